"""How far attention over integer-coded caches may be off, from its arithmetic.

Query rows enter as f16 scaled by a power of two: exact but for elements 2^-24 of the row's largest. A
logit is, in fp32, step (q.(o + c) - q.o) + lo sum q with o = 0 or 64 (4 bits), or 1024 (8 bits), sums
of D terms: each term and each sum within 2^-23 of sum |q| (off step + |lo|), off = 80 or 1280 (what
multiplies step at most), so dl <= scale (D + 8) 2^-23 sum |q| (off step + |lo|). The numerators have that
relative error, ex2's 2^-22 and, times the value's step, f16's half step 2^-11 (what falls under f16's
range: 2^-31 of the largest step a key). A value enters as mid + step (c - mid), both parts within
mag = sum_j w_j (|mid_j| + step_j N / 2). fp32 sums over the keys: 2^-23 each, 2^-18 for thousands. One
rounding of the output to bf16: 2^-8.
"""
import numpy as np

from oracle import int_cache as ic


def attention(q, kc, vc, table, L, scale, bits):
    """(reference, tolerance) of the rows q [Q, Hq, D] at the end of a request of L keys."""
    Q, Hq, D = q.shape
    N, off = 2 ** bits - 1, 80 if bits == 4 else 1280
    K, klo, kstep = ic.rows(kc, table, L, D, bits)
    V, vlo, vstep = ic.rows(vc, table, L, D, bits)
    ref = ic.attend(q, K, V, L - Q, scale)[0]
    big = np.abs(vlo + (N + 1) / 2 * vstep) + vstep * (N + 1) / 2
    mag = ic.attend(q, K, np.broadcast_to(big[..., None], V.shape), L - Q, scale)[0]
    par = np.repeat((off * kstep + np.abs(klo)).max(0), Hq // K.shape[1])
    dl = scale * (D + 8) * 2.0 ** -23 * np.abs(q).sum(-1) * par
    tol = mag * (2.0 ** -11 + 2 * dl[..., None] + 2.0 ** -18) + L * 2.0 ** -31 * vstep.max() * N
    return ref, tol + 2.0 ** -8 * (np.abs(ref) + tol)
