"""Attention over integer-coded caches with any set of visible keys, and how far the kernel may be off.

The bounds of intmodel.attention, but for the numerators' range: a row's f16 numerators times value steps
e_j step_j are scaled by a power of two under which the largest of them so far is at least 2^3, so
each is off by at most f16's half step 2^-11 of itself or by 2^-25 / 2^3 = 2^-28 of that largest one, whatever
the steps of the rows that carry no weight. Times codes of at most (N + 1) / 2 from the middle.
"""
import numpy as np

from oracle import int_cache as ic


def attention(q, kc, vc, table, L, scale, bits, gone=()):
    """(reference, tolerance) of the rows q [Q, Hq, D] at the end of a request of L keys, of which the
    positions in the logical blocks `gone` are not there; a row that sees none is zero."""
    Q, Hq, D = q.shape
    N, off = 2 ** bits - 1, 80 if bits == 4 else 1280
    B = ic.block_size_of(kc, D, bits)
    table = np.array(table)
    table[list(gone)] = 0  # any block: its rows are left out below
    K, klo, kstep = ic.rows(kc, table, L, D, bits)
    V, vlo, vstep = ic.rows(vc, table, L, D, bits)
    G = Hq // K.shape[1]
    there = ~np.isin(np.arange(L) // B, list(gone))
    big = np.abs(vlo + (N + 1) / 2 * vstep) + vstep * (N + 1) / 2
    ref, tol = np.zeros(q.shape), np.zeros(q.shape)
    for j in range(Q):
        see = np.flatnonzero(there & (np.arange(L) <= L - Q + j))
        if not len(see):
            continue
        for h in range(Hq):
            g = h // G
            x = scale * (K[see, g] @ q[j, h])
            w = np.exp(x - x.max())
            w /= w.sum()
            ref[j, h] = w @ V[see, g]
            dl = scale * (D + 8) * 2.0 ** -23 * np.abs(q[j, h]).sum() * (off * kstep[see, g] + np.abs(klo[see, g])).max()
            t = (w @ big[see, g]) * (2.0 ** -11 + 2 * dl + 2.0 ** -18) + \
                len(see) * 2.0 ** -28 * (w * vstep[see, g]).max() * (N + 1) / 2
            tol[j, h] = t + 2.0 ** -8 * (np.abs(ref[j, h]) + t)
    return ref, tol
