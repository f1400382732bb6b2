"""The calls of integer-coded caches and packed prompts from several host threads: the library runs without
the interpreter's lock (a stand-in answers whether it is held; nothing is launched), and threads with
streams and workspaces of their own get each the result of its call alone."""
import os
import subprocess
import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CALLS = ["kv_write_int", "kv_read_int", "attention_int", "attention_packed"]

PROGRAM = """
import torch
import paged_kv_cache_161_gb300 as pa

z = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype, device="cuda")
i = lambda *shape: z(*shape, dtype=torch.int32)
u = lambda *shape: z(*shape, dtype=torch.uint8)
q, kv, cache = z(3, 2, 64), z(3, 1, 64), u(4, 1, 16 * 36)
calls = dict(
    kv_write_int=lambda: pa.kv_write_int(kv, kv, cache, cache.clone(), z(3, dtype=torch.int64), bits=4),
    kv_read_int=lambda: pa.kv_read_int(z(3, 1, 64), z(3, 1, 64), cache, cache, i(2, 2), None, i(2), i(3), bits=4),
    attention_int=lambda: pa.attention_int(z(3, 2, 64), q, cache, cache, i(2, 2), i(2), i(3), bits=4, max_query_len=1,
                                           max_seq_len=9, scale=1.0, workspace=u(1 << 20)),
    attention_packed=lambda: pa.attention_packed(z(3, 2, 64), q, kv, kv, i(3), i(3), max_query_len=1, scale=1.0))
for name, call in calls.items():
    try:
        call()
        print(name, "unlocked")
    except pa.PAError as e:
        print(name, "locked" if e.status == 4 else e)
"""


def test_the_lock_is_released_in_the_library(tmp_path):
    src, lib = tmp_path / "stand_in.cpp", tmp_path / "stand_in.so"
    src.write_text('extern "C" {\nint PyGILState_Check(void);\n' +
                   "".join(f"int pa_{n}(void) {{ return PyGILState_Check() ? 4 : 0; }}\n" for n in CALLS) + "}\n")
    subprocess.run([os.environ.get("CXX", "g++"), "-shared", "-fPIC", "-o", str(lib), str(src)], check=True)
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300,
                       env={**os.environ, "LD_PRELOAD": str(lib)})
    assert r.returncode == 0, r.stderr
    assert r.stdout.split("\n")[:-1] == [f"{n} unlocked" for n in CALLS]


def test_threads_with_streams_of_their_own():
    import paged_kv_cache_161_gb300 as pa

    S, L, H, D, B = 6, 700, 2, 128, 16
    W = (L + B - 1) // B
    g = torch.Generator(device="cuda").manual_seed(0)
    rows = torch.randn((S * L, H, D), generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn((S * L, 8, D), generator=g, device="cuda").to(torch.bfloat16)
    table = torch.randperm(S * W, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(S, W).cuda()
    pos = torch.arange(L, device="cuda")
    slots = (table[:, pos // B].long() * B + pos % B).flatten()
    lens = torch.full((S,), L, dtype=torch.int32, device="cuda")
    loc = torch.arange(0, S * L + 1, L, dtype=torch.int32, device="cuda")
    one = torch.arange(S + 1, dtype=torch.int32, device="cuda")

    def run():
        kc, vc = (torch.zeros((S * W, H, B * (D // 2 + 4)), dtype=torch.uint8, device="cuda") for _ in range(2))
        k, v = torch.empty_like(rows), torch.empty_like(rows)
        packed, out = torch.empty_like(q), torch.empty_like(q[:S])
        ws = torch.empty(pa.attention_int_workspace_size(S, S, 8, H, D), dtype=torch.uint8, device="cuda")
        pa.kv_write_int(rows, -rows, kc, vc, slots, bits=4)
        pa.kv_read_int(k, v, kc, vc, table, None, lens, loc, bits=4)
        pa.attention_packed(packed, q, k, v, loc, loc, max_query_len=L, scale=D ** -0.5)
        pa.attention_int(out, q[:S], kc, vc, table, lens, one, bits=4, max_query_len=1, max_seq_len=L, scale=D ** -0.5,
                         workspace=ws)
        return kc, vc, k, v, packed, out

    want = run()
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def thread(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got[i] = run()
                torch.cuda.current_stream().synchronize()
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and pa.read_device_errors() == 0
    for result in got:
        assert all(torch.equal(a, b) for a, b in zip(result, want))
