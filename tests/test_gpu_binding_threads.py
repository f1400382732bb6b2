"""The serving-step calls let other Python threads run while they are in the library, as the ctypes
calls do: a launch may wait for room in a full queue, which a Python function queued on the stream
may have to make. A stand-in for the library, loaded before it, answers each call with whether the
interpreter's lock is held; nothing is launched."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CALLS = ["advance_batch", "norm_rope_write", "block_bounds", "block_scores", "select_blocks", "attention_sparse"]

PROGRAM = """
import torch
import paged_kv_cache_161_gb300 as pa

z = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype, device="cuda")
i = lambda *shape: z(*shape, dtype=torch.int32)
slots, kc = z(3, dtype=torch.int64), z(4, 16, 1, 64)
meta = (i(2, 2), i(2), i(3))
calls = dict(
    advance_batch=lambda: pa.advance_batch(*meta[:2], i(2), i(4), i(1), i(2), i(1), meta[2], slots, i(3), block_size=16,
                                           num_blocks=4),
    norm_rope_write=lambda: pa.norm_rope_write(z(3, 2, 64), z(3, 2, 64), z(3, 1, 64), z(3, 1, 64), None, None,
                                               z(9, 64, dtype=torch.float32), i(3), slots, kc, kc.clone()),
    block_bounds=lambda: pa.block_bounds(z(4, 1, 2, 64), kc, *meta, max_query_len=1, max_seq_len=9),
    block_scores=lambda: pa.block_scores(z(3, 1, 2, dtype=torch.float32), z(3, 2, 64), z(4, 1, 2, 64), *meta, block_size=16,
                                         max_query_len=1, max_seq_len=9),
    select_blocks=lambda: pa.select_blocks(i(3, 1, 1), z(3, 1, 2, dtype=torch.float32), *meta[1:], block_size=16),
    attention_sparse=lambda: pa.attention_sparse(z(3, 2, 64), z(3, 2, 64), kc, kc, *meta, i(3, 1, 1), max_seq_len=9, scale=1.0))
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
