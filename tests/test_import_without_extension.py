"""The ctypes calls do not need the serving-step extension: without one that loads, the package
imports, and only the serving-step calls say that it is missing."""
import os
import shutil
import subprocess
import sys

import pytest

PKG = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_161_gb300")

PROGRAM = """
from paged_kv_cache_161_gb300 import *
import paged_kv_cache_161_gb300 as pa

assert pa.lib.pa_status_string(0)
bm = BlockManager(4, 2, range(4))
bm.add_seq(7)
assert bm.append(7, 3).tolist() == [0, 1, 2]
for name in ("advance_batch", "norm_rope_write", "block_bounds", "block_scores", "select_blocks", "attention_sparse"):
    try:
        getattr(pa, name)(1, block_size=16)
    except ImportError as e:
        assert "_pa_torch.so" in str(e) and "build.py" in str(e) and name in str(e)
    else:
        raise AssertionError(name)
print("fine")
"""


@pytest.mark.parametrize("extension", [None, b"", b"\x7fELF of another machine"], ids=["missing", "empty", "foreign"])
def test_the_other_calls_work(tmp_path, extension):
    to = tmp_path / "paged_kv_cache_161_gb300"
    os.makedirs(to / "_lib")
    shutil.copy(os.path.join(PKG, "__init__.py"), to)
    shutil.copy(os.path.join(PKG, "_lib", "libpa_gb300.so"), to / "_lib")
    if extension is not None:
        (to / "_lib" / "_pa_torch.so").write_bytes(extension)
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr
