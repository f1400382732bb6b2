"""Without the extension the calls of integer-coded caches and packed prompts say that it is missing; block copies and
swaps of such caches, which are ctypes calls, do not need it."""
import os
import shutil
import subprocess
import sys

PKG = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_161_gb300")

PROGRAM = """
import torch
import paged_kv_cache_161_gb300 as pa

for name in ("kv_write_int", "kv_read_int", "attention_int", "attention_packed"):
    assert name in pa.__all__
    try:
        getattr(pa, name)(1, bits=4)
    except ImportError as e:
        assert "_pa_torch.so" in str(e) and name in str(e)
    else:
        raise AssertionError(name)
cache = torch.zeros((4, 2, 16 * 68), dtype=torch.uint8)
assert pa._block_geometry(cache, cache) == ((4, 2, 1, 16 * 68), pa.PA_FP8_E4M3)
try:
    pa._block_geometry(cache, cache[:2])
except ValueError:
    print("fine")
"""


def test_the_calls_name_the_extension(tmp_path):
    to = tmp_path / "paged_kv_cache_161_gb300"
    os.makedirs(to / "_lib")
    shutil.copy(os.path.join(PKG, "__init__.py"), to)
    shutil.copy(os.path.join(PKG, "_lib", "libpa_gb300.so"), to / "_lib")
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr
