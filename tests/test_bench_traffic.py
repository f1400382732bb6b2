"""The decode traffic that bench.py reports belongs to the sources it was measured on: it is
reported for the sources as they are, and every device file that goes into the decode kernels
counts among them."""
import os
import re

import bench

CSRC = os.path.join(bench.ROOT, "paged_kv_cache_161_gb300", "csrc")


def _device_files(name, seen):
    if name in seen:
        return
    seen.add(name)
    with open(os.path.join(CSRC, name)) as f:
        for inc in re.findall(r'#include "(\w+\.cuh)"', f.read()):
            _device_files(inc, seen)


def test_every_device_file_of_the_decode_kernels_counts():
    files = set()
    _device_files("decode_mma.cu", files)
    _device_files("decode_attention.cu", files)
    assert files == {os.path.basename(f) for f in bench.DECODE_SOURCES}


def test_the_traffic_was_measured_on_these_sources():
    assert isinstance(bench._decode_traffic(), int)


def test_a_changed_source_has_no_traffic(tmp_path, monkeypatch):
    changed = tmp_path / "mma.cuh"
    with open(os.path.join(CSRC, "mma.cuh")) as f:
        changed.write_text(f.read() + "\n")
    monkeypatch.setattr(bench, "DECODE_SOURCES", [str(changed) if f.endswith("mma.cuh") else f
                                                  for f in bench.DECODE_SOURCES])
    assert str(changed) in bench.DECODE_SOURCES and bench._decode_traffic() is None
