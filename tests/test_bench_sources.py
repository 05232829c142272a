"""The hash that ties committed counters to the GEMM's source covers its whole
translation unit: a change in any of its files makes the counters stale."""
import os
import re
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402

CSRC = os.path.join(ROOT, "float8_mixed_precision_amd", "csrc")


def _unit(name, seen):
    if name in seen:
        return seen
    seen.add(name)
    with open(os.path.join(CSRC, name)) as f:
        for inc in re.findall(r'^#include "([^"/]+)"', f.read(), re.M):
            _unit(inc, seen)
    return seen


def test_hash_covers_the_translation_unit():
    assert {os.path.basename(p) for p in bench.GEMM_SOURCES} == _unit("gemm.hip", set())


def test_hash_follows_every_source(tmp_path, monkeypatch):
    first = bench.gemm_source_hash()
    for k, path in enumerate(bench.GEMM_SOURCES):
        with open(path, "rb") as f:
            copy = tmp_path / os.path.basename(path)
            copy.write_bytes(f.read() + b"\n// changed\n")
        changed = list(bench.GEMM_SOURCES)
        changed[k] = str(copy)
        with monkeypatch.context() as m:
            m.setattr(bench, "GEMM_SOURCES", changed)
            assert bench.gemm_source_hash() != first, path
