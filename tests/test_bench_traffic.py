"""Recorded DRAM traffic counts for the source it was captured on, the headers beside it included (no GPU)."""

import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)


def test_recorded_traffic_needs_the_captured_headers(tmp_path, monkeypatch):
    import bench
    src = tmp_path / "kernel.cu"
    src.write_text('// kernel\n#include "a.cuh"\n#include <cuda.h>\n#include "../out.h"\n')
    (tmp_path / "a.cuh").write_text('#pragma once\n  # include "b.cuh"\n#include "a.cuh"\n#include "absent.cuh"\n')
    (tmp_path / "b.cuh").write_text("// deepest\n")
    (tmp_path / "profiles").mkdir()
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))

    def record():
        rec = {"w": {"source": "kernel.cu", "source_sha": bench.source_hash(str(src)), "dram_bytes_per_launch": 1000}}
        (tmp_path / "profiles" / "traffic.json").write_text(json.dumps(rec))

    for name in ("kernel.cu", "a.cuh", "b.cuh"):
        record()
        assert bench.recorded_traffic("w") == 1000
        path = tmp_path / name
        path.write_text(path.read_text() + "// changed\n")
        assert bench.recorded_traffic("w") is None, name
