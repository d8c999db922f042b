"""Host-side helpers of bench.py (no GPU): the kernel-source digest that ties a
committed rocprofv3 traffic record to the code it was measured on."""
from __future__ import annotations

import bench


def _digest_of(tmp_path, monkeypatch, text: str) -> str:
    f = tmp_path / "k.hip"
    f.write_text(text)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    monkeypatch.setitem(bench.KERNEL_SOURCES, "sgemm", ["k.hip"])
    return bench.source_digest("sgemm")


def test_digest_ignores_comments_and_layout(tmp_path, monkeypatch):
    base = _digest_of(tmp_path, monkeypatch, "int f(int x) { return x + 1; }\n")
    commented = _digest_of(tmp_path, monkeypatch,
                           "// a note\nint f(int x)  /* inline */ {\n    return x + 1;   // why\n}\n")
    assert base == commented


def test_digest_changes_with_code(tmp_path, monkeypatch):
    a = _digest_of(tmp_path, monkeypatch, "int f(int x) { return x + 1; }\n")
    b = _digest_of(tmp_path, monkeypatch, "int f(int x) { return x + 2; }\n")
    assert a != b


def test_digest_covers_included_headers():
    for kind, files in bench.KERNEL_SOURCES.items():
        assert any(f.endswith("epilogue.h") for f in files), kind
        assert any(f.endswith(f"{kind}_mfma.hip") for f in files), kind


def test_digest_covers_every_header_the_kernels_include():
    import os
    import re

    for kind, files in bench.KERNEL_SOURCES.items():
        for f in files:
            for h in re.findall(r'#include "(\w+\.h)"', open(os.path.join(bench.ROOT, f)).read()):
                if h != "plan16.h":   # (host code: which kernel runs, not what it does)
                    assert os.path.join(os.path.dirname(f), h) in files, (kind, f, h)


def test_traffic_records_belong_to_the_present_kernels():
    recs = bench._traffic_records()
    for key, r in recs.items():
        if key != "copy_calibration":
            kind = "sgemm" if "sgemm" in r["kernel"] else "hgemm"
            assert r["source_sha"] == bench.source_digest(kind), key
    for kind in ("sgemm", "hgemm"):
        assert bench.measured_traffic(kind, kind, bench.STEP_WORKLOADS[kind])


def test_kernel_names_without_the_library_s_namespaces():
    for ns in ("mi355gemm::", "mi355gemm::(anonymous namespace)::"):
        name = f"void mi355gemm::(anonymous namespace)::hgemm_dma_kernel<{ns}HgDmaCfg<256, 256, 2>, false>(mi355gemm::(anonymous namespace)::HgemmArgs)"
        assert bench._short(name) == "void hgemm_dma_kernel<HgDmaCfg<256, 256, 2>, false>"


def test_resource_summary_knows_every_profiled_kernel():
    import os

    text = open(os.path.join(bench.ROOT, "profiles", "resources.md")).read()
    assert "not found in the sources" not in text and "hgemm_dma_kernel" in text
