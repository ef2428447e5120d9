"""CPU-only: the stored traffic counters stand for the sources they were taken with,
a kernel's headers among them."""

import shutil

import bench


def test_digest_covers_the_headers_a_kernel_includes(tmp_path, monkeypatch):
    csrc = tmp_path / "csrc"
    shutil.copytree(bench.CSRC, csrc)
    monkeypatch.setattr(bench, "CSRC", str(csrc))
    kinds = sorted(bench.KERNEL_SOURCE)
    before = {k: bench.source_sha(k) for k in kinds}

    def changed(header):
        with open(csrc / header, "a") as f:
            f.write("// changed\n")
        now = {k: bench.source_sha(k) for k in kinds}
        out = {k for k in kinds if now[k] != before[k]}
        before.update(now)
        return out

    lowrank = {"lowrank", "gemm_db", "gemm_da"}
    assert changed("qn_mx.h") == lowrank                                  # included directly
    assert changed("qn_philox.h") == lowrank | {"gemm_fwd", "gemm_dx"}
    assert changed("qn_device.h") == set(kinds)
    assert changed("qn_colsum.h") == set()                                # of other kernels
    assert changed("k_codec.hip") == {"quantize", "double_quant", "dequant"}


def test_stale_counters_are_not_reported(monkeypatch):
    monkeypatch.setitem(bench.TRAFFIC, "x", {"bytes": 7, "sha256": bench.source_sha("gemv")})
    assert bench.traffic("x", "gemv") == 7
    monkeypatch.setitem(bench.TRAFFIC, "x", {"bytes": 7, "sha256": "0"})
    assert bench.traffic("x", "gemv") is None and bench.traffic("no such key", "gemv") is None
