"""Which sources a stored counter profile of the benchmark is valid for."""

from __future__ import annotations

from tests.test_bench_host import _bench


def test_other_operators_sources_do_not_void_the_layers_counters(tmp_path, monkeypatch):
    b = _bench()
    csrc = tmp_path / "mixture_experts_ffn_renorm_amd" / "csrc"
    csrc.mkdir(parents=True)
    monkeypatch.setattr(b, "ROOT", str(tmp_path))
    (csrc / "gemm_stream.hip").write_text("layer")
    first = b.kernel_source_hash()
    for name in ("qlinear.hip", "select.hip"):
        (csrc / name).write_text("operator")
        assert b.kernel_source_hash() == first
    (csrc / "gemm_stream.hip").write_text("another layer")
    second = b.kernel_source_hash()
    (csrc / "route.hip").write_text("router")
    assert len({first, second, b.kernel_source_hash()}) == 3
