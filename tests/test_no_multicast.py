"""The kernels use no cluster multicast: bench.py also runs with several ranks, and multicast copies are left to
code that only one GPU ever runs."""
import pathlib

CSRC = pathlib.Path(__file__).resolve().parent.parent / "mla_latent_cache_attention_gb300" / "csrc"


def test_no_source_uses_cluster_multicast():
    files = [f for f in CSRC.iterdir() if f.suffix in (".cu", ".cuh", ".h", ".cpp")]
    assert len(files) > 10
    assert [f.name for f in files if "multicast" in f.read_text()] == []
