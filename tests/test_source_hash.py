"""The hash that ties the committed per-launch DRAM bytes to the sources of the kernels they were measured on."""
import shutil

from sparse_attention_indexer_lt_gb300 import build


def test_the_hash_goes_by_the_measured_kernels_sources(tmp_path, monkeypatch):
    shutil.copytree(build.CSRC, tmp_path / "sources")
    shutil.copytree(build.INCLUDE, tmp_path / "include")
    want = build.source_hash()
    monkeypatch.setattr(build, "CSRC", tmp_path / "sources")
    monkeypatch.setattr(build, "INCLUDE", tmp_path / "include")
    assert build.source_hash() == want
    for path in ("sources/lt_kv4_cache.cu", "sources/lt_kv4_attention.cuh", "sources/lt_pages.cu", "include/lt_kv4.h"):
        with open(tmp_path / path, "a") as f:
            f.write("// another line\n")
        assert build.source_hash() == want, f"{path} is no part of the measured kernels"
    for path in ("sources/lt_kernels.cuh", "sources/lt_async.cuh", "sources/lt_compress.cu", "sources/lt_api.cu", "include/lt_topk.h"):
        before = build.source_hash()
        with open(tmp_path / path, "a") as f:
            f.write("// another line\n")
        assert build.source_hash() != before, path
