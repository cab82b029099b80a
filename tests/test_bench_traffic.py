"""The source hash that keys the bench's measured DRAM traffic covers the decode
and nothing else: a change of the decode drops the figures, another operator's
does not."""
import os
import shutil

import bench

CSRC = os.path.join("retrieval_sparse_attention_wave_b200", "csrc")


def test_hash_covers_the_decode_alone():
    names = {os.path.basename(f) for f in bench.decode_sources()}
    assert {"wi_decode.cu", "wi_decode_kernels.cuh", "wi_decode_bf16_d128.cu", "wi_common.cuh", "wi_plan.h",
            "wi_api.cu"} <= names
    assert not any(n.startswith(("wi_attend", "wi_serve", "wi_build", "wi_umma")) for n in names)


def test_hash_changes_with_the_decode_and_not_with_others(tmp_path, monkeypatch):
    shutil.copytree(os.path.join(bench.ROOT, CSRC), tmp_path / CSRC)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    first = bench.kernel_source_sha256()

    def after(name, text):
        with open(tmp_path / CSRC / name, "a") as f:
            f.write(text)
        return bench.kernel_source_sha256()
    assert after("wi_attend.cu", "int x;\n") == after("wi_serve.h", "int x;\n") == first
    assert after("wi_decode_kernels.cuh", "// a comment\n\n") == first
    second = after("wi_common.cuh", "int x;\n")
    assert second != first and after("wi_decode.cu", "int y;\n") not in (first, second)
