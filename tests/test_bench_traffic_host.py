"""The stored DRAM traffic of the GEMM applies to the code that it was measured on: gemm.cu and the device headers that
it includes."""
import os
import shutil

import bench


def test_a_change_in_a_header_invalidates_the_figure(tmp_path):
    sources = bench.gemm_sources()
    assert [os.path.basename(p) for p in sources] == ["gemm.cu", "tcgen05.cuh"]
    for p in sources:
        shutil.copy(p, tmp_path)
    copy = bench.gemm_sources(str(tmp_path / "gemm.cu"))
    before = bench.code_sha16(*sources)
    assert bench.code_sha16(*copy) == before
    header = tmp_path / "tcgen05.cuh"
    text = header.read_text()
    header.write_text("// a comment\n" + text)
    assert bench.code_sha16(*copy) == before
    changed = text.replace("kSuspendNs = 20000", "kSuspendNs = 1000")
    assert changed != text
    header.write_text(changed)
    assert bench.code_sha16(*copy) != before

