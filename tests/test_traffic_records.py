"""The committed DRAM records (profiles/traffic.json) belong to the kernels in the tree, and what the
bench prints of them depends on every source that a kernel is compiled from."""
import json
import os
import shutil

import pytest

import bench

with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
    RECORDS = json.load(f)


@pytest.mark.parametrize("name", sorted(RECORDS))
def test_record_is_of_the_current_source(name):
    """A record of an older kernel is retaken (its `capture` line) or taken out."""
    rec = RECORDS[name]
    assert rec["source_sha256_16"] == bench.source_hash(rec["source"])
    assert rec["dram_bytes_per_launch"] == rec["dram_bytes_read"] + rec["dram_bytes_write"]
    assert bench._traffic(name, 0) == rec["dram_bytes_per_launch"]


@pytest.mark.parametrize("source,header", [("decode_kernel.cu", "decode_tile.cuh"), ("append_kernel.cu", "append_row.cuh"),
                                           ("prefill_tc.cu", "kvq_ptx.cuh"), ("decode_kernel.cu", "decode_kernel.cu")])
def test_hash_covers_what_a_kernel_is_made_of(tmp_path, source, header):
    csrc = str(tmp_path / "package" / "csrc")
    shutil.copytree(bench.CSRC, csrc)
    shutil.copytree(os.path.join(bench.ROOT, "include"), str(tmp_path / "include"))
    before = bench.source_hash(source, csrc)
    assert before == bench.source_hash(source)
    path = os.path.join(csrc, header)
    with open(path) as f:
        text = f.read()
    with open(path, "w") as f:
        f.write("// a comment\n" + text)
    assert bench.source_hash(source, csrc) == before
    with open(path, "w") as f:
        f.write(text + "\nconstexpr int kOneMore = 1;\n")
    assert bench.source_hash(source, csrc) != before
