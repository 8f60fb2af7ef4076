"""What the compiler makes of device code whose results do not show it: a small
kernel around the code in question, compiled for gfx950, and its instructions
counted."""
import os
import re
import subprocess

import pytest

from moe_layer_amd import build as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.HIPCC), reason="hipcc not found")


def assembly(tmp_path, src):
    out = tmp_path / "probe.s"
    cmd = [B.HIPCC, *B.COMMON_FLAGS, "-I", B.CSRC, "-I", os.path.join(B.PKG, "..", "include"), "--offload-device-only",
           "-S", str(src), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return out.read_text().splitlines()


def instructions(tmp_path, body):
    """The gfx950 instructions of ``body``, HIP source behind the products' device code."""
    src = tmp_path / "probe.hip"
    src.write_text('#include "dev_rows.h"\nusing namespace moe;\n' + body)
    return [line.strip() for line in assembly(tmp_path, src) if re.match(r"\s+[a-z]+_\w+\s", line)]


def test_outputs_are_stored_past_the_caches_or_not(tmp_path):
    """store_tile has both kinds of store: of two stores that differ in that alone and
    stand in two branches the compiler makes one, a plain one."""
    code = instructions(tmp_path, """
__global__ void probe(RowsGemmArgs g, int row0, int row1, int n0) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[16 * kOutRow<128>];
    lds[threadIdx.x] = uint8_t(row0);
    __syncthreads();
    store_tile<128, 16, 64, true>(g, (lds_t*)lds, row0, row1, n0);
}
""")
    stores = [i for i in code if i.startswith("global_store_dwordx4")]
    assert any(re.search(r"\bnt\b", i) for i in stores), stores
    assert any(not re.search(r"\bnt\b", i) for i in stores), stores


def test_a_block_among_many_groups_is_found_in_one_pass(tmp_path):
    """The products of few rows read the offsets of more groups than a wave holds once:
    in one loop over pairs of neighbours, with none in front that counts all blocks."""
    pairs, kernel = {}, None
    for line in assembly(tmp_path, os.path.join(B.CSRC, "gemm_split.hip")):
        name = re.match(r"(_ZN\S*rows_split_kernel\S*):", line)
        if name or line.startswith(".Lfunc_end"):
            kernel = name.group(1) if name else None
            if name:
                pairs[kernel] = 0
        elif kernel and re.match(r"\s+global_load_dwordx2\s", line):
            pairs[kernel] += 1
    assert pairs and set(pairs.values()) == {1}, pairs
