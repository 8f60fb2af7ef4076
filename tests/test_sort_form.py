"""Which form moe_sort_rows takes below the slots that are counted in launches of
their own, by the host's rule (sorted.h), at sizes where one of the two is the
faster by 15 % or more: us of each as measured on an MI355X, 256 experts."""
import os
import subprocess

import pytest

from moe_layer_amd import build as B

# T, topk, parts, batch_parts, units, compares: us comparing, us batch
CASES = [
    (1, 8, 4, 1, 896, True),          # 3.4, 4.9
    (100, 8, 4, 1, 896, True),        # 5.9, 10.1
    (256, 8, 4, 1, 896, True),        # 9.7, 11.3
    (256, 1, 8, 2, 2048, True),       # 5.5, 7.0
    (512, 1, 2, 1, 512, True),        # 4.5, 5.9
    (128, 16, 4, 1, 896, True),       # 10.9, 14.4
    (32, 64, 4, 1, 896, True),        # 23.7, 35.1
    (32, 64, 8, 2, 2048, True),       # 25.9, 40.2
    (64, 32, 8, 2, 2048, True),       # 19.6, 24.2
    (32, 64, 1, 1, 2048, True),       # to int8, 34.8, 76.9
    (0, 8, 4, 1, 896, True),          # the batch form has no workgroup for no token
    (700, 8, 1, 1, 256, False),       # 12.0, 9.3
    (512, 8, 4, 1, 896, False),       # 17.3, 14.5
    (256, 16, 4, 1, 896, False),      # 19.0, 15.8
    (200, 64, 1, 1, 256, False),      # 67.0, 19.5
    (256, 64, 1, 1, 256, False),      # 80.8, 20.2, to int8 81.6, 21.9
    (256, 64, 4, 1, 896, False),      # 153, 41.9
    (100, 64, 8, 2, 2048, False),     # 85.2, 45.2
    (64, 64, 1, 1, 256, False),       # 30.5, 16.3
    (128, 32, 1, 1, 256, False),      # 17.7, 11.3
    (256, 16, 1, 1, 256, False),      # 11.2, 9.1
    (49152, 1, 512, 128, 131072, False),
]


@pytest.mark.skipif(not os.path.exists(B.HIPCC), reason="hipcc not found")
def test_the_faster_form_is_taken(tmp_path):
    src = tmp_path / "form.hip"
    src.write_text('#include "moe.h"\n#include "sorted.h"\n' + "".join(
        f"static_assert({'' if few else '!'}moe::few_ids({t}, {k}, {p}, {b}, {u}));\n" for t, k, p, b, u, few in CASES))
    r = subprocess.run([B.HIPCC, *B.COMMON_FLAGS, "-I", B.CSRC, "-I", os.path.join(B.PKG, "..", "include"),
                        "--offload-host-only", "-fsyntax-only", str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
