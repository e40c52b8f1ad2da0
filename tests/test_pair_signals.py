"""What tells one CTA of a pair that the other's shared memory is written: an arrival released at
cluster scope, or the completion of a copy that was issued behind the writes."""
import glob
import os
import re

import pytest
import torch

from moe_expert_layer_04_gb300 import _lib
from tests.test_launch_order import CSRC, kernels


def test_arrivals_in_another_cta_name_their_scope():
    """(Without one it is the CTA's own, which orders nothing for a thread of another.)"""
    found = 0
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        for m in re.finditer(r"mbarrier\.arrive([\w.]*)\.shared::cluster", open(path).read()):
            found += 1
            assert re.search(r"\.(release|relaxed)\.cluster", m.group(1)), (path, m.group(0))
    assert found >= 2


def test_scales_of_a_pair_are_there_before_their_codes_are_asked_for():
    body = next(b for _, n, b in kernels() if n == "mx4_gemm_kernel")
    producer = body[body.index("if (warp == 0) {", body.index("let_kernels_behind_begin(")):body.index("else if (warp == 1)")]
    wait, copy = producer.index("&sfready[j]"), producer.index("tma_load_2d")
    assert wait < copy and "rank == 1" in producer[:wait]
    scales = body[body.index("warp < kEpi0"):]
    assert re.search(r"fence_proxy_async_smem\(\);\s*__syncwarp\(\);\s*if \(lane == 0\) mbar_arrive\(&sfready\[j\]\);",
                     scales)


@pytest.mark.gpu
@pytest.mark.parametrize("cuts,R,N,K", [([], 512, 512, 2048), ([], 1024, 640, 544), ([900], 2600, 768, 8192),
                                        ([300, 301, 900], 1500, 256, 1024), ([], 2048, 2048, 544),
                                        ([900], 2600, 1032, 4096), ([300, 301, 900], 2048, 4096, 1024)])
@pytest.mark.parametrize("bits", [4, 8])
def test_scales_alone_differ(cuts, R, N, K, bits):
    """Pairs of CTAs: calls in a row whose codes are the same and whose scales are not."""
    from tests.test_gpu_fp8 import ok
    if bits == 8:
        K = (K + 127) // 128 * 128
    G, p = len(cuts) + 1, _lib.moe_mx_sf_pitch(K)
    g = torch.Generator(device="cuda").manual_seed(R + K)
    u8 = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, dtype=torch.uint8, device="cuda")
    offs = torch.tensor([0] + cuts + [R], dtype=torch.int32, device="cuda")
    a, b = u8(0, 120 if bits == 8 else 256, R, K if bits == 8 else K // 2), u8(0, 256, G, N, K // 2)
    scales = [(u8(117, 132, R, p), u8(117, 132, G, N, p)) for _ in range(3)]
    out = torch.empty(R, N, dtype=torch.bfloat16, device="cuda")

    def run(s):
        _lib.moe_mx4_matmul(a, s[0], bits, offs, G, R, b, s[1], None, 0, N, K, out)
        return out.view(torch.int16)
    alone = []
    for s in scales:
        torch.cuda.synchronize()
        alone.append(run(s).clone())
    assert not torch.equal(alone[0], alone[1])
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(600):
        wrong += (run(scales[i % 3]) != alone[i % 3]).sum()
    ok()
    assert int(wrong) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("counts,N,K", [([700, 1, 0, 900, 300], 1032, 288), ([1, 3333], 1032, 64),
                                        ([255, 257, 1, 2000, 0, 300], 1032, 1120), ([2500, 1, 129], 4104, 96)])
@pytest.mark.parametrize("bits", [4, 8])
def test_pairs_where_groups_end(counts, N, K, bits):
    """Groups that end in a pair's first row tile, with one row, or in its second."""
    from tests.test_gpu_mx4 import test_matmul as check
    check(counts, N, K if bits == 4 else (K + 127) // 128 * 128, bits, False)
