"""A kernel that may begin before the end of the kernel ahead reads what others wrote only
behind its own wait for that kernel: nothing else makes those stores visible to it."""
import re

import numpy as np
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib
from tests.test_launch_order import kernels

READS = r"__ld\w+\(|\bseq_begin\(|\bfirst_seq\(|\bbulk_load\(|\btma_load\w*\(|\bp\.\w+\[|\*p\.\w+"


def test_nothing_is_read_ahead_of_the_wait():
    """(few_experts_kernel alone works beside the kernel ahead, through signals.)"""
    seen = set()
    for _, name, body in kernels():
        at = re.search(r"griddepcontrol\.wait|wait_for_kernels_ahead\(", body)
        if at and name != "few_experts_kernel":
            seen.add(name)
            assert not re.findall(READS, body[:at.start()]), name
    assert {"balance_part_kernel", "balance_seq_kernel", "rmsnorm_kernel", "mx4_gemm_kernel"} <= seen


@pytest.mark.gpu
@pytest.mark.parametrize("T,E", [(4097, 97), (3000, 384)])
def test_offsets_that_change_ahead_of_every_call(T, E):
    """The sequences' offsets rewritten in their place ahead of each of many calls in a row:
    each call as it is alone."""
    from tests import test_gpu_balance as B
    from tests.test_gpu_fp8 import ok
    rng = np.random.default_rng(E)
    k, n = 4, 37
    z, ids = B.inputs(rng, T, E, k)
    cuts = [np.sort(np.concatenate([[0, T], rng.integers(0, T + 1, n - 1)])).astype(np.int32)
            for _ in range(3)]
    a = B.call(z, ids, B.SIG, cuts[0])
    outs = ("counts", "tokens", "load", "seq_loss", "loss", "dlogits")
    cuts = [B.dev(c) for c in cuts]
    alone = []
    for c in cuts:
        b = dict(a, seq_offsets=c, **{x: torch.empty_like(a[x]) for x in outs})
        torch.cuda.synchronize()
        _lib.moe_balance_loss(b)
        _lib.moe_balance_loss_backward(b)
        torch.cuda.synchronize()
        alone.append(b)
    assert not torch.equal(alone[0]["counts"], alone[1]["counts"])
    calls = [dict(a, **{x: torch.full_like(a[x], -7) for x in outs}) for _ in range(40)]
    torch.cuda.synchronize()
    for i, b in enumerate(calls):
        a["seq_offsets"].copy_(cuts[i * 7 // 3 % 3])
        _lib.moe_balance_loss(b)
        _lib.moe_balance_loss_backward(b)
    ok()
    for i, b in enumerate(calls):
        for x in outs:
            assert torch.equal(b[x], alone[i * 7 // 3 % 3][x]), (i, x)
