"""Offsets of sequences that descend: recorded, and every output zero, whatever the workspace
held; those of a token count that fits one CTA and of one that does not alike."""
import numpy as np
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib
from tests import test_gpu_balance as B
from tests.test_gpu_fp8 import ok

pytestmark = pytest.mark.gpu

OUT = ("counts", "tokens", "load", "seq_loss", "loss", "dlogits")


@pytest.mark.parametrize("T,offs", [(50, [0, 30, 20, 50]), (150, [0, 100, 20, 150]), (150, [0, 100, 20, 30, 40, 150]),
                                    (5000, [5000, 0]), (5000, [0, 4999, 4998, 5000, 5000, 5000]), (3, [1, 0]),
                                    (700, [-5, 650, 600, 800])])
@pytest.mark.parametrize("E,score", [(16, B.SIG), (384, B.SOFT), (97, B.SIG)])
def test_descending_offsets(T, offs, E, score):
    rng = np.random.default_rng(T + E)
    z, ids = B.inputs(rng, T, E, 2)
    offs = np.array(offs, np.int32)
    for fill in (0, 77, 255):
        b = B.call(z, ids, score, offs, ws_fill=fill)
        torch.cuda.synchronize()
        assert _lib.moe_last_device_status() == _lib.MOE_ERR_INVALID_ARG
        for n in OUT:
            assert not b[n].any(), n
    # the same workspace with offsets in order
    good = np.sort(np.clip(offs, 0, T)).astype(np.int32)
    b["seq_offsets"] = B.dev(good)
    _lib.moe_balance_loss(b)
    _lib.moe_balance_loss_backward(b)
    ok()
    B.check(b, B.reference(z.astype(np.float64), ids, score, good), z)


@pytest.mark.parametrize("T", [50, 500])
def test_offsets_outside_the_tokens_are_cut(T):
    rng = np.random.default_rng(T)
    z, ids = B.inputs(rng, T, 24, 2)
    offs = np.array([-7, 10, T - 3, T + 60, T + 50], np.int32)
    a = B.call(z, ids, B.SIG, offs)
    torch.cuda.synchronize()
    assert _lib.moe_last_device_status() == _lib.MOE_ERR_INVALID_ARG
    assert a["tokens"].tolist() == [10, T - 13, 3, 0]
    B.check(a, B.reference(z.astype(np.float64), ids, B.SIG, np.clip(offs, 0, T)), z)
