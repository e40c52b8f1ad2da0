"""Group offsets on the device that do not fit the call (the host cannot see them): the
kernels stay inside max_rows, and MOE_ERR_INVALID_ARG is recorded.  Rows of groups that
do fit are computed as ever."""
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib
from tests.test_gpu_few import n64

pytestmark = pytest.mark.gpu

GUARD = 300      # rows behind the arrays, inside the same allocation


def rows_in(t, rows):
    return t[:rows], t[rows:]


def dev(offsets):
    return torch.tensor(offsets, dtype=torch.int32, device="cuda")


def codes(*s, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(40, 60, s, generator=g, dtype=torch.uint8, device="cuda")


def matmul(R, G, offsets, N=256, K=256):
    a, b = codes(R + GUARD, K), codes(G, N, K, seed=1)
    out = torch.full((R + GUARD, N), 3.0, dtype=torch.bfloat16, device="cuda")
    s = torch.ones(R + GUARD, 2, device="cuda")
    _lib.moe_fp8_matmul(a, s, dev(offsets), G, R, b, torch.ones(G, N // 128, 2, device="cuda"), None,
                        0, N, K, out)
    torch.cuda.synchronize()
    return out, _lib.moe_last_device_status()


@pytest.mark.parametrize("R,G,good,bad", [
    (200, 3, [0, 64, 128, 200], [0, 64, 128, 437]),          # the last one past the rows
    (200, 3, [0, 64, 200, 200], [0, 64, 450, 470]),
    (7, 1, [0, 7], [0, 120]), (200, 1, [0, 200], [0, 500]),
    (200, 3, [0, 0, 128, 200], [-90, 0, 128, 200]), (7, 1, [0, 7], [-3, 7]),
    (1000, 2, [0, 500, 1000], [0, 500, 1290])])
def test_matmul(R, G, good, bad):
    want, status = matmul(R, G, good)
    assert status == _lib.MOE_OK and (want[R:] == 3.0).all()
    got, status = matmul(R, G, bad)
    assert status == _lib.MOE_ERR_INVALID_ARG
    assert (got[R:] == 3.0).all()
    assert torch.equal(got[:R], want[:R])
    assert matmul(R, G, good)[1] == _lib.MOE_OK


def test_ffn():
    R, G, d, I = 150, 2, 256, 128
    x, w13, w2 = codes(R + GUARD, d), codes(G, 2 * I, d, seed=1), codes(G, d, I, seed=2)
    one = lambda *s: torch.full(s, 0.01, device="cuda")
    out = []
    for offsets, status in (([0, 70, R], _lib.MOE_OK), ([0, 70, R + 200], _lib.MOE_ERR_INVALID_ARG)):
        hq = torch.full((R + GUARD, I), 7, dtype=torch.uint8, device="cuda")
        hs, y = torch.full((R + GUARD, 1), 5.0, device="cuda"), torch.full(
            (R + GUARD, d), 3.0, dtype=torch.bfloat16, device="cuda")
        _lib.moe_expert_ffn_fp8(x, one(R + GUARD, 2), dev(offsets), G, R, w13, one(G, 2, 2), w2,
                                one(G, 2, 1), None, 0, d, I, 7.0, hq, hs, y)
        torch.cuda.synchronize()
        assert _lib.moe_last_device_status() == status
        assert (hq[R:] == 7).all() and (hs[R:] == 5.0).all() and (y[R:] == 3.0).all()
        out.append(y[:R])
    assert torch.equal(*out)


@pytest.mark.parametrize("offsets", [[0, 100, 260, 450], [0, 300, 300, 900], [0, 260, 0, 260], [-40, 100, 200, 260]])
def test_weight_gradient(offsets):
    R, G, M, N = 260, 3, 128, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    a, b = (torch.randn(R + GUARD, c, generator=g, device="cuda").to(torch.bfloat16) for c in (M, N))
    size = _lib.moe_fp8_wgrad_workspace_size(G, R, M, N)
    ws = torch.full((size + 65536,), 9, dtype=torch.uint8, device="cuda")
    dW = torch.zeros(G, M, N, device="cuda")

    def run(offs):
        _lib.moe_fp8_wgrad(a, b, dev(offs), G, R, M, N, dW, ws[:size])
        torch.cuda.synchronize()
        return dW.clone(), _lib.moe_last_device_status()
    got, status = run(offsets)
    assert status == _lib.MOE_ERR_INVALID_ARG
    assert (ws[size:] == 9).all()
    # a first group that fits is as it is alone
    if offsets[0] == 0 and offsets[1] <= R:
        want, status = run([0, offsets[1], R, R])
        assert status == _lib.MOE_OK
        assert torch.equal(got[0], want[0])
        assert n64(got[0]).any()
