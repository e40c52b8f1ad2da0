"""Which buffers the norm's outputs may share, on the CPU (refusals) and on the GPU (results)."""
import ctypes

import numpy as np
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib

@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")
def test_two_outputs_are_not_one():
    x, r, o = ctypes.c_void_p(256), ctypes.c_void_p(512), ctypes.c_void_p(768)
    for out, y in ((o, o), (x, x)):
        a = _lib.NormArgs(T=1, d=64, eps=1e-6, format=_lib.MOE_ROWS_NONE)
        a.x, a.residual, a.weight, a.residual_out, a.y = x, r, o, out, y
        assert _lib.load().moe_rmsnorm(ctypes.byref(a), None) == _lib.MOE_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("T,d", [(40, 512), (700, 4096), (1500, 4096), (330, 16384)])
@pytest.mark.parametrize("out,y", [("x", None), ("x", "new"), ("residual", "x"), ("new", "x"), (None, "x")])
def test_shared_buffers(T, d, out, y):
    """(A row's own kernel, and many rows through the ring.)"""
    from tests import test_gpu_norm as N
    from tests.test_gpu_fp8 import ok
    rng = np.random.default_rng(T)
    w = torch.from_numpy(rng.standard_normal(d).astype(np.float32))
    x, res = N.rows(rng, T, d), None if out is None else N.rows(rng, T, d)
    want = N.forward(x, w, res)
    a = dict(want, x=x.cuda(), residual=None if out is None else res.cuda(), residual_out=None, y=None)
    pick = lambda n: None if n is None else torch.empty_like(a["x"]) if n == "new" else a[n]
    if out is not None:
        a["residual_out"] = pick(out)
    a["y"] = pick(y)
    _lib.moe_rmsnorm(a)
    ok()
    for n in ("residual_out", "y"):
        if a[n] is not None:
            assert torch.equal(a[n], want[n]), n


@pytest.mark.gpu
def test_one_buffer_for_both_is_refused():
    x, res, w = (torch.ones(n, 64, dtype=torch.bfloat16, device="cuda") for n in (3, 3, 2))
    for both in (x, res, torch.empty_like(x)):
        with pytest.raises(_lib.MoeError) as e:
            _lib.moe_rmsnorm(dict(T=3, d=64, eps=1e-6, x=x, residual=res, weight=w[0].float(),
                                  residual_out=both, y=both))
        assert e.value.status == _lib.MOE_ERR_INVALID_ARG
