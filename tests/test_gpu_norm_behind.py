"""Both directions of the norm launched behind one another with nothing between: each call may
begin before the one ahead of it ends, the backward reads what the forward ahead wrote, and all
backward calls share a workspace.  Every output of every call as it is alone, bit for bit."""
import numpy as np
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib
from tests import test_gpu_norm as N
from tests.test_gpu_fp8 import ok

pytestmark = pytest.mark.gpu

# (a row's own kernel, rows by the ring, wide rows by one CTA and by clusters of two and four)
CASES = [(1500, 4096, _lib.MOE_ROWS_FP8), (1300, 3616, _lib.MOE_ROWS_MXFP4), (700, 512, _lib.MOE_ROWS_MXFP8),
         (5, 2048, _lib.MOE_ROWS_FP8), (330, 7168, _lib.MOE_ROWS_FP8), (200, 16384, _lib.MOE_ROWS_MXFP8),
         (160, 32768, _lib.MOE_ROWS_NONE), (3, 40, _lib.MOE_ROWS_NONE)]
FWD, BWD = ("residual_out", "y", "rstd", "q", "scales"), ("dx", "d_weight")


@pytest.mark.parametrize("T,d,fmt", CASES)
def test_calls_behind_one_another(T, d, fmt):
    rng = np.random.default_rng(T + d)
    w = torch.from_numpy(rng.standard_normal(d).astype(np.float32))
    ws = torch.empty(_lib.moe_rmsnorm_bwd_workspace_size(T, d), dtype=torch.uint8, device="cuda").fill_(255)
    alone = []
    for _ in range(3):
        a = N.forward(N.rows(rng, T, d), w, N.rows(rng, T, d), fmt)
        b = dict(T=T, d=d, x=a["residual_out"], weight=a["weight"], rstd=a["rstd"], ws=ws,
                 dy=N.rows(rng, T, d).cuda(), d_residual=N.rows(rng, T, d).cuda(),
                 dx=torch.empty_like(a["x"]), d_weight=torch.empty_like(a["weight"]))
        _lib.moe_rmsnorm_backward(b)
        ok()
        alone.append((a, b))
    calls = []
    for i in range(36):
        a, b = alone[i % 3]
        new = lambda c, names: {n: c[n].clone().fill_(0x55 if c[n].dtype == torch.uint8 else -3)
                                for n in names if c.get(n) is not None}
        x = dict(a, **new(a, FWD))
        if fmt in (_lib.MOE_ROWS_MXFP8, _lib.MOE_ROWS_MXFP4):   # (bytes behind a row stay)
            x["scales"][:, d // 32:] = a["scales"][:, d // 32:]
        calls.append((x, dict(b, x=x["residual_out"], rstd=x["rstd"], **new(b, BWD))))
    torch.cuda.synchronize()
    for a, b in calls:
        _lib.moe_rmsnorm(a)
        _lib.moe_rmsnorm_backward(b)
    ok()
    for i, (a, b) in enumerate(calls):
        want_a, want_b = alone[i % 3]
        for got, want, names in ((a, want_a, FWD), (b, want_b, BWD)):
            for n in names:
                if want.get(n) is not None:
                    assert torch.equal(got[n], want[n]), (i, n)
