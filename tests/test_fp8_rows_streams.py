"""GroupedLinearFP8's forward on several streams at once: no call's quantised rows are those of
another's."""
import numpy as np
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib, layer as L
from tests.test_mx4_streams import FakeStream

BF16 = torch.bfloat16


def test_rows_of_each_stream(monkeypatch):
    made = []
    monkeypatch.setattr(_lib, "moe_fp8_wgrad_workspace_size", lambda *a: 16)
    for name in ("moe_fp8_quantize_weights", "moe_fp8_quantize", "moe_fp8_matmul"):
        monkeypatch.setattr(_lib, name, lambda *a, _n=name, **k: made.append((_n, a)))
    monkeypatch.setattr(L, "_result", lambda stream, device, *shape: torch.empty(*shape, dtype=BF16))
    p = L.GroupedLinearFP8(torch.zeros(2, 16, 144, dtype=BF16), 9)
    x, offs = torch.zeros(5, 144, dtype=BF16), torch.zeros(3, dtype=torch.int32)
    streams = [None, FakeStream(), FakeStream()]
    seen = []
    for s in streams * 2:
        made.clear()
        p.forward(x, offs, stream=s)
        (q, a), (m, b) = made
        assert m == "moe_fp8_matmul" and a[3] is b[0] and a[4] is b[1]
        assert a[3].shape == (9, 144) and a[4].shape == (9, 2)
        seen.append((a[3].data_ptr(), a[4].data_ptr()))
    assert seen[:3] == seen[3:]
    assert len({q for q, _ in seen}) == 3 and len({f for _, f in seen}) == 3


@pytest.mark.gpu
def test_streams_at_once():
    rng = np.random.default_rng(3)
    G, N, K, R = 3, 512, 1024, 2000
    t = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda().to(BF16)
    p = L.GroupedLinearFP8(t(G, N, K), R)
    offs = torch.tensor([0, 700, 701, R], dtype=torch.int32, device="cuda")
    xs = [t(R, K) * s for s in (1.0, 3.0, 0.1)]
    alone = []
    for x in xs:
        alone.append(p.forward(x, offs).clone())
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    outs = [[] for _ in xs]
    for _ in range(30):
        for s, x, o in zip(streams, xs, outs):
            o.append(p.forward(x, offs, stream=s))
    torch.cuda.synchronize()
    assert _lib.moe_last_device_status() == _lib.MOE_OK
    for o, want in zip(outs, alone):
        for y in o:
            assert torch.equal(y, want)
