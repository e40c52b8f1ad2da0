"""GroupedLinearMX4 on several streams at once and in graphs that replay at once: no call's
quantised rows are those of another's."""
import numpy as np
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib, layer as L

BF16 = torch.bfloat16


class FakeStream:
    pass


@pytest.mark.parametrize("bits,K", [(8, 128), (4, 96)])
def test_rows_of_each_stream(monkeypatch, bits, K):
    made = []
    for name in ("moe_mx_quantize", "moe_mx4_quantize", "moe_mx4_matmul"):
        monkeypatch.setattr(_lib, name, lambda *a, _n=name: made.append((_n, a)))
    monkeypatch.setattr(L, "_result", lambda stream, device, *shape: torch.empty(*shape, dtype=BF16))
    p = L.GroupedLinearMX4(torch.zeros(2, 16, K, dtype=BF16), 9, bits)
    x, offs = torch.zeros(5, K, dtype=BF16), torch.zeros(3, dtype=torch.int32)
    streams = [None, FakeStream(), FakeStream()]
    seen = []
    for s in streams * 2:
        made.clear()
        p.forward(x, offs, stream=s)
        (q, a), (m, b) = made
        assert m == "moe_mx4_matmul" and a[3] is b[0] and a[4] is b[1]
        assert a[3].shape == (9, K if bits == 8 else K // 2)
        seen.append((a[3].data_ptr(), a[4].data_ptr()))
    assert seen[:3] == seen[3:]
    assert len({q for q, _ in seen}) == 3 and len({f for _, f in seen}) == 3


def inputs(bits):
    rng = np.random.default_rng(bits)
    G, N, K, R = 3, 512, 1024, 2000
    t = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda().to(BF16)
    p = L.GroupedLinearMX4(t(G, N, K), R, bits)
    offs = torch.tensor([0, 700, 701, R], dtype=torch.int32, device="cuda")
    return p, offs, [t(R, K) * s for s in (1.0, 3.0, 0.1, 40.0)]


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 8])
def test_streams_at_once(bits):
    p, offs, xs = inputs(bits)
    alone = []
    for x in xs:
        alone.append(p.forward(x, offs).clone())
        torch.cuda.synchronize()
    assert not torch.equal(alone[0], alone[1])
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


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 8])
def test_graphs_of_one_stream_at_once(bits):
    """Two graphs captured on one stream, after a call there, replayed beside each other and
    beside calls of that stream."""
    p, offs, xs = inputs(bits)
    alone = [p.forward(x, offs).clone() for x in xs]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs, outs = [], []
    with torch.cuda.stream(st):
        p.forward(xs[2], offs)
        for x in xs[:2]:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                outs.append(p.forward(x, offs))
            graphs.append(g)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in graphs]
    for _ in range(30):
        for g, s in zip(graphs, sides):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(st):
            y = p.forward(xs[3], offs)
    torch.cuda.synchronize()
    assert _lib.moe_last_device_status() == _lib.MOE_OK
    for got, want in zip(outs + [y], [alone[0], alone[1], alone[3]]):
        assert torch.equal(got, want)
