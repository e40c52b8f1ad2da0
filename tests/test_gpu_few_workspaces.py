"""The workspaces that a layer keeps for decoding: one for a number of tokens and a
stream, a captured graph's own where that stream has none yet, new ones on demand."""
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib
from moe_expert_layer_04_gb300.layer import Dims, MoELayer
from tests.test_gpu_fp8_layer import layer_inputs

pytestmark = pytest.mark.gpu

DIMS = (12, 512, 48, 4, 256)


def build(fp8):
    T, d, E, k, I = DIMS
    w, bias, x = layer_inputs(T, d, E, k, I)
    return MoELayer(Dims(*DIMS), w, scaling=2.5, fp8=fp8), bias, x


@pytest.mark.parametrize("fp8", [False, True])
def test_streams_that_decode_as_many_tokens_at_once(fp8):
    layer, bias, x = build(fp8)
    inputs = [x, x.roll(1, 0) * -1.0, x * 0.5]
    want = [layer.forward_few(v, bias).clone() for v in inputs]
    streams = [torch.cuda.Stream() for _ in inputs]
    torch.cuda.synchronize()
    # a workspace each, zeroed in the order of its own stream
    seen = set()
    for s, v in zip(streams, inputs):
        layer.forward_few(v, bias, stream=s)
        with torch.cuda.stream(s):
            seen.add(layer._few_workspace(len(v), v.device).data_ptr())
    assert len(seen) == len(streams)
    torch.cuda.synchronize()
    outs = [[] for _ in inputs]
    for _ in range(30):
        for o, s, v in zip(outs, streams, inputs):
            o.append(layer.forward_few(v, bias, stream=s))
    torch.cuda.synchronize()
    assert _lib.moe_last_device_status() == _lib.MOE_OK
    for o, y in zip(outs, want):
        assert all(torch.equal(v, y) for v in o)


@pytest.mark.parametrize("warm", ["not", "elsewhere", "on_the_capturing_stream"])
def test_captured_calls(warm):
    """A first call inside a capture works too: the graph then has its own workspace."""
    layer, bias, x = build(True)
    want = MoELayer(Dims(*DIMS), layer.w, scaling=2.5, fp8=True).forward_few(x, bias)
    side = torch.cuda.Stream()
    if warm == "elsewhere":
        layer.forward_few(x, bias)
    if warm == "on_the_capturing_stream":
        layer.forward_few(x, bias, stream=side)
    torch.cuda.synchronize()
    y, z = torch.empty_like(x), torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        layer.forward_few(x, bias, y=y)
        layer.forward_few(x, bias, y=z)
    # before the graph ever ran, and in turn with it
    for _ in range(3):
        assert torch.equal(layer.forward_few(x, bias), want)
        y.zero_()
        z.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(z, want)
        other = layer.forward_few(x, bias, stream=side)
        side.synchronize()
        assert torch.equal(other, want)
    assert _lib.moe_last_device_status() == _lib.MOE_OK


def test_new_workspaces_on_demand():
    """(After a call that recorded MOE_ERR_TIMEOUT, which may leave counters behind.)"""
    layer, bias, x = build(True)
    want = layer.forward_few(x, bias).clone()
    ws = layer._few_workspace(len(x), x.device)
    torch.cuda.synchronize()
    layer.reset_few()
    again = layer._few_workspace(len(x), x.device)
    assert again is not ws and not again.any()
    assert torch.equal(layer.forward_few(x, bias), want)
    assert _lib.moe_last_device_status() == _lib.MOE_OK
