"""Calls with stream= from another current stream: what the layer's classes allocate
and fill for such a call belongs to that stream."""
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib
from moe_expert_layer_04_gb300.layer import Dims, GroupedLinearFP8, MoELayer
from tests.test_gpu_fp8_layer import layer_inputs

pytestmark = pytest.mark.gpu


def stream_of(t):
    """The stream whose pool the tensor's memory is from."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("no segment")


def projection(rows=64, G=3, N=256, K=128):
    gen = torch.Generator(device="cuda").manual_seed(0)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)
    p = GroupedLinearFP8(rn(G, N, K), rows)
    offsets = torch.tensor([0, 20, 20, rows], dtype=torch.int32, device="cuda")
    return p, rn(rows, K), rn(rows, N), offsets


def test_projection_on_another_stream():
    p, x, dy, offsets = projection()
    want = p.forward(x, offsets), p.backward(dy), p.dW.clone()
    side = torch.cuda.Stream()
    for i in range(20):
        side.wait_stream(torch.cuda.current_stream())
        torch.cuda._sleep(1000000)             # the current stream stays behind
        junk = torch.full((64, 256), float(i), dtype=torch.bfloat16, device="cuda")
        del junk                               # a block that the current stream still writes
        y = p.forward(x, offsets, stream=side)
        dx = p.backward(dy, stream=side)
        side.synchronize()
        assert stream_of(y) == stream_of(dx) == side.cuda_stream
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(dx, want[1]) and torch.equal(p.dW, want[2])
    assert _lib.moe_last_device_status() == _lib.MOE_OK


def test_gradient_of_no_rows_is_zeroed_on_its_stream():
    p, x, dy, offsets = projection()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20000000)
        p.dW.fill_(1.0)
    p.forward(x[:0], torch.zeros(4, dtype=torch.int32, device="cuda"), stream=side)
    p.backward(dy[:0], stream=side)
    torch.cuda.synchronize()
    assert not p.dW.any()


@pytest.mark.parametrize("fp8", [False, True])
def test_decoding_on_another_stream(fp8):
    w, bias, x = layer_inputs(9, 256, 16, 4, 128)
    layer = MoELayer(Dims(9, 256, 16, 4, 128), w, scaling=2.5, fp8=fp8)
    want = layer.forward_few(x, bias)
    side = torch.cuda.Stream()
    for i in range(20):
        side.wait_stream(torch.cuda.current_stream())
        torch.cuda._sleep(1000000)
        junk = torch.full((9, 256), float(i), dtype=torch.bfloat16, device="cuda")
        del junk
        y = layer.forward_few(x, bias, stream=side)
        side.synchronize()
        assert stream_of(y) == side.cuda_stream
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    assert _lib.moe_last_device_status() == _lib.MOE_OK


def test_result_outlives_its_last_reader():
    """A result read on the current stream and dropped: its memory does not go back to
    the other stream while that reading is still queued."""
    p, x, _, offsets = projection()
    want = p.forward(x, offsets)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    copies = []
    for _ in range(10):
        y = p.forward(x, offsets, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(2000000)
        copies.append(y.clone())
        del y
        with torch.cuda.stream(side):
            torch.full((64, 256), 9.0, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    assert all(torch.equal(c, want) for c in copies)
