"""How many weight rows the grouped calls take: the largest count passes the checks of sizes (and
is refused for the missing pointers that follow), the next one is not supported."""
import pytest

from moe_expert_layer_04_gb300 import _lib

BAD, UNS = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("G,I,want", [(1, (1 << 30) - 128, BAD), (1, 1 << 30, UNS), (1024, 1 << 20, UNS),
                                      (1023, 1 << 20, BAD)])
def test_fp8_ffn(G, I, want):
    got = _lib.load().moe_expert_ffn_fp8(None, None, None, G, 8, None, None, None, None, None, 0, 128,
                                         I, 7.0, None, None, None, None)
    assert got == want


@pytest.mark.parametrize("G,N,want", [(1, (1 << 31) - 16, BAD), (1024, (1 << 21) - 16, BAD), (1024, 1 << 21, UNS)])
def test_fp8_matmul(G, N, want):
    got = _lib.load().moe_fp8_matmul(None, None, None, G, 8, None, None, None, 0, N, 128, None, None)
    assert got == want


@pytest.mark.parametrize("G,I,want", [(1, (1 << 30) - 256, BAD), (1, (1 << 30) - 128, UNS)])
def test_mx4_ffn(G, I, want):
    got = _lib.load().moe_expert_ffn_mx4(None, None, None, G, 8, None, None, None, None, None, 0, 128,
                                         I, 7.0, None, None, None, None)
    assert got == want
