"""The balance loss on either side of the rule that gives a call one CTA or many: few and many
experts, tokens and sequences."""
import numpy as np
import pytest

from tests import test_gpu_balance as B
from tests.test_gpu_fp8 import ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,n", [(128, 384, 1), (129, 384, 1), (66, 1024, 1), (67, 1024, 1), (128, 1024, 1),
                                   (1, 1024, 3), (9, 1024, 4), (128, 16, 6), (128, 16, 7), (44, 384, 4),
                                   (45, 384, 4), (3, 97, 9), (128, 97, 4)])
@pytest.mark.parametrize("score", [B.SIG, B.SOFT])
def test_small_calls(T, E, n, score):
    rng = np.random.default_rng(T + E)
    z, ids = B.inputs(rng, T, E, 4)
    offs = np.sort(np.concatenate([[0, T], rng.integers(0, T + 1, n - 1)])).astype(np.int32)
    valid = (rng.random(T) < 0.8).astype(np.uint8)
    a = B.call(z, ids, score, offs, valid)
    ok()
    B.check(a, B.reference(z.astype(np.float64), ids, score, offs, valid), z)
