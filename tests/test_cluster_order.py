"""Order of what the CTAs of a cluster do in one another's shared memory."""
import re

import numpy as np
import pytest
import torch

from tests.test_launch_order import kernels


def test_who_writes_to_another_cta_has_waited_for_it_to_begin():
    """The shared memory of another CTA of the cluster may be accessed once that CTA runs: a
    cluster barrier stands ahead of the first address in it."""
    found = {}
    for _, name, body in kernels():
        at = re.search(r"\bdsmem_map\(|shared::cluster\.b32", body)
        if at:
            sync = re.search(r"\bcluster_sync_all\(|barrier\.cluster\.wait", body)
            found[name] = sync is not None and sync.start() < at.start()
    assert {"balance_seq_kernel", "rmsnorm_bwd_kernel", "mx4_gemm_kernel"} <= set(found)
    assert all(found.values()), found


@pytest.mark.gpu
@pytest.mark.parametrize("E", [130, 257, 384, 513, 1000])
def test_sums_of_many_clusters(E):
    """More clusters than run at once, of two to eight CTAs, again and again: the bits of the
    first call, and the loss of its terms."""
    from moe_expert_layer_04_gb300 import _lib
    from tests import test_gpu_balance as B
    from tests.test_gpu_fp8 import ok
    T, k, n = 2000, 3, 700
    rng = np.random.default_rng(E)
    z, ids = B.inputs(rng, T, E, k)
    offs = np.sort(np.concatenate([[0, T], rng.integers(0, T + 1, n - 1)])).astype(np.int32)
    a = B.call(z, ids, B.SIG, offs)
    ok()
    B.check(a, B.reference(z.astype(np.float64), ids, B.SIG, offs), z)
    first = {x: a[x].clone() for x in ("loss", "seq_loss", "load", "counts", "tokens")}
    differ = []
    for _ in range(100):
        _lib.moe_balance_loss(a)
        differ += [(a[x] != first[x]).any() for x in first]
    ok()
    assert not torch.stack(differ).any()
