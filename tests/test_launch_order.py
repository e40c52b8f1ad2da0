"""Order of kernels whose launch may precede the end of the kernel ahead
(programmatic dependent launch): whoever lets the kernel behind begin early must
itself end only after the kernel ahead, or a kernel two places behind could run
before that one's stores."""
import glob
import os
import re

import numpy as np
import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "moe_expert_layer_04_gb300", "csrc")


def kernels():
    """(file, name, body) of every __global__ function."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        text = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)
        for m in re.finditer(r"__global__", text):
            at = text.index("{", m.end())
            head = re.sub(r"__launch_bounds__\((?:[^()]|\([^()]*\))*\)", "", text[m.end():at])
            depth, end = 0, at
            while True:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
                if depth == 0:
                    break
            yield os.path.basename(path), re.search(r"(\w+)\s*\(", head).group(1), text[at:end]


def test_kernels_are_found():
    names = {n for _, n, _ in kernels()}
    assert {"few_gate_kernel", "few_experts_kernel", "fp8_gemm_kernel", "fp8_thin_kernel",
            "fp8_rows_kernel"} <= names


def test_who_lets_the_kernel_behind_begin_waits_for_the_one_ahead():
    early = [(f, n, b) for f, n, b in kernels()
             if "griddepcontrol.launch_dependents" in b or "let_kernels_behind_begin(" in b]
    assert len(early) >= 6
    missing = [(f, n) for f, n, b in early
               if "griddepcontrol.wait" not in b and "wait_for_kernels_ahead(" not in b]
    assert not missing


def blocks_around(body, at):
    """Opening braces of the blocks around place `at`."""
    stack = []
    for i, c in enumerate(body[:at]):
        if c == "{":
            stack.append(i)
        elif c == "}":
            stack.pop()
    return stack


def test_who_issues_a_bulk_copy_of_others_stores_has_the_proxy_fence():
    """The fence between generic stores and asynchronous copies works for the
    thread that executes it: it stands in a block around the copy, not in a branch
    that other lanes than the copying ones take."""
    body = next(b for _, n, b in kernels() if n == "few_experts_kernel")
    copies = [m.start() for m in re.finditer(r"\bbulk_load\(", body)]
    assert copies
    for at in copies:
        around = set(blocks_around(body, at))
        fences = [m.start() for m in re.finditer(r"fence_proxy_async_global\(", body[:at])]
        assert any(set(blocks_around(body, f)) <= around for f in fences)
    # and the lanes that store what is copied
    at = body.index("p.h[")
    after = body.index("fence_proxy_async_global(", at)
    assert set(blocks_around(body, after)) <= set(blocks_around(body, at))


def test_the_arrival_that_frees_shared_memory_takes_every_lanes_loads():
    """One lane arrives for the warp: what it arrives with depends on the values
    that all lanes have loaded (a vote), not on its own alone."""
    text = open(os.path.join(CSRC, "few.cu")).read()
    at = text.index("void arrive_after(")
    body = text[at:text.index("\n}\n", at)]
    voted = re.search(r"(\w+) = __any_sync\(0xffffffffu, \(loaded & zero\) != 0\)", body)
    assert voted
    assert re.search(r"smem_u32\(bar\) \+ " + voted.group(1), re.sub(r"\s+", " ", body))


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,fp8", [(1, 6, 2, False), (4, 64, 6, False), (2, 96, 8, True), (1, 4, 4, True)])
def test_rows_that_lanes_copy_are_the_ones_stored(T, E, k, fp8):
    """Passes of few rows, whose h each lane copies to shared memory for itself:
    two inputs in turn on one workspace, every call as it is alone."""
    from moe_expert_layer_04_gb300 import _lib
    from tests.test_gpu_few import check, make, run
    a = make(T, 256, E, k, 576, fp8)
    b = dict(a, x=make(T, 256, E, k, 576, fp8, seed=1)["x"])
    alone = []
    for c in (a, b):
        run(c)
        check(c)
        alone.append(c["y"].clone())
    wrong = []
    for i in range(300):
        w = (i * 7 // 3) % 2
        _lib.moe_layer_few((a, b)[w])
        wrong.append((a["y"] != alone[w]).any())
    assert _lib.moe_last_device_status() == _lib.MOE_OK
    assert not torch.stack(wrong).any()


@pytest.mark.gpu
def test_early_kernel_behind_the_few_token_layer_reads_its_weights():
    """A matmul launched early behind the call takes the call's routing weights
    (stored by the first of its two kernels) as its row weights."""
    from moe_expert_layer_04_gb300 import _lib
    from tests.test_gpu_few import make, n64
    T, k, N, K = 24, 4, 64, 128
    a = make(T, 256, 40, k, 128, True)
    xs = [a["x"], a["x"].roll(5, 0) * -1.0]
    rng = np.random.default_rng(0)
    q = lambda *s: torch.from_numpy(rng.integers(48, 64, s).astype(np.uint8)).cuda()   # 0.5 .. 1.875
    a_q, b_q = q(T * k, K), q(1, N, K)
    a_s, b_s = torch.ones(T * k, 1, device="cuda"), torch.ones(1, 1, 1, device="cuda")
    offs = torch.tensor([0, T * k], dtype=torch.int32, device="cuda")
    outs, want = [], []
    for i in range(60):
        a["x"] = xs[i % 2]
        out = torch.empty(T * k, N, dtype=torch.bfloat16, device="cuda")
        _lib.moe_layer_few(a)
        _lib.moe_fp8_matmul(a_q, a_s, offs, 1, T * k, b_q, b_s, a["weights"],
                            T * k, N, K, out)
        outs.append(out)
        want.append(a["weights"].clone())
    torch.cuda.synchronize()
    assert _lib.moe_last_device_status() == _lib.MOE_OK
    prod = n64(a_q.view(torch.float8_e4m3fn).float()) @ n64(b_q[0].view(torch.float8_e4m3fn).float()).T
    assert not torch.equal(want[0], want[1])
    for out, w in zip(outs, want):
        # products of these codes sum exactly in fp32; one rounding by the weight, one to bf16
        ref = n64(w).reshape(-1, 1) * prod
        assert np.max(np.abs(n64(out) / ref - 1)) <= 2.0 ** -8 + 2.0 ** -22
