"""The norm, the routing with its balance loss, the experts and their backward together, as a
block of a model runs them: MoELayer(norm_eps, balance, mx4), GroupedLinearMX4 and
moe_gate_backward.

Whole gradients are held to the layer's bounds (relative Frobenius 1e-2).  The MXFP4 layer
against plain formulas on the values that its weights stand for: what is left is MXFP8 rows, an
error of q = 0.028 for x and for h (E4M3 elements 0.0245; a block's largest, above 464 of 512
in one block of seven, saturates at 448 and adds 0.013), so 1.45 q through the gate's product
and q: 0.049, held to 0.065."""
import numpy as np
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib
from moe_expert_layer_04_gb300.layer import Dims, GroupedLinearMX4, MoELayer
from tests import mx4_ref as R
from tests.test_gpu_fp8 import bf16, codes, f64, ok
from tests.test_gpu_fp8_layer import layer_inputs, plain, randn, rel
from tests.test_gpu_mx4 import between

pytestmark = pytest.mark.gpu

EPS = 1e-5


def norm_of(v, w):
    r = 1 / np.sqrt((v * v).mean(-1, keepdims=True) + EPS)
    return v * r * w


def block(T, d, E, k, I, seed=0, **kw):
    w, bias, x = layer_inputs(T, d, E, k, I, seed)
    rng = np.random.default_rng(seed + 1)
    w["norm"] = torch.from_numpy((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)).cuda()
    res = randn(rng, 1.5, T, d)
    return MoELayer(Dims(T, d, E, k, I), w, 2.5, norm_eps=EPS, **kw), w, bias, x, res


# ------------------------------------------------------------- the MXFP4 layer

def mx4_values(w):
    """Expert weights [G, N, K] -> the values of their MXFP4 form, in float64."""
    G, N, K = w.shape
    return R.values4(*R.quantise4(f64(w).reshape(G * N, K))).reshape(G, N, K)


@pytest.mark.parametrize("T,d,E,k,I", [(1, 256, 32, 4, 128), (40, 256, 32, 4, 128), (200, 384, 33, 6, 256),
                                       (700, 640, 7, 2, 384)])
def test_mx4_layer(T, d, E, k, I):
    w, bias, x = layer_inputs(T, d, E, k, I)
    layer = MoELayer(Dims(T, d, E, k, I), w, scaling=2.5, mx4=True)
    y = f64(layer.forward(x, bias))
    ok()
    v = {n: mx4_values(w[n]) for n in ("W13", "W2")}
    want = plain(dict(w, W13=torch.from_numpy(v["W13"]), W2=torch.from_numpy(v["W2"])), bias, x, k, 2.5, 7.0)
    assert rel(y, want) <= 0.065
    # the same weights given as codes: the same bits
    q = dict(W_g=w["W_g"], **{n: getattr(layer, n) for n in ("W13_q", "W13_sf", "W2_q", "W2_sf")})
    again = MoELayer(Dims(T, d, E, k, I), q, scaling=2.5, mx4=True)
    assert torch.equal(again.forward(x, bias), layer.y)


@pytest.mark.parametrize("bits", [4, 8])
def test_projection(bits):
    rng = np.random.default_rng(bits)
    G, N, K = 5, 264, 384
    counts = [130, 0, 1, 77, 300]
    rows = sum(counts)
    w, x = randn(rng, K ** -0.5, G, N, K), randn(rng, 1.0, rows, K)
    offs = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    f = torch.rand(rows, device="cuda") + 0.5
    p = GroupedLinearMX4(w, rows + 10, bits)
    for fw in (None, f):
        y = p.forward(x, offs, row_weight=fw)
        ok()
        a = R.values4(*R.quantise4(f64(x))) if bits == 4 else R.values8(*R.quantise8(f64(x)))
        b, fr = mx4_values(w), np.ones(rows) if fw is None else f64(fw)
        lo = 0
        for g, n in enumerate(counts):
            s = slice(lo, lo + n)
            between(y[s], a[s] @ b[g].T * fr[s, None], np.abs(a[s]) @ np.abs(b[g]).T * fr[s, None], K, f"group {g}")
            lo += n
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = p.forward(x, offs, stream=side, row_weight=f)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(z, y)
    y = GroupedLinearMX4(None, rows, bits, codes=(p.w_q, p.w_sf)).forward(x, offs, row_weight=f)
    assert torch.equal(z, y)
    p.weight = w.mul_(2.0)
    p.quantize_weights()
    assert torch.equal(p.forward(x, offs, row_weight=f), 2 * z)


# ------------------------------------------------------------------ the norm

@pytest.mark.parametrize("kind", ["bf16", "mx", "fp8", "mx4"])
@pytest.mark.parametrize("residual", [False, True])
def test_layer_with_norm(kind, residual):
    T, d, E, k, I = 130, 512, 32, 4, 128
    kw = {} if kind == "bf16" else {kind: True}
    layer, w, bias, x, res = block(T, d, E, k, I, **kw)
    res = res if residual else None
    y = layer.forward(x, bias, residual=res).clone()
    ok()
    v = f64(bf16(f64(x) + f64(res))) if residual else f64(x)
    assert np.array_equal(f64(layer.residual), v)
    assert rel(f64(layer.xn), norm_of(v, f64(w["norm"]))) <= 2.0 ** -8
    bare = MoELayer(Dims(T, d, E, k, I), w, 2.5, **kw)
    other = bare.forward(layer.xn, bias)
    assert torch.equal(bare.ids, layer.ids) and torch.equal(bare.weights, layer.weights)
    if kind == "bf16":
        assert torch.equal(other, y)
        return
    # the permuted rows are the norm's codes, not those of the rounded rows
    tok = layer.row_token.long()
    assert torch.equal(layer.x_perm_q, layer.xn_q[tok])
    s = layer.x_perm_s if kind == "fp8" else layer.x_perm_sf
    used = d // 32 if kind != "fp8" else s.shape[1]
    assert torch.equal(s[:, :used], layer.xn_s[tok][:, :used])
    # ... which differ from them where the rows' rounding moves an element over a border between
    # codes: by 2^-10 on average, borders 2^-3.5 apart, one element in 91, which then is 2^-3.5
    # off: 0.0093 of x in the mean square, 1.45 of that in h (0.0135), which moves 0.0135 /
    # 2^-3.5 = 15 % of h's elements over a border, 0.034 in the mean square.  Together 0.037,
    # held to 0.05.
    assert rel(f64(y), f64(other)) <= 0.05


def test_norm_ahead_of_decoding():
    T, d, E, k, I = 64, 256, 32, 4, 128
    layer, w, bias, x, res = block(T, d, E, k, I)
    y = layer.forward(x, bias, residual=res).clone()
    kept, stream = layer.xn.clone(), layer.residual.clone()
    for n in (1, 5, 32):
        rows, v = layer.norm(x[:n].contiguous(), res[:n].contiguous())
        assert torch.equal(rows, kept[:n]) and torch.equal(v, stream[:n])
        few = layer.forward_few(rows, bias)
        ok()
        assert rel(f64(few), f64(y[:n])) <= 1e-2
    assert torch.equal(layer.xn, kept) and torch.equal(layer.residual, stream)
    rows, v = layer.norm(x[:3].contiguous())
    assert v.data_ptr() == x.data_ptr() and rows.shape == (3, d)


# --------------------------------------------------------------- the gate's part

@pytest.mark.parametrize("T,d,E", [(1, 128, 1), (3, 256, 7), (300, 384, 97), (1000, 256, 384), (129, 128, 1024),
                                   (5000, 512, 130)])
def test_gate_backward(T, d, E):
    """dz is rounded to bf16 exactly as here; sums of its products with bf16 values are fp32
    (at most one spacing, 2^-23, of the magnitudes an addition), the first result is rounded to
    bf16 and the sum again."""
    rng = np.random.default_rng(T + E)
    dz = (rng.standard_normal((T, E)) * np.exp(2 * rng.standard_normal((T, 1)))).astype(np.float32)
    x, W, dX, = randn(rng, 1.0, T, d), randn(rng, 0.05, E, d), randn(rng, 2.0, T, d)
    dW = torch.from_numpy(rng.standard_normal((E, d)).astype(np.float32)).cuda()
    z = f64(bf16(dz.astype(np.float64)))
    gx, mx = z @ f64(W), np.abs(z) @ np.abs(f64(W))
    gw, mw = z.T @ f64(x), np.abs(z).T @ np.abs(f64(x))
    ws = torch.empty(_lib.moe_gate_bwd_workspace_size(T, d, E), dtype=torch.uint8, device="cuda").fill_(255)
    for both in (True, False):
        a, b = dX.clone(), dW.clone()
        _lib.moe_gate_backward(torch.from_numpy(dz).cuda(), x, W, T, d, E, a, b if both else None, ws)
        ok()
        part = (E + 2) * 2.0 ** -23 * mx
        err = part + 2.0 ** -8 * (np.abs(gx) + part)
        want = f64(dX) + gx
        assert (np.abs(f64(a) - want) <= err + 2.0 ** -8 * (np.abs(want) + err) + 1e-30).all()
        if both:
            lim = (T + 2) * 2.0 ** -23 * mw + 2.0 ** -23 * (np.abs(gw) + np.abs(f64(dW)))
            assert (np.abs(f64(b) - f64(dW) - gw) <= lim + 1e-30).all()
        else:
            assert torch.equal(b, dW)
    b = dW.clone()
    _lib.moe_gate_backward(torch.from_numpy(dz).cuda(), x, W, T, d, E, None, b, ws)
    ok()
    assert (np.abs(f64(b) - f64(dW) - gw) <= lim + 1e-30).all()


def test_gate_backward_refusals():
    z = torch.zeros(8, 16, device="cuda")
    x, W = (torch.zeros(n, 128, dtype=torch.bfloat16, device="cuda") for n in (8, 16))
    ws = torch.empty(_lib.moe_gate_bwd_workspace_size(8, 128, 16), dtype=torch.uint8, device="cuda")
    dX, dW = torch.ones_like(x), torch.ones(16, 128, device="cuda")
    for kw, status in ((dict(T=-1), _lib.MOE_ERR_INVALID_ARG), (dict(d=192), _lib.MOE_ERR_UNSUPPORTED),
                       (dict(E=1025), _lib.MOE_ERR_UNSUPPORTED), (dict(ws=ws[:-1]), _lib.MOE_ERR_WORKSPACE),
                       (dict(ws=None), _lib.MOE_ERR_WORKSPACE), (dict(x=None), _lib.MOE_ERR_INVALID_ARG),
                       (dict(T=1 << 22), _lib.MOE_ERR_UNSUPPORTED)):
        a = dict(dlogits=z, x=x, W_g=W, T=8, d=128, E=16, dX=dX, dW_g=dW, ws=ws)
        a.update(kw)
        with pytest.raises(_lib.MoeError) as e:
            _lib.moe_gate_backward(**a)
        assert e.value.status == status
    _lib.moe_gate_backward(z, x, W, 0, 128, 16, dX, dW, None)
    ok()
    assert (dX == 1).all() and (dW == 1).all()
    assert _lib.moe_gate_bwd_workspace_size(8, 192, 16) == 0


# ------------------------------------------------------------- a training step

def autograd(layer, w, v, dY, d_res, alpha, g, softmax, offs, valid):
    """Gradients of sum(y dY) + g balance loss + sum(v d_res) by torch's autograd in float64,
    with the experts that the layer chose; v the residual stream."""
    D = layer.dims
    leaf = lambda t: torch.from_numpy(f64(t)).requires_grad_()
    v, nw, wg, w13, w2 = (leaf(t) for t in (v, w["norm"], w["W_g"], w["W13"], w["W2"]))
    x = v * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS) * nw
    z = x @ wg.T
    ids = layer.ids.long().cpu()
    s = torch.sigmoid(z)
    sel = torch.gather(s, 1, ids)
    wt = 2.5 * sel / sel.sum(1, keepdim=True)

    def ffn(rows, e):
        gu = rows @ w13[e].T
        a, u = gu[:, :D.I].clamp(max=7.0), gu[:, D.I:].clamp(-7.0, 7.0)
        return (a * torch.sigmoid(a) * u) @ w2[e].T
    y = ffn(x, D.E)
    for e in range(D.E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if len(t):
            y = y.index_add(0, t, wt[t, j, None] * ffn(x[t], e))
    p = torch.softmax(z, 1) if softmax else s / s.sum(1, keepdim=True)
    loss, n = 0.0, len(offs) - 1
    for q in range(n):
        t = torch.arange(offs[q], offs[q + 1])
        t = t[valid[t] != 0] if valid is not None else t
        if len(t):
            f = torch.bincount(ids[t].flatten(), minlength=D.E).double() * D.E / (D.k * len(t))
            loss = loss + alpha / n * (f * p[t].mean(0)).sum()
    total = (y * torch.from_numpy(f64(dY))).sum() + g * loss
    if d_res is not None:
        total = total + (v * torch.from_numpy(f64(d_res))).sum()
    total.backward()
    return dict(y=y, loss=loss, dX=v.grad, dnorm=nw.grad, dW_g=wg.grad, dW13=w13.grad, dW2=w2.grad)


def near(got, want, bound, what):
    assert rel(f64(got), want.detach().numpy()) <= bound, what


@pytest.mark.parametrize("softmax,n,padded,residual", [(False, 1, False, True), (True, 3, True, True),
                                                       (False, 4, True, False)])
@pytest.mark.parametrize("alpha", [0.5, 200.0])
def test_training_step(softmax, n, padded, residual, alpha):
    """alpha 200: the balance loss's gradient is what dW_g is made of."""
    T, d, E, k, I = 150, 256, 9, 2, 128
    layer, w, bias, x, res = block(T, d, E, k, I, backward=True, balance=alpha, sequences=n,
                                   balance_softmax=softmax)
    rng = np.random.default_rng(7)
    dY, d_res = randn(rng, 1.0, T, d), randn(rng, 1.0, T, d)
    res, d_res = (res, d_res) if residual else (None, None)
    offs = [0, 40, 40, 97, T][:n] + [T]
    valid = torch.from_numpy((rng.random(T) < 0.8).astype(np.uint8)) if padded else None
    g = torch.full((1,), 1.7, device="cuda")
    y = layer.forward(x, bias, residual=res, valid=None if valid is None else valid.cuda(),
                      seq_offsets=torch.tensor(offs, dtype=torch.int32, device="cuda") if n > 1 else None)
    dX = layer.backward(dY, d_balance=g, d_residual=d_res)
    ok()
    want = autograd(layer, w, layer.residual, dY, d_res, alpha, 1.7, softmax, offs if n > 1 else [0, T], valid)
    near(y, want["y"], 1e-2, "y")
    loss = float(want["loss"].detach())
    assert abs(float(layer.balance_loss) - loss) <= 4e-3 * loss
    near(dX, want["dX"], 1e-2, "dX")
    for name in ("dnorm", "dW_g", "dW13", "dW2"):
        near(getattr(layer, name), want[name], 1e-2, name)


def test_mx_training_step_with_norm_and_balance():
    """The MXFP8 layer's gradients are off by its quantisation: against the bf16 layer's within
    three roundings of q = 0.028 in each of two factors."""
    T, d, E, k, I = 200, 512, 8, 2, 256
    rng = np.random.default_rng(3)
    dY = randn(rng, 1.0, T, d)
    got = {}
    for mx in (False, True):
        layer, w, bias, x, res = block(T, d, E, k, I, backward=True, balance=50.0, mx=mx)
        layer.forward(x, bias, residual=res)
        layer.backward(dY)
        ok()
        got[mx] = {n: f64(getattr(layer, n)) for n in ("dX", "dnorm", "dW_g", "dW13", "dW2")}
        ids = layer.ids.clone()
        got.setdefault("ids", ids)
    assert torch.equal(got["ids"], ids)
    for name, v in got[False].items():
        assert rel(got[True][name], v) <= 0.12, name


def test_step_in_graphs_and_streams():
    """The whole step captured: replays give the eager step's bits, also after other inputs, in
    two graphs that share the layer's buffers, and on another stream."""
    T, d, E, k, I = 96, 256, 32, 4, 128
    layer, w, bias, x, res = block(T, d, E, k, I, backward=True, balance=1.0, sequences=2)
    offs = torch.tensor([0, 50, T], dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(1)
    dY, d_res = randn(rng, 1.0, T, d), randn(rng, 1.0, T, d)
    other = randn(rng, 1.0, T, d)
    names = ("y", "dX", "dnorm", "dW_g", "dW13", "dW2", "balance_loss", "balance_counts", "residual")

    def step(x, stream=None):
        layer.forward(x, bias, residual=res, seq_offsets=offs, stream=stream)
        layer.backward(dY, d_residual=d_res, stream=stream)
    kept = lambda: [getattr(layer, n).clone() for n in names]
    step(x)
    first = kept()
    step(other)
    second = kept()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for inp in (x, other):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                step(inp)
            graphs.append(g)
        for i in (0, 1, 0, 0, 1):
            for n in names:
                getattr(layer, n).zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            for n, a, b in zip(names, kept(), (first, second)[i]):
                assert torch.equal(a, b), n
    step(x, stream=side)
    torch.cuda.synchronize()
    for n, a, b in zip(names, kept(), first):
        assert torch.equal(a, b), n
    ok()


def test_tensors_of_another_device_are_refused(monkeypatch):
    """Refused by the binding, ahead of any launch (the tensors are on device 0)."""
    x, w = torch.ones(4, 128, dtype=torch.bfloat16, device="cuda"), torch.ones(128, device="cuda")
    y = torch.empty_like(x)
    q, sf = (torch.empty(4, c, dtype=torch.uint8, device="cuda") for c in (64, 16))
    monkeypatch.setattr(_lib, "_get_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        _lib.moe_rmsnorm(dict(T=4, d=128, eps=1e-6, x=x, weight=w, y=y))
    with pytest.raises(ValueError, match="current device"):
        _lib.moe_mx4_quantize(x, 4, 128, q, sf)


@pytest.mark.parametrize("kind", ["bf16", "mx4", "fp8"])
def test_balance_without_a_backward(kind):
    T, d, E, k, I = 70, 256, 32, 4, 128
    kw = {} if kind == "bf16" else {kind: True}
    layer, w, bias, x, res = block(T, d, E, k, I, balance=0.5, **kw)
    layer.forward(x, bias, residual=res)
    ok()
    s = 1 / (1 + np.exp(-f64(layer.logits)[:T]))
    counts = np.bincount(layer.ids.cpu().numpy().ravel(), minlength=E)
    assert np.array_equal(layer.balance_counts.cpu().numpy()[0], counts)
    want = 0.5 * (E * counts / (k * T)) @ (s / s.sum(1, keepdims=True)).mean(0)
    # 2^-16: what an exponential of these logits, a sum of 32 and a mean of 70 can be off by, and more
    assert abs(f64(layer.balance_loss)[0] - want) <= 2.0 ** -16 * want
    with pytest.raises(RuntimeError):
        layer.backward(x)
