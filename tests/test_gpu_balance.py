"""The balance loss, the experts' load and the gradient at the logits against their
definition in 64 bits.

Roundings: an exponential is off by at most 2^-21 (1 + |z| / 4) of itself (the fast one:
2 units of its result and the rounding of its argument), a score by that and two units; the
sum over E scores by at most 20 additions in a row (lanes in pairs, then a lane's own); so
a share p is off by at most B = 2^-20 (2 + max|z| / 4) of itself, and the mean over N tokens,
summed in chunks, by (N / 8 + 700) 2^-24 more at most."""
import numpy as np
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib
from tests.test_gpu_fp8 import f64, ok

pytestmark = pytest.mark.gpu

SIG, SOFT = _lib.MOE_SCORE_SIGMOID, _lib.MOE_SCORE_SOFTMAX
ALPHA = 0.01


def dev(a, t=None):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to("cuda", t)


def call(z, ids, score, offsets=None, valid=None, dloss=None, backward=True, ws_fill=255):
    T, E = z.shape
    k = ids.shape[1]
    n = 1 if offsets is None else len(offsets) - 1
    mk = lambda *s, t=torch.float32: torch.full(s, -5, dtype=t, device="cuda")
    a = dict(T=T, E=E, k=k, n_seq=n, score=score, alpha=ALPHA, logits=dev(z, torch.float32),
             ids=dev(ids, torch.int32), seq_offsets=dev(offsets, torch.int32),
             valid=dev(valid, torch.uint8), counts=mk(n, E, t=torch.int32),
             tokens=mk(n, t=torch.int32), load=mk(n, E), seq_loss=mk(n), loss=mk(1),
             dloss=dev(dloss, torch.float32), dlogits=mk(T, E),
             ws=torch.full((_lib.moe_balance_workspace_size(T, E, n),), ws_fill, dtype=torch.uint8,
                           device="cuda"))
    _lib.moe_balance_loss(a)
    if backward:
        _lib.moe_balance_loss_backward(a)
    return a


def shares(z, score):
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if score == SIG:
            s = 1 / (1 + np.exp(-z))
            slope = 1 / (1 + np.exp(z))
        else:
            top = z.max(1, keepdims=True)
            s = np.exp(z - np.where(np.isneginf(top), 0.0, top))
            slope = np.ones_like(z)
        tot = s.sum(1, keepdims=True)
        return np.where(tot > 0, s / tot, 0.0), slope


def reference(z, ids, score, offsets=None, valid=None, dloss=1.0):
    T, E = z.shape
    k = ids.shape[1]
    offs = [0, T] if offsets is None else offsets
    n = len(offs) - 1
    ok_t = np.ones(T, bool) if valid is None else valid != 0
    p, slope = shares(z, score)
    counts, tokens = np.zeros((n, E), int), np.zeros(n, int)
    load, seq = np.zeros((n, E)), np.zeros(n)
    dz = np.zeros((T, E))
    for q in range(n):
        t = np.arange(offs[q], offs[q + 1])
        t = t[ok_t[t]]
        tokens[q] = len(t)
        if not len(t):
            continue
        counts[q] = np.bincount(ids[t].ravel(), minlength=E)
        load[q] = E * counts[q] / (k * len(t))
        seq[q] = load[q] @ p[t].mean(0)
        dz[t] = (dloss * ALPHA / (n * len(t)) * p[t] * slope[t]
                 * (load[q] - (p[t] @ load[q])[:, None]))
    mag = np.zeros((T, E))
    for q in range(n):
        t = np.arange(offs[q], offs[q + 1])
        mag[t] = (dloss * ALPHA / (n * max(tokens[q], 1)) * p[t] * slope[t]
                  * (load[q] + (p[t] @ load[q])[:, None])) * ok_t[t, None]
    return dict(counts=counts, tokens=tokens, load=load, seq_loss=seq, loss=ALPHA * seq.sum() / n,
                dlogits=dz, mag=mag)


def check(a, r, z):
    finite = np.abs(z[np.isfinite(z)])
    B = 2.0 ** -20 * (2 + (finite.max() if finite.size else 0.0) / 4)
    assert np.array_equal(a["counts"].cpu().numpy(), r["counts"])
    assert np.array_equal(a["tokens"].cpu().numpy(), r["tokens"])
    assert np.allclose(f64(a["load"]), r["load"], rtol=2.0 ** -22, atol=0)
    lim = B + (r["tokens"] / 8 + 700) * 2.0 ** -24
    assert (np.abs(f64(a["seq_loss"]) - r["seq_loss"]) <= lim * r["seq_loss"]).all()
    assert abs(f64(a["loss"])[0] - r["loss"]) <= (lim.max() + 2.0 ** -22) * r["loss"] + 1e-30
    got = f64(a["dlogits"])
    assert (np.abs(got - r["dlogits"]) <= 4 * B * r["mag"] + 1e-37).all()


def inputs(rng, T, E, k):
    z = (rng.standard_normal((T, E)) * 1.3 + rng.standard_normal(E) * 0.5).astype(np.float32)
    ids = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
    return z, ids


SHAPES = [(1, 1, 1), (1, 16, 2), (3, 4, 4), (64, 16, 2), (40, 97, 5), (333, 128, 8), (100, 130, 3),
          (70, 257, 6), (513, 384, 6), (50, 512, 8), (30, 1024, 32), (25, 1023, 7), (9000, 20, 2),
          (129, 33, 1), (20, 700, 4)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("score", [SIG, SOFT])
def test_one_sequence(T, E, k, score):
    rng = np.random.default_rng(T + E)
    z, ids = inputs(rng, T, E, k)
    a = call(z, ids, score, dloss=np.array([0.7], np.float32))
    ok()
    check(a, reference(z.astype(np.float64), ids, score, dloss=float(np.float32(0.7))), z)


@pytest.mark.parametrize("T,E,k,n", [(100, 16, 2, 7), (2500, 96, 4, 40), (64, 33, 3, 64), (5, 8, 2, 9),
                                     (3000, 384, 6, 3)])
@pytest.mark.parametrize("score", [SIG, SOFT])
def test_sequences_and_padding(T, E, k, n, score):
    """Ragged sequences, empty ones, padding, one with nothing but padding; tokens in front of
    the first sequence and behind the last."""
    rng = np.random.default_rng(T + n)
    z, ids = inputs(rng, T, E, k)
    offs = np.sort(rng.integers(T // 20, T + 1 - T // 20, n + 1)).astype(np.int32)
    offs[1] = offs[2] if n > 2 else offs[1]
    valid = (rng.random(T) < 0.8).astype(np.uint8)
    valid[offs[0]:offs[1]] = 0
    a = call(z, ids, score, offs, valid)
    ok()
    check(a, reference(z.astype(np.float64), ids, score, offs, valid), z)


@pytest.mark.parametrize("score", [SIG, SOFT])
def test_masked_and_extreme_logits(score):
    """Experts at minus infinity or the lowest value, a token with nothing left, logits far
    out on both sides."""
    rng = np.random.default_rng(9)
    T, E, k = 60, 40, 4
    z, ids = inputs(rng, T, E, k)
    z[:, 7] = -np.inf
    z[:, 8] = np.finfo(np.float32).min
    z[5] = -np.inf
    z[6] = np.finfo(np.float32).min
    z[7, :20] = 80.0
    z[8, 3] = -80.0
    z[9] = -90.0
    a = call(z, ids, score)
    ok()
    r = reference(z.astype(np.float64), ids, score)
    assert np.isfinite(f64(a["dlogits"])).all() and np.isfinite(f64(a["loss"])).all()
    # (the lowest value is no argument of an exponential's error: shares there are 0 or equal;
    # a sigmoid below fp32's normal range, at -90, keeps few bits, but its share is 1 / E)
    z = np.where(np.abs(z) > 1e30, 0.0, z)
    for n in ("counts", "tokens"):
        assert np.array_equal(a[n].cpu().numpy(), r[n])
    rows = np.delete(np.arange(T), [5, 6, 9])
    got = f64(a["dlogits"])
    B = 2.0 ** -20 * (2 + 90 / 4)
    assert (np.abs(got - r["dlogits"])[rows] <= 4 * B * r["mag"][rows] + 1e-37).all()
    assert (got[5] == 0).all()
    assert abs(f64(a["loss"])[0] - r["loss"]) <= 0.05 * r["loss"]


def test_nan_is_kept():
    z, ids = inputs(np.random.default_rng(1), 20, 16, 2)
    z[3, 4] = np.nan
    for score in (SIG, SOFT):
        a = call(z, ids, score)
        ok()
        g = np.isnan(f64(a["dlogits"]))
        assert np.isnan(f64(a["loss"])[0]) and g[3].all() and not np.delete(g, 3, 0).any()


def test_gradient_against_differences():
    """The load held fixed, the loss's slope along random directions of the logits."""
    rng = np.random.default_rng(4)
    T, E, k = 30, 12, 3
    z, ids = inputs(rng, T, E, k)
    offs, valid = np.array([0, 11, 30], np.int32), (rng.random(T) < 0.9).astype(np.uint8)
    for score in (SIG, SOFT):
        a = call(z, ids, score, offs, valid)
        ok()

        def loss(z):
            return reference(z, ids, score, offs, valid)["loss"]
        z64, h = z.astype(np.float64), 1e-5
        for i in range(5):
            d = rng.standard_normal((T, E))
            num = (loss(z64 + h * d) - loss(z64 - h * d)) / (2 * h)
            got = (f64(a["dlogits"]) * d).sum()
            assert abs(got - num) <= 1e-5 * np.abs(f64(a["dlogits"]) * d).sum() + 1e-11


def test_no_tokens():
    z, ids = np.zeros((0, 16), np.float32), np.zeros((0, 2), np.int32)
    a = call(z, ids, SIG, np.zeros(4, np.int32))
    ok()
    assert f64(a["loss"])[0] == 0 and (a["counts"] == 0).all() and (a["tokens"] == 0).all()
    assert (f64(a["seq_loss"]) == 0).all() and (f64(a["load"]) == 0).all()


def test_bad_ids_and_offsets_are_recorded():
    rng = np.random.default_rng(2)
    z, ids = inputs(rng, 50, 16, 2)
    bad = ids.copy()
    bad[3, 1], bad[9, 0] = 16, -1
    a = call(z, bad, SIG)
    torch.cuda.synchronize()
    assert _lib.moe_last_device_status() == _lib.MOE_ERR_INVALID_ARG
    assert int(a["counts"].sum()) == 98
    for offs in ([0, 30, 20, 50], [0, 10, 400], [-7, 10, 50]):
        a = call(z, ids, SIG, np.array(offs, np.int32))
        torch.cuda.synchronize()
        assert _lib.moe_last_device_status() == _lib.MOE_ERR_INVALID_ARG
    # offsets that leave the tokens are cut to them
    assert a["tokens"].tolist() == [10, 40]


def test_same_bits_every_time():
    rng = np.random.default_rng(8)
    z, ids = inputs(rng, 5000, 384, 6)
    offs = np.array([0, 700, 701, 5000], np.int32)
    a, b = call(z, ids, SIG, offs, ws_fill=0), call(z, ids, SIG, offs, ws_fill=77)
    ok()
    for n in ("loss", "seq_loss", "load", "counts", "dlogits"):
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("score", [SIG, SOFT])
def test_most_sequences(score):
    """As many sequences as a call takes, of a token or none, some of two."""
    T, E, k, n = 70000, 8, 2, 65535
    rng = np.random.default_rng(9)
    z, ids = inputs(rng, T, E, k)
    offs = np.sort(np.concatenate([[0, T], rng.integers(0, T + 1, n - 1)])).astype(np.int32)
    a = call(z, ids, score, offs)
    ok()
    check(a, reference(z.astype(np.float64), ids, score, offs), z)


def test_places_behind_32_bits():
    """More than 2^31 logits, of which the last 70 tokens count; the gradient in their place."""
    T, E, k, m = (1 << 21) + 70, 1024, 2, 70
    z, ids = inputs(np.random.default_rng(4), m, E, k)
    logits = torch.ones(T, E, device="cuda")
    logits[-m:] = dev(z)
    all_ids, valid = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(
        T, dtype=torch.uint8, device="cuda")
    all_ids[-m:], valid[-m:] = dev(ids), 1
    f = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")
    a = dict(T=T, E=E, k=k, n_seq=1, score=SIG, alpha=ALPHA, logits=logits, ids=all_ids, valid=valid,
             counts=f(1, E, t=torch.int32), tokens=f(1, t=torch.int32), load=f(1, E), seq_loss=f(1),
             loss=f(1), dlogits=logits,
             ws=f(_lib.moe_balance_workspace_size(T, E), t=torch.uint8))
    _lib.moe_balance_loss(a)
    _lib.moe_balance_loss_backward(a)
    ok()
    for part in (logits[:5000], logits[T // 2:T // 2 + 5000], logits[-m - 5000:-m]):
        assert not part.any()
    check(dict(a, dlogits=logits[-m:]), reference(z.astype(np.float64), ids, SIG), z)


def test_one_workspace_in_a_graph():
    """Captured and replayed on a workspace that calls of other sizes have used."""
    rng = np.random.default_rng(6)
    z, ids = inputs(rng, 3000, 40, 4)
    offs = np.array([0, 10, 1700, 1700, 2990], np.int32)
    a = call(z, ids, SIG, offs, backward=False)
    r = reference(z.astype(np.float64), ids, SIG, offs)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for _ in range(2):
                _lib.moe_balance_loss(a)
                _lib.moe_balance_loss_backward(a)
        for fill in (0, 255, 77):
            a["ws"].fill_(fill)
            a["loss"].fill_(-1.0)
            a["dlogits"].fill_(-1.0)
            g.replay()
            st.synchronize()
            check(a, r, z)
    ok()
