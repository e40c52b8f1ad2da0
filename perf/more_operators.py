"""Cases of the operators around the expert layer: what feeds it, what balances
it, and its products with 4-bit weights.

  norm      the residual's addition and the root-mean-square norm ahead of the
            layer, its rows also quantised as the expert matmuls read them (FP8
            with a scale for each 128, MXFP8); and its backward
  balance   the sequence-wise balance loss of the router with the load of each
            expert, and its gradient at the gate's logits (a training step: both)
  mx4       MXFP4 (E2M1 elements, one power-of-two scale per 32): weights
            quantised and expanded again, token rows quantised (to 4 bits, or to
            8 as MXFP8) and multiplied with each group's weight, and the expert
            FFN with 4-bit weights on MXFP8 rows

`own` chooses between the plain form (elementary torch operations) and the
library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

FP8_BLOCK, MX_BLOCK = 128, 32
FP8_MAX, FP8_FLOOR = 448.0, 2.0 ** -100
EPS = 1e-6
CLAMP = 7.0
ALPHA = 1e-3
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one user decoding: the row in front of the layer, for its FP8 experts
        dict(name="norm_one", op="norm", what="fwd", T=1, d=4096, residual=True, rows="fp8"),
        # a prompt of an odd length on a narrow model, first layer (no residual yet)
        dict(name="norm_ragged_mx", op="norm", what="fwd", T=777, d=1184, residual=False,
             rows="mx"),
        # a prefill chunk
        dict(name="norm_prefill", op="norm", what="fwd", T=4096, d=4096, residual=True,
             rows="fp8"),
        # a training step's backward, with the gradient that passes the layer by
        dict(name="norm_backward", op="norm", what="bwd", T=16384, d=4096, residual=True,
             rows="none"),
        # a small layer's step
        dict(name="balance_small", op="balance", T=64, E=16, k=2, seqs=1, score="sigmoid",
             padded=False, masked=False),
        # packed sequences with padding, experts that are switched off, softmax scores
        dict(name="balance_ragged", op="balance", T=4097, E=97, k=5, seqs=37, score="softmax",
             padded=True, masked=True),
        # the training slice: 64K tokens of 16 sequences
        dict(name="balance_long", op="balance", T=65536, E=384, k=6, seqs=16, score="sigmoid",
             padded=True, masked=False),
        # weights after an optimizer step, and the values that the products will see
        dict(name="mx4_weights", op="mx4", what="weights", rows=9 * 4096, K=4096),
        # a dense projection of one token
        dict(name="mx4_project_one", op="mx4", what="project", G=1, R=1, N=4096, K=4096, bits=4),
        # expert rows of uneven counts (one expert empty, one with a single row)
        dict(name="mx4_project_ragged", op="mx4", what="project", G=33, R=12345, N=4096, K=2048,
             bits=4),
        # a short prefill over a few local experts
        dict(name="mx4_ffn_short", op="mx4", what="ffn", G=9, R=777, d=4096, I=2048),
        # a long prefill: about a thousand rows per expert
        dict(name="mx4_ffn_long", op="mx4", what="ffn", G=33, R=32768, d=4096, I=2048),
    ]


def _log(rng, lo, hi):
    """A whole number, its logarithm spread evenly over [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "balance", "mx4", "mx4", "mx4"])
    if op == "norm":
        what = rng.choice(["fwd", "fwd", "bwd"])
        rows = "none" if what == "bwd" else rng.choice(["fp8", "mx", "none"])
        return dict(op=op, what=what, T=_log(rng, 1, 16384), d=32 * rng.randint(1, 128),
                    residual=rng.random() < 0.7, rows=rows)
    if op == "balance":
        E = _log(rng, 8, 384)
        T = _log(rng, 1, 65536)
        return dict(op=op, T=T, E=E, k=rng.randint(1, 8), seqs=_log(rng, 1, 64),
                    score=rng.choice(["sigmoid", "softmax"]), padded=rng.random() < 0.5,
                    masked=rng.random() < 0.3)
    what = rng.choice(["weights", "project", "project", "ffn"])
    if what == "weights":
        return dict(op=op, what=what, rows=_log(rng, 1, 36864), K=32 * rng.randint(1, 128))
    if what == "project":
        bits = rng.choice([4, 8])
        K = 32 * _log(rng, 1, 128) if bits == 4 else 128 * _log(rng, 1, 32)
        return dict(op=op, what=what, G=_log(rng, 1, 33), R=_log(rng, 1, 12345),
                    N=8 * _log(rng, 1, 512), K=K, bits=bits)
    return dict(op=op, what=what, G=_log(rng, 1, 33), R=_log(rng, 1, 16384),
                d=128 * rng.randint(1, 32), I=128 * rng.randint(1, 16))


def _counts(R, G):
    """Rows of each group: uneven, one group empty and one with a single row
    where there are groups enough.  Fixed by (R, G)."""
    r = random.Random(R * 1000003 + G)
    w = [r.random() ** 2 + 0.05 for _ in range(G)]
    if G >= 4:
        w[r.randrange(G)] = 0.0
    c = [int(R * v / sum(w)) for v in w]
    if G >= 4 and R > G:
        c[min(range(G), key=lambda g: (c[g] == 0, c[g]))] = 1
    c[max(range(G), key=lambda g: c[g])] += R - sum(c)
    return c


# ----------------------------------------------------------------- inputs

def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed((seed * 1009 + salt) & 0x7FFFFFFF)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _activations(g, T, d):
    """Every token at its own scale, a few channels far larger."""
    x = _randn(g, T, d) * torch.exp(0.5 * _randn(g, T, 1))
    x *= torch.where(torch.rand(d, generator=g, device="cuda") < 0.01, 20.0, 1.0).to(x.dtype)
    return x


def _e2m1_bytes(g, rows, K):
    """Codes of normal values, two a byte, the even element in the low nibble."""
    out = torch.empty(rows, K // 2, dtype=torch.uint8, device="cuda")
    cut = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    for r in range(0, rows, 16384):
        v = _randn(g, min(16384, rows - r), K).float() * 2.0
        c = torch.bucketize(v.abs(), cut).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
        out[r:r + c.shape[0]] = c[:, 0::2] | (c[:, 1::2] << 4)
    return out


def _e4m3_bytes(g, rows, K):
    return (_randn(g, rows, K) * 64.0).clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(
        torch.uint8)


def _pitch(K):
    """Bytes of a row of scales: one for each 32 elements, padded to 16."""
    return (K // MX_BLOCK + 15) // 16 * 16


def _e8m0(g, rows, K, exponent):
    """Scale codes 2^(exponent - 1), 2^exponent or 2^(exponent + 1); zeros behind the row."""
    sf = torch.zeros(rows, _pitch(K), dtype=torch.uint8, device="cuda")
    sf[:, :K // MX_BLOCK] = torch.randint(126 + exponent, 129 + exponent, (rows, K // MX_BLOCK),
                                          generator=g, dtype=torch.uint8, device="cuda")
    return sf


def _weights4(g, rows, K):
    """Values of about the size 1.28 / sqrt(K)."""
    return _e2m1_bytes(g, rows, K), _e8m0(g, rows, K, round(math.log2(0.64 / math.sqrt(K))))


def _rows_plan(case):
    c = _counts(case["R"], case["G"])
    offs = np.concatenate([[0], np.cumsum(c)]).astype(np.int32)
    grp = np.repeat(np.arange(case["G"]), c)
    pos = np.arange(case["R"]) - offs[grp]
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return dict(offsets=dev(offs), grp=dev(grp.astype(np.int64)), pos=dev(pos.astype(np.int64)),
                most=max(c))


def _row_bytes(K, bits):
    return K if bits == 8 else K // 2


def prepare(case, seed):
    g = _gen(seed, 7)
    c = case
    dev = dict(device="cuda")
    bf, f32, u8 = (dict(dtype=t, **dev) for t in (torch.bfloat16, torch.float32, torch.uint8))
    s = dict(case=dict(case))
    if c["op"] == "norm":
        T, d = c["T"], c["d"]
        s["weight"] = 1.0 + 0.2 * torch.randn(d, generator=g, **dev)
        s["x"] = _activations(g, T, d)
        s["residual"] = _activations(g, T, d) if c["residual"] else None
        if c["what"] == "fwd":
            s["residual_out"] = torch.empty(T, d, **bf) if c["residual"] else None
            s["y"] = torch.empty(T, d, **bf)
            s["rstd"] = torch.empty(T, **f32)
            if c["rows"] == "fp8":
                s["q"] = torch.empty(T, d, **u8)
                s["s"] = torch.empty(T, -(-d // FP8_BLOCK), **f32)
            elif c["rows"] == "mx":
                s["q"] = torch.empty(T, d, **u8)
                s["s"] = torch.zeros(T, _pitch(d), **u8)     # the bytes behind a row stay
        else:
            s["rstd"] = 1 / torch.sqrt(s["x"].float().square().mean(1) + EPS)
            s["dy"] = _randn(g, T, d)
            s["d_residual"] = _randn(g, T, d) if c["residual"] else None
            s["dx"] = torch.empty(T, d, **bf)
            s["d_weight"] = torch.empty(d, **f32)
    elif c["op"] == "balance":
        T, E, n = c["T"], c["E"], c["seqs"]
        k = min(c["k"], E)
        z = torch.randn(T, E, generator=g, **dev) * 1.28
        z += 0.5 * torch.randn(E, generator=g, **dev)          # some experts are favoured
        if c["masked"]:                                        # experts that are switched off
            off = torch.randperm(E, generator=g, **dev)[:max(0, min(E // 8, E - k))]
            z[:, off] = -math.inf
        s["logits"] = z
        s["ids"] = z.topk(k, dim=1).indices.int()
        cut = torch.sort(torch.randint(0, T + 1, (n - 1,), generator=g, **dev)).values
        s["seq_offsets"] = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), T)]).int()
        s["valid"] = ((torch.rand(T, generator=g, **dev) < 0.9).to(torch.uint8)
                      if c["padded"] else None)
        s["dloss"] = torch.rand(1, generator=g, **dev) + 0.5
        s["counts"] = torch.empty(n, E, dtype=torch.int32, **dev)
        s["tokens"] = torch.empty(n, dtype=torch.int32, **dev)
        s["load"] = torch.empty(n, E, **f32)
        s["seq_loss"] = torch.empty(n, **f32)
        s["loss"] = torch.empty(1, **f32)
        s["dlogits"] = torch.empty(T, E, **f32)
    elif c["what"] == "weights":
        rows, K = c["rows"], c["K"]
        s["w"] = _randn(g, rows, K) * 0.02
        s["q"] = torch.empty(rows, K // 2, **u8)
        s["sf"] = torch.empty(rows, _pitch(K), **u8)
        s["out"] = torch.empty(rows, K, **bf)
    elif c["what"] == "project":
        R, G, N, K, bits = (c[n] for n in ("R", "G", "N", "K", "bits"))
        s.update(_rows_plan(c))
        s["x"] = _activations(g, R, K)
        s["b_q"], s["b_sf"] = _weights4(g, G * N, K)
        s["a_q"] = torch.empty(R, _row_bytes(K, bits), **u8)
        s["a_sf"] = torch.empty(R, _pitch(K), **u8)
        s["out"] = torch.empty(R, N, **bf)
    else:
        R, G, d, I = (c[n] for n in ("R", "G", "d", "I"))
        s.update(_rows_plan(c))
        s["x_q"], s["x_sf"] = _e4m3_bytes(g, R, d), _e8m0(g, R, d, -6)
        s["W13_q"], s["W13_sf"] = _weights4(g, G * 2 * I, d)
        s["W2_q"], s["W2_sf"] = _weights4(g, G * d, I)
        s["row_weight"] = torch.rand(R, generator=g, **dev) + 0.1
        s["h_q"] = torch.empty(R, I, **u8)
        s["h_sf"] = torch.empty(R, _pitch(I), **u8)
        s["y"] = torch.empty(R, d, **bf)
    return s


# ------------------------------------------------------------------- runs

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _typed(s, rows):
    """The quantised rows as the values that their bytes stand for."""
    q = s["q"].view(torch.float8_e4m3fn)
    return dict(q=q, s=s["s"] if rows == "fp8" else s["s"].view(torch.float8_e8m0fnu))


def _run_own(s):
    from moe_expert_layer_04_gb300 import _lib
    c = s["case"]
    if c["op"] == "norm" and c["what"] == "fwd":
        fmt = dict(none=_lib.MOE_ROWS_NONE, fp8=_lib.MOE_ROWS_FP8, mx=_lib.MOE_ROWS_MXFP8)
        _lib.moe_rmsnorm(dict(
            T=c["T"], d=c["d"], eps=EPS, format=fmt[c["rows"]], x=s["x"], residual=s["residual"],
            weight=s["weight"], residual_out=s["residual_out"], y=s["y"], rstd=s["rstd"],
            q=s.get("q"), scales=s.get("s")))
        out = dict(y=s["y"], rstd=s["rstd"], residual=s["residual_out"])
        return out if c["rows"] == "none" else dict(out, **_typed(s, c["rows"]))
    if c["op"] == "norm":
        if "ws" not in s:      # kept by the program
            s["ws"] = torch.empty(_lib.moe_rmsnorm_bwd_workspace_size(c["T"], c["d"]),
                                  dtype=torch.uint8, device="cuda")
        _lib.moe_rmsnorm_backward(dict(
            T=c["T"], d=c["d"], x=s["x"], weight=s["weight"], rstd=s["rstd"], dy=s["dy"],
            d_residual=s["d_residual"], dx=s["dx"], d_weight=s["d_weight"], ws=s["ws"]))
        return dict(dx=s["dx"], d_weight=s["d_weight"])
    if c["op"] == "balance":
        T, E, n = c["T"], c["E"], c["seqs"]
        k = min(c["k"], E)
        if "ws" not in s:
            s["ws"] = torch.empty(_lib.moe_balance_workspace_size(T, E, n), dtype=torch.uint8,
                                  device="cuda")
        score = dict(sigmoid=_lib.MOE_SCORE_SIGMOID, softmax=_lib.MOE_SCORE_SOFTMAX)[c["score"]]
        args = dict(T=T, E=E, k=k, n_seq=n, score=score, alpha=ALPHA, logits=s["logits"],
                    ids=s["ids"], seq_offsets=s["seq_offsets"], valid=s["valid"],
                    counts=s["counts"], tokens=s["tokens"], load=s["load"],
                    seq_loss=s["seq_loss"], loss=s["loss"], dloss=s["dloss"],
                    dlogits=s["dlogits"], ws=s["ws"])
        _lib.moe_balance_loss(args)
        _lib.moe_balance_loss_backward(args)
        return dict(loss=s["loss"], seq_loss=s["seq_loss"], counts=s["counts"],
                    dlogits=s["dlogits"])
    if c["what"] == "weights":
        _lib.moe_mx4_quantize(s["w"], c["rows"], c["K"], s["q"], s["sf"])
        _lib.moe_mx4_dequantize(s["q"], s["sf"], c["rows"], c["K"], s["out"])
        return s["out"]
    if c["what"] == "project":
        quantize = _lib.moe_mx4_quantize if c["bits"] == 4 else _lib.moe_mx_quantize
        quantize(s["x"], c["R"], c["K"], s["a_q"], s["a_sf"])
        _lib.moe_mx4_matmul(s["a_q"], s["a_sf"], c["bits"], s["offsets"], c["G"], c["R"],
                            s["b_q"], s["b_sf"], None, 0, c["N"], c["K"], s["out"])
        return s["out"]
    _lib.moe_expert_ffn_mx4(s["x_q"], s["x_sf"], s["offsets"], c["G"], c["R"], s["W13_q"],
                            s["W13_sf"], s["W2_q"], s["W2_sf"], s["row_weight"], c["R"], c["d"],
                            c["I"], CLAMP, s["h_q"], s["h_sf"], s["y"])
    return s["y"]


def _blocks(v, n):
    """[..., K] -> [..., ceil(K/n), n], zeros behind the row."""
    return torch.nn.functional.pad(v, (0, -v.shape[-1] % n)).unflatten(-1, (-1, n))


def _exponent(amax):
    """floor(log2) of positive numbers."""
    return torch.frexp(amax).exponent - 1


def _power(e):
    """2^e for whole e (below 2^-126 too), by its bits: a power function may be off."""
    return ((e.long() + 1023) << 52).view(torch.float64).float()


def _mx(v, top):
    """Blocks [..., 32] -> (E8M0 codes [..., 1], v / X): top is the exponent of the
    format's largest element."""
    amax = v.abs().amax(-1, keepdim=True)
    e = (_exponent(amax) - top).clamp(-127, 127)
    code = torch.where(amax > 0, e + 127, torch.zeros_like(e))
    return code, v * _power(torch.where(amax > 0, -e, torch.zeros_like(e)))


def _e2m1(v):
    """Nearest E2M1 value, ties to the even code, saturated at 6."""
    a = v.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int()
            + (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int())
    return torch.copysign(torch.tensor(E2M1, device=v.device)[code], v)


def _through_mx(v, bits):
    """fp32 rows [..., K] -> the values of their quantised form."""
    b = v.unflatten(-1, (-1, MX_BLOCK))
    code, u = _mx(b, 2 if bits == 4 else 8)
    q = _e2m1(u) if bits == 4 else u.clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).float()
    return (q * _power(code - 127)).flatten(-2)


def _expand(q, sf, K, bits):
    """Codes and scales of rows -> their values in fp32."""
    if bits == 8:
        v = q.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=q.device)
        v = torch.stack([table[(q & 15).int()], table[(q >> 4).int()]], -1).flatten(-2)
    x = _power(sf[..., :K // MX_BLOCK].int() - 127)
    return (v.unflatten(-1, (-1, MX_BLOCK)) * x.unsqueeze(-1)).flatten(-2)


def _grouped(s, v, G, most):
    """Rows of all groups -> [G, most, ...], zeros behind each group's rows."""
    out = torch.zeros(G, most, v.shape[1], dtype=v.dtype, device=v.device)
    out[s["grp"], s["pos"]] = v
    return out


def _scores(z, score):
    """The gate's scores and their shares of each token, a token without any: zeros."""
    if score == "sigmoid":
        sc = 1 / (1 + torch.exp(-z))
        total = sc.sum(1, keepdim=True)
        return sc, torch.where(total > 0, sc / total, torch.zeros_like(sc))
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(1, keepdim=True)
    return None, torch.where(total > 0, e / total, torch.zeros_like(e))


def _run_plain(s):
    c = s["case"]
    if c["op"] == "norm" and c["what"] == "fwd":
        v = s["x"]
        if c["residual"]:
            v = (v.float() + s["residual"].float()).bfloat16()
        f = v.float()
        rstd = 1 / torch.sqrt(f.square().mean(1) + EPS)
        y = f * rstd[:, None] * s["weight"]
        out = dict(y=y.bfloat16(), rstd=rstd, residual=v if c["residual"] else None)
        if c["rows"] == "fp8":
            b = _blocks(y, FP8_BLOCK)
            amax = b.abs().amax(-1, keepdim=True).clamp_min(FP8_FLOOR)
            top = torch.full_like(amax, FP8_MAX)
            q = (b * (top / amax)).to(torch.float8_e4m3fn).flatten(-2)[:, :c["d"]].contiguous()
            out.update(q=q, s=(amax / top).squeeze(-1))
        elif c["rows"] == "mx":
            code, u = _mx(_blocks(y, MX_BLOCK), 8)
            q = u.clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).flatten(-2)
            sf = torch.nn.functional.pad(code.squeeze(-1).to(torch.uint8),
                                         (0, _pitch(c["d"]) - c["d"] // MX_BLOCK))
            out.update(q=q, s=sf.view(torch.float8_e8m0fnu))
        return out
    if c["op"] == "norm":
        vh = s["x"].float() * s["rstd"][:, None]
        dy = s["dy"].float()
        wdy = dy * s["weight"]
        dx = s["rstd"][:, None] * (wdy - vh * (wdy * vh).mean(1, keepdim=True))
        if c["residual"]:
            dx = dx + s["d_residual"].float()
        return dict(dx=dx.bfloat16(), d_weight=(dy * vh).double().sum(0).float())
    if c["op"] == "balance":
        T, E, n = c["T"], c["E"], c["seqs"]
        k = min(c["k"], E)
        seq = torch.searchsorted(s["seq_offsets"], torch.arange(T, device="cuda").int(),
                                 right=True) - 1
        ok = torch.ones(T, device="cuda") if s["valid"] is None else s["valid"].float()
        sc, p = _scores(s["logits"], c["score"])
        zero = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")
        tokens = zero(n).index_add_(0, seq, ok.double())
        per = tokens.clamp_min(1.0)
        counts = zero(n * E).index_add_(0, (seq[:, None] * E + s["ids"]).flatten(),
                                        ok.double().repeat_interleave(k)).view(n, E)
        load = (counts * E / (k * per[:, None])).float()
        mean = zero(n, E).index_add_(0, seq, (p * ok[:, None]).double()) / per[:, None]
        seq_loss = (load * mean).sum(1)
        f = load[seq]
        dz = p * (f - (f * p).sum(1, keepdim=True))
        if c["score"] == "sigmoid":
            dz = dz * (1 - sc)
        dz = dz * (ok * (s["dloss"] * ALPHA / (n * per)).float()[seq])[:, None]
        return dict(loss=(ALPHA / n * seq_loss.sum()).float().view(1), seq_loss=seq_loss.float(),
                    counts=counts.int(), dlogits=dz)
    if c["what"] == "weights":
        return _through_mx(s["w"].float(), 4).bfloat16()
    if c["what"] == "project":
        G, N, K = c["G"], c["N"], c["K"]
        a = _through_mx(s["x"].float(), c["bits"])
        b = _expand(s["b_q"], s["b_sf"], K, 4).view(G, N, K)
        return torch.bmm(_grouped(s, a, G, s["most"]),
                         b.transpose(1, 2))[s["grp"], s["pos"]].bfloat16()
    G, d, I = c["G"], c["d"], c["I"]
    x = _expand(s["x_q"], s["x_sf"], d, 8)
    w13 = _expand(s["W13_q"], s["W13_sf"], d, 4).view(G, 2 * I, d)
    gu = torch.bmm(_grouped(s, x, G, s["most"]), w13.transpose(1, 2))
    del w13
    a, u = gu[..., :I].clamp(max=CLAMP), gu[..., I:].clamp(-CLAMP, CLAMP)
    h = _through_mx(a * torch.sigmoid(a) * u, 8)
    w2 = _expand(s["W2_q"], s["W2_sf"], I, 4).view(G, d, I)
    o = torch.bmm(h, w2.transpose(1, 2))[s["grp"], s["pos"]]
    return (o * s["row_weight"][:, None]).bfloat16()


# ------------------------------------------------------------------- work

def _quantised(n, bits):
    """Bytes of n elements and their scales."""
    return n * bits // 8 + n // MX_BLOCK


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["d"]
        if c["what"] == "bwd":
            return dict(bytes=n * (8 if c["residual"] else 6) + 4 * c["T"] + 8 * c["d"],
                        flops=10 * n)
        b = n * (8 if c["residual"] else 4) + 4 * c["T"] + 4 * c["d"]
        b += {"none": 0, "fp8": n + 4 * c["T"] * -(-c["d"] // FP8_BLOCK),
              "mx": _quantised(n, 8)}[c["rows"]]
        return dict(bytes=b, flops=8 * n)
    if c["op"] == "balance":
        T, E, n = c["T"], c["E"], c["seqs"]
        k = min(c["k"], E)
        # the loss needs every logit before the first gradient: two readings
        return dict(bytes=12 * T * E + 4 * T * k + 2 * T + 8 * n * E, flops=16 * T * E)
    if c["what"] == "weights":
        n = c["rows"] * c["K"]
        return dict(bytes=4 * n + 2 * _quantised(n, 4), flops=4 * n)
    used = sum(1 for n in _counts(c["R"], c["G"]) if n)
    if c["what"] == "project":
        R, N, K = c["R"], c["N"], c["K"]
        return dict(bytes=2 * R * K + used * _quantised(N * K, 4) + 2 * R * N,
                    flops=2 * R * N * K)
    R, d, I = c["R"], c["d"], c["I"]
    return dict(bytes=_quantised(R * d, 8) + used * _quantised(3 * I * d, 4)
                + 4 * R + 2 * R * d, flops=6 * R * d * I)


# ------------------------------------------------------------------ exact

def _power_64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _near(v, step, most):
    """float64 values rounded to whole steps (ties to even), saturated."""
    return torch.copysign((torch.round(v.abs() / step) * step).clamp_max(most), v)


def _e4m3_64(v):
    e = torch.frexp(v).exponent
    return _near(v, _power_64((e - 4).clamp_min(-9)), FP8_MAX)


def _e2m1_64(v):
    e = torch.frexp(v).exponent
    return _near(v, _power_64((e - 2).clamp_min(-1)), 6.0)


def _block_power(v, top):
    """The scale of blocks [..., 32] of float64 values (1 for a block of zeros)."""
    amax = v.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax).exponent - 1 - top).clamp(-127, 127)
    return _power_64(torch.where(amax > 0, e, torch.zeros_like(e)))


def _mx_64(v, bits):
    b = v.reshape(*v.shape[:-1], -1, MX_BLOCK)
    x = _block_power(b, 2 if bits == 4 else 8)
    q = _e2m1_64(b / x) if bits == 4 else _e4m3_64(b / x)
    return (q * x).reshape(v.shape)


def _values_64(q, sf, K, bits):
    if bits == 8:
        v = q.view(torch.float8_e4m3fn).double()
    else:
        v = torch.empty(q.shape[0], K, dtype=torch.float64, device="cuda")
        for half in (0, 1):
            n = (q >> (4 * half)) & 15
            m, e = (n & 1).double(), ((n >> 1) & 3).int()
            mag = torch.where(e > 0, (1 + m / 2) * _power_64(e - 1), m / 2)
            v[:, half::2] = torch.where(n >= 8, -mag, mag)
    scale = _power_64(sf[:, :K // MX_BLOCK].int() - 127)
    return v * scale.repeat_interleave(MX_BLOCK, 1)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "norm" and c["what"] == "fwd":
        v = s["x"].double()
        if c["residual"]:
            v = (v + s["residual"].double()).bfloat16().double()     # what the stream keeps
        rstd = (v.square().sum(1) / c["d"] + EPS) ** -0.5
        y = v * rstd[:, None] * s["weight"].double()
        out = dict(y=y, rstd=rstd, residual=v if c["residual"] else None)
        if c["rows"] == "fp8":
            b = torch.cat([y, y.new_zeros(c["T"], -c["d"] % FP8_BLOCK)], 1)
            b = b.view(c["T"], -1, FP8_BLOCK)
            amax = b.abs().amax(2).clamp_min(FP8_FLOOR)
            r = (FP8_MAX / amax).float().double()
            q = _e4m3_64((b * r[:, :, None]).float().double())
            out.update(q=q.view(c["T"], -1)[:, :c["d"]].contiguous(), s=amax / FP8_MAX)
        elif c["rows"] == "mx":
            b = y.view(c["T"], -1, MX_BLOCK)
            x = _block_power(b, 8)
            sf = torch.full((c["T"], _pitch(c["d"])), 2.0 ** -127, dtype=torch.float64,
                            device="cuda")
            sf[:, :c["d"] // MX_BLOCK] = x[:, :, 0]
            out.update(q=_e4m3_64(b / x).view(c["T"], -1), s=sf)
        return out
    if c["op"] == "norm":
        w, r = s["weight"].double(), s["rstd"].double()[:, None]
        x, dy = s["x"].double(), s["dy"].double()
        inner = (x * dy * w).sum(1, keepdim=True)
        dx = r * dy * w - r ** 3 * x * inner / c["d"]
        if c["residual"]:
            dx += s["d_residual"].double()
        return dict(dx=dx, d_weight=(dy * x * r).sum(0))
    if c["op"] == "balance":
        E, n = c["E"], c["seqs"]
        k = min(c["k"], E)
        offs = s["seq_offsets"].tolist()
        counts = torch.zeros(n, E, dtype=torch.int32, device="cuda")
        seq_loss = torch.zeros(n, dtype=torch.float64, device="cuda")
        dz = torch.zeros(c["T"], E, dtype=torch.float64, device="cuda")
        for q in range(n):
            rows = torch.arange(offs[q], offs[q + 1], device="cuda")
            if s["valid"] is not None:
                rows = rows[s["valid"][rows] != 0]
            if not len(rows):
                continue
            z = s["logits"][rows].double()
            counts[q] = torch.bincount(s["ids"][rows].flatten().long(), minlength=E).int()
            f = counts[q].double() * E / (k * len(rows))
            if c["score"] == "sigmoid":
                sc = torch.sigmoid(z)
                p, slope = sc / sc.sum(1, keepdim=True), 1 - sc
            else:
                p, slope = torch.softmax(z, 1), 1.0
            seq_loss[q] = (f * p.mean(0)).sum()
            dz[rows] = (p * (f - (p @ f)[:, None]) * slope
                        * (s["dloss"].double() * ALPHA / (n * len(rows))))
        return dict(loss=(ALPHA * seq_loss.sum() / n).view(1), seq_loss=seq_loss, counts=counts,
                    dlogits=dz)
    if c["what"] == "weights":
        return _mx_64(s["w"].double(), 4)
    offs = [0] + list(np.cumsum(_counts(c["R"], c["G"])))
    spans = [(g, offs[g], offs[g + 1]) for g in range(c["G"]) if offs[g + 1] > offs[g]]
    if c["what"] == "project":
        N, K = c["N"], c["K"]
        y = torch.empty(c["R"], N, dtype=torch.float64, device="cuda")
        for g, lo, hi in spans:
            rows = slice(g * N, (g + 1) * N)
            y[lo:hi] = _mx_64(s["x"][lo:hi].double(), c["bits"]) \
                @ _values_64(s["b_q"][rows], s["b_sf"][rows], K, 4).T
        return y
    d, I = c["d"], c["I"]
    y = torch.empty(c["R"], d, dtype=torch.float64, device="cuda")
    for g, lo, hi in spans:
        rows = slice(g * 2 * I, (g + 1) * 2 * I)
        gu = _values_64(s["x_q"][lo:hi], s["x_sf"][lo:hi], d, 8) \
            @ _values_64(s["W13_q"][rows], s["W13_sf"][rows], d, 4).T
        a, u = gu[:, :I].clamp(max=CLAMP), gu[:, I:].clamp(-CLAMP, CLAMP)
        h = _mx_64(a / (1 + torch.exp(-a)) * u, 8)
        rows = slice(g * d, (g + 1) * d)
        y[lo:hi] = h @ _values_64(s["W2_q"][rows], s["W2_sf"][rows], I, 4).T
    return y * s["row_weight"].double()[:, None]
