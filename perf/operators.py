"""Cases of the block-scaled FP8 operators and of the few-token layer.

Five operators of one serving and training set around the expert layer:

  few     the whole layer (gate, routing, experts, shared expert, combine) for
          1 to 32 tokens, with bf16 expert weights or with FP8 ones (E4M3
          codes, one fp32 scale per 128 x 128 block)
  quant   FP8 quantisation with a scale for each block of 128: token rows in
          the dispatch (1 x 128 blocks, each row written to its k + 1 permuted
          rows) and weights (128 x 128 blocks, both orientations)
  matmul  rows grouped by expert times each expert's weight, both in FP8 with
          block scales (also the data gradient, with the transposed weight)
  wgrad   the weight gradient dW[g] = A_g^T B_g, both operands quantised along
          the group's rows in blocks of 128
  ffn     the expert FFN on grouped rows: two FP8 matmuls around the clamped
          SwiGLU, its result quantised again

`own` chooses between the plain form (elementary torch operations in fp32,
rounded once at the end) and the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 128            # elements that share a scale
FP8_MAX = 448.0        # largest E4M3 value
AMAX_FLOOR = 2.0 ** -100   # a block's largest magnitude counts as at least this
VOCAB = 4096


# ------------------------------------------------------------------ cases

def listed():
    full = dict(d=4096, E=384, k=6, I=2048)
    return [
        # one user decoding: 7 experts' weights cross HBM for one token
        dict(name="few_bf16_one", op="few", T=1, fp8=False, hash=False, **full),
        # a small layer with odd widths, hash router, a batch that fills no tile
        dict(name="few_bf16_ragged_hash", op="few", T=23, fp8=False, hash=True, d=1152, E=97, k=5,
             I=704),
        # the largest decode batch of the call: ~150 of 384 experts are hit
        dict(name="few_bf16_batch", op="few", T=32, fp8=False, hash=False, **full),
        # one user decoding from FP8 weights
        dict(name="few_fp8_one", op="few", T=1, fp8=True, hash=False, **full),
        # a decode batch (or one request's draft tokens) from FP8 weights
        dict(name="few_fp8_sixteen", op="few", T=16, fp8=True, hash=False, **full),
        # the dispatch of a prefill chunk
        dict(name="quant_dispatch", op="quant", what="gather", T=4096, k=6, d=4096),
        # weights after an optimizer step (or at load): both orientations
        dict(name="quant_weights", op="quant", what="weights", G=9, N=4096, K=4096),
        # a dense projection of one token
        dict(name="matmul_one", op="matmul", G=1, R=1, N=4096, K=4096),
        # expert rows of uneven counts (one expert empty, one with a single row)
        dict(name="matmul_ragged", op="matmul", G=33, R=12345, N=4096, K=2048),
        # the weight gradient of the first expert matmul
        dict(name="wgrad_ragged", op="wgrad", G=9, R=6789, M=4096, N=4096),
        # a short prefill over a few local experts
        dict(name="ffn_short", op="ffn", G=9, R=777, d=4096, I=2048),
        # a long prefill: about a thousand rows per expert
        dict(name="ffn_long", op="ffn", G=33, R=32768, d=4096, I=2048),
    ]


def _log(rng, lo, hi):
    """A whole number, its logarithm spread evenly over [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["few", "few", "quant", "matmul", "wgrad", "ffn"])
    if op == "few":
        E = _log(rng, 8, 384)
        return dict(op=op, T=_log(rng, 1, 32), fp8=rng.random() < 0.5, hash=rng.random() < 0.3,
                    d=128 * rng.randint(1, 32), E=E, k=rng.randint(1, 8), I=64 * rng.randint(1, 32))
    if op == "quant":
        if rng.random() < 0.5:
            return dict(op=op, what="gather", T=_log(rng, 1, 4096), k=rng.randint(1, 8),
                        d=16 * rng.randint(1, 256))
        return dict(op=op, what="weights", G=rng.randint(1, 8), N=16 * rng.randint(1, 256),
                    K=16 * rng.randint(1, 256))
    if op == "matmul":
        return dict(op=op, G=_log(rng, 1, 33), R=_log(rng, 1, 12345), N=8 * _log(rng, 1, 512),
                    K=16 * _log(rng, 1, 256))
    if op == "wgrad":
        return dict(op=op, G=rng.randint(1, 9), R=_log(rng, 1, 6789), M=8 * rng.randint(1, 512),
                    N=8 * rng.randint(1, 512))
    return dict(op=op, G=_log(rng, 1, 33), R=_log(rng, 1, 16384), d=128 * rng.randint(1, 32),
                I=128 * rng.randint(1, 16))


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


def _codes(g, *shape):
    """E4M3 codes of values that fill the format's range, as bytes."""
    return (_randn(g, *shape) * 100.0).clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(
        torch.uint8)


def _scales(g, std, *shape):
    return (torch.rand(shape, generator=g, device="cuda") + 0.5) * (std / 100.0)


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _rows_plan(case):
    c = _counts(case["R"], case["G"])
    offs = np.concatenate([[0], np.cumsum(c)]).astype(np.int32)
    grp = np.repeat(np.arange(case["G"]), c)
    pos = np.arange(case["R"]) - offs[grp]
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return dict(offsets=dev(offs), grp=dev(grp.astype(np.int64)), pos=dev(pos.astype(np.int64)),
                most=max(c))


def prepare(case, seed):
    g = _gen(seed, 1)
    c = case
    dev = dict(device="cuda")
    s = dict(case=dict(case))
    if c["op"] == "few":
        T, d, E, k, I = (c[n] for n in ("T", "d", "E", "k", "I"))
        std = 1.28 / math.sqrt(d)
        s["x"] = _randn(g, T, d)
        s["W_g"] = _randn(g, E, d) * std
        s["bias"] = (torch.rand(2, E, generator=g, **dev) * 2 - 1) * 0.01
        s["is_vision"] = (torch.rand(T, generator=g, **dev) < 0.3).to(torch.uint8)
        s["logit_offset"] = torch.randn(E, generator=g, **dev) * 0.1
        if c["hash"]:
            s["input_ids"] = torch.randint(0, VOCAB, (T,), generator=g, dtype=torch.int32, **dev)
            s["tid2eid"] = torch.rand(VOCAB, E, generator=g, **dev).topk(k, dim=1).indices.int()
        for name, rows, cols in (("W13", 2 * I, d), ("W2", d, I)):
            std = 1.28 / math.sqrt(cols)
            if c["fp8"]:
                w = torch.empty(E + 1, rows, cols, dtype=torch.uint8, **dev)
                for e in range(0, E + 1, 32):
                    n = min(32, E + 1 - e)
                    w[e:e + n] = _codes(g, n, rows, cols)
                s[name + "_q"] = w
                s[name + "_s"] = _scales(g, std, E + 1, _blocks(rows), _blocks(cols))
            else:
                w = torch.empty(E + 1, rows, cols, dtype=torch.bfloat16, **dev)
                for e in range(0, E + 1, 32):
                    n = min(32, E + 1 - e)
                    torch.mul(_randn(g, n, rows, cols), std, out=w[e:e + n])
                s[name] = w
        s["y"] = torch.empty(T, d, dtype=torch.bfloat16, **dev)
        s["ids"] = torch.empty(T, k, dtype=torch.int32, **dev)
        s["weights"] = torch.empty(T, k, dtype=torch.float32, **dev)
    elif c["op"] == "quant" and c["what"] == "gather":
        T, d, k = c["T"], c["d"], c["k"]
        # activations: every token at its own scale, a few channels far larger
        x = _randn(g, T, d) * torch.exp(_randn(g, T, 1))
        x *= torch.where(torch.rand(d, generator=g, **dev) < 0.01, 20.0, 1.0).to(x.dtype)
        s["x"] = x
        # permuted row of each (token, slot), as the dispatch gives it
        s["slot_row"] = torch.randperm(T * k, generator=g, **dev).int()
        s["q"] = torch.empty(T * k + T, d, dtype=torch.uint8, **dev)
        s["s"] = torch.empty(T * k + T, _blocks(d), dtype=torch.float32, **dev)
    elif c["op"] == "quant":
        G, N, K = c["G"], c["N"], c["K"]
        s["w"] = _randn(g, G, N, K) * 0.02
        s["q"] = torch.empty(G, N, K, dtype=torch.uint8, **dev)
        s["s"] = torch.empty(G, _blocks(N), _blocks(K), dtype=torch.float32, **dev)
        s["qt"] = torch.empty(G, K, N, dtype=torch.uint8, **dev)
        s["st"] = torch.empty(G, _blocks(K), _blocks(N), dtype=torch.float32, **dev)
    elif c["op"] == "matmul":
        R, G, N, K = c["R"], c["G"], c["N"], c["K"]
        s.update(_rows_plan(c))
        s["a_q"], s["a_s"] = _codes(g, R, K), _scales(g, 1.0, R, _blocks(K))
        s["b_q"] = _codes(g, G, N, K)
        s["b_s"] = _scales(g, 1.28 / math.sqrt(K), G, _blocks(N), _blocks(K))
        s["row_weight"] = torch.rand(R, generator=g, **dev) + 0.1
        s["out"] = torch.empty(R, N, dtype=torch.bfloat16, **dev)
    elif c["op"] == "wgrad":
        R, G, M, N = c["R"], c["G"], c["M"], c["N"]
        s.update(_rows_plan(c))
        s["a"] = _randn(g, R, M) * torch.exp(_randn(g, R, 1) * 0.5)
        s["b"] = _randn(g, R, N)
        s["dW"] = torch.empty(G, M, N, dtype=torch.float32, **dev)
    else:
        R, G, d, I = c["R"], c["G"], c["d"], c["I"]
        s.update(_rows_plan(c))
        s["x_q"], s["x_s"] = _codes(g, R, d), _scales(g, 1.0, R, _blocks(d))
        s["W13_q"] = _codes(g, G, 2 * I, d)
        s["W13_s"] = _scales(g, 1.28 / math.sqrt(d), G, _blocks(2 * I), _blocks(d))
        s["W2_q"] = _codes(g, G, d, I)
        s["W2_s"] = _scales(g, 1.28 / math.sqrt(I), G, _blocks(d), _blocks(I))
        s["row_weight"] = torch.rand(R, generator=g, **dev) + 0.1
        s["h_q"] = torch.empty(R, I, dtype=torch.uint8, **dev)
        s["h_s"] = torch.empty(R, _blocks(I), dtype=torch.float32, **dev)
        s["y"] = torch.empty(R, d, dtype=torch.bfloat16, **dev)
    return s


SCALING, CLAMP = 2.5, 7.0


# ------------------------------------------------------------------- runs

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _fp8(t):
    return t.view(torch.float8_e4m3fn)


def _run_own(s):
    from moe_expert_layer_04_gb300 import _lib
    c = s["case"]
    if c["op"] == "few":
        T, d, E, k, I = (c[n] for n in ("T", "d", "E", "k", "I"))
        if "ws" not in s:      # zeroed once, kept by the program
            s["ws"] = torch.zeros(_lib.moe_few_workspace_size(T, d, E, k, I), dtype=torch.uint8,
                                  device="cuda")
        mode = _lib.MOE_ROUTE_HASH if c["hash"] else _lib.MOE_ROUTE_TOPK
        args = dict(T=T, d=d, E=E, k=k, I=I, scaling=SCALING, clamp=CLAMP, mode=mode,
                    vocab=VOCAB if c["hash"] else 0)
        for n in ("x", "W_g", "logit_offset", "bias", "is_vision", "input_ids", "tid2eid", "W13",
                  "W2", "W13_q", "W13_s", "W2_q", "W2_s", "y", "ids", "weights", "ws"):
            args[n] = s.get(n)
        _lib.moe_layer_few(args)
        return dict(y=s["y"], weights=s["weights"])
    if c["op"] == "quant" and c["what"] == "gather":
        _lib.moe_fp8_gather(s["x"], s["slot_row"], c["T"], c["d"], c["k"], s["q"], s["s"])
        return dict(q=_fp8(s["q"]), s=s["s"])
    if c["op"] == "quant":
        _lib.moe_fp8_quantize_weights(s["w"], c["G"], c["N"], c["K"], s["q"], s["s"], s["qt"],
                                      s["st"])
        return dict(q=_fp8(s["q"]), s=s["s"], qt=_fp8(s["qt"]), st=s["st"])
    if c["op"] == "matmul":
        _lib.moe_fp8_matmul(s["a_q"], s["a_s"], s["offsets"], c["G"], c["R"], s["b_q"], s["b_s"],
                            s["row_weight"], c["R"], c["N"], c["K"], s["out"])
        return s["out"]
    if c["op"] == "wgrad":
        if "ws" not in s:
            s["ws"] = torch.empty(
                _lib.moe_fp8_wgrad_workspace_size(c["G"], c["R"], c["M"], c["N"]),
                dtype=torch.uint8, device="cuda")
        _lib.moe_fp8_wgrad(s["a"], s["b"], s["offsets"], c["G"], c["R"], c["M"], c["N"], s["dW"],
                           s["ws"])
        return s["dW"]
    _lib.moe_expert_ffn_fp8(s["x_q"], s["x_s"], s["offsets"], c["G"], c["R"], s["W13_q"],
                            s["W13_s"], s["W2_q"], s["W2_s"], s["row_weight"], c["R"], c["d"],
                            c["I"], CLAMP, s["h_q"], s["h_s"], s["y"])
    return s["y"]


def _expand(sc, rows, cols):
    """Block scales [..., rows/128, cols/128] at every element."""
    return sc.repeat_interleave(BLOCK, -2)[..., :rows, :].repeat_interleave(BLOCK, -1)[..., :cols]


def _row_scales(sc, cols):
    return sc.repeat_interleave(BLOCK, -1)[..., :cols]


def _quantise(v, dim):
    """fp32 v with a block axis `dim` of 128 values -> (E4M3 values in fp32, scale)."""
    amax = v.abs().amax(dim, keepdim=True).clamp_min(AMAX_FLOOR)
    top = torch.full_like(amax, FP8_MAX)
    q = (v * (top / amax)).to(torch.float8_e4m3fn)
    return q, amax / top


def _pad_cols(v):
    return torch.nn.functional.pad(v, (0, -v.shape[-1] % BLOCK))


def _quantise_rows(v):
    """[rows, K] fp32 -> codes [rows, K] (float8) and scales [rows, K/128]."""
    K = v.shape[-1]
    p = _pad_cols(v).unflatten(-1, (-1, BLOCK))
    q, sc = _quantise(p, -1)
    return q.flatten(-2)[..., :K], sc.squeeze(-1)


def _grouped(s, v, G, most):
    """Rows of all groups -> [G, most, ...], zeros behind each group's rows."""
    out = torch.zeros(G, most, v.shape[1], dtype=v.dtype, device=v.device)
    out[s["grp"], s["pos"]] = v
    return out


def _silu_clamped(g, u):
    g = g.clamp(max=CLAMP)
    return g * torch.sigmoid(g) * u.clamp(-CLAMP, CLAMP)


def _expert_weights(s, name, e, rows, cols):
    """fp32 weights of the experts `e` (any index shape)."""
    if name in s:
        return s[name][e].float()
    return _fp8(s[name + "_q"][e]).float() * _expand(s[name + "_s"][e], rows, cols)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "few":
        T, d, E, k, I = (c[n] for n in ("T", "d", "E", "k", "I"))
        x = s["x"].float()
        score = torch.sigmoid(x @ s["W_g"].float().T + s["logit_offset"])
        if c["hash"]:
            ids = s["tid2eid"][s["input_ids"].long()].long()
        else:
            key = score + s["bias"][s["is_vision"].long()]
            ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
        sel = torch.gather(score, 1, ids)
        w = SCALING * sel / sel.sum(1, keepdim=True)
        every = torch.cat([ids, torch.full_like(ids[:, :1], E)], 1)   # and the shared expert
        gu = (_expert_weights(s, "W13", every, 2 * I, d) @ x[:, None, :, None]).squeeze(-1)
        h = _silu_clamped(gu[..., :I], gu[..., I:])
        o = (_expert_weights(s, "W2", every, d, I) @ h.unsqueeze(-1)).squeeze(-1)
        wt = torch.cat([w, torch.ones_like(w[:, :1])], 1)
        return dict(y=(o * wt.unsqueeze(-1)).sum(1).bfloat16(), weights=w)
    if c["op"] == "quant" and c["what"] == "gather":
        T, k = c["T"], c["k"]
        q, sc = _quantise_rows(s["x"].float())
        tok = torch.arange(T, device="cuda")
        row_token = torch.cat([torch.empty(T * k, dtype=torch.long, device="cuda"), tok])
        row_token[s["slot_row"].long()] = tok.repeat_interleave(k)
        return dict(q=_fp8(q.contiguous().view(torch.uint8)[row_token]), s=sc[row_token])
    if c["op"] == "quant":
        G, N, K = c["G"], c["N"], c["K"]
        v = torch.nn.functional.pad(s["w"].float(), (0, -K % BLOCK, 0, -N % BLOCK))
        v = v.unflatten(2, (-1, BLOCK)).unflatten(1, (-1, BLOCK)).transpose(2, 3).flatten(3)
        q, sc = _quantise(v, -1)
        q = q.view(torch.uint8).unflatten(3, (BLOCK, BLOCK)).transpose(2, 3).flatten(3)
        q = q.flatten(1, 2)[:, :N, :K].contiguous()
        sc = sc.squeeze(-1)
        return dict(q=_fp8(q), s=sc, qt=_fp8(q.transpose(1, 2).contiguous()),
                    st=sc.transpose(1, 2).contiguous())
    if c["op"] == "matmul":
        G, N, K = c["G"], c["N"], c["K"]
        a = _fp8(s["a_q"]).float() * _row_scales(s["a_s"], K)
        b = _fp8(s["b_q"]).float() * _expand(s["b_s"], N, K)
        o = torch.bmm(_grouped(s, a, G, s["most"]), b.transpose(1, 2))[s["grp"], s["pos"]]
        return (o * s["row_weight"][:, None]).bfloat16()
    if c["op"] == "wgrad":
        G = c["G"]
        most = s["most"] + -s["most"] % BLOCK

        def along_rows(v):
            p = _grouped(s, v.float(), G, most).unflatten(1, (-1, BLOCK))
            q, sc = _quantise(p, 2)
            return (q.float() * sc).flatten(1, 2)
        return torch.bmm(along_rows(s["a"]).transpose(1, 2), along_rows(s["b"]))
    G, d, I = c["G"], c["d"], c["I"]
    x = _fp8(s["x_q"]).float() * _row_scales(s["x_s"], d)
    w13 = _fp8(s["W13_q"]).float() * _expand(s["W13_s"], 2 * I, d)
    gu = torch.bmm(_grouped(s, x, G, s["most"]), w13.transpose(1, 2))
    hq, hs = _quantise_rows(_silu_clamped(gu[..., :I], gu[..., I:]))
    w2 = _fp8(s["W2_q"]).float() * _expand(s["W2_s"], d, I)
    o = torch.bmm(hq.float() * _row_scales(hs, I), w2.transpose(1, 2))[s["grp"], s["pos"]]
    return (o * s["row_weight"][:, None]).bfloat16()


# ------------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "few":
        T, d, E, k, I = (c[n] for n in ("T", "d", "E", "k", "I"))
        hit = E * (1 - (1 - k / E) ** T) + 1 if k <= E else E + 1
        elt = 1 if c["fp8"] else 2
        per = 3 * I * d * elt
        if c["fp8"]:
            per += 4 * (_blocks(2 * I) * _blocks(d) + _blocks(d) * _blocks(I))
        gate = 2 * T * k * d if c["hash"] else 2 * T * E * d
        return dict(bytes=hit * per + 2 * (min(E, T * k) if c["hash"] else E) * d + 4 * T * d,
                    flops=gate + T * (k + 1) * 6 * I * d)
    if c["op"] == "quant" and c["what"] == "gather":
        rows = c["T"] * (c["k"] + 1)
        return dict(bytes=2 * c["T"] * c["d"] + rows * (c["d"] + 4 * _blocks(c["d"])),
                    flops=3 * c["T"] * c["d"])
    if c["op"] == "quant":
        n = c["G"] * c["N"] * c["K"]
        return dict(bytes=4 * n + 8 * c["G"] * _blocks(c["N"]) * _blocks(c["K"]), flops=3 * n)
    if c["op"] == "matmul":
        R, N, K = c["R"], c["N"], c["K"]
        used = sum(1 for n in _counts(R, c["G"]) if n)
        return dict(bytes=R * (K + 4 * _blocks(K) + 2 * N + 4)
                    + used * (N * K + 4 * _blocks(N) * _blocks(K)), flops=2 * R * N * K)
    if c["op"] == "wgrad":
        R, M, N = c["R"], c["M"], c["N"]
        return dict(bytes=2 * R * (M + N) + 4 * c["G"] * M * N, flops=2 * R * M * N)
    R, d, I = c["R"], c["d"], c["I"]
    used = sum(1 for n in _counts(R, c["G"]) if n)
    return dict(bytes=R * (d + 4 * _blocks(d) + 4 + 2 * d) + used * 3 * I * d,
                flops=6 * R * d * I)


# ------------------------------------------------------------------ exact

def _e4m3_64(v):
    """float64 values rounded to the nearest E4M3 value (ties to even), as
    float64; NaN stays NaN."""
    m, e = torch.frexp(v.abs())
    step = torch.ldexp(torch.ones_like(v), (e - 4).clamp_min(-9).to(v.dtype))
    return torch.copysign((torch.round(v.abs() / step) * step).clamp_max(FP8_MAX), v)


def _quantise_64(v, dim):
    """The operator's definition on float64 values: the scale amax / 448, the
    factor 448 / amax and each product are fp32 numbers."""
    f32 = lambda t: t.float().double()
    amax = v.abs().amax(dim, keepdim=True).clamp_min(AMAX_FLOOR)
    amax = f32(amax)
    return _e4m3_64(f32(v * f32(FP8_MAX / amax))), f32(amax / FP8_MAX)


def _pad_to_block(v, dim):
    n = v.shape[dim]
    shape = list(v.shape)
    shape[dim] = -n % BLOCK
    return torch.cat([v, v.new_zeros(shape)], dim)


def _weight_64(s, name, e):
    if name in s:
        return s[name][e].double()
    q, sc = s[name + "_q"][e], s[name + "_s"][e].double()
    rows = torch.arange(q.shape[0], device="cuda") // BLOCK
    cols = torch.arange(q.shape[1], device="cuda") // BLOCK
    return _fp8(q).double() * sc[rows][:, cols]


def _rows_64(q, sc):
    cols = torch.arange(q.shape[1], device="cuda") // BLOCK
    return _fp8(q).double() * sc.double()[:, cols]


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "few":
        T, d, E, k, I = (c[n] for n in ("T", "d", "E", "k", "I"))
        x = s["x"].double()
        score = 1 / (1 + torch.exp(-(x @ s["W_g"].double().T + s["logit_offset"].double())))
        y = torch.zeros(T, d, dtype=torch.float64, device="cuda")
        w = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        pairs = {E: [(t, 1.0) for t in range(T)]}
        for t in range(T):
            if c["hash"]:
                ids = s["tid2eid"][int(s["input_ids"][t])].tolist()
            else:
                key = (score[t] + s["bias"][int(s["is_vision"][t])].double()).tolist()
                ids = sorted(range(E), key=lambda e: (-key[e], e))[:k]
            sel = score[t, ids]
            w[t] = SCALING * sel / sel.sum()
            for j, e in enumerate(ids):
                pairs.setdefault(e, []).append((t, w[t, j]))
        for e, rows in pairs.items():
            tok = torch.tensor([t for t, _ in rows], device="cuda")
            f = torch.stack([torch.as_tensor(v, dtype=torch.float64, device="cuda")
                             for _, v in rows])
            gu = x[tok] @ _weight_64(s, "W13", e).T
            g, u = gu[:, :I].clamp(max=CLAMP), gu[:, I:].clamp(-CLAMP, CLAMP)
            h = g / (1 + torch.exp(-g)) * u
            y.index_add_(0, tok, f[:, None] * (h @ _weight_64(s, "W2", e).T))
        return dict(y=y, weights=w)
    if c["op"] == "quant" and c["what"] == "gather":
        T, k, d = c["T"], c["k"], c["d"]
        q, sc = _quantise_64(_pad_to_block(s["x"].double(), 1).view(T, -1, BLOCK), 2)
        q, sc = q.view(T, -1)[:, :d], sc[:, :, 0]
        back = torch.argsort(s["slot_row"].long()) // k      # token of each routed row
        return dict(q=torch.cat([q[back], q]), s=torch.cat([sc[back], sc]))
    if c["op"] == "quant":
        G, N, K = c["G"], c["N"], c["K"]
        q = torch.empty(G, N, K, dtype=torch.float64, device="cuda")
        sc = torch.empty(G, _blocks(N), _blocks(K), dtype=torch.float64, device="cuda")
        for i in range(_blocks(N)):
            rows = s["w"][:, i * BLOCK:(i + 1) * BLOCK].double()
            v = _pad_to_block(rows, 2).view(G, rows.shape[1], -1, BLOCK)
            vq, vs = _quantise_64(v.transpose(1, 2).reshape(G, v.shape[2], -1), 2)
            q[:, i * BLOCK:(i + 1) * BLOCK] = vq.view(G, v.shape[2], rows.shape[1], BLOCK) \
                .transpose(1, 2).reshape(G, rows.shape[1], -1)[:, :, :K]
            sc[:, i] = vs[:, :, 0]
        return dict(q=q, s=sc, qt=q.transpose(1, 2).contiguous(),
                    st=sc.transpose(1, 2).contiguous())
    offs = [0] + list(np.cumsum(_counts(c["R"], c["G"])))
    spans = [(g, offs[g], offs[g + 1]) for g in range(c["G"])]
    if c["op"] == "matmul":
        y = torch.empty(c["R"], c["N"], dtype=torch.float64, device="cuda")
        a = _rows_64(s["a_q"], s["a_s"])
        for g, lo, hi in spans:
            if hi > lo:
                y[lo:hi] = a[lo:hi] @ _weight_64(s, "b", g).T
        return y * s["row_weight"].double()[:, None]
    if c["op"] == "wgrad":
        dW = torch.zeros(c["G"], c["M"], c["N"], dtype=torch.float64, device="cuda")
        for g, lo, hi in spans:
            for r in range(lo, hi, BLOCK):
                n = min(r + BLOCK, hi)
                (qa, sa), (qb, sb) = (_quantise_64(s[m][r:n].double(), 0) for m in ("a", "b"))
                dW[g] += (qa * sa).T @ (qb * sb)
        return dW
    y = torch.empty(c["R"], c["d"], dtype=torch.float64, device="cuda")
    I = c["I"]
    for g, lo, hi in spans:
        if hi == lo:
            continue
        gu = _rows_64(s["x_q"][lo:hi], s["x_s"][lo:hi]) @ _weight_64(s, "W13", g).T
        a, u = gu[:, :I].clamp(max=CLAMP), gu[:, I:].clamp(-CLAMP, CLAMP)
        h = (a / (1 + torch.exp(-a)) * u).view(hi - lo, -1, BLOCK)
        hq, hs = _quantise_64(h, 2)
        y[lo:hi] = (hq * hs).view(hi - lo, I) @ _weight_64(s, "W2", g).T
    return y * s["row_weight"].double()[:, None]
