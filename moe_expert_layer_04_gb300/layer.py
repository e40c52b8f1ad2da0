"""The routed MoE layer on one GPU, as a sequence of C-ABI calls.

This module only allocates device memory (through PyTorch) and calls the
library in order; every step of the layer runs in the library's kernels:

  forward   moe_gate_route (or moe_route) -> moe_permute -> moe_expert_ffn
            (or the one-launch moe_expert_ffn_fused) -> moe_combine
  backward  moe_backward
  decoding  moe_layer_few (at most 32 tokens, two launches)
  around it moe_rmsnorm ahead of the routing, moe_balance_loss behind it, and
            their backward (moe_gate_backward carries the loss's gradient into dX
            and dW_g)

("HyperParallel加速DeepSeek-V4.1多模态1M长序列训练" §2.3: MegaGate routing
pipeline, then MegaMoE dispatch, two expert matmuls around the clamped
SwiGLU, and result return; the shared expert of "MindSpore HyperParallel
一键开箱DeepSeek-V4.1-Flash" §01 runs as expert group E on every token.)
"""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import MOE_FLAG_BACKWARD, MOE_FLAG_RECOMPUTE, MOE_ROUTE_HASH, MOE_ROUTE_TOPK


def gate_route_supported(d: int, E: int, k: int) -> bool:
    """Shapes the one-kernel gate projection + routing (moe_gate_route) takes:
    the logits of 128 tokens for all E experts must fit in tensor memory."""
    return d % 64 == 0 and E % 32 == 0 and 32 <= E <= 512 and 1 <= k <= min(8, E)


def mx_supported(d: int, I: int) -> bool:
    """Shapes the MXFP8 expert matmuls (moe_expert_ffn_mx) take."""
    return d % 256 == 0 and I % 128 == 0


def mx4_supported(d: int, I: int) -> bool:
    """Shapes the expert FFN with MXFP4 weights (moe_expert_ffn_mx4) takes."""
    return d % 128 == 0 and I % 128 == 0


def fp8_supported(d: int, I: int) -> bool:
    """Shapes the expert FFN on FP8 rows (moe_expert_ffn_fp8) takes."""
    return d % 128 == 0 and I % 128 == 0


def norm_supported(d: int) -> bool:
    """Row lengths the norm ahead of the layer (moe_rmsnorm) takes."""
    return d % 8 == 0 and 8 <= d <= 32768


def _expect(name, t, *shape):
    """A tensor, where it is given, has the elements that a call reads or writes."""
    if t is not None and t.numel() != math.prod(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")


def _result(stream, device, *shape):
    """A bf16 tensor that a call on `stream` (None: the current one) writes and the
    caller reads on the current stream: memory of the first, kept for both."""
    if stream is None:
        return torch.empty(*shape, dtype=torch.bfloat16, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(*shape, dtype=torch.bfloat16, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


class _StreamBuffers:
    """Tensors of the given (shape, dtype)s for the calls of each stream, made at its first
    one and kept; a captured call gets its own."""

    def __init__(self, device, *specs):
        self.device, self.specs, self.kept = device, specs, {}

    def of(self, stream):
        """Those of `stream` (None: the current one), memory of that stream."""
        if self.device.type != "cuda":
            return self._of_current(stream)
        if stream is None:
            return self._of_current(_lib._stream(None))
        with torch.cuda.stream(stream):
            return self._of_current(stream.cuda_stream)

    def _of_current(self, key):
        capturing = self.device.type == "cuda" and torch.cuda.is_current_stream_capturing()
        got = None if capturing else self.kept.get(key)
        if got is None:
            got = tuple(torch.empty(*shape, dtype=t, device=self.device)
                        for shape, t in self.specs)
            if not capturing:
                self.kept[key] = got
        return got


def ffn_fused_supported(d: int, I: int) -> bool:
    """Shapes the one-launch expert FFN (moe_expert_ffn_fused) takes: 256-wide
    tiles in both matmuls."""
    return I % 128 == 0 and d % 256 == 0


@dataclass(frozen=True)
class Dims:
    T: int
    d: int
    E: int
    k: int
    I: int

    @property
    def S(self):
        return self.T * self.k

    @property
    def R(self):
        return self.T * self.k + self.T


class MoELayer:
    """Preallocated buffers for one layer shape, reused across calls.

    weights: dict with W_g [E,d], W13 [E+1,2I,d], W2 [E+1,d,I] (bf16, CUDA).
    fused_route: route with the one-kernel gate projection + routing, which
    also counts the expert load per modality (None: whenever the shape allows).
    fused_ffn: run both expert matmuls in one persistent launch
    (moe_expert_ffn_fused).  Off by default: it is bit-identical to the two
    launches and measures the same on one GPU, and its waits assume that no
    other work shares the GPU's SMs.
    mx: the low-precision variant -- the expert weights are quantised to MXFP8
    here (moe_mx_quantize; again with quantize_weights() after they change),
    each step's token rows are quantised in the dispatch (moe_mx_gather) and
    both expert matmuls take MXFP8 operands (moe_expert_ffn_mx); h between them
    is MXFP8 too.  With backward, the weights also get copies quantised along
    their other axis (moe_mx_quantize_t) and the backward runs the MX dgrad
    matmuls (moe_backward_mx).  Two launches (not fused_ffn).
    fp8: the serving variant whose expert weights are FP8 (E4M3) with one fp32
    scale per 128 x 128 block, quantised here (moe_fp8_quantize_weights; again
    with quantize_weights() after they change), or given so, as checkpoints hold
    them: weights then has W13_q [E+1,2I,d], W2_q [E+1,d,I] (E4M3 codes, as
    float8_e4m3fn or uint8) and W13_s [E+1,2I/128,d/128], W2_s [E+1,d/128,I/128]
    (fp32) in place of W13 and W2.  forward() quantises each
    step's token rows in the dispatch (moe_fp8_gather) and runs
    moe_expert_ffn_fp8; forward_few() decodes from the same weights.  Forward
    only (GroupedLinearFP8 has the matmul's gradients).
    mx4: the serving variant whose expert weights are MXFP4 (4-bit elements, one
    power of two per 32), quantised here (moe_mx4_quantize; again with
    quantize_weights() after they change), or given so: weights then has W13_q
    [E+1,2I,d/2], W2_q [E+1,d,I/2], W13_sf [E+1,2I,moe_mx_sf_pitch(d)] and W2_sf
    [E+1,d,moe_mx_sf_pitch(I)] (uint8) in place of W13 and W2.  forward() quantises
    each step's token rows to MXFP8 in the dispatch and runs moe_expert_ffn_mx4.
    Forward only.
    norm_eps: the root-mean-square norm ahead of the layer, of weight weights["norm"]
    (fp32 [d]).  forward() then takes rows of the residual stream's update x and, with
    `residual`, adds them to it first; self.residual is the stream after the addition
    (x itself without one).  In the MX, MXFP4 and FP8 layers the same kernel quantises
    the rows (of the norm's fp32 result) and the dispatch moves their codes.  backward()
    returns the gradient of x and of the residual (self.dnorm: the weight's).
    forward_few() takes rows that norm() has been through.
    balance: alpha of the router's balance loss over `sequences` sequences (softmax
    shares with balance_softmax, of sigmoid scores without).  forward() writes
    self.balance_loss [1], self.balance_counts [sequences, E] and balance_load; backward()
    adds its gradient (times d_balance) to dX and dW_g.
    """

    mx4 = False
    norm_eps = balance_alpha = None

    def __init__(self, dims: Dims, weights: dict, scaling: float, clamp: float = 7.0,
                 backward: bool = False, recompute: bool = False, device="cuda",
                 fused_route: bool | None = None, fused_ffn: bool = False, mx: bool = False,
                 fp8: bool = False, mx4: bool = False, norm_eps: float | None = None,
                 balance: float | None = None, sequences: int = 1,
                 balance_softmax: bool = False):
        self.dims = dims
        if mx4 and (mx or fp8 or fused_ffn or backward or not mx4_supported(dims.d, dims.I)):
            raise ValueError(f"the MXFP4 layer runs the forward in two launches and needs "
                             f"d % 128 == 0, I % 128 == 0 (got {dims})")
        if mx4:
            self.mx4 = True
        if fp8 and (mx or fused_ffn or backward or not fp8_supported(dims.d, dims.I)):
            raise ValueError(f"the FP8 layer runs the forward in two launches and needs "
                             f"d % 128 == 0, I % 128 == 0 (got {dims})")
        self.fp8 = bool(fp8)
        if mx and (fused_ffn or not mx_supported(dims.d, dims.I)):
            raise ValueError(f"the MXFP8 layer runs two launches and needs "
                             f"d % 256 == 0, I % 128 == 0 (got {dims})")
        self.mx = bool(mx)
        ok = gate_route_supported(dims.d, dims.E, dims.k)
        if fused_route and not ok:
            raise ValueError(f"moe_gate_route does not take the shape {dims}")
        self.fused_route = ok if fused_route is None else bool(fused_route)
        if fused_ffn and not ffn_fused_supported(dims.d, dims.I):
            raise ValueError(f"moe_expert_ffn_fused does not take the shape {dims}")
        self.fused_ffn = bool(fused_ffn)
        self.w = weights
        self.scaling = float(scaling)
        self.clamp = float(clamp)
        self.recompute = recompute
        self.backward_enabled = backward
        D = dims
        dev = torch.device(device)
        e = dict(device=dev)
        self.logits = torch.empty(D.T, D.E, dtype=torch.float32, **e)
        self.ids = torch.empty(D.T, D.k, dtype=torch.int32, **e)
        self.weights = torch.empty(D.T, D.k, dtype=torch.float32, **e)
        self.scores_sel = torch.empty(D.T, D.k, dtype=torch.float32, **e)
        self.counts = torch.empty(D.E, dtype=torch.int32, **e)
        # slots per (modality, expert), row 0 text, row 1 vision (fused routing)
        self.modality_counts = (torch.empty(2, D.E, dtype=torch.int32, **e)
                                if self.fused_route else None)
        self.offsets = torch.empty(D.E + 2, dtype=torch.int32, **e)
        self.row_token = torch.empty(D.R, dtype=torch.int32, **e)
        self.slot_row = torch.empty(D.S, dtype=torch.int32, **e)
        self.row_weight = torch.empty(D.S, dtype=torch.float32, **e)
        if self.mx:
            self._init_mx(weights, e)
        elif self.mx4:
            self._init_mx4(e)
        elif self.fp8:
            self._init_fp8(e)
        else:
            self.x_perm = torch.empty(D.R, D.d, dtype=torch.bfloat16, **e)
            self.h_perm = torch.empty(D.R, D.I, dtype=torch.bfloat16, **e)
        self.y_perm = torch.empty(D.R, D.d, dtype=torch.bfloat16, **e)
        # fp32 g|u, row-block interleaved in blocks of 32 rows (see moe.h)
        self.gu_save = (torch.empty((D.R + 31) // 32 * 32, 2 * D.I, dtype=torch.float32, **e)
                        if backward and not recompute else None)
        self.y = torch.empty(D.T, D.d, dtype=torch.bfloat16, **e)
        flags = (MOE_FLAG_BACKWARD if backward else 0) | (MOE_FLAG_RECOMPUTE if recompute else 0)
        # the MX backward has a workspace of its own
        ws = _lib.moe_workspace_size(D.T, D.d, D.E, D.k, D.I, 0 if self.mx else flags)
        if ws == 0:
            raise ValueError(f"unsupported layer shape {D}")
        self.ws = torch.empty(ws, dtype=torch.uint8, **e)
        if self.mx and backward:
            wsb = _lib.moe_backward_mx_workspace_size(D.T, D.d, D.E, D.k, D.I, recompute)
            if wsb == 0:
                raise ValueError(f"unsupported layer shape {D}")
            self.ws_bwd = torch.empty(wsb, dtype=torch.uint8, **e)
        if backward:
            self.dX = torch.empty(D.T, D.d, dtype=torch.bfloat16, **e)
            self.dW_g = torch.empty(D.E, D.d, dtype=torch.float32, **e)
            self.dW13 = torch.empty(D.E + 1, 2 * D.I, D.d, dtype=torch.float32, **e)
            self.dW2 = torch.empty(D.E + 1, D.d, D.I, dtype=torch.float32, **e)
            self.dlogits = None
            self.dweights = None
        self._few_ws = {}   # forward_few: a workspace for each number of tokens and stream
        if norm_eps is not None:
            self.norm_eps = float(norm_eps)
            self._init_norm(e)
        if balance is not None:
            self.balance_alpha = float(balance)
            self._init_balance(int(sequences), bool(balance_softmax), e)

    def _init_norm(self, e):
        D = self.dims
        w = self.w.get("norm")
        if w is None or tuple(w.shape) != (D.d,) or w.dtype != torch.float32:
            raise ValueError(f"a layer with norm_eps needs weights['norm'], fp32 [{D.d}]")
        if not norm_supported(D.d):
            raise ValueError(f"moe_rmsnorm does not take rows of {D.d}")
        self.xn = torch.empty(D.T, D.d, dtype=torch.bfloat16, **e)
        self.rstd = torch.empty(D.T, dtype=torch.float32, **e)
        self.residual = self._stream_rows = torch.empty(D.T, D.d, dtype=torch.bfloat16, **e)
        self.xn_q = self.xn_s = None
        if self.mx or self.mx4:
            self._row_format = _lib.MOE_ROWS_MXFP8
            self.xn_q = torch.empty(D.T, D.d, dtype=torch.uint8, **e)
            self.xn_s = torch.empty(D.T, _lib.moe_mx_sf_pitch(D.d), dtype=torch.uint8, **e)
        elif self.fp8:
            self._row_format = _lib.MOE_ROWS_FP8
            self.xn_q = torch.empty(D.T, D.d, dtype=torch.uint8, **e)
            self.xn_s = torch.empty(D.T, _lib.moe_fp8_scale_cols(D.d), dtype=torch.float32, **e)
        else:
            self._row_format = _lib.MOE_ROWS_NONE
        if self.backward_enabled:
            self.dnorm = torch.empty(D.d, dtype=torch.float32, **e)
            self.ws_norm = torch.empty(_lib.moe_rmsnorm_bwd_workspace_size(D.T, D.d),
                                       dtype=torch.uint8, **e)

    def _init_balance(self, n, softmax, e):
        D = self.dims
        f32, i32 = dict(dtype=torch.float32, **e), dict(dtype=torch.int32, **e)
        size = _lib.moe_balance_workspace_size(D.T, D.E, n)
        if size == 0:
            raise ValueError(f"unsupported balance loss of {n} sequences of {D}")
        self.balance_loss = torch.empty(1, **f32)
        self.balance_counts = torch.empty(n, D.E, **i32)
        self.balance_load = torch.empty(n, D.E, **f32)
        self.balance_seq_loss = torch.empty(n, **f32)
        score = _lib.MOE_SCORE_SOFTMAX if softmax else _lib.MOE_SCORE_SIGMOID
        self._balance = dict(
            T=D.T, E=D.E, k=D.k, n_seq=n, score=score, alpha=self.balance_alpha,
            logits=self.logits, ids=self.ids, counts=self.balance_counts,
            tokens=torch.empty(n, **i32), load=self.balance_load, seq_loss=self.balance_seq_loss,
            loss=self.balance_loss, ws=torch.empty(size, dtype=torch.uint8, **e))
        if self.backward_enabled:
            self._balance["dlogits"] = torch.empty(D.T, D.E, **f32)
            size = _lib.moe_gate_bwd_workspace_size(D.T, D.d, D.E)
            if size == 0:
                raise ValueError(f"unsupported balance loss of a training layer of {D}")
            self.ws_gate = torch.empty(size, dtype=torch.uint8, **e)

    def _init_mx4(self, e):
        D = self.dims
        u8 = dict(dtype=torch.uint8, **e)
        pd, pi = _lib.moe_mx_sf_pitch(D.d), _lib.moe_mx_sf_pitch(D.I)
        G = D.E + 1
        shapes = dict(W13_q=(G, 2 * D.I, D.d // 2), W13_sf=(G, 2 * D.I, pd),
                      W2_q=(G, D.d, D.I // 2), W2_sf=(G, D.d, pi))
        given = [n for n in shapes if n in self.w]
        if given and (len(given) < 4 or "W13" in self.w or "W2" in self.w):
            raise ValueError("MXFP4 weights are W13 and W2, or W13_q, W13_sf, W2_q and W2_sf")
        for name, shape in shapes.items():
            t = self.w[name] if given else torch.empty(*shape, **u8)
            if tuple(t.shape) != shape or t.dtype != torch.uint8:
                raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)}, expected uint8 {shape}")
            setattr(self, name, t)
        if not given:
            self.quantize_weights()
        self.x_perm_q = torch.empty(D.R, D.d, **u8)
        self.x_perm_sf = torch.empty(D.R, pd, **u8)
        self.h_q = torch.empty(D.R, D.I, **u8)
        self.h_sf = torch.empty(D.R, pi, **u8)

    def _init_fp8(self, e):
        D = self.dims
        f32, u8 = dict(dtype=torch.float32, **e), dict(dtype=torch.uint8, **e)
        bd, bi = _lib.moe_fp8_scale_cols(D.d), _lib.moe_fp8_scale_cols(D.I)
        G = D.E + 1
        shapes = dict(W13_q=(G, 2 * D.I, D.d), W13_s=(G, 2 * bi, bd), W2_q=(G, D.d, D.I),
                      W2_s=(G, bd, bi))
        given = [n for n in shapes if n in self.w]
        if given and (len(given) < 4 or "W13" in self.w or "W2" in self.w):
            raise ValueError("FP8 weights are W13 and W2, or W13_q, W13_s, W2_q and W2_s")
        for name, shape in shapes.items():
            codes = name.endswith("_q")
            if given:
                t = self.w[name]
                if codes and t.dtype == torch.float8_e4m3fn:
                    t = t.view(torch.uint8)
                if tuple(t.shape) != shape or t.dtype != (torch.uint8 if codes else torch.float32):
                    raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)}, expected {shape}")
            else:
                t = torch.empty(*shape, **(u8 if codes else f32))
            setattr(self, name, t)
        if not given:
            self.quantize_weights()
        self.x_perm_q = torch.empty(D.R, D.d, **u8)
        self.x_perm_s = torch.empty(D.R, bd, **f32)
        self.h_q = torch.empty(D.R, D.I, **u8)
        self.h_s = torch.empty(D.R, bi, **f32)

    def _init_mx(self, weights, e):
        D = self.dims
        u8 = dict(dtype=torch.uint8, **e)
        pd, pi = _lib.moe_mx_sf_pitch(D.d), _lib.moe_mx_sf_pitch(D.I)
        G = D.E + 1
        self.W13_q = torch.empty(G * 2 * D.I, D.d, **u8)
        self.W13_sf = torch.empty(G * 2 * D.I, pd, **u8)
        self.W2_q = torch.empty(G * D.d, D.I, **u8)
        self.W2_sf = torch.empty(G * D.d, pi, **u8)
        if self.backward_enabled:
            # the dgrad matmuls contract over d (W2) and 2I (W13)
            self.W2t_q = torch.empty(G * D.I, D.d, **u8)
            self.W2t_sf = torch.empty(G * D.I, pd, **u8)
            self.W13t_q = torch.empty(G * D.d, 2 * D.I, **u8)
            self.W13t_sf = torch.empty(G * D.d, _lib.moe_mx_sf_pitch(2 * D.I), **u8)
        self.quantize_weights()
        self.x_perm_q = torch.empty(D.R, D.d, **u8)
        self.x_perm_sf = torch.empty(D.R, pd, **u8)
        self.h_q = torch.empty(D.R, D.I, **u8)
        self.h_sf = torch.empty(D.R, pi, **u8)

    def quantize_weights(self, stream=None):
        """(MX, MXFP4 and FP8 layers) Quantise the expert weights from self.w into
        the copies the matmuls read.  MX: along d and I for the forward, and with
        backward also along d (W2) and 2I (W13) for the dgrad matmuls."""
        D = self.dims
        G = D.E + 1
        if "W13" not in self.w:
            raise RuntimeError("the layer was given quantised weights: there are none to quantise")
        W13, W2 = self.w["W13"], self.w["W2"]
        _expect("W13", W13, G, 2 * D.I, D.d)
        _expect("W2", W2, G, D.d, D.I)
        if self.mx4:
            _lib.moe_mx4_quantize(W13, G * 2 * D.I, D.d, self.W13_q, self.W13_sf, stream)
            _lib.moe_mx4_quantize(W2, G * D.d, D.I, self.W2_q, self.W2_sf, stream)
            return
        if self.fp8:
            _lib.moe_fp8_quantize_weights(W13, G, 2 * D.I, D.d, self.W13_q, self.W13_s,
                                          stream=stream)
            _lib.moe_fp8_quantize_weights(W2, G, D.d, D.I, self.W2_q, self.W2_s, stream=stream)
            return
        if self.backward_enabled:
            # one pass over each weight for both copies
            _lib.moe_mx_quantize_both(W13, G, 2 * D.I, D.d, self.W13_q, self.W13_sf,
                                      self.W13t_q, self.W13t_sf, stream)
            _lib.moe_mx_quantize_both(W2, G, D.d, D.I, self.W2_q, self.W2_sf, self.W2t_q,
                                      self.W2t_sf, stream)
            return
        _lib.moe_mx_quantize(W13, G * 2 * D.I, D.d, self.W13_q, self.W13_sf, stream)
        _lib.moe_mx_quantize(W2, G * D.d, D.I, self.W2_q, self.W2_sf, stream)

    # ------------------------------------------------------------ forward
    def route(self, x, bias, is_vision=None, logit_offset=None, mode=MOE_ROUTE_TOPK,
              input_ids=None, tid2eid=None, stream=None):
        D = self.dims
        self._rows("x", x)
        self.x = x       # the backward reads the forward's input
        if self.fused_route:
            _lib.moe_gate_route(x, self.w["W_g"], logit_offset, bias, is_vision, input_ids,
                                tid2eid, D.T, D.d, D.E, D.k, self.scaling, mode, self.logits,
                                self.ids, self.weights, self.scores_sel, self.modality_counts,
                                stream)
        else:
            _lib.moe_route(x, self.w["W_g"], logit_offset, bias, is_vision, input_ids, tid2eid,
                           D.T, D.d, D.E, D.k, self.scaling, mode, self.logits, self.ids,
                           self.weights, self.scores_sel, stream)

    def _rows(self, name, t):
        """T rows of d elements at least, where the tensor is given: what the calls read
        or write, whatever its shape says."""
        D = self.dims
        if t is not None and t.numel() < D.T * D.d:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, the layer has T = {D.T}, d = {D.d}")

    def dispatch(self, x, stream=None, codes=None):
        """The rows x [T, d] to their experts, in the type that the expert matmuls read.
        codes: (codes, scales) of these rows where they are there already, as norm() of
        dims.T rows writes them to (self.xn_q, self.xn_s): those move, and x is not read."""
        D = self.dims
        self._rows("x", x)
        low = self.mx or self.fp8 or self.mx4
        if codes is not None:
            if not low:
                raise ValueError("codes: this layer's expert matmuls read bf16 rows")
            moves = list(zip(codes, (self.x_perm_q,
                                     self.x_perm_s if self.fp8 else self.x_perm_sf)))
            for src, dst in moves:
                if tuple(src.shape) != (D.T, dst.shape[1]) or src.dtype != dst.dtype:
                    raise ValueError(f"codes: {src.dtype} {tuple(src.shape)}, expected "
                                     f"{dst.dtype} {(D.T, dst.shape[1])}")
        _lib.moe_permute(self.ids, self.weights, None if low else x, D.T, D.d, D.E, D.k,
                         self.counts, self.offsets, self.row_token, self.slot_row,
                         self.row_weight, None if low else self.x_perm, self.ws, stream)
        if codes is not None:
            for src, dst in moves:
                _lib.moe_gather_rows(src, self.row_token, dst, stream)
            return
        if self.fp8:
            _lib.moe_fp8_gather(x, self.slot_row, D.T, D.d, D.k, self.x_perm_q, self.x_perm_s,
                                stream)
        if self.mx or self.mx4:
            _lib.moe_mx_gather(x, self.slot_row, D.T, D.d, D.k, self.x_perm_q, self.x_perm_sf,
                               stream)

    def experts(self, stream=None):
        D = self.dims
        if self.mx:
            _lib.moe_expert_ffn_mx(self.x_perm_q, self.x_perm_sf, self.offsets, D.E + 1, D.R,
                                   self.W13_q, self.W13_sf, self.W2_q, self.W2_sf,
                                   self.row_weight, D.S, D.d, D.I, self.clamp, self.h_q,
                                   self.h_sf, self.y_perm, self.gu_save, stream)
            return
        if self.mx4:
            _lib.moe_expert_ffn_mx4(self.x_perm_q, self.x_perm_sf, self.offsets, D.E + 1, D.R,
                                    self.W13_q, self.W13_sf, self.W2_q, self.W2_sf,
                                    self.row_weight, D.S, D.d, D.I, self.clamp, self.h_q,
                                    self.h_sf, self.y_perm, stream)
            return
        if self.fp8:
            _lib.moe_expert_ffn_fp8(self.x_perm_q, self.x_perm_s, self.offsets, D.E + 1, D.R,
                                    self.W13_q, self.W13_s, self.W2_q, self.W2_s,
                                    self.row_weight, D.S, D.d, D.I, self.clamp, self.h_q,
                                    self.h_s, self.y_perm, stream)
            return
        if self.fused_ffn:
            _lib.moe_expert_ffn_fused(self.x_perm, self.offsets, D.E + 1, D.R, self.w["W13"],
                                      self.w["W2"], self.row_weight, D.S, D.d, D.I, self.clamp,
                                      self.gu_save, self.h_perm, self.y_perm, self.ws, stream)
            return
        _lib.moe_expert_ffn(self.x_perm, self.offsets, D.E + 1, D.R, self.w["W13"], self.w["W2"],
                            self.row_weight, D.S, D.d, D.I, self.clamp, self.gu_save,
                            self.h_perm, self.y_perm, None, stream)

    def expert_gemm1(self, stream=None):
        D = self.dims
        if self.fp8 or self.mx4:
            raise RuntimeError("this layer's expert matmuls are one call (experts())")
        if self.mx:
            _lib.moe_expert_gemm1_mx(self.x_perm_q, self.x_perm_sf, self.offsets, D.E + 1, D.R,
                                     self.W13_q, self.W13_sf, D.d, D.I, self.clamp, self.h_q,
                                     self.h_sf, self.gu_save, stream)
            return
        _lib.moe_expert_gemm1(self.x_perm, self.offsets, D.E + 1, D.R, self.w["W13"], D.d, D.I,
                              self.clamp, self.gu_save, self.h_perm, stream)

    def expert_gemm2(self, stream=None):
        D = self.dims
        if self.fp8 or self.mx4:
            raise RuntimeError("this layer's expert matmuls are one call (experts())")
        if self.mx:
            _lib.moe_expert_gemm2_mx(self.h_q, self.h_sf, self.offsets, D.E + 1, D.R, self.W2_q,
                                     self.W2_sf, self.row_weight, D.S, D.d, D.I, self.y_perm,
                                     stream)
            return
        _lib.moe_expert_gemm2(self.h_perm, self.offsets, D.E + 1, D.R, self.w["W2"],
                              self.row_weight, D.S, D.d, D.I, self.y_perm, stream)

    def combine(self, stream=None, y=None):
        D = self.dims
        self._rows("y", y)
        _lib.moe_combine(self.y_perm, self.slot_row, D.T, D.d, D.k, 1,
                         self.y if y is None else y, stream)

    def norm(self, x, residual=None, stream=None):
        """The norm ahead of the layer: (rows [T, d] bf16, the residual stream after the
        addition).  Of dims.T rows into the layer's own buffers, in a low-precision layer
        with their codes and scales (self.xn_q and self.xn_s, for dispatch()); of any other
        number, for forward_few(), new tensors."""
        D = self.dims
        if self.norm_eps is None:
            raise RuntimeError("layer built without norm_eps")
        T = int(x.shape[0])
        _expect("x", x, T, D.d)
        _expect("residual", residual, T, D.d)
        own = T == D.T
        xn = self.xn if own else _result(stream, x.device, T, D.d)
        out = None
        if residual is not None:
            out = self._stream_rows if own else _result(stream, x.device, T, D.d)
        _lib.moe_rmsnorm(dict(
            T=T, d=D.d, eps=self.norm_eps, format=self._row_format if own else _lib.MOE_ROWS_NONE,
            x=x, residual=residual, weight=self.w["norm"], residual_out=out, y=xn,
            rstd=self.rstd if own else None, q=self.xn_q if own else None,
            scales=self.xn_s if own else None), stream)
        out = x if out is None else out
        if own:
            self.residual = out       # the backward reads it
        return xn, out

    def forward(self, x, bias, is_vision=None, logit_offset=None, mode=MOE_ROUTE_TOPK,
                input_ids=None, tid2eid=None, stream=None, y=None, residual=None,
                seq_offsets=None, valid=None):
        """One forward pass; the output goes to self.y, or to `y` ([T, d] bf16)
        when given.  residual [T, d] bf16 (norm_eps layers): the residual stream that x is
        added to.  seq_offsets int32 [sequences + 1], valid uint8 [T] (balance layers): the
        loss's sequences, and which tokens count."""
        D = self.dims
        self._rows("y", y)
        if residual is not None and self.norm_eps is None:
            raise ValueError("residual: the layer was built without norm_eps")
        if self.balance_alpha is None and (seq_offsets is not None or valid is not None):
            raise ValueError("seq_offsets, valid: the layer was built without balance")
        if self.balance_alpha is not None:
            n = self._balance["n_seq"]
            if n != 1 or seq_offsets is not None:
                if seq_offsets is None:
                    raise ValueError(f"seq_offsets: the layer was built for {n} sequences")
                _expect("seq_offsets", seq_offsets, n + 1)
            _expect("valid", valid, D.T)
        if self.norm_eps is not None:
            if int(x.shape[0]) != D.T:
                raise ValueError(f"x: {int(x.shape[0])} rows, the layer has T = {D.T}")
            x, _ = self.norm(x, residual, stream)
        self.route(x, bias, is_vision, logit_offset, mode, input_ids, tid2eid, stream)
        if self.balance_alpha is not None:
            self._balance.update(seq_offsets=seq_offsets, valid=valid)   # (the backward's too)
            _lib.moe_balance_loss(self._balance, stream)
        self.dispatch(x, stream, None if self.norm_eps is None or self.xn_q is None
                      else (self.xn_q, self.xn_s))
        self.experts(stream)
        self.combine(stream, y)
        return self.y if y is None else y

    def forward_few(self, x, bias, is_vision=None, logit_offset=None, mode=MOE_ROUTE_TOPK,
                    input_ids=None, tid2eid=None, stream=None, y=None):
        """The forward of 1 to 32 tokens x [T, d] (any T, not dims.T) through
        moe_layer_few, from the layer's bf16 or FP8 weights; returns y [T, d]
        (a new tensor unless given, of the memory of `stream`).  It routes into
        buffers of its own: ids and weights of the last forward() stay.
        The workspace of a T and a stream is made at its first call and kept.  A
        captured call whose stream has one takes it (replay such a graph in turn
        with that stream's calls); else the graph gets its own, which it zeroes on
        every replay.  See reset_few()."""
        D = self.dims
        if self.mx or self.mx4:
            raise RuntimeError("moe_layer_few takes bf16 or FP8 weights")
        T = int(x.shape[0])
        _expect("x", x, T, D.d)
        _expect("logit_offset", logit_offset, D.E)
        if int(mode) == MOE_ROUTE_TOPK:
            _expect("bias", bias, 2, D.E)
            _expect("is_vision", is_vision, T)
        elif tid2eid is not None:
            _expect("input_ids", input_ids, T)
            _expect("tid2eid", tid2eid, tid2eid.shape[0], D.k)
        _expect("y", y, T, D.d)
        ws = self._few_workspace(T, x.device, stream)
        if y is None:
            y = _result(stream, x.device, T, D.d)
        w = (dict(W13_q=self.W13_q, W13_s=self.W13_s, W2_q=self.W2_q, W2_s=self.W2_s)
             if self.fp8 else dict(W13=self.w["W13"], W2=self.w["W2"]))
        _lib.moe_layer_few(dict(
            T=T, d=D.d, E=D.E, k=D.k, I=D.I, scaling=self.scaling, clamp=self.clamp,
            mode=int(mode), vocab=0 if tid2eid is None else int(tid2eid.shape[0]), x=x,
            W_g=self.w["W_g"], logit_offset=logit_offset, bias=bias, is_vision=is_vision,
            input_ids=input_ids, tid2eid=tid2eid, y=y, ws=ws, **w), stream)
        return y

    def _few_workspace(self, T, device, stream=None):
        key = T, _lib._stream(stream)
        ws = self._few_ws.get(key)
        if ws is None:
            D = self.dims
            n = _lib.moe_few_workspace_size(T, D.d, D.E, D.k, D.I)
            if n == 0:
                raise ValueError(f"moe_layer_few does not take {T} tokens of {D}")
            with torch.cuda.stream(stream):   # (None: the current one)
                ws = torch.zeros(n, dtype=torch.uint8, device=device)
                if not torch.cuda.is_current_stream_capturing():
                    self._few_ws[key] = ws
        return ws

    def reset_few(self):
        """Drops the workspaces of forward_few(), so that its next calls start from
        zeroed ones: after a call that recorded MOE_ERR_TIMEOUT
        (moe_last_device_status), which can leave counters that are not zero."""
        self._few_ws.clear()

    # ----------------------------------------------------------- backward
    def backward(self, dY, want_dlogits=False, want_dweights=False, stream=None,
                 stage_events=None, d_balance=None, d_residual=None):
        """Backward of the last forward; returns dX.  stage_events: optional
        list of MOE_BWD_STAGES + 1 torch.cuda.Event (recorded once before) that
        the library records around each of its stages.  d_balance fp32 [1] (balance
        layers; None: 1): the gradient of the balance loss.  d_residual [T, d] bf16
        (norm_eps layers): the gradient that reaches self.residual past the layer.
        want_dlogits gives the routing weights' part alone."""
        D = self.dims
        if not self.backward_enabled:
            raise RuntimeError("layer built without backward buffers")
        self._rows("dY", dY)
        if d_residual is not None and self.norm_eps is None:
            raise ValueError("d_residual: the layer was built without norm_eps")
        if d_balance is not None and self.balance_alpha is None:
            raise ValueError("d_balance: the layer was built without balance")
        self._rows("d_residual", d_residual)
        _expect("d_balance", d_balance, 1)
        self._experts_backward(dY, want_dlogits, want_dweights, stream, stage_events)
        if self.balance_alpha is not None:
            a = dict(self._balance, dloss=d_balance)
            _lib.moe_balance_loss_backward(a, stream)
            _lib.moe_gate_backward(a["dlogits"], self.x, self.w["W_g"], D.T, D.d, D.E, self.dX,
                                   self.dW_g, self.ws_gate, stream)
        if self.norm_eps is not None:
            _lib.moe_rmsnorm_backward(dict(
                T=D.T, d=D.d, x=self.residual, weight=self.w["norm"], rstd=self.rstd, dy=self.dX,
                d_residual=d_residual, dx=self.dX, d_weight=self.dnorm, ws=self.ws_norm), stream)
        return self.dX

    def _experts_backward(self, dY, want_dlogits, want_dweights, stream, stage_events):
        D = self.dims
        if want_dlogits and self.dlogits is None:
            self.dlogits = torch.empty(D.T, D.E, dtype=torch.float32, device=dY.device)
        if want_dweights and self.dweights is None:
            self.dweights = torch.empty(D.T, D.k, dtype=torch.float32, device=dY.device)
        if self.mx:
            _lib.moe_backward_mx(dict(
                T=D.T, d=D.d, E=D.E, k=D.k, I=D.I, scaling=self.scaling, clamp=self.clamp,
                x=self.x, W_g=self.w["W_g"], W13_q=self.W13_q, W13_sf=self.W13_sf,
                W2t_q=self.W2t_q, W2t_sf=self.W2t_sf, W13t_q=self.W13t_q, W13t_sf=self.W13t_sf,
                ids=self.ids, weights=self.weights, scores_sel=self.scores_sel,
                row_weight=self.row_weight, offsets=self.offsets, row_token=self.row_token,
                slot_row=self.slot_row, x_perm_q=self.x_perm_q, x_perm_sf=self.x_perm_sf, gu_save=self.gu_save,
                h_q=None if self.recompute else self.h_q,
                h_sf=None if self.recompute else self.h_sf,
                dY=dY, dX=self.dX, dW_g=self.dW_g, dW13=self.dW13, dW2=self.dW2,
                dlogits=self.dlogits if want_dlogits else None,
                dweights=self.dweights if want_dweights else None, ws=self.ws_bwd,
                stage_events=stage_events), stream)
            return
        args = dict(T=D.T, d=D.d, E=D.E, k=D.k, I=D.I, scaling=self.scaling, clamp=self.clamp,
                    flags=MOE_FLAG_RECOMPUTE if self.recompute else 0,
                    x=self.x, W_g=self.w["W_g"], W13=self.w["W13"], W2=self.w["W2"],
                    ids=self.ids, weights=self.weights, scores_sel=self.scores_sel,
                    row_weight=self.row_weight, offsets=self.offsets, row_token=self.row_token,
                    slot_row=self.slot_row,
                    x_perm=None if self.recompute else self.x_perm,
                    gu_save=None if self.recompute else self.gu_save,
                    dY=dY, dX=self.dX, dW_g=self.dW_g, dW13=self.dW13, dW2=self.dW2,
                    dlogits=self.dlogits if want_dlogits else None,
                    dweights=self.dweights if want_dweights else None, ws=self.ws,
                    stage_events=stage_events)
        _lib.moe_backward(args, stream)

    # ------------------------------------------------- steps from host memory
    def step_host(self, x_host, y_host, dY_host=None, dX_host=None, bias=None, is_vision=None,
                  logit_offset=None, mode=MOE_ROUTE_TOPK, input_ids=None, tid2eid=None,
                  stream=None, copy_stream=None):
        """One step from and to host memory through moe_layer_step_host: x_host
        ([T,d] bf16, pinned CPU) in, y_host out; with dY_host / dX_host also the
        backward (dX out, weight gradients in self.dW13 / dW2 / dW_g).  The
        routing inputs are device tensors as for forward()."""
        self._ensure_host_struct(dY_host is not None, bias, is_vision, logit_offset, mode,
                                 input_ids, tid2eid)
        self.x = self.x_dev
        _lib.moe_layer_step_host(self._host_struct, x_host, dY_host, y_host, dX_host, stream,
                                 copy_stream)

    def steps_host(self, x_hosts, y_hosts, dY_hosts=None, dX_hosts=None, bias=None,
                   is_vision=None, logit_offset=None, mode=MOE_ROUTE_TOPK, input_ids=None,
                   tid2eid=None, stream=None, copy_in_stream=None, copy_out_stream=None):
        """len(x_hosts) steps from and to host memory through
        moe_layer_steps_host, pipelined: the next step's uploads and the last
        step's downloads overlap the compute (lists of pinned CPU [T,d] bf16
        tensors; dY_hosts / dX_hosts for training steps)."""
        D = self.dims
        self._ensure_host_struct(dY_hosts is not None, bias, is_vision, logit_offset, mode,
                                 input_ids, tid2eid)
        if getattr(self, "_io2", None) is None:
            mk = lambda: torch.empty(D.T, D.d, dtype=torch.bfloat16, device=self.y.device)
            self._io2 = dict(x=mk(), y=mk(), dY=mk() if self.backward_enabled else None,
                             dX=mk() if self.backward_enabled else None)
        _lib.moe_layer_steps_host(self._host_struct, self._io2, x_hosts, dY_hosts, y_hosts,
                                  dX_hosts, stream, copy_in_stream, copy_out_stream)

    def _ensure_host_struct(self, train, bias, is_vision, logit_offset, mode, input_ids,
                            tid2eid):
        D = self.dims
        if self.mx or self.fp8 or self.mx4 or self.norm_eps is not None \
                or self.balance_alpha is not None:
            raise RuntimeError("the host-memory steps run the plain bf16 layer")
        if train and not self.backward_enabled:
            raise RuntimeError("layer built without backward buffers")
        key = (id(bias), id(is_vision), id(logit_offset), mode, id(input_ids), id(tid2eid))
        if getattr(self, "_host_key", None) != key:
            dev = self.y.device
            if getattr(self, "x_dev", None) is None:
                self.x_dev = torch.empty(D.T, D.d, dtype=torch.bfloat16, device=dev)
            if self.backward_enabled and getattr(self, "dY_dev", None) is None:
                self.dY_dev = torch.empty(D.T, D.d, dtype=torch.bfloat16, device=dev)
            self._host_refs = (bias, is_vision, logit_offset, input_ids, tid2eid)
            self._host_struct = _lib.layer_buffers(dict(
                T=D.T, d=D.d, E=D.E, k=D.k, I=D.I, scaling=self.scaling, clamp=self.clamp,
                flags=MOE_FLAG_RECOMPUTE if self.recompute else 0, mode=int(mode),
                W_g=self.w["W_g"], W13=self.w["W13"], W2=self.w["W2"],
                logit_offset=logit_offset, bias=bias, is_vision=is_vision, input_ids=input_ids,
                tid2eid=tid2eid, vocab=0 if tid2eid is None else int(tid2eid.shape[0]),
                x=self.x_dev, y=self.y,
                dY=self.dY_dev if self.backward_enabled else None,
                dX=self.dX if self.backward_enabled else None,
                logits=self.logits, ids=self.ids, weights=self.weights,
                scores_sel=self.scores_sel, modality_counts=self.modality_counts,
                counts=self.counts, offsets=self.offsets, row_token=self.row_token,
                slot_row=self.slot_row, row_weight=self.row_weight, x_perm=self.x_perm,
                h_perm=self.h_perm, y_perm=self.y_perm, gu_save=self.gu_save,
                dW_g=getattr(self, "dW_g", None), dW13=getattr(self, "dW13", None),
                dW2=getattr(self, "dW2", None), ws=self.ws))
            self._host_key = key


class GroupedLinearFP8:
    """One projection per group (expert), y[r] = x[r] W[g]^T for the rows of
    group g, with its three products in FP8 (E4M3, one fp32 scale per 128): the
    forward, the data gradient (the same matmul on the weight's transposed
    copy) and the weight gradient.

    weight: bf16 [G, N, K] (CUDA), quantised here in both orientations; again
    with quantize_weights() after it changes.  G = 1 is a dense layer.  rows:
    the most rows of a call.  offsets: int32 [G+1] on the device, the groups'
    first rows (as moe_permute writes them), the last one the number of rows.
    The buffers for the quantised rows x of a stream are made at its first call and
    kept, so that forward calls on several streams may run at once; a captured call
    has its own.  The backward is that of the last forward, whichever its stream.
    """

    def __init__(self, weight, rows: int):
        self.weight = weight
        G, N, K = self.G, self.N, self.K = tuple(map(int, weight.shape))
        self.rows = int(rows)
        n = _lib.moe_fp8_wgrad_workspace_size(G, self.rows, N, K)
        if N % 16 or K % 16 or n == 0:
            raise ValueError(f"unsupported FP8 projection [{G}, {N}, {K}] of {rows} rows")
        bn, bk = _lib.moe_fp8_scale_cols(N), _lib.moe_fp8_scale_cols(K)
        dev = weight.device
        u8, f32 = dict(dtype=torch.uint8, device=dev), dict(dtype=torch.float32, device=dev)
        self.w_q, self.w_s = torch.empty(G, N, K, **u8), torch.empty(G, bn, bk, **f32)
        self.wt_q, self.wt_s = torch.empty(G, K, N, **u8), torch.empty(G, bk, bn, **f32)
        self._buffers = _StreamBuffers(dev, ((self.rows, K), torch.uint8),
                                       ((self.rows, bk), torch.float32))
        self.dy_q, self.dy_s = torch.empty(rows, N, **u8), torch.empty(rows, bn, **f32)
        self.dW = torch.empty(G, N, K, **f32)
        self.ws = torch.empty(n, **u8)
        self.x = self.offsets = None
        self.quantize_weights()

    def quantize_weights(self, stream=None):
        _expect("weight", self.weight, self.G, self.N, self.K)
        _lib.moe_fp8_quantize_weights(self.weight, self.G, self.N, self.K, self.w_q, self.w_s,
                                      self.wt_q, self.wt_s, stream)

    def forward(self, x, offsets, stream=None):
        """y [R, N] bf16 of the rows x [R, K] bf16, R <= rows.  With `stream` the work and
        y's memory belong to that stream; the backward too then takes it."""
        R = int(x.shape[0])
        _expect("x", x, R, self.K)
        _expect("offsets", offsets, self.G + 1)
        if R > self.rows:
            raise ValueError(f"{R} rows, the buffers hold {self.rows}")
        self.x, self.offsets = x, offsets   # the backward reads them
        y = _result(stream, x.device, R, self.N)
        if R == 0:
            return y
        x_q, x_s = self._buffers.of(stream)
        _lib.moe_fp8_quantize(x, R, self.K, x_q, x_s, stream)
        _lib.moe_fp8_matmul(x_q, x_s, offsets, self.G, R, self.w_q, self.w_s, None, 0, self.N,
                            self.K, y, stream)
        return y

    def backward(self, dy, stream=None):
        """dX [R, K] bf16 of the last forward; self.dW [G, N, K] fp32."""
        if self.x is None:
            raise RuntimeError("backward() before a forward()")
        R = int(self.x.shape[0])
        _expect("dy", dy, R, self.N)
        if int(dy.shape[0]) != R:
            raise ValueError(f"dy: {int(dy.shape[0])} rows, the forward had {R}")
        dx = _result(stream, dy.device, R, self.K)
        if R == 0:
            with torch.cuda.stream(stream):   # (None: the current one)
                self.dW.zero_()
            return dx
        _lib.moe_fp8_quantize(dy, R, self.N, self.dy_q, self.dy_s, stream)
        _lib.moe_fp8_matmul(self.dy_q, self.dy_s, self.offsets, self.G, R, self.wt_q, self.wt_s,
                            None, 0, self.K, self.N, dx, stream)
        _lib.moe_fp8_wgrad(dy, self.x, self.offsets, self.G, R, self.N, self.K, self.dW, self.ws,
                           stream)
        return dx


class GroupedLinearMX4:
    """One projection per group (expert) for serving, y[r] = x[r] W[g]^T for the rows of
    group g, with MXFP4 weights (4-bit elements, one power of two per 32).

    weight: bf16 [G, N, K] (CUDA), quantised here; again with quantize_weights() after it
    changes.  Or codes=(w_q, w_sf), uint8 [G, N, K/2] and [G, N, moe_mx_sf_pitch(K)], with
    weight None.  G = 1 is a dense layer.  rows: the most rows of a call.  bits: of the rows,
    which each call quantises: 8 (MXFP8, K % 128 == 0) or 4 (MXFP4, K % 32 == 0: twice the
    tensor rate, with the rows' rounding errors those of the weights).  The buffers for the
    quantised rows of a stream are made at its first call and kept, so that calls on several
    streams may run at once; a captured call has its own."""

    def __init__(self, weight, rows: int, bits: int = 8, codes=None):
        if (weight is None) == (codes is None):
            raise ValueError("GroupedLinearMX4 takes a weight, or its codes and scales")
        if bits not in (4, 8):
            raise ValueError(f"rows of {bits} bits: 4 or 8")
        G, N, K = map(int, weight.shape if codes is None else codes[0].shape)
        if codes is not None:
            K *= 2
        if G < 1 or G > 1025 or N % 8 or K < 32 or K % (32 if bits == 4 else 128):
            raise ValueError(f"unsupported MXFP4 projection [{G}, {N}, {K}] on {bits}-bit rows")
        self.weight, self.G, self.N, self.K, self.rows, self.bits = weight, G, N, K, int(rows), bits
        pitch = _lib.moe_mx_sf_pitch(K)
        u8 = dict(dtype=torch.uint8, device=(codes[0] if weight is None else weight).device)
        if codes is None:
            self.w_q, self.w_sf = torch.empty(G, N, K // 2, **u8), torch.empty(G, N, pitch, **u8)
            self.quantize_weights()
        else:
            self.w_q, self.w_sf = codes
            _expect("codes", self.w_sf, G, N, pitch)
        self._buffers = _StreamBuffers(
            self.w_q.device, ((self.rows, K if bits == 8 else K // 2), torch.uint8),
            ((self.rows, pitch), torch.uint8))

    def quantize_weights(self, stream=None):
        if self.weight is None:
            raise RuntimeError("the projection was given quantised weights")
        _expect("weight", self.weight, self.G, self.N, self.K)
        _lib.moe_mx4_quantize(self.weight, self.G * self.N, self.K, self.w_q, self.w_sf, stream)

    def forward(self, x, offsets, stream=None, row_weight=None):
        """y [R, N] bf16 of the rows x [R, K] bf16, R <= rows; offsets int32 [G+1] on the
        device, the groups' first rows, the last one R.  row_weight fp32 [R]: factors of the
        rows.  With `stream` the work and y's memory belong to that stream."""
        R = int(x.shape[0])
        _expect("x", x, R, self.K)
        _expect("offsets", offsets, self.G + 1)
        _expect("row_weight", row_weight, R)
        if R > self.rows:
            raise ValueError(f"{R} rows, the buffers hold {self.rows}")
        y = _result(stream, x.device, R, self.N)
        if R == 0:
            return y
        quantize = _lib.moe_mx_quantize if self.bits == 8 else _lib.moe_mx4_quantize
        x_q, x_sf = self._buffers.of(stream)
        quantize(x, R, self.K, x_q, x_sf, stream)
        _lib.moe_mx4_matmul(x_q, x_sf, self.bits, offsets, self.G, R, self.w_q, self.w_sf,
                            row_weight, R, self.N, self.K, y, stream)
        return y


__all__ = ["Dims", "GroupedLinearFP8", "GroupedLinearMX4", "MoELayer", "MOE_ROUTE_TOPK", "MOE_ROUTE_HASH"]


class HostPipeline:
    """Forward passes over batches that live in pinned host memory.

    Each batch is copied to the device, run through the layer, and its output
    copied back.  Two device buffers each way and one copy stream per
    direction let batch i+1's host-to-device copy and batch i-1's
    device-to-host copy run while the layer computes batch i, so a sequence
    of batches costs about the compute alone; every batch still makes both
    copies.  Batches run in order on the caller's current stream, which
    afterwards also waits for the last copy back.
    """

    def __init__(self, layer: MoELayer):
        D = layer.dims
        dev = layer.y.device
        self.layer = layer
        self.x_dev = [torch.empty(D.T, D.d, dtype=torch.bfloat16, device=dev) for _ in range(2)]
        self.y_dev = [torch.empty(D.T, D.d, dtype=torch.bfloat16, device=dev) for _ in range(2)]
        self.h2d = torch.cuda.Stream(dev)
        self.d2h = torch.cuda.Stream(dev)
        self.x_ready = [torch.cuda.Event() for _ in range(2)]
        self.x_free = [torch.cuda.Event() for _ in range(2)]
        self.y_ready = [torch.cuda.Event() for _ in range(2)]
        self.y_free = [torch.cuda.Event() for _ in range(2)]

    def _copy_in(self, i, x_host):
        b = i % 2
        with torch.cuda.stream(self.h2d):
            self.h2d.wait_event(self.x_free[b])      # batch i-2 no longer reads x_dev[b]
            self.x_dev[b].copy_(x_host, non_blocking=True)
            self.x_ready[b].record(self.h2d)

    def run(self, xs_host, ys_host, bias, is_vision=None, logit_offset=None, **route_kw):
        """xs_host[i] ([T, d] bf16, pinned) -> layer -> ys_host[i] (pinned)."""
        comp = torch.cuda.current_stream(self.layer.y.device)
        # the copies start after everything the caller queued before
        self.h2d.wait_stream(comp)
        self.d2h.wait_stream(comp)
        n = len(xs_host)
        if n:
            self._copy_in(0, xs_host[0])
        for i in range(n):
            b = i % 2
            if i + 1 < n:
                self._copy_in(i + 1, xs_host[i + 1])
            comp.wait_event(self.x_ready[b])
            comp.wait_event(self.y_free[b])          # batch i-2's output has left y_dev[b]
            self.layer.forward(self.x_dev[b], bias, is_vision, logit_offset, y=self.y_dev[b],
                               **route_kw)
            self.x_free[b].record(comp)
            self.y_ready[b].record(comp)
            with torch.cuda.stream(self.d2h):
                self.d2h.wait_event(self.y_ready[b])
                ys_host[i].copy_(self.y_dev[b], non_blocking=True)
                self.y_free[b].record(self.d2h)
        comp.wait_stream(self.d2h)
