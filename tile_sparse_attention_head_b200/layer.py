"""The operators on both sides of the tile-sparse attention in a transformer
layer, as torch functions over the C ABI, and the attention block they form.

    h, y8 = add_rms_norm_fp8(x, delta)      residual + RMS norm, e4m3 with a scale per 128 channels
    qkv   = gemm_fp8(y8, Wqkv)              8-bit product, a scale per block of 128
    q, k, v = qkv_norm_rope(qkv)            Q/K norm, three-axis rotary positions, grid order
    o     = VedaAttention(q, k, v)
    delta = gemm_fp8(quant_fp8_heads(o), Wo)

``add_rms_norm`` and ``qkv_norm_rope`` are differentiable torch ops (their
backward runs in the library); the 8-bit forms are for inference and refuse
inputs that ask for a gradient.  ``VedaSelfAttention`` chains the calls.
Everything runs on the current stream of the tensors' device, and can be
captured into a CUDA graph; a captured ``backward()`` wants, as with torch's own
operators, that no eager graph of the same leaves is alive (torch raises
otherwise; ``torch.autograd.grad`` has no such condition).
"""
from __future__ import annotations

from typing import Optional, Sequence, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import binding as B


def _wants_grad(*tensors) -> bool:
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    return False


def _no_grad_inputs(func: str, *tensors) -> None:
    if _wants_grad(*tensors):
        raise ValueError(f"{func} is an inference operator: it has no gradient (call it under torch.no_grad())")


def _flat(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """[..., C] as rows [R, C] that the library can read in place: contiguous channels, 16-byte aligned rows that do
    not overlap; a copy only where the tensor is not like that (a broadcast one, or one that starts elsewhere)."""
    if t is None:
        return None
    if t.dim() != 2:
        t = t.reshape(t.numel() // t.shape[-1] if t.dim() and t.shape[-1] else 0, t.shape[-1] if t.dim() else 0)
    if t.is_contiguous():
        return t.clone() if t.data_ptr() & 15 else t
    rows, C = t.shape
    stride, step = t.stride()
    fits = t.data_ptr() % 16 == 0 and (step == 1 or C == 1) and (rows == 1 or (stride >= C and stride % 8 == 0))
    return t if fits else t.contiguous()


def _dense(t: Optional[torch.Tensor], shape, dtype: Optional[torch.dtype] = None) -> Optional[torch.Tensor]:
    """An upstream gradient as the library reads it: dense, 16-byte aligned, of `shape`."""
    if t is None:
        return None
    if dtype is not None and t.dtype is not dtype:
        t = t.to(dtype)
    if t.shape != shape:
        t = t.reshape(shape)
    if not t.is_contiguous():
        t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _check_stream_and_delta(x: torch.Tensor, delta: Optional[torch.Tensor]) -> None:
    if delta is not None and delta.shape != x.shape:
        raise ValueError(f"delta must have x's shape {tuple(x.shape)} (got {tuple(delta.shape)})")


# ---------------------------------------------------------------- residual and norm

def _norm_forward(x, delta, weight, eps):
    """Of rows x and delta; outputs are allocated like them (dense: an empty_like of rows with gaps has none)."""
    if delta is None:
        h, y = None, torch.empty_like(x)
    else:
        h, y = torch.empty_like(x), torch.empty_like(delta)
    B._layer_norm_forward(x, delta, weight, eps, h, y, None)
    return h, y


def _once(backward):
    """backward, with once_differentiable's guard only where a graph of the gradient is asked for (it costs several
    microseconds a call)."""
    guarded = once_differentiable(backward)

    def run(ctx, *grads):
        return guarded(ctx, *grads) if torch.is_grad_enabled() else backward(ctx, *grads)
    return run


class _AddRmsNorm(torch.autograd.Function):
    """(h, y) of residual addition and RMS norm; without a delta, y alone."""

    @staticmethod
    def forward(ctx, x, delta, weight, eps):
        x2, d2 = _flat(x), _flat(delta)
        h, y = _norm_forward(x2, d2, weight, eps)
        ctx.set_materialize_grads(False)
        ctx.like = None if delta is None else delta.dtype
        ctx.eps = eps
        if h is None:
            ctx.save_for_backward(x2 if x2.is_contiguous() else x2.contiguous(), weight)
            return y if x.dim() == 2 else y.view(x.shape)
        ctx.save_for_backward(h, weight)
        return (h, y) if x.dim() == 2 else (h.view(x.shape), y.view(x.shape))

    @staticmethod
    @_once
    def backward(ctx, *grads):
        h, weight = ctx.saved_tensors
        dh, dy = grads if len(grads) == 2 else (None, grads[0])
        want_x, want_d, want_w, _ = ctx.needs_input_grad
        if dy is None:   # only the sum itself was used: its gradient goes to both addends
            return dh if want_x else None, None if dh is None or not want_d else dh.to(ctx.like), None, None
        shape = dy.shape
        dy, dh = _dense(dy, h.shape), _dense(dh, h.shape)
        same = dy.dtype is h.dtype
        dx = torch.empty_like(h) if want_x or (want_d and same) else None
        dd = torch.empty_like(dy) if want_d and not same else None
        dw = torch.empty_like(weight) if want_w else None
        B._layer_norm_backward(h, dy, dh, weight, ctx.eps, dx, dd, dw)
        if len(shape) != 2:
            dx, dd = None if dx is None else dx.view(shape), None if dd is None else dd.view(shape)
        return dx if want_x else None, (dx if same else dd) if want_d else None, dw, None


def add_rms_norm(x: torch.Tensor, delta: Optional[torch.Tensor], weight: torch.Tensor,
                 eps: float = 1e-6) -> Tuple[torch.Tensor, torch.Tensor]:
    """(h, y): h = x + delta in x's type and y = h * (mean_c h^2 + eps)^(-1/2) * weight in delta's type.

    x and delta [..., C] of one type (bf16, fp16, fp32), or an fp32 residual
    stream x with a bf16 delta; weight [C] fp32.  delta None: h is x.  The norm
    is taken of the rounded h.  Differentiable in x, delta and weight."""
    _check_stream_and_delta(x, delta)
    if not _wants_grad(x, delta, weight):
        h, y = _norm_forward(_flat(x), _flat(delta), weight, eps)
        if x.dim() != 2:
            h, y = None if h is None else h.view(x.shape), y.view(x.shape)
        return (x if h is None else h), y
    if delta is None:
        return x, _AddRmsNorm.apply(x, None, weight, eps)
    return _AddRmsNorm.apply(x, delta, weight, eps)


def add_rms_norm_fp8(x: torch.Tensor, delta: Optional[torch.Tensor], weight: torch.Tensor,
                     eps: float = 1e-6) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(h, y8, y_scale): add_rms_norm with y as e4m3 rows [R, C] and scales [ceil(C/128), R] for gemm_fp8."""
    _no_grad_inputs("add_rms_norm_fp8", x, delta, weight)
    _check_stream_and_delta(x, delta)
    x2, d2 = _flat(x), _flat(delta)
    rows, C = x2.shape
    h = torch.empty_like(x2) if delta is not None else None
    y8 = torch.empty_like(x2, dtype=B.FP8)
    scale = x2.new_empty(((C + 127) // 128, rows), dtype=torch.float32)
    B._layer_norm_forward(x2, d2, weight, eps, h, y8, scale)
    return x if h is None else h if x.dim() == 2 else h.view(x.shape), y8, scale


# ---------------------------------------------------------------- 8-bit product

def quant_fp8(x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """[..., C] -> e4m3 rows [R, C] and a scale per row and 128 channels, [ceil(C/128), R]."""
    _no_grad_inputs("quant_fp8", x)
    return _quant(_flat(x))


def quant_fp8_heads(o: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """The attention's grid-order output [B, heads, N, d] -> e4m3 rows [B*N, heads*d] and their scales."""
    _no_grad_inputs("quant_fp8_heads", o)
    if o.dim() != 4:
        raise ValueError("o must be [B, heads, N, d]")
    return _quant(o)


def _quant(x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    rows, C = x.shape if x.dim() == 2 else (x.shape[0] * x.shape[2], x.shape[1] * x.shape[3])
    q = x.new_empty((rows, C), dtype=B.FP8)
    scale = x.new_empty(((C + 127) // 128, rows), dtype=torch.float32)
    B.veda_quant_fp8(x, q, scale)
    return q, scale


def quant_fp8_weight(w: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """A linear layer's weight [N, K] -> e4m3 and a scale per 128 x 128 block, [ceil(N/128), ceil(K/128)]."""
    w = w.detach().contiguous()
    q = torch.empty(w.shape, dtype=B.FP8, device=w.device)
    scale = torch.empty(((w.shape[0] + 127) // 128, (w.shape[1] + 127) // 128), dtype=torch.float32, device=w.device)
    B.veda_quant_fp8_weight(w, q, scale)
    return q, scale


def gemm_fp8(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
             bias: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
             out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """[M, N] = a [M, K] @ b [N, K]^T (+ bias fp32 [N]) of e4m3 operands with a scale for each block of 128."""
    _no_grad_inputs("gemm_fp8", a, a_scale, b, b_scale, bias)
    if out is None:
        return B._layer_gemm(a, a_scale, b, b_scale, bias, out_dtype)
    return B.veda_gemm_fp8(a, a_scale, b, b_scale, bias, out)


# ---------------------------------------------------------------- rotary positions

def rope_table(n: int, dim: int, theta: float = 10000.0, start: float = 0.0, step: float = 1.0,
               device="cuda") -> torch.Tensor:
    """(cos, sin) of n positions start + step*i for one axis of `dim` channels: fp32 [n, dim/2, 2], angles in fp64."""
    if dim % 2:
        raise ValueError(f"dim must be even (got {dim})")
    return B.veda_rope_table(torch.empty((n, dim // 2, 2), dtype=torch.float32, device=device), theta, start, step)


def rope_tables(grid: Sequence[int], dims: Sequence[int], theta: float = 10000.0,
                start: Sequence[float] = (0.0, 0.0, 0.0), step: Sequence[float] = (1.0, 1.0, 1.0),
                device="cuda") -> Tuple[Optional[torch.Tensor], ...]:
    """The (time, height, width) tables of a grid; dims: channels of each axis (None for an axis with none)."""
    return tuple(rope_table(n, dim, theta, a, b, device) if dim else None
                 for n, dim, a, b in zip(grid, dims, start, step))


class _QkvNormRope(torch.autograd.Function):
    """q, k, v in grid order from one packed tensor or from three."""

    @staticmethod
    def forward(ctx, rope, tables, how, wq, wk, *xs):
        q, k, v = xs[0].unbind(2) if len(xs) == 1 else xs
        shape = (rope.B, rope.heads, q.shape[1], rope.d)
        outs = tuple(q.new_empty(shape, dtype=torch.bfloat16) for _ in range(3))
        B.veda_qkv_norm_rope(rope, q, k, v, wq, wk, *outs)
        # rope holds the tables' addresses, which are this call's: backward may get other tensors (a checkpoint computes
        # the tables again, a hook moves them) and makes a struct of its own.
        ctx.sizes, ctx.how, ctx.packed = (rope.B, rope.heads, rope.d), how, len(xs) == 1
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(wq, wk, *tables, *xs)
        return outs

    @staticmethod
    @_once
    def backward(ctx, *douts):
        wq, wk, *rest = ctx.saved_tensors
        tables, xs = rest[:3], rest[3:]
        grid, pairing, norm, eps = ctx.how
        rope = B.make_rope(*ctx.sizes, grid, tables, pairing, norm, eps)
        want_wq, want_wk, *want_x = ctx.needs_input_grad[3:]
        q, k, v = xs[0].unbind(2) if ctx.packed else xs
        want = want_x * 3 if ctx.packed else want_x
        # An operand is gone through for its own gradient or its weight's (its own is written then all the same).
        need = [g is not None and (w or ww) for g, w, ww in zip(douts, want, (want_wq, want_wk, False))]
        packed = None
        if ctx.packed and want[0]:
            packed = torch.empty(xs[0].shape, dtype=q.dtype, device=q.device)
            for i, g in enumerate(douts):
                if g is None:
                    packed[:, :, i].zero_()
            dxs = list(packed.unbind(2))
        else:
            dxs = [torch.empty(q.shape, dtype=q.dtype, device=q.device) if n else None for n in need]
        if any(need):
            shape = (rope.B, rope.heads, q.shape[1], rope.d)
            d = [_dense(g, shape, torch.bfloat16) if n else None for g, n in zip(douts, need)]
            dwq = torch.empty_like(wq) if want_wq and need[0] else None
            dwk = torch.empty_like(wk) if want_wk and need[1] else None
            ws = None
            if dwq is not None or dwk is not None:
                ws = q.new_empty(B.veda_qkv_norm_rope_backward_workspace(rope, q.get_device()), dtype=torch.uint8)
            B.veda_qkv_norm_rope_backward(rope, q, k, wq, wk, *d, *(x if n else None for x, n in zip(dxs, need)),
                                          dwq, dwk, ws)
        else:
            dwq = dwk = None
        dx = (packed,) if ctx.packed else tuple(x if w else None for x, w in zip(dxs, want_x))
        return (None, None, None, dwq, dwk) + dx


def qkv_norm_rope(qkv, grid: Sequence[int], tables: Sequence[Optional[torch.Tensor]],
                  wq: Optional[torch.Tensor] = None, wk: Optional[torch.Tensor] = None, norm: str = "row",
                  eps: float = 1e-6,
                  pairing: str = "interleaved") -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """q, k, v [B, heads, N, d] bf16 for the attention from the QKV product.

    qkv: one packed tensor [B, N, 3, heads, d], or (q, k, v), each [B, N, heads,
    d]; bf16, fp16 or fp32, channels contiguous, other strides free multiples of
    8.  grid: (T, H, W) with N = T*H*W.  tables: (cos, sin) per axis (rope_tables);
    a table from a later row on moves the grid along that axis.  norm: RMS norm
    of q and k over all channels of a token ("row", weights [heads*d] fp32), over
    each head ("head", weights [d]) or "none".  pairing: "interleaved" or
    "halves" of each axis's channels.  Differentiable in qkv, wq and wk; tables
    that want a gradient are refused."""
    if isinstance(qkv, torch.Tensor):
        if qkv.dim() != 5 or qkv.shape[2] != 3:
            raise ValueError(f"qkv must be [B, N, 3, heads, d] (got {tuple(qkv.shape)})")
        xs = (qkv,)
        b, n, _, heads, d = qkv.shape
    else:
        xs = tuple(qkv)
        if len(xs) != 3 or any(t.dim() != 4 for t in xs):
            raise ValueError("qkv must be a packed tensor or (q, k, v), each [B, N, heads, d]")
        b, n, heads, d = xs[0].shape
    if len(grid) != 3 or n != grid[0] * grid[1] * grid[2]:
        raise ValueError(f"N = {n} tokens do not fill the grid {grid}")
    if norm != "none" and (wq is None or wk is None):
        raise ValueError(f"norm {norm!r} needs wq and wk")
    if norm == "none" and (wq is not None or wk is not None):
        raise ValueError("norm 'none' takes no weights")
    for t in tables:
        if t is not None and t.get_device() != xs[0].get_device():
            raise ValueError(f"a table is on {t.device}, qkv on {xs[0].device}")
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError("the tables have no gradient (detach them, or call it under torch.no_grad())")
    rope = B.make_rope(b, heads, d, grid, tables, pairing, norm, eps)
    if _wants_grad(wq, wk, *xs):
        return _QkvNormRope.apply(rope, tuple(tables), (tuple(grid), pairing, norm, eps), wq, wk, *xs)
    if len(xs) == 1:      # one allocation: with three a call on one token is a tenth slower
        outs = qkv.new_empty((3, b, heads, n, d), dtype=torch.bfloat16).unbind(0)
        B._packed_norm_rope(rope, qkv, wq, wk, outs)
    else:
        outs = tuple(xs[0].new_empty((b, heads, n, d), dtype=torch.bfloat16) for _ in range(3))
        B.veda_qkv_norm_rope(rope, *xs, wq, wk, *outs)
    return outs


# ---------------------------------------------------------------- the attention block

class VedaSelfAttention:
    """The attention block of a video transformer layer for inference, in 8-bit products:

        (x, delta) -> h = x + delta;  out = Wo attention(norm(h) Wqkv^T)

    ``attention`` is a VedaAttention; weights are given in bf16, fp16 or fp32
    and laid out in e4m3 once: w_qkv [3*heads*d, C], w_o [C, heads*d], biases fp32
    or None, norm_weight [C], wq and wk the Q/K norm's weights (see qkv_norm_rope).
    The residual stream x is bf16, fp16 or fp32 and goes through unchanged in
    type; ``out`` (bf16) is the delta of the next block.  With an fp16 stream a
    bf16 delta is brought to fp16 first: exact in fp16's normal range, to its
    step 2^-24 below, infinite above."""

    def __init__(self, attention, w_qkv: torch.Tensor, w_o: torch.Tensor, norm_weight: torch.Tensor,
                 tables: Sequence[Optional[torch.Tensor]], wq: Optional[torch.Tensor] = None,
                 wk: Optional[torch.Tensor] = None, b_qkv: Optional[torch.Tensor] = None,
                 b_o: Optional[torch.Tensor] = None, norm: str = "row", eps: float = 1e-6,
                 pairing: str = "interleaved"):
        p = attention.p
        inner, C = p.heads * p.d, norm_weight.shape[0]
        if tuple(w_qkv.shape) != (3 * inner, C) or tuple(w_o.shape) != (C, inner):
            raise ValueError(f"w_qkv must be [{3 * inner}, {C}] and w_o [{C}, {inner}] "
                             f"(got {tuple(w_qkv.shape)} and {tuple(w_o.shape)})")
        if C % 16:
            raise ValueError(f"C must be a multiple of 16 for the 8-bit products (got {C})")
        self.att, self.p, self.C = attention, p, C
        self.w_qkv, self.s_qkv = quant_fp8_weight(w_qkv)
        self.w_o, self.s_o = quant_fp8_weight(w_o)
        self.b_qkv, self.b_o = b_qkv, b_o
        self.norm_weight, self.wq, self.wk = norm_weight, wq, wk
        self.tables, self.norm, self.eps, self.pairing = tuple(tables), norm, eps, pairing

    @torch.no_grad()
    def __call__(self, x: torch.Tensor, delta: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """x, delta [B, N, C] -> (h [B, N, C] in x's type, out [B, N, C] bf16).

        One call at a time per object: the attention's selection and workspace are its own."""
        p = self.p
        if tuple(x.shape) != (p.B, p.N, self.C):
            raise ValueError(f"x must be [{p.B}, {p.N}, {self.C}] (got {tuple(x.shape)})")
        if x.device != self.w_qkv.device:
            raise ValueError(f"x is on {x.device}, the weights on {self.w_qkv.device}")
        return B._on_device(x.device, lambda: self._run(x, delta))

    def _run(self, x, delta):
        p = self.p
        if delta is not None and x.dtype is torch.float16 and delta.dtype is torch.bfloat16:
            delta = delta.to(torch.float16)
        h, y, ys = add_rms_norm_fp8(x, delta, self.norm_weight, self.eps)
        qkv = gemm_fp8(y, ys, self.w_qkv, self.s_qkv, self.b_qkv)
        q, k, v = qkv_norm_rope(qkv.view(p.B, p.N, 3, p.heads, p.d), p.grid, self.tables, self.wq, self.wk, self.norm,
                                self.eps, self.pairing)
        o, os = quant_fp8_heads(self.att(q, k, v))
        return h, gemm_fp8(o, os, self.w_o, self.s_o, self.b_o).view(p.B, p.N, self.C)
