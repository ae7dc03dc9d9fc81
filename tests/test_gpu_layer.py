"""GPU parity of the operators around the attention against plain fp64
implementations: residual + RMS norm (forward, e4m3 output, backward), the
8-bit quantisers and block-scaled product, rotary positions (forward,
backward), and the attention block they form.

Tolerances.  A rounding to a type is off by at most finfo.eps / 2 of the value
(at most half of the smallest subnormal below the normal range).  Sums of n
terms in fp32 are off by at most n * 2^-24 of the sum of the magnitudes; the
kernels add at most 32 terms per thread and then over lanes and warps in
trees, so FP32_SUM = 64 * 2^-24 bounds the statistics of a row and what is
multiplied with them (a handful of further roundings, and rsqrtf's two units
in the last place)."""
import os

import numpy as np
import pytest
import torch

from oracle import layer_oracle as L
from oracle import veda_oracle as O
from veda_synth import PRESETS, make_mlp

from parity import ATTN_MAX_ABS, ATTN_REL_L2, f64, mlp_device

pytestmark = pytest.mark.gpu

FP32_SUM = 64 * 2.0 ** -24
BF16, FP16, FP32, FP8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def V():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import tile_sparse_attention_head_b200 as V
    return V


def half_step(t):
    return torch.finfo(t).eps / 2


def low(t):
    """Half of the smallest subnormal of a type."""
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def close(got, ref, t, mag=None, rel=FP32_SUM, what=""):
    """|got - ref| <= one rounding to t + rel of the magnitudes that were added up."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    mag = np.abs(ref) if mag is None else mag
    lim = half_step(t) * (np.abs(ref) + rel * mag) + rel * mag + low(t)
    bad = ~(np.abs(got - ref) <= lim)
    assert got.shape == ref.shape, what
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(np.abs(got - ref) / lim):.3g} of the limit"


def rand(*shape, seed=0, scale=1.0, t=FP32):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(t).cuda()


STREAMS = [(BF16, BF16), (FP16, FP16), (FP32, FP32), (FP32, BF16)]
# one row; one chunk; rows that one warp holds in 1, 2 and 4 chunks a lane; a last block that is not full; a CTA per
# row with 2 and 4 chunks a thread; more rows than CTAs are launched
SHAPES = [(1, 8), (1, 5120), (3, 72), (37, 256), (5, 512), (1001, 1000), (6, 1032), (7, 4096), (3, 8192), (2, 8200),
          (2, 16384), (9001, 64), (5000, 1088)]


# ---------------------------------------------------------------- residual and norm

def norm_inputs(rows, C, tx, td, seed=0):
    x = (rand(rows, C, seed=seed) * torch.exp(0.7 * rand(C, seed=seed + 1))).to(tx)
    return x, rand(rows, C, seed=seed + 2, scale=0.3, t=td), 1 + 0.2 * rand(C, seed=seed + 3)


def norm_backward_mags(H, W, DY, DH=0.0):
    """Sums of the magnitudes that dx and dw add up."""
    r = 1 / np.sqrt((H * H).mean(1, keepdims=True) + 1e-6)
    g = np.abs(DY * W)
    return np.abs(DH) + r * (g + np.abs(H) * (g * np.abs(H)).mean(1, keepdims=True) * r * r), np.abs(DY * H * r).sum(0)


@pytest.mark.parametrize("tx,td", STREAMS)
@pytest.mark.parametrize("rows,C", SHAPES)
def test_add_rms_norm(V, rows, C, tx, td):
    x, delta, w = norm_inputs(rows, C, tx, td)
    h, y = V.add_rms_norm(x, delta, w, 1e-6)
    assert torch.equal(h, (x.float() + delta.float()).to(tx))
    assert y.dtype == td and h.dtype == tx
    close(y, L.rms_norm(f64(h), f64(w), 1e-6)[0], td, what="y")
    h2, y2 = V.add_rms_norm(x, None, w, 1e-6)
    assert h2 is x and y2.dtype == tx
    close(y2, L.rms_norm(f64(x), f64(w), 1e-6)[0], tx, what="y without a delta")


@pytest.mark.parametrize("tx,td", STREAMS)
@pytest.mark.parametrize("rows,C", SHAPES)
def test_add_rms_norm_backward(V, rows, C, tx, td):
    x, delta, w = norm_inputs(rows, C, tx, td)
    dh, dy = rand(rows, C, seed=7, t=tx), rand(rows, C, seed=8, t=td)
    leaves = [t.requires_grad_() for t in (x, delta, w)]
    h, y = V.add_rms_norm(*leaves, 1e-6)
    dx, dd, dw = torch.autograd.grad((h, y), leaves, (dh, dy))
    H, W, DY, DH = f64(h), f64(w), f64(dy), f64(dh)
    d, rw = L.rms_norm_backward(H, W, 1e-6, DY, DH)
    mag, magw = norm_backward_mags(H, W, DY, DH)
    close(dx, d, tx, mag, what="dx")
    close(dd, d, td, mag, what="ddelta")
    close(dw, rw, FP32, magw, rel=(rows + 64) * 2.0 ** -24, what="dweight")
    again = torch.autograd.grad(V.add_rms_norm(*leaves, 1e-6), leaves, (dh, dy))
    for a, b in zip(again, (dx, dd, dw)):
        assert torch.equal(a, b)


def test_add_rms_norm_gradient_against_differences(V):
    """A directional difference of the kernel's own fp32 forward.  Its rounding error is at most FP32_SUM of the
    magnitudes in the loss, over the step; what a difference of this step is off by at all is taken from fp64."""
    ts = norm_inputs(50, 80, FP32, FP32)
    dh, dy = rand(50, 80, seed=7), rand(50, 80, seed=8)
    leaves = [t.clone().requires_grad_() for t in ts]
    h, y = V.add_rms_norm(*leaves)
    grads = torch.autograd.grad((h, y), leaves, (dh, dy))
    size = ((h.double() * dh).abs().sum() + (y.double() * dy).abs().sum()).item()
    step = 0.05
    for i, g in enumerate(grads):
        v = rand(*ts[i].shape, seed=20 + i)

        def loss(s):
            hh, yy = V.add_rms_norm(*(t + (s * v if i == j else 0) for j, t in enumerate(ts)))
            return ((hh.double() * dh).sum() + (yy.double() * dy).sum()).item()

        def exact(s):
            x, d, w = (f64(t) + (s * f64(v) if i == j else 0) for j, t in enumerate(ts))
            return float(((x + d) * f64(dh)).sum() + (L.rms_norm(x + d, w, 1e-6)[0] * f64(dy)).sum())

        ana = (g.double() * v).sum().item()
        num, num64 = ((f(step) - f(-step)) / (2 * step) for f in (loss, exact))
        fine = (exact(1e-5) - exact(-1e-5)) / 2e-5
        assert abs(num - ana) <= 2 * size * FP32_SUM / step + 1.1 * abs(num64 - fine) + 1e-3, (i, num, ana, num64)


@pytest.mark.parametrize("use", ["y", "h", "y without x", "no weight", "no delta"])
def test_add_rms_norm_partial_gradients(V, use):
    x, delta, w = norm_inputs(33, 200, FP32, BF16)
    dh, dy = rand(33, 200, seed=7), rand(33, 200, seed=8, t=BF16)
    x.requires_grad_(use != "y without x")
    delta.requires_grad_(use != "no weight")
    w.requires_grad_(use != "no weight")
    if use == "no delta":
        y = V.add_rms_norm(x, None, w)[1]
        dy = dy.float()
        gx, gw = torch.autograd.grad(y, (x, w), dy)
        h = x
    else:
        h, y = V.add_rms_norm(x, delta, w)
    d, dw = L.rms_norm_backward(f64(h), f64(w), 1e-6, f64(dy))
    mag, magw = norm_backward_mags(f64(h), f64(w), f64(dy))
    if use == "no delta":
        close(gx, d, FP32, mag, what="dx")
        close(gw, dw, FP32, magw, rel=97 * 2.0 ** -24, what="dw")
    elif use == "h":
        gx, gd = torch.autograd.grad(h, (x, delta), dh)
        assert torch.equal(gx, dh) and torch.equal(gd, dh.to(BF16))
    elif use == "no weight":
        close(torch.autograd.grad(y, x, dy)[0], d, FP32, mag, what="dx")
    else:
        gs = torch.autograd.grad(y, [t for t in (x, delta, w) if t.requires_grad], dy)
        close(gs[-2], d, BF16, mag, what="ddelta")
        close(gs[-1], dw, FP32, magw, rel=97 * 2.0 ** -24, what="dw")
        if use == "y":
            close(gs[0], d, FP32, mag, what="dx")


def test_norm_strides_and_shapes(V):
    """A column slice of a wider tensor, a batch of rows, an unaligned and an expanded gradient."""
    wide = rand(40, 3 * 128, t=BF16)
    x, delta = wide[:, 128:256], wide[:, 256:]
    w = 1 + 0.2 * rand(128, seed=3)
    h, y = V.add_rms_norm(x, delta, w)
    hd, yd = V.add_rms_norm(x.contiguous(), delta.contiguous(), w)
    assert torch.equal(h, hd) and torch.equal(y, yd)
    hb, yb = V.add_rms_norm(x.view(2, 4, 5, 128), delta.view(2, 4, 5, 128), w)
    assert hb.shape == (2, 4, 5, 128) and torch.equal(yb.view(40, 128), y)
    xl = x.contiguous().requires_grad_()
    g = rand(40 * 128 + 4, t=BF16)[4:].view(40, 128)
    assert g.data_ptr() % 16 == 8
    a, = torch.autograd.grad(V.add_rms_norm(xl, delta, w)[1], xl, g)
    b, = torch.autograd.grad(V.add_rms_norm(xl, delta, w)[1], xl, g.clone())
    assert torch.equal(a, b)
    one = torch.ones((), dtype=BF16, device="cuda").expand(40, 128)
    a, = torch.autograd.grad(V.add_rms_norm(xl, delta, w)[1], xl, one)
    b, = torch.autograd.grad(V.add_rms_norm(xl, delta, w)[1], xl, one.contiguous())
    assert torch.equal(a, b)


def test_norm_special_values(V):
    """Rows of zeros, with an infinity and with a NaN leave the other rows alone."""
    x = rand(6, 1200)
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, 700] = float("nan")
    delta, w = torch.zeros_like(x), torch.ones(1200, device="cuda")
    h, y = V.add_rms_norm(x, delta, w)
    assert torch.equal(y[1], torch.zeros_like(y[1]))
    assert torch.isnan(y[2, 5]) and (y[2, 6:] == 0).all()       # x / inf
    assert torch.isnan(y[3]).all()
    assert torch.equal(y[[0, 4, 5]], V.add_rms_norm(x[[0, 4, 5]], delta[:3], w)[1])
    h, q, s = V.add_rms_norm_fp8(x, delta, w)
    assert (q[1].float() == 0).all() and (s[:, 1] == 2.0 ** -100 / 448).all()
    val = q.float() * s.t().repeat_interleave(128, 1)[:, :1200]
    assert torch.isnan(val[2, :128]).all() and (val[2, 128:] == 0).all()
    assert torch.isnan(val[3]).all()
    ok = V.add_rms_norm_fp8(x[[0, 4, 5]], delta[:3], w)
    assert torch.equal(q[[0, 4, 5]].view(torch.uint8), ok[1].view(torch.uint8)) and torch.equal(s[:, [0, 4, 5]], ok[2])


def test_norm_no_rows(V):
    x = torch.empty(0, 64, device="cuda", dtype=BF16, requires_grad=True)
    w = torch.ones(64, device="cuda", requires_grad=True)
    h, y = V.add_rms_norm(x, x.detach(), w)
    gx, gw = torch.autograd.grad(y, (x, w), torch.empty_like(y))
    assert gx.shape == (0, 64) and (gw == 0).all()
    with torch.no_grad():
        h, q, s = V.add_rms_norm_fp8(x, x, w)
    assert q.shape == (0, 64) and s.shape == (1, 0)


# ---------------------------------------------------------------- 8 bits

def check_blocks(q, scale, y, what, rel=FP32_SUM):
    """q and scale against exact rows y: scales to fp32 accuracy, values to one rounding of y / scale."""
    R, C = y.shape
    ref = L.block_scales(y)
    close(scale, ref, FP32, rel=rel, what=what + " scales")
    v = y / L.spread(ref, C)
    close(f64(q.float()), v, FP8, np.abs(v), rel=rel, what=what + " values")


@pytest.mark.parametrize("tx,td", STREAMS)
@pytest.mark.parametrize("rows,C", SHAPES)
def test_add_rms_norm_fp8(V, rows, C, tx, td):
    x, delta, w = norm_inputs(rows, C, tx, td)
    h, q, s = V.add_rms_norm_fp8(x, delta, w, 1e-6)
    assert torch.equal(h, (x.float() + delta.float()).to(tx))
    check_blocks(q, s, L.rms_norm(f64(h), f64(w), 1e-6)[0], "fp8 norm")


# A scale is one rounding of a / 448 and of 1 / 448 away from exact, its reciprocal two units more, the product one
# rounding: 2^-21 in all.
QUANT_REL = 2.0 ** -21


@pytest.mark.parametrize("t", [BF16, FP16, FP32])
@pytest.mark.parametrize("rows,C", [(1, 8), (1, 5120), (63, 120), (65, 128), (200, 1000), (129, 136)])
def test_quant_fp8(V, rows, C, t):
    x = (rand(rows, C) * torch.exp(2 * rand(rows, 1, seed=1))).to(t)
    x[0, :] = 0
    q, s = V.quant_fp8(x)
    check_blocks(q, s, f64(x), "quant", rel=QUANT_REL)
    wide = torch.zeros(rows, C + 24, dtype=t, device="cuda")
    wide[:, 8:8 + C] = x
    q2, s2 = V.quant_fp8(wide[:, 8:8 + C])
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)


@pytest.mark.parametrize("B,heads,N,d", [(1, 1, 1, 64), (2, 3, 77, 64), (1, 5, 130, 128), (2, 2, 65, 8), (1, 40, 3, 128)])
def test_quant_fp8_heads(V, B, heads, N, d):
    o = rand(B, heads, N, d, t=BF16)
    q, s = V.quant_fp8_heads(o)
    check_blocks(q, s, f64(o.transpose(1, 2).reshape(B * N, heads * d)), "quant heads", rel=QUANT_REL)
    t = o.transpose(1, 2).contiguous().transpose(1, 2)      # token order behind the same shape
    q2, s2 = V.quant_fp8_heads(t)
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)


def test_quant_special_values(V):
    x = rand(8, 256)
    x[1, 3], x[2, 200], x[3] = float("inf"), float("nan"), 1e-38
    x[4], x[5, :128] = 3e38, 2.0 ** -120
    q, s = V.quant_fp8(x)
    val = q.float() * s.t().repeat_interleave(128, 1)
    assert torch.isnan(val[1, :128]).all() and torch.isfinite(val[1, 128:]).all()
    assert torch.isnan(val[2, 128:]).all() and torch.isfinite(val[2, :128]).all()
    assert torch.isfinite(val[3:]).all()
    assert torch.allclose(val[4], x[4], rtol=2.0 ** -4)


@pytest.mark.parametrize("t", [BF16, FP16, FP32])
@pytest.mark.parametrize("N,K", [(1, 8), (128, 128), (130, 136), (257, 1000), (8, 4096)])
def test_quant_fp8_weight(V, N, K, t):
    w = (rand(N, K) * torch.exp(rand(1, K, seed=2))).to(t).requires_grad_()
    q, s = V.quant_fp8_weight(w)
    w = w.detach().float()
    for i in range(0, N, 128):
        for j in range(0, K, 128):
            b = w[i:i + 128, j:j + 128]
            ref = max(float(b.abs().max()), L.TINY) / 448
            assert abs(float(s[i // 128, j // 128]) - ref) <= QUANT_REL * ref
            v = f64(b) / ref
            close(f64(q[i:i + 128, j:j + 128].float()), v, FP8, np.abs(v), rel=QUANT_REL, what="weight")


def gemm_inputs(M, K, N, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = torch.randn(M, K, generator=g, device="cuda").to(FP8)
    b = torch.randn(N, K, generator=g, device="cuda").to(FP8)
    kb, nb = -(-K // 128), -(-N // 128)
    sa = torch.exp(torch.randn(kb, M, generator=g, device="cuda"))
    sb = torch.exp(torch.randn(nb, kb, generator=g, device="cuda")) / 30
    return a, sa, b, sb, torch.randn(N, generator=g, device="cuda")


def gemm_check(out, a, sa, b, sb, bias, what=""):
    """Products of e4m3 values are exact.  A block's 128 are added on the tensor cores (at most 128 roundings or
    truncations of 2^-23), the blocks and the bias in fp32 (a scale product, a multiply-add each): with n = 128 +
    4 blocks steps of at most 2^-23 of the sum of the magnitudes."""
    M, K = a.shape
    N = b.shape[0]
    kb = -(-K // 128)
    A = a.double() * sa.double().t().repeat_interleave(128, 1)[:, :K]
    Bw = b.double() * sb.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    ref, mag = A @ Bw.t(), A.abs() @ Bw.abs().t()
    if bias is not None:
        ref, mag = ref + bias.double(), mag + bias.double().abs()
    lim = half_step(out.dtype) * ref.abs() + (128 + 4 * kb) * 2.0 ** -23 * mag * (1 + half_step(out.dtype))
    off = (out.double() - ref).abs()
    assert bool((off <= lim).all()), f"{what}: worst {(off / lim).max().item():.3g} of the limit"


# one token, few rows, rows around every tile border, odd N and K (a K inside a block, an N inside a tile), one to many
# blocks, more tiles than SMs
GEMM = [(1, 16, 8), (1, 128, 64), (1, 5120, 1536), (1, 1552, 2056), (2, 512, 520), (3, 4096, 256), (7, 272, 1000),
        (8, 2048, 2048), (9, 144, 384), (15, 5120, 512), (16, 1536, 4608), (17, 640, 136), (31, 528, 776),
        (33, 1024, 1024), (64, 5120, 1536), (65, 400, 264), (100, 128, 2048), (127, 256, 256), (128, 384, 512),
        (129, 1040, 248), (200, 2064, 1048), (255, 640, 640), (257, 1552, 2056), (777, 1552, 2056), (1560, 1536, 1536),
        (2000, 256, 5128), (5000, 160, 264)]


@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("M,K,N", GEMM)
def test_gemm_fp8(V, M, K, N, out):
    a, sa, b, sb, bias = gemm_inputs(M, K, N)
    for with_bias in (bias, None):
        c = V.gemm_fp8(a, sa, b, sb, with_bias, out)
        V.veda_sync_status()
        assert c.dtype == out and c.shape == (M, N)
        gemm_check(c, a, sa, b, sb, with_bias)
    assert torch.equal(c, V.gemm_fp8(a, sa, b, sb, None, out))


@pytest.mark.parametrize("M", [1, 5, 40, 300])
def test_gemm_fp8_strides_and_borders(V, M):
    """Operands and output inside wider tensors; what stands around the output is left as it was."""
    K, N = 272, 264
    a, sa, b, sb, bias = gemm_inputs(M, K, N)
    wa = torch.full((M, K + 48), 448.0, device="cuda").to(FP8)
    wb = torch.full((N + 130, K + 16), 448.0, device="cuda").to(FP8)
    wa[:, 16:16 + K], wb[:N, 16:16 + K] = a, b
    room = torch.full((M + 2, N + 16), -77.0, device="cuda")
    V.gemm_fp8(wa[:, 16:16 + K], sa, wb[:N, 16:16 + K], sb, bias, out=room[1:1 + M, 8:8 + N])
    V.veda_sync_status()
    gemm_check(room[1:1 + M, 8:8 + N], a, sa, b, sb, bias)
    room[1:1 + M, 8:8 + N] = -77.0
    assert (room == -77.0).all()


def test_gemm_fp8_empty_and_special(V):
    a, sa, b, sb, _ = gemm_inputs(70, 384, 128)
    assert V.gemm_fp8(a[:0], sa[:, :0].contiguous(), b, sb).shape == (0, 128)
    clean = V.gemm_fp8(a, sa, b, sb, out_dtype=FP32)
    sa2, b2 = sa.clone(), b.clone()
    sa2[1, 5] = float("inf")
    bad = V.gemm_fp8(a, sa2, b, sb, out_dtype=FP32)
    keep = [i for i in range(70) if i != 5]
    assert not torch.isfinite(bad[5]).any() and torch.equal(bad[keep], clean[keep])
    b2.view(torch.uint8)[3, 200] = 0x7F          # NaN
    bad = V.gemm_fp8(a, sa, b2, sb, out_dtype=FP32)
    cols = [i for i in range(128) if i != 3]
    assert torch.isnan(bad[:, 3]).all() and torch.equal(bad[:, cols], clean[:, cols])


def test_gemm_fp8_refusals(V):
    a, sa, b, sb, bias = gemm_inputs(8, 256, 64)
    for args in ((a.float(), sa, b, sb), (a, sa.t().contiguous(), b, sb), (a, sa, b[:, :128], sb), (a, sa, b, sb.t().contiguous()),
                 (a, sa.double(), b, sb), (a, sa, b, sb, bias[:32]), (a, sa, b, sb, bias.half()), (a.t(), sa, b, sb)):
        with pytest.raises((ValueError, V.VedaError)):
            V.gemm_fp8(*args)
    with pytest.raises(ValueError):
        V.gemm_fp8(a, sa, b, sb, out=torch.empty(8, 72, device="cuda"))
    with pytest.raises(V.VedaError):
        V.gemm_fp8(a, sa, b, sb, out_dtype=FP16)


# ---------------------------------------------------------------- rotary positions

def rope_inputs(V, B, heads, d, grid, dims, norm, t, seed=0, start=(0.0, 0.0, 0.0)):
    n = grid[0] * grid[1] * grid[2]
    qkv = (rand(B, n, 3, heads, d, seed=seed) * torch.exp(0.3 * rand(3, heads, d, seed=seed + 1))).to(t)
    nw = {"row": heads * d, "head": d, "none": 0}[norm]
    wq, wk = ((1 + 0.2 * rand(nw, seed=seed + 2), 1 + 0.2 * rand(nw, seed=seed + 3)) if nw else (None, None))
    return qkv, wq, wk, V.rope_tables(grid, dims, start=start)


def tables64(tables, dims):
    return [None if t is None else f64(t) for t in tables]


def rope_mag(x, w, dims, norm, halves):
    """Magnitudes added up for each rotated element, grid order."""
    y = np.abs(x)
    if norm != "none":
        y = y / np.sqrt(L._mean(x * x, norm) + 1e-6) * np.abs(w.reshape(-1, x.shape[-1]))
    m = y.copy()
    for a, b, _, _ in L.pairs(dims, halves):
        m[..., a] = m[..., b] = y[..., a] + y[..., b]
    return m.transpose(0, 2, 1, 3)


# one token; a warp per token in 1, 2 and 4 chunks a lane; a CTA per token; more tokens than CTAs; partial and
# missing axes
ROPE = [(1, 1, 64, (1, 1, 1), (16, 24, 24)), (1, 1, 128, (2, 3, 5), (44, 42, 42)), (2, 3, 64, (2, 5, 3), (24, 20, 20)),
        (1, 5, 128, (3, 4, 7), (16, 32, 32)), (1, 8, 128, (2, 2, 3), (128, 0, 0)), (1, 12, 128, (5, 6, 9), (44, 42, 42)),
        (2, 40, 128, (2, 3, 4), (44, 42, 42)), (1, 67, 128, (1, 2, 3), (0, 64, 64)), (1, 9, 64, (2, 2, 2), (0, 0, 0)),
        (1, 2, 64, (9, 20, 31), (8, 16, 16)), (1, 17, 64, (7, 20, 31), (24, 20, 20))]


@pytest.mark.parametrize("norm", ["row", "head", "none"])
@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
@pytest.mark.parametrize("t", [BF16, FP16, FP32])
@pytest.mark.parametrize("B,heads,d,grid,dims", ROPE)
def test_qkv_norm_rope(V, B, heads, d, grid, dims, t, pairing, norm):
    qkv, wq, wk, tables = rope_inputs(V, B, heads, d, grid, dims, norm, t)
    douts = [rand(B, heads, qkv.shape[1], d, seed=30 + i, t=BF16) for i in range(3)]
    leaves = [x.requires_grad_() for x in (qkv, wq, wk) if x is not None]
    q, k, v = V.qkv_norm_rope(qkv, grid, tables, wq, wk, norm=norm, pairing=pairing)
    grads = torch.autograd.grad((q, k, v), leaves, douts)
    with torch.no_grad():
        for a, b in zip((q, k, v), V.qkv_norm_rope(qkv, grid, tables, wq, wk, norm=norm, pairing=pairing)):
            assert torch.equal(a, b)
    again = torch.autograd.grad(V.qkv_norm_rope(qkv, grid, tables, wq, wk, norm=norm, pairing=pairing), leaves, douts)
    for a, b in zip(again, grads):
        assert torch.equal(a, b)
    tabs, halves = tables64(tables, dims), pairing == "halves"
    for i, (out, w) in enumerate(((q, wq), (k, wk))):
        x = f64(qkv[:, :, i])
        W = None if w is None else f64(w)
        close(out, L.norm_rope(x, W, grid, dims, tabs, norm, halves, 1e-6), BF16, rope_mag(x, W, dims, norm, halves), what="qk"[i])
        dx, dw, mag, magw = L.norm_rope_backward(x, W, grid, dims, tabs, norm, halves, 1e-6, f64(douts[i]))
        close(grads[0][:, :, i], dx, t, mag, rel=2 * FP32_SUM, what="d" + "qk"[i])
        if w is not None:
            n = B * qkv.shape[1] * (heads if norm == "head" else 1)
            close(grads[1 + i], dw, FP32, magw, rel=(n + 128) * 2.0 ** -24, what="dw" + "qk"[i])
    assert torch.equal(v, qkv[:, :, 2].transpose(1, 2).to(BF16))
    assert torch.equal(grads[0][:, :, 2], douts[2].transpose(1, 2).to(t))


def test_rope_far_positions_and_moved_grid(V):
    """Angles at position 10^6 keep fp32 accuracy, and a table from a later row on moves the grid."""
    for theta, start, step in ((1e4, 0.0, 1.0), (1e4, 1e6, 1.0), (256.0, -3.0, 0.25)):
        t = V.rope_table(7, 44, theta, start, step)
        # half a step of fp32, and fp64 angles up to 10^6 off by two roundings
        assert np.abs(f64(t) - L.rope_table(7, 44, theta, start, step)).max() <= 2.0 ** -24 + 1e6 * 2.0 ** -50
    qkv, wq, wk, tables = rope_inputs(V, 1, 2, 64, (6, 2, 3), (24, 20, 20), "row", BF16)
    q, k, v = V.qkv_norm_rope(qkv, (6, 2, 3), tables, wq, wk)
    later = (tables[0][4:],) + tables[1:]
    q2, _, _ = V.qkv_norm_rope(qkv[:, 24:], (2, 2, 3), later, wq, wk)
    assert torch.equal(q2, q[:, :, 24:])


def test_rope_strides_and_separate_operands(V):
    grid, dims = (2, 3, 4), (24, 20, 20)
    qkv, wq, wk, tables = rope_inputs(V, 2, 3, 64, grid, dims, "head", FP32)
    ref = V.qkv_norm_rope(qkv, grid, tables, wq, wk, norm="head")
    xs = [x.clone() for x in qkv.unbind(2)]
    xs[1] = torch.stack((xs[1], xs[1]), 3)[:, :, :, 0]               # a head stride of 2 d
    xs[2] = xs[2].permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)    # grid order behind token order
    xs = [x.requires_grad_() for x in xs]
    out = V.qkv_norm_rope(xs, grid, tables, wq, wk, norm="head")
    for a, b in zip(out, ref):
        assert torch.equal(a, b)
    douts = [rand(2, 3, 24, 64, seed=40 + i, t=BF16) for i in range(3)]
    packed = qkv.clone().requires_grad_()
    g, = torch.autograd.grad(V.qkv_norm_rope(packed, grid, tables, wq, wk, norm="head"), packed, douts)
    for i, a in enumerate(torch.autograd.grad(out, xs, douts)):
        assert torch.equal(a, g[:, :, i])
    # only k is used: q's and v's gradients are zero or absent
    k = V.qkv_norm_rope(packed, grid, tables, wq, wk, norm="head")[1]
    gk, = torch.autograd.grad(k, packed, douts[1])
    assert torch.equal(gk[:, :, 1], g[:, :, 1]) and (gk[:, :, 0] == 0).all() and (gk[:, :, 2] == 0).all()


def test_rope_special_values(V):
    """An infinity in a channel that is not turned stays one, and other tokens do not see it."""
    grid, dims = (2, 2, 2), (8, 16, 16)
    qkv, _, _, tables = rope_inputs(V, 1, 2, 64, grid, dims, "none", BF16)
    for pairing in ("interleaved", "halves"):
        ref = V.qkv_norm_rope(qkv, grid, tables, norm="none", pairing=pairing)
        x = qkv.clone()
        x[0, 3, 0, 1, 50] = float("inf")
        q, k, v = V.qkv_norm_rope(x, grid, tables, norm="none", pairing=pairing)
        want = ref[0].clone()
        want[0, 1, 3, 50] = float("inf")
        assert torch.equal(q, want) and torch.equal(k, ref[1]) and torch.equal(v, ref[2])


def test_rope_refusals(V):
    grid, dims = (2, 3, 4), (24, 20, 20)
    qkv, wq, wk, tables = rope_inputs(V, 1, 2, 64, grid, dims, "row", BF16)
    bad = [((qkv, grid, (tables[0][:1],) + tables[1:], wq, wk), {}),             # a table shorter than the axis
           ((qkv, grid, (tables[0].cpu(),) + tables[1:], wq, wk), {}),
           ((qkv, grid, tables, wq[:64], wk), {}),
           ((qkv, grid, tables, wq, wk), dict(norm="head")),
           ((qkv.double(), grid, tables, wq, wk), {}),
           ((qkv[..., :32], grid, tables, wq, wk), {}),
           ((qkv.transpose(3, 4).contiguous().transpose(3, 4), grid, tables, wq, wk), {}),
           ((qkv, grid, V.rope_tables(grid, (24, 24, 24)), wq, wk), {})]
    for args, kw in bad:
        with pytest.raises((ValueError, V.VedaError)):
            V.qkv_norm_rope(*args, **kw)


# ---------------------------------------------------------------- streams, graphs, the whole block

def test_side_stream_and_capture(V):
    """Calls on a side stream, and a captured training step replayed on new data."""
    x, delta, w = norm_inputs(300, 768, FP32, BF16)
    grid, dims = (3, 4, 5), (24, 20, 20)
    qkv, wq, wk, tables = rope_inputs(V, 1, 4, 64, grid, dims, "row", BF16)
    a, sa, b, sb, bias = gemm_inputs(300, 768, 512)
    few = (a[:2], sa[:, :2].contiguous())
    dh, dy = rand(300, 768, seed=7), rand(300, 768, seed=8, t=BF16)
    douts = [rand(1, 4, 60, 64, seed=40 + i, t=BF16) for i in range(3)]
    leaves = [t.requires_grad_() for t in (x, delta, w)]
    rleaves = [t.requires_grad_() for t in (qkv, wq, wk)]

    def step():
        g = torch.autograd.grad(V.add_rms_norm(*leaves), leaves, (dh, dy))
        r = torch.autograd.grad(V.qkv_norm_rope(qkv, grid, tables, wq, wk), rleaves, douts)
        with torch.no_grad():
            h8 = V.add_rms_norm_fp8(*leaves)
            c = [V.gemm_fp8(a, sa, b, sb, bias), V.gemm_fp8(*few, b, sb, bias)]
        return list(g) + list(r) + [h8[0], h8[1].view(torch.uint8), h8[2]] + c

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    for i, (p, q) in enumerate(zip(got, want)):
        assert torch.equal(p, q), i
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = step()
    with torch.no_grad():
        for t in leaves + rleaves:
            t.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    for i, (p, q) in enumerate(zip(cap, step())):
        assert torch.equal(p, q), i
    V.veda_sync_status()


def test_two_streams_at_once(V):
    """The same calls on two streams, many in flight, with different sizes (so that launches with more and less shared
    memory alternate)."""
    cases = []
    for rows, C in ((700, 5120), (90, 128)):
        x, delta, w = norm_inputs(rows, C, BF16, BF16)
        cases.append((x, delta, w) + gemm_inputs(rows, C, 512))

    def calls(c):
        h, q, s = V.add_rms_norm_fp8(c[0], c[1], c[2])
        return [h, q.view(torch.uint8), s, V.gemm_fp8(*c[3:7], bias=c[7])]

    want = [calls(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for _ in range(20):
        for i, (c, st) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(st):
                got[i].append(calls(c))
    torch.cuda.synchronize()
    V.veda_sync_status()
    for i, ref in enumerate(want):
        for g in got[i]:
            for a, b in zip(g, ref):
                assert torch.equal(a, b)


def test_offsets_past_32_bits(V):
    """More than 2^31 elements: the last rows, whose offsets do not fit 32 bits, are what they are on their own."""
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of free device memory")
    rows, C, tail = (1 << 18) + 24, 8192, 24
    x = torch.zeros(rows, C, dtype=BF16, device="cuda")
    last = rand(tail, C, t=BF16)
    x[-tail:] = last
    w = 1 + 0.2 * rand(C, seed=3)
    h, y = V.add_rms_norm(x, x, w)
    h1, y1 = V.add_rms_norm(last, last, w)
    assert torch.equal(h[-tail:], h1) and torch.equal(y[-tail:], y1)
    del h, y
    leaf = x.requires_grad_()
    g, = torch.autograd.grad(V.add_rms_norm(leaf, x.detach(), w)[1], leaf, x.detach())
    one = last.clone().requires_grad_()
    g1, = torch.autograd.grad(V.add_rms_norm(one, last, w)[1], one, last)
    assert torch.equal(g[-tail:], g1)
    del g
    x = x.detach()
    h, q, s = V.add_rms_norm_fp8(x, x, w)
    h1, q1, s1 = V.add_rms_norm_fp8(last, last, w)
    assert torch.equal(q[-tail:].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s[:, -tail:], s1)
    _, _, b, sb, bias = gemm_inputs(8, C, 64)
    gemm_check(V.gemm_fp8(q, s, b, sb, bias, FP32)[-tail:], q1, s1, b, sb, bias, "far rows")
    q, s = V.quant_fp8(x)
    q1, s1 = V.quant_fp8(last)
    assert torch.equal(q[-tail:].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s[:, -tail:], s1)
    del x, h, q, s
    heads, d, grid, dims = 64, 128, (5, 256, 256), (44, 42, 42)
    n = grid[0] * grid[1] * grid[2]
    qkv = torch.zeros(1, n, 3, heads, d, dtype=BF16, device="cuda")
    qkv[:, -1] = rand(1, 3, heads, d, t=BF16)
    wq = 1 + 0.2 * rand(heads * d, seed=5)
    tables = V.rope_tables(grid, dims)
    at = tuple(t[-1:].contiguous() for t in tables)
    far = qkv[:, -1:].clone().requires_grad_()
    qkv.requires_grad_()
    out, ref = V.qkv_norm_rope(qkv, grid, tables, wq, wq), V.qkv_norm_rope(far, (1, 1, 1), at, wq, wq)
    for a, c in zip(out, ref):
        assert torch.equal(a[:, :, -1], c[:, :, 0])
    douts = [torch.zeros_like(o) for o in out]
    for i, g in enumerate(douts):
        g[:, :, -1] = rand(1, heads, d, seed=50 + i, t=BF16)
    a, = torch.autograd.grad(out, qkv, douts)
    c, = torch.autograd.grad(ref, far, [g[:, :, -1:].contiguous() for g in douts])
    assert torch.equal(a[:, -1], c[:, 0])
    V.veda_sync_status()


def block_case(V, stream_type, seed=0):
    w = PRESETS["tiny"]
    p = V.Problem(w.B, w.heads, w.d, w.S, (w.T, w.H, w.W), w.tilings)
    C, inner = 200 * 8, w.heads * w.d
    mlp = mlp_device(make_mlp(w, seed=1))
    att = V.VedaAttention(p, mlp, mlp, w.keep)
    dims = (w.d - 4 * (w.d // 6), 2 * (w.d // 6), 2 * (w.d // 6))
    tables = V.rope_tables(p.grid, dims)
    kw = dict(w_qkv=rand(3 * inner, C, seed=seed, scale=C ** -0.5), w_o=rand(C, inner, seed=seed + 1, scale=inner ** -0.5),
              norm_weight=1 + 0.2 * rand(C, seed=seed + 2), wq=1 + 0.2 * rand(inner, seed=seed + 3),
              wk=1 + 0.2 * rand(inner, seed=seed + 4), b_qkv=0.1 * rand(3 * inner, seed=seed + 5), b_o=0.1 * rand(C, seed=seed + 6))
    x, delta = rand(p.B, p.N, C, seed=seed + 7, t=stream_type), rand(p.B, p.N, C, seed=seed + 8, scale=0.3, t=BF16)
    return w, p, att, tables, dims, kw, x, delta


@pytest.mark.parametrize("stream_type", [BF16, FP32])
def test_attention_block(V, stream_type):
    """The block equals its calls in sequence, and each step of it is right for what it was given: two layers, the
    first one's output the second one's delta."""
    w, p, att, tables, dims, kw, x, delta = block_case(V, stream_type)
    block = V.VedaSelfAttention(att, tables=tables, **kw)
    for layer in range(2):
        h, out = block(x, delta)
        H, y8, ys = V.add_rms_norm_fp8(x, delta, kw["norm_weight"])
        qkv = V.gemm_fp8(y8, ys, block.w_qkv, block.s_qkv, kw["b_qkv"])
        q, k, v = V.qkv_norm_rope(qkv.view(p.B, p.N, 3, p.heads, p.d), p.grid, tables, kw["wq"], kw["wk"])
        o = att(q, k, v)
        o8, os = V.quant_fp8_heads(o)
        proj = V.gemm_fp8(o8, os, block.w_o, block.s_o, kw["b_o"]).view(out.shape)
        V.veda_sync_status()
        assert torch.equal(h, H.view(x.shape)) and torch.equal(out, proj)
        assert torch.equal(h, (x.float() + delta.float()).to(stream_type))
        check_blocks(y8, ys, L.rms_norm(f64(h).reshape(-1, h.shape[-1]), f64(kw["norm_weight"]), 1e-6)[0], "block norm")
        gemm_check(qkv, y8, ys, block.w_qkv, block.s_qkv, kw["b_qkv"], "block QKV")
        tabs = tables64(tables, dims)
        for i, (t, wt) in enumerate(((q, kw["wq"]), (k, kw["wk"]))):
            xi = f64(qkv).reshape(p.B, p.N, 3, p.heads, p.d)[:, :, i]
            close(t, L.norm_rope(xi, f64(wt), p.grid, dims, tabs, "row", False, 1e-6), BF16,
                  rope_mag(xi, f64(wt), dims, "row", False), what="block rope")
        perm = [O.tile_permute(f64(t), p.grid, w.tilings, w.S) for t in (q, k, v)]
        ref = O.sparse_attention(*perm, att.idx.cpu().numpy(), p.grid, w.tilings, w.S)
        ref = O.tile_unpermute(ref[0] if isinstance(ref, tuple) else ref, p.grid, w.tilings, w.S)
        err = np.abs(f64(o) - ref)
        assert err.max() <= ATTN_MAX_ABS and np.linalg.norm(err) <= ATTN_REL_L2 * np.linalg.norm(ref)
        gemm_check(out.view(-1, out.shape[-1]), o8, os, block.w_o, block.s_o, kw["b_o"], "block output")
        x, delta = h, out


def test_attention_block_captured(V):
    w, p, att, tables, dims, kw, x, delta = block_case(V, BF16)
    block = V.VedaSelfAttention(att, tables=tables, **kw)
    block(x, delta)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, out = block(x, delta)
    delta.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    h2, out2 = block(x, delta)
    assert torch.equal(h, h2) and torch.equal(out, out2)


def test_attention_block_refusals(V):
    w, p, att, tables, dims, kw, x, delta = block_case(V, BF16)
    with pytest.raises(ValueError, match="w_qkv must be"):
        V.VedaSelfAttention(att, tables=tables, **{**kw, "w_qkv": kw["w_qkv"][:-8]})
    block = V.VedaSelfAttention(att, tables=tables, **kw)
    with pytest.raises(ValueError, match="x must be"):
        block(x[:, 1:], delta[:, 1:])
    with pytest.raises(ValueError, match="x is on"):
        block(x.cpu(), delta.cpu())


def test_training_chain(V):
    """norm -> product -> rope -> sparse attention -> loss, with gradients through the library's backward calls,
    against the same chain of fp64 formulas given each step's stored tensors."""
    w = PRESETS["tiny"]
    p = V.Problem(w.B, w.heads, w.d, w.S, (w.T, w.H, w.W), w.tilings)
    mlp = mlp_device(make_mlp(w, seed=1))
    att = V.VedaAttention(p, mlp, mlp, w.keep)
    dims = (w.d - 4 * (w.d // 6), 2 * (w.d // 6), 2 * (w.d // 6))
    tables = V.rope_tables(p.grid, dims)
    C, inner = 256, w.heads * w.d
    x = rand(p.B, p.N, C, seed=1).requires_grad_()
    delta = rand(p.B, p.N, C, seed=2, scale=0.3, t=BF16).requires_grad_()
    nw = (1 + 0.2 * rand(C, seed=3)).requires_grad_()
    wq, wk = ((1 + 0.2 * rand(inner, seed=s)).requires_grad_() for s in (4, 5))
    W = rand(3 * inner, C, seed=6, scale=C ** -0.5, t=BF16)
    do = rand(p.B, p.heads, p.N, p.d, seed=7, t=BF16)
    h, y = V.add_rms_norm(x, delta, nw)
    qkv = y @ W.t()
    q, k, v = V.qkv_norm_rope(qkv.view(p.B, p.N, 3, p.heads, p.d), p.grid, tables, wq, wk)
    for t in (y, qkv, q, k, v):
        t.retain_grad()
    o = att.differentiable(q, k, v)
    o.backward(do)
    V.veda_sync_status()
    tabs = tables64(tables, dims)
    for i, (t, wt) in enumerate(((q, wq), (k, wk))):
        xi = f64(qkv).reshape(p.B, p.N, 3, p.heads, p.d)[:, :, i]
        dx, dw, mag, magw = L.norm_rope_backward(xi, f64(wt), p.grid, dims, tabs, "row", False, 1e-6, f64(t.grad))
        close(f64(qkv.grad).reshape(p.B, p.N, 3, p.heads, p.d)[:, :, i], dx, BF16, mag, rel=2 * FP32_SUM, what="d qkv")
        close(wt.grad, dw, FP32, magw, rel=(p.B * p.N + 128) * 2.0 ** -24, what="d qk weight")
    H, DY = f64(h).reshape(-1, C), f64(y.grad).reshape(-1, C)
    d, dnw = L.rms_norm_backward(H, f64(nw), 1e-6, DY)
    mag, magw = norm_backward_mags(H, f64(nw), DY)
    close(f64(x.grad).reshape(-1, C), d, FP32, mag, what="dx")
    close(f64(delta.grad).reshape(-1, C), d, BF16, mag, what="ddelta")
    close(nw.grad, dnw, FP32, magw, rel=(len(H) + 64) * 2.0 ** -24, what="d norm weight")


def test_loaded_library_reports_no_failed_check(V):
    """Last in this file: no kernel of the tests above recorded an error."""
    V.veda_sync_status()
    assert V.veda_bounds_checked() == (os.environ.get("VEDA_DEBUG_BOUNDS") == "1")
