"""CPU checks of the operators around the attention: refusals of the C entry
points and of the torch functions (no call here launches a kernel), and the
oracle's gradients against differences."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import layer_oracle as L

PTR = 1 << 20       # stands for a 16-byte aligned device address; no refused call reads it


@pytest.fixture(scope="module")
def V():
    import tile_sparse_attention_head_b200 as V
    return V


BF16, FP16, FP32 = 0, 1, 2
INVALID, UNSUPPORTED = 1, 2


def norm_args(scale=True, **kw):
    a = dict(rows=4, C=64, xt=BF16, x=PTR, ldx=64, dt=BF16, delta=PTR, ldd=64, w=PTR, eps=1e-6, h=PTR, y=PTR, s=PTR)
    a.update(kw)
    return [v for k, v in a.items() if scale or k != "s"] + [None]


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(C=0), dict(C=60), dict(C=16392, ldx=16392, ldd=16392), dict(xt=7), dict(dt=FP16),
    dict(xt=FP32, dt=FP16), dict(xt=BF16, dt=FP32), dict(ldx=56), dict(ldx=68), dict(ldd=56), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(w=None), dict(y=None), dict(x=PTR + 8),
    dict(delta=PTR + 2), dict(h=PTR + 4), dict(y=PTR + 4), dict(w=PTR + 4), dict(ldx=72, h=PTR)])
def test_norm_refusals(V, bad):
    for name in ("veda_add_rms_norm", "veda_add_rms_norm_fp8"):
        assert getattr(V.LIB, name)(*norm_args(name.endswith("fp8"), **bad)) != 0, bad
        assert V.LIB.veda_last_error().decode()


def test_norm_fp8_needs_a_scale(V):
    assert V.LIB.veda_add_rms_norm_fp8(*norm_args(s=None)) != 0


def test_no_rows_is_no_work(V):
    assert V.LIB.veda_add_rms_norm(*norm_args(False, rows=0)) == 0
    assert V.LIB.veda_add_rms_norm_fp8(*norm_args(rows=0)) == 0
    assert V.LIB.veda_add_rms_norm_backward(0, 64, BF16, PTR, BF16, PTR, None, PTR, 1e-6, PTR, None, None, None, 0, None) == 0
    assert V.LIB.veda_quant_fp8(1, 0, 2, 64, BF16, PTR, 0, 64, 64, PTR, PTR, None) == 0
    assert V.LIB.veda_gemm_fp8(0, 64, 64, PTR, 64, PTR, PTR, 64, PTR, None, BF16, PTR, 64, None) == 0
    assert V.LIB.veda_rope_table(0, 32, 1e4, 0.0, 1.0, PTR, None) == 0


@pytest.mark.parametrize("bad", [
    dict(h=None), dict(dy=None), dict(w=None), dict(eps=-1.0), dict(eps=float("nan")), dict(dx=None, dd=None, dw=None), dict(ws=None),
    dict(wsb=0), dict(h=PTR + 8), dict(dw=PTR + 4), dict(ws=PTR + 8), dict(C=12), dict(xt=FP16)])
def test_norm_backward_refusals(V, bad):
    a = dict(rows=4, C=64, xt=BF16, h=PTR, dt=BF16, dy=PTR, dh=PTR, w=PTR, eps=1e-6, dx=PTR, dd=PTR, dw=PTR, ws=PTR,
             wsb=16)
    a.update(bad)
    assert V.LIB.veda_add_rms_norm_backward(*a.values(), None) != 0


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(N=-1), dict(heads=0), dict(d=0), dict(d=12), dict(t=3), dict(sb=4), dict(sn=-8), dict(sh=12),
    dict(x=None), dict(q=None), dict(s=None), dict(x=PTR + 8), dict(heads=1 << 18), dict(B=1 << 20, N=1 << 20)])
def test_quant_refusals(V, bad):
    a = dict(B=1, N=8, heads=2, d=64, t=BF16, x=PTR, sb=0, sn=64, sh=512, q=PTR, s=PTR)
    a.update(bad)
    assert V.LIB.veda_quant_fp8(*a.values(), None) != 0


@pytest.mark.parametrize("bad", [dict(N=0), dict(K=0), dict(K=12), dict(t=5), dict(w=None), dict(q=PTR + 8), dict(s=None)])
def test_quant_weight_refusals(V, bad):
    a = dict(N=8, K=64, t=BF16, w=PTR, q=PTR, s=PTR)
    a.update(bad)
    assert V.LIB.veda_quant_fp8_weight(*a.values(), None) != 0


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(N=0), dict(N=12), dict(K=0), dict(K=24), dict(lda=48), dict(lda=72), dict(ldb=48), dict(ldo=56),
    dict(ldo=68), dict(t=FP16), dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(out=None),
    dict(a=PTR + 8), dict(bias=PTR + 4), dict(out=PTR + 8), dict(M=(1 << 30) + 1), dict(M=1 << 30, N=1 << 30, ldo=1 << 30)])
def test_gemm_refusals(V, bad):
    a = dict(M=8, N=64, K=64, a=PTR, lda=64, sa=PTR, b=PTR, ldb=64, sb=PTR, bias=PTR, t=BF16, out=PTR, ldo=64)
    a.update(bad)
    assert V.LIB.veda_gemm_fp8(*a.values(), None) != 0


@pytest.mark.parametrize("bad", [dict(n=-1), dict(dim=0), dict(dim=3), dict(dim=130), dict(theta=0.0),
                                 dict(theta=float("inf")), dict(start=float("nan")), dict(step=float("inf")),
                                 dict(t=None), dict(t=PTR + 4)])
def test_table_refusals(V, bad):
    a = dict(n=4, dim=32, theta=1e4, start=0.0, step=1.0, t=PTR)
    a.update(bad)
    assert V.LIB.veda_rope_table(*a.values(), None) != 0


def rope(V, **kw):
    from tile_sparse_attention_head_b200.binding import veda_rope
    from tile_sparse_attention_head_b200.binding import veda_grid
    a = dict(B=1, heads=2, d=64, grid=veda_grid(2, 3, 4), dt=16, dh=24, dw=24, tt=PTR, th=PTR, tw=PTR, pairing=0, norm=1,
             eps=1e-6)
    a.update(kw)
    return veda_rope(*a.values())


@pytest.mark.parametrize("bad", [
    dict(B=0), dict(heads=0), dict(heads=100000), dict(d=96), dict(dt=17), dict(dt=-2), dict(dt=32), dict(tt=None),
    dict(th=PTR + 4), dict(pairing=2), dict(norm=3), dict(eps=-1.0)])
def test_rope_refusals(V, bad):
    from tile_sparse_attention_head_b200.binding import veda_tokens
    t = veda_tokens(PTR, 0, 128, 64)
    r = rope(V, **bad)
    assert V.LIB.veda_qkv_norm_rope(ctypes.byref(r), BF16, ctypes.byref(t), None, None, PTR, None, PTR, None, None,
                                    None) != 0
    n = ctypes.c_size_t()
    assert V.LIB.veda_qkv_norm_rope_backward_workspace(ctypes.byref(r), ctypes.byref(n)) != 0


def test_rope_operand_refusals(V):
    from tile_sparse_attention_head_b200.binding import veda_grid, veda_tokens
    r = rope(V)
    ok = veda_tokens(PTR, 0, 128, 64)
    R = ctypes.byref

    def fwd(q=ok, w=PTR, out=PTR, t=BF16, r=r):
        return V.LIB.veda_qkv_norm_rope(R(r), t, None if q is None else R(q), None, None, w, None, out, None, None, None)

    assert fwd(q=None, out=None) != 0                          # nothing to do
    assert fwd(out=None) != 0 and fwd(q=None) != 0             # an operand without its output, and the reverse
    assert fwd(w=None) != 0 and fwd(w=PTR + 4) != 0
    assert fwd(t=9) != 0
    assert fwd(out=PTR + 8) != 0
    for bad in (veda_tokens(None, 0, 128, 64), veda_tokens(PTR + 8, 0, 128, 64), veda_tokens(PTR, 0, 132, 64),
                veda_tokens(PTR, 0, -128, 64), veda_tokens(PTR, 4, 128, 64), veda_tokens(PTR, 0, 128, 12)):
        assert fwd(q=bad) != 0
    for g in (veda_grid(0, 3, 4), veda_grid(2, 3, -1), veda_grid(1 << 20, 1 << 20, 1)):
        assert fwd(r=rope(V, grid=g)) != 0
    assert fwd(r=rope(V, B=3, grid=veda_grid(1 << 10, 1 << 10, 1 << 9))) != 0
    with pytest.raises(ValueError, match="even"):
        V.rope_table(4, 43)

    def bwd(q=ok, d_q=PTR, dq=ok, w=PTR, dw=None, ws=None, wsb=0, r=r):
        return V.LIB.veda_qkv_norm_rope_backward(R(r), BF16, None if q is None else R(q), None, w, None, d_q, None, None,
                                                 None if dq is None else R(dq), None, None, dw, None, ws, wsb, None)

    assert bwd(d_q=None, dq=None) != 0
    assert bwd(dq=None) != 0 and bwd(d_q=None) != 0
    assert bwd(q=None) != 0 and bwd(w=None) != 0               # the norm's backward reads both
    assert bwd(d_q=PTR + 8) != 0
    assert bwd(dw=PTR) != 0                                    # no workspace
    assert bwd(dw=PTR, ws=PTR, wsb=16) != 0 and bwd(dw=PTR + 4, ws=PTR, wsb=1 << 30) != 0
    assert bwd(dw=PTR, ws=PTR, wsb=1 << 30, r=rope(V, norm=0)) != 0     # no weight to have a gradient
    assert bwd(dq=veda_tokens(PTR, 0, 0, 64)) != 0             # rows that would be written twice
    assert bwd(dq=veda_tokens(PTR, 0, 128, 0)) != 0


def test_host_tensors_and_shapes_are_refused(V):
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        V.add_rms_norm(x, x, w)
    with pytest.raises(ValueError, match="CUDA tensor"):
        V.add_rms_norm_fp8(x, x, w)
    with pytest.raises(ValueError, match="shape"):
        V.add_rms_norm(x, x[:2], w)
    with pytest.raises(ValueError, match="CUDA tensor"):
        V.quant_fp8(x)
    with pytest.raises(ValueError, match="heads"):
        V.quant_fp8_heads(x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        V.quant_fp8_weight(x)
    a, s = torch.zeros(4, 64, dtype=torch.float8_e4m3fn), torch.ones(1, 4)
    with pytest.raises(ValueError, match="CUDA tensor"):
        V.gemm_fp8(a, s, a, s)
    qkv = torch.zeros(1, 24, 3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="needs wq and wk"):
        V.qkv_norm_rope(qkv, (2, 3, 4), (None, None, None))
    with pytest.raises(ValueError, match="no weights"):
        V.qkv_norm_rope(qkv, (2, 3, 4), (None, None, None), w, w, norm="none")
    with pytest.raises(ValueError, match="do not fill"):
        V.qkv_norm_rope(qkv, (2, 3, 5), (None, None, None), norm="none")
    with pytest.raises(ValueError, match="norm must be"):
        V.qkv_norm_rope(qkv, (2, 3, 4), (None, None, None), w, w, norm="both")
    with pytest.raises(ValueError, match="pairing must be"):
        V.qkv_norm_rope(qkv, (2, 3, 4), (None, None, None), norm="none", pairing="odd")
    with pytest.raises(ValueError, match="CUDA tensor"):
        V.qkv_norm_rope(qkv, (2, 3, 4), (None, None, None), norm="none")
    with pytest.raises(ValueError, match="packed"):
        V.qkv_norm_rope((qkv, qkv), (2, 3, 4), (None, None, None), norm="none")


def test_eight_bit_forms_refuse_gradients(V):
    x = torch.zeros(4, 64, requires_grad=True)
    w = torch.ones(64)
    a, s = torch.zeros(4, 64, dtype=torch.float8_e4m3fn), torch.ones(1, 4)
    for call in (lambda: V.add_rms_norm_fp8(x, None, w), lambda: V.quant_fp8(x),
                 lambda: V.quant_fp8_heads(x.view(1, 1, 4, 64)), lambda: V.gemm_fp8(a, s, a, s, bias=x[0])):
        with pytest.raises(ValueError, match="no gradient"):
            call()


# ---------------------------------------------------------------- the oracle's gradients against differences

def differences(f, x, step=1e-5):
    g = np.zeros_like(x)
    flat, out = x.reshape(-1), g.reshape(-1)
    for i in range(flat.size):
        keep = flat[i]
        flat[i] = keep + step
        up = f()
        flat[i] = keep - step
        down = f()
        flat[i] = keep
        out[i] = (up - down) / (2 * step)
    return g


def test_oracle_norm_gradient_against_differences():
    rng = np.random.default_rng(0)
    h, w = rng.standard_normal((3, 10)), 1 + 0.2 * rng.standard_normal(10)
    dy, dh = rng.standard_normal((3, 10)), rng.standard_normal((3, 10))

    def loss():
        return float((L.rms_norm(h, w, 1e-3)[0] * dy).sum() + (h * dh).sum())

    d, dw = L.rms_norm_backward(h, w, 1e-3, dy, dh)
    # central differences: error step^2 times third derivatives (order 10) + 2^-52 * 50 / step
    assert np.abs(differences(loss, h) - d).max() < 1e-7
    assert np.abs(differences(loss, w) - dw).max() < 1e-7


@pytest.mark.parametrize("norm", ["row", "head", "none"])
@pytest.mark.parametrize("halves", [False, True])
def test_oracle_rope_gradient_against_differences(norm, halves):
    rng = np.random.default_rng(1)
    grid, dims, heads, d = (2, 2, 2), (4, 2, 4), 2, 12
    x = rng.standard_normal((1, 8, heads, d))
    w = None if norm == "none" else 1 + 0.2 * rng.standard_normal(heads * d if norm == "row" else d)
    tables = [L.rope_table(n, dim, 100.0, 0.5, 1.0) for n, dim in zip(grid, dims)]
    dout = rng.standard_normal((1, heads, 8, d))

    def loss():
        return float((L.norm_rope(x, w, grid, dims, tables, norm, halves, 1e-3) * dout).sum())

    dx, dw, mag, magw = L.norm_rope_backward(x, w, grid, dims, tables, norm, halves, 1e-3, dout)
    assert np.abs(differences(loss, x) - dx).max() < 1e-7
    assert np.all(np.abs(dx) <= mag * (1 + 1e-12))
    if w is not None:
        assert np.abs(differences(loss, w) - dw).max() < 1e-7
        assert np.all(np.abs(dw) <= magw * (1 + 1e-12))


# ---------------------------------------------------------------- sizes past 32 bits

def test_sizes_past_32_bits_are_refused(V, monkeypatch):
    """ctypes passes the low 32 bits of a size that does not fit: each such size is refused before any call.  The
    tensors are broadcast, so nothing of their size is allocated."""
    B = V.binding
    made = []
    monkeypatch.setattr(B, "_device", lambda t, name: t.get_device())
    monkeypatch.setattr(B, "_call", lambda *a: made.append(a[0]))
    monkeypatch.setattr(B, "_at", lambda *a: PTR)
    monkeypatch.setattr(B, "_rows", lambda *a: (PTR, 64))
    big = (1 << 32) + 64
    f8, one = torch.zeros(1, 1, dtype=torch.float8_e4m3fn), torch.zeros(1, 1, dtype=torch.bfloat16)
    s = torch.ones(1, 1)
    x = one.expand(1, big)
    calls = [lambda: V.veda_gemm_fp8(f8.expand(big, 64), s, f8.expand(64, 64), s, None, one.expand(big, 64)),
             lambda: V.veda_gemm_fp8(f8.expand(64, 64), s, f8.expand(big, 64), s, None, one.expand(64, big)),
             lambda: V.gemm_fp8(f8.expand(big, 64), s, f8.expand(64, 64), s),
             lambda: V.gemm_fp8(f8.expand(64, big), s, f8.expand(64, big), s),
             lambda: V.veda_add_rms_norm(x, None, s, 1e-6, None, x),
             lambda: V.veda_add_rms_norm_fp8(x, None, s, 1e-6, None, f8, s),
             lambda: V.binding._layer_norm_forward(x, None, s, 1e-6, None, x, None),
             lambda: V.veda_quant_fp8_weight(one.expand(big, 64), f8, s),
             lambda: V.veda_quant_fp8_weight(x, f8, s),
             lambda: V.veda_quant_fp8(one.view(1, 1, 1, 1).expand(big, 1, 1, 1), f8, s),
             lambda: V.veda_quant_fp8(one.view(1, 1, 1, 1).expand(1, big, 1, 1), f8, s),
             lambda: V.veda_rope_table(s.view(1, 1, 1).expand(big, 16, 2)),
             lambda: V.veda_add_rms_norm_backward(x, x, None, s, 1e-6, x, None, None, None),
             lambda: V.veda_add_rms_norm_backward_workspace(4, big),
             lambda: V.make_rope(1, 2, 64, (big, 1, 1), (None, None, None)),
             lambda: V.make_rope(big, 2, 64, (1, 1, 1), (None, None, None)),
             lambda: V.make_rope(1, big, 64, (1, 1, 1), (None, None, None))]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError, match="32 bits"):
            call()
            raise AssertionError(f"call {i} was made")
    assert made == []


def test_inputs_whose_gradient_would_be_lost_are_refused(V):
    """Tables and 8-bit operands that want a gradient: there is none, and the call says so."""
    qkv = torch.zeros(1, 24, 3, 2, 64, dtype=torch.bfloat16)
    tables = tuple(torch.zeros(n, dim, 2) for n, dim in zip((2, 3, 4), (12, 10, 10)))
    tables[1].requires_grad_()
    with pytest.raises(ValueError, match="no gradient"):
        V.qkv_norm_rope(qkv, (2, 3, 4), tables, norm="none")
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA tensor"):
        V.qkv_norm_rope(qkv, (2, 3, 4), tables, norm="none")
    a, s = torch.zeros(4, 64, dtype=torch.float8_e4m3fn), torch.ones(1, 4)
    for i in (0, 2):
        args = [a, s, a, s]
        args[i] = a.clone().requires_grad_()
        with pytest.raises(ValueError, match="no gradient"):
            V.gemm_fp8(*args)


@pytest.mark.parametrize("grid", [(2 - 2 ** 32, 3, 4), (2, 3 - 2 ** 32, 4), (-2, -3, 4), (0, 3, 4)])
def test_grids_that_are_none_are_refused(V, grid):
    """A negative size may be a valid one in its low 32 bits, for which the tables are too short."""
    with pytest.raises(ValueError, match="grid dimensions"):
        V.make_rope(1, 2, 64, grid, (None, None, None), norm="none")


def test_rotary_tables_of_another_device_are_refused(V, monkeypatch):
    """The C struct holds addresses only: make_rope takes tables of one device, and the calls take operands of that
    device.  The struct keeps its tables alive."""
    import gc
    import weakref
    B = V.binding

    class On:
        """A tensor as of a device of its own."""

        def __init__(self, t, dev):
            self.t, self.dev, self.is_cuda, self.device = t, dev, True, f"cuda:{dev}"

        def get_device(self):
            return self.dev

        def __getattr__(self, name):
            return getattr(self.t, name)

    def tables(*devs):
        return tuple(On(torch.zeros(n, dim, 2), d) for n, dim, d in zip((2, 3, 4), (12, 10, 10), devs))

    with pytest.raises(ValueError, match="cuda:1"):
        V.make_rope(1, 2, 64, (2, 3, 4), tables(0, 0, 1), norm="none")
    made = []
    monkeypatch.setattr(B, "_call", lambda *a: made.append(a[0]))
    t = tables(0, 0, 0)
    r, ref = V.make_rope(1, 2, 64, (2, 3, 4), t, norm="none"), weakref.ref(t[1])
    del t
    gc.collect()
    assert ref() is not None
    x, o = (torch.zeros(s, dtype=torch.bfloat16) for s in ((1, 24, 2, 64), (1, 2, 24, 64)))
    with pytest.raises(ValueError, match="tables are on cuda:0"):
        V.veda_qkv_norm_rope(r, On(x, 1), None, None, None, None, On(o, 1), None, None)
    with pytest.raises(ValueError, match="tables are on cuda:0"):
        V.veda_qkv_norm_rope_backward(r, None, None, None, None, On(o, 1), None, None, On(x, 1), None, None, None, None, None)
    assert made == []
    V.veda_qkv_norm_rope(r, On(x, 0), None, None, None, None, On(o, 0), None, None)
    assert made == ["veda_qkv_norm_rope"]
    del r
    gc.collect()
    assert ref() is None
