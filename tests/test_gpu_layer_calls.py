"""The ways a program calls the operators around the attention: under autograd's
checkpoints and hooks, and with tensors at other places than an allocation's
start."""
import numpy as np
import pytest
import torch
from torch.utils.checkpoint import checkpoint

pytestmark = pytest.mark.gpu

BF16, FP16, FP32, FP8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def V():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import tile_sparse_attention_head_b200 as V
    return V


def rand(*shape, seed=0, scale=1.0, t=FP32):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(t).cuda()


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---------------------------------------------------------------- autograd

@pytest.mark.parametrize("norm", ["row", "none"])
@pytest.mark.parametrize("how", ["checkpoint", "save_on_cpu"])
def test_gradients_of_a_step_whose_saved_tensors_move(V, how, norm):
    """Residual, norm and rotation inside a checkpoint, or with the saved tensors on the host, and tables that live only
    as long as the call: the gradients are the plain step's, bit for bit, although other tensors have taken the tables'
    memory by the time of the backward."""
    grid, heads, d = (3, 4, 5), 2, 64
    C = 3 * heads * d
    ins = [rand(60, C, seed=1), rand(60, C, seed=2, t=BF16), 1 + 0.2 * rand(C, seed=3)]
    ins += [1 + 0.2 * rand(heads * d, seed=s) for s in (4, 5)] if norm == "row" else []
    douts = [rand(60, C, seed=6)] + [rand(1, heads, 60, d, seed=7 + i, t=BF16) for i in range(3)]

    def step(x, delta, w, wq=None, wk=None):
        h, y = V.add_rms_norm(x, delta, w)
        tables = V.rope_tables(grid, (24, 20, 20), start=(5.0, 1.0, 2.0))
        return (h,) + tuple(V.qkv_norm_rope(y.view(1, 60, 3, heads, d), grid, tables, wq, wk, norm=norm))

    def grads(run):
        leaves = [t.clone().requires_grad_() for t in ins]
        out = run(leaves)
        spoil = [torch.full((n,), 1e30, device="cuda") for n in (64, 96, 128, 128, 192, 256, 512) for _ in range(8)]
        g = torch.autograd.grad(out, leaves, douts)
        del spoil
        return g

    plain = grads(lambda leaves: step(*leaves))
    if how == "checkpoint":
        other = grads(lambda leaves: checkpoint(step, *leaves, use_reentrant=False))
    else:
        def on_cpu(leaves):
            with torch.autograd.graph.save_on_cpu(pin_memory=True):
                return step(*leaves)
        other = grads(on_cpu)
    V.veda_sync_status()
    for i, (a, b) in enumerate(zip(other, plain)):
        assert torch.equal(a, b), i


# ---------------------------------------------------------------- alignment

def at(offset, like):
    """An empty tensor like `like` that starts `offset` bytes past an allocation's start, and the memory around it."""
    n = like.numel() * like.element_size()
    room = torch.full((n + 2 * 64 + offset,), 0xA5, dtype=torch.uint8, device="cuda")
    return room[64 + offset:64 + offset + n].view(like.dtype).view(like.shape), room


def untouched(room, offset):
    return bool((room[:64 + offset] == 0xA5).all()) and bool((room[-64:] == 0xA5).all())


@pytest.mark.parametrize("C", [72, 1000, 8200])
@pytest.mark.parametrize("tx,td", [(FP32, FP32), (FP32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("off", [16, 32, 48])
def test_norm_outputs_on_16_byte_borders(V, off, tx, td, C):
    """Every tensor argument may start on any 16-byte border: inputs and outputs of the norm's calls."""
    rows = 37
    x, delta, w = rand(rows, C, seed=1, t=tx), rand(rows, C, seed=2, t=td), rand(C, seed=3)
    dh, dy = rand(rows, C, seed=4, t=tx), rand(rows, C, seed=5, t=td)

    def run(o):
        rooms = []

        def place(t, fill=True):
            p, room = at(o, t)
            if fill:
                p.copy_(t)
            rooms.append(room)
            return p
        px, pd, pw = place(x), place(delta), place(w)
        h, y, h8, y8 = (place(t, False) for t in (x, delta, x, torch.empty(rows, C, dtype=FP8)))
        s, dx, dd, dw = (place(t, False) for t in (torch.empty(-(-C // 128), rows), x, delta, w))
        V.veda_add_rms_norm(px, pd, pw, 1e-6, h, y)
        V.veda_add_rms_norm_fp8(px, pd, pw, 1e-6, h8, y8, s)
        ws = torch.empty(V.veda_add_rms_norm_backward_workspace(rows, C), dtype=torch.uint8, device="cuda")
        V.veda_add_rms_norm_backward(h, place(dy), place(dh), pw, 1e-6, dx, dd, dw, ws)
        V.veda_sync_status()
        assert all(untouched(r, o) for r in rooms)
        return h, y, h8, y8, s, dx, dd, dw

    for i, (a, b) in enumerate(zip(run(off), run(0))):
        assert same(a, b), i


@pytest.mark.parametrize("t", [FP32, BF16])
@pytest.mark.parametrize("pairing,norm", [("interleaved", "row"), ("halves", "head"), ("interleaved", "none")])
@pytest.mark.parametrize("off", [16, 32])
def test_rope_gradients_on_16_byte_borders(V, off, pairing, norm, t):
    """Inputs, outputs and gradients of the rotary calls on any 16-byte border; one of the three gradients alone too."""
    grid, heads, d, n = (2, 3, 5), 5, 128, 30
    qkv = [rand(1, n, heads, d, seed=i, t=t) for i in range(3)]
    douts = [rand(1, heads, n, d, seed=4 + i, t=BF16) for i in range(3)]
    nw = {"row": heads * d, "head": d, "none": 0}[norm]
    ws = [1 + 0.2 * rand(nw, seed=8 + i) for i in range(2)] if nw else [None, None]
    tables = V.rope_tables(grid, (44, 42, 42))
    r = V.make_rope(1, heads, d, grid, tables, pairing, norm, 1e-6)

    def run(o, only=None):
        rooms = []

        def place(x, fill=True):
            if x is None:
                return None
            p, room = at(o, x)
            if fill:
                p.copy_(x)
            rooms.append(room)
            return p
        w, xs = [place(x) for x in ws], [place(x) for x in qkv]
        outs = [place(x, False) for x in douts]
        V.veda_qkv_norm_rope(r, *xs, *w, *outs)
        grads = [place(x, False) if only in (None, i) else x.clone().zero_() for i, x in enumerate(qkv)]
        dws = [place(x, False) for x in ws]
        scratch = torch.empty(V.veda_qkv_norm_rope_backward_workspace(r), dtype=torch.uint8, device="cuda")
        V.veda_qkv_norm_rope_backward(r, xs[0], xs[1], *w, *(place(x) for x in douts), *grads, *dws, scratch)
        V.veda_sync_status()
        assert all(untouched(x, o) for x in rooms)
        return outs + grads + [x for x in dws if x is not None]

    want = run(0)
    for only in (None, 1):
        for i, (a, b) in enumerate(zip(run(off, only), want)):
            assert same(a, b), (only, i)


# ---------------------------------------------------------------- many products in flight

def test_products_in_flight_repeat_their_bits(V):
    """Products of many blocks and tiles per pair of CTAs, two streams at once: each result has the first one's bits
    (in the pair's second CTA too, whose rows are 128 to 255 of a tile), and that one is right."""
    cases = []
    for M, K, N, out in ((5000, 2560, 2560, BF16), (777, 1552, 2056, FP32), (3000, 1536, 1536, FP32), (2100, 144, 2048, BF16)):
        g = torch.Generator(device="cuda").manual_seed(M)
        a, b = (torch.randn(n, K, generator=g, device="cuda").to(FP8) for n in (M, N))
        kb = -(-K // 128)
        # scales that differ from row to row and block to block by powers of two
        sa = torch.exp2(torch.randint(-4, 5, (kb, M), generator=g, device="cuda").float())
        sb = torch.exp2(torch.randint(-4, 5, (-(-N // 128), kb), generator=g, device="cuda").float())
        cases.append((a, sa, b, sb, out))
        A = a.double() * sa.double().t().repeat_interleave(128, 1)[:, :K]
        B = b.double() * sb.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
        c = V.gemm_fp8(a, sa, b, sb, out_dtype=out)
        # products are exact; 128 additions in a block and one multiply-add per block, 2^-23 of the magnitudes each
        lim = torch.finfo(out).eps / 2 * (A @ B.t()).abs() + (128 + 4 * kb) * 2.0 ** -23 * (A.abs() @ B.abs().t()) * 1.01
        assert bool(((c.double() - A @ B.t()).abs() <= lim).all())
    want = [V.gemm_fp8(a, sa, b, sb, out_dtype=out) for a, sa, b, sb, out in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(25):
        got = []
        for i, (a, sa, b, sb, out) in enumerate(cases):
            for s in streams:
                with torch.cuda.stream(s):
                    got.append((i, V.gemm_fp8(a, sa, b, sb, out_dtype=out)))
        torch.cuda.synchronize()
        assert all(torch.equal(c, want[i]) for i, c in got)
    V.veda_sync_status()


# ---------------------------------------------------------------- the 8-bit rule

def rule(x, per_row=True):
    """The 8-bit rule in fp32 on the host, bit for bit: bytes and scales of blocks of 128 channels (and rows)."""
    x = x.float().cpu().numpy()
    R, C = x.shape
    q, nb = np.empty((R, C), np.float32), -(-C // 128)
    s = np.empty((nb, R) if per_row else (-(-R // 128), nb), np.float32)
    for j in range(nb):
        for i in range(0, R, R if per_row else 128):
            b = x[i:i + (R if per_row else 128), 128 * j:128 * j + 128]
            a = np.abs(b).max(1, keepdims=True) if per_row else np.abs(b).max(keepdims=True)
            a = np.maximum(a, np.float32(2.0 ** -100))
            q[i:i + len(b), 128 * j:128 * j + 128] = b * (np.float32(448) / a)
            (s[j:j + 1] if per_row else s[i // 128, j:j + 1])[...] = (a * (np.float32(1) / np.float32(448))).ravel()
    return torch.from_numpy(np.clip(q, -448, 448)).to(FP8), torch.from_numpy(s)


def midpoints(rows, C, seed=0):
    """Rows whose values lie on the borders between neighbouring e4m3 values once they are scaled, all exact: the
    largest of a block is 448 times a power of two."""
    g = np.random.default_rng(seed)
    grid = np.arange(0x08, 0x7E, dtype=np.uint8)
    grid = torch.from_numpy(grid).view(FP8).float().numpy()
    mid = (grid[1:] + grid[:-1]) / 2
    x = g.choice(np.concatenate((mid, grid)), (rows, C)) * g.choice([-1.0, 1.0], (rows, C))
    x[:, ::128] = 448
    return torch.from_numpy((x * np.exp2(g.integers(-20, 20, (rows, 1)))).astype(np.float32)).cuda()


@pytest.mark.parametrize("t", [FP32, BF16, FP16])
def test_quantisers_keep_the_rule_bit_for_bit(V, t):
    """448 / a is correctly rounded and multiplied once: no byte differs from the rule in fp32, on random rows and on
    the borders between e4m3 values (which bf16 and fp16 hold exactly too, within fp16's range)."""
    mid = midpoints(130, 264)
    rnd = rand(4000, 1000, seed=1) * torch.exp(2 * rand(4000, 1, seed=2))
    for x in (mid if t is not FP16 else mid.clamp(-448 * 64, 448 * 64) / 64, rnd):
        x = x.to(t)
        q, s = V.quant_fp8(x)
        rq, rs = rule(x)
        assert same(q.cpu(), rq) and same(s.cpu(), rs)
        q, s = V.quant_fp8_weight(x)
        rq, rs = rule(x, per_row=False)
        assert same(q.cpu(), rq) and same(s.cpu(), rs)
    o = rand(2, 3, 500, 64, seed=3, t=t)
    q, s = V.quant_fp8_heads(o)
    rq, rs = rule(o.transpose(1, 2).reshape(1000, 192))
    assert same(q.cpu(), rq) and same(s.cpu(), rs)


@pytest.mark.parametrize("rows,C", [(8192, 4096), (3000, 1000), (501, 256), (300, 8200)])
def test_norm_and_quantiser_have_one_rule(V, rows, C):
    """With an fp32 stream the norm's fp32 output, quantised, is its 8-bit output: the same bytes and scales."""
    x, delta, w = rand(rows, C, seed=1), rand(rows, C, seed=2, scale=0.3), 1 + 0.2 * rand(C, seed=3)
    h, y = V.add_rms_norm(x, delta, w)
    h8, q, s = V.add_rms_norm_fp8(x, delta, w)
    q2, s2 = V.quant_fp8(y)
    assert same(h, h8) and same(s, s2)
    assert same(q, q2), int((q.view(torch.uint8) != q2.view(torch.uint8)).sum())


# ---------------------------------------------------------------- the attention block

def test_attention_blocks_on_an_fp16_stream(V):
    """Two blocks in a row on an fp16 residual stream: the first one's output (bf16) is the second one's delta."""
    from parity import mlp_device
    from veda_synth import PRESETS, make_mlp
    w = PRESETS["tiny"]
    p = V.Problem(w.B, w.heads, w.d, w.S, (w.T, w.H, w.W), w.tilings)
    C, inner = 640, w.heads * w.d
    mlp = mlp_device(make_mlp(w, seed=1))
    att = V.VedaAttention(p, mlp, mlp, w.keep)
    tables = V.rope_tables(p.grid, (w.d // 4, 3 * w.d // 8, 3 * w.d // 8))
    nw, ones = 1 + 0.2 * rand(C, seed=2), torch.ones(inner, device="cuda")
    block = V.VedaSelfAttention(att, rand(3 * inner, C, seed=3, scale=C ** -0.5, t=FP16),
                                rand(C, inner, seed=4, scale=inner ** -0.5, t=FP16), nw, tables, ones, ones)
    x, delta = rand(p.B, p.N, C, seed=5, t=FP16), None
    for _ in range(2):
        h, out = block(x, delta)
        V.veda_sync_status()
        assert h.dtype == FP16 and out.dtype == BF16 and h.shape == out.shape == x.shape
        want = x if delta is None else (x.float() + delta.float()).half()
        # one rounding, and 2^-25 more where the delta is below fp16's normal range
        assert bool(((h.float() - want.float()).abs() <= 2.0 ** -24 + want.float().abs() * 2.0 ** -11).all())
        _, y8, ys = V.add_rms_norm_fp8(h, None, nw)
        qkv = V.gemm_fp8(y8, ys, block.w_qkv, block.s_qkv)
        q, k, v = V.qkv_norm_rope(qkv.view(p.B, p.N, 3, p.heads, p.d), p.grid, tables, ones, ones)
        o8, os = V.quant_fp8_heads(att(q, k, v))
        assert torch.equal(out, V.gemm_fp8(o8, os, block.w_o, block.s_o).view(out.shape))
        assert bool(torch.isfinite(out).all())
        x, delta = h, out


def test_inputs_at_any_element(V):
    """The torch functions take rows that start at any element, with gradients too."""
    x, delta, w = rand(33, 200, seed=1, t=BF16), rand(33, 200, seed=2, t=BF16), 1 + 0.2 * rand(200, seed=3)
    dy = rand(33, 200, seed=4, t=BF16)

    def odd(t):
        p = torch.empty(t.numel() + 3, dtype=t.dtype, device="cuda")[3:].view(t.shape)
        return p.copy_(t)

    def run(put):
        leaves = [put(x).requires_grad_(), put(delta).requires_grad_(), w.clone().requires_grad_()]
        h, y = V.add_rms_norm(*leaves)
        g = torch.autograd.grad((h, y), leaves, (dy, put(dy)))
        with torch.no_grad():
            return [h, y, *g, *V.add_rms_norm_fp8(*leaves), *V.quant_fp8(put(x)), *V.quant_fp8(put(x).view(3, 11, 200))]

    for i, (a, b) in enumerate(zip(run(odd), run(lambda t: t.clone()))):
        assert same(a, b), i
    V.veda_sync_status()


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("norm", ["row", "head"])
def test_gradients_of_some_rotary_inputs_alone(V, norm, packed):
    """The gradients of the weights alone, of one operand alone, and of one output alone are the full step's."""
    grid, heads, d = (2, 3, 5), 3, 64
    nw = heads * d if norm == "row" else d
    qkv = rand(2, 30, 3, heads, d, seed=1, t=BF16)
    xs = [qkv] if packed else [t.clone() for t in qkv.unbind(2)]
    ws = [1 + 0.2 * rand(nw, seed=2), 1 + 0.2 * rand(nw, seed=3)]
    douts = [rand(2, heads, 30, d, seed=4 + i, t=BF16) for i in range(3)]
    tables = V.rope_tables(grid, (24, 20, 20))

    def grads(which, used=(0, 1, 2)):
        leaves = [t.clone().requires_grad_(i in which) for i, t in enumerate(xs + ws)]
        out = V.qkv_norm_rope(leaves[0] if packed else leaves[:3], grid, tables, *leaves[-2:], norm=norm)
        return torch.autograd.grad([out[i] for i in used], [leaves[i] for i in which], [douts[i] for i in used])

    n = len(xs)
    full = grads(range(n + 2))
    for which in ([n], [n + 1], [n, n + 1], [0], [n - 1], [0, n + 1]):
        for i, g in zip(which, grads(which)):
            assert torch.equal(g, full[i]), (which, i)
    g, = grads([n], used=(0,))
    assert torch.equal(g, full[n])
    V.veda_sync_status()
