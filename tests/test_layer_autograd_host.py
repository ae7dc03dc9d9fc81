"""What the differentiable operators hand to the library, seen on the CPU: the
binding's calls are replaced by ones that write the arguments down."""
import weakref

import pytest
import torch
from torch.utils.checkpoint import checkpoint

GRID, HEADS, D = (2, 3, 4), 2, 64
N = 24


@pytest.fixture(scope="module")
def V():
    import tile_sparse_attention_head_b200 as V
    return V


class Rope:
    """Stands for the C struct: like the addresses in it, it keeps no tensor alive."""

    def __init__(self, b, heads, d, grid, tables):
        self.B, self.heads, self.d, self.grid = b, heads, d, grid
        self.tables = [weakref.ref(t) for t in tables]


@pytest.fixture
def calls(V, monkeypatch):
    """The backward calls made, each as what it was given; the gradients it writes are ones."""
    seen = []
    B = V.binding

    def forward(rope, *args):
        for t in args[-3:]:
            t.zero_()

    def backward(rope, q, k, wq, wk, d_q, d_k, d_v, dq, dk, dv, dwq, dwk, ws):
        tables = [t() for t in rope.tables]
        seen.append(dict(grid=rope.grid, tables=[None if t is None else t.clone() for t in tables],
                         wrote=[n for n, t in zip(("q", "k", "v", "wq", "wk"), (dq, dk, dv, dwq, dwk)) if t is not None]))
        for t in (dq, dk, dv, dwq, dwk):
            if t is not None:
                t.fill_(1)

    monkeypatch.setattr(B, "make_rope", lambda b, heads, d, grid, tables, *how: Rope(b, heads, d, grid, tables))
    monkeypatch.setattr(B, "veda_qkv_norm_rope", forward)
    monkeypatch.setattr(B, "veda_qkv_norm_rope_backward_workspace", lambda rope, device=None: 16)
    monkeypatch.setattr(B, "veda_qkv_norm_rope_backward", backward)
    return seen


def leaves():
    return [t.requires_grad_() for t in (torch.randn(1, N, 3, HEADS, D), torch.ones(HEADS * D), torch.ones(HEADS * D))]


def tables():
    return tuple(torch.full((n, dim, 2), float(10 * n + dim)) for n, dim in zip(GRID, (12, 10, 10)))


@pytest.mark.parametrize("how", ["plain", "checkpoint", "hooks"])
def test_rope_backward_uses_the_tables_that_autograd_kept(V, calls, how):
    """Tables that live only as long as the call: the backward's are those that autograd hands back, not the first
    call's addresses, whose memory may be another tensor's by then."""
    qkv, wq, wk = leaves()

    def call(qkv, wq, wk):
        return V.qkv_norm_rope(qkv, GRID, tables(), wq, wk)

    if how == "checkpoint":
        out = checkpoint(call, qkv, wq, wk, use_reentrant=False)
    elif how == "hooks":
        with torch.autograd.graph.saved_tensors_hooks(lambda t: t.clone(), lambda t: t):
            out = call(qkv, wq, wk)
    else:
        out = call(qkv, wq, wk)
    grads = torch.autograd.grad(out, (qkv, wq, wk), [torch.ones_like(t) for t in out])
    assert len(calls) == 1 and tuple(calls[0]["grid"]) == GRID
    for got, want in zip(calls[0]["tables"], tables()):
        assert got is not None and torch.equal(got, want)
    assert all((g == 1).all() for g in grads)


# ---------------------------------------------------------------- rows as the library reads them

@pytest.mark.parametrize("offset", [0, 1, 4, 8, 12])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_rows_are_laid_out_as_the_library_reads_them(V, dtype, offset):
    """Aligned rows are read in place; what is unaligned, overlapping or strided otherwise is copied."""
    base = torch.randn(64 * 1024).to(dtype)
    assert base.data_ptr() % 64 == 0
    aligned = offset * base.element_size() % 16 == 0
    cases = [(base[offset:offset + 24 * 64].view(24, 64), True),
             (base[offset:offset + 24 * 64].view(2, 3, 4, 64), True),
             (base[:24 * 96].view(24, 96)[:, offset:offset + 64], True),
             (base[offset:offset + 64], True),
             (base[offset:offset + 64].expand(24, 64), False),
             (base[offset:offset + 64 * 24].view(64, 24).t(), False),
             (base[:24 * 100].view(24, 100)[:, offset:offset + 64], False)]
    for t, in_place in cases:
        f = V.layer._flat(t)
        assert f.shape == (t.numel() // t.shape[-1], t.shape[-1]) and f.data_ptr() % 16 == 0
        assert torch.equal(f.reshape(t.shape), t)
        assert f.stride(1) == 1 and (f.stride(0) % 8 == 0 and f.stride(0) >= f.shape[1] or f.shape[0] == 1)
        assert (f.data_ptr() == t.data_ptr()) == (in_place and aligned)


# ---------------------------------------------------------------- what a backward goes through

@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("wants,used,wrote", [
    ("q k v wq wk", "qkv", ["q", "k", "v", "wq", "wk"]), ("q k v wq wk", "k", ["k", "wk"]),
    ("q k v", "qkv", ["q", "k", "v"]), ("wq", "qkv", ["q", "wq"]), ("wq wk", "qkv", ["q", "k", "wq", "wk"]),
    ("wk", "kv", ["k", "wk"])])
def test_rope_backward_leaves_out_what_no_one_asked_for(V, calls, packed, wants, used, wrote):
    """Frozen operands or weights, and outputs that are not used, take no part in the backward call."""
    qkv, wq, wk = leaves()
    xs = [qkv] if packed else [x.detach().clone() for x in qkv.unbind(2)]
    for t, n in zip((*xs, wq, wk), (("q",) if packed else ("q", "k", "v")) + ("wq", "wk")):
        t.requires_grad_(n in wants.split())
    out = V.qkv_norm_rope(xs[0] if packed else xs, GRID, tables(), wq, wk)
    out = [t for t, n in zip(out, "qkv") if n in used]
    ask = [t for t in (*xs, wq, wk) if t.requires_grad]
    grads = torch.autograd.grad(out, ask, [torch.ones_like(t) for t in out], allow_unused=True)
    assert [c["wrote"] for c in calls] == [wrote]
    for t, g in zip(ask, grads):
        if t is qkv:
            assert all((g[:, :, i] == (1 if n in used else 0)).all() for i, n in enumerate("qkv"))
        else:
            name = "wq" if t is wq else "wk" if t is wk else "qkv"[[x is t for x in xs].index(True)]
            assert g is None if name[-1] not in used else (g == 1).all()


def test_rope_backward_of_frozen_operands(V, calls):
    """Only v wants a gradient: q and k are not gone through; no output is used that a leaf depends on: no call."""
    xs = [x.detach().clone() for x in leaves()[0].unbind(2)]
    xs[2].requires_grad_()
    wq, wk = torch.ones(HEADS * D), torch.ones(HEADS * D)
    out = V.qkv_norm_rope(xs, GRID, tables(), wq, wk)
    g, = torch.autograd.grad(out, xs[2], [torch.ones_like(t) for t in out])
    assert calls[0]["wrote"] == ["v"] and (g == 1).all()
    out = V.qkv_norm_rope(xs, GRID, tables(), wq, wk)
    assert torch.autograd.grad(out[0], xs[2], torch.ones_like(out[0]), allow_unused=True) == (None,)
    assert len(calls) == 1
