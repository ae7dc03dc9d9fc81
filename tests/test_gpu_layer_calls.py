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
