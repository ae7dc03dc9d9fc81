"""The operators around the tile-sparse attention of one video transformer layer, as cases to measure.

Three operators: the residual's addition with its RMS norm (in the stream's type, with gradients, or in 8 bits with a
scale per block of 128 channels), the 8-bit matrix product with a scale per block of 128 (alone, or with the
quantisation of the attention's output in front of it), and the way from the QKV product to the attention's grid order
(RMS norm of Q and K, rotary positions over time, height and width, forward and backward).

Sizes: 75,600 tokens x 5,120 channels (40 heads of 128, a 21 x 45 x 80 grid) and 32,760 tokens x 1,536 channels (12 heads
of 128, a 21 x 30 x 52 grid) are this repository's benchmarked layers; the rest is generic.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -100          # blocks whose largest magnitude is below this use it instead
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# residual stream type, type of the sublayers beside it
STREAMS = {"bf16": ("bf16", "bf16"), "fp16": ("fp16", "fp16"), "fp32": ("fp32", "fp32"), "mixed": ("fp32", "bf16")}


def listed():
    return [
        # one token's residual and norm in front of an 8-bit product: a call that is all latency
        dict(name="norm8-token", kind="norm8", rows=1, C=5120, stream="bf16"),
        # the same over a whole video at the larger layer's size
        dict(name="norm8-video", kind="norm8", rows=75600, C=5120, stream="bf16"),
        # a training step of the smaller layer: a 32-bit residual stream beside 16-bit sublayers
        dict(name="norm-train-mixed", kind="norm_train", rows=32760, C=1536, stream="mixed"),
        # odd sizes, all in 32 bits: a last block of channels and a last group of rows that are not full
        dict(name="norm-train-odd", kind="norm_train", rows=1001, C=1000, stream="fp32"),
        # one token through the QKV product: the weights' bytes
        dict(name="gemm-token", kind="gemm", M=1, K=5120, N=15360, bias=False, out="bf16"),
        # a few images' worth of tokens, with a K that ends inside a block and an N that ends inside a tile
        dict(name="gemm-odd", kind="gemm", M=777, K=1552, N=2056, bias=True, out="fp32"),
        # the QKV product of the larger layer over a whole video
        dict(name="gemm-video", kind="gemm", M=75600, K=5120, N=15360, bias=True, out="bf16"),
        # the attention's output of one 30 x 52 latent frame, quantised and projected
        dict(name="proj-frame", kind="proj", B=1, heads=12, d=128, T=1, H=30, W=52, N=1536, bias=True),
        # the same for the smaller layer's whole video
        dict(name="proj-video", kind="proj", B=1, heads=12, d=128, T=21, H=30, W=52, N=1536, bias=True),
        # one token far along the time axis
        dict(name="rope-token", kind="rope", B=1, heads=40, d=128, T=1, H=1, W=1, t0=1000, norm="row",
             pairing="interleaved", dtype="bf16", dims="thirds"),
        # Q, K and V of the larger layer's whole video on their way to the attention
        dict(name="rope-video", kind="rope", B=1, heads=40, d=128, T=21, H=45, W=80, t0=0, norm="row",
             pairing="interleaved", dtype="bf16", dims="thirds"),
        # the smaller layer's, with gradients
        dict(name="rope-train", kind="rope_train", B=1, heads=12, d=128, T=21, H=30, W=52, t0=0, norm="row",
             pairing="interleaved", dtype="bf16", dims="thirds"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm8", "norm_train", "gemm", "proj", "rope", "rope_train"])
    if kind in ("norm8", "norm_train"):
        step = 16 if kind == "norm8" else 8
        C = step * _log(rng, 64 // step, 8192 // step)
        most = (75600 * 5120 if kind == "norm8" else 32760 * 1536 * 2) // C
        return dict(kind=kind, rows=_log(rng, 1, min(75600, most)), C=C, stream=rng.choice(sorted(STREAMS)))
    if kind == "gemm":
        K, N = 16 * _log(rng, 4, 512), 8 * _log(rng, 8, 2048)
        M = _log(rng, 1, min(75600, 75600 * 5120 * 15360 // (K * N)))
        return dict(kind=kind, M=M, K=K, N=N, bias=rng.random() < 0.5, out=rng.choice(["bf16", "fp32"]))
    B, heads, d = rng.choice([1, 1, 1, 2]), _log(rng, 1, 40), rng.choice([64, 128])
    T, H, W = _log(rng, 1, 31), _log(rng, 1, 45), _log(rng, 1, 80)
    most = {"proj": 75600 * 5120, "rope": 75600 * 5120, "rope_train": 32760 * 1536 * 2}[kind]
    while B * T * H * W * heads * d > most:
        T, heads = (T + 1) // 2, (heads + 1) // 2
    if kind == "proj":
        return dict(kind=kind, B=B, heads=heads, d=d, T=T, H=H, W=W, N=8 * _log(rng, 8, 1024), bias=rng.random() < 0.5)
    return dict(kind=kind, B=B, heads=heads, d=d, T=T, H=H, W=W, t0=rng.randrange(0, 200),
                norm=rng.choice(["row", "head", "none"]), pairing=rng.choice(["interleaved", "halves"]),
                dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), dims=rng.choice(["thirds", "quarters", "partial"]))


# ---------------------------------------------------------------- inputs

def _dims(d, how):
    """Channels rotated by time, height and width."""
    if how == "thirds":                       # nearly a third each, the remainder to time
        a = 2 * (d // 6)
        return d - 2 * a, a, a
    if how == "quarters":                     # a quarter to time, three eighths to each of the others
        return d // 4, 3 * d // 8, 3 * d // 8
    return d // 8, d // 4, d // 4             # the last channels keep no position


def _table(n, dim, start, device):
    """(cos, sin) of position * 10000^(-2i/dim), [n, dim/2, 2]: angles in 64 bits, rounded to 32."""
    pos = torch.arange(n, dtype=torch.float64, device=device) + start
    freq = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device=device) / dim)
    a = pos[:, None] * freq[None, :]
    return torch.stack((a.cos(), a.sin()), -1).float().contiguous()


def _fp8_rows(x):
    """[rows, C] in 32 bits -> e4m3 values and scales [blocks, rows], a scale per row and 128 channels."""
    rows, C = x.shape
    blocks = -(-C // 128)
    xp = torch.nn.functional.pad(x, (0, blocks * 128 - C)).view(rows, blocks, 128)
    a = xp.abs().amax(-1).clamp_min(TINY)
    q = (xp * (E4M3_MAX / a)[..., None]).to(torch.float8_e4m3fn)
    return q.view(rows, blocks * 128)[:, :C].contiguous(), (a / E4M3_MAX).t().contiguous()


def _fp8_weight(w):
    """[N, K] in 32 bits -> e4m3 values and scales [ceil(N/128), ceil(K/128)]."""
    N, K = w.shape
    nb, kb = -(-N // 128), -(-K // 128)
    wp = torch.nn.functional.pad(w, (0, kb * 128 - K, 0, nb * 128 - N)).view(nb, 128, kb, 128)
    a = wp.abs().amax((1, 3)).clamp_min(TINY)
    q = (wp * (E4M3_MAX / a)[:, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(nb * 128, kb * 128)[:N, :K].contiguous(), (a / E4M3_MAX).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    kind = case["kind"]
    s = {"case": case}
    if kind in ("norm8", "norm_train"):
        rows, C = case["rows"], case["C"]
        tx, td = (TYPES[t] for t in STREAMS[case["stream"]])
        # a residual stream with some channels much larger than the rest, and a sublayer's output
        s["x"] = (normal(rows, C) * torch.exp(0.7 * normal(C))).to(tx)
        s["delta"] = (0.3 * normal(rows, C)).to(td)
        s["w"] = 1 + 0.2 * normal(C)
        if kind == "norm_train":
            s["dh"], s["dy"] = normal(rows, C).to(tx), normal(rows, C).to(td)
            for t in ("x", "delta", "w"):
                s[t].requires_grad_(True)
    elif kind == "gemm":
        M, K, N = case["M"], case["K"], case["N"]
        s["a"], s["sa"] = _fp8_rows(normal(M, K) * torch.exp(0.5 * normal(K)))
        s["b"], s["sb"] = _fp8_weight(normal(N, K) / math.sqrt(K))
        s["bias"] = 0.1 * normal(N) if case["bias"] else None
    elif kind == "proj":
        tokens, C, N = case["T"] * case["H"] * case["W"], case["heads"] * case["d"], case["N"]
        s["o"] = normal(case["B"], case["heads"], tokens, case["d"]).to(torch.bfloat16)
        s["b"], s["sb"] = _fp8_weight(normal(N, C) / math.sqrt(C))
        s["bias"] = 0.1 * normal(N) if case["bias"] else None
    else:
        B, heads, d, grid = case["B"], case["heads"], case["d"], (case["T"], case["H"], case["W"])
        tokens = grid[0] * grid[1] * grid[2]
        t = TYPES[case["dtype"]]
        s["grid"], s["dims"] = grid, _dims(d, case["dims"])
        s["qkv"] = (normal(B, tokens, 3, heads, d) * torch.exp(0.3 * normal(3, heads, d))).to(t)
        n_w = {"row": heads * d, "head": d, "none": 0}[case["norm"]]
        s["wq"], s["wk"] = ((1 + 0.2 * normal(n_w), 1 + 0.2 * normal(n_w)) if n_w else (None, None))
        s["tables"] = tuple(_table(n, dim, start, "cuda")
                            for n, dim, start in zip(grid, s["dims"], (case["t0"], 0, 0)))
        # first and second channel of each rotated pair, in the pairing that splits each axis's channels in halves
        first = [o + i for o, dim in zip((0, s["dims"][0], s["dims"][0] + s["dims"][1]), s["dims"])
                 for i in range(dim // 2)]
        second = [o + dim // 2 + i for o, dim in zip((0, s["dims"][0], s["dims"][0] + s["dims"][1]), s["dims"])
                  for i in range(dim // 2)]
        s["first"], s["second"] = torch.tensor(first, device="cuda"), torch.tensor(second, device="cuda")
        if kind == "rope_train":
            s["grads"] = tuple(normal(B, heads, tokens, d).to(torch.bfloat16) for _ in range(3))
            for n in ("qkv", "wq", "wk"):
                if s[n] is not None:
                    s[n].requires_grad_(True)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    with torch.no_grad():
        return {"norm8": _norm8, "norm_train": _norm_train, "gemm": _gemm, "proj": _proj, "rope": _rope,
                "rope_train": _rope_train}[s["case"]["kind"]](s)


def _run_own(s):
    import tile_sparse_attention_head_b200 as V
    c = s["case"]
    kind = c["kind"]
    if kind == "norm8":
        return V.add_rms_norm_fp8(s["x"], s["delta"], s["w"], EPS)
    if kind == "norm_train":
        h, y = V.add_rms_norm(s["x"], s["delta"], s["w"], EPS)
        dx, dd, dw = torch.autograd.grad((h, y), (s["x"], s["delta"], s["w"]), (s["dh"], s["dy"]))
        return h, y, dx, dd, dw
    if kind == "gemm":
        return V.gemm_fp8(s["a"], s["sa"], s["b"], s["sb"], bias=s["bias"], out_dtype=TYPES[c["out"]])
    if kind == "proj":
        a, sa = V.quant_fp8_heads(s["o"])
        return V.gemm_fp8(a, sa, s["b"], s["sb"], bias=s["bias"])
    q, k, v = V.qkv_norm_rope(s["qkv"], s["grid"], s["tables"], s["wq"], s["wk"], norm=c["norm"], eps=EPS,
                              pairing=c["pairing"])
    if kind == "rope":
        return q, k, v
    leaves = [t for t in (s["qkv"], s["wq"], s["wk"]) if t is not None]
    return (q, k, v) + torch.autograd.grad((q, k, v), leaves, s["grads"])


def _norm8(s):
    h, y, _ = _add_norm(s)
    q, scale = _fp8_rows(y)
    return h, q, scale


def _add_norm(s):
    h = (s["x"].float() + s["delta"].float()).to(s["x"].dtype)
    hf = h.float()
    rstd = torch.rsqrt(hf.square().mean(-1, keepdim=True) + EPS)
    return h, hf * rstd * s["w"], rstd


def _norm_train(s):
    h, y, rstd = _add_norm(s)
    hf, dy, dh = h.float(), s["dy"].float(), s["dh"].float()
    g = dy * s["w"]
    d = dh + rstd * (g - hf * ((g * hf).mean(-1, keepdim=True) * rstd * rstd))
    dw = (dy * hf * rstd).sum(0)
    return h, y.to(s["delta"].dtype), d.to(s["x"].dtype), d.to(s["delta"].dtype), dw


def _wide(s, q, scale):
    """The values that e4m3 rows with a scale per row and 128 channels stand for, in 32 bits."""
    return q.float() * scale.t().repeat_interleave(128, 1)[:, :q.shape[1]]


def _product(s, a, sa, t):
    b = s["b"].float() * s["sb"].repeat_interleave(128, 0)[:s["b"].shape[0]].repeat_interleave(128, 1)[:, :s["b"].shape[1]]
    c = _wide(s, a, sa) @ b.t()
    return (c if s["bias"] is None else c + s["bias"]).to(t)


def _gemm(s):
    return _product(s, s["a"], s["sa"], TYPES[s["case"]["out"]])


def _proj(s):
    B, heads, n, d = s["o"].shape
    a, sa = _fp8_rows(s["o"].transpose(1, 2).reshape(B * n, heads * d).float())
    return _product(s, a, sa, torch.bfloat16)


def _angles(s):
    """cos and sin [N, 1, pairs] of every token of the grid."""
    (T, H, W), (tt, th, tw) = s["grid"], s["tables"]
    p = torch.cat((tt[:T, None, None].expand(T, H, W, -1, 2), th[None, :H, None].expand(T, H, W, -1, 2),
                   tw[None, None, :W].expand(T, H, W, -1, 2)), 3).reshape(T * H * W, 1, -1, 2)
    return p[..., 0], p[..., 1]


def _rotate(s, x, cos, sin):
    """x [B, N, heads, d] in 32 bits with its pairs turned."""
    R = sum(s["dims"])
    out = x.clone()
    if s["case"]["pairing"] == "interleaved":
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        out[..., 0:R:2], out[..., 1:R:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., s["first"]], x[..., s["second"]]
        out[..., s["first"]], out[..., s["second"]] = a * cos - b * sin, a * sin + b * cos
    return out


def _rstd(s, x):
    axes = {"row": (-1, -2), "head": -1}[s["case"]["norm"]]
    return torch.rsqrt(x.square().mean(axes, keepdim=True) + EPS)


def _normed(s, x, w):
    return x if w is None else x * _rstd(s, x) * w.view(-1, x.shape[-1])


def _rope(s):
    cos, sin = _angles(s)
    q, k, v = s["qkv"].unbind(2)
    q = _rotate(s, _normed(s, q.float(), s["wq"]), cos, sin)
    k = _rotate(s, _normed(s, k.float(), s["wk"]), cos, sin)
    return tuple(t.transpose(1, 2).to(torch.bfloat16).contiguous() for t in (q, k, v))


def _back(s, x, w, dout, cos, sin):
    """Gradients of the normed and turned x, and of w."""
    g = _rotate(s, dout.transpose(1, 2).float(), cos, -sin)
    if w is None:
        return g, None
    r, gw = _rstd(s, x), g * w.view(-1, x.shape[-1])
    axes = {"row": (-1, -2), "head": -1}[s["case"]["norm"]]
    dx = r * (gw - x * ((gw * x).mean(axes, keepdim=True) * r * r))
    dw = (g * x * r).sum((0, 1) if s["case"]["norm"] == "row" else (0, 1, 2))
    return dx, dw.reshape(-1)


def _rope_train(s):
    out = _rope(s)
    cos, sin = _angles(s)
    dq, dk, dv = s["grads"]
    q, k, v = s["qkv"].unbind(2)
    dxq, dwq = _back(s, q.float(), s["wq"], dq, cos, sin)
    dxk, dwk = _back(s, k.float(), s["wk"], dk, cos, sin)
    dqkv = torch.stack((dxq, dxk, dv.transpose(1, 2).float()), 2).to(s["qkv"].dtype)
    return out + ((dqkv,) if dwq is None else (dqkv, dwq, dwk))


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    kind = case["kind"]
    if kind in ("norm8", "norm_train"):
        n = case["rows"] * case["C"]
        bx, bd = (TYPES[t].itemsize for t in STREAMS[case["stream"]])
        if kind == "norm8":       # x, delta in; h, e4m3 and its scales out
            return {"bytes": n * (2 * bx + bd + 1) + case["rows"] * -(-case["C"] // 128) * 4 + 4 * case["C"], "flops": 6 * n}
        return {"bytes": n * (4 * bx + 4 * bd) + 8 * case["C"], "flops": 16 * n}    # and dh, dy in; dx, ddelta out
    if kind in ("gemm", "proj"):
        if kind == "proj":
            M, K, size = case["B"] * case["T"] * case["H"] * case["W"], case["heads"] * case["d"], 2
        else:
            M, K, size = case["M"], case["K"], 1
        N, out = case["N"], TYPES[case.get("out", "bf16")].itemsize
        bytes_ = M * K * size + N * K + M * N * out + 4 * (-(-K // 128)) * (-(-N // 128) + (M if kind == "gemm" else 0))
        return {"bytes": bytes_ + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    n = case["B"] * case["T"] * case["H"] * case["W"] * case["heads"] * case["d"]
    size = TYPES[case["dtype"]].itemsize
    if kind == "rope":
        return {"bytes": 3 * n * (size + 2), "flops": 2 * n * 8}
    return {"bytes": 3 * n * (2 * size + 4), "flops": 2 * n * 24}


# ---------------------------------------------------------------- the same in 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["kind"] in ("norm8", "norm_train"):
            return _exact_norm(case, s)
        if case["kind"] in ("gemm", "proj"):
            return _exact_product(case, s)
        return _exact_rope(case, s)


def _exact_blocks(y):
    """y / scale (not rounded to 8 bits) and the scales of rows in 64 bits."""
    qs, scales = [], []
    for c in range(0, y.shape[1], 128):
        b = y[:, c:c + 128]
        top = torch.clamp(torch.maximum(b.max(1).values, -b.min(1).values), min=TINY)
        qs.append(b * 448.0 / top[:, None])
        scales.append(top / 448.0)
    return torch.cat(qs, 1), torch.stack(scales)


def _exact_norm(case, s):
    total = s["x"].double() + s["delta"].double()
    h = total.to(s["x"].dtype).double()          # the stored residual is what is normalised
    inv = 1 / torch.sqrt((h * h).sum(1) / case["C"] + EPS)
    unit = h * inv[:, None]
    y = unit * s["w"].double()
    if case["kind"] == "norm8":
        q, scale = _exact_blocks(y)
        return total, q, scale
    dy = s["dy"].double()
    g = dy * s["w"].double()
    d = s["dh"].double() + inv[:, None] * (g - unit * ((g * unit).sum(1) / case["C"])[:, None])
    return total, y, d, d, (dy * unit).sum(0)


def _exact_product(case, s):
    N, K = s["b"].shape
    b = s["b"].double()
    for i in range(0, N, 128):
        for j in range(0, K, 128):
            b[i:i + 128, j:j + 128] *= s["sb"][i // 128, j // 128].double()
    if case["kind"] == "proj":
        o = s["o"].double().permute(0, 2, 1, 3).reshape(-1, K)
        q, sa = _exact_blocks(o)
        a = q.float().to(torch.float8_e4m3fn)
    else:
        a, sa = s["a"], s["sa"].double()
    out = []
    for r in range(0, a.shape[0], 16384):
        x = a[r:r + 16384].double()
        for j in range(0, K, 128):
            x[:, j:j + 128] *= sa[j // 128, r:r + 16384, None]
        c = torch.einsum("mk,nk->mn", x, b)
        out.append(c if s["bias"] is None else c + s["bias"].double())
    return torch.cat(out)


def _exact_rope(case, s):
    B, heads, d = case["B"], case["heads"], case["d"]
    T, H, W = s["grid"]
    n = torch.arange(T * H * W, device="cuda")
    places = ((n // (H * W)).double() + case["t0"], (n // W % H).double(), (n % W).double())
    pairs, turns, at = [], [], 0
    for place, dim in zip(places, s["dims"]):
        for i in range(dim // 2):
            pairs.append((at + 2 * i, at + 2 * i + 1) if case["pairing"] == "interleaved" else (at + i, at + dim // 2 + i))
            turns.append(torch.polar(torch.ones_like(place), place * 10000.0 ** (-2.0 * i / dim)))
        at += dim
    turns = torch.stack(turns, 1)[:, None, :]
    one, two = ([p[k] for p in pairs] for k in (0, 1))

    def turned(x, by):
        z = torch.complex(x[..., one], x[..., two]) * by
        y = x.clone()
        y[..., one], y[..., two] = z.real, z.imag
        return y

    def mean(x):
        return x.mean(-1, keepdim=True) if case["norm"] == "head" else x.flatten(2).mean(-1)[..., None, None]

    outs, grads, dws = [], [], []
    for i, w in ((0, s["wq"]), (1, s["wk"]), (2, None)):
        x = s["qkv"][:, :, i].double()
        unit, inv = x, None
        if w is not None:
            inv = 1 / torch.sqrt(mean(x * x) + EPS)
            unit, w = x * inv, w.double().reshape(-1, d)
        y = unit if w is None else unit * w
        outs.append((turned(y, turns) if i < 2 else y).permute(0, 2, 1, 3))
        if case["kind"] == "rope_train":
            dy = s["grads"][i].double().permute(0, 2, 1, 3)
            dy = turned(dy, turns.conj()) if i < 2 else dy
            if w is not None:
                both = (dy * unit).sum((0, 1))
                dws.append(both.sum(0) if case["norm"] == "head" else both.flatten())
                dy = inv * (dy * w - unit * mean(dy * w * unit))
            grads.append(dy)
    return tuple(outs) + ((torch.stack(grads, 2),) + tuple(dws) if grads else ())
