"""The operators around the pair-bias attention, as a training or serving
program calls them: the linear layers that feed it and read it (bias,
activation and residual in the product's epilogue) and their gradients, the
norm and rotation of queries and keys per head and its gradients, and the
clipping of the gradients by their global norm.

`listed()` names the cases, `draw()` makes more of the same ranges,
`prepare()` makes a case's inputs on the GPU, `run()` is one call, `work()`
what the call cannot do without and `exact()` its results in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")

# The attention's own sizes: 8 query heads and one key head of 128, values of
# 192, at most 8192 positions (1 Mb of sequence); a tower of width 8 * 128.
HEADS, HEAD, VALUE, FULL, WIDTH = 8, 128, 192, 8192, 1024


def listed():
    return [
        # One position through the output projection, for a single-token update.
        dict(name="linear one row", op="linear_fwd", M=1, N=WIDTH, K=HEADS * VALUE, dtype="bf16",
             out="bf16", act="none", bias=True, residual=True, preact=False),
        # The output projection of the attention at full context, with the residual stream.
        dict(name="linear out projection", op="linear_fwd", M=FULL, N=WIDTH, K=HEADS * VALUE,
             dtype="bf16", out="bf16", act="none", bias=True, residual=True, preact=False),
        # The first linear of a feed-forward block over two sequences, its
        # pre-activation kept for the backward.
        dict(name="linear feed-forward", op="linear_fwd", M=2 * FULL, N=4 * WIDTH, K=WIDTH,
             dtype="bf16", out="bf16", act="gelu", bias=True, residual=False, preact=True),
        # A ragged batch and odd widths (rows that no 16-byte load can start on).
        dict(name="linear odd sizes", op="linear_fwd", M=777, N=501, K=1003, dtype="f16",
             out="f32", act="silu", bias=True, residual=False, preact=False),
        # Gradients of the fused query and key projection at full context;
        # the weights' gradient stays in 32 bits.
        dict(name="linear grad projection", op="linear_bwd", M=FULL, N=(HEADS + 1) * HEAD, K=WIDTH,
             dtype="bf16", dx="bf16", dw="f32", act="none", db=True),
        # Gradients of a feed-forward block's second linear, through the
        # activation that made its input.
        dict(name="linear grad feed-forward", op="linear_bwd", M=FULL // 2, N=WIDTH, K=4 * WIDTH,
             dtype="bf16", dx="bf16", dw="bf16", act="gelu", db=True),
        # Queries and keys of one new position in each of four sequences.
        dict(name="qk one position", op="qk_fwd", B=4, L=1, Hq=HEADS, Hk=1, D=HEAD, R=HEAD,
             dtype="bf16", out="bf16", norm="rms", rope="halves", positions=True),
        # Queries and keys of the full context, sliced from the fused projection.
        dict(name="qk full context", op="qk_fwd", B=2, L=FULL, Hq=HEADS, Hk=1, D=HEAD, R=HEAD,
             dtype="bf16", out="bf16", norm="layer", rope="halves", positions=False),
        # Its gradients, from the attention's 32-bit ones, at a mid context
        # with positions that are alignment columns (far apart).
        dict(name="qk grad mid context", op="qk_bwd", B=2, L=FULL // 2, Hq=HEADS, Hk=1, D=HEAD,
             R=HEAD // 2, dtype="bf16", grad="f32", norm="layer", rope="interleaved",
             positions=True),
        # Ragged length, grouped keys, a head that is no power of two.
        dict(name="qk grad odd sizes", op="qk_bwd", B=3, L=333, Hq=6, Hk=2, D=100, R=50,
             dtype="f32", grad="f32", norm="rms", rope="halves", positions=True),
        # The gradients of nine blocks: matrices, biases and norms together.
        dict(name="clip nine blocks", op="clip", blocks=9, width=WIDTH, dtype="f32",
             max_norm=1.0, scale=0.01, packed=False),
        # The small tensors of one narrow block in 16 bits: latency.
        dict(name="clip one narrow block", op="clip", blocks=1, width=96, dtype="bf16",
             max_norm=0.5, scale=0.01, packed=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size of the range: half of them multiples of 8, the others as they fall."""
    n = _log(rng, lo, hi)
    return max(8, n // 8 * 8) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["linear_fwd", "linear_fwd", "linear_bwd", "linear_bwd", "qk_fwd", "qk_bwd", "clip"])
    if op == "linear_fwd":
        return dict(op=op, M=_log(rng, 1, FULL), N=_size(rng, 8, 4 * WIDTH),
                    K=_size(rng, 8, WIDTH), dtype=rng.choice(["bf16", "f16"]),
                    out=rng.choice(["same", "f32"]), act=rng.choice(ACTS),
                    bias=rng.random() < 0.7, residual=rng.random() < 0.5,
                    preact=rng.random() < 0.4)
    if op == "linear_bwd":
        return dict(op=op, M=_log(rng, 1, FULL), N=_size(rng, 8, 2 * WIDTH),
                    K=_size(rng, 8, 2 * WIDTH), dtype=rng.choice(["bf16", "f16"]),
                    dx=rng.choice(["same", "f32"]), dw=rng.choice(["same", "f32"]),
                    act=rng.choice(ACTS), db=rng.random() < 0.7)
    if op in ("qk_fwd", "qk_bwd"):
        D = rng.choice([32, 64, 128, 128, 192, 256, rng.randint(2, 256)])
        R = rng.choice([D // 2 * 2, D // 4 * 2])
        L = _log(rng, 1, FULL)
        c = dict(op=op, B=rng.randint(1, max(1, min(8, FULL // L))), L=L, Hq=rng.randint(1, 12),
                 Hk=rng.randint(1, 4), D=D, R=R, dtype=rng.choice(["bf16", "f16", "f32"]),
                 norm=rng.choice(["none", "rms", "layer"]),
                 rope=rng.choice(["halves", "interleaved"]), positions=rng.random() < 0.5)
        c["out" if op == "qk_fwd" else "grad"] = rng.choice(["bf16", "f32"])
        return c
    return dict(op=op, blocks=rng.randint(1, 8), width=_log(rng, 16, WIDTH),
                dtype=rng.choice(["f32", "bf16", "f16"]), max_norm=rng.choice([0.1, 1.0, 1e4]),
                scale=rng.choice([0.01, 0.1]), packed=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# Inputs
def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _type(case, key):
    t = case[key]
    return DTYPES[case["dtype"] if t == "same" else t]


def _clip_shapes(case):
    """The parameters of `blocks` blocks: the fused query and key projection,
    the value and output projections, the feed-forward pair, biases and norms."""
    w = case["width"]
    one = [(9 * w // 8, w), (w // 4 + 1, w), (w, w), (4 * w, w), (w, 4 * w),
           (9 * w // 8,), (w,), (4 * w,), (w,), (128,), (128,), (w,), (8, 128), (8, w)]
    return one * case["blocks"]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op in ("linear_fwd", "linear_bwd"):
        M, N, K, T = case["M"], case["N"], case["K"], DTYPES[case["dtype"]]
        s["x"] = _rand(gen, M, K).to(T)
        s["W"] = (_rand(gen, N, K) / math.sqrt(K)).to(T)
        if op == "linear_fwd":
            s["b"] = _rand(gen, N) * 0.1 if case["bias"] else None
            s["res"] = _rand(gen, M, N).to(_type(case, "out")) if case["residual"] else None
        else:
            s["dy"] = _rand(gen, M, N).to(T)
            s["z"] = _rand(gen, M, K).to(T) if case["act"] != "none" else None
    elif op in ("qk_fwd", "qk_bwd"):
        B, L, Hq, Hk, D = (case[n] for n in ("B", "L", "Hq", "Hk", "D"))
        T = DTYPES[case["dtype"]]
        fused = (_rand(gen, B, L, (Hq + Hk) * D) * 1.5 + 0.2).to(T)
        s["q"] = fused[..., :Hq * D].view(B, L, Hq, D)
        s["k"] = fused[..., Hq * D:].view(B, L, Hk, D)
        for n in ("q", "k"):
            s[n + "w"] = 1 + 0.2 * _rand(gen, D) if case["norm"] != "none" else None
            s[n + "b"] = 0.1 * _rand(gen, D) if case["norm"] == "layer" else None
        R = case["R"]
        s["freq"] = 10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R) if R else None
        if case["positions"]:  # far positions: columns of a 2^20-wide alignment
            s["pos"] = torch.randint(0, 1 << 20, (B, L), generator=gen, device="cuda").sort(-1).values
        else:
            s["pos"] = None
        if op == "qk_bwd":
            s["gq"] = _rand(gen, B, Hq, L, D).to(DTYPES[case["grad"]])
            s["gk"] = _rand(gen, B, Hk, L, D).to(DTYPES[case["grad"]])
    else:
        # Views of one flat buffer, as a program keeps its gradients: each
        # tensor on a boundary of 64 values, or end to end.
        shapes = _clip_shapes(case)
        step = 1 if case["packed"] else 64
        starts = [0]
        for shape in shapes:
            starts.append(starts[-1] + -(-math.prod(shape) // step) * step)
        s["flat"] = torch.zeros(starts[-1], dtype=DTYPES[case["dtype"]], device="cuda")
        s["grads"] = [s["flat"][at:at + math.prod(shape)].view(shape)
                      for at, shape in zip(starts, shapes)]
        for g in s["grads"]:
            g.copy_(_rand(gen, *g.shape) * case["scale"])
    return s


# ---------------------------------------------------------------------------
# One pass
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import long_context_genomics_b200 as ag

    op = s["op"]
    if op == "linear_fwd":
        return ag.ag_linear_fwd(s["x"], s["W"], bias=s["b"], act=s["act"], residual=s["res"],
                                preact=s["preact"], out_dtype=_type(s, "out"))
    if op == "linear_bwd":
        return ag.ag_linear_bwd(s["dy"], s["x"], s["W"], act=s["act"], preact=s["z"],
                                need_db=s["db"], dx_dtype=_type(s, "dx"), dW_dtype=_type(s, "dw"))
    if op == "qk_fwd":
        return ag.ag_qk_norm_rope_fwd(s["q"], s["k"], q_weight=s["qw"], k_weight=s["kw"],
                                      q_bias=s["qb"], k_bias=s["kb"], norm=s["norm"], eps=1e-6,
                                      inv_freq=s["freq"], rope=s["rope"], positions=s["pos"],
                                      out_dtype=DTYPES[s["out"]])
    if op == "qk_bwd":
        B, L, Hq, Hk, D = s["B"], s["L"], s["Hq"], s["Hk"], s["D"]
        fused = torch.empty(B, L, (Hq + Hk) * D, dtype=s["q"].dtype, device="cuda")
        grads = ag.ag_qk_norm_rope_bwd(
            s["gq"], s["gk"], s["q"], s["k"], q_weight=s["qw"], k_weight=s["kw"], q_bias=s["qb"],
            k_bias=s["kb"], norm=s["norm"], eps=1e-6, inv_freq=s["freq"], rope=s["rope"],
            positions=s["pos"], dq=fused[..., :Hq * D].view(B, L, Hq, D),
            dk=fused[..., Hq * D:].view(B, L, Hk, D))
        return (fused,) + tuple(grads[2:])
    return ag.ag_grad_clip(s["grads"], s["max_norm"]), s["flat"]


def _act(z, act):
    if act == "relu":
        return z * (z > 0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    p = 1 / (1 + torch.exp(-z))
    return p * (1 + z * (1 - p))


def _angles(s):
    pos = s["pos"]
    if pos is None:
        pos = torch.arange(s["L"], device="cuda").expand(s["B"], s["L"])
    a = pos.double()[..., None] * s["freq"]  # [B, L, R / 2], in 64 bits: positions are far
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _pairs(s, x):
    """The two members of each rotated pair, and what is not rotated."""
    R = s["R"]
    if s["rope"] == "halves":
        return x[..., :R // 2], x[..., R // 2:R], x[..., R:]
    return x[..., 0:R:2], x[..., 1:R:2], x[..., R:]


def _join(s, a, b, rest):
    if s["rope"] == "halves":
        return torch.cat([a, b, rest], -1)
    return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)


def _rotate(s, x, sign):
    if not s["R"]:
        return x
    c, sn = _angles(s)
    a, b, rest = _pairs(s, x)
    return _join(s, a * c - b * sn * sign, b * c + a * sn * sign, rest)


def _normed(s, x):
    """x [B, H, L, D] -> (normalised x, its scale)."""
    if s["norm"] == "none":
        return x, None
    if s["norm"] == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    return x * r, r


def _qk_fwd(s, x, w, b, out):
    n, _ = _normed(s, x.float().transpose(1, 2))
    if w is not None:
        n = n * w
    if b is not None:
        n = n + b
    return _rotate(s, n, 1.0).to(out)


def _qk_bwd(s, g, x, w, b):
    n, r = _normed(s, x.float().transpose(1, 2))
    g = _rotate(s, g.float(), -1.0)  # the transposed rotation
    dw = (g.double() * n).sum((0, 1, 2)).float() if w is not None else None
    db = g.double().sum((0, 1, 2)).float() if b is not None else None
    if w is not None:
        g = g * w
    if r is not None:
        d = g - n * (g * n).mean(-1, keepdim=True)
        if s["norm"] == "layer":
            d = d - g.mean(-1, keepdim=True)
        g = d * r
    return g.transpose(1, 2).flatten(2).to(x.dtype), dw, db


def _plain(s):
    op = s["op"]
    if op == "linear_fwd":
        z = s["x"].float() @ s["W"].float().T
        if s["b"] is not None:
            z = z + s["b"]
        y = _act(z, s["act"])
        if s["res"] is not None:
            y = y + s["res"].float()
        y = y.to(_type(s, "out"))
        return (y, z.to(s["x"].dtype)) if s["preact"] else y
    if op == "linear_bwd":
        dy = s["dy"].float()
        dx = dy @ s["W"].float()
        if s["z"] is not None:
            dx = dx * _act_grad(s["z"].float(), s["act"])
        dW = dy.T @ s["x"].float()
        return dx.to(_type(s, "dx")), dW.to(_type(s, "dw")), dy.sum(0) if s["db"] else None
    if op == "qk_fwd":
        out = DTYPES[s["out"]]
        return _qk_fwd(s, s["q"], s["qw"], s["qb"], out), _qk_fwd(s, s["k"], s["kw"], s["kb"], out)
    if op == "qk_bwd":
        dq, dqw, dqb = _qk_bwd(s, s["gq"], s["q"], s["qw"], s["qb"])
        dk, dkw, dkb = _qk_bwd(s, s["gk"], s["k"], s["kw"], s["kb"])
        return torch.cat([dq, dk], -1), dqw, dkw, dqb, dkb
    flat = torch.cat([g.reshape(-1) for g in s["grads"]]).double()
    norm = torch.sqrt((flat * flat).sum())
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0).float()
    [g.copy_(g.float() * coef) for g in s["grads"]]
    return norm.float(), s["flat"]


# ---------------------------------------------------------------------------
# What a pass cannot do without
def work(case):
    op = case["op"]
    size = lambda key: BYTES[case["dtype"] if case[key] == "same" else case[key]]  # noqa: E731
    if op == "linear_fwd":
        M, N, K, e = case["M"], case["N"], case["K"], BYTES[case["dtype"]]
        return {"bytes": e * (M * K + N * K) + size("out") * M * N * (1 + case["residual"])
                + e * M * N * case["preact"] + 4 * N * case["bias"], "flops": 2 * M * N * K}
    if op == "linear_bwd":
        M, N, K, e = case["M"], case["N"], case["K"], BYTES[case["dtype"]]
        return {"bytes": e * (M * N + M * K + N * K + M * K * (case["act"] != "none"))
                + size("dx") * M * K + size("dw") * N * K + 4 * N * case["db"],
                "flops": 4 * M * N * K}
    if op in ("qk_fwd", "qk_bwd"):
        n = case["B"] * case["L"] * (case["Hq"] + case["Hk"]) * case["D"]
        e = BYTES[case["dtype"]]
        pos = 8 * case["B"] * case["L"] * case["positions"]
        if op == "qk_fwd":
            return {"bytes": n * (e + size("out")) + pos, "flops": 10 * n}
        return {"bytes": n * (2 * e + size("grad")) + pos, "flops": 20 * n}
    n = sum(math.prod(shape) for shape in _clip_shapes(case))
    return {"bytes": 2 * BYTES[case["dtype"]] * n, "flops": 3 * n}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
def _exact_act(z, act, grad):
    """act(z), or its derivative by the product rule from its factor of z."""
    if act == "none":
        return torch.ones_like(z) if grad else z
    if act == "relu":
        return torch.heaviside(z, torch.zeros_like(z)) if grad else torch.clamp(z, min=0)
    if act == "gelu":
        gate, slope = torch.special.ndtr(z), torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    else:
        if act == "gelu_tanh":
            u = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z.pow(3))
            du = 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z.square())
        else:
            u, du = z, torch.ones_like(z)
        gate = torch.sigmoid(u)
        slope = gate * torch.sigmoid(-u) * du
    return gate + z * slope if grad else z * gate


def _exact_heads(s, x, w, b, g):
    """Forward (g None) or gradients, with the rotation as complex products."""
    B, L, H, D = x.shape
    R = s["R"]
    x = x.double()
    pos = s["pos"].double() if s["pos"] is not None else torch.arange(L, device=x.device).double().repeat(B, 1)
    at = torch.arange(R // 2, device=x.device)
    lo, hi = (at, at + R // 2) if s["rope"] == "halves" else (2 * at, 2 * at + 1)

    def turn(v, sign):  # v [B, L, H, D]
        v = v.clone()
        if R:
            a = pos[:, :, None] * s["freq"]
            z = torch.complex(v[..., lo], v[..., hi]) * torch.polar(torch.ones_like(a), sign * a)[:, :, None]
            v[..., lo], v[..., hi] = z.real, z.imag
        return v

    w64 = torch.ones(D, device=x.device).double() if w is None else w.double()
    b64 = torch.zeros(D, device=x.device).double() if b is None else b.double()
    if s["norm"] == "layer":
        sigma = torch.sqrt(x.var(-1, unbiased=False, keepdim=True) + 1e-6)
        n = (x - x.mean(-1, keepdim=True)) / sigma
    elif s["norm"] == "rms":
        sigma = torch.sqrt(x.square().sum(-1, keepdim=True) / D + 1e-6)
        n = x / sigma
    else:
        sigma, n = torch.ones_like(x[..., :1]), x
    if g is None:
        return turn(n * w64 + b64, 1.0).permute(0, 2, 1, 3)
    g = turn(g.double().permute(0, 2, 1, 3), -1.0)
    dw, db = torch.einsum("blhd,blhd->d", g, n), torch.einsum("blhd->d", g)
    v = g * w64
    if s["norm"] != "none":
        along = n * (v * n).sum(-1, keepdim=True) / D
        mean = v.sum(-1, keepdim=True) / D if s["norm"] == "layer" else 0.0
        v = (v - mean - along) / sigma
    return v.reshape(B, L, H * D), dw if w is not None else None, db if b is not None else None


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear_fwd":
        z = torch.einsum("mk,nk->mn", s["x"].double(), s["W"].double())
        z = z if s["b"] is None else z + s["b"].double()
        y = _exact_act(z, case["act"], False)
        y = y if s["res"] is None else y + s["res"].double()
        return (y, z) if case["preact"] else y
    if op == "linear_bwd":
        dy, x, W = (s[n].double() for n in ("dy", "x", "W"))
        dx = torch.einsum("mn,nk->mk", dy, W)
        if s["z"] is not None:
            dx = dx * _exact_act(s["z"].double(), case["act"], True)
        return dx, torch.einsum("mn,mk->nk", dy, x), torch.einsum("mn->n", dy) if case["db"] else None
    if op == "qk_fwd":
        return tuple(_exact_heads(s, s[n], s[n + "w"], s[n + "b"], None) for n in ("q", "k"))
    if op == "qk_bwd":
        (dq, dqw, dqb), (dk, dkw, dkb) = (
            _exact_heads(s, s[n], s[n + "w"], s[n + "b"], s["g" + n]) for n in ("q", "k"))
        return torch.cat([dq, dk], -1), dqw, dkw, dqb, dkb
    squares = [g.double().square().sum() for g in s["grads"]]
    norm = torch.stack(squares).sum().sqrt()
    factor = min(1.0, case["max_norm"] / (float(norm) + 1e-6))
    return norm, s["flat"].double() * factor
