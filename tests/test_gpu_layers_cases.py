"""More cases of the layers around the attention on a B200: layouts, sizes and
sums that test_gpu_layers.py does not reach.  Tolerances as derived there, or
beside the test."""
import math

import pytest
import torch

import layers_reference as ref
from test_gpu_layers import (BF16, F16, F32, _close, _gen, _half_step, _linear_bwd_case,  # noqa: F401
                             _linear_case, _ok, _randn, ag)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# Queries and keys: gradients into every layout of one buffer
def _fused(layout, B, L, D, fill):
    """A buffer and its query and key slices [B, L, H, D]."""
    t = lambda *s: torch.full(s, fill, dtype=BF16, device="cuda")  # noqa: E731
    if layout == "side by side":
        buf = t(B, L, 9 * D + 64)
        return buf, buf[..., :8 * D].view(B, L, 8, D), buf[..., 8 * D:9 * D].view(B, L, 1, D)
    if layout == "interleaved":  # each head's query, key and value together
        buf = t(B, L, 4, 3, D)
        return buf, buf[:, :, :, 0], buf[:, :, :, 1]
    buf = t(B, 10, L, D)         # the attention's own order
    return buf, buf[:, :8].transpose(1, 2), buf[:, 8:9].transpose(1, 2)


@pytest.mark.parametrize("layout", ["side by side", "interleaved", "heads first"])
@pytest.mark.parametrize("D", [128, 100])
@pytest.mark.parametrize("B,L", [(2, 1), (1, 1), (1, 9), (2, 13)])
def test_qk_bwd_into_one_buffer_of_any_layout(ag, B, L, D, layout):
    """The same values as into tensors of their own; what lies beside stays."""
    g = _gen(B + 7 * L + D)
    src, q, k = _fused(layout, B, L, D, 0.0)
    src.copy_(_randn(g, *src.shape, dtype=BF16))
    gq, gk = (_randn(g, B, t.shape[2], L, D) for t in (q, k))
    kw = dict(inv_freq=ag.ag_rope_frequencies(D))
    want = ag.ag_qk_norm_rope_bwd(gq, gk, q, k, **kw)
    buf, dq, dk = _fused(layout, B, L, D, 7.0)
    ag.ag_qk_norm_rope_bwd(gq, gk, q, k, dq=dq, dk=dk, **kw)
    _ok(ag)
    assert torch.equal(dq, want[0]) and torch.equal(dk, want[1])
    dq.fill_(7.0), dk.fill_(7.0)
    assert bool((buf == 7.0).all()), "wrote beside the gradients"


# ---------------------------------------------------------------------------
# Linear layers
@pytest.mark.parametrize("K", [64, 37])
@pytest.mark.parametrize("far", [1 << 29, (1 << 40) + 1])
def test_linear_one_row_of_any_stride(ag, far, K):
    """The last position of a long sequence: one row, whose stride is never used."""
    g, N = _gen(K), 40
    one = lambda n: torch.as_strided(torch.zeros(n, dtype=BF16, device="cuda"), (1, n), (far, 1))  # noqa: E731
    x, r, y, z, dy, dx = (one(n) for n in (K, N, N, N, N, K))
    for t in (x, r, dy):
        t.copy_(_randn(g, *t.shape, dtype=BF16))
    W = _randn(g, N, K, dtype=BF16)
    plain = [t.clone(memory_format=torch.contiguous_format) for t in (x, r, dy)]
    want = ag.ag_linear_fwd(plain[0], W, act="silu", residual=plain[1], preact=True)
    ag.ag_linear_fwd(x, W, act="silu", residual=r, preact=z, out=y)
    wdx, wdW, wdb = ag.ag_linear_bwd(plain[2], plain[0], W)
    _, dW, db = ag.ag_linear_bwd(dy, x, W, dx=dx)
    _ok(ag)
    for a, b in ((y, want[0]), (z, want[1]), (dx, wdx), (dW, wdW), (db, wdb)):
        assert torch.equal(a, b)
    w = torch.as_strided(W, (1, K), (far, 1))
    assert torch.equal(ag.ag_linear_fwd(plain[0], w), ag.ag_linear_fwd(plain[0], W[:1].clone()))


# ---------------------------------------------------------------------------
# Clipping
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,max_norm", [(8, 1e-2), (8, 1e-6), (1000, 1.0), (19, 1e-30)])
def test_clip_by_a_factor_below_the_normal_numbers(ag, dtype, n, max_norm):
    """Gradients near the largest number: the factor, formed in 64 bits, is a
    subnormal number of 32 bits, which would leave few or none of its digits.
    Two roundings to fp32 (the factor and the product) keep 2^-22."""
    g = (torch.rand(n, generator=_gen(n)) * 1e38 + 1e38).to(dtype).cuda()
    before = g.double()
    norm = ag.ag_grad_clip([g], max_norm)
    _ok(ag)
    size = float(before.square().sum().sqrt())
    want_norm = torch.tensor(size, dtype=torch.float64).float()
    assert float(norm) == math.inf if math.isinf(float(want_norm)) else (
        abs(float(norm) - size) <= size * 2.0 ** -23)
    want = before * (max_norm / size)
    _close("gradient", g, want, want.abs() * 2.0 ** -22 + _half_step(dtype, want) * 1.01
           + 2.0 ** -149)


# ---------------------------------------------------------------------------
# Queries and keys: the angles of 32-bit results
@pytest.mark.parametrize("rope", ["halves", "interleaved"])
@pytest.mark.parametrize("D", [32, 64, 128, 256, 100, 6])
@pytest.mark.parametrize("T", [BF16, F32])
def test_qk_angles_of_32_bit_results(ag, T, D, rope):
    """Rows without a norm: a rotated element is x cos - y sin, each sine and
    cosine within 2^-23 (their own, see the kernel: 1.3 units of 2^-24), the
    product and the sum each within half a unit: (2^-23 + 2 * 2^-24) (|x| + |y|),
    a quarter of what the special-function unit's 2^-21 would need.  The same
    for the gradient of 32-bit queries, which turns back."""
    g, B, L, H = _gen(D), 2, 60, 3
    q = _randn(g, B, L, H, D, dtype=T)
    pos = torch.cat([torch.arange(0, 20), torch.randint(0, 1 << 20, (20,), generator=g),
                     torch.randint(-(1 << 40), 1 << 40, (20,), generator=g)]).cuda()
    freq = ag.ag_rope_frequencies(D)
    kw = dict(norm="none", inv_freq=freq, rope=rope, positions=pos)
    out, _ = ag.ag_qk_norm_rope_fwd(q, None, out_dtype=F32, **kw)
    go = _randn(g, B, H, L, D)
    dq = ag.ag_qk_norm_rope_bwd(go, None, q, None, **kw)[0]
    _ok(ag)
    where = pos.expand(B, L)

    def mass(x):  # |x| + |y| of each element's pair
        m = x.abs()
        i = torch.arange(D, device="cuda")
        return m + m[..., (i + D // 2) % D if rope == "halves" else i ^ 1]

    unit = 2.0 ** -23 + 2 * 2.0 ** -24
    want = ref.rotate(q.double(), where, freq, rope).transpose(1, 2)
    _close("out", out, want, mass(q.double()).transpose(1, 2) * unit)
    if T == F32:
        gt = go.double().transpose(1, 2)
        want = ref.rotate(gt, where, freq, rope, -1.0)
        _close("dq", dq, want, mass(gt) * unit)


@pytest.mark.parametrize("D", [64, 36])
@pytest.mark.parametrize("out", [BF16, F32])
def test_qk_positions_without_a_phase(ag, D, out):
    """Beyond angles of 2^50 the phase is that of rounding, but a row keeps its
    length: a rotation's sine and cosine stay those of some angle."""
    q = _randn(_gen(1), 1, 6, 2, D)
    pos = torch.tensor([1 << 52, -(1 << 55), 1 << 58, 1 << 62, -(1 << 63), (1 << 63) - 1]).cuda()
    o, _ = ag.ag_qk_norm_rope_fwd(q, None, norm="none", inv_freq=ag.ag_rope_frequencies(D),
                                  positions=pos, out_dtype=out)
    _ok(ag)
    size = lambda t: t.double().square().view(*t.shape[:-1], 2, D // 2).sum(-2).sqrt()  # noqa: E731
    want = size(q).transpose(1, 2)
    assert float((size(o) / want - 1).abs().max()) <= 2.0 ** -7


# ---------------------------------------------------------------------------
# Activations element by element
@pytest.mark.parametrize("M", [8, 512])
def test_gelu_and_slope_of_every_size(ag, M):
    """Identity weights and fp32 outputs.  The kernels form z Phi(z) as max(z, 0)
    - |z| t with the tail t = Phi(-|z|) = R exp(-z^2 / 2), R a polynomial in
    u = 1 / (1 + p |z|).  Relative errors, in units of 2^-24: the exponential
    3 z^2 / 2 (three roundings of its argument) + 4 (the function unit); u 3,
    which R, of slope 2.3 at most, makes 7; R's last sums 3, and the products
    2: 16 + 3 z^2 / 2, on top of the polynomial's own fit, 9.2e-8 times
    min(30, 1 / (2 t max(|z|, 1))).  phi(z) in the slope has the exponential's
    and three roundings.  What is below the normal numbers is lost."""
    z = torch.linspace(-14, 14, M * 128).view(M, 128).to(BF16).cuda()
    eye = torch.eye(128, device="cuda").to(BF16)
    y = ag.ag_linear_fwd(z, eye, act="gelu", out_dtype=F32)
    one = torch.ones(M, 128, dtype=BF16, device="cuda")
    dx, _, _ = ag.ag_linear_bwd(one, z, eye, act="gelu", preact=z, need_dW=False, need_db=False,
                                dx_dtype=F32)
    _ok(ag)
    z = z.double()
    x = z.abs()
    phi = torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    tail = 0.5 * torch.erfc(x / math.sqrt(2))
    fit = 9.2e-8 * torch.clamp(1 / (2 * tail * x.clamp(min=1)), max=30)
    of_tail = ((16 + 1.5 * z.square()) * 2.0 ** -24 + fit) * tail
    lost = 14 * 2.0 ** -126
    want = ref.act(z, "gelu")
    _close("y", y, want, x * of_tail + 2.0 ** -24 * want.abs() + lost)
    want = ref.act_slope(z, "gelu")
    of_phi = (7 + 1.5 * z.square()) * 2.0 ** -24 * x * phi
    _close("slope", dx, want, of_tail + of_phi + 2.0 ** -24 * (want.abs() + (z > 0)) + lost)


# ---------------------------------------------------------------------------
# Linear layers of few rows: two kernels, by an estimate of their times
@pytest.mark.parametrize("M", range(1, 10))
@pytest.mark.parametrize("N,K", [(4096, 1024), (1024, 1536), (16384, 1024), (8192, 256), (64, 16384),
                                 (5001, 1003), (40, 72)])
def test_linear_few_rows_on_both_sides_of_the_rule(ag, M, N, K):
    _linear_case(ag, M, N, K, act="gelu")
    _linear_case(ag, M, N, K, T=F16, out=F32, residual=False, preact=False)


def test_linear_few_rows_take_the_tensor_cores_where_those_are_faster(ag):
    """(Only those split a sum, and so take a workspace.)  Measured, us, on the
    weight-streaming kernel and on the tensor cores: 8 x 64 x 65536 67 and 17,
    8 x 1024 x 16384 20 and 15, 2 x 64 x 65536 25 and 17; 8 x 1024 x 1536 5.5 and 8.6,
    4 x 1024 x 8192 6.7 and 13, 1 x 1024 x 16384 7.0 and 17."""
    import ctypes

    def bytes_of(M, N, K):
        n = ctypes.c_int64(-1)
        assert ag.lib.ag_linear_fwd_workspace(256, K, 512, K, M, N, K, ctypes.byref(n)) == 0
        return n.value

    for shape in ((8, 64, 65536), (8, 1024, 16384), (2, 64, 65536)):
        assert bytes_of(*shape) > 0, shape
    for shape in ((8, 1024, 1536), (4, 1024, 8192), (1, 1024, 16384)):
        assert bytes_of(*shape) == 0, shape


@pytest.mark.parametrize("M,N,K", [(4488, 4960, 392), (248, 3136, 360), (136, 2736, 72)])
def test_linear_gradients_near_the_rule_of_one_launch(ag, M, N, K):
    _linear_bwd_case(ag, M, N, K)
    _linear_bwd_case(ag, M, N, K, T=F16, dx_t=F32, dw_t=F16, act="silu")


# ---------------------------------------------------------------------------
# Long sums: nothing left out, nothing counted twice
def _whole(gen, *shape, T=BF16):
    """Whole numbers of -3 to 3 without 0: their products' sums of up to 2^20 terms
    stay below 2^24, so that fp32 holds every partial sum exactly, in any order,
    rounded or truncated."""
    v = torch.randint(1, 4, shape, generator=gen, device="cuda", dtype=torch.int8)
    return (v * (torch.randint(0, 2, shape, generator=gen, device="cuda", dtype=torch.int8) * 2 - 1)).to(T)


LONG = [(70001, 16, 24), (64, 24, 40000), (6, 40, 20001), (9, 4104, 8), (19000, 256, 256),
        (40000, 128, 128), (9000, 301, 701), (8192, 1152, 1024), (3000, 1500, 999),
        (1000, 3008, 600), (300, 200, 5000), (777, 501, 1003), (65536, 128, 128), (2048, 2048, 8),
        (8, 64, 65536), (5, 4096, 1024), (4096, 1024, 4096), (130000, 64, 61), (1, 8, 32768)]


@pytest.mark.parametrize("T", [BF16, F16])
@pytest.mark.parametrize("M,N,K", LONG)
def test_linear_sums_of_whole_numbers_are_exact(ag, M, N, K, T):
    """y, dx, dW and db of whole numbers, bit for bit: a tile, a part of a split
    sum or a part of the rows that is lost or doubled shows, whatever the length
    (a bound on rounded sums of 40000 terms lets 64 of them go)."""
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    x, W, dy = _whole(g, M, K, T=T), _whole(g, N, K, T=T), _whole(g, M, N, T=T)
    b = torch.randint(-100, 100, (N,), generator=g, device="cuda").float()
    xd, Wd, dyd = x.double(), W.double(), dy.double()
    y = ag.ag_linear_fwd(x, W, bias=b, out_dtype=F32)
    _ok(ag)
    assert torch.equal(y.double(), xd @ Wd.T + b.double())
    dx, dW, db = ag.ag_linear_bwd(dy, x, W, dx_dtype=F32)
    only_dx = ag.ag_linear_bwd(dy, x, W, dx_dtype=F32, need_dW=False, need_db=False)[0]
    only_dW = ag.ag_linear_bwd(dy, x, W, need_dx=False, need_db=False)[1]
    only_db = ag.ag_linear_bwd(dy, x, W, need_dx=False, need_dW=False)[2]
    _ok(ag)
    for got, want in ((dx, dyd @ Wd), (dW, dyd.T @ xd), (db, dyd.sum(0))):
        assert torch.equal(got.double(), want)
    assert torch.equal(only_dx, dx) and torch.equal(only_dW, dW) and torch.equal(only_db, db)


def test_the_check_of_whole_numbers_sees_a_lost_tile(ag):
    """The same comparison against oracles with 64 terms, a split's part or one
    row left out, or one counted twice."""
    g = torch.Generator(device="cuda").manual_seed(1)
    M, N, K = 16, 24, 70001
    x, W = _whole(g, M, K), _whole(g, N, K)
    y = ag.ag_linear_fwd(x, W, out_dtype=F32).double()
    _ok(ag)
    xd, Wd = x.double(), W.double()
    assert torch.equal(y, xd @ Wd.T)
    for lost in (slice(64, 128), slice(0, K // 32), slice(K - 1, K)):
        part = xd[:, lost] @ Wd[:, lost].T
        assert not torch.equal(y, xd @ Wd.T - part) and not torch.equal(y, xd @ Wd.T + part)


# ---------------------------------------------------------------------------
# The accumulator is taken over every 512 terms
@pytest.mark.parametrize("kind", ["y", "dx", "dW", "split"])
def test_linear_sums_do_not_drift(ag, kind):
    """32768 positive terms, one product to a cluster (74 tiles: no split), and a
    split one.  The tensor core truncates: each of the steps of a takeover's 512
    terms (16 terms or 8 to a step, at most 64) loses up to 2^-23 of the sum so
    far, on average of half the takeover's: 32 * 2^-23 of the whole.  The 64
    takeovers round by 2^-24 of the sum so far: 32 * 2^-24.  So 48 * 2^-23 =
    5.8e-6 bounds it, and the drift of an accumulator over the whole length
    (2048 steps of 16 terms that lose a quarter of 2^-23 on average: 256 * 2^-23
    and more; measured, 1.6e-4) lies far above."""
    n, M, N = 32768, 74 * 128, 512
    if kind == "split":
        M, N = 64, 40
    g = torch.Generator(device="cuda").manual_seed(5)
    pos = lambda *s: (torch.rand(s, generator=g, device="cuda") + 0.5).to(BF16)  # noqa: E731
    rows = slice(0, 200)
    if kind in ("y", "split"):
        x, W = pos(M, n), pos(N, n)
        got = ag.ag_linear_fwd(x, W, out_dtype=F32)[rows]
        want = x[rows].double() @ W.double().T
    elif kind == "dx":
        dy, W, x = pos(M, n), pos(n, N), pos(M, N)
        got = ag.ag_linear_bwd(dy, x, W, need_dW=False, need_db=False, dx_dtype=F32)[0][rows]
        want = dy[rows].double() @ W.double()
    else:
        dy, x, W = pos(n, M), pos(n, N), pos(M, N)
        got = ag.ag_linear_bwd(dy, x, W, need_dx=False, need_db=False)[1][rows]
        want = dy[:, rows].double().T @ x.double()
    _ok(ag)
    err = (got.double() / want - 1).abs().max()
    assert float(err) <= 48 * 2.0 ** -23


# ---------------------------------------------------------------------------
# Both gradients where TMA can write dx's rows but not dW's (two launches)
@pytest.mark.parametrize("M,N,K,act", [(777, 501, 1004, "none"), (2048, 512, 1004, "none"),
                                       (2048, 1024, 1004, "gelu"), (300, 64, 36, "silu")])
def test_linear_gradients_of_unlike_rows(ag, M, N, K, act):
    """16-bit dW of a row length that is no multiple of 8 beside fp32 dx (and a
    pre-activation with rows apart)."""
    g = _gen(M)
    dy, x = _randn(g, M, N, dtype=BF16), _randn(g, M, K, dtype=BF16)
    W = _randn(g, N, K, dtype=BF16, scale=1 / math.sqrt(N))
    z = torch.zeros(M, K + 4, dtype=BF16, device="cuda")[:, :K]
    z.copy_(_randn(g, M, K, dtype=BF16))
    dx, dW, db = ag.ag_linear_bwd(dy, x, W, act=act, preact=z if act != "none" else None,
                                  dx_dtype=F32, dW_dtype=BF16)
    _ok(ag)
    dyd, xd, Wd = dy.double(), x.double(), W.double()
    want, tol = dyd @ Wd, (N + 8) * 2.0 ** -23 * (dyd.abs() @ Wd.abs())
    if act != "none":
        tol = tol * 1.13 + want.abs() * 2.0 ** -20 * (1 + z.double().abs())
        want = want * ref.act_slope(z.double(), act)
    _close("dx", dx, want, tol * (1 + 2.0 ** -22) + _half_step(F32, want))
    want = dyd.T @ xd
    _close("dW", dW, want, (M + 8) * 2.0 ** -23 * (dyd.abs().T @ xd.abs()) * (1 + 2.0 ** -7)
           + _half_step(BF16, want))
    _close("db", db, dyd.sum(0), (M + 8) * 2.0 ** -24 * dyd.abs().sum(0) + _half_step(F32, dyd.sum(0)))


def test_linear_gradients_where_dW_starts_off_alignment(ag):
    """dW 2 bytes past a 16-byte boundary beside an aligned dx."""
    g = torch.Generator(device="cuda").manual_seed(3)
    M, N, K = 500, 136, 264
    dy, x, W = (_whole(g, *s) for s in ((M, N), (M, K), (N, K)))
    flat = torch.full((N * K + 2,), 7.0, dtype=BF16, device="cuda")
    dW = flat[1:-1].view(N, K)
    dx, _, db = ag.ag_linear_bwd(dy, x, W, dW=dW)
    wdx, wdW, wdb = ag.ag_linear_bwd(dy, x, W, dW_dtype=BF16)
    _ok(ag)
    assert torch.equal(dW, wdW) and torch.equal(db, wdb) and torch.equal(dx, wdx)
    assert float(flat[0]) == 7.0 and float(flat[-1]) == 7.0


def test_lazily_negated_views_are_refused(ag):
    """Their memory holds the values before the change of sign."""
    q = _randn(_gen(1), 1, 4, 2, 8)
    neg = torch._neg_view(q)
    assert neg.is_neg() and torch.equal(neg, -q)
    with pytest.raises(ValueError, match="negated"):
        ag.ag_qk_norm_rope_fwd(neg, None)
    with pytest.raises(ValueError, match="negated"):
        ag.ag_grad_clip([neg], 1.0)
    with pytest.raises(ValueError, match="negated"):
        ag.ag_linear_fwd(torch._neg_view(q[0, 0].to(BF16)), q[0, 1].to(BF16))
    out, _ = ag.ag_qk_norm_rope_fwd(neg.resolve_neg(), None, norm="none", out_dtype=F32)
    _ok(ag)
    assert torch.equal(out, -q.transpose(1, 2))
