"""The layers around the attention against 64-bit formulas on a B200.

Tolerances, per element, from the arithmetic (derived, not fitted):

* Products.  K exact products of 16-bit values are summed in float32 in some
  order, each addition rounded or truncated: at most K + 8 units of 2^-23 of
  the sum of the terms' magnitudes A = |x| |W|^T (the 8 covers bias and
  residual and the joining of partial sums).
* A rounding to an output type t moves a value by at most half a step,
  finfo(t).eps / 2 of its magnitude (plus half the smallest subnormal).
* An activation multiplies an error of its argument by at most 1.13 (its
  largest slope) and adds its own evaluation error, below 2^-20 (1 + |z|):
  an exponential of |z| <= 2^6 from a scaled argument errs by about |z| 2^-23.
  A derivative likewise, with slopes of slopes below 1.13 too.
* Norms.  A row's sums of D terms err by at most D / 32 + 8 additions of
  2^-24 of their terms' magnitudes, 2^-24 (D / 32 + 8) < 2^-18 relative for
  D <= 1024; a handful of further float32 operations and an angle within
  2^-21 (a reduced angle below pi in float32) keep a value within 2^-17 of its
  row's largest.  For the layer norm the mean's error is 2^-18 of the mean
  |x|, so the row's scale is max |n| + |mean| r.
* Parameter gradients sum n terms in float32 chains: n 2^-24 of the sum of
  the terms' magnitudes, on top of each term's own 2^-17.
"""
import math

import numpy as np
import pytest
import torch

import layers_reference as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def ag():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import long_context_genomics_b200 as ag

    return ag


def _randn(gen, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(dtype).cuda()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _half_step(dtype, want):
    info = torch.finfo(dtype)
    return want.abs() * info.eps / 2 + info.tiny * info.eps / 2


def _close(name, got, want, tol):
    assert got.shape == want.shape, name
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    if bool(bad.any()):
        at = int(torch.argmax((err / tol.clamp(min=1e-300)).flatten()))
        raise AssertionError(
            f"{name}: {int(bad.sum())} of {bad.numel()} beyond their bound; worst at {at}: got "
            f"{got.flatten()[at].item()}, want {want.flatten()[at].item()}, bound "
            f"{tol.flatten()[at].item():.3e}")


def _padded(t, pad, sentinel=7.0):
    """A copy of matrix t whose rows lie `pad` elements further apart, and the
    whole buffer, whose gaps hold a sentinel."""
    full = torch.full((t.shape[0], t.shape[1] + pad), sentinel, dtype=t.dtype, device=t.device)
    view = full[:, :t.shape[1]]
    view.copy_(t)
    return view, full


def _ok(ag):
    torch.cuda.synchronize()
    assert ag.ag_device_error(0) == 0


# ---------------------------------------------------------------------------
# Linear layers, forward
def _linear_case(ag, M, N, K, T=BF16, out=None, act="none", bias=True, residual=True, preact=True,
                 pad=0, seed=0):
    g = _gen(seed + M + 3 * N + 7 * K)
    x, W = _randn(g, M, K, dtype=T), _randn(g, N, K, dtype=T, scale=1 / math.sqrt(K))
    out = out or T
    b = _randn(g, N) if bias else None
    r = _randn(g, M, N, dtype=out) if residual else None
    y_t, y_full = _padded(torch.zeros(M, N, dtype=out, device="cuda"), pad)
    z_t, z_full = _padded(torch.zeros(M, N, dtype=T, device="cuda"), pad)
    if pad:
        x, _ = _padded(x, pad)
        W, _ = _padded(W, pad)
        if r is not None:
            r, _ = _padded(r, pad)
    got = ag.ag_linear_fwd(x, W, bias=b, act=act, residual=r, preact=z_t if preact else False,
                           out=y_t)
    _ok(ag)
    y, z = got if preact else (got, None)
    xd, Wd = x.double(), W.double()
    want_z = xd @ Wd.T
    A = xd.abs() @ Wd.abs().T
    if b is not None:
        want_z, A = want_z + b.double(), A + b.double().abs()
    tol_z = (K + 8) * 2.0 ** -23 * A
    want = ref.act(want_z, act)
    tol = tol_z * (1.0 if act == "none" else 1.13)
    if act != "none":
        tol = tol + 2.0 ** -20 * (1 + want_z.abs())
    if r is not None:
        want = want + r.double()
        tol = tol + 2.0 ** -23 * (want.abs() + r.double().abs())
    tol = tol * (1 + torch.finfo(out).eps) + _half_step(out, want)
    _close("y", y, want, tol)
    if preact:
        _close("preact", z, want_z, tol_z * (1 + torch.finfo(T).eps) + _half_step(T, want_z))
    if pad:
        assert bool((y_full[:, N:] == 7.0).all()), "wrote between the rows of y"
        assert bool((z_full[:, N:] == 7.0).all() or not preact), "wrote between the rows of preact"
    return got


SIZES = [(1, 8, 8), (1, 1, 1), (1, 1024, 1536), (2, 128, 256), (3, 5, 7), (7, 136, 72),
         (8, 1024, 1536), (9, 512, 512), (16, 72, 1000), (33, 200, 64), (127, 128, 128),
         (128, 256, 64), (129, 257, 65), (255, 120, 520), (256, 256, 512), (257, 264, 136),
         (300, 384, 1024), (513, 1000, 96), (777, 501, 1003), (1024, 1152, 1024),
         (2048, 64, 40), (5000, 31, 128)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear_fwd_sizes(ag, M, N, K):
    _linear_case(ag, M, N, K)


@pytest.mark.parametrize("M", [1, 100])
@pytest.mark.parametrize("T,out", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_linear_fwd_types_and_activations(ag, M, T, out, act):
    _linear_case(ag, M, 264, 192, T=T, out=out, act=act)


@pytest.mark.parametrize("bias,residual,preact", [(False, False, False), (True, False, False),
                                                  (False, True, False), (False, False, True)])
@pytest.mark.parametrize("M", [1, 200])
def test_linear_fwd_options(ag, M, bias, residual, preact):
    _linear_case(ag, M, 136, 264, bias=bias, residual=residual, preact=preact, act="gelu")


@pytest.mark.parametrize("pad", [1, 4, 8, 64])
@pytest.mark.parametrize("M,N,K", [(1, 40, 72), (5, 264, 520), (130, 136, 72), (300, 61, 37)])
def test_linear_fwd_rows_apart(ag, M, N, K, pad):
    """Row strides beyond the rows, at every alignment; the gaps stay as they were."""
    _linear_case(ag, M, N, K, pad=pad, act="silu")
    _linear_case(ag, M, N, K, pad=pad, out=F32)


@pytest.mark.parametrize("M,N,K", [(70001, 16, 24), (64, 24, 40000), (9, 4104, 8), (8, 3001, 17),
                                   (6, 40, 20001)])
def test_linear_long_sides(ag, M, N, K):
    """Many rows, long sums (split over clusters), and few rows beside wide ones."""
    _linear_case(ag, M, N, K, out=F32, preact=False)
    if M > 8:
        _linear_bwd_case(ag, M, N, K)


def test_linear_fwd_columns_of_one_buffer(ag):
    """x and y as column ranges of the same wider buffer; its other columns stay."""
    for M in (3, 500):
        g = _gen(M)
        buf = _randn(g, M, 64 + 96 + 40, dtype=BF16)
        keep = buf.clone()
        W = _randn(g, 96, 64, dtype=BF16)
        want = ag.ag_linear_fwd(buf[:, :64].contiguous(), W)
        ag.ag_linear_fwd(buf[:, :64], W, out=buf[:, 64:160])
        _ok(ag)
        assert torch.equal(buf[:, 64:160], want)
        assert torch.equal(buf[:, :64], keep[:, :64]) and torch.equal(buf[:, 160:], keep[:, 160:])
        with pytest.raises(ag.AgError, match="ALIAS"):
            ag.ag_linear_fwd(buf[:, :64], W, out=buf[:, 63:159])


def test_linear_fwd_starts_off_alignment(ag):
    """Inputs and outputs that start 2 bytes past a 16-byte boundary."""
    g = _gen(5)
    for M in (1, 150):
        flat = _randn(g, 1 + M * 72, dtype=BF16)
        x = flat[1:].view(M, 72)
        W = _randn(g, 1 + 40 * 72, dtype=BF16)[1:].view(40, 72)
        y = torch.zeros(1 + M * 40, dtype=BF16, device="cuda")
        ag.ag_linear_fwd(x, W, out=y[1:].view(M, 40))
        _ok(ag)
        want = x.double() @ W.double().T
        tol = 80 * 2.0 ** -23 * (x.double().abs() @ W.double().abs().T) + _half_step(BF16, want)
        _close("y", y[1:].view(M, 40), want, tol * 1.01)
        assert float(y[0]) == 0.0


def test_linear_fwd_in_place_residual(ag):
    for M, N, K in ((4, 64, 64), (300, 136, 4096)):
        g = _gen(M)
        x, W = _randn(g, M, K, dtype=BF16), _randn(g, N, K, dtype=BF16, scale=K ** -0.5)
        r = _randn(g, M, N, dtype=BF16)
        want = ag.ag_linear_fwd(x, W, residual=r)
        y = r.clone()
        ag.ag_linear_fwd(x, W, residual=y, out=y)
        _ok(ag)
        assert torch.equal(y, want)


def test_linear_fwd_non_finite_values_stay_in_their_rows_and_columns(ag):
    """An infinity or NaN in one row of x reaches that row of y only, one in a
    row of W that column only: nothing leaks through a tile's padding."""
    for M, N, K in ((3, 24, 40), (200, 136, 200), (130, 61, 37)):
        g = _gen(K)
        x, W = _randn(g, M, K, dtype=BF16), _randn(g, N, K, dtype=BF16)
        x[M - 1, K - 1] = math.inf
        W[N - 1, 0] = math.nan
        y = ag.ag_linear_fwd(x, W)
        _ok(ag)
        fine = torch.isfinite(y)
        assert bool(fine[:M - 1, :N - 1].all())
        assert not bool(fine[M - 1].any()) and not bool(fine[:, N - 1].any())


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M", [4, 512])
def test_activations_and_slopes_closely(ag, act, M):
    """Identity weights and fp32 outputs leave the activation and its derivative
    alone: values of order one, formed in a few fp32 operations each off by half
    a unit of 2^-23 and two special-function results of one unit: 2-norms agree
    to 2^-22."""
    x = _randn(_gen(3), M, 128, dtype=BF16)
    eye = torch.eye(128, device="cuda").to(BF16)
    y = ag.ag_linear_fwd(x, eye, act=act, out_dtype=F32)
    one = torch.ones(M, 128, dtype=BF16, device="cuda")
    dx, _, _ = ag.ag_linear_bwd(one, x, eye, act=act, preact=x, need_dW=False, need_db=False,
                                dx_dtype=F32)
    _ok(ag)
    for got, want in ((y, ref.act(x.double(), act)), (dx, ref.act_slope(x.double(), act))):
        assert float((got.double() - want).norm()) <= 2.0 ** -22 * float(want.norm())


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M,K", [(8, 8), (256, 64), (256, 61)])
def test_activations_and_slopes_of_large_values(ag, act, M, K):
    """Far from zero every activation is z or 0 and its slope 1 or 0, up to the
    largest numbers, whose squares and cubes are none any more."""
    z = torch.tensor([100.0, 1e4, 1e10, 1e13, 1e19, 1e25, 1e38, 3e38], device="cuda")
    z = torch.cat([z, -z]).repeat((M * K + 15) // 16)[:M * K].view(M, K).to(BF16)
    eye = torch.eye(K, device="cuda").to(BF16)
    y = ag.ag_linear_fwd(z, eye, act=act, out_dtype=F32)
    one = torch.ones(M, K, dtype=BF16, device="cuda")
    dx, _, _ = ag.ag_linear_bwd(one, z, eye, act=act, preact=z, need_dW=False, need_db=False,
                                dx_dtype=F32)
    _ok(ag)
    # (silu(-100) is -3.7e-42, and its slope as near to zero.)
    zero = torch.where(z > 0, 0.0, 1e-40)
    assert bool(((y - z.float().clamp(min=0)).abs() <= zero).all())
    assert bool(((dx - (z > 0).float()).abs() <= zero).all())


def test_linear_fwd_accumulates_in_32_bits(ag):
    """A long sum of equal terms beside one large term: 16-bit partial sums, or
    a truncating accumulator over the whole length, would lose it."""
    for M in (1, 64):
        K = 16384
        x = torch.ones(M, K, dtype=BF16, device="cuda")
        W = torch.full((8, K), 2.0 ** -7, dtype=BF16, device="cuda")
        W[:, 0] = 256.0
        y = ag.ag_linear_fwd(x, W, out_dtype=F32)
        _ok(ag)
        want = 256.0 + (K - 1) * 2.0 ** -7
        assert float((y - want).abs().max()) <= want * 2.0 ** -18


def test_linear_empty(ag):
    x = torch.zeros(0, 16, dtype=BF16, device="cuda")
    W = torch.zeros(8, 16, dtype=BF16, device="cuda")
    y, z = ag.ag_linear_fwd(x, W, preact=True)
    assert y.shape == (0, 8) and z.shape == (0, 8)
    dW = torch.full((8, 24), 3.0, device="cuda")
    dx, dW_got, db = ag.ag_linear_bwd(torch.zeros(0, 8, dtype=BF16, device="cuda"), x, W,
                                      dW=dW[:, :16])
    torch.cuda.synchronize()
    assert dx.shape == (0, 16) and not bool(dW[:, :16].any()) and not bool(db.any())
    assert bool((dW[:, 16:] == 3.0).all())


def test_linear_is_reproducible(ag):
    g = _gen(9)
    x, W = _randn(g, 700, 2000, dtype=BF16), _randn(g, 136, 2000, dtype=BF16)
    dy = _randn(g, 700, 136, dtype=BF16)
    first = [ag.ag_linear_fwd(x, W, out_dtype=F32), *ag.ag_linear_bwd(dy, x, W)]
    for _ in range(3):
        again = [ag.ag_linear_fwd(x, W, out_dtype=F32), *ag.ag_linear_bwd(dy, x, W)]
        assert all(torch.equal(a, b) for a, b in zip(first, again))


# ---------------------------------------------------------------------------
# Linear layers, backward
def _linear_bwd_case(ag, M, N, K, T=BF16, dx_t=None, dw_t=F32, act="none", pad=0, db=True):
    g = _gen(M + 5 * N + 11 * K)
    dx_t = dx_t or T
    dy, x = _randn(g, M, N, dtype=T), _randn(g, M, K, dtype=T)
    W = _randn(g, N, K, dtype=T, scale=1 / math.sqrt(N))
    z = _randn(g, M, K, dtype=T) if act != "none" else None
    dx_o, dx_full = _padded(torch.zeros(M, K, dtype=dx_t, device="cuda"), pad)
    dw_o, dw_full = _padded(torch.zeros(N, K, dtype=dw_t, device="cuda"), pad)
    if pad:
        dy, x, W = (_padded(t, pad)[0] for t in (dy, x, W))
        z = None if z is None else _padded(z, pad)[0]
    dx, dW, dbias = ag.ag_linear_bwd(dy, x, W, act=act, preact=z, need_db=db, dx=dx_o, dW=dw_o)
    _ok(ag)
    dyd, xd, Wd = dy.double(), x.double(), W.double()
    want, A = dyd @ Wd, dyd.abs() @ Wd.abs()
    tol = (N + 8) * 2.0 ** -23 * A
    if z is not None:
        slope = ref.act_slope(z.double(), act)
        tol = tol * 1.13 + want.abs() * 2.0 ** -20 * (1 + z.double().abs())
        want = want * slope
    _close("dx", dx, want, tol * (1 + torch.finfo(dx_t).eps) + _half_step(dx_t, want))
    want, A = dyd.T @ xd, dyd.abs().T @ xd.abs()
    _close("dW", dW, want, (M + 8) * 2.0 ** -23 * A * (1 + torch.finfo(dw_t).eps)
           + _half_step(dw_t, want))
    if db:
        _close("db", dbias, dyd.sum(0), (M + 8) * 2.0 ** -24 * dyd.abs().sum(0)
               + _half_step(F32, dyd.sum(0)))
    else:
        assert dbias is None
    if pad:
        assert bool((dx_full[:, K:] == 7.0).all()) and bool((dw_full[:, K:] == 7.0).all())


@pytest.mark.parametrize("M,N,K", SIZES + [(8192, 136, 72)])
def test_linear_bwd_sizes(ag, M, N, K):
    _linear_bwd_case(ag, M, N, K)


@pytest.mark.parametrize("T,dx_t,dw_t", [(BF16, BF16, BF16), (BF16, F32, F32), (F16, F16, F32),
                                         (F16, F32, F16)])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_linear_bwd_types_and_activations(ag, T, dx_t, dw_t, act):
    _linear_bwd_case(ag, 150, 200, 264, T=T, dx_t=dx_t, dw_t=dw_t, act=act)


@pytest.mark.parametrize("pad", [1, 4, 8])
@pytest.mark.parametrize("M,N,K", [(1, 40, 72), (130, 136, 72), (300, 61, 37)])
def test_linear_bwd_rows_apart(ag, M, N, K, pad):
    _linear_bwd_case(ag, M, N, K, pad=pad, act="gelu")


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("M,N,K", [(9, 40, 72), (257, 264, 136), (300, 61, 37), (1000, 1504, 600),
                                   (2048, 64, 40), (5000, 136, 128), (4096, 1024, 1024)])
def test_linear_bwd_of_one_gradient(ag, M, N, K, act):
    """Each gradient by itself is a launch of its own, with its own plan."""
    g = _gen(M + N + K)
    dy, x = _randn(g, M, N, dtype=BF16), _randn(g, M, K, dtype=BF16)
    W = _randn(g, N, K, dtype=BF16, scale=1 / math.sqrt(N))
    z = _randn(g, M, K, dtype=BF16) if act != "none" else None
    dx, none, _ = ag.ag_linear_bwd(dy, x, W, act=act, preact=z, need_dW=False, need_db=False)
    none2, dW, _ = ag.ag_linear_bwd(dy, x, W, act=act, preact=z, need_dx=False, need_db=False)
    _ok(ag)
    assert none is None and none2 is None
    dyd, xd, Wd = dy.double(), x.double(), W.double()
    want, tol = dyd @ Wd, (N + 8) * 2.0 ** -23 * (dyd.abs() @ Wd.abs())
    if z is not None:
        tol = tol * 1.13 + want.abs() * 2.0 ** -20 * (1 + z.double().abs())
        want = want * ref.act_slope(z.double(), act)
    _close("dx", dx, want, tol * (1 + 2.0 ** -7) + _half_step(BF16, want))
    want = dyd.T @ xd
    _close("dW", dW, want, (M + 8) * 2.0 ** -23 * (dyd.abs().T @ xd.abs()) * (1 + 2.0 ** -22)
           + _half_step(F32, want))


@pytest.mark.parametrize("M,N,K,act", [(8192, 1152, 1024, "none"), (4096, 1024, 4096, "gelu"),
                                       (19000, 256, 256, "silu"), (40000, 128, 128, "none"),
                                       (9000, 301, 701, "gelu"), (3000, 1500, 999, "none"),
                                       (1000, 3008, 600, "relu"), (300, 200, 5000, "gelu_tanh")])
def test_linear_bwd_of_many_tiles(ag, M, N, K, act):
    """More tiles of either gradient than clusters, in uneven rounds."""
    _linear_bwd_case(ag, M, N, K, act=act)


def test_linear_bwd_only_what_is_needed(ag):
    g = _gen(3)
    dy, x, W = (_randn(g, *s, dtype=BF16) for s in ((70, 48), (70, 96), (48, 96)))
    every = ag.ag_linear_bwd(dy, x, W)
    for need in ((True, False, False), (False, True, False), (False, False, True)):
        got = ag.ag_linear_bwd(dy, x, W, need_dx=need[0], need_dW=need[1], need_db=need[2])
        for wanted, a, b in zip(need, got, every):
            assert (a is not None) == wanted and (a is None or torch.equal(a, b))


def test_linear_gradients_by_differences(ag):
    """The gradients against central differences of the forward kernel, along
    a random direction: loss = sum(y c) with y = x W^T + b in fp32.  The map is
    linear, so a difference of any step is exact up to the rounding of the
    perturbed 16-bit inputs, which a step of a power of two avoids."""
    M, N, K = 40, 24, 56
    g = _gen(1)
    x = (_randn(g, M, K) * 8).round().div(8).to(BF16)  # few bits, so that x +- d is exact
    W = (_randn(g, N, K) * 8).round().div(8).to(BF16)
    d = _randn(g, M, K).sign() * 0.5
    c = _randn(g, M, N, dtype=BF16)
    loss = lambda t: (ag.ag_linear_fwd(t.to(BF16), W, out_dtype=F32).double() * c.double()).sum()  # noqa: E731
    dx, dW, db = ag.ag_linear_bwd(c, x, W, dx_dtype=F32)
    diff = (loss(x.float() + d) - loss(x.float() - d)) / 2
    along = (dx.double() * d.double()).sum()
    size = (dx.double().abs() * 0.5).sum()
    assert abs(float(diff - along)) <= float(size) * 2.0 ** -12
    db_diff = (ag.ag_linear_fwd(x, W, bias=torch.ones(N, device="cuda"), out_dtype=F32).double()
               - ag.ag_linear_fwd(x, W, out_dtype=F32).double()) * c.double()
    assert abs(float(db_diff.sum() - db.double().sum())) <= float(c.double().abs().sum()) * 2.0 ** -12


# ---------------------------------------------------------------------------
# Norm and rotation of queries and keys
def _qk_inputs(B, L, Hq, Hk, D, R, T, norm, positions, seed, layout="fused"):
    g = _gen(seed)
    if layout == "fused":
        f = _randn(g, B, L, (Hq + Hk) * D, scale=1.5).add(0.2).to(T)
        q, k = f[..., :Hq * D].view(B, L, Hq, D), f[..., Hq * D:].view(B, L, Hk, D)
    elif layout == "heads first":
        q = _randn(g, B, Hq, L, D, dtype=T).transpose(1, 2)
        k = _randn(g, B, Hk, L, D, dtype=T).transpose(1, 2)
    elif layout == "odd rows":
        q = _randn(g, B, L, Hq, D + 3, dtype=T)[..., 1:D + 1]
        k = _randn(g, B, L, Hk, D + 5, dtype=T)[..., 2:D + 2]
    else:  # one row for every batch item
        q = _randn(g, 1, L, Hq, D, dtype=T).expand(B, L, Hq, D)
        k = _randn(g, B, 1, Hk, D, dtype=T).expand(B, L, Hk, D)
    p = {n: None for n in ("qw", "kw", "qb", "kb")}
    if norm != "none":
        p["qw"], p["kw"] = 1 + 0.3 * _randn(g, D), 1 + 0.3 * _randn(g, D)
    if norm == "layer":
        p["qb"], p["kb"] = 0.2 * _randn(g, D), 0.2 * _randn(g, D)
    freq = (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).cuda() if R else None
    pos = None
    if positions == "far":
        pos = torch.randint(-(1 << 30), 1 << 40, (B, L), generator=g).cuda()
    elif positions == "shared":
        pos = torch.randint(0, 1 << 20, (L,), generator=g).cuda()
    return q, k, p, freq, pos


def _where(pos, B, L):
    if pos is None:
        return torch.arange(L, device="cuda").expand(B, L)
    return pos.expand(B, L)


def _row_scale(x, w, b, norm, eps):
    """What 2^-17 counts against: the row's largest value (see the top)."""
    n = ref.norm(x, norm, eps)
    s = n.abs().amax(-1, keepdim=True)
    if norm == "layer":
        mean = x.mean(-1, keepdim=True)
        s = s + x.abs().mean(-1, keepdim=True) / torch.sqrt((x - mean).square().mean(-1, keepdim=True) + eps)
    if w is not None:
        s = s * w.abs().max()
    if b is not None:
        s = s + b.abs().max()
    return s


def _d(t):
    return None if t is None else t.double()


def _qk_case(ag, B, L, Hq, Hk, D, R, T=BF16, out=BF16, norm="rms", rope="halves", positions=None,
             layout="fused", eps=1e-6, seed=0, grad=F32):
    q, k, p, freq, pos = _qk_inputs(B, L, Hq, Hk, D, R, T, norm, positions, seed + D + L, layout)
    kw = dict(q_weight=p["qw"], k_weight=p["kw"], q_bias=p["qb"], k_bias=p["kb"], norm=norm,
              eps=eps, inv_freq=freq, rope=rope, positions=pos)
    got = ag.ag_qk_norm_rope_fwd(q, k, out_dtype=out, **kw)
    _ok(ag)
    where = _where(pos, B, L)
    for name, o, x, w, b in (("q", got[0], q, p["qw"], p["qb"]), ("k", got[1], k, p["kw"], p["kb"])):
        want = ref.qk(x.double(), _d(w), _d(b), norm, eps, freq, rope, where)
        scale = _row_scale(x.double(), _d(w), _d(b), norm, eps).transpose(1, 2)
        _close(name + "_out", o, want, 2.0 ** -17 * scale * (1 + torch.finfo(out).eps)
               + _half_step(out, want))
    g = _gen(seed + 77)
    gq, gk = _randn(g, B, Hq, L, D, dtype=grad), _randn(g, B, Hk, L, D, dtype=grad)
    dq, dk, dqw, dkw, dqb, dkb = ag.ag_qk_norm_rope_bwd(gq, gk, q, k, **kw)
    _ok(ag)
    for name, dx, dw, db, go, x, w, b in (("dq", dq, dqw, dqb, gq, q, p["qw"], p["qb"]),
                                          ("dk", dk, dkw, dkb, gk, k, p["kw"], p["kb"])):
        xd, gd = x.double(), go.double()
        want, want_w, want_b = ref.qk_grads(gd, xd, _d(w), _d(b), norm, eps, freq, rope, where)
        n = ref.norm(xd, norm, eps)
        c = xd - xd.mean(-1, keepdim=True) if norm == "layer" else xd
        r = 1 / torch.sqrt(c.square().mean(-1, keepdim=True) + eps) if norm != "none" else 1.0
        gl = gd.transpose(1, 2)
        top = 2 * gl.abs().amax(-1, keepdim=True) * (1.0 if w is None else w.double().abs().max())
        nscale = _row_scale(xd, None, None, norm, eps) if norm != "none" else 1.0
        # dx = r (d - n mean(d n) - mean d): terms of sizes d, n^2 d and d.
        scale = r * top * (2 + nscale * n.abs().amax(-1, keepdim=True)) if norm != "none" else top
        _close(name, dx, want, 2.0 ** -17 * scale * (1 + torch.finfo(T).eps) + _half_step(T, want))
        terms = B * L * x.shape[2]
        turned = ref.rotate(gl, where, freq, rope, -1.0)
        if dw is not None:
            big = (turned.abs() * n.abs()).sum((0, 1, 2)) * terms * 2.0 ** -24
            own = (top * _row_scale(xd, None, None, norm, eps)).sum((0, 1, 2)).max() * 2.0 ** -17
            _close(name + "_weight", dw, want_w, big + own)
        else:
            assert w is None
        if db is not None:
            big = turned.abs().sum((0, 1, 2)) * terms * 2.0 ** -24
            _close(name + "_bias", db, want_b, big + top.sum((0, 1, 2)).max() * 2.0 ** -17)
        else:
            assert b is None


@pytest.mark.parametrize("norm", ["none", "rms", "layer"])
@pytest.mark.parametrize("rope", ["halves", "interleaved"])
@pytest.mark.parametrize("B,L,Hq,Hk,D,R", [
    (1, 1, 8, 1, 128, 128), (2, 33, 8, 1, 128, 128), (1, 5, 8, 1, 128, 64), (3, 17, 3, 2, 64, 32),
    (1, 9, 2, 1, 256, 256), (2, 7, 4, 4, 192, 192), (1, 6, 1, 1, 32, 0), (2, 3, 5, 1, 100, 50),
    (1, 4, 2, 1, 37, 12), (1, 3, 1, 1, 2, 2), (1, 2, 1, 1, 1, 0), (1, 5, 2, 1, 1024, 1024),
    (2, 3, 1, 2, 520, 100), (1, 7, 2, 1, 128, 40), (1, 7, 2, 1, 128, 6), (5, 41, 8, 1, 16, 16)])
def test_qk_sizes(ag, norm, rope, B, L, Hq, Hk, D, R):
    _qk_case(ag, B, L, Hq, Hk, D, R, norm=norm, rope=rope)


@pytest.mark.parametrize("T", [BF16, F16, F32])
@pytest.mark.parametrize("out", [BF16, F16, F32])
@pytest.mark.parametrize("D,R", [(128, 128), (96, 40)])
def test_qk_types(ag, T, out, D, R):
    _qk_case(ag, 2, 19, 8, 1, D, R, T=T, out=out, grad=out, norm="layer", positions="shared")


@pytest.mark.parametrize("layout", ["fused", "heads first", "odd rows", "broadcast"])
@pytest.mark.parametrize("T", [BF16, F32])
def test_qk_layouts(ag, layout, T):
    _qk_case(ag, 2, 21, 4, 2, 128, 128, T=T, layout=layout, positions="far")
    _qk_case(ag, 2, 21, 4, 2, 24, 8, T=T, layout=layout, norm="layer", rope="interleaved")


@pytest.mark.parametrize("positions", ["far", "shared", None])
@pytest.mark.parametrize("rope", ["halves", "interleaved"])
def test_qk_positions(ag, positions, rope):
    _qk_case(ag, 3, 50, 8, 1, 128, 128, positions=positions, rope=rope, out=F32, T=F32)


def test_qk_long(ag):
    _qk_case(ag, 2, 4111, 8, 1, 128, 128, norm="layer")
    _qk_case(ag, 1, 5003, 1, 1, 40, 12, norm="rms", rope="interleaved")


@pytest.mark.parametrize("Hq,Hk,D,R", [(70, 3, 128, 64), (1, 9, 64, 64), (0, 5, 128, 128),
                                       (33, 0, 100, 10), (4, 4, 8, 8), (5, 2, 16, 0)])
def test_qk_many_heads(ag, Hq, Hk, D, R):
    g = _gen(Hq + D)
    B, L = 2, 19
    q = _randn(g, B, L, Hq, D, dtype=BF16) if Hq else None
    k = _randn(g, B, L, Hk, D, dtype=BF16) if Hk else None
    w = 1 + 0.3 * _randn(g, D)
    freq = ag.ag_rope_frequencies(R) if R else None
    pos = torch.randint(0, 1 << 20, (B, L), generator=g).cuda()
    sides = [t for t in (q, k) if t is not None]
    grads = [_randn(g, B, t.shape[2], L, D) if t is not None else None for t in (q, k)]
    kw = dict(q_weight=None if q is None else w, k_weight=None if k is None else w, norm="rms",
              inv_freq=freq, positions=pos)
    outs = [o for o in ag.ag_qk_norm_rope_fwd(q, k, out_dtype=F32, **kw) if o is not None]
    got = ag.ag_qk_norm_rope_bwd(*grads, q, k, **kw)
    _ok(ag)
    for x, o, go, dx, dw in zip(sides, outs, [t for t in grads if t is not None],
                                [t for t in got[:2] if t is not None],
                                [t for t in got[2:4] if t is not None]):
        want = ref.qk(x.double(), w.double(), None, "rms", 1e-6, freq, "halves", pos)
        scale = _row_scale(x.double(), w.double(), None, "rms", 1e-6).transpose(1, 2)
        _close("out", o, want, 2.0 ** -17 * scale + _half_step(F32, want))
        wdx, wdw, _ = ref.qk_grads(go.double(), x.double(), w.double(), None, "rms", 1e-6, freq,
                                   "halves", pos)
        n = ref.norm(x.double(), "rms", 1e-6)
        r = 1 / torch.sqrt(x.double().square().mean(-1, keepdim=True) + 1e-6)
        top = 2 * go.double().transpose(1, 2).abs().amax(-1, keepdim=True) * w.double().abs().max()
        big = n.abs().amax(-1, keepdim=True)
        _close("dx", dx, wdx, 2.0 ** -17 * r * top * (2 + big * big) * (1 + 2.0 ** -7)
               + _half_step(BF16, wdx))
        terms = B * L * x.shape[2]
        turned = ref.rotate(go.double().transpose(1, 2), pos, freq, "halves", -1.0)
        _close("dw", dw, wdw, (turned.abs() * n.abs()).sum((0, 1, 2)) * terms * 2.0 ** -24
               + (top * big).sum((0, 1, 2)).max() * 2.0 ** -17)


def test_qk_zero_rows_and_eps(ag):
    """A row of zeros keeps its bias (eps > 0); with eps == 0 it has no norm."""
    q = torch.zeros(1, 3, 2, 128, dtype=BF16, device="cuda")
    q[:, 1:] = 1.5
    b = torch.linspace(-1, 1, 128, device="cuda")
    o, _ = ag.ag_qk_norm_rope_fwd(q, None, q_bias=b, norm="rms", eps=1e-6, out_dtype=F32)
    torch.cuda.synchronize()
    assert torch.equal(o[0, :, 0], b.expand(2, 128))
    o, _ = ag.ag_qk_norm_rope_fwd(q, None, norm="rms", eps=0.0, out_dtype=F32)
    torch.cuda.synchronize()
    assert bool(torch.isnan(o[0, :, 0]).all()) and bool((o[0, :, 1:] == 1.0).all())


def test_qk_non_finite_rows_stay_alone(ag):
    for D in (128, 40):
        q = _randn(_gen(2), 2, 9, 4, D, dtype=BF16)
        q[1, 3, 2, 5] = math.inf
        q[0, 8, 0, 0] = math.nan
        freq = ag.ag_rope_frequencies(D)
        o, _ = ag.ag_qk_norm_rope_fwd(q, None, inv_freq=freq)
        torch.cuda.synchronize()
        bad = ~torch.isfinite(o).all(-1)
        want = torch.zeros_like(bad)
        want[1, 2, 3] = want[0, 0, 8] = True
        assert torch.equal(bad, want)


def test_qk_one_side_and_flat_keys(ag):
    g = _gen(8)
    q, k = _randn(g, 2, 11, 8, 128, dtype=BF16), _randn(g, 2, 11, 128, dtype=BF16)
    freq = ag.ag_rope_frequencies(128)
    both = ag.ag_qk_norm_rope_fwd(q, k, inv_freq=freq)
    assert both[0].shape == (2, 8, 11, 128) and both[1].shape == (2, 11, 128)
    assert torch.equal(ag.ag_qk_norm_rope_fwd(q, None, inv_freq=freq)[0], both[0])
    assert torch.equal(ag.ag_qk_norm_rope_fwd(None, k, inv_freq=freq)[1], both[1])
    w = torch.ones(128, device="cuda")
    gq, gk = _randn(g, 2, 8, 11, 128), _randn(g, 2, 11, 128)
    all_ = ag.ag_qk_norm_rope_bwd(gq, gk, q, k, q_weight=w, k_weight=w, inv_freq=freq)
    only = ag.ag_qk_norm_rope_bwd(None, gk, None, k, k_weight=w, inv_freq=freq)
    torch.cuda.synchronize()
    assert all_[1].shape == k.shape and torch.equal(all_[1], only[1])
    assert only[0] is None and only[2] is None and torch.allclose(all_[3], only[3], rtol=1e-5, atol=1e-4)


def test_qk_bwd_into_a_fused_gradient(ag):
    """dq and dk as slices of one buffer's rows; the columns beside them stay."""
    g = _gen(4)
    B, L, H, D = 2, 13, 8, 128
    f = _randn(g, B, L, (H + 1) * D, dtype=BF16)
    q, k = f[..., :H * D].view(B, L, H, D), f[..., H * D:]
    gq, gk = _randn(g, B, H, L, D), _randn(g, B, L, D)
    freq = ag.ag_rope_frequencies(D)
    apart = ag.ag_qk_norm_rope_bwd(gq, gk, q, k, inv_freq=freq)
    buf = torch.full((B, L, (H + 1) * D + 64), 7.0, dtype=BF16, device="cuda")
    ag.ag_qk_norm_rope_bwd(gq, gk, q, k, inv_freq=freq, dq=buf[..., :H * D].view(B, L, H, D),
                           dk=buf[..., H * D:(H + 1) * D])
    torch.cuda.synchronize()
    assert torch.equal(buf[..., :H * D], apart[0].flatten(2))
    assert torch.equal(buf[..., H * D:(H + 1) * D], apart[1])
    assert bool((buf[..., (H + 1) * D:] == 7.0).all())
    with pytest.raises(ag.AgError, match="ALIAS"):
        ag.ag_qk_norm_rope_bwd(gq, gk, q, k, dq=buf[..., :H * D].view(B, L, H, D),
                               dk=buf[..., H * D - 8:(H + 1) * D - 8])
    with pytest.raises(ag.AgError, match="SHAPE"):
        ag.ag_qk_norm_rope_bwd(gq, gk, q, k, dk=buf[:1, :, :D].expand(B, L, D))


def test_qk_empty(ag):
    q = torch.zeros(2, 0, 8, 128, dtype=BF16, device="cuda")
    w = torch.ones(128, device="cuda")
    o, _ = ag.ag_qk_norm_rope_fwd(q, None, q_weight=w)
    assert o.shape == (2, 8, 0, 128)
    out = ag.ag_qk_norm_rope_bwd(torch.zeros(2, 8, 0, 128, device="cuda"), None, q, None,
                                 q_weight=w)
    torch.cuda.synchronize()
    assert out[0].shape == q.shape and not bool(out[2].any())


@pytest.mark.parametrize("norm", ["none", "rms", "layer"])
def test_qk_gradients_by_differences(ag, norm):
    """Central differences of the fp32 forward kernel along a random direction
    d with step h = 2^-6.  The error of a central difference is at most
    h^2 / 6 of the third derivative, below (3 |d| / |x|)^3 for these rows, about
    1e-3 of the gradient's size here; rounding adds 2^-20 / h = 6e-5."""
    B, L, H, D = 1, 6, 3, 128
    q, _, p, freq, pos = _qk_inputs(B, L, H, 1, D, D, F32, norm, "shared", 3)
    kw = dict(q_weight=p["qw"], q_bias=p["qb"], norm=norm, inv_freq=freq, positions=pos)
    g = _gen(6)
    c, d, h = _randn(g, B, H, L, D), _randn(g, B, L, H, D), 2.0 ** -6
    loss = lambda t: (ag.ag_qk_norm_rope_fwd(t, None, out_dtype=F32, **kw)[0].double() * c.double()).sum()  # noqa: E731
    dq = ag.ag_qk_norm_rope_bwd(c, None, q.contiguous(), None, **kw)[0]
    diff = float((loss(q + h * d) - loss(q - h * d)) / (2 * h))
    along = float((dq.double() * d.double()).sum())
    size = float((dq.double() * d.double()).square().sum().sqrt())
    assert abs(diff - along) <= 1e-2 * size


# ---------------------------------------------------------------------------
# Gradient clipping
def _clip_check(ag, grads, max_norm, eps=1e-6):
    flat = torch.cat([g.double().flatten() for g in grads])
    norm = float(flat.square().sum().sqrt())
    before = [g.clone() for g in grads]
    got = ag.ag_grad_clip(grads, max_norm, eps=eps)
    _ok(ag)
    # The sum is in 64 bits; the result is rounded once.
    assert abs(float(got) - norm) <= norm * (2.0 ** -24 + 1e-12)
    c = min(1.0, max_norm / (norm + eps)) if norm + eps > 0 else 1.0
    for g, b in zip(grads, before):
        if c == 1.0:
            assert torch.equal(g, b)
        else:  # c rounded to fp32, the product in fp32, then the type's rounding
            want = b.double() * c
            _close("gradient", g, want, want.abs() * 2.0 ** -22 + _half_step(g.dtype, want) * 1.01)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e9, math.inf])
def test_clip_types(ag, dtype, max_norm):
    g = _gen(1)
    _clip_check(ag, [_randn(g, *s, dtype=dtype) for s in ((1,), (7,), (130, 33), (40000,), (3, 5, 8),
                                                          (0, 4), (16384,), (16385,))], max_norm)


def test_clip_mixed_types_offsets_and_orders(ag):
    g = _gen(2)
    buf = _randn(g, 100000)
    half = _randn(g, 50001, dtype=BF16)
    grads = [buf[1:1002], buf[1002:1003], buf[1003:40000], half[3:17], half[17:30001],
             _randn(g, 60, 50).t(), _randn(g, 2, 3, 4, dtype=F16).permute(2, 0, 1)]
    rest = buf[40000:].clone()
    _clip_check(ag, grads, 1.0)
    assert torch.equal(buf[40000:], rest), "wrote past the last gradient"


@pytest.mark.parametrize("n", [1, 511, 512, 513, 1500])
def test_clip_many_tensors(ag, n):
    g = _gen(n)
    flat = _randn(g, n, 65)
    _clip_check(ag, [flat[i, :1 + i % 64] for i in range(n)], 0.25)
    _clip_check(ag, [flat[i, :1 + i % 64] for i in range(n)], math.inf)


@pytest.mark.parametrize("full", [31, 32, 33, 511, 512, 513])
def test_clip_many_empty_tensors(ag, full):
    """Empty tensors take no place among those of a launch, wherever they are."""
    flat = _randn(_gen(full), full, 3)
    empty = torch.zeros(0, device="cuda")
    some = list(flat)
    _clip_check(ag, some + [empty] * 600, 0.25)
    _clip_check(ag, [empty] * 600 + some, 0.125)
    _clip_check(ag, [t for s in some for t in (s, empty)], 0.0625)


def test_clip_large(ag):
    g = torch.Generator(device="cuda").manual_seed(3)
    grads = [torch.randn(n, generator=g, device="cuda") for n in (30_000_001, 5, 12_345_678)]
    _clip_check(ag, grads, 3.0)


def test_clip_range_of_magnitudes(ag):
    """Squares that overflow or vanish in 32 bits."""
    _clip_check(ag, [torch.full((1000,), 1e30, device="cuda")], 1.0)
    _clip_check(ag, [torch.full((1000,), 1e-30, device="cuda")], 1e-31, eps=0.0)


def test_clip_non_finite(ag):
    a, b = torch.ones(100, device="cuda"), torch.ones(40, dtype=BF16, device="cuda")
    a[3] = math.inf
    n = ag.ag_grad_clip([a, b], 1.0)
    torch.cuda.synchronize()
    assert float(n) == math.inf and bool(torch.isnan(a[3])) and not bool(b.any())
    assert float(a[torch.arange(100, device="cuda") != 3].abs().max()) == 0.0
    a, b = torch.ones(100, device="cuda"), torch.ones(40, dtype=BF16, device="cuda")
    a[3] = math.nan
    n = ag.ag_grad_clip([a, b], 1.0)
    torch.cuda.synchronize()
    assert math.isnan(float(n)) and bool(torch.isnan(a).all()) and bool(torch.isnan(b).all())
    a = torch.full((4,), math.inf, device="cuda")
    ag.ag_grad_clip([a], math.inf)
    torch.cuda.synchronize()
    assert bool(torch.isinf(a).all())


def test_clip_of_zeros_and_nothing(ag):
    z = torch.zeros(50, device="cuda")
    n = torch.full((1,), 5.0, device="cuda")
    assert ag.ag_grad_clip([z, None], 1.0, norm=n) is n
    torch.cuda.synchronize()
    assert float(n) == 0.0 and not bool(z.any())
    assert float(ag.ag_grad_clip([z], 0.0, eps=0.0)) == 0.0 and not bool(z.any())
    e = torch.zeros(0, device="cuda")
    assert float(ag.ag_grad_clip([e], 1.0)) == 0.0


def test_clip_of_no_tensor_through_the_c_abi(ag):
    import ctypes
    n, size = torch.full((1,), 5.0, device="cuda"), ctypes.c_int64(0)
    assert ag.lib.ag_grad_clip_workspace(0, ctypes.byref(size)) == 0
    ws = torch.zeros(size.value, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert ag.lib.ag_grad_clip(None, None, None, 0, 1.0, 0.0, n.data_ptr(), ws.data_ptr(),
                               size.value, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert float(n) == 0.0


def test_clip_refuses_overlaps(ag):
    a = torch.ones(100, device="cuda")
    for grads in ([a, a], [a[:60], a[59:]], [a[50:], a[:51]]):
        with pytest.raises(ag.AgError, match="ALIAS"):
            ag.ag_grad_clip(grads, 0.1)
    with pytest.raises(ag.AgError, match="ALIAS"):
        ag.ag_grad_clip([a[1:]], 0.1, norm=a[5])
    with pytest.raises(ValueError, match="dense"):
        ag.ag_grad_clip([a.view(10, 10)[:, :5]], 0.1)
    torch.cuda.synchronize()
    assert bool((a == 1).all())


def test_clip_is_reproducible(ag):
    g = _gen(4)
    base = [_randn(g, 100_003), _randn(g, 77), _randn(g, 999_999)]
    first = None
    for _ in range(3):
        grads = [b.clone() for b in base]
        n = ag.ag_grad_clip(grads, 1.0)
        if first is None:
            first = (n, grads)
        assert torch.equal(n, first[0]) and all(torch.equal(x, y) for x, y in zip(grads, first[1]))


# ---------------------------------------------------------------------------
# Streams, graphs, and the operators together
def _block(ag, s):
    """One attention block's forward and backward and the clipping of its
    parameters' gradients, as a training step calls them."""
    B, L, H, D = s["B"], s["L"], 8, 128
    E = H * D
    x = s["x"]
    qk = ag.ag_linear_fwd(x, s["Wqk"], bias=s["bqk"])
    v = ag.ag_linear_fwd(x, s["Wv"])
    fused = qk.view(B, L, E + D)
    kw = dict(q_weight=s["qw"], k_weight=s["kw"], norm="rms", inv_freq=s["freq"],
              positions=s["pos"])
    qh, kh = fused[..., :E].view(B, L, H, D), fused[..., E:]
    q, k = ag.ag_qk_norm_rope_fwd(qh, kh, **kw)
    vh = v.view(B, L, D)
    o, lse = ag.ag_attn_fwd(q, k, vh, s["bias"], cap=5.0)
    a = o.transpose(1, 2).reshape(B * L, E).to(BF16)
    h = ag.ag_linear_fwd(a, s["Wo"], residual=x)
    u, z = ag.ag_linear_fwd(h, s["W1"], bias=s["b1"], act="gelu", preact=True)
    y = ag.ag_linear_fwd(u, s["W2"], bias=s["b2"], residual=h)
    # Backward of sum(y * dy).
    dy = s["dy"]
    dz, dW2, db2 = ag.ag_linear_bwd(dy, u, s["W2"], act="gelu", preact=z)
    dh, dW1, db1 = ag.ag_linear_bwd(dz, h, s["W1"])
    dh = dh + dy
    da, dWo, _ = ag.ag_linear_bwd(dh, a, s["Wo"], dx_dtype=F32, need_db=False)
    do = da.view(B, L, H, D).transpose(1, 2).contiguous()
    dq, dk, dv, dbias, _ = ag.ag_attn_bwd(q, k, vh, s["bias"], lse, do, cap=5.0)
    dqk = torch.empty_like(fused)
    _, _, dqw, dkw, _, _ = ag.ag_qk_norm_rope_bwd(dq, dk, qh, kh, dq=dqk[..., :E].view(B, L, H, D),
                                                  dk=dqk[..., E:], **kw)
    dx1, dWqk, dbqk = ag.ag_linear_bwd(dqk.view(B * L, E + D), x, s["Wqk"])
    dx2, dWv, _ = ag.ag_linear_bwd(dv.to(BF16).view(B * L, D), x, s["Wv"], need_db=False)
    dx = dh.float() + dx1.float() + dx2.float()
    grads = [dWqk, dbqk, dWv, dqw, dkw, dbias, dWo, dW1, db1, dW2, db2]
    raw = [g.clone() for g in grads]
    n = ag.ag_grad_clip(grads, 0.5)
    return y, dx, raw, n, grads


def _block_inputs(B, L, seed):
    g = _gen(seed)
    E, D, F = 1024, 128, 512
    s = dict(B=B, L=L, x=_randn(g, B * L, E, dtype=BF16))
    for name, shape in (("Wqk", (E + D, E)), ("Wv", (D, E)), ("Wo", (E, E)), ("W1", (F, E)),
                        ("W2", (E, F))):
        s[name] = _randn(g, *shape, dtype=BF16, scale=shape[1] ** -0.5)
    for name, n in (("bqk", E + D), ("b1", F), ("b2", E)):
        s[name] = 0.1 * _randn(g, n)
    s["qw"], s["kw"] = 1 + 0.2 * _randn(g, D), 1 + 0.2 * _randn(g, D)
    P = -(-L // 16)
    s["bias"] = _randn(g, 8, P, P)
    s["freq"] = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).cuda()
    s["pos"] = torch.randint(0, 1 << 20, (B, L), generator=g).sort(-1).values.cuda()
    s["dy"] = _randn(g, B * L, E, dtype=BF16)
    return s


def _block_reference(s):
    """The same block in 64 bits throughout, gradients by autograd."""
    B, L, H, D = s["B"], s["L"], 8, 128
    E = H * D
    names = ["x", "Wqk", "bqk", "Wv", "qw", "kw", "bias", "Wo", "W1", "b1", "W2", "b2"]
    p = {n: s[n].double().clone().requires_grad_(True) for n in names}
    qk = (p["x"] @ p["Wqk"].T + p["bqk"]).view(B, L, E + D)
    q = ref.qk(qk[..., :E].reshape(B, L, H, D), p["qw"], None, "rms", 1e-6, s["freq"], "halves", s["pos"])
    k = ref.qk(qk[..., E:].reshape(B, L, 1, D), p["kw"], None, "rms", 1e-6, s["freq"], "halves", s["pos"])
    v = (p["x"] @ p["Wv"].T).view(B, 1, L, D)
    wide = p["bias"].repeat_interleave(16, 1).repeat_interleave(16, 2)[:, :L, :L]
    t = 5 * torch.tanh((q @ k.transpose(-1, -2) / math.sqrt(D) + wide) / 5)
    o = torch.softmax(t, -1) @ v
    h = o.transpose(1, 2).reshape(B * L, E) @ p["Wo"].T + p["x"]
    y = ref.act(h @ p["W1"].T + p["b1"], "gelu") @ p["W2"].T + p["b2"] + h
    (y * s["dy"].double()).sum().backward()
    return y.detach(), p["x"].grad, [p[n].grad for n in names[1:]]


@pytest.mark.parametrize("B,L", [(2, 40), (1, 150)])
def test_block_forward_backward_and_clip(ag, B, L):
    """The operators in a row.  Every step rounds its 16-bit outputs by at most
    2^-9 of a value in the mean square 2^-9 / sqrt(3); some ten roundings lie
    between an input and a gradient, each amplified by at most a few, so the
    2-norms agree to 3 percent."""
    s = _block_inputs(B, L, seed=L)
    y, dx, raw, n, clipped = _block(ag, s)
    _ok(ag)
    wy, wdx, wgrads = _block_reference(s)
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert rel(y, wy) <= 0.03 and rel(dx, wdx) <= 0.03
    for i, (a, b) in enumerate(zip(raw, wgrads)):
        assert rel(a, b) <= 0.03, f"gradient {i}: {rel(a, b):.3f}"
    total = math.sqrt(sum(float(g.double().square().sum()) for g in raw))
    assert abs(float(n) - total) <= total * 2.0 ** -23
    c = min(1.0, 0.5 / (total + 1e-6))
    for g, r in zip(clipped, raw):
        _close("clipped", g, r.double() * c, r.double().abs() * c * 2.0 ** -21 + 1e-30)


def test_block_on_other_streams_and_in_graphs(ag):
    """Eager, on a side stream, and two captured graphs that replay at the same
    time: the same bits (each call's workspace is its own)."""
    a, b = _block_inputs(1, 48, 1), _block_inputs(1, 48, 2)
    flat = lambda r: [r[0], r[1], *r[2], r[3], *r[4]]  # noqa: E731
    want = [[t.clone() for t in flat(_block(ag, s))] for s in (a, b)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = flat(_block(ag, a))
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want[0]))
    graphs, outs = [], []
    for s in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(flat(_block(ag, s)))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for out in outs:
            for t in out:
                t.zero_()
        torch.cuda.synchronize()
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert all(torch.equal(x, y) for x, y in zip(out, w))
    assert ag.ag_device_error(0) == 0


def test_calls_of_several_threads(ag):
    """Calls with little and with much shared memory, few and many tensors and
    several products, made by four threads at once on streams of their own."""
    import threading
    g = _gen(11)
    cases = []
    for D in (1000, 999, 331, 77):
        q, k = _randn(g, 2, 5, 2, D), _randn(g, 2, 5, D)
        w = _randn(g, D)
        x, W = _randn(g, 40 + D, 72, dtype=BF16), _randn(g, D, 72, dtype=BF16)
        cases.append((q, k, w, x, W))

    def once(q, k, w, x, W):
        kw = dict(q_weight=w, k_weight=w, norm="layer")
        fwd = ag.ag_qk_norm_rope_fwd(q, k, out_dtype=F32, **kw)
        bwd = ag.ag_qk_norm_rope_bwd(*fwd, q, k, **kw)
        y = ag.ag_linear_fwd(x, W, act="gelu")
        return [*fwd, *(t for t in bwd if t is not None), y, *ag.ag_linear_bwd(y, x, W)]

    want = [once(*c) for c in cases]
    _ok(ag)
    failed = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(40):
                    got = once(*cases[i])
                torch.cuda.current_stream().synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
        except BaseException as e:  # noqa: BLE001  (reported by the test's own thread)
            failed.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    _ok(ag)
    assert not failed, failed


def test_stream_argument(ag):
    """Each entry point on a stream given as an argument, as a Stream and as a
    raw handle: the work follows that stream's earlier work."""
    g = _gen(11)
    x0, W = _randn(g, 300, 256, dtype=BF16), _randn(g, 136, 256, dtype=BF16)
    want = ag.ag_linear_fwd(x0, W)
    torch.cuda.synchronize()
    for raw in (False, True):
        st = torch.cuda.Stream()
        x = torch.zeros_like(x0)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            torch.cuda._sleep(20_000_000)
            x.copy_(x0)
        arg = st.cuda_stream if raw else st
        y = ag.ag_linear_fwd(x, W, stream=arg)
        dx, dW, db = ag.ag_linear_bwd(y, x, W, stream=arg)
        q, _ = ag.ag_qk_norm_rope_fwd(y.view(1, 300, 1, 136), None, stream=arg)
        dq = ag.ag_qk_norm_rope_bwd(q, None, y.view(1, 300, 1, 136), None, stream=arg)[0]
        n = ag.ag_grad_clip([dW], 0.1, stream=arg)
        st.synchronize()
        assert torch.equal(y, want)
        ex = ag.ag_linear_bwd(want, x0, W)
        en = ag.ag_grad_clip([ex[1]], 0.1)
        eq, _ = ag.ag_qk_norm_rope_fwd(want.view(1, 300, 1, 136), None)
        edq = ag.ag_qk_norm_rope_bwd(eq, None, want.view(1, 300, 1, 136), None)[0]
        torch.cuda.synchronize()
        for a, b in ((dx, ex[0]), (dW, ex[1]), (db, ex[2]), (q, eq), (dq, edq), (n, en)):
            assert torch.equal(a, b)


def test_refusals_on_the_gpu(ag):
    x, W = torch.zeros(4, 8, dtype=BF16, device="cuda"), torch.zeros(6, 8, dtype=BF16, device="cuda")
    with pytest.raises(TypeError):
        ag.ag_linear_fwd(x, W.half())
    with pytest.raises(TypeError):
        ag.ag_linear_fwd(x.float(), W.float())
    with pytest.raises(TypeError):
        ag.ag_linear_fwd(x, W, out_dtype=F16)
    with pytest.raises(ValueError, match="dense"):
        ag.ag_linear_fwd(x.t().contiguous().t(), W)
    with pytest.raises(ValueError, match="bias"):
        ag.ag_linear_fwd(x, W, bias=torch.zeros(5, device="cuda"))
    with pytest.raises(ag.AgError, match="SHAPE"):
        ag.ag_linear_fwd(x[:1].expand(4, 8), W)  # rows that share one address
    with pytest.raises(ag.AgError, match="ALIAS"):
        ag.ag_linear_fwd(x, torch.zeros(8, 8, dtype=BF16, device="cuda"), out=x)
    with pytest.raises(ValueError, match="preact"):
        ag.ag_linear_bwd(torch.zeros(4, 6, dtype=BF16, device="cuda"), x, W, act="gelu")
    q = torch.zeros(1, 4, 2, 8, dtype=BF16, device="cuda")
    with pytest.raises(ag.AgError, match="SHAPE"):
        ag.ag_qk_norm_rope_fwd(q, None, inv_freq=torch.zeros(5, dtype=torch.float64, device="cuda"))
    with pytest.raises(TypeError):
        ag.ag_qk_norm_rope_fwd(q, None, inv_freq=torch.zeros(4, device="cuda"))
    with pytest.raises(TypeError):
        ag.ag_qk_norm_rope_fwd(q, None, positions=torch.zeros(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="positions"):
        ag.ag_qk_norm_rope_fwd(q, None, positions=torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ag.AgError, match="VALUE"):
        ag.ag_qk_norm_rope_fwd(q, None, eps=-1.0)
    with pytest.raises(ag.AgError, match="VALUE"):
        ag.ag_grad_clip([torch.zeros(4, device="cuda")], -1.0)
    # A workspace that is too small is refused, not overrun.
    need = torch.zeros(1, dtype=torch.int64)
    import ctypes
    n = ctypes.c_int64(0)
    assert ag.lib.ag_grad_clip_workspace(1, ctypes.byref(n)) == 0 and n.value > 0
    t, norm = torch.ones(4, device="cuda"), torch.zeros(1, device="cuda")
    ws = torch.zeros(n.value, dtype=torch.uint8, device="cuda")
    args = ((ctypes.c_void_p * 1)(t.data_ptr()), (ctypes.c_int64 * 1)(4), (ctypes.c_int * 1)(0), 1,
            1.0, 0.0, norm.data_ptr(), ws.data_ptr())
    assert ag.lib.ag_grad_clip(*args, n.value - 1, None) == 9
    torch.cuda.synchronize()
    assert bool((t == 1).all()) and int(need) == 0


# ---------------------------------------------------------------------------
# Offsets past 32 bits (8 to 26 GB on the device)
@pytest.mark.parametrize("ld", [2 ** 28, 2 ** 28 - 1])
def test_linear_rows_far_apart(ag, ld):
    """Inputs, outputs and gradients in columns of one buffer whose last rows
    start past element 2^32, with rows that TMA can and cannot address."""
    M, N, K = 18, 40, 64
    buf = torch.empty(17 * ld + 512, dtype=BF16, device="cuda")
    x, y, dy, dx = (torch.as_strided(buf, (M, n), (ld, 1), at)
                    for n, at in ((K, 0), (N, 64), (N, 128), (K, 192)))
    g = _gen(ld % 1000)
    x.copy_(_randn(g, M, K, dtype=BF16))
    dy.copy_(_randn(g, M, N, dtype=BF16))
    W = _randn(g, N, K, dtype=BF16, scale=1 / 8)
    ag.ag_linear_fwd(x, W, out=y)
    _, dW, db = ag.ag_linear_bwd(dy, x, W, dx=dx)
    _ok(ag)
    xd, Wd, dyd = x.double(), W.double(), dy.double()
    for name, got, want, mass, n in (("y", y, xd @ Wd.T, xd.abs() @ Wd.abs().T, K),
                                     ("dx", dx, dyd @ Wd, dyd.abs() @ Wd.abs(), N),
                                     ("dW", dW, dyd.T @ xd, dyd.abs().T @ xd.abs(), M),
                                     ("db", db, dyd.sum(0), dyd.abs().sum(0), M)):
        _close(name, got, want, (n + 8) * 2.0 ** -23 * mass * 1.01 + _half_step(got.dtype, want))


@pytest.mark.parametrize("D", [8, 7])
def test_qk_more_elements_than_32_bits(ag, D):
    """2^32 elements of one head, of one row at every position; the rotation
    tells the positions apart."""
    L = 2 ** 32 // D + 5
    g = _gen(D)
    row = _randn(g, D, dtype=BF16)
    q = row.expand(1, L, 1, D)
    freq = ag.ag_rope_frequencies(D // 2 * 2)
    out, _ = ag.ag_qk_norm_rope_fwd(q, None, inv_freq=freq, norm="none")
    _ok(ag)
    n = min(1000, L)
    last = torch.arange(L - n, L, device="cuda")
    for at in (torch.arange(n, device="cuda"), last):
        want = ref.qk(row.double().expand(1, n, 1, D), None, None, "none", 0.0, freq, "halves",
                      at[None])[0, 0]
        mass = row.double().abs().sum()
        _close("q", out[0, 0, at], want, mass * 2.0 ** -19 + _half_step(BF16, want))
    w = torch.ones(D, device="cuda")
    dq, _, _, _, dbias, _ = ag.ag_qk_norm_rope_bwd(out, None, q, None, q_bias=w, inv_freq=freq,
                                                   norm="none")
    _ok(ag)
    want = row.double().expand(n, D)  # turned there and back
    _close("dq", dq[0, last, 0], want, row.double().abs().sum() * (2.0 ** -18 + 2.0 ** -7)
           + _half_step(BF16, want))


def test_clip_more_elements_than_32_bits(ag):
    n = 2 ** 32 + 77
    t = torch.full((n,), 0.5, dtype=BF16, device="cuda")
    norm = ag.ag_grad_clip([t], 1024.0)
    _ok(ag)
    want = 0.5 * math.sqrt(n)
    assert abs(float(norm) - want) <= want * 2.0 ** -23
    scaled = torch.tensor(0.5 * 1024.0 / want).to(BF16).item()
    for part in (t[:1000], t[n // 2:n // 2 + 1000], t[-1000:]):
        assert bool((part == scaled).all())
