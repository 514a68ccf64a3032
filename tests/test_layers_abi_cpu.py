"""The layers' entry points without a GPU: every refusal that include/ag.h
documents comes before anything touches CUDA.  Pointers here are fake device
addresses that are never dereferenced; a call that passes every check ends at
the device (no sm_100 GPU: AG_ERR_UNSUPPORTED, no driver: AG_ERR_CUDA) or, on
a machine with a GPU, is not made."""
import ctypes
import math

import pytest
import torch

NULL, SHAPE, ALIGN, UNSUPPORTED, VALUE, CUDA, ALIAS = 1, 2, 3, 4, 5, 6, 7
MB = 1 << 20


@pytest.fixture(scope="module")
def ag():
    import long_context_genomics_b200 as ag

    return ag


def _p(i):
    """A fake device address, 64 MB apart."""
    return (i + 1) << 26


def _fwd(ag, **kw):
    a = dict(x=_p(0), ldx=64, W=_p(1), ldw=64, bias=_p(2), residual=_p(3), ldr=32, M=16, N=32,
             K=64, dtype=1, act=2, preact=_p(4), ldz=32, y=_p(5), ldy=32, y_dtype=1, ws=None,
             n=0, stream=None)
    a.update(kw)
    return ag.lib.ag_linear_fwd(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), SHAPE), (dict(N=0), SHAPE), (dict(K=0), SHAPE),
    (dict(ldx=63), SHAPE), (dict(ldw=63), SHAPE), (dict(ldy=31), SHAPE), (dict(ldr=31), SHAPE),
    (dict(ldz=31), SHAPE), (dict(ldx=0), SHAPE), (dict(ldx=-64), SHAPE),
    (dict(M=(1 << 26) + 1), UNSUPPORTED), (dict(N=(1 << 20) + 1, ldy=1 << 21), UNSUPPORTED),
    (dict(ldx=(1 << 28) + 1), UNSUPPORTED),
    (dict(dtype=0), VALUE), (dict(dtype=3), VALUE), (dict(y_dtype=2), VALUE),
    (dict(act=-1), VALUE), (dict(act=5), VALUE),
    (dict(x=None), NULL), (dict(W=None), NULL), (dict(y=None), NULL),
    (dict(x=_p(0) + 1), ALIGN), (dict(y=_p(5) + 1), ALIGN), (dict(bias=_p(2) + 2), ALIGN),
    (dict(y_dtype=0, y=_p(5) + 2), ALIGN), (dict(ws=_p(6) + 128, n=MB), ALIGN),
    (dict(y=_p(0)), ALIAS), (dict(y=_p(1) + 64), ALIAS), (dict(y=_p(2)), ALIAS),
    (dict(y=_p(4)), ALIAS), (dict(preact=_p(0)), ALIAS), (dict(preact=_p(3)), ALIAS),
    (dict(y=_p(3) + 2), ALIAS), (dict(y=_p(3), ldy=40), ALIAS),
    (dict(M=0, x=None, W=None, y=None), 0),
])
def test_linear_fwd_refusals(ag, kw, status):
    assert _fwd(ag, **kw) == status


def test_linear_fwd_takes_what_it_documents(ag):
    """Calls that pass every check on the host: only the device is missing."""
    if torch.cuda.is_available():
        pytest.skip("would launch")
    end = (UNSUPPORTED, CUDA)
    assert _fwd(ag) in end
    assert _fwd(ag, y=_p(3)) in end                              # y in place of the residual
    assert _fwd(ag, bias=None, residual=None, preact=None, ldr=0, ldz=0) in end
    # Two column ranges of one wide matrix do not overlap.
    assert _fwd(ag, x=_p(0), ldx=128, y=_p(0) + 128, ldy=128) in end
    assert _fwd(ag, x=_p(0), ldx=128, y=_p(0) + 127 * 2, ldy=128) == ALIAS


def _bwd(ag, **kw):
    a = dict(dy=_p(0), lddy=32, x=_p(1), ldx=64, W=_p(2), ldw=64, preact=_p(3), ldz=64, act=2,
             M=16, N=32, K=64, dtype=1, dx=_p(4), lddx=64, dx_dtype=1, dW=_p(5), lddw=64,
             dW_dtype=0, db=_p(6), ws=None, n=0, stream=None)
    a.update(kw)
    return ag.lib.ag_linear_bwd(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), SHAPE), (dict(N=0), SHAPE), (dict(lddy=31), SHAPE), (dict(ldx=63), SHAPE),
    (dict(ldw=63), SHAPE), (dict(lddx=63), SHAPE), (dict(lddw=63), SHAPE), (dict(ldz=63), SHAPE),
    (dict(K=(1 << 20) + 1, ldx=1 << 21, ldw=1 << 21, lddx=1 << 21, lddw=1 << 21, ldz=1 << 21),
     UNSUPPORTED),
    (dict(dtype=0), VALUE), (dict(dx_dtype=2), VALUE), (dict(dW_dtype=7), VALUE),
    (dict(act=9), VALUE), (dict(preact=None), VALUE),
    (dict(dy=None), NULL), (dict(x=None), NULL), (dict(W=None), NULL),
    (dict(dy=_p(0) + 1), ALIGN), (dict(dW=_p(5) + 2), ALIGN), (dict(db=_p(6) + 2), ALIGN),
    (dict(dx=_p(4) + 1), ALIGN),
    (dict(dx=_p(0)), ALIAS), (dict(dx=_p(3)), ALIAS), (dict(dW=_p(1)), ALIAS),
    (dict(dW=_p(4)), ALIAS), (dict(db=_p(5) + 16), ALIAS), (dict(db=_p(2)), ALIAS),
    (dict(dx=None, dW=None, db=None, dy=None), 0),
    (dict(M=0, dW=None, db=None, dy=None), 0),
])
def test_linear_bwd_refusals(ag, kw, status):
    assert _bwd(ag, **kw) == status


def test_linear_bwd_reads_only_what_a_wanted_output_needs(ag):
    if torch.cuda.is_available():
        pytest.skip("would launch")
    end = (UNSUPPORTED, CUDA)
    assert _bwd(ag) in end
    assert _bwd(ag, dx=None, W=None, preact=None, ldz=0, ldw=0, lddx=0) in end
    assert _bwd(ag, dW=None, x=None, ldx=0, lddw=0) in end
    assert _bwd(ag, dx=None, dW=None, x=None, W=None) in end


def test_linear_workspace_queries(ag):
    n = ctypes.c_int64(-1)
    f, b = ag.lib.ag_linear_fwd_workspace, ag.lib.ag_linear_bwd_workspace
    assert f(_p(0), 64, _p(1), 64, 16, 32, 64, None) == NULL
    assert f(_p(0), 63, _p(1), 64, 16, 32, 64, ctypes.byref(n)) == SHAPE
    assert f(_p(0), 64, _p(1), 64, 0, 32, 64, ctypes.byref(n)) == 0 and n.value == 0
    assert b(_p(0), 32, _p(1), 64, _p(2), 64, 16, 32, 64, None, None, None, None) == NULL
    assert b(_p(0), 31, _p(1), 64, _p(2), 64, 16, 32, 64, None, None, None,
             ctypes.byref(n)) == SHAPE
    assert b(_p(0), 32, _p(1), 64, _p(2), 64, 0, 32, 64, _p(3), _p(4), None,
             ctypes.byref(n)) == 0 and n.value == 0


def _qk(ag, **kw):
    a = dict(q=_p(0), q_sb=9 * 128 * 7, q_sl=9 * 128, q_sh=128, k=_p(0) + 8 * 256,
             k_sb=9 * 128 * 7, k_sl=9 * 128, k_sh=128, x_dtype=1, qw=_p(1), qb=None, kw=_p(2),
             kb=None, norm=1, eps=1e-6, freq=_p(3), R=128, rope=0, pos=_p(4), pos_sb=7, B=2,
             Hq=8, Hk=1, L=7, D=128, q_out=_p(5), k_out=_p(6), out_dtype=1, stream=None)
    a.update(kw)
    return ag.lib.ag_qk_norm_rope_fwd(*a.values())


QK_REFUSALS = [
    (dict(B=-1), SHAPE), (dict(L=-1), SHAPE), (dict(Hq=-1), SHAPE), (dict(D=0), SHAPE),
    (dict(R=127), SHAPE), (dict(R=130), SHAPE), (dict(R=-2), SHAPE), (dict(q_sl=-1), SHAPE),
    (dict(pos_sb=-1), SHAPE),
    (dict(D=1025), UNSUPPORTED), (dict(B=1 << 20, L=1 << 20), UNSUPPORTED),
    (dict(B=1 << 20, L=1 << 10, Hq=8), UNSUPPORTED), (dict(q_sb=1 << 60), UNSUPPORTED),
    (dict(pos_sb=1 << 60), UNSUPPORTED),
    (dict(norm=3), VALUE), (dict(eps=-1.0), VALUE), (dict(eps=math.nan), VALUE),
    (dict(eps=math.inf), VALUE), (dict(rope=2), VALUE), (dict(x_dtype=5), VALUE),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(freq=None), NULL),
    (dict(q=_p(0) + 1), ALIGN), (dict(freq=_p(3) + 4), ALIGN), (dict(pos=_p(4) + 4), ALIGN),
    (dict(qw=_p(1) + 2), ALIGN),
]


@pytest.mark.parametrize("kw,status", QK_REFUSALS + [
    (dict(out_dtype=3), VALUE), (dict(q_out=None), NULL), (dict(k_out=None), NULL),
    (dict(q_out=_p(5) + 1), ALIGN),
    (dict(q_out=_p(0)), ALIAS), (dict(k_out=_p(0) + 64), ALIAS), (dict(q_out=_p(6)), ALIAS),
    (dict(q_out=_p(1)), ALIAS), (dict(k_out=_p(3)), ALIAS), (dict(k_out=_p(4)), ALIAS),
    (dict(B=0, q=None, k=None), 0), (dict(L=0, q_out=None), 0),
    (dict(Hq=0, Hk=0, q=None, k=None), 0),
])
def test_qk_fwd_refusals(ag, kw, status):
    assert _qk(ag, **kw) == status


def _qk_bwd(ag, **kw):
    a = dict(gq=_p(7), gk=_p(8), g_dtype=0, q=_p(0), q_sb=9 * 128 * 7, q_sl=9 * 128, q_sh=128,
             k=_p(0) + 8 * 256, k_sb=9 * 128 * 7, k_sl=9 * 128, k_sh=128, x_dtype=1, qw=_p(1),
             kw=_p(2), norm=1, eps=1e-6, freq=_p(3), R=128, rope=0, pos=_p(4), pos_sb=7, B=2,
             Hq=8, Hk=1, L=7, D=128, dq=_p(5), dq_sb=9 * 128 * 7, dq_sl=9 * 128, dq_sh=128,
             dk=_p(5) + 8 * 256, dk_sb=9 * 128 * 7, dk_sl=9 * 128, dk_sh=128, dqw=_p(9),
             dqb=_p(10), dkw=_p(11), dkb=_p(12), ws=None, n=0, stream=None)
    a.update(kw)
    return ag.lib.ag_qk_norm_rope_bwd(*a.values())


@pytest.mark.parametrize("kw,status", QK_REFUSALS + [
    (dict(g_dtype=3), VALUE), (dict(gq=None), NULL), (dict(dk=None), NULL),
    (dict(gq=_p(7) + 2), ALIGN), (dict(dqw=_p(9) + 1), ALIGN), (dict(dq=_p(5) + 1), ALIGN),
    # Gradients whose elements would share addresses.
    (dict(dq_sl=0), SHAPE), (dict(dq_sh=64), SHAPE), (dict(dk_sb=64), SHAPE),
    (dict(dq_sl=8 * 128 - 1), SHAPE),
    (dict(dq=_p(0)), ALIAS), (dict(dk=_p(7)), ALIAS), (dict(dqw=_p(10)), ALIAS),
    (dict(dkb=_p(5)), ALIAS), (dict(dqb=_p(1)), ALIAS),
    (dict(dk=_p(5) + 7 * 256), ALIAS),                # dk inside dq's last head
    (dict(dk=_p(5) + 8 * 256 + 2), ALIAS),            # dk runs into the next position
    (dict(dk_sl=10 * 128), ALIAS),                    # another stride: not side by side
    (dict(B=0, dqw=None, dqb=None, dkw=None, dkb=None), 0),
])
def test_qk_bwd_refusals(ag, kw, status):
    assert _qk_bwd(ag, **kw) == status


def test_qk_bwd_takes_gradients_side_by_side(ag):
    if torch.cuda.is_available():
        pytest.skip("would launch")
    end = (UNSUPPORTED, CUDA)
    assert _qk_bwd(ag) in end
    assert _qk_bwd(ag, dk=_p(13), dk_sb=128 * 7, dk_sl=128) in end
    assert _qk_bwd(ag, Hk=0, gk=None, k=None, dk=None, dkw=None, dkb=None) in end


def _clip(ag, ptrs, counts, types, max_norm=1.0, eps=1e-6, norm=_p(20), ws=None, size=0, n=None):
    n = len(ptrs) if n is None else n
    m = max(1, len(ptrs))
    return ag.lib.ag_grad_clip((ctypes.c_void_p * m)(*ptrs), (ctypes.c_int64 * m)(*counts),
                               (ctypes.c_int * m)(*types), n, max_norm, eps, norm, ws, size, None)


def test_grad_clip_refusals(ag):
    ok = ([_p(0), _p(1)], [100, 200], [0, 1])
    assert _clip(ag, *ok, n=-1) == SHAPE
    assert _clip(ag, *ok, n=(1 << 20) + 1) == UNSUPPORTED
    assert _clip(ag, *ok, max_norm=-1.0) == VALUE
    assert _clip(ag, *ok, max_norm=math.nan) == VALUE
    assert _clip(ag, *ok, eps=-1e-6) == VALUE
    assert _clip(ag, *ok, norm=None) == NULL
    assert ag.lib.ag_grad_clip(None, None, None, 1, 1.0, 0.0, _p(20), None, 0, None) == NULL
    assert _clip(ag, [_p(0)], [-1], [0]) == SHAPE
    assert _clip(ag, [_p(0)], [(1 << 40) + 1], [0]) == SHAPE
    assert _clip(ag, [_p(0)] * 5, [1 << 40] * 5, [0] * 5) == UNSUPPORTED
    assert _clip(ag, [_p(0)], [1], [3]) == VALUE
    assert _clip(ag, [None], [1], [0]) == NULL
    assert _clip(ag, [_p(0) + 2], [1], [0]) == ALIGN
    assert _clip(ag, [_p(0) + 1], [1], [1]) == ALIGN
    assert _clip(ag, *ok, norm=_p(20) + 2) == ALIGN
    assert _clip(ag, [_p(0), _p(0)], [100, 100], [0, 0]) == ALIAS        # the same tensor twice
    assert _clip(ag, [_p(0) + 396, _p(0)], [1, 100], [0, 0]) == ALIAS    # its last element
    assert _clip(ag, [_p(0)], [100], [0], norm=_p(0) + 4) == ALIAS
    if not torch.cuda.is_available():
        end = (UNSUPPORTED, CUDA)
        assert _clip(ag, *ok) in end
        assert _clip(ag, [_p(0) + 400, _p(0)], [1, 100], [0, 0]) in end  # side by side
        assert _clip(ag, [None, _p(0)], [0, 3], [0, 0]) in end           # an empty one


def test_binding_refusals(ag):
    cpu = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ag.ag_linear_fwd(cpu, cpu)
    with pytest.raises(TypeError):
        ag.ag_linear_fwd([1.0], cpu)
    with pytest.raises(ValueError, match="CUDA"):
        ag.ag_linear_bwd(cpu, cpu, cpu)
    with pytest.raises(ValueError, match="CUDA"):
        ag.ag_qk_norm_rope_fwd(torch.zeros(1, 2, 3, 4), None)
    with pytest.raises(ValueError, match="both None"):
        ag.ag_qk_norm_rope_fwd(None, None)
    with pytest.raises(ValueError, match="CUDA"):
        ag.ag_grad_clip([cpu], 1.0)
    with pytest.raises(ValueError, match="no tensor"):
        ag.ag_grad_clip([None], 1.0)
    with pytest.raises(ValueError, match="act must be"):
        ag._code(ag.ACTIVATIONS, "swish", "act")
    assert ag._is_dense(torch.zeros(3, 4).t()) and not ag._is_dense(torch.zeros(3, 4)[:, :2])
    f = ag.ag_rope_frequencies(8, base=100.0, device="cpu")
    assert f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([1.0, 100 ** -0.25, 0.1, 100 ** -0.75]).double())


def _elements(at, n, s, D):
    i = torch.arange(D) + at
    for count, stride in zip(n, s):
        i = (i[None] + torch.arange(count)[:, None] * stride).flatten()
    return set(i.tolist())


SIDE_BY_SIDE = {
    # One position in each of two sequences: the slices' views give the length of
    # one another strides (a view of a dimension of one element may have any).
    "one position": dict(L=1, dq_sb=1152, dq_sl=1024, dk_sb=1152, dk_sl=1152),
    "one sequence": dict(B=1, dq_sb=1024, dk_sb=9 * 128 * 7),
    "one of both": dict(B=1, L=1, dq_sb=1024, dq_sl=1024, dk_sb=128, dk_sl=128),
    # [B, L, H, 3, D]: each head's query, key and value together.
    "interleaved heads": dict(Hq=4, Hk=4, dq_sb=7 * 1536, dq_sl=1536, dq_sh=384, dk_sb=7 * 1536,
                              dk_sl=1536, dk_sh=384, dk=_p(5) + 256),
    # [B, 9, L, D]: the attention's own order, the keys behind the queries.
    "heads before positions": dict(dq_sb=9 * 7 * 128, dq_sl=128, dq_sh=7 * 128, dk_sb=9 * 7 * 128,
                                   dk_sl=128, dk_sh=7 * 128, dk=_p(5) + 8 * 7 * 256),
    # [B, L, Hk, 1 + 1, D] with the keys first.
    "keys first": dict(Hq=4, Hk=4, dk=_p(5), dq=_p(5) + 256, dq_sb=7 * 1024, dq_sl=1024, dq_sh=256,
                       dk_sb=7 * 1024, dk_sl=1024, dk_sh=256),
}


@pytest.mark.parametrize("layout", SIDE_BY_SIDE)
def test_qk_bwd_takes_gradients_of_any_fused_layout(ag, layout):
    kw = SIDE_BY_SIDE[layout]
    if torch.cuda.is_available():
        pytest.skip("would launch")
    assert _qk_bwd(ag, **kw) in (UNSUPPORTED, CUDA)


def test_qk_bwd_refuses_shared_elements_exactly(ag):
    """Small layouts of every order against the sets of their elements."""
    if torch.cuda.is_available():
        pytest.skip("would launch")
    import itertools
    import random

    rng = random.Random(5)
    B, L, D, seen = 2, 3, 4, [0, 0]
    for _ in range(3000):
        heads = [rng.choice([1, 2]), rng.choice([1, 2])]
        strides = []
        for H in heads:
            n, s, inner = (B, L, H), [0, 0, 0], D
            for i in rng.choice(list(itertools.permutations(range(3)))):
                s[i] = inner + rng.choice([0, 0, 4, 4, 8, 24])
                inner = s[i] * (n[i] - 1) + inner if rng.random() < 0.5 else s[i] * n[i]
            strides.append(s)
        if rng.random() < 0.6:
            strides[1] = strides[0]
        at = rng.randrange(0, 200, 4) - 100
        a = _elements(0, (B, L, heads[0]), strides[0], D)
        b = _elements(at, (B, L, heads[1]), strides[1], D)
        if len(a) != B * L * heads[0] * D or len(b) != B * L * heads[1] * D:
            continue
        q, k = strides
        st = _qk_bwd(ag, B=B, L=L, Hq=heads[0], Hk=heads[1], D=D, R=4, pos_sb=L, dq=_p(5),
                     dq_sb=q[0], dq_sl=q[1], dq_sh=q[2], dk=_p(5) + 2 * at, dk_sb=k[0], dk_sl=k[1],
                     dk_sh=k[2])
        if st == SHAPE:  # (distinct, but not by steps over what lies inside)
            continue
        shared = bool(a & b)
        assert st == ALIAS if shared else st in (UNSUPPORTED, CUDA), (q, k, at, heads)
        seen[shared] += 1
    assert min(seen) > 200


def test_linear_stride_of_one_row_is_free(ag):
    """Nothing uses it: the last position of a long sequence is one row whose
    stride is the sequence's."""
    if torch.cuda.is_available():
        pytest.skip("would launch")
    end, far = (UNSUPPORTED, CUDA), 1 << 40
    n = ctypes.c_int64(0)
    f = ag.lib.ag_linear_fwd_workspace
    no_device = f(_p(0), 64, _p(1), 64, 1, 32, 64, ctypes.byref(n))
    assert no_device in end
    if no_device == CUDA:
        end = (CUDA,)  # so that a refusal of the stride shows
    assert _fwd(ag, M=1, ldx=far, ldr=far + 1, ldz=far + 3, ldy=far) in end
    assert _fwd(ag, N=1, ldw=far + 1) in end
    assert f(_p(0), far, _p(1), far, 1, 1, 64, ctypes.byref(n)) in end
    assert _bwd(ag, M=1, lddy=far, ldx=far, lddx=far, ldz=far) in end
    assert _bwd(ag, N=1, ldw=far, lddw=far) in end
    assert _bwd(ag, M=1, lddy=31) == SHAPE
    assert _fwd(ag, M=2, ldx=far) == UNSUPPORTED


def test_rope_frequencies_of_an_odd_dimension_are_refused(ag):
    """(3 frequencies turn 6 elements, so 5 cannot be what was meant.)"""
    for n in (5, 1, -2):
        with pytest.raises(ValueError, match="even"):
            ag.ag_rope_frequencies(n, device="cpu")
    assert ag.ag_rope_frequencies(0, device="cpu").numel() == 0
