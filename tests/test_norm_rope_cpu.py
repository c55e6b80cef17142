"""Argument checks of the norm and rotation and of the append: every refusal
is made on the host, before any launch."""
import ctypes

import pytest
import torch

from head_partitioned_distance_b200 import spa


def _fake(addr):
    return ctypes.c_void_p(addr)


P = _fake(1 << 20)  # never dereferenced: every call below fails its checks first
ODD = _fake((1 << 20) + 8)


def _s(*v):
    return (ctypes.c_int64 * len(v))(*v)


def fwd(ptrs=None, B=1, Hq=4, Hk=2, N=100, d=64, rot=64, length=100, pos=None, qs=(25600, 64, 256), ks=(12800, 64, 128),
        eps=1e-6, dtype=0):
    p = list(ptrs or [P] * 7)
    return spa._lib.spa_qk_norm_rope_fwd(*p[:5], pos, *p[5:], B, Hq, Hk, N, d, rot, length, 0, _s(*qs), _s(*ks), 0, eps,
                                         dtype, None)


REFUSALS = [
    (dict(B=0), 1), (dict(Hq=0), 1), (dict(Hk=0), 1), (dict(N=0), 1), (dict(length=0), 1), (dict(length=99), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(dtype=2), 1),
    (dict(dtype=-1), 1), (dict(d=96, rot=32), 2), (dict(rot=8), 2), (dict(rot=24), 2), (dict(rot=128), 2),
    (dict(Hq=1020, Hk=5), 2), (dict(B=1 << 16, N=1 << 16, length=1 << 16), 2), (dict(qs=(25600, 64, 257)), 2),
    (dict(qs=(25600, 60, 256)), 2), (dict(ks=(12800, 64, 4)), 2), (dict(pos=_fake((1 << 20) + 2)), 2),
]


@pytest.mark.parametrize("kw,status", REFUSALS)
def test_forward_refuses(kw, status):
    assert fwd(**kw) == status


def test_forward_refuses_pointers():
    for i in range(7):
        p = [P] * 7
        p[i] = None
        assert fwd(p) == spa.SPA_ERR_INVAL
        p[i] = ODD
        assert fwd(p) == spa.SPA_ERR_UNSUPPORTED


def test_backward_refuses():
    def bwd(p=None, qs=(25600, 64, 256), dqs=(25600, 6400, 64), d=64, N=100, length=100):
        p = list(p or [P] * 12)
        return spa._lib.spa_qk_norm_rope_bwd(*p[:7], None, *p[7:], 1, 4, 2, N, d, 64, length, 0, _s(*qs),
                                             _s(12800, 64, 128), _s(*dqs), _s(12800, 6400, 64), 0, 1e-6, 0, None)

    for i in range(12):
        p = [P] * 12
        p[i] = None
        assert bwd(p) == spa.SPA_ERR_INVAL
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 8, 11):  # dwq and dwk are written one by one
        p = [P] * 12
        p[i] = ODD
        assert bwd(p) == spa.SPA_ERR_UNSUPPORTED
    assert bwd(dqs=(25600, 6400, 63)) == spa.SPA_ERR_UNSUPPORTED
    assert bwd(dqs=(25600, 0, 64)) == spa.SPA_ERR_INVAL  # heads of a gradient on top of one another
    assert bwd(d=32) == spa.SPA_ERR_UNSUPPORTED
    assert bwd(length=50) == spa.SPA_ERR_INVAL
    assert spa.spa_qk_norm_rope_bwd_workspace_bytes(96) == 0
    assert spa.spa_qk_norm_rope_bwd_workspace_bytes(64) > 0


def test_table_refuses():
    f = lambda t=P, n=10, rot=64, base=1e4: spa._lib.spa_rope_table(t, n, rot, base, None)  # noqa: E731
    assert f(t=None) == f(n=0) == f(n=1 << 31) == f(base=0.0) == f(base=float("nan")) == spa.SPA_ERR_INVAL
    assert f(rot=24) == f(rot=0) == f(rot=144) == f(t=ODD) == spa.SPA_ERR_UNSUPPORTED


def test_append_refuses():
    def app(p=None, B=2, T=5, Hq=4, Hk=2, d=64, pages=10, page=16, width=3, rot=64, length=40, qs=(512, 64),
            vs=(512, 64), eps=1e-6, dtype=0):
        p = list(p or [P] * 12)
        return spa._lib.spa_paged_append(*p, B, T, Hq, Hk, d, pages, page, width, rot, length, _s(*qs), _s(512, 64),
                                         _s(*vs), 0, eps, dtype, None)

    for kw in (dict(B=0), dict(T=-1), dict(Hq=0), dict(pages=0), dict(width=0), dict(length=0), dict(eps=-1.0),
               dict(dtype=5)):
        assert app(**kw) == spa.SPA_ERR_INVAL, kw
    for kw in (dict(B=65536), dict(page=8), dict(page=48), dict(page=512), dict(d=80), dict(rot=80), dict(Hq=1021),
               dict(qs=(511, 64)), dict(vs=(512, 62))):
        assert app(**kw) == spa.SPA_ERR_UNSUPPORTED, kw
    for i in range(12):
        p = [P] * 12
        p[i] = None
        assert app(p) == spa.SPA_ERR_INVAL
        p[i] = _fake((1 << 20) + 2)
        assert app(p) == spa.SPA_ERR_UNSUPPORTED
    assert app([None] * 12, T=0) == spa.SPA_OK  # nothing to do, nothing launched


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    w, t = torch.ones(64), torch.zeros(3, 32, 2)
    with pytest.raises(ValueError, match="CUDA"):
        spa.qk_norm_rope_forward(x, x, w, w, t)
    with pytest.raises(ValueError, match="CUDA"):
        spa.spa_rope_table(t, 1e4)
    with pytest.raises(ValueError, match="CUDA"):
        spa.paged_append(x[0], x[0], x[0], x, x, None, None, None, w, w, t)
    with pytest.raises(ValueError, match="B, H, N, d"):
        spa.qk_norm_rope(x[0], x[0], w, w, t)


def test_paged_attention_refuses():
    def att(p=None, B=2, T=5, max_q=3, Hq=4, Hk=2, pages=10, page=16, width=3, N=48, d=64, scale=0.1, lo=None, hi=None,
            dtype=0):
        p = list(p or [P] * 9)
        a = None if lo is None else (ctypes.c_int32 * len(lo))(*lo)
        b = None if hi is None else (ctypes.c_int32 * len(hi))(*hi)
        return spa._lib.spa_paged_attn(*p, B, T, max_q, Hq, Hk, pages, page, width, N, d, scale, a, b, dtype, None)

    inval = [dict(B=0), dict(T=-1), dict(max_q=0), dict(Hq=0), dict(Hk=0), dict(Hq=5), dict(pages=0), dict(width=0),
             dict(N=0), dict(N=1 << 31), dict(N=3), dict(scale=0.0), dict(scale=float("nan")), dict(dtype=2),
             dict(lo=[0] * 4), dict(lo=[0] * 4, hi=[0] * 4), dict(lo=[-1] * 4, hi=[9] * 4),
             dict(lo=[0] * 4, hi=[49] * 4)]
    for kw in inval:
        assert att(**kw) == spa.SPA_ERR_INVAL, kw
    unsupported = [dict(B=65536), dict(Hq=258, N=300), dict(d=96), dict(page=8), dict(page=24), dict(page=512),
                   dict(pages=1 << 30)]
    for kw in unsupported:
        assert att(**kw) == spa.SPA_ERR_UNSUPPORTED, kw
    assert att([None] * 9, T=0) == spa.SPA_OK
    for i in range(9):
        p = [P] * 9
        p[i] = None
        assert att(p) == spa.SPA_ERR_INVAL
        p[i] = _fake((1 << 20) + 2)
        assert att(p) == spa.SPA_ERR_UNSUPPORTED
    p = [P] * 9
    p[6] = _fake((1 << 20) + 16)  # o is written in 32-byte stores
    assert att(p) == spa.SPA_ERR_UNSUPPORTED
    p[6], p[8] = P, _fake((1 << 20) + 128)
    assert att(p) == spa.SPA_ERR_UNSUPPORTED
    assert spa.spa_paged_attn_workspace_bytes(0, 64) == spa.spa_paged_attn_workspace_bytes(1, 96) == 0


@pytest.mark.parametrize("B,Hq,blocks", [(65534, 1, 32769), (64219, 32, 1045), (53965, 101, 394)])
def test_paged_attention_refuses_lists_at_the_32_bit_border(B, Hq, blocks):
    # the plan's 512 threads round their shares up: a list this close to 2^31
    # items would pass it on the way
    assert 2 ** 31 - 1 - 512 < B * Hq * blocks < 2 ** 31
    rows = 256 * blocks
    assert spa._lib.spa_paged_attn(*[P] * 9, B, rows, rows, Hq, Hq, 10, 16, 3, 4096, 64, 0.1, None, None, 0,
                                   None) == spa.SPA_ERR_UNSUPPORTED


def test_paged_attention_asks_for_the_length_of_the_bands():
    # the balanced bands belong to the model's length; the capacity of the page
    # table (16 * 3 here) is not that, and changes when the table grows
    q, kp = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 4, 16, 64, dtype=torch.bfloat16)
    table, cu, kv = (torch.zeros(s, dtype=torch.int32) for s in ((1, 3), (2,), (1,)))
    for bands in ({}, {"lo": [0] * 4}, {"hi": [9] * 4}):
        with pytest.raises(ValueError, match="length that the model was trained with"):
            spa.paged_attention(q, kp, kp, table, cu, kv, 2, **bands)
    # given the length, or the bands, the call goes on to its other checks
    for more in ({"N": 48}, {"lo": [0] * 4, "hi": [9] * 4}):
        with pytest.raises(ValueError, match="CUDA"):
            spa.paged_attention(q, kp, kp, table, cu, kv, 2, **more)


@pytest.mark.parametrize("rot", [17, 33, 129])
def test_rope_table_refuses_odd_columns(rot):
    # not the table of one column less
    with pytest.raises(ValueError, match="pairs"):
        spa.rope_table(10, rot, device="cpu")
