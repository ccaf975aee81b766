"""Argument checks of rope_f16, kv_append_rope and attention_paged on the host (CPU only: nothing is
launched, the addresses are never read)."""

from __future__ import annotations

import ctypes

import pytest

OK, NULL, SHAPE, ALIGN, WORKSPACE, DEVICE = 0, -1, -2, -3, -4, -5
P = 4096
F16, F32, E4M3 = 0, 1, 2


def _lib():
    from int4_weight_only_group_amd._lib import lib
    return lib()


def cache(**kw):
    from int4_weight_only_group_amd._lib import KvCache
    c = KvCache()
    a = dict(k=P, v=P, k_scale=None, v_scale=None, pages=8, page_size=16, heads=2, dim=128, stride_page=4096,
             stride_head=2048, stride_token=128, type=F16)
    a.update(kw)
    for n, x in a.items():
        setattr(c, n, x)
    return c


def rope(**kw):
    a = dict(x=P, x_type=F32, ldx=256, pos=P, freq=P, y=P, ldy=256, T=4, H=2, D=128, R=128, inter=0, inv=0, ms=1.0)
    a.update(kw)
    return _lib().rope_f16(*a.values(), None)


def append(c=None, **kw):
    a = dict(q=P, ldq=512, qo=P, ldqo=512, Hq=4, k=P, ldk=256, v=P, ldv=256, t=F32, c=c or cache(), slot=P, pos=P,
             freq=P, T=4, R=128, inter=0, ms=1.0)
    a.update(kw)
    return _lib().kv_append_rope(*a.values(), None)


def attend(c=None, ws=None, size=None, **kw):
    a = dict(q=P, ldq=512, c=c or cache(), table=P, ldt=4, W=4, kv_len=P, q_start=P, B=2, T=6, max_q=4, Hq=4,
             window=0, scale=0.1, out=P, ldo=512)
    a.update(kw)
    n = ctypes.c_size_t(0) if size is None else size
    return _lib().attention_paged(*a.values(), ws, ctypes.byref(n), None)


def test_rope_refusals():
    for n in ("x", "pos", "freq", "y"):
        assert rope(**{n: None}) == NULL
    for bad in (dict(T=0), dict(T=1 << 24), dict(H=0), dict(H=1025, ldx=1025 * 128, ldy=1025 * 128), dict(D=0),
                dict(D=12), dict(D=264), dict(R=129), dict(R=130), dict(R=-2), dict(R=7), dict(ldx=248),
                dict(ldy=248), dict(x_type=E4M3), dict(x_type=7), dict(ms=float("nan")), dict(ms=float("inf"))):
        assert rope(**bad) == SHAPE, bad
    for bad in (dict(x=P + 8), dict(y=P + 8), dict(ldx=260), dict(ldy=260), dict(pos=P + 2), dict(freq=P + 1)):
        assert rope(**bad) == ALIGN, bad


def test_append_refusals():
    for n in ("qo", "q", "k", "v", "slot", "pos", "freq"):
        assert append(**{n: None}) == NULL, n
    assert append(c=cache(k=None)) == NULL and append(c=cache(v=None)) == NULL
    for bad in (dict(T=0), dict(T=1 << 24), dict(Hq=0), dict(R=130), dict(R=3), dict(ldk=248), dict(ldv=0),
                dict(ldq=504), dict(ldqo=504), dict(t=E4M3), dict(ms=float("inf"))):
        assert append(**bad) == SHAPE, bad
    for bad in (dict(slot=P + 4), dict(k=P + 4), dict(v=P + 4), dict(q=P + 4), dict(qo=P + 4), dict(ldk=260)):
        assert append(**bad) == ALIGN, bad


CACHE_SHAPE = [dict(type=F32), dict(type=9), dict(pages=0), dict(page_size=0), dict(heads=0), dict(heads=1025),
               dict(dim=0), dict(dim=100), dict(dim=264), dict(dim=72, type=E4M3), dict(pages=1 << 20, page_size=1 << 11),
               dict(pages=1 << 40), dict(page_size=1 << 62, pages=1 << 62), dict(stride_page=-128),
               dict(stride_token=1 << 41)]
CACHE_ALIGN = [dict(k=P + 8), dict(v=P + 2), dict(stride_page=4100), dict(stride_head=2052), dict(stride_token=132),
               dict(stride_token=136, type=E4M3), dict(k_scale=P + 2, type=E4M3), dict(v_scale=P + 1, type=E4M3)]


@pytest.mark.parametrize("call", [append, attend])
def test_cache_refusals(call):
    for bad in CACHE_SHAPE:
        assert call(c=cache(**bad)) == SHAPE, bad
    for bad in CACHE_ALIGN:
        assert call(c=cache(**bad)) == ALIGN, bad


def test_attention_refusals():
    for n in ("q", "table", "kv_len", "out"):
        assert attend(**{n: None}) == NULL, n
    for bad in (dict(B=0), dict(B=(1 << 20) + 1), dict(T=0), dict(T=1 << 24), dict(max_q=0), dict(max_q=7), dict(W=0),
                dict(W=1 << 27, ldt=1 << 27), dict(ldt=3), dict(Hq=0), dict(Hq=3), dict(window=-1), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(ldq=504), dict(ldo=504),
                dict(q_start=None), dict(q_start=None, max_q=1, B=7), dict(Hq=1026, ldq=1026 * 128, ldo=1026 * 128),
                dict(T=(1 << 20) + 1, Hq=1024, ldq=1 << 17, ldo=1 << 17)):
        assert attend(**bad) == SHAPE, bad
    for bad in (dict(q=P + 8), dict(out=P + 8), dict(ldq=516), dict(ldo=516), dict(table=P + 2), dict(kv_len=P + 1),
                dict(q_start=P + 2)):
        assert attend(**bad) == ALIGN, bad


def test_attention_size_query_and_workspace():
    n = ctypes.c_size_t(123)
    big = dict(W=4096, ldt=4096, B=1, T=1, max_q=1)
    assert attend(size=n, **big) == OK
    if n.value:
        short = ctypes.c_size_t(n.value - 1)
        assert attend(ws=P, size=short, **big) == WORKSPACE
        assert attend(ws=P + 8, size=n, **big) == ALIGN


def test_no_device_is_an_error():
    import torch
    if torch.cuda.is_available():
        pytest.skip("there is a device")
    n = ctypes.c_size_t(1 << 40)
    assert attend(ws=P, size=n) == DEVICE
    assert rope() == DEVICE
    assert rope(R=0, freq=None) == DEVICE and rope(H=1, D=8, R=8) == DEVICE
    assert append() == DEVICE
    assert append(q=None, qo=None, Hq=0, ldq=0, ldqo=0) == DEVICE
    assert append(c=cache(type=E4M3, k_scale=P, v_scale=P)) == DEVICE


def test_attention_scale_keeps_its_products_normal():
    for bad in (1e-31, 1e-45, 1e31, 3e38):
        assert attend(scale=bad) == SHAPE, bad
    n = ctypes.c_size_t(0)
    assert attend(scale=1e-30, size=n) == OK and attend(scale=9.9e29, size=n) == OK


def _size(heads, G, dim=8, **kw):
    # the size query of a call; strides as of a [pages][heads][16][dim] cache
    n = ctypes.c_size_t(1)
    c = cache(heads=heads, dim=dim, stride_page=heads * 16 * dim, stride_head=16 * dim, stride_token=dim)
    ld = heads * G * dim
    return attend(c=c, size=n, ldq=ld, ldo=ld, Hq=heads * G, **{**dict(ldt=1 << 16, W=1 << 16), **kw}), n.value


def test_calls_that_no_launch_holds():
    # a launch has fewer than 2^32 threads, of workgroups of up to 256
    n = 1 << 20
    for heads, G, kw in (
            (1024, 1, dict(B=n, T=n, max_q=1, q_start=None)),  # parts (3 * 2^30 of them: past an int) and join
            (1024, 1, dict(B=n, T=n, max_q=1, q_start=None, W=1)),  # a workgroup per sequence and kv head
            (8, 16, dict(B=1 << 18, T=1 << 18, max_q=1, q_start=None)),  # the join's 16 rows of 2^21 pairs alone
            (16, 1, dict(B=n, T=n, max_q=2, W=1)),  # short ones beside others
            (1024, 1, dict(B=n, T=n, max_q=n)), (64, 17, dict(B=n - 1, T=n - 1, max_q=1 << 19))):  # tiles of many rows
        assert _size(heads, G, **kw)[0] == SHAPE, (heads, G, kw)
    # w4.h: taken while B * heads < 2^20 and T * Hq <= 2^29
    for heads, G, kw in (
            (1, 16, dict(B=n - 1, T=n - 1, max_q=1, q_start=None)), (1023, 1, dict(B=1025, T=1 << 19, max_q=512)),
            (1, 512, dict(B=n - 1, T=n, max_q=n)), (1, 1, dict(B=n - 1, T=n, max_q=2, W=2)),
            (1024, 1, dict(B=1023, T=1 << 19, max_q=1 << 19, W=2))):
        assert _size(heads, G, **kw)[0] == OK, (heads, G, kw)
