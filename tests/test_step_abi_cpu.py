"""Argument checks of norm_rope_f16, kv_append_norm_rope, kv_plan, attention_paged_tree and logits_adjust on the host (CPU
only: nothing is launched, the addresses are never read)."""

from __future__ import annotations

import ctypes

import pytest

from test_attention_abi_cpu import (ALIGN, CACHE_ALIGN, CACHE_SHAPE, DEVICE, E4M3, F32, NULL, OK, P, SHAPE, WORKSPACE,
                                    _lib, cache)

OVERLAP = -8


def norm_rope(**kw):
    a = dict(x=P, x_type=F32, ldx=256, w=P, eps=1e-6, pos=P, freq=P, y=P, ldy=256, T=4, H=2, D=128, R=128, inter=0, ms=1.0)
    a.update(kw)
    return _lib().norm_rope_f16(*a.values(), None)


def append(c=None, **kw):
    a = dict(q=P, ldq=512, qo=P, ldqo=512, Hq=4, k=P, ldk=256, v=P, ldv=256, t=F32, c=c or cache(), slot=P, pos=P,
             freq=P, qw=P, kw=P, eps=1e-6, T=4, R=128, inter=0, ms=1.0)
    a.update(kw)
    return _lib().kv_append_norm_rope(*a.values(), None)


def plan(**kw):
    a = dict(kv_len=P, new_len=P, B=4, table=P, ldt=8, W=8, owned=P, free=P, count=P, pages=64, page=16, depth=P, T=16,
             q_start=P, kv_total=P, pos=P, slot=P, status=P)
    a.update(kw)
    return _lib().kv_plan(*a.values(), None)


def attend(c=None, ws=None, size=None, **kw):
    a = dict(q=P, ldq=512, c=c or cache(), table=P, ldt=4, W=4, kv_len=P, q_start=P, mask=P, ldm=1, B=2, T=6, max_q=4,
             Hq=4, window=0, scale=0.1, out=P, ldo=512)
    a.update(kw)
    n = ctypes.c_size_t(0) if size is None else size
    return _lib().attention_paged_tree(*a.values(), ws, ctypes.byref(n), None)


def adjust(logits=P, ldl=1000, M=4, V=1000, out=P + 65536, ldo=1000, none=False, **kw):
    from int4_weight_only_group_amd._lib import LogitRules
    r = LogitRules()
    a = dict(request=P, requests=4, tokens=P, ld_tokens=50, max_tokens=50, token_len=P, prompt_len=P, repetition=P,
             frequency=P, presence=P, bias=P, bias_id=P, bias_start=P, biases=9, mask=P, ld_mask=32, masks=3, mask_row=P)
    a.update(kw)
    for n, x in a.items():
        setattr(r, n, x)
    return _lib().logits_adjust(logits, ldl, M, V, None if none else ctypes.byref(r), out, ldo, None)


def test_norm_rope_refusals():
    for n in ("x", "pos", "freq", "y"):
        assert norm_rope(**{n: None}) == NULL
    for bad in (dict(T=0), dict(T=1 << 24), dict(H=0), dict(H=1025, ldx=1025 * 128, ldy=1025 * 128), dict(D=12),
                dict(D=264), dict(R=130), dict(R=7), dict(ldx=248), dict(ldy=248), dict(x_type=E4M3),
                dict(ms=float("nan")), dict(eps=0.0), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=1e31),
                dict(eps=1e-31)):
        assert norm_rope(**bad) == SHAPE, bad
    for bad in (dict(x=P + 8), dict(y=P + 8), dict(ldx=260), dict(pos=P + 2), dict(freq=P + 1), dict(w=P + 4)):
        assert norm_rope(**bad) == ALIGN, bad


def test_append_refusals():
    for n in ("qo", "q", "k", "v", "slot", "pos", "freq"):
        assert append(**{n: None}) == NULL, n
    for bad in CACHE_SHAPE:
        assert append(c=cache(**bad)) == SHAPE, bad
    for bad in CACHE_ALIGN:
        assert append(c=cache(**bad)) == ALIGN, bad
    for bad in (dict(T=0), dict(Hq=0), dict(R=130), dict(ldk=248), dict(ldq=504), dict(t=E4M3), dict(eps=0.0),
                dict(eps=float("inf"))):
        assert append(**bad) == SHAPE, bad
    for bad in (dict(slot=P + 4), dict(k=P + 4), dict(qw=P + 4), dict(kw=P + 8)):
        assert append(**bad) == ALIGN, bad


def test_plan_refusals():
    for n in ("kv_len", "new_len", "table", "owned", "free", "count", "q_start", "kv_total", "pos", "slot", "status"):
        assert plan(**{n: None}) == NULL, n
    for bad in (dict(B=0), dict(B=(1 << 20) + 1), dict(T=0), dict(T=1 << 24), dict(W=0), dict(ldt=7), dict(page=0),
                dict(page=-1), dict(pages=0), dict(pages=1 << 27), dict(W=1 << 26, ldt=1 << 26, page=17), dict(pages=1 << 62),
                dict(page=1 << 62), dict(W=1 << 62, ldt=1 << 62), dict(B=1 << 20, W=1 << 11, ldt=1 << 11)):
        assert plan(**bad) == SHAPE, bad
    for bad in (dict(kv_len=P + 1), dict(new_len=P + 2), dict(table=P + 3), dict(owned=P + 1), dict(free=P + 2),
                dict(count=P + 2), dict(depth=P + 1), dict(q_start=P + 2), dict(kv_total=P + 2), dict(pos=P + 2),
                dict(slot=P + 4), dict(status=P + 1)):
        assert plan(**bad) == ALIGN, bad


def test_tree_refusals():
    for n in ("q", "table", "kv_len", "out", "mask"):
        assert attend(**{n: None}) == NULL, n
    for bad in CACHE_SHAPE:
        assert attend(c=cache(**bad)) == SHAPE, bad
    for bad in CACHE_ALIGN:
        assert attend(c=cache(**bad)) == ALIGN, bad
    for bad in (dict(ldm=0), dict(ldm=-1), dict(T=80, max_q=65), dict(window=3), dict(window=-1), dict(B=0), dict(T=0),
                dict(max_q=7), dict(Hq=3), dict(scale=0.0), dict(q_start=None), dict(ldq=504), dict(ldm=1 << 31)):
        assert attend(**bad) == SHAPE, bad
    assert attend(mask=P + 4) == ALIGN
    n = ctypes.c_size_t(0)
    for good in (dict(window=4), dict(window=1 << 40), dict(T=80, max_q=65, ldm=2), dict(q_start=None, max_q=1)):
        assert attend(size=n, **good) == OK, good


def test_tree_workspace():
    for kw in (dict(W=4096, ldt=4096, B=1, T=1, max_q=1), dict(W=900, ldt=900, B=3, T=90, max_q=40, ldm=1), dict()):
        n = ctypes.c_size_t(1)
        assert attend(size=n, **kw) == OK
        if n.value:
            assert attend(ws=P, size=ctypes.c_size_t(n.value - 1), **kw) == WORKSPACE
            assert attend(ws=P + 8, size=n, **kw) == ALIGN


def test_trees_that_no_launch_holds():
    def size(heads, G, dim=8, **kw):
        n = ctypes.c_size_t(1)
        c = cache(heads=heads, dim=dim, stride_page=heads * 16 * dim, stride_head=16 * dim, stride_token=dim)
        ld = heads * G * dim
        return attend(c=c, size=n, ldq=ld, ldo=ld, Hq=heads * G, **{**dict(ldt=1 << 16, W=1 << 16, ldm=1 << 14), **kw}), n.value

    n = 1 << 20
    for heads, G, dim, kw in ((1024, 1, 8, dict(B=n, T=n, max_q=1, q_start=None)), (64, 4, 256, dict(B=n, T=1 << 22, max_q=16)),
                              (1024, 1, 8, dict(B=n, T=n, max_q=n))):
        assert size(heads, G, dim, **kw)[0] == SHAPE, (heads, G, kw)
    for heads, G, dim, kw in ((1, 16, 8, dict(B=n - 1, T=n - 1, max_q=1, q_start=None)), (1, 128, 8, dict(B=n - 1, T=n, max_q=n)),
                              (1, 8, 256, dict(B=n - 1, T=1 << 23, max_q=8)), (8, 16, 128, dict(B=1 << 16, T=1 << 20, max_q=16)),
                              (1023, 1, 256, dict(B=1025, T=1 << 17, max_q=128))):
        assert size(heads, G, dim, **kw)[0] == OK, (heads, G, kw)


def test_adjust_refusals():
    assert adjust(logits=None) == NULL and adjust(out=None) == NULL and adjust(none=True) == NULL
    for n in ("token_len", "bias_id", "bias_start"):
        assert adjust(**{n: None}) == NULL, n
    big = 1 << 31
    for bad in (dict(M=0), dict(V=0), dict(V=big, ldl=big, ldo=big, ld_mask=big), dict(ldl=999), dict(ldo=999), dict(requests=0),
                dict(request=None, requests=3), dict(max_tokens=-1), dict(ld_tokens=49), dict(max_tokens=big, ld_tokens=big),
                dict(biases=-1), dict(biases=big - 1), dict(masks=0), dict(mask_row=None), dict(ld_mask=31),
                dict(M=1 << 24), dict(M=1 << 14, V=1 << 22, ldl=1 << 22, ldo=1 << 22, ld_mask=1 << 17)):
        assert adjust(**bad) == SHAPE, bad
    assert adjust(out=P, ldo=1004) == OVERLAP
    for n in ("logits", "out", "request", "tokens", "token_len", "prompt_len", "repetition", "frequency", "presence", "bias",
              "bias_id", "bias_start", "mask", "mask_row"):
        assert adjust(**{n: P + 2}) == ALIGN, n


def test_no_device_is_an_error():
    import torch
    if torch.cuda.is_available():
        pytest.skip("there is a device")
    n = ctypes.c_size_t(1 << 40)
    assert attend(ws=P, size=n) == DEVICE
    assert norm_rope() == DEVICE and norm_rope(w=None, R=0, freq=None) == DEVICE and norm_rope(R=58) == DEVICE
    assert append() == DEVICE and append(q=None, qo=None, qw=None, kw=None) == DEVICE
    assert plan() == DEVICE and plan(depth=None) == DEVICE
    assert adjust() == DEVICE and adjust(out=P) == DEVICE
    assert adjust(request=None, tokens=None, token_len=None, bias=None, mask=None) == DEVICE
