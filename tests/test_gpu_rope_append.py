"""rope_f16 and kv_append_rope against the fp64 oracle.

Bounds, per output.  The f32 path: the reduced angle is good to 1e-9 turns, cos and sin to 2 ulp of f32
(2^-22 with mscale's rounding), products and sum 3 roundings: (|a| + |b|) * mscale * 2^-20 covers it.
f16: half a step, 2^-11 of the value (2^-25 below the normal range).  e4m3: half a step, 2^-4 of the value
(2^-10 below the normal range), the f32 path's bound over the scale on top, and 2^-22 for the division.
"""

from __future__ import annotations

import numpy as np
import pytest

from oracle import attnref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import int4_weight_only_group_amd as m
    return m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def inputs(t, h, d, r, f32, seed, far=100000):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((t, h, d)).astype(np.float32 if f32 else np.float16)
    pos = rng.integers(0, far, t).astype(np.int32)
    freq = (1e4 ** (-2.0 * np.arange(r // 2) / max(r, 1))).astype(np.float32)
    return x, pos, freq


def pair_size(x, r, inter, mscale):
    """(|a| + |b|) * mscale of the pair that an element belongs to (0 where it is passed on)."""
    a, out, h = np.abs(x.astype(np.float64)), np.zeros(x.shape), r // 2
    ia, ib = (slice(0, r, 2), slice(1, r, 2)) if inter else (slice(0, h), slice(h, r))
    s = (a[..., ia] + a[..., ib]) * abs(mscale)
    out[..., ia], out[..., ib] = s, s
    return out


def close_f16(got, want, size):
    bound = np.abs(want) * 2.0 ** -11 + 2.0 ** -25 + size * 2.0 ** -20
    err = np.abs(got.astype(np.float64) - want)
    assert (err <= bound).all(), (err / bound).max()


def close_e4m3(codes, want, size, scale):
    got = ref.e4m3_values()[codes]
    y = np.clip(want / scale, -448, 448)
    bound = np.abs(y) * (2.0 ** -4 + 2.0 ** -22) + 2.0 ** -10 + size / scale * 2.0 ** -20
    err = np.abs(got - y)
    assert (err <= bound).all(), (err / bound).max()


ROPE = [  # tokens, heads, dim, rot, interleaved, f32, inverse, mscale
    (1, 1, 8, 8, False, True, False, 1.0), (1, 16, 128, 128, False, True, False, 1.0),
    (3, 5, 128, 128, True, False, True, 1.25), (64, 16, 128, 128, False, False, False, 1.0),
    (7, 2, 80, 32, True, True, False, 1.0), (7, 2, 80, 32, False, True, True, 1.0),
    (5, 3, 64, 0, False, True, False, 1.0), (5, 3, 64, 0, True, False, False, 1.0),
    (9, 2, 96, 58, False, True, False, 1.5), (9, 2, 96, 58, True, True, False, 1.5),
    (33, 7, 256, 256, False, True, True, 1.0), (33, 7, 256, 254, False, False, False, 1.0),
    (257, 4, 24, 6, True, True, False, 1.0), (1570, 2, 64, 64, False, True, False, 0.75),
    (2, 40, 72, 2, False, False, False, 1.0), (13, 18, 128, 48, False, False, True, 1.0),
]


@pytest.mark.parametrize("t,h,d,r,inter,f32,inv,ms", ROPE)
def test_rope(w4, t, h, d, r, inter, f32, inv, ms):
    x, pos, freq = inputs(t, h, d, r, f32, t + h + d)
    y = w4.rope_f16(dev(x), dev(pos), dev(freq), interleaved=inter, mscale=ms, inverse=inv).cpu().numpy()
    close_f16(y, ref.rope(x, pos, freq, interleaved=inter, mscale=ms, inverse=inv), pair_size(x, r, inter, ms))
    if r < d:
        assert np.array_equal(y[..., r:], x[..., r:].astype(np.float16))


def test_rope_far_and_negative_positions(w4):
    x, _, freq = inputs(6, 2, 128, 128, True, 3)
    pos = np.array([2 ** 31 - 1, -2 ** 31, 1 << 20, -12345, 0, -1], dtype=np.int32)
    y = w4.rope_f16(dev(x), dev(pos), dev(freq)).cpu().numpy()
    close_f16(y, ref.rope(x, pos, freq), pair_size(x, 128, False, 1.0))


@pytest.mark.parametrize("r,inter", [(128, False), (128, True), (58, False), (32, False), (32, True)])
def test_rope_in_place_and_strided_rows(w4, r, inter):
    x, pos, freq = inputs(19, 3, 128, r, False, r)
    want = w4.rope_f16(dev(x), dev(pos), dev(freq), interleaved=inter)
    rows = torch.full((19, 9, 128), 7.0, dtype=torch.float16, device="cuda")
    rows[:, 2:5] = dev(x)
    part = rows[:, 2:5]
    w4.rope_f16(part, dev(pos), dev(freq), interleaved=inter, out=part)
    assert torch.equal(part, want)
    assert (rows[:, :2] == 7).all() and (rows[:, 5:] == 7).all()


def test_rope_gradient_by_differences(w4):
    # <g, rope(x)> is linear in x, so its gradient is rope of g, inverse: against central differences
    # of the oracle, and as the adjoint of the kernel's own forward: <g, F x> = <F^T g, x> within the
    # roundings of both (2^-11 of sum |g| |Fx| and |F^T g| |x|)
    x, pos, freq = inputs(4, 2, 32, 24, True, 8)
    g, _, _ = inputs(4, 2, 32, 24, True, 9)
    grad = w4.rope_f16(dev(g), dev(pos), dev(freq), mscale=1.5, inverse=True).cpu().numpy().astype(np.float64)
    e = 1e-3
    for i in ((0, 0, 0), (1, 1, 13), (2, 0, 23), (3, 1, 31)):
        hi, lo = x.astype(np.float64), x.astype(np.float64)
        hi[i] += e
        lo[i] -= e
        diff = ((ref.rope(hi, pos, freq, mscale=1.5) - ref.rope(lo, pos, freq, mscale=1.5)) * g).sum() / (2 * e)
        assert abs(diff - grad[i]) <= abs(grad[i]) * 2.0 ** -10 + 1e-5
    y = w4.rope_f16(dev(x), dev(pos), dev(freq), mscale=1.5).cpu().numpy().astype(np.float64)
    slack = 2.0 ** -10 * (np.abs(g * y).sum() + np.abs(grad * x).sum())
    assert abs((g * y).sum() - (grad * x).sum()) <= slack


APPEND = [  # tokens, hq, hkv, dim, rot, interleaved, f32, e4m3, page, layout
    (1, 16, 2, 128, 128, False, True, False, 16, "phtd"), (64, 16, 8, 256, 256, False, True, True, 64, "phtd"),
    (37, 0, 3, 80, 32, True, False, False, 7, "pthd"), (130, 4, 1, 96, 96, False, True, True, 1, "pthd"),
    (5, 2, 2, 8, 8, False, True, False, 100, "phtd"), (33, 7, 7, 128, 58, False, False, True, 16, "kv"),
    (257, 3, 1, 64, 64, True, True, False, 32, "kv"), (9, 28, 4, 16, 6, False, True, True, 3, "phtd"),
    (700, 16, 2, 128, 128, False, True, False, 16, "phtd"),
]


def make_cache(pages, hkv, page, d, dtype, layout, fill):
    """k and v views [pages][heads][page][dim] of three memory layouts, every element `fill`."""
    code = torch.uint8 if dtype == torch.float8_e4m3fn else dtype
    if layout == "phtd":
        kv = [torch.full((pages, hkv, page, d), fill, dtype=code, device="cuda") for _ in range(2)]
    elif layout == "pthd":
        kv = [torch.full((pages, page, hkv, d), fill, dtype=code, device="cuda").transpose(1, 2) for _ in range(2)]
    else:  # both in one array
        one = torch.full((pages, 2, hkv, page, d), fill, dtype=code, device="cuda")
        kv = [one[:, 0], one[:, 1]]
    return [c.view(dtype) for c in kv]


@pytest.mark.parametrize("t,hq,hkv,d,r,inter,f32,e4m3,page,layout", APPEND)
def test_append(w4, t, hq, hkv, d, r, inter, f32, e4m3, page, layout):
    rng = np.random.default_rng(t + d)
    x, pos, freq = inputs(t, hq + 2 * hkv, d, r, f32, t)
    pages = -(-t // page) + 3
    slots = rng.permutation(pages * page)[:t].astype(np.int64)
    slots[::11] = -1  # padding tokens
    rows = dev(x)
    q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
    dtype = torch.float8_e4m3fn if e4m3 else torch.float16
    kc, vc = make_cache(pages, hkv, page, d, dtype, layout, 0x35 if e4m3 else 3.5)
    ks, vs = ((rng.random((2, hkv)) * 0.02 + 0.005).astype(np.float32) if e4m3 else (None, None))
    out = w4.kv_append_rope(k, v, kc, vc, dev(slots), dev(pos), dev(freq), q=q if hq else None, interleaved=inter,
                            k_scale=None if ks is None else dev(ks), v_scale=None if vs is None else dev(vs))
    turned = ref.rope(x[:, :hq + hkv], pos, freq, interleaved=inter)
    size = pair_size(x[:, :hq + hkv], r, inter, 1.0)
    if hq:
        close_f16(out.cpu().numpy(), turned[:, :hq], size[:, :hq])
    else:
        assert out is None
    at = np.where(slots >= 0)[0]
    page_of, off = slots[at] // page, slots[at] % page
    untouched = np.ones((pages, page), dtype=bool)
    untouched[page_of, off] = False
    for cache, want, sz, sc in ((kc, turned[:, hq:], size[:, hq:], ks),
                                (vc, x[:, hq + hkv:].astype(np.float64), np.zeros((t, hkv, d)), vs)):
        host = (cache.view(torch.uint8) if e4m3 else cache).cpu().numpy()
        got = host[page_of, :, off]
        if e4m3:
            close_e4m3(got, want[at], sz[at], sc[None, :, None].astype(np.float64))
        else:
            close_f16(got, want[at], sz[at])
        rest = host.transpose(0, 2, 1, 3)[untouched]
        assert (rest == (0x35 if e4m3 else np.float16(3.5))).all()


def test_append_v_is_one_rounding(w4):
    # V is not rotated: f16 and e4m3 caches hold exactly the rounded value, ties and saturation included
    vals = np.array([0.0, -0.0, 1 + 2.0 ** -11, 1 + 3 * 2.0 ** -11, 17.0, 19.0, -17.0, 448.0, 464.0, 1e5, -1e30,
                     2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9, 2.0 ** -26, np.inf], dtype=np.float32)
    v = np.stack([vals, vals[::-1]])[:, None, :].copy()
    k = np.zeros_like(v)
    for dtype in (torch.float16, torch.float8_e4m3fn):
        kc, vc = make_cache(1, 1, 4, 16, dtype, "phtd", 0)
        w4.kv_append_rope(dev(k), dev(v), kc, vc, dev(np.array([2, 0], dtype=np.int64)),
                          dev(np.array([5, 6], dtype=np.int32)), torch.empty(0, device="cuda"))
        if dtype == torch.float16:
            got = vc[0, 0].cpu().numpy().view(np.uint16)
            with np.errstate(over="ignore"):
                assert np.array_equal(got[[2, 0]], v[:, 0].astype(np.float16).view(np.uint16))
        else:
            assert np.array_equal(vc.view(torch.uint8)[0, 0].cpu().numpy()[[2, 0]], ref.e4m3_round(v[:, 0]))


def test_append_keeps_nan(w4):
    v = np.full((1, 1, 16), np.nan, dtype=np.float32)
    kc, vc = make_cache(1, 1, 1, 16, torch.float8_e4m3fn, "phtd", 0)
    w4.kv_append_rope(dev(v), dev(v), kc, vc, dev(np.zeros(1, np.int64)), dev(np.zeros(1, np.int32)),
                      dev(np.ones(8, np.float32)))
    assert torch.isnan(kc.float()).all() and torch.isnan(vc.float()).all()


def test_append_skips_slots_outside_the_cache(w4):
    x = np.ones((5, 1, 16), dtype=np.float32)
    slots = np.array([-1, 8, 1 << 40, -(1 << 62), 3], dtype=np.int64)
    kc, vc = make_cache(2, 1, 4, 16, torch.float16, "phtd", 0)
    q = w4.kv_append_rope(dev(x), dev(x), kc, vc, dev(slots), dev(np.zeros(5, np.int32)),
                          dev(np.ones(8, np.float32)), q=dev(x))
    assert (q == 1).all()  # the queries of padding tokens are still there
    want = torch.zeros_like(vc)
    want[0, 0, 3] = 1
    assert torch.equal(vc, want) and torch.equal(kc, want)


def test_append_far_offsets(w4):
    # elements past 2^32 of the cache
    pages, page, d = 2100, 16384, 128
    kc = torch.empty((pages, 1, page, d), dtype=torch.float16, device="cuda")
    vc = torch.empty_like(kc)
    x = np.random.default_rng(0).standard_normal((3, 1, d)).astype(np.float32)
    slots = np.array([pages * page - 1, 2, (1 << 25) + 5], dtype=np.int64)  # x 128: past 2^32 elements
    near = [kc.view(-1, d)[s - 1].clone() for s in slots.tolist()]
    w4.kv_append_rope(dev(x), dev(x), kc, vc, dev(slots), dev(np.zeros(3, np.int32)),
                      dev(np.zeros(64, np.float32)))
    for i, s in enumerate(slots.tolist()):
        for c in (kc, vc):
            assert np.array_equal(c.view(-1, d)[s].cpu().numpy(), x[i, 0].astype(np.float16))
        assert torch.equal(kc.view(-1, d)[s - 1].view(torch.int16), near[i].view(torch.int16))


def test_bindings_refuse(w4):
    x = torch.zeros((4, 2, 16), device="cuda")
    pos, freq = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(8, device="cuda")
    kc, vc = make_cache(2, 2, 4, 16, torch.float16, "phtd", 0)
    slots = torch.arange(4, device="cuda")
    ok = dict(k=x, v=x, k_cache=kc, v_cache=vc, slots=slots, positions=pos, freq=freq)
    w4.kv_append_rope(**ok)
    for bad in (dict(k=x.double()), dict(v=x.half()), dict(k=x.cpu()), dict(slots=slots.int()), dict(freq=freq.half()),
                dict(positions=pos.long()), dict(k_cache=kc.float()), dict(v_cache=vc.bfloat16()), dict(k=None)):
        with pytest.raises((TypeError, ValueError)):
            w4.kv_append_rope(**{**ok, **bad})
    for bad in (dict(k=x[:3]), dict(v=x[:, :1]), dict(slots=slots[:3]), dict(positions=pos[::2]),
                dict(k_scale=torch.ones(2, device="cuda")), dict(q=x[:3]), dict(q_out=x.half()),
                dict(q=x, q_out=torch.zeros((4, 2, 16), device="cuda")[:, :1].half()), dict(v_cache=vc[:, :, :2]),
                dict(k=x.transpose(1, 2).contiguous().transpose(1, 2)), dict(v_cache=vc.transpose(2, 3).contiguous().transpose(2, 3))):
        with pytest.raises(ValueError):
            w4.kv_append_rope(**{**ok, **bad})
    with pytest.raises(w4.W4Error):
        w4.kv_append_rope(**{**ok, "freq": torch.zeros(9, device="cuda")})  # more pairs than the head has
    with pytest.raises(ValueError):
        w4.rope_f16(x, pos, freq, out=torch.empty((4, 2, 8), dtype=torch.float16, device="cuda"))
    with pytest.raises(TypeError):
        w4.rope_f16(x, pos, freq, out=torch.empty((4, 2, 16), device="cuda"))
    with pytest.raises(w4.W4Error):
        w4.rope_f16(torch.zeros((4, 2, 12), device="cuda"), pos, freq[:4])
    with pytest.raises(w4.W4Error):
        w4.rope_f16(x[:, :, :], pos, torch.zeros(9, device="cuda"))
