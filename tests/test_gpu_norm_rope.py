"""norm_rope_f16 and kv_append_norm_rope against the fp64 oracle.

Bounds, per output: those of test_gpu_rope_append.py with the normed values in the place of x, and the norm's own f32 roundings
on top, relative to what is rotated: D squares and their sums (D + 2 roundings, each at most a half of the sum's relative error
after the root), mean, eps, root and quotient (4), the two products (2): (D / 2 + 8) * 2^-24 of |a| + |b|.
"""

from __future__ import annotations

import numpy as np
import pytest

from oracle import attnref as ref
from oracle import stepref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_rope_append import dev, inputs, pair_size, w4  # noqa: E402, F401


def sizes(y, r, inter, mscale):
    """(|a| + |b|) * mscale of an element's pair, |a| where it is passed on"""
    s = pair_size(y, r, inter, mscale)
    s[..., r:] = np.abs(y[..., r:])
    return s


def slack(d):
    return 2.0 ** -20 + (d / 2 + 8) * 2.0 ** -24


def close_f16(got, want, size):
    bound = np.abs(want) * 2.0 ** -11 + 2.0 ** -25 + size * slack(got.shape[-1])
    err = np.abs(got.astype(np.float64) - want)
    assert (err <= bound).all(), (err / bound).max()


def close_e4m3(codes, want, size, scale):
    y = np.clip(want / scale, -448, 448)
    bound = np.abs(y) * (2.0 ** -4 + 2.0 ** -22) + 2.0 ** -10 + size / scale * slack(codes.shape[-1])
    err = np.abs(ref.e4m3_values()[codes] - y)
    assert (err <= bound).all(), (err / bound).max()


CASES = [  # tokens, heads, dim, rot, interleaved, f32, mscale
    (1, 1, 8, 8, False, True, 1.0), (1, 16, 128, 128, False, True, 1.0), (3, 5, 128, 128, True, False, 1.25),
    (64, 16, 128, 128, False, False, 1.0), (7, 2, 80, 32, True, True, 1.0), (7, 2, 80, 32, False, True, 1.0),
    (5, 3, 64, 0, False, True, 1.0), (5, 3, 64, 0, True, False, 1.0), (9, 2, 96, 58, False, True, 1.5),
    (9, 2, 96, 58, True, True, 1.5), (33, 7, 256, 256, False, True, 1.0), (33, 7, 256, 254, False, False, 1.0),
    (33, 7, 256, 256, True, True, 1.0), (33, 7, 256, 16, False, True, 1.0), (257, 4, 24, 6, True, True, 1.0),
    (2600, 2, 64, 64, False, True, 0.75), (4099, 3, 80, 32, True, False, 1.0), (2, 40, 72, 2, False, False, 1.0),
    (13, 18, 128, 48, False, False, 1.0), (2, 1024, 16, 16, False, True, 1.0), (2, 1024, 16, 6, False, True, 1.0),
    (5, 1, 8, 4, False, False, 1.0), (5, 1, 8, 4, True, False, 1.0), (6, 3, 248, 240, False, True, 1.0),
    (2100, 5, 16, 16, True, True, 1.0),
]


@pytest.mark.parametrize("t,h,d,r,inter,f32,ms", CASES)
def test_norm_rope(w4, t, h, d, r, inter, f32, ms):  # noqa: F811
    x, pos, freq = inputs(t, h, d, r, f32, t + h + d)
    rng = np.random.default_rng(t)
    x = (x * rng.uniform(0.01, 20.0, (t, h, 1))).astype(x.dtype)
    weight = rng.standard_normal(d).astype(np.float32)
    for w in (weight, None):
        y = w4.norm_rope_f16(dev(x), None if w is None else dev(w), dev(pos), dev(freq), eps=1e-5, interleaved=inter,
                             mscale=ms).cpu().numpy()
        n = stepref.norm(x, w, 1e-5)
        close_f16(y, ref.rope(n, pos, freq, interleaved=inter, mscale=ms), sizes(n, r, inter, ms))


@pytest.mark.parametrize("r,inter", [(128, False), (128, True), (58, False), (32, False)])
def test_small_zero_and_odd_rows(w4, r, inter):  # noqa: F811
    # heads of zeros are zeros; of tiny values eps decides; a NaN stays in its own head
    x, pos, freq = inputs(5, 3, 128, r, True, 2)
    x[1, 1] = 0
    x[2] *= 1e-12
    x[3, 0, 7] = np.nan
    x[4] *= 1e15
    y = w4.norm_rope_f16(dev(x), None, dev(pos), dev(freq), eps=1e-6, interleaved=inter).cpu().numpy()
    assert (y[1, 1] == 0).all()
    assert np.isnan(y[3, 0]).all() and np.isfinite(y[3, 1:]).all()
    n = stepref.norm(x, None, 1e-6)
    want, size = ref.rope(n, pos, freq, interleaved=inter), sizes(n, r, inter, 1.0)
    keep = np.array([0, 1, 2, 4])
    close_f16(y[keep], want[keep], size[keep])


@pytest.mark.parametrize("r,inter", [(128, False), (128, True), (58, False), (32, False), (32, True), (0, False)])
def test_in_place_and_strided_rows(w4, r, inter):  # noqa: F811
    x, pos, freq = inputs(19, 3, 128, r, False, r)
    weight = dev(np.random.default_rng(r).standard_normal(128).astype(np.float32))
    want = w4.norm_rope_f16(dev(x), weight, dev(pos), dev(freq), interleaved=inter)
    rows = torch.full((19, 9, 128), 7.0, dtype=torch.float16, device="cuda")
    rows[:, 2:5] = dev(x)
    part = rows[:, 2:5]
    w4.norm_rope_f16(part, weight, dev(pos), dev(freq), interleaved=inter, out=part)
    assert torch.equal(part, want)
    assert (rows[:, :2] == 7).all() and (rows[:, 5:] == 7).all()


APPEND = [  # tokens, hq, hkv, dim, rot, interleaved, f32, mscale, e4m3, page
    (1, 16, 2, 128, 128, False, True, 1.0, False, 16), (1, 16, 8, 128, 128, False, True, 1.0, False, 16),
    (64, 16, 8, 256, 256, False, True, 1.0, True, 64), (33, 7, 1, 96, 58, False, False, 1.25, False, 5),
    (33, 7, 1, 96, 58, True, True, 1.25, True, 5), (9, 0, 3, 80, 32, False, True, 1.0, False, 8),
    (9, 0, 3, 80, 30, False, True, 1.0, True, 8), (300, 4, 2, 64, 64, True, False, 1.0, False, 16),
    (2500, 2, 1, 16, 16, False, True, 1.0, True, 16), (5, 3, 3, 24, 24, False, False, 1.0, False, 3),
]


@pytest.mark.parametrize("t,hq,hkv,d,r,inter,f32,ms,e4m3,page", APPEND)
def test_append(w4, t, hq, hkv, d, r, inter, f32, ms, e4m3, page):  # noqa: F811
    x, pos, freq = inputs(t, hq + 2 * hkv, d, r, f32, t + d)
    rng = np.random.default_rng(d)
    wq, wk = rng.standard_normal((2, d)).astype(np.float32)
    pages = -(-t // page) + 3
    slots = rng.permutation(pages * page)[:t].astype(np.int64)
    skipped = np.zeros(t, dtype=bool)
    skipped[t // 2::5] = t > 4
    given = np.where(skipped, rng.choice([-1, pages * page, -2 ** 62, 2 ** 62], t), slots)
    rows = dev(x)
    if e4m3:
        before = rng.integers(0, 127, (2, pages, hkv, page, d)).astype(np.uint8)
        scales = (rng.random((2, hkv)) * 0.02 + 0.01).astype(np.float32)
        kc, vc = (dev(c).view(torch.float8_e4m3fn) for c in before)
        kw = dict(k_scale=dev(scales[0]), v_scale=dev(scales[1]))
    else:
        before = rng.standard_normal((2, pages, hkv, page, d)).astype(np.float16)
        kc, vc = dev(before[0]), dev(before[1])
        kw = {}
    q = w4.kv_append_norm_rope(rows[:, hq:hq + hkv], rows[:, hq + hkv:], kc, vc, dev(given), dev(pos), dev(freq), dev(wk),
                               q=rows[:, :hq] if hq else None, q_weight=dev(wq) if hq else None, eps=1e-6,
                               interleaved=inter, mscale=ms, **kw)
    if hq:
        n = stepref.norm(x[:, :hq], wq, 1e-6)
        close_f16(q.cpu().numpy(), ref.rope(n, pos, freq, interleaved=inter, mscale=ms), sizes(n, r, inter, ms))
    else:
        assert q is None
    n = stepref.norm(x[:, hq:hq + hkv], wk, 1e-6)
    for i, (c, want, size) in enumerate(((kc, ref.rope(n, pos, freq, interleaved=inter, mscale=ms), sizes(n, r, inter, ms)),
                                         (vc, x[:, hq + hkv:].astype(np.float64), np.zeros((t, hkv, d))))):
        got = (c.view(torch.uint8) if e4m3 else c).cpu().numpy().transpose(0, 2, 1, 3).reshape(-1, hkv, d)
        old = before[i].transpose(0, 2, 1, 3).reshape(-1, hkv, d)
        at = slots[~skipped]
        if e4m3:
            close_e4m3(got[at], want[~skipped], size[~skipped], scales[i][None, :, None])
        else:
            close_f16(got[at], want[~skipped], size[~skipped])
        rest = np.setdiff1d(np.arange(pages * page), at)
        assert np.array_equal(got[rest].view(np.uint8), old[rest].view(np.uint8))


def test_norms_with_no_weights_are_weights_of_one(w4):  # noqa: F811
    x, pos, freq = inputs(6, 8, 64, 64, True, 4)
    rows, ones = dev(x), torch.ones(64, device="cuda")
    out = []
    for w in (None, ones):
        kc, vc = (torch.zeros((2, 2, 4, 64), dtype=torch.float16, device="cuda") for _ in range(2))
        q = w4.kv_append_norm_rope(rows[:, 4:6], rows[:, 6:], kc, vc, torch.arange(6, device="cuda"), dev(pos), dev(freq),
                                   w, q=rows[:, :4], q_weight=w)
        out.append((q, kc, vc))
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_bindings_refuse(w4):  # noqa: F811
    x, pos, freq = inputs(4, 2, 64, 64, True, 5)
    w = torch.ones(64, device="cuda")
    ok = dict(x=dev(x), weight=w, positions=dev(pos), freq=dev(freq))
    w4.norm_rope_f16(**ok)
    for bad in (dict(weight=w[:32]), dict(weight=torch.ones(128, device="cuda")[::2]), dict(positions=dev(pos)[:3]),
                dict(x=dev(x)[:, :, :32]), dict(weight=w.half()), dict(weight=w.cpu()), dict(x=None)):
        with pytest.raises((TypeError, ValueError)):
            w4.norm_rope_f16(**{**ok, **bad})
    for bad in (dict(eps=0.0), dict(eps=float("nan")), dict(weight=torch.ones(65, device="cuda")[1:])):
        with pytest.raises(w4.W4Error):
            w4.norm_rope_f16(**{**ok, **bad})
