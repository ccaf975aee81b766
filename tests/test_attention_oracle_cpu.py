"""The oracle of the rotary positions, the paged cache and the attention, pinned by closed forms
(CPU), and the frequencies of long contexts."""

from __future__ import annotations

import math

import numpy as np
import pytest

from oracle import attnref as ref


def test_rope_is_a_complex_product():
    rng = np.random.default_rng(0)
    x, pos = rng.standard_normal((5, 2, 12)), np.array([0, 1, 7, 1000, 123456])
    freq = np.array([1.0, 0.25, 1e-3])
    for inter in (False, True):
        y = ref.rope(x, pos, freq, interleaved=inter, mscale=1.5)
        a, b = (x[..., 0:6:2], x[..., 1:6:2]) if inter else (x[..., :3], x[..., 3:6])
        z = (a + 1j * b) * 1.5 * np.exp(1j * pos[:, None, None] * freq)
        got = (y[..., 0:6:2] + 1j * y[..., 1:6:2]) if inter else (y[..., :3] + 1j * y[..., 3:6])
        assert np.allclose(got, z, atol=1e-12)
        assert np.array_equal(y[..., 6:], x[..., 6:])
        back = ref.rope(y, pos, freq, interleaved=inter, inverse=True)
        assert np.allclose(back[..., :6], 1.5 * x[..., :6], atol=1e-12)


def test_rope_quarter_turn_and_scores_depend_on_distance():
    x = np.array([[[3.0, 4.0]]])
    assert np.allclose(ref.rope(x, [1], [math.pi / 2]), [[[-4.0, 3.0]]])
    rng = np.random.default_rng(1)
    q, k, f = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8)), np.array([1, .3, .1, .01])
    dots = [(ref.rope(q, [m + 5], f) * ref.rope(k, [m], f)).sum() for m in (0, 3, 900)]
    assert np.allclose(dots, dots[0])


def test_e4m3_table_and_rounding():
    v = ref.e4m3_values()
    assert v[0x08] == 2.0 ** -6 and v[0x01] == 2.0 ** -9 and v[0x7E] == 448 and np.isnan(v[0x7F])
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)
    assert np.array_equal(ref.e4m3_round(v[codes]), codes)
    # 17 is half way between 16 and 18: the even code (16); 19 between 18 and 20: 20
    assert v[ref.e4m3_round([17.0, 19.0, -17.0, 500.0, -1e9, 2.0 ** -10, 3 * 2.0 ** -10])].tolist() == [
        16.0, 20.0, -16.0, 448.0, -448.0, 0.0, 2.0 ** -8]
    assert np.isnan(v[ref.e4m3_round(np.nan)])


def test_attention_by_hand():
    ln3 = math.log(3.0)
    k = np.zeros((2, 1, 2, 8))
    v = np.zeros((2, 1, 2, 8))
    k[1, 0, 0, 0], k[1, 0, 1, 0], k[0, 0, 0, 0] = 0.0, ln3, np.nan  # page 0 token 0 is past the end
    v[1, 0, 0, 0], v[1, 0, 1, 0], v[0, 0, 0, 0] = 4.0, 8.0, np.inf
    q = np.zeros((2, 1, 8))
    q[:, 0, 0] = 2.0
    out, size, _ = ref.attention(q, k, v, np.array([[1, 0]]), [2], [0, 2], scale=0.5)
    assert np.allclose(out[:, 0, 0], [4.0, 0.25 * 4 + 0.75 * 8])
    assert np.allclose(size, out)
    one, _, _ = ref.attention(q, k, v, np.array([[1, 0]]), [2], [0, 2], scale=0.5, window=1)
    assert np.allclose(one[:, 0, 0], [4.0, 8.0])
    # more rows than cached tokens: the first sees nothing; no cached token: none does
    short, _, _ = ref.attention(q, k, v, np.array([[1, 0]]), [1], [0, 2], scale=0.5)
    assert np.array_equal(short[0], np.zeros((1, 8))) and short[1, 0, 0] == 4.0
    none, _, _ = ref.attention(q, k, v, np.array([[1, 0]]), [0], [0, 2], scale=0.5)
    assert np.array_equal(none, np.zeros((2, 1, 8)))


def test_attention_heads_share_a_kv_head_and_scales():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((3, 4, 8)), rng.standard_normal((3, 2, 4, 8)), rng.standard_normal((3, 2, 4, 8))
    tab = np.array([[2, 0]])
    out, _, _ = ref.attention(q, k, v, tab, [7], [0, 3], scale=0.3, k_scale=[2.0, 3.0], v_scale=[0.5, 4.0])
    for h in range(4):
        kk = np.concatenate([k[2, h // 2], k[0, h // 2]])[:7] * [2.0, 3.0][h // 2]
        vv = np.concatenate([v[2, h // 2], v[0, h // 2]])[:7] * [0.5, 4.0][h // 2]
        for i in range(3):
            e = np.exp(0.3 * kk[:5 + i] @ q[i, h])
            assert np.allclose(out[i, h], e @ vv[:5 + i] / e.sum())


def test_rope_frequencies():
    import torch
    import int4_weight_only_group_amd as w4
    f, m = w4.rope_frequencies(8, 10000.0, device="cpu")
    assert f.dtype == torch.float32 and m == 1.0
    assert np.allclose(f.numpy(), [1.0, 0.1, 0.01, 0.001], rtol=1e-7)
    f, m = w4.rope_frequencies(8, 10000.0, scaling="linear", factor=4.0, device="cpu")
    assert np.allclose(f.numpy(), np.array([1.0, 0.1, 0.01, 0.001]) / 4, rtol=1e-7) and m == 1.0
    f, _ = w4.rope_frequencies(8, 10000.0, scaling="ntk", factor=4.0, device="cpu")
    assert math.isclose(f[0], 1.0) and math.isclose(f[3], 0.001 / 4, rel_tol=1e-6)
    f, m = w4.rope_frequencies(128, 1e6, scaling="yarn", factor=4.0, original=32768, device="cpu")
    g, _ = w4.rope_frequencies(128, 1e6, device="cpu")
    turns = 32768 * g.double().numpy() / (2 * math.pi)
    ratio = (g / f).numpy()
    assert np.allclose(ratio[turns > 40], 1.0) and np.allclose(ratio[turns < 0.8], 4.0)
    assert (np.diff(ratio) >= -1e-5).all() and math.isclose(m, 0.1 * math.log(4) + 1)
    assert w4.rope_frequencies(0, device="cpu")[0].numel() == 0
    for bad in (dict(rot=7), dict(rot=8, base=1.0), dict(rot=8, factor=0.5), dict(rot=8, scaling="cubic"),
                dict(rot=8, scaling="yarn", factor=2.0), dict(rot=2, scaling="ntk", factor=2.0)):
        with pytest.raises(ValueError):
            w4.rope_frequencies(device="cpu", **bad)
