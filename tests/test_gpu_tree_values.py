"""attention_paged_tree where scores, weights and values are at the ends of their ranges, in each of its kernels; the new tokens
are chains, so that row i sees what attention_paged's does.  Bounds as in test_gpu_attention_edges.py, whose cases these are."""

from __future__ import annotations

import numpy as np
import pytest

import int4_weight_only_group_amd as binding

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_attention import dev, w4  # noqa: E402, F401
from test_gpu_attention_edges import _cache_of, _one_dim  # noqa: E402
from test_gpu_tree_attention import Tree  # noqa: E402


def chain(t):
    return binding.tree_mask(range(-1, t - 1))[0].cuda()


def _attend(w4, q, caches, table, n, **kw):  # noqa: F811
    return w4.attention_paged_tree(dev(q), *caches, table, torch.tensor([n], dtype=torch.int32, device="cuda"), chain(len(q)),
                                   q_start=torch.tensor([0, len(q)], dtype=torch.int32, device="cuda"), max_q=len(q),
                                   **kw).cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("t,n,d", [(4, 131072, 64), (20, 131072, 64), (60, 131072, 64), (20, 131072, 128), (20, 131072, 256),
                                   (20, 900, 64), (20, 900, 128), (20, 900, 256), (40, 900, 64), (40, 900, 128), (40, 900, 256)])
@pytest.mark.parametrize("below", [11.5, 20.0])
def test_many_small_weights_beside_a_large_one(w4, t, n, below, d):  # noqa: F811
    rng = np.random.default_rng(t + n)
    at = n // 3
    s = np.round(rng.uniform(-1.0, 1.0, n) * 256) / 256
    s[at] = round((below + 1) * 16) / 16
    q, k = _one_dim(2.0, s, t, 2, d)
    v = (rng.uniform(0.5, 2.0, (n, d)) * 4096).astype(np.float16)
    v[at] = 0
    got = _attend(w4, q, *_cache_of(k, v), n, scale=1.0)
    s64 = 2.0 * k[:, 0].astype(np.float64)
    w = np.exp(s64 - s64[at])
    sums, total = np.cumsum(w[:, None] * v.astype(np.float64), 0), np.cumsum(w)
    for i in range(t):
        p = n - t + i
        want = sums[p] / total[p]
        rel = 2.0 ** -11 + 2.0 ** -11 + 2 * 3 * 2.0 ** -24 * s64[at] * 2 + 2.0 ** -20 + (n / 16 + 32) * 2.0 ** -23
        assert (np.abs(got[i] - want) <= want * rel + n * 2.0 ** -36 * v.max().astype(np.float64) + 2.0 ** -25).all(), i


@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
@pytest.mark.parametrize("scale", [1.0, 1e4, 1e20, 1e30])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_scores_far_from_zero(w4, scale, order, d):  # noqa: F811
    q0 = np.array([1 / 64, 1.0, 32768.0, -32768.0])
    for t, n in ((3, 1500), (5, 40), (12, 900), (16, 2000), (24, 900), (40, 1000)):
        rng = np.random.default_rng(n)
        ints = rng.permutation(np.arange(1, n + 1))
        ints = {"rising": np.sort(ints), "falling": np.sort(ints)[::-1], "mixed": ints}[order]
        q, k = np.zeros((t, 4, d), dtype=np.float16), np.zeros((n, d), dtype=np.float16)
        q[:, :, 0], k[:, 0] = q0, ints
        v = rng.standard_normal((n, d)).astype(np.float16)
        got = _attend(w4, q, *_cache_of(k, v), n, scale=scale)
        for i in range(t):
            seen = n - t + i + 1
            s = np.outer(q0, ints[:seen].astype(np.float64)) * scale
            two = np.sort(s, 1)[:, -2:]
            w = np.exp(s - s.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            v64 = v[:seen].astype(np.float64)
            want, size = w @ v64, w @ np.abs(v64)
            off = np.where(two[:, 1] - two[:, 0] > 100, 0.0, 6 * 2.0 ** -24 * np.abs(s).max(1))[:, None]
            bound = np.abs(want) * 2.0 ** -11 + 2.0 ** -25 + size * (
                2.0 ** -11 + 2 * off + 2.0 ** -20 + (n / 16 + 32) * 2.0 ** -23) + n * 2.0 ** -36 * np.abs(v64).max()
            err = np.abs(got[i] - want)
            assert (err <= bound).all(), (t, n, i, (err / bound).max(1))


@pytest.mark.parametrize("lens,d", [([(5, 9), (4, 700)], 64), ([(20, 300), (12, 41)], 64), ([(20, 5000)], 128), ([(30, 400)], 256),
                                    ([(16, 16), (9, 90)], 256), ([(150, 400)], 128)])
def test_rows_whose_scores_are_all_minus_infinity(w4, lens, d):  # noqa: F811
    for ends in (lambda n, kv: kv, lambda n, kv: kv - n // 2 - 1):
        s = Tree(lens, 4, 2, d, 16, seed=d, kind="chain")
        s.q = np.abs(s.q) + np.float16(0.125)
        want = np.full((s.q.shape[0], 4, d), np.nan)
        for b, (n, kv) in enumerate(lens):
            for j in range(kv):
                s.host[0][s.table[b, j // 16], :, j % 16, 0] = -np.inf
            j = ends(n, kv)
            if j < kv:
                s.host[0][s.table[b, j // 16], :, j % 16, 0] = 1
                v = s.host[1][s.table[b, j // 16], :, j % 16].astype(np.float64)
                rows = np.arange(n)[kv - n + np.arange(n) >= j] + s.starts[b]
                want[rows] = np.repeat(v, 2, 0)
        s.dev = [s._place(c, "phtd") for c in s.host]
        got = s.run(w4).cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert (np.abs(got - want) <= np.abs(want) * 2.0 ** -10)[~np.isnan(want)].all()


@pytest.mark.parametrize("lens,d", [([(7, 1500)], 64), ([(20, 3000)], 64), ([(24, 3000)], 128), ([(12, 3000)], 256), ([(90, 1500)], 128)])
def test_growing_maxima(w4, lens, d):  # noqa: F811
    # scores that rise along the keys: the running maximum moves in every block
    s = Tree(lens, 2, 1, d, 16, seed=6, kind="any")
    n = lens[0][1]
    s.q[:] = np.abs(s.q)
    for j in range(n):
        s.host[0][s.table[0, j // 16], 0, j % 16] = np.float16(j * 6.0 / n) * np.ones(d, dtype=np.float16)
    s.dev[0] = dev(s.host[0])
    s.check(s.run(w4))
    s.check(s.run(w4, window=700), window=700)


@pytest.mark.parametrize("lens", [[(6, 300), (1, 1)], [(24, 1200)], [(24, 400), (20, 21)], [(200, 700)]])
def test_scales_of_the_cache_far_from_one(w4, lens):  # noqa: F811
    for scale, k_scale in ((1e-20, 1e20 / 300), (1e20, 1e-20 / 300), (1e-30, 1e-20), (1e-30, 1e-38), (1e-30, 1e-45), (1.0, 1e-45)):
        s = Tree(lens, 4, 2, 128, 16, True, seed=3)
        s.scale_k = np.full(2, k_scale, dtype=np.float32)
        s.check(s.run(w4, scale=scale), scale=scale)
        s.check(s.run(w4, scale=scale, window=240), scale=scale, window=240)


@pytest.mark.parametrize("new", [9, 24, 40, 100])
def test_infinite_values_at_seen_keys(w4, new):  # noqa: F811
    # V infinite at one new key, K finite: +-inf in the rows that see it, both signs NaN
    s = Tree([(new, new + 160)], 2, 1, 64, 16, seed=9, kind="chain")
    a, b = 160 + new // 4, 160 + new // 2
    for j, val in ((a, np.inf), (b, -np.inf)):
        s.host[1][s.table[0, j // 16], 0, j % 16, :] = np.float16(val)
    s.dev = [s._place(c, "phtd") for c in s.host]
    got = s.run(w4).cpu().numpy()
    p = 160 + np.arange(new)
    assert np.isfinite(got[p < a]).all()
    assert (got[(p >= a) & (p < b)] == np.inf).all()
    assert np.isnan(got[p >= b]).all()


def test_far_offsets(w4):  # noqa: F811
    # pages past 2^32 elements of the cache
    pages, page, d = 2100, 16384, 128
    kc = torch.empty((pages, 1, page, d), dtype=torch.float16, device="cuda")
    vc = torch.empty_like(kc)
    for new in (5, 25, 90):
        n = 100
        s = Tree([(new, n)], 2, 1, d, 128, seed=15)
        for c, h in ((kc, s.host[0]), (vc, s.host[1])):
            c[pages - 1, 0, :n] = dev(h[s.table[0, 0], 0, :n])
        got = w4.attention_paged_tree(dev(s.q), kc, vc, torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda"),
                                      dev(s.kv_len), s.mask[:, :s.words], q_start=dev(s.starts), max_q=new)
        s.check(got)
