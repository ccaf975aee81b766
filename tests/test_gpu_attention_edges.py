"""attention_paged where its definition ends: rows that see nothing in tiles of their own, scores and weights at the
ends of their ranges, workspaces that hold anything, captured calls whose keys are dealt out anew at each replay.
Bounds as in test_gpu_attention.py unless stated."""

from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_attention import Setup, dev, w4  # noqa: E402, F401


@pytest.mark.parametrize("page", [16, 64, 12])
@pytest.mark.parametrize("hq,hkv,d,e4m3", [(2, 1, 64, False), (4, 2, 64, True), (16, 2, 128, False), (2, 1, 128, True),
                                           (2, 1, 256, False), (16, 2, 256, True), (4, 2, 96, False)])
def test_row_tiles_that_see_no_key(w4, hq, hkv, d, e4m3, page):  # noqa: F811
    # more new tokens than cached ones, so that the first tiles of 64 or 128 rows see nothing; no cached tokens at all;
    # alone, beside others, with tables that are split in parts
    for lens, window in (([(200, 0)], 0), ([(300, 20)], 0), ([(300, 1)], 5), ([(150, 60), (150, 2000), (90, 0)], 0),
                         ([(1, 5), (260, 0), (2, 0), (140, 200), (130, 7)], 33), ([(700, 0), (650, 700)], 0)):
        s = Setup(lens, hq, hkv, d, page, e4m3, seed=d + page)
        print(lens, window, flush=True)
        s.check(s.run(w4, window=window), window=window)


def _cache_of(k, v, page=16):
    # [keys][dim] of one kv head as caches of whole pages, and their table, pages in another order
    n, d = k.shape
    order = np.random.default_rng(n).permutation(-(-n // page))
    caches = []
    for x in (k, v):
        c = np.zeros((len(order) * page, d), dtype=np.float16)
        c[:n] = x
        y = np.empty((len(order), 1, page, d), dtype=np.float16)
        y[order, 0] = c.reshape(-1, page, d)
        caches.append(dev(y))
    return caches, dev(order[None].astype(np.int32))


def _attend(w4, q, caches, table, n, **kw):  # noqa: F811
    return w4.attention_paged(dev(q), *caches, table, torch.tensor([n], dtype=torch.int32, device="cuda"),
                              q_start=torch.tensor([0, len(q)], dtype=torch.int32, device="cuda"), max_q=len(q),
                              **kw).cpu().numpy().astype(np.float64)


def _one_dim(q0, s, t, hq, d=64):
    # q and k of one nonzero dim, so that a score is one exact product: every key's is s[key], for rows of q0
    q, k = np.zeros((t, hq, d), dtype=np.float16), np.zeros((len(s), d), dtype=np.float16)
    q[:, :, 0], k[:, 0] = q0, np.asarray(s) / q0
    return q, k


@pytest.mark.parametrize("t,n", [(1, 131072), (3, 131072), (40, 131072), (300, 131072), (1, 300), (5, 900), (90, 900)])
@pytest.mark.parametrize("below", [11.5, 17.4, 20.0])
def test_many_small_weights_beside_a_large_one(w4, t, n, below):  # noqa: F811
    # one key, whose value is 0, has nearly all the weight; the others lie `below` nats under it and make up the result.
    # The first row (of the last position all rows see all keys but the last t) sees n - t + 1 keys.
    # Bound, relative to the result: weights to f16, 2^-11 each, or to half of f16's smallest step, 2^-25, which is 2^-36 of
    # the largest weight, 2^11; the result to f16, 2^-11 or 2^-25; scores exact but for three roundings of 2^-24 * |s| in
    # their product with scale * log2 e; exp2 2^-20; sums in f32, 2^-23 a block of 16 keys and 32 more.
    rng = np.random.default_rng(t + n)
    at = n // 3
    s = np.round(rng.uniform(-1.0, 1.0, n) * 256) / 256  # exact in f16, as are their halves
    s[at] = round((below + 1) * 16) / 16
    q, k = _one_dim(2.0, s, t, 2)
    v = (rng.uniform(0.5, 2.0, (n, 64)) * 4096).astype(np.float16)
    v[at] = 0
    got = _attend(w4, q, *_cache_of(k, v), n, scale=1.0)
    s64 = 2.0 * k[:, 0].astype(np.float64)
    w = np.exp(s64 - s64[at])
    sums, total = np.cumsum(w[:, None] * v.astype(np.float64), 0), np.cumsum(w)
    for i in range(t):
        p = n - t + i
        want = sums[p] / total[p]
        rel = 2.0 ** -11 + 2.0 ** -11 + 2 * 3 * 2.0 ** -24 * s64[at] * 2 + 2.0 ** -20 + (n / 16 + 32) * 2.0 ** -23
        assert (np.abs(got[i] - want) <= want * rel + n * 2.0 ** -36 * v.max().astype(np.float64) + 2.0 ** -25).all(), (i, np.abs(got[i] / want - 1).max())


@pytest.mark.parametrize("n", [256, 5000])
def test_few_rows_weigh_to_22_bits(w4, n):  # noqa: F811
    # Two kinds of keys in turn, of weights 1 and x and values 1 and about -1 / x, so that they cancel: what is left is
    # the weights' rounding, at the scale of 1.  One f16 a weight is off by up to 2^-12 of it, which the bound
    # refuses for these x; two are off by 2^-22.  The scores' errors are two roundings of 2^-24 * |s| log2 e < 3.
    for below in (0.3, 0.71, 1.37, 1.9):
        s = np.zeros(n)
        s[1::2] = -np.float64(np.float16(below))
        q, k = _one_dim(1.0, s, 1, 4)
        s64 = k[:, 0].astype(np.float64)
        w = np.exp(s64)
        v = np.ones((n, 64), dtype=np.float16)
        v[1::2] = -np.float16(1 / w[1])
        total = w.sum()
        want = float((w * v[:, 0].astype(np.float64)).sum() / total)
        size = float((w * np.abs(v[:, 0].astype(np.float64))).sum() / total)
        bound = abs(want) * 2.0 ** -11 + 2.0 ** -25 + size * (2.0 ** -21 + 6 * 2.0 ** -23 + 2.0 ** -20 + (n / 16 + 32) * 2.0 ** -23)
        one = np.float64(np.float16(w[1]))  # up to a power of two, the kernel's x in one f16
        off = abs(((w[::2] * v[::2, 0]).sum() + (one * v[1::2, 0].astype(np.float64)).sum()) / (w[::2].sum() + one * (n // 2)) - want)
        if n == 256:
            assert off > 2 * bound, (off, bound)  # the test tells one f16 from two
        got = _attend(w4, q, *_cache_of(k, v), n, scale=1.0)
        assert (np.abs(got - want) <= bound).all(), (below, np.abs(got - want).max(), bound)


@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
@pytest.mark.parametrize("scale", [1.0, 1e4, 1e20, 1e30])
def test_scores_far_from_zero(w4, scale, order):  # noqa: F811
    # Integer keys on one dim, so that a product q . k is exact; the rows of four heads multiply them by 1/64, 1, 32768 and
    # -32768: rows beside each other with scores of up to 2^26 * scale, all of one sign, and small ones.
    # Bound: the result and the weights to f16; a weight is off by 6 * 2^-24 of the largest score in nats, unless the
    # next one lies more than 100 nats below the largest (then all of the weight is its own).
    q0 = np.array([1 / 64, 1.0, 32768.0, -32768.0])
    for t, n in ((1, 40), (1, 1500), (4, 900), (90, 900), (300, 2000)):
        rng = np.random.default_rng(n)
        ints = rng.permutation(np.arange(1, n + 1))
        ints = {"rising": np.sort(ints), "falling": np.sort(ints)[::-1], "mixed": ints}[order]
        q, k = np.zeros((t, 4, 64), dtype=np.float16), np.zeros((n, 64), dtype=np.float16)
        q[:, :, 0], k[:, 0] = q0, ints
        v = rng.standard_normal((n, 64)).astype(np.float16)
        got = _attend(w4, q, *_cache_of(k, v), n, scale=scale)
        for i in range(t):
            seen = n - t + i + 1
            s = np.outer(q0, ints[:seen].astype(np.float64)) * scale
            two = np.sort(s, 1)[:, -2:] if seen > 1 else np.array([[-np.inf, 0]] * 4)
            w = np.exp(s - s.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            v64 = v[:seen].astype(np.float64)
            want, size = w @ v64, w @ np.abs(v64)
            off = np.where(two[:, 1] - two[:, 0] > 100, 0.0, 6 * 2.0 ** -24 * np.abs(s).max(1))[:, None]
            bound = np.abs(want) * 2.0 ** -11 + 2.0 ** -25 + size * (
                2.0 ** -11 + 2 * off + 2.0 ** -20 + (n / 16 + 32) * 2.0 ** -23) + n * 2.0 ** -36 * np.abs(v64).max()
            err = np.abs(got[i] - want)
            assert (err <= bound).all(), (t, n, i, (err / bound).max(1))


@pytest.mark.parametrize("lens,window", [([(1, 300), (1, 1)], 0), ([(5, 1200)], 33), ([(150, 400), (40, 41)], 0),
                                         ([(200, 700)], 100)])
def test_scales_of_the_cache_far_from_one(w4, lens, window):  # noqa: F811
    # the product of scale and k_scale, not each, is what a score takes: 1/300 from factors of 10^20; and down to nothing
    # (2^-149 * 1e-30), where all keys weigh the same
    for scale, k_scale in ((1e-20, 1e20 / 300), (1e20, 1e-20 / 300), (1e-30, 1e-20), (1e-30, 1e-38), (1e-30, 1e-45), (1.0, 1e-45)):
        s = Setup(lens, 4, 2, 128, 16, True, seed=3)
        s.scale_k = np.full(2, k_scale, dtype=np.float32)
        s.check(s.run(w4, scale=scale, window=window), scale=scale, window=window)


@pytest.mark.parametrize("lens,d", [([(1, 40), (1, 700)], 64), ([(1, 20000)], 128), ([(5, 9)], 64), ([(90, 300), (40, 41)], 128),
                                    ([(300, 2000)], 128), ([(150, 400)], 256)])
def test_rows_whose_scores_are_all_minus_infinity(w4, lens, d):  # noqa: F811
    # no softmax: NaN, not the 0 of a row that sees nothing; a row that sees one finite key has that key's value
    for ends in (lambda n, kv: kv, lambda n, kv: kv - n // 2 - 1):
        s = Setup(lens, 4, 2, d, 16, seed=d)
        s.q = np.abs(s.q) + np.float16(0.125)
        want = np.full((s.q.shape[0], 4, d), np.nan)
        for b, (n, kv) in enumerate(lens):
            for j in range(kv):
                s.host[0][s.table[b, j // 16], :, j % 16, 0] = -np.inf
            j = ends(n, kv)  # the one finite key, if the sequence has it
            if j < kv:
                s.host[0][s.table[b, j // 16], :, j % 16, 0] = 1
                v = s.host[1][s.table[b, j // 16], :, j % 16].astype(np.float64)
                rows = np.arange(n)[kv - n + np.arange(n) >= j] + s.starts[b]
                want[rows] = np.repeat(v, 2, 0)
        s.dev = [s._place(c, "phtd") for c in s.host]
        got = s.run(w4).cpu().numpy().astype(np.float64)
        # a weight of 2^11 (or what it is rounded to) over its own sum: the value to 2^-22, rounded to f16
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert (np.abs(got - want) <= np.abs(want) * 2.0 ** -10)[~np.isnan(want)].all()


def _workspace(w4, s, window, fill, max_q=None):  # noqa: F811
    # exactly the bytes that the call needs, filled, and 4096 more behind them that are not the call's
    need = w4.attention_workspace_bytes(s.dev[0], len(s.lens), s.q.shape[0], max_q or s.kw()["max_q"], s.hq,
                                        s.table.shape[1], window)
    ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device="cuda")
    return need, ws


@pytest.mark.parametrize("lens,hq,hkv,d,page,window,e4m3", [
    # single tokens: parts of one, of several sequences, of lengths 0 and 1 among long ones
    ([(1, 1570)], 16, 2, 128, 16, 0, False), ([(1, 5000), (1, 1), (1, 0), (1, 33)], 16, 2, 128, 100, 0, False),
    ([(1, 20011), (1, 3)], 2, 1, 64, 32, 0, True), ([(1, 3000), (1, 900)], 8, 4, 256, 16, 700, True),
    ([(1, 10 * i) for i in range(70)] + [(1, 9000)], 4, 1, 64, 16, 0, False),
    # rows of many tokens in few and in many parts, empty ones among them; both kinds together
    ([(8, 1000), (8, 300)], 16, 2, 128, 16, 0, False), ([(600, 2000)], 2, 1, 128, 16, 0, False),
    ([(200, 0), (3, 2000)], 4, 2, 64, 16, 0, False), ([(64, 6000)], 8, 1, 256, 16, 0, True),
    ([(3, 9000), (2, 100)], 8, 1, 128, 16, 0, False), ([(130, 640), (3, 70), (0, 5), (20, 4)], 8, 2, 256, 64, 0, False),
    ([(20, 2000), (1, 900), (1, 0)], 4, 2, 96, 5, 600, True),
])
def test_workspace_may_hold_anything(w4, lens, hq, hkv, d, page, window, e4m3):  # noqa: F811
    s = Setup(lens, hq, hkv, d, page, e4m3, seed=d + len(lens))
    first = None
    for fill in (0xFF, 0x00, 0x7F):  # NaN and -1; 0; 3.4e38
        need, ws = _workspace(w4, s, window, fill)
        assert need > 0  # parts are kept there
        got = s.run(w4, window=window, workspace=ws[:need])
        s.check(got, window=window)
        assert (ws[need:] == fill).all()
        first = got if first is None else first
        assert torch.equal(got, first)


def _replays(w4, s, steps, window=0):  # noqa: F811
    # two graphs of one call, which share a workspace, replayed while lengths and starts change; an eager call between
    need, ws = _workspace(w4, s, window, 0xFF)
    assert need > 0
    q, table, kv_len, starts = dev(s.q), dev(s.table), dev(s.kv_len), dev(s.starts)
    args = {**s.kw(), "q_start": starts}
    outs = [torch.empty_like(q) for _ in range(2)]

    def call(o, **kw):
        w4.attention_paged(q, *s.dev, table, kv_len, window=window, out=o, **args, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(outs[0], workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g, o in zip(graphs, outs):
        with torch.cuda.graph(g):
            call(o, workspace=ws)
    t = s.q.shape[0]
    for i, lens in enumerate(steps):
        s.lens = lens
        s.starts = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
        s.kv_len = np.array([kv for _, kv in lens], dtype=np.int32)
        kv_len.copy_(dev(s.kv_len))
        starts.copy_(dev(s.starts))
        for g, o in zip(graphs, outs):
            o.fill_(7.0)
            g.replay()
            torch.cuda.synchronize()
        eager = torch.full_like(q, 7.0)
        call(eager)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], eager) and torch.equal(outs[1], eager), i
        live = int(s.starts[-1])
        assert (eager[live:] == 7).all()
        whole, s.q = s.q, s.q[:live]
        if live:
            s.check(eager[:live], window=window)
        s.q = whole
    assert t == s.q.shape[0]


@pytest.mark.parametrize("hq,hkv,d,e4m3,window", [(4, 2, 64, False, 0), (16, 2, 128, True, 0), (2, 1, 256, False, 900)])
def test_captured_decode_replays_through_its_parts(w4, hq, hkv, d, e4m3, window):  # noqa: F811
    # of one part and of many, with nothing and with everything cached, and back
    s = Setup([(1, 3200), (1, 3200), (1, 3200)], hq, hkv, d, 16, e4m3, seed=d)
    _replays(w4, s, [[(1, a), (1, b), (1, c)] for a, b, c in (
        (30, 7, 1), (500, 1, 0), (3200, 0, 3200), (0, 0, 0), (1, 3200, 129), (128, 127, 256), (0, 1, 0), (2900, 3100, 40))], window)


@pytest.mark.parametrize("hq,hkv,d,e4m3,window", [(4, 2, 64, False, 0), (8, 4, 128, True, 0), (2, 1, 256, False, 900)])
@pytest.mark.parametrize("t", [100, 400])
def test_captured_batches_replay_through_their_parts(w4, t, hq, hkv, d, e4m3, window):  # noqa: F811
    # sequences of few rows and of many change places from replay to replay, and rows of no sequence are left
    s = Setup([(t, 3200), (0, 3200), (0, 3200)], hq, hkv, d, 16, e4m3, seed=d + t)
    _replays(w4, s, [
        [(t - 10, 3000), (5, 2000), (5, 5)], [(1, 3200), (t - 2, t - 2), (1, 0)], [(t, 3200), (0, 9), (0, 0)],
        [(t // 3, 20), (t // 3, 3200), (t // 4, 0)], [(0, 0), (0, 0), (0, 0)], [(2, 3000), (3, 1), (t - 5, 2900)],
        [(8, 64), (9, 3200), (1, 1)]], window)


@pytest.mark.parametrize("lens,hq,hkv,d,e4m3", [
    ([(1, 300), (1, 0), (1, 7000)], 16, 2, 128, False), ([(1, 200), (1, 9)], 8, 8, 64, True),
    ([(300, 300)], 16, 2, 128, False), ([(64, 6000)], 8, 1, 256, True), ([(130, 640), (3, 2000), (1, 5)], 8, 2, 64, False)])
def test_the_result_may_take_the_queries_place(w4, lens, hq, hkv, d, e4m3):  # noqa: F811
    s = Setup(lens, hq, hkv, d, 16, e4m3, seed=d)
    want = s.run(w4)
    rows = torch.full((s.q.shape[0], hq + 2, d), 5.0, device="cuda", dtype=torch.float16)
    q = rows[:, 1:hq + 1]
    q.copy_(dev(s.q))
    s.run(w4, q=q, out=q)
    assert torch.equal(q, want) and (rows[:, 0] == 5).all() and (rows[:, hq + 1] == 5).all()
