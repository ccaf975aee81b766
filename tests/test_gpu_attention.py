"""attention_paged against the fp64 oracle, element by element.

The bound of an output (size: the weighted mean of |v|; wobble: the largest sum_d |scale q_d k_d| of the row;
n: keys seen), counting roundings: the result to f16, 2^-11 of itself and 2^-25; the weights to f16, 2^-11 of size,
and 2^-25 * n * max|v| for those below f16's normal range (the largest weight is at least 1, so the sum is);
the scores in f32, dim + 8 roundings of 2^-24 * wobble each, which move a weight and the sum by as much: 2x; exp2 to
2^-21; the f32 sums over n keys in blocks of 16: (n / 16 + 32) * 2^-23 * size.
"""

from __future__ import annotations

import numpy as np
import pytest

import oracle
import synth
from oracle import attnref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import int4_weight_only_group_amd as m
    return m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Setup:
    """Sequences of (new tokens, cached tokens) over a paged cache.  Every element of the cache that no
    sequence holds is NaN or an infinity, table entries past a sequence are no page numbers."""

    def __init__(self, lens, hq, hkv, d, page, e4m3=False, layout="phtd", seed=0, sharp=1.0, scales=True):
        rng = np.random.default_rng(seed)
        self.lens, self.e4m3, self.page, self.d, self.hq, self.hkv = lens, e4m3, page, d, hq, hkv
        need = [-(-kv // page) for _, kv in lens]
        pages = sum(need) + 3
        order = rng.permutation(pages)
        self.table = rng.choice([-1, 2 ** 31 - 1, -2 ** 31, pages], size=(len(lens), max(need + [0]) + 2)).astype(np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.starts = np.concatenate([[0], np.cumsum([q for q, _ in lens])]).astype(np.int32)
        self.kv_len = np.array([kv for _, kv in lens], dtype=np.int32)
        self.q = (rng.standard_normal((int(self.starts[-1]), hq, d)) * sharp).astype(np.float16)
        held = np.zeros((pages, page), dtype=bool)
        for b, (_, kv) in enumerate(lens):
            for j in range(need[b]):
                held[self.table[b, j], :min(page, kv - j * page)] = True
        caches = []
        self.scale_k = self.scale_v = None
        for _ in range(2):
            x = rng.standard_normal((pages, hkv, page, d))
            if e4m3:
                codes = ref.e4m3_round(x * 30)
                codes[~np.broadcast_to(held[:, None, :], codes.shape[:3])] = 0x7F
                caches.append(codes)
            else:
                c = x.astype(np.float16)
                junk = rng.choice(np.array([np.nan, np.inf, -np.inf], dtype=np.float16), size=c.shape)
                caches.append(np.where(held[:, None, :, None], c, junk))
        if e4m3 and scales:
            self.scale_k, self.scale_v = (rng.random((2, hkv)) * 0.02 + 0.025).astype(np.float32)
        elif e4m3:
            self.q = (self.q / np.float16(30)).astype(np.float16)
        self.host = caches
        self.dev = [self._place(c, layout) for c in caches] if layout != "kv" else self._one(caches)

    def _place(self, c, layout):
        t = dev(c if layout == "phtd" else c.transpose(0, 2, 1, 3))
        t = t if layout == "phtd" else t.transpose(1, 2)
        return t.view(torch.float8_e4m3fn) if self.e4m3 else t

    def _one(self, caches):
        t = dev(np.stack(caches, 1))
        t = t.view(torch.float8_e4m3fn) if self.e4m3 else t
        return [t[:, 0], t[:, 1]]

    def values(self, i):
        return ref.e4m3_values()[self.host[i]] if self.e4m3 else self.host[i].astype(np.float64)

    def kw(self, **kw):
        a = dict(q_start=dev(self.starts), max_q=max(1, max(q for q, _ in self.lens)))
        if self.scale_k is not None:
            a.update(k_scale=dev(self.scale_k), v_scale=dev(self.scale_v))
        a.update(kw)
        return a

    def run(self, w4, **kw):
        q = kw.pop("q", None)
        return w4.attention_paged(dev(self.q) if q is None else q, *self.dev, dev(self.table), dev(self.kv_len),
                                  **self.kw(**kw))

    def want(self, scale=None, window=0):
        return ref.attention(self.q, self.values(0), self.values(1), self.table, self.kv_len, self.starts,
                             scale=self.d ** -0.5 if scale is None else scale, window=window, k_scale=self.scale_k,
                             v_scale=self.scale_v)

    def bound(self, want, size, wobble):
        n = float(max(self.kv_len.max(), 1))
        v = self.values(1)
        top = np.abs(v[np.isfinite(v)]).max(initial=0.0) * (1.0 if self.scale_v is None else float(self.scale_v.max()))
        return (np.abs(want) * 2.0 ** -11 + 2.0 ** -25 + n * 2.0 ** -25 * top + size *
                (2.0 ** -11 + 2 * wobble[..., None] * (self.d + 8) * 2.0 ** -24 + 2.0 ** -20 + (n / 16 + 32) * 2.0 ** -23))

    def check(self, got, scale=None, window=0):
        want, size, wobble = self.want(scale, window)
        got = got.cpu().numpy().astype(np.float64)
        err, bound = np.abs(got - want), self.bound(want, size, wobble)
        assert np.isfinite(got).all()
        assert (err <= bound).all(), (err / bound).max()
        empty = np.abs(size).sum(-1) == 0
        assert (got[empty] == 0).all()


DECODE = [  # cached tokens of each sequence (one new token each), hq, hkv, dim, page, e4m3, layout
    ([1], 1, 1, 8, 1, False, "phtd"), ([1570], 16, 2, 128, 16, False, "phtd"), ([0, 1, 5], 4, 2, 64, 16, False, "pthd"),
    ([63, 64, 65], 8, 8, 128, 16, False, "phtd"), ([127, 128, 129, 130], 16, 2, 128, 64, False, "kv"),
    ([31, 32, 33, 17, 16, 15], 7, 1, 96, 8, False, "phtd"), ([5000, 1, 0, 33], 16, 2, 128, 100, False, "pthd"),
    ([300, 2], 20, 1, 80, 3, False, "phtd"), ([200, 65], 64, 2, 64, 16, False, "phtd"), ([777], 16, 8, 256, 64, False, "phtd"),
    ([515, 4], 8, 4, 200, 7, False, "pthd"), ([1, 2, 3, 4], 2, 2, 136, 256, False, "phtd"),
    ([1570], 16, 2, 128, 16, True, "phtd"), ([63, 0, 129], 8, 4, 64, 16, True, "pthd"), ([777, 31], 16, 8, 256, 32, True, "kv"),
    ([1000, 1], 12, 4, 80, 5, True, "phtd"), ([40], 1, 1, 16, 8, True, "phtd"), ([100, 700], 32, 1, 112, 16, True, "phtd"),
    ([20011], 8, 1, 128, 16, False, "phtd"), ([20011, 3], 2, 1, 64, 32, True, "phtd"),
]


@pytest.mark.parametrize("kv,hq,hkv,d,page,e4m3,layout", DECODE)
def test_decode(w4, kv, hq, hkv, d, page, e4m3, layout):
    s = Setup([(1, n) for n in kv], hq, hkv, d, page, e4m3, layout, seed=sum(kv) + d)
    a = s.run(w4)
    s.check(a)
    # the same rows without q_start, and again: the same bits
    b = w4.attention_paged(dev(s.q), *s.dev, dev(s.table), dev(s.kv_len),
                           **{k: x for k, x in s.kw().items() if k not in ("q_start", "max_q")})
    assert torch.equal(a, b)


CHUNK = [  # (new, cached) of each sequence, hq, hkv, dim, page, window, e4m3, layout
    ([(5, 5)], 2, 1, 64, 16, 0, False, "phtd"), ([(64, 64)], 4, 4, 128, 16, 0, False, "phtd"),
    ([(130, 130)], 4, 1, 128, 16, 0, False, "pthd"), ([(8, 1000), (8, 300)], 16, 2, 128, 16, 0, False, "phtd"),
    ([(2, 3), (0, 0), (70, 200), (1, 1), (0, 9), (33, 33)], 8, 2, 128, 8, 0, False, "phtd"),
    ([(9, 4), (3, 0), (40, 20)], 4, 2, 64, 16, 0, False, "phtd"),  # more rows than cached tokens
    ([(257, 300)], 3, 1, 80, 100, 0, False, "kv"), ([(100, 333)], 2, 2, 256, 64, 0, False, "phtd"),
    ([(65, 400), (1, 129)], 8, 1, 200, 3, 0, False, "phtd"), ([(40, 77)], 28, 4, 96, 7, 0, False, "pthd"),
    ([(300, 500)], 4, 2, 128, 16, 1, False, "phtd"), ([(300, 500), (1, 900)], 4, 2, 128, 16, 100, False, "phtd"),
    ([(130, 640), (3, 70)], 8, 2, 256, 64, 64, False, "phtd"), ([(20, 700)], 16, 2, 64, 16, 333, True, "phtd"),
    ([(1, 900), (1, 77)], 16, 2, 128, 16, 129, False, "phtd"), ([(1, 900), (1, 7)], 16, 4, 128, 16, 7, True, "phtd"),
    ([(130, 130), (2, 1500)], 16, 2, 128, 16, 0, True, "phtd"), ([(70, 90)], 8, 8, 256, 64, 0, True, "kv"),
    ([(33, 70)], 6, 2, 80, 5, 0, True, "pthd"), ([(200, 1000)], 32, 1, 16, 16, 0, True, "phtd"),
    ([(600, 2000)], 2, 1, 128, 16, 0, False, "phtd"), ([(3, 9000), (2, 100)], 8, 1, 128, 16, 0, False, "phtd"),
    ([(17, 17), (1, 6000)] + [(1, 10 * i) for i in range(70)], 4, 1, 64, 16, 0, False, "phtd"),
]


@pytest.mark.parametrize("lens,hq,hkv,d,page,window,e4m3,layout", CHUNK)
def test_chunk(w4, lens, hq, hkv, d, page, window, e4m3, layout):
    s = Setup(lens, hq, hkv, d, page, e4m3, layout, seed=sum(map(sum, lens)) + d)
    a = s.run(w4, window=window)
    s.check(a, window=window)
    assert torch.equal(a, s.run(w4, window=window, max_q=s.q.shape[0], workspace=torch.full(
        (32 << 20,), 0xFF, dtype=torch.uint8, device="cuda"))) or s.check(s.run(w4, window=window, max_q=s.q.shape[0]),
                                                                        window=window) is None


@pytest.mark.parametrize("sharp,scale", [(8.0, None), (30.0, None), (1.0, 1e-6), (3.0, 2.0)])
def test_sharp_and_flat_scores(w4, sharp, scale):
    for lens in ([(1, 700), (1, 3)], [(90, 300)]):
        s = Setup(lens, 4, 1, 128, 16, seed=5, sharp=sharp)
        s.check(s.run(w4, scale=scale), scale=scale)


def test_growing_maxima(w4):
    # scores that rise along the keys: the running maximum moves in every block
    for lens in ([(1, 1500)], [(70, 700)]):
        s = Setup(lens, 2, 1, 64, 16, seed=6)
        n = lens[0][1]
        s.q[:] = np.abs(s.q)
        for j in range(n):
            s.host[0][s.table[0, j // 16], 0, j % 16] = np.float16(j * 6.0 / n) * np.ones(64, dtype=np.float16)
        s.dev[0] = dev(s.host[0])
        s.check(s.run(w4))


def test_scales_may_be_absent(w4):
    s = Setup([(1, 300), (40, 50)], 4, 2, 64, 16, True, seed=7, scales=False)
    s.check(s.run(w4))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,window", [([(20, 300)], 0), ([(200, 300)], 0), ([(4, 90)], 0), ([(150, 400)], 33),
                                         ([(3, 300), (2, 70)], 20)])
def test_what_a_row_does_not_see_does_not_reach_it(w4, lens, window, e4m3):
    # one cached token is NaN or an infinity: rows that do not see it keep their bits, the others get what
    # arithmetic with it gives (not finite)
    for junk in (np.nan, np.inf, -np.inf):
        if e4m3 and not np.isnan(junk):
            continue
        for back in (0, lens[0][0] // 2, lens[0][0] + 3):
            s = Setup(lens, 4, 2, 64, 16, e4m3, seed=8)
            clean = s.run(w4, window=window).cpu().numpy()
            n, kv = lens[0]
            j = kv - 1 - back
            for c in range(2):
                s.host[c][s.table[0, j // 16], :, j % 16] = 0x7F if e4m3 else np.float16(junk)
            s.dev = [s._place(c, "phtd") for c in s.host]
            got = s.run(w4, window=window).cpu().numpy()
            p = kv - n + np.arange(n)
            sees = (p >= j) & ((p - j < window) if window else True)
            assert np.array_equal(got[:n][~sees].view(np.uint16), clean[:n][~sees].view(np.uint16)), (junk, back)
            assert np.array_equal(got[n:], clean[n:])
            assert not np.isfinite(got[:n][sees]).any()


def test_infinite_values_at_seen_keys(w4):
    # V infinite at one key, K finite: +-inf in the rows that see it, both signs NaN
    s = Setup([(40, 200)], 2, 1, 64, 16, seed=9)
    for j, val in ((170, np.inf), (190, -np.inf)):
        s.host[1][s.table[0, j // 16], 0, j % 16, :] = np.float16(val)
    s.dev = [s._place(c, "phtd") for c in s.host]
    got = s.run(w4).cpu().numpy()
    p = 160 + np.arange(40)
    assert np.isfinite(got[p < 170]).all()
    assert (got[(p >= 170) & (p < 190)] == np.inf).all()
    assert np.isnan(got[p >= 190]).all()


def test_pages_outside_the_cache(w4):
    for lens in ([(1, 200), (1, 90)], [(50, 200), (30, 90)]):
        s = Setup(lens, 4, 2, 64, 16, seed=10)
        good = s.run(w4).cpu().numpy()
        for page in (-1, 2 ** 31 - 1, s.host[0].shape[0]):
            t = s.table.copy()
            s.table[0, 3] = page
            got = s.run(w4).cpu().numpy()
            s.table = t
            n = lens[0][0]
            assert np.isnan(got[:n]).all() and np.array_equal(got[n:], good[n:])


def test_lengths_outside_the_table(w4):
    # kv_len past the table is the table's; below 0, none.  starts past the rows end there
    s = Setup([(1, 64), (1, 40)], 2, 1, 64, 16, seed=11)
    s.table = np.ascontiguousarray(s.table[:, :4])
    s.host[0][:] = np.float16(0)
    s.host[1][:] = np.float16(1)
    s.dev = [s._place(c, "phtd") for c in s.host]
    s.kv_len = np.array([2 ** 31 - 1, -5], dtype=np.int32)
    got = s.run(w4).cpu().numpy()
    assert (got[0] == 1).all() and (got[1] == 0).all()
    s = Setup([(3, 64), (2, 40)], 2, 1, 64, 16, seed=12)
    good = s.run(w4)
    s.starts = np.array([0, 3, 9999], dtype=np.int32)  # 2 rows are there
    s.kv_len[1] = 40
    assert torch.equal(s.run(w4, max_q=5), good)


def test_rows_of_no_sequence_are_left(w4):
    for lens in ([(1, 20), (1, 0)], [(30, 40), (2, 2)]):
        s = Setup(lens, 4, 2, 64, 16, seed=13)
        t = s.q.shape[0]
        q = torch.randn((t + 7, 4, 64), device="cuda", dtype=torch.float16)
        q[:t] = dev(s.q)
        out = torch.full((t + 7, 4, 64), 9.0, device="cuda", dtype=torch.float16)
        s.run(w4, q=q, out=out)
        s.check(out[:t])
        assert (out[t:] == 9).all()


def test_strided_rows(w4):
    for lens in ([(1, 200), (1, 33)], [(90, 200), (3, 33)]):
        s = Setup(lens, 4, 2, 96, 16, seed=14)
        t = s.q.shape[0]
        rows = torch.full((t, 9, 96), 5.0, device="cuda", dtype=torch.float16)
        rows[:, 1:5] = dev(s.q)
        out = torch.full((t, 10, 96), 9.0, device="cuda", dtype=torch.float16)
        s.run(w4, q=rows[:, 1:5], out=out[:, 3:7])
        s.check(out[:, 3:7])
        assert (out[:, :3] == 9).all() and (out[:, 7:] == 9).all()


def test_far_offsets(w4):
    # pages past 2^32 elements of the cache
    pages, page, d = 2100, 16384, 128
    kc = torch.empty((pages, 1, page, d), dtype=torch.float16, device="cuda")
    vc = torch.empty_like(kc)
    for lens in ([(1, 100)], [(50, 100)]):
        s = Setup(lens, 2, 1, d, 128, seed=15)
        n = 100
        for c, h in ((kc, s.host[0]), (vc, s.host[1])):
            c[pages - 1, 0, :n] = dev(h[s.table[0, 0], 0, :n])
        got = w4.attention_paged(dev(s.q), kc, vc, torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda"),
                                 dev(s.kv_len), q_start=dev(s.starts), max_q=lens[0][0])
        s.check(got)


def test_streams_and_shared_inputs(w4):
    # two calls at once on two streams, each with its workspace; neither is the default stream
    a, b = Setup([(1, 3000)], 8, 1, 128, 16, seed=16), Setup([(100, 900)], 8, 2, 128, 16, seed=17)
    wa, wb = a.run(w4), b.run(w4)
    qa, ta, la, ka = dev(a.q), dev(a.table), dev(a.kv_len), a.kw()
    qb, tb, lb, kb = dev(b.q), dev(b.table), dev(b.kv_len), b.kw()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(4):
        with torch.cuda.stream(sa):
            oa = w4.attention_paged(qa, *a.dev, ta, la, **ka)
        with torch.cuda.stream(sb):
            ob = w4.attention_paged(qb, *b.dev, tb, lb, **kb)
        outs.append((oa, ob))
    torch.cuda.synchronize()
    for oa, ob in outs:
        assert torch.equal(oa, wa) and torch.equal(ob, wb)


def test_captured_decode_replays_as_lengths_grow(w4):
    # append + attention of one token, captured once, replayed while positions, slots and lengths move;
    # two graphs share the workspace, and each replay is compared with eager calls
    d, hq, hkv, page, steps = 64, 4, 2, 16, 5
    rng = np.random.default_rng(18)
    lens = [30, 7]
    kc = torch.zeros((16, hkv, page, d), dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    table = dev(rng.permutation(16).reshape(2, 8).astype(np.int32))
    freq, _ = w4.rope_frequencies(d)
    rows = torch.randn((steps + 40, 2, hq + 2 * hkv, d), device="cuda")
    for t in range(40):  # the cached tokens (those past a sequence's length come to be overwritten)
        pos = np.full(2, t, dtype=np.int32)
        _append(w4, rows[t], pos, table, kc, vc, freq, hq, hkv, page)
    x = torch.empty((2, hq + 2 * hkv, d), device="cuda")
    pos_d, slot_d = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    len_d, qr = torch.ones(2, dtype=torch.int32, device="cuda"), torch.empty((2, hq, d), dtype=torch.float16, device="cuda")
    out = [torch.empty((2, hq, d), dtype=torch.float16, device="cuda") for _ in range(2)]
    ws = torch.empty(max(16, w4.attention_workspace_bytes(kc, 2, 2, 1, hq, 8)), dtype=torch.uint8, device="cuda")

    def step(o):
        w4.kv_append_rope(x[:, hq:hq + hkv], x[:, hq + hkv:], kc, vc, slot_d, pos_d, freq, q=x[:, :hq], q_out=qr)
        w4.attention_paged(qr, kc, vc, table, len_d, out=o, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(out[0])
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g, o in zip(graphs, out):
        with torch.cuda.graph(g):
            step(o)
    for i in range(steps):
        pos = np.array([n + i for n in lens], dtype=np.int32)
        x.copy_(rows[40 + i])
        pos_d.copy_(dev(pos))
        slot_d.copy_(_slots(table, pos, page))
        len_d.copy_(dev(pos + 1))
        for g, o in zip(graphs, out):
            o.fill_(7.0)
            g.replay()
            torch.cuda.synchronize()
        want = w4.attention_paged(qr, kc, vc, table, dev(pos + 1))
        torch.cuda.synchronize()
        assert torch.equal(out[0], want) and torch.equal(out[1], want), i


def _slots(table, pos, page):
    p = torch.from_numpy(pos.astype(np.int64)).cuda()
    return table[torch.arange(len(pos), device="cuda"), p // page].long() * page + p % page


def _append(w4, x, pos, table, kc, vc, freq, hq, hkv, page):
    return w4.kv_append_rope(x[:, hq:hq + hkv], x[:, hq + hkv:], kc, vc, _slots(table, pos, page), dev(pos), freq,
                             q=x[:, :hq])


def test_decode_layer_from_projection_to_projection(w4):
    # q|k|v projection (int4) -> rotation and append -> attention -> output projection (int4), for a prompt
    # of 40 tokens and then a single one, each stage against the oracle on its own inputs
    hidden, hq, hkv, d, page = 512, 8, 2, 64, 16
    n = (hq + 2 * hkv) * d
    qw, sc, bi = synth.w4_weights(n, hidden, seed=3)
    ow, so, bo = synth.w4_weights(hidden, hq * d, seed=4)
    pqkv, po = w4.w4_pack(dev(qw)), w4.w4_pack(dev(ow))
    freq, _ = w4.rope_frequencies(d)
    kc = torch.zeros((8, hkv, page, d), dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    table = dev(np.array([[5, 2, 7, 0]], dtype=np.int32))
    done = 0
    for t in (40, 1):
        x = synth.activations(t, hidden, seed=t)
        if t <= 16:
            rows = w4.w4_gemv(pqkv, dev(sc), dev(bi), dev(x))
        else:
            rows = w4.gemm_f16(dev(x), w4.w4_dequant_f16_t(pqkv, dev(sc), dev(bi)))
        y_ref, bound = oracle.gemv_ref(oracle.pack(qw), sc, bi, x)
        assert oracle.check_bound(rows.cpu().numpy(), y_ref, bound)[0]
        rows = rows.view(t, hq + 2 * hkv, d)
        pos = np.arange(done, done + t, dtype=np.int32)
        slots = table[0, torch.from_numpy(pos // page).cuda().long()].long() * page + dev(pos % page).long()
        q = w4.kv_append_rope(rows[:, hq:hq + hkv], rows[:, hq + hkv:], kc, vc, slots, dev(pos), freq, q=rows[:, :hq])
        done += t
        host = rows.cpu().numpy()
        turned = ref.rope(host[:, :hq + hkv], pos, freq.cpu().numpy())
        assert np.allclose(q.cpu().numpy(), turned[:, :hq], rtol=2.0 ** -10, atol=2.0 ** -10)
        flat = kc.transpose(1, 2).reshape(-1, hkv, d)[slots].cpu().numpy()
        assert np.allclose(flat, turned[:, hq:], rtol=2.0 ** -10, atol=2.0 ** -10)
        out = w4.attention_paged(q, kc, vc, table, dev(np.array([done], dtype=np.int32)),
                                 q_start=dev(np.array([0, t], dtype=np.int32)), max_q=t)
        want, size, wobble = ref.attention(q.cpu().numpy(), kc.cpu().numpy(), vc.cpu().numpy(), table.cpu().numpy(),
                                           [done], [0, t], scale=d ** -0.5)
        err = np.abs(out.cpu().numpy() - want)
        top = np.abs(vc.cpu().numpy().astype(np.float64)).max()
        lim = (np.abs(want) * 2.0 ** -11 + 2.0 ** -25 + done * 2.0 ** -25 * top +
               size * (2.0 ** -11 + 2 * wobble[..., None] * (d + 8) * 2.0 ** -24 + 2.0 ** -20 + 35 * 2.0 ** -23))
        assert (err <= lim).all(), (err / lim).max()
        a = out.view(t, hq * d)
        if t <= 16:
            y = w4.w4_gemv(po, dev(so), dev(bo), a)
        else:
            y = w4.gemm_f16(a, w4.w4_dequant_f16_t(po, dev(so), dev(bo)))
        y_ref, bound = oracle.gemv_ref(oracle.pack(ow), so, bo, a.cpu().numpy())
        assert oracle.check_bound(y.cpu().numpy(), y_ref, bound)[0]


def test_bindings_refuse(w4):
    s = Setup([(1, 20), (1, 9)], 4, 2, 64, 16, seed=20)
    ok = dict(q=dev(s.q), k_cache=s.dev[0], v_cache=s.dev[1], table=dev(s.table), kv_len=dev(s.kv_len))
    w4.attention_paged(**ok)
    q = ok["q"]
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(table=ok["table"].long()), dict(kv_len=ok["kv_len"].long()),
                dict(out=torch.empty_like(q, dtype=torch.float32)), dict(q=None), dict(k_cache=None)):
        with pytest.raises((TypeError, ValueError, AttributeError)):
            w4.attention_paged(**{**ok, **bad})
    for bad in (dict(q=q[:, :, :32]), dict(kv_len=ok["kv_len"][:1]), dict(table=ok["table"].t()), dict(out=q[:1].clone()),
                dict(q_start=dev(s.starts[:2])), dict(v_cache=s.dev[1][:-1]), dict(k_scale=torch.ones(2, device="cuda")),
                dict(q=q.view(2, 256))):
        with pytest.raises(ValueError):
            w4.attention_paged(**{**ok, **bad})
    for bad in (dict(scale=0.0), dict(scale=float("nan")), dict(window=-1), dict(max_q=3, q_start=dev(s.starts)),
                dict(q=q[:, :3].contiguous()), dict(q=q[:1].contiguous())):
        with pytest.raises(w4.W4Error):
            w4.attention_paged(**{**ok, **bad})
