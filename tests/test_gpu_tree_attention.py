"""attention_paged_tree against the fp64 oracle; bounds as in test_gpu_attention.py."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import stepref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_attention import Setup, dev, w4  # noqa: E402, F401


def words_of(sees, words):
    """int64 [T][words] of sets of new tokens"""
    out = np.zeros((len(sees), words), dtype=np.uint64)
    for t, s in enumerate(sees):
        for j in s:
            out[t, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return out.view(np.int64)


class Tree(Setup):
    def __init__(self, lens, hq, hkv, d, page, e4m3=False, layout="phtd", seed=0, kind="tree", **kw):
        super().__init__(lens, hq, hkv, d, page, e4m3, layout, seed, **kw)
        rng = np.random.default_rng(seed + 99)
        self.sees = []
        for n, _ in lens:
            seen = []
            for i in range(n):
                if kind == "any":
                    seen.append(set(np.flatnonzero(rng.random(n) < rng.choice([0.0, 0.1, 0.7])).tolist()))
                elif kind == "none":
                    seen.append(set())
                elif kind == "chain":
                    seen.append(set(range(i + 1)))
                else:
                    p = max(i - 1 - int(rng.integers(0, 6)), -1)
                    seen.append((set(seen[p]) if p >= 0 else set()) | {i})
            self.sees += seen
        self.words = -(-max(1, max(n for n, _ in lens)) // 64)
        m = words_of(self.sees, self.words + 1)
        # bits from n on are set: they count for nothing
        at = 0
        for n, _ in lens:
            for j in range(n, 64 * (self.words + 1)):
                m.view(np.uint64)[at:at + n, j // 64] |= np.uint64(1) << np.uint64(j % 64)
            at += n
        self.mask = dev(m)

    def run(self, w4, **kw):
        q = kw.pop("q", None)
        mask = kw.pop("mask", self.mask[:, :self.words])
        return w4.attention_paged_tree(dev(self.q) if q is None else q, *self.dev, dev(self.table), dev(self.kv_len), mask,
                                       **self.kw(**kw))

    def want(self, scale=None, window=0):
        return stepref.attention(self.q, self.values(0), self.values(1), self.table, self.kv_len, self.starts, self.sees,
                                 scale=self.d ** -0.5 if scale is None else scale, window=window, k_scale=self.scale_k,
                                 v_scale=self.scale_v)


CASES = [  # (new, cached) of each sequence, hq, hkv, dim, page, window, e4m3, layout
    ([(1, 1)], 1, 1, 8, 1, 0, False, "phtd"), ([(1, 1), (1, 0), (1, 40)], 4, 2, 64, 16, 0, False, "phtd"),
    ([(8, 1570)], 16, 2, 128, 16, 0, False, "phtd"), ([(2, 3), (2, 2), (2, 900)], 8, 1, 128, 16, 0, False, "pthd"),
    ([(5, 5)], 2, 1, 64, 16, 0, False, "phtd"), ([(16, 16), (16, 47), (7, 49)], 1, 1, 64, 16, 0, False, "phtd"),
    ([(16, 1000), (3, 33)], 1, 1, 96, 5, 0, False, "kv"), ([(4, 1000), (4, 31), (3, 64)], 8, 2, 256, 64, 0, False, "phtd"),
    ([(8, 700), (2, 77)], 4, 2, 128, 16, 0, True, "phtd"), ([(4, 515), (1, 2)], 8, 2, 80, 7, 0, True, "pthd"),
    ([(3, 9000), (2, 100)], 4, 1, 128, 16, 0, False, "phtd"), ([(16, 800), (9, 300)], 1, 1, 64, 16, 100, False, "phtd"),
    ([(8, 900), (1, 7)], 2, 1, 128, 16, 8, True, "phtd"),
    # more rows than the kernel for few takes
    ([(64, 64)], 4, 4, 128, 16, 0, False, "phtd"), ([(64, 1000)], 16, 2, 128, 16, 0, False, "phtd"),
    ([(63, 130), (17, 400), (0, 0), (1, 9), (33, 40)], 8, 2, 128, 8, 0, False, "pthd"),
    ([(48, 1100), (7, 300), (30, 333)], 16, 8, 128, 32, 0, True, "phtd"), ([(65, 200)], 3, 1, 80, 100, 0, False, "kv"),
    ([(130, 333), (3, 70)], 2, 2, 256, 64, 0, False, "phtd"), ([(200, 640), (61, 500)], 8, 4, 256, 64, 256, False, "phtd"),
    ([(129, 300), (40, 3000)], 4, 2, 64, 16, 300, True, "pthd"), ([(300, 301), (5, 800)], 4, 2, 128, 16, 0, False, "phtd"),
    ([(70, 90)], 8, 8, 256, 64, 0, True, "kv"), ([(40, 77)], 28, 4, 96, 7, 40, False, "pthd"),
    ([(200, 1000)], 32, 1, 16, 16, 0, True, "phtd"), ([(24, 6000)], 16, 2, 128, 16, 0, False, "phtd"),
    ([(12, 50 + 13 * i) for i in range(40)], 4, 1, 64, 16, 0, False, "phtd"),
]


@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("lens,hq,hkv,d,page,window,e4m3,layout", CASES)
def test_trees(w4, lens, hq, hkv, d, page, window, e4m3, layout, kind):  # noqa: F811
    s = Tree(lens, hq, hkv, d, page, e4m3, layout, seed=sum(map(sum, lens)) + d, kind=kind)
    a = s.run(w4, window=window)
    s.check(a, window=window)
    # again, with a workspace of its own and a mask with more words than it needs: the same bits
    b = s.run(w4, window=window, mask=s.mask, workspace=torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda"))
    assert torch.equal(a, b)


@pytest.mark.parametrize("lens", [[(8, 700)], [(64, 700), (20, 90)], [(150, 151)], [(12, 12), (3, 3)]])
def test_rows_that_see_no_new_token(w4, lens):  # noqa: F811
    s = Tree(lens, 4, 2, 64, 16, seed=3, kind="none")
    for window in (0, 150):
        s.check(s.run(w4, window=window), window=window)


@pytest.mark.parametrize("lens", [[(8, 5), (4, 0)], [(64, 40), (20, 0), (30, 29)], [(9, 4), (3, 0), (40, 20), (2, 900)]])
@pytest.mark.parametrize("kind", ["tree", "any"])
def test_more_new_tokens_than_cached(w4, lens, kind):  # noqa: F811
    s = Tree(lens, 4, 2, 64, 16, seed=4, kind=kind)
    s.check(s.run(w4))
    s.check(s.run(w4, window=70), window=70)


@pytest.mark.parametrize("lens,hq,hkv,d,e4m3", [([(8, 900), (2, 30)], 4, 2, 64, False), ([(100, 500)], 4, 2, 128, False),
                                                ([(40, 3000), (64, 700)], 16, 2, 128, True), ([(70, 300)], 2, 1, 256, False)])
def test_a_chain_is_attention_paged(w4, lens, hq, hkv, d, e4m3):  # noqa: F811
    s = Tree(lens, hq, hkv, d, 16, e4m3, seed=5, kind="chain")
    for window in (0, 100):
        a = s.run(w4, window=window)
        s.check(a, window=window)
        s.check(Setup.run(s, w4, window=window), window=window)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,hq", [([(8, 300)], 2), ([(40, 300), (3, 70)], 4), ([(200, 333)], 4), ([(1, 40)], 4)])
def test_what_a_row_does_not_see_does_not_reach_it(w4, lens, hq, e4m3):  # noqa: F811
    # one cached token is NaN or an infinity: rows that do not see it keep their bits, the others are not finite
    for junk in (np.nan, np.inf, -np.inf):
        if e4m3 and not np.isnan(junk):
            continue
        for back in (0, lens[0][0] // 2, lens[0][0] - 1, lens[0][0] + 3):
            s = Tree(lens, hq, 2, 64, 16, e4m3, seed=8, kind="any")
            clean = s.run(w4).cpu().numpy()
            n, kv = lens[0]
            j = kv - 1 - back
            for c in range(2):
                s.host[c][s.table[0, j // 16], :, j % 16] = 0x7F if e4m3 else np.float16(junk)
            s.dev = [s._place(c, "phtd") for c in s.host]
            got = s.run(w4).cpu().numpy()
            sees = np.array([j in stepref.seen_keys(s.sees[i], kv, n) for i in range(n)])
            assert np.array_equal(got[:n][~sees].view(np.uint16), clean[:n][~sees].view(np.uint16)), (junk, back)
            assert np.array_equal(got[n:], clean[n:])
            assert not np.isfinite(got[:n][sees]).any()


def test_pages_outside_the_cache(w4):  # noqa: F811
    for lens in ([(2, 200), (1, 90)], [(50, 200), (30, 90)]):
        s = Tree(lens, 4, 2, 64, 16, seed=10)
        good = s.run(w4).cpu().numpy()
        for page in (-1, 2 ** 31 - 1, s.host[0].shape[0]):
            t = s.table.copy()
            s.table[0, 3] = page
            got = s.run(w4).cpu().numpy()
            s.table = t
            n = lens[0][0]
            assert np.isnan(got[:n]).all() and np.array_equal(got[n:], good[n:])


def test_rows_of_no_sequence_are_left(w4):  # noqa: F811
    for lens in ([(2, 20), (1, 0)], [(30, 40), (2, 2)]):
        s = Tree(lens, 4, 2, 64, 16, seed=13)
        t = s.q.shape[0]
        q = torch.randn((t + 7, 4, 64), device="cuda", dtype=torch.float16)
        q[:t] = dev(s.q)
        mask = torch.full((t + 7, s.words), -1, dtype=torch.int64, device="cuda")
        mask[:t] = s.mask[:, :s.words]
        out = torch.full((t + 7, 4, 64), 9.0, device="cuda", dtype=torch.float16)
        s.run(w4, q=q, out=out, mask=mask)
        s.check(out[:t])
        assert (out[t:] == 9).all()


def test_strided_rows_in_place(w4):  # noqa: F811
    for lens in ([(3, 200), (1, 33)], [(90, 200), (3, 33)]):
        s = Tree(lens, 4, 2, 96, 16, seed=14)
        rows = torch.full((s.q.shape[0], 9, 96), 5.0, device="cuda", dtype=torch.float16)
        rows[:, 1:5] = dev(s.q)
        s.run(w4, q=rows[:, 1:5], out=rows[:, 1:5])
        s.check(rows[:, 1:5])
        assert (rows[:, :1] == 5).all() and (rows[:, 5:] == 5).all()


def test_a_long_mask(w4):  # noqa: F811
    # a chunk whose rows see each other in both directions inside blocks of 100, and all before
    n, kv = 700, 1100
    s = Tree([(n, kv)], 2, 1, 64, 16, seed=15, kind="none")
    s.sees = [set(range(min(n, (i // 100 + 1) * 100))) for i in range(n)]
    s.mask = dev(words_of(s.sees, s.words))
    s.check(s.run(w4))


def test_streams(w4):  # noqa: F811
    a, b = Tree([(8, 3000)], 2, 1, 128, 16, seed=16), Tree([(100, 900)], 8, 2, 128, 16, seed=17)
    wa, wb = a.run(w4), b.run(w4)
    qa, ta, la, ka = dev(a.q), dev(a.table), dev(a.kv_len), a.kw()
    qb, tb, lb, kb = dev(b.q), dev(b.table), dev(b.kv_len), b.kw()
    ma, mb = a.mask[:, :a.words], b.mask[:, :b.words]
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(4):
        with torch.cuda.stream(sa):
            oa = w4.attention_paged_tree(qa, *a.dev, ta, la, ma, **ka)
        with torch.cuda.stream(sb):
            ob = w4.attention_paged_tree(qb, *b.dev, tb, lb, mb, **kb)
        outs.append((oa, ob))
    torch.cuda.synchronize()
    for oa, ob in outs:
        assert torch.equal(oa, wa) and torch.equal(ob, wb)


def test_bindings_refuse(w4):  # noqa: F811
    s = Tree([(2, 20), (1, 9)], 4, 2, 64, 16, seed=20)
    ok = dict(q=dev(s.q), k_cache=s.dev[0], v_cache=s.dev[1], table=dev(s.table), kv_len=dev(s.kv_len), mask=s.mask,
              q_start=dev(s.starts), max_q=2)
    w4.attention_paged_tree(**ok)
    for bad in (dict(mask=s.mask[:2]), dict(mask=s.mask.int()), dict(mask=s.mask.cpu()), dict(mask=None),
                dict(mask=s.mask[:, :0]), dict(mask=s.mask.t()), dict(q=None), dict(max_q=999)):
        with pytest.raises((TypeError, ValueError, AttributeError)):
            w4.attention_paged_tree(**{**ok, **bad})
    for bad in (dict(window=1), dict(scale=0.0), dict(window=-1)):
        with pytest.raises(w4.W4Error):
            w4.attention_paged_tree(**{**ok, **bad})


@pytest.mark.parametrize("b,hq,hkv,d,e4m3", [(130, 4, 1, 64, False), (300, 8, 2, 128, True), (700, 4, 2, 64, False),
                                             (1300, 4, 1, 64, True)])
@pytest.mark.parametrize("n", [3, 24, 70])
def test_many_sequences(w4, b, hq, hkv, d, e4m3, n):  # noqa: F811
    # more than a workgroup's threads, lengths from none to some; rows of one kernel and of the others
    rng = np.random.default_rng(b + n)
    if n == 70:
        b = b // 5
    kv = rng.integers(0, 90, b)
    kv[[0, b // 2]] = 1500, 400
    new = rng.integers(0, n + 1, b)
    new[b // 3] = n
    s = Tree([(int(q), int(x)) for q, x in zip(new, kv)], hq, hkv, d, 16, e4m3, seed=b, kind="any")
    s.check(s.run(w4))
    s.check(s.run(w4, window=75), window=75)


@pytest.mark.parametrize("lens,hq,hkv,d,e4m3", [
    ([(24, 5000), (11, 900), (5, 64)], 8, 2, 128, True), ([(24, 5000), (11, 900)], 8, 2, 64, False),
    ([(16, 5000), (9, 900), (1, 31)], 8, 2, 256, False), ([(24, 3000), (20, 900)], 8, 2, 256, True),
    ([(16, 9000)], 4, 1, 96, False), ([(9, 700), (8, 40), (32, 32)], 2, 2, 128, False)])
def test_the_kernel_between(w4, lens, hq, hkv, d, e4m3):  # noqa: F811
    # up to 96 rows of a tile or two, whole and half full, in one part and in many
    for window in (0, 200):
        s = Tree(lens, hq, hkv, d, 16, e4m3, seed=21, kind="any")
        s.check(s.run(w4, window=window), window=window)
    s = Tree(lens, hq, hkv, d, 7, e4m3, seed=22)
    s.check(s.run(w4))


def test_workspace_is_of_the_size_that_is_asked_for(w4):  # noqa: F811
    for lens, hq, hkv, d in (([(24, 5000), (11, 900)], 8, 2, 128), ([(100, 3000), (60, 900)], 8, 2, 64), ([(4, 3000)], 8, 2, 128)):
        s = Tree(lens, hq, hkv, d, 16, seed=23)
        need = w4.attention_workspace_bytes(s.dev[0], len(lens), s.q.shape[0], max(n for n, _ in lens), hq, s.table.shape[1],
                                            tree=True)
        assert need > 0
        ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        for fill in (0xFF, 0x00, 0x7E):
            ws[:need].fill_(fill)
            s.check(s.run(w4, workspace=ws[:need]))
            assert (ws[need:] == 0xA5).all()


def test_captured_and_replayed(w4):  # noqa: F811
    # two graphs share a workspace; lengths and masks change between replays, each is compared with the eager call
    s = Tree([(12, 400), (9, 300), (12, 40)], 8, 2, 128, 16, seed=24)
    q, t, ln, mask, kw = dev(s.q), dev(s.table), dev(s.kv_len), s.mask[:, :1].clone(), s.kw()
    out = [torch.empty_like(q) for _ in range(2)]
    kw["workspace"] = torch.empty(max(16, w4.attention_workspace_bytes(s.dev[0], 3, q.shape[0], 12, 8, t.shape[1], tree=True)),
                                  dtype=torch.uint8, device="cuda")

    def call(o):
        w4.attention_paged_tree(q, *s.dev, t, ln, mask, out=o, **kw)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.current_stream())
        call(out[0])
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g, o in zip(graphs, out):
        with torch.cuda.graph(g):
            call(o)
    for i in range(5):
        s.kv_len = np.array([400 - 90 * i, 300 - 7 * i, 40 - 5 * i], dtype=np.int32)
        s.sees = [x if (j + i) % 3 else set() for j, x in enumerate(s.sees)]
        ln.copy_(dev(s.kv_len))
        mask.copy_(dev(words_of(s.sees, 1)))
        for g, o in zip(graphs, out):
            o.fill_(7.0)
            g.replay()
        torch.cuda.synchronize()
        s.check(out[0])
        assert torch.equal(out[0], out[1])
        want = w4.attention_paged_tree(q, *s.dev, t, ln, mask, **{**kw, "workspace": None})
        assert torch.equal(out[0], want), i


@pytest.mark.parametrize("n,window", [(12, 0), (12, 40), (90, 0), (90, 95)])
def test_more_rows_than_max_q(w4, n, window):  # noqa: F811
    # of the first sequence: its rows past max_q are unspecified, the others' are right, and nothing leaves the workspace
    s = Tree([(n, 3000), (5, 700), (3, 90)], 4, 2, 64, 16, seed=25, kind="any")
    most = n * 3 // 4
    need = w4.attention_workspace_bytes(s.dev[0], 3, s.q.shape[0], most, 4, s.table.shape[1], window, tree=True)
    ws = torch.full((need + 65536,), 0xA5, dtype=torch.uint8, device="cuda")
    got = s.run(w4, window=window, max_q=most, workspace=ws[:max(need, 16)]).cpu().numpy().astype(np.float64)
    assert (ws[max(need, 16):] == 0xA5).all()
    want, size, wobble = s.want(None, window)
    keep = np.r_[n:s.q.shape[0]]
    assert (np.abs(got - want) <= s.bound(want, size, wobble))[keep].all()


@pytest.mark.parametrize("new", [3, 30, 200])
def test_starts_that_fall(w4, new):  # noqa: F811
    # starts in any order are kept in bounds: sequences then share rows, whose results are one or another's
    s = Tree([(new, 1000), (new, 1000), (new, 1000), (new, 1000)], 4, 2, 64, 16, seed=26, kind="none")
    t = s.q.shape[0]
    for starts in ([0, t, 0, t, 0], [t, 0, t, 0, t], [-9, 2 ** 31 - 1, -2 ** 31, t, 5], [new, new, 0, t, t]):
        need = w4.attention_workspace_bytes(s.dev[0], 4, t, new, 4, s.table.shape[1], tree=True)
        ws = torch.full((need + 65536,), 0xA5, dtype=torch.uint8, device="cuda")
        s.run(w4, q_start=dev(np.array(starts, dtype=np.int32)), max_q=new, workspace=ws[:max(need, 16)])
        torch.cuda.synchronize()
        assert (ws[max(need, 16):] == 0xA5).all()


def test_many_tiles_in_many_rounds(w4):  # noqa: F811
    # more tiles than parts are made for
    rng = np.random.default_rng(27)
    kv = rng.integers(20, 60, 600)
    kv[7] = 900
    s = Tree([(20, int(x)) for x in kv], 64, 8, 64, 16, seed=27, kind="any")
    s.check(s.run(w4))
