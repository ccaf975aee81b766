"""attention_paged_tree where its kernels' parts, turns and words of masks meet; bounds as in test_gpu_attention.py."""

from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import attnref  # noqa: E402
from test_gpu_attention import dev, w4  # noqa: E402, F401
from test_gpu_tree_attention import Tree, words_of  # noqa: E402


@pytest.mark.parametrize("d,e4m3", [(64, False), (64, True), (128, False), (128, True), (256, False), (256, True)])
@pytest.mark.parametrize("n", [3, 12, 16])
@pytest.mark.parametrize("old", [False, True])
def test_weights_of_few_rows_keep_22_bits(w4, d, e4m3, n, old):  # noqa: F811
    # of 16 rows at most.
    # Two keys of nearly the same score count, one with v = 1 and one with v = -1; all others have scores 16 or more below
    # theirs and v = 0.  So out = (a - b) / (a + b + the rest) is small, and its own rounding with it: 2^-11 of at most 0.032.
    # A row's a and b come from one score each: q0 k0 is exact (q and k are 0 elsewhere), times scale log2 e is off by three
    # roundings of a value below 1.45, less m (11 below the largest) one of a value below 16: 1.45 * 3 * 2^-24 + 2^-21 < 2^-20 in
    # all, times ln 2 of a weight; exp2 2^-21, two f16 2^-22.  Each is below 2^-19 off, so out below 2^-19, and the sums, of
    # 300 keys at most in blocks of 16 (which but for two weights are below 2^-23 of the largest), and the division
    # 2^-21 each.  Weights of 11 bits are off by 2^-12, and out by 2^-13.
    s = Tree([(n, n + 170)], 2, 2, d, 16, e4m3, seed=d + n, kind="tree", scales=False)
    rng = np.random.default_rng(d + n)
    # where the two stand: in a tile that all rows see whole, or among the new tokens, seen by every row (of itself and its sign)
    hot = (70, 77) if old else (170 + 1, 170 + 2)
    for t in range(n):
        s.sees[t] = s.sees[t] | {1, 2}
    s.mask = dev(words_of(s.sees, s.words))
    s.q[:] = 0
    s.q[..., 0] = rng.uniform(0.5, 1.0, (n, 2))
    code = {x: int(np.flatnonzero(attnref.e4m3_values() == x)[0]) for x in (0.0, 1.0, -1.0, 0.9375, -32.0)} if e4m3 else None

    def put(c, at, x):
        c[s.table[0, at // 16], :, at % 16, 0] = code[x] if e4m3 else x

    for c in s.host:
        c[s.table[0, :-(-(n + 170) // 16)]] = code[0.0] if e4m3 else 0.0
    for j in range(n + 170):
        put(s.host[0], j, -32.0)
    put(s.host[0], hot[0], 1.0), put(s.host[0], hot[1], 0.9375)
    for i in range(d):
        for at, x in zip(hot, (1.0, -1.0)):
            s.host[1][s.table[0, at // 16], :, at % 16, i] = code[x] if e4m3 else x
    s.dev = [s._place(c, "phtd") for c in s.host]
    got = s.run(w4, scale=1.0).cpu().numpy().astype(np.float64)
    want, size, _ = s.want(1.0)
    assert np.abs(want).max() <= 0.032 and size.max() <= 1
    err = np.abs(got - want)
    assert (err <= np.abs(want) * 2.0 ** -11 + 2.0 ** -19 + 2 * 2.0 ** -21).all(), err.max()


class Shared(Tree):
    """One head's keys, values and queries for `heads` kv heads (which share the cache's memory), so that few workgroups are left for
    the keys of each and the oracle has one head to do."""

    def __init__(self, lens, d, e4m3, heads, page=16, seed=0, group=1, **kw):
        super().__init__(lens, group, 1, d, page, e4m3, seed=seed, **kw)
        self.heads = heads

    def run(self, w4, **kw):
        kw = self.kw(**kw)
        for n in ("k_scale", "v_scale"):
            if n in kw:
                kw[n] = kw[n].repeat(self.heads)
        caches = [c.expand(-1, self.heads, -1, -1) for c in self.dev]
        self.need = w4.attention_workspace_bytes(caches[0], len(self.lens), self.q.shape[0], kw["max_q"], self.heads * self.hq,
                                                 self.table.shape[1], kw.get("window", 0), tree=True)
        q = dev(self.q).repeat(1, self.heads, 1)
        out = w4.attention_paged_tree(q, *caches, dev(self.table), dev(self.kv_len), self.mask[:, :self.words], **kw)
        out = out.view(-1, self.heads, self.hq, self.d)
        assert torch.equal(out, out[:, :1].expand_as(out))
        return out[:, 0]

    def turns(self, rows, waves):
        """32-key tiles that each wave takes at least: the workspace has a row of dims + 4 floats for each row of every part of
        a tile, and 16 bytes a tile."""
        tiles = sum(-(-n * self.hq // rows) for n, _ in self.lens)
        parts = (self.need - 16 * tiles) // (self.heads * rows * (self.d + 4) * 4) if self.need else tiles
        assert parts >= tiles
        # a tile has the parts that the others leave, at most
        return [int(kv) // (parts - tiles + 1) // (32 * waves) for _, kv in self.lens]


FORMS = [  # dims, e4m3, rows of a tile, waves, the most rows that this kernel takes
    (64, False, 64, 4, 96), (64, True, 64, 4, 96), (128, False, 64, 8, 64), (128, True, 64, 4, 96), (256, False, 32, 4, 64),
    (256, True, 32, 8, 96)]


@pytest.mark.parametrize("d,e4m3,rows,waves,most", FORMS)
@pytest.mark.parametrize("window", [False, True])
@pytest.mark.parametrize("page", [16, 7])
def test_many_turns_of_a_wave(w4, d, e4m3, rows, waves, most, window, page):  # noqa: F811
    # 17 rows and more: tiles that are fetched while others are multiplied, page numbers and buffers that come round again, maxima
    # that move from turn to turn; half full and full tiles, two tiles; with a window the first turn of some waves is not whole
    kv = 32 * waves * 24 + 75
    for i, (new, sharp) in enumerate([([24], 1.0), ([60], 8.0), ([most - 5], 1.0), ([20, 60], 8.0)]):
        s = Shared([(n, kv - 301 * j) for j, n in enumerate(new)], d, e4m3, 1024, page, seed=30 + i + d, kind="any", sharp=sharp)
        win = kv - 32 * waves * 3 + 11 if window else 0
        a = s.run(w4, window=win)
        assert min(s.turns(rows, waves)) >= 5, s.turns(rows, waves)
        s.check(a, window=win)


@pytest.mark.parametrize("d,e4m3,rows,waves,most", FORMS)
def test_many_turns_with_gaps(w4, d, e4m3, rows, waves, most):  # noqa: F811
    # the longest sequence beside others of one turn or none, and rows of two query heads
    kv = 32 * waves * 36 + 75
    s = Shared([(9, 9), (most // 2, kv), (2, 40), (0, 0), (30, 31)], d, e4m3, 512, 16, seed=40 + d, group=2, kind="any")
    s.check(s.run(w4))
    assert s.turns(rows, waves)[1] >= 5
    s.check(s.run(w4, window=200), window=200)


@pytest.mark.parametrize("d,e4m3", [(64, False), (64, True), (128, True), (256, True)])
@pytest.mark.parametrize("n", [65, 95, 96])
@pytest.mark.parametrize("old", [0, 20, 31, 407])
def test_the_second_word_of_a_mask(w4, d, e4m3, n, old):  # noqa: F811
    # 65 to 96 new tokens of a head each: tiles of keys whose bits lie in both words
    s = Tree([(n, n + old), (n - 31, n + old)], 2, 2, d, 16, e4m3, seed=n + old, kind="any")
    s.check(s.run(w4))
    s.check(s.run(w4, window=n + 3), window=n + 3)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("new", [12, 130])
@pytest.mark.parametrize("window,page", [(0, 16), (2900, 16), (0, 7)])
def test_many_turns_in_the_kernels_for_few_and_for_many(w4, d, e4m3, new, window, page):  # noqa: F811
    # two parts of 2500 keys or more: ten turns of two or four waves, or of 64 keys for all
    s = Shared([(new, 5075), (new // 2, 4800)], d, e4m3, 1024, page, seed=60 + d, kind="any", sharp=3.0)
    s.check(s.run(w4, window=window), window=window)


@pytest.mark.parametrize("new", [3, 30, 200])
@pytest.mark.parametrize("d,e4m3", [(64, False), (128, True), (256, False)])
def test_starts_that_fall_write_no_other_rows(w4, new, d, e4m3):  # noqa: F811
    # rows before and behind the call's, and the other heads of a wider row, keep what they hold
    s = Tree([(new, 700)] * 4, 4, 2, d, 16, e4m3, seed=50, kind="none")
    t = s.q.shape[0]
    for starts in ([0, t, 0, t, 0], [t, 0, t, 0, t], [-9, 2 ** 31 - 1, -2 ** 31, t, 5], [new, new, 0, t, t]):
        wide = torch.full((t + 64, 6, d), 9.0, dtype=torch.float16, device="cuda")
        s.run(w4, q_start=dev(np.array(starts, dtype=np.int32)), max_q=new, out=wide[32:32 + t, 1:5])
        torch.cuda.synchronize()
        assert (wide[:32] == 9).all() and (wide[32 + t:] == 9).all()
        assert (wide[:, 0] == 9).all() and (wide[:, 5] == 9).all()


@pytest.mark.parametrize("hq,hkv", [(4, 2), (32, 1), (130, 1)])
@pytest.mark.parametrize("b", [1, 3])
def test_a_batch_without_rows(w4, hq, hkv, b):  # noqa: F811
    # padding alone: nothing is written, whatever the workspace holds
    s = Tree([(0, 900)] * b, hq, hkv, 64, 16, seed=51)
    t = 7
    q = torch.randn((t, hq, 64), device="cuda", dtype=torch.float16)
    out = torch.full_like(q, 9.0)
    mask = torch.full((t, 1), -1, dtype=torch.int64, device="cuda")
    w4.attention_paged_tree(q, *s.dev, dev(s.table), dev(s.kv_len), mask, q_start=dev(s.starts), max_q=t, out=out,
                            workspace=torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda"))
    assert (out == 9).all()


@pytest.mark.parametrize("hq,hkv", [(4, 2), (16, 1), (32, 1), (130, 1)])
def test_one_row_each_without_starts(w4, hq, hkv):  # noqa: F811
    # of each kernel: 2, 16, 32 and 130 rows; a row sees itself, or only what is before it
    lens = [(1, 700), (1, 1), (1, 33), (1, 0), (1, 1)]
    s = Tree(lens, hq, hkv, 64, 16, seed=52)
    for bits in (1, 0, -2):  # (bits from 1 on are ignored)
        s.sees = [{0} if bits & 1 else set()] * len(lens)
        mask = torch.full((len(lens), 1), bits, dtype=torch.int64, device="cuda")
        for window in (0, 40):
            got = w4.attention_paged_tree(dev(s.q), *s.dev, dev(s.table), dev(s.kv_len), mask, window=window)
            s.check(got, window=window)


@pytest.mark.parametrize("new,hq", [(3, 2), (20, 2), (70, 4)])
def test_lengths_outside_the_table(w4, new, hq):  # noqa: F811
    # kept to 0 .. W * page size: below 0 nothing is cached, and past the table the pages that there are count
    s = Tree([(new, 96), (new, 50), (new, 64)], hq, 2, 64, 16, seed=53, kind="any")
    width = 6
    s.table = np.ascontiguousarray(s.table[:, :width])
    s.table[1] = s.table[0]
    given = np.array([2 ** 31 - 1, 97, -2 ** 31], dtype=np.int32)
    kept = np.array([96, 96, 0], dtype=np.int32)
    got = w4.attention_paged_tree(dev(s.q), *s.dev, dev(s.table), dev(given), s.mask[:, :s.words], q_start=dev(s.starts),
                                  max_q=new)
    s.kv_len = kept
    s.check(got)


@pytest.mark.parametrize("n,most", [(9, 8), (12, 3), (60, 24), (160, 40), (200, 97)])
@pytest.mark.parametrize("d,window", [(64, 0), (128, 300), (256, 0)])
def test_more_rows_than_max_q_stay_in_place(w4, n, most, d, window):  # noqa: F811
    # of the second sequence: it writes no rows but its own, whatever mask and kernel were chosen for fewer, and the others are right
    lens = [(min(most, 5), 700), (n, 900), (2, 90)]
    s = Tree(lens, 2, 2, d, 16, seed=54 + n, kind="any")
    t = s.q.shape[0]
    wide = torch.full((t + 64, 2, d), 9.0, dtype=torch.float16, device="cuda")
    got = s.run(w4, window=window, max_q=most, mask=s.mask[:, :-(-most // 64)].contiguous(), out=wide[32:32 + t])
    assert (wide[:32] == 9).all() and (wide[32 + t:] == 9).all()
    want, size, wobble = s.want(None, window)
    keep = np.r_[:lens[0][0], lens[0][0] + n:t]
    got = got.cpu().numpy().astype(np.float64)
    assert (np.abs(got - want) <= s.bound(want, size, wobble))[keep].all()


@pytest.mark.parametrize("lens,hq,hkv,d,e4m3", [
    ([(5, 4000), (3, 20)], 4, 2, 128, False), ([(20, 300), (7, 60)], 4, 2, 64, True), ([(20, 6000), (9, 900)], 4, 2, 128, False),
    ([(16, 5000)], 4, 2, 256, True), ([(100, 3000), (90, 90)], 4, 2, 64, False), ([(70, 100)], 4, 2, 256, False)])
def test_the_result_may_take_the_queries_place(w4, lens, hq, hkv, d, e4m3):  # noqa: F811
    # in each kernel, in one part and in many
    s = Tree(lens, hq, hkv, d, 16, e4m3, seed=d, kind="any")
    want = s.run(w4)
    rows = torch.full((s.q.shape[0], hq + 2, d), 5.0, device="cuda", dtype=torch.float16)
    q = rows[:, 1:hq + 1]
    q.copy_(dev(s.q))
    s.run(w4, q=q, out=q)
    assert torch.equal(q, want) and (rows[:, 0] == 5).all() and (rows[:, hq + 1] == 5).all()


@pytest.mark.parametrize("hq,hkv,d,e4m3,window", [(4, 2, 64, False, 0), (2, 2, 128, True, 0), (4, 2, 256, False, 900), (4, 4, 128, False, 300)])
@pytest.mark.parametrize("t", [6, 24, 60, 200])
def test_captured_trees_replay_through_their_parts(w4, t, hq, hkv, d, e4m3, window):  # noqa: F811
    # two graphs of one call, which share a workspace, replayed while starts, lengths and masks change: rows and keys are dealt out anew
    # each time, into one part and into many; against an eager call with a workspace of its own, and the oracle
    s = Tree([(t, 3200), (0, 3200), (0, 3200)], hq, hkv, d, 16, e4m3, seed=d + t)
    rng = np.random.default_rng(t)
    words = -(-t // 64)
    bits = rng.integers(-2 ** 63, 2 ** 63, (t, words))
    need = max(16, w4.attention_workspace_bytes(s.dev[0], 3, t, t, hq, s.table.shape[1], window, tree=True))  # (none in one part)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    q, table, kv_len, starts, mask = dev(s.q), dev(s.table), dev(s.kv_len), dev(s.starts), dev(bits)
    args = {**s.kw(), "q_start": starts, "max_q": t}
    outs = [torch.empty_like(q) for _ in range(2)]

    def call(o, **kw):
        w4.attention_paged_tree(q, *s.dev, table, kv_len, mask, window=window, out=o, **args, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(outs[0], workspace=ws[:need])
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g, o in zip(graphs, outs):
        with torch.cuda.graph(g):
            call(o, workspace=ws[:need])
    for i, lens in enumerate((
            [(t - 3, 3000), (2, 2000), (1, 5)], [(1, 3200), (t - 2, t - 2), (1, 0)], [(t, 3200), (0, 9), (0, 0)],
            [(t // 3, 20), (t // 3, 3200), (t // 4, 0)], [(0, 0), (0, 0), (0, 0)], [(2, 3000), (1, 1), (t - 4, 2900)])):
        s.lens = lens
        s.starts = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
        s.kv_len = np.array([kv for _, kv in lens], dtype=np.int32)
        s.sees = [{j for j in range(n) if bits[s.starts[b] + k, j // 64] >> (j % 64) & 1} for b, (n, _) in enumerate(lens) for k in range(n)]
        for a, x in ((kv_len, s.kv_len), (starts, s.starts), (mask, bits)):
            a.copy_(dev(x))
        for g, o in zip(graphs, outs):
            o.fill_(7.0)
            g.replay()
            torch.cuda.synchronize()
        eager = torch.full_like(q, 7.0)
        call(eager)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], eager) and torch.equal(outs[1], eager), i
        live = int(s.starts[-1])
        assert (eager[live:] == 7).all() and (ws[need:] == 0xFF).all()
        whole, s.q = s.q, s.q[:live]
        if live:
            s.check(eager[:live], window=window)
        s.q = whole
        bits = np.roll(bits, 1, axis=0)
