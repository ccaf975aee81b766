"""kv_plan against the oracle: whole numbers, equal in every place."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import stepref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_rope_append import dev, w4  # noqa: E402, F401


class State:
    """Sequences that hold the pages of `owned`, and a stack of the others."""

    def __init__(self, rng, seqs, width, page, owned, spare=10, pad=0):
        pages = int(np.sum(owned)) + spare
        order = rng.permutation(pages).astype(np.int32)
        self.page, self.width = page, width
        self.table = np.full((seqs, width), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(owned):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.owned = np.array(owned, dtype=np.int32)
        self.free = np.full(pages, 77, dtype=np.int32)
        self.free[:pages - at] = order[at:]
        self.count = pages - at
        wide = torch.full((seqs, width + pad), -7, dtype=torch.int32, device="cuda")
        self.wide, self.d_table = wide, wide[:, :width]
        self.d_table.copy_(dev(self.table))
        self.d_owned, self.d_free = dev(self.owned), dev(self.free)
        self.d_count = torch.tensor([self.count], dtype=torch.int32, device="cuda")

    def step(self, w4, kv_len, new_len, rows, depth=None, **kw):
        kv_len, new_len = np.asarray(kv_len, dtype=np.int32), np.asarray(new_len, dtype=np.int32)
        want = stepref.plan(kv_len, new_len, self.table, self.owned, self.free, self.count, self.page, rows, depth)
        out = w4.kv_plan(dev(kv_len), dev(new_len), self.d_table, self.d_owned, self.d_free, self.d_count, self.page, rows,
                         depth=None if depth is None else dev(np.asarray(depth, dtype=np.int32)), **kw)
        self.check(out, want)
        return out, want

    def check(self, out, want):
        for got, name in zip((*out, self.d_table, self.d_owned, self.d_free, self.d_count),
                             ("q_start", "kv_total", "pos", "slot", "status", "table", "owned", "free", "count")):
            assert np.array_equal(got.cpu().numpy().reshape(-1), np.array(want[name]).reshape(-1)), name
        self.table, self.owned = np.array(want["table"], dtype=np.int32), np.array(want["owned"], dtype=np.int32)
        self.free, self.count = np.array(want["free"], dtype=np.int32), want["count"]


@pytest.mark.parametrize("seqs,page,new", [(1, 1, 1), (1, 16, 100), (3, 16, 1), (64, 16, 1), (63, 5, 7), (65, 64, 40),
                                           (257, 16, 30), (1024, 8, 3), (1025, 8, 3), (2500, 16, 2)])
def test_steps_of_a_batch(w4, seqs, page, new):  # noqa: F811
    # a few steps: sequences grow, are cut back, end and start again
    rng = np.random.default_rng(seqs + page)
    width = 40 + 400 // page
    kv = rng.integers(0, 20 * page, seqs)
    s = State(rng, seqs, width, page, -(-kv // page), spare=seqs * (3 + new // page), pad=3)
    for step in range(4):
        n = rng.integers(0, new + 1, seqs) if step else np.full(seqs, new)
        rows = max(1, int(n.sum()) + [0, 5][step % 2])
        (_, total, _, _, status), _ = s.step(w4, kv, n, rows, rng.integers(0, 9, rows) if step == 2 else None)
        kv = total.cpu().numpy().copy()
        cut = rng.random(seqs)
        kv = np.where(cut < 0.2, 0, np.where(cut < 0.5, np.maximum(kv - rng.integers(0, new + 1, seqs), 0), kv))
    assert (s.wide[:, width:] == -7).all()


@pytest.mark.parametrize("seqs,spare", [(1, 0), (5, 1), (64, 7), (64, 0), (300, 40), (1500, 100)])
def test_a_stack_that_does_not_cover_the_step(w4, seqs, spare):  # noqa: F811
    rng = np.random.default_rng(seqs)
    kv = rng.integers(0, 60, seqs)
    s = State(rng, seqs, 30, 4, -(-kv // 4), spare=spare)
    n = rng.integers(0, 9, seqs)
    (_, total, _, _, status), want = s.step(w4, kv, n, max(1, int(n.sum())))
    if spare < seqs:
        assert max(want["status"]) > 0
    # what lacked is tried again when others have ended
    kv = total.cpu().numpy().copy()
    kv[::3] = 0
    n = np.where(status.cpu().numpy() > 0, n, 0)
    s.step(w4, kv, n, max(1, int(n.sum())))


def test_what_does_not_fit(w4):  # noqa: F811
    rng = np.random.default_rng(1)
    s = State(rng, 9, 6, 4, [1, 2, 0, 6, 1, 1, 0, 3, 0])
    big, low = 2 ** 31 - 1, -2 ** 31
    s.step(w4, [4, big, low, 24, -1, 2, 0, 10, 5], [1, 1, 1, 1, 3, low, big, 2, 2], 12)
    s = State(rng, 3, 4, 8, [1, 1, 1])
    s.step(w4, [8, 8, 8], [5, 6, 7], 11)  # rows of the last two do not fit
    s.step(w4, [8, 8, 8], [big, big, 1], 20)


def test_corrupt_state_stays_in_bounds(w4):  # noqa: F811
    # owned past the table, a height past the stack, entries that are no pages: bounded as written in w4.h
    rng = np.random.default_rng(2)
    s = State(rng, 4, 5, 4, [2, 3, 1, 2], spare=6)
    s.owned[:] = [9, -3, 1, 2 ** 31 - 1]
    s.d_owned.copy_(dev(s.owned))
    s.count = 99
    s.d_count.fill_(99)
    s.table[0, 0], s.table[2, 0] = -5, 2 ** 31 - 1
    s.d_table.copy_(dev(s.table))
    s.step(w4, [5, 6, 2, 3], [1, 4, 1, 1], 8)


def test_large_rows_and_long_tables(w4):  # noqa: F811
    rng = np.random.default_rng(3)
    for seqs, new in ((1, 5000), (3, 9000), (300, 31), (5000, 1), (4097, 3)):
        kv = rng.integers(0, 100, seqs)
        s = State(rng, seqs, 9200 // 16, 16, -(-kv // 16), spare=seqs * (new // 16 + 2))
        n = np.where(rng.random(seqs) < 0.3, 0, new)
        n[0] = new
        s.step(w4, kv, n, int(n.sum()) + 9, rng.integers(0, new, int(n.sum()) + 9))


def test_lengths_in_place_and_captured(w4):  # noqa: F811
    # kv_total is kv_len: a captured decode step advances by itself; every replay is compared with the oracle
    rng = np.random.default_rng(4)
    seqs, rows = 6, 8
    kv = np.array([3, 15, 16, 0, 31, 47], dtype=np.int32)
    s = State(rng, seqs, 8, 16, -(-kv // 16), spare=20)
    d_kv, n = dev(kv), np.array([1, 1, 1, 1, 1, 1], dtype=np.int32)
    d_n = dev(n)
    i32 = dict(dtype=torch.int32, device="cuda")
    out = (torch.empty(seqs + 1, **i32), d_kv, torch.empty(rows, **i32), torch.empty(rows, dtype=torch.int64, device="cuda"),
           torch.empty(seqs, **i32))

    def call():
        w4.kv_plan(d_kv, d_n, s.d_table, s.d_owned, s.d_free, s.d_count, 16, rows, out=out)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.current_stream())
        want = stepref.plan(kv, n, s.table, s.owned, s.free, s.count, 16, rows)
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    s.check(out, want)
    kv = np.array(want["kv_total"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(20):
        if i == 7:  # one is cut back, one ends
            kv[1], kv[2] = 5, 0
            d_kv.copy_(dev(kv.astype(np.int32)))
        want = stepref.plan(kv, n, s.table, s.owned, s.free, s.count, 16, rows)
        g.replay()
        torch.cuda.synchronize()
        s.check(out, want)
        kv = np.array(want["kv_total"])


def test_bindings_refuse(w4):  # noqa: F811
    rng = np.random.default_rng(5)
    s = State(rng, 3, 4, 8, [1, 1, 1])
    z = torch.zeros(3, dtype=torch.int32, device="cuda")
    ok = dict(kv_len=z, new_len=z, table=s.d_table, owned=s.d_owned, free=s.d_free, free_count=s.d_count, page_size=8, rows=4)
    w4.kv_plan(**ok)
    for bad in (dict(kv_len=z[:2]), dict(new_len=z.long()), dict(table=s.d_table.t()), dict(owned=z.cpu()), dict(free=None),
                dict(free_count=z), dict(depth=z), dict(free=s.d_free[::2]), dict(table=z),
                dict(out=(z, z, z, z.long(), z))):
        with pytest.raises((TypeError, ValueError, AttributeError)):
            w4.kv_plan(**{**ok, **bad})
    for bad in (dict(page_size=0), dict(rows=0), dict(page_size=1 << 30)):
        with pytest.raises((w4.W4Error, ValueError)):
            w4.kv_plan(**{**ok, **bad})


def test_pages_of_many_sequences_move_at_once(w4):  # noqa: F811
    # long sequences end and others take their places, some pages, many or none each
    rng = np.random.default_rng(6)
    for seqs in (3, 200, 256, 257, 1024, 1100):
        width = 300
        kv = rng.integers(0, width * 4 - 20, seqs)
        s = State(rng, seqs, width, 4, -(-kv // 4), spare=seqs * 40)
        for _ in range(3):
            kv = np.where(rng.random(seqs) < 0.4, rng.integers(0, width * 4 - 20, seqs), kv)
            n = rng.integers(0, 3, seqs)
            (_, total, _, _, _), _ = s.step(w4, kv, n, max(1, int(n.sum())))
            kv = total.cpu().numpy().copy()
