"""kv_plan, kv_append_norm_rope and logits_adjust at the ends of what their arguments may be, and in calls beside each other."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import stepref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_logits_adjust import Rules  # noqa: E402
from test_gpu_plan import State  # noqa: E402
from test_gpu_rope_append import dev, inputs, w4  # noqa: E402, F401


@pytest.mark.parametrize("seqs", [1, 3, 300, 1025])
def test_large_pages(w4, seqs):  # noqa: F811
    # a page of 2^28 tokens, tables of four: lengths up to 2^30, slots up to 2^31
    rng = np.random.default_rng(seqs)
    page = 1 << 28
    for kv, n in ((0, 1), (page - 1, 1), (page - 1, 2), (4 * page - 3, 3), (4 * page - 3, 4), (4 * page, 0), (4 * page, 1), (2 ** 31 - 1, 1)):
        s = State(rng, seqs, 4, page, [min(4, -(-kv // page))] + [0] * (seqs - 1), spare=2)
        given = np.zeros(seqs, dtype=np.int64)
        rows = np.zeros(seqs, dtype=np.int64)
        given[0], rows[0] = kv, n
        s.step(w4, given, rows, 5)


def test_long_tables_of_single_tokens(w4):  # noqa: F811
    # pages of one token: a sequence that takes and gives back many at once, alone and beside others
    rng = np.random.default_rng(3)
    for seqs, width in ((1, 70000), (5, 70000), (1030, 2000)):
        s = State(rng, seqs, width, 1, [0] * seqs, spare=width + 10)
        kv, n = np.zeros((2, seqs), dtype=np.int64)
        n[0] = width - 1
        s.step(w4, kv, n, width + 5)
        kv[0], n[0] = width - 1, 1
        s.step(w4, kv, n, 3)
        kv[0], n[0] = 2, 1
        kv[-1], n[-1] = (0, width - 7) if seqs > 1 else (2, 1)
        s.step(w4, kv, n, width)


@pytest.mark.parametrize("inter,r", [(False, 128), (True, 128), (False, 58)])
def test_queries_normed_in_place(w4, inter, r):  # noqa: F811
    # q_out is q, a column block of the projection's rows; k and v stay as they are
    t, hq, hkv, d = 37, 6, 2, 128
    x, pos, freq = inputs(t, hq + 2 * hkv, d, r, False, 5)
    rng = np.random.default_rng(r)
    wq, wk = (dev(w) for w in rng.standard_normal((2, d)).astype(np.float32))
    out = []
    for place in (False, True):
        rows = dev(x)
        kc, vc = (torch.zeros((5, hkv, 8, d), dtype=torch.float16, device="cuda") for _ in range(2))
        q = rows[:, :hq]
        got = w4.kv_append_norm_rope(rows[:, hq:hq + hkv], rows[:, hq + hkv:], kc, vc, torch.arange(t, device="cuda"), dev(pos), dev(freq),
                                     wk, q=q, q_weight=wq, q_out=q if place else None, interleaved=inter)
        assert torch.equal(rows[:, hq:], dev(x)[:, hq:])
        out.append((got.clone(), kc, vc))
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_calls_on_two_streams(w4):  # noqa: F811
    rng = np.random.default_rng(9)
    r = [Rules(9, 20000, 4, 700, 20, "row", seed=s) for s in (1, 2)]
    x, kw = [dev(a.logits) for a in r], [a.kw() for a in r]
    t, pages = 300, 40
    rows = [torch.randn((t, 8, 64), device="cuda") for _ in range(2)]
    pos = torch.arange(t, dtype=torch.int32, device="cuda")
    freq, _ = w4.rope_frequencies(64, 1e4)
    weight = torch.rand(64, device="cuda") + 0.5
    kv, new = (rng.integers(0, 90, (2, 50)), rng.integers(0, 6, (2, 50)))
    order = dev(rng.permutation(2000).astype(np.int32))

    def all_of(i):
        caches = [torch.zeros((pages, 2, 8, 64), dtype=torch.float16, device="cuda") for _ in range(2)]
        q = w4.kv_append_norm_rope(rows[i][:, 4:6], rows[i][:, 6:], *caches, torch.arange(t, device="cuda"), pos, freq, weight,
                                   q=rows[i][:, :4], q_weight=weight)
        table = torch.full((50, 12), -1, dtype=torch.int32, device="cuda")
        owned, free = torch.zeros(50, dtype=torch.int32, device="cuda"), order.clone()
        count = torch.full((1,), 2000, dtype=torch.int32, device="cuda")
        plan = w4.kv_plan(kv_dev[i], new_dev[i], table, owned, free, count, 8, 260)
        return [w4.logits_adjust(x[i], **kw[i]), q, *caches, *plan, table, owned, free, count]

    kv_dev, new_dev = ([dev(a.astype(np.int32)) for a in y] for y in (kv, new))
    want = [all_of(0), all_of(1)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(3):
        for i, st in enumerate(streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append((i, all_of(i)))
    torch.cuda.synchronize()
    for i, g in got:
        for a, b in zip(g, want[i]):
            assert torch.equal(a, b)
    r[0].check(want[0][0])
    p = stepref.plan(kv[0], new[0], np.full((50, 12), -1), [0] * 50, order.cpu().numpy(), 2000, 8, 260)
    assert want[0][8].tolist() == p["status"] and want[0][7].tolist() == p["slot"]
