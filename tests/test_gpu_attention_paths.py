"""attention_paged over the ways its work is cut: many sequences, windows that end inside a page, tiles of 64 and
of 128 rows in one part and in several; bounds as in test_gpu_attention.py."""

from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_attention import Setup, dev, w4  # noqa: E402, F401


@pytest.mark.parametrize("n,kv,window,hq,hkv,d,page,e4m3", [
    # the window's first key is not a multiple of 16, so a part more than the window alone would need
    (16, 1000, 240, 1, 1, 64, 16, False), (16, 1000, 240, 2, 2, 128, 16, True), (15, 999, 241, 1, 1, 64, 16, False),
    (16, 1001, 496, 1, 1, 128, 8, False), (8, 1003, 247, 2, 1, 256, 16, False), (3, 1003, 254, 4, 1, 64, 100, True),
    (1, 1007, 256, 4, 1, 64, 16, False), (1, 1000, 257, 1, 1, 96, 5, False),
])
def test_window_from_the_middle_of_a_page(w4, n, kv, window, hq, hkv, d, page, e4m3):  # noqa: F811
    for lens in ([(n, kv)], [(n, kv + i) for i in range(5)], [(n, kv), (n, 3), (n, kv + 1)]):
        s = Setup(lens, hq, hkv, d, page, e4m3, seed=n + kv + len(lens))
        s.check(s.run(w4, window=window), window=window)


@pytest.mark.parametrize("hq,hkv,d,e4m3", [(4, 2, 64, False), (2, 1, 256, False), (2, 2, 128, True)])
@pytest.mark.parametrize("b", [129, 300, 700])
def test_many_sequences_decode(w4, b, hq, hkv, d, e4m3):  # noqa: F811
    rng = np.random.default_rng(b + d)
    kv = rng.integers(0, 60, b)
    kv[[0, b // 2, b - 1]] = 700, 300, 0
    s = Setup([(1, int(x)) for x in kv], hq, hkv, d, 16, e4m3, seed=b)
    s.check(s.run(w4))
    s.check(s.run(w4, window=33), window=33)


@pytest.mark.parametrize("hq,hkv,d,e4m3", [(4, 2, 64, False), (2, 1, 256, True), (16, 2, 128, False)])
def test_many_sequences_mixed(w4, hq, hkv, d, e4m3):  # noqa: F811
    rng = np.random.default_rng(d)
    n = rng.integers(0, 4, 300)
    n[[3, 70, 140, 299]] = 90, 33, 0, 40
    lens = [(int(a), int(a + rng.integers(0, 90))) for a in n]
    s = Setup(lens, hq, hkv, d, 16, e4m3, seed=d + 1)
    s.check(s.run(w4))


@pytest.mark.parametrize("lens,hq,hkv,d,page,window,e4m3", [
    # 64 rows a tile: one part; three; two at 256 dims; pages that no wave's rows fit
    ([(300, 300)], 32, 8, 64, 16, 0, False), ([(300, 2000)], 16, 2, 128, 16, 0, False),
    ([(300, 2000)], 16, 2, 128, 16, 0, True), ([(500, 1500)], 16, 2, 256, 64, 0, False),
    ([(500, 1400)], 16, 2, 256, 64, 0, True), ([(260, 2500)], 32, 4, 64, 8, 0, True),
    ([(120, 700), (121, 800), (122, 650)], 32, 8, 64, 12, 0, False), ([(300, 1500)], 48, 8, 128, 16, 700, False),
    ([(200, 900)], 32, 16, 256, 16, 333, True), ([(400, 3000)], 16, 1, 104, 20, 0, False),
    # 128 rows: one part; three at 256 dims; two of few dims
    ([(700, 900), (650, 700)], 32, 8, 128, 16, 0, False), ([(700, 900), (650, 700)], 32, 8, 128, 16, 250, True),
    ([(700, 1000)], 32, 8, 112, 7, 0, False), ([(150, 2000)], 64, 8, 256, 16, 0, False),
    ([(150, 2000)], 64, 8, 256, 24, 0, True), ([(64, 6000)], 512, 128, 8, 16, 0, False),
])
def test_tiles_and_parts(w4, lens, hq, hkv, d, page, window, e4m3):  # noqa: F811
    s = Setup(lens, hq, hkv, d, page, e4m3, seed=d + len(lens))
    a = s.run(w4, window=window)
    s.check(a, window=window)
    assert torch.equal(a, s.run(w4, window=window))


def test_decode_step_of_a_padded_batch(w4):  # noqa: F811
    # rows of no sequence: slot -1, no cached tokens, anything in q, k and v.  They get zeros and touch nothing
    d, hq, hkv, page, b = 64, 4, 2, 16, 6
    gen = torch.Generator(device="cuda").manual_seed(3)
    kc, vc = (torch.randn((8, hkv, page, d), device="cuda", generator=gen, dtype=torch.float16) for _ in range(2))
    qkv = torch.randn((b, hq + 2 * hkv, d), device="cuda", generator=gen)
    lens = torch.tensor([20, 0, 33, 0, 1, 0], dtype=torch.int32, device="cuda")
    table = torch.tensor([[0, 1, -1], [-1] * 3, [2, 3, 4], [9, 9, 9], [5, -1, -1], [0, 1, 2]], dtype=torch.int32,
                         device="cuda")
    slots = torch.tensor([1 * page + 3, -1, 4 * page, -1, 5 * page, -1], device="cuda")
    pos = (lens - 1).clamp_min(0)
    freq, mscale = w4.rope_frequencies(d)
    live = lens > 0

    def step(qkv, rows):
        k2, v2 = kc.clone(), vc.clone()
        q = w4.kv_append_rope(qkv[rows][:, hq:hq + hkv], qkv[rows][:, hq + hkv:], k2, v2, slots[rows], pos[rows], freq,
                              q=qkv[rows][:, :hq], mscale=mscale)
        return w4.attention_paged(q, k2, v2, table[rows], lens[rows]), k2, v2

    want, wk, wv = step(qkv, live)
    qkv[~live] = float("nan")
    got, gk, gv = step(qkv, torch.ones_like(live))
    assert torch.equal(got[live], want) and (got[~live] == 0).all()
    assert torch.equal(gk, wk) and torch.equal(gv, wv)


def test_a_prompt_in_chunks_is_the_prompt_at_once(w4):  # noqa: F811
    # append and attention of 300 tokens at once, and of 1, 17, 100 and 182 after each other: the caches bit by bit,
    # the rows to two f16 roundings of a result and of the weights
    d, hq, hkv, page, t = 128, 8, 2, 16, 300
    gen = torch.Generator(device="cuda").manual_seed(4)
    qkv = torch.randn((t, hq + 2 * hkv, d), device="cuda", generator=gen)
    freq, mscale = w4.rope_frequencies(d, 1e6)
    table = torch.randperm(24, device="cuda", generator=gen).to(torch.int32)[None, :19].contiguous()
    pos = torch.arange(t, dtype=torch.int32, device="cuda")
    slots = table[0, (pos // page).long()].long() * page + pos % page
    outs, caches = [], []
    for cuts in ([0, 300], [0, 1, 18, 118, 300]):
        kc, vc = (torch.zeros((24, hkv, page, d), dtype=torch.float16, device="cuda") for _ in range(2))
        rows = []
        for a, e in zip(cuts, cuts[1:]):
            q = w4.kv_append_rope(qkv[a:e, hq:hq + hkv], qkv[a:e, hq + hkv:], kc, vc, slots[a:e], pos[a:e], freq,
                                  q=qkv[a:e, :hq], mscale=mscale)
            rows.append(w4.attention_paged(q, kc, vc, table, torch.tensor([e], dtype=torch.int32, device="cuda"),
                                           q_start=torch.tensor([0, e - a], dtype=torch.int32, device="cuda"),
                                           max_q=e - a))
        outs.append(torch.cat(rows))
        caches.append((kc, vc))
    assert torch.equal(caches[0][0], caches[1][0]) and torch.equal(caches[0][1], caches[1][1])
    # each side: 2^-11 of the result, 2^-11 of the mean |v| (at most max |v|) for the weights
    top = caches[0][1].abs().max().float()
    assert (outs[0].float() - outs[1].float()).abs().max() <= 4 * 2.0 ** -11 * top


def test_append_and_attention_on_another_stream(w4):  # noqa: F811
    # two streams, each with its cache; the calls go to the stream that is current
    d, hq, hkv, page = 64, 4, 1, 16
    gen = torch.Generator(device="cuda").manual_seed(5)
    freq, mscale = w4.rope_frequencies(d)
    data = []
    for i in range(2):
        qkv = torch.randn((200, hq + 2 * hkv, d), device="cuda", generator=gen)
        caches = [torch.zeros((13, hkv, page, d), dtype=torch.float16, device="cuda") for _ in range(2)]
        data.append((qkv, *caches, torch.arange(13, dtype=torch.int32, device="cuda")[None],
                     torch.arange(200, device="cuda"), torch.arange(200, dtype=torch.int32, device="cuda"),
                     torch.tensor([200], dtype=torch.int32, device="cuda"),
                     torch.tensor([0, 200], dtype=torch.int32, device="cuda")))

    def run(qkv, kc, vc, table, slots, pos, n, starts):
        q = w4.kv_append_rope(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], kc, vc, slots, pos, freq, q=qkv[:, :hq],
                              mscale=mscale)
        return w4.attention_paged(q, kc, vc, table, n, q_start=starts, max_q=200)

    want = [run(*x) for x in data]
    for x in data:
        x[1].zero_(), x[2].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s, x in zip(streams, data):
        with torch.cuda.stream(s):
            got.append(run(*x))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("hq,hkv,d,e4m3", [(4, 2, 64, False), (2, 1, 256, False), (2, 2, 128, True)])
@pytest.mark.parametrize("b", [129, 300, 700])
def test_many_sequences_and_long_ones(w4, b, hq, hkv, d, e4m3):  # noqa: F811
    # the keys of all sequences are dealt out in parts, to workgroups that look at one or several sequences a thread
    rng = np.random.default_rng(b + d)
    kv = rng.integers(0, 40, b)
    kv[[0, b // 2, b - 1]] = 300, 2500, 1100
    s = Setup([(1, int(x)) for x in kv], hq, hkv, d, 16, e4m3, seed=b)
    s.check(s.run(w4))
    lens = [(int(a), int(a + x)) for a, x in zip(rng.integers(0, 3, b), kv)]
    s = Setup(lens, hq, hkv, d, 16, e4m3, seed=b + 1)
    s.check(s.run(w4))


@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (2, 2, 128), (16, 2, 256)])
def test_a_sequence_longer_than_max_q_leaves_the_others_theirs(w4, hq, hkv, d):  # noqa: F811
    # rows past max_q of a sequence are unspecified; the first max_q of each are right
    for lens, max_q in (([(300, 300), (50, 70), (60, 60), (2, 90)], 60), ([(40, 900), (1, 700), (1, 3)], 1),
                        ([(90, 95), (3, 40), (200, 210)], 3)):
        s = Setup(lens, hq, hkv, d, 16, seed=d)
        got = s.run(w4, max_q=max_q).cpu().numpy().astype(np.float64)
        want, size, wobble = s.want()
        keep = np.concatenate([a + np.arange(min(n, max_q)) for a, (n, _) in zip(s.starts, lens)])
        assert (np.abs(got - want) <= s.bound(want, size, wobble))[keep].all()
