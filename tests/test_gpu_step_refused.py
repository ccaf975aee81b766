"""A step of which kv_plan refuses some sequences: the others' rows and the whole cache are as if the refused had no rows."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import attnref, stepref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_rope_append import dev, w4  # noqa: E402, F401

HQ, HKV, D, PAGE, WIDTH = 4, 2, 64, 8, 12


@pytest.mark.parametrize("new", [3, 20, 60])
@pytest.mark.parametrize("e4m3", [False, True])
def test_a_step_with_refused_sequences(w4, new, e4m3):  # noqa: F811
    # five sequences: the second lacks pages (those behind it lack none), the fourth is longer than its table
    rng = np.random.default_rng(new)
    kv = np.array([9, 16, 24, PAGE * WIDTH, 3], dtype=np.int32)
    n = np.array([new, new + 8, 0, 2, 1], dtype=np.int32)
    pages = 50
    table = np.full((5, WIDTH), -1, dtype=np.int32)
    order = rng.permutation(pages)
    owned, at = [-(-(9 + new) // PAGE), 2, 3, WIDTH, 1], 0
    for b, k in enumerate(owned):
        table[b, :k] = order[at:at + k]
        at += k
    free = np.concatenate([order[at:], order[:at]]).astype(np.int32)
    count = 0  # of free pages: the first sequence has what it needs, the second lacks some
    rows = int(n.sum()) + 2
    want = stepref.plan(kv, n, table, owned, free, count, PAGE, rows)
    assert want["status"][0] == 0 and want["status"][1] > 0 and want["status"][2:] == [0, -1, 0]
    d_table = dev(table)
    plan = w4.kv_plan(dev(kv), dev(n), d_table, dev(np.array(owned, dtype=np.int32)), dev(free),
                      torch.tensor([count], dtype=torch.int32, device="cuda"), PAGE, rows)
    q_start, kv_total, pos, slots, status = plan
    for got, name in zip((*plan, d_table), ("q_start", "kv_total", "pos", "slot", "status", "table")):
        assert np.array_equal(got.cpu().numpy().reshape(-1), np.array(want[name]).reshape(-1)), name
    # a refused sequence keeps its length and has no slots: its rows do not stand where the plan's lengths say
    assert want["kv_total"][1] == kv[1] and want["kv_total"][3] == kv[3]

    held = [rng.standard_normal((pages, HKV, PAGE, D)) for _ in range(2)]
    held = [attnref.e4m3_round(x * 30) if e4m3 else x.astype(np.float16) for x in held]
    caches = [dev(x).view(torch.float8_e4m3fn) if e4m3 else dev(x) for x in held]
    scales = dict(k_scale=torch.full((HKV,), 0.03, device="cuda"), v_scale=torch.full((HKV,), 0.03, device="cuda")) if e4m3 else {}
    x = dev(rng.standard_normal((rows, HQ + 2 * HKV, D)).astype(np.float16))
    freq, _ = w4.rope_frequencies(D, 1e4)
    q = w4.kv_append_norm_rope(x[:, HQ:HQ + HKV], x[:, HQ + HKV:], *caches, slots, pos, freq, None, q=x[:, :HQ], **scales)
    # nothing but the accepted rows' slots has changed
    after = [c.view(torch.uint8).cpu().numpy() if e4m3 else c.cpu().numpy() for c in caches]
    mine = np.zeros((pages, PAGE), dtype=bool)
    for s in want["slot"]:
        if s >= 0:
            mine[s // PAGE, s % PAGE] = True
    for a, b in zip(held, after):
        same = (a.view(np.uint8) == b.view(np.uint8)).reshape(pages, HKV, PAGE, -1).all(-1)
        assert same[np.broadcast_to(~mine[:, None, :], same.shape)].all()
        assert not same[np.broadcast_to(mine[:, None, :], same.shape)].all()

    sees = [set(range(i + 1)) for b in range(5) for i in range(n[b])]
    words = -(-int(n.max()) // 64)
    mask = np.zeros((rows, words), dtype=np.uint64)
    for t, s in enumerate(sees):
        for j in s:
            mask[t, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    out = torch.full((rows, HQ, D), 9.0, dtype=torch.float16, device="cuda")
    w4.attention_paged_tree(q, *caches, d_table, kv_total, dev(mask.view(np.int64)), q_start=q_start, max_q=int(n.max()), out=out,
                            **scales)
    values = [attnref.e4m3_values()[c] if e4m3 else c.astype(np.float64) for c in after]
    sc = np.full(HKV, 0.03, dtype=np.float32) if e4m3 else None
    keep = np.concatenate([np.arange(want["q_start"][b], want["q_start"][b + 1]) for b in (0, 4)])
    # the oracle's tables: the refused have no rows
    alone = [0, n[0], n[0], n[0], n[0], n[0] + 1]
    ref, size, wobble = stepref.attention(q.cpu().numpy()[keep], *values, want["table"], want["kv_total"], alone,
                                          [sees[t] for t in keep], scale=D ** -0.5, k_scale=sc, v_scale=sc)
    # counted as in test_gpu_attention.py
    keys, top = max(want["kv_total"]), max(np.abs(v[np.isfinite(v)]).max() for v in values) * (0.03 if e4m3 else 1.0)
    lim = (np.abs(ref) * 2.0 ** -11 + 2.0 ** -25 + keys * 2.0 ** -25 * top +
           size * (2.0 ** -11 + 2 * wobble[..., None] * (D + 8) * 2.0 ** -24 + 2.0 ** -20 + (keys / 16 + 32) * 2.0 ** -23))
    err = np.abs(out.cpu().numpy().astype(np.float64)[keep] - ref)
    assert (err <= lim).all(), (err / lim).max()
    assert (out[-2:] == 9).all()  # padding
