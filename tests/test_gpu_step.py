"""Decode steps with drafted tokens from end to end: kv_plan, kv_append_norm_rope, attention_paged_tree, the projections around
them, logits_adjust and logits_argmax_topk, each stage against the oracle on its own inputs, over steps that accept a part of
what was drafted; and the step captured into one graph."""

from __future__ import annotations

import numpy as np
import pytest

import oracle
import synth
from oracle import attnref, stepref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_norm_rope import close_f16, sizes  # noqa: E402
from test_gpu_rope_append import dev, w4  # noqa: E402, F401

HIDDEN, HQ, HKV, D, PAGE, WIDTH, VOCAB, EPS = 256, 4, 2, 64, 8, 12, 3001, 1e-6


class Engine:
    """Weights, caches and the state of three requests."""

    def __init__(self, w4, seed, e4m3):
        rng = np.random.default_rng(seed)
        self.w4, self.rng, self.e4m3 = w4, rng, e4m3
        n = (HQ + 2 * HKV) * D
        qw, sc, bi = synth.w4_weights(n, HIDDEN, seed=seed)
        self.qkv = (w4.w4_pack(dev(qw)), dev(sc), dev(bi))
        self.head_host = synth.head_f16(HQ * D, VOCAB + 7, seed=seed)[:, :VOCAB + 7]
        self.head = dev(self.head_host)
        self.wq, self.wk = rng.uniform(0.5, 1.5, (2, D)).astype(np.float32)
        self.freq, _ = w4.rope_frequencies(D, 1e4)
        self.pages = 40
        kind = torch.float8_e4m3fn if e4m3 else torch.float16
        self.kc, self.vc = (torch.zeros((self.pages, HKV, PAGE, D), device="cuda").to(kind) for _ in range(2))
        self.scales = dict(k_scale=torch.full((HKV,), 0.02, device="cuda"),
                           v_scale=torch.full((HKV,), 0.02, device="cuda")) if e4m3 else {}
        self.table = torch.full((3, WIDTH), -1, dtype=torch.int32, device="cuda")
        self.owned = torch.zeros(3, dtype=torch.int32, device="cuda")
        self.free = dev(rng.permutation(self.pages).astype(np.int32))
        self.count = torch.tensor([self.pages], dtype=torch.int32, device="cuda")
        self.kv = np.zeros(3, dtype=np.int32)
        self.history = np.zeros((3, 64), dtype=np.int32)
        self.length = np.zeros(3, dtype=np.int32)

    def values(self, c):
        host = c.view(torch.uint8).cpu().numpy() if self.e4m3 else c.cpu().numpy()
        return attnref.e4m3_values()[host] if self.e4m3 else host.astype(np.float64)

    def step(self, parents):
        """One pass over the sequences' new tokens (parents[b]: their trees); returns what was chosen for each row."""
        w4, t = self.w4, sum(map(len, parents))
        rows = t + 2  # two rows of padding
        new = np.array([len(p) for p in parents], dtype=np.int32)
        masks = [w4.tree_mask(p) for p in parents]
        mask = torch.zeros((rows, 1), dtype=torch.int64)
        depth = torch.zeros(rows, dtype=torch.int32)
        at = 0
        for m, d in masks:
            if len(d):
                mask[at:at + len(d)], depth[at:at + len(d)] = m, d
            at += len(d)
        before = [x.cpu().numpy().copy() for x in (self.table, self.owned, self.free, self.count)]
        plan = w4.kv_plan(dev(self.kv), dev(new), self.table, self.owned, self.free, self.count, PAGE, rows,
                          depth=depth.cuda())
        q_start, kv_total, pos, slots, status = plan
        want = stepref.plan(self.kv, new, before[0], before[1], before[2], before[3][0], PAGE, rows, depth.numpy())
        for got, name in zip((q_start, kv_total, pos, slots, status, self.table, self.owned, self.count),
                             ("q_start", "kv_total", "pos", "slot", "status", "table", "owned", "count")):
            assert np.array_equal(got.cpu().numpy().reshape(-1), np.array(want[name]).reshape(-1)), name
        assert want["status"] == [0, 0, 0]

        x = self.rng.standard_normal((rows, HIDDEN)).astype(np.float16)
        qkv = w4.gemm_f16(dev(x), w4.w4_dequant_f16_t(*self.qkv)).view(rows, HQ + 2 * HKV, D)
        q = w4.kv_append_norm_rope(qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], self.kc, self.vc, slots, pos, self.freq,
                                   dev(self.wk), q=qkv[:, :HQ], q_weight=dev(self.wq), eps=EPS, **self.scales)
        host = qkv.cpu().numpy()
        n = stepref.norm(host[:, :HQ], self.wq, EPS)
        close_f16(q.cpu().numpy(), attnref.rope(n, pos.cpu().numpy(), self.freq.cpu().numpy()), sizes(n, D, False, 1.0))

        sees, at = [], 0
        for p in parents:
            bits = mask[at:at + len(p), 0].numpy().view(np.uint64)
            sees += [{j for j in range(len(p)) if int(b) >> j & 1} for b in bits]
            at += len(p)
        out = torch.zeros((rows, HQ, D), dtype=torch.float16, device="cuda")
        w4.attention_paged_tree(q, self.kc, self.vc, self.table, kv_total, mask.cuda(), q_start=q_start, max_q=int(new.max()),
                                out=out, **self.scales)
        ks, vs = (s.cpu().numpy() for s in self.scales.values()) if self.scales else (None, None)
        k, v = self.values(self.kc), self.values(self.vc)
        ref, size, wobble = stepref.attention(q.cpu().numpy()[:t], k, v, self.table.cpu().numpy(), want["kv_total"],
                                              want["q_start"], sees, scale=D ** -0.5, k_scale=ks, v_scale=vs)
        keys, top = max(want["kv_total"]), np.abs(v[np.isfinite(v)]).max() * (1.0 if vs is None else 0.02)
        lim = (np.abs(ref) * 2.0 ** -11 + 2.0 ** -25 + keys * 2.0 ** -25 * top +
               size * (2.0 ** -11 + 2 * wobble[..., None] * (D + 8) * 2.0 ** -24 + 2.0 ** -20 + (keys / 16 + 32) * 2.0 ** -23))
        err = np.abs(out.cpu().numpy()[:t] - ref)
        assert (err <= lim).all(), (err / lim).max()
        assert (out[t:] == 0).all()

        logits = w4.gemm_f16(out[:t].view(t, HQ * D), self.head)[:, :VOCAB]
        y, bound = oracle.gemm_ref(out[:t].cpu().numpy().reshape(t, HQ * D), self.head_host)
        assert oracle.check_bound(logits.cpu().numpy(), y[:, :VOCAB], bound[:, :VOCAB])[0]
        request = np.repeat(np.arange(3), new).astype(np.int32)
        allowed = self.rng.random((t, VOCAB)) < 0.3
        words = -(-VOCAB // 32)
        bits = np.zeros((t, 32 * words), dtype=bool)
        bits[:, :VOCAB] = allowed
        grammar = (bits.reshape(t, words, 32) * (np.uint64(1) << np.arange(32, dtype=np.uint64))).sum(-1).astype(np.uint32)
        r, f, p = self.rng.uniform(1.0, 1.5, 3).astype(np.float32), np.full(3, 0.3, np.float32), np.full(3, 0.1, np.float32)
        given = w4.logits_adjust(logits, tokens=dev(self.history), token_len=dev(self.length), repetition=dev(r),
                                 frequency=dev(f), presence=dev(p), request=dev(request), mask=dev(grammar.view(np.int32)))
        ref, size = stepref.adjust(logits.cpu().numpy(), request, self.history, self.length, None, r, f, p, None,
                                   [set(np.flatnonzero(a).tolist()) for a in allowed])
        got = given.cpu().numpy()
        assert np.array_equal(np.isneginf(got), ~allowed)
        assert (np.abs(got[allowed] - ref[allowed]) <= size[allowed] * 5 * 2.0 ** -24).all()
        idx, _ = w4.logits_argmax_topk(given, 5)
        assert np.array_equal(idx.cpu().numpy(), np.argsort(-got, axis=1, kind="stable")[:, :5])
        return plan, qkv, idx.cpu().numpy()

    def accept(self, plan, qkv, paths):
        """Keeps the tokens paths[b] of each sequence's new ones, in order: they are appended anew where they belong."""
        q_start, _, pos, _, _ = (x.cpu().numpy() for x in plan)
        rows = np.concatenate([q_start[b] + np.array(p, dtype=np.int64) for b, p in enumerate(paths)]).astype(np.int64)
        table = self.table.cpu().numpy()
        at = np.concatenate([self.kv[b] + np.arange(len(p)) for b, p in enumerate(paths)])
        seq = np.repeat(np.arange(3), [len(p) for p in paths])
        assert np.array_equal(pos[rows], at)  # a path's depths follow each other
        slots = table[seq, at // PAGE].astype(np.int64) * PAGE + at % PAGE
        part = qkv[dev(rows)]
        self.w4.kv_append_norm_rope(part[:, HQ:HQ + HKV], part[:, HQ + HKV:], self.kc, self.vc, dev(slots),
                                    dev(at.astype(np.int32)), self.freq, dev(self.wk), eps=EPS, **self.scales)
        for b, p in enumerate(paths):
            self.kv[b] += len(p)
            for _ in p:
                self.history[b, self.length[b] % 64] = self.rng.integers(0, VOCAB)
                self.length[b] = min(self.length[b] + 1, 64)


@pytest.mark.parametrize("e4m3", [False, True])
def test_steps(w4, e4m3):  # noqa: F811
    e = Engine(w4, 31, e4m3)
    prompts = [20, 5, 11]
    plan, qkv, _ = e.step([list(range(-1, n - 1)) for n in prompts])
    e.accept(plan, qkv, [list(range(n)) for n in prompts])
    # trees; a path through each is kept: 0 - 2 - 4, nothing, 1
    plan, qkv, _ = e.step([[-1, -1, 0, 0, 2, 2, 4], [-1, 0, 1], [-1, -1, 1, 2, 0]])
    e.accept(plan, qkv, [[0, 2, 4], [], [1]])
    assert e.kv.tolist() == [23, 5, 12]
    # one ends and another takes its place; single tokens beside it
    e.kv[0], e.length[0] = 0, 0
    plan, qkv, _ = e.step([list(range(-1, 17)), [-1], [-1, 0, 0, 1, 1, 2, 2, 3, 3]])
    e.accept(plan, qkv, [list(range(18)), [0], [0, 2, 5]])
    e.step([[-1], [-1], [-1]])


def test_a_captured_step(w4):  # noqa: F811
    # plan, append, attention and logits in one graph: lengths advance on the device; each replay against eager calls on
    # copies of the same state
    rng = np.random.default_rng(33)
    b, rows, v = 3, 12, 1000
    parents = [[-1, 0, 0], [-1, -1, 1, 2], [-1, 0]]
    new = dev(np.array([3, 4, 2], dtype=np.int32))
    mask = torch.zeros((rows, 1), dtype=torch.int64)
    depth = torch.zeros(rows, dtype=torch.int32)
    at = 0
    for p in parents:
        m, d = w4.tree_mask(p)
        mask[at:at + len(p)], depth[at:at + len(p)] = m, d
        at += len(p)
    mask, depth = mask.cuda(), depth.cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    freq, _ = w4.rope_frequencies(D, 1e4)
    weight = torch.ones(D, device="cuda")
    head = torch.randn((HQ * D, v), device="cuda", dtype=torch.float16)
    tokens, lens = torch.randint(0, v, (b, 30), **i32), torch.full((b,), 30, **i32)
    request = torch.tensor([0] * 3 + [1] * 4 + [2] * 2 + [0] * 3, **i32)
    one = torch.full((b,), 1.3, device="cuda")

    def state():
        return dict(kv=torch.tensor([5, 0, 15], **i32), table=torch.full((b, 16), -1, **i32), owned=torch.zeros(b, **i32),
                    free=torch.arange(60, **i32), count=torch.tensor([60], **i32),
                    kc=torch.zeros((60, HKV, PAGE, D), dtype=torch.float16, device="cuda"),
                    vc=torch.zeros((60, HKV, PAGE, D), dtype=torch.float16, device="cuda"),
                    x=torch.zeros((rows, HQ + 2 * HKV, D), device="cuda"),
                    plan=(torch.empty(b + 1, **i32), None, torch.empty(rows, **i32),
                          torch.empty(rows, dtype=torch.int64, device="cuda"), torch.empty(b, **i32)),
                    q=torch.empty((rows, HQ, D), dtype=torch.float16, device="cuda"),
                    o=torch.zeros((rows, HQ, D), dtype=torch.float16, device="cuda"),
                    y=torch.empty((rows, v), device="cuda"), z=torch.empty((rows, v), device="cuda"),
                    ws=torch.empty(1 << 24, dtype=torch.uint8, device="cuda"))

    def step(s):
        plan = (s["plan"][0], s["kv"], *s["plan"][2:])
        w4.kv_plan(s["kv"], new, s["table"], s["owned"], s["free"], s["count"], PAGE, rows, depth=depth, out=plan)
        x = s["x"]
        w4.kv_append_norm_rope(x[:, HQ:HQ + HKV], x[:, HQ + HKV:], s["kc"], s["vc"], plan[3], plan[2], freq, weight,
                               q=x[:, :HQ], q_weight=weight, q_out=s["q"])
        w4.attention_paged_tree(s["q"], s["kc"], s["vc"], s["table"], s["kv"], mask, q_start=plan[0], max_q=4, out=s["o"],
                                workspace=s["ws"])
        w4.gemm_f16(s["o"].view(rows, HQ * D), head, out=s["y"], workspace=s["ws"])
        w4.logits_adjust(s["y"], tokens=tokens, token_len=lens, repetition=one, request=request, out=s["z"])

    a, e, spare = state(), state(), state()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.current_stream())
        step(spare)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(a)
    for i in range(6):
        rows_in = torch.from_numpy(rng.standard_normal(tuple(a["x"].shape)).astype(np.float32)).cuda()
        for s in (a, e):
            s["x"].copy_(rows_in)
            if i == 3:  # a part was not accepted
                s["kv"] -= torch.tensor([2, 3, 0], **i32)
        g.replay()
        torch.cuda.synchronize()
        step(e)
        torch.cuda.synchronize()
        for n in ("kv", "table", "owned", "free", "count", "kc", "vc", "q", "o", "z"):
            assert torch.equal(a[n], e[n]), (i, n)
        for x, y in zip(a["plan"], e["plan"]):
            assert x is None or torch.equal(x, y)
