"""logits_adjust against the fp64 oracle.

Bound, per output: at most four f32 roundings (the quotient or product, the frequency's term and the subtractions or their
fused form, the bias), each at most 2^-24 of the sum of the sizes of what has been added up: 5 * 2^-24 of that sum
covers them.  Masked logits are -infinity, logits that nothing changes keep their bits.
"""

from __future__ import annotations

import numpy as np
import pytest

from oracle import stepref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_rope_append import dev, w4  # noqa: E402, F401


class Rules:
    def __init__(self, m, v, requests=None, length=50, biases=5, masks="row", penalties=True, seed=0, junk=True):
        rng = np.random.default_rng(seed)
        s = m if requests is None else requests
        self.m, self.v, self.s = m, v, s
        self.logits = (rng.standard_normal((m, v)) * 4).astype(np.float32)
        self.request = None if requests is None else rng.integers(0, s, m).astype(np.int32)
        self.tokens = self.token_len = self.prompt_len = self.repetition = self.frequency = self.presence = None
        if penalties:
            self.tokens = (v * rng.random((s, length)) ** 3).astype(np.int32)
            if junk and length:
                at = rng.random((s, length)) < 0.1
                self.tokens[at] = rng.choice([-1, v, 2 ** 31 - 1, -2 ** 31], int(at.sum()))
            self.token_len = rng.integers(0, length + 1, s).astype(np.int32)
            self.token_len[0] = length
            self.prompt_len = rng.integers(-3, length + 9, s).astype(np.int32)
            self.repetition = rng.uniform(0.7, 2.0, s).astype(np.float32)
            self.frequency = rng.uniform(-0.5, 1.0, s).astype(np.float32)
            self.presence = rng.uniform(-0.5, 1.0, s).astype(np.float32)
        self.bias = None
        if biases is not None:
            n = rng.integers(0, biases + 1, s) if biases else np.zeros(s, dtype=int)
            self.bias = [[(int(t), np.float32(b)) for t, b in zip(rng.choice([-1, 0, v // 2, v - 1, v, int(rng.integers(v))], k),
                                                                 rng.standard_normal(k) * 5)] for k in n]
        self.allowed = self.mask = self.mask_row = None
        if masks == "row":
            self.mask_bits = rng.random((m, v)) < 0.4
            self.mask_bits[m // 2] = False  # a row of which nothing is allowed
            self.allowed = [set(np.flatnonzero(r).tolist()) for r in self.mask_bits]
        elif masks == "some":
            self.mask_bits = rng.random((3, v)) < 0.9
            self.mask_row = rng.choice([0, 1, 2, -1, 3, -2 ** 31, 2 ** 31 - 1], m).astype(np.int32)
            self.allowed = [set(np.flatnonzero(self.mask_bits[g]).tolist()) if 0 <= g < 3 else None for g in self.mask_row]
        if masks:
            n = -(-v // 32)
            bits = rng.random((self.mask_bits.shape[0], 32 * (n + 1))) < 0.5  # past V: anything
            bits[:, :v] = self.mask_bits
            w = (bits.reshape(bits.shape[0], n + 1, 32) * (np.uint64(1) << np.arange(32, dtype=np.uint64))).sum(-1)
            self.mask = w.astype(np.uint32).view(np.int32)

    def kw(self):
        a = {}
        for n in ("request", "tokens", "token_len", "prompt_len", "repetition", "frequency", "presence", "mask", "mask_row"):
            x = getattr(self, n)
            if x is not None:
                a[n] = dev(x)
        if self.bias is not None:
            flat = [e for b in self.bias for e in b]
            a["bias_start"] = dev(np.cumsum([0] + [len(b) for b in self.bias]).astype(np.int32))
            a["bias_id"] = dev(np.array([t for t, _ in flat], dtype=np.int32))
            a["bias"] = dev(np.array([x for _, x in flat], dtype=np.float32))
        return a

    def check(self, got, logits=None):
        logits = self.logits if logits is None else logits
        want, size = stepref.adjust(logits, self.request, self.tokens, self.token_len, self.prompt_len, self.repetition,
                                    self.frequency, self.presence, self.bias, self.allowed)
        got = got.cpu().numpy()
        masked = np.isneginf(want)
        assert np.array_equal(np.isneginf(got), masked)
        same = ~masked & (want == logits)
        assert np.array_equal(got[same], logits[same])
        err, bound = np.abs(got[~masked] - want[~masked]), size[~masked] * 5 * 2.0 ** -24
        assert (err <= bound).all(), (err / bound).max()


CASES = [  # rows, vocabulary, requests, history, biases, masks, penalties
    (1, 1, None, 3, 2, None, True), (1, 5, None, 7, 3, "row", True), (1, 151936, None, 1570, 20, None, True),
    (3, 4095, None, 100, 9, "row", True), (3, 4096, 2, 100, 9, "some", True), (2, 4097, None, 5000, None, None, True),
    (9, 1001, 4, 30, 40, "some", True), (5, 32000, None, 0, 5, "row", True), (5, 32001, 3, 1, None, "row", True),
    (64, 2000, None, 257, 300, "some", True), (2, 262144, 1, 20001, 7, "row", True), (4, 777, None, 9, None, "row", False),
    (4, 776, None, 9, 6, None, False), (4, 776, 2, 9, 6, "some", False), (3, 500, None, 9, None, None, False),
    (300, 130, 7, 64, 3, "some", True), (2, 50257, None, 70000, 1000, None, True),
    (5, 9000, 2, 64, 20000, "row", True), (70, 40000, 3, 300, 30, "row", True), (40, 70000, 5, 3000, None, "some", True),
]


@pytest.mark.parametrize("m,v,requests,length,biases,masks,penalties", CASES)
def test_rules(w4, m, v, requests, length, biases, masks, penalties):  # noqa: F811
    r = Rules(m, v, requests, length, biases, masks, penalties, seed=m + v)
    x, kw = dev(r.logits), r.kw()
    a = w4.logits_adjust(x, **kw)
    r.check(a)
    assert np.array_equal(x.cpu().numpy(), r.logits)
    # in place, and rows that are not 16-byte aligned: the same bits
    w4.logits_adjust(x, out=x, **kw)
    assert torch.equal(x, a)
    wide = torch.full((m, v + 7), 3.0, device="cuda")
    wide[:, 3:3 + v] = dev(r.logits)
    out = torch.full((m, v + 6), 8.0, device="cuda")
    w4.logits_adjust(wide[:, 3:3 + v], out=out[:, 1:1 + v], **kw)
    assert torch.equal(out[:, 1:1 + v], a)
    assert (out[:, 0] == 8).all() and (out[:, 1 + v:] == 8).all() and (wide[:, :3] == 3).all() and (wide[:, 3 + v:] == 3).all()
    w4.logits_adjust(wide[:, 3:3 + v], out=wide[:, 3:3 + v], **kw)
    assert torch.equal(wide[:, 3:3 + v], a) and (wide[:, :3] == 3).all() and (wide[:, 3 + v:] == 3).all()


def test_each_penalty_alone(w4):  # noqa: F811
    for name in ("repetition", "frequency", "presence", "prompt_len", None):
        r = Rules(3, 300, None, 60, None, None, seed=2)
        for n in ("repetition", "frequency", "presence", "prompt_len"):
            if n != name:
                setattr(r, n, None)
        r.check(w4.logits_adjust(dev(r.logits), **r.kw()))


def test_requests_that_are_none(w4):  # noqa: F811
    r = Rules(6, 700, 3, 40, 8, "row", seed=3)
    r.request = np.array([0, -1, 3, 2, -2 ** 31, 2 ** 31 - 1], dtype=np.int32)
    r.check(w4.logits_adjust(dev(r.logits), **r.kw()))


def test_not_finite_logits(w4):  # noqa: F811
    # infinities and NaN: masked ones are -infinity, the others go through the arithmetic
    r = Rules(4, 600, None, 200, 4, "row", seed=4)
    rng = np.random.default_rng(5)
    x = r.logits.copy()
    at = rng.random(x.shape) < 0.3
    x[at] = rng.choice(np.array([np.nan, np.inf, -np.inf], dtype=np.float32), int(at.sum()))
    got = w4.logits_adjust(dev(x), **r.kw()).cpu().numpy()
    allowed = r.mask_bits
    assert np.isneginf(got[~allowed]).all()
    odd = at & allowed
    assert np.array_equal(got[odd], x[odd], equal_nan=True)


def test_starts_and_lengths_outside(w4):  # noqa: F811
    # token_len past the row and below 0, bias_start past the entries, falling and below 0
    r = Rules(4, 400, None, 30, None, None, seed=6)
    kw = r.kw()
    kw["token_len"] = dev(np.array([99, 2 ** 31 - 1, -1, -2 ** 31], dtype=np.int32))
    r.token_len = np.array([30, 30, 0, 0])
    entries = [(5, np.float32(1.0)), (6, np.float32(2.0)), (5, np.float32(4.0))]
    kw["bias_id"] = dev(np.array([t for t, _ in entries], dtype=np.int32))
    kw["bias"] = dev(np.array([b for _, b in entries], dtype=np.float32))
    kw["bias_start"] = dev(np.array([-5, 2, 2 ** 31 - 1, 1, -2 ** 31], dtype=np.int32))
    r.bias = [entries[:2], entries[2:], [], []]
    r.check(w4.logits_adjust(dev(r.logits), **kw))


def test_selection_takes_masked_rows(w4):  # noqa: F811
    # logits_argmax_topk behind it: fewer tokens allowed than k, one, and none
    for v, k in ((1000, 8), (5000, 8), (151936, 40), (151936, 64), (151936, 200), (9000, 256)):
        rng = np.random.default_rng(v + k)
        x = rng.standard_normal((5, v)).astype(np.float32)
        allowed = np.zeros((5, v), dtype=bool)
        allowed[0] = rng.random(v) < 0.5
        allowed[1, rng.choice(v, 3, replace=False)] = True
        allowed[2, v - 1] = True
        allowed[4, :] = True
        n = -(-v // 32)
        bits = np.zeros((5, 32 * n), dtype=bool)
        bits[:, :v] = allowed
        mask = (bits.reshape(5, n, 32) * (np.uint64(1) << np.arange(32, dtype=np.uint64))).sum(-1).astype(np.uint32)
        y = w4.logits_adjust(dev(x), mask=dev(mask.view(np.int32)))
        idx, val = w4.logits_argmax_topk(y, k)
        host = np.where(allowed, x, -np.inf)
        want = np.argsort(-host, axis=1, kind="stable")[:, :k]
        assert np.array_equal(idx.cpu().numpy(), want), (v, k)
        assert np.array_equal(val.cpu().numpy(), np.take_along_axis(host, want, 1)), (v, k)


def test_far_offsets(w4):  # noqa: F811
    # rows past 2^31 elements of the logits
    m, v = 17000, 131072
    x = torch.zeros((m, v), device="cuda")
    for row in (0, m - 1):
        x[row] = torch.arange(v, device="cuda") * 0.5
    tokens = torch.full((m, 2), -1, dtype=torch.int32, device="cuda")
    tokens[m - 1, 0], tokens[m - 1, 1] = v - 1, v - 1
    ln = torch.full((m,), 2, dtype=torch.int32, device="cuda")
    w4.logits_adjust(x, tokens=tokens, token_len=ln, presence=torch.ones(m, device="cuda"), out=x)
    assert float(x[m - 1, v - 1]) == (v - 1) * 0.5 - 1 and float(x[m - 1, v - 2]) == (v - 2) * 0.5
    assert float(x[0, v - 1]) == (v - 1) * 0.5 and not x[1:m - 1].any()


def test_captured_and_replayed(w4):  # noqa: F811
    r = Rules(5, 3001, 3, 90, 12, "some", seed=7)
    x, kw = dev(r.logits), r.kw()
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.current_stream())
        w4.logits_adjust(x, out=out, **kw)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.logits_adjust(x, out=out, **kw)
    for i in range(4):
        r.logits = np.roll(r.logits, i + 1, axis=1)
        r.token_len = np.minimum(r.token_len + i, 90).astype(np.int32)
        x.copy_(dev(r.logits))
        kw["token_len"].copy_(dev(r.token_len))
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        r.check(out)
        assert torch.equal(out, w4.logits_adjust(x, **kw))


def test_bindings_refuse(w4):  # noqa: F811
    r = Rules(3, 100, None, 20, 4, "row", seed=8)
    x, kw = dev(r.logits), r.kw()
    w4.logits_adjust(x, **kw)
    i = torch.zeros(3, dtype=torch.int32, device="cuda")
    for bad in (dict(token_len=None), dict(token_len=i[:2]), dict(tokens=None), dict(tokens=kw["tokens"].long()),
                dict(repetition=i), dict(frequency=kw["frequency"][:2]), dict(bias=None), dict(bias_id=None),
                dict(bias_start=i), dict(mask=None, mask_row=i), dict(mask=kw["mask"][:, :3]), dict(mask=kw["mask"].t()),
                dict(mask_row=i[:2]), dict(request=i[:2]), dict(out=x[:2].clone()), dict(out=x.half()), dict(presence=x)):
        with pytest.raises((TypeError, ValueError)):
            w4.logits_adjust(x, **{**kw, **bad})
    for bad in (dict(mask=kw["mask"][:2]), dict(tokens=None, token_len=None, prompt_len=None, repetition=None, frequency=None,
                                                presence=None, bias_start=kw["bias_start"][:2])):
        with pytest.raises(w4.W4Error):
            w4.logits_adjust(x, **{**kw, **bad})
