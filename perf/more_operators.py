"""The operators of a decode step with drafted tokens: block tables and slot maps from request lengths, norms of
queries and keys with the rotary positions on their way into the paged cache, the attention of a tree of drafted
tokens over it, and penalties, biases and grammar masks on the logits.  Cases, inputs, a plain form of each
(elementary torch operations in 32 bits, angles in 64) and the values of their definitions in 64 bits.

Layouts: x, q, k, v [tokens][heads][dim]; caches [pages][kv heads][page size][dim], f16 or e4m3 with one f32
scale per kv head; table int32 [sequences][pages of a sequence], -1 where a sequence has none; slots int64
[tokens] = page * page size + offset, -1: none; tree masks int64 [tokens][words], bit j % 64 of word j / 64: sees new token j of its
sequence; grammar masks int32 [masks][words], bit v % 32 of word v / 32: token v is allowed.
"""

from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0


# --------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of each of 64 sequences, some of which have just taken another's place
        dict(name="plan_decode_64", op="plan", seqs=64, new=1, new_min=1, kv=8192, kv_min=1, page=16, tree=False, short=0),
        # prompt chunks beside single tokens, 256 sequences of a long table: the rows of a large step
        dict(name="plan_mixed_256", op="plan", seqs=256, new=201, new_min=0, kv=16384, kv_min=0, page=16, tree=False,
             short=0),
        # one token of the Qwen3-1.7B heads, straight from the f32 rows of the q|k|v projection
        dict(name="norm_append_1", op="append", tokens=1, hq=16, hkv=8, dim=128, rot=128, interleaved=False, mscale=1.0,
             far=4096, f32=True, e4m3=False, page=16, pages=128),
        # one token of each of 64 sequences, the Gemma-shaped heads, an 8-bit cache
        dict(name="norm_append_64_e4m3", op="append", tokens=64, hq=16, hkv=8, dim=256, rot=256, interleaved=False,
             mscale=1.0, far=8192, f32=True, e4m3=True, page=64, pages=24),
        # a long odd prompt chunk
        dict(name="norm_append_8191", op="append", tokens=8191, hq=16, hkv=8, dim=128, rot=128, interleaved=False,
             mscale=1.0, far=8192, f32=True, e4m3=False, page=16, pages=520),
        # queries alone, part of each head turned in neighbouring pairs, f16
        dict(name="norm_rope_4099", op="norm", tokens=4099, heads=16, dim=80, rot=32, interleaved=True, mscale=1.1386,
             far=32768, f32=False),
        # eight drafted tokens of one sequence: the smallest call, where latency counts
        dict(name="tree_8", op="tree", seqs=1, new=8, new_min=8, kv=1570, kv_min=1570, hq=16, hkv=2, dim=128, page=16,
             window=0, e4m3=False),
        # 16 sequences with trees of 7 to 48 tokens, the Qwen3-1.7B heads, an 8-bit cache
        dict(name="tree_16x48_e4m3", op="tree", seqs=16, new=48, new_min=7, kv=8192, kv_min=301, hq=16, hkv=8, dim=128,
             page=32, window=0, e4m3=True),
        # wide trees behind long contexts, the Gemma-shaped heads, a sliding window
        dict(name="tree_4x200_window", op="tree", seqs=4, new=200, new_min=61, kv=16384, kv_min=9001, hq=16, hkv=8,
             dim=256, page=64, window=4096, e4m3=False),
        # one row of the Qwen2.5-3B vocabulary, penalties and biases
        dict(name="logits_1", op="logits", rows=1, requests=1, vocab=151936, tokens=1570, biases=20, masks=0),
        # 64 requests with long histories, grammars for half of them
        dict(name="logits_64", op="logits", rows=64, requests=64, vocab=151936, tokens=8191, biases=64, masks=32),
        # the drafted tokens of four requests, each with a grammar state of its own, the Gemma-shaped vocabulary
        dict(name="logits_tree_100", op="logits", rows=100, requests=4, vocab=262144, tokens=20001, biases=7, masks=100),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("plan", "norm", "append", "append", "tree", "tree", "tree", "logits", "logits"))
    page = rng.choice((8, 16, 16, 32, 64, 100))
    if op == "plan":
        seqs, new = _log(rng, 1, 1024), 1 if rng.random() < 0.4 else _log(rng, 2, 64)
        return dict(op=op, seqs=seqs, new=new, new_min=rng.randint(0, new), kv=_log(rng, 64, 16384), kv_min=rng.randint(0, 60),
                    page=page, tree=new > 1 and rng.random() < 0.5, short=rng.choice((0, 0, 1, 5)))
    if op == "logits":
        rows = _log(rng, 1, 100)
        return dict(op=op, rows=rows, requests=rows if rng.random() < 0.5 else rng.randint(1, rows),
                    vocab=rng.choice((32000, 50257, 151936, 151936, 262144, rng.randint(1000, 262144))),
                    tokens=_log(rng, 1, 20000), biases=rng.choice((0, 3, 300)), masks=rng.choice((0, 1, rows)))
    dim = rng.choice((64, 80, 96, 128, 128, 256))
    hkv, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 7, 8))
    e4m3 = rng.random() < 0.4
    if op in ("norm", "append"):
        rot = dim if rng.random() < 0.6 else 2 * rng.randint(1, dim // 2)
        shared = dict(op=op, tokens=_log(rng, 1, 8192), dim=dim, rot=rot, interleaved=rng.random() < 0.4,
                      mscale=rng.choice((1.0, 1.25)), far=_log(rng, 8192, 1 << 20), f32=rng.random() < 0.6)
        if op == "norm":
            return dict(heads=min(16, hkv * group), **shared)
        return dict(hq=hkv * group if hkv * group <= 16 else hkv, hkv=hkv, e4m3=e4m3, page=page,
                    pages=-(-shared["tokens"] // page) + rng.randint(1, 20), **shared)
    seqs = _log(rng, 1, 16)
    new = _log(rng, 2, max(4, min(256, 4096 // (seqs * group))))
    kv = new + _log(rng, 30, max(64, min(65536 // (seqs * hkv), 7 * 10 ** 9 // (seqs * new * hkv * group * dim))))
    return dict(op=op, seqs=seqs, new=new, new_min=rng.randint(1, new), kv=kv, kv_min=rng.randint(new, kv), hq=hkv * group,
                hkv=hkv, dim=dim, page=page, window=new + _log(rng, 16, 4096) if rng.random() < 0.25 else 0, e4m3=e4m3)


def _spread(n, lo, hi, step):
    """n whole numbers from lo to hi, the first of them hi"""
    return [hi] + [lo + int(round((hi - lo) * ((b * step) % 1.0))) for b in range(1, n)]


def _new(case):
    return _spread(case["seqs"], case["new_min"], case["new"], 0.7548776662)


def _tree_lengths(case):
    """(new tokens, cached tokens with them) of each sequence"""
    return [(n, max(n, kv)) for n, kv in zip(_new(case), _spread(case["seqs"], case["kv_min"], case["kv"], 0.6180339887))]


def _histories(case):
    return _spread(case["requests"], min(case["tokens"], 1 + case["tokens"] // 16), case["tokens"], 0.6180339887)


def work(case):
    op = case["op"]
    if op == "plan":
        rows, seqs = sum(_new(case)), case["seqs"]
        return {"bytes": rows * (16 + 4 * case["tree"]) + seqs * 28, "flops": 4 * rows + 8 * seqs}
    if op == "norm":
        e = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": e * ((4 if case["f32"] else 2) + 2) + case["tokens"] * 4 + case["rot"] * 2 + case["dim"] * 4,
                "flops": 4 * e + 3 * case["tokens"] * case["heads"] * case["rot"]}
    if op == "append":
        e, kv = (case["tokens"] * n * case["dim"] for n in (case["hq"] + 2 * case["hkv"], 2 * case["hkv"]))
        turned = case["tokens"] * (case["hq"] + case["hkv"])
        return {"bytes": e * (4 if case["f32"] else 2) + 2 * (e - kv) + kv * (1 if case["e4m3"] else 2) + 12 * case["tokens"],
                "flops": turned * (4 * case["dim"] + 3 * case["rot"])}
    if op == "tree":
        keys = pairs = new = 0
        for n, kv in _tree_lengths(case):
            old = min(kv - n, case["window"] or kv)
            keys += old + n
            new += n
            pairs += n * (old + min(n, 8))  # a drafted token has a few ancestors
        return {"bytes": keys * 2 * case["hkv"] * case["dim"] * (1 if case["e4m3"] else 2) + 4 * new * case["hq"] * case["dim"],
                "flops": 4 * pairs * case["hq"] * case["dim"]}
    e = case["rows"] * case["vocab"]
    return {"bytes": 8 * e + case["masks"] * case["vocab"] // 8 + 4 * sum(_histories(case)), "flops": 2 * e}


# -------------------------------------------------------------------------------- inputs

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _starts(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def _cache(case, gen, pages):
    shape = (pages, case["hkv"], case["page"], case["dim"])
    caches, scales = [], []
    for _ in range(2):
        x = torch.randn(shape, device=DEV, generator=gen, dtype=torch.float16)
        if case["e4m3"]:
            s = 0.02 + 0.01 * torch.rand(case["hkv"], device=DEV, generator=gen)
            x = (x.float() / s[:, None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            scales.append(s)
        else:
            scales.append(None)
        caches.append(x)
    return {"k_cache": caches[0], "v_cache": caches[1], "k_scale": scales[0], "v_scale": scales[1]}


def _ancestors(parent):
    """for each token of a tree the set of tokens from its root to itself, as bits of an integer"""
    sets = []
    for i, p in enumerate(parent):
        sets.append((sets[p] if p >= 0 else 0) | 1 << i)
    return sets


def _prepare_plan(case, gen, st):
    seqs, page = case["seqs"], case["page"]
    new = _new(case)
    # lengths of two steps that take turns: some requests grow, some end and others take their places
    now = torch.randint(case["kv_min"], case["kv"] + 1, (seqs,), device=DEV, generator=gen)
    fresh = torch.randint(case["kv_min"], case["kv"] + 1, (seqs,), device=DEV, generator=gen)
    other = torch.where(torch.rand(seqs, device=DEV, generator=gen) < 0.3, fresh, now + 1)
    new_len = torch.tensor(new, device=DEV)
    need = [(x + new_len + page - 1) // page for x in (now, other)]
    owned = (now + page - 1) // page
    st["width"] = -(-(case["kv"] + 1 + case["new"]) // page) + 2
    pages = seqs * st["width"]
    order = torch.randperm(pages, device=DEV, generator=gen).to(torch.int32)
    st["table"] = torch.full((seqs, st["width"]), -1, dtype=torch.int32, device=DEV)
    held = torch.arange(st["width"], device=DEV) < owned[:, None]
    taken = int(owned.sum())
    st["table"][held] = order[:taken]
    left = pages - taken
    if case["short"]:  # a stack that does not cover the step
        left = max(0, int((need[0] - owned).sum()) - case["short"])
    st["free"], st["free_count"] = order.roll(-taken), _ints([left])
    st["owned"] = owned.to(torch.int32)
    st["kv_len"] = [now.to(torch.int32), other.to(torch.int32)]
    st["new_len"] = _ints(new)
    st["rows"] = sum(new) + 3  # three rows of padding
    st["depth"] = None
    if case["tree"]:
        start = _ints(_starts(new))
        i = torch.arange(st["rows"], device=DEV)
        at = i - start[torch.searchsorted(start[1:], i, right=True).clamp(max=seqs - 1)]
        st["depth"] = (torch.rand(st["rows"], device=DEV, generator=gen) * (at + 1)).to(torch.int32)
    st["step"] = 0


def _prepare_rotation(case, gen, st):
    t, dim = case["tokens"], case["dim"]
    dt = torch.float32 if case["f32"] else torch.float16
    st["freq"] = (1e6 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])).float().to(DEV)
    st["positions"] = torch.randint(0, case["far"], (t,), device=DEV, generator=gen, dtype=torch.int32)
    st["weights"] = [1.0 + 0.3 * torch.randn(dim, device=DEV, generator=gen) for _ in range(2)]
    size = 0.2 + 3.0 * torch.rand((t, 1, 1), device=DEV, generator=gen)  # rows of a projection differ in size
    if case["op"] == "norm":
        st["x"] = (size * torch.randn((t, case["heads"], dim), device=DEV, generator=gen)).to(dt)
        return
    hq, hkv = case["hq"], case["hkv"]
    # the rows of a q|k|v projection; q, k and v are its column blocks
    rows = (size * torch.randn((t, hq + 2 * hkv, dim), device=DEV, generator=gen)).to(dt)
    st["q"], st["k"], st["v"] = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
    st.update(_cache(case, gen, case["pages"]))
    st["slots"] = torch.randperm(case["pages"] * case["page"], device=DEV, generator=gen)[:t].contiguous()


def _prepare_tree(case, gen, st):
    lens, ps = _tree_lengths(case), case["page"]
    need = [-(-kv // ps) for _, kv in lens]
    st["table"] = torch.full((len(lens), max(need) + 3), -1, dtype=torch.int32, device=DEV)  # room to grow
    order = torch.randperm(sum(need) + 5, device=DEV, generator=gen).to(torch.int32)
    for b, (n, at) in enumerate(zip(need, _starts(need))):
        st["table"][b, :n] = order[at:at + n]
    starts = _starts([n for n, _ in lens])
    words = -(-case["new"] // 64)
    pick = torch.rand(starts[-1], device=DEV, generator=gen).tolist()
    flat = []
    for b, (n, _) in enumerate(lens):
        # a token hangs on one of the four before it, or starts a branch behind the context
        parent = [max(i - 1 - int(5 * pick[starts[b] + i]), -1) for i in range(n)]
        for bits in _ancestors(parent):
            flat += [(w ^ (1 << 63)) - (1 << 63) for w in ((bits >> (64 * k)) & ((1 << 64) - 1) for k in range(words))]
    st["mask"] = torch.tensor(flat, dtype=torch.int64, device=DEV).view(starts[-1], words)
    st.update(_cache(case, gen, sum(need) + 5))
    st["q"] = torch.randn((starts[-1], case["hq"], case["dim"]), device=DEV, generator=gen, dtype=torch.float16)
    st["kv_len"], st["q_start"] = _ints([kv for _, kv in lens]), _ints(starts)
    st["max_q"], st["max_kv"] = max(n for n, _ in lens), max(kv for _, kv in lens)
    st["scale"] = case["dim"] ** -0.5
    st["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)


def _prepare_logits(case, gen, st):
    m, s, v = case["rows"], case["requests"], case["vocab"]

    def uniform(*shape):
        return torch.rand(shape, device=DEV, generator=gen)

    st["logits"] = 4.0 * torch.randn((m, v), device=DEV, generator=gen)
    # text repeats itself: tokens are drawn with a strong preference for a few
    st["tokens"] = (v * uniform(s, case["tokens"]) ** 4).to(torch.int32).clamp(max=v - 1)
    st["token_len"] = _ints(_histories(case))
    st["prompt_len"] = (st["token_len"] * uniform(s)).to(torch.int32)
    st["repetition"] = 1.0 + 0.5 * uniform(s)
    st["frequency"], st["presence"] = 0.5 * uniform(s), 0.8 * uniform(s)
    st["request"] = None if m == s else (torch.arange(m, device=DEV) * s // m).to(torch.int32)
    st["bias_start"] = st["bias_id"] = st["bias"] = st["mask"] = st["mask_row"] = None
    if case["biases"]:
        st["bias_start"] = _ints([case["biases"] * i for i in range(s + 1)])
        st["bias_id"] = (v * uniform(s * case["biases"])).to(torch.int32).clamp(max=v - 1)
        st["bias"] = 10.0 * torch.randn(s * case["biases"], device=DEV, generator=gen)
    if case["masks"]:
        words = (case["masks"], -(-v // 32))
        st["mask"] = torch.randint(-2 ** 31, 2 ** 31, words, device=DEV, generator=gen, dtype=torch.int32)
        st["mask"] &= torch.randint(-2 ** 31, 2 ** 31, words, device=DEV, generator=gen, dtype=torch.int32)
        if case["masks"] < m:  # some rows are free to take any token
            st["mask_row"] = torch.arange(m, device=DEV, dtype=torch.int32)
            st["mask_row"][st["mask_row"] >= case["masks"]] = -1


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = {"case": case}
    {"plan": _prepare_plan, "norm": _prepare_rotation, "append": _prepare_rotation, "tree": _prepare_tree,
     "logits": _prepare_logits}[case["op"]](case, gen, st)
    return st


# ----------------------------------------------------------------------------- the calls

def run(st):
    case = st["case"]
    op = case["op"]
    if op == "plan":
        kv_len = st["kv_len"][st["step"] % 2]
        st["step"] += 1
        if own:
            import int4_weight_only_group_amd as w4
            out = w4.kv_plan(kv_len, st["new_len"], st["table"], st["owned"], st["free"], st["free_count"], case["page"],
                             st["rows"], depth=st["depth"])
        else:
            out = _plan(st, kv_len)
        return (*out, st["table"], st["owned"], st["free"], st["free_count"])
    if own:
        import int4_weight_only_group_amd as w4
        if op == "norm":
            return w4.norm_rope_f16(st["x"], st["weights"][0], st["positions"], st["freq"], eps=1e-6,
                                    interleaved=case["interleaved"], mscale=case["mscale"])
        if op == "append":
            q = w4.kv_append_norm_rope(st["k"], st["v"], st["k_cache"], st["v_cache"], st["slots"], st["positions"],
                                       st["freq"], st["weights"][1], q=st["q"], q_weight=st["weights"][0], eps=1e-6,
                                       interleaved=case["interleaved"], mscale=case["mscale"],
                                       k_scale=st["k_scale"], v_scale=st["v_scale"])
            return q, st["k_cache"], st["v_cache"]
        if op == "tree":
            return w4.attention_paged_tree(st["q"], st["k_cache"], st["v_cache"], st["table"], st["kv_len"], st["mask"],
                                           q_start=st["q_start"], max_q=st["max_q"], scale=st["scale"],
                                           window=case["window"], k_scale=st["k_scale"], v_scale=st["v_scale"],
                                           workspace=st["workspace"])
        return w4.logits_adjust(st["logits"], tokens=st["tokens"], token_len=st["token_len"], prompt_len=st["prompt_len"],
                                repetition=st["repetition"], frequency=st["frequency"], presence=st["presence"],
                                bias_start=st["bias_start"], bias_id=st["bias_id"], bias=st["bias"], mask=st["mask"],
                                mask_row=st["mask_row"], request=st["request"])
    if op == "norm":
        cos, sin = _turns(st)
        return _rotate(_normed(st["x"], st["weights"][0]), cos, sin, case["interleaved"]).half()
    if op == "append":
        cos, sin = _turns(st)
        q = _rotate(_normed(st["q"], st["weights"][0]), cos, sin, case["interleaved"]).half()
        k = _rotate(_normed(st["k"], st["weights"][1]), cos, sin, case["interleaved"])
        page, off = st["slots"] // case["page"], st["slots"] % case["page"]
        st["k_cache"][page, :, off] = _stored(k, st["k_scale"])
        st["v_cache"][page, :, off] = _stored(st["v"].float(), st["v_scale"])
        return q, st["k_cache"], st["v_cache"]
    return _attend(st) if op == "tree" else _adjust(st)


def _plan(st, kv_len):
    page, rows, table = st["case"]["page"], st["rows"], st["table"]
    old, new = kv_len.long(), st["new_len"].long()
    need, owned = (old + new + page - 1) // page, st["owned"].long()
    j = torch.arange(st["width"], device=DEV)
    count, size = st["free_count"].long(), st["free"].numel()
    # pages past what a sequence needs go back; one more element takes what is not written
    back = (j >= need[:, None]) & (j < owned[:, None])
    at = torch.where(back, count + back.flatten().cumsum(0).view_as(back) - 1, size)
    free = torch.cat((st["free"], st["free"][:1])).scatter(0, at.flatten(), table.flatten())[:size]
    count = count + back.sum()
    want = (need - owned).clamp(min=0)
    granted = (want == 0) | (want.cumsum(0) <= count)
    take = (j >= owned[:, None]) & (j < need[:, None]) & granted[:, None]
    rank = take.flatten().cumsum(0).view_as(take) - 1
    table.copy_(torch.where(take, free[(count - 1 - rank).clamp(0, size - 1)], torch.where(back, -1, table)))
    st["free"].copy_(free)
    st["free_count"].copy_(count - take.sum())
    st["owned"].copy_(torch.where(granted, need, owned))
    end = new.cumsum(0)
    i = torch.arange(rows, device=DEV)
    seq = torch.searchsorted(end, i, right=True)
    real, seq = seq < new.numel(), seq.clamp(max=new.numel() - 1)
    step = i - (end - new)[seq]
    at = old[seq] + step
    slots = table[seq, (at // page).clamp(max=st["width"] - 1)].long() * page + at % page
    positions = old[seq] + (step if st["depth"] is None else st["depth"])
    return (torch.cat((end.new_zeros(1), end)).int(), torch.where(granted, old + new, old).int(),
            torch.where(real, positions, 0).int(), torch.where(real & granted[seq], slots, -1),
            torch.where(granted, 0, want).int())


def _turns(st):
    a = st["positions"].double()[:, None] * st["freq"].double()  # far positions: angles in 64 bits
    m = st["case"]["mscale"]
    return (a.cos() * m).float()[:, None], (a.sin() * m).float()[:, None]


def _normed(x, weight):
    x = x.float()
    return x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * weight


def _rotate(x, cos, sin, interleaved):
    r = 2 * cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., r:]), -1)


def _stored(x, scale):
    if scale is None:
        return x.half()
    return (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _gathered(cache, scale, table, tokens):
    """f32 [sequences][kv heads][tokens][dim] of the cached values."""
    ps = cache.shape[2]
    x = cache[table[:, :-(-tokens // ps)].clamp(min=0).long()].float()
    x = x.transpose(1, 2).flatten(2, 3)[:, :, :tokens]
    return x if scale is None else x * scale[:, None, None]


def _attend(st):
    case, q_start, kv_len = st["case"], st["q_start"].long(), st["kv_len"].long()
    k = _gathered(st["k_cache"], st["k_scale"], st["table"], st["max_kv"])
    v = _gathered(st["v_cache"], st["v_scale"], st["table"], st["max_kv"])
    b, hkv, tokens, dim = k.shape
    mq, group = st["max_q"], case["hq"] // hkv
    i, j = torch.arange(mq, device=DEV), torch.arange(tokens, device=DEV)
    q_len = q_start[1:] - q_start[:-1]
    at = (q_start[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][at].float().reshape(b, mq, hkv, group, dim).permute(0, 2, 3, 1, 4).reshape(b, hkv, group * mq, dim)
    s = (q @ k.transpose(2, 3)).mul_(st["scale"]).view(b, hkv, group, mq, tokens)
    bits = (st["mask"][at][..., None] >> torch.arange(64, device=DEV) & 1).flatten(2)[..., :mq].bool()
    bits &= i < q_len[:, None, None]
    old = (kv_len - q_len)[:, None, None]  # cached tokens before the drafted ones, which are key old and on
    node = j - old
    seen = torch.gather(bits, 2, node.clamp(0, mq - 1).expand(b, mq, tokens)) & (node >= 0) & (node < mq)
    past = node < 0
    if case["window"]:
        past = past & (j > old + bits.sum(-1, keepdim=True) - 1 - case["window"])
    s.masked_fill_(~(seen | past)[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    s.sub_(top.masked_fill_(top == -math.inf, 0.0)).exp_()
    total = s.sum(-1, keepdim=True)
    o = (s.view(b, hkv, group * mq, tokens) @ v).view(b, hkv, group, mq, dim) / total.masked_fill_(total == 0, 1.0)
    t = torch.arange(st["q"].shape[0], device=DEV)
    seq = torch.searchsorted(q_start[1:], t, right=True)
    return o[seq, :, :, t - q_start[seq]].reshape(t.numel(), case["hq"], dim).half()


def _adjust(st):
    case = st["case"]
    s, v = case["requests"], case["vocab"]
    of = slice(None) if st["request"] is None else st["request"].long()
    i, ids = torch.arange(case["tokens"], device=DEV), st["tokens"].long()
    said = (i >= st["prompt_len"][:, None]) & (i < st["token_len"][:, None])
    count = torch.zeros((s, v), device=DEV).scatter_add_(1, ids, said.float())
    seen = torch.zeros((s, v), device=DEV).scatter_add_(1, ids, (i < st["token_len"][:, None]).float()) > 0
    count, seen = count[of], seen[of]
    r, f, p = (st[n][of][:, None] for n in ("repetition", "frequency", "presence"))
    x = torch.where(seen, torch.where(st["logits"] > 0, st["logits"] / r, st["logits"] * r), st["logits"])
    x = x - f * count - p * (count > 0)
    if st["bias"] is not None:
        n = case["biases"]
        last = torch.zeros((s, v), dtype=torch.int64, device=DEV)  # of the same token twice the later counts
        last.scatter_reduce_(1, st["bias_id"].long().view(s, n), torch.arange(1, s * n + 1, device=DEV).view(s, n), "amax")
        x = x + torch.where(last > 0, st["bias"][(last - 1).clamp(min=0)], 0.0)[of]
    if st["mask"] is not None:
        allowed = (st["mask"][..., None] >> torch.arange(32, device=DEV, dtype=torch.int32) & 1).flatten(1)[:, :v].bool()
        if st["mask_row"] is not None:
            allowed = allowed[st["mask_row"].clamp(min=0).long()] | (st["mask_row"] < 0)[:, None]
        x = x.masked_fill(~allowed, -math.inf)
    return x


# -------------------------------------------------------------- the definitions in 64 bits

def _exact_plan(case, st):
    page = case["page"]
    old, new = st["kv_len"][0].tolist(), st["new_len"].tolist()
    table, owned = st["table"].tolist(), st["owned"].tolist()
    held = st["free"].tolist()
    count = st["free_count"].tolist()[0]
    need = [-(-(a + n) // page) for a, n in zip(old, new)]
    for b, row in enumerate(table):
        for j in range(need[b], owned[b]):
            held[count], row[j] = row[j], -1
            count += 1
        owned[b] = min(owned[b], need[b])
    starts, total, positions, slots, status = [0], [], [], [], []
    left = count
    for b, row in enumerate(table):
        want = need[b] - owned[b]
        left -= want
        fine = want == 0 or left >= 0
        for j in range(owned[b], need[b] if fine else 0):
            count -= 1
            row[j] = held[count]
        owned[b] = need[b] if fine else owned[b]
        status.append(0 if fine else want)
        total.append(old[b] + new[b] if fine else old[b])
        for i in range(new[b]):
            at = old[b] + i
            positions.append(at if st["depth"] is None else old[b] + int(st["depth"][starts[-1] + i]))
            slots.append(row[at // page] * page + at % page if fine else -1)
        starts.append(starts[-1] + new[b])
    pad = st["rows"] - starts[-1]
    out = [_ints(x) for x in (starts, total, positions + [0] * pad, status, table, owned, held, [count])]
    return (*out[:3], torch.tensor(slots + [-1] * pad, dtype=torch.int64, device=DEV), *out[3:])


def _exact_rotation(case, st):
    f64 = torch.float64
    turn = torch.polar(torch.full((case["tokens"], case["rot"] // 2), case["mscale"], dtype=f64, device=DEV),
                       st["positions"].to(f64)[:, None] * st["freq"].to(f64)[None])

    def turned(x, weight):
        y, r = x.to(f64), case["rot"]
        y = y / torch.sqrt(torch.linalg.vector_norm(y, dim=-1, keepdim=True) ** 2 / case["dim"] + 1e-6) * weight.to(f64)
        even = slice(0, r, 2) if case["interleaved"] else slice(0, r // 2)
        odd = slice(1, r, 2) if case["interleaved"] else slice(r // 2, r)
        z = torch.complex(y[..., even], y[..., odd]) * turn[:, None]
        y[..., even], y[..., odd] = z.real, z.imag
        return y

    if case["op"] == "norm":
        return turned(st["x"], st["weights"][0])
    out = [turned(st["q"], st["weights"][0])]
    for x, cache, scale in ((turned(st["k"], st["weights"][1]), st["k_cache"], st["k_scale"]),
                            (st["v"].to(f64), st["v_cache"], st["v_scale"])):
        if scale is not None:
            x = x / scale.to(f64)[None, :, None]
        c = cache.to(f64).transpose(1, 2).reshape(-1, case["hkv"], case["dim"])
        c[st["slots"]] = x
        out.append(c.view(case["pages"], case["page"], case["hkv"], case["dim"]).transpose(1, 2).contiguous())
    return tuple(out)


def _exact_tree(case, st):
    f64 = torch.float64
    t0, outs, group = 0, [], case["hq"] // case["hkv"]
    for b, (n, kv) in enumerate(_tree_lengths(case)):
        ids, old = st["table"][b, :-(-kv // case["page"])].long(), kv - n
        hidden = torch.zeros((n, kv), dtype=torch.bool, device=DEV)
        for j in range(n):  # a column for each drafted token
            hidden[:, old + j] = (st["mask"][t0:t0 + n, j // 64] >> (j % 64)) & 1 == 0
        if case["window"]:
            depth = (~hidden[:, old:]).sum(1) - 1
            hidden[:, :old] = torch.arange(old, device=DEV) <= (old + depth - case["window"])[:, None]
        heads = []
        for h in range(case["hq"]):
            g = h // group
            k = st["k_cache"][ids, g].reshape(-1, case["dim"])[:kv].to(f64)
            v = st["v_cache"][ids, g].reshape(-1, case["dim"])[:kv].to(f64)
            if case["e4m3"]:
                k, v = k * st["k_scale"][g].to(f64), v * st["v_scale"][g].to(f64)
            s = st["q"][t0:t0 + n, h].to(f64) @ k.T * st["scale"]
            s[hidden] = -math.inf
            heads.append(torch.softmax(s, -1) @ v)
        outs.append(torch.stack(heads, 1))
        t0 += n
    return torch.cat(outs)


def _exact_logits(case, st):
    x, v = st["logits"].double(), case["vocab"]
    bits = 1 << torch.arange(32, device=DEV, dtype=torch.int64)
    for m in range(case["rows"]):
        s = m if st["request"] is None else int(st["request"][m])
        history, at = st["tokens"][s, :int(st["token_len"][s])].long(), int(st["prompt_len"][s])
        seen = history.unique()
        y = x[m, seen]
        r = st["repetition"][s].double()
        x[m, seen] = torch.maximum(y, y * 0) / r + torch.minimum(y, y * 0) * r
        said = torch.bincount(history[at:], minlength=v)
        x[m] -= st["frequency"][s].double() * said + st["presence"][s].double() * said.clamp(max=1)
        n = case["biases"]
        given = {int(i): b for i, b in zip(st["bias_id"][s * n:s * n + n], st["bias"][s * n:s * n + n].double())} if n else {}
        if given:
            x[m, torch.tensor(list(given), device=DEV)] += torch.stack(list(given.values()))
        if st["mask"] is not None:
            g = m if st["mask_row"] is None else int(st["mask_row"][m])
            if g >= 0:
                allowed = ((st["mask"][g].long()[:, None] & bits) != 0).reshape(-1)[:v]
                x[m, ~allowed] = -math.inf
    return x


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("norm", "append"):
        return _exact_rotation(case, st)
    return {"plan": _exact_plan, "tree": _exact_tree, "logits": _exact_logits}[case["op"]](case, st)
