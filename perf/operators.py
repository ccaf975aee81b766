"""The operators between the q|k|v projection and the output projection of a decoder layer:
rotary positions, the append of keys and values to a paged cache, and the attention of new
tokens over that cache.  Cases, inputs, a plain form of each (elementary torch operations in
32 bits, angles in 64) and the values of their definitions in 64 bits.

Layouts: x, q, k, v [tokens][heads][dim]; caches [pages][kv heads][page size][dim], f16 or
e4m3 with one f32 scale per kv head; table int32 [sequences][pages of a sequence], -1 where a
sequence has none; slots int64 [tokens] = page * page size + offset.
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
        # queries of one decode step of 64 sequences, positions far into a long context
        dict(name="rope_decode_64", op="rope", tokens=64, heads=16, dim=128, rot=128, interleaved=False,
             inverse=False, mscale=1.0, far=131072, f32=True),
        # part of each head, neighbouring pairs, rotated back (the gradient of the rotation): a long odd chunk
        dict(name="rope_inverse_8191", op="rope", tokens=8191, heads=16, dim=80, rot=32, interleaved=True,
             inverse=True, mscale=1.1386, far=32768, f32=False),
        # one token of the Qwen2.5-3B shapes, straight from the f32 rows of the q|k|v projection
        dict(name="append_decode_1", op="append", tokens=1, hq=16, hkv=2, dim=128, rot=128, interleaved=False,
             mscale=1.0, far=4096, f32=True, e4m3=False, page=16, pages=128),
        # one token of each of 64 sequences, the Gemma-shaped heads, an 8-bit cache
        dict(name="append_decode_64_e4m3", op="append", tokens=64, hq=16, hkv=8, dim=256, rot=256,
             interleaved=False, mscale=1.0, far=8192, f32=True, e4m3=True, page=64, pages=24),
        # the tokens of a long prompt chunk
        dict(name="append_prefill_8192", op="append", tokens=8192, hq=16, hkv=2, dim=128, rot=128,
             interleaved=False, mscale=1.0, far=8192, f32=True, e4m3=False, page=16, pages=520),
        # one sequence, one token: the smallest call of a local engine, where latency counts
        dict(name="attend_decode_1", op="attend", seqs=1, q=1, q_min=1, kv=1570, kv_min=1570, hq=16, hkv=2,
             dim=128, page=16, window=0, e4m3=False),
        # a batch of 64 sequences of very different lengths, the Qwen3-1.7B heads, an 8-bit cache
        dict(name="attend_decode_64_e4m3", op="attend", seqs=64, q=1, q_min=1, kv=8192, kv_min=1, hq=16, hkv=8,
             dim=128, page=32, window=0, e4m3=True),
        # eight long contexts: the cache's bytes and nothing else
        dict(name="attend_decode_8_long", op="attend", seqs=8, q=1, q_min=1, kv=65536, kv_min=61001, hq=16, hkv=2,
             dim=128, page=16, window=0, e4m3=False),
        # eight draft tokens of four sequences (speculative verification)
        dict(name="attend_verify_8", op="attend", seqs=4, q=8, q_min=8, kv=16384, kv_min=9001, hq=16, hkv=2,
             dim=128, page=16, window=0, e4m3=False),
        # a whole prompt of 1570 tokens
        dict(name="attend_prompt_1570", op="attend", seqs=1, q=1570, q_min=1570, kv=1570, kv_min=1570, hq=16,
             hkv=2, dim=128, page=16, window=0, e4m3=False),
        # a ragged batch with a sliding window, the Gemma-shaped heads
        dict(name="attend_ragged_window", op="attend", seqs=6, q=700, q_min=1, kv=4001, kv_min=900, hq=16, hkv=8,
             dim=256, page=64, window=1024, e4m3=False),
        # a chunk of 4096 tokens behind 12288 cached ones
        dict(name="attend_chunk_4096", op="attend", seqs=1, q=4096, q_min=4096, kv=16384, kv_min=16384, hq=16,
             hkv=2, dim=128, page=16, window=0, e4m3=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dim = rng.choice((64, 80, 96, 128, 128, 256))
    hkv, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 7, 8))
    page = rng.choice((8, 16, 16, 32, 64, 100))
    kind = rng.choice(("rope", "append", "decode", "decode", "chunk", "chunk"))
    e4m3 = rng.random() < 0.4
    if kind in ("rope", "append"):
        rot = dim if rng.random() < 0.6 else 2 * rng.randint(1, dim // 2)
        shared = dict(tokens=_log(rng, 1, 8192), dim=dim, rot=rot, interleaved=rng.random() < 0.4,
                      mscale=rng.choice((1.0, 1.25)), far=_log(rng, 8192, 1 << 20), f32=rng.random() < 0.6)
        if kind == "rope":
            return dict(op="rope", heads=min(16, hkv * group), inverse=rng.random() < 0.5, **shared)
        hq = hkv * group if hkv * group <= 16 else hkv
        return dict(op="append", hq=hq, hkv=hkv, e4m3=e4m3, page=page,
                    pages=-(-shared["tokens"] // page) + rng.randint(1, 20), **shared)
    window = _log(rng, 16, 4096) if rng.random() < 0.3 else 0
    shared = dict(op="attend", hq=hkv * group, hkv=hkv, dim=dim, page=page, window=window, e4m3=e4m3)
    if kind == "decode":
        seqs = _log(rng, 1, 64)
        kv = _log(rng, 64, max(128, 131072 // (seqs * hkv)))
        return dict(seqs=seqs, q=1, q_min=1, kv=kv, kv_min=rng.randint(1 + kv // 8, kv), **shared)
    seqs = _log(rng, 1, 8)
    q = _log(rng, 2, max(4, 4096 // (seqs * group)))
    kv = q + _log(rng, 1, max(2, 16384 // (seqs * hkv)))
    return dict(seqs=seqs, q=q, q_min=rng.randint(1, q), kv=kv, kv_min=rng.randint(q, kv), **shared)


def _lengths(case):
    """(new tokens, cached tokens with them) of each sequence, spread between the case's bounds."""
    n, out = case["seqs"], []
    for b in range(n):
        f, g = (b * 0.6180339887 + (b + 1 == n)) % 1.0 if n > 1 else 1.0, (b * 0.7548776662) % 1.0
        if b == 0:
            f = g = 1.0  # the longest of each is there
        q = case["q_min"] + int(round((case["q"] - case["q_min"]) * g))
        out.append((q, max(q, case["kv_min"] + int(round((case["kv"] - case["kv_min"]) * f)))))
    return out


def work(case):
    if case["op"] == "rope":
        e = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": e * ((4 if case["f32"] else 2) + 2) + case["tokens"] * 4 + case["rot"] * 2,
                "flops": 3 * case["tokens"] * case["heads"] * case["rot"]}
    if case["op"] == "append":
        heads = case["hq"] + 2 * case["hkv"]
        e, kv = case["tokens"] * heads * case["dim"], case["tokens"] * 2 * case["hkv"] * case["dim"]
        q = case["tokens"] * case["hq"] * case["dim"]
        return {"bytes": e * (4 if case["f32"] else 2) + 2 * q + kv * (1 if case["e4m3"] else 2) + 12 * case["tokens"],
                "flops": 3 * case["tokens"] * (case["hq"] + case["hkv"]) * case["rot"]}
    keys = pairs = new = 0
    for q, kv in _lengths(case):
        w = case["window"] or kv
        keys += min(kv, w + q - 1)
        new += q
        full = min(max(0, kv - w), q)  # the last `full` queries see w keys, the others all before them
        part = q - full
        pairs += full * w + part * (kv - q) + part * (part + 1) // 2
    return {"bytes": keys * 2 * case["hkv"] * case["dim"] * (1 if case["e4m3"] else 2) + 4 * new * case["hq"] * case["dim"],
            "flops": 4 * pairs * case["hq"] * case["dim"]}


# -------------------------------------------------------------------------------- inputs

def _frequencies(rot):
    return (1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().to(DEV)


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


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = {"case": case}
    if case["op"] in ("rope", "append"):
        t, dim = case["tokens"], case["dim"]
        dt = torch.float32 if case["f32"] else torch.float16
        st["freq"] = _frequencies(case["rot"])
        st["positions"] = torch.randint(0, case["far"], (t,), device=DEV, generator=gen, dtype=torch.int32)
        if case["op"] == "rope":
            st["x"] = torch.randn((t, case["heads"], dim), device=DEV, generator=gen, dtype=dt)
            return st
        hq, hkv = case["hq"], case["hkv"]
        # the rows of a q|k|v projection; q, k and v are its column blocks
        rows = torch.randn((t, hq + 2 * hkv, dim), device=DEV, generator=gen, dtype=dt)
        st["q"], st["k"], st["v"] = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
        st.update(_cache(case, gen, case["pages"]))
        st["slots"] = torch.randperm(case["pages"] * case["page"], device=DEV, generator=gen)[:t].contiguous()
        return st
    lens = _lengths(case)
    ps = case["page"]
    need = [-(-kv // ps) for _, kv in lens]
    width = max(need) + 3  # a table row has room for the sequence to grow
    order = torch.randperm(sum(need) + 5, device=DEV, generator=gen).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    starts = [0]
    for q, _ in lens:
        starts.append(starts[-1] + q)
    st.update(_cache(case, gen, sum(need) + 5))
    st["q"] = torch.randn((starts[-1], case["hq"], case["dim"]), device=DEV, generator=gen, dtype=torch.float16)
    st["table"] = table
    st["kv_len"] = torch.tensor([kv for _, kv in lens], dtype=torch.int32, device=DEV)
    st["q_start"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    st["max_q"], st["max_kv"] = max(q for q, _ in lens), max(kv for _, kv in lens)
    st["scale"] = case["dim"] ** -0.5
    st["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    return st


# ----------------------------------------------------------------------------- the calls

def run(st):
    case = st["case"]
    if own:
        import int4_weight_only_group_amd as w4
        if case["op"] == "rope":
            return w4.rope_f16(st["x"], st["positions"], st["freq"], interleaved=case["interleaved"],
                               mscale=case["mscale"], inverse=case["inverse"])
        if case["op"] == "append":
            q = w4.kv_append_rope(st["k"], st["v"], st["k_cache"], st["v_cache"], st["slots"], st["positions"],
                                  st["freq"], q=st["q"], interleaved=case["interleaved"], mscale=case["mscale"],
                                  k_scale=st["k_scale"], v_scale=st["v_scale"])
            return q, st["k_cache"], st["v_cache"]
        return w4.attention_paged(st["q"], st["k_cache"], st["v_cache"], st["table"], st["kv_len"],
                                  q_start=st["q_start"], max_q=st["max_q"], scale=st["scale"],
                                  window=case["window"], k_scale=st["k_scale"], v_scale=st["v_scale"],
                                  workspace=st["workspace"])
    if case["op"] == "rope":
        cos, sin = _turns(st, -1.0 if case["inverse"] else 1.0)
        return _rotate(st["x"].float(), cos, sin, case["interleaved"]).half()
    if case["op"] == "append":
        cos, sin = _turns(st, 1.0)
        q = _rotate(st["q"].float(), cos, sin, case["interleaved"]).half()
        k = _rotate(st["k"].float(), cos, sin, case["interleaved"])
        page, off = st["slots"] // case["page"], st["slots"] % case["page"]
        st["k_cache"][page, :, off] = _stored(k, st["k_scale"])
        st["v_cache"][page, :, off] = _stored(st["v"].float(), st["v_scale"])
        return q, st["k_cache"], st["v_cache"]
    return _attend(st)


def _turns(st, sign):
    a = st["positions"].double()[:, None] * st["freq"].double()  # far positions: angles in 64 bits
    m = st["case"]["mscale"]
    return (a.cos() * m).float()[:, None], (a.sin() * (m * sign)).float()[:, None]


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
    i, j = torch.arange(mq, device=k.device), torch.arange(tokens, device=k.device)
    q_len = q_start[1:] - q_start[:-1]
    at = (q_start[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][at].float().reshape(b, mq, hkv, group, dim).permute(0, 2, 3, 1, 4).reshape(b, hkv, group * mq, dim)
    s = (q @ k.transpose(2, 3)).mul_(st["scale"]).view(b, hkv, group, mq, tokens)
    last = (kv_len - q_len)[:, None, None] + i[:, None]  # the last key that a query sees
    seen = (j <= last) & (j < kv_len[:, None, None])
    if case["window"]:
        seen &= j > last - case["window"]
    s.masked_fill_(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    s.sub_(top.masked_fill_(top == -math.inf, 0.0)).exp_()
    total = s.sum(-1, keepdim=True)
    o = (s.view(b, hkv, group * mq, tokens) @ v).view(b, hkv, group, mq, dim) / total.masked_fill_(total == 0, 1.0)
    t = torch.arange(st["q"].shape[0], device=k.device)
    seq = torch.searchsorted(q_start[1:], t, right=True)
    return o[seq, :, :, t - q_start[seq]].reshape(t.numel(), case["hq"], dim).half()


# -------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "attend":
        t0, outs = 0, []
        group, ps = case["hq"] // case["hkv"], case["page"]
        for b, (nq, nkv) in enumerate(_lengths(case)):
            ids = st["table"][b, :-(-nkv // ps)].long()
            pos = torch.arange(nkv - nq, nkv, device=DEV)[:, None]
            key = torch.arange(nkv, device=DEV)
            hidden = key > pos
            if case["window"]:
                hidden = hidden | (key <= pos - case["window"])
            heads = []
            for h in range(case["hq"]):
                g = h // group
                k = st["k_cache"][ids, g].reshape(-1, case["dim"])[:nkv].to(f64)
                v = st["v_cache"][ids, g].reshape(-1, case["dim"])[:nkv].to(f64)
                if case["e4m3"]:
                    k, v = k * st["k_scale"][g].to(f64), v * st["v_scale"][g].to(f64)
                s = st["q"][t0:t0 + nq, h].to(f64) @ k.T * st["scale"]
                s[hidden] = -math.inf
                heads.append(torch.softmax(s, -1) @ v)
            outs.append(torch.stack(heads, 1))
            t0 += nq
        return torch.cat(outs)
    turn = torch.polar(torch.full((case["tokens"], case["rot"] // 2), case["mscale"], dtype=f64, device=DEV),
                       st["positions"].to(f64)[:, None] * st["freq"].to(f64)[None])
    if case.get("inverse"):
        turn = turn.conj()

    def turned(x):
        y, r = x.to(f64).clone(), case["rot"]
        even = slice(0, r, 2) if case["interleaved"] else slice(0, r // 2)
        odd = slice(1, r, 2) if case["interleaved"] else slice(r // 2, r)
        z = torch.complex(y[..., even], y[..., odd]) * turn[:, None]
        y[..., even], y[..., odd] = z.real, z.imag
        return y

    if case["op"] == "rope":
        return turned(st["x"])
    out = [turned(st["q"])]
    for x, cache, scale in ((turned(st["k"]), st["k_cache"], st["k_scale"]), (st["v"].to(f64), st["v_cache"], st["v_scale"])):
        if scale is not None:
            x = x / scale.to(f64)[None, :, None]
        c = cache.to(f64).transpose(1, 2).reshape(-1, case["hkv"], case["dim"])
        c[st["slots"]] = x
        out.append(c.view(case["pages"], case["page"], case["hkv"], case["dim"]).transpose(1, 2).contiguous())
    return tuple(out)
