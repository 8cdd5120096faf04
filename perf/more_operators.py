"""Attention and its 4-bit key/value cache as they are measured: attention over
packed prompts, writing keys and values into the cache, attention of new tokens
over the cache (with the weights that eviction goes by), and eviction.

`own` selects between the plain form (elementary torch operations in fp32) and
the library's operators; `exact` evaluates the definitions in float64.

A cache has pages of 64 tokens; a sequence's table names its pages, and place p
of the sequence is token p % 64 of page table[p // 64].  Rows of keys and values
are held as E2M1 codes with a scale per group: NVFP4 16 elements, E4M3, times
one fp32 scale of all keys (values); MXFP4 32 elements, E8M0.
"""
import math
import random

import torch

own = False

PAGE = 64
GROUP = {"nvfp4": 16, "mxfp4": 32}
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # a short question to a small model: launch latency
        dict(name="prompt_tiny", op="prompt", dtype="bf16", hq=4, hkv=2, d=64, b=1, most=37, past=0, mix=0, lse=False),
        # prompts of several users in one batch; 48 heads of 128 over a hidden size of 6144
        dict(name="prompt_packed", op="prompt", dtype="bf16", hq=48, hkv=8, d=128, b=8, most=3001, past=0, mix=1,
             lse=False),
        # one long document; 32 heads of 128 over a hidden size of 4096
        dict(name="prompt_long", op="prompt", dtype="fp16", hq=32, hkv=8, d=128, b=1, most=16384, past=0, mix=0,
             lse=False),
        # chunks of long prompts over the keys of the chunks before them, large heads
        dict(name="prompt_chunks", op="prompt", dtype="bf16", hq=16, hkv=2, d=256, b=2, most=1024, past=9000, mix=2,
             lse=True),
        # one decode step of 32 users: launch latency
        dict(name="append_step", op="append", dtype="bf16", fmt="nvfp4", hkv=8, d=128, b=32, most=1, past=5000, mix=3,
             scaled=True),
        # the prompts of a batch
        dict(name="append_prompts", op="append", dtype="fp16", fmt="mxfp4", hkv=8, d=128, b=5, most=9999, past=700,
             mix=4, scaled=False),
        # one user's short conversation with a small model: launch latency
        dict(name="attend_tiny", op="attend", dtype="bf16", fmt="nvfp4", hq=4, hkv=2, d=64, b=1, rows=1, most=100, mix=0,
             track=False),
        # one user, a context of 128 thousand tokens
        dict(name="attend_long", op="attend", dtype="bf16", fmt="nvfp4", hq=64, hkv=8, d=128, b=1, rows=1, most=131069,
             mix=0, track=False),
        # a serving batch with contexts of all lengths
        dict(name="attend_batch", op="attend", dtype="bf16", fmt="nvfp4", hq=48, hkv=8, d=128, b=64, rows=1, most=30011,
             mix=5, track=False),
        # a token and three drafts for each user, with the weights kept for eviction
        dict(name="attend_drafts", op="attend", dtype="fp16", fmt="mxfp4", hq=32, hkv=4, d=128, b=16, rows=4, most=16000,
             mix=6, track=True),
        # eviction after a short conversation: launch latency
        dict(name="evict_small", op="evict", fmt="mxfp4", hkv=2, d=64, b=2, most=700, keep=256, recent=64, sinks=4,
             mix=7),
        # half of long contexts leaves the cache
        dict(name="evict_long", op="evict", fmt="nvfp4", hkv=8, d=128, b=8, most=32768, keep=12000, recent=1024,
             sinks=4, mix=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "append", "attend", "attend", "attend", "evict"])
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    mix = rng.randint(10, 10 ** 6)
    if op == "prompt":
        hq = hkv * rng.choice([1, 2, 4, 5, 8])
        b = _log(rng, 1, 16)
        # pairs of all sequences stay below those of 32 heads of 128 over 16384 tokens
        top = int(math.sqrt(16384.0 ** 2 * 32 * 128 / (hq * d * b)))
        past = rng.choice([0, 0, _log(rng, 1, 8192)])
        most = _log(rng, 1, min(16384, top) if past == 0 else min(2048, top // 4))
        return dict(op=op, dtype=rng.choice(["bf16", "fp16"]), hq=hq, hkv=hkv, d=d, b=b, most=most, past=past, mix=mix,
                    lse=rng.random() < 0.3)
    if op == "append":
        b = _log(rng, 1, 64)
        most = _log(rng, 1, min(8192, 40000 // b))
        return dict(op=op, dtype=rng.choice(["bf16", "fp16", "fp32"]), fmt=rng.choice(["nvfp4", "mxfp4"]),
                    hkv=rng.choice([1, 2, 4]), d=d, b=b, most=most, past=_log(rng, 1, 5000), mix=mix,
                    scaled=rng.random() < 0.5)
    if op == "attend":
        b = _log(rng, 1, 64)
        rows = rng.choice([1, 1, 2, 4, 8, 16])
        most = _log(rng, 1, min(131072, 5000000 // (b * hkv * (d // 64))))
        return dict(op=op, dtype=rng.choice(["bf16", "fp16"]), fmt=rng.choice(["nvfp4", "nvfp4", "mxfp4"]),
                    hq=hkv * rng.choice([1, 4, 5, 8, 16]), hkv=hkv, d=d, b=b, rows=rows, most=most, mix=mix,
                    track=rng.random() < 0.3)
    b = _log(rng, 1, 16)
    most = _log(rng, 64, min(65536, 2000000 // (b * hkv * (d // 64))))
    keep = _log(rng, 32, most)
    recent = rng.choice([0, keep // 8, keep // 2])
    return dict(op=op, fmt=rng.choice(["nvfp4", "mxfp4"]), hkv=hkv, d=d, b=b, most=most, keep=keep, recent=recent,
                sinks=rng.choice([0, 4]), mix=mix)


def _lengths(c):
    """Tokens that come with this call, and tokens after it, of each sequence."""
    r = random.Random(c["mix"])
    new, all_ = [], []
    for i in range(c["b"]):
        n = c["most"] if i == 0 else _log(r, max(1, c["most"] // 16), c["most"])
        past = c.get("past", 0)
        past = 0 if past == 0 else r.randint(past // 2, past)
        new.append(n)
        all_.append(n + past)
    return new, all_


def _starts(n):
    out = [0]
    for v in n:
        out.append(out[-1] + v)
    return out


def _kept(c):
    return [min(n, c["keep"]) for n in _lengths(c)[0]]


def work(case):
    c = case
    new, full = _lengths(c)
    d, hkv = c["d"], c["hkv"]
    if c["op"] == "prompt":
        s, hq = SIZE[c["dtype"]], c["hq"]
        pairs = sum(n * (a - n) + n * (n + 1) // 2 for n, a in zip(new, full))
        b = s * d * (2 * sum(new) * hq + 2 * sum(full) * hkv) + (4 * sum(new) * hq if c["lse"] else 0)
        return {"bytes": b, "flops": 4 * pairs * hq * d}
    row = d // 2 + d // GROUP[c["fmt"]]
    if c["op"] == "append":
        # rows in, codes and scales out, and read back as the values they stand for
        n = sum(new) * hkv * 2
        return {"bytes": n * (d * SIZE[c["dtype"]] + 2 * row + 4 * d), "flops": 2 * n * d}
    if c["op"] == "attend":
        seen = sum(max(0, a - r) for a in new for r in range(c["rows"]))
        b = 2 * sum(new) * hkv * row + 2 * 2 * c["b"] * c["rows"] * c["hq"] * d
        return {"bytes": b + (8 * sum(new) * hkv if c["track"] else 0), "flops": 4 * seen * c["hq"] * d}
    # weights and positions come in and are read; about keep (1 - keep / n) tokens move; what is kept is read back in bf16
    moved = sum(int(k * (1.0 - k / n)) for n, k in zip(new, _kept(c)))
    kept = sum(_kept(c))
    return {"bytes": hkv * (8 * sum(new) + moved * (4 * row + 16) + kept * (2 * row + 4 * d)), "flops": hkv * 4 * sum(new)}


# ---- inputs ----------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _table(g, full):
    """The pages of each sequence, in the order that a pool hands them out after some use."""
    need = [(n + PAGE - 1) // PAGE for n in full]
    width, total = max(max(need), 1), sum(need)
    order = torch.randperm(total + 3, generator=g, device="cuda").to(torch.int32)[:total]
    table = torch.zeros(len(full), width, dtype=torch.int32, device="cuda")
    for i, (s, n) in enumerate(zip(_starts(need), need)):
        table[i, :n] = order[s:s + n]
    return table, total + 3


_LUT = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _lut(device):
    return torch.tensor(_LUT + [-v for v in _LUT], device=device)


def _pow2(e):
    """2^e in float64 from whole exponents, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _cached(g, pages, hkv, d, fmt, size):
    """Codes and scales of `pages` full pages as quantising leaves them: every group has a code of 6."""
    grp = GROUP[fmt]
    codes = torch.randint(0, 256, (pages, hkv, PAGE, d // 2), generator=g, device="cuda", dtype=torch.uint8)
    # the largest is at any element of a group: here the first or the second
    lead = codes.view(pages, hkv, PAGE, d // grp, grp // 2)[..., 0]
    low = (lead & 16) == 0
    lead.copy_(torch.where(low, lead | 7, lead | 112))
    shape = (pages, hkv, PAGE, d // grp)
    if fmt == "nvfp4":
        # code values have a root mean square of 3; some channels are larger for all tokens
        s = _randn(g, *shape).mul_(0.3).exp_()
        s *= torch.exp(0.5 * _randn(g, 1, hkv, 1, d // grp)) * (size / 3.0)
        scales = s.clamp_(2.0 ** -6, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        e = torch.randint(-1, 2, shape, generator=g, device="cuda") + int(round(math.log2(size / 3.0)))
        scales = (e + 127).to(torch.uint8)
    return codes, scales


def _values(codes, scales, fmt, gs):
    """The fp32 values of codes [..., d/2] and scales [..., d/g]."""
    both = torch.stack((codes & 15, codes >> 4), dim=-1).reshape(*codes.shape[:-1], -1)
    v = _lut(codes.device)[both.to(torch.int32)]
    if fmt == "nvfp4":
        s = scales.view(torch.float8_e4m3fn).to(torch.float32)
    else:
        s = _pow2(scales.to(torch.int64) - 127).to(torch.float32)
    v = (v.view(*s.shape, -1) * s.unsqueeze(-1)).reshape(v.shape)
    return v if gs is None else v * gs


def _fill(cache, st, full):
    """Puts the cached tokens into the library's cache the way a program does: appends them.  They are
    representable, so the cache holds the same codes and scales."""
    c = st["case"]
    for b, n in enumerate(full):
        for p0 in range(0, n, 16384):
            n1 = min(n - p0, 16384)
            rows = st["table"][b, p0 // PAGE:(p0 + n1 + PAGE - 1) // PAGE].to(torch.int64)
            kv = []
            for side in ("k", "v"):
                x = _values(st[side][0][rows], st[side][1][rows], c["fmt"], None)
                kv.append(x.transpose(1, 2).reshape(-1, c["hkv"], c["d"])[:n1])
            cache.append(kv[0], kv[1], st["table"][b:b + 1], _ints([p0 + n1]))


def prepare(case, seed):
    c = case
    g = _gen(seed)
    st = {"case": c}
    new, full = _lengths(c)
    d, hkv = c["d"], c["hkv"]
    if c["op"] == "prompt":
        dt = DTYPE[c["dtype"]]
        T, S, hq = sum(new), sum(full), c["hq"]
        st["new"], st["full"] = new, full
        st["starts"], st["key_starts"] = _ints(_starts(new)), _ints(_starts(full))
        if T == S:
            # queries, keys and values are parts of one projection's rows
            x = _randn(g, T, (hq + 2 * hkv) * d)
            x[:, :hq * d] *= 1.5
            x = x.to(dt)
            st["q"] = x[:, :hq * d].view(T, hq, d)
            st["k"] = x[:, hq * d:(hq + hkv) * d].view(T, hkv, d)
            st["v"] = x[:, (hq + hkv) * d:].view(T, hkv, d)
        else:
            st["q"] = (_randn(g, T, hq, d) * 1.5).to(dt)
            st["k"] = _randn(g, S, hkv, d).to(dt)
            st["v"] = _randn(g, S, hkv, d).to(dt)
        return st
    if c["op"] == "append":
        dt = DTYPE[c["dtype"]]
        T = sum(new)
        st["new"] = new
        st["lens"], st["starts"] = _ints(full), _ints(_starts(new))
        st["table"], pages = _table(g, full)
        # some channels of the keys are large for all tokens; tokens differ in size
        st["k"] = (_randn(g, T, hkv, d) * torch.exp(0.7 * _randn(g, 1, hkv, d))).to(dt)
        st["v"] = (_randn(g, T, hkv, d) * torch.exp(0.3 * _randn(g, T, hkv, 1))).to(dt)
        st["gs"] = (None, None)
        if c["fmt"] == "nvfp4" and c["scaled"]:
            st["gs"] = (torch.full((1,), 0.037, device="cuda"), torch.full((1,), 0.0113, device="cuda"))
        if own:
            from hbm_expert_slot_amd.ops import KV4Cache
            st["cache"] = KV4Cache(pages, hkv, d, c["fmt"], k_scale=st["gs"][0], v_scale=st["gs"][1])
        return st
    st["lens"] = _ints(new)
    st["table"], pages = _table(g, new)
    st["k"] = _cached(g, pages, hkv, d, c["fmt"], 1.0)
    st["v"] = _cached(g, pages, hkv, d, c["fmt"], 1.0)
    if c["op"] == "attend":
        st["q"] = (_randn(g, c["b"], c["rows"], c["hq"], d) * 1.5).to(DTYPE[c["dtype"]])
        track = c["track"]
        if track:
            st["weights0"] = torch.rand(pages, hkv, PAGE, generator=g, device="cuda") * 2.0
            st["weights"] = torch.empty_like(st["weights0"])
    else:
        track = True
        st["kept"] = _kept(c)
        st["starts"] = _ints(_starts(st["kept"]))
        # a few tokens have most of the weight; many have little, in steps, so that some are equal
        w = torch.rand(pages, hkv, PAGE, generator=g, device="cuda")
        st["weights0"] = torch.where(w < 0.2, torch.floor(w * 64.0) / 64.0, w ** -0.7)
        at = torch.zeros(pages, 1, PAGE, dtype=torch.int32, device="cuda")
        for b, n in enumerate(new):
            rows = st["table"][b, :(n + PAGE - 1) // PAGE].to(torch.int64)
            at[rows, 0] = torch.arange(len(rows) * PAGE, dtype=torch.int32, device="cuda").view(-1, PAGE)
        st["positions0"] = at.expand(pages, hkv, PAGE).contiguous()
        st["weights"], st["positions"] = torch.empty_like(st["weights0"]), torch.empty_like(st["positions0"])
    if own:
        from hbm_expert_slot_amd.ops import KV4Cache
        st["cache"] = KV4Cache(pages, hkv, d, c["fmt"], track=track)
        _fill(st["cache"], st, new)
        if track:
            st["weights"], st["positions"] = st["cache"].weights, st["cache"].positions
    return st


# ---- one pass --------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    from hbm_expert_slot_amd import ops
    c = st["case"]
    if c["op"] == "prompt":
        if c["lse"]:
            return ops.prompt_attention(st["q"], st["k"], st["v"], st["starts"], st["key_starts"], return_lse=True)
        return ops.prompt_attention(st["q"], st["k"], st["v"], st["starts"], st["key_starts"])
    cache = st["cache"]
    if c["op"] == "append":
        cache.append(st["k"], st["v"], st["table"], st["lens"], st["starts"])
        return cache.read(st["table"], st["lens"], st["k"].shape[0], st["starts"], dtype=torch.float32)
    if c["op"] == "attend":
        if not c["track"]:
            return cache.attend(st["q"], st["table"], st["lens"])
        # the weights as the steps before have left them
        cache.weights.copy_(st["weights0"])
        return cache.attend(st["q"], st["table"], st["lens"], accumulate=True), cache.weights
    # the weights and positions as the steps before have left them
    cache.weights.copy_(st["weights0"])
    cache.positions.copy_(st["positions0"])
    lens = cache.evict(st["table"], st["lens"], c["keep"], recent=c["recent"], sinks=c["sinks"])
    k, v = cache.read(st["table"], lens, sum(st["kept"]), st["starts"], dtype=torch.bfloat16)
    return k, v, cache.weights, cache.positions, lens


def _plain_round(v, lut):
    """Index of the nearest table value to each v >= 0, ties to the even index."""
    idx = torch.zeros_like(v, dtype=torch.int32)
    for i in range(len(lut) - 1):
        mid = 0.5 * (lut[i] + lut[i + 1])
        idx += ((v >= mid) if i % 2 else (v > mid)).to(torch.int32)
    return idx


def _plain_quant(x, fmt, gs):
    # float64 where a value can lie next to a rounding border
    b = x.to(torch.float64).view(*x.shape[:-1], -1, GROUP[fmt])
    amax = b.abs().amax(-1)
    if fmt == "nvfp4":
        gd = 1.0 if gs is None else gs.to(torch.float64)
        a = torch.clamp(amax / (6.0 * gd), max=448.0)
        _, e = torch.frexp(a)
        step = _pow2(torch.clamp(e - 1, min=-6) - 3)
        full = torch.round(a / step) * step * gd
    else:
        _, e = torch.frexp(amax)
        full = _pow2(torch.clamp(e - 3, -127, 127))
    q = b.abs() / torch.where(full > 0, full, torch.ones_like(full)).unsqueeze(-1)
    code = _plain_round(q, _LUT)
    v = torch.tensor(_LUT, device=x.device, dtype=torch.float64)[code] * torch.sign(b) * full.unsqueeze(-1)
    return v.reshape(x.shape).to(torch.float32)


def _plain_attend(q, k, v, ahead, scale, want_p=False):
    """q [hkv, rows, d] against k, v [hkv, n, d], all fp32; row i sees keys j < ahead[i].  Heads one at a time
    where the scores of all are large."""
    n = k.shape[1]
    seen = torch.arange(n, device=q.device) < ahead.unsqueeze(1)
    outs, lses, ps = [], [], []
    for h in range(q.shape[0]):
        s = (q[h] @ k[h].t()) * scale
        s = torch.where(seen, s, torch.full_like(s, -math.inf))
        m = s.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        p = torch.exp(s - m)
        t = p.sum(-1, keepdim=True)
        lses.append((m + torch.log(t)).squeeze(-1))
        p = p / torch.where(t > 0, t, torch.ones_like(t))
        outs.append(p @ v[h])
        if want_p:
            ps.append(p.sum(0))
    return torch.stack(outs), torch.stack(lses), torch.stack(ps) if want_p else None


def _gather(side, table_row, n, fmt):
    """The first n places of a sequence as fp32 [hkv, n, d]."""
    rows = table_row[:(n + PAGE - 1) // PAGE].to(torch.int64)
    x = _values(side[0][rows], side[1][rows], fmt, None)
    return x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])[:, :n]


def _run_plain(st):
    c = st["case"]
    d, hkv = c["d"], c["hkv"]
    if c["op"] == "prompt":
        g = c["hq"] // hkv
        out = torch.empty(st["q"].shape, dtype=st["q"].dtype, device=st["q"].device)
        lse = torch.empty(out.shape[:2], dtype=torch.float32, device=out.device)
        q0 = k0 = 0
        for n, a in zip(st["new"], st["full"]):
            k = st["k"][k0:k0 + a].to(torch.float32).transpose(0, 1)
            v = st["v"][k0:k0 + a].to(torch.float32).transpose(0, 1)
            ahead = torch.arange(a - n + 1, a + 1, device=out.device)
            for h in range(c["hq"]):
                q = st["q"][q0:q0 + n, h].to(torch.float32).unsqueeze(0)
                o, l, _ = _plain_attend(q, k[h // g:h // g + 1], v[h // g:h // g + 1], ahead, 1.0 / math.sqrt(d))
                out[q0:q0 + n, h] = o[0].to(out.dtype)
                lse[q0:q0 + n, h] = l[0]
            q0 += n
            k0 += a
        return (out, lse) if c["lse"] else out
    if c["op"] == "append":
        return _plain_quant(st["k"], c["fmt"], st["gs"][0]), _plain_quant(st["v"], c["fmt"], st["gs"][1])
    new = _lengths(c)[0]
    if c["op"] == "attend":
        r, g = c["rows"], c["hq"] // hkv
        out = torch.empty_like(st["q"])
        if c["track"]:
            st["weights"].copy_(st["weights0"])
        for b, n in enumerate(new):
            k = _gather(st["k"], st["table"][b], n, c["fmt"])
            v = _gather(st["v"], st["table"][b], n, c["fmt"])
            q = st["q"][b].to(torch.float32).view(r, hkv, g, d).transpose(0, 1).reshape(hkv, r * g, d)
            ahead = torch.arange(n - r + 1, n + 1, device=out.device).repeat_interleave(g)
            o, _, p = _plain_attend(q, k, v, ahead, 1.0 / math.sqrt(d), c["track"])
            out[b] = o.view(hkv, r, g, d).transpose(0, 1).reshape(r, c["hq"], d).to(out.dtype)
            if c["track"]:
                pages = (n + PAGE - 1) // PAGE
                add = torch.zeros(hkv, pages * PAGE, device=out.device)
                add[:, :n] = p
                st["weights"][st["table"][b, :pages].to(torch.int64)] += add.view(hkv, pages, PAGE).transpose(0, 1)
        return (out, st["weights"]) if c["track"] else out
    w, at = st["weights"], st["positions"]
    w.copy_(st["weights0"])
    at.copy_(st["positions0"])
    for b, (n, keep) in enumerate(zip(new, st["kept"])):
        if n <= keep:
            continue
        place = torch.arange(n, device=w.device)
        page, slot = st["table"][b].to(torch.int64)[place // PAGE], place % PAGE
        for h in range(hkv):
            p = at[page, h, slot]
            always = (p < c["sinks"]) | (p > p.max() - c["recent"])
            key = torch.where(always, torch.full_like(w[page, h, slot], math.inf), w[page, h, slot])
            order = torch.sort(key, descending=True, stable=True)[1][:keep]
            stays = torch.zeros(n, dtype=torch.bool, device=w.device)
            stays[order] = True
            free = torch.nonzero(~stays[:keep]).flatten()
            move = torch.nonzero(stays[keep:]).flatten() + keep
            pf, sf, pm, sm = page[free], slot[free], page[move], slot[move]
            for t in (w, at, *st["k"], *st["v"]):
                t[pf, h, sf] = t[pm, h, sm]
    ks, vs = [], []
    for b, n in enumerate(st["kept"]):
        ks.append(_gather(st["k"], st["table"][b], n, c["fmt"]).transpose(0, 1))
        vs.append(_gather(st["v"], st["table"][b], n, c["fmt"]).transpose(0, 1))
    lens = torch.clamp(st["lens"], max=c["keep"])
    return torch.cat(ks).to(torch.bfloat16), torch.cat(vs).to(torch.bfloat16), w, at, lens


# ---- the definitions in float64 ----------------------------------------------

def _e2m1_64(nib):
    """E2M1 from its fields: sign, two exponent bits (bias 1), one mantissa bit."""
    n = nib.to(torch.int64)
    ex, man = (n >> 1) & 3, (n & 1).to(torch.float64)
    mag = torch.where(ex == 0, 0.5 * man, (1.0 + 0.5 * man) * _pow2(ex - 1))
    return torch.where(n > 7, -mag, mag)


def _e4m3_64(b):
    """E4M3 from its fields: four exponent bits (bias 7), three mantissa bits."""
    n = b.to(torch.int64)
    ex, man = (n >> 3) & 15, (n & 7).to(torch.float64)
    mag = torch.where(ex == 0, man / 512.0, (1.0 + man / 8.0) * _pow2(ex - 7))
    return torch.where(n > 127, -mag, mag)


def _rows_64(side, pages, h, n, fmt):
    codes, scales = side[0][pages, h].reshape(-1, side[0].shape[3])[:n], side[1][pages, h].reshape(-1, side[1].shape[3])[:n]
    x = torch.empty(n, codes.shape[1] * 2, dtype=torch.float64, device=codes.device)
    x[:, 0::2] = _e2m1_64(codes & 15)
    x[:, 1::2] = _e2m1_64(codes >> 4)
    s = _e4m3_64(scales) if fmt == "nvfp4" else _pow2(scales.to(torch.int64) - 127)
    return x * s.repeat_interleave(GROUP[fmt], dim=1)


def _softmax_rows_64(q, k, v, first):
    """Rows of q against the keys; row i sees `first + i` of them."""
    z = (q @ k.t()) / math.sqrt(q.shape[1])
    col = torch.arange(k.shape[0], device=q.device).unsqueeze(0)
    row = torch.arange(q.shape[0], device=q.device).unsqueeze(1)
    z.masked_fill_(col >= first + row, -math.inf)
    lse = torch.logsumexp(z, dim=1)
    z.sub_(lse.clamp(min=-1e300).unsqueeze(1)).exp_()
    return z @ v, lse, z


def _quant_64(x, fmt, gs):
    g = GROUP[fmt]
    w = x.to(torch.float64)
    a = w.abs().reshape(-1, g)
    big = a.amax(-1)
    if fmt == "nvfp4":
        gs = 1.0 if gs is None else gs.to(torch.float64)
        grid = _e4m3_64(torch.arange(127, device=w.device))            # 0 .. 448
        t = big / (6.0 * gs)
        mids = 0.5 * (grid[1:] + grid[:-1])
        lo = torch.searchsorted(mids, t, right=False)                  # ties: the lower value
        hi = torch.searchsorted(mids, t, right=True)                   # ties: the upper value
        d = grid[torch.where(lo % 2 == 0, lo, hi)] * gs
    else:
        # the exponent field of the float64 value (0 for a block of zeros)
        ex = (big.view(torch.int64) >> 52) - 1023
        d = _pow2(torch.clamp(ex - 2, -127, 127))
    values = _e2m1_64(torch.arange(8, device=w.device))
    borders = 0.5 * (values[1:] + values[:-1])
    out = torch.empty_like(a)
    for i in range(0, a.shape[0], 1 << 20):
        ai, di = a[i:i + (1 << 20)], d[i:i + (1 << 20)]
        cut = (di.unsqueeze(-1) * borders).unsqueeze(-2)               # exact products
        code = (ai.unsqueeze(-1) > cut).sum(-1)
        tie = (ai.unsqueeze(-1) == cut).any(-1) & (code % 2 == 1)
        code = torch.where((di > 0).unsqueeze(-1), code + tie.to(code.dtype), torch.zeros_like(code))
        out[i:i + (1 << 20)] = values[code] * di.unsqueeze(-1)
    return torch.copysign(out.view(w.shape), w)


def _pages_of(st, b, n):
    return st["table"][b, :(n + PAGE - 1) // PAGE].to(torch.int64)


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    f64 = dict(dtype=torch.float64, device="cuda")
    new, full = _lengths(c)
    if c["op"] == "prompt":
        out, lse = torch.zeros(st["q"].shape, **f64), torch.zeros(st["q"].shape[:2], **f64)
        q0 = k0 = 0
        for n, a in zip(new, full):
            for h in range(c["hq"]):
                j = h * c["hkv"] // c["hq"]
                k, v = st["k"][k0:k0 + a, j].to(torch.float64), st["v"][k0:k0 + a, j].to(torch.float64)
                for r in range(0, n, 2048):
                    m = min(2048, n - r)
                    q = st["q"][q0 + r:q0 + r + m, h].to(torch.float64)
                    top = a - n + r + m
                    o, l, _ = _softmax_rows_64(q, k[:top], v[:top], a - n + r + 1)
                    out[q0 + r:q0 + r + m, h], lse[q0 + r:q0 + r + m, h] = o, l
            q0, k0 = q0 + n, k0 + a
        return (out, lse) if c["lse"] else out
    if c["op"] == "append":
        return _quant_64(st["k"], c["fmt"], st["gs"][0]), _quant_64(st["v"], c["fmt"], st["gs"][1])
    if c["op"] == "attend":
        out = torch.zeros(st["q"].shape, **f64)
        w = st["weights0"].to(torch.float64) if c["track"] else None
        g = c["hq"] // c["hkv"]
        for b, n in enumerate(new):
            pages = _pages_of(st, b, n)
            for j in range(c["hkv"]):
                k, v = (_rows_64(st[s], pages, j, n, c["fmt"]) for s in ("k", "v"))
                p = torch.zeros(len(pages) * PAGE, **f64)
                for h in range(j * g, j * g + g):
                    o, l, z = _softmax_rows_64(st["q"][b, :, h].to(torch.float64), k, v, n - c["rows"] + 1)
                    out[b, :, h] = o
                    p[:n] += z.sum(0)
                if c["track"]:
                    w[pages, j] += p.view(-1, PAGE)
        return (out, w) if c["track"] else out
    # whole numbers and moved values: by counting larger weights on the host
    w, at = st["weights0"].cpu(), st["positions0"].cpu()
    table = st["table"].cpu().to(torch.int64)
    ks, vs = [], []
    for b, (n, keep) in enumerate(zip(new, st["kept"])):
        place = torch.arange(n)
        page, slot = table[b][place // PAGE], place % PAGE
        source = torch.arange(keep).repeat(c["hkv"], 1)
        if n > keep:
            for h in range(c["hkv"]):
                p, x = at[page, h, slot], w[page, h, slot].to(torch.float64)
                x[(p < c["sinks"]) | (p > int(p.max()) - c["recent"])] = math.inf
                least = torch.sort(x)[0][n - keep]                      # the keep-th largest
                stays = x > least
                equal = torch.nonzero(x == least).flatten()
                stays[equal[:keep - int(stays.sum())]] = True
                free = torch.nonzero(~stays[:keep]).flatten()
                source[h, free] = torch.nonzero(stays[keep:]).flatten() + keep
            old_w, old_at = w[page].clone(), at[page].clone()           # [n, hkv, 64] by place
            for h in range(c["hkv"]):
                src = source[h]
                w[page[:keep], h, slot[:keep]] = old_w[src, h, src % PAGE]
                at[page[:keep], h, slot[:keep]] = old_at[src, h, src % PAGE]
        for side, outs in (("k", ks), ("v", vs)):
            cols = []
            for h in range(c["hkv"]):
                x = _rows_64(st[side], _pages_of(st, b, n), h, n, c["fmt"])
                cols.append(x[source[h].cuda()])
            outs.append(torch.stack(cols, dim=1))
    return torch.cat(ks), torch.cat(vs), w.cuda().to(torch.float64), at.cuda(), _ints(st["kept"])
