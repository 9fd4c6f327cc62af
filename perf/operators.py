"""Performance cases of the serving-step operators: block tables and slot maps
built from request lengths (kv_plan), the 4-bit paged KV cache (kv4_append,
kv4_gather, kv4_decode_attention) and the log probabilities of given tokens
(token_logprobs).

Every case runs in two forms on the same inputs: the plain form, elementary
torch operations in 32 bits (64 where 32 lose what matters), and, with
``own`` set, the calls a user makes of this package.  ``exact`` gives the
same outputs from the definitions in 64 bits, written apart from both.

The 4-bit cache holds, per layer and separately for K and V, a uint8 tensor
[num_blocks, kv_heads, page_size / 16, 9 * head_dim]: each tile of 16 tokens
of one kv head is its e2m1 codes [16, head_dim / 2] (element 2j in the low
nibble of byte j) followed by its e4m3 scales [16, head_dim / 16], one per 16
consecutive elements; an element stands for code * scale * s with one fp32 s
per layer.
"""
import math
import random

import torch

own = False

DEV = "cuda"
F32, F64, BF16, I32, I64, U8 = torch.float32, torch.float64, torch.bfloat16, torch.int32, torch.int64, torch.uint8


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 64 running requests, one new token each: the smallest plan, pure latency
        dict(name="plan-decode-64", op="plan", batch=64, page=16, kind="decode", max_ctx=16384, tokens=64, short=False,
             lens_seed=1),
        # continuous batching: prompt chunks of some requests beside single tokens of the others
        dict(name="plan-mixed-509", op="plan", batch=509, page=32, kind="mixed", max_ctx=8192, tokens=16384,
             short=False, lens_seed=2),
        # the new keys and values of one decode step (32 requests), written and read back
        dict(name="append-decode-32", op="append", tokens=32, hq=32, hkv=8, d=128, page=16),
        # a large prompt chunk, k and v taken from the fused projection's rows
        dict(name="append-prompt-8191", op="append", tokens=8191, hq=32, hkv=8, d=128, page=64),
        # a short cached prefix read back for a dense prompt attention, narrow heads
        dict(name="gather-prefix-777", op="gather", tokens=777, hkv=2, d=64, page=48),
        # long cached prefixes of several requests read back in bf16
        dict(name="gather-prefix-65536", op="gather", tokens=65536, hkv=8, d=128, page=16),
        # one request, a short context: latency
        dict(name="attend-1x1021", op="attend", batch=1, kind="equal", max_len=1021, hq=32, hkv=8, d=128, page=16,
             qn=1, window=0, lens_seed=3),
        # a uniform decode batch
        dict(name="attend-8x4096", op="attend", batch=8, kind="equal", max_len=4096, hq=32, hkv=8, d=128, page=16,
             qn=1, window=0, lens_seed=4),
        # a ragged decode batch up to long contexts
        dict(name="attend-ragged-48x32768", op="attend", batch=48, kind="ragged", max_len=32768, hq=32, hkv=8, d=128,
             page=16, qn=1, window=0, lens_seed=5),
        # several query tokens per request (drafted tokens being verified), five query heads per kv head
        dict(name="attend-verify-16x8192", op="attend", batch=16, kind="ragged", max_len=8192, hq=40, hkv=8, d=128,
             page=64, qn=4, window=0, lens_seed=6),
        # the lm_head's logits of one sequence: latency over a long row
        dict(name="logprobs-1x152064", op="logprobs", rows=1, vocab=152064, k=20, dtype="bf16", pad=0, masked=False),
        # scoring a prompt: every position's logits
        dict(name="logprobs-2048x152064", op="logprobs", rows=2048, vocab=152064, k=20, dtype="bf16", pad=0,
             masked=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "gather", "attend", "attend", "attend", "logprobs", "logprobs"])
    if op == "plan":
        batch = _log(rng, 1, 1024)
        kind = rng.choice(["decode", "mixed"])
        page = rng.choice([16, 32, 48, 64, 128, 256])
        tokens = batch if kind == "decode" else max(4 * batch, _log(rng, 64, 32768))
        return dict(op=op, batch=batch, page=page, kind=kind, max_ctx=_log(rng, 16, 32768), tokens=tokens,
                    short=rng.random() < 0.25, lens_seed=rng.randrange(1 << 30))
    if op in ("append", "gather"):
        hkv = rng.choice([1, 2, 4, 8])
        d = rng.choice([64, 128])
        case = dict(op=op, tokens=_log(rng, 1, 8191 if op == "append" else 65536), hkv=hkv, d=d,
                    page=rng.choice([16, 32, 48, 64, 128, 256]))
        if op == "append":
            case["hq"] = hkv * rng.choice([1, 4, 5, 8])
        return case
    if op == "attend":
        while True:
            hkv = rng.choice([1, 2, 4, 8])
            case = dict(op=op, batch=_log(rng, 1, 48), kind=rng.choice(["equal", "ragged"]),
                        max_len=_log(rng, 1, 32768), hq=hkv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16]), hkv=hkv,
                        d=rng.choice([64, 128]), page=rng.choice([16, 32, 48, 64, 128, 256]),
                        qn=rng.choice([1, 1, 1, 2, 4, 7]), window=rng.choice([0, 0, 0, 128, 1000, 4096]),
                        lens_seed=rng.randrange(1 << 30))
            w, top = work(case), work(listed()[8])
            if w["bytes"] <= top["bytes"] and w["flops"] <= 2 * top["flops"]:
                return case
    while True:
        case = dict(op=op, rows=_log(rng, 1, 2048), vocab=_log(rng, 1000, 152064), k=rng.choice([1, 2, 5, 20, 32]),
                    dtype=rng.choice(["bf16", "f32"]), pad=rng.choice([0, 0, 1, 8, 64]), masked=rng.random() < 0.25)
        if work(case)["bytes"] <= work(listed()[11])["bytes"]:
            return case


def _lens(case):
    """The lengths of a plan or attend case: a fixed function of the case."""
    rng = random.Random(case["lens_seed"])
    if case["op"] == "attend":
        if case["kind"] == "equal":
            lens = [case["max_len"]] * case["batch"]
        else:
            lens = [_log(rng, 1, case["max_len"]) for _ in range(case["batch"])]
            lens[rng.randrange(case["batch"])] = case["max_len"]
        qls = [min(n, rng.randint(1, case["qn"])) for n in lens]
        return lens, qls
    ctx = [rng.randint(0, case["max_ctx"]) for _ in range(case["batch"])]
    if case["kind"] == "decode":
        return ctx, [1] * case["batch"]
    new, left = [], case["tokens"] - case["batch"]
    for i in range(case["batch"]):
        n = rng.choice([0, 1, 1, 1, 1, 1])
        if left > 0 and rng.random() < 0.1:
            more = min(left, _log(rng, 1, 4096))
            n, left = n + more, left - more
        new.append(n)
    return ctx, new


def _visible(case):
    """Keys that the rows of each sequence can see at all: a window hides the oldest."""
    lens, qls = _lens(case)
    return [n if not case["window"] else min(n, case["window"] + q - 1) for n, q in zip(lens, qls)]


def work(case):
    """Bytes and operations a pass cannot do without: inputs read once, outputs written once."""
    op = case["op"]
    if op == "plan":
        ctx, new = _lens(case)
        p = case["page"]
        pages = sum((c + n + p - 1) // p - (c + p - 1) // p for c, n in zip(ctx, new))
        b, t = case["batch"], case["tokens"]
        return {"bytes": 4 * (2 * b + 2 * b + 1 + 2 * pages + 3 * t + b), "flops": 0}
    if op == "append":
        e = 2 * case["tokens"] * case["hkv"] * case["d"]       # elements of k and v
        held = e // 2 + e // 16
        return {"bytes": 2 * e + held + held + 2 * e + 4 * case["tokens"], "flops": 0}
    if op == "gather":
        e = 2 * case["tokens"] * case["hkv"] * case["d"]
        return {"bytes": e // 2 + e // 16 + 2 * e + 4 * case["tokens"], "flops": 0}
    if op == "attend":
        lens, qls = _lens(case)
        vis = _visible(case)
        held = case["hkv"] * case["d"] * 9 // 16
        rows = sum(qls) * case["hq"]
        flops = 0
        for n, q in zip(lens, qls):
            for i in range(q):
                seen = n - q + i + 1
                flops += 4 * case["hq"] * case["d"] * (min(seen, case["window"]) if case["window"] else seen)
        pages = sum((n + case["page"] - 1) // case["page"] for n in vis)
        return {"bytes": 2 * held * sum(vis) + 4 * rows * case["d"] + 4 * rows + 4 * pages + 8 * case["batch"],
                "flops": flops}
    size = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": case["rows"] * (size * case["vocab"] + 4 + 8 + 8 * case["k"]),
            "flops": 4 * case["rows"] * case["vocab"]}


# ------------------------------------------------------- the 4-bit format, plain
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)          # e2m1


def _encode(x, s):
    """x [..., D] -> e2m1 codes (0..15) and e4m3 scale bytes [..., D / 16]:
    scale = e4m3(amax / (6 s)), code = e2m1(x / (s * scale)), each quotient
    and product one fp32 rounding; a group whose scale is 0 holds zeros."""
    g = x.to(F32).unflatten(-1, (-1, 16))
    amax = g.abs().amax(-1)
    sc = (amax / (s * 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    den = (sc.to(F32) * s).unsqueeze(-1)
    q = torch.where(den > 0, g / den, torch.zeros_like(g))
    a = q.abs()
    mag = ((a > 0.25).to(U8) + (a >= 0.75).to(U8) + (a > 1.25).to(U8) + (a >= 1.75).to(U8) + (a > 2.5).to(U8)
           + (a >= 3.5).to(U8) + (a > 5.0).to(U8))              # halfway goes to the even code
    return (mag + 8 * (q < 0).to(U8)).flatten(-2), sc.view(U8)


def _decode(codes, scales, s):
    """Codes [..., D] and scale bytes [..., D / 16] -> fp32 values."""
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), dtype=F32, device=codes.device)
    sc = scales.view(torch.float8_e4m3fn).to(F32).unsqueeze(-1)
    return ((table[codes.long()].unflatten(-1, (-1, 16)) * sc) * s).flatten(-2)


def _views(cache, d):
    """The code bytes [nb, hkv, tiles, 16, d / 2] and scales [.., 16, d / 16] of a cache."""
    return cache[..., :8 * d].unflatten(-1, (16, d // 2)), cache[..., 8 * d:].unflatten(-1, (16, d // 16))


def _place(slots, page):
    slots = slots.long()
    return slots // page, slots % page // 16, slots % 16


def _store(x, slots, s, cache, page):
    codes, scales = _encode(x, s)
    keep = slots >= 0
    blk, tile, row = _place(slots[keep], page)
    cv, sv = _views(cache, x.shape[-1])
    cv[blk, :, tile, row] = (codes[..., 0::2] | (codes[..., 1::2] << 4))[keep]
    sv[blk, :, tile, row] = scales[keep]


def _load(cache, slots, s, page, d):
    """fp32 values [T, hkv, d] of the tokens at slots; zeros where a slot is -1."""
    blk, tile, row = _place(slots.clamp(min=0), page)
    cv, sv = _views(cache, d)
    b = cv[blk, :, tile, row]
    x = _decode(torch.stack((b & 15, b >> 4), -1).flatten(-2), sv[blk, :, tile, row], s)
    return torch.where((slots >= 0)[:, None, None], x, torch.zeros_like(x))


# --------------------------------------------------------------- preparation
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _fill_cache(g, shape, s, mean):
    """A cache of quantized normal values: its tiles are drawn from 2048 quantized ones."""
    nb, hkv, tiles, nbytes = shape
    d = nbytes // 9
    x = torch.randn((2048 * 16, 1, d), generator=g, device=DEV, dtype=F32) + mean
    pool = torch.zeros((2048, 1, 1, nbytes), dtype=U8, device=DEV)
    _store(x.to(BF16), torch.arange(2048 * 16, device=DEV), s, pool, 16)
    pick = torch.randint(0, 2048, (nb * hkv * tiles,), generator=g, device=DEV)
    return pool.view(2048, nbytes)[pick].view(shape)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case=case)
    if op == "plan":
        ctx, new = _lens(case)
        p, b = case["page"], case["batch"]
        held = [(c + p - 1) // p for c in ctx]
        need = sum((c + n + p - 1) // p for c, n in zip(ctx, new)) - sum(held)
        st["max_blocks"] = max((c + n + p - 1) // p for c, n in zip(ctx, new)) + 3
        used = 11                                               # free blocks that earlier steps took
        spare = need // 2 if case["short"] else need + 40       # a pool that runs out, or does not
        st["num_blocks"] = sum(held) + used + spare
        perm = torch.randperm(st["num_blocks"], generator=g, device=DEV).to(I32)
        col = torch.arange(st["max_blocks"], device=DEV)[None]
        hold = torch.tensor(held, device=DEV)
        first = torch.cumsum(hold, 0) - hold
        st["table"] = torch.where(col < hold[:, None], perm[(first[:, None] + col).clamp(max=st["num_blocks"] - 1)],
                                  torch.full_like(perm[:1], -1))
        st["free"] = perm[sum(held):].contiguous()
        st["head"] = torch.tensor([used], dtype=I32, device=DEV)
        st["ctx"] = torch.tensor(ctx, dtype=I32, device=DEV)
        st["new"] = torch.tensor(new, dtype=I32, device=DEV)
        return st
    if op == "logprobs":
        dt = BF16 if case["dtype"] == "bf16" else F32
        m, v = case["rows"], case["vocab"]
        full = torch.empty((m, v + case["pad"]), dtype=dt, device=DEV)
        for i in range(0, m, 256):                              # a model's logits: a normal bulk, a few tall ones
            x = torch.randn((min(256, m - i), v + case["pad"]), generator=g, device=DEV) * 2.0
            tall = torch.randint(0, v, (x.shape[0], 8), generator=g, device=DEV)
            x.scatter_add_(1, tall, torch.rand(tall.shape, generator=g, device=DEV) * 12)
            full[i:i + 256] = x.to(dt)
        st["logits"] = full[:, :v]
        st["targets"] = torch.randint(0, v, (m,), generator=g, device=DEV).to(I32)
        if case["masked"]:                                      # constrained decoding: most of the vocabulary is shut
            open_ = torch.rand((m, v), generator=g, device=DEV) < max(0.05, 64.0 / v)
            open_.scatter_(1, st["targets"].long()[:, None], True)
            open_[:, :40] = True
            st["logits"].masked_fill_(~open_, -math.inf)
        return st
    hkv, d, page = case["hkv"], case["d"], case["page"]
    st["ks"] = torch.tensor([5.5 / 2688], device=DEV)
    st["vs"] = torch.tensor([6.0 / 2688], device=DEV)
    if op in ("append", "gather"):
        t = case["tokens"]
        nb = (t + page - 1) // page + 3
        st["slots"] = torch.randperm(nb * page, generator=g, device=DEV)[:t].to(I32)
        if t > 8:
            st["slots"][t - 1] = -1                             # padding of a captured step
        shape = (nb, hkv, page // 16, 9 * d)
        if op == "append":
            hq = case["hq"]
            qkv = torch.randn((t, (hq + 2 * hkv) * d), generator=g, device=DEV).to(BF16)
            st["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
            st["v"] = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
            st["kc"] = torch.zeros(shape, dtype=U8, device=DEV)
            st["vc"] = torch.zeros(shape, dtype=U8, device=DEV)
        else:
            st["kc"] = _fill_cache(g, shape, st["ks"], 0.0)
            st["vc"] = _fill_cache(g, shape, st["vs"], 0.25)
        return st
    lens, qls = _lens(case)
    need = [(n + page - 1) // page for n in lens]
    nb = sum(need) + 3
    shape = (nb, hkv, page // 16, 9 * d)
    st["kc"] = _fill_cache(g, shape, st["ks"], 0.0)
    st["vc"] = _fill_cache(g, shape, st["vs"], 0.25)
    perm = torch.randperm(nb, generator=g, device=DEV).to(I32)
    table = torch.full((len(lens), max(need)), -1, dtype=I32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    table = table.to(DEV)
    st["table"] = torch.where(table >= 0, perm[table.clamp(min=0).long()], table)
    st["lens"] = torch.tensor(lens, dtype=I32, device=DEV)
    cu = [0]
    for q in qls:
        cu.append(cu[-1] + q)
    st["cu"] = torch.tensor(cu, dtype=I32, device=DEV)
    qkv = torch.randn((cu[-1], (case["hq"] + 2 * hkv) * d), generator=g, device=DEV).to(BF16) * 1.5
    st["q"] = qkv[:, :case["hq"] * d].unflatten(1, (case["hq"], d))
    st["sm"] = d ** -0.5
    if own:
        import fp8_block_scaled_02_gb300 as fp8bs
        st["ws"] = fp8bs.kv4_workspace(d, DEV)
    return st


# ----------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    import fp8_block_scaled_02_gb300 as fp8bs
    case = st["case"]
    op = case["op"]
    if op == "plan":
        p = fp8bs.kv_plan(st["ctx"], st["new"], st["table"], st["free"], st["head"], case["page"], st["num_blocks"],
                          case["tokens"])
        return dict(seq_lens=p.seq_lens, cu_new=p.cu_new, slots=p.slots, positions=p.positions, requests=p.requests,
                    free_head=p.free_head, table=st["table"])
    if op == "append":
        fp8bs.kv4_append(st["k"], st["v"], st["slots"], st["ks"], st["vs"], st["kc"], st["vc"])
        k, v = fp8bs.kv4_gather(st["kc"], st["vc"], st["slots"], st["ks"], st["vs"])
        return dict(k=k, v=v)
    if op == "gather":
        k, v = fp8bs.kv4_gather(st["kc"], st["vc"], st["slots"], st["ks"], st["vs"])
        return dict(k=k, v=v)
    if op == "attend":
        many = case["qn"] > 1
        o, lse = fp8bs.kv4_decode_attention(st["q"], st["kc"], st["vc"], st["ks"], st["vs"], st["table"], st["lens"],
                                            case["max_len"], st["sm"], st["ws"], cu_q=st["cu"] if many else None,
                                            max_q=case["qn"], window=case["window"], return_lse=True)
        return dict(o=o, lse=lse)
    r = fp8bs.token_logprobs(st["logits"], st["targets"], case["k"])
    return dict(logprobs=r.logprobs, entropy=r.entropy, top_ids=r.top_ids, top_logprobs=r.top_logprobs)


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "plan":
        return _plan_plain(st)
    if op == "append":
        for x, s, c in ((st["k"], st["ks"], st["kc"]), (st["v"], st["vs"], st["vc"])):
            _store(x, st["slots"], s, c, case["page"])
    if op in ("append", "gather"):
        k = _load(st["kc"], st["slots"], st["ks"], case["page"], case["d"]).to(BF16)
        v = _load(st["vc"], st["slots"], st["vs"], case["page"], case["d"]).to(BF16)
        return dict(k=k, v=v)
    if op == "attend":
        return _attend_plain(st)
    return _logprobs_plain(st)


def _plan_plain(st):
    case = st["case"]
    p, t, b = case["page"], case["tokens"], case["batch"]
    ctx, new, head = st["ctx"].long(), st["new"].long(), st["head"].long()
    n_free = st["free"].numel()
    cap = st["max_blocks"] * p
    cu = torch.zeros(b + 1, dtype=I64, device=DEV)
    cu[1:] = torch.cumsum(new.clamp(min=0), 0)
    ok = (ctx >= 0) & (new >= 0) & (ctx + new <= cap) & (cu[1:] <= t)
    have = (ctx + p - 1) // p
    need = torch.where(ok, (ctx + new + p - 1) // p - have, torch.zeros_like(ctx))
    upto = torch.cumsum(need, 0)
    granted = ok & ((need == 0) | (head + upto <= n_free))
    seq = torch.where(granted, ctx + new, ctx.clamp(0, cap))
    taken = torch.where(granted, upto, torch.zeros_like(upto)).max()
    j = torch.arange(t, device=DEV)
    req = torch.searchsorted(cu[1:].contiguous(), j, right=True)
    live = req < b
    r = req.clamp(max=b - 1)
    pos = ctx[r] + j - cu[r]
    live_ok = live & granted[r]
    pg = (pos // p).clamp(0, st["max_blocks"] - 1)
    fresh = pg >= have[r]
    pick = (head + upto[r] - need[r] + pg - have[r]).clamp(0, max(n_free - 1, 0))
    blk = torch.where(fresh, st["free"][pick].long() if n_free else torch.full_like(pg, -1), st["table"][r, pg].long())
    bad = (blk < 0) | (blk >= st["num_blocks"])
    minus = torch.full_like(j, -1)
    table = st["table"]
    opens = live_ok & fresh & (pos % p == 0)
    table.view(-1).index_put_(((r * st["max_blocks"] + pg)[opens],), torch.where(bad, minus, blk)[opens].to(I32))
    return dict(seq_lens=seq.to(I32), cu_new=cu.to(I32),
                slots=torch.where(live_ok & ~bad, blk * p + pos % p, minus).to(I32),
                positions=torch.where(live_ok, pos, minus).to(I32), requests=torch.where(live, req, minus).to(I32),
                free_head=(head + taken).to(I32), table=table)


def _attend_plain(st):
    case = st["case"]
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    lens, qls = _lens(case)
    out = torch.empty((sum(qls), hq, d), dtype=BF16, device=DEV)
    lse = torch.empty((sum(qls), hq), dtype=F32, device=DEV)
    at = 0
    for b, (n, q) in enumerate(zip(lens, qls)):
        i = torch.arange(n, device=DEV)
        slots = st["table"][b].long()[i // page] * page + i % page
        k = _load(st["kc"], slots, st["ks"], page, d).transpose(0, 1)                    # [hkv, n, d]
        v = _load(st["vc"], slots, st["vs"], page, d).transpose(0, 1)
        x = st["q"][at:at + q].to(F32).view(q, hkv, hq // hkv, d).permute(1, 0, 2, 3).reshape(hkv, -1, d)
        s = (x @ k.transpose(1, 2) * st["sm"]).view(hkv, q, hq // hkv, n)
        own_pos = (n - q + torch.arange(q, device=DEV))[None, :, None, None]
        dead = i > own_pos
        if case["window"]:
            dead = dead | (i <= own_pos - case["window"])
        s = s.masked_fill(dead, -math.inf)
        m = s.amax(-1, keepdim=True)
        e = torch.exp(s - m)
        z = e.sum(-1, keepdim=True)
        o = ((e / z).view(hkv, -1, n) @ v).view(hkv, q, hq // hkv, d)
        out[at:at + q] = o.permute(1, 0, 2, 3).reshape(q, hq, d).to(BF16)
        lse[at:at + q] = (m + torch.log(z)).squeeze(-1).permute(1, 0, 2).reshape(q, hq)
        at += q
    return dict(o=out, lse=lse)


def _logprobs_plain(st):
    case = st["case"]
    m, v, k = case["rows"], case["vocab"], case["k"]
    lp = torch.empty(m, dtype=F32, device=DEV)
    ent = torch.empty(m, dtype=F32, device=DEV)
    ids = torch.empty((m, k), dtype=I32, device=DEV)
    tops = torch.empty((m, k), dtype=F32, device=DEV)
    back = (v - 1 - torch.arange(v, device=DEV))[None]
    for i in range(0, m, 128):
        x = st["logits"][i:i + 128].to(F32)
        top = x.amax(-1, keepdim=True)
        y = x - top
        e = torch.exp(y)
        z = e.sum(-1, keepdim=True)
        lz = torch.log(z)
        lp[i:i + 128] = (y.gather(1, st["targets"][i:i + 128].long()[:, None]) - lz).squeeze(1)
        ent[i:i + 128] = (lz - torch.where(e > 0, y * e, e).sum(-1, keepdim=True) / z).squeeze(1)
        if k:
            bits = x.view(I32)                                  # an order of integers: the value, then the lowest index
            key = torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF).long() * (1 << 32) + back
            best = v - 1 - (torch.topk(key, k, dim=1).values & 0xFFFFFFFF)
            ids[i:i + 128] = best.to(I32)
            tops[i:i + 128] = y.gather(1, best) - lz
    return dict(logprobs=lp, entropy=ent, top_ids=ids, top_logprobs=tops)


# ------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return dict(plan=_plan_exact, append=_append_exact, gather=_append_exact, attend=_attend_exact,
                logprobs=_logprobs_exact)[case["op"]](st)


def _plan_exact(st):
    case = st["case"]
    p, t, nb = case["page"], case["tokens"], st["num_blocks"]
    ctx, new, table, free = (st[n].cpu().tolist() for n in ("ctx", "new", "table", "free"))
    head0 = int(st["head"])
    cap = st["max_blocks"] * p
    asked, head = head0, head0
    seq, cu = [], [0]
    slots, positions, requests = [-1] * t, [-1] * t, [-1] * t
    for b, (c, n) in enumerate(zip(ctx, new)):
        first = cu[-1]
        cu.append(first + max(n, 0))
        for i in range(first, min(cu[-1], t)):
            requests[i] = b
        good = c >= 0 and n >= 0 and c + n <= cap and cu[-1] <= t
        have = -(-c // p)
        need = -(-(c + n) // p) - have if good else 0
        if good and need and asked + need > len(free):
            good = False
        at = asked
        asked += need
        seq.append(c + n if good else min(max(c, 0), cap))
        if not good:
            continue
        if need:
            head = asked
        for i in range(need):
            f = free[at + i]
            table[b][have + i] = f if 0 <= f < nb else -1
        for i in range(n):
            positions[first + i] = c + i
            blk = table[b][(c + i) // p]
            if 0 <= blk < nb:
                slots[first + i] = blk * p + (c + i) % p
    ints = dict(seq_lens=seq, cu_new=cu, slots=slots, positions=positions, requests=requests, free_head=[head],
                table=table)
    return {n: torch.tensor(v, dtype=I64) for n, v in ints.items()}


def _e4m3_values(dev):
    """The 127 non-negative finite e4m3 values in the order of their codes."""
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:127], dtype=F64, device=dev)


def _nearest(a, values):
    """The index of the nearest of the ascending values; halfway takes the even index."""
    hi = torch.searchsorted(values, a.contiguous()).clamp(1, len(values) - 1)
    lo = hi - 1
    up, down = values[hi] - a, a - values[lo]
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def _append_exact(st):
    """What the tokens' slots hold after the call, unrounded."""
    case = st["case"]
    e4 = _e4m3_values(DEV)
    e2 = torch.tensor(MAGNITUDES, dtype=F64, device=DEV)
    res = {}
    for name, sname, cname in (("k", "ks", "kc"), ("v", "vs", "vc")):
        s = st[sname].double()
        if case["op"] == "append":
            x = st[name].double()
            x = x.reshape(*x.shape[:-1], -1, 16)
            six = (6.0 * s).float().double()
            sc = e4[_nearest((x.abs().amax(-1) / six).float().double(), e4)]
            den = (sc * s).float().double()[..., None]
            quot = (x / torch.where(den > 0, den, torch.ones_like(den))).float().double()
            val = torch.where(den > 0, torch.sign(quot) * e2[_nearest(quot.abs(), e2)], torch.zeros_like(x))
            val = (val * sc[..., None] * s).flatten(-2)
        else:
            d, page = case["d"], case["page"]
            slot = st["slots"].long().clamp(min=0)
            tiles = st[cname][slot // page, :, slot % page // 16].long()                  # [T, hkv, 9 d]
            row = (slot % 16)[:, None, None]
            byte = torch.arange(d // 2, device=DEV)[None, None] + row * (d // 2)
            code = tiles.gather(2, byte.expand(-1, tiles.shape[1], -1))
            nib = torch.stack((code % 16, code // 16), -1).flatten(-2)
            at = 8 * d + torch.arange(d // 16, device=DEV)[None, None] + row * (d // 16)
            sc = e4[tiles.gather(2, at.expand(-1, tiles.shape[1], -1)).clamp(max=126)]
            val = e2[nib % 8] * torch.where(nib >= 8, -1.0, 1.0) * sc.repeat_interleave(16, -1) * s
        res[name] = torch.where((st["slots"] >= 0)[:, None, None], val, torch.zeros_like(val))
    return res


def _attend_exact(st):
    case = st["case"]
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    lens, qls = _lens(case)
    if sum(lens) * hkv * d > 1 << 30:
        return None
    e4 = _e4m3_values(DEV)
    signed = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), dtype=F64, device=DEV)
    o_all, l_all = [], []
    at = 0
    for b, (n, q) in enumerate(zip(lens, qls)):
        pages = st["table"][b, :(n + page - 1) // page].long()
        kv = []
        for cname, sname in (("kc", "ks"), ("vc", "vs")):
            t = st[cname][pages].permute(1, 0, 2, 3).reshape(hkv, -1, 9 * d)              # tiles in order
            by = t[..., :8 * d].reshape(hkv, -1, d // 2)
            sc = e4[t[..., 8 * d:].reshape(hkv, -1, d // 16).long().clamp(max=126)]
            x = torch.empty((hkv, by.shape[1], d), dtype=F64, device=DEV)
            x[..., 0::2] = signed[(by % 16).long()]
            x[..., 1::2] = signed[(by // 16).long()]
            kv.append((x.view(hkv, -1, d // 16, 16) * sc[..., None]).view(hkv, -1, d)[:, :n] * st[sname].double())
        k, v = kv
        for i in range(q):
            last = n - q + i
            lo = max(0, last - case["window"] + 1) if case["window"] else 0
            x = st["q"][at + i].double().view(hkv, hq // hkv, d)
            s = torch.einsum("hgd,hnd->hgn", x, k[:, lo:last + 1]) * st["sm"]
            l_all.append(torch.logsumexp(s, -1).reshape(hq))
            o_all.append(torch.einsum("hgn,hnd->hgd", torch.softmax(s, -1), v[:, lo:last + 1]).reshape(hq, d))
        at += q
    return dict(o=torch.stack(o_all), lse=torch.stack(l_all))


def _logprobs_exact(st):
    case = st["case"]
    k = case["k"]
    lp, ent, ids, tops = [], [], [], []
    for i in range(0, case["rows"], 32):
        x = st["logits"][i:i + 32].double()
        lse = torch.logsumexp(x, 1, keepdim=True)
        logp = x - lse
        lp.append(logp.gather(1, st["targets"][i:i + 32].long()[:, None])[:, 0])
        pr = torch.exp(logp)
        ent.append(-torch.where(pr > 0, pr * logp, torch.zeros_like(pr)).sum(1))
        val, idx = torch.sort(x, dim=1, descending=True, stable=True)
        ids.append(idx[:, :k])
        tops.append(val[:, :k] - lse)
    return dict(logprobs=torch.cat(lp), entropy=torch.cat(ent), top_ids=torch.cat(ids), top_logprobs=torch.cat(tops))
