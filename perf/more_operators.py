"""Performance cases of what a step does between its linears and its attention:
the norm and rotation of queries and keys on their way into a paged cache
(kv4_rope_append, kv_rope_append), the routing to experts and the weighted sum
of their outputs (moe_route, moe_combine), and the choice of the next token
(sample_tokens).

Every case runs in two forms on the same inputs: the plain form, elementary
torch operations in 32 bits (64 where 32 lose what matters), and, with
``own`` set, the calls a user makes of this package.  ``exact`` gives the
same outputs from the definitions in 64 bits, written apart from both.

rope: a head vector a (bf16), with norm weights w: r = 1 / sqrt(mean a^2 + eps)
rounded once, n = (a r) w; the pair (n1, n2) of a position's (cos, sin):
(n1 cos - n2 sin, n2 cos + n1 sin); every product, sum and difference one fp32
rounding.  q is then bf16, k and v go to the cache: e4m3(x / scale), or e2m1
codes with an e4m3 scale per 16 elements.
route: scores s = softmax(x) or sigmoid(x); with a bias the experts are chosen by
s + bias in multiples of 2^-44, without by x; groups by the sum of their best
one or two scores, in the same multiples; weights are the chosen s.
sample: w = exp((x - max) / T); of the order by value, then index, the first
tokens that top-k, top-p (of the top-k's mass) and min-p all keep; the first
random number picks a block of 1024 token ids by the kept mass, the second the
token in it.
"""
import math

import torch

own = False

DEV = "cuda"
F32, F64, BF16, I32, I64, U8 = torch.float32, torch.float64, torch.bfloat16, torch.int32, torch.int64, torch.uint8
E4M3 = torch.float8_e4m3fn
EPS = 1e-6
BLOCK = 1024                                                    # token ids that the first random number tells apart
UNIT = 2.0 ** 44                                                # of biased scores


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 64 requests, 4-bit cache: latency
        dict(name="rope4-decode-64", op="rope", bits=4, tokens=64, hq=32, hkv=8, d=128, page=16, rot=128, norm=True,
             pairs=False),
        # a prompt chunk into the 4-bit cache, read back for a dense prompt attention
        dict(name="rope4-prompt-8191", op="rope", bits=4, tokens=8191, hq=32, hkv=8, d=128, page=64, rot=128, norm=True,
             pairs=False),
        # one request's next token, FP8 cache: the smallest call
        dict(name="rope8-decode-1", op="rope", bits=8, tokens=1, hq=32, hkv=8, d=128, page=16, rot=128, norm=True,
             pairs=False),
        # a prompt chunk into the FP8 cache: half of each head rotated in adjacent pairs, no norm
        dict(name="rope8-prompt-4099", op="rope", bits=8, tokens=4099, hq=64, hkv=8, d=128, page=32, rot=64, norm=False,
             pairs=True),
        # the router of a decode step: the top 12 of 256 by softmax
        dict(name="route-decode-32x256", op="route", tokens=32, experts=256, topk=12, scoring="softmax", bias=False,
             groups=1, topk_groups=1, group_top=1, dtype="f32"),
        # the router of a prompt: sigmoid scores, a bias for balance, the best 4 of 8 groups
        dict(name="route-prompt-8192x256", op="route", tokens=8192, experts=256, topk=8, scoring="sigmoid", bias=True,
             groups=8, topk_groups=4, group_top=2, dtype="f32"),
        # the experts' outputs of a decode step, added to the residual stream
        dict(name="combine-decode-32", op="combine", tokens=32, topk=12, n=4096, residual=True, dropped=False),
        # the same of a prompt
        dict(name="combine-prompt-2048", op="combine", tokens=2048, topk=12, n=4096, residual=True, dropped=False),
        # one sequence's next token: latency over a long row
        dict(name="sample-1x152064", op="sample", rows=1, vocab=152064, kind="top_p", dtype="bf16", pad=0, masked=False),
        # a decode batch whose requests each bring their own settings
        dict(name="sample-64x152064", op="sample", rows=64, vocab=152064, kind="mixed", dtype="bf16", pad=0,
             masked=False),
        # many short fp32 rows of an odd length
        dict(name="sample-256x32003", op="sample", rows=256, vocab=32003, kind="mixed", dtype="f32", pad=0,
             masked=False),
        # rollouts: many sequences, temperature only
        dict(name="sample-512x152064", op="sample", rows=512, vocab=152064, kind="temperature", dtype="bf16", pad=0,
             masked=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "route", "route", "combine", "sample", "sample", "sample"])
    if op == "rope":
        bits = rng.choice([4, 8])
        hkv = rng.choice([1, 2, 4, 8])
        d = rng.choice([64, 128]) if bits == 4 else 128
        return dict(op=op, bits=bits, tokens=_log(rng, 1, 8191), hq=hkv * rng.choice([1, 2, 3, 4]), hkv=hkv, d=d,
                    page=rng.choice([16, 32, 48, 64, 128, 256]), rot=rng.choice([16, 32, 64, d]), norm=rng.random() < 0.6,
                    pairs=rng.random() < 0.3)
    if op == "route":
        groups, topk_groups, group_top = rng.choice([(1, 1, 1), (1, 1, 1), (4, 2, 1), (8, 4, 2), (8, 3, 2)])
        experts = groups * _log(rng, 4, 512 // groups)
        most = min(16, experts * topk_groups // groups)
        return dict(op=op, tokens=_log(rng, 1, 8192), experts=experts, topk=rng.randint(1, most),
                    scoring=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                    topk_groups=topk_groups, group_top=group_top, dtype=rng.choice(["f32", "f32", "bf16"]))
    if op == "combine":
        return dict(op=op, tokens=_log(rng, 1, 2048), topk=rng.randint(1, 12), n=8 * _log(rng, 8, 512),
                    residual=rng.random() < 0.6, dropped=rng.random() < 0.3)
    while True:
        case = dict(op=op, rows=_log(rng, 1, 512), vocab=_log(rng, 1000, 152064),
                    kind=rng.choice(["temperature", "top_p", "top_k", "mixed", "mixed"]),
                    dtype=rng.choice(["bf16", "f32"]), pad=rng.choice([0, 0, 1, 8, 64]), masked=rng.random() < 0.2)
        if work(case)["bytes"] <= work(listed()[-1])["bytes"] and (case["kind"] == "temperature" or case["rows"] <= 256):
            return case


def work(case):
    """Bytes and operations a pass cannot do without: inputs read once, outputs written once."""
    op = case["op"]
    t = case.get("tokens")
    if op == "rope":
        row = (case["hq"] + 2 * case["hkv"]) * case["d"]
        kv = 2 * t * case["hkv"] * case["d"]
        held = kv * 9 // 16 if case["bits"] == 4 else kv
        back = held + 2 * kv if case["bits"] == 4 else 0          # the 4-bit cases read the cache back in bf16
        return {"bytes": 2 * t * row + 2 * t * case["hq"] * case["d"] + held + back + 4 * t * case["rot"] + 8 * t,
                "flops": t * (case["hq"] + case["hkv"]) * (3 * case["rot"] + (4 * case["d"] if case["norm"] else 0))}
    if op == "route":
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": t * (size * case["experts"] + 8 * case["topk"]), "flops": 4 * t * case["experts"]}
    if op == "combine":
        rows = case["topk"] + 1 + (1 if case["residual"] else 0)
        return {"bytes": t * (2 * case["n"] * rows + 4 * case["topk"]), "flops": 2 * t * case["topk"] * case["n"]}
    size = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": case["rows"] * (size * case["vocab"] + 8 + 8), "flops": 3 * case["rows"] * case["vocab"]}


# --------------------------------------------------------------- preparation
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rand(g, lo, hi, n):
    return lo + (hi - lo) * torch.rand(n, generator=g, device=DEV)


def _angles(positions, rot):
    """cos and sin of the rotated pairs [positions, rot], the angles in 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=F64) / rot)
    a = torch.arange(positions, device=DEV, dtype=F64)[:, None] * freq
    return torch.cat((torch.cos(a), torch.sin(a)), 1).to(F32)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case=case)
    t = case.get("tokens")
    if op == "rope":
        hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
        qkv = torch.randn((t, (hq + 2 * hkv) * d), generator=g, device=DEV).to(BF16)  # the fused projection's rows
        st["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        st["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        st["v"] = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        most = 32768
        if t <= 64:                                             # decode: every request at a place of its own
            st["pos"] = torch.randint(0, most, (t,), generator=g, device=DEV).to(I32)
        else:                                                   # a prompt chunk
            first = int(torch.randint(0, most - t, (1,), generator=g, device=DEV))
            st["pos"] = torch.arange(first, first + t, device=DEV).to(I32)
        st["table"] = _angles(most, case["rot"])
        nb = (t + page - 1) // page + 3
        st["slots"] = torch.randperm(nb * page, generator=g, device=DEV)[:t].to(I32)
        if case["norm"]:
            st["qw"] = (1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(BF16)
            st["kw"] = (1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(BF16)
        top = 2688.0 if case["bits"] == 4 else 448.0
        st["ks"] = torch.tensor([8.0 / top], device=DEV)
        st["vs"] = torch.tensor([6.0 / top], device=DEV)
        shape = (nb, hkv, page // 16, 9 * d) if case["bits"] == 4 else (nb, page, hkv, d)
        st["kc"] = torch.zeros(shape, dtype=U8, device=DEV)
        st["vc"] = torch.zeros(shape, dtype=U8, device=DEV)
        return st
    if op == "route":
        x = torch.randn((t, case["experts"]), generator=g, device=DEV) * 1.5
        st["logits"] = x if case["dtype"] == "f32" else x.to(BF16)
        if case["bias"]:
            st["bias"] = torch.randn(case["experts"], generator=g, device=DEV) * 0.05
        return st
    if op == "combine":
        st["y"] = torch.randn((t, case["topk"], case["n"]), generator=g, device=DEV).to(BF16)
        w = torch.rand((t, case["topk"]), generator=g, device=DEV) + 0.05
        st["w"] = w / w.sum(1, keepdim=True)
        st["ids"] = torch.randint(0, 256, (t, case["topk"]), generator=g, device=DEV).to(I32)
        if case["dropped"]:                                     # slots that no expert had room for
            st["ids"][torch.rand(st["ids"].shape, generator=g, device=DEV) < 0.1] = -1
        if case["residual"]:
            st["res"] = torch.randn((t, case["n"]), generator=g, device=DEV).to(BF16)
        return st
    m, v = case["rows"], case["vocab"]
    full = torch.randn((m, v + case["pad"]), generator=g, device=DEV).mul_(2.0)  # a model's logits: a normal bulk
    tall = torch.randint(0, v, (m, 8), generator=g, device=DEV)                  # and a few tall ones
    full.scatter_add_(1, tall, torch.rand(tall.shape, generator=g, device=DEV) * 12)
    full = full.to(BF16 if case["dtype"] == "bf16" else F32)
    st["logits"] = full[:, :v]
    if case["masked"]:                                          # constrained decoding: most of the vocabulary is shut
        open_ = torch.rand((m, v), generator=g, device=DEV) < max(0.05, 64.0 / v)
        open_[:, :40] = True
        st["logits"].masked_fill_(~open_, -math.inf)
    st["u"] = torch.rand((m, 2), generator=g, device=DEV)
    kind = case["kind"]
    st["temperature"] = _rand(g, 0.5, 1.3, m)
    if kind in ("top_p", "mixed"):
        st["top_p"] = _rand(g, 0.8, 0.98, m)
    if kind in ("top_k", "mixed"):
        st["top_k"] = torch.randint(1, 201, (m,), generator=g, device=DEV).to(I32)
    if kind == "mixed":                                         # each setting off for some rows; some are greedy
        pick = torch.rand((3, m), generator=g, device=DEV)
        st["top_p"] = torch.where(pick[0] < 0.4, torch.ones_like(st["top_p"]), st["top_p"])
        st["top_k"] = torch.where(pick[1] < 0.4, torch.zeros_like(st["top_k"]), st["top_k"])
        st["min_p"] = torch.where(pick[2] < 0.6, torch.zeros_like(st["u"][:, 0]), _rand(g, 0.02, 0.1, m))
        st["temperature"] = torch.where(pick[2] > 0.9, torch.zeros_like(st["temperature"]), st["temperature"])
    return st


# ----------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    import fp8_block_scaled_02_gb300 as fp8bs
    case = st["case"]
    op = case["op"]
    if op == "rope":
        append = fp8bs.kv4_rope_append if case["bits"] == 4 else fp8bs.kv_rope_append
        q = append(st["q"], st["k"], st["v"], st["pos"], st["slots"], st["table"], st["ks"], st["vs"], st["kc"], st["vc"],
                   q_norm=st.get("qw"), k_norm=st.get("kw"), eps=EPS, interleaved=case["pairs"])
        if case["bits"] == 8:
            return dict(q=q, k=st["kc"].view(E4M3), v=st["vc"].view(E4M3))
        k, v = fp8bs.kv4_gather(st["kc"], st["vc"], st["slots"], st["ks"], st["vs"])
        return dict(q=q, k=k, v=v)
    if op == "route":
        ids, weights = fp8bs.moe_route(st["logits"], case["topk"], scoring=case["scoring"], bias=st.get("bias"),
                                       groups=case["groups"], topk_groups=case["topk_groups"],
                                       group_top=case["group_top"], renormalize=True, scale=1.0)
        return dict(ids=ids, weights=weights)
    if op == "combine":
        return dict(out=fp8bs.moe_combine(st["y"], st["w"], ids=st["ids"], num_experts=256, residual=st.get("res")))
    r = fp8bs.sample_tokens(st["logits"], st["u"], st["temperature"], top_k=st.get("top_k"), top_p=st.get("top_p"),
                            min_p=st.get("min_p"))
    return dict(tokens=r.tokens, logprobs=r.logprobs)


def _run_plain(st):
    return dict(rope=_rope_plain, route=_route_plain, combine=_combine_plain, sample=_sample_plain)[st["case"]["op"]](st)


MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)          # e2m1


def _turn(x, w, cos, sin, rot, pairs):
    """The head vectors x [T, H, D] normed (w) and rotated, in fp32."""
    x = x.to(F32)
    if w is not None:
        ms = x.to(F64).square().mean(-1, keepdim=True)
        x = (x * (ms + torch.tensor(EPS, dtype=F32).to(F64).item()).rsqrt().to(F32)) * w.to(F32)
    y = x[..., :rot]
    a, b = (y[..., 0::2], y[..., 1::2]) if pairs else (y[..., :rot // 2], y[..., rot // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((a, b), -1).flatten(-2) if pairs else torch.cat((a, b), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _encode4(x, s):
    """fp32 x [..., D] -> e2m1 codes (0..15) and e4m3 scale bytes [..., D / 16]."""
    g = x.unflatten(-1, (-1, 16))
    sc = (g.abs().amax(-1) / (s * 6.0)).clamp(max=448.0).to(E4M3)
    den = (sc.to(F32) * s).unsqueeze(-1)
    q = torch.where(den > 0, g / den, torch.zeros_like(g))
    a = q.abs()
    mag = ((a > 0.25).to(U8) + (a >= 0.75).to(U8) + (a > 1.25).to(U8) + (a >= 1.75).to(U8) + (a > 2.5).to(U8)
           + (a >= 3.5).to(U8) + (a > 5.0).to(U8))              # halfway goes to the even code
    return (mag + 8 * (q < 0).to(U8)).flatten(-2), sc.view(U8)


def _rope_plain(st):
    case = st["case"]
    rot, d, page = case["rot"], case["d"], case["page"]
    turn = st["table"][st["pos"].long()][:, None]
    cos, sin = turn[..., :rot // 2], turn[..., rot // 2:]
    q = _turn(st["q"], st.get("qw"), cos, sin, rot, case["pairs"]).to(BF16)
    k = _turn(st["k"], st.get("kw"), cos, sin, rot, case["pairs"])
    v = st["v"].to(F32)
    slots = st["slots"].long()
    if case["bits"] == 8:
        for x, s, c in ((k, st["ks"], st["kc"]), (v, st["vs"], st["vc"])):
            c.flatten(0, 1)[slots] = (x / s).clamp(-448.0, 448.0).to(E4M3).view(U8)
        return dict(q=q, k=st["kc"].view(E4M3), v=st["vc"].view(E4M3))
    blk, tile, row = slots // page, slots % page // 16, slots % 16
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), dtype=F32, device=DEV)
    out = dict(q=q)
    for name, x, s, c in (("k", k, st["ks"], st["kc"]), ("v", v, st["vs"], st["vc"])):
        code, sc = _encode4(x, s)
        cv, sv = c[..., :8 * d].unflatten(-1, (16, d // 2)), c[..., 8 * d:].unflatten(-1, (16, d // 16))
        cv[blk, :, tile, row] = code[..., 0::2] | (code[..., 1::2] << 4)
        sv[blk, :, tile, row] = sc
        b = cv[blk, :, tile, row]
        code = torch.stack((b & 15, b >> 4), -1).flatten(-2)
        sc = sv[blk, :, tile, row].view(E4M3).to(F32).unsqueeze(-1)
        out[name] = ((table[code.long()].unflatten(-1, (-1, 16)) * sc) * s).flatten(-2).to(BF16)
    return out


def _route_plain(st):
    case = st["case"]
    x = st["logits"].to(F64)
    if case["scoring"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True))
        s = e / e.sum(1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-x))
    c = torch.round((s + st["bias"].to(F64) if case["bias"] else s) * UNIT)
    choice = c if case["bias"] else x
    g = case["groups"]
    if g > 1:
        score = torch.topk(c.unflatten(1, (g, -1)), case["group_top"], dim=2).values.sum(2)
        order = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        live = torch.zeros_like(score, dtype=torch.bool).scatter_(1, order, True)
        choice = choice.masked_fill(~live.repeat_interleave(case["experts"] // g, 1), -math.inf)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :case["topk"]]
    w = s.gather(1, ids)
    return dict(ids=ids.to(I32), weights=(w / w.sum(1, keepdim=True)).to(F32))


def _combine_plain(st):
    w = torch.where(st["ids"] >= 0, st["w"], torch.zeros_like(st["w"]))
    out = (w[:, :, None] * st["y"].to(F32)).sum(1)
    return dict(out=(out + st["res"].to(F32) if st["case"]["residual"] else out).to(BF16))


def _sample_plain(st):
    case = st["case"]
    v = case["vocab"]
    x = st["logits"].to(F32) + 0.0
    t = st["temperature"].to(F64)[:, None]
    greedy = t == 0
    w = torch.exp((x.to(F64) - x.amax(1, keepdim=True).to(F64)) / torch.where(greedy, torch.ones_like(t), t))
    ids = torch.arange(v, device=DEV)
    if "top_k" in st or "top_p" in st:
        bits = x.view(I32)                                      # an order of integers: the value, then the lowest index
        key = torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF).to(I64) * (1 << 32) + (v - 1 - ids)
        order = v - 1 - (torch.sort(key, dim=1, descending=True).values & 0xFFFFFFFF)
        ws = w.gather(1, order)
        keep = (ids == 0) | ~greedy
        if "top_k" in st:
            k = st["top_k"][:, None]
            keep = keep & ((ids < k) | (k <= 0))
        if "min_p" in st:
            keep = keep & (ws >= st["min_p"].to(F64)[:, None])
        if "top_p" in st:
            p = st["top_p"].to(F64)[:, None]
            of_k = torch.where((ids < k) | (k <= 0), ws, torch.zeros_like(ws)) if "top_k" in st else ws
            upto = torch.cumsum(of_k, 1)
            before = torch.cat((torch.zeros_like(upto[:, :1]), upto[:, :-1]), 1)
            keep = keep & ((p >= 1) | (before < p * upto[:, -1:]) | (ids == 0))
        w = torch.where(torch.zeros_like(keep).scatter_(1, order, keep), w, torch.zeros_like(w))
    blocks = torch.nn.functional.pad(w, (0, -v % BLOCK)).unflatten(1, (-1, BLOCK))
    upto = torch.cumsum(blocks.sum(2), 1)
    u = st["u"].to(F64)
    b = (upto <= u[:, :1] * upto[:, -1:]).sum(1)
    inside = torch.cumsum(blocks[torch.arange(len(b), device=DEV), b], 1)
    token = b * BLOCK + (inside <= u[:, 1:] * inside[:, -1:]).sum(1)
    logp = torch.log(w.gather(1, token[:, None]) / upto[:, -1:])[:, 0]
    return dict(tokens=token.to(I32), logprobs=logp.to(F32))


# ------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return dict(rope=_rope_exact, route=_route_exact, combine=_combine_exact, sample=_sample_exact)[case["op"]](st)


def _once(x):
    """x rounded to fp32, held in 64 bits."""
    return x.to(F32).to(F64)


def _e4m3_values():
    """The 127 non-negative finite e4m3 values in the order of their codes."""
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:127], dtype=F64, device=DEV)


def _nearest(a, values):
    """The nearest of the ascending values; halfway takes the even index."""
    hi = torch.searchsorted(values, a.contiguous()).clamp(1, len(values) - 1)
    lo = hi - 1
    up, down = values[hi] - a, a - values[lo]
    return values[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)]


def _rope_exact(st):
    """q without any rounding; what k's and v's places in the cache hold, by the roundings that the format defines."""
    case = st["case"]
    d, rot, hkv = case["d"], case["rot"], case["hkv"]
    half = rot // 2
    at = torch.arange(rot, device=DEV)
    first, second = (at[0::2], at[1::2]) if case["pairs"] else (at[:half], at[half:])
    ang = st["table"].index_select(0, st["pos"]).to(F64)
    c, s = ang[:, None, :half], ang[:, None, half:]

    def turned(x, w, rnd):
        x = x.to(F64)
        if w is not None:
            r = rnd(1.0 / torch.sqrt((x * x).sum(-1, keepdim=True) / d + float(torch.tensor(EPS, dtype=F32))))
            x = rnd(rnd(x * r) * w.to(F64))
        o = x.clone()
        o[..., first] = rnd(rnd(x[..., first] * c) - rnd(x[..., second] * s))
        o[..., second] = rnd(rnd(x[..., second] * c) + rnd(x[..., first] * s))
        return o

    res = dict(q=turned(st["q"], st.get("qw"), lambda z: z))
    e4 = _e4m3_values()
    e2 = torch.tensor(MAGNITUDES, dtype=F64, device=DEV)
    for name, x, sc in (("k", turned(st["k"], st.get("kw"), _once), st["ks"].to(F64)),
                        ("v", st["v"].to(F64), st["vs"].to(F64))):
        if case["bits"] == 8:
            z = _once(x / sc)
            held = torch.zeros((st["kc"].shape[0] * case["page"], hkv, d), dtype=F64, device=DEV)
            held[st["slots"].long()] = torch.sign(z) * _nearest(z.abs(), e4)
            res[name] = held.view(st["kc"].shape)
            continue
        g = x.reshape(*x.shape[:-1], -1, 16)
        scale = _nearest(_once(g.abs().amax(-1) / _once(6.0 * sc)), e4)
        den = _once(scale * sc)[..., None]
        z = _once(g / torch.where(den > 0, den, torch.ones_like(den)))
        val = torch.where(den > 0, torch.sign(z) * _nearest(z.abs(), e2), torch.zeros_like(z))
        res[name] = (val * scale[..., None] * sc).flatten(-2)
    return res


def _route_exact(st):
    case = st["case"]
    t, e, g = case["tokens"], case["experts"], case["groups"]
    x = st["logits"].to(F64)
    s = torch.softmax(x, 1) if case["scoring"] == "softmax" else torch.sigmoid(x)
    c = torch.round((s + (st["bias"].to(F64) if case["bias"] else 0.0)) * UNIT)
    live = torch.ones((t, e), dtype=torch.bool, device=DEV)
    if g > 1:
        best = torch.sort(c.view(t, g, e // g), dim=2, descending=True).values[..., :case["group_top"]].sum(2)
        i = torch.arange(g, device=DEV)
        ahead = (best[:, None, :] > best[:, :, None]) | ((best[:, None, :] == best[:, :, None]) & (i[None, :] < i[:, None]))
        live = (ahead.sum(2) < case["topk_groups"]).repeat_interleave(e // g, 1)
    choice = torch.where(live, c if case["bias"] else x, torch.full_like(x, -math.inf))
    picked = []
    for _ in range(case["topk"]):                               # the best that is left, the lowest of equals
        top = (choice == choice.amax(1, keepdim=True)).to(I32).argmax(1, keepdim=True)
        picked.append(top)
        choice = choice.scatter(1, top, -math.inf)
    ids = torch.cat(picked, 1)
    w = s.gather(1, ids)
    return dict(ids=ids, weights=w / w.sum(1, keepdim=True))


def _combine_exact(st):
    w = st["w"].to(F64) * (st["ids"] >= 0)
    out = torch.einsum("tj,tjn->tn", w, st["y"].to(F64))
    return dict(out=out + st["res"].to(F64) if st["case"]["residual"] else out)


def _sample_exact(st):
    case = st["case"]
    m, v = case["rows"], case["vocab"]
    tokens, logps = [], []
    for r in range(m):
        x = st["logits"][r].to(F64)
        t = float(st["temperature"][r])
        val, idx = torch.sort(x, descending=True, stable=True)
        w = torch.exp((val - val[0]) / t) if t > 0 else torch.ones_like(val)
        n = v if t > 0 else 1
        k = int(st["top_k"][r]) if "top_k" in st else 0
        if k > 0:
            n = min(n, k)
        allowed = n
        if "top_p" in st and float(st["top_p"][r]) < 1 and n > 1:
            upto = torch.cumsum(w[:n], 0)
            allowed = min(allowed, int((upto < float(st["top_p"][r]) * upto[-1]).sum()) + 1)
        if "min_p" in st and t > 0:
            allowed = max(1, min(allowed, int((w >= float(st["min_p"][r])).sum())))
        kept = torch.zeros(-(-v // BLOCK) * BLOCK, dtype=F64, device=DEV)
        kept[idx[:allowed]] = w[:allowed]
        kept = kept.view(-1, BLOCK)
        mass = kept.sum(1)
        b = int(torch.searchsorted(torch.cumsum(mass, 0), mass.sum() * float(st["u"][r, 0]), right=True))
        i = int(torch.searchsorted(torch.cumsum(kept[b], 0), mass[b] * float(st["u"][r, 1]), right=True))
        tokens.append(b * BLOCK + i)
        logps.append(torch.log(kept[b, i] / mass.sum()))
    return dict(tokens=torch.tensor(tokens, dtype=I64), logprobs=torch.stack(logps))
