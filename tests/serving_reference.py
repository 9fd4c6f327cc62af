"""Plain numpy references, in 64 bits, of the serving-step operators: the
paging plan, the 4-bit KV cache and token log probabilities.  Written from
the definitions in include/fp8bs.h, one request, group or row at a time;
where a definition has an fp32 rounding, it is made with numpy's float32."""
import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1_SIGNED = np.concatenate([E2M1, -E2M1])


def e4m3_values():
    """The values of the codes 0 .. 126 (the non-negative finite ones)."""
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return np.array(v[:127])


E4M3 = e4m3_values()


def nearest(a, values):
    """Index of the nearest of the ascending values, halfway to the even
    index, saturating at the last."""
    a = np.asarray(a, dtype=np.float64)
    hi = np.clip(np.searchsorted(values, a), 1, len(values) - 1)
    up, down = values[hi] - a, a - values[hi - 1]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def bf16_to_f64(bits):
    return (np.asarray(bits, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def f32_to_bf16_bits(v):
    """Nearest-even bf16 bits of finite float32 values."""
    u = np.asarray(v, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


# -------------------------------------------------------------- 4-bit cache
def encode(x_bits, s):
    """bf16 bits [..., D] -> codes [..., D], scale codes [..., D / 16]."""
    x = bf16_to_f64(x_bits).astype(np.float32)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    s = np.float32(s)
    with np.errstate(over="ignore", divide="ignore", invalid="ignore", under="ignore"):
        sc = nearest((np.abs(g).max(-1) / (np.float32(6) * s)).astype(np.float32), E4M3)
        den = (s * E4M3[sc].astype(np.float32)).astype(np.float32)[..., None]
        q = np.where(den > 0, g / np.where(den > 0, den, np.float32(1)), np.float32(0)).astype(np.float32)
    mag = nearest(np.abs(q), E2M1)
    codes = np.where(den > 0, mag + 8 * np.signbit(q), 0)
    return codes.reshape(x.shape).astype(np.uint8), sc.astype(np.uint8)


def split(cache):
    """Views of a cache: code bytes [nb, hkv, tiles, 16, D / 2], scales [.., 16, D / 16]."""
    nb, hkv, tiles, nbytes = cache.shape
    d = nbytes // 9
    return (cache[..., :8 * d].reshape(nb, hkv, tiles, 16, d // 2),
            cache[..., 8 * d:].reshape(nb, hkv, tiles, 16, d // 16))


def append(x_bits, slots, s, cache):
    """A copy of the cache with the tokens stored at their slots."""
    out = cache.copy()
    nb, hkv, tiles, nbytes = out.shape
    d, page = nbytes // 9, tiles * 16
    codes, sc = encode(x_bits, s)
    for t, slot in enumerate(slots):
        if not 0 <= slot < nb * page:
            continue
        blk, off = divmod(int(slot), page)
        tile, r = divmod(off, 16)
        for h in range(hkv):
            c = codes[t, h]
            out[blk, h, tile, r * (d // 2):(r + 1) * (d // 2)] = c[0::2] | (c[1::2] << 4)
            out[blk, h, tile, 8 * d + r * (d // 16):8 * d + (r + 1) * (d // 16)] = sc[t, h]
    return out


def decode(cache):
    """code * scale of every token, [slots, hkv, D] float64 (NaN where a scale is NaN)."""
    nb, hkv, tiles, nbytes = cache.shape
    d = nbytes // 9
    by = cache[..., :8 * d].reshape(nb, hkv, tiles * 16, d // 2)
    sc = cache[..., 8 * d:].reshape(nb, hkv, tiles * 16, d // 16)
    table = np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]])
    x = np.empty((nb, hkv, tiles * 16, d))
    x[..., 0::2], x[..., 1::2] = E2M1_SIGNED[by & 15], E2M1_SIGNED[by >> 4]
    x = x.reshape(nb, hkv, tiles * 16, d // 16, 16) * table[sc][..., None]
    return x.reshape(nb, hkv, tiles * 16, d).transpose(0, 2, 1, 3).reshape(-1, hkv, d)


def gather_bits(cache, slots, s):
    """bf16 bits [T, hkv, D] of the cached tokens."""
    x = decode(cache)
    ok = (slots >= 0) & (slots < len(x))
    v = (x[np.where(ok, slots, 0)].astype(np.float32) * np.float32(s)).astype(np.float32)
    return np.where(ok[:, None, None], f32_to_bf16_bits(v), 0).astype(np.uint16)


def attention(q_bits, cu, kc, vc, ks, vs, table, lens, sm, window=0):
    """float64 o [T, Hq, D], lse [T, Hq], and the largest sum_d |q k| sm of each
    row (what the rounding of its scores scales with)."""
    q = bf16_to_f64(q_bits)
    t, hq, d = q.shape
    nb, hkv, tiles, _ = kc.shape
    page = tiles * 16
    k, v = decode(kc) * float(np.float32(ks)), decode(vc) * float(np.float32(vs))
    o, lse, mag = np.zeros((t, hq, d)), np.full((t, hq), -np.inf), np.zeros((t, hq))
    for b, n in enumerate(lens):
        rows = range(cu[b], cu[b + 1])
        for i, row in enumerate(rows):
            p = n - len(rows) + i
            lo = max(0, p - window + 1) if window else 0
            pos = np.arange(lo, p + 1)
            blk = table[b, pos // page] if len(pos) else pos
            ok = (blk >= 0) & (blk < nb)
            idx = (blk * page + pos % page)[ok]
            if not len(idx):
                continue
            for h in range(hq):
                g = h // (hq // hkv)
                s = sm * (k[idx, g] @ q[row, h])
                m = s.max()
                e = np.exp(s - m)
                o[row, h] = (e / e.sum()) @ v[idx, g]
                lse[row, h] = m + math.log(e.sum())
                mag[row, h] = abs(sm) * (np.abs(k[idx, g]) @ np.abs(q[row, h])).max()
    return o, lse, mag


def lse_bound(lse, mag, d):
    """fp32 scores: d products summed with at most one truncation (2^-23) a
    step and three roundings of the scale; exp2 and log within 2^-21 of the
    sum; one rounding of the result."""
    return (d + 8) * 2.0 ** -23 * mag + 2.0 ** -20 + 2.0 ** -22 * np.where(np.isfinite(lse), np.abs(lse), 0)


# -------------------------------------------------------------- paging plan
def plan(ctx, new, table, free, head, page, num_blocks, num_tokens):
    """dict of the plan's arrays, one request after the other, and the error bits."""
    table = np.array(table, dtype=np.int64)
    cap, err = table.shape[1] * page, 0
    head_ok = 0 <= head <= len(free)
    if not head_ok:
        err |= 16
    seq, cu, asked, taken = [], [0], 0, 0
    slots, pos, req = (np.full(num_tokens, -1, dtype=np.int64) for _ in range(3))
    for b, (c, n) in enumerate(zip(ctx, new)):
        at = cu[-1]
        cu.append(at + max(n, 0))
        req[at:cu[-1]] = b
        good = c >= 0 and n >= 0 and c + n <= cap and cu[-1] <= num_tokens
        if not good:
            err |= 16
            seq.append(min(max(c, 0), cap))
            continue
        have = -(-c // page)
        need = -(-(c + n) // page) - have
        mine, asked = asked, asked + need
        if need and not (head_ok and head + asked <= len(free)):
            err |= 32
            seq.append(c)
            continue
        taken = asked if need else taken
        seq.append(c + n)
        for i in range(need):
            f = free[head + mine + i]
            table[b, have + i] = f if 0 <= f < num_blocks else -1
        for i in range(n):
            pos[at + i] = c + i
            blk = table[b, (c + i) // page]
            if 0 <= blk < num_blocks:
                slots[at + i] = blk * page + (c + i) % page
            else:
                err |= 16
    return dict(seq_lens=np.array(seq, dtype=np.int64), cu_new=np.minimum(cu, 2 ** 31 - 1), slots=slots, positions=pos,
                requests=req, free_head=np.array([head + taken]), table=table), err


# -------------------------------------------------------- log probabilities
def logprobs(x, targets, top):
    """x float64 [M, V]: dict of logprobs, entropy, top_ids, top_logprobs, and
    per row |t / l| = the mean distance to the maximum."""
    m, v = x.shape
    lp, ent, dist = np.zeros(m), np.zeros(m), np.zeros(m)
    ids, tops = np.zeros((m, top), dtype=np.int64), np.zeros((m, top))
    for r in range(m):
        mx = x[r].max()
        logp = x[r].copy()                              # a row of nothing but -inf stays so
        if mx != -np.inf:
            e = np.exp(x[r] - mx)
            logp = (x[r] - mx) - math.log(e.sum())      # not x - lse: lse would lose the log beside a large mx
            p = e / e.sum()
            ent[r] = -np.sum(p[p > 0] * logp[p > 0])
            dist[r] = np.sum(p[p > 0] * (mx - x[r][p > 0]))
        lp[r] = logp[targets[r]] if 0 <= targets[r] < v else 0.0
        order = np.lexsort((np.arange(v), -x[r]))[:top]
        ids[r], tops[r] = order, logp[order]
    return dict(logprobs=lp, entropy=ent, top_ids=ids, top_logprobs=tops), dist
