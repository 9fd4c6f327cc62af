"""Plain numpy references, in 64 bits, of what a step does between its linears
and its attention: norm and rotation into a paged cache, routing to experts
and the weighted sum of their outputs, sampling.  Written from the definitions
in include/fp8bs.h, one head, token or row at a time; where a definition has an
fp32 rounding, it is made with numpy's float32."""
import math

import numpy as np

import serving_reference as serving
from serving_reference import E4M3, bf16_to_f64, nearest

F32 = np.float32


# -------------------------------------------------- norm and rotation, caches
def turned(x_bits, w_bits, eps, cos, sin, interleaved, rounded=True):
    """bf16 bits [T, H, D], norm weights' bits [D] or None, cos and sin [T, R / 2] fp32 -> [T, H, D] float64:
    every step rounded to fp32 as defined, or none."""
    rnd = (lambda v: v.astype(F32).astype(np.float64)) if rounded else (lambda v: v)
    x = bf16_to_f64(x_bits)
    if w_bits is not None:
        with np.errstate(divide="ignore", invalid="ignore"):
            r = rnd(1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(F32(eps))))
            x = rnd(rnd(x * r) * bf16_to_f64(w_bits))
    half = cos.shape[1]
    a, b = (np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved else (np.arange(half), np.arange(half) + half)
    c, s = cos.astype(np.float64)[:, None], sin.astype(np.float64)[:, None]
    out = x.copy()
    out[..., a] = rnd(rnd(x[..., a] * c) - rnd(x[..., b] * s))
    out[..., b] = rnd(rnd(x[..., b] * c) + rnd(x[..., a] * s))
    return out


def e4m3_codes(v):
    """float32 -> e4m3 bytes, nearest even, saturating, the sign kept, NaN 0x7F."""
    v = np.asarray(v, dtype=F32)
    nan = np.isnan(v)
    mag = nearest(np.minimum(np.abs(np.where(nan, 0, v)).astype(np.float64), 448.0), E4M3)
    return np.where(nan, 0x7F, mag + 128 * np.signbit(v)).astype(np.uint8)


def store8(x, slots, s, cache):
    """A copy of the FP8 cache [nb, page, H, D] with x [T, H, D] (fp32 values) stored at the slots."""
    out = cache.copy()
    flat = out.reshape(-1, *cache.shape[2:])
    with np.errstate(over="ignore", invalid="ignore"):
        codes = e4m3_codes(x.astype(F32) / F32(s))
    for t, slot in enumerate(slots):
        if 0 <= slot < len(flat):
            flat[slot] = codes[t]
    return out


def store4(x, slots, s, cache):
    """A copy of the 4-bit cache with x [T, H, D] (fp32 values) stored at the slots."""
    out = cache.copy()
    codes_of, scales_of = serving.split(out)
    d, page = x.shape[-1], cache.shape[2] * 16
    g = x.astype(F32).reshape(*x.shape[:-1], d // 16, 16)
    with np.errstate(all="ignore"):
        amax = np.abs(g).max(-1)                               # NaN if there is one
        quot = (amax / (F32(6) * F32(s))).astype(F32)
        sc = np.where(np.isnan(quot), 0x7F, nearest(np.minimum(np.where(np.isnan(quot), 0, quot), 448), E4M3))
        den = (F32(s) * np.where(sc == 0x7F, np.nan, E4M3[np.minimum(sc, 126)]).astype(F32)).astype(F32)[..., None]
        ok = den > 0
        q = np.where(ok, g / np.where(ok, den, F32(1)), F32(0)).astype(F32)
        mag = nearest(np.minimum(np.abs(np.where(np.isnan(q), 0, q)), 6), serving.E2M1)
    codes = np.where(ok, mag + 8 * np.signbit(q), 0).reshape(x.shape).astype(np.uint8)
    for t, slot in enumerate(slots):
        if 0 <= slot < cache.shape[0] * page:
            blk, off = divmod(int(slot), page)
            codes_of[blk, :, off // 16, off % 16] = codes[t][:, 0::2] | (codes[t][:, 1::2] << 4)
            scales_of[blk, :, off // 16, off % 16] = sc[t].astype(np.uint8)
    return out


# ------------------------------------------------------------------- routing
UNIT = 2.0 ** 44


def route(x, topk, scoring, bias=None, groups=1, topk_groups=1, group_top=1, renormalize=True, scale=1.0):
    """x [M, E] float64 -> ids [M, topk], weights [M, topk] float64."""
    m, e = x.shape
    ids, weights = np.zeros((m, topk), dtype=np.int64), np.zeros((m, topk))
    for t in range(m):
        if scoring == "softmax":
            with np.errstate(invalid="ignore"):
                top = np.max(x[t])                              # NaN if there is one
                s = np.exp(x[t] - top) if top != -math.inf else np.zeros(e)
                s = s / s.sum() if s.sum() != 0 else s
        else:
            with np.errstate(over="ignore"):
                s = 1.0 / (1.0 + np.exp(-x[t]))
        b = 0.0 if bias is None else np.clip(np.asarray(bias, dtype=np.float64), -65536, 65536)
        c = np.rint((s + b) * UNIT)
        choice = c if bias is not None else x[t]
        live = list(range(e))
        if groups > 1:
            per = e // groups
            low = np.where(np.isnan(c), -2.0 ** 61 + 1, c)
            best = [sum(sorted(low[g * per:(g + 1) * per])[::-1][:group_top]) for g in range(groups)]
            chosen = sorted(range(groups), key=lambda g: (-best[g], g))[:topk_groups]
            live = [i for i in range(e) if i // per in chosen]
        picked = sorted(live, key=lambda i: (1, 0, i) if np.isnan(choice[i]) else (0, -choice[i], i))[:topk]
        w = s[picked]
        if renormalize:
            w = w / w.sum() if w.sum() != 0 else np.zeros(topk)
        ids[t], weights[t] = picked, w * scale
    return ids, weights


def combine(y, w, ids=None, num_experts=0, residual=None):
    """float64 y [M, K, N], w [M, K] -> [M, N]; slots without an expert add nothing."""
    out = np.zeros((y.shape[0], y.shape[2])) if residual is None else residual.astype(np.float64).copy()
    for t in range(y.shape[0]):
        for j in range(y.shape[1]):
            if ids is None or 0 <= ids[t, j] < num_experts:
                out[t] += w[t, j] * y[t, j]
    return out


# ------------------------------------------------------------------ sampling
BLOCK = 1024


def kept_tokens(x, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The kept tokens of a row (float64), best first, and the weights of all."""
    order = np.lexsort((np.arange(len(x)), -x))
    top = x[order[0]]
    if temperature == 0:
        w = np.zeros(len(x))
        w[order[0]] = 1.0
        return order[:1], w
    w = np.exp((x - top) / temperature)
    n = len(x) if top_k <= 0 else min(top_k, len(x))
    keep = n
    if top_p < 1:
        upto = np.cumsum(w[order[:n]])
        keep = min(keep, int((upto < top_p * upto[-1]).sum()) + 1)
    if min_p > 0:
        keep = min(keep, int((w[order] >= min(min_p, 1.0)).sum()))
    return order[:max(keep, 1)], w


def sample(x, u0, u1, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log probability, how near a random number came to a border of its choice) of a row: -1 for one without a
    finite largest logit or with settings that cannot be."""
    x = np.asarray(x, dtype=np.float64)
    if np.isnan(x).any() or not np.isfinite(x.max()):
        return -1, 0.0, 1.0
    if not (0 <= temperature < math.inf) or math.isnan(top_p) or math.isnan(min_p):
        return -1, 0.0, 1.0
    kept, w = kept_tokens(x, temperature, top_k, top_p, min_p)
    mass = np.zeros(-(-len(x) // BLOCK) * BLOCK)
    mass[kept] = w[kept]
    mass = mass.reshape(-1, BLOCK)
    blocks = np.cumsum(mass.sum(1))
    b = int((blocks <= u0 * blocks[-1]).sum())
    inside = np.cumsum(mass[b])
    i = int((inside <= u1 * inside[-1]).sum())
    near = min(np.abs(blocks / blocks[-1] - u0)[blocks < blocks[-1]].min(initial=1.0),
               np.abs(inside / inside[-1] - u1)[inside < inside[-1]].min(initial=1.0))
    return b * BLOCK + i, math.log(mass[b, i] / blocks[-1]), near
