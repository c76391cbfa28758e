"""Plain forms of the serving and norm operators for the tests: numpy, from the definitions, in 64 bits or, where a
contract fixes every rounding (the codes), in float32 one operation at a time.  Nothing here comes from the library."""
import math

import numpy as np

EPS32 = np.float32(1e-5)


def bf16_round(x):
    """float32 -> the nearest bfloat16 value, ties to even, as float32."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    r = (u + np.uint32(0x7FFF) + ((u >> np.uint32(16)) & np.uint32(1))) & np.uint32(0xFFFF0000)
    return r.view(np.float32)


# ------------------------------------------------------------------ plan

def plan(cached, added, free, taken, table, block, T):
    """(table, total, row_start, slots, positions, taken_out), one request after the other."""
    B, width = table.shape
    table = table.copy()
    total, row_start = np.zeros(B, np.int64), np.zeros(B + 1, np.int64)
    slots, positions = np.full(T, -1, np.int64), np.full(T, -1, np.int64)
    row, at = 0, max(int(taken), 0)
    for b in range(B):
        c, n = max(int(cached[b]), 0), max(int(added[b]), 0)
        n = min(n, 2 ** 31 - 1 - c)
        total[b] = c + n
        row_start[b] = min(row, T)
        had, want = min(-(-c // block), width), min(-(-(c + n) // block), width)
        for j in range(had, want):
            table[b, j] = free[at] if at < len(free) else -1
            at += 1
        for i in range(min(n, max(0, T - row))):
            p = c + i
            positions[row + i] = p
            if p // block < want and table[b, p // block] >= 0:
                slots[row + i] = int(table[b, p // block]) * block + p % block
        row += n
    row_start[B] = min(row, T)
    return table, total, row_start, slots, positions, at


# ------------------------------------------------------------------ cache

def codes_of(x, gamma, bits):
    """Codes of float32 values under gamma, each float32 operation rounded once."""
    L = np.float32(2 ** bits - 1)
    r = L / (np.float32(2.0) * (np.float32(gamma) + EPS32))
    return np.clip(np.rint(np.asarray(x, np.float32) * r + np.float32(0.5) * L), 0, L).astype(np.uint8)


def append(x, slots, codes, scales, bits):
    """The cache after the rows x [T][H][D] (float32 values) went to their slots, one row after the other over each
    block: codes [n][H][block][D] and scales [n][H] are copied."""
    codes, scales = codes.copy(), scales.copy()
    n, H, block, D = codes.shape
    L = np.float32(2 ** bits - 1)
    T, t = len(slots), 0
    while t < T:
        s = int(slots[t])
        if s < 0 or s >= n * block:
            t += 1
            continue
        page, place = divmod(s, block)
        e = t + 1
        while e < T and slots[e] == s + (e - t) and place + (e - t) < block:
            e += 1
        for h in range(H):
            rows = np.asarray(x[t:e, h], np.float32)
            old = scales[page, h] if place else np.float32(0)
            gamma = max(old, np.abs(rows).max())
            if place and gamma > old:
                u = old / L
                value = (np.float32(2) * codes[page, h, :place].astype(np.float32) - L) * u
                codes[page, h, :place] = codes_of(value, gamma, bits)
            codes[page, h, place:place + (e - t)] = codes_of(rows, gamma, bits)
            scales[page, h] = gamma
        t = e
    return codes, scales


def values(codes, scales, bits):
    """What the codes stand for, in 64 bits."""
    L = 2.0 ** bits - 1
    return (2.0 * codes.astype(np.float64) - L) * (scales.astype(np.float64) / L)[..., None, None]


# ------------------------------------------------------------------ attention

def attention(q, row_start, total, table, k, v, scale, v_scales=None):
    """64-bit causal attention over pages: q [T][Hq][D], k and v the cache's values [n][H][block][D], v_scales the
    gammas of v.  Returns (o, mass, reach, crest): o NaN in rows of no request, mass = sum_j p_j |v_j| (what relative
    errors of the weights act on), reach = the largest scale * sum_d |q_d k_jd| of a row (what relative errors of a
    score's products act on), crest = the largest p_j gamma_j (what the smallest step of a weight is a part of)."""
    T, Hq, D = q.shape
    n, H, block, _ = k.shape
    B, width = table.shape
    o = np.full((T, Hq, D), np.nan)
    mass, reach, crest = np.zeros((T, Hq, D)), np.zeros((T, Hq, 1)), np.zeros((T, Hq, 1))
    gamma = np.abs(v).max((2, 3)) if v_scales is None else np.asarray(v_scales, np.float64)
    for b in range(B):
        lo, hi = int(row_start[b]), int(row_start[b + 1])
        for t in range(lo, hi):
            keys = max(0, min(int(total[b]) - hi + t + 1, width * block))
            ids = table[b, :-(-keys // block)].astype(np.int64)
            good = (ids >= 0) & (ids < n)
            seen = np.repeat(good, block)[:keys]
            if not seen.any():
                o[t] = 0.0
                continue
            safe = np.where(good, ids, 0)
            for h in range(H):
                kk = k[safe, h].reshape(-1, D)[:keys][seen]
                vv = v[safe, h].reshape(-1, D)[:keys][seen]
                rows = slice(h * (Hq // H), (h + 1) * (Hq // H))
                qq = q[t, rows].astype(np.float64)
                s = qq @ kk.T * scale
                p = np.exp(s - s.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                o[t, rows] = p @ vv
                mass[t, rows] = p @ np.abs(vv)
                reach[t, rows, 0] = (np.abs(qq) @ np.abs(kk).T).max(-1) * abs(scale)
                crest[t, rows, 0] = (p * np.repeat(gamma[safe, h], block)[:keys][seen]).max(-1)
    return o, mass, reach, crest


def attention_tolerance(o, mass, reach, crest, keys, q_f32, o_f32):
    """How far an element may be off, counted from the contract: the output's rounding (half a step: 2^-8 bf16, 2^-24
    float); the weights' rounding to fp16, 2^-11 (float q: two parts, 2^-22); a score's error moves its weight and the
    sum: twice 2^-18 reach (22-bit products, at most 32 float accumulation steps of 2^-23 each, which truncate) and
    2^-20 for the exponential and the scaling; and float accumulation over the keys in steps of 16.  A weight times its
    block's gamma is held on a scale where the row's largest lies in [2^7, 2^15]: what is below fp16's normal numbers
    there is off by half its smallest step, 2^-25, at most 2^-32 of crest for a key; weights that underflow float,
    2^-126."""
    weights = (2.0 ** -22 if q_f32 else 2.0 ** -11) + 2 * (2.0 ** -18 * reach + 2.0 ** -20) + (keys / 16 + 8) * 2.0 ** -23
    return (2.0 ** -24 if o_f32 else 2.0 ** -8) * np.abs(o) + weights * mass + keys * (2.0 ** -32 * crest + 2.0 ** -126)


# ------------------------------------------------------------------ residual, RMSNorm, quantizer

def add_rms_quant(x, r, gain, bits, bf16):
    """(h, t, codes, scales): x, r float32 values; every float32 operation rounded once, sums in 64 bits."""
    x = np.asarray(x, np.float32)
    K = x.shape[1]
    h = x if r is None else x + np.asarray(r, np.float32)
    if bf16:
        h = bf16_round(h)
    ms = np.array([[math.fsum(float(v) * float(v) for v in row) / K] for row in h]).astype(np.float32)
    rstd = np.float32(1) / np.sqrt(ms + EPS32)
    t = h * rstd
    if gain is not None:
        t = t * np.asarray(gain, np.float32)
    if bits == 8:
        c, lo, hi = np.float32(127), -128, 127
        stat = np.abs(t).max(1)
    else:
        c, lo, hi = np.float32(math.sqrt(7.0)), -8, 7
        stat = np.array([math.fsum(abs(float(v)) for v in row) / K for row in t]).astype(np.float32)
    rr = c / (stat + EPS32)
    q = np.clip(np.rint(t.astype(np.float64) * rr.astype(np.float64)[:, None]), lo, hi).astype(np.int8)
    return h, t, q, stat / c


def rms_value(h, gain):
    """The normalised value in 64 bits (the quantizer passed straight through)."""
    h = np.asarray(h, np.float64)
    t = h / np.sqrt((h * h).mean(1, keepdims=True) + 1e-5)
    return t if gain is None else t * np.asarray(gain, np.float64)


def add_rms_backward(h, gain, g_t, g_h):
    """(g_x, g_gain, per-element size of the terms of g_x) in 64 bits."""
    h, g_t = np.asarray(h, np.float64), np.asarray(g_t, np.float64)
    K = h.shape[1]
    rstd = 1.0 / np.sqrt((h * h).mean(1, keepdims=True) + 1e-5)
    n = h * rstd
    g_u = g_t if gain is None else g_t * np.asarray(gain, np.float64)
    c = (g_u * n).sum(1, keepdims=True) / K
    g_x = rstd * (g_u - n * c)
    size = rstd * (np.abs(g_u) + np.abs(n) * (np.abs(g_u * n).sum(1, keepdims=True) / K))
    if g_h is not None:
        g_x = g_x + np.asarray(g_h, np.float64)
        size = size + np.abs(np.asarray(g_h, np.float64))
    return g_x, (g_t * n).sum(0), size
