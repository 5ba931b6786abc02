"""64-bit definitions of the latent cache's attention and of eviction by
attention weight, with bounds of what arithmetic in fewer bits may differ by.

Every bound counts roundings: half a step of a bf16 is 2^-8 of the value, of a
fp32 2^-24, and tensor cores may cut an fp32 sum instead of rounding it, 2^-23.
"""
import numpy as np

CUT = 2.0 ** -23   # one fp32 addition
F32 = 2.0 ** -24   # one rounding to fp32
BF16 = 2.0 ** -8   # one rounding to bf16
TWO = 2.0 ** -16   # a value in two bf16 parts: the second rounds what the first left
EXP = 2.0 ** -20   # the exponential, the logarithm and the products around them


def rows(cache, table, n, bs):
    """The first n rows [n, ..., D] of the pages [NB, ..., bs, D] that a table names."""
    t = np.arange(n)
    if cache.ndim == 3:
        return np.asarray(cache[table[t // bs], t % bs], dtype=np.float64)
    return np.asarray(cache[table[t // bs], :, t % bs], dtype=np.float64)


def append(latent, rope, slots, cache):
    nb, bs, _ = cache.shape
    for t, s in enumerate(slots):
        if 0 <= s < nb * bs:
            cache[s // bs, s % bs] = np.concatenate([latent[t], rope[t]])


def softmax(s):
    """softmax over the last axis; -inf where masked; rows without any entry are zero."""
    m = s.max(-1, keepdims=True)
    e = np.exp(s - np.where(np.isfinite(m), m, 0.0))
    total = e.sum(-1, keepdims=True)
    return e / np.where(total > 0, total, 1.0)


def attend(q, k, v, scale, limit, dk=None, dv=None, dp=BF16):
    """out [R, Dv] and its bound in fp32, before a rounding of the output: q [R, D],
    k [T, D], v [T, Dv]; row r sees the first limit[r] keys.  dk, dv: by how
    much the kernel's keys and values may differ from these; dp: the rounding of
    the probabilities."""
    R, T = q.shape[0], k.shape[0]
    if T == 0:
        return np.zeros((R, v.shape[1])), np.zeros((R, v.shape[1]))
    hide = np.arange(T)[None] >= np.asarray(limit)[:, None]
    s = np.where(hide, -np.inf, scale * (q @ k.T))
    ds = (q.shape[1] + 4) * CUT * abs(scale) * (np.abs(q) @ np.abs(k).T)
    if dk is not None:
        ds = ds + abs(scale) * (np.abs(q) @ dk.T)
    d = np.where(hide, 0.0, ds).max(1, keepdims=True)
    p = softmax(s)
    mass = p @ np.abs(v)
    rel = 2 * np.expm1(2 * d) + EXP + dp + (T + 64) * CUT
    tol = rel * mass
    if dv is not None:
        tol = tol + (1 + rel) * (p @ dv)
    return p @ v, tol


def decode(q, cache, tables, lens, scale, latent, dp=BF16):
    """q [B, Q, H, D] -> (out [B, Q, H, latent], bound)."""
    B, Q, H, _ = q.shape
    bs = cache.shape[1]
    out, tol = np.zeros((B, Q, H, latent)), np.zeros((B, Q, H, latent))
    for i in range(B):
        x = rows(cache, tables[i], int(lens[i]), bs)
        for j in range(Q):
            limit = np.full(H, max(0, int(lens[i]) - Q + 1 + j))
            out[i, j], tol[i, j] = attend(q[i, j].astype(np.float64), x, x[:, :latent], scale, limit, dp=dp)
    return out, tol


def to_bf16(x):
    """Nearest bf16 (ties to even) of float64 values, as float64."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256.0), e - 8)


def expanded(c, w, two=False, f32=False):
    """c [T, L] by w [D, L]: bf16 values [T, D], and by how much a kernel's may
    differ: a whole step where fp32 arithmetic may round to the other side.
    f32: the values themselves, and what fp32 sums leave; two: a wider bound, with
    room for a second part of 8 bits."""
    x = c @ w.T
    slack = (c.shape[1] + 4) * CUT * (np.abs(c) @ np.abs(w).T)
    if f32:
        return x, slack
    if two:
        return x, slack + TWO * (np.abs(x) + slack)
    r = to_bf16(x)
    return r, np.maximum(np.abs(to_bf16(x + slack) - r), np.abs(to_bf16(x - slack) - r))


def prefill(q, cache, w_k, w_v, cu, start, tables, scale, two=False, f32=False):
    """q [T, H, head + rope] -> (out [T, H, head], bound); keys, values and
    probabilities rounded to bf16, or (f32) to nothing below fp32; two: as f32 with
    the bound of 16 bits."""
    T, H, _ = q.shape
    head, latent = w_k.shape[1:]
    bs = cache.shape[1]
    out, tol = np.zeros((T, H, head)), np.zeros((T, H, head))
    for i in range(len(start)):
        n, a = int(cu[i + 1] - cu[i]), int(start[i])
        if n == 0:
            continue
        x = rows(cache, tables[i], a + n, bs)
        for h in range(H):
            k, dk = expanded(x[:, :latent], w_k[h].astype(np.float64), two, f32)
            v, dv = expanded(x[:, :latent], w_v[h].astype(np.float64), two, f32)
            k = np.concatenate([k, x[:, latent:]], 1)
            dk = np.concatenate([dk, np.zeros_like(x[:, latent:])], 1)
            o, t = attend(q[cu[i]:cu[i + 1], h].astype(np.float64), k, v, scale, a + 1 + np.arange(n), dk, dv,
                          F32 if f32 else TWO if two else BF16)
            out[cu[i]:cu[i + 1], h], tol[cu[i]:cu[i + 1], h] = o, t
    return out, tol


def weights(before, q, k_cache, tables, lens, scale):
    """before [B, M] fp32, q [B, W, H, D], k_cache [NB, Hkv, bs, D] -> (after, bound)."""
    B, W, H, D = q.shape
    hkv, bs = k_cache.shape[1], k_cache.shape[2]
    out = np.asarray(before, dtype=np.float64).copy()
    tol = np.zeros_like(out)
    for i in range(B):
        n = int(lens[i])
        if n == 0:
            continue
        k = rows(k_cache, tables[i], n, bs)
        for j in range(W):
            if n - W + 1 + j <= 0:
                continue
            hide = np.arange(n) >= n - W + 1 + j
            for h in range(H):
                x, kk = q[i, j, h].astype(np.float64), k[:, h // (H // hkv)]
                ds = (D + 4) * CUT * abs(scale) * (np.abs(kk) @ np.abs(x))
                d = np.where(hide, 0.0, ds).max()
                p = softmax(np.where(hide, -np.inf, scale * (kk @ x)))
                out[i, :n] += p
                tol[i, :n] += p * (2 * np.expm1(2 * d) + EXP + (n + 64) * CUT)
        tol[i, :n] += (W * H + 4) * CUT * np.abs(out[i, :n])
    return out, tol


def select(weights, start, lens, counts, recent):
    """(keep, weights after): the kept positions of all sequences one behind the other."""
    w = np.array(weights)
    keep = []
    for i in range(len(lens)):
        a, b, n = int(start[i]), int(lens[i]), int(counts[i])
        late = min(recent, n)
        cand = np.where(np.isnan(w[i, a:b - late]), -np.inf, w[i, a:b - late])
        # NaN below everything: behind every number, -inf included
        rank = np.lexsort((np.arange(len(cand)), np.isnan(w[i, a:b - late]), -cand))[: n - late]
        pick = np.concatenate([a + np.sort(rank), np.arange(b - late, b)]).astype(np.int64)
        row = w[i].copy()
        row[a:b] = 0
        row[a:a + n] = w[i, pick]
        w[i] = row
        keep.append(pick)
    return np.concatenate(keep), w
