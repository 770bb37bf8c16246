"""A plain 64-bit implementation of the 4-bit key / value cache and of attention over it,
written from the definitions in include/qmm.h (numpy, loops; nothing of the CUDA path)."""
import math

import numpy as np

TILE = 16


def param_halves(mode):
    return 2 if mode == "asym" else 1


def tile_bytes(dim, G, mode):
    return TILE * (dim + 2 * G * 2 * param_halves(mode))


def key_word(dim, n, tok):
    if dim == 64:
        return 2 * (n % 4) + n // 4
    p = n % 4 + 4 * (n // 16)
    if dim == 256:
        p ^= 4 * (tok % 2)
    return 4 * p + (n // 4) % 4


def value_word(dim, n, tok):
    per = dim // 64                      # words per piece of dim / 16 bytes
    piece = n // per
    if dim == 128:
        piece ^= 4 * ((tok // 2) % 2)
    elif dim == 256:
        piece ^= 2 * (tok % 4)
    return piece * per + n % per


def quantize(x, group, mode):
    """x [..., dim] float64 (fp16 / bf16 values) -> codes, scales (fp16), zeros (fp16 or None)."""
    dim = x.shape[-1]
    L = dim if group == -1 else group
    g = np.where(np.isnan(x), 0.0, x).reshape(*x.shape[:-1], dim // L, L)
    lo, hi = np.minimum(g.min(-1), 0), np.maximum(g.max(-1), 0)
    f32 = np.float32
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if mode == "sym":
            span = np.abs(g).max(-1).astype(f32) / f32(7)
        else:
            span = (hi - lo).astype(f32) / f32(15)
        s = np.minimum(span, f32(4096)).astype(np.float16)
        d = np.where(s > 0, s, np.float16(1)).astype(np.float64)
        if mode == "sym":
            z = np.full(s.shape, 8.0)
        else:
            z = np.where(s > 0, np.clip(np.rint(-lo / d), 0, 15), 0.0) + 0.0     # an integer: never -0
        q = np.clip(np.rint(g / d[..., None]) + z[..., None], 0, 15)
    q = np.where((s > 0)[..., None], q, z[..., None])
    return q.reshape(x.shape).astype(np.uint8), s, (z.astype(np.float16) if mode == "asym" else None)


def decode(q, s, z, group):
    dim = q.shape[-1]
    L = dim if group == -1 else group
    g = q.astype(np.float64).reshape(*q.shape[:-1], dim // L, L)
    zz = 8.0 if z is None else z.astype(np.float64)[..., None]
    return ((g - zz) * s.astype(np.float64)[..., None]).reshape(q.shape)


def write_row(cache, page_len, slot, head, which, q, s, z):
    """Put one row's codes and parameters into the cache bytes [pages][heads][tiles][bytes]."""
    dim = len(q)
    tile = cache[slot // page_len, head, slot % page_len // TILE]
    tok = slot % TILE
    for n in range(dim // 8):
        w = value_word(dim, n, tok) if which else key_word(dim, n, tok)
        at = which * TILE * dim // 2 + tok * dim // 2 + 4 * w
        for i in range(4):
            tile[at + i] = q[8 * n + 2 * i] | (q[8 * n + 2 * i + 1] << 4)
    par = s if z is None else np.stack([s, z], -1).reshape(-1)
    raw = par.astype(np.float16).view(np.uint8)
    at = TILE * dim + (which * TILE + tok) * len(raw)
    tile[at:at + len(raw)] = raw


def store(cache, page_len, k, v, slots, group, mode):
    for i, slot in enumerate(slots):
        if slot < 0 or slot >= cache.shape[0] * page_len:
            continue
        for which, x in ((0, k), (1, v)):
            q, s, z = quantize(x[i], group, mode)
            for h in range(x.shape[1]):
                write_row(cache, page_len, slot, h, which, q[h], s[h], None if z is None else z[h])


def read_rows(cache, page_len, dim, slots, group, mode):
    """(K~, V~) [len(slots)][heads][dim] float64."""
    heads = cache.shape[1]
    G = 1 if group == -1 else dim // group
    out = np.zeros((2, len(slots), heads, dim))
    d = np.arange(dim)
    for i, slot in enumerate(slots):
        tile = cache[slot // page_len, :, slot % page_len // TILE]
        tok = slot % TILE
        for which in (0, 1):
            word = np.array([value_word(dim, n, tok) if which else key_word(dim, n, tok) for n in range(dim // 8)])
            at = which * TILE * dim // 2 + tok * dim // 2 + 4 * word[d // 8] + d % 8 // 2
            q = (tile[:, at] >> (4 * (d % 2)).astype(np.uint8)) & 15
            nb = 2 * G * param_halves(mode)
            pa = TILE * dim + (which * TILE + tok) * nb
            par = np.ascontiguousarray(tile[:, pa:pa + nb]).view(np.float16).reshape(heads, G, -1)
            z = par[..., 1] if mode == "asym" else None
            out[which, i] = decode(q, par[..., 0], z, group)
    return out[0], out[1]


def attend(q, keys, values, scale, window):
    """One sequence: q [m, H, dim] its last m tokens' queries, keys / values [n, KV, dim].
    Returns float64 (out, lse, sum_t p |v|, largest sum |q||k| scale, largest step of the visible
    values: at most a seventh of their largest magnitude, see quantize())."""
    m, H, dim = q.shape
    n, KV = keys.shape[0], keys.shape[1]
    out = np.zeros((m, H, dim))
    spread = np.zeros((m, H, dim))
    lse = np.full((m, H), -math.inf)
    dots, step = np.zeros((m, H)), np.zeros((m, H))
    for i in range(m):
        pos = n - m + i
        first = max(0, pos - window + 1) if window else 0
        if pos < 0 or first > pos:
            continue
        for h in range(H):
            k, v = keys[first:pos + 1, h * KV // H], values[first:pos + 1, h * KV // H]
            x = scale * (k @ q[i, h])
            top = x.max()
            e = np.exp(x - top)
            out[i, h] = (e @ v) / e.sum()
            spread[i, h] = (e @ np.abs(v)) / e.sum()
            lse[i, h] = top + math.log(e.sum())
            step[i, h] = np.abs(v).max() / 7 * (1 + 2.0 ** -10)
            dots[i, h] = abs(scale) * (np.abs(k) @ np.abs(q[i, h])).max()
    return out, lse, spread, dots, step


def bounds(out, spread, dots, dim, dtype, step, rounded_keys=False):
    """Largest error of the kernel's output and of its log-sum-exp.  `step`: attend()'s, for a
    format with one scale per token, else 0.  `rounded_keys`: the kernel for many rows per key
    head takes keys as fp16((q - z) s), half a step 2^-11 off in each term of a logit.

    Logits: fp32 sums of at most dim + 8 exact products and their scales, and the
    exponential's argument and result, at most (dim + 16) 2^-24 + 2^-21 of the largest
    sum of magnitudes, on numerator and denominator.  Values and probabilities: one fp16
    rounding each, half a step 2^-11.  Output: half a step of its type (fp16 2^-11, bf16
    2^-8; 2^-25 absolute for fp16 below its normals).  Sums over tokens in fp32: 2^-18
    covers 2^6 additions of halves of 2^-24 in any order of a few thousand terms.

    One scale per token: value codes enter the MMAs as unsigned fp16 subnormals q 2^-20, and
    the zero-points' share is subtracted from the sums.  An MMA adds 16 products and the
    accumulator aligned to the largest of their exponents, 24 bits kept; a subnormal counts with
    the exponent of 2^-14, 2^6 above its unit.  So one MMA errs by at most 17 2^-24 2^6 of the
    largest P s it adds, whatever the codes: over all MMAs at most 17 2^-18 of sum P s, which is
    at most `step` after the division by sum P."""
    logit = (dots + 1.0) * ((dim + 16) * 2.0 ** -24 + 2.0 ** -21)
    if rounded_keys:
        logit = logit + 2.0 ** -11 * dots
    half = 2.0 ** -11 if dtype == "f16" else 2.0 ** -8
    rel = 2 * 2.0 ** -11 * 1.01 + np.expm1(2 * logit)[..., None] + 2.0 ** -18
    return rel * spread * (1 + half) + 17 * 2.0 ** -18 * step[..., None] + half * np.abs(out) + 2.0 ** -24, 2 * logit + 2.0 ** -18
