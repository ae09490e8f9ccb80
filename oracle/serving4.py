"""Plain float64 / integer restatement of the serving step's other operators (norms and rotary positions, the 4-bit
paged cache and attention over it, verification of drafted tokens): loops over requests, tokens and heads, from the
definitions in include/moe.h."""
from __future__ import annotations

import numpy as np

from oracle import serving as S

# byte of each of 16 tokens' scales
SCALE_BYTE = [4 * (t % 8 // 2) + 2 * (t // 8) + t % 2 for t in range(16)]
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])


def rotate(x, positions, freqs, axes=None, interleaved=False, gamma=None, eps=1e-5, factor=1.0):
    """Rows x [n][heads][D] at positions [n_axes][n] -> (y, tol): y in float64 and how far a result in 32 bits may be
    off that is rounded once to bf16: 2^-8 |y| + 2^-19 factor (|a| + |b|) of a pair (a, b).  A norm's sum of up to 256
    squares in pieces of at most 13 additions, its root and the products: below 2^-20.5 relative; a sine's or
    cosine's argument and itself: below 2^-21; the rotation's own products and sum: 2^-23."""
    y = np.asarray(x, np.float64).copy()
    n, H, D = y.shape
    if gamma is not None:
        with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
            y = y / np.sqrt((y * y).mean(-1, keepdims=True) + np.float64(np.float32(eps))) * np.asarray(gamma, np.float64)
    size = np.abs(y)
    out, pairs = y.copy(), len(freqs)
    for i in range(pairs):
        axis = 0 if axes is None else int(axes[i])
        angle = np.asarray(positions, np.float64).reshape(-1, n)[axis] * freqs[i]
        c, s = np.cos(angle)[:, None] * factor, np.sin(angle)[:, None] * factor
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        out[:, :, a] = y[:, :, a] * c - y[:, :, b] * s
        out[:, :, b] = y[:, :, b] * c + y[:, :, a] * s
        size[:, :, a] = size[:, :, b] = factor * (np.abs(y[:, :, a]) + np.abs(y[:, :, b]))
    return out, 2.0 ** -8 * np.abs(out) + 2.0 ** -19 * size + 1e-40


def exponent(amax):
    """ceil(log2(amax / 6)) for amax at least 6 * 2^-126, at most 125."""
    a = max(float(amax), 6 * 2.0 ** -126)
    if np.isinf(a):
        return 125
    m, e = np.frexp(a / 6)
    return min(int(e) - (1 if m == 0.5 else 0), 125)


def e2m1(x):
    """Codes of the nearest E2M1 values, ties to the even code; beyond +-6 saturated, NaN +6, -0 as 0."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    code = np.zeros(x.shape, np.uint8)
    for limit, tie_up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a > limit) | ((a == limit) & tie_up)
    code = np.where(np.isnan(x), 7, code | np.where(x < 0, 8, 0))
    return code.astype(np.uint8)


def page_bytes(P, D):
    return P * D // 16 * 17


def unpack(cache, P, D):
    """Cache [pages][kv][bytes] -> codes [2][pages][P][kv][D], scale bytes [2][pages][P][kv][D / 32]."""
    n, kv = cache.shape[:2]
    half, few, nb = P * D // 2, P * D // 32, D // 32
    codes, scales = np.empty((2, n, P, kv, D), np.uint8), np.empty((2, n, P, kv, nb), np.uint8)
    for side in range(2):
        c = cache[:, :, side * half:(side + 1) * half].reshape(n, kv, nb, P, 16)
        both = np.stack([c & 15, c >> 4], -1).reshape(n, kv, nb, P, 32)
        codes[side] = both.transpose(0, 3, 1, 2, 4).reshape(n, P, kv, D)
        s = cache[:, :, 2 * half + side * few:2 * half + (side + 1) * few].reshape(n, kv, nb, P // 16, 16)[..., SCALE_BYTE]
        scales[side] = s.reshape(n, kv, nb, P).transpose(0, 3, 1, 2)
    return codes, scales


def pack(codes, scales):
    _, n, P, kv, D = codes.shape
    half, few, nb = P * D // 2, P * D // 32, D // 32
    cache = np.empty((n, kv, page_bytes(P, D)), np.uint8)
    for side in range(2):
        c = codes[side].reshape(n, P, kv, nb, 32).transpose(0, 2, 3, 1, 4)
        cache[:, :, side * half:(side + 1) * half] = (c[..., 0::2] | c[..., 1::2] << 4).reshape(n, kv, half)
        s = np.empty((n, kv, nb, P // 16, 16), np.uint8)
        s[..., SCALE_BYTE] = scales[side].transpose(0, 2, 3, 1).reshape(n, kv, nb, P // 16, 16)
        cache[:, :, 2 * half + side * few:2 * half + (side + 1) * few] = s.reshape(n, kv, few)
    return cache


def scale_value(byte):
    """Scale bytes as numbers: 0 counts as 0, what is above 252 as 252."""
    b = np.minimum(np.asarray(byte, np.int64), 252)
    return np.where(b == 0, 0.0, 2.0 ** (b - 127.0))


def values(codes, scales):
    """What codes [..., D] with scales [..., D / 32] stand for."""
    return E2M1[codes] * np.repeat(scale_value(scales), 32, -1)


def append(cache, P, xk, xv, slots):
    """The cache after rows xk, xv [n][kv][D] (float) went to slots."""
    D = xk.shape[2]
    codes, scales = unpack(cache, P, D)
    for t, s in enumerate(slots):
        if not 0 <= s < cache.shape[0] * P:
            continue
        page, o = divmod(int(s), P)
        for side, x in enumerate((xk, xv)):
            for h in range(x.shape[1]):
                for b in range(D // 32):
                    block = np.asarray(x[t, h, 32 * b:32 * b + 32], np.float64)
                    a = np.abs(block)[~np.isnan(block)]
                    k = exponent(a.max() if a.size else 0.0)
                    scales[side, page, o, h, b] = k + 127
                    codes[side, page, o, h, 32 * b:32 * b + 32] = e2m1(block * 2.0 ** -k)
    return pack(codes, scales)


def read(cache, P, D, slots):
    """Keys and values [n][kv][D] (float64) at slots, all of them in the cache."""
    codes, scales = unpack(cache, P, D)
    page, o = np.asarray(slots) // P, np.asarray(slots) % P
    return [values(codes[s][page, o], scales[s][page, o]) for s in range(2)]


def attend(cache, P, q, starts, lens, table, window=0, sinks=None, scale=None, weight=2.0 ** -11, floor=2.0 ** -31, flush=2.0 ** -120):
    """-> (out, tol): out [rows][heads][D] float64 (NaN rows where no sequence has one), and how far a result may be
    off that holds probabilities to `weight` of themselves, scores and sums in 32 bits, and rounds once to bf16: with
    A = sum_t p_t |v_t| and B = max_t scale sum_d |q_d k_td|,
        2^-8 |out| + A (2 weight + 2 (D + 8) 2^-24 B + 2^-18) + floor F + flush max_t 2^(e_t) sum_t |code_td|.
    A score is a sum of D products, off by at most (D + 4) 2^-24 B in 32 bits; turning it into a power of two and its
    argument's rounding add at most 4 * 2^-24 B, since |s| <= B.  Each p_t is off by that relative to itself, which
    moves numerator and denominator by at most A times it; `weight` for the rounding of p (half a step: 2^-11 and the
    power of two's own error in fp16, 2^-8 in bf16), and as much again for the sums; 2^-18 where 2 weight is nothing.
    F = max_t (p_t 2^(e_t)) sum_t |code_td| over a block of 32 dims, with e_t the token's exponent: fp16 weights
    2^(s - m + e_t - E), E at most 4 above e_t, m at most 11 below the largest score when it was set and never more than
    15 below one since, so 2^7 at least for the token of the largest score; below 2^-14 they are off by up to half of fp16's smallest step, 2^-25: 2^-32 of the largest,
    doubled for parts with references of their own.
    F counts on a weight of 2^-21 of the largest or more for the token that counts most in a dim: one of 2^-31 may be taken
    as 0, and a result that such tokens alone make up (the others' codes being 0) is none.
    The last term, for such weights on tokens of the largest scales: 2^-120, where scales are within 2^120 of one another
    less than the floor.  0 where all of a row's weights are of one size."""
    D, H = q.shape[2], q.shape[1]
    kv, n_pages = cache.shape[1], cache.shape[0]
    codes, scales = unpack(cache, P, D)
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    out, tol = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    for b in range(len(lens)):
        s, e = int(starts[b]), int(starts[b + 1])
        for r in range(s, e):
            p = int(lens[b]) - (e - r)
            seen = np.arange(max(0, p - window + 1) if window else 0, max(p + 1, 0))
            seen = seen[seen // P < table.shape[1]]
            pages = table[b, seen // P] if len(seen) else seen
            ok = (pages >= 0) & (pages < n_pages)
            pages, at = pages[ok], (seen % P)[ok]
            if not len(pages):
                out[r] = tol[r] = 0.0
                continue
            k, v = (values(codes[i][pages, at], scales[i][pages, at]) for i in range(2))
            ve = np.repeat(scale_value(scales[1][pages, at]), 32, -1)
            for h in range(H):
                g = h // (H // kv)
                qv = np.asarray(q[r, h], np.float64)
                x = scale * (k[:, g] @ qv)
                m = max(x.max(), sinks[h]) if sinks is not None else x.max()
                w = np.exp(x - m)
                w = w / (w.sum() + (np.exp(sinks[h] - m) if sinks is not None else 0.0))
                out[r, h] = w @ v[:, g]
                B = scale * (np.abs(k[:, g]) @ np.abs(qv)).max()
                F = (w[:, None] * ve[:, g]).max(0) * np.abs(E2M1[codes[1][pages, at, g]]).sum(0)
                F = floor * F + flush * ve[:, g].max(0) * np.abs(E2M1[codes[1][pages, at, g]]).sum(0)
                tol[r, h] = F + 2.0 ** -8 * np.abs(out[r, h]) + \
                    w @ np.abs(v[:, g]) * (2 * weight + 2 * (D + 8) * 2.0 ** -24 * B + 2.0 ** -18)
    return out, tol + 1e-30


def probabilities(logits, t, k, p, min_p):
    """What a row's token is drawn from; all 0 for a row without a token."""
    w = S.kept(logits, t, k, p, min_p)
    return w / w.sum() if w.any() else w


def verify(ps, drafts, qs, u, draw):
    """One sequence: ps the rows' probabilities, qs the drafts' ones (None: certain), u one a row.
    -> (accepted, the rest's weights at the row of the draw, the least |u q - p| on the way there)."""
    n, V, near = len(ps), len(ps[0]), np.inf
    for j in range(n - 1):
        x = int(drafts[j])
        q = np.zeros(V)
        if qs is None:
            if 0 <= x < V:
                q[x] = 1.0
        else:
            q = np.clip(np.nan_to_num(np.asarray(qs[j], np.float64), nan=0.0), 0.0, 1.0)
        if 0 <= x < V:
            near = min(near, abs(float(u[j]) * q[x] - ps[j][x]) / max(ps[j][x], 1e-30) if ps[j][x] else np.inf)
            if float(u[j]) * q[x] < ps[j][x]:
                continue
        rest = np.maximum(ps[j] - q, 0.0)
        return j, rest if rest.any() else ps[j], near
    return n - 1, ps[n - 1], near
