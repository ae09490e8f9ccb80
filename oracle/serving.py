"""Plain float64 / integer restatement of the serving operators (page tables, the 8-bit paged cache and
attention over it, sampling): loops over requests, tokens and heads, from the definitions in include/moe.h."""
from __future__ import annotations

import numpy as np

INT_MAX = 2 ** 31 - 1
# token of 16 at each byte of a value block
PLACE = [0, 1, 8, 9, 2, 3, 10, 11, 4, 5, 12, 13, 6, 7, 14, 15]


def pages_assign(P, cached, fresh, free, n_free, table, max_tokens):
    """-> dict(free, counts, table, starts, lens, slots, positions); inputs are not changed."""
    free, table = list(map(int, free)), np.array(table, np.int32)
    n, width = table.shape
    cap = len(free)
    top = min(max(int(n_free), 0), cap)
    have = [max(int(c), 0) for c in cached]
    held = [min(-(-h // P), width) for h in have]
    for b in range(n):
        if fresh[b] < 0:
            for j in range(held[b]):
                if table[b, j] >= 0 and top < cap:
                    free[top] = int(table[b, j])
                    top += 1
    missing, starts, lens, slots, pos = 0, [0], [], [], []
    for b in range(n):
        add = int(fresh[b])
        if add < 0:
            lens.append(0)
            starts.append(starts[-1])
            continue
        for j in range(held[b], min(-(-(have[b] + add) // P), width)):
            if top > 0:
                top -= 1
                table[b, j] = free[top]
            else:
                missing += 1
                table[b, j] = -1
        for i in range(add):
            t = have[b] + i
            pg = int(table[b, t // P]) if t // P < width else -1
            slots.append(pg * P + t % P if pg >= 0 else -1)
            pos.append(t)
        lens.append(have[b] + add)
        starts.append(starts[-1] + add)
    tail = max(0, max_tokens - len(slots))
    return dict(free=np.array(free, np.int32), counts=np.array([top, missing], np.int32), table=table,
                starts=np.array(starts, np.int32), lens=np.array(lens, np.int32),
                slots=np.array((slots + [-1] * tail)[:max_tokens], np.int32),
                positions=np.array((pos + [-1] * tail)[:max_tokens], np.int32))


def _e4m3_values():
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = np.nan if (c & 127) == 127 else (-x if c & 128 else x)
    return v


E4M3 = _e4m3_values()


def e4m3(x):
    """Codes of the nearest E4M3 values, ties to the even code; beyond +-448 saturated, NaN the NaN code."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    safe = np.where(np.isnan(a) | (a == 0), 1.0, a)
    q = 2.0 ** (np.maximum(np.frexp(safe)[1] - 1, -6) - 3)
    r = np.rint(safe / q) * q                       # half to even: q steps alternate even and odd codes
    code = np.searchsorted(E4M3[:127], r)
    code = np.where(a == 0, 0, code) | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 127, code).astype(np.uint8)


def exponent(amax):
    """ceil(log2(amax / 448)) for amax at least 448 * 2^-126 and at most the largest float."""
    a = min(max(float(amax), 448 * 2.0 ** -126), float(np.finfo(np.float32).max))
    m, e = np.frexp(a / 448)
    return int(e) - (1 if m == 0.5 else 0)



def unpack(k, v, P, D):
    """Code arrays [pages][kv][P * D] -> codes [pages][P][kv][D], keys and values."""
    n, kv = k.shape[:2]
    kk = k.reshape(n, kv, D // 16, P, 16).transpose(0, 3, 1, 2, 4).reshape(n, P, kv, D)
    vv = np.empty((n, P, kv, D), np.uint8)
    blocks = v.reshape(n, kv, P // 16, D, 16)
    for byte, tok in enumerate(PLACE):
        vv[:, tok::16] = blocks[..., byte].transpose(0, 2, 1, 3)
    return kk, vv


def pack(kk, vv):
    n, P, kv, D = kk.shape
    k = kk.reshape(n, P, kv, D // 16, 16).transpose(0, 2, 3, 1, 4).reshape(n, kv, P * D)
    blocks = np.empty((n, kv, P // 16, D, 16), np.uint8)
    for byte, tok in enumerate(PLACE):
        blocks[..., byte] = vv[:, tok::16].transpose(0, 2, 1, 3)
    return np.ascontiguousarray(k), blocks.reshape(n, kv, P * D)


def append(k, v, ks, vs, P, xk, xv, slots):
    """New (k, v, ks, vs) after appending rows xk, xv [n][kv][D] (float) at slots."""
    D, kv, pages = xk.shape[2], xk.shape[1], k.shape[0]
    kk, vv = unpack(k, v, P, D)
    ks, vs = ks.copy(), vs.copy()
    t = 0
    while t < len(slots):
        s = int(slots[t])
        if not 0 <= s < pages * P:
            t += 1
            continue
        z = t + 1
        while z < len(slots) and slots[z] == slots[z - 1] + 1 and slots[z] % P:
            z += 1
        page, o = divmod(s, P)
        for codes, scales, x in ((kk, ks, xk), (vv, vs, xv)):
            for h in range(kv):
                new = np.asarray(x[t:z, h], np.float64)
                a = np.abs(new)[~np.isnan(new)]
                byte = exponent(a.max() if a.size else 0.0) + 127
                if o:
                    old = int(scales[page, h])
                    if byte > old:
                        codes[page, :o, h] = e4m3(E4M3[codes[page, :o, h]] * 2.0 ** (old - byte))
                    byte = max(byte, old)
                scales[page, h] = byte
                codes[page, o:o + z - t, h] = e4m3(new * 2.0 ** (127 - byte))
        t = z
    return (*pack(kk, vv), ks, vs)


def attend(k, v, ks, vs, P, q, starts, lens, table, window=0, sinks=None, scale=None, floor=2.0 ** -39):
    """-> (out, tol): out [rows][heads][D] float64 (NaN rows where no sequence has one), and how far a result may
    be off that holds probabilities in 11 bits or more, scores and sums in 32 bits, and rounds once to bf16:
    with A = sum_t p_t |v_t| and B = max_t scale sum_d |q_d k_td|,
        2^-8 |out| + A (2^-10 + 2 (D + 8) 2^-24 B) + floor F + 2^-110 sum_t |v_t|.
    A score is a sum of D products, off by at most (D + 4) 2^-24 B in 32 bits; turning it into a power of two
    and its argument's rounding add at most 4 * 2^-24 B, since |s| <= B.  Each p_t is off by that relative to
    itself, which moves numerator and denominator by at most A times it; 2^-11 A for the rounding of p, and as
    much again for the sums.
    F = max_t (p_t 2^(e_t)) sum_t |code_td|, with e_t the value page's exponent: weights p_t 2^(e_t) held in fp16,
    scaled so that the largest is at most 2^15, are off by up to half of fp16's smallest step, 2^-25, where they
    are below 2^-14: 2^-40 of the largest (2^-39 where another unit's reference was up to twice as large).  The kernel for prompts moves
    its reference only when passed by 2^8, and scales the reference to 2^7: 2^-25 / 2^7, doubled likewise: 2^-31.
    The last term: the factor that turns p_t into its fp16 weight, 2^(15 + e_t - N) with 2^N = max_u p_u 2^(e_u), is
    held to 2^126, so weights with e_t - N > 111 come out too small; for those p_t <= 2^(N - e_t) < 2^-111."""
    D, H, kv = q.shape[2], q.shape[1], k.shape[1]
    kk, vv = unpack(k, v, P, D)
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    out = np.full(q.shape, np.nan)
    tol = np.full(q.shape, np.nan)
    for b in range(len(lens)):
        s, e = int(starts[b]), int(starts[b + 1])
        for r in range(s, e):
            p = int(lens[b]) - (e - r)
            seen = [t for t in range(max(0, p - window + 1) if window else 0, p + 1)
                    if t // P < table.shape[1] and 0 <= table[b, t // P] < k.shape[0]]
            pages = [int(table[b, t // P]) for t in seen]
            at = [t % P for t in seen]
            for h in range(H):
                g = h // (H // kv)
                if not seen:
                    out[r, h] = tol[r, h] = 0.0
                    continue
                kt = E4M3[kk[pages, at, g]] * 2.0 ** (ks[pages, g].astype(np.float64) - 127)[:, None]
                vt = E4M3[vv[pages, at, g]] * 2.0 ** (vs[pages, g].astype(np.float64) - 127)[:, None]
                x = scale * (kt @ np.asarray(q[r, h], np.float64))
                m = max(x.max(), sinks[h]) if sinks is not None else x.max()
                w = np.exp(x - m)
                den = w.sum() + (np.exp(sinks[h] - m) if sinks is not None else 0.0)
                out[r, h] = (w / den) @ vt
                B = scale * (np.abs(kt) @ np.abs(np.asarray(q[r, h], np.float64))).max()
                ve = vs[pages, g].astype(np.float64) - 127
                F = (w / den * 2.0 ** ve).max() * np.abs(E4M3[vv[pages, at, g]]).sum(0)
                tol[r, h] = floor * F + 2.0 ** -110 * np.abs(vt).sum(0) + 2.0 ** -8 * np.abs(out[r, h]) + (w / den) @ np.abs(vt) * (2.0 ** -10 + 2 * (D + 8) * 2.0 ** -24 * B)
    return out, tol + 1e-30


def kept(logits, t, k, p, min_p):
    """Weights of one row's kept tokens (0 for the others), in order of index."""
    x = np.asarray(logits, np.float64)
    V = len(x)
    ok = ~np.isnan(x) & (x > -np.inf)
    if not ok.any():
        return np.zeros(V)
    top = x[ok].max()
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(ok, np.where(x == top, 1.0, np.exp((x - top) / t) if t > 0 else 0.0), 0.0)
    order = np.argsort(np.where(ok, -x, np.inf), kind="stable")
    order = order[:ok.sum()]
    if not t > 0:
        order = order[:1]
    elif 0 < k < V:
        order = order[:k]
    if p < 1 and t > 0:
        before = np.cumsum(w[order]) - w[order]
        keep = before < p * w[order].sum()
        keep[0] = True
        order = order[keep]
    order = order[w[order] >= min(min_p, 1.0)]
    out = np.zeros(V)
    out[order] = w[order]
    return out


def sample(w, u):
    """The token at which the running sum of the kept weights exceeds u times their total; -1 without one."""
    if not w.any():
        return -1
    c = np.cumsum(w)
    return min(int((c <= u * c[-1]).sum()), int(np.flatnonzero(w)[-1]))
