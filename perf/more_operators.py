"""Workloads of the serving step's other operators: norms and rotary positions of queries and keys, the 4-bit
paged key/value cache (append and read, attention) and the verification of drafted tokens.  Each case is one call
as a serving loop makes it; `run` computes it in plain torch operations, or through the framework's own entry
points where `own` is true.

Cache layout (both sides read and write the same bytes): per page of P tokens and kv head, P * D * 17 / 16 bytes:
key codes [D / 32][P][16] (the 32 dims of a block together, dim 2 i in the low nibble of byte i), value codes
likewise, key scales [D / 32][P], value scales.  Codes are E2M1, scales E8M0 (value 2^(s - 127)); a scale row holds
token 2 t + e of 16 (t < 4, e < 2) at byte 4 t + e and token 8 + 2 t + e at byte 4 t + 2 + e.
"""
import math
import zlib

import numpy as np
import torch

own = False

# Shapes: gpt-oss attention (64 query heads, 8 kv heads, dims of 64, window 128 on alternate layers) as this
# repository's benchmark has it, and generic ones with dims of 128.


def listed():
    return [
        # one decode step of a small server: 64 sequences, one token each, far positions, heads normed
        dict(name="rotate_decode_64", op="rotate", tokens=64, heads=64, kv=8, dim=64, pairs=32, axes=1, norm=True,
             interleaved=False, far=131000),
        # a ragged batch of prompts, an odd number of tokens, dims of 128, no norms
        dict(name="rotate_prompts_4099", op="rotate", tokens=4099, heads=32, kv=4, dim=128, pairs=64, axes=1, norm=False,
             interleaved=False, far=8000),
        # images and video among text: positions of time, height and width, heads normed
        dict(name="rotate_video_15k", op="rotate", tokens=15001, heads=28, kv=4, dim=128, pairs=64, axes=3, norm=True,
             interleaved=False, far=2000),
        # one decode step's keys and values of 48 sequences, and what the cache now holds of them
        dict(name="cache4_decode_48", op="cache", seqs=48, kv=8, dim=64, page=16, ctx=900, new=1),
        # ragged prompts' keys and values, pages that begin and end inside them
        dict(name="cache4_prompts_16k", op="cache", seqs=21, kv=8, dim=128, page=32, ctx=300, new=1500),
        # the smallest call: one request, short context, a full layer with sinks
        dict(name="attend4_one_131", op="attend", seqs=1, heads=64, kv=8, dim=64, page=16, ctx=131, new=1, window=0,
             sinks=True, ragged=False),
        # the repository's own decode workload: 16 sequences with 4096 visible tokens, full layer
        dict(name="attend4_decode_16x4096", op="attend", seqs=16, heads=64, kv=8, dim=64, page=64, ctx=4096, new=1,
             window=0, sinks=True, ragged=False),
        # a step that verifies four drafted tokens a sequence: five rows each over ragged contexts
        dict(name="attend4_drafts_24x5", op="attend", seqs=24, heads=64, kv=8, dim=64, page=32, ctx=7000, new=5,
             window=0, sinks=True, ragged=True),
        # a large ragged decode batch with dims of 128 and an odd number of query heads per kv head
        dict(name="attend4_ragged_96_d128", op="attend", seqs=96, heads=20, kv=4, dim=128, page=32, ctx=12000, new=1,
             window=0, sinks=False, ragged=True),
        # ragged prompts attending over what is cached before them and themselves
        dict(name="attend4_prompts_4x900", op="attend", seqs=4, heads=32, kv=8, dim=128, page=32, ctx=2700, new=900,
             window=0, sinks=False, ragged=True),
        # one interactive request with four drafted tokens: fp32 logits of a 32 K vocabulary, top-k and top-p
        dict(name="verify_one_32k", op="verify", seqs=1, drafts=4, vocab=32001, type="float32", k=50, p=0.95, min_p=0.0,
             mixed=False, probs=True),
        # a decode batch with up to four drafted tokens each, settings of their own, bf16 logits (many equal)
        dict(name="verify_64_128k_mixed", op="verify", seqs=64, drafts=4, vocab=128000, type="bfloat16", k=100, p=0.95,
             min_p=0.02, mixed=True, probs=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "cache", "attend", "attend", "verify"])
    if op == "rotate":
        kv, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
        heads = kv * rng.choice([1, 3, 4, 7, 8])
        return dict(op=op, tokens=_log(rng, 1, max(2, min(16000, 15001 * 32 * 128 // ((heads + kv) * dim)))), heads=heads, kv=kv,
                    dim=dim, pairs=rng.choice([dim // 2, dim // 4]), axes=rng.choice([1, 1, 2, 3]), norm=rng.random() < 0.5,
                    interleaved=rng.random() < 0.3, far=_log(rng, 10, 1000000))
    if op == "cache":
        new = _log(rng, 1, 1500)
        return dict(op=op, seqs=_log(rng, 1, 64 if new < 100 else 20), kv=rng.choice([1, 2, 3, 4, 8]),
                    dim=rng.choice([64, 128]), page=rng.choice([16, 32, 64]), ctx=_log(rng, 1, 1000), new=new)
    if op == "attend":
        kv, group, dim = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 5, 7, 8, 12, 16]), rng.choice([64, 128])
        new = 1 if rng.random() < 0.4 else rng.randint(2, 8) if rng.random() < 0.5 else _log(rng, 9, 700)
        ctx = max(new, _log(rng, 1, 12000 if new <= 8 else 2500))
        most = (96 * 12000 * 4 * 128) // (ctx * kv * dim)
        if new > 1:
            most = min(most, 1200 * 32 * 2500 // (new * kv * group * ctx))
        return dict(op=op, seqs=_log(rng, 1, max(1, min(128, most))), heads=kv * group, kv=kv, dim=dim,
                    page=rng.choice([16, 32, 64]), ctx=ctx, new=new, window=rng.choice([0, 0, 1, 100, 128, 1000]),
                    sinks=rng.random() < 0.5, ragged=rng.random() < 0.7)
    seqs, drafts = _log(rng, 1, 64), rng.randint(0, 7)
    return dict(op=op, seqs=seqs, drafts=drafts, vocab=_log(rng, 2, min(200000, 320 * 128000 // (seqs * (drafts + 1)))),
                type=rng.choice(["float32", "bfloat16"]), k=rng.choice([1, 20, 1000]), p=rng.choice([1.0, 0.95, 0.8, 0.3]),
                min_p=rng.choice([0.0, 0.0, 0.05]), mixed=rng.random() < 0.5, probs=rng.random() < 0.7)


# ---------------------------------------------------------------- inputs

_VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]
_PLACE = [4 * (t % 8 // 2) + 2 * (t // 8) + t % 2 for t in range(16)]    # byte of each of 16 tokens' scales


def _fixed(case):
    """Lengths are the same for every seed, so that outputs keep their shapes, in an order of the seed's own."""
    return np.random.RandomState(zlib.crc32(repr(sorted((k, v) for k, v in case.items() if k != "name")).encode()))


def _lengths(case, rs):
    """(cached or visible tokens, new tokens) of each sequence, on the host."""
    n, S, fixed = case["new"], case["seqs"], _fixed(case)
    if case["op"] == "cache":
        have, new = fixed.randint(0, case["ctx"] + 1, S), fixed.randint(max(1, n // 2), n + 1, S)
    elif case["ragged"]:
        new = fixed.randint(max(1, n // 3), n + 1, S)
        have = np.maximum(new, fixed.randint(1, case["ctx"] + 1, S))
        new[0], have[0] = n, case["ctx"]
    else:
        have, new = np.full(S, case["ctx"], np.int64), np.full(S, n, np.int64)
    order = rs.permutation(S)
    return have[order], new[order]


def _cache(pages, case, g):
    """A filled cache [pages][kv][P * D * 17 / 16] of normally distributed keys and values; blocks differ in size."""
    kv, D, P = case["kv"], case["dim"], case["page"]
    limits = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    place = torch.tensor(_PLACE, device="cuda")
    cache = torch.zeros((pages, kv, P * D * 17 // 16), dtype=torch.uint8, device="cuda")
    half, few = P * D // 2, P * D // 32
    for side, spread in ((0, 1.5), (1, 1.0)):
        for lo in range(0, pages, 4096):
            n = min(4096, pages - lo)
            x = torch.randn((n, kv, D // 32, P, 32), generator=g, device="cuda") * spread
            x *= torch.exp2(torch.randint(0, 3, (n, kv, D // 32, P, 1), generator=g, device="cuda").float())
            e = torch.ceil(torch.log2(x.abs().amax(-1) / 6))
            x /= torch.exp2(e)[..., None]
            code = torch.bucketize(x.abs(), limits, out_int32=True) + torch.where(x < 0, 8, 0)
            code = (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)
            cache[lo:lo + n, :, side * half:(side + 1) * half] = code.reshape(n, kv, -1)
            s = torch.empty((n, kv, D // 32, P // 16, 16), dtype=torch.uint8, device="cuda")
            s[..., place] = (e + 127).to(torch.uint8).view(n, kv, D // 32, P // 16, 16)
            at = 2 * half + side * few
            cache[lo:lo + n, :, at:at + few] = s.reshape(n, kv, -1)
    return cache


def _tables(per_seq, width, rs):
    """A table of distinct pages in random order, -1 behind each sequence's last; and the pages."""
    total = int(per_seq.sum())
    order = rs.permutation(total).astype(np.int32)
    t = np.full((len(per_seq), width), -1, np.int32)
    at = 0
    for b, c in enumerate(per_seq):
        t[b, :c] = order[at:at + c]
        at += c
    return t, max(total, 1)


def _dev(a, dt=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dt is None else t.to(dt)


def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "rotate":
        n, H, kv, D, pairs, axes = (case[k] for k in ("tokens", "heads", "kv", "dim", "pairs", "axes"))
        rows = torch.randn((n, H + 2 * kv, D), generator=g, device="cuda")      # of one projection
        rows *= torch.exp2(2 * torch.randn((n, H + 2 * kv, 1), generator=g, device="cuda"))
        rows = rows.to(torch.bfloat16)
        if axes == 1:     # the positions of a few sequences' tokens
            pos = (rs.randint(0, case["far"], max(1, n // 500))[:, None] + np.arange(-(-n // max(1, n // 500)))).ravel()[None, :n]
        else:             # frames of a grid
            w = max(1, int(math.sqrt(n / 8)))
            i = np.arange(n)
            pos = np.stack([i // (w * w), i // w % w, i % w])[:axes] + rs.randint(0, case["far"])
        freqs = (150000.0 if D == 64 else 1e6) ** (-np.arange(pairs) / pairs)
        of = np.sort(np.arange(pairs) % axes).astype(np.uint8)                   # sections of the pairs, an axis each
        gamma = [1 + 0.1 * torch.randn(D, generator=g, device="cuda") for _ in range(2)] if case["norm"] else [None, None]
        st.update(q=rows[:, :H], k=rows[:, H:H + kv], positions=_dev(pos, torch.int32), freqs=freqs, of=of,
                  angle=_dev(freqs), axis=_dev(of, torch.long), q_gamma=gamma[0], k_gamma=gamma[1],
                  q_out=torch.zeros((n, H, D), dtype=torch.bfloat16, device="cuda"),
                  k_out=torch.zeros((n, kv, D), dtype=torch.bfloat16, device="cuda"))
        if own:
            from mxfp4_mixture_experts_rms_gb300 import moe
            st["plan"] = moe.Rotary(D, freqs, axes=of, interleaved=case["interleaved"], q_gamma=gamma[0], k_gamma=gamma[1],
                                    eps=1e-6)
    elif case["op"] == "cache":
        S, P, kv, D = case["seqs"], case["page"], case["kv"], case["dim"]
        cached, new = _lengths(case, rs)
        per = -(-(cached + new) // P)
        t, pages = _tables(per, int(per.max()), rs)
        n = int(new.sum())
        seq = np.repeat(np.arange(S), new)
        pos = np.concatenate([cached[b] + np.arange(new[b]) for b in range(S)])
        slots = t[seq, pos // P] * P + pos % P
        # keys and values as slices of one projection's rows
        both = torch.randn((n, 2 * kv, D), generator=g, device="cuda")
        both *= 1 + 3 * torch.rand((n, 1, 1), generator=g, device="cuda")
        both = both.to(torch.bfloat16)
        st.update(cache=_cache(pages, case, g), slots=_dev(slots, torch.int32), xk=both[:, :kv], xv=both[:, kv:],
                  k_out=torch.zeros((n, kv, D), dtype=torch.bfloat16, device="cuda"),
                  v_out=torch.zeros((n, kv, D), dtype=torch.bfloat16, device="cuda"))
        if own:
            from mxfp4_mixture_experts_rms_gb300 import moe
            st["plan"] = moe.Kv4(kv, kv, D, P, pages, cache=st["cache"])
    elif case["op"] == "attend":
        P, kv, D, H = case["page"], case["kv"], case["dim"], case["heads"]
        vis, new = _lengths(case, rs)
        per = -(-vis // P)
        t, pages = _tables(per, -(-case["ctx"] // P), rs)
        n = int(new.sum())
        q = (torch.randn((n, H, D), generator=g, device="cuda") * 0.7).to(torch.bfloat16)
        sinks = torch.randn(H, generator=g, device="cuda") if case["sinks"] else None
        st.update(cache=_cache(pages, case, g), q=q, sinks=sinks, table=_dev(t), lens=_dev(vis, torch.int32),
                  starts=None if case["new"] == 1 else _dev(np.concatenate([[0], np.cumsum(new)]), torch.int32),
                  out=torch.zeros_like(q))
        if own:
            from mxfp4_mixture_experts_rms_gb300 import moe
            st["plan"] = moe.Kv4(H, kv, D, P, pages, sliding_window=case["window"], sinks=sinks, cache=st["cache"])
    else:
        S, V = case["seqs"], case["vocab"]
        rows = _fixed(case).randint(max(1, case["drafts"]), case["drafts"] + 2, S)    # the drafts and one more
        starts = np.concatenate([[0], np.cumsum(rows[rs.permutation(S)])])
        n = int(starts[-1])
        x = torch.randn((n, V), generator=g, device="cuda") * 2.5
        step = max(1, V // 40)
        x[:, ::step] += 6.0 * torch.rand((n, len(range(0, V, step))), generator=g, device="cuda")
        # a smaller model's probabilities, and the tokens that it drew from them
        near = x + torch.randn((n, V), generator=g, device="cuda")
        q = torch.softmax(near / 0.8, -1)
        drafts = (near / 0.8 - torch.log(-torch.log(torch.rand((n, V), generator=g, device="cuda").clamp(1e-9, 1 - 1e-6)))).argmax(-1)
        temp, k, p, mp = (np.full(S, z) for z in (0.8, case["k"], case["p"], case["min_p"]))
        if case["mixed"]:
            temp = rs.choice([0.0, 0.6, 0.8, 1.0], S)
            k = np.where((p >= 1) | (rs.rand(S) < 0.5), k, 0)
            mp = mp * rs.choice([0, 1], S)
        st.update(x=x.to(getattr(torch, case["type"])), probs=q if case["probs"] else None, drafts=drafts.int(),
                  u=torch.rand(n, generator=g, device="cuda"), draws=torch.rand(S, generator=g, device="cuda"),
                  starts=_dev(starts, torch.int32), temperature=_dev(temp, torch.float32), top_k=_dev(k, torch.int32),
                  top_p=_dev(p, torch.float32), min_p=_dev(mp, torch.float32),
                  ids=torch.zeros(n, dtype=torch.int32, device="cuda"), accepted=torch.zeros(S, dtype=torch.int32, device="cuda"))
        if own:
            from mxfp4_mixture_experts_rms_gb300 import moe
            st["plan"] = moe.Verify(n)
    return st


# ---------------------------------------------------------------- the plain forms

def _rotate(s):
    c = s["case"]
    pairs = c["pairs"]
    turn = s["positions"].double()[s["axis"]].T * s["angle"]         # [tokens][pairs], in 64 bits: positions may be far
    turn = torch.remainder(turn, 2 * math.pi)
    cos, sin = turn.cos().float()[:, None], turn.sin().float()[:, None]
    done = []
    for x, gamma in ((s["q"], s["q_gamma"]), (s["k"], s["k_gamma"])):
        x = x.float()
        if gamma is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gamma
        if c["interleaved"]:
            a, b = x[..., 0:2 * pairs:2], x[..., 1:2 * pairs:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :pairs], x[..., pairs:2 * pairs]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        done.append(torch.cat([y, x[..., 2 * pairs:]], -1).to(torch.bfloat16))
    return dict(q=done[0], k=done[1])


def _parts(cache, c):
    """The cache's codes and scales as views: two of [pages][kv][D / 32][P][16], two of [pages][kv][D / 32][P]."""
    kv, D, P = c["kv"], c["dim"], c["page"]
    half, few = P * D // 2, P * D // 32
    codes = [cache[:, :, i * half:(i + 1) * half].view(-1, kv, D // 32, P, 16) for i in range(2)]
    return codes + [cache[:, :, 2 * half + i * few:2 * half + (i + 1) * few].view(-1, kv, D // 32, P) for i in range(2)]


def _rows_of(cache, c, page, off):
    """Keys and values [..., kv, D] in fp32 of the tokens at places `off` of pages `page`."""
    values = torch.tensor(_VALUES, device="cuda")
    place = torch.tensor(_PLACE, device="cuda")
    at = off // 16 * 16 + place[off % 16]
    kc, vc, ks, vs = _parts(cache, c)
    done = []
    for codes, scales in ((kc, ks), (vc, vs)):
        b = codes[page, :, :, off]                       # [..., kv, D / 32, 16]
        x = torch.stack([values[(b & 15).int()], values[(b >> 4).int()]], -1).flatten(-2)
        done.append((x * torch.exp2(scales[page, :, :, at].float() - 127)[..., None]).flatten(-2))
    return done


def _cache_rows(s):
    c = s["case"]
    kv, D, P = c["kv"], c["dim"], c["page"]
    slots = s["slots"].long()
    page, off = slots // P, slots % P
    place = torch.tensor(_PLACE, device="cuda")
    kc, vc, ks, vs = _parts(s["cache"], c)
    limits = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    for codes, scales, x in ((kc, ks, s["xk"]), (vc, vs, s["xv"])):
        x = x.float().view(-1, kv, D // 32, 32)
        e = torch.frexp(x.abs().amax(-1).clamp(min=6 * 2.0 ** -126))
        e = (e.exponent - 3 + (e.mantissa > 0.75)).clamp(max=125)         # ceil(log2(amax / 6))
        m = (x.abs() * torch.exp2(-e.float())[..., None]).contiguous()
        up = torch.bucketize(m, limits, right=True)                        # ties upwards
        code = torch.where(torch.bucketize(m, limits) % 2 == 0, torch.bucketize(m, limits), up)   # ties to the even code
        code = code + torch.where(x < 0, 8, 0)
        codes[page, :, :, off] = (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)
        scales[page, :, :, off // 16 * 16 + place[off % 16]] = (e + 127).to(torch.uint8)
    k, v = _rows_of(s["cache"], c, page, off)
    return dict(k=k.to(torch.bfloat16), v=v.to(torch.bfloat16))


def _attend(s):
    c = s["case"]
    P, kv, D, H, win, n = c["page"], c["kv"], c["dim"], c["heads"], c["window"], c["new"]
    G, S, W = H // kv, s["lens"].numel(), s["table"].shape[1]
    lens = s["lens"].long()
    starts = torch.arange(S + 1, device="cuda") if s["starts"] is None else s["starts"].long()
    new = starts[1:] - starts[:-1]
    i = torch.arange(n, device="cuda")[None]
    there = i < new[:, None]                              # rows of a padded batch that exist
    row = torch.where(there, starts[:-1, None] + i, 0)
    span = min(W * P, win + n - 1) if win else W * P
    lo = (lens - new - win + 1).clamp(min=0) if win else torch.zeros_like(lens)
    pos = lo[:, None] + torch.arange(span, device="cuda")
    page = s["table"].long().gather(1, (pos // P).clamp(max=W - 1))
    seen = (pos < lens[:, None]) & (pos // P < W) & (page >= 0)
    k, v = _rows_of(s["cache"], c, torch.where(seen, page, 0), pos % P)
    v = torch.where(seen[:, :, None, None], v, 0.0)
    q = s["q"].float()[row].view(S, n, kv, G, D)
    at = (lens - new)[:, None] + torch.arange(n, device="cuda")
    ok = seen[:, None] & (pos[:, None] <= at[:, :, None])
    if win:
        ok = ok & (pos[:, None] > at[:, :, None] - win)
    x = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(S, kv, G * n, D), k.permute(0, 2, 3, 1)) / math.sqrt(D)
    x = torch.where(ok[:, None, None], x.view(S, kv, G, n, span), -math.inf)
    top = x.amax(-1, keepdim=True)
    sink = None if s["sinks"] is None else s["sinks"].view(1, kv, G, 1, 1)
    if sink is not None:
        top = torch.maximum(top, sink)
    top = torch.where(top == -math.inf, 0.0, top)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    if sink is not None:
        total = total + torch.exp(sink - top)
    o = torch.matmul(x.view(S, kv, G * n, span), v.permute(0, 2, 1, 3)).view(S, kv, G, n, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(S, n, H, D)
    out = torch.zeros((s["q"].shape[0] + 1, H, D), dtype=torch.bfloat16, device="cuda")
    out[torch.where(there, row, out.shape[0] - 1)] = o.to(torch.bfloat16)
    return out[:-1]


def _target(s, of):
    """Probabilities (64 bits) from which each row's token is drawn: temperature, top-k, top-p, min-p."""
    x = s["x"].double()
    x = torch.where(torch.isnan(x), -math.inf, x)
    top = x.amax(-1, keepdim=True)
    t, k, p, mp = (s[n][of][:, None] for n in ("temperature", "top_k", "top_p", "min_p"))
    t, k, p, mp = t.double(), k.long(), p.double(), mp.double()
    w = torch.where(x == top, 1.0, torch.where(t > 0, torch.exp((x - top) / torch.where(t > 0, t, 1.0)), 0.0))
    w = torch.where(x == -math.inf, 0.0, w)
    V = x.shape[1]
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    k = torch.where(t > 0, torch.where((k <= 0) | (k > V), V, k), 1)
    ws = torch.where(torch.arange(V, device="cuda")[None] < k, ws, 0.0)
    before = ws.cumsum(-1) - ws
    keep = (ws > 0) & ((p >= 1) | (before < p * ws.sum(-1, keepdim=True))) & (ws >= mp)
    keep[:, 0] = ws[:, 0] > 0
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, ws, 0.0))
    total = w.sum(-1, keepdim=True)
    return torch.where(total > 0, w / total, 0.0)


def _verify(s):
    starts = s["starts"].long()
    n, V = s["x"].shape
    S = starts.numel() - 1
    row = torch.arange(n, device="cuda")
    of = torch.searchsorted(starts[1:], row, right=True)                  # each row's sequence
    p = _target(s, of)
    last = row == starts[1:][of] - 1
    d = s["drafts"].long()
    q = torch.zeros_like(p).scatter_(1, d[:, None], 1.0) if s["probs"] is None else s["probs"].double()
    q = torch.where(last[:, None], 0.0, q)
    px, qx = p.gather(1, d[:, None])[:, 0], q.gather(1, d[:, None])[:, 0]
    ok = ~last & (s["u"].double() * qx < px)
    # of each sequence: the first row that is not accepted
    stop = torch.full((S,), n, device="cuda").scatter_reduce(0, of, torch.where(ok, n, row), "amin")
    rest = (p[stop] - q[stop]).clamp(min=0)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, p[stop])
    c = rest.cumsum(-1)
    pick = (c <= s["draws"].double()[:, None] * c[:, -1:]).sum(-1)
    pick = torch.minimum(pick, torch.where(rest > 0, torch.arange(V, device="cuda")[None], -1).amax(-1))
    at = stop[of]
    ids = torch.where(row < at, d, torch.where(row == at, pick[of], -1))
    return dict(ids=ids.int(), accepted=(stop - starts[:-1]).int())


def _own(s):
    c = s["case"]
    if c["op"] == "rotate":
        s["plan"].apply(s["q"], s["k"], s["positions"], s["q_out"], s["k_out"])
        return dict(q=s["q_out"], k=s["k_out"])
    if c["op"] == "cache":
        s["plan"].append(s["xk"], s["xv"], s["slots"])
        s["plan"].read(s["slots"], s["k_out"], s["v_out"])
        return dict(k=s["k_out"], v=s["v_out"])
    if c["op"] == "attend":
        s["plan"].attend(s["q"], s["lens"], s["table"], s["out"], starts=s["starts"], max_new=c["new"])
        return s["out"]
    s["plan"].run(s["x"], s["drafts"], s["u"], s["draws"], s["starts"], s["ids"], s["accepted"], draft_probs=s["probs"],
                  temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
    return dict(ids=s["ids"], accepted=s["accepted"])


def run(state):
    if own:
        return _own(state)
    return dict(rotate=_rotate, cache=_cache_rows, attend=_attend, verify=_verify)[state["case"]["op"]](state)


# ---------------------------------------------------------------- work

def work(case):
    """Averages where lengths are drawn (each uniform over its range)."""
    if case["op"] == "rotate":
        n = case["tokens"] * (case["heads"] + case["kv"]) * case["dim"]
        return dict(bytes=4 * n + 4 * case["axes"] * case["tokens"], flops=(6 if case["norm"] else 3) * n)
    if case["op"] == "cache":
        tok = case["seqs"] * 0.75 * max(1, case["new"])
        # read, written as codes and scales, those read again, written
        return dict(bytes=tok * (case["kv"] * case["dim"] * 2 * (4 + 17 / 16) + 8), flops=4 * tok * case["kv"] * case["dim"])
    if case["op"] == "attend":
        S, n, ctx, D = case["seqs"], case["new"], case["ctx"], case["dim"]
        if case["ragged"]:
            n = max(1, n * 2 / 3)
            ctx = (n * n + ctx * ctx) / (2 * ctx)
        pairs = n * (min(ctx, case["window"]) if case["window"] else ctx - (n - 1) / 2)
        seen = min(ctx, case["window"] + n - 1) if case["window"] else ctx
        return dict(bytes=S * (seen * case["kv"] * D * 17 / 16 + n * case["heads"] * D * 4),
                    flops=4 * S * pairs * case["heads"] * D)
    size = 4 if case["type"] == "float32" else 2
    rows = case["seqs"] * (case["drafts"] + 0.5)
    # the logits of every row, the draft's probabilities of one row a sequence
    return dict(bytes=(rows * size + (4 * case["seqs"] if case["probs"] else 0)) * case["vocab"], flops=3 * rows * case["vocab"])


# ---------------------------------------------------------------- from the definitions, in 64 bits

def _exact_rotate(case, s):
    n, pairs = case["tokens"], case["pairs"]
    pos, freqs = s["positions"].cpu().numpy().astype(np.float64), s["freqs"]
    a = np.stack([pos[s["of"][i]] * freqs[i] for i in range(pairs)], 1)
    cos, sin = _dev(np.cos(a)).view(n, 1, pairs), _dev(np.sin(a)).view(n, 1, pairs)
    out = {}
    for name in ("q", "k"):
        y = s[name].double().clone()
        if s[name + "_gamma"] is not None:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / case["dim"] + 1e-6) * s[name + "_gamma"].double()
        first = slice(0, 2 * pairs, 2) if case["interleaved"] else slice(0, pairs)
        second = slice(1, 2 * pairs, 2) if case["interleaved"] else slice(pairs, 2 * pairs)
        a, b = y[..., first].clone(), y[..., second].clone()
        y[..., first] = cos * a - sin * b
        y[..., second] = sin * a + cos * b
        out[name] = y
    return out


def _exact_block(x):
    """Blocks [..., 32] (float64): the values they stand for in E2M1 with an E8M0 scale."""
    a = x.abs().amax(-1, keepdim=True).clamp(min=6 * 2.0 ** -126)
    k = torch.ceil(torch.log2(a / 6))
    k = torch.where(6 * torch.exp2(k - 1) >= a, k - 1, k)                  # where log2 rounded up
    k = torch.where(6 * torch.exp2(k) < a, k + 1, k).clamp(-126, 125)      # or down
    m = (x.abs() * torch.exp2(-k)).clamp(max=6.0)
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    return torch.copysign(torch.round(m / step) * step * torch.exp2(k), x)


def _exact_attend(case, s):
    P, kv, D, H, win = case["page"], case["kv"], case["dim"], case["heads"], case["window"]
    lens, table = s["lens"].tolist(), s["table"]
    starts = list(range(len(lens) + 1)) if s["starts"] is None else s["starts"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    nibble = torch.tensor(_VALUES, dtype=torch.float64, device="cuda")
    order = sorted(range(16), key=lambda t: _PLACE[t])
    back = torch.tensor([order.index(t) for t in range(16)], device="cuda")
    for b, L in enumerate(lens):
        a, z = starts[b], starts[b + 1]
        lo = max(0, L - (z - a) - win + 1) // P if win else 0
        page = s["cache"][table[b, lo:-(-L // P)].long()]                  # [pages][kv][bytes]
        n, half, few = page.shape[0], P * D // 2, P * D // 32
        both = []
        for side in range(2):
            codes = page[:, :, side * half:(side + 1) * half].reshape(n, kv, D // 32, P, 16)
            scale = page[:, :, 2 * half + side * few:2 * half + (side + 1) * few].reshape(n, kv, D // 32, P // 16, 16)[..., back]
            x = torch.empty((n, kv, D // 32, P, 32), dtype=torch.float64, device="cuda")
            x[..., 0::2], x[..., 1::2] = nibble[(codes % 16).long()], nibble[(codes // 16).long()]
            x *= torch.exp2(scale.reshape(n, kv, D // 32, P, 1).double() - 127)
            both.append(x.permute(0, 3, 1, 2, 4).reshape(n * P, kv, D))
        k, v = both
        kp = lo * P + torch.arange(n * P, device="cuda")
        qp = L - (z - a) + torch.arange(z - a, device="cuda")
        hide = kp[None] > qp[:, None]
        if win:
            hide |= kp[None] <= qp[:, None] - win
        for h in range(H):
            x = s["q"][a:z, h].double() @ k[:, h // (H // kv)].T / math.sqrt(D)
            x = x.masked_fill(hide, -math.inf)
            if s["sinks"] is not None:
                x = torch.cat([x, s["sinks"][h].double().expand(z - a, 1)], 1)
            out[a:z, h] = torch.softmax(x, -1)[:, :n * P] @ v[:, h // (H // kv)]
    return out


def exact(case, seed):
    if case["op"] == "verify":
        return None   # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "rotate":
        return _exact_rotate(case, s)
    if case["op"] == "cache":
        blocks = lambda x: x.double().reshape(x.shape[0], case["kv"], -1, 32)   # noqa: E731
        return {n: _exact_block(blocks(x)).reshape(x.shape) for n, x in (("k", s["xk"]), ("v", s["xv"]))}
    return _exact_attend(case, s)
