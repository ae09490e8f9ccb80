"""The serving operators' workloads: page tables, the 8-bit paged key/value cache (append and
attention) and sampling.  Each case is one call as a serving loop makes it; `run` computes it in
plain torch operations, or through the framework's own entry points where `own` is true.

Cache layout (both sides read and write the same bytes): codes are E4M3; per page of P tokens and
kv head, keys as [D / 16][P][16] (16 consecutive dims of a token together) and values as
[P / 16][D][16], token 2 t + e of 16 (t < 4, e < 2) at byte 4 t + e and token 8 + 2 t + e at byte
4 t + 2 + e; one E8M0 scale byte per page and kv head, value 2^(s - 127).
"""
import math
import zlib

import numpy as np
import torch

own = False

# Shapes: gpt-oss attention (64 query heads, 8 kv heads, dims of 64, window 128 on alternate
# layers) as this repository's benchmark has it, and generic ones with dims of 128.


def listed():
    return [
        # one decode step of a small server: 64 requests, one token each, a few cross into a new page, some finish
        dict(name="pages_decode_64", op="pages", seqs=64, page=16, ctx=4096, new=1, done=4),
        # admission of a large ragged batch: prompts and running requests together
        dict(name="pages_ragged_2048", op="pages", seqs=2048, page=16, ctx=8192, new=600, done=100),
        # one decode step's keys and values of 48 sequences into partly filled pages
        dict(name="append_decode_48", op="append", seqs=48, kv=8, dim=64, page=16, ctx=900, new=1),
        # ragged prompts' keys and values, pages that begin and end inside them
        dict(name="append_prompts_16k", op="append", seqs=21, kv=8, dim=128, page=32, ctx=300, new=1500),
        # the smallest call: one request, short context, a sliding and sink layer's shape
        dict(name="attend_one_131", op="attend", seqs=1, heads=64, kv=8, dim=64, page=16, ctx=131, new=1, window=0,
             sinks=True, ragged=False),
        # the repository's own decode workload: 16 sequences with 4096 visible tokens, full layer
        dict(name="attend_decode_16x4096", op="attend", seqs=16, heads=64, kv=8, dim=64, page=64, ctx=4096, new=1,
             window=0, sinks=True, ragged=False),
        # its sliding layer: 128 tokens of long contexts
        dict(name="attend_window_32x8191", op="attend", seqs=32, heads=64, kv=8, dim=64, page=16, ctx=8191, new=1,
             window=128, sinks=True, ragged=False),
        # a ragged batch with dims of 128 and an odd number of query heads per kv head
        dict(name="attend_ragged_96_d128", op="attend", seqs=96, heads=20, kv=4, dim=128, page=32, ctx=12000, new=1,
             window=0, sinks=False, ragged=True),
        # ragged prompts attending over what is cached before them and themselves
        dict(name="attend_prompts_3x1024", op="attend", seqs=3, heads=64, kv=8, dim=64, page=64, ctx=2900, new=1024,
             window=0, sinks=True, ragged=True),
        # one interactive request: fp32 logits of a 32 K vocabulary, top-k and top-p
        dict(name="sample_one_32k", op="sample", rows=1, vocab=32001, type="float32", k=50, p=0.95, min_p=0.0, mixed=False),
        # a decode batch: fp32 logits of a 200 K vocabulary, nucleus only
        dict(name="sample_16x200k", op="sample", rows=16, vocab=200000, type="float32", k=0, p=0.9, min_p=0.0, mixed=False),
        # a large batch of requests with settings of their own, bf16 logits (many equal)
        dict(name="sample_256x128k_mixed", op="sample", rows=256, vocab=128000, type="bfloat16", k=100, p=0.95,
             min_p=0.02, mixed=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "append", "attend", "attend", "sample"])
    if op == "pages":
        seqs = _log(rng, 1, 2048)
        return dict(op=op, seqs=seqs, page=rng.choice([16, 32, 64]), ctx=_log(rng, 1, 8192),
                    new=_log(rng, 1, 600), done=rng.randrange(0, seqs // 2 + 1))
    if op == "append":
        new = _log(rng, 1, 1500)
        return dict(op=op, seqs=_log(rng, 1, 64 if new < 100 else 20), kv=rng.choice([1, 2, 3, 4, 8]),
                    dim=rng.choice([64, 128]), page=rng.choice([16, 32, 64]), ctx=_log(rng, 1, 1000), new=new)
    if op == "attend":
        kv, group, dim = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 5, 7, 8, 12, 16]), rng.choice([64, 128])
        new = 1 if rng.random() < 0.6 else _log(rng, 2, 700)
        ctx = max(new, _log(rng, 1, 12000 if new == 1 else 2500))
        most = (96 * 12000 * 4 * 128) // (ctx * kv * dim) if new == 1 else 1200 * 64 * 2500 // (new * kv * group * ctx)
        return dict(op=op, seqs=_log(rng, 1, max(1, min(128, most))), heads=kv * group, kv=kv, dim=dim,
                    page=rng.choice([16, 32, 64]), ctx=ctx, new=new, window=rng.choice([0, 0, 1, 100, 128, 1000]),
                    sinks=rng.random() < 0.5, ragged=rng.random() < 0.7)
    rows = _log(rng, 1, 256)
    return dict(op=op, rows=rows, vocab=_log(rng, 2, min(260000, 256 * 128000 // rows)),
                type=rng.choice(["float32", "bfloat16"]), k=rng.choice([0, 1, 20, 1000]),
                p=rng.choice([1.0, 0.95, 0.8, 0.3]), min_p=rng.choice([0.0, 0.0, 0.05]), mixed=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs

_PLACE = [0, 1, 8, 9, 2, 3, 10, 11, 4, 5, 12, 13, 6, 7, 14, 15]   # token at each byte of a value block
_BYTE = [_PLACE.index(i) for i in range(16)]                       # byte of each token


def _lengths(case, rs):
    """(cached or visible tokens, new tokens) of each sequence, on the host: the same lengths for
    every seed, so that outputs keep their shapes, in an order of the seed's own."""
    n, S = case["new"], case["seqs"]
    fixed = np.random.RandomState(zlib.crc32(repr(sorted((k, v) for k, v in case.items() if k != "name")).encode()))
    if case["op"] == "pages":
        have, new = fixed.randint(0, case["ctx"] + 1, S), fixed.randint(1, n + 1, S)
        new[:case["done"]] = -1
    elif case["op"] == "append":
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
    """A filled cache: codes and scales of normally distributed keys and values."""
    kv, D, P = case["kv"], case["dim"], case["page"]
    made = []
    for spread in (1.5, 1.0):
        x = torch.randn((pages, kv, P * D), generator=g, device="cuda") * spread
        s = torch.randint(0, 3, (pages, kv), generator=g, device="cuda")   # pages differ in size
        x = x * torch.exp2(s.float())[:, :, None]
        e = torch.ceil(torch.log2(x.abs().amax(-1) / 448))
        codes = (x / torch.exp2(e)[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        made += [codes, (e + 127).to(torch.uint8)]
        del x
    return made[0], made[2], made[1], made[3]


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
    if case["op"] == "pages":
        S, P = case["seqs"], case["page"]
        cached, fresh = _lengths(case, rs)
        W = -(-(case["ctx"] + case["new"]) // P)
        held = -(-cached // P)
        t, used = _tables(held, W, rs)
        pool = used + int((-(-(cached + np.maximum(fresh, 0)) // P) - held).sum()) + 17
        free = np.full(pool, -1, np.int32)
        rest = rs.permutation(np.arange(used, pool)).astype(np.int32)
        free[:len(rest)] = rest
        tokens = int(np.maximum(fresh, 0).sum()) + 3
        st.update(cached=_dev(cached, torch.int32), fresh=_dev(fresh, torch.int32), table=_dev(t), free=_dev(free),
                  counts=_dev(np.array([len(rest), 0], np.int32)),
                  counts_out=torch.zeros(2, dtype=torch.int32, device="cuda"),
                  starts=torch.zeros(S + 1, dtype=torch.int32, device="cuda"),
                  lens=torch.zeros(S, dtype=torch.int32, device="cuda"),
                  slots=torch.zeros(tokens, dtype=torch.int32, device="cuda"),
                  positions=torch.zeros(tokens, dtype=torch.int32, device="cuda"))
    elif case["op"] == "append":
        S, P, kv, D = case["seqs"], case["page"], case["kv"], case["dim"]
        cached, new = _lengths(case, rs)
        per = -(-(cached + new) // P)
        t, pages = _tables(per, int(per.max()), rs)
        k, v, ks, vs = _cache(pages, case, g)
        n = int(new.sum())
        seq = np.repeat(np.arange(S), new)
        pos = np.concatenate([cached[b] + np.arange(new[b]) for b in range(S)])
        slots = t[seq, pos // P] * P + pos % P
        # keys and values as slices of one projection's rows
        both = torch.randn((n, 2 * kv, D), generator=g, device="cuda")
        both *= 1 + 3 * torch.rand((n, 1, 1), generator=g, device="cuda")
        both = both.to(torch.bfloat16)
        st.update(k=k, v=v, ks=ks, vs=vs, slots=_dev(slots, torch.int32), xk=both[:, :kv], xv=both[:, kv:])
        if own:
            from mxfp4_mixture_experts_rms_gb300 import moe
            st["plan"] = moe.Kv8(kv, kv, D, P, pages, cache=(k, v, ks, vs))
    elif case["op"] == "attend":
        S, P, kv, D, QH = case["seqs"], case["page"], case["kv"], case["dim"], case["heads"]
        vis, new = _lengths(case, rs)
        per = -(-vis // P)
        t, pages = _tables(per, -(-case["ctx"] // P), rs)
        k, v, ks, vs = _cache(pages, case, g)
        n = int(new.sum())
        q = (torch.randn((n, QH, D), generator=g, device="cuda") * 0.7).to(torch.bfloat16)
        sinks = torch.randn(QH, generator=g, device="cuda") if case["sinks"] else None
        st.update(k=k, v=v, ks=ks, vs=vs, q=q, sinks=sinks, table=_dev(t), lens=_dev(vis, torch.int32),
                  starts=None if case["new"] == 1 else _dev(np.concatenate([[0], np.cumsum(new)]), torch.int32),
                  out=torch.zeros_like(q))
        if own:
            from mxfp4_mixture_experts_rms_gb300 import moe
            st["plan"] = moe.Kv8(QH, kv, D, P, pages, sliding_window=case["window"], sinks=sinks, cache=(k, v, ks, vs))
    else:
        R, V = case["rows"], case["vocab"]
        x = torch.randn((R, V), generator=g, device="cuda") * 2.5
        x[:, :: max(1, V // 40)] += 6.0 * torch.rand((R, len(range(0, V, max(1, V // 40)))), generator=g, device="cuda")
        temp, k, p, mp = (np.full(R, z) for z in (0.8, case["k"], case["p"], case["min_p"]))
        if case["mixed"]:
            temp = rs.choice([0.0, 0.6, 1.0, 1.3], R)
            k = k * rs.choice([0, 1], R)
            p = np.where(rs.rand(R) < 0.5, p, 1.0)
            mp = mp * rs.choice([0, 1], R)
        st.update(x=x.to(getattr(torch, case["type"])), u=torch.rand(R, generator=g, device="cuda"),
                  temperature=_dev(temp, torch.float32), top_k=_dev(k, torch.int32), top_p=_dev(p, torch.float32),
                  min_p=_dev(mp, torch.float32), ids=torch.zeros(R, dtype=torch.int32, device="cuda"))
    return st


# ---------------------------------------------------------------- the plain forms

def _pages(s):
    c = s["case"]
    P, (S, W) = c["page"], s["table"].shape
    cached, fresh = s["cached"].long(), s["fresh"].long()
    gone, new = fresh < 0, fresh.clamp(min=0)
    held = ((cached + P - 1) // P).clamp(max=W)
    j = torch.arange(W, device="cuda")[None]
    back = gone[:, None] & (j < held[:, None]) & (s["table"] >= 0)
    at = torch.where(back.flatten(), s["counts"][0] + back.flatten().cumsum(0) - 1, s["free"].numel())
    free = torch.cat([s["free"], s["free"].new_zeros(1)]).scatter_(0, at, s["table"].flatten())[:-1]
    n1 = s["counts"][0] + back.sum()
    want = torch.where(gone, 0, ((cached + new + P - 1) // P).clamp(max=W) - held)
    src = n1 - 1 - ((want.cumsum(0) - want)[:, None] + j - held[:, None])
    page = torch.where(src >= 0, free[src.clamp(0, free.numel() - 1)], -1)
    table = torch.where((j >= held[:, None]) & (j < (held + want)[:, None]), page, s["table"])
    ends = new.cumsum(0)
    starts = torch.cat([ends.new_zeros(1), ends])
    tok = torch.arange(s["slots"].numel(), device="cuda")
    b = torch.searchsorted(ends, tok, right=True).clamp(max=S - 1)
    pos = cached[b] + tok - starts[b]
    pg = table[b, (pos // P).clamp(0, W - 1)].long()
    live = tok < ends[-1]
    slots = torch.where(live & (pos // P < W) & (pg >= 0), pg * P + pos % P, -1)
    left = n1 - want.sum()
    return dict(table=table.int(), free=free, counts=torch.stack([left.clamp(min=0), (-left).clamp(min=0)]).int(),
                starts=starts.int(), lens=torch.where(gone, 0, cached + new).int(), slots=slots.int(),
                positions=torch.where(live, pos, -1).int())


def _append(s):
    c = s["case"]
    P, kv, D = c["page"], c["kv"], c["dim"]
    page, off = s["slots"].long() // P, s["slots"].long() % P
    pages = s["ks"].shape[0]
    first = torch.full((pages,), P, device="cuda", dtype=torch.long).scatter_reduce(0, page, off, "amin")[page]
    tok = torch.arange(P, device="cuda")
    # index of (token of the page, kv head, dim) in a page's bytes
    h, d = torch.arange(kv, device="cuda")[:, None], torch.arange(D, device="cuda")[None]
    at_k = (h * P * D + d // 16 * P * 16 + d % 16)[None] + (tok * 16)[:, None, None]
    byte = torch.tensor(_BYTE, device="cuda")
    at_v = (h * P * D + d * 16)[None] + (tok // 16 * D * 16 + byte[tok % 16])[:, None, None]
    done = []
    for codes, scale, x, at in ((s["k"], s["ks"], s["xk"], at_k), (s["v"], s["vs"], s["xv"], at_v)):
        x = x.float()
        amax = x.abs().amax(-1).clamp(min=448 * 2.0 ** -126)
        e = torch.frexp(amax / 448)
        e = torch.where(e.mantissa == 0.5, e.exponent - 1, e.exponent) + 127
        most = torch.zeros((pages, kv), device="cuda", dtype=e.dtype).scatter_reduce(0, page[:, None].expand(-1, kv), e, "amax")[page]
        old = scale[page].to(e.dtype)
        now = torch.where(first[:, None] > 0, torch.maximum(most, old), most)
        flat = codes.view(pages, -1)
        had = flat[page[:, None, None, None], at[None]]
        was = had.view(torch.float8_e4m3fn).float() * torch.exp2((old - now).float())[:, None, :, None]
        was = torch.where((tok < first[:, None])[:, :, None, None], was.to(torch.float8_e4m3fn).view(torch.uint8), had)
        flat[page[:, None, None, None], at[None]] = was
        flat[page[:, None, None], at[off]] = (x * torch.exp2(127 - now.float())[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scale[page] = now.to(torch.uint8)
        done.append((flat, scale))
    return _held(s)


def _held(s):
    return dict(k=s["k"].view(torch.float8_e4m3fn), v=s["v"].view(torch.float8_e4m3fn), ks=s["ks"], vs=s["vs"])


def _rows(s):
    """(token of each sequence's row, rows of a padded batch that exist, row index)."""
    c, n = s["case"], s["case"]["new"]
    S = s["lens"].numel()
    starts = torch.arange(S + 1, device="cuda") if s["starts"] is None else s["starts"].long()
    new = starts[1:] - starts[:-1]
    i = torch.arange(n, device="cuda")[None]
    there = i < new[:, None]
    return new, there, torch.where(there, starts[:-1, None] + i, 0)


def _attend(s):
    c = s["case"]
    P, kv, D, QH, win = c["page"], c["kv"], c["dim"], c["heads"], c["window"]
    G, S, W = QH // kv, s["lens"].numel(), s["table"].shape[1]
    lens = s["lens"].long()
    new, there, row = _rows(s)
    n = row.shape[1]
    span = min(W * P, win + n - 1) if win else W * P
    lo = (lens - new - win + 1).clamp(min=0) if win else torch.zeros_like(lens)
    pos = lo[:, None] + torch.arange(span, device="cuda")
    page = s["table"].long().gather(1, (pos // P).clamp(max=W - 1))
    seen = (pos < lens[:, None]) & (pos // P < W) & (page >= 0)
    page, off = torch.where(seen, page, 0), pos % P
    k = s["k"].view(-1, kv, D // 16, P, 16)[page, :, :, off].reshape(S, span, kv, D)
    byte = torch.tensor(_BYTE, device="cuda")
    v = s["v"].view(-1, kv, P // 16, D, 16)[page, :, off // 16, :, byte[off % 16]]
    k = k.view(torch.float8_e4m3fn).float() * torch.exp2(s["ks"][page].float() - 127)[..., None]
    v = v.view(torch.float8_e4m3fn).float() * torch.exp2(s["vs"][page].float() - 127)[..., None]
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
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(S, n, QH, D)
    out = torch.zeros((s["q"].shape[0] + 1, QH, D), dtype=torch.bfloat16, device="cuda")
    out[torch.where(there, row, out.shape[0] - 1)] = o.to(torch.bfloat16)
    return out[:-1]


def _sample(s):
    x = s["x"].double()
    x = torch.where(torch.isnan(x), -math.inf, x)
    top = x.amax(-1, keepdim=True)
    t = s["temperature"].double()[:, None]
    w = torch.where(x == top, 1.0, torch.where(t > 0, torch.exp((x - top) / torch.where(t > 0, t, 1.0)), 0.0))
    w = torch.where(x == -math.inf, 0.0, w)
    V = x.shape[1]
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    k = s["top_k"].long()[:, None]
    k = torch.where(t > 0, torch.where((k <= 0) | (k > V), V, k), 1)
    ws = torch.where(torch.arange(V, device="cuda")[None] < k, ws, 0.0)
    before = ws.cumsum(-1) - ws
    p = s["top_p"].double()[:, None]
    keep = (ws > 0) & ((p >= 1) | (before < p * ws.sum(-1, keepdim=True))) & (ws >= s["min_p"].double()[:, None])
    keep[:, 0] = ws[:, 0] > 0
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, ws, 0.0))
    c = w.cumsum(-1)
    pick = (c <= s["u"].double()[:, None] * c[:, -1:]).sum(-1)
    last = torch.where(w > 0, torch.arange(V, device="cuda")[None], -1).amax(-1)
    return torch.minimum(pick, last).int()


def _own(s):
    from mxfp4_mixture_experts_rms_gb300 import moe
    op = s["case"]["op"]
    if op == "pages":
        moe.pages_assign(s["case"]["page"], s["cached"], s["fresh"], s["free"], s["counts"], s["counts_out"], s["table"],
                         s["starts"], s["lens"], s["slots"], s["positions"])
        return dict(table=s["table"], free=s["free"], counts=s["counts_out"], starts=s["starts"], lens=s["lens"],
                    slots=s["slots"], positions=s["positions"])
    if op == "append":
        s["plan"].append(s["xk"], s["xv"], s["slots"])
        return _held(s)
    if op == "attend":
        s["plan"].attend(s["q"], s["lens"], s["table"], s["out"], starts=s["starts"], max_new=s["case"]["new"])
        return s["out"]
    moe.sample(s["x"], s["u"], s["ids"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
               min_p=s["min_p"])
    return s["ids"]


def run(state):
    if own:
        return _own(state)
    return dict(pages=_pages, append=_append, attend=_attend, sample=_sample)[state["case"]["op"]](state)


# ---------------------------------------------------------------- work

def work(case):
    """Averages where lengths are drawn (each uniform over its range)."""
    if case["op"] == "pages":
        S, P = case["seqs"], case["page"]
        tok = (S - case["done"]) * (case["new"] + 1) / 2
        back = case["done"] * (case["ctx"] / 2 / P + 0.5)
        return dict(bytes=S * 8 + 8 * tok + tok / P * 8 + back * 8 + 8 * S, flops=0)
    if case["op"] == "append":
        tok = case["seqs"] * 0.75 * max(1, case["new"])
        return dict(bytes=tok * (case["kv"] * case["dim"] * 2 * 3 + 4) + tok / case["page"] * case["kv"] * 2, flops=0)
    if case["op"] == "attend":
        S, n, ctx, D = case["seqs"], case["new"], case["ctx"], case["dim"]
        if case["ragged"]:
            n = max(1, n * 2 / 3)
            ctx = (n * n + ctx * ctx) / (2 * ctx)
        pairs = n * (min(ctx, case["window"]) if case["window"] else ctx - (n - 1) / 2)
        seen = min(ctx, case["window"] + n - 1) if case["window"] else ctx
        return dict(bytes=S * (seen * case["kv"] * D * 2 + n * case["heads"] * D * 4),
                    flops=4 * S * pairs * case["heads"] * D)
    size = 4 if case["type"] == "float32" else 2
    return dict(bytes=case["rows"] * (case["vocab"] * size + 24), flops=3 * case["rows"] * case["vocab"])


# ---------------------------------------------------------------- from the definitions, in 64 bits

def _round8(x):
    """To the nearest value of E4M3, ties to even; |x| at most 448."""
    e = (torch.frexp(x.abs().clamp(min=2.0 ** -30)).exponent - 1).clamp(min=-6).double()
    q = torch.exp2(e - 3)
    return torch.round(x / q) * q


def _unpack(s, case):
    """Codes' values (float64) as [pages][token][kv][dim], keys and values."""
    P, kv, D = case["page"], case["kv"], case["dim"]
    k = s["k"].view(torch.float8_e4m3fn).double().view(-1, kv, D // 16, P, 16).permute(0, 3, 1, 2, 4).reshape(-1, P, kv, D)
    v = s["v"].view(torch.float8_e4m3fn).double().view(-1, kv, P // 16, D, 16)
    v = v[..., _BYTE].permute(0, 2, 4, 1, 3).reshape(-1, P, kv, D)
    return k, v


def _exact_append(case, s):
    P, kv, D = case["page"], case["kv"], case["dim"]
    slots = s["slots"].cpu().numpy()
    k, v = _unpack(s, case)
    done = {}
    order = np.argsort(slots, kind="stable")
    for name, vals, scale, x in (("k", k, s["ks"], s["xk"].double()), ("v", v, s["vs"], s["xv"].double())):
        sc = scale.double() - 127
        at = 0
        while at < len(order):   # the tokens of one page
            pg, to = slots[order[at]] // P, at
            while to < len(order) and slots[order[to]] // P == pg:
                to += 1
            t = torch.from_numpy(order[at:to]).cuda()
            first, y = int(slots[order[at]] % P), x[t]
            a = y.abs().amax((0, 2))
            e = torch.ceil(torch.log2(a / 448)).clamp(min=-126)
            e = torch.where(448 * torch.exp2(e - 1) >= a, e - 1, e).clamp(min=-126)   # where log2 rounded up
            if first:
                e = torch.maximum(e, sc[pg])
                vals[pg, :first] = _round8(vals[pg, :first] * torch.exp2(sc[pg] - e)[None, :, None])
            vals[pg, first:first + len(t)] = _round8(y * torch.exp2(-e)[None, :, None])
            sc[pg] = e
            at = to
        done[name + "s"] = sc + 127
        if name == "k":
            done[name] = vals.view(-1, P, kv, D // 16, 16).permute(0, 2, 3, 1, 4).reshape(-1, kv, P * D)
        else:
            done[name] = vals.view(-1, P // 16, 16, kv, D)[:, :, _PLACE].permute(0, 3, 1, 4, 2).reshape(-1, kv, P * D)
    return dict(k=done["k"], v=done["v"], ks=None, vs=None)


def _exact_attend(case, s):
    P, kv, D, QH, win = case["page"], case["kv"], case["dim"], case["heads"], case["window"]
    lens, table = s["lens"].tolist(), s["table"]
    starts = list(range(len(lens) + 1)) if s["starts"] is None else s["starts"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, L in enumerate(lens):
        a, z = starts[b], starts[b + 1]
        lo = max(0, L - (z - a) - win + 1) // P if win else 0
        pg = table[b, lo:-(-L // P)].long()
        k, v = _unpack(dict(k=s["k"][pg], v=s["v"][pg]), case)
        k = (k * torch.exp2(s["ks"][pg].double() - 127)[:, None, :, None]).reshape(-1, kv, D)
        v = (v * torch.exp2(s["vs"][pg].double() - 127)[:, None, :, None]).reshape(-1, kv, D)
        kp = lo * P + torch.arange(k.shape[0], device="cuda")
        qp = L - (z - a) + torch.arange(z - a, device="cuda")
        hide = kp[None] > qp[:, None]
        if win:
            hide |= kp[None] <= qp[:, None] - win
        for h in range(QH):
            x = s["q"][a:z, h].double() @ k[:, h // (QH // kv)].T / math.sqrt(D)
            x = x.masked_fill(hide, -math.inf)
            if s["sinks"] is not None:
                x = torch.cat([x, s["sinks"][h].double().expand(z - a, 1)], 1)
            out[a:z, h] = torch.softmax(x, -1)[:, :k.shape[0]] @ v[:, h // (QH // kv)]
    return out


def exact(case, seed):
    if case["op"] == "append":
        return _exact_append(case, prepare(case, seed))
    if case["op"] == "attend":
        return _exact_attend(case, prepare(case, seed))
    return None   # whole numbers only
