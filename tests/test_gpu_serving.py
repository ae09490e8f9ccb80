"""The serving operators on the GPU against oracle/serving.py (64 bits): page tables, the 8-bit paged
cache's append, the attention over it, sampling, and a run of them together.

Tolerances.  Page tables and codes are whole numbers: equal.  Attention: oracle.serving.attend gives with each
output how far it may be off, from the roundings' sizes.  Sampling: a weight e^z, z <= 0, is off by at most
(2^-22 + |z| 2^-22) of itself, and |z| e^z <= 0.37, so running sums are within 2^-20 of the total; the token
must be one whose interval of the running sum, widened by 2^-18 of the total, holds u times the total."""
import numpy as np
import pytest

from oracle import serving as S

pytestmark = pytest.mark.gpu


def moe():
    from mxfp4_mixture_experts_rms_gb300 import moe as m
    return m


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(x):
    """x rounded to bf16: the tensor on the GPU, and its values."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


# ---------------------------------------------------------------- page tables

def run_pages(P, cached, fresh, free, n_free, table, max_tokens, in_place=False):
    import torch
    n = len(cached)
    t = dict(free=dev(np.asarray(free, np.int32)), table=dev(np.asarray(table, np.int32)))
    counts = dev(np.array([n_free, 77], np.int32))
    out = counts if in_place else torch.full((2,), 99, dtype=torch.int32, device="cuda")
    z = lambda k: torch.full((k,), 12345, dtype=torch.int32, device="cuda")   # noqa: E731
    starts, lens, slots, pos = z(n + 1), z(n), z(max_tokens), z(max_tokens)
    moe().pages_assign(P, dev(np.asarray(cached, np.int32)), dev(np.asarray(fresh, np.int32)), t["free"], counts, out, t["table"],
                       starts, lens, slots, pos)
    got = dict(free=t["free"], counts=out, table=t["table"], starts=starts, lens=lens, slots=slots, positions=pos)
    return {k: v.cpu().numpy() for k, v in got.items()}


def check_pages(P, cached, fresh, free, n_free, table, max_tokens, **kw):
    got = run_pages(P, cached, fresh, free, n_free, table, max_tokens, **kw)
    ref = S.pages_assign(P, cached, fresh, free, n_free, table, max_tokens)
    for k, v in ref.items():
        assert np.array_equal(got[k], v), k


def pages_case(rng, n, P, width, most, new, gone, short=0):
    cached = rng.integers(0, most + 1, n)
    fresh = rng.integers(0, new + 1, n)
    fresh[rng.random(n) < gone] = -1
    held = np.minimum(-(-cached // P), width)
    need = np.minimum(-(-(cached + np.maximum(fresh, 0)) // P), width) - held
    ids = rng.permutation(int(held.sum() + need.sum()) + 9).astype(np.int32)
    table, at = rng.integers(-5, 99, (n, width)).astype(np.int32), 0
    for b in range(n):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.full(len(ids) + 3, -7, np.int32)
    rest = ids[at:]
    n_free = max(0, len(rest) - short)
    free[:n_free] = rest[:n_free]
    return cached, fresh, free, n_free, table, int(np.maximum(fresh, 0).sum())


@pytest.mark.parametrize("n,P,width,most,new,gone", [
    (1, 16, 3, 0, 1, 0.0), (1, 16, 4, 40, 1, 1.0), (2, 64, 5, 100, 200, 0.0), (33, 16, 20, 250, 60, 0.3), (64, 32, 9, 256, 1, 0.1),
    (700, 16, 40, 600, 40, 0.2), (4096, 16, 12, 150, 30, 0.1), (5, 1, 50, 20, 20, 0.4), (40, 48, 6, 200, 100, 0.2),
    (300, 64, 130, 8000, 300, 0.05)])
def test_pages_assign(n, P, width, most, new, gone):
    rng = np.random.default_rng(n * 7 + P)
    c = pages_case(rng, n, P, width, most, new, gone)
    check_pages(P, *c[:5], c[5] + 13)
    check_pages(P, *c[:5], max(0, c[5] - 5), in_place=True)     # room for fewer tokens than there are


def test_pages_assign_shortage_overflow_and_odd_inputs():
    rng = np.random.default_rng(5)
    c = pages_case(rng, 50, 16, 30, 300, 90, 0.1, short=70)     # too few pages
    check_pages(16, *c[:5], c[5] + 2)
    c = pages_case(rng, 20, 16, 4, 100, 90, 0.0)                # past the table's width
    check_pages(16, *c[:5], c[5])
    c = pages_case(rng, 9, 16, 12, 100, 50, 0.5)
    c[4][:, 1] = -1                                             # entries without a page are not given back
    check_pages(16, *c[:5], c[5])
    cached, fresh, free, n_free, table, tok = pages_case(rng, 6, 16, 12, 100, 50, 0.5)
    check_pages(16, cached, fresh, free[:n_free + 2], n_free, table, tok)       # pushes past the capacity are dropped
    check_pages(16, -np.abs(cached), np.maximum(fresh, 0), free, n_free, table, tok)    # negative lengths count as none
    check_pages(16, np.zeros(0, int), np.zeros(0, int), free, n_free, np.zeros((0, 3), np.int32), 4)
    check_pages(16, [3, 4], [0, 0], free, 0, np.zeros((2, 1), np.int32), 1)     # nothing to do


def test_pages_assign_of_more_tokens_than_a_wave_of_threads():
    rng = np.random.default_rng(8)
    c = pages_case(rng, 37, 64, 400, 9000, 16000, 0.1)
    got = run_pages(64, *c[:5], c[5] + 1)
    ref = S.pages_assign(64, *c[:5], c[5] + 1)
    for k, v in ref.items():
        assert np.array_equal(got[k], v), k


# ---------------------------------------------------------------- append

def random_cache(rng, pages, kv, P, D, lo=112, hi=130):
    codes = [rng.integers(0, 256, (pages, kv, P * D)).astype(np.uint8) for _ in range(2)]
    for c in codes:
        c[(c & 127) == 127] = 5
    return [*codes, *(rng.integers(lo, hi, (pages, kv)).astype(np.uint8) for _ in range(2))]


def run_append(c, P, D, xk, xv, slots, split=None):
    """-> arrays after the append; xk, xv numpy bf16 values; split: sizes of consecutive calls."""
    pages, kv = c[2].shape
    d = [dev(x) for x in c]
    plan = moe().Kv8(kv, kv, D, P, pages, cache=d)
    both, _ = bf16(np.concatenate([xk, xv], 1))         # rows of one projection: strided keys and values
    sl, at = dev(np.asarray(slots, np.int32)), 0
    for n in split or [len(slots)]:
        plan.append(both[at:at + n, :kv], both[at:at + n, kv:], sl[at:at + n])
        at += n
    return [x.cpu().numpy() for x in d]


def tokens(rng, n, kv, D, spread=6):
    x = rng.normal(0, 1, (n, kv, D)) * 2.0 ** rng.integers(-spread, spread, (n, 1, 1))
    return bf16(x)[1]


@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv", [1, 3, 8])
def test_append(P, D, kv):
    rng = np.random.default_rng(P + D + kv)
    c = random_cache(rng, 23, kv, P, D)
    order = rng.permutation(23)
    slots = []
    # a run inside a page, one that starts a page, one over several pages, a page to the end, padding
    for i, (page, off, n) in enumerate([(0, 3, 5), (1, 0, 7), (2, P - 1, 1), (3, 1, P - 1), (4, 0, P), (5, 0, 1)]):
        slots += [order[page] * P + off + j for j in range(n)] + ([-1] if i % 2 else [])
    for page in (7, 9, 12):
        slots += list(order[page] * P + np.arange(P)) + list(order[page + 1] * P + np.arange(P // 2 + 1))
    slots += [-1, 23 * P, 2 ** 31 - 1, -2 ** 31]
    xk, xv = tokens(rng, len(slots), kv, D), tokens(rng, len(slots), kv, D)
    got = run_append(c, P, D, xk, xv, slots)
    ref = S.append(*c, P, xk, xv, slots)
    for g, r in zip(got, ref):
        assert np.array_equal(g, r)


@pytest.mark.parametrize("P,D", [(16, 64), (64, 128)])
def test_append_token_by_token_rounds_again(P, D):
    rng = np.random.default_rng(3)
    c = random_cache(rng, 4, 2, P, D)
    slots = list(range(P + 3, 3 * P - 2))
    xk, xv = tokens(rng, len(slots), 2, D, 9), tokens(rng, len(slots), 2, D, 9)
    got = run_append(c, P, D, xk, xv, slots, split=[1] * len(slots))
    ref = c
    for i in range(len(slots)):
        ref = S.append(*ref, P, xk[i:i + 1], xv[i:i + 1], slots[i:i + 1])
    for g, r in zip(got, ref):
        assert np.array_equal(g, r)


def test_append_of_many_tokens_and_of_odd_values():
    rng = np.random.default_rng(4)
    P, D, kv, n = 32, 64, 2, 1500
    c = random_cache(rng, 60, kv, P, D)
    slots = np.concatenate([np.arange(5, 700), np.arange(30 * P + 1, 30 * P + 1 + n - 695)])
    xk, xv = tokens(rng, n, kv, D), tokens(rng, n, kv, D)
    xk[40, 0, 3] = np.inf
    xk[100, 1, 5] = -np.inf
    xk[200, 1, :] = np.nan
    xv[300, 0, 7] = np.nan
    xk[400:440], xv[400:440] = 0.0, 2.0 ** -133         # nothing, and subnormals
    xv[900:960] = -0.0
    xk[1000:1100] *= 2.0 ** 100
    got = run_append(c, P, D, xk, xv, slots)
    ref = S.append(*c, P, bf16(xk)[1], bf16(xv)[1], slots)
    for g, r in zip(got, ref):
        assert np.array_equal(g, r)


# ---------------------------------------------------------------- attention

def sequences(rng, P, lens, rows, width, pages, kv, D, poison=True, **cache):
    """A cache with each sequence's tokens on pages of its own, NaN everywhere else."""
    c = random_cache(rng, pages, kv, P, D, **cache)
    order, at = rng.permutation(pages), 0
    table = rng.integers(-3, pages + 3, (len(lens), width)).astype(np.int32)     # entries past a sequence are anything
    kk, vv = S.unpack(c[0], c[1], P, D)
    used = np.zeros((pages, P), bool)
    for b, L in enumerate(lens):
        n = min(-(-L // P), width)
        table[b, :n] = order[at:at + n]
        for j in range(n):
            used[order[at + j], :min(P, L - j * P)] = True
        at += n
    assert at <= pages
    if poison:
        kk[~used] = 127
        vv[~used] = 127
        c[:2] = S.pack(kk, vv)
        free = order[at:]
        c[2][free], c[3][free] = 255, 255
    return c, table


def check_attend(rng, P, D, kv, H, lens, rows, window=0, sinks=True, width=None, pages=None, scale=None, spread=0.25,
                 max_new=None, extra=0, poison=True, change=None, **cache):
    import torch
    lens, rows = list(lens), list(rows)
    width = width or max(1, -(-max(lens) // P))
    pages = pages or sum(-(-L // P) for L in lens) + 3
    c, table = sequences(rng, P, lens, rows, width, pages, kv, D, poison, **cache)
    if change:
        change(c, table)
    starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    n = int(starts[-1]) + extra
    qd, q = bf16(rng.normal(0, spread, (n, H + 2, D)))
    qd, q = qd[:, 1:H + 1], q[:, 1:H + 1]                # rows of a wider projection
    s = rng.normal(0, 2, H).astype(np.float32) if sinks else None
    plan = moe().Kv8(H, kv, D, P, pages, sliding_window=window, softmax_scale=scale, sinks=None if s is None else dev(s),
                     cache=[dev(x) for x in c])
    out = torch.full((n, H, D), 7.5, dtype=torch.bfloat16, device="cuda")
    one = all(r == 1 for r in rows) and extra == 0
    most = max_new if max_new is not None else max(rows + [1])
    for use in ([False, True] if one else [True]):      # with and without starts
        out.fill_(7.5)
        plan.attend(qd, dev(np.array(lens, np.int32)), dev(table), out, starts=dev(starts) if use else None, max_new=most)
        got = out.double().cpu().numpy()
        # more than 64 rows (new tokens x query heads of a kv head) a sequence: the kernel for prompts
        ref, tol = S.attend(*c, P, q, starts, lens, table, window, s, scale, 2.0 ** -31 if most * (H // kv) > 64 else 2.0 ** -39)
        for b in range(len(lens)):
            a, z = starts[b], min(starts[b] + most, starts[b + 1])
            nan = np.isnan(ref[a:z])
            assert np.array_equal(np.isnan(got[a:z]), nan), b
            far = np.abs(got[a:z] - ref[a:z])[~nan] / tol[a:z][~nan]
            assert not far.size or far.max() <= 1, (b, far.max())
            assert np.all(got[z:starts[b + 1]] == 7.5)
        assert np.all(got[starts[-1]:] == 7.5)          # rows of no sequence
    return got


@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv,H", [(1, 1), (2, 16), (3, 9), (2, 20), (1, 16), (4, 4)])
def test_attend_one_token_a_sequence(P, D, kv, H):
    rng = np.random.default_rng(P * D + H)
    check_attend(rng, P, D, kv, H, [1, 2, P - 1, P, P + 1, 63, 64, 65, 200, 0, 333], [1] * 11, sinks=H % 2 == 0)


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 128, 1000])
@pytest.mark.parametrize("P,D", [(16, 64), (64, 128)])
def test_attend_sliding_window(window, P, D):
    rng = np.random.default_rng(window)
    check_attend(rng, P, D, 2, 8, [1, 5, 64, 127, 128, 129, 500], [1] * 7, window=window)
    check_attend(rng, P, D, 2, 8, [5, 64, 200, 129], [5, 3, 40, 1], window=window, sinks=False)


@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv,H", [(2, 2), (1, 5), (2, 16), (1, 16), (2, 22)])
def test_attend_several_tokens_a_sequence(P, D, kv, H):
    rng = np.random.default_rng(P * D + H + 1)
    check_attend(rng, P, D, kv, H, [2, 3, 40, 65, 130, 1], [2, 1, 4, 3, 5, 0])                    # a few
    check_attend(rng, P, D, kv, H, [70, 33, 150, 9, 260], [70, 1, 37, 9, 130], sinks=False)       # prompts


def test_attend_long_contexts_and_many_sequences():
    rng = np.random.default_rng(11)
    check_attend(rng, 64, 64, 1, 8, [9000], [1])                       # one sequence over the whole GPU
    check_attend(rng, 16, 128, 1, 2, [3000, 1, 2500], [1, 1, 1])
    check_attend(rng, 16, 64, 1, 1, list(rng.integers(0, 40, 700)), [1] * 700)
    check_attend(rng, 32, 64, 2, 16, [1500, 700], [400, 3], max_new=400)


def test_attend_rows_that_see_nothing():
    rng = np.random.default_rng(12)
    got = check_attend(rng, 16, 64, 1, 4, [0, 3, 0], [1, 1, 1])
    assert np.all(got[[0, 2]] == 0)
    # more rows than tokens: the first rows stand before the sequence's beginning
    got = check_attend(rng, 16, 64, 2, 4, [3, 0, 20], [5, 3, 40], sinks=False)
    assert np.all(got[:2] == 0) and np.all(got[5:8] == 0) and np.all(got[8:28] == 0)


@pytest.mark.parametrize("rows", [[1, 1, 1], [5, 60, 2]])
def test_attend_lengths_and_starts_out_of_range(rows):
    import torch
    rng = np.random.default_rng(18)
    P, D, kv, H, n = 16, 64, 2, 8, sum(rows)
    c, table = sequences(rng, P, [64, 64, 64], rows, 4, 20, kv, D, poison=False)
    plan = moe().Kv8(H, kv, D, P, 20, cache=[dev(x) for x in c])
    qd, q = bf16(rng.normal(0, 0.25, (n, H, D)))
    out = torch.full((n, H, D), 7.5, dtype=torch.bfloat16, device="cuda")
    starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    # a length below 0 is none; the sequence between keeps its own
    plan.attend(qd, dev(np.array([-2 ** 31, 64, -5], np.int32)), dev(table), out, starts=dev(starts), max_new=max(rows))
    got = out.double().cpu().numpy()
    ref, tol = S.attend(*c, P, q, starts, [0, 64, 0], table, floor=2.0 ** -31)
    assert (np.abs(got - ref) / tol).max() <= 1
    assert np.all(got[:starts[1]] == 0) and np.all(got[starts[2]:] == 0)
    # starts past the rows, before them and going back: nothing outside out's rows is written
    guard = torch.full((n + 40, H, D), 7.5, dtype=torch.bfloat16, device="cuda")
    for bad in ([0, n + 5, 2 * n, 2 ** 31 - 1], [-7, -3, 1, n], [n, 2, 1, 0], [2 ** 31 - 1] * 4):
        guard.fill_(7.5)
        plan.attend(qd, dev(np.array([64, 64, 64], np.int32)), dev(table), guard[20:20 + n], starts=dev(np.array(bad, np.int32)), max_new=max(rows))
        assert bool((guard[:20] == 7.5).all()) and bool((guard[20 + n:] == 7.5).all())
    assert plan.device_status() == 0


def test_attend_pages_that_are_not_there():
    rng = np.random.default_rng(13)

    def change(c, table):
        table[0, 1], table[1, 0], table[1, 1], table[2, :] = -1, c[2].shape[0], 2 ** 31 - 1, -2 ** 31

    for rows in ([1, 1, 1], [3, 30, 70]):
        check_attend(rng, 32, 64, 2, 8, [100, 70, 90], rows, change=change, sinks=True)
        check_attend(rng, 32, 64, 2, 8, [100, 70, 90], rows, change=change, sinks=False)
    # lengths past the table's width: the tokens behind it are not seen
    check_attend(rng, 16, 64, 1, 2, [100, 40], [1, 1], width=2, pages=20)
    check_attend(rng, 16, 64, 1, 2, [100, 40], [30, 20], width=2, pages=20)


@pytest.mark.parametrize("rows", [[1, 1], [20, 70]])
def test_attend_padding_and_row_limits(rows):
    rng = np.random.default_rng(14)
    check_attend(rng, 16, 64, 2, 4, [90, 200], rows, extra=5, max_new=max(rows))
    if max(rows) > 1:
        check_attend(rng, 16, 64, 2, 4, [90, 200], rows, max_new=7)     # later rows are left as they were


@pytest.mark.parametrize("rows", [[1, 1, 1], [9, 40, 3]])
def test_attend_scales_far_apart(rows):
    rng = np.random.default_rng(15)

    def change(c, table):
        c[3][...] = rng.integers(100, 150, c[3].shape)      # value pages from 2^-27 to 2^22 times the codes
        c[3][table[1, 0]] = 1                               # a page of (nearly) nothing still counts in the sum

    check_attend(rng, 16, 64, 2, 8, [100, 70, 333], rows, change=change)
    # scores up to about 100, one key far above the rest, and a sink that takes nearly all
    check_attend(rng, 16, 64, 1, 8, [300, 64, 1000], rows, lo=124, hi=128, spread=0.02, scale=1.0)


@pytest.mark.parametrize("P,D", [(16, 64), (64, 128)])
@pytest.mark.parametrize("rows", [[3, 2, 1], [70, 33, 200]])
@pytest.mark.parametrize("window", [0, 20])
def test_attend_nan_values_reach_only_rows_that_see_them(P, D, rows, window):
    rng = np.random.default_rng(17)
    lens = [100, 75, 333]

    def change(c, table):
        kk, vv = S.unpack(c[0], c[1], P, D)
        for b, t in ((0, 99), (0, 40), (1, 74 - rows[1] // 2), (2, 332 - rows[2] // 2)):   # a last token, ones before
            vv[table[b, t // P], t % P, b % 2, 3 + b] = 127
        c[:2] = S.pack(kk, vv)

    check_attend(rng, P, D, 2, 8, lens, rows, window=window, change=change)


def test_attend_two_streams_graph_replay_and_repeats():
    import torch
    rng = np.random.default_rng(16)
    P, D, kv, H, lens = 16, 64, 2, 16, [700, 33, 1000, 5]
    c, table = sequences(rng, P, lens, [1] * 4, 64, 120, kv, D, poison=False)
    d = [dev(x) for x in c]
    qd, q = bf16(rng.normal(0, 0.25, (4, H, D)))
    plans = [moe().Kv8(H, kv, D, P, 120, cache=d) for _ in range(2)]
    ld, td = dev(np.array(lens, np.int32)), dev(table)
    outs = [torch.zeros((4, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):     # two calls at once, a workspace each
        for p, o, s in zip(plans, outs, streams):
            p.attend(qd, ld, td, o, stream=s)
    torch.cuda.synchronize()
    ref, tol = S.attend(*c, P, q, range(5), lens, table)
    for o in outs:
        assert (np.abs(o.double().cpu().numpy() - ref) / tol).max() <= 1
    assert torch.equal(outs[0], outs[1])
    # two graphs over one workspace, replayed in turn, with lengths that change between replays
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            plans[0].attend(qd, ld, td, o)
        graphs.append(g)
    for lens in ([700, 33, 1000, 5], [1, 500, 64, 0], [1000, 1000, 1000, 1000]):
        ld.copy_(torch.tensor(lens, dtype=torch.int32))
        for o, g in zip(outs, graphs):
            o.fill_(3.0)
            g.replay()
            g.replay()
        torch.cuda.synchronize()
        ref, tol = S.attend(*c, P, q, range(5), lens, table)
        for o in outs:
            assert (np.abs(o.double().cpu().numpy() - ref) / tol).max() <= 1


def test_attend_empty_calls_change_nothing():
    import torch
    p = moe().Kv8(4, 2, 64, 16, 3)
    z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device="cuda")   # noqa: E731
    q = z(0, 4, 64, t=torch.bfloat16)
    p.attend(q, z(0), z(0, 2), q.clone())
    q, o = z(3, 4, 64, t=torch.bfloat16), torch.full((3, 4, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    p.attend(q, z(0), z(0, 2), o, starts=z(1), max_new=3)
    p.attend(q, z(2), z(2, 0), o, starts=z(3), max_new=3)       # no rows in any sequence
    assert bool((o == 2.0).all())
    p.attend(q, z(3), z(3, 0), o)                               # a table without entries: nothing is seen
    assert bool((o == 0.0).all())
    with pytest.raises(moe().MoeError):
        p.attend(q, z(3), z(3, 1), q)                           # in place
    with pytest.raises(moe().MoeError):
        p.attend(q[:, :, ::2], z(3), z(3, 1), o)


# ---------------------------------------------------------------- sampling

def check_sample(x, u, t=None, k=None, p=None, mp=None, dtype="float32", stride=0):
    import torch
    n, V = x.shape
    full = torch.full((n, V + stride), 50.0)                     # what lies behind a row is not read
    full[:, :V] = torch.from_numpy(np.asarray(x, np.float32))
    full = full.to(getattr(torch, dtype))
    vals = full[:, :V].double().numpy()
    ids = torch.full((n,), -9, dtype=torch.int32, device="cuda")
    par = {}
    for name, v, ty in (("temperature", t, np.float32), ("top_k", k, np.int32), ("top_p", p, np.float32), ("min_p", mp, np.float32)):
        if v is not None:
            par[name] = dev(np.broadcast_to(np.asarray(v, ty), (n,)).copy())
    u = np.broadcast_to(np.asarray(u, np.float32), (n,)).copy()
    moe().sample(full.cuda()[:, :V], dev(u), ids, **par)
    got = ids.cpu().numpy()
    at = lambda a, i, d: float(np.broadcast_to(np.asarray(a, np.float32), (n,))[i]) if a is not None else d   # noqa: E731
    for r in range(n):
        w = S.kept(vals[r], at(t, r, 1.0), int(at(k, r, 0)), at(p, r, 1.0), at(mp, r, 0.0))
        want = S.sample(w, float(u[r]))
        if got[r] == want:
            continue
        assert want >= 0 and 0 <= got[r] < V and w[got[r]] > 0, (r, got[r], want)
        c = np.cumsum(w)
        goal, slack = float(u[r]) * c[-1], 2.0 ** -18 * c[-1]
        assert c[got[r]] - w[got[r]] <= goal + slack and goal - slack <= c[got[r]], (r, got[r], want)
    return got


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("V", [1, 2, 7, 32, 1000, 1024, 1025, 4099, 50001, 201000])
def test_sample(V, dtype):
    rng = np.random.default_rng(V)
    n = 12
    x = rng.normal(0, 3, (n, V))
    u = rng.random(n)
    check_sample(x, u, dtype=dtype)
    check_sample(x, u, t=0.7, k=40, p=0.9, mp=0.02, dtype=dtype, stride=3)
    t = rng.choice([0.0, 0.5, 1.0, 2.0], n)
    k = rng.choice([-1, 0, 1, 3, 50, V, V + 5], n)
    p = rng.choice([0.0, 0.1, 0.5, 0.99, 1.0, 1.5], n)
    mp = rng.choice([0.0, 0.01, 0.3, 1.0, 2.0], n)
    check_sample(x, u, t=t, k=k, p=p, dtype=dtype, stride=1)
    check_sample(x, u, t=t, k=k, p=p, mp=mp, dtype=dtype)
    check_sample(x, u, t=t, p=p, dtype=dtype)


@pytest.mark.parametrize("n,V,dtype", [(16, 200000, "float32"), (21, 40000, "bfloat16"), (45, 130000, "bfloat16"), (80, 131072, "bfloat16"),
                                       (90, 201000, "float32"), (1, 1 << 22, "float32"), (2, (1 << 22) - 3, "bfloat16"),
                                       (160, 5000, "float32")])
def test_sample_batches_of_all_shapes(n, V, dtype):
    # from one row over many CTAs to rows that share the device, kept in shared memory and not
    rng = np.random.default_rng(n + V)
    x = rng.normal(0, 3, (n, V)).astype(np.float32)
    pick = lambda *v: rng.choice(v, n)   # noqa: E731
    check_sample(x, rng.random(n), t=pick(0.5, 0.9, 1.3), k=pick(0, 40, 700), p=pick(0.9, 0.3, 1.0), mp=pick(0.0, 0.02), dtype=dtype)


def test_two_streams_of_page_tables_and_sampling():
    import torch
    rng = np.random.default_rng(23)
    x = dev(rng.normal(0, 2, (40, 30011)).astype(np.float32))
    u = dev(rng.random(40).astype(np.float32))
    k, p = dev(np.full(40, 900, np.int32)), dev(np.full(40, 0.9, np.float32))
    streams = [torch.cuda.Stream() for _ in range(2)]
    out = []
    for _ in range(2):
        i = lambda *a: torch.zeros(a, dtype=torch.int32, device="cuda")   # noqa: E731
        out.append(dict(ids=i(40), table=i(700, 9), starts=i(701), lens=i(700), slots=i(9000), free=torch.arange(6000, dtype=torch.int32, device="cuda"),
                        counts=torch.tensor([6000, 0], dtype=torch.int32, device="cuda")))
    cached, fresh = i(700), dev(rng.integers(0, 14, 700).astype(np.int32))
    torch.cuda.synchronize()
    for turn in range(10):      # no entry point keeps anything of another call's
        for s, o in zip(streams, out):
            moe().pages_assign(16, cached, fresh, o["free"], o["counts"], o["counts"], o["table"], o["starts"], o["lens"], o["slots"], stream=s)
            moe().sample(x, u, o["ids"], top_k=k, top_p=p, stream=s)
    torch.cuda.synchronize()
    for n in out[0]:
        assert torch.equal(out[0][n], out[1][n]), n
    # 10 times 657 pages of 6000: the last call got 87 of its own
    pages = int((fresh > 0).sum())
    assert pages == 657 and out[0]["counts"].tolist() == [0, 10 * pages - 6000]
    once = torch.zeros_like(out[0]["ids"])
    moe().sample(x, u, once, top_k=k, top_p=p)
    assert torch.equal(once, out[0]["ids"])


def test_bindings_refuse_other_types():
    import torch
    M = moe()
    z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device="cuda")   # noqa: E731
    f = lambda *s: z(*s, t=torch.float32)   # noqa: E731
    calls = [lambda: M.sample(z(2, 8, t=torch.float16), f(2), z(2)), lambda: M.sample(f(2, 8), z(2), z(2)),
             lambda: M.sample(f(2, 8), f(2), f(2)), lambda: M.sample(f(2, 8), f(2), z(2), top_k=f(2)),
             lambda: M.sample(f(2, 8), f(2), z(2), temperature=z(2)), lambda: M.sample(f(2, 8), f(2), z(3))]
    plan = M.Kv8(4, 2, 64, 16, 3)
    b = lambda n, h, t=torch.bfloat16: z(n, h, 64, t=t)   # noqa: E731
    calls += [lambda: plan.append(b(2, 2, torch.float16), b(2, 2), z(2)), lambda: plan.append(b(2, 2), b(2, 2), f(2)),
              lambda: plan.append(b(2, 2), b(3, 2), z(2)), lambda: plan.append(b(2, 4), b(2, 4), z(2)),
              lambda: plan.attend(b(2, 4, torch.float16), z(2), z(2, 1), b(2, 4)), lambda: plan.attend(b(2, 4), f(2), z(2, 1), b(2, 4)),
              lambda: plan.attend(b(2, 4), z(2), z(2, 1), b(3, 4)), lambda: plan.attend(b(2, 4), z(2), z(3, 1), b(2, 4))]
    for n, c in enumerate(calls):
        with pytest.raises(M.MoeError):
            c()
            raise AssertionError(f"call {n} was not refused")
    assert plan.device_status() == 0


def test_bindings_refuse_tensors_of_another_device(monkeypatch):
    import torch
    M = moe()
    z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device="cuda")   # noqa: E731
    b = lambda n, h: z(n, h, 64, t=torch.bfloat16)   # noqa: E731
    plan = M.Kv8(4, 2, 64, 16, 3)
    plan.append(b(1, 2), b(1, 2), z(1))
    monkeypatch.setattr(M, "_raw_stream", (M._raw_stream[0], lambda: 1))     # as where the current device is the second
    for call in (lambda: plan.append(b(1, 2), b(1, 2), z(1)), lambda: plan.attend(b(1, 4), z(1), z(1, 1), b(1, 4)),
                 lambda: M.sample(z(1, 4, t=torch.float32), z(1, t=torch.float32), z(1)), plan.device_status,
                 lambda: M.pages_assign(16, z(1), z(1), z(4), z(2), z(2), z(1, 2), z(2), torch.ones(1, dtype=torch.int32, device="cuda"), z(3))):
        with pytest.raises(M.MoeError, match="device"):
            call()


def test_sample_equal_and_odd_logits():
    rng = np.random.default_rng(1)
    V = 3001
    u = rng.random(16)
    x = rng.integers(-3, 4, (16, V)).astype(np.float64)          # few distinct values, -0 among them
    x[:, ::7] *= -0.0
    check_sample(x, u, k=rng.integers(1, V, 16), p=0.7)
    check_sample(x, u, k=rng.integers(1, 50, 16), p=1.0)
    check_sample(x, u, p=rng.random(16))
    check_sample(np.zeros((16, V)), u, k=rng.integers(1, V, 16), p=rng.random(16))
    y = rng.normal(0, 2, (16, V))
    y[:, rng.integers(0, V, 900)] = np.nan
    y[:, rng.integers(0, V, 900)] = -np.inf
    check_sample(y, u, k=100, p=0.8)
    y[3], y[4, :], y[5, :] = np.nan, -np.inf, -1e30
    y[6], y[7, 5], y[8, [3, 9, 700]] = -np.inf, 3e38, np.inf
    y[6, 17] = -3e38
    got = check_sample(y, u, t=0.8, p=0.9)
    assert got[3] == -1 and got[4] == -1 and got[6] == 17 and got[7] == 5 and got[8] in (3, 9, 700)
    y = rng.normal(0, 1, (16, V)) + 1e4                            # far from zero; close together
    check_sample(y, u, t=rng.choice([1e-6, 0.01, 1.0, 100.0], 16), p=0.95)
    check_sample(rng.normal(0, 30, (16, V)), u, k=500, p=0.999999, mp=1e-9)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_sample_where_the_threshold_is_hard_to_find(dtype):
    """Many logits within one step of the first histogram, far below its range, or at its bins' edges."""
    rng = np.random.default_rng(9)
    V, n = 60000, 8
    u = rng.random(n)
    p = np.array([0.01, 0.3, 0.5, 0.9, 0.99, 0.9999, 0.7, 0.2])
    k = np.array([1, 7, 100, 3000, 30000, 59999, 50, 2])
    near = rng.normal(0, 1e-3, (n, V))
    far = rng.normal(0, 1, (n, V)) - 40
    far[:, 777] = 9.0
    edges = np.repeat(rng.normal(0, 4, (n, 60)), 1000, 1)
    for x in (near, far, edges, np.zeros((n, V)), rng.normal(0, 3, (n, V))):
        check_sample(x, u, p=p, dtype=dtype)
        check_sample(x, u, k=k, dtype=dtype)
        check_sample(x, u, k=k, p=p, t=0.9, dtype=dtype)
    check_sample(rng.normal(0, 1, (2, 1200000)), u[:2], p=0.9, dtype=dtype)       # more than shared memory holds
    check_sample(rng.normal(0, 1, (2, 1200000)), u[:2], k=70000, p=0.9, dtype=dtype)


def test_sample_the_ends_of_u():
    x = np.random.default_rng(2).normal(0, 1, (4, 777))
    first = check_sample(x, 0.0, p=0.5)
    last = check_sample(x, np.float32(1 - 2.0 ** -24), p=0.5)
    for r in range(4):
        keep = np.flatnonzero(S.kept(np.float32(x[r]), 1.0, 0, 0.5, 0.0))
        assert first[r] == keep[0] and last[r] == keep[-1]


def test_sample_many_rows_and_distribution():
    rng = np.random.default_rng(3)
    check_sample(rng.normal(0, 2, (700, 999)), rng.random(700), t=0.9, k=rng.integers(0, 30, 700), p=0.9)
    # one row's distribution over an even grid of u: counts within one of the exact ones
    x = rng.normal(0, 1, 20)
    n = 4096
    u = (np.arange(n) + 0.5) / n
    got = check_sample(np.tile(x, (n, 1)), u, k=9)
    w = S.kept(np.float32(x), 1.0, 9, 1.0, 0.0)
    assert np.all(np.abs(np.bincount(got, minlength=20) - n * w / w.sum()) <= 1.01)


# ---------------------------------------------------------------- together

def test_a_serving_run_of_all_operators_and_its_graph():
    """Requests come, grow by ragged numbers of tokens, finish and give their pages back; each step assigns pages,
    appends, attends and samples.  The whole run once call by call and once as a captured step replayed."""
    import torch
    m = moe()
    P, D, kv, H, pages, n, W, V, steps, cap = 16, 64, 2, 8, 40, 6, 12, 500, 14, 160
    rng = np.random.default_rng(21)
    plan_steps = []
    lens = np.zeros(n, np.int64)
    for _ in range(steps):
        fresh = np.where(rng.random(n) < 0.5, 1, rng.integers(0, 27, n))
        fresh = np.where((lens + fresh > 100) | (rng.random(n) < 0.1), -1, fresh)
        plan_steps.append(fresh)
        lens = np.where(fresh < 0, 0, lens + fresh)
    sinks = rng.normal(0, 1, H).astype(np.float32)
    xs = [rng.normal(0, 1, (cap, H + 2 * kv, D)) for _ in range(steps)]
    us = [rng.random(n).astype(np.float32) for _ in range(steps)]
    head = rng.normal(0, 0.1, (H * D, V)).astype(np.float32)

    def run(graph):
        z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device="cuda")   # noqa: E731
        plan = m.Kv8(H, kv, D, P, pages, sinks=dev(sinks), sliding_window=50)
        free, counts, table = dev(np.arange(pages, dtype=np.int32)), dev(np.array([pages, 0], np.int32)), z(n, W)
        have, fresh, lens, starts, slots = z(n), z(n), z(n), z(n + 1), z(cap)
        rows = z(cap, H + 2 * kv, D, t=torch.bfloat16)
        out, u, ids, hd = z(cap, H, D, t=torch.bfloat16), z(n, t=torch.float32), z(n), dev(head)

        def step():
            m.pages_assign(P, have, fresh, free, counts, counts, table, starts, lens, slots)
            plan.append(rows[:, H:H + kv], rows[:, H + kv:], slots)
            plan.attend(rows[:, :H], lens, table, out, starts=starts, max_new=27)
            last = (starts[1:].long() - 1).clamp(min=0)
            m.sample(out[last].float().view(n, -1) @ hd, u, ids, top_k=None, temperature=None)
            have.copy_(lens)

        g = None
        seen = []
        for s in range(steps):
            fresh.copy_(dev(plan_steps[s].astype(np.int32)))
            rows.copy_(bf16(xs[s])[0])
            u.copy_(dev(us[s]))
            out.zero_()
            if graph and g is None:
                side = torch.cuda.Stream()
                side.wait_stream(torch.cuda.current_stream())
                keep = [t.clone() for t in (have, free, counts, table, plan.k, plan.v, plan.k_scale, plan.v_scale)]
                with torch.cuda.stream(side):
                    step()                                       # a first run outside the capture
                torch.cuda.current_stream().wait_stream(side)
                for t, c in zip((have, free, counts, table, plan.k, plan.v, plan.k_scale, plan.v_scale), keep):
                    t.copy_(c)
                out.zero_()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    step()
            g.replay() if graph else step()
            seen.append([t.cpu().numpy().copy() for t in (table, starts, lens, slots, counts, plan.k, plan.v, plan.k_scale,
                                                          plan.v_scale, ids)] + [out.double().cpu().numpy()])
        return seen

    calls, replays = run(False), run(True)
    for a, b in zip(calls, replays):
        assert all(np.array_equal(x, y) for x, y in zip(a, b))
    free, n_free, table, have = np.arange(pages, dtype=np.int32), pages, np.zeros((n, W), np.int32), np.zeros(n, np.int64)
    cache = [np.zeros((pages, kv, P * D), np.uint8)] * 2 + [np.zeros((pages, kv), np.uint8)] * 2
    for s in range(steps):
        r = S.pages_assign(P, have, plan_steps[s], free, n_free, table, cap)
        free, n_free, table, have = r["free"], int(r["counts"][0]), r["table"], r["lens"].astype(np.int64)
        assert r["counts"][1] == 0 and r["starts"][-1] <= cap
        x = bf16(xs[s])[1]
        cache = list(S.append(*cache, P, x[:, H:H + kv], x[:, H + kv:], r["slots"]))
        got = calls[s]
        for g, w in zip(got[:9], (table, r["starts"], r["lens"], r["slots"], r["counts"], *cache)):
            assert np.array_equal(g, w), s
        ref, tol = S.attend(*cache, P, x[:, :H], r["starts"], r["lens"], table, 50, sinks, floor=2.0 ** -31)
        a = slice(0, int(r["starts"][-1]))
        assert (np.abs(got[10][a] - ref[a]) / tol[a]).max() <= 1, s
        assert np.all(got[10][a.stop:] == 0)
