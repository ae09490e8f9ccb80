"""The serving operators on the GPU where they are easily wrong, against oracle/serving.py: tokens that weigh next to
nothing beside another, parameters that are not numbers, thresholds among nearly equal tokens;
plans made while streams are busy; NaN in every hidden place; the largest
windows; a sequence that goes on past the rows;
scores that need more than 24 bits; page
tables and free lists of nearly 2^31 entries.

Tolerances are those of test_gpu_serving.py."""
import numpy as np
import pytest

import test_gpu_serving as base
from oracle import serving as S

pytestmark = pytest.mark.gpu
LAST = np.float32(1 - 2.0 ** -24)       # the largest u


# ---------------------------------------------------------------- page tables

def big_pages(n, width, cached, fresh, table_fill, capacity, n_free, tokens):
    """A call with P = 1; -> (table, free, counts_out, starts, lens, slots) on the GPU, and the table's and list's given tails."""
    import torch
    i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    table = torch.full((n, width), table_fill, dtype=torch.int32, device="cuda")
    free = torch.full((capacity,), 5, dtype=torch.int32, device="cuda")
    free[:min(n_free, 3000)] = torch.arange(min(n_free, 3000), dtype=torch.int32, device="cuda")
    counts, out = i([n_free, 0]), i([0, 0])
    cached, fresh = i([cached] * n), i([fresh] * n)
    starts, lens, slots = i([9] * (n + 1)), i([9] * n), i([9] * tokens)
    return table, free, counts, out, cached, fresh, starts, lens, slots


@pytest.mark.parametrize("room", [2047, 2048, 2049, 5000])
@pytest.mark.parametrize("n", [40, 1024, 1025])
def test_pages_assign_around_the_sizes_of_one_cta(n, room):
    rng = np.random.default_rng(n + room)
    c = base.pages_case(rng, n, 16, 64, 900, 1 if n > 100 else 100, 0.2)
    base.check_pages(16, *c[:5], room)
    base.check_pages(16, *c[:5], room, in_place=True)


WIDE = (2 ** 31 - 1) // 4096


def test_pages_assign_of_nearly_2_31_wanted_pages():
    import torch
    table, free, counts, out, cached, fresh, starts, lens, slots = big_pages(4096, WIDE, 0, WIDE, 7, 1000, 1000, 1500)
    base.moe().pages_assign(1, cached, fresh, free, counts, out, table, starts, lens, slots)
    flat = table.view(-1)
    assert out.tolist() == [0, 4096 * WIDE - 1000]
    assert torch.equal(flat[:1000], torch.arange(999, -1, -1, dtype=torch.int32, device="cuda"))
    assert bool((flat[1000:] == -1).all())
    assert torch.equal(slots[:1000], flat[:1000]) and bool((slots[1000:] == -1).all())
    assert starts[-1].item() == 4096 * WIDE and bool((lens == WIDE).all())


def test_pages_assign_of_nearly_2_31_entries_given_back():
    import torch
    table, free, counts, out, cached, fresh, starts, lens, slots = big_pages(4096, WIDE, WIDE, -1, -1, 5000, 4, 10)
    places = [0, 1, WIDE - 1, WIDE, 2000 * WIDE + 17, 4096 * WIDE - 2, 4096 * WIDE - 1]
    table.view(-1)[torch.tensor(places, device="cuda")] = torch.arange(100, 107, dtype=torch.int32, device="cuda")
    base.moe().pages_assign(1, cached, fresh, free, counts, out, table, starts, lens, slots)
    assert out.tolist() == [11, 0] and free[:13].tolist() == [0, 1, 2, 3, *range(100, 107), 5, 5]
    assert bool((starts == 0).all()) and bool((lens == 0).all()) and bool((slots == -1).all())


def test_pages_assign_with_a_full_free_list_of_2_31_entries():
    import torch
    most = 2 ** 31 - 1
    for n in (40, 3000):        # one kernel, and two
        table, free, counts, out, cached, fresh, starts, lens, slots = big_pages(n, 20, 16, -1, 77, most, most, 30)
        cached[-1], fresh[-1] = 0, 3
        free[-3:] = torch.tensor([21, 22, 23], dtype=torch.int32, device="cuda")
        base.moe().pages_assign(1, cached, fresh, free, counts, out, table, starts, lens, slots)
        assert out.tolist() == [most - 3, 0]                    # what was given back had no room
        assert table[-1, :4].tolist() == [23, 22, 21, 77] and slots[:4].tolist() == [23, 22, 21, -1]
        assert free[-3:].tolist() == [21, 22, 23] and bool((free[3000:-3] == 5).all())
        del table, free


# ---------------------------------------------------------------- sampling

@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("V,top,n", [(128000, 29.5, 6), (200000, 31.0, 6), (5000, 35.0, 6), (20000, 40.0, 200), (1200000, 30.0, 2)])
def test_sample_tokens_far_below_another(V, top, n, dtype):
    rng = np.random.default_rng(V)
    x = rng.normal(0, 0.25, (n, V)).astype(np.float32)
    x[np.arange(n), V - 1 - np.arange(n) * 7] = top
    vals = base.bf16(x)[1] if dtype == "bfloat16" else x
    for kw in (dict(), dict(k=V // 2), dict(mp=1e-25), dict(k=V - 1, t=0.9)):
        got = base.check_sample(x, 0.0, dtype=dtype, **kw)
        for r in range(n):      # at u = 0 the first kept token, however little it weighs
            w = S.kept(vals[r], kw.get("t", 1.0), kw.get("k", 0), 1.0, kw.get("mp", 0.0))
            assert got[r] == np.flatnonzero(w)[0]
        base.check_sample(x, np.resize(np.float32([1e-30, 2.0 ** -24, LAST, 0.5, 2.0 ** -60]), n), dtype=dtype, **kw)


def test_sample_ranked_tokens_far_below_the_first():
    rng = np.random.default_rng(1)
    x = rng.normal(0, 0.25, (8, 3000)).astype(np.float32)
    x[:, 2990] = 36.0
    got = base.check_sample(x, 0.0, k=100)
    assert all(got[r] == np.flatnonzero(S.kept(x[r], 1.0, 100, 1.0, 0.0))[0] for r in range(8))


@pytest.mark.parametrize("n", [3, 300])
def test_sample_nan_temperature_takes_the_first_token(n):
    rng = np.random.default_rng(2)
    x = rng.normal(0, 1, (n, 3000))
    t = np.where(np.arange(n) % 3 == 1, 0.8, np.nan)
    got = base.check_sample(x, rng.random(n), t=t, p=0.9)
    nan = np.isnan(t)
    assert np.array_equal(got[nan], np.argmax(np.float32(x), 1)[nan])
    base.check_sample(x[:3], rng.random(3), t=[np.inf, -np.inf, np.nan], k=50)


def test_sample_nan_top_p_and_min_p_are_none():
    import torch
    rng = np.random.default_rng(13)
    for k in (0, 40, 900):
        x, u = base.dev(rng.normal(0, 2, (9, 5000)).astype(np.float32)), base.dev(rng.random(9).astype(np.float32))
        nan, some = np.full(9, np.nan, np.float32), np.where(np.arange(9) % 2, np.nan, 0.02).astype(np.float32)
        kk = base.dev(np.full(9, k, np.int32))
        ids = [torch.zeros(9, dtype=torch.int32, device="cuda") for _ in range(4)]
        base.moe().sample(x, u, ids[0], top_k=kk)
        base.moe().sample(x, u, ids[1], top_k=kk, top_p=base.dev(nan), min_p=base.dev(nan))
        base.moe().sample(x, u, ids[2], top_k=kk, top_p=base.dev(nan), min_p=base.dev(some))
        base.moe().sample(x, u, ids[3], top_k=kk, min_p=base.dev(np.nan_to_num(some)))
        assert torch.equal(ids[0], ids[1]) and torch.equal(ids[2], ids[3])


@pytest.mark.parametrize("V,std,t,p", [(128000, 0.02, 1.0, 0.5), (128000, 0.02, 1.0, 0.4), (200000, 2.5, 30.0, 0.5), (128000, 2.5, 200.0, 0.8),
                                       (60000, 1e-3, 1.0, 0.5), (1000003, 0.5, 3.0, 0.6), (1 << 22, 0.3, 2.0, 0.7)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_sample_nucleus_of_nearly_equal_tokens(V, std, t, p, dtype):
    # the border's bin holds more than a list does, on both sides of 0: with a border a few tokens off, most draws are others
    rng = np.random.default_rng(V)
    n = 24 if V < 10 ** 6 else 4
    x = rng.normal(0, std, (n, V)).astype(np.float32)
    u = rng.random(n)
    base.check_sample(x, u, t=t, p=p, dtype=dtype)
    base.check_sample(x, u, t=t, p=p, k=V * 3 // 4, dtype=dtype)


def check_border(x, u, p, dtype):
    """As test_gpu_serving.check_sample, where p of the sum falls on a token's end: sums are within 2^-20 of the row's
    total S, so the prefix that reaches p S is that of some p' S with |p' - p| <= 2^-20, one token more or fewer where
    a token weighs more than that, and every running sum over the kept ones is that of this other prefix."""
    import torch
    n = len(x)
    full = torch.from_numpy(np.asarray(x, np.float32)).to(getattr(torch, dtype))
    p, u = np.asarray(p, np.float32), np.asarray(u, np.float32)
    ids = torch.full((n,), -9, dtype=torch.int32, device="cuda")
    base.moe().sample(full.cuda(), base.dev(u), ids, top_p=base.dev(p))
    got, vals = ids.cpu().numpy(), full.double().numpy()
    for r in range(n):
        ok = []
        for d in (0.0, -2.0 ** -20, 2.0 ** -20):
            w = S.kept(vals[r], 1.0, 0, float(p[r]) + d, 0.0)
            c = np.cumsum(w)
            goal, slack = float(u[r]) * c[-1], 2.0 ** -18 * c[-1]
            ok.append(w[got[r]] > 0 and c[got[r]] - w[got[r]] <= goal + slack and goal - slack <= c[got[r]])
        assert any(ok), r


@pytest.mark.parametrize("V", [20000, 200000])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_sample_nucleus_at_the_edges_of_bins(V, dtype):
    # equal tokens whose weights are 2^(-i / 16), p where their sums end: the first histogram's rounding may name the bin next to it
    rng = np.random.default_rng(7)
    n = 24 if V < 10 ** 5 else 6
    level = -np.log(2) / 16 * rng.integers(0, 40, (n, V))
    w = np.sort(np.exp(level), 1)[:, ::-1]
    for shift in (-1e-6, 0.0, 1e-6):
        at = rng.integers(50, V - 50, n)
        p = np.cumsum(w, 1)[np.arange(n), at] / w.sum(1) + shift
        check_border(level, rng.random(n), p, dtype)


@pytest.mark.parametrize("gap,steps", [(22.5, 150), (23.0, 90), (25.0, 15), (26.5, 4), (27.2, 2)])
@pytest.mark.parametrize("k", [0, 100000])
def test_sample_nucleus_that_ends_far_below_the_first(gap, steps, k):
    # one token next to 1, the others e^-gap each, 1 - p about half of them; the largest u then falls just before the
    # last kept ones.  Of their sum: weights are within 2^-21 of themselves and the first token's lane (of at least
    # 512) loses what others it has, V / 512 of V: 2^-9 in all.
    rng = np.random.default_rng(3)
    V, n = 128000, 4
    x = rng.normal(0, 0.3, (n, V)).astype(np.float32) - np.float32(gap)
    x[:, 0] = 0.0
    p = np.float32(1 - steps * 2.0 ** -24)
    got = base.check_sample(x, LAST, p=p, k=k)
    for r in range(n):
        w = S.kept(x[r], 1.0, k, float(p), 0.0)
        c = np.cumsum(w) - 1                                # of the others, up to each token
        goal = max(float(LAST) * (1 + c[-1]) - 1, 0.0)      # 0: the first token itself
        assert abs(c[got[r]] - goal) <= 2.0 ** -9 * c[-1], r


@pytest.mark.parametrize("gap", [20.0, 24.0, 30.0])
def test_sample_nucleus_cuts_equal_tokens_far_below_the_first(gap):
    # top-k ends among equal tokens, and top-p leaves half of the kept ones of them: counted by u at their ends
    V, n, k = 40000, 4, 30000
    x = np.full((n, V), -gap, np.float32)
    x[:, 0] = 0.0
    tail = (k - 1) * np.exp(-gap)
    p = np.float32(1 - 0.5 * tail)
    got = base.check_sample(x, LAST, p=p, k=k)
    c = np.cumsum(S.kept(x[0], 1.0, k, float(p), 0.0)) - 1
    goal = max(float(LAST) * (1 + c[-1]) - 1, 0.0)
    assert np.all(np.abs(c[got] - goal) <= 2.0 ** -9 * c[-1])


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("busy", ["default", "own"])
def test_a_plan_made_while_streams_are_busy(busy):
    # its workspace is cleared after what is queued on the block of memory that it gets, and before its own first call
    import torch
    rng = np.random.default_rng(8)
    P, D, kv, H, lens = 64, 64, 1, 8, [9000, 20, 4000]
    c, table = base.sequences(rng, P, lens, [1] * 3, 141, 220, kv, D, poison=False)
    d, ld, td = [base.dev(x) for x in c], base.dev(np.array(lens, np.int32)), base.dev(table)
    qd, q = base.bf16(rng.normal(0, 0.25, (3, H, D)))
    size = base.moe().Kv8(H, kv, D, P, 220, cache=d).ws.numel()
    ref, tol = S.attend(*c, P, q, range(4), lens, table)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            old = torch.empty(size, dtype=torch.uint8, device="cuda")
            with torch.cuda.stream(torch.cuda.default_stream() if busy == "default" else side):
                torch.cuda._sleep(20_000_000)               # some 10 ms
            old.fill_(255)
            del old
            plan = base.moe().Kv8(H, kv, D, P, 220, cache=d)
            out = torch.zeros((3, H, D), dtype=torch.bfloat16, device="cuda")
            plan.attend(qd, ld, td, out)
        side.synchronize()
        assert (np.abs(out.double().cpu().numpy() - ref) / tol).max() <= 1
        assert plan.device_status() == 0


@pytest.mark.parametrize("P,D", [(16, 64), (32, 128), (64, 64)])
@pytest.mark.parametrize("H", [4, 16])
def test_attend_nan_in_every_place_behind_a_sequence(P, D, H):
    # what a sequence does not see is set to 0 in shared memory by other lanes than those that read it
    rng = np.random.default_rng(9)
    base.check_attend(rng, P, D, 1, H, list(range(1, 130)), [1] * 129)
    base.check_attend(rng, P, D, 1, H, list(range(40, 140)), [1] * 100, window=37)
    base.check_attend(rng, P, D, 1, H, list(range(4, 70)), [3] * 66, sinks=False)


@pytest.mark.parametrize("rows", [[6, 1], [40, 3]])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 4, 2 ** 30])
def test_attend_the_largest_windows(rows, window):
    # with rows before the sequence's beginning: position - window goes past 32 bits
    rng = np.random.default_rng(4)
    base.check_attend(rng, 16, 64, 2, 8, [3, 200], rows, window=window)
    base.check_attend(rng, 64, 128, 2, 8, [rows[0] - 1, 200], rows, window=window, sinks=False)


@pytest.mark.parametrize("rows", [[5, 7, 4], [30, 90, 8]])
@pytest.mark.parametrize("window", [0, 20])
def test_attend_a_sequence_that_goes_on_past_the_rows(rows, window):
    # as where the page tables had room for fewer tokens than there are: the rows that are there keep their positions
    import torch
    rng = np.random.default_rng(5)
    P, D, kv, H, lens = 16, 64, 2, 8, [50, 130, 70]
    c, table = base.sequences(rng, P, lens, rows, 9, 30, kv, D, poison=False)
    starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    qd, q = base.bf16(rng.normal(0, 0.25, (starts[-1], H, D)))
    plan = base.moe().Kv8(H, kv, D, P, 30, sliding_window=window, cache=[base.dev(x) for x in c])
    ref, tol = S.attend(*c, P, q, starts, lens, table, window, floor=2.0 ** -31)
    for n in (starts[1] + 2, starts[2] - 1, starts[2] + 1):
        out = torch.full((starts[-1], H, D), 7.5, dtype=torch.bfloat16, device="cuda")
        plan.attend(qd[:n], base.dev(np.array(lens, np.int32)), base.dev(table), out[:n], starts=base.dev(starts), max_new=max(rows))
        got = out.double().cpu().numpy()
        assert (np.abs(got[:n] - ref[:n]) / tol[:n]).max() <= 1
        assert np.all(got[n:] == 7.5)


@pytest.mark.parametrize("rows", [[1, 1], [3, 2], [40, 70]])
@pytest.mark.parametrize("P,D,lo", [(16, 64, 135), (16, 64, 150), (64, 128, 155), (32, 64, 170)])
def test_attend_large_scores(rows, P, D, lo):
    # up to 2^60: their rounding is more than 1, and the largest one's weight still 1
    rng = np.random.default_rng(6)

    def change(c, table):
        c[3][...] = rng.integers(120, 130, c[3].shape)      # the values' scales as usual

    base.check_attend(rng, P, D, 2, 8, [100, 333], rows, lo=lo, hi=lo + 3, change=change, spread=4.0)
    base.check_attend(rng, P, D, 1, 8, [100, 333], rows, lo=lo, hi=lo + 3, change=change, spread=4.0, window=70)


@pytest.mark.parametrize("rows", [[1, 1], [40, 30]])
@pytest.mark.parametrize("P", [16, 64])
def test_attend_one_large_score_takes_all(rows, P):
    # every query and key a multiple of one direction: the last seen key is the longest by far, and its value the result
    import torch
    rng = np.random.default_rng(10)
    D, lens = 64, [90, 120]
    c, table = base.sequences(rng, P, lens, rows, 8, 20, 1, D, poison=False)
    kk, vv = S.unpack(c[0], c[1], P, D)
    for b, L in enumerate(lens):
        for t in range(L):
            kk[table[b, t // P], t % P] = 0x38 + t % 8          # 1 .. 1.875 times the page's scale
            c[2][table[b, t // P]] = 127 + 24 + 2 * (t // P)
    vv[...] = rng.integers(0x30, 0x40, vv.shape)                # values of one sign and size
    c[:2] = S.pack(kk, vv)
    c[3][...] = 127
    starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    n = int(starts[-1])
    qd, q = base.bf16(np.full((n, 4, D), 3.0))
    plan = base.moe().Kv8(4, 1, D, P, 20, cache=[base.dev(x) for x in c])
    out = torch.zeros((n, 4, D), dtype=torch.bfloat16, device="cuda")
    plan.attend(qd, base.dev(np.array(lens, np.int32)), base.dev(table), out, starts=base.dev(starts), max_new=max(rows))
    got = out.double().cpu().numpy()
    ref, _ = S.attend(*c, P, q, starts, lens, table)
    # scores differ by 2^24 and more or not at all: sums of values and weights of exactly 1, and one division, in fp32
    assert (np.abs(got - ref) <= np.abs(ref) * (2.0 ** -8 + 2.0 ** -16)).all()


@pytest.mark.parametrize("n,V,dtype", [(76, 90000, "float32"), (100, 60000, "float32"), (120, 131072, "bfloat16"), (152, 43000, "float32"),
                                       (30, 210000, "float32"), (310, 170000, "float32")])
def test_sample_row_counts_between_one_and_two_ctas_an_sm(n, V, dtype):
    rng = np.random.default_rng(n)
    x = rng.normal(0, 3, (n, V)).astype(np.float32)
    pick = lambda *v: rng.choice(v, n)   # noqa: E731
    base.check_sample(x, rng.random(n), t=pick(0.5, 0.9), k=pick(0, 40, 700), p=pick(0.9, 0.3, 1.0), mp=pick(0.0, 0.02), dtype=dtype)


@pytest.mark.parametrize("rows", [1, 30])
def test_attend_out_beside_q_in_one_array(rows):
    import torch
    rng = np.random.default_rng(11)
    P, D, kv, H, lens = 16, 64, 2, 4, [50, 130]
    c, table = base.sequences(rng, P, lens, [rows] * 2, 9, 30, kv, D, poison=False)
    plan = base.moe().Kv8(H, kv, D, P, 30, cache=[base.dev(x) for x in c])
    ld, td, n = base.dev(np.array(lens, np.int32)), base.dev(table), 2 * rows
    starts = np.array([0, rows, n], np.int32)
    for first in (0, 1):        # q before out and behind it
        both, vals = base.bf16(rng.normal(0, 0.25, (n, 2 * H + 1, D)))
        q, out = (both[:, :H], both[:, H + 1:]) if first == 0 else (both[:, H + 1:], both[:, :H])
        qv = vals[:, :H] if first == 0 else vals[:, H + 1:]
        plan.attend(q, ld, td, out, starts=base.dev(starts), max_new=rows)
        ref, tol = S.attend(*c, P, qv, starts, lens, table, floor=2.0 ** -31)
        assert (np.abs(out.double().cpu().numpy() - ref) / tol).max() <= 1
        assert np.array_equal(q.double().cpu().numpy(), qv) and np.array_equal(both[:, H].double().cpu().numpy(), vals[:, H])
    both = torch.zeros((n, 2 * H, D), dtype=torch.bfloat16, device="cuda")
    for off in (0, 1, H - 1):   # overlapping in every row
        if n > 1:
            with pytest.raises(base.moe().MoeError, match="overlap"):
                plan.attend(both[:, :H], ld, td, both[:, off:off + H], starts=base.dev(starts), max_new=rows)


@pytest.mark.parametrize("lens,rows", [([100, 70], [1, 1]), ([900, 20], [1, 1]), ([100, 70], [40, 30])])
@pytest.mark.parametrize("sinks", [False, True])
def test_attend_values_of_the_smallest_scales(lens, rows, sinks):
    # pages from 2^-127 on; outputs are bf16 numbers still (2^-126, its smallest normal one, absolutely)
    import torch
    rng = np.random.default_rng(12)
    P, D, kv, H = 16, 64, 2, 4
    c, table = base.sequences(rng, P, lens, rows, 64, 80, kv, D, poison=False)
    for lo, hi in ((0, 6), (4, 12), (12, 40)):
        c[3][...] = rng.integers(lo, hi, c[3].shape)
        s = rng.normal(0, 2, H).astype(np.float32) if sinks else None
        starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        qd, q = base.bf16(rng.normal(0, 0.25, (starts[-1], H, D)))
        plan = base.moe().Kv8(H, kv, D, P, 80, sinks=None if s is None else base.dev(s), cache=[base.dev(x) for x in c])
        out = torch.zeros((int(starts[-1]), H, D), dtype=torch.bfloat16, device="cuda")
        plan.attend(qd, base.dev(np.array(lens, np.int32)), base.dev(table), out, starts=base.dev(starts), max_new=max(rows))
        # the oracle's absolute 1e-30 is not for these: its other terms at the same scores, values scaled by 2^90
        up = [*c[:3], (c[3] + 90).astype(np.uint8)]
        ref, tol = S.attend(*up, P, q, starts, lens, table, 0, s, None, 2.0 ** -31)
        got = out.double().cpu().numpy() * 2.0 ** 90
        assert (np.abs(got - ref) <= tol + 2.0 ** (90 - 126 - 8)).all(), (lo, (np.abs(got - ref) / tol).max())


@pytest.mark.parametrize("p", [0.0, 1e-9, 1e-4, 0.3, 0.999])
@pytest.mark.parametrize("k", [2, 40, 511, 512, 900, 1500])
def test_sample_nucleus_among_the_equal_tokens_that_top_k_left(p, k):
    rng = np.random.default_rng(14)
    base.check_sample(rng.integers(-2, 3, (8, 4909)), rng.random(8), k=k, p=p)
    base.check_sample(np.zeros((8, 1448)), rng.random(8), k=k, p=p, dtype="bfloat16")
    base.check_sample(np.full((8, 20000), 9984.0), rng.random(8), t=0.1, k=k, p=p)


@pytest.mark.parametrize("V", [2, 30, 700, 30000])
@pytest.mark.parametrize("mp", [1.0, 2.0])
def test_sample_min_p_of_one_keeps_the_largest_only(V, mp):
    # weights of the others within 2^-24 of 1
    rng = np.random.default_rng(15)
    x = -np.abs(rng.normal(0, 1e-7, (12, V))).astype(np.float32)
    x[6:, ::3] = x[6:].max(1, keepdims=True)            # and with many that are the largest
    u = rng.random(12)
    want = [S.sample(np.where(r == r.max(), 1.0, 0.0), float(np.float32(v))) for r, v in zip(x, u)]
    for kw in (dict(), dict(t=0.7), dict(k=V // 2 + 1), dict(k=600), dict(p=0.999), dict(k=5, p=0.9)):
        got = base.check_sample(x, u, mp=mp, **kw)
        if not kw or "t" in kw:
            assert list(got) == want


@pytest.mark.parametrize("rows", [[1, 1], [40, 33]])
def test_append_and_attend_past_32_bit_offsets(rows):
    # the last pages of a cache of 4.6 GB a side: byte offsets past 2^32, against a cache of those pages alone
    import torch
    rng = np.random.default_rng(16)
    P, D, kv, H, pages, lens = 64, 128, 8, 16, 70000, [200, 130]
    plan = base.moe().Kv8(H, kv, D, P, pages)
    used = np.array([69999, 69998, 40000, 65537, 65536, 32769, 1])
    c = base.random_cache(rng, len(used), kv, P, D)
    at = torch.from_numpy(used).cuda()
    for t, x in zip((plan.k, plan.v, plan.k_scale, plan.v_scale), c):
        t[at] = base.dev(x)
    small = np.array([[0, 1, 2, 3], [4, 5, 6, -1]], np.int32)
    table = np.where(small < 0, -1, used[small]).astype(np.int32)
    starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    n = int(starts[-1])
    pos = [np.arange(L - r, L) for L, r in zip(lens, rows)]
    near = np.concatenate([small[b, p // P] * P + p % P for b, p in enumerate(pos)])
    far = np.concatenate([table[b, p // P] * P + p % P for b, p in enumerate(pos)]).astype(np.int32)
    kd, k = base.bf16(rng.normal(0, 1, (n, kv, D)))
    vd, v = base.bf16(rng.normal(0, 1, (n, kv, D)))
    plan.append(kd, vd, base.dev(far))
    ref = S.append(*c, P, k, v, near)
    for t, x in zip((plan.k, plan.v, plan.k_scale, plan.v_scale), ref):
        assert np.array_equal(t[at].cpu().numpy(), x)
    qd, q = base.bf16(rng.normal(0, 0.25, (n, H, D)))
    out = torch.zeros((n, H, D), dtype=torch.bfloat16, device="cuda")
    plan.attend(qd, base.dev(np.array(lens, np.int32)), base.dev(table), out, starts=base.dev(starts), max_new=max(rows))
    want, tol = S.attend(*ref, P, q, starts, lens, small, floor=2.0 ** -31)
    assert (np.abs(out.double().cpu().numpy() - want) / tol).max() <= 1


def test_a_status_that_was_set_is_told_once_and_clears_the_tickets():
    # as a wait that gave up leaves the workspace: the status word, and tickets of jobs that were not joined
    import torch
    rng = np.random.default_rng(17)
    P, D, kv, H, lens = 64, 64, 1, 8, [9000, 5000]
    c, table = base.sequences(rng, P, lens, [1] * 2, 141, 230, kv, D, poison=False)
    plan = base.moe().Kv8(H, kv, D, P, 230, cache=[base.dev(x) for x in c])
    head = plan.ws[(-plan.ws.data_ptr()) % 256:][:8192].view(torch.int32)
    assert plan.device_status() == 0
    head[0], head[1] = 1, 90
    head[16:16 + 160] = 1
    assert plan.device_status() == 1 and plan.device_status() == 0 and bool((head == 0).all())
    qd, q = base.bf16(rng.normal(0, 0.25, (2, H, D)))
    out = torch.zeros((2, H, D), dtype=torch.bfloat16, device="cuda")
    plan.attend(qd, base.dev(np.array(lens, np.int32)), base.dev(table), out)
    ref, tol = S.attend(*c, P, q, range(3), lens, table)
    assert (np.abs(out.double().cpu().numpy() - ref) / tol).max() <= 1 and bool((head == 0).all())


@pytest.mark.parametrize("lens,rows", [([9000, 20, 4000, 700], [1] * 4), ([3000, 50, 900, 1], [8, 3, 5, 1]), ([700, 333, 90, 1500], [300, 33, 90, 1])])
def test_attend_repeats_itself_exactly(lens, rows):
    # joins in a fixed order, whichever CTA comes last
    import torch
    rng = np.random.default_rng(18)
    P, D, kv, H = 32, 64, 2, 16
    c, table = base.sequences(rng, P, lens, rows, -(-max(lens) // P), sum(-(-n // P) for n in lens) + 1, kv, D, poison=False)
    plan = base.moe().Kv8(H, kv, D, P, c[2].shape[0], cache=[base.dev(x) for x in c])
    qd, _ = base.bf16(rng.normal(0, 0.25, (sum(rows), H, D)))
    ld, td = base.dev(np.array(lens, np.int32)), base.dev(table)
    starts = base.dev(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32))
    outs = [torch.zeros((sum(rows), H, D), dtype=torch.bfloat16, device="cuda") for _ in range(12)]
    for i, o in enumerate(outs):
        if i % 3 == 2:      # other work beside it
            torch.randn(1 << 22, device="cuda").sort()
        plan.attend(qd, ld, td, o, starts=starts, max_new=max(rows))
    assert all(torch.equal(o, outs[0]) for o in outs)
