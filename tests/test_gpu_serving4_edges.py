"""Edges of the serving step's other operators on the GPU: largest sizes and values, busy streams, shared workspaces, states
left by earlier calls.  Tolerances as in test_gpu_serving4.py."""
import numpy as np
import pytest

from oracle import serving4 as S4
from tests import test_gpu_serving4 as base

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("busy", ["default", "own"])
def test_a_plan_made_while_streams_are_busy(busy):
    # its workspace is cleared after what is queued on the block of memory that it gets, and before its own first call
    import torch
    rng = np.random.default_rng(8)
    P, D, kv, H, lens = 64, 64, 1, 8, [9000, 20, 4000]
    c, table = base.sequences(rng, P, lens, 141, 220, kv, D)
    d, ld, td = base.dev(c), base.dev(np.array(lens, np.int32)), base.dev(table)
    qd, q = base.bf16(rng.normal(0, 0.25, (3, H, D)))
    size = base.moe().Kv4(H, kv, D, P, 220, cache=d).ws.numel()
    ref, tol = S4.attend(c, P, q, range(4), lens, table)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            old = torch.empty(size, dtype=torch.uint8, device="cuda")
            with torch.cuda.stream(torch.cuda.default_stream() if busy == "default" else side):
                torch.cuda._sleep(20_000_000)               # some 10 ms
            old.fill_(255)
            del old
            plan = base.moe().Kv4(H, kv, D, P, 220, cache=d)
            out = torch.zeros((3, H, D), dtype=torch.bfloat16, device="cuda")
            plan.attend(qd, ld, td, out)
        side.synchronize()
        base.close(out.double().cpu().numpy(), ref, tol)
        assert plan.device_status() == 0


@pytest.mark.parametrize("P,D", [(16, 64), (32, 128), (64, 64)])
@pytest.mark.parametrize("H", [4, 16])
def test_attend_anything_in_every_place_behind_a_sequence(P, D, H):
    rng = np.random.default_rng(9)
    base.check_attend(rng, P, D, 1, H, list(range(1, 130)), [1] * 129)
    base.check_attend(rng, P, D, 1, H, list(range(40, 140)), [1] * 100, window=37)
    base.check_attend(rng, P, D, 1, H, list(range(4, 70)), [3] * 66, sinks=False)


@pytest.mark.parametrize("rows,H", [([6, 1], 8), ([40, 3], 8), ([40] * 80, 32)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 4, 2 ** 30])
def test_attend_the_largest_windows(rows, H, window):
    # with rows before the sequence's beginning: position - window goes past 32 bits
    rng = np.random.default_rng(4)
    many = len(rows) > 2
    lens = [3, 100] + [5] * (len(rows) - 2)
    rows = rows[:2] + [1] * (len(rows) - 2)
    base.check_attend(rng, 16, 64, 2, H, lens, rows, window=window, prompts=many)
    base.check_attend(rng, 64, 128, 2, H, [rows[0] - 1] + lens[1:], rows, window=window, sinks=False, prompts=many)


@pytest.mark.parametrize("rows", [[5, 7, 4], [30, 90, 8]])
@pytest.mark.parametrize("window", [0, 20])
def test_attend_a_sequence_that_goes_on_past_the_rows(rows, window):
    # as where the page tables had room for fewer tokens than there are: the rows that are there keep their positions
    import torch
    rng = np.random.default_rng(5)
    P, D, kv, H, lens = 16, 64, 2, 8, [50, 130, 70]
    c, table = base.sequences(rng, P, lens, 9, 30, kv, D)
    starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    qd, q = base.bf16(rng.normal(0, 0.25, (starts[-1], H, D)))
    plan = base.moe().Kv4(H, kv, D, P, 30, sliding_window=window, cache=base.dev(c))
    ref, tol = S4.attend(c, P, q, starts, lens, table, window)
    for n in (starts[1] + 2, starts[2] - 1, starts[2] + 1):
        out = torch.full((starts[-1], H, D), 7.5, dtype=torch.bfloat16, device="cuda")
        plan.attend(qd[:n], base.dev(np.array(lens, np.int32)), base.dev(table), out[:n], starts=base.dev(starts), max_new=max(rows))
        got = out.double().cpu().numpy()
        base.close(got[:n], ref[:n], tol[:n])
        assert np.all(got[n:] == 7.5)


@pytest.mark.parametrize("rows,kv,H", [([1, 1], 2, 8), ([3, 2], 2, 8), ([40, 70], 2, 8), ([30] + [2] * 23, 8, 64)])
@pytest.mark.parametrize("P,D,lo", [(16, 64, 135), (16, 64, 150), (64, 128, 155), (32, 64, 170)])
def test_attend_large_scores(rows, kv, H, P, D, lo):
    # up to 2^60: their rounding is more than 1, and the largest one's weight still 1
    rng = np.random.default_rng(6)

    def change(c, table):
        codes, scales = S4.unpack(c, P, D)
        scales[1] = rng.integers(120, 130, scales[1].shape)      # the values' scales as usual
        return S4.pack(codes, scales)

    lens = [100, 333] + [40] * (len(rows) - 2)
    many = True if len(rows) > 2 else None
    base.check_attend(rng, P, D, kv, H, lens, rows, lo=lo, hi=lo + 3, change=change, spread=4.0, poison=False, prompts=many)
    base.check_attend(rng, P, D, kv, H, lens, rows, lo=lo, hi=lo + 3, change=change, spread=4.0, window=70, poison=False, prompts=many)


@pytest.mark.parametrize("D,most", [(64, 12), (128, 6)])
def test_attend_prompts_of_more_sequences_than_lanes(D, most):
    rng = np.random.default_rng(18)
    rows = np.minimum(rng.integers(0, most + 1, 40), 3)
    rows[[5, 39]] = most
    check = lambda lens, **kw: base.check_attend(rng, 16, D, 8, 64, lens, rows, max_new=most, prompts=True, **kw)
    check(rows + rng.integers(0, 90, 40))
    check(rows + rng.integers(-2, 200, 40).clip(0), window=50)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("width", [None, 3, 9])
def test_attend_prompts_of_equal_sequences_and_past_the_table(D, width):
    # tiles of the same length, of none, and of more tokens than their table has
    rng = np.random.default_rng(19)
    rows = [33, 33, 0, 33, 1, 33, 70] + [33] * 13
    lens = [160, 160, 160, 20, 160, 160, 300] + [160] * 12 + [0]
    base.check_attend(rng, 16, D, 8, 64, lens, rows, width=width, max_new=70, prompts=True)


def test_attend_large_scores_among_usual_ones():
    # scores that pass 2^17 only behind the first tokens, and rows that do beside rows that do not
    rng = np.random.default_rng(7)

    def change(c, table):
        codes, scales = S4.unpack(c, 16, 64)
        scales[0][:, :, :, :] = 125
        for t in (70, 150, 151):
            scales[0][table[0, t // 16], t % 16] = 150
        return S4.pack(codes, scales)

    for rows in ([1, 1], [5, 2], [30, 40]):
        base.check_attend(rng, 16, 64, 1, 8, [300, 64], rows, change=change, spread=1.0, poison=False)


@pytest.mark.parametrize("rows", [[1, 1], [3, 2], [40, 33]])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale,spread,lo", [(1e-25, 2.0 ** -40, 224), (None, 2.0 ** -118, 224), (2e-30, 2.0 ** -6, 222), (1e20, 2.0 ** -100, 124)])
def test_attend_small_queries_and_large_keys(rows, D, scale, spread, lo):
    # a row's scale, undone, times softmax_scale is far below fp32's smallest number, the scores are not
    rng = np.random.default_rng(17)

    def change(c, table):
        codes, scales = S4.unpack(c, 16, D)
        scales[1] = rng.integers(120, 130, scales[1].shape)
        return S4.pack(codes, scales)

    base.check_attend(rng, 16, D, 2, 8, [300, 64], rows, scale=scale, spread=spread, lo=lo, hi=lo + 3, change=change, poison=False)


@pytest.mark.parametrize("rows", [[1, 1], [3, 2], [40, 33]])
def test_append_read_and_attend_past_32_bit_offsets(rows):
    # the last pages of a cache of 4.9 GB: byte offsets past 2^32, against a cache of those pages alone
    import torch
    rng = np.random.default_rng(16)
    P, D, kv, H, pages, lens = 64, 128, 8, 16, 70000, [200, 130]
    plan = base.moe().Kv4(H, kv, D, P, pages)
    used = np.array([69999, 69998, 61684, 65537, 65536, 32769, 1])
    c = base.random_cache(rng, len(used), kv, P, D)
    at = torch.from_numpy(used).cuda()
    plan.cache[at] = base.dev(c)
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
    ref = S4.append(c, P, k, v, near)
    assert np.array_equal(plan.cache[at].cpu().numpy(), ref)
    kd.zero_(), vd.zero_()
    plan.read(base.dev(far), kd, vd)
    for t, x in zip((kd, vd), S4.read(ref, P, D, near)):
        assert np.array_equal(t.double().cpu().numpy(), x)
    qd, q = base.bf16(rng.normal(0, 0.25, (n, H, D)))
    out = torch.zeros((n, H, D), dtype=torch.bfloat16, device="cuda")
    plan.attend(qd, base.dev(np.array(lens, np.int32)), base.dev(table), out, starts=base.dev(starts), max_new=max(rows))
    base.close(out.double().cpu().numpy(), *S4.attend(ref, P, q, starts, lens, small))


def test_prompts_past_32_bit_offsets():
    import torch
    rng = np.random.default_rng(17)
    P, D, kv, H, pages = 64, 128, 8, 8, 70000
    rows = np.array([17] + [3] * 30)
    lens = rows + rng.integers(0, 90, 31)
    plan = base.moe().Kv4(H, kv, D, P, pages)
    used = rng.permutation(np.arange(69000, 70000))[:70]
    c, small = base.sequences(rng, P, lens, 2, 70, kv, D)
    small = np.where((small >= 0) & (small < 70), small, -1).astype(np.int32)
    plan.cache[torch.from_numpy(used).cuda()] = base.dev(c)
    table = np.where(small < 0, -1, used[small]).astype(np.int32)
    starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    qd, q = base.bf16(rng.normal(0, 0.25, (starts[-1], H, D)))
    out = torch.zeros_like(qd)
    assert base.for_prompts(31, kv, H, 17, D)
    plan.attend(qd, base.dev(lens.astype(np.int32)), base.dev(table), out, starts=base.dev(starts), max_new=17)
    base.close(out.double().cpu().numpy(), *S4.attend(c, P, q, starts, lens, small, weight=2.0 ** -8))


def test_a_status_that_was_set_is_told_once_and_clears_the_tickets():
    # as a wait that gave up leaves the workspace: the status word, and tickets of jobs that were not joined
    import torch
    rng = np.random.default_rng(17)
    P, D, kv, H, lens = 64, 64, 1, 8, [9000, 5000]
    c, table = base.sequences(rng, P, lens, 141, 230, kv, D)
    plan = base.moe().Kv4(H, kv, D, P, 230, cache=base.dev(c))
    head = plan.ws[(-plan.ws.data_ptr()) % 256:][:8192].view(torch.int32)
    assert plan.device_status() == 0
    head[0], head[1] = 1, 95
    head[16:16 + 160] = 1
    assert plan.device_status() == 1 and plan.device_status() == 0 and bool((head == 0).all())
    qd, q = base.bf16(rng.normal(0, 0.25, (2, H, D)))
    out = torch.zeros((2, H, D), dtype=torch.bfloat16, device="cuda")
    plan.attend(qd, base.dev(np.array(lens, np.int32)), base.dev(table), out)
    base.close(out.double().cpu().numpy(), *S4.attend(c, P, q, range(3), lens, table))
    assert bool((head == 0).all())


@pytest.mark.parametrize("lens,rows", [([9000, 20, 4000, 700], [1] * 4), ([3000, 50, 900, 1], [8, 3, 5, 1]), ([700, 333, 90, 1500], [300, 33, 90, 1])])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_repeats_itself_exactly(lens, rows, D):
    # joins in a fixed order, whichever CTA comes last
    import torch
    rng = np.random.default_rng(18)
    P, kv, H = 32, 2, 16
    pages = sum(-(-n // P) for n in lens) + 1
    c, table = base.sequences(rng, P, lens, -(-max(lens) // P), pages, kv, D)
    plan = base.moe().Kv4(H, kv, D, P, pages, cache=base.dev(c))
    qd, _ = base.bf16(rng.normal(0, 0.25, (sum(rows), H, D)))
    ld, td = base.dev(np.array(lens, np.int32)), base.dev(table)
    starts = base.dev(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32))
    outs = [torch.zeros((sum(rows), H, D), dtype=torch.bfloat16, device="cuda") for _ in range(12)]
    for i, o in enumerate(outs):
        if i % 3 == 2:      # other work beside it
            torch.randn(1 << 22, device="cuda").sort()
        plan.attend(qd, ld, td, o, starts=starts, max_new=max(rows))
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_plans_of_two_shapes_share_a_workspace():
    import torch
    rng = np.random.default_rng(19)
    made = []
    big = None
    for D, H, lens in ((128, 8, [3000, 70]), (64, 16, [5000, 300])):
        pages = sum(-(-n // 32) for n in lens) + 1
        c, table = base.sequences(rng, 32, lens, -(-max(lens) // 32), pages, 1, D)
        plan = base.moe().Kv4(H, 1, D, 32, pages, cache=base.dev(c), workspace=big)
        big = big or plan
        qd, q = base.bf16(rng.normal(0, 0.25, (2, H, D)))
        made.append((plan, qd, base.dev(np.array(lens, np.int32)), base.dev(table), torch.zeros_like(qd), S4.attend(c, 32, q, range(3), lens, table)))
    for _ in range(5):
        for plan, qd, ld, td, out, _ in made:
            plan.attend(qd, ld, td, out)
    for _, _, _, _, out, (ref, tol) in made:
        base.close(out.double().cpu().numpy(), ref, tol)
    with pytest.raises(base.moe().MoeError):
        base.moe().Kv4(4, 1, 128, 32, 4, workspace=made[1][0].__class__(4, 1, 64, 32, 4))


@pytest.mark.parametrize("rows", [[1, 1], [5, 2], [40, 33]])
def test_attend_out_beside_q_in_one_array(rows):
    import torch
    rng = np.random.default_rng(20)
    P, D, kv, H, lens = 32, 128, 1, 4, [70, 300]
    c, table = base.sequences(rng, P, lens, 10, 16, kv, D)
    starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    both, x = base.bf16(rng.normal(0, 0.25, (starts[-1], 2 * H + 1, D)))
    plan = base.moe().Kv4(H, kv, D, P, 16, cache=base.dev(c))
    plan.attend(both[:, :H], base.dev(np.array(lens, np.int32)), base.dev(table), both[:, H + 1:], starts=base.dev(starts), max_new=max(rows))
    got = both.double().cpu().numpy()
    base.close(got[:, H + 1:], *S4.attend(c, P, x[:, :H], starts, lens, table))
    assert np.array_equal(got[:, :H + 1], x[:, :H + 1])
    for bad in (both[:, H - 1:2 * H - 1], both[:, :H]):
        with pytest.raises(base.moe().MoeError):
            plan.attend(both[:, :H], base.dev(np.array(lens, np.int32)), base.dev(table), bad, starts=base.dev(starts), max_new=max(rows))


def test_rotate_on_a_stream_into_strided_places_of_one_array():
    import torch
    rng = np.random.default_rng(21)
    n, H, kv, D = 300, 6, 2, 128
    x = rng.normal(0, 1, (n, H + kv, D))
    xd, x = base.bf16(x)
    to = torch.full((n, H + kv + 2, D), 7.5, dtype=torch.bfloat16, device="cuda")
    pos = rng.integers(0, 4000, n).astype(np.int32)
    freqs = rng.random(64)
    plan, side = base.moe().Rotary(D, freqs), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan.apply(xd[:, :H], xd[:, H:], base.dev(pos), to[:, 2:H + 2], to[:, H + 2:], stream=side)
    side.synchronize()
    got = to.double().cpu().numpy()
    base.close(got[:, 2:], *S4.rotate(x, pos, freqs))
    assert np.all(got[:, :2] == 7.5)
    for bad in ((xd[:, :H], xd[:, H:], xd[:, 1:H + 1], to[:, :kv]), (xd[:, :H], xd[:, H:], to[:, :H], to[:, H - 1:H + 1])):
        with pytest.raises(base.moe().MoeError):
            plan.apply(bad[0], bad[1], base.dev(pos), bad[2], bad[3])


def test_verify_calls_of_fewer_rows_and_none():
    import torch
    rng = np.random.default_rng(22)
    plan = base.moe().Verify(6)
    z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device="cuda")   # noqa: E731
    acc = z(3) + 9
    plan.run(z(0, 50, t=torch.float32), z(0), z(0, t=torch.float32), z(3, t=torch.float32), z(4), z(0), acc)
    assert acc.tolist() == [0, 0, 0]
    plan.run(z(0, 50, t=torch.float32), z(0), z(0, t=torch.float32), z(0, t=torch.float32), z(1), z(0), z(0))
    with pytest.raises(base.moe().MoeError):
        plan.run(z(7, 50, t=torch.float32), z(7), z(7, t=torch.float32), z(3, t=torch.float32), z(4), z(7), acc)
    # starts past the rows: what is there is a sequence's end
    x = rng.normal(0, 1, (4, 50)).astype(np.float32)
    ids = z(4) + 77
    plan.run(base.dev(x), base.dev(np.argmax(x, 1).astype(np.int32)), z(4, t=torch.float32), z(3, t=torch.float32),
             base.dev(np.array([1, 3, 9, 12], np.int32)), ids, acc, top_k=base.dev(np.array([1, 1, 1], np.int32)))
    assert acc.tolist() == [1, 0, 0] and ids.tolist() == [77, int(np.argmax(x[1])), int(np.argmax(x[2])), int(np.argmax(x[3]))]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_verify_draws_from_wide_nuclei(dtype):
    # tens of thousands of tokens kept: the drawn one is the oracle's own, or beside a border that is as near
    rng = np.random.default_rng(23)
    V, n = 60000, 24
    x = rng.normal(0, 1.0, (2 * n, V))
    q, d = base.drafted(rng, x, 0.7)
    base.check_verify(rng, x, [2] * n, d, q, p=0.95, dtype=dtype)
    base.check_verify(rng, x, [2] * n, d, q, t=1.7, dtype=dtype)
