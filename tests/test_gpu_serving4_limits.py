"""The serving step's other operators at the limits that include/moe.h states, on the GPU.  Tolerances as in
test_gpu_serving4.py, or derived at the test."""
import numpy as np
import pytest

from oracle import serving4 as S4
from tests import test_gpu_serving4 as base

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- attention

def check_scales(rng, P, D, kv, H, lens, rows, scales_of, window=0, lo=118, hi=131, prompts=False, spread=0.1):
    """Attention where scales_of (sequence, position, block or None, scale byte) says how large values are.  Scores are within
    a few units of one another, so that no weight is next to nothing: what a row sees counts (flush = 0)."""
    import torch
    width, pages = -(-max(lens) // P), sum(-(-L // P) for L in lens) + 2
    c, table = base.sequences(rng, P, lens, width, pages, kv, D, poison=False, lo=lo, hi=hi)
    codes, scales = S4.unpack(c, P, D)
    scales[0] = rng.integers(124, 128, scales[0].shape)
    for b, t, block, byte in scales_of:
        scales[1][table[b, t // P], t % P, :, slice(None) if block is None else block] = byte
    c = S4.pack(codes, scales)
    starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    qd, q = base.bf16(rng.normal(0, spread, (starts[-1], H, D)))
    plan = base.moe().Kv4(H, kv, D, P, pages, sliding_window=window, cache=base.dev(c))
    out = torch.full((starts[-1], H, D), 7.5, dtype=torch.bfloat16, device="cuda")
    assert base.for_prompts(len(lens), kv, H, max(rows), D) == prompts
    plan.attend(qd, base.dev(np.array(lens, np.int32)), base.dev(table), out, starts=base.dev(starts), max_new=max(rows))
    ref, tol = S4.attend(c, P, q, starts, lens, table, window, weight=2.0 ** -8 if prompts else 2.0 ** -11, flush=0.0)
    base.close(out.double().cpu().numpy(), ref, tol)
    assert plan.device_status() == 0


@pytest.mark.parametrize("P,D", [(16, 64), (32, 128), (64, 64), (64, 128), (32, 64)])
@pytest.mark.parametrize("kv,H", [(1, 1), (1, 8), (2, 6), (1, 16)])
def test_attend_scales_that_only_some_rows_see(P, D, kv, H):
    """Drafted rows of which the last one's values are as large as they can be, and tokens that slide out of the window."""
    rng = np.random.default_rng(P + D + H)
    for byte in (252, 255, 200):
        check_scales(rng, P, D, kv, H, [230, 70], [5, 2], [(0, 229, None, byte), (1, 69, 0, byte)])
        check_scales(rng, P, D, kv, H, [321, 70], [5, 2], [(0, 317, 1, byte), (0, 320, 0, byte)], lo=40, hi=60)
    # positions 225 .. 229 see the last 100: 127 is seen by rows 0 and 1, 126 by row 0
    check_scales(rng, P, D, kv, H, [230, 300], [5, 3], [(0, 127, None, 252), (0, 126, None, 250), (1, 199, 1, 252)], window=100)
    check_scales(rng, P, D, kv, H, [230, 300], [5, 3], [(0, 127, None, 252), (0, 160, 0, 150), (0, 229, 0, 252)], window=100, lo=30, hi=50)


@pytest.mark.parametrize("D,kv,H", [(64, 1, 8), (128, 1, 2), (128, 2, 8)])
def test_attend_scales_that_only_some_rows_see_across_shares(D, kv, H):
    """The same where a sequence is shared by many warps and CTAs: the joins' exponents are the rows' own."""
    rng = np.random.default_rng(D + H)
    check_scales(rng, 32, D, kv, H, [6000], [5], [(0, 5999, None, 252)])
    check_scales(rng, 32, D, kv, H, [6000], [5], [(0, 3002, None, 252), (0, 4500, 0, 10), (0, 1500, 1, 190)], window=2995, lo=60, hi=70)
    check_scales(rng, 32, D, kv, H, [2500, 90, 3000], [3, 2, 4], [(0, 2499, 0, 252), (1, 89, None, 252), (2, 2998, 1, 252)], lo=50, hi=60)


@pytest.mark.parametrize("rows,H", [([1], 1), ([1], 8), ([3], 8)])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_scales_of_every_size_in_one_row(rows, H, D):
    """Every row sees them all: the largest ones are the result, whatever order they come in."""
    rng = np.random.default_rng(H + D)
    up = [(0, t, None, int(b)) for t, b in zip(range(700), np.linspace(1, 252, 700))]
    for what in (up, [(0, 699 - t, None, b) for _, t, _, b in up], [(0, t, None, int(rng.integers(1, 253))) for t in range(700)],
                 [(0, t, int(rng.integers(0, D // 32)), int(rng.integers(1, 253))) for t in range(0, 700, 3)]):
        check_scales(rng, 16, D, 1, H, [700], rows, what)
    check_scales(rng, 32, D, 1, H, [40], rows, [(0, t, None, int(rng.integers(1, 253))) for t in range(40)])


@pytest.mark.parametrize("D,kv,H,most", [(64, 8, 16, 100), (128, 8, 8, 17)])
def test_attend_scales_that_only_some_rows_of_prompts_see(D, kv, H, most):
    rng = np.random.default_rng(most)
    n = 6 if D == 64 else 31
    rows = np.minimum(rng.integers(1, most + 1, n), 20)
    rows[0] = most
    lens = rows + rng.integers(0, 100, n)
    check_scales(rng, 32, D, kv, H, lens, rows, [(b, int(L) - 1, None, 252) for b, L in enumerate(lens)] + [(0, int(lens[0]) - 40, 0, 250)], prompts=True)


@pytest.mark.parametrize("D,H", [(64, 1), (64, 8), (128, 8)])
@pytest.mark.parametrize("window", [0, 30, 2 ** 31 - 1])
def test_attend_rows_far_before_their_sequence(D, H, window):
    """starts that end at 2^31 - 1: the rows that are there stand almost 2^31 before the sequence's first token, and see nothing."""
    import torch
    rng = np.random.default_rng(H)
    P, lens = 64, [67, 100]
    c, table = base.sequences(rng, P, lens, 2, 6, 1, D)
    qd, _ = base.bf16(rng.normal(0, 0.25, (7, H, D)))
    out = torch.full((7, H, D), 7.5, dtype=torch.bfloat16, device="cuda")
    plan = base.moe().Kv4(H, 1, D, P, 6, sliding_window=window, cache=base.dev(c))
    for first in (0, 2):
        out.fill_(7.5)
        plan.attend(qd, base.dev(np.array(lens, np.int32)), base.dev(table), out, starts=base.dev(np.array([first, 2 ** 31 - 1, 2 ** 31 - 1], np.int32)), max_new=9)
        assert bool((out[:first] == 7.5).all()) and bool((out[first:] == 0).all())


# ---------------------------------------------------------------- verification

@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("below", [0.90625, 0.69921875, 0.30078125])
def test_verify_sums_of_the_largest_vocabulary(below, dtype):
    """2^22 tokens of one weight, which 32-bit sums round the same way every time: a lane's 1024 are off by up to 2^-16.3.
    Drafted tokens with u 2^-17.4 of p below p, and above it."""
    V = 1 << 22
    x = np.full((8, V), -below, np.float32)
    x[:, 77] = 0.0
    p = S4.probabilities(x[0], 1.0, 0, 1.0, 0.0)[5]
    u = np.array([p * (1 - 2.0 ** -17.4), 0.5, p * (1 + 2.0 ** -17.4), 0.5] * 2)
    ids, acc = base.check_verify(np.random.default_rng(1), x, [2, 2, 2, 2], np.array([5, 0, 9, 0, V - 1, 0, V // 2, 0]), None, u=u, dtype=dtype)
    assert list(acc) == [1, 0, 1, 0]


def below_a_share(n):
    """1 / n in fp32, which for these n is less than 1 / n: a residual of known size, some 2^-25 of it."""
    q = np.float32(1.0 / n)
    assert float(q) < 1.0 / n
    return q


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n,step", [(11, 3), (1009, 7), (50021, 7), (100019, 3), (149993, 1000), (4100013, 3), (3333331, 1000)])
def test_verify_residuals_of_next_to_nothing(n, step, dtype):
    """n equal logits, so that p is 1 / n to the last bit, and drafts' probabilities that are 1 / n rounded down at every
    step-th token and more than 1 / n at the others: the residual is the rounding, the same at each of those tokens, and 0 at
    the others.  Sums within 2^-20 of their totals choose the token of the middle of each share exactly, or one that is as
    near as that."""
    while float(np.float32(1.0 / n)) >= 1.0 / n:
        n += 1
    q = np.full(n, np.nextafter(below_a_share(n), np.float32(1)), np.float32)
    some = np.arange(2 % n, n, step)
    q[some] = below_a_share(n)
    q[0] = 2.0 / n                                       # the drafted token: not accepted at u = 0.9
    B = 24 if n < 1e6 else 9
    pick = np.linspace(0, len(some) - 1, B).round().astype(int)
    draws = ((pick + 0.5) / len(some)).astype(np.float32)
    import torch
    z = lambda k: torch.zeros(k, dtype=torch.int32, device="cuda")   # noqa: E731
    ids, acc = z(2 * B), z(B)
    x = torch.zeros((2 * B, n), dtype=getattr(torch, dtype), device="cuda")
    base.moe().Verify(2 * B).run(x, z(2 * B), torch.full((2 * B,), 0.9, device="cuda"), base.dev(draws), base.dev(np.arange(0, 2 * B + 1, 2, dtype=np.int32)),
                                 ids, acc, draft_probs=base.dev(np.tile(q, (2 * B, 1))))
    got = ids.cpu().numpy()[::2]
    assert not acc.any() and np.isin(got, some).all()
    at = np.searchsorted(some, got)
    slack = 2.0 ** -20 * len(some)
    assert np.all(np.abs(at + 0.5 - draws.astype(np.float64) * len(some)) <= 0.5 + slack)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_verify_of_single_rows_draws_what_sample_draws(dtype):
    """Rows without drafts against the sampler at the same random numbers: the same token, but where the share lies within the
    two sums' bounds (2^-19) of a border."""
    import torch
    rng = np.random.default_rng(9)
    n, V = 300, 4001
    x = torch.from_numpy(rng.normal(0, 2.5, (n, V)).astype(np.float32)).to(getattr(torch, dtype)).cuda()
    t, k = rng.choice([0.0, 0.6, 1.0, 1.4], n).astype(np.float32), rng.choice([0, 1, 40, 900], n).astype(np.int32)
    p, mp = rng.choice([1.0, 0.95, 0.5], n).astype(np.float32), rng.choice([0.0, 0.02], n).astype(np.float32)
    u = rng.random(n).astype(np.float32)
    z = lambda k: torch.zeros(k, dtype=torch.int32, device="cuda")   # noqa: E731
    a, b, acc = z(n), z(n), z(n)
    opt = dict(temperature=base.dev(t), top_k=base.dev(k), top_p=base.dev(p), min_p=base.dev(mp))
    base.moe().sample(x, base.dev(u), a, **opt)
    base.moe().Verify(n).run(x, z(n), base.dev(u), base.dev(u), base.dev(np.arange(n + 1, dtype=np.int32)), b, acc, **opt)
    a, b, x = a.cpu().numpy(), b.cpu().numpy(), x.double().cpu().numpy()
    assert not acc.any()
    for i in np.flatnonzero(a != b):
        c = np.cumsum(S4.probabilities(x[i], float(t[i]), int(k[i]), float(p[i]), float(mp[i])))
        lo, hi = sorted((a[i], b[i]))
        assert abs(float(u[i]) - c[lo]) <= 2.0 ** -19 and c[hi - 1] - c[lo] <= 2.0 ** -19, i


# ---------------------------------------------------------------- angles

def test_rotate_negative_frequencies_keep_their_angles():
    """Far positions whose angles are whole turns but for their frequencies' last bits: sines of next to nothing show the
    angle's error, which is at most 2^-25 of a turn.  (The frequency's own product with the position is exact to 2^-40.)"""
    import torch
    pos = 2 ** 31 - 1
    turns = np.array([256, 768, 1280, 1792, 2304, 2816, 1, 12345] * 4)
    freqs = np.where(np.arange(32) % 16 < 8, -1, 1) * 2 * np.pi * turns / pos
    x = np.zeros((1, 1, 64))
    x[..., 32:] = 1.0                                     # (0, 1) -> (-sin, cos)
    xd, _ = base.bf16(x)
    base.moe().Rotary(64, freqs).apply(xd, None, base.dev(np.array([pos], np.int32)))
    got, angle = xd.double().cpu().numpy()[0, 0], freqs * pos
    assert np.all(np.abs(got[:32] + np.sin(angle)) <= 2 * np.pi * 2.0 ** -25)
    assert np.all(got[32:] == 1.0)
