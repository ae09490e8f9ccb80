"""The serving step's other operators on the GPU against oracle/serving4.py (64 bits): norms and rotary positions, the
4-bit paged cache (append, read, attention), the verification of drafted tokens, and a run of them together.

Tolerances.  Codes, scales and what is read are equal.  Rotations and attention: the oracle gives with each output how
far it may be off, from the roundings' sizes.  Verification: a weight e^z, z <= 0, is off by at most
(2^-22 + |z| 2^-22) of itself, and |z| e^z <= 0.37, so probabilities and running sums are within 2^-20 of the total; a
drafted token may be taken either way where u q(x) is within 2^-18 of p(x), and the drawn token must be one whose
interval of the running sum, widened by 2^-18 of p's total, holds its share of the total."""
import numpy as np
import pytest

from oracle import serving as S
from oracle import serving4 as S4

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


def close(got, ref, tol):
    nan = np.isnan(ref)
    assert not (np.isnan(got) != nan).any()
    far = (np.abs(got - ref) / tol)[~nan]
    assert not far.size or far.max() <= 1, far.max()


# ---------------------------------------------------------------- norms and rotary positions

def check_rotate(rng, n, H, kv, D, pairs, axes=1, interleaved=False, norm=True, far=5000, factor=1.0, eps=1e-6, rows=None, in_place=False,
                 positions=None, freqs=None):
    import torch
    x = rng.normal(0, 1, (n, H + 2 * kv, D)) * 2.0 ** rng.integers(-6, 7, (n, H + 2 * kv, 1)) if rows is None else rows
    xd, x = bf16(x)
    freqs = 10000.0 ** (-np.arange(pairs) / max(pairs, 1)) if freqs is None else freqs
    of = None if axes == 1 else rng.integers(0, axes, pairs)
    pos = rng.integers(0, far, (axes, n)).astype(np.int32) if positions is None else positions
    gq, gk = (rng.normal(1, 0.2, D).astype(np.float32) for _ in range(2))
    plan = moe().Rotary(D, freqs, axes=of, n_axes=axes, interleaved=interleaved, eps=eps, factor=factor,
                        q_gamma=dev(gq) if norm else None, k_gamma=dev(gk) if norm else None)
    q, k = xd[:, :H], xd[:, H:H + kv]                    # places of one projection's rows
    if in_place:
        before = xd.clone()
        plan.apply(q, k, dev(pos if axes > 1 else pos[0]))
        qo, ko = q, k
        assert torch.equal(before[:, H + kv:], xd[:, H + kv:])
    else:
        qo, ko = (torch.full((n, h, D), 7.5, dtype=torch.bfloat16, device="cuda") for h in (H, kv))
        plan.apply(q, k, dev(pos), qo, ko)
    live = (pos >= 0).all(0)
    for o, src, g in ((qo, x[:, :H], gq), (ko, x[:, H:H + kv], gk)):
        got = o.double().cpu().numpy()
        ref, tol = S4.rotate(src, pos, freqs, of, interleaved, g if norm else None, eps, factor)
        close(got[live], ref[live], tol[live])
        assert np.array_equal(got[~live], src[~live] if in_place else np.full_like(got[~live], 7.5), equal_nan=True)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_rotate(D, interleaved, norm):
    rng = np.random.default_rng(D + interleaved)
    check_rotate(rng, 1, 1, 1, D, D // 2, interleaved=interleaved, norm=norm)
    check_rotate(rng, 37, 10, 2, D, D // 2, interleaved=interleaved, norm=norm, far=2 ** 31 - 1)
    check_rotate(rng, 33, 5, 1, D, 8, interleaved=interleaved, norm=norm, factor=1.37)              # most dims stay
    check_rotate(rng, 20, 3, 3, D, D // 4, axes=3, interleaved=interleaved, norm=norm, in_place=True)
    check_rotate(rng, 9, 2, 1, D, 0, interleaved=interleaved, norm=norm)                            # norms alone
    check_rotate(rng, 9, 200, 1, D, D // 2, axes=4, interleaved=interleaved, norm=norm)


def test_rotate_many_tokens_padded_rows_and_one_side():
    import torch
    rng = np.random.default_rng(1)
    pos = rng.integers(0, 9000, (1, 1501)).astype(np.int32)
    pos[0, [0, 7, 1500]] = -1
    pos[0, 900:1000] = -(2 ** 31)
    check_rotate(rng, 1501, 6, 2, 64, 32, positions=pos)
    check_rotate(rng, 1501, 6, 2, 64, 32, positions=pos, in_place=True)
    pos = rng.integers(0, 90, (3, 700)).astype(np.int32)
    pos[2, 100:200] = -5                                  # any axis
    check_rotate(rng, 700, 3, 1, 128, 64, axes=3, positions=pos)
    xd, x = bf16(rng.normal(0, 1, (5, 4, 64)))
    out = torch.empty_like(xd)
    plan = moe().Rotary(64, [0.5] * 32)
    plan.apply(xd, None, dev(np.arange(5, dtype=np.int32)), out)
    close(out.double().cpu().numpy(), *S4.rotate(x, np.arange(5), [0.5] * 32))
    plan.apply(xd[:0], xd[:0], dev(np.zeros(0, np.int32)))


@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_rotate_odd_values(eps):
    """Squares that 32 bits do not hold, rows of nothing, infinities and NaN: only their own heads show them."""
    rng = np.random.default_rng(2)
    x = rng.normal(0, 1, (12, 5, 64))
    x[0] *= 1e30
    x[1] *= 1e-30
    x[2, 1] = 0.0
    x[3, 0, 5], x[4, 1, 60], x[5, 2, 0] = np.inf, -np.inf, np.nan
    x[6] *= 2.0 ** 126
    x[7, :, 1:] = 0.0
    with np.errstate(invalid="ignore", divide="ignore"):
        check_rotate(rng, 12, 3, 1, 64, 0, rows=x, eps=eps)
        x[3:6] = 1.0
        check_rotate(rng, 12, 3, 1, 64, 32, rows=x, eps=eps)
    xd, _ = bf16(np.where(np.arange(64) == 3, np.nan, np.ones((2, 2, 64))))
    xd[1, 0] = 1.0
    out = xd.clone()
    moe().Rotary(64, [1.0] * 16).apply(xd, None, dev(np.zeros(2, np.int32)), out)
    bad = np.isnan(out.double().cpu().numpy())
    assert set(np.flatnonzero(bad[0, 0])) == {3, 19} and not bad[1, 0].any()    # its pair, no others


def test_rotate_far_positions_keep_their_angles():
    rng = np.random.default_rng(3)
    pos = np.array([[0, 1, 2 ** 24 + 1, 2 ** 31 - 1, 123456789]], np.int32)
    check_rotate(rng, 5, 2, 1, 64, 32, positions=pos, freqs=np.concatenate([[1.0, 2.0, 7.25, -0.75, 1e-9, 0.0, 3.0, 0.1], rng.random(24)]))


# ---------------------------------------------------------------- the cache

def random_cache(rng, pages, kv, P, D, lo=118, hi=131):
    codes = rng.integers(0, 16, (2, pages, P, kv, D)).astype(np.uint8)
    return S4.pack(codes, rng.integers(lo, hi, (2, pages, P, kv, D // 32)).astype(np.uint8))


def tokens(rng, n, kv, D, spread=6):
    x = rng.normal(0, 1, (n, kv, D)) * 2.0 ** rng.integers(-spread, spread, (n, kv, 1)) * 2.0 ** rng.integers(-3, 3, (n, kv, D))
    return bf16(x)[1]


def run_append(c, P, D, xk, xv, slots, calls=1):
    d = dev(c)
    plan = moe().Kv4(c.shape[1], c.shape[1], D, P, c.shape[0], cache=d)
    both, _ = bf16(np.concatenate([xk, xv], 1))
    sl = dev(np.asarray(slots, np.int32))
    for part in np.array_split(np.arange(len(slots)), calls):
        a, z = part[0], part[-1] + 1
        plan.append(both[a:z, :xk.shape[1]], both[a:z, xk.shape[1]:], sl[a:z])
    return plan, d.cpu().numpy()


@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv", [1, 3, 8])
def test_append_and_read(P, D, kv):
    import torch
    rng = np.random.default_rng(P + D + kv)
    c = random_cache(rng, 9, kv, P, D)
    slots = rng.permutation(9 * P)[:70]                  # in any order
    slots = np.concatenate([slots[:30], [-1, 9 * P, 2 ** 31 - 1, -2 ** 31], slots[30:]])
    xk, xv = tokens(rng, len(slots), kv, D), tokens(rng, len(slots), kv, D)
    ref = S4.append(c, P, xk, xv, slots)
    plan, got = run_append(c, P, D, xk, xv, slots)
    assert np.array_equal(got, ref)
    assert np.array_equal(run_append(c, P, D, xk, xv, slots, calls=9)[1], ref)
    both = torch.full((len(slots), 2 * kv + 1, D), 7.5, dtype=torch.bfloat16, device="cuda")
    plan.read(dev(slots.astype(np.int32)), both[:, :kv], both[:, kv + 1:])
    live = (slots >= 0) & (slots < 9 * P)
    got = both.double().cpu().numpy()
    k, v = S4.read(ref, P, D, slots[live])
    assert np.array_equal(got[live, :kv], k) and np.array_equal(got[live, kv + 1:], v)
    assert np.all(got[:, kv] == 7.5) and np.all(got[~live] == 7.5)


def test_append_odd_values_and_the_codes_of_the_activation_encoder():
    import torch
    rng = np.random.default_rng(4)
    P, D, kv, n = 32, 64, 2, 200
    c = random_cache(rng, 8, kv, P, D)
    xk, xv = tokens(rng, n, kv, D), tokens(rng, n, kv, D)
    _, got = run_append(c, P, D, xk, xv, np.arange(n))
    codes, scales = S4.unpack(got, P, D)
    for side, x in enumerate((xk, xv)):                  # the same blocks through moe_mx_quantize_fp4
        xd = bf16(x)[0].view(torch.int16)
        cd, sd = torch.empty(n * kv * D // 2, dtype=torch.uint8, device="cuda"), torch.empty(n * kv * D // 32, dtype=torch.uint8, device="cuda")
        moe().mx_quantize_fp4(xd.view(n * kv, D), cd, sd)
        both = cd.cpu().numpy().reshape(n, kv, D // 2)
        both = np.stack([both & 15, both >> 4], -1).reshape(n, kv, D)
        assert np.array_equal(codes[side].reshape(-1, kv, D)[:n], both)
        assert np.array_equal(scales[side].reshape(-1, kv, D // 32)[:n], sd.cpu().numpy().reshape(n, kv, -1))
    xk[3, 0, 3], xk[4, 1, 5], xk[5, 1, :], xv[6, 0, 7] = np.inf, -np.inf, np.nan, np.nan
    xk[40:44], xv[40:44] = 0.0, 2.0 ** -133              # nothing, and subnormals
    xv[90:96] = -0.0
    xk[100:110] = np.where(rng.random((10, kv, D)) < 0.5, -1, 1) * 3.3e38
    xv[110:120] *= 2.0 ** -125
    xk[120:130] = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -5.0, -2.5], (10, kv, D))    # ties
    _, got = run_append(c, P, D, xk, xv, np.arange(n))
    assert np.array_equal(got, S4.append(c, P, bf16(xk)[1], bf16(xv)[1], np.arange(n)))


# ---------------------------------------------------------------- attention

def for_prompts(seqs, kv, H, most, D):
    """Does the kernel for prompts take a call (weights in bf16), or that for a few new tokens (in fp16)?  By the rule that the
    choice is made by; where it is told otherwise a test fails by its tolerance or tests less."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows, heads = most * (H // kv), seqs * kv
    tenths = (30 if rows <= 128 else 40) if D == 64 else (16 if rows <= 128 else 21)
    return rows > 16 and 10 * heads * -(-rows // 16) >= -(-heads * -(-rows // 256) // sms) * sms * tenths


def sequences(rng, P, lens, width, pages, kv, D, poison=True, **cache):
    """A cache with each sequence's tokens on pages of its own, anything everywhere else."""
    c = random_cache(rng, pages, kv, P, D, **cache)
    order, at = rng.permutation(pages), 0
    table = rng.integers(-3, pages + 3, (len(lens), width)).astype(np.int32)     # entries past a sequence are anything
    codes, scales = S4.unpack(c, P, D)
    used = np.zeros((pages, P), bool)
    for b, L in enumerate(lens):
        n = min(-(-L // P), width)
        table[b, :n] = order[at:at + n]
        for j in range(n):
            used[order[at + j], :min(P, L - j * P)] = True
        at += n
    assert at <= pages
    if poison:
        codes[:, ~used] = rng.integers(0, 16, codes[:, ~used].shape)
        scales[:, ~used] = rng.choice([0, 1, 200, 252, 253, 254, 255], scales[:, ~used].shape)
        c = S4.pack(codes, scales)
    return c, table


def check_attend(rng, P, D, kv, H, lens, rows, window=0, sinks=True, width=None, pages=None, scale=None, spread=0.25,
                 max_new=None, extra=0, poison=True, change=None, prompts=None, **cache):
    import torch
    lens, rows = list(lens), list(rows)
    width = width or max(1, -(-max(lens) // P))
    pages = pages or sum(-(-L // P) for L in lens) + 3
    c, table = sequences(rng, P, lens, width, pages, kv, D, poison, **cache)
    if change:
        c = change(c, table)
    starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    n = int(starts[-1]) + extra
    qd, q = bf16(rng.normal(0, spread, (n, H + 2, D)))
    qd, q = qd[:, 1:H + 1], q[:, 1:H + 1]                # rows of a wider projection
    s = rng.normal(0, 2, H).astype(np.float32) if sinks else None
    plan = moe().Kv4(H, kv, D, P, pages, sliding_window=window, softmax_scale=scale, sinks=None if s is None else dev(s), cache=dev(c))
    out = torch.full((n, H, D), 7.5, dtype=torch.bfloat16, device="cuda")
    one = all(r == 1 for r in rows) and extra == 0
    most = max_new if max_new is not None else max(rows + [1])
    many = for_prompts(len(lens), kv, H, most, D)        # weights in bf16
    assert prompts is None or prompts == many
    for use in ([False, True] if one else [True]):      # with and without starts
        out.fill_(7.5)
        plan.attend(qd, dev(np.array(lens, np.int32)), dev(table), out, starts=dev(starts) if use else None, max_new=most)
        got = out.double().cpu().numpy()
        ref, tol = S4.attend(c, P, q, starts, lens, table, window, s, scale, weight=2.0 ** -8 if many else 2.0 ** -11)
        for b in range(len(lens)):
            a, z = starts[b], min(starts[b] + most, starts[b + 1])
            close(got[a:z], ref[a:z], tol[a:z])
            assert np.all(got[z:starts[b + 1]] == 7.5)
        assert np.all(got[starts[-1]:] == 7.5)          # rows of no sequence
    assert plan.device_status() == 0
    return got


@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv,H", [(1, 1), (2, 16), (3, 9), (2, 20), (1, 16), (4, 4)])
def test_attend_one_token_a_sequence(P, D, kv, H):
    rng = np.random.default_rng(P * D + H)
    check_attend(rng, P, D, kv, H, [1, 2, P - 1, P, P + 1, 63, 64, 65, 200, 0, 333], [1] * 11, sinks=H % 2 == 0)


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 128, 1000, 2 ** 31 - 1])
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


@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("D,kv,H,most", [(64, 8, 16, 100), (64, 2, 32, 200), (128, 8, 8, 17), (128, 4, 20, 40), (128, 1, 16, 260)])
def test_attend_prompts(P, D, kv, H, most):
    rng = np.random.default_rng(P + H + most)
    n = {(64, 16): 6, (64, 32): 5, (128, 8): 31, (128, 20): 9, (128, 16): 6}[D, H]
    rows = np.minimum(rng.integers(1, most + 1, n), rng.integers(1, 60, n))      # (the oracle is slow)
    rows[0] = most
    lens = rows + rng.integers(0, 150, n)
    lens[0] = most
    lens[1], rows[1] = rows[1] // 2, rows[1]                                     # rows before the sequence's beginning
    check_attend(rng, P, D, kv, H, lens, rows, max_new=most, prompts=True, sinks=bool(P % 64))
    check_attend(rng, P, D, kv, H, lens, rows, max_new=most, prompts=True, window=37, extra=3)


@pytest.mark.parametrize("D", [64, 128])
def test_attend_many_rows_over_few_keys_and_the_other_way_round(D):
    # one sequence: the streaming kernel whatever its rows
    rng = np.random.default_rng(D)
    check_attend(rng, 32, D, 1, 8, [700], [90], prompts=False)
    check_attend(rng, 32, D, 1, 16, [90], [90], prompts=False, window=20)
    check_attend(rng, 16, D, 2, 2, [500, 30], [300, 7], prompts=False)


def test_attend_long_contexts_and_many_sequences():
    rng = np.random.default_rng(11)
    check_attend(rng, 64, 64, 1, 8, [9000], [1])                       # one sequence over the whole GPU
    check_attend(rng, 32, 128, 2, 16, [5000, 700], [5, 1])
    check_attend(rng, 16, 128, 1, 2, [3000, 1, 2500], [1, 1, 1])
    check_attend(rng, 16, 64, 1, 1, list(rng.integers(0, 40, 700)), [1] * 700)
    check_attend(rng, 32, 64, 2, 16, [1500, 700], [300, 3], max_new=300)


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
    c, table = sequences(rng, P, [64, 64, 64], 4, 20, kv, D)
    plan = moe().Kv4(H, kv, D, P, 20, cache=dev(c))
    qd, q = bf16(rng.normal(0, 0.25, (n, H, D)))
    out = torch.full((n, H, D), 7.5, dtype=torch.bfloat16, device="cuda")
    starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    # a length below 0 is none; the sequence between keeps its own
    plan.attend(qd, dev(np.array([-2 ** 31, 64, -5], np.int32)), dev(table), out, starts=dev(starts), max_new=max(rows))
    got = out.double().cpu().numpy()
    close(got, *S4.attend(c, P, q, starts, [0, 64, 0], table))
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
        table[0, 1], table[1, 0], table[1, 1], table[2, :] = -1, c.shape[0], 2 ** 31 - 1, -2 ** 31
        return c

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


@pytest.mark.parametrize("rows", [[1, 1, 1], [3, 4, 2], [9, 40, 3]])
def test_attend_scales_far_apart(rows):
    rng = np.random.default_rng(15)

    def apart(c, table):
        codes, scales = S4.unpack(c, 16, 64)
        scales[1] = rng.integers(100, 150, scales[1].shape)     # values from 2^-27 to 2^22 times the codes
        scales[1][table[1, 0]] = 1                              # (nearly) nothing still counts in the sum
        return S4.pack(codes, scales)

    def blocks(c, table):
        codes, scales = S4.unpack(c, 16, 64)
        scales[1][..., 0], scales[1][..., 1] = rng.integers(60, 64, scales[1].shape[:-1]), rng.integers(190, 194, scales[1].shape[:-1])
        return S4.pack(codes, scales)

    check_attend(rng, 16, 64, 2, 8, [100, 70, 333], rows, change=apart)
    check_attend(rng, 16, 64, 2, 8, [100, 70, 333], rows, change=blocks)     # a head's halves
    # scores up to about 100, one key far above the rest, and a sink that takes nearly all
    check_attend(rng, 16, 64, 1, 8, [300, 64, 1000], rows, lo=124, hi=128, spread=0.02, scale=1.0)
    # the smallest scales, of which some are 0
    check_attend(rng, 16, 64, 2, 8, [100, 70, 333], rows, lo=1, hi=4, scale=1e20)


@pytest.mark.parametrize("rows", [[1, 1], [4, 33]])
def test_attend_queries_that_are_not_finite_or_far_apart(rows):
    import torch
    rng = np.random.default_rng(19)
    P, D, kv, H, lens = 32, 128, 1, 4, [70, 300]
    c, table = sequences(rng, P, lens, 10, 16, kv, D)
    starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    x = rng.normal(0, 0.25, (starts[-1], H, D))
    x[0, 1, 3], x[1, 2, 7] = np.nan, np.inf
    x[0, 0] *= 2.0 ** -30
    x[1, 0] = 0.0
    qd, q = bf16(x)
    out = torch.empty_like(qd)
    plan = moe().Kv4(H, kv, D, P, 16, cache=dev(c))
    plan.attend(qd, dev(np.array(lens, np.int32)), dev(table), out, starts=dev(starts), max_new=max(rows))
    got = out.double().cpu().numpy()
    q[0, 1], q[1, 2] = 0, 0
    ref, tol = S4.attend(c, P, q, starts, lens, table)
    assert np.isnan(got[0, 1]).all() and np.isnan(got[1, 2]).all()
    got[0, 1], got[1, 2], ref[0, 1], ref[1, 2] = 0, 0, 0, 0
    close(got, ref, tol)


def test_attend_two_streams_graph_replay_and_repeats():
    import torch
    rng = np.random.default_rng(16)
    P, D, kv, H, lens = 16, 64, 2, 16, [700, 33, 1000, 5]
    c, table = sequences(rng, P, lens, 64, 120, kv, D, poison=False)     # (longer lengths below see other places)
    d = dev(c)
    qd, q = bf16(rng.normal(0, 0.25, (4, H, D)))
    plans = [moe().Kv4(H, kv, D, P, 120, cache=d) for _ in range(2)]
    ld, td = dev(np.array(lens, np.int32)), dev(table)
    outs = [torch.zeros((4, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):     # two calls at once, a workspace each
        for p, o, s in zip(plans, outs, streams):
            p.attend(qd, ld, td, o, stream=s)
    torch.cuda.synchronize()
    ref, tol = S4.attend(c, P, q, range(5), lens, table)
    for o in outs:
        close(o.double().cpu().numpy(), ref, tol)
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
        ref, tol = S4.attend(c, P, q, range(5), lens, table)
        for o in outs:
            close(o.double().cpu().numpy(), ref, tol)


def test_attend_empty_calls_change_nothing():
    import torch
    p = moe().Kv4(4, 2, 64, 16, 3)
    z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device="cuda")   # noqa: E731
    q = z(0, 4, 64, t=torch.bfloat16)
    p.attend(q, z(0), z(0, 2), q.clone())
    p.append(z(0, 2, 64, t=torch.bfloat16), z(0, 2, 64, t=torch.bfloat16), z(0))
    p.read(z(0), z(0, 2, 64, t=torch.bfloat16), z(0, 2, 64, t=torch.bfloat16))
    q, o = z(3, 4, 64, t=torch.bfloat16), torch.full((3, 4, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    p.attend(q, z(0), z(0, 2), o, starts=z(1), max_new=3)
    p.attend(q, z(2), z(2, 0), o, starts=z(3), max_new=3)       # no rows in any sequence
    assert bool((o == 2.0).all())
    p.attend(q, z(3), z(3, 0), o)                               # a table without entries: nothing is seen
    assert bool((o == 0.0).all())


# ---------------------------------------------------------------- verification

def check_verify(rng, x, rows, drafts, qs=None, u=None, draws=None, t=None, k=None, p=None, mp=None, dtype="float32", extra=0, stride=0):
    """x [n][V]; rows: rows of each sequence; drafts [n]; qs [n][V] or None.  -> (ids, accepted)"""
    import torch
    starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    n, V, B = x.shape[0], x.shape[1], len(rows)
    wide = torch.full((n, V + stride), 9.0)
    wide[:, :V] = torch.from_numpy(np.asarray(x, np.float32))
    xd = wide.to(getattr(torch, dtype)).cuda()[:, :V]
    x = xd.double().cpu().numpy()
    u = rng.random(n).astype(np.float32) if u is None else np.asarray(u, np.float32)
    draws = rng.random(B).astype(np.float32) if draws is None else np.asarray(draws, np.float32)
    full = lambda v, dt: None if v is None else np.broadcast_to(np.asarray(v, dt), (B,)).copy()   # noqa: E731
    t, k, p, mp = full(t, np.float32), full(k, np.int32), full(p, np.float32), full(mp, np.float32)
    ids, acc = torch.full((n,), 77, dtype=torch.int32, device="cuda"), torch.full((B,), 77, dtype=torch.int32, device="cuda")
    opt = lambda v: None if v is None else dev(v)   # noqa: E731
    moe().Verify(n).run(xd, dev(np.asarray(drafts, np.int32)), dev(u), dev(draws), dev(starts), ids, acc,
                        draft_probs=None if qs is None else dev(np.asarray(qs, np.float32)), temperature=opt(t), top_k=opt(k), top_p=opt(p),
                        min_p=opt(mp))
    ids, acc = ids.cpu().numpy(), acc.cpu().numpy()
    qs = None if qs is None else np.asarray(qs, np.float32)
    for b in range(B):
        s, e = starts[b], starts[b + 1]
        if s == e:
            assert acc[b] == 0
            continue
        ps = [S4.probabilities(x[r], 1.0 if t is None else float(t[b]), 0 if k is None else int(k[b]), 1.0 if p is None else float(p[b]),
                               0.0 if mp is None else float(mp[b])) for r in range(s, e)]
        a, rest, near = S4.verify(ps, drafts[s:e], None if qs is None else qs[s:e], u[s:e], draws[b])
        if acc[b] != a:
            assert near < 2.0 ** -18, (b, acc[b], a, near)
            continue
        assert np.array_equal(ids[s:s + a], drafts[s:s + a]) and np.all(ids[s + a + 1:e] == -1)
        got = ids[s + a]
        if not rest.any():
            assert got == -1
            continue
        c = np.cumsum(rest)
        share, slack = float(draws[b]) * c[-1], 2.0 ** -18
        assert rest[got] > 0 or c[-1] < 2.0 ** -16, (b, got)
        assert c[got] - rest[got] - slack <= share <= c[got] + slack, (b, got, S.sample(rest, float(draws[b])))
    assert np.all(ids[starts[-1]:] == 77)
    return ids, acc


def drafted(rng, x, noise=1.0, t=0.8):
    near = x + rng.normal(0, noise, x.shape)
    q = np.exp((near - near.max(-1, keepdims=True)) / t)
    q /= q.sum(-1, keepdims=True)
    return q.astype(np.float32), np.array([rng.choice(x.shape[1], p=row / row.sum()) for row in q.astype(np.float64)])


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 1000, 32001, 150000])
def test_verify(V, dtype):
    rng = np.random.default_rng(V)
    rows = [5, 1, 2, 0, 8, 3]
    x = rng.normal(0, 2.5, (sum(rows) + 2, V))
    q, d = drafted(rng, x)
    check_verify(rng, x, rows, d, q, dtype=dtype)
    check_verify(rng, x, rows, d, None, dtype=dtype, stride=3)
    check_verify(rng, x, rows, d, q, t=[0.7, 0.0, 1.3, 1.0, 0.8, 0.8], k=[50, 3, 0, 1, V, 2], p=[0.9, 0.5, 1.0, 0.9, 0.95, 1.0],
                 mp=[0, 0.1, 0.02, 0, 0, 1.0], dtype=dtype)
    check_verify(rng, np.round(x), rows, d, q, k=[5, 20, 2, 1, 40, 7], p=0.8, dtype=dtype)       # equal logits, some left out


def test_verify_accepts_all_none_and_the_first_ones():
    rng = np.random.default_rng(2)
    V, rows = 400, [6, 6, 6, 6]
    x = rng.normal(0, 1, (24, V))
    q = np.exp(x) / np.exp(x).sum(-1, keepdims=True)
    _, d = drafted(rng, x)
    u = np.full(24, 0.5)
    assert np.all(check_verify(rng, x, rows, d, q, u=u)[1] == 5)              # q = p: all of them
    assert np.all(check_verify(rng, x, rows, np.argmin(x, 1), None, u=np.full(24, 0.99))[1] == 0)
    d = np.argmax(x, 1)
    d[[3, 8, 18]] = [-1, V, 2 ** 31 - 1]                                      # not in the vocabulary
    ids, acc = check_verify(rng, x, rows, d, None, t=0.0)
    assert list(acc) == [3, 2, 5, 0]
    assert ids[3] == np.argmax(x[3]) and ids[5] == -1
    check_verify(rng, x, rows, d, np.where(rng.random((24, V)) < 0.3, np.nan, 5.0), u=u)   # no probabilities at all
    check_verify(rng, x, rows, d, -q, u=u)


def test_verify_many_rows_of_one_sequence_and_many_sequences():
    rng = np.random.default_rng(3)
    x = rng.normal(0, 2, (70, 300))
    q, d = drafted(rng, x, 0.05)
    assert check_verify(rng, x, [70], d, q, u=np.full(70, 0.4))[1][0] > 33
    rows = list(rng.integers(0, 4, 700))
    x = rng.normal(0, 2, (sum(rows) + 5, 90))
    q, d = drafted(rng, x)
    check_verify(rng, x, rows, d, q, k=rng.integers(0, 20, 700), p=0.9)


def test_verify_ties_at_the_limit():
    """Drafted tokens among equal logits of which top-k keeps the first ones: those are accepted, later ones not."""
    rng = np.random.default_rng(4)
    V = 5000
    x = np.full((12, V), -3.0)
    x[:, 100::7] = 1.0                                                        # 700 equal ones
    kept_ = list(range(100, V, 7))
    d = np.array([kept_[0], kept_[39], kept_[40], 0] * 3)
    u = np.zeros(12)
    for k, want in ((40, 2), (41, 3), (39, 1), (700, 3)):
        assert np.all(check_verify(rng, x, [4, 4, 4], d, None, u=u, k=k, dtype="bfloat16")[1] == want)
    x[:, 0] = 2.0
    assert np.all(check_verify(rng, x, [4, 4, 4], d, None, u=u, k=41)[1] == 2)


def test_verify_rows_without_a_token_and_of_one_token():
    rng = np.random.default_rng(5)
    x = rng.normal(0, 1, (8, 50))
    x[1], x[4], x[6, 3] = -np.inf, np.nan, np.inf
    q, d = drafted(rng, np.nan_to_num(x, nan=0.0, posinf=9.0, neginf=-9.0))
    ids, acc = check_verify(rng, x, [3, 2, 3], d, q, u=np.zeros(8))
    assert ids[1] == -1 and acc[0] == 1 and ids[4] == -1
    assert ids[5] == d[5] or ids[6] in (-1, 3)


def test_verify_draws_have_the_target_s_distribution():
    """Over an even grid of random numbers the first token's counts are those of p, whatever q is."""
    rng = np.random.default_rng(6)
    V, n = 12, 64
    x = rng.normal(0, 1.5, V)
    near = x + rng.normal(0, 1.5, V)
    q = np.exp(near) / np.exp(near).sum()
    p = S4.probabilities(np.float32(x), 1.0, 9, 1.0, 0.0)
    # the drafted token by its share of q, then u and the draw over grids
    counts, share = np.zeros(V), (np.arange(n) + 0.5) / n
    uu, dd = np.meshgrid(share, share, indexing="ij")
    for tok in range(V):
        X, Q = np.tile(x, (2 * n * n, 1)), np.tile(q, (2 * n * n, 1))
        ids, _ = check_verify(rng, X, [2] * (n * n), np.full(2 * n * n, tok), Q, u=np.repeat(uu.ravel(), 2), draws=dd.ravel(), k=9)
        counts += q[tok] * np.bincount(ids[::2], minlength=V) / (n * n)
    assert np.abs(counts - p).max() <= 2.0 / n          # each grid is off by at most a step


def test_verify_in_a_graph_and_on_two_streams():
    import torch
    rng = np.random.default_rng(7)
    rows = [4, 1, 5]
    x = rng.normal(0, 2, (10, 3000)).astype(np.float32)
    q, d = drafted(rng, x)
    z = lambda k: torch.zeros(k, dtype=torch.int32, device="cuda")   # noqa: E731
    xd, qd, dd, sd = dev(x), dev(q), dev(d.astype(np.int32)), dev(np.array([0, 4, 5, 10], np.int32))
    u, w = torch.rand(10, device="cuda"), torch.rand(3, device="cuda")
    k = dev(np.array([20, 0, 5], np.int32))
    made = [(moe().Verify(10), z(10), z(3)) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    for _ in range(10):
        for (plan, ids, acc), s in zip(made, streams):
            plan.run(xd, dd, u, w, sd, ids, acc, draft_probs=qd, top_k=k, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(made[0][1], made[1][1]) and torch.equal(made[0][2], made[1][2])
    plan, ids, acc = made[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.run(xd, dd, u, w, sd, ids, acc, draft_probs=qd, top_k=k)
    for seed in range(4):
        u.copy_(torch.rand(10, device="cuda")), w.copy_(torch.rand(3, device="cuda"))
        sd.copy_(torch.tensor([[0, 4, 5, 10], [0, 0, 9, 10], [0, 3, 7, 9], [1, 4, 5, 6]][seed], dtype=torch.int32))
        ids.fill_(77)
        g.replay()
        one, other = ids.clone(), (z(10) + 77, z(3))
        made[1][0].run(xd, dd, u, w, sd, *other, draft_probs=qd, top_k=k)
        assert torch.equal(one, other[0]) and torch.equal(acc, other[1])


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("D,H,kv", [(64, 16, 2), (128, 6, 2)])
def test_a_run_with_drafted_tokens_and_its_graph(D, H, kv):
    """Requests decode with drafted tokens: each step assigns pages, turns queries and keys, appends, attends, verifies, and
    goes on behind the tokens that were accepted.  The whole run once call by call and once as a captured step replayed."""
    import torch
    m = moe()
    P, n, W, V, steps, most, pages = 16, 5, 12, 300, 7, 5, 80
    cap = n * most + 3
    rng = np.random.default_rng(D)
    rows_of = [rng.integers(1, most + 1, n) for _ in range(steps)]                # the drafts and one more
    xs = [bf16(rng.normal(0, 1, (cap, H + 2 * kv, D)))[0] for _ in range(steps)]
    extra = [[rng.random(cap), rng.random(n), rng.integers(0, V, cap)] for _ in range(steps)]
    head = rng.normal(0, 0.3, (H * D, V)).astype(np.float32)
    gamma, freqs = rng.normal(1, 0.1, (2, D)).astype(np.float32), 1e4 ** (-np.arange(D // 2) / (D // 2))

    def run(graph):
        z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device="cuda")   # noqa: E731
        cache = m.Kv4(H, kv, D, P, pages, sliding_window=40)
        rotary, verify = m.Rotary(D, freqs, q_gamma=dev(gamma[0]), k_gamma=dev(gamma[1])), m.Verify(cap)
        free, counts, table = dev(np.arange(pages, dtype=np.int32)), dev(np.array([pages, 0], np.int32)), z(n, W)
        have, fresh, lens, starts, slots, pos = z(n), z(n), z(n), z(n + 1), z(cap), z(cap)
        x, q, k = z(cap, H + 2 * kv, D, t=torch.bfloat16), z(cap, H, D, t=torch.bfloat16), z(cap, kv, D, t=torch.bfloat16)
        out, logits, hd = z(cap, H, D, t=torch.bfloat16), z(cap, V, t=torch.float32), dev(head)
        u, draws, drafts, ids, accepted = z(cap, t=torch.float32), z(n, t=torch.float32), z(cap), z(cap), z(n)

        def step():
            m.pages_assign(P, have, fresh, free, counts, counts, table, starts, lens, slots, pos)
            rotary.apply(x[:, :H], x[:, H:H + kv], pos, q, k)
            cache.append(k, x[:, H + kv:], slots)
            cache.attend(q, lens, table, out, starts=starts, max_new=most)
            torch.mm(out.view(cap, -1).float(), hd, out=logits)
            verify.run(logits, drafts, u, draws, starts, ids, accepted, top_k=None, temperature=None)
            have.add_(accepted + 1)

        kept_ = (have, free, counts, table, cache.cache, q, k, out, ids)
        seen, g = [], None
        for s in range(steps):
            fresh.copy_(dev(rows_of[s].astype(np.int32)))
            x.copy_(xs[s])
            u.copy_(dev(extra[s][0].astype(np.float32))), draws.copy_(dev(extra[s][1].astype(np.float32)))
            drafts.copy_(dev(extra[s][2].astype(np.int32)))
            if s % 2:      # drafted tokens that the last step's logits like best
                drafts.copy_(logits.argmax(-1))
            q.zero_(), k.zero_(), out.zero_(), ids.zero_()
            if graph and g is None:
                side = torch.cuda.Stream()
                side.wait_stream(torch.cuda.current_stream())
                old = [t.clone() for t in kept_]
                with torch.cuda.stream(side):
                    step()                                       # a first run outside the capture
                torch.cuda.current_stream().wait_stream(side)
                for t, c in zip(kept_, old):
                    t.copy_(c)
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    step()
            g.replay() if graph else step()
            seen.append([t.cpu().numpy().copy() for t in (table, starts, lens, slots, pos, counts, cache.cache, ids, accepted, drafts, logits, have)] +
                        [t.double().cpu().numpy() for t in (q, k, out)])
        return seen

    eager, replayed = run(False), run(True)
    for a, b in zip(eager, replayed):
        assert all(np.array_equal(x, y) for x, y in zip(a, b))
    free, n_free, table, have = np.arange(pages, dtype=np.int32), pages, np.zeros((n, W), np.int32), np.zeros(n, np.int64)
    cache = np.zeros((pages, kv, S4.page_bytes(P, D)), np.uint8)
    for s in range(steps):
        t, starts, lens, slots, pos, counts, c, ids, accepted, drafts, logits, after, q, k, out = eager[s]
        r = S.pages_assign(P, have, rows_of[s], free, n_free, table, cap)
        free, n_free, table = r["free"], int(r["counts"][0]), r["table"]
        for got, want in ((t, table), (starts, r["starts"]), (lens, r["lens"]), (slots, r["slots"]), (pos, r["positions"]), (counts, r["counts"])):
            assert np.array_equal(got, want), s
        e, x = int(starts[-1]), xs[s].double().cpu().numpy()
        for got, src, ga in ((q, x[:, :H], gamma[0]), (k, x[:, H:H + kv], gamma[1])):
            ref, tol = S4.rotate(src[:e], pos[None, :e], freqs, gamma=ga)
            close(got[:e], ref, tol)
            assert np.all(got[e:] == 0)                          # rows of no token
        cache = S4.append(cache, P, k, x[:, H + kv:], slots)
        assert np.array_equal(c, cache), s
        ref, tol = S4.attend(cache, P, q, starts, lens, table, 40)
        close(out[:e], ref[:e], tol[:e])
        for b in range(n):
            a, z = int(starts[b]), int(starts[b + 1])
            ps = [S4.probabilities(logits[i], 1.0, 0, 1.0, 0.0) for i in range(a, z)]
            took, rest, near = S4.verify(ps, drafts[a:z], None, extra[s][0][a:z].astype(np.float32), extra[s][1][b])
            assert accepted[b] == took or near < 2.0 ** -18
            if accepted[b] == took:
                assert np.array_equal(ids[a:a + took], drafts[a:a + took]) and np.all(ids[a + took + 1:z] == -1)
                cum, got = np.cumsum(rest), ids[a + took]
                share = float(np.float32(extra[s][1][b])) * cum[-1]
                assert cum[got] - rest[got] - 2.0 ** -18 <= share <= cum[got] + 2.0 ** -18
        have = have + accepted + 1
        assert np.array_equal(after, have)
