"""The serving oracle (page tables, 8-bit cache, attention over it, sampling) against other statements of
the same things, and the host-side refusals of the serving entry points.  No GPU."""
import ctypes as C

import numpy as np
import pytest

from mxfp4_mixture_experts_rms_gb300 import build, moe
from oracle import serving as S


@pytest.fixture(scope="module")
def L():
    build.build()
    return moe.load()


def test_e4m3_encoding_is_the_nearest_value_with_ties_to_even():
    torch = pytest.importorskip("torch")
    vals = S.E4M3[:127]
    assert vals[126] == 448 and vals[1] == 2.0 ** -9 and np.all(np.diff(vals) > 0)
    mid = (vals[:-1] + vals[1:]) / 2
    codes = S.e4m3(mid)
    assert np.all(codes % 2 == 0) and np.all((codes == np.arange(126)) | (codes == np.arange(1, 127)))
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(0, 1, 4000) * 2.0 ** rng.integers(-12, 9, 4000), mid, -mid, vals, -vals])
    x = x[np.abs(x) <= 448].astype(np.float32)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(S.e4m3(x), ref)
    assert list(S.e4m3([np.inf, -1e30, np.nan])) == [126, 254, 127]


def test_the_page_exponent_is_the_smallest_that_fits():
    for a in [448.0, 448.5, 447.0, 1.0, 1.75, 1.7578125, 3.5, 2.0 ** -100, 3e38]:
        k = S.exponent(a)
        assert a <= 448 * 2.0 ** k and a > 448 * 2.0 ** (k - 1)
    assert S.exponent(0.0) == -126 and S.exponent(np.inf) == S.exponent(np.finfo(np.float32).max) == 120


@pytest.mark.parametrize("P,D", [(16, 64), (32, 128), (64, 64)])
def test_the_cache_layout_is_a_permutation(P, D):
    rng = np.random.default_rng(1)
    kk, vv = rng.integers(0, 256, (2, 3, P, 2, D)).astype(np.uint8)
    k, v = S.pack(kk, vv)
    a, b = S.unpack(k, v, P, D)
    assert np.array_equal(a, kk) and np.array_equal(b, vv)
    # one byte of each by hand: token 9, dim 37, kv head 1
    assert k[2, 1].reshape(D // 16, P, 16)[37 // 16, 9, 37 % 16] == kk[2, 9, 1, 37]
    assert v[2, 1].reshape(P // 16, D, 16)[0, 37, 4 * 0 + 2 + 1] == vv[2, 9, 1, 37]


def test_appending_in_pieces_keeps_the_values_near():
    rng = np.random.default_rng(2)
    P, D, kv = 16, 64, 1
    x = rng.normal(0, 1, (40, kv, D)) * 2.0 ** rng.integers(-3, 4, (40, 1, 1))
    z = [np.zeros((4, kv, P * D), np.uint8), np.zeros((4, kv, P * D), np.uint8), np.full((4, kv), 200, np.uint8),
         np.full((4, kv), 200, np.uint8)]
    slots = np.arange(40) + P
    one = S.append(*z, P, x, -x, slots)
    c = z
    for i in range(40):
        c = S.append(*c, P, x[i:i + 1], -x[i:i + 1], slots[i:i + 1])
    assert np.array_equal(one[2], c[2]) and np.array_equal(one[3], c[3])     # the same exponents in the end
    for got in (one, c):
        kk, vv = S.unpack(got[0], got[1], P, D)
        val = S.E4M3[kk] * 2.0 ** (got[2].astype(float) - 127)[:, None, :, None]
        val = val.reshape(-1, kv, D)[slots]
        step = 2.0 ** (got[2].astype(float) - 127)[slots // P][:, :, None] * 2.0 ** -9
        assert np.all(np.abs(val - x) <= np.maximum(np.abs(x) * 2.0 ** -4, 2 * step))


def test_attention_oracle_against_matrices():
    rng = np.random.default_rng(3)
    P, D, kv, H, pages = 16, 64, 2, 6, 7
    c = S.pack(*rng.integers(0, 120, (2, pages, P, kv, D)).astype(np.uint8))
    ks, vs = rng.integers(116, 120, (2, pages, kv)).astype(np.uint8)
    table = np.array([[3, 0, 5], [6, 1, -1]], np.int32)
    lens, starts = [37, 20], [0, 3, 4]
    q = rng.normal(0, 0.1, (4, H, D))
    sinks = rng.normal(0, 1, H)
    out, _ = S.attend(*c, ks, vs, P, q, starts, lens, table, window=10, sinks=sinks)
    kk, vv = S.unpack(*c, P, D)
    for b in range(2):
        pg = table[b][table[b] >= 0]
        K = (S.E4M3[kk[pg]] * 2.0 ** (ks[pg].astype(float) - 127)[:, None, :, None]).reshape(-1, kv, D)
        V = (S.E4M3[vv[pg]] * 2.0 ** (vs[pg].astype(float) - 127)[:, None, :, None]).reshape(-1, kv, D)
        for r in range(starts[b], starts[b + 1]):
            p = lens[b] - (starts[b + 1] - r)
            x = np.einsum("hd,thd->ht", q[r], np.repeat(K, 3, 1)) / 8
            t = np.arange(K.shape[0])
            x[:, (t > p) | (t <= p - 10)] = -np.inf
            x = np.concatenate([x, sinks[:, None]], 1)
            w = np.exp(x - x.max(1, keepdims=True))
            w = w[:, :-1] / w.sum(1, keepdims=True)
            assert np.allclose(np.einsum("ht,thd->hd", w, np.repeat(V, 3, 1)), out[r], rtol=1e-12, atol=1e-12)


def test_pages_oracle_keeps_every_page_once():
    rng = np.random.default_rng(4)
    P, W, pool = 16, 8, 60
    free, n_free = rng.permutation(pool).astype(np.int32), pool
    table, lens = np.full((12, W), -1, np.int32), np.zeros(12, np.int64)
    for step in range(60):
        fresh = rng.integers(0, 30, 12)
        fresh[rng.random(12) < 0.25] = -1
        r = S.pages_assign(P, lens, fresh, free, n_free, table, 400)
        free, n_free, table, lens = r["free"], r["counts"][0], r["table"], r["lens"].astype(np.int64)
        lens = np.minimum(lens, W * P)
        held = [table[b, : -(-lens[b] // P)] for b in range(12)]
        used = np.concatenate(held)
        used = used[used >= 0]
        assert len(np.unique(used)) == len(used) and len(used) + n_free == pool
        assert not set(used) & set(free[:n_free])
        s = r["slots"][r["slots"] >= 0]
        assert len(np.unique(s)) == len(s)
        if r["counts"][1]:      # a shortage: those tokens are lost, the request starts again
            lens[:] = 0
            free, n_free, table = rng.permutation(pool).astype(np.int32), pool, np.full((12, W), -1, np.int32)


def test_sampling_oracle_cases():
    x = np.array([1.0, 3.0, 3.0, np.nan, -np.inf, 2.0])
    assert list(np.flatnonzero(S.kept(x, 0.0, 0, 1.0, 0.0))) == [1]            # greedy: the lower index
    assert list(np.flatnonzero(S.kept(x, 1.0, 2, 1.0, 0.0))) == [1, 2]
    assert list(np.flatnonzero(S.kept(x, 1.0, 1, 1.0, 0.0))) == [1]            # ties: the lower index first
    assert list(np.flatnonzero(S.kept(x, 1.0, 0, 0.39, 0.0))) == [1]           # 1 / (2 + e^-1 + e^-2) = 0.3995
    assert list(np.flatnonzero(S.kept(x, 1.0, 0, 0.5, 0.0))) == [1, 2]
    assert list(np.flatnonzero(S.kept(x, 1.0, 0, 0.0, 0.0))) == [1]
    assert list(np.flatnonzero(S.kept(x, 1.0, 0, 1.0, 0.3))) == [1, 2, 5]      # e^-1 = 0.37 and e^-2 = 0.14
    w = S.kept(x, 1.0, 0, 1.0, 0.0)
    assert S.sample(w, 0.0) == 0 and S.sample(w, 0.9999999) == 5
    assert S.sample(S.kept(np.array([np.nan, -np.inf]), 1.0, 0, 1.0, 0.0), 0.5) == -1
    rng = np.random.default_rng(5)
    x = rng.normal(0, 2, 50)
    w = S.kept(x, 0.7, 0, 1.0, 0.0)
    assert np.allclose(w / w.sum(), np.exp(x / 0.7) / np.exp(x / 0.7).sum())


def test_pages_assign_refusals(L):
    P = C.c_void_p
    a = [P(0x1000 * (i + 1)) for i in range(12)]

    def call(page=16, n=2, cached=a[0], fresh=a[1], free=a[2], cap=8, counts=a[3], co=a[4], table=a[5], w=4, starts=a[6],
             lens=a[7], slots=a[8], pos=a[9], mt=5):
        return L.moe_pages_assign(page, n, cached, fresh, free, cap, counts, co, table, w, starts, lens, slots, pos, mt, None)

    for bad in (dict(page=0), dict(page=65537), dict(n=-1), dict(n=4097), dict(cap=-1), dict(w=-1), dict(mt=-1),
                dict(n=4096, w=2 ** 20), dict(cached=None), dict(fresh=None), dict(free=None), dict(counts=None), dict(co=None),
                dict(table=None), dict(starts=None), dict(lens=None), dict(slots=None), dict(cached=P(0x1002)),
                dict(pos=P(0x2001)), dict(lens=a[0]), dict(lens=a[1]), dict(starts=a[0]), dict(starts=P(0x1ffc)), dict(starts=P(0x1ff8))):
        assert call(**bad) == moe.MOE_EINVAL, bad
        assert L.moe_last_error()


def test_kv8_refusals(L):
    P = C.c_void_p
    for bad in ((0, 1, 64, 16, 4), (8, 0, 64, 16, 4), (9, 2, 64, 16, 4), (34, 2, 64, 16, 4), (8, 2, 96, 16, 4),
                (8, 2, 64, 24, 4), (8, 2, 64, 128, 4), (8, 2, 64, 16, 0), (8, 2, 64, 64, 2 ** 26), (512, 257, 64, 16, 4)):
        assert not L.moe_kv8_create(*bad), bad
        assert b"moe_kv8_create" in L.moe_last_error()
    h = P(L.moe_kv8_create(8, 2, 64, 16, 4))
    x, y, s, o = P(0x10000), P(0x20000), P(0x30000), P(0x40000)
    app = lambda k=x, v=y, ks=128, vs=128, sl=s, n=3: L.moe_kv8_append(h, k, v, ks, vs, sl, n, None)   # noqa: E731
    att = lambda q=x, qs=512, st=None, le=s, t=y, w=4, n=2, mn=1, r=2, out=o, os_=512: L.moe_kv8_attend(   # noqa: E731
        h, q, qs, st, le, t, w, n, mn, r, out, os_, None)
    assert app() == moe.MOE_ENOTREADY and att() == moe.MOE_ENOTREADY
    word = C.c_int(7)
    assert L.moe_kv8_get_device_status(h, C.byref(word), None) == moe.MOE_ENOTREADY and word.value == 7
    assert L.moe_kv8_get_device_status(None, C.byref(word), None) == moe.MOE_EINVAL
    assert L.moe_kv8_get_device_status(h, None, None) == moe.MOE_EINVAL
    assert L.moe_kv8_set_cache(h, x, None, s, s) == moe.MOE_EINVAL
    assert L.moe_kv8_set_cache(h, P(0x10008), y, s, s) == moe.MOE_EINVAL
    assert L.moe_kv8_set_cache(h, x, y, s, P(0x30001)) == moe.MOE_OK          # scales: any byte
    assert att() == moe.MOE_ENOTREADY                                         # no workspace
    assert L.moe_kv8_workspace_bytes(h) > 0 and L.moe_kv8_workspace_bytes(None) == 0
    assert L.moe_kv8_set_workspace(h, P(0x10080), 1 << 30) == moe.MOE_EINVAL
    assert L.moe_kv8_set_workspace(h, P(0x10000), 100) == moe.MOE_ENOMEM
    assert L.moe_kv8_set_i(h, b"sliding_window", -1) == moe.MOE_EINVAL
    assert L.moe_kv8_set_i(h, b"window", 1) == moe.MOE_EINVAL
    assert L.moe_kv8_set_i(h, b"sliding_window", 128) == moe.MOE_OK
    for v in (0.0, -1.0, float("inf"), float("nan"), 1e31):
        assert L.moe_kv8_set_f(h, b"softmax_scale", v) == moe.MOE_EINVAL
    assert L.moe_kv8_set_f(h, b"softmax_scale", 0.2) == moe.MOE_OK
    assert L.moe_kv8_set_sinks(h, P(0x1002)) == moe.MOE_EINVAL and L.moe_kv8_set_sinks(h, None) == moe.MOE_OK
    assert app(n=0) == moe.MOE_OK
    for bad in (dict(n=-1), dict(k=None), dict(v=None), dict(sl=None), dict(k=P(0x10008)), dict(sl=P(0x30002)),
                dict(ks=120), dict(vs=132), dict(ks=127)):
        assert app(**bad) == moe.MOE_EINVAL, bad
    L.moe_kv8_destroy(h)
    L.moe_kv8_destroy(None)
    assert L.moe_kv8_append(None, x, y, 128, 128, s, 1, None) == moe.MOE_EINVAL
    assert L.moe_kv8_attend(None, x, 512, None, s, y, 4, 2, 1, 2, o, 512, None) == moe.MOE_EINVAL


def test_sample_refusals(L):
    P = C.c_void_p
    x, u, ids = P(0x10000), P(0x20000), P(0x30000)
    call = lambda x=x, bf=0, n=2, V=10, st=10, t=None, k=None, p=None, m=None, u=u, ids=ids: L.moe_sample(   # noqa: E731
        x, bf, n, V, st, t, k, p, m, u, ids, None)
    assert call(n=0) == moe.MOE_OK
    for bad in (dict(n=-1), dict(V=0), dict(V=2 ** 24 + 1, st=2 ** 25), dict(st=9), dict(bf=2), dict(x=None), dict(u=None),
                dict(ids=None), dict(x=P(0x10002)), dict(bf=1, x=P(0x10001)), dict(t=P(2)), dict(k=P(1)), dict(p=P(3)),
                dict(m=P(2)), dict(u=P(2)), dict(ids=P(2))):
        assert call(**bad) == moe.MOE_EINVAL, bad


def test_bindings_refuse_what_the_library_cannot_see():
    torch = pytest.importorskip("torch")
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(moe.MoeError):       # host tensors
        moe.sample(torch.zeros((4, 8)), torch.zeros(4), i)
    with pytest.raises(moe.MoeError):
        moe.pages_assign(16, i, i, i, i, i[:2], torch.zeros((4, 2), dtype=torch.int32), torch.zeros(5, dtype=torch.int32), i, i)
