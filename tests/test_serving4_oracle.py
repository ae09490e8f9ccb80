"""Oracle pins and host-side refusals of the serving step's other operators (no GPU)."""
import ctypes as C
import types

import numpy as np
import pytest

from mxfp4_mixture_experts_rms_gb300 import build, moe
from oracle import serving as S
from oracle import serving4 as S4


@pytest.fixture(scope="module")
def L():
    build.build()
    return moe.load()


def test_e2m1_encoding_is_the_nearest_value_with_ties_to_even():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.normal(0, 3, 4000), [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 1e9, np.inf]])
    for y in (x, -x):
        code = S4.e2m1(y)
        best = np.abs(np.clip(y, -6, 6)[:, None] - S4.E2M1[None]).min(1)
        assert np.array_equal(np.abs(S4.E2M1[code] - np.clip(y, -6, 6)), best)
        two = (np.abs(np.clip(y, -6, 6)[:, None] - S4.E2M1[None, :8] * np.where(y < 0, -1, 1)[:, None]) == best[:, None]).sum(1) == 2
        assert two[-11:-4].all() and np.all(code[two] % 2 == 0)
    assert S4.e2m1([np.nan, -0.0]).tolist() == [7, 0]


def test_the_block_exponent_is_the_smallest_that_fits():
    for a in list(np.random.default_rng(2).random(200) * 100) + [6.0, 3.0, 6 * 2.0 ** 40, 5.9999]:
        k = S4.exponent(a)
        assert 6 * 2.0 ** (k - 1) < a <= 6 * 2.0 ** k
    assert S4.exponent(0) == -126 and S4.exponent(np.inf) == 125 and S4.exponent(3.3e38) == 125


@pytest.mark.parametrize("P,D", [(16, 64), (32, 128), (64, 64)])
def test_the_cache_layout_is_a_permutation(P, D):
    rng = np.random.default_rng(3)
    cache = rng.integers(0, 256, (3, 2, S4.page_bytes(P, D))).astype(np.uint8)
    codes, scales = S4.unpack(cache, P, D)
    assert np.array_equal(S4.pack(codes, scales), cache)
    # the places that the header names: token 21 (of P > 16) or 5, kv head 1, value dims 32 .. 34
    t = 21 if P > 16 else 5
    at = P * D // 2 + P * 16 + t * 16
    assert cache[2, 1, at] == codes[1, 2, t, 1, 32] | codes[1, 2, t, 1, 33] << 4
    assert cache[2, 1, P * D + P * D // 32 + P + (t & ~15) + 4 * 2 + 1] == scales[1, 2, t, 1, 1]


def test_append_and_read_oracle():
    rng = np.random.default_rng(4)
    x = rng.normal(0, 1, (6, 2, 64))
    cache = S4.append(np.zeros((2, 2, S4.page_bytes(16, 64)), np.uint8), 16, x, -2 * x, [3, -1, 31, 0, 16, 40])
    k, v = S4.read(cache, 16, 64, [3, 31, 0, 16])
    assert np.array_equal(v, -2 * k)
    amax = np.abs(x[[0, 2, 3, 4]].reshape(4, 2, 2, 32)).max(-1)
    assert np.all(np.abs(k - x[[0, 2, 3, 4]]).reshape(4, 2, 2, 32).max(-1) <= amax / 4)


def test_rotation_oracle():
    """Against complex numbers; scores depend on the distance alone."""
    rng = np.random.default_rng(5)
    x, freqs = rng.normal(0, 1, (4, 2, 64)), rng.random(32)
    pos = np.array([[0, 3, 10, 17]])
    y, _ = S4.rotate(x, pos, freqs, interleaved=True)
    z = (x[..., 0::2] + 1j * x[..., 1::2]) * np.exp(1j * pos[0][:, None, None] * freqs)
    assert np.allclose(y[..., 0::2], z.real) and np.allclose(y[..., 1::2], z.imag)
    assert np.allclose(y[0], x[0])
    a, b = (S4.rotate(x, pos + s, freqs)[0] for s in (0, 1000))
    assert np.allclose((a[1] * a[3]).sum(-1), (b[1] * b[3]).sum(-1))
    n, _ = S4.rotate(x, pos, freqs[:0], gamma=np.ones(64), eps=0.0)
    assert np.allclose((n * n).mean(-1), 1)
    # several axes: each pair by its own
    of = np.arange(32) % 3
    y, _ = S4.rotate(x, np.stack([pos[0], 2 * pos[0], 0 * pos[0]]), freqs, of)
    w, _ = S4.rotate(x, pos, np.where(of == 0, freqs, np.where(of == 1, 2 * freqs, 0)))
    assert np.allclose(y, w)


def test_attention_oracle_against_the_8_bit_one():
    """The same values in either cache give the same attention."""
    rng = np.random.default_rng(6)
    P, D, kv, H = 16, 64, 2, 6
    codes, scales = rng.integers(0, 16, (2, 5, P, kv, D)).astype(np.uint8), np.full((2, 5, P, kv, D // 32), 127, np.uint8)
    cache = S4.pack(codes, scales)
    e4 = S.e4m3(S4.E2M1[codes])
    k8, v8 = S.pack(e4[0], e4[1])
    q = rng.normal(0, 0.3, (7, H, D))
    table, one = np.array([[3, 1, -1], [4, 0, 2]], np.int32), np.full((5, kv), 127, np.uint8)
    sinks = rng.normal(0, 1, H)
    for window in (0, 5):
        a = S4.attend(cache, P, q, [0, 3, 7], [20, 41], table, window, sinks)[0]
        b = S.attend(k8, v8, one, one, P, q, [0, 3, 7], [20, 41], table, window, sinks)[0]
        assert np.allclose(a, b, atol=1e-12)


def test_verification_keeps_the_target_s_distribution():
    """The exact probability of each first token over u and the draw is p's."""
    rng = np.random.default_rng(7)
    p, q = rng.random(6), rng.random(6)
    p, q = p / p.sum(), q / q.sum()
    p[2] = 0.0
    p /= p.sum()
    got = np.zeros(6)
    for x in range(6):
        take = min(1.0, p[x] / q[x])
        got[x] += q[x] * take
        if take < 1:
            a, rest, _ = S4.verify([p, p], [x, 0], [q, q], [(take + 1) / 2, 0], 0.5)
            assert a == 0
            got += q[x] * (1 - take) * rest / rest.sum()
        if take > 0:
            assert S4.verify([p, p], [x, 0], [q, q], [take * 0.999, 0], 0.5)[0] == 1
    assert np.allclose(got, p)
    assert S4.verify([p, p], [2, 0], None, [0.0, 0], 0.5)[0] == 0          # a token of no weight
    a, rest, _ = S4.verify([p, p], [0, 0], None, [0.9999, 0], 0.5)
    assert a == 0 and rest[0] == 0 and np.allclose(rest[1:], p[1:])


def test_rotary_refusals(L):
    P = C.c_void_p
    for bad in ((32, 16, 1, 0), (96, 32, 1, 0), (64, 33, 1, 0), (64, 4, 1, 0), (64, 40, 1, 0), (64, -8, 1, 0), (64, 32, 0, 0),
                (64, 32, 5, 0), (64, 32, 1, 2)):
        assert not L.moe_rotary_create(*bad), bad
        assert b"moe_rotary_create" in L.moe_last_error()
    h = P(L.moe_rotary_create(64, 32, 2, 0))
    x, y, p = 0x100000, 0x200000, P(0x300000)

    def call(q=x, qs=640, qh=8, k=x + 1024, ks=640, kh=2, pos=p, ps=5, n=5, qo=y, qos=640, ko=y + 1024, kos=640):
        return L.moe_rotary_apply(h, q, qs, qh, k, ks, kh, pos, ps, n, qo, qos, ko, kos, None)

    assert call() == moe.MOE_ENOTREADY
    assert L.moe_rotary_set_freqs(h, None, None) == moe.MOE_EINVAL
    assert L.moe_rotary_set_freqs(h, P(0x1004), None) == moe.MOE_EINVAL
    assert L.moe_rotary_set_freqs(h, P(0x1008), P(0x1001)) == moe.MOE_OK
    assert L.moe_rotary_set_norm(h, P(0x1008), None) == moe.MOE_EINVAL and L.moe_rotary_set_norm(None, None, None) == moe.MOE_EINVAL
    for key, v in ((b"eps", -1.0), (b"eps", float("nan")), (b"factor", 0.0), (b"factor", float("inf")), (b"base", 1.0)):
        assert L.moe_rotary_set_f(h, key, v) == moe.MOE_EINVAL
    assert call(n=0) == moe.MOE_OK and call(qh=0, kh=0) == moe.MOE_OK
    for bad in (dict(n=-1), dict(qh=-1), dict(kh=65537), dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(pos=None),
                dict(pos=P(0x300002)), dict(ps=4), dict(q=x + 4), dict(ko=y + 1026), dict(qs=508), dict(kos=642), dict(kos=124),
                dict(qo=x + 8), dict(qo=x, qos=1280), dict(ko=x), dict(qo=x + 1024), dict(ko=y + 8), dict(ko=y + 1016),
                dict(ko=y + 1024 + 128)):
        assert call(**bad) == moe.MOE_EINVAL, bad
        assert L.moe_last_error()
    assert L.moe_rotary_apply(None, x, 512, 8, None, 0, 0, p, 5, 5, y, 512, None, 0, None) == moe.MOE_EINVAL
    L.moe_rotary_destroy(h)
    L.moe_rotary_destroy(None)


def test_kv4_refusals(L):
    P = C.c_void_p
    for bad in ((0, 1, 64, 16, 4), (8, 0, 64, 16, 4), (9, 2, 64, 16, 4), (34, 2, 64, 16, 4), (8, 2, 96, 16, 4),
                (8, 2, 64, 24, 4), (8, 2, 64, 128, 4), (8, 2, 64, 16, 0), (8, 2, 64, 64, 2 ** 26), (512, 257, 64, 16, 4)):
        assert not L.moe_kv4_create(*bad), bad
        assert b"moe_kv4_create" in L.moe_last_error()
    h = P(L.moe_kv4_create(8, 2, 64, 16, 4))
    assert L.moe_kv4_page_bytes(h) == 2 * S4.page_bytes(16, 64) and L.moe_kv4_page_bytes(None) == 0
    x, y, s, o = 0x10000, 0x20000, P(0x30000), 0x40000
    app = lambda k=x, v=y, ks=128, vs=128, sl=s, n=3: L.moe_kv4_append(h, k, v, ks, vs, sl, n, None)   # noqa: E731
    rd = lambda k=x, v=y, ks=128, vs=128, sl=s, n=3: L.moe_kv4_read(h, sl, n, k, v, ks, vs, None)      # noqa: E731
    att = lambda q=x, qs=512, st=None, le=s, t=P(y), w=4, n=2, mn=1, r=2, out=o, os_=512: L.moe_kv4_attend(   # noqa: E731
        h, q, qs, st, le, t, w, n, mn, r, out, os_, None)
    assert app() == rd() == att() == moe.MOE_ENOTREADY
    word = C.c_int(7)
    assert L.moe_kv4_get_device_status(h, C.byref(word), None) == moe.MOE_ENOTREADY and word.value == 7
    assert L.moe_kv4_get_device_status(None, C.byref(word), None) == moe.MOE_EINVAL
    assert L.moe_kv4_get_device_status(h, None, None) == moe.MOE_EINVAL
    assert L.moe_kv4_set_cache(h, None) == moe.MOE_EINVAL and L.moe_kv4_set_cache(h, P(0x10008)) == moe.MOE_EINVAL
    assert L.moe_kv4_set_cache(h, P(x)) == moe.MOE_OK
    assert att() == moe.MOE_ENOTREADY                                         # no workspace
    assert L.moe_kv4_workspace_bytes(h) > 0 and L.moe_kv4_workspace_bytes(None) == 0
    assert L.moe_kv4_set_workspace(h, P(0x10080), 1 << 30) == moe.MOE_EINVAL
    assert L.moe_kv4_set_workspace(h, P(0x10000), 100) == moe.MOE_ENOMEM
    assert L.moe_kv4_set_i(h, b"sliding_window", -1) == moe.MOE_EINVAL
    assert L.moe_kv4_set_i(h, b"window", 1) == moe.MOE_EINVAL
    assert L.moe_kv4_set_i(h, b"sliding_window", 128) == moe.MOE_OK
    for v in (0.0, -1.0, float("inf"), float("nan"), 1e31):
        assert L.moe_kv4_set_f(h, b"softmax_scale", v) == moe.MOE_EINVAL
    assert L.moe_kv4_set_sinks(h, P(0x1002)) == moe.MOE_EINVAL and L.moe_kv4_set_sinks(h, None) == moe.MOE_OK
    assert app(n=0) == moe.MOE_OK and rd(n=0) == moe.MOE_OK
    for bad in (dict(n=-1), dict(n=2 ** 30 + 1), dict(k=None), dict(v=None), dict(sl=None), dict(k=0x10008), dict(sl=P(0x30002)),
                dict(ks=120), dict(vs=132), dict(ks=127)):
        assert app(**bad) == moe.MOE_EINVAL and rd(**bad) == moe.MOE_EINVAL, bad
    assert rd(v=x) == moe.MOE_EINVAL and rd(v=x + 128) == moe.MOE_EINVAL and rd(v=x + 128, ks=256, vs=256) == moe.MOE_EINVAL
    L.moe_kv4_destroy(h)
    L.moe_kv4_destroy(None)
    assert L.moe_kv4_append(None, x, y, 128, 128, s, 1, None) == moe.MOE_EINVAL
    assert L.moe_kv4_attend(None, x, 512, None, s, P(y), 4, 2, 1, 2, o, 512, None) == moe.MOE_EINVAL


def test_verify_refusals(L):
    P = C.c_void_p
    a = [P(0x10000 * (i + 1)) for i in range(13)]

    def call(x=a[0], bf=0, n=6, V=10, st=10, d=a[1], q=a[2], qs=10, starts=a[3], B=2, t=a[4], k=a[5], p=a[6], mp=a[7], u=a[8], w=a[9],
             ids=a[10], acc=a[11], ws=a[12], size=6 * 24):
        return L.moe_verify(x, bf, n, V, st, d, q, qs, starts, B, t, k, p, mp, u, w, ids, acc, ws, size, None)

    assert L.moe_verify_workspace_bytes(6) == 6 * 24 and L.moe_verify_workspace_bytes(0) == 0 and L.moe_verify_workspace_bytes(-3) == 0
    assert call(B=0) == moe.MOE_OK
    for bad in (dict(n=-1), dict(n=2 ** 24 + 1), dict(V=0), dict(V=2 ** 24 + 1, st=2 ** 25), dict(st=9), dict(qs=9), dict(bf=2), dict(B=-1),
                dict(B=65537), dict(x=None), dict(d=None), dict(starts=None), dict(u=None), dict(w=None), dict(ids=None), dict(acc=None),
                dict(ws=None), dict(x=P(0x10002)), dict(bf=1, x=P(0x10001)), dict(d=P(2)), dict(q=P(2)), dict(starts=P(1)), dict(t=P(2)),
                dict(k=P(1)), dict(p=P(3)), dict(mp=P(2)), dict(u=P(2)), dict(w=P(2)), dict(ids=P(2)), dict(acc=P(2)), dict(ws=P(0x10008)),
                dict(ids=a[1]), dict(ids=P(0x20000 + 20)), dict(d=P(a[10].value - 20)), dict(ids=a[8]), dict(ids=a[3]), dict(acc=P(a[3].value + 8)),
                dict(acc=a[9]), dict(acc=a[4]), dict(acc=P(a[10].value + 20)), dict(acc=P(a[10].value - 4)), dict(ids=a[7])):
        assert call(**bad) == moe.MOE_EINVAL, bad
        assert L.moe_last_error()
    assert call(size=6 * 24 - 1) == moe.MOE_ENOMEM


# ---------------------------------------------------------------- bindings (tensors of two devices are stand-ins)

torch = pytest.importorskip("torch")
from tests.test_serving_bindings import B2, F4, I4, Library, Tensor  # noqa: E402


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(moe, "_lib", lib)
    monkeypatch.setattr(moe, "_raw_stream", (lambda device: 0, lambda: 0))
    return lib


def calls(lib):
    def args(**k):
        return {n: Tensor(*v) for n, v in k.items()}
    c = object.__new__(moe.Kv4)
    c.L, c.h, c.q_heads, c.kv_heads, c.head_dim, c.page_size, c.n_pages, c.device = lib, None, 4, 2, 64, 16, 3, 0
    c.cache, c.ws, c.sinks = Tensor(torch.uint8, 3, 2, 1088), Tensor(torch.uint8, 512), None
    r = object.__new__(moe.Rotary)
    r.L, r.h, r.head_dim, r.n_axes, r.device = lib, None, 64, 1, 0
    v = object.__new__(moe.Verify)
    v.L, v.max_rows, v.bytes, v.device, v.ws = lib, 4, 96, 0, Tensor(torch.uint8, 96)
    return {
        "rotary": (lambda a, s: r.apply(stream=s, **a), args(q=(B2, 3, 4, 64), k=(B2, 3, 2, 64), positions=(I4, 3), q_out=(B2, 3, 4, 64),
                                                           k_out=(B2, 3, 2, 64))),
        "append": (lambda a, s: c.append(stream=s, **a), args(k=(B2, 3, 2, 64), v=(B2, 3, 2, 64), slots=(I4, 3))),
        "read": (lambda a, s: c.read(stream=s, **a), args(k=(B2, 3, 2, 64), v=(B2, 3, 2, 64), slots=(I4, 3))),
        "attend": (lambda a, s: c.attend(stream=s, **a), args(
            q=(B2, 3, 4, 64), lens=(I4, 2), table=(I4, 2, 3), out=(B2, 3, 4, 64), starts=(I4, 3))),
        "verify": (lambda a, s: v.run(stream=s, **a), args(
            logits=(F4, 4, 9), drafts=(I4, 4), u=(F4, 4), draws=(F4, 2), starts=(I4, 3), ids=(I4, 4), accepted=(I4, 2), draft_probs=(F4, 4, 9),
            temperature=(F4, 2), top_k=(I4, 2), top_p=(F4, 2), min_p=(F4, 2))),
    }


@pytest.mark.parametrize("name", ["rotary", "append", "read", "attend", "verify"])
def test_every_tensor_and_the_stream_are_on_the_current_device(lib, name):
    call, args = calls(lib)[name]
    call(args, None)
    assert lib.calls == 1
    for t in args.values():
        t.at = 1
        with pytest.raises(moe.MoeError, match="device"):
            call(args, None)
        t.at = 0
    for t in args.values():
        t.at = 1
    with pytest.raises(moe.MoeError, match="device"):
        call(args, None)
    for t in args.values():
        t.at = 0
    stream = types.SimpleNamespace(cuda_stream=7, device=torch.device("cuda", 1))
    with pytest.raises(moe.MoeError, match="device"):
        call(args, stream)
    assert lib.calls == 1
    stream.device = torch.device("cuda", 0)
    call(args, stream)
    assert lib.calls == 2


@pytest.mark.parametrize("name", ["rotary", "append", "read", "attend", "verify"])
def test_bindings_refuse_other_types_and_shapes(lib, name):
    call, args = calls(lib)[name]
    for key, t in args.items():
        kept = t.dtype
        t.dtype = torch.float16
        with pytest.raises(moe.MoeError):
            call(args, None)
        t.dtype = kept
    for key, t in args.items():
        if key in ("table", "q", "logits", "lens"):    # (other arguments follow these)
            continue
        kept = t.shape
        t.shape = (kept[0] + 1, *kept[1:])
        with pytest.raises(moe.MoeError):
            call(args, None)
        t.shape = kept
    assert lib.calls == 0


def test_rotary_plans_refuse_axes_that_are_not_there(monkeypatch):
    with pytest.raises(moe.MoeError, match="axes"):
        moe.Rotary(64, [1.0] * 8, axes=[0] * 7)
    with pytest.raises(moe.MoeError, match="axes"):
        moe.Rotary(64, [1.0] * 8, axes=[0, 1, 2, 0, 0, 0, 0, 0], n_axes=2)
    with pytest.raises(moe.MoeError, match="axes"):
        moe.Rotary(64, [1.0] * 8, axes=[-1] * 8)
