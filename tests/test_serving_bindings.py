"""The serving operators' bindings refuse tensors and streams that are not on the current device.  No GPU: tensors of
two devices are stand-ins, and the library's entry points count their calls."""
import types

import pytest

from mxfp4_mixture_experts_rms_gb300 import moe as M

torch = pytest.importorskip("torch")


class Tensor:
    is_cuda = True

    def __init__(self, dtype, *shape, device=0):
        self.dtype, self.shape, self.at = dtype, shape, device

    def get_device(self):
        return self.at

    def is_contiguous(self):
        return True

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def data_ptr(self):
        return 4096

    def stride(self, i=None):
        s, n = [], 1
        for k in reversed(self.shape):
            s.insert(0, n)
            n *= k
        return tuple(s) if i is None else s[i]


class Library:
    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def entry(*args):
            self.calls += 1
            return 0
        return entry


I4, F4, B2 = torch.int32, torch.float32, torch.bfloat16


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(M, "_lib", lib)
    monkeypatch.setattr(M, "_raw_stream", (lambda device: 0, lambda: 0))
    return lib


def plan(lib):
    p = object.__new__(M.Kv8)
    p.L, p.h, p.q_heads, p.kv_heads, p.head_dim, p.page_size, p.n_pages = lib, None, 4, 2, 64, 16, 3
    p.k = p.v = Tensor(torch.uint8, 3, 2, 16 * 64)
    p.k_scale = p.v_scale = Tensor(torch.uint8, 3, 2)
    p.ws, p.sinks, p.device = Tensor(torch.uint8, 512), None, 0
    return p


def calls(lib):
    """name -> (call, its tensors by name)"""
    def args(**k):
        return {n: Tensor(*v) for n, v in k.items()}
    p = plan(lib)
    return {
        "pages_assign": (lambda a, s: M.pages_assign(16, stream=s, **a), args(
            cached=(I4, 2), fresh=(I4, 2), free_pages=(I4, 4), counts=(I4, 2), counts_out=(I4, 2), table=(I4, 2, 3), starts=(I4, 3),
            lens=(I4, 2), slots=(I4, 5), positions=(I4, 5))),
        "append": (lambda a, s: p.append(stream=s, **a), args(k=(B2, 3, 2, 64), v=(B2, 3, 2, 64), slots=(I4, 3))),
        "attend": (lambda a, s: p.attend(stream=s, **a), args(
            q=(B2, 3, 4, 64), lens=(I4, 2), table=(I4, 2, 3), out=(B2, 3, 4, 64), starts=(I4, 3))),
        "sample": (lambda a, s: M.sample(stream=s, **a), args(
            logits=(F4, 2, 9), u=(F4, 2), ids=(I4, 2), temperature=(F4, 2), top_k=(I4, 2), top_p=(F4, 2), min_p=(F4, 2))),
    }


@pytest.mark.parametrize("name", ["pages_assign", "append", "attend", "sample"])
def test_every_tensor_is_on_the_current_device(lib, name):
    call, args = calls(lib)[name]
    call(args, None)
    assert lib.calls == 1
    for k, t in args.items():
        t.at = 1
        with pytest.raises(M.MoeError, match="device"):
            call(args, None)
        t.at = 0
    for t in args.values():
        t.at = 1
    with pytest.raises(M.MoeError, match="device"):
        call(args, None)
    assert lib.calls == 1


@pytest.mark.parametrize("name", ["pages_assign", "append", "attend", "sample"])
def test_the_stream_is_one_of_the_current_device(lib, name):
    call, args = calls(lib)[name]
    stream = types.SimpleNamespace(cuda_stream=7, device=torch.device("cuda", 1))
    with pytest.raises(M.MoeError, match="device"):
        call(args, stream)
    assert lib.calls == 0
    stream.device = torch.device("cuda", 0)
    call(args, stream)
    assert lib.calls == 1


def test_a_plan_is_used_on_its_cache_s_device(lib, monkeypatch):
    p = plan(lib)
    monkeypatch.setattr(M, "_raw_stream", (lambda device: 0, lambda: 1))     # the current device is the second
    b = lambda n, h: Tensor(B2, n, h, 64, device=1)   # noqa: E731
    i = lambda *s: Tensor(I4, *s, device=1)           # noqa: E731
    for call in (lambda: p.append(b(3, 2), b(3, 2), i(3)), lambda: p.attend(b(2, 4), i(2), i(2, 1), b(2, 4)), p.device_status):
        with pytest.raises(M.MoeError, match="device"):
            call()
    assert lib.calls == 0


def test_a_plan_s_arrays_are_on_one_device(lib):
    def make(sinks=0, **at):
        u = lambda n, *s: Tensor(torch.uint8, *s, device=at.get(n, 0))   # noqa: E731
        cache = (u("k", 3, 2, 1024), u("v", 3, 2, 1024), u("k_scale", 3, 2), u("v_scale", 3, 2))
        M.Kv8(4, 2, 64, 16, 3, cache=cache, sinks=Tensor(F4, 4, device=sinks), workspace=types.SimpleNamespace(ws=u("ws", 4096)))

    for bad in (dict(v=1), dict(k=1), dict(k_scale=1), dict(v_scale=1), dict(sinks=1), dict(ws=1)):
        with pytest.raises(M.MoeError, match="device"):
            lib.moe_kv8_create = lambda *a: 99
            lib.moe_kv8_workspace_bytes = lambda *a: 256
            make(**bad)


def test_rows_of_an_empty_batch_have_any_strides(lib):
    p = plan(lib)
    q, k, i = Tensor(B2, 0, 4, 64), Tensor(B2, 0, 2, 64), Tensor(I4, 0)
    for t in (q, k):
        t.stride = lambda n=None: (0, 1, 1) if n is None else (0, 1, 1)[n]
    p.attend(q, i, Tensor(I4, 0, 3), q)
    p.append(k, k, i)
    assert lib.calls == 2
