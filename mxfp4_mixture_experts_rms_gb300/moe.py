"""Thin ctypes binding of ``include/moe.h`` (argument marshalling only).

Every step of the block runs in the CUDA kernels of ``lib/libmoe.so``; this
module only passes device pointers and sizes.  PyTorch provides device memory
and streams.  There is no fallback: if the library is missing or fails to
load, every call raises.
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np

from . import build as _build

MOE_OK, MOE_EINVAL, MOE_ESHAPE, MOE_ENOTREADY, MOE_ECUDA, MOE_ENOMEM, MOE_EDEVICE = 0, -1, -2, -3, -4, -5, -6
_STATUS_NAMES = {0: "MOE_OK", -1: "MOE_EINVAL", -2: "MOE_ESHAPE", -3: "MOE_ENOTREADY", -4: "MOE_ECUDA",
                 -5: "MOE_ENOMEM", -6: "MOE_EDEVICE"}

_lib = None

EXPORTS = ["moe_plan_create", "moe_plan_destroy", "moe_plan_set_i", "moe_plan_set_f", "moe_plan_path_for",
           "moe_workspace_bytes",
           "moe_set_workspace", "moe_load_weights", "moe_forward", "moe_forward_ex", "moe_get_expert_counts",
           "moe_get_permutation", "moe_debug_dequant", "moe_profile_read", "moe_get_device_status",
           "moe_get_cache_state",
           "moe_forward_noalloc", "moe_cast_f32_to_bf16", "moe_mx_quantize_fp4", "moe_locality_create",
           "moe_locality_record", "moe_locality_attach", "moe_locality_read", "moe_locality_reset",
           "moe_locality_destroy", "moe_attn_create", "moe_attn_set_i", "moe_attn_set_f", "moe_attn_workspace_bytes",
           "moe_attn_set_workspace", "moe_attn_set_cache", "moe_attn_load_weights", "moe_attn_decode", "moe_attn_prefill",
           "moe_attn_destroy", "moe_attn_get_device_status", "moe_pages_assign", "moe_kv8_create", "moe_kv8_set_i",
           "moe_kv8_set_f", "moe_kv8_set_cache", "moe_kv8_set_sinks", "moe_kv8_workspace_bytes",
           "moe_kv8_set_workspace", "moe_kv8_append", "moe_kv8_attend", "moe_kv8_destroy", "moe_kv8_get_device_status",
           "moe_sample", "moe_rotary_create", "moe_rotary_set_f", "moe_rotary_set_freqs", "moe_rotary_set_norm",
           "moe_rotary_apply", "moe_rotary_destroy", "moe_kv4_create", "moe_kv4_set_i", "moe_kv4_set_f", "moe_kv4_page_bytes",
           "moe_kv4_set_cache", "moe_kv4_set_sinks", "moe_kv4_workspace_bytes", "moe_kv4_set_workspace", "moe_kv4_append",
           "moe_kv4_read", "moe_kv4_attend", "moe_kv4_get_device_status", "moe_kv4_destroy", "moe_verify_workspace_bytes",
           "moe_verify",
           "moe_last_error"]


class LocalityStats(C.Structure):
    _fields_ = [("hist", C.c_void_p), ("weight_hist", C.c_void_p), ("layer_records", C.c_void_p),
                ("adjacent_pairs", C.c_void_p), ("overlap_sum", C.c_void_p), ("jaccard_sum", C.c_void_p),
                ("cache_hits", C.c_void_p), ("cache_weight_hits", C.c_void_p), ("caps", C.c_void_p),
                ("n_caps", C.c_int)]


class AttnWeights(C.Structure):
    _fields_ = [("gamma", C.c_void_p), ("wq", C.c_void_p), ("wk", C.c_void_p), ("wv", C.c_void_p),
                ("wo", C.c_void_p), ("bq", C.c_void_p), ("bk", C.c_void_p), ("bv", C.c_void_p),
                ("bo", C.c_void_p), ("sinks", C.c_void_p)]


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class Mat(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("bias", C.c_void_p)]


class Weights(C.Structure):
    _fields_ = [("gamma", C.c_void_p), ("router_w", C.c_void_p), ("router_b", C.c_void_p),
                ("gate", Mat), ("up", Mat), ("down", Mat),
                ("sh_gate", Mat), ("sh_up", Mat), ("sh_down", Mat)]


def lib_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True):
    """Load ``libmoe.so`` (building it first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    if build_if_missing and not _build.up_to_date():
        _build.build()
    if not os.path.exists(_build.LIB):
        raise MoeError(MOE_ENOTREADY, f"CUDA library not built: {_build.LIB}")
    L = C.CDLL(_build.LIB)
    P, I, LL, D, SZ = C.c_void_p, C.c_int, C.c_longlong, C.c_double, C.c_size_t
    L.moe_plan_create.restype = P
    L.moe_plan_create.argtypes = [I, I, I, I, C.c_float, C.c_float, C.c_float]
    L.moe_plan_destroy.restype = None
    L.moe_plan_destroy.argtypes = [P]
    L.moe_plan_set_i.argtypes = [P, C.c_char_p, LL]
    L.moe_plan_set_f.argtypes = [P, C.c_char_p, D]
    L.moe_plan_path_for.argtypes = [P, I]
    L.moe_workspace_bytes.restype = SZ
    L.moe_workspace_bytes.argtypes = [P, I]
    L.moe_set_workspace.argtypes = [P, P, SZ]
    L.moe_load_weights.argtypes = [P, C.POINTER(Weights)]
    L.moe_forward.argtypes = [P, P, I, P, P, P]
    L.moe_forward_ex.argtypes = [P, P, I, P, P, P, P, P]
    L.moe_get_expert_counts.argtypes = [P, P, P]
    L.moe_get_permutation.argtypes = [P, P, P, P, P]
    L.moe_debug_dequant.argtypes = [P, I, I, P, P]
    L.moe_get_device_status.argtypes = [P, C.POINTER(I), P]
    L.moe_get_cache_state.argtypes = [P, P, P, P]
    L.moe_profile_read.argtypes = [P, C.POINTER(C.c_double), C.POINTER(I), I]
    L.moe_forward_noalloc.argtypes = [P, P, I, P, P, P]
    L.moe_cast_f32_to_bf16.argtypes = [P, P, SZ, P]
    L.moe_mx_quantize_fp4.argtypes = [P, SZ, SZ, P, P, P]
    L.moe_locality_create.restype = P
    L.moe_locality_create.argtypes = [I, I, I, P, I]
    L.moe_locality_record.argtypes = [P, I, P, P, I, LL, P]
    L.moe_locality_attach.argtypes = [P, P, I]
    L.moe_locality_read.argtypes = [P, C.POINTER(LocalityStats)]
    L.moe_locality_reset.argtypes = [P, P]
    L.moe_locality_destroy.restype = None
    L.moe_locality_destroy.argtypes = [P]
    L.moe_attn_create.restype = P
    L.moe_attn_create.argtypes = [I, I, I, I, I, I]
    L.moe_attn_set_i.argtypes = [P, C.c_char_p, LL]
    L.moe_attn_set_f.argtypes = [P, C.c_char_p, D]
    L.moe_attn_workspace_bytes.restype = SZ
    L.moe_attn_workspace_bytes.argtypes = [P]
    L.moe_attn_set_workspace.argtypes = [P, P, SZ]
    L.moe_attn_set_cache.argtypes = [P, P, P]
    L.moe_attn_load_weights.argtypes = [P, C.POINTER(AttnWeights)]
    L.moe_attn_decode.argtypes = [P, P, I, P, P, P]
    L.moe_attn_prefill.argtypes = [P, P, I, I, I, P, P]
    L.moe_attn_get_device_status.argtypes = [P, C.POINTER(I), P]
    L.moe_attn_destroy.restype = None
    L.moe_attn_destroy.argtypes = [P]
    L.moe_pages_assign.argtypes = [I, I, P, P, P, I, P, P, P, I, P, P, P, P, I, P]
    L.moe_kv8_create.restype = P
    L.moe_kv8_create.argtypes = [I, I, I, I, I]
    L.moe_kv8_set_i.argtypes = [P, C.c_char_p, LL]
    L.moe_kv8_set_f.argtypes = [P, C.c_char_p, D]
    L.moe_kv8_set_cache.argtypes = [P, P, P, P, P]
    L.moe_kv8_set_sinks.argtypes = [P, P]
    L.moe_kv8_workspace_bytes.restype = SZ
    L.moe_kv8_workspace_bytes.argtypes = [P]
    L.moe_kv8_set_workspace.argtypes = [P, P, SZ]
    L.moe_kv8_append.argtypes = [P, P, P, LL, LL, P, I, P]
    L.moe_kv8_attend.argtypes = [P, P, LL, P, P, P, I, I, I, I, P, LL, P]
    L.moe_kv8_get_device_status.argtypes = [P, C.POINTER(I), P]
    L.moe_kv8_destroy.restype = None
    L.moe_kv8_destroy.argtypes = [P]
    L.moe_sample.argtypes = [P, I, I, I, LL, P, P, P, P, P, P, P]
    L.moe_rotary_create.restype = P
    L.moe_rotary_create.argtypes = [I, I, I, I]
    L.moe_rotary_set_f.argtypes = [P, C.c_char_p, D]
    L.moe_rotary_set_freqs.argtypes = [P, P, P]
    L.moe_rotary_set_norm.argtypes = [P, P, P]
    L.moe_rotary_apply.argtypes = [P, P, LL, I, P, LL, I, P, LL, I, P, LL, P, LL, P]
    L.moe_rotary_destroy.restype = None
    L.moe_rotary_destroy.argtypes = [P]
    L.moe_kv4_create.restype = P
    L.moe_kv4_create.argtypes = [I, I, I, I, I]
    L.moe_kv4_set_i.argtypes = [P, C.c_char_p, LL]
    L.moe_kv4_set_f.argtypes = [P, C.c_char_p, D]
    L.moe_kv4_page_bytes.restype = SZ
    L.moe_kv4_page_bytes.argtypes = [P]
    L.moe_kv4_set_cache.argtypes = [P, P]
    L.moe_kv4_set_sinks.argtypes = [P, P]
    L.moe_kv4_workspace_bytes.restype = SZ
    L.moe_kv4_workspace_bytes.argtypes = [P]
    L.moe_kv4_set_workspace.argtypes = [P, P, SZ]
    L.moe_kv4_append.argtypes = [P, P, P, LL, LL, P, I, P]
    L.moe_kv4_read.argtypes = [P, P, I, P, P, LL, LL, P]
    L.moe_kv4_attend.argtypes = [P, P, LL, P, P, P, I, I, I, I, P, LL, P]
    L.moe_kv4_get_device_status.argtypes = [P, C.POINTER(I), P]
    L.moe_kv4_destroy.restype = None
    L.moe_kv4_destroy.argtypes = [P]
    L.moe_verify_workspace_bytes.restype = SZ
    L.moe_verify_workspace_bytes.argtypes = [I]
    L.moe_verify.argtypes = [P, I, I, I, LL, P, P, LL, P, I, P, P, P, P, P, P, P, P, P, SZ, P]
    L.moe_last_error.restype = C.c_char_p
    L.moe_last_error.argtypes = []
    for name in EXPORTS:
        if name not in ("moe_plan_create", "moe_plan_destroy", "moe_workspace_bytes", "moe_last_error",
                        "moe_locality_create", "moe_locality_destroy", "moe_attn_create", "moe_attn_destroy",
                        "moe_attn_workspace_bytes", "moe_kv8_create", "moe_kv8_destroy", "moe_kv8_workspace_bytes"):
            getattr(L, name).restype = C.c_int
    _lib = L
    return L


def _check(rc: int):
    if rc != MOE_OK:
        raise MoeError(rc, load().moe_last_error().decode())


def _ptr(t):
    """Device address of a tensor the library reads or writes as one dense
    row-major array; a strided view would be misread, so it is refused."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise MoeError(MOE_EINVAL, "tensors passed to the library must be contiguous")
    return t.data_ptr()


def _stream_ptr(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


def cast_f32_to_bf16(src, dst, stream=None):
    """dst (int16/uint16 bits, device) = bf16_rne(src (float32, device)); enqueued on `stream`."""
    assert src.numel() == dst.numel()
    _check(load().moe_cast_f32_to_bf16(C.c_void_p(_ptr(src)), C.c_void_p(_ptr(dst)), int(src.numel()),
                                       _stream_ptr(stream)))


def mx_quantize_fp4(x, codes, scales, stream=None):
    """FP4 activation encoding of x (bf16 bits as int16/uint16, device, [rows][cols])
    into codes (uint8 [rows][cols/2]) and E8M0 scales (uint8 [rows][cols/32]),
    both device tensors; enqueued on `stream`."""
    rows, cols = x.shape
    assert codes.numel() == rows * cols // 2 and scales.numel() == rows * cols // 32
    _check(load().moe_mx_quantize_fp4(C.c_void_p(_ptr(x)), rows, cols, C.c_void_p(_ptr(codes)),
                                      C.c_void_p(_ptr(scales)), _stream_ptr(stream)))


class DeviceBlock:
    """Device copies (torch tensors) of one block's weights, in the canonical layout."""

    def __init__(self, blk: dict, device="cuda"):
        import torch
        shape = blk["shape"]
        self.shape = shape

        def up(a, dt=None):
            if isinstance(a, torch.Tensor):   # already a tensor (e.g. drawn on the device)
                return a.to(device).contiguous()
            a = np.ascontiguousarray(a)
            t = torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a)
            return t.to(device)

        self.gamma = up(blk["gamma"])
        self.router_w = up(blk["router_w"])
        self.router_b = up(blk["router_b"])
        self.mats = {m: (up(blk["codes"][m]), up(blk["scales"][m]), up(blk["bias"][m])) for m in ("gate", "up", "down")}
        self.shared = None
        if shape.n_shared:
            sh = blk["shared"]
            self.shared = {m: (up(sh["codes"][m]), up(sh["scales"][m]), up(sh["bias"][m])) for m in ("gate", "up", "down")}

    def cstruct(self) -> Weights:
        w = Weights()
        w.gamma, w.router_w, w.router_b = _ptr(self.gamma), _ptr(self.router_w), _ptr(self.router_b)
        for m in ("gate", "up", "down"):
            c, s, b = self.mats[m]
            setattr(w, m, Mat(_ptr(c), _ptr(s), _ptr(b)))
            if self.shared is not None:
                c, s, b = self.shared[m]
                setattr(w, "sh_" + m, Mat(_ptr(c), _ptr(s), _ptr(b)))
        return w


class HostStoreBlock(DeviceBlock):
    """A block's weights for a plan with an expert cache: the routed experts'
    matrices in pinned host memory (the store the cache copies from), the
    router, the norm weight and the shared expert on the device."""

    def __init__(self, blk: dict, device="cuda"):
        super().__init__(blk, device)
        self.mats = {m: tuple(t.cpu().pin_memory() for t in v) for m, v in self.mats.items()}


class Plan:
    """One block shape: owns the plan handle and a torch-allocated workspace."""

    def __init__(self, shape, max_tokens: int = 4096, device="cuda", **opts):
        self.L = load()
        self.shape = shape
        h = self.L.moe_plan_create(shape.hidden, shape.expert_hidden, shape.n_experts, shape.top_k,
                                   shape.swiglu_alpha, shape.swiglu_limit, shape.weight_scale)
        if not h:
            raise MoeError(MOE_ESHAPE, self.L.moe_last_error().decode())
        self.h = C.c_void_p(h)
        self.set_i("n_shared_experts", shape.n_shared)
        self.set_f("rms_eps", shape.rms_eps)
        self.set_i("max_tokens", max_tokens)
        for k, v in opts.items():
            self.set_i(k, int(v))
        self.max_tokens = max_tokens
        self.device = device
        self.ws = None
        self.weights = None

    def set_i(self, key: str, v: int):
        _check(self.L.moe_plan_set_i(self.h, key.encode(), int(v)))

    def set_f(self, key: str, v: float):
        _check(self.L.moe_plan_set_f(self.h, key.encode(), float(v)))

    def path_for(self, tokens: int) -> int:
        """1 if a forward of `tokens` tokens runs the GEMV decode path, 2 the
        grouped GEMM, 3 the block-scaled FP4 grouped GEMM (act_fp4 plans)."""
        rc = int(self.L.moe_plan_path_for(self.h, int(tokens)))
        _check(min(rc, 0))
        return rc

    def workspace_bytes(self, max_tokens: int = 0) -> int:
        return int(self.L.moe_workspace_bytes(self.h, max_tokens))

    def alloc_workspace(self):
        import torch
        n = self.workspace_bytes()
        self.ws = torch.empty(n + 256, dtype=torch.uint8, device=self.device)
        p = self.ws.data_ptr()
        off = (-p) % 256
        _check(self.L.moe_set_workspace(self.h, C.c_void_p(p + off), n))
        return self

    def load_weights(self, dev: DeviceBlock):
        self.weights = dev  # keep alive
        self._wstruct = dev.cstruct()
        _check(self.L.moe_load_weights(self.h, C.byref(self._wstruct)))
        return self

    def forward(self, x, out, ids=None, stream=None):
        _check(self.L.moe_forward(self.h, C.c_void_p(_ptr(x)), int(x.shape[0]), C.c_void_p(_ptr(out)),
                                  C.c_void_p(_ptr(ids)), _stream_ptr(stream)))

    def forward_ex(self, x, out, ids=None, route_w=None, xhat=None, stream=None):
        _check(self.L.moe_forward_ex(self.h, C.c_void_p(_ptr(x)), int(x.shape[0]), C.c_void_p(_ptr(out)),
                                     C.c_void_p(_ptr(ids)), C.c_void_p(_ptr(route_w)), C.c_void_p(_ptr(xhat)),
                                     _stream_ptr(stream)))

    def expert_counts(self, out, stream=None):
        _check(self.L.moe_get_expert_counts(self.h, C.c_void_p(_ptr(out)), _stream_ptr(stream)))

    def permutation(self, offsets, perm_token, perm_slot, stream=None):
        """offsets [E + n_shared + 1]; perm_token / perm_slot of at least
        max_tokens * (top_k + n_shared) entries (the extent the library copies)."""
        R = self.max_tokens * (self.shape.top_k + self.shape.n_shared)
        if perm_token.numel() < R or perm_slot.numel() < R:
            raise MoeError(MOE_EINVAL, f"perm_token / perm_slot need {R} entries")
        if offsets.numel() < self.shape.n_experts + self.shape.n_shared + 1:
            raise MoeError(MOE_EINVAL, "offsets needs n_experts + n_shared + 1 entries")
        _check(self.L.moe_get_permutation(self.h, C.c_void_p(_ptr(offsets)), C.c_void_p(_ptr(perm_token)),
                                          C.c_void_p(_ptr(perm_slot)), _stream_ptr(stream)))

    def debug_dequant(self, expert: int, which: int, out, stream=None):
        _check(self.L.moe_debug_dequant(self.h, int(expert), int(which), C.c_void_p(_ptr(out)), _stream_ptr(stream)))

    def profile_read(self, n_slots: int = 4):
        """(total ms, launches) per kernel slot since the last read (profile option)."""
        ms = (C.c_double * n_slots)()
        cnt = (C.c_int * n_slots)()
        _check(self.L.moe_profile_read(self.h, ms, cnt, n_slots))
        return list(ms), list(cnt)

    def device_status(self, stream=None) -> int:
        s = C.c_int(0)
        rc = self.L.moe_get_device_status(self.h, C.byref(s), _stream_ptr(stream))
        if rc not in (MOE_OK, MOE_EDEVICE):
            _check(rc)
        return s.value

    def cache_state(self, stream=None):
        """Expert cache of a plan made with expert_cache_slots: (slot of each
        expert, -1 when not resident; cumulative hits; misses; forwards)."""
        slots = np.empty(self.shape.n_experts, np.int32)
        stats = np.zeros(3, np.int64)
        _check(self.L.moe_get_cache_state(self.h, slots.ctypes.data_as(C.c_void_p),
                                          stats.ctypes.data_as(C.c_void_p), _stream_ptr(stream)))
        return slots, int(stats[0]), int(stats[1]), int(stats[2])

    def close(self):
        if getattr(self, "h", None):
            self.L.moe_plan_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Locality:
    """Expert-locality statistics of the routing (ds4.c expert locality
    profiler; goosedump gpt_oss.rs ExpertRouteProfile), kept on the device."""

    def __init__(self, n_layers: int, n_experts: int, top_k: int, caps=()):
        import numpy as np
        self.L = load()
        self.n_layers, self.n_experts, self.top_k = n_layers, n_experts, top_k
        arr = (C.c_int * max(len(caps), 1))(*[int(c) for c in caps])
        h = self.L.moe_locality_create(n_layers, n_experts, top_k, arr, len(caps))
        if not h:
            raise MoeError(MOE_EINVAL, self.L.moe_last_error().decode())
        self.h = C.c_void_p(h)
        self._np = np

    def record(self, layer: int, ids, route_w, first_pos: int, stream=None):
        _check(self.L.moe_locality_record(self.h, int(layer), C.c_void_p(_ptr(ids)), C.c_void_p(_ptr(route_w)),
                                          int(ids.shape[0]), int(first_pos), _stream_ptr(stream)))

    def attach(self, plan, layer: int):
        _check(self.L.moe_locality_attach(plan.h, self.h, int(layer)))

    def reset(self, stream=None):
        _check(self.L.moe_locality_reset(self.h, _stream_ptr(stream)))

    def read(self) -> dict:
        np = self._np
        L, E = self.n_layers, self.n_experts
        out = dict(hist=np.zeros((L, E), np.uint64), weight_hist=np.zeros((L, E), np.float64),
                   layer_records=np.zeros(L, np.uint64), adjacent_pairs=np.zeros(L, np.uint64),
                   overlap_sum=np.zeros(L, np.float64), jaccard_sum=np.zeros(L, np.float64),
                   cache_hits=np.zeros((16, L), np.uint64), cache_weight_hits=np.zeros((16, L), np.float64),
                   caps=np.zeros(16, np.int32))
        st = LocalityStats(*[out[k].ctypes.data for k in ("hist", "weight_hist", "layer_records", "adjacent_pairs",
                                                          "overlap_sum", "jaccard_sum", "cache_hits",
                                                          "cache_weight_hits", "caps")], 0)
        _check(self.L.moe_locality_read(self.h, C.byref(st)))
        n = st.n_caps
        out["caps"] = out["caps"][:n].copy()
        out["cache_hits"] = out["cache_hits"][:n].copy()
        out["cache_weight_hits"] = out["cache_weight_hits"][:n].copy()
        return out

    def close(self):
        if getattr(self, "h", None):
            self.L.moe_locality_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class AttnPlan:
    """One layer's attention decode step (moe_attn_*): the plan, a torch-allocated
    workspace and fp16 key/value caches [max_seqs][max_ctx][kv_heads][64]."""

    def __init__(self, hidden: int, q_heads: int, kv_heads: int, max_seqs: int, max_ctx: int, head_dim: int = 64,
                 sliding_window: int = 0, out_bf16: bool = False, prefill_rows: int = 0, device="cuda"):
        import torch
        self.L = load()
        h = self.L.moe_attn_create(hidden, q_heads, kv_heads, head_dim, max_seqs, max_ctx)
        if not h:
            raise MoeError(MOE_EINVAL, self.L.moe_last_error().decode())
        self.h = C.c_void_p(h)
        self.hidden, self.q_heads, self.kv_heads, self.max_seqs, self.max_ctx = hidden, q_heads, kv_heads, max_seqs, max_ctx
        _check(self.L.moe_attn_set_i(self.h, b"sliding_window", int(sliding_window)))
        _check(self.L.moe_attn_set_i(self.h, b"out_bf16", int(out_bf16)))
        if prefill_rows:
            _check(self.L.moe_attn_set_i(self.h, b"prefill_rows", int(prefill_rows)))
        n = int(self.L.moe_attn_workspace_bytes(self.h))
        self.ws = torch.empty(n + 256, dtype=torch.uint8, device=device)
        off = (-self.ws.data_ptr()) % 256
        _check(self.L.moe_attn_set_workspace(self.h, C.c_void_p(self.ws.data_ptr() + off), n))
        self.k_cache = torch.zeros((max_seqs, max_ctx, kv_heads, head_dim), dtype=torch.float16, device=device)
        self.v_cache = torch.zeros_like(self.k_cache)
        _check(self.L.moe_attn_set_cache(self.h, C.c_void_p(self.k_cache.data_ptr()),
                                         C.c_void_p(self.v_cache.data_ptr())))
        self.weights = None

    def load_weights(self, wts: dict):
        """wts: device tensors gamma, wq, wk, wv, wo (bf16 bits as int16), bq, bk, bv, bo, sinks (float32)."""
        self.weights = wts
        self._w = AttnWeights(*[_ptr(wts[k]) for k in ("gamma", "wq", "wk", "wv", "wo", "bq", "bk", "bv", "bo",
                                                        "sinks")])
        _check(self.L.moe_attn_load_weights(self.h, C.byref(self._w)))
        return self

    def decode(self, x, positions, out, stream=None):
        _check(self.L.moe_attn_decode(self.h, C.c_void_p(_ptr(x)), int(x.shape[0]), C.c_void_p(_ptr(positions)),
                                      C.c_void_p(_ptr(out)), _stream_ptr(stream)))

    def prefill(self, x, seq: int, pos0: int, out, stream=None):
        """x: bf16 bits [n][hidden] (n new tokens of cache sequence seq at positions pos0 ..)."""
        _check(self.L.moe_attn_prefill(self.h, C.c_void_p(_ptr(x)), int(x.shape[0]), int(seq), int(pos0),
                                       C.c_void_p(_ptr(out)), _stream_ptr(stream)))

    def set_i(self, key: str, value: int):
        _check(self.L.moe_attn_set_i(self.h, key.encode(), int(value)))

    def device_status(self, stream=None) -> int:
        s = C.c_int(0)
        rc = self.L.moe_attn_get_device_status(self.h, C.byref(s), _stream_ptr(stream))
        if rc not in (MOE_OK, MOE_EDEVICE):
            _check(rc)
        return s.value

    def close(self):
        if getattr(self, "h", None):
            self.L.moe_attn_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_DTYPES = {}    # "i4", "f4", "f8", "u1", "b2": int32, float32, float64, uint8, bfloat16


def _dtypes():
    import torch
    _DTYPES.update(i4=torch.int32, f4=torch.float32, f8=torch.float64, u1=torch.uint8, b2=torch.bfloat16)
    return _DTYPES


_raw_stream = None


def _device(t, what: str) -> int:
    """The current device; `t`, a tensor of the call, must be on it."""
    global _raw_stream
    if t is None or not t.is_cuda:
        raise MoeError(MOE_EINVAL, f"{what}: a CUDA tensor is needed")
    if _raw_stream is None:
        import torch
        _raw_stream = (torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice)
    device = _raw_stream[1]()
    if t.get_device() != device:
        raise MoeError(MOE_EINVAL, f"{what} is on device {t.get_device()}, the current device is {device}")
    return device


def _arg(t, kind: str, device: int, count=None, what="tensor", none=False):
    """Address of a dense tensor on `device` of type `kind` and (where given)
    `count` elements; None passes where `none` allows it."""
    if t is None and none:
        return None
    if t is None or t.dtype is not (_DTYPES or _dtypes())[kind] or t.get_device() != device or not t.is_contiguous() or \
            (count is not None and t.numel() != count):
        raise MoeError(MOE_EINVAL, f"{what}: a contiguous CUDA tensor of {_dtypes()[kind]} on device {device}"
                                   + (f" ({count} elements)" if count is not None else "") + " is needed")
    return t.data_ptr()


def _stream(stream, device: int):
    """cudaStream_t of `stream`, one of `device`, or of the current one."""
    if stream is None:
        return _raw_stream[0](device)
    if stream.device.index != device:
        raise MoeError(MOE_EINVAL, f"the stream is of device {stream.device.index}, the current device is {device}")
    return stream.cuda_stream


def _head_rows(t, heads: int, dim: int, device: int, what: str):
    """(address, row stride) of bf16 rows [n][heads][dim], dense but for the stride from row to row."""
    shape = t.shape
    if t.get_device() != device or t.dtype is not (_DTYPES or _dtypes())["b2"] or len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise MoeError(MOE_EINVAL, f"{what}: a CUDA tensor of bf16 rows [n][{heads}][{dim}] on device {device} is needed")
    s0, s1, s2 = t.stride()
    if shape[0] and (s2 != 1 or (s1 != dim and heads > 1)):     # (an empty tensor's strides say nothing)
        raise MoeError(MOE_EINVAL, f"{what}: the heads of a row must lie side by side")
    return t.data_ptr(), s0 if shape[0] > 1 else heads * dim


def pages_assign(page_size: int, cached, fresh, free_pages, counts, counts_out, table, starts, lens, slots, positions=None,
                 stream=None):
    """Block tables and slot maps from request lengths (moe_pages_assign): int32 device tensors cached [n],
    fresh [n] (below 0: finished), free_pages [capacity], counts [>= 1], counts_out [2], table [n][width],
    starts [n + 1], lens [n], slots [max_tokens], positions [max_tokens] or None."""
    n, width = table.shape
    tokens, d = slots.numel(), _device(table, "table")
    rc = (_lib or load()).moe_pages_assign(
        int(page_size), n, _arg(cached, "i4", d, n, "cached"), _arg(fresh, "i4", d, n, "fresh"),
        _arg(free_pages, "i4", d, None, "free_pages"), free_pages.numel(), _arg(counts, "i4", d, None, "counts"),
        _arg(counts_out, "i4", d, 2, "counts_out"), _arg(table, "i4", d, None, "table"), width, _arg(starts, "i4", d, n + 1, "starts"),
        _arg(lens, "i4", d, n, "lens"), _arg(slots, "i4", d, None, "slots"), _arg(positions, "i4", d, tokens, "positions", none=True),
        tokens, _stream(stream, d))
    if rc:
        _check(rc)


class Kv8:
    """One layer's paged key/value cache in 8 bits (moe_kv8_*): the plan, its workspace, and the arrays of
    codes and scales k, v [n_pages][kv_heads][page_size * head_dim], k_scale, v_scale [n_pages][kv_heads]
    (uint8; `cache` = (k, v, k_scale, v_scale) to use given ones).  `workspace`: another plan, used on the
    same stream, whose workspace this one shares.  All of a plan's arrays are on one device, which is the
    current one where its methods are called."""

    def __init__(self, q_heads: int, kv_heads: int, head_dim: int, page_size: int, n_pages: int, sliding_window: int = 0,
                 softmax_scale: float | None = None, sinks=None, cache=None, workspace: "Kv8 | None" = None, device="cuda"):
        import torch
        self.L = load()
        h = self.L.moe_kv8_create(q_heads, kv_heads, head_dim, page_size, n_pages)
        if not h:
            raise MoeError(MOE_EINVAL, self.L.moe_last_error().decode())
        self.h = C.c_void_p(h)
        self.q_heads, self.kv_heads, self.head_dim, self.page_size, self.n_pages = q_heads, kv_heads, head_dim, page_size, n_pages
        _check(self.L.moe_kv8_set_i(self.h, b"sliding_window", int(sliding_window)))
        if softmax_scale is not None:
            _check(self.L.moe_kv8_set_f(self.h, b"softmax_scale", float(softmax_scale)))
        codes, scales = (n_pages, kv_heads, page_size * head_dim), (n_pages, kv_heads)
        n_scales, n_codes = n_pages * kv_heads, n_pages * kv_heads * page_size * head_dim
        if cache is None:
            cache = [torch.zeros(s, dtype=torch.uint8, device=device) for s in (codes, codes, scales, scales)]
        self.k, self.v, self.k_scale, self.v_scale = cache
        d = self.device = self.k.get_device()   # whose tensors and streams the calls take
        if d < 0:
            raise MoeError(MOE_EINVAL, "k: a CUDA tensor is needed")
        _check(self.L.moe_kv8_set_cache(self.h, _arg(self.k, "u1", d, n_codes, "k"), _arg(self.v, "u1", d, n_codes, "v"),
                                        _arg(self.k_scale, "u1", d, n_scales, "k_scale"), _arg(self.v_scale, "u1", d, n_scales, "v_scale")))
        self.sinks = sinks
        _check(self.L.moe_kv8_set_sinks(self.h, _arg(sinks, "f4", d, q_heads, "sinks", none=True)))
        n = int(self.L.moe_kv8_workspace_bytes(self.h))
        self.ws = torch.empty(n + 256, dtype=torch.uint8, device=self.k.device) if workspace is None else workspace.ws
        if self.ws.numel() < n + 256:
            raise MoeError(MOE_ENOMEM, "the shared workspace is too small for this plan")
        at = _arg(self.ws, "u1", d, None, "workspace")
        with torch.cuda.device(d):
            _check(self.L.moe_kv8_set_workspace(self.h, at + (-at) % 256, n))

    def _on(self, t, what: str) -> int:
        """The current device; `t` must be on it, and the plan too."""
        d = _device(t, what)
        if d != self.device:
            raise MoeError(MOE_EINVAL, f"the cache is on device {self.device}, the current device is {d}")
        return d

    def append(self, k, v, slots, stream=None):
        """k, v: bf16 [n][kv_heads][head_dim] (rows may be strided); slots: int32 [n]."""
        d = self._on(k, "k")
        kp, ks = _head_rows(k, self.kv_heads, self.head_dim, d, "k")
        vp, vs = _head_rows(v, self.kv_heads, self.head_dim, d, "v")
        n = k.shape[0]
        if v.shape[0] != n:
            raise MoeError(MOE_EINVAL, "k and v must have the same number of rows")
        rc = self.L.moe_kv8_append(self.h, kp, vp, ks, vs, _arg(slots, "i4", d, n, "slots"), n, _stream(stream, d))
        if rc:
            _check(rc)

    def attend(self, q, lens, table, out, starts=None, max_new: int = 1, stream=None):
        """q, out: bf16 [n_rows][q_heads][head_dim] (rows may be strided); lens int32 [n_seqs]; table int32
        [n_seqs][width]; starts int32 [n_seqs + 1] (None: one row a sequence); max_new: most rows of a sequence."""
        d = self._on(q, "q")
        qp, qs = _head_rows(q, self.q_heads, self.head_dim, d, "q")
        op, os_ = _head_rows(out, self.q_heads, self.head_dim, d, "out")
        n, width = table.shape
        if out.shape[0] != q.shape[0]:
            raise MoeError(MOE_EINVAL, "q and out must have the same number of rows")
        rc = self.L.moe_kv8_attend(self.h, qp, qs, _arg(starts, "i4", d, n + 1, "starts", none=True), _arg(lens, "i4", d, n, "lens"),
                                   _arg(table, "i4", d, None, "table"), width, n, max_new, q.shape[0], op, os_, _stream(stream, d))
        if rc:
            _check(rc)

    def device_status(self, stream=None) -> int:
        s = C.c_int(0)
        rc = self.L.moe_kv8_get_device_status(self.h, C.byref(s), _stream(stream, self._on(self.ws, "the plan")))
        if rc not in (MOE_OK, MOE_EDEVICE):
            _check(rc)
        return s.value

    def close(self):
        if getattr(self, "h", None):
            self.L.moe_kv8_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def sample(logits, u, ids, temperature=None, top_k=None, top_p=None, min_p=None, stream=None):
    """Next tokens (moe_sample): logits [n][vocab] fp32 or bf16 (rows may be strided), u float32 [n] in [0, 1), ids
    int32 [n]; temperature, top_p, min_p float32 [n] and top_k int32 [n], each may be None."""
    shape, kinds = logits.shape, _DTYPES or _dtypes()
    bf16 = logits.dtype is kinds["b2"]
    d = _device(logits, "logits")
    if len(shape) != 2 or not (bf16 or logits.dtype is kinds["f4"]) or (logits.stride(1) != 1 and shape[1] > 1):
        raise MoeError(MOE_EINVAL, "logits: a CUDA tensor of fp32 or bf16 rows is needed")
    n, vocab = shape
    rc = (_lib or load()).moe_sample(
        logits.data_ptr(), bf16, n, vocab, logits.stride(0) if n > 1 else vocab,
        _arg(temperature, "f4", d, n, "temperature", none=True), _arg(top_k, "i4", d, n, "top_k", none=True),
        _arg(top_p, "f4", d, n, "top_p", none=True), _arg(min_p, "f4", d, n, "min_p", none=True), _arg(u, "f4", d, n, "u"),
        _arg(ids, "i4", d, n, "ids"), _stream(stream, d))
    if rc:
        _check(rc)


class Rotary:
    """Norms and rotary positions of queries and keys (moe_rotary_*): the plan and its table.  freqs: radians a
    position of each pair of dims (host, float64; a multiple of 8 of them, at most head_dim / 2); axes: the axis
    of positions that turns each pair (host; None: one axis); pairs are dims i and i + len(freqs), or with
    `interleaved` 2 i and 2 i + 1.  q_gamma, k_gamma: float32 [head_dim] device tensors, None: that side is not
    normed.  factor: of the sines and cosines.  All arrays are on one device, which is the current one where
    apply is called."""

    def __init__(self, head_dim: int, freqs, axes=None, n_axes: int | None = None, interleaved: bool = False, q_gamma=None,
                 k_gamma=None, eps: float = 1e-5, factor: float = 1.0, device="cuda"):
        import torch
        self.L = load()
        freqs = np.ascontiguousarray(freqs, np.float64).reshape(-1)
        if axes is not None:
            axes = np.asarray(axes).reshape(-1)
            if len(axes) != len(freqs) or (len(axes) and (axes.min() < 0 or axes.max() > 255)):
                raise MoeError(MOE_EINVAL, "axes: one of 0 .. 255 for each of freqs is needed")
        most = 0 if axes is None or not len(axes) else int(axes.max())
        self.head_dim, self.n_axes = int(head_dim), most + 1 if n_axes is None else int(n_axes)
        if self.n_axes <= most:
            raise MoeError(MOE_EINVAL, f"axes: one is {most}, there are {self.n_axes}")
        h = self.L.moe_rotary_create(self.head_dim, len(freqs), self.n_axes, int(bool(interleaved)))
        if not h:
            raise MoeError(MOE_EINVAL, self.L.moe_last_error().decode())
        self.h = C.c_void_p(h)
        _check(self.L.moe_rotary_set_f(self.h, b"eps", float(eps)))
        _check(self.L.moe_rotary_set_f(self.h, b"factor", float(factor)))
        self.freqs = torch.from_numpy(freqs if len(freqs) else np.zeros(1)).to(device)
        self.axes = None if axes is None else torch.from_numpy(np.ascontiguousarray(axes, np.uint8)).to(device)
        self.q_gamma, self.k_gamma = q_gamma, k_gamma
        d = self.device = self.freqs.get_device()
        if d < 0:
            raise MoeError(MOE_EINVAL, "the table: a CUDA device is needed")
        _check(self.L.moe_rotary_set_freqs(self.h, _arg(self.freqs, "f8", d, None, "freqs"), _arg(self.axes, "u1", d, None, "axes", none=True)))
        _check(self.L.moe_rotary_set_norm(self.h, _arg(q_gamma, "f4", d, self.head_dim, "q_gamma", none=True),
                                          _arg(k_gamma, "f4", d, self.head_dim, "k_gamma", none=True)))

    def apply(self, q, k, positions, q_out=None, k_out=None, stream=None):
        """q, k: bf16 [n][heads][head_dim] (rows may be strided; k may be None); positions: int32 [n], or
        [n_axes][n]; q_out, k_out: likewise, None: in place."""
        d = _device(q, "q")
        if d != self.device:
            raise MoeError(MOE_EINVAL, f"the table is on device {self.device}, the current device is {d}")
        n = q.shape[0]
        if positions.shape != ((n,) if self.n_axes == 1 and len(positions.shape) == 1 else (self.n_axes, n)):
            raise MoeError(MOE_EINVAL, f"positions: shape ({self.n_axes}, {n})" + (f" or ({n},)" if self.n_axes == 1 else "") + " is needed")
        sides = []
        for x, out, what in ((q, q_out, "q"), (k, k_out, "k")):
            if x is None and out is None and what == "k":
                sides.append((None, 0, 0, None, 0))
                continue
            if x is None or len(x.shape) != 3:
                raise MoeError(MOE_EINVAL, f"{what}: a CUDA tensor of bf16 rows [n][heads][{self.head_dim}] is needed")
            heads, out = x.shape[1], x if out is None else out
            xp, xs = _head_rows(x, heads, self.head_dim, d, what)
            op, os_ = _head_rows(out, heads, self.head_dim, d, what + "_out")
            if x.shape[0] != n or out.shape[0] != n:
                raise MoeError(MOE_EINVAL, "q, k and the outputs must have the same number of rows")
            sides.append((xp, xs, heads, op, os_))
        (qp, qs, qh, qop, qos), (kp, ks, kh, kop, kos) = sides
        rc = self.L.moe_rotary_apply(self.h, qp, qs, qh, kp, ks, kh, _arg(positions, "i4", d, None, "positions"), n, n, qop, qos, kop, kos,
                                     _stream(stream, d))
        if rc:
            _check(rc)

    def close(self):
        if getattr(self, "h", None):
            self.L.moe_rotary_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Kv4:
    """One layer's paged key/value cache in 4 bits (moe_kv4_*): the plan, its workspace, and the cache, uint8
    [n_pages][kv_heads][page_size * head_dim * 17 / 16] (`cache` to use a given one).  `workspace`: another plan,
    used on the same stream, whose workspace this one shares.  All of a plan's arrays are on one device, which is
    the current one where its methods are called."""

    def __init__(self, q_heads: int, kv_heads: int, head_dim: int, page_size: int, n_pages: int, sliding_window: int = 0,
                 softmax_scale: float | None = None, sinks=None, cache=None, workspace: "Kv4 | None" = None, device="cuda"):
        import torch
        self.L = load()
        h = self.L.moe_kv4_create(q_heads, kv_heads, head_dim, page_size, n_pages)
        if not h:
            raise MoeError(MOE_EINVAL, self.L.moe_last_error().decode())
        self.h = C.c_void_p(h)
        self.q_heads, self.kv_heads, self.head_dim, self.page_size, self.n_pages = q_heads, kv_heads, head_dim, page_size, n_pages
        _check(self.L.moe_kv4_set_i(self.h, b"sliding_window", int(sliding_window)))
        if softmax_scale is not None:
            _check(self.L.moe_kv4_set_f(self.h, b"softmax_scale", float(softmax_scale)))
        page = int(self.L.moe_kv4_page_bytes(self.h))
        if cache is None:
            cache = torch.zeros((n_pages, kv_heads, page // kv_heads), dtype=torch.uint8, device=device)
        self.cache = cache
        d = self.device = cache.get_device()   # whose tensors and streams the calls take
        if d < 0:
            raise MoeError(MOE_EINVAL, "cache: a CUDA tensor is needed")
        _check(self.L.moe_kv4_set_cache(self.h, _arg(cache, "u1", d, n_pages * page, "cache")))
        self.sinks = sinks
        _check(self.L.moe_kv4_set_sinks(self.h, _arg(sinks, "f4", d, q_heads, "sinks", none=True)))
        n = int(self.L.moe_kv4_workspace_bytes(self.h))
        self.ws = torch.empty(n + 256, dtype=torch.uint8, device=cache.device) if workspace is None else workspace.ws
        if self.ws.numel() < n + 256:
            raise MoeError(MOE_ENOMEM, "the shared workspace is too small for this plan")
        at = _arg(self.ws, "u1", d, None, "workspace")
        with torch.cuda.device(d):
            _check(self.L.moe_kv4_set_workspace(self.h, at + (-at) % 256, n))

    _on = Kv8._on

    def _rows(self, k, v, slots, d):
        kp, ks = _head_rows(k, self.kv_heads, self.head_dim, d, "k")
        vp, vs = _head_rows(v, self.kv_heads, self.head_dim, d, "v")
        n = k.shape[0]
        if v.shape[0] != n:
            raise MoeError(MOE_EINVAL, "k and v must have the same number of rows")
        return kp, vp, ks, vs, _arg(slots, "i4", d, n, "slots"), n

    def append(self, k, v, slots, stream=None):
        """k, v: bf16 [n][kv_heads][head_dim] (rows may be strided); slots: int32 [n]."""
        d = self._on(k, "k")
        kp, vp, ks, vs, at, n = self._rows(k, v, slots, d)
        rc = self.L.moe_kv4_append(self.h, kp, vp, ks, vs, at, n, _stream(stream, d))
        if rc:
            _check(rc)

    def read(self, slots, k, v, stream=None):
        """What the cache holds at slots into k, v, as append takes them."""
        d = self._on(k, "k")
        kp, vp, ks, vs, at, n = self._rows(k, v, slots, d)
        rc = self.L.moe_kv4_read(self.h, at, n, kp, vp, ks, vs, _stream(stream, d))
        if rc:
            _check(rc)

    def attend(self, q, lens, table, out, starts=None, max_new: int = 1, stream=None):
        """q, out: bf16 [n_rows][q_heads][head_dim] (rows may be strided); lens int32 [n_seqs]; table int32
        [n_seqs][width]; starts int32 [n_seqs + 1] (None: one row a sequence); max_new: most rows of a sequence."""
        d = self._on(q, "q")
        qp, qs = _head_rows(q, self.q_heads, self.head_dim, d, "q")
        op, os_ = _head_rows(out, self.q_heads, self.head_dim, d, "out")
        n, width = table.shape
        if out.shape[0] != q.shape[0]:
            raise MoeError(MOE_EINVAL, "q and out must have the same number of rows")
        rc = self.L.moe_kv4_attend(self.h, qp, qs, _arg(starts, "i4", d, n + 1, "starts", none=True), _arg(lens, "i4", d, n, "lens"),
                                   _arg(table, "i4", d, None, "table"), width, n, max_new, q.shape[0], op, os_, _stream(stream, d))
        if rc:
            _check(rc)

    def device_status(self, stream=None) -> int:
        s = C.c_int(0)
        rc = self.L.moe_kv4_get_device_status(self.h, C.byref(s), _stream(stream, self._on(self.ws, "the plan")))
        if rc not in (MOE_OK, MOE_EDEVICE):
            _check(rc)
        return s.value

    def close(self):
        if getattr(self, "h", None):
            self.L.moe_kv4_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Verify:
    """Verification of drafted tokens (moe_verify) in calls of at most max_rows rows: holds their workspace, which
    is on the device that is current where it is made.  Calls that can overlap on the GPU need one each."""

    def __init__(self, max_rows: int, device="cuda"):
        import torch
        self.L, self.max_rows = load(), int(max_rows)
        n = int(self.L.moe_verify_workspace_bytes(self.max_rows))
        self.ws = torch.empty(max(n, 16), dtype=torch.uint8, device=device)
        self.bytes, self.device = n, self.ws.get_device()
        if self.device < 0:
            raise MoeError(MOE_EINVAL, "the workspace: a CUDA device is needed")

    def run(self, logits, drafts, u, draws, starts, ids, accepted, draft_probs=None, temperature=None, top_k=None, top_p=None,
            min_p=None, stream=None):
        """logits [n][vocab] fp32 or bf16 (rows may be strided): sequence b's rows are starts[b] .. starts[b + 1] - 1
        (int32 [n_seqs + 1]); drafts int32 [n], draft_probs fp32 [n][vocab] (rows may be strided; None: drafted tokens
        were certain), u float32 [n], draws float32 [n_seqs], in [0, 1); temperature, top_p, min_p float32 [n_seqs]
        and top_k int32 [n_seqs], each may be None.  Writes ids int32 [n] and accepted int32 [n_seqs]."""
        shape, kinds = logits.shape, _DTYPES or _dtypes()
        bf16 = logits.dtype is kinds["b2"]
        d = _device(logits, "logits")
        if d != self.device:
            raise MoeError(MOE_EINVAL, f"the workspace is on device {self.device}, the current device is {d}")
        if len(shape) != 2 or not (bf16 or logits.dtype is kinds["f4"]) or (shape[0] and logits.stride(1) != 1 and shape[1] > 1):
            raise MoeError(MOE_EINVAL, "logits: a CUDA tensor of fp32 or bf16 rows is needed")
        n, vocab = shape
        probs, probs_stride = None, 0
        if draft_probs is not None:
            if draft_probs.dtype is not kinds["f4"] or draft_probs.get_device() != d or draft_probs.shape != shape or \
                    (n and draft_probs.stride(1) != 1 and vocab > 1):
                raise MoeError(MOE_EINVAL, f"draft_probs: a CUDA tensor of fp32 rows [{n}][{vocab}] on device {d} is needed")
            probs, probs_stride = draft_probs.data_ptr(), draft_probs.stride(0) if n > 1 else vocab
        S = starts.numel() - 1
        rc = self.L.moe_verify(
            logits.data_ptr(), bf16, n, vocab, logits.stride(0) if n > 1 else vocab, _arg(drafts, "i4", d, n, "drafts"), probs, probs_stride,
            _arg(starts, "i4", d, None, "starts"), S, _arg(temperature, "f4", d, S, "temperature", none=True),
            _arg(top_k, "i4", d, S, "top_k", none=True), _arg(top_p, "f4", d, S, "top_p", none=True),
            _arg(min_p, "f4", d, S, "min_p", none=True), _arg(u, "f4", d, n, "u"), _arg(draws, "f4", d, S, "draws"),
            _arg(ids, "i4", d, n, "ids"), _arg(accepted, "i4", d, S, "accepted"), _arg(self.ws, "u1", d, None, "workspace"), self.bytes,
            _stream(stream, d))
        if rc:
            _check(rc)
