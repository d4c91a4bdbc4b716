"""Python binding of libmoe_offload.so (the C ABI in include/moe_offload.h).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels. torch supplies device memory (tensors) and streams. There is no
fallback: without the built library every call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_offload.so")

MOE_OK, MOE_E_INVALID, MOE_E_NOMEM, MOE_E_HOST_NOMEM, MOE_E_HIP, MOE_E_UNSUPPORTED, MOE_E_STATE = range(7)
ACT_F32, ACT_BF16 = 0, 1
HOST_COMPUTE_NONE, HOST_COMPUTE_MISSES, HOST_COMPUTE_LAYER = 0, 1, 2


class Config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("group_size", ctypes.c_int32), ("num_layers", ctypes.c_int32),
                ("act_dtype", ctypes.c_int32), ("max_tokens", ctypes.c_int32), ("hbm_slots", ctypes.c_int32),
                ("gemm_min_tokens", ctypes.c_int32), ("prefill_stage_slots", ctypes.c_int32),
                ("weight_bits", ctypes.c_int32), ("prefetch_slots", ctypes.c_int32)]


class LayerWeights(ctypes.Structure):
    _fields_ = [("router_w", ctypes.c_void_p), ("router_b", ctypes.c_void_p), ("experts", ctypes.c_void_p)]


class Routing(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("topk_ids", ctypes.c_void_p), ("topk_w", ctypes.c_void_p),
                ("counts", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("sorted", ctypes.c_void_p),
                ("inv", ctypes.c_void_p)]


class Stats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("forwards", "tokens", "hits", "misses", "bytes_hbm", "bytes_host",
                                              "bytes_copied", "promotions", "evictions", "host_computed",
                                              "prefetched")]

    def as_dict(self):
        return {n: int(getattr(self, n)) for n, _ in self._fields_}


class CachePolicy(ctypes.Structure):
    _fields_ = [("decay", ctypes.c_double), ("max_promotions", ctypes.c_int32), ("overlap", ctypes.c_int32),
                ("want_resident", ctypes.c_void_p)]


class PlanInfo(ctypes.Structure):
    _fields_ = [("device", ctypes.c_int32), ("gpu_numa_node", ctypes.c_int32), ("host_pool_node", ctypes.c_int32),
                ("numa_bound", ctypes.c_int32), ("internal_expert_bytes", ctypes.c_int64),
                ("host_pool_bytes", ctypes.c_int64), ("hbm_slot_bytes", ctypes.c_int64),
                ("workspace_bytes", ctypes.c_int64)]

    def as_dict(self):
        return {n: int(getattr(self, n)) for n, _ in self._fields_}


class LinkCeilings(ctypes.Structure):
    _fields_ = [("hbm_read_gbps", ctypes.c_double), ("host_read_gbps", ctypes.c_double),
                ("h2d_copy_gbps", ctypes.c_double)]


class RmsNormArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("act_dtype", ctypes.c_int32),
                ("add_dtype", ctypes.c_int32), ("eps", ctypes.c_float), ("x", ctypes.c_void_p),
                ("ld_x", ctypes.c_int64), ("add", ctypes.c_void_p), ("ld_add", ctypes.c_int64),
                ("weight", ctypes.c_void_p), ("x_out", ctypes.c_void_p), ("ld_x_out", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("ld_out", ctypes.c_int64), ("q_out", ctypes.c_void_p),
                ("ld_q", ctypes.c_int64), ("s_out", ctypes.c_void_p)]


class QuantizeArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("act_dtype", ctypes.c_int32), ("x", ctypes.c_void_p),
                ("ld_x", ctypes.c_int64), ("q_out", ctypes.c_void_p), ("ld_q", ctypes.c_int64),
                ("s_out", ctypes.c_void_p)]


class Int8MatmulArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("q_x", ctypes.c_void_p), ("ld_x", ctypes.c_int64), ("s_x", ctypes.c_void_p),
                ("q_w", ctypes.c_void_p), ("ld_w", ctypes.c_int64), ("s_w", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("y_in", ctypes.c_void_p), ("ld_y", ctypes.c_int64),
                ("res", ctypes.c_void_p), ("ld_res", ctypes.c_int64), ("out", ctypes.c_void_p),
                ("ld_out", ctypes.c_int64)]


class Int8FfnArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("q_x", ctypes.c_void_p), ("ld_x", ctypes.c_int64), ("s_x", ctypes.c_void_p),
                ("q_gu", ctypes.c_void_p), ("ld_gu", ctypes.c_int64), ("s_gu", ctypes.c_void_p),
                ("q_dn", ctypes.c_void_p), ("ld_dn", ctypes.c_int64), ("s_dn", ctypes.c_void_p),
                ("y_in", ctypes.c_void_p), ("ld_y", ctypes.c_int64), ("res", ctypes.c_void_p),
                ("ld_res", ctypes.c_int64), ("out", ctypes.c_void_p), ("ld_out", ctypes.c_int64),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


KERNELS = ["router", "route", "gateup", "down", "combine", "gemm_gateup", "gemm_down", "stage"]


class KernelTimes(ctypes.Structure):
    _fields_ = [("launches", ctypes.c_int64 * 8), ("total_ms", ctypes.c_double * 8)]


class MoeError(RuntimeError):
    def __init__(self, status, fn, msg):
        super().__init__("%s failed: %s (%s)" % (fn, _status_name(status), msg))
        self.status = status


_lib = None


def _status_name(s):
    return ["MOE_OK", "MOE_E_INVALID", "MOE_E_NOMEM", "MOE_E_HOST_NOMEM", "MOE_E_HIP", "MOE_E_UNSUPPORTED",
            "MOE_E_STATE"][s] if 0 <= s < 7 else str(s)


def load_library(path: str = LIB_PATH, with_torch: bool = True):
    """Load the library. With torch, torch is imported first so that the library
    binds to the same HIP runtime as torch's tensors and streams."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError("libmoe_offload.so is not built (%s): run __graft_entry__.build() or "
                           "python expert_offloaded_ffn_moe_amd/build.py" % path)
    if with_torch:
        import torch  # noqa: F401
    lib = ctypes.CDLL(path)
    vp, i32, st = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int
    lib.moe_expert_bytes.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(ctypes.c_size_t)]
    lib.moe_plan_create.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(LayerWeights), vp, vp, ctypes.POINTER(vp)]
    lib.moe_plan_load_layer.argtypes = [vp, i32, ctypes.POINTER(LayerWeights), vp, vp]
    lib.moe_plan_get_info.argtypes = [vp, ctypes.POINTER(PlanInfo)]
    lib.moe_measure_link_ceilings.argtypes = [ctypes.c_size_t, ctypes.c_size_t, i32, vp, ctypes.POINTER(LinkCeilings)]
    lib.moe_debug_fail_alloc.argtypes = [i32, i32]
    lib.moe_plan_set_host_compute.argtypes = [vp, i32, i32, i32]
    lib.moe_prefetch.argtypes = [vp, i32, i32, vp, vp, i32, vp, vp]
    lib.moe_plan_prefetch_slots.argtypes = [vp, i32, vp]
    lib.moe_debug_live_allocs.argtypes = [ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int64)]
    lib.moe_layer_forward.argtypes = [vp, i32, i32, vp, vp, vp, ctypes.POINTER(Routing), vp]
    lib.moe_layer_forward_noalloc.argtypes = [vp, i32, i32, vp, vp, vp, ctypes.POINTER(Routing), vp]
    lib.moe_layer_forward_residual.argtypes = [vp, i32, i32, vp, vp, vp, vp, ctypes.POINTER(Routing), vp]
    lib.moe_cache_update.argtypes = [vp, i32, ctypes.POINTER(CachePolicy), vp]
    lib.moe_plan_stats.argtypes = [vp, i32, ctypes.POINTER(Stats)]
    lib.moe_plan_reset_stats.argtypes = [vp]
    lib.moe_plan_residency.argtypes = [vp, i32, vp]
    lib.moe_plan_profile.argtypes = [vp, i32]
    lib.moe_plan_kernel_times.argtypes = [vp, ctypes.POINTER(KernelTimes)]
    lib.moe_rms_norm.argtypes = [vp, vp]  # a RmsNormArgs
    lib.moe_quantize_rows.argtypes = [vp, vp]  # a QuantizeArgs
    lib.moe_int8_matmul.argtypes = [vp, vp]  # a Int8MatmulArgs
    lib.moe_int8_ffn_workspace.argtypes = [i32, i32, i32, ctypes.POINTER(ctypes.c_size_t)]
    lib.moe_int8_ffn.argtypes = [vp, vp]  # a Int8FfnArgs
    lib.moe_plan_destroy.argtypes = [vp]
    lib.moe_plan_destroy.restype = None
    lib.moe_status_str.argtypes = [st]
    lib.moe_status_str.restype = ctypes.c_char_p
    lib.moe_last_error.restype = ctypes.c_char_p
    for fn in ("moe_expert_bytes", "moe_plan_create", "moe_plan_load_layer", "moe_layer_forward",
               "moe_layer_forward_noalloc", "moe_layer_forward_residual",
               "moe_cache_update", "moe_plan_stats", "moe_plan_reset_stats", "moe_plan_residency",
               "moe_plan_profile", "moe_plan_kernel_times", "moe_plan_get_info", "moe_measure_link_ceilings",
               "moe_debug_fail_alloc", "moe_debug_live_allocs", "moe_plan_set_host_compute",
               "moe_prefetch", "moe_plan_prefetch_slots", "moe_rms_norm", "moe_quantize_rows", "moe_int8_matmul",
               "moe_int8_ffn_workspace", "moe_int8_ffn"):
        getattr(lib, fn).restype = st
    _lib = lib
    return lib


def _check(status, fn):
    if status != MOE_OK:
        raise MoeError(status, fn, _lib.moe_last_error().decode())


def _ptr(t):
    """Device/host address of a torch tensor or numpy array (None -> NULL)."""
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        assert t.flags["C_CONTIGUOUS"]
        return t.ctypes.data
    assert t.is_contiguous()
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def measure_link_ceilings(hbm_bytes=1 << 30, host_bytes=1 << 30, iters=5, stream=None) -> dict:
    """Streaming-read GB/s over device memory and over pinned device-mapped host memory,
    and host -> device copy GB/s (moe_measure_link_ceilings)."""
    lib = load_library()
    out = LinkCeilings()
    _check(lib.moe_measure_link_ceilings(hbm_bytes, host_bytes, iters, _stream(stream), ctypes.byref(out)),
           "moe_measure_link_ceilings")
    return {n: float(getattr(out, n)) for n, _ in out._fields_}


def debug_fail_alloc(kind: int, n: int):
    """Test hook: the n-th next device (kind 0) or pinned host (kind 1) allocation fails."""
    lib = load_library()
    _check(lib.moe_debug_fail_alloc(kind, n), "moe_debug_fail_alloc")


def debug_live_allocs():
    """(device, pinned host) allocations the library currently holds."""
    lib = load_library()
    d, h = ctypes.c_int64(), ctypes.c_int64()
    _check(lib.moe_debug_live_allocs(ctypes.byref(d), ctypes.byref(h)), "moe_debug_live_allocs")
    return int(d.value), int(h.value)


def make_config(H, I, E, k, G, act="bf16", num_layers=1, max_tokens=16, hbm_slots=None, gemm_min_tokens=0,
                prefill_stage_slots=0, weight_bits=4, prefetch_slots=0):
    return Config(H, I, E, k, G, num_layers, ACT_BF16 if act == "bf16" else ACT_F32, max_tokens,
                  E if hbm_slots is None else hbm_slots, gemm_min_tokens, prefill_stage_slots, weight_bits,
                  prefetch_slots)


def expert_bytes(cfg: Config) -> int:
    lib = load_library()
    out = ctypes.c_size_t()
    _check(lib.moe_expert_bytes(ctypes.byref(cfg), ctypes.byref(out)), "moe_expert_bytes")
    return int(out.value)


def _layer_weights(router_w, router_b, experts):
    """(LayerWeights, the arrays it points into, kept alive by the caller)."""
    rw = np.ascontiguousarray(router_w)
    rb = None if router_b is None else np.ascontiguousarray(router_b, dtype=np.float32)
    ex = np.ascontiguousarray(experts, dtype=np.uint8)
    return LayerWeights(_ptr(rw), _ptr(rb), _ptr(ex)), (rw, rb, ex)


# ---- dense operators beside the routed layer
#
# Tensors are on one GPU, matrices two-dimensional with consecutive elements in a row and
# rows that do not overlap (any row stride from their length on; an expanded row is
# refused), vectors packed. The work runs on `stream` (default: torch's current
# stream of that GPU); the GPU need not be the current one.


# A call of a few tokens takes less time on the GPU than a handful of Python calls, so the
# checks below read each tensor's properties once, and the arguments are packed into the
# bytes of their C struct at once (0.4 us less than filling the ctypes mirror).


def _packer(mirror):
    """Struct.pack of a ctypes mirror's layout."""
    codes = {ctypes.c_int32: "i", ctypes.c_float: "f", ctypes.c_int64: "q", ctypes.c_void_p: "P", ctypes.c_size_t: "N"}
    s = struct.Struct("@" + "".join(codes[c] for _, c in mirror._fields_))
    assert s.size == ctypes.sizeof(mirror)
    return s.pack


_pack_norm, _pack_quantize = _packer(RmsNormArgs), _packer(QuantizeArgs)
_pack_matmul, _pack_ffn = _packer(Int8MatmulArgs), _packer(Int8FfnArgs)


class _Torch:
    """What the dense operators take of torch, once it is imported."""
    acts = None  # torch dtype -> moe_act_dtype; None until then


def _load_torch():
    import torch
    load_library()
    _Torch.f32, _Torch.bf16, _Torch.i8, _Torch.u8 = torch.float32, torch.bfloat16, torch.int8, torch.uint8
    _Torch.stream, _Torch.device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    _Torch.acts = {torch.bfloat16: ACT_BF16, torch.float32: ACT_F32}


def _refuse(fn, msg):
    raise MoeError(MOE_E_INVALID, fn, msg)


def _refuse_numbers(fn, **numbers):
    """For what struct.error says of a number that its field of the ABI cannot hold."""
    _refuse(fn, "out of range: %s" % ", ".join("%s = %s" % n for n in numbers.items()))


def _refuse_tensor(fn, name, t, shape, dtype, dev):
    if t.dtype is not dtype:
        _refuse(fn, "%s has dtype %s, not %s" % (name, t.dtype, dtype))
    if t.get_device() < 0:
        _refuse(fn, "%s is not on a GPU" % name)
    if t.get_device() != dev:
        _refuse(fn, "%s is on another GPU than the other tensors" % name)
    if t.shape != shape:
        _refuse(fn, "%s has shape %s, not %s" % (name, tuple(t.shape), shape))
    _refuse(fn, "%s: the elements of a row are not consecutive" % name)


def _mat(fn, name, t, rows, cols, dtype, dev):
    """(address, row stride) of a matrix, (0, 0) for None."""
    if t is None:
        return 0, 0
    if t.dtype is dtype and t.get_device() == dev and t.shape == (rows, cols):
        if t.is_contiguous():
            return t.data_ptr(), cols
        ld, step = t.stride()
        if step == 1 or cols == 1:
            if rows == 1:  # its stride says nothing, and may be less than its length
                return t.data_ptr(), cols
            if ld >= cols:
                return t.data_ptr(), ld
            # a broadcast row among them: the ABI's stride of 0 stands for packed rows
            _refuse(fn, "%s: its rows overlap (row stride %d for %d elements): pass a tensor that holds every row" % (name, ld, cols))
    _refuse_tensor(fn, name, t, (rows, cols), dtype, dev)


def _vec(fn, name, t, n, dtype, dev):
    """Address of a packed vector, 0 for None."""
    if t is None:
        return 0
    if t.dtype is dtype and t.get_device() == dev and t.shape == (n,) and t.is_contiguous():
        return t.data_ptr()
    _refuse_tensor(fn, name, t, (n,), dtype, dev)


def _act_of(fn, name, t):
    """moe_act_dtype of a tensor."""
    act = _Torch.acts.get(t.dtype)
    if act is None:
        _refuse(fn, "%s has dtype %s, not bfloat16 or float32" % (name, t.dtype))
    return act


def _shape2(fn, name, t):
    s = t.shape
    if len(s) != 2:
        _refuse(fn, "%s has %d dimensions, not 2" % (name, len(s)))
    return s


def _run(fn, name, args, dev, stream):
    """Enqueue on `stream`, by default torch's current stream of GPU `dev`."""
    if dev < 0:
        _refuse(name, "the tensors are not on a GPU")
    if stream is None:
        s = _Torch.stream(dev)
    else:
        if getattr(stream, "device_index", dev) != dev:
            _refuse(name, "the stream is on another GPU than the tensors")
        s = _stream(stream)
    if dev == _Torch.device():
        status = fn(args, s)
    else:
        import torch
        with torch.cuda.device(dev):
            status = fn(args, s)
    if status != MOE_OK:
        _check(status, name)


def rms_norm(x, weight, eps=1e-6, add=None, x_out=None, out=None, q_out=None, s_out=None, stream=None):
    """Root-mean-square norm of s = x + add (add: x's dtype, or float32 such as forward()'s y):
    x_out = s rounded to x's dtype, out = the norm in x's dtype, q_out int8 [T, H] and s_out
    float32 [T] = its codes and scales; any of the outputs may be None (moe_rms_norm)."""
    if _Torch.acts is None:
        _load_torch()
    fn, f32 = "moe_rms_norm", _Torch.f32
    T, H = _shape2(fn, "x", x)
    dt, dev = x.dtype, x.get_device()
    act = _act_of(fn, "x", x)
    adt = dt if add is None else add.dtype
    if adt is not dt and adt is not f32:
        _refuse(fn, "add has dtype %s, not %s or float32" % (adt, dt))
    try:
        a = _pack_norm(T, H, act, act if adt is dt else ACT_F32, eps, *_mat(fn, "x", x, T, H, dt, dev),
                       *_mat(fn, "add", add, T, H, adt, dev), _vec(fn, "weight", weight, H, dt, dev),
                       *_mat(fn, "x_out", x_out, T, H, dt, dev), *_mat(fn, "out", out, T, H, dt, dev),
                       *_mat(fn, "q_out", q_out, T, H, _Torch.i8, dev), _vec(fn, "s_out", s_out, T, f32, dev))
    except struct.error:
        _refuse_numbers(fn, T=T, H=H, eps=eps)
    _run(_lib.moe_rms_norm, fn, a, dev, stream)


def quantize_rows(x, q_out, s_out, stream=None):
    """int8 codes q_out [T, H] and float32 scales s_out [T] of the rows of x [T, H]
    (moe_quantize_rows): activations, or a weight matrix, whose rows are its channels."""
    if _Torch.acts is None:
        _load_torch()
    fn = "moe_quantize_rows"
    T, H = _shape2(fn, "x", x)
    dev = x.get_device()
    try:
        a = _pack_quantize(T, H, _act_of(fn, "x", x), *_mat(fn, "x", x, T, H, x.dtype, dev),
                           *_mat(fn, "q_out", q_out, T, H, _Torch.i8, dev), _vec(fn, "s_out", s_out, T, _Torch.f32, dev))
    except struct.error:
        _refuse_numbers(fn, T=T, H=H)
    _run(_lib.moe_quantize_rows, fn, a, dev, stream)


def int8_matmul(q_x, s_x, q_w, s_w, out, bias=None, y_in=None, res=None, stream=None):
    """out [T, N] = act(s_x s_w (q_x @ q_w.T) + bias + y_in + res), q_x int8 [T, K], q_w int8
    [N, K]; bias float32 [N], y_in float32 [T, N], res in out's dtype; out may be y_in or
    res (moe_int8_matmul)."""
    if _Torch.acts is None:
        _load_torch()
    fn, f32, i8 = "moe_int8_matmul", _Torch.f32, _Torch.i8
    T, K = _shape2(fn, "q_x", q_x)
    N = _shape2(fn, "q_w", q_w)[0]
    dt, dev = out.dtype, q_x.get_device()
    try:
        a = _pack_matmul(T, N, K, _act_of(fn, "out", out), *_mat(fn, "q_x", q_x, T, K, i8, dev),
                         _vec(fn, "s_x", s_x, T, f32, dev), *_mat(fn, "q_w", q_w, N, K, i8, dev),
                         _vec(fn, "s_w", s_w, N, f32, dev), _vec(fn, "bias", bias, N, f32, dev),
                         *_mat(fn, "y_in", y_in, T, N, f32, dev), *_mat(fn, "res", res, T, N, dt, dev),
                         *_mat(fn, "out", out, T, N, dt, dev))
    except struct.error:
        _refuse_numbers(fn, T=T, N=N, K=K)
    _run(_lib.moe_int8_matmul, fn, a, dev, stream)
    return out


def int8_ffn_workspace(T, H, I) -> int:
    """Bytes of workspace that int8_ffn needs for T tokens (moe_int8_ffn_workspace)."""
    lib = load_library()
    n = ctypes.c_size_t()
    if not all(-(1 << 31) <= v < 1 << 31 for v in (T, H, I)):  # ctypes would drop their high bits
        _refuse_numbers("moe_int8_ffn_workspace", T=T, H=H, I=I)
    _check(lib.moe_int8_ffn_workspace(T, H, I, ctypes.byref(n)), "moe_int8_ffn_workspace")
    return int(n.value)


def int8_ffn(q_x, s_x, q_gu, s_gu, q_dn, s_dn, out, workspace, y_in=None, res=None, stream=None):
    """Gated feed-forward block on 8-bit codes: q_x int8 [T, H], q_gu int8 [2I, H] (gate rows,
    then up rows), q_dn int8 [H, I]; out [T, H] = act(block + y_in + res). workspace: a uint8
    tensor of int8_ffn_workspace(T, H, I) bytes, one for each call in flight (moe_int8_ffn)."""
    if _Torch.acts is None:
        _load_torch()
    fn, f32, i8 = "moe_int8_ffn", _Torch.f32, _Torch.i8
    T, H = _shape2(fn, "q_x", q_x)
    I = _shape2(fn, "q_dn", q_dn)[1]
    dt, dev, n = out.dtype, q_x.get_device(), workspace.numel()
    try:
        a = _pack_ffn(T, H, I, _act_of(fn, "out", out), *_mat(fn, "q_x", q_x, T, H, i8, dev),
                      _vec(fn, "s_x", s_x, T, f32, dev), *_mat(fn, "q_gu", q_gu, 2 * I, H, i8, dev),
                      _vec(fn, "s_gu", s_gu, 2 * I, f32, dev), *_mat(fn, "q_dn", q_dn, H, I, i8, dev),
                      _vec(fn, "s_dn", s_dn, H, f32, dev), *_mat(fn, "y_in", y_in, T, H, f32, dev),
                      *_mat(fn, "res", res, T, H, dt, dev), *_mat(fn, "out", out, T, H, dt, dev),
                      _vec(fn, "workspace", workspace, n, _Torch.u8, dev), n)
    except struct.error:
        _refuse_numbers(fn, T=T, H=H, I=I)
    _run(_lib.moe_int8_ffn, fn, a, dev, stream)
    return out


class Plan:
    """A residency plan: pools, pointer tables and workspace of `cfg.num_layers` layers.

    layers: optional list of (router_w, router_b, experts) per layer, loaded at create;
    initial_hbm: optional host [L, E] int (1 = the expert starts in an HBM slot)."""

    def __init__(self, cfg: Config, layers=None, initial_hbm=None, stream=None):
        self.lib = load_library()
        self.cfg = cfg
        h = ctypes.c_void_p()
        arr, keep, ih = None, [], None
        if layers is not None:
            assert len(layers) == cfg.num_layers
            arr = (LayerWeights * len(layers))()
            for i, (rw, rb, ex) in enumerate(layers):
                arr[i], k = _layer_weights(rw, rb, ex)
                keep.append(k)
            if initial_hbm is not None:
                ih = np.ascontiguousarray(initial_hbm, dtype=np.int32)
                assert ih.shape == (cfg.num_layers, cfg.num_experts)
        _check(self.lib.moe_plan_create(ctypes.byref(cfg), arr, _ptr(ih), _stream(stream), ctypes.byref(h)),
               "moe_plan_create")
        self.handle = h

    def load_layer(self, layer, router_w: np.ndarray, router_b, experts: np.ndarray, resident=None, stream=None):
        """router_w: host [E, H] float32 (f32 plans) or uint16 bf16 bits (bf16 plans);
        router_b: host [E] float32 or None; experts: host uint8 [E, expert_bytes];
        resident: host [E] int (1 = the expert starts in an HBM slot) or None."""
        w, keep = _layer_weights(router_w, router_b, experts)
        res = None if resident is None else np.ascontiguousarray(resident, dtype=np.int32)
        _check(self.lib.moe_plan_load_layer(self.handle, layer, ctypes.byref(w), _ptr(res), _stream(stream)),
               "moe_plan_load_layer")
        del keep

    def forward(self, layer, x, y, logits_in=None, route=None, stream=None):
        """x: cuda tensor [T, H] (float32 or bfloat16); y: cuda float32 [T, H];
        route: optional dict of cuda tensors named like the moe_routing fields."""
        T = int(x.shape[0])
        r = None
        if route is not None:
            r = Routing(*[_ptr(route.get(n)) for n, _ in Routing._fields_])
        _check(self.lib.moe_layer_forward(self.handle, layer, T, _ptr(x), _ptr(logits_in), _ptr(y),
                                          ctypes.byref(r) if r is not None else None, _stream(stream)),
               "moe_layer_forward")
        return y

    def forward_residual(self, layer, x, y, x_out, logits_in=None, route=None, stream=None):
        """forward() that also writes x_out = x + y in x's dtype (the residual stream's
        next value), from the kernel that writes y."""
        T = int(x.shape[0])
        r = None
        if route is not None:
            r = Routing(*[_ptr(route.get(n)) for n, _ in Routing._fields_])
        _check(self.lib.moe_layer_forward_residual(self.handle, layer, T, _ptr(x), _ptr(logits_in), _ptr(y),
                                                   _ptr(x_out), ctypes.byref(r) if r is not None else None,
                                                   _stream(stream)), "moe_layer_forward_residual")
        return y

    def forward_noalloc(self, layer, x, y, logits_in=None, route=None, stream=None):
        """forward() through moe_layer_forward_noalloc: the workspace comes from the
        library's static per-device array, and the call allocates nothing."""
        T = int(x.shape[0])
        r = None
        if route is not None:
            r = Routing(*[_ptr(route.get(n)) for n, _ in Routing._fields_])
        _check(self.lib.moe_layer_forward_noalloc(self.handle, layer, T, _ptr(x), _ptr(logits_in), _ptr(y),
                                                  ctypes.byref(r) if r is not None else None, _stream(stream)),
               "moe_layer_forward_noalloc")
        return y

    def cache_update(self, layer=-1, decay=0.9, max_promotions=8, overlap=False, want_resident=None, stream=None):
        """overlap=True: the pipelined update (decisions lag one update; copies on the
        plan's copy stream, promoted experts switched to HBM by the next update).
        want_resident: host [E] (one layer) or [L, E] (layer = -1) ints, the residency
        set to move to instead of the frequency policy's choice."""
        want = None if want_resident is None else np.ascontiguousarray(want_resident, dtype=np.int32)
        pol = CachePolicy(decay, max_promotions, 1 if overlap else 0, _ptr(want))
        _check(self.lib.moe_cache_update(self.handle, layer, ctypes.byref(pol), _stream(stream)),
               "moe_cache_update")

    def prefetch(self, layer, x=None, logits_in=None, candidates=0, predicted_out=None, stream=None):
        """Predict the layer's experts from x (cuda [T, H], the layer's router applied to
        it) or logits_in (cuda float32 [T, E]) and copy the host-read ones among them
        into the layer's prefetch slots, on the plan's prefetch stream, after the work
        enqueued on `stream` so far. predicted_out: optional cuda int32 [prefetch_slots]."""
        src = logits_in if logits_in is not None else x
        T = int(src.shape[0])
        _check(self.lib.moe_prefetch(self.handle, layer, T, _ptr(x), _ptr(logits_in), candidates,
                                     _ptr(predicted_out), _stream(stream)), "moe_prefetch")

    def prefetch_slots(self, layer) -> np.ndarray:
        """Expert held by each prefetch slot of the layer (-1 none); waits for its prefetch."""
        out = np.empty(self.cfg.prefetch_slots, dtype=np.int32)
        _check(self.lib.moe_plan_prefetch_slots(self.handle, layer, out.ctypes.data), "moe_plan_prefetch_slots")
        return out

    def set_host_compute(self, layer=-1, mode=HOST_COMPUTE_MISSES, threads=0):
        """Where the layer's experts are computed: HOST_COMPUTE_NONE (the GPU, offloaded ones
        read over the host link), HOST_COMPUTE_MISSES (the host cores compute the offloaded
        ones), HOST_COMPUTE_LAYER (the host cores compute all of them)."""
        _check(self.lib.moe_plan_set_host_compute(self.handle, layer, mode, threads), "moe_plan_set_host_compute")

    def info(self) -> dict:
        out = PlanInfo()
        _check(self.lib.moe_plan_get_info(self.handle, ctypes.byref(out)), "moe_plan_get_info")
        return out.as_dict()

    def stats(self, layer=-1) -> dict:
        s = Stats()
        _check(self.lib.moe_plan_stats(self.handle, layer, ctypes.byref(s)), "moe_plan_stats")
        return s.as_dict()

    def reset_stats(self):
        _check(self.lib.moe_plan_reset_stats(self.handle), "moe_plan_reset_stats")

    def residency(self, layer) -> np.ndarray:
        out = np.empty(self.cfg.num_experts, dtype=np.int32)
        _check(self.lib.moe_plan_residency(self.handle, layer, out.ctypes.data), "moe_plan_residency")
        return out

    def profile(self, enable: bool):
        _check(self.lib.moe_plan_profile(self.handle, 1 if enable else 0), "moe_plan_profile")

    def kernel_times(self) -> dict:
        """{kernel class: (launches, total ms)} of the recorded launches."""
        kt = KernelTimes()
        _check(self.lib.moe_plan_kernel_times(self.handle, ctypes.byref(kt)), "moe_plan_kernel_times")
        return {n: (int(kt.launches[i]), float(kt.total_ms[i])) for i, n in enumerate(KERNELS)}

    def destroy(self):
        if self.handle:
            self.lib.moe_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass
