"""Python binding of libnvfp4.so: the functions of include/nvfp4.h,
include/nvfp4_attn.h and include/nvfp4_attn_long.h, same names.

Argument marshalling only: torch tensors supply device memory and the current
stream; every step of the computation runs in the library's HIP kernels.  If
the library is not built, every call raises -- there is no fallback path.
"""
import ctypes
import os
import warnings

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4.so")

NVFP4_OK = 0
NVFP4_ERR_NULL = 1
NVFP4_ERR_SHAPE = 2
NVFP4_ERR_ALIGN = 3
NVFP4_ERR_DTYPE = 4
NVFP4_ERR_WORKSPACE = 5
NVFP4_ERR_ARG = 6
NVFP4_ERR_HIP = 7
NVFP4_F32 = 0
NVFP4_BF16 = 1

EXPORTED = (
    "nvfp4_abi_version", "nvfp4_status_str", "nvfp4_last_error", "nvfp4_packed_bytes", "nvfp4_pack",
    "nvfp4_unpack", "nvfp4_gemv_workspace_bytes", "nvfp4_gemv", "nvfp4_gemm_workspace_bytes", "nvfp4_gemm",
    "nvfp4_gemv_batched_workspace_bytes", "nvfp4_gemv_batched", "nvfp4_gemm_batched_workspace_bytes",
    "nvfp4_gemm_batched", "nvfp4_moe_workspace_bytes", "nvfp4_moe_grouped", "nvfp4_quantize_workspace_bytes",
    "nvfp4_quantize", "nvfp4_expert_cache_reset", "nvfp4_moe_streamed", "nvfp4_mx_packed_bytes", "nvfp4_mx_pack",
    "nvfp4_mx_unpack", "nvfp4_w4a4_workspace_bytes", "nvfp4_w4a4_gemm", "nvfp4_w4a4_batched_workspace_bytes",
    "nvfp4_w4a4_batched", "nvfp4_gemv_batched_noalloc",
)

# include/nvfp4_attn.h
NVFP4_ROPE_HALF = 0
NVFP4_ROPE_INTERLEAVED = 1
NVFP4_ROPE_NONE = 0
NVFP4_ROPE_LINEAR = 1
NVFP4_ROPE_YARN = 2
NVFP4_KV_BF16 = 0
NVFP4_KV_E4M3 = 1
NVFP4_KV_NVFP4 = 2
NVFP4_ATTN_COUNTER_BYTES = 1024

EXPORTED_ATTN = (
    "nvfp4_rope_freqs", "nvfp4_rope", "nvfp4_kv_cache_bytes", "nvfp4_kv_append", "nvfp4_kv_read",
    "nvfp4_attn_decode_workspace_bytes", "nvfp4_attn_decode",
)

# include/nvfp4_attn_long.h
NVFP4_SELECT_COUNTER_BYTES = 4096

EXPORTED_ATTN_LONG = (
    "nvfp4_attn_shared_workspace_bytes", "nvfp4_attn_shared", "nvfp4_kv_bounds", "nvfp4_kv_select_workspace_bytes",
    "nvfp4_kv_select", "nvfp4_attn_decode_heads", "nvfp4_attn_weigh_workspace_bytes", "nvfp4_attn_weigh",
    "nvfp4_kv_evict_workspace_bytes", "nvfp4_kv_evict",
)


class Nvfp4Error(RuntimeError):
    def __init__(self, status, message):
        super().__init__(message)
        self.status = status


class Problem(ctypes.Structure):
    """Mirror of struct nvfp4_problem."""
    _fields_ = [
        ("packed", ctypes.c_void_p), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
        ("tensor_scale", ctypes.c_float), ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
        ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64),
    ]


class MoeArgs(ctypes.Structure):
    """Mirror of struct nvfp4_moe_args."""
    _fields_ = [
        ("tokens", ctypes.c_int64), ("experts", ctypes.c_int64), ("top_k", ctypes.c_int64),
        ("hidden", ctypes.c_int64), ("inter", ctypes.c_int64),
        ("x", ctypes.c_void_p), ("router_logits", ctypes.c_void_p),
        ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
        ("stride_gate", ctypes.c_size_t), ("stride_up", ctypes.c_size_t), ("stride_down", ctypes.c_size_t),
        ("scale_gate", ctypes.c_void_p), ("scale_up", ctypes.c_void_p), ("scale_down", ctypes.c_void_p),
        ("y", ctypes.c_void_p), ("y_dtype", ctypes.c_int),
        ("topk_ids", ctypes.c_void_p), ("topk_weights", ctypes.c_void_p),
        ("expert_counts", ctypes.c_void_p), ("expert_offsets", ctypes.c_void_p), ("perm", ctypes.c_void_p),
        ("dbg_gate", ctypes.c_void_p), ("dbg_up", ctypes.c_void_p), ("dbg_h", ctypes.c_void_p),
        ("dbg_down", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class ExpertCache(ctypes.Structure):
    """Mirror of struct nvfp4_expert_cache."""
    _fields_ = [
        ("experts", ctypes.c_int64), ("slots", ctypes.c_int64),
        ("host_gate", ctypes.c_void_p), ("host_up", ctypes.c_void_p), ("host_down", ctypes.c_void_p),
        ("dev_gate", ctypes.c_void_p), ("dev_up", ctypes.c_void_p), ("dev_down", ctypes.c_void_p),
        ("stride_gate", ctypes.c_size_t), ("stride_up", ctypes.c_size_t), ("stride_down", ctypes.c_size_t),
        ("dev_slot_of", ctypes.c_void_p), ("host_counts", ctypes.c_void_p), ("host_slot_stage", ctypes.c_void_p),
        ("slot_of", ctypes.c_void_p), ("expert_in", ctypes.c_void_p), ("last_use", ctypes.c_void_p),
        ("clock", ctypes.c_uint64),
        ("last_active", ctypes.c_int64), ("last_fetched", ctypes.c_int64), ("last_bytes", ctypes.c_size_t),
    ]


class RopeConfig(ctypes.Structure):
    """Mirror of struct nvfp4_rope_config."""
    _fields_ = [
        ("rot_dim", ctypes.c_int64), ("base", ctypes.c_double), ("scaling", ctypes.c_int), ("factor", ctypes.c_double),
        ("original_max", ctypes.c_double), ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double),
    ]


class RopeArgs(ctypes.Structure):
    """Mirror of struct nvfp4_rope_args."""
    _fields_ = [
        ("tokens", ctypes.c_int64), ("heads", ctypes.c_int64), ("head_dim", ctypes.c_int64), ("rot_dim", ctypes.c_int64),
        ("layout", ctypes.c_int), ("inverse", ctypes.c_int), ("magnitude", ctypes.c_float),
        ("positions", ctypes.c_void_p), ("freqs", ctypes.c_void_p),
        ("x", ctypes.c_void_p), ("x_dtype", ctypes.c_int), ("ldx", ctypes.c_int64),
        ("y", ctypes.c_void_p), ("y_dtype", ctypes.c_int), ("ldy", ctypes.c_int64),
    ]


class KvCacheDesc(ctypes.Structure):
    """Mirror of struct nvfp4_kv_cache."""
    _fields_ = [
        ("pool", ctypes.c_void_p), ("pages", ctypes.c_int64), ("page_size", ctypes.c_int64),
        ("kv_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64), ("format", ctypes.c_int),
        ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float),
    ]


class KvAppendArgs(ctypes.Structure):
    """Mirror of struct nvfp4_kv_append_args."""
    _fields_ = [
        ("cache", ctypes.POINTER(KvCacheDesc)), ("tokens", ctypes.c_int64), ("slots", ctypes.c_void_p),
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int),
        ("ldk", ctypes.c_int64), ("ldv", ctypes.c_int64),
        ("freqs", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("rot_dim", ctypes.c_int64),
        ("layout", ctypes.c_int), ("magnitude", ctypes.c_float),
        ("q_heads", ctypes.c_int64), ("q", ctypes.c_void_p), ("ldq", ctypes.c_int64),
        ("q_out", ctypes.c_void_p), ("ldqo", ctypes.c_int64),
    ]


class AttnArgs(ctypes.Structure):
    """Mirror of struct nvfp4_attn_args."""
    _fields_ = [
        ("cache", ctypes.POINTER(KvCacheDesc)), ("batch", ctypes.c_int64), ("q_heads", ctypes.c_int64),
        ("q", ctypes.c_void_p), ("ldq", ctypes.c_int64), ("page_table", ctypes.c_void_p),
        ("table_width", ctypes.c_int64), ("seq_lens", ctypes.c_void_p), ("scale", ctypes.c_float),
        ("window", ctypes.c_int64), ("out", ctypes.c_void_p), ("ldo", ctypes.c_int64), ("lse", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class AttnSharedArgs(ctypes.Structure):
    """Mirror of struct nvfp4_attn_shared_args."""
    _fields_ = [("attn", AttnArgs), ("prefix_table", ctypes.c_void_p), ("prefix_width", ctypes.c_int64),
                ("prefix_len", ctypes.c_void_p)]


class AttnWeighArgs(ctypes.Structure):
    """Mirror of struct nvfp4_attn_weigh_args."""
    _fields_ = [("attn", AttnArgs), ("weights", ctypes.c_void_p), ("decay", ctypes.c_float), ("weights_out", ctypes.c_void_p)]


class KvSelectArgs(ctypes.Structure):
    """Mirror of struct nvfp4_kv_select_args."""
    _fields_ = [
        ("cache", ctypes.POINTER(KvCacheDesc)), ("batch", ctypes.c_int64), ("q_heads", ctypes.c_int64),
        ("q", ctypes.c_void_p), ("ldq", ctypes.c_int64), ("bounds", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
        ("table_width", ctypes.c_int64), ("seq_lens", ctypes.c_void_p), ("budget", ctypes.c_int64),
        ("pages_out", ctypes.c_void_p), ("lens_out", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class KvEvictArgs(ctypes.Structure):
    """Mirror of struct nvfp4_kv_evict_args."""
    _fields_ = [
        ("batch", ctypes.c_int64), ("kv_heads", ctypes.c_int64), ("page_size", ctypes.c_int64), ("weights", ctypes.c_void_p),
        ("page_table", ctypes.c_void_p), ("table_width", ctypes.c_int64), ("seq_lens", ctypes.c_void_p),
        ("budget", ctypes.c_int64), ("sink", ctypes.c_int64), ("recent", ctypes.c_int64), ("table_out", ctypes.c_void_p),
        ("lens_out", ctypes.c_void_p), ("weights_out", ctypes.c_void_p), ("freed", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


_lib = None


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m bit_quantized_decode_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, i64, sz, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    sig = {
        "nvfp4_abi_version": (I, []),
        "nvfp4_status_str": (ctypes.c_char_p, [I]),
        "nvfp4_last_error": (ctypes.c_char_p, []),
        "nvfp4_packed_bytes": (I, [i64, i64, ctypes.POINTER(sz)]),
        "nvfp4_pack": (I, [P, P, i64, i64, P, P]),
        "nvfp4_unpack": (I, [P, i64, i64, P, P, P]),
        "nvfp4_gemv_workspace_bytes": (I, [i64, i64, ctypes.POINTER(sz)]),
        "nvfp4_gemv": (I, [P, i64, i64, ctypes.c_float, P, P, P, sz, P]),
        "nvfp4_gemm_workspace_bytes": (I, [i64, i64, i64, ctypes.POINTER(sz)]),
        "nvfp4_gemm": (I, [P, i64, i64, ctypes.c_float, P, i64, i64, P, i64, I, P, sz, P]),
        "nvfp4_gemv_batched_workspace_bytes": (I, [ctypes.POINTER(Problem), I, ctypes.POINTER(sz)]),
        "nvfp4_gemv_batched": (I, [ctypes.POINTER(Problem), I, P, sz, P]),
        "nvfp4_gemv_batched_noalloc": (I, [ctypes.POINTER(Problem), I, P]),
        "nvfp4_gemm_batched_workspace_bytes": (I, [ctypes.POINTER(Problem), I, i64, ctypes.POINTER(sz)]),
        "nvfp4_gemm_batched": (I, [ctypes.POINTER(Problem), I, i64, I, P, sz, P]),
        "nvfp4_moe_workspace_bytes": (I, [ctypes.POINTER(MoeArgs), ctypes.POINTER(sz)]),
        "nvfp4_moe_grouped": (I, [ctypes.POINTER(MoeArgs), P]),
        "nvfp4_quantize_workspace_bytes": (I, [ctypes.POINTER(sz)]),
        "nvfp4_quantize": (I, [P, I, i64, i64, i64, P, P, P, P, sz, P]),
        "nvfp4_expert_cache_reset": (I, [ctypes.POINTER(ExpertCache)]),
        "nvfp4_moe_streamed": (I, [ctypes.POINTER(MoeArgs), ctypes.POINTER(ExpertCache), P]),
        "nvfp4_mx_packed_bytes": (I, [i64, i64, ctypes.POINTER(sz)]),
        "nvfp4_mx_pack": (I, [P, P, i64, i64, P, P]),
        "nvfp4_mx_unpack": (I, [P, i64, i64, P, P, P]),
        "nvfp4_w4a4_workspace_bytes": (I, [i64, i64, ctypes.POINTER(sz)]),
        "nvfp4_w4a4_gemm": (I, [P, i64, i64, ctypes.c_float, P, i64, i64, P, i64, I, P, sz, P]),
        "nvfp4_w4a4_batched_workspace_bytes": (I, [ctypes.POINTER(Problem), I, i64, ctypes.POINTER(sz)]),
        "nvfp4_w4a4_batched": (I, [ctypes.POINTER(Problem), I, i64, I, P, sz, P]),
        "nvfp4_rope_freqs": (I, [ctypes.POINTER(RopeConfig), P, ctypes.POINTER(ctypes.c_float)]),
        "nvfp4_rope": (I, [ctypes.POINTER(RopeArgs), P]),
        "nvfp4_kv_cache_bytes": (I, [ctypes.POINTER(KvCacheDesc), ctypes.POINTER(sz)]),
        "nvfp4_kv_append": (I, [ctypes.POINTER(KvAppendArgs), P]),
        "nvfp4_kv_read": (I, [ctypes.POINTER(KvCacheDesc), P, i64, P, i64, P, i64, I, P]),
        "nvfp4_attn_decode_workspace_bytes": (I, [ctypes.POINTER(AttnArgs), ctypes.POINTER(sz)]),
        "nvfp4_attn_decode": (I, [ctypes.POINTER(AttnArgs), P]),
        "nvfp4_attn_shared_workspace_bytes": (I, [ctypes.POINTER(AttnSharedArgs), ctypes.POINTER(sz)]),
        "nvfp4_attn_shared": (I, [ctypes.POINTER(AttnSharedArgs), P]),
        "nvfp4_kv_bounds": (I, [ctypes.POINTER(KvCacheDesc), P, i64, P, P]),
        "nvfp4_kv_select_workspace_bytes": (I, [ctypes.POINTER(KvSelectArgs), ctypes.POINTER(sz)]),
        "nvfp4_kv_select": (I, [ctypes.POINTER(KvSelectArgs), P]),
        "nvfp4_attn_decode_heads": (I, [ctypes.POINTER(AttnArgs), P]),
        "nvfp4_attn_weigh_workspace_bytes": (I, [ctypes.POINTER(AttnWeighArgs), ctypes.POINTER(sz)]),
        "nvfp4_attn_weigh": (I, [ctypes.POINTER(AttnWeighArgs), P]),
        "nvfp4_kv_evict_workspace_bytes": (I, [ctypes.POINTER(KvEvictArgs), ctypes.POINTER(sz)]),
        "nvfp4_kv_evict": (I, [ctypes.POINTER(KvEvictArgs), P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def check(status):
    if status != NVFP4_OK:
        L = lib()
        raise Nvfp4Error(status, f"{L.nvfp4_status_str(status).decode()}: {L.nvfp4_last_error().decode()}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# Zero-initialised workspaces, one per (device, kind), reused across calls in
# stream order.  "split" serves the GEMV / GEMM split-K reductions, whose
# counters every call leaves at zero; "moe" holds the MoE intermediates.  The
# two kinds never share memory, so MoE scratch cannot disturb the counters.
_workspaces = {}


def workspace(nbytes, device, kind="split"):
    if nbytes == 0:
        return None
    key = (str(device), kind)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


def abi_version():
    return lib().nvfp4_abi_version()


def packed_bytes(n, k):
    out = ctypes.c_size_t()
    check(lib().nvfp4_packed_bytes(n, k, ctypes.byref(out)))
    return out.value


def pack(codes, scales, stream=None):
    """codes uint8 [n][k/2], scales uint8 [n][k/16] (device) -> packed uint8 buffer."""
    n, kh = codes.shape
    k = 2 * kh
    packed = torch.empty(packed_bytes(n, k), dtype=torch.uint8, device=codes.device)
    check(lib().nvfp4_pack(_ptr(codes), _ptr(scales), n, k, _ptr(packed), _stream(stream)))
    return packed


def mx_packed_bytes(rows, k):
    out = ctypes.c_size_t()
    check(lib().nvfp4_mx_packed_bytes(rows, k, ctypes.byref(out)))
    return out.value


def mx_pack(codes, scales, stream=None):
    """Canonical NVFP4 codes [n][k/2], scales [n][k/16] (device) -> MX tiles for nvfp4_w4a4_gemm."""
    n, kh = codes.shape
    k = 2 * kh
    out = torch.empty(mx_packed_bytes(n, k), dtype=torch.uint8, device=codes.device)
    check(lib().nvfp4_mx_pack(_ptr(codes), _ptr(scales), n, k, _ptr(out), _stream(stream)))
    return out


def mx_unpack(mx, rows, k, stream=None):
    codes = torch.empty((rows, k // 2), dtype=torch.uint8, device=mx.device)
    scales = torch.empty((rows, k // 32), dtype=torch.uint8, device=mx.device)
    check(lib().nvfp4_mx_unpack(_ptr(mx), rows, k, _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


def w4a4_workspace_bytes(m, k):
    out = ctypes.c_size_t()
    check(lib().nvfp4_w4a4_workspace_bytes(m, k, ctypes.byref(out)))
    return out.value


def w4a4_x_tiles(ws, m, k):
    """The MX tiles of x that the last nvfp4_w4a4_gemm left in workspace ws."""
    off = w4a4_workspace_bytes(m, k) - mx_packed_bytes(m, k)
    return ws[off:off + mx_packed_bytes(m, k)]


def w4a4_gemm(mx, n, k, tensor_scale, x, y=None, y_dtype=torch.bfloat16, ws=None, stream=None):
    """y[m][n] = s_t * x' W'^T over MX FP4 operands (see nvfp4_w4a4_gemm); ws (zeroed
    before its first use) receives the schedule's counters and x's MX tiles."""
    m = x.shape[0]
    if y is None:
        y = torch.empty((m, n), dtype=y_dtype, device=x.device)
    if ws is None:
        ws = workspace(w4a4_workspace_bytes(m, k), x.device, kind="w4a4")
    dt = NVFP4_BF16 if y.dtype == torch.bfloat16 else NVFP4_F32
    check(lib().nvfp4_w4a4_gemm(_ptr(mx), n, k, float(tensor_scale), _ptr(x), m, x.stride(0), _ptr(y), y.stride(0),
                                dt, _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))
    return y


def w4a4_batched_workspace_bytes(items, m):
    """Workspace bytes nvfp4_w4a4_batched needs for these problems at m activation rows."""
    need = ctypes.c_size_t()
    check(lib().nvfp4_w4a4_batched_workspace_bytes(problems(items), len(items), m, ctypes.byref(need)))
    return need.value


def w4a4_batched(items, ws=None, stream=None):
    """Several W4A4 products sharing m and the output dtype:
    items = [(mx_tiles, n, k, tensor_scale, x [m][ldx], y [m][ldy])]."""
    arr = problems(items)
    m = items[0][4].shape[0] if items else 0
    dt = NVFP4_BF16 if items and items[0][5].dtype == torch.bfloat16 else NVFP4_F32
    if ws is None and items:
        ws = workspace(w4a4_batched_workspace_bytes(items, m), items[0][4].device, kind="w4a4")
    check(lib().nvfp4_w4a4_batched(arr, len(items), m, dt, _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))


def w4a4_batched_prepared(items, ws=None, stream=None):
    """nvfp4_w4a4_batched with its arguments marshalled once: returns a
    zero-argument callable that only makes the library call."""
    arr = problems(items)
    m = items[0][4].shape[0] if items else 0
    dt = NVFP4_BF16 if items and items[0][5].dtype == torch.bfloat16 else NVFP4_F32
    if ws is None and items:
        ws = workspace(w4a4_batched_workspace_bytes(items, m), items[0][4].device, kind="w4a4")
    fn, n, wsp, wsb = lib().nvfp4_w4a4_batched, len(items), _ptr(ws), 0 if ws is None else ws.numel()
    keep = (items, ws)

    def call():
        check(fn(arr, n, m, dt, wsp, wsb, _stream(stream)))
        return keep

    return call


def quantize_workspace_bytes():
    out = ctypes.c_size_t()
    check(lib().nvfp4_quantize_workspace_bytes(ctypes.byref(out)))
    return out.value


def quantize(w, codes=None, scales=None, tensor_scale=None, ws=None, stream=None):
    """NVFP4-encode w (device, float32 or bfloat16, [n][k], rows may be strided):
    returns (codes uint8 [n][k/2], scales uint8 [n][k/16], tensor_scale float32 [1])."""
    n, k = w.shape
    dtype = {torch.float32: NVFP4_F32, torch.bfloat16: NVFP4_BF16}[w.dtype]
    dev = w.device
    if codes is None:
        codes = torch.empty((n, k // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((n, k // 16), dtype=torch.uint8, device=dev)
    if tensor_scale is None:
        tensor_scale = torch.empty(1, dtype=torch.float32, device=dev)
    if ws is None:
        ws = workspace(quantize_workspace_bytes(), dev, kind="quantize")
    check(lib().nvfp4_quantize(_ptr(w), dtype, n, k, w.stride(0) if n > 0 else k, _ptr(codes), _ptr(scales),
                               _ptr(tensor_scale), _ptr(ws), ws.numel(), _stream(stream)))
    return codes, scales, tensor_scale


def unpack(packed, n, k, stream=None):
    codes = torch.empty((n, k // 2), dtype=torch.uint8, device=packed.device)
    scales = torch.empty((n, k // 16), dtype=torch.uint8, device=packed.device)
    check(lib().nvfp4_unpack(_ptr(packed), n, k, _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


def gemv_workspace_bytes(n, k):
    out = ctypes.c_size_t()
    check(lib().nvfp4_gemv_workspace_bytes(n, k, ctypes.byref(out)))
    return out.value


def gemv(packed, n, k, tensor_scale, x, y=None, ws=None, stream=None):
    """y[n] fp32 = s_t * W x, x bf16 [k] (device)."""
    if y is None:
        y = torch.empty(n, dtype=torch.float32, device=x.device)
    need = gemv_workspace_bytes(n, k)
    if ws is None:
        ws = workspace(need, x.device)
    check(lib().nvfp4_gemv(_ptr(packed), n, k, float(tensor_scale), _ptr(x), _ptr(y), _ptr(ws),
                           0 if ws is None else ws.numel(), _stream(stream)))
    return y


def gemm_workspace_bytes(m, n, k):
    out = ctypes.c_size_t()
    check(lib().nvfp4_gemm_workspace_bytes(m, n, k, ctypes.byref(out)))
    return out.value


def gemm(packed, n, k, tensor_scale, x, y=None, y_dtype=torch.bfloat16, ws=None, stream=None):
    """y[m][n] = s_t * x W^T, x bf16 [m][ldx] (device, row stride x.stride(0))."""
    m = x.shape[0]
    if y is None:
        y = torch.empty((m, n), dtype=y_dtype, device=x.device)
    dt = NVFP4_BF16 if y.dtype == torch.bfloat16 else NVFP4_F32
    need = gemm_workspace_bytes(m, n, k)
    if ws is None:
        ws = workspace(need, x.device)
    check(lib().nvfp4_gemm(_ptr(packed), n, k, float(tensor_scale), _ptr(x), m, x.stride(0), _ptr(y), y.stride(0),
                           dt, _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))
    return y


def problems(items):
    """ctypes array of Problem from (packed, n, k, tensor_scale, x, y) tuples of tensors."""
    arr = (Problem * len(items))()
    for i, (packed, n, k, st, x, y) in enumerate(items):
        arr[i].packed = packed.data_ptr()
        arr[i].n, arr[i].k, arr[i].tensor_scale = n, k, float(st)
        arr[i].x = x.data_ptr()
        arr[i].ldx = x.stride(0) if x.dim() == 2 else k
        arr[i].y = y.data_ptr()
        arr[i].ldy = y.stride(0) if y.dim() == 2 else n
    return arr


def gemv_batched(items, ws=None, stream=None):
    """Several GEMVs in one launch: items = [(packed, n, k, tensor_scale, x [k], y fp32 [n]), ...]."""
    arr = problems(items)
    L = lib()
    need = ctypes.c_size_t()
    check(L.nvfp4_gemv_batched_workspace_bytes(arr, len(items), ctypes.byref(need)))
    if ws is None and items:
        ws = workspace(need.value, items[0][4].device)
    check(L.nvfp4_gemv_batched(arr, len(items), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))


def gemv_batched_noalloc(items, stream=None):
    """nvfp4_gemv_batched_noalloc: the batched GEMV with the library's static
    device scratch instead of a workspace (same items as gemv_batched)."""
    arr = problems(items)
    check(lib().nvfp4_gemv_batched_noalloc(arr, len(items), _stream(stream)))


def gemv_batched_prepared(items, ws=None, stream=None):
    """nvfp4_gemv_batched with its arguments marshalled once: returns a
    zero-argument callable that only makes the library call (for tight
    launch loops)."""
    arr = problems(items)
    L = lib()
    need = ctypes.c_size_t()
    check(L.nvfp4_gemv_batched_workspace_bytes(arr, len(items), ctypes.byref(need)))
    if ws is None and items:
        ws = workspace(need.value, items[0][4].device)
    fn, n, wsp, wsb = L.nvfp4_gemv_batched, len(items), _ptr(ws), 0 if ws is None else ws.numel()
    keep = (items, ws)  # the tensors must outlive the callable

    def call():
        # The stream is looked up per call (None: the current one), so that a
        # call under graph capture lands on the capturing stream.
        check(fn(arr, n, wsp, wsb, _stream(stream)))
        return keep

    return call


def gemm_batched_workspace_bytes(items, m):
    """Workspace bytes nvfp4_gemm_batched needs for these problems at m activation rows."""
    arr = problems(items)
    need = ctypes.c_size_t()
    check(lib().nvfp4_gemm_batched_workspace_bytes(arr, len(items), m, ctypes.byref(need)))
    return need.value


def gemm_batched(items, ws=None, stream=None):
    """Several GEMMs sharing m and the output dtype: items = [(packed, n, k, tensor_scale, x [m][ldx], y [m][ldy])]."""
    arr = problems(items)
    L = lib()
    m = items[0][4].shape[0] if items else 0
    dt = NVFP4_BF16 if items and items[0][5].dtype == torch.bfloat16 else NVFP4_F32
    need = ctypes.c_size_t()
    check(L.nvfp4_gemm_batched_workspace_bytes(arr, len(items), m, ctypes.byref(need)))
    if ws is None and items:
        ws = workspace(need.value, items[0][4].device)
    check(L.nvfp4_gemm_batched(arr, len(items), m, dt, _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))


def gemm_batched_prepared(items, ws=None, stream=None):
    """nvfp4_gemm_batched with its arguments marshalled once: returns a
    zero-argument callable that only makes the library call."""
    arr = problems(items)
    L = lib()
    m = items[0][4].shape[0] if items else 0
    dt = NVFP4_BF16 if items and items[0][5].dtype == torch.bfloat16 else NVFP4_F32
    need = ctypes.c_size_t()
    check(L.nvfp4_gemm_batched_workspace_bytes(arr, len(items), m, ctypes.byref(need)))
    if ws is None and items:
        ws = workspace(need.value, items[0][4].device)
    fn, n, wsp, wsb = L.nvfp4_gemm_batched, len(items), _ptr(ws), 0 if ws is None else ws.numel()
    keep = (items, ws)

    def call():
        check(fn(arr, n, m, dt, wsp, wsb, _stream(stream)))
        return keep

    return call


def moe_args(**kw):
    a = MoeArgs()
    for key, val in kw.items():
        if isinstance(val, torch.Tensor):
            val = val.data_ptr()
        setattr(a, key, val)
    return a


def moe_workspace_bytes(tokens, experts, top_k, hidden, inter):
    a = moe_args(tokens=tokens, experts=experts, top_k=top_k, hidden=hidden, inter=inter)
    out = ctypes.c_size_t()
    check(lib().nvfp4_moe_workspace_bytes(ctypes.byref(a), ctypes.byref(out)))
    return out.value


def moe_grouped(x, logits, top_k, w_gate, w_up, w_down, stride_gate, stride_up, stride_down,
                scale_gate, scale_up, scale_down, inter, y_dtype=torch.float32, debug=False, ws=None,
                outputs=None, stream=None):
    """The routed expert layer.  Returns a dict of the outputs (see nvfp4_moe_grouped).
    w_gate may be an ExpertStream (then w_up, w_down and the strides are taken from it)."""
    streamed = w_gate if isinstance(w_gate, ExpertStream) else None
    if streamed is not None:
        w_gate, w_up, w_down = streamed.dev
        stride_gate, stride_up, stride_down = streamed.strides
    tokens, hidden = x.shape
    experts = logits.shape[1]
    dev = x.device
    o = outputs if outputs is not None else {}
    flat = tokens * top_k
    o.setdefault("y", torch.empty((tokens, hidden), dtype=y_dtype, device=dev))
    o.setdefault("topk_ids", torch.empty((tokens, top_k), dtype=torch.int32, device=dev))
    o.setdefault("topk_weights", torch.empty((tokens, top_k), dtype=torch.float32, device=dev))
    o.setdefault("expert_counts", torch.empty(experts, dtype=torch.int32, device=dev))
    o.setdefault("expert_offsets", torch.empty(experts + 1, dtype=torch.int32, device=dev))
    o.setdefault("perm", torch.empty(flat, dtype=torch.int32, device=dev))
    if debug:
        o.setdefault("dbg_gate", torch.empty((flat, inter), dtype=torch.float32, device=dev))
        o.setdefault("dbg_up", torch.empty((flat, inter), dtype=torch.float32, device=dev))
        o.setdefault("dbg_h", torch.empty((flat, inter), dtype=torch.bfloat16, device=dev))
        o.setdefault("dbg_down", torch.empty((flat, hidden), dtype=torch.float32, device=dev))
    if ws is None:
        ws = workspace(moe_workspace_bytes(tokens, experts, top_k, hidden, inter), dev, kind="moe")
    a = moe_args(
        tokens=tokens, experts=experts, top_k=top_k, hidden=hidden, inter=inter, x=x, router_logits=logits,
        w_gate=w_gate, w_up=w_up, w_down=w_down, stride_gate=stride_gate, stride_up=stride_up,
        stride_down=stride_down, scale_gate=scale_gate, scale_up=scale_up, scale_down=scale_down,
        y=o["y"], y_dtype=NVFP4_BF16 if o["y"].dtype == torch.bfloat16 else NVFP4_F32,
        topk_ids=o["topk_ids"], topk_weights=o["topk_weights"], expert_counts=o["expert_counts"],
        expert_offsets=o["expert_offsets"], perm=o["perm"],
        dbg_gate=o.get("dbg_gate"), dbg_up=o.get("dbg_up"), dbg_h=o.get("dbg_h"), dbg_down=o.get("dbg_down"),
        workspace=ws, workspace_bytes=0 if ws is None else ws.numel(),
    )
    if streamed is not None:
        check(lib().nvfp4_moe_streamed(ctypes.byref(a), ctypes.byref(streamed.cache), _stream(stream)))
    else:
        check(lib().nvfp4_moe_grouped(ctypes.byref(a), _stream(stream)))
    return o


class ExpertStream:
    """Routed experts streamed from pinned host memory through a device cache
    of `slots` expert slots (nvfp4_moe_streamed).  pool_*: the packed expert
    pools (uint8 tensors, expert e at e * stride_*, any device); they are
    copied once into pinned host memory.  Pass the object as w_gate to
    moe_grouped (w_up / w_down / strides: None); its device slot pools then
    stand in for the weights."""

    def __init__(self, pool_gate, pool_up, pool_down, stride_gate, stride_up, stride_down, experts, slots, device):
        import numpy as np
        self.host = [torch.empty(p.numel(), dtype=torch.uint8, pin_memory=True) for p in (pool_gate, pool_up, pool_down)]
        for h, p in zip(self.host, (pool_gate, pool_up, pool_down)):
            h.copy_(p.reshape(-1))
        strides = (stride_gate, stride_up, stride_down)
        self.dev = [torch.empty(slots * st, dtype=torch.uint8, device=device) for st in strides]
        self.dev_slot_of = torch.zeros(experts, dtype=torch.int32, device=device)
        self.host_counts = torch.zeros(experts, dtype=torch.int32, pin_memory=True)
        self.host_stage = torch.zeros(experts, dtype=torch.int32, pin_memory=True)
        self.slot_of = np.full(experts, -1, np.int32)
        self.expert_in = np.full(slots, -1, np.int32)
        self.last_use = np.zeros(slots, np.uint64)
        c = ExpertCache()
        c.experts, c.slots = experts, slots
        c.host_gate, c.host_up, c.host_down = (h.data_ptr() for h in self.host)
        c.dev_gate, c.dev_up, c.dev_down = (d.data_ptr() for d in self.dev)
        c.stride_gate, c.stride_up, c.stride_down = strides
        c.dev_slot_of = self.dev_slot_of.data_ptr()
        c.host_counts = self.host_counts.data_ptr()
        c.host_slot_stage = self.host_stage.data_ptr()
        c.slot_of = self.slot_of.ctypes.data
        c.expert_in = self.expert_in.ctypes.data
        c.last_use = self.last_use.ctypes.data
        self.cache = c
        self.strides = strides
        self.reset()

    def reset(self):
        check(lib().nvfp4_expert_cache_reset(ctypes.byref(self.cache)))

    def stats(self):
        c = self.cache
        return {"active": c.last_active, "fetched": c.last_fetched, "bytes": c.last_bytes}


def moe_grouped_prepared(*args, **kw):
    """moe_grouped with its arguments marshalled once (same arguments):
    returns (call, outputs), call() making only the library call."""
    o = moe_grouped(*args, **kw)   # one real call builds and validates everything
    x, logits, top_k = args[0], args[1], args[2]
    tokens, hidden = x.shape
    experts = logits.shape[1]
    inter = args[12]
    ws = kw.get("ws")
    if ws is None:
        ws = workspace(moe_workspace_bytes(tokens, experts, top_k, hidden, inter), x.device, kind="moe")
    a = moe_args(
        tokens=tokens, experts=experts, top_k=top_k, hidden=hidden, inter=inter, x=x, router_logits=logits,
        w_gate=args[3], w_up=args[4], w_down=args[5], stride_gate=args[6], stride_up=args[7],
        stride_down=args[8], scale_gate=args[9], scale_up=args[10], scale_down=args[11],
        y=o["y"], y_dtype=NVFP4_BF16 if o["y"].dtype == torch.bfloat16 else NVFP4_F32,
        topk_ids=o["topk_ids"], topk_weights=o["topk_weights"], expert_counts=o["expert_counts"],
        expert_offsets=o["expert_offsets"], perm=o["perm"],
        dbg_gate=o.get("dbg_gate"), dbg_up=o.get("dbg_up"), dbg_h=o.get("dbg_h"), dbg_down=o.get("dbg_down"),
        workspace=ws, workspace_bytes=ws.numel(),
    )
    fn, ref, stream = lib().nvfp4_moe_grouped, ctypes.byref(a), kw.get("stream")
    keep = (args, kw, o, ws, a)

    def call():
        check(fn(ref, _stream(stream)))
        return keep

    return call, o


# ---- the attention side (include/nvfp4_attn.h) ---------------------------------
#
# Every call here runs on the device of its tensors, whichever is current, on
# `stream` or that device's current stream.  A call told its stream keeps the
# memory of its tensors from reuse until it has run; what it makes belongs to that
# stream, as if made with it current.  Each *_prepared() checks and
# marshals its arguments once and returns a zero-argument callable that makes
# the library call and returns the outputs, the same buffers each time; called with
# another stream current than when it was made, it keeps their memory likewise.

def _device_of(stream, **tensors):
    """The one GPU that all given tensors, and `stream` if it is given, are on."""
    dev = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be on the GPU, not on {t.device}")
        if dev is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, other arguments on {dev}")
        dev = t.device
    if stream is not None and stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    return dev


def _rows(t, name, dtypes, heads=None, head_dim=None, tokens=None):
    """The leading dimension of t [tokens][heads][head_dim] after checking its shape and strides."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens][heads][head_dim], not {tuple(t.shape)}")
    for want, got, what in ((tokens, t.shape[0], "tokens"), (heads, t.shape[1], "heads"), (head_dim, t.shape[2], "head_dim")):
        if want is not None and want != got:
            raise ValueError(f"{name} has {got} {what}, expected {want}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {dtypes}, not {t.dtype}")
    if t.numel() and ((t.shape[2] > 1 and t.stride(2) != 1) or (t.shape[1] > 1 and t.stride(1) != t.shape[2])):
        raise ValueError(f"{name}: the heads of a row must be contiguous (strides {t.stride()})")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


def _vector(t, name, dtype, shape):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {tuple(shape)}, not {tuple(t.shape)} with strides {t.stride()}")
    return t.data_ptr()


def _dtype_code(t):
    return NVFP4_BF16 if t.dtype == torch.bfloat16 else NVFP4_F32


_ACTIVATIONS = (torch.float32, torch.bfloat16)


def _new(make, device, stream):
    """make() with device current, and stream too if one is given: memory made there may be reused on that stream only."""
    with torch.cuda.device(device):
        if stream is None:
            return make()
        with torch.cuda.stream(stream):
            return make()


# The current stream's handle by device index.  torch.cuda.current_stream() makes a Stream object for it, 2.7 us
# of a call's 6.2; without the short way, that one.
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda index: torch.cuda.current_stream(index).cuda_stream)


def _caller(fn, args, device, stream, outputs, keep):
    """The callable of a prepared call: fn(*args, stream) on the tensors' device."""
    index, given = device.index, None if stream is None else stream.cuda_stream
    known = {_current_raw_stream(index)}

    def claim(s):
        # The caller may let go of the callable, or of its tensors, while a call is still queued on a stream that is not theirs:
        # their memory waits for that stream.
        for t in keep:
            t = getattr(t, "pool", getattr(t, "freqs", t))      # of a cache, of a table
            if isinstance(t, torch.Tensor):
                t.record_stream(s)

    if stream is not None:
        claim(stream)

    def call():
        # The current stream is looked up per call, so that a call under graph capture lands on the capturing stream.
        handle = _current_raw_stream(index) if given is None else given
        if given is None and handle not in known:
            claim(torch.cuda.current_stream(index))
            known.add(handle)
        if torch.cuda.current_device() == index:
            status = fn(*args, handle)
        else:
            with torch.cuda.device(index):
                status = fn(*args, handle)
        if status != NVFP4_OK:
            check(status)
        return outputs

    call.keep = keep   # the tensors and structures must outlive the callable
    call.outputs = outputs
    return call


def _clearing(call, ws, counter_bytes, device, stream):
    """The callable of a call prepared under capture.  Its workspace was zeroed by a node of that graph, so that a call
    outside it, or in another graph, may come before that is written: each call clears the counters itself."""
    @torch.inference_mode()     # where the workspace may have been made, and may be written
    def clear():
        ws[:counter_bytes].zero_()

    def clear_and_call():
        _new(clear, device, stream)
        return call()

    clear_and_call.keep, clear_and_call.outputs = call.keep, call.outputs
    return clear_and_call


class RopeTable:
    """A device table of rotary frequencies (nvfp4_rope_freqs, or the caller's own: 64-bit fractions of a turn, at least
    rot_dim / 2 of them), with the layout and magnitude that go with it."""

    def __init__(self, freqs, rot_dim, layout, magnitude):
        self.freqs, self.rot_dim, self.layout, self.magnitude = freqs, rot_dim, layout, magnitude

    def address(self):
        """The table's address, after a check that it holds what the kernels read."""
        f = self.freqs
        if f.dtype not in (torch.int64, torch.uint64):
            raise TypeError(f"a rotary table's frequencies must be 64-bit integers, not {f.dtype}")
        if not f.is_contiguous() or f.numel() < self.rot_dim // 2:
            raise ValueError(f"a rotary table for rot_dim {self.rot_dim} must hold {self.rot_dim // 2} contiguous frequencies, "
                             f"not {tuple(f.shape)} with strides {f.stride()}")
        return f.data_ptr()


def rope_freqs(rot_dim, base=10000.0, scaling=None):
    """(freqs, magnitude): the host table as int64 bit patterns [rot_dim / 2].  scaling: None,
    ("linear", factor) or ("yarn", factor, original_max[, beta_fast, beta_slow])."""
    c = RopeConfig(rot_dim=rot_dim, base=base, scaling=NVFP4_ROPE_NONE, factor=1.0, beta_fast=32.0, beta_slow=1.0)
    if scaling is not None:
        kind, *rest = scaling
        fields = {"linear": ("factor",), "yarn": ("factor", "original_max", "beta_fast", "beta_slow")}.get(kind)
        if fields is None or not rest or len(rest) > len(fields) or (kind == "yarn" and len(rest) not in (2, 4)):
            raise ValueError(f"unknown rotary scaling {scaling!r}")
        c.scaling = NVFP4_ROPE_LINEAR if kind == "linear" else NVFP4_ROPE_YARN
        for field, value in zip(fields, rest):
            setattr(c, field, value)
    freqs = torch.zeros(max(rot_dim, 0) // 2, dtype=torch.int64)
    magnitude = ctypes.c_float()
    check(lib().nvfp4_rope_freqs(ctypes.byref(c), _ptr(freqs), ctypes.byref(magnitude)))
    return freqs, magnitude.value


def rope_table(rot_dim, base=10000.0, layout="half", scaling=None, device="cuda"):
    """A RopeTable on `device`; layout: "half" or "interleaved", the rest as in rope_freqs."""
    code = {"half": NVFP4_ROPE_HALF, "interleaved": NVFP4_ROPE_INTERLEAVED}.get(layout)
    if code is None:
        raise ValueError(f"unknown rotary layout {layout!r}")
    freqs, magnitude = rope_freqs(rot_dim, base, scaling)
    return RopeTable(freqs.to(device), rot_dim, code, magnitude)


def rope_prepared(x, positions, table, out=None, dtype=None, inverse=False, stream=None):
    """rope() with its arguments marshalled once: returns a zero-argument callable that returns `out`."""
    ldx = _rows(x, "x", _ACTIVATIONS)
    tokens, heads, head_dim = x.shape
    if out is not None and dtype is not None and out.dtype != dtype:
        raise TypeError(f"out is {out.dtype}, dtype {dtype}")
    freqs = table.address()
    dev = _device_of(stream, x=x, positions=positions, freqs=table.freqs, out=out)
    if out is None:
        out = _new(lambda: torch.empty((tokens, heads, head_dim), dtype=dtype or x.dtype, device=dev), dev, stream)
    ldy = _rows(out, "out", _ACTIVATIONS, heads, head_dim, tokens)
    a = RopeArgs(tokens=tokens, heads=heads, head_dim=head_dim, rot_dim=table.rot_dim, layout=table.layout,
                 inverse=int(inverse), magnitude=table.magnitude,
                 positions=_vector(positions, "positions", torch.int32, (tokens,)), freqs=freqs,
                 x=x.data_ptr(), x_dtype=_dtype_code(x), ldx=ldx, y=out.data_ptr(), y_dtype=_dtype_code(out), ldy=ldy)
    return _caller(lib().nvfp4_rope, (ctypes.byref(a),), dev, stream, out, (a, x, positions, table, out))


def rope(x, positions, table, out=None, dtype=None, inverse=False, stream=None):
    """Rotary positions: x [tokens][heads][head_dim] (fp32 or bf16; the rows may be strided), positions int32
    [tokens].  Returns out (x itself turns in place; by default a new tensor of `dtype` or x's).
    inverse=True turns back: the gradient of rope() is rope(inverse=True) of the output's gradient."""
    return rope_prepared(x, positions, table, out, dtype, inverse, stream)()


class KvCache:
    """A paged key-value cache (struct nvfp4_kv_cache) with its pool.  fmt: NVFP4_KV_BF16, NVFP4_KV_E4M3 or
    NVFP4_KV_NVFP4 (whose tensor scales are k_scale and v_scale).  A token's slot is page * page_size + offset."""

    def __init__(self, pages, page_size, kv_heads, head_dim, fmt, k_scale=1.0, v_scale=1.0, device="cuda", pool=None):
        self.desc = KvCacheDesc(pool=None, pages=pages, page_size=page_size, kv_heads=kv_heads, head_dim=head_dim,
                                format=fmt, k_scale=k_scale, v_scale=v_scale)
        need = ctypes.c_size_t()
        check(lib().nvfp4_kv_cache_bytes(ctypes.byref(self.desc), ctypes.byref(need)))
        if pool is None:
            pool = torch.empty(need.value, dtype=torch.uint8, device=device)
        if pool.dtype != torch.uint8 or not pool.is_contiguous() or pool.numel() < need.value:
            raise ValueError(f"pool must be contiguous uint8 of at least {need.value} bytes")
        self.pool = pool
        self.desc.pool = pool.data_ptr()
        self.pages, self.page_size, self.kv_heads, self.head_dim, self.fmt = pages, page_size, kv_heads, head_dim, fmt


def _kv_append(cache, k, v, slots, positions, table, q, q_out, stream):
    tokens = k.shape[0]
    ldk = _rows(k, "k", _ACTIVATIONS, cache.kv_heads, cache.head_dim)
    ldv = _rows(v, "v", (k.dtype,), cache.kv_heads, cache.head_dim, tokens)
    freqs = None if table is None else table.address()
    dev = _device_of(stream, pool=cache.pool, k=k, v=v, slots=slots, positions=positions if table is not None else None,
                     freqs=None if table is None else table.freqs, q=q, q_out=q_out)
    a = KvAppendArgs(cache=ctypes.pointer(cache.desc), tokens=tokens, slots=_vector(slots, "slots", torch.int64, (tokens,)),
                     k=k.data_ptr(), v=v.data_ptr(), dtype=_dtype_code(k), ldk=ldk, ldv=ldv)
    if table is not None:
        if positions is None:
            raise ValueError("a rotary table needs positions")
        # A table that turns nothing (rot_dim 0) has no memory of its own: any aligned address stands for it.
        a.freqs = freqs or cache.pool.data_ptr()
        a.positions = _vector(positions, "positions", torch.int32, (tokens,))
        a.rot_dim, a.layout, a.magnitude = table.rot_dim, table.layout, table.magnitude
    elif positions is not None:
        warnings.warn("positions without a rotary table are not used: the keys are stored as they are", stacklevel=3)
    if q is not None:
        a.ldq = _rows(q, "q", (k.dtype,), None, cache.head_dim, tokens)
        if q_out is None:
            q_out = _new(lambda: torch.empty(q.shape, dtype=torch.bfloat16, device=dev), dev, stream)
        a.ldqo = _rows(q_out, "q_out", (torch.bfloat16,), q.shape[1], cache.head_dim, tokens)
        a.q_heads, a.q, a.q_out = q.shape[1], q.data_ptr(), q_out.data_ptr()
    return _caller(lib().nvfp4_kv_append, (ctypes.byref(a),), dev, stream, q_out,
                   (a, cache, k, v, slots, positions, table, q, q_out))


def kv_append_prepared(cache, k, v, slots, positions=None, table=None, q=None, q_out=None, stream=None):
    """kv_append() with its arguments marshalled once: returns a zero-argument callable that returns q_out."""
    return _kv_append(cache, k, v, slots, positions, table, q, q_out, stream)


def kv_append(cache, k, v, slots, positions=None, table=None, q=None, q_out=None, stream=None):
    """Write k, v [tokens][kv_heads][head_dim] (fp32 or bf16) into the cache at slots (int64; outside the pool:
    skipped).  With table (and positions, int32) k is turned first, and q [tokens][q_heads][head_dim] into q_out
    (bf16), which is returned.  Without a table k is stored as it is, and positions only raise a warning."""
    return _kv_append(cache, k, v, slots, positions, table, q, q_out, stream)()


def kv_read_prepared(cache, slots, k_out=None, v_out=None, dtype=torch.bfloat16, stream=None):
    """kv_read() with its arguments marshalled once: returns a zero-argument callable that returns (k_out, v_out)."""
    tokens = slots.shape[0]
    dev = _device_of(stream, pool=cache.pool, slots=slots, k_out=k_out, v_out=v_out)
    shape = (tokens, cache.kv_heads, cache.head_dim)
    if k_out is None and v_out is None:
        k_out, v_out = (_new(lambda: torch.empty(shape, dtype=dtype, device=dev), dev, stream) for _ in range(2))
    ld, codes = [0, 0], set()
    for i, t in enumerate((k_out, v_out)):
        if t is not None:
            ld[i] = _rows(t, ("k_out", "v_out")[i], _ACTIVATIONS, cache.kv_heads, cache.head_dim, tokens)
            codes.add(_dtype_code(t))
    if len(codes) != 1:
        raise TypeError("k_out and v_out must have the same dtype")
    args = (ctypes.byref(cache.desc), _vector(slots, "slots", torch.int64, (tokens,)), tokens, _ptr(k_out), ld[0],
            _ptr(v_out), ld[1], codes.pop())
    return _caller(lib().nvfp4_kv_read, args, dev, stream, (k_out, v_out), (cache, slots, k_out, v_out))


def kv_read(cache, slots, k_out=None, v_out=None, dtype=torch.bfloat16, stream=None):
    """The values the cache holds at slots (int64): (k, v), each [tokens][kv_heads][head_dim], new tensors of `dtype`.
    Given one of k_out and v_out, only that one is read, in its own dtype.  Rows of slots outside the pool are left as they were."""
    return kv_read_prepared(cache, slots, k_out, v_out, dtype, stream)()


def _attn_workspace(nbytes, device, stream, kind="attn"):
    """The workspace of attention calls without one of their own (kind "select": of page selections).  Calls on one
    stream run one after the other and share; calls on others have another.  Under capture the graph gets one of its
    own, zeroed by a node of the graph: replays may overlap with anything."""
    def make():
        return torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)

    with torch.cuda.device(device):
        if _new(torch.cuda.is_current_stream_capturing, device, stream):   # of the stream that the call runs on
            return _new(make, device, stream)
        s = torch.cuda.current_stream() if stream is None else stream
        key = (str(device), kind, s.cuda_stream)
        ws = _workspaces.get(key)
        if ws is None or ws.numel() < nbytes:
            ws = _workspaces[key] = _new(make, device, stream)
        return ws


def _workspace_of(need, ws, device, stream, prepared, kind):
    """(the workspace of a call that needs `need` bytes, whether it was made for a call prepared under capture)."""
    if ws is not None or not need:
        return ws, False
    if not prepared:
        return _attn_workspace(need, device, stream, kind), False
    ws = _new(lambda: torch.zeros(need, dtype=torch.uint8, device=device), device, stream)
    return ws, _new(torch.cuda.is_current_stream_capturing, device, stream)


def _check_ws(ws):
    if ws is not None and not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous, not {tuple(ws.shape)} with strides {ws.stride()}")


def _attn(q, cache, page_table, seq_lens, scale, window, out, lse, ws, stream, prepared, fn="nvfp4_attn_decode", wrap=None,
          result=None, **tensors):
    """The callable of an attention: `fn` with AttnArgs, or with wrap(AttnArgs), a structure that has them as `attn`; tensors:
    those that wrap() uses, and result: one more that the call returns."""
    ldq = _rows(q, "q", (torch.bfloat16,), None, cache.head_dim)
    batch, q_heads, head_dim = q.shape
    if not isinstance(lse, torch.Tensor) and lse is not True and lse:
        raise TypeError(f"lse must be True, False or a tensor, not {lse!r}")
    _check_ws(ws)
    dev = _device_of(stream, pool=cache.pool, q=q, page_table=page_table, seq_lens=seq_lens, out=out, ws=ws,
                     lse=lse if isinstance(lse, torch.Tensor) else None, **tensors)
    heads = page_table.dim() == 3 and fn == "nvfp4_attn_decode"
    if page_table.dim() != 2 and not heads:
        raise ValueError(f"page_table must be [batch][pages], not {tuple(page_table.shape)}")
    if out is None:
        out = _new(lambda: torch.empty((batch, q_heads, head_dim), dtype=torch.bfloat16, device=dev), dev, stream)
    if lse is True:
        lse = _new(lambda: torch.empty((batch, q_heads), dtype=torch.float32, device=dev), dev, stream)
    width = page_table.shape[-1]
    a = AttnArgs(cache=ctypes.pointer(cache.desc), batch=batch, q_heads=q_heads, q=q.data_ptr(), ldq=ldq,
                 page_table=_vector(page_table, "page_table", torch.int32,
                                    (batch, cache.kv_heads, width) if heads else (batch, width)),
                 table_width=width, seq_lens=_vector(seq_lens, "seq_lens", torch.int32, (batch,)),
                 scale=head_dim ** -0.5 if scale is None else scale, window=window, out=out.data_ptr(),
                 ldo=_rows(out, "out", (torch.bfloat16,), q_heads, head_dim, batch))
    if isinstance(lse, torch.Tensor):
        a.lse = _vector(lse, "lse", torch.float32, (batch, q_heads))
    args = a if wrap is None else wrap(a)
    need = ctypes.c_size_t()
    check(getattr(lib(), f"{fn}_workspace_bytes")(ctypes.byref(args), ctypes.byref(need)))
    ws, captured = _workspace_of(need.value, ws, dev, stream, prepared, "attn")
    if ws is not None:
        attn = a if wrap is None else args.attn
        attn.workspace, attn.workspace_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    outputs = (out,) + ((lse,) if isinstance(lse, torch.Tensor) else ()) + (() if result is None else (result,))
    call = _caller(getattr(lib(), "nvfp4_attn_decode_heads" if heads else fn), (ctypes.byref(args),), dev, stream,
                   outputs if len(outputs) > 1 else out,
                   (a, args, cache, q, page_table, seq_lens, out, lse, ws, *tensors.values()))
    return _clearing(call, ws, NVFP4_ATTN_COUNTER_BYTES, dev, stream) if captured else call


def attn_decode_prepared(q, cache, page_table, seq_lens, scale=None, window=0, out=None, lse=None, ws=None, stream=None):
    """attn_decode() with its arguments marshalled once and a workspace of its own: returns a zero-argument callable
    that returns what attn_decode() does.  Its calls, and replays of graphs that captured them, must not overlap.
    The workspace is zeroed on `stream`, or the stream that is current here: a call on another waits for that one."""
    return _attn(q, cache, page_table, seq_lens, scale, window, out, lse, ws, stream, True)


def attn_decode(q, cache, page_table, seq_lens, scale=None, window=0, out=None, lse=None, ws=None, stream=None):
    """Attention of one new token per sequence over the cache: q bf16 [batch][q_heads][head_dim], page_table int32
    [batch][pages], or [batch][kv_heads][pages] for pages of each kv head's own (as kv_select() gives them), seq_lens int32
    [batch] (with the new token), scale 1 / sqrt(head_dim) by default.  Returns out (bf16 like q), or (out, lse) if lse is
    True or a float32 [batch][q_heads] tensor.  ws: a workspace, zeroed before its first use, that no other running call has; the
    attentions below and kv_select() may have the same one, the calls of include/nvfp4.h not."""
    return _attn(q, cache, page_table, seq_lens, scale, window, out, lse, ws, stream, False)()


# ---- reading less of a long cache (include/nvfp4_attn_long.h) --------------------
#
# As the calls above; *_prepared() as there, a workspace of its own for each.

def _attn_shared(q, cache, prefix_pages, prefix_len, page_table, seq_lens, scale, out, lse, ws, stream, prepared):
    if prefix_pages.dim() != 1:
        raise ValueError(f"prefix_pages must be [pages], not {tuple(prefix_pages.shape)}")
    width = prefix_pages.shape[0]

    def wrap(a):
        return AttnSharedArgs(attn=a, prefix_table=_vector(prefix_pages, "prefix_pages", torch.int32, (width,)),
                              prefix_width=width, prefix_len=_vector(prefix_len, "prefix_len", torch.int32, (1,)))
    return _attn(q, cache, page_table, seq_lens, scale, 0, out, lse, ws, stream, prepared, "nvfp4_attn_shared", wrap,
                 prefix_pages=prefix_pages, prefix_len=prefix_len)


def attn_shared_prepared(q, cache, prefix_pages, prefix_len, page_table, seq_lens, scale=None, out=None, lse=None, ws=None,
                         stream=None):
    """attn_shared() prepared, as attn_decode_prepared() is."""
    return _attn_shared(q, cache, prefix_pages, prefix_len, page_table, seq_lens, scale, out, lse, ws, stream, True)


def attn_shared(q, cache, prefix_pages, prefix_len, page_table, seq_lens, scale=None, out=None, lse=None, ws=None, stream=None):
    """attn_decode() where every sequence's tokens follow a prefix that all share, which is read once: prefix_pages int32
    [pages], prefix_len int32 [1] (its tokens); page_table and seq_lens are of the sequences' own tokens after it, the
    new one among them.  A length below 0: a free place of the batch (zeros, lse -inf)."""
    return _attn_shared(q, cache, prefix_pages, prefix_len, page_table, seq_lens, scale, out, lse, ws, stream, False)()


def kv_bounds_prepared(cache, pages, bounds=None, stream=None):
    """kv_bounds() with its arguments marshalled once: returns a zero-argument callable that returns bounds."""
    if pages.dim() != 1:
        raise ValueError(f"pages must be [n], not {tuple(pages.shape)}")
    dev = _device_of(stream, pool=cache.pool, pages=pages, bounds=bounds)
    shape = (cache.pages, cache.kv_heads, 2, cache.head_dim)
    if bounds is None:
        bounds = _new(lambda: torch.zeros(shape, dtype=torch.bfloat16, device=dev), dev, stream)
    n = pages.shape[0]
    args = (ctypes.byref(cache.desc), _vector(pages, "pages", torch.int32, (n,)), n,
            _vector(bounds, "bounds", torch.bfloat16, shape))
    return _caller(lib().nvfp4_kv_bounds, args, dev, stream, bounds, (cache, pages, bounds))


def kv_bounds(cache, pages, bounds=None, stream=None):
    """The smallest and largest key of each channel in the pages (int32 ids; outside the pool: skipped), which must be
    full: written to bounds bf16 [cache.pages][kv_heads][2][head_dim], by default a new tensor of zeros.  Returns bounds."""
    return kv_bounds_prepared(cache, pages, bounds, stream)()


def _kv_select(q, cache, bounds, page_table, seq_lens, budget, pages_out, lens_out, ws, stream, prepared):
    ldq = _rows(q, "q", (torch.bfloat16,), None, cache.head_dim)
    batch, q_heads, head_dim = q.shape
    if page_table.dim() != 2:
        raise ValueError(f"page_table must be [batch][pages], not {tuple(page_table.shape)}")
    _check_ws(ws)
    dev = _device_of(stream, pool=cache.pool, q=q, bounds=bounds, page_table=page_table, seq_lens=seq_lens,
                     pages_out=pages_out, lens_out=lens_out, ws=ws)
    shape = (batch, cache.kv_heads, budget)
    a = KvSelectArgs(cache=ctypes.pointer(cache.desc), batch=batch, q_heads=q_heads, q=q.data_ptr(), ldq=ldq,
                     bounds=_vector(bounds, "bounds", torch.bfloat16, (cache.pages, cache.kv_heads, 2, head_dim)),
                     page_table=_vector(page_table, "page_table", torch.int32, (batch, page_table.shape[1])),
                     table_width=page_table.shape[1], seq_lens=_vector(seq_lens, "seq_lens", torch.int32, (batch,)),
                     budget=budget)
    need = ctypes.c_size_t()
    check(lib().nvfp4_kv_select_workspace_bytes(ctypes.byref(a), ctypes.byref(need)))
    if pages_out is None:
        pages_out = _new(lambda: torch.empty(shape, dtype=torch.int32, device=dev), dev, stream)
    if lens_out is None:
        lens_out = _new(lambda: torch.empty((batch,), dtype=torch.int32, device=dev), dev, stream)
    a.pages_out = _vector(pages_out, "pages_out", torch.int32, shape)
    a.lens_out = _vector(lens_out, "lens_out", torch.int32, (batch,))
    ws, captured = _workspace_of(need.value, ws, dev, stream, prepared, "select")
    if ws is not None:
        a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    call = _caller(lib().nvfp4_kv_select, (ctypes.byref(a),), dev, stream, (pages_out, lens_out),
                   (a, cache, q, bounds, page_table, seq_lens, pages_out, lens_out, ws))
    return _clearing(call, ws, NVFP4_SELECT_COUNTER_BYTES, dev, stream) if captured else call


def kv_select_prepared(q, cache, bounds, page_table, seq_lens, budget, pages_out=None, lens_out=None, ws=None, stream=None):
    """kv_select() prepared, as attn_decode_prepared() is; its .outputs are the buffers that it fills."""
    return _kv_select(q, cache, bounds, page_table, seq_lens, budget, pages_out, lens_out, ws, stream, True)


def kv_select(q, cache, bounds, page_table, seq_lens, budget, pages_out=None, lens_out=None, ws=None, stream=None):
    """The pages that each kv head's queries q (as in attn_decode()) attend to: the last one, and those of the others that
    bounds (kv_bounds()) rank highest, `budget` at most.  Returns (pages int32 [batch][kv_heads][budget], lens int32
    [batch]), a page table and lengths for attn_decode().  ws: as in attn_decode()."""
    return _kv_select(q, cache, bounds, page_table, seq_lens, budget, pages_out, lens_out, ws, stream, False)()


def _attn_weigh(q, cache, page_table, seq_lens, weights, decay, weights_out, scale, window, out, lse, ws, stream, prepared):
    if weights_out is None:
        weights_out = weights
    if weights_out is None or (weights is None and decay != 0):
        raise ValueError("without weights, decay must be 0 and weights_out given")
    shape = (q.shape[0], cache.kv_heads, page_table.shape[-1])

    def wrap(a):
        return AttnWeighArgs(attn=a, decay=decay, weights_out=_vector(weights_out, "weights_out", torch.float32, shape),
                             weights=None if weights is None else _vector(weights, "weights", torch.float32, shape))
    return _attn(q, cache, page_table, seq_lens, scale, window, out, lse, ws, stream, prepared, "nvfp4_attn_weigh", wrap,
                 weights_out, weights=weights, weights_out=weights_out)


def attn_weigh_prepared(q, cache, page_table, seq_lens, weights, decay=1.0, weights_out=None, scale=None, window=0, out=None,
                        lse=None, ws=None, stream=None):
    """attn_weigh() prepared, as attn_decode_prepared() is."""
    return _attn_weigh(q, cache, page_table, seq_lens, weights, decay, weights_out, scale, window, out, lse, ws, stream, True)


def attn_weigh(q, cache, page_table, seq_lens, weights, decay=1.0, weights_out=None, scale=None, window=0, out=None, lse=None,
               ws=None, stream=None):
    """attn_decode(), and the attention weight that its query heads give to each page added to decay * weights: float32
    [batch][kv_heads][pages], updated in place unless weights_out is given.  Returns (out, weights_out), or (out, lse,
    weights_out) with lse.  weights may be None if decay is 0."""
    return _attn_weigh(q, cache, page_table, seq_lens, weights, decay, weights_out, scale, window, out, lse, ws, stream, False)()


def kv_evict_prepared(weights, page_table, seq_lens, page_size, budget, sink=0, recent=1, table_out=None, lens_out=None,
                      freed=None, weights_out=None, stream=None):
    """kv_evict() with its arguments marshalled once: returns a zero-argument callable that returns its outputs."""
    if weights.dim() != 3:
        raise ValueError(f"weights must be [batch][kv_heads][pages], not {tuple(weights.shape)}")
    batch, kv_heads, width = weights.shape
    dev = _device_of(stream, weights=weights, page_table=page_table, seq_lens=seq_lens, table_out=table_out,
                     lens_out=lens_out, freed=freed, weights_out=weights_out)
    a = KvEvictArgs(batch=batch, kv_heads=kv_heads, page_size=page_size,
                    weights=_vector(weights, "weights", torch.float32, (batch, kv_heads, width)),
                    page_table=_vector(page_table, "page_table", torch.int32, (batch, width)), table_width=width,
                    seq_lens=_vector(seq_lens, "seq_lens", torch.int32, (batch,)), budget=budget, sink=sink, recent=recent)
    need = ctypes.c_size_t()
    check(lib().nvfp4_kv_evict_workspace_bytes(ctypes.byref(a), ctypes.byref(need)))

    def output(t, name, dtype, *shape):
        if t is None:
            t = _new(lambda: torch.empty(shape, dtype=dtype, device=dev), dev, stream)
        setattr(a, name, _vector(t, name, dtype, shape))
        return t

    outputs = (output(table_out, "table_out", torch.int32, batch, budget), output(lens_out, "lens_out", torch.int32, batch),
               output(freed, "freed", torch.int32, batch, width),
               output(weights_out, "weights_out", torch.float32, batch, kv_heads, budget))
    ws = _new(lambda: torch.empty(need.value, dtype=torch.uint8, device=dev), dev, stream) if need.value else None
    if ws is not None:
        a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel()
    return _caller(lib().nvfp4_kv_evict, (ctypes.byref(a),), dev, stream, outputs,
                   (a, weights, page_table, seq_lens, ws, *outputs))


def kv_evict(weights, page_table, seq_lens, page_size, budget, sink=0, recent=1, table_out=None, lens_out=None, freed=None,
             weights_out=None, stream=None):
    """Keeps up to `budget` pages of each sequence: the last `recent`, the first `sink`, and the others by their weights
    (attn_weigh()) over all kv heads.  Returns (table_out int32 [batch][budget], lens_out int32 [batch], freed int32
    [batch][pages], weights_out float32 [batch][kv_heads][budget]): the kept pages in order with the lengths and weights
    that go with them, and the pages dropped; -1 and 0 behind them."""
    return kv_evict_prepared(weights, page_table, seq_lens, page_size, budget, sink, recent, table_out, lens_out, freed,
                             weights_out, stream)()
