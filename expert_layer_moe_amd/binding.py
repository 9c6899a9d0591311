"""ctypes binding of libmoe_amd.so: argument marshalling only.

Every step of the layer runs in the library's HIP kernels; this module only
checks tensor shapes / dtypes / devices and passes raw device pointers and the
current HIP stream.  PyTorch provides device memory and streams.  The calls of
the 4-bit operators and the norm do the same in compiled code (csrc/calls.cpp).
There is no fallback: if the library is missing, loading raises; if the compiled
calls for this interpreter and torch are, the first such call does.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
from typing import Optional

import torch

from .build import calls_path

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libmoe_amd.so")
CALLS_PATH = calls_path()

MOE_F32, MOE_BF16, MOE_FP8_E4M3 = 0, 1, 2
MOE_LAYOUT_ROW_MAJOR, MOE_LAYOUT_FRAG16 = 0, 1
_STATUS = {0: "MOE_OK", -1: "MOE_ERR_INVALID_ARG", -2: "MOE_ERR_UNSUPPORTED",
           -3: "MOE_ERR_WORKSPACE", -4: "MOE_ERR_HIP"}

EXPORTS = ["moe_workspace_size", "moe_route", "moe_align", "moe_forward",
           "moe_forward_few", "moe_few_workspace_size", "moe_gemm_fp8",
           "moe_gemm_fp8_kernel", "moe_quant_fp8", "moe_silu_mul_quant_fp8",
           "moe_quant_mxfp4", "moe_silu_mul_quant_mxfp4", "moe_dequant_mxfp4", "moe_gemm_mxfp4",
           "moe_gemm_mxfp4_kernel",
           "moe_add_rms_norm", "moe_add_rms_norm_quant_fp8",
           "moe_forward_noalloc", "moe_forward_signaled", "moe_block_signal_count", "moe_set_signal_wait_us", "moe_set_one_launch",
           "moe_pack_weights", "moe_set_path_thresholds", "moe_set_fp8_mfma", "moe_status_str", "moe_num_stages", "moe_stage_name",
           "moe_profile_enable", "moe_profile_read"]


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_STATUS.get(status, status)}: {msg}")
        self.status = status


class moe_desc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("E", ctypes.c_int32),
                ("n_shared", ctypes.c_int32), ("I", ctypes.c_int32),
                ("act_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32),
                ("w13_scale", ctypes.c_void_p), ("w2_scale", ctypes.c_void_p),
                ("block_m", ctypes.c_int32), ("w_layout", ctypes.c_int32)]


class moe_gemm_desc(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("lda", ctypes.c_int64), ("ldb", ctypes.c_int64),
                ("ld_as", ctypes.c_int64), ("ldo", ctypes.c_int64)]


class moe_quant_desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("cols", ctypes.c_int32),
                ("in_dtype", ctypes.c_int32), ("ld_in", ctypes.c_int64),
                ("ld_codes", ctypes.c_int64), ("ld_scales", ctypes.c_int64)]


class moe_mx_gemm_desc(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("lda", ctypes.c_int64), ("ldb", ctypes.c_int64),
                ("ld_as", ctypes.c_int64), ("ld_bs", ctypes.c_int64), ("ldo", ctypes.c_int64)]


class moe_norm_desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("res_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("eps", ctypes.c_float), ("ld_x", ctypes.c_int64),
                ("ld_res", ctypes.c_int64), ("ld_res_out", ctypes.c_int64),
                ("ld_out", ctypes.c_int64), ("ld_codes", ctypes.c_int64),
                ("ld_scales", ctypes.c_int64)]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmoe_amd.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build() "
                           "(the MoE layer has no fallback path)")
    lib = ctypes.CDLL(path)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    D = ctypes.POINTER(moe_desc)
    lib.moe_workspace_size.argtypes = [D, I32]
    lib.moe_workspace_size.restype = SZ
    lib.moe_route.argtypes = [D, P, P, P, I32, P, P, P, P, SZ, P]
    lib.moe_route.restype = ctypes.c_int
    lib.moe_align.argtypes = [D, P, I32, I32, P, P, P, P, P, SZ, P]
    lib.moe_align.restype = ctypes.c_int
    lib.moe_forward.argtypes = [D, P, P, P, P, P, I32, P, P, SZ, P]
    lib.moe_forward.restype = ctypes.c_int
    lib.moe_forward_noalloc.argtypes = [D, P, P, P, P, P, I32, P, P]
    lib.moe_forward_noalloc.restype = ctypes.c_int
    lib.moe_forward_signaled.argtypes = [D, P, P, P, P, P, I32, P, P, SZ, P, P, P]
    lib.moe_forward_signaled.restype = ctypes.c_int
    lib.moe_block_signal_count.argtypes = [D]
    lib.moe_block_signal_count.restype = SZ
    lib.moe_set_signal_wait_us.argtypes = [I32]
    lib.moe_set_signal_wait_us.restype = ctypes.c_int
    lib.moe_set_one_launch.argtypes = [I32]
    lib.moe_set_one_launch.restype = ctypes.c_int
    lib.moe_few_workspace_size.argtypes = [D, I32]
    lib.moe_few_workspace_size.restype = SZ
    lib.moe_forward_few.argtypes = [D, P, P, P, P, P, I32, P, P, SZ, P]
    lib.moe_forward_few.restype = ctypes.c_int
    lib.moe_gemm_fp8.argtypes = [ctypes.POINTER(moe_gemm_desc), P, P, P, P, P, P]
    lib.moe_gemm_fp8.restype = ctypes.c_int
    lib.moe_gemm_fp8_kernel.argtypes = [ctypes.POINTER(moe_gemm_desc)]
    lib.moe_gemm_fp8_kernel.restype = ctypes.c_char_p
    for name in ("moe_quant_fp8", "moe_silu_mul_quant_fp8", "moe_quant_mxfp4",
                 "moe_silu_mul_quant_mxfp4", "moe_dequant_mxfp4"):
        getattr(lib, name).argtypes = [ctypes.POINTER(moe_quant_desc), P, P, P, P]
        getattr(lib, name).restype = ctypes.c_int
    lib.moe_gemm_mxfp4.argtypes = [ctypes.POINTER(moe_mx_gemm_desc), P, P, P, P, P, P]
    lib.moe_gemm_mxfp4.restype = ctypes.c_int
    lib.moe_gemm_mxfp4_kernel.argtypes = [ctypes.POINTER(moe_mx_gemm_desc)]
    lib.moe_gemm_mxfp4_kernel.restype = ctypes.c_char_p
    lib.moe_add_rms_norm.argtypes = [ctypes.POINTER(moe_norm_desc), P, P, P, P, P, P]
    lib.moe_add_rms_norm.restype = ctypes.c_int
    lib.moe_add_rms_norm_quant_fp8.argtypes = [ctypes.POINTER(moe_norm_desc)] + [P] * 8
    lib.moe_add_rms_norm_quant_fp8.restype = ctypes.c_int
    lib.moe_pack_weights.argtypes = [D, P, P, P, P, P]
    lib.moe_pack_weights.restype = ctypes.c_int
    lib.moe_set_fp8_mfma.argtypes = [I32]
    lib.moe_set_fp8_mfma.restype = ctypes.c_int
    lib.moe_set_path_thresholds.argtypes = [I32, I32]
    lib.moe_set_path_thresholds.restype = ctypes.c_int
    lib.moe_status_str.argtypes = [ctypes.c_int]
    lib.moe_status_str.restype = ctypes.c_char_p
    lib.moe_num_stages.argtypes = []
    lib.moe_num_stages.restype = ctypes.c_int
    lib.moe_stage_name.argtypes = [ctypes.c_int]
    lib.moe_stage_name.restype = ctypes.c_char_p
    lib.moe_profile_enable.argtypes = [ctypes.c_int]
    lib.moe_profile_enable.restype = ctypes.c_int
    lib.moe_profile_read.argtypes = [ctypes.POINTER(ctypes.c_double),
                                     ctypes.POINTER(ctypes.c_int32), I32]
    lib.moe_profile_read.restype = ctypes.c_int
    _lib = lib
    return lib


_calls = None


def _load_calls():
    """The compiled calls, with this library's entry points."""
    global _calls
    lib = load_library()
    if not os.path.exists(CALLS_PATH):
        raise RuntimeError(f"{CALLS_PATH} is missing: build it with __graft_entry__.build(), with this "
                           "interpreter and torch")
    loader = importlib.machinery.ExtensionFileLoader("_moe_calls", CALLS_PATH)
    calls = importlib.util.module_from_spec(
        importlib.util.spec_from_file_location("_moe_calls", CALLS_PATH, loader=loader))
    loader.exec_module(calls)
    entries = (lib.moe_quant_mxfp4, lib.moe_silu_mul_quant_mxfp4, lib.moe_dequant_mxfp4,
               lib.moe_gemm_mxfp4, lib.moe_add_rms_norm, lib.moe_add_rms_norm_quant_fp8)
    calls.bind(*(ctypes.cast(e, ctypes.c_void_p).value for e in entries),
               torch._C._cuda_getCurrentRawStream, _empty, _check)
    _calls = calls
    return calls


def _check(status: int):
    if status != 0:
        raise MoeError(status, load_library().moe_status_str(status).decode())


_DT = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.uint8: MOE_FP8_E4M3}


def make_desc(T, H, E, I, n_shared=0, act_dtype=MOE_BF16, w_dtype=MOE_BF16,
              w13_scale: Optional[torch.Tensor] = None,
              w2_scale: Optional[torch.Tensor] = None, block_m=0,
              w_layout=MOE_LAYOUT_ROW_MAJOR) -> moe_desc:
    return moe_desc(T, H, E, n_shared, I, act_dtype, w_dtype,
                    _ptr(w13_scale), _ptr(w2_scale), block_m, w_layout)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _dev(t: Optional[torch.Tensor], name: str, dtype=None, shape=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _act(desc):
    return torch.float32 if desc.act_dtype == MOE_F32 else torch.bfloat16


def _w(desc):
    return {MOE_F32: torch.float32, MOE_BF16: torch.bfloat16,
            MOE_FP8_E4M3: torch.uint8}[desc.w_dtype]


def moe_workspace_size(desc: moe_desc, topk: int) -> int:
    return int(load_library().moe_workspace_size(ctypes.byref(desc), topk))


def alloc_workspace(desc: moe_desc, topk: int, device="cuda") -> torch.Tensor:
    n = moe_workspace_size(desc, topk)
    if n == 0:
        raise MoeError(-1, "invalid descriptor")
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_route(desc, x, valid_rows, router_w, topk, topk_ids, topk_w, logits=None,
              workspace=None, stream=None):
    T, H, E = desc.T, desc.H, desc.E
    ws = workspace if workspace is not None else alloc_workspace(desc, topk, x.device)
    _check(load_library().moe_route(
        ctypes.byref(desc), _dev(x, "x", _act(desc), (T, H)),
        _dev(valid_rows, "valid_rows", torch.uint8, (T,)),
        _dev(router_w, "router_w", _act(desc), (E, H)), topk,
        _dev(topk_ids, "topk_ids", torch.int32, (T, topk)),
        _dev(topk_w, "topk_w", torch.float32, (T, topk)),
        _dev(logits, "logits", torch.float32, (T, E)),
        _dev(ws, "workspace", torch.uint8), ws.numel(), _stream(stream)))
    return ws


def moe_align(desc, topk_ids, topk, block_m, sorted_ids, block_expert,
              expert_offsets, n_post_padded, workspace=None, stream=None):
    T, E, ns = desc.T, desc.E, desc.n_shared
    cap = T * (topk + ns) + (E + ns) * (block_m - 1)
    if sorted_ids.numel() < cap or block_expert.numel() < (cap + block_m - 1) // block_m:
        raise ValueError("sorted_ids / block_expert below the documented capacity")
    if expert_offsets.numel() < E + ns + 1:
        raise ValueError("expert_offsets holds E + n_shared + 1 entries")
    _check(load_library().moe_align(
        ctypes.byref(desc), _dev(topk_ids, "topk_ids", torch.int32, (T, topk)), topk,
        block_m, _dev(sorted_ids, "sorted_ids", torch.int32),
        _dev(block_expert, "block_expert", torch.int32),
        _dev(expert_offsets, "expert_offsets", torch.int32),
        _dev(n_post_padded, "n_post_padded", torch.int32, (1,)),
        _dev(workspace, "workspace", torch.uint8),
        0 if workspace is None else workspace.numel(), _stream(stream)))


def moe_forward(desc, x, valid_rows, router_w, w13, w2, topk, out, workspace,
                stream=None):
    T, H, E, I, ns = desc.T, desc.H, desc.E, desc.I, desc.n_shared
    _check(load_library().moe_forward(
        ctypes.byref(desc), _dev(x, "x", _act(desc), (T, H)),
        _dev(valid_rows, "valid_rows", torch.uint8, (T,)),
        _dev(router_w, "router_w", _act(desc), (E, H)),
        _dev(w13, "w13", _w(desc), (E + ns, 2 * I, H)),
        _dev(w2, "w2", _w(desc), (E + ns, H, I)), topk,
        _dev(out, "out", _act(desc), (T, H)),
        _dev(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream)))


def moe_forward_noalloc(desc, x, valid_rows, router_w, w13, w2, topk, out, stream=None):
    """moe_forward in the library's fixed device scratch (no workspace)."""
    T, H, E, I, ns = desc.T, desc.H, desc.E, desc.I, desc.n_shared
    _check(load_library().moe_forward_noalloc(
        ctypes.byref(desc), _dev(x, "x", _act(desc), (T, H)),
        _dev(valid_rows, "valid_rows", torch.uint8, (T,)),
        _dev(router_w, "router_w", _act(desc), (E, H)),
        _dev(w13, "w13", _w(desc), (E + ns, 2 * I, H)),
        _dev(w2, "w2", _w(desc), (E + ns, H, I)), topk,
        _dev(out, "out", _act(desc), (T, H)), _stream(stream)))


def moe_block_signal_count(desc: moe_desc) -> int:
    """Entries of moe_forward_signaled's completion counters."""
    return int(load_library().moe_block_signal_count(ctypes.byref(desc)))


def moe_forward_signaled(desc, x, valid_rows, router_w, w13, w2, topk, out, workspace,
                         block_signal, stream=None, consumer_stream=None):
    """moe_forward with per-(expert, 64-row block) completion counters
    (block_signal, int32 [E + n_shared, ceil(T / 64)]) and the combine waiting
    on them on consumer_stream (None: the current stream, like `stream`)."""
    T, H, E, I, ns = desc.T, desc.H, desc.E, desc.I, desc.n_shared
    _check(load_library().moe_forward_signaled(
        ctypes.byref(desc), _dev(x, "x", _act(desc), (T, H)),
        _dev(valid_rows, "valid_rows", torch.uint8, (T,)),
        _dev(router_w, "router_w", _act(desc), (E, H)),
        _dev(w13, "w13", _w(desc), (E + ns, 2 * I, H)),
        _dev(w2, "w2", _w(desc), (E + ns, H, I)), topk,
        _dev(out, "out", _act(desc), (T, H)),
        _dev(workspace, "workspace", torch.uint8), workspace.numel(),
        _dev(block_signal, "block_signal", torch.int32, (E + ns, (T + 63) // 64)),
        _stream(stream), _stream(consumer_stream)))


def moe_set_signal_wait_us(us: int = 10000):
    """Time bound of each wait of the signaled combine (process-wide)."""
    _check(load_library().moe_set_signal_wait_us(us))


def moe_set_one_launch(enable: bool = False):
    """Calls where every segment streams: gate/up and down in one launch
    (True) or two (False, the default).  Process-wide."""
    _check(load_library().moe_set_one_launch(1 if enable else 0))


# ---- few token rows, fp8 block-scale product, token quantisation -----------------
FEW_MAX_ROWS = 16   # MOE_FEW_MAX_ROWS


def _device_of(*tensors) -> int:
    """The GPU that all the tensors (None: absent) are on."""
    device = -1
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d < 0:
                raise ValueError("tensors must be on the GPU")
            if device >= 0 and d != device:
                raise ValueError(f"tensors on cuda:{device} and cuda:{d}: one GPU expected")
            device = d
    return device


def _enqueue(entry, device: int, stream, *args):
    """Calls a library entry point with that GPU current, on the given stream
    or its current one."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(device)
    else:
        if stream.device_index != device:
            raise ValueError(f"stream on {stream.device}, tensors on cuda:{device}")
        raw = stream.cuda_stream
    if device == torch._C._cuda_getDevice():
        status = entry(*args, raw)
    else:
        with torch.cuda.device(device):
            status = entry(*args, raw)
    if status:
        _check(status)


def _empty(shape, dtype, device, stream):
    """A new tensor [rows, columns] for a result written on `stream` (its
    memory is reused in that stream's order)."""
    if stream is None:
        return torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _row_stride(t: torch.Tensor, name: str, dtypes, rows: int, cols: int) -> int:
    """Row stride of a rows x cols matrix with contiguous rows (0: dense, or one
    row, whose stride says nothing)."""
    if t.dtype not in dtypes or t.shape != (rows, cols):
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)}, expected "
                         f"{' or '.join(map(str, dtypes))} ({rows}, {cols})")
    if t.is_contiguous():
        return 0
    row, col = t.stride()
    if col != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous rows")
    if rows == 1:
        return 0
    if row < cols:
        raise ValueError(f"{name} has rows that overlap (stride {row})")
    return row


def _sizes(*sizes):
    """The descriptors hold 32 bits, and ctypes would keep the low ones of more."""
    if max(sizes) > 0x7fffffff:
        raise ValueError(f"sizes {sizes}: less than 2^31 expected")


_CODES = (torch.uint8, torch.float8_e4m3fn)
_F32 = (torch.float32,)
_FLOATS = (torch.float32, torch.bfloat16)


def moe_few_workspace_size(desc: moe_desc, topk: int) -> int:
    return int(load_library().moe_few_workspace_size(ctypes.byref(desc), topk))


def alloc_few_workspace(desc: moe_desc, topk: int, device="cuda") -> torch.Tensor:
    n = moe_few_workspace_size(desc, topk)
    if n == 0:
        raise MoeError(-2, "not a layer of a few rows (bf16 activations, 1 to "
                           f"{FEW_MAX_ROWS} rows, a hidden size of 128 n)")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _dense(t, name: str, dtype, *shape):
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)}, expected contiguous {dtype} {shape}")


def moe_forward_few(desc, x, valid_rows, router_w, w13, w2, topk, out, workspace,
                    stream=None):
    """moe_forward for at most FEW_MAX_ROWS token rows, in two or three
    launches."""
    T, H, E, I, ne = desc.T, desc.H, desc.E, desc.I, desc.E + desc.n_shared
    act, w = _act(desc), _w(desc)
    _dense(x, "x", act, T, H)
    _dense(out, "out", act, T, H)
    _dense(router_w, "router_w", act, E, H)
    _dense(w13, "w13", w, ne, 2 * I, H)
    _dense(w2, "w2", w, ne, H, I)
    valid = None
    if valid_rows is not None:
        _dense(valid_rows, "valid_rows", torch.uint8, T)
        valid = valid_rows.data_ptr()
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace: contiguous torch.uint8 expected")
    _enqueue(load_library().moe_forward_few,
             _device_of(router_w, w13, w2, x, valid_rows, out, workspace), stream,
             ctypes.byref(desc), x.data_ptr(), valid, router_w.data_ptr(), w13.data_ptr(),
             w2.data_ptr(), topk, out.data_ptr(), workspace.data_ptr(), workspace.numel())


def moe_gemm_fp8(a, a_scale, b, b_scale, out=None, out_dtype=torch.bfloat16, stream=None):
    """out [M, N] = (a * a_scale) (b * b_scale)^T of e4m3fn codes (uint8 or
    float8_e4m3fn) a [M, K], b [N, K]; a_scale [M, ceil(K/128)], b_scale
    [ceil(N/128), ceil(K/128)] fp32.  a, b, a_scale and out may have wider
    rows (row strides); out is allocated here when not given."""
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError("a and b are matrices")
    M, K = a.shape
    N = b.shape[0]
    _sizes(M, N, K)
    nb = (K + 127) // 128
    lda = _row_stride(a, "a", _CODES, M, K)
    ldb = _row_stride(b, "b", _CODES, N, K)
    ld_as = _row_stride(a_scale, "a_scale", _F32, M, nb)
    if _row_stride(b_scale, "b_scale", _F32, (N + 127) // 128, nb) not in (0, nb):
        raise ValueError("b_scale must be contiguous")
    if out is None:
        if out_dtype not in _FLOATS:
            raise ValueError(f"out_dtype {out_dtype}: float32 or bfloat16 expected")
        out, ldo = _empty((M, N), out_dtype, a.device, stream), 0
    else:
        ldo = _row_stride(out, "out", _FLOATS, M, N)
    _enqueue(load_library().moe_gemm_fp8, _device_of(a, a_scale, b, b_scale, out), stream,
             moe_gemm_desc(M, N, K, _DT[out.dtype], lda, ldb, ld_as, ldo), a.data_ptr(),
             a_scale.data_ptr(), b.data_ptr(), b_scale.data_ptr(), out.data_ptr())
    return out


def moe_gemm_fp8_kernel(M: int, N: int, K: int, out_dtype=torch.bfloat16) -> str:
    """The kernel that moe_gemm_fp8 takes for these sizes ("rows 16", "tile 64 x
    32", ...)."""
    _sizes(M, N, K)
    if out_dtype not in _FLOATS:
        raise ValueError(f"out_dtype {out_dtype}: float32 or bfloat16 expected")
    name = load_library().moe_gemm_fp8_kernel(
        ctypes.byref(moe_gemm_desc(M, N, K, _DT[out_dtype], 0, 0, 0, 0)))
    if name is None:
        raise MoeError(-2, "sizes that moe_gemm_fp8 does not take")
    return name.decode()


def _quant(entry, x, per_col, codes, scales, stream):
    if x.dim() != 2:
        raise ValueError(f"a matrix expected, not {tuple(x.shape)}")
    M, n = x.shape
    if n % per_col != 0:
        raise ValueError(f"a matrix of {per_col} n columns expected, not {tuple(x.shape)}")
    cols = n // per_col
    _sizes(M, cols)
    nb = (cols + 127) // 128
    ld_in = _row_stride(x, "input", _FLOATS, M, n)
    given = codes, scales
    ld_codes = ld_scales = 0
    if codes is None:
        codes = _empty((M, cols), torch.uint8, x.device, stream)
    else:
        ld_codes = _row_stride(codes, "codes", _CODES, M, cols)
    if scales is None:
        scales = _empty((M, nb), torch.float32, x.device, stream)
    else:
        ld_scales = _row_stride(scales, "scales", _F32, M, nb)
    _enqueue(entry, _device_of(x, *given), stream,
             moe_quant_desc(M, cols, _DT[x.dtype], ld_in, ld_codes, ld_scales), x.data_ptr(),
             codes.data_ptr(), scales.data_ptr())
    return codes, scales


def moe_quant_fp8(x, codes=None, scales=None, stream=None):
    """Token rows x [M, K] (bf16 or fp32; rows may be strided) -> e4m3fn codes
    [M, K] (uint8) and fp32 scales [M, ceil(K/128)], allocated here when not
    given.  Returns (codes, scales)."""
    return _quant(load_library().moe_quant_fp8, x, 1, codes, scales, stream)


def moe_silu_mul_quant_fp8(gu, codes=None, scales=None, stream=None):
    """moe_quant_fp8 of SiLU(g) * u for gu [M, 2 I] (gate columns, then up)."""
    return _quant(load_library().moe_silu_mul_quant_fp8, gu, 2, codes, scales, stream)


# ---- 4-bit microscaled floats ---------------------------------------------------
# (Results that a call of these or of the norm allocates lie in one allocation if they
# take up to 1 MB together, which is free when the last of them is: each is a tensor of its
# own that may be kept, resized or used on other streams.  But a file of one holds the bytes
# ahead of it too, torch.save takes several of different types only as clones (their
# storages begin at one address), and one that torch hands to another process keeps the
# allocation for good.  A call with a `stream` allocates each by itself.)
def moe_quant_mxfp4(x, codes=None, scales=None, stream=None):
    """Token or weight rows x [M, K] (bf16 or fp32; rows may be strided; K a
    multiple of 32) -> e2m1 codes [M, K/2] (uint8, two to a byte, the first in
    the low half) and e8m0 scale codes [M, K/32] (uint8 or, if given,
    float8_e8m0fnu), allocated here when not given.  Returns (codes, scales)."""
    return (_calls or _load_calls()).quant_mxfp4(x, codes, scales, stream)


def moe_silu_mul_quant_mxfp4(gu, codes=None, scales=None, stream=None):
    """moe_quant_mxfp4 of SiLU(g) * u for gu [M, 2 I] (gate columns, then up)."""
    return (_calls or _load_calls()).silu_mul_quant_mxfp4(gu, codes, scales, stream)


def moe_dequant_mxfp4(codes, scales, out=None, out_dtype=torch.bfloat16, stream=None):
    """The values [M, K] (bf16 or fp32, exact) of e2m1 codes [M, K/2] under e8m0
    scale codes [M, K/32]; out is allocated here when not given."""
    return (_calls or _load_calls()).dequant_mxfp4(codes, scales, out, out_dtype, stream)


def moe_gemm_mxfp4(a, a_scale, b, b_scale, out=None, out_dtype=torch.bfloat16, stream=None):
    """out [M, N] = a b^T of e2m1 codes a [M, K/2], b [N, K/2] (uint8, two to a
    byte) under e8m0 scale codes a_scale [M, K/32], b_scale [N, K/32] (uint8 or
    float8_e8m0fnu).  All may have wider rows (row strides); out is allocated
    here when not given."""
    return (_calls or _load_calls()).gemm_mxfp4(a, a_scale, b, b_scale, out, out_dtype, stream)


def moe_gemm_mxfp4_kernel(M: int, N: int, K: int) -> str:
    """The kernel that moe_gemm_mxfp4 takes for these sizes ("rows 16", "tile 64 x
    128", ...)."""
    _sizes(M, N, K)
    name = load_library().moe_gemm_mxfp4_kernel(
        ctypes.byref(moe_mx_gemm_desc(M, N, K, _DT[torch.bfloat16], 0, 0, 0, 0, 0)))
    if name is None:
        raise MoeError(-2, "sizes that moe_gemm_mxfp4 does not take")
    return name.decode()


# ---- root-mean-square norm with the residual's addition ---------------------------
def moe_add_rms_norm(x, residual, weight, eps=1e-6, out=None, residual_out=None,
                     out_dtype=torch.bfloat16, stream=None):
    """r = x + residual (as stored in residual_out, of residual's type), out =
    r / sqrt(mean(r^2) + eps) * weight, for rows x, residual [M, H] (bf16 or
    fp32, H a multiple of 16) and weight [H].  residual None: r = x.
    residual_out may be residual, out may be x; both are allocated here when not
    given.  Returns (out, residual_out), the latter None without a residual."""
    return (_calls or _load_calls()).add_rms_norm(x, residual, weight, eps, out, residual_out,
                                                  out_dtype, stream)


def moe_add_rms_norm_quant_fp8(x, residual, weight, eps=1e-6, codes=None, scales=None,
                               residual_out=None, out=None, stream=None):
    """moe_add_rms_norm's result in moe_quant_fp8's codes [M, H] (uint8) and
    scales [M, ceil(H/128)], of its fp32 values; these themselves go to `out`
    (bf16 or fp32) only if it is given.  Returns (codes, scales, residual_out)."""
    return (_calls or _load_calls()).add_rms_norm_quant_fp8(
        x, residual, weight, eps, codes, scales, residual_out, out, stream)


SCRATCH_BYTES = 64 << 20   # MOE_SCRATCH_BYTES


def moe_pack_weights(desc, w13, w2, w13_packed=None, w2_packed=None, stream=None):
    """Row-major w13 / w2 -> the MFMA fragment layout (MOE_LAYOUT_FRAG16).
    Returns the packed tensors (allocated here when not given)."""
    ne, H, I = desc.E + desc.n_shared, desc.H, desc.I
    w13_packed = torch.empty_like(w13) if w13_packed is None else w13_packed
    w2_packed = torch.empty_like(w2) if w2_packed is None else w2_packed
    wd = _w(desc)
    _check(load_library().moe_pack_weights(
        ctypes.byref(desc), _dev(w13, "w13", wd, (ne, 2 * I, H)),
        _dev(w2, "w2", wd, (ne, H, I)),
        _dev(w13_packed, "w13_packed", wd, (ne, 2 * I, H)),
        _dev(w2_packed, "w2_packed", wd, (ne, H, I)), _stream(stream)))
    return w13_packed, w2_packed


def moe_set_path_thresholds(gemm_min_rows: int = 128, gemm_min_tiles: int = -1):
    """Segments above gemm_min_rows rows use the tiled GEMM kernels once their
    tiles number gemm_min_tiles (-1 = fill the chip).  Process-wide."""
    _check(load_library().moe_set_path_thresholds(gemm_min_rows, gemm_min_tiles))


def moe_set_fp8_mfma(enable: bool = False):
    """fp8 weights on the tiled gate/up GEMM: fp8 MFMA on two-term token
    codes (True) or bf16 MFMA on dequantised weights (False, the default).
    Process-wide; size workspaces after choosing."""
    _check(load_library().moe_set_fp8_mfma(1 if enable else 0))


def moe_status_str(status: int) -> str:
    return load_library().moe_status_str(status).decode()


# ---- measurement hooks -------------------------------------------------------
def stage_names():
    lib = load_library()
    return [lib.moe_stage_name(i).decode() for i in range(lib.moe_num_stages())]


def moe_profile_enable(stages=None):
    """Time the named stages (None or [] = off, "all" = every stage)."""
    if stages == "all":
        mask = -1
    else:
        names = stage_names()
        mask = 0
        for s in stages or []:
            mask |= 1 << names.index(s)
    _check(load_library().moe_profile_enable(mask))


def moe_profile_read():
    lib = load_library()
    n = lib.moe_num_stages()
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int32 * n)()
    _check(lib.moe_profile_read(ms, cnt, n))
    return {name: (ms[i], cnt[i]) for i, name in enumerate(stage_names())}
