"""Python binding of libtq (ternary-weight GEMV/GEMM for AMD gfx950).

Argument marshalling only: every step of the computation runs in libtq's HIP
kernels (or, for packing, in its host C++ code).  PyTorch supplies device
memory and streams.  The functions carry the C ABI's names (see
include/tq.h); device tensors must be contiguous, on the GPU and 16-byte
aligned.  If libtq.so is missing the import fails loudly -- there is no
fallback.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtq.so")

TQ_FMT_B3 = 0
TQ_FMT_2B = 1
TQ_FMT_BP = 2
TQ_FMT_B3R = 3  # B3 bytes in row-major group order (the layout without the re-tiling)
TQ_F16 = 0
TQ_F32 = 1
TQ_STREAM_READ_WGS = 8192
TQ_ROPE_HALVES = 0  # rotated pairs: element i with i + rot / 2
TQ_ROPE_PAIRS = 1   # ... 2i with 2i + 1
GROUP = 128
KV_PAGE = 64
GEMV_MAX_M = 16
STACK_MAX_ROWS = 4

_STATUS = {0: "TQ_OK", -1: "TQ_ERR_NULL", -2: "TQ_ERR_SHAPE", -3: "TQ_ERR_ALIGN",
           -4: "TQ_ERR_VALUE", -5: "TQ_ERR_FORMAT", -6: "TQ_ERR_DTYPE", -7: "TQ_ERR_SIZE",
           -8: "TQ_ERR_HIP"}

EXPORTS = ("tq_status_str", "tq_packed_bytes", "tq_pack", "tq_unpack", "tq_quant_act",
           "tq_gemv_workspace_bytes", "tq_gemv", "tq_gemv_gate_up_swiglu",
           "tq_gemm_workspace_bytes", "tq_gemm", "tq_debug_unpack", "tq_debug_group_sums",
           "tq_gemv_quant_workspace_bytes", "tq_gemv_quant",
           "tq_decode_stack_workspace_bytes", "tq_decode_stack", "tq_hadamard_quant_act",
           "tq_ternarize", "tq_debug_stream_read", "tq_debug_gate_up_sums",
           "tq_debug_gemv_quant_sums", "tq_decode_stack_persistent",
           "tq_gemv_noalloc", "tq_noalloc_scratch_bytes",
           "tq_decode_stack_batch_workspace_bytes", "tq_decode_stack_batch",
           "tq_debug_gemv_quant_rows_sums", "tq_workspace_clear", "tq_workspace_check",
           "tq_rope_table", "tq_kv_append", "tq_kv_attn_workspace_bytes", "tq_kv_attn",
           "tq_residual_norm", "tq_debug_kv_read")


class TqLayer(ctypes.Structure):
    """Packed weights of one layer (device addresses), as tq_layer in tq.h."""
    _fields_ = [("qkv", ctypes.c_void_p), ("o", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("up", ctypes.c_void_p), ("down", ctypes.c_void_p)]


class TQError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {_STATUS.get(status, status)} ({status})")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libtq.so not built ({LIB_PATH}); run ternary_weight_base_amd/build.py")
    L = ctypes.CDLL(LIB_PATH)
    P, I64, SZ, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    F, F64 = ctypes.c_float, ctypes.c_double
    sig = {
        "tq_status_str": ([I], ctypes.c_char_p),
        "tq_packed_bytes": ([I, I64, I64], SZ),
        "tq_pack": ([I, I64, I64, P, P, P, SZ], I),
        "tq_unpack": ([I, I64, I64, P, SZ, P, P], I),
        "tq_quant_act": ([I, I64, I64, P, P, P, P], I),
        "tq_gemv_workspace_bytes": ([I, I64, I64, I64], SZ),
        "tq_gemv": ([I, I64, I64, I64, P, P, P, P, P, SZ, P], I),
        "tq_gemv_gate_up_swiglu": ([I, I64, I64, I64, P, P, P, P, P, P, SZ, P], I),
        "tq_gemm_workspace_bytes": ([I, I64, I64, I64], SZ),
        "tq_gemm": ([I, I64, I64, I64, P, P, P, P, P, SZ, P], I),
        "tq_debug_unpack": ([I, I64, I64, P, P, P], I),
        "tq_debug_group_sums": ([I, I64, I64, I64, P, P, P, I, P], I),
        "tq_gemv_quant_workspace_bytes": ([I, I64, I64, I], SZ),
        "tq_gemv_quant": ([I, I64, I64, P, P, I, P, P, I64, P, P, P, P, SZ, P], I),
        "tq_decode_stack_workspace_bytes": ([I, I64, I64, I64, I64, I64], SZ),
        "tq_decode_stack": ([I, I64, I64, I64, I64, I64, P, P, P, P, P, P, P, P, P, SZ, P], I),
        "tq_decode_stack_persistent": ([I, I64, I64, I64, I64, I64, P, P, P, P, P, P, P, P, P, SZ, P], I),
        "tq_decode_stack_batch_workspace_bytes": ([I, I64, I64, I64, I64, I64, I64], SZ),
        "tq_debug_gemv_quant_rows_sums": ([I, I64, I64, I64, P, P, I, P, P, I64, P, P, P], I),
        "tq_decode_stack_batch": ([I, I64, I64, I64, I64, I64, I64, P, P, P, P, P, P, P, P, P, SZ, P], I),
        "tq_gemv_noalloc": ([I, I64, I64, I64, P, P, P, P, P], I),
        "tq_noalloc_scratch_bytes": ([], SZ),
        "tq_hadamard_quant_act": ([I, I64, I64, P, P, P, P, P], I),
        "tq_ternarize": ([I64, I64, P, P, P], I),
        "tq_debug_stream_read": ([P, SZ, P, I64, P], I),
        "tq_debug_gate_up_sums": ([I, I64, I64, I64, P, P, P, P, P], I),
        "tq_debug_gemv_quant_sums": ([I, I64, I64, P, P, I, P, P, I64, P, P, P], I),
        "tq_workspace_clear": ([P, SZ, P], I),
        "tq_workspace_check": ([P, SZ, P, P], I),
        "tq_rope_table": ([I64, I64, F64, P], I),
        "tq_kv_append": ([I, I64, I64, I64, I64, I64, P, I64, P, I64, I64, I, P, P, P, I64, P, P, P, P, I64, P,
                          P], I),
        "tq_kv_attn_workspace_bytes": ([I64, I64, I64, I64, I64, I64], SZ),
        "tq_kv_attn": ([I64, I64, I64, I64, I64, P, I64, P, P, P, I64, P, P, P, P, I64, I64, F, I64, I64, P, I64,
                        P, SZ, P], I),
        "tq_residual_norm": ([I, I, I, I64, I64, P, P, P, I64, F64, P, P, P, F64, P, P, P, P], I),
        "tq_debug_kv_read": ([I, I64, I64, I64, P, P, P, P, P, I64, P, P], I),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    return L


lib = _load()


def _check(rc: int, what: str):
    if rc != 0:
        raise TQError(rc, what)


def _ptr(t) -> int:
    """Device address of a torch tensor (or None -> NULL)."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch
    return torch.cuda.current_stream().cuda_stream


def tq_status_str(status: int) -> str:
    return lib.tq_status_str(status).decode()


# ---- host: packed format ------------------------------------------------

def tq_packed_bytes(fmt: int, N: int, K: int) -> int:
    return int(lib.tq_packed_bytes(fmt, N, K))


def tq_pack(fmt: int, trits: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """trits int8 [N][K], scales fp16 bits uint16 [N][K/128] -> packed uint8 blob (host)."""
    t = np.ascontiguousarray(trits, dtype=np.int8)
    s = np.ascontiguousarray(scales, dtype=np.uint16)
    N, K = t.shape
    nbytes = tq_packed_bytes(fmt, N, K)
    out = np.empty(max(nbytes, 1), dtype=np.uint8)
    _check(lib.tq_pack(fmt, N, K, t.ctypes.data, s.ctypes.data, out.ctypes.data, nbytes),
           "tq_pack")
    return out


def tq_ternarize(w: np.ndarray):
    """fp32 weights [N][K] (host) -> (trits int8 [N][K], fp16 scale bits uint16 [N][K/128])."""
    w = np.ascontiguousarray(w, dtype=np.float32)
    N, K = w.shape
    t = np.empty((N, K), dtype=np.int8)
    s = np.empty((N, max(K // GROUP, 1)), dtype=np.uint16)
    _check(lib.tq_ternarize(N, K, w.ctypes.data, t.ctypes.data, s.ctypes.data), "tq_ternarize")
    return t, s


def tq_unpack(fmt: int, blob: np.ndarray, N: int, K: int):
    """Inverse of tq_pack -> (trits int8 [N][K], scales uint16 [N][K/128])."""
    b = np.ascontiguousarray(blob, dtype=np.uint8)
    t = np.empty((N, K), dtype=np.int8)
    s = np.empty((N, K // GROUP), dtype=np.uint16)
    _check(lib.tq_unpack(fmt, N, K, b.ctypes.data, b.size, t.ctypes.data, s.ctypes.data),
           "tq_unpack")
    return t, s


# ---- device ---------------------------------------------------------------

def tq_quant_act(x, q, a_scale, stream=None) -> None:
    """x [M][K] fp16/fp32 (device) -> q int8 [M][K], a_scale fp32 [M]."""
    import torch
    dtype = {torch.float16: TQ_F16, torch.float32: TQ_F32}.get(x.dtype, -1)
    M, K = x.shape
    _check(lib.tq_quant_act(dtype, M, K, _ptr(x), _ptr(q), _ptr(a_scale), _stream(stream)),
           "tq_quant_act")


def tq_hadamard_quant_act(x, signs, q, a_scale, stream=None) -> None:
    """x [M][K] fp16/fp32 (device), signs int8 [K] -> q int8 [M][K], a_scale
    fp32 [M] of the block-64 Hadamard-rotated rows."""
    import torch
    dtype = {torch.float16: TQ_F16, torch.float32: TQ_F32}.get(x.dtype, -1)
    M, K = x.shape
    _check(lib.tq_hadamard_quant_act(dtype, M, K, _ptr(x), _ptr(signs), _ptr(q), _ptr(a_scale),
                                     _stream(stream)), "tq_hadamard_quant_act")


def tq_gemv_workspace_bytes(fmt: int, M: int, N: int, K: int) -> int:
    return int(lib.tq_gemv_workspace_bytes(fmt, M, N, K))


def tq_gemm_workspace_bytes(fmt: int, M: int, N: int, K: int) -> int:
    return int(lib.tq_gemm_workspace_bytes(fmt, M, N, K))


def _ws(ws):
    return (None, 0) if ws is None else (_ptr(ws), ws.numel() * ws.element_size())


def tq_gemv(fmt, M, N, K, W, q, a_scale, y, ws=None, stream=None) -> None:
    wp, wb = _ws(ws)
    _check(lib.tq_gemv(fmt, M, N, K, _ptr(W), _ptr(q), _ptr(a_scale), _ptr(y), wp, wb,
                       _stream(stream)), "tq_gemv")


def tq_gemv_noalloc(fmt, M, N, K, W, q, a_scale, y, stream=None) -> None:
    """tq_gemv with the library's own fixed device scratch array as workspace."""
    _check(lib.tq_gemv_noalloc(fmt, M, N, K, _ptr(W), _ptr(q), _ptr(a_scale), _ptr(y), _stream(stream)),
           "tq_gemv_noalloc")


def tq_gemv_gate_up_swiglu(fmt, M, N, K, Wg, Wu, q, a_scale, h, ws=None, stream=None) -> None:
    wp, wb = _ws(ws)
    _check(lib.tq_gemv_gate_up_swiglu(fmt, M, N, K, _ptr(Wg), _ptr(Wu), _ptr(q), _ptr(a_scale),
                                      _ptr(h), wp, wb, _stream(stream)), "tq_gemv_gate_up_swiglu")


def tq_gemm(fmt, M, N, K, W, q, a_scale, y, ws=None, stream=None) -> None:
    wp, wb = _ws(ws)
    _check(lib.tq_gemm(fmt, M, N, K, _ptr(W), _ptr(q), _ptr(a_scale), _ptr(y), wp, wb,
                       _stream(stream)), "tq_gemm")


def tq_debug_unpack(fmt, N, K, W, trits, stream=None) -> None:
    _check(lib.tq_debug_unpack(fmt, N, K, _ptr(W), _ptr(trits), _stream(stream)),
           "tq_debug_unpack")


def tq_debug_group_sums(fmt, M, N, K, W, q, S, use_gemm_path=False, stream=None) -> None:
    _check(lib.tq_debug_group_sums(fmt, M, N, K, _ptr(W), _ptr(q), _ptr(S), int(use_gemm_path),
                                   _stream(stream)), "tq_debug_group_sums")


def tq_debug_gate_up_sums(fmt, M, N, K, Wg, Wu, q, S, stream=None) -> None:
    """S int32 [2][M][N][K/128]: the gate and up group sums of tq_gemv_gate_up_swiglu's kernel."""
    _check(lib.tq_debug_gate_up_sums(fmt, M, N, K, _ptr(Wg), _ptr(Wu), _ptr(q), _ptr(S),
                                     _stream(stream)), "tq_debug_gate_up_sums")


def tq_debug_gemv_quant_sums(fmt, N, K, W, Wu, x, S, x_bmax=None, a_scale=None, stream=None) -> None:
    """S int32 [nmat][N][K/128] (and a_scale fp32 [1]) from tq_gemv_quant's kernel,
    which quantises x (fp16 [K], or fp32 [K] with x_bmax) inside the launch."""
    import torch
    dtype = {torch.float16: TQ_F16, torch.float32: TQ_F32}.get(x.dtype, -1)
    nb = 0 if x_bmax is None else x_bmax.numel()
    _check(lib.tq_debug_gemv_quant_sums(fmt, N, K, _ptr(W), _ptr(Wu), dtype, _ptr(x), _ptr(x_bmax), nb,
                                        _ptr(S), _ptr(a_scale), _stream(stream)),
           "tq_debug_gemv_quant_sums")


def tq_debug_gemv_quant_rows_sums(fmt, rows, N, K, W, Wu, x, S, x_bmax=None, a_scale=None,
                                  stream=None) -> None:
    """S int32 [nmat][rows][N][K/128] (and a_scale fp32 [rows]) from the batch
    stack's kernel over `rows` token rows of x (fp16 [rows][K], or fp32 with
    x_bmax [rows][K/64])."""
    import torch
    dtype = {torch.float16: TQ_F16, torch.float32: TQ_F32}.get(x.dtype, -1)
    nb = 0 if x_bmax is None else K // 64
    _check(lib.tq_debug_gemv_quant_rows_sums(fmt, rows, N, K, _ptr(W), _ptr(Wu), dtype, _ptr(x),
                                             _ptr(x_bmax), nb, _ptr(S), _ptr(a_scale), _stream(stream)),
           "tq_debug_gemv_quant_rows_sums")


def tq_workspace_clear(ws, stream=None) -> None:
    """Zero-fill a workspace tensor (device, 16-byte aligned, size a multiple
    of 16 bytes) on the stream: the state every workspace-taking call expects."""
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.tq_workspace_clear(_ptr(ws), nbytes, _stream(stream)), "tq_workspace_clear")


def tq_workspace_check(ws, count, stream=None) -> None:
    """count (device int32/uint32 [>= 1]) receives the number of non-zero
    32-bit words of the workspace tensor ws (0: fit for the next call)."""
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.tq_workspace_check(_ptr(ws), nbytes, _ptr(count), _stream(stream)), "tq_workspace_check")


def tq_debug_stream_read(src, sink, stream=None) -> None:
    """Read every byte of src (device tensor, size a multiple of 16) once;
    sink (int32/uint32 [>= TQ_STREAM_READ_WGS]) receives per-workgroup XORs."""
    nbytes = src.numel() * src.element_size()
    _check(lib.tq_debug_stream_read(_ptr(src), nbytes, _ptr(sink), sink.numel(), _stream(stream)),
           "tq_debug_stream_read")


def tq_gemv_quant_workspace_bytes(fmt, N, K, gate_up=False) -> int:
    return int(lib.tq_gemv_quant_workspace_bytes(fmt, N, K, int(bool(gate_up))))


def tq_gemv_quant(fmt, N, K, W, Wu, x, y, x_bmax=None, y_bmax=None, ws=None, stream=None,
                  y_signs=None) -> None:
    """y = W . quant(x) (or SwiGLU of W, Wu) for one token x [K] fp16 / fp32
    (device); fp32 x needs x_bmax, its K/64 block maxima.  y_signs (int8 [N])
    stores y Hadamard-rotated per 64-row block."""
    import torch
    dtype = {torch.float16: TQ_F16, torch.float32: TQ_F32}.get(x.dtype, -1)
    nb = 0 if x_bmax is None else x_bmax.numel()
    wp, wb = _ws(ws)
    _check(lib.tq_gemv_quant(fmt, N, K, _ptr(W), _ptr(Wu), dtype, _ptr(x), _ptr(x_bmax), nb,
                             _ptr(y), _ptr(y_bmax), _ptr(y_signs), wp, wb, _stream(stream)),
           "tq_gemv_quant")


def tq_decode_stack_workspace_bytes(fmt, layers, hidden, inter, qkv_out, o_in) -> int:
    return int(lib.tq_decode_stack_workspace_bytes(fmt, layers, hidden, inter, qkv_out, o_in))


def tq_decode_stack(fmt, layers, hidden, inter, qkv_out, o_in, weights, x_in, a_in,
                    y_qkv, y_o, h, y_out, ws, stream=None, ffn_signs=None, persistent=False) -> None:
    """weights: list of (qkv, o, gate, up, down) device tensors per layer (or a
    ctypes array of TqLayer built once with stack_layers()).  ffn_signs (int8
    [layers][hidden]) rotates the FFN input online.  persistent=True calls
    tq_decode_stack_persistent (one launch per 32 layers) instead of one
    launch per projection."""
    arr = weights if isinstance(weights, ctypes.Array) else stack_layers(weights)
    wp, wb = _ws(ws)
    fn = lib.tq_decode_stack_persistent if persistent else lib.tq_decode_stack
    _check(fn(fmt, layers, hidden, inter, qkv_out, o_in, ctypes.cast(arr, ctypes.c_void_p),
              _ptr(x_in), _ptr(a_in), _ptr(y_qkv), _ptr(y_o), _ptr(h), _ptr(y_out), _ptr(ffn_signs),
              wp, wb, _stream(stream)), "tq_decode_stack_persistent" if persistent else "tq_decode_stack")


def tq_decode_stack_batch_workspace_bytes(fmt, rows, layers, hidden, inter, qkv_out, o_in) -> int:
    return int(lib.tq_decode_stack_batch_workspace_bytes(fmt, rows, layers, hidden, inter, qkv_out, o_in))


def tq_decode_stack_batch(fmt, rows, layers, hidden, inter, qkv_out, o_in, weights, x_in, a_in,
                          y_qkv, y_o, h, y_out, ws, stream=None, ffn_signs=None) -> None:
    """tq_decode_stack for `rows` token rows per launch: x_in [layers][rows][hidden],
    a_in [layers][rows][o_in], outputs [layers][rows][N]."""
    arr = weights if isinstance(weights, ctypes.Array) else stack_layers(weights)
    wp, wb = _ws(ws)
    _check(lib.tq_decode_stack_batch(fmt, rows, layers, hidden, inter, qkv_out, o_in,
                                     ctypes.cast(arr, ctypes.c_void_p), _ptr(x_in), _ptr(a_in),
                                     _ptr(y_qkv), _ptr(y_o), _ptr(h), _ptr(y_out), _ptr(ffn_signs),
                                     wp, wb, _stream(stream)), "tq_decode_stack_batch")


# ---- device: between the projections of a layer --------------------------

def tq_rope_table(positions: int, rot: int, base: float) -> np.ndarray:
    """fp32 [positions][2][rot/2] (host): cosines and sines of each position's angles."""
    t = np.empty((max(positions, 1), 2, max(rot // 2, 1)), dtype=np.float32)
    _check(lib.tq_rope_table(positions, rot, base, t.ctypes.data), "tq_rope_table")
    return t


class _Torch:
    """What the calls below take from torch, looked up once: a decode step
    makes these calls by the hundred, and the host's time is theirs."""
    f16 = None

    @classmethod
    def get(cls):
        if cls.f16 is None:
            import torch
            cls.f32, cls.i32, cls.u8, cls.i8 = torch.float32, torch.int32, torch.uint8, torch.int8
            cls.acts = {torch.float16: TQ_F16, torch.float32: TQ_F32}
            cls.available = torch.cuda.is_available
            # the current device without the check that torch is initialised, and the
            # stream's handle without a Stream object, where torch has them
            cls.device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
            cls.stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: torch.cuda.current_stream(d).cuda_stream)
            cls.f16 = torch.float16
        return cls


def _bad(what, name, t, dtype, shape, dev):
    """The error that a tensor's check found."""
    if t.dtype is not dtype:
        return ValueError(f"{what}: {name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        return ValueError(f"{what}: {name} must be on the current GPU (cuda:{dev}), got {t.device}")
    if tuple(t.shape) != tuple(shape):
        return ValueError(f"{what}: {name} must have shape {list(shape)}, got {list(t.shape)}")
    return ValueError(f"{what}: {name} must be contiguous")


def _need(what, name, t, dtype, shape, dev):
    """Checks that t is a contiguous tensor of that type and shape on GPU `dev`, the
    current one, whose stream the call takes; -> its address."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise _bad(what, name, t, dtype, shape, dev)
    return t.data_ptr()


def _rows_need(what, name, t, dtype, shape, dev):
    """The same for rows that may lie apart; -> (address, elements from row to row)."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        raise _bad(what, name, t, dtype, shape, dev)
    if t.is_contiguous():
        n = shape[1]
        return t.data_ptr(), n if len(shape) == 2 else n * shape[2]
    if not t[0].is_contiguous():
        raise ValueError(f"{what}: {name} must be contiguous within a row")
    return t.data_ptr(), t.stride(0)


def _cache_need(what, T, cu_rows, kv_len, page_table, k_cache, v_cache, k_scale, v_scale, dev):
    """Checks the cache's tensors; -> (seqs, kv_heads, head_dim, their arguments in the library's order)."""
    i32, f32 = T.i32, T.f32
    if k_cache.dim() != 4 or page_table.dim() != 2:
        raise ValueError(f"{what}: k_cache must have shape [pages][kv_heads][{KV_PAGE}][head_dim], page_table two dimensions")
    pages, heads, page, dim = k_cache.shape
    seqs, width = page_table.shape
    per = (pages, heads)
    # one expression where all is well: seven calls of _need would be most of a call's host time
    if not (cu_rows.dtype is kv_len.dtype is page_table.dtype is i32 and k_cache.dtype is v_cache.dtype is T.u8
            and k_scale.dtype is v_scale.dtype is f32
            and cu_rows.get_device() == kv_len.get_device() == page_table.get_device() == k_cache.get_device()
            == v_cache.get_device() == k_scale.get_device() == v_scale.get_device() == dev
            and cu_rows.shape == (seqs + 1,) and kv_len.shape == (seqs,) and page == KV_PAGE
            and v_cache.shape == (pages, heads, dim, KV_PAGE) and k_scale.shape == per and v_scale.shape == per
            and cu_rows.is_contiguous() and kv_len.is_contiguous() and page_table.is_contiguous() and k_cache.is_contiguous()
            and v_cache.is_contiguous() and k_scale.is_contiguous() and v_scale.is_contiguous()):
        for name, t, dtype, shape in (("cu_rows", cu_rows, i32, (seqs + 1,)), ("kv_len", kv_len, i32, (seqs,)),
                                      ("page_table", page_table, i32, (seqs, width)),
                                      ("k_cache", k_cache, T.u8, (pages, heads, KV_PAGE, dim)),
                                      ("v_cache", v_cache, T.u8, (pages, heads, dim, KV_PAGE)),
                                      ("k_scale", k_scale, f32, per), ("v_scale", v_scale, f32, per)):
            _need(what, name, t, dtype, shape, dev)
    return seqs, heads, dim, (cu_rows.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(), width, k_cache.data_ptr(),
                              v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages)


def _current(T, stream, t):
    """(index of the current GPU, the call's stream as an integer) for a call on t and others."""
    if t.get_device() < 0 and not T.available():
        return -1, 0  # nothing can run: the checks do, and the library reports the launch
    dev = T.device()  # (host memory is refused against it: a kernel must not be given its address)
    if stream is None:
        return dev, T.stream(dev)
    return dev, stream if isinstance(stream, int) else stream.cuda_stream


def tq_kv_append(qkv, rope, cu_rows, kv_len, page_table, k_cache, v_cache, k_scale, v_scale, q_out=None,
                 rope_mode=TQ_ROPE_HALVES, q_heads=None, stream=None) -> None:
    """Append the rows of qkv [rows][(q_heads + 2 kv_heads) head_dim] (fp16 or
    fp32; rows may be strided) to the paged cache, rotating keys and queries
    by rope [positions][2][rot/2] (fp32, as tq_rope_table; None: no rotation);
    the rotated queries go to q_out fp16 [rows][q_heads][head_dim]."""
    what, T = "tq_kv_append", _Torch.get()
    dev, st = _current(T, stream, k_cache)
    seqs, heads, dim, cache = _cache_need(what, T, cu_rows, kv_len, page_table, k_cache, v_cache, k_scale, v_scale, dev)
    if qkv.dim() != 2:
        raise ValueError(f"{what}: qkv must have two dimensions")
    rows, width = qkv.shape
    if q_heads is None:
        q_heads = width // max(dim, 1) - 2 * heads
    x, stride = _rows_need(what, "qkv", qkv, qkv.dtype, (rows, (q_heads + 2 * heads) * dim), dev)
    q = None if q_out is None else _need(what, "q_out", q_out, T.f16, (rows, q_heads, dim), dev)
    r, rope_rows, rot = None, 0, 0
    if rope is not None:
        if rope.dim() != 3:
            raise ValueError(f"{what}: rope must have shape [positions][2][rot/2]")
        rope_rows, _, half = rope.shape
        rot = 2 * half
        r = _need(what, "rope", rope, T.f32, (rope_rows, 2, half), dev)
    rc = lib.tq_kv_append(T.acts.get(qkv.dtype, -1), rows, seqs, q_heads, heads, dim, x, stride, r, rope_rows, rot, rope_mode,
                          *cache, q, st)
    if rc:
        raise TQError(rc, what)


def tq_kv_attn_workspace_bytes(rows, seqs, q_heads, kv_heads, head_dim, max_kv_len) -> int:
    return int(lib.tq_kv_attn_workspace_bytes(rows, seqs, q_heads, kv_heads, head_dim, max_kv_len))


def kv_attn_workspace(rows, seqs, q_heads, kv_heads, head_dim, max_kv_len, device="cuda"):
    """A zero-filled workspace tensor for tq_kv_attn (None when it needs none)."""
    import torch
    nbytes = tq_kv_attn_workspace_bytes(rows, seqs, q_heads, kv_heads, head_dim, max_kv_len)
    return torch.zeros((nbytes + 15) // 16 * 4, dtype=torch.int32, device=device) if nbytes else None


def tq_kv_attn(q, cu_rows, kv_len, page_table, k_cache, v_cache, k_scale, v_scale, out, max_kv_len,
               softmax_scale=None, window=0, sinks=0, ws=None, stream=None) -> None:
    """out = attention of q over the cache, both fp16 [rows][q_heads][head_dim]
    (rows may be strided).  max_kv_len: the largest kv_len (a host number).
    softmax_scale defaults to head_dim ** -0.5; window > 0 limits a row to its
    last `window` keys and the first `sinks` ones."""
    what, T = "tq_kv_attn", _Torch.get()
    dev, st = _current(T, stream, k_cache)
    seqs, heads, dim, cache = _cache_need(what, T, cu_rows, kv_len, page_table, k_cache, v_cache, k_scale, v_scale, dev)
    if q.dim() != 3:
        raise ValueError(f"{what}: q must have three dimensions")
    rows, q_heads, _ = q.shape
    shape = (rows, q_heads, dim)
    qp, qs = _rows_need(what, "q", q, T.f16, shape, dev)
    op, os_ = _rows_need(what, "out", out, T.f16, shape, dev)
    wp, wb = None, 0
    if ws is not None:
        if ws.get_device() != dev or not ws.is_contiguous():
            raise ValueError(f"{what}: ws must be contiguous and on the current GPU")
        wp, wb = ws.data_ptr(), ws.numel() * ws.element_size()
    rc = lib.tq_kv_attn(rows, seqs, q_heads, heads, dim, qp, qs, *cache, max_kv_len,
                        dim ** -0.5 if softmax_scale is None else softmax_scale, window, sinks, op, os_, wp, wb, st)
    if rc:
        raise TQError(rc, what)


def tq_residual_norm(y, res, res_out, pre_w=None, x=None, q=None, a_scale=None, post_w=None, gate=None,
                     res_scale=1.0, eps=1e-6, stream=None) -> None:
    """res_out = res + res_scale * gate * norm(y; post_w); x (fp16 / fp32) and / or
    q, a_scale (int8, fp32 [M]) = norm(res_out; pre_w).  All [M][H]; gate [H] or
    [M][H] (rows may be strided); y None: norm(res) only."""
    what, T = "tq_residual_norm", _Torch.get()
    dev, st = _current(T, stream, res)
    if res.dim() != 2:
        raise ValueError(f"{what}: res must have two dimensions")
    M, H = shape = res.shape
    f32, row, rt = T.f32, (H,), res.dtype
    yt = rt if y is None else y.dtype
    gp, gs = None, 0
    if gate is not None:
        if gate.dim() == 2:
            gp, gs = _rows_need(what, "gate", gate, yt, shape, dev)
        else:
            gp = _need(what, "gate", gate, yt, row, dev)
    # (one expression where all is well, as for the cache's tensors)
    if not (res.get_device() == dev and res.is_contiguous()
            and (y is None or y.get_device() == dev and y.shape == shape and y.is_contiguous())
            and (res_out is None or res_out.dtype is rt and res_out.get_device() == dev and res_out.shape == shape
                 and res_out.is_contiguous())
            and (post_w is None or post_w.dtype is f32 and post_w.get_device() == dev and post_w.shape == row
                 and post_w.is_contiguous())
            and (pre_w is None or pre_w.dtype is f32 and pre_w.get_device() == dev and pre_w.shape == row
                 and pre_w.is_contiguous())
            and (x is None or x.get_device() == dev and x.shape == shape and x.is_contiguous())
            and (q is None or q.dtype is T.i8 and q.get_device() == dev and q.shape == shape and q.is_contiguous())
            and (a_scale is None or a_scale.dtype is f32 and a_scale.get_device() == dev and a_scale.shape == (M,)
                 and a_scale.is_contiguous())):
        for name, t, dtype, size in (("res", res, rt, shape), ("y", y, yt, shape), ("res_out", res_out, rt, shape),
                                     ("post_w", post_w, f32, row), ("pre_w", pre_w, f32, row),
                                     ("x", x, None if x is None else x.dtype, shape), ("q", q, T.i8, shape),
                                     ("a_scale", a_scale, f32, (M,))):
            if t is not None:
                _need(what, name, t, dtype, size, dev)
    acts = T.acts
    rc = lib.tq_residual_norm(
        TQ_F32 if y is None else acts.get(yt, -1), acts.get(rt, -1), TQ_F32 if x is None else acts.get(x.dtype, -1), M, H,
        None if y is None else y.data_ptr(), None if post_w is None else post_w.data_ptr(), gp, gs, res_scale, res.data_ptr(),
        None if res_out is None else res_out.data_ptr(), None if pre_w is None else pre_w.data_ptr(), eps,
        None if x is None else x.data_ptr(), None if q is None else q.data_ptr(),
        None if a_scale is None else a_scale.data_ptr(), st)
    if rc:
        raise TQError(rc, what)


def tq_debug_kv_read(pages, k_cache, v_cache, k_scale, v_scale, values, stream=None) -> None:
    """values (fp16 / fp32 [2][n][kv_heads][64][head_dim]) of the cache pages named by pages (int32 [n])."""
    what, T = "tq_debug_kv_read", _Torch.get()
    dev, st = _current(T, stream, k_cache)
    if k_cache.dim() != 4 or pages.dim() != 1:
        raise ValueError(f"{what}: k_cache must have four dimensions, pages one")
    num, heads, page, dim = k_cache.shape
    n, per = pages.shape[0], (num, heads)
    shape = (2, n, heads, KV_PAGE, dim)
    if not (pages.dtype is T.i32 and k_cache.dtype is v_cache.dtype is T.u8 and k_scale.dtype is v_scale.dtype is T.f32
            and pages.get_device() == k_cache.get_device() == v_cache.get_device() == k_scale.get_device()
            == v_scale.get_device() == values.get_device() == dev
            and page == KV_PAGE and v_cache.shape == (num, heads, dim, KV_PAGE) and k_scale.shape == per and v_scale.shape == per
            and values.shape == shape and pages.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()
            and k_scale.is_contiguous() and v_scale.is_contiguous() and values.is_contiguous()):
        for name, t, dtype, size in (("pages", pages, T.i32, (n,)), ("k_cache", k_cache, T.u8, (num, heads, KV_PAGE, dim)),
                                     ("v_cache", v_cache, T.u8, (num, heads, dim, KV_PAGE)), ("k_scale", k_scale, T.f32, per),
                                     ("v_scale", v_scale, T.f32, per), ("values", values, values.dtype, shape)):
            _need(what, name, t, dtype, size, dev)
    rc = lib.tq_debug_kv_read(T.acts.get(values.dtype, -1), n, heads, dim, pages.data_ptr(), k_cache.data_ptr(),
                              v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), num, values.data_ptr(), st)
    if rc:
        raise TQError(rc, what)


def stack_timeouts(ws) -> int:
    """Waits of the persistent decode stack that gave up (the workspace's first
    32-bit word; 0 after correct calls).  Synchronises with the device."""
    return int(ws.view(-1)[0:1].view(-1).cpu().numpy().view("uint32")[0]) if ws is not None else 0


def stack_layers(weights):
    """Host array of TqLayer from [(qkv, o, gate, up, down), ...] device tensors."""
    arr = (TqLayer * len(weights))()
    for i, w in enumerate(weights):
        arr[i] = TqLayer(*[_ptr(t) for t in w])
    return arr


def workspace(fmt: int, M: int, N: int, K: int, device="cuda"):
    """A zero-filled workspace tensor sized for tq_gemv / tq_gemm on this shape
    (None when the shape needs none).  Allocation is the caller's: this helper
    uses torch, never the library."""
    import torch
    nbytes = max(tq_gemv_workspace_bytes(fmt, min(M, GEMV_MAX_M), N, K),
                 tq_gemm_workspace_bytes(fmt, M, N, K))
    if nbytes == 0:
        return None
    return torch.zeros((nbytes + 15) // 16 * 4, dtype=torch.int32, device=device)
