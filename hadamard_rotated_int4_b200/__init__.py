"""Python binding of libhbl.so, the sm_100a H-BitLinear library (BitNet v2).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  torch supplies device memory and the current CUDA stream.  There is
no CPU fallback: calls raise if the library is not built or the device is not
an sm_100 GPU.

Names follow include/hbl.h:
  pack_ternary(W)                         -> (W_packed int32 view [N, K/16], alpha [1])
  norm_fwht(X)                            -> V fp32 [M, K]
  norm_fwht_quant(X, act_bits)            -> (codes uint8, scales fp32 [M], rowsum int32 [M])
  ternary_gemm(codes, scales, rowsum, act_bits, K, W_packed, alpha)  -> Y bf16 [M, N] (, acc)
  hbitlinear_forward(X, W_packed, alpha, act_bits)                   -> Y bf16 [M, N]
  hbitlinear_forward_hostio(X_host, W_packed, alpha, act_bits, Y_host, ws)
  ternary_gemv_noalloc(codes, scales, rowsum, act_bits, K, W_packed, alpha)  -> Y (, acc)
  norm_transform(X, flags)                -> V fp32 [M, K]       (variants: NORM_* flags)
  norm_quant(X, act_bits, flags)          -> (codes, scales, rowsum)
  bitlinear_forward(X, W_packed, alpha, act_bits, flags)            -> Y bf16 [M, N]
  rotate_weights(W, signs)                -> W_rot fp32 [N, K]
  kv_quant(X, bits)                       -> (codes uint8 [rows, D*bits/8], scales fp32 [rows])
  kv_cache_alloc(pages, page_size, heads, D, bits, device)          -> KvCache (paged, low-bit)
  kv_cache_write(cache, K, V, cu_seqlens, kv_lens, block_table)     (quantises new rows into pages)
  kv_cache_read(cache, cu_seqlens, kv_lens, block_table, rows)      -> (K, V) [rows, heads, D]
  kv_attention(Q, cache, cu_seqlens, kv_lens, block_table)          -> O bf16 [rows, q heads, D] (, lse)
"""
import ctypes
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libhbl.so")

HBL_OK = 0
STATUS_NAMES = {0: "HBL_OK", 1: "HBL_ERR_INVALID_ARG", 2: "HBL_ERR_SHAPE", 3: "HBL_ERR_ALIGNMENT",
                4: "HBL_ERR_UNSUPPORTED_ARCH", 5: "HBL_ERR_WORKSPACE", 6: "HBL_ERR_CUDA",
                7: "HBL_ERR_TIMEOUT"}
OP_PACK_TERNARY, OP_TERNARY_GEMM, OP_HBITLINEAR_FORWARD, OP_HBITLINEAR_FORWARD_HOSTIO = 0, 1, 2, 3
ACT_INT4_I32, ACT_INT8_I32 = 0x104, 0x108  # one byte per code, 32-row interleaved layout
ACT_INT4_BYTES = 0x204                      # INT4 codes one byte each, row-major
NORM_LAYERNORM, NORM_NO_HADAMARD = 1, 2     # variant flags of norm_transform / norm_quant / bitlinear_forward
PATH_AUTO, PATH_TC_SS, PATH_GEMV, PATH_TC_TS, PATH_TC_TMA, PATH_TC_DECODE = 0, 1, 2, 3, 4, 5
PATH_TC_PACKED, PATH_TC_PAIR = 6, 7
EXPORTS = ("hbl_status_string", "hbl_version", "hbl_workspace_size", "hbl_workspace_size_path",
           "hbl_pack_ternary", "hbl_norm_fwht", "hbl_norm_fwht_quant", "hbl_ternary_gemm",
           "hbl_ternary_gemm_path", "hbl_hbitlinear_forward", "hbl_hbitlinear_forward_path",
           "hbl_hbitlinear_forward_hostio",
           "hbl_ternary_gemv_noalloc", "hbl_norm_transform", "hbl_norm_quant",
           "hbl_bitlinear_forward", "hbl_rotate_weights", "hbl_kv_quant",
           "hbl_kv_cache_write", "hbl_kv_cache_read", "hbl_kv_attention_workspace",
           "hbl_kv_attention",
           "hbl_expand_ternary", "hbl_ternary_gemm_s8w", "hbl_selftest_bounded_wait",
           "hbl_selftest_clock_wait", "hbl_probe_tc_int8")

_lib = None
_kv_calls = {}  # the KV calls once more, taking packed bytes for their structs


class _CacheArgs(ctypes.Structure):  # hbl_kv_cache
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_codes", "k_scales", "v_codes", "v_scales")] + \
               [(n, ctypes.c_int) for n in ("num_pages", "page_size", "num_kv_heads", "head_dim",
                                            "bits")]


class _BatchArgs(ctypes.Structure):  # hbl_kv_batch
    _fields_ = [(n, ctypes.c_void_p) for n in ("cu_seqlens", "kv_lens", "block_table")] + \
               [(n, ctypes.c_int) for n in ("num_seqs", "pages_per_seq", "rows")]


class _AttnArgs(ctypes.Structure):  # hbl_kv_attn
    _fields_ = [("Q", ctypes.c_void_p), ("q_row_stride", ctypes.c_int64),
                ("q_head_stride", ctypes.c_int64), ("O", ctypes.c_void_p),
                ("o_row_stride", ctypes.c_int64), ("o_head_stride", ctypes.c_int64),
                ("lse", ctypes.c_void_p), ("num_heads", ctypes.c_int), ("max_rows", ctypes.c_int),
                ("max_kv", ctypes.c_int), ("scale", ctypes.c_float), ("causal", ctypes.c_int),
                ("window", ctypes.c_int)]


class HblError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__("%s failed: %s (%s)" % (what, STATUS_NAMES.get(status, status),
                                                  lib().hbl_status_string(status).decode()))


def lib():
    """Load libhbl.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libhbl.so is not built (run __graft_entry__.build() or "
                               "python hadamard_rotated_int4_b200/build.py)")
        L = ctypes.CDLL(LIB_PATH)
        P, I, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.hbl_status_string.restype = ctypes.c_char_p
        L.hbl_status_string.argtypes = [I]
        L.hbl_version.restype = I
        L.hbl_version.argtypes = []
        L.hbl_workspace_size.restype = I
        L.hbl_workspace_size.argtypes = [I, I, I, I, I, ctypes.POINTER(SZ)]
        L.hbl_workspace_size_path.restype = I
        L.hbl_workspace_size_path.argtypes = [I, I, I, I, I, I, ctypes.POINTER(SZ)]
        L.hbl_pack_ternary.restype = I
        L.hbl_pack_ternary.argtypes = [P, I, I, F, P, P, P, SZ, P]
        L.hbl_norm_fwht.restype = I
        L.hbl_norm_fwht.argtypes = [P, P, I, I, F, P, P, P]
        L.hbl_norm_fwht_quant.restype = I
        L.hbl_norm_fwht_quant.argtypes = [P, P, I, I, F, F, I, P, P, P, P, P]
        L.hbl_ternary_gemm.restype = I
        L.hbl_ternary_gemm.argtypes = [P, P, P, I, I, I, P, P, I, P, P, P, SZ, P, P]
        L.hbl_ternary_gemm_path.restype = I
        L.hbl_ternary_gemm_path.argtypes = [P, P, P, I, I, I, P, P, I, P, P, P, SZ, P, I, P]
        L.hbl_hbitlinear_forward.restype = I
        L.hbl_hbitlinear_forward.argtypes = [P, P, I, I, I, P, P, I, F, F, P, P, SZ, P, P]
        L.hbl_hbitlinear_forward_path.restype = I
        L.hbl_hbitlinear_forward_path.argtypes = [P, P, I, I, I, P, P, I, F, F, P, P, SZ, P, I, P]
        L.hbl_hbitlinear_forward_hostio.restype = I
        L.hbl_hbitlinear_forward_hostio.argtypes = [P, P, I, I, I, P, P, I, F, F, P, P, SZ, P, P]
        L.hbl_ternary_gemv_noalloc.restype = I
        L.hbl_ternary_gemv_noalloc.argtypes = [P, P, P, I, I, I, P, P, I, P, P, P, P]
        U, I64 = ctypes.c_uint, ctypes.c_int64
        L.hbl_norm_transform.restype = I
        L.hbl_norm_transform.argtypes = [P, P, I, I, F, U, P, P, P]
        L.hbl_norm_quant.restype = I
        L.hbl_norm_quant.argtypes = [P, P, I, I, F, F, I, U, P, P, P, P, P]
        L.hbl_bitlinear_forward.restype = I
        L.hbl_bitlinear_forward.argtypes = [P, P, I, I, I, P, P, I, U, F, F, P, P, SZ, P, P]
        L.hbl_rotate_weights.restype = I
        L.hbl_rotate_weights.argtypes = [P, P, I, I, P, P, P]
        L.hbl_kv_quant.restype = I
        L.hbl_kv_quant.argtypes = [P, I64, I, I, F, P, P, P, P]
        CA, BA, AA = (ctypes.POINTER(t) for t in (_CacheArgs, _BatchArgs, _AttnArgs))
        L.hbl_kv_cache_write.restype = I
        L.hbl_kv_cache_write.argtypes = [CA, BA, P, I64, I64, P, I64, I64, F, P, P]
        L.hbl_kv_cache_read.restype = I
        L.hbl_kv_cache_read.argtypes = [CA, BA, P, P, I, P, P]
        L.hbl_kv_attention_workspace.restype = I
        L.hbl_kv_attention_workspace.argtypes = [CA, BA, AA, ctypes.POINTER(SZ)]
        L.hbl_kv_attention.restype = I
        L.hbl_kv_attention.argtypes = [CA, BA, AA, P, SZ, P, P]
        for name in ("hbl_kv_cache_write", "hbl_kv_cache_read", "hbl_kv_attention_workspace",
                     "hbl_kv_attention"):
            f = L[name]
            f.restype = I
            f.argtypes = [P if t in (CA, BA, AA) else t for t in getattr(L, name).argtypes]
            _kv_calls[name] = f
        L.hbl_expand_ternary.restype = I
        L.hbl_expand_ternary.argtypes = [P, I, I, P, P, P]
        L.hbl_ternary_gemm_s8w.restype = I
        L.hbl_ternary_gemm_s8w.argtypes = [P, P, I, I, I, P, P, I, P, P, P, P]
        L.hbl_selftest_bounded_wait.restype = I
        L.hbl_selftest_bounded_wait.argtypes = [I, I, P, P]
        L.hbl_selftest_clock_wait.restype = I
        L.hbl_selftest_clock_wait.argtypes = [I, I, I, P, P]
        L.hbl_probe_tc_int8.restype = I
        L.hbl_probe_tc_int8.argtypes = [I, I, P, P]
        _lib = L
    return _lib


def _check(status, what):
    if status != HBL_OK:
        raise HblError(status, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    import torch

    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dev(t, dtype, name):
    import torch

    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def workspace_size(op, M, K, N, act_bits, path=PATH_AUTO):
    """Workspace bytes of `op` on GEMM back end `path` (PATH_*)."""
    out = ctypes.c_size_t(0)
    _check(lib().hbl_workspace_size_path(op, M, K, N, act_bits, int(path), ctypes.byref(out)),
           "workspace_size")
    return out.value


def _workspace(nbytes, device):
    import torch

    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def new_status(device):
    import torch

    return torch.zeros(4, dtype=torch.int32, device=device)


def pack_ternary(W, eps=1e-5, ws=None):
    import torch

    _dev(W, torch.float32, "W")
    N, K = W.shape
    packed = torch.empty((N, K // 16), dtype=torch.int32, device=W.device)
    alpha = torch.empty(4, dtype=torch.float32, device=W.device)
    need = workspace_size(OP_PACK_TERNARY, 0, K, N, 0)
    if ws is None:
        ws = _workspace(need, W.device)
    _check(lib().hbl_pack_ternary(_ptr(W), N, K, float(eps), _ptr(packed), _ptr(alpha), _ptr(ws),
                                  ws.numel(), _stream()), "hbl_pack_ternary")
    return packed, alpha[:1]


def norm_fwht(X, gain=None, norm_eps=1e-6, status=None):
    import torch

    _dev(X, torch.bfloat16, "X")
    M, K = X.shape
    V = torch.empty((M, K), dtype=torch.float32, device=X.device)
    _check(lib().hbl_norm_fwht(_ptr(X), _ptr(gain), M, K, float(norm_eps), _ptr(V), _ptr(status),
                               _stream()), "hbl_norm_fwht")
    return V


def codes_shape(M, K, act_bits):
    if act_bits in (ACT_INT4_I32, ACT_INT8_I32):
        return ((M + 31) // 32 * 32, K)
    return (M, K // 2 if act_bits == 4 else K)


def norm_fwht_quant(X, act_bits, gain=None, norm_eps=1e-6, quant_eps=1e-5, out=None,
                    status=None):
    import torch

    _dev(X, torch.bfloat16, "X")
    M, K = X.shape
    if out is None:
        codes = torch.empty(codes_shape(M, K, act_bits), dtype=torch.uint8, device=X.device)
        scales = torch.empty(max(M, 4), dtype=torch.float32, device=X.device)
        rowsum = torch.empty(max(M, 4), dtype=torch.int32, device=X.device)
    else:
        codes, scales, rowsum = out
    _check(lib().hbl_norm_fwht_quant(_ptr(X), _ptr(gain), M, K, float(norm_eps),
                                     float(quant_eps), int(act_bits), _ptr(codes), _ptr(scales),
                                     _ptr(rowsum), _ptr(status), _stream()),
           "hbl_norm_fwht_quant")
    return codes, scales[:M], rowsum[:M]


def ternary_gemm(codes, scales, rowsum, act_bits, K, W_packed, alpha, want_acc=False, ws=None,
                 out=None, status=None, path=PATH_AUTO):
    """hbl_ternary_gemm (hbl_ternary_gemm_path for a back end other than PATH_AUTO:
    PATH_TC_SS tensor cores with both operands staged by threads, PATH_GEMV
    CUDA-core GEMV, PATH_TC_TS tensor cores with activations in TMEM,
    PATH_TC_TMA TMA-fed tensor cores for one-byte codes, PATH_TC_DECODE the
    decode-batch tensor-core kernel for one-byte codes and M <= 128,
    PATH_TC_PACKED the large-batch tensor-core kernel on the packed weights,
    PATH_TC_PAIR the TMA-fed large-batch kernel on pairs of SMs)."""
    import torch

    M = scales.shape[0]  # the interleaved layouts pad the codes buffer to 32 rows
    N = W_packed.shape[0]
    Y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16,
                                                device=codes.device)
    acc = torch.empty((M, N), dtype=torch.int32, device=codes.device) if want_acc else None
    need = workspace_size(OP_TERNARY_GEMM, M, K, N, act_bits, path)
    if ws is None:
        ws = _workspace(need, codes.device)
    _check(lib().hbl_ternary_gemm_path(_ptr(codes), _ptr(scales), _ptr(rowsum), int(act_bits), M,
                                       K, _ptr(W_packed), _ptr(alpha), N, _ptr(Y), _ptr(acc),
                                       _ptr(ws), ws.numel(), _ptr(status), int(path), _stream()),
           "hbl_ternary_gemm")
    return (Y, acc) if want_acc else Y


def ternary_gemv_noalloc(codes, scales, rowsum, act_bits, K, W_packed, alpha, want_acc=False,
                         out=None, status=None):
    """hbl_ternary_gemv_noalloc: the split-K GEMV with the library's fixed scratch
    array (no workspace argument; the library allocates nothing)."""
    import torch

    M = scales.shape[0]
    N = W_packed.shape[0]
    Y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16,
                                                device=codes.device)
    acc = torch.empty((M, N), dtype=torch.int32, device=codes.device) if want_acc else None
    _check(lib().hbl_ternary_gemv_noalloc(_ptr(codes), _ptr(scales), _ptr(rowsum),
                                          int(act_bits), M, K, _ptr(W_packed), _ptr(alpha), N,
                                          _ptr(Y), _ptr(acc), _ptr(status), _stream()),
           "hbl_ternary_gemv_noalloc")
    return (Y, acc) if want_acc else Y


def hbitlinear_forward(X, W_packed, alpha, act_bits, gain=None, norm_eps=1e-6, quant_eps=1e-5,
                       ws=None, out=None, status=None, path=PATH_AUTO):
    """hbl_hbitlinear_forward (hbl_hbitlinear_forward_path for another GEMM back end)."""
    import torch

    _dev(X, torch.bfloat16, "X")
    M, K = X.shape
    N = W_packed.shape[0]
    Y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    if ws is None:
        ws = _workspace(workspace_size(OP_HBITLINEAR_FORWARD, M, K, N, act_bits, path), X.device)
    _check(lib().hbl_hbitlinear_forward_path(_ptr(X), _ptr(gain), M, K, N, _ptr(W_packed),
                                             _ptr(alpha), int(act_bits), float(norm_eps),
                                             float(quant_eps), _ptr(Y), _ptr(ws), ws.numel(),
                                             _ptr(status), int(path), _stream()),
           "hbl_hbitlinear_forward")
    return Y


def hbitlinear_forward_hostio(X_host, W_packed, alpha, act_bits, Y_host, ws, gain=None,
                              norm_eps=1e-6, quant_eps=1e-5, status=None):
    """Host bf16 X in, host bf16 Y out (pinned memory makes the copies asynchronous)."""
    M, K = X_host.shape
    N = W_packed.shape[0]
    _check(lib().hbl_hbitlinear_forward_hostio(_ptr(X_host), _ptr(gain), M, K, N, _ptr(W_packed),
                                               _ptr(alpha), int(act_bits), float(norm_eps),
                                               float(quant_eps), _ptr(Y_host), _ptr(ws),
                                               ws.numel(), _ptr(status), _stream()),
           "hbl_hbitlinear_forward_hostio")
    return Y_host


# ------------------------------------------------------------------ variants

def norm_transform(X, flags=0, gain=None, norm_eps=1e-6, status=None):
    """hbl_norm_transform: V = T(N(X)) with NORM_LAYERNORM / NORM_NO_HADAMARD flags."""
    import torch

    _dev(X, torch.bfloat16, "X")
    M, K = X.shape
    V = torch.empty((M, K), dtype=torch.float32, device=X.device)
    _check(lib().hbl_norm_transform(_ptr(X), _ptr(gain), M, K, float(norm_eps), int(flags),
                                    _ptr(V), _ptr(status), _stream()), "hbl_norm_transform")
    return V


def norm_quant(X, act_bits, flags=0, gain=None, norm_eps=1e-6, quant_eps=1e-5, out=None,
               status=None):
    import torch

    _dev(X, torch.bfloat16, "X")
    M, K = X.shape
    if out is None:
        codes = torch.empty(codes_shape(M, K, act_bits), dtype=torch.uint8, device=X.device)
        scales = torch.empty(max(M, 4), dtype=torch.float32, device=X.device)
        rowsum = torch.empty(max(M, 4), dtype=torch.int32, device=X.device)
    else:
        codes, scales, rowsum = out
    _check(lib().hbl_norm_quant(_ptr(X), _ptr(gain), M, K, float(norm_eps), float(quant_eps),
                                int(act_bits), int(flags), _ptr(codes), _ptr(scales),
                                _ptr(rowsum), _ptr(status), _stream()), "hbl_norm_quant")
    return codes, scales[:M], rowsum[:M]


def bitlinear_forward(X, W_packed, alpha, act_bits, flags=0, gain=None, norm_eps=1e-6,
                      quant_eps=1e-5, ws=None, out=None, status=None):
    import torch

    _dev(X, torch.bfloat16, "X")
    M, K = X.shape
    N = W_packed.shape[0]
    Y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    if ws is None:
        ws = _workspace(workspace_size(OP_HBITLINEAR_FORWARD, M, K, N, act_bits), X.device)
    _check(lib().hbl_bitlinear_forward(_ptr(X), _ptr(gain), M, K, N, _ptr(W_packed),
                                       _ptr(alpha), int(act_bits), int(flags), float(norm_eps),
                                       float(quant_eps), _ptr(Y), _ptr(ws), ws.numel(),
                                       _ptr(status), _stream()), "hbl_bitlinear_forward")
    return Y


def rotate_weights(W, signs=None, out=None, status=None):
    """hbl_rotate_weights: W_rot = FWHT(W * signs) / sqrt(K) per row (out may be W)."""
    import torch

    _dev(W, torch.float32, "W")
    N, K = W.shape
    if signs is not None:
        _dev(signs, torch.float32, "signs")
    Wr = out if out is not None else torch.empty_like(W)
    _check(lib().hbl_rotate_weights(_ptr(W), _ptr(signs), N, K, _ptr(Wr), _ptr(status),
                                    _stream()), "hbl_rotate_weights")
    return Wr


def kv_code_bytes(D, bits):
    return D * bits // 8


def kv_quant(X, bits, eps=1e-5, out=None, status=None):
    """hbl_kv_quant over the last dimension (one head of one token per row)."""
    import torch

    _dev(X, torch.bfloat16, "X")
    D = X.shape[-1]
    rows = X.numel() // D if D else 0
    if out is None:
        codes = torch.empty((rows, kv_code_bytes(D, bits)), dtype=torch.uint8, device=X.device)
        scales = torch.empty(max(rows, 4), dtype=torch.float32, device=X.device)
    else:
        codes, scales = out
    _check(lib().hbl_kv_quant(_ptr(X), rows, D, int(bits), float(eps), _ptr(codes),
                              _ptr(scales), _ptr(status), _stream()), "hbl_kv_quant")
    return codes, scales[:rows]


# ------------------------------------------------------- paged low-bit KV cache
# These calls run once per layer and token, so their marshalling is kept short:
# the structs are packed bytes, the stream is asked for by device index, and torch
# is looked up by the first KvCache (without which there is no call), not by each call.

_torch = None

_pack_cache = struct.Struct("@PPPPiiiii4x").pack         # hbl_kv_cache
_pack_batch = struct.Struct("@PPPiii4x").pack           # hbl_kv_batch
_pack_attn = struct.Struct("@PqqPqqPiiifii").pack       # hbl_kv_attn


class KvCache:
    """A paged low-bit K/V cache: uint8 codes [pages, heads, page_size, D*bits/8]
    and fp32 scales [pages, heads, page_size], for K and for V (hbl_kv_cache).

    Its tensors and sizes are fixed (a larger pool is another KvCache): their addresses
    are packed once, for all calls.  A call on a cache whose tensors' memory has been
    resized or exchanged since is refused."""

    __slots__ = ("_tensors", "_sizes", "_device", "_index", "_at", "_args")

    k_codes = property(lambda self: self._tensors[0])
    k_scales = property(lambda self: self._tensors[1])
    v_codes = property(lambda self: self._tensors[2])
    v_scales = property(lambda self: self._tensors[3])
    num_pages = property(lambda self: self._sizes[0])
    num_kv_heads = property(lambda self: self._sizes[1])
    page_size = property(lambda self: self._sizes[2])
    head_dim = property(lambda self: self._sizes[3])
    bits = property(lambda self: self._sizes[4])
    device = property(lambda self: self._device)

    def __init__(self, k_codes, k_scales, v_codes, v_scales, head_dim):
        global _torch
        if _torch is None:
            import torch as _torch

        u8, f32 = _torch.uint8, _torch.float32
        if not (k_codes.dtype is u8 and v_codes.dtype is u8 and k_scales.dtype is f32 and
                v_scales.dtype is f32 and k_codes.is_cuda and k_codes.is_contiguous() and
                v_codes.is_contiguous() and k_scales.is_contiguous() and
                v_scales.is_contiguous()):
            _dev(k_codes, u8, "k_codes")
            _dev(v_codes, u8, "v_codes")
            _dev(k_scales, f32, "k_scales")
            _dev(v_scales, f32, "v_scales")
        shape, code_shape = k_scales.shape, k_codes.shape
        if len(shape) != 3 or len(code_shape) != 4 or code_shape[:3] != shape or \
                v_codes.shape != code_shape or v_scales.shape != shape:
            raise ValueError("codes must be [pages, heads, page_size, D*bits/8] and scales "
                             "[pages, heads, page_size], alike for K and V")
        self._device = device = k_codes.device
        if not device == v_codes.device == k_scales.device == v_scales.device:
            raise ValueError("the cache's tensors must be on one device")
        head_dim = int(head_dim)
        nbytes = code_shape[3]
        bits = nbytes * 8 // head_dim if head_dim > 0 else 0
        if head_dim < 1 or kv_code_bytes(head_dim, bits) != nbytes:
            raise ValueError("the codes' last dimension must be head_dim * bits / 8 bytes")
        self._index = device.index
        self._tensors = (k_codes, k_scales, v_codes, v_scales)
        self._sizes = (shape[0], shape[1], shape[2], head_dim, bits)
        self._at = at = tuple([t.data_ptr() for t in self._tensors])
        self._args = _pack_cache(*at, shape[0], shape[2], shape[1], head_dim, bits)


def kv_cache_alloc(num_pages, page_size, num_kv_heads, head_dim, bits, device):
    """An empty KvCache (its pages need no initial values)."""
    import torch

    shape = (num_pages, num_kv_heads, page_size)
    codes = [torch.empty(shape + (kv_code_bytes(head_dim, bits),), dtype=torch.uint8,
                         device=device) for _ in range(2)]
    scales = [torch.empty(shape, dtype=torch.float32, device=device) for _ in range(2)]
    return KvCache(codes[0], scales[0], codes[1], scales[1], head_dim)


def _kv_batch(cache, cu_seqlens, kv_lens, block_table, rows):
    """hbl_kv_batch of int32 CUDA tensors on the cache's device."""
    i32, device = _torch.int32, cache._device
    for t in (cu_seqlens, kv_lens, block_table):
        if not isinstance(t, _torch.Tensor) or t.dtype is not i32 or t.device != device or \
                not t.is_contiguous():
            _dev(t, i32, "each of cu_seqlens, kv_lens and block_table")
            raise ValueError("cu_seqlens, kv_lens and block_table must be on the cache's device")
    n, cu, table = kv_lens.shape, cu_seqlens.shape, block_table.shape
    if len(n) != 1 or len(cu) != 1 or len(table) != 2 or cu[0] != n[0] + 1 or table[0] != n[0]:
        raise ValueError("kv_lens must be [seqs], cu_seqlens [seqs + 1] and block_table "
                         "[seqs, pages]")
    return _pack_batch(cu_seqlens.data_ptr(), kv_lens.data_ptr(), block_table.data_ptr(), n[0],
                       table[1], rows)


def _kv_rows(t, cache, name, heads=None):
    """Checks a strided bf16 [rows, heads, D] tensor; returns its strides."""
    if not isinstance(t, _torch.Tensor) or t.dtype is not _torch.bfloat16 or \
            t.device != cache._device:
        if not isinstance(t, _torch.Tensor) or not t.is_cuda:
            raise TypeError("%s must be a CUDA tensor" % name)
        if t.dtype != _torch.bfloat16:
            raise TypeError("%s must be %s, got %s" % (name, _torch.bfloat16, t.dtype))
        raise ValueError("%s must be on the cache's device" % name)
    shape = t.shape
    if len(shape) != 3 or shape[2] != cache._sizes[3] or (heads is not None and shape[1] != heads):
        raise ValueError("%s must be [rows, heads, head_dim] like the cache" % name)
    sr, sh, sd = t.stride()
    if sd != 1:
        raise ValueError("%s must be contiguous in its last dimension" % name)
    # the stride of a dimension of one is never used
    return sr if shape[0] > 1 else 0, sh if shape[1] > 1 else 0


def _kv_overlap(rows, heads, D, a, b=None):
    """Whether two strided [rows, heads, D] tensors share an element, each given as (first
    element, row stride, head stride), strides not negative; without b, whether
    elements of a are elements of a twice."""
    if rows == 0 or heads == 0:
        return False
    if b is None:
        # one dimension's steps hold the other's whole extent
        for (n, s), (m, t) in (((heads, a[2]), (rows, a[1])), ((rows, a[1]), (heads, a[2]))):
            if (n == 1 or s >= D) and (m == 1 or t >= (n - 1) * (s if n > 1 else 0) + D):
                return False
    else:
        ends = [at + (rows - 1) * r + (heads - 1) * h + D for at, r, h in (a, b)]
        if ends[0] <= b[0] or ends[1] <= a[0]:
            return False
        if a[1] == b[1] and a[1] > 0:  # side by side in rows of one stride
            width, off = (heads - 1) * a[2] + D, (b[0] - a[0]) % a[1]
            if width <= off and off + (heads - 1) * b[2] + D <= a[1]:
                return False
    import torch

    # all pieces of D elements in order: two neighbours that overlap, of either tensor
    starts = [(at + torch.arange(rows)[:, None] * r + torch.arange(heads) * h).flatten()
              for at, r, h in ((a,) if b is None else (a, b))]
    if b is None:
        order = starts[0].sort().values
        return bool((order[1:] - order[:-1] < D).any())
    first = starts[0].sort().values
    next_ = torch.searchsorted(first, starts[1] - D, right=True)  # the first that ends behind
    return bool((first[next_.clamp(max=len(first) - 1)] - starts[1]).abs().lt(D).any())


def _kv_call(what, cache, *args):
    """Calls the library on the cache's device and that device's current stream."""
    k, ks, v, vs = cache._tensors
    if (k.data_ptr(), ks.data_ptr(), v.data_ptr(), vs.data_ptr()) != cache._at:
        raise ValueError("a tensor of the cache has been resized or exchanged")
    if _lib is None:
        lib()
    index = cache._index
    stream = _torch._C._cuda_getCurrentRawStream(index)
    if index == _torch._C._cuda_getDevice():
        status = _kv_calls[what](*args, stream)
    else:
        with _torch.cuda.device(index):
            status = _kv_calls[what](*args, stream)
    if status != HBL_OK:
        raise HblError(status, what)


def _kv_status(status, cache):
    if status is None:
        return None
    _dev(status, _torch.int32, "status")
    if status.device != cache._device:
        raise ValueError("status must be on the cache's device")
    return status.data_ptr()


def kv_cache_write(cache, K, V, cu_seqlens, kv_lens, block_table, eps=1e-5, status=None):
    """hbl_kv_cache_write: quantise the packed new rows K, V [rows, heads, D] (any
    row and head strides that are multiples of 8) into the batch's pages."""
    ks = _kv_rows(K, cache, "K", cache._sizes[1])
    vs = _kv_rows(V, cache, "V", cache._sizes[1])
    rows = K.shape[0]
    if V.shape[0] != rows:
        raise ValueError("K and V must have the same shape")
    batch = _kv_batch(cache, cu_seqlens, kv_lens, block_table, rows)
    _kv_call("hbl_kv_cache_write", cache, cache._args, batch, K.data_ptr(), ks[0], ks[1],
             V.data_ptr(), vs[0], vs[1], float(eps), _kv_status(status, cache))


def kv_cache_read(cache, cu_seqlens, kv_lens, block_table, rows, dtype=None, out=None,
                  status=None):
    """hbl_kv_cache_read: the last cu_seqlens[b+1] - cu_seqlens[b] positions of each
    sequence as (K, V) [rows, heads, D], bf16 (default) or torch.float32."""
    rows = int(rows)
    shape = (rows, cache._sizes[1], cache._sizes[3])
    if out is None:
        dtype = _torch.bfloat16 if dtype is None else dtype
        if dtype not in (_torch.bfloat16, _torch.float32):
            raise TypeError("dtype must be torch.bfloat16 or torch.float32, got %s" % dtype)
        if rows < 0:
            raise ValueError("rows must not be negative")
        like = cache._tensors[1] if dtype is _torch.float32 else None
        K = like.new_empty(shape) if like is not None else \
            _torch.empty(shape, dtype=dtype, device=cache._device)
        V = _torch.empty_like(K)
    else:
        K, V = out
        dtype = K.dtype if dtype is None else dtype
        if dtype not in (_torch.bfloat16, _torch.float32):
            raise TypeError("out must be torch.bfloat16 or torch.float32, got %s" % dtype)
        for t in (K, V):
            _dev(t, dtype, "out")
            if tuple(t.shape) != shape or t.device != cache._device:
                raise ValueError("out must be two [rows, heads, D] tensors on the cache's device")
        if abs(K.data_ptr() - V.data_ptr()) < K.numel() * K.element_size():
            raise ValueError("out must be two tensors that do not overlap")
    batch = _kv_batch(cache, cu_seqlens, kv_lens, block_table, rows)
    _kv_call("hbl_kv_cache_read", cache, cache._args, batch, K.data_ptr(), V.data_ptr(),
             1 if dtype == _torch.float32 else 0, _kv_status(status, cache))
    return K, V


def _kv_attention_bytes(cache_args, batch, args):
    if _lib is None:
        lib()
    need = ctypes.c_size_t(0)
    _check(_kv_calls["hbl_kv_attention_workspace"](cache_args, batch, args, ctypes.byref(need)),
           "hbl_kv_attention_workspace")
    return need.value


def kv_attention_workspace_size(rows, num_heads, cache, num_seqs, pages_per_seq, max_rows=0,
                                max_kv=0, causal=True, window=0):
    """Workspace bytes of kv_attention for these sizes."""
    batch = _pack_batch(0, 0, 0, int(num_seqs), int(pages_per_seq), int(rows))
    args = _pack_attn(0, 0, 0, 0, 0, 0, 0, int(num_heads), int(max_rows or 0), int(max_kv or 0),
                      1.0, 1 if causal else 0, int(window))
    return _kv_attention_bytes(cache._args, batch, args)


def kv_attention(Q, cache, cu_seqlens, kv_lens, block_table, max_rows=None, max_kv=None,
                 scale=None, causal=True, window=0, want_lse=False, ws=None, out=None,
                 status=None):
    """hbl_kv_attention: the packed rows Q [rows, q heads, D] attend to everything
    their sequences have cached, their own positions among it.  scale defaults to
    1/sqrt(D); window 0 is none.  max_rows (no sequence has more rows) and max_kv
    (about the longest sequence) are host-side sizes that the launch is planned
    with; without them the row count and the block table's width are taken.
    out may be Q itself, but must not overlap it otherwise.  Returns O (out if given), with want_lse also lse fp32 [rows, q heads]."""
    q_row, q_head = _kv_rows(Q, cache, "Q")
    rows, heads, D = Q.shape
    q_ptr = Q.data_ptr()
    if out is None:
        out = _torch.empty_like(Q) if Q.is_contiguous() else Q.new_empty((rows, heads, D))
        o_row, o_head = heads * D, D
        o_ptr = out.data_ptr()
    else:
        o_row, o_head = _kv_rows(out, cache, "out", heads)
        if out.shape[0] != rows:
            raise ValueError("out must have Q's shape")
        # rows of heads that hold D values each, apart from Q, need no closer look
        o_ptr, width, down = out.data_ptr(), (heads - 1) * o_head + D, rows - 1
        if (o_head < D and heads > 1 or o_row < width and down) and \
                _kv_overlap(rows, heads, D, (0, o_row, o_head)):
            raise ValueError("out's rows and heads must not overlap one another")
        if q_ptr < o_ptr + 2 * (down * o_row + width) and \
                o_ptr < q_ptr + 2 * (down * q_row + (heads - 1) * q_head + D):
            # (Q itself will do: a row is read before it is written, by the same CTA)
            q, o = (q_ptr >> 1, q_row, q_head), (o_ptr >> 1, o_row, o_head)
            if q != o and _kv_overlap(rows, heads, D, q, o):
                raise ValueError("out must not overlap Q, unless it is Q")
    lse = cache._tensors[1].new_empty((rows, heads)) if want_lse else None
    batch = _kv_batch(cache, cu_seqlens, kv_lens, block_table, rows)
    args = _pack_attn(q_ptr, q_row, q_head, o_ptr, o_row, o_head,
                      lse.data_ptr() if want_lse else 0, heads, max_rows or 0, max_kv or 0,
                      D ** -0.5 if scale is None else scale, 1 if causal else 0, window)
    if ws is None:
        nbytes = _kv_attention_bytes(cache._args, batch, args)
        if nbytes:
            ws = cache._tensors[0].new_empty(nbytes)
    else:
        if not isinstance(ws, _torch.Tensor) or not ws.is_cuda or ws.device != cache._device or \
                not ws.is_contiguous():
            raise ValueError("ws must be a contiguous tensor on the cache's device")
        nbytes = ws.numel() * ws.element_size()
    _kv_call("hbl_kv_attention", cache, cache._args, batch, args,
             None if ws is None else ws.data_ptr(), nbytes, _kv_status(status, cache))
    return (out, lse) if want_lse else out


# ------------------------------------------------------- expanded weights

def expand_ternary(W_packed, K, out=None, status=None):
    """hbl_expand_ternary: packed 2-bit weights -> int8 t in {-1, 0, 1} [N, K]."""
    import torch

    N = W_packed.shape[0]
    Ws = out if out is not None else torch.empty((N, K), dtype=torch.int8,
                                                 device=W_packed.device)
    _check(lib().hbl_expand_ternary(_ptr(W_packed), N, K, _ptr(Ws), _ptr(status), _stream()),
           "hbl_expand_ternary")
    return Ws


def ternary_gemm_s8w(codes, scales, act_bits, W_s8, alpha, want_acc=False, out=None,
                     status=None):
    """hbl_ternary_gemm_s8w: the TMA-fed tensor-core GEMM on expanded weights."""
    import torch

    M = scales.shape[0]
    N, K = W_s8.shape
    Y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16,
                                                device=codes.device)
    acc = torch.empty((M, N), dtype=torch.int32, device=codes.device) if want_acc else None
    _check(lib().hbl_ternary_gemm_s8w(_ptr(codes), _ptr(scales), int(act_bits), M, K, _ptr(W_s8),
                                      _ptr(alpha), N, _ptr(Y), _ptr(acc), _ptr(status),
                                      _stream()), "hbl_ternary_gemm_s8w")
    return (Y, acc) if want_acc else Y


def selftest_bounded_wait(arrive, timeout_us, status):
    """hbl_selftest_bounded_wait: the bounded-wait failure path on one probe kernel."""
    _check(lib().hbl_selftest_bounded_wait(int(bool(arrive)), int(timeout_us), _ptr(status),
                                           _stream()), "hbl_selftest_bounded_wait")


def selftest_clock_wait(arrive, aborted, limit_clocks, status):
    """hbl_selftest_clock_wait: the attention kernels' wait on one probe kernel."""
    _check(lib().hbl_selftest_clock_wait(int(bool(arrive)), int(bool(aborted)), int(limit_clocks),
                                         _ptr(status), _stream()), "hbl_selftest_clock_wait")


def probe_tc_int8(ctas, mmas_per_cta, status):
    """hbl_probe_tc_int8: back-to-back 128 x 256 x 32 kind::i8 MMAs from shared
    memory on `ctas` SMs (time it with events on the current stream)."""
    _check(lib().hbl_probe_tc_int8(int(ctas), int(mmas_per_cta), _ptr(status), _stream()),
           "hbl_probe_tc_int8")


OPS_PER_PROBE_MMA = 2 * 128 * 256 * 32


def measure_int8_tensor_peak(ctas, mmas_per_cta=1 << 15, reps=5):
    """Best-of-reps dense INT8 rate (TOPS) from the probe, with its launch timed
    by CUDA events on the current stream; returns (tops, status word)."""
    import torch

    status = new_status(torch.device("cuda", torch.cuda.current_device()))
    probe_tc_int8(ctas, 64, status)  # warm-up (shared-memory attribute, clocks)
    torch.cuda.synchronize()
    best = None
    for _ in range(reps):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        probe_tc_int8(ctas, mmas_per_cta, status)
        b.record()
        torch.cuda.synchronize()
        t = a.elapsed_time(b) * 1e-3
        best = t if best is None else min(best, t)
    tops = ctas * mmas_per_cta * OPS_PER_PROBE_MMA / best / 1e12
    return tops, int(status[0].item())
