"""Python binding of the B200 FP8 block-scaled NT GEMM library (libdg.so).

Argument marshalling only: every function here forwards torch tensors' device
pointers, their sizes and the current CUDA stream to the C ABI of
``include/dg.h`` with the same name.  All arithmetic runs in the sm_100a kernels
of ``libdg.so``; there is no fallback.  If the library is missing the first call
raises ``RuntimeError`` (build it with ``__graft_entry__.build()`` or
``python -m moe_grouped_gemm_weight_b200.build``).

Layouts (see include/dg.h):
  A   uint8 / float8_e4m3fn [M, K]          (masked: [G, M_max, K])
  sa  float32, transposed: sa[kb*sa_stride + m] (masked: per group blocks)
  B   uint8 / float8_e4m3fn [N, K] or [G, N, K]
  sb  float32 [ceil(N/128), K/128] or [G, ceil(N/128), K/128]
  D   bfloat16 [M, N]                        (masked: [G, M_max, N])
"""
from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdg.so")

DG_OK, DG_ERR_INVALID_ARG, DG_ERR_UNSUPPORTED, DG_ERR_MISALIGNED, DG_ERR_CUDA = range(5)
DG_DEVERR_TIMEOUT, DG_DEVERR_BAD_M_INDEX, DG_DEVERR_BAD_MASKED_M, DG_DEVERR_NOT_POW2 = 1, 2, 4, 8
DG_DEVERR_BAD_K_OFFSET = 16
DG_DEVERR_BAD_EXPERT = 32
DG_DEVERR_BAD_SEQ_OFFSET = 64
DG_DTYPE_BF16, DG_DTYPE_FP32 = 0, 1
DG_SCORE_SOFTMAX, DG_SCORE_SIGMOID = 0, 1
DG_ACT_NONE, DG_ACT_RELU, DG_ACT_GELU, DG_ACT_GELU_TANH, DG_ACT_SILU = range(5)

_lock = threading.Lock()
_lib = None
torch = None  # imported by the first call that takes tensors: plans, sizes and switches work without it


class DGError(RuntimeError):
    def __init__(self, func: str, status: int, message: str):
        super().__init__(f"{func}: {message} (status {status})")
        self.status = status


class Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in
                ("block_m", "block_n", "stages", "m_blocks", "n_blocks", "tiles", "grid", "smem_bytes",
                 "swap_ab", "split_k", "tail_split")]

    def as_dict(self) -> dict:
        return {n: getattr(self, n) for n, _ in self._fields_}


def lib() -> ctypes.CDLL:
    """The loaded libdg.so (raises RuntimeError if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"CUDA library {LIB_PATH} is missing: run __graft_entry__.build() first")
            L = ctypes.CDLL(LIB_PATH)
            P, I = ctypes.c_void_p, ctypes.c_int
            L.dg_fp8_gemm_nt.restype = I
            L.dg_fp8_gemm_nt.argtypes = [P, P, P, I, P, P, I, I, I, P]
            for nm in ("dg_fp8_gemm_nn", "dg_fp8_gemm_tn", "dg_fp8_gemm_tt"):
                getattr(L, nm).restype = I
                getattr(L, nm).argtypes = [P, P, P, I, P, P, I, I, I, P]
            L.dg_k_grouped_fp8_gemm_tn.restype = I
            L.dg_k_grouped_fp8_gemm_tn.argtypes = [P, P, P, I, P, P, P, I, I, I, I, P]
            L.dg_fp8_gemm_nt_ue8m0.restype = I
            L.dg_fp8_gemm_nt_ue8m0.argtypes = [P, P, P, I, P, P, I, I, I, P]
            L.dg_fp8_gemm_nt_noalloc.restype = I
            L.dg_fp8_gemm_nt_noalloc.argtypes = [P, P, P, I, P, P, I, I, I, P]
            L.dg_to_fp8_1x128.restype = I
            L.dg_to_fp8_1x128.argtypes = [P, P, I, P, I, I, P]
            L.dg_to_fp8_128x128.restype = I
            L.dg_to_fp8_128x128.argtypes = [P, P, P, I, I, P]
            L.dg_grouped_contiguous_nt.restype = I
            L.dg_grouped_contiguous_nt.argtypes = [P, P, P, I, P, P, P, I, I, I, I, P]
            L.dg_grouped_masked_nt.restype = I
            L.dg_grouped_masked_nt.argtypes = [P, P, P, I, P, P, P, I, I, I, I, I, P]
            F = ctypes.c_float
            for nm, at in (
                    ("dg_route_topk", [P, P, P, I, P, I, I, I, I, I, I, I, I, F, P]),
                    ("dg_route_topk_bwd", [P, P, P, I, P, I, I, I, I, I, F, P]),
                    ("dg_get_layout_rows", [I, I, I]),
                    ("dg_route_layout", [P, P, P, P, P, P, I, I, I, I, I, P]),
                    ("dg_dispatch_fp8_1x128", [P, P, I, P, P, I, I, I, I, I, P]),
                    ("dg_combine", [P, P, P, P, I, I, I, I, P]),
                    ("dg_combine_bwd", [P, P, P, I, P, P, I, P, P, P, P, P, I, I, I, I, P]),
                    ("dg_swiglu_fp8", [P, P, I, P, P, I, P, P, I, I, I, P]),
                    ("dg_swiglu_fp8_bwd", [P, P, I, P, P, I, P, P, P, P, P, I, P, I, I, P]),
                    ("dg_fp8_1x128_to_128x128", [P, P, P, P, I, P, I, I, P]),
                    ("dg_fp8_gemm_nt_epilogue", [P, P, P, P, I, P, P, I, P, P, P, I, P, I, I, I, P]),
                    ("dg_get_bias_workspace", [I, I]),
                    ("dg_epilogue_bwd", [P, P, I, P, P, I, P, P, P, P, I, I, I, P]),
                    ("dg_norm_residual", [P, P, P, P, I, P, P, I, P, P, P, P, I, I, I, F, F, P]),
                    ("dg_get_norm_workspace", [I, I]),
                    ("dg_norm_residual_bwd", [P, P, P, P, P, P, P, P, P, I, P, P, P, P, P, I, I, I, F, P]),
                    ("dg_get_balance_workspace", [I, I, I]),
                    ("dg_balance_loss", [P, P, P, P, P, I, P, P, I, I, I, I, I, F, P]),
                    ("dg_balance_loss_bwd", [P, P, P, P, I, P, P, I, I, I, I, I, F, P])):
                getattr(L, nm).restype = I
                getattr(L, nm).argtypes = at
            L.dg_set_pdl.restype = None
            L.dg_set_pdl.argtypes = [I]
            L.dg_get_pdl.restype = I
            L.dg_get_pdl.argtypes = []
            L.dg_set_num_sms.restype = None
            L.dg_set_num_sms.argtypes = [I]
            L.dg_get_num_sms.restype = I
            L.dg_get_num_sms.argtypes = []
            L.dg_get_m_alignment_for_contiguous_layout.restype = I
            L.dg_get_m_alignment_for_contiguous_layout.argtypes = []
            L.dg_get_tma_aligned_size.restype = I
            L.dg_get_tma_aligned_size.argtypes = [I, I]
            L.dg_get_device_error.restype = I
            L.dg_get_device_error.argtypes = [ctypes.POINTER(I)]
            L.dg_get_workspace_count.restype = I
            L.dg_get_workspace_count.argtypes = []
            L.dg_status_string.restype = ctypes.c_char_p
            L.dg_status_string.argtypes = [I]
            L.dg_last_error_message.restype = ctypes.c_char_p
            L.dg_last_error_message.argtypes = []
            L.dg_selftest_bounded_wait.restype = I
            L.dg_selftest_bounded_wait.argtypes = [P]
            L.dg_make_plan.restype = I
            L.dg_make_plan.argtypes = [I, I, I, I, I, I, ctypes.POINTER(Plan)]
            L.dg_make_plan_ue8m0.restype = I
            L.dg_make_plan_ue8m0.argtypes = [I, I, I, I, ctypes.POINTER(Plan)]
            _lib = L
    return _lib


_CALLS = ("dg_route_topk", "dg_route_topk_bwd", "dg_route_layout", "dg_dispatch_fp8_1x128", "dg_combine",
          "dg_combine_bwd", "dg_swiglu_fp8", "dg_swiglu_fp8_bwd", "dg_fp8_1x128_to_128x128",
          "dg_fp8_gemm_nt_epilogue", "dg_epilogue_bwd",
          "dg_norm_residual", "dg_norm_residual_bwd", "dg_balance_loss", "dg_balance_loss_bwd")
_calls = None


def _need_torch() -> None:
    global torch
    if torch is None:
        import torch


def _marshal():
    """The calls around the GEMMs as vector calls (csrc/dg_pycall.cpp), bound to the loaded library."""
    global _calls
    L = lib()
    _need_torch()
    try:
        from . import _dgcall
    except ImportError as e:
        path = os.path.join(_HERE, "_dgcall.so")
        why = f"does not load ({e})" if os.path.exists(path) else "is missing"
        raise RuntimeError(f"the extension {path} {why}: run __graft_entry__.build() first") from e
    for name in _CALLS:
        _dgcall.bind(name, ctypes.cast(getattr(L, name), ctypes.c_void_p).value)
    _calls = _dgcall
    return _calls


def _check(func: str, status: int) -> None:
    if status != DG_OK:
        L = lib()
        msg = L.dg_last_error_message().decode() or L.dg_status_string(status).decode()
        raise DGError(func, status, msg)


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _cdiv(a: int, b: int) -> int:
    return -(-a // b)


def _sa_need(kblocks: int, sa_stride: int, rows: int) -> int:
    """Elements of a transposed scale array sa[kb*sa_stride + m] that the
    library touches for kb < kblocks, m < rows."""
    return 0 if kblocks <= 0 or rows <= 0 else (kblocks - 1) * int(sa_stride) + rows


def _check_dim(func: str, what: str, got: int, want: int) -> None:
    if got != want:
        raise DGError(func, DG_ERR_INVALID_ARG, f"{what} is {got}, expected {want}")


def _check_args(func: str, *specs) -> None:
    """Check the tensor arguments before their pointers cross the C boundary.

    Each spec is (name, tensor, element bytes, elements the call touches).  The
    C ABI takes plain device pointers and cannot see extents, so a tensor that
    is too short, strided, of another element type, or not on the current CUDA
    device would be read or written outside its memory by the kernels.  Such a
    call raises DGError (DG_ERR_INVALID_ARG) here and launches nothing.  None
    passes through: the library itself reports a null pointer."""
    given = [sp for sp in specs if sp[1] is not None]
    for name, t, esize, need in given:
        if t.element_size() != esize:
            raise DGError(func, DG_ERR_INVALID_ARG,
                          f"{name} has {t.element_size()}-byte elements, the call takes {esize}-byte ones")
        if not t.is_contiguous():
            raise DGError(func, DG_ERR_INVALID_ARG, f"{name} is not contiguous")
        if t.numel() < need:
            raise DGError(func, DG_ERR_INVALID_ARG, f"{name} holds {t.numel()} elements, the call touches {need}")
    for name, t, _, _ in given:
        if t.device.type != "cuda":
            raise DGError(func, DG_ERR_INVALID_ARG, f"{name} is not on a CUDA device ({t.device})")
    if given:
        _need_torch()
        cur = torch.cuda.current_device()
        for name, t, _, _ in given:
            if t.device.index != cur:
                raise DGError(func, DG_ERR_INVALID_ARG, f"{name} is on {t.device}, the current device is cuda:{cur}")


def _check_dense(func: str, D, A, sa, sa_stride, B, sb, M: int, N: int, K: int, b_k: int) -> None:
    """Arguments of a dense call: D [M][N] bf16, A with M*K codes, sa
    transposed per 1x128, B with N*K codes (its K extent b_k), sb
    [ceil(N/128)][K/128]."""
    _check_dim(func, "K of B", b_k, K)
    nkb = _cdiv(K, 128)
    _check_args(func, ("D", D, 2, M * N), ("A", A, 1, M * K), ("sa", sa, 4, _sa_need(nkb, sa_stride, M)),
                ("B", B, 1, N * K), ("sb", sb, 4, _cdiv(N, 128) * nkb))


def _stream(stream) -> int:
    if stream is None:
        _need_torch()
        return int(torch.cuda.current_stream().cuda_stream)
    return int(stream if isinstance(stream, int) else stream.cuda_stream)


def dg_fp8_gemm_nt(D, A, sa, sa_stride: int, B, sb, stream=None) -> None:
    """Dense D[M,N] = scaled A[M,K] . B[N,K]^T (sizes taken from A and B)."""
    M, K = A.shape[-2], A.shape[-1]
    N = B.shape[-2]
    _check_dense("dg_fp8_gemm_nt", D, A, sa, sa_stride, B, sb, M, N, K, B.shape[-1])
    _check("dg_fp8_gemm_nt", lib().dg_fp8_gemm_nt(_ptr(D), _ptr(A), _ptr(sa), int(sa_stride), _ptr(B), _ptr(sb),
                                                  M, N, K, _stream(stream)))


def dg_fp8_gemm_nn(D, A, sa, sa_stride: int, B, sb, stream=None) -> None:
    """D[M,N] = scaled A . B^T with A [M,K] and B stored [K,N]."""
    M, K = A.shape[-2], A.shape[-1]
    N = B.shape[-1]
    _check_dense("dg_fp8_gemm_nn", D, A, sa, sa_stride, B, sb, M, N, K, B.shape[-2])
    _check("dg_fp8_gemm_nn", lib().dg_fp8_gemm_nn(_ptr(D), _ptr(A), _ptr(sa), int(sa_stride), _ptr(B), _ptr(sb),
                                                  M, N, K, _stream(stream)))


def dg_fp8_gemm_tn(D, A, sa, sa_stride: int, B, sb, stream=None) -> None:
    """D[M,N] = scaled A . B^T with A stored [K,M] and B stored [K,N]."""
    K, M = A.shape[-2], A.shape[-1]
    N = B.shape[-1]
    _check_dense("dg_fp8_gemm_tn", D, A, sa, sa_stride, B, sb, M, N, K, B.shape[-2])
    _check("dg_fp8_gemm_tn", lib().dg_fp8_gemm_tn(_ptr(D), _ptr(A), _ptr(sa), int(sa_stride), _ptr(B), _ptr(sb),
                                                  M, N, K, _stream(stream)))


def dg_fp8_gemm_tt(D, A, sa, sa_stride: int, B, sb, stream=None) -> None:
    """D[M,N] = scaled A . B^T with A stored [K,M] and B [N,K]."""
    K, M = A.shape[-2], A.shape[-1]
    N = B.shape[-2]
    _check_dense("dg_fp8_gemm_tt", D, A, sa, sa_stride, B, sb, M, N, K, B.shape[-1])
    _check("dg_fp8_gemm_tt", lib().dg_fp8_gemm_tt(_ptr(D), _ptr(A), _ptr(sa), int(sa_stride), _ptr(B), _ptr(sb),
                                                  M, N, K, _stream(stream)))


def dg_k_grouped_fp8_gemm_tn(D, A, sa, sa_stride: int, B, sb, k_offsets, stream=None) -> None:
    """K-grouped GEMM: A stored [K,M], B stored [K,N], k_offsets int32 [G+1] on the
    device, D [G,M,N]."""
    K, M = A.shape[-2], A.shape[-1]
    N = B.shape[-1]
    G = k_offsets.numel() - 1
    func = "dg_k_grouped_fp8_gemm_tn"
    _check_dim(func, "K of B", B.shape[-2], K)
    nkb = _cdiv(K, 128)
    _check_args(func, ("D", D, 2, max(G, 0) * M * N), ("A", A, 1, M * K), ("sa", sa, 4, _sa_need(nkb, sa_stride, M)),
                ("B", B, 1, N * K), ("sb", sb, 4, _cdiv(N, 128) * nkb), ("k_offsets", k_offsets, 4, G + 1))
    _check("dg_k_grouped_fp8_gemm_tn",
           lib().dg_k_grouped_fp8_gemm_tn(_ptr(D), _ptr(A), _ptr(sa), int(sa_stride), _ptr(B), _ptr(sb),
                                          _ptr(k_offsets), G, M, N, K, _stream(stream)))


def dg_fp8_gemm_nt_ue8m0(D, A, sa, sa_stride: int, B, sb, stream=None) -> None:
    """dg_fp8_gemm_nt for power-of-two sa / sb, scaled inside the tensor core."""
    M, K = A.shape[-2], A.shape[-1]
    N = B.shape[-2]
    _check_dense("dg_fp8_gemm_nt_ue8m0", D, A, sa, sa_stride, B, sb, M, N, K, B.shape[-1])
    _check("dg_fp8_gemm_nt_ue8m0", lib().dg_fp8_gemm_nt_ue8m0(_ptr(D), _ptr(A), _ptr(sa), int(sa_stride), _ptr(B),
                                                            _ptr(sb), M, N, K, _stream(stream)))


def dg_fp8_gemm_nt_noalloc(D, A, sa, sa_stride: int, B, sb, stream=None) -> None:
    """dg_fp8_gemm_nt without device allocation: the K-split scratch is a static
    16 MiB array shared by every call on the device, so calls that overlap on
    the GPU race.  Make the first call on each device before any stream capture."""
    M, K = A.shape[-2], A.shape[-1]
    N = B.shape[-2]
    _check_dense("dg_fp8_gemm_nt_noalloc", D, A, sa, sa_stride, B, sb, M, N, K, B.shape[-1])
    _check("dg_fp8_gemm_nt_noalloc",
           lib().dg_fp8_gemm_nt_noalloc(_ptr(D), _ptr(A), _ptr(sa), int(sa_stride), _ptr(B), _ptr(sb),
                                        M, N, K, _stream(stream)))


def dg_to_fp8_1x128(Q, sa, sa_stride: int, X, stream=None) -> None:
    """Activation cast: bf16 X [M,K] -> e4m3 Q [M,K] (uint8) and sa[kb*sa_stride + m]."""
    M, K = X.shape[-2], X.shape[-1]
    _check_args("dg_to_fp8_1x128", ("Q", Q, 1, M * K), ("sa", sa, 4, _sa_need(_cdiv(K, 128), sa_stride, M)),
                ("X", X, 2, M * K))
    _check("dg_to_fp8_1x128", lib().dg_to_fp8_1x128(_ptr(Q), _ptr(sa), int(sa_stride), _ptr(X), M, K,
                                                    _stream(stream)))


def dg_to_fp8_128x128(Q, sb, W, stream=None) -> None:
    """Weight cast: bf16 W [N,K] -> e4m3 Q [N,K] (uint8) and sb [ceil(N/128), K/128]."""
    N, K = W.shape[-2], W.shape[-1]
    _check_args("dg_to_fp8_128x128", ("Q", Q, 1, N * K), ("sb", sb, 4, _cdiv(N, 128) * _cdiv(K, 128)),
                ("W", W, 2, N * K))
    _check("dg_to_fp8_128x128", lib().dg_to_fp8_128x128(_ptr(Q), _ptr(sb), _ptr(W), N, K, _stream(stream)))


def dg_grouped_contiguous_nt(D, A, sa, sa_stride: int, B, sb, m_indices, stream=None) -> None:
    """Contiguous-layout grouped GEMM; B is [G,N,K], m_indices int32 [M_total]."""
    M, K = A.shape[-2], A.shape[-1]
    func = "dg_grouped_contiguous_nt"
    _check_dim(func, "rank of B", B.dim(), 3)
    G, N = B.shape[0], B.shape[1]
    _check_dim(func, "K of B", B.shape[2], K)
    nkb = _cdiv(K, 128)
    _check_args(func, ("D", D, 2, M * N), ("A", A, 1, M * K), ("sa", sa, 4, _sa_need(nkb, sa_stride, M)),
                ("B", B, 1, G * N * K), ("sb", sb, 4, G * _cdiv(N, 128) * nkb), ("m_indices", m_indices, 4, M))
    _check("dg_grouped_contiguous_nt",
           lib().dg_grouped_contiguous_nt(_ptr(D), _ptr(A), _ptr(sa), int(sa_stride), _ptr(B), _ptr(sb),
                                          _ptr(m_indices), M, N, K, G, _stream(stream)))


def dg_grouped_masked_nt(D, A, sa, sa_stride: int, B, sb, masked_m, expected_m: int = 0, stream=None) -> None:
    """Masked-layout grouped GEMM; A is [G,M_max,K], masked_m int32 [G] on the device."""
    func = "dg_grouped_masked_nt"
    _check_dim(func, "rank of A", A.dim(), 3)
    _check_dim(func, "rank of B", B.dim(), 3)
    G, Mmax, K = A.shape
    N = B.shape[1]
    _check_dim(func, "group count of B", B.shape[0], G)
    _check_dim(func, "K of B", B.shape[2], K)
    nkb = _cdiv(K, 128)
    _check_args(func, ("D", D, 2, G * Mmax * N), ("A", A, 1, G * Mmax * K),
                ("sa", sa, 4, _sa_need(G * nkb, sa_stride, Mmax)), ("B", B, 1, G * N * K),
                ("sb", sb, 4, G * _cdiv(N, 128) * nkb), ("masked_m", masked_m, 4, G))
    _check("dg_grouped_masked_nt",
           lib().dg_grouped_masked_nt(_ptr(D), _ptr(A), _ptr(sa), int(sa_stride), _ptr(B), _ptr(sb),
                                      _ptr(masked_m), G, Mmax, N, K, int(expected_m), _stream(stream)))


def _rank_error(func: str, of_rows=(), **tensors) -> DGError:
    """What is wrong with the tensors that a call's sizes come from: rank 2, or (`of_rows`) any but 0."""
    for n, t in tensors.items():
        if not isinstance(t, torch.Tensor) or t.dim() != (2 if n not in of_rows else max(t.dim(), 1)):
            return DGError(func, DG_ERR_INVALID_ARG, f"{n} must be a tensor of " + ("rows" if n in of_rows else "rank 2"))
    return DGError(func, DG_ERR_INVALID_ARG, f"bad sizes of {', '.join(tensors)}")


def _shape1(func: str, name: str, t) -> int:
    if not isinstance(t, torch.Tensor) or t.dim() != 1:
        raise DGError(func, DG_ERR_INVALID_ARG, f"{name} must be a tensor of rank 1")
    return t.shape[0]


# Kinds of elements, as the extension's check of a call's tensors numbers them.
_U8, _BF16, _F32, _I32 = 1, 2, 4, 5


def _check_tensors(func: str, names: str, *triples) -> int:
    """_check_args for the calls around the GEMMs, and the current device's index.

    `triples` are (tensor, kind, elements the call touches) one after the other,
    `names` their names.  The extension checks them in one go (a decoding step
    makes these calls every few microseconds); what is wrong is looked up only
    for the message."""
    cur = _calls.fits(*triples)
    if cur >= 0:
        return cur
    kinds = {_BF16: torch.bfloat16, _F32: torch.float32, _I32: torch.int32}
    given = [(name, *triples[3 * i:3 * i + 3]) for i, name in enumerate(names.split()) if triples[3 * i] is not None]
    for name, t, kind, need in given:
        if not isinstance(t, torch.Tensor) or t.layout != torch.strided:
            raise DGError(func, DG_ERR_INVALID_ARG, f"{name} must be a dense tensor")
        if t.element_size() != 1 if kind == _U8 else t.dtype != kinds[kind]:
            raise DGError(func, DG_ERR_INVALID_ARG, f"{name} is {t.dtype}, the call takes "
                          + ("1-byte elements" if kind == _U8 else str(kinds[kind])))
        if not t.is_contiguous():
            raise DGError(func, DG_ERR_INVALID_ARG, f"{name} is not contiguous")
        if t.numel() < need:
            raise DGError(func, DG_ERR_INVALID_ARG, f"{name} holds {t.numel()} elements, the call touches {need}")
    for name, t, _, _ in given:
        if t.device.type != "cuda":
            raise DGError(func, DG_ERR_INVALID_ARG, f"{name} is not on a CUDA device ({t.device})")
    cur = torch.cuda.current_device()
    for name, t, _, _ in given:
        if t.get_device() != cur:
            raise DGError(func, DG_ERR_INVALID_ARG, f"{name} is on {t.device}, the current device is cuda:{cur}")
    raise DGError(func, DG_ERR_INVALID_ARG, f"an argument is missing or not a tensor: {names}")


def _raw_stream(stream, device: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return _stream(stream)


def _logits_dtype(func: str, logits) -> int:
    if logits.dtype == torch.bfloat16:
        return DG_DTYPE_BF16
    if logits.dtype == torch.float32:
        return DG_DTYPE_FP32
    raise DGError(func, DG_ERR_INVALID_ARG, f"logits are {logits.dtype}, the call takes bfloat16 or float32")


def _scales_need(nkb: int, stride: int, rows: int, group_rows: int) -> int:
    """Elements of a transposed scale array over rows, in one block (group_rows 0) or one per group."""
    if group_rows > 0 and rows >= group_rows:
        return _sa_need(rows // group_rows * nkb, stride, group_rows)
    return _sa_need(nkb, stride, rows)


def dg_route_topk(topk_idx, topk_w, logits, bias=None, n_groups: int = 1, topk_groups: int = 1, group_top: int = 1,
                  score: int = DG_SCORE_SOFTMAX, renorm: bool = False, scale: float = 1.0, stream=None) -> None:
    """The k experts of each token: logits [T,E] (bfloat16 or float32), optional
    float32 bias [E] -> int32 topk_idx [T,k] and float32 topk_w [T,k]."""
    func = "dg_route_topk"
    calls = _calls or _marshal()
    try:
        T, E = logits.shape
        Ti, k = topk_idx.shape
    except (AttributeError, ValueError):
        raise _rank_error(func, logits=logits, topk_idx=topk_idx) from None
    _check_dim(func, "token count of topk_idx", Ti, T)
    dt = _logits_dtype(func, logits)
    kind = _BF16 if dt == DG_DTYPE_BF16 else _F32
    dev = _check_tensors(func, "topk_idx topk_w logits bias",
                         topk_idx, _I32, T * k, topk_w, _F32, T * k, logits, kind, T * E, bias, _F32, E)
    status = calls.dg_route_topk(topk_idx, topk_w, logits, dt, bias, T, E, k, n_groups, topk_groups, group_top,
                                 score, 1 if renorm else 0, scale, _raw_stream(stream, dev))
    if status != DG_OK:
        _check(func, status)


def dg_route_topk_bwd(dlogits, dw, logits, topk_idx, score: int = DG_SCORE_SOFTMAX, renorm: bool = False,
                      scale: float = 1.0, stream=None) -> None:
    """Gradient of dg_route_topk: float32 dw [T,k] -> dlogits [T,E] (the logits' type)."""
    func = "dg_route_topk_bwd"
    calls = _calls or _marshal()
    try:
        T, E = logits.shape
        Ti, k = topk_idx.shape
    except (AttributeError, ValueError):
        raise _rank_error(func, logits=logits, topk_idx=topk_idx) from None
    _check_dim(func, "token count of topk_idx", Ti, T)
    dt = _logits_dtype(func, logits)
    kind = _BF16 if dt == DG_DTYPE_BF16 else _F32
    if isinstance(dlogits, torch.Tensor) and dlogits.dtype != logits.dtype:
        raise DGError(func, DG_ERR_INVALID_ARG, f"dlogits are {dlogits.dtype}, logits {logits.dtype}")
    dev = _check_tensors(func, "dlogits dw logits topk_idx",
                         dlogits, kind, T * E, dw, _F32, T * k, logits, kind, T * E, topk_idx, _I32, T * k)
    status = calls.dg_route_topk_bwd(dlogits, dw, logits, dt, topk_idx, T, E, k, score, 1 if renorm else 0, scale,
                                     _raw_stream(stream, dev))
    if status != DG_OK:
        _check(func, status)


def dg_get_layout_rows(T: int, k: int, E: int) -> int:
    """Rows that dg_route_layout's contiguous form needs for any choice of experts; -1 for sizes it does not take."""
    sizes = [int(x) for x in (T, k, E)]
    if any(abs(x) > 0x7FFFFFFF for x in sizes):  # ctypes would keep the low 32 bits
        return -1
    return int(lib().dg_get_layout_rows(*sizes))


def dg_route_layout(row_of, m_indices, slot_of, group_offsets, counts, topk_idx, max_rows: int = 0,
                    stream=None) -> None:
    """The grouped layout of topk_idx [T,k] (all int32): row_of [T,k],
    m_indices and slot_of [rows], group_offsets [E+1], counts [E]; contiguous,
    or masked with max_rows rows per group."""
    func = "dg_route_layout"
    calls = _calls or _marshal()
    try:
        T, k = topk_idx.shape
    except (AttributeError, ValueError):
        raise _rank_error(func, topk_idx=topk_idx) from None
    rows, E = _shape1(func, "m_indices", m_indices), _shape1(func, "counts", counts)
    dev = _check_tensors(func, "row_of m_indices slot_of group_offsets counts topk_idx",
                         row_of, _I32, T * k, m_indices, _I32, rows, slot_of, _I32, rows, group_offsets, _I32, E + 1,
                         counts, _I32, E, topk_idx, _I32, T * k)
    status = calls.dg_route_layout(row_of, m_indices, slot_of, group_offsets, counts, topk_idx, T, k, E, rows,
                                   max_rows, _raw_stream(stream, dev))
    if status != DG_OK:
        _check(func, status)


def dg_dispatch_fp8_1x128(Q, sa, sa_stride: int, X, row_of, group_rows: int = 0, stream=None) -> None:
    """Cast bf16 X [T,K] into the rows of the layout: e4m3 Q [rows,K] (or
    [G,M_max,K]) and its transposed scales; group_rows = M_max when masked."""
    func = "dg_dispatch_fp8_1x128"
    calls = _calls or _marshal()
    try:
        T, K = X.shape
        Ti, k = row_of.shape
        n, Kq = Q.numel(), Q.shape[-1]
    except (AttributeError, ValueError, TypeError, IndexError):
        raise _rank_error(func, ("Q",), X=X, row_of=row_of, Q=Q) from None
    _check_dim(func, "token count of row_of", Ti, T)
    _check_dim(func, "K of Q", Kq, K)
    rows = n // K if K else 0
    dev = _check_tensors(func, "Q sa X row_of",
                         Q, _U8, rows * K, sa, _F32, _scales_need(_cdiv(K, 128), sa_stride, rows, group_rows),
                         X, _BF16, T * K, row_of, _I32, T * k)
    status = calls.dg_dispatch_fp8_1x128(Q, sa, sa_stride, X, row_of, T, k, K, rows, group_rows,
                                         _raw_stream(stream, dev))
    if status != DG_OK:
        _check(func, status)


def dg_combine(out, Y, row_of, w=None, stream=None) -> None:
    """out [T,N] = sum over slots of w [T,k] (None: ones) times the rows of Y
    ([rows,N] or [G,M_max,N]), bf16; without w the backward pass of the dispatch."""
    func = "dg_combine"
    calls = _calls or _marshal()
    try:
        T, N = out.shape
        Ti, k = row_of.shape
        n, Ny = Y.numel(), Y.shape[-1]
    except (AttributeError, ValueError, TypeError, IndexError):
        raise _rank_error(func, ("Y",), out=out, row_of=row_of, Y=Y) from None
    _check_dim(func, "token count of row_of", Ti, T)
    _check_dim(func, "N of Y", Ny, N)
    rows = n // N if N else 0
    dev = _check_tensors(func, "out Y row_of w",
                         out, _BF16, T * N, Y, _BF16, rows * N, row_of, _I32, T * k, w, _F32, T * k)
    status = calls.dg_combine(out, Y, row_of, w, T, k, N, rows, _raw_stream(stream, dev))
    if status != DG_OK:
        _check(func, status)


def dg_combine_bwd(dw, Qr, sr, sr_stride: int, Qc, sc, sc_stride: int, dout, Y, row_of, slot_of, w,
                   stream=None) -> None:
    """Gradient of dg_combine (contiguous layout): dout [T,N] -> dY [rows,N]
    cast per 1x128 (Qr, sr) and per 128x1 (Qc, sc), and float32 dw [T,k]."""
    func = "dg_combine_bwd"
    calls = _calls or _marshal()
    try:
        T, N = dout.shape
        Ti, k = row_of.shape
        rows, Ny = Y.shape
    except (AttributeError, ValueError):
        raise _rank_error(func, dout=dout, row_of=row_of, Y=Y) from None
    _check_dim(func, "token count of row_of", Ti, T)
    _check_dim(func, "N of Y", Ny, N)
    dev = _check_tensors(func, "dw Qr sr Qc sc dout Y row_of slot_of w",
                         dw, _F32, T * k, Qr, _U8, rows * N, sr, _F32, _sa_need(_cdiv(N, 128), sr_stride, rows),
                         Qc, _U8, rows * N, sc, _F32, _sa_need(_cdiv(rows, 128), sc_stride, N), dout, _BF16, T * N,
                         Y, _BF16, rows * N, row_of, _I32, T * k, slot_of, _I32, rows, w, _F32, T * k)
    status = calls.dg_combine_bwd(dw, Qr, sr, sr_stride, Qc, sc, sc_stride, dout, Y, row_of, slot_of, w, T, k, N,
                                  rows, _raw_stream(stream, dev))
    if status != DG_OK:
        _check(func, status)


def dg_swiglu_fp8(Q, sa, sa_stride: int, H, C=None, cs=None, cs_stride: int = 0, m_indices=None, group_rows: int = 0,
                  stream=None) -> None:
    """silu(gate) * up of bf16 H [rows,2F] (or [G,M_max,2F]) -> e4m3 Q [rows,F]
    and sa; with C and cs also the e4m3 checkpoint of gate and up [rows,2F]."""
    func = "dg_swiglu_fp8"
    calls = _calls or _marshal()
    try:
        n, width, Fq = H.numel(), H.shape[-1], Q.shape[-1]
    except (AttributeError, TypeError, IndexError):
        raise _rank_error(func, ("H", "Q"), H=H, Q=Q) from None
    F = width // 2
    _check_dim(func, "last extent of H", width, 2 * F)
    _check_dim(func, "F of Q", Fq, F)
    rows = n // (2 * F) if F else 0
    dev = _check_tensors(func, "Q sa H C cs m_indices",
                         Q, _U8, rows * F, sa, _F32, _scales_need(_cdiv(F, 128), sa_stride, rows, group_rows),
                         H, _BF16, rows * 2 * F, C, _U8, rows * 2 * F,
                         cs if C is not None else None, _F32, _scales_need(2 * _cdiv(F, 128), cs_stride, rows, group_rows),
                         m_indices, _I32, rows)
    status = calls.dg_swiglu_fp8(Q, sa, sa_stride, C, cs, cs_stride, H, m_indices, rows, F, group_rows,
                                 _raw_stream(stream, dev))
    if status != DG_OK:
        _check(func, status)


def dg_swiglu_fp8_bwd(Qr, sr, sr_stride: int, Qc, sc, sc_stride: int, Qa, sb, dA, C, cs, cs_stride: int,
                      m_indices=None, stream=None) -> None:
    """Backward of dg_swiglu_fp8 from its checkpoint (contiguous layout): bf16
    dA [rows,F] -> dH [rows,2F] cast per 1x128 (Qr, sr) and per 128x1 (Qc, sc),
    and the activation again per 128x128 (Qa [rows,F], sb [F/128, rows/128])."""
    func = "dg_swiglu_fp8_bwd"
    calls = _calls or _marshal()
    try:
        rows, F = dA.shape
        width = C.shape[-1]
    except (AttributeError, ValueError, TypeError, IndexError):
        raise _rank_error(func, ("C",), dA=dA, C=C) from None
    _check_dim(func, "last extent of C", width, 2 * F)
    dev = _check_tensors(func, "Qr sr Qc sc Qa sb dA C cs m_indices",
                         Qr, _U8, rows * 2 * F, sr, _F32, _sa_need(2 * _cdiv(F, 128), sr_stride, rows),
                         Qc, _U8, rows * 2 * F, sc, _F32, _sa_need(_cdiv(rows, 128), sc_stride, 2 * F),
                         Qa, _U8, rows * F, sb, _F32, _cdiv(F, 128) * _cdiv(rows, 128), dA, _BF16, rows * F,
                         C, _U8, rows * 2 * F, cs, _F32, _sa_need(2 * _cdiv(F, 128), cs_stride, rows),
                         m_indices, _I32, rows)
    status = calls.dg_swiglu_fp8_bwd(Qr, sr, sr_stride, Qc, sc, sc_stride, Qa, sb, dA, C, cs, cs_stride, m_indices,
                                     rows, F, _raw_stream(stream, dev))
    if status != DG_OK:
        _check(func, status)


def dg_fp8_1x128_to_128x128(Qb, sb, Q, sa, sa_stride: int, m_indices=None, stream=None) -> None:
    """e4m3 Q [rows,K] with scales per 1x128 -> Qb [rows,K] with scales per
    128x128, sb [K/128, rows/128] (contiguous layout)."""
    func = "dg_fp8_1x128_to_128x128"
    calls = _calls or _marshal()
    try:
        rows, K = Q.shape
    except (AttributeError, ValueError):
        raise _rank_error(func, Q=Q) from None
    dev = _check_tensors(func, "Qb sb Q sa m_indices",
                         Qb, _U8, rows * K, sb, _F32, _cdiv(K, 128) * _cdiv(rows, 128), Q, _U8, rows * K,
                         sa, _F32, _sa_need(_cdiv(K, 128), sa_stride, rows), m_indices, _I32, rows)
    status = calls.dg_fp8_1x128_to_128x128(Qb, sb, Q, sa, sa_stride, m_indices, rows, K, _raw_stream(stream, dev))
    if status != DG_OK:
        _check(func, status)


def _int32_sizes(*sizes) -> bool:
    return all(abs(int(x)) <= 0x7FFFFFFF for x in sizes)  # ctypes would keep the low 32 bits


def dg_fp8_gemm_nt_epilogue(D, A, sa, sa_stride: int, B, sb, bias=None, act: int = DG_ACT_NONE, residual=None, Z=None,
                            Q=None, sq=None, sq_stride: int = 0, stream=None) -> None:
    """z = scaled A[M,K] . B[N,K]^T + bias [N], v = act(z) + residual [M,N]: bf16 D
    (v) and Z (z), and v as e4m3 Q [M,N] with its transposed scales sq (any of
    D, Z, Q may be None, but not all; D may be the residual)."""
    func = "dg_fp8_gemm_nt_epilogue"
    calls = _calls or _marshal()
    try:
        M, K = A.shape
        N, Kb = B.shape
    except (AttributeError, ValueError):
        raise _rank_error(func, A=A, B=B) from None
    _check_dim(func, "K of B", Kb, K)
    nkb, nnb = _cdiv(K, 128), _cdiv(N, 128)
    dev = _check_tensors(func, "D A sa B sb bias residual Z Q sq",
                         D, _BF16, M * N, A, _U8, M * K, sa, _F32, _sa_need(nkb, sa_stride, M), B, _U8, N * K,
                         sb, _F32, nnb * nkb, bias, _F32, N, residual, _BF16, M * N, Z, _BF16, M * N, Q, _U8, M * N,
                         sq if Q is not None else None, _F32, _sa_need(nnb, sq_stride, M))
    status = calls.dg_fp8_gemm_nt_epilogue(D, Z, Q, sq, sq_stride, A, sa, sa_stride, B, sb, bias, act, residual, M, N,
                                           K, _raw_stream(stream, dev))
    if status != DG_OK:
        _check(func, status)


def dg_get_bias_workspace(M: int, N: int) -> int:
    """Floats of dg_epilogue_bwd's workspace; -1 for sizes it does not take."""
    return int(lib().dg_get_bias_workspace(int(M), int(N))) if _int32_sizes(M, N) else -1


def dg_epilogue_bwd(Qr, sr, sr_stride: int, Qc, sc, sc_stride: int, dD, Z=None, act: int = DG_ACT_NONE, dbias=None,
                    ws=None, stream=None) -> None:
    """Gradient of dg_fp8_gemm_nt_epilogue: bf16 dD and Z [M,N] -> dz cast per
    1x128 (Qr [M,N], sr) and per 128x1 (Qc [M rounded up to 128, N], sc), and the
    float32 bias gradient dbias [N]."""
    func = "dg_epilogue_bwd"
    calls = _calls or _marshal()
    try:
        M, N = dD.shape
    except (AttributeError, ValueError):
        raise _rank_error(func, dD=dD) from None
    mb, nb = _cdiv(M, 128), _cdiv(N, 128)
    dev = _check_tensors(func, "Qr sr Qc sc dD Z dbias ws",
                         Qr, _U8, M * N, sr, _F32, _sa_need(nb, sr_stride, M), Qc, _U8, 128 * mb * N,
                         sc, _F32, _sa_need(mb, sc_stride, N), dD, _BF16, M * N,
                         Z if act != DG_ACT_NONE else None, _BF16, M * N, dbias, _F32, N,
                         ws if dbias is not None else None, _F32, mb * N)
    status = calls.dg_epilogue_bwd(Qr, sr, sr_stride, Qc, sc, sc_stride, dbias, ws, dD, Z, act, M, N,
                                   _raw_stream(stream, dev))
    if status != DG_OK:
        _check(func, status)


def _stream_dtype(func: str, *tensors) -> int:
    """Element type of the residual stream: that of the first tensor given."""
    for t in tensors:
        if isinstance(t, torch.Tensor):
            if t.dtype == torch.bfloat16:
                return DG_DTYPE_BF16
            if t.dtype == torch.float32:
                return DG_DTYPE_FP32
            raise DGError(func, DG_ERR_INVALID_ARG, f"the stream is {t.dtype}, the call takes bfloat16 or float32")
    return DG_DTYPE_BF16


def dg_norm_residual(U, X, Y=None, H=None, Q=None, sq=None, sq_stride: int = 0, rstd=None, w_post=None, gate=None,
                     w_pre=None, post_norm: bool = False, scale: float = 1.0, eps: float = 1e-6, stream=None) -> None:
    """u = x + scale * gate[t] * w_post * (norm of) y into U [T,N] (X's type,
    bfloat16 or float32), and h = w_pre * norm of u as bf16 H [T,N] and as e4m3 Q
    [T,N] with its transposed scales sq; float32 rstd [T,2] for the gradient.
    Outputs that are None are left out; X or Y may be None."""
    func = "dg_norm_residual"
    calls = _calls or _marshal()
    try:
        T, N = (X if X is not None else Y).shape
    except (AttributeError, ValueError):
        raise _rank_error(func, **({"X": X} if X is not None else {"Y": Y})) from None
    dt = _stream_dtype(func, X, U)
    kind = _BF16 if dt == DG_DTYPE_BF16 else _F32
    dev = _check_tensors(func, "U X Y H Q sq rstd w_post gate w_pre",
                         U, kind, T * N, X, kind, T * N, Y, _BF16, T * N, H, _BF16, T * N, Q, _U8, T * N,
                         sq if Q is not None else None, _F32, _sa_need(_cdiv(N, 128), sq_stride, T),
                         rstd, _F32, 2 * T, w_post, _F32, N, gate, _F32, T, w_pre, _F32, N)
    status = calls.dg_norm_residual(U, H, Q, sq, sq_stride, rstd, X, dt, Y, w_post, gate, w_pre, T, N,
                                    1 if post_norm else 0, scale, eps, _raw_stream(stream, dev))
    if status != DG_OK:
        _check(func, status)


def dg_get_norm_workspace(T: int, N: int) -> int:
    """Floats of dg_norm_residual_bwd's workspace; -1 for sizes it does not take."""
    return int(lib().dg_get_norm_workspace(int(T), int(N))) if _int32_sizes(T, N) else -1


def dg_norm_residual_bwd(dX, dU, dH, U, Y, rstd, dY=None, dgate=None, dw_post=None, dw_pre=None, ws=None, w_post=None,
                         gate=None, w_pre=None, post_norm: bool = False, scale: float = 1.0, stream=None) -> None:
    """Gradient of dg_norm_residual: dU [T,N] (U's type) and bf16 dH [T,N] (either
    may be None: zeros) -> dX [T,N] (U's type), bf16 dY [T,N], float32 dgate [T],
    dw_post and dw_pre [N] (with ws); outputs that are None are left out."""
    func = "dg_norm_residual_bwd"
    calls = _calls or _marshal()
    try:
        T, N = U.shape
    except (AttributeError, ValueError):
        raise _rank_error(func, U=U) from None
    dt = _stream_dtype(func, U)
    kind = _BF16 if dt == DG_DTYPE_BF16 else _F32
    sums = dw_post is not None or dw_pre is not None
    dev = _check_tensors(func, "dX dU dH U Y rstd dY dgate dw_post dw_pre ws w_post gate w_pre",
                         dX, kind, T * N, dU, kind, T * N, dH, _BF16, T * N, U, kind, T * N, Y, _BF16, T * N,
                         rstd, _F32, 2 * T, dY, _BF16, T * N, dgate, _F32, T, dw_post, _F32, N, dw_pre, _F32, N,
                         ws if sums else None, _F32, max(dg_get_norm_workspace(T, N), 0) if sums else 0,
                         w_post, _F32, N, gate, _F32, T, w_pre, _F32, N)
    status = calls.dg_norm_residual_bwd(dX, dY, dgate, dw_post, dw_pre, ws, dU, dH, U, dt, Y, rstd, w_post, gate, w_pre,
                                        T, N, 1 if post_norm else 0, scale, _raw_stream(stream, dev))
    if status != DG_OK:
        _check(func, status)


def dg_get_balance_workspace(T: int, E: int, S: int = 1) -> int:
    """Floats of dg_balance_loss's workspace; -1 for sizes it does not take."""
    return int(lib().dg_get_balance_workspace(int(T), int(E), int(S))) if _int32_sizes(T, E, S) else -1


def dg_balance_loss(loss, counts, probs, logits, topk_idx, ws, seq_offsets=None, score: int = DG_SCORE_SOFTMAX,
                    coef: float = 1.0, stream=None) -> None:
    """Balance loss of a router: logits [T,E] and int32 topk_idx [T,k] -> float32
    loss [1], int32 counts [S,E] and float32 mean probabilities probs [S,E] (or
    None) of the sequences between int32 seq_offsets [S+1] (None: one of all tokens)."""
    func = "dg_balance_loss"
    calls = _calls or _marshal()
    try:
        T, E = logits.shape
        Ti, k = topk_idx.shape
        S, Ec = counts.shape
    except (AttributeError, ValueError):
        raise _rank_error(func, logits=logits, topk_idx=topk_idx, counts=counts) from None
    _check_dim(func, "token count of topk_idx", Ti, T)
    _check_dim(func, "E of counts", Ec, E)
    dt = _logits_dtype(func, logits)
    kind = _BF16 if dt == DG_DTYPE_BF16 else _F32
    dev = _check_tensors(func, "loss counts probs logits topk_idx ws seq_offsets",
                         loss, _F32, 1, counts, _I32, S * E, probs, _F32, S * E, logits, kind, T * E,
                         topk_idx, _I32, T * k, ws, _F32, max(dg_get_balance_workspace(T, E, S), 0),
                         seq_offsets, _I32, S + 1)
    status = calls.dg_balance_loss(loss, counts, probs, ws, logits, dt, topk_idx, seq_offsets, T, E, k, S, score, coef,
                                   _raw_stream(stream, dev))
    if status != DG_OK:
        _check(func, status)


def dg_balance_loss_bwd(dlogits, logits, counts, k: int, dloss=None, add=None, seq_offsets=None,
                        score: int = DG_SCORE_SOFTMAX, coef: float = 1.0, stream=None) -> None:
    """Gradient of dg_balance_loss with k choices per token: dlogits [T,E] (the
    logits' type) = add [T,E] (or zeros) + float32 dloss [1] (or 1) times the
    loss's gradient; counts [S,E] as the forward call wrote them."""
    func = "dg_balance_loss_bwd"
    calls = _calls or _marshal()
    try:
        T, E = logits.shape
        S, Ec = counts.shape
    except (AttributeError, ValueError):
        raise _rank_error(func, logits=logits, counts=counts) from None
    _check_dim(func, "E of counts", Ec, E)
    dt = _logits_dtype(func, logits)
    kind = _BF16 if dt == DG_DTYPE_BF16 else _F32
    for name, t in (("dlogits", dlogits), ("add", add)):
        if isinstance(t, torch.Tensor) and t.dtype != logits.dtype:
            raise DGError(func, DG_ERR_INVALID_ARG, f"{name} are {t.dtype}, logits {logits.dtype}")
    dev = _check_tensors(func, "dlogits logits counts dloss add seq_offsets",
                         dlogits, kind, T * E, logits, kind, T * E, counts, _I32, S * E, dloss, _F32, 1,
                         add, kind, T * E, seq_offsets, _I32, S + 1)
    status = calls.dg_balance_loss_bwd(dlogits, add, dloss, logits, dt, counts, seq_offsets, T, E, k, S, score, coef,
                                       _raw_stream(stream, dev))
    if status != DG_OK:
        _check(func, status)


def dg_set_pdl(enable) -> None:
    """Programmatic dependent launch on (True), off (False) or default (None: DG_PDL=1)."""
    lib().dg_set_pdl(-1 if enable is None else int(bool(enable)))


def dg_get_pdl() -> bool:
    return bool(lib().dg_get_pdl())


def dg_set_num_sms(n: int) -> None:
    lib().dg_set_num_sms(int(n))


def dg_get_num_sms() -> int:
    return int(lib().dg_get_num_sms())


def dg_get_m_alignment_for_contiguous_layout() -> int:
    return int(lib().dg_get_m_alignment_for_contiguous_layout())


def dg_get_tma_aligned_size(x: int, elem_bytes: int) -> int:
    return int(lib().dg_get_tma_aligned_size(int(x), int(elem_bytes)))


def dg_get_device_error() -> int:
    code = ctypes.c_int(0)
    _check("dg_get_device_error", lib().dg_get_device_error(ctypes.byref(code)))
    return int(code.value)


def dg_get_workspace_count() -> int:
    return int(lib().dg_get_workspace_count())


def dg_make_plan(mode: int, rows: int, N: int, K: int, G: int, num_sms: int) -> dict:
    pl = Plan()
    _check("dg_make_plan", lib().dg_make_plan(int(mode), int(rows), int(N), int(K), int(G), int(num_sms),
                                              ctypes.byref(pl)))
    return pl.as_dict()


def dg_make_plan_ue8m0(M: int, N: int, K: int, num_sms: int) -> dict:
    pl = Plan()
    _check("dg_make_plan_ue8m0", lib().dg_make_plan_ue8m0(int(M), int(N), int(K), int(num_sms), ctypes.byref(pl)))
    return pl.as_dict()


def dg_selftest_bounded_wait(stream=None) -> None:
    """Enqueue the bounded-wait self-test kernel (sets DG_DEVERR_TIMEOUT after ~1 s)."""
    _check("dg_selftest_bounded_wait", lib().dg_selftest_bounded_wait(_stream(stream)))


def dg_status_string(status: int) -> str:
    return lib().dg_status_string(int(status)).decode()


def dg_get_col_major_tma_aligned_tensor(s):
    """[M, nkb] (or [G, M, nkb]) float32 scales -> (flat transposed TMA-aligned tensor, sa_stride).

    Layout helper for callers (the pages' get_col_major_tma_aligned_tensor);
    runs as torch tensor ops outside the timed path."""
    _need_torch()
    grouped = s.dim() == 3
    s3 = s if grouped else s.unsqueeze(0)
    G, M, nkb = s3.shape
    stride = dg_get_tma_aligned_size(M, 4)
    out = torch.zeros(G, nkb, stride, dtype=torch.float32, device=s.device)
    out[:, :, :M] = s3.transpose(1, 2)
    return out.reshape(-1).contiguous(), stride
