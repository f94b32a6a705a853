"""Residual binarized weights on AMD Instinct MI355X: Python face of librb.

Thin wrappers over the C ABI in include/rb.h. PyTorch provides device buffers and the
current HIP stream; every computation runs in librb's HIP kernels. Functions take and
return CUDA (HIP) tensors on the current device and enqueue on the current stream.

  planes, g = pack(W, k)                         residual sign planes + row scales
  y = gemv(planes, g, h, x, K)                   y = sum_i g_i (.) (B_i (h_i (.) x)), M <= 16
  y = gemm_small(planes, g, h, x, K)             same on the matrix cores, larger M
  y = gemv_variant(planes, g, h, x, K, mu=, zero_one=)   {0, s} planes / per-row offset
  idx = codebook_encode(sign_plane, K, C, v)     nearest binary codeword per v-block
  y = codebook_gemv(idx, C, v, s, group, x, K)   product on codebook indices
  C, idx, M = codebook_learn(sign_plane, K, C0, v, iters)   binary K-means codebook learning
  planes, g, h = svid_init(W, k)                 function-aware initialization of k paths
  planes, What = qat_derive(W, g, h)             coupled training: paths derived from W
  Y, planes, What = qat_forward(W, g, h, X)      ... and the layer's product Y = X What^T
  dW, dX, dg, dh = qat_backward(dY, X, What, planes, g, h)   straight-through backward
  qat_autotune(X, dY, What, Y, dW, dX)           pick the fastest GEMM kernels for a shape
  Y, Z = qat_linear(X, What, bias, act, residual)   Y = act(X What^T + bias) + residual
  dZ, db = qat_linear_backward(dY, Z, act)       ... and its epilogue's gradients
  S, X, stats = resnorm_forward(Y, R, w_pre)     S = alpha R + gate norm_post(Y), X = norm_pre(S)
  grads = resnorm_backward(dX, dS, Y, S, stats, w_pre)   ... and its gradients
  adamw_step(plan, step, lr)                     AdamW over many tensors (adamw_plan), states in 32 or 8 bits
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from ._lib import (RB_F16, RB_F32, RB_BF16, RB_OP_CODEBOOK_GEMV, RB_OP_GEMM_SMALL, RB_OP_GEMV,
                   RB_OP_QAT_BACKWARD, RB_OP_QAT_LINEAR, RB_OP_QAT_LINEAR_BACKWARD, RB_OP_RESNORM_BACKWARD, RB_OP_SVID_INIT, RB_QAT_ENGINE_AUTO, RB_QAT_ENGINE_MFMA,
                   RB_QAT_ENGINE_ROCBLAS, RbError, check, lib)

__all__ = ["pack", "gemv", "gemv_variant", "gemm_small", "codebook_encode", "codebook_gemv", "codebook_mstep",
           "codebook_distinct", "codebook_learn", "svid_init", "qat_derive",
           "qat_forward", "qat_matmul", "qat_backward", "qat_autotune", "qat_linear", "qat_linear_backward", "resnorm_forward",
           "resnorm_backward", "adamw_plan", "adamw_step", "AdamWPlan", "workspace",
           "workspace_bytes", "storage_bits_per_weight", "version", "RbError", "lib"]

_DT = {torch.float32: RB_F32, torch.float16: RB_F16, torch.bfloat16: RB_BF16}


def _dt(t: torch.dtype) -> int:
    if t not in _DT:
        raise TypeError(f"unsupported dtype {t}")
    return _DT[t]


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("librb takes device tensors")
    if not t.is_contiguous():
        raise ValueError("librb takes contiguous tensors")
    return t.data_ptr()


def _ptr_rows(t: torch.Tensor | None):
    """A matrix whose rows may be strided (unit stride within a row; the row stride is passed
    to the library as the leading dimension)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("librb takes device tensors")
    if t.dim() < 1 or t.stride(-1) != 1 or any(t.stride(d) < 0 for d in range(t.dim())):
        raise ValueError("librb takes matrices with unit stride along rows")
    if t.dim() == 3 and t.stride(0) != t.shape[1] * t.stride(1):
        raise ValueError("librb takes plane stacks with planes stored back to back")
    return t.data_ptr()


# the handle alone costs a tenth of what a Stream object does (0.3 against 2.8 us per call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream():
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch.cuda.current_device())


def version() -> int:
    return lib.rb_version()


def workspace_bytes(op: int, k: int, N: int, K: int, M: int) -> int:
    return int(lib.rb_workspace_bytes(op, k, N, K, M))


def storage_bits_per_weight(N: int, K: int, k: int, scale_dtype=torch.float16, has_h: bool = True) -> float:
    return float(lib.rb_storage_bits_per_weight(N, K, k, _dt(scale_dtype), int(has_h)))


def workspace(op: int, k: int, N: int, K: int, M: int, device=None) -> torch.Tensor | None:
    """A zero-filled workspace for the given operation (None when it needs none)."""
    n = workspace_bytes(op, k, N, K, M)
    if n == 0:
        return None
    return torch.zeros((n + 15) // 16 * 16, dtype=torch.uint8, device=device or "cuda")


def pack(W: torch.Tensor, k: int, h: torch.Tensor | None = None, group: int = 0,
         scale_dtype=torch.float16, ldp: int | None = None, planes: torch.Tensor | None = None,
         d_status: torch.Tensor | None = None):
    """Residual sign planes (int32 storage of the uint32 words, [k][N][ldp]) and scales
    ([k][N] or [k][N][ceil(K/group)]) of W [N][K] (fp32/fp16/bf16)."""
    N, K = W.shape
    Kw = (K + 31) // 32
    ldp = Kw if ldp is None else ldp
    if planes is None:
        planes = torch.zeros((k, N, ldp), dtype=torch.int32, device=W.device)
    shape = (k, N) if group == 0 else (k, N, (K + group - 1) // group)
    g = torch.empty(shape, dtype=scale_dtype, device=W.device)
    check("rb_pack", lib.rb_pack(_ptr(W), _dt(W.dtype), N, K, W.stride(0), k, group, _ptr(h),
                                 _dt(scale_dtype), _ptr(planes), ldp, _ptr(g), _ptr(d_status),
                                 _stream()))
    return planes, g


def _product(fn_name: str, planes, g, h, x, K, y_dtype, ws, y, op):
    k, N, ldp = planes.shape
    M = x.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=y_dtype, device=x.device)
    if ws is None:
        ws = workspace(op, k, N, K, M, device=x.device)
    fn = getattr(lib, fn_name)
    check(fn_name, fn(_ptr(planes), ldp, _ptr(g), _ptr(h), _dt(g.dtype), k, N, K, _ptr(x),
                      _dt(x.dtype), M, _ptr(y), _dt(y.dtype), _ptr(ws),
                      0 if ws is None else ws.numel(), _stream()))
    return y


def gemv(planes, g, h, x, K: int, y_dtype=torch.float16, ws=None, y=None):
    """y [M][N] = sum_i g_i (.) (B_i (h_i (.) x)) for x [M][K], M <= 16."""
    return _product("rb_gemv", planes, g, h, x, K, y_dtype, ws, y, RB_OP_GEMV)


def gemv_variant(planes, g, h, x, K: int, mu=None, zero_one: bool = False, y_dtype=torch.float16, ws=None,
                 y=None):
    """rb_gemv with {0, 1} planes (zero_one) and/or a per-row offset mu [N] (scale dtype, h None)."""
    k, N, ldp = planes.shape
    M = x.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=y_dtype, device=x.device)
    if ws is None:
        ws = workspace(RB_OP_GEMV, k, N, K, M, device=x.device)
    check("rb_gemv_variant", lib.rb_gemv_variant(_ptr(planes), ldp, _ptr(g), _ptr(h), _ptr(mu), int(zero_one),
                                                 _dt(g.dtype), k, N, K, _ptr(x), _dt(x.dtype), M, _ptr(y),
                                                 _dt(y.dtype), _ptr(ws), 0 if ws is None else ws.numel(),
                                                 _stream()))
    return y


def gemm_small(planes, g, h, x, K: int, y_dtype=torch.float16, ws=None, y=None):
    """Same product on the matrix cores, for larger batches (x fp16)."""
    return _product("rb_gemm_small", planes, g, h, x, K, y_dtype, ws, y, RB_OP_GEMM_SMALL)


def codebook_encode(sign_plane: torch.Tensor, K: int, codebook: torch.Tensor, v: int, table: bool = False,
                    ws: torch.Tensor | None = None):
    """uint16 indices (int16 storage) [N][ceil(K/v)] of the nearest codewords; with table=True
    through the nearest-codeword table of all 2^v patterns (v <= 24; same result)."""
    N, ldp = sign_plane.shape
    nb = (K + v - 1) // v
    idx = torch.empty((N, nb), dtype=torch.int16, device=sign_plane.device)
    if not table:
        check("rb_codebook_encode", lib.rb_codebook_encode(_ptr(sign_plane), ldp, N, K, _ptr(codebook),
                                                           codebook.numel(), v, _ptr(idx), _stream()))
        return idx
    if ws is None:
        ws = torch.empty(max(4, lib.rb_codebook_table_bytes(v)), dtype=torch.uint8, device=sign_plane.device)
    check("rb_codebook_encode_table", lib.rb_codebook_encode_table(_ptr(sign_plane), ldp, N, K, _ptr(codebook),
                                                                   codebook.numel(), v, _ptr(idx), _ptr(ws),
                                                                   ws.numel(), _stream()))
    return idx


def codebook_gemv(idx, codebook, v: int, s, group: int, x, K: int, ws=None, y=None):
    N = idx.shape[0]
    M = x.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=x.device)
    if ws is None:
        ws = workspace(RB_OP_CODEBOOK_GEMV, 1, N, K, M, device=x.device)
    check("rb_codebook_gemv", lib.rb_codebook_gemv(_ptr(idx), _ptr(codebook), codebook.numel(), v,
                                                   _ptr(s), group, N, K, _ptr(x), M, _ptr(y),
                                                   _ptr(ws), 0 if ws is None else ws.numel(),
                                                   _stream()))
    return y


def _learn_ws(N: int, K: int, c: int, v: int, device, ws):
    if ws is None:
        ws = torch.empty(max(4, lib.rb_codebook_learn_workspace_bytes(N, K, c, v)), dtype=torch.uint8, device=device)
    return ws


def codebook_mstep(sign_plane: torch.Tensor, K: int, idx: torch.Tensor, codebook: torch.Tensor, v: int,
                   counts: bool = True, ws: torch.Tensor | None = None):
    """One M-step of binary K-means, in place on `codebook` ([c] int32 storage of the words);
    returns the member count per codeword ([c] int32 storage) or None."""
    N, ldp = sign_plane.shape
    c = codebook.numel()
    cnt = torch.empty(c, dtype=torch.int32, device=codebook.device) if counts else None
    ws = _learn_ws(N, K, c, v, codebook.device, ws)
    check("rb_codebook_mstep", lib.rb_codebook_mstep(_ptr(sign_plane), ldp, N, K, v, _ptr(idx), _ptr(codebook), c,
                                                     _ptr(cnt), _ptr(ws), ws.numel(), _stream()))
    return cnt


def codebook_distinct(sign_plane: torch.Tensor, K: int, codebook: torch.Tensor, v: int,
                      ws: torch.Tensor | None = None) -> torch.Tensor:
    """Number of distinct v-column blocks (a device int32 tensor); if below the codebook size,
    the codebook (in place) becomes those blocks in ascending order."""
    N, ldp = sign_plane.shape
    c = codebook.numel()
    nd = torch.empty(1, dtype=torch.int32, device=codebook.device)
    ws = _learn_ws(N, K, c, v, codebook.device, ws)
    check("rb_codebook_distinct", lib.rb_codebook_distinct(_ptr(sign_plane), ldp, N, K, v, _ptr(codebook), c,
                                                           _ptr(nd), _ptr(ws), ws.numel(), _stream()))
    return nd


def codebook_learn(sign_plane: torch.Tensor, K: int, codebook: torch.Tensor, v: int, iters: int,
                   idx: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """Binary K-means from the initial `codebook` (updated in place): returns (codebook, idx
    [N][ceil(K/v)] uint16 as int16 storage, number of distinct blocks as a device int32)."""
    N, ldp = sign_plane.shape
    c = codebook.numel()
    nb = (K + v - 1) // v
    idx = torch.empty((N, nb), dtype=torch.int16, device=codebook.device) if idx is None else idx
    nd = torch.empty(1, dtype=torch.int32, device=codebook.device)
    ws = _learn_ws(N, K, c, v, codebook.device, ws)
    check("rb_codebook_learn", lib.rb_codebook_learn(_ptr(sign_plane), ldp, N, K, v, _ptr(codebook), c, iters,
                                                     _ptr(idx), _ptr(nd), _ptr(ws), ws.numel(), _stream()))
    return codebook, idx, nd


def svid_init(W: torch.Tensor, k: int, T: int = 20, P: int = 4, s_in: torch.Tensor | None = None,
              s_out: torch.Tensor | None = None, a_in: float = 0.0, a_out: float = 0.0,
              ldp: int | None = None, ws: torch.Tensor | None = None):
    """Function-aware initialization of k residual paths of W [N][K] (fp32, row stride a
    multiple of 4): sign planes [k][N][ldp] (int32 storage of the uint32 words) and fp32 scales
    g [k][N], h [k][K], after T Gauss-Seidel sweeps of residual SVID with P power iterations
    per path update; s_in [K] / s_out [N] (fp32, > 0) are the I/O importance vectors."""
    N, K = W.shape
    Kw = (K + 31) // 32
    ldp = Kw if ldp is None else ldp
    if K % 4 != 0 or not W.is_contiguous():
        # rows of a multiple of 4 floats (16-byte rows), as the entry point requires
        Wp = torch.zeros((N, (K + 3) // 4 * 4), dtype=W.dtype, device=W.device)
        Wp[:, :K] = W
        W = Wp
    planes = torch.zeros((k, N, ldp), dtype=torch.int32, device=W.device)
    g = torch.empty((k, N), dtype=torch.float32, device=W.device)
    h = torch.empty((k, K), dtype=torch.float32, device=W.device)
    if ws is None:
        ws = torch.empty((workspace_bytes(RB_OP_SVID_INIT, k, N, K, 1) + 15) // 16 * 16, dtype=torch.uint8,
                         device=W.device)
    check("rb_svid_init", lib.rb_svid_init(_ptr(W), _dt(W.dtype), N, K, W.stride(0), k, T, P, _ptr(s_in),
                                           _ptr(s_out), a_in, a_out, _ptr(planes), ldp, _ptr(g), _ptr(h),
                                           _ptr(ws), ws.numel(), _stream()))
    return planes, g, h


def qat_derive(W: torch.Tensor, g: torch.Tensor, h: torch.Tensor, a_dtype=torch.bfloat16,
               planes: torch.Tensor | None = None, What: torch.Tensor | None = None):
    """Coupled-training derivation: from the shared fp32 weight W [N][K] (rows may be strided)
    and fp32 scales g [k][N], h [k][K], the k sign planes [k][N][ceil(K/32)] (int32 storage)
    and the effective weight What [N][K] in a_dtype (fp16 or bf16)."""
    N, K = W.shape
    k = g.shape[0]
    planes = torch.zeros((k, N, (K + 31) // 32), dtype=torch.int32, device=W.device) if planes is None else planes
    What = torch.empty((N, K), dtype=a_dtype, device=W.device) if What is None else What
    check("rb_qat_derive", lib.rb_qat_derive(_ptr_rows(W), N, K, W.stride(0), k, _ptr(g), _ptr(h), _ptr_rows(planes),
                                             planes.stride(1), _ptr_rows(What), _dt(What.dtype), What.stride(0),
                                             _stream()))
    return planes, What


def qat_forward(W: torch.Tensor, g: torch.Tensor, h: torch.Tensor, X: torch.Tensor, y_dtype=None,
                planes: torch.Tensor | None = None, What: torch.Tensor | None = None,
                Y: torch.Tensor | None = None):
    """Coupled-training forward: the derivation, then Y [M][N] = X What^T for X [M][K] (fp16 or
    bf16, rows may be strided); y_dtype fp32 or X's type (default). Returns (Y, planes, What)."""
    N, K = W.shape
    M = X.shape[0]
    k = g.shape[0]
    planes = torch.zeros((k, N, (K + 31) // 32), dtype=torch.int32, device=W.device) if planes is None else planes
    What = torch.empty((N, K), dtype=X.dtype, device=W.device) if What is None else What
    Y = torch.empty((M, N), dtype=y_dtype or X.dtype, device=W.device) if Y is None else Y
    check("rb_qat_forward", lib.rb_qat_forward(_ptr_rows(W), N, K, W.stride(0), k, _ptr(g), _ptr(h), _ptr_rows(X),
                                               _dt(X.dtype), M, X.stride(0), _ptr_rows(planes), planes.stride(1),
                                               _ptr_rows(What), What.stride(0), _ptr_rows(Y), _dt(Y.dtype), Y.stride(0),
                                               _stream()))
    return Y, planes, What


def qat_matmul(X: torch.Tensor, What: torch.Tensor, Y: torch.Tensor | None = None, y_dtype=None,
               engine: int = RB_QAT_ENGINE_AUTO):
    """The coupled-training forward's product alone: Y [M][N] = X What^T for X [M][K] and What
    [N][K] (fp16 or bf16, rows may be strided), Y fp32 or the operand type (default), on
    `engine` (RB_QAT_ENGINE_AUTO, _MFMA: the library's matrix-core kernel, _ROCBLAS)."""
    M, K = X.shape
    N = What.shape[0]
    Y = torch.empty((M, N), dtype=y_dtype or X.dtype, device=X.device) if Y is None else Y
    check("rb_qat_matmul", lib.rb_qat_matmul(_ptr_rows(X), _dt(X.dtype), M, X.stride(0), _ptr_rows(What),
                                             What.stride(0), N, K, _ptr_rows(Y), _dt(Y.dtype), Y.stride(0), engine,
                                             _stream()))
    return Y


def qat_backward(dY: torch.Tensor, X: torch.Tensor, What: torch.Tensor, planes: torch.Tensor, g: torch.Tensor,
                 h: torch.Tensor, dx_dtype=None, ws: torch.Tensor | None = None, dW: torch.Tensor | None = None,
                 dX: torch.Tensor | None = None, dg: torch.Tensor | None = None, dh: torch.Tensor | None = None):
    """Coupled-training backward from dY [M][N]: dW = dY^T X (fp32 [N][K]), dX = dY What
    ([M][K], dx_dtype fp32 or the activation type), dg [k][N] and dh [k][K] (fp32)."""
    M, N = dY.shape
    K = X.shape[1]
    k = g.shape[0]
    dev = dY.device
    dW = torch.empty((N, K), dtype=torch.float32, device=dev) if dW is None else dW
    dX = torch.empty((M, K), dtype=dx_dtype or X.dtype, device=dev) if dX is None else dX
    dg = torch.empty((k, N), dtype=torch.float32, device=dev) if dg is None else dg
    dh = torch.empty((k, K), dtype=torch.float32, device=dev) if dh is None else dh
    if ws is None:
        ws = torch.empty(max(16, workspace_bytes(RB_OP_QAT_BACKWARD, k, N, K, M)), dtype=torch.uint8, device=dev)
    check("rb_qat_backward", lib.rb_qat_backward(_ptr_rows(dY), _dt(dY.dtype), M, dY.stride(0), _ptr_rows(X), X.stride(0),
                                                 _ptr_rows(What), What.stride(0), _ptr_rows(planes), planes.stride(1),
                                                 _ptr(g), _ptr(h), k, N, K, _ptr_rows(dW), dW.stride(0), _ptr_rows(dX),
                                                 _dt(dX.dtype), dX.stride(0), _ptr(dg), _ptr(dh), _ptr(ws),
                                                 ws.numel(), _stream()))
    return dW, dX, dg, dh


def qat_autotune(X: torch.Tensor, dY: torch.Tensor, What: torch.Tensor, Y: torch.Tensor, dW: torch.Tensor,
                 dX: torch.Tensor):
    """Time the GEMM kernels rocBLAS offers for this layer shape on these buffers and keep the
    fastest for later qat_forward / qat_backward calls of the same shape (synchronising; Y, dW
    and dX are overwritten)."""
    M, K = X.shape
    N = What.shape[0]
    check("rb_qat_autotune", lib.rb_qat_autotune(_ptr_rows(X), _ptr_rows(dY), _dt(X.dtype), M, X.stride(0),
                                                 dY.stride(0), _ptr_rows(What), What.stride(0), N, K, _ptr_rows(Y),
                                                 _dt(Y.dtype), Y.stride(0), _ptr_rows(dW), dW.stride(0),
                                                 _ptr_rows(dX), _dt(dX.dtype), dX.stride(0), _stream()))



_ACT = {"none": _lib.RB_ACT_NONE, "relu": _lib.RB_ACT_RELU, "gelu": _lib.RB_ACT_GELU,
        "gelu_tanh": _lib.RB_ACT_GELU_TANH, "silu": _lib.RB_ACT_SILU}


def _vec(name: str, t: torch.Tensor | None, n: int):
    """A contiguous fp32 device vector of n elements, or None."""
    if t is None:
        return None
    if t.dtype is not torch.float32 or t.numel() != n:
        raise ValueError(f"{name} is an fp32 vector of {n} elements")
    return _ptr(t)


def _rows(name: str, t: torch.Tensor | None, M: int, N: int, dtype):
    """(pointer, row stride) of an M x N matrix of this type, or (None, 0)."""
    if t is None:
        return None, 0
    if t.dtype is not dtype or t.shape != (M, N):
        raise ValueError(f"{name} is a {dtype} matrix of shape {(M, N)}")
    if not t.is_cuda:
        raise ValueError("librb takes device tensors")
    if t.is_contiguous():
        return t.data_ptr(), N
    ld, step = t.stride()
    if (step != 1 and N > 1) or (ld < N and M > 1):
        raise ValueError("librb takes matrices with unit stride along rows")
    return t.data_ptr(), ld if M > 1 else max(ld, N)


@functools.lru_cache(maxsize=4096)
def _ws_bytes(op: int, N: int, K: int, M: int) -> int:
    return workspace_bytes(op, 1, N, K, M)


def qat_linear(X: torch.Tensor, What: torch.Tensor, bias: torch.Tensor | None = None, act: str = "none",
               residual: torch.Tensor | None = None, y_dtype=None, save_z: bool = False,
               Y: torch.Tensor | None = None, Z: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """The layer's product with its epilogue: Z = X What^T + bias, Y = act(Z) + residual, for X [M][K]
    and What [N][K] (fp16 or bf16, rows may be strided), an fp32 `bias` [N], `act` one of "none",
    "relu", "gelu", "gelu_tanh", "silu" and a `residual` [M][N] in Y's type (fp32 or X's, the default;
    it may be Y itself). Returns (Y, Z); Z, in X's type, is kept for the backward if `save_z` or
    given, else None."""
    M, K = X.shape
    N = What.shape[0]
    dt = X.dtype
    if Y is None:
        Y = torch.empty((M, N), dtype=y_dtype or (dt if residual is None else residual.dtype), device=X.device)
    if Z is None and save_z:
        Z = torch.empty((M, N), dtype=dt, device=X.device)
    n = _ws_bytes(RB_OP_QAT_LINEAR, N, K, M)
    if ws is None and n:
        ws = torch.empty(n, dtype=torch.uint8, device=X.device)
    xp, ldx = _rows("X", X, M, K, dt)
    wp, ldw = _rows("What", What, N, K, dt)
    yp, ldy = _rows("Y", Y, M, N, Y.dtype)
    rp, ldr = _rows("residual", residual, M, N, Y.dtype)
    zp, ldz = _rows("Z", Z, M, N, dt)
    check("rb_qat_linear", lib.rb_qat_linear(xp, _dt(dt), M, ldx, wp, ldw, N, K, _vec("bias", bias, N), _ACT[act], rp, ldr,
                                             zp, ldz, yp, _dt(Y.dtype), ldy, _ptr(ws), 0 if ws is None else ws.numel(),
                                             _stream()))
    return Y, Z


def qat_linear_backward(dY: torch.Tensor, Z: torch.Tensor | None, act: str = "none", bias: bool = True, a_dtype=None,
                        dZ: torch.Tensor | None = None, db: torch.Tensor | None = None,
                        ws: torch.Tensor | None = None):
    """The epilogue's gradients from dY [M][N] (fp32 or the activation type) and the forward's Z (not
    needed for act "none"): (dZ, db), dZ = dY act'(Z) in the activation type (Z's, or `a_dtype`; what
    qat_backward takes as its dY) and, with `bias`, db = its column sums, fp32 [N]."""
    M, N = dY.shape
    dt = a_dtype or (Z.dtype if Z is not None else dZ.dtype if dZ is not None else dY.dtype)
    if dZ is None:
        dZ = torch.empty((M, N), dtype=dt, device=dY.device)
    if not bias:
        db = None
    elif db is None:
        db = torch.empty(N, dtype=torch.float32, device=dY.device)
    n = _ws_bytes(RB_OP_QAT_LINEAR_BACKWARD, N, 1, M)
    if ws is None and bias and n:
        ws = torch.empty(n, dtype=torch.uint8, device=dY.device)
    dyp, lddy = _rows("dY", dY, M, N, dY.dtype)
    zp, ldz = _rows("Z", Z, M, N, dt)
    dzp, lddz = _rows("dZ", dZ, M, N, dt)
    check("rb_qat_linear_backward", lib.rb_qat_linear_backward(dyp, _dt(dY.dtype), M, N, lddy, zp, _dt(dt), ldz, _ACT[act],
                                                               dzp, lddz, _vec("db", db, N), _ptr(ws),
                                                               0 if ws is None else ws.numel(), _stream()))
    return dZ, db


_NORM = {"none": _lib.RB_NORM_NONE, "rms": _lib.RB_NORM_RMS, "layer": _lib.RB_NORM_LAYER}


def _gate_rows(gate, M: int, D: int, dtype):
    """(pointer, row stride) of a gate: an fp32 vector (stride 0) or rows."""
    if gate is not None and gate.dim() == 1:
        return _vec("gate", gate, D), 0
    return _rows("gate", gate, M, D, dtype)


def resnorm_forward(Y: torch.Tensor, R: torch.Tensor | None, w_pre: torch.Tensor | None, w_post=None, b_pre=None,
                    b_post=None, gate=None, alpha: float = 1.0, eps: float = 1e-6, pre: str = "rms",
                    post: str | None = None, S: torch.Tensor | None = None, X: torch.Tensor | None = None,
                    stats: torch.Tensor | None = None):
    """Between two blocks: S = alpha R + gate * norm_post(Y), X = norm_pre(S). Y [M][D] is the block's
    output, R [M][D] the stream (Y's type or fp32; None: no residual), `gate` an fp32 vector [D], rows
    [M][D] of Y's type or None; `pre` and `post` name the norms ("none", "rms", "layer"; post
    defaults to "rms" where w_post is given), w_* and b_* are fp32 [D]. Returns (S, X, stats): S in
    R's type, X in Y's (None for pre "none", which takes no X), stats [M][4] fp32 for the backward."""
    M, D = Y.shape
    post = post or ("none" if w_post is None else "rms")
    sdt = R.dtype if R is not None else S.dtype if S is not None else Y.dtype
    if S is None:
        S = torch.empty((M, D), dtype=sdt, device=Y.device)
    if X is None and pre != "none":
        X = torch.empty((M, D), dtype=Y.dtype, device=Y.device)
    if stats is None:
        stats = torch.empty((M, 4), dtype=torch.float32, device=Y.device)
    dt = Y.dtype
    yp, ldy = _rows("Y", Y, M, D, dt)
    rp, ldr = _rows("R", R, M, D, sdt)
    gp, ldg = _gate_rows(gate, M, D, dt)
    sp, lds = _rows("S", S, M, D, sdt)
    xp, ldx = _rows("X", X, M, D, dt)
    check("rb_resnorm_forward", lib.rb_resnorm_forward(
        yp, _dt(dt), M, D, ldy, rp, _dt(sdt), ldr, gp, ldg, alpha, _NORM[post], _vec("w_post", w_post, D),
        _vec("b_post", b_post, D), _NORM[pre], _vec("w_pre", w_pre, D), _vec("b_pre", b_pre, D), eps, sp, lds, xp, ldx,
        _vec("stats", stats, 4 * M), _stream()))
    return S, X, stats


def resnorm_backward(dX: torch.Tensor | None, dS: torch.Tensor | None, Y: torch.Tensor, S: torch.Tensor,
                     stats: torch.Tensor, w_pre: torch.Tensor | None, w_post=None, b_post=None, gate=None,
                     alpha: float = 1.0, pre: str = "rms", post: str | None = None, bias: bool = False,
                     dY: torch.Tensor | None = None, dR: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                     out: dict | None = None):
    """Gradients of resnorm_forward's inputs from those of X (dX; None for pre "none") and S (dS; None: zero), in a dict:
    dY, dR, dgate (like the gate), dw_pre, dw_post and, with `bias`, db_pre, db_post (fp32 [D]); None
    where there is no such input. `out` holds buffers for any of the vectors' or the gate's gradients, by
    these names. Other arguments as in the forward call."""
    M, D = Y.shape
    dev, dt, sdt = Y.device, Y.dtype, S.dtype
    post = post or ("none" if w_post is None else "rms")
    has_pre, has_post = pre != "none", post != "none"
    if dY is None:
        dY = torch.empty((M, D), dtype=dt, device=dev)
    if dR is None:
        dR = torch.empty((M, D), dtype=sdt, device=dev)
    # the vectors' gradients that are not given lie in one buffer
    names = [n for n, there in (("dw_pre", has_pre), ("db_pre", has_pre and bias), ("dw_post", has_post),
                                ("db_post", has_post and bias), ("dgate", gate is not None and gate.dim() == 1)) if there]
    vec = dict(zip(names, torch.empty((len(names), D), dtype=torch.float32, device=dev).unbind(0))) if names else {}
    given, out = out, {"dY": dY, "dR": dR, "dgate": None, "dw_pre": None, "dw_post": None, "db_pre": None,
                       "db_post": None, **vec}
    if gate is not None and gate.dim() != 1 and not (given and "dgate" in given):
        out["dgate"] = torch.empty((M, D), dtype=dt, device=dev)
    for k, t in (given or {}).items():
        if k == "dgate" and gate is not None and gate.dim() != 1:
            _rows(k, t, M, D, dt)
        elif k not in vec:
            raise ValueError(f"there is no gradient {k} to write")
        else:
            _vec(k, t, D)
        out[k] = t
    if ws is None:
        ws = torch.empty(_ws_bytes(RB_OP_RESNORM_BACKWARD, D, 1, M), dtype=torch.uint8, device=dev)
    dxp, lddx = _rows("dX", dX, M, D, dt)
    dsp, ldds = _rows("dS", dS, M, D, sdt)
    yp, ldy = _rows("Y", Y, M, D, dt)
    sp, lds = _rows("S", S, M, D, sdt)
    gp, ldg = _gate_rows(gate, M, D, dt)
    dyp, lddy = _rows("dY", dY, M, D, dt)
    drp, lddr = _rows("dR", dR, M, D, sdt)
    dg, lddg = out["dgate"], D
    if dg is not None and dg.dim() == 2:
        dg, lddg = _rows("dgate", dg, M, D, dt)
    else:
        dg = _ptr(dg)
    check("rb_resnorm_backward", lib.rb_resnorm_backward(
        dxp, _dt(dt), M, D, lddx, dsp, _dt(sdt), ldds, yp, ldy, sp, lds, _vec("stats", stats, 4 * M), gp, ldg, alpha,
        _NORM[post], _vec("w_post", w_post, D), _vec("b_post", b_post, D), _NORM[pre], _vec("w_pre", w_pre, D), dyp,
        lddy, drp, lddr, dg, lddg, _ptr(out["dw_post"]), _ptr(out["db_post"]), _ptr(out["dw_pre"]),
        _ptr(out["db_pre"]), _ptr(ws), ws.numel(), _stream()))
    return out


class AdamWPlan:
    """The tensors of an optimizer, as adamw_step reads them: keeps the parameters, gradients and
    states alive and their table on the device. m, v (and m_scale, v_scale with 8-bit states) are
    lists in the parameters' order."""

    def __init__(self, params, grads, state_bits, m, v, m_scale, v_scale, table, chunks):
        self.params, self.grads, self.state_bits = params, grads, state_bits
        self.m, self.v, self.m_scale, self.v_scale = m, v, m_scale, v_scale
        self.table, self.chunks = table, chunks


def adamw_plan(params, grads, state_bits: int = 32, m=None, v=None, m_scale=None, v_scale=None, weight_decay=0.0,
               lr_mult=1.0) -> AdamWPlan:
    """Lay out one AdamW step over `params` and their `grads` (lists of contiguous device tensors,
    fp32 / fp16 / bf16). States are made, zero, unless given: fp32 with state_bits 32, with 8
    torch.float8_e4m3fn (m, and sqrt(v) in v) and an fp32 scale per 256 elements. `weight_decay` and
    `lr_mult` are numbers or lists of one per tensor. The gradients are read from these tensors at
    every step: write new ones into them."""
    params, grads, n = list(params), list(grads), len(params)
    if state_bits not in (8, 32):
        raise ValueError("state_bits must be 8 or 32")
    if n == 0:
        raise ValueError("adamw_plan needs a tensor at least")
    sdt = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
    each = lambda x: list(x) if isinstance(x, (list, tuple)) else [x] * n  # noqa: E731
    wd, lm = each(weight_decay), each(lr_mult)
    m = [torch.zeros(p.shape, dtype=sdt, device=p.device) for p in params] if m is None else list(m)
    v = [torch.zeros(p.shape, dtype=sdt, device=p.device) for p in params] if v is None else list(v)
    rows = [(p.numel() + 255) // 256 for p in params]
    if state_bits == 8:
        m_scale, v_scale = ([torch.ones(r, device=p.device) for r, p in zip(rows, params)] if s is None else list(s)
                            for s in (m_scale, v_scale))
    else:
        m_scale, v_scale = [None] * n, [None] * n
    if not all(len(x) == n for x in (grads, wd, lm, m, v, m_scale, v_scale)):
        raise ValueError("adamw_plan takes as many of each as there are parameters")
    t = (_lib.AdamwTensor * n)()
    for i in range(n):
        p, g = params[i], grads[i]
        if any(x.numel() != p.numel() for x in (g, m[i], v[i])) or m[i].dtype != sdt or v[i].dtype != sdt:
            raise ValueError(f"tensor {i}: gradient and states must match the parameter, states in {sdt}")
        if any(x.device != p.device for x in (g, m[i], v[i], params[0])):
            raise ValueError(f"tensor {i}: all tensors of a plan live on one device")
        if state_bits == 8 and any(s.numel() != rows[i] or s.dtype != torch.float32 or s.device != p.device
                                   for s in (m_scale[i], v_scale[i])):
            raise ValueError(f"tensor {i}: scales are fp32, one per 256 elements")
        t[i] = _lib.AdamwTensor(_ptr(p), _ptr(g), _ptr(m[i]), _ptr(v[i]), _ptr(m_scale[i]), _ptr(v_scale[i]),
                                p.numel(), lm[i], wd[i], _dt(p.dtype), _dt(g.dtype))
    image = torch.zeros(lib.rb_adamw_plan_bytes(ctypes.byref(t), n), dtype=torch.uint8)
    chunks = ctypes.c_int64()
    check("rb_adamw_plan", lib.rb_adamw_plan(ctypes.byref(t), n, state_bits, ctypes.c_void_p(image.data_ptr()),
                                             image.numel(), ctypes.byref(chunks)))
    return AdamWPlan(params, grads, state_bits, m, v, m_scale, v_scale, image.to(params[0].device), chunks.value)


def adamw_step(plan: AdamWPlan, step: int, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
               grad_scale: torch.Tensor | None = None, skip: torch.Tensor | None = None, seed: int = 0) -> None:
    """Step number `step` (1, 2, ...) of AdamW over the plan's tensors, in place, in one launch.
    `grad_scale` (device fp32) multiplies the gradients; the step changes nothing where `skip`
    (device int32) is not 0; `seed` feeds the rounding of 8-bit states."""
    if grad_scale is not None and grad_scale.dtype != torch.float32:
        raise TypeError("grad_scale is a device fp32")
    if skip is not None and skip.dtype != torch.int32:
        raise TypeError("skip is a device int32")
    check("rb_adamw_step", lib.rb_adamw_step(_ptr(plan.table), plan.chunks, plan.state_bits, step, lr, beta1, beta2,
                                             eps, _ptr(grad_scale), _ptr(skip), seed & 0xFFFFFFFF, _stream()))
