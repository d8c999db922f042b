"""Python binding of libmi355gemm.so: row-major GEMM on one MI355X.

The functions take the same arguments as the C ABI in
``include/mi355gemm.h`` and only marshal them (the ``_ex`` forms add the
transA/transB flags of C = alpha*op(A)op(B) + beta*C): every step of the computation
runs in the library's HIP kernels.  Operands may be torch CUDA tensors (their
``data_ptr()`` is passed; dtype, device and storage extent are checked first so
that a wrong buffer is refused on the host instead of faulting the GPU) or raw
integer device addresses (passed as they are).  ``stream`` may be None (torch's
current stream), a ``torch.cuda.Stream`` or a raw ``hipStream_t`` integer.

The functions at the end (routing, grouped products, combining, adapters) run on
the device their tensors (and a ``torch.cuda.Stream``) are on, refuse more than one
device, and where they need a workspace take ``workspace=`` or let torch allocate it.

If the library is not built, importing works but every call raises
``GemmLibraryMissing``: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import os

__all__ = ["gemm_f32", "gemm_f16_f32acc", "gemm_batched_f16_f32acc",
           "gemm_f32_ex", "gemm_f16_f32acc_ex", "gemm_batched_f16_f32acc_ex",
           "gemm_bf16_f32acc", "gemm_batched_bf16_f32acc", "gemm_bf16_f32acc_ex", "gemm_batched_bf16_f32acc_ex",
           "gemm_f16_f32acc_noalloc",
           "moe_route_f32", "moe_route_workspace", "moe_route_f32_grad",
           "gemm_grouped_f16_f32acc_ex", "gemm_grouped_bf16_f32acc_ex",
           "gemm_grouped_wgrad_f16_f32acc", "gemm_grouped_wgrad_bf16_f32acc",
           "moe_combine_f32", "moe_combine_grad_f16", "moe_combine_grad_bf16",
           "gemm_lora_f16_f32acc_ex", "gemm_lora_bf16_f32acc_ex", "gemm_lora_workspace",
           "status_string",
           "GemmError", "GemmLibraryMissing", "LIB_PATH", "load_library", "EXPORTS"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmi355gemm.so")
EXPORTS = ("gemm_f32", "gemm_f16_f32acc", "gemm_batched_f16_f32acc",
           "gemm_f32_ex", "gemm_f16_f32acc_ex", "gemm_batched_f16_f32acc_ex",
           "gemm_bf16_f32acc", "gemm_batched_bf16_f32acc", "gemm_bf16_f32acc_ex", "gemm_batched_bf16_f32acc_ex",
           "gemm_f16_f32acc_noalloc",
           "moe_route_f32", "moe_route_workspace", "moe_route_f32_grad",
           "gemm_grouped_f16_f32acc_ex", "gemm_grouped_bf16_f32acc_ex",
           "gemm_grouped_wgrad_f16_f32acc", "gemm_grouped_wgrad_bf16_f32acc",
           "moe_combine_f32", "moe_combine_grad_f16", "moe_combine_grad_bf16",
           "gemm_lora_f16_f32acc_ex", "gemm_lora_bf16_f32acc_ex", "gemm_lora_workspace",
           "gemm_status_string")

_lib = None


class GemmError(RuntimeError):
    """A non-zero status returned by the library."""

    def __init__(self, status: int, fn: str):
        self.status = status
        super().__init__(f"{fn} failed with status {status}: {status_string(status)}")


class GemmLibraryMissing(RuntimeError):
    """libmi355gemm.so has not been built (run dense_gemm_optimisation_f32_amd.build)."""


def load_library(path: str = LIB_PATH):
    """Load (once) and return the ctypes handle of the library."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise GemmLibraryMissing(f"{path} is missing; build it with "
                                 "`python -m dense_gemm_optimisation_f32_amd.build`")
    lib = ctypes.CDLL(path)
    i, f, vp, ll = ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_longlong
    lib.gemm_f32.argtypes = [i, i, i, f, vp, i, vp, i, f, vp, i, vp]
    lib.gemm_f32.restype = i
    lib.gemm_f16_f32acc.argtypes = [i, i, i, f, vp, i, vp, i, f, vp, i, vp]
    lib.gemm_f16_f32acc.restype = i
    lib.gemm_batched_f16_f32acc.argtypes = [i, i, i, f, vp, i, ll, vp, i, ll, f, vp, i, ll, i, vp]
    lib.gemm_batched_f16_f32acc.restype = i
    lib.gemm_f32_ex.argtypes = [i, i] + lib.gemm_f32.argtypes
    lib.gemm_f32_ex.restype = i
    lib.gemm_f16_f32acc_ex.argtypes = [i, i] + lib.gemm_f16_f32acc.argtypes
    lib.gemm_f16_f32acc_ex.restype = i
    lib.gemm_batched_f16_f32acc_ex.argtypes = [i, i] + lib.gemm_batched_f16_f32acc.argtypes
    lib.gemm_batched_f16_f32acc_ex.restype = i
    for name, base in (("gemm_bf16_f32acc", lib.gemm_f16_f32acc),
                       ("gemm_batched_bf16_f32acc", lib.gemm_batched_f16_f32acc),
                       ("gemm_bf16_f32acc_ex", lib.gemm_f16_f32acc_ex),
                       ("gemm_batched_bf16_f32acc_ex", lib.gemm_batched_f16_f32acc_ex)):
        fn = getattr(lib, name)
        fn.argtypes = base.argtypes
        fn.restype = i
    lib.gemm_f16_f32acc_noalloc.argtypes = lib.gemm_f16_f32acc.argtypes
    lib.gemm_f16_f32acc_noalloc.restype = i
    lib.moe_route_f32.argtypes = [i, i, vp, i, vp, i, i, i, i, i, i, f, vp, vp, vp, vp, vp, vp, ll, vp]
    lib.moe_route_f32_grad.argtypes = [i, i, vp, i, i, i, i, f, vp, vp, vp, i, vp]
    lib.moe_combine_f32.argtypes = [i, i, i, vp, i, i, vp, vp, f, vp, i, vp]
    for t in ("f16", "bf16"):
        getattr(lib, f"gemm_grouped_{t}_f32acc_ex").argtypes = [i, i, i, i, i, f, vp, i, i, vp, vp, i, ll, vp, f, vp, i, vp]
        getattr(lib, f"gemm_grouped_wgrad_{t}_f32acc").argtypes = [i, i, i, i, f, vp, i, i, vp, vp, i, i, vp, vp, f, vp, i,
                                                                   ll, vp]
        getattr(lib, f"moe_combine_grad_{t}").argtypes = [i, i, i, vp, i, vp, i, i, vp, vp, vp, i, vp, vp]
        getattr(lib, f"gemm_lora_{t}_f32acc_ex").argtypes = [i, i, i, i, i, i, f, vp, i, vp, i, vp, i, ll, vp, i, ll, vp, vp,
                                                             vp, f, vp, i, vp, ll, vp]
    for name in ("moe_route_f32", "moe_route_f32_grad", "moe_combine_f32", "gemm_grouped_f16_f32acc_ex",
                 "gemm_grouped_bf16_f32acc_ex", "gemm_grouped_wgrad_f16_f32acc", "gemm_grouped_wgrad_bf16_f32acc",
                 "moe_combine_grad_f16", "moe_combine_grad_bf16", "gemm_lora_f16_f32acc_ex", "gemm_lora_bf16_f32acc_ex"):
        getattr(lib, name).restype = i
    lib.moe_route_workspace.argtypes = [i, i, i]
    lib.moe_route_workspace.restype = ll
    lib.gemm_lora_workspace.argtypes = [i, i, i, i]
    lib.gemm_lora_workspace.restype = ll
    lib.gemm_status_string.argtypes = [i]
    lib.gemm_status_string.restype = ctypes.c_char_p
    if path == LIB_PATH:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().gemm_status_string(int(status)).decode()


def _extent(rows: int, cols: int, ld: int) -> int:
    return 0 if rows <= 0 or cols <= 0 else (rows - 1) * ld + cols


def _is_tensor(x) -> bool:
    return type(x).__module__.startswith("torch") and hasattr(x, "data_ptr")


def _ptr(x, name: str, dtype_name: str | None, need: int):
    """Device address of an operand, checking torch tensors against the extent read or written."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if _is_tensor(x):
        if x.device.type != "cuda":
            raise ValueError(f"{name} must be a CUDA tensor, got device {x.device}")
        if dtype_name is not None and str(x.dtype) != dtype_name:
            raise TypeError(f"{name} must have dtype {dtype_name}, got {x.dtype}")
        if need > 0:
            st = x.untyped_storage()
            avail = (st.nbytes() - (x.data_ptr() - st.data_ptr())) // x.element_size()
            if avail < need:
                raise ValueError(f"{name} holds {avail} elements from its start; the call needs {need}")
        return x.data_ptr()
    raise TypeError(f"{name}: expected a torch tensor or an integer device address, got {type(x)}")


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _needs(M, N, K, alpha, lda, ldb, ldc, batch=1, sA=0, sB=0, sC=0, transA=0, transB=0):
    reads_ab = K > 0 and alpha != 0 and M > 0 and N > 0
    nb = max(batch - 1, 0)
    a_rows, a_cols = (K, M) if transA else (M, K)
    b_rows, b_cols = (N, K) if transB else (K, N)
    na = _extent(a_rows, a_cols, lda) + nb * sA if reads_ab else 0
    nbb = _extent(b_rows, b_cols, ldb) + nb * sB if reads_ab else 0
    nc = _extent(M, N, ldc) + nb * sC if batch > 0 else 0
    return na, nbb, nc


def gemm_f32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> None:
    """C <- alpha*A*B + beta*C, fp32 (see gemm_f32 in include/mi355gemm.h)."""
    lib = load_library()
    na, nb, nc = _needs(M, N, K, alpha, lda, ldb, ldc)
    rc = lib.gemm_f32(M, N, K, alpha, _ptr(A, "A", "torch.float32", na), lda,
                      _ptr(B, "B", "torch.float32", nb), ldb, beta,
                      _ptr(C, "C", "torch.float32", nc), ldc, _stream(stream))
    if rc != 0:
        raise GemmError(rc, "gemm_f32")


def gemm_f16_f32acc(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> None:
    """C <- alpha*A*B + beta*C with fp16 A, B and fp32 accumulation and C."""
    lib = load_library()
    na, nb, nc = _needs(M, N, K, alpha, lda, ldb, ldc)
    rc = lib.gemm_f16_f32acc(M, N, K, alpha, _ptr(A, "A", "torch.float16", na), lda,
                             _ptr(B, "B", "torch.float16", nb), ldb, beta,
                             _ptr(C, "C", "torch.float32", nc), ldc, _stream(stream))
    if rc != 0:
        raise GemmError(rc, "gemm_f16_f32acc")


def gemm_f16_f32acc_noalloc(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> None:
    """gemm_f16_f32acc for callers that cannot allocate: its K split keeps its partial tiles in one
    static buffer per GPU (calls that overlap on one GPU must not be made)."""
    lib = load_library()
    na, nb, nc = _needs(M, N, K, alpha, lda, ldb, ldc)
    rc = lib.gemm_f16_f32acc_noalloc(M, N, K, alpha, _ptr(A, "A", "torch.float16", na), lda,
                                     _ptr(B, "B", "torch.float16", nb), ldb, beta,
                                     _ptr(C, "C", "torch.float32", nc), ldc, _stream(stream))
    if rc != 0:
        raise GemmError(rc, "gemm_f16_f32acc_noalloc")


def gemm_batched_f16_f32acc(M, N, K, alpha, A, lda, strideA, B, ldb, strideB, beta, C, ldc, strideC,
                            batch_count, stream=None) -> None:
    """Strided-batched form of gemm_f16_f32acc (member b at A + b*strideA etc.)."""
    lib = load_library()
    na, nb, nc = _needs(M, N, K, alpha, lda, ldb, ldc, batch_count, strideA, strideB, strideC)
    rc = lib.gemm_batched_f16_f32acc(M, N, K, alpha, _ptr(A, "A", "torch.float16", na), lda, strideA,
                                     _ptr(B, "B", "torch.float16", nb), ldb, strideB, beta,
                                     _ptr(C, "C", "torch.float32", nc), ldc, strideC, batch_count,
                                     _stream(stream))
    if rc != 0:
        raise GemmError(rc, "gemm_batched_f16_f32acc")


def gemm_f32_ex(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> None:
    """C <- alpha*op(A)*op(B) + beta*C, fp32; transA: A stored K x M, transB: B stored N x K."""
    lib = load_library()
    tA, tB = int(transA), int(transB)   # values other than 0/1 are refused by the library
    na, nb, nc = _needs(M, N, K, alpha, lda, ldb, ldc, transA=tA, transB=tB)
    rc = lib.gemm_f32_ex(tA, tB, M, N, K, alpha, _ptr(A, "A", "torch.float32", na), lda,
                         _ptr(B, "B", "torch.float32", nb), ldb, beta,
                         _ptr(C, "C", "torch.float32", nc), ldc, _stream(stream))
    if rc != 0:
        raise GemmError(rc, "gemm_f32_ex")


def gemm_f16_f32acc_ex(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> None:
    """gemm_f16_f32acc with op(A)/op(B) (see gemm_f32_ex)."""
    lib = load_library()
    tA, tB = int(transA), int(transB)   # values other than 0/1 are refused by the library
    na, nb, nc = _needs(M, N, K, alpha, lda, ldb, ldc, transA=tA, transB=tB)
    rc = lib.gemm_f16_f32acc_ex(tA, tB, M, N, K, alpha, _ptr(A, "A", "torch.float16", na), lda,
                                _ptr(B, "B", "torch.float16", nb), ldb, beta,
                                _ptr(C, "C", "torch.float32", nc), ldc, _stream(stream))
    if rc != 0:
        raise GemmError(rc, "gemm_f16_f32acc_ex")


def gemm_batched_f16_f32acc_ex(transA, transB, M, N, K, alpha, A, lda, strideA, B, ldb, strideB, beta, C, ldc,
                               strideC, batch_count, stream=None) -> None:
    """gemm_batched_f16_f32acc with op(A)/op(B) (see gemm_f32_ex)."""
    lib = load_library()
    tA, tB = int(transA), int(transB)   # values other than 0/1 are refused by the library
    na, nb, nc = _needs(M, N, K, alpha, lda, ldb, ldc, batch_count, strideA, strideB, strideC, tA, tB)
    rc = lib.gemm_batched_f16_f32acc_ex(tA, tB, M, N, K, alpha, _ptr(A, "A", "torch.float16", na), lda, strideA,
                                        _ptr(B, "B", "torch.float16", nb), ldb, strideB, beta,
                                        _ptr(C, "C", "torch.float32", nc), ldc, strideC, batch_count,
                                        _stream(stream))
    if rc != 0:
        raise GemmError(rc, "gemm_batched_f16_f32acc_ex")


def gemm_bf16_f32acc(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> None:
    """C <- alpha*A*B + beta*C with bf16 A, B and fp32 accumulation and C."""
    lib = load_library()
    na, nb, nc = _needs(M, N, K, alpha, lda, ldb, ldc)
    rc = lib.gemm_bf16_f32acc(M, N, K, alpha, _ptr(A, "A", "torch.bfloat16", na), lda,
                              _ptr(B, "B", "torch.bfloat16", nb), ldb, beta,
                              _ptr(C, "C", "torch.float32", nc), ldc, _stream(stream))
    if rc != 0:
        raise GemmError(rc, "gemm_bf16_f32acc")


def gemm_batched_bf16_f32acc(M, N, K, alpha, A, lda, strideA, B, ldb, strideB, beta, C, ldc, strideC,
                             batch_count, stream=None) -> None:
    """Strided-batched form of gemm_bf16_f32acc."""
    lib = load_library()
    na, nb, nc = _needs(M, N, K, alpha, lda, ldb, ldc, batch_count, strideA, strideB, strideC)
    rc = lib.gemm_batched_bf16_f32acc(M, N, K, alpha, _ptr(A, "A", "torch.bfloat16", na), lda, strideA,
                                      _ptr(B, "B", "torch.bfloat16", nb), ldb, strideB, beta,
                                      _ptr(C, "C", "torch.float32", nc), ldc, strideC, batch_count,
                                      _stream(stream))
    if rc != 0:
        raise GemmError(rc, "gemm_batched_bf16_f32acc")


def gemm_bf16_f32acc_ex(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> None:
    """gemm_bf16_f32acc with op(A)/op(B) (see gemm_f32_ex)."""
    lib = load_library()
    tA, tB = int(transA), int(transB)   # values other than 0/1 are refused by the library
    na, nb, nc = _needs(M, N, K, alpha, lda, ldb, ldc, transA=tA, transB=tB)
    rc = lib.gemm_bf16_f32acc_ex(tA, tB, M, N, K, alpha, _ptr(A, "A", "torch.bfloat16", na), lda,
                                 _ptr(B, "B", "torch.bfloat16", nb), ldb, beta,
                                 _ptr(C, "C", "torch.float32", nc), ldc, _stream(stream))
    if rc != 0:
        raise GemmError(rc, "gemm_bf16_f32acc_ex")


def gemm_batched_bf16_f32acc_ex(transA, transB, M, N, K, alpha, A, lda, strideA, B, ldb, strideB, beta, C, ldc,
                                strideC, batch_count, stream=None) -> None:
    """gemm_batched_bf16_f32acc with op(A)/op(B) (see gemm_f32_ex)."""
    lib = load_library()
    tA, tB = int(transA), int(transB)   # values other than 0/1 are refused by the library
    na, nb, nc = _needs(M, N, K, alpha, lda, ldb, ldc, batch_count, strideA, strideB, strideC, tA, tB)
    rc = lib.gemm_batched_bf16_f32acc_ex(tA, tB, M, N, K, alpha, _ptr(A, "A", "torch.bfloat16", na), lda,
                                         strideA, _ptr(B, "B", "torch.bfloat16", nb), ldb, strideB, beta,
                                         _ptr(C, "C", "torch.float32", nc), ldc, strideC, batch_count,
                                         _stream(stream))
    if rc != 0:
        raise GemmError(rc, "gemm_batched_bf16_f32acc_ex")


# ------------------------------------------------------------------ products whose right operand is chosen per row
#
# These calls serve single tokens, whose kernels take a few microseconds, so their
# marshalling is kept short: one test of an operand's properties where all is as
# expected, sizes of workspaces remembered by the sizes they belong to.
_torch = None
_Tensor = _device = _raw_stream = None   # torch.Tensor; the current device's index; its current stream's handle
_DTYPES = {}


class _Elsewhere(Exception):
    """An operand or the stream is on another device than the current one."""

    def __init__(self, index: int):
        self.index = index


def _load_torch():
    global _torch, _Tensor, _device, _raw_stream
    import torch

    _Tensor, _device, _raw_stream = torch.Tensor, torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    _DTYPES.update(float32=torch.float32, float16=torch.float16, bfloat16=torch.bfloat16, int32=torch.int32)
    _torch = torch
    return torch


def _on_operands_device(fn):
    """Run ``fn`` with the device current that its tensors and its stream are on (one for all of them)."""

    @functools.wraps(fn)
    def call(*args, **kwargs):
        try:
            return fn(*args, **kwargs)
        except _Elsewhere as e:
            index = e.index
        with _torch.cuda.device(index):
            try:
                return fn(*args, **kwargs)
            except _Elsewhere as e:
                raise ValueError(f"{fn.__name__}: operands or stream on more than one device: cuda:{index} and cuda:{e.index}") from None

    return call


def _strided(x, name: str, dtype_name: str, need: int, packed: bool = False):
    """Device address of an operand of which the call reads or writes ``need`` elements; the short way is a contiguous
    tensor on the current device that holds them."""
    if type(x) is _Tensor:
        if (x.is_cuda and x.dtype is _DTYPES[dtype_name] and x.numel() >= need and x.is_contiguous()
                and x.get_device() == _device()):
            return x.data_ptr()
    elif x is None or type(x) is int:
        return x
    torch = _torch or _load_torch()
    if isinstance(x, torch.Tensor) and x.is_cuda:
        if x.get_device() != _device():
            raise _Elsewhere(x.get_device())
        if packed and not x.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    return _ptr(x, name, "torch." + dtype_name, need)


def _packed(x, name: str, dtype_name: str, need: int):
    """Device address of an array the kernels read or write without strides."""
    return _strided(x, name, dtype_name, need, True)


def _call(fn, args, stream, workspace=None, workspace_bytes=None) -> None:
    """Run library function ``fn`` on ``stream``, or on the current stream.  With ``workspace_bytes`` the call takes a
    workspace: the caller's, or one that torch's allocator hands out for that stream (graph capture included) and
    takes back in its order."""
    if stream is None:
        if _torch is None:
            _load_torch()
        h = _raw_stream(_device())
    else:
        h = _stream(stream)
        at = getattr(stream, "device", None)   # (a raw handle has none)
        if at is not None:
            if _torch is None:
                _load_torch()
            if at.index != _device():
                raise _Elsewhere(at.index)
    if workspace_bytes is None:
        rc = fn(*args, h)
    else:
        if workspace is None and workspace_bytes > 0:
            torch = _torch or _load_torch()
            if stream is None:
                workspace = torch.empty(workspace_bytes, dtype=torch.uint8, device="cuda")   # (the current device)
            else:
                with torch.cuda.stream(torch.cuda.ExternalStream(h)):
                    workspace = torch.empty(workspace_bytes, dtype=torch.uint8, device="cuda")
            rc = fn(*args, workspace.data_ptr(), workspace_bytes, h)
        else:
            rc = fn(*args, *_room(workspace, workspace_bytes), h)
    if rc != 0:
        raise GemmError(rc, fn.__name__)


def _room(workspace, need: int):
    """Address and bytes the library may use: what a tensor's storage holds from its start, or for a raw address what the call needs."""
    if workspace is None or type(workspace) is int:
        return workspace, need
    if workspace.is_cuda and workspace.get_device() != (_torch or _load_torch()).cuda.current_device():
        raise _Elsewhere(workspace.get_device())
    at = _ptr(workspace, "workspace", None, 0)
    st = workspace.untyped_storage()
    return at, st.nbytes() - (at - st.data_ptr())


@functools.lru_cache(maxsize=None)
def _function(name: str):
    return getattr(load_library(), name)


@functools.lru_cache(maxsize=1024)
def moe_route_workspace(T, E, k) -> int:
    """Bytes of workspace moe_route_f32 needs for its sorted choices (0: none)."""
    return load_library().moe_route_workspace(T, E, k)


@_on_operands_device
def moe_route_f32(T, E, logits, ldl, bias, score, groups, group_k, group_top, k, renorm, scale, ids, weights, offsets=None,
                  rows=None, slots=None, workspace=None, stream=None) -> None:
    """Each of T tokens chooses k of E experts (ids, weights), and the choices sorted by expert (offsets, rows, slots)."""
    n = max(T, 0) * max(k, 0)
    args = (T, E, _strided(logits, "logits", "float32", _extent(T, E, ldl)), ldl, _packed(bias, "bias", "float32", E),
            int(score), groups, group_k, group_top, k, int(renorm), scale, _packed(ids, "ids", "int32", n),
            _packed(weights, "weights", "float32", n), _packed(offsets, "offsets", "int32", E + 1),
            _packed(rows, "rows", "int32", n), _packed(slots, "slots", "int32", n))
    need = moe_route_workspace(T, E, k) if offsets is not None else 0
    _call(_function("moe_route_f32"), args, stream, workspace, need)


@_on_operands_device
def moe_route_f32_grad(T, E, logits, ldl, score, k, renorm, scale, ids, dweights, dlogits, lddl, stream=None) -> None:
    """dlogits from dweights: the gradient of moe_route_f32's weights in its logits."""
    n = max(T, 0) * max(k, 0)
    args = (T, E, _strided(logits, "logits", "float32", _extent(T, E, ldl)), ldl, int(score), k, int(renorm), scale,
            _packed(ids, "ids", "int32", n), _packed(dweights, "dweights", "float32", n),
            _strided(dlogits, "dlogits", "float32", _extent(T, E, lddl)), lddl)
    _call(_function("moe_route_f32_grad"), args, stream)


def _grouped(t, dtype_name, transB, groups, R, N, K, alpha, A, M, lda, rows, B, ldb, strideB, offsets, beta, C, ldc, stream):
    tB = int(transB)
    work = groups > 0 and R > 0 and N > 0
    reads = work and K > 0 and alpha != 0 and M > 0
    b = _extent(*((N, K) if tB else (K, N)), ldb) + max(groups - 1, 0) * strideB
    args = (tB, groups, R, N, K, alpha, _strided(A, "A", dtype_name, _extent(M, K, lda) if reads else 0), M, lda,
            _packed(rows, "rows", "int32", R if reads else 0), _strided(B, "B", dtype_name, b if reads else 0), ldb, strideB,
            _packed(offsets, "offsets", "int32", groups + 1 if work else 0), beta,
            _strided(C, "C", "float32", _extent(R, N, ldc)), ldc)
    _call(_function(f"gemm_grouped_{t}_f32acc_ex"), args, stream)


@_on_operands_device
def gemm_grouped_f16_f32acc_ex(transB, groups, R, N, K, alpha, A, M, lda, rows, B, ldb, strideB, offsets, beta, C, ldc,
                               stream=None) -> None:
    """C[r,:] <- alpha*A[rows[r],:]*op(B_g) + beta*C[r,:] for the rows r of every group g; fp16 A and B, fp32 C."""
    _grouped("f16", "float16", transB, groups, R, N, K, alpha, A, M, lda, rows, B, ldb, strideB, offsets, beta, C, ldc,
             stream)


@_on_operands_device
def gemm_grouped_bf16_f32acc_ex(transB, groups, R, N, K, alpha, A, M, lda, rows, B, ldb, strideB, offsets, beta, C, ldc,
                                stream=None) -> None:
    """gemm_grouped_f16_f32acc_ex with bf16 A and B."""
    _grouped("bf16", "bfloat16", transB, groups, R, N, K, alpha, A, M, lda, rows, B, ldb, strideB, offsets, beta, C, ldc,
             stream)


def _wgrad(t, dtype_name, groups, R, M, N, alpha, A, a_rows, lda, rowsA, B, b_rows, ldb, rowsB, offsets, beta, C, ldc, strideC,
           stream):
    work = groups > 0 and M > 0 and N > 0
    reads = work and R > 0 and alpha != 0 and a_rows > 0 and b_rows > 0
    args = (groups, R, M, N, alpha, _strided(A, "A", dtype_name, _extent(a_rows, M, lda) if reads else 0), a_rows, lda,
            _packed(rowsA, "rowsA", "int32", R if reads else 0),
            _strided(B, "B", dtype_name, _extent(b_rows, N, ldb) if reads else 0), b_rows, ldb,
            _packed(rowsB, "rowsB", "int32", R if reads else 0),
            _packed(offsets, "offsets", "int32", groups + 1 if reads else 0), beta,
            _strided(C, "C", "float32", _extent(M, N, ldc) + (groups - 1) * strideC if work else 0), ldc, strideC)
    _call(_function(f"gemm_grouped_wgrad_{t}_f32acc"), args, stream)


@_on_operands_device
def gemm_grouped_wgrad_f16_f32acc(groups, R, M, N, alpha, A, a_rows, lda, rowsA, B, b_rows, ldb, rowsB, offsets, beta, C, ldc,
                                  strideC, stream=None) -> None:
    """C_g <- alpha * sum over group g's rows r of A[rowsA[r],:]^T B[rowsB[r],:] + beta*C_g; fp16 A and B, fp32 C."""
    _wgrad("f16", "float16", groups, R, M, N, alpha, A, a_rows, lda, rowsA, B, b_rows, ldb, rowsB, offsets, beta, C, ldc,
           strideC, stream)


@_on_operands_device
def gemm_grouped_wgrad_bf16_f32acc(groups, R, M, N, alpha, A, a_rows, lda, rowsA, B, b_rows, ldb, rowsB, offsets, beta, C, ldc,
                                   strideC, stream=None) -> None:
    """gemm_grouped_wgrad_f16_f32acc with bf16 A and B."""
    _wgrad("bf16", "bfloat16", groups, R, M, N, alpha, A, a_rows, lda, rowsA, B, b_rows, ldb, rowsB, offsets, beta, C, ldc,
           strideC, stream)


@_on_operands_device
def moe_combine_f32(T, k, N, Y, R, ldy, slots, weights, beta, C, ldc, stream=None) -> None:
    """C[t,:] <- sum_j weights[t,j]*Y[slots[t,j],:] + beta*C[t,:] (weights None: ones)."""
    n = max(T, 0) * max(k, 0) if N > 0 else 0
    args = (T, k, N, _strided(Y, "Y", "float32", _extent(R, N, ldy) if n else 0), R, ldy,
            _packed(slots, "slots", "int32", n), _packed(weights, "weights", "float32", n), beta,
            _strided(C, "C", "float32", _extent(T, N, ldc)), ldc)
    _call(_function("moe_combine_f32"), args, stream)


def _combine_grad(t, dtype_name, T, k, N, dC, lddc, Y, R, ldy, slots, weights, dY, lddy, dweights, stream):
    n = max(T, 0) * max(k, 0)
    args = (T, k, N, _strided(dC, "dC", "float32", _extent(T, N, lddc)), lddc,
            _strided(Y, "Y", "float32", _extent(R, N, ldy) if n else 0), R, ldy, _packed(slots, "slots", "int32", n),
            _packed(weights, "weights", "float32", n), _strided(dY, "dY", dtype_name, _extent(R, N, lddy) if n else 0), lddy,
            _packed(dweights, "dweights", "float32", n))
    _call(_function(f"moe_combine_grad_{t}"), args, stream)


@_on_operands_device
def moe_combine_grad_f16(T, k, N, dC, lddc, Y, R, ldy, slots, weights, dY, lddy, dweights, stream=None) -> None:
    """The gradient of moe_combine_f32: dY in fp16 (what the grouped products take) and dweights in fp32."""
    _combine_grad("f16", "float16", T, k, N, dC, lddc, Y, R, ldy, slots, weights, dY, lddy, dweights, stream)


@_on_operands_device
def moe_combine_grad_bf16(T, k, N, dC, lddc, Y, R, ldy, slots, weights, dY, lddy, dweights, stream=None) -> None:
    """moe_combine_grad_f16 with dY in bf16."""
    _combine_grad("bf16", "bfloat16", T, k, N, dC, lddc, Y, R, ldy, slots, weights, dY, lddy, dweights, stream)


@functools.lru_cache(maxsize=1024)
def gemm_lora_workspace(M, N, K, rank) -> int:
    """Bytes of workspace gemm_lora_f16_f32acc_ex and its bf16 form need."""
    return load_library().gemm_lora_workspace(M, N, K, rank)


def _lora(t, dtype_name, transB, M, N, K, rank, adapters, alpha, A, lda, B, ldb, LA, ldla, strideLA, LB, ldlb, strideLB, scales,
          ranks, ids, beta, C, ldc, workspace, stream):
    tB = int(transB)
    na = nb = nc = 0
    if M > 0 and N > 0:
        nc = (M - 1) * ldc + N
        if K > 0 and alpha != 0:
            na = (M - 1) * lda + K
            nb = (N - 1) * ldb + K if tB else (K - 1) * ldb + N
    thin = na > 0 and adapters > 0
    last = max(adapters - 1, 0)
    args = (tB, M, N, K, rank, adapters, alpha, _strided(A, "A", dtype_name, na), lda, _strided(B, "B", dtype_name, nb), ldb,
            _strided(LA, "LA", dtype_name, _extent(rank, K, ldla) + last * strideLA if thin else 0), ldla, strideLA,
            _strided(LB, "LB", dtype_name, _extent(N, rank, ldlb) + last * strideLB if thin else 0), ldlb, strideLB,
            _packed(scales, "scales", "float32", adapters if thin else 0),
            _packed(ranks, "ranks", "int32", adapters if thin else 0),
            _packed(ids, "ids", "int32", M if thin else 0), beta, _strided(C, "C", "float32", nc), ldc)
    need = gemm_lora_workspace(M, N, K, rank) if thin else 0
    _call(_function(f"gemm_lora_{t}_f32acc_ex"), args, stream, workspace, need)


@_on_operands_device
def gemm_lora_f16_f32acc_ex(transB, M, N, K, rank, adapters, alpha, A, lda, B, ldb, LA, ldla, strideLA, LB, ldlb, strideLB, scales,
                            ranks, ids, beta, C, ldc, workspace=None, stream=None) -> None:
    """C[i,:] <- alpha*(A[i,:]*op(B) + scales[a]*(A[i,:]*LA_a^T)*LB_a^T) + beta*C[i,:], a = ids[i]; fp16 inputs, fp32 C."""
    _lora("f16", "float16", transB, M, N, K, rank, adapters, alpha, A, lda, B, ldb, LA, ldla, strideLA, LB, ldlb, strideLB,
          scales, ranks, ids, beta, C, ldc, workspace, stream)


@_on_operands_device
def gemm_lora_bf16_f32acc_ex(transB, M, N, K, rank, adapters, alpha, A, lda, B, ldb, LA, ldla, strideLA, LB, ldlb, strideLB,
                             scales, ranks, ids, beta, C, ldc, workspace=None, stream=None) -> None:
    """gemm_lora_f16_f32acc_ex with bf16 inputs."""
    _lora("bf16", "bfloat16", transB, M, N, K, rank, adapters, alpha, A, lda, B, ldb, LA, ldla, strideLA, LB, ldlb, strideLB,
          scales, ranks, ids, beta, C, ldc, workspace, stream)
