"""ctypes binding of libgemm_f32.so (include/gemm_f32.h, gemm_f32_rows.h), same names.

Argument marshalling only: every step of the product runs in the library's
HIP kernels.  ``matmul`` is a convenience over ``gemm_f32`` that takes torch
tensors for device memory and the current torch stream; it validates layout
and raises on any non-zero status.  ``route``, ``expert_map``, ``grouped_matmul``,
``combine``, ``adapter_matmul`` and the ``*_grad`` functions do the same for the
products whose second matrix is chosen row by row.  There is no fallback: if the library is
missing and cannot be built, loading raises.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(PKG, "libgemm_f32.so")

GEMM_F32_OK = 0
GEMM_F32_ERR_DIM = 1
GEMM_F32_ERR_LD = 2
GEMM_F32_ERR_NULL = 3
GEMM_F32_ERR_LAUNCH = 4
GEMM_F32_ERR_CONFIG = 5
GEMM_F32_ERR_ALIGN = 6
GEMM_F32_ERR_SCRATCH = 7
GEMM_F32_ERR_TYPE = 8
GEMM_F32_ERR_OPTION = 9
GEMM_F32_ERR_WORKSPACE = 10
GEMM_F32_SCRATCH_BYTES = 4 << 20

GEMM_F32_TYPE_F32, GEMM_F32_TYPE_BF16, GEMM_F32_TYPE_F16 = 0, 1, 2
GEMM_F32_SCORE_SOFTMAX, GEMM_F32_SCORE_SIGMOID = 0, 1
GEMM_F32_MAX_EXPERTS = 1024
GEMM_F32_MAX_CHOSEN = 64
GEMM_F32_MAX_RANK = 256

_lib = None


class GemmError(RuntimeError):
    def __init__(self, status: int, what: str = "gemm_f32"):
        self.status = status
        super().__init__(f"{what}: status {status} ({gemm_f32_status_string(status)})")


def load() -> ctypes.CDLL:
    """The HIP library (built in-tree first if it is not there yet)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIBRARY):
            from . import build
            build.build()
        lib = ctypes.CDLL(LIBRARY)
        i, p = ctypes.c_int, ctypes.c_void_p
        gemm_args = [i, i, i, p, i, p, i, p, i, p]
        lib.gemm_f32.argtypes = gemm_args
        lib.gemm_f32.restype = i
        lib.gemm_f32_with_config.argtypes = [i] + gemm_args
        lib.gemm_f32_with_config.restype = i
        lib.gemm_f32_num_configs.argtypes = []
        lib.gemm_f32_num_configs.restype = i
        lib.gemm_f32_config_name.argtypes = [i]
        lib.gemm_f32_config_name.restype = ctypes.c_char_p
        ip = ctypes.POINTER(ctypes.c_int)
        lib.gemm_f32_config_info.argtypes = [i, ip, ip, ip, ip, ip]
        lib.gemm_f32_config_info.restype = i
        lib.gemm_f32_describe.argtypes = [i, i, i, i, p, i, p, i, p, i, ctypes.c_char_p, i]
        lib.gemm_f32_describe.restype = i
        lib.gemm_f32_ws_size.argtypes = [i, i, i]
        lib.gemm_f32_ws_size.restype = ctypes.c_size_t
        lib.gemm_f32_ws.argtypes = [i, i, i, p, i, p, i, p, i, p, ctypes.c_size_t, p]
        lib.gemm_f32_ws.restype = i
        lib.gemm_f32_ws_noalloc.argtypes = gemm_args
        lib.gemm_f32_ws_noalloc.restype = i
        lib.gemm_f32_device_peak.argtypes = [i, ip, ip, ctypes.POINTER(ctypes.c_double)]
        lib.gemm_f32_device_peak.restype = i
        z, f, l = ctypes.c_size_t, ctypes.c_float, ctypes.c_int64
        for name, res, args in (
                ("route", i, [i, i, i, i, p, i, p, i, i, i, i, i, f, p, p, p]),
                ("route_grad", i, [i, i, i, i, p, i, i, i, f, p, p, p, i, p]),
                ("expert_map_ws_size", z, [i, i]),
                ("expert_map", i, [i, i, p, p, p, p, p, z, p]),
                ("grouped", i, [i, i, i, i, i, p, p, i, i, p, i, p, i, l, p, i, p]),
                ("grouped_grad_x", i, [i, i, i, i, i, p, p, i, p, i, l, p, i, p]),
                ("grouped_grad_w", i, [i, i, i, i, i, p, p, i, i, p, i, p, i, p, i, l, p]),
                ("combine", i, [i, i, i, i, i, p, p, p, i, p, i, p]),
                ("combine_grad", i, [i, i, i, i, i, p, p, p, i, p, i, p, i, p, p]),
                ("adapters_ws_size", z, [i, i, i, i, i]),
                ("adapters", i, [i, i, i, i, i, i, p, i, p, i, p, i, l, p, i, l, p, p, p, i, p, z, p])):
            fn = getattr(lib, "gemm_f32_" + name)
            fn.argtypes, fn.restype = args, res
        lib.gemm_f32_status_string.argtypes = [i]
        lib.gemm_f32_status_string.restype = ctypes.c_char_p
        _lib = lib
    return _lib


INT32_MIN, INT32_MAX = -(1 << 31), (1 << 31) - 1


def _ints(**vals):
    """Refuses values a C int cannot hold: ctypes would wrap them silently
    (2^32 + 1000 becomes 1000), turning an oversized size or leading
    dimension into a different, valid-looking one."""
    for name, v in vals.items():
        if not INT32_MIN <= int(v) <= INT32_MAX:
            raise ValueError(f"{name} = {v} does not fit the C ABI's 32-bit int")


# --- the C ABI, one function per exported symbol ---------------------------
def gemm_f32(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    """C := A . B on `stream`; A, B, C are device addresses (ints)."""
    _ints(M=M, N=N, K=K, lda=lda, ldb=ldb, ldc=ldc)
    return load().gemm_f32(M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_f32_with_config(config, M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    _ints(config=config, M=M, N=N, K=K, lda=lda, ldb=ldb, ldc=ldc)
    return load().gemm_f32_with_config(config, M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_f32_num_configs() -> int:
    return load().gemm_f32_num_configs()


def gemm_f32_config_name(config: int) -> str:
    return load().gemm_f32_config_name(config).decode()


def gemm_f32_config_info(config: int, occupancy: bool = False) -> dict:
    """{'bm', 'bn', 'bk', 'threads'} (+ 'blocks_per_cu' if occupancy, needs a GPU)."""
    vals = [ctypes.c_int(0) for _ in range(5)]
    ptrs = [ctypes.byref(v) for v in vals]
    if not occupancy:
        ptrs[4] = None
    rc = load().gemm_f32_config_info(config, *ptrs)
    if rc != GEMM_F32_OK:
        raise GemmError(rc, "gemm_f32_config_info")
    out = dict(bm=vals[0].value, bn=vals[1].value, bk=vals[2].value, threads=vals[3].value)
    if occupancy:
        out["blocks_per_cu"] = vals[4].value
    return out


def gemm_f32_ws_size(M, N, K) -> int:
    """Workspace bytes the split-K plan for this shape needs (0: not split)."""
    _ints(M=M, N=N, K=K)
    return load().gemm_f32_ws_size(M, N, K)


def gemm_f32_ws(M, N, K, A, lda, B, ldb, C, ldc, workspace, workspace_bytes, stream=0) -> int:
    """C := A . B, split over K through `workspace` when the shape calls for it."""
    _ints(M=M, N=N, K=K, lda=lda, ldb=ldb, ldc=ldc)
    return load().gemm_f32_ws(M, N, K, A, lda, B, ldb, C, ldc, workspace, workspace_bytes, stream)


def gemm_f32_ws_noalloc(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    """C := A . B like gemm_f32_ws, split over K through the library's own
    static scratch (allocates nothing; overlapping calls on one GPU race)."""
    _ints(M=M, N=N, K=K, lda=lda, ldb=ldb, ldc=ldc)
    return load().gemm_f32_ws_noalloc(M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_f32_device_peak(device: int = 0) -> dict:
    """{'compute_units', 'clock_khz', 'tflops'}: the FP32 matrix-core peak derived
    from the device's properties (needs a GPU)."""
    cu, khz, tf = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_double(0.0)
    rc = load().gemm_f32_device_peak(device, ctypes.byref(cu), ctypes.byref(khz), ctypes.byref(tf))
    if rc != GEMM_F32_OK:
        raise GemmError(rc, "gemm_f32_device_peak")
    return dict(compute_units=cu.value, clock_khz=khz.value, tflops=tf.value)


def gemm_f32_describe(config, M, N, K, A, lda, B, ldb, C, ldc) -> tuple[int, str]:
    """(status, description) of what gemm_f32_with_config would enqueue."""
    _ints(config=config, M=M, N=N, K=K, lda=lda, ldb=ldb, ldc=ldc)
    buf = ctypes.create_string_buffer(256)
    rc = load().gemm_f32_describe(config, M, N, K, A, lda, B, ldb, C, ldc, buf, len(buf))
    return rc, buf.value.decode()


# --- include/gemm_f32_rows.h ------------------------------------------------
def gemm_f32_route(type, T, E, k, logits, ldl, bias, score, groups, keep_groups, group_top, normalize, scale,
                   weight, index, stream=0) -> int:
    """k of E experts for each of T rows of logits."""
    _ints(T=T, E=E, k=k, ldl=ldl, groups=groups, keep_groups=keep_groups, group_top=group_top)
    return load().gemm_f32_route(type, T, E, k, logits, ldl, bias, score, groups, keep_groups, group_top, normalize,
                                 scale, weight, index, stream)


def gemm_f32_route_grad(type, T, E, k, logits, ldl, score, normalize, scale, index, dweight, dlogits, lddl,
                        stream=0) -> int:
    """Gradient of the logits from that of gemm_f32_route's weights."""
    _ints(T=T, E=E, k=k, ldl=ldl, lddl=lddl)
    return load().gemm_f32_route_grad(type, T, E, k, logits, ldl, score, normalize, scale, index, dweight, dlogits,
                                      lddl, stream)


def gemm_f32_expert_map_ws_size(S, E) -> int:
    """Workspace bytes of gemm_f32_expert_map (0: none)."""
    _ints(S=S, E=E)
    return load().gemm_f32_expert_map_ws_size(S, E)


def gemm_f32_expert_map(S, E, index, offsets, order, position, workspace=0, workspace_bytes=0, stream=0) -> int:
    """Slots in the order of their experts."""
    _ints(S=S, E=E)
    return load().gemm_f32_expert_map(S, E, index, offsets, order, position, workspace, workspace_bytes, stream)


def gemm_f32_grouped(type, G, P, N, K, offsets, order, per_row, rows, X, ldx, W, ldw, stride_w, Y, ldy,
                     stream=0) -> int:
    """Y(p,:) = X(r(p),:) . W_g for every place p of group g."""
    _ints(G=G, P=P, N=N, K=K, per_row=per_row, rows=rows, ldx=ldx, ldw=ldw, ldy=ldy)
    return load().gemm_f32_grouped(type, G, P, N, K, offsets, order, per_row, rows, X, ldx, W, ldw, stride_w, Y, ldy,
                                   stream)


def gemm_f32_grouped_grad_x(type, G, P, N, K, offsets, dY, lddy, W, ldw, stride_w, dX, lddx, stream=0) -> int:
    """dX(p,:) = dY(p,:) . W_g^T."""
    _ints(G=G, P=P, N=N, K=K, lddy=lddy, ldw=ldw, lddx=lddx)
    return load().gemm_f32_grouped_grad_x(type, G, P, N, K, offsets, dY, lddy, W, ldw, stride_w, dX, lddx, stream)


def gemm_f32_grouped_grad_w(type, G, P, N, K, offsets, order, per_row, rows, X, ldx, dY, lddy, dW, lddw, stride_dw,
                            stream=0) -> int:
    """dW_g = sum over group g's places of X(r(p),:)^T . dY(p,:)."""
    _ints(G=G, P=P, N=N, K=K, per_row=per_row, rows=rows, ldx=ldx, lddy=lddy, lddw=lddw)
    return load().gemm_f32_grouped_grad_w(type, G, P, N, K, offsets, order, per_row, rows, X, ldx, dY, lddy, dW, lddw,
                                          stride_dw, stream)


def gemm_f32_combine(type, T, k, N, P, position, weight, Y, ldy, out, ldo, stream=0) -> int:
    """out(t,:) = sum over j of weight * Y(position,:)."""
    _ints(T=T, k=k, N=N, P=P, ldy=ldy, ldo=ldo)
    return load().gemm_f32_combine(type, T, k, N, P, position, weight, Y, ldy, out, ldo, stream)


def gemm_f32_combine_grad(type, T, k, N, P, position, weight, Y, ldy, dout, lddo, dY, lddy, dweight, stream=0) -> int:
    """Gradients of gemm_f32_combine: of Y and of the weights."""
    _ints(T=T, k=k, N=N, P=P, ldy=ldy, lddo=lddo, lddy=lddy)
    return load().gemm_f32_combine_grad(type, T, k, N, P, position, weight, Y, ldy, dout, lddo, dY, lddy, dweight,
                                        stream)


def gemm_f32_adapters_ws_size(type, T, N, K, R) -> int:
    """Workspace bytes of gemm_f32_adapters (0: none)."""
    _ints(T=T, N=N, K=K, R=R)
    return load().gemm_f32_adapters_ws_size(type, T, N, K, R)


def gemm_f32_adapters(type, T, N, K, R, n, X, ldx, W, ldw, A, lda, stride_a, B, ldb, stride_b, adapter, scale, Y, ldy,
                      workspace, workspace_bytes, stream=0) -> int:
    """Y(t,:) = X(t,:) . W + scale[a] * (X(t,:) . A_a) . B_a, a = adapter[t]."""
    _ints(T=T, N=N, K=K, R=R, n=n, ldx=ldx, ldw=ldw, lda=lda, ldb=ldb, ldy=ldy)
    return load().gemm_f32_adapters(type, T, N, K, R, n, X, ldx, W, ldw, A, lda, stride_a, B, ldb, stride_b, adapter,
                                    scale, Y, ldy, workspace, workspace_bytes, stream)


def gemm_f32_status_string(status: int) -> str:
    return load().gemm_f32_status_string(status).decode()


def config_names() -> list[str]:
    return [gemm_f32_config_name(c) for c in range(gemm_f32_num_configs())]


# --- torch convenience -------------------------------------------------------
def _row_major(t, rows: int, cols: int, name: str) -> int:
    """Leading dimension of a 2-D float32 CUDA tensor with unit column stride."""
    import torch
    if t.dtype != torch.float32 or t.dim() != 2 or not t.is_cuda:
        raise TypeError(f"{name} must be a 2-D float32 tensor on a GPU")
    if tuple(t.shape) != (rows, cols):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(rows, cols)}")
    s0, s1 = t.stride()
    if rows > 0 and cols > 1 and s1 != 1:
        raise ValueError(f"{name} must have unit column stride")
    if rows > 1 and s0 < cols:
        raise ValueError(f"{name} rows overlap")
    return max(s0 if rows > 1 else cols, cols, 1)


def matmul(A, B, out=None, config: int = -1, stream=None):
    """out = A @ B via gemm_f32 on the current (or given) torch stream."""
    import torch
    M, K = A.shape
    K2, N = B.shape
    if K2 != K:
        raise ValueError("inner dimensions differ")
    lda = _row_major(A, M, K, "A")
    ldb = _row_major(B, K, N, "B")
    _ints(M=M, N=N, K=K, lda=lda, ldb=ldb)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    ldc = _row_major(out, M, N, "out")
    if stream is None:
        stream = torch.cuda.current_stream(A.device)
    rc = gemm_f32_with_config(config, M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb,
                              out.data_ptr(), ldc, stream.cuda_stream)
    if rc != GEMM_F32_OK:
        raise GemmError(rc)
    return out


# --- torch convenience: products whose second matrix is chosen row by row -----
# Matrices are float32, bfloat16 or float16 tensors of one GPU with unit stride
# in their last dimension (rows may be further apart); index tensors are
# int32, weights float32, both contiguous.  Work is enqueued on `stream` (the
# tensors' device's current stream if None; one of that device), whichever device is current;
# outputs and workspaces are allocated under that stream.  A call that runs on
# another stream than the one its inputs were made on needs the caller's own
# synchronisation, and outputs passed in must not overlap inputs.
_types = None


def _type(t) -> int:
    global _types
    if _types is None or _lib is None:
        import torch
        load()
        _types = {torch.float32: GEMM_F32_TYPE_F32, torch.bfloat16: GEMM_F32_TYPE_BF16,
                  torch.float16: GEMM_F32_TYPE_F16}
    if t.dtype not in _types:
        raise TypeError(f"element type {t.dtype} is not float32, bfloat16 or float16")
    return _types[t.dtype]


def _matrix(t, name: str, like=None, shape=None) -> int:
    """Leading dimension of a matrix (or of a stack of them)."""
    if not t.is_cuda:
        raise TypeError(f"{name} must be on a GPU")
    if like is not None and (t.dtype != like.dtype or t.device != like.device):
        raise TypeError(f"{name} is {t.dtype} on {t.device}, expected {like.dtype} on {like.device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    rows, cols = t.shape[-2], t.shape[-1]
    s0, s1 = t.stride()[-2:]
    if rows > 0 and cols > 1 and s1 != 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    if rows > 1 and s0 < cols:
        raise ValueError(f"{name} rows overlap")
    return max(s0 if rows > 1 else cols, cols, 1)


def _stack(t, name: str, ld: int) -> int:
    """Elements between the matrices of a stack [n, rows, cols]."""
    need = t.shape[1] * ld
    if t.shape[0] <= 1:
        return need
    s = t.stride(0)
    if s < need:
        # a last row that ends before the leading dimension does is no overlap,
        # but the C ABI asks for whole rows between matrices
        raise ValueError(f"{name}'s matrices are {s} elements apart, need at least {need}")
    return s


def _vector(t, name: str, dtype, device, shape) -> int:
    """Address of a contiguous tensor of numbers that goes with the matrices."""
    if t.dtype != dtype or t.device != device:
        raise TypeError(f"{name} is {t.dtype} on {t.device}, expected {dtype} on {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


_current_device = _current_raw_stream = None


def _here(device) -> int:
    """The current stream of `device`, the current device (a HIP stream address)."""
    global _current_device, _current_raw_stream
    if _current_raw_stream is None:                  # the last one set: other threads may be here too
        import torch
        _current_device = torch.cuda.current_device
        # the raw address, without the Stream object around it where torch offers it
        _current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                      lambda index: torch.cuda.current_stream(index).cuda_stream)
    return _current_raw_stream(device.index)


def _elsewhere(device, stream) -> bool:
    """Whether a call has to be made under another device or stream than the current ones."""
    return stream is not None or (_current_device or _device_now)() != device.index


def _device_now() -> int:
    import torch
    return torch.cuda.current_device()


def _call_on(device, stream, fn, *args, **kwargs):
    """fn with the tensors' device and the given stream (of that device) made current."""
    import torch
    if stream is not None and stream.device != device:
        raise ValueError(f"the stream is one of {stream.device}, the tensors are on {device}")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        return fn(*args, **kwargs)


def _fit(*sizes):
    """Refuses sizes that a C int cannot hold (ctypes would wrap them)."""
    for size in (max(sizes), min(sizes)):
        if not INT32_MIN <= size <= INT32_MAX:
            raise ValueError(f"size {size} does not fit the C ABI's 32-bit int")


def _check(rc: int, what: str):
    if rc != GEMM_F32_OK:
        raise GemmError(rc, what)


def _score(score: str) -> int:
    if score == "softmax":
        return GEMM_F32_SCORE_SOFTMAX
    if score == "sigmoid":
        return GEMM_F32_SCORE_SIGMOID
    raise ValueError(f"score {score!r} is neither 'softmax' nor 'sigmoid'")


def route(logits, k: int, *, bias=None, score: str = "softmax", groups: int = 1, keep_groups: int = 1,
          group_top: int = 1, normalize: bool = False, scale: float = 1.0, stream=None):
    """(weight [T, k] float32, index [T, k] int32): the k experts of each row of logits [T, E].

    Scores are the row's softmax or sigmoid; bias [E] (float32) is added for
    the choice only.  With groups > 1 only the keep_groups groups with the largest sum
    of their group_top best biased scores stay.  `normalize` divides a row's
    weights by their sum, `scale` multiplies them.  An expert whose logit or bias is
    -inf is not available; index is -1 (weight 0) where fewer than k are.
    """
    import torch
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    type_, ldl, mode = _type(logits), _matrix(logits, "logits"), _score(score)
    device = logits.device
    if _elsewhere(device, stream):
        return _call_on(device, stream, route, logits, k, bias=bias, score=score, groups=groups,
                        keep_groups=keep_groups, group_top=group_top, normalize=normalize, scale=scale)
    T, E = logits.shape
    _fit(T, E, k, ldl, groups, keep_groups, group_top)
    b = 0 if bias is None else _vector(bias, "bias", torch.float32, device, (E,))
    weight = logits.new_empty((T, max(k, 0)), dtype=torch.float32)
    index = logits.new_empty((T, max(k, 0)), dtype=torch.int32)
    _check(_lib.gemm_f32_route(type_, T, E, k, logits.data_ptr(), ldl, b, mode, groups, keep_groups, group_top,
                               bool(normalize), scale, weight.data_ptr(), index.data_ptr(), _here(device)),
           "gemm_f32_route")
    return weight, index


def route_grad(logits, index, dweight, *, score: str = "softmax", normalize: bool = False, scale: float = 1.0,
               out=None, stream=None):
    """Gradient [T, E] of the logits, in their type, from that of route()'s weights."""
    import torch
    if logits.dim() != 2 or index.dim() != 2:
        raise ValueError("logits must be [T, E] and index [T, k]")
    type_, ldl, mode = _type(logits), _matrix(logits, "logits"), _score(score)
    device = logits.device
    if _elsewhere(device, stream):
        return _call_on(device, stream, route_grad, logits, index, dweight, score=score, normalize=normalize,
                        scale=scale, out=out)
    T, E = logits.shape
    k = index.shape[1]
    i = _vector(index, "index", torch.int32, device, (T, k))
    w = _vector(dweight, "dweight", torch.float32, device, (T, k))
    if out is None:
        out = logits.new_empty((T, E))
    ldo = _matrix(out, "out", logits, (T, E))
    _fit(T, E, k, ldl, ldo)
    _check(_lib.gemm_f32_route_grad(type_, T, E, k, logits.data_ptr(), ldl, mode, bool(normalize), scale, i, w,
                                    out.data_ptr(), ldo, _here(device)), "gemm_f32_route_grad")
    return out


def expert_map(index, experts: int, *, stream=None):
    """(offsets [experts + 1], order [S], position like index): slots by expert.

    Slot s is the s-th element of index (int32, any shape).  Places
    offsets[e] .. offsets[e + 1] of order hold the slots of expert e in rising
    order; position is each slot's place.  Slots whose expert is outside 0 .. experts - 1
    are left out: position -1, and -1 at the end of order.
    """
    import torch
    if not index.is_cuda:
        raise TypeError("index must be on a GPU")
    device = index.device
    i = _vector(index, "index", torch.int32, device, index.shape)
    if _elsewhere(device, stream):
        return _call_on(device, stream, expert_map, index, experts)
    S = index.numel()
    need = gemm_f32_expert_map_ws_size(S, experts)
    offsets = index.new_empty(max(experts, 0) + 1)
    order = index.new_empty(S)
    position = torch.empty_like(index)
    ws = index.new_empty(need, dtype=torch.uint8) if need else None
    _check(_lib.gemm_f32_expert_map(S, experts, i, offsets.data_ptr(), order.data_ptr(), position.data_ptr(),
                                    ws.data_ptr() if need else 0, need, _here(device)), "gemm_f32_expert_map")
    return offsets, order, position


def _grouped_args(X, offsets, order):
    """What forward and weight gradient have in common: places, rows, addresses."""
    import torch
    G = offsets.numel() - 1
    if G < 0:
        raise ValueError("offsets must have one number more than there are groups")
    o = _vector(offsets, "offsets", torch.int32, X.device, (G + 1,))
    if order is None:
        return G, X.shape[0], o, 0
    return G, order.numel(), o, _vector(order, "order", torch.int32, X.device, (order.numel(),))


def grouped_matmul(X, W, offsets, *, order=None, per_row: int = 1, out=None, stream=None):
    """Y [P, N]: rows of X times the matrix W[g] ([G, K, N]) of the group their place is in.

    Place p is in group g when offsets[g] <= p < offsets[g + 1].  Its row of
    X is p, or order[p] // per_row (expert_map's order, and k choices per
    row).  Rows of `out` in no group are left as they were.
    """
    import torch
    if X.dim() != 2 or W.dim() != 3:
        raise ValueError("X must be [rows, K] and W [G, K, N]")
    type_, ldx = _type(X), _matrix(X, "X")
    device = X.device
    if _elsewhere(device, stream):
        return _call_on(device, stream, grouped_matmul, X, W, offsets, order=order, per_row=per_row, out=out)
    G, P, o, r = _grouped_args(X, offsets, order)
    rows, K = X.shape
    N = W.shape[2]
    ldw = _matrix(W, "W", X, (G, K, N))
    stride = _stack(W, "W", ldw)
    if out is None:
        out = X.new_empty((P, N))
    ldy = _matrix(out, "out", X, (P, N))
    _fit(G, P, N, K, per_row, rows, ldx, ldw, ldy)
    _check(_lib.gemm_f32_grouped(type_, G, P, N, K, o, r, per_row, rows, X.data_ptr(), ldx, W.data_ptr(), ldw, stride,
                                 out.data_ptr(), ldy, _here(device)), "gemm_f32_grouped")
    return out


def grouped_grad_x(dY, W, offsets, *, out=None, stream=None):
    """dX [P, K] of grouped_matmul's places: rows of dY [P, N] times W[g]^T.

    With an order, the gradient of X is combine(dX, position) over a row's places.
    """
    import torch
    if dY.dim() != 2 or W.dim() != 3:
        raise ValueError("dY must be [P, N] and W [G, K, N]")
    type_, lddy = _type(dY), _matrix(dY, "dY")
    device = dY.device
    if _elsewhere(device, stream):
        return _call_on(device, stream, grouped_grad_x, dY, W, offsets, out=out)
    G, P, o, _ = _grouped_args(dY, offsets, None)
    N, K = dY.shape[1], W.shape[1]
    ldw = _matrix(W, "W", dY, (G, K, N))
    stride = _stack(W, "W", ldw)
    if out is None:
        out = dY.new_empty((P, K))
    lddx = _matrix(out, "out", dY, (P, K))
    _fit(G, P, N, K, lddy, ldw, lddx)
    _check(_lib.gemm_f32_grouped_grad_x(type_, G, P, N, K, o, dY.data_ptr(), lddy, W.data_ptr(), ldw, stride,
                                        out.data_ptr(), lddx, _here(device)), "gemm_f32_grouped_grad_x")
    return out


def grouped_grad_w(X, dY, offsets, *, order=None, per_row: int = 1, out=None, stream=None):
    """dW [G, K, N] of grouped_matmul from the gradient dY [P, N] of its places."""
    import torch
    if X.dim() != 2 or dY.dim() != 2:
        raise ValueError("X must be [rows, K] and dY [P, N]")
    type_, ldx = _type(X), _matrix(X, "X")
    device = X.device
    if _elsewhere(device, stream):
        return _call_on(device, stream, grouped_grad_w, X, dY, offsets, order=order, per_row=per_row, out=out)
    G, P, o, r = _grouped_args(X, offsets, order)
    rows, K = X.shape
    N = dY.shape[1]
    lddy = _matrix(dY, "dY", X, (P, N))
    if out is None:
        out = X.new_empty((G, K, N))
    lddw = _matrix(out, "out", X, (G, K, N))
    stride = _stack(out, "out", lddw)
    _fit(G, P, N, K, per_row, rows, ldx, lddy, lddw)
    _check(_lib.gemm_f32_grouped_grad_w(type_, G, P, N, K, o, r, per_row, rows, X.data_ptr(), ldx, dY.data_ptr(), lddy,
                                        out.data_ptr(), lddw, stride, _here(device)), "gemm_f32_grouped_grad_w")
    return out


def combine(Y, position, weight=None, *, out=None, stream=None):
    """out [T, N]: for each row of position [T, k] the sum of weight [T, k] times rows of Y [P, N].

    Positions outside 0 .. P - 1 add nothing; weight None: 1.
    """
    import torch
    if Y.dim() != 2 or position.dim() != 2:
        raise ValueError("Y must be [P, N] and position [T, k]")
    type_, ldy = _type(Y), _matrix(Y, "Y")
    device = Y.device
    if _elsewhere(device, stream):
        return _call_on(device, stream, combine, Y, position, weight, out=out)
    P, N = Y.shape
    T, k = position.shape
    at = _vector(position, "position", torch.int32, device, (T, k))
    w = 0 if weight is None else _vector(weight, "weight", torch.float32, device, (T, k))
    if out is None:
        out = Y.new_empty((T, N))
    ldo = _matrix(out, "out", Y, (T, N))
    _fit(T, k, N, P, ldy, ldo)
    _check(_lib.gemm_f32_combine(type_, T, k, N, P, at, w, Y.data_ptr(), ldy, out.data_ptr(), ldo, _here(device)),
           "gemm_f32_combine")
    return out


def combine_grad(dout, Y, position, weight=None, *, out=None, stream=None):
    """[dY [P, N], dweight [T, k]] of combine() from dout [T, N].

    Rows of dY that no position names are left as they were in `out` (undefined if it is None).
    """
    import torch
    if Y.dim() != 2 or position.dim() != 2:
        raise ValueError("Y must be [P, N] and position [T, k]")
    type_, ldy = _type(Y), _matrix(Y, "Y")
    device = Y.device
    if _elsewhere(device, stream):
        return _call_on(device, stream, combine_grad, dout, Y, position, weight, out=out)
    P, N = Y.shape
    T, k = position.shape
    lddo = _matrix(dout, "dout", Y, (T, N))
    at = _vector(position, "position", torch.int32, device, (T, k))
    w = 0 if weight is None else _vector(weight, "weight", torch.float32, device, (T, k))
    if out is None:
        out = Y.new_empty((P, N))
    lddy = _matrix(out, "out", Y, (P, N))
    dweight = Y.new_empty((T, k), dtype=torch.float32)
    _fit(T, k, N, P, ldy, lddo, lddy)
    _check(_lib.gemm_f32_combine_grad(type_, T, k, N, P, at, w, Y.data_ptr(), ldy, dout.data_ptr(), lddo,
                                      out.data_ptr(), lddy, dweight.data_ptr(), _here(device)),
           "gemm_f32_combine_grad")
    return [out, dweight]


def adapter_matmul(X, W, A, B, adapter, scale=None, *, out=None, workspace=None, stream=None):
    """Y [T, N] = X W, plus scale[a] (X A[a]) B[a] for each row's adapter a = adapter[t].

    X [T, K], W [K, N], A [n, K, R], B [n, R, N], adapter [T] int32 (outside
    0 .. n - 1: none), scale [n] float32 or None (1).  `workspace` is a uint8
    tensor of at least gemm_f32_adapters_ws_size bytes, allocated if None.
    """
    import torch
    if X.dim() != 2 or W.dim() != 2 or A.dim() != 3 or B.dim() != 3:
        raise ValueError("X must be [T, K], W [K, N], A [n, K, R] and B [n, R, N]")
    type_, ldx = _type(X), _matrix(X, "X")
    device = X.device
    if _elsewhere(device, stream):
        return _call_on(device, stream, adapter_matmul, X, W, A, B, adapter, scale, out=out, workspace=workspace)
    T, K = X.shape
    N, n, R = W.shape[1], A.shape[0], A.shape[2]
    ldw, lda, ldb = _matrix(W, "W", X, (K, N)), _matrix(A, "A", X, (n, K, R)), _matrix(B, "B", X, (n, R, N))
    sa, sb = _stack(A, "A", lda), _stack(B, "B", ldb)
    a = _vector(adapter, "adapter", torch.int32, device, (T,))
    c = 0 if scale is None else _vector(scale, "scale", torch.float32, device, (n,))
    if out is None:
        out = X.new_empty((T, N))
    ldy = _matrix(out, "out", X, (T, N))
    _fit(T, N, K, R, n, ldx, ldw, lda, ldb, ldy)
    if workspace is None:
        workspace = X.new_empty(_lib.gemm_f32_adapters_ws_size(type_, T, N, K, R), dtype=torch.uint8)
    elif workspace.dtype != torch.uint8 or workspace.device != device or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous uint8 tensor on the operands' device")
    _check(_lib.gemm_f32_adapters(type_, T, N, K, R, n, X.data_ptr(), ldx, W.data_ptr(), ldw, A.data_ptr(), lda, sa,
                                  B.data_ptr(), ldb, sb, a, c, out.data_ptr(), ldy, workspace.data_ptr(),
                                  workspace.numel(), _here(device)), "gemm_f32_adapters")
    return out
