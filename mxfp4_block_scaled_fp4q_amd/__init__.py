"""Python binding of libfp4q, the block-scaled MXFP4 linear-layer hot path for
AMD MI355X (gfx950).

Argument marshalling only: every step runs in the HIP kernels behind the C ABI
declared in ``include/libfp4q.h``; torch supplies device memory and the
current stream.  There is no fallback: if ``libfp4q.so`` has not been built,
loading the library raises.
"""
import ctypes as _ct
import os as _os

_HERE = _os.path.dirname(_os.path.abspath(__file__))
LIB_PATH = _os.path.join(_HERE, "libfp4q.so")

F32, BF16 = 0, 1
ROW, COL = 0, 1
RNE, SR = 0, 1
STE, DGE = 0, 1
SILU, GELU = 0, 1
LAYER_NORM, RMS_NORM = 0, 1

STATUS = {0: "FP4Q_OK", 1: "FP4Q_ERR_INVALID", 2: "FP4Q_ERR_UNSUPPORTED",
          3: "FP4Q_ERR_ALIGNMENT", 4: "FP4Q_ERR_WORKSPACE", 5: "FP4Q_ERR_HIP"}

EXPORTS = ["fp4q_channel_mask", "fp4q_quantize_masked", "fp4q_gemm_hcp_split",
           "fp4q_quantize", "fp4q_quantize_dual", "fp4q_dequantize", "fp4q_grad_estimate",
           "fp4q_gemm",
           "fp4q_gemm_dge", "fp4q_gemm_quant", "fp4q_hcp_workspace_bytes",
           "fp4q_hcp_residual_add", "fp4q_hcp_residual_add_noalloc",
           "fp4q_gemm_hcp", "fp4q_hot_channels_workspace_bytes", "fp4q_hot_channels",
           "fp4q_quantize_2d", "fp4q_quantize_2d_tile", "fp4q_quantize_rht", "fp4q_occ_max_nnz",
           "fp4q_occ_workspace_bytes", "fp4q_occ_quantize", "fp4q_occ_spmm",
           "fp4q_gemm_gated", "fp4q_gemm_gated_grad", "fp4q_layer_norm",
           "fp4q_layer_norm_grad_workspace_bytes", "fp4q_layer_norm_grad", "fp4q_adamw_step",
           "fp4q_adamw_table", "fp4q_adamw_step_table",
           "fp4q_set_next_launch", "fp4q_status_string",
           "fp4q_last_error", "fp4q_abi_version"]


class Fp4qError(RuntimeError):
    def __init__(self, status, detail):
        super().__init__(f"{STATUS.get(status, status)}: {detail}")
        self.status = status


class AdamwTensor(_ct.Structure):
    """One tensor of an AdamW step (fp4q_adamw_tensor_t)."""
    _fields_ = [("param", _ct.c_void_p), ("grad", _ct.c_void_p), ("exp_avg", _ct.c_void_p),
                ("exp_avg_sq", _ct.c_void_p), ("exp_avg_scales", _ct.c_void_p),
                ("exp_avg_sq_scales", _ct.c_void_p), ("copy", _ct.c_void_p),
                ("numel", _ct.c_int64), ("weight_decay", _ct.c_double)]


_lib = None


def lib():
    """Load libfp4q.so (raises if it is not built)."""
    global _lib
    if _lib is None:
        if not _os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run "
                              "mxfp4_block_scaled_fp4q_amd/build.py (or __graft_entry__.build())")
        L = _ct.CDLL(LIB_PATH)
        P, I64, I32, U64, F, SZ, D = (_ct.c_void_p, _ct.c_int64, _ct.c_int32, _ct.c_uint64,
                                      _ct.c_float, _ct.c_size_t, _ct.c_double)
        sig = {
            "fp4q_quantize": (I32, [P, I32, I64, I64, I64, I32, I32, I32, U64, U64, P, P, P]),
            "fp4q_quantize_dual": (I32, [P, I32, I64, I64, I64, I32, I32, U64, I32, U64, U64, P, P,
                                         P, P, P]),
            "fp4q_dequantize": (I32, [P, P, I64, I64, I32, P, I32, P]),
            "fp4q_grad_estimate": (I32, [I32, P, I32, P, I32, I64, I64, I32, I32, F, F, P, I32,
                                         P]),
            "fp4q_gemm": (I32, [I64, I64, I64, P, P, P, P, I32, P, I32, I64, I32, P]),
            "fp4q_hcp_workspace_bytes": (SZ, [I64, I64, I32]),
            "fp4q_hcp_residual_add": (I32, [I64, I64, I64, P, P, P, P, P, P, P, I32, P, P, SZ,
                                            P]),
            "fp4q_hcp_residual_add_noalloc": (I32, [I64, I64, I64, P, P, P, P, P, P, P, I32, P,
                                                    P]),
            "fp4q_gemm_dge": (I32, [I64, I64, I64, P, P, P, P, P, I32, F, F, P, I64, P]),
            "fp4q_gemm_quant": (I32, [I64, I64, I64, P, P, P, P, P, I64, P, P, P]),
            "fp4q_channel_mask": (I32, [P, I32, I64, P, P]),
            "fp4q_quantize_masked": (I32, [P, I32, I64, I64, I64, I32, I32, I32, U64, U64, P, P,
                                           P, P]),
            "fp4q_gemm_hcp_split": (I32, [I64, I64, I64, P, P, P, P, P, P, P, I32, P, I64, P, SZ,
                                          P]),
            "fp4q_gemm_hcp": (I32, [I64, I64, I64, P, P, P, P, P, P, P, I32, P, I64, P, SZ, P]),
            "fp4q_hot_channels_workspace_bytes": (SZ, [I64, I64]),
            "fp4q_quantize_2d": (I32, [P, I64, I64, I64, I32, U64, U64, P, P, P, P, P]),
            "fp4q_quantize_2d_tile": (I32, [P, I64, I64, I64, I32, I32, U64, U64, P, P, P, P, P]),
            "fp4q_quantize_rht": (I32, [P, I64, I64, I64, I32, P, I32, U64, U64, P, P, P]),
            "fp4q_occ_max_nnz": (I64, [I64, I64, _ct.c_double]),
            "fp4q_occ_workspace_bytes": (SZ, [I64, I64]),
            "fp4q_occ_quantize": (I32, [P, I64, I64, I64, _ct.c_double, I32, U64, U64, P, P, P, P,
                                        P, I64, P, P, SZ, P]),
            "fp4q_occ_spmm": (I32, [I64, I64, I64, P, P, P, P, I64, P, I64, P]),
            "fp4q_hot_channels": (I32, [P, I64, I64, I64, I32, P, P, P, SZ, P]),
            "fp4q_gemm_gated": (I32, [I64, I64, I64, P, P, P, P, P, P, I32, P, I64, P, P, I64,
                                      P]),
            "fp4q_gemm_gated_grad": (I32, [I64, I64, I64, P, P, P, P, I32, P, P, I64, P, P, I64,
                                           P]),
            "fp4q_layer_norm": (I32, [I32, P, I32, I64, I64, I64, P, P, I32, D, P, I32, I64, P, P,
                                      P]),
            "fp4q_layer_norm_grad_workspace_bytes": (SZ, [I64, I64]),
            "fp4q_layer_norm_grad": (I32, [I32, P, I32, I64, P, I32, I64, I64, I64, P, I32, P, P,
                                           P, I64, P, P, P, SZ, P]),
            "fp4q_adamw_step": (I32, [P, I32, I32, I32, D, D, D, D, I64, U64, P, P]),
            "fp4q_adamw_table": (I32, [P, I32, I32, P, P, P]),
            "fp4q_adamw_step_table": (I32, [P, I32, I64, I32, I32, D, D, D, D, I64, U64, P, P]),
            "fp4q_set_next_launch": (I32, [P, P, _ct.c_uint32]),
            "fp4q_status_string": (_ct.c_char_p, [I32]),
            "fp4q_last_error": (_ct.c_char_p, []),
            "fp4q_abi_version": (I32, []),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(status):
    if status != 0:
        raise Fp4qError(status, lib().fp4q_last_error().decode())


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _dt(t):
    torch = _torch_module or _torch()
    if t.dtype is torch.bfloat16:
        return BF16
    if t.dtype is torch.float32:
        return F32
    raise TypeError(f"libfp4q takes bf16 or fp32 tensors, got {t.dtype}")


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    c = (_torch_module or _torch())._C
    # the current stream's handle, without building a Stream object per call
    return c._cuda_getCurrentRawStream(c._cuda_getDevice())


_empty_strided_cuda = None


def _allocator(t, stream):
    """An f(size, stride, dtype) that makes uninitialised contiguous tensors on
    t's device: torch's shortest way to one where this torch has it and the
    device is the current one (0.7 us a tensor against 1.4), else new_empty.
    The short way passes the dispatcher by, so it is not taken where a dispatch
    mode watches or deterministic algorithms ask for memory that is filled.

    The tensors belong to `stream`, which the call's kernels run on: memory of
    the current stream's pool may still be in use by that stream's pending work,
    and would go back there when a result is dropped, written or not.  They are
    recorded on the current stream, where the caller may read them."""
    global _empty_strided_cuda
    if stream is not None:
        cuda = _torch().cuda
        current = cuda.current_stream()
        if current.cuda_stream != stream.cuda_stream:
            def on_stream(size, stride, dtype):
                with cuda.stream(stream):
                    out = t.new_empty(size, dtype=dtype)
                out.record_stream(current)
                return out
            return on_stream
    c = (_torch_module or _torch())._C
    if _empty_strided_cuda is None:
        guards = getattr(getattr(c, "_dynamo", None), "guards", None)
        _empty_strided_cuda = (hasattr(c, "_len_torch_dispatch_stack")
                               and getattr(guards, "_empty_strided_cuda", False))
    if (_empty_strided_cuda and t.get_device() == c._cuda_getDevice()
            and not c._len_torch_dispatch_stack() and not c._get_deterministic_algorithms()):
        return _empty_strided_cuda
    return lambda size, stride, dtype: t.new_empty(size, dtype=dtype)


def _halves(empty, rows, cols, dtype):
    """The two [rows, cols] halves of one [rows, 2 cols] tensor that `empty`
    (an _allocator) makes."""
    ld = 2 * cols
    both = empty((rows, ld), (ld, 1), dtype)
    return both.as_strided((rows, cols), (ld, 1)), both.as_strided((rows, cols), (ld, 1), cols)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("libfp4q takes device (cuda) tensors")


def _need(t, name, dtype, shape=None, dense=True):
    """Raise unless t has the dtype (and shape) the C call reads it as and,
    with dense, is contiguous (the C call takes no strides for it)."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _scratch(nbytes, device, stream):
    """Caller-less workspace for one call: allocated from torch's pool and,
    when the kernels run on a stream other than the current one, recorded on
    that stream so the pool does not hand the block to other work before
    those kernels finish."""
    torch = _torch()
    ws = torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)
    if stream is not None:
        ws.record_stream(stream)
    return ws


def _hcp_operands(x, xq_codes, xq_scales, w, wq_codes, wq_scales, hot_idx):
    """Shapes and dtypes of the hot-channel calls' operands; returns M, N, K."""
    torch = _torch()
    _need_cuda(x, xq_codes, xq_scales, w, wq_codes, wq_scales, hot_idx)
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x and w must be 2-D")
    M, K = x.shape
    N = w.shape[1]
    _need(x, "x", torch.bfloat16)
    _need(w, "w", torch.bfloat16, (K, N))
    _need(xq_codes, "xq_codes", torch.uint8, (M, K // 2))
    _need(xq_scales, "xq_scales", torch.uint8, (M, K // 32))
    _need(wq_codes, "wq_codes", torch.uint8, (N, K // 2))
    _need(wq_scales, "wq_scales", torch.uint8, (N, K // 32))
    _need(hot_idx, "hot_idx", torch.int32)
    if hot_idx.dim() != 1:
        raise ValueError("hot_idx must be 1-D")
    return M, N, K


def quantize(x, block=32, axis=ROW, rounding=RNE, seed=0, rng_offset=0, codes=None, scales=None,
             stream=None):
    """Fused MXFP4 quantisation of a 2-D bf16/fp32 tensor (row stride from x).
    Returns (codes uint8, scales uint8): ROW -> [R, C/2], [R, C/block];
    COL -> [C, R/2], [C, R/block] (the K-major quantisation of x^T)."""
    torch = _torch()
    _need_cuda(x)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    rows, cols = x.shape
    if axis == ROW:
        cshape, sshape = (rows, cols // 2), (rows, cols // block)
    else:
        cshape, sshape = (cols, rows // 2), (cols, rows // block)
    if codes is None:
        codes = torch.empty(cshape, dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(sshape, dtype=torch.uint8, device=x.device)
    _check(lib().fp4q_quantize(_ptr(x), _dt(x), rows, cols, x.stride(0), block, axis, rounding,
                               seed, rng_offset, _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


def quantize_dual(x, block=32, round_row=RNE, seed_row=0, round_col=RNE, seed_col=0,
                  rng_offset=0, out=None, stream=None):
    """Both orientations in one pass: returns ((row codes, row scales),
    (col codes, col scales)), identical to quantize(x, block, ROW, round_row,
    seed_row, rng_offset) and quantize(x, block, COL, round_col, seed_col,
    rng_offset).  `out` may give the four output tensors."""
    torch = _torch()
    _need_cuda(x)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    rows, cols = x.shape
    if out is None:
        u8 = dict(dtype=torch.uint8, device=x.device)
        out = (torch.empty((rows, cols // 2), **u8), torch.empty((rows, cols // block), **u8),
               torch.empty((cols, rows // 2), **u8), torch.empty((cols, rows // block), **u8))
    rc, rs, cc, cs = out
    _check(lib().fp4q_quantize_dual(_ptr(x), _dt(x), rows, cols, x.stride(0), block, round_row,
                                    seed_row, round_col, seed_col, rng_offset, _ptr(rc), _ptr(rs),
                                    _ptr(cc), _ptr(cs), _stream(stream)))
    return (rc, rs), (cc, cs)


def dequantize(codes, scales, block=32, out_dtype=None, out=None, stream=None):
    """codes [R, K/2] + scales [R, K/block] -> dense [R, K] bf16 (default) or fp32."""
    torch = _torch()
    _need_cuda(codes, scales)
    rows, k = codes.shape[0], codes.shape[1] * 2
    if out is None:
        out = torch.empty((rows, k), dtype=out_dtype or torch.bfloat16, device=codes.device)
    _check(lib().fp4q_dequantize(_ptr(codes), _ptr(scales), rows, k, block, _ptr(out), _dt(out),
                                 _stream(stream)))
    return out


def grad_estimate(mode, x, grad, block=32, axis=ROW, k=5.0, clamp_max=3.0, out_dtype=None,
                  out=None, stream=None):
    """STE (mode 0) or DGE (mode 1) backward of the quantiser: out = grad * d."""
    torch = _torch()
    _need_cuda(x, grad)
    rows, cols = grad.shape
    if out is None:
        out = torch.empty((rows, cols), dtype=out_dtype or grad.dtype, device=grad.device)
    xdt = _dt(x) if x is not None else F32
    _check(lib().fp4q_grad_estimate(mode, _ptr(x), xdt, _ptr(grad), _dt(grad), rows, cols, block,
                                    axis, float(k), float(clamp_max), _ptr(out), _dt(out),
                                    _stream(stream)))
    return out


def gemm(a_codes, a_scales, b_codes, b_scales, out_dtype=None, c=None, accumulate=False,
         block=32, stream=None):
    """C[M,N] (+)= deq(A) deq(B)^T with A [M, K/2]+[M, K/32], B [N, K/2]+[N, K/32]."""
    torch = _torch()
    _need_cuda(a_codes, a_scales, b_codes, b_scales)
    M, N, K = a_codes.shape[0], b_codes.shape[0], a_codes.shape[1] * 2
    if b_codes.shape[1] * 2 != K:
        raise ValueError("A and B K dimensions differ")
    if c is None:
        c = torch.empty((M, N), dtype=out_dtype or torch.bfloat16, device=a_codes.device)
    _check(lib().fp4q_gemm(M, N, K, _ptr(a_codes), _ptr(a_scales), _ptr(b_codes),
                           _ptr(b_scales), block, _ptr(c), _dt(c), c.stride(0),
                           1 if accumulate else 0, _stream(stream)))
    return c


ANY_ORDER = 1


def set_next_launch(start_event=None, stop_event=None, any_order=False):
    """Options for the next kernel this thread launches through the library:
    hipEvent_t handles (ints or ctypes pointers, or None) that its dispatch
    records at its start and end, and whether it may start before earlier
    work on its stream has finished (the caller vouches that it does not
    depend on that work)."""
    _check(lib().fp4q_set_next_launch(start_event, stop_event, ANY_ORDER if any_order else 0))


def hcp_workspace_bytes(M, N, n_hot):
    return int(lib().fp4q_hcp_workspace_bytes(M, N, n_hot))


def hcp_residual_add(x, xq_codes, xq_scales, w, wq_codes, wq_scales, hot_idx, y, workspace=None,
                     stream=None):
    """y[M,N] (fp32, in place) += sum_{c in hot} X[:,c] W[c,:] - Xq[:,c] Wq[c,:]."""
    torch = _torch()
    M, N, K = _hcp_operands(x, xq_codes, xq_scales, w, wq_codes, wq_scales, hot_idx)
    _need_cuda(y)
    _need(y, "y", torch.float32, (M, N))
    n_hot = hot_idx.numel()
    if workspace is None:
        workspace = _scratch(hcp_workspace_bytes(M, N, n_hot), x.device, stream)
    _check(lib().fp4q_hcp_residual_add(M, N, K, _ptr(x), _ptr(xq_codes), _ptr(xq_scales), _ptr(w),
                                       _ptr(wq_codes), _ptr(wq_scales), _ptr(hot_idx), n_hot,
                                       _ptr(y), _ptr(workspace), workspace.numel(),
                                       _stream(stream)))
    return y


HCP_NOALLOC_MAX_BYTES = 64 << 20


def hcp_residual_add_noalloc(x, xq_codes, xq_scales, w, wq_codes, wq_scales, hot_idx, y,
                             stream=None):
    """hcp_residual_add without a workspace (fp4q_hcp_residual_add_noalloc):
    the library's own 64 MiB device scratch holds the gathered operands;
    nothing is allocated.  Calls overlapping on one GPU race."""
    torch = _torch()
    M, N, K = _hcp_operands(x, xq_codes, xq_scales, w, wq_codes, wq_scales, hot_idx)
    _need_cuda(y)
    _need(y, "y", torch.float32, (M, N))
    _check(lib().fp4q_hcp_residual_add_noalloc(M, N, K, _ptr(x), _ptr(xq_codes), _ptr(xq_scales),
                                               _ptr(w), _ptr(wq_codes), _ptr(wq_scales),
                                               _ptr(hot_idx), hot_idx.numel(), _ptr(y),
                                               _stream(stream)))
    return y


def gemm_hcp(x, xq_codes, xq_scales, w, wq_codes, wq_scales, hot_idx, y=None, workspace=None,
             stream=None):
    """Y[M,N] (fp32) = Xq Wq + sum_{c in hot} X[:,c] W[c,:] - Xq[:,c] Wq[c,:], in one GEMM
    kernel (fp4q_gemm_hcp); returns y."""
    torch = _torch()
    M, N, K = _hcp_operands(x, xq_codes, xq_scales, w, wq_codes, wq_scales, hot_idx)
    n_hot = hot_idx.numel()
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    _need_cuda(y)
    _need(y, "y", torch.float32, (M, N), dense=False)
    if y.stride(1) != 1:
        raise ValueError("y must have unit column stride")
    if workspace is None:
        workspace = _scratch(hcp_workspace_bytes(M, N, n_hot), x.device, stream)
    _check(lib().fp4q_gemm_hcp(M, N, K, _ptr(x), _ptr(xq_codes), _ptr(xq_scales), _ptr(w),
                               _ptr(wq_codes), _ptr(wq_scales), _ptr(hot_idx), n_hot, _ptr(y),
                               y.stride(0), _ptr(workspace), workspace.numel(), _stream(stream)))
    return y


def gemm_dge(a_codes, a_scales, b_codes, b_scales, x, k=5.0, clamp_max=3.0, out=None,
             stream=None):
    """out[M,N] (fp32) = deq(A) deq(B)^T times the DGE derivative of x (bf16 [M,N],
    column blocks of 32), in one kernel (fp4q_gemm_dge); returns out."""
    torch = _torch()
    _need_cuda(a_codes, a_scales, b_codes, b_scales, x)
    M, N, K = a_codes.shape[0], b_codes.shape[0], a_codes.shape[1] * 2
    if b_codes.shape[1] * 2 != K:
        raise ValueError("A and B K dimensions differ")
    if tuple(x.shape) != (M, N):
        raise ValueError("x must be [M, N]")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=a_codes.device)
    _check(lib().fp4q_gemm_dge(M, N, K, _ptr(a_codes), _ptr(a_scales), _ptr(b_codes),
                               _ptr(b_scales), _ptr(x), _dt(x), k, clamp_max, _ptr(out),
                               out.stride(0), _stream(stream)))
    return out


def gemm_quant(a_codes, a_scales, b_codes, b_scales, c=None, write_c=True, out=None,
               stream=None):
    """C = deq(A) deq(B)^T in bf16 (written unless write_c is False) and C's ROW
    block-32 nearest-even quantisation, in one kernel (fp4q_gemm_quant).
    Returns (c or None, (codes, scales))."""
    torch = _torch()
    _need_cuda(a_codes, a_scales, b_codes, b_scales)
    M, N, K = a_codes.shape[0], b_codes.shape[0], a_codes.shape[1] * 2
    if b_codes.shape[1] * 2 != K:
        raise ValueError("A and B K dimensions differ")
    if write_c and c is None:
        c = torch.empty((M, N), dtype=torch.bfloat16, device=a_codes.device)
    if not write_c:
        c = None
    if out is None:
        u8 = dict(dtype=torch.uint8, device=a_codes.device)
        out = (torch.empty((M, N // 2), **u8), torch.empty((M, N // 32), **u8))
    _check(lib().fp4q_gemm_quant(M, N, K, _ptr(a_codes), _ptr(a_scales), _ptr(b_codes),
                                 _ptr(b_scales), _ptr(c), c.stride(0) if c is not None else N,
                                 _ptr(out[0]), _ptr(out[1]), _stream(stream)))
    return c, out


def channel_mask(idx, length, out=None, stream=None):
    """uint32 bit mask over `length` positions with the bits of idx set
    (fp4q_channel_mask); returns the mask tensor."""
    torch = _torch()
    _need_cuda(idx)
    if out is None:
        out = torch.empty(((length + 31) // 32,), dtype=torch.int32, device=idx.device)
    _check(lib().fp4q_channel_mask(_ptr(idx), idx.numel(), length, _ptr(out), _stream(stream)))
    return out


def quantize_masked(x, zero_mask, block=32, axis=ROW, rounding=RNE, seed=0, rng_offset=0,
                    codes=None, scales=None, stream=None):
    """fp4q_quantize of x with the zero_mask positions along the block axis
    taken as zeros (fp4q_quantize_masked); returns (codes, scales)."""
    torch = _torch()
    _need_cuda(x, zero_mask)
    R, C = x.shape
    if codes is None:
        shape_c = (R, C // 2) if axis == ROW else (C, R // 2)
        shape_s = (R, C // block) if axis == ROW else (C, R // block)
        codes = torch.empty(shape_c, dtype=torch.uint8, device=x.device)
        scales = torch.empty(shape_s, dtype=torch.uint8, device=x.device)
    _check(lib().fp4q_quantize_masked(_ptr(x), _dt(x), R, C, x.stride(0), block, axis, rounding,
                                      seed, rng_offset, _ptr(zero_mask), _ptr(codes),
                                      _ptr(scales), _stream(stream)))
    return codes, scales


def gemm_hcp_split(x, xq_codes, xq_scales, w, wq_codes, wq_scales, hot_idx, y=None,
                   workspace=None, stream=None):
    """Y[M,N] (fp32) = Xq' Wq' + X[:, hot] W[hot, :] in one kernel
    (fp4q_gemm_hcp_split; xq, wq quantised with the hot channels zeroed)."""
    torch = _torch()
    M, N, K = _hcp_operands(x, xq_codes, xq_scales, w, wq_codes, wq_scales, hot_idx)
    n_hot = hot_idx.numel()
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    _need_cuda(y)
    _need(y, "y", torch.float32, (M, N), dense=False)
    if y.stride(1) != 1:
        raise ValueError("y must have unit column stride")
    if workspace is None:
        workspace = _scratch(hcp_workspace_bytes(M, N, n_hot), x.device, stream)
    _check(lib().fp4q_gemm_hcp_split(M, N, K, _ptr(x), _ptr(xq_codes), _ptr(xq_scales), _ptr(w),
                                     _ptr(wq_codes), _ptr(wq_scales), _ptr(hot_idx), n_hot,
                                     _ptr(y), y.stride(0), _ptr(workspace), workspace.numel(),
                                     _stream(stream)))
    return y


def hot_channels_workspace_bytes(rows, cols):
    return int(lib().fp4q_hot_channels_workspace_bytes(rows, cols))


def hot_channels(x, n_hot, hot_idx=None, err=None, want_err=False, workspace=None, stream=None):
    """The n_hot channels (columns) of the bf16 x with the largest ROW block-32
    quantisation error, ascending (fp4q_hot_channels).  Returns hot_idx, or
    (hot_idx, err) when want_err (err: fp32 per-channel errors)."""
    torch = _torch()
    _need_cuda(x)
    _need(x, "x", torch.bfloat16, dense=False)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    R, C = x.shape
    if hot_idx is None:
        hot_idx = torch.empty((max(n_hot, 0),), dtype=torch.int32, device=x.device)
    _need_cuda(hot_idx)
    _need(hot_idx, "hot_idx", torch.int32)
    if err is None and want_err:
        err = torch.empty((C,), dtype=torch.float32, device=x.device)
    if err is not None:
        _need_cuda(err)
        _need(err, "err", torch.float32, (C,))
    if workspace is None:
        workspace = _scratch(hot_channels_workspace_bytes(R, C), x.device, stream)
    _check(lib().fp4q_hot_channels(_ptr(x), R, C, x.stride(0), n_hot,
                                   _ptr(hot_idx) if n_hot > 0 else None,
                                   _ptr(err) if err is not None else None, _ptr(workspace),
                                   workspace.numel(), _stream(stream)))
    return (hot_idx, err) if want_err else hot_idx


def quantize_2d(x, rounding=RNE, seed=0, rng_offset=0, out=None, stream=None, tile=32):
    """One E8M0 scale per tile x tile square of the bf16 x (fp4q_quantize_2d,
    or fp4q_quantize_2d_tile for tile 16).  Returns (row_codes, row_scales,
    col_codes, col_scales): the same codes in the ROW layout [R, C/2],
    [R, C/tile] and the COL layout [C, R/2], [C, R/tile]."""
    torch = _torch()
    _need_cuda(x)
    R, C = x.shape
    if out is None:
        dev = x.device
        out = (torch.empty((R, C // 2), dtype=torch.uint8, device=dev),
               torch.empty((R, C // tile), dtype=torch.uint8, device=dev),
               torch.empty((C, R // 2), dtype=torch.uint8, device=dev),
               torch.empty((C, R // tile), dtype=torch.uint8, device=dev))
    if tile == 32:
        _check(lib().fp4q_quantize_2d(_ptr(x), R, C, x.stride(0), rounding, seed, rng_offset,
                                      *(_ptr(t) for t in out), _stream(stream)))
    else:
        _check(lib().fp4q_quantize_2d_tile(_ptr(x), R, C, x.stride(0), tile, rounding, seed,
                                           rng_offset, *(_ptr(t) for t in out), _stream(stream)))
    return out


def quantize_rht(x, signs, axis=ROW, rounding=RNE, seed=0, rng_offset=0, codes=None, scales=None,
                 stream=None):
    """Block-32 quantisation of c * H32 * D * x along the block axis
    (fp4q_quantize_rht); signs: int32/uint32 device bit mask over that axis.
    Returns (codes, scales) in the layout of quantize(x, 32, axis)."""
    torch = _torch()
    _need_cuda(x, signs)
    R, C = x.shape
    if codes is None:
        shape_c = (R, C // 2) if axis == ROW else (C, R // 2)
        shape_s = (R, C // 32) if axis == ROW else (C, R // 32)
        codes = torch.empty(shape_c, dtype=torch.uint8, device=x.device)
        scales = torch.empty(shape_s, dtype=torch.uint8, device=x.device)
    _check(lib().fp4q_quantize_rht(_ptr(x), R, C, x.stride(0), axis, _ptr(signs), rounding, seed,
                                   rng_offset, _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


def occ_max_nnz(rows, cols, quantile=0.99):
    return int(lib().fp4q_occ_max_nnz(rows, cols, quantile))


def occ_quantize(x, quantile=0.99, rounding=RNE, seed=0, rng_offset=0, workspace=None,
                 stream=None):
    """Outlier clamping and compensation (fp4q_occ_quantize).  Returns
    (codes, scales, row_ptr, col_idx, vals, threshold): the ROW block-32
    quantisation of the clamped x, the residual in CSR (arrays sized by the
    bound fp4q_occ_max_nnz; row_ptr[-1] entries are used) and T's bf16 bits."""
    torch = _torch()
    _need_cuda(x)
    _need(x, "x", torch.bfloat16, dense=False)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    R, C = x.shape
    dev = x.device
    cap = occ_max_nnz(R, C, quantile)
    codes = torch.empty((R, C // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((R, C // 32), dtype=torch.uint8, device=dev)
    row_ptr = torch.empty((R + 1,), dtype=torch.int64, device=dev)
    col_idx = torch.empty((max(cap, 1),), dtype=torch.int32, device=dev)
    vals = torch.empty((max(cap, 1),), dtype=torch.float32, device=dev)
    thr = torch.empty((8,), dtype=torch.int16, device=dev)
    if workspace is None:
        workspace = _scratch(lib().fp4q_occ_workspace_bytes(R, C), dev, stream)
    _check(lib().fp4q_occ_quantize(_ptr(x), R, C, x.stride(0), quantile, rounding, seed,
                                   rng_offset, _ptr(codes), _ptr(scales), _ptr(row_ptr),
                                   _ptr(col_idx), _ptr(vals), cap, _ptr(thr), _ptr(workspace),
                                   workspace.numel(), _stream(stream)))
    return codes, scales, row_ptr, col_idx, vals, thr[:1]


def occ_spmm(row_ptr, col_idx, vals, w, y, stream=None):
    """y[M, N] (fp32, in place) += R W for the CSR residual R (fp4q_occ_spmm)."""
    torch = _torch()
    _need_cuda(row_ptr, col_idx, vals, w, y)
    _need(row_ptr, "row_ptr", torch.int64)
    _need(col_idx, "col_idx", torch.int32)
    _need(vals, "vals", torch.float32)
    _need(w, "w", torch.bfloat16, dense=False)
    _need(y, "y", torch.float32, dense=False)
    if w.stride(1) != 1 or y.stride(1) != 1:
        raise ValueError("w and y must have unit column stride")
    M, N = y.shape
    K = w.shape[0]
    _check(lib().fp4q_occ_spmm(M, N, K, _ptr(row_ptr), _ptr(col_idx), _ptr(vals), _ptr(w),
                               w.stride(0), _ptr(y), y.stride(0), _stream(stream)))
    return y


def _rows(t, name, dtype=None, shape=None):
    """Row stride of a 2-D device tensor with unit column stride (the stride
    of a single row, or of columns one element wide, is free)."""
    size = t.shape
    if (t.is_cuda and len(size) == 2 and t.is_contiguous() and (dtype is None or t.dtype is dtype)
            and (shape is None or size == shape)):
        return size[1]
    _need_cuda(t)
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and size != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(size)}")
    if len(size) != 2 or (t.stride(1) != 1 and size[1] != 1):
        raise ValueError(f"{name} must be 2-D with unit column stride")
    return t.stride(0) if size[0] > 1 else max(t.stride(0), size[1])


def _codes(codes, scales, name, rows=None, K=None):
    """Checks one K-major block-32 operand; returns its rows and K."""
    u8, size = _torch().uint8, codes.shape
    if len(size) == 2:
        if rows is None:
            rows = size[0]
        if K is None:
            K = 2 * size[1]
        if (codes.dtype is u8 and scales.dtype is u8 and size == (rows, K // 2)
                and scales.shape == (rows, K // 32) and codes.is_contiguous()
                and scales.is_contiguous() and codes.is_cuda and scales.is_cuda):
            return rows, K
    _need_cuda(codes, scales)  # one of these says what is wrong
    if len(size) != 2:
        raise ValueError(f"{name}_codes must be 2-D")
    _need(codes, f"{name}_codes", u8, (rows, K // 2))
    _need(scales, f"{name}_scales", u8, (rows, K // 32))
    return rows, K


def gemm_gated(x_codes, x_scales, gate_codes, gate_scales, up_codes, up_scales, act=SILU,
               save=False, h=None, gate=None, up=None, stream=None):
    """act(X Wg^T) * (X Wu^T) of quantised operands in one kernel
    (fp4q_gemm_gated): x_codes [M, K/2], the weights' codes [F, K/2] (rows of
    one packed array will do).  Returns h (bf16 [M, F]), or (h, gate, up)
    where save is set or gate and up are given; with save alone they are the
    halves of one [M, 2F] tensor."""
    bf16 = _torch().bfloat16
    M, K = _codes(x_codes, x_scales, "x")
    F, _ = _codes(gate_codes, gate_scales, "gate", K=K)
    _codes(up_codes, up_scales, "up", F, K)
    if (gate is None) != (up is None):
        raise ValueError("gate and up are given both or neither")
    ldgu, empty = 0, _allocator(x_codes, stream)
    if gate is not None:
        ldgu = _rows(gate, "gate", bf16, (M, F))
        if _rows(up, "up", bf16, (M, F)) != ldgu:
            raise ValueError("gate and up must have the same row stride")
    elif save:
        gate, up = _halves(empty, M, F, bf16)
        ldgu = 2 * F
    if h is None:
        h, ldh = empty((M, F), (F, 1), bf16), F
    else:
        ldh = _rows(h, "h", bf16, (M, F))
    status = lib().fp4q_gemm_gated(
        M, F, K, x_codes.data_ptr(), x_scales.data_ptr(), gate_codes.data_ptr(),
        gate_scales.data_ptr(), up_codes.data_ptr(), up_scales.data_ptr(), act, h.data_ptr(), ldh,
        _ptr(gate), _ptr(up), ldgu, _stream(stream))
    if status:
        _check(status)
    return h if gate is None else (h, gate, up)


def gemm_gated_grad(dy_codes, dy_scales, w_codes, w_scales, gate, up, act=SILU, d_gate=None,
                    d_up=None, stream=None):
    """Gradients of the gated block's two products behind its down projection
    (fp4q_gemm_gated_grad): dy_codes [M, K/2], w_codes [F, K/2], gate and up
    bf16 [M, F] as gemm_gated returned them.  Returns (d_gate, d_up), bf16,
    the halves of one [M, 2F] tensor unless given (not in gate's or up's
    memory)."""
    bf16 = _torch().bfloat16
    M, K = _codes(dy_codes, dy_scales, "dy")
    F, _ = _codes(w_codes, w_scales, "w", K=K)
    ldgu = _rows(gate, "gate", bf16, (M, F))
    if _rows(up, "up", bf16, (M, F)) != ldgu:
        raise ValueError("gate and up must have the same row stride")
    if (d_gate is None) != (d_up is None):
        raise ValueError("d_gate and d_up are given both or neither")
    if d_gate is None:
        d_gate, d_up = _halves(_allocator(dy_codes, stream), M, F, bf16)
        ldd = 2 * F
    else:
        ldd = _rows(d_gate, "d_gate", bf16, (M, F))
        if _rows(d_up, "d_up", bf16, (M, F)) != ldd:
            raise ValueError("d_gate and d_up must have the same row stride")
    status = lib().fp4q_gemm_gated_grad(
        M, F, K, dy_codes.data_ptr(), dy_scales.data_ptr(), w_codes.data_ptr(), w_scales.data_ptr(),
        act, gate.data_ptr(), up.data_ptr(), ldgu, d_gate.data_ptr(), d_up.data_ptr(), ldd,
        _stream(stream))
    if status:
        _check(status)
    return d_gate, d_up


def _vec(t, name, dtype, n):
    """Checks a contiguous device vector of n elements (dtype None: any)."""
    if t.shape == (n,) and t.is_cuda and t.is_contiguous() and (dtype is None or t.dtype is dtype):
        return
    _need_cuda(t)
    _need(t, name, t.dtype if dtype is None else dtype, (n,))


def _affine(weight, bias, cols):
    """Dtype code of the norm's weight and bias vectors."""
    if weight is not None:
        _vec(weight, "weight", None, cols)
    if bias is None:
        return F32 if weight is None else _dt(weight)
    _vec(bias, "bias", None, cols)
    if weight is not None and weight.dtype != bias.dtype:
        raise TypeError("weight and bias must have the same dtype")
    return _dt(bias)


def layer_norm(x, weight=None, bias=None, eps=1e-5, kind=LAYER_NORM, y=None, out_dtype=None,
               stats=True, mean=None, rstd=None, stream=None):
    """Layer norm (or RMS norm) of the rows of x (fp4q_layer_norm).  Returns
    (y, mean, rstd): y of out_dtype (x's by default), mean and rstd fp32 per
    row for layer_norm_grad (mean None for RMS_NORM, both None without
    stats)."""
    f32 = _torch().float32
    ldx = _rows(x, "x")
    R, C = x.shape
    xdt = ydt = _dt(x)
    wdt = _affine(weight, bias, C)
    empty = _allocator(x, stream)
    if y is None:
        ldy = C
        y = empty((R, C), (C, 1), x.dtype if out_dtype is None else out_dtype)
        if out_dtype is not None:
            ydt = _dt(y)
    else:
        ldy, ydt = _rows(y, "y", shape=(R, C)), _dt(y)
    if mean is not None:
        _vec(mean, "mean", f32, R)
    elif stats and kind == LAYER_NORM:
        mean = empty((R,), (1,), f32)
    if rstd is not None:
        _vec(rstd, "rstd", f32, R)
    elif stats:
        rstd = empty((R,), (1,), f32)
    status = lib().fp4q_layer_norm(kind, x.data_ptr(), xdt, R, C, ldx, _ptr(weight), _ptr(bias), wdt,
                                   eps, y.data_ptr(), ydt, ldy, _ptr(mean), _ptr(rstd),
                                   _stream(stream))
    if status:
        _check(status)
    return y, mean, rstd


def layer_norm_grad_workspace_bytes(rows, cols):
    return int(lib().fp4q_layer_norm_grad_workspace_bytes(rows, cols))


def layer_norm_grad(dy, x, weight, mean, rstd, kind=LAYER_NORM, dx=None, want_weight=True,
                    want_bias=True, dweight=None, dbias=None, workspace=None, stream=None):
    """Backward pass of layer_norm (fp4q_layer_norm_grad).  Returns (dx,
    dweight, dbias): dx of x's dtype, the others fp32 (None where not
    wanted)."""
    f32 = _torch().float32
    ldx = _rows(x, "x")
    R, C = x.shape
    lddy = _rows(dy, "dy", shape=(R, C))
    wdt = _affine(weight, None, C)
    empty = _allocator(x, stream)
    if dx is None:
        dx, lddx = empty((R, C), (C, 1), x.dtype), C
    else:
        lddx = _rows(dx, "dx", x.dtype, (R, C))
    if mean is not None:
        _vec(mean, "mean", f32, R)
    if rstd is not None:
        _vec(rstd, "rstd", f32, R)
    if dweight is not None:
        _vec(dweight, "dweight", f32, C)
    elif want_weight:
        dweight = empty((C,), (1,), f32)
    if dbias is not None:
        _vec(dbias, "dbias", f32, C)
    elif want_bias:
        dbias = empty((C,), (1,), f32)
    nbytes = 0
    if dweight is not None or dbias is not None:
        if workspace is None:
            nbytes = lib().fp4q_layer_norm_grad_workspace_bytes(R, C)
            workspace = empty((nbytes,), (1,), _torch().uint8)
        else:
            _need_cuda(workspace)
            _need(workspace, "workspace", workspace.dtype)
            nbytes = workspace.numel() * workspace.element_size()
    status = lib().fp4q_layer_norm_grad(kind, dy.data_ptr(), _dt(dy), lddy, x.data_ptr(), _dt(x), R, C,
                                        ldx, _ptr(weight), wdt, _ptr(mean), _ptr(rstd),
                                        dx.data_ptr(), lddx, _ptr(dweight), _ptr(dbias),
                                        _ptr(workspace), nbytes, _stream(stream))
    if status:
        _check(status)
    return dx, dweight, dbias


class AdamwPlan:
    """The tensors of an AdamW step, checked once (see adamw_plan).  Holds
    their memory (through tensors of its own, which a later `param.data = ...`
    leaves as they are) and, for more tensors than one launch takes as kernel
    arguments, their table in device memory."""
    ARGUMENTS = 44

    def __init__(self, array, n, bits, grad_dtype, tensors):
        self.array, self.n, self.bits, self.grad_dtype = array, n, bits, grad_dtype
        self.tensors = tensors
        self.table, self.chunks, self.streams = None, 0, set()
        if n > self.ARGUMENTS:
            torch = _torch()
            size, chunks = _ct.c_size_t(0), _ct.c_int64(0)
            fill = lib().fp4q_adamw_table
            _check(fill(array, n, bits, None, _ct.byref(size), _ct.byref(chunks)))
            host = torch.empty(size.value + 16, dtype=torch.uint8)
            host = host[-host.data_ptr() % 16:][:size.value]
            _check(fill(array, n, bits, host.data_ptr(), _ct.byref(size), _ct.byref(chunks)))
            self.table, self.chunks = host.to(tensors[0][0].device), chunks.value
            self.streams.add(_stream(None))

    def read_on(self, handle, stream):
        """The table is about to be read on a stream: its memory is not to be
        reused before that work is done, should the plan be dropped."""
        if handle not in self.streams:
            self.table.record_stream(_torch().cuda.current_stream() if stream is None else stream)
            self.streams.add(handle)


def adamw_state(param, bits=32):
    """Zero moments for one parameter: (exp_avg, exp_avg_sq, exp_avg_scales,
    exp_avg_sq_scales); the scales are None for bits=32."""
    torch = _torch()
    n = param.numel()
    if bits == 32:
        return (torch.zeros(n, dtype=torch.float32, device=param.device),
                torch.zeros(n, dtype=torch.float32, device=param.device), None, None)
    if bits != 8:
        raise ValueError("bits must be 8 or 32")
    return tuple(torch.zeros(k, dtype=torch.uint8, device=param.device)
                 for k in (n, n, (n + 31) // 32, (n + 31) // 32))


def adamw_plan(params, grads, exp_avg, exp_avg_sq, exp_avg_scales=None, exp_avg_sq_scales=None,
               copies=None, weight_decay=0.0):
    """Checks the tensors of an AdamW step and keeps their addresses for
    adamw_step.  params: contiguous fp32 tensors; grads: fp32 or bf16, one
    dtype; exp_avg, exp_avg_sq: fp32, or uint8 (E4M3 codes of m and of
    sqrt(v)) with the uint8 scales, ceil(numel/32) per tensor; copies: bf16
    tensors to receive the new params, or None; weight_decay: a number, or
    one per tensor.

    A plan is of addresses and holds the memory behind them.  It is made anew
    when a tensor gets other memory (gradients that are set to None and made
    again, param.data = ...): an old plan would step with the old gradients and
    write to the old parameters.  Gradients that are zeroed in place, or
    written over as layer_norm_grad's dweight= and gemm's c= do, keep theirs."""
    torch = _torch()
    n = len(params)
    bits = 8 if exp_avg_scales is not None else 32
    if (exp_avg_scales is None) != (exp_avg_sq_scales is None):
        raise ValueError("exp_avg_scales and exp_avg_sq_scales are given both or neither")
    state = torch.uint8 if bits == 8 else torch.float32
    none = [None] * n
    if not isinstance(weight_decay, (list, tuple)):
        weight_decay = [weight_decay] * n
    cols = dict(params=params, grads=grads, exp_avg=exp_avg, exp_avg_sq=exp_avg_sq,
                exp_avg_scales=exp_avg_scales or none, exp_avg_sq_scales=exp_avg_sq_scales or none,
                copies=copies or none, weight_decay=weight_decay)
    for name, c in cols.items():
        if len(c) != n:
            raise ValueError(f"{name} must have one entry per tensor ({n}), got {len(c)}")
    gdtype = grads[0].dtype if n else torch.float32
    if gdtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"grads must be bf16 or fp32, got {gdtype}")
    array = (AdamwTensor * max(n, 1))()
    for i, (p, g, m, v, ms, vs, c, wd) in enumerate(zip(*cols.values())):
        k = p.numel()
        nb = (k + 31) // 32
        for t, name, dtype, size in ((p, "param", torch.float32, k), (g, "grad", gdtype, k),
                                     (m, "exp_avg", state, k), (v, "exp_avg_sq", state, k),
                                     (ms, "exp_avg_scales", torch.uint8, nb),
                                     (vs, "exp_avg_sq_scales", torch.uint8, nb),
                                     (c, "copy", torch.bfloat16, k)):
            if t is None:
                continue
            _need_cuda(t)
            if t.dtype != dtype or t.numel() != size or not t.is_contiguous():
                _need(t, f"{name} {i}", dtype)
                raise ValueError(f"{name} {i} must have {size} elements, got {t.numel()}")
        array[i] = AdamwTensor(*(0 if t is None else t.data_ptr() for t in (p, g, m, v, ms, vs, c)),
                               k, wd)
    return AdamwPlan(array, n, bits, BF16 if gdtype == torch.bfloat16 else F32,
                     [tuple(t if t is None else t.detach() for t in row)
                      for row in zip(*list(cols.values())[:-1])])


def adamw_step(plan, lr, step, beta1=0.9, beta2=0.999, eps=1e-8, seed=0, grad_scale=None,
               stream=None):
    """One AdamW step over the plan's tensors, in place (fp4q_adamw_step).
    step counts from 1; seed: the stochastic rounding of 8-bit moments;
    grad_scale: a device fp32 scalar that multiplies the gradients.  A graph
    that captured the step reads the plan's memory at every replay: the plan is
    kept as long as the graph."""
    if grad_scale is not None:
        _need_cuda(grad_scale)
        _need(grad_scale, "grad_scale", _torch().float32)
        if grad_scale.numel() != 1:
            raise ValueError(f"grad_scale must have one element, got {grad_scale.numel()}")
    handle = _stream(stream)
    if plan.table is None:
        _check(lib().fp4q_adamw_step(plan.array, plan.n, plan.bits, plan.grad_dtype, lr, beta1, beta2,
                                     eps, step, seed, _ptr(grad_scale), handle))
    else:
        plan.read_on(handle, stream)
        _check(lib().fp4q_adamw_step_table(plan.table.data_ptr(), plan.n, plan.chunks, plan.bits,
                                           plan.grad_dtype, lr, beta1, beta2, eps, step, seed,
                                           _ptr(grad_scale), handle))
