"""GB300 (sm_103a) block-scaled quantization: bf16 -> MXFP8 / NVFP4.

Thin Python binding over libmxq.so, whose C ABI is declared in
``include/mxq.h``.  The functions here carry the same names as the C entry
points and only marshal arguments: they allocate outputs with torch when the
caller does not pass them, pass raw device pointers and the current CUDA
stream, and raise ``MxqError`` on a non-zero status.  Every step of the
quantization runs in the library's kernels; there is no fallback path, and
importing this package fails if libmxq.so cannot be loaded.

No call synchronises, so that what goes wrong on the GPU (a wait that ran out,
group offsets that are out of order) is only seen in ``dev_err``, a zeroed
[1] int32 CUDA tensor that the caller passes and reads.  With ``stream``, an
output that is not passed in is still allocated on the current stream: order
the one after the other.
"""
import ctypes

import torch

from . import _lib

ROWWISE = 1
COLWISE = 2
DBIAS = 4
ACT_GELU_TANH = 8
NVFP4_2D = 16
ACT_SILU = 32
SCALE_RCEIL = 64
SCALE_SWIZZLED = 128
OUT_F32 = 256


def scale_shape(R, C, flags):
    """Shape of an [R][C] scale matrix as written under `flags`: padded to
    128 x 4 tiles with SCALE_SWIZZLED, else [R, C]."""
    if flags & SCALE_SWIZZLED:
        return (-(-R // 128) * 128, -(-C // 4) * 4)
    return (R, C)
OP_ROWCOL = 0
OP_NVFP4 = 1
OP_DACT = 2
OP_ROWCOL_HOST = 3
OP_GROUPED_GEMM = 4
OP_GROUPED_WGRAD = 5
OP_NVFP4_GEMV = 6
DEVERR_TIMEOUT = 1
DEVERR_OFFSETS = 2

STATUS_NAMES = {0: "MXQ_OK", 1: "MXQ_EINVAL", 2: "MXQ_ESHAPE", 3: "MXQ_EALIGN",
                4: "MXQ_EARCH", 5: "MXQ_EWORKSPACE", 6: "MXQ_ECUDA"}


class MxqError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = _lib.lib().mxq_status_string(status).decode()
        super().__init__(f"{where}: {msg} (status {status})")


def library_path():
    return _lib.LIB_PATH


def _check(status, where):
    if status != 0:
        raise MxqError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _input(x, name="x"):
    if not isinstance(x, torch.Tensor) or x.dtype != torch.bfloat16 or x.dim() != 2:
        raise TypeError(f"{name} must be a 2-D torch.bfloat16 tensor")
    if not x.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if x.size(1) > 1 and x.stride(1) != 1:
        raise ValueError(f"{name} needs a unit column stride")
    return x.stride(0) if x.size(0) > 1 else x.size(1)


def _empty(shape, dtype, device):
    return torch.empty(shape, dtype=dtype, device=device)


def mxq_workspace_bytes(op, M, K, flags):
    return int(_lib.lib().mxq_workspace_bytes(op, M, K, flags))


def mx_quantize_rowcol(x, flags=ROWWISE | COLWISE, *, q_row=None, s_row=None, q_col=None,
                       s_col=None, dbias=None, workspace=None, dev_err=None, stream=None):
    """bf16 x[M, K] -> MXFP8.  Returns a dict with q_row [M,K] / s_row
    [M,K/32] (ROWWISE), q_col [K,M] / s_col [K,M/32] (COLWISE), dbias [K]
    fp32 (DBIAS); codes and scales are torch.uint8."""
    ldx = _input(x)
    M, K = x.shape
    dev = x.device
    out = {}
    if flags & ROWWISE:
        out["q_row"] = q_row if q_row is not None else _empty((M, K), torch.uint8, dev)
        out["s_row"] = s_row if s_row is not None else _empty(scale_shape(M, K // 32, flags),
                                                              torch.uint8, dev)
    if flags & COLWISE:
        out["q_col"] = q_col if q_col is not None else _empty((K, M), torch.uint8, dev)
        out["s_col"] = s_col if s_col is not None else _empty(scale_shape(K, M // 32, flags),
                                                              torch.uint8, dev)
    ws_bytes = 0
    if flags & DBIAS:
        out["dbias"] = dbias if dbias is not None else _empty((K,), torch.float32, dev)
        if workspace is None:
            need = mxq_workspace_bytes(OP_ROWCOL, M, K, flags)
            workspace = _empty((max(need, 16),), torch.uint8, dev)
        ws_bytes = workspace.numel() * workspace.element_size()
    st = _lib.lib().mx_quantize_rowcol(
        _ptr(x), M, K, ldx, flags, _ptr(out.get("q_row")), _ptr(out.get("s_row")),
        _ptr(out.get("q_col")), _ptr(out.get("s_col")), _ptr(out.get("dbias")),
        _ptr(workspace), ws_bytes, _ptr(dev_err), _stream(stream))
    _check(st, "mx_quantize_rowcol")
    return out


def mx_quantize_rowcol_dbias_noalloc(x, flags=ROWWISE | COLWISE, *, q_row=None, s_row=None,
                                     q_col=None, s_col=None, dbias=None, dev_err=None,
                                     stream=None):
    """mx_quantize_rowcol with dbias, for callers that cannot allocate a
    workspace: the library keeps the band sums in its own fixed 8 MiB
    device array (see include/mxq.h for the limit, and for ordering calls
    that share it).  Outputs not passed in are allocated here with torch,
    as in the other bindings; pass them all to allocate nothing."""
    ldx = _input(x)
    M, K = x.shape
    dev = x.device
    out = {}
    if flags & ROWWISE:
        out["q_row"] = q_row if q_row is not None else _empty((M, K), torch.uint8, dev)
        out["s_row"] = s_row if s_row is not None else _empty(scale_shape(M, K // 32, flags),
                                                              torch.uint8, dev)
    if flags & COLWISE:
        out["q_col"] = q_col if q_col is not None else _empty((K, M), torch.uint8, dev)
        out["s_col"] = s_col if s_col is not None else _empty(scale_shape(K, M // 32, flags),
                                                              torch.uint8, dev)
    out["dbias"] = dbias if dbias is not None else _empty((K,), torch.float32, dev)
    st = _lib.lib().mx_quantize_rowcol_dbias_noalloc(
        _ptr(x), M, K, ldx, flags, _ptr(out.get("q_row")), _ptr(out.get("s_row")),
        _ptr(out.get("q_col")), _ptr(out.get("s_col")), _ptr(out["dbias"]), _ptr(dev_err),
        _stream(stream))
    _check(st, "mx_quantize_rowcol_dbias_noalloc")
    return out


def mx_quantize_rowcol_host(x, flags=ROWWISE | COLWISE, *, q_row=None, s_row=None, q_col=None,
                            s_col=None, workspace=None, stream=None):
    """mx_quantize_rowcol of a bf16 matrix in host memory: outputs in host
    memory (page-locked when allocated here), computed by panels pipelined
    through the device.  Returns once the work is enqueued; synchronise the
    stream before reading the outputs."""
    if not isinstance(x, torch.Tensor) or x.dtype != torch.bfloat16 or x.dim() != 2:
        raise TypeError("x must be a 2-D torch.bfloat16 tensor")
    if x.is_cuda:
        raise TypeError("x must be in host memory (use mx_quantize_rowcol for device tensors)")
    if x.size(1) > 1 and x.stride(1) != 1:
        raise ValueError("x needs a unit column stride")
    M, K = x.shape
    ldx = x.stride(0) if M > 1 else K

    def host(shape, given):
        return given if given is not None else torch.empty(shape, dtype=torch.uint8).pin_memory()

    out = {}
    if flags & ROWWISE:
        out["q_row"] = host((M, K), q_row)
        out["s_row"] = host(scale_shape(M, K // 32, flags), s_row)
    if flags & COLWISE:
        out["q_col"] = host((K, M), q_col)
        out["s_col"] = host(scale_shape(K, M // 32, flags), s_col)
    if workspace is None:
        need = mxq_workspace_bytes(OP_ROWCOL_HOST, M, K, flags)
        workspace = _empty((max(need, 256),), torch.uint8, torch.device("cuda"))
    st = _lib.lib().mx_quantize_rowcol_host(
        _ptr(x), M, K, ldx, flags, _ptr(out.get("q_row")), _ptr(out.get("s_row")),
        _ptr(out.get("q_col")), _ptr(out.get("s_col")), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "mx_quantize_rowcol_host")
    return out


def mx_quantize_gated(x, flags=ROWWISE | COLWISE, *, q_row=None, s_row=None, q_col=None,
                      s_col=None, dev_err=None, stream=None):
    """Gated MXFP8 of x[M, 2N] = [gate | up]; y = silu(gate) * up (SwiGLU,
    the default) or gelu_tanh(gate) * up (flags | ACT_GELU_TANH: GeGLU) in
    fp32, quantized like mx_quantize_rowcol (outputs sized by N)."""
    ldx = _input(x)
    M, W = x.shape
    if W % 2:
        raise ValueError("x must hold [gate | up] halves of equal width")
    N = W // 2
    dev = x.device
    out = {}
    if flags & ROWWISE:
        out["q_row"] = q_row if q_row is not None else _empty((M, N), torch.uint8, dev)
        out["s_row"] = s_row if s_row is not None else _empty(scale_shape(M, N // 32, flags),
                                                              torch.uint8, dev)
    if flags & COLWISE:
        out["q_col"] = q_col if q_col is not None else _empty((N, M), torch.uint8, dev)
        out["s_col"] = s_col if s_col is not None else _empty(scale_shape(N, M // 32, flags),
                                                              torch.uint8, dev)
    st = _lib.lib().mx_quantize_gated(
        _ptr(x), M, N, ldx, flags, _ptr(out.get("q_row")), _ptr(out.get("s_row")),
        _ptr(out.get("q_col")), _ptr(out.get("s_col")), _ptr(dev_err), _stream(stream))
    _check(st, "mx_quantize_gated")
    return out


def _mx_outputs(M, K, flags, dev, q_row, s_row, q_col, s_col):
    out = {}
    if flags & ROWWISE:
        out["q_row"] = q_row if q_row is not None else _empty((M, K), torch.uint8, dev)
        out["s_row"] = s_row if s_row is not None else _empty(scale_shape(M, K // 32, flags),
                                                              torch.uint8, dev)
    if flags & COLWISE:
        out["q_col"] = q_col if q_col is not None else _empty((K, M), torch.uint8, dev)
        out["s_col"] = s_col if s_col is not None else _empty(scale_shape(K, M // 32, flags),
                                                              torch.uint8, dev)
    return out


def mx_quantize_dact(grad, x, flags, *, q_row=None, s_row=None, q_col=None, s_col=None,
                     dbias=None, workspace=None, dev_err=None, stream=None):
    """Backward MXFP8: y = grad * act'(x) for grad, x [M, K] bf16, with act
    gelu_tanh (flags | ACT_GELU_TANH) or silu (flags | ACT_SILU); outputs as
    mx_quantize_rowcol, dbias = column sums of y with DBIAS."""
    ldg = _input(grad, "grad")
    ldx = _input(x)
    M, K = x.shape
    if tuple(grad.shape) != (M, K):
        raise ValueError("grad and x shapes differ")
    dev = x.device
    out = _mx_outputs(M, K, flags, dev, q_row, s_row, q_col, s_col)
    ws_bytes = 0
    if flags & DBIAS:
        out["dbias"] = dbias if dbias is not None else _empty((K,), torch.float32, dev)
        if workspace is None:
            need = mxq_workspace_bytes(OP_DACT, M, K, flags)
            workspace = _empty((max(need, 16),), torch.uint8, dev)
        ws_bytes = workspace.numel() * workspace.element_size()
    st = _lib.lib().mx_quantize_dact(
        _ptr(grad), _ptr(x), M, K, ldg, ldx, flags, _ptr(out.get("q_row")),
        _ptr(out.get("s_row")), _ptr(out.get("q_col")), _ptr(out.get("s_col")),
        _ptr(out.get("dbias")), _ptr(workspace), ws_bytes, _ptr(dev_err), _stream(stream))
    _check(st, "mx_quantize_dact")
    return out


def mx_quantize_dgated(grad, x, flags=ROWWISE | COLWISE, *, q_row=None, s_row=None, q_col=None,
                       s_col=None, dev_err=None, stream=None):
    """Backward of the gated activation: grad [M, N], x [M, 2N] = [gate |
    up]; y [M, 2N] = [grad * up * act'(gate) | grad * act(gate)] with act
    silu (default) or gelu_tanh (flags | ACT_GELU_TANH), quantized like
    mx_quantize_rowcol (outputs sized by 2N)."""
    ldg = _input(grad, "grad")
    ldx = _input(x)
    M, W = x.shape
    if W % 2 or tuple(grad.shape) != (M, W // 2):
        raise ValueError("x must be [M, 2N] = [gate | up] and grad [M, N]")
    N = W // 2
    out = _mx_outputs(M, W, flags, x.device, q_row, s_row, q_col, s_col)
    st = _lib.lib().mx_quantize_dgated(
        _ptr(grad), _ptr(x), M, N, ldg, ldx, flags, _ptr(out.get("q_row")),
        _ptr(out.get("s_row")), _ptr(out.get("q_col")), _ptr(out.get("s_col")), _ptr(dev_err),
        _stream(stream))
    _check(st, "mx_quantize_dgated")
    return out


def bf16_amax(x, *, out=None, stream=None):
    """Largest |x| as a 1-element fp32 device tensor."""
    ldx = _input(x)
    M, K = x.shape
    if out is None:
        out = _empty((1,), torch.float32, x.device)
    st = _lib.lib().bf16_amax(_ptr(x), M, K, ldx, _ptr(out), _stream(stream))
    _check(st, "bf16_amax")
    return out


def nvfp4_quantize_transpose(x, flags=ROWWISE | COLWISE, *, amax=None, global_scale=None,
                             q_row=None, s_row=None, q_t=None, s_t=None, workspace=None,
                             dev_err=None, stream=None):
    """bf16 x[M, K] -> NVFP4: q_row [M,K/2] / s_row [M,K/16] (ROWWISE),
    q_t [K,M/2] / s_t [K,M/16] (COLWISE), global_scale [1] fp32.  `amax`
    (1-element fp32 device tensor) skips the internal amax pass; flags | NVFP4_2D
    takes one scale per 16x16 block."""
    ldx = _input(x)
    M, K = x.shape
    dev = x.device
    out = {"global_scale": global_scale if global_scale is not None
           else _empty((1,), torch.float32, dev)}
    if flags & ROWWISE:
        out["q_row"] = q_row if q_row is not None else _empty((M, K // 2), torch.uint8, dev)
        out["s_row"] = s_row if s_row is not None else _empty((M, K // 16), torch.uint8, dev)
    if flags & COLWISE:
        out["q_t"] = q_t if q_t is not None else _empty((K, M // 2), torch.uint8, dev)
        out["s_t"] = s_t if s_t is not None else _empty((K, M // 16), torch.uint8, dev)
    ws_bytes = 0
    if amax is None:
        if workspace is None:
            workspace = _empty((16,), torch.uint8, dev)
        ws_bytes = workspace.numel() * workspace.element_size()
    st = _lib.lib().nvfp4_quantize_transpose(
        _ptr(x), M, K, ldx, flags, _ptr(amax), _ptr(out["global_scale"]),
        _ptr(out.get("q_row")), _ptr(out.get("s_row")), _ptr(out.get("q_t")),
        _ptr(out.get("s_t")), _ptr(workspace), ws_bytes, _ptr(dev_err), _stream(stream))
    _check(st, "nvfp4_quantize_transpose")
    return out


_OUT_FLAGS = {torch.bfloat16: 0, torch.float32: OUT_F32}
_U8, _I32, _F32 = torch.uint8, torch.int32, torch.float32


# The products' calls take microseconds on the GPU, so their bindings look at
# each tensor once and cheaply, and say what is wrong only once something is.
def _operand(t, name, dim, dtype=_U8):
    """Shape of a contiguous CUDA tensor of this type and rank."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.is_contiguous():
        shape = t.shape
        if len(shape) == dim:
            return shape
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.dim() != dim:
        raise TypeError(f"{name} must be a {dim}-D {dtype} tensor")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    raise ValueError(f"{name} must be contiguous")


_several = None        # whether there is more than one CUDA device, once it is known


def _one_device(*tensors):
    """Every tensor lies on the current device, to which the launch goes.  With one
    device there is no other, and the calls do not come here (it is 1 us a call)."""
    global _several
    if _several is None:
        _several = torch.cuda.device_count() > 1
    if _several:
        found = {t.get_device() for t in tensors if isinstance(t, torch.Tensor)}
        found.add(torch.cuda.current_device())
        if len(found) > 1:
            raise ValueError(f"operands, output and current device differ: devices {sorted(found)}")


def _product_out(out, shape, out_dtype, like):
    """The output tensor (allocated when not given), its row stride and the
    flags of its type."""
    if out is None:
        flags = _OUT_FLAGS.get(out_dtype)
        if flags is None:
            raise TypeError("the output type is torch.bfloat16 or torch.float32")
        return torch.empty(shape, dtype=out_dtype, device=like.device), max(shape[-1], 1), flags
    if not isinstance(out, torch.Tensor):
        raise TypeError("out must be a tensor")
    if tuple(out.shape) != shape or not out.is_cuda:
        raise ValueError(f"out must be a CUDA tensor of shape {shape}")
    if out.dtype not in _OUT_FLAGS:
        raise TypeError("the output type is torch.bfloat16 or torch.float32")
    if shape[-1] > 1 and out.stride(-1) != 1:
        raise ValueError("out needs a unit column stride")
    return out, out.stride(-2) if shape[-2] > 1 else max(shape[-1], 1), _OUT_FLAGS[out.dtype]


def _err_ptr(dev_err):
    if dev_err is None:
        return None
    if not isinstance(dev_err, torch.Tensor) or not dev_err.is_cuda \
            or dev_err.element_size() != 4 or dev_err.numel() < 1:
        raise TypeError("dev_err must be a [1] int32 CUDA tensor")
    return dev_err.data_ptr()


def _raw_stream(stream, like):
    """The cudaStream_t of `stream`, or of the current stream of the tensor's
    device (as a number; torch.cuda.current_stream() builds an object first,
    3 us)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(like.get_device())


def mx_grouped_gemm(x_q, x_s, w_q, w_s, offsets, *, out=None, out_dtype=torch.bfloat16,
                    dev_err=None, stream=None):
    """Rows sorted by expert times their experts' weights: x_q [M,K] / x_s
    [M,K/32] and w_q [E,N,K] / w_s [E,N,K/32] as mx_quantize_rowcol writes
    them (ROWWISE, row-major scales), offsets [E+1] int32; returns [M,N]
    bf16 or fp32.  Rows in no group are not written.  For the input gradient
    pass the gradient's rows and the weights' COLWISE codes [E,K,N].  fp32
    outputs are exact to 2^-20 of their norm: the tensor cores cut sums off
    (include/mxq.h).  Offsets that decrease or leave [0, M] set DEVERR_OFFSETS
    in dev_err and nothing is written: an output allocated here then holds
    whatever its memory held."""
    M, K = _operand(x_q, "x_q", 2)
    E, N, Kw = _operand(w_q, "w_q", 3)
    if Kw != K or _operand(x_s, "x_s", 2) != (M, K // 32) \
            or _operand(w_s, "w_s", 3) != (E, N, K // 32):
        raise ValueError("x_q [M,K], x_s [M,K/32], w_q [E,N,K] and w_s [E,N,K/32] do not agree")
    if _operand(offsets, "offsets", 1, _I32) != (E + 1,):
        raise ValueError("offsets must have one entry more than there are experts")
    out, ldo, flags = _product_out(out, (M, N), out_dtype, x_q)
    if _several is not False:
        _one_device(x_q, x_s, w_q, w_s, offsets, out, dev_err)
    st = _lib.lib().mx_grouped_gemm(
        x_q.data_ptr(), x_s.data_ptr(), w_q.data_ptr(), w_s.data_ptr(), offsets.data_ptr(), M, N,
        K, E, flags, out.data_ptr(), ldo, _err_ptr(dev_err), _raw_stream(stream, x_q))
    _check(st, "mx_grouped_gemm")
    return out


def mx_grouped_wgrad(g_q, g_s, x_q, x_s, offsets, *, out=None, out_dtype=torch.float32,
                     dev_err=None, stream=None):
    """The weights' gradients of mx_grouped_gemm: g_q [N,M] / g_s [N,M/32]
    and x_q [K,M] / x_s [K,M/32] as mx_quantize_rowcol writes them
    (COLWISE), offsets [E+1] int32, multiples of 32; returns [E,N,K] fp32 or
    bf16, exact as mx_grouped_gemm's.  Offsets that break this set
    DEVERR_OFFSETS in dev_err and nothing is written, as there."""
    N, M = _operand(g_q, "g_q", 2)
    K, Mx = _operand(x_q, "x_q", 2)
    if Mx != M or _operand(g_s, "g_s", 2) != (N, M // 32) \
            or _operand(x_s, "x_s", 2) != (K, M // 32):
        raise ValueError("g_q [N,M], g_s [N,M/32], x_q [K,M] and x_s [K,M/32] do not agree")
    E = _operand(offsets, "offsets", 1, _I32)[0] - 1
    if E < 0:
        raise ValueError("offsets must have one entry more than there are experts")
    out, _, flags = _product_out(out, (E, N, K), out_dtype, g_q)
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    if _several is not False:
        _one_device(g_q, g_s, x_q, x_s, offsets, out, dev_err)
    st = _lib.lib().mx_grouped_wgrad(
        g_q.data_ptr(), g_s.data_ptr(), x_q.data_ptr(), x_s.data_ptr(), offsets.data_ptr(), M, N,
        K, E, flags, out.data_ptr(), _err_ptr(dev_err), _raw_stream(stream, g_q))
    _check(st, "mx_grouped_wgrad")
    return out


def nvfp4_gemv(x, w_q, w_s, global_scale, *, experts=None, share=1, out=None,
               out_dtype=torch.bfloat16, dev_err=None, stream=None):
    """Few rows times NVFP4 weights as nvfp4_quantize_transpose writes them
    (ROWWISE): x [T,K] bf16 with w_q [N,K/2] / w_s [N,K/16] / global_scale
    [1], or with experts [T*share] int32 and w_q [E,N,K/2] / w_s [E,N,K/16] /
    global_scale [E], where `share` output rows in turn read one row of x
    and a row whose expert is not in [0, E) is zero.  Returns [T*share,N]
    bf16 or fp32."""
    ldx = _input(x)
    T, K = x.shape
    if experts is None:
        E, lead, ids = 1, (), None
        N = _operand(w_q, "w_q", 2)[0]
    else:
        E, N, _ = _operand(w_q, "w_q", 3)
        if _operand(experts, "experts", 1, _I32) != (T * share,):
            raise ValueError("experts must have T * share entries")
        lead, ids = (E,), experts.data_ptr()
    if K % 2 or w_q.shape != lead + (N, K // 2) \
            or _operand(w_s, "w_s", len(lead) + 2) != lead + (N, K // 16):
        raise ValueError("x [T,K], w_q [(E,) N,K/2] and w_s [(E,) N,K/16] do not agree")
    if _operand(global_scale, "global_scale", 1, _F32) != (E,):
        raise ValueError("global_scale must have one entry for each expert")
    out, ldo, flags = _product_out(out, (T * share, N), out_dtype, x)
    if _several is not False:
        _one_device(x, w_q, w_s, global_scale, experts, out, dev_err)
    st = _lib.lib().nvfp4_gemv(
        x.data_ptr(), ldx, w_q.data_ptr(), w_s.data_ptr(), global_scale.data_ptr(), ids, T, share,
        N, K, E, flags, out.data_ptr(), ldo, _err_ptr(dev_err), _raw_stream(stream, x))
    _check(st, "nvfp4_gemv")
    return out


_PLAN_FIELDS = {OP_GROUPED_GEMM: ("ctas", "cols", "few", "split", "tiles", "grid"),
                OP_GROUPED_WGRAD: ("ctas", "cols", "few", "split", "tiles", "grid"),
                OP_NVFP4_GEMV: ("toks", "tiles", "cluster", "cap", "items", "grid", "uneven")}


def mxq_product_plan(op, M, N, K, E, flags=0, *, num_sms=None):
    """How a product's call is cut on a GPU of num_sms SMs (the current device's
    by default; with num_sms no device is needed), as a dict; see include/mxq.h.
    OP_NVFP4_GEMV takes M = T * share, and E = 0 for a call without experts."""
    if num_sms is None:
        num_sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    plan = (ctypes.c_int32 * 7)()
    _check(_lib.lib().mxq_product_plan(op, M, N, K, E, flags, num_sms, plan), "mxq_product_plan")
    return dict(zip(_PLAN_FIELDS[op], plan))


def mxq_selftest_bounded_wait(timeout_ns, dev_err, *, stream=None):
    """Run the bounded-wait self test (see include/mxq.h); the kernel sets
    DEVERR_TIMEOUT in dev_err (a 1-element int32 device tensor)."""
    st = _lib.lib().mxq_selftest_bounded_wait(int(timeout_ns), _ptr(dev_err), _stream(stream))
    _check(st, "mxq_selftest_bounded_wait")
