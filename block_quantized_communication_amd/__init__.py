"""Python binding of libzpq, the ZeRO++ block-quantized communication kernels
for MI355X (gfx950).

Argument marshalling only: every step runs in the HIP kernels of libzpq.so,
called through its C ABI (include/zpq.h).  PyTorch supplies device memory and
the current stream.  There is no fallback: if libzpq.so is missing or a call
fails, an exception is raised.

Functions (names follow the C ABI):
  quant_i8(x, block)                         -> (codes int8 [n], scales f32 [n/block])
  dequant_i8(codes, scales, block, dtype)    -> y [n]
  qgz_reorder_quant_i4(grad, L, N, block)    -> (codes uint8 [n/2], scales f32 [n/block])
  qgz_dequant_reduce_requant_i4(codes, scales, n_src, chunk, block,
                                out_dtype=None, divisor=1.0)
      out_dtype None: hop-1 mode, -> (codes uint8 [chunk/2], scales f32 [chunk/block])
      out_dtype set : hop-2 mode, -> averaged values [chunk] of that dtype
Each also accepts preallocated outputs (out=...) so that timed loops allocate
nothing.

Around the communication path (tensors need their element's alignment only):
  TensorList(tensors)                        a list laid out once for grad_sumsq
  grad_sumsq(tensors)                        -> sum of squares, f64 [1]
  AdamW(params, grads, ...)                  the optimizer step over many tensors, states in 32 or 8 bits
  state8_unpack / state8_pack                8-bit states to and from floats
  embedding(ids, table, scale)               -> scaled rows; embedding_i8: from qwZ codes and scales
  embedding_grad(ids, dy, rows, scale)       -> dense gradient of the table
  quant_f8(x, tile, along)                   8-bit floats in blocks of 128 along rows, columns or both, or in tiles
  dequant_f8, transpose_f8                   their values; the transposed matrix of tiles
  matmul_f8(a, b)                            a @ b.T of two such matrices
  orthogonalize(x)                           nearest orthogonal matrices, by Newton-Schulz products
  Muon(params, grads, ...)                   the optimizer step with orthogonalised updates, for matrices
"""
import bisect
import contextlib
import ctypes
import functools
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libzpq.so")

ZPQ_F32, ZPQ_F16, ZPQ_BF16 = 0, 1, 2
STATUS = {0: "ok", 1: "null pointer", 2: "bad size", 3: "bad block", 4: "misaligned pointer",
          5: "bad dtype", 6: "bad output mode", 7: "launch failed", 8: "bad argument",
          9: "output overlaps input"}

EXPORTS = ("zpq_quant_i8", "zpq_dequant_i8", "zpq_quant_i8_tensor", "zpq_qgz_reorder_quant_i4",
           "zpq_qgz_dequant_reduce_requant_i4", "zpq_status_str", "zpq_abi_version",
           "zpq_list_make", "zpq_grad_sumsq", "zpq_adamw_plan_make", "zpq_adamw_step",
           "zpq_adamw_step_at",
           "zpq_state8_unpack", "zpq_state8_pack", "zpq_embedding", "zpq_embedding_i8",
           "zpq_embedding_grad_bytes", "zpq_embedding_grad", "zpq_quant_f8", "zpq_dequant_f8",
           "zpq_transpose_f8", "zpq_matmul_f8_bytes", "zpq_matmul_f8",
           "zpq_orthogonalize_bytes", "zpq_orthogonalize", "zpq_muon_plan_bytes", "zpq_muon_plan_make",
           "zpq_muon_step")

STATE_BLOCK = 256          # elements that share an exponent byte in 8-bit optimizer states
LIST_FIXED_BYTES = 20736   # ZPQ_LIST_BYTES(0)


class _List(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("elems", ctypes.c_int64), ("chunks", ctypes.c_int64),
                ("count", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class _AdamwTensor(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("g", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("m_exp", ctypes.c_void_p), ("v_exp", ctypes.c_void_p),
                ("copy", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("weight_decay", ctypes.c_double)]


class _AdamwPlan(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("elems", ctypes.c_int64), ("chunks", ctypes.c_int64),
                ("count", ctypes.c_int32), ("p_dtype", ctypes.c_int32),
                ("g_dtype", ctypes.c_int32), ("copy_dtype", ctypes.c_int32),
                ("state_bits", ctypes.c_int32)]


class _AdamwHyper(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("grad_scale", ctypes.c_double),
                ("max_norm", ctypes.c_double), ("step", ctypes.c_int64),
                ("seed", ctypes.c_uint64)]


class _F8(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("kind", ctypes.c_int32),
                ("tile", ctypes.c_int32)]


class _MuonMatrix(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("g", ctypes.c_void_p), ("m", ctypes.c_void_p), ("copy", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("weight_decay", ctypes.c_double),
                ("scale", ctypes.c_double)]


class _MuonPlan(ctypes.Structure):
    _fields_ = [("memory", ctypes.c_void_p), ("matrices", ctypes.POINTER(_MuonMatrix)), ("count", ctypes.c_int32),
                ("p_dtype", ctypes.c_int32), ("g_dtype", ctypes.c_int32), ("copy_dtype", ctypes.c_int32)]


class _MuonHyper(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("momentum", ctypes.c_double), ("grad_scale", ctypes.c_double),
                ("max_norm", ctypes.c_double), ("coeffs", ctypes.POINTER(ctypes.c_double)), ("steps", ctypes.c_int32),
                ("nesterov", ctypes.c_int32)]


class ZpqError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: libzpq status {status} ({_status_str(status)})")


_lib = None


def lib():
    """The loaded libzpq (ctypes.CDLL) with argument types set."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run "
                              "`python -m block_quantized_communication_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        L.zpq_quant_i8.argtypes = [vp, i32, i64, i32, vp, vp, vp]
        L.zpq_dequant_i8.argtypes = [vp, vp, i64, i32, vp, i32, vp]
        L.zpq_quant_i8_tensor.argtypes = [vp, i32, i64, vp, vp, vp]
        L.zpq_qgz_reorder_quant_i4.argtypes = [vp, i32, i64, i32, i32, i32, vp, vp, vp]
        L.zpq_qgz_dequant_reduce_requant_i4.argtypes = [vp, vp, i32, i64, i32, vp, vp, vp, i32,
                                                        f32, vp]
        L.zpq_list_make.argtypes = [vp, vp, i32, i32, vp, i64, ctypes.POINTER(_List), vp]
        L.zpq_grad_sumsq.argtypes = [ctypes.POINTER(_List), vp, i32, vp]
        L.zpq_adamw_plan_make.argtypes = [ctypes.POINTER(_AdamwTensor), i32, i32, i32, i32, i32, vp,
                                          i64, ctypes.POINTER(_AdamwPlan), vp]
        L.zpq_adamw_step.argtypes = [ctypes.POINTER(_AdamwPlan), ctypes.POINTER(_AdamwHyper), vp, vp]
        L.zpq_adamw_step_at.argtypes = [ctypes.POINTER(_AdamwPlan), vp, vp, vp]
        L.zpq_state8_unpack.argtypes = [vp, vp, i64, i32, vp, i32, vp]
        L.zpq_state8_pack.argtypes = [vp, i32, i64, i32, vp, vp, vp]
        L.zpq_embedding.argtypes = [vp, i32, i64, i64, i64, vp, i32, i64, i64, f32, vp, i32, i64, vp]
        L.zpq_embedding_i8.argtypes = [vp, vp, i64, i64, i32, vp, i32, i64, i64, f32, vp, i32, i64,
                                       vp]
        L.zpq_embedding_grad_bytes.argtypes = [i64, i64, i64, ctypes.POINTER(i64)]
        L.zpq_embedding_grad.argtypes = [vp, i32, i64, vp, i32, i64, i64, i64, i64, i64, f32, vp,
                                         i32, i64, i32, vp, i64, vp]
        L.zpq_quant_f8.argtypes = [vp, i32, i64, i64, i64, i32, i32, vp, vp, vp, vp, vp]
        L.zpq_dequant_f8.argtypes = [vp, i32, vp, i64, i64, i32, vp, i32, i64, vp]
        L.zpq_transpose_f8.argtypes = [vp, vp, i64, i64, vp, vp, vp]
        L.zpq_matmul_f8_bytes.argtypes = [i64, i64, i64, ctypes.POINTER(i64)]
        L.zpq_matmul_f8.argtypes = [ctypes.POINTER(_F8), ctypes.POINTER(_F8), i64, i64, i64, vp, i32, i64, i32, vp,
                                    i64, vp]
        L.zpq_orthogonalize_bytes.argtypes = [i64, i64, i64, ctypes.POINTER(i64)]
        L.zpq_orthogonalize.argtypes = [vp, i32, i64, i64, i64, i64, i64, ctypes.POINTER(ctypes.c_double), i32, vp, i32, i64,
                                        i64, vp, i64, vp]
        L.zpq_muon_plan_bytes.argtypes = [ctypes.POINTER(_MuonMatrix), i32, ctypes.POINTER(i64)]
        L.zpq_muon_plan_make.argtypes = [ctypes.POINTER(_MuonMatrix), i32, i32, i32, i32, vp, i64, ctypes.POINTER(_MuonPlan), vp]
        L.zpq_muon_step.argtypes = [ctypes.POINTER(_MuonPlan), ctypes.POINTER(_MuonHyper), vp, vp]
        for f in (L.zpq_quant_i8, L.zpq_dequant_i8, L.zpq_quant_i8_tensor,
                  L.zpq_qgz_reorder_quant_i4, L.zpq_qgz_dequant_reduce_requant_i4,
                  L.zpq_list_make, L.zpq_grad_sumsq, L.zpq_adamw_plan_make, L.zpq_adamw_step,
                  L.zpq_adamw_step_at, L.zpq_state8_unpack, L.zpq_state8_pack, L.zpq_embedding, L.zpq_embedding_i8,
                  L.zpq_embedding_grad_bytes, L.zpq_embedding_grad, L.zpq_quant_f8, L.zpq_dequant_f8,
                  L.zpq_transpose_f8, L.zpq_matmul_f8_bytes, L.zpq_matmul_f8, L.zpq_orthogonalize_bytes,
                  L.zpq_orthogonalize, L.zpq_muon_plan_bytes, L.zpq_muon_plan_make, L.zpq_muon_step):
            f.restype = ctypes.c_int
        L.zpq_status_str.argtypes = [ctypes.c_int]
        L.zpq_status_str.restype = ctypes.c_char_p
        L.zpq_abi_version.argtypes = []
        L.zpq_abi_version.restype = ctypes.c_int32
        _lib = L
    return _lib


def _status_str(status):
    try:
        return lib().zpq_status_str(status).decode()
    except Exception:
        return STATUS.get(status, "unknown")


def _torch():
    import torch
    return torch


def dtype_code(dt):
    torch = _torch()
    codes = {torch.float32: ZPQ_F32, torch.float16: ZPQ_F16, torch.bfloat16: ZPQ_BF16}
    if dt not in codes:
        raise ValueError(f"unsupported element type {dt} (float32, float16 or bfloat16)")
    return codes[dt]


def torch_dtype(code):
    torch = _torch()
    return {ZPQ_F32: torch.float32, ZPQ_F16: torch.float16, ZPQ_BF16: torch.bfloat16}[code]


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(stream, device):
    torch = _torch()
    s = torch.cuda.current_stream(device) if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(rc, where):
    if rc != 0:
        raise ZpqError(rc, where)


def _gpu(t, name, device=None):
    """t must be a contiguous tensor on a GPU (on `device` when given): the
    library receives raw device pointers and checks neither."""
    if not t.is_cuda or not t.is_contiguous() or (device is not None and t.device != device):
        where = "a GPU" if device is None else str(device)
        raise ValueError(f"{name}: need a contiguous tensor on {where}, got "
                         f"{tuple(t.shape)} on {t.device}"
                         f"{'' if t.is_contiguous() else ' (not contiguous)'}")
    return t.device


def _need(t, dtype, numel, name, device):
    _gpu(t, name, device)
    if t.dtype != dtype or t.numel() != numel:
        raise ValueError(f"{name}: need {numel} elements of {dtype}, got {t.numel()} of {t.dtype}")


def _blocks(n, block):
    return n // block if block > 0 else 0       # a bad block is refused by the library


def quant_i8(x, block=256, out=None, stream=None):
    """qwZ INT8 block quantization: x (fp32/fp16/bf16, CUDA) -> (codes, scales)."""
    torch = _torch()
    dev = _gpu(x, "x")
    n = x.numel()
    if out is None:
        out = (torch.empty(n, dtype=torch.int8, device=dev),
               torch.empty(_blocks(n, block), dtype=torch.float32, device=dev))
    codes, scales = out
    _need(codes, torch.int8, n, "codes", dev)
    _need(scales, torch.float32, _blocks(n, block), "scales", dev)
    rc = lib().zpq_quant_i8(_ptr(x), dtype_code(x.dtype), n, block, _ptr(codes), _ptr(scales),
                            _stream(stream, dev))
    _check(rc, "zpq_quant_i8")
    return codes, scales


def quant_i8_tensor(x, out=None, stream=None):
    """Non-blocked INT8 quantization, one scale for all of x -> (codes, scale[1])."""
    torch = _torch()
    dev = _gpu(x, "x")
    n = x.numel()
    if out is None:
        out = (torch.empty(n, dtype=torch.int8, device=dev),
               torch.empty(1, dtype=torch.float32, device=dev))
    codes, scale = out
    _need(codes, torch.int8, n, "codes", dev)
    _need(scale, torch.float32, 1, "scale", dev)
    rc = lib().zpq_quant_i8_tensor(_ptr(x), dtype_code(x.dtype), n, _ptr(codes), _ptr(scale),
                                   _stream(stream, dev))
    _check(rc, "zpq_quant_i8_tensor")
    return codes, scale


def dequant_i8(codes, scales, block=256, dtype=None, out=None, stream=None):
    """qwZ INT8 block dequantization: (codes, scales) -> y of `dtype`."""
    torch = _torch()
    dev = _gpu(codes, "codes")
    n = codes.numel()
    _need(codes, torch.int8, n, "codes", dev)
    _need(scales, torch.float32, _blocks(n, block), "scales", dev)
    if out is None:
        out = torch.empty(n, dtype=dtype or torch.float16, device=dev)
    _need(out, out.dtype, n, "out", dev)
    rc = lib().zpq_dequant_i8(_ptr(codes), _ptr(scales), n, block, _ptr(out),
                              dtype_code(out.dtype), _stream(stream, dev))
    _check(rc, "zpq_dequant_i8")
    return out


def qgz_reorder_quant_i4(grad, local_ranks, nodes, block=128, out=None, stream=None):
    """qgZ slice reorder + INT4 block quantization -> (codes [n/2], scales [n/block])."""
    torch = _torch()
    dev = _gpu(grad, "grad")
    n = grad.numel()
    if out is None:
        out = (torch.empty(n // 2, dtype=torch.uint8, device=dev),
               torch.empty(_blocks(n, block), dtype=torch.float32, device=dev))
    codes, scales = out
    _need(codes, torch.uint8, n // 2, "codes", dev)
    _need(scales, torch.float32, _blocks(n, block), "scales", dev)
    rc = lib().zpq_qgz_reorder_quant_i4(_ptr(grad), dtype_code(grad.dtype), n, local_ranks, nodes,
                                        block, _ptr(codes), _ptr(scales), _stream(stream, dev))
    _check(rc, "zpq_qgz_reorder_quant_i4")
    return codes, scales


def qgz_dequant_reduce_requant_i4(in_codes, in_scales, n_src, chunk, block=128, out_dtype=None,
                                  divisor=1.0, out=None, stream=None):
    """qgZ receive side of one all-to-all hop.  Hop 1 (out_dtype None and out
    None or a (codes, scales) pair): -> (codes [chunk/2], scales [chunk/block]);
    hop 2: -> values [chunk] of out_dtype (or of out's type)."""
    torch = _torch()
    dev = _gpu(in_codes, "in_codes")
    _need(in_codes, torch.uint8, n_src * (chunk // 2), "in_codes", dev)
    _need(in_scales, torch.float32, n_src * _blocks(chunk, block), "in_scales", dev)
    if out_dtype is None and (out is None or isinstance(out, tuple)):
        if out is None:
            out = (torch.empty(chunk // 2, dtype=torch.uint8, device=dev),
                   torch.empty(_blocks(chunk, block), dtype=torch.float32, device=dev))
        oc, os_ = out
        _need(oc, torch.uint8, chunk // 2, "out_codes", dev)
        _need(os_, torch.float32, _blocks(chunk, block), "out_scales", dev)
        rc = lib().zpq_qgz_dequant_reduce_requant_i4(
            _ptr(in_codes), _ptr(in_scales), n_src, chunk, block, _ptr(oc), _ptr(os_),
            ctypes.c_void_p(0), 0, ctypes.c_float(1.0), _stream(stream, dev))
        _check(rc, "zpq_qgz_dequant_reduce_requant_i4")
        return oc, os_
    if out is None:
        out = torch.empty(chunk, dtype=out_dtype, device=dev)
    _need(out, out.dtype, chunk, "out", dev)
    rc = lib().zpq_qgz_dequant_reduce_requant_i4(
        _ptr(in_codes), _ptr(in_scales), n_src, chunk, block, ctypes.c_void_p(0),
        ctypes.c_void_p(0), _ptr(out), dtype_code(out.dtype), ctypes.c_float(divisor),
        _stream(stream, dev))
    _check(rc, "zpq_qgz_dequant_reduce_requant_i4")
    return out


def abi_version():
    return int(lib().zpq_abi_version())


# ---------------------------------------------------------------------------
# Around the communication path: optimizer step, gradient norm, embedding.
#
# The smallest of these calls take less time on the GPU than here, so the checks
# are plain comparisons and pointers go to ctypes as integers.
_here = contextlib.nullcontext()
_codes = {}


def _code(dt):
    c = _codes.get(dt)
    if c is None:
        c = _codes[dt] = dtype_code(dt)
    return c


@functools.lru_cache(maxsize=None)
def _raw_stream():
    """Device index -> pointer of its current stream: torch's short way, which is not
    public, where it is there."""
    torch = _torch()
    return getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on(stream, device):
    """(stream pointer, context): what a call allocates comes from the pool of
    the stream that it runs on, so that freeing it is ordered with its use."""
    torch = _torch()
    if stream is None:
        index = device.index
        raw = _raw_stream()(index)
        if index == torch.cuda.current_device():
            return raw, _here
        return raw, torch.cuda.stream(torch.cuda.current_stream(device))
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
    return stream.cuda_stream, torch.cuda.stream(stream)


class _Held:
    """Memory that a handle owns, with the stream that it was allocated on.  `used` tells
    the allocator of every other stream, so that memory of a handle that goes is
    not given out again while work there is under way."""

    def __init__(self):
        self.tensors, self.on = [], {}

    def add(self, tensors, home):
        for t in tensors:
            self.tensors.append((t, home))
            for raw, s in self.on.items():
                if raw != home:
                    t.record_stream(s)

    def used(self, raw, stream, device):
        if raw not in self.on:
            s = self.on[raw] = _torch().cuda.current_stream(device) if stream is None else stream
            for t, home in self.tensors:
                if raw != home:
                    t.record_stream(s)


def _one_device(tensors, name):
    """The tensors' common GPU; each must be contiguous and there."""
    dev = None
    for i, t in enumerate(tensors):
        dev = _gpu(t, f"{name}[{i}]", dev)
    return dev


def _one_dtype(tensors, name):
    kinds = {t.dtype for t in tensors}
    if len(kinds) != 1:
        raise ValueError(f"{name}: need tensors of one type, got {sorted(map(str, kinds))}")
    return _code(next(iter(kinds)))


class TensorList:
    """Tensors of one type on one GPU, laid out once for grad_sumsq.  Keeps the
    tensors; their storage must not be replaced (set_, resize_) meanwhile.  The
    table is written on `stream` (the current one by default) and also holds the
    partial sums of the call that runs: later calls must come after it and one
    after the other, in stream order.  A captured graph holds the table's address:
    keep the list as long as the graph.  Of a list made during a capture the table is
    written by each replay, not before the first."""

    def __init__(self, tensors, stream=None):
        self.tensors = list(tensors)
        if not self.tensors:
            raise ValueError("tensors: need at least one")
        self.device = _one_device(self.tensors, "tensors")
        dt = _one_dtype(self.tensors, "tensors")
        self._allocate(len(self.tensors), stream)
        self._lay_out([t.data_ptr() for t in self.tensors], [t.numel() for t in self.tensors], dt, stream)

    def _allocate(self, count, stream):
        self._c = _List()
        self._ref = ctypes.byref(self._c)
        self._held = _Held()
        st, ctx = _on(stream, self.device)
        with ctx:
            self._table = _torch().empty(count * 32 + LIST_FIXED_BYTES, dtype=_torch().uint8, device=self.device)
        self._held.add([self._table], st)

    def _lay_out(self, ptrs, sizes, dt, stream):
        n = len(ptrs)
        st, ctx = _on(stream, self.device)
        self._held.used(st, stream, self.device)
        with ctx:
            _check(lib().zpq_list_make((ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*sizes), n, dt,
                                       self._table.data_ptr(), self._table.numel(), self._ref, st),
                   "zpq_list_make")


def grad_sumsq(tensors, out=None, accumulate=False, stream=None):
    """Sum of squares of all elements, in float64 -> out [1] (out[0] += with
    accumulate: several lists, one norm).  tensors: a TensorList, or tensors."""
    torch = _torch()
    tl = tensors if isinstance(tensors, TensorList) else TensorList(tensors, stream=stream)
    st, ctx = _on(stream, tl.device)
    tl._held.used(st, stream, tl.device)
    with ctx:
        if out is not None:
            _need(out, torch.float64, 1, "out", tl.device)
        elif accumulate:
            raise ValueError("accumulate needs out")
        else:
            out = torch.empty(1, dtype=torch.float64, device=tl.device)
        _check(lib().zpq_grad_sumsq(tl._ref, out.data_ptr(), accumulate, st), "zpq_grad_sumsq")
    return out


class AdamW:
    """The AdamW step over many tensors in one launch.

    params        tensors of one type (float32, or float16 / bfloat16 without a master copy), updated in place
    grads         their gradients, of one type
    copies        with float32 params: float16 or bfloat16 tensors that receive the new weights
    weight_decay  one number, or one per tensor
    state_bits    32 (float32 moments) or 8 (zpq.h, zpq_adamw_step)
    exp_avg, exp_avg_sq
                  existing moments, one per tensor: float32 tensors, or with 8 bits pairs (codes
                  uint8 [n], exponents uint8 [ceil(n / 256)]); zeros are made where not given
    seed          of the random rounding of 8-bit states

    Tensors are kept and their addresses laid out once, on `stream` (the current
    one by default; later calls must come after it in stream order): storage must
    not be replaced meanwhile; set_grads() takes other gradients.  A captured graph
    holds addresses of this object's memory: keep it as long as the graph.  Made, or
    given gradients, during a capture, it has them from the first replay on."""

    def __init__(self, params, grads, copies=None, lr=1e-3, betas=(0.9, 0.999), eps=1e-8,
                 weight_decay=0.01, state_bits=32, exp_avg=None, exp_avg_sq=None, seed=0, stream=None):
        torch = _torch()
        self.params = list(params)
        if not self.params:
            raise ValueError("params: need at least one tensor")
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits: 8 or 32, got {state_bits}")
        self.device = _one_device(self.params, "params")
        self._pd = _one_dtype(self.params, "params")
        self.state_bits, self.lr, self.betas, self.eps, self.seed = state_bits, lr, tuple(betas), eps, seed
        count = len(self.params)
        self.weight_decay = list(weight_decay) if hasattr(weight_decay, "__len__") else [weight_decay] * count
        if len(self.weight_decay) != count:
            raise ValueError(f"weight_decay: need {count} numbers, got {len(self.weight_decay)}")
        self.copies = None if copies is None else list(copies)
        self._cd = -1
        if self.copies is not None:
            self._match(self.copies, "copies")
            self._cd = _one_dtype(self.copies, "copies")
            if self._cd == ZPQ_F32 or self._pd != ZPQ_F32:
                raise ValueError("copies: need float16 or bfloat16 tensors beside float32 params")
        self._held = _Held()
        st, ctx = _on(stream, self.device)
        with ctx:
            self.exp_avg = self._state(exp_avg, "exp_avg")
            self.exp_avg_sq = self._state(exp_avg_sq, "exp_avg_sq")
        for given, made in ((exp_avg, self.exp_avg), (exp_avg_sq, self.exp_avg_sq)):
            if given is None:
                self._held.add([t for x in made for t in (x if state_bits == 8 else (x,))], st)
        self._tables = {}                              # of each gradient type: the plan's table, the norm's list
        self._sizes = [p.numel() for p in self.params]
        self._rows = (_AdamwTensor * count)()
        spans = []                                     # of what the step writes
        for i, (r, p) in enumerate(zip(self._rows, self.params)):
            m, v = self.exp_avg[i], self.exp_avg_sq[i]
            written = [p] if self.copies is None else [p, self.copies[i]]
            if self.state_bits == 8:
                (m, me), (v, ve) = m, v
                r.m_exp, r.v_exp = me.data_ptr(), ve.data_ptr()
                written += [me, ve]
            r.p, r.m, r.v, r.n = p.data_ptr(), m.data_ptr(), v.data_ptr(), self._sizes[i]
            if self.copies is not None:
                r.copy = self.copies[i].data_ptr()
            r.weight_decay = self.weight_decay[i]
            if self._sizes[i]:
                spans += [(a, a + t.numel() * t.element_size()) for t in written + [m, v] for a in (t.data_ptr(),)]
        spans.sort()
        self._starts, self._ends = [a for a, _ in spans], [b for _, b in spans]
        if any(b > a for b, a in zip(self._ends, self._starts[1:])):
            raise ValueError("params, copies and moments overlap in memory (tied weights are one tensor)")
        self.set_grads(grads, stream=stream)

    def _match(self, tensors, name):
        if len(tensors) != len(self.params):
            raise ValueError(f"{name}: need {len(self.params)} tensors, got {len(tensors)}")
        for i, (t, p) in enumerate(zip(tensors, self.params)):
            _gpu(t, f"{name}[{i}]", self.device)
            if t.numel() != p.numel():
                raise ValueError(f"{name}[{i}]: need {p.numel()} elements, got {t.numel()}")

    def _state(self, given, name):
        torch = _torch()
        if self.state_bits == 32:
            if given is None:
                return [torch.zeros(p.numel(), dtype=torch.float32, device=self.device) for p in self.params]
            given = list(given)
            self._match(given, name)
            for i, t in enumerate(given):
                _need(t, torch.float32, t.numel(), f"{name}[{i}]", self.device)
            return given
        if given is None:
            zeros = lambda n: torch.zeros(n, dtype=torch.uint8, device=self.device)  # noqa: E731
            return [(zeros(p.numel()), zeros(-(-p.numel() // STATE_BLOCK))) for p in self.params]
        given = [tuple(x) for x in given]
        if any(len(x) != 2 for x in given):
            raise ValueError(f"{name}: need (codes, exponents) pairs with state_bits=8")
        self._match([c for c, _ in given], name)
        for i, (c, e) in enumerate(given):
            _need(c, torch.uint8, c.numel(), f"{name}[{i}] codes", self.device)
            _need(e, torch.uint8, -(-c.numel() // STATE_BLOCK), f"{name}[{i}] exponents", self.device)
        return given

    def set_grads(self, grads, stream=None):
        """Take these gradients from the next call on (in stream order).  A captured
        norm or step takes them too, from its next replay on: the tables stay where
        they are.  Gradients of another type have tables of their own; a graph that
        was captured with the earlier type goes on with its last gradients, which
        are kept for it."""
        grads = list(grads)
        self._match(grads, "grads")
        gd = _one_dtype(grads, "grads")
        width = grads[0].element_size()
        ptrs = [g.data_ptr() for g in grads]
        starts, ends = self._starts, self._ends
        for r, a, n in zip(self._rows, ptrs, self._sizes):
            r.g = a
            j = bisect.bisect_right(starts, a)
            if n and ((j and ends[j - 1] > a) or (j < len(starts) and starts[j] < a + n * width)):
                raise ValueError("grads overlap what the step writes")
        st, ctx = _on(stream, self.device)
        self._held.used(st, stream, self.device)
        plan = _AdamwPlan()
        with ctx:
            if gd not in self._tables:
                made = TensorList.__new__(TensorList)
                made.device = self.device
                made._allocate(len(grads), stream)
                self._tables[gd] = _torch().empty(len(grads) * 128 + 64, dtype=_torch().uint8, device=self.device), made
                self._held.add([self._tables[gd][0]], st)
            table, made = self._tables[gd]
            _check(lib().zpq_adamw_plan_make(self._rows, len(grads), self._pd, gd, self._cd, self.state_bits,
                                             table.data_ptr(), table.numel(), ctypes.byref(plan), st),
                   "zpq_adamw_plan_make")
            made._lay_out(ptrs, self._sizes, gd, stream)
            made.tensors = grads
            self._plan, self._ref, self._list, self.grads = plan, ctypes.byref(plan), made, grads

    def grad_sumsq(self, out=None, accumulate=False, stream=None):
        """Sum of squares of the gradients -> float64 [1] (see grad_sumsq)."""
        return grad_sumsq(self._list, out=out, accumulate=accumulate, stream=stream)

    def step(self, step, lr=None, grad_scale=1.0, sumsq=None, max_norm=None, stream=None):
        """Step number `step` (from 1), or a DeviceHyper.  sumsq: float64 [1] on the GPU, the
        squared norm of the unscaled gradients over all ranks; where it is not
        finite nothing changes.  max_norm: clip the scaled gradients to it
        (needs sumsq)."""
        norm = None
        if sumsq is not None:
            _need(sumsq, _torch().float64, 1, "sumsq", self.device)
            norm = sumsq.data_ptr()
        if isinstance(step, DeviceHyper):
            if lr is not None or max_norm is not None or grad_scale != 1.0:
                raise ValueError("lr, grad_scale and max_norm come from the DeviceHyper")
            if step.clips and norm is None:
                raise ValueError("max_norm needs sumsq")
            if step.data.device != self.device:
                raise ValueError(f"step: need a DeviceHyper on {self.device}, got one on {step.data.device}")
            st, ctx = _on(stream, self.device)
            self._held.used(st, stream, self.device)
            step._held.used(st, stream, self.device)
            with ctx:
                _check(lib().zpq_adamw_step_at(self._ref, step.data.data_ptr(), norm, st), "zpq_adamw_step_at")
            return
        if norm is None and max_norm is not None:
            raise ValueError("max_norm needs sumsq")
        h = self._hyper(step, lr, grad_scale, max_norm)
        st, ctx = _on(stream, self.device)
        self._held.used(st, stream, self.device)
        with ctx:
            _check(lib().zpq_adamw_step(self._ref, ctypes.byref(h), norm, st), "zpq_adamw_step")

    def _hyper(self, step, lr, grad_scale, max_norm):
        return _AdamwHyper(self.lr if lr is None else lr, self.betas[0], self.betas[1], self.eps, grad_scale,
                           _INF if max_norm is None else max_norm, step, self.seed)

    def device_hyper(self, step=1, lr=None, grad_scale=1.0, max_norm=None):
        """These hyperparameters in GPU memory, for step() in a captured graph."""
        return DeviceHyper(self._hyper(step, lr, grad_scale, max_norm), self.device, max_norm is not None)


class DeviceHyper:
    """A step's hyperparameters in GPU memory, read when the step runs: lr,
    grad_scale and max_norm are float64 [1] tensors, step an int64 [1] one, to be
    written in stream order (h.step.add_(1) in the graph, h.lr.fill_(x) before a
    replay).  Values out of range make the step do nothing.  max_norm counts only
    where step() gets a sumsq (one made with max_norm insists on it).  From
    AdamW.device_hyper, not during a capture."""

    def __init__(self, values, device, clips):
        torch = _torch()
        self.data = torch.frombuffer(bytearray(values), dtype=torch.float64).to(device)
        self.clips = clips
        self._held = _Held()
        self._held.add([self.data], _on(None, self.data.device)[0])
        self.lr, self.grad_scale, self.max_norm = self.data[0:1], self.data[4:5], self.data[5:6]
        self.step = self.data[6:7].view(torch.int64)


_INF = float("inf")


def state8_unpack(codes, exps, moment, dtype=None, out=None, stream=None):
    """Values of an 8-bit state of one tensor: moment 1 (exp_avg) or 2 (exp_avg_sq)."""
    torch = _torch()
    dev = _gpu(codes, "codes")
    n = codes.numel()
    if codes.dtype != torch.uint8:
        raise ValueError(f"codes: need uint8, got {codes.dtype}")
    _need(exps, torch.uint8, -(-n // STATE_BLOCK), "exps", dev)
    st, ctx = _on(stream, dev)
    with ctx:
        if out is None:
            out = torch.empty(n, dtype=dtype or torch.float32, device=dev)
        else:
            _need(out, out.dtype, n, "out", dev)
        _check(lib().zpq_state8_unpack(codes.data_ptr(), exps.data_ptr(), n, moment, out.data_ptr(),
                                       _code(out.dtype), st), "zpq_state8_unpack")
    return out


def state8_pack(x, moment, out=None, stream=None):
    """A float state as 8 bits, rounded to nearest -> (codes, exponents)."""
    torch = _torch()
    dev = _gpu(x, "x")
    n = x.numel()
    st, ctx = _on(stream, dev)
    with ctx:
        if out is None:
            out = (torch.empty(n, dtype=torch.uint8, device=dev),
                   torch.empty(-(-n // STATE_BLOCK), dtype=torch.uint8, device=dev))
        codes, exps = out
        _need(codes, torch.uint8, n, "codes", dev)
        _need(exps, torch.uint8, -(-n // STATE_BLOCK), "exps", dev)
        _check(lib().zpq_state8_pack(x.data_ptr(), _code(x.dtype), n, moment, codes.data_ptr(),
                                     exps.data_ptr(), st), "zpq_state8_pack")
    return codes, exps


def _ids(ids):
    torch = _torch()
    dev = _gpu(ids, "ids")
    if ids.dtype == torch.int64:
        return dev, 8
    if ids.dtype == torch.int32:
        return dev, 4
    raise ValueError(f"ids: need int32 or int64, got {ids.dtype}")


def _rows(t, name, device):
    """t as rows: a 2-D tensor on `device` whose rows are contiguous (they may
    lie further apart); returns (rows, dim, distance of rows)."""
    if t.dim() == 2 and t.device == device:
        n, d = t.shape
        ld, step = t.stride()
        if step == 1 or d <= 1:
            if n <= 1:
                return n, d, d
            if ld >= d:
                return n, d, ld
            raise ValueError(f"{name}: rows overlap (strides {tuple(t.stride())})")
    raise ValueError(f"{name}: need a 2-D tensor on {device} with contiguous rows, got "
                     f"{tuple(t.shape)} with strides {tuple(t.stride())} on {t.device}")


def _rows_of(t, name, device, rows, dim):
    """The distance of t's rows; t must be [rows, dim]."""
    n, d, ld = _rows(t, name, device)
    if n != rows or d != dim:
        raise ValueError(f"{name}: need {rows} x {dim}, got {tuple(t.shape)}")
    return ld


def _lookup_out(ids, dim, out, dtype, dev):
    """(output, distance of its rows)."""
    if out is None:
        return _torch().empty(ids.shape + (dim,), dtype=dtype, device=dev), dim
    return out, _rows_of(out if out.dim() == 2 else out.view(-1, out.shape[-1]), "out", dev, ids.numel(), dim)


def embedding(ids, table, scale=1.0, first=0, out_dtype=None, out=None, stream=None):
    """scale * table[ids - first] -> [*ids.shape, dim]; zeros where ids - first is
    not a row (padding, another shard's rows).  table [rows, dim]: float32,
    float16 or bfloat16, rows may lie apart."""
    dev, ib = _ids(ids)
    rows, dim, ld = _rows(table, "table", dev)
    st, ctx = _on(stream, dev)
    with ctx:
        out, lo = _lookup_out(ids, dim, out, out_dtype or table.dtype, dev)
        _check(lib().zpq_embedding(table.data_ptr(), _code(table.dtype), rows, dim, ld, ids.data_ptr(), ib,
                                   ids.numel(), first, scale, out.data_ptr(), _code(out.dtype), lo, st),
               "zpq_embedding")
    return out


def embedding_i8(ids, codes, scales, rows, dim, block=256, scale=1.0, first=0, out_dtype=None, out=None,
                 stream=None):
    """The same from a table as qwZ gathers it: int8 codes and one float32 scale
    per block of them (at least rows * dim; padding after it is not read)."""
    torch = _torch()
    dev, ib = _ids(ids)
    _gpu(codes, "codes", dev)
    _gpu(scales, "scales", dev)
    if codes.dtype != torch.int8 or codes.numel() < rows * dim:
        raise ValueError(f"codes: need {rows * dim} elements of int8, got {codes.numel()} of {codes.dtype}")
    if scales.dtype != torch.float32 or (block > 0 and scales.numel() < -(-rows * dim // block)):
        raise ValueError(f"scales: need {-(-rows * dim // max(block, 1))} elements of float32, got "
                         f"{scales.numel()} of {scales.dtype}")
    st, ctx = _on(stream, dev)
    with ctx:
        out, lo = _lookup_out(ids, dim, out, out_dtype or torch.float16, dev)
        _check(lib().zpq_embedding_i8(codes.data_ptr(), scales.data_ptr(), rows, dim, block, ids.data_ptr(), ib,
                                      ids.numel(), first, scale, out.data_ptr(), _code(out.dtype), lo, st),
               "zpq_embedding_i8")
    return out


@functools.lru_cache(maxsize=256)
def _grad_bytes(tokens, rows, dim):
    need = ctypes.c_int64()
    _check(lib().zpq_embedding_grad_bytes(tokens, rows, dim, ctypes.byref(need)), "zpq_embedding_grad_bytes")
    return need.value


def embedding_grad(ids, dy, rows, scale=1.0, first=0, padding=None, out_dtype=None, out=None,
                   accumulate=False, stream=None):
    """Dense gradient of the lookup: row r gets scale * the sum of dy over the
    tokens with ids - first == r (added to out with accumulate) -> [rows, dim].
    Ids outside and `padding` count for nothing.  The same ids give the same
    order of additions."""
    torch = _torch()
    dev, ib = _ids(ids)
    if dy.dim() != 2:
        _gpu(dy, "dy", dev)
        dy = dy.view(-1, dy.shape[-1])
    n, dim, ld = _rows(dy, "dy", dev)
    if n != ids.numel():
        raise ValueError(f"dy: need {ids.numel()} rows, got {n}")
    need = _grad_bytes(n, rows, dim)
    st, ctx = _on(stream, dev)
    with ctx:
        if out is not None:
            lo = _rows_of(out, "out", dev, rows, dim)
        elif accumulate:
            raise ValueError("accumulate needs out")
        else:
            out, lo = torch.empty((rows, dim), dtype=out_dtype or dy.dtype, device=dev), dim
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        _check(lib().zpq_embedding_grad(dy.data_ptr(), _code(dy.dtype), ld, ids.data_ptr(), ib, n, first,
                                        first - 1 if padding is None else padding, rows, dim, scale,
                                        out.data_ptr(), _code(out.dtype), lo, accumulate, ws.data_ptr(), need,
                                        st), "zpq_embedding_grad")
    return out


# ---------------------------------------------------------------------------
# Matrix products of the step, from 8-bit floating-point blocks of 128.  A matrix
# [rows, cols] is a pair: codes [rows, 128 * kb] of torch.float8_e4m3fn or float8_e5m2, and
# exponent bytes, uint8 [rows, kb4], or [ceil(rows / 128), kb4] of tiles (zpq.h).
F8_BLOCK = 128


@functools.lru_cache(maxsize=None)
def _kinds():
    torch = _torch()
    return {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}


def _kind(dtype, name):
    k = _kinds().get(dtype)
    if k is None:
        raise ValueError(f"{name}: need float8_e4m3fn or float8_e5m2, got {dtype}")
    return k


def _f8_shapes(rows, cols, tile):
    """Shapes of the codes and the exponent bytes of a [rows, cols] matrix."""
    kb = -(-cols // F8_BLOCK)
    return (rows, kb * F8_BLOCK), (-(-rows // F8_BLOCK) if tile else rows, -(-kb // 4) * 4)


@functools.lru_cache(maxsize=4096)
def _f8_shape(shape, dtype, scales, scales_dtype, name):
    """(kind, rows, blocks of a row, tile) of codes and scales of these shapes and types."""
    kind = _kind(dtype, f"{name} codes")
    if len(shape) != 2 or shape[1] % F8_BLOCK or len(scales) != 2 or scales_dtype != _torch().uint8:
        raise ValueError(f"{name}: need codes [rows, 128 * blocks] and uint8 scales [rows, blocks4], got "
                         f"{tuple(shape)} and {tuple(scales)} of {scales_dtype}")
    rows, width = shape
    of_rows, of_tiles = _f8_shapes(rows, width, False)[1], _f8_shapes(rows, width, True)[1]
    if tuple(scales) not in (of_rows, of_tiles):
        raise ValueError(f"{name} scales: need {of_rows} or, of tiles, {of_tiles}, got {tuple(scales)}")
    return kind, rows, width // F8_BLOCK, tuple(scales) != of_rows


def _f8_pair(pair, name, device=None):
    """Checks codes and scales; (device, kind, rows, blocks of a row, tile)."""
    codes, scales = pair
    dev = _gpu(codes, f"{name} codes", device)
    _gpu(scales, f"{name} scales", dev)
    return (dev,) + _f8_shape(codes.shape, codes.dtype, scales.shape, scales.dtype, name)


def _f8_cols(cols, blocks, name):
    """The matrix's columns: all of its blocks unless given."""
    if cols is None:
        return blocks * F8_BLOCK
    if cols < 0 or -(-cols // F8_BLOCK) != blocks:
        raise ValueError(f"{name}: {cols} columns are not {blocks} blocks")
    return cols


def _f8_new(out, name, rows, cols, tile, dtype, dev):
    """Codes and scales to be written: checked, or made."""
    torch = _torch()
    c, s = _f8_shapes(rows, cols, tile)
    if out is None:
        return torch.empty(c, dtype=dtype, device=dev), torch.empty(s, dtype=torch.uint8, device=dev)
    codes, scales = out
    _gpu(codes, f"{name} codes", dev)
    _gpu(scales, f"{name} scales", dev)
    if codes.dtype != dtype or tuple(codes.shape) != c or scales.dtype != torch.uint8 or tuple(scales.shape) != s:
        raise ValueError(f"{name}: need {c} of {dtype} and {s} of uint8, got {tuple(codes.shape)} of {codes.dtype} and "
                         f"{tuple(scales.shape)} of {scales.dtype}")
    return codes, scales


def quant_f8(x, tile=False, along="rows", dtype=None, out=None, stream=None):
    """x [rows, cols] (float32, float16 or bfloat16; rows may lie apart) as 8-bit floats
    with a power-of-two scale for each 128 elements of a row, or with tile for each 128 x 128.

    along  "rows": -> (codes, scales); "cols": those of the transposed matrix; "both": ((codes,
           scales), (codes, scales) of the transposed matrix), reading x once.  What a
           weight gradient sums over is the tokens: it takes "cols" of both its operands
    dtype  torch.float8_e4m3fn (default) or torch.float8_e5m2
    out    what is returned, to be written into"""
    torch = _torch()
    if along not in ("rows", "cols", "both"):
        raise ValueError(f"along: rows, cols or both, got {along!r}")
    if not x.is_cuda:
        raise ValueError(f"x: need a tensor on a GPU, got one on {x.device}")
    dtype = dtype or torch.float8_e4m3fn
    kind, dev = _kind(dtype, "dtype"), x.device
    rows, cols, ld = _rows(x, "x", dev)
    st, ctx = _on(stream, dev)
    with ctx:
        first, second = out if along == "both" and out is not None else (out, out)
        a = b = (None, None)
        if along != "cols":
            a = _f8_new(first, "out", rows, cols, tile, dtype, dev)
        if along != "rows":
            b = _f8_new(second, "out", cols, rows, tile, dtype, dev)
        ptrs = [None if t is None else t.data_ptr() for t in a + b]
        _check(lib().zpq_quant_f8(x.data_ptr(), _code(x.dtype), rows, cols, ld, kind, tile, *ptrs, st), "zpq_quant_f8")
    return (a, b) if along == "both" else a if along == "rows" else b


def dequant_f8(codes, scales, cols=None, dtype=None, out=None, stream=None):
    """The values of an 8-bit matrix -> [rows, cols] of dtype (bfloat16 by default); cols: of
    the matrix, where they are not whole blocks."""
    torch = _torch()
    dev, kind, rows, blocks, tile = _f8_pair((codes, scales), "matrix")
    cols = _f8_cols(cols, blocks, "cols")
    st, ctx = _on(stream, dev)
    with ctx:
        if out is None:
            out, ld = torch.empty((rows, cols), dtype=dtype or torch.bfloat16, device=dev), cols
        else:
            ld = _rows_of(out, "out", dev, rows, cols)
        _check(lib().zpq_dequant_f8(codes.data_ptr(), kind, scales.data_ptr(), rows, cols, tile, out.data_ptr(),
                                    _code(out.dtype), ld, st), "zpq_dequant_f8")
    return out


def transpose_f8(codes, scales, cols=None, out=None, stream=None):
    """The transposed matrix of one in tiles -> (codes, scales), the same values."""
    dev, kind, rows, blocks, tile = _f8_pair((codes, scales), "matrix")
    if not tile and scales.shape != _f8_shapes(rows, blocks * F8_BLOCK, True)[1]:
        raise ValueError("scales: need those of tiles")
    cols = _f8_cols(cols, blocks, "cols")
    st, ctx = _on(stream, dev)
    with ctx:
        to = _f8_new(out, "out", cols, rows, True, codes.dtype, dev)
        _check(lib().zpq_transpose_f8(codes.data_ptr(), scales.data_ptr(), rows, cols, to[0].data_ptr(),
                                      to[1].data_ptr(), st), "zpq_transpose_f8")
    return to


@functools.lru_cache(maxsize=1024)
def _matmul_bytes(m, n, k):
    need = ctypes.c_int64()
    _check(lib().zpq_matmul_f8_bytes(m, n, k, ctypes.byref(need)), "zpq_matmul_f8_bytes")
    return need.value


def matmul_f8(a, b, out_dtype=None, out=None, accumulate=False, stream=None):
    """a @ b.T for 8-bit matrices a [m, k] and b [n, k], pairs as quant_f8 gives them (of either
    type, along rows or in tiles) -> [m, n] of out_dtype (bfloat16 by default), or
    out, added to it with accumulate.  Sums are in binary32 for float32 and float16 results.  For
    bfloat16 ones, at twice the rate, the matrix core cuts products off 2^-13 below the largest of 8
    neighbours: up to 9e-5 of the result as a root mean square, where its rounding is 1.7e-3
    (zpq.h).  A pair says its columns in whole blocks only: a and b need as many blocks, and the
    shorter one counts as padded with the zeros that it is quantized with.  With x, dy [tokens, .]
    and w [outputs, inputs]: y = x w^T; dx = dy w = matmul_f8(dy, transpose_f8(*w)); dw = dy^T x, of
    both along their columns."""
    torch = _torch()
    dev, ka, m, blocks, ta = _f8_pair(a, "a")
    _, kb, n, blocks_b, tb = _f8_pair(b, "b", dev)
    if blocks != blocks_b:
        raise ValueError(f"a has {blocks} blocks in a row, b has {blocks_b}")
    k = blocks * F8_BLOCK
    need = _matmul_bytes(m, n, k)
    st, ctx = _on(stream, dev)
    with ctx:
        if out is not None:
            ld = _rows_of(out, "out", dev, m, n)
        elif accumulate:
            raise ValueError("accumulate needs out")
        else:
            out, ld = torch.empty((m, n), dtype=out_dtype or torch.bfloat16, device=dev), n
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        _check(lib().zpq_matmul_f8(_F8(a[0].data_ptr(), a[1].data_ptr(), ka, ta), _F8(b[0].data_ptr(), b[1].data_ptr(), kb, tb),
                                   m, n, k, out.data_ptr(), _code(out.dtype), ld, accumulate,
                                   None if ws is None else ws.data_ptr(), need, st), "zpq_matmul_f8")
    return out


# ---------------------------------------------------------------------------
# Orthogonalised updates.
NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)      # five times: singular values to between 0.7 and 1.2


@functools.lru_cache(maxsize=64)
def _coeffs(coeffs, steps):
    """(host array [steps][3], steps): one triple for every step, or one for each."""
    flat = [c for triple in coeffs for c in triple] if hasattr(coeffs[0], "__len__") else list(coeffs) * steps
    if len(flat) != 3 * steps:
        raise ValueError(f"coeffs: need three numbers, or three for each of {steps} steps")
    return (ctypes.c_double * max(len(flat), 1))(*flat), steps


def _coeffs_of(coeffs, steps):
    return _coeffs(tuple(tuple(c) if hasattr(c, "__len__") else float(c) for c in coeffs), int(steps))


@functools.lru_cache(maxsize=256)
def _orthogonalize_bytes(count, rows, cols):
    need = ctypes.c_int64()
    _check(lib().zpq_orthogonalize_bytes(count, rows, cols, ctypes.byref(need)), "zpq_orthogonalize_bytes")
    return need.value


def _stack(t, name, device):
    """t as matrices: 2-D, or 3-D with equally spaced ones, their rows contiguous (they may lie apart);
    (count, rows, cols, distance of rows, of matrices)."""
    if t.dim() == 2:
        return (1,) + _rows(t, name, device) + (0,)
    if t.dim() == 3 and t.device == device:
        count, rows, cols = t.shape
        apart, ld, step = t.stride()
        if count == 0 or rows == 0 or cols == 0:
            return count, rows, cols, cols, rows * cols
        if step == 1 or cols == 1:
            ld = cols if rows == 1 else ld
            span = (rows - 1) * ld + cols
            if ld >= cols and (count == 1 or apart >= span):
                return count, rows, cols, ld, apart if count > 1 else span
        raise ValueError(f"{name}: rows or matrices overlap, or rows are not contiguous (strides {tuple(t.stride())})")
    raise ValueError(f"{name}: need a 2-D or 3-D tensor on {device}, got {tuple(t.shape)} on {t.device}")


def orthogonalize(x, steps=5, coeffs=NEWTON_SCHULZ, out_dtype=None, out=None, stream=None):
    """x [rows, cols], or [count, rows, cols] of one shape, with its singular values driven towards 1
    by `steps` Newton-Schulz steps X <- a X + (b A + c A A) X, A = X X^T, from X = x / |x| -> out_dtype
    (bfloat16 by default, or float16).  coeffs: (a, b, c), or one triple for each step.  Zeros stay
    zeros; a matrix that is not finite comes out as NaN."""
    torch = _torch()
    if not x.is_cuda:
        raise ValueError(f"x: need a tensor on a GPU, got one on {x.device}")
    dev = x.device
    count, rows, cols, ld, apart = _stack(x, "x", dev)
    c, steps = _coeffs_of(coeffs, steps)
    need = _orthogonalize_bytes(count, rows, cols)
    st, ctx = _on(stream, dev)
    with ctx:
        if out is None:
            out = torch.empty(x.shape, dtype=out_dtype or torch.bfloat16, device=dev)
        elif out.shape != x.shape:
            raise ValueError(f"out: need {tuple(x.shape)}, got {tuple(out.shape)}")
        _, _, _, lo, apart_o = _stack(out, "out", dev)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        _check(lib().zpq_orthogonalize(x.data_ptr(), _code(x.dtype), count, rows, cols, ld, apart, c, steps, out.data_ptr(),
                                       _code(out.dtype), lo, apart_o, None if ws is None else ws.data_ptr(), need, st),
               "zpq_orthogonalize")
    return out


class Muon:
    """The Muon step over many matrices: momentum, orthogonalised by Newton-Schulz products, added
    to the weights.  For a layer's matrices; its vectors and embeddings are AdamW's.

    params        matrices of one type (float32, or float16 / bfloat16 without a master copy), updated in place
    grads         their gradients, of one type
    copies        with float32 params: float16 or bfloat16 tensors that receive the new weights
    weight_decay  one number, or one per matrix
    scale         of the orthogonal update, one number or one per matrix; by default
                  0.2 * sqrt(max(rows, cols)), about the size of an AdamW update at the same lr
    momenta       existing momenta, float32, one per matrix; zeros are made where not given

    Whole matrices: a rank of a sharded step gives those that it owns.  Tensors are kept and
    their addresses laid out once, on `stream` (the current one by default; later calls must come
    after it in stream order): storage must not be replaced meanwhile; set_grads() takes other
    gradients.  The object's memory, which the steps work in, holds about 14 bytes for each element
    of the matrices that are worked on at a time: its largest one, or consecutive ones up to 2^26
    elements and 1 GiB; and up to 0.5 GiB for parts of long sums (zpq.h).  A captured graph holds
    its addresses: keep the object as long as the graph."""

    def __init__(self, params, grads, copies=None, lr=1e-3, momentum=0.95, nesterov=True, weight_decay=0.0, scale=None,
                 steps=5, coeffs=NEWTON_SCHULZ, momenta=None, stream=None):
        torch = _torch()
        self.params = list(params)
        if not self.params:
            raise ValueError("params: need at least one matrix")
        self.device = _one_device(self.params, "params")
        for i, p in enumerate(self.params):
            if p.dim() != 2:
                raise ValueError(f"params[{i}]: need a matrix, got {tuple(p.shape)}")
        self._pd = _one_dtype(self.params, "params")
        self.lr, self.momentum, self.nesterov = lr, momentum, nesterov
        self._c, self.steps = _coeffs_of(coeffs, steps)
        count = len(self.params)
        if scale is None:
            scale = [0.2 * max(p.shape) ** 0.5 for p in self.params]
        self.weight_decay, self.scale = (list(v) if hasattr(v, "__len__") else [v] * count for v in (weight_decay, scale))
        for name in ("weight_decay", "scale"):
            if len(getattr(self, name)) != count:
                raise ValueError(f"{name}: need {count} numbers, got {len(getattr(self, name))}")
        self.copies = None if copies is None else list(copies)
        self._cd = -1
        if self.copies is not None:
            self._match(self.copies, "copies")
            self._cd = _one_dtype(self.copies, "copies")
            if self._cd == ZPQ_F32 or self._pd != ZPQ_F32:
                raise ValueError("copies: need float16 or bfloat16 tensors beside float32 params")
        self._held = _Held()
        st, ctx = _on(stream, self.device)
        with ctx:
            if momenta is None:
                self.momenta = [torch.zeros(p.shape, dtype=torch.float32, device=self.device) for p in self.params]
                self._held.add(self.momenta, st)
            else:
                self.momenta = list(momenta)
                self._match(self.momenta, "momenta")
                for i, t in enumerate(self.momenta):
                    _need(t, torch.float32, t.numel(), f"momenta[{i}]", self.device)
        self._rows = (_MuonMatrix * count)()
        spans = []                                     # of what the step writes
        for i, (r, p, m) in enumerate(zip(self._rows, self.params, self.momenta)):
            written = [p, m] if self.copies is None else [p, m, self.copies[i]]
            r.p, r.m, (r.rows, r.cols) = p.data_ptr(), m.data_ptr(), p.shape
            if self.copies is not None:
                r.copy = self.copies[i].data_ptr()
            r.weight_decay, r.scale = self.weight_decay[i], self.scale[i]
            if p.numel():
                spans += [(a, a + t.numel() * t.element_size()) for t in written for a in (t.data_ptr(),)]
        spans.sort()
        self._starts, self._ends = [a for a, _ in spans], [b for _, b in spans]
        if any(b > a for b, a in zip(self._ends, self._starts[1:])):
            raise ValueError("params, copies and momenta overlap in memory (tied weights are one matrix)")
        need = ctypes.c_int64()
        _check(lib().zpq_muon_plan_bytes(self._rows, count, ctypes.byref(need)), "zpq_muon_plan_bytes")
        with ctx:
            self._memory = torch.empty(need.value, dtype=torch.uint8, device=self.device)
        self._held.add([self._memory], st)
        self._list = None
        self.set_grads(grads, stream=stream)

    def _match(self, tensors, name):
        if len(tensors) != len(self.params):
            raise ValueError(f"{name}: need {len(self.params)} tensors, got {len(tensors)}")
        for i, (t, p) in enumerate(zip(tensors, self.params)):
            _gpu(t, f"{name}[{i}]", self.device)
            if t.shape != p.shape:
                raise ValueError(f"{name}[{i}]: need {tuple(p.shape)}, got {tuple(t.shape)}")

    def set_grads(self, grads, stream=None):
        """Take these gradients, of the type of the first ones, from the next call on (in stream order), also
        in a captured norm or step."""
        grads = list(grads)
        self._match(grads, "grads")
        gd = _one_dtype(grads, "grads")
        if self._list is not None and gd != self._gd:
            raise ValueError(f"grads: need {self.grads[0].dtype}, got {grads[0].dtype}")
        width = grads[0].element_size()
        starts, ends = self._starts, self._ends
        for g in grads:
            a, n = g.data_ptr(), g.numel()
            j = bisect.bisect_right(starts, a)
            if n and ((j and ends[j - 1] > a) or (j < len(starts) and starts[j] < a + n * width)):
                raise ValueError("grads overlap what the step writes")
        st, ctx = _on(stream, self.device)
        self._held.used(st, stream, self.device)
        plan = _MuonPlan()
        for r, g in zip(self._rows, grads):
            r.g = g.data_ptr()
        with ctx:
            made = self._list
            if made is None:
                made = TensorList.__new__(TensorList)
                made.device = self.device
                made._allocate(len(grads), stream)
            _check(lib().zpq_muon_plan_make(self._rows, len(grads), self._pd, gd, self._cd, self._memory.data_ptr(),
                                            self._memory.numel(), ctypes.byref(plan), st), "zpq_muon_plan_make")
            made._lay_out([g.data_ptr() for g in grads], [g.numel() for g in grads], gd, stream)
            made.tensors = grads
            self._plan, self._ref, self._list, self.grads, self._gd = plan, ctypes.byref(plan), made, grads, gd

    def grad_sumsq(self, out=None, accumulate=False, stream=None):
        """Sum of squares of the gradients -> float64 [1] (see grad_sumsq)."""
        return grad_sumsq(self._list, out=out, accumulate=accumulate, stream=stream)

    def step(self, lr=None, grad_scale=1.0, sumsq=None, max_norm=None, stream=None):
        """One step.  sumsq: float64 [1] on the GPU, the squared norm of the unscaled gradients over all
        ranks and optimizers; where it is not finite nothing changes.  max_norm: clip the scaled
        gradients to it (needs sumsq).  lr, momentum, grad_scale and max_norm are numbers of this call: a
        captured step goes on with those it was captured with (there is no DeviceHyper for it; capture it
        again to change them), while sumsq and the gradients are read at each replay."""
        norm = None
        if sumsq is not None:
            _need(sumsq, _torch().float64, 1, "sumsq", self.device)
            norm = sumsq.data_ptr()
        elif max_norm is not None:
            raise ValueError("max_norm needs sumsq")
        h = _MuonHyper(self.lr if lr is None else lr, self.momentum, grad_scale, _INF if max_norm is None else max_norm,
                       self._c, self.steps, self.nesterov)
        st, ctx = _on(stream, self.device)
        self._held.used(st, stream, self.device)
        with ctx:
            _check(lib().zpq_muon_step(self._ref, ctypes.byref(h), norm, st), "zpq_muon_step")
