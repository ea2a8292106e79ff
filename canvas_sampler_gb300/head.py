"""The 8-bit output head: from hidden states to tokens with the vocabulary table in 8 bits.

PyTorch tensors in, pointers out (include/ds_sampler.h, "8-bit output head"); every computation is
one of the library's CUDA kernels. The four operators stand alone; OutputHead runs them together:

    head = OutputHead(E, norm_weight)                        # quantises E once
    logits, h = head.logits(x, residual)                     # norm -> 8-bit rows -> product
    token, prob = head.sample(x, u, residual, top_p=p)       # and a token per row

A call enqueues its work on `stream` (the current stream of the tensors' device by default),
allocates its outputs there and shares no workspace with any other call. There is no backward pass:
tensors that require a gradient are refused unless gradients are off (torch.no_grad()).
"""
from __future__ import annotations

import struct
from contextlib import contextmanager
from ctypes import byref, c_int32
from functools import lru_cache

import torch

from . import _lib as C

# PyTorch's own cheap forms of an allocation on the current device, the current device and a raw
# stream (0.9, 0.1 and 0.1 us on the host, where the public ones take 1.5, 0.2 and 2 us), else these.
# Allocations made so pass by the dispatcher, as the launches do.
try:
    from torch._C._dynamo.guards import _empty_strided_cuda
except ImportError:
    def _empty_strided_cuda(size, stride, dtype):
        return torch.empty_strided(size, stride, dtype=dtype, device="cuda")
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)

_FP8 = {"e4m3": (C.DS_FP8_E4M3, torch.float8_e4m3fn), "e5m2": (C.DS_FP8_E5M2, torch.float8_e5m2)}
_FP8_CODE = {t: c for c, t in _FP8.values()}
_DTYPES = {torch.bfloat16: C.DS_DTYPE_BF16, torch.float32: C.DS_DTYPE_FP32}
_OUT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_IMPLS = {"auto": C.DS_IMPL_AUTO, "tensor": C.DS_IMPL_TENSOR, "simt": C.DS_IMPL_SIMT}
BLOCK = 128


@lru_cache(maxsize=None)
def _entry(name: str):
    return C.packed_call(name, getattr(C, name + "_args"))


def _choice(name: str, table: dict, key):
    try:
        return table[key]
    except (KeyError, TypeError):
        raise ValueError(f"{name} must be one of {sorted(table)}, got {key!r}") from None


def _refuse_gradient(name: str) -> None:
    """These operators have no backward pass: outputs would leave the graph without a word."""
    if torch.is_grad_enabled():
        raise ValueError(f"{name} wants a gradient, which these operators do not give: call them "
                         "under torch.no_grad() or with detached tensors")


def _rows(name: str, t, shape: tuple, dtypes, dev: int) -> int:
    """Check a [rows, columns] argument whose columns are adjacent; the elements from one row to
    the next. A lone row has no next one: any stride that keeps its start's alignment serves."""
    if isinstance(t, torch.Tensor) and t.requires_grad:
        _refuse_gradient(name)
    if isinstance(t, torch.Tensor) and t.shape == shape and t.dtype in dtypes and \
            t.get_device() == dev and dev >= 0:
        s = t.stride()
        if s[1] == 1 or shape[1] <= 1:
            if shape[0] <= 1:
                return -(-shape[1] // 16) * 16
            if s[0] >= shape[1]:
                return s[0]
            raise ValueError(f"{name}: rows must not overlap")
        raise ValueError(f"{name}: columns must be adjacent in memory")
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D tensor")
    if t.get_device() < 0:
        raise ValueError(f"{name} must be on the device")
    if t.get_device() != dev:
        raise ValueError(f"{name}: expected cuda:{dev}, got {t.device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: expected {' or '.join(map(str, dtypes))}, got {t.dtype}")
    raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _vector(name: str, t, n: int, dtype, dev: int) -> int:
    """Check an [n] argument; its address, 0 for None."""
    if t is None:
        return 0
    if isinstance(t, torch.Tensor) and t.requires_grad:
        _refuse_gradient(name)
    if isinstance(t, torch.Tensor) and t.shape == (n,) and t.dtype is dtype and \
            t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape ({n},) on cuda:{dev}")


def _shape(name: str, t) -> tuple:
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D tensor")
    return t.shape


@contextmanager
def _elsewhere(dev: int, stream):
    """The tensors' device is current and outputs are allocated on the stream that writes them."""
    with torch.cuda.device(dev):
        if stream is None:
            yield torch.cuda.current_stream().cuda_stream
            return
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=dev)
        with torch.cuda.stream(stream):
            yield stream.cuda_stream


def _run(work, dev: int, stream):
    """work(raw stream) where the tensors live. A stream object has to be of their device (of a bare
    handle only the caller knows that)."""
    if stream is not None:
        on = getattr(stream, "device", None)
        if on is not None and on.index != dev:
            raise ValueError(f"stream: expected one of cuda:{dev}, got one of {on}")
    if stream is None and _current_device() == dev:  # (a tensor is on it: CUDA is up)
        return work(_raw_stream(dev))
    with _elsewhere(dev, stream) as raw:
        return work(raw)


def _call(name: str, raw: int, *fields) -> None:
    pack, fn = _entry(name)
    try:
        packed = pack(*fields)
    except (struct.error, OverflowError) as e:  # a number that its field cannot hold
        raise ValueError(f"{name}: {e}") from None
    status = fn(packed, raw)
    if status:
        C.check(status, name)


def _empty(rows: int, cols: int, dtype) -> torch.Tensor:
    return _empty_strided_cuda((rows, cols), (cols or 1, 1), dtype)


def _empty_codes(rows: int, cols: int, t8) -> torch.Tensor:
    """Codes whose rows start on 16-byte boundaries, as the tensor-core product wants them."""
    return _empty_strided_cuda((rows, cols), (-(-cols // 16) * 16 or 1, 1), t8)


_FLOATS = tuple(_DTYPES)
_CODES8 = tuple(_FP8_CODE)
_F32 = (torch.float32,)


def rmsnorm_fp8(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, *,
                eps: float = 1e-6, weight_offset: float = 0.0, fp8: str = "e4m3",
                out_h: torch.Tensor | None = None, stream=None):
    """ds_rmsnorm_fp8: h = x + residual, its norm in 8 bits. Returns (q [R, d], scales
    [R, ceil(d / 128)], h); h is x itself without a residual and out_h, else out_h (which may be x
    or residual) or a new tensor."""
    shape = R, d = _shape("x", x)
    dev, dt = x.get_device(), x.dtype
    x_stride = _rows("x", x, shape, _FLOATS, dev)
    if weight is None:
        raise ValueError("weight is required")
    w = _vector("weight", weight, d, dt, dev)
    r = r_stride = h_stride = 0
    if residual is not None:
        r_stride = _rows("residual", residual, shape, (dt,), dev)
        r = residual.data_ptr()
    if out_h is not None:
        h_stride = _rows("out_h", out_h, shape, (dt,), dev)
    code, t8 = _choice("fp8", _FP8, fp8)

    def work(raw):
        q = _empty_codes(R, d, t8)
        nb = -(-d // BLOCK)
        scales = _empty(R, nb, torch.float32)
        h, hs = out_h, h_stride
        if h is None and residual is not None:
            h, hs = _empty(R, d, dt), d
        _call("ds_rmsnorm_fp8", raw, R, d, _DTYPES[dt], code, eps, weight_offset, 0, x.data_ptr(),
              x_stride, r, r_stride, w, 0 if h is None else h.data_ptr(), hs, q.data_ptr(),
              -(-d // 16) * 16, scales.data_ptr(), nb)
        return q, scales, (x if h is None else h)

    return _run(work, dev, stream)


def quantize_fp8(x: torch.Tensor, *, block_rows: int = 128, fp8: str = "e4m3", stream=None):
    """ds_quantize_fp8: the 8-bit form of x [R, C] in blocks of block_rows (1 or 128) x 128.
    Returns (q [R, C], scales [ceil(R / block_rows), ceil(C / 128)])."""
    shape = R, cols = _shape("x", x)
    dev = x.get_device()
    x_stride = _rows("x", x, shape, _FLOATS, dev)
    if block_rows not in (1, BLOCK):
        raise ValueError(f"block_rows must be 1 or {BLOCK}")
    code, t8 = _choice("fp8", _FP8, fp8)

    def work(raw):
        q = _empty_codes(R, cols, t8)
        nb = -(-cols // BLOCK)
        scales = _empty(-(-R // block_rows), nb, torch.float32)
        _call("ds_quantize_fp8", raw, R, cols, _DTYPES[x.dtype], code, block_rows, x.data_ptr(),
              x_stride, q.data_ptr(), -(-cols // 16) * 16, scales.data_ptr(), nb)
        return q, scales

    return _run(work, dev, stream)


def matmul_fp8(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor, *,
               out_dtype: str = "bf16", out: torch.Tensor | None = None, impl: str = "auto",
               stream=None) -> torch.Tensor:
    """ds_matmul_fp8: [M, N] = A . B^T of 8-bit A [M, K] (scales [M, ceil(K / 128)]) and B [N, K]
    (scales [ceil(N / 128), ceil(K / 128)])."""
    M, K = _shape("a", a)
    N = _shape("b", b)[0]
    dev, nb, dt = a.get_device(), -(-K // BLOCK), _choice("out_dtype", _OUT, out_dtype)
    how = _choice("impl", _IMPLS, impl)
    strides = (_rows("a", a, (M, K), _CODES8, dev), _rows("a_scales", a_scales, (M, nb), _F32, dev),
               _rows("b", b, (N, K), _CODES8, dev),
               _rows("b_scales", b_scales, (-(-N // BLOCK), nb), _F32, dev))
    given = 0 if out is None else _rows("out", out, (M, N), (dt,), dev)

    def work(raw):
        o, os = out, given
        if o is None:
            o, os = _empty(M, N, dt), (N if M > 1 else -(-N // 16) * 16)
        _call("ds_matmul_fp8", raw, M, N, K, _FP8_CODE[a.dtype], _FP8_CODE[b.dtype], _DTYPES[dt],
              how, a.data_ptr(), strides[0], a_scales.data_ptr(), strides[1], b.data_ptr(),
              strides[2], b_scales.data_ptr(), strides[3], o.data_ptr(), os)
        return o

    return _run(work, dev, stream)


def sample_logits(logits: torch.Tensor, u: torch.Tensor, *, temperature: torch.Tensor | None = None,
                  top_k: torch.Tensor | None = None, top_p: torch.Tensor | None = None,
                  min_p: torch.Tensor | None = None, done: torch.Tensor | None = None,
                  out: tuple[torch.Tensor, torch.Tensor] | None = None, stream=None):
    """ds_sample_logits: a token per row of logits [R, V] by the random numbers u [R]. The
    filters are [R] tensors (top_k int32, the others float32) or None for off. Rows with done
    (uint8 [R]) set are left as `out` has them. Returns (token int32 [R], prob float32 [R])."""
    shape = R, V = _shape("logits", logits)
    dev = logits.get_device()
    stride = _rows("logits", logits, shape, _FLOATS, dev)
    if u is None:
        raise ValueError("u is required")
    f32 = torch.float32
    given = (_vector("temperature", temperature, R, f32, dev),
             _vector("top_k", top_k, R, torch.int32, dev), _vector("top_p", top_p, R, f32, dev),
             _vector("min_p", min_p, R, f32, dev), _vector("u", u, R, f32, dev),
             _vector("done", done, R, torch.uint8, dev))
    if out is not None:
        if out[0] is None or out[1] is None:
            raise ValueError("out: expected a pair of tensors")
        _vector("out[0]", out[0], R, torch.int32, dev)
        _vector("out[1]", out[1], R, f32, dev)
    elif done is not None:
        raise ValueError("done leaves rows untouched: pass out")

    def work(raw):
        token, prob = out if out is not None else (
            _empty_strided_cuda((R,), (1,), torch.int32), _empty_strided_cuda((R,), (1,), f32))
        _call("ds_sample_logits", raw, R, V, _DTYPES[logits.dtype], 0, logits.data_ptr(), stride,
              *given, token.data_ptr(), prob.data_ptr())
        return token, prob

    return _run(work, dev, stream)


def head_status(device=None, stream=None) -> int:
    """ds_head_status of a device (the current one by default): 0, or a DS_ERR_* code. Its error word
    is shared by all callers and streams of the device, and taken by this call."""
    v = c_int32()
    dev = torch.cuda.current_device() if device is None else torch.device(device).index

    def work(raw):
        C.check(C.load_library().ds_head_status(raw, byref(v)), "ds_head_status")
        return v.value

    return _run(work, torch.cuda.current_device() if dev is None else dev, stream)


class OutputHead:
    """A final norm and a vocabulary table held in 8 bits, from hidden states to tokens.

    E [V, d] (bf16 or fp32, on the device) is quantised once, in 128 x 128 blocks, on the current
    stream; norm_weight [d] has the hidden states' type. Both are constants here: parameters are taken
    without their gradients. The constructor returns when the table is
    ready (unless it is being captured into a graph), so calls on any stream may follow it. Calls share
    nothing but these read-only weights.
    """

    def __init__(self, E: torch.Tensor, norm_weight: torch.Tensor, *, eps: float = 1e-6,
                 weight_offset: float = 0.0, fp8: str = "e4m3", out_dtype: str = "bf16"):
        self.vocab, self.d = _shape("E", E)
        if norm_weight is None:
            raise ValueError("norm_weight is required")
        E, norm_weight = E.detach(), norm_weight.detach()
        _choice("fp8", _FP8, fp8)
        _choice("out_dtype", _OUT, out_dtype)
        _vector("norm_weight", norm_weight, self.d, norm_weight.dtype, E.get_device())
        self.q, self.scales = quantize_fp8(E, fp8=fp8)
        with torch.cuda.device(E.device):
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()
        self.norm_weight, self.eps, self.weight_offset = norm_weight, eps, weight_offset
        self.fp8, self.out_dtype = fp8, out_dtype

    def logits(self, x: torch.Tensor, residual: torch.Tensor | None = None, *, stream=None):
        """(logits [R, V], h [R, d]) of hidden states x [R, d] (+ residual)."""
        q, s, h = rmsnorm_fp8(x, self.norm_weight, residual, eps=self.eps,
                              weight_offset=self.weight_offset, fp8=self.fp8, stream=stream)
        return matmul_fp8(q, s, self.q, self.scales, out_dtype=self.out_dtype, stream=stream), h

    def sample(self, x: torch.Tensor, u: torch.Tensor, residual: torch.Tensor | None = None, *,
               stream=None, **filters):
        """(token [R], prob [R]) of hidden states x; filters as for sample_logits."""
        logits, _ = self.logits(x, residual, stream=stream)
        return sample_logits(logits, u, stream=stream, **filters)
