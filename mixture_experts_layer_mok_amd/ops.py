"""Torch-facing row operators and MXFP4 operators over the C ABI, for expert functions that
are not the layer's own:

    pos, offsets = layer.schedule_tables()             # views of the schedule's tables
    rows = permute(x, pos, torch.empty(max_rows, D))   # tokens to expert order
    codes, scales = quantize_mx4(rows)
    h = grouped_mx4(codes, scales, offsets, w_codes, w_scales)
    ...
    y = unpermute(rows, pos, weights)                  # and back, weighted
    d_rows, d_weights = unpermute_backward(dy, rows, pos, weights, d_rows)
    dx = permute_backward(d_rows, pos)

Ordinary calls run through the extension module _fast (the same checks and the same C entry
point in native code); what it does not take runs through the code here, which has the
messages.  Without an extension module that fits the running torch, every call does.

Every function checks its tensors (ValueError), makes one call of the C entry point of the
same name (MokError for what that refuses) on the tensors' device and returns without
synchronising.  Autograd records none of them: inputs may require grad, results do not, and the
gradients are functions of their own (for an autograd.Function to call).  Outputs that are
passed in count as changed in place, so that a backward pass which saved one raises.

Value tensors are bf16, fp16 or fp32 matrices whose rows are contiguous; the first lies at a
multiple of 16 bytes, the distance between them may be any multiple of 8 elements.  `stream` is
a torch stream or a raw handle; by default the current stream of the tensors' device.  Outputs
may be passed in; those allocated here belong to the stream the work runs on.
"""
from __future__ import annotations

import ctypes
import warnings

import torch

from . import _lib as L

_TYPES = {torch.bfloat16: L.MOK_TYPE_BF16, torch.float16: L.MOK_TYPE_FP16,
          torch.float32: L.MOK_TYPE_FP32}
_MAX = 2**31 - 1  # sizes that the entry points take as 32 bits


# Every check here runs on every call, so the ones that pass do little: messages are made only
# for what is refused.


def _matrix(name, t, rows=-1, cols=-1, dtype=None, write=False) -> tuple:
    """Checks a matrix with contiguous rows; returns (address, elements from row to row, end
    address)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: a tensor is wanted")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name}: a matrix is wanted")
    r, c = shape
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name}: {dtype} is wanted, not {t.dtype}")
    if (rows >= 0 and r != rows) or (cols >= 0 and c != cols):
        raise ValueError(f"{name}: {rows if rows >= 0 else 'any'} x {cols if cols >= 0 else 'any'} "
                         f"is wanted, not {r} x {c}")
    if c > _MAX:
        raise ValueError(f"{name}: a row has at most {_MAX} elements")
    ld, step = t.stride()
    if step != 1 and c > 1 and r > 0:  # (of no rows the strides say nothing)
        raise ValueError(f"{name}: rows must be contiguous")
    if r <= 1:
        ld = c  # the stride of a single row says nothing
    elif write and ld < c:
        raise ValueError(f"{name}: rows of an output overlap")
    p = t.data_ptr()
    return p, ld, p + ((r - 1) * ld + c) * t.element_size() if r and c else p


def _flat(name, t, shape, dtype) -> tuple:
    """Checks a contiguous tensor; returns (address, end address)."""
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype is not dtype or \
            not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor of shape {tuple(shape)} is wanted")
    p = t.data_ptr()
    return p, p + t.numel() * t.element_size()


def _type(name, t) -> int:
    try:
        return _TYPES[t.dtype]
    except (KeyError, AttributeError):
        raise ValueError(f"{name}: a bfloat16, float16 or float32 tensor is wanted") from None


def _apart(name, lo, hi, inputs) -> None:
    """An output [lo, hi) shares no memory with the inputs ((name, start, end) each)."""
    for other, a, b in inputs:
        if lo < b and a < hi and a != b and lo != hi:
            raise ValueError(f"{name} overlaps {other}")


def _same_device(dev, *tensors) -> None:
    for t in tensors:
        if t.device != dev:
            raise ValueError("the tensors are on different devices")
    if dev.type != "cuda":
        raise ValueError("the tensors must be on a GPU")


class _On:
    """The tensors' device made current where it is not, or the given stream made current
    (what is allocated inside belongs to it); gives the stream's handle."""

    __slots__ = ("index", "stream", "guard")

    def __init__(self, dev, stream):
        self.index, self.stream, self.guard = dev.index, stream, None

    def __enter__(self):
        s = self.stream
        if s is None:
            if self.index != torch.cuda.current_device():
                self.guard = torch.cuda.device(self.index)
                self.guard.__enter__()
            return _raw_stream(self.index)
        if isinstance(s, int):
            s = torch.cuda.ExternalStream(s, device=self.index)
        if s.device.index != self.index:
            raise ValueError("the stream is of another device than the tensors")
        self.guard = torch.cuda.stream(s)
        self.guard.__enter__()
        return s.cuda_stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)
        return False


# the current stream's handle without making a Stream object of it, where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(fn: str, *args) -> None:
    if not _bound:
        _bind(L.load())
    getattr(L, fn)(*args)


_fast = None  # the extension module, from the first call on, where there is one that fits
_bound = False  # it has been looked for


def _bind(lib) -> None:
    """Gives the extension module the library's entry points."""
    global _fast, _bound
    _bound = True
    try:
        from . import _fast as module

        fits = getattr(module, "torch_version", "unknown")
        if fits != torch.__version__:
            raise ImportError(f"it is built for torch {fits}")
    except ImportError as e:
        warnings.warn(f"the extension module _fast is not used ({e}); calls take a few microseconds "
                      "more of host time.  `python -m mixture_experts_layer_mok_amd.build` makes it",
                      RuntimeWarning, stacklevel=2)
        return
    names = ("mok_permute", "mok_permute_bwd", "mok_unpermute", "mok_unpermute_bwd",
             "mok_quantize_mx4", "mok_dequantize_mx4", "mok_grouped_mx4")
    module.bind(getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device), _raw_stream,
                *(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names))
    _fast = module


def _written(*outs) -> None:
    """Outputs passed in (None: made by the call): a graph that saved one finds it changed."""
    for t in outs:
        if t is not None and not t.is_inference():
            torch.autograd.graph.increment_version(t)


def _pos(pos) -> tuple:
    if not isinstance(pos, torch.Tensor) or pos.dim() != 2 or pos.dtype is not torch.int32 or \
            not pos.is_contiguous():
        raise ValueError("pos: a contiguous int32 matrix [tokens, top_k] is wanted")
    T, k = pos.shape
    if k > _MAX:
        raise ValueError(f"pos: a row has at most {_MAX} elements")
    p = pos.data_ptr()
    return T, k, p, p + 4 * T * k


def permute(x, pos, out, stream=None):
    """out[pos[t, j]] = x[t] for every pair with 0 <= pos < len(out); the other rows of out
    stay as they are.  x [T, D], pos [T, k] int32, out [max_rows, D]; returns out."""
    if stream is None and _fast is not None:
        done = _fast.permute(x, pos, out)
        if done is not None:
            return done
    T, k, pp, pe = _pos(pos)
    ty = _type("x", x)
    px, ld_x, xe = _matrix("x", x, T)
    D = x.shape[1]
    po, ld_o, oe = _matrix("out", out, -1, D, x.dtype, True)
    n = out.shape[0]
    _apart("out", po, oe, (("x", px, xe), ("pos", pp, pe)))
    dev = x.device
    _same_device(dev, pos, out)
    with _On(dev, stream) as st:
        _call("mok_permute", ty, px, ld_x, pp, T, k, D, po, ld_o, n, st)
    _written(out)
    return out


def _sum_rows(fn, rows, pos, weights, out, stream):
    T, k, pp, pe = _pos(pos)
    ty = _type("rows", rows)
    pr, ld_r, re = _matrix("rows", rows)
    n, D = rows.shape
    dev = rows.device
    inputs = [("rows", pr, re), ("pos", pp, pe)]
    pw = ()
    if weights is not None:
        w, we = _flat("weights", weights, (T, k), torch.float32)
        inputs.append(("weights", w, we))
        pw = (w,)
        _same_device(dev, weights)
    _same_device(dev, pos)
    given = out
    with _On(dev, stream) as st:
        if out is None:
            out = torch.empty(T, D, dtype=rows.dtype, device=dev)
        po, ld_o, oe = _matrix("out", out, T, D, rows.dtype, True)
        _apart("out", po, oe, inputs)
        _same_device(dev, out)
        _call(fn, ty, pr, ld_r, n, pp, *pw, T, k, D, po, ld_o, st)
    _written(given)
    return out


def permute_backward(d_rows, pos, out=None, stream=None):
    """Gradient of permute with respect to x: out[t] = sum over j of d_rows[pos[t, j]]."""
    if stream is None and _fast is not None:
        done = _fast.permute_backward(d_rows, pos, out)
        if done is not None:
            return done
    return _sum_rows("mok_permute_bwd", d_rows, pos, None, out, stream)


def unpermute(rows, pos, weights, out=None, stream=None):
    """out[t] = sum over j, ascending, of weights[t, j] * rows[pos[t, j]]; pairs whose pos is
    outside [0, len(rows)) are skipped.  rows [max_rows, D], weights [T, k] float32."""
    if stream is None and _fast is not None:
        done = _fast.unpermute(rows, pos, weights, out)
        if done is not None:
            return done
    if weights is None:
        raise ValueError("weights: a contiguous float32 tensor [tokens, top_k] is wanted")
    return _sum_rows("mok_unpermute", rows, pos, weights, out, stream)


def unpermute_backward(dy, rows, pos, weights, d_rows, d_weights=None, stream=None):
    """Gradients of unpermute: d_rows[pos[t, j]] = weights[t, j] * dy[t] (other rows of d_rows
    stay as they are) and d_weights[t, j] = <dy[t], rows[pos[t, j]]> (0 for pairs without a
    row).  Returns (d_rows, d_weights)."""
    if stream is None and _fast is not None:
        done = _fast.unpermute_backward(dy, rows, pos, weights, d_rows, d_weights)
        if done is not None:
            return done
    T, k, pp, pe = _pos(pos)
    ty = _type("rows", rows)
    pr, ld_r, re = _matrix("rows", rows)
    n, D = rows.shape
    py, ld_y, ye = _matrix("dy", dy, T, D, rows.dtype)
    pd, ld_d, de = _matrix("d_rows", d_rows, n, D, rows.dtype, True)
    pw, we = _flat("weights", weights, (T, k), torch.float32)
    dev = rows.device
    _same_device(dev, dy, pos, weights, d_rows)
    given = d_weights
    with _On(dev, stream) as st:
        if d_weights is None:
            d_weights = torch.empty(T, k, dtype=torch.float32, device=dev)
        pdw, dwe = _flat("d_weights", d_weights, (T, k), torch.float32)
        _same_device(dev, d_weights)
        inputs = (("dy", py, ye), ("rows", pr, re), ("pos", pp, pe), ("weights", pw, we))
        _apart("d_rows", pd, de, inputs)
        _apart("d_weights", pdw, dwe, inputs + (("d_rows", pd, de),))
        _call("mok_unpermute_bwd", ty, py, ld_y, pr, ld_r, n, pp, pw, T, k, D, pd, ld_d, pdw, st)
    _written(d_rows, given)
    return d_rows, d_weights


def _rows_of(name, t, cols, rows=-1, dtype=None, write=False) -> tuple:
    """A tensor [..., cols] as the matrix of its rows: (address, elements from row to row, end
    address, rows)."""
    if not isinstance(t, torch.Tensor) or t.dim() < 1 or t.shape[-1] != cols:
        raise ValueError(f"{name}: a tensor with a last axis of {cols} is wanted")
    if t.dim() != 2:
        try:
            t = t.view(-1, cols)
        except RuntimeError:
            raise ValueError(f"{name}: rows must lie at one distance") from None
    return (*_matrix(name, t, rows, cols, dtype, write), t.shape[0])


def quantize_mx4(src, codes=None, scales=None, stream=None):
    """MXFP4 codes [..., K / 2] and scales [..., K / 32] (uint8) of src [..., K], in blocks of
    32 along its last axis.  Returns (codes, scales)."""
    if stream is None and _fast is not None:
        done = _fast.quantize_mx4(src, codes, scales)
        if done is not None:
            return done
    ty = _type("src", src)
    K = src.shape[-1] if src.dim() else 0
    if K == 0 or K % 32:
        raise ValueError("src: a last axis that is a multiple of 32 is wanted")
    ps, ld_s, se, n = _rows_of("src", src, K)
    dev = src.device
    _same_device(dev)
    given = codes, scales
    with _On(dev, stream) as st:
        if codes is None:
            codes = torch.empty(*src.shape[:-1], K // 2, dtype=torch.uint8, device=dev)
        if scales is None:
            scales = torch.empty(*src.shape[:-1], K // 32, dtype=torch.uint8, device=dev)
        pc, ld_c, ce, _ = _rows_of("codes", codes, K // 2, n, torch.uint8, True)
        pq, ld_q, qe, _ = _rows_of("scales", scales, K // 32, n, torch.uint8, True)
        _same_device(dev, codes, scales)
        _apart("codes", pc, ce, (("src", ps, se),))
        _apart("scales", pq, qe, (("src", ps, se), ("codes", pc, ce)))
        _call("mok_quantize_mx4", ty, ps, ld_s, n, K, pc, ld_c, pq, ld_q, st)
    _written(*given)
    return codes, scales


def dequantize_mx4(codes, scales, dtype=torch.bfloat16, out=None, stream=None):
    """The values of MXFP4 codes [..., K / 2] and scales [..., K / 32], [..., K] in `dtype` (or
    in out's)."""
    if stream is None and _fast is not None:
        done = _fast.dequantize_mx4(codes, scales, dtype, out)
        if done is not None:
            return done
    if not isinstance(codes, torch.Tensor) or codes.dim() < 1 or codes.shape[-1] % 16 or \
            codes.shape[-1] == 0:
        raise ValueError("codes: a tensor with a last axis that is a multiple of 16 is wanted")
    K = codes.shape[-1] * 2
    pc, ld_c, ce, n = _rows_of("codes", codes, K // 2, -1, torch.uint8)
    pq, ld_q, qe, _ = _rows_of("scales", scales, K // 32, n, torch.uint8)
    if out is None and dtype not in _TYPES:
        raise ValueError("dtype: bfloat16, float16 or float32 is wanted")
    dev = codes.device
    _same_device(dev, scales)
    given = out
    with _On(dev, stream) as st:
        if out is None:
            out = torch.empty(*codes.shape[:-1], K, dtype=dtype, device=dev)
        ty = _type("out", out)
        po, ld_o, oe, _ = _rows_of("out", out, K, n, None, True)
        _same_device(dev, out)
        _apart("out", po, oe, (("codes", pc, ce), ("scales", pq, qe)))
        _call("mok_dequantize_mx4", pc, ld_c, pq, ld_q, n, K, ty, po, ld_o, st)
    _written(given)
    return out


def grouped_mx4(a, a_scales, offsets, b, b_scales, out=None, dtype=torch.bfloat16, stream=None):
    """out[r] = B[e] A[r] for the rows r of [offsets[e], offsets[e + 1]), every expert e; the
    other rows of out stay as they are (undefined where out is allocated here).

    a [max_rows, K / 2] MXFP4 codes (quantize_mx4), or [max_rows, K] MXFP8 codes
    (mok_quantize_mx), uint8, with a_scales [max_rows, K / 32]; offsets [E + 1] int32, on the
    device; b [E, N, K / 2] MXFP4 codes with b_scales [E, N, K / 32], contiguous; out
    [max_rows, N] bf16 or fp32."""
    if stream is None and _fast is not None:
        done = _fast.grouped_mx4(a, a_scales, offsets, b, b_scales, dtype, out)
        if done is not None:
            return done
    if not isinstance(b, torch.Tensor) or b.dim() != 3 or b.shape[2] % 16 or b.shape[2] == 0:
        raise ValueError("b: a tensor [E, N, K / 2] with K a multiple of 32 is wanted")
    E, N, half = b.shape
    if E > _MAX or N > _MAX:
        raise ValueError(f"b: at most {_MAX} experts and columns")
    K = 2 * half
    pb, be = _flat("b", b, (E, N, half), torch.uint8)
    pq, qe = _flat("b_scales", b_scales, (E, N, K // 32), torch.uint8)
    pf, fe = _flat("offsets", offsets, (E + 1,), torch.int32)
    pa, ld_a, ae = _matrix("a", a, dtype=torch.uint8)
    n, width = a.shape
    if width != half and width != K:
        raise ValueError(f"a: {half} (MXFP4) or {K} (MXFP8) columns are wanted, not {width}")
    pas, ld_as, ase = _matrix("a_scales", a_scales, n, K // 32, torch.uint8)
    if out is None and dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("dtype: bfloat16 or float32 is wanted")
    dev = a.device
    _same_device(dev, a_scales, offsets, b, b_scales)
    given = out
    with _On(dev, stream) as st:
        if out is None:
            out = torch.empty(n, N, dtype=dtype, device=dev)
        po, ld_o, oe = _matrix("out", out, n, N, None, True)
        if out.dtype is not torch.bfloat16 and out.dtype is not torch.float32:
            raise ValueError("out: bfloat16 or float32 is wanted")
        _same_device(dev, out)
        _apart("out", po, oe, (("a", pa, ae), ("a_scales", pas, ase), ("offsets", pf, fe),
                               ("b", pb, be), ("b_scales", pq, qe)))
        _call("mok_grouped_mx4", L.MOK_MX_E2M1 if width == half else L.MOK_MX_E4M3, pa, ld_a, pas,
              ld_as, n, pf, E, pb, pq, N, K, _TYPES[out.dtype], po, ld_o, st)
    _written(given)
    return out
