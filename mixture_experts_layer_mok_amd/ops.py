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

Every function checks its tensors (ValueError), makes one call of the C entry point of the
same name (MokError for what that refuses) on the tensors' device and returns without
synchronising.  Value tensors are bf16, fp16 or fp32 matrices whose rows are contiguous;
the distance between rows may be any multiple of 8 elements.  `stream` is a torch stream
or a raw handle; by default the current stream of the tensors' device.  Outputs may be
passed in; those allocated here belong to the stream the work runs on.
"""
from __future__ import annotations

import torch

from . import _lib as L

_TYPES = {torch.bfloat16: L.MOK_TYPE_BF16, torch.float16: L.MOK_TYPE_FP16,
          torch.float32: L.MOK_TYPE_FP32}


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _matrix(name: str, t: torch.Tensor, rows=None, cols=None, dtype=None, write=False) -> int:
    """Checks a matrix with contiguous rows; returns the elements from row to row."""
    _need(isinstance(t, torch.Tensor) and t.dim() == 2, f"{name}: a matrix is wanted")
    _need(dtype is None or t.dtype == dtype, f"{name}: {dtype} is wanted, not {t.dtype}")
    _need(rows is None or t.shape[0] == rows, f"{name}: {rows} rows are wanted")
    _need(cols is None or t.shape[1] == cols, f"{name}: {cols} columns are wanted")
    _need(t.shape[1] <= 1 or t.stride(1) == 1, f"{name}: rows must be contiguous")
    if t.shape[0] <= 1:
        return max(t.shape[1], 1)  # the stride of a single row says nothing
    _need(not write or t.stride(0) >= t.shape[1], f"{name}: rows of an output overlap")
    return t.stride(0)


def _contiguous(name: str, t: torch.Tensor, shape, dtype) -> None:
    _need(isinstance(t, torch.Tensor) and tuple(t.shape) == tuple(shape) and t.dtype == dtype and
          t.is_contiguous(), f"{name}: a contiguous {dtype} tensor of shape {tuple(shape)} is wanted")


def _type(name: str, t: torch.Tensor) -> int:
    _need(isinstance(t, torch.Tensor) and t.dtype in _TYPES,
          f"{name}: bfloat16, float16 or float32 is wanted")
    return _TYPES[t.dtype]


def _span(t: torch.Tensor) -> tuple[int, int]:
    p = t.data_ptr()
    if t.numel() == 0:
        return p, p
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return p, p + (last + 1) * t.element_size()


def _apart(outputs: dict, inputs: dict) -> None:
    """Outputs share no memory with inputs or with one another."""
    spans = [(n, *_span(t)) for n, t in outputs.items()]
    for i, (n, lo, hi) in enumerate(spans):
        for m, a, b in spans[i + 1:] + [(m, *_span(t)) for m, t in inputs.items()]:
            _need(hi <= a or b <= lo or lo == hi or a == b, f"{n} overlaps {m}")


class _On:
    """The device and stream of a call: the tensors' device is current inside, and what is
    allocated inside belongs to the stream."""

    def __init__(self, stream, *tensors):
        dev = tensors[0].device
        _need(all(t.device == dev for t in tensors), "the tensors are on different devices")
        _need(dev.type == "cuda", "the tensors must be on a GPU")
        self.index = dev.index
        self.stream = stream
        self.guard = None

    def __enter__(self):
        if self.stream is None:
            if self.index != torch.cuda.current_device():
                self.guard = torch.cuda.device(self.index)
                self.guard.__enter__()
            return torch.cuda.current_stream(self.index).cuda_stream
        s = self.stream
        if isinstance(s, int):
            s = torch.cuda.ExternalStream(s, device=self.index)
        _need(s.device.index == self.index, "the stream is of another device than the tensors")
        self.guard = torch.cuda.stream(s)
        self.guard.__enter__()
        return s.cuda_stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)
        return False


def _pos(pos: torch.Tensor) -> tuple[int, int]:
    _need(isinstance(pos, torch.Tensor) and pos.dim() == 2 and pos.dtype == torch.int32 and
          pos.is_contiguous(), "pos: a contiguous int32 matrix [tokens, top_k] is wanted")
    return pos.shape[0], pos.shape[1]


def permute(x, pos, out, stream=None):
    """out[pos[t, j]] = x[t] for every pair with 0 <= pos < len(out); the other rows of out
    stay as they are.  x [T, D], pos [T, k] int32, out [max_rows, D]; returns out."""
    T, k = _pos(pos)
    ty = _type("x", x)
    ld_x = _matrix("x", x, rows=T)
    ld_o = _matrix("out", out, cols=x.shape[1], dtype=x.dtype, write=True)
    _apart({"out": out}, {"x": x, "pos": pos})
    with _On(stream, x, pos, out) as st:
        L.mok_permute(ty, x, ld_x, pos, T, k, x.shape[1], out, ld_o, out.shape[0], st)
    return out


def permute_backward(d_rows, pos, out=None, stream=None):
    """Gradient of permute with respect to x: out[t] = sum over j of d_rows[pos[t, j]]."""
    T, k = _pos(pos)
    ty = _type("d_rows", d_rows)
    ld_r = _matrix("d_rows", d_rows)
    n, D = d_rows.shape
    with _On(stream, d_rows, pos, *(() if out is None else (out,))) as st:
        if out is None:
            out = torch.empty(T, D, dtype=d_rows.dtype, device=d_rows.device)
        ld_o = _matrix("out", out, rows=T, cols=D, dtype=d_rows.dtype, write=True)
        _apart({"out": out}, {"d_rows": d_rows, "pos": pos})
        L.mok_permute_bwd(ty, d_rows, ld_r, n, pos, T, k, D, out, ld_o, st)
    return out


def unpermute(rows, pos, weights, out=None, stream=None):
    """out[t] = sum over j, ascending, of weights[t, j] * rows[pos[t, j]]; pairs whose pos is
    outside [0, len(rows)) are skipped.  rows [max_rows, D], weights [T, k] float32."""
    T, k = _pos(pos)
    ty = _type("rows", rows)
    ld_r = _matrix("rows", rows)
    n, D = rows.shape
    _contiguous("weights", weights, (T, k), torch.float32)
    with _On(stream, rows, pos, weights, *(() if out is None else (out,))) as st:
        if out is None:
            out = torch.empty(T, D, dtype=rows.dtype, device=rows.device)
        ld_o = _matrix("out", out, rows=T, cols=D, dtype=rows.dtype, write=True)
        _apart({"out": out}, {"rows": rows, "pos": pos, "weights": weights})
        L.mok_unpermute(ty, rows, ld_r, n, pos, weights, T, k, D, out, ld_o, st)
    return out


def unpermute_backward(dy, rows, pos, weights, d_rows, d_weights=None, stream=None):
    """Gradients of unpermute: d_rows[pos[t, j]] = weights[t, j] * dy[t] (other rows of d_rows
    stay as they are) and d_weights[t, j] = <dy[t], rows[pos[t, j]]> (0 for pairs without a
    row).  Returns (d_rows, d_weights)."""
    T, k = _pos(pos)
    ty = _type("rows", rows)
    ld_r = _matrix("rows", rows)
    n, D = rows.shape
    ld_y = _matrix("dy", dy, rows=T, cols=D, dtype=rows.dtype)
    ld_d = _matrix("d_rows", d_rows, rows=n, cols=D, dtype=rows.dtype, write=True)
    _contiguous("weights", weights, (T, k), torch.float32)
    with _On(stream, dy, rows, pos, weights, d_rows,
             *(() if d_weights is None else (d_weights,))) as st:
        if d_weights is None:
            d_weights = torch.empty(T, k, dtype=torch.float32, device=rows.device)
        _contiguous("d_weights", d_weights, (T, k), torch.float32)
        _apart({"d_rows": d_rows, "d_weights": d_weights},
               {"dy": dy, "rows": rows, "pos": pos, "weights": weights})
        L.mok_unpermute_bwd(ty, dy, ld_y, rows, ld_r, n, pos, weights, T, k, D, d_rows, ld_d,
                            d_weights, st)
    return d_rows, d_weights


def _rows_of(name: str, t: torch.Tensor, cols: int) -> tuple[torch.Tensor, int]:
    """A tensor [..., cols] as the matrix of its rows (a view), and their distance."""
    _need(t.dim() >= 1 and t.shape[-1] == cols, f"{name}: a last axis of {cols} is wanted")
    if t.dim() != 2:
        try:
            t = t.view(-1, cols)
        except RuntimeError:
            raise ValueError(f"{name}: rows must lie at one distance") from None
    return t, _matrix(name, t)


def quantize_mx4(src, codes=None, scales=None, stream=None):
    """MXFP4 codes [..., K / 2] and scales [..., K / 32] (uint8) of src [..., K], in blocks of
    32 along its last axis.  Returns (codes, scales)."""
    ty = _type("src", src)
    _need(src.dim() >= 1 and src.shape[-1] % 32 == 0 and src.shape[-1] > 0,
          "src: a last axis that is a multiple of 32 is wanted")
    K = src.shape[-1]
    s, ld_s = _rows_of("src", src, K)
    with _On(stream, src, *(t for t in (codes, scales) if t is not None)) as st:
        if codes is None:
            codes = torch.empty(*src.shape[:-1], K // 2, dtype=torch.uint8, device=src.device)
        if scales is None:
            scales = torch.empty(*src.shape[:-1], K // 32, dtype=torch.uint8, device=src.device)
        ld_c, ld_sc = _codes_and_scales("codes", codes, scales, s.shape[0], K // 2, K, True)
        _apart({"codes": codes, "scales": scales}, {"src": src})
        L.mok_quantize_mx4(ty, s, ld_s, s.shape[0], K, codes, ld_c, scales, ld_sc, st)
    return codes, scales


def _codes_and_scales(name, codes, scales, rows, width, K, write=False):
    out = []
    for n, t, w in ((name, codes, width), (f"scales of {name}", scales, K // 32)):
        _need(isinstance(t, torch.Tensor) and t.dtype == torch.uint8, f"{n}: uint8 is wanted")
        m, _ = _rows_of(n, t, w)
        out.append(_matrix(n, m, rows=rows, write=write))
    return out


def dequantize_mx4(codes, scales, dtype=torch.bfloat16, out=None, stream=None):
    """The values of MXFP4 codes [..., K / 2] and scales [..., K / 32], [..., K] in `dtype` (or
    in out's)."""
    _need(isinstance(codes, torch.Tensor) and codes.dim() >= 1, "codes: a tensor is wanted")
    K = codes.shape[-1] * 2
    _need(K > 0 and K % 32 == 0, "codes: a last axis that is a multiple of 16 is wanted")
    c, ld_c = _rows_of("codes", codes, K // 2)
    _, ld_sc = _codes_and_scales("codes", codes, scales, c.shape[0], K // 2, K)
    _need(dtype in _TYPES, "dtype: bfloat16, float16 or float32 is wanted")
    with _On(stream, codes, scales, *(() if out is None else (out,))) as st:
        if out is None:
            out = torch.empty(*codes.shape[:-1], K, dtype=dtype, device=codes.device)
        ty = _type("out", out)
        o, _ = _rows_of("out", out, K)
        ld_o = _matrix("out", o, rows=c.shape[0], write=True)
        _apart({"out": out}, {"codes": codes, "scales": scales})
        L.mok_dequantize_mx4(c, ld_c, scales, ld_sc, c.shape[0], K, ty, o, ld_o, st)
    return out


def grouped_mx4(a, a_scales, offsets, b, b_scales, out=None, dtype=torch.bfloat16, stream=None):
    """out[r] = B[e] A[r] for the rows r of [offsets[e], offsets[e + 1]), every expert e; the
    other rows of out stay as they are (undefined where out is allocated here).

    a [max_rows, K / 2] MXFP4 codes (quantize_mx4), or [max_rows, K] MXFP8 codes
    (mok_quantize_mx), uint8, with a_scales [max_rows, K / 32]; offsets [E + 1] int32, on the
    device; b [E, N, K / 2] MXFP4 codes with b_scales [E, N, K / 32], contiguous; out
    [max_rows, N] bf16 or fp32."""
    _need(isinstance(b, torch.Tensor) and b.dim() == 3, "b: a tensor [E, N, K / 2] is wanted")
    E, N, half = b.shape
    K = 2 * half
    _need(K > 0 and K % 32 == 0, "b: a last axis that is a multiple of 16 is wanted")
    _contiguous("b", b, (E, N, half), torch.uint8)
    _contiguous("b_scales", b_scales, (E, N, K // 32), torch.uint8)
    _contiguous("offsets", offsets, (E + 1,), torch.int32)
    _need(isinstance(a, torch.Tensor) and a.dim() == 2 and a.shape[1] in (half, K),
          f"a: a matrix of {half} (MXFP4) or {K} (MXFP8) columns is wanted")
    fmt = L.MOK_MX_E2M1 if a.shape[1] == half else L.MOK_MX_E4M3
    n = a.shape[0]
    ld_a, ld_as = _codes_and_scales("a", a, a_scales, n, a.shape[1], K)
    _need(dtype in (torch.bfloat16, torch.float32), "dtype: bfloat16 or float32 is wanted")
    with _On(stream, a, a_scales, offsets, b, b_scales, *(() if out is None else (out,))) as st:
        if out is None:
            out = torch.empty(n, N, dtype=dtype, device=a.device)
        _need(out.dtype in (torch.bfloat16, torch.float32), "out: bfloat16 or float32 is wanted")
        ld_o = _matrix("out", out, rows=n, cols=N, write=True)
        _apart({"out": out}, {"a": a, "a_scales": a_scales, "offsets": offsets, "b": b,
                              "b_scales": b_scales})
        L.mok_grouped_mx4(fmt, a, ld_a, a_scales, ld_as, n, offsets, E, b, b_scales, N, K,
                          _TYPES[out.dtype], out, ld_o, st)
    return out
