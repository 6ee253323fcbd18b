"""The sublayer in 8 bits, on torch tensors.

Argument marshalling only, as in the package itself: RMS norm with the
residual's addition, 8-bit values with scales, the experts' product of such
values, and the weight gradient from rows that were kept in them.  The functions
carry the C ABI's names (include/ns_hip.h).  Nothing here is recorded by
autograd: every gradient is a call of its own.

8-bit values are torch.float8_e4m3fn, their scales powers of two
(torch.float8_e8m0fnu), one for each 128 columns of a row or each 128 x 128 block
of a weight.

    n = ns_rms_norm(x, gamma, residual, outputs="scaled")        # n.total, n.q, n.scales
    w, wt = ns_quantize_weights(master, transposed=True)
    y = ns_experts_product_scaled(n.q, n.scales, *w, r.offsets, r.rows)
    # backward, from the rows kept in 8 bits
    dw = ns_experts_weight_grad_scaled(dy, n.q, n.scales, r.offsets, r.rows)
    dx = ns_experts_product_scaled(*ns_quantize(dy), *wt, r.offsets)      # sorted rows
    dh = ns_experts_combine(dx, r.slots)
    dx, dgamma = ns_rms_norm_backward(dh, n.total, gamma, n.rstd, dtotal=dout)
"""

from typing import NamedTuple, Optional

import torch

from .sublayer import _call, _code, _dense, _out, _out_like, _ptr, _rows_of

BLOCK = 128
EIGHT, SCALE = torch.float8_e4m3fn, torch.float8_e8m0fnu


class Scaled(NamedTuple):
    """Values in 8 bits: q float8_e4m3fn, scales float8_e8m0fnu."""
    q: torch.Tensor
    scales: torch.Tensor


class RMSNorm(NamedTuple):
    """What ns_rms_norm returns; what was not asked for is None."""
    y: Optional[torch.Tensor]
    rstd: torch.Tensor                # fp32 [rows]
    total: torch.Tensor               # x + residual, or x itself
    q: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]


def _blocks(n):
    return -(-n // BLOCK)


def _row_scales(shape):
    return (*shape[:-1], _blocks(shape[-1]))


def _eight_like(t, name, like):
    """t, checked, or a new tensor: 8-bit values of like's shape."""
    if t is None and like.is_contiguous():
        return torch.empty_like(like, dtype=EIGHT)  # (takes less time than torch.empty)
    return _out(t, name, like, EIGHT, like.shape)


def _weight_scales(shape):
    return (*shape[:-2], _blocks(shape[-2]), _blocks(shape[-1]))


# -------------------------------------------------------------- RMS norm


def ns_rms_norm(x, weight=None, residual=None, eps=1e-6, outputs="same", y=None, rstd=None, total=None, q=None,
                scales=None):
    """RMS norm over the last dimension of t = x + residual (x alone without one): an RMSNorm.

    x, residual: [..., cols] fp32 or bf16 (matrices may have spaced rows).
    weight: [cols] fp32 or bf16, or None.  outputs: "same" (y in x's type),
    "scaled" (y as 8-bit rows, cols a multiple of 16) or "both".
    """
    if outputs not in ("same", "scaled", "both"):
        raise ValueError(f"outputs must be 'same', 'scaled' or 'both', got {outputs!r}")
    rows, cols, ld = _rows_of(x, "x")
    dt = _code(x.dtype)
    ldr = cols
    if residual is not None:
        if residual.shape != x.shape or residual.dtype != x.dtype or residual.device != x.device:
            raise ValueError("residual must match x in shape, dtype and device")
        ldr = _rows_of(residual, "residual")[2]
        total = _out_like(total, "total", x)
    elif total is not None:
        raise ValueError("total without a residual")
    if weight is not None:
        _dense(weight, "weight", x, None, (cols,))
    if outputs != "scaled":
        y = _out_like(y, "y", x)
    elif y is not None:
        raise ValueError("y with outputs='scaled'")
    if outputs != "same":
        q = _eight_like(q, "q", x)
        scales = _out(scales, "scales", x, SCALE, _row_scales(x.shape))
    elif q is not None or scales is not None:
        raise ValueError("q or scales with outputs='same'")
    rstd = _out(rstd, "rstd", x, torch.float32, (rows,))
    _call("ns_rms_norm", x, x.data_ptr(), ld, _ptr(residual), ldr, _ptr(weight), _ptr(total), _ptr(y), _ptr(q),
          _ptr(scales), rstd.data_ptr(), rows, cols, dt, dt if weight is None else _code(weight.dtype), eps)
    return RMSNorm(y, rstd, x if residual is None else total, q, scales)


def ns_rms_norm_backward(dy, x, weight, rstd, dtotal=None, dx=None, dweight=None):
    """(dx, dweight) of ns_rms_norm; x is what the norm was taken of (its total).  dx is the gradient of x and of the
    residual alike; dtotal, the gradient that reaches total from elsewhere, is added to it.  dweight has weight's type
    and is None without a weight."""
    rows, cols, ld = _rows_of(x, "x")
    ldd, ldt = _rows_of(dy, "dy")[2], cols
    if dy.shape != x.shape or dy.dtype != x.dtype or dy.device != x.device:
        raise ValueError("dy must match x in shape, dtype and device")
    if dtotal is not None:
        if dtotal.shape != x.shape or dtotal.dtype != x.dtype or dtotal.device != x.device:
            raise ValueError("dtotal must match x in shape, dtype and device")
        ldt = _rows_of(dtotal, "dtotal")[2]
    _dense(rstd, "rstd", x, torch.float32, (rows,))
    pt = x.dtype
    if weight is not None:
        pt = _dense(weight, "weight", x, None, (cols,)).dtype
        dweight = _out(dweight, "dweight", x, pt, (cols,))
    elif dweight is not None:
        raise ValueError("dweight without a weight")
    dx = _out_like(dx, "dx", x)
    _call("ns_rms_norm_backward", x, dy.data_ptr(), ldd, x.data_ptr(), ld, _ptr(weight), rstd.data_ptr(), _ptr(dtotal),
          ldt, dx.data_ptr(), _ptr(dweight), rows, cols, _code(x.dtype), _code(pt))
    return dx, dweight


# ---------------------------------------------------------- quantization


def ns_quantize(x, q=None, scales=None):
    """x [..., cols] fp32 or bf16 (a matrix may have spaced rows), cols a multiple of 16, as 8-bit rows: a Scaled with
    scales [..., ceil(cols / 128)]."""
    rows, cols, ld = _rows_of(x, "x")
    q = _eight_like(q, "q", x)
    scales = _out(scales, "scales", x, SCALE, _row_scales(x.shape))
    _call("ns_quantize", x, x.data_ptr(), ld, q.data_ptr(), scales.data_ptr(), rows, cols, _code(x.dtype))
    return Scaled(q, scales)


def ns_quantize_weights(w, transposed=False):
    """w [fan_out, fan_in] or [experts, fan_out, fan_in], multiples of 16, as 8-bit weights: a Scaled with scales
    [..., ceil(fan_out / 128), ceil(fan_in / 128)].  transposed: a pair of them, the second of the same values
    transposed, for the gradient of the product's input."""
    _dense(w, "w")
    if w.dim() not in (2, 3):
        raise ValueError("w must be [fan_out, fan_in] or [experts, fan_out, fan_in]")
    fan_out, fan_in = w.shape[-2:]
    turned = (*w.shape[:-2], fan_in, fan_out)
    a = Scaled(_out(None, "q", w, EIGHT, w.shape), _out(None, "scales", w, SCALE, _weight_scales(w.shape)))
    b = Scaled(None, None)
    if transposed:
        b = Scaled(_out(None, "q", w, EIGHT, turned), _out(None, "scales", w, SCALE, _weight_scales(turned)))
    _call("ns_quantize_weights", w, w.data_ptr(), a.q.data_ptr(), a.scales.data_ptr(), _ptr(b.q), _ptr(b.scales),
          1 if w.dim() == 2 else w.shape[0], fan_out, fan_in, _code(w.dtype))
    return (a, b) if transposed else a


def ns_dequantize(q, scales, dtype=torch.bfloat16, out=None):
    """The values of 8-bit rows or weights (their scales' shape says which), in fp32 or bf16."""
    _dense(q, "q", None, EIGHT)
    if q.dim() < 1:
        raise ValueError("q must have rows")
    _dense(scales, "scales", q, SCALE)
    cols = q.shape[-1]
    if scales.shape == _row_scales(q.shape):
        matrices, rows, block_rows = 1, (q.numel() // cols if cols else 0), 1
    elif q.dim() in (2, 3) and scales.shape == _weight_scales(q.shape):
        matrices, rows, block_rows = (1 if q.dim() == 2 else q.shape[0]), q.shape[-2], BLOCK
    else:
        raise ValueError(f"scales of the shape {tuple(scales.shape)} belong neither to rows nor to weights of the shape "
                         f"{tuple(q.shape)}")
    code = _code(dtype)
    out = torch.empty_like(q, dtype=dtype) if out is None else _dense(out, "out", q, dtype, q.shape)
    _call("ns_dequantize", q, q.data_ptr(), scales.data_ptr(), out.data_ptr(), matrices, rows, cols, block_rows,
          code)
    return out


# --------------------------------------------------- the experts' products


def _scaled_rows(x, x_scales, rows):
    """(n_x, fan_in, n_rows) of 8-bit x read through rows (or not)."""
    _dense(x, "x", None, EIGHT)
    if x.dim() != 2:
        raise ValueError("x must be [n_x, fan_in]")
    n_x, fan_in = x.shape
    _dense(x_scales, "x_scales", x, SCALE, (n_x, _blocks(fan_in)))
    if rows is None:
        return n_x, fan_in, n_x
    _dense(rows, "rows", x, torch.int32)
    return n_x, fan_in, rows.numel()


def ns_experts_product_scaled(x, x_scales, w, w_scales, offsets=None, rows=None, dtype=torch.bfloat16, y=None):
    """y[i] = x[rows[i]] @ w[e].T for expert e's sorted rows offsets[e] .. offsets[e + 1], of 8-bit rows and weights.

    x, x_scales: 8-bit rows [n_x, fan_in]; w, w_scales: 8-bit weights [experts, fan_out, fan_in]; offsets, rows: int32,
    from ns_route (rows None: x is sorted already).  Without offsets there is one expert, which has all rows, and w may
    be [fan_out, fan_in]: a linear layer.  Returns y [n_rows, fan_out] in dtype: bf16, from products that are cut off at
    2^-13 of the largest of eight neighbours, or fp32, from exact ones, at half the rate (to be had in bf16 by rounding
    them: where large products cancel).  Rows that no expert has are not written.  With ns_quantize_weights' transposed weights and dy in 8 bits
    it is the gradient of x, row by row.
    """
    n_x, fan_in, n_rows = _scaled_rows(x, x_scales, rows)
    _dense(w, "w", x, EIGHT)
    if w.dim() not in (2, 3) or (w.dim() == 2 and offsets is not None):
        raise ValueError("w must be [experts, fan_out, fan_in] (or [fan_out, fan_in] without offsets)")
    experts, fan_out, w_in = (1, *w.shape) if w.dim() == 2 else w.shape
    if w_in != fan_in:
        raise ValueError(f"w takes rows of {w_in}, x has rows of {fan_in}")
    _dense(w_scales, "w_scales", x, SCALE, _weight_scales(w.shape))
    if offsets is not None:
        _dense(offsets, "offsets", x, torch.int32, (experts + 1,))
    elif experts != 1:
        raise ValueError("without offsets there is one expert")
    y = _out(y, "y", x, dtype, (n_rows, fan_out))
    _call("ns_experts_product_scaled", x, x.data_ptr(), x_scales.data_ptr(), n_x, _ptr(rows), w.data_ptr(),
          w_scales.data_ptr(), _ptr(offsets), y.data_ptr(), n_rows, experts, fan_out, fan_in, _code(dtype))
    return y


def ns_experts_weight_grad_scaled(dy, x, x_scales, offsets=None, rows=None, dw=None):
    """dw[e] = dy[i].T @ x[rows[i]] over expert e's sorted rows, from x kept in 8 bits: [experts, fan_out, fan_in] in
    dy's type (bf16 or fp32), zero for an expert without rows.  Without offsets there is one expert, which has all rows,
    and dw is [fan_out, fan_in]: a linear layer."""
    n_x, fan_in, n_rows = _scaled_rows(x, x_scales, rows)
    if offsets is not None:
        _dense(offsets, "offsets", x, torch.int32)
        if offsets.dim() != 1 or offsets.numel() < 2:
            raise ValueError("offsets must be [experts + 1]")
    if dy.dim() != 2:
        raise ValueError("dy must be [n_rows, fan_out]")
    experts, fan_out = 1 if offsets is None else offsets.numel() - 1, dy.shape[1]
    _dense(dy, "dy", x, None, (n_rows, fan_out))
    dw = _out(dw, "dw", x, dy.dtype, (fan_out, fan_in) if offsets is None else (experts, fan_out, fan_in))
    _call("ns_experts_weight_grad_scaled", x, dy.data_ptr(), x.data_ptr(), x_scales.data_ptr(), n_x, _ptr(rows),
          _ptr(offsets), dw.data_ptr(), n_rows, experts, fan_out, fan_in, _code(dy.dtype))
    return dw
