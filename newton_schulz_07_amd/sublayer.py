"""The mixture-of-experts sublayer's operators, on torch tensors.

Argument marshalling only, as in the package itself: layer norm, routing of
tokens to experts, the experts' products with their gradients, and the
weighted sum of the experts' outputs.  The functions carry the C ABI's names
(include/ns_hip.h).  Nothing here is recorded by autograd: every gradient is a
call of its own.

    r = ns_route(logits, top_k=8)
    y = ns_experts_product(x, w, r.offsets, r.rows)
    out = ns_experts_combine(y, r.slots, r.weights)
    # backward
    dy, dweights = ns_experts_combine_backward(dout, y, r.slots, r.weights)
    dx = ns_experts_combine(ns_experts_input_grad(dy, w, r.offsets), r.slots)
    dw = ns_experts_weight_grad(dy, x, r.offsets, r.rows)   # [experts, fan_out, fan_in]
    dlogits = ns_route_backward(logits, r.ids, dweights)
"""

from typing import NamedTuple

import torch

from . import NS_DTYPE_BF16, NS_DTYPE_F32, _check, lib

NS_SCORE_SOFTMAX, NS_SCORE_SIGMOID = 0, 1
SCORES = {"softmax": NS_SCORE_SOFTMAX, "sigmoid": NS_SCORE_SIGMOID}


class Routing(NamedTuple):
    """What ns_route returns.  offsets, rows and slots are None if no plan was asked for."""
    ids: torch.Tensor       # int32 [..., top_k]
    weights: torch.Tensor   # fp32 [..., top_k]
    offsets: torch.Tensor   # int32 [experts + 1]
    rows: torch.Tensor      # int32 [tokens * top_k]
    slots: torch.Tensor     # int32 [..., top_k]


_stream_of = torch._C._cuda_getCurrentRawStream  # the device's current stream, without an object around it
_current_device = torch._C._cuda_getDevice
_functions = {}


def _call(name, like, *args):
    """lib().name(*args, stream) on the device of `like` and its current stream."""
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(lib(), name)
    dev = like.get_device()
    if _current_device() == dev:
        status = fn(*args, _stream_of(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _stream_of(dev))
    if status:
        _check(status)


def _rows_of(t, name):
    """(rows, cols, leading dimension) of a GPU tensor [..., cols] whose rows are evenly spaced."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dim() == 2:
        rows, cols = t.shape
        ld, unit = t.stride()
        if (unit == 1 or cols == 1) and (ld >= cols or rows <= 1):
            return rows, cols, (ld if rows > 1 else cols)
        raise ValueError(f"{name} must have contiguous rows")
    if t.dim() < 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, or a matrix with contiguous rows")
    cols = t.shape[-1]
    return (t.numel() // cols if cols else 0), cols, cols


def _dense(t, name, like=None, dtype=None, shape=None):
    """t, checked: on the GPU (of `like`), contiguous, of this dtype and shape."""
    if (t.is_cuda and t.is_contiguous() and (dtype is None or t.dtype == dtype) and (shape is None or t.shape == shape)
            and (like is None or t.get_device() == like.get_device())):
        return t
    if not t.is_cuda or (like is not None and t.device != like.device):
        raise ValueError(f"{name} must be a tensor on {'the GPU' if like is None else like.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")


def _out(t, name, like, dtype, shape):
    # (sizes one by one: torch takes longer over a tuple)
    return torch.empty(*shape, dtype=dtype, device=like.device) if t is None else _dense(t, name, like, dtype, shape)


def _out_like(t, name, like):
    if t is None and like.is_contiguous():
        return torch.empty_like(like)
    return _out(t, name, like, like.dtype, like.shape)


def _code(dtype):
    if dtype == torch.bfloat16:
        return NS_DTYPE_BF16
    if dtype == torch.float32:
        return NS_DTYPE_F32
    raise TypeError(f"unsupported dtype {dtype}: use torch.float32 or torch.bfloat16")


def _ptr(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------ layer norm


def ns_layer_norm(x, weight=None, bias=None, eps=1e-5, y=None, mean=None, rstd=None):
    """(y, mean, rstd) of a layer norm over the last dimension of x.

    x: [..., cols] fp32 or bf16 (a matrix may have spaced rows).  weight and
    bias: [cols], both fp32 or both bf16, or None.  mean, rstd: fp32 [rows],
    for the backward pass.
    """
    rows, cols, ld = _rows_of(x, "x")
    p = weight if weight is not None else bias
    if weight is not None:
        _dense(weight, "weight", x, None, (cols,))
    if bias is not None:
        _dense(bias, "bias", x, p.dtype, (cols,))
    y = _out_like(y, "y", x)
    mean = _out(mean, "mean", x, torch.float32, (rows,))
    rstd = _out(rstd, "rstd", x, torch.float32, (rows,))
    dt = _code(x.dtype)
    _call("ns_layer_norm", x, x.data_ptr(), ld, _ptr(weight), _ptr(bias), y.data_ptr(), mean.data_ptr(),
          rstd.data_ptr(), rows, cols, dt, dt if p is None else _code(p.dtype), eps)
    return y, mean, rstd


def ns_layer_norm_backward(dy, x, weight, mean, rstd, bias=True, dx=None, dweight=None, dbias=None):
    """(dx, dweight, dbias) of ns_layer_norm; dweight is None without a weight, dbias if `bias` is False.
    dweight and dbias have weight's type (fp32 without one)."""
    rows, cols, ld = _rows_of(x, "x")
    drows, dcols, ldd = _rows_of(dy, "dy")
    if dy.shape != x.shape or dy.dtype != x.dtype or dy.device != x.device:
        raise ValueError("dy must match x in shape, dtype and device")
    _dense(mean, "mean", x, torch.float32, (rows,))
    _dense(rstd, "rstd", x, torch.float32, (rows,))
    pt = torch.float32
    if weight is not None:
        pt = _dense(weight, "weight", x, None, (cols,)).dtype
        dweight = _out(dweight, "dweight", x, pt, (cols,))
    elif dweight is not None:
        raise ValueError("dweight without a weight")
    if bias:
        dbias = _out(dbias, "dbias", x, pt, (cols,))
    elif dbias is not None:
        raise ValueError("dbias with bias=False")
    dx = _out_like(dx, "dx", x)
    _call("ns_layer_norm_backward", x, dy.data_ptr(), ldd, x.data_ptr(), ld, _ptr(weight), mean.data_ptr(),
          rstd.data_ptr(), dx.data_ptr(), _ptr(dweight), _ptr(dbias), rows, cols, _code(x.dtype),
          _code(pt))
    return dx, dweight, dbias


# --------------------------------------------------------------- routing


def _score(score):
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}, got {score!r}")
    return SCORES[score]


def ns_route(logits, top_k, bias=None, groups=1, top_groups=1, group_best=2, score="softmax", renormalize=True,
             scale=1.0, plan=True):
    """Chooses top_k experts for each token: a Routing.

    logits: [..., experts] fp32 or bf16; -inf takes an expert out (it comes
    last, with weight 0).  bias: fp32 [experts], moves the choice only.
    groups, top_groups, group_best: only experts of the best top_groups of
    `groups` groups of neighbours, ranked by their group_best largest scores
    (with the bias; experts taken out add nothing).  score: "softmax" or
    "sigmoid".  plan=False: no offsets, rows and slots.
    """
    tokens, experts, ld = _rows_of(logits, "logits")
    code = _score(score)
    if bias is not None:
        _dense(bias, "bias", logits, torch.float32, (experts,))
    dev = logits.device
    ids = torch.empty(*logits.shape[:-1], top_k, dtype=torch.int32, device=dev)
    weights = torch.empty(*logits.shape[:-1], top_k, dtype=torch.float32, device=dev)
    offsets = rows = slots = None
    if plan:
        slots = torch.empty_like(ids)
        rows = torch.empty(tokens * top_k, dtype=torch.int32, device=dev)
        offsets = torch.empty(experts + 1, dtype=torch.int32, device=dev)
    _call("ns_route", logits, logits.data_ptr(), ld, _ptr(bias), ids.data_ptr(), weights.data_ptr(),
          _ptr(offsets), _ptr(rows), _ptr(slots), tokens, experts, top_k, groups, top_groups, group_best, code,
          1 if renormalize else 0, scale, _code(logits.dtype))
    return Routing(ids, weights, offsets, rows, slots)


def ns_route_backward(logits, ids, dweights, score="softmax", renormalize=True, scale=1.0, dlogits=None):
    """dlogits of ns_route from dweights, with the forward pass's arguments and its ids."""
    tokens, experts, ld = _rows_of(logits, "logits")
    code = _score(score)
    _dense(ids, "ids", logits, torch.int32)
    if ids.shape[:-1] != logits.shape[:-1]:
        raise ValueError("ids must have logits' leading shape")
    _dense(dweights, "dweights", logits, torch.float32, ids.shape)
    dlogits = _out_like(dlogits, "dlogits", logits)
    _call("ns_route_backward", logits, logits.data_ptr(), ld, ids.data_ptr(), dweights.data_ptr(),
          dlogits.data_ptr(), tokens, experts, ids.shape[-1], code, 1 if renormalize else 0, scale,
          _code(logits.dtype))
    return dlogits


# --------------------------------------------------- the experts' products


def _sorted_rows(x, rows, experts, offsets):
    """(n_x, fan_in, ldx, n_rows) of x read through rows (or not)."""
    n_x, fan_in, ld = _rows_of(x, "x")
    _dense(offsets, "offsets", x, torch.int32, (experts + 1,))
    if rows is None:
        return n_x, fan_in, ld, n_x
    _dense(rows, "rows", x, torch.int32)
    return n_x, fan_in, ld, rows.numel()


def ns_experts_product(x, w, offsets, rows=None, y=None):
    """y[i] = x[rows[i]] @ w[e].T for expert e's sorted rows offsets[e] .. offsets[e + 1].

    x: [n_x, fan_in]; w: [experts, fan_out, fan_in]; offsets, rows: int32,
    from ns_route (rows None: x is sorted already).  Returns y [n_rows,
    fan_out]; rows that no expert has (offsets that end below n_rows) are not
    written.
    """
    experts, fan_out, w_in = _dense(w, "w", x, x.dtype).shape
    n_x, fan_in, ld, n_rows = _sorted_rows(x, rows, experts, offsets)
    if w_in != fan_in:
        raise ValueError(f"w takes rows of {w_in}, x has rows of {fan_in}")
    y = _out(y, "y", x, x.dtype, (n_rows, fan_out))
    _call("ns_experts_product", x, x.data_ptr(), ld, n_x, _ptr(rows), w.data_ptr(), offsets.data_ptr(),
          y.data_ptr(), n_rows, experts, fan_out, fan_in, _code(x.dtype))
    return y


def ns_experts_input_grad(dy, w, offsets, dx=None):
    """dx[i] = dy[i] @ w[e] for the sorted rows: [n_rows, fan_in], rows that no expert has not written.
    ns_experts_combine(dx, slots) adds them up to the gradient of x."""
    experts, fan_out, fan_in = _dense(w, "w", dy, dy.dtype).shape
    n_rows = dy.shape[0]
    _dense(dy, "dy", w, None, (n_rows, fan_out))
    _dense(offsets, "offsets", dy, torch.int32, (experts + 1,))
    dx = _out(dx, "dx", dy, dy.dtype, (n_rows, fan_in))
    _call("ns_experts_input_grad", dy, dy.data_ptr(), w.data_ptr(), offsets.data_ptr(), dx.data_ptr(), n_rows,
          experts, fan_out, fan_in, _code(dy.dtype))
    return dx


def ns_experts_weight_grad(dy, x, offsets, rows=None, dw=None):
    """dw[e] = dy[i].T @ x[rows[i]] over expert e's sorted rows: [experts, fan_out, fan_in], zero for an expert
    without rows."""
    experts = offsets.numel() - 1
    n_x, fan_in, ld, n_rows = _sorted_rows(x, rows, experts, offsets)
    if dy.dim() != 2:
        raise ValueError("dy must be [n_rows, fan_out]")
    fan_out = dy.shape[1]
    _dense(dy, "dy", x, x.dtype, (n_rows, fan_out))
    dw = _out(dw, "dw", x, x.dtype, (experts, fan_out, fan_in))
    _call("ns_experts_weight_grad", x, dy.data_ptr(), x.data_ptr(), ld, n_x, _ptr(rows), offsets.data_ptr(),
          dw.data_ptr(), n_rows, experts, fan_out, fan_in, _code(x.dtype))
    return dw


# ---------------------------------------------------------------- combine


def _slots_of(slots, weights, like):
    _dense(slots, "slots", like, torch.int32)
    if slots.dim() < 1:
        raise ValueError("slots must be [..., top_k]")
    if weights is not None:
        _dense(weights, "weights", like, torch.float32, slots.shape)
    top_k = slots.shape[-1]
    return (slots.numel() // top_k if top_k else 0), top_k


def ns_experts_combine(y, slots, weights=None, out=None):
    """out[t] = sum_j weights[t, j] * y[slots[t, j]] (weights None: the plain sum): [..., cols] for slots
    [..., top_k]."""
    if y.dim() != 2:
        raise ValueError("y must be [n_rows, cols]")
    _dense(y, "y")
    tokens, top_k = _slots_of(slots, weights, y)
    n_rows, cols = y.shape
    out = _out(out, "out", y, y.dtype, (*slots.shape[:-1], cols))
    _call("ns_experts_combine", y, y.data_ptr(), slots.data_ptr(), _ptr(weights), out.data_ptr(), tokens,
          top_k, n_rows, cols, _code(y.dtype))
    return out


def ns_experts_combine_backward(dout, y, slots, weights=None, dy=None, dweights=None):
    """(dy, dweights) of ns_experts_combine; dweights is None without weights.

    No two slots may be the same.  Rows of y that are more than there are slots have a gradient of zero; where there
    are as many slots as rows, but some out of range, the rows that none names are not written: pass a dy of zeros.
    """
    if y.dim() != 2:
        raise ValueError("y must be [n_rows, cols]")
    _dense(y, "y")
    tokens, top_k = _slots_of(slots, weights, y)
    n_rows, cols = y.shape
    _dense(dout, "dout", y, y.dtype, (*slots.shape[:-1], cols))
    if dy is None and tokens * top_k != n_rows:
        dy = torch.zeros_like(y)  # rows that no slot names are not written
    dy = _out_like(dy, "dy", y)
    if weights is not None:
        dweights = _out_like(dweights, "dweights", weights)
    elif dweights is not None:
        raise ValueError("dweights without weights")
    _call("ns_experts_combine_backward", y, dout.data_ptr(), y.data_ptr(), slots.data_ptr(), _ptr(weights),
          dy.data_ptr(), _ptr(dweights), tokens, top_k, n_rows, cols, _code(y.dtype))
    return dy, dweights
