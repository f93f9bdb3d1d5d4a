"""The other end of the tied table and the residual stream: embedding with its
gradient by sorted tokens, dropout from a counter-based generator, layer norm,
4-bit rows.

Argument marshalling only (the C ABI is include/invariant_layers.h), as in
token_ops.py; what is said there of HIP graphs holds here too.

Dropout's mask is never stored: it is a function of (seed, draw, row number,
column), and the backward pass computes it again.  seed is an integer, or a
one-element int64 tensor on the device that is read when the kernel runs, so
that a captured graph draws anew whenever the tensor changes; between a forward
and its backward it must stay as it is.  draw tells the calls of one seed apart
(a layer's number), first_row numbers a part of a batch as the whole would.
"""

import torch

from . import _lib
from .ops import _DTYPES, _INDEX, _dtype_code, _nbytes, _ptr, _row_vector
from .token_ops import (Fp4Rows, _call, _first_order, _fp4_operand, _norm_out, _norm_rows,
                        _norm_weight, _same_device, _stride, _workspace)


def _ids(t, device):
    if t.dtype not in _INDEX:
        raise TypeError("token_ids must be int64 or int32")
    if t.device != device:
        raise ValueError("token_ids must be on the table's device")
    return t.contiguous(), t.numel(), _INDEX[t.dtype]


def _table(t, name):
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1) or not t.is_cuda:
        raise ValueError(f"{name} must be [V, H] with contiguous rows on a ROCm device")
    return t.shape[0], t.shape[1], _stride(t)


def embedding_fwd(token_ids, weight, scale=1.0, ignore_index=-100, out=None, out_dtype=None):
    """Rows of weight [V, H] (float32, bfloat16, float16, or Fp4Rows) by token,
    times scale: [*token_ids.shape, H] in the weight's dtype (out_dtype, bfloat16
    unless given, from Fp4Rows).  token_ids int64 or int32; one equal to
    ignore_index gives a row of zeros, any other outside [0, V) a row of NaN."""
    fp4 = isinstance(weight, Fp4Rows)
    if fp4:
        v, h = _fp4_operand(weight, "weight")
        dev, dtype = weight.data.device, out_dtype or torch.bfloat16
    else:
        v, h, ld = _table(weight, "weight")
        dev, dtype = weight.device, weight.dtype
        if out_dtype not in (None, dtype):
            raise ValueError("out_dtype is for Fp4Rows; other tables give rows of their own dtype")
    if dtype not in _DTYPES:
        raise TypeError("rows must be float32, bfloat16 or float16")
    tok, n, tcode = _ids(token_ids, dev)
    shape = (*token_ids.shape, h)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev)
    elif tuple(out.shape) != shape or out.dtype != dtype or out.device != dev:
        raise ValueError(f"out must be a {dtype} tensor of shape {shape}")
    po, _, _, ld_o = _norm_rows(out, "out")
    if fp4:
        _call("embedding_fp4_fwd", dev, weight.data.data_ptr(), _stride(weight.data),
              weight.scale.data_ptr(), _stride(weight.scale), v, h, tok.data_ptr(), tcode, n,
              int(ignore_index), float(scale), _DTYPES[dtype], po, ld_o)
    else:
        _call("embedding_fwd", dev, weight.data_ptr(), ld, v, h, _DTYPES[dtype], tok.data_ptr(),
              tcode, n, int(ignore_index), float(scale), po, ld_o)
    return out


def embedding_bwd(token_ids, grad, num_rows, scale=1.0, ignore_index=-100, out_dtype=None,
                  dweight_out=None, accumulate=False, workspace=None):
    """Gradient [num_rows, H] of embedding_fwd's weight from grad
    [*token_ids.shape, H], in grad's dtype (out_dtype: that or float32): for every
    token the sum over its occurrences in ascending order, in float32, rounded
    once.  accumulate adds it to dweight_out, e.g. the dweight of a tied LM head
    (linear_token_logp_bwd), and leaves the rows of absent tokens as they are."""
    pg, n, h, ld_g = _norm_rows(grad, "grad")
    dev = grad.device
    tok, nt, tcode = _ids(token_ids, dev)
    if tuple(grad.shape[:-1]) != tuple(token_ids.shape):
        raise ValueError("grad must be [*token_ids.shape, H]")
    code = _dtype_code(grad)
    v = int(num_rows)
    if dweight_out is None:
        if accumulate:
            raise ValueError("accumulate needs the dweight_out that it adds to")
        dweight_out = torch.empty(v, h, dtype=out_dtype or grad.dtype, device=dev)
    if out_dtype not in (None, dweight_out.dtype):
        raise ValueError("dweight_out must be of out_dtype")
    if dweight_out.dtype not in (grad.dtype, torch.float32):
        raise TypeError("dweight must be float32 or of grad's dtype")
    v2, h2, ld = _table(dweight_out, "dweight_out")
    if (v2, h2) != (v, h) or dweight_out.device != dev:
        raise ValueError("dweight_out must be [num_rows, H] on grad's device")
    ws = _workspace(workspace, _lib.lib().embedding_bwd_workspace_bytes(nt, v, h), dev)
    _call("embedding_bwd", dev, pg, ld_g, code, tok.data_ptr(), tcode, nt, v, h, int(ignore_index),
          float(scale), _DTYPES[dweight_out.dtype], int(bool(accumulate)), dweight_out.data_ptr(),
          ld, _ptr(ws), _nbytes(ws))
    return dweight_out


# The backward passes of the autograd functions run in a thread of their own, where
# every object of the interpreter that they touch comes from another core's cache:
# what the forward has checked is not checked again, sizes come along as integers
# (training calls on few rows: layer norm 142 -> 126 to 131 us, dropout 84 -> 74, embedding
# 97 -> 88; a call of nothing but tensors handed on takes 40 to 67).  Hooks on saved
# tensors may have moved them: addresses and strides are those of the backward.
class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, token_ids, weight, scale, ignore_index):
        out = embedding_fwd(token_ids, weight, scale, ignore_index)
        tok, n, tcode = _ids(token_ids, weight.device)
        v, h = weight.shape
        ctx.save_for_backward(tok)
        ctx.sizes = (_DTYPES[weight.dtype], tcode, n, v, h, ignore_index, scale,
                     _lib.lib().embedding_bwd_workspace_bytes(n, v, h))
        return out

    @staticmethod
    @_first_order
    def backward(ctx, g):
        (tok,) = ctx.saved_tensors
        code, tcode, n, v, h, ignore_index, scale, nbytes = ctx.sizes
        g = g.contiguous()
        dw = torch.empty((v, h), dtype=g.dtype, device=g.device)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=g.device)
        _call("embedding_bwd", g.device, g.data_ptr(), h, code, tok.data_ptr(), tcode, n, v, h,
              ignore_index, scale, code, 0, dw.data_ptr(), h, ws.data_ptr(), nbytes)
        return None, dw, None, None


def embedding(token_ids, weight, scale=1.0, ignore_index=-100):
    """Differentiable embedding_fwd of a weight [V, H] (not Fp4Rows): its gradient
    is whole, in the weight's dtype."""
    if isinstance(weight, Fp4Rows):
        raise TypeError("4-bit rows have no gradient: embedding_fwd looks them up")
    return _Embedding.apply(token_ids, weight, float(scale), int(ignore_index))


def _seed(seed, device):
    """(value, pointer or None) of a seed."""
    if isinstance(seed, torch.Tensor):
        if seed.dtype != torch.int64 or seed.numel() != 1 or seed.device != device:
            raise ValueError("a seed tensor must be one int64 on the rows' device")
        return 0, seed.data_ptr()
    value = int(seed) & (2 ** 64 - 1)
    return value - 2 ** 64 if value >= 2 ** 63 else value, None


def _place(draw, first_row):
    """(draw, first_row) as the library's integers hold them."""
    draw, first_row = int(draw), int(first_row)
    if draw >> 32 or first_row >> 63:
        raise ValueError("draw must be in [0, 2^32) and first_row in [0, 2^63)")
    return draw, first_row


def _dropout(x, residual, out, drop):
    """(out, the sizes of its backward)."""
    px, n, h, ld_x = _norm_rows(x, "x")
    code = _dtype_code(x)
    pr, ld_r = None, 0
    if residual is not None:
        pr, _, _, ld_r = _norm_rows(residual, "residual", x)
    out, po, ld_o = _norm_out(out, "out", x, h)
    _call("dropout_fwd", x.device, px, ld_x, pr, ld_r, code, n, h, *drop, po, ld_o)
    return out, (code, n, h)


def _dropout_args(p, seed, draw, first_row, device):
    if seed is None:
        if p:
            raise ValueError("dropout needs a seed")
        seed = 0
    return (float(p), *_seed(seed, device), *_place(draw, first_row))


def dropout_fwd(x, p, seed, residual=None, draw=0, first_row=0, out=None):
    """residual + dropped(x) (dropped(x) without a residual), rounded once to x's
    dtype: an element of x [*lead, H] (float32, bfloat16, float16) is dropped with
    probability p (to 2^-16), the others are scaled by the reciprocal of what is
    kept.  seed may be None where p is 0.  out may be x or residual."""
    return _dropout(x, residual, out, _dropout_args(p, seed, draw, first_row, x.device))[0]


def dropout_bwd(grad, p, seed, draw=0, first_row=0, dx_out=None):
    """Gradient of dropout_fwd's x from that of its output (which is the
    residual's gradient itself).  dx_out may be grad."""
    return dropout_fwd(grad, p, seed, None, draw, first_row, dx_out)


def _seed_again(drop, saved):
    """drop with the seed where it is now: hooks on saved tensors may have moved it."""
    return (*drop[:2], saved[0].data_ptr(), *drop[3:]) if saved else drop


def _dropout_back(g, drop, code, n, h):
    """dropout's gradient of x from contiguous rows g."""
    dx = torch.empty_like(g)
    _call("dropout_fwd", g.device, g.data_ptr(), h, None, 0, code, n, h, *drop, dx.data_ptr(), h)
    return dx


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, p, seed, residual, draw, first_row):
        drop = _dropout_args(p, seed, draw, first_row, x.device)
        out, sizes = _dropout(x, residual, None, drop)
        if drop[2] is not None:
            ctx.save_for_backward(seed)
        ctx.sizes = (drop, *sizes)
        return out

    @staticmethod
    @_first_order
    def backward(ctx, g):
        saved = ctx.saved_tensors  # a seed that has changed raises
        drop, code, n, h = ctx.sizes
        g = g.contiguous()
        need = ctx.needs_input_grad
        dx = _dropout_back(g, _seed_again(drop, saved), code, n, h) if need[0] else None
        return dx, None, None, g if need[3] else None, None, None


def dropout(x, p, seed, residual=None, draw=0, first_row=0):
    """Differentiable dropout_fwd; the mask is computed again in the backward."""
    return _Dropout.apply(x, float(p), seed, residual, int(draw), int(first_row))


def _norm_bias(bias, x):
    return _norm_weight(bias, x, "bias") if bias is not None else None


def _drop_args(p, seed, draw, first_row, device):
    """The library's (p, seed, its address, draw, first row)."""
    if not p:
        return 0.0, 0, None, 0, 0
    return _dropout_args(p, seed, draw, first_row, device)


def _layer_norm_forward(x, weight, bias, residual, eps, drop, stats, y_out, sum_out):
    """(y, s, the sizes of its backward), with the rows' means and then their rstd in
    stats [2 N] (or None)."""
    px, n, h, ld_x = _norm_rows(x, "x")
    code = _dtype_code(x)
    pw, pb = _norm_weight(weight, x), _norm_bias(bias, x)
    y, py, ld_y = _norm_out(y_out, "y_out", x, h)
    pr, ld_r, ps, ld_s, s = None, 0, None, 0, x
    if residual is not None:
        pr, _, _, ld_r = _norm_rows(residual, "residual", x)
    if residual is not None or drop[0] or sum_out is not None:
        s, ps, ld_s = _norm_out(sum_out, "sum_out", x, h)
    pm = stats.data_ptr() if stats is not None else None
    _call("layer_norm_fwd", x.device, px, ld_x, pr, ld_r, pw, pb, code, n, h, eps, *drop, py, ld_y,
          ps, ld_s, pm, pm + 4 * n if pm is not None else None)
    return y, s, (code, n, h, drop)


def _stats(x):
    return torch.empty(2 * (x.numel() // x.shape[-1] if x.numel() else 0), dtype=torch.float32,
                       device=x.device)


def layer_norm_fwd(x, weight, bias=None, residual=None, eps=1e-5, dropout=0.0, seed=None, draw=0,
                   first_row=0, return_stats=False, y_out=None, sum_out=None):
    """Layer norm of s = residual + dropped(x) (dropout_fwd's arguments; s = x
    without either), rounded to x's dtype before it is normed: (y, s, mean, rstd),
    y = (s - mean(s)) / sqrt(var(s) + eps) * weight + bias, mean and rstd [N]
    float32 (None unless asked for).  x [*lead, H] float32, bfloat16 or float16,
    weight and bias [H].  sum_out receives s and may be x or residual."""
    if not x.is_cuda:
        raise ValueError("tensors must be on a ROCm device")
    stats = _stats(x) if return_stats else None
    y, s, _ = _layer_norm_forward(x, weight, bias, residual, float(eps),
                                  _drop_args(dropout, seed, draw, first_row, x.device), stats,
                                  y_out, sum_out)
    mean, rstd = stats.view(2, -1) if return_stats else (None, None)
    return y, s, mean, rstd


def layer_norm_bwd(s, weight, mean, rstd, grad_y, grad_sum=None, dropout=0.0, seed=None, draw=0,
                   first_row=0, need_dresidual=True, need_dweight=True, need_dbias=True,
                   dx_out=None, dresidual_out=None, workspace=None):
    """(dx, dresidual, dweight, dbias) of layer_norm_fwd from its stored sum s,
    mean, rstd and the gradients of y and (where given) of s.  Without dropout
    dresidual is dx itself.  dx_out and dresidual_out may be grad_y or grad_sum,
    not one another; what is not needed is None."""
    p_s, n, h, ld_s = _norm_rows(s, "s")
    mean, rstd = _row_vector(mean, n, "mean"), _row_vector(rstd, n, "rstd")
    dev = s.device
    _same_device(dev, mean=mean, rstd=rstd)
    drop = _drop_args(dropout, seed, draw, first_row, dev)
    code = _dtype_code(s)
    pw = _norm_weight(weight, s)
    pg, _, _, ld_g = _norm_rows(grad_y, "grad_y", s)
    pd, ld_d = None, 0
    if grad_sum is not None:
        pd, _, _, ld_d = _norm_rows(grad_sum, "grad_sum", s)
    dx, px, ld_x = _norm_out(dx_out, "dx_out", s, h)
    dres, pr, ld_r = dx, None, 0
    if not need_dresidual:
        dres = None
    elif drop[0]:
        dres, pr, ld_r = _norm_out(dresidual_out, "dresidual_out", s, h)
    if dresidual_out is not None and pr is None:
        raise ValueError("dresidual_out is for a gradient through dropout that is asked for")
    dw = torch.empty_like(weight) if need_dweight else None
    db = torch.empty_like(weight) if need_dbias else None
    ws = None
    if need_dweight or need_dbias:
        ws = _workspace(workspace, _lib.lib().layer_norm_bwd_workspace_bytes(n, h), dev)
    _call("layer_norm_bwd", dev, p_s, ld_s, pw, mean.data_ptr(), rstd.data_ptr(), pg, ld_g, pd,
          ld_d, code, n, h, *drop, px, ld_x, pr, ld_r, _ptr(dw), _ptr(db), _ptr(ws), _nbytes(ws))
    return dx, dres, dw, db


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, eps, p, seed, draw, first_row):
        if not x.is_cuda:
            raise ValueError("tensors must be on a ROCm device")
        stats = _stats(x)
        drop = _drop_args(p, seed, draw, first_row, x.device)
        y, s, sizes = _layer_norm_forward(x, weight, bias, residual, eps, drop, stats, None, None)
        if drop[2] is not None:
            ctx.save_for_backward(s, weight, stats, seed)
        else:
            ctx.save_for_backward(s, weight, stats)
        ctx.sizes = (*sizes, _lib.lib().layer_norm_bwd_workspace_bytes(*sizes[1:3]))
        ctx.set_materialize_grads(False)
        return y if residual is None else (y, s)

    @staticmethod
    @_first_order
    def backward(ctx, gy, gs=None):
        s, weight, stats, *held = ctx.saved_tensors  # a seed that has changed raises
        code, n, h, drop, nbytes = ctx.sizes
        drop = _seed_again(drop, held)
        need_x, need_w, need_b, need_r = ctx.needs_input_grad[:4]
        # gradients may come in broadcast (a row for all rows, one value for all)
        gs = gs.contiguous() if gs is not None else None
        if gy is None:  # only the stored sum was used, or nothing
            dx = gs
            if drop[0] and need_x and gs is not None:
                dx = _dropout_back(gs, drop, code, n, h)
            dw = torch.zeros_like(weight) if need_w else None
            db = torch.zeros_like(weight) if need_b else None
            return dx, dw, db, gs, None, None, None, None, None
        gy = gy.contiguous()
        ld_s = h
        if s.dtype != gy.dtype or not s.is_contiguous():
            _, _, _, ld_s = _norm_rows(s, "s", gy)
        dx = dres = torch.empty_like(gy)
        pr = pw = pb = ws = None
        dw = db = None
        if drop[0] and need_r:
            dres = torch.empty_like(gy)
            pr = dres.data_ptr()
        if need_w:
            dw = torch.empty_like(weight)
            pw = dw.data_ptr()
        if need_b:
            db = torch.empty_like(weight)
            pb = db.data_ptr()
        if need_w or need_b:
            ws = torch.empty(nbytes, dtype=torch.uint8, device=gy.device)
        pm = stats.data_ptr()
        _call("layer_norm_bwd", gy.device, s.data_ptr(), ld_s, weight.data_ptr(), pm, pm + 4 * n,
              gy.data_ptr(), h, gs.data_ptr() if gs is not None else None, h, code, n, h, *drop,
              dx.data_ptr(), h, pr, h, pw, pb, ws.data_ptr() if ws is not None else None,
              nbytes)
        return dx, dw, db, dres if need_r else None, None, None, None, None, None


def layer_norm(x, weight, bias=None, residual=None, eps=1e-5, dropout=0.0, seed=None, draw=0,
               first_row=0):
    """Differentiable layer_norm_fwd: y, or (y, s) with a residual."""
    return _LayerNorm.apply(x, weight, bias, residual, float(eps), float(dropout), seed, int(draw),
                            int(first_row))


def quantize_rows_fp4(x):
    """x [N, H] (float32, bfloat16, float16; H a multiple of 32) as Fp4Rows, e.g. a
    frozen table that embedding_fwd and linear_token_logp_fwd share, made once per
    weight version.  A group's scale is the smallest power of two that brings it
    within 6, the greatest e2m1 value."""
    if x.dim() != 2:
        raise ValueError("x must be [N, H]")
    px, n, h, ld = _norm_rows(x, "x")
    code = _dtype_code(x)
    data = torch.empty(n, h // 2, dtype=torch.uint8, device=x.device)
    scale = torch.empty(n, h // 32, dtype=torch.uint8, device=x.device)
    _call("fp4_quantize", x.device, px, ld, code, n, h, data.data_ptr(), h // 2, scale.data_ptr(),
          h // 32)
    return Fp4Rows(data, scale)
