"""Token operators: several given tokens a row, entropy, the most probable
tokens, their gradients, 8-bit rows and the root-mean-square norm.

Argument marshalling only (the C ABI is include/invariant_tokens.h): PyTorch
supplies device memory and the current HIP stream; the library checks the
rest and its status becomes a LogpError.

Every function can be captured into a HIP graph.  A training step is captured
with the *_bwd functions, or through autograd while no eager autograd graph of
the same leaves is alive (torch ties a leaf's accumulation to the stream that
it was first used on, and would wait there for the capturing one).
"""

from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._lib import check
from .ops import (_DTYPES, _INDEX, _dtype_code, _linear_operands, _nbytes, _padded_logits,
                  _prepared, _prepared_buffer, _ptr, _rounding, _row_vector, _rows, _saved_stride)


class TokenLogp(NamedTuple):
    """What the token operators return (float32; lse and entropy one a row):
    logp [*lead, M] of the given tokens, lse, entropy (None unless asked for),
    top_logp and top_ids [*lead, k] of the most probable tokens (ids int64,
    -1 on padding rows)."""

    logp: torch.Tensor
    lse: torch.Tensor
    entropy: Optional[torch.Tensor]
    top_logp: torch.Tensor
    top_ids: torch.Tensor


class QuantizedRows(NamedTuple):
    """8-bit rows: data [N, H] float8_e4m3fn with contiguous rows and one
    float32 scale a row; row r stands for data[r] * scale[r]."""

    data: torch.Tensor
    scale: torch.Tensor


class Fp4Rows(NamedTuple):
    """4-bit rows: data [N, H / 2] uint8, two e2m1 values a byte (the even
    column in the low half), and scale [N, H / 32] uint8, one byte b for every 32
    columns, which stands for 2^(b - 127); both with contiguous rows."""

    data: torch.Tensor
    scale: torch.Tensor


_functions = {}  # the library's, by name


def _call(name, device, *args):
    """The library function on the device's current stream (its last
    argument), with that device current; a non-zero status raises."""
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(_lib.lib(), name)
    index = device.index
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if st:
        check(name, st)


def _first_order(backward):
    """once_differentiable, at no cost where no second derivative is asked for."""
    guarded = once_differentiable(backward)

    def run(ctx, *grads):
        return guarded(ctx, *grads) if torch.is_grad_enabled() else backward(ctx, *grads)

    return run


def _tokens(t, n, lead, device):
    """token_ids [*lead, M] (or None) -> (contiguous tensor or None, M, code)."""
    if t is None:
        return None, 0, _lib.LOGP_I64
    if t.dtype not in _INDEX:
        raise TypeError("token_ids must be int64 or int32")
    if t.device != device:
        raise ValueError("token_ids must be on the rows' device")
    if t.dim() < 1 or tuple(t.shape[:-1]) != tuple(lead):
        raise ValueError("token_ids must be [*lead, M] with the rows' leading dimensions")
    return t.contiguous(), t.shape[-1], _INDEX[t.dtype]


def _row_grad(x, n, k, name, device):
    """A gradient or saved value with k entries a row ([*lead, k], the leading
    dimensions flattened or not), as contiguous float32."""
    if x.dim() < 1 or x.shape[-1] != k or x.numel() != n * k or x.device != device:
        raise ValueError(f"{name} must be [*lead, {k}], one entry per row and token, on the rows' "
                         "device")
    return x.to(torch.float32).contiguous()


def _token_grad(grad_logp, n, m, device):
    """The given tokens' gradient, None without tokens (where one that has
    entries would be lost)."""
    if m:
        return _row_grad(grad_logp, n, m, "grad_logp", device)
    if grad_logp is not None and grad_logp.numel():
        raise ValueError("grad_logp needs the token_ids that it belongs to")
    return None


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} must be on {device}")


def _out(x, shape, dtype, device, name):
    if x is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if x.dtype != dtype or tuple(x.shape) != tuple(shape) or not x.is_contiguous() or x.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    return x


class _Outputs:
    """Output buffers of a forward, checked or allocated."""

    NAMES = ("logp_out", "lse_out", "entropy_out", "top_logp_out", "top_ids_out")

    def __init__(self, n, lead, m, k, entropy, device, given):
        for name in given:
            if name not in self.NAMES:
                raise TypeError(f"unexpected argument {name}")
        if not entropy and given.get("entropy_out") is not None:
            raise ValueError("entropy_out needs return_entropy")
        f = torch.float32
        self.logp = _out(given.get("logp_out"), (*lead, m), f, device, "logp_out")
        self.lse = _out(given.get("lse_out"), (n,), f, device, "lse_out")
        self.entropy = (_out(given.get("entropy_out"), (n,), f, device, "entropy_out")
                        if entropy else None)
        self.top_logp = _out(given.get("top_logp_out"), (*lead, k), f, device, "top_logp_out")
        self.top_ids = _out(given.get("top_ids_out"), (*lead, k), torch.int64, device, "top_ids_out")

    def pointers(self):
        return (self.logp.data_ptr(), self.lse.data_ptr(), _ptr(self.entropy),
                self.top_logp.data_ptr(), self.top_ids.data_ptr())

    def result(self):
        return TokenLogp(self.logp, self.lse, self.entropy, self.top_logp, self.top_ids)


def _workspace(given, need, device):
    if given is not None:
        if not given.is_contiguous() or given.device != device:
            raise ValueError("workspace must be a contiguous tensor on the rows' device")
        return given
    return torch.empty(need, dtype=torch.uint8, device=device) if need else None


def token_logp_fwd(logits, token_ids=None, top_k=0, ignore_index=-100, tile_width=4096,
                   return_entropy=False, workspace=None, **outputs):
    """Log-probabilities of the given tokens, row lse, entropy and the top_k
    most probable tokens of logits [*lead, V] (float32, bfloat16, float16), as
    a TokenLogp.  token_ids [*lead, M] int64 or int32, or None (M = 0): an
    entry equal to ignore_index gives 0; a row whose entries are all ignored is
    padding and is not read.  Alternatives come greatest first, the lowest
    index first among equals.  Output buffers may be passed as logp_out,
    lse_out, entropy_out, top_logp_out and top_ids_out."""
    x2, v, ld = _rows(logits)
    n, lead, dev = x2.shape[0], logits.shape[:-1], logits.device
    tok, m, tcode = _tokens(token_ids, n, lead, dev)
    code = _dtype_code(logits)
    k = int(top_k)
    if not 0 <= k <= _lib.LOGP_MAX_TOP:
        raise ValueError(f"top_k must be 0 to {_lib.LOGP_MAX_TOP}")
    out = _Outputs(n, lead, m, k, return_entropy, dev, outputs)
    L = _lib.lib()
    need = L.token_logp_fwd_workspace_bytes(n, v, code, int(tile_width), k)
    ws = _workspace(workspace, need, dev)
    _call("token_logp_fwd", dev, x2.data_ptr(), code, n, v, ld, _ptr(tok), tcode, m,
          int(ignore_index), int(tile_width), k, *out.pointers(), _ptr(ws), _nbytes(ws))
    return out.result()


def token_logp_bwd(logits, lse, token_ids=None, grad_logp=None, top_ids=None, grad_top_logp=None,
                   ignore_index=-100, entropy=None, grad_entropy=None, dlogits_out=None):
    """Gradient of the logits from those of token_logp_fwd's logp ([*lead, M]),
    top_logp ([*lead, k], with the forward's top_ids) and entropy ([N]), each
    of which may be absent; in the logits dtype and shape.  dlogits_out may be
    the logits themselves."""
    x2, v, ld = _rows(logits)
    n, lead, dev = x2.shape[0], logits.shape[:-1], logits.device
    tok, m, tcode = _tokens(token_ids, n, lead, dev)
    code = _dtype_code(logits)
    if (top_ids is None) != (grad_top_logp is None):
        raise ValueError("top_ids and grad_top_logp go together")
    if (entropy is None) != (grad_entropy is None):
        raise ValueError("entropy and grad_entropy go together")
    if m and grad_logp is None:
        raise ValueError("grad_logp is needed for the given tokens")
    g = _token_grad(grad_logp, n, m, dev)
    ids, k, gt = _alternatives(top_ids, grad_top_logp, n, dev)
    lse = _row_vector(lse, n, "lse")
    ent, gent = _row_vector(entropy, n, "entropy"), _row_vector(grad_entropy, n, "grad_entropy")
    _same_device(dev, lse=lse, entropy=ent, grad_entropy=gent)
    if dlogits_out is None:
        dlogits_out = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
    d2, v2, ld_out = _rows(dlogits_out)
    if v2 != v or d2.shape[0] != n or dlogits_out.dtype != logits.dtype or dlogits_out.device != dev:
        raise ValueError("dlogits_out must match the logits shape, dtype and device")
    _call("token_logp_bwd", dev, x2.data_ptr(), code, n, v, ld, _ptr(tok), tcode, m,
          int(ignore_index), _ptr(ids), k, lse.data_ptr(), _ptr(g), _ptr(gt), _ptr(ent),
          _ptr(gent), d2.data_ptr(), ld_out)
    return dlogits_out


def _alternatives(top_ids, grad_top_logp, n, dev):
    if top_ids is None:
        return None, 0, None
    if top_ids.dtype != torch.int64 or top_ids.device != dev or top_ids.dim() < 1:
        raise ValueError("top_ids must be the forward's int64 [*lead, k]")
    k = top_ids.shape[-1]
    if top_ids.numel() != n * k:
        raise ValueError("top_ids must have one row per logits row")
    return top_ids.contiguous(), k, _row_grad(grad_top_logp, n, k, "grad_top_logp", dev)


class _TokenLogp(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, token_ids, top_k, ignore_index, tile_width, with_entropy):
        r = token_logp_fwd(logits, token_ids, top_k, ignore_index, tile_width, with_entropy)
        ctx.save_for_backward(logits, token_ids, r.lse, r.entropy, r.top_ids)
        ctx.ignore_index = ignore_index
        ctx.mark_non_differentiable(r.lse, r.top_ids)
        ctx.set_materialize_grads(False)
        return tuple(r)

    @staticmethod
    @once_differentiable
    def backward(ctx, g, _lse, g_entropy, g_top, _ids):
        logits, token_ids, lse, entropy, top_ids = ctx.saved_tensors
        if token_ids is not None and g is None:
            g = torch.zeros(token_ids.shape, dtype=torch.float32, device=logits.device)
        with_top = g_top is not None and top_ids.shape[-1] > 0
        with_ent = g_entropy is not None
        d = token_logp_bwd(logits, lse, token_ids, g, top_ids if with_top else None,
                           g_top if with_top else None, ctx.ignore_index,
                           entropy if with_ent else None,
                           g_entropy.float().contiguous() if with_ent else None)
        return d, None, None, None, None, None


def batch_invariant_token_logp(logits, token_ids=None, top_k=0, ignore_index=-100,
                               tile_width=4096, return_entropy=False):
    """Differentiable token_logp_fwd: gradients flow through logp, top_logp
    (the log-probabilities of the tokens that were the most probable) and
    entropy into logits; lse and top_ids carry none."""
    return TokenLogp(*_TokenLogp.apply(logits, token_ids, int(top_k), int(ignore_index),
                                       int(tile_width), bool(return_entropy)))


def _q8_operand(q, name):
    if q.data.dtype != torch.float8_e4m3fn or q.data.dim() != 2 or q.data.stride(1) != 1:
        raise TypeError(f"{name}.data must be [rows, H] float8_e4m3fn with contiguous rows")
    if (q.scale.dtype != torch.float32 or q.scale.shape != q.data.shape[:1]
            or not q.scale.is_contiguous() or q.scale.device != q.data.device):
        raise TypeError(f"{name}.scale must be contiguous float32 with one entry per row")
    return q.data.shape


def _fp4_operand(q, name):
    """[rows, H] of 4-bit rows."""
    for part in q:
        if part.dtype != torch.uint8 or part.dim() != 2 or (part.stride(1) != 1 and part.shape[1] > 1):
            raise TypeError(f"{name}: Fp4Rows hold [rows, H / 2] and [rows, H / 32] uint8 with "
                            "contiguous rows")
    rows, h = q.data.shape[0], 2 * q.data.shape[1]
    if h % 32 or tuple(q.scale.shape) != (rows, h // 32):
        raise ValueError(f"{name}: Fp4Rows take H a multiple of 32 and one scale for 32 columns")
    if not q.data.is_cuda or q.scale.device != q.data.device:
        raise ValueError(f"{name} must be on one ROCm device")
    return rows, h


def _stride(t):
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def linear_token_logp_fwd(hidden, weight, token_ids=None, top_k=0, ignore_index=-100,
                          temperature=1.0, return_entropy=False, round_logits=False,
                          prepared_weight=None, logits_out=None, row_chunk=0, workspace=None,
                          **outputs):
    """token_logp_fwd through the LM head without keeping the logits: hidden
    [N, H] and weight [V, H] bfloat16, logits = hidden weight^T / temperature;
    token_ids [N, M].  hidden and weight may both be QuantizedRows: the 8-bit
    head of frozen weights (no round_logits, prepared_weight or logits_out).
    weight may be Fp4Rows: the 4-bit head of frozen weights, with the bits of the
    bfloat16 weight they stand for (no prepared_weight or logits_out).
    round_logits and prepared_weight: as linear_logp_fwd.  logits_out [N, V]
    float32 (or bfloat16 with round_logits) receives the unscaled logits for
    linear_token_logp_bwd.  row_chunk: rows taken at a time, which bounds the
    workspace (0 = the library's default); any value gives the same bits."""
    q8, fp4 = isinstance(hidden, QuantizedRows), isinstance(weight, Fp4Rows)
    if q8 != isinstance(weight, QuantizedRows):
        raise TypeError("hidden and weight must both be QuantizedRows, or neither")
    L = _lib.lib()
    k = int(top_k)
    if not 0 <= k <= _lib.LOGP_MAX_TOP:
        raise ValueError(f"top_k must be 0 to {_lib.LOGP_MAX_TOP}")
    z = logits_out
    if q8:
        if round_logits or prepared_weight is not None or z is not None:
            raise ValueError("the 8-bit head takes no round_logits, prepared_weight or logits_out")
        n, h = _q8_operand(hidden, "hidden")
        v, h2 = _q8_operand(weight, "weight")
        if h2 != h:
            raise ValueError("hidden and weight must share H")
        if not hidden.data.is_cuda or weight.data.device != hidden.data.device:
            raise ValueError("hidden and weight must be on one ROCm device")
        ld_h = hidden.data.stride(0) if n > 1 else h
        ld_w = weight.data.stride(0) if v > 1 else h
        dev, pw = hidden.data.device, None
        flags = _lib.LOGP_TOKEN_Q8
    elif fp4:
        if prepared_weight is not None or z is not None:
            raise ValueError("the 4-bit head takes no prepared_weight or logits_out")
        if hidden.dtype != torch.bfloat16 or hidden.dim() != 2 or hidden.stride(1) != 1:
            raise TypeError("hidden must be [N, H] bfloat16 with contiguous rows")
        v, h = _fp4_operand(weight, "weight")
        n, dev, pw = hidden.shape[0], hidden.device, None
        if hidden.shape[1] != h:
            raise ValueError("hidden and weight must share H")
        if weight.data.device != dev:
            raise ValueError("hidden and weight must be on one ROCm device")
        ld_h = hidden.stride(0) if n > 1 else h
        flags = _lib.LOGP_TOKEN_FP4 | (_lib.LOGP_TOKEN_ROUND_BF16 if round_logits else 0)
    else:
        n, h, v, ld_h, ld_w = _linear_operands(hidden, weight)
        dev = hidden.device
        if not hidden.is_cuda or weight.device != dev:
            raise ValueError("hidden and weight must be on one ROCm device")
        pw = _prepared(_prepared_buffer(prepared_weight, weight), L, v, h, dev)
        if z is not None and (z.dim() != 2 or tuple(z.shape) != (n, v) or z.stride(1) != 1
                              or z.device != dev):
            raise ValueError("logits_out must be [N, V] with contiguous rows")
        if z is not None and z.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("logits_out must be float32, or bfloat16 with round_logits")
        flags = ((_lib.LOGP_TOKEN_KEEPS_LOGITS if z is not None else 0)
                 | (_lib.LOGP_TOKEN_ROUND_BF16 if round_logits else 0))
    tok, m, tcode = _tokens(token_ids, n, (n,), dev)
    out = _Outputs(n, (n,), m, k, return_entropy, dev, outputs)
    need = L.linear_token_logp_fwd_workspace_bytes(n, h, v, m, k, flags, int(row_chunk))
    ws = _workspace(workspace, need, dev)
    if q8:
        _call("linear_token_logp_q8_fwd", dev, hidden.data.data_ptr(), ld_h,
              hidden.scale.data_ptr(), weight.data.data_ptr(), ld_w, weight.scale.data_ptr(), n, h,
              v, _ptr(tok), tcode, m, int(ignore_index), float(temperature), k, *out.pointers(),
              int(row_chunk), _ptr(ws), _nbytes(ws))
    elif fp4:
        _call("linear_token_logp_fp4_fwd", dev, hidden.data_ptr(), ld_h, weight.data.data_ptr(),
              _stride(weight.data), weight.scale.data_ptr(), _stride(weight.scale), n, h, v,
              _ptr(tok), tcode, m, int(ignore_index), float(temperature), _rounding(round_logits), k,
              *out.pointers(), int(row_chunk), _ptr(ws), _nbytes(ws))
    else:
        _call("linear_token_logp_fwd", dev, hidden.data_ptr(), ld_h, weight.data_ptr(), ld_w, n, h,
              v, _ptr(tok), tcode, m, int(ignore_index), float(temperature),
              _rounding(round_logits), k, *out.pointers(), _ptr(z),
              _DTYPES[z.dtype] if z is not None else 0,
              (z.stride(0) if n > 1 else v) if z is not None else 0, _ptr(pw), _nbytes(pw),
              int(row_chunk), _ptr(ws), _nbytes(ws))
    return out.result()


def linear_token_logp_bwd(hidden, weight, lse, token_ids=None, logp=None, grad_logp=None,
                          top_ids=None, top_logp=None, grad_top_logp=None, ignore_index=-100,
                          temperature=1.0, entropy=None, grad_entropy=None, round_logits=False,
                          saved_logits=None, prepared_weight=None, need_dhidden=True,
                          need_dweight=True, out_dtype=torch.float32, vocab_chunk=0,
                          workspace=None, dhidden_out=None, dweight_out=None):
    """Backward of linear_token_logp_fwd: (dhidden [N, H] or None, dweight
    [V, H] or None) in out_dtype, from the forward's lse, logp, top_ids,
    top_logp and entropy and the upstream gradients (top_ids and entropy only
    where gradients come in for them).  dhidden is summed in segments of the
    vocabulary; vocab_chunk is rounded up to whole ones.  The rest: as
    linear_logp_bwd."""
    n, h, v, ld_h, ld_w = _linear_operands(hidden, weight)
    dev = hidden.device
    if not hidden.is_cuda or weight.device != dev:
        raise ValueError("hidden and weight must be on one ROCm device")
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out_dtype must be float32 or bfloat16")
    L = _lib.lib()
    pw = _prepared(_prepared_buffer(prepared_weight, weight), L, v, h, dev)
    tok, m, tcode = _tokens(token_ids, n, (n,), dev)
    if m and (logp is None or grad_logp is None):
        raise ValueError("logp and grad_logp are needed for the given tokens")
    if len({top_ids is None, top_logp is None, grad_top_logp is None}) != 1:
        raise ValueError("top_ids, top_logp and grad_top_logp go together")
    if (entropy is None) != (grad_entropy is None):
        raise ValueError("entropy and grad_entropy go together")
    lp = _row_grad(logp, n, m, "logp", dev) if m else None
    g = _token_grad(grad_logp, n, m, dev)
    ids, k, gt = _alternatives(top_ids, grad_top_logp, n, dev)
    tl = _row_grad(top_logp, n, k, "top_logp", dev) if ids is not None else None
    lse = _row_vector(lse, n, "lse")
    ent, gent = _row_vector(entropy, n, "entropy"), _row_vector(grad_entropy, n, "grad_entropy")
    _same_device(dev, lse=lse, entropy=ent, grad_entropy=gent)
    z = saved_logits
    if z is not None and (z.dim() != 2 or tuple(z.shape) != (n, v) or z.stride(1) != 1
                          or z.dtype not in (torch.float32, torch.bfloat16) or z.device != dev):
        raise ValueError("saved_logits must be [N, V] float32 / bfloat16 with contiguous rows")
    outs = []
    for o, rows, need in ((dhidden_out, n, need_dhidden), (dweight_out, v, need_dweight)):
        if not need:
            outs.append(None)
            continue
        if o is None:
            o = torch.empty(rows, h, dtype=out_dtype, device=dev)
        if (o.dtype != out_dtype or tuple(o.shape) != (rows, h) or o.stride(1) != 1
                or o.device != dev):
            raise ValueError("output buffers must be [rows, H] of out_dtype, rows contiguous")
        outs.append(o)
    dh, dw = outs
    flags = ((_lib.LOGP_BWD_DHIDDEN if dh is not None else 0)
             | (_lib.LOGP_BWD_DWEIGHT if dw is not None else 0)
             | (_lib.LOGP_BWD_PREPARED if pw is not None else 0)
             | (_lib.LOGP_BWD_SAVED_LOGITS if z is not None else 0)
             | (_lib.LOGP_BWD_BF16_OUT if out_dtype == torch.bfloat16 else 0))
    need = L.linear_token_logp_bwd_workspace_bytes(n, h, v, flags, int(vocab_chunk))
    ws = _workspace(workspace, need, dev)
    _call("linear_token_logp_bwd", dev, hidden.data_ptr(), ld_h, weight.data_ptr(), ld_w, n, h, v,
          _ptr(tok), tcode, m, int(ignore_index), _ptr(ids), k, float(temperature),
          _rounding(round_logits), _ptr(z), _DTYPES[z.dtype] if z is not None else 0,
          _saved_stride(z, n, v) if z is not None else 0, _ptr(pw), _nbytes(pw), lse.data_ptr(),
          _ptr(lp), _ptr(tl), _ptr(g), _ptr(gt), _ptr(ent), _ptr(gent), _DTYPES[out_dtype], _ptr(dh),
          (dh.stride(0) if n > 1 else h) if dh is not None else 0, _ptr(dw),
          (dw.stride(0) if v > 1 else h) if dw is not None else 0, int(vocab_chunk), _ptr(ws),
          _nbytes(ws))
    return dh, dw


class _LinearTokenLogp(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, token_ids, top_k, ignore_index, temperature, with_entropy,
                round_logits, save_logits, prepared_weight):
        z = None
        if save_logits:
            z = _padded_logits(hidden.shape[0], weight.shape[0],
                               torch.bfloat16 if round_logits else torch.float32, hidden.device)
        r = linear_token_logp_fwd(hidden, weight, token_ids, top_k, ignore_index, temperature,
                                  with_entropy, round_logits, prepared_weight, z)
        ctx.save_for_backward(hidden, weight, token_ids, z, *r)
        ctx.options = (ignore_index, temperature, round_logits, prepared_weight)
        ctx.mark_non_differentiable(r.lse, r.top_ids)
        ctx.set_materialize_grads(False)
        return tuple(r)

    @staticmethod
    @once_differentiable
    def backward(ctx, g, _lse, g_entropy, g_top, _ids):
        hidden, weight, token_ids, z, logp, lse, entropy, top_logp, top_ids = ctx.saved_tensors
        ignore_index, temperature, round_logits, prepared = ctx.options
        if prepared is not None:
            prepared.check(weight)
        if token_ids is not None and g is None:
            g = torch.zeros(token_ids.shape, dtype=torch.float32, device=hidden.device)
        with_top = g_top is not None and top_ids.shape[-1] > 0
        with_ent = g_entropy is not None
        dh, dw = linear_token_logp_bwd(
            hidden, weight, lse, token_ids, logp, g, top_ids if with_top else None,
            top_logp if with_top else None, g_top if with_top else None, ignore_index, temperature,
            entropy if with_ent else None, g_entropy.float().contiguous() if with_ent else None,
            round_logits, z, prepared, ctx.needs_input_grad[0], ctx.needs_input_grad[1],
            torch.bfloat16)
        return dh, dw, None, None, None, None, None, None, None, None


def linear_token_logp(hidden, weight, token_ids=None, top_k=0, ignore_index=-100, temperature=1.0,
                      return_entropy=False, round_logits=False, save_logits=False,
                      prepared_weight=None):
    """Differentiable linear_token_logp_fwd for bfloat16 hidden [N, H] and
    weight [V, H]: gradients (bfloat16) flow through logp, top_logp and
    entropy.  save_logits keeps the logits from forward to backward ([N, V]
    float32, bfloat16 with round_logits), which then computes one product less;
    the same bits.  prepared_weight: as linear_logp."""
    if isinstance(weight, (QuantizedRows, Fp4Rows)):
        raise TypeError("8-bit and 4-bit rows have no gradient: linear_token_logp_fwd scores them")
    return TokenLogp(*_LinearTokenLogp.apply(hidden, weight, token_ids, int(top_k),
                                             int(ignore_index), float(temperature),
                                             bool(return_entropy), bool(round_logits),
                                             bool(save_logits), prepared_weight))


def _norm_rows(x, name, like=None):
    """[*lead, H] -> (pointer, n, h, row stride); leading dimensions must
    flatten without a copy."""
    if not x.is_cuda:
        raise ValueError("tensors must be on a ROCm device")
    shape = x.shape
    if like is not None and (shape != like.shape or x.dtype != like.dtype
                             or x.get_device() != like.get_device()):
        raise ValueError(f"{name} must match x in shape, dtype and device")
    dim = len(shape)
    if dim and x.is_contiguous():
        h = shape[-1]
        return x.data_ptr(), x.numel() // h if h else 0, h, h
    if dim < 1 or x.stride(-1) != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    h = shape[-1]
    x2 = x if dim == 2 else x.view(-1, h)
    return x2.data_ptr(), x2.shape[0], h, x2.stride(0) if x2.shape[0] > 1 else h


def _norm_out(given, name, like, h):
    """An output like `like`: (tensor, pointer, row stride)."""
    if given is None:
        o = (torch.empty_like(like) if like.is_contiguous()
             else torch.empty(like.shape, dtype=like.dtype, device=like.device))
        return o, o.data_ptr(), h
    p, _, _, ld = _norm_rows(given, name, like)
    return given, p, ld


def _norm_weight(weight, x, name="weight"):
    if (weight.dim() != 1 or weight.shape[0] != x.shape[-1] or weight.dtype != x.dtype
            or weight.get_device() != x.get_device() or not weight.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous [H] of x's dtype and device")
    return weight.data_ptr()


def rms_norm_fwd(x, weight, residual=None, eps=1e-6, return_rstd=False, y_out=None, sum_out=None):
    """Root-mean-square norm of s = x + residual (rounded to x's dtype, then
    normed; s = x without a residual): (y, s, rstd), y = s / sqrt(mean(s^2) +
    eps) * weight, rstd [N] float32 (None unless asked for).  x [*lead, H]
    float32, bfloat16 or float16, weight [H].  sum_out receives s (a copy of x
    without a residual) and may be x or residual (in place)."""
    px, n, h, ld_x = _norm_rows(x, "x")
    code = _dtype_code(x)
    pw = _norm_weight(weight, x)
    dev = x.device
    y, py, ld_y = _norm_out(y_out, "y_out", x, h)
    pr, ld_r, ps, ld_s, s = None, 0, None, 0, x
    if residual is not None:
        pr, _, _, ld_r = _norm_rows(residual, "residual", x)
    if residual is not None or sum_out is not None:
        s, ps, ld_s = _norm_out(sum_out, "sum_out", x, h)
    rstd = torch.empty(n, dtype=torch.float32, device=dev) if return_rstd else None
    _call("rms_norm_fwd", dev, px, ld_x, pr, ld_r, pw, code, n, h, float(eps), py, ld_y, ps, ld_s,
          _ptr(rstd))
    return y, s, rstd


def rms_norm_bwd(s, weight, rstd, grad_y, grad_sum=None, need_dweight=True, dx_out=None,
                 workspace=None):
    """(dx, dweight or None) of rms_norm_fwd from its stored sum s, rstd and
    the gradients of y and (where given) of s; dx is the gradient of x and of
    the residual.  dx_out may be grad_y or grad_sum."""
    p_s, n, h, ld_s = _norm_rows(s, "s")
    code = _dtype_code(s)
    pw = _norm_weight(weight, s)
    pg, _, _, ld_g = _norm_rows(grad_y, "grad_y", s)
    pd, ld_d = None, 0
    if grad_sum is not None:
        pd, _, _, ld_d = _norm_rows(grad_sum, "grad_sum", s)
    rstd = _row_vector(rstd, n, "rstd")
    _same_device(s.device, rstd=rstd)
    dev = s.device
    dx, px, ld_x = _norm_out(dx_out, "dx_out", s, h)
    dw = torch.empty(h, dtype=s.dtype, device=dev) if need_dweight else None
    L = _lib.lib()
    ws = _workspace(workspace, L.rms_norm_bwd_workspace_bytes(n, h), dev) if need_dweight else None
    _call("rms_norm_bwd", dev, p_s, ld_s, pw, rstd.data_ptr(), pg, ld_g, pd, ld_d, code, n, h, px,
          ld_x, _ptr(dw), _ptr(ws), _nbytes(ws))
    return dx, dw


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, s, rstd = rms_norm_fwd(x, weight, residual, eps, return_rstd=True)
        ctx.save_for_backward(s, weight, rstd)
        ctx.fused = residual is not None
        ctx.set_materialize_grads(False)
        return (y, s) if ctx.fused else y

    @staticmethod
    @once_differentiable
    def backward(ctx, gy, gs=None):
        s, weight, rstd = ctx.saved_tensors
        need_w = ctx.needs_input_grad[1]
        if gy is None:  # only the stored sum was used
            return gs, torch.zeros_like(weight) if need_w else None, gs if ctx.fused else None, None
        # gradients may come in broadcast (a row for all rows, one value for all)
        gs = gs.contiguous() if gs is not None else None
        dx, dw = rms_norm_bwd(s, weight, rstd, gy.contiguous(), gs, need_dweight=need_w)
        return dx, dw, dx if ctx.fused else None, None


def rms_norm(x, weight, residual=None, eps=1e-6):
    """Differentiable rms_norm_fwd: y, or (y, x + residual) with a residual."""
    return _RmsNorm.apply(x, weight, residual, float(eps))


def _quantize(x, weight, residual, eps, sum_out):
    px, n, h, ld_x = _norm_rows(x, "x")
    code = _dtype_code(x)
    pw = _norm_weight(weight, x) if weight is not None else None
    dev = x.device
    pr, ld_r, ps, ld_s, s = None, 0, None, 0, x
    if residual is not None:
        pr, _, _, ld_r = _norm_rows(residual, "residual", x)
    if residual is not None or sum_out is not None:
        s, ps, ld_s = _norm_out(sum_out, "sum_out", x, h)
    q = torch.empty(n, h, dtype=torch.float8_e4m3fn, device=dev)
    scale = torch.empty(n, dtype=torch.float32, device=dev)
    _call("rms_norm_q8_fwd", dev, px, ld_x, pr, ld_r, pw, code, n, h, float(eps), q.data_ptr(), h,
          scale.data_ptr(), ps, ld_s)
    return QuantizedRows(q, scale), s


def rms_norm_quantized(x, weight, residual=None, eps=1e-6, sum_out=None):
    """rms_norm_fwd with 8-bit rows as output: (QuantizedRows [N, H], s).  A
    row's scale is its greatest magnitude / 448, at least 2^-126 (0 for a row
    of zeros); the norm's fp32 result is rounded once, to 8 bits."""
    return _quantize(x, weight, residual, eps, sum_out)


def quantize_rows(x):
    """x [N, H] (float32, bfloat16, float16) as QuantizedRows, e.g. a frozen
    LM-head weight, made once per weight version."""
    return _quantize(x, None, None, 0.0, None)[0]


def norm_linear_token_logp(x, norm_weight, weight, token_ids=None, residual=None, eps=1e-6,
                           top_k=0, ignore_index=-100, temperature=1.0, return_entropy=False,
                           round_logits=False, save_logits=False, prepared_weight=None):
    """The tail of a decoder, from the last layer's output to the tokens'
    log-probabilities: rms_norm(x + residual) through the LM head, as a
    TokenLogp.  x [N, H] bfloat16.  With a bfloat16 weight [V, H] it is
    differentiable in x, residual, norm_weight and weight (rms_norm, then
    linear_token_logp); with a QuantizedRows weight the normed rows are
    quantised in the norm and the 8-bit head scores them, with Fp4Rows the 4-bit
    head scores them as they are (no gradient through either).  The gradient of
    norm_weight sums over all rows, padding rows (whose part is 0) included: they
    must be finite for it."""
    if isinstance(weight, (QuantizedRows, Fp4Rows)):
        fp4 = isinstance(weight, Fp4Rows)
        bits = 4 if fp4 else 8
        if fp4 and (save_logits or prepared_weight is not None):
            raise ValueError("the 4-bit head takes no save_logits or prepared_weight")
        if not fp4 and (round_logits or save_logits or prepared_weight is not None):
            raise ValueError("the 8-bit head takes no round_logits, save_logits or prepared_weight")
        if torch.is_grad_enabled() and any(t is not None and t.requires_grad
                                           for t in (x, norm_weight, residual)):
            raise ValueError(f"the {bits}-bit head has no gradient: call it under torch.no_grad()")
        if fp4:
            y, _, _ = rms_norm_fwd(x, norm_weight, residual, eps)
            return linear_token_logp_fwd(y, weight, token_ids, top_k, ignore_index, temperature,
                                         return_entropy, round_logits)
        hidden, _ = rms_norm_quantized(x, norm_weight, residual, eps)
        return linear_token_logp_fwd(hidden, weight, token_ids, top_k, ignore_index, temperature,
                                     return_entropy)
    y = rms_norm(x, norm_weight, residual, eps)
    if residual is not None:
        y = y[0]
    return linear_token_logp(y, weight, token_ids, top_k, ignore_index, temperature, return_entropy,
                             round_logits, save_logits, prepared_weight)
