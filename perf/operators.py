"""The cases on which the token operators are measured, and their plain forms.

Operators (N rows, V vocabulary columns, H hidden columns, M given tokens and k alternatives a row):

  token         log-probabilities of M given tokens, row log-sum-exp, entropy and the k most probable tokens
                of a [N, V] matrix of logits; token_train adds the gradient of the logits
  linear        the same through the language-model head, logits = hidden @ weight.T / T; linear_train adds the
                gradients of hidden and weight
  norm          root-mean-square norm of x + residual; norm_train adds the gradients of x, residual and weight;
                norm_q8 gives the normed rows in 8 bits (e4m3) with one scale a row
  linear_q8     the language-model head on 8-bit hidden and weight rows with their scales

run() computes the plain form in 32 bits where `own` is false, and makes the framework's calls where it is true.
"""

import math

import torch

own = False

IGNORE = -100  # a token entry to leave out; a row whose entries are all left out is padding
EPS = 1e-6
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}
E4M3_MAX = 448.0


def listed():
    return [
        # one sequence's next token: its log-probability and 5 alternatives (latency)
        dict(name="token-decode-1", op="token", n=1, v=151936, m=1, k=5, dtype="bf16", entropy=False),
        # a batch of rollouts scored with 20 alternatives and the entropy, 5% padding rows
        dict(name="token-score-4096", op="token", n=4096, v=151936, m=1, k=20, dtype="bf16", entropy=True),
        # fp32 logits of an odd vocabulary (rows not 16-byte aligned), the longest list of alternatives
        dict(name="token-odd-fp32", op="token", n=509, v=50257, m=4, k=64, dtype="fp32", entropy=False),
        # distillation on a teacher's 16 tokens a position, with an entropy bonus
        dict(name="token-train-4096", op="token_train", n=4096, v=128256, m=16, k=0, dtype="bf16", entropy=True),
        # decoding 16 sequences from their hidden rows, 20 alternatives each
        dict(name="linear-decode-16", op="linear", n=16, h=4096, v=151936, m=1, k=20, temperature=0.7, entropy=False),
        # scoring 4096 positions from their hidden rows, 20 alternatives each
        dict(name="linear-score-4096", op="linear", n=4096, h=4096, v=151936, m=1, k=20, temperature=1.0, entropy=True),
        # distillation through the head on a teacher's 8 tokens a position
        dict(name="linear-train-2048", op="linear_train", n=2048, h=4096, v=151936, m=8, k=0, temperature=1.0, entropy=False),
        # the last norm while decoding 16 sequences (latency)
        dict(name="norm-decode-16", op="norm", n=16, h=4096, dtype="bf16"),
        # the last norm of a training step, forward and backward
        dict(name="norm-train-8192", op="norm_train", n=8192, h=4096, dtype="bf16"),
        # the last norm before an 8-bit head, a ragged number of rows
        dict(name="norm-q8-4095", op="norm_q8", n=4095, h=5120, dtype="bf16"),
        # decoding 32 sequences through an 8-bit head (the weight's bytes count)
        dict(name="linear-q8-decode-32", op="linear_q8", n=32, h=4096, v=151936, m=1, k=0, temperature=1.0, entropy=False),
        # scoring 4096 positions with an 8-bit reference model's head
        dict(name="linear-q8-score-4096", op="linear_q8", n=4096, h=4096, v=151936, m=1, k=0, temperature=1.0, entropy=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["token", "token_train", "linear", "linear_train", "norm", "norm_train", "norm_q8", "linear_q8"])
    if op.startswith("norm"):
        return dict(op=op, n=_log_int(rng, 1, 8192), h=8 * _log_int(rng, 16, 1024) - rng.choice([0, 0, 0, 3]),
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    m, k = rng.choice([1, 1, 2, 5, 16, 32]), rng.choice([0, 1, 5, 20, 64])
    v = _log_int(rng, 1000, 151936)
    case = dict(op=op, n=_log_int(rng, 1, 2048), v=v, m=m, k=k, entropy=rng.random() < 0.5)
    if op.startswith("token"):
        case["dtype"] = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    else:
        case["h"] = 64 * _log_int(rng, 4, 64)
        case["temperature"] = rng.choice([1.0, 1.0, 0.7, 1.3])
    if op == "linear_q8":
        case["k"] = 0
    return case


def _grid(shape, step, std, gen):
    """Normal values on a grid of `step`, at most 127 steps, as weights and activations of an 8-bit model in bf16 are: sums of their products are exact in 32 bits,
    so which of two tokens is the more probable does not hang on the order of a sum."""
    x = torch.randn(shape, generator=gen, device=gen.device)
    return x.mul_(std / step).round_().clamp_(-127, 127).mul_(step).to(torch.bfloat16)


def _quantized(x):
    scale = x.abs().amax(1) / E4M3_MAX
    return (x / scale[:, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    s = dict(case=case)
    n, op = case["n"], case["op"]
    if op.startswith("norm"):
        h, t = case["h"], TYPES[case["dtype"]]
        s["x"] = randn(n, h).to(t)
        s["residual"] = (3 * randn(n, h)).to(t)
        s["weight"] = (1 + 0.1 * randn(h)).to(t)
        if op == "norm_train":
            s["dy"] = randn(n, h).to(t)
            s["dsum"] = randn(n, h).to(t)
            for k in ("x", "residual", "weight"):
                s[k].requires_grad_()
        return s
    v, m = case["v"], case["m"]
    # given tokens: any that is not masked below; one entry in 20 is left out, and with it one row in 20 for m = 1
    tokens = torch.randint(0, v - v // 64, (n, m), generator=gen, device=dev)
    drop = torch.rand(n, m, generator=gen, device=dev) < 0.05
    drop[0, 0] = False
    s["tokens"] = tokens.masked_fill_(drop, IGNORE)
    if op.startswith("token"):
        s["logits"] = (3 * randn(n, v)).to(TYPES[case["dtype"]])
        s["logits"][:, v - v // 64:] = -math.inf  # the vocabulary's padding columns are masked
    elif op == "linear_q8":
        s["hidden"], s["hidden_scale"] = _quantized(randn(n, case["h"]))
        s["weight"], s["weight_scale"] = _quantized(randn(v, case["h"]).mul_(0.02))
    else:
        s["hidden"] = _grid((n, case["h"]), 1 / 16, 1.0, gen)
        s["weight"] = _grid((v, case["h"]), 1 / 1024, 0.02, gen)
    if op.endswith("train"):
        s["g"] = randn(n, m)
        if case["k"]:
            s["g_top"] = randn(n, case["k"])
        if case["entropy"]:
            s["g_entropy"] = 0.01 * randn(n)
        for k in ("logits", "hidden", "weight"):
            if k in s:
                s[k].requires_grad_()
    return s


# ---- the plain forms -----------------------------------------------------------------------------------------


def _top(x, k):
    """The k largest of each row, the lowest index first among equals: one whole number a value that orders by (value, -index)."""
    bits = (x + 0.0).view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).to(torch.int64) << 32
    key += torch.arange(x.shape[1] - 1, -1, -1, device=x.device)
    return x.shape[1] - 1 - (key.topk(k, dim=1).values & 0xFFFFFFFF)


def _scores(x, tokens, case):
    """The outputs of the token operators on 32-bit logits x, and what their gradient needs."""
    active = (tokens != IGNORE).any(1)
    given = tokens != IGNORE
    top = x.amax(1)
    d = x - top[:, None]
    e = d.exp()
    total = e.sum(1)
    lse = top + total.log()
    out = {"logp": torch.where(given, x.gather(1, tokens.clamp(min=0)) - lse[:, None], 0.0),
           "lse": torch.where(active, lse, 0.0)}
    if case["entropy"]:
        moment = (e * torch.where(e > 0, d, 0.0)).sum(1)
        out["entropy"] = torch.where(active, total.log() - moment / total, 0.0)
    if case["k"]:
        ids = _top(x, case["k"])
        out["top_logp"] = torch.where(active[:, None], x.gather(1, ids) - lse[:, None], 0.0)
        out["top_ids"] = torch.where(active[:, None], ids, -1)
    return out, lse, active


def _dscores(x, out, lse, active, s):
    """The gradient of 32-bit logits x."""
    case, tokens = s["case"], s["tokens"]
    g = s["g"] * (tokens != IGNORE)
    whole = g.sum(1)
    logp = x - lse[:, None]
    p = logp.exp() * active[:, None]
    if case["k"]:
        g_top = s["g_top"] * active[:, None]
        whole = whole + g_top.sum(1)
    d = p * -whole[:, None]
    if case["entropy"]:
        d -= p * torch.where(p > 0, logp + out["entropy"][:, None], 0.0) * s["g_entropy"][:, None]
    d.scatter_add_(1, tokens.clamp(min=0), g)
    if case["k"]:
        d.scatter_add_(1, out["top_ids"].clamp(min=0), g_top)
    return d


def _norm(s):
    t = s["x"].dtype
    total = (s["x"].float() + s["residual"].float()).to(t)  # the residual stream is stored in its type, and its stored rows are normed
    f = total.float()
    scale = (f.square().mean(1, keepdim=True) + EPS).rsqrt()
    return total, f, scale


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op.startswith("norm"):
        total, f, scale = _norm(s)
        w = s["weight"].float()
        y = f * scale * w
        if op == "norm":
            return {"y": y.to(total.dtype), "sum": total}
        if op == "norm_q8":
            most = y.abs().amax(1, keepdim=True)
            return {"q": (y * (E4M3_MAX / most)).to(torch.float8_e4m3fn), "scale": (most / E4M3_MAX)[:, 0], "sum": total}
        dy = s["dy"].float()
        unit, dunit = f * scale, dy * w
        dx = s["dsum"].float() + scale * (dunit - unit * (dunit * unit).mean(1, keepdim=True))
        return {"y": y.to(total.dtype), "sum": total, "dx": dx.to(total.dtype), "dresidual": dx.to(total.dtype),
                "dweight": (dy * unit).sum(0).to(total.dtype)}
    if op.startswith("token"):
        x = s["logits"].float()
        out, lse, active = _scores(x, s["tokens"], case)
        if op == "token_train":
            out["dlogits"] = _dscores(x, out, lse, active, s).to(s["logits"].dtype)
        return out
    hidden, weight = s["hidden"].float(), s["weight"].float()
    x = hidden @ weight.T
    if op == "linear_q8":
        x = x * s["hidden_scale"][:, None] * s["weight_scale"]
    if case["temperature"] != 1.0:
        x = x * (1.0 / case["temperature"])
    out, lse, active = _scores(x, s["tokens"], case)
    if op == "linear_train":
        dz = _dscores(x, out, lse, active, s) * (1.0 / case["temperature"])
        out["dhidden"] = (dz @ weight).to(torch.bfloat16)
        out["dweight"] = (dz.T @ hidden).to(torch.bfloat16)
    return out


# ---- the framework's calls -----------------------------------------------------------------------------------


def _named(r, case):
    out = {"logp": r.logp, "lse": r.lse}
    if case["entropy"]:
        out["entropy"] = r.entropy
    if case["k"]:
        out["top_logp"], out["top_ids"] = r.top_logp, r.top_ids
    return out


def _grads(r, s, inputs):
    outs, grads = [r.logp], [s["g"]]
    if s["case"]["k"]:
        outs.append(r.top_logp)
        grads.append(s["g_top"])
    if s["case"]["entropy"]:
        outs.append(r.entropy)
        grads.append(s["g_entropy"])
    return torch.autograd.grad(outs, inputs, grads)


def _ours(s):
    import invariant_token_log_amd as itl

    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        y, total, _ = itl.rms_norm_fwd(s["x"], s["weight"], residual=s["residual"], eps=EPS)
        return {"y": y, "sum": total}
    if op == "norm_q8":
        q, total = itl.rms_norm_quantized(s["x"], s["weight"], residual=s["residual"], eps=EPS)
        return {"q": q.data, "scale": q.scale, "sum": total}
    if op == "norm_train":
        y, total = itl.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS)
        dx, dresidual, dweight = torch.autograd.grad([y, total], [s["x"], s["residual"], s["weight"]], [s["dy"], s["dsum"]])
        return {"y": y, "sum": total, "dx": dx, "dresidual": dresidual, "dweight": dweight}
    if op == "token":
        return _named(itl.token_logp_fwd(s["logits"], s["tokens"], top_k=case["k"], ignore_index=IGNORE,
                                         return_entropy=case["entropy"]), case)
    if op == "token_train":
        r = itl.batch_invariant_token_logp(s["logits"], s["tokens"], top_k=case["k"], ignore_index=IGNORE,
                                           return_entropy=case["entropy"])
        return {**_named(r, case), "dlogits": _grads(r, s, [s["logits"]])[0]}
    if op == "linear_train":
        r = itl.linear_token_logp(s["hidden"], s["weight"], s["tokens"], top_k=case["k"], ignore_index=IGNORE,
                                  temperature=case["temperature"], return_entropy=case["entropy"],
                                  save_logits=True)  # 1.2 GB of 288 until the backward, which then computes one product less
        dhidden, dweight = _grads(r, s, [s["hidden"], s["weight"]])
        return {**_named(r, case), "dhidden": dhidden, "dweight": dweight}
    hidden, weight = s["hidden"], s["weight"]
    if op == "linear_q8":
        hidden, weight = itl.QuantizedRows(hidden, s["hidden_scale"]), itl.QuantizedRows(weight, s["weight_scale"])
    return _named(itl.linear_token_logp_fwd(hidden, weight, s["tokens"], top_k=case["k"], ignore_index=IGNORE,
                                            temperature=case["temperature"], return_entropy=case["entropy"]), case)


def run(state):
    if own:
        return _ours(state)
    with torch.no_grad():
        return _plain(state)


# ---- what a pass cannot do without ---------------------------------------------------------------------------


def work(case):
    n, op = case["n"], case["op"]
    if op.startswith("norm"):
        h, size = case["h"], SIZE[case["dtype"]]
        cells = n * h
        if op == "norm":
            return {"bytes": 4 * cells * size + h * size, "flops": 5 * cells}
        if op == "norm_q8":
            return {"bytes": 3 * cells * size + cells + 4 * n + h * size, "flops": 7 * cells}
        return {"bytes": 8 * cells * size + 2 * h * size, "flops": 15 * cells}
    v, small = case["v"], n * (12 * case["m"] + 12 * case["k"] + 8)
    if op == "token":
        return {"bytes": n * v * SIZE[case["dtype"]] + small, "flops": 4 * n * v}
    if op == "token_train":
        return {"bytes": 2 * n * v * SIZE[case["dtype"]] + 2 * small, "flops": 8 * n * v}
    size = 1 if op == "linear_q8" else 2
    times = 3 if op == "linear_train" else 1
    moved = (2 if op == "linear_train" else 1) * size * (n + v) * case["h"]
    return {"bytes": moved + small, "flops": times * 2 * n * v * case["h"]}


# ---- the definition, in 64 bits ------------------------------------------------------------------------------


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    wide = {k: v.detach().double() for k, v in s.items() if torch.is_tensor(v) and v.dtype != torch.int64}
    with torch.enable_grad():
        if op.startswith("norm"):
            stored = (wide["x"] + wide["residual"]).to(TYPES[case["dtype"]])
            a, w = stored.double().requires_grad_(), wide["weight"].requires_grad_()
            y = a / torch.sqrt(torch.mean(a * a, -1, keepdim=True) + EPS) * w
            if op == "norm":
                return {"y": y.detach(), "sum": wide["x"] + wide["residual"]}
            if op == "norm_q8":
                scale = y.detach().abs().amax(-1) / E4M3_MAX
                return {"q": y.detach() / scale[:, None], "scale": scale, "sum": wide["x"] + wide["residual"]}
            da, dw = torch.autograd.grad([y, a * 1.0], [a, w], [wide["dy"], wide["dsum"]])
            return {"y": y.detach(), "sum": wide["x"] + wide["residual"], "dx": da, "dresidual": da, "dweight": dw}
        if op.startswith("token"):
            leaves = [wide["logits"].requires_grad_()]
            x = leaves[0]
        else:
            leaves = [wide["hidden"].requires_grad_(), wide["weight"].requires_grad_()]
            x = torch.mm(leaves[0], leaves[1].t())
            if op == "linear_q8":
                x = x * wide["hidden_scale"][:, None] * wide["weight_scale"][None, :]
            x = x / case["temperature"]
        if not op.endswith("train"):
            x = x.detach()
        keep = s["tokens"].ne(IGNORE)
        row = keep.any(-1)
        logp = torch.log_softmax(x, -1)
        out = {"logp": logp.gather(-1, s["tokens"].masked_fill(~keep, 0)).masked_fill(~keep, 0),
               "lse": torch.logsumexp(x, -1).masked_fill(~row, 0)}
        if case["entropy"]:
            out["entropy"] = -(logp.exp() * logp.clamp_min(-1e300)).sum(-1).masked_fill(~row, 0)
        if case["k"]:
            out["top_logp"] = logp.topk(case["k"], -1).values.masked_fill(~row[:, None], 0)
            out["top_ids"] = None
        if op.endswith("train"):
            ends = [(out["logp"], "g"), (out.get("top_logp"), "g_top"), (out.get("entropy"), "g_entropy")]
            ends = [(o, wide[g]) for o, g in ends if g in wide]
            grads = torch.autograd.grad([o for o, _ in ends], leaves, [g for _, g in ends])
            names = ["dlogits"] if op == "token_train" else ["dhidden", "dweight"]
            out.update(zip(names, grads))
    return {k: o.detach() if o is not None else None for k, o in out.items()}
