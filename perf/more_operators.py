"""The cases on which the operators around the token operators are measured, and their plain forms.

Operators (N rows, H hidden columns, V vocabulary rows):

  embed          rows of a [V, H] table by token, times a scale; embed_train adds the table's gradient, whole
  embed_fp4      the same lookup from a table in 4 bits
  dropout_train  residual + dropout(x) from a counter-based generator, and the gradient of x
  norm           layer norm of x + residual; norm_train adds dropout on x and the gradients of x, residual, weight and bias
  linear_fp4     log-probabilities, row log-sum-exp, entropy and the k most probable tokens through a language-model
                 head in 4 bits

4-bit rows: two e2m1 values a byte, the even column in the low half, and one scale byte b for every 32 columns, which
stands for 2^(b - 127).  Dropout: Philox-4x32-10 with the key seed (low word, high word) and the counter (column / 8,
row, row / 2^32, draw) gives eight 16-bit numbers u, two a word, the low half first; column 8 c + i is kept where u[i] >=
round(65536 p), and scaled by 65536 / (65536 - round(65536 p)).

run() computes the plain form in 32 bits where `own` is false, and makes the framework's calls where it is true.
"""

import math

import numpy as np
import torch

own = False

IGNORE = -100  # a token that is left out: its row is zeros and takes no gradient
EPS = 1e-5
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DRAW = 5  # the layer's number within a training step


def listed():
    return [
        # the tokens of 16 sequences that decode together (latency)
        dict(name="embed-decode-16", op="embed", n=16, h=4096, v=151936, dtype="bf16"),
        # a training batch of text, a few tokens very often, 5% padding: the rows and the whole table's gradient
        dict(name="embed-train-16384", op="embed_train", n=16384, h=4096, v=151936, dtype="bf16"),
        # an odd vocabulary and rows that start off 16 bytes
        dict(name="embed-odd-fp32", op="embed_train", n=2047, h=1597, v=50257, dtype="fp32"),
        # a prompt's tokens from the table that a 4-bit head shares
        dict(name="embed-fp4-4096", op="embed_fp4", n=4096, h=4096, v=151936),
        # the residual stream of a training step behind an attention or a feed-forward layer
        dict(name="dropout-train-8192", op="dropout_train", n=8192, h=4096, dtype="bf16", p=0.1, residual=True),
        # dropout of an odd number of fp32 columns, nothing added
        dict(name="dropout-odd-fp32", op="dropout_train", n=509, h=5003, dtype="fp32", p=0.25, residual=False),
        # the norm of a decoding step (latency)
        dict(name="norm-decode-16", op="norm", n=16, h=4096, dtype="bf16"),
        # the norm of a training step behind dropout and the residual's addition, forward and backward
        dict(name="norm-train-8192", op="norm_train", n=8192, h=4096, dtype="bf16", p=0.1),
        # odd rows in fp16 without dropout, forward and backward
        dict(name="norm-odd-fp16", op="norm_train", n=2047, h=5117, dtype="fp16", p=0.0),
        # one sequence's next token through the 4-bit head: its log-probability and 5 alternatives
        dict(name="linear-fp4-decode-1", op="linear_fp4", n=1, h=4096, v=151936, m=1, k=5, temperature=1.0, entropy=False),
        # decoding 32 sequences, 20 alternatives each
        dict(name="linear-fp4-decode-32", op="linear_fp4", n=32, h=4096, v=151936, m=1, k=20, temperature=0.7, entropy=False),
        # scoring a prompt of 1000 positions
        dict(name="linear-fp4-score-1000", op="linear_fp4", n=1000, h=4096, v=151936, m=1, k=0, temperature=1.0, entropy=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["embed", "embed_train", "embed_train", "embed_fp4", "dropout_train", "norm", "norm_train", "norm_train",
                     "linear_fp4", "linear_fp4"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("embed", "embed_train"):
        return dict(op=op, n=_log_int(rng, 1, 16384), h=8 * _log_int(rng, 8, 256) - rng.choice([0, 0, 3]),
                    v=_log_int(rng, 1000, 151936), dtype=dtype)
    if op == "embed_fp4":
        return dict(op=op, n=_log_int(rng, 1, 8192), h=32 * _log_int(rng, 2, 128), v=_log_int(rng, 1000, 151936))
    if op == "linear_fp4":
        return dict(op=op, n=_log_int(rng, 1, 1000), h=64 * _log_int(rng, 4, 64), v=_log_int(rng, 1000, 151936),
                    m=rng.choice([1, 1, 2, 5]), k=rng.choice([0, 1, 5, 20, 64]), temperature=rng.choice([1.0, 1.0, 0.7, 1.3]),
                    entropy=rng.random() < 0.5)
    case = dict(op=op, n=_log_int(rng, 1, 8192), h=8 * _log_int(rng, 16, 1024) - rng.choice([0, 0, 0, 3]), dtype=dtype)
    if op != "norm":
        case["p"] = rng.choice([0.1, 0.1, 0.05, 0.2, 0.5] + ([0.0, 0.0] if op == "norm_train" else []))
    if op == "dropout_train":
        case["residual"] = rng.random() < 0.7
    return case


def _grid(shape, step, std, gen):
    """Normal values on a grid of `step`, at most 127 steps: with 4-bit weights the sums of products are exact in 32 bits, so which of two tokens is the
    more probable does not hang on the order of a sum."""
    x = torch.randn(shape, generator=gen, device=gen.device)
    return x.mul_(std / step).round_().clamp_(-127, 127).mul_(step).to(torch.bfloat16)


def _to_fp4(x):
    """x [V, H] as (codes [V, H / 2], scale bytes [V, H / 32]): the smallest power of two that brings a group of 32 within 6, values rounded to nearest even."""
    v, h = x.shape
    g = x.view(v, h // 32, 32)
    most = g.abs().amax(2, keepdim=True).clamp_min(1e-30)
    e = torch.ceil(torch.log2(most / 6.0))
    a = (g * torch.exp2(-e)).view(v, h)
    m = a.abs()
    code = torch.zeros(v, h, dtype=torch.uint8, device=x.device)
    for i, t in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += (m > t if i % 2 == 0 else m >= t)
    code |= (a < 0).to(torch.uint8) << 3
    return code[:, ::2] | (code[:, 1::2] << 4), (e[:, :, 0] + 127).to(torch.uint8)


def _table_fp4(v, h, gen):
    codes = torch.empty(v, h // 2, dtype=torch.uint8, device=gen.device)
    scales = torch.empty(v, h // 32, dtype=torch.uint8, device=gen.device)
    for i in range(0, v, 16384):
        codes[i:i + 16384], scales[i:i + 16384] = _to_fp4(torch.randn(min(16384, v - i), h, generator=gen, device=gen.device).mul_(0.02))
    return codes, scales


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    s = dict(case=case)
    n, h, op = case["n"], case["h"], case["op"]
    t = TYPES[case.get("dtype", "bf16")]
    if op.startswith("embed"):
        v = case["v"]
        # tokens as in text: a few of them very often; one in 20 is padding
        ids = (torch.rand(n, generator=gen, device=dev, dtype=torch.float64).pow_(3) * v).long().clamp_(max=v - 1)
        pad = torch.rand(n, generator=gen, device=dev) < 0.05
        pad[0] = False
        s["ids"] = ids.masked_fill_(pad, IGNORE)
        s["scale"] = math.sqrt(h)
        if op == "embed_fp4":
            s["codes"], s["scales"] = _table_fp4(v, h, gen)
            return s
        s["table"] = randn(v, h).mul_(0.02).to(t)
        if op == "embed_train":
            s["dy"] = randn(n, h).to(t)
            s["table"].requires_grad_()
        return s
    if op == "linear_fp4":
        v, m = case["v"], case["m"]
        tokens = torch.randint(0, v, (n, m), generator=gen, device=dev)
        drop = torch.rand(n, m, generator=gen, device=dev) < 0.05
        drop[0, 0] = False
        s["tokens"] = tokens.masked_fill_(drop, IGNORE)
        s["hidden"] = _grid((n, h), 1 / 16, 1.0, gen)
        s["codes"], s["scales"] = _table_fp4(v, h, gen)
        return s
    s["seed"] = torch.randint(0, 2**62, (1,), generator=gen, device=dev)
    s["x"] = randn(n, h).to(t)
    if op != "dropout_train" or case["residual"]:
        s["residual"] = (3 * randn(n, h) + 0.5).to(t)
    if op == "dropout_train":
        s["dy"] = randn(n, h).to(t)
        s["x"].requires_grad_()
        return s
    s["weight"] = (1 + 0.1 * randn(h)).to(t)
    s["bias"] = (0.1 * randn(h)).to(t)
    if op == "norm_train":
        s["dy"] = randn(n, h).to(t)
        s["dsum"] = randn(n, h).to(t)
        for k in ("x", "residual", "weight", "bias"):
            s[k].requires_grad_()
    return s


# ---- the plain forms -----------------------------------------------------------------------------------------


def _kept(n, h, p, seed):
    """Which elements [n, h] dropout keeps, and their factor: Philox-4x32-10 in whole numbers of 64 bits."""
    low = 0xFFFFFFFF
    chunks = (h + 7) // 8
    row = torch.arange(n, device=seed.device)[:, None].expand(n, chunks)
    c0, c1, c2 = torch.arange(chunks, device=seed.device).expand(n, chunks), row & low, row >> 32
    c3 = torch.full_like(c0, DRAW)
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # 64-bit products modulo 2^64: both halves are right
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([c0, c1, c2, c3], 2)
    u = torch.stack([words & 0xFFFF, words >> 16], 3).view(n, chunks * 8)[:, :h]
    least = int(p * 65536 + 0.5)
    return u >= least, 65536.0 / (65536 - least)


def _dropped(s):
    x, p = s["x"].float(), s["case"].get("p", 0.0)
    if not p:
        return x, None, 1.0
    keep, factor = _kept(*x.shape, p, s["seed"])
    return torch.where(keep, x * factor, 0.0), keep, factor


def _from_fp4(codes, scales):
    """4-bit rows as 32-bit values."""
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    out = torch.empty(codes.shape[0], codes.shape[1] * 2, device=codes.device)
    for i in range(0, codes.shape[0], 16384):
        c = codes[i:i + 16384]
        f = torch.stack([lut[(c & 15).long()], lut[(c >> 4).long()]], 2).view(c.shape[0], -1, 32)
        out[i:i + 16384] = (f * torch.exp2(scales[i:i + 16384].float() - 127)[:, :, None]).view(c.shape[0], -1)
    return out


def _top(x, k):
    """The k largest of each row, the lowest index first among equals: one whole number a value that orders by (value, -index)."""
    bits = (x + 0.0).view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).to(torch.int64) << 32
    key += torch.arange(x.shape[1] - 1, -1, -1, device=x.device)
    return x.shape[1] - 1 - (key.topk(k, dim=1).values & 0xFFFFFFFF)


def _scores(x, tokens, case):
    """Log-probabilities, row log-sum-exp, entropy and alternatives of 32-bit logits x."""
    given = tokens != IGNORE
    active = given.any(1)
    top = x.amax(1)
    d = x - top[:, None]
    e = d.exp()
    total = e.sum(1)
    lse = top + total.log()
    out = {"logp": torch.where(given, x.gather(1, tokens.clamp(min=0)) - lse[:, None], 0.0), "lse": torch.where(active, lse, 0.0)}
    if case["entropy"]:
        out["entropy"] = torch.where(active, total.log() - (e * d).sum(1) / total, 0.0)
    if case["k"]:
        ids = _top(x, case["k"])
        out["top_logp"] = torch.where(active[:, None], x.gather(1, ids) - lse[:, None], 0.0)
        out["top_ids"] = torch.where(active[:, None], ids, -1)
    return out


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op.startswith("embed"):
        ids, live = s["ids"].clamp(min=0), s["ids"] != IGNORE
        if op == "embed_fp4":
            rows = _from_fp4(s["codes"][ids], s["scales"][ids])
            return {"y": torch.where(live[:, None], rows * s["scale"], 0.0).to(torch.bfloat16)}
        t = s["table"].dtype
        out = {"y": torch.where(live[:, None], s["table"][ids].float() * s["scale"], 0.0).to(t)}
        if op == "embed_train":
            d = torch.zeros(s["table"].shape, device=ids.device)
            d.index_add_(0, ids[live], s["dy"].float()[live])
            out["dtable"] = d.mul_(s["scale"]).to(t)
        return out
    if op == "linear_fp4":
        x = s["hidden"].float() @ _from_fp4(s["codes"], s["scales"]).T
        if case["temperature"] != 1.0:
            x = x * (1.0 / case["temperature"])
        return _scores(x, s["tokens"], case)
    x, keep, factor = _dropped(s)
    t = s["x"].dtype
    total = (x + s["residual"].float() if "residual" in s else x).to(t)  # the residual stream is stored in its type
    if op == "dropout_train":
        return {"sum": total, "dx": torch.where(keep, s["dy"].float() * factor, 0.0).to(t)}
    f, w = total.float(), s["weight"].float()
    f = f - f.mean(1, keepdim=True)
    scale = (f.square().mean(1, keepdim=True) + EPS).rsqrt()
    unit = f * scale
    out = {"y": (unit * w + s["bias"].float()).to(t), "sum": total}
    if op == "norm_train":
        dy = s["dy"].float()
        g = dy * w
        ds = s["dsum"].float() + scale * (g - g.mean(1, keepdim=True) - unit * (g * unit).mean(1, keepdim=True))
        out["dresidual"] = ds.to(t)
        out["dx"] = (ds if keep is None else torch.where(keep, ds * factor, 0.0)).to(t)
        out["dweight"], out["dbias"] = (dy * unit).sum(0).to(t), dy.sum(0).to(t)
    return out


# ---- the framework's calls -----------------------------------------------------------------------------------


def _ours(s):
    import invariant_token_log_amd as itl

    case, op = s["case"], s["case"]["op"]
    if op == "embed":
        return {"y": itl.embedding_fwd(s["ids"], s["table"], scale=s["scale"], ignore_index=IGNORE)}
    if op == "embed_fp4":
        return {"y": itl.embedding_fwd(s["ids"], itl.Fp4Rows(s["codes"], s["scales"]), scale=s["scale"], ignore_index=IGNORE)}
    if op == "embed_train":
        y = itl.embedding(s["ids"], s["table"], scale=s["scale"], ignore_index=IGNORE)
        return {"y": y, "dtable": torch.autograd.grad(y, s["table"], s["dy"])[0]}
    if op == "dropout_train":
        y = itl.dropout(s["x"], case["p"], s["seed"], residual=s.get("residual"), draw=DRAW)
        return {"sum": y, "dx": torch.autograd.grad(y, s["x"], s["dy"])[0]}
    if op == "norm":
        y, total, _, _ = itl.layer_norm_fwd(s["x"], s["weight"], s["bias"], residual=s["residual"], eps=EPS)
        return {"y": y, "sum": total}
    if op == "norm_train":
        y, total = itl.layer_norm(s["x"], s["weight"], s["bias"], residual=s["residual"], eps=EPS, dropout=case["p"],
                                  seed=s["seed"], draw=DRAW)
        grads = torch.autograd.grad([y, total], [s["x"], s["residual"], s["weight"], s["bias"]], [s["dy"], s["dsum"]])
        return {"y": y, "sum": total, **dict(zip(("dx", "dresidual", "dweight", "dbias"), grads))}
    r = itl.linear_token_logp_fwd(s["hidden"], itl.Fp4Rows(s["codes"], s["scales"]), s["tokens"], top_k=case["k"], ignore_index=IGNORE,
                                  temperature=case["temperature"], return_entropy=case["entropy"])
    out = {"logp": r.logp, "lse": r.lse}
    if case["entropy"]:
        out["entropy"] = r.entropy
    if case["k"]:
        out["top_logp"], out["top_ids"] = r.top_logp, r.top_ids
    return out


def run(state):
    if own:
        return _ours(state)
    with torch.no_grad():
        return _plain(state)


# ---- what a pass cannot do without ---------------------------------------------------------------------------


def work(case):
    n, h, op = case["n"], case["h"], case["op"]
    cells, size = n * h, SIZE[case.get("dtype", "bf16")]
    if op == "embed_fp4":
        return {"bytes": cells * (1 / 2 + 1 / 32 + 2) + 8 * n, "flops": 2 * cells}
    if op == "embed":
        return {"bytes": 2 * cells * size + 8 * n, "flops": cells}
    if op == "embed_train":
        return {"bytes": (3 * cells + case["v"] * h) * size + 16 * n, "flops": 2 * cells + case["v"] * h}
    if op == "linear_fp4":
        return {"bytes": case["v"] * h * (1 / 2 + 1 / 32) + 2 * cells + n * (12 * case["m"] + 12 * case["k"] + 8),
                "flops": 2 * cells * case["v"]}
    if op == "dropout_train":
        return {"bytes": (5 if case["residual"] else 4) * cells * size, "flops": 4 * cells}
    if op == "norm":
        return {"bytes": (4 * cells + 2 * h) * size, "flops": 8 * cells}
    return {"bytes": ((9 if case["p"] else 8) * cells + 4 * h) * size, "flops": 24 * cells}


# ---- the definition, in 64 bits ------------------------------------------------------------------------------


def _mask64(n, h, p, seed):
    """The kept elements once more, in numpy's unsigned numbers."""
    u, low = np.uint64, np.uint64(0xFFFFFFFF)
    half = u(32)
    wide = (h + 7) // 8
    at = np.arange(n * wide, dtype=np.uint64)
    ctr = [at % u(wide), at // u(wide), np.zeros_like(at), np.full_like(at, DRAW)]
    key = [u(seed & 0xFFFFFFFF), u(seed >> 32)]
    for _ in range(10):
        first, third = u(0xD2511F53) * ctr[0], u(0xCD9E8D57) * ctr[2]
        ctr = [(third >> half) ^ ctr[1] ^ key[0], third & low, (first >> half) ^ ctr[3] ^ key[1], first & low]
        key = [(key[0] + u(0x9E3779B9)) & low, (key[1] + u(0xBB67AE85)) & low]
    lanes = np.stack(ctr, -1).astype("<u4").view("<u2").reshape(n, wide * 8)[:, :h]
    return torch.from_numpy((lanes >= math.floor(p * 65536 + 0.5)).copy())


def _wide_fp4(codes, scales):
    pair = torch.stack([codes.bitwise_and(15), codes.bitwise_right_shift(4)], -1).flatten(1)
    out = torch.empty(pair.shape, dtype=torch.float64, device=pair.device)
    for i in range(0, len(pair), 8192):
        q = pair[i:i + 8192].to(torch.int32)
        mantissa, exponent = q & 1, (q >> 1) & 3
        # e2m1: 2^(e - 1) (1 + m / 2), or m / 2 where e is 0
        value = torch.where(exponent == 0, mantissa * 0.5, torch.ldexp(1.0 + 0.5 * mantissa.double(), exponent - 1))
        value = torch.where(q >= 8, -value, value).double()
        out[i:i + 8192] = torch.ldexp(value, scales[i:i + 8192].to(torch.int32).sub_(127).repeat_interleave(32, 1))
    return out


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    n, h = case["n"], case["h"]
    if op.startswith("embed"):
        live = s["ids"].ne(IGNORE).nonzero()[:, 0]
        ids = s["ids"][live]
        y = torch.zeros(n, h, dtype=torch.float64, device=ids.device)
        if op == "embed_fp4":
            y[live] = _wide_fp4(s["codes"][ids], s["scales"][ids]) * s["scale"]
            return {"y": y}
        table = s["table"].detach()
        y[live] = table[ids].double() * s["scale"]
        if op == "embed":
            return {"y": y}
        d = torch.zeros(table.shape, dtype=torch.float64, device=ids.device)
        return {"y": y, "dtable": d.index_put_((ids,), s["dy"][live].double() * s["scale"], accumulate=True)}
    if op == "linear_fp4":
        x = torch.mm(s["hidden"].double(), _wide_fp4(s["codes"], s["scales"]).t()) / case["temperature"]
        keep = s["tokens"].ne(IGNORE)
        row = keep.any(-1)
        logp = torch.log_softmax(x, -1)
        out = {"logp": logp.gather(-1, s["tokens"].masked_fill(~keep, 0)).masked_fill(~keep, 0),
               "lse": torch.logsumexp(x, -1).masked_fill(~row, 0)}
        if case["entropy"]:
            out["entropy"] = -(logp.exp() * logp).sum(-1).masked_fill(~row, 0)
        if case["k"]:
            out["top_logp"] = logp.topk(case["k"], -1).values.masked_fill(~row[:, None], 0)
            out["top_ids"] = None
        return out
    x = s["x"].detach().double()
    factor = None
    if case.get("p"):
        kept = _mask64(n, h, case["p"], int(s["seed"].item())).to(x.device)
        factor = kept.double() / (1 - math.floor(case["p"] * 65536 + 0.5) / 65536)
        x = x * factor
    total = x + s["residual"].detach().double() if "residual" in s else x
    if op == "dropout_train":
        return {"sum": total, "dx": s["dy"].double() * factor}
    with torch.enable_grad():
        a = total.to(TYPES[case["dtype"]]).double().requires_grad_()
        w, b = s["weight"].detach().double().requires_grad_(), s["bias"].detach().double().requires_grad_()
        y = (a - a.mean(-1, keepdim=True)) / torch.sqrt(a.var(-1, correction=0, keepdim=True) + EPS) * w + b
        out = {"y": y.detach(), "sum": total}
        if op == "norm_train":
            ds, dw, db = torch.autograd.grad([y, a * 1.0], [a, w, b], [s["dy"].double(), s["dsum"].double()])
            out.update(dx=ds if factor is None else ds * factor, dresidual=ds, dweight=dw, dbias=db)
    return out
