"""Plain float64 forms of the token operators and the norm, for the tests:
straight from their definitions, on the CPU, one value at a time where that is
the plainest way."""

import torch


def ranked(x, k):
    """Indices of the k greatest of each row of x (NaN as -inf), the lowest
    index first among equals."""
    x = torch.where(torch.isnan(x), -torch.inf, x.double())
    return torch.sort(-x, dim=1, stable=True).indices[:, :k]


def token_scores(x, tokens, k, ignore=-100):
    """x [N, V] float64, tokens [N, M] or None -> dict of logp, lse, entropy,
    top_logp, top_ids and active, padding rows filled as documented."""
    n, v = x.shape
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - lse[:, None])
    ent = -torch.where(p > 0, p * (x - lse[:, None]), 0.0).sum(1)
    if tokens is None or tokens.shape[1] == 0:
        active = torch.ones(n, dtype=torch.bool)
        logp = torch.zeros(n, 0, dtype=torch.float64)
    else:
        tokens = tokens.cpu().long()
        active = (tokens != ignore).any(1)
        inside = (tokens >= 0) & (tokens < v)
        logp = x.gather(1, torch.where(inside, tokens, 0)) - lse[:, None]
        logp = torch.where(inside, logp, torch.nan)
        logp = torch.where(tokens == ignore, 0.0, logp)
    ids = ranked(x, k)
    top = x.gather(1, ids) - lse[:, None]
    zero = ~active
    logp[zero], lse, ent = 0.0, lse.masked_fill(zero, 0.0), ent.masked_fill(zero, 0.0)
    return {"logp": logp, "lse": lse, "entropy": ent, "top_logp": top.masked_fill(zero[:, None], 0.0),
            "top_ids": ids.masked_fill(zero[:, None], -1), "active": active}


def token_gradient(x, tokens, g, ids=None, g_top=None, g_ent=None, ignore=-100):
    """The formula's gradient of the float64 logits x, entry by entry, and the
    magnitudes a rounding of its terms can reach."""
    n, v = x.shape
    s = token_scores(x, tokens, 0, ignore)
    p = torch.exp(x - torch.logsumexp(x, 1)[:, None])
    d = torch.zeros_like(x)
    size = torch.zeros_like(x)
    for r in range(n):
        if not s["active"][r]:
            continue
        entries = []
        if tokens is not None:
            entries += [(int(t), float(a)) for t, a in zip(tokens[r], g[r]) if int(t) != ignore]
        if ids is not None:
            entries += [(int(t), float(a)) for t, a in zip(ids[r], g_top[r]) if int(t) >= 0]
        for t, a in entries:
            d[r] -= a * p[r]
            size[r] += abs(a) * p[r]
            if 0 <= t < v:
                d[r, t] += a
                size[r, t] += abs(a)
        if g_ent is not None:
            logp = torch.where(p[r] > 0, x[r] - torch.logsumexp(x[r], 0), 0.0)
            d[r] -= float(g_ent[r]) * p[r] * (logp + s["entropy"][r])
            size[r] += abs(float(g_ent[r])) * p[r] * (logp.abs() + s["entropy"][r])
    return d, size


def norm_forward(s, w, eps):
    """(y, rstd) of the stored sum s, float64."""
    s, w = s.double(), w.double()
    rstd = 1.0 / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    return s * rstd * w, rstd


def norm_gradient(s, w, dy, ds, eps):
    s, w, dy = s.double(), w.double(), dy.double()
    _, rstd = norm_forward(s, w, eps)
    u = s * rstd
    dx = rstd * (dy * w - u * (dy * w * u).mean(-1, keepdim=True))
    if ds is not None:
        dx = dx + ds.double()
    return dx, (dy * u).reshape(-1, s.shape[-1]).sum(0)
