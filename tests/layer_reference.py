"""Plain float64 forms of the embedding, dropout, the layer norm and 4-bit rows,
for the tests: straight from their definitions, on the CPU."""

import numpy as np
import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def philox(counter, key):
    """One block of Philox-4x32-10: four words from four and two (Python
    integers)."""
    c, k, low = list(counter), list(key), 0xFFFFFFFF
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & low, (a >> 32) ^ c[3] ^ k[1], a & low]
        k = [(k[0] + 0x9E3779B9) & low, (k[1] + 0xBB67AE85) & low]
    return c


def kept(n, h, p, seed, draw=0, first_row=0):
    """(mask [n, h] of the kept elements, their factor)."""
    u, low, half = np.uint64, np.uint64(0xFFFFFFFF), np.uint64(32)
    chunks = (h + 7) // 8
    row = (np.arange(n, dtype=np.uint64) + u(first_row)).repeat(chunks)
    c = [np.tile(np.arange(chunks, dtype=np.uint64), n), row & low, row >> half,
         np.full(n * chunks, draw, dtype=np.uint64)]
    k = [u(seed & 0xFFFFFFFF), u((seed >> 32) & 0xFFFFFFFF)]
    for _ in range(10):
        a, b = u(0xD2511F53) * c[0], u(0xCD9E8D57) * c[2]
        c = [(b >> half) ^ c[1] ^ k[0], b & low, (a >> half) ^ c[3] ^ k[1], a & low]
        k = [(k[0] + u(0x9E3779B9)) & low, (k[1] + u(0xBB67AE85)) & low]
    words = np.stack(c, 1)
    numbers = np.stack([words & u(0xFFFF), words >> u(16)], 2).reshape(n, 8 * chunks)[:, :h]
    least = int(np.floor(p * 65536 + 0.5))
    factor = float(np.float32(65536 / (65536 - least))) if least < 65536 else 0.0
    return torch.from_numpy(numbers >= u(least)), factor


def dropped(x, p, seed, draw=0, first_row=0):
    """x float64 with its dropped elements 0 and the others scaled."""
    mask, factor = kept(*x.shape, p, seed, draw, first_row)
    return torch.where(mask, x.double() * factor, 0.0)


def layer_norm(s, w, b, eps):
    """(y, mean, rstd) of rows s, float64."""
    s, w = s.double(), w.double()
    m = s.mean(1, keepdim=True)
    rs = 1.0 / torch.sqrt(((s - m) ** 2).mean(1, keepdim=True) + eps)
    y = (s - m) * rs * w
    return (y if b is None else y + b.double()), m, rs


def layer_norm_gradient(s, w, dy, ds, eps):
    """(d, dweight, dbias): d is the gradient of s."""
    _, m, rs = layer_norm(s, w, None, eps)
    dy, u = dy.double(), (s.double() - m) * rs
    g = dy * w.double()
    d = rs * (g - g.mean(1, keepdim=True) - u * (g * u).mean(1, keepdim=True))
    return (d if ds is None else d + ds.double()), (dy * u).sum(0), dy.sum(0)


def embedding_gradient(ids, dy, v, scale, ignore):
    d = torch.zeros(v, dy.shape[1], dtype=torch.float64)
    for i, t in enumerate(ids.tolist()):
        if t != ignore and 0 <= t < v:
            d[t] += dy[i].double() * scale
    return d


def fp4_values(data, scale):
    """4-bit rows (uint8 tensors) as float64."""
    data, scale = data.cpu().long(), scale.cpu().long()
    table = torch.tensor(E2M1 + [-x for x in E2M1], dtype=torch.float64)
    q = torch.stack([table[data & 15], table[data >> 4]], 2).flatten(1)
    factor = torch.where(scale == 255, torch.nan, 2.0 ** (scale.double() - 127))
    return q * factor.repeat_interleave(32, 1)


def to_fp4(x):
    """x [n, h] float64 -> (codes [n, h], scale bytes [n, h / 32]) from the
    definition: the first of the scales 2^-126 .. 2^125 that brings a group within
    6, the nearest of the eight magnitudes, an even code at a tie."""
    n, h = x.shape
    codes, scales = torch.zeros(n, h, dtype=torch.long), torch.zeros(n, h // 32, dtype=torch.long)
    for r in range(n):
        for g in range(h // 32):
            part = x[r, 32 * g:32 * g + 32].double()
            if not torch.isfinite(part).all():
                scales[r, g] = 255
                continue
            b = 1
            while b < 252 and part.abs().max() > 6 * 2.0 ** (b - 127):
                b += 1
            scales[r, g] = b
            for j, val in enumerate(part.tolist()):
                a = abs(val) / 2.0 ** (b - 127)
                best = min(range(8), key=lambda c: (abs(E2M1[c] - a), c % 2))
                codes[r, 32 * g + j] = best + 8 * (np.signbit(val))
    return codes, scales
