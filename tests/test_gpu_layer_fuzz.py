"""Randomised runs of the embedding, dropout, the layer norm and the 4-bit rows:
sizes near every bound of a kernel's choice and between them, types, strides,
row chunks, outputs asked for; fixed seeds, so that runs repeat, and the case's
own line is printed before it runs.  ITL_FUZZ_EXAMPLES=N (N > 0): N examples a
block, for a longer run.  References and tolerances are those of the
targeted tests: exact for the lookups, the embedding's sums and the 4-bit head
(against the bf16 head on the decoded weight), derived there for the rest."""

import os
import random

import pytest
import torch

import invariant_token_log_amd as itl
from gpu_helpers import dev
from layer_reference import TYPES, dropped, fp4_values
from test_gpu_dropout import close
from test_gpu_fp4 import given, same
from test_gpu_layer_norm import EPS, SEED, check_forward, check_gradient, rows, weights

pytestmark = pytest.mark.gpu

BLOCKS = range(10)
EXAMPLES = int(os.environ.get("ITL_FUZZ_EXAMPLES", "0")) or 50


def size(r, most, bounds=()):
    """1 to `most`: next to one of the bounds, or spread over the logarithm."""
    near = [b for b in bounds if b < most]
    if near and r.random() < 0.5:
        return max(1, min(most, r.choice(near) + r.choice([-1, 0, 0, 1])))
    return max(1, min(most, round(most ** r.random())))


def examples(name, block):
    for i in range(EXAMPLES):
        yield random.Random(f"{name} {block} {i}"), 100000 * block + i


def say(**case):
    print(" ".join(f"{k}={v}" for k, v in case.items()), flush=True)


def padded(t, pad):
    """t on the device, its rows `pad` elements apart more than they need be."""
    return torch.empty(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=dev())[:, :t.shape[1]].copy_(t)


@pytest.mark.parametrize("block", BLOCKS)
def test_head(block):
    for r, seed in examples("head", block):
        n = size(r, 1100, (1, 16, 32, 64, 128, 256, 512, 768, 1024))
        h = 64 * size(r, 40, (1, 2, 3, 4, 8, 12, 16, 32))
        v = size(r, min(9000, 1500000 // h), (1, 32, 64, 128, 256, 512, 1024, 2048, 4096))
        pad, hpad, m = r.choice([0, 0, 1, 3, 4]), r.choice([0, 0, 8, 24]), r.choice([0, 1, 1, 3])
        k = min(v, r.choice([0, 0, 1, 5, 20]) if m else r.choice([1, 5, 20]))
        kw = dict(top_k=k, return_entropy=r.random() < 0.5, temperature=r.choice([1.0, 0.7]), round_logits=r.random() < 0.3)
        chunk = r.choice([0, 0, 256, 512])
        say(seed=seed, n=n, h=h, v=v, pad=pad, hpad=hpad, m=m, chunk=chunk, **kw)
        gen = torch.Generator().manual_seed(seed)
        data = torch.randint(0, 256, (v, h // 2), generator=gen, dtype=torch.uint8)
        scale = torch.randint(112, 123, (v, h // 32), generator=gen, dtype=torch.uint8)
        w = fp4_values(data, scale).bfloat16().to(dev())
        x = padded(torch.randn(n, h, generator=gen).bfloat16(), hpad)
        tok = given(n, v, m, seed) if m else None
        got = itl.linear_token_logp_fwd(x, itl.Fp4Rows(padded(data, 16 * pad), padded(scale, pad)), tok, row_chunk=chunk, **kw)
        same(got, itl.linear_token_logp_fwd(x, w, tok, **kw))


@pytest.mark.parametrize("block", BLOCKS)
def test_embedding(block):
    for r, seed in examples("embedding", block):
        n = size(r, 40000, (1, 4, 32, 33, 64, 2048, 4096, 16384, 32768))
        h = size(r, min(5000, 2000000 // n + 1), (1, 8, 64, 256, 512, 1024, 2048, 4096))
        v = size(r, min(2000000, 8000000 // h + 1), (1, 64, 1000, (1 << 20) - 1))
        name = r.choice(list(TYPES))
        dtype, index = TYPES[name], r.choice([torch.int64, torch.int64, torch.int32])
        ypad, tpad = r.choice([0, 0, 1, 8]), r.choice([0, 0, 3, 8])
        power, f32, add = r.choice([1, 3, 8]), r.random() < 0.4, r.random() < 0.4
        say(seed=seed, n=n, h=h, v=v, dtype=name, index=index, ypad=ypad, tpad=tpad, power=power, f32=f32, add=add)
        gen = torch.Generator().manual_seed(seed)
        ids = (torch.rand(n, generator=gen, dtype=torch.float64) ** power * (v + 1)).long()  # v: invalid
        ids[torch.rand(n, generator=gen) < 0.1] = -100
        live = (ids >= 0) & (ids < v)
        ids_d = ids.to(index).to(dev())
        # sixteenths, at most 2^15.3 of them to a token: sums below 2^20 sixteenths, exact in fp32
        dy = torch.randint(-16, 17, (n, h), generator=gen).float() / 16
        old = (torch.randint(-8, 9, (v, h), generator=gen).float() / 8).to(torch.float32 if f32 else dtype)
        want = torch.zeros(v, h, dtype=torch.float64).index_add_(0, ids[live], dy[live].double()) * 0.5
        want = (want + old.double() if add else want).to(old.dtype)
        out = padded(old, tpad)
        got = itl.embedding_bwd(ids_d, padded(dy.to(dtype), ypad), v, scale=0.5, dweight_out=out, accumulate=add)
        assert got is out and torch.equal(got.cpu(), want)
        table = torch.randn(v, h, generator=gen).to(dtype)
        y = itl.embedding_fwd(ids_d, padded(table, tpad), scale=0.75).cpu()
        assert torch.equal(y[live], (table[ids[live]].float() * 0.75).to(dtype))
        assert not y[ids == -100].any() and y[ids == v].isnan().all()


@pytest.mark.parametrize("block", BLOCKS)
def test_rows_of_four_bits(block):
    for r, seed in examples("rows", block):
        h = 32 * size(r, 300, (1, 2, 8, 32, 64, 128, 256))
        v = size(r, min(5000, 600000 // h + 1), (1, 64, 256))
        n = size(r, min(40000, 2000000 // h + 1), (1, 4, 64, 1024, 4096, 16384))
        name, scale, pad = r.choice(list(TYPES)), r.choice([1.0, 0.75, 1.3]), r.choice([0, 0, 1, 8])
        say(seed=seed, n=n, h=h, v=v, dtype=name, scale=scale, pad=pad)
        gen = torch.Generator().manual_seed(seed)
        x = (torch.randn(v, h, generator=gen) * torch.exp2(torch.randint(-9, 9, (v, 1), generator=gen))).to(TYPES[name])
        q = itl.quantize_rows_fp4(padded(x, pad))
        values, step = fp4_values(q.data, q.scale), 2.0 ** (q.scale.cpu().double() - 127).repeat_interleave(32, 1)
        a = x.double().abs() / step
        # within 6 of the least scale, and half the distance between neighbours: 1/4 below 2, 1/2 to 4, 1 to 6
        assert ((a.view(v, -1, 32).amax(2) <= 6) & (a.view(v, -1, 32).amax(2) > 3)).all()
        assert ((values - x.double()).abs() <= step * torch.where(a < 2, 0.25, torch.where(a < 4, 0.5, 1.0))).all()
        ids = torch.randint(-1, v + 1, (n,), generator=gen)
        live = (ids >= 0) & (ids < v)
        y = itl.embedding_fwd(ids.to(dev()), q, scale=scale, ignore_index=-1, out_dtype=TYPES[name]).cpu()
        assert torch.equal(y[live], (values.float()[ids[live]] * torch.tensor(scale)).to(TYPES[name]))
        assert not y[ids == -1].any() and y[ids == v].isnan().all()


@pytest.mark.parametrize("block", BLOCKS)
def test_norm_and_dropout(block):
    ends = (1, 8, 512, 1024, 2048, 4096, 6144, 8192, 12288, 16384, 24576, 32768)
    for r, seed in examples("norm", block):
        h = size(r, 40000, ends)
        n = size(r, min(3000, 400000 // h + 1), (1, 4, 102, 256, 512, 1024, 2048))
        name, p, pad, draw = r.choice(list(TYPES)), r.choice([0.0, 0.1, 0.5]), r.choice([0, 0, 1, 8]), r.randrange(1 << 32)
        residual, bias, with_ds = r.random() < 0.7, r.random() < 0.7, r.random() < 0.5
        say(seed=seed, n=n, h=h, dtype=name, p=p, pad=pad, draw=draw, residual=residual, bias=bias, with_ds=with_ds)
        x, xd = rows(n, h, name, seed, pad=pad)
        c, cd = rows(n, h, name, seed + 1, 3.0, 0.5, pad) if residual else (None, None)
        w, b = weights(h, name)
        wd = w.to(dev())
        y, s, mean, rstd = itl.layer_norm_fwd(xd, wd, b.to(dev()) if bias else None, residual=cd, eps=EPS, dropout=p, seed=SEED,
                                              draw=draw, return_stats=True)
        if p:
            close(s, dropped(x.double(), p, SEED, draw) + (c.double() if residual else 0.0), name)
            assert torch.equal(itl.dropout_fwd(xd, p, SEED, residual=cd, draw=draw), s)
        else:
            assert torch.equal(s.cpu(), (x.float() + c.float()).to(TYPES[name]) if residual else x)
        check_forward(y, mean, rstd, s.cpu(), w, b if bias else None, name)
        dy, dyd = rows(n, h, name, seed + 2, pad=pad)
        ds, dsd = rows(n, h, name, seed + 3, pad=pad) if with_ds else (None, None)
        got = itl.layer_norm_bwd(s, wd, mean, rstd, dyd, dsd, dropout=p, seed=SEED, draw=draw)
        check_gradient(got, s.cpu(), w, dy, ds, name, p, draw)
