"""Dropout with the residual's addition against the generator's definition.

The mask is compared exactly.  Values: the factor is one fp32 number, the product
and the residual's addition are rounded together or not at all to fp32, half a
step of 2^-24, and the result rounds once to its type: eps / 2 of it (fp16
subnormals: 2^-25)."""

import pytest
import torch

import invariant_token_log_amd as itl
from gpu_helpers import dev
from layer_reference import TYPES, dropped, kept

pytestmark = pytest.mark.gpu

SEED = 0x0123456789ABCDEF
LENGTHS = [1, 7, 8, 9, 100, 1021, 2048, 2056, 4096, 5003]


def rows(n, h, dtype, seed, pad=0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(n, h, generator=gen).to(TYPES[dtype])
    buf = torch.zeros(n, h + pad, dtype=x.dtype, device=dev())[:, :h]
    buf.copy_(x)
    return x, buf


def close(got, ref, dtype):
    got, half = got.detach().double().cpu(), torch.finfo(TYPES[dtype]).eps / 2
    bound = ref.abs() * (half * (1 + 2.0 ** -20) + 2.0 ** -23) + (2.0 ** -25 if dtype == "fp16" else 0)
    assert ((got - ref).abs() <= bound).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("h", LENGTHS)
def test_forward(h, dtype):
    n, p = 11, 0.3
    for residual, pad in ((True, 0), (False, 0), (True, 3)):
        x, xd = rows(n, h, dtype, h, pad)
        r, rd = rows(n, h, dtype, h + 1, pad) if residual else (None, None)
        y = itl.dropout_fwd(xd, p, SEED, residual=rd, draw=3)
        ref = dropped(x.double(), p, SEED, 3)
        close(y, ref + r.double() if residual else ref, dtype)


@pytest.mark.parametrize("p", [0.0, 2.0 ** -17 - 1e-9, 2.0 ** -16, 0.1, 0.5, 0.999, 1 - 2.0 ** -16, 1 - 2.0 ** -18, 1.0])
def test_mask(p):
    n, h = 300, 1003
    x = torch.ones(n, h, device=dev())
    mask, factor = kept(n, h, p, SEED)
    y = itl.dropout_fwd(x, p, SEED).cpu()
    assert torch.equal(y != 0, mask if factor else torch.zeros_like(mask))
    assert (y[mask] == torch.tensor(factor, dtype=torch.float32)).all()
    share = mask.float().mean().item()
    assert abs(share - (1 - p)) <= 6 * (p * (1 - p) / (n * h)) ** 0.5 + 2.0 ** -16


def test_known_block():
    """The generator's published answers for a counter and key of zeros, and of
    all ones."""
    from layer_reference import philox

    assert philox([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert philox([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    # the first chunk of row 0 and of a row past 2^32, at several thresholds
    for row in (0, 5 * 2 ** 32 + 77):
        words = philox([0, row % 2 ** 32, row // 2 ** 32, 9], [SEED % 2 ** 32, SEED >> 32])
        numbers = [w >> s & 0xFFFF for w in words for s in (0, 16)]
        for least in sorted(numbers):
            y = itl.dropout_fwd(torch.ones(1, 8, device=dev()), least / 65536, SEED, draw=9, first_row=row)
            assert [v != 0 for v in y[0].tolist()] == [u >= least for u in numbers]


@pytest.mark.parametrize("seed", [0, -1, 2 ** 63, 2 ** 64 - 1, SEED])
def test_seeds_and_draws(seed):
    x = torch.ones(40, 264, device=dev())
    for draw in (0, 1, 2 ** 32 - 1):
        got = itl.dropout_fwd(x, 0.5, seed, draw=draw).cpu() != 0
        assert torch.equal(got, kept(40, 264, 0.5, seed % 2 ** 64, draw)[0])
        at = torch.tensor([seed - 2 ** 64 if seed >= 2 ** 63 else seed], device=dev())
        assert torch.equal(itl.dropout_fwd(x, 0.5, at, draw=draw).cpu() != 0, got)


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_alone_strided_and_in_place(dtype):
    x, xd = rows(13, 333, dtype, 1)
    r, rd = rows(13, 333, dtype, 2)
    y = itl.dropout_fwd(xd, 0.2, SEED, residual=rd, draw=1)
    # a row alone, a later part of the batch
    assert torch.equal(itl.dropout_fwd(xd[5:6], 0.2, SEED, residual=rd[5:6], draw=1, first_row=5), y[5:6])
    assert torch.equal(itl.dropout_fwd(xd[4:], 0.2, SEED, residual=rd[4:], draw=1, first_row=4), y[4:])
    _, xp = rows(13, 333, dtype, 1, pad=5)
    assert torch.equal(itl.dropout_fwd(xp, 0.2, SEED, residual=rd, draw=1), y)
    wide = torch.full((13, 340), 7.0, dtype=TYPES[dtype], device=dev())
    itl.dropout_fwd(xd, 0.2, SEED, residual=rd, draw=1, out=wide[:, :333])
    assert torch.equal(wide[:, :333], y) and (wide[:, 333:] == 7).all()
    for which in ("x", "residual"):
        a, b = xd.clone(), rd.clone()
        out = itl.dropout_fwd(a, 0.2, SEED, residual=b, draw=1, out=a if which == "x" else b)
        assert torch.equal(out, y)
    lead = itl.dropout_fwd(xd.view(1, 13, 333), 0.2, SEED, residual=rd.view(1, 13, 333), draw=1)
    assert torch.equal(lead[0], y)


def test_infinities_and_nan_where_dropped():
    mask, factor = kept(6, 50, 0.5, SEED)
    for bad in (torch.inf, -torch.inf, torch.nan):
        x = torch.where(mask, 1.0, bad).to(dev())
        r = torch.full((6, 50), 2.0, device=dev())
        y = itl.dropout_fwd(x, 0.5, SEED, residual=r).cpu()
        assert torch.equal(y, torch.where(mask, 2.0 + factor, 2.0))
        x = torch.where(mask, bad, 1.0).to(dev())
        y = itl.dropout_fwd(x, 0.5, SEED, residual=r).cpu()
        assert torch.equal(y[~mask], torch.full_like(y[~mask], 2.0)) and not y[mask].isfinite().any()


@pytest.mark.parametrize("dtype", TYPES)
def test_gradient(dtype):
    n, h, p = 7, 99, 0.4
    x, xd = rows(n, h, dtype, 5)
    r, rd = rows(n, h, dtype, 6)
    g, gd = rows(n, h, dtype, 7)
    a, b = xd.requires_grad_(), rd.requires_grad_()
    seed = torch.tensor([SEED], device=dev())
    y = itl.dropout(a, p, seed, residual=b, draw=2)
    dx, dr = torch.autograd.grad(y, [a, b], gd)
    close(dx, dropped(g.double(), p, SEED, 2), dtype)
    assert torch.equal(dr, gd)
    # a linear map: its own transpose
    if dtype == "fp32":
        e = torch.zeros_like(x)
        e[3, 17] = 1.0
        d = itl.dropout_fwd(xd.detach() + e.to(dev()), p, SEED, draw=2) - itl.dropout_fwd(xd.detach(), p, SEED, draw=2)
        assert abs((d * gd).sum().item() - dx[3, 17].item()) <= 1e-5
    g1 = torch.tensor(0.5, dtype=TYPES[dtype], device=dev()).expand(n, h)  # broadcast
    full = torch.autograd.grad(itl.dropout(a, p, seed, draw=2), a, g1)[0]
    assert torch.equal(full, itl.dropout_bwd(g1.contiguous(), p, SEED, draw=2))


def test_seed_changed_before_the_backward():
    x = torch.randn(4, 64, device=dev(), requires_grad=True)
    seed = torch.tensor([1], device=dev())
    y = itl.dropout(x, 0.5, seed)
    seed.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_empty_and_many_short_rows():
    assert itl.dropout_fwd(torch.empty(0, 64, device=dev()), 0.5, 1).shape == (0, 64)
    x = torch.ones(70000, 3, device=dev())
    assert torch.equal(itl.dropout_fwd(x, 0.5, 1).cpu() != 0, kept(70000, 3, 0.5, 1)[0])


def test_graph_draws_anew():
    """A captured call reads its seed when it is replayed."""
    x = torch.randn(64, 512, device=dev())
    seed = torch.zeros(1, dtype=torch.int64, device=dev())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        itl.dropout_fwd(x, 0.3, seed)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = itl.dropout_fwd(x, 0.3, seed)
    for k in range(4):
        seed.fill_(SEED + k)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, itl.dropout_fwd(x, 0.3, SEED + k))


@pytest.mark.parametrize("place", [dict(draw=-1), dict(draw=2 ** 32), dict(draw=2 ** 64), dict(first_row=-1),
                                   dict(first_row=2 ** 63), dict(first_row=2 ** 64 + 1)])
def test_refused_places(place):
    """Numbers past the generator's counter, and those a 64-bit integer would wrap."""
    x = torch.ones(2, 64, device=dev())
    with pytest.raises(ValueError, match="draw must be"):
        itl.dropout(x, 0.5, SEED, **place)
    with pytest.raises(ValueError, match="draw must be"):
        itl.layer_norm(x, x[0], dropout=0.5, seed=SEED, **place)


def test_last_places():
    """The last draw, and rows past 2^32: a part of a batch is numbered as the whole."""
    x = torch.ones(4, 64, device=dev())
    y = itl.dropout_fwd(x, 0.5, SEED, draw=2 ** 32 - 1, first_row=2 ** 32 - 2)
    assert torch.equal(y.cpu(), dropped(x.cpu(), 0.5, SEED, 2 ** 32 - 1, 2 ** 32 - 2).float())
    assert torch.equal(y[2:], itl.dropout_fwd(x[2:], 0.5, SEED, draw=2 ** 32 - 1, first_row=2 ** 32))


def test_widest_rows():
    """Rows of 2^24 elements, the most: the ends are as the same columns' of the plain form."""
    h = 2 ** 24
    x = torch.ones(1, h, dtype=torch.bfloat16, device=dev())
    y = itl.dropout_fwd(x, 0.25, SEED)
    again = itl.dropout_fwd(x[:, :4096].contiguous(), 0.25, SEED)
    assert torch.equal(y[:, :4096], again) and int((y != 0).sum()) + int((y == 0).sum()) == h
    assert abs(float((y == 0).float().mean()) - 0.25) < 6 * (0.1875 / h) ** 0.5
    with pytest.raises(RuntimeError):
        itl.dropout_fwd(torch.empty(1, h + 8, dtype=torch.bfloat16, device=dev()), 0.25, SEED)


@pytest.mark.parametrize("dtype", TYPES)
def test_without_a_seed(dtype):
    """Nothing is dropped: x itself, or the sum rounded once; both gradients whole."""
    x, xd = rows(5, 77, dtype, 1)
    r, rd = rows(5, 77, dtype, 2)
    assert torch.equal(itl.dropout_fwd(xd, 0.0, None), xd) and torch.equal(itl.dropout_bwd(xd, 0, None), xd)
    a, b = xd.clone().requires_grad_(), rd.clone().requires_grad_()
    y = itl.dropout(a, 0.0, None, residual=b)
    assert torch.equal(y.cpu(), (x.float() + r.float()).to(TYPES[dtype]))
    da, db = torch.autograd.grad(y, [a, b], xd)
    assert torch.equal(da, xd) and torch.equal(db, xd)
