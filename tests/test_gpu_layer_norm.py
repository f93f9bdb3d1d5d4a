"""The layer norm with dropout and the residual's addition, and its gradient,
against the plain float64 forms.

Tolerances.  The stored sum is one fp32 operation rounded to its type: without
dropout equal to torch's, with it equal to dropout_fwd's.  A sum of h terms joins
chains of at most h / 256 + 16 terms with 22 more additions: k = (h / 256 + 40)
2^-24 of the sum of magnitudes.  So the mean is off by dm = k mean|s| + 2^-24
|m|, the variance relatively by k + 2^-22 + dm^2 / (var + eps), rstd by half of
that and 2^-22, and u = (s - m) rstd by du = |u| (k / 2 + 2^-21 + dm^2 / (var +
eps)) + dm rstd.  y = u w + b: |w| du + 2^-23 (|u w| + |b|), then eps / 2.  d = ds +
rstd (g - mean g - u mean(g u)): 2 k + 2^-20 of the magnitudes' sum, and du where u
stands.  dweight: (n + 64) 2^-24 + 2^-22 of sum |dy u| and sum |dy| du; dbias: (n +
64) 2^-24 of sum |dy|; each then rounds by eps / 2 (fp16 subnormals: 2^-25)."""

import pytest
import torch

import invariant_token_log_amd as itl
from gpu_helpers import dev
from layer_reference import TYPES, dropped, kept, layer_norm, layer_norm_gradient

pytestmark = pytest.mark.gpu

EPS, SEED = 1e-5, 0x7F4A7C159E3779B9
# one element, fewer than a chunk, odd, both sides of each team's end, the rows
# that are read again
LENGTHS = [1, 7, 64, 100, 1021, 1024, 1032, 2048, 4096, 5120, 8185, 8192, 8200, 12296, 16385, 20000, 32776, 65536]


def rows(n, h, dtype, seed, scale=1.0, mean=0.0, pad=0):
    gen = torch.Generator().manual_seed(seed)
    x = (mean + scale * torch.randn(n, h, generator=gen)).to(TYPES[dtype])
    buf = torch.zeros(n, h + pad, dtype=x.dtype, device=dev())[:, :h]
    buf.copy_(x)
    return x, buf


def weights(h, dtype):
    gen = torch.Generator().manual_seed(h + 9)
    w, b = 1 + 0.1 * torch.randn(h, generator=gen), 0.3 * torch.randn(h, generator=gen)
    return w.to(TYPES[dtype]), b.to(TYPES[dtype])


def within(a, ref, bound, dtype):
    half = torch.finfo(TYPES[dtype]).eps / 2
    sub = 2.0 ** -25 if dtype == "fp16" else 0.0
    a = a.detach().double().cpu()
    bad = ~((a - ref).abs() <= bound + half * (ref.abs() + bound) + sub)
    assert not bad.any(), (bad.nonzero()[:4], a[bad][:4], ref[bad][:4])


def unit_error(s, eps=EPS):
    """(k, dm, rel rstd, u, du, rstd) of the docstring."""
    h = s.shape[1]
    s = s.double()
    k = (h / 256 + 40) * 2.0 ** -24
    m = s.mean(1, keepdim=True)
    var = ((s - m) ** 2).mean(1, keepdim=True) + eps
    rs = var ** -0.5
    dm = k * s.abs().mean(1, keepdim=True) + 2.0 ** -24 * m.abs()
    u = (s - m) * rs
    rel = k / 2 + 2.0 ** -21 + dm ** 2 / var
    return k, dm, rel, u, u.abs() * rel + dm * rs, rs


def check_forward(y, mean, rstd, s, w, b, dtype):
    ref, m, rs = layer_norm(s, w, b, EPS)
    k, dm, rel, u, du, _ = unit_error(s)
    wd = w.double().abs()
    within(y, ref, wd * du + 2.0 ** -23 * ((u * wd).abs() + (b.double().abs() if b is not None else 0.0)), dtype)
    assert ((mean.double().cpu() - m[:, 0]).abs() <= dm[:, 0] + 1e-40).all()
    assert ((rstd.double().cpu() - rs[:, 0]).abs() <= rel[:, 0] * rs[:, 0]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("h", LENGTHS)
def test_forward(h, dtype):
    n = 5 if h > 4096 else 9
    w, b = weights(h, dtype)
    wd, bd = w.to(dev()), b.to(dev())
    for residual, p, bias, pad in ((True, 0.0, True, 0), (False, 0.0, False, 0), (True, 0.2, True, 0),
                                   (False, 0.2, False, 0), (True, 0.2, True, 3)):
        x, xd = rows(n, h, dtype, h, pad=pad)
        r, rd = rows(n, h, dtype, h + 1, 3.0, 0.5, pad) if residual else (None, None)
        y, s, mean, rstd = itl.layer_norm_fwd(xd, wd, bd if bias else None, residual=rd, eps=EPS, dropout=p, seed=SEED,
                                              draw=4, return_stats=True)
        if p:
            assert torch.equal(s, itl.dropout_fwd(xd, p, SEED, residual=rd, draw=4))
        else:
            assert torch.equal(s.cpu(), x if r is None else (x.float() + r.float()).to(TYPES[dtype]))
        check_forward(y, mean, rstd, s.cpu(), w, b if bias else None, dtype)
        # the fused call has the bits of the addition and a norm
        y2, _, _, _ = itl.layer_norm_fwd(s.contiguous(), wd, bd if bias else None, eps=EPS)
        assert torch.equal(y2, y)


@pytest.mark.parametrize("h", [64, 1021, 4096, 20000, 65536])
def test_far_from_zero(h):
    """A mean of a thousand standard deviations, and a row of one value."""
    x, xd = rows(4, h, "fp32", h, 1.0, 1000.0)
    xd[1] = x[1] = 7.25
    w, b = weights(h, "fp32")
    y, s, mean, rstd = itl.layer_norm_fwd(xd, w.to(dev()), b.to(dev()), eps=EPS, return_stats=True)
    check_forward(y, mean, rstd, x, w, b, "fp32")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("h", [1, 100, 1024, 4096, 5121, 20000, 40000])
def test_rows_alone_strided_and_in_place(h, dtype):
    x, xd = rows(11, h, dtype, 3)
    r, rd = rows(11, h, dtype, 4, 3.0)
    w, b = (t.to(dev()) for t in weights(h, dtype))
    for p in (0.0, 0.3):
        def run(a, c, first=0, **out):
            return itl.layer_norm_fwd(a, w, b, residual=c, eps=EPS, dropout=p, seed=SEED, first_row=first, **out)[:2]

        y, s = run(xd, rd)
        one, s1 = run(xd[4:5], rd[4:5], 4)
        assert torch.equal(one, y[4:5]) and torch.equal(s1, s[4:5])
        _, xp = rows(11, h, dtype, 3, pad=5)
        yp, sp = run(xp, rd)
        assert torch.equal(yp, y) and torch.equal(sp, s)
        a, c = xd.clone(), rd.clone()
        yi, si = run(a, c, sum_out=c, y_out=a)
        assert torch.equal(yi, y) and torch.equal(si, s) and si.data_ptr() == c.data_ptr()
        a, c = xd.clone(), rd.clone()
        yi, si = run(a, c, sum_out=a)
        assert torch.equal(yi, y) and torch.equal(si, s)
    a = xd.clone()
    y, _, _, _ = itl.layer_norm_fwd(xd, w, b, eps=EPS)
    assert torch.equal(itl.layer_norm_fwd(a, w, b, eps=EPS, y_out=a)[0], y)


def check_gradient(got, s, w, dy, ds, dtype, p=0.0, draw=0):
    dx, dres, dw, db = got
    n = s.shape[0]
    ref, rw, rb = layer_norm_gradient(s, w, dy, ds, EPS)
    k, dm, rel, u, du, rs = unit_error(s)
    g = (dy.double() * w.double()).abs()
    mean = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    size = g + mean(g) + u.abs() * mean(g * u.abs())
    bound = rs * ((2 * k + 2.0 ** -20 + rel) * size + du * mean(g * u.abs()) + u.abs() * mean(g * du))
    bound = bound + (2.0 ** -22 * ds.double().abs() if ds is not None else 0.0)
    if dres is not None:
        within(dres, ref, bound, dtype)
    if p:
        mask, factor = kept(*s.shape, p, SEED, draw)
        ref, bound = torch.where(mask, ref * factor, 0.0), torch.where(mask, bound * factor + 2.0 ** -23 * ref.abs(), 0.0)
    within(dx, ref, bound, dtype)
    dyd = dy.double().abs()
    if dw is not None:
        within(dw, rw, ((n + 64) * 2.0 ** -24 + 2.0 ** -22) * (dyd * u.abs()).sum(0) + (dyd * du).sum(0), dtype)
    if db is not None:
        within(db, rb, (n + 64) * 2.0 ** -24 * dyd.sum(0), dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,h", [(1, 1), (3, 100), (70, 1021), (2, 1024), (5, 2048), (1500, 4096), (4100, 64), (3, 8192),
                                 (3, 12280), (300, 12296), (3, 20000), (2, 65536)])
def test_gradient(n, h, dtype):
    s, sd = rows(n, h, dtype, h, 1.5, 0.3)
    dy, dyd = rows(n, h, dtype, h + 1)
    ds, dsd = rows(n, h, dtype, h + 2)
    w, b = weights(h, dtype)
    wd = w.to(dev())
    _, _, mean, rstd = itl.layer_norm_fwd(sd, wd, eps=EPS, return_stats=True)
    for with_ds, p in ((True, 0.0), (False, 0.0), (True, 0.3), (False, 0.3)):
        def run(g, d, **kw):
            return itl.layer_norm_bwd(sd, wd, mean, rstd, g, d if with_ds else None, dropout=p, seed=SEED, draw=6, **kw)

        got = run(dyd, dsd)
        check_gradient(got, s, w, dy, ds if with_ds else None, dtype, p, 6)
        if not p:
            assert got[1] is got[0]
        assert all(torch.equal(a, c) for a, c in zip(run(dyd, dsd), got))  # a fixed order
        # in place over both gradients; parts that are not asked for
        g2, d2 = dyd.clone(), dsd.clone()
        kw = dict(dx_out=g2, dresidual_out=d2) if p and with_ds else dict(dx_out=g2)
        again = run(g2, d2, **kw)
        assert all(torch.equal(a, c) for a, c in zip(again, got))
        part = run(dyd, dsd, need_dweight=False, need_dresidual=False)
        assert part[1] is None and part[2] is None and torch.equal(part[0], got[0]) and torch.equal(part[3], got[3])
        part = run(dyd, dsd, need_dweight=False, need_dbias=False)
        assert part[2] is None and part[3] is None and torch.equal(part[0], got[0])


@pytest.mark.parametrize("h", [100, 1021, 4096, 8200, 20000])
def test_gradient_strided_and_alone(h):
    s, sd = rows(6, h, "bf16", 1, pad=7)
    dy, dyd = rows(6, h, "bf16", 2, pad=3)
    ds, dsd = rows(6, h, "bf16", 3, pad=1)
    w = weights(h, "bf16")[0].to(dev())
    _, _, mean, rstd = itl.layer_norm_fwd(sd, w, return_stats=True)
    want = itl.layer_norm_bwd(sd.contiguous(), w, mean, rstd, dyd.contiguous(), dsd.contiguous(), dropout=0.2, seed=SEED)
    wide = torch.full((6, h + 5), 9.0, dtype=torch.bfloat16, device=dev())
    got = itl.layer_norm_bwd(sd, w, mean, rstd, dyd, dsd, dropout=0.2, seed=SEED, dx_out=wide[:, :h])
    assert all(torch.equal(a, c) for a, c in zip(got, want)) and (wide[:, h:] == 9).all()
    one = itl.layer_norm_bwd(sd[2:3], w, mean[2:3], rstd[2:3], dyd[2:3], dsd[2:3], dropout=0.2, seed=SEED, first_row=2)
    assert torch.equal(one[0], want[0][2:3]) and torch.equal(one[1], want[1][2:3])


@pytest.mark.parametrize("p", [0.0, 0.3])
def test_autograd_and_differences(p):
    n, h = 4, 96
    x, xd = rows(n, h, "fp32", 2)
    r, rd = rows(n, h, "fp32", 3, 2.0)
    gy, gyd = rows(n, h, "fp32", 4)
    gs, gsd = rows(n, h, "fp32", 5)
    w, b = weights(h, "fp32")
    leaves = [t.to(dev()).requires_grad_() for t in (x, r, w, b)]
    seed = torch.tensor([SEED], device=dev())
    y, s = itl.layer_norm(leaves[0], leaves[2], leaves[3], residual=leaves[1], eps=EPS, dropout=p, seed=seed, draw=1)
    grads = torch.autograd.grad([y, s], leaves, [gyd, gsd])

    def loss(a, c, ww, bb):
        t = (dropped(a, p, SEED, 1) if p else a) + c
        return (layer_norm(t, ww, bb, EPS)[0] * gy.double()).sum() + (t * gs.double()).sum()

    base = [t.double() for t in (x, r, w, b)]
    gen = torch.Generator().manual_seed(8)
    for i, g in enumerate(grads):
        for _ in range(3):
            d = torch.randn(base[i].shape, generator=gen, dtype=torch.float64)
            step = 1e-5
            up, down = ([t + (sgn * step * d if j == i else 0) for j, t in enumerate(base)] for sgn in (1, -1))
            slope = (loss(*up) - loss(*down)) / (2 * step)
            size = (g.double().cpu() * d).abs().sum()
            assert abs((g.double().cpu() * d).sum() - slope) <= 1e-5 * size + 1e-6


def test_partial_use():
    """Only one output used, no residual, no bias, leaves without gradients."""
    x, xd = rows(5, 72, "bf16", 1)
    r, rd = rows(5, 72, "bf16", 2)
    w, b = (t.to(dev()) for t in weights(72, "bf16"))
    g = torch.randn(5, 72, device=dev()).bfloat16()
    a, c, ww, bb = (t.clone().requires_grad_() for t in (xd, rd, w, b))
    y, s = itl.layer_norm(a, ww, bb, residual=c, dropout=0.4, seed=SEED)
    da, dc, dw, db = torch.autograd.grad(s, [a, c, ww, bb], g)
    assert torch.equal(da, itl.dropout_bwd(g, 0.4, SEED)) and torch.equal(dc, g) and not dw.any() and not db.any()
    y, s = itl.layer_norm(a, ww, bb, residual=c, dropout=0.4, seed=SEED)
    only = torch.autograd.grad(y, [a, c, ww, bb], g)
    _, sd, mean, rstd = itl.layer_norm_fwd(xd, w, b, residual=rd, dropout=0.4, seed=SEED, return_stats=True)
    want = itl.layer_norm_bwd(sd, w, mean, rstd, g, dropout=0.4, seed=SEED)
    assert all(torch.equal(p, q) for p, q in zip(only, want))
    y = itl.layer_norm(a, w)
    da, = torch.autograd.grad(y, a, g)
    _, _, mean, rstd = itl.layer_norm_fwd(xd, w, return_stats=True)
    assert torch.equal(da, itl.layer_norm_bwd(xd, w, mean, rstd, g)[0])
    y = itl.layer_norm(xd, ww, bb, dropout=0.4, seed=SEED)
    dw, db = torch.autograd.grad(y, [ww, bb], g.float().sum().bfloat16().expand(5, 72))
    assert dw.shape == (72,) and db.shape == (72,)


@pytest.mark.parametrize("dtype", TYPES)
def test_infinities_and_nan_stay_in_their_row(dtype):
    x, xd = rows(6, 300, dtype, 1)
    w, b = (t.to(dev()) for t in weights(300, dtype))
    y, _, _, _ = itl.layer_norm_fwd(xd, w, b)
    xd[1, 7], xd[3, 9] = torch.inf, torch.nan
    z, _, _, _ = itl.layer_norm_fwd(xd, w, b)
    assert z[1].isnan().all() and z[3].isnan().all()
    assert torch.equal(z[[0, 2, 4, 5]], y[[0, 2, 4, 5]])


def test_empty_batch():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=dev())
    w = torch.ones(64, dtype=torch.bfloat16, device=dev())
    y, s, mean, rstd = itl.layer_norm_fwd(x, w, w, residual=x, dropout=0.1, seed=1, return_stats=True)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    dx, dr, dw, db = itl.layer_norm_bwd(x, w, mean, rstd, x, dropout=0.1, seed=1)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()


def test_graph_replays():
    """Forward and backward captured, replayed with new inputs and seeds between
    eager calls."""
    n, h = 96, 2048
    x, r, dy = (torch.randn(n, h, device=dev()).bfloat16() for _ in range(3))
    w, b = (t.to(dev()) for t in weights(h, "bf16"))
    seed = torch.zeros(1, dtype=torch.int64, device=dev())

    def step(sd):
        y, s, mean, rstd = itl.layer_norm_fwd(x, w, b, residual=r, dropout=0.2, seed=sd, return_stats=True)
        return (y, s, *itl.layer_norm_bwd(s, w, mean, rstd, dy, dropout=0.2, seed=sd))

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step(seed)
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(seed)
    for k in range(4):
        for t in (x, r, dy):
            t.copy_(torch.randn(n, h, device=dev()))
        seed.fill_(SEED + k)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(out, step(SEED + k)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("h", [6144, 6145, 24576, 24577, 32761, 32768])
def test_forward_at_more_ends_of_the_teams(h, dtype):
    """Chunks a thread on both sides of three and four; the longest rows in registers."""
    test_forward(h, dtype)


# Rows of every team and chunk count of the gradient, whole chunks and not, more than twice
# as many as there are teams (1024 of 64 threads, 512 or 256 of the others; 102 to 73 groups of
# rows where they are read again, past 8192 elements in fp32 and 12288): a team walks two or
# three rows, the next one's loads ahead.
SEVERAL = [(2100, 505), (2100, 512), (2100, 1021), (2100, 1024), (1100, 2045), (1100, 2048), (1100, 4093), (1100, 4096),
           (600, 5117), (600, 5120), (600, 8185), (600, 8192), (600, 8200), (600, 12281), (600, 12288), (160, 12297)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,h", SEVERAL)
def test_gradient_of_several_rows_a_team(n, h, dtype):
    s, sd = rows(n, h, dtype, h, 1.5, 0.3)
    dy, dyd = rows(n, h, dtype, h + 1)
    ds, dsd = rows(n, h, dtype, h + 2)
    w = weights(h, dtype)[0]
    wd = w.to(dev())
    _, _, mean, rstd = itl.layer_norm_fwd(sd, wd, eps=EPS, return_stats=True)

    def run(g, d, p, **kw):
        return itl.layer_norm_bwd(sd, wd, mean, rstd, g, d, dropout=p, seed=SEED, draw=6, **kw)

    got = run(dyd, dsd, 0.3)
    check_gradient(got, s, w, dy, ds, dtype, 0.3, 6)
    assert all(torch.equal(a, c) for a, c in zip(run(dyd, dsd, 0.3), got))
    g2, d2 = dyd.clone(), dsd.clone()
    assert all(torch.equal(a, c) for a, c in zip(run(g2, d2, 0.3, dx_out=g2, dresidual_out=d2), got))
    # without dropout: dx is what dresidual is with it; the sums over the rows are the same
    plain = run(dyd, dsd, 0.0)
    assert torch.equal(plain[0], got[1]) and torch.equal(plain[2], got[2]) and torch.equal(plain[3], got[3])
    # a row alone, the last and one in the middle
    for r in (n // 2 + 1, n - 1):
        one = itl.layer_norm_bwd(sd[r:r + 1], wd, mean[r:r + 1], rstd[r:r + 1], dyd[r:r + 1], dsd[r:r + 1], dropout=0.3,
                                 seed=SEED, draw=6, first_row=r)
        assert torch.equal(one[0], got[0][r:r + 1]) and torch.equal(one[1], got[1][r:r + 1])
    # nothing but y was used
    only = run(dyd, None, 0.0)
    check_gradient((only[0][-4:], None, None, None), s[-4:], w, dy[-4:], None, dtype)
    assert torch.equal(only[2], got[2]) and torch.equal(only[3], got[3])
