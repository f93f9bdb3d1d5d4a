"""The residual root-mean-square norm, its 8-bit form and its gradient against
the plain float64 forms.

Tolerances.  The stored sum is one fp32 addition rounded to its type: equal to
torch's.  y: the sum of squares of h terms, a square root, a division and two
products are off by at most (h / 512 + 24) 2^-24 relative (each thread adds at
most h / 64 / 8 * 8 terms in turn, twelve more additions join them, and their
roundings are not aligned), taken as 2e-6 + h 2^-33; the output rounds by eps /
2.  dx = ds + rstd (a - u c): each term carries that and the mean's own error,
taken as 1e-5 of |ds| + rstd (|a| + |u| mean|a u|), then eps / 2.  dweight: n
terms in fp32, (n + 64) 2^-24 of sum |dy u| at most, plus 1e-5 of it, then eps /
2.  8 bits: the value before rounding is within 4e-6 of the exact one, so q lies
between the roundings of the two ends; the scale within 4e-6."""

import pytest
import torch

import invariant_token_log_amd as itl
from gpu_helpers import dev
from token_reference import norm_forward, norm_gradient

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6
# one element, fewer than a chunk, odd, one team of each width and both sides
# of its end, several chunks a thread
LENGTHS = [1, 7, 64, 100, 1021, 1024, 1032, 2048, 4096, 5120, 8185, 8192, 8200, 20000, 65536]


def make(n, h, dtype, seed, residual=True, pad=0):
    gen = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]

    def rows(scale):
        x = (scale * torch.randn(n, h, generator=gen)).to(t)
        buf = torch.zeros(n, h + pad, dtype=t, device=dev())[:, :h]
        buf.copy_(x)
        return x, buf

    x, xd = rows(1.0)
    r, rd = rows(3.0) if residual else (None, None)
    w = (1 + 0.1 * torch.randn(h, generator=gen)).to(t)
    return x, xd, r, rd, w


def within(a, ref, bound, dtype):
    t = TYPES[dtype]
    half = torch.finfo(t).eps / 2
    sub = 2.0 ** -25 if t == torch.float16 else 0.0
    a = a.detach().double().cpu()
    bad = ~((a - ref).abs() <= bound + half * (ref.abs() + bound) + sub)
    assert not bad.any(), (bad.nonzero()[:4], a[bad][:4], ref[bad][:4])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("h", LENGTHS)
def test_forward(h, dtype):
    n = 5 if h > 4096 else 9
    for residual, pad in ((True, 0), (False, 0), (True, 3)):
        x, xd, r, rd, w = make(n, h, dtype, seed=h, residual=residual, pad=pad)
        y, s, rstd = itl.rms_norm_fwd(xd, w.to(dev()), residual=rd, eps=EPS, return_rstd=True)
        want = x if r is None else (x.float() + r.float()).to(TYPES[dtype])
        assert torch.equal(s.cpu(), want)
        ref, rs = norm_forward(want, w, EPS)
        rel = 2e-6 + h * 2.0 ** -33
        assert ((rstd.double().cpu() - rs[:, 0]).abs() <= rel * rs[:, 0]).all()
        within(y, ref, rel * ref.abs(), dtype)
        # the fused call has the bits of an addition and a norm
        y2, _, _ = itl.rms_norm_fwd(s.contiguous(), w.to(dev()), eps=EPS)
        assert torch.equal(y2, y)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("h", [1, 100, 1024, 4096, 5121, 20000])
def test_rows_alone_strided_and_in_place(h, dtype):
    x, xd, r, rd, w = make(11, h, dtype, seed=3)
    wd = w.to(dev())
    y, s, _ = itl.rms_norm_fwd(xd, wd, residual=rd, eps=EPS)
    one, s1, _ = itl.rms_norm_fwd(xd[4:5], wd, residual=rd[4:5], eps=EPS)
    assert torch.equal(one, y[4:5]) and torch.equal(s1, s[4:5])
    _, xp, _, rp, _ = make(11, h, dtype, seed=3, pad=5)
    yp, sp, _ = itl.rms_norm_fwd(xp, wd, residual=rp, eps=EPS)
    assert torch.equal(yp, y) and torch.equal(sp, s)
    xi, ri = xd.clone(), rd.clone()
    yi, si, _ = itl.rms_norm_fwd(xi, wd, residual=ri, eps=EPS, sum_out=ri, y_out=xi)
    assert torch.equal(yi, y) and torch.equal(si, s) and si.data_ptr() == ri.data_ptr()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,h", [(1, 1), (3, 100), (70, 1021), (2, 1024), (5, 2048), (1500, 4096),
                                 (4100, 64), (3, 8192), (3, 20000), (2, 65536)])
def test_gradient(n, h, dtype):
    gen = torch.Generator().manual_seed(n + h)
    x, xd, _, _, w = make(n, h, dtype, seed=h, residual=False)
    dy = torch.randn(n, h, generator=gen).to(TYPES[dtype])
    ds = torch.randn(n, h, generator=gen).to(TYPES[dtype])
    _, _, rstd = itl.rms_norm_fwd(xd, w.to(dev()), eps=EPS, return_rstd=True)
    for with_ds in (True, False):
        dx, dw = itl.rms_norm_bwd(xd, w.to(dev()), rstd, dy.to(dev()), ds.to(dev()) if with_ds else None)
        rx, rw = norm_gradient(x, w, dy, ds if with_ds else None, EPS)
        _, rs = norm_forward(x, w, EPS)
        a, u = (dy.double() * w.double()).abs(), (x.double() * rs).abs()
        size = rs * (a + u * (a * u).mean(1, keepdim=True)) + (ds.double().abs() if with_ds else 0.0)
        within(dx, rx, (1e-5 + h * 2.0 ** -33) * size, dtype)
        total = (dy.double() * x.double() * rs).abs().sum(0)
        within(dw, rw, (1e-5 + (n + 64) * 2.0 ** -24) * total, dtype)
        again = itl.rms_norm_bwd(xd, w.to(dev()), rstd, dy.to(dev()), ds.to(dev()) if with_ds else None)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)  # a fixed order
    # in place over either gradient; without the weight's
    g = dy.to(dev())
    dx2, none = itl.rms_norm_bwd(xd, w.to(dev()), rstd, g, need_dweight=False, dx_out=g)
    assert none is None and torch.equal(dx2, dx)


def test_autograd_and_differences():
    n, h = 4, 96
    x, xd, r, rd, w = make(n, h, "fp32", seed=2)
    gen = torch.Generator().manual_seed(4)
    gy, gs = torch.randn(n, h, generator=gen), torch.randn(n, h, generator=gen)
    leaves = [t.clone().requires_grad_() for t in (xd, rd, w.to(dev()))]
    y, s = itl.rms_norm(leaves[0], leaves[2], residual=leaves[1], eps=EPS)
    ((y * gy.to(dev())).sum() + (s * gs.to(dev())).sum()).backward()
    assert torch.equal(leaves[0].grad, leaves[1].grad)

    def objective(a, b):
        return float((norm_forward(a + r.double(), b, EPS)[0] * gy).sum() + ((a + r.double()) * gs).sum())

    step = 1e-5
    for i in range(4):
        u, v = torch.randn(n, h, generator=gen).double(), torch.randn(h, generator=gen).double()
        xx, ww = x.double(), w.double()
        want = (objective(xx + step * u, ww) - objective(xx - step * u, ww)) / (2 * step)
        got = (leaves[0].grad.double().cpu() * u)
        assert abs(want - float(got.sum())) <= 1e-5 * float(got.abs().sum()) + 1e-6
        want = (objective(xx, ww + step * v) - objective(xx, ww - step * v)) / (2 * step)
        got = (leaves[2].grad.double().cpu() * v)
        assert abs(want - float(got.sum())) <= 1e-5 * float(got.abs().sum()) + 1e-6
    # only one of the outputs used; broadcast gradients
    for use in (0, 1):
        a = xd.clone().requires_grad_()
        itl.rms_norm(a, leaves[2], residual=rd, eps=EPS)[use].sum().backward()
        assert torch.isfinite(a.grad).all()
    a = xd.view(2, 2, h).clone().requires_grad_()
    itl.rms_norm(a, w.to(dev())).sum().backward()
    assert a.grad.shape == (2, 2, h)


def test_broadcast_gradients():
    """A gradient that is one row or one value for all rows (an expanded
    tensor), for y and for the stored sum."""
    x, xd, r, rd, w = make(6, 80, "fp32", seed=9)
    g = torch.randn(80, generator=torch.Generator().manual_seed(2)).to(dev())
    wd = w.to(dev())

    def grads(gy, gs):
        a = xd.clone().requires_grad_()
        y, s = itl.rms_norm(a, wd, residual=rd, eps=EPS)
        torch.autograd.backward([y, s], [gy, gs])
        return a.grad

    full = grads(g.expand(6, 80).contiguous(), torch.full((6, 80), 0.5, device=dev()))
    assert torch.equal(grads(g.expand(6, 80), torch.tensor(0.5, device=dev()).expand(6, 80)), full)


def e4m3(d):
    return d.clamp(-448.0, 448.0).float().to(torch.float8_e4m3fn).double()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("h", [1, 7, 100, 1024, 4096, 5121, 20000])
def test_quantized(h, dtype):
    n = 6
    x, xd, r, rd, w = make(n, h, dtype, seed=h)
    for mode in ("residual", "plain", "rows"):
        if mode == "rows":
            q, t = itl.quantize_rows(xd), x.double()
        else:
            q, s = itl.rms_norm_quantized(xd, w.to(dev()), residual=rd if mode == "residual" else None,
                                          eps=EPS)
            want = (x.float() + r.float()).to(TYPES[dtype]) if mode == "residual" else x
            assert torch.equal(s.cpu(), want)
            t, _ = norm_forward(want, w, EPS)
        rel = 4e-6 + h * 2.0 ** -33
        scale = t.abs().amax(1) / 448.0
        assert ((q.scale.double().cpu() - scale).abs() <= rel * scale).all()
        v, got = t / scale[:, None], q.data.cpu().double()
        ends = e4m3(v * (1 - rel)), e4m3(v * (1 + rel))
        assert ((got >= torch.minimum(*ends)) & (got <= torch.maximum(*ends))).all()


def test_quantized_edges():
    """A row of zeros, one with an infinity, one with a NaN, one of the type's
    largest values; the rows next to them keep their values."""
    x = torch.randn(5, 300, generator=torch.Generator().manual_seed(0))
    x[1] = 0.0
    x[2, 7] = torch.inf
    x[3, 9] = torch.nan
    x[4] = torch.finfo(torch.float32).max / 2
    q = itl.quantize_rows(x.to(dev()))
    val = q.data.float() * q.scale[:, None]
    assert torch.equal(val[1], torch.zeros(300, device=dev())) and q.scale[1] == 0
    assert val[2].isnan().all() and val[3].isnan().all()
    assert torch.isfinite(val[0]).all() and torch.equal(q.data[4].float(), torch.full((300,), 448.0, device=dev()))
    y, _, _ = itl.rms_norm_fwd(x.to(dev())[:2], torch.ones(300, device=dev()), eps=EPS)
    assert (y[1] == 0).all()


def test_quantized_tiny_rows():
    """Rows whose 448 / max|t| would pass fp32's range: the scale stays at
    2^-126.  Half a step of e4m3 is 2^-4 of the value, 2^-10 below 2^-6; the
    fp32 factor and product move a value by less than 2^-20 of itself."""
    x = torch.randn(5, 300, generator=torch.Generator().manual_seed(1))
    x = x * torch.tensor([1e-30, 1e-36, 1e-37, 1e-38, 1e-41])[:, None]
    x[:, 5] = 0.0
    q = itl.quantize_rows(x.to(dev()))
    scale = x.double().abs().amax(1).clamp(min=448 * 2.0 ** -126) / 448
    assert ((q.scale.double().cpu() - scale).abs() <= 2.0 ** -23 * scale).all()
    val = q.data.double().cpu() * q.scale.double().cpu()[:, None]
    bound = x.double().abs() * (2.0 ** -4 + 2.0 ** -20) + scale[:, None] * 2.0 ** -10 * (1 + 2.0 ** -20)
    assert ((val - x.double()).abs() <= bound).all()


def test_empty_batch():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=dev())
    w = torch.ones(64, dtype=torch.bfloat16, device=dev())
    y, s, rstd = itl.rms_norm_fwd(x, w, residual=x, return_rstd=True)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    dx, dw = itl.rms_norm_bwd(x, w, rstd, x)
    assert dx.shape == (0, 64) and (dw == 0).all()
    assert itl.quantize_rows(x).data.shape == (0, 64)
