"""Several given tokens a row, entropy and alternatives from logits, and their
gradient, against the plain float64 forms.

Tolerances.  logp, lse and the alternatives' logp: the bound of the logp path
(gpu_helpers).  Entropy: that and 1e-6 of the row's spread, as for logp_fwd.
Gradients: a term g or g p of size |t| carries the forward's lse tolerance
through exp (1e-5 + 1e-5 |x - lse|) and at most M + k + 8 roundings of
2^-24, so the fp32 value is within (4e-5 + 1e-5 |x - lse|) sum|t| of the exact
one for M + k <= 320 (320 * 2^-24 = 1.9e-5); the output then rounds once, by at
most eps / 2 of its type."""

import itertools

import pytest
import torch

import invariant_token_log_amd as itl
from gpu_helpers import ATOL, RTOL, bits, dev
from token_reference import ranked, token_gradient, token_scores

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
WIDTH = {"bf16": 512, "fp16": 512, "fp32": 256}


def make(n, v, m, dtype, seed, ld=None, offset=0, drop=0.2):
    gen = torch.Generator().manual_seed(seed)
    x = (3 * torch.randn(n, v, generator=gen)).to(TYPES[dtype])
    ld = ld or v
    buf = torch.full((n * ld + offset + 16,), 77.0, dtype=TYPES[dtype], device=dev())
    view = buf[offset:offset + n * ld].view(n, ld)[:, :v]
    view.copy_(x)
    tok = torch.randint(0, v, (n, m), generator=gen)
    tok[torch.rand(n, m, generator=gen) < drop] = -100
    return x, view, tok


def close(a, ref, what, extra=0.0):
    a = a.detach().double().cpu()
    same = torch.isfinite(ref)
    assert torch.equal(torch.isnan(a), torch.isnan(ref)), what
    assert torch.equal(a[~same & ~torch.isnan(ref)], ref[~same & ~torch.isnan(ref)]), what
    err = (a - ref).abs()
    bound = ATOL + RTOL * ref.abs() + extra
    bad = same & ~(err <= bound)
    assert not bad.any(), (what, err[bad][:5], ref[bad][:5])


def check_forward(x, r, tok, k):
    ref = token_scores(x.double(), tok, k)
    close(r.logp, ref["logp"], "logp")
    close(r.lse, ref["lse"], "lse")
    if r.entropy is not None:
        fin = torch.where(torch.isfinite(x), x.double(), 0.0)
        close(r.entropy, ref["entropy"], "entropy", 1e-6 * (fin.amax(1) - fin.amin(1)))
    assert torch.equal(r.top_ids.cpu(), ref["top_ids"])
    close(r.top_logp, ref["top_logp"], "top_logp")
    return ref


# sizes: one column, fewer columns than lanes, one group and its neighbours, odd
# rows (no 16-byte alignment), a tile's end inside the row, many tiles
SIZES = [(1, 1, 1, 1), (3, 5, 2, 5), (4, 63, 1, 7), (2, 64, 0, 64), (5, 127, 3, 1), (3, 129, 1, 64),
         (2, 511, 256, 3), (3, 512, 1, 20), (7, 1000, 5, 33), (4, 4097, 2, 64), (2, 40001, 1, 20),
         (1, 151936, 1, 5)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,m,k", SIZES)
def test_forward(n, v, m, k, dtype):
    for width in (WIDTH[dtype], 4096):
        x, view, tok = make(n, v, m, dtype, seed=n * v + m)
        r = itl.token_logp_fwd(view, tok.to(dev()) if m else None, top_k=k, return_entropy=True,
                               tile_width=width)
        check_forward(x, r, tok, k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("ld,offset", [(1005, 0), (1008, 8), (1016, 3), (1001, 1)])
def test_strides_and_alignment(ld, offset, dtype):
    """Row strides and starts other than 16-byte multiples: the values, and the
    bits of the packed rows."""
    x, view, tok = make(6, 1000, 3, dtype, seed=5, ld=ld, offset=offset)
    r = itl.token_logp_fwd(view, tok.to(dev()), top_k=9, return_entropy=True)
    check_forward(x, r, tok, 9)
    q = itl.token_logp_fwd(x.to(dev()), tok.to(dev()).int(), top_k=9, return_entropy=True)
    for a, b in zip(r, q):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,v,width", [("bf16", 151936, 4096), ("fp16", 5000, 512), ("fp32", 30000, 2048)])
def test_same_bits_as_logp_fwd(dtype, v, width):
    x, view, tok = make(9, v, 1, dtype, seed=3)
    t = tok.to(dev())
    logp, lse, ent = itl.logp_fwd(view, t[:, 0], tile_width=width, return_entropy=True)
    for k in (0, 20):
        r = itl.token_logp_fwd(view, t, top_k=k, return_entropy=True, tile_width=width)
        assert torch.equal(bits(r.logp[:, 0]), bits(logp))
        assert torch.equal(bits(r.lse), bits(lse))
        assert torch.equal(bits(r.entropy), bits(ent))


@pytest.mark.parametrize("dtype", TYPES)
def test_ties_and_masks(dtype):
    """Constant rows, two plateaus, a single live column, nothing live, -0
    against +0, an infinite logit and a NaN: which alternatives come out and in
    which order."""
    v, k = 1500, 64
    x = torch.randn(8, v, generator=torch.Generator().manual_seed(1)).to(TYPES[dtype]).float()
    x[0] = 2.5
    x[1] = -1.0
    x[1, 700:900] = 3.0
    x[2] = -torch.inf
    x[2, 1234] = 0.5
    x[3] = -torch.inf
    x[4] = 0.0
    x[4, ::3] = -0.0
    x[5, 77] = torch.nan
    x[6] = torch.finfo(TYPES[dtype]).min
    x[6, 5] = 0.0
    x[7, 3] = torch.inf
    x = x.to(TYPES[dtype])
    r = itl.token_logp_fwd(x.to(dev()), None, top_k=k)
    ids = ranked(x, k)
    keep = [0, 1, 2, 3, 4, 6]
    assert torch.equal(r.top_ids.cpu()[keep], ids[keep])
    lse = torch.logsumexp(x.double(), 1)
    close(r.lse[[0, 1, 2, 4, 6]], lse[[0, 1, 2, 4, 6]], "lse")
    top = x.double().gather(1, ids) - lse[:, None]
    for row in (0, 1, 2, 4, 6):
        close(r.top_logp[row], top[row], row)
    assert r.top_logp[3].isnan().all() and r.top_logp[5].isnan().all()  # nothing live; a NaN
    assert ((r.top_ids >= 0) & (r.top_ids < v)).all()
    assert r.top_ids[7, 0].item() == 3


def test_many_equal_groups_overflow_the_list():
    """More candidates than the ranking list holds: every column equals one of
    three values, so whole groups tie at every cut."""
    gen = torch.Generator().manual_seed(2)
    x = torch.randint(0, 3, (5, 20000), generator=gen).to(torch.bfloat16)
    for k in (1, 20, 64):
        r = itl.token_logp_fwd(x.to(dev()), None, top_k=k)
        assert torch.equal(r.top_ids.cpu(), ranked(x, k))
    x = torch.arange(20000).flip(0).to(torch.float32).repeat(2, 1)  # ascending from the end
    x[1] = x[1].flip(0)
    r = itl.token_logp_fwd(x.to(dev()), None, top_k=64)
    assert torch.equal(r.top_ids.cpu(), ranked(x, 64))


def test_invalid_ignored_and_padding():
    x, view, _ = make(5, 300, 1, "bf16", seed=8)
    tok = torch.tensor([[1, -100, 299], [-100, -100, -100], [300, 5, -1], [7, 7, 7], [-5, -100, 0]])
    for dt in (torch.int64, torch.int32):
        r = itl.token_logp_fwd(view, tok.to(dev(), dt), top_k=4, return_entropy=True)
        ref = check_forward(x, r, tok, 4)
        assert not ref["active"][1]
        assert (bits(r.logp)[1] == 0).all() and r.lse[1] == 0 and r.entropy[1] == 0
        assert (r.top_ids[1] == -1).all() and (r.top_logp[1] == 0).all()
    view[1] = torch.nan  # a padding row is not read
    assert torch.isfinite(itl.token_logp_fwd(view, tok.to(dev())).lse).all()


def test_rows_do_not_depend_on_the_batch():
    x, view, tok = make(70, 9000, 3, "bf16", seed=4, drop=0.0)
    r = itl.token_logp_fwd(view, tok.to(dev()), top_k=11, return_entropy=True)
    for i in (0, 33, 69):
        one = itl.token_logp_fwd(view[i:i + 1], tok[i:i + 1].to(dev()), top_k=11, return_entropy=True)
        for a, b in zip(r, one):
            assert torch.equal(a[i:i + 1], b)
    # fewer alternatives are the head of more, and leave the rest as it is
    few = itl.token_logp_fwd(view, tok.to(dev()), top_k=2)
    assert torch.equal(few.top_ids, r.top_ids[:, :2]) and torch.equal(few.top_logp, r.top_logp[:, :2])
    assert torch.equal(few.logp, r.logp)


def check_gradient(d, x, ref, size, lse):
    d = d.detach().double().cpu()
    t = d.new_tensor(torch.finfo(x.dtype).eps / 2)
    dl = torch.where(torch.isfinite(x), x.double() - lse[:, None], 0.0).abs()
    bound = (4e-5 + 1e-5 * dl) * size
    bound = bound + t * (ref.abs() + bound) + size * 2.0 ** -126
    if x.dtype == torch.float16:
        bound = bound + 2.0 ** -25  # half a subnormal step
    bad = ~((d - ref).abs() <= bound)
    assert not bad.any(), (bad.nonzero()[:4], d[bad][:4], ref[bad][:4])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,m,k,ent", [(1, 1, 1, 0, False), (4, 37, 3, 2, True), (3, 1000, 1, 0, True),
                                         (5, 2050, 16, 0, False), (3, 3001, 70, 64, True),
                                         (2, 4096, 256, 64, True), (3, 600, 0, 5, False),
                                         (2, 600, 0, 0, True)])
def test_gradient(n, v, m, k, ent, dtype):
    x, view, tok = make(n, v, m, dtype, seed=v + m)
    if m >= 3:
        tok[0, 1] = tok[0, 0] = v // 2  # the same token twice
        tok[n - 1] = -100               # a padding row
        tok[0, 2] = v + 3               # invalid
    gen = torch.Generator().manual_seed(9)
    g, gt, ge = torch.randn(n, m, generator=gen), torch.randn(n, k, generator=gen), torch.randn(n, generator=gen)
    t = tok.to(dev()) if m else None
    f = itl.token_logp_fwd(view, t, top_k=k, return_entropy=ent)
    d = itl.token_logp_bwd(view, f.lse, t, g.to(dev()) if m else None, f.top_ids if k else None,
                           gt.to(dev()) if k else None, entropy=f.entropy,
                           grad_entropy=ge.to(dev()) if ent else None)
    ids = f.top_ids.cpu() if k else None
    ref, size = token_gradient(x.double(), tok if m else None, g, ids, gt, ge if ent else None)
    check_gradient(d, x, ref, size, torch.logsumexp(x.double(), 1))
    if m >= 3:
        assert (d[n - 1] == 0).all()
    # in place, the same bits
    own = view.clone()
    itl.token_logp_bwd(own, f.lse, t, g.to(dev()) if m else None, f.top_ids if k else None,
                       gt.to(dev()) if k else None, entropy=f.entropy,
                       grad_entropy=ge.to(dev()) if ent else None, dlogits_out=own)
    assert torch.equal(own, d)


def test_gradient_against_differences():
    """The autograd function against central differences of the float64
    objective in random directions: a difference quotient of step h is off by
    h^2 and the direction's sum by the tolerance of its terms."""
    n, v, m, k = 3, 200, 4, 3
    x, view, tok = make(n, v, m, "fp32", seed=6)
    leaf = view.clone().requires_grad_()
    gen = torch.Generator().manual_seed(1)
    g, gt, ge = torch.randn(n, m, generator=gen), torch.randn(n, k, generator=gen), torch.randn(n, generator=gen)
    r = itl.batch_invariant_token_logp(leaf, tok.to(dev()), top_k=k, return_entropy=True)
    ((r.logp * g.to(dev())).sum() + (r.top_logp * gt.to(dev())).sum()
     + (r.entropy * ge.to(dev())).sum()).backward()
    ids = r.top_ids.cpu()

    def objective(y):
        s = token_scores(y, tok, 0)
        live = s["active"].double()
        top = y.gather(1, ids.clamp(min=0)) - torch.logsumexp(y, 1)[:, None]
        return float((s["logp"] * g).sum() + (top * gt * live[:, None]).sum() + (s["entropy"] * ge).sum())

    step = 1e-5
    for i in range(5):
        u = torch.randn(n, v, generator=gen, dtype=torch.float64)
        want = (objective(x.double() + step * u) - objective(x.double() - step * u)) / (2 * step)
        got = float((leaf.grad.double().cpu() * u).sum())
        assert abs(want - got) <= 1e-4 * float((leaf.grad.double().cpu() * u).abs().sum()) + 1e-6


def test_parts_of_the_gradient_may_be_absent():
    x, view, tok = make(4, 500, 2, "fp32", seed=12)
    for name, kw in itertools.product(("logp", "top_logp", "entropy"), (0,)):
        leaf = view.clone().requires_grad_()
        r = itl.batch_invariant_token_logp(leaf, tok.to(dev()), top_k=3, return_entropy=True)
        getattr(r, name).sum().backward()
        assert torch.isfinite(leaf.grad).all() and leaf.grad.abs().sum() > 0
    leaf = view.clone().requires_grad_()
    r = itl.batch_invariant_token_logp(leaf, None, top_k=2)
    assert r.entropy is None and r.logp.shape == (4, 0) and not r.lse.requires_grad
    r.top_logp.sum().backward()
    lead = itl.token_logp_fwd(view.view(2, 2, 500), tok.view(2, 2, 2).to(dev()), top_k=3)
    assert lead.logp.shape == (2, 2, 2) and lead.top_ids.shape == (2, 2, 3)


def test_second_derivative_is_refused():
    _, view, tok = make(2, 50, 1, "fp32", seed=1)
    leaf = view.clone().requires_grad_()
    d, = torch.autograd.grad(itl.batch_invariant_token_logp(leaf, tok.to(dev())).logp.square().sum(), leaf,
                             create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        d.sum().backward()


def test_one_row_without_leading_dimensions():
    x, view, tok = make(1, 700, 3, "bf16", seed=13, drop=0.0)
    one = itl.token_logp_fwd(view[0], tok[0].to(dev()), top_k=4)
    two = itl.token_logp_fwd(view, tok.to(dev()), top_k=4)
    assert one.logp.shape == (3,) and one.top_ids.shape == (4,)
    assert torch.equal(one.logp, two.logp[0]) and torch.equal(one.top_ids, two.top_ids[0])


def test_empty_batch():
    x = torch.empty(0, 100, dtype=torch.bfloat16, device=dev())
    r = itl.token_logp_fwd(x, torch.empty(0, 3, dtype=torch.int64, device=dev()), top_k=2,
                           return_entropy=True)
    assert r.logp.shape == (0, 3) and r.top_ids.shape == (0, 2)
    assert itl.token_logp_bwd(x, r.lse, torch.empty(0, 3, dtype=torch.int64, device=dev()),
                              r.logp).shape == (0, 100)


def test_past_two_to_the_31_elements():
    """Rows whose offset passes 2^31 elements, forward and backward."""
    n, v = 14200, 151936
    x = torch.zeros(n, v, dtype=torch.bfloat16, device=dev())
    last = (3 * torch.randn(2, v, generator=torch.Generator().manual_seed(3))).to(torch.bfloat16)
    x[-2:] = last.to(dev())
    tok = torch.full((n, 2), -100, dtype=torch.int64, device=dev())
    tok[-2:] = torch.tensor([[5, v - 1], [v // 2, 5]], device=dev())
    r = itl.token_logp_fwd(x, tok, top_k=20, return_entropy=True)
    one = itl.token_logp_fwd(x[-2:].clone(), tok[-2:], top_k=20, return_entropy=True)
    for a, b in zip(r, one):
        assert torch.equal(a[-2:], b)
    g = torch.ones(n, 2, device=dev())
    d1 = itl.token_logp_bwd(x[-2:].clone(), one.lse, tok[-2:], g[-2:])
    itl.token_logp_bwd(x, r.lse, tok, g, dlogits_out=x)
    assert torch.equal(x[-2:], d1) and not x[:-2].any()


def test_graph_replays():
    """Forward and backward captured together, replayed with new inputs and
    eager work in between: the eager bits each time."""
    n, v, m, k = 16, 33000, 3, 7
    x = torch.empty(n, v, dtype=torch.bfloat16, device=dev())
    t = torch.zeros(n, m, dtype=torch.int64, device=dev())
    g, gt = torch.zeros(n, m, device=dev()), torch.zeros(n, k, device=dev())

    def step():
        f = itl.token_logp_fwd(x, t, top_k=k, return_entropy=True)
        return (*f, itl.token_logp_bwd(x, f.lse, t, g, f.top_ids, gt))

    def fill(seed):
        gen = torch.Generator().manual_seed(seed)
        x.copy_((3 * torch.randn(n, v, generator=gen)).to(torch.bfloat16))
        t.copy_(torch.randint(0, v, (n, m), generator=gen))
        g.copy_(torch.randn(n, m, generator=gen))
        gt.copy_(torch.randn(n, k, generator=gen))

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (1, 2, 3):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b), seed
        torch.cuda.synchronize()


def test_two_streams_at_once():
    """Two calls on two streams, each with a workspace of its own."""
    cases = [make(64, 30000, 2, "bf16", seed=s) for s in (1, 2)]
    want = [itl.token_logp_fwd(v, t.to(dev()), top_k=5) for _, v, t in cases]
    torch.cuda.synchronize()
    got = [None, None]
    for i, (_, v, t) in enumerate(cases):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got[i] = itl.token_logp_fwd(v, t.to(dev()), top_k=5)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a.logp, b.logp) and torch.equal(a.top_ids, b.top_ids)
