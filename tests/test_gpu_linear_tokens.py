"""The token operators through the LM head (bf16 and 8-bit), their gradients,
and the decoder's tail as a whole, against the plain float64 forms.

Tolerances.  Inputs on a grid (hidden k / 16, weight k / 1024) make every sum
of products exact in fp32, so the alternatives' order is exact and logp and lse
keep the logits' bound.  Gradients: dz rounds to bf16 once, so dhidden and
dweight are within 2^-8 of sum |dz||W| (|dz||h|), plus 1e-3 of what an entry's
own column carries and 1e-6, as for linear_logp's backward; bf16 outputs round
by 2^-8 more.  8-bit head: products of e4m3 values are exact in fp32; a matrix
instruction adds 16 of them and H / 16 such sums follow, within (16 + H / 16)
2^-23 sum |h w| of the exact logit, which moves logp and lse by at most twice
that."""

import pytest
import torch

import invariant_token_log_amd as itl
from gpu_helpers import ATOL, RTOL, bits, dev
from token_reference import norm_forward, norm_gradient, ranked, token_gradient, token_scores

pytestmark = pytest.mark.gpu


def grid(shape, step, std, gen):
    return (torch.randn(shape, generator=gen) * (std / step)).round().clamp(-127, 127) * step


def make(n, h, v, m, seed, drop=0.15):
    gen = torch.Generator().manual_seed(seed)
    hid, w = grid((n, h), 1 / 16, 1.0, gen), grid((v, h), 1 / 1024, 0.05, gen)
    tok = torch.randint(0, v, (n, m), generator=gen)
    tok[torch.rand(n, m, generator=gen) < drop] = -100
    return hid, w, tok


def close(a, ref, what, extra=0.0):
    a = a.detach().double().cpu()
    assert torch.equal(torch.isnan(a), torch.isnan(ref)), what
    bad = ~((a - ref).abs() <= ATOL + RTOL * ref.abs() + extra) & ~torch.isnan(ref)
    assert not bad.any(), (what, a[bad][:5], ref[bad][:5])


def check(r, z, tok, k, extra=0.0):
    ref = token_scores(z, tok, k)
    close(r.logp, ref["logp"], "logp", extra)
    close(r.lse, ref["lse"], "lse", extra)
    if r.entropy is not None:
        close(r.entropy, ref["entropy"], "entropy", extra * 20 + 2e-5)
    assert torch.equal(r.top_ids.cpu(), ref["top_ids"])
    close(r.top_logp, ref["top_logp"], "top_logp", extra)


# one row to many (64-, 128- and 256-row tiles, more than one row chunk), odd
# vocabularies, fewer columns than a tile
SIZES = [(1, 64, 5, 1, 5), (3, 128, 255, 2, 20), (64, 192, 1000, 1, 64), (65, 64, 257, 3, 1),
         (130, 256, 3001, 1, 20), (300, 320, 700, 5, 8), (600, 64, 5000, 1, 20), (5, 64, 40000, 0, 9)]


@pytest.mark.parametrize("n,h,v,m,k", SIZES)
def test_forward(n, h, v, m, k):
    hid, w, tok = make(n, h, v, m, seed=n + v)
    a, b = hid.to(dev(), torch.bfloat16), w.to(dev(), torch.bfloat16)
    t = tok.to(dev()) if m else None
    z = hid.double() @ w.double().T
    for temp in (1.0, 0.7):
        r = itl.linear_token_logp_fwd(a, b, t, top_k=k, temperature=temp, return_entropy=True)
        inv = float(torch.tensor(1.0 / temp, dtype=torch.float64).float())
        check(r, (z.float() * inv).double(), tok, k)
        # row chunks, a prepared weight and kept logits: the same bits
        kept = torch.empty(n, v, device=dev())
        for kw in (dict(row_chunk=256), dict(prepared_weight=itl.prepare_weight(b)), dict(logits_out=kept)):
            q = itl.linear_token_logp_fwd(a, b, t, top_k=k, temperature=temp, return_entropy=True, **kw)
            for x, y in zip(r, q):
                assert torch.equal(x, y), kw.keys()
        act = token_scores(z, tok, 0)["active"]
        assert torch.equal(kept.cpu()[act], z.float()[act])


def test_same_bits_as_linear_logp():
    hid, w, tok = make(200, 256, 2000, 1, seed=5)
    hid = torch.randn(200, 256, generator=torch.Generator().manual_seed(1))
    a, b, t = hid.to(dev(), torch.bfloat16), w.to(dev(), torch.bfloat16), tok.to(dev())
    for rnd in (False, True):
        ref = itl.linear_logp_fwd(a, b, t[:, 0], return_entropy=True, round_logits=rnd)
        for k in (0, 6):
            r = itl.linear_token_logp_fwd(a, b, t, top_k=k, return_entropy=True, round_logits=rnd)
            assert torch.equal(bits(r.logp[:, 0]), bits(ref[0]))
            assert torch.equal(bits(r.lse), bits(ref[1])) and torch.equal(bits(r.entropy), bits(ref[2]))
        one = itl.linear_token_logp_fwd(a[7:8], b, t[7:8], top_k=6, return_entropy=True, round_logits=rnd)
        for x, y in zip(one, r):
            assert torch.equal(x, y[7:8])


def test_rounded_logits_order():
    """With the logits rounded to bf16 many columns tie; the lowest comes first."""
    hid, w, tok = make(40, 128, 4000, 2, seed=6)
    a, b = hid.to(dev(), torch.bfloat16), w.to(dev(), torch.bfloat16)
    z = (hid.double() @ w.double().T).float().to(torch.bfloat16)
    r = itl.linear_token_logp_fwd(a, b, tok.to(dev()), top_k=33, round_logits=True)
    check(r, z.double(), tok, 33)
    zero = itl.linear_token_logp_fwd(torch.zeros_like(a), b, None, top_k=64)
    assert torch.equal(zero.top_ids, torch.arange(64, device=dev()).expand(40, 64))


@pytest.mark.parametrize("n,h,v,m,k,ent,temp", [(1, 64, 300, 1, 0, False, 1.0), (5, 128, 700, 3, 4, True, 0.7),
                                                (200, 64, 513, 16, 0, False, 1.0),
                                                (70, 192, 1000, 70, 64, True, 1.3),
                                                (3, 64, 300, 0, 5, False, 1.0)])
def test_gradient(n, h, v, m, k, ent, temp):
    hid, w, tok = make(n, h, v, m, seed=n + m)
    if m >= 3:
        tok[0, 1] = tok[0, 0] = v // 2
        tok[n - 1] = -100
        tok[0, 2] = v + 1
    gen = torch.Generator().manual_seed(3)
    g, gt, ge = torch.randn(n, m, generator=gen), torch.randn(n, k, generator=gen), torch.randn(n, generator=gen)
    a, b = hid.to(dev(), torch.bfloat16), w.to(dev(), torch.bfloat16)
    t = tok.to(dev()) if m else None
    kept = torch.empty(n, (v + 3) // 4 * 4, device=dev())[:, :v]
    f = itl.linear_token_logp_fwd(a, b, t, top_k=k, temperature=temp, return_entropy=ent, logits_out=kept)
    args = dict(token_ids=t, logp=f.logp if m else None, grad_logp=g.to(dev()) if m else None,
                top_ids=f.top_ids if k else None, top_logp=f.top_logp if k else None,
                grad_top_logp=gt.to(dev()) if k else None, temperature=temp, entropy=f.entropy,
                grad_entropy=ge.to(dev()) if ent else None)
    dh, dw = itl.linear_token_logp_bwd(a, b, f.lse, **args)
    inv = 1.0 / temp
    x = hid.double() @ w.double().T * inv
    dx, size = token_gradient(x, tok if m else None, g, f.top_ids.cpu() if k else None, gt, ge if ent else None)
    dz, size = dx * inv, size * inv
    wd, hd = w.double(), hid.double()
    bound_h = 2.0 ** -8 * dz.abs() @ wd.abs() + 1e-4 * size @ wd.abs() + 1e-6
    bound_w = 2.0 ** -8 * dz.abs().T @ hd.abs() + 1e-4 * size.T @ hd.abs() + 1e-6
    assert ((dh.double().cpu() - dz @ wd).abs() <= bound_h).all()
    assert ((dw.double().cpu() - dz.T @ hd).abs() <= bound_w).all()
    # kept logits, a prepared weight, vocabulary chunks: the same bits
    for kw in (dict(saved_logits=kept), dict(prepared_weight=itl.prepare_weight(b)), dict(vocab_chunk=256)):
        dh2, dw2 = itl.linear_token_logp_bwd(a, b, f.lse, **args, **kw)
        assert torch.equal(dh2, dh) and torch.equal(dw2, dw), kw.keys()
    # through autograd, in bf16
    la, lb = a.clone().requires_grad_(), b.clone().requires_grad_()
    r = itl.linear_token_logp(la, lb, t, top_k=k, temperature=temp, return_entropy=ent, save_logits=m > 1)
    outs = [(r.logp, g)] if m else []
    outs += [(r.top_logp, gt)] if k else []
    outs += [(r.entropy, ge)] if ent else []
    torch.autograd.backward([o for o, _ in outs], [q.to(dev()) for _, q in outs])
    assert torch.equal(la.grad, dh.to(torch.bfloat16)) and torch.equal(lb.grad, dw.to(torch.bfloat16))


@pytest.mark.parametrize("bf16", [False, True])
def test_gradient_over_many_columns(bf16):
    """Four segments of the vocabulary (9216 columns each): few rows (one
    product a segment), the same in chunks, and many rows (a tile walks them)
    give a row the same bits; the bound is test_gradient's."""
    h, v, few, many = 320, 16384 * 2 + 700, 5, 8300
    gen = torch.Generator().manual_seed(4)
    hid = torch.randn(many, h, generator=gen).to(torch.bfloat16)
    w = (0.05 * torch.randn(v, h, generator=gen)).to(torch.bfloat16)
    tok = torch.randint(0, v, (many, 2), generator=gen)
    tok[1, 0], tok[2, 1], tok[3, 0] = 9216, 9215, v - 1
    g = torch.randn(many, 2, generator=gen)
    b = w.to(dev())
    pw = itl.prepare_weight(b)

    def grads(n, **kw):
        a, t = hid[:n].to(dev()), tok[:n].to(dev())
        f = itl.linear_token_logp_fwd(a, b, t)
        return itl.linear_token_logp_bwd(a, b, f.lse, t, f.logp, g[:n].to(dev()),
                                         out_dtype=torch.bfloat16 if bf16 else torch.float32, **kw)

    dh, dw = grads(few)
    x = hid[:few].double() @ w.double().T
    dz, size = token_gradient(x, tok[:few], g[:few], None, None, None)
    wd, hd = w.double(), hid[:few].double()
    out = 2.0 ** -8 if bf16 else 0.0
    ref_h, ref_w = dz @ wd, dz.T @ hd
    bound_h = 2.0 ** -8 * dz.abs() @ wd.abs() + 1e-4 * size @ wd.abs() + 1e-6
    bound_w = 2.0 ** -8 * dz.abs().T @ hd.abs() + 1e-4 * size.T @ hd.abs() + 1e-6
    assert ((dh.double().cpu() - ref_h).abs() <= bound_h + out * (ref_h.abs() + bound_h)).all()
    assert ((dw.double().cpu() - ref_w).abs() <= bound_w + out * (ref_w.abs() + bound_w)).all()
    for kw in (dict(vocab_chunk=1), dict(vocab_chunk=32768), dict(prepared_weight=pw), dict(need_dweight=False),
               dict(prepared_weight=pw, vocab_chunk=16384)):
        dh2, dw2 = grads(few, **kw)
        assert torch.equal(dh2, dh), kw.keys()
        assert dw2 is None or torch.equal(dw2, dw), kw.keys()
    for kw in (dict(), dict(need_dweight=False), dict(vocab_chunk=16384, prepared_weight=pw)):
        assert torch.equal(grads(many, **kw)[0][:few], dh), kw.keys()


def quant(n, h, v, seed):
    gen = torch.Generator().manual_seed(seed)
    rows = lambda r, s: itl.quantize_rows((s * torch.randn(r, h, generator=gen)).to(dev()))  # noqa: E731
    return rows(n, 1.0), rows(v, 0.05)


@pytest.mark.parametrize("n,h,v,m,k", [(1, 64, 5, 1, 0), (7, 128, 300, 2, 0), (32, 192, 1000, 1, 3),
                                       (33, 320, 257, 1, 0), (64, 64, 513, 3, 0), (100, 256, 700, 1, 0),
                                       (128, 448, 600, 2, 0), (129, 64, 1000, 1, 0), (300, 192, 2000, 2, 0),
                                       (257, 320, 515, 1, 0), (600, 128, 5000, 1, 2)])
def test_8bit_head(n, h, v, m, k):
    a, b = quant(n, h, v, seed=n + h)
    tok = torch.randint(0, v, (n, m), generator=torch.Generator().manual_seed(n))
    tok[0, 0] = -100
    hd = a.data.cpu().double() * a.scale.cpu().double()[:, None]
    wd = b.data.cpu().double() * b.scale.cpu().double()[:, None]
    z = hd @ wd.T / 0.9
    extra = float((2 * (16 + h / 16) * 2.0 ** -23 * (hd.abs() @ wd.abs().T)).max()) / 0.9
    r = itl.linear_token_logp_fwd(a, b, tok.to(dev()), top_k=k, temperature=0.9, return_entropy=True)
    ref = token_scores(z, tok, k)
    close(r.logp, ref["logp"], "logp", extra)
    close(r.lse, ref["lse"], "lse", extra)
    close(r.entropy, ref["entropy"], "entropy", 20 * extra + 2e-5)
    if k:
        close(r.top_logp, ref["top_logp"], "top_logp", extra)
        got = z.gather(1, r.top_ids.cpu().clamp(min=0))
        want = z.gather(1, ranked(z, k))
        assert ((got - want).abs() <= 2 * extra)[ref["active"]].all()
    # a row alone (the narrow tile), row chunks: the same bits
    for i in (n - 1, n // 2):
        one = itl.linear_token_logp_fwd(itl.QuantizedRows(a.data[i:i + 1], a.scale[i:i + 1].contiguous()), b,
                                        tok[i:i + 1].to(dev()), top_k=k, temperature=0.9, return_entropy=True)
        for x, y in zip(one, r):
            assert torch.equal(x, y[i:i + 1])
    c = itl.linear_token_logp_fwd(a, b, tok.to(dev()), top_k=k, temperature=0.9, return_entropy=True, row_chunk=256)
    for x, y in zip(c, r):
        assert torch.equal(x, y)


def test_8bit_strided_operands():
    a, b = quant(40, 128, 600, seed=2)
    def wide(q):
        buf = torch.zeros(q.data.shape[0], 160, dtype=torch.uint8, device=dev())
        buf[:, :128] = q.data.view(torch.uint8)
        return itl.QuantizedRows(buf.view(torch.float8_e4m3fn)[:, :128], q.scale)
    r = itl.linear_token_logp_fwd(a, b, None, top_k=4)
    s = itl.linear_token_logp_fwd(wide(a), wide(b), None, top_k=4)
    assert torch.equal(r.top_ids, s.top_ids) and torch.equal(r.lse, s.lse)


def test_decoder_tail():
    """Norm, head and token log-probabilities together, as a training step and
    as 8-bit scoring."""
    n, h, v, m, k = 37, 128, 900, 3, 4
    gen = torch.Generator().manual_seed(7)
    x, r, nw = torch.randn(n, h, generator=gen), 2 * torch.randn(n, h, generator=gen), 1 + 0.1 * torch.randn(h, generator=gen)
    w = 0.05 * torch.randn(v, h, generator=gen)
    tok = torch.randint(0, v, (n, m), generator=gen)
    leaves = [t.to(dev(), torch.bfloat16).requires_grad_() for t in (x, r, nw, w)]
    lx, lr, ln, lw = leaves
    out = itl.norm_linear_token_logp(lx, ln, lw, tok.to(dev()), residual=lr, top_k=k, return_entropy=True)
    g = torch.randn(n, m, generator=gen)
    out.logp.backward(g.to(dev()))
    # the parts, called one after the other
    y, s = itl.rms_norm(lx.detach(), ln.detach(), residual=lr.detach())
    parts = itl.linear_token_logp_fwd(y, lw.detach(), tok.to(dev()), top_k=k, return_entropy=True)
    for a, b in zip(out, parts):
        assert torch.equal(a, b)
    dh, dw = itl.linear_token_logp_bwd(y, lw.detach(), parts.lse, tok.to(dev()), parts.logp, g.to(dev()), out_dtype=torch.bfloat16)
    assert torch.equal(lw.grad, dw)
    sd = s.cpu()
    dx, dn = norm_gradient(sd, nw.to(torch.bfloat16), dh.cpu(), None, 1e-6)
    assert ((lx.grad.double().cpu() - dx).abs() <= 2.0 ** -8 * dx.abs() + 1e-5 * dx.abs().amax()).all()
    assert torch.equal(lx.grad, lr.grad)
    assert ((ln.grad.double().cpu() - dn).abs() <= 2.0 ** -8 * dn.abs() + 1e-5 * dn.abs().amax()).all()
    # 8 bits: the norm's rows and a weight quantised once
    qw = itl.quantize_rows(lw.detach())
    with torch.no_grad():
        q = itl.norm_linear_token_logp(lx, ln, qw, tok.to(dev()), residual=lr, top_k=k)
    rows, _ = itl.rms_norm_quantized(lx.detach(), ln.detach(), residual=lr.detach())
    direct = itl.linear_token_logp_fwd(rows, qw, tok.to(dev()), top_k=k)
    assert torch.equal(q.logp, direct.logp) and torch.equal(q.top_ids, direct.top_ids)
    # e4m3 rounds by 2^-4 at most: far from the bf16 head's only by the rounding of 128 products
    hd, wd = norm_forward(sd, nw.to(torch.bfloat16), 1e-6)[0], lw.detach().double().cpu()
    off = 2 * (2 * 2.0 ** -4 + 2.0 ** -8 + 2.0 ** -8) * (hd.abs() @ wd.abs().T).amax(1, keepdim=True)
    assert ((q.logp.double().cpu() - out.logp.detach().double().cpu()).abs() <= off).all()
    with pytest.raises(ValueError, match="no gradient"):
        itl.norm_linear_token_logp(lx, ln, qw, tok.to(dev()), residual=lr)


def test_graph_replays_tail():
    """Norm and head, bf16 and 8-bit, captured and replayed with new inputs."""
    n, h, v = 140, 128, 3000
    x = torch.zeros(n, h, dtype=torch.bfloat16, device=dev())
    tok = torch.zeros(n, 2, dtype=torch.int64, device=dev())
    gen = torch.Generator().manual_seed(1)
    nw = torch.ones(h, dtype=torch.bfloat16, device=dev())
    w = (0.05 * torch.randn(v, h, generator=gen)).to(dev(), torch.bfloat16)
    qw = itl.quantize_rows(w)
    g = torch.ones(n, 2, device=dev())

    def step():
        y, s, rstd = itl.rms_norm_fwd(x, nw, residual=x, return_rstd=True)
        f = itl.linear_token_logp_fwd(y, w, tok, top_k=5, return_entropy=True)
        dh, dw = itl.linear_token_logp_bwd(y, w, f.lse, tok, f.logp, g, out_dtype=torch.bfloat16)
        dx, dn = itl.rms_norm_bwd(s, nw, rstd, dh)
        q, _ = itl.rms_norm_quantized(x, nw, residual=x)
        return [*f, dw, dx, dn, *itl.linear_token_logp_fwd(q, qw, tok, top_k=5)[:2]]

    def fill(seed):
        gn = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn(n, h, generator=gn).to(torch.bfloat16))
        tok.copy_(torch.randint(0, v, (n, 2), generator=gn))

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
        for i, (a, b) in enumerate(zip(out, step())):
            assert torch.equal(a, b), (seed, i)
        torch.cuda.synchronize()


def test_empty_batch():
    a = torch.empty(0, 64, dtype=torch.bfloat16, device=dev())
    w = torch.randn(300, 64, device=dev()).to(torch.bfloat16)
    r = itl.linear_token_logp_fwd(a, w, torch.empty(0, 2, dtype=torch.int64, device=dev()), top_k=3)
    assert r.logp.shape == (0, 2)
    dh, dw = itl.linear_token_logp_bwd(a, w, r.lse, torch.empty(0, 2, dtype=torch.int64, device=dev()),
                                       r.logp, r.logp)
    assert dh.shape == (0, 64) and (dw == 0).all()
