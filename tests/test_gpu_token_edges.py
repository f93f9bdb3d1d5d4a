"""Values, sizes and launches at the edges of the token operators: NaN and
infinite logits, vocabularies past one register block of tiles, row chunks,
against the plain float64 forms.

Inputs of the heads are small whole numbers or lie on a grid, so that every sum
of products is exact in fp32 and the order of the alternatives is exact too;
logp and lse keep the bound of the logp path (gpu_helpers)."""

import pytest
import torch

import invariant_token_log_amd as itl
from gpu_helpers import ATOL, RTOL, bits, dev
from invariant_token_log_amd import _lib
from token_reference import ranked, token_gradient, token_scores

pytestmark = pytest.mark.gpu


def same(a, b):
    """Equal bits, NaN included."""
    for x, y in zip(a, b):
        if x is not None:
            x, y = x.contiguous(), y.contiguous()
            view = torch.int64 if x.dtype == torch.int64 else torch.int32
            assert torch.equal(x.view(view), y.view(view))


def head_operands(n, h, v, q8, seed):
    """(hidden, weight) for the head and the exact logits z (float64): bf16
    rows, or 8-bit rows with scales that are powers of two."""
    gen = torch.Generator().manual_seed(seed)
    hid = torch.randint(-4, 5, (n, h), generator=gen).float()
    w = torch.randint(-4, 5, (v, h), generator=gen).float()
    z = (hid @ w.T).double()  # whole numbers of at most 16 h: exact in fp32
    if not q8:
        return hid.to(dev(), torch.bfloat16), w.to(dev(), torch.bfloat16), z
    s = 2.0 ** torch.randint(-2, 2, (v,), generator=gen)
    rows = lambda x, scale: itl.QuantizedRows(x.to(dev()).to(torch.float8_e4m3fn), scale.to(dev()))  # noqa: E731
    return rows(hid, torch.ones(n)), rows(w, s), z * s.double()


def put_nan(weight, columns):
    """The weight with NaN in the given rows: their logits are NaN in every row."""
    if isinstance(weight, itl.QuantizedRows):
        scale = weight.scale.clone()
        scale[columns] = torch.nan
        return itl.QuantizedRows(weight.data, scale)
    weight = weight.clone()
    weight[columns, 1] = torch.nan
    return weight


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("n,h,v", [(5, 64, 3000), (140, 64, 2500), (600, 128, 1000), (3, 64, 170001)])
def test_nan_logits_through_the_head(n, h, v, q8):
    """A NaN logit ranks as -inf: the other columns of its tile keep their
    places, also when it lies beside the row's greatest logits, when a tile
    holds nothing else and when a whole row is NaN."""
    a, b, z = head_operands(n, h, v, q8, seed=n + v)
    beside = [c ^ 1 for c in z.argmax(1)[:3].tolist() if c ^ 1 < v]
    last = list(range(v // 256 * 256, v))  # the last tile, whole
    for columns in (beside, last, beside + last):
        x = z.clone()
        x[:, columns] = torch.nan
        bn = put_nan(b, columns)
        for k in (1, 20, 64):
            r = itl.linear_token_logp_fwd(a, bn, None, top_k=k, temperature=0.5, return_entropy=True)
            assert torch.equal(r.top_ids.cpu(), ranked(x, k)), (len(columns), k)
            assert r.lse.isnan().all() and r.top_logp.isnan().all() and r.entropy.isnan().all()
    if q8:
        scale = a.scale.clone()
        scale[1] = torch.nan
        an = itl.QuantizedRows(a.data, scale)
    else:
        an = a.clone()
        an[1, 3] = torch.nan
    r = itl.linear_token_logp_fwd(an, b, None, top_k=9)
    assert torch.equal(r.top_ids[1].cpu(), torch.arange(9)) and r.lse[1].isnan()
    other = [i for i in range(n) if i != 1]
    ref = itl.linear_token_logp_fwd(a, b, None, top_k=9)
    same([t[other] for t in (r.lse, r.top_logp, r.top_ids)], [t[other] for t in (ref.lse, ref.top_logp, ref.top_ids)])


def test_infinite_logits_through_the_head():
    """+inf comes first, -inf last, and 0 * inf is a NaN."""
    a, b, z = head_operands(40, 64, 1500, False, seed=3)
    b[700] = 0.0
    b[700, 0] = torch.inf
    z[:, 700] = a[:, 0].cpu().double() * torch.inf
    assert z[:, 700].isnan().any() and (z[:, 700] == torch.inf).any() and (z[:, 700] == -torch.inf).any()
    for k in (1, 64):
        r = itl.linear_token_logp_fwd(a, b, None, top_k=k)
        assert torch.equal(r.top_ids.cpu(), ranked(z, k))
    low = z[:, 700] == -torch.inf
    lse = torch.logsumexp(z[low], 1)
    assert ((r.lse.cpu().double()[low] - lse).abs() <= ATOL + RTOL * lse.abs()).all()
    assert not torch.isfinite(r.lse.cpu()[~low]).any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_nan_logits_streamed(dtype):
    """The same from logits, with an infinite logit beside it."""
    x = torch.randn(6, 5003, generator=torch.Generator().manual_seed(1)).to(dtype)
    x[0, 100] = torch.nan
    x[1, x[1].argmax() ^ 1] = torch.nan
    x[2, :] = torch.nan
    x[3, 7], x[3, 8] = torch.inf, torch.nan
    x[4, 9], x[4, 300] = torch.inf, -torch.inf
    for k in (1, 20, 64):
        r = itl.token_logp_fwd(x.to(dev()), None, top_k=k)
        assert torch.equal(r.top_ids.cpu(), ranked(x, k))
        assert r.lse[:4].isnan().all() and torch.isfinite(r.lse[5])


# a tile is tile_width columns: here 4096, the default
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_tile_of_nothing_but_nan(dtype):
    """A tile whose only values are NaN (and -inf) is no empty tile: the row's
    lse is NaN, as for a NaN beside other values.  Rows without one, and rows
    and tiles of -inf alone, keep their values."""
    v = 3 * 4096 + 5
    x = torch.randn(8, v, generator=torch.Generator().manual_seed(2)).to(dtype)
    x[0, -1] = torch.nan                     # beside four other values
    x[1, -5:] = torch.nan                    # the last tile, whole
    x[2, 4096:8192] = -torch.inf
    x[2, 5000] = torch.nan                   # one NaN in a masked tile
    x[3, 4096:8192] = torch.nan              # a whole tile
    x[4] = torch.nan                         # a whole row
    x[5, 4096:8192] = -torch.inf             # a masked tile
    x[6] = -torch.inf                        # a masked row
    nan = torch.tensor([True] * 5 + [False] * 3)
    t = torch.full((8, 1), 17, dtype=torch.int64, device=dev())
    xd = x.to(dev())
    for k in (0, 5):
        r = itl.token_logp_fwd(xd, t, top_k=k, return_entropy=True)
        assert torch.equal(r.lse.isnan().cpu(), nan)
        assert r.logp[:5].isnan().all() and r.entropy[:5].isnan().all() and r.top_logp[:5].isnan().all()
        assert r.lse[6] == -torch.inf and r.logp[6].isnan()
        ref = token_scores(x[[5, 7]].double(), t[[5, 7]], k)
        assert ((r.lse[[5, 7]].cpu().double() - ref["lse"]).abs() <= ATOL + RTOL * ref["lse"].abs()).all()
        for shards in (1, 19):  # of v = 19 * 647
            logp, lse, ent = itl.logp_fwd(xd, t[:, 0], num_shards=shards, return_entropy=True)
            assert torch.equal(lse.isnan().cpu(), nan) and logp[:5].isnan().all() and ent[:5].isnan().all()
            for a, b in ((lse, r.lse), (logp, r.logp[:, 0])):
                assert torch.equal(bits(a)[5:], bits(b)[5:])


@pytest.mark.parametrize("h", [64, 128, 192])
def test_8bit_head_of_one_step(h):
    """Many rows on one pair of K steps (h = 64, 128), where a single barrier
    stands between the scales and targets in LDS and their reads: scales and
    targets that differ from row to row and column to column, every row."""
    n, v = 1100, 2600
    a, b, z = head_operands(n, h, v, True, seed=h)
    gen = torch.Generator().manual_seed(h)
    s = 2.0 ** torch.randint(-3, 2, (n,), generator=gen)
    a, z = itl.QuantizedRows(a.data, s.to(dev())), z * s.double()[:, None]
    tok = torch.randint(0, v, (n, 1), generator=gen)
    tok[torch.rand(n, 1, generator=gen) < 0.1] = -100
    for k in (0, 7):
        r = itl.linear_token_logp_fwd(a, b, tok.to(dev()), top_k=k, return_entropy=True)
        ref = token_scores(z, tok, k)
        for got, want in ((r.logp, ref["logp"]), (r.lse, ref["lse"])):
            assert ((got.double().cpu() - want).abs() <= ATOL + RTOL * want.abs()).all()
        assert torch.equal(r.top_ids.cpu(), ref["top_ids"])


def test_more_rows_than_one_grid_holds():
    """2^26 rows and a few, one column: more workgroups than one launch takes.
    Each row as in a batch of its own, beside a launch's end and at the last."""
    n = (1 << 26) + 7
    x = torch.empty(n, 1, dtype=torch.bfloat16, device=dev()).normal_(generator=torch.Generator(dev()).manual_seed(1))
    r = torch.empty_like(x).normal_(generator=torch.Generator(dev()).manual_seed(2))
    w = torch.full((1,), 1.5, dtype=torch.bfloat16, device=dev())
    y, s, rstd = itl.rms_norm_fwd(x, w, residual=r, return_rstd=True)
    q, sq = itl.rms_norm_quantized(x, w, residual=r)
    assert torch.equal(s, (x.float() + r.float()).to(torch.bfloat16)) and torch.equal(sq, s)
    ends = [(i << 22) - 3 for i in range(1, 17)] + [0, n - 9]
    for i in ends:
        part = slice(i, i + 9)
        y1, s1, rstd1 = itl.rms_norm_fwd(x[part], w, residual=r[part], return_rstd=True)
        q1, _ = itl.rms_norm_quantized(x[part], w, residual=r[part])
        assert torch.equal(y[part], y1) and torch.equal(rstd[part], rstd1)
        assert torch.equal(q.data[part].view(torch.uint8), q1.data.view(torch.uint8))
        assert torch.equal(q.scale[part], q1.scale)
    assert torch.isfinite(y).all() and (rstd > 0).all()


@pytest.mark.parametrize("m,k,kept,q8", [(1, 0, False, False), (0, 0, False, False), (2, 3, True, False),
                                         (1, 0, False, True), (0, 0, False, True)])
def test_row_chunks_without_logits_in_the_workspace(m, k, kept, q8):
    """Several chunks, a part of one and one that takes the tiles for few rows:
    the bits of the rows taken together."""
    n, h, v = 805, 128, 1500
    a, b, _ = head_operands(n, h, v, q8, seed=m)
    tok = torch.randint(0, v, (n, m), generator=torch.Generator().manual_seed(5)).to(dev()) if m else None
    if m:
        tok[3] = -100
    outs = []
    for chunk in (0, 256, 300):
        z = torch.zeros(n, v, device=dev()) if kept else None
        extra = dict(logits_out=z) if kept else {}
        r = itl.linear_token_logp_fwd(a, b, tok, top_k=k, return_entropy=True, row_chunk=chunk, **extra)
        outs.append([*r, z])
    for o in outs[1:]:
        same(outs[0], o)


def test_backwards_refuse_gradients_in_another_layout():
    n, v, h, m, k = 4, 300, 64, 3, 2
    a, b, z = head_operands(n, h, v, False, seed=9)
    x, tok = z.float().to(dev()), torch.randint(0, v, (n, m), generator=torch.Generator().manual_seed(1)).to(dev())
    g, gt = torch.ones(n, m, device=dev()), torch.ones(n, k, device=dev())
    f = itl.token_logp_fwd(x, tok, top_k=k)
    e = itl.linear_token_logp_fwd(a, b, tok, top_k=k)
    tops = dict(top_ids=f.top_ids, grad_top_logp=gt)
    d = itl.token_logp_bwd(x, f.lse, tok, g, **tops)
    assert torch.equal(itl.token_logp_bwd(x.view(2, 2, v), f.lse, tok.view(2, 2, m), g, **tops).view(n, v), d)
    for bad in (g.t().contiguous(), g.view(-1)):
        with pytest.raises(ValueError, match="grad_logp"):
            itl.token_logp_bwd(x, f.lse, tok, bad)
        with pytest.raises(ValueError, match="grad_logp"):
            itl.linear_token_logp_bwd(a, b, e.lse, tok, e.logp, bad)
    with pytest.raises(ValueError, match="grad_top_logp"):
        itl.token_logp_bwd(x, f.lse, tok, g, top_ids=f.top_ids, grad_top_logp=gt.t())


def test_backwards_refuse_a_gradient_without_its_tokens():
    n, v, h, m, k = 4, 300, 64, 3, 2
    a, b, z = head_operands(n, h, v, False, seed=9)
    x, g, gt = z.float().to(dev()), torch.ones(n, m, device=dev()), torch.ones(n, k, device=dev())
    f, e = itl.token_logp_fwd(x, None, top_k=k), itl.linear_token_logp_fwd(a, b, None, top_k=k)
    with pytest.raises(ValueError, match="token_ids"):
        itl.token_logp_bwd(x, f.lse, None, g, top_ids=f.top_ids, grad_top_logp=gt)
    with pytest.raises(ValueError, match="token_ids"):
        itl.linear_token_logp_bwd(a, b, e.lse, None, g, g, top_ids=e.top_ids, top_logp=e.top_logp, grad_top_logp=gt)
    # no tokens, and a gradient of none of them
    leaf = x.clone().requires_grad_()
    r = itl.batch_invariant_token_logp(leaf, None, top_k=k)
    (r.logp.sum() + r.top_logp.sum()).backward()
    assert torch.isfinite(leaf.grad).all()


@pytest.mark.parametrize("h", [100, 2048])
def test_norm_writes_a_given_sum_without_a_residual(h):
    gen = torch.Generator().manual_seed(h)
    x = torch.randn(5, h, generator=gen).to(dev(), torch.bfloat16)
    w = torch.ones(h, dtype=torch.bfloat16, device=dev())
    y, _, _ = itl.rms_norm_fwd(x, w)
    for norm in (lambda t, s: itl.rms_norm_fwd(t, w, sum_out=s)[:2], lambda t, s: itl.rms_norm_quantized(t, w, sum_out=s)):
        buf = torch.full_like(x, 7.0)
        _, s = norm(x, buf)
        assert s is buf and torch.equal(buf, x)
        own = x.clone()  # in place
        _, s = norm(own, own)
        assert s is own and torch.equal(own, x)
    own, buf = x.clone(), torch.empty_like(x)  # y over x, x kept beside it
    y2, s, _ = itl.rms_norm_fwd(own, w, y_out=own, sum_out=buf)
    assert torch.equal(own, y) and torch.equal(buf, x)


def test_saved_logits_that_overlap_are_refused():
    n, v, h = 4, 304, 64
    a, b, z = head_operands(n, h, v, False, seed=11)
    tok = torch.randint(0, v, (n, 1), generator=torch.Generator().manual_seed(1)).to(dev())
    f = itl.linear_token_logp_fwd(a, b, tok)
    g = torch.ones(n, 1, device=dev())
    one = z[:1].float().to(dev())
    for bad in (one.expand(n, v), torch.zeros(4 * v, device=dev()).as_strided((n, v), (v - 4, 1))):
        with pytest.raises(itl.LogpError) as e:
            itl.linear_token_logp_bwd(a, b, f.lse, tok, f.logp, g, saved_logits=bad)
        assert e.value.status == itl._lib.LOGP_ERR_SHAPE
        with pytest.raises(itl.LogpError) as e:
            itl.linear_logp_bwd(a, b, tok[:, 0], f.lse, g[:, 0], saved_logits=bad)
        assert e.value.status == itl._lib.LOGP_ERR_SHAPE
    dh, _ = itl.linear_token_logp_bwd(a, b, f.lse, tok, f.logp, g)
    assert torch.equal(itl.linear_token_logp_bwd(a, b, f.lse, tok, f.logp, g, saved_logits=z.float().to(dev()))[0], dh)
    d1, _ = itl.linear_token_logp_bwd(a[:1], b, f.lse[:1], tok[:1], f.logp[:1], g[:1], saved_logits=one)
    assert torch.equal(d1, dh[:1])


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("n,v", [(2, 163840), (5, 163841), (140, 164100), (600, 201088), (3, 262144)])
def test_head_past_one_block_of_tiles(n, v, q8):
    """Vocabularies around 163840 columns, where the tables of a row no longer
    fit one block of registers in the merge and in the selection; rows on both
    sides of every tile and of two waves a row, a row alone, a row of equal
    logits.  The merge's chain over T tiles is off by at most T 2^-24 in the sum
    and the moment, which moves the entropy by twice that of the mean distance
    to the maximum."""
    h, k = 64, 20
    a, b, _ = head_operands(n, h, v, q8, seed=v)
    if q8:
        a.data.view(torch.uint8)[1] = 0
        hd, wd = a.data.cpu().double(), b.data.cpu().double() * b.scale.cpu().double()[:, None]
    else:
        a[1] = 0.0
        hd, wd = a.cpu().double(), b.cpu().double()
    rows = sorted({0, 1, n // 2, n - 1})
    tok = torch.randint(0, v, (n, 2), generator=torch.Generator().manual_seed(3))
    tok[0] = torch.tensor([v - 1, 0])
    r = itl.linear_token_logp_fwd(a, b, tok.to(dev()), top_k=k, temperature=16.0, return_entropy=True)
    x = hd[rows] @ wd.T / 16.0  # exact
    ref = token_scores(x, tok[rows], k)
    at = lambda t: t[rows].double().cpu()  # noqa: E731
    assert torch.equal(r.top_ids[rows].cpu(), ref["top_ids"])
    for got, want in ((r.logp, ref["logp"]), (r.lse, ref["lse"]), (r.top_logp, ref["top_logp"])):
        assert ((at(got) - want).abs() <= ATOL + RTOL * want.abs()).all()
    chain = 2 * (v + 127) // 128 * 2.0 ** -24 * (x.amax(1) - ref["lse"] + ref["entropy"])
    assert ((at(r.entropy) - ref["entropy"]).abs() <= ATOL + RTOL * ref["entropy"] + chain).all()
    for i in rows:
        one = itl.QuantizedRows(a.data[i:i + 1], a.scale[i:i + 1]) if q8 else a[i:i + 1]
        s = itl.linear_token_logp_fwd(one, b, tok[i:i + 1].to(dev()), top_k=k, temperature=16.0, return_entropy=True)
        same([t[i:i + 1] for t in r], s)


@pytest.mark.parametrize("bf16", [False, True])
def test_gradient_through_segments_of_the_vocabulary(bf16):
    """Three segments of 4096 columns, with several tokens (one twice, one
    invalid, some at a segment's edge), alternatives, entropy and temperature:
    few rows (every segment a product of its own, then their sum) against
    float64 within test_gpu_linear_tokens' bounds; many rows (a tile walks the
    segments) give a row the bits of the few; dweight of the many against
    float64.  The workspace tells which of the two runs."""
    h, v, few, many, m, k, temp = 320, 9000, 6, 16640, 3, 4, 0.7
    gen = torch.Generator().manual_seed(8)
    hid = (torch.randn(many, h, generator=gen) * 16).round().clamp(-127, 127) / 16
    w = (torch.randn(v, h, generator=gen) * 51).round().clamp(-127, 127) / 1024
    tok = torch.randint(0, v, (many, m), generator=gen)
    tok[0, 1] = tok[0, 0]
    tok[1] = -100
    tok[2, 0] = v + 5
    tok[3] = torch.tensor([4095, 4096, 8192])
    tok[4, 0] = v - 1
    g, gt, ge = torch.randn(many, m, generator=gen), torch.randn(many, k, generator=gen), torch.randn(many, generator=gen)
    out = torch.bfloat16 if bf16 else torch.float32
    b = w.to(dev(), torch.bfloat16)
    pw = itl.prepare_weight(b)
    ops = [t.to(dev()) for t in (hid.to(torch.bfloat16), tok, g, gt, ge)]

    def grads(part, **kw):
        a, t, gp, gtp, gep = (o[part] for o in ops)
        f = itl.linear_token_logp_fwd(a, b, t, top_k=k, temperature=temp, return_entropy=True)
        return itl.linear_token_logp_bwd(a, b, f.lse, t, f.logp, gp, f.top_ids, f.top_logp, gtp, temperature=temp,
                                         entropy=f.entropy, grad_entropy=gep, out_dtype=out, **kw), f

    def need(n, chunk=0):
        flags = _lib.LOGP_BWD_DHIDDEN | _lib.LOGP_BWD_DWEIGHT
        np_, vc = (n + 255) // 256 * 256, min(chunk or 32768, 9216)
        rest = 2 * np_ * h * 2 + np_ * vc * 2  # the hidden rows twice, dz
        return _lib.lib().linear_token_logp_bwd_workspace_bytes(n, h, v, flags, chunk) - rest

    assert need(few) >= 3 * few * h * 4                # every segment's part
    assert need(many) < 4 * many * h and need(many, 8192) < 4 * many * h  # none: the tiles walk

    (dh, dw), f = grads(slice(0, few))
    inv = 1.0 / temp
    wd, hd = w.double(), hid[:few].double()
    dx, size = token_gradient(hd @ wd.T * inv, tok[:few], g[:few], f.top_ids.cpu(), gt[:few], ge[:few])
    dz, size = dx * inv, size * inv
    half = 2.0 ** -8 if bf16 else 0.0

    def inside(got, want, bound):
        assert ((got.double() - want).abs() <= bound + half * (want.abs() + bound)).all()

    inside(dh.cpu(), dz @ wd, 2.0 ** -8 * dz.abs() @ wd.abs() + 1e-4 * size @ wd.abs() + 1e-6)
    inside(dw.cpu(), dz.T @ hd, 2.0 ** -8 * dz.abs().T @ hd.abs() + 1e-4 * size.T @ hd.abs() + 1e-6)
    for kw in (dict(vocab_chunk=4096), dict(vocab_chunk=8192), dict(prepared_weight=pw), dict(prepared_weight=pw, vocab_chunk=8192)):
        (d2, w2), _ = grads(slice(0, few), **kw)
        assert torch.equal(d2, dh) and torch.equal(w2, dw), kw.keys()
    (dhm, dwm), fm = grads(slice(0, many))
    assert torch.equal(dhm[:few], dh) and not dhm[1].any()
    tail = slice(many - few, many)
    assert torch.equal(dhm[tail], grads(tail)[0][0])
    for kw in (dict(vocab_chunk=4096), dict(vocab_chunk=8192), dict(prepared_weight=pw), dict(prepared_weight=pw, vocab_chunk=8192),
               dict(need_dweight=False), dict(need_dweight=False, vocab_chunk=8192)):
        (d2, w2), _ = grads(slice(0, many), **kw)
        assert torch.equal(d2, dhm) and (w2 is None or torch.equal(w2, dwm)), kw.keys()
    # dweight of all rows, the formula in 64 bits on the device
    hd, wd = ops[0].double(), b.double()
    x = torch.mm(hd, wd.t().contiguous()) * inv
    lse = torch.logsumexp(x, 1, keepdim=True)
    p = torch.exp(x - lse)
    given = ops[1] != -100
    act = given.any(1, keepdim=True).double()
    gd, gtd = ops[2].double() * given, ops[3].double() * act
    logp = x - lse
    ent = -(p * logp).sum(1, keepdim=True)
    total = (gd.sum(1) + gtd.sum(1))[:, None]
    gent = ops[4].double()[:, None]
    d = (-p * total - gent * p * (logp + ent)) * act
    size = (p * (gd.abs().sum(1) + gtd.abs().sum(1))[:, None] + gent.abs() * p * (logp.abs() + ent)) * act
    inside_v = (ops[1] >= 0) & (ops[1] < v)
    d.scatter_add_(1, ops[1].clamp(0, v - 1), gd * inside_v)
    size.scatter_add_(1, ops[1].clamp(0, v - 1), gd.abs() * inside_v)
    d.scatter_add_(1, fm.top_ids.clamp(min=0), gtd)
    size.scatter_add_(1, fm.top_ids.clamp(min=0), gtd.abs())
    d, size = (d * inv).t().contiguous(), (size * inv).t().contiguous()
    inside(dwm, torch.mm(d, hd), 2.0 ** -8 * torch.mm(d.abs(), hd.abs()) + 1e-4 * torch.mm(size, hd.abs()) + 1e-6)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n,v", [(3, 163841), (600, 164100), (2, 262144)])
def test_logits_past_one_block_of_groups(n, v, dtype):
    """The same from logits: more groups of 128 columns (64 of fp32) than the
    selection's registers hold at once; a row of equal logits, a row alone."""
    gen = torch.Generator().manual_seed(v)
    rows = sorted({0, 1, n - 1})
    x = torch.zeros(n, v, dtype=dtype, device=dev())
    some = (3 * torch.randn(len(rows), v, generator=gen)).to(dtype)
    some[1] = 0.5
    x[rows] = some.to(dev())
    tok = torch.randint(0, v, (n, 2), generator=gen)
    for k in (1, 20, 64):
        r = itl.token_logp_fwd(x, tok.to(dev()), top_k=k, return_entropy=True)
        ref = token_scores(some.double(), tok[rows], k)
        assert torch.equal(r.top_ids[rows].cpu(), ref["top_ids"])
        for got, want in ((r.logp, ref["logp"]), (r.lse, ref["lse"]), (r.top_logp, ref["top_logp"])):
            assert ((got[rows].double().cpu() - want).abs() <= ATOL + RTOL * want.abs()).all()
        for i in rows:
            same([t[i:i + 1] for t in r], itl.token_logp_fwd(x[i:i + 1], tok[i:i + 1].to(dev()), top_k=k,
                                                             return_entropy=True))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_entropy_beside_tiles_of_the_lowest_value(dtype):
    """Whole tiles masked with the type's lowest value (and with -inf, or far
    below the rest) add nothing to the entropy."""
    v, low = 3 * 4096 + 5, torch.finfo(dtype).min
    x = (3 * torch.randn(5, v, generator=torch.Generator().manual_seed(6))).to(dtype)
    x[0, 4096:8192] = low
    x[1, 5:] = low
    x[2, 4096:] = -torch.inf
    x[2, 8192:] = low
    x[3, :4096] = low / 4
    ref = token_scores(x.double(), None, 0)
    near = torch.where(x.double() < -1e4, 0.0, x.double())  # masked columns carry no weight
    bound = ATOL + RTOL * ref["entropy"] + 1e-6 * (near.amax(1) - near.amin(1))
    xd, t = x.to(dev()), torch.zeros(5, dtype=torch.int64, device=dev())
    r = itl.token_logp_fwd(xd, None, top_k=3, return_entropy=True)
    for got in (r.entropy, itl.logp_fwd(xd, t, return_entropy=True)[2]):
        assert ((got.double().cpu() - ref["entropy"]).abs() <= bound).all()
    d = itl.token_logp_bwd(xd, r.lse, entropy=r.entropy, grad_entropy=torch.ones(5, device=dev()))
    assert torch.isfinite(d).all() and (d[0, 4096:8192] == 0).all() and (d[1, 5:] == 0).all()


@pytest.mark.parametrize("q8", [False, True])
def test_entropy_of_the_head_beside_far_tiles(q8):
    """A whole tile whose logits are near the lowest fp32 value."""
    h, v = 64, 1000
    gen = torch.Generator().manual_seed(7)
    hid, w = torch.ones(3, h), torch.randint(-4, 5, (v, h), generator=gen).float() / 64
    w[256:512] = 0.0
    big = 2.0 ** 127  # times -1.75 = -2.98e38
    if q8:
        w[256:512, 0] = -1.75
        scale = torch.ones(v)
        scale[256:512] = big
        a = itl.QuantizedRows(hid.to(dev()).to(torch.float8_e4m3fn), torch.ones(3, device=dev()))
        b = itl.QuantizedRows(w.to(dev()).to(torch.float8_e4m3fn), scale.to(dev()))
    else:
        w[256:512, 0] = -1.75 * big
        a, b = hid.to(dev(), torch.bfloat16), w.to(dev(), torch.bfloat16)
    x = hid.double() @ w.double().T
    x[:, 256:512] = -1.75 * big
    ref = token_scores(x, None, 0)
    r = itl.linear_token_logp_fwd(a, b, None, return_entropy=True)
    for got, want in ((r.lse, ref["lse"]), (r.entropy, ref["entropy"])):
        assert ((got.double().cpu() - want).abs() <= 2 * ATOL + RTOL * want.abs()).all()
    if not q8:
        got = itl.linear_logp_fwd(a, b, torch.zeros(3, dtype=torch.int64, device=dev()), return_entropy=True)[2]
        assert ((got.double().cpu() - ref["entropy"]).abs() <= 2 * ATOL + RTOL * ref["entropy"]).all()


@pytest.mark.parametrize("value", [torch.nan, torch.inf])
@pytest.mark.parametrize("n", [6, 40, 300])
def test_what_a_padding_row_holds_stays_there(n, value):
    """Hidden rows, gradients and kept logits of padding rows may be anything:
    no output and no gradient of the batch shows it, dweight included."""
    h, v = 128, 1000
    gen = torch.Generator().manual_seed(n)
    a = torch.randn(n, h, generator=gen).to(dev(), torch.bfloat16)
    b = (0.05 * torch.randn(v, h, generator=gen)).to(dev(), torch.bfloat16)
    tok = torch.randint(0, v, (n, 2), generator=gen).to(dev())
    pads = [2, n - 1]
    tok[pads] = -100
    g, ge = torch.randn(n, 2, generator=gen).to(dev()), torch.randn(n, generator=gen).to(dev())
    pw = itl.prepare_weight(b)

    def tokens(fill, saved, out, prepared):
        x, gx, gex = a.clone(), g.clone(), ge.clone()
        z = torch.zeros(n, v, device=dev()) if saved else None
        for t in (x, gx, gex):
            t[pads] = fill
        f = itl.linear_token_logp_fwd(x, b, tok, top_k=3, return_entropy=True, logits_out=z)
        if saved:
            z[pads] = fill
        gt = torch.full((n, 3), 0.5, device=dev())
        gt[pads] = fill
        return (*f, *itl.linear_token_logp_bwd(x, b, f.lse, tok, f.logp, gx, f.top_ids, f.top_logp, gt, entropy=f.entropy,
                                               grad_entropy=gex, saved_logits=z, out_dtype=out, prepared_weight=prepared))

    def single(fill, t):
        x, gx = a.clone(), g[:, 0].clone()
        x[pads] = fill
        gx[pads] = fill
        logp, lse = itl.linear_logp_fwd(x, b, t)
        return logp, lse, *itl.linear_logp_bwd(x, b, t, lse, gx)

    for saved, out, prepared in ((False, torch.float32, None), (True, torch.bfloat16, None), (False, torch.bfloat16, pw)):
        for one, two in zip(tokens(0.0, saved, out, prepared), tokens(value, saved, out, prepared)):
            assert torch.isfinite(two).all() and torch.equal(one, two)
    for t in (tok[:, 0].contiguous(), tok[:, 0].int()):
        for one, two in zip(single(0.0, t), single(value, t)):
            assert torch.isfinite(two).all() and torch.equal(one, two)


def test_heads_on_two_streams_at_once():
    """Both heads on two streams, many rows (the tile queue is in the call's own
    workspace) and few, forward and backward: the bits of one call after the other."""
    cases = []
    for n, seed in ((700, 1), (40, 2)):
        a, b, _ = head_operands(n, 128, 6000, False, seed)
        qa, qb, _ = head_operands(n, 128, 6000, True, seed)
        tok = torch.randint(0, 6000, (n, 2), generator=torch.Generator().manual_seed(seed)).to(dev())
        cases.append((a, b, qa, qb, tok, torch.ones(n, 2, device=dev())))

    def run(a, b, qa, qb, tok, g):
        f = itl.linear_token_logp_fwd(a, b, tok, top_k=5, return_entropy=True)
        dh, dw = itl.linear_token_logp_bwd(a, b, f.lse, tok, f.logp, g)
        return [*f, dh, dw, *itl.linear_token_logp_fwd(qa, qb, tok, top_k=5, return_entropy=True)]

    want = [run(*c) for c in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for c in cases:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(run(*c))
        torch.cuda.synchronize()
        for x, y in zip(want, got):
            same(x, y)


@pytest.mark.parametrize("n", [30, 16400])
def test_graph_replays_of_the_segmented_backward(n):
    """The backward through several vocabulary segments, in parts (30 rows) and
    walked (16400), captured and replayed with new inputs and eager work between."""
    h, v, m, k = 320, 9000, 2, 3
    a = torch.zeros(n, h, dtype=torch.bfloat16, device=dev())
    tok = torch.zeros(n, m, dtype=torch.int64, device=dev())
    g, gt = torch.zeros(n, m, device=dev()), torch.zeros(n, k, device=dev())
    w = (0.05 * torch.randn(v, h, generator=torch.Generator().manual_seed(1))).to(dev(), torch.bfloat16)

    def step():
        f = itl.linear_token_logp_fwd(a, w, tok, top_k=k, return_entropy=True)
        return [*f, *itl.linear_token_logp_bwd(a, w, f.lse, tok, f.logp, g, f.top_ids, f.top_logp, gt, entropy=f.entropy,
                                               grad_entropy=g[:, 0].contiguous(), out_dtype=torch.bfloat16)]

    def fill(seed):
        gen = torch.Generator(dev()).manual_seed(seed)
        a.normal_(generator=gen)
        tok.copy_(torch.randint(0, v, (n, m), generator=gen, device=dev()))
        tok[seed] = -100
        g.normal_(generator=gen)
        gt.normal_(generator=gen)

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
        for i, (x, y) in enumerate(zip(out, step())):
            assert torch.equal(x, y), (seed, i)
        torch.cuda.synchronize()


@pytest.mark.parametrize("n", [5, 16640])
def test_strided_outputs_of_the_segmented_backward(n):
    """dhidden and dweight in views with longer, unaligned rows, in parts and
    walked: the same bits, and nothing written beside them."""
    h, v = 320, 9000
    a, b, _ = head_operands(n, h, v, False, seed=n)
    tok = torch.randint(0, v, (n, 2), generator=torch.Generator().manual_seed(n)).to(dev())
    g = torch.randn(n, 2, generator=torch.Generator().manual_seed(n)).to(dev())
    f = itl.linear_token_logp_fwd(a, b, tok, temperature=50.0)
    for dtype in (torch.float32, torch.bfloat16):
        want = itl.linear_token_logp_bwd(a, b, f.lse, tok, f.logp, g, temperature=50.0, out_dtype=dtype)
        bufs = [torch.full((rows, h + 5), 9.0, dtype=dtype, device=dev()) for rows in (n, v)]
        got = itl.linear_token_logp_bwd(a, b, f.lse, tok, f.logp, g, temperature=50.0, out_dtype=dtype,
                                        dhidden_out=bufs[0][:, 3:h + 3], dweight_out=bufs[1][:, 3:h + 3])
        for x, y, buf in zip(want, got, bufs):
            assert torch.equal(x, y) and (buf[:, :3] == 9).all() and (buf[:, h + 3:] == 9).all()
