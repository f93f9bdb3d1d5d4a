"""4-bit rows and the LM head on them.

The quantisation is compared exactly with its definition.  The head's outputs are
compared bit for bit with the bf16 head on the decoded weight (whose values are
exact in bf16; tests/test_gpu_linear_tokens.py holds that head to the float64
forms), and once with the float64 form itself, within the bound stated there for
log-probabilities, 1e-5 + 1e-5 of the value."""

import pytest
import torch

import invariant_token_log_amd as itl
from gpu_helpers import bits, dev
from layer_reference import TYPES, fp4_values, to_fp4
from token_reference import token_scores

pytestmark = pytest.mark.gpu


def table(v, h, seed=0, pad=0):
    gen = torch.Generator().manual_seed(seed)
    data = torch.randint(0, 256, (v, h // 2), generator=gen, dtype=torch.uint8)
    scale = torch.randint(116, 122, (v, h // 32), generator=gen, dtype=torch.uint8)
    q = itl.Fp4Rows(torch.zeros(v, h // 2 + 16 * pad, dtype=torch.uint8, device=dev())[:, :h // 2].copy_(data),
                    torch.zeros(v, h // 32 + pad, dtype=torch.uint8, device=dev())[:, :h // 32].copy_(scale))
    return q, fp4_values(data, scale)


def rows(n, h, seed=1):
    return torch.randn(n, h, generator=torch.Generator().manual_seed(seed)).bfloat16()


def given(n, v, m, seed=2):
    gen = torch.Generator().manual_seed(seed)
    t = torch.randint(0, v, (n, m), generator=gen)
    t[torch.rand(n, m, generator=gen) < 0.1] = -100
    return t.to(dev())


def same(a, b):
    for x, y, name in zip(a, b, a._fields):
        if x is None:
            assert y is None
        else:
            assert torch.equal(x if x.dtype == torch.int64 else bits(x), y if y.dtype == torch.int64 else bits(y)), name


@pytest.mark.parametrize("n,h,v", [(1, 64, 1), (1, 64, 300), (5, 128, 256), (3, 192, 257), (16, 256, 1000), (32, 320, 515),
                                   (33, 448, 5003), (64, 512, 300), (65, 576, 700), (200, 1024, 999), (256, 1600, 513),
                                   (448, 448, 1100), (449, 448, 1100), (500, 1024, 5003), (7, 4096, 3001), (40, 4096, 777),
                                   (128, 192, 513), (129, 64, 300), (129, 128, 1), (150, 192, 257), (257, 320, 515),
                                   (511, 576, 5003), (130, 4096, 777), (1025, 1088, 4097)])
def test_head_has_the_bits_of_the_decoded_weight(n, h, v):
    q, values = table(v, h)
    w = values.bfloat16().to(dev())
    assert torch.equal(w.double().cpu(), values)
    x = rows(n, h).to(dev())
    k = min(v, 7)
    for m, top, ent, temp, rounded in ((1, 0, False, 1.0, False), (1, k, True, 0.7, False), (3, k, False, 1.0, True),
                                       (0, 1, True, 1.3, False), (4, 0, True, 1.0, False), (1, 0, True, 1.0, True)):
        tok = given(n, v, m) if m else None
        kw = dict(top_k=top, return_entropy=ent, temperature=temp, round_logits=rounded)
        same(itl.linear_token_logp_fwd(x, q, tok, **kw), itl.linear_token_logp_fwd(x, w, tok, **kw))


@pytest.mark.parametrize("n", [9, 460])
def test_head_against_the_definition(n):
    h, v = 256, 2001
    q, values = table(v, h, 5)
    x, tok = rows(n, h), given(n, v, 2)
    got = itl.linear_token_logp_fwd(x.to(dev()), q, tok, top_k=5, return_entropy=True)
    ref = token_scores(x.double() @ values.T, tok, 5)
    for name in ("logp", "lse", "entropy", "top_logp"):
        a, b = getattr(got, name).double().cpu(), ref[name]
        assert ((a - b).abs() <= 1e-5 + 1e-5 * b.abs()).all(), name


def test_rows_alone_strided_and_chunked():
    h, v = 384, 901
    q, values = table(v, h)
    wide, _ = table(v, h, pad=3)
    x = rows(600, h)
    buf = torch.zeros(600, h + 8, dtype=torch.bfloat16, device=dev())[:, :h].copy_(x)
    tok = given(600, v, 1)
    whole = itl.linear_token_logp_fwd(x.to(dev()), q, tok, top_k=3)
    same(itl.linear_token_logp_fwd(buf, wide, tok, top_k=3), whole)
    same(itl.linear_token_logp_fwd(buf, wide, tok.int(), top_k=3, row_chunk=256), whole)
    for lo, hi in ((0, 1), (10, 40), (100, 200), (30, 478), (30, 479)):
        part = itl.linear_token_logp_fwd(x[lo:hi].to(dev()), wide, tok[lo:hi], top_k=3)
        same(part, itl.TokenLogp(whole.logp[lo:hi], whole.lse[lo:hi], None, whole.top_logp[lo:hi], whole.top_ids[lo:hi]))
    lead = itl.linear_token_logp_fwd(x[:0].to(dev()), q, tok[:0], top_k=3)
    assert lead.logp.shape == (0, 1)


@pytest.mark.parametrize("n", [4, 470])
def test_scales_of_nan_and_the_ends(n):
    """A group of NaN makes its column's logit NaN in every row; the smallest and
    the greatest scales decode as the bf16 values they stand for."""
    h, v = 128, 300
    q, _ = table(v, h)
    q.scale[7, 1] = 0
    q.scale[8, 0] = 1
    x = rows(n, h)
    w = fp4_values(q.data, q.scale).bfloat16().to(dev())
    tok = given(n, v, 1)
    same(itl.linear_token_logp_fwd(x.to(dev()), q, tok, top_k=4), itl.linear_token_logp_fwd(x.to(dev()), w, tok, top_k=4))
    q.scale[250, 2] = 255
    r = itl.linear_token_logp_fwd(x.to(dev()), q, None, top_k=4)
    assert r.lse.isnan().all() and (r.top_ids != 250).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize(dtype):
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(9, 96, generator=gen) * torch.exp2(torch.randint(-20, 20, (9, 3), generator=gen)).repeat_interleave(32, 1)
    if dtype == "fp16":
        x = x.clamp(-60000, 60000)
    x[0] = 0.0
    x[1, :32] = torch.tensor([6.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25] * 2 + [-6.0, -5.0, -3.5, -2.5, -1.75, -1.25, -0.75, -0.25] * 2)
    x[1, 32:64] = x[1, :32] * 1.0078125  # a step of bf16 past each tie
    x[1, 64:] = 6.0
    x[2, 5], x[3, 40], x[4, 95] = torch.nan, torch.inf, -torch.inf
    x = x.to(TYPES[dtype])
    q = itl.quantize_rows_fp4(x.to(dev()))
    codes, scales = to_fp4(x.double())
    assert torch.equal(q.scale.cpu().long(), scales)
    data = q.data.cpu().long()
    live = (scales != 255).repeat_interleave(32, 1)
    got = torch.stack([data & 15, data >> 4], 2).flatten(1)
    assert torch.equal(got[live], codes[live])
    value = itl.embedding_fwd(torch.arange(9, device=dev()), q, out_dtype=torch.float32).cpu()
    assert value[~live].isnan().all() and torch.equal(value[live].double(), fp4_values(q.data, q.scale)[live])


def test_quantize_ends_of_the_range():
    """The largest finite values saturate, the smallest keep the least scale."""
    most = torch.finfo(torch.float32).max
    x = torch.zeros(4, 32)
    x[0, :3] = torch.tensor([most, -most, most / 4])
    x[1, :2] = torch.tensor([2.0 ** -126, -2.0 ** -140])
    x[2, :2] = torch.tensor([6 * 2.0 ** 125, 4.9 * 2.0 ** 125])
    x[3, 0] = 6.1 * 2.0 ** -126
    q = itl.quantize_rows_fp4(x.to(dev()))
    assert q.scale.flatten().tolist() == [252, 1, 252, 2]
    value = itl.embedding_fwd(torch.arange(4, device=dev()), q, out_dtype=torch.float32).cpu().double()
    assert value[0, :3].tolist() == [6 * 2.0 ** 125, -6 * 2.0 ** 125, 2.0 ** 126]
    assert value[1, :2].tolist() == [2.0 ** -126, 0.0] and value[3, 0] == 6 * 2.0 ** -126


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_shapes(dtype):
    for n, h, pad in ((1, 32, 0), (3, 64, 5), (2000, 96, 0), (5, 4096, 8), (2, 20000, 0)):
        x = torch.randn(n, h, generator=torch.Generator().manual_seed(n)).to(TYPES[dtype])
        buf = torch.zeros(n, h + pad, dtype=x.dtype, device=dev())[:, :h].copy_(x)
        q = itl.quantize_rows_fp4(buf)
        value = fp4_values(q.data, q.scale)
        scale = 2.0 ** (q.scale.cpu().double() - 127)
        step = scale.repeat_interleave(32, 1)
        # half the distance between neighbours: 1/4 below 2, 1/2 to 4, 1 to 6
        a = x.double().abs() / step
        assert (a.view(n, -1, 32).amax(2) <= 6).all() and (a.view(n, -1, 32).amax(2) > 3).all()
        assert ((value - x.double()).abs() <= step * torch.where(a < 2, 0.25, torch.where(a < 4, 0.5, 1.0))).all()
    assert itl.quantize_rows_fp4(torch.empty(0, 64, device=dev())).data.shape == (0, 32)


def test_tied_table_from_tokens_to_tokens():
    """One 4-bit table at both ends: lookup, norm, head, as a decoding step runs
    them; captured and replayed with new tokens."""
    v, h, n = 3000, 512, 12
    weight = torch.randn(v, h, generator=torch.Generator().manual_seed(0)).mul_(0.05)
    q = itl.quantize_rows_fp4(weight.bfloat16().to(dev()))
    norm = torch.ones(h, dtype=torch.bfloat16, device=dev())
    ids = torch.zeros(n, dtype=torch.int64, device=dev())

    def step():
        x = itl.embedding_fwd(ids, q, scale=h ** 0.5)
        return itl.norm_linear_token_logp(x, norm, q, ids[:, None], top_k=4)

    with torch.no_grad():
        step()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        w = fp4_values(q.data, q.scale)
        for k in range(3):
            ids.copy_(torch.randint(0, v, (n,), generator=torch.Generator().manual_seed(k)))
            graph.replay()
            torch.cuda.synchronize()
            same(step(), out)
            x = (w[ids.cpu()].float() * torch.tensor(h ** 0.5)).bfloat16()
            y, _, _ = itl.rms_norm_fwd(x.to(dev()), norm)
            ref = token_scores(y.double().cpu() @ w.T, ids[:, None], 4)
            assert ((out.logp.double().cpu() - ref["logp"]).abs() <= 1e-5 + 1e-5 * ref["logp"].abs()).all()
            assert ((out.top_logp.double().cpu() - ref["top_logp"]).abs() <= 1e-5 + 1e-5 * ref["top_logp"].abs()).all()


def test_no_gradient():
    q, _ = table(100, 64)
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device=dev(), requires_grad=True)
    w = torch.ones(64, dtype=torch.bfloat16, device=dev())
    with pytest.raises(ValueError, match="no gradient"):
        itl.norm_linear_token_logp(x, w, q)
    with pytest.raises(ValueError, match="4-bit head takes no"):
        itl.norm_linear_token_logp(x.detach(), w, q, save_logits=True)


@pytest.mark.parametrize("n", [60, 100, 700])
def test_head_captured_and_on_two_streams(n):
    """Each kernel of the head replayed with new rows between eager calls, and two
    calls at once."""
    h, v = 512, 9000
    q, _ = table(v, h)
    x, tok = rows(n, h).to(dev()), given(n, v, 1)

    def run():
        return itl.linear_token_logp_fwd(x, q, tok, top_k=3, return_entropy=True)

    run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for k in range(3):
        x.copy_(rows(n, h, seed=10 + k))
        graph.replay()
        torch.cuda.synchronize()
        same(run(), out)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for st in streams:
        with torch.cuda.stream(st):
            outs.append(run())
    torch.cuda.synchronize()
    same(outs[0], out)
    same(outs[1], out)


def alike(a, b):
    """same, any NaN being like another."""
    for x, y, name in zip(a, b, a._fields):
        if x is not None:
            assert torch.equal(x.isnan(), y.isnan()) and torch.equal(x[~x.isnan()], y[~y.isnan()]), name


@pytest.mark.parametrize("n", [4, 20, 40, 100, 470])
@pytest.mark.parametrize("h", [128, 192])
@pytest.mark.parametrize("lo,hi,codes", [(0, 0, 0xFF), (1, 1, 0xFF), (0, 3, 0xFF), (2, 2, 0xFF), (127, 128, 0xFF), (126, 129, 0xFF),
                                         (199, 202, 0xFF), (252, 252, 0xFF), (249, 252, 0xFF), (253, 253, 0xBB), (251, 254, 0xBB)])
def test_every_scale_reaches_the_logits(lo, hi, codes, h, n):
    """All groups of all columns have scale bytes from lo to hi, and the hidden rows a
    power of two that brings the logits near 1 to 100 (past 252 magnitudes up to 3/2: greater
    ones pass the range).  Hidden values are eighths and codes halves of powers of two: with
    three bits of the scales' span a logit is a sum of 192 multiples of a unit, each at most 15
    * 12 * 8 of it, so below 2^24 units and exact in fp32, whatever the order.  So
    log-probabilities are off by the stated 1e-5 + 1e-5 of the value and by the rounding of
    the log-sum-exp, 2^-24 of it."""
    v = 300
    gen = torch.Generator().manual_seed(lo + h)
    data = torch.randint(0, 256, (v, h // 2), generator=gen, dtype=torch.uint8) & codes
    scale = torch.randint(lo, hi + 1, (v, h // 32), generator=gen, dtype=torch.uint8)
    values = fp4_values(data, scale)
    w = values.bfloat16()
    assert torch.equal(w.double(), values)
    power = min(max(124 - hi, -125), 124)
    x = torch.randint(8, 16, (n, h), generator=gen) * (2 * torch.randint(0, 2, (n, h), generator=gen) - 1)
    x = (x.double() * 2.0 ** (power - 3)).bfloat16()
    z = x.double() @ values.T
    assert (z != 0).float().mean() > 0.9 and torch.equal(z.float().double(), z) and 0.1 < z.abs().max() < 1000
    tok = given(n, v, 3)
    kw = dict(top_k=64, return_entropy=True)
    got = itl.linear_token_logp_fwd(x.to(dev()), itl.Fp4Rows(data.to(dev()), scale.to(dev())), tok, **kw)
    same(got, itl.linear_token_logp_fwd(x.to(dev()), w.to(dev()), tok, **kw))
    ref = token_scores(z, tok, 64)
    for name in ("logp", "lse", "top_logp"):
        a, b = getattr(got, name).double().cpu(), ref[name]
        assert ((a - b).abs() <= 1e-5 + 1e-5 * b.abs() + 2.0 ** -24 * ref["lse"].abs().view(-1, *[1] * (b.dim() - 1))).all(), name


@pytest.mark.parametrize("n", [4, 20, 40, 100, 470])
@pytest.mark.parametrize("b,least", [(253, 4), (254, 2)])
def test_values_past_the_range_are_infinities(b, least, n):
    """Under the scale bytes 253 and 254 magnitudes from 4 and from 2 on: their column's
    logit is an infinity, or a NaN where both signs meet; others keep theirs."""
    h, v = 128, 300
    q, _ = table(v, h)
    code = {2: 4, 4: 6}[least]
    x = rows(n, h).abs().clamp(min=0.25)
    tok = torch.tensor([[3, 7, 8, 200]]).repeat(n, 1).to(dev())
    without = itl.linear_token_logp_fwd(x.to(dev()), q, tok, top_k=20)
    q.scale[7], q.data[7] = b, 0x11 * (code | 8)  # an infinity below
    got = itl.linear_token_logp_fwd(x.to(dev()), q, tok, top_k=20, return_entropy=True)
    w = fp4_values(q.data, q.scale).bfloat16().to(dev())
    assert (w[7] == -torch.inf).all() and w[:7].isfinite().all() and w[8:].isfinite().all()
    alike(got, itl.linear_token_logp_fwd(x.to(dev()), w, tok, top_k=20, return_entropy=True))
    assert (got.logp[:, 1] == -torch.inf).all() and got.logp[:, [0, 2, 3]].isfinite().all() and got.lse.isfinite().all()
    assert (got.top_ids != 7).all() and (got.lse <= without.lse).all()
    for data in (0x11 * code, code | 0x80 | code << 4):  # above; both
        q.data[7] = data
        w = fp4_values(q.data, q.scale).bfloat16().to(dev())
        got = itl.linear_token_logp_fwd(x.to(dev()), q, tok, top_k=20, return_entropy=True)
        alike(got, itl.linear_token_logp_fwd(x.to(dev()), w, tok, top_k=20, return_entropy=True))
        assert not got.lse.isfinite().any()
    # one step below the least such magnitude stays in the range
    q.data[7] = 0x11 * (code - 1)
    assert fp4_values(q.data, q.scale)[7].bfloat16().isfinite().all()


@pytest.mark.parametrize("dtype", TYPES)
def test_lookup_at_the_ends_of_the_scales(dtype):
    """Values are decoded in fp32, where they are exact or, past its range (bytes 253 and 254), an
    infinity that the call's scale leaves one."""
    data = torch.arange(256, dtype=torch.uint8).view(8, 32).repeat(1, 2)[:, :64]
    codes = torch.arange(256, dtype=torch.uint8).repeat(8)[:8 * 64].view(8, 64)
    scale = torch.tensor([0, 1, 2, 127, 252, 253, 254, 255], dtype=torch.uint8).repeat_interleave(4).view(8, 4)
    for data in (data, codes):
        q = itl.Fp4Rows(data.to(dev()), scale.to(dev()))
        values = fp4_values(data, scale).float()
        for by in (1.0, 0.5, 2.0 ** 60):
            got = itl.embedding_fwd(torch.arange(8, device=dev()), q, scale=by, out_dtype=TYPES[dtype]).cpu()
            want = (values * torch.tensor(by)).to(TYPES[dtype])
            assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got[:7], want[:7]) and got[7].isnan().all()
