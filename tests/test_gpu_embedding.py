"""The embedding, its gradient by sorted tokens and the lookup from 4-bit rows
against the plain forms.

The lookup is one fp32 product rounded to the type: equal to torch's.  The
gradient of rows on a grid of 1/16 with a power-of-two scale is exact in fp32
whatever the order, so it equals the rounding of the exact sum.  Other rows: L
occurrences are added with at most 32 + L / 256 + 8 roundings on a chain, the scale
and the table's old value take two more: (L / 256 + 44) 2^-24 of the sum of
magnitudes, then eps / 2."""

import pytest
import torch

import invariant_token_log_amd as itl
from gpu_helpers import dev
from layer_reference import TYPES, embedding_gradient, fp4_values

pytestmark = pytest.mark.gpu


def table(v, h, dtype, seed=0, pad=0):
    gen = torch.Generator().manual_seed(seed)
    w = torch.randn(v, h, generator=gen).to(TYPES[dtype])
    buf = torch.zeros(v, h + pad, dtype=w.dtype, device=dev())[:, :h]
    buf.copy_(w)
    return w, buf


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("h", [1, 7, 8, 100, 1021, 2048, 2056, 4096])
def test_lookup(h, dtype):
    v = 37
    ids = torch.tensor([0, 36, 5, 5, -100, 12, 37, -1, 2 ** 40, 3])
    for pad, index in ((0, torch.int64), (3, torch.int32)):
        t = ids if index == torch.int64 else ids.clamp(max=1000).to(index)
        w, wd = table(v, h, dtype, pad=pad)
        y = itl.embedding_fwd(t.to(dev()), wd, scale=1.7).cpu()
        live = (ids >= 0) & (ids < v)
        want = (w[ids[live]].float() * torch.tensor(1.7, dtype=torch.float32)).to(TYPES[dtype])
        assert torch.equal(y[live], want)
        assert not y[4].any() and y[6:9].isnan().all()
        one = itl.embedding_fwd(t[3:4].to(dev()), wd, scale=1.7).cpu()
        assert torch.equal(one, y[3:4])
    wide = torch.full((2, 5, h + 6), 3.0, dtype=TYPES[dtype], device=dev())
    out = itl.embedding_fwd(ids.view(2, 5).to(dev()), table(v, h, dtype)[1], out=wide[:, :, :h])
    plain = itl.embedding_fwd(ids.to(dev()), table(v, h, dtype)[1])
    assert torch.equal(out.reshape(10, h).nan_to_num(9.0), plain.nan_to_num(9.0)) and (wide[:, :, h:] == 3).all()
    # an ignore_index inside the vocabulary
    y = itl.embedding_fwd(ids.to(dev()), table(v, h, dtype)[1], ignore_index=5).cpu()
    assert not y[2:4].any() and y[4].isnan().all()


def test_lookup_many_rows():
    w, wd = table(1000, 24, "bf16")
    ids = torch.randint(0, 1000, (300001,), generator=torch.Generator().manual_seed(1))
    assert torch.equal(itl.embedding_fwd(ids.to(dev()), wd).cpu(), w[ids])
    assert itl.embedding_fwd(ids[:0].to(dev()), wd).shape == (0, 24)
    assert torch.equal(itl.embedding_fwd(ids[0].to(dev()), wd).cpu(), w[ids[0]])


def draw_ids(n, v, kind, gen):
    if kind == "one":
        ids = torch.full((n,), v // 2)
    elif kind == "text":
        ids = (torch.rand(n, generator=gen, dtype=torch.float64) ** 4 * v).long().clamp(max=v - 1)
    elif kind == "once":
        ids = torch.randperm(max(v, n), generator=gen)[:n] % v
    else:  # runs around the piece length, side by side
        lengths = [31, 32, 33, 1, 64, 65, 63, 96, 2, 97, 40]
        ids = torch.cat([torch.full((m,), i) for i, m in enumerate(lengths)])
        ids = ids.repeat((n + len(ids) - 1) // len(ids))[:n] % v
        ids = ids[torch.randperm(n, generator=gen)]
    drop = torch.rand(n, generator=gen)
    ids[drop < 0.05] = -100
    ids[drop > 0.98] = v + 3  # invalid: left out
    return ids


CASES = [(1, 1, "one"), (1, 50, "one"), (3, 5, "text"), (32, 4, "one"), (33, 4, "one"), (64, 100, "once"),
         (527, 40, "runs"), (1000, 333, "text"), (2047, 90, "text"), (2048, 700, "once"), (2049, 5, "text"), (4095, 1000, "text"), (4096, 7, "one"), (4097, 300, "text"),
         (8200, 64, "runs"), (9000, 20000, "once"), (500, 1500000, "text"), (12289, 3, "text"), (20000, 1500000, "text"), (16384, 900, "once"), (16385, 900, "text"),
         (70000, 400, "text"), (131073, 2000, "text"), (270000, 50, "runs")]


@pytest.mark.parametrize("n,v,kind", CASES)
def test_gradient_exact(n, v, kind):
    """Exact sums: every type, both outputs, written or added."""
    gen = torch.Generator().manual_seed(n + v)
    ids = draw_ids(n, v, kind, gen)
    h = 40 if v < 100000 else 8
    grid = torch.randint(-15, 16, (n, h), generator=gen).float() / 16
    live = (ids >= 0) & (ids < v)
    ref = torch.zeros(v, h, dtype=torch.float64).index_add_(0, ids[live], grid[live].double() * 0.5)
    for dtype in TYPES:
        dy = grid.to(TYPES[dtype])
        for out_dtype in {TYPES[dtype], torch.float32}:
            d = itl.embedding_bwd(ids.to(dev()), dy.to(dev()), v, scale=0.5, out_dtype=out_dtype)
            assert d.dtype == out_dtype and torch.equal(d.cpu(), ref.to(out_dtype))
            base = torch.randint(-8, 9, (v, h), generator=gen).float().to(out_dtype)
            out = base.to(dev())
            got = itl.embedding_bwd(ids.int().to(dev()), dy.to(dev()), v, scale=0.5, dweight_out=out, accumulate=True)
            assert got is out and torch.equal(out.cpu(), (ref + base.double()).to(out_dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("h", [1, 7, 100, 512, 513, 1021, 2056, 4096])
def test_gradient_widths(h, dtype):
    n, v = 700, 60
    gen = torch.Generator().manual_seed(h)
    ids = draw_ids(n, v, "runs", gen)
    dy = torch.randn(n, h, generator=gen).to(TYPES[dtype])
    ref = embedding_gradient(ids, dy, v, 2.5, -100)
    size = embedding_gradient(ids, dy.abs(), v, 2.5, -100)
    most = torch.bincount(ids[(ids >= 0) & (ids < v)]).max().item()
    bound = (most / 256 + 44) * 2.0 ** -24 * size
    half = torch.finfo(TYPES[dtype]).eps / 2
    got = itl.embedding_bwd(ids.to(dev()), dy.to(dev()), v, scale=2.5)
    assert ((got.double().cpu() - ref).abs() <= bound + half * (ref.abs() + bound) + 2.0 ** -25 * (dtype == "fp16")).all()
    assert torch.equal(itl.embedding_bwd(ids.to(dev()), dy.to(dev()), v, scale=2.5), got)
    # strided and unaligned rows, columns past them left alone
    dyp = torch.zeros(n, h + 3, dtype=dy.dtype, device=dev())[:, :h].copy_(dy)
    wide = torch.full((v, h + 5), 4.0, dtype=dy.dtype, device=dev())
    itl.embedding_bwd(ids.to(dev()), dyp, v, scale=2.5, dweight_out=wide[:, :h])
    assert torch.equal(wide[:, :h], got) and (wide[:, h:] == 4).all()


def test_gradient_depends_on_a_tokens_own_rows():
    """The same occurrences in another batch: the same bits; NaN in the rows of
    left-out tokens stays out."""
    gen = torch.Generator().manual_seed(3)
    n, v, h = 6000, 500, 72
    ids = draw_ids(n, v, "text", gen)
    dy = torch.randn(n, h, generator=gen)
    dy[(ids < 0) | (ids >= v)] = torch.nan
    d = itl.embedding_bwd(ids.to(dev()), dy.to(dev()), v)
    assert not d.isnan().any()
    for t in ids[(ids >= 0) & (ids < v)].unique()[:12].tolist():
        mine = ids == t
        alone = itl.embedding_bwd(ids[mine].to(dev()), dy[mine].to(dev()), v)
        assert torch.equal(alone[t], d[t]) and alone.count_nonzero() == alone[t].count_nonzero()


def test_gradient_empty_and_absent():
    ids = torch.full((50,), -100, device=dev())
    dy = torch.ones(50, 16, device=dev())
    out = torch.full((9, 16), 5.0, device=dev())
    assert not itl.embedding_bwd(ids, dy, 9, dweight_out=out).any()
    out.fill_(5.0)
    assert (itl.embedding_bwd(ids, dy, 9, dweight_out=out, accumulate=True) == 5).all()
    assert not itl.embedding_bwd(ids[:0], dy[:0], 9, dweight_out=out).any()
    out.fill_(5.0)
    assert (itl.embedding_bwd(ids[:0], dy[:0], 9, dweight_out=out, accumulate=True) == 5).all()


def test_autograd():
    w, wd = table(50, 24, "fp32")
    ids = torch.tensor([[3, 3, 7], [49, -100, 3]], device=dev())
    a = wd.requires_grad_()
    y = itl.embedding(ids, a, scale=3.0)
    g = torch.randn(2, 3, 24, device=dev())
    d, = torch.autograd.grad(y, a, g)
    ref = embedding_gradient(ids.cpu().flatten(), g.cpu().view(6, 24), 50, 3.0, -100)
    assert ((d.double().cpu() - ref).abs() <= 2.0 ** -20 * (1 + ref.abs())).all()
    e = torch.zeros_like(wd)
    e[3, 5] = 1.0
    slope = ((itl.embedding_fwd(ids, wd.detach() + e, scale=3.0) - itl.embedding_fwd(ids, wd.detach(), scale=3.0)) * g).sum()
    assert abs(slope.item() - d[3, 5].item()) <= 1e-4
    y = itl.embedding(ids, a, scale=3.0)
    one, = torch.autograd.grad(y, a, torch.tensor(2.0, device=dev()).expand(2, 3, 24))
    assert one[3, 0] == 18 and one[7, 0] == 6 and one[0].eq(0).all()


def test_streams_and_graph():
    """Captured and replayed with new tokens between eager calls, and two calls on
    two streams at once."""
    v, h = 3000, 256
    ids = torch.zeros(5000, dtype=torch.int64, device=dev())
    dy = torch.empty(5000, h, dtype=torch.bfloat16, device=dev())

    def fill(k):
        gen = torch.Generator().manual_seed(k)
        ids.copy_(draw_ids(5000, v, "text", gen))
        dy.copy_(torch.randn(5000, h, generator=gen))

    fill(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        itl.embedding_bwd(ids, dy, v)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d = itl.embedding_bwd(ids, dy, v)
    for k in (1, 2, 3):
        fill(k)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d, itl.embedding_bwd(ids, dy, v))
    want = itl.embedding_bwd(ids, dy, v)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for st in streams:
        with torch.cuda.stream(st):
            outs.append(itl.embedding_bwd(ids, dy, v))
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


@pytest.mark.parametrize("out_dtype", TYPES)
@pytest.mark.parametrize("h", [32, 96, 2048, 4096])
def test_lookup_fp4(h, out_dtype):
    v = 29
    gen = torch.Generator().manual_seed(h)
    data = torch.randint(0, 256, (v, h // 2), generator=gen, dtype=torch.uint8)
    scale = torch.randint(100, 140, (v, h // 32), generator=gen, dtype=torch.uint8)
    scale[3, 0], scale[4, 0] = 0, 255
    ids = torch.tensor([0, 28, 3, 4, -100, 29, 7, 7])
    q = itl.Fp4Rows(data.to(dev()), scale.to(dev()))
    y = itl.embedding_fwd(ids.to(dev()), q, scale=1.3, out_dtype=TYPES[out_dtype])
    values = fp4_values(data, scale).float()  # exact
    live = torch.tensor([0, 1, 2, 3, 6, 7])
    want = (values[ids[live]] * torch.tensor(1.3, dtype=torch.float32)).to(TYPES[out_dtype])
    got = y.cpu()[live]
    assert torch.equal(got.nan_to_num(9.0), want.nan_to_num(9.0)) and torch.equal(got.isnan(), want.isnan())
    assert not y[4].any() and y[5].isnan().all()
    wide = torch.zeros(v, h // 2 + 16, dtype=torch.uint8, device=dev())
    wide[:, :h // 2] = q.data
    rows = itl.Fp4Rows(wide[:, :h // 2], torch.cat([q.scale, q.scale], 1)[:, :h // 32])
    again = itl.embedding_fwd(ids.int().to(dev()), rows, scale=1.3, out_dtype=TYPES[out_dtype])
    assert torch.equal(again.nan_to_num(9.0), y.nan_to_num(9.0))


def test_widest_rows():
    """Rows of 2^24 elements, the most, with a token of two pieces, one of one and one absent."""
    h, n = 2 ** 24, 34
    dy = torch.zeros(n, h, dtype=torch.bfloat16, device=dev())
    dy[:, 0], dy[:, h - 1], dy[:, h // 2 + 3] = 0.5, 1.0, 2.0
    ids = torch.tensor([1] * 17 + [0] + [1] * 16, device=dev())
    g = itl.embedding_bwd(ids, dy, 3)
    for c, x in ((0, 0.5), (h - 1, 1.0), (h // 2 + 3, 2.0), (1, 0.0), (h - 2, 0.0)):
        assert g[:, c].tolist() == [x, 33 * x, 0.0]
    assert int(torch.count_nonzero(g)) == 6
    assert torch.equal(itl.embedding_fwd(ids[16:18], g), g[[1, 0]])


def test_lookup_fp4_many_rows():
    gen = torch.Generator().manual_seed(4)
    data = torch.randint(0, 256, (1000, 16), generator=gen, dtype=torch.uint8)
    scale = torch.randint(110, 130, (1000, 1), generator=gen, dtype=torch.uint8)
    ids = torch.randint(-1, 1001, (300001,), generator=gen)
    ids[300000], ids[299998], ids[7] = 3, 1000, -100
    y = itl.embedding_fwd(ids.to(dev()), itl.Fp4Rows(data.to(dev()), scale.to(dev()))).double().cpu()
    live = (ids >= 0) & (ids < 1000)
    assert torch.equal(y[live], fp4_values(data, scale)[ids[live]]) and not y[7].any()
    assert y[~live & (ids != -100)].isnan().all()


@pytest.mark.parametrize("dtype,h,ld", [("fp32", 100, 105), ("bf16", 101, 103), ("fp16", 96, 104)])
@pytest.mark.parametrize("n", [0, 1000, 5000])
def test_gradient_into_a_large_table_with_gaps(n, dtype, h, ld):
    """More rows than are cleared beside the sort and the merge (40 and 32 MB): the absent ones
    of the rest go row by row.  Gaps stay as they are, and the rows behind the table."""
    v = 2 ** 27 // (h * (4 if dtype == "fp32" else 2)) + 37
    gen = torch.Generator().manual_seed(n + h)
    ids = torch.randint(0, v, (n,), generator=gen)
    if n:
        ids[:8] = torch.tensor([0, v - 1, v - 2, v - 64, v - 65, v // 2, v // 2, -100])
        ids[100:140] = v - 5  # several pieces among absent rows
        ids[200:264] = torch.arange(v - 300, v - 236)  # a whole block of 64 present
    grid = (torch.randint(-15, 16, (n, h), generator=gen).float() / 16).to(TYPES[dtype])
    live = ids >= 0
    want = torch.zeros(v, h).index_add_(0, ids[live], grid[live].float())  # exact: few sixteenths a sum
    wide = torch.full((v + 2, ld), 3.0, dtype=TYPES[dtype], device=dev())
    got = itl.embedding_bwd(ids.to(dev()), grid.to(dev()), v, dweight_out=wide[:v, :h])
    assert got.data_ptr() == wide.data_ptr() and torch.equal(got.cpu(), want.to(TYPES[dtype]))
    assert (wide[:, h:] == 3).all() and (wide[v:] == 3).all()
    # the same sums without gaps
    assert torch.equal(itl.embedding_bwd(ids.to(dev()), grid.to(dev()), v), got)
    # added: absent rows stay too
    wide.fill_(3.0)
    itl.embedding_bwd(ids.to(dev()), grid.to(dev()), v, dweight_out=wide[:v, :h], accumulate=True)
    assert torch.equal(wide[:v, :h].cpu(), (want + 3).to(TYPES[dtype]))
    assert (wide[:, h:] == 3).all() and (wide[v:] == 3).all()
