"""The operators in a row, as a model with a tied table runs them: embedding,
dropout and layer norm on the residual stream, the LM head's log-probabilities,
and all the way back, the table's gradient being the head's plus the
embedding's.

Tolerances of the whole chain.  Activations and their gradients are rounded to
bf16 between the operators: about ten roundings of 2^-9 on average, at most 2^-8
each, that a gradient passes, so the relative distance of a whole gradient from
the float64 one (taken with the same masks) stays below 10 * 2^-8."""

import contextlib
import math

import pytest
import torch
import torch.utils.checkpoint

import invariant_token_log_amd as itl
from gpu_helpers import dev
from layer_reference import dropped

pytestmark = pytest.mark.gpu

V, H, N, P, SEED = 1009, 256, 96, 0.1, 0x1234567
EPS = 1e-5


def model(seed):
    gen = torch.Generator().manual_seed(seed)
    table = (torch.randn(V, H, generator=gen) * 0.05).bfloat16()
    w = (1 + 0.1 * torch.randn(2, H, generator=gen)).bfloat16()
    b = (0.1 * torch.randn(2, H, generator=gen)).bfloat16()
    ids = torch.randint(0, V, (N,), generator=gen)
    ids[::7] = 5  # one token often
    targets = torch.randint(0, V, (N, 1), generator=gen)
    ids[-6:], targets[-6:] = -100, -100  # a padded end
    return table, w, b, ids, targets


def loss64(table, w, b, ids, targets, seed):
    """-sum of the log-probabilities of x1 = drop(E[ids] sqrt(H)), x2 = x1 +
    drop(norm(x1)), norm(x2) through E, and x2's norm weights."""
    def norm(x, i):
        m = x.mean(1, keepdim=True)
        return (x - m) / torch.sqrt(((x - m) ** 2).mean(1, keepdim=True) + EPS) * w[i] + b[i]

    def drop(x, draw):
        keep = dropped(torch.ones(N, H, dtype=torch.float64), P, seed, draw)
        return x * keep

    live = ids >= 0
    x1 = drop(torch.where(live[:, None], table[ids.clamp(min=0)], 0.0) * math.sqrt(H), 0)
    x2 = x1 + drop(norm(x1, 0), 1)
    logp = torch.log_softmax(norm(x2, 1) @ table.T, 1).gather(1, targets.clamp(min=0))[:, 0]
    return -(logp * (targets[:, 0] >= 0)).sum()


def reference(parts, seed):
    table, w, b, ids, targets = parts
    leaves = [t.double().requires_grad_() for t in (table, w, b)]
    loss = loss64(*leaves, ids, targets, seed)
    return loss.item(), torch.autograd.grad(loss, leaves)


def near(got, want):
    got = got.double().cpu()
    assert (got - want).norm() <= 10 * 2.0 ** -8 * want.norm()


def test_training_step_through_autograd():
    parts = model(1)
    table, w, b = (t.to(dev()).requires_grad_() for t in parts[:3])
    ids, targets = parts[3].to(dev()), parts[4].to(dev())
    seed = torch.tensor([SEED], device=dev())
    x1 = itl.dropout(itl.embedding(ids, table, scale=math.sqrt(H)), P, seed, draw=0)
    y = itl.layer_norm(x1, w[0], b[0], eps=EPS)
    y, _ = itl.layer_norm(y, w[1], b[1], residual=x1, eps=EPS, dropout=P, seed=seed, draw=1)
    loss = -itl.linear_token_logp(y, table, targets).logp.sum()
    loss.backward()
    value, grads = reference(parts, SEED)
    assert abs(loss.item() - value) <= 1e-2 * abs(value)
    for got, want in zip((table.grad, w.grad, b.grad), grads):
        near(got, want)


def step(table, w, b, ids, targets, seed, dtable):
    """The same step in the library's own calls; the table's gradient of both ends
    in one fp32 buffer."""
    x0 = itl.embedding_fwd(ids, table, scale=math.sqrt(H))
    x1 = itl.dropout_fwd(x0, P, seed, draw=0)
    y0, s0, m0, r0 = itl.layer_norm_fwd(x1, w[0], b[0], eps=EPS, return_stats=True)
    y1, s1, m1, r1 = itl.layer_norm_fwd(y0, w[1], b[1], residual=x1, eps=EPS, dropout=P, seed=seed, draw=1, return_stats=True)
    r = itl.linear_token_logp_fwd(y1, table, targets)
    g = torch.full_like(r.logp, -1.0)
    dy1, _ = itl.linear_token_logp_bwd(y1, table, r.lse, targets, r.logp, g, out_dtype=torch.float32, dweight_out=dtable)
    dy0, dx1, dw1, db1 = itl.layer_norm_bwd(s1, w[1], m1, r1, dy1.bfloat16(), dropout=P, seed=seed, draw=1)
    dx1, _, dw0, db0 = itl.layer_norm_bwd(s0, w[0], m0, r0, dy0, dx1)
    itl.embedding_bwd(ids, itl.dropout_bwd(dx1, P, seed, draw=0), V, scale=math.sqrt(H), dweight_out=dtable, accumulate=True)
    return r.logp, dtable, torch.stack([dw0, dw1]), torch.stack([db0, db1])


def test_training_step_captured():
    """Captured once and replayed with new tokens, weights and seeds between eager
    steps."""
    parts = [t.to(dev()) for t in model(2)]
    seed = torch.tensor([SEED], device=dev())
    dtable = torch.empty(V, H, device=dev())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(*parts, seed, dtable)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*parts, seed, dtable)
    for k in range(3, 6):
        fresh = model(k)
        for a, c in zip(parts, fresh):
            a.copy_(c)
        seed.fill_(SEED + k)
        graph.replay()
        torch.cuda.synchronize()
        eager = step(*parts, SEED + k, torch.empty(V, H, device=dev()))
        assert all(torch.equal(a, c) for a, c in zip(out, eager))
        value, grads = reference(fresh, SEED + k)
        assert abs(-out[0].sum().item() - value) <= 1e-2 * abs(value)
        for got, want in zip(out[1:], grads):
            near(got, want)


@pytest.mark.parametrize("call", ["embedding", "dropout", "layer_norm"])
def test_second_derivative_is_refused(call):
    x = torch.randn(4, 64, device=dev(), requires_grad=True)
    w = torch.ones(64, device=dev(), requires_grad=True)
    if call == "embedding":
        y, leaf = itl.embedding(torch.tensor([1, 3], device=dev()), x), x
    elif call == "dropout":
        y, leaf = itl.dropout(x, 0.3, 1), x
    else:
        y, leaf = itl.layer_norm(x, w), x
    g = torch.ones_like(y, requires_grad=True)
    d, = torch.autograd.grad(y, leaf, g, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        d.sum().backward()


def test_past_two_to_the_31_elements():
    """A table, rows and gradients whose last elements lie past 2^31."""
    v, h = 300000, 8192
    table = torch.zeros(v, h, dtype=torch.bfloat16, device=dev())
    ids = torch.tensor([v - 1, 0, v - 2, v - 1], device=dev())
    gen = torch.Generator().manual_seed(1)
    rows = torch.randint(-8, 9, (4, h), generator=gen).bfloat16().to(dev())
    itl.embedding_bwd(ids, rows, v, dweight_out=table)
    assert torch.equal(table[v - 1], rows[0] + rows[3]) and torch.equal(table[v - 2], rows[2])
    assert torch.equal(table[0], rows[1]) and not table[1:v - 2].any()
    itl.embedding_bwd(ids, rows, v, dweight_out=table, accumulate=True)
    assert torch.equal(table[v - 1], 2 * (rows[0] + rows[3]))
    assert torch.equal(itl.embedding_fwd(ids, table)[2], 2 * rows[2])
    # the last rows of a long batch, alone and within it
    w = torch.ones(h, dtype=torch.bfloat16, device=dev())
    table[-3:] = torch.randn(3, h, device=dev())
    out = torch.empty_like(table)
    itl.dropout_fwd(table, 0.5, 7, residual=table, out=out)
    assert torch.equal(out[-3:], itl.dropout_fwd(table[-3:], 0.5, 7, residual=table[-3:], first_row=v - 3))
    y, _, mean, rstd = itl.layer_norm_fwd(table, w, w, y_out=out, return_stats=True)
    one, _, m1, r1 = itl.layer_norm_fwd(table[-3:], w, w, return_stats=True)
    assert torch.equal(y[-3:], one) and torch.equal(mean[-3:], m1) and torch.equal(rstd[-3:], r1)
    dx, _, _, _ = itl.layer_norm_bwd(table, w, mean, rstd, out, need_dweight=False, need_dbias=False, dx_out=out)
    d1, _, _, _ = itl.layer_norm_bwd(table[-3:], w, m1, r1, one, need_dweight=False, need_dbias=False)
    assert torch.equal(dx[-3:], d1)
    q = itl.quantize_rows_fp4(table)
    last = itl.quantize_rows_fp4(table[-3:])
    assert torch.equal(q.data[-3:], last.data) and torch.equal(q.scale[-3:], last.scale)
    assert torch.equal(itl.embedding_fwd(ids, q)[0], itl.embedding_fwd(torch.tensor([2], device=dev()), last)[0])


def test_saved_tensors_that_hooks_move():
    """Saved tensors that live elsewhere between forward and backward: a strided row
    comes back contiguous, a seed at another address (its first place is used again)."""
    gen = torch.Generator().manual_seed(3)
    buf = torch.randn(33, 136, generator=gen).to(dev())
    w, b = torch.randn(2, 128, generator=gen).to(dev())
    g = torch.randn(33, 128, generator=gen).to(dev())
    ids = torch.randint(0, 50, (33,), generator=gen).to(dev())

    def grads(hooks):
        x = buf[:, :128].detach().requires_grad_()
        table = torch.randn(50, 128, generator=torch.Generator().manual_seed(4)).to(dev()).requires_grad_()
        with hooks:
            seed = torch.tensor([77], device=dev())
            y = itl.layer_norm(x, w, b)
            z, s = itl.layer_norm(x, w, b, residual=itl.embedding(ids, table), dropout=0.3, seed=seed, draw=1)
            u = itl.dropout(x, 0.4, seed, draw=2)
            del seed
        over = [torch.full((1,), 5 + i, dtype=torch.int64, device=dev()) for i in range(64)]
        out = torch.autograd.grad([y, z, s, u], [x, table], [g, g, g, g])
        del over
        return out

    want = grads(contextlib.nullcontext())
    got = grads(torch.autograd.graph.save_on_cpu())
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("p", [0.0, 0.3])
def test_one_tensor_in_two_places(p):
    """Rows that are their own residual: their gradient is the sum of both, and two leaves get
    buffers of their own; the sum over the rows in place of both."""
    gen = torch.Generator().manual_seed(6)
    x, g = torch.randn(2, 37, 520, generator=gen).to(dev())
    w = torch.randn(520, generator=gen).to(dev())
    a, b, c = (x.clone().requires_grad_() for _ in range(3))
    y, s = itl.layer_norm(a, w, w, residual=a, dropout=p, seed=3)
    d, = torch.autograd.grad([y, s], a, [g, g])
    torch.autograd.backward(itl.layer_norm(b, w, w, residual=c, dropout=p, seed=3), [g, g])
    assert torch.equal(d, b.grad + c.grad) and b.grad.data_ptr() != c.grad.data_ptr()
    i = x.clone()
    y2, _, _, _ = itl.layer_norm_fwd(i, w, w, residual=i, dropout=p, seed=3, sum_out=i)
    assert torch.equal(y2, y) and torch.equal(i, s)
    d, = torch.autograd.grad(itl.dropout(a, p, 3, residual=a), a, g)
    assert torch.equal(d, itl.dropout_bwd(g, p, 3) + g)


def test_autograd_on_streams_and_again():
    """Forward on a side stream and backward on another, a graph used twice, a forward that is
    run again for its backward: the same gradient every time."""
    gen = torch.Generator().manual_seed(7)
    table = torch.randn(500, 520, generator=gen).to(dev()).requires_grad_()
    w = torch.randn(520, generator=gen).to(dev())
    ids = torch.randint(0, 500, (3000,), generator=gen).to(dev())
    g = torch.randn(3000, 520, generator=gen).to(dev())

    def step():
        e = itl.embedding(ids, table, 2.0)
        return itl.dropout(itl.layer_norm(e, w, w), 0.2, 9, residual=e)

    out = step()
    want, = torch.autograd.grad(out, table, g, retain_graph=True)
    got = [torch.autograd.grad(out, table, g)[0],
           torch.autograd.grad(torch.utils.checkpoint.checkpoint(step, use_reentrant=False), table, g)[0]]
    main = torch.cuda.current_stream()
    for side in [torch.cuda.Stream() for _ in range(2)]:
        side.wait_stream(main)
        with torch.cuda.stream(side):
            out = step()
        main.wait_stream(side)
        got.append(torch.autograd.grad(out, table, g)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(d, want) for d in got)
