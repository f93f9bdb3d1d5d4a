"""Refusals of the embedding, dropout, the layer norm and 4-bit rows, on the
host: every bad argument gets its documented status before any HIP call, and the
binding's own checks raise before any device work (nothing here touches a
device)."""

import os

import pytest
import torch

import invariant_token_log_amd as itl
from invariant_token_log_amd import _lib, layer_ops
from invariant_token_log_amd.build import LIB_PATH, build

P = 0x10000  # a non-NULL, 256-byte aligned address that the checks never dereference
Q = 0x20000
BIG = 1 << 60
OK = _lib.LOGP_OK
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(LIB_PATH):
        build()
    return _lib.lib()


def expect(fn, base, cases):
    """Each case changes some arguments of a good call and names the status."""
    for status, change in cases:
        args = {**base, **change}
        assert set(args) == set(base), change
        assert fn(*args.values()) == status, (change, status)


def test_embedding(L):
    base = dict(table=P, ld_t=64, v=100, h=64, dtype=1, tokens=P, tdt=0, n=5, ignore=-100, scale=1.0, out=P, ld_o=64,
                stream=None)
    expect(L.embedding_fwd, base, [
        (_lib.LOGP_ERR_DTYPE, dict(dtype=3)), (_lib.LOGP_ERR_DTYPE, dict(tdt=2)), (_lib.LOGP_ERR_SHAPE, dict(n=-1)),
        (_lib.LOGP_ERR_SHAPE, dict(n=1 << 31)), (_lib.LOGP_ERR_SHAPE, dict(v=0)), (_lib.LOGP_ERR_SHAPE, dict(v=(1 << 31) + 1)),
        (_lib.LOGP_ERR_SHAPE, dict(h=0)), (_lib.LOGP_ERR_SHAPE, dict(h=(1 << 24) + 1, ld_t=BIG, ld_o=BIG)),
        (_lib.LOGP_ERR_SHAPE, dict(ld_t=63)), (_lib.LOGP_ERR_SHAPE, dict(ld_o=63)), (_lib.LOGP_ERR_VALUE, dict(scale=INF)),
        (_lib.LOGP_ERR_VALUE, dict(scale=NAN)), (_lib.LOGP_ERR_NULL, dict(table=None)), (_lib.LOGP_ERR_NULL, dict(tokens=None)),
        (_lib.LOGP_ERR_NULL, dict(out=None)), (OK, dict(n=0, table=None, tokens=None, out=None)),
    ])
    base = dict(data=P, ld_d=32, scales=P, ld_s=2, v=100, h=64, tokens=P, tdt=0, n=5, ignore=-100, scale=1.0, odt=1, out=P,
                ld_o=64, stream=None)
    expect(L.embedding_fp4_fwd, base, [
        (_lib.LOGP_ERR_DTYPE, dict(odt=-1)), (_lib.LOGP_ERR_DTYPE, dict(tdt=7)), (_lib.LOGP_ERR_SHAPE, dict(h=48, ld_d=32)),
        (_lib.LOGP_ERR_SHAPE, dict(ld_d=31)), (_lib.LOGP_ERR_SHAPE, dict(ld_s=1)), (_lib.LOGP_ERR_SHAPE, dict(ld_o=60)),
        (_lib.LOGP_ERR_NULL, dict(data=None)), (_lib.LOGP_ERR_NULL, dict(scales=None)), (_lib.LOGP_ERR_ALIGN, dict(data=P + 8)),
        (_lib.LOGP_ERR_ALIGN, dict(ld_d=40)), (_lib.LOGP_ERR_VALUE, dict(scale=-INF)),
        (OK, dict(n=0, data=None, scales=None, tokens=None, out=None)),
    ])


def test_embedding_gradient(L):
    need = L.embedding_bwd_workspace_bytes(5000, 100, 60)
    # id, pos, start; the tiles' keys; two partial rows of 64 columns for 32 tokens
    assert need == 3 * 20224 + 40192 + 2 * 157 * 64 * 4 + (-2 * 157 * 64 * 4) % 256
    assert L.embedding_bwd_workspace_bytes(32, 100, 60) == 3 * 256
    for bad in ((0, 100, 60), (-1, 100, 60), ((1 << 24) + 1, 100, 60), (5, 0, 60), (5, 100, 0)):
        assert L.embedding_bwd_workspace_bytes(*bad) == 0
    base = dict(dy=P, ld_y=60, dtype=1, tokens=P, tdt=1, n=5000, v=100, h=60, ignore=-100, scale=1.0, odt=1, add=0, d=P,
                ld_t=60, ws=P, ws_bytes=need, stream=None)
    expect(L.embedding_bwd, base, [
        (_lib.LOGP_ERR_DTYPE, dict(dtype=5)), (_lib.LOGP_ERR_DTYPE, dict(odt=2)), (_lib.LOGP_ERR_DTYPE, dict(tdt=-1)),
        (_lib.LOGP_ERR_SHAPE, dict(n=(1 << 24) + 1)), (_lib.LOGP_ERR_SHAPE, dict(ld_y=59)), (_lib.LOGP_ERR_SHAPE, dict(ld_t=59)),
        (_lib.LOGP_ERR_VALUE, dict(add=2)), (_lib.LOGP_ERR_VALUE, dict(scale=NAN)), (_lib.LOGP_ERR_NULL, dict(dy=None)),
        (_lib.LOGP_ERR_NULL, dict(tokens=None)), (_lib.LOGP_ERR_NULL, dict(d=None)), (_lib.LOGP_ERR_WORKSPACE, dict(ws=None)),
        (_lib.LOGP_ERR_WORKSPACE, dict(ws=P + 64)), (_lib.LOGP_ERR_WORKSPACE, dict(ws_bytes=need - 1)),
        (OK, dict(n=0, add=1, dy=None, tokens=None, d=None, ws=None)), (_lib.LOGP_ERR_NULL, dict(n=0, d=None)),
    ])


def test_dropout(L):
    base = dict(x=P, ld_x=64, r=P, ld_r=64, dtype=1, n=5, h=64, p=0.1, seed=1, at=None, draw=0, first=0, out=P, ld_o=64,
                stream=None)
    expect(L.dropout_fwd, base, [
        (_lib.LOGP_ERR_DTYPE, dict(dtype=3)), (_lib.LOGP_ERR_SHAPE, dict(n=-1)), (_lib.LOGP_ERR_SHAPE, dict(h=0)),
        (_lib.LOGP_ERR_SHAPE, dict(ld_x=63)), (_lib.LOGP_ERR_SHAPE, dict(ld_r=63)), (_lib.LOGP_ERR_SHAPE, dict(ld_o=63)),
        (_lib.LOGP_ERR_VALUE, dict(p=-0.01)), (_lib.LOGP_ERR_VALUE, dict(p=1.01)), (_lib.LOGP_ERR_VALUE, dict(p=NAN)),
        (_lib.LOGP_ERR_VALUE, dict(draw=-1)), (_lib.LOGP_ERR_VALUE, dict(draw=1 << 32)), (_lib.LOGP_ERR_VALUE, dict(first=-1)),
        (_lib.LOGP_ERR_VALUE, dict(first=(1 << 63) - 1)), (_lib.LOGP_ERR_NULL, dict(x=None)), (_lib.LOGP_ERR_NULL, dict(out=None)),
        (OK, dict(n=0, x=None, r=None, out=None)),
    ])


def test_layer_norm(L):
    base = dict(x=P, ld_x=64, r=P, ld_r=64, w=P, b=P, dtype=1, n=5, h=64, eps=1e-5, p=0.1, seed=1, at=None, draw=0, first=0,
                y=P, ld_y=64, s=P, ld_s=64, mean=P, rstd=P, stream=None)
    expect(L.layer_norm_fwd, base, [
        (_lib.LOGP_ERR_DTYPE, dict(dtype=3)), (_lib.LOGP_ERR_SHAPE, dict(n=-1)), (_lib.LOGP_ERR_SHAPE, dict(h=0)),
        (_lib.LOGP_ERR_SHAPE, dict(h=65537, ld_x=BIG, ld_r=BIG, ld_y=BIG, ld_s=BIG)), (_lib.LOGP_ERR_SHAPE, dict(ld_x=63)),
        (_lib.LOGP_ERR_SHAPE, dict(ld_r=63)), (_lib.LOGP_ERR_SHAPE, dict(ld_y=63)), (_lib.LOGP_ERR_SHAPE, dict(ld_s=63)),
        (_lib.LOGP_ERR_VALUE, dict(eps=-1.0)), (_lib.LOGP_ERR_VALUE, dict(eps=INF)), (_lib.LOGP_ERR_VALUE, dict(p=1.5)),
        (_lib.LOGP_ERR_VALUE, dict(draw=-1)), (_lib.LOGP_ERR_NULL, dict(x=None)), (_lib.LOGP_ERR_NULL, dict(w=None)),
        (_lib.LOGP_ERR_NULL, dict(y=None)), (_lib.LOGP_ERR_NULL, dict(s=None)), (_lib.LOGP_ERR_NULL, dict(r=None, s=None)),
        (_lib.LOGP_ERR_NULL, dict(p=0.0, s=None)), (OK, dict(n=0, x=None, w=None, y=None, s=None)),
    ])
    need = L.layer_norm_bwd_workspace_bytes(5, 64)
    assert need == 5 * 64 * 8 and L.layer_norm_bwd_workspace_bytes(0, 64) == 0
    assert L.layer_norm_bwd_workspace_bytes(5, 65537) == 0
    base = dict(s=P, ld_s=64, w=P, mean=P, rstd=P, dy=P, ld_dy=64, ds=P, ld_ds=64, dtype=1, n=5, h=64, p=0.1, seed=1, at=None,
                draw=0, first=0, dx=P, ld_dx=64, dr=Q, ld_dr=64, dw=P, db=P, ws=P, ws_bytes=need, stream=None)
    expect(L.layer_norm_bwd, base, [
        (_lib.LOGP_ERR_DTYPE, dict(dtype=3)), (_lib.LOGP_ERR_SHAPE, dict(n=-1)), (_lib.LOGP_ERR_SHAPE, dict(h=0)),
        (_lib.LOGP_ERR_SHAPE, dict(ld_s=63)), (_lib.LOGP_ERR_SHAPE, dict(ld_dy=63)), (_lib.LOGP_ERR_SHAPE, dict(ld_ds=63)),
        (_lib.LOGP_ERR_SHAPE, dict(ld_dx=63)), (_lib.LOGP_ERR_SHAPE, dict(ld_dr=63)), (_lib.LOGP_ERR_VALUE, dict(p=-1.0)),
        (_lib.LOGP_ERR_VALUE, dict(p=0.0)), (_lib.LOGP_ERR_VALUE, dict(dr=P)), (_lib.LOGP_ERR_NULL, dict(s=None)),
        (_lib.LOGP_ERR_NULL, dict(w=None)), (_lib.LOGP_ERR_NULL, dict(mean=None)), (_lib.LOGP_ERR_NULL, dict(rstd=None)),
        (_lib.LOGP_ERR_NULL, dict(dy=None)), (_lib.LOGP_ERR_NULL, dict(dx=None)), (_lib.LOGP_ERR_WORKSPACE, dict(ws=None)),
        (_lib.LOGP_ERR_WORKSPACE, dict(ws=P + 8)), (_lib.LOGP_ERR_WORKSPACE, dict(ws_bytes=need - 1)),
        (OK, dict(n=0, dw=None, db=None, s=None, dx=None)),
    ])


def test_fp4_rows(L):
    base = dict(x=P, ld_x=64, dtype=1, n=5, h=64, d=P, ld_d=32, s=P, ld_s=2, stream=None)
    expect(L.fp4_quantize, base, [
        (_lib.LOGP_ERR_DTYPE, dict(dtype=4)), (_lib.LOGP_ERR_SHAPE, dict(n=-1)), (_lib.LOGP_ERR_SHAPE, dict(h=0)),
        (_lib.LOGP_ERR_SHAPE, dict(h=40)), (_lib.LOGP_ERR_SHAPE, dict(ld_x=63)), (_lib.LOGP_ERR_SHAPE, dict(ld_d=31)),
        (_lib.LOGP_ERR_SHAPE, dict(ld_s=1)), (_lib.LOGP_ERR_NULL, dict(x=None)), (_lib.LOGP_ERR_NULL, dict(d=None)),
        (_lib.LOGP_ERR_NULL, dict(s=None)), (_lib.LOGP_ERR_ALIGN, dict(d=P + 4)), (_lib.LOGP_ERR_ALIGN, dict(ld_d=36)),
        (OK, dict(n=0, x=None, d=None, s=None)),
    ])


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(4, 64), torch.ones(64)
    ids, g = torch.zeros(4, dtype=torch.int64), torch.zeros(4, 64)
    for call in (lambda: itl.embedding_fwd(ids, torch.zeros(9, 64)), lambda: itl.embedding(ids, torch.zeros(9, 64)),
                 lambda: itl.embedding_bwd(ids, g, 9), lambda: itl.dropout_fwd(x, 0.1, 1), lambda: itl.dropout(x, 0.1, 1),
                 lambda: itl.dropout_bwd(x, 0.1, 1), lambda: itl.layer_norm_fwd(x, w), lambda: itl.layer_norm(x, w),
                 lambda: itl.layer_norm_bwd(x, w, x[:, 0], x[:, 0], x), lambda: itl.quantize_rows_fp4(x),
                 lambda: itl.embedding_fwd(ids, itl.Fp4Rows(torch.zeros(9, 32, dtype=torch.uint8),
                                                            torch.zeros(9, 2, dtype=torch.uint8)))):
        with pytest.raises(ValueError, match="ROCm device"):
            call()


def test_binding_checks_4_bit_rows():
    data, scale = torch.zeros(9, 32, dtype=torch.uint8), torch.zeros(9, 2, dtype=torch.uint8)
    for d, s, error in ((data.int(), scale, TypeError), (data, scale.float(), TypeError), (data[0], scale, TypeError),
                        (data.t(), scale, TypeError), (data[:, :24], scale, ValueError), (data, scale[:8], ValueError),
                        (data, scale[:, :1], ValueError)):
        with pytest.raises(error, match="Fp4Rows"):
            itl.embedding_fwd(torch.zeros(4, dtype=torch.int64), itl.Fp4Rows(d, s))


def test_seeds():
    dev = torch.device("cpu")
    assert layer_ops._seed(-1, dev) == (-1, None) and layer_ops._seed(2 ** 64 - 1, dev) == (-1, None)
    assert layer_ops._seed(2 ** 63, dev) == (-2 ** 63, None) and layer_ops._seed(5, dev) == (5, None)
    for bad in (torch.zeros(2, dtype=torch.int64), torch.zeros(1), torch.zeros(1, dtype=torch.int32)):
        with pytest.raises(ValueError, match="seed"):
            layer_ops._seed(bad, dev)
    with pytest.raises(ValueError, match="seed"):
        layer_ops._drop_args(0.1, None, 0, 0, dev)
    assert layer_ops._drop_args(0.0, None, 3, 4, dev) == (0.0, 0, None, 0, 0)


def test_rows_of_few_bits_have_no_gradient():
    q = itl.Fp4Rows(torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8))
    with pytest.raises(TypeError, match="no gradient"):
        itl.embedding(torch.zeros(2, dtype=torch.int64), q)
    for rows in (q, itl.QuantizedRows(torch.zeros(4, 64), torch.zeros(4))):
        with pytest.raises(TypeError, match="no gradient"):
            itl.linear_token_logp(torch.zeros(2, 32), rows)


def test_head(L):
    flags = _lib.LOGP_TOKEN_FP4
    need = L.linear_token_logp_fwd_workspace_bytes(8, 128, 3000, 2, 3, flags, 0)
    assert need == L.linear_token_logp_fwd_workspace_bytes(8, 128, 3000, 2, 3, 0, 0)
    many = L.linear_token_logp_fwd_workspace_bytes(449, 128, 3000, 2, 3, flags, 0)
    assert many == L.linear_token_logp_fwd_workspace_bytes(449, 128, 3000, 2, 3, 0, 0)
    for bad in (flags | 1, flags | 4, 16):
        assert L.linear_token_logp_fwd_workspace_bytes(8, 128, 3000, 2, 3, bad, 0) == 0
    base = dict(h_ptr=P, ld_h=128, d=P, ld_d=64, s=P, ld_s=4, n=8, h=128, v=3000, tokens=P, tdt=0, m=2, ignore=-100, temp=1.0,
                rnd=0, k=3, logp=P, lse=P, ent=None, top=P, ids=P, rows=0, ws=P, ws_bytes=need, stream=None)
    expect(L.linear_token_logp_fp4_fwd, base, [
        (_lib.LOGP_ERR_SHAPE, dict(n=-1)), (_lib.LOGP_ERR_SHAPE, dict(h=96)), (_lib.LOGP_ERR_SHAPE, dict(v=0)),
        (_lib.LOGP_ERR_SHAPE, dict(m=257)), (_lib.LOGP_ERR_SHAPE, dict(ld_h=127)), (_lib.LOGP_ERR_SHAPE, dict(ld_d=63)),
        (_lib.LOGP_ERR_SHAPE, dict(ld_s=3)), (_lib.LOGP_ERR_SHAPE, dict(rows=-1)),
        (_lib.LOGP_ERR_SHAPE, dict(ld_h=(1 << 25) + 8)), (_lib.LOGP_ERR_SHAPE, dict(ld_d=(1 << 23) + 16)),
        (_lib.LOGP_ERR_SHAPE, dict(ld_s=(1 << 23) + 1)), (_lib.LOGP_ERR_VALUE, dict(k=65)),
        (_lib.LOGP_ERR_VALUE, dict(temp=0.0)), (_lib.LOGP_ERR_VALUE, dict(rnd=2)), (_lib.LOGP_ERR_DTYPE, dict(tdt=3)),
        (_lib.LOGP_ERR_NULL, dict(h_ptr=None)), (_lib.LOGP_ERR_NULL, dict(d=None)), (_lib.LOGP_ERR_NULL, dict(s=None)),
        (_lib.LOGP_ERR_NULL, dict(tokens=None)), (_lib.LOGP_ERR_NULL, dict(logp=None)), (_lib.LOGP_ERR_NULL, dict(ids=None)),
        (_lib.LOGP_ERR_ALIGN, dict(h_ptr=P + 8)), (_lib.LOGP_ERR_ALIGN, dict(ld_h=132)), (_lib.LOGP_ERR_ALIGN, dict(d=P + 8)),
        (_lib.LOGP_ERR_ALIGN, dict(ld_d=72)), (_lib.LOGP_ERR_WORKSPACE, dict(ws=None)),
        (_lib.LOGP_ERR_WORKSPACE, dict(ws_bytes=need - 1)), (OK, dict(n=0, h_ptr=None, d=None, s=None, ws=None)),
    ])


def test_head_binding():
    q = itl.Fp4Rows(torch.zeros(9, 32, dtype=torch.uint8), torch.zeros(9, 2, dtype=torch.uint8))
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="4-bit head takes no"):
        itl.linear_token_logp_fwd(x, q, logits_out=torch.zeros(4, 9))
    with pytest.raises(TypeError, match="bfloat16"):
        itl.linear_token_logp_fwd(x.float(), q)
    with pytest.raises(TypeError, match="QuantizedRows"):
        itl.linear_token_logp_fwd(itl.QuantizedRows(x.to(torch.float8_e4m3fn), torch.ones(4)), q)
    with pytest.raises(ValueError, match="ROCm device"):
        itl.linear_token_logp_fwd(x, q)


def test_embedding_gradient_workspace_of_long_batches(L):
    """Past eight tiles of 2048 tokens the keys are merged twice, in two buffers."""
    def keys(n):
        return L.embedding_bwd_workspace_bytes(n, 100, 8) - 3 * ((4 * n + 255) // 256 * 256) - \
            (2 * ((n + 31) // 32) * 32 + 255) // 256 * 256

    assert keys(2048) == 0 and keys(2304) == 8 * 2304 and keys(16384) == 8 * 16384 and keys(16640) == 16 * 16640


def test_dropout_without_a_seed():
    """As in the layer norm: none is needed where nothing is dropped, and one is asked for
    by name elsewhere (the rows' device is looked at next)."""
    x = torch.zeros(2, 8)
    for call in (itl.dropout_fwd, itl.dropout_bwd, itl.dropout):
        for p in (0, 0.0):
            with pytest.raises(ValueError, match="ROCm device"):
                call(x, p, None)
        for p in (0.5, NAN, -1.0):
            with pytest.raises(ValueError, match="needs a seed"):
                call(x, p, None)
    assert layer_ops._dropout_args(0.0, None, 3, 4, x.device) == (0.0, 0, None, 3, 4)
