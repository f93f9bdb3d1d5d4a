"""Refusals of the token operators and the norm, on the host: every bad
argument gets its documented status before any HIP call, and the binding's own
checks raise before any device work (nothing here touches a device)."""

import os

import pytest
import torch

import invariant_token_log_amd as itl
from invariant_token_log_amd import _lib, token_ops
from invariant_token_log_amd.build import LIB_PATH, build

P = 0x10000  # a non-NULL, 256-byte aligned address that the checks never dereference
BIG = 1 << 60
OK = _lib.LOGP_OK


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


def test_token_forward(L):
    base = dict(logits=P, dtype=1, n=4, v=5000, ld=5000, tokens=P, tdt=0, m=2, ignore=-100, tile=4096, k=3,
                logp=P, lse=P, ent=None, top=P, ids=P, ws=P, ws_bytes=BIG, stream=None)
    need = L.token_logp_fwd_workspace_bytes(4, 5000, 1, 4096, 3)
    assert need == 3 * 256 + 1024  # m, s, w of 4 x 2 tiles; 4 x 64 group keys
    expect(L.token_logp_fwd, base, [
        (_lib.LOGP_ERR_DTYPE, dict(dtype=3)), (_lib.LOGP_ERR_DTYPE, dict(tdt=2)),
        (_lib.LOGP_ERR_SHAPE, dict(n=-1)), (_lib.LOGP_ERR_SHAPE, dict(v=0)), (_lib.LOGP_ERR_SHAPE, dict(ld=4999)),
        (_lib.LOGP_ERR_SHAPE, dict(m=-1)), (_lib.LOGP_ERR_SHAPE, dict(m=257)), (_lib.LOGP_ERR_SHAPE, dict(n=0, m=257)),
        (_lib.LOGP_ERR_TILE, dict(tile=1000)), (_lib.LOGP_ERR_TILE, dict(dtype=0, tile=8192)),
        (_lib.LOGP_ERR_SHAPE, dict(v=512 * 4097, ld=512 * 4097, tile=512)),
        (_lib.LOGP_ERR_VALUE, dict(k=-1)), (_lib.LOGP_ERR_VALUE, dict(k=65)), (_lib.LOGP_ERR_VALUE, dict(v=2, k=3)),
        (_lib.LOGP_ERR_NULL, dict(logits=None)), (_lib.LOGP_ERR_NULL, dict(tokens=None)),
        (_lib.LOGP_ERR_NULL, dict(logp=None)), (_lib.LOGP_ERR_NULL, dict(top=None)),
        (_lib.LOGP_ERR_NULL, dict(ids=None)),
        (_lib.LOGP_ERR_WORKSPACE, dict(ws=None)), (_lib.LOGP_ERR_WORKSPACE, dict(ws=P + 16)),
        (_lib.LOGP_ERR_WORKSPACE, dict(ws_bytes=need - 1)),
        (OK, dict(n=0, logits=None, tokens=None, logp=None, ws=None)),
    ])
    assert L.token_logp_fwd_workspace_bytes(4, 5000, 1, 1000, 3) == 0
    assert L.token_logp_fwd_workspace_bytes(4, 5000, 1, 4096, 65) == 0


def test_token_backward(L):
    base = dict(logits=P, dtype=1, n=4, v=5000, ld=5000, tokens=P, tdt=0, m=2, ignore=-100, ids=P, k=3, lse=P, g=P,
                gt=P, ent=None, gent=None, d=P, ld_out=5000, stream=None)
    expect(L.token_logp_bwd, base, [
        (_lib.LOGP_ERR_DTYPE, dict(dtype=-1)), (_lib.LOGP_ERR_DTYPE, dict(tdt=9)),
        (_lib.LOGP_ERR_SHAPE, dict(ld_out=4999)), (_lib.LOGP_ERR_SHAPE, dict(ld=1)), (_lib.LOGP_ERR_SHAPE, dict(m=300)),
        (_lib.LOGP_ERR_VALUE, dict(k=65)), (_lib.LOGP_ERR_NULL, dict(lse=None)), (_lib.LOGP_ERR_NULL, dict(g=None)),
        (_lib.LOGP_ERR_NULL, dict(gt=None)), (_lib.LOGP_ERR_NULL, dict(ids=None)), (_lib.LOGP_ERR_NULL, dict(d=None)),
        (_lib.LOGP_ERR_NULL, dict(tokens=None)), (_lib.LOGP_ERR_NULL, dict(ent=P)), (_lib.LOGP_ERR_NULL, dict(gent=P)),
        (OK, dict(n=0, logits=None, d=None)),
    ])


def head_base():
    return dict(h_ptr=P, ld_h=128, w_ptr=P, ld_w=128, n=8, h=128, v=3000, tokens=P, tdt=0, m=2, ignore=-100, temp=1.0,
                rnd=0, k=3, logp=P, lse=P, ent=None, top=P, ids=P, z=None, zdt=0, ld_z=0, prep=None, prep_bytes=0,
                rows=0, ws=P, ws_bytes=BIG, stream=None)


def test_head_forward(L):
    base = head_base()
    need = L.linear_token_logp_fwd_workspace_bytes(8, 128, 3000, 2, 3, 0, 0)
    prep = L.linear_logp_prepared_bytes(3000, 128)
    expect(L.linear_token_logp_fwd, base, [
        (_lib.LOGP_ERR_SHAPE, dict(h=96)), (_lib.LOGP_ERR_SHAPE, dict(h=0)), (_lib.LOGP_ERR_SHAPE, dict(n=-1)),
        (_lib.LOGP_ERR_SHAPE, dict(v=0)), (_lib.LOGP_ERR_SHAPE, dict(ld_h=64)), (_lib.LOGP_ERR_SHAPE, dict(ld_w=64)),
        (_lib.LOGP_ERR_SHAPE, dict(v=(1 << 31) + 1)), (_lib.LOGP_ERR_SHAPE, dict(rows=-1)),
        (_lib.LOGP_ERR_SHAPE, dict(m=257)), (_lib.LOGP_ERR_VALUE, dict(k=65)), (_lib.LOGP_ERR_VALUE, dict(v=2, k=3)),
        (_lib.LOGP_ERR_VALUE, dict(temp=0.0)), (_lib.LOGP_ERR_VALUE, dict(temp=float("nan"))),
        (_lib.LOGP_ERR_VALUE, dict(temp=1e-40)), (_lib.LOGP_ERR_VALUE, dict(rnd=2)), (_lib.LOGP_ERR_DTYPE, dict(tdt=5)),
        (_lib.LOGP_ERR_DTYPE, dict(z=P, zdt=1, ld_z=3000)), (_lib.LOGP_ERR_SHAPE, dict(z=P, ld_z=2999)),
        (_lib.LOGP_ERR_ALIGN, dict(h_ptr=P + 2)), (_lib.LOGP_ERR_ALIGN, dict(w_ptr=P + 8)),
        (_lib.LOGP_ERR_ALIGN, dict(ld_w=132)), (_lib.LOGP_ERR_NULL, dict(w_ptr=None)),
        (_lib.LOGP_ERR_NULL, dict(tokens=None)), (_lib.LOGP_ERR_NULL, dict(logp=None)),
        (_lib.LOGP_ERR_NULL, dict(ids=None)), (_lib.LOGP_ERR_SHAPE, dict(prep=P, prep_bytes=prep - 1)),
        (_lib.LOGP_ERR_ALIGN, dict(prep=P + 8, prep_bytes=prep)), (_lib.LOGP_ERR_WORKSPACE, dict(ws=None)),
        (_lib.LOGP_ERR_WORKSPACE, dict(ws_bytes=need - 1)), (OK, dict(n=0, h_ptr=None, w_ptr=None, ws=None)),
    ])
    # the logits' part of the workspace: none for one given token and nothing else, a row chunk's otherwise
    small = L.linear_token_logp_fwd_workspace_bytes(8192, 128, 30000, 1, 0, 0, 0)
    chunk = L.linear_token_logp_fwd_workspace_bytes(8192, 128, 30000, 1, 5, 0, 256)
    whole = L.linear_token_logp_fwd_workspace_bytes(8192, 128, 30000, 1, 5, 0, 8192)
    kept = L.linear_token_logp_fwd_workspace_bytes(8192, 128, 30000, 1, 5, _lib.LOGP_TOKEN_KEEPS_LOGITS, 0)
    assert chunk < whole and whole - kept == 8192 * 30000 * 4 and 256 * 30000 * 4 < chunk < 2 * 256 * 30000 * 4
    assert small < kept + 4096
    assert L.linear_token_logp_fwd_workspace_bytes(8, 96, 30000, 1, 5, 0, 0) == 0


def test_8bit_head(L):
    base = dict(h_ptr=P, ld_h=128, hs=P, w_ptr=P, ld_w=128, ws_=P, n=8, h=128, v=3000, tokens=P, tdt=0, m=2,
                ignore=-100, temp=1.0, k=0, logp=P, lse=P, ent=None, top=None, ids=None, rows=0, ws=P, ws_bytes=BIG,
                stream=None)
    expect(L.linear_token_logp_q8_fwd, base, [
        (_lib.LOGP_ERR_SHAPE, dict(h=100)), (_lib.LOGP_ERR_SHAPE, dict(ld_w=64)),
        (_lib.LOGP_ERR_SHAPE, dict(ld_h=(1 << 23) + 16)), (_lib.LOGP_ERR_ALIGN, dict(h_ptr=P + 4)),
        (_lib.LOGP_ERR_ALIGN, dict(ld_h=136)), (_lib.LOGP_ERR_NULL, dict(hs=None)), (_lib.LOGP_ERR_NULL, dict(ws_=None)),
        (_lib.LOGP_ERR_NULL, dict(k=2)), (_lib.LOGP_ERR_VALUE, dict(temp=-1.0)), (_lib.LOGP_ERR_VALUE, dict(k=100)),
        (_lib.LOGP_ERR_WORKSPACE, dict(ws=None)), (OK, dict(n=0, h_ptr=None)),
    ])


def test_head_backward(L):
    base = dict(h_ptr=P, ld_h=128, w_ptr=P, ld_w=128, n=8, h=128, v=3000, tokens=P, tdt=0, m=2, ignore=-100, ids=P, k=3,
                temp=1.0, rnd=0, z=None, zdt=0, ld_z=0, prep=None, prep_bytes=0, lse=P, logp=P, top=P, g=P, gt=P,
                ent=None, gent=None, odt=0, dh=P, ld_dh=128, dw=P, ld_dw=128, chunk=0, ws=P, ws_bytes=BIG, stream=None)
    need = L.linear_token_logp_bwd_workspace_bytes(8, 128, 3000, 3, 0)
    assert need == L.linear_logp_bwd_workspace_bytes(8, 128, 3000, 256, 3, 0) + 512
    expect(L.linear_token_logp_bwd, base, [
        (_lib.LOGP_ERR_SHAPE, dict(h=60)), (_lib.LOGP_ERR_SHAPE, dict(chunk=-1)), (_lib.LOGP_ERR_SHAPE, dict(ld_dh=64)),
        (_lib.LOGP_ERR_SHAPE, dict(ld_dw=64)), (_lib.LOGP_ERR_DTYPE, dict(odt=2)), (_lib.LOGP_ERR_NULL, dict(dh=None, dw=None)),
        (_lib.LOGP_ERR_NULL, dict(logp=None)), (_lib.LOGP_ERR_NULL, dict(top=None)), (_lib.LOGP_ERR_NULL, dict(g=None)),
        (_lib.LOGP_ERR_NULL, dict(gt=None)), (_lib.LOGP_ERR_NULL, dict(lse=None)), (_lib.LOGP_ERR_NULL, dict(ent=P)),
        (_lib.LOGP_ERR_DTYPE, dict(z=P, zdt=1, ld_z=3000)), (_lib.LOGP_ERR_ALIGN, dict(z=P + 4, ld_z=3000)),
        (_lib.LOGP_ERR_SHAPE, dict(z=P, ld_z=2996)), (_lib.LOGP_ERR_VALUE, dict(temp=float("inf"))),
        (_lib.LOGP_ERR_WORKSPACE, dict(ws_bytes=need - 1)), (_lib.LOGP_ERR_ALIGN, dict(w_ptr=P + 2)),
        (OK, dict(n=0, dw=None)),
    ])


def test_norm(L):
    base = dict(x=P, ld_x=100, r=P, ld_r=100, w=P, dtype=1, n=4, h=100, eps=1e-6, y=P, ld_y=100, s=P, ld_s=100, rstd=None,
                stream=None)
    expect(L.rms_norm_fwd, base, [
        (_lib.LOGP_ERR_DTYPE, dict(dtype=4)), (_lib.LOGP_ERR_SHAPE, dict(h=0)), (_lib.LOGP_ERR_SHAPE, dict(h=65537, ld_x=1 << 20)),
        (_lib.LOGP_ERR_SHAPE, dict(ld_x=99)), (_lib.LOGP_ERR_SHAPE, dict(ld_r=99)), (_lib.LOGP_ERR_SHAPE, dict(ld_s=99)),
        (_lib.LOGP_ERR_SHAPE, dict(ld_y=99)), (_lib.LOGP_ERR_SHAPE, dict(n=-1)), (_lib.LOGP_ERR_SHAPE, dict(n=1 << 31)),
        (_lib.LOGP_ERR_VALUE, dict(eps=-1.0)), (_lib.LOGP_ERR_VALUE, dict(eps=float("nan"))),
        (_lib.LOGP_ERR_NULL, dict(x=None)), (_lib.LOGP_ERR_NULL, dict(w=None)), (_lib.LOGP_ERR_NULL, dict(y=None)),
        (_lib.LOGP_ERR_NULL, dict(s=None)), (OK, dict(n=0, x=None)),
    ])
    base = dict(x=P, ld_x=100, r=None, ld_r=0, w=None, dtype=0, n=4, h=100, eps=0.0, q=P, ld_q=100, scale=P, s=None, ld_s=0,
                stream=None)
    expect(L.rms_norm_q8_fwd, base, [
        (_lib.LOGP_ERR_SHAPE, dict(ld_q=50)), (_lib.LOGP_ERR_NULL, dict(q=None)), (_lib.LOGP_ERR_NULL, dict(scale=None)),
        (_lib.LOGP_ERR_NULL, dict(r=P, ld_r=100)), (_lib.LOGP_ERR_DTYPE, dict(dtype=-1)), (OK, dict(n=0)),
    ])
    base = dict(s=P, ld_s=100, w=P, rstd=P, dy=P, ld_dy=100, ds=None, ld_ds=0, dtype=2, n=4, h=100, dx=P, ld_dx=100, dw=P,
                ws=P, ws_bytes=BIG, stream=None)
    need = L.rms_norm_bwd_workspace_bytes(4, 100)
    assert need == 1792  # four partial rows of 100
    expect(L.rms_norm_bwd, base, [
        (_lib.LOGP_ERR_SHAPE, dict(ld_dy=1)), (_lib.LOGP_ERR_SHAPE, dict(ds=P, ld_ds=1)), (_lib.LOGP_ERR_SHAPE, dict(ld_dx=99)),
        (_lib.LOGP_ERR_NULL, dict(rstd=None)), (_lib.LOGP_ERR_NULL, dict(dx=None)), (_lib.LOGP_ERR_WORKSPACE, dict(ws=None)),
        (_lib.LOGP_ERR_WORKSPACE, dict(ws_bytes=need - 1)), (_lib.LOGP_ERR_DTYPE, dict(dtype=3)), (OK, dict(n=0, dw=None)),
    ])


def test_binding_refuses_before_device_work():
    """CPU tensors and mismatched arguments never reach the library."""
    bf = torch.bfloat16
    x, tok = torch.zeros(4, 100, dtype=bf), torch.zeros(4, 2, dtype=torch.int64)
    with pytest.raises(ValueError, match="ROCm"):
        itl.token_logp_fwd(x, tok)
    with pytest.raises(ValueError, match="ROCm"):
        itl.batch_invariant_token_logp(x, tok, top_k=2)
    with pytest.raises(ValueError, match="ROCm"):
        itl.linear_token_logp_fwd(x[:, :64].contiguous(), x[:, :64].contiguous(), tok)
    with pytest.raises(TypeError, match="both"):
        itl.linear_token_logp_fwd(itl.QuantizedRows(x, x), x)
    with pytest.raises(ValueError, match="ROCm"):
        itl.rms_norm_fwd(x, x[0])
    with pytest.raises(ValueError, match="ROCm"):
        itl.quantize_rows(x)
    q = itl.QuantizedRows(torch.zeros(4, 64, dtype=torch.float8_e4m3fn), torch.zeros(4))
    with pytest.raises(ValueError, match="ROCm"):
        itl.linear_token_logp_fwd(q, q)
    with pytest.raises(ValueError, match="8-bit head"):
        itl.linear_token_logp_fwd(q, q, round_logits=True)
    with pytest.raises(TypeError, match="scale"):
        itl.linear_token_logp_fwd(q, itl.QuantizedRows(q.data, q.scale.half()))
    with pytest.raises(ValueError, match="8-bit head"):
        itl.norm_linear_token_logp(x, x[0], q, save_logits=True)
    for bad in (65, -1):
        with pytest.raises(ValueError, match="top_k"):
            itl.linear_token_logp_fwd(q, q, top_k=bad)


def test_output_names():
    """An output buffer under a name that does not exist, or of an output that
    was not asked for, is refused rather than left unwritten."""
    outputs = lambda ent, **given: token_ops._Outputs(2, (2,), 1, 0, ent, torch.device("cpu"), given)
    with pytest.raises(TypeError):
        outputs(False, logps_out=torch.empty(2, 1))
    with pytest.raises(ValueError):
        outputs(False, entropy_out=torch.empty(2))
    e = torch.empty(2)
    assert outputs(True, entropy_out=e).entropy is e
