"""Workspace sizes and the binding's own checks at the edges of the token
operators, on the host (nothing here touches a device)."""

import os

import pytest
import torch

from invariant_token_log_amd import _lib, token_ops
from invariant_token_log_amd.build import LIB_PATH, build


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(LIB_PATH):
        build()
    return _lib.lib()


# one token; tokens and alternatives with kept logits; nothing but the lse
@pytest.mark.parametrize("m,k,flags", [(1, 0, 0), (3, 5, _lib.LOGP_TOKEN_KEEPS_LOGITS), (0, 0, 0),
                                       (1, 0, _lib.LOGP_TOKEN_Q8), (0, 0, _lib.LOGP_TOKEN_Q8)])
def test_row_chunk_bounds_the_workspace(L, m, k, flags):
    """row_chunk bounds the workspace whether or not it holds logits, and the
    default does too."""
    need = lambda n, chunk: L.linear_token_logp_fwd_workspace_bytes(n, 128, 30000, m, k, flags, chunk)  # noqa: E731
    assert need(1 << 20, 256) == need(256, 0) < need(512, 0)
    assert need(1 << 20, 300) == need(512, 0)
    assert need(1 << 20, 0) == need(65536, 0) > need(65536, 4096)
    assert need(100, 256) == need(100, 0)


def test_gradients_in_another_layout_are_refused():
    """As many entries in another layout are no [*lead, M] gradient."""
    cpu = torch.device("cpu")
    g = torch.arange(6.0).view(2, 3)
    for good in (g, g.double(), g.view(2, 1, 3), g.repeat(1, 2)[:, :3]):
        assert torch.equal(token_ops._row_grad(good, 2, 3, "grad_logp", cpu).view(2, 3), g)
    for bad in (g.t(), g.reshape(-1), g.view(3, 2), g.view(1, 6), torch.zeros(4, 3), torch.zeros(())):
        with pytest.raises(ValueError, match="grad_logp"):
            token_ops._row_grad(bad, 2, 3, "grad_logp", cpu)
    ids = torch.zeros(2, 3, dtype=torch.int64)
    with pytest.raises(ValueError, match="grad_top_logp"):
        token_ops._alternatives(ids, g.t(), 2, cpu)
    assert token_ops._alternatives(ids, g, 2, cpu)[1] == 3


def test_gradient_without_tokens_is_refused():
    """A gradient of log-probabilities without the tokens that it belongs to
    would be lost."""
    cpu = torch.device("cpu")
    g = torch.arange(6.0).view(2, 3)
    with pytest.raises(ValueError, match="token_ids"):
        token_ops._token_grad(g, 2, 0, cpu)
    assert token_ops._token_grad(torch.empty(2, 0), 2, 0, cpu) is None
    assert token_ops._token_grad(None, 2, 0, cpu) is None
    assert torch.equal(token_ops._token_grad(g, 2, 3, cpu), g)


def test_saved_logits_keep_their_row_stride():
    """Rows that overlap keep their stride for the library to refuse: taken as
    v columns apart, rows past the first would be read behind the data."""
    from invariant_token_log_amd.ops import _saved_stride

    row = torch.zeros(1, 8)
    assert _saved_stride(row.expand(5, 8), 5, 8) == 0
    assert _saved_stride(torch.zeros(40).as_strided((5, 8), (4, 1)), 5, 8) == 4
    assert _saved_stride(torch.zeros(5, 12)[:, :8], 5, 8) == 12
    assert _saved_stride(row, 1, 8) == 8
    assert _saved_stride(torch.zeros(1, 12)[:, :8], 1, 8) == 12
