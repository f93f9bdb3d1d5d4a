"""Workspace sizes and the binding's own checks at the edges of the token
operators, on the host (nothing here touches a device)."""

import os

import pytest

from invariant_token_log_amd import _lib
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
