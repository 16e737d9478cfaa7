"""Calls of the cache entry points that have to be taken, without a GPU: pointers are fake, and nothing is
launched or the launch fails for want of a device (LI_ERR_CUDA), which is not a refusal."""
import ctypes

import pytest

from sparse_attention_token_lightning_b200 import build as libbuild
from sparse_attention_token_lightning_b200 import li
from test_rope_cache_host import _DENSE_ATTN, _cache, _cattn


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return li.lib()


@pytest.mark.parametrize("kw", [dict(batch=0), dict(s1=0), dict(_DENSE_ATTN, batch=0, codes=None, descale=None),
                                dict(batch=0, q=None, sparse_indices=None)])
def test_attention_without_rows_needs_no_pointers(L, kw):
    """An empty tensor has no address: with a rope part as without."""
    for rope in (dict(), dict(Dr=64, q_rope=None, k_rope=0x70000), dict(Dr=64, q_rope=None, k_rope=None)):
        assert L.li_cache_attention(ctypes.byref(_cattn(**kw, **rope)), None, None, None, None) == 0, (kw, rope)
