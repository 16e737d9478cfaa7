"""Calls of the cache entry points that have to be taken or refused, without a GPU: pointers are fake, and
nothing is launched."""
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


@pytest.mark.parametrize("kw", [dict(x_batch_stride=127, x_row_stride=256), dict(x_batch_stride=128, x_row_stride=255),
                                dict(x_batch_stride=1151, x_row_stride=128), dict(x_batch_stride=0, x_row_stride=128)])
def test_read_refuses_batches_that_overlap(L, kw):
    assert L.li_cache_read(ctypes.byref(_cache(**kw)), None) == 1, kw
