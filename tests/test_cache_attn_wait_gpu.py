"""The last wait of a cache attention launch: when it runs out, the call says so.

In the test build (libli_lastwaittest.so) a wait gives up after 1 ms and no unit's last value product is
announced, so the softmax warps' wait before the output runs out with every other role done. The
product itself ends in microseconds: nothing is in flight when the kernel leaves."""
import time

import pytest
import torch

import cache_attn_ref as ref
from sparse_attention_token_lightning_b200 import build, li

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(B=1, S1=2, S2=128, G=16, Dm=128, Dr=0, topk=128),
                                dict(B=3, S1=1, S2=400, G=40, Dm=512, Dr=64, topk=129),
                                dict(B=1, S1=200, S2=200, G=16, Dm=512, Dr=64, topk=150, causal=True),
                                dict(B=1, S1=1, S2=2000, G=16, Dm=512, Dr=64, topk=1500)])
def test_the_last_wait_is_reported(monkeypatch, kw):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    p = ref.make(seed=11, **kw)
    before = p.call(li.cache_attention, return_stats=True)
    monkeypatch.setattr(li, "_lib", li.load(build.build_last_wait_test()))
    t0 = time.perf_counter()
    with pytest.raises(li.LiError) as e:
        p.call(li.cache_attention)
    assert e.value.status == 5 and time.perf_counter() - t0 < 20.0       # LI_ERR_DEVICE_TIMEOUT
    monkeypatch.undo()
    assert all(torch.equal(a, b) for a, b in zip(before, p.call(li.cache_attention, return_stats=True)))
