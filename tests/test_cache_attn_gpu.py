"""Attention over the E4M3 cache (li_cache_attention) against a 64-bit form; tolerances are derived
in cache_attn_ref from the kernel's arithmetic."""
import os
import subprocess
import sys
import time

import pytest
import torch

import cache_attn_ref as ref
from sparse_attention_token_lightning_b200 import build, li

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    li.lib()


def run(p, **kw):
    out, smax, ssum = p.call(li.cache_attention, return_stats=True, **kw)
    torch.cuda.synchronize()
    return out, smax, ssum


CASES = {
    # B, S1, S2, G, Dm, Dr, topk, block
    "one_tile": dict(B=1, S1=2, S2=128, G=16, Dm=128, Dr=0, topk=128),
    "one_key": dict(B=2, S1=1, S2=40, G=16, Dm=512, Dr=64, topk=1),
    "single_token": dict(B=1, S1=1, S2=3000, G=16, Dm=512, Dr=64, topk=2048),
    "decode": dict(B=5, S1=1, S2=1000, G=16, Dm=512, Dr=64, topk=700),
    "odd_heads": dict(B=3, S1=2, S2=300, G=5, Dm=256, Dr=64, topk=129, block=17),
    "one_head": dict(B=1, S1=4, S2=200, G=1, Dm=384, Dr=0, topk=200, block=1),
    "heads17": dict(B=2, S1=3, S2=400, G=17, Dm=512, Dr=64, topk=300),
    "heads32": dict(B=2, S1=2, S2=500, G=32, Dm=512, Dr=64, topk=385, block=1024),
    "heads40": dict(B=2, S1=1, S2=500, G=40, Dm=256, Dr=0, topk=500, block=48),
    "heads128": dict(B=2, S1=2, S2=600, G=128, Dm=512, Dr=64, topk=512),
    "causal": dict(B=1, S1=200, S2=200, G=16, Dm=512, Dr=64, topk=150, causal=True),
    "many_rows": dict(B=1, S1=700, S2=260, G=8, Dm=128, Dr=64, topk=200, causal=True),
    "many_rows_32": dict(B=2, S1=300, S2=300, G=20, Dm=128, Dr=0, topk=64, causal=True),
    "dense": dict(B=3, S1=4, S2=333, G=16, Dm=512, Dr=64, topk=200, block=None),
    "any_scales": dict(B=2, S1=3, S2=400, G=16, Dm=256, Dr=64, topk=300, pow2=False),
    "wild_scales": dict(B=2, S1=2, S2=300, G=16, Dm=128, Dr=64, topk=256, spread=6.0, q_std=0.01),
    "peaked": dict(B=2, S1=3, S2=900, G=16, Dm=512, Dr=64, topk=900, scale=0.5),
    "flat": dict(B=1, S1=2, S2=900, G=32, Dm=512, Dr=64, topk=900, q_std=1e-3),
    # two, four and eight CTAs to a row (the single token above: eight)
    "shared_by_two": dict(B=40, S1=1, S2=700, G=16, Dm=256, Dr=64, topk=600),
    "shared_by_two_32": dict(B=35, S1=1, S2=700, G=24, Dm=128, Dr=0, topk=641),
    "shared_by_four": dict(B=5, S1=4, S2=900, G=7, Dm=512, Dr=0, topk=777, block=48),
    "shared_by_eight": dict(B=1, S1=2, S2=1200, G=32, Dm=512, Dr=64, topk=1153, pow2=False),
    "topk8192": dict(B=1, S1=2, S2=9000, G=16, Dm=128, Dr=0, topk=8192),
}


@pytest.mark.parametrize("name", list(CASES))
def test_parity(name):
    p = ref.make(seed=len(name), **CASES[name])
    rows = None if p.q.shape[0] * p.q.shape[1] <= 40 else [0, 1, 2, 63, 127, 128, 150, p.q.shape[1] - 1]
    ref.check(p, *run(p), rows=rows, label=name)


def test_holes_repeats_and_rows_without_keys():
    p = ref.make(3, 20, 400, 16, 256, 64, 300, seed=1)
    g = torch.Generator().manual_seed(2)
    p.idx[torch.rand(p.idx.shape, generator=g) < 0.3] = -1
    p.idx[0, 3] = -1                        # nothing selected
    p.idx[1, 4] = -1
    p.idx[1, 4, 0, 299] = 7                 # one key, the last entry
    p.idx[2, 5, 0, :128] = -1               # an empty first tile
    p.idx[0, 9, 0, 10:40] = p.idx[0, 9, 0].max()
    p.idx[2, :, 0, :] = torch.where(torch.arange(300) % 2 == 0, p.idx[2, :, 0, :], -5)
    ref.check(p, *run(p))
    # few rows, so that empty pieces meet full ones in the joined result
    one = ref.make(1, 1, 3000, 16, 512, 64, 2048, seed=3)
    one.idx[0, 0, 0, 100:1800] = -1
    ref.check(one, *run(one))
    none = ref.make(1, 1, 3000, 40, 512, 64, 2048, seed=3)
    none.idx[:] = -1
    ref.check(none, *run(none))


@pytest.mark.parametrize("G", [16, 40])
def test_extreme_queries(G):
    """q of every magnitude, zero heads, one large element per head (the split's range), and a
    reference that moves in every tile (scores that rise along the selection)."""
    p = ref.make(1, 6, 700, G, 512, 64, 600, seed=4)
    p.q[0, 0] *= 2.0 ** -60
    p.q_rope[0, 0] *= 0
    p.q[0, 1] = 0
    p.q[0, 2, :, 5] = 3000.0
    p.q[0, 3, 1:4] = 0
    p.q[0, 4] *= 2.0 ** 70
    p.q[0, 4] *= (torch.arange(512) == 3)
    p.q[0, 4] *= 2.0 ** -75
    # rising scores: selection sorted by the score of head 0
    k = (p.codes.double() * p.descale.double()[..., None, None]).reshape(-1, 512)
    at = ref.row_keys(p, 0, p.idx[0, 5, 0])
    order = (k[at] @ p.q[0, 5, 0].double()).argsort()
    p.idx[0, 5, 0] = p.idx[0, 5, 0][order]
    p.q[0, 5, 0] *= 4
    ref.check(p, *run(p))


def test_non_finite_values_show_and_stay_in_their_rows():
    p = ref.make(1, 4, 300, 16, 256, 64, 200, seed=5)
    p.idx[0, 1, 0, 50] = 17
    p.idx[0, (0, 2, 3)] = torch.where(p.idx[0, (0, 2, 3)] == 17, torch.full_like(p.idx[0, (0, 2, 3)], 18),
                                      p.idx[0, (0, 2, 3)])
    bs = p.codes.shape[1]
    blk, off = int(p.table[0, 17 // bs]), 17 % bs
    p.codes.view(torch.uint8)[blk, off, 0, 9] = 127         # a NaN code in key 17
    p.q[0, 2, 3, 4] = float("inf")
    out, smax, ssum = run(p)
    assert torch.isnan(out[0, 1].float()).all()
    assert torch.isnan(out[0, 2, 3].float()).all()
    ref.check(p, out, smax, ssum, rows=[0, 3])
    q2 = p.q.clone()
    q2[0, 2, 3, 4] = 1.0
    p.q = q2
    ref.check(p, *run(p), rows=[0, 2, 3])


def test_unselected_rows_are_not_read():
    """Cache rows that nothing selects may hold anything: NaN codes, scales and rope parts change no
    bit, also where a short selection fills its tile."""
    p = ref.make(2, 3, 500, 16, 512, 64, 90, seed=6)
    a = run(p)
    used = torch.zeros(p.descale.numel(), dtype=torch.bool)
    for b in range(2):
        for i in range(3):
            used[ref.row_keys(p, b, p.idx[b, i, 0])] = True
    p.codes.view(torch.uint8).view(-1, 512)[~used] = 255
    p.descale.view(-1)[~used] = float("nan")
    p.k_rope.view(-1, 64)[~used] = float("inf")
    for x, y in zip(a, run(p)):
        assert torch.equal(x, y)


def test_bad_entries_are_reported_and_select_nothing():
    p = ref.make(2, 3, 100, 16, 128, 0, 64, block=16, seed=7)
    clean = run(p)

    def bits(p):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = p.call(li.cache_attention, return_stats=True, check=False, device_status=st)
        torch.cuda.synchronize()
        return int(st), out

    assert bits(p)[0] == 0
    p.idx[0, 0, 0, 5] = 100
    p.idx[1, 2, 0, 63] = 2 ** 31 - 1
    b, out = bits(p)
    assert b == li.DEVERR_LENGTHS
    ref.check(p, *out)
    with pytest.raises(li.LiError):
        p.call(li.cache_attention)
    p = ref.make(2, 3, 100, 16, 128, 0, 64, block=16, seed=7)
    p.table[0, 2] = -1
    p.table[1, 3] = p.codes.shape[0]
    b, out = bits(p)
    assert b == li.DEVERR_TABLE
    ref.check(p, *out)
    p = ref.make(2, 3, 100, 16, 128, 0, 64, block=16, seed=7)
    at = int(ref.row_keys(p, 0, p.idx[0, 1, 0])[3])
    for bad in (0.0, -1.0, float("nan"), float("inf"), 1e-38):
        p.descale.view(-1)[at] = bad
        b, out = bits(p)
        assert b == li.DEVERR_DESCALE
        q = ref.make(2, 3, 100, 16, 128, 0, 64, block=16, seed=7)
        flat = torch.tensor([[int(r) for r in ref.row_keys(q, bb, torch.arange(100))] for bb in range(2)])
        pos = (flat == at).nonzero()[0]
        q.idx[pos[0]] = torch.where(q.idx[pos[0]] == int(pos[1]), torch.full_like(q.idx[pos[0]], -1), q.idx[pos[0]])
        ref.check(q, *out)
    assert clean[0].shape == (2, 3, 16, 128)


def test_reruns_graphs_and_streams_are_bit_identical():
    p = ref.make(3, 2, 2500, 32, 512, 64, 2048, seed=8)
    c = lambda t: t.cuda()  # noqa: E731
    t = dict(q_rope=c(p.q_rope), rope_cache=c(p.k_rope), block_table=c(p.table), s2=p.s2)
    q, codes, descale, idx = c(p.q), c(p.codes), c(p.descale), c(p.idx)
    a = li.cache_attention(q, codes, descale, idx, p.scale, **t)
    for _ in range(3):
        assert torch.equal(a, li.cache_attention(q, codes, descale, idx, p.scale, **t))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [li.cache_attention(q, codes, descale, idx, p.scale, stream=side, check=False, **t)]
    outs.append(li.cache_attention(q, codes, descale, idx, p.scale, check=False, **t))   # two at once
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    q2 = torch.zeros_like(q)
    with torch.cuda.graph(graph):
        outs.append(li.cache_attention(q2, codes, descale, idx, p.scale, check=False, **t))
    q2.copy_(q)
    graph.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(a, o)


@pytest.mark.parametrize("name", ["single_token", "shared_by_two", "causal", "heads128"])
def test_a_wait_that_runs_out_is_reported(monkeypatch, name):
    """The test build gives up a wait after 1 ms and gathers nothing: the first product's wait runs out,
    every role leaves, the CTAs of a cluster still meet, and the call reports it. The context stays
    usable: the library's own call gives the same bits as before."""
    p = ref.make(seed=len(name), **CASES[name])
    before = run(p)
    monkeypatch.setattr(li, "_lib", li.load(build.build_wait_test()))
    t0 = time.perf_counter()
    with pytest.raises(li.LiError) as e:
        run(p)
    assert e.value.status == 5 and time.perf_counter() - t0 < 20.0       # LI_ERR_DEVICE_TIMEOUT
    monkeypatch.undo()
    assert all(torch.equal(a, b) for a, b in zip(before, run(p)))


FIRST_CALL = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import cache_attn_ref as ref
from sparse_attention_token_lightning_b200 import li
p = ref.make(1, 200, 200, 16, 512, 64, 150, causal=True, seed=6)
c = lambda t: t.cuda()
args = c(p.q), c(p.codes), c(p.descale), c(p.idx), p.scale
kw = dict(q_rope=c(p.q_rope), rope_cache=c(p.k_rope), block_table=c(p.table), s2=p.s2, check=False)
outs = [li.cache_attention(*args, **kw) for _ in range(4)]
torch.cuda.synchronize()
ref.check(p, outs[0], rows=range(0, 200, 3))
assert all(torch.equal(outs[0], o) for o in outs[1:])
"""


def test_the_first_call_of_a_process():
    """A cold start spreads the kernel's roles in time as no later call does: its bits are those of
    every other call."""
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_CALL.format(root=os.path.dirname(tests), tests=tests)
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)


def test_no_rows():
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    for B, S1 in ((0, 3), (2, 0)):
        out, smax, ssum = li.cache_attention(
            z(B, S1, 16, 128, dtype=torch.bfloat16), z(B, 9, 1, 128, dtype=torch.float8_e4m3fn), z(B, 9),
            z(B, S1, 1, 4, dtype=torch.int32), 0.1, return_stats=True)
        assert out.shape == (B, S1, 16, 128) and smax.shape == (B, 1, S1, 16)
