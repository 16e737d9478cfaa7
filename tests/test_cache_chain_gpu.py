"""The rotation, the quantised cache, the indexer over it and the attention over what it selects, run
together as a model layer does, and on the bounds-checked build of the library.

Each stage is checked against its 64-bit form on what the stage before left on the device, with
that stage's own tolerance (rotation: test_rope_gpu; attention: cache_attn_ref; the codes and the
selection are exact)."""
import math
import os
import subprocess
import sys

import pytest
import torch

import cache_attn_ref
import parity
import rope_cache_ref as ref
from sparse_attention_token_lightning_b200 import build, li, synthetic

pytestmark = pytest.mark.gpu

LENS, S1, HEADS, TOPK, BLOCK, G = [300, 129, 1], 2, 8, 40, 16, 20


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    li.lib()


class Layer:
    """Inputs of one layer, its caches, and the calls that fill and read them. The last sequence has
    one key and two query rows, so its first row selects nothing."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
        B, T = len(LENS), sum(LENS)
        self.pb = synthetic.quantized(synthetic.paged(LENS, S1, HEADS, TOPK, block_size=BLOCK, seed=31)).to("cuda")
        self.qi, self.ki = r(B, S1, HEADS, 128), r(T, 1, 128)
        self.q, self.kv = r(B, S1, G, 576), r(T, 576)               # fused projections: 512 + 64
        cu = [0]
        for n in LENS:
            cu.append(cu[-1] + n)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
        self.cu, self.lens = i32(cu), i32(LENS)
        self.kpos = i32([j for n in LENS for j in range(n)])
        self.qpos = i32([[max(n - S1 + i, 0) for i in range(S1)] for n in LENS])
        self.plain = li.rope_frequencies(64)
        self.yarn = li.rope_frequencies(64, scaling="yarn", factor=4.0)
        f8 = lambda *s: torch.zeros(*s, dtype=torch.float8_e4m3fn, device="cuda")  # noqa: E731
        nb = self.pb.k.shape[0]
        self.ki8, self.kis = f8(nb, BLOCK, 1, 128), torch.ones(nb, BLOCK, device="cuda")
        self.qi8, self.qis = f8(B, S1, HEADS, 128), torch.ones(B, S1, HEADS, device="cuda")
        self.kv8, self.kvs = f8(nb, BLOCK, 1, 512), torch.ones(nb, BLOCK, device="cuda")
        self.kr = torch.zeros(nb, BLOCK, 1, 64, dtype=torch.bfloat16, device="cuda")
        self.prob = self.pb.replace(q=self.qi8, q_descale=self.qis.view(self.pb.q_descale.shape), k=self.ki8,
                                    k_descale=self.kis.view(self.pb.k_descale.shape))
        self.table = self.pb.block_table
        self.scale = 1.0 / math.sqrt(576)

    def step(self, check=True):
        where = dict(cu_seqlens=self.cu, seqused_k=self.lens, block_table=self.table, check=check)
        # the indexer's keys and queries: the first half of each head turns
        self.ki_r = li.rope(self.ki, self.kpos, self.plain)
        li.cache_write(self.ki_r, self.ki8, self.kis, **where)
        self.qi_r = li.rope(self.qi, self.qpos, self.plain)
        li.cache_write(self.qi_r.view(1, -1, 128), self.qi8.view(1, -1, 128), self.qis.view(1, -1), check=check)
        # the attention's: the last 64 of 576
        self.kv_r = li.rope(self.kv.view(-1, 1, 576), self.kpos, self.yarn, offset=512, interleaved=True)
        li.cache_write(self.kv_r[..., :512], self.kv8, self.kvs, rope=self.kv_r[..., 512:], rope_cache=self.kr,
                       pow2=True, **where)
        self.q_r = li.rope(self.q, self.qpos, self.yarn, offset=512, interleaved=True)
        q, qr = self.q_r[..., :512].contiguous(), self.q_r[..., 512:].contiguous()
        self.idx, _ = li.indexer(self.prob, check=check)
        self.out = li.cache_attention(q, self.kv8, self.kvs, self.idx, self.scale, q_rope=qr, rope_cache=self.kr,
                                      block_table=self.table, check=check)
        # the way back through the rotation
        self.dq = li.rope_grad(self.out.new_ones(self.q.shape) * self.q, self.qpos, self.yarn, offset=512,
                               interleaved=True)
        return [self.ki_r, self.qi_r, self.kv_r, self.q_r, self.ki8.view(torch.uint8), self.kis,
                self.kv8.view(torch.uint8), self.kvs, self.kr, self.idx, self.out, self.dq]


def _rotated(y, x, pos, freqs, offset, interleaved, grad=False):
    f = list(freqs.freq)[:freqs.rope_dim // 2]
    want, terms = ref.rotate(x.cpu(), pos.cpu(), f, freqs.magnitude, offset, interleaved, grad)
    tol = terms * 2.0 ** -21 + want.abs() * 2 * ref.HALF_STEP[x.dtype]
    assert ((y.cpu().double() - want).abs() <= tol).all()


def _written(y, codes, scales, pow2, lens, table):
    want, s = ref.quantise(y.cpu().reshape(-1, y.shape[-1]), pow2)
    at = [slot for _, slot in ref.places(lens, table.tolist(), BLOCK, cu=[0] + torch.tensor(lens).cumsum(0).tolist())]
    assert torch.equal(codes.cpu().view(torch.uint8).reshape(-1, y.shape[-1])[at], want)
    assert torch.equal(scales.cpu().reshape(-1)[at], s)
    return at


def test_a_layer(orc):
    m = Layer(1)
    m.step()
    _rotated(m.ki_r, m.ki, m.kpos, m.plain, 0, False)
    _rotated(m.qi_r, m.qi, m.qpos, m.plain, 0, False)
    _rotated(m.kv_r, m.kv.view(-1, 1, 576), m.kpos, m.yarn, 512, True)
    _rotated(m.q_r, m.q, m.qpos, m.yarn, 512, True)
    _rotated(m.dq, m.q, m.qpos, m.yarn, 512, True, grad=True)
    _written(m.ki_r, m.ki8, m.kis, False, LENS, m.table)
    at = _written(m.kv_r[..., :512], m.kv8, m.kvs, True, LENS, m.table)
    assert torch.equal(m.kr.cpu().reshape(-1, 64)[at], m.kv_r.cpu()[:, 0, 512:])
    want, s = ref.quantise(m.qi_r.cpu().reshape(-1, 128))
    assert torch.equal(m.qi8.cpu().view(torch.uint8).view(-1, 128), want) and torch.equal(m.qis.cpu().view(-1), s)
    cpu = m.prob.to("cpu")
    idx, val = li.indexer(m.prob)
    assert torch.equal(idx, m.idx)
    parity.check(orc, cpu, parity.as_rows(idx, cpu.topk), parity.as_rows(val, cpu.topk), label="layer")
    assert (m.idx[2, 0] < 0).all() and (m.idx[2, 1] >= 0).sum() == 1
    p = cache_attn_ref.CacheAttn(m.q_r[..., :512].cpu(), m.kv8.cpu(), m.kvs.cpu(), m.idx.cpu(), m.scale,
                                 m.q_r[..., 512:].cpu(), m.kr.cpu(), m.table.cpu(), m.table.shape[1] * BLOCK)
    cache_attn_ref.check(p, m.out, label="layer")


def test_a_layer_captured_twice_and_replayed():
    """Two layers' graphs, replayed on two streams at once on inputs that changed after the capture."""
    a, b, w = Layer(2), Layer(3), Layer(4)
    w.step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for m in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(m.step(check=False))
        graphs.append(g)
    for m in (a, b):
        for x in (m.qi, m.ki, m.q, m.kv):
            x.normal_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for m, got in ((a, outs[0]), (b, outs[1])):
        got = [t.clone() for t in got]
        for x, y in zip(got, m.step()):
            assert torch.equal(x, y)


def test_the_bounds_checked_build_agrees(monkeypatch):
    release, checked = li.lib(), li.load(build.build_debug())
    a, b = Layer(5), Layer(5)
    first = a.step()
    monkeypatch.setattr(li, "_lib", checked)
    second = b.step()                   # raises on any status bit
    x = torch.empty(sum(LENS), 512, dtype=torch.bfloat16, device="cuda")
    back = [x.clone(), x.clone()]
    for m, lib, y in ((a, release, back[0]), (b, checked, back[1])):
        monkeypatch.setattr(li, "_lib", lib)
        li.cache_read(m.kv8, m.kvs, y, cu_seqlens=m.cu, seqused_k=m.lens, block_table=m.table)
    torch.cuda.synchronize()
    for u, v in zip(first + back[:1], second + back[1:]):
        assert torch.equal(u, v)


def test_offsets_past_32_bits():
    """Rows whose codes, rope parts and strided source lie beyond 2^32 bytes of their buffers."""
    nb, block, dim = 140_000, 64, 512                       # 4.6 GB of codes
    if torch.cuda.mem_get_info()[0] < 20e9:
        pytest.skip("needs 20 GB")
    codes = torch.empty(nb, block, 1, dim, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(nb, block, device="cuda")
    kr = torch.empty(nb, block, 1, 64, dtype=torch.bfloat16, device="cuda")
    n, g = 200, torch.Generator().manual_seed(7)
    assert (nb - 5) * block * dim > 2 ** 32
    table = torch.tensor([[nb - 1, 0, nb - 3, nb - 2]], dtype=torch.int32, device="cuda")
    src = torch.empty(n, 12_000_000, dtype=torch.bfloat16, device="cuda")       # rows 24 MB apart: 4.8 GB
    x, r = src[:, -576:-64], src[:, -64:]
    x.copy_(torch.randn(n, dim, generator=g))
    r.copy_(torch.randn(n, 64, generator=g))
    lens, cu = torch.tensor([n], dtype=torch.int32).cuda(), torch.tensor([0, n], dtype=torch.int32).cuda()
    li.cache_write(x, codes, scales, rope=r, rope_cache=kr, seqused_k=lens, block_table=table, cu_seqlens=cu)
    want, s = ref.quantise(x.cpu())
    at = torch.tensor([slot for _, slot in ref.places([n], table.tolist(), block, cu=[0, n])]).cuda()
    got = codes.view(torch.uint8).view(-1, dim)[at]
    assert torch.equal(got.cpu(), want) and torch.equal(scales.view(-1)[at].cpu(), s)
    assert torch.equal(kr.view(-1, 64)[at], r)
    back, rope = torch.zeros_like(src[:, :512]), torch.zeros_like(src[:, :64])
    li.cache_read(codes, scales, back, rope_cache=kr, rope_out=rope, seqused_k=lens, block_table=table, cu_seqlens=cu)
    assert torch.equal(back.cpu(), (got.view(torch.float8_e4m3fn).cpu().float() * s[:, None]).to(torch.bfloat16))
    assert torch.equal(rope, r)
    q, qr = (torch.randn(1, 2, 16, d, generator=g).to(torch.bfloat16) for d in (512, 64))
    idx = torch.stack([torch.randperm(n, generator=g)[:150] for _ in range(2)]).view(1, 2, 1, 150).int()
    out = li.cache_attention(q.cuda(), codes, scales, idx.cuda(), 0.05, q_rope=qr.cuda(), rope_cache=kr,
                             block_table=table, s2=n)
    small = torch.tensor([[0, 1, 2, 3]], dtype=torch.int32)         # the same keys in a small cache
    pick = lambda t: t[table[0].long()].cpu()  # noqa: E731
    p = cache_attn_ref.CacheAttn(q, pick(codes.view(torch.uint8)).view(torch.float8_e4m3fn), pick(scales), idx, 0.05,
                                 qr, pick(kr), small, n)
    cache_attn_ref.check(p, out, label="far rows")
    freqs = li.rope_frequencies(64)
    pos = torch.arange(n, device="cuda")
    y = li.rope(r.unsqueeze(1), pos, freqs, out=torch.empty_like(src)[:, :64].unsqueeze(1))
    _rotated(y, r.unsqueeze(1), pos, freqs, 0, False)


FIRST_CAPTURE = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import test_cache_chain_gpu as chain
from sparse_attention_token_lightning_b200 import li
m = chain.Layer(6)
freqs, x = m.plain, m.qi.clone()
idx = torch.zeros(3, 2, 1, 9, dtype=torch.int32, device="cuda")
q = m.q[..., :512].contiguous()
g = torch.cuda.CUDAGraph()
def calls():
    li.rope(x, m.qpos, freqs, out=y)
    li.cache_write(m.kv[:, :512], m.kv8, m.kvs, cu_seqlens=m.cu, seqused_k=m.lens, block_table=m.table, check=False)
    return li.cache_attention(q, m.kv8, m.kvs, idx, 0.1, block_table=m.table, check=False)
y = torch.zeros_like(x)
with torch.cuda.graph(g):
    out = calls()
g.replay()
torch.cuda.synchronize()
first = y.clone(), out.clone(), m.kv8.view(torch.uint8).clone()
y.zero_()
again = calls()
torch.cuda.synchronize()
assert torch.equal(first[0], y) and torch.equal(first[1], again) and torch.equal(first[2], m.kv8.view(torch.uint8))
assert first[0].abs().sum() > 0 and first[1].abs().sum() > 0
"""


def test_the_first_calls_of_a_process_are_captured():
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_CAPTURE.format(root=os.path.dirname(tests), tests=tests)
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)
