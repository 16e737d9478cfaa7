"""Rotary positions (li_rope, li_rope_grad) against a 64-bit form.

Tolerance, from the kernel's arithmetic: the angle's remainder (at most half a turn) is rounded
once to fp32 (2^-25 of a half turn, 2^-25 pi radians), sincospif is within 2 ulp (2^-22 of 1 at
most), the magnitude, the two products and their sum add four roundings of 2^-24: in all less than
2^-21 of m (|x_u| + |x_v|); the output's own rounding adds half a step of its type relative to
the value (denormal results of fp16: half of 2^-24).
"""
import pytest
import torch

import rope_cache_ref as ref
from sparse_attention_token_lightning_b200 import li

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    li.lib()


def check(y, x, pos, freq, mag, offset, interleaved, grad=False):
    want, terms = ref.rotate(x.cpu(), pos.cpu(), freq, mag, offset, interleaved, grad)
    tol = terms * 2.0 ** -21 + want.abs() * 2 * ref.HALF_STEP[x.dtype]
    if x.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    off = (y.cpu().double() - want).abs()
    assert (off <= tol).all(), f"off by {(off - tol).max():.3g} over the tolerance"
    same = terms == 0
    assert torch.equal(y.cpu()[same], x.cpu()[same])     # outside the rotated part: bit for bit


CASES = {
    # lead, heads, dim, rope, offset, interleaved
    "index_q": ((1, 300), 64, 128, 64, 0, False),
    "index_k": ((1, 3000), 1, 128, 64, 0, False),
    "attn_q_rope": ((2, 70), 16, 64, 64, 0, True),
    "tail_of_head": ((2, 33), 5, 576, 64, 512, True),
    "tail_half": ((77,), 3, 192, 128, 64, False),
    "one_row": ((1,), 1, 2, 2, 0, True),
    "odd_everything": ((13, 7), 3, 37, 10, 9, False),
    "odd_interleaved": ((41,), 2, 27, 6, 21, True),
    "rope256": ((9,), 2, 264, 256, 8, False),
    "half_of_12": ((50,), 4, 48, 12, 8, False),
    "many_heads": ((3,), 128, 64, 16, 48, True),
}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("name", list(CASES))
def test_rotation_and_gradient(name, dtype):
    lead, heads, dim, n, offset, inter = CASES[name]
    g = torch.Generator().manual_seed(len(name) + heads)
    x = torch.randn(*lead, heads, dim, generator=g).to(dtype)
    pos = torch.randint(-5, 5000, lead, generator=g)
    freqs = li.rope_frequencies(n)
    f, m = ref.frequencies(n)
    for p in (pos, pos.to(torch.int32)):
        y = li.rope(x.cuda(), p.cuda(), freqs, offset=offset, interleaved=inter)
        check(y, x, p, f, m, offset, inter)
    dx = li.rope_grad(x.cuda(), pos.cuda(), freqs, offset=offset, interleaved=inter)
    check(dx, x, pos, f, m, offset, inter, grad=True)


@pytest.mark.parametrize("scaling,factor", [("linear", 8.0), ("yarn", 40.0), ("yarn", 1.0)])
def test_far_positions_and_scaled_frequencies(scaling, factor):
    """Positions up to 2^40 (fp32 angles would be off by whole turns) with scaled frequencies."""
    g = torch.Generator().manual_seed(3)
    pos = torch.cat([torch.randint(0, 1 << 20, (60,), generator=g),
                     torch.randint(1 << 30, 1 << 40, (20,), generator=g), torch.tensor([0, 1, -1])])
    x = torch.randn(len(pos), 4, 64, generator=g)
    freqs = li.rope_frequencies(64, scaling=scaling, factor=factor)
    f, m = ref.frequencies(64, scaling=scaling, factor=factor)
    assert abs(freqs.magnitude - m) <= 2.0 ** -24 * m
    y = li.rope(x.cuda(), pos.cuda(), freqs, interleaved=True)
    # the 64-bit angle itself carries 2^-52 of its size: 2^40 radians are 2^-12 off in both forms
    near = pos.abs() < 1 << 21
    check(y[near.cuda()], x[near], pos[near], f, m, 0, True)
    want, terms = ref.rotate(x, pos, f, m, 0, True)
    assert ((y.cpu().double() - want).abs() <= terms * 2.0 ** -10).all()


def test_strided_rows_heads_and_in_place():
    """Views: the rope part of a fused projection (row stride beyond heads x dim), heads in front of
    rows, and in place; elements outside the views keep their values."""
    g = torch.Generator().manual_seed(4)
    freqs, (f, m) = li.rope_frequencies(64), ref.frequencies(64)
    fused = torch.randn(50, 4 * 64 + 24, generator=g).to(torch.bfloat16).cuda()
    pos = torch.arange(50).cuda()
    view = fused[:, 8:8 + 256].view(50, 4, 64)
    keep = fused.clone()
    y = li.rope(view, pos, freqs)
    check(y, view, pos, f, m, 0, False)
    out = li.rope(view, pos, freqs, out=view)
    assert out is view and torch.equal(view, y)
    assert torch.equal(fused[:, :8], keep[:, :8]) and torch.equal(fused[:, 264:], keep[:, 264:])
    # (heads, rows, dim) storage
    hrd = torch.randn(3, 50, 64, generator=g).to(torch.float16).cuda()
    x = hrd.transpose(0, 1)
    y = li.rope(x, pos, freqs, interleaved=True, out=torch.empty_like(hrd).transpose(0, 1))
    check(y, x, pos, f, m, 0, True)
    # an unaligned start: element by element
    odd = torch.randn(50 * 64 + 1, generator=g).to(torch.bfloat16).cuda()[1:].view(50, 1, 64)
    check(li.rope(odd, pos, freqs), odd, pos, f, m, 0, False)
    # in place on part of the head: the rest is not touched
    z = torch.randn(50, 2, 96, generator=g).cuda()
    was = z.clone()
    li.rope(z, pos, freqs, offset=16, interleaved=True, out=z)
    check(z, was, pos, f, m, 16, True)


def test_gradient_against_differences():
    """The map is linear, so a central difference of sum(dy * rope(x)) along each coordinate is its
    derivative up to fp32 rounding: 2 h terms of size |dy| |y| 2^-21."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(3, 2, 12, generator=g)
    dy = torch.randn(3, 2, 12, generator=g)
    pos = torch.tensor([0, 7, 100000])
    freqs = li.rope_frequencies(8, scaling="yarn", factor=4.0)
    for inter in (False, True):
        f = lambda t: (li.rope(t.cuda(), pos.cuda(), freqs, offset=4, interleaved=inter).cpu().double() * dy.double()).sum()  # noqa: E731,B023
        dx = li.rope_grad(dy.cuda(), pos.cuda(), freqs, offset=4, interleaved=inter).cpu().double()
        h = 0.5
        for i in range(x.numel()):
            e = torch.zeros_like(x).view(-1)
            e[i] = h
            e = e.view_as(x)
            diff = (f(x + e) - f(x - e)) / (2 * h)
            assert abs(float(diff) - float(dx.view(-1)[i])) <= 72 * 4.0 * 2.0 ** -21 / h


def test_gradient_undoes_the_rotation():
    g = torch.Generator().manual_seed(6)
    x = torch.randn(100, 4, 64, generator=g).cuda()
    pos = torch.randint(0, 1 << 20, (100,), generator=g).cuda()
    freqs = li.rope_frequencies(64)
    back = li.rope_grad(li.rope(x, pos, freqs), pos, freqs)
    assert (back - x).abs().max() <= 2.0 ** -19 * x.abs().max()


def test_non_finite_inputs_stay_in_their_pair():
    x = torch.ones(2, 1, 8, device="cuda")
    x[0, 0, 2], x[1, 0, 5] = float("nan"), float("inf")
    y = li.rope(x, torch.tensor([1, 2], device="cuda"), li.rope_frequencies(8), interleaved=True)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[0, 0, 2:4] = True
    want[1, 0, 4:6] = True
    assert torch.equal(bad, want)


def test_empty_and_graph_and_stream():
    freqs, (f, m) = li.rope_frequencies(64), ref.frequencies(64)
    e = li.rope(torch.empty(0, 4, 64, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), freqs)
    assert e.shape == (0, 4, 64)
    x = torch.randn(20, 4, 64, device="cuda")
    pos = torch.arange(20, device="cuda")
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = li.rope(x, pos, freqs, stream=side)
    side.synchronize()
    check(y, x, pos, f, m, 0, False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        li.rope(x, pos, freqs, out=out)
    x.normal_()
    pos += 1000
    graph.replay()
    torch.cuda.synchronize()
    check(out, x, pos, f, m, 0, False)
