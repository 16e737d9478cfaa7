"""Calls of the rotation, cache and cache attention that their documentation allows, at its edges."""
import pytest
import torch

from sparse_attention_token_lightning_b200 import li

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    li.lib()


def zeros(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


@pytest.mark.parametrize("B,S1,paged", [(0, 3, False), (2, 0, False), (0, 3, True), (2, 0, True)])
def test_attention_without_rows_and_with_a_rope_part(B, S1, paged):
    n = 5 if paged else B
    kw = dict(block_table=zeros(B, 2, dtype=torch.int32)) if paged else {}
    bf = torch.bfloat16
    out = li.cache_attention(zeros(B, S1, 16, 128, dtype=bf), zeros(n, 9, 1, 128, dtype=torch.float8_e4m3fn), zeros(n, 9),
                             zeros(B, S1, 1, 4, dtype=torch.int32), 0.1, q_rope=zeros(B, S1, 16, 64, dtype=bf),
                             rope_cache=zeros(n, 9, 1, 64, dtype=bf), return_stats=True, **kw)
    assert [t.shape for t in out] == [(B, S1, 16, 128), (B, 1, S1, 16), (B, 1, S1, 16)]


def test_read_into_rows_outside_batches():
    """x as a (B, S, D) view of (S, B, D) storage, read and written."""
    g = torch.Generator().manual_seed(1)
    codes = torch.randn(3, 20, 1, 64, generator=g).to(torch.float8_e4m3fn).cuda()
    scale = torch.rand(3, 20, generator=g).cuda() + 0.5
    store = zeros(20, 3, 64)
    out, _ = li.cache_read(codes, scale, store.transpose(0, 1))
    assert torch.equal(out, codes.squeeze(2).float() * scale.unsqueeze(-1))
    again, s2 = torch.zeros_like(codes), torch.zeros_like(scale)
    li.cache_write(store.transpose(0, 1), again, s2)
    want, ws = torch.zeros_like(codes), torch.zeros_like(scale)
    li.cache_write(out.contiguous(), want, ws)
    assert torch.equal(again.view(torch.uint8), want.view(torch.uint8)) and torch.equal(s2, ws)


def test_the_rotated_part_goes_straight_to_q_rope():
    """The rotated part of a fused query into a tensor of its own, as cache_attention() takes it."""
    g = torch.Generator().manual_seed(2)
    q = torch.randn(2, 3, 16, 192, generator=g).to(torch.bfloat16).cuda()
    pos, freqs = torch.arange(6, device="cuda").view(2, 3), li.rope_frequencies(64)
    whole = li.rope(q, pos, freqs, offset=128, interleaved=True)
    part = li.rope(q[..., 128:], pos, freqs, interleaved=True, out=torch.empty_like(q[..., 128:]).contiguous())
    assert part.is_contiguous() and torch.equal(part, whole[..., 128:])


def test_no_call_is_recorded_by_autograd():
    """Outputs have no history, also of inputs that require grad; rope_grad() is the rotation's gradient."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(5, 2, 64, generator=g).cuda().requires_grad_()
    pos, freqs = torch.arange(5, device="cuda"), li.rope_frequencies(64)

    class Rope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return li.rope(x, pos, freqs)

        @staticmethod
        def backward(ctx, dy):
            return li.rope_grad(dy.contiguous(), pos, freqs)
    assert not li.rope(x, pos, freqs).requires_grad
    dy = torch.randn(5, 2, 64, generator=g).cuda()
    Rope.apply(x).backward(dy)
    assert torch.equal(x.grad, li.rope_grad(dy, pos, freqs)) and x.grad.abs().sum() > 0
