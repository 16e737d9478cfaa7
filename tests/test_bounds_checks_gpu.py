"""The bounds checks of the rotation, cache and cache attention kernels, seen to fail.

The bounds-checked build must agree with the release build (test_cache_chain_gpu, test_debug_build_gpu); that
says nothing of a check that is not there. In libli_tighttest.so every buffer counts one element fewer than
it has, so an ordinary call that touches a buffer's last element fails that buffer's check: the access is
left out, and reported where the call has a status word. Every access stays inside its buffer."""
import pytest
import torch

from sparse_attention_token_lightning_b200 import build, li

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tight():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    li.lib()
    return li.load(build.build_tight_test())


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rope,offset", [(64, 64, 0), (64, 32, 0), (64, 32, 32), (66, 32, 33)])
def test_rotation(monkeypatch, tight, interleaved, dim, rope, offset):
    x = torch.randn(7, 3, dim, generator=torch.Generator().manual_seed(dim)).to(torch.bfloat16).cuda()
    pos, freqs = torch.arange(7, device="cuda"), li.rope_frequencies(rope)
    want = li.rope(x, pos, freqs, offset, interleaved)
    monkeypatch.setattr(li, "_lib", tight)
    got = li.rope(x, pos, freqs, offset, interleaved, out=torch.full_like(x, 99))
    left = got == 99
    assert left[-1, -1, -1] and not left[:-1].any() and not left[:, :-1].any() and left.sum() <= 16
    assert torch.equal(got[~left], want[~left])


def cache_calls(lib, monkeypatch, lens, table, used=None):
    """(written cache rows, status of the write, rows read, status of the read) of two batches of four rows over
    blocks of four, five of them."""
    monkeypatch.setattr(li, "_lib", lib)
    x = torch.ones(2, 4, 64, device="cuda")
    r = torch.ones(2, 4, 16, device="cuda")
    codes = torch.zeros(5, 4, 1, 64, dtype=torch.float8_e4m3fn, device="cuda")
    scale, rc, st = torch.zeros(5, 4, device="cuda"), torch.zeros(5, 4, 1, 16, device="cuda"), i32([0, 0])
    kw = dict(seqused_k=i32(lens), block_table=i32(table), check=False, seqused=None if used is None else i32(used))
    li.cache_write(x, codes, scale, rope=r, rope_cache=rc, device_status=st[:1], **kw)
    written = (scale.view(-1) != 0).nonzero().view(-1).tolist()
    assert (rc.view(-1, 16)[:, 0] != 0).nonzero().view(-1).tolist() == written
    out, rout = torch.zeros_like(x), torch.zeros_like(r)
    li.cache_read(torch.ones_like(scale).view(5, 4, 1, 1).expand(5, 4, 1, 64).to(torch.float8_e4m3fn).contiguous(),
                  torch.ones_like(scale), out, rope_cache=torch.ones_like(rc), rope_out=rout, device_status=st[1:], **kw)
    read = (out.view(8, 64)[:, 0] != 0).nonzero().view(-1).tolist()
    assert (rout.view(8, 16)[:, 0] != 0).nonzero().view(-1).tolist() == read
    return written, int(st[0]), read, int(st[1])


@pytest.mark.parametrize("lens,table,used,unwritten,unread", [
    ((4, 4), ((0, 1), (2, 3)), None, {11}, {7}),                # the last row of x and rope
    ((4, 4), ((4, 1), (2, 3)), None, {19, 11}, {3, 7}),         # and the cache's last row
    ((4, 8), ((0, 1), (2, 3)), None, {12, 13, 14, 15}, {4, 5, 6, 7}),   # the table's last entry
    ((4, 3), ((0, 1), (2, 3)), (4, 3), set(), set()),           # none of them used
])
def test_cache(monkeypatch, tight, lens, table, used, unwritten, unread):
    want = cache_calls(li.lib(), monkeypatch, lens, table, used)
    assert want[1] == want[3] == 0 and unwritten <= set(want[0]) and unread <= set(want[2])
    got = cache_calls(tight, monkeypatch, lens, table, used)
    assert set(got[0]) == set(want[0]) - unwritten and set(got[2]) == set(want[2]) - unread
    # the write reads every row of x, in use or not
    assert got[1] == 0x100 and got[3] == (0x100 if unread else 0)       # LI_DEVERR_BOUNDS


@pytest.mark.parametrize("G", [16, 40])
def test_attention(monkeypatch, tight, G):
    g = torch.Generator().manual_seed(G)
    bf = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    q, qr, kr = bf(2, 2, G, 128), bf(2, 2, G, 64), bf(9, 4, 1, 64)
    codes = torch.randn(9, 4, 1, 128, generator=g).to(torch.float8_e4m3fn).cuda()
    scale = torch.ones(9, 4, device="cuda")
    table = i32([[0, 8, 2, 3], [4, 5, 6, 7]])
    idx = i32([[0, 3, 7, 9, 1, 2], [0, 1, 2, 3, 4, 8], [0, 1, 12, 2, 15, 8], [1, 5, 6, 2, 3, 4]]).view(2, 2, 1, 6)

    def run(lib, idx):
        st = i32([0])
        monkeypatch.setattr(li, "_lib", lib)
        out = li.cache_attention(q, codes, scale, idx, 0.1, q_rope=qr, rope_cache=kr, block_table=table, check=False,
                                 return_stats=True, device_status=st)
        return [t.transpose(1, 2).reshape(4, G, -1) if i else t.reshape(4, G, -1) for i, t in enumerate(out)], int(st)
    release = li.lib()
    got, bits = run(tight, idx)
    assert bits == 0x100 | li.DEVERR_TABLE      # a table entry that is not read counts as a block outside
    # row 0 loses position 7 (the cache's last row), row 2 positions 12 and 15 (the table's last entry); the last
    # row's outputs are not stored
    idx[0, 0, 0, 2] = idx[1, 0, 0, 2] = idx[1, 0, 0, 4] = -1
    want, bits = run(release, idx)
    assert bits == 0
    for a, b in zip(got, want):
        assert torch.equal(a[:3], b[:3])
