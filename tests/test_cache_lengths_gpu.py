"""li_cache_write and li_cache_read with packed lengths that are wrong: reported, and no block of the cache or
row of the call is touched that the call does not own."""
import pytest
import torch

from sparse_attention_token_lightning_b200 import li

pytestmark = pytest.mark.gpu

D, BLOCK = 64, 4


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    li.lib()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def both(cu, lens, rows):
    """(status of the write, cache rows written, status of the read, rows read) of `rows` rows of sequences that
    end at cu[1:], each with two blocks of its own, and two spare blocks at either end of the cache."""
    B = len(cu) - 1
    table = torch.arange(2, 2 + 2 * B, dtype=torch.int32, device="cuda").view(B, 2)
    grid = (2 * B + 4, BLOCK)
    g = torch.Generator().manual_seed(B)
    x = torch.randn(rows, D, generator=g).to(torch.bfloat16).cuda()
    codes = torch.zeros(*grid, 1, D, dtype=torch.float8_e4m3fn, device="cuda")
    descale, st, st2 = torch.zeros(grid, device="cuda"), i32([0]), i32([0])
    kw = dict(seqused_k=i32(lens), block_table=table, cu_seqlens=i32(cu), check=False)
    li.cache_write(x, codes, descale, device_status=st, **kw)
    written = (descale.view(-1) != 0).nonzero().view(-1).tolist()
    coded = (codes.view(torch.uint8).view(-1, D) != 0).any(-1).nonzero().view(-1).tolist()
    assert set(coded) <= set(written)
    full = torch.ones(*grid, 1, D, device="cuda").to(torch.float8_e4m3fn)
    out = torch.full((rows + 3, D), 7.0, device="cuda")             # the call's rows and three behind them
    li.cache_read(full, torch.full(grid, 2.0, device="cuda"), out[:rows], device_status=st2, **kw)
    assert (out[rows:] == 7).all() and ((out == 7) | (out == 2)).all()
    return int(st), written, int(st2), (out[:rows, 0] == 2).nonzero().view(-1).tolist()


@pytest.mark.parametrize("cu,rows", [((0, 6, 2, 8), 8), ((0, 3, 3, 2, 8), 8), ((-1, 4, 6, 8), 8), ((0, 4, 6, 9), 8),
                                     ((5, 0, 0, 0), 8), ((0, 2, 1), 8), ((0, 2 ** 31 - 1, 8), 8)])
def test_ends_out_of_order_are_reported(cu, rows):
    wst, written, rst, read = both(cu, [8] * (len(cu) - 1), rows)
    assert wst == rst == li.DEVERR_LENGTHS
    own = range(2 * BLOCK, (2 + 2 * (len(cu) - 1)) * BLOCK)
    assert set(written) <= set(own)


@pytest.mark.parametrize("at", [1, 31, 32, 200, 299])
def test_one_end_among_hundreds(at):
    cu = list(range(0, 602, 2))
    assert both(cu, [3] * 300, 600)[::2] == (0, 0)
    cu[at] = cu[at - 1] - 1 if at > 1 else -1
    assert both(cu, [8] * 300, 600)[::2] == (li.DEVERR_LENGTHS, li.DEVERR_LENGTHS)


def test_rows_before_and_behind_the_sequences_are_left():
    wst, written, rst, read = both((2, 4, 4, 7), [2, 0, 4], 9)
    assert (wst, rst) == (0, 0) and read == [2, 3, 4, 5, 6]
    assert written == [8, 9, 25, 26, 27]            # positions 0, 1 of the first and 1 .. 3 of the third


def test_lengths_that_end_before_they_begin():
    """The last end lies before the one ahead of it: rows 0 .. 3 are the last of seven of a sequence with
    four keys, so only row 3 has a position."""
    wst, written, rst, read = both((0, 7, 4), [4, 4], 8)
    assert wst == rst == li.DEVERR_LENGTHS
    assert written == [8] and read == [3]


def test_the_call_raises():
    with pytest.raises(li.LiError):
        li.cache_write(torch.ones(8, D, device="cuda"), torch.zeros(8, 4, 1, D, device="cuda").to(torch.float8_e4m3fn),
                       torch.zeros(8, 4, device="cuda"), seqused_k=i32([8, 8, 8]), cu_seqlens=i32([0, 6, 2, 8]),
                       block_table=torch.arange(6, dtype=torch.int32, device="cuda").view(3, 2))
