"""The quantised key cache (li_cache_write, li_cache_read) against a 64-bit form. Codes, scales and
what is read back are exact: the scale is one correctly rounded quotient, a code is the nearest
E4M3 value to the exact quotient (ties to even), a value read back is one rounded product."""
import pytest
import torch

import rope_cache_ref as ref
from sparse_attention_token_lightning_b200 import li, synthetic

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    li.lib()


def _bytes(t):
    return t.view(torch.uint8).cpu()


def _paged(lens, block, g, spare=2):
    nb = [-(-n // block) for n in lens]
    perm = torch.randperm(sum(nb) + spare, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(1, max(nb))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(nb):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, sum(nb) + spare


CASES = {
    # dim, rope, dtype, block (None: dense), S or packed lengths, used, prefix per batch, pow2
    "index_keys": (128, 0, torch.bfloat16, 64, [5, 130, 1, 0, 77], None, [3, 0, 64, 9, 1], False),
    "latent": (512, 64, torch.bfloat16, 64, 40, [40, 1, 0, 17], [0, 100, 5, 63], True),
    "one_token": (512, 64, torch.bfloat16, 64, 1, None, [0, 700, 63], True),
    "odd_block": (384, 8, torch.float16, 17, 33, None, [1, 50], False),
    "block_of_one": (16, 16, torch.float32, 1, [9, 4], None, [0, 3], False),
    "wide_fp32": (1024, 256, torch.float32, 100, 21, [20, 21], [7, 0], True),
    "dense": (256, 0, torch.float16, None, 50, [50, 20], [0, 3], False),
    "dim_48": (48, 24, torch.bfloat16, 5, [11, 2], None, [0, 8], True),
    "block_1024": (128, 64, torch.float16, 1024, 300, None, [900], False),
}


def _problem(name, seed=0):
    dim, rope, dt, block, rows, used, prefix, pow2 = CASES[name]
    g = torch.Generator().manual_seed(seed)
    B = len(prefix)
    packed = isinstance(rows, list)
    n = rows if packed else (used or [rows] * B)
    lens = [a + b for a, b in zip(n, prefix)]
    # TND: three rows behind the last sequence
    shape = (sum(rows) + 3,) if packed else (B, rows)
    x = torch.randn(*shape, dim, generator=g) * torch.exp(2 * torch.randn(*shape, 1, generator=g))
    r = torch.randn(*shape, rope, generator=g).to(dt) if rope else None
    cu = [0]
    for v in n:
        cu.append(cu[-1] + v)
    kw = dict(seqused_k=torch.tensor(lens, dtype=torch.int32))
    if packed:
        kw["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32)
    elif used:
        kw["seqused"] = torch.tensor(used, dtype=torch.int32)
    if block:
        kw["block_table"], nb = _paged(lens, block, g)
        grid = (nb, block)
    else:
        grid = (B, max(lens) + 2)
    at = ref.places(lens, kw["block_table"].tolist() if block else None, block or 1,
                    S=None if packed else rows, cu=cu if packed else None, used=None if packed else n,
                    k_len=grid[1])
    return x.to(dt), r, grid, kw, at, pow2


def _cuda(kw):
    return {k: v.cuda() for k, v in kw.items()}


@pytest.mark.parametrize("name", list(CASES))
def test_write_then_read(name):
    x, r, grid, kw, at, pow2 = _problem(name)
    D = x.shape[-1]
    codes = torch.full((*grid, 1, D), 3.0).to(torch.float8_e4m3fn).cuda()
    descale = torch.full(grid, -7.0).cuda()
    rc = torch.full((*grid, 1, r.shape[-1]), 5.0, dtype=x.dtype).cuda() if r is not None else None
    want_c, want_s = _bytes(codes).view(-1, D).clone(), descale.cpu().view(-1).clone()
    want_r = rc.cpu().view(-1, r.shape[-1]).clone() if r is not None else None
    src = torch.tensor([a for a, _ in at], dtype=torch.int64)
    dst = torch.tensor([b for _, b in at], dtype=torch.int64)
    want_c[dst], want_s[dst] = ref.quantise(x.reshape(-1, D)[src], pow2)
    li.cache_write(x.cuda(), codes, descale, rope=None if r is None else r.cuda(), rope_cache=rc,
                   pow2=pow2, **_cuda(kw))
    assert torch.equal(descale.cpu().view(-1), want_s)
    assert torch.equal(_bytes(codes).view(-1, D), want_c)
    if r is not None:
        want_r[dst] = r.reshape(-1, r.shape[-1])[src]
        assert torch.equal(rc.cpu().view(-1, r.shape[-1]), want_r)
    # back, in every type; rows that take no part keep what they held
    for dt in (torch.bfloat16, torch.float16, torch.float32):
        out = torch.full(x.shape, 9.0, dtype=dt).cuda()
        rout = rc2 = None
        if r is not None:
            rc2 = rc.to(dt)
            rout = torch.full(r.shape, 9.0, dtype=dt).cuda()
        li.cache_read(codes, descale, out, rope_cache=rc2, rope_out=rout, **_cuda(kw))
        want = torch.full(x.shape, 9.0, dtype=dt).view(-1, D)
        want[src] = (want_c[dst].view(torch.float8_e4m3fn).double() * want_s[dst].double()[:, None]).to(dt)
        assert torch.equal(out.cpu().view(-1, D), want)
        if r is not None:
            wr = torch.full(r.shape, 9.0, dtype=dt).view(-1, r.shape[-1])
            wr[src] = rc2.cpu().view(-1, r.shape[-1])[dst]
            assert torch.equal(rout.cpu().view(-1, r.shape[-1]), wr)


def _rows(x, pow2=False, **kw):
    """Quantise rows x (n, D) into a dense cache of one batch: (bytes, scales)."""
    n, D = x.shape
    codes = torch.empty(1, n, D, dtype=torch.float8_e4m3fn, device="cuda")
    descale = torch.empty(1, n, device="cuda")
    li.cache_write(x.cuda().unsqueeze(0), codes, descale, pow2=pow2, **kw)
    return _bytes(codes).view(n, D), descale.cpu().view(n)


@pytest.mark.parametrize("pow2", [False, True])
def test_quotients_at_the_borders(pow2):
    """fp32 rows whose quotients lie on a border between two codes or within a few ulp of it: an
    fp32 quotient would round onto the border for some of them."""
    g = torch.Generator().manual_seed(1)
    mags = ref.MAGS
    mids = ((mags[1:] + mags[:-1]) / 2)
    rows = []
    for _ in range(200):
        s = float((torch.rand(1, generator=g) * 3 + 0.01).float())
        base = torch.empty(256)
        base[0] = 448.0 * s
        m = mids[torch.randint(0, len(mids), (255,), generator=g)].double() * s
        m = m.float()
        k = torch.randint(-2, 3, (255,), generator=g, dtype=torch.int32)
        base[1:] = (m.view(torch.int32) + k).view(torch.float32)
        base[1:] *= torch.sign(torch.rand(255, generator=g) - 0.5)
        rows.append(base)
    x = torch.stack(rows)
    got_c, got_s = _rows(x, pow2)
    want_c, want_s = ref.quantise(x, pow2)
    assert torch.equal(got_s, want_s)
    bad = (got_c != want_c).sum()
    assert bad == 0, f"{int(bad)} codes differ"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("pow2", [False, True])
def test_extreme_rows(dtype, pow2):
    """Rows of zeros (with signs), the largest and smallest values of the type, one element, NaN and
    infinities among finite elements, nothing finite at all."""
    big = torch.finfo(dtype).max
    tiny = torch.finfo(dtype).smallest_normal
    x = torch.zeros(9, 32)
    x[1] = -0.0
    x[2, 5] = big
    x[3] = torch.linspace(-1, 1, 32) * tiny
    x[4, 31] = -1.0
    x[5] = torch.linspace(-3, 3, 32)
    x[5, 7], x[5, 8], x[5, 9] = float("nan"), float("inf"), float("-inf")
    x[6] = float("nan")
    x[7] = float("inf")
    x[8] = torch.linspace(-big / 2, big / 2, 32)
    x = x.to(dtype)
    got_c, got_s = _rows(x, pow2)
    want_c, want_s = ref.quantise(x, pow2)
    assert torch.equal(got_s, want_s)
    nan = (want_c & 127) == 127
    assert torch.equal((got_c & 127) == 127, nan)
    assert torch.equal(got_c[~nan], want_c[~nan])


@pytest.mark.parametrize("dim,dtype", [(16, torch.float32), (48, torch.bfloat16), (496, torch.float16),
                                       (528, torch.bfloat16), (1008, torch.bfloat16), (1024, torch.float32)])
def test_many_rows(dim, dtype):
    """Enough rows that a lane takes more of each (more than eight elements a thread of the device),
    dims that do not divide by the lanes."""
    n = 148 * 2048 * 8 // dim + 77
    g = torch.Generator().manual_seed(dim)
    x = torch.randn(1, n, dim, generator=g).to(dtype)
    x[0, :, -1] *= 9                        # the last element counts in every row's maximum
    codes = torch.zeros(1, n, 1, dim, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.zeros(1, n, device="cuda")
    li.cache_write(x.cuda(), codes, scale)
    want, s = ref.quantise(x[0])
    assert torch.equal(_bytes(codes).view(n, dim), want) and torch.equal(scale.cpu()[0], s)
    back = li.cache_read(codes, scale, torch.zeros(1, n, dim, dtype=dtype, device="cuda"))[0]
    assert torch.equal(back.cpu()[0], (codes.cpu().float().view(n, dim) * s[:, None]).to(dtype))


def test_strided_rows():
    """x and rope as column ranges of one projection, at an aligned and an unaligned start, and rows
    of a longer batch; reading back into such views leaves the other columns alone."""
    g = torch.Generator().manual_seed(2)
    for shift in (0, 1):
        fused = torch.randn(3, 30, 128 + 16 + 8 + shift, generator=g).to(torch.bfloat16).cuda()
        x, r = fused[:, 4:24, shift:128 + shift], fused[:, 4:24, 128 + shift:144 + shift]
        codes = torch.zeros(3, 20, 1, 128, dtype=torch.float8_e4m3fn, device="cuda")
        descale, rc = torch.zeros(3, 20, device="cuda"), torch.zeros(3, 20, 1, 16, dtype=torch.bfloat16, device="cuda")
        li.cache_write(x, codes, descale, rope=r, rope_cache=rc)
        want_c, want_s = ref.quantise(x.reshape(-1, 128).cpu())
        assert torch.equal(_bytes(codes).view(-1, 128), want_c) and torch.equal(descale.cpu().view(-1), want_s)
        assert torch.equal(rc.squeeze(2), r)
        back = torch.full_like(fused, 2.0)
        li.cache_read(codes, descale, back[:, 4:24, shift:128 + shift], rope_cache=rc,
                      rope_out=back[:, 4:24, 128 + shift:144 + shift])
        want = (want_c.view(torch.float8_e4m3fn).double() * want_s.double()[:, None]).to(torch.bfloat16)
        assert torch.equal(back[:, 4:24, shift:128 + shift].cpu().reshape(-1, 128), want)
        assert torch.equal(back[:, 4:24, 128 + shift:144 + shift], r)
        back[:, 4:24, shift:144 + shift] = 2.0
        assert (back == 2.0).all()


def test_bad_lengths_and_table_entries_are_reported():
    """Rows whose position lies outside the sequence or whose block is none are skipped and reported;
    the others are written."""
    x = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def run(seq, table, **kw):
        codes = torch.zeros(6, 4, 1, 64, dtype=torch.float8_e4m3fn, device="cuda")
        descale = torch.zeros(6, 4, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        li.cache_write(x, codes, descale, seqused_k=seq, block_table=table, device_status=st,
                       check=False, **kw)
        torch.cuda.synchronize()
        return int(st), (descale.cpu().view(-1) != 0).nonzero().view(-1).tolist()

    table = i32(0, 1, 2, 3).view(2, 2)
    assert run(i32(4, 8), table) == (0, [0, 1, 2, 3, 12, 13, 14, 15])
    # batch 0 holds fewer keys than rows (positions -2, -1 are none); batch 1 runs past its table
    bits, rows = run(i32(2, 9), table)
    assert bits == li.DEVERR_LENGTHS and rows == [0, 1, 13, 14, 15]
    bits, rows = run(i32(-1, 4), table)
    assert bits == li.DEVERR_LENGTHS and rows == [8, 9, 10, 11]
    bits, rows = run(i32(4, 4), i32(-1, 1, 6, 3).view(2, 2))
    assert bits == li.DEVERR_TABLE and rows == []
    bits, rows = run(i32(4, 4), table, seqused=i32(9, -3))
    assert bits == li.DEVERR_LENGTHS and rows == [0, 1, 2, 3]
    with pytest.raises(li.LiError):
        li.cache_write(x, torch.zeros(6, 4, 1, 64, dtype=torch.float8_e4m3fn, device="cuda"),
                       torch.zeros(6, 4, device="cuda"), seqused_k=i32(2, 9), block_table=table)
    # packed rows with lengths that decrease: reported, nothing outside is touched
    flat = x.view(8, 64)
    codes = torch.zeros(6, 4, 1, 64, dtype=torch.float8_e4m3fn, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    li.cache_write(flat, codes, torch.zeros(6, 4, device="cuda"), seqused_k=i32(4, 4),
                   block_table=table, cu_seqlens=i32(0, 7, 4), device_status=st, check=False)
    torch.cuda.synchronize()


def test_empty_calls():
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    f8 = dict(dtype=torch.float8_e4m3fn)
    li.cache_write(z(0, 5, 64), z(0, 9, 64, **f8), z(0, 9))
    li.cache_write(z(2, 0, 64), z(2, 9, 64, **f8), z(2, 9))
    li.cache_write(z(0, 64), z(1, 4, 64, **f8), z(1, 4), cu_seqlens=z(2, dtype=torch.int32),
                   seqused_k=z(1, dtype=torch.int32), block_table=z(1, 1, dtype=torch.int32))


def test_captured_and_on_another_stream():
    x, r, grid, kw, at, pow2 = _problem("latent", 4)
    kw = _cuda(kw)
    x, r = x.cuda(), r.cuda()
    mk = lambda: (torch.zeros(*grid, 1, 512, dtype=torch.float8_e4m3fn, device="cuda"),  # noqa: E731
                  torch.zeros(grid, device="cuda"),
                  torch.zeros(*grid, 1, 64, dtype=torch.bfloat16, device="cuda"))
    a, b, c = mk(), mk(), mk()
    li.cache_write(x, a[0], a[1], rope=r, rope_cache=a[2], pow2=pow2, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    li.cache_write(x, b[0], b[1], rope=r, rope_cache=b[2], pow2=pow2, stream=side, **kw)
    side.synchronize()
    y = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        li.cache_write(y, c[0], c[1], rope=r, rope_cache=c[2], pow2=pow2, check=False, **kw)
    y.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    for u, v, w in zip(a, b, c):
        assert torch.equal(_bytes(u), _bytes(v)) and torch.equal(_bytes(u), _bytes(w))


def test_the_indexer_reads_what_was_written(orc):
    """Keys written into a paged cache and queries quantised by the same call are the fp8 indexer's
    k / k_descale and q / q_descale: its selection over them is the oracle's."""
    pb = synthetic.paged([300, 129, 64], 2, 8, 40, block_size=16, seed=31)
    dev = synthetic.quantized(pb).to("cuda")
    # the logical keys of each batch, written in two steps: all but the last two, then those
    codes = torch.zeros_like(dev.k)
    descale = torch.ones_like(dev.k_descale)
    lens, bt = pb.seqused_k.tolist(), pb.block_table
    keys = [torch.stack([pb.k[int(bt[b, j // 16]), j % 16, 0] for j in range(n)]) for b, n in enumerate(lens)]
    for part in (0, 1):
        rows = [k[-2:] if part else k[:-2] for k in keys]
        cu = [0]
        for t in rows:
            cu.append(cu[-1] + len(t))
        seq = torch.tensor(lens) - (0 if part else 2)
        li.cache_write(torch.cat(rows).cuda(), codes, descale, seqused_k=seq.int().cuda(),
                       block_table=dev.block_table, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    q = torch.zeros_like(dev.q)
    qs = torch.ones_like(dev.q_descale)
    li.cache_write(pb.q.cuda().view(1, -1, 128), q.view(1, -1, 128), qs.view(1, -1))
    got = dev.replace(q=q, q_descale=qs, k=codes, k_descale=descale)
    want_q, want_s = ref.quantise(pb.q.reshape(-1, 128))
    assert torch.equal(_bytes(q).view(-1, 128), want_q) and torch.equal(qs.cpu().view(-1), want_s)
    idx, val = li.indexer(got)
    import parity
    cpu = got.to("cpu")
    parity.check(orc, cpu, parity.as_rows(idx, cpu.topk), parity.as_rows(val, cpu.topk),
                 label="written cache")
