"""li_cache_attention where its 8-bit weights and its normaliser could lose keys, against a 64-bit form.

Scores come from the rope part alone (q = 0), so that scales of any size leave them small. With u = 2^-24,
A the largest sum of magnitudes of a row's scores and n its keys, a score is off by ex = 2 u (64 + 8) A and
an exponent by ey = 2^-21 (A + max |log2 scale| + 8); the normaliser by 2 (ex + ey) + (n + 8) 2 u of itself;
a weight by 2^-9 + 2^-11 of itself (two E4M3 parts by way of fp16) or by FLOOR of the row's largest weight
(with its scale), and the output by half a step of bf16, 2^-8 of itself."""
import pytest
import torch

from sparse_attention_token_lightning_b200 import li

pytestmark = pytest.mark.gpu

FLOOR = 2.0 ** -21      # half of the lo part's last step, 2^-14, where the largest weight is at least 2^7


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    li.lib()


def attend(idx, codes, descale, k_rope, q_rope, scale=1.0, **kw):
    """(out, softmax_max, softmax_sum) over a dense cache of one batch: codes (S2, D) as values, idx (S1, topk),
    q_rope (S1, G, 64)."""
    S1, G = q_rope.shape[:2]
    D = codes.shape[1]
    c = lambda t: t.unsqueeze(0).cuda()  # noqa: E731
    out = li.cache_attention(torch.zeros(1, S1, G, D, dtype=torch.bfloat16, device="cuda"),
                             c(codes.to(torch.float8_e4m3fn)).unsqueeze(2), c(descale.float()),
                             c(idx.int()).unsqueeze(2), scale, q_rope=c(q_rope.to(torch.bfloat16)),
                             rope_cache=c(k_rope.to(torch.bfloat16)).unsqueeze(2), return_stats=True, **kw)
    torch.cuda.synchronize()
    return [t.cpu().double() for t in (out[0][0], out[1][0, 0], out[2][0, 0])]


def check(got, idx, codes, descale, k_rope, q_rope, scale=1.0, floor=FLOOR):
    out, smax, ssum = got
    codes, descale = codes.to(torch.float8_e4m3fn).double(), descale.float().double()
    k_rope, q_rope = (t.to(torch.bfloat16).double() for t in (k_rope, q_rope))
    u = 2.0 ** -24
    for r in range(idx.shape[0]):
        at = idx[r][idx[r] >= 0].long()
        n = at.numel()
        k = codes[at] * descale[at][:, None]
        x = scale * q_rope[r] @ k_rope[at].T
        A = (scale * q_rope[r].abs() @ k_rope[at].abs().T).amax(-1)
        m = x.amax(-1)
        w = torch.exp(x - m[:, None])
        l = w.sum(-1)
        ex, ey = 2 * u * 72 * A, 2.0 ** -21 * (A + descale[at].log2().abs().max() + 8)
        err = 2 * (ex + ey) + (n + 8) * 2 * u
        assert ((smax[r] - m).abs() <= ex + ey).all(), f"row {r}: softmax_max"
        assert ((ssum[r] - l).abs() <= err * l).all(), f"row {r}: softmax_sum {ssum[r]} for {l}"
        o = w @ k / l[:, None]
        E = w @ k.abs() / l[:, None]
        top = (w * descale[at]).amax(-1) * 448 / l
        tol = 2.0 ** -8 * o.abs() + (2.0 ** -9 + 2.0 ** -11 + err)[:, None] * E + (n * floor * top)[:, None]
        off = (out[r] - o).abs()
        assert (off <= tol).all(), f"row {r}: out off by {(off / tol).max():.3g} of the tolerance"


def _codes(S2, D, g):
    return torch.randn(S2, D, generator=g).clamp(-3, 3) * 149.0


@pytest.mark.parametrize("G", [16, 40])
@pytest.mark.parametrize("low,high", [(-71, 60), (-100, 100), (100, -100), (-100, 40)])
@pytest.mark.parametrize("topk,at", [(2, (0, 1)), (300, (3, 200)), (300, (200, 3)), (2048, (0, 1500)),
                                     (2048, (1500, 0)), (2048, (100, 101))])
def test_scales_far_apart(G, low, high, topk, at):
    """Keys of equal scores whose scales lie up to 2^200 apart have equal shares: in one tile, in two tiles
    of a CTA in either order (the reference moves) and in two CTAs of a cluster."""
    g = torch.Generator().manual_seed(topk)
    codes, descale = _codes(40, 128, g), torch.ones(40)
    descale[5], descale[6] = 2.0 ** low, 2.0 ** high
    idx = torch.full((2, topk), -1)
    idx[:, at[0]], idx[:, at[1]] = 5, 6
    q_rope, k_rope = torch.randn(2, G, 64, generator=g), torch.zeros(40, 64)
    got = attend(idx, codes, descale, k_rope, q_rope)
    assert (got[1] == 0).all()
    check(got, idx, codes, descale, k_rope, q_rope)


@pytest.mark.parametrize("rows,topk", [(3, 700), (1, 2048), (200, 300)])
def test_scales_of_every_size(rows, topk):
    """Scales over the whole accepted range, 2^-100 to 2^100, with scores of their own."""
    g = torch.Generator().manual_seed(rows)
    S2 = 2100
    codes, descale = _codes(S2, 256, g), torch.exp2(torch.rand(S2, generator=g) * 200 - 100)
    descale[:2] = torch.tensor([2.0 ** -100, 2.0 ** 100])
    idx = torch.stack([torch.randperm(S2, generator=g)[:topk] for _ in range(rows)])
    idx[0, -1], idx[0, 7] = 0, 1
    q_rope, k_rope = 2 * torch.randn(rows, 16, 64, generator=g), torch.randn(S2, 64, generator=g)
    some = slice(None, None, 1 + rows // 8)
    got = attend(idx, codes, descale, k_rope, q_rope, scale=0.125)
    check([t[some] for t in got], idx[some], codes, descale, k_rope, q_rope[some], scale=0.125)


@pytest.mark.parametrize("rows", [1, 100])
@pytest.mark.parametrize("n", [2048, 8192])
@pytest.mark.parametrize("sink", [0, 777, 2047])
def test_a_sink_with_a_long_tail(rows, n, sink):
    """One key takes nearly all of the weight, and thousands of others, each too small to count, have values
    where it has none: what they are worth together arrives, to n FLOOR. The tail's weights are e^-10 ...
    e^-17.5 (2^-14 ... 2^-25) of the sink's, by head; shared by eight CTAs (one row) or not (100)."""
    codes, descale = torch.zeros(n, 128), torch.ones(n)
    codes[:, 64:], k_rope = 448.0, torch.zeros(n, 64)
    k_rope[:, 0] = -1
    codes[sink] = torch.cat([torch.full((64,), 448.0), torch.zeros(64)])
    k_rope[sink] = 0
    q_rope = torch.zeros(rows, 16, 64)
    q_rope[:, :, 0] = 10 + 0.5 * torch.arange(16)
    idx = torch.arange(n).expand(rows, n).contiguous()
    got = attend(idx, codes, descale, k_rope, q_rope)
    check([t[::33] for t in got], idx[::33], codes, descale, k_rope, q_rope[::33])


@pytest.mark.parametrize("rows,topk", [(2, 2048), (170, 1536)])
def test_holes_where_keys_were(rows, topk):
    """Entries that select nothing in the places where a tile four tiles earlier (the lookups' ring) had keys
    that outweigh all others: a mark that arrived late would give them weight. Whole tiles, halves and single
    entries of every tile in turn."""
    g = torch.Generator().manual_seed(topk)
    S2 = 2100
    codes, descale = _codes(S2, 128, g), torch.exp2(torch.randint(-3, 4, (S2,), generator=g).float())
    k_rope, q_rope = torch.randn(S2, 64, generator=g), torch.randn(rows, 16, 64, generator=g)
    idx = torch.stack([torch.randperm(S2, generator=g)[:topk] for _ in range(rows)])
    tile, lane = torch.arange(topk) // 128, torch.arange(topk) % 128
    hole = torch.where(tile % 8 < 4, torch.zeros(topk, dtype=torch.bool),
                       torch.where(tile % 4 == 0, torch.ones(topk, dtype=torch.bool), (lane + tile) % 2 == 0))
    idx[:, hole] = -1
    some = slice(None, None, 1 + rows // 8)
    first = attend(idx, codes, descale, k_rope, q_rope, scale=0.2)
    check([t[some] for t in first], idx[some], codes, descale, k_rope, q_rope[some], scale=0.2)
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(first, attend(idx, codes, descale, k_rope, q_rope, scale=0.2)))


@pytest.mark.parametrize("G,topk,S1", [(16, 300, 3), (40, 300, 3), (16, 2048, 1), (40, 1500, 1)])
@pytest.mark.parametrize("what", ["code", "k_rope", "q nan", "q inf", "q -inf", "q_rope"])
def test_not_a_number_in_all_three_outputs(G, topk, S1, what):
    """A NaN of a key is a NaN of its rows' outputs, maximum and sum, one of a head of q (or an infinity there) of
    that head's; other rows and heads keep their bits. Uncut rows and rows cut between CTAs."""
    g = torch.Generator().manual_seed(G + topk)
    S2, D = topk + 50, 128
    codes = _codes(S2, D, g).to(torch.float8_e4m3fn).view(1, S2, 1, D)
    kr = torch.randn(1, S2, 1, 64, generator=g).to(torch.bfloat16)
    q, qr = (torch.randn(1, S1, G, d, generator=g).to(torch.bfloat16) for d in (D, 64))
    idx = torch.stack([torch.randperm(S2 - 1, generator=g)[:topk] for _ in range(S1)]).view(1, S1, 1, topk).int()
    idx[0, 0, 0, topk // 2] = S2 - 1                # a key that row 0 alone selects

    def run():
        out = li.cache_attention(q.cuda(), codes.cuda(), torch.ones(1, S2, device="cuda"), idx.cuda(), 0.05,
                                 q_rope=qr.cuda(), rope_cache=kr.cuda(), return_stats=True)
        return [t.cpu() for t in (out[0][0], out[1][0, 0], out[2][0, 0])]
    clean = run()
    hit = torch.zeros(S1, G, dtype=torch.bool)
    if what in ("code", "k_rope"):
        hit[0] = True
        if what == "code":
            codes.view(torch.uint8)[0, S2 - 1, 0, 77] = 255
        else:
            kr[0, S2 - 1, 0, 13] = float("nan")
    else:
        hit[S1 - 1, G - 3] = True
        (qr if what == "q_rope" else q)[0, S1 - 1, G - 3, 5] = float(what.split()[-1] if what != "q_rope" else "nan")
    for a, b in zip(clean, run()):
        assert torch.isfinite(a).all()
        assert torch.isnan(b[hit]).all() and torch.equal(a[~hit], b[~hit])
