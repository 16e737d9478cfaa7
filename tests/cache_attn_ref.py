"""Problems and the 64-bit form of the attention over an E4M3 cache, with the error bounds of the
kernel's arithmetic.

With u = 2^-24, D = Dm + Dr, A = max over a row's selected keys of the dot product of magnitudes
(scale included), Q = the head's largest |q|, K = max over the keys of scale sum_d |k_d|:
  scores     fp32 sums of exact products of q's parts and the codes (the tensor cores may truncate:
             2 u per term); Q is scaled to [2^7, 2^8) and the lo part ends in steps of 2^-9 / 16, so
             q is off by 2^-14 there at most, 2^-21 of Q:  ex = 2 u (D + 8) A + 2^-21 Q K
  weights    2^(y - ref) with |y| <= A log2(e) + |log2 descale| rounded a few times:
             ey = 2^-21 (A + max |log2 descale| + 8); rounded to fp16 (2^-11) and held
             to 2^-9 in two E4M3 parts (hi is off by 2^-4 at most, a rest below that by 2^-5 of
             2^-4): 2^-9 + 2^-11; and to 2^-14, half of lo's last step, where the row's largest is
             at least 2^4: 2^-18 of it
  softmax_max   ex + ey;   softmax_sum / l:  2 (ex + ey) + (n + 8) 2 u
  out        half a step of bf16 of the value (2^-8), and over E = sum p |k| / l:
             (2^-9 + 2^-11 + 2 (ex + ey) + (n + 8) 4 u) E + n 2^-18 max(p descale) 448 / l
"""
import math
from dataclasses import dataclass

import torch


@dataclass
class CacheAttn:
    q: torch.Tensor
    codes: torch.Tensor             # paged (NB, bs, 1, Dm) or dense (B, S2, 1, Dm)
    descale: torch.Tensor
    idx: torch.Tensor
    scale: float
    q_rope: torch.Tensor = None
    k_rope: torch.Tensor = None
    table: torch.Tensor = None
    s2: int = 0

    def call(self, fn, **kw):
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        return fn(c(self.q), c(self.codes), c(self.descale), c(self.idx), self.scale, q_rope=c(self.q_rope),
                  rope_cache=c(self.k_rope), block_table=c(self.table),
                  s2=self.s2 if self.table is not None else None, **kw)


def make(B, S1, S2, G, Dm, Dr, topk, block=64, causal=False, seed=0, q_std=2.0, scale=None,
         spread=0.3, pow2=True, table_rows=None):
    """A problem: rows quantised with a scale each (spread: their log's deviation), distinct keys of
    each row's window in random order, -1 behind; block None: a dense cache."""
    g = torch.Generator().manual_seed(seed)
    if block is None:
        grid, table = (B, S2), None
    else:
        nb = -(-S2 // block)
        table = torch.randperm(B * nb + 2, generator=g)[:B * nb].reshape(B, nb).to(torch.int32)
        grid = (B * nb + 2, block)
    x = torch.randn(*grid, 1, Dm, generator=g)
    s = x.abs().amax(-1) / 448.0
    if pow2:
        s = torch.exp2(torch.ceil(torch.log2(s)))
    codes = (x / s.unsqueeze(-1)).to(torch.float8_e4m3fn)
    s = s * torch.exp2(torch.round(spread * torch.randn(s.shape, generator=g) / math.log(2)) if pow2
                       else spread * torch.randn(s.shape, generator=g))
    q = (q_std * torch.randn(B, S1, G, Dm, generator=g)).to(torch.bfloat16)
    qr = (q_std * torch.randn(B, S1, G, Dr, generator=g)).to(torch.bfloat16) if Dr else None
    kr = torch.randn(*grid, 1, Dr, generator=g).to(torch.bfloat16) if Dr else None
    idx = torch.full((B, S1, 1, topk), -1, dtype=torch.int32)
    n = min(topk, S2)
    u = torch.rand(B, S1, S2, generator=g)
    if causal:
        j, i = torch.arange(S2)[None, None], torch.arange(S1)[None, :, None]
        u = torch.where(j <= i + S2 - S1, u, u - 2)
    val, at = torch.topk(u, n, dim=-1)
    idx[:, :, 0, :n] = torch.where(val >= 0, at, torch.full_like(at, -1)).to(torch.int32)
    return CacheAttn(q, codes, s.squeeze(-1).contiguous(), idx, scale or 1.0 / math.sqrt(Dm + Dr), qr, kr,
                     table, S2)


def row_keys(p, b, sel):
    """Cache rows (flat) of the positions sel of batch b that select a key."""
    ok = (sel >= 0) & (sel < p.s2)
    v = sel[ok].long()
    if p.table is None:
        return b * p.codes.shape[1] + v
    bs = p.codes.shape[1]
    blk = p.table[b][v // bs].long()
    good = (blk >= 0) & (blk < p.codes.shape[0])
    return (blk * bs + v % bs)[good]


def check(p, out, smax=None, ssum=None, rows=None, label=""):
    B, S1, G, Dm = p.q.shape
    codes = p.codes.reshape(-1, Dm).double()
    desc = p.descale.reshape(-1).double()
    kr = None if p.k_rope is None else p.k_rope.reshape(-1, p.k_rope.shape[-1]).double()
    out = out.cpu().double().reshape(B * S1, G, Dm)
    smax = None if smax is None else smax.cpu().double().reshape(B * S1, G)
    ssum = None if ssum is None else ssum.cpu().double().reshape(B * S1, G)
    D = Dm + (0 if kr is None else kr.shape[-1])
    for r in (range(B * S1) if rows is None else rows):
        b, i = divmod(r, S1)
        at = row_keys(p, b, p.idx[b, i, 0])
        where = f"{label} row {r}"
        if at.numel() == 0:
            assert (out[r] == 0).all(), where
            if smax is not None:
                assert torch.isneginf(smax[r]).all() and (ssum[r] == 0).all(), where
            continue
        k = codes[at] * desc[at][:, None]
        q = p.q[b, i].double()
        x = p.scale * (q @ k.T)
        A = p.scale * (q.abs() @ k.abs().T)
        if kr is not None:
            x = x + p.scale * (p.q_rope[b, i].double() @ kr[at].T)
            A = A + p.scale * (p.q_rope[b, i].double().abs() @ kr[at].abs().T)
        A = A.amax(-1, keepdim=True)                                     # (G, 1)
        n = at.numel()
        u = 2.0 ** -24
        ex = 2 * u * (D + 8) * A + 2.0 ** -21 * q.abs().amax(-1, keepdim=True) * p.scale * k.abs().sum(-1).max()
        ey = 2.0 ** -21 * (A + desc[at].log2().abs().max() + 8)
        m = x.amax(-1, keepdim=True)
        w = torch.exp(x - m)
        l = w.sum(-1, keepdim=True)
        if smax is not None:
            assert ((smax[r] - m[:, 0]).abs() <= (ex + ey)[:, 0]).all(), \
                f"{where}: softmax_max off by {(smax[r] - m[:, 0]).abs().max():.3g}"
            rel = ((ssum[r] - l[:, 0]).abs() / l[:, 0])
            assert (rel <= (2 * (ex + ey) + (n + 8) * 2 * u)[:, 0]).all(), f"{where}: softmax_sum off by {rel.max():.3g}"
        o = (w @ k) / l
        E = (w @ k.abs()) / l
        tol = o.abs() * 2.0 ** -8 + (2.0 ** -9 + 2.0 ** -11 + 2 * (ex + ey) + (n + 8) * 4 * u) * E + \
            n * 2.0 ** -18 * 448 * (w * desc[at]).amax(-1, keepdim=True) / l
        off = (out[r] - o).abs()
        bad = (off > tol).nonzero()
        assert bad.numel() == 0, (f"{where}: out off by {off.max():.3g} (tolerance there {tol[off == off.max()].max():.3g}) "
                                  f"at head/dim {bad[0].tolist()}, {bad.shape[0]} of {off.numel()}")
