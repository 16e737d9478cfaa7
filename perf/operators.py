"""Measured cases of the operators around the quantised key cache: rotary positions (forward and
gradient), writing keys into an E4M3 cache, reading them back, and the attention over selected
rows of that cache.

``run`` computes them in plain form (elementary torch operations in 32 bits, 64 where angles or
the borders between two codes ask for it) or, where ``own`` is true, through the calls of
``sparse_attention_token_lightning_b200.li``. ``exact`` gives the same outputs from the
definitions in 64 bits.

Formulas
  rotation   a pair (a, b) of a row at position p with frequency f and magnitude m becomes
             m (a cos pf - b sin pf, a sin pf + b cos pf); the gradient is the transposed map
  write      s = max(amax |x| / 448, 2^-90) per row (1 for a row of zeros), rounded once to fp32,
             or the smallest power of two that is no less; codes = E4M3(x / s); row i of batch b
             goes to position L2_b - L1_b + i of the batch's key sequence
  read       codes * s, rows as above
  attention  x = scale (q . k + q_rope . k_rope), o = sum softmax(x) k over the selected rows,
             k = codes * s
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3_MAX = 448.0
DEV = "cuda"


# ---- cases --------------------------------------------------------------------------------------

def listed():
    return [
        # the indexer's queries of a 4096-token prefill: 64 heads of 128 dims, half of each rotated
        dict(name="rope_index_q_prefill", op="rope", rows=4096, heads=64, dim=128, rope=64,
             offset=0, interleaved=False, dtype="bf16", grad=False, max_pos=4096, far=False,
             factor=1.0),
        # one decode step of 64 sequences: the attention's rope part, far positions, YaRN
        dict(name="rope_decode_yarn", op="rope", rows=64, heads=16, dim=64, rope=64, offset=0,
             interleaved=True, dtype="bf16", grad=False, max_pos=163840, far=True, factor=40.0),
        # training: the gradient through the rope dims of 512 + 64 dim query heads, fp32 gradients
        dict(name="rope_grad_query", op="rope", rows=2999, heads=16, dim=576, rope=64, offset=512,
             interleaved=True, dtype="fp32", grad=True, max_pos=2999, far=False, factor=1.0),
        # a packed prefill of 8 sequences writes its indexer keys (one scale per key)
        dict(name="write_index_keys", op="write", batch=8, total=32768, packed=True, dim=128,
             rope=0, dtype="bf16", block=64, pow2=False, prefix=0),
        # one decode step of 64 sequences writes its latent keys and rope parts
        dict(name="write_latent_decode", op="write", batch=64, total=64, packed=False, dim=512,
             rope=64, dtype="bf16", block=64, pow2=True, prefix=4096),
        # a chunk of a long prefill, rows of a fused projection (512 + 64), block size 48
        dict(name="write_latent_chunk", op="write", batch=2, total=65536, packed=False, dim=512,
             rope=64, dtype="bf16", block=48, pow2=True, prefix=5000),
        # the cached prefix of 4 ragged sequences back to bf16 for a dense prefill
        dict(name="read_latent_prefix", op="read", batch=4, total=65536, packed=False, dim=512,
             rope=64, dtype="bf16", block=64, pow2=True, prefix=0),
        # the last few indexer keys of 32 sequences in fp32, small odd blocks
        dict(name="read_index_tail", op="read", batch=32, total=1120, packed=True, dim=128,
             rope=0, dtype="fp32", block=17, pow2=False, prefix=2000),
        # one decode step of 64 sequences over caches of up to 32768 keys
        dict(name="attn_decode", op="attn", batch=64, s1=1, keys=32768, heads=16, dim=512,
             rope=64, topk=2048, block=64, causal=True),
        # a single token of a single sequence: latency
        dict(name="attn_single_token", op="attn", batch=1, s1=1, keys=16384, heads=16, dim=512,
             rope=64, topk=2048, block=64, causal=True),
        # causal prefill over its own cache, early rows with few keys
        dict(name="attn_prefill", op="attn", batch=1, s1=2048, keys=2048, heads=16, dim=512,
             rope=64, topk=1024, block=64, causal=True),
        # three drafted tokens a sequence, 128 heads, odd selection and block sizes, no rope part
        dict(name="attn_128_heads", op="attn", batch=7, s1=3, keys=5001, heads=128, dim=256,
             rope=0, topk=777, block=48, causal=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attn", "attn"])
    if op == "rope":
        rope = rng.choice([16, 32, 64, 128])
        dim = rope + 8 * rng.choice([0, 0, 1, 8, 16, 64])
        offset = rng.choice([0, dim - rope])
        heads = rng.randint(1, 64)
        rows = _log(rng, 1, max(2, 30_000_000 // (heads * dim)))
        return dict(op="rope", rows=rows, heads=heads, dim=dim, rope=rope, offset=offset,
                    interleaved=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    grad=rng.random() < 0.5, max_pos=_log(rng, 64, 1 << 20),
                    far=rng.random() < 0.5, factor=rng.choice([1.0, 4.0, 40.0]))
    if op in ("write", "read"):
        dim = rng.choice([128, 256, 384, 512])
        batch = _log(rng, 1, 64)
        packed = rng.random() < 0.5
        total = max(batch, _log(rng, batch, 60000))
        if not packed:
            total = total // batch * batch
        return dict(op=op, batch=batch, total=total, packed=packed, dim=dim,
                    rope=rng.choice([0, 64]), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    block=rng.choice([16, 64, 128, rng.randint(1, 200)]),
                    pow2=rng.random() < 0.5, prefix=rng.choice([0, _log(rng, 10, 5000)]))
    heads = rng.choice([rng.randint(1, 16), rng.randint(17, 32), 16, 64, 128])
    topk = _log(rng, 1, 2048)
    pairs = 1_500_000 * 16 // max(16, heads)
    rows = _log(rng, 1, max(1, min(4096, pairs // topk)))
    batch = rng.randint(1, rows) if rows < 64 and rng.random() < 0.7 else 1
    s1 = rows // batch
    # up to three times the selection, but always at least the rows of a causal sequence
    keys = max(s1, min(32768, int(topk * rng.uniform(0.7, 3.0))), 1)
    return dict(op="attn", batch=batch, s1=s1, keys=keys, heads=heads,
                dim=rng.choice([128, 256, 512, 512]), rope=rng.choice([0, 64, 64]), topk=topk,
                block=rng.choice([16, 64, 64, rng.randint(1, 200)]), causal=rng.random() < 0.8)


# ---- inputs -------------------------------------------------------------------------------------

def _lengths(total, batch, g):
    """`batch` lengths >= 1 that sum to `total`."""
    cut = torch.rand(batch, generator=g, device=DEV).add_(0.05).cumsum(0)
    edges = (cut / cut[-1] * (total - batch)).long() + torch.arange(1, batch + 1, device=DEV)
    edges[-1] = total
    return torch.diff(edges, prepend=edges.new_zeros(1))


def _table(lens, block, most, g):
    """A block table over `lens` keys per batch (at most `most` in all) with blocks in random
    order, -1 behind the last one, in a cache with room for `most` keys and a spare block."""
    nb = (lens + block - 1) // block
    width = max(1, int(nb.max()))
    used = torch.arange(width, device=DEV)[None, :] < nb[:, None]
    blocks = most // block + lens.numel() + 1
    perm = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    table = torch.full((lens.numel(), width), -1, dtype=torch.int32, device=DEV)
    table[used] = perm[:int(nb.sum())]
    return table, blocks


def _quantised(shape, dtype, g):
    """Random key rows held as E4M3 codes with a power-of-two scale per row."""
    x = torch.randn(shape, generator=g, device=DEV)
    x *= torch.exp(0.3 * torch.randn(shape[:-1], generator=g, device=DEV)).unsqueeze(-1)
    s = torch.exp2(torch.ceil(torch.log2(x.abs().amax(-1) / E4M3_MAX)))
    return (x / s.unsqueeze(-1)).to(dtype), s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c = case
    if c["op"] == "rope":
        dt = DTYPES[c["dtype"]]
        x = torch.randn(c["rows"], c["heads"], c["dim"], generator=g, device=DEV).to(dt)
        if c["far"]:
            pos = torch.randint(0, c["max_pos"], (c["rows"],), generator=g, device=DEV)
        else:
            pos = torch.arange(c["rows"], device=DEV) % c["max_pos"]
        return dict(case=c, x=x, pos=pos)
    if c["op"] in ("write", "read"):
        B, total, D, R = c["batch"], c["total"], c["dim"], c["rope"]
        dt = DTYPES[c["dtype"]]
        if c["packed"]:
            lens = _lengths(total, B, g)
            cu = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).to(torch.int32)
            used, shape = None, (total,)
        else:
            S = total // B
            lens = torch.randint(S // 2 + 1, S + 1, (B,), generator=g, device=DEV)
            lens[0] = S
            cu, used, shape = None, lens.to(torch.int32), (B, S)
        prefix = torch.randint(0, c["prefix"] + 1, (B,), generator=g, device=DEV)
        seqused = (lens + prefix).to(torch.int32)
        table, nb = _table(seqused.long(), c["block"], total + B * c["prefix"], g)
        st = dict(case=c, cu=cu, used=used, seqused=seqused, table=table)
        if c["op"] == "write":
            # the two parts are column ranges of one projection's rows
            fused = torch.randn(*shape, D + R, generator=g, device=DEV).to(dt)
            st["x"], st["r"] = fused[..., :D], fused[..., D:] if R else None
            st["codes"] = torch.zeros(nb, c["block"], 1, D, dtype=torch.float8_e4m3fn, device=DEV)
            st["descale"] = torch.ones(nb, c["block"], device=DEV)
            st["rcache"] = torch.zeros(nb, c["block"], 1, R, dtype=dt, device=DEV) if R else None
        else:
            st["codes"], st["descale"] = _quantised((nb, c["block"], 1, D), torch.float8_e4m3fn, g)
            st["descale"] = st["descale"].squeeze(-1).contiguous()
            st["rcache"] = (torch.randn(nb, c["block"], 1, R, generator=g, device=DEV).to(dt)
                            if R else None)
            st["out"] = torch.zeros(*shape, D, dtype=dt, device=DEV)
            st["rout"] = torch.zeros(*shape, R, dtype=dt, device=DEV) if R else None
        return st
    B, S1, K, G, D, R = c["batch"], c["s1"], c["keys"], c["heads"], c["dim"], c["rope"]
    lens = torch.randint(max(K // 2, S1), K + 1, (B,), generator=g, device=DEV)
    lens[0] = K
    table, nb = _table(lens, c["block"], B * K, g)
    codes, descale = _quantised((nb, c["block"], 1, D), torch.float8_e4m3fn, g)
    q = (2.0 * torch.randn(B, S1, G, D, generator=g, device=DEV)).to(torch.bfloat16)
    qr = kr = None
    if R:
        qr = (2.0 * torch.randn(B, S1, G, R, generator=g, device=DEV)).to(torch.bfloat16)
        kr = torch.randn(nb, c["block"], 1, R, generator=g, device=DEV).to(torch.bfloat16)
    # the selected keys of each row: distinct positions of its window in random order
    idx = torch.full((B, S1, 1, c["topk"]), -1, dtype=torch.int32, device=DEV)
    kk = min(c["topk"], K)
    j = torch.arange(K, device=DEV)
    for b in range(B):
        last = lens[b] - S1 + torch.arange(S1, device=DEV) if c["causal"] else (lens[b] - 1).expand(S1)
        u = torch.rand(S1, K, generator=g, device=DEV)
        u = torch.where(j[None, :] <= last[:, None], u, u - 2.0)
        val, at = torch.topk(u, kk, dim=-1)
        idx[b, :, 0, :kk] = torch.where(val >= 0, at, torch.full_like(at, -1)).to(torch.int32)
    return dict(case=c, q=q, qr=qr, codes=codes, descale=descale.squeeze(-1).contiguous(), kr=kr,
                idx=idx, table=table, scale=1.0 / math.sqrt(D + R))


# ---- the operators in plain form ----------------------------------------------------------------

def _frequencies(dim, factor, base=10000.0, original=4096, fast=32.0, slow=1.0):
    """Angles per position of the dim / 2 pairs and the magnitude: plain, or YaRN for factor > 1."""
    i = torch.arange(dim // 2, dtype=torch.float64, device=DEV)
    f = base ** (-2.0 * i / dim)
    if factor <= 1.0:
        return f, 1.0
    turn = [dim * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (fast, slow)]
    low, high = max(math.floor(turn[0]), 0), min(math.ceil(turn[1]), dim - 1)
    ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0


def _rope_plain(st):
    c, x = st["case"], st["x"]
    f, m = _frequencies(c["rope"], c["factor"])
    a = st["pos"].double()[:, None] * f[None, :]
    cos, sin = ((m * t).float()[:, None, :] for t in (torch.cos(a), torch.sin(a)))
    if c["grad"]:
        sin = -sin
    y = x.clone()
    part = x[..., c["offset"]:c["offset"] + c["rope"]].float()
    out = torch.empty_like(part)
    h = c["rope"] // 2
    u, v = (slice(0, None, 2), slice(1, None, 2)) if c["interleaved"] else (slice(0, h), slice(h, None))
    out[..., u] = part[..., u] * cos - part[..., v] * sin
    out[..., v] = part[..., u] * sin + part[..., v] * cos
    y[..., c["offset"]:c["offset"] + c["rope"]] = out.to(x.dtype)
    return y


def _slots(st):
    """Cache row of every row of the call, flat, and which rows take part."""
    c, block = st["case"], st["case"]["block"]
    seq = st["seqused"].long()
    if c["packed"]:
        cu = st["cu"].long()
        r = torch.arange(c["total"], device=DEV)
        b = torch.searchsorted(cu[1:], r, right=True)
        pos = seq[b] - (cu[b + 1] - cu[b]) + (r - cu[b])
        ok = torch.ones_like(r, dtype=torch.bool)
    else:
        i = torch.arange(c["total"] // c["batch"], device=DEV)[None, :]
        used = st["used"].long()[:, None]
        pos, ok = (seq[:, None] - used + i).reshape(-1), (i < used).reshape(-1)
        b = torch.arange(c["batch"], device=DEV).repeat_interleave(i.numel())
    at = torch.where(ok, pos, torch.zeros_like(pos))
    return st["table"][b, at // block].long() * block + at % block, ok


def _spare(st):
    """First row of a block that no batch uses."""
    n = st["codes"].shape[0]
    seen = torch.zeros(n + 1, device=DEV)
    t = st["table"].reshape(-1).long()
    seen[torch.where(t < 0, torch.full_like(t, n), t)] = 1
    return torch.argmin(seen[:n]) * st["case"]["block"]


def _write_plain(st):
    c = st["case"]
    D, R = c["dim"], c["rope"]
    slot, ok = _slots(st)
    spare = _spare(st)
    # a row that takes no part writes a spare row's old values back to it
    slot = torch.where(ok, slot, spare)
    x = st["x"].reshape(-1, D).double()
    amax = x.abs().amax(-1)
    s = (amax / E4M3_MAX).clamp_min(2.0 ** -90)
    if c["pow2"]:
        mant, exp = torch.frexp(amax)
        s = torch.ldexp(torch.ones_like(amax), (exp - 9 + (mant > 0.875)).clamp_min(-90))
    s = torch.where(amax > 0, s, torch.ones_like(s)).float()
    q = x / s[:, None].double()
    # to E4M3 by rounding to multiples of its step (ties to even), then an exact conversion
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
    q = torch.round(q / step) * step
    codes, descale = st["codes"].view(-1, D), st["descale"].view(-1)
    byte = lambda t: t.view(torch.uint8)  # noqa: E731
    byte(codes)[slot] = torch.where(ok[:, None], byte(q.float().to(codes.dtype)), byte(codes)[spare][None])
    descale[slot] = torch.where(ok, s, descale[spare])
    out = [st["codes"], st["descale"]]
    if R:
        rc = st["rcache"].view(-1, R)
        rc[slot] = torch.where(ok[:, None], st["r"].reshape(-1, R), rc[spare][None])
        out.append(st["rcache"])
    return out


def _read_plain(st):
    c = st["case"]
    slot, ok = _slots(st)
    slot = torch.where(ok, slot, torch.zeros_like(slot))
    D, R = c["dim"], c["rope"]
    rows = st["codes"].view(-1, D).view(torch.uint8)[slot].view(torch.float8_e4m3fn).float()
    rows = rows * st["descale"].view(-1)[slot][:, None]
    out = st["out"].view(-1, D)
    out.copy_(torch.where(ok[:, None], rows.to(out.dtype), out))
    if not R:
        return [st["out"]]
    rout = st["rout"].view(-1, R)
    rout.copy_(torch.where(ok[:, None], st["rcache"].view(-1, R)[slot], rout))
    return [st["out"], st["rout"]]


def _selected(st):
    """Cache row of every selected key [rows, topk] and which entries select one."""
    c, block = st["case"], st["case"]["block"]
    rows = c["batch"] * c["s1"]
    idx = st["idx"].reshape(rows, -1).long()
    ok = idx >= 0
    at = idx.clamp_min(0)
    b = torch.arange(c["batch"], device=DEV).repeat_interleave(c["s1"])[:, None]
    slot = st["table"][b, at // block].long() * block + at % block
    return torch.where(ok, slot, torch.zeros_like(slot)), ok


def _attn_plain(st):
    c = st["case"]
    G, D, R = c["heads"], c["dim"], c["rope"]
    slot, ok = _selected(st)
    codes, descale = st["codes"].view(-1, D), st["descale"].view(-1)
    if slot.numel() > codes.shape[0]:                        # prefill: the cache once, then rows
        k = (codes.float() * descale[:, None])[slot]
    else:                                                    # decode: the selected rows only
        k = codes.view(torch.uint8)[slot].view(codes.dtype).float() * descale[slot].unsqueeze(-1)
    x = torch.bmm(st["q"].reshape(-1, G, D).float(), k.transpose(1, 2))
    if R:
        kr = st["kr"].view(-1, R)[slot].float()
        x += torch.bmm(st["qr"].reshape(-1, G, R).float(), kr.transpose(1, 2))
    x = (x * st["scale"]).masked_fill(~ok[:, None, :], float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.bmm(p, k) / p.sum(-1, keepdim=True)
    return o.to(torch.bfloat16).view(c["batch"], c["s1"], G, D)


def run(state):
    c, st = state["case"], state
    if own:
        return _own(st)
    return {"rope": _rope_plain, "write": _write_plain, "read": _read_plain,
            "attn": _attn_plain}[c["op"]](st)


def _own(st):
    from sparse_attention_token_lightning_b200 import li
    c = st["case"]
    if c["op"] == "rope":
        freqs = li.rope_frequencies(c["rope"], scaling="yarn" if c["factor"] > 1 else None,
                                    factor=c["factor"])
        call = li.rope_grad if c["grad"] else li.rope
        return call(st["x"], st["pos"], freqs, offset=c["offset"], interleaved=c["interleaved"])
    if c["op"] in ("write", "read"):
        where = dict(seqused_k=st["seqused"], block_table=st["table"], cu_seqlens=st["cu"],
                     seqused=st["used"], check=False)
        if c["op"] == "write":
            li.cache_write(st["x"], st["codes"], st["descale"], rope=st["r"],
                           rope_cache=st["rcache"], pow2=c["pow2"], **where)
            return [t for t in (st["codes"], st["descale"], st["rcache"]) if t is not None]
        li.cache_read(st["codes"], st["descale"], st["out"], rope_cache=st["rcache"],
                      rope_out=st["rout"], **where)
        return [t for t in (st["out"], st["rout"]) if t is not None]
    return li.cache_attention(st["q"], st["codes"], st["descale"], st["idx"], st["scale"],
                              q_rope=st["qr"], rope_cache=st["kr"], block_table=st["table"],
                              s2=c["keys"], check=False)


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    c = case
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if c["op"] == "rope":
        n = c["rows"] * c["heads"] * c["dim"]
        return {"bytes": 2.0 * n * size[c["dtype"]] + 8 * c["rows"],
                "flops": 3.0 * c["rows"] * c["heads"] * c["rope"]}
    if c["op"] in ("write", "read"):
        # ragged dense batches use three quarters of their rows on average
        rows = c["total"] * (1.0 if c["packed"] else 0.75 + 0.25 / c["batch"])
        e = size[c["dtype"]]
        return {"bytes": rows * (c["dim"] * (e + 1) + 4 + 2 * c["rope"] * e), "flops": 2.0 * rows * c["dim"]}
    # keys selected: a row takes min(topk, its window); windows average three quarters of `keys`
    rows = c["batch"] * c["s1"]
    if c["causal"] and c["s1"] > 1 and c["s1"] == c["keys"]:
        n = min(c["topk"], c["keys"])
        pairs = c["batch"] * (n * (n + 1) / 2 + (c["keys"] - n) * n)
    else:
        pairs = float(rows * min(c["topk"], c["keys"]))
    key_bytes = c["dim"] + 4 + 2 * c["rope"]
    distinct = min(pairs, c["batch"] * c["keys"])
    return {"bytes": distinct * key_bytes + 4.0 * rows * c["topk"] +
            rows * c["heads"] * (2 * (c["dim"] + c["rope"]) + 2 * c["dim"]),
            "flops": 2.0 * pairs * c["heads"] * (2 * c["dim"] + c["rope"])}


# ---- the definitions in 64 bits -------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    c = case
    if c["op"] == "rope":
        n = c["rope"]
        f, m = _frequencies(n, c["factor"])
        z = torch.polar(torch.full_like(f, m).expand(c["rows"], -1), st["pos"].double()[:, None] * f)
        if c["grad"]:
            z = z.conj()
        y = st["x"].double()
        part = y[..., c["offset"]:c["offset"] + n].reshape(c["rows"], c["heads"], *((n // 2, 2) if c["interleaved"] else (2, n // 2)))
        if not c["interleaved"]:
            part = part.transpose(-1, -2)
        w = torch.view_as_real(torch.view_as_complex(part.contiguous()) * z[:, None, :])
        if not c["interleaved"]:
            w = w.transpose(-1, -2)
        y[..., c["offset"]:c["offset"] + n] = w.reshape(c["rows"], c["heads"], n)
        return y
    if c["op"] in ("write", "read"):
        D, R, block = c["dim"], c["rope"], c["block"]
        seq, table = st["seqused"].tolist(), st["table"].tolist()
        S = None if c["packed"] else c["total"] // c["batch"]
        cu = st["cu"].tolist() if c["packed"] else [b * S for b in range(c["batch"] + 1)]
        used = [cu[b + 1] - cu[b] for b in range(c["batch"])] if c["packed"] else st["used"].tolist()
        src, dst = [], []
        for b in range(c["batch"]):
            p0 = seq[b] - used[b]
            src += range(cu[b], cu[b] + used[b])
            dst += [table[b][p // block] * block + p % block for p in range(p0, p0 + used[b])]
        src, dst = torch.tensor(src, device=DEV), torch.tensor(dst, device=DEV)
        if c["op"] == "read":
            out = st["out"].double()
            out.view(-1, D)[src] = st["codes"].view(-1, D).view(torch.uint8)[dst].view(torch.float8_e4m3fn).double() * st["descale"].view(-1)[dst].double()[:, None]
            if not R:
                return [out]
            rout = st["rout"].double()
            rout.view(-1, R)[src] = st["rcache"].view(-1, R)[dst].double()
            return [out, rout]
        x = st["x"].reshape(-1, D)[src].double()
        amax = x.abs().amax(1)
        if c["pow2"]:
            s = torch.ones_like(amax)
            grid = torch.exp2(torch.arange(-90, 40, dtype=torch.float64, device=DEV))
            s = grid[torch.searchsorted(grid * E4M3_MAX, amax)]     # the first with 448 s >= amax
        else:
            s = torch.maximum(amax / E4M3_MAX, torch.full_like(amax, 2.0 ** -90)).float().double()
        s[amax == 0] = 1.0
        # nearest of the 127 magnitudes of the format, the even code where two are as near
        mags = torch.arange(127, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double()
        t = (x / s[:, None]).abs()
        hi = torch.searchsorted(mags, t).clamp_max(126)
        lo = (hi - 1).clamp_min(0)
        up, down = mags[hi] - t, t - mags[lo]
        code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
        codes = st["codes"].double()
        codes.view(-1, D)[dst] = torch.sign(x) * mags[code]
        descale = st["descale"].double()
        descale.view(-1)[dst] = s
        if not R:
            return [codes, descale]
        rc = st["rcache"].double()
        rc.view(-1, R)[dst] = st["r"].reshape(-1, R)[src].double()
        return [codes, descale, rc]
    G, D, R, block = c["heads"], c["dim"], c["rope"], c["block"]
    out = torch.zeros(c["batch"] * c["s1"], G, D, dtype=torch.float64, device=DEV)
    logical = torch.arange(c["keys"], device=DEV)
    step = max(1, 200_000_000 // (c["keys"] * G))
    for b in range(c["batch"]):
        # the batch's keys in order, then a count of each row's selections as weights
        page = st["table"][b].long()
        page = page[(logical // block).clamp_max(page.numel() - 1)].clamp_min(0)
        rows = page * block + logical % block
        k = st["codes"].view(-1, D)[rows].double() * st["descale"].view(-1)[rows].double()[:, None]
        kr = st["kr"].view(-1, R)[rows].double() if R else None
        for i in range(0, c["s1"], step):
            sel = st["idx"][b, i:i + step, 0].long()
            n = torch.zeros(sel.shape[0], c["keys"] + 1, dtype=torch.float64, device=DEV)
            n.scatter_add_(1, torch.where(sel < 0, torch.full_like(sel, c["keys"]), sel), torch.ones_like(sel, dtype=torch.float64))
            n = n[:, None, :-1]
            x = st["q"][b, i:i + step].double() @ k.T
            if R:
                x = x + st["qr"][b, i:i + step].double() @ kr.T
            w = n * torch.exp(st["scale"] * x - torch.where(n > 0, st["scale"] * x, -torch.inf).amax(-1, keepdim=True)).where(n > 0, torch.zeros((), dtype=torch.float64, device=DEV))
            r0 = b * c["s1"] + i
            out[r0:r0 + sel.shape[0]] = (w @ k) / w.sum(-1, keepdim=True)
    return out.view(c["batch"], c["s1"], G, D)
