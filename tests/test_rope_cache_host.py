"""The rotary and cache entry points without a GPU: struct mirrors, host-side refusals (every pointer
is fake and never dereferenced), and the frequencies, which are host arithmetic."""
import ctypes
import math
import subprocess
from pathlib import Path

import pytest
import torch

import rope_cache_ref as ref
from sparse_attention_token_lightning_b200 import build as libbuild
from sparse_attention_token_lightning_b200 import li

ROOT = Path(__file__).resolve().parents[1]


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return li.lib()


@pytest.mark.parametrize("cls,cname", [(li.LiRopeArgs, "li_rope_args"),
                                       (li.LiRopeScaling, "li_rope_scaling"),
                                       (li.LiCacheArgs, "li_cache_args")])
def test_mirrors_match_the_header(tmp_path, cls, cname):
    names = [f for f, _ in cls._fields_]
    prog = tmp_path / "p.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "li.h"\nint main(void){\n'
                    f'printf("%zu\\n", sizeof({cname}));\n' +
                    "".join(f'printf("%zu\\n", offsetof({cname}, {n}));\n' for n in names) + "return 0;}\n")
    subprocess.run(["gcc", "-std=c11", "-I", str(ROOT / "include"), str(prog), "-o", str(tmp_path / "p")],
                   check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "p")], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == [ctypes.sizeof(cls)] + [getattr(cls, n).offset for n in names]
    assert f"#define LI_ROPE_MAX_PAIRS {li.ROPE_MAX_PAIRS}" in (ROOT / "include" / "li.h").read_text()


def _rope(**kw):
    # no rows: a valid set is accepted without a launch; refusals come before that
    a = li.LiRopeArgs(0x10000, 0x20000, 0x30000, 0, 512, 128, 512, 128, 4, 128, 64, 0, 0, 0, 64, 1.0)
    for k, v in kw.items():
        if k == "freq0":
            a.freq[0] = v
        else:
            setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(dtype=-1), dict(rope_dim=0), dict(rope_dim=3), dict(rope_dim=258),
    dict(heads=0), dict(heads=1025), dict(head_dim=62), dict(head_dim=4098), dict(rope_offset=-1),
    dict(rope_offset=65), dict(interleaved=2), dict(position_bits=16), dict(rows=-1),
    dict(magnitude=float("nan")), dict(freq0=float("inf")), dict(x_row_stride=-1),
    dict(y_head_stride=(1 << 31) + 1),
    # with rows: missing or misaligned pointers, in place with other strides, rows that overlap
    dict(rows=5, x=None), dict(rows=5, positions=None), dict(rows=5, y=0x20001),
    dict(rows=5, positions=0x30004), dict(rows=5, y=0x10000, y_row_stride=1024),
    dict(rows=5, y_row_stride=511), dict(rows=5, y_head_stride=127), dict(rows=5, y_row_stride=0)])
def test_rope_refusals(L, kw):
    for f in (L.li_rope, L.li_rope_grad):
        assert f(ctypes.byref(_rope(**kw)), None) == 1, kw
        assert li.li_last_error_string()


def test_rope_limits(L):
    assert L.li_rope(None, None) == 1
    assert L.li_rope(ctypes.byref(_rope()), None) == 0
    assert L.li_rope(ctypes.byref(_rope(rows=1 << 31)), None) == 2


def _cache(**kw):
    a = li.LiCacheArgs()
    a.x, a.codes, a.descale = 0x10000, 0x20000, 0x30000
    a.seqused_k, a.block_table, a.block_table_stride = 0x40000, 0x50000, 4
    a.x_batch_stride, a.x_row_stride = 128 * 9, 128
    a.batch, a.x_len, a.num_blocks, a.block_size, a.dim = 2, 9, 8, 16, 128
    a.layout_k = 2
    for k, v in kw.items():
        setattr(a, k, v)
    return a


_DENSE = dict(layout_k=0, block_table=None, block_table_stride=0, num_blocks=0, block_size=0, k_len=20)


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(dtype=-1), dict(pow2=2), dict(dim=0), dict(dim=120), dict(dim=1040),
    dict(rope_dim=12), dict(rope_dim=264), dict(rope_dim=-8), dict(batch=-1), dict(x_len=-1),
    dict(layout_x=2), dict(layout_x=1), dict(cu_seqlens=0x60000), dict(layout_k=1),
    dict(block_size=0), dict(block_size=1025), dict(num_blocks=0), dict(block_table_stride=0),
    dict(block_table=None), dict(seqused_k=None), dict(x=None), dict(codes=None),
    dict(descale=None), dict(rope_dim=64), dict(rope=0x60000, rope_cache=0x70000),
    dict(rope_dim=64, rope=0x60000), dict(rope_dim=64, rope=0x60000, rope_cache=0x70008),
    dict(x=0x10001), dict(codes=0x20008), dict(descale=0x30002), dict(seqused=0x60002),
    dict(device_status=0x60001), dict(reserved=1), dict(x_row_stride=-1),
    dict(x_batch_stride=1 << 41), dict(_DENSE, k_len=-1), dict(_DENSE, num_blocks=3),
    dict(_DENSE, block_table=0x50000)])
def test_cache_refusals(L, kw):
    for f in (L.li_cache_write, L.li_cache_read):
        assert f(ctypes.byref(_cache(**kw)), None) == 1, kw
        assert li.li_last_error_string()


@pytest.mark.parametrize("kw", [dict(x_row_stride=127), dict(x_row_stride=0), dict(x_batch_stride=128 * 8),
                                dict(rope_dim=64, rope=0x60000, rope_cache=0x70000, rope_row_stride=63)])
def test_cache_read_refuses_rows_that_overlap(L, kw):
    assert L.li_cache_read(ctypes.byref(_cache(**kw)), None) == 1, kw


def test_cache_limits(L):
    assert L.li_cache_write(None, None) == 1
    assert L.li_cache_write(ctypes.byref(_cache(batch=0)), None) == 0
    assert L.li_cache_read(ctypes.byref(_cache(x_len=0, x=None)), None) == 0
    big = dict(batch=1 << 16, x_len=1 << 16)
    assert L.li_cache_write(ctypes.byref(_cache(**big)), None) == 2
    assert L.li_cache_write(ctypes.byref(_cache(num_blocks=1 << 25, block_size=128)), None) == 2
    assert L.li_cache_write(ctypes.byref(_cache(**dict(_DENSE, batch=1 << 16, k_len=1 << 16))), None) == 2


@pytest.mark.parametrize("n", [2, 64, 128, 256])
@pytest.mark.parametrize("scaling,factor,original", [(None, 1.0, 4096), ("linear", 8.0, 4096),
                                                     ("yarn", 40.0, 4096), ("yarn", 4.0, 32768),
                                                     ("yarn", 0.5, 1), ("yarn", 1.0, 4096)])
def test_frequencies(L, n, scaling, factor, original):
    got = li.rope_frequencies(n, scaling=scaling, factor=factor, original_max=original)
    f, m = ref.frequencies(n, scaling=scaling, factor=factor, original=original)
    assert all(math.isclose(a, b, rel_tol=1e-14) for a, b in zip(got.freq, f))
    assert got.magnitude == torch.tensor(m).item()


@pytest.mark.parametrize("kw", [
    dict(base=1.0), dict(base=float("nan")), dict(scaling="linear", factor=0.0),
    dict(scaling="yarn", factor=float("inf")), dict(scaling="yarn", beta_slow=0.0),
    dict(scaling="yarn", beta_fast=0.5), dict(scaling="yarn", original_max=0),
    dict(scaling="yarn", magnitude_coef=-1.0), dict(rope_dim=0), dict(rope_dim=258), dict(rope_dim=7)])
def test_frequency_refusals(L, kw):
    kw = dict(kw)
    with pytest.raises(li.LiError):
        li.rope_frequencies(kw.pop("rope_dim", 64), **kw)


def test_binding_refuses_host_tensors_and_wrong_shapes(L):
    freqs = li.rope_frequencies(8)
    with pytest.raises(ValueError):
        li.rope(torch.zeros(3, 2, 8), torch.zeros(3, dtype=torch.int64), freqs)
    with pytest.raises(ValueError):
        li.rope_frequencies(64, scaling="cubic")
    with pytest.raises(ValueError):
        li.RopeFrequencies(64, [1.0] * 31)
    with pytest.raises(ValueError):
        li.cache_write(torch.zeros(1, 3, 64), torch.zeros(1, 3, 64), torch.zeros(1, 3))
    flat = lambda t: li._row_stride(t.shape, t.stride(), t.dim() - 2, "x")  # noqa: E731
    assert flat(torch.zeros(4, 5, 2, 8)) == (20, 16)
    assert flat(torch.zeros(1, 5, 2, 8)[:, ::2]) == (3, 32)
    assert flat(torch.zeros(2, 8)) == (1, 0)
    assert flat(torch.zeros(0, 5, 2, 8))[0] == 0
    with pytest.raises(ValueError):
        flat(torch.zeros(4, 5, 2, 8)[:, :3])


def test_cache_attention_mirror_matches_the_header(tmp_path):
    test_mirrors_match_the_header(tmp_path, li.LiCacheAttnArgs, "li_cache_attn_args")


def _cattn(**kw):
    a = li.LiCacheAttnArgs()
    a.q, a.codes, a.descale, a.sparse_indices = 0x10000, 0x20000, 0x30000, 0x40000
    a.block_table, a.block_table_stride, a.num_blocks, a.block_size = 0x50000, 4, 9, 16
    a.scale, a.batch, a.s1, a.s2, a.G, a.Dm, a.topk, a.layout_k = 0.05, 2, 3, 64, 16, 512, 32, 2
    for k, v in kw.items():
        setattr(a, k, v)
    return a


_DENSE_ATTN = dict(layout_k=0, block_table=None, block_table_stride=0, num_blocks=0, block_size=0)


@pytest.mark.parametrize("kw", [
    dict(G=0), dict(G=129), dict(Dm=64), dict(Dm=200), dict(Dm=640), dict(Dr=32), dict(Dr=64),
    dict(Dr=64, q_rope=0x60000), dict(q_rope=0x60000, k_rope=0x70000), dict(topk=0), dict(topk=8193),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(batch=-1), dict(s1=-1), dict(s2=0), dict(s2=-1), dict(q=None), dict(codes=None),
    dict(descale=None), dict(sparse_indices=None), dict(block_table=None), dict(layout_k=1),
    dict(block_size=0), dict(block_size=1025), dict(num_blocks=0), dict(block_table_stride=3),
    dict(_DENSE_ATTN, block_size=4), dict(_DENSE_ATTN, block_table=0x50000), dict(q=0x10008),
    dict(codes=0x20008), dict(descale=0x30002), dict(sparse_indices=0x40001),
    dict(device_status=0x60002), dict(reserved=1),
    dict(Dr=64, q_rope=0x60008, k_rope=0x70000), dict(Dr=64, q_rope=0x60000, k_rope=0x70008)])
def test_cache_attention_refusals(L, kw):
    assert L.li_cache_attention(ctypes.byref(_cattn(**kw)), 0x200000, None, None, None) == 1, kw
    assert li.li_last_error_string()


def test_cache_attention_outputs_and_limits(L):
    def run(out, m=None, s=None, **kw):
        return L.li_cache_attention(ctypes.byref(_cattn(**kw)), out, m, s, None)
    assert run(None) == 1 and run(0x200008) == 1
    assert run(0x200000, 0x300000) == 1 and run(0x200000, 0x300000, 0x400002) == 1
    assert run(0x200000, batch=1 << 14, s1=1 << 11) == 2
    assert run(0x200000, num_blocks=1 << 25, block_size=128) == 2
    # every head count and size of key fits; no rows need no launch
    for G in (1, 16, 17, 32, 33, 128):
        for Dm in (128, 256, 384, 512):
            for rope in (dict(), dict(Dr=64, q_rope=0x60000, k_rope=0x70000)):
                assert run(None, batch=0, G=G, Dm=Dm, **rope) == 0
