"""Writing the 8-bit KV cache and reading it back (CUDA, through the C ABI) against the float64 oracle: codes and
scales bit by bit, values to their rounding."""
import numpy as np
import pytest
import torch

import oracle
import structured_causal_attention_b200 as hd
from tests.gpu_util import need_gpu
from tests.q8_util import garbage_cache, on_host, rows, same_cache

pytestmark = pytest.mark.gpu

FMTS = ["e4m3", "int8"]


def _i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def _write(cache, host, k, v, fmt, off=None, length=None):
    """One write on both sides; returns the oracle's cache."""
    hd.kv_write_q8(k.cuda(), v.cuda(), cache, _i32(off), _i32(length))
    torch.cuda.synchronize()
    return {x: oracle.kv_write_q8(t, *host[x], cache.n, cache.block_tokens, fmt, off, length)
            for x, t in (("k", k), ("v", v))}


SHAPES = [
    # B, L, n, Hkv, D, Tcap, bt, offsets, lengths
    (2, 24, 4, 2, 128, 30, 8, None, None),
    (3, 13, 3, 1, 64, 20, 5, [0, 4, 7], [13, 0, 1]),      # ragged, empty, one token; ends inside blocks
    (2, 1, 4, 3, 128, 17, 16, [16, 15], None),             # a decode step: a block's first token, and its last
    (1, 1, 1, 1, 64, 1, 1, None, None),                    # one token in all
    (2, 40, 2, 2, 64, 64, 64, [24, 3], [40, 37]),          # a block larger than the chunk
    (1, 70, 8, 2, 128, 80, 32, [10], None),
    (2, 9, 3, 5, 64, 9, 1, [0, 0], [9, 5]),                # a scale for every token
    (1, 300, 1, 1, 128, 301, 300, [1], None),              # one long block, exactly to the end
    (1, 30, 2, 1, 64, 33, 7, [3], None),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("shape", SHAPES, ids=[str(s) for s in SHAPES])
def test_write_is_the_definitions(shape, fmt):
    """Into memory that held anything, over a first part written before."""
    need_gpu()
    B, L, n, Hkv, D, Tcap, bt, off, length = shape
    cache = garbage_cache(B, Tcap, n, Hkv, D, fmt, bt, seed=L)
    host = on_host(cache)
    if off is not None and max(off) > 0:
        head = max(off)
        k, v = rows((B, head * n, Hkv, D), L + 1, n, 3), rows((B, head * n, Hkv, D), L + 2, n, 3)
        host = _write(cache, host, k, v, fmt, None, off)
        same_cache(cache, host)
    # twice the size: many begun blocks have their scale raised
    k, v = rows((B, L * n, Hkv, D), L + 3, n, 3) * 2, rows((B, L * n, Hkv, D), L + 4, n, 3) * 2
    host = _write(cache, host, k, v, fmt, off, length)
    same_cache(cache, host)
    again = _write(cache, host, k, v, fmt, off, length)  # the same tokens again: nothing changes
    same_cache(cache, host)
    same_cache(cache, again)
    assert hd.hd_device_status() == hd.HD_OK


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("shape", SHAPES, ids=[str(s) for s in SHAPES])
def test_read_is_the_definitions(shape, fmt):
    need_gpu()
    B, L, n, Hkv, D, Tcap, bt, off, length = shape
    cache = garbage_cache(B, Tcap, n, Hkv, D, fmt, bt, seed=L + 9)
    host = _write(cache, on_host(cache), rows((B, Tcap * n, Hkv, D), L, n, 3), rows((B, Tcap * n, Hkv, D), L + 1, n, 3), fmt)
    k, v = hd.kv_read_q8(cache, L, _i32(off), _i32(length))
    for got, x in ((k, "k"), (v, "v")):
        want = oracle.kv_read_q8(*host[x], n, bt, fmt, L, off, length)
        # a code times a scale of 8 significant bits is exact in fp32 and then rounded once
        assert torch.equal(got.cpu(), torch.tensor(want, dtype=torch.float32).to(torch.bfloat16))
    assert hd.hd_device_status() == hd.HD_OK


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_behind_a_sequence_are_zeros(fmt):
    need_gpu()
    B, L, n, Hkv, D, bt = 3, 6, 2, 2, 64, 4
    cache = garbage_cache(B, 10, n, Hkv, D, fmt, bt)
    x = rows((B, 10 * n, Hkv, D), 1, n)
    host = _write(cache, on_host(cache), x, x, fmt)
    out = tuple(torch.full((B, L * n, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    off, length = [0, 2, 4], [6, 0, 3]
    hd.kv_read_q8(cache, L, _i32(off), _i32(length), out=out)
    want = torch.tensor(oracle.kv_read_q8(*host["k"], n, bt, fmt, L, off, length), dtype=torch.float32).to(torch.bfloat16)
    assert (want[1] == 0).all() and torch.equal(out[0].cpu(), want) and torch.equal(out[1].cpu(), want)


@pytest.mark.parametrize("fmt", FMTS)
def test_every_scale_border_and_tie(fmt):
    """Largest magnitudes over all 8-bit significands and exponents at both ends, and values that fall on ties."""
    need_gpu()
    D, n = 64, 1
    tops = [m * 2.0 ** e for m in range(128, 256) for e in (-70, -66, -12, -7, 0, 20, 110)] + [0.0, 2.0 ** -133, 2.0 ** -126]
    k = torch.zeros(1, len(tops), 1, D, dtype=torch.float32)
    steps = torch.arange(D, dtype=torch.float32)
    for i, a in enumerate(tops):
        s = oracle.kv_q8.scale_for(a, fmt)
        k[0, i, 0] = ((steps + 0.5) * s * (1 if fmt == "int8" else 2.0 ** -4)).clamp(max=a)  # ties, where bf16 holds them
        k[0, i, 0, 1::2] *= -1
        k[0, i, 0, 0] = a
    k = k.to(torch.bfloat16)
    assert torch.equal(k[0, :, 0].float().abs().amax(dim=1), torch.tensor(tops, dtype=torch.float32))
    cache = garbage_cache(1, len(tops), n, 1, D, fmt, 1)
    same_cache(cache, _write(cache, on_host(cache), k, -k, fmt))


@pytest.mark.parametrize("fmt", FMTS)
def test_the_largest_values(fmt):
    """Rows up to bf16's largest value, 255 * 2^120: codes and scales are the definition's, and a code whose value
    rounds past it (256 * 2^120 in E4M3, 127 scales in INT8) reads as infinity. A code times its scale has at
    most 15 significant bits, so fp32 holds it and the one rounding is the one to bf16."""
    need_gpu()
    D, n = 64, 1
    tops = [m * 2.0 ** 120 for m in range(128, 256)]
    share = torch.arange(D, 0, -1, dtype=torch.float64) / D
    k = torch.stack([share * a for a in tops]).reshape(1, len(tops), 1, D)
    k[..., 1::2] *= -1
    k = k.to(torch.float32).to(torch.bfloat16)
    assert k.isfinite().all() and k[0, -1, 0, 0] == torch.finfo(torch.bfloat16).max
    cache = garbage_cache(1, len(tops), n, 1, D, fmt, 1)
    host = _write(cache, on_host(cache), k, -k, fmt)
    same_cache(cache, host)
    for got, name in zip(hd.kv_read_q8(cache, len(tops)), "kv"):
        want = torch.tensor(oracle.kv_read_q8(*host[name], n, 1, fmt, len(tops))).to(torch.float32).to(torch.bfloat16)
        assert want.isinf().any() and torch.equal(got.cpu(), want)
    assert hd.hd_device_status() == hd.HD_OK


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_value_that_is_no_number_marks_its_block(fmt, bad):
    """The block's scale of that stream and head is NaN, stays so for later rows, and goes when it starts afresh."""
    need_gpu()
    B, n, Hkv, D, bt, Tcap = 1, 2, 2, 64, 4, 12
    cache = garbage_cache(B, Tcap, n, Hkv, D, fmt, bt)
    k, v = rows((B, 6 * n, Hkv, D), 1, n), rows((B, 6 * n, Hkv, D), 2, n)
    k[0, 5 * n + 1, 1, 3] = bad  # token 5 (block 1), stream 1, head 1
    host = _write(cache, on_host(cache), k, v, fmt)
    same_cache(cache, host)
    assert np.isnan(host["k"][1]).sum() == np.isnan(on_host(garbage_cache(B, Tcap, n, Hkv, D, fmt, bt))["k"][1])[:, :, 2:].sum() + 1
    k1, v1 = rows((B, n, Hkv, D), 3, n), rows((B, n, Hkv, D), 4, n)
    host = _write(cache, host, k1, v1, fmt, [6])
    same_cache(cache, host)
    got = hd.kv_read_q8(cache, 7)[0].isnan()
    want = torch.zeros_like(got)
    want[0, [4 * n + 1, 5 * n + 1, 6 * n + 1], 1] = True
    assert torch.equal(got, want)
    host = _write(cache, host, k1, v1, fmt, [4])  # token 4 begins block 1
    same_cache(cache, host)
    assert not np.isnan(host["k"][1][0, :, 1]).any()
    assert hd.hd_device_status() == hd.HD_OK


@pytest.mark.parametrize("off,length,bad", [
    ([-1, 2], [3, 3], 0), ([0, 8], [3, 3], 1), ([0, 2], [3, -1], 1), ([5, 2], [0, 4], 1), ([2, 10], [2, 1], 1),
    ([0, 2 ** 31 - 1], [3, 3], 1),
])
def test_a_range_outside_is_left_alone(off, length, bad):
    """... on both ways, and the other sequence is served. (Here the rows given are 3 tokens, the cache 10.)"""
    need_gpu()
    B, L, n, Hkv, D, bt = 2, 3, 2, 1, 64, 4
    cache = garbage_cache(B, 10, n, Hkv, D, "int8", bt)
    before = on_host(cache)
    hd.hd_device_status(clear=True)
    k, v = rows((B, L * n, Hkv, D), 1, n), rows((B, L * n, Hkv, D), 2, n)
    good = 1 - bad
    warm = [0, 0]
    warm[good] = off[good]
    first = rows((B, 10 * n, Hkv, D), 3, n), rows((B, 10 * n, Hkv, D), 4, n)
    host = _write(cache, before, *first, "int8", None, warm)
    _write(cache, host, k, v, "int8", off, length)
    assert hd.hd_device_status(clear=True) == hd.HD_ERR_DEVICE_INDEX
    host = {x: oracle.kv_write_q8(t, *host[x], n, bt, "int8", off, length) for x, t in (("k", k), ("v", v))}
    same_cache(cache, host)
    assert np.array_equal(on_host(cache)["k"][0][bad], before["k"][0][bad])
    out = tuple(torch.full((B, L * n, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    hd.kv_read_q8(cache, L, _i32(off), _i32(length), out=out)
    assert hd.hd_device_status(clear=True) == hd.HD_ERR_DEVICE_INDEX
    assert (out[0][bad] == 0).all() and (out[1][bad] == 0).all()
    want = oracle.kv_read_q8(*host["k"], n, bt, "int8", L, off, length)[good, :length[good] * n]
    assert torch.equal(out[0][good, :length[good] * n].cpu(), torch.tensor(want, dtype=torch.float32).to(torch.bfloat16))


def test_helpers_refuse():
    need_gpu()
    cache = hd.kv_cache_q8(2, 8, 2, 1, 64, torch.int8, 4)
    k = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    bad = [
        lambda: hd.kv_write_q8(k.float(), k, cache), lambda: hd.kv_write_q8(k, k[:1], cache),
        lambda: hd.kv_write_q8(k[:, :3].contiguous(), k[:, :3].contiguous(), cache),  # not whole tokens
        lambda: hd.kv_write_q8(k.transpose(0, 1), k.transpose(0, 1), cache), lambda: hd.kv_write_q8(k, k, cache, i.long()),
        lambda: hd.kv_write_q8(k, k, cache, i[:1]), lambda: hd.kv_write_q8(k, k, cache, i, i.cpu()),
        lambda: hd.kv_write_q8(k, k, cache._replace(k=cache.k.view(torch.uint8))),
        lambda: hd.kv_write_q8(k, k, cache._replace(block_tokens=8)), lambda: hd.kv_write_q8(k, k, cache._replace(n=3)),
        lambda: hd.kv_write_q8(k, k, cache._replace(v_scale=cache.v_scale.half())),
        lambda: hd.kv_read_q8(cache, 2, out=(k, k[:, :2].contiguous())), lambda: hd.kv_read_q8(cache, 2, out=(k.float(), k)),
        lambda: hd.decode_attn_q8(k, cache, i.long(), hd.INTRA), lambda: hd.decode_attn_q8(k, cache, i, hd.INTRA),
        lambda: hd.decode_attn_final_q8(k[:, :2].contiguous(), cache, i, hd.INTRA),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()


def test_no_tokens_is_no_work():
    need_gpu()
    cache = garbage_cache(2, 8, 2, 1, 64, "int8", 4)
    before = on_host(cache)
    empty = torch.zeros(2, 0, 1, 64, dtype=torch.bfloat16, device="cuda")
    hd.kv_write_q8(empty, empty, cache)
    same_cache(cache, before)
    assert hd.kv_read_q8(cache, 0)[0].shape == (2, 0, 1, 64)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 codes: its last tokens are written and read where they belong."""
    need_gpu()
    B, n, Hkv, D, bt, Tcap = 2, 8, 16, 128, 16, 150_000  # 4.9e9 codes in each of K and V
    cache = hd.kv_cache_q8(B, Tcap, n, Hkv, D, torch.int8, bt)
    k, v = rows((B, 3 * n, Hkv, D), 1, n), rows((B, 3 * n, Hkv, D), 2, n)
    off = _i32([Tcap - 3, Tcap - 3])
    hd.kv_write_q8(k.cuda(), v.cuda(), cache, off)
    got = hd.kv_read_q8(cache, 3, off)
    last = [Tcap - 3 - (Tcap - 3) // bt * bt] * B  # the same tokens of a short cache, as far into their block
    for x, t in (("k", k), ("v", v)):
        host = np.zeros((B, 2 * bt * n, Hkv, D), np.uint8), np.zeros((B, Hkv, 2, n))
        host = oracle.kv_write_q8(t, *host, n, bt, "int8", last)
        want = oracle.kv_read_q8(*host, n, bt, "int8", 3, last)
        assert torch.equal(got["kv".index(x)].cpu(), torch.tensor(want, dtype=torch.float32).to(torch.bfloat16))
    assert int((cache.k[0] != 0).sum()) == int((cache.k[0, -3 * n:] != 0).sum())  # and nothing else
    assert hd.hd_device_status() == hd.HD_OK
