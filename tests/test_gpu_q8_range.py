"""Decode attention against the 8-bit KV cache where sizes are far apart: queries and keys whose products are ordinary
though neither is, and V blocks of very different scales, against the float64 oracle on the values that the cache holds."""
import numpy as np
import pytest
import torch

import oracle
import structured_causal_attention_b200 as hd
from structured_causal_attention_b200 import synthetic as syn
from tests.gpu_util import need_gpu
from tests.q8_util import check_attention, garbage_cache, on_host, rows

pytestmark = pytest.mark.gpu

FMTS = ["e4m3", "int8"]
HEADS = [2, 12, 24, 40]  # of one KV head, n = 1: a row tile of 8, of 16, of 32, and two of 32


def _attend(k, v, q, n, fmt, bt, mode, W, scale, spare=0):
    """The step for the last of the rows' tokens, checked against the oracle."""
    B, S, Hkv, D = k.shape
    T = S // n
    cache = garbage_cache(B, T + spare, n, Hkv, D, fmt, bt)
    hd.kv_write_q8(k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), cache,
                   lengths=torch.full((B,), T, dtype=torch.int32, device="cuda"))
    seqlen = torch.full((B,), T, dtype=torch.int32)
    out, lse = hd.decode_attn_q8(q.cuda(), cache, seqlen.cuda(), mode, W, scale)
    torch.cuda.synchronize()
    assert hd.hd_device_status() == hd.HD_OK
    with np.errstate(over="ignore"):  # (the check forms the weights of hidden keys too)
        check_attention(out, lse, q, on_host(cache), n, bt, fmt, seqlen, mode, W, scale, False)
    return out, lse


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq", HEADS)
def test_large_queries_over_small_keys(Hq, D, fmt):
    """Query rows of +-2^124 over keys at the smallest scale, 2^-60: a query times a code passes fp32, the scores (up to
    2^68) do not. Each row's largest score is 2^64 and more above its others, so its output is that key's V.

    Every product here is exact; what is rounded of a score is scale * log2 e (two roundings of 2^-24 with the
    constant's), times the key's scale, times the dot product, its reference (-13), + log2 l and * ln 2 (with the
    constant's, 2^-25): eight of at most 2^-24 of it, 2^-21."""
    need_gpu()
    T = 300
    rng = np.random.default_rng(Hq)
    sign = np.where(np.arange(Hq) % 2 == 0, 1.0, -1.0)
    q = np.zeros((1, 1, Hq, D))
    q[0, 0, np.arange(Hq), np.arange(Hq)] = 2.0 ** 124 * sign
    code = 8.0 * rng.integers(-12, 13, (T, D))  # exact in both formats
    best = rng.permutation(T)[:Hq]
    code[best, np.arange(Hq)] = 112.0 * sign
    k = torch.tensor(code * 2.0 ** -60).view(1, T, 1, D)
    v = rows((1, T, 1, D), 3, 1)
    cache = garbage_cache(1, T, 1, 1, D, fmt, 16)
    hd.kv_write_q8(k.to(torch.bfloat16).cuda(), v.cuda(), cache)
    assert (cache.k_scale == 2.0 ** -60).all()
    seqlen = torch.tensor([T], dtype=torch.int32, device="cuda")
    out, lse = hd.decode_attn_q8(torch.tensor(q).to(torch.bfloat16).cuda(), cache, seqlen, hd.CROSS_FULL, 0, 0.125)
    want = 2.0 ** 124 * 112 * 2.0 ** -60 * 0.125
    assert (lse[0, :, 0].double() - want).abs().max().item() <= 2.0 ** -21 * want
    held = torch.tensor(oracle.kv_values_q8(*on_host(cache)["v"], 1, 16, fmt)[0, best, 0])
    got = out[0, 0].double().cpu()  # (a weight alone: rounded to fp16 and divided by itself, and the rounding to bf16)
    assert bool(((got - held).abs() <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -20) * held.abs()).all())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq", HEADS)
def test_zero_keys_in_a_block_of_a_large_scale(Hq, D, fmt):
    """Keys of zeros share a block with one of 2^40 that the window leaves out: their scores with queries of 2^118 are
    zero, though the query's size times the block's scale passes fp32."""
    need_gpu()
    T = 150
    q = (syn.normal_bf16((1, 1, Hq, D), 1).double() * 2.0 ** 118).to(torch.bfloat16)
    k = torch.zeros(1, T, 1, D, dtype=torch.float64)
    k[0, 3] = 2.0 ** 40
    _, lse = _attend(k, rows((1, T, 1, D), 3, 1), q, 1, fmt, 16, hd.CROSS_WINDOW, T - 4, 0.125)
    assert (lse.cpu().double() - np.log(T - 4)).abs().max() < 2.0 ** -11
