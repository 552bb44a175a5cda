"""Decode attention against the 8-bit KV cache where sizes are far apart: queries and keys whose products are ordinary
though neither is, and V blocks of very different scales, against the float64 oracle on the values that the cache holds."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import structured_causal_attention_b200 as hd
from structured_causal_attention_b200 import synthetic as syn
from tests.gpu_util import need_gpu
from tests.q8_util import check_attention, garbage_cache, on_host, rows
from tests.test_gpu_guard_bands import Guarded, _libs, _run, _status_ok

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


SPANS = [  # exponents of the V of the first, middle and last third of the blocks (None: zeros, whose scale is 2^-60)
    (100, None, None), (None, None, 100), (None, 100, None), (None, 90, 100), (100, -50, -50), (-50, -50, 100),
    (20, None, None), (None, None, 20), (118, 118, None), (None, 30, None),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("Hq", HEADS)
@pytest.mark.parametrize("T", [40, 300, 9000], ids=["warp", "whole", "in_parts"])
@pytest.mark.parametrize("span", SPANS, ids=[str(s) for s in SPANS])
def test_values_of_scales_far_apart(span, T, Hq, fmt):
    """Every key counts in the softmax's sum, whatever its V's scale: V blocks of zeros (or near the smallest scale) beside
    V of 2^20 to 2^118, before and behind them, in a warp's tiles, in other warps' and in other CTAs'."""
    need_gpu()
    D = 64
    q = syn.normal_bf16((1, 1, Hq, D), 1)
    q[0, 0, 0] = 0  # equal weights
    part = np.minimum(np.arange(T) // 16 * 3 // max(1, -(-T // 16)), 2)
    size = np.array([0.0 if e is None else 2.0 ** e for e in span])[part]
    v = rows((1, T, 1, D), 3, 1).double() * torch.tensor(size).view(1, T, 1, 1)
    k = rows((1, T, 1, D), 2, 1).double()
    _, lse = _attend(k, v, q, 1, fmt, 16, hd.CROSS_FULL, 0, 0.125, spare=3)
    assert abs(lse[0, 0, 0].item() - np.log(T)) < 2.0 ** -11


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("final", [False, True], ids=["streams", "final"])
@pytest.mark.parametrize("mode", [hd.INTRA, hd.CROSS_FULL, hd.CROSS_WINDOW], ids=["INTRA", "CROSS_FULL", "CROSS_WINDOW"])
@pytest.mark.parametrize("shape", [(3, 4, 200, 8, 2, 128, 150), (5, 3, 3000, 14, 2, 64, 1100), (2, 2, 6000, 6, 3, 128, 5999)],
                         ids=["whole", "in_parts", "long"])
def test_scales_far_apart_in_every_mode(shape, mode, final, fmt):
    """A ragged batch whose V blocks of tokens, streams and heads are zeros, of 2^-40 or of 2^90, one sequence's ordinary."""
    need_gpu()
    B, n, T, Hq, Hkv, D, W = shape
    bt = 16
    rng = np.random.default_rng(T)
    k, v = rows((B, T * n, Hkv, D), 1, n).double(), rows((B, T * n, Hkv, D), 2, n).double()
    size = rng.choice([0.0, 2.0 ** -40, 2.0 ** 90], (B, -(-T // bt), n, Hkv))
    size[1] = 1.0
    v *= torch.tensor(size[:, np.arange(T) // bt]).reshape(B, T * n, Hkv, 1)
    seqlen = torch.tensor(rng.integers(1, T + 1, B), dtype=torch.int32)
    seqlen[0] = T
    cache = garbage_cache(B, T + 1, n, Hkv, D, fmt, bt)
    hd.kv_write_q8(k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), cache, lengths=seqlen.cuda())
    q = syn.normal_bf16((B, 1 if final else n, Hq, D), 3)
    call = hd.decode_attn_final_q8 if final else hd.decode_attn_q8
    out, lse = call(q.cuda(), cache, seqlen.cuda(), mode, W, 0.1)
    again = call(q.cuda(), cache, seqlen.cuda(), mode, W, 0.1)
    torch.cuda.synchronize()
    assert hd.hd_device_status() == hd.HD_OK
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    check_attention(out, lse, q, on_host(cache), n, bt, fmt, seqlen, mode, W, 0.1, final)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("Hq", HEADS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_scales_far_apart_beside_a_block_that_is_no_number(bad, Hq, fmt):
    """The last token's second stream holds a NaN or infinity in a block of its own, which the first stream's query does
    not see: its rows are what the other keys make them, with V blocks of zeros and of 2^100 among these."""
    need_gpu()
    n, bt, D, g = 2, 16, 64, Hq // 2
    T = 3 * bt + 1
    q = syn.normal_bf16((1, n, g, D), 1)
    k, v = rows((1, T * n, 1, D), 2, n).double(), rows((1, T * n, 1, D), 3, n).double()
    v[:, :bt * n] = 0
    v[:, bt * n:2 * bt * n] *= 2.0 ** 100
    clean = _attend(k, v, q, n, fmt, bt, hd.CROSS_FULL, 0, 0.125)
    for x in (k, v):
        held = x[0, -1].clone()
        x[0, -1, 0, 5] = bad
        cache = garbage_cache(1, T, n, 1, D, fmt, bt)
        hd.kv_write_q8(k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), cache)
        out, lse = hd.decode_attn_q8(q.cuda(), cache, torch.tensor([T], dtype=torch.int32, device="cuda"), hd.CROSS_FULL, 0, 0.125)
        x[0, -1] = held
        assert torch.equal(out[:, 0], clean[0][:, 0]) and torch.equal(lse[:, :, 0], clean[1][:, :, 0])
        assert out[:, 1].isnan().all() and lse[:, :, 1].isnan().all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("which", ["libhd", "libhd_checked"])
@pytest.mark.parametrize("T", [20, 3000], ids=["whole", "in_parts"])
def test_scales_far_apart_guarded(T, which, fmt):
    """Between guard bands, with a workspace of exactly the bytes asked for, and in the bounds-checked build."""
    need_gpu()
    lib = _libs()[which]
    B, n, Hq, Hkv, D, bt = 2, 3, 6, 2, 64, 8
    k, v = rows((B, T * n, Hkv, D), 1, n).double(), rows((B, T * n, Hkv, D), 2, n).double()
    v *= torch.tensor(np.random.default_rng(1).choice([0.0, 2.0 ** 90], (B, T * n // 12, 1))).repeat_interleave(12, 1)[..., None]
    c = garbage_cache(B, T, n, Hkv, D, fmt, bt)
    hd.kv_write_q8(k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), c)
    g = Guarded()
    held = [g.like(t.view(torch.uint8)) for t in c[:4]]
    seqlen = torch.tensor([T, T - 7], dtype=torch.int32)
    qh = syn.normal_bf16((B, n, Hq, D), 3)
    q, sl = g.like(qh.cuda()), g.like(seqlen.cuda())
    need = lib.hd_decode_q8_workspace_bytes(B, n, T, Hq, Hkv, D)
    ws, out, lse = g.empty((need,), torch.uint8), g.empty((B, n, Hq, D), torch.bfloat16), g.empty((B, Hq, n), torch.float32)
    _run(lib, "hd_decode_attn_q8", q, *held, sl, out, lse, B, n, T, Hq, Hkv, D, hd.HD_Q8_E4M3 if fmt == "e4m3" else hd.HD_Q8_INT8,
         bt, hd.CROSS_FULL, 0, ctypes.c_float(0.125), ws, need)
    g.check_bands()
    _status_ok(lib)
    check_attention(out, lse, qh, on_host(c), n, bt, fmt, seqlen, hd.CROSS_FULL, 0, 0.125, False)
