"""Decode attention against the 8-bit KV cache (CUDA, through the C ABI) against the float64 oracle on the values that
the cache holds."""
import math

import numpy as np
import pytest
import torch

import oracle
import structured_causal_attention_b200 as hd
from structured_causal_attention_b200 import synthetic as syn
from tests.gpu_util import need_gpu
from tests.q8_util import DTYPES, check_attention, garbage_cache, on_host, rows, same_cache

pytestmark = pytest.mark.gpu

MODES = [hd.INTRA, hd.CROSS_FULL, hd.CROSS_WINDOW]
IDS = ["INTRA", "CROSS_FULL", "CROSS_WINDOW"]
FMTS = ["e4m3", "int8"]


def _filled(B, Tcap, n, Hkv, D, fmt, bt, seqlen, seed, spread=1.0):
    """A cache with seqlen[b] tokens written and arbitrary bytes behind them."""
    cache = garbage_cache(B, Tcap, n, Hkv, D, fmt, bt, seed=seed)
    k, v = (rows((B, Tcap * n, Hkv, D), seed + i, n, spread).cuda() for i in (1, 2))
    hd.kv_write_q8(k, v, cache, lengths=seqlen.cuda())
    return cache


def _attend(q, cache, seqlen, mode, W, scale, final):
    fn = hd.decode_attn_final_q8 if final else hd.decode_attn_q8
    out, lse = fn(q.cuda(), cache, seqlen.cuda(), mode, W, scale)
    torch.cuda.synchronize()
    return out, lse


def _lengths(B, T, seed, ragged):
    s = torch.full((B,), T, dtype=torch.int32)
    if ragged:
        s = torch.randint(1, T + 1, (B,), generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        s[0] = T
        s[-1] = 1
    return s


SHAPES = [
    # B, n, tokens, Tcap, Hq, Hkv, D, W, bt, ragged
    (3, 3, 20, 30, 6, 2, 64, 4, 8, True),
    (2, 4, 700, 701, 16, 4, 128, 37, 16, False),
    (4, 4, 100, 128, 32, 4, 128, 9, 16, True),     # 32 rows a KV head
    (1, 8, 4, 5, 2, 1, 64, 2, 1, False),
    (2, 1, 333, 400, 4, 4, 128, 50, 24, True),      # n = 1: ordinary decode
    (2, 4, 1, 4, 8, 8, 64, 1, 16, False),           # the first token
    (3, 2, 1000, 1100, 4, 1, 128, 300, 64, True),
    (2, 3, 500, 500, 14, 2, 64, 499, 7, True),      # 21 rows, a window of nearly all
    (1, 8, 200, 216, 64, 8, 128, 25, 16, False),    # 64 rows
    (1, 5, 129, 130, 3, 3, 64, 13, 1000, False),    # a block longer than the cache
    (70, 2, 600, 601, 3, 1, 64, 100, 16, True),      # more sequences than a warp has lanes, of all lengths
    (40, 1, 1300, 1300, 9, 3, 128, 1299, 8, True),   # pieces that hold the ends of several sequences
]


@pytest.mark.parametrize("final", [False, True], ids=["streams", "final"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("mode", MODES, ids=IDS)
@pytest.mark.parametrize("shape", SHAPES, ids=[str(s) for s in SHAPES])
def test_decode_is_the_definitions(shape, mode, fmt, final):
    need_gpu()
    B, n, T, Tcap, Hq, Hkv, D, W, bt, ragged = shape
    seqlen = _lengths(B, T, T, ragged)
    cache = _filled(B, Tcap, n, Hkv, D, fmt, bt, seqlen, T + n)
    q = syn.normal_bf16((B, 1 if final else n, Hq, D), T + 5)
    out, lse = _attend(q, cache, seqlen, mode, W, D ** -0.5, final)
    assert hd.hd_device_status() == hd.HD_OK
    check_attention(out, lse, q, on_host(cache), n, cache.block_tokens, fmt, seqlen, mode, W, D ** -0.5, final)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("final", [False, True], ids=["streams", "final"])
def test_blocks_of_very_different_size(fmt, final):
    """V's blocks, streams and heads differ by 2^+-30 and K's by 2^+-4: small blocks count where large ones do not."""
    need_gpu()
    B, n, T, Hq, Hkv, D, bt = 2, 2, 90, 4, 2, 64, 8
    rng = np.random.default_rng(5)
    k, v = (rows((B, T * n, Hkv, D), i, n).double() for i in (6, 7))
    blocks = np.arange(T * n) // n // bt
    k = k * torch.tensor(2.0 ** rng.integers(-4, 2, 12)[blocks])[None, :, None, None]
    v = v * torch.tensor(2.0 ** rng.integers(-30, 30, 12)[blocks])[None, :, None, None]
    v[:, :, 1] *= 2.0 ** -20
    v[:, 1::2] *= 2.0 ** 9
    cache = garbage_cache(B, T + 3, n, Hkv, D, fmt, bt)
    hd.kv_write_q8(k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), cache)
    seqlen = torch.tensor([T, T - 30], dtype=torch.int32)
    q = syn.normal_bf16((B, 1 if final else n, Hq, D), 8)
    for mode in MODES:
        for W in (1, 9):
            out, lse = _attend(q, cache, seqlen, mode, W, 0.125, final)
            check_attention(out, lse, q, on_host(cache), n, cache.block_tokens, fmt, seqlen, mode, W, 0.125, final)


@pytest.mark.parametrize("fmt", FMTS)
def test_queries_of_any_size(fmt):
    """Rows of zeros, of 2^-120 (scores of zero), and of 2^100 with scores kept small by K; one large channel."""
    need_gpu()
    B, n, T, H, D = 1, 4, 70, 1, 64
    seqlen = torch.tensor([T], dtype=torch.int32)
    q = syn.normal_bf16((B, n, H, D), 3)
    q[0, 0] = 0
    q[0, 1] *= 2.0 ** -120
    q[0, 2, 0, 5] = 30.0
    for size in (1.0, 2.0 ** 40):
        cache = garbage_cache(B, T, n, H, D, fmt, 16)
        k = (rows((B, T * n, H, D), 4, n).double() / size).to(torch.bfloat16)
        v = rows((B, T * n, H, D), 5, n)
        hd.kv_write_q8(k.cuda(), v.cuda(), cache)
        qs = (q.double() * size).to(torch.bfloat16)
        out, lse = _attend(qs, cache, seqlen, hd.CROSS_FULL, 0, 0.125, False)
        check_attention(out, lse, qs, on_host(cache), n, cache.block_tokens, fmt, seqlen, hd.CROSS_FULL, 0, 0.125, False)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("final", [False, True], ids=["streams", "final"])
def test_a_heavy_first_key_and_many_light_ones(fmt, final):
    """One key holds weight 1 and 20000 others 2^-14 each: the small weights have to keep their sizes."""
    need_gpu()
    B, n, T, H, D = 1, 1, 20000, 1, 64
    k = torch.zeros(B, T, H, D)
    k[0, 0, 0, 0] = 14 * math.log(2)
    v = torch.zeros(B, T, H, D)
    v[0, 0] = 1
    v[0, 1:] = 3
    cache = garbage_cache(B, T + 1, n, H, D, fmt, 16)
    hd.kv_write_q8(k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), cache, lengths=torch.tensor([T], dtype=torch.int32).cuda())
    q = torch.zeros(B, n, H, D, dtype=torch.bfloat16)
    q[..., 0] = 1
    seqlen = torch.tensor([T], dtype=torch.int32)
    out, lse = _attend(q, cache, seqlen, hd.CROSS_FULL, 0, 1.0, final)
    check_attention(out, lse, q, on_host(cache), n, cache.block_tokens, fmt, seqlen, hd.CROSS_FULL, 0, 1.0, final)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("which", ["k", "v"])
def test_only_what_a_query_sees_reaches_it(fmt, which):
    """A block marked as no number, of stream 2, head 1: under INTRA the other streams' outputs are what they were, under
    CROSS_WINDOW all are once it is out of the window, and where it is seen the output is NaN."""
    need_gpu()
    B, n, T, Hq, Hkv, D, bt = 1, 4, 200, 4, 2, 64, 16
    seqlen = torch.tensor([T], dtype=torch.int32)
    k, v = rows((B, T * n, Hkv, D), 1, n), rows((B, T * n, Hkv, D), 2, n)
    q = syn.normal_bf16((B, n, Hq, D), 3)

    def outs(mode, W, final):
        cache = garbage_cache(B, T, n, Hkv, D, fmt, bt)
        hd.kv_write_q8(k.cuda(), v.cuda(), cache)
        return _attend(q[:, -1:] if final else q, cache, seqlen, mode, W, 0.125, final)

    cases = [(hd.INTRA, 0, False), (hd.INTRA, 0, True), (hd.CROSS_FULL, 0, False), (hd.CROSS_WINDOW, 20, False),
             (hd.CROSS_WINDOW, 20, True), (hd.CROSS_FULL, 0, True)]
    clean = [outs(*c) for c in cases]
    (k if which == "k" else v)[0, 50 * n + 2, 1, 7] = float("nan")  # token 50: block 3, tokens 48 .. 63
    for c, (o0, l0) in zip(cases, clean):
        o1, l1 = outs(*c)
        sees = torch.zeros(o0.shape[:3], dtype=torch.bool, device="cuda")
        if c[0] != hd.CROSS_WINDOW:
            streams = slice(None) if c[0] == hd.CROSS_FULL else (slice(0, 0) if c[2] else slice(2, 3))
            sees[0, streams, 2:] = True
        assert torch.equal(o1[~sees], o0[~sees])
        assert o1[sees].isnan().all()
        lsees = sees.transpose(1, 2)
        assert torch.equal(l1[~lsees], l0[~lsees]) and l1[lsees].isnan().all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("final", [False, True], ids=["streams", "final"])
@pytest.mark.parametrize("T", [12, 1500], ids=["whole", "in_parts"])
def test_bad_seqlen_on_device(T, fmt, final):
    need_gpu()
    B, n, Hq, Hkv, D = 5, 2, 4, 2, 64
    good = torch.tensor([1, T, T, T, T], dtype=torch.int32)
    cache = _filled(B, T, n, Hkv, D, fmt, 4, good, 1)
    q = syn.normal_bf16((B, 1 if final else n, Hq, D), 2)
    hd.hd_device_status(clear=True)
    seqlen = torch.tensor([0, T, T + 1, -5, T], dtype=torch.int32)
    for mode in MODES:
        out, lse = _attend(q, cache, seqlen, mode, 700, 0.125, final)
        assert hd.hd_device_status(clear=True) == hd.HD_ERR_DEVICE_INDEX
        for b in (0, 2, 3):
            assert (out[b] == 0).all() and (lse[b] == -math.inf).all()
        ok = cache._replace(**{x: getattr(cache, x)[[1, 4]] for x in ("k_scale", "v_scale")},
                            **{x: getattr(cache, x).view(torch.uint8)[[1, 4]].view(DTYPES[fmt]) for x in ("k", "v")})
        check_attention(out[[1, 4]], lse[[1, 4]], q[[1, 4]], on_host(ok), n, 4, fmt, seqlen[[1, 4]], mode, 700, 0.125, final)
    none = torch.zeros(B, dtype=torch.int32)
    out, lse = _attend(q, cache, none, hd.CROSS_FULL, 0, 0.125, final)
    assert hd.hd_device_status(clear=True) == hd.HD_ERR_DEVICE_INDEX
    assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_a_generation_from_prompt_to_tokens(fmt):
    """The calls as they are used: a ragged prompt written with its padding, steps appended one token at a time (RoPE at
    the physical positions first), and each step attended to, all streams and the last alone; then the same steps from a
    captured graph."""
    need_gpu()
    B, L, n, Hq, Hkv, D, bt, Tcap, steps = 3, 21, 4, 8, 2, 64, 16, 40, 12
    cache = garbage_cache(B, Tcap, n, Hkv, D, fmt, bt)
    empty = on_host(cache)
    lens = torch.tensor([21, 1, 16], dtype=torch.int32)
    k, v = rows((B, L * n, Hkv, D), 1, n).cuda(), rows((B, L * n, Hkv, D), 2, n).cuda()
    hd.rope_(None, k, n)
    hd.kv_write_q8(k, v, cache, lengths=lens.cuda())
    host = {x: oracle.kv_write_q8(t.cpu(), *empty[x], n, bt, fmt, None, lens.tolist()) for x, t in (("k", k), ("v", v))}
    prompt = tuple(t.clone() for t in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale))
    news = [[rows((B, n, h, D), 10 * i + j, n).cuda() * (1 + i % 3) for j, h in enumerate((Hq, Hkv, Hkv))] for i in range(steps)]

    def step(q, k, v, tokens):  # tokens: int32 [B], cached before; the call advances it
        hd.rope_(q, k, n, token_offset=tokens)
        hd.kv_write_q8(k, v, cache, tokens)
        tokens += 1
        return (hd.decode_attn_q8(q, cache, tokens, hd.CROSS_WINDOW, 9),
                hd.decode_attn_final_q8(q[:, -1:].contiguous(), cache, tokens, hd.INTRA))

    eager, tokens = [], lens.cuda()
    for i in range(steps):
        q, kk, vv = (t.clone() for t in news[i])
        eager.append(step(q, kk, vv, tokens))
        for x, t in (("k", kk), ("v", vv)):
            host[x] = oracle.kv_write_q8(t.cpu(), *host[x], n, bt, fmt, (lens + i).tolist())
        same_cache(cache, host)
        for (out, lse), qq, mode, W, fin in ((eager[-1][0], q, hd.CROSS_WINDOW, 9, False),
                                             (eager[-1][1], q[:, -1:], hd.INTRA, 0, True)):
            check_attention(out, lse, qq.cpu(), host, n, bt, fmt, lens + i + 1, mode, W, D ** -0.5, fin)
    assert hd.hd_device_status() == hd.HD_OK

    for dst, src in zip((cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale), prompt):
        dst.copy_(src)
    q, kk, vv = (torch.empty_like(t) for t in news[0])
    tokens = lens.cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(q, kk, vv, tokens)
    for i in range(steps):
        for dst, src in zip((q, kk, vv), news[i]):
            dst.copy_(src)
        graph.replay()
        for (o, l), (eo, el) in zip(got, eager[i]):
            assert torch.equal(o, eo) and torch.equal(l, el)
    assert tokens.tolist() == (lens + steps).tolist()


def test_two_calls_at_once_and_on_another_stream():
    """Calls with workspaces of their own on two streams at once give what each gives alone, run after run."""
    need_gpu()
    B, n, T, Hq, Hkv, D = 4, 4, 900, 16, 4, 128
    seqlen = _lengths(B, T, 3, True).cuda()
    caches = [_filled(B, T, n, Hkv, D, f, 16, seqlen.cpu(), 4) for f in FMTS]
    q = syn.normal_bf16((B, n, Hq, D), 5).cuda()
    alone = [hd.decode_attn_q8(q, c, seqlen, hd.CROSS_FULL) for c in caches]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in caches]
    for _ in range(10):
        got = []
        for s, c in zip(streams, caches):
            with torch.cuda.stream(s):
                got.append(hd.decode_attn_q8(q, c, seqlen, hd.CROSS_FULL))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("final", [False, True], ids=["streams", "final"])
@pytest.mark.parametrize("mode", MODES, ids=IDS)
def test_decode_workload(mode, fmt, final):
    """B8, n4, 16384 prior tokens (65540 cache rows), 32/8 heads, D128; two sequences vs the oracle, every row."""
    need_gpu()
    w = syn.WORKLOADS["decode"]
    B, n, T, Hq, Hkv, D = w["B"], w["n"], w["T"] + 1, w["Hq"], w["Hkv"], w["D"]
    seqlen = torch.full((B,), T, dtype=torch.int32)
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = hd.kv_cache_q8(B, T, n, Hkv, D, torch.int8 if fmt == "int8" else torch.float8_e4m3fn)
    k, v = (torch.randn(B, T * n, Hkv, D, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    hd.kv_write_q8(k, v, cache)
    q = syn.normal_bf16((B, 1 if final else n, Hq, D), 2)
    out, lse = _attend(q, cache, seqlen, mode, 1024, w["scale"], final)
    assert hd.hd_device_status() == hd.HD_OK
    for b in (0, B - 1):
        at = slice(b, b + 1)
        one = cache._replace(**{x: getattr(cache, x)[at] for x in ("k", "v", "k_scale", "v_scale")})
        check_attention(out[at], lse[at], q[at], on_host(one), n, cache.block_tokens, fmt, seqlen[at], mode, 1024, w["scale"], final)


def test_other_stream_by_argument_and_shared_workspace_in_order():
    """The stream argument, and one workspace for calls that follow one another on a stream."""
    need_gpu()
    B, n, T, Hq, Hkv, D = 2, 4, 1500, 16, 4, 64
    seqlen = _lengths(B, T, 3, False).cuda()
    cache = _filled(B, T, n, Hkv, D, "int8", 16, seqlen.cpu(), 4)
    q = [syn.normal_bf16((B, n, Hq, D), 5 + i).cuda() for i in range(3)]
    alone = [hd.decode_attn_q8(x, cache, seqlen, hd.CROSS_FULL) for x in q]
    ws = torch.empty(hd.hd_decode_q8_workspace_bytes(B, n, T, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [hd.decode_attn_q8(x, cache, seqlen, hd.CROSS_FULL, stream=s, workspace=ws) for x in q]
    s.synchronize()
    for a, b in zip(alone, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("fmt", FMTS)
def test_cache_past_32_bits(fmt):
    """Codes beyond 2^32 elements: the second sequence's keys lie there."""
    need_gpu()
    B, n, Hq, Hkv, D, bt, Tcap = 2, 8, 16, 16, 128, 16, 300_000
    cache = hd.kv_cache_q8(B, Tcap, n, Hkv, D, torch.int8 if fmt == "int8" else torch.float8_e4m3fn, bt)
    T = 40
    k, v = rows((B, T * n, Hkv, D), 1, n), rows((B, T * n, Hkv, D), 2, n)
    hd.kv_write_q8(k.cuda(), v.cuda(), cache)
    seqlen = torch.tensor([T, T], dtype=torch.int32)
    q = syn.normal_bf16((B, n, Hq, D), 3)
    out, lse = _attend(q, cache, seqlen, hd.CROSS_FULL, 0, 0.1, False)
    short = cache._replace(**{x: getattr(cache, x)[:, :T * n].contiguous() for x in ("k", "v")},
                           **{x: getattr(cache, x)[:, :, :-(-T // bt)].contiguous() for x in ("k_scale", "v_scale")})
    check_attention(out, lse, q, on_host(short), n, bt, fmt, seqlen, hd.CROSS_FULL, 0, 0.1, False)
    # and its last keys: the last stream's window of 16 tokens is exactly the last 16 tokens' rows
    seqlen = torch.tensor([T, Tcap], dtype=torch.int32)
    hd.kv_write_q8(k[:, :16 * n].contiguous().cuda(), v[:, :16 * n].contiguous().cuda(), cache,
                   torch.tensor([0, Tcap - 16], dtype=torch.int32, device="cuda"))
    out, lse = _attend(q[:, -1:], cache, seqlen, hd.CROSS_WINDOW, 16, 0.1, True)
    tail = hd.KVCacheQ8(cache.k[1:, -16 * n:], cache.v[1:, -16 * n:], cache.k_scale[1:, :, -1:], cache.v_scale[1:, :, -1:], n, bt)
    check_attention(out[1:], lse[1:], q[1:, -1:], on_host(tail), n, bt, fmt, torch.tensor([16]), hd.CROSS_FULL, 0, 0.1, True)


@pytest.mark.parametrize("as_handle", [False, True], ids=["stream", "handle"])
def test_memory_of_a_call_on_another_stream_is_its_own(as_handle):
    """A call on a stream that is still busy: what the caller allocates and writes meanwhile does not reach it."""
    need_gpu()
    B, n, T, Hq, Hkv, D = 2, 4, 1500, 16, 4, 64
    seqlen = _lengths(B, T, 3, False).cuda()
    cache = _filled(B, T, n, Hkv, D, "int8", 16, seqlen.cpu(), 4)
    q = syn.normal_bf16((B, n, Hq, D), 5).cuda()
    alone = hd.decode_attn_q8(q, cache, seqlen, hd.CROSS_FULL)
    read = hd.kv_read_q8(cache, 100)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    s = side.cuda_stream if as_handle else side
    size = hd.hd_decode_q8_workspace_bytes(B, n, T, Hq, Hkv, D)
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # ~10 ms
    out, lse = hd.decode_attn_q8(q, cache, seqlen, hd.CROSS_FULL, stream=s)
    k, v = hd.kv_read_q8(cache, 100, stream=s)
    others = [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
    side.synchronize()
    assert torch.equal(out, alone[0]) and torch.equal(lse, alone[1])
    assert torch.equal(k, read[0]) and torch.equal(v, read[1])
    assert all(bool((x == 0xFF).all()) for x in others)
    zero = hd.decode_attn_q8(q, cache, seqlen, hd.CROSS_FULL, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(zero[0], alone[0])
