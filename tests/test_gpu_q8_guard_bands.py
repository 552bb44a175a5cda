"""The 8-bit cache's entry points write only what is theirs: guard bands around every buffer, inputs unchanged, through
libhd.so and through the bounds-checked libhd_checked.so (whose status word must stay clear)."""
import ctypes
import math

import pytest
import torch

import oracle
import structured_causal_attention_b200 as hd
from structured_causal_attention_b200 import synthetic as syn
from tests.q8_util import check_attention, garbage_cache, on_host, rows, same_cache
from tests.test_gpu_guard_bands import Guarded, _libs, _run, _status_ok

pytestmark = pytest.mark.gpu

FMTS = ["e4m3", "int8"]


@pytest.fixture(scope="module")
def libs():
    return _libs()


def _guarded_cache(g, B, Tcap, n, Hkv, D, fmt, bt):
    c = garbage_cache(B, Tcap, n, Hkv, D, fmt, bt, seed=Tcap)
    like = {x: g.empty(tuple(t.shape), t.dtype) for x, t in zip(("k", "v", "k_scale", "v_scale"), c[:4])}
    for x, t in zip(("k", "v", "k_scale", "v_scale"), c[:4]):
        like[x].view(torch.uint8).copy_(t.view(torch.uint8))
    return hd.KVCacheQ8(like["k"], like["v"], like["k_scale"], like["v_scale"], n, bt)


SHAPES = [  # B, L, n, Hkv, D, Tcap, bt, offsets, lengths
    (2, 9, 3, 2, 64, 17, 5, [8, 3], [9, 4]),      # exactly to the end of the cache
    (3, 1, 4, 3, 128, 20, 16, [19, 0, 15], None),
    (1, 100, 1, 1, 128, 101, 64, [1], None),
    (2, 40, 8, 1, 64, 40, 40, None, [40, 0]),
]


@pytest.mark.parametrize("which", ["libhd", "libhd_checked"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("shape", SHAPES, ids=[str(s) for s in SHAPES])
def test_write_and_read_guarded(libs, which, fmt, shape):
    lib = libs[which]
    B, L, n, Hkv, D, Tcap, bt, off, length = shape
    g = Guarded()
    c = _guarded_cache(g, B, Tcap, n, Hkv, D, fmt, bt)
    code = hd.HD_Q8_E4M3 if fmt == "e4m3" else hd.HD_Q8_INT8
    host = on_host(c)
    kh, vh = rows((B, Tcap * n, Hkv, D), 1, n), rows((B, Tcap * n, Hkv, D), 2, n)
    k, v = g.like(kh.cuda()), g.like(vh.cuda())
    _run(lib, "hd_kv_write_q8", k, v, 0, 0, *c[:4], B, Tcap, n, Tcap, Hkv, D, code, bt)  # the whole cache
    host = {x: oracle.kv_write_q8(t, *host[x], n, bt, fmt) for x, t in (("k", kh), ("v", vh))}
    k2h, v2h = rows((B, L * n, Hkv, D), 3, n) * 4, rows((B, L * n, Hkv, D), 4, n) * 4
    k2, v2 = g.like(k2h.cuda()), g.like(v2h.cuda())
    o = 0 if off is None else g.like(torch.tensor(off, dtype=torch.int32, device="cuda"))
    m = 0 if length is None else g.like(torch.tensor(length, dtype=torch.int32, device="cuda"))
    _run(lib, "hd_kv_write_q8", k2, v2, o, m, *c[:4], B, L, n, Tcap, Hkv, D, code, bt)
    host = {x: oracle.kv_write_q8(t, *host[x], n, bt, fmt, off, length) for x, t in (("k", k2h), ("v", v2h))}
    same_cache(c, host)
    ok, ov = g.empty((B, L * n, Hkv, D), torch.bfloat16), g.empty((B, L * n, Hkv, D), torch.bfloat16)
    _run(lib, "hd_kv_read_q8", *c[:4], o, m, ok, ov, B, L, n, Tcap, Hkv, D, code, bt)
    g.check_bands()
    _status_ok(lib)
    same_cache(c, host)
    for dev_t, host_t in ((k, kh), (v, vh), (k2, k2h), (v2, v2h)):
        assert torch.equal(dev_t.cpu(), host_t)
    for got, x in ((ok, "k"), (ov, "v")):
        want = oracle.kv_read_q8(*host[x], n, bt, fmt, L, off, length)
        assert torch.equal(got.cpu(), torch.tensor(want, dtype=torch.float32).to(torch.bfloat16))


DECODE = [  # B, n, tokens, Tcap, Hq, Hkv, D, W, bt
    (3, 3, 41, 45, 6, 2, 64, 4, 8),
    (2, 4, 300, 300, 32, 4, 128, 70, 16),   # 32 rows a KV head; parts joined
    (1, 5, 1100, 1101, 20, 4, 64, 300, 24),  # 25 rows
    (2, 2, 2000, 2003, 8, 4, 128, 900, 64),
]


@pytest.mark.parametrize("which", ["libhd", "libhd_checked"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("mode", [hd.INTRA, hd.CROSS_FULL, hd.CROSS_WINDOW], ids=["INTRA", "CROSS_FULL", "CROSS_WINDOW"])
@pytest.mark.parametrize("final", [False, True], ids=["streams", "final"])
@pytest.mark.parametrize("shape", DECODE, ids=[str(s) for s in DECODE])
def test_decode_guarded(libs, which, fmt, mode, final, shape):
    """With a workspace of exactly the bytes asked for, twice (what it held before does not matter)."""
    lib = libs[which]
    B, n, T, Tcap, Hq, Hkv, D, W, bt = shape
    scale = 1.0 / math.sqrt(D)
    g = Guarded()
    c = _guarded_cache(g, B, Tcap, n, Hkv, D, fmt, bt)
    code = hd.HD_Q8_E4M3 if fmt == "e4m3" else hd.HD_Q8_INT8
    sh = torch.tensor([T, 1, T // 2][:B], dtype=torch.int32)
    k, v = rows((B, Tcap * n, Hkv, D), 1, n).cuda(), rows((B, Tcap * n, Hkv, D), 2, n).cuda()
    sl = g.like(sh.cuda())
    _run(lib, "hd_kv_write_q8", k, v, 0, sl, *c[:4], B, Tcap, n, Tcap, Hkv, D, code, bt)
    before = on_host(c)
    qh = syn.normal_bf16((B, 1 if final else n, Hq, D), 3)
    q = g.like(qh.cuda())
    size = lib.hd_decode_final_q8_workspace_bytes if final else lib.hd_decode_q8_workspace_bytes
    need = size(B, n, Tcap, Hq, Hkv, D)
    ws = g.empty((need,), torch.uint8)
    name = "hd_decode_attn_final_q8" if final else "hd_decode_attn_q8"
    outs = []
    for _ in range(2):
        out, lse = g.empty(tuple(qh.shape), torch.bfloat16), g.empty((B, Hq, qh.shape[1]), torch.float32)
        _run(lib, name, q, *c[:4], sl, out, lse, B, n, Tcap, Hq, Hkv, D, code, bt, mode, W, ctypes.c_float(scale), ws, need)
        outs.append((out, lse))
    g.check_bands()
    _status_ok(lib)
    same_cache(c, before)
    assert torch.equal(q.cpu(), qh) and torch.equal(sl.cpu(), sh)
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    check_attention(*outs[0], qh, before, n, bt, fmt, sh, mode, W, scale, final)
