"""The 8-bit cache's entry points refuse bad arguments on the host, before any launch (no GPU needed)."""
import pytest
import torch

import structured_causal_attention_b200 as hd
from structured_causal_attention_b200.build import build

FAKE = 0x10000  # an aligned, never-dereferenced address: validation fails first


@pytest.fixture(scope="module")
def lib():
    build()
    return hd.lib()


ROWS = dict(k=FAKE, v=FAKE, off=FAKE, len=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, B=2, L=8, n=4, Tcap=64, Hkv=2,
            D=128, fmt=hd.HD_Q8_E4M3, bt=16)
BAD_ROWS = [
    (dict(k=0), 1), (dict(v=0), 1), (dict(kc=0), 1), (dict(vc=0), 1), (dict(ks=0), 1), (dict(vs=0), 1),
    (dict(k=FAKE + 8), 1), (dict(v=FAKE + 2), 1), (dict(kc=FAKE + 4), 1), (dict(vc=FAKE + 1), 1),
    (dict(ks=FAKE + 4), 1), (dict(vs=FAKE + 8), 1), (dict(B=0), 1), (dict(L=0), 1), (dict(n=0), 1), (dict(Tcap=0), 1),
    (dict(Hkv=0), 1), (dict(D=0), 1), (dict(fmt=2), 1), (dict(fmt=-1), 1), (dict(bt=0), 1), (dict(bt=-4), 1),
    (dict(bt=1025), 2), (dict(D=96), 2), (dict(D=256), 2), (dict(Tcap=1 << 27), 2), (dict(L=1 << 27), 2),
    (dict(L=1 << 24, Hkv=8), 2),  # more than 2^31 chunks of 8 elements a sequence
]


@pytest.mark.parametrize("kw,code", BAD_ROWS)
@pytest.mark.parametrize("which", ["write", "read"])
def test_write_and_read_refuse(lib, which, kw, code):
    a = dict(ROWS, **kw)
    sizes = [a[x] for x in ("B", "L", "n", "Tcap", "Hkv", "D", "fmt", "bt")]
    if which == "write":
        st = lib.hd_kv_write_q8(a["k"], a["v"], a["off"], a["len"], a["kc"], a["vc"], a["ks"], a["vs"], *sizes, None)
    else:
        st = lib.hd_kv_read_q8(a["kc"], a["vc"], a["ks"], a["vs"], a["off"], a["len"], a["k"], a["v"], *sizes, None)
    assert st == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), 1), (dict(kc=0), 1), (dict(vc=0), 1), (dict(ks=0), 1), (dict(vs=0), 1), (dict(sl=0), 1), (dict(out=0), 1),
    (dict(lse=0), 1), (dict(ws=0), 1), (dict(q=FAKE + 8), 1), (dict(kc=FAKE + 8), 1), (dict(vs=FAKE + 4), 1),
    (dict(out=FAKE + 2), 1), (dict(ws=FAKE + 8), 1), (dict(B=0), 1), (dict(n=-1), 1), (dict(Tcap=0), 1), (dict(Hq=3), 1),
    (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(fmt=2), 1), (dict(bt=0), 1), (dict(bt=2000), 2), (dict(mode=3), 1),
    (dict(mode=-1), 1), (dict(mode=hd.CROSS_WINDOW, W=0), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(D=80), 2), (dict(Tcap=1 << 27), 2), (dict(short=1), 1),
])
@pytest.mark.parametrize("final", [False, True], ids=["streams", "final"])
def test_decode_refuses(lib, final, kw, code):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, sl=FAKE, out=FAKE, lse=FAKE, B=2, n=4, Tcap=100, Hq=16, Hkv=4,
             D=128, fmt=hd.HD_Q8_INT8, bt=16, mode=hd.CROSS_FULL, W=1, scale=0.1, ws=FAKE, short=0)
    size = hd.hd_decode_final_q8_workspace_bytes if final else hd.hd_decode_q8_workspace_bytes
    need = size(2, 4, 100, 16, 4, 128)
    assert need > 0
    a.update(kw)
    fn = lib.hd_decode_attn_final_q8 if final else lib.hd_decode_attn_q8
    st = fn(*[a[x] for x in ("q", "kc", "vc", "ks", "vs", "sl", "out", "lse", "B", "n", "Tcap", "Hq", "Hkv", "D", "fmt",
                             "bt", "mode", "W", "scale", "ws")], (1 << 40) if not a["short"] else need - 1, None)
    assert st == code


def test_workspace_of_bad_sizes_is_zero(lib):
    for size in (hd.hd_decode_q8_workspace_bytes, hd.hd_decode_final_q8_workspace_bytes):
        assert size(0, 4, 100, 16, 4, 128) == 0
        assert size(2, 4, 100, 15, 4, 128) == 0


def test_helpers_refuse_cpu_tensors(lib):
    x = torch.zeros(1, 8, 2, 64, dtype=torch.bfloat16)
    cache = hd.kv_cache_q8(1, 4, 2, 2, 64, torch.int8, device="cpu")
    with pytest.raises(ValueError):
        hd.kv_write_q8(x, x, cache)
    with pytest.raises(ValueError):
        hd.kv_read_q8(cache, 4)
    with pytest.raises(ValueError):
        hd.decode_attn_q8(x[:, :2], cache, torch.ones(1, dtype=torch.int32), hd.INTRA)


def test_binding_raises_on_error(lib):
    with pytest.raises(hd.HDError) as e:
        hd.hd_kv_write_q8(FAKE, FAKE, 0, 0, FAKE, FAKE, FAKE, FAKE, 1, 8, 4, 64, 2, 96, 0, 16, stream=0)
    assert e.value.status == hd.HD_ERR_UNSUPPORTED


# (each of these has a product that passes 32 or 64 bits; the queries' rows of the first come to 2^32)
@pytest.mark.parametrize("sizes", [
    (1, 65536, 1, 65536, 1, 64), (2**31 - 1, 2**28, 1, 2**31 - 1, 1, 128), (2**31 - 1, 1, 1, 2, 1, 64),
    (1, 1, 2**28, 2**31 - 1, 2**31 - 1, 128), (1, 1, 2**31 - 1, 1, 1, 64), (1, 2, 1, 2**30, 1, 64),
    (8, 4, 2**26, 32, 8, 128), (1, 1, 100, 4, 4, 2**31 - 1),
])
@pytest.mark.parametrize("final", [False, True], ids=["streams", "final"])
def test_sizes_past_the_counters_are_refused(lib, final, sizes):
    """No product of sizes wraps: the workspace's size is 0 and the call refused, for each mode."""
    size = hd.hd_decode_final_q8_workspace_bytes if final else hd.hd_decode_q8_workspace_bytes
    assert size(*sizes) == 0
    fn = lib.hd_decode_attn_final_q8 if final else lib.hd_decode_attn_q8
    for mode in (hd.INTRA, hd.CROSS_FULL, hd.CROSS_WINDOW):
        st = fn(*[FAKE] * 8, *sizes, hd.HD_Q8_INT8, 16, mode, 1, 0.1, FAKE, 2**63, None)
        assert st == hd.HD_ERR_UNSUPPORTED


@pytest.mark.parametrize("other", ["0x10000", b"0x10000", 65536.0, [FAKE]])
def test_only_tensors_and_addresses_are_pointers(lib, other):
    """Text and bytes are no device pointers, though ctypes would pass their host address."""
    assert hd._lib.ptr(None) == 0 and hd._lib.ptr(FAKE) == FAKE
    with pytest.raises(AttributeError):
        hd._lib.ptr(other)
