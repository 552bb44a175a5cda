"""What the 8-bit cache's calls and helpers say of sizes and arguments that they do not take."""
import pytest
import torch

import structured_causal_attention_b200 as hd
from structured_causal_attention_b200.build import build

FAKE = 0x10000  # an aligned, never-dereferenced address: validation fails first


@pytest.fixture(scope="module")
def lib():
    build()
    return hd.lib()


@pytest.mark.parametrize("final", [False, True], ids=["streams", "final"])
@pytest.mark.parametrize("sizes,code", [
    # B, n, Tcap, Hq, Hkv, D
    ((2, 4, 100, 16, 4, 96), hd.HD_ERR_UNSUPPORTED), ((1, 1, 2**28 + 1, 4, 4, 64), hd.HD_ERR_UNSUPPORTED),
    ((8, 4, 2**26, 32, 8, 128), hd.HD_ERR_UNSUPPORTED), ((2, 4, 100, 16, 4, 128), hd.HD_ERR_INVALID_ARG),
    ((2, 4, 100, 15, 4, 128), hd.HD_ERR_INVALID_ARG),
])
def test_sizes_are_judged_before_the_workspace(lib, sizes, code, final):
    """The workspace of sizes that are not supported has 0 bytes, and no address: the sizes are what is wrong."""
    fn = lib.hd_decode_attn_final_q8 if final else lib.hd_decode_attn_q8
    size = lib.hd_decode_final_q8_workspace_bytes if final else lib.hd_decode_q8_workspace_bytes
    assert (size(*sizes) == 0) == (code == hd.HD_ERR_UNSUPPORTED or sizes[3] % sizes[4] != 0)
    for mode in (hd.INTRA, hd.CROSS_FULL, hd.CROSS_WINDOW):
        assert fn(*[FAKE] * 8, *sizes, hd.HD_Q8_INT8, 16, mode, 1, 0.1, None, 0, None) == code


@pytest.mark.gpu
@pytest.mark.parametrize("call,rows", [(hd.decode_attn_q8, 2), (hd.decode_attn_final_q8, 1)], ids=["streams", "final"])
def test_helpers_name_unsupported_sizes(call, rows):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    cache = hd.kv_cache_q8(1, 10, 2, 2, 96, torch.int8)
    q = torch.zeros(1, rows, 4, 96, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(hd.HDError) as e:
        call(q, cache, torch.ones(1, dtype=torch.int32, device="cuda"), hd.CROSS_FULL)
    assert e.value.status == hd.HD_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(block_tokens=0), dict(block_tokens=-16), dict(n=0), dict(Tcap=0), dict(B=0), dict(Hkv=0),
                                dict(D=0), dict(dtype=torch.bfloat16), dict(dtype=torch.uint8), dict(dtype=torch.float8_e5m2)])
def test_a_cache_of_bad_sizes_is_not_made(kw):
    a = dict(B=1, Tcap=8, n=2, Hkv=2, D=64, dtype=torch.int8, block_tokens=16, device="cpu")
    hd.kv_cache_q8(**a)
    with pytest.raises(ValueError):
        hd.kv_cache_q8(**dict(a, **kw))
