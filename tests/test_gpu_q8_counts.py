"""Full-size decode steps against the 8-bit cache in which one key lost or counted twice shows.

q = 0, so every visible key weighs 1 / N. Channel 0 of V is 1 everywhere; each position has a second 1, in one of the
other channels of one head, so that a (head, channel) has about 64 of the 65540 positions, and its output, their share,
moves by a part in 64 when one of them is lost or read twice - against 2^-8 of the rounding to bf16."""
import numpy as np
import pytest
import torch

import oracle
import structured_causal_attention_b200 as hd
from structured_causal_attention_b200 import synthetic as syn
from tests.gpu_util import need_gpu
from tests.q8_util import DTYPES, on_host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("final", [False, True], ids=["streams", "final"])
@pytest.mark.parametrize("ragged", [False, True], ids=["even", "ragged"])
def test_every_key_counts_once(fmt, final, ragged):
    """An output is a sum of N equal weights' share over their sum: off by the weight's rounding to fp16 (2^-11), by the
    roundings of the sums (at most 600 terms follow one another in a lane, and an MMA's sum is right to 2^-23: 2^-13) and
    to bf16 (2^-8): within 2^-8 + 2^-10 of it, where one key is 1/65 of it or more. An lse is log N, off by the sum's
    roundings (600 of 2^-24: 2^-14) and by those of the reference, the logarithm and their product: 2^-14 + 2^-19."""
    need_gpu()
    w = syn.WORKLOADS["decode"]
    B, n, T, Hq, Hkv, D, W, bt = w["B"], w["n"], w["T"] + 1, w["Hq"], w["Hkv"], w["D"], 1024, 16
    rng = np.random.default_rng(1)
    channel = rng.permutation(np.arange(T * n) % (Hkv * (D - 1)))  # of the position: head * (D - 1) + channel - 1
    head, at = channel // (D - 1), channel % (D - 1) + 1
    v = torch.zeros(1, T * n, Hkv, D)
    v[..., 0] = 1
    v[0, torch.arange(T * n), torch.tensor(head), torch.tensor(at)] = 1
    v = v.to(torch.bfloat16).cuda().expand(B, -1, -1, -1).contiguous()
    cache = hd.kv_cache_q8(B, T, n, Hkv, D, DTYPES[fmt], bt)
    hd.kv_write_q8(torch.ones_like(v), v, cache)
    assert bool((cache.v_scale == cache.v_scale.flatten()[0]).all())
    first = on_host(cache._replace(**{x: getattr(cache, x)[:1, :n] for x in ("k", "v")}))["v"]
    one = oracle.kv_values_q8(*first, n, bt, fmt)[0, 0, 0, 0]  # what 1 is held as
    seqlen = np.full(B, T)
    if ragged:
        seqlen[1:] = rng.integers(T // 2, T, B - 1)
    sl = torch.tensor(seqlen, dtype=torch.int32, device="cuda")
    nq = 1 if final else n
    q = torch.zeros(B, nq, Hq, D, dtype=torch.bfloat16, device="cuda")
    call = hd.decode_attn_final_q8 if final else hd.decode_attn_q8
    p = np.arange(T * n)
    for mode in (hd.INTRA, hd.CROSS_FULL, hd.CROSS_WINDOW):
        out, lse = call(q, cache, sl, mode, W, 1.0)
        got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for b in range(B):
            for s in range(nq):
                own = (seqlen[b] - 1) * n + n - nq + s
                seen = oracle.visible(own, p, n, mode, W)
                N = seen.sum()
                share = np.zeros((Hkv, D))
                np.add.at(share, (head[seen], at[seen]), one / N)
                share[:, 0] = one
                want = np.repeat(share, Hq // Hkv, axis=0)
                err = np.abs(got[b, s] - want)
                assert (err <= (2.0 ** -8 + 2.0 ** -10) * want).all(), (mode, b, s, (err / np.maximum(want, 1e-30)).max())
                assert np.abs(got_lse[b, :, s] - np.log(N)).max() <= 2.0 ** -14 + 2.0 ** -19
    assert hd.hd_device_status() == hd.HD_OK
