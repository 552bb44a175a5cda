"""Helpers shared by the tests of the 8-bit KV cache (no method arithmetic here)."""
import numpy as np
import torch

import oracle
import structured_causal_attention_b200 as hd

DTYPES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def rows(shape, seed, n, spread=1.0):
    """bf16 [B, L*n, Hkv, D] rows, each stream and head of its own size (powers of two within 2^+-spread)."""
    rng = np.random.default_rng(seed)
    B, S, Hkv, D = shape
    size = 2.0 ** rng.uniform(-spread, spread, (n, Hkv, 1))
    x = rng.standard_normal((B, S // n, n, Hkv, D)) * size
    return torch.tensor(x.reshape(shape), dtype=torch.float32).to(torch.bfloat16)


def garbage_cache(B, Tcap, n, Hkv, D, fmt, bt, seed=0, device="cuda"):
    """A cache whose memory holds arbitrary bytes, NaN codes and scales among them: nothing was written yet."""
    g = torch.Generator().manual_seed(seed)

    def codes():
        x = torch.randint(0, 256, (B, Tcap * n, Hkv, D), generator=g, dtype=torch.int64).to(torch.uint8)
        x[:, :, :, ::3] = 0x7F
        return x.view(DTYPES[fmt]).to(device)

    def scale():
        s = torch.full((B, Hkv, -(-Tcap // bt), n), float("nan"))
        s[:, :, ::2] = 1e30
        return s.to(device)

    return hd.KVCacheQ8(codes(), codes(), scale(), scale(), n, bt)


def on_host(cache):
    """{"k": (bytes, scales), "v": ...} of a cache, as the oracle takes them."""
    return {x: (getattr(cache, x).view(torch.uint8).cpu().numpy(), getattr(cache, x + "_scale").double().cpu().numpy())
            for x in ("k", "v")}


def same_cache(cache, want):
    """The cache's bytes and scales are the oracle's, bit by bit (-0 and 0 are both a zero code)."""
    for x in ("k", "v"):
        codes, scale = on_host(cache)[x]
        assert np.array_equal(scale, want[x][1], equal_nan=True), f"{x} scales"
        assert np.array_equal(codes, want[x][0]), f"{x} codes"


def check_attention(out, lse, q, host, n, bt, fmt, seqlen, mode, W, scale, final):
    """Against the oracle on the values that a cache holds; host: on_host() of it, or the oracle's.

    An output is off by its rounding to bf16 (2^-8 of it, half a step) and by the weights': each weight
    p_j vs_j is rounded to fp16 (2^-11 of it), and its score is off by E, which changes it by E (and the sum
    by as much). E: the dot product accumulates D products in fp32 (D / 16 roundings of at most 2^-23 of
    sum |q k|), and the exponent's roundings are four of 2^-24 of at most |score| + 60 each: with scores and
    sum |q k| * scale below 2^8 here, less than 2^-12 + 2^-14. (A query element is held to 2^-40 of the row's
    largest.) So |error| <= 2^-8 |O| + (2^-11 + 2 E) sum p |v| < 2^-8 |O| + 2^-9 sum p |v|.
    A weight far below the row's largest is a subnormal fp16: the largest is in [2^13, 2^14] there, so it is
    off by at most 2^-25 / 2^13 = 2^-38 of the largest, times its code (at most 448, or 127); over N keys that
    adds 2^-38 N 448 max_j p_j vs_j. An lse is off by E and the roundings of the sum and the logarithm, below
    2^-11 in all (plus 2^-22 of it)."""
    k, v = (oracle.kv_values_q8(*host[x], n, bt, fmt) for x in ("k", "v"))
    seqlen = np.asarray(seqlen.cpu() if hasattr(seqlen, "cpu") else seqlen)
    want, want_lse = oracle.decode_attn(q, k, v, seqlen, n, mode, W, scale, final_only=final)
    size, _ = oracle.decode_attn(q, k, np.abs(v), seqlen, n, mode, W, scale, final_only=final)
    got = out.detach().double().cpu().numpy()
    assert got.shape == want.shape and np.isfinite(got).all()
    floor = np.zeros(want.shape[:3] + (1,))
    g = q.shape[2] // k.shape[2]
    qd = q.detach().double().cpu().numpy()
    for b, tokens in enumerate(seqlen):
        p = np.arange(tokens * n)
        at = (tokens - 1) * n + np.arange(n - q.shape[1], n)
        seen = oracle.visible(at[:, None], p[None, :], n, mode, W)
        for h in range(q.shape[2]):
            weight = np.exp(scale * qd[b, :, h] @ k[b, :tokens * n, h // g].T - want_lse[b, h][:, None])
            weight = np.where(seen, weight * host["v"][1][b, h // g, p // n // bt, p % n], 0)
            floor[b, :, h, 0] = 2.0 ** -38 * 448 * seen.sum(axis=1) * weight.max(axis=1)
    bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * size + floor + 1e-300
    worst = float((np.abs(got - want) / bound).max())
    assert worst <= 1, f"out: {worst:.3f} of the bound"
    got_lse = lse.detach().double().cpu().numpy()
    err = np.abs(got_lse - want_lse) / (2.0 ** -11 + 2.0 ** -22 * np.abs(want_lse))
    assert err.max() <= 1, f"lse: {float(err.max()):.3f} of the bound"
