"""CPU oracle: an 8-bit KV cache, written and read back.

TEST INFRASTRUCTURE ONLY; the library never calls it.

Source (page "微信WeLM提出Hidden Decoding：大模型推理新范式", tahou.com): section
"中间流的作用验证", each stream keeps its own KV state. The 8-bit formats are not
on the pages; this is their definition.

codes [B, Tcap*n, Hkv, D] (numpy uint8: the bytes), scales float64
[B, Hkv, ceil(Tcap / bt), n]; the scale of block j, stream s and head h covers
tokens j*bt .. (j+1)*bt - 1 of stream s. value = code * scale.

  e4m3  sign, 4 exponent bits (bias 7), 3 mantissa bits, no infinity, largest
        448; scale = the smallest power of two with absmax <= 448 * scale
  int8  two's complement; scale = absmax / 127 rounded up to 8 significant bits

No scale is smaller than 2^-60. Rounding is to nearest, ties to even.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

from .attention import _f64

MIN_SCALE = 2.0 ** -60


def _e4m3_values():
    """The value of every byte, from the format's definition (0x7f and 0xff are NaN)."""
    v = np.zeros(256)
    for byte in range(256):
        exponent, mantissa = (byte >> 3) & 15, byte & 7
        if exponent == 15 and mantissa == 7:
            v[byte] = np.nan
            continue
        size = mantissa / 8 * 2.0 ** -6 if exponent == 0 else (1 + mantissa / 8) * 2.0 ** (exponent - 7)
        v[byte] = -size if byte & 128 else size
    return v


E4M3 = _e4m3_values()


def code_values(codes, fmt):
    """Bytes -> the values of the codes, float64."""
    codes = np.asarray(codes, dtype=np.uint8)
    return E4M3[codes] if fmt == "e4m3" else codes.view(np.int8).astype(np.float64)


def encode(x, fmt):
    """Values over their scale -> bytes: nearest code, ties to the even one."""
    x = np.asarray(x, dtype=np.float64)
    if fmt == "int8":
        return np.rint(x).astype(np.int8).view(np.uint8)
    sizes = E4M3[:127]  # 0 .. 448, ascending; the byte is the index
    a = np.abs(x)
    hi = np.clip(np.searchsorted(sizes, a), 0, 126)
    lo = np.clip(hi - 1, 0, 126)
    up, down = sizes[hi] - a, a - sizes[lo]
    byte = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    byte = np.where(sizes[hi] == a, hi, byte)
    return (byte | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def scale_for(absmax, fmt):
    """The scale that values up to ``absmax`` need, in exact arithmetic."""
    a = Fraction(float(absmax))
    if a == 0:
        return MIN_SCALE
    want = a / 448 if fmt == "e4m3" else a / 127
    j = math.frexp(float(want))[1] + 2
    while Fraction(2) ** (j - 1) >= want:
        j -= 1  # the smallest power of two that is not below what is wanted
    if fmt == "e4m3":
        return max(float(Fraction(2) ** j), MIN_SCALE)
    step = Fraction(2) ** (j - 8)  # 8 significant bits below 2^j
    return max(float(-(-want // step) * step), MIN_SCALE)


def kv_write_q8(x, codes, scale, n, bt, fmt, token_offset=None, lengths=None):
    """Write x [B, L*n, Hkv, D] (K or V) at tokens token_offset[b] ..; returns (codes, scale), new arrays."""
    x = _f64(x)
    B, S, Hkv, D = x.shape
    L = S // n
    codes = np.array(codes, dtype=np.uint8)
    scale = np.array(scale, dtype=np.float64)
    Tcap = codes.shape[1] // n
    for b in range(B):
        t0 = 0 if token_offset is None else int(token_offset[b])
        t1 = t0 + (L if lengths is None else int(lengths[b]))
        if t0 < 0 or t1 < t0 or t1 - t0 > L or t1 > Tcap:
            continue
        for j in range(t0 // bt, -(-t1 // bt)):
            lo, hi = max(t0, j * bt), min(t1, (j + 1) * bt)
            if lo >= hi:
                continue
            for s in range(n):
                for h in range(Hkv):
                    new = x[b, [(t - t0) * n + s for t in range(lo, hi)], h]
                    old = scale[b, h, j, s] if j * bt < t0 else 0.0
                    at = [t * n + s for t in range(lo, hi)]
                    if not np.isfinite(new).all() or np.isnan(old):
                        scale[b, h, j, s] = np.nan
                        codes[b, at, h] = 0
                        continue
                    now = max(old, scale_for(np.abs(new).max(), fmt))
                    if j * bt < t0 and now > old:
                        was = [t * n + s for t in range(j * bt, t0)]
                        codes[b, was, h] = encode(code_values(codes[b, was, h], fmt) * old / now, fmt)
                    scale[b, h, j, s] = now
                    codes[b, at, h] = encode(new / now, fmt)
    return codes, scale


def kv_values_q8(codes, scale, n, bt, fmt):
    """The whole cache as float64 values [B, Tcap*n, Hkv, D]."""
    codes = np.asarray(codes, dtype=np.uint8)
    p = np.arange(codes.shape[1])
    s = np.asarray(scale, dtype=np.float64)[:, :, p // n // bt, p % n]  # [B, Hkv, positions]
    return code_values(codes, fmt) * np.moveaxis(s, 1, 2)[..., None]


def kv_read_q8(codes, scale, n, bt, fmt, L, token_offset=None, lengths=None):
    """float64 [B, L*n, Hkv, D]: tokens token_offset[b] .., zeros behind lengths[b] and for a range outside."""
    v = kv_values_q8(codes, scale, n, bt, fmt)
    B, S, Hkv, D = v.shape
    out = np.zeros((B, L * n, Hkv, D))
    for b in range(B):
        t0 = 0 if token_offset is None else int(token_offset[b])
        m = L if lengths is None else int(lengths[b])
        if t0 >= 0 and 0 <= m <= L and (t0 + m) * n <= S:
            out[b, :m * n] = v[b, t0 * n:(t0 + m) * n]
    return out
