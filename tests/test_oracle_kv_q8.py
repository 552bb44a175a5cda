"""Pins of the 8-bit cache's oracle: the formats against torch's types and hand-worked values, the scales
against their definitions, writing in pieces against writing at once, and planted mistakes."""
import inspect
import types

import numpy as np
import pytest
import torch

import oracle
import oracle.kv_q8 as kv


def test_e4m3_bytes_are_the_formats_values():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(kv.E4M3, want, equal_nan=True)


def test_e4m3_rounds_as_torch_does():
    x = torch.cat([torch.randn(4000, generator=torch.Generator().manual_seed(1)) * 2.0 ** e for e in range(-10, 8)])
    x = x.clamp(-448, 448)
    mid = torch.tensor((kv.E4M3[:126] + kv.E4M3[1:127]) / 2, dtype=torch.float32)  # every tie
    x = torch.cat([x, mid, -mid, torch.zeros(1), torch.tensor([-0.0])])
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kv.encode(x.double().numpy(), "e4m3"), want)


@pytest.mark.parametrize("absmax,fmt,want", [
    (448.0, "e4m3", 1.0), (450.0, "e4m3", 2.0), (7.0, "e4m3", 2.0 ** -6), (0.0, "e4m3", 2.0 ** -60),
    (2.0 ** -100, "e4m3", 2.0 ** -60), (127.0, "int8", 1.0), (254.0, "int8", 2.0), (0.0, "int8", 2.0 ** -60),
    (128.0, "int8", 1.0 + 2.0 ** -6), (1.0, "int8", 2.0 ** -7 * (1 + 2.0 ** -6)),
])
def test_scales_worked_by_hand(absmax, fmt, want):
    assert kv.scale_for(absmax, fmt) == want


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_scale_is_the_smallest_that_holds_the_value(fmt):
    for m in range(128, 256):
        for e in (-20, -1, 0, 3, 40):
            a = m * 2.0 ** e
            s = kv.scale_for(a, fmt)
            top = 448 if fmt == "e4m3" else 127
            assert top * s >= a
            # the next smaller scale: half, or one step of 8 significant bits (the upper half of an fp32) less
            bits = np.float32(s).view(np.uint32)
            below = s / 2 if fmt == "e4m3" else float((bits - np.uint32(0x10000)).view(np.float32))
            assert top * below < a
            if fmt == "int8":
                assert float(np.float32(s).view(np.uint32) & 0xffff) == 0  # 8 significant bits


def test_int8_ties_are_exact_or_far():
    """x / scale, both of 8 significant bits, is a tie or at least 1/1020 away from one (so the rounded code
    does not depend on the arithmetic); enumerated."""
    a, b = np.meshgrid(np.arange(128, 256), np.arange(128, 256))
    for e in range(-10, 8):
        r = a * 2.0 ** e / b
        r = r[r <= 127.5]
        d = np.abs(r - (np.floor(r) + 0.5))
        assert ((d == 0) | (d >= 1 / 1020)).all()


def _cache(B, Tcap, n, Hkv, D, bt):
    return np.zeros((B, Tcap * n, Hkv, D), np.uint8), np.zeros((B, Hkv, -(-Tcap // bt), n))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_a_falling_range_is_the_same_written_at_once_or_token_by_token(fmt):
    """Each block's largest value comes first, so no scale is raised: pieces and the whole agree."""
    rng = np.random.default_rng(3)
    B, L, n, Hkv, D, bt = 2, 13, 3, 2, 4, 5
    x = torch.tensor(rng.standard_normal((B, L * n, Hkv, D))).to(torch.bfloat16).double().numpy()
    x.reshape(B, L, n, Hkv, D)[:, ::bt] = 8.0
    whole = kv.kv_write_q8(x, *_cache(B, 16, n, Hkv, D, bt), n, bt, fmt)
    piece = _cache(B, 16, n, Hkv, D, bt)
    for t in range(L):
        piece = kv.kv_write_q8(x[:, t * n:(t + 1) * n], *piece, n, bt, fmt, token_offset=[t] * B)
    assert np.array_equal(whole[0], piece[0]) and np.array_equal(whole[1], piece[1])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_values_are_within_half_a_step(fmt):
    rng = np.random.default_rng(4)
    B, L, n, Hkv, D, bt = 2, 11, 2, 2, 8, 4
    x = torch.tensor(rng.standard_normal((B, L * n, Hkv, D)) * 3).to(torch.bfloat16).double().numpy()
    codes, scale = kv.kv_write_q8(x, *_cache(B, L, n, Hkv, D, bt), n, bt, fmt)
    got = oracle.kv_read_q8(codes, scale, n, bt, fmt, L)
    s = scale[:, :, np.arange(L * n) // n // bt, np.arange(L * n) % n]
    s = np.moveaxis(s, 1, 2)[..., None]
    # int8: half a step of the scale; e4m3: half of 2^-3 of the value's power of two, or of 2^-9
    half = s / 2 if fmt == "int8" else np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10)
    assert (np.abs(got - x) <= half).all()


def test_a_raised_scale_rounds_the_earlier_codes_again():
    codes, scale = _cache(1, 4, 1, 1, 2, 4)
    codes, scale = kv.kv_write_q8(np.array([[[[127.0, 3.0]]]]), codes, scale, 1, 4, "int8")
    assert scale[0, 0, 0, 0] == 1 and codes[0, 0, 0].tolist() == [127, 3]
    codes, scale = kv.kv_write_q8(np.array([[[[254.0, 1.0]]]]), codes, scale, 1, 4, "int8", token_offset=[1])
    assert scale[0, 0, 0, 0] == 2
    assert codes[0, 0, 0].tolist() == [64, 2]  # 63.5 and 1.5: ties to even
    assert codes[0, 1, 0].tolist() == [127, 0]


MUTANTS = [
    ("scale not raised", "now = max(old, scale_for(np.abs(new).max(), fmt))", "now = old or scale_for(np.abs(new).max(), fmt)"),
    ("codes kept as they were", "encode(code_values(codes[b, was, h], fmt) * old / now, fmt)", "codes[b, was, h]"),
    ("ties upwards", "np.rint(x)", "np.floor(x + 0.5)"),
    ("rounded down scale", "float(-(-want // step) * step)", "float((want // step) * step)"),
    ("448 as 256", "a / 448", "a / 256"),
    ("block not started afresh", "if j * bt < t0 else 0.0", "if True else 0.0"),
]


@pytest.mark.parametrize("name,old,new", MUTANTS, ids=[m[0] for m in MUTANTS])
def test_planted_mistakes_are_seen(name, old, new, monkeypatch):
    src = inspect.getsource(kv)
    assert src.count(old) == 1, old
    mod = types.ModuleType("kv_q8_mutant")
    mod.__dict__["__package__"] = "oracle"
    exec(compile(src.replace(old, new), "kv_q8_mutant", "exec"), mod.__dict__)
    monkeypatch.setitem(globals(), "kv", mod)
    caught = 0
    for check in (test_a_raised_scale_rounds_the_earlier_codes_again,
                  lambda: test_scale_is_the_smallest_that_holds_the_value("int8"),
                  lambda: test_scale_is_the_smallest_that_holds_the_value("e4m3"),
                  lambda: test_scales_worked_by_hand(450.0, "e4m3", 2.0),
                  _rewritten_block_forgets):
        try:
            check()
        except AssertionError:
            caught += 1
    assert caught


def _rewritten_block_forgets():
    codes, scale = _cache(1, 4, 1, 1, 2, 4)
    codes, scale = kv.kv_write_q8(np.full((1, 2, 1, 2), 127.0), codes, scale, 1, 4, "int8")
    codes, scale = kv.kv_write_q8(np.full((1, 2, 1, 2), 0.5), codes, scale, 1, 4, "int8")
    assert scale[0, 0, 0, 0] < 1


def test_rewritten_block_forgets_its_scale():
    _rewritten_block_forgets()
