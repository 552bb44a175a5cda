"""What is measured of the 8-bit KV cache: writing it, reading it back, and the decode attention over it.

The cache holds K and V of the expanded sequence (n streams a token, stream s of token t at position
t*n + s) as one byte an element, codes [B, Tcap*n, Hkv, D], with fp32 scales [B, Hkv, blocks, n]: one for
each block of `bt` tokens, each stream and each head. A value is code * scale.

  e4m3  scale = the smallest power of two with absmax <= 448 * scale
  int8  scale = absmax / 127 rounded up to 8 significant bits
        (both at least 2^-60); code = value / scale, rounded to nearest, ties to even

Writing tokens [t0, t0 + len): a block whose first token is among them starts afresh; a block that was
begun before keeps its scale, or raises it to what the new rows need, and then its earlier codes are
rounded again at the new scale. Reading gives code * scale in bf16. A decode step is the attention of the
new token's n stream queries (or the last stream's alone) over the cached positions that the mask shows:
0 INTRA (same stream), 1 CROSS_FULL, 2 CROSS_WINDOW (the last n*W positions).

A case that writes also reads the written blocks back, as a prefill does that attends to what the cache
holds, so that the codes come out as the values that they stand for.
"""
import math

import torch

own = False

INTRA, CROSS_FULL, CROSS_WINDOW = 0, 1, 2
MIN_SCALE = 2.0 ** -60
DTYPES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


# ------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # a serving step's append: one token for each of 8 sequences of about 16384 tokens, inside a block
        dict(name="write_token", op="write", fmt="int8", bt=16, B=8, n=4, Hkv=8, D=128, L=1, Tcap=16400,
             first=16000, ragged=True),
        # a prompt of two long sequences, written whole (the sliding-window layer's sizes)
        dict(name="write_prompt", op="write", fmt="e4m3", bt=16, B=2, n=4, Hkv=8, D=128, L=8192, Tcap=8208,
             first=0, ragged=False),
        # a chunk of prompts that differ in length, appended inside blocks: padded rows, odd sizes
        dict(name="write_chunk", op="write", fmt="int8", bt=32, B=5, n=3, Hkv=2, D=64, L=331, Tcap=1501,
             first=700, ragged=True),
        # a long cached prefix read back as bf16, for the prefill that goes on from it
        dict(name="read_prefix", op="read", fmt="int8", bt=16, B=1, n=4, Hkv=8, D=128, L=32768, Tcap=32768,
             first=0, ragged=False),
        # pieces of different lengths from inside their sequences, blocks that end inside the range
        dict(name="read_chunk", op="read", fmt="e4m3", bt=8, B=5, n=3, Hkv=2, D=64, L=333, Tcap=1501,
             first=700, ragged=True),
        # the first tokens of one short sequence: latency
        dict(name="decode_short", op="decode", fmt="e4m3", bt=16, B=1, n=4, Hq=4, Hkv=4, D=64, T=63, Tcap=64,
             mode=CROSS_FULL, W=0, ragged=False),
        # decode at a small batch against a long cache
        dict(name="decode8", op="decode", fmt="e4m3", bt=16, B=8, n=4, Hq=32, Hkv=8, D=128, T=16384, Tcap=16385,
             mode=CROSS_FULL, W=0, ragged=False),
        # decode at a large batch against a long cache
        dict(name="decode64", op="decode", fmt="int8", bt=16, B=64, n=4, Hq=32, Hkv=8, D=128, T=16384,
             Tcap=16385, mode=CROSS_FULL, W=0, ragged=False),
        # a sliding-window layer's step, sequences of different lengths
        dict(name="decode_window", op="decode", fmt="int8", bt=16, B=8, n=4, Hq=32, Hkv=8, D=128, T=16384,
             Tcap=16385, mode=CROSS_WINDOW, W=1024, ragged=True),
        # an intra-stream layer with three streams and seven query heads a KV head: 21 rows share a key
        dict(name="decode_intra_odd", op="decode", fmt="e4m3", bt=24, B=3, n=3, Hq=14, Hkv=2, D=64, T=5003,
             Tcap=5021, mode=INTRA, W=0, ragged=True),
        # a mirror layer's step: the last stream's query over all streams' keys
        dict(name="final8", op="final", fmt="int8", bt=16, B=8, n=4, Hq=32, Hkv=8, D=128, T=16384, Tcap=16385,
             mode=CROSS_FULL, W=0, ragged=False),
        # a mirror layer of the intra-stream kind: only the last stream's rows are read
        dict(name="final8_intra", op="final", fmt="e4m3", bt=16, B=8, n=4, Hq=32, Hkv=8, D=128, T=16384,
             Tcap=16385, mode=INTRA, W=0, ragged=True),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    c = dict(op=rng.choice(["write", "read", "decode", "decode", "final"]), fmt=rng.choice(["e4m3", "int8"]),
             bt=rng.choice([8, 16, 16, 24, 32, 64]), n=rng.choice([1, 2, 3, 4, 4, 8]), D=rng.choice([64, 128]),
             Hkv=rng.randint(1, 8), ragged=rng.random() < 0.7)
    if c["op"] in ("write", "read"):
        c["B"] = _spread(rng, 1, 16)
        c["L"] = _spread(rng, 1, 8192)
        c["L"] = max(1, min(c["L"], 2 ** 28 // (c["B"] * c["n"] * c["Hkv"] * c["D"])))
        c["first"] = rng.choice([0, rng.randint(0, 4 * c["bt"]), _spread(rng, 1, 2048)])
        c["Tcap"] = c["first"] + c["L"] + 3 * c["bt"] + rng.randint(0, 20)
        return c
    c["B"] = _spread(rng, 1, 64)
    c["Hq"] = c["Hkv"] * rng.randint(1, 8)
    c["T"] = _spread(rng, 1, 16384)
    c["T"] = max(1, min(c["T"], 2 ** 30 // (c["B"] * c["n"] * c["Hkv"] * c["D"])))
    c["Tcap"] = c["T"] + 1 + rng.choice([0, rng.randint(0, 100)])
    c["mode"] = rng.choice([INTRA, CROSS_FULL, CROSS_WINDOW])
    c["W"] = _spread(rng, 1, 2 * c["T"]) if c["mode"] == CROSS_WINDOW else 0
    return c


# ------------------------------------------------------------------------------------ inputs, on the GPU

def _rows(gen, shape):
    """bf16 rows [..., n, Hkv, D] as K and V have them: each stream and head of its own size, a few channels larger."""
    n, Hkv, D = shape[-3:]
    size = torch.exp2(torch.randn(n, Hkv, 1, device="cuda", generator=gen))
    channel = 1 + 7 * (torch.rand(Hkv, D, device="cuda", generator=gen) < 0.03)
    return (torch.randn(*shape, device="cuda", generator=gen) * (size * channel)).to(torch.bfloat16)


def _need(amax, fmt):
    """The scale that rows of this largest magnitude need, in the arithmetic of amax's type."""
    if fmt == "e4m3":
        m, e = torch.frexp(amax)  # amax = m * 2^e, 0.5 <= m < 1, and 448 = 0.875 * 2^9
        s = torch.exp2((e - 9 + (m > 0.875)).to(amax.dtype))
        return torch.where(amax > 0, s, 0).clamp(min=MIN_SCALE)
    m, e = torch.frexp(amax / torch.full_like(amax, 127))  # a division: times 1/127 would miss the borders
    return torch.ldexp(torch.ceil(m * 256) / 256, e).clamp(min=MIN_SCALE)


def _coded(x, fmt):
    """x (values over their scale) as codes."""
    if fmt == "e4m3":
        return x.to(torch.float8_e4m3fn)
    return torch.round(x).to(torch.int8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, n, Hkv, D, bt, fmt, Tcap = (case[x] for x in ("B", "n", "Hkv", "D", "bt", "fmt", "Tcap"))
    nb = -(-Tcap // bt)
    state = dict(case=case)
    for name in ("k", "v"):
        codes = torch.zeros(B, nb * bt, n, Hkv, D, dtype=DTYPES[fmt], device="cuda")
        scale = torch.zeros(B, Hkv, nb, n, device="cuda")
        for b in range(B):
            x = _rows(gen, (nb, bt, n, Hkv, D)).float()
            if case["op"] == "write":
                x[-(-case["first"] // bt):] = 0  # behind the sequence: not written yet
            s = _need(x.abs().amax(dim=(1, 4)), fmt)  # [nb, n, Hkv]
            codes[b] = _coded(x / s[:, None, :, :, None], fmt).view(nb * bt, n, Hkv, D)
            scale[b] = s.permute(2, 0, 1)
        state[name + "_codes"] = codes[:, :Tcap].contiguous().view(B, Tcap * n, Hkv, D)
        state[name + "_scale"] = scale
        del codes

    def ints(lo, hi):
        return torch.randint(lo, hi + 1, (B,), device="cuda", generator=gen).to(torch.int32)

    if case["op"] in ("write", "read"):
        L, first = case["L"], case["first"]
        offset = ints(max(0, first - 2 * bt), first) if case["ragged"] else ints(first, first)
        length = None
        if case["ragged"] and L > 1:
            length = ints(0, L)
            length[0] = L
        state |= dict(offset=offset, length=length)
        if case["op"] == "write":
            state |= dict(k=_rows(gen, (B, L, n, Hkv, D)).view(B, L * n, Hkv, D) * 2,
                          v=_rows(gen, (B, L, n, Hkv, D)).view(B, L * n, Hkv, D) * 2)
            start = offset // bt * bt  # the written blocks, from their first token on
            state |= dict(start=start.to(torch.int32), held=(offset - start + (L if length is None else length)).to(torch.int32))
        return state
    nq = n if case["op"] == "decode" else 1
    state["q"] = torch.randn(B, nq, case["Hq"], D, device="cuda", generator=gen).to(torch.bfloat16)
    state["seqlen"] = ints(1, case["T"] + 1) if case["ragged"] else ints(case["T"] + 1, case["T"] + 1)
    if case["ragged"]:
        state["seqlen"][0] = case["T"] + 1
    return state


# -------------------------------------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    return {"write": _write, "read": _read, "decode": _attend, "final": _attend}[case["op"]](state, case)


def _own(state, case):
    import structured_causal_attention_b200 as hd

    cache = hd.KVCacheQ8(state["k_codes"], state["v_codes"], state["k_scale"], state["v_scale"], case["n"], case["bt"])
    if case["op"] == "write":
        hd.kv_write_q8(state["k"], state["v"], cache, state["offset"], state["length"])
        k, v = hd.kv_read_q8(cache, _held_tokens(case), state["start"], state["held"])
        return dict(k=k, v=v, k_scale=cache.k_scale, v_scale=cache.v_scale)
    if case["op"] == "read":
        k, v = hd.kv_read_q8(cache, case["L"], state["offset"], state["length"])
        return dict(k=k, v=v)
    attend = hd.decode_attn_q8 if case["op"] == "decode" else hd.decode_attn_final_q8
    out, lse = attend(state["q"], cache, state["seqlen"], case["mode"], case["W"], case["D"] ** -0.5)
    return dict(out=out, lse=lse)


def _held_tokens(case):
    """Tokens that are read back of a sequence after a write: its new ones and those before them in their block."""
    return case["L"] + case["bt"] - 1


def _tokens(start, count, Tcap):
    """Token numbers [B, count] from start[b] on, and the same with those behind the cache moved to its last."""
    tok = start.long()[:, None] + torch.arange(count, device=start.device)
    return tok, tok.clamp(max=Tcap - 1)


def _values(codes, scale, start, held, count, case):
    """bf16 [B, count*n, Hkv, D]: `held[b]` tokens from start[b] on, as the cache holds them; zeros behind them."""
    B, n, Hkv, D, bt, Tcap = (case[x] for x in ("B", "n", "Hkv", "D", "bt", "Tcap"))
    tok, at = _tokens(start, count, Tcap)
    rows = torch.arange(B, device=codes.device)[:, None]
    x = codes.view(B, Tcap, n, Hkv, D).view(torch.uint8)[rows, at].view(codes.dtype).float()
    s = scale.permute(0, 2, 3, 1)[rows, at // bt]  # [B, count, n, Hkv]
    x = x * s[..., None]
    if held is not None:
        x = x * (tok < (start + held).long()[:, None])[:, :, None, None, None]
    return x.to(torch.bfloat16).view(B, count * n, Hkv, D)


def _read(state, case):
    return {name: _values(state[name + "_codes"], state[name + "_scale"], state["offset"], state["length"], case["L"], case)
            for name in ("k", "v")}


def _write(state, case):
    out = {}
    for name in ("k", "v"):
        _write_one(state[name], state[name + "_codes"], state[name + "_scale"], state, case)
        out[name] = _values(state[name + "_codes"], state[name + "_scale"], state["start"], state["held"], _held_tokens(case), case)
        out[name + "_scale"] = state[name + "_scale"]
    return out


def _write_one(x, codes, scale, state, case):
    B, n, Hkv, D, bt, L, Tcap, fmt = (case[c] for c in ("B", "n", "Hkv", "D", "bt", "L", "Tcap", "fmt"))
    offset, dev = state["offset"].long()[:, None], x.device
    length = L if state["length"] is None else state["length"].long()[:, None]
    count = -(-(L + bt - 1) // bt)  # blocks that L tokens can touch, wherever they begin
    start = state["start"]
    tok, _ = _tokens(start, count * bt, Tcap)  # the cache is long enough for all of them
    rows = torch.arange(B, device=dev)[:, None]
    blocks = start.long()[:, None] // bt + torch.arange(count, device=dev)
    source = tok - offset
    new = (source >= 0) & (source < length)
    fresh = x.view(B, L, n, Hkv, D)[rows, source.clamp(0, L - 1)].float() * new[:, :, None, None, None]
    need = _need(fresh.view(B, count, bt, n, Hkv, D).abs().amax(dim=(2, 5)), fmt)  # [B, count, n, Hkv]
    before = scale.permute(0, 2, 3, 1)[rows, blocks]
    begun = (blocks * bt < offset)[:, :, None, None]
    touched = new.view(B, count, bt).any(dim=2)[:, :, None, None]
    after = torch.where(begun, torch.maximum(before, need), need)
    after = torch.where(touched, after, before)
    wide = after.repeat_interleave(bt, dim=1)[..., None]
    was = before.repeat_interleave(bt, dim=1)[..., None]
    old = codes.view(B, Tcap, n, Hkv, D).view(torch.uint8)[rows, tok].view(codes.dtype)
    again = _coded(old.float() * was / wide.clamp(min=MIN_SCALE), fmt)
    kept = torch.where((tok < offset)[:, :, None, None, None], again.view(torch.uint8), old.view(torch.uint8))
    coded = _coded(fresh / wide.clamp(min=MIN_SCALE), fmt).view(torch.uint8)
    codes.view(B, Tcap, n, Hkv, D).view(torch.uint8)[rows, tok] = torch.where(new[:, :, None, None, None], coded, kept)
    scale.permute(0, 2, 3, 1)[rows, blocks] = after


def _attend(state, case):
    B, n, Hq, Hkv, D, bt, Tcap, mode, W = (case[x] for x in ("B", "n", "Hq", "Hkv", "D", "bt", "Tcap", "mode", "W"))
    q, dev = state["q"], state["q"].device
    nq, g = q.shape[1], Hq // Hkv
    pos = torch.arange(Tcap * n, device=dev)

    def wide(codes, scale):
        return codes.float().mul_(scale[:, :, pos // (n * bt), pos % n].transpose(1, 2)[..., None])

    rows = q.float().view(B, nq, Hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, nq * g, D)
    s = torch.matmul(rows, wide(state["k_codes"], state["k_scale"]).permute(0, 2, 3, 1)).mul_(D ** -0.5)
    at = (state["seqlen"].long() - 1)[:, None] * n + torch.arange(n - nq, n, device=dev)  # the queries' positions [B, nq]
    shown = pos <= at[..., None]
    if mode == INTRA:
        shown &= pos % n == (at % n)[..., None]
    if mode == CROSS_WINDOW:
        shown &= at[..., None] - pos < n * W
    s = s.view(B, Hkv, nq, g, Tcap * n).masked_fill_(~shown[:, None, :, None, :], -math.inf)
    top = s.amax(dim=-1, keepdim=True)
    p = s.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, nq * g, Tcap * n), wide(state["v_codes"], state["v_scale"]).transpose(1, 2))
    o = o.view(B, Hkv, nq, g, D) / total
    lse = (top + total.log())[..., 0]  # [B, Hkv, nq, g]
    return dict(out=o.permute(0, 2, 1, 3, 4).reshape(B, nq, Hq, D).to(torch.bfloat16),
                lse=lse.permute(0, 1, 3, 2).reshape(B, Hq, nq))


# ----------------------------------------------------------------------------- the work of one pass

def work(case):
    B, n, Hkv, D, bt = (case[x] for x in ("B", "n", "Hkv", "D", "bt"))
    ragged = 0.5 if case["ragged"] else 1.0  # lengths are drawn evenly; the first sequence has the full one
    if case["op"] in ("write", "read"):
        L = case["L"]
        tokens = L + (B - 1) * (max(1, L * ragged) if L > 1 else L)
        values = tokens * n * Hkv * D * 2  # of K and V
        scales = tokens / bt * n * Hkv * 2 * 4
        if case["op"] == "read":
            return dict(bytes=int(3 * values + scales), flops=int(values))
        back = values + (bt / 2 if case["first"] else 0) * B * n * Hkv * D * 2  # what is read back
        return dict(bytes=int(3 * values + scales + 2 * back), flops=int(3 * values))
    T, Hq, mode, W = case["T"] + 1, case["Hq"], case["mode"], case["W"]
    nq = n if case["op"] == "decode" else 1
    tokens = T + (B - 1) * T * ragged
    if mode == CROSS_WINDOW:
        full = min(1.0, W / T)
        tokens = min(T, W) + (B - 1) * T * ((full - full * full / 2) if case["ragged"] else full)
    held = tokens * n if case["op"] == "decode" or mode != INTRA else tokens  # positions that are read
    seen = held if mode != INTRA else tokens  # keys of one query
    return dict(bytes=int(2 * held * Hkv * (D + 4 / bt) + 2 * 2 * B * nq * Hq * D + 4 * B * nq * Hq + 4 * B),
                flops=int(4 * seen * nq * Hq * D))


# --------------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] in ("write", "read"):
        return _exact_rows(state, case)
    return _exact_attention(state, case)


def _near8(x, fmt):
    """float64 values over their scale, at the nearest that 8 bits hold (ties to even)."""
    if fmt == "int8":
        return torch.round(x)
    tiny = x.abs().clamp(min=2.0 ** -6)
    step = torch.exp2(torch.floor(torch.log2(tiny)) - 3)
    return torch.round(x / step) * step


def _exact_scale(most, fmt):
    """The scale for a largest magnitude, from its definition, as Python does it."""
    if most == 0:
        return MIN_SCALE
    if fmt == "e4m3":
        s = 2.0 ** (math.frexp(most)[1] - 10)
        while most > 448 * s:
            s *= 2
        return max(s, MIN_SCALE)
    unit = 2.0 ** (math.frexp(most / 127)[1] - 8)  # one step of 8 significant bits
    whole = math.floor(most / 127 / unit)
    while whole * unit * 127 < most:
        whole += 1
    return max(whole * unit, MIN_SCALE)


def _exact_rows(state, case):
    B, n, Hkv, D, bt, L, Tcap, fmt = (case[x] for x in ("B", "n", "Hkv", "D", "bt", "L", "Tcap", "fmt"))
    nb = -(-Tcap // bt)
    if case["op"] == "write" and B * n * Hkv * (L // bt + 2) > 400_000:
        return None  # block by block, this would take too long
    offset = state["offset"].tolist()
    length = [L] * B if state["length"] is None else state["length"].tolist()
    out = {}
    for name in ("k", "v"):
        codes = state[name + "_codes"].view(B, Tcap, n, Hkv, D).to(torch.float64)
        scale = state[name + "_scale"].to(torch.float64).permute(0, 2, 3, 1).clone()  # [B, nb, n, Hkv]
        if case["op"] == "write":
            x = state[name].view(B, L, n, Hkv, D).to(torch.float64)
            for b in range(B):
                t0, t1 = offset[b], offset[b] + length[b]
                for j in range(t0 // bt, -(-t1 // bt) if t1 > t0 else 0):
                    lo, hi = max(t0, j * bt), min(t1, (j + 1) * bt)
                    rows = x[b, lo - t0:hi - t0]
                    most = rows.abs().amax(dim=(0, 3)).tolist()  # [n][Hkv]
                    s = torch.tensor([[_exact_scale(m, fmt) for m in r] for r in most], dtype=torch.float64, device=x.device)
                    if j * bt < t0:
                        old = scale[b, j].clone()
                        s = torch.maximum(s, old)
                        codes[b, j * bt:t0] = _near8(codes[b, j * bt:t0] * old[..., None] / s[..., None], fmt)
                    scale[b, j] = s
                    codes[b, lo:hi] = _near8(rows / s[..., None], fmt)
            start, held, count = state["start"].tolist(), state["held"].tolist(), _held_tokens(case)
            out[name + "_scale"] = scale.permute(0, 3, 1, 2)
        else:
            start, held, count = offset, length, L
        back = torch.zeros(B, count, n, Hkv, D, dtype=torch.float64, device=codes.device)
        for b in range(B):
            at = torch.arange(start[b], start[b] + held[b], device=codes.device)
            back[b, :held[b]] = codes[b, at] * scale[b, at // bt][..., None]
        out[name] = back.view(B, count * n, Hkv, D)
        del codes
    assert nb == state["k_scale"].shape[2]
    return out


def _exact_attention(state, case):
    B, n, Hq, Hkv, D, bt, mode, W = (case[x] for x in ("B", "n", "Hq", "Hkv", "D", "bt", "mode", "W"))
    q = state["q"].to(torch.float64)
    nq, g, dev = q.shape[1], Hq // Hkv, q.device
    out = torch.zeros(B, nq, Hq, D, dtype=torch.float64, device=dev)
    lse = torch.zeros(B, Hq, nq, dtype=torch.float64, device=dev)
    for b, tokens in enumerate(state["seqlen"].tolist()):
        for s in range(nq):
            stream = s + n - nq
            p = (tokens - 1) * n + stream
            at = torch.arange(max(0, p - n * W + 1) if mode == CROSS_WINDOW else 0, p + 1, device=dev)
            if mode == INTRA:
                at = at[at % n == stream]
            for h in range(Hkv):
                ks = state["k_scale"][b, h, at // n // bt, at % n].to(torch.float64)
                vs = state["v_scale"][b, h, at // n // bt, at % n].to(torch.float64)
                k, v = (state[x][b, :, h].view(torch.uint8)[at].view(state[x].dtype).to(torch.float64) * y[:, None]
                        for x, y in (("k_codes", ks), ("v_codes", vs)))
                score = q[b, s, h * g:(h + 1) * g] @ k.T / math.sqrt(D)
                lse[b, h * g:(h + 1) * g, s] = torch.logsumexp(score, dim=1)
                out[b, s, h * g:(h + 1) * g] = torch.softmax(score, dim=1) @ v
    return dict(out=out, lse=lse)
