"""Hidden Decoding hot path on B200: a C-ABI CUDA library and its Python binding.

The library (``libhd.so``, built from ``csrc/`` by ``build.py``) implements the
data-parallel hot path of Hidden Decoding with Stream-Factorized Attention
(page "微信WeLM提出Hidden Decoding：大模型推理新范式", tahou.com):

* ``hd_expand_embed``  interleaved n-table embedding gather (stream k of token i
  at position (i-1)n+k);
* ``hd_rope_expanded``  rotary position embedding of q and k at the physical
  positions p = t*n + s (continuous positions over the expanded sequence);
* ``hd_final_readout`` / ``hd_lm_head_ce``  the final stream's hidden rows and the
  LM-head cross-entropy on them (the only supervised stream), logits never
  materialised;
* ``hd_attn_fwd`` / ``hd_attn_bwd``  attention over the expanded sequence with
  intra-stream, cross-stream full-causal and cross-stream sliding-window masks,
  optionally with final-stream-only queries (KV-mirror);
* ``hd_decode_attn_final``  the final stream's query alone (KV-mirror layers);
* ``hd_decode_attn``  the n stream queries of a new token against the
  interleaved per-stream KV cache;
* ``hd_kv_write_q8`` / ``hd_kv_read_q8``  an 8-bit KV cache (e4m3 or int8, a scale
  for each block of tokens, stream and head): quantised as it is written, read
  back as bf16;
* ``hd_decode_attn_q8`` / ``hd_decode_attn_final_q8``  the decode steps against it.

The C names are re-exported from ``_lib`` (pointer + size arguments). The
tensor helpers below (``expand_embed``, ``rope_``, ``attn_fwd``, ``attn_bwd``,
``decode_attn``, ``decode_attn_final``, and those of the 8-bit cache) allocate outputs and workspace with
torch and call the same C entry points; torch is used for device memory and streams only.
"""
from __future__ import annotations

import functools
from typing import Any, NamedTuple

from ._lib import (  # noqa: F401
    HD_ERR_CUDA,
    HD_ERR_DEVICE_INDEX,
    HD_ERR_INVALID_ARG,
    HD_ERR_TIMEOUT,
    HD_ERR_UNSUPPORTED,
    HD_OK,
    HD_Q8_E4M3,
    HD_Q8_INT8,
    HDError,
    hd_attn_bwd,
    hd_attn_bwd_workspace_bytes,
    hd_attn_fwd,
    hd_decode_attn,
    hd_decode_attn_final,
    hd_decode_attn_final_q8,
    hd_decode_attn_noalloc,
    hd_decode_attn_q8,
    hd_decode_final_q8_workspace_bytes,
    hd_decode_final_workspace_bytes,
    hd_decode_q8_workspace_bytes,
    hd_decode_workspace_bytes,
    hd_device_status,
    hd_expand_embed,
    hd_final_readout,
    hd_kv_read_q8,
    hd_kv_write_q8,
    hd_lm_head_ce,
    hd_lm_head_ce_bwd,
    hd_lm_head_ce_bwd_workspace_bytes,
    hd_lm_head_ce_workspace_bytes,
    hd_rope_expanded,
    hd_selftest_wait_timeout,
    lib,
    status_string,
)

INTRA, CROSS_FULL, CROSS_WINDOW = 0, 1, 2


def _need_cuda(*ts):
    for t in ts:
        if not t.is_cuda:
            raise ValueError("tensors must live on a CUDA device (the library has no CPU path)")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def expand_embed(ids, tables, stream=None):
    """ids int32 [B, L], tables [n, V, d] -> out [B, L*n, d] (tables' dtype)."""
    import torch

    _need_cuda(ids, tables)
    B, L = ids.shape
    n, V, d = tables.shape
    out = torch.empty((B, L * n, d), dtype=tables.dtype, device=tables.device)
    hd_expand_embed(ids, tables, out, B, L, n, V, d, tables.element_size(), stream)
    return out


def rope_(q, k, n, final_only=False, base=10000.0, token_offset=None, stream=None):
    """Rotate q [B, Sq, Hq, D] and k [B, n*L, Hkv, D] bf16 in place at their physical positions.

    Either may be None. ``token_offset`` (int32 [B] on the device) gives the
    tokens that precede the rows of each sequence. Returns (q, k).
    """
    ts = [t for t in (q, k, token_offset) if t is not None]
    _need_cuda(*ts)
    ref = k if k is not None else q
    B, D = ref.shape[0], ref.shape[-1]
    if k is not None:
        L = k.shape[1] // n
    else:
        L = q.shape[1] if final_only else q.shape[1] // n
    Hq = q.shape[2] if q is not None else 0
    Hkv = k.shape[2] if k is not None else 0
    hd_rope_expanded(q, k, token_offset, B, L, n, Hq, Hkv, D, final_only, base, stream)
    return q, k


def attn_fwd(q, k, v, n, mode, W=0, final_only=False, scale=None, stream=None):
    """q [B, Sq, Hq, D], k/v [B, n*L, Hkv, D] bf16 -> (out bf16 like q, lse fp32 [B, Hq, Sq])."""
    import torch

    _need_cuda(q, k, v)
    B, S, Hkv, D = k.shape
    L = S // n
    Hq = q.shape[2]
    if scale is None:
        scale = D ** -0.5
    out = torch.empty_like(q)
    lse = torch.empty((B, Hq, q.shape[1]), dtype=torch.float32, device=q.device)
    hd_attn_fwd(q, k, v, out, lse, B, L, n, Hq, Hkv, D, mode, W, final_only, scale, stream)
    return out, lse


def attn_bwd(q, k, v, out, lse, dout, n, mode, W=0, final_only=False, scale=None, stream=None,
             workspace=None):
    """Gradients (dq, dk, dv) in bf16; the fp32 workspace is allocated if not given."""
    import torch

    _need_cuda(q, k, v, out, lse, dout)
    B, S, Hkv, D = k.shape
    L = S // n
    Hq = q.shape[2]
    if scale is None:
        scale = D ** -0.5
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    nbytes = hd_attn_bwd_workspace_bytes(B, L, n, Hq, Hkv, D, final_only)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    hd_attn_bwd(q, k, v, out, lse, dout, dq, dk, dv, B, L, n, Hq, Hkv, D, mode, W, final_only, scale,
                workspace, workspace.numel() * workspace.element_size(), stream)
    return dq, dk, dv


def decode_attn(q, k_cache, v_cache, seqlen, mode, W=0, scale=None, stream=None, workspace=None):
    """q [B, n, Hq, D]; caches [B, Tcap*n, Hkv, D]; seqlen int32 [B] (tokens incl. the new one)."""
    import torch

    _need_cuda(q, k_cache, v_cache, seqlen)
    B, n, Hq, D = q.shape
    Hkv = k_cache.shape[2]
    Tcap = k_cache.shape[1] // n
    if scale is None:
        scale = D ** -0.5
    out = torch.empty_like(q)
    lse = torch.empty((B, Hq, n), dtype=torch.float32, device=q.device)
    nbytes = hd_decode_workspace_bytes(B, n, Tcap, Hq, Hkv, D)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    hd_decode_attn(q, k_cache, v_cache, seqlen, out, lse, B, n, Tcap, Hq, Hkv, D, mode, W, scale,
                   workspace, workspace.numel() * workspace.element_size(), stream)
    return out, lse


def decode_attn_final(q, k_cache, v_cache, seqlen, n, mode, W=0, scale=None, stream=None,
                      workspace=None):
    """q [B, 1, Hq, D] (stream n-1 of the new token); caches [B, Tcap*n, Hkv, D]; seqlen int32 [B].

    Returns (out [B, 1, Hq, D] bf16, lse [B, Hq, 1] fp32).
    """
    import torch

    _need_cuda(q, k_cache, v_cache, seqlen)
    B, one, Hq, D = q.shape
    if one != 1:
        raise ValueError("q must be [B, 1, Hq, D]")
    Hkv = k_cache.shape[2]
    Tcap = k_cache.shape[1] // n
    if scale is None:
        scale = D ** -0.5
    out = torch.empty_like(q)
    lse = torch.empty((B, Hq, 1), dtype=torch.float32, device=q.device)
    nbytes = hd_decode_final_workspace_bytes(B, n, Tcap, Hq, Hkv, D)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    hd_decode_attn_final(q, k_cache, v_cache, seqlen, out, lse, B, n, Tcap, Hq, Hkv, D, mode, W,
                         scale, workspace, workspace.numel() * workspace.element_size(), stream)
    return out, lse


def final_readout(x, n, stream=None):
    """x [B, n*L, d] -> the final stream's rows [B, L, d] (positions t*n + n-1)."""
    import torch

    _need_cuda(x)
    B, S, d = x.shape
    L = S // n
    out = torch.empty((B, L, d), dtype=x.dtype, device=x.device)
    hd_final_readout(x, out, B, L, n, d, x.element_size(), stream)
    return out


def lm_head_ce(x, w, labels, n, stream=None, workspace=None):
    """x bf16 [B, n*L, d], w bf16 [V, d], labels int32 [B, L] -> (loss, lse) fp32 [B, L]."""
    import torch

    _need_cuda(x, w, labels)
    B, S, d = x.shape
    L = S // n
    V = w.shape[0]
    loss = torch.empty((B, L), dtype=torch.float32, device=x.device)
    lse = torch.empty((B, L), dtype=torch.float32, device=x.device)
    nbytes = hd_lm_head_ce_workspace_bytes(B, L, V)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    hd_lm_head_ce(x, w, labels, loss, lse, B, L, n, d, V, workspace,
                  workspace.numel() * workspace.element_size(), stream)
    return loss, lse


def lm_head_ce_bwd(x, w, labels, lse, n, grad_scale=1.0, stream=None, workspace=None):
    """Gradients of sum(loss) * grad_scale: (dh bf16 [B, L, d], dw fp32 [V, d])."""
    import torch

    _need_cuda(x, w, labels, lse)
    B, S, d = x.shape
    L = S // n
    V = w.shape[0]
    dh = torch.empty((B, L, d), dtype=torch.bfloat16, device=x.device)
    dw = torch.empty((V, d), dtype=torch.float32, device=x.device)
    nbytes = hd_lm_head_ce_bwd_workspace_bytes(B, L, V)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    hd_lm_head_ce_bwd(x, w, labels, lse, grad_scale, dh, dw, B, L, n, d, V, workspace,
                      workspace.numel() * workspace.element_size(), stream)
    return dh, dw


class KVCacheQ8(NamedTuple):
    """An 8-bit KV cache: codes [B, Tcap*n, Hkv, D], float8_e4m3fn or int8 (the format), and fp32 scales
    [B, Hkv, ceil(Tcap / block_tokens), n]. ``kv_cache_q8`` makes one. Other contiguous tensors of these shapes do
    where their storage starts on 16-byte boundaries, with scales of 0 (any, where each block is written from its
    first token on): a write that enters a block behind its first token goes by the scale that it finds."""

    k: Any
    v: Any
    k_scale: Any
    v_scale: Any
    n: int
    block_tokens: int


def kv_cache_q8(B, Tcap, n, Hkv, D, dtype, block_tokens=16, device="cuda"):
    """An empty 8-bit cache for ``Tcap`` tokens; ``dtype`` is torch.float8_e4m3fn or torch.int8."""
    import torch

    if min(B, Tcap, n, Hkv, D, block_tokens) < 1:
        raise ValueError("sizes and block_tokens must be positive")
    if dtype not in (torch.float8_e4m3fn, torch.int8):
        raise ValueError("dtype must be float8_e4m3fn or int8")
    k, v = (torch.zeros((B, Tcap * n, Hkv, D), dtype=dtype, device=device) for _ in range(2))
    k_scale, v_scale = (torch.zeros((B, Hkv, -(-Tcap // block_tokens), n), dtype=torch.float32, device=device)
                        for _ in range(2))
    return KVCacheQ8(k, v, k_scale, v_scale, n, block_tokens)


def _cache_q8(cache):
    """(B, Tcap, Hkv, D, format) of a KVCacheQ8, its tensors checked against one another."""
    import torch

    k, v, k_scale, v_scale, n, block_tokens = cache
    _need_cuda(k, v, k_scale, v_scale)
    if v.dtype != k.dtype or k.dtype not in (torch.float8_e4m3fn, torch.int8):
        raise ValueError("codes must be float8_e4m3fn or int8, k and v alike")
    shape = k.shape
    if n < 1 or block_tokens < 1 or len(shape) != 4 or shape[1] % n:
        raise ValueError("codes must be [B, Tcap*n, Hkv, D]")
    B, S, Hkv, D = shape
    Tcap = S // n
    want = (B, Hkv, -(-Tcap // block_tokens), n)
    if v.shape != shape or k_scale.shape != want or v_scale.shape != want:
        raise ValueError(f"k and v must be alike and the scales {list(want)}")
    if k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32:
        raise ValueError("scales must be float32")
    return B, Tcap, Hkv, D, HD_Q8_E4M3 if k.dtype == torch.float8_e4m3fn else HD_Q8_INT8


def _call_on(ts, call, *args):
    """call(*args) with the one device of the tensors ``ts`` (``None`` among them is passed over) current."""
    import torch

    index = ts[0].get_device()
    for t in ts:
        if t is not None and t.get_device() != index:
            raise ValueError("tensors must live on one device")
    if index == torch.cuda.current_device():
        return call(*args)
    with torch.cuda.device(index):
        return call(*args)


def _within(stream, device):
    """``stream`` (a torch stream or a handle) as the current one: a context. What is allocated in it is the
    stream's own, so that no other stream is given the memory while the stream's kernels use it."""
    import torch

    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError("the stream must be of the tensors' device")
    return torch.cuda.stream(stream)


def _index_q8(t, B, what):
    import torch

    if t is not None:
        _need_cuda(t)
        if t.dtype != torch.int32 or t.shape != (B,):
            raise ValueError(f"{what} must be int32 [B]")


def kv_write_q8(k, v, cache, token_offset=None, lengths=None, stream=None):
    """Quantise k, v bf16 [B, L*n, Hkv, D] into ``cache`` (a KVCacheQ8) from token ``token_offset[b]`` on
    (int32 [B]; None: 0). ``lengths`` (int32 [B]) gives the tokens of each sequence in a padded batch. What the last
    written block holds behind the written tokens no longer counts: to replace a token, write those behind it in its
    block again too."""
    import torch

    _need_cuda(k, v)
    B, Tcap, Hkv, D, fmt = _cache_q8(cache)
    if stream is not None:
        with _within(stream, k.device):
            return kv_write_q8(k, v, cache, token_offset, lengths)
    if k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16:
        raise ValueError("k and v must be bfloat16")
    shape = k.shape
    L = shape[1] // cache.n if len(shape) == 4 else 0
    if shape != (B, L * cache.n, Hkv, D) or v.shape != shape:
        raise ValueError(f"k and v must be [{B}, L*{cache.n}, {Hkv}, {D}]")
    _index_q8(token_offset, B, "token_offset")
    _index_q8(lengths, B, "lengths")
    codes = cache[:4]
    if L:
        _call_on((*codes, k, v, token_offset, lengths), hd_kv_write_q8, k, v, token_offset, lengths, *codes, B, L,
                 cache.n, Tcap, Hkv, D, fmt, cache.block_tokens)


def kv_read_q8(cache, L, token_offset=None, lengths=None, out=None, stream=None):
    """(k, v) bf16 [B, L*n, Hkv, D]: ``L`` tokens of each sequence from ``token_offset[b]`` on, or the first
    ``lengths[b]`` of them and zeros behind. ``out``: two buffers to use."""
    import torch

    B, Tcap, Hkv, D, fmt = _cache_q8(cache)
    if stream is not None:
        with _within(stream, cache.k.device):
            return kv_read_q8(cache, L, token_offset, lengths, out)
    _index_q8(token_offset, B, "token_offset")
    _index_q8(lengths, B, "lengths")
    shape = (B, L * cache.n, Hkv, D)
    if out is None:
        out = cache.k.new_empty(shape, dtype=torch.bfloat16), cache.k.new_empty(shape, dtype=torch.bfloat16)
    k, v = out
    _need_cuda(k, v)
    if k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16 or k.shape != shape or v.shape != shape:
        raise ValueError(f"out must be two bfloat16 tensors {list(shape)}")
    codes = cache[:4]
    if L:
        _call_on((*codes, token_offset, lengths, k, v), hd_kv_read_q8, *codes, token_offset, lengths, k, v, B, L,
                 cache.n, Tcap, Hkv, D, fmt, cache.block_tokens)
    return k, v


def _decode_q8(q, cache, seqlen, mode, W, scale, stream, workspace, final):
    import torch

    _need_cuda(q, seqlen)
    if stream is not None:
        with _within(stream, q.device):
            return _decode_q8(q, cache, seqlen, mode, W, scale, None, workspace, final)
    B, Tcap, Hkv, D, fmt = _cache_q8(cache)
    n = cache.n
    nq = 1 if final else n
    shape = q.shape
    Hq = shape[2] if len(shape) == 4 else 0
    if q.dtype != torch.bfloat16 or shape != (B, nq, Hq, D):
        raise ValueError(f"q must be bfloat16 [{B}, {nq}, Hq, {D}]")
    _index_q8(seqlen, B, "seqlen")
    if workspace is not None:
        _need_cuda(workspace)
    if scale is None:
        scale = D ** -0.5
    out = torch.empty_like(q)
    lse = q.new_empty((B, Hq, nq), dtype=torch.float32)
    if workspace is None:
        workspace = q.new_empty(_decode_q8_bytes(q.get_device(), final, B, n, Tcap, Hq, Hkv, D), dtype=torch.uint8)
    codes = cache[:4]
    _call_on((q, *codes, seqlen, workspace), hd_decode_attn_final_q8 if final else hd_decode_attn_q8, q, *codes, seqlen,
             out, lse, B, n, Tcap, Hq, Hkv, D, fmt, cache.block_tokens, mode, W, scale, workspace,
             workspace.numel() * workspace.element_size())
    return out, lse


@functools.lru_cache(maxsize=256)
def _decode_q8_bytes(index, final, *sizes):
    """The workspace's size on device ``index`` (it goes by the sizes and the number of its SMs)."""
    import torch

    with torch.cuda.device(index):
        return (hd_decode_final_q8_workspace_bytes if final else hd_decode_q8_workspace_bytes)(*sizes)


def decode_attn_q8(q, cache, seqlen, mode, W=0, scale=None, stream=None, workspace=None):
    """decode_attn against a KVCacheQ8: q bf16 [B, n, Hq, D]; seqlen int32 [B] (tokens incl. the new one)."""
    return _decode_q8(q, cache, seqlen, mode, W, scale, stream, workspace, False)


def decode_attn_final_q8(q, cache, seqlen, mode, W=0, scale=None, stream=None, workspace=None):
    """decode_attn_final against a KVCacheQ8: q bf16 [B, 1, Hq, D] (stream n-1 of the new token)."""
    return _decode_q8(q, cache, seqlen, mode, W, scale, stream, workspace, True)
