"""An attention layer for serving, composed from the library's calls: NVFP4
projections around attention over an NVFP4 key/value cache.

  qkv = x Wqkv^T       the NVFP4 linear layer's forward (linear.fprop)
  q, cache <- qkv      nvfp4_kv_append: the queries and keys rotated, keys and
                       values quantized into the cache's pages, one launch
  o = attention(q)     nvfp4_kv_attention over the cache
  y = o Wo^T           linear.fprop

The same call takes a decode step (one token of each sequence), several
drafted tokens of each, a prompt, a chunk of one, or a mixture (cu_q; every
sequence then takes the kernel that max_q asks for, so that prompts and single
tokens go faster in calls of their own). The four steps run in the library's
kernels; around them torch fills and copies x and o up to a multiple of 16
tokens where they are not one, and finds seq where it is not given. What a serving program keeps between calls is made once: the weights
(layer_weights), the cache (nvfp4_kv_cache), the rotation table
(nvfp4_rope_table) and two workspaces (nvfp4_workspace, nvfp4_kv_workspace).
"""
from __future__ import annotations

from . import _torch, nvfp4_kv_append, nvfp4_kv_attention, nvfp4_workspace
from .linear import fprop, quantize_weight


def layer_weights(wqkv, wo, stream=None) -> dict:
    """Wqkv [(heads + 2 kv_heads) head_dim][hidden] (the queries' rows, the
    keys', the values') and Wo [hidden][heads head_dim], bf16 -> NVFP4."""
    return {"qkv": quantize_weight(wqkv, stream=stream), "out": quantize_weight(wo, stream=stream)}


def _rows16(x):
    """x [tokens][n] with zero rows up to a multiple of 16 tokens, which the
    NVFP4 GEMM takes."""
    tokens, n = x.shape
    if tokens % 16 == 0:
        return x
    padded = x.new_zeros((tokens + 15) // 16 * 16, n)
    padded[:tokens] = x
    return padded


def _sequences(seq, cu_q, max_q, tokens, batch, device):
    """Each token's sequence as nvfp4_kv_append takes it, by what the attention
    takes the tokens for: max_q of each sequence, or cu_q's."""
    torch = _torch()
    if cu_q is not None and max_q is None:
        raise ValueError("cu_q needs max_q, the most tokens of one sequence")
    if seq is not None or (max_q in (None, 1) and (cu_q is None or tokens == batch)):
        return seq  # without it, one of each
    at = torch.arange(tokens, dtype=torch.int32, device=device)
    if cu_q is None:
        return at // max_q
    return torch.bucketize(at, cu_q[1:], out_int32=True, right=True)


def attention_layer(x, weights: dict, cache: dict, positions, page_table, lens, table, kv_workspace, heads: int,
                    seq=None, cu_q=None, max_q: int | None = None, interleaved: bool = False, causal: bool = True,
                    window: int = 0, ws=None, stream=None):
    """y [tokens][hidden] (bf16) from x [tokens][hidden] (bf16); the tokens'
    keys and values join the cache. Token t is token positions[t] of sequence
    seq[t] (None: found from cu_q or max_q, by a torch kernel or two where a
    sequence may have more than one; a program that runs many layers gives it);
    lens holds the sequences' lengths with these
    tokens, cu_q where each sequence's tokens begin, at most max_q of each
    (None: max_q, 1 by default, of each)."""
    torch = _torch()
    kv_heads, head_dim = cache["data"].shape[1], cache["data"].shape[3] // 18
    tokens = x.shape[0]
    with torch.cuda.stream(stream) if stream is not None else torch.cuda.device(x.device):
        seq = _sequences(seq, cu_q, max_q, tokens, page_table.shape[0], x.device)
        ws = nvfp4_workspace(x.device) if ws is None else ws
        qkv = fprop(_rows16(x), weights["qkv"], ws=ws, out_dtype=torch.bfloat16)[:tokens]
        qkv = qkv.view(tokens, heads + 2 * kv_heads, head_dim)
        q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
        nvfp4_kv_append(cache, k, v, positions, page_table, seq=seq, table=table, interleaved=interleaved, q=q, q_out=q)
        o = nvfp4_kv_attention(q, cache, page_table, lens, kv_workspace, cu_q=cu_q, max_q=max_q, causal=causal,
                               window=window)
        y = fprop(_rows16(o.view(tokens, heads * head_dim)), weights["out"], ws=ws, out_dtype=torch.bfloat16)
    return y[:tokens]
