"""NVFP4 key/value cache: rotary positions, appending, reading back and
attention over the cache (include/nvfp4_kv.h).

Argument marshalling only, as in the package's other calls: every step runs
in the HIP kernels, outputs are allocated with torch.empty (on the stream
given), and there is no fallback. Tensors of heads are [tokens][heads]
[head_dim] and may be views (of a fused projection's output, say) as long as
head_dim is contiguous and every token and head starts on 16 bytes.

A cache is a dict: "data", uint8 [num_pages][kv_heads][page_size / 16]
[18 * head_dim], and "k_amax", "v_amax", float32 [1]; nvfp4_kv_cache makes
one.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

from . import BF16, F32, Nvfp4Error, _check, _device, _torch, lib

F16 = 2  # a dtype beside F32 and BF16
KV_WORKSPACE_BYTES = 64 << 20
_INTERLEAVED, _ADJOINT, _CAUSAL = 0x1, 0x2, 0x1
_SCALINGS = {None: 0, "linear": 1, "base": 2, "parts": 3}


def bind(L):
    """Argument types of the calls declared in include/nvfp4_kv.h."""
    P, I64, U32, I, D, F = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32, ctypes.c_int, ctypes.c_double,
                            ctypes.c_float)
    cache = [I64, I64, I64, I64, P, P]  # num_pages, kv_heads, page_size, head_dim, k_amax, v_amax
    L.nvfp4_rope_table.argtypes = [I64, I64, D, I, D, D, D, D, D, P, P]
    L.nvfp4_rope.argtypes = [P, I, I64, I64, I64, I64, I64, P, P, I64, I64, U32, P, I64, I64, P]
    L.nvfp4_kv_append.argtypes = [P, P, I, I64, I64, I64, P, P, I64, I64, I64, I64, I64, P, P, P, I64, I64, P, I64,
                                  I64, U32, P, *cache, P]
    L.nvfp4_kv_read.argtypes = [P, *cache, I64, P, P, P, I64, I64, P, P, I, P]
    L.nvfp4_kv_attention.argtypes = [P, I, I64, I64, I64, I64, P, I64, P, *cache, P, I64, I64, P, F, I64, U32, P, P,
                                     P, P]
    for name in ("nvfp4_rope_table", "nvfp4_rope", "nvfp4_kv_append", "nvfp4_kv_read", "nvfp4_kv_attention"):
        getattr(L, name).restype = I


# --------------------------------------------------------------- marshalling
#
# A decode step's kernels take a few microseconds, so the checks are kept to
# a few attribute reads where nothing is wrong; what is wrong is found out
# after that.

class _Names:
    """torch's names that the checks use, looked up once."""

    def __init__(self):
        torch = _torch()
        self.torch, self.Tensor, self.empty, self.empty_like = torch, torch.Tensor, torch.empty, torch.empty_like
        self.int32, self.uint8, self.f32 = torch.int32, torch.uint8, torch.float32
        self.dtypes = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
        # (the tensors that are asked about it are on the GPU: it is initialised)
        self.device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        # the stream's handle without a Stream object around it, where torch has that
        self.stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)


_names = None


def _n() -> _Names:
    global _names
    if _names is None:
        _names = _Names()
    return _names


def _like(n, t, shape):
    """An uninitialised contiguous tensor of t's dtype and shape (given), on
    its device."""
    out = n.empty_like(t)
    return out if out.is_contiguous() else t.new_empty(shape)


def _dtype(n, t, name, f32=True):
    code = n.dtypes.get(t)
    if code is None or (code == F32 and not f32):
        raise TypeError(f"{name} must be bfloat16 or float16" + (" or float32" if f32 else "") + f", got {t}")
    return code


def _heads(n, t, name, like=None):
    """A [tokens][heads][head_dim] tensor on the GPU -> its shape, its token
    and its head stride; `like`: the tensor whose dtype and device it must
    have."""
    if not isinstance(t, n.Tensor) or t.get_device() < 0:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must be 3-D [tokens][heads][head_dim]")
    if like is not None and (t.dtype is not like.dtype or t.get_device() != like.get_device()):
        raise TypeError(f"{name} must be {like.dtype} on {like.device}, got {t.dtype} on {t.device}")
    tokens, h, d = t.shape
    ts, hs, ds = t.stride()
    if ds != 1 and d > 1:
        raise ValueError(f"{name}: head_dim must be contiguous")
    # The stride of a dimension of one element says nothing.
    return tokens, h, d, (h * d if tokens <= 1 else ts), (d if h == 1 else hs)


def _whole(n, t, name, dtype, index, count=None):
    """A contiguous tensor of this dtype on GPU `index` (with `count`
    elements) -> its address."""
    try:
        if (t.dtype is dtype and t.get_device() == index and t.is_contiguous()
                and (count is None or t.numel() == count)):
            return t.data_ptr()
    except AttributeError:  # no tensor
        pass
    if isinstance(t, n.Tensor):
        if t.get_device() == index:
            if t.dtype is not dtype:
                raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
            raise ValueError(f"{name} must have {count} elements, got {list(t.shape)}")
    raise TypeError(f"{name} must be a tensor on cuda:{index}")


def _elsewhere(n, index, stream):
    """Whether the call has to be made in another context than the caller's."""
    return stream is not None or n.device() != index


def _on(n, index, stream):
    """The context in which outputs are allocated and the call is made: the
    tensors' device, and the stream given (so that the allocator ties what is
    allocated here to the stream that writes it)."""
    stack = contextlib.ExitStack()
    stack.enter_context(n.torch.cuda.device(index))
    if stream is not None:
        stack.enter_context(n.torch.cuda.stream(stream))
    return stack


def _out(n, out, name, shape, dtype, index):
    if out is None:
        return n.torch.empty(shape, dtype=dtype, device=n.torch.device("cuda", index))
    _whole(n, out, name, dtype, index)
    if tuple(out.shape) != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(out.shape)}")
    return out


def _cache_args(n, cache, index):
    data = cache["data"]
    ptr = _whole(n, data, "cache data", n.uint8, index)
    if data.dim() != 4 or data.shape[3] % 18 != 0:
        raise ValueError("cache data must be uint8 [num_pages][kv_heads][page_size / 16][18 * head_dim]")
    pages, heads, tiles, rec = data.shape
    return ptr, (pages, heads, 16 * tiles, rec // 18, _whole(n, cache["k_amax"], "k_amax", n.f32, index, 1),
                 _whole(n, cache["v_amax"], "v_amax", n.f32, index, 1))


def _table_args(n, page_table, index):
    ptr = _whole(n, page_table, "page_table", n.int32, index)
    if page_table.dim() != 2:
        raise ValueError("page_table must be int32 [batch][pages of a sequence]")
    return ptr, *page_table.shape


def _rope_args(n, table, index):
    """(pointer, max_pos, rot_dim) of a rotation table."""
    ptr = _whole(n, table, "table", n.f32, index)
    if table.dim() != 3 or table.shape[1] != 2:
        raise ValueError("table must be float32 [max_pos][2][rot_dim / 2]")
    max_pos, _, half = table.shape
    return ptr, max_pos, 2 * half


def _ints(n, t, name, count, index):
    return None if t is None else _whole(n, t, name, n.int32, index, count)


# ------------------------------------------------------------------ the API

def nvfp4_rope_table(max_pos: int, rot_dim: int, base: float = 10000.0, scaling: str | None = None,
                     factor: float = 1.0, original_len: float = 0.0, low: float = 1.0, high: float = 32.0,
                     amplitude: float = 1.0, device=None, out=None, stream=None):
    """Cosines and sines of the rotation's angles: float32 [max_pos][2]
    [rot_dim / 2], made once and kept. scaling, for contexts longer than the
    model was trained on (original_len): None; "linear" (positions divided by
    factor); "base" (a larger base); "parts" (pairs that turn more than `high`
    times over original_len stay, those below `low` are divided by factor, a
    ramp between). amplitude multiplies both."""
    n = _n()
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {list(_SCALINGS)}")
    device = _device(device)
    if device.type == "cuda" and device.index is None:
        device = n.torch.device("cuda", n.torch.cuda.current_device())
    with _on(n, device.index, stream):
        out = _out(n, out, "out", (max_pos, 2, rot_dim // 2), n.f32, device.index)
        _check(lib().nvfp4_rope_table(max_pos, rot_dim, base, _SCALINGS[scaling], factor, original_len, low, high,
                                      amplitude, out.data_ptr(), n.stream(device.index)))
    return out


def nvfp4_rope(x, positions, table, interleaved: bool = False, adjoint: bool = False, out=None, stream=None):
    """Rotates the first rot_dim elements of every head of x [tokens][heads]
    [head_dim] (bfloat16, float16 or float32) by its token's position (int32
    [tokens]). interleaved: pairs (2i, 2i + 1), otherwise (i, i + rot_dim / 2).
    adjoint: the gradient of the rotation (dx from dy). out: may be x itself."""
    n = _n()
    tokens, h, d, *xs = _heads(n, x, "x")
    dt = _dtype(n, x.dtype, "x")
    dev = x.get_device()
    if _elsewhere(n, dev, stream):
        with _on(n, dev, stream):
            return nvfp4_rope(x, positions, table, interleaved, adjoint, out)
    pos = _ints(n, positions, "positions", tokens, dev)
    tab, max_pos, rot = _rope_args(n, table, dev)
    if out is None:
        out = _like(n, x, (tokens, h, d))
        ys = h * d, d
    else:
        *shape, yt, yh = _heads(n, out, "out", x)
        if shape != [tokens, h, d]:
            raise ValueError(f"out must be {[tokens, h, d]}, got {shape}")
        ys = yt, yh
    flags = (_INTERLEAVED if interleaved else 0) | (_ADJOINT if adjoint else 0)
    _check(lib().nvfp4_rope(x.data_ptr(), dt, tokens, h, d, *xs, pos, tab, max_pos, rot, flags, out.data_ptr(), *ys,
                            n.stream(dev)))
    return out


def nvfp4_kv_cache(num_pages: int, kv_heads: int, head_dim: int, k_amax, v_amax, page_size: int = 64, device=None):
    """An empty cache. k_amax, v_amax: the largest magnitudes that keys (after
    the rotation) and values are taken to have, as numbers or float32 [1]
    tensors (from nvfp4_amax of a calibration run); larger ones saturate.
    page_size: a power of two from 16 to 32768; head_dim: 64, 128 or 256."""
    torch = _torch()
    if not 16 <= page_size <= 32768 or page_size & (page_size - 1) or head_dim not in (64, 128, 256):
        raise Nvfp4Error(-2, f"a cache has pages of a power of two from 16 to 32768 tokens and heads of 64, 128 or 256 "
                             f"elements, got {page_size} and {head_dim}")
    device = _device(device)

    def amax(a):
        return a if isinstance(a, torch.Tensor) else torch.full((1,), float(a), dtype=torch.float32, device=device)

    data = torch.zeros((num_pages, kv_heads, page_size // 16, 18 * head_dim), dtype=torch.uint8, device=device)
    return {"data": data, "k_amax": amax(k_amax), "v_amax": amax(v_amax)}


def nvfp4_kv_append(cache, k, v, positions, page_table, seq=None, table=None, interleaved: bool = False, q=None,
                    q_out=None, stream=None):
    """Quantizes k and v [tokens][kv_heads][head_dim] into the cache, k rotated
    on the way (table, as nvfp4_rope; None: not rotated). Token t is token
    positions[t] of sequence seq[t] (int32; seq None: of sequence t, at most
    batch tokens), whose pages are row seq[t] of page_table (int32 [batch]
    [pages]). A negative position marks padding. With q [tokens][heads][head_dim], also rotates the
    queries in the same launch and returns them (q_out: may be q itself);
    otherwise returns None."""
    n = _n()
    like_k = tokens, kh, d, *ks = _heads(n, k, "k")
    dt = _dtype(n, k.dtype, "k")
    like_v = _heads(n, v, "v", k)
    if like_v != like_k and (like_v[:3] != like_k[:3] or k.numel() > 0):
        raise ValueError("k and v must have the same shape and strides")
    dev = k.get_device()
    if _elsewhere(n, dev, stream):
        with _on(n, dev, stream):
            return nvfp4_kv_append(cache, k, v, positions, page_table, seq, table, interleaved, q, q_out)
    data, dims = _cache_args(n, cache, dev)
    if kh != dims[1] or d != dims[3]:
        raise ValueError(f"k must be [tokens][{dims[1]}][{dims[3]}] for this cache, got {list(k.shape)}")
    pos = _ints(n, positions, "positions", tokens, dev)
    sq = _ints(n, seq, "seq", tokens, dev)
    pages, batch, stride = _table_args(n, page_table, dev)
    tab, max_pos, rot = (None, 0, 0) if table is None else _rope_args(n, table, dev)
    if table is None and (q is not None or interleaved):
        raise ValueError("q and interleaved need a rotation table")
    qp, qo, heads, qs, qos = None, None, 0, (0, 0), (0, 0)
    if q is not None:
        qt, heads, qd, *qs = _heads(n, q, "q", k)
        if qt != tokens or qd != d:
            raise ValueError(f"q must be [{tokens}][heads][{d}], got {list(q.shape)}")
        if q_out is None:
            q_out = _like(n, q, (tokens, heads, d))
            qos = heads * d, d
        else:
            *shape, yt, yh = _heads(n, q_out, "q_out", k)
            if shape != [tokens, heads, d]:
                raise ValueError(f"q_out must be {[tokens, heads, d]}, got {shape}")
            qos = yt, yh
        qp, qo = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    if tokens == 0:
        return q_out
    _check(lib().nvfp4_kv_append(k.data_ptr(), v.data_ptr(), dt, tokens, *ks, qp, qo, heads, *qs, *qos, pos, sq, pages,
                                 batch, stride, tab, max_pos, rot, _INTERLEAVED if interleaved else 0, data, *dims,
                                 n.stream(dev)))
    return q_out


def nvfp4_kv_read(cache, positions, page_table, seq=None, out_dtype=None, out=None, stream=None):
    """The keys and values that the cache holds for a list of tokens (named as
    in nvfp4_kv_append) -> (k, v), each [tokens][kv_heads][head_dim] of
    out_dtype (bfloat16 by default, or float16, float32). out: a pair of
    tensors to write to."""
    n = _n()
    out_dtype = n.torch.bfloat16 if out_dtype is None else out_dtype
    dt = _dtype(n, out_dtype, "out_dtype")
    dev = cache["data"].get_device()
    if dev < 0:
        raise TypeError("the cache must be on the GPU")
    if _elsewhere(n, dev, stream):
        with _on(n, dev, stream):
            return nvfp4_kv_read(cache, positions, page_table, seq, out_dtype, out)
    data, dims = _cache_args(n, cache, dev)
    if not isinstance(positions, n.Tensor) or positions.dim() != 1:
        raise ValueError("positions must be int32 [tokens]")
    tokens = positions.shape[0]
    pos = _ints(n, positions, "positions", tokens, dev)
    sq = _ints(n, seq, "seq", tokens, dev)
    pages, batch, stride = _table_args(n, page_table, dev)
    shape = (tokens, dims[1], dims[3])
    ok, ov = out or (None, None)
    at = cache["data"].device
    k = n.empty(shape, dtype=out_dtype, device=at) if ok is None else _out(n, ok, "out", shape, out_dtype, dev)
    v = n.empty_like(k) if ov is None else _out(n, ov, "out", shape, out_dtype, dev)
    if tokens > 0:
        _check(lib().nvfp4_kv_read(data, *dims, tokens, pos, sq, pages, batch, stride, k.data_ptr(), v.data_ptr(), dt,
                                   n.stream(dev)))
    return k, v


def nvfp4_kv_workspace(device=None):
    """A zero-filled workspace for nvfp4_kv_attention."""
    torch = _torch()
    return torch.zeros(KV_WORKSPACE_BYTES // 4, dtype=torch.int32, device=_device(device))


def nvfp4_kv_attention(q, cache, page_table, lens, workspace, cu_q=None, max_q: int | None = None, scale: float | None = None,
                       causal: bool = True, window: int = 0, out=None, return_lse: bool = False, lse=None,
                       stream=None):
    """Attention of q [total_q][heads][head_dim] (bfloat16 or float16; heads a
    multiple of the cache's) over the cached tokens -> [total_q][heads]
    [head_dim] of q's dtype, or with return_lse (or an lse tensor) the pair of
    it and the log-sum-exp, float32 [total_q][heads].

    lens: int32 [batch], the cached tokens of each sequence, the queries' own
    among them (they are appended first). cu_q: int32 [batch + 1], where each
    sequence's queries begin, at most max_q each (given with it; queries past
    that are NaN); None: max_q (1 by default) for every sequence. Query i of n sits at position lens - n + i and sees the tokens
    up to itself (causal) and after its position - window (window > 0);
    without either all of them. One that sees nothing gives 0 and -inf.
    scale: 1 / sqrt(head_dim) by default. workspace: from nvfp4_kv_workspace,
    kept between calls; calls that overlap in time need different ones."""
    n = _n()
    tokens, h, d, *qs = _heads(n, q, "q")
    dt = _dtype(n, q.dtype, "q", f32=False)
    if max_q is None:
        if cu_q is not None:
            raise ValueError("cu_q needs max_q, the most queries of one sequence")
        max_q = 1
    dev = q.get_device()
    if _elsewhere(n, dev, stream):
        with _on(n, dev, stream):
            return nvfp4_kv_attention(q, cache, page_table, lens, workspace, cu_q, max_q, scale, causal, window, out,
                                      return_lse, lse)
    data, dims = _cache_args(n, cache, dev)
    if d != dims[3]:
        raise ValueError(f"q must be [tokens][heads][{dims[3]}] for this cache, got {list(q.shape)}")
    pages, batch, stride = _table_args(n, page_table, dev)
    ln = _ints(n, lens, "lens", batch, dev)
    cu = _ints(n, cu_q, "cu_q", batch + 1, dev)
    ws = _whole(n, workspace, "workspace", n.int32, dev)
    if 4 * workspace.numel() < KV_WORKSPACE_BYTES:
        raise ValueError(f"workspace must hold {KV_WORKSPACE_BYTES} bytes")
    out = _like(n, q, (tokens, h, d)) if out is None else _out(n, out, "out", (tokens, h, d), q.dtype, dev)
    if return_lse or lse is not None:
        lse = _out(n, lse, "lse", (tokens, h), n.f32, dev)
    if tokens > 0:
        _check(lib().nvfp4_kv_attention(
            q.data_ptr(), dt, tokens, h, *qs, cu, max_q, data, *dims, pages, batch, stride, ln,
            1.0 / math.sqrt(d) if scale is None else scale, window, _CAUSAL if causal else 0, out.data_ptr(),
            None if lse is None else lse.data_ptr(), ws, n.stream(dev)))
    return out if lse is None else (out, lse)
