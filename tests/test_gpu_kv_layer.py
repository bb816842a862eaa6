"""GPU: the attention layer (fp4_block_scaled_amax_amd/attention.py) and the
cache's operators used together: a prompt, then single tokens, against the
64-bit attention of the same projections; and a prompt taken whole against the
same prompt taken token by token."""
import math

import numpy as np
import pytest
import torch

import kv_plain as P
import workloads as W

pytestmark = pytest.mark.gpu

F = None


def setup_module(module):
    global F
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp4_block_scaled_amax_amd as pkg
    from fp4_block_scaled_amax_amd import attention, linear

    pkg.lib()  # raises if the HIP library is missing: no fallback
    F = pkg
    F.layer, F.lin = attention, linear


def bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_prompt_then_tokens():
    """Three sequences: prompts of 21, 1 and 16 tokens in one call, then two
    decode steps. The projections' own outputs (the NVFP4 linear layer's, with
    its tests) are what the 64-bit form starts from; o against it within the
    attention's bound, y as the linear layer's of that o."""
    hidden, heads, kv_heads, D, page = 256, 4, 2, 64, 16
    rng = np.random.default_rng(21)
    w = F.layer.layer_weights(bf16(W.weight((heads + 2 * kv_heads) * D, hidden, seed=5)),
                              bf16(W.weight(hidden, heads * D, seed=6)))
    table = F.nvfp4_rope_table(64, D)
    cache = F.nvfp4_kv_cache(12, kv_heads, D, 4.0, 4.0, page_size=page)
    pages = torch.randperm(12, device="cuda").to(torch.int32).view(3, 4)
    ws, kws = F.nvfp4_workspace(), F.nvfp4_kv_workspace()
    lens = [0, 0, 0]
    for news in ([21, 1, 16], [1, 1, 1], [1, 1, 1]):
        tokens = sum(news)
        x = torch.from_numpy(rng.standard_normal((tokens, hidden)).astype(np.float32)).bfloat16().cuda()
        pos = np.concatenate([np.arange(n, n + k) for n, k in zip(lens, news)]).astype(np.int32)
        seq = np.repeat(np.arange(3), news).astype(np.int32)
        lens = [n + k for n, k in zip(lens, news)]
        cu = i32(np.cumsum([0] + news).tolist())
        y = F.layer.attention_layer(x, w, cache, i32(pos.tolist()), pages, i32(lens), table, kws, heads,
                                    seq=i32(seq.tolist()), cu_q=cu, max_q=max(news), ws=ws)
        assert y.shape == (tokens, hidden) and y.dtype == torch.bfloat16
        # the same steps apart
        pad = F.layer._rows16(x)
        assert pad.shape[0] % 16 == 0 and not pad[tokens:].any()
        qkv = F.lin.fprop(pad, w["qkv"], ws=ws, out_dtype=torch.bfloat16)[:tokens].view(tokens, -1, D)
        turned = P.rotate(qkv[:, :heads].float().cpu().numpy(), pos, table.cpu().numpy(), False)
        q = torch.from_numpy(turned).bfloat16()
        data, tab = cache["data"].cpu().numpy(), pages.cpu().numpy()
        o = F.nvfp4_kv_attention(q.cuda(), cache, pages, i32(lens), kws, cu_q=cu, max_q=max(news))
        at = 0
        for b, (n, k) in enumerate(zip(lens, news)):
            for h in range(kv_heads):
                ks, vs = (np.stack([P.read(data, tab, b, p, h, keys, 4.0) for p in range(n)]) for keys in (True, False))
                # what was cached: exactly what the rotated keys of these tokens quantize to
                new = P.rotate(qkv[at:at + k, heads + h:heads + h + 1].float().cpu().numpy(), pos[at:at + k],
                               table.cpu().numpy(), False)[:, 0]
                for i in range(k):
                    codes, scales = P.quantize_row(new[i], 4.0)
                    sg = float(np.float32(4.0) / np.float32(2688.0))
                    assert np.array_equal(ks[n - k + i], P.E2M1[codes] * np.repeat(P.E4M3[scales], 16) * sg)
                for g in range(2 * h, 2 * h + 2):
                    rows = q[at:at + k, g].double().numpy()
                    want, _, mag = P.attention(rows, ks, vs, 1 / math.sqrt(D), np.zeros(k, int), n - k + np.arange(k) + 1)
                    got = o[at:at + k, g].double().cpu().numpy()
                    assert (np.abs(got - want) <= (2.0 ** -11 + 2.0 ** -14) * mag + 2.0 ** -8 * np.abs(want)).all()
            at += k
        again = F.lin.fprop(F.layer._rows16(o.view(tokens, -1)), w["out"], ws=ws, out_dtype=torch.bfloat16)[:tokens]
        assert torch.equal(y, again)


@pytest.mark.parametrize("window", [0, 40])
def test_whole_prompt_equals_token_by_token(window):
    """150 tokens appended and attended at once, in chunks, and one by one:
    the same bytes in the cache, and outputs that differ by the two kernels'
    roundings alone (twice the attention's bound, with sum p |v| below the
    largest value, 8)."""
    n, heads, kv_heads, D = 150, 8, 2, 128
    gen = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.randn(n, heads + 2 * kv_heads, D, device="cuda", generator=gen).bfloat16()
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
    table, ws = F.nvfp4_rope_table(n, D), F.nvfp4_kv_workspace()
    pages = i32([[2, 0, 1]])
    outs, datas = [], []
    for size in (n, 47, 5, 1):
        cache = F.nvfp4_kv_cache(3, kv_heads, D, 6.0, 6.0, page_size=64)
        o = []
        for at in range(0, n, size):
            end = min(n, at + size)
            pos = torch.arange(at, end, dtype=torch.int32, device="cuda")
            turned = F.nvfp4_kv_append(cache, k[at:end], v[at:end], pos, pages, seq=torch.zeros_like(pos), table=table,
                                       q=q[at:end])
            o.append(F.nvfp4_kv_attention(turned, cache, pages, i32([end]), ws, max_q=end - at, window=window))
        outs.append(torch.cat(o))
        datas.append(cache["data"])
    for o, d in zip(outs[1:], datas[1:]):
        assert torch.equal(d, datas[0])
        assert (o.float() - outs[0].float()).abs().max().item() <= 2 * (2.0 ** -11 + 2.0 ** -14 + 2.0 ** -8) * 8

@pytest.mark.parametrize("cu", [False, True])
def test_several_tokens_of_each_without_seq(cu):
    """Without seq the tokens belong to the sequences as the attention takes
    them: max_q of each, or by cu_q. The same outputs and cache as with it."""
    hidden, heads, kv_heads, D, page, B = 256, 4, 2, 64, 16, 3
    rng = np.random.default_rng(22)
    w = F.layer.layer_weights(bf16(W.weight((heads + 2 * kv_heads) * D, hidden, seed=5)),
                              bf16(W.weight(hidden, heads * D, seed=6)))
    table, kws, ws = F.nvfp4_rope_table(64, D), F.nvfp4_kv_workspace(), F.nvfp4_workspace()
    pages = i32([[7, 1, 2], [0, 4, 5], [3, 6, 8]])
    for news in ([4, 4, 4], [1, 1, 1]) if not cu else ([2, 0, 5], [0, 1, 0], [1, 1, 0], [1, 1, 1]):
        tokens = sum(news)
        x = torch.from_numpy(rng.standard_normal((tokens, hidden)).astype(np.float32)).bfloat16().cuda()
        pos = i32(np.concatenate([np.arange(9, 9 + k) for k in news]).tolist())
        seq = i32(np.repeat(np.arange(B), news).tolist())
        rest = dict(max_q=max(news), cu_q=i32(np.cumsum([0] + news).tolist()) if cu else None, ws=ws)
        got = []
        for s in (seq, None):
            cache = F.nvfp4_kv_cache(9, kv_heads, D, 4.0, 4.0, page_size=page)
            y = F.layer.attention_layer(x, w, cache, pos, pages, i32([9 + k for k in news]), table, kws, heads, seq=s, **rest)
            got.append((y, cache["data"]))
        assert got[0][1].any()
        assert torch.equal(got[0][1], got[1][1])
        assert torch.equal(got[0][0], got[1][0])
