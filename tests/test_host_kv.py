"""Host-side checks of the key/value cache's C ABI (no GPU needed): every
refusal comes before any HIP call, and the plain forms that the GPU tests
compare with agree with each other and with the definitions."""
import ctypes
import math

import numpy as np
import pytest

import fp4_block_scaled_amax_amd as F
import kv_plain
import oracle
from fp4_block_scaled_amax_amd import build as B

P = ctypes.c_void_p
A, MIS, NULL = P(4096), P(4104), None


@pytest.fixture(scope="module")
def L():
    if B.is_stale():
        B.build()
    return F.lib()


def test_rope_table_validation(L):
    f = lambda n=16, r=32, base=1e4, kind=0, factor=1.0, l0=0.0, lo=1.0, hi=32.0, amp=1.0, t=A: L.nvfp4_rope_table(  # noqa: E731
        n, r, base, kind, factor, l0, lo, hi, amp, t, NULL)
    assert f(t=NULL) == -1
    assert f(kind=4) == -4
    assert f(base=1.0) == -4
    assert f(base=math.nan) == -4
    assert f(factor=0.5) == -4
    assert f(amp=math.inf) == -4
    assert f(kind=3, factor=4.0) == -4            # no original length
    assert f(kind=3, l0=1.0, lo=4.0, hi=4.0) == -4
    assert f(r=8) == -2
    assert f(n=0) == -2
    assert f(n=1 << 40) == -6
    assert f(t=MIS) == -3


def test_rope_validation(L):
    def f(x=A, dt=1, n=4, h=2, d=64, xs=(128, 64), pos=A, t=A, maxp=16, r=32, fl=0, y=A, ys=(128, 64)):
        return L.nvfp4_rope(x, dt, n, h, d, *xs, pos, t, maxp, r, fl, y, *ys, NULL)
    assert f(dt=3) == -4
    assert f(fl=4) == -4
    assert f(ys=(256, 64)) == -4                  # in place with other strides
    assert f(n=-1) == -2
    assert f(h=0) == -2
    assert f(d=72) == -2
    assert f(r=80) == -2
    assert f(r=24) == -2
    assert f(r=0) == -2
    assert f(maxp=0) == -2
    assert f(xs=(-128, 64)) == -2
    assert f(xs=(132, 64)) == -3
    assert f(dt=0, xs=(130, 64)) == -3
    assert f(y=MIS) == -3
    assert f(x=NULL) == -1
    assert f(pos=NULL) == -1
    assert f(t=NULL) == -1
    assert f(n=1 << 40, xs=(1 << 40, 64)) == -6
    assert f(n=0, x=NULL, y=NULL, pos=NULL) == 0  # nothing to do


def test_append_validation(L):
    def f(k=A, v=A, dt=1, n=4, ks=(128, 64), q=A, qo=A, h=2, qs=(128, 64), qos=(128, 64), pos=A, seq=NULL, pt=A, b=1,
          ps=2, t=A, maxp=16, r=32, fl=0, data=A, np_=4, kh=2, page=16, d=64, ka=A, va=A):
        return L.nvfp4_kv_append(k, v, dt, n, *ks, q, qo, h, *qs, *qos, pos, seq, pt, b, ps, t, maxp, r, fl, data, np_,
                                 kh, page, d, ka, va, NULL)
    assert f(dt=5) == -4
    assert f(fl=2) == -4                          # the adjoint is nvfp4_rope's
    assert f(t=NULL, q=NULL, qo=NULL, h=0) == -4  # rot_dim without a table
    assert f(qs=(256, 64)) == -4                  # in place with other strides
    for name in ("data", "ka", "va", "pt", "k", "v", "pos", "qo", "q", "t"):
        assert f(**{name: NULL}) == -1, name
    assert f(h=0) == -1                           # queries but no heads
    assert f(page=8) == -2
    assert f(page=48) == -2
    assert f(page=65536) == -2
    assert f(d=96, r=32) == -2
    assert f(r=96) == -2
    assert f(n=-1) == -2
    assert f(np_=0) == -2
    assert f(b=0) == -2
    assert f(ks=(100, 64)) == -3
    assert f(data=MIS) == -3
    assert f(k=MIS) == -3
    assert f(pos=P(4097)) == -3
    assert f(np_=1 << 40) == -6
    assert f(ps=1 << 40) == -6
    assert f(n=0, k=NULL, v=NULL, pos=NULL) == 0


def test_read_validation(L):
    def f(data=A, n=4, pos=A, k=A, v=A, dt=1, page=16, d=64):
        return L.nvfp4_kv_read(data, 4, 2, page, d, A, A, n, pos, NULL, A, 1, 2, k, v, dt, NULL)
    assert f(dt=9) == -4
    assert f(data=NULL) == -1
    assert f(pos=NULL) == -1
    assert f(k=NULL, v=NULL) == -1
    assert f(page=24) == -2
    assert f(d=32) == -2
    assert f(n=-2) == -2
    assert f(k=MIS) == -3
    assert f(n=0, pos=NULL, k=NULL, v=NULL) == 0


def test_attention_validation(L):
    def f(q=A, dt=1, n=4, h=4, qs=(256, 64), cu=NULL, mq=2, data=A, np_=4, kh=2, page=16, d=64, pt=A, b=2, ps=2, lens=A,
          scale=0.125, w=0, fl=1, out=A, lse=NULL, ws=A):
        return L.nvfp4_kv_attention(q, dt, n, h, *qs, cu, mq, data, np_, kh, page, d, A, A, pt, b, ps, lens, scale, w,
                                    fl, out, lse, ws, NULL)
    assert f(dt=0) == -4                          # 16-bit queries only
    assert f(fl=2) == -4
    for scale in (0.0, -1.0, math.nan, math.inf):
        assert f(scale=scale) == -4
    for name in ("q", "data", "pt", "lens", "out", "ws"):
        assert f(**{name: NULL}) == -1, name
    assert f(h=3) == -2
    assert f(n=5) == -2                           # not batch * max_q without cu_q
    assert f(mq=0) == -2
    assert f(w=-1) == -2
    assert f(d=80) == -2
    assert f(qs=(256, 60)) == -3
    assert f(ws=MIS) == -3
    assert f(out=MIS) == -3
    assert f(lse=P(4098)) == -3
    assert f(cu=A, n=1 << 40, mq=2) == -6
    assert f(cu=A, mq=1 << 31) == -6
    assert f(cu=A, n=0, q=NULL, out=NULL) == 0


def test_division_by_a_launch_constant():
    """kernels.h's DivBy: n / d = (n mul) >> 32 >> s with mul = ceil(2^(32 + s)
    / d), 2^s >= d > 2^(s - 1), for every n < 2^31; checked at the ends of
    every quotient step that could fail (multiples of d, and one less)."""
    rng = np.random.default_rng(0)
    for d in [1, 2, 3, 5, 6, 7, 10, 12, 24, 100, 255, 1 << 13, (1 << 20) - 1, 1 << 20] + rng.integers(1, 1 << 20, 50).tolist():
        s = 0
        while (1 << s) < d:
            s += 1
        mul = ((1 << (32 + s)) + d - 1) // d
        assert mul < 1 << 33
        top = ((1 << 31) - 1) // d
        for k in {0, 1, 2, top // 2, top - 1, top} | set(rng.integers(0, top + 1, 50).tolist()):
            for n in (k * d - 1, k * d, k * d + d - 1):
                if 0 <= n < 1 << 31:
                    assert n * mul < 1 << 64
                    assert (n * mul >> 32) >> s == n // d


@pytest.mark.parametrize("D", [64, 128, 256])
def test_record_layout_is_a_bijection(D):
    """Every nibble and scale byte of a record belongs to one element of one
    token, and a record is 18 D bytes."""
    seen = np.zeros((18 * D, 2), int)
    for keys in (True, False):
        for t in range(16):
            code, shift, scale = kv_plain.places(D, t, keys)
            np.add.at(seen, (code, shift // 4), 1)
            np.add.at(seen, (scale, 0), 1)
            np.add.at(seen, (scale, 1), 1)
    assert (seen == 1).all()


def test_plain_quantizer_is_the_oracles():
    """On BF16 values the plain block quantizer equals the oracle's rowwise
    quantization byte for byte."""
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((6, 128)) * 3).astype(np.float32)
    bits = (x.view(np.uint32) >> 16).astype(np.uint16)
    x = (bits.astype(np.uint32) << 16).view(np.float32)
    amax = np.float32(9.0)
    codes, scales = oracle.quantize_1d_rows(bits, oracle.global_scale(amax))
    for r in range(6):
        c, s = kv_plain.quantize_row(x[r], amax)
        assert np.array_equal(s, np.asarray(scales)[r])
        assert np.array_equal(c[0::2] | (c[1::2] << 4), np.asarray(codes)[r])


def test_plain_rotation_in_64_bits():
    """A pair turns by its angle: complex multiplication, and the adjoint
    undoes it."""
    rng = np.random.default_rng(2)
    ang = rng.uniform(0, 7, (5, 8))
    table = np.stack([np.cos(ang), np.sin(ang)], 1)
    x = rng.standard_normal((5, 3, 32))
    pos = np.arange(5)
    for il in (False, True):
        y = kv_plain.rotate(x, pos, table, il, dtype=np.float64)
        a, b = (x[..., :16:2], x[..., 1:16:2]) if il else (x[..., :8], x[..., 8:16])
        z = (a + 1j * b) * np.exp(1j * ang)[:, None]
        ya, yb = (y[..., :16:2], y[..., 1:16:2]) if il else (y[..., :8], y[..., 8:16])
        assert np.abs(ya + 1j * yb - z).max() < 1e-14
        assert np.abs(kv_plain.rotate(y, pos, table, il, True, np.float64) - x).max() < 1e-14
        assert np.array_equal(y[..., 16:], x[..., 16:])


def test_grids_that_no_launch_holds_are_refused(L):
    """A grid has fewer than 2^32 threads along x and 65536 workgroups along
    y: sizes past that are refused before any HIP call."""
    def append(n=4, h=2, kh=2, d=64):
        hs = 64 * h
        return L.nvfp4_kv_append(A, A, 1, n, 64 * kh, 64, A, A, h, hs, 64, hs, 64, A, NULL, A, 1, 2, A, 16, 32, 0, A, 4,
                                 kh, 16, d, A, A, NULL)

    def read(n=4, kh=2, d=64):
        return L.nvfp4_kv_read(A, 4, kh, 16, d, A, A, n, A, NULL, A, 1, 2, A, A, 1, NULL)

    def attention(n=4, h=4, kh=2, b=2, mq=2, cu=A):
        return L.nvfp4_kv_attention(A, 1, n, h, 64 * h, 64, cu, mq, A, 4, kh, 16, 64, A, A, A, b, 2, A, 0.125, 0, 1, A,
                                    NULL, A, NULL)
    assert append(n=1 << 28) == -6
    assert append(h=1 << 20) == -6
    assert append(kh=60000, d=256) == -6
    assert read(n=1 << 28) == -6
    assert read(kh=60000, d=256) == -6
    assert attention(b=1 << 23) == -6
    assert attention(n=1 << 20, mq=1 << 20, b=1 << 12) == -6
    assert attention(n=1 << 30, b=1 << 10, mq=1 << 20, cu=NULL) == -6


def test_more_queries_than_max_q_allows_are_refused(L):
    """With cu_q too, a call has at most max_q queries for each sequence."""
    def f(n, mq, b=2, cu=A):
        return L.nvfp4_kv_attention(A, 1, n, 4, 256, 64, cu, mq, A, 4, 2, 16, 64, A, A, A, b, 2, A, 0.125, 0, 1, A, NULL, A,
                                    NULL)
    assert f(5, 2) == -2
    assert f(3, 1) == -2
    assert f(1 << 30, (1 << 29) - 1) == -6        # a grid that no launch holds comes first


def test_tokens_of_no_sequence_are_refused(L):
    """Without seq, token t belongs to sequence t: there are batch of them."""
    def append(n, b, q=A, h=2):
        return L.nvfp4_kv_append(A, A, 1, n, 128, 64, q, q, h, 128, 64, 128, 64, A, NULL, A, b, 2, A, 16, 32, 0, A, 4, 2,
                                 16, 64, A, A, NULL)

    def read(n, b):
        return L.nvfp4_kv_read(A, 4, 2, 16, 64, A, A, n, A, NULL, A, b, 2, A, A, 1, NULL)
    assert append(4, 3) == -2
    assert append(2, 1, q=NULL, h=0) == -2
    assert read(4, 3) == -2


def test_the_layer_finds_each_tokens_sequence():
    """seq from max_q or cu_q, sequences without tokens among them; none where
    every sequence has one token, and the given one as it is."""
    import torch

    from fp4_block_scaled_amax_amd.attention import _sequences

    cpu = torch.device("cpu")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    assert _sequences(None, None, None, 3, 3, cpu) is None
    assert _sequences(None, None, 1, 3, 3, cpu) is None
    assert _sequences(None, i32([0, 1, 2, 3]), 1, 3, 3, cpu) is None
    given = i32([2, 0])
    assert _sequences(given, i32([0, 1, 1, 2]), 1, 2, 3, cpu) is given
    with pytest.raises(ValueError, match="max_q"):
        _sequences(given, i32([0, 1, 1, 2]), None, 2, 3, cpu)
    for news, max_q in (([4, 4, 4], 4), ([2, 0, 5], 5), ([0, 0, 3], 7), ([1, 0, 1], 1), ([0, 1, 0, 1, 1], 1)):
        want = i32(np.repeat(np.arange(len(news)), news).tolist())
        got = _sequences(None, i32(np.cumsum([0] + news).tolist()), max_q, sum(news), len(news), cpu)
        assert got.dtype == torch.int32 and torch.equal(got, want)
    got = _sequences(None, None, 4, 12, 3, cpu)
    assert got.dtype == torch.int32 and torch.equal(got, i32([0, 0, 0, 0, 1, 1, 1, 1, 2, 2, 2, 2]))


def test_outputs_that_overlap_themselves_are_refused(L):
    """A result whose tokens or heads share elements (a broadcast view) has no
    value; any other strides are taken, nested or not (here up to the missing
    input: nothing is launched)."""
    def rope(n, h, d, ys):
        return L.nvfp4_rope(NULL, 1, n, h, d, 0, 0, A, A, 16, 16, 0, A, *ys, NULL)

    def append(n, h, ys):
        return L.nvfp4_kv_append(NULL, A, 1, n, 128, 64, A, A, h, 64 * h, 64, *ys, A, A, A, 1, 2, A, 16, 32, 0, A, 4, 2, 16,
                                 64, A, A, NULL)
    rng = np.random.default_rng(5)
    cases = [(4, 2, 64, (0, 64)), (4, 2, 64, (128, 0)), (4, 1, 64, (56, 0)), (1, 3, 64, (0, 32)), (4, 2, 64, (64, 64)),
             (4, 3, 64, (128, 64)), (2, 4, 64, (64, 128)), (2, 2, 64, (192, 128)), (3, 3, 64, (192, 128)),
             (1, 1, 64, (0, 0)), (5, 1, 64, (64, 0)), (4, 2, 64, (128, 64)), (4, 2, 64, (64, 256))]
    cases += [(int(n), int(h), 16, (8 * int(a), 8 * int(b))) for n, h, a, b in rng.integers(1, 13, (400, 4))]
    refused = 0
    for n, h, d, ys in cases:
        at = (np.arange(n)[:, None, None] * ys[0] + np.arange(h)[:, None] * ys[1] + np.arange(d)).reshape(-1)
        apart = len(set(at.tolist())) == len(at)
        refused += not apart
        assert rope(n, h, d, ys) == (-1 if apart else -2), (n, h, d, ys)
        if d == 64:
            assert append(n, h, ys) == (-1 if apart else -2), (n, h, d, ys)
    assert 100 < refused < len(cases) - 100


def test_attention_of_no_sequences(L):
    """An empty batch is nothing to do; queries of no sequence are refused."""
    def f(n, b, pt=NULL, scale=0.125, cu=NULL):
        return L.nvfp4_kv_attention(NULL, 1, n, 4, 256, 64, cu, 1, A, 4, 2, 16, 64, A, A, pt, b, 2, NULL, scale, 0, 1, NULL,
                                    NULL, A, NULL)
    assert f(0, 0) == 0
    assert f(0, 0, pt=A, cu=A) == 0
    assert f(0, 0, scale=-1.0) == -4
    assert f(1, 0, pt=A) == -2
    assert f(1, 0, pt=A, cu=A) == -2


def test_caches_that_no_call_takes_are_refused():
    """A page of 24 tokens would become one of 16, at other places than the
    caller's page table says."""
    for page, d in ((24, 64), (0, 64), (8, 64), (-16, 64), (48, 128), (65536, 64), (16, 96), (16, 0)):
        with pytest.raises(F.Nvfp4Error, match="ERR_SHAPE"):
            F.nvfp4_kv_cache(2, 1, d, 8.0, 8.0, page_size=page, device="cpu")
    cache = F.nvfp4_kv_cache(2, 3, 128, 8.0, 8.0, page_size=32, device="cpu")
    assert cache["data"].shape == (2, 3, 2, 18 * 128)


def test_device_0_is_the_first_gpu(monkeypatch):
    """A device given as 0 is that one, not the current one."""
    import torch

    asked = []
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **k: asked.append(torch.device(device)))
    for make in (F.nvfp4_workspace, F.nvfp4_kv_workspace, lambda d=None: F.nvfp4_kv_cache(
            2, 1, 64, torch.ones(1), torch.ones(1), device=d)):
        for given, want in ((0, "cuda:0"), (1, "cuda:1"), ("cuda:0", "cuda:0"), (None, "cuda"), (torch.device("cpu"), "cpu")):
            make(given)
            assert asked.pop() == torch.device(want)


def test_the_kernels_division_by_a_launch_constant(tmp_path):
    """The same with csrc/div_by.h itself, compiled for the host: every divisor
    up to 4096, powers of two and their neighbours, and large ones, at both ends
    of quotient steps from the first to the last."""
    import os
    import subprocess

    source, program = tmp_path / "div.cpp", tmp_path / "div"
    source.write_text(r"""
#include <stdio.h>
#include <initializer_list>
#include "div_by.h"
static uint64_t seed = 1;
static uint64_t draw() { return (seed = seed * 6364136223846793005ull + 1442695040888963407ull) >> 33; }  // 31 bits
static int wrong = 0;
static void check(uint32_t d)
{
    const nvfp4::DivBy by = nvfp4::DivBy::of(d);
    const uint64_t last = 0x7FFFFFFFull / d;
    auto at = [&](uint64_t q) {
        for (uint64_t n : {q * d - 1, q * d, q * d + 1, q * d + d - 1})
            if (n <= 0x7FFFFFFFull && by.div((uint32_t)n) != n / d && wrong++ < 5)
                printf("%llu / %u: %u\n", (unsigned long long)n, d, by.div((uint32_t)n));
    };
    for (uint64_t q = 0; q < 8; ++q) {
        at(q);
        at(last - (q < last ? q : last));
    }
    for (int i = 0; i < 32; ++i)
        at(draw() % (last + 1));
}
int main()
{
    for (uint32_t d = 1; d <= 4096; ++d)
        check(d);
    for (uint32_t b = 2; b < 31; ++b)
        for (int i = -1; i <= 1; ++i)
            check((1u << b) + i);
    for (int i = 0; i < 20000; ++i)
        check((uint32_t)(draw() >> (i % 20)) + 1);
    printf("%d wrong\n", wrong);
    return wrong != 0;
}
""")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", os.path.join(os.path.dirname(B.__file__), "csrc"), "-o",
                    str(program), str(source)], check=True)
    done = subprocess.run([str(program)], capture_output=True, text=True, timeout=60)
    assert done.returncode == 0 and done.stdout == "0 wrong\n", done.stdout
