// Appending keys and values to the NVFP4 cache (rotated and quantized on the
// way) and reading them back. See include/nvfp4_kv.h for the contract and
// the record layout.
#include "heads.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 16;                  // tokens of a workgroup
constexpr int kSlots = kThreads / kTokens;   // 16-element units of each token in a workgroup

// 16 binary32 values -> 8 bytes of codes and the block's scale byte, by the
// steps of nvfp4_quantize_1d.
__device__ __forceinline__ uint2 quantize_block(const float (&x)[16], float sg, uint32_t& byte)
{
    uint32_t b = 0u;
#pragma unroll
    for (int j = 0; j < 16; ++j)
        b = max(b, __float_as_uint(x[j]) & 0x7FFFFFFFu);
    byte = block_scale_byte(b, 6.0f * sg);
    const float r = unit_reciprocal(byte, sg);
    uint32_t w[2] = {fresh_word(), fresh_word()};
    // A ratio can be NaN only where r is not finite, or the block's maximum is
    // not (times an r of 0, which an amax of 0 gives).
    if (fabsf(r) <= 3.402823466e38f && b < 0x7F800000u) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            w[h] = put_pair<kEncHw, 0>(w[h], x[8 * h + 0], x[8 * h + 1], r, 0u, 0u);
            w[h] = put_pair<kEncHw, 1>(w[h], x[8 * h + 2], x[8 * h + 3], r, 0u, 0u);
            w[h] = put_pair<kEncHw, 2>(w[h], x[8 * h + 4], x[8 * h + 5], r, 0u, 0u);
            w[h] = put_pair<kEncHw, 3>(w[h], x[8 * h + 6], x[8 * h + 7], r, 0u, 0u);
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            w[h] = put_pair<kEncHwSafe, 0>(w[h], x[8 * h + 0], x[8 * h + 1], r, 0u, 0u);
            w[h] = put_pair<kEncHwSafe, 1>(w[h], x[8 * h + 2], x[8 * h + 3], r, 0u, 0u);
            w[h] = put_pair<kEncHwSafe, 2>(w[h], x[8 * h + 4], x[8 * h + 5], r, 0u, 0u);
            w[h] = put_pair<kEncHwSafe, 3>(w[h], x[8 * h + 6], x[8 * h + 7], r, 0u, 0u);
        }
    }
    return make_uint2(w[0], w[1]);
}

// Keys are rotated in binary32 and quantized without a rounding in between;
// a block of 16 elements is one thread's (its maximum needs no exchange). Its
// partners of a rotation with the halves apart are loaded again by the thread
// of the other half: those bytes come from the cache.
//
// A workgroup holds 16 tokens x 16 units of 16 elements: of the queries
// (blockIdx.y below q_blocks) with the units of a token side by side, which
// makes its loads and stores contiguous; of the keys and values with tokens
// side by side, so that a prompt's tokens fill whole records from one
// workgroup (one L2). (Tokens side by side for the queries too: 57 us where
// this takes 43.)
//
// Memory bounds it: 8192 tokens of 32 + 2 x 8 heads of 128, bf16, 181 MB in 41
// us (4.4 TB/s, a large copy reaches 5.05); 64 tokens 4.7 us, an empty launch
// 2.3.
template <class T, int D>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(KvAppendArgs a, int q_blocks, bool stream_q)
{
    constexpr int kUnits = D / 16;
    const int half = a.rot_dim >> 1;
    if ((int)blockIdx.y < q_blocks) {
        const int64_t t = (int64_t)blockIdx.x * kTokens + threadIdx.x / kSlots;
        const int slot = blockIdx.y * kSlots + (threadIdx.x & (kSlots - 1));
        const int h = slot / kUnits, j = slot % kUnits;
        if (t >= a.tokens || h >= a.heads)
            return;
        const int pos = a.positions[t];
        const Unit u = unit_of(j, a.rot_dim, a.interleaved);
        const char* x = static_cast<const char*>(a.q) + (t * a.q_ts + h * a.q_hs) * T::kBytes;
        char* y = static_cast<char*>(a.q_out) + (t * a.qo_ts + h * a.qo_hs) * T::kBytes;
        float lo[8], hi[8];
        load8<T>(x + u.lo * T::kBytes, lo);
        load8<T>(x + u.hi * T::kBytes, hi);
        if (pos < 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                lo[i] = hi[i] = 0.0f;
        } else if (u.pairs) {
            turn_unit(lo, hi, load_turn(a.table, pos, a.max_pos, half, 8 * j, 0u), a.interleaved);
        }
        if constexpr (T::kBytes == 2 && D >= 128) {
            if (stream_q) {
                store16_stream(y + u.lo * T::kBytes, pack8<T>(lo));
                store16_stream(y + u.hi * T::kBytes, pack8<T>(hi));
                return;
            }
        }
        store8<T>(y + u.lo * T::kBytes, lo);
        store8<T>(y + u.hi * T::kBytes, hi);
        return;
    }
    const int64_t t = (int64_t)blockIdx.x * kTokens + (threadIdx.x & (kTokens - 1));
    const int slot = ((int)blockIdx.y - q_blocks) * kSlots + threadIdx.x / kTokens;
    const int h = slot / kUnits, j = slot % kUnits;
    if (t >= a.tokens || h >= 2 * a.c.kv_heads)
        return;
    const int pos = a.positions[t];
    const bool key = h < a.c.kv_heads;
    const int kh = h - (key ? 0 : a.c.kv_heads);
    const Place p = place_of(a.c, pos, a.seq != nullptr ? a.seq[t] : (int)t);
    if (!p.there)
        return;
    const char* x = static_cast<const char*>(key ? a.k : a.v) + (t * a.kv_ts + kh * a.kv_hs) * T::kBytes;
    float e[2][8];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        // 8 elements from i on; with the halves apart their partners are
        // half further or half back.
        const int i = 16 * j + 8 * g;
        load8<T>(x + i * T::kBytes, e[g]);
        if (key && i < a.rot_dim) {
            if (a.interleaved) {
                const Turn w = load_turn(a.table, pos, a.max_pos, half, 8 * j, 0u);
                float y[8];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    y[2 * m] = turn_a(e[g][2 * m], e[g][2 * m + 1], w.c[4 * g + m], w.s[4 * g + m]);
                    y[2 * m + 1] = turn_b(e[g][2 * m], e[g][2 * m + 1], w.c[4 * g + m], w.s[4 * g + m]);
                }
#pragma unroll
                for (int m = 0; m < 8; ++m)
                    e[g][m] = y[m];
            } else {
                const bool first = i < half;
                const Turn w = load_turn(a.table, pos, a.max_pos, half, first ? i : i - half, 0u);
                float o[8];
                load8<T>(x + (first ? i + half : i - half) * T::kBytes, o);
#pragma unroll
                for (int m = 0; m < 8; ++m)
                    e[g][m] = first ? turn_a(e[g][m], o[m], w.c[m], w.s[m]) : turn_b(o[m], e[g][m], w.c[m], w.s[m]);
            }
        }
    }
    float b[16];
#pragma unroll
    for (int m = 0; m < 16; ++m)
        b[m] = e[m >> 3][m & 7];
    uint32_t byte;
    const uint2 codes = quantize_block(b, global_scale_from_amax(*(key ? a.c.k_amax : a.c.v_amax)), byte);
    uint8_t* rec = a.data + (p.record + ((int64_t)kh << (a.c.page_shift - 4))) * Record<D>::kBytes;
    if (key) {
        *reinterpret_cast<uint2*>(rec + Record<D>::key_codes(p.t, j)) = codes;
        rec[Record<D>::key_scale(p.t, j)] = (uint8_t)byte;
    } else {
        uint8_t* to = rec + Record<D>::value_codes(p.t, j);
        if constexpr (D == 64) {
            uint16_t* w = reinterpret_cast<uint16_t*>(to);
            w[0] = (uint16_t)codes.x, w[4] = (uint16_t)(codes.x >> 16);
            w[8] = (uint16_t)codes.y, w[12] = (uint16_t)(codes.y >> 16);
        } else if constexpr (D == 128) {
            uint32_t* w = reinterpret_cast<uint32_t*>(to);
            w[0] = codes.x, w[4] = codes.y;
        } else {
            *reinterpret_cast<uint2*>(to) = codes;
        }
        rec[Record<D>::value_scale(p.t, j)] = (uint8_t)byte;
    }
}

// The same tiling: one 16-element block per thread, decoded as
// nvfp4_dequantize does. 8192 tokens of 2 x 8 heads of 128 to bf16: 10.4 to
// 11.4 us (43 MB, 3.8 to 4.1 TB/s).
template <class T, int D>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvReadArgs a)
{
    constexpr int kUnits = D / 16;
    const int64_t t = (int64_t)blockIdx.x * kTokens + (threadIdx.x & (kTokens - 1));
    const int slot = blockIdx.y * kSlots + threadIdx.x / kTokens;
    const int h = slot / kUnits, j = slot % kUnits;
    if (t >= a.tokens || h >= 2 * a.c.kv_heads)
        return;
    const bool key = h < a.c.kv_heads;
    const int kh = key ? h : h - a.c.kv_heads;
    char* out = static_cast<char*>(key ? a.k_out : a.v_out);
    if (out == nullptr)
        return;
    out += ((t * a.c.kv_heads + kh) * D + 16 * j) * T::kBytes;
    const int pos = a.positions[t];
    const Place p = place_of(a.c, pos, a.seq != nullptr ? a.seq[t] : (int)t);
    float v[2][8];
    if (p.there) {
        const uint8_t* rec = a.data + (p.record + ((int64_t)kh << (a.c.page_shift - 4))) * Record<D>::kBytes;
        uint32_t w[2];
        uint32_t byte;
        if (key) {
            const uint2 c = *reinterpret_cast<const uint2*>(rec + Record<D>::key_codes(p.t, j));
            w[0] = c.x, w[1] = c.y;
            byte = rec[Record<D>::key_scale(p.t, j)];
        } else {
            const uint8_t* from = rec + Record<D>::value_codes(p.t, j);
            if constexpr (D == 64) {
                const uint16_t* s = reinterpret_cast<const uint16_t*>(from);
                w[0] = s[0] | ((uint32_t)s[4] << 16), w[1] = s[8] | ((uint32_t)s[12] << 16);
            } else if constexpr (D == 128) {
                const uint32_t* s = reinterpret_cast<const uint32_t*>(from);
                w[0] = s[0], w[1] = s[4];
            } else {
                const uint2 c = *reinterpret_cast<const uint2*>(from);
                w[0] = c.x, w[1] = c.y;
            }
            byte = rec[Record<D>::value_scale(p.t, j)];
        }
        const float sg = global_scale_from_amax(*(key ? a.c.k_amax : a.c.v_amax));
        const float s = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(byte, 1.0f, false)[0];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const auto x = m == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[g], 1.0f, 0)
                               : m == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[g], 1.0f, 1)
                               : m == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[g], 1.0f, 2)
                                        : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[g], 1.0f, 3);
                v[g][2 * m] = (x[0] * s) * sg;
                v[g][2 * m + 1] = (x[1] * s) * sg;
            }
        }
    } else {
        const float fill = pos < 0 ? 0.0f : __uint_as_float(0x7FC00000u);
#pragma unroll
        for (int m = 0; m < 8; ++m)
            v[0][m] = v[1][m] = fill;
    }
    store8<T>(out, v[0]);
    store8<T>(out + 8 * T::kBytes, v[1]);
}

template <template <class, int> class Run, class... A>
hipError_t by_type_and_dim(int dtype, int head_dim, A&&... args)
{
    if (dtype == kBf16)
        return head_dim == 64    ? Run<Bf16, 64>::go(args...)
               : head_dim == 128 ? Run<Bf16, 128>::go(args...)
                                 : Run<Bf16, 256>::go(args...);
    if (dtype == kF16)
        return head_dim == 64    ? Run<F16, 64>::go(args...)
               : head_dim == 128 ? Run<F16, 128>::go(args...)
                                 : Run<F16, 256>::go(args...);
    return head_dim == 64    ? Run<F32, 64>::go(args...)
           : head_dim == 128 ? Run<F32, 128>::go(args...)
                             : Run<F32, 256>::go(args...);
}

dim3 grid_of(int64_t tokens, int64_t heads, int head_dim)
{
    const int64_t slots = heads * (head_dim / 16);
    return dim3((unsigned)((tokens + kTokens - 1) / kTokens), (unsigned)((slots + kSlots - 1) / kSlots));
}

template <class T, int D>
struct Append {
    static hipError_t go(const KvAppendArgs& a, hipStream_t stream)
    {
        const unsigned q_blocks = grid_of(a.tokens, a.heads, D).y;
        dim3 grid = grid_of(a.tokens, 2 * a.c.kv_heads, D);
        grid.y += q_blocks;
        // More rotated queries than the XCDs' L2s hold (8 x 4 MiB) are written
        // past them: they would only be pushed out, at the launch's end. Whole
        // lines are, that is, 16-bit heads of 128 and more, aligned. (8192
        // tokens of 32 x 128: 41 us, 47 through the caches; half rotated 41 and
        // 44; 4096 tokens, just the L2s' size, 24 and 23; heads of 64 elements
        // 30 and 26.)
        const bool stream_q = T::kBytes == 2 && D >= 128 && a.tokens * a.heads * D * 2 > ((int64_t)32 << 20) &&
                              (a.qo_ts | a.qo_hs) % 64 == 0 && reinterpret_cast<uintptr_t>(a.q_out) % 128 == 0;
        hipLaunchKernelGGL((kv_append_kernel<T, D>), grid, dim3(kThreads), 0, stream, a, (int)q_blocks, stream_q);
        return hipGetLastError();
    }
};

template <class T, int D>
struct Read {
    static hipError_t go(const KvReadArgs& a, hipStream_t stream)
    {
        hipLaunchKernelGGL((kv_read_kernel<T, D>), grid_of(a.tokens, 2 * a.c.kv_heads, D), dim3(kThreads), 0,
                           stream, a);
        return hipGetLastError();
    }
};

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t stream)
{
    return by_type_and_dim<Append>(a.dtype, a.c.head_dim, a, stream);
}

hipError_t launch_kv_read(const KvReadArgs& a, hipStream_t stream)
{
    return by_type_and_dim<Read>(a.dtype, a.c.head_dim, a, stream);
}

}  // namespace nvfp4
