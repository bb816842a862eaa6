// One wave's part of attention over the NVFP4 cache: 32 cached tokens at a
// time against NT tiles of 16 query rows, everything in registers.
//
// Layouts (lane l, c = l % 16, g = l / 16). Scores are formed transposed,
// S^T [token][row] = K Q^T, and so is the output, O^T [element][row] =
// V^T P^T, with v_mfma_f32_16x16x32_f16:
//  - K operand of a 16-token tile: lane holds token c, elements g D/4 ..,
//    which is 16 (D = 128) contiguous bytes of codes of the record.
//  - S^T comes out with row c in every lane, tokens 4 g + i: two tiles give a
//    lane 8 weights of one row, which is the P^T operand of the second
//    product as it stands (its 8 K-elements are the tokens 4 g + i of both
//    tiles). No exchange between lanes, and every statistic of a row is a
//    scalar per lane.
//  - V^T operand: lane holds the elements c D/16 .. of the same 8 tokens; a
//    record keeps those of 4 tokens together, and their scales too. The
//    nibbles of two tokens are paired by shift and bit-select before they are
//    converted, so that a convert gives two tokens of one element.
//  - O^T: lane holds row c, elements g D/4 + i D/16 + n of product n.
// Codes are decoded exactly (e2m1 * e4m3 is a binary16 value): one convert
// and one packed multiply per two codes.
//
// The softmax is a running one: with m the maximum so far, a part of the
// tokens gives l = sum exp2(s - m) and o = sum exp2(s - m) v, and parts join
// as l = l1 exp2(m1 - m) + l2 exp2(m2 - m), o likewise, so that every cached
// byte is read once. m, l and o are binary32. The weights are rounded to
// binary16 for their product with the values: the values are exact in it, the
// matrix cores take both operands in one type, and 11 bits of a weight are 3
// more than the output's in bf16 and as many as it has in f16.
#pragma once

#include "heads.h"

namespace nvfp4 {

typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(4))) float floatx4;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

// Weights are kept as 2^kBias exp2(s - m): a row's running maximum m is
// raised only when a score passes it by kSlack (in log2), so a weight is at
// most 2^(kBias + kSlack) = 2^14, inside binary16, and a weight is held to
// its 11 bits down to 2^-20 of the maximum's.
constexpr float kBias = 6.0f;
constexpr float kSlack = 8.0f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xFF800000u); }

// Maximum (sum) over the four lanes that share l % 16.
__device__ __forceinline__ float across16_max(float v)
{
    const uint32_t u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t w = __float_as_uint(fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1])));
    const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float across16_sum(float v)
{
    const uint32_t u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t w = __float_as_uint(__uint_as_float(a[0]) + __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Two codes (byte SEL of w) times a pair of scales.
template <int SEL>
__device__ __forceinline__ f16x2_t decode2(uint32_t w, f16x2_t s)
{
    return __builtin_bit_cast(f16x2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, SEL)) * s;
}
__device__ __forceinline__ f16x2_t decode2(uint32_t w, int sel, f16x2_t s)
{
    return sel == 0 ? decode2<0>(w, s) : sel == 1 ? decode2<1>(w, s) : sel == 2 ? decode2<2>(w, s) : decode2<3>(w, s);
}

// Two E4M3 bytes (the low or the high half of w) as binary16.
template <bool HIGH>
__device__ __forceinline__ f16x2_t scales2(uint32_t w)
{
    return __builtin_bit_cast(f16x2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HIGH));
}

__device__ __forceinline__ f16x8 join8(f16x2_t a, f16x2_t b, f16x2_t c, f16x2_t d)
{
    return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A lane's part of one record.
template <int D>
struct Tile {
    uint32_t k[D / 32];  // token c's key codes, elements g D/4 ..
    uint32_t v[D / 32];  // tokens 4 g .. + 3, elements c D/16 ..: [token][D / 128 words] (D = 64: half words)
    uint32_t ks;         // D / 64 scale bytes
    uint32_t vs;         // the four tokens' scales of the lane's block
};

template <int D>
__device__ __forceinline__ Tile<D> load_tile(const uint8_t* rec, int lane)
{
    const int c = lane & 15, g = lane >> 4;
    Tile<D> t;
    const uint8_t* kp = rec + lane * (D / 8);
    const uint8_t* vp = rec + Record<D>::kValueCodes + lane * (D / 8);
    if constexpr (D == 64) {
        const uint2 a = *reinterpret_cast<const uint2*>(kp), b = *reinterpret_cast<const uint2*>(vp);
        t.k[0] = a.x, t.k[1] = a.y;
        t.v[0] = b.x, t.v[1] = b.y;
        t.ks = rec[Record<D>::kKeyScales + lane];
    } else {
#pragma unroll
        for (int i = 0; i < D / 128; ++i) {
            const uint4 a = load16(kp + 16 * i), b = load16(vp + 16 * i);
            t.k[4 * i] = a.x, t.k[4 * i + 1] = a.y, t.k[4 * i + 2] = a.z, t.k[4 * i + 3] = a.w;
            t.v[4 * i] = b.x, t.v[4 * i + 1] = b.y, t.v[4 * i + 2] = b.z, t.v[4 * i + 3] = b.w;
        }
        if constexpr (D == 128)
            t.ks = *reinterpret_cast<const uint16_t*>(rec + Record<D>::kKeyScales + 2 * lane);
        else
            t.ks = *reinterpret_cast<const uint32_t*>(rec + Record<D>::kKeyScales + 4 * lane);
    }
    t.vs = *reinterpret_cast<const uint32_t*>(rec + Record<D>::kValueScales + (c * D / 256) * 16 + 4 * g);
    return t;
}

// The nibbles of tokens (0, 1) and (2, 3) of a tile side by side: byte b of
// word w holds two tokens' codes of one element, where it belongs as
// pair_word / pair_byte say.
template <int D>
__device__ __forceinline__ void pair_tokens(const uint32_t (&v)[D / 32], uint32_t (&out)[D / 32])
{
    constexpr uint32_t kLow = 0x0F0F0F0Fu;
    auto lo = [](uint32_t a, uint32_t b) { return (a & kLow) | ((b << 4) & ~kLow); };
    auto hi = [](uint32_t a, uint32_t b) { return ((a >> 4) & kLow) | (b & ~kLow); };
    if constexpr (D == 64) {
        // word 0: tokens 0 | 1 << 16, word 1: tokens 2 | 3 << 16
        const uint32_t a = __builtin_amdgcn_perm(v[1], v[0], 0x05040100u);  // tokens 0 and 2
        const uint32_t b = __builtin_amdgcn_perm(v[1], v[0], 0x07060302u);  // tokens 1 and 3
        out[0] = lo(a, b);
        out[1] = hi(a, b);
    } else {
        constexpr int W = D / 128;  // words of a token
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int w = 0; w < W; ++w) {
                out[2 * (W * p + w)] = lo(v[2 * p * W + w], v[(2 * p + 1) * W + w]);
                out[2 * (W * p + w) + 1] = hi(v[2 * p * W + w], v[(2 * p + 1) * W + w]);
            }
    }
}
template <int D>
constexpr int pair_word(int p, int n)
{
    return D == 64 ? (n & 1) : 2 * ((D / 128) * p + (n >> 3)) + (n & 1);
}
template <int D>
constexpr int pair_byte(int p, int n)
{
    return D == 64 ? 2 * p + (n >> 1) : (n & 7) >> 1;
}

// What a lane's rows see: token t is seen by row c of tile n when
// lo[n] <= t < hi[n].
template <int NT>
struct Sight {
    int lo[NT], hi[NT];
};

template <int D, int NT>
struct Rows {
    f16x8 q[NT][D / 32];
    float f[NT];   // log2 of a weight per unit of the raw product
    float m[NT];   // the running maximum times f (log2), -inf before the first token
    float l[NT];   // this lane's part of the sum of weights
    floatx4 o[NT][D / 16];
};

// This lane's part of 16 NT query rows as they lie in memory: rows r0 .. of
// the kv head's (token r / G, head r % G; rows: how many there are).
template <int D, int NT>
struct RawRows {
    uint4 v[NT][D / 32];
};

template <int D, int NT>
__device__ __forceinline__ void load_rows(RawRows<D, NT>& raw, const KvAttentionArgs& a, int64_t q0, int kv_head,
                                          int r0, int rows, int G, int lane)
{
    const int c = lane & 15, g = lane >> 4;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = r0 + 16 * n + c;
        const int tok = r < rows ? r / G : 0;
        const char* p = static_cast<const char*>(a.q) +
                        ((q0 + tok) * a.q_ts + (kv_head * G + r - tok * G) * a.q_hs + g * (D / 4)) * 2;
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
            raw.v[n][k] = r < rows ? load16(p + 16 * k) : make_uint4(0u, 0u, 0u, 0u);
    }
}

// The largest |element| of 16-bit words, as its bits (their order is the
// magnitudes'; a NaN's are above infinity's).
template <int N>
__device__ __forceinline__ uint32_t top_bits(const uint4 (&raw)[N])
{
    uint32_t bits = 0u;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            bits = pk_max_u16(bits, word_at(raw[k], j) & 0x7FFF7FFFu);
    return max(bits >> 16, bits & 0xFFFFu);
}

// Infinite elements become NaN (x 0 + x): they leave no finite score, so that the
// softmax is NaN; as -inf such scores would be taken for those of masked tokens.
// (A row that sees nothing gives 0 all the same.) BF16 rows get their NaN with
// their scaling.
__device__ __forceinline__ f16x8 nan_for_infinity(uint4 raw)
{
    const f16x8 x = __builtin_bit_cast(f16x8, raw);
    return __builtin_elementwise_fma(x, (f16x8)(_Float16)0.0f, x);
}

template <class T, int D, int NT>
__device__ __forceinline__ void start_rows(Rows<D, NT>& w, const RawRows<D, NT>& raw, const KvAttentionArgs& a)
{
    const float sg = global_scale_from_amax(*a.c.k_amax);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        w.f[n] = a.scale * kLog2e * sg;
        if constexpr (__is_same(T, Bf16)) {
            // The row is brought to binary16's range by a power of two that
            // puts its largest element into [2^13, 2^14): 8 bits fit down to
            // 2^-17, that is 2^-30 of the largest; smaller elements are rounded
            // to multiples of 2^-24. The inverse goes into the logits' factor.
            const float top = across16_max(__uint_as_float(top_bits(raw.v[n]) << 16));
            int e = (int)((__float_as_uint(top) >> 23) & 255u) - 127;  // floor(log2) of a normal number
            e = min(max(13 - e, -126), 126);
            const bool scale = top > 0.0f && top < __uint_as_float(0x7F800000u);
            const float up = scale ? __uint_as_float((uint32_t)(e + 127) << 23) : top == 0.0f ? 1.0f : __uint_as_float(0x7FC00000u);
            w.f[n] *= scale ? __uint_as_float((uint32_t)(127 - e) << 23) : 1.0f;
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w.q[n][k][j] = (_Float16)(bf16_at(raw.v[n][k], j) * up);
        } else {
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
                w.q[n][k] = nan_for_infinity(raw.v[n][k]);
        }
        w.m[n] = neg_inf();
        w.l[n] = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            w.o[n][i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    }
}

// The bytes of a word of E4M3 scales that are NaN, one bit each (bit 7 of
// the byte).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t s)
{
    return ((s & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// 32 tokens from t0 on. masked (uniform): some row does not see some of them
// (tokens past the end, before a window, after a query, in a hole): `sight`
// says which; there[u] is whether tile u is in the cache at all.
template <int D, int NT>
__device__ __forceinline__ void attend(Rows<D, NT>& w, const Tile<D> (&tile)[2], int t0, const Sight<NT>& sight,
                                       int seen_lo, int seen_hi, const bool (&there)[2], bool masked, int lane)
{
    const int g = lane >> 4;
    floatx4 s[NT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        f16x2_t sc[D / 64];
        if constexpr (D == 64) {
            const f16x2_t a = scales2<false>(tile[u].ks);
            sc[0] = f16x2_t{a[0], a[0]};
        } else {
            const f16x2_t a = scales2<false>(tile[u].ks);
            sc[0] = f16x2_t{a[0], a[0]}, sc[1] = f16x2_t{a[1], a[1]};
            if constexpr (D == 256) {
                const f16x2_t b = scales2<true>(tile[u].ks);
                sc[2] = f16x2_t{b[0], b[0]}, sc[3] = f16x2_t{b[1], b[1]};
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
            s[n][u] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
            const uint32_t x = tile[u].k[k];
            const f16x2_t e = sc[k >> 1];
            const f16x8 kf = join8(decode2<0>(x, e), decode2<1>(x, e), decode2<2>(x, e), decode2<3>(x, e));
#pragma unroll
            for (int n = 0; n < NT; ++n)
                s[n][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, w.q[n][k], s[n][u], 0, 0, 0);
        }
    }

    // Weights. A row's maximum is raised only when it is passed by more than
    // kSlack (or when there is none yet): what was summed is then rescaled.
    f16x8 p[NT];
    uint32_t attended[NT];  // masked: bit 4 u + i, this lane's row sees token 16 u + 4 g + i
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        attended[n] = 0u;
        if (masked) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = t0 + 16 * u + 4 * g + i;
                    const bool ok = there[u] && t >= sight.lo[n] && t < sight.hi[n];
                    attended[n] |= ok ? 1u << (4 * u + i) : 0u;
                    s[n][u][i] = ok ? s[n][u][i] : neg_inf();
                }
        }
        // Scores in log2. (The product comes first: it leaves the maximum with
        // operands that are known to be in canonical form.)
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            e[i] = s[n][i >> 2][i & 3] * w.f[n];
        float top = fmaxf(fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3])), fmaxf(fmaxf(e[4], e[5]), fmaxf(e[6], e[7])));
        // -inf times an f of 0 is NaN, and a row that sees nothing here has
        // no say: both leave the comparison false.
        if (__any(top > w.m[n] + kSlack)) {
            top = across16_max(top);
            const bool raise = top > w.m[n];
            const float down = raise ? __builtin_amdgcn_exp2f(w.m[n] - top) : 1.0f;
            w.m[n] = raise ? top : w.m[n];
            w.l[n] *= down;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                w.o[n][i] *= down;
        }
        // A row that has seen nothing yet has only -inf scores here.
        const float base = kBias - (w.m[n] == neg_inf() ? 0.0f : w.m[n]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            e[i] = __builtin_amdgcn_exp2f(e[i] + base);
        if (masked) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                e[i] = (attended[n] >> i) & 1u ? e[i] : 0.0f;
        }
        w.l[n] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            p[n][i] = (_Float16)e[i];
    }

    uint32_t vs[2] = {tile[0].vs, tile[1].vs};
    if (masked) {
        // Tokens that no row sees may hold anything: their scales become 0.
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = t0 + 16 * u + 4 * g + i;
                if (!there[u] || t < seen_lo || t >= seen_hi)
                    vs[u] &= ~(0xFFu << (8 * i));
            }
        // A value that is NaN reaches the rows that see its token and no
        // other: it is left out of the product (0 times NaN is NaN), and the
        // rows that see it get their NaN by themselves.
        const uint32_t bad[2] = {nan_bytes(vs[0]), nan_bytes(vs[1])};
        if (__any((bad[0] | bad[1]) != 0u)) {
            f16x8 which;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                which[i] = (bad[i >> 2] >> (8 * (i & 3))) & 0x80u ? (_Float16)1.0f : (_Float16)0.0f;
#pragma unroll
            for (int u = 0; u < 2; ++u)
                vs[u] &= ~((bad[u] >> 7) * 0xFFu);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                f16x8 sees;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    sees[i] = (attended[n] >> i) & 1u ? (_Float16)1.0f : (_Float16)0.0f;
                const floatx4 hit = __builtin_amdgcn_mfma_f32_16x16x32_f16(which, sees, floatx4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
#pragma unroll
                for (int x = 0; x < D / 16; ++x)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w.o[n][x][i] = hit[i] > 0.0f ? __uint_as_float(0x7FC00000u) : w.o[n][x][i];
            }
        }
    }
    uint32_t pv[2][D / 32];
    pair_tokens<D>(tile[0].v, pv[0]);
    pair_tokens<D>(tile[1].v, pv[1]);
    const f16x2_t sv[2][2] = {{scales2<false>(vs[0]), scales2<true>(vs[0])},
                              {scales2<false>(vs[1]), scales2<true>(vs[1])}};
#pragma unroll
    for (int x = 0; x < D / 16; ++x) {
        const f16x8 vf = join8(decode2(pv[0][pair_word<D>(0, x)], pair_byte<D>(0, x), sv[0][0]),
                               decode2(pv[0][pair_word<D>(1, x)], pair_byte<D>(1, x), sv[0][1]),
                               decode2(pv[1][pair_word<D>(0, x)], pair_byte<D>(0, x), sv[1][0]),
                               decode2(pv[1][pair_word<D>(1, x)], pair_byte<D>(1, x), sv[1][1]));
#pragma unroll
        for (int n = 0; n < NT; ++n)
            w.o[n][x] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, p[n], w.o[n][x], 0, 0, 0);
    }
}

}  // namespace nvfp4
