// Attention over the NVFP4 key/value cache for many query rows per sequence:
// prompts and chunks of prompts. See include/nvfp4_kv.h for the contract.
//
// A workgroup holds 32 query rows per wave (rows of one kv head: the G heads
// of a token side by side) and walks the cached tokens in steps of 32. Its
// threads decode the keys and values once, exactly, to binary16 in LDS, a
// stage (one record of 16 tokens per wave) at a time, and every wave
// multiplies them with its rows on v_mfma_f32_32x32x16_f16:
//  - scores transposed, S^T [token][row] = K Q^T: a row is a lane (l % 32),
//    its tokens the two lanes that share it, so a row's statistics are a
//    scalar per lane and one exchange;
//  - the weights are the second product's operand as they stand: O^T = V^T
//    P^T, whose K-elements of a lane are the tokens that the lane's registers
//    hold (4 h .. and 8 + 4 h .. of 16, h = l / 32).
// LDS holds both operands in chunks of 16 bytes, the 32 lanes that share a
// chunk side by side, so fragment reads are contiguous (no conflicts). V^T's
// rows are the elements c D/16 + x in the order x 16 + c: what a decoding
// lane has (c fixed, x running) then goes to consecutive 16-byte slots across
// the lanes, and the output's elements of a lane come out contiguous.
//
// Per step the weights cost about as many vector cycles (an exponential is
// eight) as the products cost matrix cycles, so neither may wait for the
// other: in step h a wave turns the scores of step h into weights while the
// matrix cores form the scores of step h + 1 and add the values of step
// h - 1, all in one stretch of code without a branch. Steps at the edges
// (masked, first, last) take the same operations one after the other.
//
// The products bound it. 8192 tokens, 32 heads of 128 over 8, causal: 508 to 539
// us by card, 1.02 to 1.08 PFLOP/s of the pairs that are seen (a large library matrix product
// reaches 1.36 in bf16 and 1.22 in f16), matrix cores and vector units busy in
// 52 % of the cycles each, at the 1.9 GHz that the power allows; 2048 tokens
// over 8192: 231 to 251 us, 0.96 to 1.04 PFLOP/s (one workgroup for each compute unit, whose
// rows see 6144 to 8192 tokens: the last are waited for); 4096 tokens, 16 heads
// of 256: 172 us, 800 TFLOP/s. The same products, loads and weights one after
// the other took 700 us for the first.
#include <atomic>

#include "kv_parts.h"

namespace nvfp4 {

namespace {

typedef __attribute__((ext_vector_type(16))) float floatx16;
typedef __attribute__((ext_vector_type(4))) _Float16 f16x4;

// The weights of a step are formed with the maximum known before it; where a
// lane's 16 come to more than this together, one may pass binary16's range.
constexpr float kMost = 32768.0f;

// H steps of 32 tokens are a stage. Three buffers each for keys and values:
// in stage n the keys of stages n and n + 1 and the values of stages n - 1 and
// n are read, and keys n + 2 and values n + 1 are written.
template <int D, int W>
struct Stages {
    static constexpr int H = D == 256 ? 1 : 2;
    static constexpr int kTokens = 32 * H;
    static constexpr int kTiles = 2 * H;
    static constexpr int kBytes = kTokens * D * 2;
    static constexpr int kRows = 32 * W;
    static constexpr size_t kSlotFloats = (size_t)kRows * (D + 2);
    alignas(16) uint8_t keys[3][kBytes];
    alignas(16) uint8_t values[3][kBytes];
    uint32_t holes[3];  // number + 1 of the last stage in this buffer that is not wholly in the cache
    uint32_t nans;      // whether there were NaN values that some row does not see
};

__device__ __forceinline__ float halves_max(float v)
{
    const uint32_t u = __float_as_uint(v);
    const auto b = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float halves_sum(float v)
{
    const uint32_t u = __float_as_uint(v);
    const auto b = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

template <int D>
__device__ __forceinline__ void load_codes(uint32_t (&w)[D / 32], const uint8_t* p)
{
    if constexpr (D == 64) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        w[0] = x.x, w[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < D / 128; ++i) {
            const uint4 x = load16(p + 16 * i);
            w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
        }
    }
}

// Decodes a lane's keys (token c of record `tile`, elements g D/4 ..) to LDS.
template <int D>
__device__ __forceinline__ void keys_to_lds(uint8_t* keys, const uint32_t (&w)[D / 32], uint32_t scales, int tile, int lane)
{
    constexpr int kTokens = Stages<D, 8>::kTokens;
    const int c = lane & 15, g = lane >> 4;
    f16x2_t sc[D / 64];
    const f16x2_t a = scales2<false>(scales);
    sc[0] = f16x2_t{a[0], a[0]};
    if constexpr (D >= 128)
        sc[1] = f16x2_t{a[1], a[1]};
    if constexpr (D == 256) {
        const f16x2_t b = scales2<true>(scales);
        sc[2] = f16x2_t{b[0], b[0]}, sc[3] = f16x2_t{b[1], b[1]};
    }
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
        const f16x2_t e = sc[k >> 1];
        const f16x8 x = join8(decode2<0>(w[k], e), decode2<1>(w[k], e), decode2<2>(w[k], e), decode2<3>(w[k], e));
        *reinterpret_cast<f16x8*>(keys + ((g * (D / 32) + k) * kTokens + 16 * tile + c) * 16) = x;
    }
}

// ... and a lane's values (tokens 4 g .., elements c D/16 ..).
template <int D>
__device__ __forceinline__ void values_to_lds(uint8_t* values, const uint32_t (&w)[D / 32], uint32_t scales, int tile,
                                              int lane)
{
    const int c = lane & 15, g = lane >> 4;
    uint32_t p[D / 32];
    pair_tokens<D>(w, p);
    const f16x2_t s0 = scales2<false>(scales), s1 = scales2<true>(scales);
    uint8_t* const to = values + ((2 * tile + (g & 1)) * D + c) * 16 + (g >> 1) * 8;
#pragma unroll
    for (int x = 0; x < D / 16; ++x) {
        const f16x2_t a = decode2(p[pair_word<D>(0, x)], pair_byte<D>(0, x), s0);
        const f16x2_t b = decode2(p[pair_word<D>(1, x)], pair_byte<D>(1, x), s1);
        *reinterpret_cast<f16x4*>(to + x * 256) = f16x4{a[0], a[1], b[0], b[1]};
    }
}

// The largest of 16 scores. (maximum, not fmax: it takes the products'
// results as they are, and a NaN may come out, which no comparison lets in.)
__device__ __forceinline__ float max16(const floatx16& s)
{
    float a = __builtin_elementwise_maximum(__builtin_elementwise_maximum(s[0], s[1]), s[2]);
    float b = __builtin_elementwise_maximum(__builtin_elementwise_maximum(s[3], s[4]), s[5]);
#pragma unroll
    for (int i = 6; i < 14; i += 4) {
        a = __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, s[i]), s[i + 1]);
        b = __builtin_elementwise_maximum(__builtin_elementwise_maximum(b, s[i + 2]), s[i + 3]);
    }
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), __builtin_elementwise_maximum(s[14], s[15]));
}

// What a workgroup has to do: rows r0 .. r1 of a (sequence, kv head), and the
// tokens that they see between them in `stages` stages from base0 on, split
// into `parts` stretches.
struct Piece {
    Seq s;
    int b, kh, rows, r0, r1;
    int seen_lo, seen_hi, base0, stages, parts;
};

// Stages that a part has at least. (4 or 8: 150 queries over 3212 tokens 36 or
// 41 us where 2 take 31, 64 over 1710 21.5 or 26 where 2 take 21.)
constexpr int kMinStages = 2;

// Heads run fastest (with 8 of them each XCD keeps one head's cache in its
// L2), then a sequence's rows, those with the most tokens to see first, then
// sequences. (Workgroups go to the chip's engines in turn, so that sequences
// side by side would each stay on some of them: four prompts of 2000 tokens 193
// us that way, 144 so; 16 short ones of 250 to 500 tokens 53 and 60, for their
// longest rows do not all come first.)
template <int D, int W>
__device__ __forceinline__ Piece piece_of(const KvAttentionArgs& a, int id, int row_tiles, int parts_most)
{
    typedef Stages<D, W> St;
    const int G = a.heads / a.c.kv_heads;
    Piece p;
    p.kh = id % a.c.kv_heads;
    id /= a.c.kv_heads;
    p.b = id / row_tiles;
    p.r0 = (row_tiles - 1 - (id - p.b * row_tiles)) * St::kRows;
    p.s = seq_of(a, p.b);
    p.rows = p.s.nq * G;
    p.r1 = min(p.r0 + St::kRows, p.rows) - 1;
    p.seen_lo = first_seen(a, p.s, p.r0 / G);
    p.seen_hi = end_seen(a, p.s, p.r1 / G);
    p.base0 = p.seen_lo & ~15;
    p.stages = max(1, (p.seen_hi - p.base0 + St::kTokens - 1) / St::kTokens);
    p.parts = max(1, min(parts_most, p.stages / kMinStages));
    return p;
}

// Partial results, as the lanes hold them: [wave][D / 32][4][lane] of 4
// elements, then a maximum and a sum for each row.
template <int D, int W>
__device__ __forceinline__ float* slot_of(const KvAttentionArgs& a, int item, int parts_most, int part)
{
    return reinterpret_cast<float*>(reinterpret_cast<char*>(a.workspace) + kCounterBytes) +
           ((size_t)item * parts_most + part) * Stages<D, W>::kSlotFloats;
}

template <class T, int D, int W>
__global__ __launch_bounds__(64 * W) void kv_prompt_kernel(KvAttentionArgs a, int row_tiles, int parts_most)
{
    typedef Stages<D, W> St;
    constexpr int H = St::H, kTokens = St::kTokens, kTiles = St::kTiles;
    static_assert(W >= 2 * kTiles, "a wave decodes the keys or the values of one record of a stage");
    __shared__ St lds;
    const int lane = threadIdx.x & 63;
    const int wave = uniform((int)threadIdx.x >> 6);
    const int q = lane & 31, h2 = lane >> 5;
    const int G = a.heads / a.c.kv_heads;
    const Piece piece = piece_of<D, W>(a, blockIdx.x, row_tiles, parts_most);
    const Seq& s = piece.s;
    const int b = piece.b, kh = piece.kh, rows = piece.rows, r0 = piece.r0, r1 = piece.r1, parts = piece.parts;
    const int part = blockIdx.y;
    if (s.past > 0 && part == 0 && r0 == 0)
        write_past<T, D>(a, s, kh, G, 64 * W);
    if (r0 >= rows || part >= parts)
        return;
    const int seen_lo = piece.seen_lo, seen_hi = piece.seen_hi;
    const int all_lo = first_seen(a, s, r1 / G), all_hi = end_seen(a, s, r0 / G);
    // Its stages: stretches that differ by one at most.
    const int each = piece.stages / parts, more = piece.stages - each * parts;
    const int stages = each + (part < more ? 1 : 0);
    const int base = piece.base0 + (part * each + min(part, more)) * kTokens;

    // This wave's rows, and what they see of the tokens: lane by lane, and
    // (uniform) what all of them see.
    const int rw = r0 + 32 * wave;
    const bool active = rw < rows;  // a wave without rows only decodes
    const int row = min(rw + q, rows - 1);
    const int lo = first_seen(a, s, row / G), hi = end_seen(a, s, row / G);
    const int w_all_lo = first_seen(a, s, min(rw + 31, rows - 1) / G), w_all_hi = end_seen(a, s, min(rw, rows - 1) / G);
    uint4 raw_q[D / 16];
    {
        const int tok = row / G;
        const char* p = static_cast<const char*>(a.q) + ((s.q0 + tok) * a.q_ts + (kh * G + row - tok * G) * a.q_hs + 8 * h2) * 2;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
            raw_q[k] = load16(p + 32 * k);
    }

    const int32_t* pages = a.c.page_table + (int64_t)b * a.c.table_stride;
    const int tile_mask = (1 << (a.c.page_shift - 4)) - 1;
    const int mine = wave & (kTiles - 1);  // the wave's record of a stage
    const bool decodes = wave < 2 * kTiles;  // of 12 waves, the first 8
    const bool has_keys = wave < kTiles;   // it decodes keys, or values
    // The page of a token, -1 for a hole and for a token that no row sees.
    const auto page_at = [&](int t) {
        const int p = t < seen_hi ? pages[t >> a.c.page_shift] : -1;
        return (uint32_t)p < (uint32_t)a.c.num_pages ? p : -1;
    };
    // The wave's record of a stage: its codes and scales as they lie in memory.
    // Lane i holds the page of the record of stage 64 j + i, so that the loop
    // reads the page table once in 64 stages.
    uint32_t codes[D / 32], scales = 0u;
    int page = -1, page_lanes = -1;
    const uint32_t code_at = (has_keys ? 0 : Record<D>::kValueCodes) + lane * (D / 8);
    const uint32_t scale_at = has_keys ? Record<D>::kKeyScales + lane * (D / 64)
                                       : Record<D>::kValueScales + ((lane & 15) * D / 256) * 16 + 4 * (lane >> 4);
    const auto fetch = [&](int n) {
        if (!decodes)
            return;
        if ((n & 63) == 0)
            page_lanes = page_at(base + min(n + lane, stages) * kTokens + 16 * mine);
        page = __builtin_amdgcn_readlane(page_lanes, n & 63);
        const int t = base + n * kTokens + 16 * mine;
        const int64_t rec = (((int64_t)max(page, 0) * a.c.kv_heads + kh) << (a.c.page_shift - 4)) + ((t >> 4) & tile_mask);
        const uint8_t* p = a.data + rec * Record<D>::kBytes;  // uniform; the lane's part is a 32-bit offset
        load_codes<D>(codes, p + code_at);
        if (has_keys)
            scales = D == 64    ? *reinterpret_cast<const uint8_t*>(p + scale_at)
                     : D == 128 ? *reinterpret_cast<const uint16_t*>(p + scale_at)
                                : *reinterpret_cast<const uint32_t*>(p + scale_at);
        else
            scales = *reinterpret_cast<const uint32_t*>(p + scale_at);
    };
    // ... decoded into buffer `slot`.
    const auto decode = [&](int n, int slot) {
        if (!decodes)
            return;
        const int t = base + n * kTokens + 16 * mine;
        if (t < all_lo || t + 16 > all_hi || page < 0) {
            // Some row does not see some of these tokens. Those that no row
            // sees may hold anything: their scales become 0. NaN values of the
            // others are left out and put in at the end. (Any number of lanes
            // may write a flag, all the same value.)
            if (has_keys) {
                if (t + (lane & 15) < seen_lo || t + (lane & 15) >= seen_hi)
                    scales = 0u;
                else if (page < 0) {
                    scales = ~0u;  // NaN scores: the step finds out why
                    lds.holes[slot] = (uint32_t)n + 1u;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int u = t + 4 * (lane >> 4) + i;
                    if (page < 0 || u < seen_lo || u >= seen_hi)
                        scales &= ~(0xFFu << (8 * i));
                }
                const uint32_t bad = nan_bytes(scales);
                scales &= ~((bad >> 7) * 0xFFu);
                if (bad != 0u)
                    lds.nans = 1u;
            }
        }
        if (has_keys)
            keys_to_lds<D>(lds.keys[slot], codes, scales, mine, lane);
        else
            values_to_lds<D>(lds.values[slot], codes, scales, mine, lane);
    };

    if (threadIdx.x < 3)
        lds.holes[threadIdx.x] = 0u;
    if (threadIdx.x == 0)
        lds.nans = 0u;
    fetch(0);

    // The rows in binary16 (a BF16 row scaled by a power of two, infinities NaN, as
    // in kv_stream.h).
    f16x8 qf[D / 16];
    float f = a.scale * kLog2e * global_scale_from_amax(*a.c.k_amax);
    if constexpr (__is_same(T, Bf16)) {
        const float top = halves_max(__uint_as_float(top_bits(raw_q) << 16));
        int e = (int)((__float_as_uint(top) >> 23) & 255u) - 127;
        e = min(max(13 - e, -126), 126);
        const bool scale = top > 0.0f && top < __uint_as_float(0x7F800000u);
        const float up = scale ? __uint_as_float((uint32_t)(e + 127) << 23) : top == 0.0f ? 1.0f : __uint_as_float(0x7FC00000u);
        f *= scale ? __uint_as_float((uint32_t)(127 - e) << 23) : 1.0f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                qf[k][j] = (_Float16)(bf16_at(raw_q[k], j) * up);
    } else {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
            qf[k] = nan_for_infinity(raw_q[k]);
    }
    float m = neg_inf(), l = 0.0f;
    floatx16 o[D / 32];
#pragma unroll
    for (int x = 0; x < D / 32; ++x)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            o[x][i] = 0.0f;

    // Keys run a stage further ahead than values do.
    __syncthreads();  // lds.holes, lds.nans
    decode(0, 0);
    if (stages > 1) {
        fetch(1);
        if (has_keys) {
            decode(1, 1);
            if (stages > 2)
                fetch(2);
        }
    }
    __syncthreads();

    // Where a lane's fragments lie in a buffer.
    const uint32_t key_lane = (h2 * kTokens + q) * 16, value_lane = (h2 * D + q) * 16;
    const auto key_frag = [&](int slot, int half, int k) {
        return *reinterpret_cast<const f16x8*>(&lds.keys[0][0] + (slot * St::kBytes + half * 512 + key_lane) +
                                               2 * k * kTokens * 16);
    };
    const auto value_frag = [&](int slot, int half, int y, int x) {
        return *reinterpret_cast<const f16x8*>(&lds.values[0][0] + (slot * St::kBytes + half * 4 * D * 16 + value_lane) +
                                               (2 * y * D + 32 * x) * 16);
    };

    bool ready = false;  // every row has a maximum
    // The first fragments of a step are read at the end of the one before: the
    // loads' latency is under way while that one decides on its weights.
    // (Not across a stage of one step: its next keys come with the barrier.)
    constexpr int kTurns = D / 16, kDeep = 2, kEarly = H == 2 ? kDeep : 0;
    f16x8 kf[kTurns + kEarly], vf[kTurns + kEarly];
    const auto read = [&](int k, int ks, int kh2, int vs, int vh, int at) {
        vf[at] = value_frag(vs, vh, k / (D / 32), k % (D / 32));
        kf[at] = key_frag(ks, kh2, k);
    };
    // The step at token t0 (of stage n, whose keys are in buffer `own`):
    // weights from sc (its scores) to p; scores of the next step's keys (buffer
    // ks, half kh2) to sn; the last step's values (buffer vs, half vh) with
    // their weights pp to o. ks2 .. vh2: the same of the step after. The first
    // step has weights of 0 for values that are there, and the last one reads
    // keys that are not (scores that nothing is made of).
    const auto step = [&](int t0, int n, int own, int ks, int kh2, int vs, int vh, int ks2, int kh3, int vs2, int vh2,
                          floatx16& sc, floatx16& sn, f16x8 (&pp)[2], f16x8 (&p)[2]) {
        const bool masked = t0 < w_all_lo || t0 + 32 > w_all_hi;
        const float shift = kBias - m;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            sn[i] = 0.0f;
        // 16 elements of D at a time: the fragments kDeep turns on are read,
        // then two products, each with its share of the weights' arithmetic
        // to fill its cycles.
        float e[16], sum[2] = {0.0f, 0.0f};
        // At raised priority: of the two waves of a SIMD the one with products to
        // issue goes first, the other's decoding fills in (533 -> 523 us).
        __builtin_amdgcn_s_setprio(1);
        const auto weigh = [&](int i) { e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i], f, shift)); };
        // The first turn has none: the last scores are still on their way.
        constexpr auto turn_of = [](int i) { return 1 + (i / 2) * (kTurns - 1) / 8; };
        uint32_t pairs[8];
        const auto keep = [&](int i) {  // weights i and i + 1
            sum[0] += e[i];
            sum[1] += e[i + 1];
            pairs[i >> 1] = __builtin_bit_cast(uint32_t, f16x2_t{(_Float16)e[i], (_Float16)e[i + 1]});
            asm volatile("" : "+v"(pairs[i >> 1]), "+v"(sum[0]), "+v"(sum[1]));  // here, not past the branch below
        };
#pragma unroll
        for (int k = kEarly; k < kDeep; ++k)
            read(k, ks, kh2, vs, vh, k);
#pragma unroll
        for (int k = 0; k < kTurns; ++k) {
            if (k + kDeep < kTurns)
                read(k + kDeep, ks, kh2, vs, vh, k + kDeep);
            else if (k + kDeep - kTurns < kEarly)
                read(k + kDeep - kTurns, ks2, kh3, vs2, vh2, k + kDeep);
            const int x = k % (D / 32);
            o[x] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[k], pp[k / (D / 32)], o[x], 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 16; i += 2)
                if (turn_of(i) == k)
                    weigh(i);
            __builtin_amdgcn_sched_barrier(0);  // the turns stay in this order
            sn = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf[k], qf[k], sn, 0, 0, 0);
#pragma unroll
            for (int i = 1; i < 16; i += 2)
                if (turn_of(i) == k)
                    weigh(i);
#pragma unroll
            for (int i = 0; i < 16; i += 2)
                if (turn_of(i + 1) == k - 1)
                    keep(i);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < 16; i += 2)
            if (turn_of(i + 1) == kTurns - 1)
                keep(i);
#pragma unroll
        for (int y = 0; y < 2; ++y)
            p[y] = __builtin_bit_cast(f16x8, u32x4{pairs[4 * y], pairs[4 * y + 1], pairs[4 * y + 2], pairs[4 * y + 3]});
#pragma unroll
        for (int k = 0; k < kEarly; ++k) {
            kf[k] = kf[kTurns + k];
            vf[k] = vf[kTurns + k];
        }
        __builtin_amdgcn_s_setprio(0);
        float total = sum[0] + sum[1];
        if (masked || !ready || __any(!(total <= kMost))) {
            // Some row does not see all of the tokens (there is a hole), has no
            // maximum yet, or has passed its maximum by so much that a weight
            // could leave binary16: the weights again, from the maximum of
            // what is seen. (-inf times an f of 0 is NaN, which raises
            // nothing.)
            // Register i is token 8 (i / 4) + 4 h2 + i % 4 of the step.
            uint32_t there = 3u;  // which of the step's two records are in the cache
            if (uniform((int)lds.holes[own]) == n + 1)
                there = (page_at(t0) >= 0 ? 1u : 0u) | (page_at(t0 + 16) >= 0 ? 2u : 0u);
            const int from_lo = lo - t0 - 4 * h2, from_hi = hi - t0 - 4 * h2;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int x = 8 * (i >> 2) + (i & 3);
                sc[i] = x >= from_lo && x < from_hi && ((there >> (i >> 3)) & 1u) ? sc[i] : neg_inf();
                if ((i & 3) == 3)
                    __builtin_amdgcn_sched_barrier(0);  // few registers at a time
            }
            const float top = halves_max(max16(sc) * f);
            const bool raise = top > m;
            const float down = raise ? __builtin_amdgcn_exp2f(m - top) : 1.0f;
            m = raise ? top : m;
            ready = !__any(m == neg_inf());
            l *= down;
#pragma unroll
            for (int x = 0; x < D / 32; ++x)
                o[x] *= down;
            const float from = kBias - (m == neg_inf() ? 0.0f : m);
            total = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float w = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i], f, from));
                w = sc[i] == neg_inf() ? 0.0f : w;
                total += w;
                p[i >> 3][i & 7] = (_Float16)w;
                if ((i & 3) == 3)
                    __builtin_amdgcn_sched_barrier(0);
            }
        }
        l += total;
    };
    // Keys of stage n + 2 or values of stage n + 1 into the buffer that both
    // belong in (their own), and what comes after them from memory.
    const auto ahead = [&](int n, int slot1, int slot2) {
        const int d = n + (has_keys ? 2 : 1);
        if (decodes && d < stages) {
            decode(d, has_keys ? slot2 : slot1);
            if (d + 1 < stages)
                fetch(d + 1);
        }
    };
    if (!active) {
        // A wave without rows only decodes. (It passes as many barriers as the
        // others, in a loop of its own: the steps' registers are not carried
        // around them here.)
        int now = 0, next = 1, last = 2;
        for (int n = 0; n < stages; ++n) {
            ahead(n, next, last);
            __syncthreads();
            const int x = now;
            now = next, next = last, last = x;
        }
    } else {
        floatx16 sa, sb;
        f16x8 pa[2], pb[2];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            sa[i] = 0.0f;
            pb[i >> 3][i & 7] = (_Float16)0.0f;
        }
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
            sa = __builtin_amdgcn_mfma_f32_32x32x16_f16(key_frag(0, 0, k), qf[k], sa, 0, 0, 0);
        int now = 0, next = 1, last = 2;  // buffers of stages n, n + 1, n + 2 (which is n - 1's)
        int t0 = base;
        // The last step's values once no scores are left to be formed.
        const auto finish = [&](int slot, f16x8 (&pp)[2]) {
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int x = 0; x < D / 32; ++x)
                    o[x] = __builtin_amdgcn_mfma_f32_32x32x16_f16(value_frag(slot, H - 1, y, x), pp[y], o[x], 0, 0, 0);
        };
        if constexpr (H == 2) {
#pragma unroll
            for (int k = 0; k < kEarly; ++k)
                read(k, now, 1, now, 1, k);
            for (int n = 0; n < stages; ++n, t0 += kTokens) {
                if (has_keys)
                    ahead(n, next, last);
                step(t0, n, now, now, 1, n == 0 ? now : last, 1, next, 0, now, 0, sa, sb, pb, pa);
                if (!has_keys)
                    ahead(n, next, last);
                step(t0 + 32, n, now, next, 0, now, 0, next, 1, now, 1, sb, sa, pa, pb);
                __syncthreads();
                const int x = now;
                now = next, next = last, last = x;
            }
            finish(last, pb);
        } else {
            int n = 0;
            for (; n + 1 < stages; n += 2, t0 += 2 * kTokens) {
                ahead(n, next, last);
                step(t0, n, now, next, 0, n == 0 ? now : last, 0, last, 0, now, 0, sa, sb, pb, pa);
                __syncthreads();
                ahead(n + 1, last, now);
                step(t0 + kTokens, n + 1, next, last, 0, now, 0, now, 0, next, 0, sb, sa, pa, pb);
                __syncthreads();
                const int x = now;
                now = last, last = next, next = x;
            }
            if (n < stages) {
                step(t0, n, now, next, 0, n == 0 ? now : last, 0, last, 0, now, 0, sa, sb, pb, pa);
                __syncthreads();
                finish(now, pa);
            } else {
                finish(last, pb);
            }
        }
    }

    // An opaque zero keeps what follows from being formed ahead of the loop.
    uint32_t zero = 0u;
    asm volatile("" : "+v"(zero));
    const int local = 32 * wave + q + (int)zero;
    const int half = h2 + (int)zero;
    __syncthreads();
    if (lds.nans != 0u && active) {
        // NaN values that some row does not see were left out of the products:
        // 1 where an element of a token is one, times 1 where a row sees it,
        // says where they belong.
        for (int t = base; t < min(base + stages * kTokens, seen_hi); t += 16) {
            const int pg = page_at(t);
            if (pg < 0 || (t >= all_lo && t + 16 <= all_hi))
                continue;
            const int64_t rec = (((int64_t)pg * a.c.kv_heads + kh) << (a.c.page_shift - 4)) + ((t >> 4) & tile_mask);
            const uint8_t* vs = a.data + rec * Record<D>::kBytes + Record<D>::kValueScales;
            f16x8 sees;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int u = t + 8 * (i >> 2) + 4 * half + (i & 3);
                sees[i] = u >= lo && u < hi ? (_Float16)1.0f : (_Float16)0.0f;
            }
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
                const int slot = 32 * x + q;
                const int blk = ((slot & 15) * (D / 16) + (slot >> 4)) >> 4;
                f16x8 which;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t byte = vs[blk * 16 + 8 * (i >> 2) + 4 * half + (i & 3)];
                    which[i] = (byte & 0x7Fu) == 0x7Fu ? (_Float16)1.0f : (_Float16)0.0f;
                }
                floatx16 hit;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    hit[i] = 0.0f;
                hit = __builtin_amdgcn_mfma_f32_32x32x16_f16(which, sees, hit, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    o[x][i] = hit[i] > 0.0f ? __uint_as_float(0x7FC00000u) : o[x][i];
            }
        }
    }

    // Register i of o[x] is slot 32 x + 8 (i / 4) + 4 h2 + i % 4, so registers
    // with the same i % 8 (over x and i / 8) are D / 16 consecutive elements.
    l = halves_sum(l);
    const float vg = global_scale_from_amax(*a.c.v_amax);
    if (parts > 1) {
        float* const slot = slot_of<D, W>(a, blockIdx.x, parts_most, part);
        float* const to = slot + (wave * (D / 8) * 64 + lane + (int)zero) * 4;
        if (active) {
#pragma unroll
            for (int x = 0; x < D / 32; ++x)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    *reinterpret_cast<floatx4*>(to + (x * 4 + k) * 256) =
                        floatx4{o[x][4 * k], o[x][4 * k + 1], o[x][4 * k + 2], o[x][4 * k + 3]};
            if (half == 0)
                *reinterpret_cast<float2*>(slot + St::kRows * D + 2 * local) = make_float2(m, l);
        }
        return;
    }
    if (r0 + local < rows) {
        const int tok = (r0 + local) / G;
        const int64_t out_row = (s.q0 + tok) * a.heads + kh * G + (r0 + local - tok * G);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = 8 * (i >> 2) + 4 * half + (i & 3);
            constexpr int N = D == 64 ? 4 : 8;
#pragma unroll
            for (int e = 0; e < D / 16; e += N) {
                float v[N];
#pragma unroll
                for (int j = 0; j < N; ++j)
                    v[j] = o[(e + j) >> 1][i + 8 * (j & 1)];
                write_row<T, D>(a, out_row, c * (D / 16) + e, m, l, v, vg);
            }
        }
    }
}

// Joins the parts: a workgroup for a half (registers 4 j .. and 8 + 4 j .. of
// every o[x]) or, of 256-element heads, a quarter of a wave's rows' elements;
// its four waves take every fourth part, in their order, and are joined in LDS.
// In a launch of its own: joined by the workgroup that finishes last, 64
// queries over 1710 tokens took 61 us (with this 19), 256 over 9251 128 us (49).
constexpr int kJoinWaves = 4;

template <class T, int D, int W>
__global__ __launch_bounds__(64 * kJoinWaves) void kv_join_kernel(KvAttentionArgs a, int row_tiles, int parts_most)
{
    typedef Stages<D, W> St;
    constexpr int N = D == 64 ? 4 : 8;  // elements side by side in memory, of each of 4 registers
    __shared__ floatx4 lds_v[kJoinWaves - 1][N][64];
    __shared__ float2 lds_ml[kJoinWaves - 1][64];
    const Piece piece = piece_of<D, W>(a, blockIdx.x, row_tiles, parts_most);
    const int lane = threadIdx.x & 63, own = uniform((int)threadIdx.x >> 6), y = blockIdx.y;
    const int wave = y % W, j = y / W & 1, first = y / (2 * W) * N;
    const int local = 32 * wave + (lane & 31), half = lane >> 5;
    if (piece.parts == 1 || piece.r0 + 32 * wave >= piece.rows)
        return;
    const float vg = global_scale_from_amax(*a.c.v_amax);
    floatx4 v[N];
#pragma unroll
    for (int e = 0; e < N; ++e)
        v[e] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    float m = neg_inf(), l = 0.0f;
#pragma unroll 4
    for (int p = own; p < piece.parts; p += kJoinWaves) {
        const float* const slot = slot_of<D, W>(a, blockIdx.x, parts_most, p);
        const float* const from = slot + (wave * (D / 8) * 64 + lane) * 4;
        const float2 ml = *reinterpret_cast<const float2*>(slot + St::kRows * D + 2 * local);
        floatx4 x[N];
#pragma unroll
        for (int e = 0; e < N; ++e)
            x[e] = *reinterpret_cast<const floatx4*>(from + (((first + e) >> 1) * 4 + 2 * (e & 1) + j) * 256);
        const Factors f = join_of(m, l, ml.x, ml.y);
#pragma unroll
        for (int e = 0; e < N; ++e)
            v[e] = v[e] * f.mine + x[e] * f.other;
    }
    if (own > 0) {
#pragma unroll
        for (int e = 0; e < N; ++e)
            lds_v[own - 1][e][lane] = v[e];
        lds_ml[own - 1][lane] = make_float2(m, l);
    }
    __syncthreads();
    if (own > 0 || piece.r0 + local >= piece.rows)
        return;
#pragma unroll
    for (int k = 0; k < kJoinWaves - 1; ++k) {
        const float2 ml = lds_ml[k][lane];
        const Factors f = join_of(m, l, ml.x, ml.y);
#pragma unroll
        for (int e = 0; e < N; ++e)
            v[e] = v[e] * f.mine + lds_v[k][e][lane] * f.other;
    }
    const int G = a.heads / a.c.kv_heads;
    const int tok = (piece.r0 + local) / G;
    const int64_t out_row = (piece.s.q0 + tok) * a.heads + piece.kh * G + (piece.r0 + local - tok * G);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x[N];
#pragma unroll
        for (int k = 0; k < N; ++k)
            x[k] = v[k][i];
        write_row<T, D>(a, out_row, (8 * j + 4 * half + i) * (D / 16) + first, m, l, x, vg);
    }
}

int compute_units()
{
    static std::atomic<int> cache[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64)
        return 0;
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n > 0)
        return n;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
        return 0;
    cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

// How a launch is cut, and what it is taken to cost (tenths of a microsecond).
struct Plan {
    int64_t row_tiles, items, parts, cost;
};

template <int D, int W>
Plan plan(const KvAttentionArgs& a, int cus)
{
    typedef Stages<D, W> St;
    Plan w;
    w.row_tiles = (a.max_q * (a.heads / a.c.kv_heads) + St::kRows - 1) / St::kRows;
    w.items = w.row_tiles * a.c.batch * a.c.kv_heads;
    // The tokens may be split into parts, as far as a workgroup's rows can see
    // enough of them (the table's capacity, or the window behind the first
    // row's token up to the last one's): with fewer workgroups than compute
    // units, or where that fills the last round of them. What a choice costs,
    // in tenths of a microsecond: rounds of workgroups, each its stages and 5
    // (7 where partial results are written), and with parts the second launch
    // and the partial results' way to memory and back. (17 x 8 pieces over up
    // to 4096 tokens: 99 us whole, 85 in three parts and two rounds; 80 pieces
    // of 227 tokens 22 us in three parts, 19.5 whole; 12 x 8 over 4096 64 us in
    // two parts, 67 in five.)
    constexpr int64_t kSlots = (int64_t)((kWorkspaceBytes - kCounterBytes) / (St::kSlotFloats * 4));
    const int64_t capacity = a.c.table_stride << a.c.page_shift;
    const int64_t behind = a.window + St::kRows / (a.heads / a.c.kv_heads) + 1;
    const int64_t seen = a.causal && a.window > 0 && behind < capacity ? behind : capacity;
    const int64_t stages = (seen + 15 + St::kTokens - 1) / St::kTokens;
    constexpr int64_t kStage = D == 64 ? (W == 8 ? 12 : 16) : D == 128 ? 20 : 13;
    int64_t most = kSlots / w.items < stages / kMinStages ? kSlots / w.items : stages / kMinStages;
    most = most < 2 * cus / w.items ? most : 2 * cus / w.items;
    const auto rounds = [&](int64_t n) { return (n + cus - 1) / cus; };
    w.parts = 1;
    w.cost = rounds(w.items) * (stages * kStage + 50);
    for (int64_t p = 2; p <= most; ++p) {
        const int64_t cost = rounds(w.items * p) * (stages * kStage / p + 70) + 60 +
                             w.items * p * (int64_t)St::kSlotFloats / 62500;  // 2 x 4 bytes at 5 TB/s
        if (cost < w.cost)
            w.cost = cost, w.parts = p;
    }
    return w;
}

template <class T, int D, int W>
hipError_t go(const KvAttentionArgs& a, const Plan& w, hipStream_t stream)
{
    hipLaunchKernelGGL((kv_prompt_kernel<T, D, W>), dim3((unsigned)w.items, (unsigned)w.parts), dim3(64 * W), 0, stream, a,
                       (int)w.row_tiles, (int)w.parts);
    if (w.parts > 1) {
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        hipLaunchKernelGGL((kv_join_kernel<T, D, W>), dim3((unsigned)w.items, (D == 256 ? 4 : 2) * W),
                           dim3(64 * kJoinWaves), 0, stream,
                           a, (int)w.row_tiles, (int)w.parts);
    }
    return hipGetLastError();
}

// Heads of 64 elements leave registers for three waves of a SIMD: 12 waves, of
// which 8 decode, where that does not cost a round of workgroups (8192 tokens
// 334 us, 8 waves 356; 5 x 117 queries over 24,341 tokens 277 and 307; 4096
// tokens 104 and 94).
template <class T>
hipError_t by_dim(const KvAttentionArgs& a, hipStream_t stream)
{
    const int cus = compute_units();
    if (cus <= 0)
        return hipErrorInvalidDevice;
    switch (a.c.head_dim) {
    case 64: {
        const Plan w8 = plan<64, 8>(a, cus), w12 = plan<64, 12>(a, cus);
        return w8.cost <= w12.cost ? go<T, 64, 8>(a, w8, stream) : go<T, 64, 12>(a, w12, stream);
    }
    case 128:
        return go<T, 128, 8>(a, plan<128, 8>(a, cus), stream);
    default:
        return go<T, 256, 4>(a, plan<256, 4>(a, cus), stream);
    }
}

}  // namespace

hipError_t launch_kv_prompt(const KvAttentionArgs& a, hipStream_t stream)
{
    return a.dtype == kBf16 ? by_dim<Bf16>(a, stream) : by_dim<F16>(a, stream);
}

}  // namespace nvfp4
