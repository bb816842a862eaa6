// Attention over the NVFP4 key/value cache: few query rows per sequence (the
// streaming kernel). See include/nvfp4_kv.h for the contract, kv_stream.h for
// a wave's inner loop.
#include <atomic>

#include "kv_parts.h"

namespace nvfp4 {

namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kBlock = 32 * kWaves;  // tokens that a workgroup takes at a time

// Blocks that a part has at least. (1: 777 tokens in 10.0 us where 2 take 10.3,
// but 200 in 9.6 where 2 take 7.9; 4: 777 in 11.5, 3000 in 12.0 and 11.2.)
constexpr int kMinChunk = 2;

// Blocks of kBlock tokens that the queries of a sequence see between them
// (one at least where there are queries: somebody has to write their zeros).
__device__ __forceinline__ int blocks_of(const KvAttentionArgs& a, const Seq& s)
{
    if (s.nq <= 0)
        return 0;
    const int lo = first_seen(a, s, 0) & ~31, hi = end_seen(a, s, s.nq - 1);
    return max(1, (hi - lo + kBlock - 1) / kBlock);
}

// Partial results that a thread joins on its own, at most. (4 to 16 measure
// alike; without a limit the join of 124 parts took half of 94 us.)
constexpr int kAlone = 16;

// Where an element of a row lies in LDS and in a partial result.
template <int D, int NT>
struct Joint {
    static constexpr int kRows = 16 * NT;
    static constexpr int kPitch = D + 4;
    static constexpr size_t kSlotFloats = kRows * (D + 2);
    float o[kWaves][kRows][kPitch];
    float m[kWaves][kRows], l[kWaves][kRows];
    uint32_t last;
};

__device__ __forceinline__ int ceil_div(int a, int b) { return (int)(((unsigned)a + (unsigned)b - 1u) / (unsigned)b); }

// Inclusive sums over the wave's lanes: within rows of 16, then across them
// (lane shifts and row broadcasts of the vector unit, no LDS).
__device__ __forceinline__ int wave_scan(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);   // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);   // row_shr:2
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);   // row_shr:4
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);   // row_shr:8
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15 to rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31 to rows 2 and 3
    return v;
}

// A workgroup's share of a launch of the streaming kernel.
struct Share {
    Seq s;
    int b, kh;        // sequence (-1: no share), kv head (times tiles: a tile of its rows)
    int part, parts;  // part of how many of the (sequence, head)
    int slot0;        // slot of the first of them, where there are several
};

// Every (sequence, kv head, tile of its rows) is cut into equal parts of at
// most `chunk` blocks, a workgroup each; chunk is found from lens, the same by every workgroup, so
// that there are about `target` parts in all (0: nothing is cut), or fewer
// where parts of 4 blocks are, down to `few` (one for a compute unit): what
// is left to stream is then less than starting and joining parts takes (16
// sequences of 9 blocks: 17.3 us in 192 parts, 21.6 in 320). Parts are whole
// numbers: where they come out as more than target (more than the device
// holds at once), a larger chunk keeps them from taking a second round (32
// sequences of 16 to 64 blocks, 8 heads: 62 us without). 32-bit sums: the
// launch has seen to it.
__device__ __forceinline__ Share share_of(const KvAttentionArgs& a, int tiles, int target, int few, int lane)
{
    const int H = a.c.kv_heads * tiles, B = a.c.batch;
    // What is known of the first 64 sequences stays in the lanes.
    Seq mine{0, 0, 0, 0, 0};
    int blocks0 = 0;
    if (lane < B) {
        mine = seq_of(a, lane);
        blocks0 = blocks_of(a, mine);
    }
    const auto blocks_at = [&](int b0) {
        return b0 == 0 ? blocks0 : b0 + lane < B ? blocks_of(a, seq_of(a, b0 + lane)) : 0;
    };
    int chunk = 0x7FFFFFFF;
    if (target > 0) {
        int sum = 0;
        for (int b0 = 0; b0 < B; b0 += 64)
            sum += blocks_at(b0);
        const int total = __builtin_amdgcn_readlane(wave_scan(sum), 63) * H;
        target = min(target, max(few, total >> 2));
        chunk = max(kMinChunk, ceil_div(total, target));
        if (B * H < target)
            for (int again = 0; again < 4; ++again) {
                int n = 0;
                for (int b0 = 0; b0 < B; b0 += 64)
                    n += ceil_div(blocks_at(b0), chunk);
                const int count = __builtin_amdgcn_readlane(wave_scan(n), 63) * H;
                if (count <= target)
                    break;
                chunk = max(chunk + 1, (int)((float)chunk * (float)count / (float)target));
            }
    }
    Share w{Seq{0, 0, 0, 0, 0}, -1, 0, 0, 1, 0};
    int id = blockIdx.x;
    for (int b0 = 0; b0 < B; b0 += 64) {
        const int parts = ceil_div(blocks_at(b0), chunk);
        const int cut = parts > 1 ? parts : 0;
        const int upto = wave_scan(parts), upto_cut = wave_scan(cut);
        const uint64_t past = __ballot(id < upto * H);
        if (past != 0) {
            const int at = __ffsll((unsigned long long)past) - 1;
            w.b = b0 + at;
            w.parts = __builtin_amdgcn_readlane(parts, at);
            id -= (__builtin_amdgcn_readlane(upto, at) - w.parts) * H;
            w.slot0 += (__builtin_amdgcn_readlane(upto_cut, at) - (w.parts > 1 ? w.parts : 0)) * H;
            w.kh = id / w.parts;
            w.part = id - w.kh * w.parts;
            w.slot0 += w.kh * w.parts;
            if (b0 == 0) {
                w.s.q0 = __builtin_amdgcn_readlane((int)mine.q0, at);  // below total_q, 31 bits
                w.s.nq = __builtin_amdgcn_readlane(mine.nq, at);
                w.s.past = __builtin_amdgcn_readlane(mine.past, at);
                w.s.len = __builtin_amdgcn_readlane(mine.len, at);
                w.s.pos0 = __builtin_amdgcn_readlane(mine.pos0, at);
            } else {
                w.s = seq_of(a, w.b);
            }
            break;
        }
        id -= __builtin_amdgcn_readlane(upto, 63) * H;
        w.slot0 += __builtin_amdgcn_readlane(upto_cut, 63) * H;
    }
    return w;
}

// Waves of a SIMD that the kernel is compiled for: as many as its registers
// allow without going through memory. (Left to itself the compiler aims at
// one, and keeps the output in accumulation registers that every step copies
// from and to.)
template <int D, int NT>
constexpr int kWavesPerSimd = D == 64 ? (NT == 1 ? 4 : 3) : D == 128 ? (NT == 1 ? 3 : 2) : (NT == 1 ? 2 : 1);

// The streaming kernel: one part of a (sequence, kv head, 16 NT of its rows)
// per workgroup, the waves 32 tokens each of every 128. One that is not cut is written at once.
// The parts of others go to the workspace, and the workgroup that finishes
// last joins them, in their order, so that results do not depend on who that
// is.
//
// Reading the cache bounds it: 18 D bytes for 16 tokens of a head, each once
// for all rows of the head; two register sets per wave, and two to three
// workgroups on a compute unit, keep the loads in flight. Two sequences of
// 131,072 tokens, 8 heads of 128: 302 MB in 67.7 us (4.5 TB/s); 32 sequences
// of 2048 to 8192: 189 MB in 47 us (4.0 TB/s; 34.5 us of it the loop, the rest
// finding the parts, rows, and joining); one sequence of 777 tokens 10.2 us,
// of which 2.5 are an empty launch, 3 find and start the parts, 1.8 stream,
// 2.9 join: a chain of dependent loads, each about 0.8 us.
template <class T, int D, int NT>
__global__ __launch_bounds__(kThreads, (kWavesPerSimd<D, NT>)) void kv_stream_kernel(KvAttentionArgs a, int tiles, int target, int few)
{
    __shared__ Joint<D, NT> lds;
    constexpr int kRows = 16 * NT;
    const int lane = threadIdx.x & 63;
    const int wave = uniform((int)threadIdx.x >> 6);
    const int c = lane & 15;
    const int G = a.heads / a.c.kv_heads;
    const Share share = share_of(a, tiles, target, few, lane);
    if (share.b < 0)
        return;
    const Seq s = share.s;
    const int part = share.part, parts = share.parts, slot0 = share.slot0;
    // Rows r0 .. of the kv head: `rows` of them.
    const int kh = share.kh / tiles, r0 = (share.kh - kh * tiles) * kRows;
    const int rows = min(s.nq * G - r0, kRows);
    if (rows <= 0 && r0 > 0)
        return;
    RawRows<D, NT> raw;
    load_rows<D, NT>(raw, a, s.q0, kh, r0, r0 + rows, G, lane);
    const int seen_lo = first_seen(a, s, 0), seen_hi = end_seen(a, s, s.nq - 1);
    const int all_lo = first_seen(a, s, (r0 + rows - 1) / G), all_hi = end_seen(a, s, r0 / G);
    const int32_t* pages = a.c.page_table + (int64_t)share.b * a.c.table_stride;
    // The item's blocks in `parts` stretches that differ by one at most.
    const int blocks = blocks_of(a, s), each = blocks / parts, more = blocks - each * parts;
    const int k0 = part * each + min(part, more), k1 = k0 + each + (part < more ? 1 : 0);
    const int base = seen_lo & ~31;
    const int end = min(seen_hi, base + k1 * kBlock);
    const int tile_mask = (1 << (a.c.page_shift - 4)) - 1;

    // Two sets of registers: the loads of the next 32 tokens are under way
    // while these are worked on, and the page numbers of those after them.
    const auto pages_at = [&](int t0, int (&page)[2]) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
            page[x] = t0 + 16 * x < end ? pages[(t0 + 16 * x) >> a.c.page_shift] : -1;
    };
    const auto load = [&](int t0, const int (&page)[2], Tile<D> (&tile)[2], bool (&there)[2]) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            there[x] = (uint32_t)page[x] < (uint32_t)a.c.num_pages;
            const int64_t rec = (((int64_t)(there[x] ? page[x] : 0) * a.c.kv_heads + kh) << (a.c.page_shift - 4)) +
                                (((t0 >> 4) + x) & tile_mask);
            tile[x] = load_tile<D>(a.data + rec * Record<D>::kBytes, lane);
        }
    };
    Rows<D, NT> w;
    Sight<NT> sight;
    const auto work = [&](int t0, const Tile<D> (&tile)[2], const bool (&there)[2]) {
        const bool masked = t0 < all_lo || t0 + 32 > all_hi || !there[0] || !there[1];
        attend<D, NT>(w, tile, t0, sight, seen_lo, seen_hi, there, masked, lane);
    };
    int t0 = base + k0 * kBlock + 32 * wave;
    Tile<D> ta[2], tb[2];
    bool ha[2], hb[2];
    int page[2];
    if (t0 < end) {
        pages_at(t0, page);
        load(t0, page, ta, ha);
        pages_at(t0 + kBlock, page);
    }
    start_rows<T, D, NT>(w, raw, a);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int i = (r0 + min(16 * n + c, rows - 1)) / G;
        sight.lo[n] = first_seen(a, s, i);
        sight.hi[n] = end_seen(a, s, i);
    }
    if (t0 < end) {
        for (;;) {
            const int t1 = t0 + kBlock;
            if (t1 < end)
                load(t1, page, tb, hb);
            pages_at(t1 + kBlock, page);
            __builtin_amdgcn_sched_barrier(0);
            work(t0, ta, ha);
            if (t1 >= end)
                break;
            t0 = t1 + kBlock;
            if (t0 < end)
                load(t0, page, ta, ha);
            pages_at(t0 + kBlock, page);
            __builtin_amdgcn_sched_barrier(0);
            work(t1, tb, hb);
            if (t0 >= end)
                break;
        }
    }

    // The waves' results side by side in LDS. An opaque zero keeps the
    // addresses of what follows from being formed ahead of the loop above
    // (they would stay in registers throughout it).
    uint32_t zero = 0u;
    asm volatile("" : "+v"(zero));
    const int tid = threadIdx.x + (int)zero;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = 16 * n + (tid & 15);
        const float l = across16_sum(w.l[n]);
        if ((tid & 63) < 16) {
            lds.m[wave][r] = w.m[n];
            lds.l[wave][r] = l;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int x = 0; x < D / 16; ++x)
                lds.o[wave][r][((tid & 63) >> 4) * (D / 4) + i * (D / 16) + x] = w.o[n][x][i];
    }
    // (Behind the loop: a store ahead of it keeps its uniform loads out of the
    // scalar cache, 32 sequences of 2048 to 8192 tokens 51 us for 46.5.)
    if (s.past > 0 && part == 0 && r0 == 0)
        write_past<T, D>(a, s, kh, G, kThreads);
    __syncthreads();
    const float vg = global_scale_from_amax(*a.c.v_amax);
    float* const slots = reinterpret_cast<float*>(reinterpret_cast<char*>(a.workspace) + kCounterBytes);
    float* const slot = slots + (int64_t)(slot0 + part) * Joint<D, NT>::kSlotFloats;
    // A partial result: maxima and sums, then the rows.
    const auto put_unit = [&](float* to, int r, int d, float m, float l, const float (&v)[8]) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            put2(to + 2 * kRows + r * D + d + 2 * j, v[2 * j], v[2 * j + 1]);
        if (d == 0)
            put2(to + 2 * r, m, l);
    };
    for (int i = tid; i < rows * (D / 8); i += kThreads) {
        const int r = i / (D / 8), d = i % (D / 8) * 8;
        float m = lds.m[0][r], l = lds.l[0][r], v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = lds.o[0][r][d + j];
#pragma unroll
        for (int k = 1; k < kWaves; ++k) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = lds.o[k][r][d + j];
            merge(m, l, v, lds.m[k][r], lds.l[k][r], x);
        }
        if (parts == 1) {
            const int tok = (r0 + r) / G;
            write_row<T, D>(a, (s.q0 + tok) * a.heads + kh * G + (r0 + r - tok * G), d, m, l, v, vg);
        } else {
            put_unit(slot, r, d, m, l, v);
        }
    }
    if (parts == 1)
        return;

    // Groups of threads take every `way`th partial result; then they are joined
    // in LDS.
    const int units = rows * (D / 8);
    const int way = max(1, kThreads / units);  // 1 where the rows fill the workgroup
    float* const mine = slots + (int64_t)slot0 * Joint<D, NT>::kSlotFloats;
    // Joins n results, `step` slots apart from the item's slot `at` on; what
    // comes out is the output, or (last false) replaces the first of them.
    const auto join = [&](int at, int step, int n, bool last) {
        for (int i0 = 0; i0 < units; i0 += kThreads) {
            const int i = way > 1 ? tid % units : i0 + tid;
            const int grp = way > 1 ? tid / units : 0;
            const bool on = i < units && grp < way;
            const int r = i / (D / 8), d = i % (D / 8) * 8;
            float m = neg_inf(), l = 0.0f, v[8] = {};
            if (on) {
#pragma unroll 4
                for (int p = grp; p < n; p += way) {
                    const float* from = mine + (int64_t)(at + p * step) * Joint<D, NT>::kSlotFloats;
                    const float2 ml = get2(from + 2 * r);
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 y = get2(from + 2 * kRows + r * D + d + 2 * j);
                        x[2 * j] = y.x, x[2 * j + 1] = y.y;
                    }
                    merge(m, l, v, ml.x, ml.y, x);
                }
            }
            __syncthreads();  // the rows' maxima and sums are read by other threads than write them
            if (way > 1) {
                // kThreads times 8 elements, a maximum and a sum fit where the
                // waves' results were.
                float* const flat = &lds.o[0][0][0];
                static_assert(sizeof(lds.o) >= kThreads * 10 * sizeof(float), "LDS");
                if (on) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        flat[tid * 8 + j] = v[j];
                    flat[kThreads * 8 + 2 * tid] = m;
                    flat[kThreads * 8 + 2 * tid + 1] = l;
                }
                __syncthreads();
                if (on && grp == 0) {
                    for (int k = 1; k < way; ++k) {
                        const int o = k * units + i;
                        float x[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            x[j] = flat[o * 8 + j];
                        merge(m, l, v, flat[kThreads * 8 + 2 * o], flat[kThreads * 8 + 2 * o + 1], x);
                    }
                }
                __syncthreads();  // a second join writes there again
            }
            if (on && grp == 0) {
                if (last) {
                    const int tok = (r0 + r) / G;
                    write_row<T, D>(a, (s.q0 + tok) * a.heads + kh * G + (r0 + r - tok * G), d, m, l, v, vg);
                } else {
                    put_unit(mine + (int64_t)at * Joint<D, NT>::kSlotFloats, r, d, m, l, v);
                }
            }
        }
    };
    // Whether this workgroup is the last of n that are counted at an item's
    // slot's number (and the count is 0 again).
    const auto last_of = [&](int at, int n) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's stores have arrived
        __syncthreads();
        if (tid == 0) {
            uint32_t* const counter = a.workspace + slot0 + at;
            const uint32_t done = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            lds.last = done + 1 == (uint32_t)n;
            if (lds.last)
                __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        return lds.last != 0u;
    };
    // Many parts are joined in two levels (a thread's loads of kAlone parts are
    // under way four at a time, each about 2 us): groups of about as many as
    // there are groups, counted at their second slot, then their results,
    // counted at the item's first.
    int group = 1;
    if (parts > kAlone * way) {
        group = max(2, (int)__builtin_sqrtf((float)parts));
        const int first = part / group * group, n = min(group, parts - first);
        if (n > 1) {
            if (!last_of(first + 1, n))
                return;
            join(first, 1, n, false);
        }
    }
    const int count = (parts + group - 1) / group;
    if (last_of(0, count))
        join(0, group, count, true);
}

// Workgroups of the kernel that the device holds at once, and its compute
// units (looked up on first use per device).
template <class T, int D, int NT>
int stream_capacity(int& cus)
{
    static std::atomic<int> cache[64], units[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64)
        return 0;
    int n = cache[dev].load(std::memory_order_acquire);
    cus = units[dev].load(std::memory_order_relaxed);
    if (n > 0)
        return n;
    int per_cu = 0;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(
            &per_cu, reinterpret_cast<const void*>(kv_stream_kernel<T, D, NT>), kThreads, 0) != hipSuccess ||
        hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
        return 0;
    n = (per_cu > 0 ? per_cu : 1) * cus;
    if (n > 0) {
        units[dev].store(cus, std::memory_order_relaxed);
        cache[dev].store(n, std::memory_order_release);
    }
    return n;
}

template <class T, int D, int NT>
hipError_t stream(const KvAttentionArgs& a, int tiles, hipStream_t stream)
{
    int cus = 0;
    const int n = stream_capacity<T, D, NT>(cus);
    if (n <= 0)
        return hipErrorInvalidDevice;
    // A cut item has at least 2 parts of more than half a chunk, so cut items
    // have at most 2 target parts, each with a slot (and a counter).
    constexpr int kSlots = (int)((kWorkspaceBytes - kCounterBytes) / (Joint<D, NT>::kSlotFloats * 4));
    // Two workgroups for a compute unit stream as fast as three; where an item
    // has only a few parts, three even out that they are whole numbers (two
    // sequences of 131,072 tokens, 8 heads: 67.7 and 74 us; 32 sequences of
    // 2048 to 8192: 48.7 and 46.4 us).
    const int64_t items = (int64_t)a.c.batch * a.c.kv_heads * tiles;
    int target = 6 * items <= 2 * cus && 2 * cus < n ? 2 * cus : n;
    target = target < kSlots / 2 ? target : kSlots / 2;
    target = target < kMaxSlots / 2 ? target : kMaxSlots / 2;
    // Workgroups: a part for each item, and target more at most; nor more
    // than there are chunks in the pages that the table has room for.
    // (More blocks than 31 bits count: nothing is cut.)
    const int64_t blocks = ((a.c.table_stride << a.c.page_shift) + 31 + kBlock - 1) / kBlock;
    if (blocks > 0x7FFFFFFF / items)
        target = 0;
    const int64_t chunks = items * ((blocks + kMinChunk - 1) / kMinChunk);
    const int64_t grid = items + target < chunks ? items + target : chunks;
    hipLaunchKernelGGL((kv_stream_kernel<T, D, NT>), dim3((unsigned)grid), dim3(kThreads), 0, stream, a, tiles,
                       target, cus);
    return hipGetLastError();
}

template <class T, int D>
hipError_t go(const KvAttentionArgs& a, hipStream_t s)
{
    // Up to kMost rows of a kv head stream, each 32 of them the cache for
    // themselves; more are a prompt, whose workgroups decode it once for up to
    // 256 rows but come one to a compute unit, so that a sequence's parts are
    // not evened out. 32 sequences of 2048 to 8192 tokens, us here and there:
    // 36 rows of 64 elements 66 and 108, 128 rows 97 and 114; 64 rows of 128
    // elements 107 and 137, 128 rows 160 and 143; 36 rows of 256 elements 156
    // and 145. One sequence of 10^5 tokens, 64 rows of 128: 93 and 95.
    constexpr int kMost = D == 64 ? 128 : D == 128 ? 64 : 32;
    const int64_t rows = a.max_q * (a.heads / a.c.kv_heads);
    if (rows <= 16)
        return stream<T, D, 1>(a, 1, s);
    if (rows <= kMost)
        return stream<T, D, 2>(a, (int)((rows + 31) / 32), s);
    return launch_kv_prompt(a, s);
}

}  // namespace

hipError_t launch_kv_attention(const KvAttentionArgs& a, hipStream_t stream)
{
    const bool bf16 = a.dtype == kBf16;
    switch (a.c.head_dim) {
    case 64:
        return bf16 ? go<Bf16, 64>(a, stream) : go<F16, 64>(a, stream);
    case 128:
        return bf16 ? go<Bf16, 128>(a, stream) : go<F16, 128>(a, stream);
    default:
        return bf16 ? go<Bf16, 256>(a, stream) : go<F16, 256>(a, stream);
    }
}

}  // namespace nvfp4
