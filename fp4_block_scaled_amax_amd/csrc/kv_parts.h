// What the attention kernels share: a sequence's rows and visible tokens, the
// workspace, and how partial results are kept and joined.
#pragma once

#include "kv_stream.h"

namespace nvfp4 {

// Workspace: a counter for each slot, then the slots (partial results).
constexpr int kMaxSlots = 8192;
constexpr size_t kCounterBytes = kMaxSlots * 4;
constexpr size_t kWorkspaceBytes = 64u << 20;  // NVFP4_KV_WORKSPACE_BYTES

// Relaxed device-scope accesses: they go past the XCDs' own L2s, which are
// not coherent with each other, without flushing them.
__device__ __forceinline__ void put2(float* p, float a, float b)
{
    const uint64_t v = ((uint64_t)__float_as_uint(b) << 32) | __float_as_uint(a);
    __hip_atomic_store(reinterpret_cast<uint64_t*>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 get2(const float* p)
{
    const uint64_t v = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}

// Scalars of one sequence: its queries' rows in q (the nq that are computed,
// and `past` more than max_q allows), its visible tokens, and the position of
// its first query. (pos0 is no less than -2^30: queries are fewer than that, so
// one before the first token stays there, and no sum below passes 31 bits.)
struct Seq {
    int64_t q0;
    int nq, past, len, pos0;
};

__device__ __forceinline__ Seq seq_of(const KvAttentionArgs& a, int b)
{
    Seq s;
    int64_t n = a.max_q;
    if (a.cu_q != nullptr) {
        s.q0 = a.cu_q[b];
        const int64_t end = min((int64_t)a.cu_q[b + 1], a.total_q);
        n = s.q0 < 0 ? 0 : max((int64_t)0, end - s.q0);
    } else {
        s.q0 = b * a.max_q;
    }
    s.nq = (int)min(n, a.max_q);
    s.past = (int)(n - s.nq);
    s.len = (int)max((int64_t)0, min((int64_t)a.lens[b], a.c.table_stride << a.c.page_shift));
    s.pos0 = (int)max(s.len - n, -((int64_t)1 << 30));
    return s;
}

// Tokens [lo, hi) that query i of a sequence sees.
__device__ __forceinline__ int first_seen(const KvAttentionArgs& a, const Seq& s, int i)
{
    return a.window > 0 ? max(0, s.pos0 + i - a.window + 1) : 0;
}
__device__ __forceinline__ int end_seen(const KvAttentionArgs& a, const Seq& s, int i)
{
    return a.causal ? max(0, s.pos0 + i + 1) : s.len;
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Merges a running maximum and sum with another part's, and gives the factors
// of their elements. A part that saw nothing has m = -inf and l = 0; one whose
// scores were all NaN has m = -inf and l = NaN, which must stay.
struct Factors {
    float mine, other;
};
__device__ __forceinline__ Factors join_of(float& m, float& l, float pm, float pl)
{
    const float top = fmaxf(m, pm);
    const float fa = m == top ? 1.0f : m == neg_inf() ? 1.0f : __builtin_amdgcn_exp2f(m - top);
    const float fb = pm == top ? 1.0f : pm == neg_inf() ? 1.0f : __builtin_amdgcn_exp2f(pm - top);
    l = l * fa + pl * fb;
    m = top;
    return Factors{fa, fb};
}
__device__ __forceinline__ void merge(float& m, float& l, float (&v)[8], float pm, float pl, const float (&pv)[8])
{
    const Factors f = join_of(m, l, pm, pl);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = v[j] * f.mine + pv[j] * f.other;
}

// Elements d .. d + N - 1 (N 4 or 8) of a finished row, and its log-sum-exp.
// (One division for the row's elements: a sum of weights is between 2^-2 and
// 2^45 where there is one, so its inverse is a normal number.)
template <class T, int D, int N>
__device__ __forceinline__ void write_row(const KvAttentionArgs& a, int64_t row, int d, float m, float l, float (&v)[N],
                                          float vg)
{
    const float inverse = 1.0f / l;
#pragma unroll
    for (int j = 0; j < N; ++j)
        v[j] = l == 0.0f ? 0.0f : v[j] * inverse * vg;
    char* const to = static_cast<char*>(a.out) + (row * D + d) * 2;
    if constexpr (N == 8)
        store8<T>(to, v);
    else
        *reinterpret_cast<uint2*>(to) = make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
    if (a.lse != nullptr && d == 0)
        a.lse[row] = l == 0.0f ? neg_inf() : (m - kBias + __builtin_amdgcn_logf(l)) * kLn2;
}

// NaN for the queries of a sequence that max_q leaves out (only the device knows
// of them), by the workgroup that has the first rows of a kv head.
template <class T, int D>
__device__ __forceinline__ void write_past(const KvAttentionArgs& a, const Seq& s, int kv_head, int G, int threads)
{
    const float nan = __uint_as_float(0x7FC00000u);
    const float v[8] = {nan, nan, nan, nan, nan, nan, nan, nan};
    const int64_t units = (int64_t)s.past * G * (D / 8);
    for (int64_t i = threadIdx.x; i < units; i += threads) {
        const int64_t r = i / (D / 8), tok = r / G;
        const int64_t row = (s.q0 + s.nq + tok) * a.heads + kv_head * G + (r - tok * G);
        const int d = (int)(i % (D / 8)) * 8;
        store8<T>(static_cast<char*>(a.out) + (row * D + d) * 2, v);
        if (a.lse != nullptr && d == 0)
            a.lse[row] = nan;
    }
}

}  // namespace nvfp4
