// Rotary positions: the table of cosines and sines, and the rotation itself
// (forward and adjoint). See include/nvfp4_kv.h for the contract.
#include "heads.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;

// One thread per (position, pair). The angle p f_i is formed and reduced in
// 64 bits: at p = 10^6 a binary32 angle would be off by 0.03.
__global__ __launch_bounds__(kThreads) void rope_table_kernel(RopeTableArgs a)
{
    const int half = a.rot_dim >> 1;
    const int64_t n = a.max_pos * half;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        const int64_t p = i / half;
        const int k = (int)(i - p * half);
        double f = pow(a.base, -2.0 * k / a.rot_dim);
        if (a.linear)
            f /= a.factor;
        if (a.parts) {
            const double turns = a.original_len * f / 6.283185307179586476925;
            const double w = fmin(fmax((turns - a.low) / (a.high - a.low), 0.0), 1.0);
            f = f * (w + (1.0 - w) / a.factor);
        }
        double s, c;
        sincos((double)p * f, &s, &c);
        float* row = a.table + p * (2 * half) + k;
        row[0] = (float)(a.amplitude * c);
        row[half] = (float)(a.amplitude * s);
    }
}

// Each pair (a, b) becomes (a c - b s, b c + a s): a rotation by the angle of
// the token's position, whose transpose (the gradient) has -s. Three
// operations an element against 4 bytes moved (16-bit dtypes): memory bounds
// it, launches where there are few tokens.
//
// One thread per unit of 16 elements (8 pairs, or 16 elements that pass
// through): two 16-byte loads and stores per thread for 16-bit dtypes, all
// issued before the first is used. Neighbouring threads take neighbouring
// units of a head, so the halves of a head are read in spans of 8 threads x 16
// bytes; the table's row is read by all heads of a token and stays in the
// caches. The split into token, head and unit is one multiplication each (a
// division by a launch constant).
//
// Measured: 8192 tokens x 32 heads x 128, bf16 26.3 to 28 us a call, by card, with
// six inputs in turn, which then come from memory (4.8 to 5.1 TB/s; a large copy
// reaches 5.05), 22 to 24 with two, which the last-level cache holds in part; 4095 x 16 x 256 binary32, 64 elements rotated, 27.6 us (4.9 TB/s); 64
// tokens 3.0 us, an empty launch 2.3.
template <class T>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a, int64_t token0, uint32_t units, bool stream_y)
{
    const uint32_t id = blockIdx.x * kThreads + threadIdx.x;
    if (id >= units)
        return;
    const uint32_t th = a.by_units.div(id);  // token and head
    const int j = (int)(id - th * a.by_units.d);
    const uint32_t tl = a.by_heads.div(th);
    const int h = (int)(th - tl * a.by_heads.d);
    const int64_t t = token0 + tl;
    const Unit u = unit_of(j, a.rot_dim, a.interleaved);
    const char* x = static_cast<const char*>(a.x) + (t * a.x_ts + h * a.x_hs) * T::kBytes;
    char* y = static_cast<char*>(a.y) + (t * a.y_ts + h * a.y_hs) * T::kBytes;
    float lo[8], hi[8];
    load8<T>(x + u.lo * T::kBytes, lo);
    load8<T>(x + u.hi * T::kBytes, hi);
    if (u.pairs)
        turn_unit(lo, hi, load_turn(a.table, a.positions[t], a.max_pos, a.rot_dim >> 1, 8 * j, a.sign),
                  a.interleaved);
    if constexpr (T::kBytes == 2) {
        if (stream_y) {
            store16_stream(y + u.lo * T::kBytes, pack8<T>(lo));
            store16_stream(y + u.hi * T::kBytes, pack8<T>(hi));
            return;
        }
    }
    store8<T>(y + u.lo * T::kBytes, lo);
    store8<T>(y + u.hi * T::kBytes, hi);
}

}  // namespace

hipError_t launch_rope_table(const RopeTableArgs& a, hipStream_t stream)
{
    const int64_t n = a.max_pos * (a.rot_dim >> 1);
    const int64_t blocks = (n + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(rope_table_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(kThreads), 0,
                       stream, a);
    return hipGetLastError();
}

hipError_t launch_rope(const RopeArgs& a, hipStream_t stream)
{
    // Unit indexes are 31-bit: more tokens than that go in several launches.
    const int64_t per_token = (int64_t)a.by_heads.d * a.by_units.d;
    const int64_t most = ((int64_t)1 << 30) / per_token;
    // A result larger than the XCDs' L2s (8 x 4 MiB) is written past them: it
    // would only be pushed out, at the launch's end. Whole lines are, that is,
    // 16-bit heads of 128 and more, aligned. (From memory: 26.3 us where the caches take
    // 27.7, 27.4 and 28.3 with neighbouring pairs; heads of 64 elements alike;
    // binary32, whose threads write half lines, 70 and 27.)
    const int64_t head_dim = 16 * (int64_t)a.by_units.d;
    const bool stream_y = head_dim >= 128 && a.tokens * per_token * 32 > ((int64_t)32 << 20) &&
                          (a.y_ts | a.y_hs) % 64 == 0 && reinterpret_cast<uintptr_t>(a.y) % 128 == 0;
    for (int64_t t0 = 0; t0 < a.tokens; t0 += most) {
        const int64_t n = (a.tokens - t0 < most ? a.tokens - t0 : most) * per_token;
        const dim3 grid((unsigned)((n + kThreads - 1) / kThreads));
        if (a.dtype == kBf16)
            hipLaunchKernelGGL(rope_kernel<Bf16>, grid, dim3(kThreads), 0, stream, a, t0, (uint32_t)n,
                               stream_y);
        else if (a.dtype == kF16)
            hipLaunchKernelGGL(rope_kernel<F16>, grid, dim3(kThreads), 0, stream, a, t0, (uint32_t)n,
                               stream_y);
        else
            hipLaunchKernelGGL(rope_kernel<F32>, grid, dim3(kThreads), 0, stream, a, t0, (uint32_t)n,
                               stream_y);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

}  // namespace nvfp4
