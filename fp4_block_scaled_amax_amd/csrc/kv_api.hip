// C ABI entry points of the key/value cache: argument validation (before any
// HIP call), then the launch. See include/nvfp4_kv.h for the contract of
// each call.
#include "../../include/nvfp4_kv.h"

#include <math.h>

#include "kernels.h"

namespace {

constexpr int64_t kMaxElements = (int64_t)1 << 46;
constexpr int64_t kMaxInt = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxLen = (int64_t)1 << 30;  // tokens of a sequence, rows of a kv head
// A grid has fewer than 2^32 threads along x and at most 65535 workgroups
// along y; append and read put 16 tokens on a workgroup of x, and 16 blocks of
// 16 elements on one of y.
constexpr int64_t kMaxTokens = ((int64_t)1 << 28) - 16;
constexpr int64_t kMaxUnits = 65535 * 16;
constexpr int64_t kMaxItems = (int64_t)1 << 21;  // pieces of 128 rows: at most 4 workgroups of 256 threads

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int status_of(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP; }

bool dtype_ok(int dtype) { return dtype == NVFP4_F32 || dtype == NVFP4_BF16 || dtype == NVFP4_F16; }

// Strides of a [tokens][heads][head_dim] tensor: whole 16-byte vectors, not
// negative, and the last element inside the index range.
int strides_status(int dtype, int64_t tokens, int64_t heads, int64_t head_dim, int64_t ts, int64_t hs)
{
    const int64_t granule = dtype == NVFP4_F32 ? 4 : 8;
    if (ts < 0 || hs < 0)
        return NVFP4_ERR_SHAPE;
    if (ts % granule != 0 || hs % granule != 0)
        return NVFP4_ERR_ALIGN;
    if (ts > kMaxElements || hs > kMaxElements || (tokens > 0 && ts > kMaxElements / tokens) ||
        hs > kMaxElements / heads || head_dim > kMaxElements)
        return NVFP4_ERR_SIZE;
    return NVFP4_OK;
}

// Whether two heads of a tensor that is written share elements: some token's
// head begins less than head_dim from another's. Where the larger stride is past
// all that the smaller one spans none does; otherwise its multiples are looked
// at, each beside the nearest of the smaller's.
bool overlaps(int64_t tokens, int64_t heads, int64_t head_dim, int64_t ts, int64_t hs)
{
    if (tokens <= 1 || heads <= 1)
        return (tokens > 1 && ts < head_dim) || (heads > 1 && hs < head_dim);
    const int64_t few = ts < hs ? ts : hs, n_few = ts < hs ? tokens : heads;
    const int64_t far = ts < hs ? hs : ts, n_far = ts < hs ? heads : tokens;
    if (few < head_dim)
        return true;
    if (far >= (n_few - 1) * few + head_dim)
        return false;
    for (int64_t k = 1; k < n_far && k * far / few < n_few; ++k) {
        const int64_t past = k * far % few;
        if (past < head_dim || (few - past < head_dim && k * far / few + 1 < n_few))
            return true;
    }
    return false;
}

// The rotation's table: rot_dim elements of a head, rows below max_pos.
int rope_status(int64_t head_dim, int64_t max_pos, int64_t rot_dim, uint32_t flags, uint32_t known)
{
    if ((flags & ~known) != 0)
        return NVFP4_ERR_FLAGS;
    if (rot_dim <= 0 || rot_dim % 16 != 0 || rot_dim > head_dim || max_pos <= 0)
        return NVFP4_ERR_SHAPE;
    if (max_pos > kMaxInt)
        return NVFP4_ERR_SIZE;
    return NVFP4_OK;
}

// The cache and the page table; c receives them.
int cache_status(const uint8_t* data, int64_t num_pages, int64_t kv_heads, int64_t page_size, int64_t head_dim,
                 const float* k_amax, const float* v_amax, const int32_t* page_table, int64_t batch,
                 int64_t table_stride, nvfp4::KvCacheArgs& c)
{
    if (data == nullptr || k_amax == nullptr || v_amax == nullptr || page_table == nullptr)
        return NVFP4_ERR_NULL;
    if (num_pages <= 0 || kv_heads <= 0 || batch <= 0 || table_stride <= 0 || page_size < 16 || page_size > 32768 ||
        (page_size & (page_size - 1)) != 0 || (head_dim != 64 && head_dim != 128 && head_dim != 256))
        return NVFP4_ERR_SHAPE;
    if (num_pages > kMaxInt || kv_heads > 65535 || batch > kMaxInt || table_stride > kMaxLen / page_size)
        return NVFP4_ERR_SIZE;
    if (!aligned16(data) || !aligned4(k_amax) || !aligned4(v_amax) || !aligned4(page_table))
        return NVFP4_ERR_ALIGN;
    c = nvfp4::KvCacheArgs{};
    c.num_pages = num_pages;
    c.kv_heads = (int)kv_heads;
    while (((int64_t)1 << c.page_shift) < page_size)
        ++c.page_shift;
    c.head_dim = (int)head_dim;
    c.k_amax = k_amax;
    c.v_amax = v_amax;
    c.page_table = page_table;
    c.batch = (int)batch;
    c.table_stride = table_stride;
    return NVFP4_OK;
}

}  // namespace

extern "C" {

int nvfp4_rope_table(int64_t max_pos, int64_t rot_dim, double base, int scaling, double factor,
                     double original_len, double low, double high, double amplitude, float* table,
                     hipStream_t stream)
{
    if (table == nullptr)
        return NVFP4_ERR_NULL;
    if (scaling < NVFP4_ROPE_PLAIN || scaling > NVFP4_ROPE_PARTS || !(base > 1.0) || !isfinite(base) ||
        !isfinite(amplitude) || !(factor >= 1.0) || !isfinite(factor))
        return NVFP4_ERR_FLAGS;
    if (scaling == NVFP4_ROPE_PARTS &&
        (!(original_len > 0.0) || !isfinite(original_len) || !(low < high) || !isfinite(low) || !isfinite(high)))
        return NVFP4_ERR_FLAGS;
    if (max_pos <= 0 || rot_dim <= 0 || rot_dim % 16 != 0)
        return NVFP4_ERR_SHAPE;
    if (max_pos > kMaxInt || rot_dim > (1 << 20))
        return NVFP4_ERR_SIZE;
    if (!aligned16(table))
        return NVFP4_ERR_ALIGN;
    nvfp4::RopeTableArgs a{};
    a.max_pos = max_pos;
    a.rot_dim = (int)rot_dim;
    a.base = scaling == NVFP4_ROPE_BASE ? base * pow(factor, (double)rot_dim / (double)(rot_dim - 2)) : base;
    a.factor = factor;
    a.original_len = original_len;
    a.low = low;
    a.high = high;
    a.amplitude = amplitude;
    a.linear = scaling == NVFP4_ROPE_LINEAR;
    a.parts = scaling == NVFP4_ROPE_PARTS;
    a.table = table;
    return status_of(nvfp4::launch_rope_table(a, stream));
}

int nvfp4_rope(const void* x, int dtype, int64_t tokens, int64_t heads, int64_t head_dim,
               int64_t x_token_stride, int64_t x_head_stride, const int32_t* positions,
               const float* table, int64_t max_pos, int64_t rot_dim, uint32_t flags, void* y,
               int64_t y_token_stride, int64_t y_head_stride, hipStream_t stream)
{
    if (!dtype_ok(dtype))
        return NVFP4_ERR_FLAGS;
    if (tokens < 0 || heads <= 0 || head_dim <= 0 || head_dim % 16 != 0)
        return NVFP4_ERR_SHAPE;
    int st = rope_status(head_dim, max_pos, rot_dim, flags, NVFP4_ROPE_INTERLEAVED | NVFP4_ROPE_ADJOINT);
    if (st != NVFP4_OK)
        return st;
    if (heads > (1 << 20) || head_dim > (1 << 13))
        return NVFP4_ERR_SIZE;
    if ((st = strides_status(dtype, tokens, heads, head_dim, x_token_stride, x_head_stride)) != NVFP4_OK ||
        (st = strides_status(dtype, tokens, heads, head_dim, y_token_stride, y_head_stride)) != NVFP4_OK)
        return st;
    if (overlaps(tokens, heads, head_dim, y_token_stride, y_head_stride))
        return NVFP4_ERR_SHAPE;
    if (tokens == 0)
        return NVFP4_OK;
    if (x == nullptr || y == nullptr || positions == nullptr || table == nullptr)
        return NVFP4_ERR_NULL;
    if (!aligned16(x) || !aligned16(y) || !aligned16(table) || !aligned4(positions))
        return NVFP4_ERR_ALIGN;
    if (x == y && (x_token_stride != y_token_stride || x_head_stride != y_head_stride))
        return NVFP4_ERR_FLAGS;
    nvfp4::RopeArgs a{};
    a.x = x;
    a.y = y;
    a.dtype = dtype;
    a.tokens = tokens;
    a.by_heads = nvfp4::DivBy::of((uint32_t)heads);
    a.by_units = nvfp4::DivBy::of((uint32_t)(head_dim / 16));
    a.x_ts = x_token_stride;
    a.x_hs = x_head_stride;
    a.y_ts = y_token_stride;
    a.y_hs = y_head_stride;
    a.positions = positions;
    a.table = table;
    a.max_pos = (int)max_pos;
    a.rot_dim = (int)rot_dim;
    a.interleaved = (flags & NVFP4_ROPE_INTERLEAVED) != 0;
    a.sign = (flags & NVFP4_ROPE_ADJOINT) ? 0x80000000u : 0u;
    return status_of(nvfp4::launch_rope(a, stream));
}

int nvfp4_kv_append(const void* k, const void* v, int dtype, int64_t tokens,
                    int64_t kv_token_stride, int64_t kv_head_stride, const void* q, void* q_out,
                    int64_t heads, int64_t q_token_stride, int64_t q_head_stride,
                    int64_t q_out_token_stride, int64_t q_out_head_stride, const int32_t* positions,
                    const int32_t* seq, const int32_t* page_table, int64_t batch,
                    int64_t table_stride, const float* table, int64_t max_pos, int64_t rot_dim,
                    uint32_t flags, uint8_t* data, int64_t num_pages, int64_t kv_heads,
                    int64_t page_size, int64_t head_dim, const float* k_amax, const float* v_amax,
                    hipStream_t stream)
{
    if (!dtype_ok(dtype))
        return NVFP4_ERR_FLAGS;
    nvfp4::KvAppendArgs a{};
    int st = cache_status(data, num_pages, kv_heads, page_size, head_dim, k_amax, v_amax, page_table, batch,
                          table_stride, a.c);
    if (st != NVFP4_OK)
        return st;
    if (tokens < 0 || heads < 0)
        return NVFP4_ERR_SHAPE;
    if ((q != nullptr) != (heads > 0) || (q_out != nullptr) != (heads > 0) || (heads > 0 && table == nullptr))
        return NVFP4_ERR_NULL;
    if (table != nullptr) {
        if ((st = rope_status(head_dim, max_pos, rot_dim, flags, NVFP4_ROPE_INTERLEAVED)) != NVFP4_OK)
            return st;
    } else if (rot_dim != 0 || flags != 0) {
        return NVFP4_ERR_FLAGS;
    }
    if (tokens > kMaxTokens || heads > kMaxUnits || (heads + 2 * kv_heads) * (head_dim / 16) > kMaxUnits - 16)
        return NVFP4_ERR_SIZE;
    if ((st = strides_status(dtype, tokens, kv_heads, head_dim, kv_token_stride, kv_head_stride)) != NVFP4_OK)
        return st;
    if (heads > 0 &&
        ((st = strides_status(dtype, tokens, heads, head_dim, q_token_stride, q_head_stride)) != NVFP4_OK ||
         (st = strides_status(dtype, tokens, heads, head_dim, q_out_token_stride, q_out_head_stride)) != NVFP4_OK))
        return st;
    if (heads > 0 && overlaps(tokens, heads, head_dim, q_out_token_stride, q_out_head_stride))
        return NVFP4_ERR_SHAPE;
    if (tokens == 0)
        return NVFP4_OK;
    if (k == nullptr || v == nullptr || positions == nullptr)
        return NVFP4_ERR_NULL;
    if (!aligned16(k) || !aligned16(v) || !aligned16(q) || !aligned16(q_out) || !aligned16(table) ||
        !aligned4(positions) || !aligned4(seq))
        return NVFP4_ERR_ALIGN;
    if (heads > 0 && q == q_out && (q_token_stride != q_out_token_stride || q_head_stride != q_out_head_stride))
        return NVFP4_ERR_FLAGS;
    if (seq == nullptr && tokens > batch)
        return NVFP4_ERR_SHAPE;  // tokens of no sequence
    a.data = data;
    a.k = k;
    a.v = v;
    a.q = q;
    a.q_out = q_out;
    a.dtype = dtype;
    a.tokens = tokens;
    a.heads = (int)heads;
    a.kv_ts = kv_token_stride;
    a.kv_hs = kv_head_stride;
    a.q_ts = q_token_stride;
    a.q_hs = q_head_stride;
    a.qo_ts = q_out_token_stride;
    a.qo_hs = q_out_head_stride;
    a.positions = positions;
    a.seq = seq;
    a.table = table;
    a.max_pos = (int)max_pos;
    a.rot_dim = (int)rot_dim;
    a.interleaved = (flags & NVFP4_ROPE_INTERLEAVED) != 0;
    return status_of(nvfp4::launch_kv_append(a, stream));
}

int nvfp4_kv_read(const uint8_t* data, int64_t num_pages, int64_t kv_heads, int64_t page_size,
                  int64_t head_dim, const float* k_amax, const float* v_amax, int64_t tokens,
                  const int32_t* positions, const int32_t* seq, const int32_t* page_table,
                  int64_t batch, int64_t table_stride, void* k_out, void* v_out, int out_dtype,
                  hipStream_t stream)
{
    if (!dtype_ok(out_dtype))
        return NVFP4_ERR_FLAGS;
    nvfp4::KvReadArgs a{};
    const int st = cache_status(data, num_pages, kv_heads, page_size, head_dim, k_amax, v_amax, page_table, batch,
                                table_stride, a.c);
    if (st != NVFP4_OK)
        return st;
    if (tokens < 0)
        return NVFP4_ERR_SHAPE;
    if (tokens > kMaxTokens || 2 * kv_heads * (head_dim / 16) > kMaxUnits)
        return NVFP4_ERR_SIZE;
    if (tokens == 0)
        return NVFP4_OK;
    if (positions == nullptr || (k_out == nullptr && v_out == nullptr))
        return NVFP4_ERR_NULL;
    if (!aligned16(k_out) || !aligned16(v_out) || !aligned4(positions) || !aligned4(seq))
        return NVFP4_ERR_ALIGN;
    if (seq == nullptr && tokens > batch)
        return NVFP4_ERR_SHAPE;  // tokens of no sequence
    a.data = data;
    a.tokens = tokens;
    a.positions = positions;
    a.seq = seq;
    a.k_out = k_out;
    a.v_out = v_out;
    a.dtype = out_dtype;
    return status_of(nvfp4::launch_kv_read(a, stream));
}

int nvfp4_kv_attention(const void* q, int dtype, int64_t total_q, int64_t heads,
                       int64_t q_token_stride, int64_t q_head_stride, const int32_t* cu_q,
                       int64_t max_q, const uint8_t* data, int64_t num_pages, int64_t kv_heads,
                       int64_t page_size, int64_t head_dim, const float* k_amax,
                       const float* v_amax, const int32_t* page_table, int64_t batch,
                       int64_t table_stride, const int32_t* lens, float scale, int64_t window,
                       uint32_t flags, void* out, float* lse, void* workspace, hipStream_t stream)
{
    if ((dtype != NVFP4_BF16 && dtype != NVFP4_F16) || (flags & ~NVFP4_KV_CAUSAL) != 0 || !(scale > 0.0f) ||
        !isfinite(scale))
        return NVFP4_ERR_FLAGS;
    if (batch == 0 && total_q == 0)
        return NVFP4_OK;  // no sequences (and perhaps no page table)
    nvfp4::KvAttentionArgs a{};
    int st = cache_status(data, num_pages, kv_heads, page_size, head_dim, k_amax, v_amax, page_table, batch,
                          table_stride, a.c);
    if (st != NVFP4_OK)
        return st;
    if (total_q < 0 || max_q < 1 || window < 0 || heads <= 0 || heads % kv_heads != 0 ||
        (cu_q == nullptr && (max_q > kMaxLen || total_q != batch * max_q)))
        return NVFP4_ERR_SHAPE;
    if (total_q > kMaxInt || max_q > kMaxLen || heads > 65535 || max_q > kMaxLen / (heads / kv_heads))
        return NVFP4_ERR_SIZE;
    const int64_t tiles = ((max_q < total_q ? max_q : total_q) * (heads / kv_heads) + 127) / 128;
    if (batch > kMaxItems / kv_heads || tiles > kMaxItems / (batch * kv_heads))
        return NVFP4_ERR_SIZE;
    if (total_q > batch * max_q)
        return NVFP4_ERR_SHAPE;  // some sequence has more than max_q
    if ((st = strides_status(dtype, total_q, heads, head_dim, q_token_stride, q_head_stride)) != NVFP4_OK)
        return st;
    if (total_q == 0)
        return NVFP4_OK;
    if (q == nullptr || lens == nullptr || out == nullptr || workspace == nullptr)
        return NVFP4_ERR_NULL;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || !aligned4(cu_q) || !aligned4(lens) ||
        !aligned4(lse))
        return NVFP4_ERR_ALIGN;
    a.data = data;
    a.q = q;
    a.dtype = dtype;
    a.total_q = total_q;
    a.max_q = max_q < total_q ? max_q : total_q;
    a.heads = (int)heads;
    a.q_ts = q_token_stride;
    a.q_hs = q_head_stride;
    a.cu_q = cu_q;
    a.lens = lens;
    a.scale = scale;
    a.window = window < kMaxLen ? (int)window : 0;  // no sequence is longer: no window
    a.causal = (flags & NVFP4_KV_CAUSAL) != 0;
    a.out = out;
    a.lse = lse;
    a.workspace = static_cast<uint32_t*>(workspace);
    return status_of(nvfp4::launch_kv_attention(a, stream));
}

}  // extern "C"
