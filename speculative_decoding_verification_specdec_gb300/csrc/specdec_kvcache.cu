/*
 * specdec_kvcache.cu -- the paged key-value cache for GB300 (sm_103a): rows of a step written into
 * their pages (keys rotated, heads quantised on the way) and tokens read back; C-ABI entry points
 * in include/specdec.h.
 *
 * Quantisation: an e4m3 head (one token, one head) carries the power of two 2^e with
 * max |x| in (224, 448] 2^e. Scaling by a power of two is exact, so the only rounding is the one to
 * e4m3's three mantissa bits (relative error at most 2^-4), and the scale takes one byte.
 *
 * Both kernels only move data: bound by HBM. Measured on one GB300, calls through the binding: a prompt
 * into a bf16 cache 40.6 us where the copy rate would take 32.2 (79 %); prefixes out of an e4m3 cache 123.6 us for
 * 109.6 (89 %; 139 before four units a thread were in flight). A step's rows into an e4m3 cache take 4 us on
 * the GPU and 15.2 through the binding: small calls are bound by the host.
 */
#include "specdec_rows.cuh"

namespace {

using namespace specdec;

constexpr int kThreads = 256;
constexpr int kMaxRows = 32;
constexpr int kReadBatch = 4;             // units of 16 elements a thread has in flight

struct Table {
    const int32_t* block_table;
    int64_t block_stride;
    int32_t max_blocks;
};

struct WriteArgs {
    const void *k, *v;
    int64_t row_stride, head_stride;
    int32_t rows, rows_per_cta;
    int32_t has_rope;
    specdec_rope_t rope;
    const int32_t* positions;
    specdec_kv_cache_t cache;
    Table table;
    const int32_t *cached, *cu;
    int32_t B;
    uint32_t* status;
};

struct RowSlot {
    int64_t at;        // element offset of (page, head 0, slot)
    int64_t exp_at;    // byte offset of the same in k_exp, v_exp
    int64_t position;
    int32_t live;
};

__device__ __forceinline__ RowSlot no_slot() { return RowSlot{0, 0, 0, 0}; }

// Page and slot of token i of request b; a bad page id is reported and leaves the row dead (-1).
__device__ __forceinline__ RowSlot slot_of(const specdec_kv_cache_t& c, const Table& t, int b, int64_t i, uint32_t* status)
{
    const int page = __ldg(t.block_table + b * t.block_stride + i / c.page_size);
    RowSlot r = no_slot();
    if (page < 0 || page >= c.num_pages) {
        if (status) atomicOr(status + b, SPECDEC_ST_BAD_PAGE);
        r.live = -1;
        return r;
    }
    const int slot = (int)(i % c.page_size);
    r.at = page * c.page_stride + slot * c.slot_stride;
    r.exp_at = (int64_t)page * c.num_kv_heads * c.page_size + slot;
    r.live = 1;
    return r;
}

__device__ __forceinline__ bool fits(const specdec_kv_cache_t& c, const Table& t, int64_t tokens)
{
    return tokens <= (int64_t)t.max_blocks * c.page_size;
}

// The exponent of an e4m3 head: smallest e >= -126 with top <= 448 2^e (0 for a head of zeros).
// top = m 2^x with m in [0.5, 1), 448 = 0.875 2^9.
__device__ __forceinline__ int e4m3_exponent(float top)
{
    if (top == 0.f) return 0;
    int x;
    const float m = frexpf(top, &x);
    return max(m <= 0.875f ? x - 9 : x - 8, -126);
}

// N finite (or NaN) values times a power of two, to nearest e4m3, of which the largest is at most 448.
template <int N> __device__ __forceinline__ void store_e4m3(uint8_t* p, const float* x, float inverse_scale)
{
    if constexpr (N == 1) {
        *p = (uint8_t)__nv_cvt_float_to_fp8(x[0] * inverse_scale, __NV_SATFINITE, __NV_E4M3);
    } else {
        static_assert(N == 8, "an 8-byte store");
        uint32_t two[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            two[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * inverse_scale, x[2 * i + 1] * inverse_scale), __NV_SATFINITE, __NV_E4M3);
        *reinterpret_cast<uint2*>(p) = make_uint2(two[0] | two[1] << 16, two[2] | two[3] << 16);
    }
}

// A head is held by a group of kLanes lanes, kUnits units of 2V elements a lane, so that its largest
// magnitude is a shuffle reduction and its elements are read once. The group's first head is read before the rows'
// places are known.
// V = 8: 16-byte runs, groups of 8 lanes (head_dim <= 128); V = 1 takes any even rot_dim and any
// alignment of the inputs with a warp a head.
template <typename T, typename C, int V, int kLanes, int kUnits>
__global__ void __launch_bounds__(kThreads, 6) specdec_kv_write_kernel(const WriteArgs a)
{
    extern __shared__ float2 cs[];                                 // [rows_per_cta][rot_dim / 2]
    __shared__ RowSlot slots[kMaxRows];
    after_predecessor();
    const specdec_kv_cache_t& c = a.cache;
    const int tid = threadIdx.x;
    const int64_t row0 = (int64_t)blockIdx.x * a.rows_per_cta;
    const int n = (int)min((int64_t)a.rows_per_cta, a.rows - row0);
    const int half = a.has_rope ? a.rope.rot_dim / 2 : 0;
    const int units = c.head_dim / (2 * V), H = c.num_kv_heads, total = n * 2 * H;
    const int lane = tid % kLanes, group = tid / kLanes;
    constexpr int kGroups = kThreads / kLanes;

    Raw<T, V> raw[kUnits][2];
    const Place step(kGroups, 2 * H, 1);
    Place ahead(group, 2 * H, 1), at = ahead;                      // row, and head of K (below H) or V, next to read, to write
    auto fetch = [&](bool in) {
        if (in) {
            const int is_v = ahead.h >= H, h = ahead.h - is_v * H;
            const T* src = static_cast<const T*>(is_v ? a.v : a.k) + (row0 + ahead.r) * a.row_stride + h * a.head_stride;
#pragma unroll
            for (int q = 0; q < kUnits; ++q) {
                const int u = lane + q * kLanes;
                if (u >= units) continue;
                int first, second;
                unit_runs<V>(u, 2 * half, a.rope.interleaved, &first, &second);
                raw[q][0].load(src + first);
                raw[q][1].load(src + second);
            }
        }
        ahead.move(step, 2 * H, 1);
    };
    const int there = rows_there(a.cu, a.B, row0, n) * 2 * H;
    fetch(group < there);

    if (a.status)
        for (int64_t b = (int64_t)blockIdx.x * kThreads + tid; b < a.B; b += (int64_t)gridDim.x * kThreads) {
            if (!rows_ok(a.cu, a.B, (int)b, a.rows)) atomicOr(a.status + b, SPECDEC_ST_BAD_OFFSETS);
            else if (a.cached[b] < 0 || !fits(c, a.table, (int64_t)a.cached[b] + a.cu[b + 1] - a.cu[b] + 1))
                atomicOr(a.status + b, SPECDEC_ST_BAD_LENGTH);
        }
    int b = owner_of<kThreads>(a.B, row0, [&](int i) { return (int64_t)__ldg(a.cu + i) + i; });
    if (tid < n) {
        const int64_t t = row0 + tid;
        b = max(b, 0);
        while (b < a.B && t > (int64_t)__ldg(a.cu + b + 1) + b) ++b;
        RowSlot r = no_slot();
        if (b < a.B && rows_ok(a.cu, a.B, b, a.rows)) {
            const int64_t j = t - __ldg(a.cu + b) - b, k = (int64_t)__ldg(a.cu + b + 1) - __ldg(a.cu + b);
            const int64_t cached = __ldg(a.cached + b);
            if (j >= 0 && cached >= 0 && fits(c, a.table, cached + k + 1)) {
                r = slot_of(c, a.table, b, cached + j, a.status);
                r.position = a.positions ? a.positions[t] : cached + j;
            }
        }
        slots[tid] = r;
    }
    __syncthreads();
    for (int i = tid; i < n * half; i += kThreads) {
        const int r = i / half;
        cs[i] = turn(slots[r].position, __ldg(a.rope.freq + (i - r * half)), a.rope.amplitude);
    }
    __syncthreads();

    // (whole warps go round together: the reduction needs their lanes)
    for (int round = 0; round < total; round += kGroups, at.move(step, 2 * H, 1)) {
        const bool in = round + group < total;
        if (round > 0) fetch(round + group < there);
        const int r = in ? at.r : 0, is_v = at.h >= H, h = at.h - is_v * H;
        const bool live = in && slots[r].live == 1;
        float x[kUnits][2 * V];
        float top = 0.f;
        if (live) {
#pragma unroll
            for (int q = 0; q < kUnits; ++q) {
                const int u = lane + q * kLanes;
                if (u >= units) continue;
                raw[q][0].to(x[q]);
                raw[q][1].to(x[q] + V);
                if (!is_v) rotate_unit<V>(x[q], u, 2 * half, a.rope.interleaved, cs + r * half);
#pragma unroll
                for (int i = 0; i < 2 * V; ++i) top = fmaxf(top, fabsf(x[q][i]));      // (fmaxf passes over NaN)
            }
        }
        int e = 0;
        if constexpr (sizeof(C) == 1) {
            if (__any_sync(0xffffffffu, top == INFINITY)) {
                // infinities become NaN and leave the scale to the others
                top = 0.f;
                if (live) {
#pragma unroll
                    for (int q = 0; q < kUnits; ++q)
                        if (lane + q * kLanes < units)
#pragma unroll
                            for (int i = 0; i < 2 * V; ++i) {
                                if (fabsf(x[q][i]) == INFINITY) x[q][i] = NAN;
                                top = fmaxf(top, fabsf(x[q][i]));
                            }
                }
            }
#pragma unroll
            for (int off = kLanes / 2; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            e = e4m3_exponent(top);
        }
        if (!live) continue;
        const RowSlot& slot = slots[r];
        C* dst = static_cast<C*>(is_v ? c.v : c.k) + slot.at + h * c.head_stride;
#pragma unroll
        for (int q = 0; q < kUnits; ++q) {
            const int u = lane + q * kLanes;
            if (u >= units) continue;
            int first, second;
            unit_runs<V>(u, 2 * half, a.rope.interleaved, &first, &second);
            if constexpr (sizeof(C) == 1) {
                const float inv = __uint_as_float((uint32_t)(127 - e) << 23);     // 2^-e, e in [-126, 120]
                store_e4m3<V>(reinterpret_cast<uint8_t*>(dst) + first, x[q], inv);
                store_e4m3<V>(reinterpret_cast<uint8_t*>(dst) + second, x[q] + V, inv);
            } else {
                Raw<C, V> y;
                y.from(x[q]);
                y.store(dst + first);
                y.from(x[q] + V);
                y.store(dst + second);
            }
        }
        if constexpr (sizeof(C) == 1)
            if (lane == 0) (is_v ? c.v_exp : c.k_exp)[slot.exp_at + (int64_t)h * c.page_size] = (uint8_t)(e + 127);
    }
}

template <typename T, typename C> specdec_status_t launch_write(WriteArgs a, cudaStream_t stream)
{
    const specdec_kv_cache_t& c = a.cache;
    const int rot = a.has_rope ? a.rope.rot_dim : 0;
    const int64_t per = 16 / (int64_t)sizeof(T);
    const bool wide = rot % 16 == 0 && aligned_to(a.k, 16) && aligned_to(a.v, 16) && a.row_stride % per == 0 &&
                      a.head_stride % per == 0;
    // rows for 608 CTAs (four on each of 152 SMs), up to eight heads a group; never fewer than fill a CTA
    const int groups = wide ? kThreads / 8 : kThreads / 32, heads = 2 * c.num_kv_heads, batch = 8 * groups;
    if (heads >= 1 << 24) return SPECDEC_ERR_UNSUPPORTED;          // (32-bit places within a CTA's rows)
    const int64_t wave = ((int64_t)a.rows + 607) / 608, most = (batch + heads - 1) / heads, fill = (groups + heads - 1) / heads;
    int64_t rpc = wave < most ? wave : most;
    rpc = rpc > fill ? rpc : fill;
    rpc = rpc > kMaxRows ? kMaxRows : rpc;
    a.rows_per_cta = (int)rpc;
    const unsigned grid = (unsigned)(((int64_t)a.rows + rpc - 1) / rpc);
    const size_t smem = (size_t)rpc * (rot / 2) * sizeof(float2);
    const cudaError_t e = wide ? launch_dependent(specdec_kv_write_kernel<T, C, 8, 8, 1>, grid, kThreads, smem, stream, a)
                               : launch_dependent(specdec_kv_write_kernel<T, C, 1, 32, 2>, grid, kThreads, smem, stream, a);
    return e == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

template <typename T> specdec_status_t launch_write_to(const WriteArgs& a, cudaStream_t stream)
{
    if (a.cache.dtype == SPECDEC_BF16) return launch_write<T, __nv_bfloat16>(a, stream);
    if (a.cache.dtype == SPECDEC_F16) return launch_write<T, __half>(a, stream);
    return launch_write<T, __nv_fp8_e4m3>(a, stream);
}

struct ReadArgs {
    specdec_kv_cache_t cache;
    Table table;
    const int32_t* first;
    const int64_t* cu_len;
    int32_t B, rows_per_cta;
    int64_t rows;
    void *out_k, *out_v;
    int64_t out_row, out_head;
    uint32_t* status;
};

// Offsets and range of request b: 0 fine, else the status bit.
__device__ __forceinline__ uint32_t read_fault(const ReadArgs& a, int b)
{
    const int64_t r0 = a.cu_len[b], r1 = a.cu_len[b + 1], end = a.cu_len[a.B];
    if (a.cu_len[0] != 0 || r0 < 0 || r1 < r0 || r1 > end || r1 > a.rows) return SPECDEC_ST_BAD_OFFSETS;
    const int32_t f = a.first ? a.first[b] : 0;
    if (f < 0 || (r1 > r0 && !fits(a.cache, a.table, f + (r1 - r0)))) return SPECDEC_ST_BAD_LENGTH;
    return 0;
}

// Units of 16 elements; kWide: the outputs take 16-byte stores.
template <typename C, typename T, bool kWide>
__global__ void __launch_bounds__(kThreads, 4) specdec_kv_read_kernel(const ReadArgs a)
{
    __shared__ RowSlot slots[kMaxRows];
    after_predecessor();
    const specdec_kv_cache_t& c = a.cache;
    const int tid = threadIdx.x;
    const int64_t row0 = (int64_t)blockIdx.x * a.rows_per_cta;
    const int n = (int)min((int64_t)a.rows_per_cta, a.rows - row0);
    if (a.status)
        for (int64_t b = (int64_t)blockIdx.x * kThreads + tid; b < a.B; b += (int64_t)gridDim.x * kThreads) {
            const uint32_t f = read_fault(a, (int)b);
            if (f) atomicOr(a.status + b, f);
        }
    int b = owner_of<kThreads>(a.B, row0, [&](int i) { return (int64_t)__ldg((const long long*)a.cu_len + i); });
    if (tid < n) {
        const int64_t t = row0 + tid;
        b = max(b, 0);
        while (b < a.B && t >= a.cu_len[b + 1]) ++b;
        RowSlot r = no_slot();
        if (b < a.B && t >= a.cu_len[b] && read_fault(a, b) == 0)
            r = slot_of(c, a.table, b, (a.first ? a.first[b] : 0) + (t - a.cu_len[b]), a.status);
        slots[tid] = r;
    }
    __syncthreads();
    const int units = c.head_dim / 16, H = c.num_kv_heads, row_units = 2 * H * units, total = n * row_units;
    const Place step(kThreads, 2 * H, units);
    Place at(tid, 2 * H, units);
    for (int base = tid; base < total; base += kReadBatch * kThreads) {
        Raw<C, 16> raw[kReadBatch];
        float scale[kReadBatch];
        T* out[kReadBatch];                                        // nullptr: nothing to write
#pragma unroll
        for (int q = 0; q < kReadBatch; ++q, at.move(step, 2 * H, units)) {
            out[q] = nullptr;
            scale[q] = 1.f;
            if (base + q * kThreads >= total) continue;
            const int r = at.r, u = at.u, is_v = at.h >= H, h = at.h - is_v * H;
            const RowSlot& slot = slots[r];
            T* const to = static_cast<T*>(is_v ? a.out_v : a.out_k);
            if (!slot.live || !to) continue;
            out[q] = to + (row0 + r) * a.out_row + h * a.out_head + u * 16;
            if (slot.live > 0) {
                raw[q].load(static_cast<const C*>(is_v ? c.v : c.k) + slot.at + h * c.head_stride + u * 16);
                if constexpr (sizeof(C) == 1) scale[q] = exp_value((is_v ? c.v_exp : c.k_exp)[slot.exp_at + (int64_t)h * c.page_size]);
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) raw[q].e[e] = C();    // a bad page reads as zeros
            }
        }
#pragma unroll
        for (int q = 0; q < kReadBatch; ++q) {
            if (!out[q]) continue;
            float x[16];
            raw[q].to(x);
            if constexpr (sizeof(C) == 1) {
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] *= scale[q];
            }
            if constexpr (kWide) {
                Raw<T, 16> y;
                y.from(x);
                y.store(out[q]);
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) out[q][e] = from_float<T>(x[e]);
            }
        }
    }
}

template <typename C, typename T> specdec_status_t launch_read(ReadArgs a, cudaStream_t stream)
{
    const int64_t per = 16 / (int64_t)sizeof(T);
    const bool wide = aligned_to(a.out_k, 16) && aligned_to(a.out_v, 16) && a.out_row % per == 0 && a.out_head % per == 0;
    const int units = a.cache.head_dim / 16;
    const int64_t row_units = (int64_t)2 * a.cache.num_kv_heads * units;
    if (row_units >= 1 << 24) return SPECDEC_ERR_UNSUPPORTED;      // (32-bit places within a CTA's rows)
    // as the write's: one wave's rows, up to 16 units a thread, never fewer than fill a CTA
    const int64_t wave = (a.rows + 607) / 608, most = (16 * kThreads + row_units - 1) / row_units,
                  fill = (kThreads + row_units - 1) / row_units;
    int64_t rpc = wave < most ? wave : most;
    rpc = rpc > fill ? rpc : fill;
    rpc = rpc > kMaxRows ? kMaxRows : rpc;
    a.rows_per_cta = (int)rpc;
    const int64_t grid = (a.rows + rpc - 1) / rpc;
    if (grid > 0x7fffffff) return SPECDEC_ERR_UNSUPPORTED;
    const cudaError_t e = wide ? launch_dependent(specdec_kv_read_kernel<C, T, true>, (unsigned)grid, kThreads, 0, stream, a)
                               : launch_dependent(specdec_kv_read_kernel<C, T, false>, (unsigned)grid, kThreads, 0, stream, a);
    return e == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

template <typename C> specdec_status_t launch_read_to(const ReadArgs& a, specdec_dtype_t out, cudaStream_t stream)
{
    if (out == SPECDEC_F32) return launch_read<C, float>(a, stream);
    if (out == SPECDEC_BF16) return launch_read<C, __nv_bfloat16>(a, stream);
    return launch_read<C, __half>(a, stream);
}

}  // namespace

extern "C" specdec_status_t specdec_kv_write(const void* k, const void* v, specdec_dtype_t dtype, int32_t rows,
                                             int64_t row_stride, int64_t head_stride, const specdec_rope_t* rope,
                                             const int32_t* positions, const specdec_kv_cache_t* cache,
                                             const int32_t* block_table, int32_t max_blocks, int64_t block_stride,
                                             const int32_t* cached_len, const int32_t* cu_num_draft, int32_t B,
                                             uint32_t* status, void* stream)
{
    if (!is_float_type(dtype)) return SPECDEC_ERR_UNSUPPORTED;
    specdec_status_t rc = check_cache(cache);
    if (rc != SPECDEC_OK) return rc;
    if (rope && (rc = check_rope(rope, cache->head_dim)) != SPECDEC_OK) return rc;
    if (rows < 0 || B < 0 || max_blocks < 0 || block_stride < 0 || row_stride < 0 || head_stride < 0)
        return SPECDEC_ERR_INVALID_ARG;
    if (rows == 0 || B == 0) return SPECDEC_OK;
    if (!k || !v || !block_table || !cached_len || !cu_num_draft) return SPECDEC_ERR_INVALID_ARG;
    const size_t es = elem_bytes(dtype);
    if (!aligned_to(k, es) || !aligned_to(v, es) || !aligned_to(positions, 4) || !aligned_to(block_table, 4) ||
        !aligned_to(cached_len, 4) || !aligned_to(cu_num_draft, 4) || !aligned_to(status, 4))
        return SPECDEC_ERR_INVALID_ARG;
    WriteArgs a = {k, v, row_stride, head_stride, rows, 0, rope != nullptr, rope ? *rope : specdec_rope_t{nullptr, 0, 0, 1.f},
                   positions, *cache, {block_table, block_stride, max_blocks}, cached_len, cu_num_draft, B, status};
    if (dtype == SPECDEC_F32) return launch_write_to<float>(a, (cudaStream_t)stream);
    if (dtype == SPECDEC_BF16) return launch_write_to<__nv_bfloat16>(a, (cudaStream_t)stream);
    return launch_write_to<__half>(a, (cudaStream_t)stream);
}

extern "C" specdec_status_t specdec_kv_read(const specdec_kv_cache_t* cache, const int32_t* block_table,
                                            int32_t max_blocks, int64_t block_stride, const int32_t* first,
                                            const int64_t* cu_len, int32_t B, int64_t rows, void* out_k, void* out_v,
                                            specdec_dtype_t out_dtype, int64_t out_row_stride, int64_t out_head_stride,
                                            uint32_t* status, void* stream)
{
    if (!is_float_type(out_dtype)) return SPECDEC_ERR_UNSUPPORTED;
    const specdec_status_t rc = check_cache(cache);
    if (rc != SPECDEC_OK) return rc;
    if (rows < 0 || B < 0 || max_blocks < 0 || block_stride < 0 || out_row_stride < 0 || out_head_stride < 0)
        return SPECDEC_ERR_INVALID_ARG;
    if (rows == 0 || B == 0) return SPECDEC_OK;
    if (!block_table || !cu_len || (!out_k && !out_v)) return SPECDEC_ERR_INVALID_ARG;
    const size_t es = elem_bytes(out_dtype);
    if (!aligned_to(out_k, es) || !aligned_to(out_v, es) || !aligned_to(block_table, 4) || !aligned_to(first, 4) ||
        !aligned_to(cu_len, 8) || !aligned_to(status, 4))
        return SPECDEC_ERR_INVALID_ARG;
    const ReadArgs a = {*cache, {block_table, block_stride, max_blocks}, first, cu_len, B, 0, rows, out_k, out_v,
                        out_row_stride, out_head_stride, status};
    if (cache->dtype == SPECDEC_BF16) return launch_read_to<__nv_bfloat16>(a, out_dtype, (cudaStream_t)stream);
    if (cache->dtype == SPECDEC_F16) return launch_read_to<__half>(a, out_dtype, (cudaStream_t)stream);
    return launch_read_to<__nv_fp8_e4m3>(a, out_dtype, (cudaStream_t)stream);
}
