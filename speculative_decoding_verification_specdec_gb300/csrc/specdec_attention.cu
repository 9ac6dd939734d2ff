/*
 * specdec_attention.cu -- attention of a verify step's rows over the paged key-value cache for
 * GB300 (sm_103a); C-ABI entry point in include/specdec.h.
 *
 * One CTA per (request row, query head): every warp takes each fourth token, a lane holds up to four
 * elements of the head, the score is a shuffle sum, and a running (m, l, O) keeps the softmax in
 * one pass over the tokens; the four warps' states are joined in shared memory.
 */
#include <cmath>

#include "specdec_rows.cuh"

namespace {

using namespace specdec;

constexpr int kThreads = 128;

struct Args {
    const void* q;
    void* out;
    float* lse;
    int32_t rows, num_heads;
    int64_t q_row, q_head, out_row, out_head;
    specdec_kv_cache_t cache;
    const int32_t* block_table;
    int64_t block_stride;
    int32_t max_blocks;
    const int32_t *cached, *cu;
    int32_t B, max_k, window;
    float scale;
    uint32_t* status;
};

template <typename T, typename C>
__global__ void __launch_bounds__(kThreads) specdec_paged_attention_kernel(const Args a)
{
    __shared__ float sm[4], sl[4], so[4][128];
    const specdec_kv_cache_t& c = a.cache;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, D = c.head_dim;
    const int64_t t = blockIdx.x;
    const int hq = blockIdx.y, h = hq / (a.num_heads / c.num_kv_heads);
    if (a.status && hq == 0)
        for (int64_t b = t * kThreads + tid; b < a.B; b += (int64_t)gridDim.x * kThreads)
            if (!offsets_ok(a.cu, a.B, (int)b)) atomicOr(a.status + b, SPECDEC_ST_BAD_OFFSETS);
    const int b = owner_of<kThreads>(a.B, t, [&](int i) { return (int64_t)__ldg(a.cu + i) + i; });
    if (b < 0 || !offsets_ok(a.cu, a.B, b)) return;
    const int64_t j = t - a.cu[b] - b, k = a.cu[b + 1] - a.cu[b];
    if (j > k) return;
    const int64_t cached = a.cached[b], last = cached + j;
    uint32_t fault = 0;
    if (k > a.max_k) fault = SPECDEC_ST_K_TOO_LARGE;
    else if (cached < 0 || cached + k + 1 > (int64_t)a.max_blocks * c.page_size) fault = SPECDEC_ST_BAD_LENGTH;
    if (fault && a.status && tid == 0) atomicOr(a.status + b, fault);

    float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
    const T* qp = static_cast<const T*>(a.q) + t * a.q_row + hq * a.q_head;
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = lane + 32 * e < D ? to_float<T>(qp[lane + 32 * e]) : 0.f;
    const int64_t begin = fault ? 1 : (a.window > 0 ? max((int64_t)0, last - a.window + 1) : 0), end = fault ? 0 : last + 1;
    for (int64_t i = begin + warp; i < end; i += 4) {
        const int page = a.block_table[b * a.block_stride + i / c.page_size];
        const bool good = page >= 0 && page < c.num_pages;
        if (!good && a.status && lane == 0) atomicOr(a.status + b, SPECDEC_ST_BAD_PAGE);
        const int slot = (int)(i % c.page_size);
        const int64_t at = (good ? page : 0) * c.page_stride + h * c.head_stride + slot * c.slot_stride;
        const int64_t ex = ((int64_t)(good ? page : 0) * c.num_kv_heads + h) * c.page_size + slot;
        float ks = 1.f, vs = 1.f;
        if constexpr (sizeof(C) == 1) { ks = exp_value(c.k_exp[ex]); vs = exp_value(c.v_exp[ex]); }
        float s = 0.f, v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool in = good && lane + 32 * e < D;
            s += in ? q[e] * to_float<C>(static_cast<const C*>(c.k)[at + lane + 32 * e]) : 0.f;
            v[e] = in ? to_float<C>(static_cast<const C*>(c.v)[at + lane + 32 * e]) * vs : 0.f;
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= ks * a.scale;
        const float mn = fmaxf(m, s);
        if (mn == -INFINITY && s == s) continue;                   // nothing seen yet (a NaN score stays)
        const float f = expf(m - mn), p = expf(s - mn);
        m = mn;
        l = l * f + p;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = o[e] * f + p * v[e];
    }
    if (lane == 0) { sm[warp] = m; sl[warp] = l; }
#pragma unroll
    for (int e = 0; e < 4; ++e) so[warp][lane + 32 * e] = o[e];
    __syncthreads();
    const float mm = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    float ll = 0.f, oo = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float f = sm[w] == -INFINITY ? 0.f : expf(sm[w] - mm);
        ll += sl[w] * f;
        oo += so[w][tid] * f;
    }
    T* out = static_cast<T*>(a.out) + t * a.out_row + hq * a.out_head;
    if (tid < D) out[tid] = from_float<T>(ll > 0.f || ll != ll ? oo / ll : 0.f);
    if (a.lse && tid == 0) a.lse[t * a.num_heads + hq] = mm + logf(ll);
}

}  // namespace

extern "C" size_t specdec_paged_attention_workspace_size(int32_t B, int32_t max_k, int32_t num_heads,
                                                         int32_t num_kv_heads, int32_t head_dim)
{
    if (B <= 0 || max_k < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0) return 0;
    return 16;
}

extern "C" specdec_status_t specdec_paged_attention(
    const void* q, specdec_dtype_t dtype, int32_t rows, int32_t num_heads, int64_t q_row_stride, int64_t q_head_stride,
    const specdec_kv_cache_t* cache, const int32_t* block_table, int32_t max_blocks, int64_t block_stride,
    const int32_t* cached_len, const int32_t* cu_num_draft, int32_t B, int32_t max_k, float scale, int32_t window,
    void* out, int64_t out_row_stride, int64_t out_head_stride, float* lse, uint32_t* status, void* workspace,
    size_t workspace_bytes, int32_t wait_limit_us, void* stream)
{
    if (dtype != SPECDEC_BF16 && dtype != SPECDEC_F16) return SPECDEC_ERR_UNSUPPORTED;
    const specdec_status_t rc = check_cache(cache);
    if (rc != SPECDEC_OK) return rc;
    if (cache->dtype != SPECDEC_E4M3 && cache->dtype != dtype) return SPECDEC_ERR_UNSUPPORTED;
    if (rows < 0 || B < 0 || max_blocks < 0 || block_stride < 0 || max_k < 0 || max_k > SPECDEC_KMAX || num_heads < 1 ||
        num_heads % cache->num_kv_heads != 0 || window < 0 || !std::isfinite(scale) || wait_limit_us < -1 ||
        wait_limit_us > 2000000)
        return SPECDEC_ERR_INVALID_ARG;
    const int64_t st[4] = {q_row_stride, q_head_stride, out_row_stride, out_head_stride};
    for (int64_t s : st)
        if (s < 0 || s % 8 != 0) return SPECDEC_ERR_INVALID_ARG;
    if (rows == 0 || B == 0) return SPECDEC_OK;
    if (!q || !out || !block_table || !cached_len || !cu_num_draft || !workspace) return SPECDEC_ERR_INVALID_ARG;
    if (!aligned_to(q, 16) || !aligned_to(out, 16) || !aligned_to(workspace, 16) || !aligned_to(block_table, 4) ||
        !aligned_to(cached_len, 4) || !aligned_to(cu_num_draft, 4) || !aligned_to(lse, 4) || !aligned_to(status, 4) ||
        workspace_bytes < specdec_paged_attention_workspace_size(B, max_k, num_heads, cache->num_kv_heads, cache->head_dim))
        return SPECDEC_ERR_INVALID_ARG;
    const Args a = {q, out, lse, rows, num_heads, q_row_stride, q_head_stride, out_row_stride, out_head_stride, *cache,
                    block_table, block_stride, max_blocks, cached_len, cu_num_draft, B, max_k, window, scale, status};
    const dim3 grid((unsigned)rows, (unsigned)num_heads);
    const cudaStream_t s = (cudaStream_t)stream;
    if (dtype == SPECDEC_BF16) {
        if (cache->dtype == SPECDEC_BF16) specdec_paged_attention_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
        else specdec_paged_attention_kernel<__nv_bfloat16, __nv_fp8_e4m3><<<grid, kThreads, 0, s>>>(a);
    } else {
        if (cache->dtype == SPECDEC_F16) specdec_paged_attention_kernel<__half, __half><<<grid, kThreads, 0, s>>>(a);
        else specdec_paged_attention_kernel<__half, __nv_fp8_e4m3><<<grid, kThreads, 0, s>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}
