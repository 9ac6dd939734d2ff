/*
 * specdec_rope.cu -- rotary positions for GB300 (sm_103a); C-ABI entry points in include/specdec.h.
 *
 * Every pair (a, b) of a head's first rot_dim elements turns by the row's position times the
 * pair's frequency. All heads of a row share the angles, so a CTA takes whole rows: its threads first
 * put the rows' cosines and sines into shared memory (rot_dim / 2 pairs a row, one sincospif each),
 * then rotate the heads in 32-byte units. Bound by HBM: every element is read and written once.
 *
 * A thread has four units in flight and reads the first of them before the rows' places are known; few rows
 * are spread over many CTAs. Measured on one GB300, calls through the binding: a prompt whose floor at the
 * copy rate is 29.8 us takes 41.6 (72 %, 4.9 TB/s). The look at the requests' total before the first read, which keeps
 * rows behind it unread, costs 0.5 us of it (1.0 before the first requests' offsets were read beside it). Four units
 * and many CTAs took 1280 query rows from 10.2 to 8.2 us; without the binding they take 4 to 6: the host bounds small calls.
 */
#include <cmath>

#include "specdec_rows.cuh"

namespace {

using namespace specdec;

constexpr int kThreads = 256;
constexpr int kBatch = 4;                 // units a thread has in flight
constexpr int kMaxRows = 16;              // rows a CTA takes at most

struct RopeArgs {
    const void* x;
    void* out;
    int32_t rows, heads, head_dim, units, rows_per_cta, inverse;
    int64_t x_row, x_head, out_row, out_head;
    specdec_rope_t rope;
    const int32_t *positions, *cu, *cached;
    int32_t B;
};

// The first batch is read before the rows' positions are known (only that the requests have so many rows): their
// chain of reads and the angles then cost nothing on top of it.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 3) specdec_rope_kernel(const RopeArgs a)
{
    extern __shared__ float2 cs[];                                 // [rows_per_cta][rot_dim / 2]
    __shared__ int64_t pos[kMaxRows];
    __shared__ int live[kMaxRows];
    after_predecessor();
    const int tid = threadIdx.x, half = a.rope.rot_dim / 2;
    const int64_t row0 = (int64_t)blockIdx.x * a.rows_per_cta;
    const int n = (int)min((int64_t)a.rows_per_cta, a.rows - row0);
    const int row_units = a.heads * a.units, total = n * row_units;
    auto start = [&](int i) { return (int64_t)__ldg(a.cu + i) + i; };
    const int64_t first_start = !a.positions && tid < a.B ? start(tid) : 0;        // (on its way beside the offsets' total)
    const int there = a.positions ? total : rows_there(a.cu, a.B, row0, n) * row_units;
    Raw<T, V> v[kBatch][2];
    const Place step(kThreads, a.heads, a.units);
    Place ahead(tid, a.heads, a.units), at = ahead;                // of the next unit to read, to write
    auto fetch = [&](int base) {
#pragma unroll
        for (int q = 0; q < kBatch; ++q, ahead.move(step, a.heads, a.units)) {
            if (base + q * kThreads >= there) continue;
            int first, second;
            unit_runs<V>(ahead.u, a.rope.rot_dim, a.rope.interleaved, &first, &second);
            const T* x = static_cast<const T*>(a.x) + (row0 + ahead.r) * a.x_row + ahead.h * a.x_head;
            v[q][0].load(x + first);
            v[q][1].load(x + second);
        }
    };
    fetch(tid);
    int b = 0;
    if (!a.positions) b = owner_of<kThreads>(a.B, row0, first_start, start);
    if (tid < n) {
        const int64_t t = row0 + tid;
        if (a.positions) {
            pos[tid] = a.positions[t];
            live[tid] = 1;
        } else {
            b = max(b, 0);
            while (b < a.B && t > (int64_t)__ldg(a.cu + b + 1) + b) ++b;
            const int64_t j = b < a.B ? t - __ldg(a.cu + b) - b : -1;
            const int32_t c = b < a.B ? __ldg(a.cached + b) : -1;
            live[tid] = j >= 0 && c >= 0 && rows_ok(a.cu, a.B, b, a.rows);
            pos[tid] = (int64_t)c + j;
        }
    }
    __syncthreads();
    for (int i = tid; i < n * half; i += kThreads) {
        const int r = i / half;
        float2 t = turn(pos[r], __ldg(a.rope.freq + (i - r * half)), a.rope.amplitude);
        if (a.inverse) t.y = -t.y;
        cs[i] = t;
    }
    __syncthreads();
    for (int base = tid; base < total; base += kBatch * kThreads) {
        if (base != tid) fetch(base);
#pragma unroll
        for (int q = 0; q < kBatch; ++q, at.move(step, a.heads, a.units)) {
            if (base + q * kThreads >= total || !live[at.r]) continue;
            int first, second;
            unit_runs<V>(at.u, a.rope.rot_dim, a.rope.interleaved, &first, &second);
            float x[2 * V];
            v[q][0].to(x);
            v[q][1].to(x + V);
            rotate_unit<V>(x, at.u, a.rope.rot_dim, a.rope.interleaved, cs + at.r * half);
            T* out = static_cast<T*>(a.out) + (row0 + at.r) * a.out_row + at.h * a.out_head;
            Raw<T, V> y;
            y.from(x);
            y.store(out + first);
            y.from(x + V);
            y.store(out + second);
        }
    }
}

template <typename T>
specdec_status_t launch_rope(RopeArgs a, cudaStream_t stream)
{
    // 16-byte runs of eight 16-bit elements (four of fp32) where head, rotated part, strides and
    // pointers allow; element by element otherwise
    constexpr int kV = 16 / (int)sizeof(T);
    const int64_t st[4] = {a.x_row, a.x_head, a.out_row, a.out_head};
    bool wide = a.head_dim % (2 * kV) == 0 && a.rope.rot_dim % (2 * kV) == 0 && aligned_to(a.x, 16) && aligned_to(a.out, 16);
    for (int64_t s : st) wide = wide && s % kV == 0;
    const int V = wide ? kV : 1;
    a.units = a.head_dim / (2 * V);
    const int64_t row_units = (int64_t)a.heads * a.units;
    if (row_units >= 1 << 24) return SPECDEC_ERR_UNSUPPORTED;      // (32-bit places within a CTA's rows)
    // rows for 608 CTAs (four on each of 152 SMs; 80 registers let three run at once, the rest of so small a grid follows
    // as they end), up to a batch of units a thread; never fewer than fill a CTA
    const int64_t wave = ((int64_t)a.rows + 607) / 608, batch = (kBatch * kThreads + row_units - 1) / row_units,
                  fill = (kThreads + row_units - 1) / row_units;
    int64_t rpc = wave < batch ? wave : batch;
    rpc = rpc > fill ? rpc : fill;
    rpc = rpc > kMaxRows ? kMaxRows : rpc;
    a.rows_per_cta = (int)rpc;
    const unsigned grid = (unsigned)(((int64_t)a.rows + a.rows_per_cta - 1) / a.rows_per_cta);
    const size_t smem = (size_t)a.rows_per_cta * (a.rope.rot_dim / 2) * sizeof(float2);
    const cudaError_t e = wide ? launch_dependent(specdec_rope_kernel<T, kV>, grid, kThreads, smem, stream, a)
                               : launch_dependent(specdec_rope_kernel<T, 1>, grid, kThreads, smem, stream, a);
    return e == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

}  // namespace

extern "C" specdec_status_t specdec_rope_frequencies(int32_t rot_dim, double theta, specdec_rope_scaling_t scaling,
                                                     double factor, int64_t original_len, double beta_fast,
                                                     double beta_slow, uint64_t* freq, float* amplitude)
{
    const double kTwoPi = 6.283185307179586476925286766559;
    if (!freq || rot_dim < 2 || (rot_dim & 1) || rot_dim > 256 || !(theta >= 1.0) || !std::isfinite(theta))
        return SPECDEC_ERR_INVALID_ARG;
    if (scaling != SPECDEC_ROPE_PLAIN && scaling != SPECDEC_ROPE_LINEAR && scaling != SPECDEC_ROPE_BY_PARTS)
        return SPECDEC_ERR_INVALID_ARG;
    if (scaling != SPECDEC_ROPE_PLAIN && (!(factor > 0.0) || !std::isfinite(factor))) return SPECDEC_ERR_INVALID_ARG;
    if (scaling == SPECDEC_ROPE_BY_PARTS &&
        (original_len < 1 || !(beta_fast > beta_slow) || !std::isfinite(beta_fast) || !std::isfinite(beta_slow)))
        return SPECDEC_ERR_INVALID_ARG;
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(theta, -2.0 * i / rot_dim);
        if (scaling == SPECDEC_ROPE_LINEAR) f /= factor;
        if (scaling == SPECDEC_ROPE_BY_PARTS) {
            double w = ((double)original_len * f / kTwoPi - beta_slow) / (beta_fast - beta_slow);
            w = w < 0.0 ? 0.0 : w > 1.0 ? 1.0 : w;
            f *= w + (1.0 - w) / factor;
        }
        if (!std::isfinite(f)) return SPECDEC_ERR_INVALID_ARG;     // (a factor whose reciprocal is none)
        const double turns = std::fmod(f / kTwoPi, 1.0);
        freq[i] = (uint64_t)std::ldexp(turns, 64);                 // turns < 1: fits; what is under 2^-64 turn is dropped
    }
    if (amplitude)
        *amplitude = scaling == SPECDEC_ROPE_BY_PARTS && factor > 1.0 ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
    return SPECDEC_OK;
}

extern "C" specdec_status_t specdec_rope(const void* x, void* out, specdec_dtype_t dtype, int32_t rows, int32_t heads,
                                         int32_t head_dim, int64_t x_row_stride, int64_t x_head_stride,
                                         int64_t out_row_stride, int64_t out_head_stride, const specdec_rope_t* rope,
                                         int32_t inverse, const int32_t* positions, const int32_t* cu_num_draft,
                                         const int32_t* cached_len, int32_t B, void* stream)
{
    if (!is_float_type(dtype)) return SPECDEC_ERR_UNSUPPORTED;
    if (head_dim < 2 || (head_dim & 1) || head_dim > 256) return SPECDEC_ERR_UNSUPPORTED;
    if (rows < 0 || heads < 1 || B < 0 || !rope) return SPECDEC_ERR_INVALID_ARG;
    if (x_row_stride < 0 || x_head_stride < 0 || out_row_stride < 0 || out_head_stride < 0) return SPECDEC_ERR_INVALID_ARG;
    const specdec_status_t rc = check_rope(rope, head_dim);
    if (rc != SPECDEC_OK) return rc;
    if (rows == 0 || (!positions && B == 0)) return SPECDEC_OK;
    if (!x || !out || (!positions && (!cu_num_draft || !cached_len))) return SPECDEC_ERR_INVALID_ARG;
    const size_t es = elem_bytes(dtype);
    if (!aligned_to(x, es) || !aligned_to(out, es) || !aligned_to(positions, 4) || !aligned_to(cu_num_draft, 4) ||
        !aligned_to(cached_len, 4))
        return SPECDEC_ERR_INVALID_ARG;
    RopeArgs a = {x, out, rows, heads, head_dim, 0, 0, inverse != 0, x_row_stride, x_head_stride, out_row_stride,
                  out_head_stride, *rope, positions, cu_num_draft, cached_len, B};
    if (dtype == SPECDEC_F32) return launch_rope<float>(a, (cudaStream_t)stream);
    if (dtype == SPECDEC_BF16) return launch_rope<__nv_bfloat16>(a, (cudaStream_t)stream);
    return launch_rope<__half>(a, (cudaStream_t)stream);
}
