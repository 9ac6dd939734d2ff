/*
 * specdec_rows.cuh -- what the cache operators share: the ragged row layout, element types,
 * rotary angles, the checks of a cache description.
 */
#ifndef SPECDEC_ROWS_CUH
#define SPECDEC_ROWS_CUH

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

#include "specdec.h"

namespace specdec {

inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline size_t elem_bytes(specdec_dtype_t t)
{
    return t == SPECDEC_F32 ? 4 : t == SPECDEC_E4M3 ? 1 : 2;
}

inline bool is_float_type(specdec_dtype_t t) { return t == SPECDEC_F32 || t == SPECDEC_BF16 || t == SPECDEC_F16; }

inline specdec_status_t check_rope(const specdec_rope_t* r, int32_t head_dim)
{
    if (!r->freq || !aligned_to(r->freq, 8) || r->rot_dim < 2 || (r->rot_dim & 1) || r->rot_dim > head_dim ||
        (r->interleaved != 0 && r->interleaved != 1))
        return SPECDEC_ERR_INVALID_ARG;
    return SPECDEC_OK;
}

inline bool cache_head_dim(int32_t d) { return d >= 16 && d <= 128 && d % 16 == 0; }

inline specdec_status_t check_cache(const specdec_kv_cache_t* c)
{
    if (!c) return SPECDEC_ERR_INVALID_ARG;
    if (c->dtype != SPECDEC_BF16 && c->dtype != SPECDEC_F16 && c->dtype != SPECDEC_E4M3) return SPECDEC_ERR_UNSUPPORTED;
    const int ps = c->page_size, es = (int)elem_bytes(c->dtype);
    if (ps != 16 && ps != 32 && ps != 64 && ps != 128 && ps != 256) return SPECDEC_ERR_UNSUPPORTED;
    if (!cache_head_dim(c->head_dim)) return SPECDEC_ERR_UNSUPPORTED;
    if (!c->k || !c->v || !aligned_to(c->k, 16) || !aligned_to(c->v, 16) || c->num_pages < 1 || c->num_kv_heads < 1)
        return SPECDEC_ERR_INVALID_ARG;
    const int64_t st[3] = {c->page_stride, c->head_stride, c->slot_stride};
    for (int64_t s : st)
        if (s < 0 || s > ((int64_t)1 << 38) || (s * es) % 16 != 0) return SPECDEC_ERR_INVALID_ARG;
    if (c->dtype == SPECDEC_E4M3 ? (!c->k_exp || !c->v_exp) : (c->k_exp || c->v_exp)) return SPECDEC_ERR_INVALID_ARG;
    if (!aligned_to(c->k_exp, 16) || !aligned_to(c->v_exp, 16)) return SPECDEC_ERR_INVALID_ARG;
    return SPECDEC_OK;
}

// These kernels are launched as programmatic dependents of what the stream holds before them: a launch is set up while
// its predecessor still runs, and waits for its end (and its writes) here, before anything else is read or written.
// The next launch may be set up from here on.
__device__ __forceinline__ void after_predecessor()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... P, typename... A>
inline cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A&&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
    if (e != cudaSuccess) (void)cudaGetLastError();
    return e;
}

// Whether request b's rows are known: offsets as SPECDEC_ST_BAD_OFFSETS describes them.
__device__ __forceinline__ bool offsets_ok(const int32_t* cu, int32_t B, int b)
{
    const int32_t a0 = __ldg(cu + b), a1 = __ldg(cu + b + 1);
    return __ldg(cu) == 0 && a0 >= 0 && a1 >= a0 && a1 <= __ldg(cu + B);
}

// And whether there are as many rows as they name.
__device__ __forceinline__ bool rows_ok(const int32_t* cu, int32_t B, int b, int64_t rows)
{
    return offsets_ok(cu, B, b) && (int64_t)__ldg(cu + b + 1) + b < rows;
}

// Of n rows from row0 on, how many the requests have (as far as the offsets' total says): those behind are not read.
__device__ __forceinline__ int rows_there(const int32_t* cu, int32_t B, int64_t row0, int n)
{
    return (int)max((int64_t)0, min((int64_t)n, (int64_t)__ldg(cu + B) + B - row0));
}

// The request that owns row t, by counting the requests that start at or before it (every thread
// of the CTA calls it; one round of independent loads per 256 requests, where a search would
// wait out a chain of them). `first` is start(threadIdx.x), which the caller may have read ahead.
// The caller checks that the request really holds the row.
template <int kThreads, typename Start>
__device__ __forceinline__ int owner_of(int32_t B, int64_t t, int64_t first, Start start)
{
    int n = 0;
    for (int base = 0; base < B; base += kThreads) {
        const int b = base + (int)threadIdx.x;
        n += __syncthreads_count(b < B && (base == 0 ? first : start(b)) <= t);
    }
    return n - 1;
}
template <int kThreads, typename Start>
__device__ __forceinline__ int owner_of(int32_t B, int64_t t, Start start)
{
    return owner_of<kThreads>(B, t, (int)threadIdx.x < B ? start((int)threadIdx.x) : 0, start);
}

// cos and sin of position * freq (units of 2^-64 turn): the product wraps modulo one turn, the
// nearest quarter is taken off in integers, and all of the rest, at most an eighth of a turn, goes to fp32
// once, with a relative error of 2^-24 however small it is.
__device__ __forceinline__ float2 turn(int64_t position, uint64_t freq, float amplitude)
{
    const uint64_t phase = (uint64_t)position * freq;
    const uint32_t quarter = (uint32_t)((phase + (1ull << 61)) >> 62);
    const int64_t rest = (int64_t)(phase - ((uint64_t)quarter << 62));
    float s, c;
    sincospif(__ll2float_rn(rest) * 0x1p-63f, &s, &c);
    const float cq = (quarter & 1u) ? s : c, sq = (quarter & 1u) ? c : s;
    return make_float2(((quarter + 1u) & 2u) ? -cq * amplitude : cq * amplitude,
                       (quarter & 2u) ? -sq * amplitude : sq * amplitude);
}

template <typename T> __device__ __forceinline__ float to_float(T x);
template <> __device__ __forceinline__ float to_float<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float to_float<__half>(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float to_float<__nv_fp8_e4m3>(__nv_fp8_e4m3 x) { return (float)x; }

template <typename T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ float from_float<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }

// N consecutive elements as they lie: read and written in 16-byte accesses where N elements fill them, in 8-byte ones
// where they fill those (the caller knows the address to be aligned then), else one by one; the halves of a
// load and its use may so be far apart.
template <typename T, int N> struct Raw {
    static constexpr int kBytes = N * (int)sizeof(T);
    static constexpr bool kWide = kBytes % 8 == 0 && N > 1;
    alignas(16) T e[N];
    __device__ __forceinline__ void load(const T* p)
    {
        if constexpr (kBytes % 16 == 0 && kWide) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i) reinterpret_cast<uint4*>(e)[i] = reinterpret_cast<const uint4*>(p)[i];
        } else if constexpr (kWide) {
#pragma unroll
            for (int i = 0; i < kBytes / 8; ++i) reinterpret_cast<uint2*>(e)[i] = reinterpret_cast<const uint2*>(p)[i];
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) e[i] = p[i];
        }
    }
    __device__ __forceinline__ void store(T* p) const
    {
        if constexpr (kBytes % 16 == 0 && kWide) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i) reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(e)[i];
        } else if constexpr (kWide) {
#pragma unroll
            for (int i = 0; i < kBytes / 8; ++i) reinterpret_cast<uint2*>(p)[i] = reinterpret_cast<const uint2*>(e)[i];
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) p[i] = e[i];
        }
    }
    __device__ __forceinline__ void to(float* x) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = to_float<T>(e[i]);
    }
    __device__ __forceinline__ void from(const float* x)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = from_float<T>(x[i]);
    }
};

// A place in rows of heads of units that moves on by a fixed number of units, without divisions on the way.
struct Place {
    int r, h, u;
    __device__ __forceinline__ Place(int i, int heads, int units)
    {
        const int w = i / units;
        u = i - w * units;
        r = w / heads;
        h = w - r * heads;
    }
    __device__ __forceinline__ void move(const Place& by, int heads, int units)
    {
        u += by.u;
        h += by.h;
        r += by.r;
        if (u >= units) u -= units, ++h;
        if (h >= heads) h -= heads, ++r;
    }
};

// A head is taken in units of 2V elements: the two runs of V that rotate together (half layout), 2V
// consecutive ones (interleaved layout, and the elements behind rot_dim). Needs rot_dim and
// head_dim to be multiples of 2V. Offsets of unit u's two runs:
template <int V>
__device__ __forceinline__ void unit_runs(int u, int rot_dim, int interleaved, int* first, int* second)
{
    const int half = rot_dim / 2;
    if (!interleaved && u * V < half) {
        *first = u * V;
        *second = half + u * V;
    } else {
        *first = 2 * u * V;
        *second = 2 * u * V + V;
    }
}

// Rotates unit u (already loaded) by the row's table cs[pair]; a unit behind rot_dim stays.
template <int V>
__device__ __forceinline__ void rotate_unit(float* x, int u, int rot_dim, int interleaved, const float2* cs)
{
    if (u * V >= rot_dim / 2) return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float2 t = cs[u * V + i];
        if (interleaved) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = a * t.x - b * t.y;
            x[2 * i + 1] = b * t.x + a * t.y;
        } else {
            const float a = x[i], b = x[V + i];
            x[i] = a * t.x - b * t.y;
            x[V + i] = b * t.x + a * t.y;
        }
    }
}

// The scale of an e4m3 head: the value of an exponent byte (0 is 2^-127, 255 stands for no number).
__device__ __forceinline__ float exp_value(uint32_t byte)
{
    return byte == 255u ? __int_as_float(0x7fffffff) : __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

}  // namespace specdec

#endif  // SPECDEC_ROWS_CUH
