/*
 * specdec_distill.cu -- distillation of a drafter from the top logits of a teacher for GB300 (sm_103a): loss, gradient and
 * backward pass; C-ABI entry points in include/specdec.h.
 *
 * Of a row z and a list of ids with the teacher's log-probabilities, with s = softmax(z / temperature), targets t_i on the list,
 * r = 1 - sum t left for all other ids together and M = sum t + r:
 *
 *   loss     w (sum_i t_i (ln t_i - ln s_i) + r (ln r - ln rho)),   rho = sum of s outside the list
 *   gradient w / temperature (M s_j - t_j) on the list, w / temperature (M s_j - r s_j / rho) outside
 *
 * rho is summed over the other ids alone (one minus the listed would lose it where the student is sure): the listed
 * elements are taken out of the row in shared memory. Outside the list the gradient is one exponential times one number,
 * e_j (M / S - r / S_rest).
 *
 * A row is held by a cluster of CTAs, a slice each, in shared memory: it is read from HBM once, for the sums and for the gradient.
 */
#include <atomic>

#include "specdec_logits.cuh"

namespace {

using namespace specdec;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kTileBytes = 100 * 1024;             // the most of a row that a CTA holds at once: two CTAs an SM

struct Args {
    const void* logits;
    int64_t row_stride;
    int32_t V, rows;
    const int32_t* ids;                            // [rows, n]
    const float* logprobs;                         // [rows, n]
    int32_t n;
    float scale, scale_low;                        // log2(e) / temperature as a sum of two
    double inverse;                                // 1 / temperature
    int32_t rest;                                  // 1: what the list leaves is a category; 0: the list is renormalised
    const float* weight;                           // [rows] (backward: the loss's gradient) or nullptr
    float* loss;
    float* stats;                                  // [rows, 2]: ln of the sums of exp(z / temperature), of all ids and of those outside the list
    void* grad;
    int64_t grad_stride;
    uint32_t* status;
    int32_t slice, tile;                           // vectors of a CTA, and of what it holds at once (the slice, or a part)
};

constexpr double kLn2 = 0.69314718055994530941723;

// NaN stays; -infinity becomes the lowest number, so that its product with the scale's small part is no NaN.
__device__ __forceinline__ float not_below_lowest(float x)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(-3.402823466e38f));
    return y;
}
__device__ __forceinline__ float exponent(float z, const Args& a, float ref)
{
    return fmaf(z, a.scale_low, fmaf(z, a.scale, -ref));
}

// Thread i's entry of the list: id, -1 where there is none or it does not count.
struct Entry {
    int32_t id;
    float lp;
    uint32_t fault;
};

// `ids` is filled for the CTA; a barrier is inside.
__device__ __forceinline__ Entry read_entry(const Args& a, int64_t r, int32_t* ids)
{
    const int tid = threadIdx.x;
    Entry e = {-1, -INFINITY, 0};
    if (tid < a.n) {
        e.id = __ldg(a.ids + r * a.n + tid);
        e.lp = __ldg(a.logprobs + r * a.n + tid);
        ids[tid] = e.id;
    }
    __syncthreads();
    if (tid < a.n && e.id != -1) {
        bool bad = e.id < 0 || e.id >= a.V || !(e.lp < INFINITY);
        for (int j = 0; j < tid; ++j) bad |= ids[j] == e.id;
        if (bad) {
            e.id = -1;
            e.fault = SPECDEC_ST_BAD_TARGET;
        }
    }
    return e;
}

// Sums over the CTA of a double a thread; every thread gets it. Two barriers.
__device__ __forceinline__ double sum_64(double x, double* part, int threads)
{
    const int warps = (threads + 31) / 32, warp = threadIdx.x >> 5;
    if (warp < warps) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if ((threadIdx.x & 31) == 0) part[warp] = x;
    }
    __syncthreads();
    double sum = 0.0;
    for (int w = 0; w < warps; ++w) sum += part[w];
    __syncthreads();
    return sum;
}

struct Targets {
    double r, mass;                                // what is left to the rest; the sum of all
    double t;                                      // this thread's
    double log_t;                                  // and its logarithm
};

__device__ __forceinline__ Targets targets_of(const Args& a, const Entry& e, double* part)
{
    Targets t;
    t.log_t = (double)e.lp;
    t.t = e.id >= 0 ? exp((double)e.lp) : 0.0;
    const double sum = sum_64(t.t, part, a.n);
    t.r = 0.0;
    t.mass = sum;
    if (a.rest) {
        t.r = fmax(0.0, 1.0 - sum);
        t.mass = sum + t.r;
    } else if (sum > 0.0) {
        t.t /= sum;
        t.log_t -= log(sum);
        t.mass = 1.0;
    }
    return t;
}

// Store of a vector's elements, those inside the row.
template <typename T> __device__ __forceinline__ void store_vector(const Row<T>& row, T* to, bool aligned, int32_t v, const float* x)
{
    const int32_t at = row.first(v);
    Raw<T, kPer<T>> y;
    y.from(x);
    if (aligned && row.whole(at)) {
        *reinterpret_cast<uint4*>(to + at) = *reinterpret_cast<const uint4*>(y.e);
    } else {
#pragma unroll
        for (int i = 0; i < kPer<T>; ++i)
            if (at + i >= 0 && at + i < row.V) to[at + i] = y.e[i];
    }
}

// Whether the gradient's row lies on the 16-byte grid as the logits' does.
template <typename T> __device__ __forceinline__ bool same_grid(const T* x, const T* y)
{
    return ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(y)) & 15) == 0;
}

__device__ __forceinline__ uint32_t cluster_rank() { uint32_t r; asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r)); return r; }
__device__ __forceinline__ uint32_t cluster_size() { uint32_t r; asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r)); return r; }
__device__ __forceinline__ uint32_t in_cta(const void* p, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void put_64(uint32_t to, double x) { asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(to), "d"(x) : "memory"); }
__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

struct Shared {
    double part[kWarps];
    double peer_S[kMaxCluster], peer_ref[kMaxCluster];
    double inverse_all, each;                      // M over the sum of all at all_ref; weight / temperature
    float refs[kWarps], sums[kWarps];
    float factor, all_ref;
    int32_t ids[SPECDEC_TOP_MAX];
};

template <typename T, bool kGrad> __global__ void __launch_bounds__(kThreads) specdec_distill_kernel(const Args a)
{
    extern __shared__ __align__(16) unsigned char held[];
    __shared__ Shared s;
    after_predecessor();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int64_t r = blockIdx.x / size;
    const T* const z = static_cast<const T*>(a.logits) + r * a.row_stride;
    T* const g = static_cast<T*>(a.grad) + r * a.grad_stride;
    const Row<T> row(z, a.V);
    const int32_t v0 = min((int32_t)rank * a.slice, row.vectors), v1 = min(v0 + a.slice, row.vectors);
    const float w = a.weight ? a.weight[r] : 1.f;
    const bool aligned = kGrad && same_grid(z, g);
    if (w == 0.f) {
        if (kGrad) {
            const float zero[kPer<T>] = {};
            for (int32_t v = v0 + tid; v < v1; v += kThreads) store_vector(row, g, aligned, v, zero);
        }
        if (rank == 0 && tid == 0) {
            a.loss[r] = 0.f;
            if (a.stats) a.stats[2 * r] = a.stats[2 * r + 1] = 0.f;
        }
        return;
    }
    asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");     // (waited for before any CTA writes to another)
    Raw<T, kPer<T>>* const mine = reinterpret_cast<Raw<T, kPer<T>>*>(held);
    auto fetch = [&](int32_t from, int32_t to) {
        for (int32_t v = from + tid; v < to; v += kThreads) {
            const int32_t at = row.first(v);
            if (row.whole(at)) {
                async_copy_16(smem_u32(mine + (v - from)), z + at, 16);
            } else {
                Raw<T, kPer<T>> x;
#pragma unroll
                for (int i = 0; i < kPer<T>; ++i) x.e[i] = at + i >= 0 && at + i < a.V ? z[at + i] : neg_inf<T>();
                mine[v - from] = x;
            }
        }
    };
    fetch(v0, min(v0 + a.tile, v1));

    // the list: targets, and the student's logits there, which every CTA of the cluster reads before any of them writes
    const Entry e = read_entry(a, r, s.ids);
    float top = e.id >= 0 ? to_float<T>(z[e.id]) : -INFINITY;
    float top_ref = ceilf(top * a.scale);
    if (top_ref == -INFINITY) top = -INFINITY;                        // (the lowest numbers, where masks put them)
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top_ref = fmaxf(top_ref, __shfl_xor_sync(0xffffffffu, top_ref, o));
    if (lane == 0) s.refs[warp] = top_ref;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i) top_ref = fmaxf(top_ref, s.refs[i]);
    // Every CTA takes the targets and the listed exponentials in 64 bits: a loss near zero is a small difference of their logarithms.
    const Targets t = targets_of(a, e, s.part);
    const double scale = (double)a.scale + (double)a.scale_low;
    const double up = top == -INFINITY ? -INFINITY : (double)top * scale - (double)top_ref;
    const double S_top = sum_64(exp2(up), s.part, a.n);
    double cross = 0.0;                            // sum of t_i (ln t_i - (z_i / temperature - top_ref ln 2))
    if (rank == 0) cross = sum_64(t.t > 0.0 ? t.t * (t.log_t - up * kLn2) : 0.0, s.part, a.n);
    const bool any = t.mass > 0.0;                 // (an empty list that leaves nothing asks for nothing)

    // the sums over this CTA's part of the row without the listed
    float ref = -INFINITY, S = 0.f;
    for (int32_t from = v0; from < v1; from += a.tile) {
        const int32_t to = min(from + a.tile, v1);
        if (from != v0) {
            __syncthreads();
            fetch(from, to);
        }
        async_copy_wait();
        __syncthreads();
        const int32_t at = e.id - row.first(from);
        if (e.id >= 0 && at >= 0 && at < (to - from) * kPer<T>) reinterpret_cast<T*>(held)[at] = neg_inf<T>();
        __syncthreads();
        for (int32_t v = tid; v < to - from; v += kThreads) {
            const Raw<T, kPer<T>> x = mine[v];
            const float m = vector_max(x);
            if (m * a.scale > ref) {
                const float up_ref = ceilf(m * a.scale);
                S *= reference_step(ref, up_ref);
                ref = up_ref;
            }
            float f[kPer<T>];
            x.to(f);
            const float base = ref == -INFINITY ? 0.f : ref;
            float part = 0.f;
#pragma unroll
            for (int i = 0; i < kPer<T>; ++i) part += exp2_fast(exponent(not_below_lowest(f[i]), a, base));
            S += part;
        }
    }
    warp_join(ref, S);
    if (lane == 0) {
        s.refs[warp] = ref;
        s.sums[warp] = S;
    }
    __syncthreads();
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    if (tid < (int)size) {
        // every CTA gets every CTA's sum: thread i writes into CTA i
        float top_all = -INFINITY;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) top_all = fmaxf(top_all, s.refs[i]);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) sum += (double)s.sums[i] * reference_step_64(s.refs[i], top_all);
        put_64(in_cta(&s.peer_S[rank], tid), sum);
        put_64(in_cta(&s.peer_ref[rank], tid), (double)top_all);
    }
    cluster_barrier();

    float rest_ref = -INFINITY;
    for (uint32_t i = 0; i < size; ++i) rest_ref = fmaxf(rest_ref, (float)s.peer_ref[i]);
    if (tid == 0) {
        double S_rest = 0.0;
        for (uint32_t i = 0; i < size; ++i) S_rest += s.peer_S[i] * reference_step_64((float)s.peer_ref[i], rest_ref);
        const float all_ref = fmaxf(rest_ref, top_ref);
        const double S_all = S_rest * reference_step_64(rest_ref, all_ref) + S_top * reference_step_64(top_ref, all_ref);
        // Where the student leaves nothing to the rest there is no such category.
        const bool tail = S_rest > 0.0 || S_rest != S_rest;
        const double left = tail ? t.r : 0.0, mass = tail ? t.mass : t.mass - t.r;
        const bool none = !(S_all > 0.0) && S_all == S_all;           // no finite logit
        const bool still = none || !any;                              // no gradient
        s.each = still ? 0.0 : (double)w * a.inverse;
        s.inverse_all = none ? 0.0 : mass / S_all;
        s.all_ref = none ? 0.f : all_ref;
        s.factor = still ? 0.f : (float)((s.inverse_all * reference_step_64(rest_ref, all_ref) - (tail ? left / S_rest : 0.0)) * s.each);
        if (rank == 0) {
            const double log_all = log(S_all) + (double)all_ref * kLn2, log_rest = log(S_rest) + (double)rest_ref * kLn2;
            double loss = 0.0;
            if (none) {
                loss = any ? INFINITY : 0.0;
            } else if (any) {
                const double sum = t.mass - t.r;
                loss = cross + (sum > 0.0 ? sum * (log_all - (double)top_ref * kLn2) : 0.0);
                if (left > 0.0) loss += left * (log(left) - (log_rest - log_all));
            }
            a.loss[r] = (float)((double)w * loss);
            if (a.stats) {
                a.stats[2 * r] = (float)log_all;
                a.stats[2 * r + 1] = (float)log_rest;
            }
        }
    }
    if (rank == 0 && a.status) {
        const uint32_t empty = tid == 0 && !(fmaxf(rest_ref, top_ref) > -INFINITY) ? SPECDEC_ST_EMPTY_MASK_ROW : 0u;
        if (e.fault | empty) atomicOr(a.status + r, e.fault | empty);
    }
    if constexpr (!kGrad) return;
    __syncthreads();
    const float factor = s.factor, base = rest_ref == -INFINITY ? 0.f : rest_ref;
    for (int32_t from = v0; from < v1; from += a.tile) {
        const int32_t to = min(from + a.tile, v1);
        if (a.tile < a.slice) {
            __syncthreads();
            fetch(from, to);
            async_copy_wait();
            __syncthreads();
        }
        for (int32_t v = tid; v < to - from; v += kThreads) {
            float f[kPer<T>];
            mine[v].to(f);
#pragma unroll
            for (int i = 0; i < kPer<T>; ++i) f[i] = exp2_fast(exponent(not_below_lowest(f[i]), a, base)) * factor;
            store_vector(row, g, aligned, from + v, f);
        }
    }
    __syncthreads();
    if (e.id >= 0 && e.id >= row.first(v0) && e.id < row.first(v1)) {
        const double share = top == -INFINITY ? 0.0 : exp2((double)top * scale - (double)s.all_ref) * s.inverse_all;
        g[e.id] = from_float<T>((float)((share - t.t) * s.each));
    }
}

// The gradient from the sums that a forward pass kept: element by element, a CTA a chunk of a row.
constexpr int kChunk = 8;                          // vectors a thread

template <typename T> __global__ void __launch_bounds__(kThreads) specdec_distill_backward_kernel(const Args a, const int32_t chunks)
{
    __shared__ double part[kWarps];
    __shared__ int32_t ids[SPECDEC_TOP_MAX];
    __shared__ float s_factor;
    after_predecessor();
    const int tid = threadIdx.x;
    const int64_t r = blockIdx.x / (uint32_t)chunks;
    const int32_t v0 = (int32_t)(blockIdx.x - r * chunks) * (kChunk * kThreads);
    const T* const z = static_cast<const T*>(a.logits) + r * a.row_stride;
    T* const g = static_cast<T*>(a.grad) + r * a.grad_stride;
    const Row<T> row(z, a.V);
    if (v0 >= row.vectors) return;
    const bool aligned = same_grid(z, g);
    const float w = a.weight ? a.weight[r] : 1.f;
    if (w == 0.f) {
        const float zero[kPer<T>] = {};
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
            if (v0 + i * kThreads + tid < row.vectors) store_vector(row, g, aligned, v0 + i * kThreads + tid, zero);
        return;
    }
    Raw<T, kPer<T>> x[kChunk];
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
        const int32_t v = v0 + i * kThreads + tid, at = row.first(v);
        if (v < row.vectors && row.whole(at)) {
            *reinterpret_cast<uint4*>(x[i].e) = *reinterpret_cast<const uint4*>(z + at);
        } else {
#pragma unroll
            for (int k = 0; k < kPer<T>; ++k) x[i].e[k] = at + k >= 0 && at + k < a.V ? z[at + k] : neg_inf<T>();
        }
    }
    const Entry e = read_entry(a, r, ids);
    const Targets t = targets_of(a, e, part);
    const double each = (double)w * a.inverse;
    const double log_all = (double)a.stats[2 * r], log_rest = (double)a.stats[2 * r + 1];
    // the exponentials of this kernel are taken at the rest's sum, or where there is none at that of all
    const bool tail = !(log_rest == -INFINITY), none = log_all == -INFINITY || !(t.mass > 0.0);
    const double left = tail ? t.r : 0.0, mass = tail ? t.mass : t.mass - t.r;
    const float ref = (float)ceil((tail ? log_rest : none ? 0.0 : log_all) / kLn2);
    if (tid == 0) {
        const double rest = tail ? left * exp((double)ref * kLn2 - log_rest) : 0.0;
        s_factor = none ? 0.f : (float)((mass * exp((double)ref * kLn2 - log_all) - rest) * each);
    }
    const int32_t at = e.id;
    const bool here = at >= 0 && at >= row.first(v0) && at < row.first(min(v0 + kChunk * kThreads, row.vectors));
    const float top = here ? to_float<T>(z[at]) : 0.f;                // (before the row is written: the gradient may lie over it)
    __syncthreads();
    const float factor = s_factor;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
        const int32_t v = v0 + i * kThreads + tid;
        if (v >= row.vectors) continue;
        float f[kPer<T>];
        x[i].to(f);
#pragma unroll
        for (int k = 0; k < kPer<T>; ++k) f[k] = exp2_fast(exponent(not_below_lowest(f[k]), a, ref)) * factor;
        store_vector(row, g, aligned, v, f);
    }
    __syncthreads();
    if (here) {
        const double share = top == -INFINITY ? 0.0 : mass * exp((double)top * ((double)a.scale + (double)a.scale_low) * kLn2 - log_all);
        g[at] = from_float<T>(none ? 0.f : (float)((share - t.t) * each));
    }
    if (v0 == 0 && a.status && e.fault) atomicOr(a.status + r, e.fault);
}

// ---------------------------------------------------------------- host

struct Shape {
    int32_t cluster, slice, tile;
};

// A row goes to the fewest CTAs that keep three of them on an SM (64 KB each), more where the rows alone do not
// fill the GPU; what is longer than eight times kTileBytes is read a second time for the gradient.
template <typename T> Shape shape_of(int32_t rows, int32_t V)
{
    const int32_t vectors = most_vectors<T>(V);
    int32_t cluster = 1;
    auto slice = [&] { return (vectors + cluster - 1) / cluster; };
    while (cluster < kMaxCluster && (slice() > 64 * 1024 / 16 || ((int64_t)rows * cluster < 304 && slice() > 8 * 1024 / 16))) cluster *= 2;
    const int32_t s = (slice() + 7) / 8 * 8;
    return Shape{cluster, s, s < kTileBytes / 16 ? s : kTileBytes / 16};
}

cudaError_t launch_clusters(void (*kernel)(Args), const Args& a, const Shape& shape, std::atomic<uint64_t>& allowed, cudaStream_t stream)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = 1ull << (dev & 63);
    for (int attempt = allowed.load() & bit ? 0 : 1; e == cudaSuccess; ++attempt) {
        // (once a device; again where a launch fails, for a device may have been reset)
        if (attempt > 0) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileBytes);
        if (e != cudaSuccess) break;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)((int64_t)a.rows * shape.cluster));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = (size_t)shape.tile * 16;
        cfg.stream = stream;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim = {(unsigned)shape.cluster, 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        if (cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess) {
            allowed |= bit;
            return cudaSuccess;
        }
        if (attempt > 0) e = cudaErrorUnknown;
        (void)cudaGetLastError();
    }
    (void)cudaGetLastError();
    return e;
}

template <typename T> specdec_status_t launch_forward(Args a, cudaStream_t stream)
{
    static std::atomic<uint64_t> allowed[2];
    const Shape shape = shape_of<T>(a.rows, a.V);
    if ((int64_t)a.rows * shape.cluster > 0x7fffffff) return SPECDEC_ERR_UNSUPPORTED;
    a.slice = shape.slice;
    a.tile = shape.tile;
    const cudaError_t e = a.grad ? launch_clusters(specdec_distill_kernel<T, true>, a, shape, allowed[1], stream)
                                 : launch_clusters(specdec_distill_kernel<T, false>, a, shape, allowed[0], stream);
    return e == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

template <typename T> specdec_status_t launch_backward(const Args& a, cudaStream_t stream)
{
    const int32_t chunks = (most_vectors<T>(a.V) + kChunk * kThreads - 1) / (kChunk * kThreads);
    if ((int64_t)a.rows * chunks > 0x7fffffff) return SPECDEC_ERR_UNSUPPORTED;
    const cudaError_t e = launch_dependent(specdec_distill_backward_kernel<T>, (unsigned)((int64_t)a.rows * chunks), kThreads, 0, stream, a, chunks);
    return e == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

specdec_status_t check_distill(const void* logits, specdec_dtype_t dtype, int32_t rows, int32_t V, int64_t row_stride,
                               const int32_t* top_ids, const float* top_logprobs, int32_t n, double temperature, int32_t rest,
                               const float* weight, const float* stats, const void* grad, int64_t grad_row_stride, const uint32_t* status)
{
    const specdec_status_t rc = check_logits(logits, dtype, rows, V, row_stride);
    if (rc != SPECDEC_OK) return rc;
    if (n < 1 || n > SPECDEC_TOP_MAX || !usable_temperature(temperature) || (rest != 0 && rest != 1) || grad_row_stride < 0)
        return SPECDEC_ERR_INVALID_ARG;
    if (rows == 0) return SPECDEC_OK;
    if (!top_ids || !top_logprobs || !aligned_to(top_ids, 4) || !aligned_to(top_logprobs, 4) || !aligned_to(weight, 4) ||
        !aligned_to(stats, 4) || !aligned_to(status, 4) || !aligned_to(grad, elem_bytes(dtype)) || (grad && rows > 1 && grad_row_stride < V))
        return SPECDEC_ERR_INVALID_ARG;
    return SPECDEC_OK;
}

Args args_of(const void* logits, int32_t rows, int32_t V, int64_t row_stride, const int32_t* top_ids, const float* top_logprobs, int32_t n,
             double temperature, int32_t rest, const float* weight, float* loss, float* stats, void* grad, int64_t grad_row_stride,
             uint32_t* status)
{
    const double c = scale_of(temperature);
    return Args{logits, row_stride, V, rows, top_ids, top_logprobs, n, (float)c, (float)(c - (double)(float)c), 1.0 / temperature, rest,
                weight, loss, stats, grad, grad_row_stride, status, 0, 0};
}

}  // namespace

extern "C" specdec_status_t specdec_distill(const void* logits, specdec_dtype_t dtype, int32_t rows, int32_t V, int64_t row_stride,
                                            const int32_t* top_ids, const float* top_logprobs, int32_t n, double temperature,
                                            int32_t rest, const float* weight, float* loss, float* stats, void* grad,
                                            int64_t grad_row_stride, uint32_t* status, void* stream)
{
    const specdec_status_t rc = check_distill(logits, dtype, rows, V, row_stride, top_ids, top_logprobs, n, temperature, rest, weight,
                                              stats, grad, grad_row_stride, status);
    if (rc != SPECDEC_OK || rows == 0) return rc;
    if (!loss || !aligned_to(loss, 4)) return SPECDEC_ERR_INVALID_ARG;
    const Args a = args_of(logits, rows, V, row_stride, top_ids, top_logprobs, n, temperature, rest, weight, loss, stats, grad,
                           grad_row_stride, status);
    if (dtype == SPECDEC_F32) return launch_forward<float>(a, (cudaStream_t)stream);
    if (dtype == SPECDEC_BF16) return launch_forward<__nv_bfloat16>(a, (cudaStream_t)stream);
    return launch_forward<__half>(a, (cudaStream_t)stream);
}

extern "C" specdec_status_t specdec_distill_backward(const void* logits, specdec_dtype_t dtype, int32_t rows, int32_t V,
                                                     int64_t row_stride, const int32_t* top_ids, const float* top_logprobs, int32_t n,
                                                     double temperature, int32_t rest, const float* stats, const float* grad_loss,
                                                     void* grad, int64_t grad_row_stride, uint32_t* status, void* stream)
{
    const specdec_status_t rc = check_distill(logits, dtype, rows, V, row_stride, top_ids, top_logprobs, n, temperature, rest, grad_loss,
                                              stats, grad, grad_row_stride, status);
    if (rc != SPECDEC_OK || rows == 0) return rc;
    if (!stats || !grad) return SPECDEC_ERR_INVALID_ARG;
    const Args a = args_of(logits, rows, V, row_stride, top_ids, top_logprobs, n, temperature, rest, grad_loss, nullptr,
                           const_cast<float*>(stats), grad, grad_row_stride, status);
    if (dtype == SPECDEC_F32) return launch_backward<float>(a, (cudaStream_t)stream);
    if (dtype == SPECDEC_BF16) return launch_backward<__nv_bfloat16>(a, (cudaStream_t)stream);
    return launch_backward<__half>(a, (cudaStream_t)stream);
}
