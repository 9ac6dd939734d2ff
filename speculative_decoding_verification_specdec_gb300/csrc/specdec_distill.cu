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
#include <cmath>

#include "specdec_logits.cuh"

namespace {

using namespace specdec;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBackThreads = 256;
constexpr int kMaxCluster = 8;
constexpr int kTileBytes = 100 * 1024;             // the most of a row that a CTA holds at once: two CTAs an SM

struct Args {
    const void* logits;
    int64_t row_stride;
    int32_t V, rows;
    const int32_t* ids;                            // [rows, n]
    const float* logprobs;                         // [rows, n]
    int32_t n;
    float scale, scale_low;                        // log2(e) / temperature as a sum of two positive numbers
    float inverse;                                 // 1 / temperature
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

// z log2(e) / temperature - ref: scale and scale_low are both positive, so that -infinity stays what it is.
__device__ __forceinline__ float exponent(float z, const Args& a, float ref)
{
    return fmaf(z, a.scale_low, fmaf(z, a.scale, -ref));
}
// 2 to that, two at a time; kLow: with scale_low.
template <bool kLow> struct Exponentials {
    Pair c, low, less;
    __device__ __forceinline__ Exponentials(const Args& a, float ref)
        : c(pair_of(a.scale, a.scale)), low(pair_of(a.scale_low, a.scale_low)), less(pair_of(-ref, -ref))
    {
    }
    __device__ __forceinline__ Pair operator()(Pair z) const
    {
        return exp2_2(kLow ? fma_2(z, low, fma_2(z, c, less)) : fma_2(z, c, less));
    }
};

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
    if (tid < (a.n + 31) / 32 * 32) {                                 // (whole warps)
        const uint32_t same = __match_any_sync(0xffffffffu, e.id);
        bool bad = e.id < -1 || e.id >= a.V || !(e.lp < INFINITY) || (same & ((1u << (tid & 31)) - 1u)) != 0;
        const int4* before = reinterpret_cast<const int4*>(ids);
        for (int j = 0; j < tid / 32 * 8; ++j) {
            const int4 four = before[j];
            bad |= four.x == e.id || four.y == e.id || four.z == e.id || four.w == e.id;
        }
        if (bad && e.id != -1) {
            e.id = -1;
            e.fault = SPECDEC_ST_BAD_TARGET;
        }
    }
    return e;
}

template <typename F> __device__ __forceinline__ F warp_sum(F x)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ float warp_max(float x)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

constexpr int kListWarps = SPECDEC_TOP_MAX / 32;   // the warps that hold entries

// 2^y to 2^-43 relative in some fifteen 64-bit operations (this part has few of them): y = k + f with k whole, v = f ln 2 / 8,
// exp(v) by its series (|v| < 0.044: from the fourth power on in fp32, whose 2^-24 is 2^-46 of the sum), squared three times.
__device__ __forceinline__ double exp2_64(double y)
{
    if (!(y > -1000.0)) return y != y ? y : 0.0;
    const double shifted = y + 0x1.8p52, k = shifted - 0x1.8p52;
    const double v = (y - k) * (kLn2 / 8.0), square = v * v;
    const float x = (float)v;
    const float series = fmaf(fmaf(fmaf(x, 1.f / 5040.f, 1.f / 720.f), x, 1.f / 120.f), x, 1.f / 24.f);
    double e = fma(fma(square, (double)series, fma(v, 1.0 / 6.0, 0.5)), square, v) + 1.0;
    e *= e;
    e *= e;
    e *= e;
    return e * __hiloint2double((1023 + (int)fmin(k, 1023.0)) << 20, 0);
}

// What the list asks for. A target is exp(lp - shift) * norm; where the list is renormalised, shift is its largest log-probability,
// so that a list of small ones keeps its shares.
struct Asked {
    float shift, norm, listed, rest;               // listed, rest: the masses of the targets and of what is left
};
struct ListPart {
    double sum;                                    // in 64 bits: the rest is what it leaves of one
    float shift;
};
constexpr double kLog2e = 1.4426950408889634073599;
__device__ __forceinline__ double target_64(const Entry& e, float shift) { return e.id >= 0 ? exp2_64(((double)e.lp - (double)shift) * kLog2e) : 0.0; }
__device__ __forceinline__ ListPart list_part(const Entry& e, int has_rest)       // a warp's
{
    float shift = 0.f;
    if (!has_rest) {
        shift = warp_max(e.id >= 0 ? e.lp : -INFINITY);
        if (shift == -INFINITY) shift = 0.f;
    }
    return ListPart{warp_sum(target_64(e, shift)), shift};
}
__device__ __forceinline__ Asked asked_of(const ListPart* parts, int n, int has_rest)
{
    Asked a = {0.f, 1.f, 0.f, 0.f};
    const int warps = (n + 31) / 32;
    if (has_rest) {
        double sum = 0.0;
        for (int i = 0; i < warps; ++i) sum += parts[i].sum;
        a.listed = (float)sum;
        a.rest = (float)fmax(0.0, 1.0 - sum);
        return a;
    }
    float shift = -INFINITY, sum = 0.f;
    for (int i = 0; i < warps; ++i)
        if (parts[i].sum > 0.0) shift = fmaxf(shift, parts[i].shift);
    for (int i = 0; i < warps; ++i)
        if (parts[i].sum > 0.0) sum += (float)parts[i].sum * expf(parts[i].shift - shift);
    if (sum > 0.f) {
        a.shift = shift;
        a.norm = 1.f / sum;
        a.listed = 1.f;
    }
    return a;
}
__device__ __forceinline__ float target_of(const Entry& e, const Asked& a) { return expf(e.lp - a.shift) * a.norm; }

// Store of a vector's elements, those inside the row.
template <typename T> __device__ __forceinline__ void store_vector(const Row<T>& row, T* to, bool aligned, int32_t v, const Raw<T, kPer<T>>& x)
{
    const int32_t at = row.first(v);
    if (aligned && row.whole(at)) {
        *reinterpret_cast<uint4*>(to + at) = *reinterpret_cast<const uint4*>(x.e);
    } else {
#pragma unroll
        for (int i = 0; i < kPer<T>; ++i)
            if (at + i >= 0 && at + i < row.V) to[at + i] = x.e[i];
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
__device__ __forceinline__ void put_32(uint32_t to, float x) { asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(x) : "memory"); }
__device__ __forceinline__ void put_64(uint32_t to, double x) { asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(to), "d"(x) : "memory"); }
__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

struct Shared {
    double peer_S[kMaxCluster];
    float peer_ref[kMaxCluster];
    float refs[kWarps], sums[kWarps];
    float top_ref[kListWarps], top_sum[kListWarps];
    ListPart list[kListWarps];
    Asked asked;
    double list_64[kListWarps][3];
    alignas(16) int32_t ids[SPECDEC_TOP_MAX];
};

template <typename T, bool kGrad> __global__ void __launch_bounds__(kThreads, 2) specdec_distill_kernel(const Args a)
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
            const Raw<T, kPer<T>> zero = {};
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
    // (but for the row's first and last vector, every vector lies inside it)
    const int32_t whole0 = row.lead ? 1 : 0, whole1 = (row.lead + a.V) / kPer<T>;
    auto fetch = [&](int32_t from, int32_t to) {
        const int32_t end = min(to, whole1);
        for (int32_t v = max(from, whole0) + tid; v < end; v += kThreads) async_copy_16(smem_u32(mine + (v - from)), z + row.first(v), 16);
        if (tid < 2) {
            const int32_t v = tid == 0 ? 0 : row.vectors - 1;
            if ((v < whole0 || v >= whole1) && v >= from && v < to) load_vector(row, v, mine[v - from]);
        }
    };
    fetch(v0, min(v0 + a.tile, v1));

    // the list: targets, and the student's logits there, which every CTA of the cluster reads before any of them writes
    const Entry e = read_entry(a, r, s.ids);
    float top = e.id >= 0 ? to_float<T>(z[e.id]) : -INFINITY;
    if (warp < kListWarps) {
        float ref = ceilf(top * a.scale);
        if (ref == -INFINITY) top = -INFINITY;                        // (the lowest numbers, where masks put them)
        ref = warp_max(ref);
        const float sum = warp_sum(top == -INFINITY ? 0.f : exp2_fast(exponent(top, a, ref)));
        const ListPart part = list_part(e, a.rest);
        if (lane == 0) {
            s.top_ref[warp] = ref;
            s.top_sum[warp] = sum;
            s.list[warp] = part;
        }
    }

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
            const float m = Maximum<T>::of(x).value();
            if (m * a.scale > ref) {
                const float up = ceilf(m * a.scale);
                S *= reference_step(ref, up);
                ref = up;
            }
            const Exponentials<true> e2(a, ref == -INFINITY ? 0.f : ref);
            Pair part = e2(elements(x, 0));
#pragma unroll
            for (int i = 1; i < kPer<T> / 2; ++i) part = add_2(part, e2(elements(x, i)));
            S += both(part).x + both(part).y;
        }
    }
    warp_join(ref, S);
    if (lane == 0) {
        s.refs[warp] = ref;
        s.sums[warp] = S;
    }
    __syncthreads();
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    if (warp == 0) {
        const Asked asked = asked_of(s.list, a.n, a.rest);
        if (lane == 0) s.asked = asked;
        // every CTA gets every CTA's sum: lane i writes into CTA i
        const float one = s.refs[lane % kWarps], all = warp_max(one);
        double sum = (double)s.sums[lane % kWarps] * reference_step_64(one, all);
#pragma unroll
        for (int o = kWarps / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane < (int)size) {
            put_64(in_cta(&s.peer_S[rank], lane), sum);
            put_32(in_cta(&s.peer_ref[rank], lane), all);
        }
    }
    cluster_barrier();

    float rest_ref = -INFINITY, top_ref = -INFINITY, S_rest = 0.f, S_top = 0.f;
    for (uint32_t i = 0; i < size; ++i) rest_ref = fmaxf(rest_ref, s.peer_ref[i]);
    for (uint32_t i = 0; i < size; ++i) S_rest += (float)s.peer_S[i] * reference_step(s.peer_ref[i], rest_ref);
#pragma unroll
    for (int i = 0; i < kListWarps; ++i) top_ref = fmaxf(top_ref, s.top_ref[i]);
#pragma unroll
    for (int i = 0; i < kListWarps; ++i) S_top += s.top_sum[i] * reference_step(s.top_ref[i], top_ref);
    const Asked asked = s.asked;
    const bool asks = asked.listed + asked.rest > 0.f;                // (an empty list that leaves nothing asks for nothing)
    const float all_ref = fmaxf(rest_ref, top_ref);
    const float S_rest_all = S_rest * reference_step(rest_ref, all_ref), S_top_all = S_top * reference_step(top_ref, all_ref);
    const float S_all = S_rest_all + S_top_all;
    const bool none = all_ref == -INFINITY && !(S_all != S_all);      // no finite logit
    // Where the student leaves nothing to the rest there is no such category.
    const bool tail = !(S_rest == 0.f);
    const float left = tail ? asked.rest : 0.f;

    if constexpr (kGrad) {
        // outside the list: e_j (M / S - r / S_rest), which is (S_rest sum t - r S_top) / (S S_rest) without the cancellation of M and r
        const float each = none || !asks ? 0.f : w * a.inverse, mass = asked.listed + left, per_all = none ? 0.f : mass / S_all;
        const float base = rest_ref == -INFINITY ? 0.f : rest_ref;
        const float factor = tail ? ((asked.listed * S_rest_all - left * S_top_all) / S_all) / S_rest * each : 0.f;
        const Exponentials<sizeof(T) == 4> e2(a, base);
        const Pair factors = pair_of(factor, factor);
        for (int32_t from = v0; from < v1; from += a.tile) {
            const int32_t to = min(from + a.tile, v1);
            if (a.tile < a.slice) {
                __syncthreads();
                fetch(from, to);
                async_copy_wait();
                __syncthreads();
            }
            auto change = [&](int32_t v) {
                Raw<T, kPer<T>> x = mine[v - from];
#pragma unroll
                for (int i = 0; i < kPer<T> / 2; ++i) put_elements(x, i, mul_2(e2(elements(x, i)), factors));
                return x;
            };
            if (aligned) {
                const int32_t end = min(to, whole1);
                for (int32_t v = max(from, whole0) + tid; v < end; v += kThreads) {
                    const Raw<T, kPer<T>> x = change(v);
                    *reinterpret_cast<uint4*>(g + row.first(v)) = *reinterpret_cast<const uint4*>(x.e);
                }
                if (tid < 2) {
                    const int32_t v = tid == 0 ? 0 : row.vectors - 1;
                    if ((v < whole0 || v >= whole1) && v >= from && v < to) store_vector(row, g, false, v, change(v));
                }
            } else {
                for (int32_t v = from + tid; v < to; v += kThreads) store_vector(row, g, false, v, change(v));
            }
        }
        __syncthreads();
        if (e.id >= 0 && e.id >= row.first(v0) && e.id < row.first(v1)) {
            const float share = top == -INFINITY ? 0.f : exp2_fast(exponent(top, a, all_ref)) * per_all;
            g[e.id] = from_float<T>((share - target_of(e, asked)) * each);
        }
    }
    if (rank != 0) return;

    // The loss in 64 bits: near zero it is a small difference of logarithms.
    if (a.status && (e.fault || (tid == 0 && none))) atomicOr(a.status + r, e.fault | (tid == 0 && none ? SPECDEC_ST_EMPTY_MASK_ROW : 0u));
    if (warp < kListWarps) {
        const double up = top == -INFINITY ? -INFINITY : (double)top * ((double)a.scale + (double)a.scale_low) - (double)top_ref;
        const double t = target_64(e, asked.shift), sum = warp_sum(t), listed = warp_sum(exp2_64(up)), cross = warp_sum(t > 0.0 ? t * ((double)e.lp - up * kLn2) : 0.0);
        if (lane == 0) {
            s.list_64[warp][0] = sum;
            s.list_64[warp][1] = listed;
            s.list_64[warp][2] = cross;
        }
    }
    __syncthreads();
    if (tid == 0) {
        double sum = 0.0, listed = 0.0, cross = 0.0, others = 0.0;
        for (int i = 0; i < kListWarps; ++i) {
            sum += s.list_64[i][0];
            listed += s.list_64[i][1];
            cross += s.list_64[i][2];
        }
        for (uint32_t i = 0; i < size; ++i) others += s.peer_S[i] * reference_step_64(s.peer_ref[i], rest_ref);
        const double log_all = log(others * reference_step_64(rest_ref, all_ref) + listed * reference_step_64(top_ref, all_ref)) + (double)all_ref * kLn2;
        const double log_rest = log(others) + (double)rest_ref * kLn2;
        double loss = 0.0;
        if (none) {
            loss = asks ? INFINITY : 0.0;
        } else if (asks) {
            const double r_64 = a.rest && tail ? fmax(0.0, 1.0 - sum) : 0.0;
            if (sum > 0.0) {
                // sum of t_i (ln t_i - ln s_i) where t_i = exp(lp_i), and where they are renormalised
                loss = cross + sum * (log_all - (double)top_ref * kLn2);
                if (!a.rest) loss = loss / sum - log(sum) - (double)asked.shift;
            }
            if (r_64 > 0.0) loss += r_64 * (log(r_64) - (log_rest - log_all));
        }
        a.loss[r] = (float)((double)w * loss);
        if (a.stats) {
            a.stats[2 * r] = (float)log_all;
            a.stats[2 * r + 1] = (float)log_rest;
        }
    }
}

// log2(e) x = whole - less, whole a whole number (x's, rounded up) and 0 <= less <= 1 without the product's rounding.
__device__ __forceinline__ void in_octaves(float x, float* whole, float* less)
{
    constexpr float kHigh = 1.44269504f, kLow = (float)(1.4426950408889634073599 - (double)kHigh);
    const float p = x * kHigh;
    *whole = ceilf(p);
    *less = (*whole - p) - fmaf(x, kHigh, -p) - x * kLow;
}

// The gradient from the sums that a forward pass kept: element by element, a CTA a chunk of a row. All in fp32: the sums come in fp32.
constexpr int kChunk = 8;                          // vectors a thread

template <typename T> __global__ void __launch_bounds__(kBackThreads) specdec_distill_backward_kernel(const Args a, const int32_t chunks)
{
    __shared__ ListPart parts[kListWarps];
    __shared__ __align__(16) int32_t ids[SPECDEC_TOP_MAX];
    after_predecessor();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t r = blockIdx.x / (uint32_t)chunks;
    const int32_t v0 = (int32_t)(blockIdx.x - r * chunks) * (kChunk * kBackThreads);
    const T* const z = static_cast<const T*>(a.logits) + r * a.row_stride;
    T* const g = static_cast<T*>(a.grad) + r * a.grad_stride;
    const Row<T> row(z, a.V);
    if (v0 >= row.vectors) return;
    const bool aligned = same_grid(z, g);
    const float w = a.weight ? a.weight[r] : 1.f;
    if (w == 0.f) {
        const Raw<T, kPer<T>> zero = {};
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
            if (v0 + i * kBackThreads + tid < row.vectors) store_vector(row, g, aligned, v0 + i * kBackThreads + tid, zero);
        return;
    }
    Raw<T, kPer<T>> x[kChunk];
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
        const int32_t v = v0 + i * kBackThreads + tid, at = row.first(v);
        if (v < row.vectors && row.whole(at)) {
            *reinterpret_cast<uint4*>(x[i].e) = *reinterpret_cast<const uint4*>(z + at);
        } else {
#pragma unroll
            for (int k = 0; k < kPer<T>; ++k) x[i].e[k] = at + k >= 0 && at + k < a.V ? z[at + k] : neg_inf<T>();
        }
    }
    const float lse = a.stats[2 * r], lse_rest = a.stats[2 * r + 1];
    const Entry e = read_entry(a, r, ids);
    const bool here = e.id >= 0 && e.id >= row.first(v0) && e.id < row.first(min(v0 + kChunk * kBackThreads, row.vectors));
    const float top = here ? to_float<T>(z[e.id]) : 0.f;              // (before the row is written: the gradient may lie over it)
    if (warp < kListWarps) {
        const ListPart part = list_part(e, a.rest);
        if (lane == 0) parts[warp] = part;
    }
    __syncthreads();
    const Asked asked = asked_of(parts, a.n, a.rest);
    // the exponentials of this kernel are taken at the rest's sum; where there is none, no element is outside the list
    const bool tail = !(lse_rest == -INFINITY), none = lse == -INFINITY || !(asked.listed + asked.rest > 0.f);
    const float left = tail ? asked.rest : 0.f, each = none ? 0.f : w * a.inverse;
    float all, all_less, ref, ref_less;
    in_octaves(none ? 0.f : lse, &all, &all_less);
    in_octaves(tail ? lse_rest : 0.f, &ref, &ref_less);
    const float factor = tail ? ((asked.listed + left) * exp2f(ref - all + all_less) - left * exp2f(ref_less)) * each : 0.f;
    const Exponentials<sizeof(T) == 4> e2(a, ref);
    const Pair factors = pair_of(factor, factor);
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
        const int32_t v = v0 + i * kBackThreads + tid;
        if (v >= row.vectors) continue;
#pragma unroll
        for (int k = 0; k < kPer<T> / 2; ++k) put_elements(x[i], k, mul_2(e2(elements(x[i], k)), factors));
        store_vector(row, g, aligned, v, x[i]);
    }
    __syncthreads();
    if (here) {
        const float share = exp2f(exponent(top, a, all) + all_less) * (asked.listed + left);
        g[e.id] = from_float<T>((share - target_of(e, asked)) * each);
    }
    if (v0 == 0 && a.status && e.fault) atomicOr(a.status + r, e.fault);
}

// ---------------------------------------------------------------- host

struct Shape {
    int32_t cluster, slice, tile;
};

// A row goes to the fewest CTAs that keep two of them on an SM, more where the rows alone do not
// fill the GPU; what is longer than eight times kTileBytes is read a second time for the gradient.
template <typename T> Shape shape_of(int32_t rows, int32_t V)
{
    const int32_t vectors = most_vectors<T>(V);
    int32_t cluster = 1;
    auto slice = [&] { return (vectors + cluster - 1) / cluster; };
    while (cluster < kMaxCluster && (slice() > kTileBytes / 16 || ((int64_t)rows * cluster < 304 && slice() > 8 * 1024 / 16))) cluster *= 2;
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
    const int32_t chunks = (most_vectors<T>(a.V) + kChunk * kBackThreads - 1) / (kChunk * kBackThreads);
    if ((int64_t)a.rows * chunks > 0x7fffffff) return SPECDEC_ERR_UNSUPPORTED;
    const cudaError_t e = launch_dependent(specdec_distill_backward_kernel<T>, (unsigned)((int64_t)a.rows * chunks), kBackThreads, 0, stream, a, chunks);
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
    // (the first rounded towards zero and the second at least a little above it: the kernels rely on their signs)
    const double c = scale_of(temperature);
    const float high = std::nextafterf((float)c, 0.f), low = std::fmax((float)(c - (double)high), 1e-30f);
    return Args{logits, row_stride, V, rows, top_ids, top_logprobs, n, high, low, (float)(1.0 / temperature), rest,
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
