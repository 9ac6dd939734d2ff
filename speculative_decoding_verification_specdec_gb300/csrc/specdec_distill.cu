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
 * A row is held by a cluster of CTAs, a part each, in shared memory: it is read from HBM once, for the sums and for the gradient.
 * Measured on one GB300: 2048 rows of 151936 bf16 logits against 64 ids, loss and gradient, 270 us, 68 % of what reading and
 * writing them once takes at the copy rate (a forward and a backward pass of their own: 157 + 185). Its bound is a row's chain of
 * barriers, which the other CTAs of an SM fill. The backward kernel goes element by element: 700 rows of 128256 fp32 logits in 107.5 us, 98 %.
 */
#include <atomic>
#include <cmath>
#include <cstddef>

#include "specdec_logits.cuh"

namespace {

using namespace specdec;

constexpr int kRowWarps = 8;                       // of a CTA, at most, that hold its part of a row
constexpr int kLaneVectors = 20;                   // of a thread, where that many warps are enough
constexpr int kBackThreads = 256;
constexpr int kMaxCluster = 16;
constexpr int kSliceBytes = 70 * 1024;             // of a row in a CTA: three CTAs an SM
constexpr int kSmallBytes = 44 * 1024;             // five of them, of four warps
constexpr int kMostBytes = 200 * 1024;             // and where sixteen CTAs hold the row only so

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
    int32_t slice;                                 // vectors of a row in a CTA
};

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

__device__ __forceinline__ float warp_max(float x)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

constexpr int kEntries = SPECDEC_TOP_MAX / 32;     // of a lane of the warp that holds the list
constexpr float kMostLogProbability = 0.5f;        // where the list is not renormalised: rounding may bring one above 0, not so far

// The list as one warp holds it: entry lane + 32 c in a lane's c-th place.
struct List {
    int32_t ids[kEntries];
    float lps[kEntries];
    __device__ __forceinline__ void read(const Args& a, int64_t r)
    {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int c = 0; c < kEntries; ++c) {
            const int j = lane + 32 * c;
            ids[c] = j < a.n ? a.ids[r * a.n + j] : -1;
            lps[c] = j < a.n ? a.logprobs[r * a.n + j] : -INFINITY;
        }
    }
};

// An entry that lies in one part of a row.
struct Own {
    int32_t id;
    float lp, top;                                 // top: the student's logit
};
// The entries that lie in elements begin .. end - 1, side by side in own, but for those that do not count: a repeated id (which lies
// in the same part as its first listing), or no log-probability. One warp; returns how many, and the status bits of this lane's
// entries (ids outside the vocabulary lie in no part: they count for the first).
__device__ __forceinline__ int own_entries(const Args& a, const List& list, int32_t begin, int32_t end, Own* own, uint32_t* fault)
{
    const int lane = threadIdx.x & 31;
    const uint32_t below = (1u << lane) - 1u;
    int found = 0;
    *fault = 0;
#pragma unroll
    for (int c = 0; c < kEntries; ++c) {
        if (32 * c >= a.n) continue;
        const int32_t id = list.ids[c];
        if ((id < -1 || id >= a.V) && begin <= 0) *fault = SPECDEC_ST_BAD_TARGET;
        const bool here = id >= max(begin, 0) && id < min(end, a.V);
        const uint32_t all = __ballot_sync(0xffffffffu, here);
        if (here) own[found + __popc(all & below)] = Own{id, list.lps[c], 0.f};
        found += __popc(all);
    }
    __syncwarp();
    // (from the last 32 to the first, so that those before are still as they were listed)
    for (int j0 = (found - 1) / 32 * 32; found > 0 && j0 >= 0; j0 -= 32) {
        const int j = j0 + lane;
        const Own o = own[j < found ? j : 0];
        bool counts = (__match_any_sync(0xffffffffu, j < found ? o.id : -2 - lane) & below) == 0 &&
                      o.lp <= (a.rest ? kMostLogProbability : 3.402823466e38f);
        for (int k = 0; k < j0; ++k) counts &= own[k].id != o.id;
        if (j < found && !counts) {
            own[j].top = 1.f;                      // marked
            *fault = SPECDEC_ST_BAD_TARGET;
        }
    }
    if (!__any_sync(0xffffffffu, *fault)) return found;
    int kept = 0;
    for (int j0 = 0; j0 < found; j0 += 32) {
        const int j = j0 + lane;
        const Own o = own[j < found ? j : 0];
        const bool counts = j < found && o.top == 0.f;
        const uint32_t all = __ballot_sync(0xffffffffu, counts);
        __syncwarp();
        if (counts) own[kept + __popc(all & below)] = o;              // (never behind where it is read)
        kept += __popc(all);
        __syncwarp();
    }
    return kept;
}

// exp(lp - shift), a target (0 from 2^-125 down, -infinity among it).
__device__ __forceinline__ Two target_of(float lp, float shift)
{
    return lp - shift < -90.f ? Two{0.f, 0.f} : exp2_two(two_sum(lp, -shift) * SPECDEC_TWO(kLog2e));
}
// Targets add up as whole numbers of 2^-54, so that what they leave of one is exact (128 of exp(0.5) stay below 2^63 of them).
constexpr float kFixed = 0x1p54f;
__device__ __forceinline__ long long fixed_of(Two x) { return __float2ll_rn(x.hi * kFixed) + __float2ll_rn(x.lo * kFixed); }
__device__ __forceinline__ float from_fixed(long long x) { return __ll2float_rn(x) * (1.f / kFixed); }

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
__device__ __forceinline__ void put_64(uint32_t to, long long x) { asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(to), "l"(x) : "memory"); }
// (A thread that has written nothing for others: a release would wait for its own copies and stores in flight.)
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// ---------------------------------------------------------------- forward

// Persistent clusters, row after row. All warps of a CTA but two hold its part of the row in shared memory, each thread its own
// vectors, and fetch the next row's into their places as they finish with them. One warp holds the list: it takes the listed
// elements out of the row, sums their part and exchanges the CTAs' sums. Another works the loss out while the others go on. What
// a CTA knows of a row meets the others' by distributed shared memory and one cluster barrier a row.

// What one CTA of a cluster knows of a row.
struct Part {
    long long fixed;                               // the sum of the targets in 2^-54 (rest = 1)
    Two rest, top, targets, cross;                 // sums of exponentials outside and on the list; of the targets (rest = 0); of t (ln t - z / temperature)
    float rest_ref, top_ref, shift;
    int32_t endless;                               // whether a target lies where the student has -infinity
    long long unused;
};
constexpr int kPartWords = sizeof(Part) / 8;
static_assert(kPartWords == 8, "a power of two");
struct Shared {
    Part peer[2][kMaxCluster];                     // two rows': a CTA may be one ahead
    Part part;
    float refs[kRowWarps], sums[kRowWarps];
    float factor, base;                            // of the gradient outside the list: e_j relative to base, times factor
    Own own[2][SPECDEC_TOP_MAX];                   // of this row and of the one before, or after
};

// The parts of all CTAs together: the lanes of each half of a warp hold one each.
__device__ __forceinline__ float half_max(float x)
{
#pragma unroll
    for (int o = kMaxCluster / 2; o >= 1; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
template <typename F> __device__ __forceinline__ F half_sum(F x)
{
#pragma unroll
    for (int o = kMaxCluster / 2; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ Two half_sum(Two x)
{
#pragma unroll
    for (int o = kMaxCluster / 2; o >= 1; o >>= 1) x = x + shuffle_xor(x, o);
    return x;
}

// All CTAs' parts together, by one warp.
struct Total {
    float rest_ref, all_ref, S_rest, S_rest_all, S_top_all, S_all, listed, left;      // listed, left: the masses of the targets and of the rest
    bool none, asks, tail;                         // no finite logit; whether anything is asked for; whether there is a rest
    __device__ __forceinline__ Total(const Args& a, const Part* peer, uint32_t size)
    {
        const int i = threadIdx.x % kMaxCluster;
        const bool there = i < (int)size;
        const Part& one = peer[there ? i : 0];
        const float one_rest = there ? one.rest_ref : -INFINITY, one_top = there ? one.top_ref : -INFINITY;
        rest_ref = half_max(one_rest);
        all_ref = fmaxf(rest_ref, half_max(one_top));
        S_rest = half_sum(there ? one.rest.hi * reference_step(one_rest, rest_ref) : 0.f);
        S_top_all = half_sum(there ? one.top.hi * reference_step(one_top, all_ref) : 0.f);
        S_rest_all = S_rest * reference_step(rest_ref, all_ref);
        S_all = S_rest_all + S_top_all;
        tail = !(S_rest == 0.f);                   // (where the student leaves nothing to the rest there is no such category)
        left = 0.f;
        if (a.rest) {
            const long long fixed = half_sum(there ? one.fixed : 0ll), unit = (long long)kFixed;
            listed = from_fixed(fixed);
            if (fixed < unit) left = from_fixed(unit - fixed);
        } else {
            listed = half_max(there && one.targets.hi > 0.f ? 1.f : 0.f);
        }
        asks = listed + left > 0.f;
        if (!tail) left = 0.f;
        none = all_ref == -INFINITY && !(S_all != S_all);
    }
    // The largest log-probability of a list that is renormalised, and one over the sum of exp(lp - shift).
    __device__ __forceinline__ float shift(const Args& a, const Part* peer, uint32_t size) const
    {
        if (a.rest || !asks) return 0.f;
        const int i = threadIdx.x % kMaxCluster;
        return half_max(i < (int)size && peer[i].targets.hi > 0.f ? peer[i].shift : -INFINITY);
    }
    __device__ __forceinline__ float norm(const Args& a, const Part* peer, uint32_t size, float shift) const
    {
        if (a.rest || !asks) return 1.f;
        const int i = threadIdx.x % kMaxCluster;
        return 1.f / half_sum(i < (int)size && peer[i].targets.hi > 0.f ? peer[i].targets.hi * expf(peer[i].shift - shift) : 0.f);
    }
};

// A CTA's part of a row: vectors begin .. begin + count - 1, of which those from number `whole` on, `wholes` of them, lie in it as a whole.
template <typename T> struct Slice {
    Row<T> row;
    int32_t begin, count, whole, wholes;
    __device__ __forceinline__ Slice(const Args& a, int64_t r, int32_t rank)
        : row(static_cast<const T*>(a.logits) + r * a.row_stride, a.V)
    {
        begin = min(rank * a.slice, row.vectors);
        count = min(begin + a.slice, row.vectors) - begin;
        whole = max(row.lead ? 1 : 0, begin) - begin;
        wholes = max(min((row.lead + a.V) / kPer<T>, begin + count) - begin - whole, 0);
    }
    __device__ __forceinline__ bool is_whole(int32_t i) const { return (uint32_t)(i - whole) < (uint32_t)wholes; }
    __device__ __forceinline__ const T* at(int32_t i) const { return row.p + row.first(begin + i); }
};

template <typename T, bool kGrad> __global__ void __launch_bounds__((kRowWarps + 2) * 32, 3) specdec_distill_kernel(const Args a)
{
    extern __shared__ __align__(16) unsigned char held[];
    __shared__ Shared s;
    after_predecessor();
    constexpr int kPairs = kPer<T> / 2;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x - 64;
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int64_t clusters = gridDim.x / size;
    auto weight_of = [&](int64_t r) { return a.weight ? a.weight[r] : 1.f; };
    const int64_t first = blockIdx.x / size;       // the cluster's rows: from this one on, `clusters` apart
    // Every thread goes through every row's barriers, whether the row has a weight or not, so that no weight that changes under
    // the call can part them; it arrives at the cluster's barrier once at the start and once a row, and waits for each phase.
    auto meet = [&] { barrier_sync(1, threads + 32); };               // the row's warps and the list's

    if (tid < threads) {
        // ---- the warps that hold the row
        Raw<T, kPer<T>>* const mine = reinterpret_cast<Raw<T, kPer<T>>*>(held) + tid;
        const uint32_t mine_at = smem_u32(mine);
        bool live = weight_of(first) != 0.f;
        if (live) {
            const Slice<T> now(a, first, rank);
            for (int32_t i = tid; i < now.count; i += threads)
                if (now.is_whole(i)) async_copy_16(mine_at + (i - tid) * 16, now.at(i), 16);
        }
        cluster_arrive_relaxed();                                     // (no CTA writes to one that has not started)
        for (int64_t r = first; r < a.rows; r += clusters) {
            const Slice<T> now(a, r, rank);
            const int64_t after = min(r + clusters, (int64_t)a.rows - 1);
            const bool next_live = r + clusters < a.rows && weight_of(after) != 0.f;
            async_copy_wait();
            meet();                                                   // A: the row has landed; the list's warp takes the listed out
            meet();                                                   // B
            const Slice<T> next(a, after, rank);
            const int32_t count = live ? now.count : 0, coming = next_live ? next.count : 0;
            const char* const source = reinterpret_cast<const char*>(next.at(0));
            auto fetch = [&](int32_t i) {                             // vector i of the next row into the place that this thread is done with
                if (next.is_whole(i)) async_copy_16(mine_at + (i - tid) * 16, source + (int64_t)i * 16, 16);
            };
            float ref = -INFINITY;
            Pair sum = pair_of(0.f, 0.f);
            auto fold = [&](const Raw<T, kPer<T>>& x, const Exponentials<true>& e2) {
                Pair some = e2(elements(x, 0));
#pragma unroll
                for (int k = 1; k < kPairs; ++k) some = add_2(some, e2(elements(x, k)));
                sum = add_2(sum, some);
            };
            auto raise = [&](float m) {
                m *= a.scale;
                if (m > ref) {
                    const float up = ceilf(m), step = reference_step(ref, up);
                    sum = mul_2(sum, pair_of(step, step));
                    ref = up;
                }
            };
            int32_t i = tid;
            for (; i + threads < count; i += 2 * threads) {
                const Raw<T, kPer<T>> x = mine[i - tid], y = mine[i - tid + threads];
                raise(larger(Maximum<T>::of(x), Maximum<T>::of(y)).value());
                const Exponentials<true> e2(a, ref == -INFINITY ? 0.f : ref);
                fold(x, e2);
                fold(y, e2);
                if (!kGrad) {
                    if (i < coming) fetch(i);
                    if (i + threads < coming) fetch(i + threads);
                }
            }
            if (i < count) {
                const Raw<T, kPer<T>> x = mine[i - tid];
                raise(Maximum<T>::of(x).value());
                fold(x, Exponentials<true>(a, ref == -INFINITY ? 0.f : ref));
            }
            // (a row off the 16-byte grid may have one vector more or less than the next)
            if (!kGrad)
                for (; i < coming; i += threads) fetch(i);
            float S = both(sum).x + both(sum).y;
            warp_join(ref, S);
            if (lane == 0) {
                s.refs[warp] = ref;
                s.sums[warp] = S;
            }
            meet();                                                   // D: the sums are there
            cluster_wait();                                           // (the phase before: the list's warp has waited for it)
            cluster_arrive_relaxed();
            if constexpr (kGrad) {
                T* const g = static_cast<T*>(a.grad) + r * a.grad_stride;
                const bool aligned = same_grid(now.row.p, g);
                T* const to = g + now.row.first(now.begin);
                meet();                                               // E: the factor is there
                const Exponentials<sizeof(T) == 4> e2(a, s.base);
                const Pair factors = pair_of(s.factor, s.factor);
                for (i = tid; i < now.count; i += threads) {
                    Raw<T, kPer<T>> x = {};
                    if (live) {
                        x = mine[i - tid];
#pragma unroll
                        for (int k = 0; k < kPairs; ++k) put_elements(x, k, mul_2(e2(elements(x, k)), factors));
                    }
                    if (i < coming) fetch(i);
                    if (aligned && now.is_whole(i)) *reinterpret_cast<uint4*>(to + (int64_t)i * kPer<T>) = *reinterpret_cast<const uint4*>(x.e);
                    else store_vector(now.row, g, false, now.begin + i, x);
                }
                for (; i < coming; i += threads) fetch(i);
            }
            live = next_live;
        }
        if (kGrad) meet();                                            // F: the row is written, the listed may go over it
        cluster_wait();
        return;
    }

    if (tid < threads + 32) {
        // ---- the list's warp
        List list;
        list.read(a, first);
        // The row's ends, where a vector lies partly outside it: an element a lane, the first vector's and the last one's.
        T end_element;
        auto read_ends = [&](const Slice<T>& z) {
            const int32_t v = lane < kPer<T> ? 0 : z.row.vectors - 1, at = z.row.first(v) + lane % kPer<T>;
            end_element = lane < 2 * kPer<T> && at >= 0 && at < a.V ? z.row.p[at] : neg_inf<T>();
        };
        auto put_ends = [&](const Slice<T>& z) {
            const int32_t i = (lane < kPer<T> ? 0 : z.row.vectors - 1) - z.begin;
            if (lane < 2 * kPer<T> && i >= 0 && i < z.count && !z.is_whole(i)) reinterpret_cast<T*>(held)[i * kPer<T> + lane % kPer<T>] = end_element;
        };
        // the entries of a row that lie here; none of a row without a weight
        auto own_of = [&](int64_t row, float w, Own* own) {
            if (w == 0.f) return 0;
            const Slice<T> z(a, row, rank);
            read_ends(z);
            uint32_t fault;
            const int n = own_entries(a, list, z.row.first(z.begin), z.row.first(z.begin + z.count), own, &fault);
            if (a.status && fault) atomicOr(a.status + row, fault);
            return n;
        };
        float w = weight_of(first);
        int owned = own_of(first, w, s.own[0]), late_count = 0;
        T* late = nullptr;                                            // where the listed elements' gradients go once all others are written
        auto write_late = [&](const Own* own) {
            for (int j = lane; j < late_count; j += 32) late[own[j].id] = from_float<T>(own[j].top);
            __syncwarp();
        };
        cluster_arrive();
        cluster_wait();                                               // (every CTA has started)
        int turn = 0;
        for (int64_t r = first; r < a.rows; r += clusters, turn ^= 1) {
            Own* const own = s.own[turn];
            const Slice<T> now(a, r, rank);
            meet();                                                   // A
            const int32_t begin = now.row.first(now.begin);
            if (w != 0.f) put_ends(now);
            __syncwarp();
            for (int j = lane; j < owned; j += 32) {
                T* const e = reinterpret_cast<T*>(held) + (own[j].id - begin);
                const float top = to_float<T>(*e);
                own[j].top = top * a.scale == -INFINITY ? -INFINITY : top;    // (the lowest numbers, where masks put them)
                *e = neg_inf<T>();
            }
            meet();                                                   // B
            if (kGrad) write_late(s.own[turn ^ 1]);
            const int64_t after = r + clusters;
            float next_w = 0.f;
            if (after < a.rows) {                                     // (read well before they are asked)
                next_w = weight_of(after);
                list.read(a, after);
            }
            Part part = {0, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, -INFINITY, -INFINITY, a.rest ? 0.f : -INFINITY, 0, 0};
            if (owned) {
                for (int j = lane; j < owned; j += 32) {
                    part.top_ref = fmaxf(part.top_ref, ceilf(own[j].top * a.scale));
                    if (!a.rest) part.shift = fmaxf(part.shift, own[j].lp);
                }
                part.top_ref = warp_max(part.top_ref);
                if (!a.rest) part.shift = warp_max(part.shift);
                const float base = part.top_ref == -INFINITY ? 0.f : part.top_ref, origin = part.shift == -INFINITY ? 0.f : part.shift;
                for (int j0 = 0; j0 < owned; j0 += 32) {
                    const bool in = j0 + lane < owned;
                    const Own o = own[in ? j0 + lane : 0];
                    const bool number = o.top > -INFINITY || o.top != o.top;
                    // z log2(e) / temperature
                    const Two up = two_product(o.top, a.scale) + Two{o.top * a.scale_low, 0.f};
                    const Two target = target_of(o.lp, origin);
                    if (in && number) part.top = part.top + exp2_two(up + Two{-base, 0.f});
                    if (in) {
                        if (a.rest) part.fixed += fixed_of(target);
                        else part.targets = part.targets + target;
                        if (target.hi > 0.f && number) part.cross = part.cross + target * (Two{o.lp, 0.f} - up * SPECDEC_TWO(kLn2));
                        else if (target.hi > 0.f) part.endless = 1;
                    }
                }
                part.top = warp_sum(part.top);
                part.cross = warp_sum(part.cross);
                part.endless = __any_sync(0xffffffffu, part.endless);
                if (a.rest)
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) part.fixed += __shfl_xor_sync(0xffffffffu, part.fixed, o);
                else part.targets = warp_sum(part.targets);
            }
            if (!kGrad && r != first) cluster_wait();                 // (the phase before)
            if (lane == 0) s.part = part;
            meet();                                                   // D
            {
                const bool holds = lane < threads / 32;
                const float one = holds ? s.refs[lane] : -INFINITY, rest_ref = half_max(one);      // (of the lower half)
                const Two rest = half_sum(Two{holds ? s.sums[lane] * reference_step(one, rest_ref) : 0.f, 0.f});
                if (lane == 0) {
                    s.part.rest_ref = rest_ref;
                    s.part.rest = rest;
                }
            }
            __syncwarp();
            // to every CTA, eight bytes a lane at a time
            for (int i = lane; i < kPartWords * (int)size; i += 32)
                put_64(in_cta(&s.peer[turn][rank], i / kPartWords) + i % kPartWords * 8, reinterpret_cast<const long long*>(&s.part)[i % kPartWords]);
            cluster_arrive();
            if constexpr (kGrad) {
                cluster_wait();
                const Total all(a, s.peer[turn], size);
                const float each = all.none || !all.asks ? 0.f : w * a.inverse;
                // outside the list: e_j (M / S - r / S_rest), which is (S_rest sum t - r S_top) / (S S_rest) without the cancellation of M and r
                if (lane == 0) {
                    s.factor = all.tail ? ((all.listed * all.S_rest_all - all.left * all.S_top_all) / all.S_all) / all.S_rest * each : 0.f;
                    s.base = all.rest_ref == -INFINITY ? 0.f : all.rest_ref;
                }
                meet();                                               // E
                const float shift = all.shift(a, s.peer[turn], size), norm = all.norm(a, s.peer[turn], size, shift);
                const float per_all = all.none ? 0.f : (all.listed + all.left) / all.S_all;
                late = static_cast<T*>(a.grad) + r * a.grad_stride;
                late_count = owned;
                for (int j = lane; j < owned; j += 32) {
                    const Own o = own[j];
                    const float share = o.top == -INFINITY ? 0.f : exp2_fast(exponent(o.top, a, all.all_ref)) * per_all;
                    own[j].top = (share - expf(o.lp - shift) * norm) * each;
                }
            }
            if (after < a.rows) owned = own_of(after, next_w, s.own[turn ^ 1]);
            w = next_w;
        }
        if constexpr (kGrad) {
            meet();                                                   // F
            write_late(s.own[turn ^ 1]);
        } else {
            cluster_wait();
        }
        return;
    }

    // ---- the loss's warp
    cluster_arrive_relaxed();
    cluster_wait();
    cluster_arrive_relaxed();
    int turn = 0;
    for (int64_t r = first; r < a.rows; r += clusters, turn ^= 1) {
        const float w = weight_of(r);
        cluster_wait();
        const bool there = lane % kMaxCluster < (int)size;
        const Part one = s.peer[turn][there ? lane % kMaxCluster : 0];
        const Total all(a, s.peer[turn], size);
        const float shift = all.shift(a, s.peer[turn], size);
        if (r + clusters < a.rows) cluster_arrive_relaxed();          // (nothing of the row is read behind this)
        if (rank == 0 && w == 0.f) {
            if (lane == 0) a.loss[r] = 0.f;
            if (lane < 2 && a.stats) a.stats[2 * r + lane] = 0.f;
        } else if (rank == 0) {
            // The loss in pairs of floats: near zero it is a small difference of logarithms.
            const Two zero = {0.f, 0.f};
            const bool some = there && (a.rest ? one.fixed > 0 : one.targets.hi > 0.f);
            const long long whole = (long long)(one.fixed >> 32) << 32;       // (its upper half is exact in fp32)
            const Two given = a.rest ? two_sum(from_fixed(whole), from_fixed(one.fixed - whole)) : one.targets;
            const Two rest = half_sum(there ? times(one.rest, reference_step(one.rest_ref, all.rest_ref)) : zero);
            const Two top = half_sum(there ? times(one.top, reference_step(one.top_ref, all.all_ref)) : zero);
            const Two by = !some ? zero : a.rest ? Two{1.f, 0.f} : target_of(one.shift, shift);
            const Two sum = half_sum(some ? given * by : zero), cross = half_sum(some ? one.cross * by : zero);
            const bool endless = __any_sync(0xffffffffu, there && one.endless);
            const Two remains = a.rest && all.tail ? Two{1.f, 0.f} - sum : zero;
            const Two logs = log2_two(lane == 0 ? times(rest, reference_step(all.rest_ref, all.all_ref)) + top : lane == 1 ? rest : lane == 2 ? remains : sum);
            auto log_of = [&](int l, float ref) {                     // natural; what is no number stays so
                const Two x = {__shfl_sync(0xffffffffu, logs.hi, l), __shfl_sync(0xffffffffu, logs.lo, l)};
                return x.hi - x.hi == 0.f ? (x + Two{ref, 0.f}) * SPECDEC_TWO(kLn2) : Two{x.hi, 0.f};
            };
            const Two log_all = log_of(0, all.all_ref), log_rest = log_of(1, all.rest_ref), log_r = log_of(2, 0.f), log_sum = log_of(3, 0.f);
            if (lane == 0) {
                Two loss = zero;
                if (all.asks && !all.none) {
                    // sum of t_i (ln t_i - ln s_i) where t_i = exp(lp_i), and where they are renormalised
                    if (sum.hi > 0.f) {
                        loss = cross + sum * log_all;
                        if (!a.rest) loss = loss * reciprocal(sum) - log_sum - Two{shift, 0.f};
                    }
                    if (remains.hi > 0.f) loss = loss + remains * (log_r - (log_rest - log_all));
                }
                a.loss[r] = all.asks && (all.none || endless) ? w * INFINITY : w * loss.hi;
                if (a.stats) {
                    a.stats[2 * r] = log_all.hi;
                    a.stats[2 * r + 1] = log_rest.hi;
                }
                if (a.status && all.none) atomicOr(a.status + r, SPECDEC_ST_EMPTY_MASK_ROW);
            }
        }
    }
}

// ---------------------------------------------------------------- backward

// log2(e) x = whole - less, whole a whole number (x's, rounded up) and 0 <= less <= 1 without the product's rounding.
__device__ __forceinline__ void in_octaves(float x, float* whole, float* less)
{
    constexpr float kHigh = (float)kLog2e, kLow = (float)(kLog2e - (double)kHigh);
    const float p = x * kHigh;
    *whole = ceilf(p);
    *less = (*whole - p) - fmaf(x, kHigh, -p) - x * kLow;
}

// The gradient from the sums that a forward pass kept: element by element, a CTA a chunk of a row. All in fp32: the sums come in fp32.
constexpr int kChunk = 8;                          // vectors a thread

template <typename T> __global__ void __launch_bounds__(kBackThreads) specdec_distill_backward_kernel(const Args a, const int32_t chunks)
{
    __shared__ Own own[SPECDEC_TOP_MAX];           // of the list, what lies in this chunk
    __shared__ float s_listed, s_left, s_shift, s_norm;
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
    int owned = 0;
    if (warp == 0) {
        List list;
        list.read(a, r);
        uint32_t fault;
        // targets are summed over the whole list: every entry that counts, wherever it lies
        const int32_t begin = row.first(v0), end = row.first(min(v0 + kChunk * kBackThreads, row.vectors));
        const int all_owned = own_entries(a, list, 0, a.V, own, &fault);
        if (a.status && v0 == 0 && fault) atomicOr(a.status + r, fault);
        float shift = a.rest ? 0.f : -INFINITY, sum = 0.f;
        long long fixed = 0;
        if (!a.rest) {
            for (int j = lane; j < all_owned; j += 32) shift = fmaxf(shift, own[j].lp);
            shift = warp_max(shift);
            if (shift == -INFINITY) shift = 0.f;
        }
        for (int j0 = 0; j0 < all_owned; j0 += 32) {
            const bool in = j0 + lane < all_owned;
            Own o = own[in ? j0 + lane : 0];
            if (a.rest) fixed += in ? fixed_of(target_of(o.lp, 0.f)) : 0;
            else sum += in ? expf(o.lp - shift) : 0.f;
            const bool here = in && o.id >= begin && o.id < end;
            const uint32_t all = __ballot_sync(0xffffffffu, here);
            // (the student's logit is read before the row is written: the gradient may lie over it)
            if (here) {
                o.top = to_float<T>(z[o.id]);
                own[owned + __popc(all & ((1u << lane) - 1u))] = o;  // (never behind where it is read)
            }
            owned += __popc(all);
            __syncwarp();
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            fixed += __shfl_xor_sync(0xffffffffu, fixed, o);
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        if (lane == 0) {
            const long long unit = (long long)kFixed;
            s_listed = a.rest ? from_fixed(fixed) : sum > 0.f ? 1.f : 0.f;
            s_left = a.rest && fixed < unit ? from_fixed(unit - fixed) : 0.f;
            s_shift = shift;
            s_norm = a.rest || !(sum > 0.f) ? 1.f : 1.f / sum;
        }
    }
    __syncthreads();
    const float listed = s_listed, left_over = s_left;
    // the exponentials of this kernel are taken at the rest's sum; where there is none, no element is outside the list
    const bool tail = !(lse_rest == -INFINITY), none = lse == -INFINITY || !(listed + left_over > 0.f);
    const float left = tail ? left_over : 0.f, each = none ? 0.f : w * a.inverse;
    float all, all_less, ref, ref_less;
    in_octaves(none ? 0.f : lse, &all, &all_less);
    in_octaves(tail ? lse_rest : 0.f, &ref, &ref_less);
    const float factor = tail ? ((listed + left) * exp2f(ref - all + all_less) - left * exp2f(ref_less)) * each : 0.f;
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
    for (int j = tid; warp == 0 && j < owned; j += 32) {
        const Own o = own[j];
        const float share = exp2f(exponent(o.top, a, all) + all_less) * (listed + left);
        g[o.id] = from_float<T>((share - expf(o.lp - s_shift) * s_norm) * each);
    }
}

// ---------------------------------------------------------------- host

struct Shape {
    int32_t cluster, slice, threads;
};

// A row goes to the fewest CTAs that keep three of them on an SM, more where the rows alone do not fill the GPU, and at most to
// sixteen. A part of up to 44 KB has four warps or fewer, so that five CTAs share an SM: while some wait for the others of their
// cluster, the rest read and write. Measured, 2048 bf16 rows against 64 ids with the gradient: V = 151936 (38 KB parts) 267 us with
// four warps, 416 with eight; V = 128256 (64 KB parts) 276 and 217.
template <typename T> Shape shape_of(int32_t rows, int32_t V)
{
    const int32_t vectors = most_vectors<T>(V);
    int32_t cluster = 1;
    auto slice = [&] { return (vectors + cluster - 1) / cluster; };
    while (cluster < kMaxCluster && (slice() > kSliceBytes / 16 || ((int64_t)rows * cluster < 152 && slice() > 8 * 1024 / 16))) cluster *= 2;
    const int32_t most = slice() > kSmallBytes / 16 ? kRowWarps : 4, warps = (slice() + 32 * kLaneVectors - 1) / (32 * kLaneVectors);
    return Shape{cluster, slice(), ((slice() > kSmallBytes / 16 || warps > most ? most : warps) + 2) * 32};
}

// What a kernel remembers: the devices on which it may have its shared memory and clusters of sixteen, and how many clusters of the
// shape last asked for are resident at once (the shape in the upper half).
struct Memory {
    std::atomic<uint64_t> allowed{0}, resident{0};
};

cudaError_t launch_clusters(void (*kernel)(Args), const Args& a, const Shape& shape, Memory& memory, cudaStream_t stream)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = 1ull << (dev & 63);
    for (int attempt = memory.allowed.load() & bit ? 0 : 1; e == cudaSuccess; ++attempt) {
        // (once a device; again where a launch fails, for a device may have been reset)
        if (attempt > 0) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostBytes);
            if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) break;
        }
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)shape.cluster);
        cfg.blockDim = dim3((unsigned)shape.threads);
        cfg.dynamicSmemBytes = (size_t)shape.slice * 16;
        cfg.stream = stream;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {(unsigned)shape.cluster, 1, 1};
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const uint64_t key = (uint64_t)(dev & 63) << 58 | (uint64_t)shape.cluster << 52 | (uint64_t)(shape.threads / 32) << 47 | (uint64_t)shape.slice << 32;
        uint64_t known = memory.resident.load();
        if ((known >> 32) != (key >> 32)) {
            int clusters = 0;
            e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
            if (e != cudaSuccess || clusters < 1) {
                (void)cudaGetLastError();
                if (e == cudaSuccess || attempt > 0) return e != cudaSuccess ? e : cudaErrorInvalidConfiguration;
                e = cudaSuccess;
                continue;
            }
            known = key | (uint32_t)clusters;
            memory.resident = known;
        }
        const uint32_t clusters = (uint32_t)known;
        cfg.numAttrs = 2;
        cfg.gridDim = dim3((clusters < (uint32_t)a.rows ? clusters : (uint32_t)a.rows) * (unsigned)shape.cluster);
        if (cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess) {
            memory.allowed |= bit;
            return cudaSuccess;
        }
        (void)cudaGetLastError();
        if (attempt > 0) e = cudaErrorUnknown;
    }
    (void)cudaGetLastError();
    return e;
}

template <typename T> specdec_status_t launch_forward(Args a, cudaStream_t stream)
{
    static Memory memory[2];
    const Shape shape = shape_of<T>(a.rows, a.V);
    if (shape.slice > kMostBytes / 16) return SPECDEC_ERR_UNSUPPORTED;
    a.slice = shape.slice;
    const cudaError_t e = a.grad ? launch_clusters(specdec_distill_kernel<T, true>, a, shape, memory[1], stream)
                                 : launch_clusters(specdec_distill_kernel<T, false>, a, shape, memory[0], stream);
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
                weight, loss, stats, grad, grad_row_stride, status, 0};
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
