/*
 * specdec_top.cu -- the best ids of rows of logits, and a beam step's selection, for GB300 (sm_103a); C-ABI entry points in
 * include/specdec.h.
 *
 * Two kernels for the rows, a third for the beams:
 *
 *   stream   reads every row once. A warp takes a unit of 256 vectors (4 KB), a lane 8 of them, 512 bytes apart: their sum of
 *            exponentials goes into the unit's (reference, sum) pair, and the largest element of every 128 bytes (a
 *            group) is kept.
 *   select   a CTA a row: joins the sums, and finds the n best elements through the groups' maxima. The n-th largest of 256
 *            numbers, each the largest of some groups' maxima, is a lower bound of the n-th best element, so that only
 *            the groups that reach it (about n) are read again.
 *   merge    a CTA a request: the beams' lists hold everything that can survive; a candidate's rank is its place in its
 *            own list plus, by bisection, how many entries of each other list come before it.
 *
 * The stream is bound by HBM: 2048 rows of 128256 bf16 logits in 78.8 us, 98 % of the measured copy rate (eight 16-byte loads a
 * thread in flight, no shared memory; 3 % of the bytes go into the groups' maxima and their second reading). The selection takes 20 us more of
 * that call's 97.6, bound by instructions (issue 70 %). 128 threads a row: 102; its 64-bit sums: 106; groups of a lane's own
 * eight vectors, which are 512 bytes apart: 117, for 64 of them are 32 KB of DRAM bursts a row where 128 contiguous bytes are 8.
 * Under a bitmask only vectors with an allowed id are loaded: 768 rows of 151936 fp32 logits with 5 % allowed in 48.8 us (157 MB of 467 read),
 * 105 when every vector was gone through. A beam step over 1024 rows of 128256 fp32 logits: 87.9 us, 88 % of the copy rate.
 */
#include "specdec_logits.cuh"

namespace {

using namespace specdec;

constexpr int kThreads = 256;                      // of the stream and the merge
constexpr int kUnitVectors = 256;                  // a warp's: 8 a lane
constexpr int kLaneVectors = kUnitVectors / 32, kGroupVectors = kUnitVectors / 32;
constexpr int kSelectThreads = 256;
constexpr int kBounds = 256;                       // the numbers of which the n-th largest bounds the n-th best element
constexpr int kMaxGroups = 1024, kMaxFound = 1024;
constexpr int kMaxMerge = 4096;                    // candidates of one request

struct StreamArgs {
    const void* logits;
    int64_t row_stride, rows;
    int32_t V, units;
    const int32_t* bitmask;
    int32_t words;
    float scale;
    const float* scores;                           // beams: a row whose beam is finished, or whose score is not finite, is not read
    const uint8_t* finished;
    float2* sums;                                  // [rows, units]
    void* maxima;                                  // [rows, units, 32], the logits' type
};

// (Scores and flags past L1: the call before may have written them in place of its own, a line's parts by several CTAs that had read
// it, while this kernel had been set up already.)
__device__ __forceinline__ bool live_beam(const float* scores, const uint8_t* finished, int64_t row)
{
    return !scores || (isfinite(__ldcg(scores + row)) && !(finished && __ldcg(finished + row)));
}

template <typename T> __global__ void __launch_bounds__(kThreads) specdec_rows_stream_kernel(const StreamArgs a)
{
    after_predecessor();
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t r = unit / a.units;
    if (r >= a.rows || !live_beam(a.scores, a.finished, r)) return;
    const int u = (int)(unit - r * a.units);
    const Row<T> row(static_cast<const T*>(a.logits) + r * a.row_stride, a.V);
    const int v0 = u * kUnitVectors + lane;
    Raw<T, kPer<T>> x[kLaneVectors];
#pragma unroll
    for (int i = 0; i < kLaneVectors; ++i) load_vector(row, v0 + i * 32, x[i]);
    Maximum<T> part[kLaneVectors];
#pragma unroll
    for (int i = 0; i < kLaneVectors; ++i) part[i] = Maximum<T>::of(x[i]);
    Maximum<T> own = part[0];
#pragma unroll
    for (int i = 1; i < kLaneVectors; ++i) own = larger(own, part[i]);
    float m = own.value();
    if (!(m > -INFINITY)) m = -INFINITY;           // (nothing but NaN)
    float ref = m == -INFINITY ? m : whole_reference(m, a.scale), S = 0.f;
    const float from = m == -INFINITY ? 0.f : ref;
    const Pair c = pair_of(a.scale, a.scale), less = pair_of(-from, -from);
    Pair sum = pair_of(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kLaneVectors; ++i) {
        Pair some = exp2_2(fma_2(elements(x[i], 0), c, less));
#pragma unroll
        for (int e = 1; e < kPer<T> / 2; ++e) some = add_2(some, exp2_2(fma_2(elements(x[i], e), c, less)));
        sum = add_2(sum, some);
    }
    S = both(sum).x + both(sum).y;
    // The maxima of 8 neighbouring lanes' i-th vectors, 128 bytes, meet in the i-th of those lanes: three exchanges, of 4, 2 and 1.
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) {
        const bool high = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const Maximum<T> kept = high ? part[i + o] : part[i], given = high ? part[i] : part[i + o];
            part[i] = larger(kept, Maximum<T>::from(__shfl_xor_sync(0xffffffffu, given.bits(), o)));
        }
    }
    static_cast<T*>(a.maxima)[unit * 32 + (lane & 7) * 4 + (lane >> 3)] = from_float<T>(part[0].value());
    warp_join(ref, S);
    if (lane == 0) a.sums[unit] = make_float2(ref, S);
}

// The same under a bitmask. A lane takes the mask of one group; the vectors in which an id is allowed are listed side by side
// for the warp, and only those are loaded, a lane one. (Where 5 % of the ids are allowed that is a twelfth of fp32's vectors and an eighth
// of the 16-bit types'; with all allowed the list is the whole unit, and 1024 rows of 128256
// bf16 logits take 81 us where no mask takes 48. Four loads a lane in flight took registers, and with them warps: 48.7 -> 59.5 with 5 %.)
template <typename T> __global__ void __launch_bounds__(kThreads) specdec_rows_stream_masked_kernel(const StreamArgs a)
{
    constexpr int kWords = 8 * kPer<T> / 32;       // of a group's mask
    __shared__ uint16_t listed[kThreads / 32][kUnitVectors];
    __shared__ uint32_t best[kThreads / 32][32];
    after_predecessor();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + warp;
    const int64_t r = unit / a.units;
    if (r >= a.rows || !live_beam(a.scores, a.finished, r)) return;
    const int u = (int)(unit - r * a.units);
    const Row<T> row(static_cast<const T*>(a.logits) + r * a.row_stride, a.V);
    const int32_t* const words = a.bitmask + r * a.words;
    // bits of the group's elements first .. first + 32 kWords - 1; what lies outside the row is 0
    const int32_t v0 = u * kUnitVectors, first = row.first(v0 + lane * kGroupVectors);
    uint32_t bits[kWords + 1];
#pragma unroll
    for (int i = 0; i <= kWords; ++i) {
        const int32_t w = (first >> 5) + i;        // (first may be negative: the first group of a row off the grid)
        bits[i] = w >= 0 && w < a.words && (i < kWords || (first & 31)) ? (uint32_t)words[w] : 0u;
    }
    best[warp][lane] = 0;
    uint32_t some[kWords];                         // a bit for each vector with one
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        bits[i] = __funnelshift_r(bits[i], bits[i + 1], first & 31);
        const int32_t at = first + i * 32;
        if (at < 0) bits[i] &= at > -32 ? 0xffffffffu << -at : 0u;
        if (at + 32 > a.V) bits[i] &= at < a.V ? (1u << (a.V - at)) - 1u : 0u;
        uint32_t t = bits[i] | bits[i] >> 1;
        t |= t >> 2;
        if (kPer<T> == 8) t |= t >> 4;
        some[i] = t & (kPer<T> == 8 ? 0x01010101u : 0x11111111u);
        mine += __popc(some[i]);
    }
    int to = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, to, o);
        if (lane >= o) to += y;
    }
    const int count = __shfl_sync(0xffffffffu, to, 31);
    to -= mine;
#pragma unroll
    for (int i = 0; i < kGroupVectors; ++i) {
        const int bit = i * kPer<T> % 32, word = i * kPer<T> / 32;
        if (some[word] >> bit & 1) listed[warp][to++] = (uint16_t)(lane * kGroupVectors + i | (bits[word] >> bit & ((1u << kPer<T>) - 1u)) << 8);
    }
    __syncwarp();
    float ref = -INFINITY;
    Pair sum = pair_of(0.f, 0.f);
    const Pair c = pair_of(a.scale, a.scale);
    for (int j = lane; j < count; j += 32) {
        const uint32_t entry = listed[warp][j];
        const int i = entry & 255;
        Raw<T, kPer<T>> x;
        load_vector(row, v0 + i, x);
        apply_bits<T>(x, entry >> 8);
        const float m = Maximum<T>::of(x).value();
        const uint32_t key = order_key(m);
        if (key) {
            atomicMax(&best[warp][i / kGroupVectors], key);
            const float up = whole_reference(m, a.scale);
            if (up > ref) {
                const float step = reference_step(ref, up);
                sum = mul_2(sum, pair_of(step, step));
                ref = up;
            }
        }
        const float from = ref == -INFINITY ? 0.f : ref;
        const Pair less = pair_of(-from, -from);
        Pair part = exp2_2(fma_2(elements(x, 0), c, less));
#pragma unroll
        for (int e = 1; e < kPer<T> / 2; ++e) part = add_2(part, exp2_2(fma_2(elements(x, e), c, less)));
        sum = add_2(sum, part);
    }
    __syncwarp();
    const uint32_t key = best[warp][lane];
    static_cast<T*>(a.maxima)[unit * 32 + lane] = from_float<T>(key ? key_value(key) : -INFINITY);
    float S = both(sum).x + both(sum).y;
    warp_join(ref, S);
    if (lane == 0) a.sums[unit] = make_float2(ref, S);
}

struct SelectArgs {
    StreamArgs s;
    int32_t n;
    int32_t* ids;                                  // [rows, n], -1 behind the last
    float* logprobs;                               // [rows, n] or nullptr
    float* lse;                                    // [rows] or nullptr
    uint32_t* status;                              // [rows] or nullptr
    float* values;                                 // beams: the elements [rows, n], -infinity behind the last
    double* sums;                                  // beams: ln of the sum of exp, [rows]
};

// The value of a bound on keys: of what lies below every key, the lowest number (-infinity and NaN are never at or above it).
__device__ __forceinline__ float bound_value(uint32_t key) { return key <= 0x00800000u ? -3.402823466e38f : key_value(key); }

// The largest t, a multiple of 2^low, with at least n of some numbers (count(t) of them) at or above it.
template <typename Count> __device__ __forceinline__ uint32_t nth_largest(int n, int low, Count count)
{
    uint32_t t = 0;
    for (int bit = 31; bit >= low; --bit) {
        const uint32_t next = t | 1u << bit;
        if (count(next) >= n) t = next;
    }
    return t;
}

// The sum of one number a thread, the same in every thread; two barriers.
template <int kCount> __device__ __forceinline__ int block_sum(int x, int* part)
{
    x = __reduce_add_sync(0xffffffffu, x);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kCount / 32; ++w) sum += part[w];
    __syncthreads();
    return sum;
}

template <typename T> struct Select {
    const SelectArgs& a;
    const int64_t r;
    const Row<T> row;
    const int32_t* words;

    __device__ __forceinline__ Select(const SelectArgs& args, int64_t at)
        : a(args), r(at), row(static_cast<const T*>(args.s.logits) + at * args.s.row_stride, args.s.V),
          words(args.s.bitmask ? args.s.bitmask + at * args.s.words : nullptr)
    {
    }
    __device__ __forceinline__ void load(int32_t v, Raw<T, kPer<T>>& x) const
    {
        load_vector(row, v, x);
        if (words) apply_bits<T>(x, vector_bits(row, words, v));
    }
    // Calls f(key, element) for every element of vector v that is at least `bound`.
    template <typename F> __device__ __forceinline__ void each_from(float bound, int32_t v, F f) const
    {
        Raw<T, kPer<T>> x;
        load(v, x);
        if (!(Maximum<T>::of(x).value() >= bound)) return;
        const int32_t at = row.first(v);
#pragma unroll
        for (int e = 0; e < kPer<T>; ++e) {
            const float z = to_float<T>(x.e[e]);
            if (z >= bound) f(order_key(z), at + e);
        }
    }
    // Calls f(key, element) for every element of vector v (key 0: it cannot be chosen).
    template <typename F> __device__ __forceinline__ void each(int32_t v, F f) const
    {
        Raw<T, kPer<T>> x;
        load(v, x);
        const int32_t at = row.first(v);
#pragma unroll
        for (int e = 0; e < kPer<T>; ++e) f(order_key(to_float<T>(x.e[e])), at + e);
    }
};

// (z scale - log_sum) ln 2
__device__ __forceinline__ float log_probability(float z, float scale, Two log_sum)
{
    const Two zc = two_product(z, scale);
    return ((zc.hi - log_sum.hi) + (zc.lo - log_sum.lo)) * (float)kLn2;
}

// An element as one number: by value, then the lower index first. Never 0.
__device__ __forceinline__ unsigned long long composite(uint32_t key, int32_t at)
{
    return (unsigned long long)key << 32 | (uint32_t)~at;
}

template <typename T> __global__ void __launch_bounds__(kSelectThreads, 8) specdec_rows_select_kernel(const SelectArgs a)
{
    constexpr int kWarps = kSelectThreads / 32, kMine = kMaxFound / kSelectThreads, kSides = kBounds / kSelectThreads;
    __shared__ unsigned long long found[kMaxFound];
    __shared__ int32_t groups[kMaxGroups];
    __shared__ uint32_t bounds[kBounds];
    __shared__ Two row_sum;
    __shared__ uint32_t bound;
    __shared__ int counts[kWarps];
    __shared__ int num_groups, num_found;
    after_predecessor();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.n;
    const int64_t r = blockIdx.x;
    if (!live_beam(a.s.scores, a.s.finished, r)) return;
    const Select<T> sel(a, r);
    if (tid == 0) num_groups = num_found = 0;

    // 256 numbers, each the largest of a set of the row's elements: of every 256th vector of the groups' maxima, where those are
    // too few of every 256th group, and in rows of fewer than 2 n groups of every 256th vector of the row itself
    const T* const maxima = static_cast<const T*>(a.s.maxima) + r * a.s.units * 32;
    const int32_t vectors = a.s.units * 32 / kPer<T>;
    auto largest = [&](int32_t v) {
        Raw<T, kPer<T>> x;
        x.load(maxima + v * kPer<T>);
        return order_key(Maximum<T>::of(x).value());
    };
#pragma unroll
    for (int side = 0; side < kSides; ++side) {
        uint32_t top = 0;
        const int32_t first = tid + side * kSelectThreads;
        if (vectors >= kBounds) {
            for (int32_t v = first; v < vectors; v += kBounds) top = max(top, largest(v));
        } else if (sel.row.vectors / kGroupVectors >= 2 * n) {
            for (int32_t g = first; g < vectors * kPer<T>; g += kBounds) top = max(top, order_key(to_float<T>(maxima[g])));
        } else {
            for (int32_t v = first; v < sel.row.vectors; v += kBounds) {
                Raw<T, kPer<T>> x;
                sel.load(v, x);
                top = max(top, order_key(Maximum<T>::of(x).value()));
            }
        }
        bounds[tid + side * kSelectThreads] = top;
    }
    __syncthreads();
    if (warp == 0) {
        // the n-th largest of them, its upper 16 bits (a lower bound of a lower bound)
        uint32_t mine[kBounds / 32];
#pragma unroll
        for (int i = 0; i < kBounds / 32; ++i) mine[i] = bounds[lane + i * 32];
        const uint32_t t = nth_largest(n, 16, [&](uint32_t t) {
            int c = 0;
#pragma unroll
            for (int i = 0; i < kBounds / 32; ++i) c += mine[i] >= t;
            return (int)__reduce_add_sync(0xffffffffu, c);
        });
        if (lane == 0) bound = max(t, 1u);
    } else if (warp == 1) {
        // the row's sum, in pairs of floats and always in the same order
        const float2* sums = a.s.sums + r * a.s.units;
        float ref = -INFINITY;
        for (int u = lane; u < a.s.units; u += 32) ref = fmaxf(ref, sums[u].x);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
        Two S = {0.f, 0.f};
        for (int u = lane; u < a.s.units; u += 32) S = S + Two{sums[u].y * reference_step(sums[u].x, ref), 0.f};
        S = log2_two(warp_sum(S));
        // in units of the exponents
        if (lane == 0) row_sum = S.hi - S.hi == 0.f && ref > -INFINITY ? Two{ref, 0.f} + S : Two{S.hi + ref, 0.f};
    }
    __syncthreads();
    const uint32_t least = bound;
    const float least_value = bound_value(least);
    for (int32_t v = tid; v < vectors; v += kSelectThreads) {
        Raw<T, kPer<T>> x;
        x.load(maxima + v * kPer<T>);
        if (!(Maximum<T>::of(x).value() >= least_value)) continue;
#pragma unroll
        for (int e = 0; e < kPer<T>; ++e)
            if (to_float<T>(x.e[e]) >= least_value) {
                const int at = atomicAdd(&num_groups, 1);
                if (at < kMaxGroups) groups[at] = v * kPer<T> + e;
            }
    }
    __syncthreads();
    const int want = num_groups;
    if (want <= kMaxGroups) {
        for (int i = tid; i < want * kGroupVectors; i += kSelectThreads)
            sel.each_from(least_value, groups[i / kGroupVectors] * kGroupVectors + i % kGroupVectors, [&](uint32_t key, int32_t at) {
                const int to = atomicAdd(&num_found, 1);
                if (to < kMaxFound) found[to] = composite(key, at);
            });
    }
    __syncthreads();
    int have = num_found;
    if (want > kMaxGroups || have > kMaxFound) {
        // So many groups or elements reach the bound that they do not fit (equal values for the most part): the n-th largest
        // key from counts over the row itself, what lies above it, and of its equals the first ones.
        __syncthreads();
        if (tid == 0) num_found = 0;
        const uint32_t nth = max(1u, nth_largest(n, kKeyLow<T>, [&](uint32_t t) {
            int mine = 0;
            for (int32_t v = tid; v < sel.row.vectors; v += kSelectThreads) sel.each(v, [&](uint32_t key, int32_t) { mine += key >= t; });
            return block_sum<kSelectThreads>(mine, counts);
        }));
        const uint32_t above = nth | ((1u << kKeyLow<T>) - 1u);       // (a key's low bits follow from the others)
        for (int32_t v = tid; v < sel.row.vectors; v += kSelectThreads)
            sel.each(v, [&](uint32_t key, int32_t at) {
                if (key > above) found[atomicAdd(&num_found, 1)] = composite(key, at);
            });
        __syncthreads();
        have = num_found;
        for (int32_t v0 = 0; v0 < sel.row.vectors && have < n; v0 += kSelectThreads) {
            int mine = 0;
            if (v0 + tid < sel.row.vectors) sel.each(v0 + tid, [&](uint32_t key, int32_t) { mine += key >= nth && key <= above; });
            int before = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, before, o);
                if (lane >= o) before += y;
            }
            if (lane == 31) counts[warp] = before;
            __syncthreads();
            int to = have + before - mine, sum = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) to += counts[w];
                sum += counts[w];
            }
            if (mine && to < n)
                sel.each(v0 + tid, [&](uint32_t key, int32_t at) {
                    if (key >= nth && key <= above && to < n) found[to++] = composite(key, at);
                });
            have = min(n, have + sum);
            __syncthreads();
        }
    } else if (have > 384) {
        // few rows come here (wide ties, small vocabularies): the n-th largest first, so that ranks are counted among few
        unsigned long long mine[kMine];
#pragma unroll
        for (int i = 0; i < kMine; ++i) mine[i] = tid + i * kSelectThreads < have ? found[tid + i * kSelectThreads] : 0;
        const uint32_t nth = max(1u, nth_largest(n, kKeyLow<T>, [&](uint32_t t) {
            int c = 0;
#pragma unroll
            for (int i = 0; i < kMine; ++i) c += (uint32_t)(mine[i] >> 32) >= t;
            return block_sum<kSelectThreads>(c, counts);
        }));
        if (tid == 0) num_found = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kMine; ++i)
            if ((uint32_t)(mine[i] >> 32) >= nth) found[atomicAdd(&num_found, 1)] = mine[i];
        __syncthreads();
        have = num_found;
    }

    // ranks among what was found: they are the places, whatever the order of the finding was
    const Two log_sum = row_sum;
    for (int i = tid; i < have; i += kSelectThreads) {
        const unsigned long long me = found[i];
        int rank = 0;
        for (int j = 0; j < have; ++j) rank += found[j] > me;
        if (rank >= n) continue;
        const float z = key_value((uint32_t)(me >> 32));
        a.ids[r * n + rank] = (int32_t)~(uint32_t)me;
        if (a.values) a.values[r * n + rank] = z;
        if (a.logprobs) a.logprobs[r * n + rank] = log_sum.hi == -INFINITY ? -INFINITY : log_probability(z, a.s.scale, log_sum);
    }
    for (int i = have + tid; i < n; i += kSelectThreads) {
        a.ids[r * n + i] = -1;
        if (a.values) a.values[r * n + i] = -INFINITY;
        if (a.logprobs) a.logprobs[r * n + i] = -INFINITY;
    }
    if (tid == 0) {
        const bool number = log_sum.hi - log_sum.hi == 0.f;
        const Two natural = number ? log_sum * SPECDEC_TWO(kLn2) : log_sum;
        if (a.lse) a.lse[r] = natural.hi;
        if (a.sums) a.sums[r] = number ? ((double)log_sum.hi + (double)log_sum.lo) / (double)a.s.scale : (double)log_sum.hi;
        if (a.status && have == 0) atomicOr(a.status + r, SPECDEC_ST_EMPTY_MASK_ROW);
    }
}

struct MergeArgs {
    const float* values;                           // [B * beams, n]
    const int32_t* ids;
    const double* sums;
    const float* scores;
    const uint8_t* finished;
    int32_t beams, n, end_token;
    int32_t *rows, *tokens;
    float* next;
    uint8_t* ended;
    uint32_t* status;
};

constexpr long long kNone = (long long)0x8000000000000000ull;        // below every score's key

// A signed number that orders doubles as they are ordered.
__device__ __forceinline__ long long order_key_64(double x)
{
    const long long b = __double_as_longlong(x + 0.0);
    return b ^ (b < 0 ? 0x7fffffffffffffffll : 0);
}

__global__ void __launch_bounds__(kThreads) specdec_beam_merge_kernel(const MergeArgs a)
{
    extern __shared__ long long keys[];                              // [beams][n], each beam's best first
    __shared__ int counts[kThreads / 32];
    __shared__ float scores[SPECDEC_TOP_MAX];                        // read once: the outputs may lie over the inputs
    __shared__ uint8_t done[SPECDEC_TOP_MAX];
    __shared__ long long least;                                      // the best of the beams' n-th: what is below it has n before it
    after_predecessor();
    const int tid = threadIdx.x, n = a.n, total = a.beams * n;
    const int64_t b = blockIdx.x, row0 = b * a.beams;
    if (tid < a.beams) {
        scores[tid] = __ldcg(a.scores + row0 + tid);
        done[tid] = a.finished && __ldcg(a.finished + row0 + tid);
    }
    if (tid == 0) least = kNone;
    __syncthreads();
    int valid = 0;
    uint32_t bad = 0;
    for (int i = tid; i < total; i += kThreads) {
        const int w = i / n, k = i - w * n;
        const float score = scores[w];
        long long key = kNone;
        if (!isfinite(score)) {
            if (score != -INFINITY) bad |= SPECDEC_ST_BAD_SCORE;
        } else if (done[w]) {
            if (k == 0) key = order_key_64((double)score);
        } else {
            const double s = (double)score + ((double)a.values[(row0 + w) * n + k] - a.sums[row0 + w]);
            const bool there = a.ids[(row0 + w) * n + k] >= 0;
            if (there && isfinite(s)) key = order_key_64(s);
            else if (k == 0) bad |= !there || a.sums[row0 + w] == -INFINITY ? SPECDEC_ST_EMPTY_MASK_ROW : SPECDEC_ST_BAD_SCORE;
        }
        keys[i] = key;
        valid += key != kNone;
    }
    if (a.status && bad) atomicOr(a.status + b, bad);
    valid = block_sum<kThreads>(valid, counts);                      // (its barriers also publish the keys)
    if (tid < a.beams) atomicMax(&least, keys[tid * n + n - 1]);
    __syncthreads();
    for (int i = tid; i < total; i += kThreads) {
        const int w = i / n, k = i - w * n;
        const long long key = keys[i];
        if (key == kNone || key < least) continue;
        int rank = k;
        for (int o = 0; o < a.beams && rank < n; ++o) {
            if (o == w) continue;
            // entries of beam o before this one: those above it, and its equals where o is the lower beam
            const long long* list = keys + o * n;
            int lo = 0, hi = n;
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                const bool before = o < w ? list[mid] >= key : list[mid] > key;
                lo = before ? mid + 1 : lo;
                hi = before ? hi : mid;
            }
            rank += lo;
        }
        if (rank >= n) continue;
        const int32_t token = done[w] ? a.end_token : a.ids[(row0 + w) * n + k];
        const float score = scores[w];
        a.rows[b * n + rank] = (int32_t)(row0 + w);
        a.tokens[b * n + rank] = token;
        a.next[b * n + rank] = done[w] ? score : (float)((double)score + ((double)a.values[(row0 + w) * n + k] - a.sums[row0 + w]));
        if (a.ended) a.ended[b * n + rank] = done[w] || (a.end_token >= 0 && token == a.end_token);
    }
    for (int i = min(valid, n) + tid; i < n; i += kThreads) {
        a.rows[b * n + i] = -1;
        a.tokens[b * n + i] = -1;
        a.next[b * n + i] = -INFINITY;
        if (a.ended) a.ended[b * n + i] = 0;
    }
}

// ---------------------------------------------------------------- host

inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

inline int32_t units_of(int32_t V, specdec_dtype_t dtype)
{
    const int32_t v = dtype == SPECDEC_F32 ? most_vectors<float>(V) : most_vectors<__half>(V);
    return (v + kUnitVectors - 1) / kUnitVectors;
}

struct Layout {
    size_t sums, maxima, values, ids, logs, end;
};

// Where the parts of a workspace lie; n = 0: without the beams' lists.
inline Layout layout_of(int64_t rows, int32_t V, specdec_dtype_t dtype, int32_t n)
{
    const size_t units = (size_t)rows * units_of(V, dtype);
    Layout l;
    l.sums = 0;
    l.maxima = round_up(units * sizeof(float2), 16);
    l.values = round_up(l.maxima + units * 32 * elem_bytes(dtype), 16);
    l.ids = l.values + round_up((size_t)rows * n * 4, 16);
    l.logs = l.ids + round_up((size_t)rows * n * 4, 16);
    l.end = l.logs + (n ? round_up((size_t)rows * 8, 16) : 0);
    return l;
}

inline bool sizes_fit(int64_t rows, int32_t V, specdec_dtype_t dtype)
{
    return (rows * units_of(V, dtype) + kThreads / 32 - 1) / (kThreads / 32) <= 0x7fffffff && rows <= 0x7fffffff;
}

template <typename T> specdec_status_t launch_rows(const StreamArgs& s, const SelectArgs& a, cudaStream_t stream)
{
    const int64_t units = s.rows * s.units;
    const unsigned grid = (unsigned)((units + kThreads / 32 - 1) / (kThreads / 32));
    cudaError_t e = s.bitmask ? launch_dependent(specdec_rows_stream_masked_kernel<T>, grid, kThreads, 0, stream, s)
                              : launch_dependent(specdec_rows_stream_kernel<T>, grid, kThreads, 0, stream, s);
    if (e == cudaSuccess) e = launch_dependent(specdec_rows_select_kernel<T>, (unsigned)s.rows, kSelectThreads, 0, stream, a);
    return e == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

specdec_status_t launch_rows(const StreamArgs& s, SelectArgs a, specdec_dtype_t dtype, cudaStream_t stream)
{
    a.s = s;
    if (dtype == SPECDEC_F32) return launch_rows<float>(s, a, stream);
    if (dtype == SPECDEC_BF16) return launch_rows<__nv_bfloat16>(s, a, stream);
    return launch_rows<__half>(s, a, stream);
}

}  // namespace

extern "C" size_t specdec_top_logits_workspace_size(int32_t rows, int32_t V, specdec_dtype_t dtype)
{
    if (rows <= 0 || V < 1 || V > kMaxVocab || !is_float_type(dtype) || !sizes_fit(rows, V, dtype)) return 0;
    return layout_of(rows, V, dtype, 0).values;
}

extern "C" specdec_status_t specdec_top_logits(const void* logits, specdec_dtype_t dtype, int32_t rows, int32_t V,
                                               int64_t row_stride, const int32_t* bitmask, double temperature, int32_t n,
                                               int32_t* out_ids, float* out_logprobs, float* lse, uint32_t* status,
                                               void* workspace, size_t workspace_bytes, void* stream)
{
    const specdec_status_t rc = check_logits(logits, dtype, rows, V, row_stride);
    if (rc != SPECDEC_OK) return rc;
    if (n < 1 || n > SPECDEC_TOP_MAX || !usable_temperature(temperature)) return SPECDEC_ERR_INVALID_ARG;
    if (rows == 0) return SPECDEC_OK;
    if (!out_ids || !out_logprobs || !workspace) return SPECDEC_ERR_INVALID_ARG;
    if (!aligned_to(bitmask, 4) || !aligned_to(out_ids, 4) || !aligned_to(out_logprobs, 4) || !aligned_to(lse, 4) || !aligned_to(status, 4) ||
        !aligned_to(workspace, 16))
        return SPECDEC_ERR_INVALID_ARG;
    if (!sizes_fit(rows, V, dtype)) return SPECDEC_ERR_UNSUPPORTED;
    const Layout l = layout_of(rows, V, dtype, 0);
    if (workspace_bytes < l.values) return SPECDEC_ERR_INVALID_ARG;
    char* const w = static_cast<char*>(workspace);
    const StreamArgs s = {logits, row_stride, rows, V, units_of(V, dtype), bitmask, (V + 31) / 32, (float)scale_of(temperature), nullptr, nullptr,
                          reinterpret_cast<float2*>(w + l.sums), w + l.maxima};
    const SelectArgs a = {s, n, out_ids, out_logprobs, lse, status, nullptr, nullptr};
    return launch_rows(s, a, dtype, (cudaStream_t)stream);
}

extern "C" size_t specdec_beam_select_workspace_size(int32_t B, int32_t beams, int32_t V, specdec_dtype_t dtype, int32_t n)
{
    if (B <= 0 || beams < 1 || beams > SPECDEC_TOP_MAX || V < 1 || V > kMaxVocab || !is_float_type(dtype) || n < 1 || n > SPECDEC_TOP_MAX ||
        (int64_t)beams * n > kMaxMerge || !sizes_fit((int64_t)B * beams, V, dtype))
        return 0;
    return layout_of((int64_t)B * beams, V, dtype, n).end;
}

extern "C" specdec_status_t specdec_beam_select(const void* logits, specdec_dtype_t dtype, int32_t B, int32_t beams, int32_t V,
                                                int64_t row_stride, const int32_t* bitmask, const float* scores,
                                                const uint8_t* finished, int32_t end_token, int32_t n, int32_t* out_rows,
                                                int32_t* out_tokens, float* out_scores, uint8_t* out_finished, uint32_t* status,
                                                void* workspace, size_t workspace_bytes, void* stream)
{
    if (B < 0 || beams < 1 || n < 1 || n > SPECDEC_TOP_MAX || beams > SPECDEC_TOP_MAX) return SPECDEC_ERR_INVALID_ARG;
    const int64_t rows = (int64_t)B * beams;
    const specdec_status_t rc = check_logits(logits, dtype, rows, V, row_stride);
    if (rc != SPECDEC_OK) return rc;
    if (end_token < -1 || end_token >= V || (finished && end_token < 0)) return SPECDEC_ERR_INVALID_ARG;
    if ((int64_t)beams * n > kMaxMerge) return SPECDEC_ERR_UNSUPPORTED;
    if (B == 0) return SPECDEC_OK;
    if (!scores || !out_rows || !out_tokens || !out_scores || !workspace) return SPECDEC_ERR_INVALID_ARG;
    if (!aligned_to(bitmask, 4) || !aligned_to(scores, 4) || !aligned_to(out_rows, 4) || !aligned_to(out_tokens, 4) ||
        !aligned_to(out_scores, 4) || !aligned_to(status, 4) || !aligned_to(workspace, 16))
        return SPECDEC_ERR_INVALID_ARG;
    if (!sizes_fit(rows, V, dtype)) return SPECDEC_ERR_UNSUPPORTED;
    const Layout l = layout_of(rows, V, dtype, n);
    if (workspace_bytes < l.end) return SPECDEC_ERR_INVALID_ARG;
    char* const w = static_cast<char*>(workspace);
    const StreamArgs s = {logits, row_stride, rows, V, units_of(V, dtype), bitmask, (V + 31) / 32, (float)scale_of(1.0), scores, finished,
                          reinterpret_cast<float2*>(w + l.sums), w + l.maxima};
    const SelectArgs a = {s, n, reinterpret_cast<int32_t*>(w + l.ids), nullptr, nullptr, nullptr, reinterpret_cast<float*>(w + l.values),
                          reinterpret_cast<double*>(w + l.logs)};
    const specdec_status_t done = launch_rows(s, a, dtype, (cudaStream_t)stream);
    if (done != SPECDEC_OK) return done;
    const MergeArgs m = {a.values, a.ids, a.sums, scores, finished, beams, n, end_token, out_rows, out_tokens, out_scores, out_finished, status};
    const cudaError_t e = launch_dependent(specdec_beam_merge_kernel, (unsigned)B, kThreads, (size_t)beams * n * 8, (cudaStream_t)stream, m);
    return e == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}
