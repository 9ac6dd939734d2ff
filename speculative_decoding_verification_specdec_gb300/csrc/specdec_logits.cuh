/*
 * specdec_logits.cuh -- what the operators on rows of logits beside the verify share: a row as 16-byte vectors whatever
 * its alignment, mask bits, keys that order floats, and the folds of a softmax's sum.
 */
#ifndef SPECDEC_LOGITS_CUH
#define SPECDEC_LOGITS_CUH

#include "specdec_rows.cuh"
#include "specdec_tensor.cuh"

namespace specdec {

constexpr int32_t kMaxVocab = 1 << 30;             // element numbers within a row stay in 32 bits

template <typename T> constexpr int kPer = 16 / (int)sizeof(T);        // elements of a vector

template <typename T> __device__ __forceinline__ T neg_inf() { return from_float<T>(-INFINITY); }

// A row's elements lie in vectors on the 16-byte grid: vector v holds elements v * per - lead .. + per - 1, of which the
// first and the last may lie outside the row. Those vectors are taken element by element, so that nothing outside the row is touched.
template <typename T> struct Row {
    const T* p;
    int32_t V, lead, vectors;
    __device__ __forceinline__ Row(const T* row, int32_t vocab) : p(row), V(vocab)
    {
        lead = (int32_t)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
        vectors = (lead + vocab + kPer<T> - 1) / kPer<T>;
    }
    __device__ __forceinline__ int32_t first(int32_t v) const { return v * kPer<T> - lead; }
    __device__ __forceinline__ bool whole(int32_t at) const { return at >= 0 && at + kPer<T> <= V; }
};

// The most vectors that a row of V elements takes, wherever it starts.
template <typename T> inline __host__ __device__ int32_t most_vectors(int32_t V) { return (V + 2 * kPer<T> - 2) / kPer<T>; }

// 16 bytes that are read once: not kept in L1.
__device__ __forceinline__ uint4 load_once(const void* p)
{
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

// Vector v, -infinity for what lies outside the row (v may lie behind it as a whole).
template <typename T> __device__ __forceinline__ void load_vector(const Row<T>& row, int32_t v, Raw<T, kPer<T>>& x)
{
    const int32_t at = row.first(v);
    if (row.whole(at)) {
        *reinterpret_cast<uint4*>(x.e) = load_once(row.p + at);
    } else {
#pragma unroll
        for (int i = 0; i < kPer<T>; ++i) x.e[i] = at + i >= 0 && at + i < row.V ? row.p[at + i] : neg_inf<T>();
    }
}

// Mask bits of vector v's elements, bit i for element i; bits outside the row are 0. words: the row's ceil(V / 32) words.
template <typename T> __device__ __forceinline__ uint32_t vector_bits(const Row<T>& row, const int32_t* words, int32_t v)
{
    const int32_t at = row.first(v), lo = max(at, 0), hi = min(at + kPer<T>, row.V) - 1;
    if (hi < lo) return 0;
    const uint32_t a = (uint32_t)words[lo >> 5], b = (lo >> 5) == (hi >> 5) ? 0u : (uint32_t)words[hi >> 5];
    const uint32_t bits = __funnelshift_r(a, b, lo & 31) & ((2u << (hi - lo)) - 1u);
    return bits << (lo - at);
}

template <typename T> __device__ __forceinline__ void apply_bits(Raw<T, kPer<T>>& x, uint32_t bits)
{
#pragma unroll
    for (int i = 0; i < kPer<T>; ++i)
        if (!(bits >> i & 1)) x.e[i] = neg_inf<T>();
}

// An unsigned number that orders floats as they are ordered; 0 for what is never chosen (-infinity and NaN). -0 and 0 are equal.
__device__ __forceinline__ uint32_t order_key(float x)
{
    if (!(x > -INFINITY)) return 0;
    const int32_t b = __float_as_int(x + 0.f);
    return (uint32_t)b ^ (b < 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
// Bits of a key under which those of T's values are all alike.
template <typename T> constexpr int kKeyLow = 0;
template <> constexpr int kKeyLow<__nv_bfloat16> = 16;
template <> constexpr int kKeyLow<__half> = 13;

// The temperatures taken: 2^(z log2(e) / t) then vanishes for the lowest fp32 number, and z / t of ordinary logits is finite.
inline bool usable_temperature(double t) { return t >= 1e-4 && t <= 1e4; }
inline double scale_of(double temperature) { return 1.4426950408889634073599 / temperature; }

// A sum of exponentials is S 2^ref with ref a whole number: references differ by whole numbers, so that sums are joined by
// exact powers of two. An empty sum has ref = -infinity, S = 0. (The lowest fp32 numbers, where masks put them, have a product
// beyond fp32: the reference stays finite, and their terms are 0.)
__device__ __forceinline__ float whole_reference(float m, float c) { return ceilf(fmaxf(m * c, -3.0e38f)); }

// 2^(a - b) for references a <= b: exact, and 0 where a is an empty sum's or the power is under fp32's normal numbers.
__device__ __forceinline__ float reference_step(float a, float b)
{
    const int d = (int)fmaxf(a - b, -127.f);
    return d == -127 ? 0.f : __int_as_float((127 + d) << 23);
}

// A number as the sum of two floats, |lo| at most half an ulp of hi: 2^-46 or so from additions and products by fp32's own
// instructions. This part has few 64-bit ones: a warp's takes an SM some 16 clocks.
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two two_ordered(float a, float b)         // |a| >= |b|, or a = 0
{
    const float s = __fadd_rn(a, b);
    return Two{s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Two two_sum(float a, float b)
{
    const float s = __fadd_rn(a, b), c = __fsub_rn(s, a);
    return Two{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, c)), __fsub_rn(b, c))};
}
__device__ __forceinline__ Two two_product(float a, float b)
{
    const float p = __fmul_rn(a, b);
    return Two{p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ Two operator+(Two a, Two b)
{
    const Two s = two_sum(a.hi, b.hi);
    return two_ordered(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ Two operator-(Two a) { return Two{-a.hi, -a.lo}; }
__device__ __forceinline__ Two operator-(Two a, Two b) { return a + -b; }
__device__ __forceinline__ Two operator*(Two a, Two b)
{
    const Two p = two_product(a.hi, b.hi);
    return two_ordered(p.hi, __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, p.lo)));
}
__device__ __forceinline__ Two times(Two a, float power_of_two) { return Two{a.hi * power_of_two, a.lo * power_of_two}; }
// A constant, to 48 bits.
#define SPECDEC_TWO(x) (::specdec::Two{(float)(x), (float)((x) - (double)(float)(x))})
constexpr double kLn2 = 0.69314718055994530941723, kLog2e = 1.4426950408889634073599;

// 2^y to 2^-42: y = k + f with k whole, v = f ln 2 / 8, exp(v) by its series (|v| < 0.044: from the fourth power on in fp32),
// squared three times. 0 below 2^-125.
__device__ __forceinline__ Two exp2_two(Two y)
{
    if (!(y.hi > -125.f)) return Two{y.hi != y.hi ? y.hi : 0.f, 0.f};
    const float k = rintf(y.hi);
    const Two v = two_ordered(__fsub_rn(y.hi, k), y.lo) * SPECDEC_TWO(kLn2 / 8.0), square = v * v;
    const float x = v.hi, fourth = square.hi * square.hi;
    const float series = fmaf(fmaf(fmaf(x, 1.f / 5040.f, 1.f / 720.f), x, 1.f / 120.f), x, 1.f / 24.f) * fourth;
    Two e = square * (v * SPECDEC_TWO(1.0 / 6.0) + Two{0.5f, 0.f}) + v + Two{series, 0.f};
    e = Two{1.f, 0.f} + e;
    e = e * e;
    e = e * e;
    e = e * e;
    return times(times(e, __int_as_float((127 + (int)k / 2) << 23)), __int_as_float((127 + (int)k - (int)k / 2) << 23));
}
// log2 x, x > 0 and no subnormal: fp32's, put right by one step of Newton's method (-infinity for 0; infinity and NaN stay).
__device__ __forceinline__ Two log2_two(Two x)
{
    if (!(x.hi > 0.f) || x.hi == INFINITY) return Two{x.hi == 0.f ? -INFINITY : x.hi, 0.f};
    const int e = (__float_as_int(x.hi) >> 23) - 127;
    const float down = __int_as_float((127 - e / 2) << 23), more = __int_as_float((127 - (e - e / 2)) << 23);
    const Two m = times(times(x, down), more);
    const float y = log2f(m.hi);
    const Two d = m * exp2_two(Two{-y, 0.f}) + Two{-1.f, 0.f};
    return two_sum((float)e, y) + d * SPECDEC_TWO(kLog2e) + Two{-0.5f * (float)kLog2e * d.hi * d.hi, 0.f};
}
__device__ __forceinline__ Two shuffle_xor(Two x, int o)
{
    return Two{__shfl_xor_sync(0xffffffffu, x.hi, o), __shfl_xor_sync(0xffffffffu, x.lo, o)};
}
__device__ __forceinline__ Two reciprocal(Two x)
{
    const float r = 1.f / x.hi;
    return Two{r, 0.f} + (Two{1.f, 0.f} - x * Two{r, 0.f}) * Two{r, 0.f};
}
// The sum of one number a lane, the same in every lane.
__device__ __forceinline__ Two warp_sum(Two x)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) x = x + shuffle_xor(x, o);
    return x;
}

// Two fp32 numbers in a register pair: one instruction adds or multiplies both.
typedef unsigned long long Pair;
__device__ __forceinline__ Pair pair_of(float x, float y)
{
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
    return p;
}
__device__ __forceinline__ float2 both(Pair p)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
    return f;
}
__device__ __forceinline__ Pair fma_2(Pair a, Pair b, Pair c)
{
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ Pair add_2(Pair a, Pair b)
{
    Pair d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Pair mul_2(Pair a, Pair b)
{
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Pair exp2_2(Pair a)
{
    const float2 f = both(a);
    return pair_of(exp2_fast(f.x), exp2_fast(f.y));
}

// Elements 2 i and 2 i + 1 of a vector.
__device__ __forceinline__ Pair elements(const Raw<float, 4>& x, int i) { return pair_of(x.e[2 * i], x.e[2 * i + 1]); }
__device__ __forceinline__ Pair elements(const Raw<__nv_bfloat16, 8>& x, int i)
{
    const uint32_t w = reinterpret_cast<const uint32_t*>(x.e)[i];
    return pair_of(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ Pair elements(const Raw<__half, 8>& x, int i)
{
    const float2 f = __half22float2(reinterpret_cast<const __half2*>(x.e)[i]);
    return pair_of(f.x, f.y);
}
__device__ __forceinline__ void put_elements(Raw<float, 4>& x, int i, Pair p)
{
    const float2 f = both(p);
    x.e[2 * i] = f.x;
    x.e[2 * i + 1] = f.y;
}
__device__ __forceinline__ void put_elements(Raw<__nv_bfloat16, 8>& x, int i, Pair p)
{
    const float2 f = both(p);
    reinterpret_cast<__nv_bfloat162*>(x.e)[i] = __floats2bfloat162_rn(f.x, f.y);
}
__device__ __forceinline__ void put_elements(Raw<__half, 8>& x, int i, Pair p)
{
    const float2 f = both(p);
    reinterpret_cast<__half2*>(x.e)[i] = __floats2half2_rn(f.x, f.y);
}

// Joins the lanes' sums; every lane gets the warp's.
__device__ __forceinline__ void warp_join(float& ref, float& S)
{
    float top = ref;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    S *= reference_step(ref, top);                     // (NaN stays)
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
    ref = top;
}

// Maxima of vectors as they are kept on the way: a float, or a pair of 16-bit numbers whose larger one counts. NaN is passed over.
template <typename T> struct Maximum;
template <> struct Maximum<float> {
    float x;
    __device__ __forceinline__ static Maximum of(const Raw<float, 4>& v) { return {fmaxf(fmaxf(v.e[0], v.e[1]), fmaxf(v.e[2], v.e[3]))}; }
    __device__ __forceinline__ friend Maximum larger(Maximum a, Maximum b) { return {fmaxf(a.x, b.x)}; }
    __device__ __forceinline__ float value() const { return x; }
    __device__ __forceinline__ uint32_t bits() const { return __float_as_uint(x); }
    __device__ __forceinline__ static Maximum from(uint32_t b) { return {__uint_as_float(b)}; }
};
template <> struct Maximum<__nv_bfloat16> {
    uint32_t x;
    __device__ __forceinline__ friend Maximum larger(Maximum a, Maximum b)
    {
        Maximum m;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(m.x) : "r"(a.x), "r"(b.x));
        return m;
    }
    __device__ __forceinline__ static Maximum of(const Raw<__nv_bfloat16, 8>& v)
    {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(v.e);
        return larger(larger(Maximum{p[0]}, Maximum{p[1]}), larger(Maximum{p[2]}, Maximum{p[3]}));
    }
    __device__ __forceinline__ float value() const { return fmaxf(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)); }
    __device__ __forceinline__ uint32_t bits() const { return x; }
    __device__ __forceinline__ static Maximum from(uint32_t b) { return {b}; }
};
template <> struct Maximum<__half> {
    uint32_t x;
    __device__ __forceinline__ friend Maximum larger(Maximum a, Maximum b)
    {
        Maximum m;
        asm("max.f16x2 %0, %1, %2;" : "=r"(m.x) : "r"(a.x), "r"(b.x));
        return m;
    }
    __device__ __forceinline__ static Maximum of(const Raw<__half, 8>& v)
    {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(v.e);
        return larger(larger(Maximum{p[0]}, Maximum{p[1]}), larger(Maximum{p[2]}, Maximum{p[3]}));
    }
    __device__ __forceinline__ float value() const
    {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
        return fmaxf(f.x, f.y);
    }
    __device__ __forceinline__ uint32_t bits() const { return x; }
    __device__ __forceinline__ static Maximum from(uint32_t b) { return {b}; }
};

inline specdec_status_t check_logits(const void* logits, specdec_dtype_t dtype, int64_t rows, int32_t V, int64_t row_stride)
{
    if (!is_float_type(dtype)) return SPECDEC_ERR_UNSUPPORTED;
    if (rows < 0 || V < 1 || row_stride < 0) return SPECDEC_ERR_INVALID_ARG;
    if (V > kMaxVocab) return SPECDEC_ERR_UNSUPPORTED;
    if (rows == 0) return SPECDEC_OK;
    if (!logits || !aligned_to(logits, elem_bytes(dtype)) || (rows > 1 && row_stride < V)) return SPECDEC_ERR_INVALID_ARG;
    return SPECDEC_OK;
}

}  // namespace specdec

#endif  // SPECDEC_LOGITS_CUH
