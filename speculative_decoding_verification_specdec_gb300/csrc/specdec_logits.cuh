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
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
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
    const uint32_t a = (uint32_t)__ldg(words + (lo >> 5)), b = (lo >> 5) == (hi >> 5) ? 0u : (uint32_t)__ldg(words + (hi >> 5));
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

// 2^(a - b) for references a <= b: exact, and 0 where a is an empty sum's or the power is under the type's normal numbers.
__device__ __forceinline__ float reference_step(float a, float b)
{
    const int d = (int)fmaxf(a - b, -127.f);
    return d == -127 ? 0.f : __int_as_float((127 + d) << 23);
}
__device__ __forceinline__ double reference_step_64(float a, float b)
{
    const int d = (int)fmaxf(a - b, -1023.f);
    return d == -1023 ? 0.0 : __hiloint2double((1023 + d) << 20, 0);
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
