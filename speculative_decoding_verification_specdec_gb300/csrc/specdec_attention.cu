/*
 * specdec_attention.cu -- attention of a verify step's rows over the paged key-value cache for
 * GB300 (sm_103a); C-ABI entry points in include/specdec.h.
 *
 * Mathematics. The (k_b + 1) * G query rows that share one key-value head of request b are the N
 * columns of two products over a tile of 128 tokens (padded to N = 16, 32, 64, 96 or 128):
 *     S^T [128 tokens, N] = K Q^T          O^T [D, N] += V^T P^T,   P = exp2(c S - m)
 * with tokens (and head elements) as the 128 rows of tcgen05.mma: the work grows with the rows there
 * are, not with a row tile of 128, and the keys and values go from TMA's swizzled tiles into the
 * products as they lie (V^T is V read with its rows contiguous). The softmax is one pass: a column keeps
 * a reference m and the sum l of its weights; m moves only when a score exceeds it by more than 8
 * (in log2), so that the common tile needs no maximum across lanes, only a vote, and O^T, which
 * stays in tensor memory, is rarely rescaled. exp2(c S - m) <= 2^8 is exact to its rounding whatever m is.
 *
 * Work. The tiles of every (request, key-value head, row block) are numbered through the batch, each such
 * item preceded by kItem units for what it costs to start and end it; CTA i of P takes the i-th of P equal
 * runs of units, whatever the lengths and without the host knowing them. A CTA that holds only part of an item
 * writes (m, l, O) to its workspace slot, and specdec_paged_join_kernel joins the parts in the order of the CTAs.
 *
 * Warps, one CTA an SM: for the softmax 4 to each group of 16 or 32 columns (a lane quarter of tensor memory each),
 * and with at most 32 columns two such sets that take the tiles in turn, each with its own m, l and O; 4 that
 * widen e4m3 values to f16 tiles in shared memory (exact); two that feed TMA (keys, values); one for each
 * product; one that hands out the work and fetches Q (with many columns the scores' warp does that too).
 *
 * e4m3 keys go into the product as they lie, with Q taken apart into e4m3 pieces: widening them as well took
 * 427 us where this takes 355 (128 requests of up to 8000 tokens, 24 rows a key head).
 *
 * Bound by HBM: every visible key and value is read once per row block. Measured on one GB300: 64 requests of 1000
 * to 32000 bf16 tokens, up to 72 rows a key head (4.8 GB): 716 to 725 us by the card, 6.7 TB/s, 98 to 99 % of the measured copy rate.
 * Over e4m3 a tile is 32 KB and takes 0.84 us with 16 columns (the copy rate would be 0.74) and 1.07 with 32, by the
 * latency of the chain scores - weights - product of a tile; with short contexts an item costs 4 to 9 us to start
 * and end, most of it instructions that are run once an item and not in the instruction cache.
 */
#include <cuda.h>

#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstddef>
#include <type_traits>

#include "specdec_rows.cuh"
#include "specdec_tensor.cuh"

namespace {

using namespace specdec;

constexpr int kTile = 128;                               // tokens
constexpr int kNone = -100000, kUnset = 100000;          // no exponent: below, above every other
constexpr int kPartly = 4096;                            // added to the exponent of a token that some rows do not see
constexpr int kItem = 3;                                 // what starting and ending an item costs, in tiles
constexpr float kLazy = 8.f;                             // how far (log2) a score may pass the reference
constexpr uint32_t kWaitNs = 2000000000u;                // a wait's default limit
constexpr unsigned long long kDrainNs = 1000000000ull;   // more time for copies in flight before a CTA leaves
constexpr int kSmemBytes = 227 * 1024;
constexpr int kJoinThreads = 512;                        // of the join: four rows of 128 elements, or eight of 64

// An item that a CTA begins and others go on with: its first row, rows and first column's row, head, and the last CTA
// (below 0: none).
struct Split {
    int32_t row0, rows, first, head, last;
};

struct Args {
    const void* q;
    void* out;
    float* lse;
    int32_t rows, num_heads, group;
    int64_t q_row, q_head, out_row, out_head;
    specdec_kv_cache_t cache;
    const int32_t* block_table;
    int64_t block_stride;
    int32_t max_blocks;
    const int32_t *cached, *cu;
    int32_t B, max_k, window;
    float scale_log2;                                    // scale * log2(e)
    uint32_t* status;
    Split* split;                                        // [P]: the item that CTA i leaves to the next ones
    float* parts;                                        // [2 P] slots of N (D + 2) floats
    uint32_t wait_ns;
};

// ---------------------------------------------------------------- the batch's units

struct Request {
    int64_t cached;
    int32_t row0, rows, blocks;                          // first row, rows a key-value head, row blocks
    int32_t first_tile, tiles;
    uint32_t fault;
    __device__ __forceinline__ int64_t units(int heads) const { return tiles ? (int64_t)heads * blocks * (tiles + kItem) : 0; }
};

// Tokens that a request may have: its row of block_table, and what keeps token numbers and their tiles within 32 bits.
__host__ __device__ __forceinline__ int64_t most_tokens(int32_t max_blocks, int32_t page_size)
{
    const int64_t held = (int64_t)max_blocks * page_size, most = (int64_t)INT32_MAX - kTile;
    return held < most ? held : most;
}

template <int N> __device__ __noinline__ Request request_of(const Args& a, int b)
{
    Request r = {0, 0, 0, 0, 0, 0, 0};
    const int32_t c0 = __ldg(a.cu + b), k = __ldg(a.cu + b + 1) - c0;
    if (!rows_ok(a.cu, a.B, b, a.rows)) {
        r.fault = SPECDEC_ST_BAD_OFFSETS;
        return r;
    }
    r.row0 = c0 + b;
    r.cached = __ldg(a.cached + b);
    if (k > a.max_k) {
        r.fault = SPECDEC_ST_K_TOO_LARGE;
    } else if (r.cached < 0 || r.cached + k + 1 > most_tokens(a.max_blocks, a.cache.page_size)) {
        r.fault = SPECDEC_ST_BAD_LENGTH;
    } else {
        r.rows = (k + 1) * a.group;
        r.blocks = (r.rows + N - 1) / N;
        r.first_tile = a.window > 0 && r.cached >= a.window ? (int32_t)((r.cached - a.window + 1) / kTile) : 0;
        r.tiles = (int32_t)((r.cached + k + kTile) / kTile) - r.first_tile;
    }
    return r;
}

// The first unit of CTA i. With fewer units than CTAs the first ones take one each, so that no CTA between two
// parts of an item is without a part.
__device__ __noinline__ int64_t quotient(int64_t x, int64_t y)           // x, y >= 0; 32-bit division where it will do
{
    return (x | y) >> 32 ? x / y : (int64_t)((uint32_t)x / (uint32_t)y);
}
__device__ __forceinline__ int64_t cta_begin(int64_t units, int i, int P)
{
    const int64_t each = quotient(units, P), rest = units - each * P;
    return each * i + min((int64_t)i, rest);
}

// What a CTA does of one item: tiles [t0, t1), numbered in the request.
struct Task {
    int32_t b, h, block, t0, t1;                         // b < 0: no more
    int32_t begin, end;                                  // whether they hold the item's first tile, and its last
    int32_t row0, rows, cached;
    int64_t last_unit;                                   // of the whole item
};

// Walks a CTA's units item by item.
template <int N> struct Walker {
    const Args& a;
    int64_t u, u_end, base;
    int b;
    Request r;
    __device__ __forceinline__ Walker(const Args& a_, int64_t begin, int64_t end, int b0, int64_t base0)
        : a(a_), u(begin), u_end(end), base(base0), b(b0)
    {
        if (u < u_end) r = request_of<N>(a, b);
    }
    __device__ __forceinline__ bool next(Task& w)
    {
        do {
            if (!step(w)) return false;
        } while (w.t1 <= w.t0);
        return true;
    }
    __device__ __forceinline__ bool step(Task& w)
    {
        w.b = -1;
        if (u >= u_end) return false;
        const int H = a.cache.num_kv_heads;
#pragma unroll 1
        while (u >= base + r.units(H)) {
            base += r.units(H);
            r = request_of<N>(a, ++b);
        }
        const int per = r.tiles + kItem;
        const int64_t local = u - base, item = quotient(local, per);
        const int at = (int)(local - item * per), tile = max(at - kItem, 0);
        const int n = (int)min((int64_t)(per - at), u_end - u);
        u += n;
        w.b = b;
        w.h = (int)quotient(item, r.blocks);
        w.block = (int)(item - (int64_t)w.h * r.blocks);
        w.t0 = r.first_tile + tile;
        w.t1 = r.first_tile + at + n - kItem;            // (t0 or less: none of the item's tiles are the CTA's)
        w.begin = tile == 0;
        w.end = at + n == per;
        w.row0 = r.row0;
        w.rows = r.rows;
        w.cached = (int32_t)r.cached;
        w.last_unit = base + item * per + per - 1;
        return true;
    }
};

// Whether either of two packed values has all bits of its exponent set: one more there carries into the sign's place.
template <typename M> __device__ __forceinline__ uint32_t not_finite(uint32_t two)
{
    constexpr uint32_t kOne = std::is_same<M, __half>::value ? 0x04000400u : 0x00800080u;
    return ((two & 0x7fff7fffu) + kOne) & 0x80008000u;
}

// ln of the sum of a column's weights: log2's approximation is off by 2^-22 near a sum of one, else by two units in its
// own last place, and so of the size of the other roundings of a long sum
__device__ __forceinline__ float lse_of(bool any, float ref, float sum)
{
    return any ? (ref + __log2f(sum)) * 0.69314718055994531f : -INFINITY;
}

// ---------------------------------------------------------------- shapes

template <typename T_, bool kFp8_, int N_, int DB_> struct Shape {
    using T = T_;                                        // type of q and out
    using M = std::conditional_t<kFp8_, __half, T_>;     // type of the second product's operands
    static constexpr bool kFp8 = kFp8_;
    // e4m3 keys are multiplied by Q as e4m3 too, taken apart into pieces whose sum it is: four significant bits
    // each (and the sign of the rest), so two for bf16's eight and three for f16's eleven
    static constexpr int kPieces = std::is_same<T_, __nv_bfloat16>::value ? 2 : 3;
    static constexpr int N = N_, DB = DB_, DP = 64 * DB_;
    // softmax warps: kCol groups of NC columns, and for few columns two sets of them that take the tiles in turn
    static constexpr int kCol = N >= 64 ? N / 32 : 1, NC = N / kCol, kPar = N <= 32 ? 2 : 1, kGroups = kPar * kCol;
    static constexpr int kQ = N >= 96 && DB == 2 ? 1 : 2;                // Q buffers
    static constexpr int kSoftWarps = 4 * kGroups, kConvWarps = kFp8 ? 4 : 0;
    // With many columns, and over e4m3 from 32, the warp that issues the scores also fetches Q: one warp less leaves
    // the softmax's threads registers that are worth more than Q fetched ahead (bf16, 96 columns, 64 requests of up to
    // 32000 tokens: 739 against 795 us; e4m3, 32 columns, 128 requests of up to 8000: 314 against 349).
    static constexpr bool kOneWarp = N >= 96 || (kFp8_ && N >= 32);
    static constexpr int kProducer = kSoftWarps + kConvWarps, kScores = kProducer + 2, kValues = kProducer + 3,
                         kLoader = kOneWarp ? kScores : kProducer + 4, kWarps = kProducer + (kOneWarp ? 4 : 5);
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kAhead = kFp8 ? 4 : 2;                          // tiles that the copies look ahead
    // Tasks between the loader and the slowest role. The copies of a tile are issued once the tile kAhead further is
    // known, which may be as many tasks further, and the loader hands out a task only when the task kTasks before is
    // taken and, before it, fetches the Q of one that waits for the item two before to end: which needs the copies
    // of at most two items after that. kAhead + 4 tasks keep the two from waiting for one another.
    static constexpr int kTasks = 8;
    static_assert(kTasks >= kAhead + 4, "tasks ahead");
    static constexpr int kSlotBytes = kTile * DP * (kFp8 ? 1 : 2);
    static constexpr int kQBytes = N * DP * (kFp8 ? kPieces : 2), kPBytes = N * kTile * 2, kV16Bytes = kFp8 ? kTile * DP * 2 : 0;
    static constexpr int kMiscBytes = (kFp8 ? 16 : 13) * 1024;
    static constexpr int kRoom = kSmemBytes - 1024 - kMiscBytes - kQ * kQBytes - kPar * kPBytes - 2 * kV16Bytes;
    static constexpr int kSlots = kRoom / kSlotBytes > 12 ? 12 : kRoom / kSlotBytes;
    static constexpr int kKSlots = kSlots / 2, kVSlots = kSlots - kKSlots;
    // where things lie behind the 1024-byte boundary that the ring starts at (up to 1023 bytes behind the base)
    static constexpr int kV16At = kSlots * kSlotBytes, kQAt = kV16At + 2 * kV16Bytes, kPAt = kQAt + kQ * kQBytes,
                         kMiscAt = kPAt + kPar * kPBytes, kSmem = 1024 + kMiscAt + kMiscBytes;
    static_assert(kSmem <= kSmemBytes, "shared memory");
    static constexpr int kTmem = (kPar + 2) * N;                         // O, two S
    static constexpr int kTmemColumns = kTmem <= 64 ? 64 : kTmem <= 128 ? 128 : kTmem <= 256 ? 256 : 512;
    static constexpr int kSlotFloats = N * (DP + 2);
    static_assert(kKSlots + kAhead <= 12 && kVSlots + kAhead <= 12, "a tile's scales stay in their ring of 16 until it is done with");
    static_assert(kKSlots >= 2 && kTmem <= 512, "shape does not fit the SM");
};

template <typename S> struct Misc {
    uint64_t full[S::kSlots], empty[S::kSlots];
    uint64_t s_full[2], pv_done[2], p_full[2], done[2], q_full[2], q_empty[2], v16_full[2], drained;
    uint64_t task_full[S::kTasks], task_free[S::kTasks];
    Task task[S::kTasks];
    int64_t begin, end, base, units;
    int64_t warp_units[32];
    int first_b;
    int expired;
    uint32_t tmem;
    uint32_t poison[2][4];                               // tokens of a tile whose values are taken one by one
    alignas(16) float red[S::kPar][4][S::N];             // a column's value in each warp of its group
    alignas(16) float fac[S::kPar][S::N];
    float ref[S::kPar][S::N];
    int red_e[4 * S::kGroups], ref_e[S::kPar];
    alignas(16) int32_t last[2][S::N];                   // last token that a column sees (-1: no column)
    alignas(16) int2 place[2][S::N];                     // a column's row of q and out, and its query head (row -1: no column)
    alignas(16) int64_t out_at[2][S::N];                 // and where it lies in out
    alignas(16) float qscale[2][S::kFp8 ? S::N : 4];
    alignas(16) int32_t pages[2][8][8];                  // of keys and of values: page ids of the tiles looked ahead to
    alignas(16) uint8_t scales[2][S::kFp8 ? 16 : 1][kTile];              // and exponents of their e4m3 keys and values
    // E, the exponent that a group takes the values' scales by, and that which a token's must pass to raise it. E follows from
    // the scales alone, so that the groups of a tile agree on it, and from tokens that every row sees: one that some rows
    // do not see would cost these rows' weights their bits if its scale were far above theirs, so above E + 4 it is
    // added by hand (heavy). Until a tile holds a token that every row sees, E is the smallest scale so far and
    // lift_over below all. (Here and not in registers, where they cost spills: 314 us where 321 for 128 requests of up to
    // 8000 tokens, 24 rows a key head.)
    int scale_e[S::kGroups], lift_over[S::kGroups], red_low[4 * S::kGroups];
};

// ---------------------------------------------------------------- the kernel

template <typename S>
__global__ void __launch_bounds__(S::kThreads, 1)
specdec_paged_attention_kernel(const Args a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap)
{
    using T = typename S::T;
    using M = typename S::M;
    constexpr int N = S::N, NC = S::NC, DP = S::DP;
    extern __shared__ unsigned char raw[];
    unsigned char* const ring = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    unsigned char* const v16 = ring + S::kV16At;
    unsigned char* const qbuf = ring + S::kQAt;
    unsigned char* const pbuf = ring + S::kPAt;
    Misc<S>& ms = *reinterpret_cast<Misc<S>*>(ring + S::kMiscAt);
    static_assert(sizeof(Misc<S>) <= S::kMiscBytes, "misc");
    static_assert(offsetof(Misc<S>, last) % 16 == 0 && offsetof(Misc<S>, qscale) % 16 == 0 && offsetof(Misc<S>, scales) % 16 == 0 &&
                  offsetof(Misc<S>, pages) % 16 == 0 && offsetof(Misc<S>, fac) % 16 == 0, "8- and 16-byte accesses");
    static_assert(S::kSlotBytes % 1024 == 0 && S::kQBytes % 1024 == 0 && S::kPBytes % 1024 == 0, "swizzled tiles");

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, P = gridDim.x;
    const specdec_kv_cache_t& c = a.cache;
    const int H = c.num_kv_heads;
    volatile int* const expired = &ms.expired;
    auto bar = [](uint64_t& b) { return smem_u32(&b); };
    auto wait = [&](uint64_t& b, uint32_t parity) { return bar_wait(smem_u32(&b), parity & 1u, a.wait_ns, expired); };

    // ---- set-up: barriers, tensor memory, the CTA's units
    if (tid == 0) {
#pragma unroll 1
        for (int s = 0; s < S::kSlots; ++s) {
            bar_init(bar(ms.full[s]), 1);
            // given back by the product that read it; of e4m3 also by the softmax (the scales), values by the converters
            bar_init(bar(ms.empty[s]), !S::kFp8 ? 1 : s < S::kKSlots ? 1 + 4 * S::kCol : 4 + 4 * S::kCol);
        }
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            bar_init(bar(ms.s_full[i]), 1);
            bar_init(bar(ms.pv_done[i]), 1);
            bar_init(bar(ms.p_full[i]), 4 * S::kCol);
            bar_init(bar(ms.done[i]), S::kSoftWarps);
            bar_init(bar(ms.q_full[i]), 1);
            // given back by the scores' last product; a single buffer also by the softmax's warps, once they have seen it
            // full: else the loader could fill it twice before a late one looks, whose phase then never comes. (Of two
            // buffers the next filling waits for the item to be done.)
            bar_init(bar(ms.q_empty[i]), S::kQ == 1 ? 1 + S::kSoftWarps : 1);
            bar_init(bar(ms.v16_full[i]), 4);
        }
        for (int i = 0; i < S::kTasks; ++i) {
            bar_init(bar(ms.task_full[i]), 1);
            bar_init(bar(ms.task_free[i]), S::kThreads / 32);
        }
        bar_init(bar(ms.drained), 2);
        ms.expired = 0;
        if constexpr (S::kFp8)
            for (int i = 0; i < S::kGroups; ++i) ms.scale_e[i] = kUnset, ms.lift_over[i] = kNone;
        for (int i = 0; i < 8; ++i) ms.poison[i >> 2][i & 3] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == S::kScores) tmem_alloc(smem_u32(&ms.tmem), S::kTmemColumns);
    after_predecessor();
    {
        // every thread sums the units of consecutive requests, a scan over the threads places them
        const int per = (a.B + S::kThreads - 1) / S::kThreads, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
        int64_t mine = 0;
#pragma unroll 1
        for (int b = b0; b < b1; ++b) mine += request_of<N>(a, b).units(H);
        int64_t upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += x;
        }
        if (lane == 31) ms.warp_units[warp] = upto;
        __syncthreads();
        int64_t before = upto - mine, units = 0;
#pragma unroll 1
        for (int w = 0; w < S::kThreads / 32; ++w) {
            if (w < warp) before += ms.warp_units[w];
            units += ms.warp_units[w];
        }
        const int64_t begin = cta_begin(units, blockIdx.x, P);
        if (mine > 0 && begin >= before && begin < before + mine) {      // the loader walks on from here
            ms.first_b = b0;
            ms.base = before;
        }
        if (tid == 0) {
            ms.begin = begin;
            ms.end = cta_begin(units, blockIdx.x + 1, P);
            ms.units = units;
        }
    }
    tmem_before();
    __syncthreads();
    tmem_after();
    const uint32_t tmem = ms.tmem;
    const uint32_t t_o = tmem, t_s = tmem + S::kPar * N;
    // ring slot of a tile's keys, and of its values
    auto k_slot = [](uint32_t n) { return n % S::kKSlots; };
    auto v_slot = [](uint32_t n) { return S::kKSlots + n % S::kVSlots; };
    // The next task, copied out of the loader's ring; false: none is left (or a wait has expired).
    auto take = [&](uint32_t q, Task& w) {
        const int s = q % S::kTasks;
        const bool ok = __all_sync(0xffffffffu, wait(ms.task_full[s], q / S::kTasks));
        if (ok) {
            w = ms.task[s];
            __syncwarp();
            if (lane == 0) bar_arrive(bar(ms.task_free[s]));
        }
        return ok && w.b >= 0;
    };
    Task w;
    if (tid == 0) a.split[blockIdx.x].last = -1;         // this thread may fill it in below

    // ================================================================ the tasks, a few ahead; Q, its scales and its columns' places
    // (of the loader's warp, or the scores'; then(q) once Q is there)
    [[maybe_unused]] auto load_items = [&](auto then) {
        Walker<N> walk(a, ms.begin, ms.end, ms.first_b, ms.base);
        uint32_t sent = 0;
        bool more = true;
        auto send = [&]() {
            if (!more) return;
            Task x;
            more = walk.next(x);                         // (the last one says that no more come)
            const int s = sent % S::kTasks;
            if (sent >= (uint32_t)S::kTasks && !__all_sync(0xffffffffu, wait(ms.task_free[s], sent / S::kTasks - 1))) {
                more = false;
                return;
            }
            if (lane == 0) {
                ms.task[s] = x;
                bar_arrive(bar(ms.task_full[s]));
            }
            ++sent;
        };
#pragma unroll 1
        for (uint32_t i = 0;; ++i) {
            send();
            if (i + 1 < (uint32_t)S::kTasks - 1) continue;               // the first tasks before the first Q
            const uint32_t q = i + 2 - S::kTasks;
            if (!take(q, w)) break;
            const uint32_t qb = q % S::kQ, tb = q & 1;
            if (q >= 2) wait(ms.done[tb], (q >> 1) - 1);                 // the tables' last item is done with
            if (q >= (uint32_t)S::kQ) wait(ms.q_empty[qb], q / S::kQ - 1);
#pragma unroll 1
            for (int n = lane; n < N; n += 32) {
                const int r = w.block * N + n, j = r / a.group, g = r - j * a.group;
                const bool real = r < w.rows;
                const int2 at = real ? make_int2(w.row0 + j, w.h * a.group + g) : make_int2(-1, 0);
                ms.place[tb][n] = at;
                ms.out_at[tb][n] = real ? at.x * a.out_row + at.y * a.out_head : -1;
                ms.last[tb][n] = real ? w.cached + j : -1;
            }
            __syncwarp();
            unsigned char* const dst = qbuf + qb * S::kQBytes;
            constexpr int kChunks = N * (DP / 8) / 32;                   // of 16 bytes, a lane
            // chunk i of this lane: its column, its place in the head, and where it comes from (nullptr: zeros)
            auto column = [&](int i) { return (lane & 7) + 8 * ((lane + 32 * i) / DP); };
            auto piece = [&](int i) { return ((lane + 32 * i) >> 3) % (DP / 8); };
            auto source = [&](int i) -> const T* {
                const int2 at = ms.place[tb][column(i)];
                return at.x >= 0 && piece(i) * 8 < c.head_dim ? static_cast<const T*>(a.q) + at.x * a.q_row + at.y * a.q_head + piece(i) * 8 : nullptr;
            };
            auto target = [&](int i) { return dst + ((column(i) >> 3) * (DP / 8) + piece(i)) * 128 + (column(i) & 7) * 16; };
            if constexpr (!S::kFp8) {
#pragma unroll 4
                for (int i = 0; i < kChunks; ++i) {
                    const T* src = source(i);
                    async_copy_16(smem_u32(target(i)), src ? src : static_cast<const T*>(a.q), src ? 16 : 0);
                }
                async_copy_wait();
            } else {
                // Eight rows at a time: lanes of the same number modulo 8 hold a row, kRow chunks each; the next eight
                // rows are on their way while these are taken apart.
                // A power of two brings the row's largest magnitude to [128, 256): a piece is the nearest e4m3 number to
                // what the pieces before it leave, in all exact to 2^-10, e4m3's half step at its smallest, so to
                // 2^-17 of the row's largest element at worst. What is not finite becomes NaN.
                constexpr int kRow = DP / 32;
                auto read = [&](int base, uint4 (&v)[kRow]) {
#pragma unroll
                    for (int u = 0; u < kRow; ++u) {
                        const T* src = source(base + u);
                        v[u] = src ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0);
                    }
                };
                uint4 now[kRow], next[kRow];
                read(0, now);
#pragma unroll 1
                for (int base = 0; base < kChunks; base += kRow) {
                    if (base + kRow < kChunks) read(base + kRow, next);
                    float z[kRow][8], top = 0.f;
#pragma unroll
                    for (int u = 0; u < kRow; ++u) {
                        const T* y = reinterpret_cast<const T*>(&now[u]);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            z[u][k] = to_float<T>(y[k]);
                            top = fmaxf(top, fabsf(z[u][k]));            // (fmaxf passes over NaN)
                        }
                    }
                    if (__any_sync(0xffffffffu, top == INFINITY)) {
                        top = 0.f;
#pragma unroll
                        for (int u = 0; u < kRow; ++u)
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                if (fabsf(z[u][k]) == INFINITY) z[u][k] = NAN;
                                top = fmaxf(top, fabsf(z[u][k]));
                            }
                    }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                    const int n = column(base);
                    const int e = top > 0.f ? max((int)(__float_as_uint(top) >> 23) - 126, -100) : 8;
                    const float inv = __uint_as_float((uint32_t)(127 + 8 - e) << 23);
                    if (lane < 8) ms.qscale[tb][n] = __uint_as_float((uint32_t)(127 + e - 8) << 23);
#pragma unroll
                    for (int u = 0; u < kRow; ++u) {
                        const int at = piece(base + u);
                        unsigned char* const d = dst + ((n >> 3) * (DP / 16) + (at >> 1)) * 128 + (n & 7) * 16 + (at & 1) * 8;
#pragma unroll
                        for (int p = 0; p < S::kPieces; ++p) {
                            uint32_t two[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float scale = p == 0 ? inv : 1.f;
                                const float2 x = make_float2(z[u][2 * k] * scale, z[u][2 * k + 1] * scale);
                                two[k] = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
                                const float2 back = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two[k], __NV_E4M3)));
                                z[u][2 * k] = x.x - back.x;
                                z[u][2 * k + 1] = x.y - back.y;
                            }
                            *reinterpret_cast<uint2*>(d + p * N * DP) = make_uint2(two[0] | two[1] << 16, two[2] | two[3] << 16);
                        }
                    }
#pragma unroll
                    for (int u = 0; u < kRow; ++u) now[u] = next[u];
                }
            }
            fence_async();
            __syncwarp();
            if (lane == 0) bar_arrive(bar(ms.q_full[qb]));
            then(q);
        }
    };

    if (warp == S::kProducer || warp == S::kProducer + 1) {
        // ================================================================ keys (one warp) and values (the other) into the ring
        // (a page of 16 slots takes copies of 2 KB: one warp for both streams took 879 us where two take 739)
        const bool is_v = warp != S::kProducer;
        const int ps = c.page_size, bits = __ffs(ps) - 1, row_bits = min(bits, 7), rows = 1 << row_bits, pages = kTile >> row_bits;
        const CUtensorMap* const map = is_v ? &vmap : &kmap;
        const uint32_t slots = is_v ? S::kVSlots : S::kKSlots;
        // A tile on its way. Its page ids are on their way to shared memory while the two tiles before it are issued, an
        // e4m3 tile's scales (which need the ids) too, so its ids four tiles: a read that had to land in a register
        // would hold up each turn of the loop. Tasks follow one another without a break.
        struct Ahead {
            int first, used, h, slot0, b;                // its pages first .. used - 1 (used 0: no more tiles), head, ...
        };
        constexpr int kAhead = S::kAhead;
        uint32_t q = 0, n = 0, issued = 0;               // tasks so far, tiles, those whose copies were issued
        int t = 0, t_end = 0, len = 0;
        bool more = true;
        Ahead x[kAhead + 1];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) x[i] = {0, 0, 0, 0, 0};
#pragma unroll 1
        for (int k = 0;; ++k) {                          // looks at tile k, issues tile k - kAhead
            async_copy_wait_but_one();                   // what was under way two turns ago has landed
            __syncwarp();
            Ahead& ahead = x[kAhead];
            ahead = {0, 0, 0, 0, 0};
            if (t == t_end && more) {
                more = take(q++, w);
                t = w.t0;
                t_end = w.t1;
                len = w.cached + w.rows / a.group;
            }
            if (more) {
                const int32_t token0 = t * kTile;
                ahead.used = min(pages, (len - token0 + rows - 1) >> row_bits);
                ahead.first = a.window > 0 ? max(w.cached - a.window + 1 - token0, 0) >> row_bits : 0;   // (no row sees those before)
                ahead.h = w.h;
                ahead.b = w.b;
                ahead.slot0 = token0 & (ps - 1) & ~(rows - 1);
                if (lane < 8) {
                    int32_t* const to = &ms.pages[is_v][k & 7][lane];
                    if (lane >= ahead.first && lane < ahead.used)
                        async_copy_4(smem_u32(to), a.block_table + w.b * a.block_stride + ((token0 + (lane << row_bits)) >> bits));
                    else
                        *to = -1;
                }
                ++t;
            }
            if constexpr (S::kFp8) {
                const Ahead& y = x[2];                   // tile k - 2: 16 of its scales a lane (without a page the smallest: zeros raise no exponent)
                if (y.used > 0 && lane < 8) {
                    const int pg = ms.pages[is_v][(k - 2) & 7][(lane << 4) >> row_bits];
                    uint8_t* const to = &ms.scales[is_v][(k - 2) & 15][lane * 16];
                    if (pg >= 0 && pg < c.num_pages)
                        async_copy_16(smem_u32(to), (is_v ? c.v_exp : c.k_exp) + ((((int64_t)pg * H + y.h) << bits) + y.slot0 + ((lane << 4) & (rows - 1))), 16);
                    else
                        *reinterpret_cast<uint4*>(to) = make_uint4(0x01010101, 0x01010101, 0x01010101, 0x01010101);
                }
            }
            async_copy_commit();
            if (k >= kAhead) {
                const Ahead& x0 = x[0];
                if (x0.used == 0) break;
                const int page = lane < 8 ? ms.pages[is_v][n & 7][lane] : -1;
                const bool bad = lane >= x0.first && lane < x0.used && (page < 0 || page >= c.num_pages);
                if (bad && a.status) atomicOr(a.status + x0.b, SPECDEC_ST_BAD_PAGE);
                const int from = bad ? c.num_pages : page;       // past the end: the copy reads zeros
                const uint32_t s = is_v ? v_slot(n) : k_slot(n);
                if (n >= slots) wait(ms.empty[s], n / slots - 1);
                if (!__any_sync(0xffffffffu, *expired)) {
                    issued = n + 1;
                    const uint32_t fb = bar(ms.full[s]), dst = smem_u32(ring) + s * S::kSlotBytes;
                    __syncwarp();
                    if (elected()) bar_expect(fb, (x0.used - x0.first) * rows * DP * (S::kFp8 ? 1 : 2));
#pragma unroll 1
                    for (int p = x0.first; p < x0.used; ++p) {
                        const int pg = __shfl_sync(0xffffffffu, from, p);
                        if (elected()) {
                            if constexpr (S::kFp8) {
                                tma_load_4d(dst + p * rows * DP, map, fb, 0, x0.slot0, x0.h, pg);
                            } else {
#pragma unroll
                                for (int d = 0; d < S::DB; ++d)
                                    tma_load_4d(dst + d * (kTile * 128) + p * rows * 128, map, fb, d * 64, x0.slot0, x0.h, pg);
                            }
                        }
                        __syncwarp();
                    }
                }
                ++n;
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) x[i] = x[i + 1];
        }
        async_copy_wait();
        // nothing may still be on its way into shared memory when the CTA leaves
        __syncwarp();
        if (*expired && lane == 0) {
            const unsigned long long t0 = time_ns();
#pragma unroll 1
            for (uint32_t i = issued > slots ? issued - slots : 0; i < issued; ++i)
                while (!bar_test(bar(ms.full[is_v ? v_slot(i) : k_slot(i)]), (i / slots) & 1u) && time_ns() - t0 < kDrainNs) {}
        }
    } else if (warp == S::kScores) {
        // ================================================================ S^T = K Q^T
        // (the two products are issued by a warp each: what a warp does between its products, some hundred instructions
        // that wait for one another, is longer than the products of few columns)
        constexpr uint32_t ds = product(std::is_same<M, __nv_bfloat16>::value, 0, 128, N);
        const uint32_t ring0 = smem_u32(ring), q0 = smem_u32(qbuf);
        uint32_t n = 0;                                  // tiles of the CTA
        auto item = [&](uint32_t q, bool have_q) {
            const uint32_t qb = q % S::kQ;
            const uint64_t qo = operand(q0 + qb * S::kQBytes, 128, DP * (S::kFp8 ? 8 : 16), kNoSwizzle);
#pragma unroll 1
            for (int t = w.t0; t < w.t1; ++t, ++n) {
                const uint32_t slot = k_slot(n);
                bool ok = wait(ms.full[slot], n / S::kKSlots) && have_q;
                if (n >= 2) ok = wait(ms.p_full[n & 1], (n >> 1) - 1) && ok;             // the scores of tile n - 2 are read
                if (__all_sync(0xffffffffu, ok) && elected()) {
                    tmem_after();
                    const uint32_t d = t_s + (n & 1) * N;
                    if constexpr (S::kFp8) {
                        // 16 elements to 16 bytes of a row; the pieces of Q one after the other into the same sums
                        const uint64_t ko = operand(ring0 + slot * S::kSlotBytes, 0, DP * 8, DP == 128 ? kSwizzle128 : kSwizzle64);
#pragma unroll
                        for (int p = 0; p < S::kPieces; ++p)
#pragma unroll
                            for (int k = 0; k < DP / 32; ++k)
                                mma_ss_e4m3(d, ko + k * (32 >> 4), qo + p * (N * DP >> 4) + k * (256 >> 4), ds, p > 0 || k > 0);
                    } else {
                        const uint64_t ko = operand(ring0 + slot * S::kSlotBytes, 0, 1024, kSwizzle128);
#pragma unroll
                        for (int k = 0; k < DP / 16; ++k)
                            mma_ss(d, ko + (k / 4) * (kTile * 128 >> 4) + (k % 4) * (32 >> 4), qo + k * (256 >> 4), ds, k > 0);
                    }
                    mma_commit(bar(ms.s_full[n & 1]));
                    mma_commit(bar(ms.empty[slot]));
                    if (t + 1 == w.t1) mma_commit(bar(ms.q_empty[qb]));
                }
                __syncwarp();
            }
        };
        if constexpr (S::kOneWarp) {
            load_items([&](uint32_t q) { item(q, true); });
        } else {
            for (uint32_t q = 0; take(q, w); ++q) item(q, wait(ms.q_full[q % S::kQ], q / S::kQ));
        }
    } else if (warp == S::kValues) {
        // ================================================================ O^T += V^T P^T
        constexpr uint32_t dv = product(std::is_same<M, __nv_bfloat16>::value, 1, 128, N);
        const uint32_t ring0 = smem_u32(ring), p0 = smem_u32(pbuf), v0 = smem_u32(v16);
        // one block of 64 elements (DB = 1): the rows 64 .. 127 read the block again and are not used
        constexpr uint32_t lead = S::DB == 2 ? kTile * 128 : 0;
        uint32_t n = 0;
        for (uint32_t q = 0; take(q, w); ++q) {
            const bool o_free = q == 0 || wait(ms.done[(q - 1) & 1], (q - 1) >> 1);
#pragma unroll 1
            for (int t = w.t0; t < w.t1; ++t, ++n) {
                const uint32_t slot = v_slot(n);
                bool ok = S::kFp8 ? wait(ms.v16_full[n & 1], n >> 1) : wait(ms.full[slot], n / S::kVSlots);
                ok = wait(ms.p_full[n & 1], n >> 1) && ok && o_free;
                if (__all_sync(0xffffffffu, ok) && elected()) {
                    tmem_after();
                    const uint32_t acc = t_o + n % S::kPar * N;
                    const uint64_t vo = operand(S::kFp8 ? v0 + (n & 1) * S::kV16Bytes : ring0 + slot * S::kSlotBytes, lead, 1024, kSwizzle128);
                    const uint64_t po = operand(p0 + n % S::kPar * S::kPBytes, 128, 2048, kNoSwizzle);
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        mma_ss(acc, vo + k * (2048 >> 4), po + k * (256 >> 4), dv, t - w.t0 >= S::kPar || k > 0);
                    mma_commit(bar(ms.pv_done[n & 1]));
                    if constexpr (!S::kFp8) mma_commit(bar(ms.empty[slot]));
                }
                __syncwarp();
            }
        }
    } else if (!S::kOneWarp && warp == S::kLoader) {
        load_items([](uint32_t) {});
    } else if (S::kFp8 && warp >= S::kSoftWarps) {
        // ================================================================ e4m3 values -> f16 (exact), a token a thread
        const int row = tid & 127;
        uint32_t n = 0;
        for (uint32_t q = 0; take(q, w); ++q) {
#pragma unroll 1
            for (int t = w.t0; t < w.t1; ++t, ++n) {
                const uint32_t slot = v_slot(n);
                wait(ms.full[slot], n / S::kVSlots);
                const unsigned char* const src = ring + slot * S::kSlotBytes + row * DP;
                uint4 x[DP / 16];                        // 16 codes each
#pragma unroll
                for (int ch = 0; ch < DP / 16; ++ch)
                    x[ch] = *reinterpret_cast<const uint4*>(src + (DP == 128 ? ch ^ (row & 7) : ch ^ ((row >> 1) & 3)) * 16);
                __syncwarp();
                if (lane == 0) bar_arrive(bar(ms.empty[slot]));
                if (n >= 2) wait(ms.pv_done[n & 1], (n >> 1) - 1);       // the product of tile n - 2 has read the buffer
                // the layout of a 16-bit tile of TMA's
                unsigned char* const dst = v16 + (n & 1) * S::kV16Bytes + row * 128;
#pragma unroll
                for (int ch = 0; ch < DP / 16; ++ch) {
                    const uint32_t codes[4] = {x[ch].x, x[ch].y, x[ch].z, x[ch].w};
                    uint32_t r[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
                            : "=r"(r[2 * k]), "=r"(r[2 * k + 1]) : "r"(codes[k]));
                    unsigned char* const d = dst + (ch / 4) * (kTile * 128);
                    *reinterpret_cast<uint4*>(d + ((2 * (ch % 4)) ^ (row & 7)) * 16) = make_uint4(r[0], r[1], r[2], r[3]);
                    *reinterpret_cast<uint4*>(d + ((2 * (ch % 4) + 1) ^ (row & 7)) * 16) = make_uint4(r[4], r[5], r[6], r[7]);
                }
                fence_async();
                __syncwarp();
                if (lane == 0) bar_arrive(bar(ms.v16_full[n & 1]));
            }
        }
    } else {
        // ================================================================ softmax
        const int wq = warp & 3, gt = tid & 127, grp = warp >> 2;        // lane quarter, thread of the group, group:
        const int par = grp / S::kCol, cg = grp % S::kCol;               // which tiles, which columns
        const int col0 = cg * NC, id = 1 + grp, id_par = 9 + par;        // barriers of the group, of the tile's groups
        constexpr int kParThreads = 128 * S::kCol;
        const int tq = lane >> 2, cq = 2 * (lane & 3);                   // token and column within an 8 x 8 matrix
        const uint32_t quarter = (uint32_t)wq << 21;                     // lane 32 wq
        uint32_t n = 0;
        for (uint32_t q = 0;; ++q) {
            // (all of the softmax's threads go on, or none)
            if (barrier_or(7, 128 * S::kGroups, !take(q, w))) break;
            const uint32_t tb = q & 1;
            wait(ms.q_full[q % S::kQ], q / S::kQ);
            if constexpr (S::kQ == 1) {
                __syncwarp();
                if (lane == 0) bar_arrive(bar(ms.q_empty[0]));
            }
            const int row_first = w.block * N, row_last = min(row_first + N, w.rows) - 1;
            const int32_t seen_all = w.cached + row_first / a.group, seen_any = w.cached + row_last / a.group;
            const int32_t from_all = a.window > 0 ? seen_any - a.window + 1 : 0, from_any = a.window > 0 ? seen_all - a.window + 1 : 0;
            float m[NC / 4], l[NC / 4];
#pragma unroll
            for (int i = 0; i < NC / 4; ++i) m[i] = -FLT_MAX, l[i] = 0.f;
            // One tile; kMasked: it holds a token that some row does not see.
            auto tile = [&](auto masked, const int t) {
                constexpr bool kMasked = decltype(masked)::value;
                const int32_t token0 = t * kTile;
                [[maybe_unused]] const uint32_t ks = k_slot(n), vs = v_slot(n);
                const uint32_t acc = t_o + par * N + quarter + col0;
                // the product before this one that reads P's buffer and adds to O
                auto last_product = [&]() {
                    if (t - S::kPar >= w.t0) wait(ms.pv_done[(n - S::kPar) & 1], (n - S::kPar) >> 1);
                };
                [[maybe_unused]] float kscale[4];
                [[maybe_unused]] int ve[4];
                if constexpr (S::kFp8) {
                    wait(ms.full[ks], n / S::kKSlots);
                    wait(ms.full[vs], n / S::kVSlots);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tok = 32 * wq + 8 * i + tq;
                        kscale[i] = exp_value(ms.scales[0][n & 15][tok]) * a.scale_log2;
                        ve[i] = (int)ms.scales[1][n & 15][tok] - 127;
                        // a token that no row sees may hold anything
                        if constexpr (kMasked) {
                            if (token0 + tok > seen_any || token0 + tok < from_any) ve[i] = kNone;
                            else if (token0 + tok > seen_all || token0 + tok < from_all) ve[i] += kPartly;
                        }
                    }
                    __syncwarp();
                    if (lane == 0) {                                     // the scales are read: the slots may go
                        bar_arrive(bar(ms.empty[ks]));
                        bar_arrive(bar(ms.empty[vs]));
                    }
                }
                // the exponent by which token i may raise E; that which it has; whether one is heavy
                [[maybe_unused]] auto lift = [&](int i) { return ve[i] >= 128 ? kNone : ve[i]; };
                [[maybe_unused]] auto own = [&](int i) { return kMasked && ve[i] > kPartly - 200 ? ve[i] - kPartly : ve[i]; };
                [[maybe_unused]] auto heavy = [&](int e) { return kMasked && e > ms.scale_e[grp] + 4 && e < 128; };
                wait(ms.s_full[n & 1], n >> 1);
                tmem_after();
                const uint32_t s_at = t_s + (n & 1) * N + quarter + col0;
                float x[2][NC / 8][4];
                auto fetch = [&]() {
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                        for (int r = 0; r < NC / 8; r += 2)
                            tmem_ld_16x16(s_at + ((uint32_t)hf << 20) + r * 8, x[hf][r], x[hf][r + 1]);
                    tmem_wait_ld();
                };
                // f(score, its scale to log2 units, whether its row sees its token, its column's number)
                auto each = [&](auto f) {
#pragma unroll
                    for (int r = 0; r < NC / 8; ++r) {
                        float2 qs = make_float2(1.f, 1.f);
                        if constexpr (S::kFp8) qs = *reinterpret_cast<const float2*>(&ms.qscale[tb][col0 + 8 * r + cq]);
                        int2 last = make_int2(0, 0);
                        if constexpr (kMasked) {
                            // in the tile's own numbering of this thread's tokens
                            last = *reinterpret_cast<const int2*>(&ms.last[tb][col0 + 8 * r + cq]);
                            last.x -= token0 + 32 * wq + tq;
                            last.y -= token0 + 32 * wq + tq;
                        }
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                [[maybe_unused]] const int i = 2 * hf + (e >> 1);
                                float scale = a.scale_log2;
                                if constexpr (S::kFp8) scale = kscale[i];
                                if constexpr (S::kFp8) scale *= (e & 1) ? qs.y : qs.x;
                                bool seen = true;
                                if constexpr (kMasked) {
                                    const int32_t lt = (e & 1) ? last.y : last.x;
                                    // (a difference that wraps, under a window next to 2^31, has lt < 0 and so no say)
                                    seen = 8 * i <= lt && (a.window == 0 || 8 * i > (int32_t)((uint32_t)lt - (uint32_t)a.window));
                                }
                                f(x[hf][r][e], scale, seen, 2 * r + (e & 1));
                            }
                    }
                };
                fetch();
                float over = -INFINITY;
                each([&](float& z, float scale, bool seen, int ci) {
                    z = seen ? fmaf(z, scale, -m[ci]) : -INFINITY;
                    over = fmaxf(over, z);
                });
                bool move = over > kLazy;
                if constexpr (S::kFp8) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        move = move || lift(i) > ms.lift_over[grp] ||
                               (kMasked && ms.lift_over[grp] == kNone && own(i) > kNone && own(i) < min(ms.scale_e[grp], 128));
                }
                if (barrier_or(id, 128, move)) {
                    // the references move to the columns' maxima so far, and E to the values' largest exponent if one passes it
                    fetch();
                    float top[NC / 4];
#pragma unroll
                    for (int i = 0; i < NC / 4; ++i) top[i] = -INFINITY;
                    each([&](float& z, float scale, bool seen, int ci) {
                        z = seen ? z * scale : -INFINITY;
                        top[ci] = fmaxf(top[ci], z);
                    });
#pragma unroll
                    for (int i = 0; i < NC / 4; ++i) {
#pragma unroll
                        for (int off = 4; off <= 16; off <<= 1) top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], off));
                    }
                    if (tq == 0) {
#pragma unroll
                        for (int i = 0; i < NC / 4; ++i) ms.red[par][wq][col0 + 8 * (i >> 1) + cq + (i & 1)] = top[i];
                    }
                    if constexpr (S::kFp8) {
                        int et = kNone, low = kUnset;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            et = max(et, lift(i));
                            if (kMasked && own(i) > kNone && own(i) < 128) low = min(low, own(i));
                        }
                        et = __reduce_max_sync(0xffffffffu, et);
                        if constexpr (kMasked) low = __reduce_min_sync(0xffffffffu, low);
                        if (lane == 0) {
                            ms.red_e[4 * grp + wq] = et;
                            if constexpr (kMasked) ms.red_low[4 * grp + wq] = low;
                        }
                    }
                    barrier_sync(id, 128);
                    float e_fac = 1.f;
                    if constexpr (S::kFp8) {
                        const int E = ms.scale_e[grp], lift_over = ms.lift_over[grp];
                        int et = kNone, low = E;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            et = max(et, ms.red_e[4 * grp + i]);
                            if constexpr (kMasked) low = min(low, ms.red_low[4 * grp + i]);
                        }
                        const bool firm = et > lift_over;
                        int to = E;
                        if (firm) to = max(et, -126);
                        else if (kMasked && lift_over == kNone) to = max(low, -126);
                        if (to != E) {
                            const int d = min(E - to, 127);
                            e_fac = E == kUnset || d < -126 ? 0.f : __uint_as_float((uint32_t)(127 + d) << 23);
                        }
                        barrier_sync(id, 128);
                        if (gt == 0) {
                            ms.scale_e[grp] = to;
                            if (firm) ms.lift_over[grp] = to + 4;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < NC / 4; ++i) {
                        const int col = col0 + 8 * (i >> 1) + cq + (i & 1);
                        const float now = fmaxf(fmaxf(fmaxf(ms.red[par][0][col], ms.red[par][1][col]), fmaxf(ms.red[par][2][col], ms.red[par][3][col])), m[i]);
                        const float f = exp2_fast(m[i] - now);
                        l[i] *= f;
                        m[i] = now;
                        if (wq == 0 && tq == 0) ms.fac[par][col] = f * e_fac;
                    }
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                        for (int r = 0; r < NC / 8; ++r)
#pragma unroll
                            for (int e = 0; e < 4; ++e) x[hf][r][e] -= m[2 * r + (e & 1)];
                    barrier_sync(id, 128);
                    if (t - S::kPar >= w.t0) {
                        // O^T: this thread's lane is an element of the head, its columns the group's
                        last_product();
                        tmem_after();
#pragma unroll 1
                        for (int i = 0; i < NC; i += 16) {
                            float o[16];
                            uint32_t r[16];
                            tmem_ld_32x16(acc + i, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k) r[k] = __float_as_uint(o[k] * ms.fac[par][col0 + i + k]);
                            tmem_st_32x16(acc + i, r);
                        }
                        tmem_wait_st();
                    }
                }
                // weights, their sums, and P^T as the second product takes it: 8 x 8 blocks of 128 bytes
                last_product();
                unsigned char* const pt = pbuf + par * S::kPBytes;
                [[maybe_unused]] float vw[4];
                if constexpr (S::kFp8) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int e = own(i), de = e - ms.scale_e[grp];
                        vw[i] = e >= 128 ? __int_as_float(0x7fffffff) : heavy(e) ? 1.f : de < -126 ? 0.f : __uint_as_float((uint32_t)(127 + de) << 23);
                    }
                }
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int r = 0; r < NC / 8; r += 2) {
                        uint32_t packed[4];
#pragma unroll
                        for (int rr = 0; rr < 2; ++rr)
#pragma unroll
                            for (int s = 0; s < 2; ++s) {
                                float p0 = exp2_fast(x[hf][r + rr][2 * s]), p1 = exp2_fast(x[hf][r + rr][2 * s + 1]);
                                l[2 * (r + rr)] += p0;
                                l[2 * (r + rr) + 1] += p1;
                                if constexpr (S::kFp8) {
                                    const float v = vw[2 * hf + s];
                                    // (a scale that is no number stays out of the rows that do not see its token)
                                    p0 = kMasked && p0 == 0.f ? 0.f : p0 * v;
                                    p1 = kMasked && p1 == 0.f ? 0.f : p1 * v;
                                }
                                if constexpr (std::is_same<M, __half>::value) {
                                    const __half2 h2 = __floats2half2_rn(p0, p1);
                                    packed[2 * rr + s] = *reinterpret_cast<const uint32_t*>(&h2);
                                } else {
                                    const __nv_bfloat162 h2 = __floats2bfloat162_rn(p0, p1);
                                    packed[2 * rr + s] = *reinterpret_cast<const uint32_t*>(&h2);
                                }
                            }
                        // matrices (r, tokens 0-7), (r, tokens 8-15), (r + 1, ..), (r + 1, ..) of this half
                        const int mi = lane >> 3, col_group = col0 / 8 + r + (mi >> 1), token_group = 4 * wq + 2 * hf + (mi & 1);
                        store_matrices_t(smem_u32(pt) + (col_group * 16 + token_group) * 128 + (lane & 7) * 16, packed[0], packed[1],
                                         packed[2], packed[3]);
                    }
                bool poisoned = false;
                uint32_t* const pz = ms.poison[n & 1];
                if constexpr (kMasked) {
                    // values of tokens that no row sees become zeros (a weight of zero times NaN is NaN); those that some
                    // rows see and others do not, and that are heavy or not finite, become zeros here and are added by hand below
                    unsigned char* vt;
                    if constexpr (S::kFp8) {
                        wait(ms.v16_full[n & 1], n >> 1);
                        vt = v16 + (n & 1) * S::kV16Bytes;
                    } else {
                        wait(ms.full[vs], n / S::kVSlots);
                        vt = ring + vs * S::kSlotBytes;
                    }
                    if (cg == 0) {
                        const int32_t tok = token0 + gt;
                        const bool none = tok > seen_any || tok < from_any, some = tok > seen_all || tok < from_all;
                        bool clear = none;
                        if (!none && some) {
                            if constexpr (S::kFp8) clear = heavy((int)ms.scales[1][n & 15][gt] - 127);
#pragma unroll 2
                            for (int ch = 0; ch < DP / 8; ++ch) {
                                const uint4 v4 = *reinterpret_cast<const uint4*>(vt + (ch / 8) * (kTile * 128) + gt * 128 + (((ch % 8) ^ (gt & 7)) * 16));
                                clear = clear || (not_finite<M>(v4.x) | not_finite<M>(v4.y) | not_finite<M>(v4.z) | not_finite<M>(v4.w)) != 0;
                            }
                            if (clear) atomicOr(&pz[wq], 1u << lane);
                        }
                        if (clear) {
#pragma unroll 4
                            for (int ch = 0; ch < DP / 8; ++ch)
                                *reinterpret_cast<uint4*>(vt + (ch / 8) * (kTile * 128) + gt * 128 + ((ch % 8) ^ (gt & 7)) * 16) = make_uint4(0, 0, 0, 0);
                        }
                    }
                    barrier_sync(id_par, kParThreads);
                    poisoned = (pz[0] | pz[1] | pz[2] | pz[3]) != 0;
                }
                fence_async();
                tmem_before();
                __syncwarp();
                if (lane == 0) bar_arrive(bar(ms.p_full[n & 1]));
                if constexpr (kMasked) {
                    if (poisoned) {
                        wait(ms.pv_done[n & 1], n >> 1);
                        tmem_after();
                        const int d = gt;                                // this thread's element of the head
#pragma unroll 1
                        for (int tk = 0; tk < kTile; ++tk) {
                            if (!(pz[tk >> 5] >> (tk & 31) & 1u)) continue;
                            const int32_t tok = token0 + tk;
                            const int page = __ldg(a.block_table + w.b * a.block_stride + tok / c.page_size);
                            float v = 0.f;
                            if (d < c.head_dim && page >= 0 && page < c.num_pages) {
                                const int64_t at = page * c.page_stride + w.h * c.head_stride + tok % c.page_size * c.slot_stride + d;
                                if constexpr (S::kFp8) {
                                    const int e = (int)ms.scales[1][n & 15][tk] - 127;
                                    v = to_float<__nv_fp8_e4m3>(static_cast<const __nv_fp8_e4m3*>(c.v)[at]);
                                    if (heavy(e)) v = ldexpf(v, e - ms.scale_e[grp]);  // (its weights are without their scale)
                                }
                                else v = to_float<M>(static_cast<const M*>(c.v)[at]);
                            }
#pragma unroll 1
                            for (int i = 0; i < NC; i += 16) {
                                float o[16];
                                uint32_t r[16];
                                tmem_ld_32x16(acc + i, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 16; ++k) {
                                    const int col = col0 + i + k, lt = ms.last[tb][col];
                                    const bool seen = tok <= lt && (a.window == 0 || tok > lt - a.window);
                                    const float p = to_float<M>(*reinterpret_cast<const M*>(pt + ((col >> 3) * 16 + (tk >> 3)) * 128 + (col & 7) * 16 + (tk & 7) * 2));
                                    r[k] = __float_as_uint(seen && p != 0.f ? fmaf(p, v, o[k]) : o[k]);
                                }
                                tmem_st_32x16(acc + i, r);
                                tmem_wait_st();
                            }
                        }
                        barrier_sync(id_par, kParThreads);
                        if (cg == 0 && gt < 4) pz[gt] = 0;
                        barrier_sync(id_par, kParThreads);
                        tmem_before();
                    }
                }
            };
#pragma unroll 1
            for (int t = w.t0; t < w.t1; ++t, ++n) {
                if (S::kPar == 2 && (int)(n & 1) != par) continue;
                const int32_t token0 = t * kTile;
                if (token0 + kTile - 1 > seen_all || token0 < from_all) tile(std::true_type{}, t);
                else tile(std::false_type{}, t);
            }
            // ---- the item's (part of) result
            const uint32_t last_n = n - 1;
#pragma unroll
            for (int i = 0; i < NC / 4; ++i) {
#pragma unroll
                for (int off = 4; off <= 16; off <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
            }
            if (tq == 0) {
#pragma unroll
                for (int i = 0; i < NC / 4; ++i) {
                    const int col = col0 + 8 * (i >> 1) + cq + (i & 1);
                    ms.red[par][wq][col] = l[i];
                    if (wq == 0) ms.ref[par][col] = m[i];
                }
            }
            if (S::kFp8 && cg == 0 && gt == 0) ms.ref_e[par] = ms.scale_e[grp];
            const bool whole = w.begin && w.end;
            float* const part = a.parts + (int64_t)(2 * blockIdx.x + (w.begin ? 1 : 0)) * S::kSlotFloats;
            barrier_sync(7, 128 * S::kGroups);
            if (S::kFp8 && gt == 0) {                                    // (all have read them)
                ms.scale_e[grp] = kUnset;
                ms.lift_over[grp] = kNone;
            }
            if (tid < N) {
                // the column's sum, over both sets of tiles at one reference, and each set's factor for O
                float ref = ms.ref[0][tid], sum = 0.f, f[S::kPar];
                if constexpr (S::kPar == 2) ref = fmaxf(ref, ms.ref[1][tid]);
#pragma unroll
                for (int p = 0; p < S::kPar; ++p) {
                    const float s = ms.red[p][0][tid] + ms.red[p][1][tid] + ms.red[p][2][tid] + ms.red[p][3][tid];
                    f[p] = s == 0.f ? 0.f : S::kPar == 1 ? 1.f : exp2_fast(ms.ref[p][tid] - ref);
                    sum += s == 0.f ? 0.f : s * f[p];
                }
                const bool any = !(sum == 0.f);                          // (a NaN sum is one)
#pragma unroll
                for (int p = 0; p < S::kPar; ++p) {
                    float y = f[p];
                    if constexpr (S::kFp8) {
                        const int e = ms.ref_e[p];
                        if (e != kUnset) y *= __uint_as_float((uint32_t)(127 + e) << 23);
                    }
                    ms.fac[p][tid] = !any ? 0.f : whole ? y * __frcp_rn(sum) : y;
                }
                if (whole) {
                    const int2 at = ms.place[tb][tid];
                    if (a.lse && at.x >= 0) a.lse[(int64_t)at.x * a.num_heads + at.y] = lse_of(any, ref, sum);
                } else {
                    part[N * DP + tid] = ref;
                    part[N * DP + N + tid] = sum;
                }
            }
            wait(ms.pv_done[last_n & 1], last_n >> 1);                   // (products end in order)
            tmem_after();
            barrier_sync(7, 128 * S::kGroups);
            const int d = gt;
            constexpr int kEach = N / S::kGroups;                        // columns that a group writes
#pragma unroll 1
            for (int i = 0; i < kEach; i += 8) {
                const int first = grp * kEach + i;
                float o[S::kPar][8];
#pragma unroll
                for (int p = 0; p < S::kPar; ++p) tmem_ld_32x8(t_o + p * N + quarter + first, o[p]);
                tmem_wait_ld();
                // (every read before the first write, and no branch between them)
                int64_t at[8];
                float y[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    at[k] = ms.out_at[tb][first + k];
                    y[k] = 0.f;
#pragma unroll
                    for (int p = 0; p < S::kPar; ++p) {
                        const float f = ms.fac[p][first + k];
                        y[k] += f == 0.f ? 0.f : o[p][k] * f;            // (O is not set where its set had no tile)
                    }
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const bool mine = at[k] >= 0 && d < c.head_dim;
                    if (whole && mine) static_cast<T*>(a.out)[at[k] + d] = from_float<T>(y[k]);
                    if (!whole && mine) part[(first + k) * DP + d] = y[k];
                }
            }
            if (tid == 0 && w.begin && !w.end) {
                // the CTA of the item's last unit
                int lastc = (int)min((int64_t)P - 1, quotient(w.last_unit, max((int64_t)1, quotient(ms.units, P))));
                while (cta_begin(ms.units, lastc + 1, P) <= w.last_unit) ++lastc;
                while (cta_begin(ms.units, lastc, P) > w.last_unit) --lastc;
                a.split[blockIdx.x] = {w.row0, w.rows, w.block * N, w.h, lastc};
            }
            tmem_before();
            __syncwarp();
            if (lane == 0) bar_arrive(bar(ms.done[q & 1]));
        }
        // requests that the kernel does not take: their bits, and zeros in the rows that are known
#pragma unroll 1
        for (int b = blockIdx.x; b < a.B; b += P) {
            const Request r = request_of<N>(a, b);
            if (!r.fault) continue;
            if (tid == 0 && a.status) atomicOr(a.status + b, r.fault);
            if (r.fault == SPECDEC_ST_BAD_OFFSETS) continue;
            const int64_t k1 = (int64_t)a.cu[b + 1] - a.cu[b] + 1;
#pragma unroll 1
            for (int64_t i = tid; i < k1 * a.num_heads; i += 128 * S::kGroups) {
                const int64_t row = r.row0 + quotient(i, a.num_heads), hq = i - quotient(i, a.num_heads) * a.num_heads;
                if (a.lse) a.lse[row * a.num_heads + hq] = -INFINITY;
                T* out = static_cast<T*>(a.out) + row * a.out_row + hq * a.out_head;
#pragma unroll 1
                for (int d = 0; d < c.head_dim; d += 8) *reinterpret_cast<uint4*>(out + d) = make_uint4(0, 0, 0, 0);
            }
        }
    }
    tmem_before();
    __syncthreads();
    tmem_after();
    if (*expired && tid == 0 && a.status && ms.begin < ms.end) {
        // every request that the CTA has a unit of
        int64_t base = ms.base;
#pragma unroll 1
        for (int b = ms.first_b; b < a.B && base < ms.end; ++b) {
            const int64_t n = request_of<N>(a, b).units(H);
            if (n > 0) atomicOr(a.status + b, SPECDEC_ST_DEVICE_TIMEOUT);
            base += n;
        }
    }
    if (*expired && (warp == S::kScores || warp == S::kValues)) {
        // products issued so far end by themselves: wait for them
        if (elected()) mma_commit(bar(ms.drained));
        __syncwarp();
    }
    if (warp == S::kScores) {
        if (*expired) {
            const unsigned long long t0 = time_ns();
            while (!bar_test(bar(ms.drained), 0) && time_ns() - t0 < kDrainNs) {}
            __syncwarp();
        }
        tmem_free(tmem, S::kTmemColumns);
    }
}

// Joins the parts of the item that CTA blockIdx.x of the kernel above left to its successors: slot 2 i + 1, then
// slot 2 j of each CTA j up to the last. A warp takes 32 elements of a row: its lanes hold the parts' factors, and
// the parts' elements are summed in their order.
template <typename T, int N, int DP>
__global__ void __launch_bounds__(kJoinThreads) specdec_paged_join_kernel(const Args a)
{
    after_predecessor();
    const Split s = a.split[blockIdx.x];
    if (s.last < 0) return;
    constexpr int64_t kSlot = N * (DP + 2);
    constexpr int kWarps = DP / 32, kRows = kJoinThreads / DP;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = (warp % kWarps) * 32 + lane, i = blockIdx.x, n = s.last - i + 1;
    const float* const head = a.parts + (2 * (int64_t)i + 1) * kSlot;
    const float* const tail = a.parts + 2 * (int64_t)i * kSlot;
    auto part = [&](int j) { return j == 0 ? head : tail + 2 * j * kSlot; };
#pragma unroll 1
    for (int col = blockIdx.y * kRows + warp / kWarps; col < N; col += gridDim.y * kRows) {
        const int row = s.first + col;
        if (row >= s.rows) return;
        float m = -FLT_MAX;
#pragma unroll 1
        for (int j = lane; j < n; j += 32) m = fmaxf(m, part(j)[N * DP + col]);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        float l = 0.f, o = 0.f;
#pragma unroll 1
        for (int j0 = 0; j0 < n; j0 += 32) {
            float f = 0.f;
            if (j0 + lane < n) {
                const float* p = part(j0 + lane) + N * DP + col;
                f = exp2_fast(p[0] - m);
                l += p[N] * f;
            }
            const int up = min(32, n - j0);
#pragma unroll 1
            for (int j = 0; j < up; j += 8) {                            // eight parts' elements in flight
                float x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = j + k < up ? part(j0 + j + k)[col * DP + d] : 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float fk = __shfl_sync(0xffffffffu, f, j + k);
                    o = j + k < up ? fmaf(x[k], fk, o) : o;
                }
            }
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        const int j = row / a.group, g = row - j * a.group;
        const int64_t t = s.row0 + j, hq = s.head * a.group + g;
        const bool any = !(l == 0.f);
        if (d < a.cache.head_dim) static_cast<T*>(a.out)[t * a.out_row + hq * a.out_head + d] = from_float<T>(any ? o * __frcp_rn(l) : 0.f);
        if (d == 0 && a.lse) a.lse[t * a.num_heads + hq] = lse_of(any, m, l);
    }
}

// ---------------------------------------------------------------- host side

int sm_count()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) == cudaSuccess && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && n > 0)
        return n;
    (void)cudaGetLastError();
    return 152;
}

int row_tile(int32_t max_k, int32_t group)
{
    const int64_t rows = ((int64_t)max_k + 1) * group;
    return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 96 ? 96 : 128;
}

// A window that no request can be longer than hides nothing: it is none (0). One that is left is below most_tokens, and
// a tile's first token lies at most SPECDEC_KMAX behind `cached`, so that cached - window + 1 - token0, the copies' smallest
// difference, is at least -32 - (2^31 - 130) + 1 and does not wrap.
int32_t window_of(int32_t window, int32_t max_blocks, int32_t page_size)
{
    return window >= most_tokens(max_blocks, page_size) ? 0 : window;
}

size_t split_bytes(int P) { return ((size_t)P * sizeof(Split) + 255) / 256 * 256; }

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Encode encoder()
{
    static const Encode e = [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            fn = nullptr;
        }
        return reinterpret_cast<Encode>(fn);
    }();
    return e;
}

// [pages, heads, slots, elements] in tiles of one page's slots (at most 128) and 128 bytes (64 for an e4m3 head of up to 64)
bool tile_map(CUtensorMap* map, const specdec_kv_cache_t& c, void* base)
{
    const int es = (int)elem_bytes(c.dtype);
    const cuuint64_t size[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.num_kv_heads, (cuuint64_t)c.num_pages};
    auto bytes = [&](int64_t stride, int64_t n) { return (cuuint64_t)(n > 1 ? stride * es : 16); };
    const cuuint64_t stride[3] = {bytes(c.slot_stride, c.page_size), bytes(c.head_stride, c.num_kv_heads), bytes(c.page_stride, c.num_pages)};
    const int inner = es == 1 && c.head_dim <= 64 ? 64 : es == 1 ? 128 : 64;
    const cuuint32_t box[4] = {(cuuint32_t)inner, (cuuint32_t)(c.page_size < kTile ? c.page_size : kTile), 1, 1}, step[4] = {1, 1, 1, 1};
    const CUtensorMapDataType type = es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : c.dtype == SPECDEC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const CUtensorMapSwizzle swizzle = inner * es == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    return encoder()(map, type, 4, base, size, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename S> specdec_status_t launch(const Args& a, cudaStream_t stream, int P)
{
    static_assert(sizeof(CUtensorMap) == 128, "tensor map");
    CUtensorMap kmap, vmap;
    if (!encoder()) return SPECDEC_ERR_CUDA;
    if (!tile_map(&kmap, a.cache, a.cache.k) || !tile_map(&vmap, a.cache, a.cache.v)) return SPECDEC_ERR_INVALID_ARG;
    constexpr int smem = S::kSmem;
    static_assert(1023 + S::kMiscAt + (int)sizeof(Misc<S>) <= smem, "shared memory, wherever its base lies");
    auto kernel = specdec_paged_attention_kernel<S>;
    // the kernel's shared memory is allowed at its first launch (and again where a context has been reset since)
    static std::atomic<uint64_t> allowed{0};             // devices, by bit
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return SPECDEC_ERR_CUDA;
    }
    const uint64_t bit = 1ull << (dev & 63);
    for (int attempt = allowed.load() & bit ? 0 : 1;; ++attempt) {
        if (attempt > 0 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
            (void)cudaGetLastError();
            return SPECDEC_ERR_CUDA;
        }
        if (launch_dependent(kernel, P, S::kThreads, smem, stream, a, kmap, vmap) == cudaSuccess) break;
        if (attempt > 0) return SPECDEC_ERR_CUDA;
    }
    allowed |= bit;
    if (launch_dependent(specdec_paged_join_kernel<typename S::T, S::N, S::DP>, dim3((unsigned)P, 4), kJoinThreads, 0, stream, a) != cudaSuccess)
        return SPECDEC_ERR_CUDA;
    return SPECDEC_OK;
}

template <typename T, bool kFp8, int DB> specdec_status_t launch_rows(const Args& a, int N, cudaStream_t s, int P)
{
    if (N == 16) return launch<Shape<T, kFp8, 16, DB>>(a, s, P);
    if (N == 32) return launch<Shape<T, kFp8, 32, DB>>(a, s, P);
    if (N == 64) return launch<Shape<T, kFp8, 64, DB>>(a, s, P);
    if (N == 96) return launch<Shape<T, kFp8, 96, DB>>(a, s, P);
    return launch<Shape<T, kFp8, 128, DB>>(a, s, P);
}

template <typename T> specdec_status_t launch_type(const Args& a, int N, cudaStream_t s, int P)
{
    const bool fp8 = a.cache.dtype == SPECDEC_E4M3, one = a.cache.head_dim <= 64;
    if (fp8) return one ? launch_rows<T, true, 1>(a, N, s, P) : launch_rows<T, true, 2>(a, N, s, P);
    return one ? launch_rows<T, false, 1>(a, N, s, P) : launch_rows<T, false, 2>(a, N, s, P);
}

}  // namespace

extern "C" size_t specdec_paged_attention_workspace_size(int32_t B, int32_t max_k, int32_t num_heads,
                                                         int32_t num_kv_heads, int32_t head_dim)
{
    if (B <= 0 || max_k < 0 || max_k > SPECDEC_KMAX || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0 ||
        !cache_head_dim(head_dim))
        return 0;
    const int P = sm_count(), group = num_heads / num_kv_heads, DP = head_dim <= 64 ? 64 : 128;
    return split_bytes(P) + (size_t)2 * P * row_tile(max_k, group) * (DP + 2) * sizeof(float);
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
    const int P = sm_count(), group = num_heads / cache->num_kv_heads;
    const Args a = {q, out, lse, rows, num_heads, group, q_row_stride, q_head_stride, out_row_stride, out_head_stride, *cache,
                    block_table, block_stride, max_blocks, cached_len, cu_num_draft, B, max_k,
                    window_of(window, max_blocks, cache->page_size), scale * 1.4426950408889634f,
                    status, static_cast<Split*>(workspace), reinterpret_cast<float*>(static_cast<char*>(workspace) + split_bytes(P)),
                    wait_limit_us < 0 ? kWaitNs : (uint32_t)wait_limit_us * 1000u};
    const int N = row_tile(max_k, group);
    return dtype == SPECDEC_BF16 ? launch_type<__nv_bfloat16>(a, N, (cudaStream_t)stream, P) : launch_type<__half>(a, N, (cudaStream_t)stream, P);
}
