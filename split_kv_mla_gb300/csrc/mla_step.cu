// mla_step.cu -- what lies between two steps of a decode loop: the beams' next
// tokens (selection), their states in their new order (reordering), and the next
// step's page tables, lengths, slots and positions (extension).  See
// include/mla_decode.h for the contracts.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "mla_internal.h"
#include "mla_launch.h"
#include "mla_softmax.cuh"

namespace mla {
namespace {

// ---- beam selection -------------------------------------------------------------------------
//
// The logits are read once.  For a row's score order only x matters, and the K best
// of a request lie in the K best groups of columns, when groups are ordered by their
// largest score and then by their index: each of those groups has a candidate at
// least as good as the K-th of them, and a candidate outside them is behind all of
// these (a group is a range of columns, so of equal scores the lower index is also in
// the lower group).  So
//   scan   streams the rows and leaves, for each 256 columns, their maximum, and for
//          each 4 KB segment of a row its maximum m and sum of e^(x - m);
//   pick   (a CTA per request) joins a row's segments, takes the K best groups by
//          their maxima, reads those 256 logits of each again and takes the K best.
// What scan does per logit does not depend on the data, and pick reads 1/64 of the
// bytes and K groups.
//
// A segment's sum is relative to its own maximum, so its largest term is 1, and is
// held in fp32; which column goes to which lane does not depend on a row's address,
// so equal rows give equal sums and their equal candidates are taken by their index.

constexpr int kGroup = 256;             // columns
constexpr int kLongPieces = 8;          // 16-byte loads of a lane per segment, of large calls
constexpr int kShortPieces = 2;         // and of small ones
constexpr int kScanThreads = 256;
constexpr int kPickThreads = 512;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kPickList = 1024;
static_assert(kPickWarps == 16, "the halves of 16 warps are the 32 parts that pick_best takes");
constexpr int kMaxVocab = 1 << 20;

struct SelectArgs {
    const void* logits;
    int64_t row_stride;
    const float* scores;
    const uint8_t* finished;
    int32_t batch, beams, vocab, select, end_token;
    int32_t groups;        // of a row
    int32_t segments;      // of a row
    int64_t rows;
    float* group_max;      // [rows, groups]
    float2* parts;         // [rows, segments]: maximum, sum
    int32_t* tokens;
    int32_t* parents;
    float* scores_out;
    uint8_t* finished_out;
    uint32_t* err;
};

template <typename T>
struct LogitType;

template <>
struct LogitType<__nv_bfloat16> {
    static constexpr uint32_t kNone = 0xFF80u;   // -inf
    static __device__ __forceinline__ float2 unpack(uint32_t w)
    {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
    {
        const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                         *reinterpret_cast<const __nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&m);
    }
};

template <>
struct LogitType<__half> {
    static constexpr uint32_t kNone = 0xFC00u;
    static __device__ __forceinline__ float2 unpack(uint32_t w)
    {
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
    {
        const __half2 m = __hmax2(*reinterpret_cast<const __half2*>(&a),
                                  *reinterpret_cast<const __half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&m);
    }
};

template <typename T>
constexpr int kElements = 16 / (int)sizeof(T);   // of a 16-byte piece

template <typename T, int PIECES>
constexpr int kSegment = PIECES * 32 * kElements<T>;   // columns

// Maximum of a piece (a NaN is passed over: the sum shows it).
template <typename T>
__device__ __forceinline__ float piece_max(const uint4& v)
{
    if constexpr (sizeof(T) == 4) {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                     fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    } else {
        using L = LogitType<T>;
        const float2 m = L::unpack(L::max2(L::max2(v.x, v.y), L::max2(v.z, v.w)));
        return fmaxf(m.x, m.y);
    }
}

template <typename T, class F>
__device__ __forceinline__ void each_logit(const uint4& v, F&& f)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            f(i, __uint_as_float(w[i]));
        } else {
            const float2 p = LogitType<T>::unpack(w[i]);
            f(2 * i, p.x);
            f(2 * i + 1, p.y);
        }
    }
}

// Columns [col, col + elements) of a row of `vocab`, -inf behind its end, one by one.
template <typename T>
__device__ __noinline__ uint4 load_edge(const T* row, int col, int vocab)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            w[i] = col + i < vocab ? __ldg(reinterpret_cast<const uint32_t*>(row) + col + i)
                                   : 0xFF800000u;
        } else {
            const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
            const uint32_t none = LogitType<T>::kNone;
            const uint32_t lo = col + 2 * i < vocab ? __ldg(p + col + 2 * i) : none;
            const uint32_t hi = col + 2 * i + 1 < vocab ? __ldg(p + col + 2 * i + 1) : none;
            w[i] = lo | hi << 16;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The same.  Pieces of an aligned row are one load.  Otherwise a piece lies in two
// aligned ones, and is shifted out of them where both are inside the row.
template <typename T, bool ALIGNED>
__device__ __forceinline__ uint4 load_piece(const T* row, int col, int vocab)
{
    if constexpr (ALIGNED) {
        if (col + kElements<T> <= vocab)
            return __ldcs(reinterpret_cast<const uint4*>(row + col));
    } else {
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + col);
        const uint32_t off = (uint32_t)at & 15u;
        const uintptr_t from = at - off;
        if (from >= reinterpret_cast<uintptr_t>(row) &&
            from + 32 <= reinterpret_cast<uintptr_t>(row + vocab)) {
            const uint4 a = __ldg(reinterpret_cast<const uint4*>(from));
            const uint4 b = __ldg(reinterpret_cast<const uint4*>(from) + 1);
            uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            if (off & 8u) {
#pragma unroll
                for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
            }
            if (off & 4u) {
#pragma unroll
                for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
            }
            const uint32_t s = (off & 2u) * 8u;
            return make_uint4(__funnelshift_r(w[0], w[1], s), __funnelshift_r(w[1], w[2], s),
                              __funnelshift_r(w[2], w[3], s), __funnelshift_r(w[3], w[4], s));
        }
    }
    return load_edge(row, col, vocab);
}

// Floats as integers in the same order.
__device__ __forceinline__ int ordered(float x)
{
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7FFFFFFF);
}

__device__ __forceinline__ float from_ordered(int i)
{
    return __int_as_float(i ^ ((i >> 31) & 0x7FFFFFFF));
}

__device__ __forceinline__ bool row_is_live(const SelectArgs& a, int64_t row)
{
    return __ldg(a.scores + row) != -INFINITY &&
           (a.finished == nullptr || __ldg(a.finished + row) == 0);
}

// A warp per segment.  The rows of beams without candidates are not read, except where
// a call is so small that its logits are asked for before it is known which those are.
template <typename T, bool ALIGNED, int PIECES>
__global__ void __launch_bounds__(kScanThreads)
scan_kernel(const SelectArgs a)
{
    constexpr bool kEager = PIECES == kShortPieces;
    constexpr int E = kElements<T>;
    constexpr int kPerGroup = kGroup / (32 * E);         // pieces of a group
    constexpr int kGroups = PIECES / kPerGroup;          // groups of a segment
    wait_for_predecessor();
    allow_dependents();
    const int lane = threadIdx.x & 31;
    const uint32_t id = blockIdx.x * (kScanThreads / 32) + (threadIdx.x >> 5);   // below 2^31
    const int64_t row = id / (uint32_t)a.segments;
    const int seg = (int)(id % (uint32_t)a.segments);
    if (row >= a.rows) return;
    const bool live = row_is_live(a, row);
    if (!kEager && !live) return;
    const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
    const int c0 = seg * kSegment<T, PIECES> + lane * E;
    uint4 v[PIECES];
#pragma unroll
    for (int p = 0; p < PIECES; ++p) v[p] = load_piece<T, ALIGNED>(x, c0 + p * 32 * E, a.vocab);
    if (kEager && !live) return;

    int most = INT32_MIN, mine = 0;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        float m = piece_max<T>(v[g * kPerGroup]);
#pragma unroll
        for (int p = 1; p < kPerGroup; ++p) m = fmaxf(m, piece_max<T>(v[g * kPerGroup + p]));
        const int r = __reduce_max_sync(0xffffffffu, ordered(m));
        most = max(most, r);
        if (lane == g) mine = r;
    }
    const int group = seg * kGroups + lane;
    if (lane < kGroups && group < a.groups) a.group_max[row * a.groups + group] = from_ordered(mine);

    const float top = from_ordered(most);
    const float ref = top == -INFINITY ? 0.f : top;
    constexpr float kLog2e = 1.4426950408889634f;
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int p = 0; p < PIECES; ++p)
        each_logit<T>(v[p], [&](int i, float t) { sum[i & 1] += ex2_approx((t - ref) * kLog2e); });
    float s = sum[0] + sum[1];
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (lane == 0) a.parts[row * a.segments + seg] = make_float2(top, s);
}

// (hi, lo) of a + b.
__device__ __forceinline__ float2 two_sum(float a, float b)
{
    const float s = __fadd_rn(a, b);
    const float t = __fsub_rn(s, a);
    return make_float2(s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t)));
}

// score - m - ln(sum) as a sum of two floats, so that a candidate's score is rounded
// once: the scores of different beams that fp32 tells apart come out in their order.
// ln(sum) = e ln 2 + ln f with f in [0.75, 1.5); ln 2 in two parts, of which the first
// has 12 bits, so that e times it is exact.
__device__ __forceinline__ float2 row_base(float score, float m, float sum)
{
    int e = ((__float_as_int(sum) >> 23) & 255) - 127;
    float f = __int_as_float((__float_as_int(sum) & 0x7FFFFF) | 0x3F800000);
    if (f >= 1.5f) {
        f *= 0.5f;
        ++e;
    }
    constexpr double kLn2 = 0.69314718055994530942;
    constexpr double kHigh = 2839.0 / 4096.0;
    const float2 a = two_sum(score, -m);
    const float2 b = two_sum(a.x, -(float)e * (float)kHigh);
    const float rest = (a.y + b.y) - fmaf((float)e, (float)(kLn2 - kHigh), logf(f));
    const float hi = __fadd_rn(b.x, rest);
    return make_float2(hi, __fadd_rn(__fsub_rn(b.x, hi), rest));
}

// A score as a number in its order; 0 for what is no candidate (-inf, or the NaN that
// the base of a beam without candidates makes).
__device__ __forceinline__ uint32_t rank_of(float2 base, float x)
{
    const float2 s = two_sum(base.x, x);
    const float score = __fadd_rn(__fadd_rn(s.x, __fadd_rn(s.y, base.y)), 0.f);   // -0 as +0
    return score > -INFINITY ? (uint32_t)ordered(score) ^ 0x80000000u : 0u;
}

// With the index, a lower one first; 0: none.
__device__ __forceinline__ uint64_t candidate(uint32_t rank, uint32_t index)
{
    return rank == 0 ? 0 : (uint64_t)rank << 32 | (0xFFFFFFFFu - index);
}

__device__ __forceinline__ uint32_t index_of(uint64_t c) { return 0xFFFFFFFFu - (uint32_t)c; }

__device__ __forceinline__ float score_of(uint64_t c)
{
    return from_ordered((int)((uint32_t)(c >> 32) ^ 0x80000000u));
}

struct Picker {
    uint32_t best[32];            // of each half of a warp
    uint64_t list[kPickList];
    uint64_t last[kPickWarps];
    uint32_t least;
    int count;
};

// The K largest of the CTA's candidates: done(k, c) is called once for each k < K, by
// some thread, with the k-th of them (0 where there are fewer).  best is the largest
// rank among this thread's, and each(least, f) calls f(candidate) for each of this
// thread's of at least that rank.  Of the best of 32 parts the K-th is at or below the
// K-th of all: what is not below it is listed and ranked by counting.  A list that
// would overflow (many equal scores, or a part that holds most of the best and many) is
// not used: the K are taken one after the other.
template <class Each, class Done>
__device__ __forceinline__ void pick_best(Picker& p, int K, uint32_t best, Each&& each, Done&& done)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t half = lane < 16 ? 0xFFFFu : 0xFFFF0000u;
    best = __reduce_max_sync(half, best);
    if ((lane & 15) == 0) p.best[2 * warp + (lane >> 4)] = best;
    if (tid == 0) {
        p.count = 0;
        p.least = 1;
    }
    __syncthreads();
    if (warp == 0) {
        const uint32_t mine = p.best[lane];
        int above = 0;
#pragma unroll
        for (int w = 0; w < 32; ++w) {
            const uint32_t other = p.best[w];
            above += other > mine || (other == mine && w < lane) ? 1 : 0;
        }
        if (above == K - 1 && mine != 0) p.least = mine;
    }
    __syncthreads();
    each(p.least, [&](uint64_t c) {
        const int at = atomicAdd(&p.count, 1);
        if (at < kPickList) p.list[at] = c;
    });
    __syncthreads();
    const int n = p.count;
    if (n <= kPickList) {
        for (int i = tid; i < n; i += kPickThreads) {
            const uint64_t mine = p.list[i];
            int above = 0;
            for (int j = 0; j < n; ++j) above += p.list[j] > mine ? 1 : 0;
            if (above < K) done(above, mine);
        }
        if (tid >= n && tid < K) done(tid, 0);
    } else {
        uint64_t last = ~0ull;
        for (int k = 0; k < K; ++k) {
            uint64_t next = 0;
            each(1, [&](uint64_t c) { next = c < last && c > next ? c : next; });
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) {
                const uint64_t other = __shfl_xor_sync(0xffffffffu, next, off);
                next = other > next ? other : next;
            }
            if (lane == 0) p.last[warp] = next;
            __syncthreads();
            last = p.last[0];
#pragma unroll
            for (int w = 1; w < kPickWarps; ++w) last = p.last[w] > last ? p.last[w] : last;
            if (tid == 0) done(k, last);
            __syncthreads();
        }
    }
}

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kPickThreads)
pick_kernel(const SelectArgs a)
{
    constexpr int E = kElements<T>;
    constexpr int kPerGroup = kGroup / (32 * E);
    constexpr int kItems = 8;      // group maxima of a thread that stay in registers
    constexpr int kParts = 4;      // parts of a row, of a lane
    constexpr int kTurns = MLA_MAX_BEAMS / kPickWarps;
    __shared__ Picker p;
    __shared__ uint64_t taken[MLA_MAX_BEAMS];
    __shared__ float2 base[MLA_MAX_BEAMS];   // -inf: no candidates; of an ended beam its score
    __shared__ uint32_t ended;               // bit per beam
    wait_for_predecessor();
    allow_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row0 = (int64_t)blockIdx.x * a.beams;
    const int K = a.select, W = a.beams;
    const uint32_t G = (uint32_t)a.groups, items = (uint32_t)W * G;

    const float* maxima = a.group_max + row0 * G;
    float gm[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const uint32_t i = tid + k * kPickThreads;
        gm[k] = i < items ? __ldcg(maxima + i) : 0.f;
    }
    if (tid < 32) {
        const bool e = tid < W && a.finished != nullptr && a.finished[row0 + tid] != 0;
        const uint32_t bits = __ballot_sync(0xffffffffu, e);
        if (tid == 0) ended = bits;
    }
#pragma unroll 1
    for (int w = warp; w < W; w += kPickWarps) {
        const int64_t row = row0 + w;
        const float2* parts = a.parts + row * a.segments;
        const float own = __ldg(a.scores + row);
        const bool is_ended = a.finished != nullptr && a.finished[row] != 0;
        float2 t[kParts];
        float m = -INFINITY, s = 0.f;
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
            const int i = lane + 32 * k;
            t[k] = i < a.segments ? __ldcg(parts + i) : make_float2(-INFINITY, 0.f);
        }
#pragma unroll
        for (int k = 0; k < kParts; ++k) m = fmaxf(m, t[k].x);
        for (int i = lane + 32 * kParts; i < a.segments; i += 32) m = fmaxf(m, __ldcg(parts + i).x);
        m = from_ordered(__reduce_max_sync(0xffffffffu, ordered(m)));
        const float ref = m == -INFINITY ? 0.f : m;
        constexpr float kLog2e = 1.4426950408889634f;
#pragma unroll
        for (int k = 0; k < kParts; ++k) s += t[k].y * ex2_approx((t[k].x - ref) * kLog2e);
        for (int i = lane + 32 * kParts; i < a.segments; i += 32) {
            const float2 u = __ldcg(parts + i);
            s += u.y * ex2_approx((u.x - ref) * kLog2e);
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        if (lane == 0) {
            // (what is not read of a beam without candidates may be anything)
            const bool none = own == -INFINITY;
            // a NaN or +inf among the logits makes the sum one
            const bool bad = !none && (!(own < INFINITY) || (!is_ended && !(s < INFINITY)));
            if (bad) atomicOr(a.err, MLA_DEVERR_BAD_LOGITS);
            if (none || bad || (!is_ended && s == 0.f)) base[w] = make_float2(-INFINITY, 0.f);
            else base[w] = is_ended ? make_float2(own, 0.f) : row_base(own, m, s);
        }
    }
    __syncthreads();

    // groups: item i of beam i / G
    const uint32_t ends = ended;
    const uint32_t step_w = kPickThreads / G, step_g = kPickThreads % G;
    auto rank_item = [&](uint32_t w, uint32_t g, float x) {
        if ((ends >> w) & 1u) x = g == 0 ? 0.f : -INFINITY;
        return rank_of(base[w], x);
    };
    auto next_item = [&](uint32_t& w, uint32_t& g) {
        w += step_w;
        g += step_g;
        if (g >= G) {
            g -= G;
            ++w;
        }
    };
    uint32_t rank[kItems], best = 0;
    uint32_t w = (uint32_t)tid / G, g = (uint32_t)tid % G;
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        rank[k] = w < (uint32_t)W ? rank_item(w, g, gm[k]) : 0u;
        best = max(best, rank[k]);
        next_item(w, g);
    }
    const uint32_t w8 = w, g8 = g;   // of the first item that is not in registers
    for (uint32_t i = tid + kItems * kPickThreads; i < items; i += kPickThreads) {
        best = max(best, rank_item(w, g, __ldcg(maxima + i)));
        next_item(w, g);
    }
    pick_best(
        p, K, best,
        [&](uint32_t least, auto&& take) {
#pragma unroll
            for (int k = 0; k < kItems; ++k)
                if (rank[k] >= least) take(candidate(rank[k], tid + k * kPickThreads));
            uint32_t iw = w8, ig = g8;
            for (uint32_t i = tid + kItems * kPickThreads; i < items; i += kPickThreads) {
                const uint32_t r = rank_item(iw, ig, __ldcg(maxima + i));
                if (r >= least) take(candidate(r, i));
                next_item(iw, ig);
            }
        },
        [&](int k, uint64_t c) { taken[k] = c; });
    __syncthreads();

    // the logits of a warp's groups, eight a lane
    uint4 v[kTurns][kPerGroup];
    uint32_t column[kTurns], beam[kTurns], top[kTurns];
    best = 0;
#pragma unroll
    for (int q = 0; q < kTurns; ++q) {
        const int k = warp + q * kPickWarps;
        const uint64_t mine = k < K ? taken[k] : 0;
        const uint32_t i = index_of(mine);
        beam[q] = mine != 0 ? i / G : 0u;
        column[q] = (i - beam[q] * G) * kGroup + lane * E;
        top[q] = 0;
        if (mine == 0) continue;
        if ((ends >> beam[q]) & 1u) {
            column[q] = a.end_token;
            top[q] = lane == 0 ? rank_of(base[beam[q]], 0.f) : 0u;
        } else {
            const T* x = static_cast<const T*>(a.logits) + (row0 + beam[q]) * a.row_stride;
            float m = -INFINITY;
#pragma unroll
            for (int z = 0; z < kPerGroup; ++z)
                v[q][z] = load_piece<T, ALIGNED>(x, column[q] + z * 32 * E, a.vocab);
#pragma unroll
            for (int z = 0; z < kPerGroup; ++z) m = fmaxf(m, piece_max<T>(v[q][z]));
            top[q] = rank_of(base[beam[q]], m);
        }
        best = max(best, top[q]);
    }
    const int64_t out = (int64_t)blockIdx.x * K;
    pick_best(
        p, K, best,
        [&](uint32_t least, auto&& take) {
#pragma unroll
            for (int q = 0; q < kTurns; ++q) {
                if (top[q] < least) continue;
                const uint32_t first = beam[q] * (uint32_t)a.vocab + column[q];
                if ((ends >> beam[q]) & 1u) {
                    take(candidate(top[q], first));
                } else {
#pragma unroll
                    for (int z = 0; z < kPerGroup; ++z)
                        each_logit<T>(v[q][z], [&](int i, float x) {
                            const uint32_t r = rank_of(base[beam[q]], x);
                            if (r >= least) take(candidate(r, first + z * 32 * E + i));
                        });
                }
            }
        },
        [&](int k, uint64_t c) {
            int token = -1, w = 0;
            float score = -INFINITY;
            bool end = true;
            if (c != 0) {
                const uint32_t i = index_of(c);
                w = (int)(i / (uint32_t)a.vocab);
                token = (int)(i - (uint32_t)w * a.vocab);
                score = score_of(c);
                end = token == a.end_token || ((ends >> w) & 1u) != 0;
            }
            a.tokens[out + k] = token;
            a.parents[out + k] = (int32_t)(row0 + w);
            a.scores_out[out + k] = score;
            if (a.finished_out != nullptr) a.finished_out[out + k] = end ? 1 : 0;
        });
}

template <typename T, bool ALIGNED, int PIECES>
cudaError_t launch_scan(SelectArgs& a, cudaStream_t s)
{
    a.segments = (a.vocab + kSegment<T, PIECES> - 1) / kSegment<T, PIECES>;
    const int64_t warps = a.rows * a.segments;
    const int64_t ctas = (warps + kScanThreads / 32 - 1) / (kScanThreads / 32);
    return launch_dependent(scan_kernel<T, ALIGNED, PIECES>, dim3((unsigned)ctas), kScanThreads, s,
                            true, a);
}

// Segments of 1 KB instead of 4 while they are no more than the GPU's SMs hold at a time.
constexpr int64_t kShortWarps = 152 * 32;

template <typename T, bool ALIGNED>
cudaError_t launch_select(SelectArgs a, cudaStream_t s)
{
    const int64_t n = kSegment<T, kShortPieces>;
    const bool small = a.rows * ((a.vocab + n - 1) / n) <= kShortWarps;
    const cudaError_t e = small ? launch_scan<T, ALIGNED, kShortPieces>(a, s)
                                : launch_scan<T, ALIGNED, kLongPieces>(a, s);
    if (e != cudaSuccess) return e;
    return launch_dependent(pick_kernel<T, ALIGNED>, dim3((unsigned)a.batch), kPickThreads, s, true, a);
}

template <typename T>
cudaError_t launch_select_of(const SelectArgs& a, cudaStream_t s)
{
    const bool aligned = aligned16(a.logits) &&
                         (a.rows == 1 || a.row_stride * (int64_t)sizeof(T) % 16 == 0);
    return aligned ? launch_select<T, true>(a, s) : launch_select<T, false>(a, s);
}

bool select_shape_ok(int64_t batch, int64_t beams, int64_t vocab)
{
    return batch >= 1 && batch <= 65535 && beams >= 1 && beams <= MLA_MAX_BEAMS && vocab >= 1 &&
           vocab <= kMaxVocab;
}

int64_t select_groups(int64_t vocab) { return (vocab + kGroup - 1) / kGroup; }

// Bytes of the segments' parts: short segments are no more than kShortWarps, long ones
// most for fp32.
int64_t select_part_bytes(int64_t rows, int64_t vocab)
{
    const int64_t n = kSegment<float, kLongPieces>;
    const int64_t parts = rows * ((vocab + n - 1) / n);
    return align256((parts > kShortWarps ? parts : kShortWarps) * (int64_t)sizeof(float2));
}

// ---- beam state reordering ------------------------------------------------------------------
//
// A copy: bounded by HBM for large states, by latency for small ones.  A CTA takes a
// part of one row.  Units are the largest that both tensors' rows are aligned to.

constexpr int kReorderThreads = 256;
constexpr int kReorderTurns = 4;   // units in flight per thread

struct ReorderArgs {
    const uint8_t* state;
    int64_t state_stride;
    int32_t num_parents;
    int64_t row_bytes;
    int32_t elem_bytes;
    const int32_t* parents;
    int32_t num_rows;
    const int32_t* lens;
    const int32_t* tokens;
    uint8_t* out;
    int64_t out_stride;
    int32_t* out_lens;
    uint32_t parts;        // CTAs of a row
    uint32_t* err;
};

template <typename U>
__global__ void __launch_bounds__(kReorderThreads)
reorder_kernel(const ReorderArgs a)
{
    wait_for_predecessor();
    allow_dependents();
    const uint32_t f = blockIdx.x / a.parts, part = blockIdx.x - f * a.parts;
    const bool first = part == 0 && threadIdx.x == 0;
    const int32_t p = __ldg(a.parents + f);
    if (p < 0 || p >= a.num_parents) {
        if (first) {
            atomicOr(a.err, MLA_DEVERR_BAD_TABLE);
            if (a.out_lens != nullptr) a.out_lens[f] = 0;
        }
        return;
    }
    int64_t bytes = a.row_bytes;
    uint8_t* out = a.out + f * a.out_stride;
    if (a.lens != nullptr) {
        const int64_t room = a.row_bytes / a.elem_bytes;
        const int64_t want = __ldg(a.lens + p);
        const int64_t len = want < 0 ? 0 : want > room ? room : want;
        bytes = len * a.elem_bytes;
        if (first) {
            const bool add = a.tokens != nullptr && len < room;
            if (add) *reinterpret_cast<int32_t*>(out + bytes) = __ldg(a.tokens + f);
            if (a.out_lens != nullptr) a.out_lens[f] = (int32_t)(len + (add ? 1 : 0));
            if (len != want || (a.tokens != nullptr && !add)) atomicOr(a.err, MLA_DEVERR_BAD_LENGTH);
        }
    }
    const uint8_t* in = a.state + p * a.state_stride;
    const int64_t units = bytes / (int64_t)sizeof(U);
    const U* from = reinterpret_cast<const U*>(in);
    U* to = reinterpret_cast<U*>(out);
    const int64_t step = (int64_t)a.parts * kReorderThreads * kReorderTurns;
    for (int64_t i = (int64_t)part * (kReorderThreads * kReorderTurns) + threadIdx.x; i < units;
         i += step) {
        U v[kReorderTurns];
#pragma unroll
        for (int k = 0; k < kReorderTurns; ++k)
            if (i + k * kReorderThreads < units) v[k] = __ldg(from + i + k * kReorderThreads);
#pragma unroll
        for (int k = 0; k < kReorderTurns; ++k)
            if (i + k * kReorderThreads < units) to[i + k * kReorderThreads] = v[k];
    }
    // what is left of the last unit
    const int64_t at = units * (int64_t)sizeof(U) + threadIdx.x;
    if (part == 0 && at < bytes) out[at] = in[at];
}

// ---- cache extension --------------------------------------------------------------------------
//
// Bytes: 8 per entry that is kept, 12 (16 with a list of free slots) per token.
// Every CTA sums the requests' lengths and counts by itself, in shared memory, and
// fills its part of the new table from there: one launch.  A kernel that left the sums
// for a second one took 7.5 us where this takes 4.9 (8 requests of 8192), and looking a
// request up in global memory, per entry, 103 us where this takes 9 (512 of 1024 to
// 8192).  More requests than shared memory is given for go that way:
//   sums   (one CTA) the requests' lengths and counts, their sums, the cursor;
//   fill   a thread per entry of the new table and per token.

constexpr int kExtendThreads = 256;
constexpr int kExtendRequests = 2048;   // 32 KB of sums
constexpr int kExtendSpan = 8;          // entries in flight per thread
constexpr int kExtendCtas = 4 * 152;
constexpr int kLeadTokens = 2048;       // that one CTA takes
constexpr int kSumThreads = 1024;
constexpr int kFillThreads = 256;

struct ExtendArgs {
    const int32_t* kv_indices;
    int64_t num_indices;
    const int32_t* kv_indptr;
    const int32_t* seq_lens;
    int32_t num_parents;
    const int32_t* parents;
    const int32_t* new_tokens;
    int32_t num_requests;
    const int32_t* free_slots;
    int64_t num_free;
    const int32_t* cursor;
    int64_t pool_rows;
    const int32_t* prefix_len;
    int32_t* new_indices;
    int64_t total;
    int32_t* new_indptr;
    int32_t* new_lens;
    int32_t* slots;
    int32_t* positions;
    int64_t num_tokens;
    int32_t* token_indptr;
    int32_t* new_cursor;
    uint32_t* err;
};

// What request f keeps: entries [from, from + length) of kv_indices.
struct Kept {
    int32_t from, length;
};

__device__ __forceinline__ Kept kept_of(const ExtendArgs& a, int f, uint32_t& bad)
{
    const int p = a.parents == nullptr ? f : __ldg(a.parents + f);
    if (p < 0 || p >= a.num_parents) {
        bad |= MLA_DEVERR_BAD_TABLE;
        return Kept{0, 0};
    }
    const int64_t from = __ldg(a.kv_indptr + p), to = __ldg(a.kv_indptr + p + 1);
    const int64_t want = __ldg(a.seq_lens + p);
    if (from < 0 || to > a.num_indices || to < from) {
        bad |= MLA_DEVERR_BAD_TABLE;
        return Kept{0, 0};
    }
    const int64_t len = want < 0 ? 0 : want > to - from ? to - from : want;
    if (len != want) bad |= MLA_DEVERR_BAD_LENGTH;
    return Kept{(int32_t)from, (int32_t)len};
}

// a + b, or 2^32 - 1 where that is less: sums of lengths and counts, whose use is
// bounded by less than 2^31.
__device__ __forceinline__ uint32_t add_up(uint32_t a, uint32_t b)
{
    const uint32_t s = a + b;
    return s < a ? 0xFFFFFFFFu : s;
}

__device__ __forceinline__ uint32_t warp_scan(uint32_t v, int lane)
{
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v = add_up(v, u);
    }
    return v;
}

// Sum of the threads before this one's, and of all; `part` holds one sum per warp.
template <int WARPS>
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* part, uint32_t& all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t sum = warp_scan(v, lane);
    uint32_t before = __shfl_up_sync(0xffffffffu, sum, 1);
    if (lane == 0) before = 0;
    __syncthreads();
    if (lane == 31) part[warp] = sum;
    __syncthreads();
    const uint32_t w = warp_scan(lane < WARPS ? part[lane] : 0u, lane);
    all = __shfl_sync(0xffffffffu, w, 31);
    const uint32_t warps = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return warp > 0 ? add_up(warps, before) : before;
}

// The number of the token's free slot, in 32 bits as the cursor, to its slot (-1: none).
__device__ __forceinline__ int32_t free_slot(const ExtendArgs& a, int32_t number, uint32_t& bad)
{
    if (number < 0 || number >= (a.free_slots == nullptr ? a.pool_rows : a.num_free)) {
        bad |= MLA_DEVERR_NO_SLOT;
        return -1;
    }
    const int32_t slot = a.free_slots == nullptr ? number : __ldg(a.free_slots + number);
    if (slot >= 0 && slot < a.pool_rows) return slot;
    bad |= MLA_DEVERR_BAD_SLOT;
    return -1;
}

// The last f in [lo, hi) with start[f] <= i (start[lo] <= i).
__device__ __forceinline__ int last_at_most(const int32_t* start, int lo, int hi, int32_t i)
{
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

// CTA 0 writes what is per request, and with `spread` false all of what is per token,
// so that it alone reads the cursor that it then moves (which may be one and the
// same); the others copy.
__global__ void __launch_bounds__(kExtendThreads)
extend_kernel(const ExtendArgs a, bool spread, bool move_cursor)
{
    extern __shared__ int32_t sums[];
    __shared__ uint32_t part[kExtendThreads / 32];
    wait_for_predecessor();
    allow_dependents();
    const int tid = threadIdx.x, lane = tid & 31, F = a.num_requests;
    int32_t* const start = sums;              // [F + 1] of the new table
    int32_t* const token = start + F + 1;     // [F + 1] tokens before
    int32_t* const length = token + F + 1;    // [F] kept
    int32_t* const from = length + F;         // [F] kv_indices of the new table's entry 0
    const bool lead = blockIdx.x == 0;
    const uint32_t room = (uint32_t)a.total, token_room = (uint32_t)a.num_tokens;
    uint32_t bad = 0;
    for (int f = tid; f < F; f += kExtendThreads) {
        int n = a.new_tokens == nullptr ? 1 : __ldg(a.new_tokens + f);
        if (n < 0) {
            n = 0;
            bad |= MLA_DEVERR_BAD_LENGTH;
        }
        const Kept k = kept_of(a, f, bad);
        token[f] = n;
        length[f] = k.length;
        from[f] = k.from;
    }
    __syncthreads();
    const int per = (F + kExtendThreads - 1) / kExtendThreads;
    const int f0 = min(tid * per, F), f1 = min(f0 + per, F);
    uint32_t mine = 0, all;
    for (int f = f0; f < f1; ++f) mine = add_up(mine, token[f]);
    uint32_t at = block_scan<kExtendThreads / 32>(mine, part, all);
    for (int f = f0; f < f1; ++f) {
        const uint32_t n = token[f];
        token[f] = (int32_t)min(at, token_room);
        at = add_up(at, n);
    }
    if (all > token_room) bad |= MLA_DEVERR_BAD_TABLE;
    const int tokens = (int)min(all, token_room);
    if (tid == 0) token[F] = tokens;
    __syncthreads();
    mine = 0;
    for (int f = f0; f < f1; ++f) mine = add_up(mine, length[f] + (token[f + 1] - token[f]));
    at = block_scan<kExtendThreads / 32>(mine, part, all);
    for (int f = f0; f < f1; ++f) {
        start[f] = (int32_t)min(at, room);
        from[f] -= start[f];
        at = add_up(at, length[f] + (token[f + 1] - token[f]));
    }
    if (all > room) bad |= MLA_DEVERR_BAD_TABLE;
    const int32_t total = (int32_t)min(all, room);
    if (tid == 0) start[F] = total;
    __syncthreads();

    if (lead || spread) {
        const int step = spread ? (int)gridDim.x * kExtendThreads : kExtendThreads;
        const int32_t cursor = a.num_tokens > 0 ? __ldg(a.cursor) : 0;
        const int32_t prefix = a.prefix_len == nullptr ? 0 : __ldg(a.prefix_len);
        for (int64_t t = (int64_t)(spread ? blockIdx.x : 0) * kExtendThreads + tid; t < a.num_tokens;
             t += step) {
            int32_t slot = -1, position = 0;
            if (t < tokens) {
                const int f = last_at_most(token, 0, F, (int32_t)t);
                const int32_t j = length[f] + ((int32_t)t - token[f]);
                position = j + prefix;
                if (j < start[f + 1] - start[f]) {
                    slot = free_slot(a, (int32_t)((uint32_t)cursor + (uint32_t)t), bad);
                    a.new_indices[start[f] + j] = slot;
                }
            }
            a.slots[t] = slot;
            a.positions[t] = position;
        }
    }
    if (lead) {
        for (int f = tid; f <= F; f += kExtendThreads) {
            a.new_indptr[f] = start[f];
            a.token_indptr[f] = token[f];
            if (f < F) a.new_lens[f] = start[f + 1] - start[f];
        }
        if (move_cursor) {
            const uint32_t c = tid == 0 ? (uint32_t)a.cursor[0] : 0;
            __syncthreads();   // every thread has read it
            if (tid == 0) a.new_cursor[0] = (int32_t)(c + (uint32_t)tokens);
        }
        if (bad != 0) atomicOr(a.err, bad);
        return;
    }
    if (spread && (bad & (MLA_DEVERR_NO_SLOT | MLA_DEVERR_BAD_SLOT)) != 0) atomicOr(a.err, bad);

    // a warp's part of the table, and the requests in it
    constexpr int kSpan = 32 * kExtendSpan;   // entries at a time
    const int warps = ((int)gridDim.x - 1) * (kExtendThreads / 32);
    const int warp = ((int)blockIdx.x - 1) * (kExtendThreads / 32) + (tid >> 5);
    const int64_t run = ((int64_t)total + (int64_t)warps * kSpan - 1) / ((int64_t)warps * kSpan) * kSpan;
    const int64_t begin = warp * run;
    if (begin >= total) return;
    const int32_t end = (int32_t)min(begin + run, (int64_t)total);
    int lo = last_at_most(start, 0, F, (int32_t)begin);
    for (int32_t i0 = (int32_t)begin; i0 < end; i0 += kSpan) {
        const int32_t past = min(i0 + kSpan, end);
        if (start[lo + 1] <= i0) lo = last_at_most(start, lo + 1, F, i0);
        int32_t v[kExtendSpan];
        if (start[lo + 1] >= past) {   // one request's
            const int32_t until = min(past, start[lo] + length[lo]);
            const int32_t* src = a.kv_indices + from[lo];
#pragma unroll
            for (int k = 0; k < kExtendSpan; ++k) {
                const int32_t i = i0 + 32 * k + lane;
                if (i < until) v[k] = __ldg(src + i);
            }
#pragma unroll
            for (int k = 0; k < kExtendSpan; ++k) {
                const int32_t i = i0 + 32 * k + lane;
                if (i < until) a.new_indices[i] = v[k];
            }
            continue;
        }
        const int hi = last_at_most(start, lo, F, past - 1) + 1;
        bool kept[kExtendSpan];
#pragma unroll
        for (int k = 0; k < kExtendSpan; ++k) {
            const int32_t i = i0 + 32 * k + lane;
            kept[k] = i < past;
            if (kept[k]) {
                const int f = last_at_most(start, lo, hi, i);
                kept[k] = i - start[f] < length[f];
                if (kept[k]) v[k] = __ldg(a.kv_indices + (from[f] + i));
            }
        }
#pragma unroll
        for (int k = 0; k < kExtendSpan; ++k)
            if (kept[k]) a.new_indices[i0 + 32 * k + lane] = v[k];
    }
}

// The cursor in place, when every CTA of the kernel before has read it.
__global__ void cursor_kernel(const ExtendArgs a)
{
    wait_for_predecessor();
    allow_dependents();
    a.new_cursor[0] = (int32_t)((uint32_t)a.cursor[0] + (uint32_t)a.token_indptr[a.num_requests]);
}

__global__ void __launch_bounds__(kSumThreads)
sums_kernel(const ExtendArgs a)
{
    __shared__ uint32_t part[32];
    wait_for_predecessor();
    allow_dependents();
    const int tid = threadIdx.x;
    const uint32_t room = (uint32_t)a.total, token_room = (uint32_t)a.num_tokens;
    uint32_t tokens = 0, entries = 0;   // of the requests before this turn's
    uint32_t bad = 0;
    for (int f0 = 0; f0 < a.num_requests; f0 += kSumThreads) {
        const int f = f0 + tid;
        uint32_t n = 0, length = 0;
        if (f < a.num_requests) {
            const int32_t want = a.new_tokens == nullptr ? 1 : __ldg(a.new_tokens + f);
            n = max(want, 0);
            if (want < 0) bad |= MLA_DEVERR_BAD_LENGTH;
            length = kept_of(a, f, bad).length;
        }
        uint32_t all;
        const uint32_t t = add_up(tokens, block_scan<kSumThreads / 32>(n, part, all));
        const uint32_t first_token = min(t, token_room);
        length += min(add_up(t, n), token_room) - first_token;
        tokens = add_up(tokens, all);
        const uint32_t e = add_up(entries, block_scan<kSumThreads / 32>(length, part, all));
        const uint32_t first = min(e, room);
        entries = add_up(entries, all);
        if (f < a.num_requests) {
            a.token_indptr[f] = (int32_t)first_token;
            a.new_indptr[f] = (int32_t)first;
            a.new_lens[f] = (int32_t)(min(add_up(e, length), room) - first);
        }
    }
    if (tokens > token_room || entries > room) bad |= MLA_DEVERR_BAD_TABLE;
    if (tid == 0) {
        const uint32_t n = min(tokens, token_room);
        a.token_indptr[a.num_requests] = (int32_t)n;
        a.new_indptr[a.num_requests] = (int32_t)min(entries, room);
        // modulo 2^32, so that fill has the cursor from the new one
        a.new_cursor[0] = (int32_t)((uint32_t)a.cursor[0] + n);
    }
    if (bad != 0) atomicOr(a.err, bad);
}

// The last f with indptr[f] <= i, of n >= 1 (indptr[0] <= i).
__device__ __forceinline__ int find_request(const int32_t* indptr, int n, int64_t i)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldcg(indptr + mid) <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kFillThreads)
fill_kernel(const ExtendArgs a, uint32_t entry_ctas)
{
    wait_for_predecessor();
    allow_dependents();
    const int F = a.num_requests;
    uint32_t bad = 0;
    if (blockIdx.x < entry_ctas) {
        const int64_t i = (int64_t)blockIdx.x * kFillThreads + threadIdx.x;
        if (i >= __ldcg(a.new_indptr + F)) return;
        const int f = find_request(a.new_indptr, F, i);
        const Kept k = kept_of(a, f, bad);
        const int64_t j = i - __ldcg(a.new_indptr + f);
        if (j < k.length) a.new_indices[i] = __ldg(a.kv_indices + k.from + j);
        return;
    }
    const int64_t t = (int64_t)(blockIdx.x - entry_ctas) * kFillThreads + threadIdx.x;
    if (t >= a.num_tokens) return;
    const int32_t tokens = __ldcg(a.token_indptr + F);
    int32_t slot = -1, position = 0;
    if (t < tokens) {
        const int f = find_request(a.token_indptr, F, t);
        const Kept k = kept_of(a, f, bad);
        bad = 0;   // the sums have told
        const int64_t j = k.length + (t - __ldcg(a.token_indptr + f));
        position = (int32_t)(j + (a.prefix_len == nullptr ? 0 : __ldg(a.prefix_len)));
        if (j < __ldcg(a.new_lens + f)) {
            slot = free_slot(a, (int32_t)((uint32_t)__ldcg(a.new_cursor) - (uint32_t)tokens + (uint32_t)t),
                             bad);
            a.new_indices[__ldcg(a.new_indptr + f) + j] = slot;
        }
    }
    a.slots[t] = slot;
    a.positions[t] = position;
    if (bad != 0) atomicOr(a.err, bad);
}

// Whether n bytes at p and m bytes at q have one in common.
bool overlap(const void* p, int64_t n, const void* q, int64_t m)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p != nullptr && q != nullptr && n > 0 && m > 0 && a < b + (uintptr_t)m &&
           b < a + (uintptr_t)n;
}

// Whether two sets of rows of `bytes` have one in common: n rows at p, `ps` apart, and m
// at q, `qs` apart.  Rows of one stride may lie between one another; otherwise sets
// that reach into each other are taken to have one.
bool rows_overlap(const void* p, int64_t n, int64_t ps, const void* q, int64_t m, int64_t qs,
                  int64_t bytes)
{
    if (n < 1 || m < 1 || bytes < 1 ||
        !overlap(p, (n - 1) * ps + bytes, q, (m - 1) * qs + bytes))
        return false;
    if (ps != qs || ps < 1) return true;
    const int64_t d = reinterpret_cast<const char*>(q) - reinterpret_cast<const char*>(p);
    const int64_t in = (d % ps + ps) % ps;   // of a row of q in the rows of p
    return in < bytes || ps - in < bytes;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

int64_t mla_beam_select_workspace_bytes(int32_t batch, int32_t beams, int32_t vocab)
{
    if (!select_shape_ok(batch, beams, vocab)) return 0;
    const int64_t rows = (int64_t)batch * beams;
    return MLA_WORKSPACE_HEADER_BYTES + select_part_bytes(rows, vocab) +
           align256(rows * select_groups(vocab) * 4);
}

int mla_beam_select(const void* logits, int32_t dtype, int64_t row_stride, const float* scores,
                    const uint8_t* finished, int32_t batch, int32_t beams, int32_t vocab,
                    int32_t num_select, int32_t end_token, int32_t* tokens, int32_t* parents,
                    float* scores_out, uint8_t* finished_out, void* workspace,
                    int64_t workspace_bytes, void* stream)
{
    if (batch < 0 || beams < 1 || vocab < 1 || num_select < 1) return MLA_ERR_INVALID_ARG;
    if (dtype != MLA_DTYPE_BF16 && dtype != MLA_DTYPE_F16 && dtype != MLA_DTYPE_F32)
        return MLA_ERR_INVALID_ARG;
    if (end_token < -1 || end_token >= vocab || (finished != nullptr && end_token < 0))
        return MLA_ERR_INVALID_ARG;
    if (num_select > MLA_MAX_BEAMS) return MLA_ERR_UNSUPPORTED_SHAPE;
    if (batch == 0) return MLA_OK;
    if (!select_shape_ok(batch, beams, vocab)) return MLA_ERR_UNSUPPORTED_SHAPE;
    const int64_t rows = (int64_t)batch * beams;
    const int64_t picks = (int64_t)batch * num_select;
    if (!logits || !scores || !tokens || !parents || !scores_out || row_stride < 0)
        return MLA_ERR_INVALID_ARG;
    if ((overlap(scores_out, picks * 4, scores, rows * 4) &&
         (scores_out != scores || num_select != beams)) ||
        (overlap(finished_out, picks, finished, rows) &&
         (finished_out != finished || num_select != beams)))
        return MLA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(logits) & (dtype == MLA_DTYPE_F32 ? 3u : 1u)) != 0)
        return MLA_ERR_MISALIGNED;
    int rc = check_header(workspace, workspace_bytes);
    if (rc != MLA_OK) return rc;
    if (workspace_bytes < mla_beam_select_workspace_bytes(batch, beams, vocab))
        return MLA_ERR_WORKSPACE_TOO_SMALL;
    rc = device_ok();
    if (rc != MLA_OK) return rc;

    SelectArgs a{};
    a.logits = logits;
    a.row_stride = row_stride;
    a.scores = scores;
    a.finished = finished;
    a.batch = batch;
    a.beams = beams;
    a.vocab = vocab;
    a.select = num_select;
    a.end_token = end_token;
    a.groups = (int32_t)select_groups(vocab);
    a.rows = rows;
    char* p = static_cast<char*>(workspace);
    a.err = reinterpret_cast<uint32_t*>(p);
    a.parts = reinterpret_cast<float2*>(p + MLA_WORKSPACE_HEADER_BYTES);
    a.group_max = reinterpret_cast<float*>(p + MLA_WORKSPACE_HEADER_BYTES +
                                           select_part_bytes(rows, vocab));
    a.tokens = tokens;
    a.parents = parents;
    a.scores_out = scores_out;
    a.finished_out = finished_out;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return status_of(dtype == MLA_DTYPE_F32   ? launch_select_of<float>(a, s)
                     : dtype == MLA_DTYPE_F16 ? launch_select_of<__half>(a, s)
                                              : launch_select_of<__nv_bfloat16>(a, s));
}

int mla_beam_reorder(const void* state, int64_t state_stride, int32_t num_parents,
                     int64_t row_bytes, int32_t elem_bytes, const int32_t* parents,
                     int32_t num_rows, const int32_t* lens, const int32_t* tokens, void* out,
                     int64_t out_stride, int32_t* out_lens, void* workspace,
                     int64_t workspace_bytes, void* stream)
{
    if (num_parents < 0 || num_rows < 0 || row_bytes < 0 || state_stride < 0 || out_stride < 0)
        return MLA_ERR_INVALID_ARG;
    if (elem_bytes != 1 && elem_bytes != 2 && elem_bytes != 4 && elem_bytes != 8)
        return MLA_ERR_UNSUPPORTED_SHAPE;
    if (row_bytes % elem_bytes != 0 || row_bytes / elem_bytes > INT32_MAX)
        return MLA_ERR_UNSUPPORTED_SHAPE;
    if (((tokens != nullptr || out_lens != nullptr) && lens == nullptr) ||
        (out_lens != nullptr && out_lens == lens))
        return MLA_ERR_INVALID_ARG;
    if (tokens != nullptr && elem_bytes != 4) return MLA_ERR_UNSUPPORTED_SHAPE;
    if (num_rows == 0) return MLA_OK;
    if (!parents || (row_bytes > 0 && (!out || (num_parents > 0 && !state))) ||
        (num_rows > 1 && out_stride < row_bytes) ||
        rows_overlap(state, num_parents, state_stride, out, num_rows, out_stride, row_bytes))
        return MLA_ERR_INVALID_ARG;
    uintptr_t bits = reinterpret_cast<uintptr_t>(state) | reinterpret_cast<uintptr_t>(out);
    if (num_parents > 1) bits |= (uintptr_t)state_stride;
    if (num_rows > 1) bits |= (uintptr_t)out_stride;
    if (tokens != nullptr && (bits & 3u) != 0) return MLA_ERR_MISALIGNED;
    int rc = check_header(workspace, workspace_bytes);
    if (rc != MLA_OK) return rc;
    rc = device_ok();
    if (rc != MLA_OK) return rc;

    ReorderArgs a{static_cast<const uint8_t*>(state), state_stride, num_parents, row_bytes,
                  elem_bytes, parents, num_rows, lens, tokens, static_cast<uint8_t*>(out),
                  out_stride, out_lens, 1, static_cast<uint32_t*>(workspace)};
    const int unit = (bits & 15u) == 0 ? 16 : (bits & 7u) == 0 ? 8 : (bits & 3u) == 0 ? 4
                                                       : (bits & 1u) == 0 ? 2 : 1;
    const int64_t per = (int64_t)unit * kReorderThreads * kReorderTurns;
    const int64_t parts = (row_bytes + per - 1) / per;
    const int64_t most = INT32_MAX / num_rows;   // CTAs of the grid; a CTA loops over the rest
    a.parts = (uint32_t)(parts < 1 ? 1 : parts < most ? parts : most);
    const dim3 grid((unsigned)(a.parts * (uint32_t)num_rows));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto* kernel = unit == 16  ? reorder_kernel<uint4>
                   : unit == 8 ? reorder_kernel<uint2>
                   : unit == 4 ? reorder_kernel<uint32_t>
                   : unit == 2 ? reorder_kernel<uint16_t>
                               : reorder_kernel<uint8_t>;
    return status_of(launch_dependent(kernel, grid, kReorderThreads, s, true, a));
}

int mla_cache_extend(const int32_t* kv_indices, int64_t num_indices, const int32_t* kv_indptr,
                     const int32_t* seq_lens, int32_t num_parents, const int32_t* parents,
                     const int32_t* new_tokens, int32_t num_requests, const int32_t* free_slots,
                     int64_t num_free, const int32_t* cursor, int64_t pool_rows,
                     const int32_t* prefix_len, int32_t* new_indices, int64_t total,
                     int32_t* new_indptr, int32_t* new_lens, int32_t* slots, int32_t* positions,
                     int64_t num_tokens, int32_t* token_indptr, int32_t* new_cursor,
                     void* workspace, int64_t workspace_bytes, void* stream)
{
    if (num_indices < 0 || num_parents < 0 || num_requests < 0 || num_free < 0 || pool_rows < 0 ||
        total < 0 || num_tokens < 0)
        return MLA_ERR_INVALID_ARG;
    if (num_indices > INT32_MAX || total > INT32_MAX || num_tokens > INT32_MAX ||
        pool_rows > INT32_MAX || num_free > INT32_MAX)
        return MLA_ERR_UNSUPPORTED_SHAPE;
    if (!kv_indptr || !cursor || !new_indptr || !token_indptr || !new_cursor ||
        (num_indices > 0 && !kv_indices) || (num_parents > 0 && !seq_lens) ||
        (num_requests > 0 && !new_lens) || (total > 0 && !new_indices) ||
        (num_tokens > 0 && (!slots || !positions)))
        return MLA_ERR_INVALID_ARG;
    if (parents == nullptr && num_requests > num_parents) return MLA_ERR_INVALID_ARG;
    struct Range {
        const void* p;
        int64_t n;
    };
    const int64_t F = num_requests, P = num_parents;
    const Range in[] = {{kv_indices, num_indices}, {kv_indptr, P + 1}, {seq_lens, P}, {parents, F},
                        {new_tokens, F}, {free_slots, num_free}, {cursor, 1}, {prefix_len, 1}};
    const Range out[] = {{new_indices, total}, {new_indptr, F + 1}, {new_lens, F},
                         {slots, num_tokens}, {positions, num_tokens}, {token_indptr, F + 1},
                         {new_cursor, 1}};
    for (const Range& o : out)
        for (const Range& i : in)
            if (overlap(o.p, o.n * 4, i.p, i.n * 4) && !(o.p == new_cursor && i.p == cursor))
                return MLA_ERR_INVALID_ARG;
    int rc = check_header(workspace, workspace_bytes);
    if (rc != MLA_OK) return rc;
    rc = device_ok();
    if (rc != MLA_OK) return rc;

    const ExtendArgs a{kv_indices, num_indices, kv_indptr, seq_lens, num_parents, parents,
                       new_tokens, num_requests, free_slots, num_free, cursor, pool_rows,
                       prefix_len, new_indices, total, new_indptr, new_lens, slots, positions,
                       num_tokens, token_indptr, new_cursor, static_cast<uint32_t*>(workspace)};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (num_requests <= kExtendRequests) {
        const int64_t per = kExtendThreads * kExtendSpan;
        const int64_t most = (total + per - 1) / per;
        const bool spread = num_tokens > kLeadTokens;
        const bool in_place = new_cursor == cursor;
        const dim3 grid((unsigned)(1 + (most < 1 ? 1 : most < kExtendCtas ? most : kExtendCtas)));
        const int bytes = (4 * num_requests + 2) * 4;
        cudaError_t e = launch_dependent_shared(extend_kernel, grid, kExtendThreads, bytes, s, true, a,
                                                spread, !(spread && in_place));
        if (e == cudaSuccess && spread && in_place)
            e = launch_dependent(cursor_kernel, dim3(1), 1, s, true, a);
        return status_of(e);
    }
    cudaError_t e = launch_dependent(sums_kernel, dim3(1), kSumThreads, s, true, a);
    const int64_t entry_ctas = num_requests == 0 ? 0 : (total + kFillThreads - 1) / kFillThreads;
    const int64_t token_ctas = (num_tokens + kFillThreads - 1) / kFillThreads;
    if (e == cudaSuccess && entry_ctas + token_ctas > 0)
        e = launch_dependent(fill_kernel, dim3((unsigned)(entry_ctas + token_ctas)), kFillThreads, s,
                             true, a, (uint32_t)entry_ctas);
    return status_of(e);
}

}  // extern "C"
