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
constexpr int kPieces = 8;              // 16-byte loads of a lane per segment
constexpr int kScanThreads = 256;
constexpr int kPickThreads = 1024;
constexpr int kPickList = 1024;
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

template <typename T>
constexpr int kSegment = kPieces * 32 * kElements<T>;   // columns

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

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kScanThreads)
scan_kernel(const SelectArgs a)
{
    constexpr int E = kElements<T>;
    constexpr int kPerGroup = kGroup / (32 * E);         // pieces of a group
    constexpr int kGroups = kPieces / kPerGroup;         // groups of a segment
    wait_for_predecessor();
    allow_dependents();
    const int lane = threadIdx.x & 31;
    const uint32_t id = blockIdx.x * (kScanThreads / 32) + (threadIdx.x >> 5);   // below 2^31
    const int64_t row = id / (uint32_t)a.segments;
    const int seg = (int)(id % (uint32_t)a.segments);
    if (row >= a.rows || !row_is_live(a, row)) return;
    const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
    const int c0 = seg * kSegment<T> + lane * E;
    uint4 v[kPieces];
#pragma unroll
    for (int p = 0; p < kPieces; ++p) v[p] = load_piece<T, ALIGNED>(x, c0 + p * 32 * E, a.vocab);

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
    for (int p = 0; p < kPieces; ++p)
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

// A candidate as a number: its score, then the lower index; 0: none.
__device__ __forceinline__ uint64_t candidate(float score, uint32_t index)
{
    if (!(score > -INFINITY)) return 0;
    const uint32_t s = (uint32_t)ordered(score + 0.f) ^ 0x80000000u;   // -0 as +0
    return (uint64_t)s << 32 | (0xFFFFFFFFu - index);
}

__device__ __forceinline__ uint32_t index_of(uint64_t c) { return 0xFFFFFFFFu - (uint32_t)c; }

__device__ __forceinline__ float score_of(uint64_t c)
{
    return from_ordered((int)((uint32_t)(c >> 32) ^ 0x80000000u));
}

__device__ __forceinline__ uint64_t candidate_of(float2 base, float x, uint32_t index)
{
    if (x == -INFINITY) return 0;
    const float2 s = two_sum(base.x, x);
    return candidate(__fadd_rn(s.x, __fadd_rn(s.y, base.y)), index);
}

__device__ __forceinline__ uint64_t warp_max(uint64_t v)
{
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return (uint64_t)hi << 32 | lo;
}

struct Picker {
    uint64_t best[kPickThreads / 32];   // of each warp
    uint64_t list[kPickList];
    uint64_t taken[MLA_MAX_BEAMS];
    uint64_t least;
    int count;
};

// The K largest of the CTA's candidates (distinct numbers, 0 for none) in p.taken, in
// order.  each(f) calls f for each of this thread's.  With K of 32 warps' best at hand,
// all of the K largest are at or above the K-th of those: what is, is listed and
// ranked by counting.  A list that would overflow (one warp holds most of them, and
// many) is not used: the K are taken one after the other.
template <class Each>
__device__ __forceinline__ void pick_best(Picker& p, int K, Each&& each)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint64_t best = 0;
    each([&](uint64_t c) { best = c > best ? c : best; });
    best = warp_max(best);
    if (lane == 0) p.best[warp] = best;
    if (tid == 0) {
        p.count = 0;
        p.least = 1;
    }
    __syncthreads();
    if (warp == 0) {
        const uint64_t mine = p.best[lane];
        int rank = 0;
#pragma unroll
        for (int w = 0; w < kPickThreads / 32; ++w) rank += p.best[w] > mine ? 1 : 0;
        if (rank == K - 1 && mine != 0) p.least = mine;
    }
    __syncthreads();
    const uint64_t least = p.least;
    each([&](uint64_t c) {
        if (c >= least) {
            const int at = atomicAdd(&p.count, 1);
            if (at < kPickList) p.list[at] = c;
        }
    });
    __syncthreads();
    const int n = p.count;
    if (n <= kPickList) {
        if (tid < n) {
            const uint64_t mine = p.list[tid];
            int rank = 0;
            for (int i = 0; i < n; ++i) rank += p.list[i] > mine ? 1 : 0;
            if (rank < K) p.taken[rank] = mine;
        }
        if (tid >= n && tid < K) p.taken[tid] = 0;
    } else {
        uint64_t last = ~0ull;
        for (int k = 0; k < K; ++k) {
            uint64_t next = 0;
            each([&](uint64_t c) { next = c < last && c > next ? c : next; });
            next = warp_max(next);
            __syncthreads();
            if (lane == 0) p.best[warp] = next;
            __syncthreads();
            last = warp_max(p.best[lane]);
            if (tid == 0) p.taken[k] = last;
        }
    }
    __syncthreads();
}

enum : int { kRowDead = 0, kRowLive = 1, kRowEnded = 2 };

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kPickThreads)
pick_kernel(const SelectArgs a)
{
    constexpr int E = kElements<T>;
    constexpr int kPerGroup = kGroup / (32 * E);
    __shared__ Picker p;
    __shared__ float2 base[MLA_MAX_BEAMS];   // (own score, -) of a beam that has ended
    __shared__ int state[MLA_MAX_BEAMS];
    wait_for_predecessor();
    allow_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row0 = (int64_t)blockIdx.x * a.beams;
    const int K = a.select;

    if (warp < a.beams) {
        const int64_t row = row0 + warp;
        const float own = a.scores[row];
        const bool ended = a.finished != nullptr && a.finished[row] != 0;
        float m = -INFINITY, s = 0.f;
        if (own != -INFINITY && !ended) {
            const float2* parts = a.parts + row * a.segments;
            for (int i = lane; i < a.segments; i += 32) m = fmaxf(m, __ldcg(&parts[i]).x);
            m = from_ordered(__reduce_max_sync(0xffffffffu, ordered(m)));
            const float ref = m == -INFINITY ? 0.f : m;
            constexpr float kLog2e = 1.4426950408889634f;
            for (int i = lane; i < a.segments; i += 32) {
                const float2 t = __ldcg(&parts[i]);
                s += t.y * ex2_approx((t.x - ref) * kLog2e);
            }
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        }
        if (lane == 0) {
            // a NaN or +inf among the logits makes the sum one
            const bool bad = !(own < INFINITY) || (!ended && own != -INFINITY && !(s < INFINITY));
            if (bad) atomicOr(a.err, MLA_DEVERR_BAD_LOGITS);
            const bool dead = bad || own == -INFINITY || (!ended && s == 0.f);
            state[warp] = dead ? kRowDead : ended ? kRowEnded : kRowLive;
            base[warp] = dead || ended ? make_float2(own, 0.f) : row_base(own, m, s);
        }
    }
    __syncthreads();

    const uint32_t items = (uint32_t)a.beams * (uint32_t)a.groups;
    pick_best(p, K, [&](auto&& take) {
        for (uint32_t i = tid; i < items; i += kPickThreads) {
            const uint32_t w = i / (uint32_t)a.groups;
            const int st = state[w];
            if (st == kRowLive)
                take(candidate_of(base[w], __ldcg(a.group_max + row0 * a.groups + i), i));
            else if (st == kRowEnded && i == w * a.groups)
                take(candidate(base[w].x, i));
        }
    });

    // a warp's group, eight logits a lane
    uint64_t c[kPerGroup * E];
#pragma unroll
    for (int i = 0; i < kPerGroup * E; ++i) c[i] = 0;
    const uint64_t mine = warp < K ? p.taken[warp] : 0;
    if (mine != 0) {
        const uint32_t g = index_of(mine);
        const uint32_t w = g / (uint32_t)a.groups;
        if (state[w] == kRowEnded) {
            if (lane == 0) c[0] = candidate(base[w].x, w * a.vocab + a.end_token);
        } else {
            const T* x = static_cast<const T*>(a.logits) + (row0 + w) * a.row_stride;
            const int col = (int)(g - w * a.groups) * kGroup + lane * E;
            const float2 b = base[w];
#pragma unroll
            for (int q = 0; q < kPerGroup; ++q) {
                const int c0 = col + q * 32 * E;
                const uint4 v = load_piece<T, ALIGNED>(x, c0, a.vocab);
                each_logit<T>(v, [&](int i, float t) {
                    c[q * E + i] = candidate_of(b, t, w * a.vocab + c0 + i);
                });
            }
        }
    }
    __syncthreads();   // everyone has read taken
    pick_best(p, K, [&](auto&& take) {
#pragma unroll
        for (int i = 0; i < kPerGroup * E; ++i) take(c[i]);
    });

    if (tid < K) {
        const uint64_t t = p.taken[tid];
        const int64_t at = (int64_t)blockIdx.x * K + tid;
        int token = -1, w = 0;
        float score = -INFINITY;
        bool end = true;
        if (t != 0) {
            const uint32_t i = index_of(t);
            w = (int)(i / (uint32_t)a.vocab);
            token = (int)(i - (uint32_t)w * a.vocab);
            score = score_of(t);
            end = token == a.end_token || state[w] == kRowEnded;
        }
        a.tokens[at] = token;
        a.parents[at] = (int32_t)(row0 + w);
        a.scores_out[at] = score;
        if (a.finished_out != nullptr) a.finished_out[at] = end ? 1 : 0;
    }
}

template <typename T, bool ALIGNED>
cudaError_t launch_select(SelectArgs a, cudaStream_t s)
{
    a.segments = (a.vocab + kSegment<T> - 1) / kSegment<T>;
    const int64_t warps = a.rows * a.segments;
    const int64_t ctas = (warps + kScanThreads / 32 - 1) / (kScanThreads / 32);
    cudaError_t e = launch_dependent(scan_kernel<T, ALIGNED>, dim3((unsigned)ctas), kScanThreads, s,
                                     true, a);
    if (e == cudaSuccess)
        e = launch_dependent(pick_kernel<T, ALIGNED>, dim3((unsigned)a.batch), kPickThreads, s, true,
                             a);
    return e;
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

// Bytes of the segments' parts (most for fp32, whose segments are shortest).
int64_t select_part_bytes(int64_t rows, int64_t vocab)
{
    const int64_t n = kSegment<float>;
    return align256(rows * ((vocab + n - 1) / n) * (int64_t)sizeof(float2));
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
// sums   (one CTA) the requests' lengths and counts, their sums, the cursor;
// fill   a thread per entry of the new table and per token.
// Bytes: 8 per entry that is kept, 12 (16 with a list of free slots) per token.

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

__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane)
{
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += u;
    }
    return v;
}

// Inclusive sums over the CTA's threads; `part` holds one sum per warp.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* part, int64_t& all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = warp_scan(v, lane);
    __syncthreads();
    if (lane == 31) part[warp] = v;
    __syncthreads();
    const int64_t w = warp_scan(part[lane], lane);
    all = __shfl_sync(0xffffffffu, w, 31);
    const int64_t before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return v + (warp > 0 ? before : 0);
}

__global__ void __launch_bounds__(kSumThreads)
sums_kernel(const ExtendArgs a)
{
    __shared__ int64_t part[32];
    wait_for_predecessor();
    allow_dependents();
    const int tid = threadIdx.x;
    int64_t tokens = 0, entries = 0;   // of the requests before this turn's
    uint32_t bad = 0;
    for (int f0 = 0; f0 < a.num_requests; f0 += kSumThreads) {
        const int f = f0 + tid;
        int64_t n = 0, length = 0;
        if (f < a.num_requests) {
            n = a.new_tokens == nullptr ? 1 : __ldg(a.new_tokens + f);
            if (n < 0) {
                n = 0;
                bad |= MLA_DEVERR_BAD_LENGTH;
            }
            length = kept_of(a, f, bad).length;
        }
        int64_t all;
        const int64_t last = tokens + block_scan(n, part, all);
        const int64_t begin = min(last - n, a.num_tokens), end = min(last, a.num_tokens);
        if (end - begin != n) bad |= MLA_DEVERR_BAD_TABLE;
        tokens += all;
        length += end - begin;
        const int64_t until = entries + block_scan(length, part, all);
        const int64_t first = min(until - length, a.total), past = min(until, a.total);
        if (past - first != length) bad |= MLA_DEVERR_BAD_TABLE;
        entries += all;
        if (f < a.num_requests) {
            a.token_indptr[f] = (int32_t)begin;
            a.new_indptr[f] = (int32_t)first;
            a.new_lens[f] = (int32_t)(past - first);
        }
    }
    if (tid == 0) {
        const int64_t n = min(tokens, a.num_tokens);
        a.token_indptr[a.num_requests] = (int32_t)n;
        a.new_indptr[a.num_requests] = (int32_t)min(entries, a.total);
        // modulo 2^32, so that fill has the cursor from the new one
        a.new_cursor[0] = (int32_t)((uint32_t)a.cursor[0] + (uint32_t)n);
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
            // the number of the free slot, in 32 bits as the cursor
            const int64_t number = (int32_t)((uint32_t)__ldcg(a.new_cursor) - (uint32_t)tokens +
                                             (uint32_t)t);
            if (number < 0 || number >= (a.free_slots == nullptr ? a.pool_rows : a.num_free)) {
                bad = MLA_DEVERR_NO_SLOT;
            } else {
                slot = a.free_slots == nullptr ? (int32_t)number : __ldg(a.free_slots + number);
                if (slot < 0 || slot >= a.pool_rows) {
                    slot = -1;
                    bad = MLA_DEVERR_BAD_SLOT;
                }
            }
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
    cudaError_t e = launch_dependent(sums_kernel, dim3(1), kSumThreads, s, true, a);
    const int64_t entry_ctas = num_requests == 0 ? 0 : (total + kFillThreads - 1) / kFillThreads;
    const int64_t token_ctas = (num_tokens + kFillThreads - 1) / kFillThreads;
    if (e == cudaSuccess && entry_ctas + token_ctas > 0)
        e = launch_dependent(fill_kernel, dim3((unsigned)(entry_ctas + token_ctas)), kFillThreads, s,
                             true, a, (uint32_t)entry_ctas);
    return status_of(e);
}

}  // extern "C"
