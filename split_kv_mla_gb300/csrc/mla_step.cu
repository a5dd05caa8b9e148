// mla_step.cu -- what lies between two steps of a decode loop: the beams' next
// tokens (selection), their states in their new order (reordering), and the next
// step's page tables, lengths, slots and positions (extension).  See
// include/mla_decode.h for the contracts.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstddef>

#include "mla_internal.h"
#include "mla_launch.h"
#include "mla_softmax.cuh"
#include "mla_spans.h"

namespace mla {
namespace {

// The kernels here start while the preceding one runs, which may write what they read, as one
// call's outputs are the next one's inputs: nothing is read before the wait for it, and nothing
// by __ldg, which is for what stays as it is for as long as the kernel runs.  (Extension reads
// by __ldcg: behind its barriers and stores plain loads wait, 4.6 us for 8 x 8192 and not 4.3.)

// ---- beam selection -------------------------------------------------------------------------
//
// The logits are read once.  For a row's score order only x matters, and the K best
// of a request lie in the K best groups of columns, when groups are ordered by their
// largest score and then by their index: each of those groups has a candidate at
// least as good as the K-th of them, and a candidate outside them is behind all of
// these (a group is a range of columns, so of equal scores the lower index is also in
// the lower group).  So
//   scan   streams the rows and leaves, for each 256 columns, their maximum, and for
//          each segment of a row (1 to 4 KB) its maximum m and sum of e^(x - m);
//   pick   (a CTA per request) joins a row's segments, takes the K best groups by
//          their maxima, reads those 256 logits of each again and takes the K best.
// What scan does per logit does not depend on the data, and pick reads 1/64 of the
// bytes, K groups, and of rows with a token of more than two thirds of their mass one
// segment.
//
// A segment's sum is relative to its own maximum, so its largest term is 1, and is
// held in fp32; which column goes to which lane does not depend on a row's address,
// so equal rows give equal sums and their equal candidates are taken by their index.
// Where one token has most of a row's mass, the logarithm is that of 1 + t with a small t,
// of which a sum that has the 1 has lost all below 2^-24 (scores of -2e-8 came out as 0).
// There pick sums the maximum's segment again without it, 0.6 to 1.8 us of a call whose
// rows are such.  (In scan, where every segment has a maximum, leaving the 1 out took every
// call longer: 11.7 -> 13.5 us for 32 x 4 of 100003 fp16, by its registers.)

constexpr int kGroup = 256;             // columns
constexpr int kShortPieces = 2, kMiddlePieces = 4, kLongPieces = 8;   // 16-byte loads of a lane
                                                                    // per segment
constexpr int kScanThreads = 256;
constexpr int kPickThreads = 512;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kPickList = 1024;
constexpr int kParts = 4;               // of a row, that a lane of pick asks for at once
constexpr float kPeakedSum = 1.5f;      // of a row, its maximum's term being 1
constexpr int kMaxVocab = 1 << 20;
constexpr int kPlaceBits = 20;          // of a column
static_assert(kMaxVocab <= 1 << kPlaceBits && MLA_MAX_BEAMS <= 1 << (32 - kPlaceBits), "");

struct SelectArgs {
    const void* logits;
    int64_t row_stride;
    const float* scores;
    const uint8_t* finished;
    int32_t batch, beams, vocab, select, end_token;
    int32_t groups;        // of a row
    int32_t segments;      // of a row
    int32_t segment_groups;
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
__device__ __forceinline__ void each_pair(const uint4& v, F&& f)
{
    if constexpr (sizeof(T) == 4) {
        f(make_float2(__uint_as_float(v.x), __uint_as_float(v.y)));
        f(make_float2(__uint_as_float(v.z), __uint_as_float(v.w)));
    } else {
        f(LogitType<T>::unpack(v.x));
        f(LogitType<T>::unpack(v.y));
        f(LogitType<T>::unpack(v.z));
        f(LogitType<T>::unpack(v.w));
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
            w[i] = col + i < vocab ? reinterpret_cast<const uint32_t*>(row)[col + i]
                                   : 0xFF800000u;
        } else {
            const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
            const uint32_t none = LogitType<T>::kNone;
            const uint32_t lo = col + 2 * i < vocab ? p[col + 2 * i] : none;
            const uint32_t hi = col + 2 * i + 1 < vocab ? p[col + 2 * i + 1] : none;
            w[i] = lo | hi << 16;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Segment `seg` of a row, -inf behind the row's end: PIECES of a lane.  Of an aligned row a
// lane's piece is 16 bytes, neighbours in neighbouring lanes.  Otherwise, in every row of
// the call, its words are 128 bytes apart, and those of a row of 16-bit logits that
// starts on an odd one are shifted out of two.  (Pieces shifted out of two aligned ones
// took 31 us a call for 57 MB, this way it is 21.)
template <typename T, int PIECES>
struct Segment {
    uint4 v[PIECES];
};

template <typename T, bool ALIGNED, int PIECES>
__device__ __forceinline__ void load_segment(const SelectArgs& a, int64_t row, int seg, int lane,
                                             Segment<T, PIECES>& s)
{
    constexpr int E = kElements<T>;
    const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
    const int c0 = seg * kSegment<T, PIECES>;
    if constexpr (ALIGNED) {
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            const int col = c0 + (p * 32 + lane) * E;
            s.v[p] = col + E <= a.vocab ? __ldcs(reinterpret_cast<const uint4*>(x + col))
                                        : load_edge(x, col, a.vocab);
        }
    } else {
        constexpr int N = 4 * PIECES;
        uint32_t w[N];
        if constexpr (sizeof(T) == 4) {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(x) + c0 + lane;
            const int left = a.vocab - c0 - lane;
#pragma unroll
            for (int k = 0; k < N; ++k) w[k] = 32 * k < left ? __ldcs(p + 32 * k) : 0xFF800000u;
        } else {
            const uintptr_t at = reinterpret_cast<uintptr_t>(x + c0);
            const int odd = (int)(at >> 1) & 1;
            const uint32_t* p = reinterpret_cast<const uint32_t*>(at - 2 * odd) + lane;
            if (c0 - odd < 0 || c0 + kSegment<T, PIECES> + odd > a.vocab) {   // the row's ends
                const uint16_t* h = reinterpret_cast<const uint16_t*>(x) + c0 + 2 * lane;
                const int left = a.vocab - c0 - 2 * lane;
                constexpr uint32_t none = LogitType<T>::kNone;
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const uint32_t lo = 64 * k < left ? h[64 * k] : none;
                    const uint32_t hi = 64 * k + 1 < left ? h[64 * k + 1] : none;
                    w[k] = lo | hi << 16;
                }
            } else if (odd) {
#pragma unroll
                for (int k = 0; k < N; ++k)
                    w[k] = __funnelshift_r(p[32 * k], p[32 * k + 1], 16);
            } else {
#pragma unroll
                for (int k = 0; k < N; ++k) w[k] = __ldcs(p + 32 * k);
            }
        }
#pragma unroll
        for (int q = 0; q < PIECES; ++q)
            s.v[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    }
}

// The column of a lane's i-th logit of a segment, from the lane's first on, and that.
template <typename T, bool ALIGNED>
__device__ __forceinline__ int column_step(int i)
{
    constexpr int E = kElements<T>, N = E / 4;   // logits of a word
    return ALIGNED ? i / E * 32 * E + i % E : i / N * 32 * N + i % N;
}

template <typename T, bool ALIGNED>
__device__ __forceinline__ int first_column(int lane)
{
    return lane * (ALIGNED ? kElements<T> : kElements<T> / 4);
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

// Maximum over the warp (a NaN is passed over).
__device__ __forceinline__ float warp_max(float x)
{
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
    return m;
}

__device__ __forceinline__ bool row_is_live(const SelectArgs& a, int64_t row)
{
    const float score = a.scores[row];
    const uint8_t finished = a.finished == nullptr ? 0 : a.finished[row];
    return score != -INFINITY && finished == 0;
}

// A segment's group maxima and its part.
template <typename T, int PIECES>
__device__ __forceinline__ void scan_segment(const SelectArgs& a, int64_t row, int seg, int lane,
                                             const Segment<T, PIECES>& s)
{
    constexpr int kPerGroup = kGroup / (32 * kElements<T>);   // pieces of a group
    constexpr int kGroups = PIECES / kPerGroup;               // groups of a segment
    float top = -INFINITY, mine = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        float m = piece_max<T>(s.v[g * kPerGroup]);
#pragma unroll
        for (int p = 1; p < kPerGroup; ++p) m = fmaxf(m, piece_max<T>(s.v[g * kPerGroup + p]));
        m = warp_max(m);
        top = fmaxf(top, m);
        if (lane == g) mine = m;
    }
    const int group = seg * kGroups + lane;
    if (lane < kGroups && group < a.groups) a.group_max[row * a.groups + group] = mine;

    const float ref = top == -INFINITY ? 0.f : top;
    constexpr float kLog2e = 1.4426950408889634f;
    const float2 back = make_float2(-ref, -ref), scale = make_float2(kLog2e, kLog2e);
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int p = 0; p < PIECES; ++p)
        each_pair<T>(s.v[p], [&](float2 t) {
            t = __fmul2_rn(__fadd2_rn(t, back), scale);
            sum = __fadd2_rn(sum, make_float2(ex2_approx(t.x), ex2_approx(t.y)));
        });
    float all = sum.x + sum.y;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) all += __shfl_xor_sync(0xffffffffu, all, off);
    if (lane == 0) a.parts[row * a.segments + seg] = make_float2(top, all);
}

// A warp per segment.  The rows of beams without candidates are not read.  (Warps that
// take several segments, the next one's logits in flight while they work on one, were
// slower with 16 to 40 of them on an SM: 45.5 us for 268 MB, 44.3 this way.)
template <typename T, bool ALIGNED, int PIECES>
__global__ void __launch_bounds__(kScanThreads)
scan_kernel(const SelectArgs a)
{
    wait_for_predecessor();
    allow_dependents();
    const int lane = threadIdx.x & 31;
    const uint32_t id = blockIdx.x * (kScanThreads / 32) + (threadIdx.x >> 5);   // below 2^31
    const int64_t row = id / (uint32_t)a.segments;
    const int seg = (int)(id % (uint32_t)a.segments);
    if (row >= a.rows || !row_is_live(a, row)) return;
    Segment<T, PIECES> s;
    load_segment<T, ALIGNED, PIECES>(a, row, seg, lane, s);
    scan_segment<T, PIECES>(a, row, seg, lane, s);
}

// (hi, lo) of a + b.
__device__ __forceinline__ float2 two_sum(float a, float b)
{
    const float s = __fadd_rn(a, b);
    const float t = __fsub_rn(s, a);
    return make_float2(s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t)));
}

// score - m - ln(sum) as a sum of floats, the largest first, so that a candidate's score is
// rounded once: the scores of different beams that fp32 tells apart come out in their order,
// as far as the sums are that exact (which is within 2^-15 of the logarithm).
// ln(sum) = e ln 2 + ln f with f in [0.75, 1.5); ln 2 in two parts, of which the first
// has 12 bits, so that e times it is exact.
__device__ __forceinline__ float3 row_base(float score, float m, float sum)
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
    const float2 c = two_sum(b.x, (a.y + b.y) - fmaf((float)e, (float)(kLn2 - kHigh), logf(f)));
    return make_float3(c.x, c.y, 0.f);
}

// The same of a row whose maximum, which it has once, has more than two thirds of its mass:
// of 1 + t with t the sum of e^(x - m) over the others.  The segment of the maximum is summed
// again without it, and the other segments' sums are joined by expf, as their maxima are far
// below m; head are those that the lane has.
template <typename T, bool ALIGNED>
__device__ __forceinline__ float3 peaked_base(const SelectArgs& a, int64_t row, int lane, float score,
                                              float m, const float2 (&head)[kParts])
{
    constexpr int kPerGroup = kGroup / (32 * kElements<T>);
    constexpr int kAtOnce = kPerGroup == 1 ? 2 : 4;   // groups (four of 16-bit logits spill)
    constexpr float kLog2e = 1.4426950408889634f;
    const float2* parts = a.parts + row * a.segments;
    float2 sum = make_float2(0.f, 0.f);
    uint32_t at = 0;
    auto join = [&](uint32_t i, float2 u) {
        if (u.x == m) at = i;
        else sum.x += u.y * expf(u.x - m);
    };
#pragma unroll
    for (int k = 0; k < kParts; ++k) join(lane + 32 * k, head[k]);
#pragma unroll 1
    for (int i = lane + 32 * kParts; i < a.segments; i += 32) join(i, __ldcg(parts + i));
    int g = (int)__reduce_max_sync(0xffffffffu, at) * a.segment_groups;
    const int end = min(g + a.segment_groups, a.groups);
#pragma unroll 1
    for (; g < end; g += kAtOnce) {
        Segment<T, kPerGroup> v[kAtOnce];
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q)
            if (g + q < end) load_segment<T, ALIGNED, kPerGroup>(a, row, g + q, lane, v[q]);
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) {
            if (g + q >= end) break;
#pragma unroll
            for (int p = 0; p < kPerGroup; ++p)
                each_pair<T>(v[q].v[p], [&](float2 x) {
                    sum.x += x.x == m ? 0.f : ex2_approx((x.x - m) * kLog2e);
                    sum.y += x.y == m ? 0.f : ex2_approx((x.y - m) * kLog2e);
                });
        }
    }
    float rest = sum.x + sum.y;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, off);
    // m last, and all three: the score and the logarithm may both be far below it
    const float2 u = two_sum(score, -log1pf(rest)), b = two_sum(u.x, -m);
    return make_float3(b.x, b.y, u.y);
}

// A score as a number in its order; 0 for what is no candidate (-inf, or the NaN that
// the base of a beam without candidates makes).
__device__ __forceinline__ uint32_t rank_of(float3 base, float x)
{
    const float2 s = two_sum(base.x, x), t = two_sum(s.x, base.y);
    const float rest = __fadd_rn(__fadd_rn(t.y, s.y), base.z);
    const float score = __fadd_rn(__fadd_rn(t.x, rest), 0.f);   // -0 as +0
    return score > -INFINITY ? (uint32_t)ordered(score) ^ 0x80000000u : 0u;
}

// A candidate of a beam as a number: by rank, then by the lower beam and the lower place
// (a column or a group) in it.
__device__ __forceinline__ uint64_t candidate(uint32_t rank, uint32_t beam, uint32_t place)
{
    return (uint64_t)rank << 32 | (0xFFFFFFFFu - (beam << kPlaceBits | place));
}

__device__ __forceinline__ uint32_t beam_of(uint64_t c) { return ~(uint32_t)c >> kPlaceBits; }

__device__ __forceinline__ uint32_t place_of(uint64_t c)
{
    return ~(uint32_t)c & ((1u << kPlaceBits) - 1u);
}

__device__ __forceinline__ float score_of(uint64_t c)
{
    return from_ordered((int)((uint32_t)(c >> 32) ^ 0x80000000u));
}

__device__ __forceinline__ uint64_t warp_max(uint64_t v)
{
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return (uint64_t)hi << 32 | lo;
}

// The next place of a list in shared memory.  (A few lanes of a warp ask at a time: their
// additions one after the other are shorter than the code that makes one of them.)
__device__ __forceinline__ int next_place(int* count)
{
    int at;
    asm volatile("atom.shared.add.u32 %0, [%1], 1;" : "=r"(at) : "r"(smem_u32(count)) : "memory");
    return at;
}

constexpr int kChunk = 8;          // candidates of a thread at a time
constexpr int kPickSlots = 256;
constexpr int kManyThreads = 48;

struct Picker {
    uint32_t best[2][32];               // of each part: of the groups, of the logits
    uint32_t least[2];
    int slots[2], count[2];
    alignas(16) float x[kPickSlots][kChunk];   // logits (group maxima) of the threads that have any
    int beam[kPickSlots], place[kPickSlots];
    uint64_t list[kPickList];
    uint64_t warps[kPickWarps];
    float3 base[MLA_MAX_BEAMS];         // -inf: no candidates; of an ended beam its score
    int ended[MLA_MAX_BEAMS];
};

static_assert(offsetof(Picker, x) % 16 == 0 && kChunk % 4 == 0, "chunks are stored as float4");

// The K-th largest of the parts' best, or 1 if there are not that many, after a barrier.  The
// threads of a lane are one of 32 parts of the CTA's candidates, and best is the largest
// rank of this thread's: K candidates or more have the rank returned, or a larger one.
__device__ __forceinline__ uint32_t rank_of_part(Picker& p, int round, int K, uint32_t best)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    atomicMax(&p.best[round][lane], best);
    __syncthreads();
    const uint32_t other = p.best[round][lane];
#pragma unroll
    for (int h = 0; h < 32 / kPickWarps; ++h) {
        const int part = warp * (32 / kPickWarps) + h;
        const uint32_t mine = __shfl_sync(0xffffffffu, other, part);
        const uint32_t above = __ballot_sync(0xffffffffu, other > mine || (other == mine && lane < part));
        if (lane == 0 && __popc(above) == K - 1 && mine != 0) p.least[round] = mine;
    }
    __syncthreads();
    return p.least[round];
}

// Lists the CTA's candidates with ranks of at least `least`, and returns how many, after a
// barrier.  each(f) calls f(beam, place, x) for the threads that have any, of kChunk
// logits x at a time, of which the i-th lies at place + step(i).  Those threads, a few,
// hand their logits over, and a thread for each ranks them (1,600 cycles; with the eight
// ranked in the threads themselves 2,150).  Lists that would overflow (many equal scores,
// or most of the best in few groups, and many) are not used: the K largest are then taken
// one after the other.
template <class Each, class Step>
__device__ __forceinline__ int list_candidates(Picker& p, int round, int K, uint32_t least,
                                               Each&& each, Step&& step)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint64_t last = ~0ull;
#pragma unroll 1
    for (int k = -1; k < K; ++k) {   // -1: the list; else the k-th by itself
        uint64_t next = 0;
        each([&](int beam, int place, const float (&x)[kChunk]) {
            if (k < 0) {
                const int at = next_place(&p.slots[round]);
                if (at >= kPickSlots) return;
                float4* to = reinterpret_cast<float4*>(p.x[at]);
                to[0] = make_float4(x[0], x[1], x[2], x[3]);
                to[1] = make_float4(x[4], x[5], x[6], x[7]);
                p.beam[at] = beam;
                p.place[at] = place;
            } else {
#pragma unroll 1
                for (int i = 0; i < kChunk; ++i) {   // (short code: it is rarely reached)
                    float xi = x[0];
#pragma unroll
                    for (int j = 1; j < kChunk; ++j) xi = i == j ? x[j] : xi;
                    const uint32_t r = rank_of(p.base[beam], xi);
                    const uint64_t c = candidate(r, beam, place + step(i));
                    if (r >= least && c < last && c > next) next = c;
                }
            }
        });
        __syncthreads();
        if (k < 0) {
            const int slots = p.slots[round];
            if (slots <= kPickSlots) {
                for (int t = tid; t < slots * kChunk; t += kPickThreads) {
                    const int slot = t / kChunk, i = t % kChunk, beam = p.beam[slot];
                    const uint32_t r = rank_of(p.base[beam], p.x[slot][i]);
                    if (r >= least) {
                        const int at = next_place(&p.count[round]);
                        if (at < kPickList) p.list[at] = candidate(r, beam, p.place[slot] + step(i));
                    }
                }
                __syncthreads();
                if (p.count[round] <= kPickList) return p.count[round];
            }
            continue;
        }
        next = warp_max(next);
        if (lane == 0) p.warps[warp] = next;
        __syncthreads();
        last = warp_max(p.warps[lane % kPickWarps]);
        if (tid == 0) p.list[k] = last;
    }
    __syncthreads();
    return K;
}

// done(k, x) for each of the K largest x of n listed, the k-th, by counting those above:
// a warp for each of a few, a thread for each of many.
template <class Done>
__device__ __forceinline__ void rank_list(const uint64_t* list, int n, int K, Done&& done)
{
    const int tid = threadIdx.x, lane = tid & 31;
    if (n <= 32) {
        const uint64_t other = lane < n ? list[lane] : 0;
        for (int i = tid >> 5; i < n; i += kPickWarps) {
            const uint64_t mine = list[i];
            const int above = __popc(__ballot_sync(0xffffffffu, other > mine));
            if (lane == 0 && above < K) done(above, mine);
        }
        return;
    }
#pragma unroll 1
    for (int i = tid; i < n; i += kPickThreads) {
        const uint64_t mine = list[i];
        int above = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) above += list[j] > mine ? 1 : 0;
        if (above < K) done(above, mine);
    }
}

// Bounded by latency: a request is one SM's, and a warp's instructions follow one another
// at four cycles and more, so what counts is the longest chain of them.  A beam belongs to
// one warp or several, each with the beam's base for itself, so that all a request needs
// is asked for at once.  Groups' maxima are candidates, so the rank that K of them reach
// bounds the logits' too, and only those that are left in the end are put in order.
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kPickThreads)
pick_kernel(const SelectArgs a)
{
    constexpr int E = kElements<T>;
    constexpr int kPerGroup = kGroup / (32 * E);
    constexpr int kTurns = MLA_MAX_BEAMS / kPickWarps;
    static_assert(kPerGroup * E == kChunk, "a lane's logits of a group are one chunk");
    __shared__ Picker p;
    __shared__ uint64_t groups[MLA_MAX_BEAMS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int K = a.select, W = a.beams, G = a.groups;
    const int share = W < kPickWarps ? kPickWarps / W : 1;   // warps of a beam
    const int beam0 = warp / share, part0 = warp % share;
    if (tid < 64) p.best[tid >> 5][tid & 31] = 0;
    if (tid < 2) {
        p.least[tid] = 1;
        p.slots[tid] = p.count[tid] = 0;
    }
    __syncthreads();
    wait_for_predecessor();
    allow_dependents();
    const int64_t row0 = (int64_t)blockIdx.x * W;

    // A thread's groups in beam w are first_group(w) + 32 share k.  (Turned by the beam, so
    // that beams of a few groups do not all lie in the same lanes.)
    auto first_group = [&](int w) { return part0 * 32 + ((lane + 5 * w) & 31); };
    float x[kChunk];
    auto load_maxima = [&](int w, int g) {
        const float* maxima = a.group_max + (row0 + w) * G;
#pragma unroll
        for (int k = 0; k < kChunk; ++k) {
            x[k] = g < G ? __ldcg(maxima + g) : -INFINITY;
            g += 32 * share;
        }
    };
    auto largest = [&] {
        return fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])),
                     fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
    };
    uint32_t best = 0;   // largest rank of the thread's beams
#pragma unroll 1
    for (int w = beam0; w < W; w += kPickWarps) {
        const int64_t row = row0 + w;
        const float2* parts = a.parts + row * a.segments;
        const float own = a.scores[row];
        const bool is_ended = a.finished != nullptr && a.finished[row] != 0;
        float2 t[kParts];
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
            const int i = lane + 32 * k;
            t[k] = i < a.segments ? __ldcg(parts + i) : make_float2(-INFINITY, 0.f);
        }
        const int g0 = first_group(w);
        load_maxima(w, g0);
        float m = -INFINITY, s = 0.f;
#pragma unroll
        for (int k = 0; k < kParts; ++k) m = fmaxf(m, t[k].x);
        // of rows with more parts (kParts at once, whatever is made of the loop: one
        // after the other they took 10.6 us for 1 x 1 x 1048576, this way 9.0)
        auto more_parts = [&](auto&& each) {
#pragma unroll 1
            for (int i = lane + 32 * kParts; i < a.segments; i += 32 * kParts) {
                float2 u[kParts];
#pragma unroll
                for (int k = 0; k < kParts; ++k)
                    u[k] = i + 32 * k < a.segments ? __ldcg(parts + i + 32 * k) : make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int k = 0; k < kParts; ++k) each(u[k]);
            }
        };
        more_parts([&](float2 u) { m = fmaxf(m, u.x); });
        m = warp_max(m);
        const float ref = m == -INFINITY ? 0.f : m;
        constexpr float kLog2e = 1.4426950408889634f;
#pragma unroll
        for (int k = 0; k < kParts; ++k) s += t[k].y * ex2_approx((t[k].x - ref) * kLog2e);
        more_parts([&](float2 u) { s += u.y * ex2_approx((u.x - ref) * kLog2e); });
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        // (what is not read of a beam without candidates may be anything)
        const bool none = own == -INFINITY;
        // a NaN or +inf among the logits makes the sum one
        const bool bad = !none && (!(own < INFINITY) || (!is_ended && !(s < INFINITY)));
        float3 b = make_float3(-INFINITY, 0.f, 0.f);
        if (!none && !bad && (is_ended || s != 0.f))
            b = is_ended ? make_float3(own, 0.f, 0.f)
                : __builtin_expect(s < kPeakedSum, 0)
                    ? peaked_base<T, ALIGNED>(a, row, lane, own, m, t)
                    : row_base(own, m, s);
        if (lane == 0 && part0 == 0) {
            p.base[w] = b;
            p.ended[w] = is_ended ? 1 : 0;
            if (bad) atomicOr(a.err, MLA_DEVERR_BAD_LOGITS);
        }
        if (is_ended) {   // its one candidate is in its first group
#pragma unroll
            for (int k = 0; k < kChunk; ++k) x[k] = -INFINITY;
            if (g0 == 0) x[0] = 0.f;
        }
        float most = largest();
        if (!is_ended) {
            const float* maxima = a.group_max + row * G;
#pragma unroll 4
            for (int g = g0 + 32 * share * kChunk; g < G; g += 32 * share)
                most = fmaxf(most, __ldcg(maxima + g));
        }
        best = max(best, rank_of(b, most));
    }
    // Round 0 finds the groups, round 1 their logits.  (One copy of the code for both: a
    // jump to code for the first time is 700 cycles.)
    Segment<T, kPerGroup> v[kTurns];   // a warp's groups, eight logits a lane
    int beam[kTurns] = {}, column[kTurns] = {}, n = 0;
    uint32_t top[kTurns] = {}, least = 1;
    auto unpack = [&](int q) {   // into x; an ended beam's one candidate is lane 0's
        if (p.ended[beam[q]] != 0) {
#pragma unroll
            for (int i = 0; i < kChunk; ++i) x[i] = -INFINITY;
            if (lane == 0) x[0] = 0.f;
        } else {
#pragma unroll
            for (int z = 0; z < kPerGroup; ++z)
                each_logit<T>(v[q].v[z], [&](int i, float t) { x[z * E + i] = t; });
        }
    };
    bool reload = W > kPickWarps;   // (of two beams only the last's maxima are there)
#pragma unroll 1
    for (int round = 0; round < 2; ++round) {
        bool bound = true;
        if (round == 1) {
#pragma unroll
            for (int q = 0; q < kTurns; ++q) {
                const int k = warp + q * kPickWarps;
                beam[q] = -1;
                if (k >= n) continue;
                const uint64_t c = groups[k];
                const int g = (int)place_of(c);
                beam[q] = (int)beam_of(c);
                column[q] = g * kGroup + first_column<T, ALIGNED>(lane);
                if (p.ended[beam[q]] == 0)
                    load_segment<T, ALIGNED, kPerGroup>(a, row0 + beam[q], g, lane, v[q]);
            }
            best = 0;
#pragma unroll
            for (int q = 0; q < kTurns; ++q) {
                top[q] = 0;
                if (beam[q] < 0) continue;
                unpack(q);
                top[q] = rank_of(p.base[beam[q]], largest());
                best = max(best, top[q]);
            }
            // Where few groups hold most of the best (beams far ahead of the others, of a
            // small vocabulary), the groups' bound leaves many logits, and theirs is needed.
            bound = __syncthreads_count(best >= least) > kManyThreads;
        }
        if (bound) least = max(least, rank_of_part(p, round, K, best));
        n = list_candidates(
            p, round, K, least,
            [&](auto&& take) {
                if (best < least) return;
                if (round == 1) {
#pragma unroll
                    for (int q = 0; q < kTurns; ++q) {
                        if (top[q] < least) continue;
                        unpack(q);
                        take(beam[q], p.ended[beam[q]] != 0 ? a.end_token : column[q], x);
                    }
                    return;
                }
#pragma unroll 1
                for (int w = beam0; w < W; w += kPickWarps) {
                    const int g0 = first_group(w);
                    const bool is_ended = p.ended[w] != 0;
                    if (is_ended) {
#pragma unroll
                        for (int k = 0; k < kChunk; ++k) x[k] = -INFINITY;
                        if (g0 == 0) x[0] = 0.f;
                    }
                    const float3 b = p.base[w];
#pragma unroll 1
                    for (int g = g0; g < G; g += 32 * share * kChunk) {
                        if (reload && !is_ended) load_maxima(w, g);
                        if (rank_of(b, largest()) >= least) take(w, g, x);
                        if (is_ended) break;
                        reload = reload || g + 32 * share * kChunk < G;
                    }
                }
            },
            [&](int i) { return round == 0 ? 32 * share * i : column_step<T, ALIGNED>(i); });
        if (round == 1) break;
        // (up to 32 groups, more than K, are looked at as they are)
        if (n > MLA_MAX_BEAMS) {
            rank_list(p.list, n, K, [&](int k, uint64_t c) { groups[k] = c; });
            n = K;
        } else if (tid < n) {
            groups[tid] = p.list[tid];
        }
        __syncthreads();
    }
    const int64_t out = (int64_t)blockIdx.x * K;
    auto put = [&](int k, int token, int w, float score, bool end) {
        a.tokens[out + k] = token;
        a.parents[out + k] = (int32_t)(row0 + w);
        a.scores_out[out + k] = score;
        if (a.finished_out != nullptr) a.finished_out[out + k] = end ? 1 : 0;
    };
    rank_list(p.list, n, K, [&](int k, uint64_t c) {
        const int w = (int)beam_of(c), token = (int)place_of(c);
        put(k, token, w, score_of(c), token == a.end_token || p.ended[w] != 0);
    });
    if (tid >= n && tid < K) put(tid, -1, 0, -INFINITY, true);
}

// Segments are as long as leaves the GPU's SMs a wave of warps, 64 each: 4 KB, 2 or 1; and
// not so short that a row has more parts than pick asks for at once.
// (us per call with 4 / 2 / 1 KB: 64 x 8 beams of 131072 fp32 logits 50.0 / 52.0 / -,
// 32 x 4 of 100003 fp16 13.5 / 12.4 / 14.4, 8 x 8 of 50001 bf16 15.0 / - / 10.6.)
constexpr int64_t kScanWarps = 152 * 64;

template <typename T, bool ALIGNED, int PIECES>
cudaError_t launch_scan(SelectArgs& a, cudaStream_t s)
{
    a.segments = (a.vocab + kSegment<T, PIECES> - 1) / kSegment<T, PIECES>;
    a.segment_groups = kSegment<T, PIECES> / kGroup;
    const int64_t ctas = (a.rows * a.segments + kScanThreads / 32 - 1) / (kScanThreads / 32);
    return launch_dependent(scan_kernel<T, ALIGNED, PIECES>, dim3((unsigned)ctas), kScanThreads, s,
                            true, a);
}

template <typename T, bool ALIGNED>
cudaError_t launch_select(SelectArgs a, cudaStream_t s)
{
    auto parts = [&](int64_t columns) { return (a.vocab + columns - 1) / columns; };   // of a row
    const int64_t many = parts(kSegment<T, kLongPieces>), some = parts(kSegment<T, kMiddlePieces>),
                  few = parts(kSegment<T, kShortPieces>);
    const cudaError_t e =
        a.rows * many >= kScanWarps || some > 32 * kParts ? launch_scan<T, ALIGNED, kLongPieces>(a, s)
        : a.rows * some >= kScanWarps || few > 32 * kParts
            ? launch_scan<T, ALIGNED, kMiddlePieces>(a, s)
            : launch_scan<T, ALIGNED, kShortPieces>(a, s);
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

// Bytes of the segments' parts.  Segments shorter than the longest are taken while those of
// twice their length are less than a wave.
int64_t select_part_bytes(int64_t rows, int64_t vocab)
{
    const int64_t n = kSegment<float, kLongPieces>;
    const int64_t parts = rows * ((vocab + n - 1) / n);
    return align256((parts > 2 * kScanWarps ? parts : 2 * kScanWarps) * (int64_t)sizeof(float2));
}

// ---- beam state reordering ------------------------------------------------------------------
//
// A copy: bounded by HBM for large states, by latency for small ones.  A CTA takes a
// part of one row, in 16-byte pieces of out.  Where rows of state and out do not lie at the
// same place of 16 bytes, a piece is shifted out of two aligned ones of state (512 rows of
// 65535 bf16: 21.5 us, 43.7 by the 2 bytes that they are aligned to, 19 for 65536), and
// the few bytes at a row's ends are copied one by one.

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

// Bytes [shift, shift + 16) of two pieces, 0 < shift < 16.
__device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, uint32_t shift)
{
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (shift & 8u) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (shift & 4u) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    const uint32_t s = (shift & 3u) * 8u;
    return make_uint4(__funnelshift_r(w[0], w[1], s), __funnelshift_r(w[1], w[2], s),
                      __funnelshift_r(w[2], w[3], s), __funnelshift_r(w[3], w[4], s));
}

template <bool ALIGNED>
__global__ void __launch_bounds__(kReorderThreads)
reorder_kernel(const ReorderArgs a)
{
    wait_for_predecessor();
    allow_dependents();
    const uint32_t f = blockIdx.x / a.parts, part = blockIdx.x - f * a.parts;
    const bool first = part == 0 && threadIdx.x == 0;
    const int32_t p = a.parents[f];
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
        const int64_t want = a.lens[p];
        const int64_t len = want < 0 ? 0 : want > room ? room : want;
        bytes = len * a.elem_bytes;
        if (first) {
            const bool add = a.tokens != nullptr && len < room;
            if (add) *reinterpret_cast<int32_t*>(out + bytes) = a.tokens[f];
            if (a.out_lens != nullptr) a.out_lens[f] = (int32_t)(len + (add ? 1 : 0));
            if (len != want || (a.tokens != nullptr && !add)) atomicOr(a.err, MLA_DEVERR_BAD_LENGTH);
        }
    }
    const uint8_t* in = a.state + p * a.state_stride;
    // pieces [begin, end) of out from its byte `head` on, of which piece j is shifted out of
    // pieces j and j + 1 of state from its byte head - shift on, both inside the row
    int64_t head = 0, begin = 0, end = bytes / 16;
    uint32_t shift = 0;
    if constexpr (!ALIGNED) {
        head = (int64_t)((16u - (uint32_t)reinterpret_cast<uintptr_t>(out)) & 15u);
        if (head > bytes) head = bytes;
        end = (bytes - head) / 16;
        shift = (uint32_t)reinterpret_cast<uintptr_t>(in + head) & 15u;
        if (shift != 0) {
            begin = head < (int64_t)shift ? 1 : 0;
            const int64_t whole = (a.row_bytes - head + shift) / 16 - 1;
            end = end < whole ? end : whole;
        }
        if (end <= begin) begin = end = 0;
    }
    const uint4* from = reinterpret_cast<const uint4*>(in + head - shift);
    uint4* to = reinterpret_cast<uint4*>(out + head);
    const int64_t step = (int64_t)a.parts * kReorderThreads * kReorderTurns;
    for (int64_t i = begin + (int64_t)part * (kReorderThreads * kReorderTurns) + threadIdx.x; i < end;
         i += step) {
        uint4 v[kReorderTurns];
        if (ALIGNED || shift == 0) {
#pragma unroll
            for (int k = 0; k < kReorderTurns; ++k)
                if (i + k * kReorderThreads < end) v[k] = from[i + k * kReorderThreads];
        } else {
#pragma unroll
            for (int k = 0; k < kReorderTurns; ++k)
                if (i + k * kReorderThreads < end) {
                    const uint4* q = from + i + k * kReorderThreads;
                    v[k] = shifted(q[0], q[1], shift);
                }
        }
#pragma unroll
        for (int k = 0; k < kReorderTurns; ++k)
            if (i + k * kReorderThreads < end) to[i + k * kReorderThreads] = v[k];
    }
    // what lies before and behind those, at most 31 and 63 bytes
    if (part == 0) {
        const int64_t before = begin == end ? 0 : head + begin * 16;
        const int64_t behind = begin == end ? 0 : head + end * 16;
        if ((int64_t)threadIdx.x < before) out[threadIdx.x] = in[threadIdx.x];
        for (int64_t at = behind + threadIdx.x; at < bytes; at += kReorderThreads) out[at] = in[at];
    }
}

// ---- cache extension --------------------------------------------------------------------------
//
// Bytes: 8 per entry that is kept, 12 (16 with a list of free slots) per token.
// Every CTA sums the requests' lengths and counts by itself, in shared memory, and
// fills its part of the new table from there: one launch.  A kernel that left the sums
// for a second one took 7.5 us where this takes 4.3 (8 requests of 8192), and looking a
// request up in global memory, per entry, 103 us where this takes 8.8 (512 of 1024 to
// 8192).  More requests than shared memory is given for go that way:
//   sums   (one CTA) the requests' lengths and counts, their sums, the cursor;
//   fill   a warp per 256 entries of the new table, a thread per token.

constexpr int kExtendThreads = 512;
constexpr int kExtendRequests = 2048;   // 32 KB of sums
constexpr int kShortSpan = 8, kLongSpan = 16;   // entries in flight per thread
constexpr int kExtendCtas = 2 * 152;
constexpr int kLeadTokens = 2048;       // that one CTA takes
constexpr int kSumThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kFillSpan = 256;          // entries of a warp

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
    const int p = a.parents == nullptr ? f : __ldcg(a.parents + f);
    if (p < 0 || p >= a.num_parents) {
        bad |= MLA_DEVERR_BAD_TABLE;
        return Kept{0, 0};
    }
    const int64_t from = __ldcg(a.kv_indptr + p), to = __ldcg(a.kv_indptr + p + 1);
    const int64_t want = __ldcg(a.seq_lens + p);
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
    const int32_t slot = a.free_slots == nullptr ? number : __ldcg(a.free_slots + number);
    if (slot >= 0 && slot < a.pool_rows) return slot;
    bad |= MLA_DEVERR_BAD_SLOT;
    return -1;
}

// The last f in [lo, hi) with start[f] <= i (start[lo] <= i).
__device__ __forceinline__ int last_at_most(const int32_t* start, int lo, int hi, int32_t i)
{
    while (hi - lo > 1) {
        const int mid = middle(lo, hi);
        if (start[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

// CTA 0 writes what is per request, and with `spread` false all of what is per token,
// so that it alone reads the cursor that it then moves (which may be one and the
// same); the others copy.
// (Four CTAs on an SM for short spans: with three, at 40 registers, the next call's CTAs
// start later, 7.4 us a call instead of 6.6 for 1.1 million entries; the same with three
// of two for long spans, 9.8 instead of 7.8 for 2.4 million.)
template <int SPAN>
__global__ void __launch_bounds__(kExtendThreads, SPAN == kShortSpan ? 4 : 2)
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
        int n = a.new_tokens == nullptr ? 1 : __ldcg(a.new_tokens + f);
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
    for (int f = f0; f < f1; ++f) mine = add_up(mine, token_place(length[f], token[f + 1] - token[f]));
    at = block_scan<kExtendThreads / 32>(mine, part, all);
    for (int f = f0; f < f1; ++f) {
        start[f] = (int32_t)min(at, room);
        from[f] -= start[f];
        at = add_up(at, token_place(length[f], token[f + 1] - token[f]));
    }
    if (all > room) bad |= MLA_DEVERR_BAD_TABLE;
    const int32_t total = (int32_t)min(all, room);
    if (tid == 0) start[F] = total;
    __syncthreads();

    if (lead || spread) {
        const int step = spread ? (int)gridDim.x * kExtendThreads : kExtendThreads;
        const int32_t cursor = a.num_tokens > 0 ? __ldcg(a.cursor) : 0;
        const int32_t prefix = a.prefix_len == nullptr ? 0 : __ldcg(a.prefix_len);
        for (int64_t t = (int64_t)(spread ? blockIdx.x : 0) * kExtendThreads + tid; t < a.num_tokens;
             t += step) {
            int32_t slot = -1, position = 0;
            if (t < tokens) {
                const int f = last_at_most(token, 0, F, (int32_t)t);
                const uint32_t j = token_place(length[f], (uint32_t)t - (uint32_t)token[f]);
                position = (int32_t)(j + (uint32_t)prefix);
                if (has_place(start[f], start[f + 1], j)) {
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
    constexpr int kSpan = 32 * SPAN;   // entries at a time
    const uint32_t warps = (gridDim.x - 1) * (kExtendThreads / 32);
    const uint32_t warp = (blockIdx.x - 1) * (kExtendThreads / 32) + (tid >> 5);
    const Run run = warp_run((uint32_t)total, warp, warps, kSpan);
    if (run.begin >= run.end) return;
    int lo = last_at_most(start, 0, F, (int32_t)run.begin);
    for (uint32_t i0 = run.begin; i0 < run.end; i0 += kSpan) {
        const uint32_t past = span_end(i0, run.end, kSpan);
        if (start[lo + 1] <= (int32_t)i0) lo = last_at_most(start, lo + 1, F, (int32_t)i0);
        // the lane's entries are 32 apart from its first on: those below `left`
        int32_t* const dst = a.new_indices + (i0 + lane);
        int32_t v[SPAN];
        if (start[lo + 1] >= (int32_t)past) {   // one request's
            const uint32_t until = min(past, kept_end(start[lo], start[lo + 1], length[lo]));
            const int32_t left = (int32_t)(until - i0) - lane;
            const int32_t* src = a.kv_indices + from[lo] + (i0 + lane);
#pragma unroll
            for (int k = 0; k < SPAN; ++k)
                if (32 * k < left) v[k] = __ldcg(src + 32 * k);
#pragma unroll
            for (int k = 0; k < SPAN; ++k)
                if (32 * k < left) dst[32 * k] = v[k];
            continue;
        }
        const int hi = last_at_most(start, lo, F, (int32_t)past - 1) + 1;
        const int32_t left = (int32_t)(past - i0) - lane;
        bool kept[SPAN];
#pragma unroll
        for (int k = 0; k < SPAN; ++k) {
            kept[k] = 32 * k < left;
            if (kept[k]) {
                const int32_t i = (int32_t)i0 + lane + 32 * k;
                const int f = last_at_most(start, lo, hi, i);
                kept[k] = i - start[f] < length[f];
                if (kept[k]) v[k] = __ldcg(a.kv_indices + (from[f] + i));
            }
        }
#pragma unroll
        for (int k = 0; k < SPAN; ++k)
            if (kept[k]) dst[32 * k] = v[k];
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
    const uint32_t F = (uint32_t)a.num_requests;
    for (uint32_t f0 = 0; f0 < F; f0 += kSumThreads) {
        const uint32_t f = f0 + tid;
        uint32_t n = 0, length = 0;
        if (f < F) {
            const int32_t want = a.new_tokens == nullptr ? 1 : __ldcg(a.new_tokens + f);
            n = max(want, 0);
            if (want < 0) bad |= MLA_DEVERR_BAD_LENGTH;
            length = kept_of(a, (int)f, bad).length;
        }
        uint32_t all;
        const uint32_t t = add_up(tokens, block_scan<kSumThreads / 32>(n, part, all));
        const uint32_t first_token = min(t, token_room);
        length += min(add_up(t, n), token_room) - first_token;
        tokens = add_up(tokens, all);
        const uint32_t e = add_up(entries, block_scan<kSumThreads / 32>(length, part, all));
        const uint32_t first = min(e, room);
        entries = add_up(entries, all);
        if (f < F) {
            a.token_indptr[f] = (int32_t)first_token;
            a.new_indptr[f] = (int32_t)first;
            a.new_lens[f] = (int32_t)(min(add_up(e, length), room) - first);
        }
    }
    if (tokens > token_room || entries > room) bad |= MLA_DEVERR_BAD_TABLE;
    if (tid == 0) {
        const uint32_t n = min(tokens, token_room);
        a.token_indptr[F] = (int32_t)n;
        a.new_indptr[F] = (int32_t)min(entries, room);
        // modulo 2^32, so that fill has the cursor from the new one
        a.new_cursor[0] = (int32_t)((uint32_t)a.cursor[0] + n);
    }
    if (bad != 0) atomicOr(a.err, bad);
}

// The last f in [lo, hi) with indptr[f] <= i (indptr[lo] <= i).
__device__ __forceinline__ int find_request(const int32_t* indptr, int lo, int hi, int64_t i)
{
    while (hi - lo > 1) {
        const int mid = middle(lo, hi);
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
        // a warp's span, and the requests in it
        const int lane = threadIdx.x & 31;
        const int64_t total = __ldcg(a.new_indptr + F);
        const int64_t i0 = ((int64_t)blockIdx.x * (kFillThreads / 32) + (threadIdx.x >> 5)) * kFillSpan;
        if (i0 >= total) return;
        const int64_t past = min(i0 + kFillSpan, total);
        const int lo = find_request(a.new_indptr, 0, F, i0);
        const int hi = __ldcg(a.new_indptr + lo + 1) >= past
                           ? lo + 1 : find_request(a.new_indptr, lo, F, past - 1) + 1;
        const Kept own = kept_of(a, lo, bad);
        const int64_t start = __ldcg(a.new_indptr + lo);
        int32_t v[kFillSpan / 32];
        bool kept[kFillSpan / 32];
#pragma unroll
        for (int k = 0; k < kFillSpan / 32; ++k) {
            const int64_t i = i0 + 32 * k + lane;
            kept[k] = i < past;
            if (!kept[k]) continue;
            Kept from = own;
            int64_t j = i - start;
            if (hi - lo > 1) {
                const int f = find_request(a.new_indptr, lo, hi, i);
                from = kept_of(a, f, bad);
                j = i - __ldcg(a.new_indptr + f);
            }
            kept[k] = j < from.length;
            if (kept[k]) v[k] = __ldcg(a.kv_indices + from.from + j);
        }
#pragma unroll
        for (int k = 0; k < kFillSpan / 32; ++k)
            if (kept[k]) a.new_indices[i0 + 32 * k + lane] = v[k];
        return;
    }
    const int64_t t = (int64_t)(blockIdx.x - entry_ctas) * kFillThreads + threadIdx.x;
    if (t >= a.num_tokens) return;
    const int32_t tokens = __ldcg(a.token_indptr + F);
    int32_t slot = -1, position = 0;
    if (t < tokens) {
        const int f = find_request(a.token_indptr, 0, F, t);
        const Kept k = kept_of(a, f, bad);
        bad = 0;   // the sums have told
        const int64_t j = k.length + (t - __ldcg(a.token_indptr + f));
        position = (int32_t)(j + (a.prefix_len == nullptr ? 0 : __ldcg(a.prefix_len)));
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

struct Bytes {
    const void* p;
    int64_t n;
};

bool overlap(const Bytes& a, const Bytes& b) { return overlap(a.p, a.n, b.p, b.n); }

// Whether one of n rows of `bytes` at p, `stride` apart, has a byte in common with b.
bool rows_reach(const void* p, int64_t n, int64_t stride, int64_t bytes, const Bytes& b)
{
    if (p == nullptr || b.p == nullptr || n < 1 || bytes < 1 || b.n < 1) return false;
    const int64_t at = reinterpret_cast<const char*>(b.p) - static_cast<const char*>(p);
    // the first row that does not end before b
    const int64_t r = at < bytes || stride < 1 ? 0 : (at - bytes) / stride + 1;
    return r < n && r * stride < at + b.n && at < r * stride + bytes;
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
    const int64_t element = dtype == MLA_DTYPE_F32 ? 4 : 2;
    const Bytes in[2] = {{scores, rows * 4}, {finished, rows}};
    const Bytes out[4] = {{scores_out, picks * 4}, {finished_out, picks}, {tokens, picks * 4},
                          {parents, picks * 4}};
    auto on_logits = [&](const Bytes& b) {
        return rows_reach(logits, rows, row_stride * element, vocab * element, b);
    };
    for (int i = 0; i < 4; ++i) {
        // scores_out as scores and finished_out as finished, entry by entry
        const bool in_place = i < 2 && out[i].p == in[i].p && num_select == beams;
        for (int k = 0; k < 2; ++k)
            if (overlap(out[i], in[k]) && !(i == k && in_place)) return MLA_ERR_INVALID_ARG;
        for (int k = 0; k < i; ++k)
            if (overlap(out[i], out[k])) return MLA_ERR_INVALID_ARG;
        // (flags in place are an input as well, and where inputs lie is the caller's)
        if (!(i == 1 && in_place) && on_logits(out[i])) return MLA_ERR_INVALID_ARG;
    }
    if ((reinterpret_cast<uintptr_t>(logits) & (dtype == MLA_DTYPE_F32 ? 3u : 1u)) != 0)
        return MLA_ERR_MISALIGNED;
    int rc = check_header(workspace, workspace_bytes);
    if (rc != MLA_OK) return rc;
    const Bytes scratch = {workspace, mla_beam_select_workspace_bytes(batch, beams, vocab)};
    if (workspace_bytes < scratch.n) return MLA_ERR_WORKSPACE_TOO_SMALL;
    for (const Bytes& b : {in[0], in[1], out[0], out[1], out[2], out[3]})
        if (overlap(scratch, b)) return MLA_ERR_INVALID_ARG;
    if (on_logits(scratch)) return MLA_ERR_INVALID_ARG;
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
    if ((tokens != nullptr || out_lens != nullptr) && lens == nullptr) return MLA_ERR_INVALID_ARG;
    if (tokens != nullptr && elem_bytes != 4) return MLA_ERR_UNSUPPORTED_SHAPE;
    if (num_rows == 0) return MLA_OK;
    if (!parents || (row_bytes > 0 && (!out || (num_parents > 0 && !state))) ||
        (num_rows > 1 && out_stride < row_bytes) ||
        rows_overlap(state, num_parents, state_stride, out, num_rows, out_stride, row_bytes))
        return MLA_ERR_INVALID_ARG;
    const int64_t F = num_rows, span = (F - 1) * out_stride + row_bytes;
    const Bytes in[] = {{parents, F * 4}, {tokens, F * 4}, {lens, (int64_t)num_parents * 4}};
    const Bytes rows = {out, span}, counts = {out_lens, F * 4};
    auto on_state = [&](const Bytes& b) {
        return rows_reach(state, num_parents, state_stride, row_bytes, b);
    };
    for (const Bytes& i : in)
        if (overlap(counts, i) || overlap(rows, i)) return MLA_ERR_INVALID_ARG;
    if (overlap(counts, rows) || on_state(counts)) return MLA_ERR_INVALID_ARG;
    uintptr_t bits = reinterpret_cast<uintptr_t>(state) | reinterpret_cast<uintptr_t>(out);
    if (num_parents > 1) bits |= (uintptr_t)state_stride;
    if (num_rows > 1) bits |= (uintptr_t)out_stride;
    if (tokens != nullptr && (bits & 3u) != 0) return MLA_ERR_MISALIGNED;
    int rc = check_header(workspace, workspace_bytes);
    if (rc != MLA_OK) return rc;
    const Bytes header = {workspace, MLA_WORKSPACE_HEADER_BYTES};
    for (const Bytes& b : {rows, counts, in[0], in[1], in[2]})
        if (overlap(header, b)) return MLA_ERR_INVALID_ARG;
    if (on_state(header)) return MLA_ERR_INVALID_ARG;
    rc = device_ok();
    if (rc != MLA_OK) return rc;

    ReorderArgs a{static_cast<const uint8_t*>(state), state_stride, num_parents, row_bytes,
                  elem_bytes, parents, num_rows, lens, tokens, static_cast<uint8_t*>(out),
                  out_stride, out_lens, 1, static_cast<uint32_t*>(workspace)};
    const int64_t per = (int64_t)16 * kReorderThreads * kReorderTurns;
    const int64_t parts = (row_bytes + per - 1) / per;
    const int64_t most = INT32_MAX / num_rows;   // CTAs of the grid; a CTA loops over the rest
    a.parts = (uint32_t)(parts < 1 ? 1 : parts < most ? parts : most);
    const dim3 grid((unsigned)(a.parts * (uint32_t)num_rows));
    return status_of(launch_dependent((bits & 15u) == 0 ? reorder_kernel<true> : reorder_kernel<false>,
                                      grid, kReorderThreads, static_cast<cudaStream_t>(stream), true, a));
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
    const int64_t F = num_requests, P = num_parents;
    const Bytes in[] = {{kv_indices, num_indices * 4}, {kv_indptr, (P + 1) * 4}, {seq_lens, P * 4},
                        {parents, F * 4}, {new_tokens, F * 4}, {free_slots, num_free * 4},
                        {cursor, 4}, {prefix_len, 4}};
    const Bytes out[] = {{new_indices, total * 4}, {new_indptr, (F + 1) * 4}, {new_lens, F * 4},
                         {slots, num_tokens * 4}, {positions, num_tokens * 4},
                         {token_indptr, (F + 1) * 4}, {new_cursor, 4}};
    for (const Bytes& o : out) {
        for (const Bytes& i : in)
            if (overlap(o, i) && !(o.p == new_cursor && i.p == cursor)) return MLA_ERR_INVALID_ARG;
        for (const Bytes* other = out; other != &o; ++other)
            if (overlap(o, *other)) return MLA_ERR_INVALID_ARG;
    }
    int rc = check_header(workspace, workspace_bytes);
    if (rc != MLA_OK) return rc;
    const Bytes header = {workspace, MLA_WORKSPACE_HEADER_BYTES};
    for (const Bytes& o : out)
        if (overlap(header, o)) return MLA_ERR_INVALID_ARG;
    for (const Bytes& i : in)
        if (overlap(header, i)) return MLA_ERR_INVALID_ARG;
    rc = device_ok();
    if (rc != MLA_OK) return rc;

    const ExtendArgs a{kv_indices, num_indices, kv_indptr, seq_lens, num_parents, parents,
                       new_tokens, num_requests, free_slots, num_free, cursor, pool_rows,
                       prefix_len, new_indices, total, new_indptr, new_lens, slots, positions,
                       num_tokens, token_indptr, new_cursor, static_cast<uint32_t*>(workspace)};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (num_requests <= kExtendRequests) {
        // (twice the entries in flight once that saves a turn of every warp: 9.6 -> 8.5 us
        // for 2.4 million entries, but 5.0 -> 6.1 for 65,536)
        const bool large = total > (int64_t)kExtendCtas * kExtendThreads * kShortSpan;
        const bool spread = num_tokens > kLeadTokens;
        // A CTA per SM while that leaves a thread two entries or more, then one for each turn
        // of its threads: every CTA sums all the requests (65,536 entries by 17, 33 and 65
        // CTAs: 5.0, 4.4 and 4.2 us; 1.1 million by 152, 260 and 305: 6.8, 6.5 and 7.5).
        const int64_t units = spread && num_tokens > total ? num_tokens : total;
        auto ctas = [&](int64_t per_thread) {
            return (units + per_thread * kExtendThreads - 1) / (per_thread * kExtendThreads);
        };
        const int64_t spans = ctas(large ? kLongSpan : kShortSpan), pairs = ctas(2);
        const int64_t few = pairs < kExtendCtas / 2 ? pairs : kExtendCtas / 2;
        const int64_t most = spans > few ? spans : few;
        const bool in_place = new_cursor == cursor;
        const dim3 grid((unsigned)(1 + (most < 1 ? 1 : most < kExtendCtas ? most : kExtendCtas)));
        const int bytes = (4 * num_requests + 2) * 4;
        cudaError_t e = launch_dependent_shared(
            large ? extend_kernel<kLongSpan> : extend_kernel<kShortSpan>, grid, kExtendThreads, bytes, s,
            true, a, spread, !(spread && in_place));
        if (e == cudaSuccess && spread && in_place)
            e = launch_dependent(cursor_kernel, dim3(1), 1, s, true, a);
        return status_of(e);
    }
    cudaError_t e = launch_dependent(sums_kernel, dim3(1), kSumThreads, s, true, a);
    constexpr int64_t per = kFillThreads / 32 * kFillSpan;
    const int64_t entry_ctas = num_requests == 0 ? 0 : (total + per - 1) / per;
    const int64_t token_ctas = (num_tokens + kFillThreads - 1) / kFillThreads;
    if (e == cudaSuccess && entry_ctas + token_ctas > 0)
        e = launch_dependent(fill_kernel, dim3((unsigned)(entry_ctas + token_ctas)), kFillThreads, s,
                             true, a, (uint32_t)entry_ctas);
    return status_of(e);
}

}  // extern "C"
