// mla_cache.cu -- what writes and manages the paged fp8 cache: append (norm,
// rotation, e4m3, page write, with the queries in the same launch), fork and
// compaction.  See include/mla_decode.h for the contracts.
//
// All three move bytes once and compute little, so HBM bounds them; the point
// of every kernel here is to keep many 16-byte loads of whole 128-byte lines in
// flight and to spend few launches.
#include <cuda_bf16.h>

#include <cmath>

#include "mla_internal.h"
#include "mla_sm100.cuh"

namespace mla {
namespace {

using sm100::f32x2_to_e4m3x2;

// Launches kernel as a programmatic dependent of the preceding kernel on the
// stream: it may be scheduled while that one drains and waits for its
// completion (griddepcontrol.wait) before it reads anything.
// With `overlap` false it starts only when all earlier work on the stream is
// done (after a memset, which is no kernel to depend on).
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, int threads,
                             cudaStream_t stream, bool overlap, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = overlap ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

__device__ __forceinline__ void wait_for_predecessor()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void allow_dependents()
{
    asm volatile("griddepcontrol.launch_dependents;");
}

// ---- append ---------------------------------------------------------------------------------
//
// A row of 64 K columns belongs to eight lanes; lane l holds columns 64 k + 8 l
// .. + 7 for k < K, so each of its K loads is one of eight neighbouring 16-byte
// pieces (a whole 128-byte line per row), all K are in flight together, and the
// last one holds the eight RoPE columns 8 l .. 8 l + 7 whatever K is.  The mean
// of squares is a three-step shuffle; interleaved pairs sit in one lane, the
// partners of half-split pairs four lanes apart.

constexpr int kAppendThreads = 256;
constexpr int kRowLanes = 8;
constexpr int kAppendRows = kAppendThreads / kRowLanes;   // rows at a time per CTA

struct AppendArgs {
    const uint16_t* kv;
    int64_t kv_stride;
    const uint16_t* kv_weight;
    int32_t kv_norm_cols;
    const int32_t* slots;
    uint8_t* pool;
    int64_t pool_rows;
    float inv_scale;
    const uint16_t* q;
    int64_t q_token_stride, q_head_stride;
    const uint16_t* q_weight;
    int32_t q_norm;
    uint16_t* q_nope;
    uint16_t* q_pe;
    const int32_t* positions;
    const float* cos_sin;
    int64_t max_positions;
    int32_t half_split;
    float eps;
    int32_t tokens, heads;
    uint32_t kv_ctas;        // CTAs 0 .. kv_ctas-1 append rows, the others take queries
    uint32_t* err;
};

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

// Streaming accesses: every byte is used once.
__device__ __forceinline__ uint4 load_once(const uint16_t* p)
{
    return __ldcs(reinterpret_cast<const uint4*>(p));
}

// The angles of one lane's RoPE columns: cosine and sine per column, the sine
// with the sign of its column's term.
struct Turn {
    float c[8], s[8];
};

__device__ __forceinline__ Turn load_turn(const float* row, int l, bool half)
{
    Turn t;
    if (half) {
        const int a = (8 * l) & 31;   // columns i and i + 32 share angle i
        const float sign = l < 4 ? -1.f : 1.f;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const float4 c = __ldg(reinterpret_cast<const float4*>(row + a) + q);
            const float4 s = __ldg(reinterpret_cast<const float4*>(row + 32 + a) + q);
            t.c[4 * q] = c.x; t.c[4 * q + 1] = c.y; t.c[4 * q + 2] = c.z; t.c[4 * q + 3] = c.w;
            t.s[4 * q] = sign * s.x; t.s[4 * q + 1] = sign * s.y;
            t.s[4 * q + 2] = sign * s.z; t.s[4 * q + 3] = sign * s.w;
        }
    } else {
        const float4 c = __ldg(reinterpret_cast<const float4*>(row) + l);
        const float4 s = __ldg(reinterpret_cast<const float4*>(row + 32) + l);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t.c[2 * i] = t.c[2 * i + 1] = cc[i];
            t.s[2 * i] = -ss[i];
            t.s[2 * i + 1] = ss[i];
        }
    }
    return t;
}

// x_j c_j + (partner of x_j) s_j.  The whole warp calls it.
__device__ __forceinline__ void rotate(float (&x)[8], const Turn& t, bool half)
{
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float far = __shfl_xor_sync(0xffffffffu, x[j], 4);
        y[j] = half ? far : x[j ^ 1];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = x[j] * t.c[j] + y[j] * t.s[j];
}

// Sum over the eight lanes of a row (every lane ends with it).
__device__ __forceinline__ float row_sum(float v)
{
#pragma unroll
    for (int off = kRowLanes / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// 1 / rms over the row's first `norm_cols` columns (1 without a norm).  The whole
// warp calls it.
template <int K>
__device__ __forceinline__ float inv_rms(const uint4 (&v)[K], int norm_cols, float eps)
{
    if (norm_cols == 0) return 1.f;
    const int n = norm_cols / 64;   // pieces of this lane that take part
    float sq = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (k < n) {
            float x[8];
            unpack8(v[k], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) sq = fmaf(x[j], x[j], sq);
        }
    return 1.f / sqrtf(row_sum(sq) / (float)norm_cols + eps);
}

// Piece k of a row, normed: x_j r w_j (w = 1 without weights).
__device__ __forceinline__ void norm_piece(uint4 v, int k, float r, const uint16_t* weight, int l,
                                           float (&x)[8])
{
    unpack8(v, x);
    if (weight != nullptr) {
        float w[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(weight + 64 * k + 8 * l)), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] * r * w[j];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= r;
    }
}

// The position of token t, or -1 (reported by the caller's lane 0) if it is
// outside the table.
__device__ __forceinline__ int64_t position_of(const AppendArgs& a, int t)
{
    const int64_t p = __ldg(a.positions + t);
    return p >= 0 && p < a.max_positions ? p : -1;
}

template <int K>
__device__ __forceinline__ void append_row(const AppendArgs& a, int64_t t, int l)
{
    const bool on = t < a.tokens;
    const int32_t slot = on ? __ldg(a.slots + t) : -1;
    const int64_t pos = on ? position_of(a, (int)t) : -1;
    const bool inside = slot >= 0 && slot < a.pool_rows;
    if (on && l == 0) {
        if (slot >= 0 && !inside) atomicOr(a.err, MLA_DEVERR_BAD_SLOT);
        if (pos < 0) atomicOr(a.err, MLA_DEVERR_BAD_POSITION);
    }
    const bool write = inside && pos >= 0;
    uint4 v[K];
#pragma unroll
    for (int k = 0; k < K; ++k)
        v[k] = write ? load_once(a.kv + t * a.kv_stride + 64 * k + 8 * l) : make_uint4(0, 0, 0, 0);
    const Turn turn = load_turn(a.cos_sin + (write ? pos : 0) * 64, l, a.half_split != 0);
    const float r = inv_rms<K>(v, a.kv_norm_cols, a.eps);
    uint8_t* row = a.pool + (int64_t)(write ? slot : 0) * (64 * K) + 8 * l;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float x[8];
        if (64 * k < a.kv_norm_cols) norm_piece(v[k], k, r, a.kv_weight, l, x);
        else unpack8(v[k], x);
        if (k == K - 1) rotate(x, turn, a.half_split != 0);
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = (uint32_t)f32x2_to_e4m3x2(x[4 * i] * a.inv_scale, x[4 * i + 1] * a.inv_scale) |
                   ((uint32_t)f32x2_to_e4m3x2(x[4 * i + 2] * a.inv_scale,
                                              x[4 * i + 3] * a.inv_scale) << 16);
        if (write) *reinterpret_cast<uint2*>(row + 64 * k) = make_uint2(w[0], w[1]);
    }
}

// U heads of one token per eight lanes, their loads in flight together and the
// angles loaded once.
template <int K, int U>
__device__ __forceinline__ void query_rows(const AppendArgs& a, int64_t first, int g, int l)
{
    // group `first` + g: the CTA's first one is found once, the others from it
    const uint32_t per = (uint32_t)(a.heads + U - 1) / U;
    const uint32_t off = (uint32_t)(first % per) + g;
    const int64_t t = first / per + off / per;
    const int h0 = (int)(off % per) * U;
    const bool on = t < a.tokens;
    const int64_t pos = on ? position_of(a, (int)t) : -1;
    if (on && pos < 0 && l == 0 && h0 == 0) atomicOr(a.err, MLA_DEVERR_BAD_POSITION);
    const bool half = a.half_split != 0;
    const uint16_t* q = a.q + (on ? t : 0) * a.q_token_stride + 8 * l;
    uint4 v[U][K];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < K; ++k)
            v[u][k] = on && h0 + u < a.heads ? load_once(q + (h0 + u) * a.q_head_stride + 64 * k)
                                             : make_uint4(0, 0, 0, 0);
    const Turn turn = load_turn(a.cos_sin + (pos >= 0 ? pos : 0) * 64, l, half);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const bool write = pos >= 0 && h0 + u < a.heads;
        const int64_t row = t * a.heads + h0 + u;
        const float r = inv_rms<K>(v[u], a.q_norm ? 64 * K : 0, a.eps);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            uint4 y = v[u][k];   // without a norm the other columns pass through
            if (a.q_norm || k == K - 1) {
                float x[8];
                if (a.q_norm) norm_piece(y, k, r, a.q_weight, l, x);
                else unpack8(y, x);
                if (k == K - 1) rotate(x, turn, half);
                y = pack8(x);
            }
            uint16_t* to = k < K - 1 ? a.q_nope + row * (64 * (K - 1)) + 64 * k : a.q_pe + row * 64;
            if (write) __stcs(reinterpret_cast<uint4*>(to + 8 * l), y);
        }
    }
}

// Heads per eight lanes: about six 16-byte loads of queries in flight a lane.
template <int K>
constexpr int kHeads = K == 1 ? 4 : K <= 3 ? 2 : 1;

template <int KKV, int KQ>
__global__ void __launch_bounds__(kAppendThreads, 4)
append_kernel(const AppendArgs a)
{
    wait_for_predecessor();
    allow_dependents();
    const int g = threadIdx.x / kRowLanes, l = threadIdx.x % kRowLanes;
    if (blockIdx.x < a.kv_ctas)
        append_row<KKV>(a, (int64_t)blockIdx.x * kAppendRows + g, l);
    else
        query_rows<KQ, kHeads<KQ>>(a, (int64_t)(blockIdx.x - a.kv_ctas) * kAppendRows, g, l);
}

template <int KKV, int KQ>
cudaError_t launch_append(AppendArgs a, bool kv, cudaStream_t stream)
{
    const int64_t groups = (int64_t)a.tokens * ((a.heads + kHeads<KQ> - 1) / kHeads<KQ>);
    const int64_t kv_ctas = kv ? ((int64_t)a.tokens + kAppendRows - 1) / kAppendRows : 0;
    const int64_t ctas = kv_ctas + (groups + kAppendRows - 1) / kAppendRows;
    if (ctas == 0) return cudaSuccess;
    a.kv_ctas = (uint32_t)kv_ctas;
    return launch_dependent(append_kernel<KKV, KQ>, dim3((unsigned)ctas), kAppendThreads, stream,
                            true, a);
}

template <int KKV>
cudaError_t launch_append_q(const AppendArgs& a, bool kv, int kq, cudaStream_t stream)
{
    switch (kq) {
    case 1: return launch_append<KKV, 1>(a, kv, stream);
    case 2: return launch_append<KKV, 2>(a, kv, stream);
    case 3: return launch_append<KKV, 3>(a, kv, stream);
    case 4: return launch_append<KKV, 4>(a, kv, stream);
    case 5: return launch_append<KKV, 5>(a, kv, stream);
    case 6: return launch_append<KKV, 6>(a, kv, stream);
    case 7: return launch_append<KKV, 7>(a, kv, stream);
    case 8: return launch_append<KKV, 8>(a, kv, stream);
    default: return launch_append<KKV, 9>(a, kv, stream);
    }
}

// ---- row copies (fork, compaction) ------------------------------------------------------------
//
// A warp copies kCopyRows rows at a time: their 16-byte pieces, 36 (or 32) a
// row, are dealt out over the lanes in order, nine (eight) loads in flight per
// lane, neighbouring lanes on neighbouring pieces.

constexpr int kCopyThreads = 256;
constexpr int kCopyRows = 8;

// Lane first + i, i < kCopyRows, of the warp holds row i's source and destination
// slot (dst < 0: none).  The whole warp calls it.
template <int WIDTH>
__device__ __forceinline__ void copy_rows(uint8_t* pool, int32_t src, int32_t dst, int lane,
                                          int first = 0)
{
    constexpr int kPieces = WIDTH / 16;
    constexpr int kPer = kCopyRows * kPieces / 32;
    static_assert(kCopyRows * kPieces % 32 == 0, "pieces deal out evenly");
    uint4 v[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = lane + 32 * k, row = i / kPieces, piece = i % kPieces;
        const int32_t from = __shfl_sync(0xffffffffu, src, first + row);
        const int32_t to = __shfl_sync(0xffffffffu, dst, first + row);
        if (to >= 0)
            v[k] = __ldcs(reinterpret_cast<const uint4*>(pool + (int64_t)from * WIDTH) + piece);
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = lane + 32 * k, row = i / kPieces, piece = i % kPieces;
        const int32_t to = __shfl_sync(0xffffffffu, dst, first + row);
        if (to >= 0) __stcs(reinterpret_cast<uint4*>(pool + (int64_t)to * WIDTH) + piece, v[k]);
    }
}

constexpr int64_t kForkManyEntries = 1 << 17;

struct ForkArgs {
    uint8_t* pool;
    int64_t pool_rows;
    const int32_t* kv_indices;
    int64_t num_indices;
    const int32_t* kv_indptr;
    int32_t num_parents;
    const int32_t* parents;
    const int32_t* keep;
    const int32_t* child_indptr;
    int32_t num_children;
    const int32_t* fresh;
    int64_t num_fresh;
    const int32_t* fresh_indptr;
    int32_t* table;
    int64_t total;
    uint32_t* err;
};

// Table entry i and, if its row is copied, where from and to (dst -1: not).
__device__ __forceinline__ void fork_entry(const ForkArgs& a, int64_t i, int32_t& src,
                                           int32_t& dst)
{
    src = dst = -1;
    if (i >= a.total || i < __ldg(a.child_indptr)) return;
    // the child whose range holds i: the last f with child_indptr[f] <= i
    int lo = 0, hi = a.num_children;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.child_indptr + mid) <= i) lo = mid;
        else hi = mid;
    }
    const int f = lo;
    if (i >= __ldg(a.child_indptr + f + 1)) return;   // past the last child
    const int64_t j = i - __ldg(a.child_indptr + f);
    const int32_t p = __ldg(a.parents + f);
    const int64_t past = j - __ldg(a.keep + f);
    uint32_t bad = 0;
    int32_t entry = -1;
    if (p < 0 || p >= a.num_parents) {
        bad = MLA_DEVERR_BAD_TABLE;
    } else {
        const int64_t base = __ldg(a.kv_indptr + p);
        if (base + j >= __ldg(a.kv_indptr + p + 1)) {
            bad = MLA_DEVERR_BAD_LENGTH;
        } else if (base < 0 || base + j >= a.num_indices) {
            bad = MLA_DEVERR_BAD_TABLE;
        } else {
            const int32_t from = __ldg(a.kv_indices + base + j);
            if (past < 0) {
                entry = from;
                if (from < 0 || from >= a.pool_rows) bad = MLA_DEVERR_BAD_SLOT;
            } else {
                // keep[f] < 0 copies every row, the first to the first fresh slot
                const int64_t n = past < j ? past : j;
                const int64_t at = __ldg(a.fresh_indptr + f) + n;
                if (at < 0 || at >= __ldg(a.fresh_indptr + f + 1) || at >= a.num_fresh) {
                    bad = MLA_DEVERR_BAD_TABLE;
                } else {
                    entry = __ldg(a.fresh + at);
                    if (from < 0 || from >= a.pool_rows || entry < 0 || entry >= a.pool_rows) {
                        bad = MLA_DEVERR_BAD_SLOT;
                    } else {
                        src = from;
                        dst = entry;
                    }
                }
            }
        }
    }
    if (bad != 0) atomicOr(a.err, bad);
    a.table[i] = entry;
}

// A warp takes B * kCopyRows table entries, one per lane, and copies their rows in
// B turns.
template <int WIDTH, int B>
__global__ void __launch_bounds__(kCopyThreads)
fork_kernel(const ForkArgs a)
{
    wait_for_predecessor();
    allow_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t warp = (int64_t)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5);
    int32_t src = -1, dst = -1;
    if (lane < B * kCopyRows) fork_entry(a, warp * (B * kCopyRows) + lane, src, dst);
    const uint32_t any = __ballot_sync(0xffffffffu, dst >= 0);
#pragma unroll
    for (int b = 0; b < B; ++b)
        if ((any >> (b * kCopyRows)) & ((1u << kCopyRows) - 1u))
            copy_rows<WIDTH>(a.pool, src, dst, lane, b * kCopyRows);
}

// ---- compaction -------------------------------------------------------------------------------
//
// Live slots are bits of a bitmap.  With u(s) the number of live slots below s,
// L = u(pool_rows) and U = u(L), slot s < L that is not live is hole number
// s - u(s), and live slot s >= L is tail row number u(s) - U; there are L - U of
// each, and tail row k moves into hole k.  Sources lie at or past L and
// destinations below it, so the moves run in any order.
//   mark    sets the bits;
//   count   the live slots of each chunk of 8192 (only for large pools);
//   place   ranks: u at every bitmap word, the lists of holes and of tail rows;
//   move    copies the tail rows and rewrites the table.
// A small pool's mark and place are one CTA's work on a bitmap in shared memory
// (rank_kernel).  (One cooperative launch for everything, its phases parted by
// grid barriers of about 2 us, took 13.4, 20.0 and 77 us for the pools of 8192,
// 131072 and 1048576 rows that take 7.2, 16.4 and 70 this way.)

constexpr int64_t kMoveCtas = 4 * 152;
constexpr int kPlaceThreads = 256;                       // one bitmap word each
constexpr int64_t kChunkSlots = kPlaceThreads * 32;

struct CompactArgs {
    uint8_t* pool;
    int64_t pool_rows;
    const int32_t* kv_indices;
    int64_t num_indices;
    int32_t* new_indices;
    int32_t* live;
    uint32_t* err;
    uint32_t* bits;       // [words] live bitmap, words = chunks * kPlaceThreads
    int32_t* below;       // [words] u at the word's first slot
    int32_t* counts;      // [chunks]
    int32_t* totals;      // L, U
    int32_t* holes;       // [pool_rows / 2]
    int32_t* tail;        // [pool_rows / 2]
    int32_t chunks;
};

constexpr int kMarkEntries = 4;   // per thread

__global__ void __launch_bounds__(kCopyThreads)
mark_kernel(const CompactArgs a)
{
    wait_for_predecessor();
    allow_dependents();
    const int64_t i0 = (int64_t)blockIdx.x * (kMarkEntries * kCopyThreads) + threadIdx.x;
    int32_t s[kMarkEntries];
#pragma unroll
    for (int k = 0; k < kMarkEntries; ++k) {
        const int64_t i = i0 + k * kCopyThreads;
        s[k] = i < a.num_indices ? __ldg(a.kv_indices + i) : -1;
    }
#pragma unroll
    for (int k = 0; k < kMarkEntries; ++k) {
        if (s[k] < 0) continue;
        if (s[k] < a.pool_rows) atomicOr(a.bits + (s[k] >> 5), 1u << (s[k] & 31));
        else atomicOr(a.err, MLA_DEVERR_BAD_SLOT);
    }
}

// Sum over the CTA's threads; every thread gets it.  `part` holds one word per
// warp; a barrier precedes its reuse.
__device__ __forceinline__ int block_sum(int v, int* part)
{
    v = __reduce_add_sync(0xffffffffu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int w = 0; w < kPlaceThreads / 32; ++w) s += part[w];
    return s;
}

// A warp's 32 bitmap words from `word` on, one per lane with u at its first slot:
// their holes and tail rows into the lists, a word at a time, a slot per lane.
__device__ __forceinline__ void list_slots(const CompactArgs& a, uint32_t bits, int u, int64_t word,
                                           int L, int U)
{
    const int lane = threadIdx.x & 31;
    const uint32_t lower = (1u << lane) - 1u;
    for (int w = 0; w < 32; ++w) {
        const uint32_t b = __shfl_sync(0xffffffffu, bits, w);
        const int un = __shfl_sync(0xffffffffu, u, w) + __popc(b & lower);   // u at this slot
        const int64_t s = (word + w) * 32 + lane;
        const bool live = (b >> lane) & 1u;
        if (live && s >= L) a.tail[un - U] = (int32_t)s;
        if (!live && s < L) a.holes[s - un] = (int32_t)s;
    }
}

__global__ void __launch_bounds__(kPlaceThreads)
count_kernel(const CompactArgs a)
{
    __shared__ int part[kPlaceThreads / 32];
    wait_for_predecessor();
    allow_dependents();
    const int n = block_sum(__popc(__ldcg(a.bits + (int64_t)blockIdx.x * kPlaceThreads + threadIdx.x)),
                            part);
    if (threadIdx.x == 0) a.counts[blockIdx.x] = n;
}

// DIRECT: every CTA reads the whole bitmap (at most kDirectWords words, 32 a
// thread) and needs no counts.
constexpr int kDirectLoads = 8;   // of four words, per thread
constexpr int64_t kDirectWords = 4 * kDirectLoads * kPlaceThreads;

template <bool DIRECT>
__global__ void __launch_bounds__(kPlaceThreads)
place_kernel(const CompactArgs a)
{
    __shared__ int part[kPlaceThreads / 32];
    wait_for_predecessor();
    allow_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c = blockIdx.x;
    // L, the live slots below this chunk, and U
    int all = 0, before = 0, L, U;
    if constexpr (DIRECT) {
        uint4 b[kDirectLoads];
        auto first_of = [&](int k) { return (k * kPlaceThreads + tid) * 4; };   // word
#pragma unroll
        for (int k = 0; k < kDirectLoads; ++k) {
            b[k] = make_uint4(0u, 0u, 0u, 0u);
            if (first_of(k) < a.chunks * kPlaceThreads)
                b[k] = __ldcg(reinterpret_cast<const uint4*>(a.bits + first_of(k)));
        }
#pragma unroll
        for (int k = 0; k < kDirectLoads; ++k) {
            const int n = __popc(b[k].x) + __popc(b[k].y) + __popc(b[k].z) + __popc(b[k].w);
            all += n;
            before += first_of(k) < c * kPlaceThreads ? n : 0;
        }
        L = block_sum(all, part);
        before = block_sum(before, part);
        int under = 0;
#pragma unroll
        for (int k = 0; k < kDirectLoads; ++k) {
            const uint32_t w[4] = {b[k].x, b[k].y, b[k].z, b[k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = L - (first_of(k) + i) * 32;   // slots of this word below L
                under += n <= 0 ? 0 : __popc(n >= 32 ? w[i] : w[i] & ((1u << n) - 1u));
            }
        }
        U = block_sum(under, part);
    } else {
        for (int i = tid; i < a.chunks; i += kPlaceThreads) {
            const int n = __ldcg(a.counts + i);
            all += n;
            before += i < c ? n : 0;
        }
        L = block_sum(all, part);
        before = block_sum(before, part);
        // the chunks below L's chunk, and the bits of L's chunk below L
        const int lc = (int)(L / kChunkSlots);
        int under = 0;
        for (int i = tid; i < lc; i += kPlaceThreads) under += __ldcg(a.counts + i);
        if (lc < a.chunks) {
            const int64_t first = lc * kChunkSlots + (int64_t)tid * 32;
            const int64_t n = L - first;   // slots of this word below L
            const uint32_t w = __ldcg(a.bits + (int64_t)lc * kPlaceThreads + tid);
            under += n <= 0 ? 0 : __popc(n >= 32 ? w : w & ((1u << n) - 1u));
        }
        U = block_sum(under, part);
    }
    if (c == 0 && tid == 0) {
        a.totals[0] = L;
        a.totals[1] = U;
        a.live[0] = L;
    }
    // u at this thread's word
    const int64_t word = (int64_t)c * kPlaceThreads + tid;
    const uint32_t bits = __ldcg(a.bits + word);
    const int mine = __popc(bits);
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
    }
    __syncthreads();
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    int u = before + incl - mine;
    for (int w = 0; w < warp; ++w) u += part[w];
    a.below[word] = u;
    list_slots(a, bits, u, word - lane, L, U);
}

// Pools of at most kSmallRows rows whose tables have at most kSmallEntries
// entries: bitmap, ranks and lists by one CTA, one launch instead of a clear and
// three kernels.  (Measured: 8192 rows and 5,600 entries 9 us against 12 us; one
// CTA took 33 us for 131072 rows and 122,000 entries, the kernels 14.)
constexpr int kRankThreads = 1024;
constexpr int64_t kSmallRows = 32 * kRankThreads / 2;
constexpr int64_t kSmallEntries = 1 << 15;

__global__ void __launch_bounds__(kRankThreads)
rank_kernel(const CompactArgs a)
{
    constexpr int kWords = (int)(kSmallRows / 32);
    __shared__ uint32_t map[kWords];
    __shared__ int part[kRankThreads / 32];
    __shared__ int under_s;
    wait_for_predecessor();
    allow_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < kWords) map[tid] = 0;
    if (tid == 0) under_s = 0;
    __syncthreads();
    constexpr int kAhead = 8;
    for (int64_t i0 = tid; i0 < a.num_indices; i0 += kAhead * kRankThreads) {
        int32_t s[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            s[k] = i0 + k * kRankThreads < a.num_indices ? __ldg(a.kv_indices + i0 + k * kRankThreads) : -1;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (s[k] < 0) continue;
            if (s[k] < a.pool_rows) atomicOr(map + (s[k] >> 5), 1u << (s[k] & 31));
            else atomicOr(a.err, MLA_DEVERR_BAD_SLOT);
        }
    }
    __syncthreads();
    // ranks: a word per thread of the first half
    const uint32_t bits = tid < kWords ? map[tid] : 0u;
    int incl = __popc(bits);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
    }
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    int before = 0, L = 0;
    for (int w = 0; w < kRankThreads / 32; ++w) {
        const int n = part[w];
        before += w < warp ? n : 0;
        L += n;
    }
    // live slots below L
    const int n = L - tid * 32;
    int under = n <= 0 ? 0 : __popc(n >= 32 ? bits : bits & ((1u << n) - 1u));
    under = __reduce_add_sync(0xffffffffu, under);
    if (lane == 0) atomicAdd(&under_s, under);
    __syncthreads();
    const int U = under_s;
    if (tid == 0) {
        a.totals[0] = L;
        a.totals[1] = U;
        a.live[0] = L;
    }
    const int u = before + incl - __popc(bits);
    if (tid < a.chunks * kPlaceThreads) {   // whole warps
        a.bits[tid] = bits;
        a.below[tid] = u;
    }
    // the lists, the words dealt out over all warps
    __shared__ int below[kWords];
    if (tid < kWords) below[tid] = u;
    __syncthreads();
    const uint32_t lower = (1u << lane) - 1u;
    for (int w = warp; w < kWords; w += kRankThreads / 32) {
        const int64_t s = w * 32 + lane;
        if (w * 32 >= a.pool_rows) break;
        const uint32_t b = map[w];
        const int un = below[w] + __popc(b & lower);
        const bool live = (b >> lane) & 1u;
        if (live && s >= L) a.tail[un - U] = (int32_t)s;
        if (!live && s < L) a.holes[s - un] = (int32_t)s;
    }
}

// CTAs 0 .. move_ctas-1 copy the tail rows, eight a turn of a warp with the next
// turn's slots on their way; the others rewrite the table.
template <int WIDTH>
__global__ void __launch_bounds__(kCopyThreads, 4)
move_kernel(const CompactArgs a, int move_ctas)
{
    wait_for_predecessor();
    allow_dependents();
    const int32_t L = __ldcg(a.totals), U = __ldcg(a.totals + 1);
    const int lane = threadIdx.x & 31;
    if ((int)blockIdx.x < move_ctas) {
        const int moves = L - U;
        const int step = move_ctas * (kCopyThreads / 32) * kCopyRows;
        int k = ((int)blockIdx.x * (kCopyThreads / 32) + (int)(threadIdx.x >> 5)) * kCopyRows;
        int32_t src = -1, dst = -1;
        auto slots = [&](int at) {
            src = dst = -1;
            if (lane < kCopyRows && at + lane < moves) {
                src = __ldcg(a.tail + at + lane);
                dst = __ldcg(a.holes + at + lane);
            }
        };
        slots(k);
        for (; k < moves; k += step) {
            const int32_t s = src, d = dst;
            slots(moves - k > step ? k + step : moves);
            copy_rows<WIDTH>(a.pool, s, d, lane);
        }
        return;
    }
    const int64_t threads = (int64_t)(gridDim.x - move_ctas) * kCopyThreads;
    for (int64_t i = (int64_t)(blockIdx.x - move_ctas) * kCopyThreads + threadIdx.x;
         i < a.num_indices; i += threads) {
        const int32_t s = __ldcg(a.kv_indices + i);
        int32_t to = s;
        if (s >= L && s < a.pool_rows) {
            const int rank = __ldcg(a.below + (s >> 5)) +
                             __popc(__ldcg(a.bits + (s >> 5)) & ((1u << (s & 31)) - 1u)) - U;
            to = __ldcg(a.holes + rank);
        }
        a.new_indices[i] = to;
    }
}

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }
int64_t compact_chunks(int64_t rows) { return (rows + kChunkSlots - 1) / kChunkSlots; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_header(const void* ws, int64_t bytes)
{
    if (!ws) return MLA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return MLA_ERR_MISALIGNED;
    return bytes < MLA_WORKSPACE_HEADER_BYTES ? MLA_ERR_WORKSPACE_TOO_SMALL : MLA_OK;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? MLA_OK : MLA_ERR_LAUNCH_FAILED; }

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

int mla_cache_append(const void* kv, int64_t kv_stride, const void* kv_weight,
                     int32_t kv_norm_cols, const int32_t* slots, void* pool, int64_t pool_rows,
                     int32_t row_bytes, float kv_scale, const void* q, int64_t q_token_stride,
                     int64_t q_head_stride, const void* q_weight, int32_t q_norm, int32_t q_cols,
                     void* q_nope, void* q_pe, const int32_t* positions, const float* cos_sin,
                     int64_t max_positions, int32_t half_split, float eps, int32_t num_tokens,
                     int32_t num_heads, void* workspace, int64_t workspace_bytes, void* stream)
{
    if (num_tokens < 0 || num_heads < 0 || max_positions < 0) return MLA_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0.f) return MLA_ERR_INVALID_ARG;
    if (kv != nullptr) {
        if (row_bytes != 576 && row_bytes != 512) return MLA_ERR_UNSUPPORTED_SHAPE;
        if (kv_norm_cols != 0 && kv_norm_cols != row_bytes - 64 && kv_norm_cols != row_bytes)
            return MLA_ERR_UNSUPPORTED_SHAPE;
        if (!std::isfinite(kv_scale) || kv_scale == 0.f || !std::isfinite(1.f / kv_scale))
            return MLA_ERR_INVALID_ARG;
    }
    if (num_heads > 0 && (q_cols < 64 || q_cols > 576 || q_cols % 64 != 0 || num_heads > 128))
        return MLA_ERR_UNSUPPORTED_SHAPE;
    if (num_tokens == 0) return MLA_OK;
    if ((q != nullptr) != (num_heads > 0)) return MLA_ERR_INVALID_ARG;
    if (!positions || !cos_sin || max_positions < 1) return MLA_ERR_INVALID_ARG;
    if (!aligned16(cos_sin)) return MLA_ERR_MISALIGNED;
    if (kv != nullptr) {
        if (!slots || !pool || pool_rows < 1) return MLA_ERR_INVALID_ARG;
        if (!aligned16(kv) || !aligned16(kv_weight) || !aligned16(pool) || kv_stride % 8 != 0)
            return MLA_ERR_MISALIGNED;
    }
    if (q != nullptr) {
        if (!q_pe || (q_cols > 64 && !q_nope)) return MLA_ERR_INVALID_ARG;
        if (!aligned16(q) || !aligned16(q_weight) || !aligned16(q_nope) || !aligned16(q_pe) ||
            q_token_stride % 8 != 0 || q_head_stride % 8 != 0)
            return MLA_ERR_MISALIGNED;
    }
    int rc = check_header(workspace, workspace_bytes);
    if (rc != MLA_OK) return rc;
    rc = device_ok();
    if (rc != MLA_OK) return rc;

    AppendArgs a{};
    a.kv = static_cast<const uint16_t*>(kv);
    a.kv_stride = kv_stride;
    a.kv_weight = static_cast<const uint16_t*>(kv_weight);
    a.kv_norm_cols = kv_norm_cols;
    a.slots = slots;
    a.pool = static_cast<uint8_t*>(pool);
    a.pool_rows = pool_rows;
    a.inv_scale = kv != nullptr ? 1.f / kv_scale : 1.f;
    a.q = static_cast<const uint16_t*>(q);
    a.q_token_stride = q_token_stride;
    a.q_head_stride = q_head_stride;
    a.q_weight = static_cast<const uint16_t*>(q_weight);
    a.q_norm = q_norm;
    a.q_nope = static_cast<uint16_t*>(q_nope);
    a.q_pe = static_cast<uint16_t*>(q_pe);
    a.positions = positions;
    a.cos_sin = cos_sin;
    a.max_positions = max_positions;
    a.half_split = half_split;
    a.eps = eps;
    a.tokens = num_tokens;
    a.heads = num_heads;
    a.err = static_cast<uint32_t*>(workspace);
    const int kq = q != nullptr ? q_cols / 64 : 1;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return status_of(row_bytes == 512 ? launch_append_q<8>(a, kv != nullptr, kq, s)
                                      : launch_append_q<9>(a, kv != nullptr, kq, s));
}

int mla_cache_fork(void* pool, int64_t pool_rows, int32_t row_bytes, const int32_t* kv_indices,
                   int64_t num_indices, const int32_t* kv_indptr, int32_t num_parents,
                   const int32_t* parents, const int32_t* keep, const int32_t* child_indptr,
                   int32_t num_children, const int32_t* fresh, int64_t num_fresh,
                   const int32_t* fresh_indptr, int32_t* table, int64_t total, void* workspace,
                   int64_t workspace_bytes, void* stream)
{
    if (num_parents < 0 || num_children < 0 || num_indices < 0 || num_fresh < 0 || total < 0)
        return MLA_ERR_INVALID_ARG;
    if (row_bytes != 576 && row_bytes != 512) return MLA_ERR_UNSUPPORTED_SHAPE;
    if (total > INT32_MAX) return MLA_ERR_UNSUPPORTED_SHAPE;
    if (num_children == 0 || total == 0) return MLA_OK;
    if (!pool || pool_rows < 1 || !kv_indptr || !parents || !keep || !child_indptr ||
        !fresh_indptr || !table || (num_indices > 0 && !kv_indices) || (num_fresh > 0 && !fresh))
        return MLA_ERR_INVALID_ARG;
    if (!aligned16(pool)) return MLA_ERR_MISALIGNED;
    int rc = check_header(workspace, workspace_bytes);
    if (rc != MLA_OK) return rc;
    rc = device_ok();
    if (rc != MLA_OK) return rc;
    const ForkArgs a{static_cast<uint8_t*>(pool), pool_rows, kv_indices, num_indices, kv_indptr,
                     num_parents, parents, keep, child_indptr, num_children, fresh, num_fresh,
                     fresh_indptr, table, total, static_cast<uint32_t*>(workspace)};
    // Four turns a warp amortise the look-up of its entries once every SM has
    // work without that.
    const bool many = total > kForkManyEntries;
    const int64_t per = kCopyThreads / 32 * kCopyRows * (many ? 4 : 1);
    const dim3 grid((unsigned)((total + per - 1) / per));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto* kernel = row_bytes == 576 ? (many ? fork_kernel<576, 4> : fork_kernel<576, 1>)
                                    : (many ? fork_kernel<512, 4> : fork_kernel<512, 1>);
    return status_of(launch_dependent(kernel, grid, kCopyThreads, s, true, a));
}

int64_t mla_cache_compact_workspace_bytes(int64_t pool_rows)
{
    if (pool_rows < 1 || pool_rows > INT32_MAX) return 0;
    const int64_t chunks = compact_chunks(pool_rows);
    return MLA_WORKSPACE_HEADER_BYTES + 2 * align256(chunks * kPlaceThreads * 4) +
           align256(chunks * 4) + 256 + 2 * align256((pool_rows / 2 + 1) * 4);
}

int mla_cache_compact(void* pool, int64_t pool_rows, int32_t row_bytes,
                      const int32_t* kv_indices, int64_t num_indices, int32_t* new_indices,
                      int32_t* live, void* workspace, int64_t workspace_bytes, void* stream)
{
    if (num_indices < 0 || pool_rows < 1) return MLA_ERR_INVALID_ARG;
    if (row_bytes != 576 && row_bytes != 512) return MLA_ERR_UNSUPPORTED_SHAPE;
    if (pool_rows > INT32_MAX || num_indices > INT32_MAX) return MLA_ERR_UNSUPPORTED_SHAPE;
    if (!pool || !live || (num_indices > 0 && (!kv_indices || !new_indices)))
        return MLA_ERR_INVALID_ARG;
    if (!aligned16(pool)) return MLA_ERR_MISALIGNED;
    int rc = check_header(workspace, workspace_bytes);
    if (rc != MLA_OK) return rc;
    if (workspace_bytes < mla_cache_compact_workspace_bytes(pool_rows))
        return MLA_ERR_WORKSPACE_TOO_SMALL;
    rc = device_ok();
    if (rc != MLA_OK) return rc;

    CompactArgs a{};
    a.pool = static_cast<uint8_t*>(pool);
    a.pool_rows = pool_rows;
    a.kv_indices = kv_indices;
    a.num_indices = num_indices;
    a.new_indices = new_indices;
    a.live = live;
    a.chunks = (int32_t)compact_chunks(pool_rows);
    char* p = static_cast<char*>(workspace);
    a.err = reinterpret_cast<uint32_t*>(p);
    p += MLA_WORKSPACE_HEADER_BYTES;
    const int64_t words = align256((int64_t)a.chunks * kPlaceThreads * 4);
    a.bits = reinterpret_cast<uint32_t*>(p);
    a.below = reinterpret_cast<int32_t*>(p + words);
    p += 2 * words;
    a.counts = reinterpret_cast<int32_t*>(p);
    p += align256((int64_t)a.chunks * 4);
    a.totals = reinterpret_cast<int32_t*>(p);
    p += 256;
    a.holes = reinterpret_cast<int32_t*>(p);
    a.tail = reinterpret_cast<int32_t*>(p + align256((pool_rows / 2 + 1) * 4));

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (pool_rows <= kSmallRows && num_indices <= kSmallEntries) {
        e = launch_dependent(rank_kernel, dim3(1), kRankThreads, s, true, a);
    } else {
        e = cudaMemsetAsync(a.bits, 0, (size_t)a.chunks * kPlaceThreads * 4, s);
        const int64_t per = kMarkEntries * kCopyThreads;
        if (e == cudaSuccess && num_indices > 0)
            e = launch_dependent(mark_kernel, dim3((unsigned)((num_indices + per - 1) / per)),
                                 kCopyThreads, s, false, a);
        const bool direct = (int64_t)a.chunks * kPlaceThreads <= kDirectWords;
        if (e == cudaSuccess && !direct)
            e = launch_dependent(count_kernel, dim3((unsigned)a.chunks), kPlaceThreads, s,
                                 num_indices > 0, a);
        if (e == cudaSuccess)
            e = launch_dependent(direct ? place_kernel<true> : place_kernel<false>,
                                 dim3((unsigned)a.chunks), kPlaceThreads, s,
                                 !direct || num_indices > 0, a);
    }
    if (e == cudaSuccess) {
        // one turn a warp in the worst case, at most four CTAs an SM of a full GPU
        // (a CTA loops over the rest)
        const int64_t turn = kCopyThreads / 32 * kCopyRows;
        const int64_t most = (pool_rows / 2 + turn - 1) / turn;
        const int64_t remap = (num_indices + kCopyThreads - 1) / kCopyThreads;
        const int move_ctas = (int)(most < kMoveCtas ? most : kMoveCtas);
        const int remap_ctas = (int)(remap < kMoveCtas ? remap : kMoveCtas);
        if (move_ctas + remap_ctas > 0)
            e = launch_dependent(row_bytes == 576 ? move_kernel<576> : move_kernel<512>,
                                 dim3((unsigned)(move_ctas + remap_ctas)), kCopyThreads, s, true, a,
                                 move_ctas);
    }
    return status_of(e);
}

}  // extern "C"
