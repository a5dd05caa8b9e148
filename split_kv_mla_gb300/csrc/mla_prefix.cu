// mla_prefix.cu -- decode of a batch whose requests share a prefix: the
// prefix's keys are attended once by the query rows of the whole batch, 64 rows
// per tile, instead of once per request.  See mla_prefix_decode in
// include/mla_decode.h for the contract.
//
// Three kernels:
//
// * prepare: gathers the keys' rows through their slot lists into 128-key
//   blocks laid out exactly as the MMA reads them (mla_layout.cuh), and splits
//   each query row into two e4m3 terms the same way.  Both are then fetched with
//   plain bulk copies of whole 16 KB chunks: a row gather cannot feed 64-row
//   tiles (160 tile::gather4 copies of a block take ~3,800 cycles, as long as
//   all its MMAs), and every tile reads the same prefix blocks.
// * prefix_split: a tile's blocks are the prefix's, then those of the requests
//   that have rows in the tile (their own keys, masked for the other requests'
//   rows); or, where the requests' own keys are long, the prefix's alone and
//   the split kernel (mla_split_kernel.cuh) does the others.  Per CTA runs of
//   (tile, block) pairs; per block
//     S^T[128 keys x 128] = K[128 x 576] . [q_hi | q_lo]^T      one MMA chain
//     p = 2^(s - m),  O^T[512 x 64] += V^T[512 x 128] . (p_hi + p_lo)
//   with K and V e4m3 as they are stored.  A query row, scaled to max |q| in
//   [128, 256), is q_hi + 2^-5 q_lo, both e4m3: exact for a bf16 element within
//   2^-14 of the row's maximum and off by at most 2^-22 of that maximum below.
//   Where that could move a logit by 2^-11, the row's tile adds a third term, the
//   rest in e5m2 in q_lo's units: exact within 2^-18 of the maximum, off by at most
//   2^-26 of it below.
//   p = p_hi + p_lo is an e4m3 term and the residual in e5m2, whose 2^-16
//   smallest step lets both terms accumulate into the same columns without a
//   scale of their own (a second set of columns does not fit: O^T takes 256 of
//   TMEM's 512 columns at 64 rows, the two S^T buffers the others).  The pair is
//   off by at most 4.2e-3 of p (1.3e-3 in the mean square; rounding to bf16: 3.9e-3
//   and 1.6e-3) down to 2^-12 of the row's reference, by 1.4e-2 at 2^-14 and 0.11
//   from 2^-17 on.  O is divided by the sum of what was fed, so common errors cancel.
// * prefix_merge: joins a row's partials by their base-2 LSEs.
//
// What bounds the split kernel: shared memory's 128 bytes a cycle.  A block of
// 128 keys and 64 rows reads 18 x 8 KB for QK (both terms stacked along N, so K
// is read once) and 32 x 6 KB for P.V (V once per term), the bulk copies write
// 72 KB and the softmax 16 KB: 435 KB, 3,400 cycles, against 2,176 of
// multiplying at the bf16 rate.  It takes 1.92 us, about 3,700 (the MMAs alone, back
// to back: 18 x 73 + 32 x 58 = 3,170).  More rows per tile would read less per
// row, but O^T and the S^T buffers fill TMEM and the stages, queries and P fill
// shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "mla_internal.h"
#include "mla_layout.cuh"
#include "mla_sm100.cuh"
#include "mla_softmax.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kDv = 512, kDr = 64, kWidth = kDv + kDr;
constexpr int kRows = kPrefixRows;
constexpr int kKeys = kPrefixKeys;
constexpr int kChunk = kKeys * 128;           // bytes of one 128-column chunk of 128 rows
constexpr int kRopeBytes = kKeys * 64;
static_assert(4 * kChunk + kRopeBytes == kPrefixImage, "image of a block or a query tile");
static_assert(2 * kRows == kKeys, "a query tile's two terms have a block's layout");
constexpr int kQLoBits = 5;                   // q_lo is stored times 2^5
constexpr float kQLoBack = 1.f / (1 << kQLoBits);
// The largest error of a base-2 logit that a tile's two terms may leave (by a bound
// with every key at +-448; with random keys a thirtieth of it): half the LSE's bar.
constexpr float kThirdAbove = 1.f / 2048.f;
// Two terms carry a scaled bf16 element of at least 2^-7 exactly; of a smaller one
// they leave up to 2^-15.
constexpr float kTwoTerms = 1.f / 128.f, kTwoTermsLeave = 1.f / 32768.f;

// A grid kernel launched as a programmatic dependent of its predecessor.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, int threads, int smem,
                       cudaStream_t stream, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// The prefix's length: the device value clamped to its list (prepare reports one
// outside), or the list's own length.
__device__ __forceinline__ int prefix_length(const PrefixArgs& a)
{
    if (a.prefix_len == nullptr) return a.prefix_cap;
    return min(max(__ldcg(a.prefix_len), 0), a.prefix_cap);
}

// The own blocks' images follow those that the longest prefix takes.
__device__ __forceinline__ int prefix_image_blocks(const PrefixArgs& a)
{
    return (a.prefix_cap + kKeys - 1) / kKeys;
}

// Request b's own keys: how many are in use, and where its table starts.  A
// length outside its table is clamped (the caller reports it), as is a table
// that reaches past the plan's entries.
__device__ __forceinline__ int own_length(const PrefixArgs& a, int b, int& first)
{
    first = __ldg(a.kv_indptr + b);
    const int cap = __ldg(a.kv_indptr + b + 1) - first;
    const int len = min(max(__ldg(a.seq_lens + b), 0), max(cap, 0));
    return first < 0 || first > a.total_keys ? 0 : min(len, a.total_keys - first);
}

// The block of the own images where request b's keys start.
__device__ __forceinline__ int own_block0(int first, int b) { return first / kKeys + b; }

// Requests that have rows in tile t: [first, last].
__device__ __forceinline__ void tile_requests(const PrefixArgs& a, int64_t t, int& b0, int& b1)
{
    const int64_t per = (int64_t)a.q_len * a.num_heads;
    b0 = (int)(t * kRows / per);
    b1 = (int)((min(t * kRows + kRows, a.rows) - 1) / per);
}

// How a tile's blocks are dealt out.  With `splits`, CTA t * splits + s takes the
// s-th of equal parts of tile t; else the tile-major sequence of all U blocks is
// cut into equal runs, CTA g taking blocks [g U / G, (g + 1) U / G), G <= U.
// Then the CTA of block u is:
__device__ __forceinline__ int64_t cta_of(int64_t u, int64_t U, int64_t G)
{
    return ((u + 1) * G - 1) / U;
}
// The first block of part s of `splits` equal parts of nb < 2^24 blocks.
__device__ __forceinline__ uint32_t part_begin(uint32_t nb, int s, int splits)
{
    return nb * (uint32_t)s / (uint32_t)splits;
}
// A run of CTA g in tile t leaves its partial rows in slot g with `splits`, in
// slot g + t without (runs follow one another by a step of g or of t).

// ---- prepare ----------------------------------------------------------------------------------

constexpr int kPrepThreads = 256;
constexpr int kPrepKeys = 32;     // keys per CTA
constexpr int kPrepRows = kPrepThreads / 32;   // query rows per CTA, one per warp

// The top bits of v's bytes that are e4m3fn NaN codes (magnitude 0x7f).
__device__ __forceinline__ uint32_t nan_bits(uint32_t v)
{
    return ((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}
// v with its NaN codes as zeros.
__device__ __forceinline__ uint32_t without_nan(uint32_t v)
{
    return v & ~((nan_bits(v) >> 7) * 0xffu);
}

// Keys [k0, k0 + 32) of a list of `len` into rows k0 % 128 .. of block k0 / 128 of
// `image`, as zero rows past the list's end and for bad slots.  A tile's rows need
// not all see a key, and 0 x NaN is NaN in P.V: NaN codes become zeros here and
// their keys are marked, so that the rows that see such a key (and only they)
// take a NaN logit.  flags: valid and marked keys, a bit each.  The whole CTA.
__device__ __forceinline__ void prepare_keys(const PrefixArgs& a, const int32_t* list, int k0,
                                             int len, uint8_t* image, uint2* flags)
{
    __shared__ int32_t slots[kPrepKeys];
    const int tid = threadIdx.x;
    flags += k0 / kPrepKeys;
    if (tid < kPrepKeys) {
        int32_t s = k0 + tid < len ? __ldg(list + k0 + tid) : -1;
        if (k0 + tid < len && (s < 0 || s >= a.pool_rows)) {
            atomicOr(a.err, MLA_DEVERR_BAD_SLOT);
            s = -1;
        }
        slots[tid] = s;
        const uint32_t valid = __ballot_sync(0xffffffffu, s >= 0);
        if (tid == 0) *flags = make_uint2(valid, 0u);
    }
    __syncthreads();
    image += k0 / kKeys * kPrefixImage;
    const int row0 = k0 % kKeys;
    constexpr int kPieces = kWidth / 16;
    constexpr int kPer = (kPrepKeys * kPieces + kPrepThreads - 1) / kPrepThreads;
    uint4 v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int p = tid + i * kPrepThreads, row = p / kPieces;
        v[i] = make_uint4(0, 0, 0, 0);
        if (p < kPrepKeys * kPieces && slots[row] >= 0)
            v[i] = __ldg(reinterpret_cast<const uint4*>(a.pool + (int64_t)slots[row] * kWidth) +
                         p % kPieces);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int p = tid + i * kPrepThreads, row = p / kPieces;
        if (p >= kPrepKeys * kPieces) continue;
        if ((nan_bits(v[i].x) | nan_bits(v[i].y) | nan_bits(v[i].z) | nan_bits(v[i].w)) != 0) {
            atomicOr(&flags->y, 1u << row);
            v[i] = make_uint4(without_nan(v[i].x), without_nan(v[i].y), without_nan(v[i].z),
                              without_nan(v[i].w));
        }
        *reinterpret_cast<uint4*>(image + tile_offset(row0 + row, p % kPieces * 16, kKeys)) = v[i];
    }
}

// Quarter c % 4 of own block c / 4, if a request's keys reach it.
__device__ void prepare_own(const PrefixArgs& a, int c)
{
    const int block = c / 4, lane = threadIdx.x & 31;
    // the last request whose first block is at most `block`: 32 probes a step
    int lo = 0, n = a.batch;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int b = lo + lane * step;
        const bool le = lane * step < n && (lane == 0 || own_block0(__ldg(a.kv_indptr + b), b) <= block);
        const int hit = 31 - __clz(__ballot_sync(0xffffffffu, le));
        lo += hit * step;
        n = min(step, n - hit * step);
    }
    int first;
    const int len = own_length(a, lo, first);
    const int k0 = (block - own_block0(first, lo)) * kKeys + c % 4 * kPrepKeys;
    if (k0 < 0 || k0 >= (len + kKeys - 1) / kKeys * kKeys) return;
    const int64_t at = prefix_image_blocks(a) + own_block0(first, lo);
    prepare_keys(a, a.kv_indices + first, k0, len, a.k_image + at * kPrefixImage, a.k_flags + at * 4);
}

// Blocks before each tile, by one CTA; it also reports bad lengths.
__device__ void prepare_tiles(const PrefixArgs& a)
{
    __shared__ int64_t part[kPrepThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int len = prefix_length(a);
    if (tid == 0 && a.prefix_len != nullptr && __ldcg(a.prefix_len) != len)
        atomicOr(a.err, MLA_DEVERR_BAD_LENGTH);
    int64_t before = 0;
    for (int64_t t0 = 0; t0 < a.tiles; t0 += kPrepThreads) {
        const int64_t t = t0 + tid;
        int64_t mine = 0;
        if (t < a.tiles) {
            mine = (len + kKeys - 1) / kKeys;
            if (a.joined || a.own_splits == 0) {   // (else the split kernel reports)
                int b0, b1;
                tile_requests(a, t, b0, b1);
                for (int b = b0; b <= b1; ++b) {
                    int first;
                    const int n = own_length(a, b, first);
                    if (n != __ldg(a.seq_lens + b)) atomicOr(a.err, MLA_DEVERR_BAD_LENGTH);
                    mine += (n + kKeys - 1) / kKeys;   // none without entries
                }
            }
        }
        int64_t incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += v;
        }
        __syncthreads();
        if (lane == 31) part[warp] = incl;
        __syncthreads();
        int64_t base = before;
        for (int w = 0; w < kPrepThreads / 32; ++w) {
            if (w < warp) base += part[w];
            before += part[w];
        }
        if (t < a.tiles) a.tile_start[t] = base + incl - mine;
    }
    if (tid == 0) a.tile_start[a.tiles] = before;
}

// x * 2^k as two multiplications by powers of two (mul_pow2 with its branches taken
// once: k is a row's).
struct Pow2 {
    float a, b;
    __device__ __forceinline__ explicit Pow2(int k)
    {
        const int k0 = min(max(k, -126), 127);
        a = __uint_as_float((uint32_t)(k0 + 127) << 23);
        b = __uint_as_float((uint32_t)(k - k0 + 127) << 23);
    }
    __device__ __forceinline__ float operator()(float x) const { return x * a * b; }
};

// Query row `item`, eight columns (lane + 32 i) 8 .. + 7 per lane and i, and the
// largest magnitude in it.  The whole warp.
constexpr int kQueryVec = (kWidth / 8 + 31) / 32;
__device__ __forceinline__ float load_query(const PrefixArgs& a, int64_t item, int lane,
                                            uint4 (&v)[kQueryVec])
{
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kQueryVec; ++i) {
        const int c = (lane + 32 * i) * 8;
        v[i] = make_uint4(0, 0, 0, 0);
        if (item < a.rows && c < kWidth)
            v[i] = c < kDv ? __ldg(reinterpret_cast<const uint4*>(a.q_lat + item * kDv + c))
                           : __ldg(reinterpret_cast<const uint4*>(a.q_pe + item * kDr + (c - kDv)));
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[k] << 16)),
                                     fabsf(__uint_as_float(w[k] & 0xFFFF0000u))));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    return amax;
}

// Query row `item` (one warp) into its tile's image, rows 0..63 the high terms
// and 64..127 the low ones; its logit scale and the positions it sees, with the
// sign bit set if the row wants its third term.
__device__ void prepare_query(const PrefixArgs& a, int64_t item)
{
    const int lane = threadIdx.x & 31;
    if (item >= (int64_t)a.tiles * kRows) return;
    const bool on = item < a.rows;
    uint4 v[kQueryVec];
    const float amax = load_query(a, item, lane, v);
    const int sh = q_shift(amax);
    const Pow2 scale(sh);
    uint8_t* image = a.q_image + item / kRows * kPrefixImage;
    const int row = (int)(item % kRows);
    int small = 0;   // elements that the two terms do not carry exactly
#pragma unroll
    for (int i = 0; i < kQueryVec; ++i) {
        const int c = (lane + 32 * i) * 8;
        if (c >= kWidth) continue;
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint16_t h[4], l[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float x0 = scale(__uint_as_float(w[k] << 16));
            const float x1 = scale(__uint_as_float(w[k] & 0xFFFF0000u));
            split_pair<kQLoBits>(x0, x1, h[k], l[k]);
            small += (x0 != 0.f && fabsf(x0) < kTwoTerms ? 1 : 0) +
                     (x1 != 0.f && fabsf(x1) < kTwoTerms ? 1 : 0);
        }
        *reinterpret_cast<uint2*>(image + tile_offset(row, c, kKeys)) =
            make_uint2((uint32_t)h[0] | ((uint32_t)h[1] << 16), (uint32_t)h[2] | ((uint32_t)h[3] << 16));
        *reinterpret_cast<uint2*>(image + tile_offset(kRows + row, c, kKeys)) =
            make_uint2((uint32_t)l[0] | ((uint32_t)l[1] << 16), (uint32_t)l[2] | ((uint32_t)l[3] << 16));
    }
    small = __reduce_add_sync(0xffffffffu, small);
    if (lane == 0) {
        // (rows past the batch's last see everything: a mask would cost every block)
        int64_t win = INT32_MAX;
        if (on) {
            // draft row t sees positions <= P + S_b - q_len + t, the prefix's first
            const int64_t r = item / a.num_heads;
            const int b = (int)(r / a.q_len), t = (int)(r % a.q_len);
            const int cap = __ldg(a.kv_indptr + b + 1) - __ldg(a.kv_indptr + b);
            const int len = min(max(__ldg(a.seq_lens + b), 0), max(cap, 0));
            const int64_t P = prefix_length(a);
            win = max((int64_t)0, P + len - a.q_len + t + 1);
            win = min(win, a.joined ? (int64_t)INT32_MAX : P);
        }
        // (an infinite query has no finite terms: its logits are NaN)
        const float cq = !on ? 0.f : isinf(amax) ? CUDART_NAN_F : mul_pow2(a.logit_scale, -sh);
        const bool third = (float)small * (kTwoTermsLeave * 448.f) * fabsf(cq) > kThirdAbove;
        a.q_scale[item] = cq;
        a.q_window[item] = (int32_t)win | (third ? INT32_MIN : 0);
    }
}

// CTA 0 ranks the tiles, then own_ctas CTAs of own keys (the longest chain of
// loads first), query_ctas of queries and the rest of prefix keys.
__global__ void __launch_bounds__(kPrepThreads)
prefix_prepare_kernel(const PrefixArgs a, int own_ctas, int query_ctas)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    int c = (int)blockIdx.x - 1;
    if (c < 0) {
        prepare_tiles(a);
    } else if (c < own_ctas) {
        prepare_own(a, c);
    } else if ((c -= own_ctas) < query_ctas) {
        prepare_query(a, (int64_t)c * kPrepRows + (threadIdx.x >> 5));
    } else {
        c -= query_ctas;
        const int len = prefix_length(a);
        if (c * kPrepKeys < (len + kKeys - 1) / kKeys * kKeys)
            prepare_keys(a, a.prefix_indices, c * kPrepKeys, len, a.k_image, a.k_flags);
    }
}

// ---- prefix_split -----------------------------------------------------------------------------
//
// Warp 0 loads, warp 1 issues the MMAs, warp 2 looks up the tile's requests, warps 2
// and 3 write third terms, warps 4-11 are two softmax sets of four warps; set s owns
// query rows 32 s .. 32 s + 31, warp w % 4 of a set the TMEM lanes (keys) 32 (w % 4)
// .. + 31, one key per thread, as in the split kernel.
//
// A stage's four latent chunks are released one by one, as the P.V MMAs of that
// chunk finish, so the next block's chunks stream in behind them; the RoPE
// chunk, which only QK reads, has one buffer.  QK of block j + 1 runs while the
// softmax works on block j, and P.V of block j - 1 before it.
//
// A tile with a row that wants its third term holds those terms (64 rows, 36 KB) in
// one of the two stages, where warps 2 and 3 write them from the queries when a run
// starts.  All of its blocks then pass through the other stage, each chunk behind the
// P.V of the block before, and QK makes a second pass over the block, which adds the
// third terms to the low terms' columns of S^T.  (Measured: 64 requests of 128 heads
// on 32768 positions 462 us without such a row, 757 with one in the batch, 836 with
// all rows; 4 of 16 heads on 1024 18.5, 23.0 and 38.2.  Nothing else held those 36
// KB: shared memory is full, and the workspace's layout is the plan's.  A loop of its
// own for such tiles slowed the others: the roles' loops together just fill the
// instruction cache, 82 % of whose requests hit without that code, 70 % with it.)

constexpr int kThreads = 384;
constexpr int kLoadWarp = 0, kMmaWarp = 1, kTileWarp = 2, kSoftmaxWarp0 = 4;
constexpr int kSets = 2, kSetRows = kRows / kSets;
constexpr int kSoftmaxWarps = 4 * kSets;
// 168 registers a thread at launch (384 x 168 <= 65536); the first warpgroup
// gives back what the softmax warpgroups take.  (With 56 and 224 the MMA role's
// descriptors spilled: 528 us instead of 463 at 64 requests of 128 heads.)
constexpr uint32_t kRegsLow = 72, kRegsHigh = 216;
static_assert(128 * kRegsLow + 256 * kRegsHigh <= 384 * 168, "register split");

// Softmax constants, in base-2 logit units: a row's reference moves when a
// logit passes it by more than kTau, then to the block's maximum plus
// kHeadroom; p is fed as 2^(s - m + kShift) <= 2^8.75 < 448.
constexpr float kTau = 2.75f, kShift = 6.f, kHeadroom = 1.f;
constexpr float kTop = kTau + kShift;

constexpr int kOffRope = 2 * 4 * kChunk;
constexpr int kOffQ = kOffRope + kRopeBytes;
constexpr int kOffP = kOffQ + (int)kPrefixImage;
constexpr int kPTerm = kKeys * kRows;            // bytes of one term of P^T
constexpr int kOffMisc = kOffP + 2 * kPTerm;
constexpr uint32_t kColS = 0, kColO = 256, kTmemCols = 512;
static_assert(kOffQ % 1024 == 0 && kOffP % 1024 == 0, "swizzle atoms");
static_assert(kRows * kDv * 4 <= kOffRope, "the epilogue stages its rows in the idle stages");
static_assert(2 * kRows * 128 <= kChunk && kRows * 64 <= kRows * 128, "the third terms fit in a stage");

struct PrefixShared {
    uint64_t k_full[2][4], k_empty[2][4];   // per stage and chunk
    uint64_t r_full, r_empty, q_full, q3_full;
    uint64_t s_full[2], s_free[2];
    uint64_t p_full, pv_done;
    uint64_t mma_drain;   // after an abort: every MMA issued has completed
    uint64_t never;       // tests of the timeout path
    uint32_t tmem_base;
    int abort;
    alignas(16) float cq[kRows];
    alignas(16) int win[kRows];
    alignas(16) float delta[kRows];   // a reference's step
    alignas(16) float scale[kRows];   // 2^step; epilogue: 1 / the sum of what the MMA consumed
    uint32_t set_now[kSets], shrunk[kSets];   // rows that got a reference, that moved theirs
    int stop[kSets];
    alignas(16) float red[kSoftmaxWarps][32];
    // the tile's requests: own blocks before each, where its images start
    uint64_t own_full;
    int own_before[kRows + 1];
    int own_image[kRows];
};
constexpr int kSmemBytes = kOffMisc + (int)sizeof(PrefixShared);
static_assert(kSmemBytes <= 227 * 1024, "one CTA's dynamic shared memory limit");

// p (two rows) as an e4m3 term and the residual as an e5m2 term; returns the
// sums that the MMA will see.  fp16 holds p <= 448 and the residual exactly
// enough: p to 2^-12 of itself, the difference exactly.
__device__ __forceinline__ float2 split_p(float a, float b, uint16_t& hi, uint16_t& lo)
{
    uint32_t p, back, rest, low, sum;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(p) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hi) : "r"(p));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(hi));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(p), "r"(back));
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(lo) : "r"(rest));
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(low) : "h"(lo));
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(sum) : "r"(back), "r"(low));
    return __half22float2(*reinterpret_cast<const __half2*>(&sum));
}

// A run: blocks [x0, x1) of a tile's nb, of which `shared` are the prefix's and the
// others its requests' own.  The own blocks are spread evenly among the
// prefix's, so that no run is made of own blocks alone: there every request's
// first block would start its rows' softmax anew (measured, with the own blocks
// behind the prefix's the CTAs that had them took 34 us, the others 24).  `j0`
// blocks went before in this CTA (the pipeline's phases go on counting), `run`
// runs.
struct Run {
    int64_t tile;
    int x0, x1, nb;
    int shared;
    int64_t slot;   // where its partial rows go
    int64_t j0;
    int run;
};

// Walks a run's blocks in order: block x is own if floor((x + 1) no / nb) is past
// floor(x no / nb) = y, no the tile's own blocks, and then own block y; else block
// x - y of the prefix.
struct Walk {
    int x, y, k;      // k: number in the tile of own block y's request (once looked up)
    int64_t acc;      // x no mod nb
    __device__ __forceinline__ explicit Walk(const Run& r) : x(r.x0), k(0)
    {
        y = 0;
        acc = 0;
        if (r.nb > r.shared) {
            const int64_t t = (int64_t)r.x0 * (r.nb - r.shared);
            y = (int)(t / r.nb);
            acc = t % r.nb;
        }
    }
    __device__ __forceinline__ bool own(const Run& r) const
    {
        return acc + (r.nb - r.shared) >= r.nb;
    }
    __device__ __forceinline__ void next(const Run& r)
    {
        const bool o = own(r);
        acc += (r.nb - r.shared) - (o ? r.nb : 0);
        y += o ? 1 : 0;
        ++x;
    }
    // The image of the block (an own one's request looked up by warp 2).
    __device__ __forceinline__ int64_t image(const Run& r, const PrefixShared& ms)
    {
        if (!own(r)) return x - y;
        while (y >= ms.own_before[k + 1]) ++k;
        return (int64_t)ms.own_image[k] + (y - ms.own_before[k]);
    }
};

// Two of the tile's rows per lane, negative if one wants its third term, and whether
// any of the tile's does.  The whole warp.
__device__ __forceinline__ int32_t third_flags(const PrefixArgs& a, const Run& r, int lane)
{
    const int32_t* w = a.q_window + r.tile * kRows + lane;
    return __ldcg(w) | __ldcg(w + 32);
}
__device__ __forceinline__ bool any_third(int32_t flags)
{
    return __any_sync(0xffffffffu, flags < 0);
}

// The stage that holds block jj of the run.
__device__ __forceinline__ int stage_of(const Run& r, int64_t jj, bool third)
{
    return (int)((third ? r.j0 : jj) & 1);
}

// Where a run keeps its tile's third terms: their chunks as far apart as those of the
// other terms (so that QK's second pass differs from its first in a base address), the
// RoPE chunk in the first gap.
constexpr int kThirdRope = kRows * 128;
__device__ __forceinline__ int third_at(int row, int c)
{
    const int at = tile_offset(row, c, kRows);
    return c < kDv ? at + c / 128 * (kChunk - kRows * 128) : at - 4 * kRows * 128 + kThirdRope;
}
__device__ __forceinline__ uint32_t third_offset(const Run& r)
{
    return (uint32_t)((r.j0 + 1) & 1) * (4 * kChunk);
}

// Warp 2: the run's tile's requests into shared memory.
__device__ __forceinline__ void tile_role(const PrefixArgs& a, PrefixShared& ms, const Run& r,
                                          int lane)
{
    int b0 = 0, b1 = -1, before = 0;
    if (r.nb > r.shared) tile_requests(a, r.tile, b0, b1);
    for (int k0 = 0; b0 + k0 <= b1; k0 += 32) {   // at most 64: a request has a row or more
        const int b = b0 + k0 + lane;
        int n = 0;
        if (b <= b1) {
            int first;
            n = (own_length(a, b, first) + kKeys - 1) / kKeys;
            ms.own_image[k0 + lane] = prefix_image_blocks(a) + own_block0(first, b);
        }
        int incl = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += v;
        }
        if (b <= b1) ms.own_before[k0 + lane] = before + incl - n;
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) ms.own_before[b1 - b0 + 1] = before;
    __syncwarp();
    if (lane == 0) mbar_arrive(&ms.own_full);
}

__device__ __forceinline__ void load_role(const PrefixArgs& a, uint8_t* smem, PrefixShared& ms,
                                          const Run& r, int lane)
{
    volatile int* abort_flag = &ms.abort;
    const int n = r.x1 - r.x0;
    Walk walk(r);
    bool looked = false;   // the tile's requests are known
    int64_t issued = 0, ropes = 0;   // latent chunks and RoPE chunks of this run
    const int32_t flags = third_flags(a, r, lane);   // (the first block goes to one stage either way)
    bool third = false;
    if (lane == 0) {
        mbar_arrive_expect_tx(&ms.q_full, (uint32_t)kPrefixImage);
        bulk_load(smem + kOffQ, a.q_image + r.tile * kPrefixImage, (uint32_t)kPrefixImage,
                  &ms.q_full);
    }
    bool ok = true;
    for (int j = 0; j < n && ok; ++j) {
        const int64_t jj = r.j0 + j;
        const int st = (int)(jj & 1);
        if (j == 1) third = any_third(flags);
        const int mem = stage_of(r, jj, third);
        const int64_t before = jj - (third ? 1 : 2);   // the block that was there
        if (!looked && walk.own(r)) {
            ok = looked = warp_wait(&ms.own_full, (uint32_t)r.run & 1, abort_flag, 0, a.wait_limit);
            if (!ok) break;
        }
        const uint8_t* src = a.k_image + walk.image(r, ms) * kPrefixImage;
        walk.next(r);
        for (int c = 0; c < 4 && ok; ++c) {
            if (before >= 0)
                ok = warp_wait(&ms.k_empty[before & 1][c], (uint32_t)(before >> 1) & 1, abort_flag,
                               0, a.wait_limit);
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&ms.k_full[st][c], kChunk);
                bulk_load(smem + mem * 4 * kChunk + c * kChunk, src + c * kChunk, kChunk,
                          &ms.k_full[st][c]);
            }
            ++issued;
        }
        if (!ok) break;
        if (jj >= 1)
            ok = warp_wait(&ms.r_empty, (uint32_t)(jj - 1) & 1, abort_flag, 0, a.wait_limit);
        if (!ok) break;
        if (lane == 0) {
            mbar_arrive_expect_tx(&ms.r_full, kRopeBytes);
            bulk_load(smem + kOffRope, src + 4 * kChunk, kRopeBytes, &ms.r_full);
        }
        ++ropes;
    }
    // Never go on with copies in flight: the last two blocks' chunks, the RoPE
    // chunk and the query tile must land.  A fresh flag and the full bound keep
    // this going after an abort; otherwise they have landed long ago or soon will.
    volatile int drain = 0;
    for (int64_t i = issued > 8 ? issued - 8 : 0; i < issued; ++i) {
        const int64_t jj = r.j0 + (i >> 2);
        warp_wait(&ms.k_full[jj & 1][i & 3], (uint32_t)(jj >> 1) & 1, &drain);
    }
    if (ropes > 0) warp_wait(&ms.r_full, (uint32_t)(r.j0 + ropes - 1) & 1, &drain);
    warp_wait(&ms.q_full, (uint32_t)r.run & 1, &drain);
}

// After an abort, MMAs already issued may still be running: wait for them (with the
// full bound) before the CTA releases TMEM and its stages.  The MMA warp.
__device__ __forceinline__ void drain_after_abort(PrefixShared& ms)
{
    if (__shfl_sync(0xffffffffu, *static_cast<volatile int*>(&ms.abort) != 0 ? 1 : 0, 0) != 0) {
        umma_commit_warp(&ms.mma_drain);
        volatile int drain = 0;
        warp_wait(&ms.mma_drain, 0, &drain);
    }
    __syncwarp();
}

__device__ __forceinline__ void mma_role(const PrefixArgs& a, uint32_t smem_base, uint32_t tmem,
                                         PrefixShared& ms, const Run& r)
{
    volatile int* abort_flag = &ms.abort;
    const int n = r.x1 - r.x0;
    constexpr uint32_t id_qk = idesc_e4m3(128, 2 * kRows, false, false);
    constexpr uint32_t id_hi = idesc_e4m3(128, kRows, true, true);
    constexpr uint32_t id_lo = idesc_e4m3(128, kRows, true, true, true);
    const uint64_t k_lat = smem_desc(smem_base, 16, 1024, kSw128);
    const uint64_t k_rope = smem_desc(smem_base + kOffRope, 16, 512, kSw64);
    const uint64_t q_lat = smem_desc(smem_base + kOffQ, 16, 1024, kSw128);
    const uint64_t q_rope = smem_desc(smem_base + kOffQ + 4 * kChunk, 16, 512, kSw64);
    const uint64_t v_lat = smem_desc(smem_base, kChunk, 1024, kSw128);
    const uint64_t p_hi = smem_desc(smem_base + kOffP, 128, 2048, kSwNone);
    const uint64_t p_lo = smem_desc(smem_base + kOffP + kPTerm, 128, 2048, kSwNone);
    auto ready = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __shfl_sync(0xffffffffu, mbar_try_wait(bar, parity) ? 1 : 0, 0) != 0;
    };
    // the third terms: a second pass of QK, into the low terms' columns
    constexpr uint32_t id_q3 = idesc_e4m3(128, kRows, false, false, true);
    const bool third = any_third(third_flags(a, r, threadIdx.x & 31));
    bool ok = warp_wait(&ms.q_full, (uint32_t)r.run & 1, abort_flag, 0, a.wait_limit);
    if (third && ok) ok = warp_wait(&ms.q3_full, (uint32_t)r.run & 1, abort_flag, 0, a.wait_limit);
    int next_qk = 0, next_pv = 0;
    long long t_last = clock64();
    for (uint32_t idle = 0; ok && next_pv < n;) {
        bool did = false;
        const int64_t jp = r.j0 + next_pv, jq = r.j0 + next_qk;
        if (next_pv < next_qk && ready(&ms.p_full, (uint32_t)jp & 1)) {
            tc_fence_after();
            const int st = (int)(jp & 1);
            const uint64_t v0 = v_lat + (uint64_t)((stage_of(r, jp, third) * 4 * kChunk) >> 4);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint64_t v = v0 + (uint64_t)((c * kChunk + kk * 4096) >> 4);
                    const uint64_t off = (uint64_t)((kk * 512) >> 4);
                    const uint32_t d = tmem + kColO + c * kRows;
                    umma_f8_warp(d, v, p_hi + off, id_hi, (next_pv > 0 || kk > 0) ? 1u : 0u);
                    umma_f8_warp(d, v, p_lo + off, id_lo, 1u);
                }
                umma_commit_warp(&ms.k_empty[st][c]);
            }
            umma_commit_warp(&ms.pv_done);
            ++next_pv;
            did = true;
        }
        if (next_qk < n) {
            const int st = (int)(jq & 1);
            const uint32_t ph = (uint32_t)(jq >> 1) & 1;
            if (ready(&ms.k_full[st][0], ph) &&
                (jq < 2 || ready(&ms.s_free[st], (uint32_t)((jq - 2) >> 1) & 1))) {
                tc_fence_after();
                const uint64_t k0 = k_lat + (uint64_t)((stage_of(r, jq, third) * 4 * kChunk) >> 4);
                uint64_t q0 = q_lat, q1 = q_rope;
                uint32_t id = id_qk, d = tmem + kColS + st * 2 * kRows;
#pragma unroll 1
                for (int pass = 0;; ++pass) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (c > 0 && ok)
                            ok = warp_wait(&ms.k_full[st][c], ph, abort_flag, 0, a.wait_limit);
                        if (ok) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                umma_f8_warp(d, k0 + (uint64_t)((c * kChunk + kk * 32) >> 4),
                                             q0 + (uint64_t)((c * kChunk + kk * 32) >> 4), id,
                                             (c > 0 || kk > 0) ? 1u : (uint32_t)pass);
                        }
                    }
                    if (ok) ok = warp_wait(&ms.r_full, (uint32_t)jq & 1, abort_flag, 0, a.wait_limit);
                    if (!ok) break;
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk)
                        umma_f8_warp(d, k_rope + (uint64_t)((kk * 32) >> 4),
                                     q1 + (uint64_t)((kk * 32) >> 4), id, 1u);
                    if (!third || pass > 0) break;
                    q0 = smem_desc(smem_base + third_offset(r), 16, 1024, kSw128);
                    q1 = smem_desc(smem_base + third_offset(r) + kThirdRope, 16, 512, kSw64);
                    id = id_q3;
                    d += kRows;
                }
                if (!ok) break;
                umma_commit_warp(&ms.s_full[st]);
                umma_commit_warp(&ms.r_empty);
                ++next_qk;
                did = true;
            }
        }
        if (did) {
            idle = 0;
            continue;
        }
        if ((++idle & 63u) == 0) {
            const long long now = clock64();
            if (__shfl_sync(0xffffffffu, *abort_flag, 0) != 0) break;
            if (idle == 64) t_last = now;   // first check of this idle stretch
            else if (__shfl_sync(0xffffffffu, now - t_last > a.wait_limit ? 1 : 0, 0) != 0) {
                *abort_flag = 1;
                break;
            }
        }
    }
    drain_after_abort(ms);
}

// Row `item`'s third terms into row `row` of the 64 at `tile`: what split_pair leaves
// of q_lo, in q_lo's units.  One warp.
__device__ __forceinline__ void third_terms(const PrefixArgs& a, int64_t item, int row, int lane,
                                            uint8_t* tile)
{
    uint4 v[kQueryVec];
    const Pow2 scale(q_shift(load_query(a, item, lane, v)));
#pragma unroll
    for (int i = 0; i < kQueryVec; ++i) {
        const int c = (lane + 32 * i) * 8;
        if (c >= kWidth) continue;
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint16_t t[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float x0 = scale(__uint_as_float(w[k] << 16));
            const float x1 = scale(__uint_as_float(w[k] & 0xFFFF0000u));
            uint16_t h, l;
            const float2 p = split_pair<kQLoBits>(x0, x1, h, l);
            t[k] = f32x2_to_e5m2x2((x0 - p.x) * (1 << kQLoBits), (x1 - p.y) * (1 << kQLoBits));
        }
        *reinterpret_cast<uint2*>(tile + third_at(row, c)) =
            make_uint2((uint32_t)t[0] | ((uint32_t)t[1] << 16), (uint32_t)t[2] | ((uint32_t)t[3] << 16));
    }
}

// Warps 2 and 3: the third terms of a tile that wants them, 32 rows each, zeros for
// the rows that do not (so a row's result does not depend on its tile's others); warp
// 2 looks up the tile's requests first.
__device__ __forceinline__ void third_role(const PrefixArgs& a, uint8_t* smem, PrefixShared& ms,
                                           const Run& r, int warp, int lane)
{
    const int row0 = (warp - kTileWarp) * 32;
    const int32_t flags = third_flags(a, r, lane);
    const uint32_t mine = __ballot_sync(0xffffffffu, __ldcg(a.q_window + r.tile * kRows + row0 + lane) < 0);
    if (warp == kTileWarp) tile_role(a, ms, r, lane);
    if (any_third(flags)) {
        uint8_t* tile = smem + third_offset(r);
#pragma unroll 1
        for (int k = 0; k < 32; ++k) {
            const int row = row0 + k;
            if ((mine >> k) & 1u) {
                third_terms(a, r.tile * kRows + row, row, lane, tile);
            } else {
                for (int c = lane * 16; c < kWidth; c += 512)
                    *reinterpret_cast<uint4*>(tile + third_at(row, c)) = make_uint4(0, 0, 0, 0);
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
    }
    if (lane == 0) mbar_arrive(&ms.q3_full);
}

__device__ __forceinline__ void softmax_role(const PrefixArgs& a, uint8_t* smem, uint32_t tmem,
                                             PrefixShared& ms, const Run& r, int warp, int lane)
{
    constexpr int R = kSetRows;
    volatile int* abort_flag = &ms.abort;
    const int set = (warp - kSoftmaxWarp0) / 4;
    const int quad = warp & 3;
    const uint32_t bar_id = 1u + (uint32_t)set;
    const int r0 = set * R;
    const int ti = quad * 32 + lane;                  // key within a block == TMEM lane
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    float* red = &ms.red[set * 4][0];
    float* redt = reinterpret_cast<float*>(smem + kOffP) + set * 128;   // epilogue: P is idle
    const int n = r.x1 - r.x0;

    // the rows' logit scales and windows (every set its own rows)
    if (ti < R) {
        ms.cq[r0 + ti] = __ldcg(a.q_scale + r.tile * kRows + r0 + ti);
        ms.win[r0 + ti] = __ldcg(a.q_window + r.tile * kRows + r0 + ti) & INT32_MAX;
    }
    softmax_bar(bar_id);
    int win_min = ms.win[r0 + lane];
    // rows without a reference yet, as bits (the same in every thread of the set);
    // a row that sees nothing never gets one
    uint32_t unset = __ballot_sync(0xffffffffu, win_min > 0);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        win_min = min(win_min, __shfl_xor_sync(0xffffffffu, win_min, off));

    // x = logit - m + kShift, nm = kShift - m (0 while the row has no reference)
    float nm[R], l[R], lt[R];
#pragma unroll
    for (int k = 0; k < R; ++k) nm[k] = l[k] = lt[k] = 0.f;
    bool alive = true;
    if (a.stall_probe) warp_wait(&ms.never, 0, abort_flag, 0, a.wait_limit);
    // the requests of the tile, for the blocks of their own keys
    const int P = prefix_length(a);
    const int per = a.q_len * a.num_heads;
    int row0 = 0;   // row of the tile's first request's first row, among the set's
    if (r.nb > r.shared) {
        int b0, b1;
        tile_requests(a, r.tile, b0, b1);
        row0 = (int)((int64_t)b0 * per - r.tile * kRows) - r0;
    }
    // one block ahead: its keys' flags, and where its first key is and whose
    Walk walk(r);
    bool looked = false;
    uint2 flags_next;   // valid and marked keys of this warp's 32
    int pos_next, k_next;   // k_next < 0: a prefix block
    auto look_ahead = [&]() {
        const bool own = walk.own(r);
        if (own && !looked)
            looked = warp_wait(&ms.own_full, (uint32_t)r.run & 1, abort_flag, 0, a.wait_limit);
        flags_next = make_uint2(0u, 0u);
        if (!own || looked) flags_next = __ldcg(a.k_flags + walk.image(r, ms) * 4 + quad);
        k_next = own ? walk.k : -1;
        pos_next = own ? P + (walk.y - (looked ? ms.own_before[walk.k] : 0)) * kKeys
                       : (walk.x - walk.y) * kKeys;
        walk.next(r);
    };
    look_ahead();
    for (int j = 0; j < n; ++j) {
        const int64_t jj = r.j0 + j;
        const int st = (int)(jj & 1);
        const uint32_t valid = flags_next.x, marked = flags_next.y;
        const int pos0 = pos_next, k_now = k_next;
        if (j + 1 < n) look_ahead();
        const bool ok = warp_wait(&ms.s_full[st], (uint32_t)(jj >> 1) & 1, abort_flag, 0,
                                  a.wait_limit);
        float x[R];
        if (ok) {
            tc_fence_after();
            const uint32_t sa = lanes + kColS + st * 2 * kRows + r0;
            uint32_t h0[16], l0[16], h1[16], l1[16];
            tmem_ld16(sa, h0);
            tmem_ld16(sa + kRows, l0);
            tmem_ld16(sa + 16, h1);
            tmem_ld16(sa + kRows + 16, l1);
            tmem_wait_ld();
            reg_fence(h0);
            reg_fence(l0);
            reg_fence(h1);
            reg_fence(l1);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                x[k] = fmaf(__uint_as_float(l0[k]), kQLoBack, __uint_as_float(h0[k]));
                x[16 + k] = fmaf(__uint_as_float(l1[k]), kQLoBack, __uint_as_float(h1[k]));
            }
        } else {
#pragma unroll
            for (int k = 0; k < R; ++k) x[k] = -CUDART_INF_F;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.s_free[st]);
#pragma unroll
        for (int g = 0; g < R / 4; ++g) {
            const float4 c = reinterpret_cast<const float4*>(ms.cq + r0)[g];
            x[4 * g] = fmaf(x[4 * g], c.x, nm[4 * g]);
            x[4 * g + 1] = fmaf(x[4 * g + 1], c.y, nm[4 * g + 1]);
            x[4 * g + 2] = fmaf(x[4 * g + 2], c.z, nm[4 * g + 2]);
            x[4 * g + 3] = fmaf(x[4 * g + 3], c.w, nm[4 * g + 3]);
        }
        // masked: keys past their list or with a bad slot, positions that a row does
        // not see, and own keys of another request than the row's.  `vis` has a bit
        // per row that sees this thread's key.  (The rolled loop keeps the code of
        // this rare path short: unrolled, it cost 2,500 cycles, most of them
        // fetching it.)
        uint32_t vis = 0xffffffffu;
        if (k_now >= 0 || valid != 0xffffffffu || marked != 0 || pos0 + kKeys > win_min) {
            const int pos = pos0 + ti;
            const float bump = (marked >> lane) & 1u ? CUDART_NAN_F : 0.f;   // a key with NaN codes
            vis = 0;
            if ((valid >> lane) & 1u) {
#pragma unroll 1
                for (int g = 0; g < R / 4; ++g) {
                    const int4 w = reinterpret_cast<const int4*>(ms.win + r0)[g];
                    vis |= ((pos < w.x ? 1u : 0u) | (pos < w.y ? 2u : 0u) |
                            (pos < w.z ? 4u : 0u) | (pos < w.w ? 8u : 0u)) << (4 * g);
                }
            }
            if (k_now >= 0) {   // only the rows of the key's request
                const int first = row0 + k_now * per;
                const int lo = max(first, 0), hi = min(first + per, R);
                vis &= hi <= lo ? 0u : (0xffffffffu >> (32 - (hi - lo))) << lo;
            }
#pragma unroll
            for (int k = 0; k < R; ++k) x[k] = (vis >> k) & 1u ? x[k] + bump : -CUDART_INF_F;
        }
        float top = x[0];
#pragma unroll
        for (int k = 1; k < R; ++k) top = fmaxf(top, x[k]);
        const bool need = top > kTop || (unset & vis) != 0 || !ok;
        if (softmax_bar_or(bar_id, need)) {
            // block maxima per row, then one lane per row of the set's first warp
            // decides on the row's new reference
            {
                float v[R];
#pragma unroll
                for (int k = 0; k < R; ++k) v[k] = x[k];
                red[quad * 32 + lane] = warp_transpose_reduce<R, true>(v, lane);
            }
            softmax_bar(bar_id);
            if (quad == 0) {
                const float bm = fmaxf(fmaxf(red[lane], red[32 + lane]),
                                       fmaxf(red[64 + lane], red[96 + lane]));
                const bool first = (unset >> lane) & 1u;
                const bool move = bm > (first ? -CUDART_INF_F : kTop);
                const float delta = move ? (kShift - kHeadroom) - bm : 0.f;
                ms.delta[r0 + lane] = delta;
                ms.scale[r0 + lane] = move && !first ? ex2_approx(delta) : 1.f;
                const uint32_t set_now = __ballot_sync(0xffffffffu, move && first);
                const uint32_t shrunk = __ballot_sync(0xffffffffu, move && !first);
                if (lane == 0) {
                    ms.set_now[set] = set_now;
                    ms.shrunk[set] = shrunk;
                    ms.stop[set] = *abort_flag;   // a warp that gave up: all of the set stop
                }
            }
            softmax_bar(bar_id);
            if (ms.stop[set] != 0) {
                alive = false;
                break;
            }
            unset &= ~ms.set_now[set];
            uint32_t moved = ms.shrunk[set];
#pragma unroll
            for (int g = 0; g < R / 4; ++g) {
                const float4 d = reinterpret_cast<const float4*>(ms.delta + r0)[g];
                nm[4 * g] += d.x;
                nm[4 * g + 1] += d.y;
                nm[4 * g + 2] += d.z;
                nm[4 * g + 3] += d.w;
                x[4 * g] += d.x;
                x[4 * g + 1] += d.y;
                x[4 * g + 2] += d.z;
                x[4 * g + 3] += d.w;
            }
            if (moved != 0) {   // sums and O so far shrink with the reference's step
#pragma unroll
                for (int g = 0; g < R / 4; ++g) {
                    const float4 f = reinterpret_cast<const float4*>(ms.scale + r0)[g];
                    l[4 * g] *= f.x;
                    l[4 * g + 1] *= f.y;
                    l[4 * g + 2] *= f.z;
                    l[4 * g + 3] *= f.w;
                    lt[4 * g] *= f.x;
                    lt[4 * g + 1] *= f.y;
                    lt[4 * g + 2] *= f.z;
                    lt[4 * g + 3] *= f.w;
                }
            }
            if (moved != 0 &&
                warp_wait(&ms.pv_done, (uint32_t)(jj - 1) & 1, abort_flag, 0, a.wait_limit)) {
                // O^T holds the blocks before: scale the moved rows' columns
                tc_fence_after();
#pragma unroll 1
                while (moved != 0) {
                    const int row = __ffs(moved) - 1;
                    moved &= moved - 1;
                    const float f = ms.scale[r0 + row];
                    uint32_t o[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[c] = tmem_ld1(lanes + kColO + c * kRows + r0 + row);
                    tmem_wait_ld();
                    reg_fence(o);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        tmem_st1(lanes + kColO + c * kRows + r0 + row,
                                 __float_as_uint(__uint_as_float(o[c]) * f));
                }
                tmem_wait_st();
            }
        }
        // P^T is stored as 16-row columns of 128 keys x 16 bytes, e4m3 terms
        // then e5m2 terms
        uint32_t hw[R / 4], lw[R / 4];
#pragma unroll
        for (int k = 0; k < R; k += 4) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                x[k + u] = ex2_approx(x[k + u]);
                l[k + u] += x[k + u];
            }
            uint16_t h0, l0, h1, l1;
            const float2 t0 = split_p(x[k], x[k + 1], h0, l0);
            const float2 t1 = split_p(x[k + 2], x[k + 3], h1, l1);
            lt[k] += t0.x;
            lt[k + 1] += t0.y;
            lt[k + 2] += t1.x;
            lt[k + 3] += t1.y;
            hw[k / 4] = (uint32_t)h0 | ((uint32_t)h1 << 16);
            lw[k / 4] = (uint32_t)l0 | ((uint32_t)l1 << 16);
        }
        // the buffer is free when the P.V of the block before has finished
        if (jj >= 1)
            warp_wait(&ms.pv_done, (uint32_t)(jj - 1) & 1, abort_flag, 0, a.wait_limit);
        uint8_t* prow = smem + kOffP + ti * 16 + (r0 / 16) * 2048;
#pragma unroll
        for (int g = 0; g < R / 16; ++g) {
            *reinterpret_cast<uint4*>(prow + g * 2048) =
                make_uint4(hw[4 * g], hw[4 * g + 1], hw[4 * g + 2], hw[4 * g + 3]);
            *reinterpret_cast<uint4*>(prow + kPTerm + g * 2048) =
                make_uint4(lw[4 * g], lw[4 * g + 1], lw[4 * g + 2], lw[4 * g + 3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.p_full);
    }

    // ---- epilogue: sums over the keys, then the rows out of TMEM, normalised by
    // what the MMA consumed (lt), and the LSE from the exact p (l) -------------------------
    bool have;
    {
        const float sum = warp_transpose_reduce<R, false>(l, lane);
        const float fed = warp_transpose_reduce<R, false>(lt, lane);
        red[quad * 32 + lane] = sum;
        have = alive && warp_wait(&ms.pv_done, (uint32_t)(r.j0 + n - 1) & 1, abort_flag, 0,
                                  a.wait_limit);
        if (have) tc_fence_after();
        redt[quad * 32 + lane] = fed;
    }
    softmax_bar(bar_id);
    if (ti < R) {
        const float fed = (redt[ti] + redt[32 + ti]) + (redt[64 + ti] + redt[96 + ti]);
        ms.scale[r0 + ti] = have && fed != 0.f ? 1.f / fed : 0.f;   // NaN stays NaN
    }
    softmax_bar(bar_id);
    float* stage = reinterpret_cast<float*>(smem);   // fp32 [64][512]
    float scl[R];
#pragma unroll
    for (int g = 0; g < R / 4; ++g) {
        const float4 s = reinterpret_cast<const float4*>(ms.scale + r0)[g];
        scl[4 * g] = s.x;
        scl[4 * g + 1] = s.y;
        scl[4 * g + 2] = s.z;
        scl[4 * g + 3] = s.w;
    }
    // (without `have` the columns may hold anything: the rows are zero then.  The loop
    // is rolled for the instruction cache: unrolled, 44.4 us instead of 42.6 at 64
    // requests of 16 heads with 1000 + 1000 positions, 18.9 instead of 18.5 at 4 of 16.)
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        tmem_ld32(lanes + kColO + c * kRows + r0, o);
        tmem_wait_ld();
        reg_fence(o);
#pragma unroll
        for (int k = 0; k < R; ++k)
            stage[(r0 + k) * kDv + c * 128 + ti] = scl[k] != 0.f ? __uint_as_float(o[k]) * scl[k] : 0.f;
    }
    tc_fence_before();
    fence_proxy_async_smem();
    softmax_bar(bar_id);
    if (ti < R) {
        const int64_t item = r.tile * kRows + r0 + ti;
        if (item < a.rows) {
            const float sum = (red[ti] + red[32 + ti]) + (red[64 + ti] + red[96 + ti]);
            float m = 0.f;
#pragma unroll
            for (int k = 0; k < R; ++k)
                if (k == ti) m = nm[k];
            const int64_t at = r.slot * kRows + r0 + ti;
            a.lse_part[at] = sum != 0.f ? log2f(sum) - m : -CUDART_INF_F;
            bulk_store(a.o_part + at * kDv, stage + (r0 + ti) * kDv, kDv * 4);
            bulk_commit();
            bulk_wait_read();
        }
    }
}

__global__ void __launch_bounds__(kThreads, 1)
prefix_split_kernel(const PrefixArgs a)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    PrefixShared& ms = *reinterpret_cast<PrefixShared*>(smem + kOffMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // the next kernel (the requests' own keys) may be scheduled as SMs fall idle
    asm volatile("griddepcontrol.launch_dependents;");
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            for (int c = 0; c < 4; ++c) {
                mbar_init(&ms.k_full[i][c], 1);
                mbar_init(&ms.k_empty[i][c], 1);
            }
            mbar_init(&ms.s_full[i], 1);
            mbar_init(&ms.s_free[i], kSoftmaxWarps);
        }
        mbar_init(&ms.r_full, 1);
        mbar_init(&ms.r_empty, 1);
        mbar_init(&ms.q_full, 1);
        mbar_init(&ms.q3_full, 2);
        mbar_init(&ms.p_full, kSoftmaxWarps);
        mbar_init(&ms.pv_done, 1);
        mbar_init(&ms.mma_drain, 1);
        mbar_init(&ms.own_full, 1);
        mbar_init(&ms.never, 1);
        ms.abort = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&ms.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    // the images come from the kernel before
    asm volatile("griddepcontrol.wait;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ms.tmem_base;
    const uint32_t smem_base = smem_u32(smem);

    // this CTA's share: `left` blocks from block x of `tile` on
    const int64_t g = blockIdx.x;
    int64_t tile = 0, left = 0, tile_nb = -1;   // blocks of `tile`, -1: not read yet
    int x = 0;
    if (a.splits > 0) {
        tile = (int)blockIdx.x / a.splits;
        const int s = (int)blockIdx.x % a.splits;
        tile_nb = __ldcg(a.tile_start + tile + 1) - __ldcg(a.tile_start + tile);
        x = (int)part_begin((uint32_t)tile_nb, s, a.splits);
        left = (int)part_begin((uint32_t)tile_nb, s + 1, a.splits) - x;
    } else {
        const int64_t U = __ldcg(a.tile_start + a.tiles), G = min((int64_t)gridDim.x, U);
        if (g < G) {
            const int64_t u = g * U / G;
            left = (g + 1) * U / G - u;
            // the last tile that starts at or before u: 32 probes a step
            int64_t n = a.tiles;
            while (n > 1) {
                const int64_t step = (n + 31) / 32;
                const bool le = lane * step < n && __ldcg(a.tile_start + tile + lane * step) <= u;
                const int hit = 31 - __clz(__ballot_sync(0xffffffffu, le));
                tile += hit * step;
                n = min(step, n - hit * step);
            }
            x = (int)(u - __ldcg(a.tile_start + tile));
        }
    }
    const int shared = (prefix_length(a) + kKeys - 1) / kKeys;
    int64_t j0 = 0;
    int idx = 0;
    // the next run, past tiles without blocks; false at the end
    Run r;
    auto next_run = [&]() -> bool {
        while (left > 0) {
            const int64_t nb = tile_nb >= 0 ? tile_nb
                                            : __ldcg(a.tile_start + tile + 1) - __ldcg(a.tile_start + tile);
            tile_nb = -1;
            if (nb > x) {
                r.tile = tile;
                r.nb = (int)nb;
                r.x0 = x;
                r.x1 = (int)min(nb, x + left);
                r.shared = shared;
                r.slot = a.splits > 0 ? g : g + tile;
                r.j0 = j0;
                r.run = idx;
                left -= r.x1 - r.x0;
                j0 += r.x1 - r.x0;
                ++idx;
                ++tile;
                x = 0;
                return true;
            }
            ++tile;
            x = 0;
        }
        return false;
    };
    // Registers move from the first warpgroup to the softmax warpgroups; each
    // branch below holds all of its warpgroups' remaining code.  Every thread
    // meets at the barrier that ends a run.
    if (warp < kSoftmaxWarp0) {
        regs_lower<kRegsLow>();
        while (next_run()) {
            if (warp == kLoadWarp) load_role(a, smem, ms, r, lane);
            else if (warp == kMmaWarp) mma_role(a, smem_base, tmem, ms, r);
            else third_role(a, smem, ms, r, warp, lane);
            tc_fence_before();
            const bool stop = __syncthreads_or(ms.abort);
            tc_fence_after();
            if (stop) break;
        }
    } else {
        regs_raise<kRegsHigh>();
        while (next_run()) {
            softmax_role(a, smem, tmem, ms, r, warp, lane);
            tc_fence_before();
            const bool stop = __syncthreads_or(ms.abort);
            tc_fence_after();
            if (stop) break;
        }
    }
    if (tid == 0 && ms.abort) atomicOr(a.err, MLA_DEVERR_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ---- prefix_merge -----------------------------------------------------------------------------
//
// A CTA's warps are rows x G groups of partials x W column parts: a lane has 16 / W
// columns of every G-th partial (group g: g, g + G, ...), the groups' sums are
// added in increasing g.  Few rows have few warps, so as many take a row as leave
// one wave of CTAs (two an SM), each with up to 20 (10) partials' loads in flight;
// with many rows one warp does, two partials at a time.  (Measured: 512 rows of 19
// partials 5.0 us at W = 4 against 7.9 at 1; 1024 of 9 4.4 at 2 against 7.6 at 1;
// 8192 of 2 to 3 9.6 at 1 against 16.4 at 2.)  Few rows of many partials are a small
// batch on a long prefix: there four groups share them.
// The row's partials are those of the runs of its tile and, without joined
// tiles, the split kernel's: M = max lse, w = 2^(lse - M), o = sum w o_s / sum w,
// summed in increasing order, lse = M + log2 sum w.  A partial of weight 0 is
// not added.  The first partials are loaded before the weights are known.

constexpr int kMergeMax = 2 * MLA_MAX_SPLITS;   // partials of one tile or one request: 256 each
constexpr int64_t kMergeRows4 = 512, kMergeRows2 = 1024;   // rows up to which W is 4, 2
constexpr int kMergeManyParts = 20;   // partials above which four groups share a row's

template <int W, int G>
__global__ void __launch_bounds__(32 * (G > 1 ? W * G : 8))
prefix_merge_kernel(const PrefixArgs a)
{
    constexpr int kQuads = 4 / W;        // groups of four columns per lane
    constexpr int kAhead = W == 1 ? 2 : 5 * W;   // partials in flight per lane
    constexpr int kWarps = G > 1 ? W * G : 8;
    constexpr int kMergeRows = kWarps / (W * G);
    static_assert(kRows % kMergeRows == 0, "a CTA's rows are in one tile");
    static_assert(G == 1 || kMergeRows == 1, "the groups of a row are a CTA");
    __shared__ float weights[G > 1 ? 1 : kWarps][kMergeMax];
    __shared__ float4 group_sum[G > 1 ? G - 1 : 1][G > 1 ? W : 1][32];
    __shared__ float row_sum_s;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t item = (int64_t)blockIdx.x * kMergeRows + warp / (W * G);
    const int group = G > 1 ? warp / W : 0;
    const int col = warp % W * (128 * kQuads) + lane * 4;   // and every 128 columns on
    const int64_t tile = (int64_t)blockIdx.x * kMergeRows / kRows;
    if (item >= a.rows) return;   // whole warps, and no barrier follows
    float* w_s = weights[G > 1 ? 0 : warp];
    // the tile's runs: slots [s0, s0 + np); a run without blocks has left nothing
    int64_t s0 = 0;
    int np = 0;
    uint32_t nb = 0;
    if (a.ctas > 0) {
        const int64_t u0 = __ldcg(a.tile_start + tile), u1 = __ldcg(a.tile_start + tile + 1);
        nb = (uint32_t)(u1 - u0);
        if (a.splits > 0) {   // (the partials' loads need not wait for nb)
            s0 = tile * a.splits;
            np = a.splits;
        } else if (nb > 0) {
            const int64_t U = __ldcg(a.tile_start + a.tiles), ctas = min((int64_t)a.ctas, U);
            const int64_t g0 = cta_of(u0, U, ctas);
            s0 = g0 + tile;
            np = (int)(cta_of(u1 - 1, U, ctas) - g0) + 1;
        }
    }
    auto left_out = [&](int i) {   // equal parts of few blocks: some are empty
        return a.splits > 0 && part_begin(nb, i, a.splits) == part_begin(nb, i + 1, a.splits);
    };
    const int n = np + a.own_splits;
    const float* own = a.o_own + item * a.own_splits * kDv + col;
    const float* part = a.o_part + (s0 * kRows + item % kRows) * kDv + col;
    const float* lse_part = a.lse_part + s0 * kRows + item % kRows;
    struct Cols {
        float4 v[kQuads];   // columns col + 128 q .. + 3
    };
    auto load = [&](int i) {
        const float* row = i < np ? part + (int64_t)i * (kRows * kDv) : own + (int64_t)(i - np) * kDv;
        Cols c;
#pragma unroll
        for (int q = 0; q < kQuads; ++q) c.v[q] = __ldcg(reinterpret_cast<const float4*>(row + 128 * q));
        return c;
    };
    Cols ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (group + i * G < n) ahead[i] = load(group + i * G);
    // the weights: by every warp for itself, or by the CTA's first for all
    float m = -CUDART_INF_F, sum = 0.f;
    if (G == 1 || warp == 0) {
        for (int i = lane; i < n; i += 32) {
            float l = -CUDART_INF_F;
            if (i >= np) l = __ldcg(a.lse_own + item * a.own_splits + (i - np));
            else if (!left_out(i)) l = __ldcg(lse_part + i * kRows);
            w_s[i] = l;
            m = fmaxf(m, l);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        for (int i = lane; i < n; i += 32) {
            const float w = w_s[i] == -CUDART_INF_F ? 0.f : exp2f(w_s[i] - m);
            sum += w;
            w_s[i] = w * (i < np ? a.kv_scale : a.own_scale);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (lane == 0 && warp % W == 0 && a.lse != nullptr)
            a.lse[item] = sum != 0.f ? m + log2f(sum) : -CUDART_INF_F;
        if (G > 1 && lane == 0) row_sum_s = sum;
    }
    if constexpr (G > 1) {
        __syncthreads();
        sum = row_sum_s;
    } else {
        __syncwarp();
    }
    Cols acc;
#pragma unroll
    for (int q = 0; q < kQuads; ++q) acc.v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float w, const Cols& c) {
        if (w != 0.f) {
#pragma unroll
            for (int q = 0; q < kQuads; ++q) {
                acc.v[q].x += w * c.v[q].x;
                acc.v[q].y += w * c.v[q].y;
                acc.v[q].z += w * c.v[q].z;
                acc.v[q].w += w * c.v[q].w;
            }
        }
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (group + i * G < n) add(w_s[group + i * G], ahead[i]);
    for (int i0 = group + kAhead * G; i0 < n; i0 += kAhead * G) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i0 + i * G < n) ahead[i] = load(i0 + i * G);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i0 + i * G < n) add(w_s[i0 + i * G], ahead[i]);
    }
    if constexpr (G > 1) {
        static_assert(G == 1 || kQuads == 1, "one float4 per lane and group");
        if (group > 0) group_sum[group - 1][warp % W][lane] = acc.v[0];
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int g = 0; g < G - 1; ++g) {
            const float4 x = group_sum[g][warp % W][lane];
            acc.v[0].x += x.x;
            acc.v[0].y += x.y;
            acc.v[0].z += x.z;
            acc.v[0].w += x.w;
        }
    }
    const float f = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int q = 0; q < kQuads; ++q) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.v[q].x * f, acc.v[q].y * f);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.v[q].z * f, acc.v[q].w * f);
        *reinterpret_cast<uint2*>(a.o + item * kDv + col + 128 * q) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
}

}  // namespace

cudaError_t launch_prefix_split(const PrefixArgs& a, cudaStream_t stream)
{
    static DeviceOnce once;
    cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(prefix_split_kernel,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    });
    if (e != cudaSuccess) return e;
    const int64_t key_ctas = prefix_blocks(a.prefix_cap) * (kKeys / kPrepKeys);
    const int64_t own_ctas =
        a.joined ? prefix_own_blocks(a.total_keys, a.batch) * (kKeys / kPrepKeys) : 0;
    const int64_t query_ctas = (int64_t)a.tiles * (kRows / kPrepRows);
    e = launch_pdl(prefix_prepare_kernel, dim3((unsigned)(1 + own_ctas + query_ctas + key_ctas)),
                   kPrepThreads, 0, stream, a, (int)own_ctas, (int)query_ctas);
    if (e != cudaSuccess) return e;
    return launch_pdl(prefix_split_kernel, dim3((unsigned)a.ctas), kThreads, kSmemBytes, stream, a);
}

cudaError_t launch_prefix_merge(const PrefixArgs& a, cudaStream_t stream)
{
    auto launch = [&](auto* kernel, int rows, int threads) {
        return launch_pdl(kernel, dim3((unsigned)((a.rows + rows - 1) / rows)), threads, 0, stream, a);
    };
    const int parts = (a.splits > 0 ? a.splits : a.ctas / a.tiles) + a.own_splits;
    if (a.rows <= kMergeRows4 && parts > kMergeManyParts)
        return launch(prefix_merge_kernel<4, 4>, 1, 512);
    if (a.rows <= kMergeRows4) return launch(prefix_merge_kernel<4, 1>, 2, 256);
    if (a.rows <= kMergeRows2) return launch(prefix_merge_kernel<2, 1>, 4, 256);
    return launch(prefix_merge_kernel<1, 1>, 8, 256);
}

}  // namespace mla
