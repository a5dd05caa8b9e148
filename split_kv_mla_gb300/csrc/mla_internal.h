// mla_internal.h -- host-side declarations shared by the libmla translation units.
#pragma once
#include <atomic>
#include <cstdint>
#include <mutex>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/mla_decode.h"

namespace mla {

// Runs a set-up step (a kernel attribute, a symbol lookup: state the runtime
// keeps per device) once for each device that is current when run() is called.
// Thread-safe; a step that fails is tried again on the next call.
class DeviceOnce {
public:
    template <class F>
    cudaError_t run(F&& step)
    {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
        if (done_[dev].load(std::memory_order_acquire)) return cudaSuccess;
        std::lock_guard<std::mutex> lock(mu_);
        if (done_[dev].load(std::memory_order_relaxed)) return cudaSuccess;
        e = step();
        if (e == cudaSuccess) done_[dev].store(true, std::memory_order_release);
        return e;
    }

private:
    static constexpr int kMaxDevices = 64;
    std::atomic<bool> done_[kMaxDevices]{};
    std::mutex mu_;
};

// Parameters of one split-kernel launch (dense or sparse).
// Largest batch for which the split kernel orders requests longest first.
constexpr int kLongFirstMaxBatch = 256;

struct SplitArgs {
    const uint16_t* q_lat;      // bf16 [rows, H, d_v]  (dense q_lat / sparse q_nope)
    const uint16_t* q_pe;       // bf16 [rows, H, d_rope]
    const uint8_t* pool;        // e4m3fn [pool_rows, d_v + d_rope]
    int64_t pool_rows;
    const int32_t* seq_lens;    // dense: [batch]; sparse: NULL (every token has topk entries)
    const int32_t* kv_indices;  // dense: flat slot list; sparse: [tokens, topk]
    const int32_t* kv_indptr;   // dense: [batch+1]; sparse: NULL (token t starts at t*topk)
    int32_t topk;               // sparse only
    int32_t batch;              // requests (dense) or tokens (sparse)
    int32_t q_len;              // 1 for sparse
    int32_t num_heads;
    int32_t d_v, d_rope;
    int32_t num_splits, rows_per_cta, head_blocks;
    float logit_scale;          // scale * kv_scale * log2(e): raw fp8 dot -> base-2 logit
    float out_scale;            // kv_scale: raw fp8 V units -> output units
    uint16_t* o;                // bf16 [rows, H, d_v]   (written when num_splits == 1)
    float* o_f32;               // fp32 [rows, H, d_v] instead of o, or NULL
    float* lse;                 // fp32 [rows, H] or NULL
    float* o_part;              // fp32 [rows*H, ns, d_v] (num_splits > 1)
    float* lse_part;            // fp32 [rows*H, ns]
    uint32_t* err;              // workspace error word
    int sparse;
    // sparse only: a second (compressed) cache, extra_indices [tokens, extra_topk]
    // into extra_pool [extra_rows, d_v + d_rope]; extra_topk 0 without one
    const uint8_t* extra_pool = nullptr;
    int64_t extra_rows = 0;
    const int32_t* extra_indices = nullptr;
    int32_t extra_topk = 0;
    // dense only: grid slice z takes the z-th longest request (batch at most
    // kLongFirstMaxBatch)
    int32_t long_first = 0;
    // decode context parallelism (dense only): local key i is global position
    // i * cp_world + cp_rank; glen [batch] global lengths, or NULL to use seq_lens
    const int32_t* glen = nullptr;
    int32_t cp_rank = 0;
    int32_t cp_world = 1;
    // fused merge (plan.merge_cluster > 1): per (request x head block, cluster
    // rank) arrival tickets in the workspace header, zero between calls
    uint32_t* tickets = nullptr;
    // phase time stamps (builds with MLA_TRACE only): kTraceSlots per CTA
    unsigned long long* trace = nullptr;
    // cycle bound of the pipeline's waits (mla_debug_wait_limit; the waits that
    // drain copies and MMAs before the CTA exits keep the full bound)
    long long wait_limit = 2000000000ll;
    // tests of the timeout path: the softmax warps first wait on a barrier that
    // nothing completes, so that wait runs out while copies are in flight
    int32_t stall_probe = 0;
};

// The pipeline wait bound that launches use (mla_debug_wait_limit sets it),
// and whether that call armed the unsatisfiable wait of the timeout tests.
long long pipeline_wait_limit();
bool stall_probe_armed();

// Phase stamps of a traced build (compiled with -DMLA_TRACE): per CTA of the
// split kernel, globaltimer nanoseconds at kTraceSlots points, for at most
// kTraceCtas CTAs (linear CTA index x + grid_x (y + grid_y z)).
constexpr int kTraceSlots = 12;
constexpr int kTraceCtas = 8192;
// ... followed by per-block events of the first kTraceBlockCtas CTAs.
constexpr int kTraceBlockCtas = 4;
constexpr int kTraceBlocks = 64;
constexpr int kTraceBlockEvents = 8;
constexpr int kTraceWords =
    kTraceCtas * kTraceSlots + kTraceBlockCtas * kTraceBlocks * kTraceBlockEvents;

// Merge-ticket counters in the workspace header: after the 256-byte error-word
// area, one uint32 per (tile, cluster rank) of a fused-merge launch.
constexpr int64_t kErrorAreaBytes = 256;
constexpr int64_t kMaxTickets = (MLA_WORKSPACE_HEADER_BYTES - kErrorAreaBytes) / 4;
// Largest number of (row, cluster) partials one CTA of the last cluster merges
// from the workspace in a fused merge (its slice rows x the tile's clusters).
constexpr int kMaxMergeTerms = 32;

// Kernel variants (mla_plan_t::variant).  Value 1 belonged to a CUDA-core
// bring-up kernel that the tcgen05 kernel replaced; it is rejected.
enum Variant : int32_t {
    kVariantTc = 2,   // tcgen05 + TMA split kernel, then the split-K reduce kernel
};

// The split kernel; mc > 1 fuses the split-K merge (clusters of mc splits).
cudaError_t launch_split_tc(const SplitArgs& a, const mla_plan_t& plan, int mc,
                            cudaStream_t stream);

// Workspace bytes that a plan needs, recomputed from its shape and split count.
int64_t needed_workspace(const mla_plan_t* plan);

// 2-D uint8 tensor map of the pool (row_bytes columns x rows) with one-row
// boxes of `box` columns (the shape tile::gather4 reads); false on failure.
bool make_row_map(CUtensorMap* m, const void* pool, int64_t rows, int row_bytes, int box,
                  CUtensorMapSwizzle sw);

// Merge of decode-context-parallel ranks' bf16 shares (mla_dcp_lse_merge_ranks).
cudaError_t launch_dcp_merge(const void* parts, bool parts_f32, const float* lse_in,
                             int32_t world, int64_t rows, int32_t d_v, uint16_t* o, float* lse,
                             cudaStream_t stream);

// ---- shared-prefix decode (mla_prefix.cu) -----------------------------------------------
constexpr int kPrefixRows = 64;       // query rows of a tile
constexpr int kPrefixKeys = 128;      // keys of a block
constexpr int64_t kPrefixImage = 73728;   // bytes of a block's (a query tile's) operand image

// Parameters of one shared-prefix call's kernels.
struct PrefixArgs {
    const uint16_t* q_lat;       // bf16 [batch * q_len, H, 512]
    const uint16_t* q_pe;        // bf16 [batch * q_len, H, 64]
    const uint8_t* pool;         // e4m3fn [pool_rows, 576]
    int64_t pool_rows;
    const int32_t* prefix_indices;
    const int32_t* prefix_len;   // device length, or NULL: prefix_cap
    int32_t prefix_cap;          // entries of prefix_indices
    const int32_t* seq_lens;     // the requests' own keys
    const int32_t* kv_indices;
    const int32_t* kv_indptr;
    int32_t total_keys;          // entries of kv_indices that joined tiles may read
    int32_t batch, q_len, num_heads;
    int64_t rows;                // batch * q_len * num_heads
    int32_t tiles;               // ceil(rows / kPrefixRows)
    int32_t ctas;                // CTAs of the prefix kernel
    int32_t splits;              // CTAs per tile, or 0: equal runs of the tiles' sequence
    int32_t joined;              // a tile's blocks are the prefix's and its requests' own
    float logit_scale;           // scale * kv_scale * log2(e)
    float kv_scale;
    // workspace
    uint32_t* err;
    uint8_t* k_image;            // [prefix blocks, then own blocks][kPrefixImage]
    uint2* k_flags;              // [blocks][4]: bits of 32 valid keys, of keys with NaN codes
    uint8_t* q_image;            // [tiles][kPrefixImage]: e4m3 terms of the queries
    float* q_scale;              // [tiles * 64] raw dot -> base-2 logit
    int32_t* q_window;           // [tiles * 64] positions the row sees; sign bit: the row
                                 // wants its query's third term
    int64_t* tile_start;         // [tiles + 1] blocks before the tile
    float* o_part;               // [slots][64][512], normalised
    float* lse_part;             // [slots][64]
    // without joined tiles: the requests' own keys as partial rows of the split kernel
    const float* o_own;          // [rows, own_splits, 512]
    const float* lse_own;        // [rows, own_splits]
    int32_t own_splits;          // 0: none
    float own_scale;             // o_own's units -> output units
    uint16_t* o;                 // bf16 [rows, 512]
    float* lse;                  // fp32 [rows] or NULL
    long long wait_limit;
    int32_t stall_probe;
};

// Blocks of the prefix, and room for the requests' own: request b's start at
// block kv_indptr[b] / 128 + b.
inline int64_t prefix_blocks(int64_t cap) { return (cap + kPrefixKeys - 1) / kPrefixKeys; }
inline int64_t prefix_own_blocks(int64_t total_keys, int64_t batch)
{
    return total_keys / kPrefixKeys + batch;
}

// The operand images of the prefix and the queries, and the prefix's partials.
cudaError_t launch_prefix_split(const PrefixArgs& a, cudaStream_t stream);
// Merge of the prefix's and the requests' own partials into o and lse.
cudaError_t launch_prefix_merge(const PrefixArgs& a, cudaStream_t stream);

// MLA_OK when the current device is one the library runs on, else a status.
int device_ok();

// Gather probe (mla_debug_gather).
cudaError_t launch_gather_probe(const void* pool, int64_t pool_rows, int32_t row_bytes,
                                const int32_t* indices, int64_t n, uint8_t* out, uint32_t* err,
                                cudaStream_t stream);
// Split-K reduce; writes o as bf16, or as fp32 when out_f32.
cudaError_t launch_splitk_reduce(const float* o_part, const float* lse_part, int64_t rows,
                                 int32_t num_splits, int32_t d_v, float out_scale, void* o,
                                 bool out_f32, float* lse, cudaStream_t stream);

}  // namespace mla
