// mla_spans.h -- the whole-number arithmetic of cache extension: which entries of the new
// table a warp copies, which of a request's are kept, and which take its tokens.  Tables,
// lengths and counts go up to 2^31 - 1, so what is added to them is held in 32 bits without
// a sign, where neither two of them nor one and a span overflow.  For host code too.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define MLA_HD __host__ __device__ __forceinline__
#else
#define MLA_HD inline
#endif

namespace mla {

// Entries [begin, end) of a table of `total` that warp number `warp` of `warps` takes, in
// whole spans where it takes more than one.  begin is below 2^32 for 2^19 warps of spans of
// up to 2^12; nothing of the table where begin >= end.
struct Run {
    uint32_t begin, end;
};

MLA_HD Run warp_run(uint32_t total, uint32_t warp, uint32_t warps, uint32_t span)
{
    uint32_t run = (total + warps - 1) / warps;
    run = run > span ? (run + span - 1) / span * span : (run + 31) / 32 * 32;
    const uint32_t begin = warp * run;
    return Run{begin, begin >= total || total - begin < run ? total : begin + run};
}

// The end of the span at i0 < end.
MLA_HD uint32_t span_end(uint32_t i0, uint32_t end, uint32_t span)
{
    return end - i0 > span ? i0 + span : end;
}

// The end of what a request keeps, whose entries are [start, next) and of which the first
// `length` are kept, or as many as have room.
MLA_HD uint32_t kept_end(uint32_t start, uint32_t next, uint32_t length)
{
    return length < next - start ? start + length : next;
}

// The place in its request of the n-th token behind `length` kept entries, and whether the
// request's entries [start, next) of the table have it.
MLA_HD uint32_t token_place(uint32_t length, uint32_t n) { return length + n; }

MLA_HD bool has_place(uint32_t start, uint32_t next, uint32_t place)
{
    return place < next - start;
}

// Between lo and hi: lo itself where hi is the next.  (Of a fork's children too.)
MLA_HD int32_t middle(int32_t lo, int32_t hi)
{
    return (int32_t)(((uint32_t)lo + (uint32_t)hi) >> 1);
}

}  // namespace mla
