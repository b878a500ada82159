// What the kernels that move rows into and out of the 8-bit paged cache share: which 16 positions a warp owns.
#pragma once

#include "tq_elem.cuh"
#include "tq_fp8.cuh"

namespace tq {
namespace {

constexpr int kWarps = 8;
constexpr int kRows = 16;  // tokens a warp holds

// Where one warp works: 16 positions of a block.
struct Place {
    bool live;       // the unit has tokens there
    int blk;         // the block's id, not checked yet (-1: past the block table)
    int64_t row0;    // packed row of the warp's first token (may lie before the sequence's first)
    int64_t pos;     // its position
    int first;       // offset of the warp's 16 tokens in the block
    int lo, hi;      // offsets in the block of the new tokens: lo <= t < hi
    int head, side;
};

// The 16 tokens from `first` on of unit u's block: everything but the head and the side.
__device__ __forceinline__ Place place_of_unit(const Fp8Geometry& g, const Fp8Batch& b, uint32_t u, int first, int32_t* status) {
    Place p;
    p.first = first;
    p.head = p.side = 0;
    p.live = false;
    p.blk = -1;
    p.row0 = 0;
    p.pos = 0;
    p.lo = p.hi = 0;
    if (u >= fp8_units(b.num_tokens, b.batch, g.bs, 2)) return p;
    const Fp8Seq q = fp8_seq_of_unit(b, u, g.bs, 2);
    const int s = q.b, c0 = q.row0, n = q.n, start = q.start;
    const int64_t j = (int64_t)u - q.base;
    if (n <= 0 || j < 0) return p;
    if (start < 0) {
        if (j == 0 && (threadIdx.x & 31) == 0) flag(status, TQ_FLAG_BAD_SLOT);
        return p;
    }
    const int64_t blk_i = (start >> g.bs_shift) + j;  // the block of the sequence
    const int64_t pos0 = blk_i << g.bs_shift;
    if (pos0 >= (int64_t)start + n) return p;
    if (blk_i < b.max_blocks) p.blk = __ldg(b.block_table + (int64_t)s * b.max_blocks + blk_i);
    p.live = true;
    p.row0 = (int64_t)c0 + (pos0 - start) + p.first;
    p.pos = pos0 + p.first;
    p.lo = start > pos0 ? (int)(start - pos0) : 0;
    p.hi = (int)min((int64_t)g.bs, (int64_t)start + n - pos0);
    return p;
}
// Work item `w` (16 tokens) of the launch; 2^wpb_shift warps per block of tokens.
__device__ __forceinline__ Place find_place(const Fp8Geometry& g, const Fp8Batch& b, int64_t w, int wpb_shift,
                                            int32_t* status) {
    const int64_t item = w >> wpb_shift;
    const uint32_t uh = (uint32_t)(item >> 1);  // the host keeps the grid, and so this, below 2^31
    const uint32_t u = uh / (uint32_t)g.hkv;
    Place p = place_of_unit(g, b, u, (int)(w & ((1 << wpb_shift) - 1)) * kRows, status);
    p.side = (int)(item & 1);
    p.head = (int)(uh - u * (uint32_t)g.hkv);
    return p;
}
// Whether the place's block lies in the pool (else it is flagged); its page is (blk * hkv + head) * 2 + side.
__device__ __forceinline__ bool page_of(const Fp8Geometry& g, const Place& p, int32_t* status, int64_t& page) {
    if (p.blk < 0 || p.blk >= g.num_blocks) {
        if (p.live && (threadIdx.x & 31) == 0) flag(status, TQ_FLAG_BAD_SLOT);
        return false;
    }
    page = ((int64_t)p.blk * g.hkv + p.head) * 2 + p.side;
    return true;
}

// Four codes times 2^d, d <= 0; exact but for those that become subnormal.
__device__ __forceinline__ uint32_t scale_codes(uint32_t v, int d) {
    if (d == 0) return v;
    const float m = fp8_pow2(max(d, -100));
    const float2 x = fp8_to_float2(v & 0xFFFFu), y = fp8_to_float2(v >> 16);
    return fp8_cvt2(x.x * m, x.y * m) | (fp8_cvt2(y.x * m, y.y * m) << 16);
}
// The same for `rows` rows of codes, by a warp.
__device__ __forceinline__ void move_codes(uint8_t* codes, int rows, int d) {
    for (int r = 0; r < rows; ++r) {
        uint32_t* c = reinterpret_cast<uint32_t*>(codes + (int64_t)r * kHeadDim) + (threadIdx.x & 31);
        *c = scale_codes(*c, d);
    }
}

// CTAs of a launch over all 16-token pieces of a batch's blocks, heads and sides.
inline int64_t fp8_row_grid(const Fp8Geometry& g, const Fp8Batch& b) {
    const int64_t warps = (fp8_units(b.num_tokens, b.batch, g.bs, 2) * g.hkv * 2) << (g.bs_shift - 4);
    return (warps + kWarps - 1) / kWarps;
}

}  // namespace
}  // namespace tq
