// Keeping the accepted path of a tree of drafts in the 8-bit paged cache: the
// codes of positions start + kept[r] move to positions start + r, whose blocks may
// have other scales.
//
// A block that receives codes takes the largest exponent of the blocks they come
// from and, where it holds earlier positions of the sequence, of its own; codes move by
// c -> c 2^(e_from - e), which is exact but for those that become subnormal.
//
// With r <= kept[r], nothing that is written lies in front of what is still to be read, if
// the rows go in order.  So one CTA takes a (sequence, head, side) and goes through the
// places 128 at a time, which is a whole number of blocks: every row of the 128 is in
// registers, and every exponent known, before any of them is written.  A warp has 16
// places; a lane looks one of them up, so that the chain of loads (kept row, block id,
// scale, codes) is paid once for all of them.  Earlier positions of the first block are
// rows that come from where they are.
//
// What bounds it is that chain of loads and how many CTAs there are: 64 sequences x 8 heads
// with a few kept nodes 5.3 us; 32 sequences x 20 heads with up to 700 kept, in blocks of 64, 22 us
// (35 MB read, 0.4 of the copy's rate); a CTA going through the same rows 16 at a time took 370,
// the next step's ids and kept rows read ahead 26 (more registers, fewer CTAs an SM), one barrier a
// step 24 (a CTA's warps drift apart).
#include <cuda_runtime.h>

#include <climits>

#include "tq_fp8_rows.cuh"

namespace tq {
namespace {

constexpr int kPlaces = kWarps * kRows;  // of a CTA's step

__global__ void __launch_bounds__(kWarps * 32) fp8_keep_kernel(const Fp8KeepArgs a) {
    const Fp8Geometry& g = a.g;
    __shared__ int tops[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t hs = blockIdx.x >> 1;
    const int side = (int)(blockIdx.x & 1), b = (int)(hs / g.hkv), h = (int)(hs - (int64_t)b * g.hkv);
    const int c0 = fp8_clamp_cu(a.b.cu, b, a.b.num_tokens), n = fp8_clamp_cu(a.b.cu, b + 1, a.b.num_tokens) - c0;
    const int start = __ldg(a.b.start + b);
    if (n <= 0) return;
    if (start < 0) {
        if (threadIdx.x == 0) flag(a.status, TQ_FLAG_BAD_SLOT);
        return;
    }
    const int32_t* table = a.b.block_table + (int64_t)b * a.b.max_blocks;
    // the page that holds a position of the sequence, or -1
    auto page_of_pos = [&](int64_t p) -> int64_t {
        const int64_t j = p >> g.bs_shift;
        const int id = j < a.b.max_blocks ? __ldg(table + j) : -1;
        return id >= 0 && id < g.num_blocks ? ((int64_t)id * g.hkv + h) * 2 + side : -1;
    };
    const int64_t first = (int64_t)start >> g.bs_shift << g.bs_shift;  // the first block's first position
    const int64_t end = (int64_t)start + n;
    const int group = warp >> (g.bs_shift - 4) << (g.bs_shift - 4);    // the first warp of this one's block
    for (int64_t p0 = first; p0 < end; p0 += kPlaces) {
        const int64_t mine = p0 + warp * kRows;                        // the warp's places, of one block
        // lane i (and i + 16) looks up place i: its codes' row in the pool (-1: it gets none), their exponent
        const int64_t p = mine + (lane & 15);
        int64_t from = -1;
        int e_from = INT_MIN;
        const int64_t page = mine < end ? page_of_pos(mine) : -1;
        const int e_own = page >= 0 ? fp8_exp_of(g.scales[page]) : 0;
        if (page >= 0 && p < end) {
            if (p < start) {
                from = (page << g.bs_shift) + (p & (g.bs - 1));
                e_from = e_own;
            } else {
                const int r = (int)(p - start), k = __ldg(a.kept + c0 + r);
                const int64_t s = (int64_t)start + k, of = k >= r ? page_of_pos(s) : -1;
                if (of >= 0) {
                    from = (of << g.bs_shift) + (s & (g.bs - 1));
                    e_from = fp8_exp_of(g.scales[of]);
                }
            }
        }
        if (p >= start && p < end && from < 0 && lane < 16) flag(a.status, TQ_FLAG_BAD_SLOT);
        // four rows at a time, 16 bytes a lane
        uint4 code[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = __shfl_sync(0xFFFFFFFFu, from, 4 * i + (lane >> 3));
            code[i] = make_uint4(0, 0, 0, 0);
            if (row >= 0) code[i] = *(reinterpret_cast<const uint4*>(g.pool + row * kHeadDim) + (lane & 7));
        }
        const int top = __reduce_max_sync(0xFFFFFFFFu, e_from);
        if (lane == 0) tops[warp] = top;
        __syncthreads();  // all rows are read, and all exponents
        int e = INT_MIN;
        for (int w = 0; w < g.bs >> 4; ++w) e = max(e, tops[group + w]);
        if (page >= 0 && e != INT_MIN) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = 4 * i + (lane >> 3);
                const int64_t row = __shfl_sync(0xFFFFFFFFu, from, at);
                const int d = __shfl_sync(0xFFFFFFFFu, e_from, at) - e;
                const int64_t to = (page << g.bs_shift) + (mine & (g.bs - 1)) + at;
                if (row >= 0 && (row != to || d != 0))
                    *(reinterpret_cast<uint4*>(g.pool + to * kHeadDim) + (lane & 7)) =
                        make_uint4(scale_codes(code[i].x, d), scale_codes(code[i].y, d), scale_codes(code[i].z, d), scale_codes(code[i].w, d));
            }
            if (warp == group && lane == 0 && e != e_own) g.scales[page] = fp8_pow2(e);
        }
        __syncthreads();  // (the next step reads what this one has not written, and tops again)
    }
}

}  // namespace

bool fp8_keep_counts(const Fp8Geometry& g, int batch) { return (int64_t)batch * g.hkv * 2 < INT_MAX; }

int launch_fp8_keep(const Fp8KeepArgs& a, void* stream) {
    return (int)launch_programmatic(fp8_keep_kernel, dim3((unsigned)((int64_t)a.b.batch * a.g.hkv * 2)), dim3(kWarps * 32), 0,
                                    reinterpret_cast<cudaStream_t>(stream), a);
}

}  // namespace tq
