// Keeping the accepted path of a tree of drafts in the 8-bit paged cache: the
// codes of positions start + kept[r] move to positions start + r, whose blocks may
// have other scales.
//
// A block that receives codes takes the largest exponent of the blocks they come
// from and, where it holds earlier positions of the sequence, of its own; codes move by
// c -> c 2^(e_from - e), which is exact but for those that become subnormal.  With
// r <= kept[r] a position's codes are read before, or at the same time as, anything is
// written over them, if the rows go in order: one warp takes a (sequence, head, side)
// and goes through its rows in order, those of a block with the block's final exponent.
#include <cuda_runtime.h>

#include <climits>

#include "tq_fp8_rows.cuh"

namespace tq {
namespace {

constexpr int kBatch = 16;  // rows that a warp has in flight

__global__ void __launch_bounds__(kWarps * 32) fp8_keep_kernel(const Fp8KeepArgs a) {
    const Fp8Geometry& g = a.g;
    const int lane = threadIdx.x & 31;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t hs = item >> 1;
    const int side = (int)(item & 1), b = (int)(hs / g.hkv), h = (int)(hs - (int64_t)b * g.hkv);
    if (b >= a.b.batch) return;
    const int c0 = fp8_clamp_cu(a.b.cu, b, a.b.num_tokens), n = fp8_clamp_cu(a.b.cu, b + 1, a.b.num_tokens) - c0;
    const int start = __ldg(a.b.start + b);
    if (n <= 0) return;
    if (start < 0) {
        if (lane == 0) flag(a.status, TQ_FLAG_BAD_SLOT);
        return;
    }
    const int32_t* row = a.b.block_table + (int64_t)b * a.b.max_blocks;
    // the page that holds a position of the sequence, or -1
    auto page_of_pos = [&](int64_t p) -> int64_t {
        const int64_t j = p >> g.bs_shift;
        const int id = j < a.b.max_blocks ? __ldg(row + j) : -1;
        return id >= 0 && id < g.num_blocks ? ((int64_t)id * g.hkv + h) * 2 + side : -1;
    };
    // where row r comes from: its page (-1: it is skipped) and slot
    auto source = [&](int r, int& slot) -> int64_t {
        const int k = __ldg(a.kept + c0 + r);
        const int64_t p = (int64_t)start + k;
        slot = (int)(p & (g.bs - 1));
        return k >= r ? page_of_pos(p) : -1;
    };
    const int64_t stride = (int64_t)g.bs * kHeadDim;
    for (int r0 = 0; r0 < n;) {  // block by block
        const int64_t p0 = (int64_t)start + r0;
        const int off = (int)(p0 & (g.bs - 1)), m = min(g.bs - off, n - r0);
        const int64_t page = page_of_pos(p0);
        const int e_own = page >= 0 ? fp8_exp_of(g.scales[page]) : 0;
        int e = off > 0 && page >= 0 ? e_own : INT_MIN;
        bool bad = page < 0;
        for (int i = lane; i < m; i += 32) {
            int slot;
            const int64_t from = source(r0 + i, slot);
            if (from >= 0) e = max(e, fp8_exp_of(g.scales[from]));
            else bad = true;
        }
        e = __reduce_max_sync(0xFFFFFFFFu, e);
        if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) flag(a.status, TQ_FLAG_BAD_SLOT);
        if (page >= 0 && e != INT_MIN) {
            uint8_t* dst = g.pool + page * stride;
            for (int i0 = 0; i0 < m; i0 += kBatch) {  // a lane holds 4 codes of a row
                uint32_t code[kBatch];
                int d[kBatch];  // what the row's exponent changes by; 1: skipped
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    d[i] = 1;
                    code[i] = 0;
                    if (i0 + i < m) {
                        int slot;
                        const int64_t from = source(r0 + i0 + i, slot);
                        if (from >= 0) {
                            d[i] = (from == page ? e_own : fp8_exp_of(g.scales[from])) - e;
                            code[i] = *(reinterpret_cast<const uint32_t*>(g.pool + from * stride + (int64_t)slot * kHeadDim) + lane);
                        }
                    }
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (d[i] <= 0)
                        *(reinterpret_cast<uint32_t*>(dst + (int64_t)(off + i0 + i) * kHeadDim) + lane) = scale_codes(code[i], d[i]);
                __syncwarp();
            }
            if (off > 0 && e > e_own) move_codes(dst, off, e_own - e);
            __syncwarp();
            if (lane == 0) g.scales[page] = fp8_pow2(e);
            __syncwarp();
        }
        r0 += m;
    }
}

}  // namespace

bool fp8_keep_counts(const Fp8Geometry& g, int batch) { return (int64_t)batch * g.hkv * 2 / kWarps < (1 << 30); }

int launch_fp8_keep(const Fp8KeepArgs& a, void* stream) {
    const int64_t warps = (int64_t)a.b.batch * a.g.hkv * 2;
    return (int)launch_programmatic(fp8_keep_kernel, dim3((unsigned)((warps + kWarps - 1) / kWarps)), dim3(kWarps * 32), 0,
                                    reinterpret_cast<cudaStream_t>(stream), a);
}

}  // namespace tq
