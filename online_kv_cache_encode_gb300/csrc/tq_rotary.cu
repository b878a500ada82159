// Rotary positions: the table of a position's cosines and sines, and the
// rotation of rows of heads (or by the transposed matrix, which is the gradient).
//
// What bounds the rotation is the rows themselves, read and written once: 2 T H d
// times the element size, plus a table row of 4 rot bytes a token.  A warp takes one
// token and up to 16 heads of 128 dims (4 KB of 16-bit elements in flight), so a lane
// reads the cosines and sines of its pairs once for all of them.
//
// 32768 tokens x 64 heads of bf16: 165 us, 0.99 of what a copy of the rows takes (scalar
// products 211, two-wide ones 197, addresses by steps and three CTAs an SM 166, whose 80
// registers cost the 16-bit wide variants 16 to 20 bytes of spills); one token of 64 sequences, 32
// heads: 2.8 us, of which the launch is the most.
#include <cuda_runtime.h>

#include "tq_decode_impl.cuh"
#include "tq_rotary.cuh"

namespace tq {
namespace {

constexpr int kRotWarps = 8;
constexpr int kRotHeads = 16;  // heads of a warp

template <typename T, bool INTER, bool WIDE>
__global__ void __launch_bounds__(kRotWarps * 32, 3) rotary_kernel(const RotaryArgs a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    grid_launch_dependents();
    const int parts = (a.heads + kRotHeads - 1) / kRotHeads;
    const int64_t item = (int64_t)blockIdx.x * kRotWarps + warp;
    const int64_t token = item / parts;
    if (token >= a.tokens) return;
    const int h0 = (int)(item - token * parts) * kRotHeads;
    const int32_t p = __ldg(a.positions + token);
    if (p < 0 || p >= a.r.positions) {  // the row stays as it was
        if (lane == 0) flag(a.status, TQ_FLAG_BAD_SLOT);
        return;
    }
    rotate_heads<T, INTER, WIDE, 4>(a.r, a.r.table + (int64_t)p * a.r.rot, a.transpose != 0,
                          static_cast<const T*>(a.x) + token * a.x_token + h0 * a.x_head, a.x_head,
                          static_cast<T*>(a.out) + token * a.out_token + h0 * a.out_head, a.out_head, min(kRotHeads, a.heads - h0), a.d);
}

struct Frequencies {
    double f[kRotaryMaxDim / 2];
};
__global__ void rotary_table_kernel(const __grid_constant__ Frequencies f, int half, double magnitude, int64_t positions, float* table) {
    grid_dependency_wait();
    grid_launch_dependents();
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < positions * half; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t p = i / half;
        const int j = (int)(i - p * half);
        double s, c;
        sincos((double)p * f.f[j], &s, &c);
        table[p * 2 * half + j] = (float)(magnitude * c);
        table[p * 2 * half + half + j] = (float)(magnitude * s);
    }
}

template <typename T, bool INTER>
int launch(const RotaryArgs& a, cudaStream_t s) {
    const int64_t warps = a.tokens * ((a.heads + kRotHeads - 1) / kRotHeads);
    const dim3 grid((unsigned)((warps + kRotWarps - 1) / kRotWarps)), block(kRotWarps * 32);
    if (32 % (a.d / (2 * Elem<T>::V)) == 0) return (int)launch_programmatic(rotary_kernel<T, INTER, true>, grid, block, 0, s, a);
    return (int)launch_programmatic(rotary_kernel<T, INTER, false>, grid, block, 0, s, a);
}
template <typename T>
int launch(const RotaryArgs& a, cudaStream_t s) {
    return a.r.interleaved ? launch<T, true>(a, s) : launch<T, false>(a, s);
}

}  // namespace

bool rotary_counts(int64_t tokens, int heads) {
    return tokens * ((heads + kRotHeads - 1) / kRotHeads) / kRotWarps < (1 << 30);
}

int launch_rotary(const RotaryArgs& a, void* stream) {
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (a.dtype == TQ_F32) return launch<float>(a, s);
    return a.dtype == TQ_BF16 ? launch<__nv_bfloat16>(a, s) : launch<__half>(a, s);
}

int launch_rotary_table(const double* frequencies, int rot, double magnitude, int64_t positions, float* table, void* stream) {
    Frequencies f{};
    for (int i = 0; i < rot / 2; ++i) f.f[i] = frequencies[i];
    const int64_t blocks = (positions * (rot / 2) + 255) / 256;
    return (int)launch_programmatic(rotary_table_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0,
                                    reinterpret_cast<cudaStream_t>(stream), f, rot / 2, magnitude, positions, table);
}

}  // namespace tq
