// The 8-bit paged cache: writing new keys and values into it, and reading it
// back.
//
// A block of bs tokens of one KV head and side (K or V) holds e4m3 codes c and
// one scale s = 2^e, x ~ c s.  Writing takes the least e with max|x| <= 448 2^e
// over the block's new rows, or the block's present e where it already holds
// earlier positions of the sequence and that is larger; the earlier rows move to
// a larger scale by c -> c 2^(e_old - e).  A power of two costs a floating code
// nothing but range (its relative step is the same at every scale, and less
// than one of its 15 binades stays unused), and makes that move exact down to
// the subnormal codes.
//
// One warp owns 16 tokens of one (block, head, side), a whole block goes to
// neighbouring warps of one CTA, and a block is touched by no other: no
// atomics, and the same bytes every time.  Both kernels only move data: T x hkv
// x 256 x (1 + element size) bytes is what they cannot do without.
#include <cuda_runtime.h>

#include "tq_fp8.cuh"

namespace tq {
namespace {

constexpr int kWarps = 8;
constexpr int kRows = 16;  // tokens a warp holds

// Where one warp works: 16 positions of a block.
struct Place {
    bool live;       // the unit has tokens and its block lies in the pool
    int64_t page;    // (block * hkv + head) * 2 + side
    int64_t row0;    // packed row of the warp's first token (may lie before the sequence's first)
    int first;       // offset of the warp's 16 tokens in the block
    int lo, hi;      // offsets in the block of the new tokens: lo <= t < hi
    int head, side;
};

// Work item `w` (16 tokens) of the launch; WPB = warps per block of tokens.
__device__ __forceinline__ Place find_place(const Fp8Geometry& g, const Fp8Batch& b, int64_t w, int wpb_shift,
                                            int32_t* status) {
    Place p;
    const int64_t item = w >> wpb_shift;
    p.first = (int)(w & ((1 << wpb_shift) - 1)) * kRows;
    p.side = (int)(item & 1);
    const int64_t uh = item >> 1;
    const int64_t u = uh / g.hkv;
    p.head = (int)(uh - u * g.hkv);
    p.live = false;
    p.page = 0;
    p.row0 = 0;
    p.lo = p.hi = 0;
    if (u >= fp8_units(b.num_tokens, b.batch, g.bs_shift)) return p;
    const int s = fp8_seq_of_unit(b.cu, b.batch, b.num_tokens, u, g.bs_shift);
    const int c0 = fp8_clamp_cu(b.cu, s, b.num_tokens), c1 = fp8_clamp_cu(b.cu, s + 1, b.num_tokens);
    const int n = c1 - c0, start = __ldg(b.start + s);
    const int64_t j = u - ((int64_t)(c0 >> g.bs_shift) + 2 * (int64_t)s);
    if (n <= 0 || j < 0) return p;
    if (start < 0) {
        if (j == 0 && (threadIdx.x & 31) == 0) flag(status, TQ_FLAG_BAD_SLOT);
        return p;
    }
    const int64_t blk_i = (start >> g.bs_shift) + j;  // the block of the sequence
    const int64_t pos0 = blk_i << g.bs_shift;
    if (pos0 >= (int64_t)start + n) return p;
    const int blk = blk_i < b.max_blocks ? __ldg(b.block_table + (int64_t)s * b.max_blocks + blk_i) : -1;
    if (blk < 0 || blk >= g.num_blocks) {
        if ((threadIdx.x & 31) == 0) flag(status, TQ_FLAG_BAD_SLOT);
        return p;
    }
    p.live = true;
    p.page = ((int64_t)blk * g.hkv + p.head) * 2 + p.side;
    p.row0 = (int64_t)c0 + (pos0 - start) + p.first;
    p.lo = start > pos0 ? (int)(start - pos0) : 0;
    p.hi = (int)min((int64_t)g.bs, (int64_t)start + n - pos0);
    return p;
}

template <typename T>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int V = 4;  // elements of a 16-byte piece
    static __device__ __forceinline__ void get(const uint4& r, float (&x)[4]) {
        x[0] = __uint_as_float(r.x); x[1] = __uint_as_float(r.y); x[2] = __uint_as_float(r.z); x[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int V = 8;
    static __device__ __forceinline__ void get(const uint4& r, float (&x)[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Elem<__half> {
    static constexpr int V = 8;
    static __device__ __forceinline__ void get(const uint4& r, float (&x)[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// A lane holds 16-byte pieces: LPR lanes make a row of 128 elements, a warp
// RPI rows at a time.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) fp8_write_kernel(const Fp8WriteArgs a, int wpb_shift) {
    using E = Elem<T>;
    constexpr int V = E::V, LPR = kHeadDim / V, RPI = 32 / LPR, IT = kRows / RPI;
    __shared__ float tops[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    const Place p = find_place(a.g, a.b, (int64_t)blockIdx.x * kWarps + warp, wpb_shift, a.status);
    const int sub = lane / LPR, col = (lane % LPR) * V;
    const T* src = static_cast<const T*>(p.side ? a.V : a.K) + p.row0 * (p.side ? a.v_token : a.k_token) +
                   p.head * (p.side ? a.v_head : a.k_head) + col;
    const int64_t step = p.side ? a.v_token : a.k_token;
    uint4 raw[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int r = i * RPI + sub, t = p.first + r;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (p.live && t >= p.lo && t < p.hi) raw[i] = __ldg(reinterpret_cast<const uint4*>(src + r * step));
    }
    // the block's scale as earlier tokens left it
    const int e_old = p.live && p.lo > 0 ? fp8_exp_of(a.g.scales[p.page]) : kFp8MinExp;
    float top = 0.f;
    bool odd = false;  // an inf or a NaN among the new rows
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        float x[V];
        E::get(raw[i], x);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const bool f = finite(x[k]);
            odd |= !f;
            top = fmaxf(top, f ? fabsf(x[k]) : 0.f);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (__any_sync(0xFFFFFFFFu, odd) && lane == 0) flag(a.status, TQ_FLAG_NONFINITE);
    if (wpb_shift) {  // the block's warps are neighbours of one CTA
        if (lane == 0) tops[warp] = top;
        __syncthreads();
        for (int w = 0; w < 1 << wpb_shift; ++w) top = fmaxf(top, tops[(warp >> wpb_shift << wpb_shift) + w]);
    }
    if (!p.live) return;
    const int e = max(fp8_exponent(top), e_old);
    if (p.first == 0 && lane == 0) a.g.scales[p.page] = fp8_pow2(e);
    const float inv = fp8_pow2(-e);
    uint8_t* dst = a.g.pool + p.page * ((int64_t)a.g.bs * kHeadDim) + (int64_t)p.first * kHeadDim + col;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int r = i * RPI + sub, t = p.first + r;
        float x[V];
        E::get(raw[i], x);
        uint32_t w[V / 4];
#pragma unroll
        for (int k = 0; k < V; k += 4) {
#pragma unroll
            for (int m = 0; m < 4; ++m) x[k + m] = x[k + m] != x[k + m] ? 0.f : x[k + m] * inv;  // NaN is stored as 0
            w[k / 4] = fp8_cvt2(x[k], x[k + 1]) | (fp8_cvt2(x[k + 2], x[k + 3]) << 16);
        }
        if (t >= p.lo && t < p.hi) {
            if constexpr (V == 8) *reinterpret_cast<uint2*>(dst + r * kHeadDim) = make_uint2(w[0], w[V / 4 - 1]);
            else *reinterpret_cast<uint32_t*>(dst + r * kHeadDim) = w[0];
        }
    }
    if (p.lo > p.first && e > e_old) {  // earlier rows move to the larger scale
        const float m = fp8_pow2(max(e_old - e, -100));
        for (int r = 0; r < min(p.lo - p.first, kRows); ++r) {
            uint32_t* c = reinterpret_cast<uint32_t*>(a.g.pool + p.page * ((int64_t)a.g.bs * kHeadDim) +
                                                      (int64_t)(p.first + r) * kHeadDim) + lane;
            const uint32_t v = *c;
            const float2 x = fp8_to_float2(v & 0xFFFFu), y = fp8_to_float2(v >> 16);
            *c = fp8_cvt2(x.x * m, x.y * m) | (fp8_cvt2(y.x * m, y.y * m) << 16);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) fp8_read_kernel(const Fp8ReadArgs a, int wpb_shift) {
    using E = Elem<T>;
    constexpr int V = E::V, LPR = kHeadDim / V, RPI = 32 / LPR, IT = kRows / RPI;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    const Place p = find_place(a.g, a.b, (int64_t)blockIdx.x * kWarps + warp, wpb_shift, a.status);
    if (!p.live) return;
    const int sub = lane / LPR, col = (lane % LPR) * V;
    const float s = __ldg(a.g.scales + p.page);
    const uint8_t* src = a.g.pool + p.page * ((int64_t)a.g.bs * kHeadDim) + (int64_t)p.first * kHeadDim + col;
    T* dst = static_cast<T*>(p.side ? a.V : a.K) + (p.row0 * a.g.hkv + p.head) * kHeadDim + col;
    const int64_t step = (int64_t)a.g.hkv * kHeadDim;
    uint2 raw[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int r = i * RPI + sub, t = p.first + r;
        raw[i] = make_uint2(0, 0);
        if (t >= p.lo && t < p.hi) {
            if constexpr (V == 8) raw[i] = __ldg(reinterpret_cast<const uint2*>(src + r * kHeadDim));
            else raw[i].x = __ldg(reinterpret_cast<const uint32_t*>(src + r * kHeadDim));
        }
    }
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int r = i * RPI + sub, t = p.first + r;
        const uint32_t w[2] = {raw[i].x, raw[i].y};
        float x[V];
#pragma unroll
        for (int k = 0; k < V; k += 2) {
            const float2 f = fp8_to_float2((w[k / 4] >> (8 * (k % 4))) & 0xFFFFu);
            x[k] = f.x * s;
            x[k + 1] = f.y * s;
        }
        if (t >= p.lo && t < p.hi) *reinterpret_cast<uint4*>(dst + r * step) = E::put(x);
    }
}

template <typename Args>
bool grid_of(const Args& a, int& wpb_shift, int64_t& ctas) {
    wpb_shift = a.g.bs_shift - 4;
    const int64_t warps = (fp8_units(a.b.num_tokens, a.b.batch, a.g.bs_shift) * a.g.hkv * 2) << wpb_shift;
    ctas = (warps + kWarps - 1) / kWarps;
    return ctas <= 0x7FFFFFFF;
}

}  // namespace

int launch_fp8_write(const Fp8WriteArgs& a, void* stream) {
    int shift;
    int64_t ctas;
    if (!grid_of(a, shift, ctas)) return (int)cudaErrorInvalidConfiguration;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)ctas), block(kWarps * 32);
    if (a.dtype == TQ_F32) return (int)launch_programmatic(fp8_write_kernel<float>, grid, block, 0, s, a, shift);
    if (a.dtype == TQ_BF16) return (int)launch_programmatic(fp8_write_kernel<__nv_bfloat16>, grid, block, 0, s, a, shift);
    return (int)launch_programmatic(fp8_write_kernel<__half>, grid, block, 0, s, a, shift);
}

int launch_fp8_read(const Fp8ReadArgs& a, void* stream) {
    int shift;
    int64_t ctas;
    if (!grid_of(a, shift, ctas)) return (int)cudaErrorInvalidConfiguration;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)ctas), block(kWarps * 32);
    if (a.dtype == TQ_F32) return (int)launch_programmatic(fp8_read_kernel<float>, grid, block, 0, s, a, shift);
    if (a.dtype == TQ_BF16) return (int)launch_programmatic(fp8_read_kernel<__nv_bfloat16>, grid, block, 0, s, a, shift);
    return (int)launch_programmatic(fp8_read_kernel<__half>, grid, block, 0, s, a, shift);
}

}  // namespace tq
