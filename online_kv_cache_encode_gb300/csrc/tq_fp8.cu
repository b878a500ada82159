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
    bool live;       // the unit has tokens there
    int blk;         // the block's id, not checked yet (-1: past the block table)
    int64_t row0;    // packed row of the warp's first token (may lie before the sequence's first)
    int first;       // offset of the warp's 16 tokens in the block
    int lo, hi;      // offsets in the block of the new tokens: lo <= t < hi
    int head, side;
};

// Work item `w` (16 tokens) of the launch; 2^wpb_shift warps per block of tokens.
__device__ __forceinline__ Place find_place(const Fp8Geometry& g, const Fp8Batch& b, int64_t w, int wpb_shift,
                                            int32_t* status) {
    Place p;
    const int64_t item = w >> wpb_shift;
    p.first = (int)(w & ((1 << wpb_shift) - 1)) * kRows;
    p.side = (int)(item & 1);
    const uint32_t uh = (uint32_t)(item >> 1);  // the host keeps the grid, and so this, below 2^31
    const uint32_t u = uh / (uint32_t)g.hkv;
    p.head = (int)(uh - u * (uint32_t)g.hkv);
    p.live = false;
    p.blk = -1;
    p.row0 = 0;
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
    p.lo = start > pos0 ? (int)(start - pos0) : 0;
    p.hi = (int)min((int64_t)g.bs, (int64_t)start + n - pos0);
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

// A 16-byte piece of a row: V elements.  top() is the largest magnitude as an
// integer (magnitudes order as their bits do, infinities and NaN above all).
template <typename T>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int V = 4;
    static constexpr uint32_t kInf = 0x7F800000u;
    static __device__ __forceinline__ uint32_t top(const uint4& r, uint32_t m) {
        return max(max(m, max(r.x & 0x7FFFFFFFu, r.y & 0x7FFFFFFFu)), max(r.z & 0x7FFFFFFFu, r.w & 0x7FFFFFFFu));
    }
    static __device__ __forceinline__ uint32_t join(uint32_t m) { return m; }
    static __device__ __forceinline__ float value(uint32_t m) { return __uint_as_float(m); }
    static __device__ __forceinline__ void get(const uint4& r, float (&x)[4]) {
        x[0] = __uint_as_float(r.x); x[1] = __uint_as_float(r.y); x[2] = __uint_as_float(r.z); x[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
// Two 16-bit elements in a word: magnitudes and maxima two at a time.
struct Elem16 {
    static constexpr int V = 8;
    static __device__ __forceinline__ uint32_t top(const uint4& r, uint32_t m) {
        const uint32_t a = __vmaxu2(r.x & 0x7FFF7FFFu, r.y & 0x7FFF7FFFu), b = __vmaxu2(r.z & 0x7FFF7FFFu, r.w & 0x7FFF7FFFu);
        return __vmaxu2(m, __vmaxu2(a, b));
    }
    static __device__ __forceinline__ uint32_t join(uint32_t m) { return max(m & 0xFFFFu, m >> 16); }
};
template <>
struct Elem<__nv_bfloat16> : Elem16 {
    static constexpr uint32_t kInf = 0x7F80u;
    static __device__ __forceinline__ float value(uint32_t m) { return __uint_as_float(m << 16); }
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
struct Elem<__half> : Elem16 {
    static constexpr uint32_t kInf = 0x7C00u;
    static __device__ __forceinline__ float value(uint32_t m) { return __half2float(__ushort_as_half((unsigned short)m)); }
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
// Five CTAs an SM (48 registers) hide the look-up's chain of loads: 33 us for 32K x 8 heads of bf16, 41 at four, 35 with
// CTAs that go from item to item and look the next one up ahead.  A warp of fp32 rows holds twice the registers (two CTAs
// an SM: 55 us for the same rows, 0.90 of HBM).
template <typename T>
__global__ void __launch_bounds__(kWarps * 32, sizeof(T) == 4 ? 2 : 5) fp8_write_kernel(const Fp8WriteArgs a, int wpb_shift) {
    using E = Elem<T>;
    constexpr int V = E::V, LPR = kHeadDim / V, RPI = 32 / LPR, IT = kRows / RPI;
    __shared__ uint32_t tops[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    const Place p = find_place(a.g, a.b, (int64_t)blockIdx.x * kWarps + warp, wpb_shift, a.status);
    const int sub = lane / LPR, col = (lane % LPR) * V;
    const int64_t step = p.side ? a.v_token : a.k_token;
    const T* src = static_cast<const T*>(p.side ? a.V : a.K) + p.row0 * step + p.head * (p.side ? a.v_head : a.k_head) + col;
    // the rows are on their way before the block's id is looked at
    uint4 raw[IT];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int r = i * RPI + sub, t = p.first + r;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (t >= p.lo && t < p.hi) raw[i] = __ldcs(reinterpret_cast<const uint4*>(src + r * step));
    }
    int64_t page = 0;
    const bool there = page_of(a.g, p, a.status, page);
    // the block's scale as earlier tokens left it
    const int e_old = there && p.lo > 0 ? fp8_exp_of(a.g.scales[page]) : kFp8MinExp;
#pragma unroll
    for (int i = 0; i < IT; ++i) top = E::top(raw[i], top);
    top = __reduce_max_sync(0xFFFFFFFFu, E::join(top));
    const bool odd = top >= E::kInf;  // an inf or a NaN among the new rows: the maximum of the others
    if (odd) {
        float best = 0.f;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            float x[V];
            E::get(raw[i], x);
#pragma unroll
            for (int k = 0; k < V; ++k) best = fmaxf(best, finite(x[k]) ? fabsf(x[k]) : 0.f);
        }
        T b = (T)best;  // exact: one of the elements
        if constexpr (V == 4) top = __float_as_uint(best);
        else top = *reinterpret_cast<const unsigned short*>(&b);
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        if (lane == 0) flag(a.status, TQ_FLAG_NONFINITE);
    }
    if (wpb_shift) {  // the block's warps are neighbours of one CTA
        if (lane == 0) tops[warp] = top;
        __syncthreads();
        for (int w = 0; w < 1 << wpb_shift; ++w) top = max(top, tops[(warp >> wpb_shift << wpb_shift) + w]);
    }
    if (!there) return;
    const int e = max(fp8_exponent(E::value(top)), e_old);
    if (p.first == 0 && lane == 0) a.g.scales[page] = fp8_pow2(e);
    const float inv = fp8_pow2(-e);
    uint8_t* dst = a.g.pool + page * ((int64_t)a.g.bs * kHeadDim) + (int64_t)p.first * kHeadDim + col;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int r = i * RPI + sub, t = p.first + r;
        float x[V];
        E::get(raw[i], x);
        if (odd) {
#pragma unroll
            for (int k = 0; k < V; ++k) x[k] = x[k] != x[k] ? 0.f : x[k];  // NaN is stored as 0
        }
        uint32_t w[V / 4];
#pragma unroll
        for (int k = 0; k < V; k += 4) w[k / 4] = fp8_cvt2(x[k] * inv, x[k + 1] * inv) | (fp8_cvt2(x[k + 2] * inv, x[k + 3] * inv) << 16);
        if (t >= p.lo && t < p.hi) {
            if constexpr (V == 8) *reinterpret_cast<uint2*>(dst + r * kHeadDim) = make_uint2(w[0], w[V / 4 - 1]);
            else *reinterpret_cast<uint32_t*>(dst + r * kHeadDim) = w[0];
        }
    }
    if (p.lo > p.first && e > e_old) {  // earlier rows move to the larger scale
        const float m = fp8_pow2(max(e_old - e, -100));
        for (int r = 0; r < min(p.lo - p.first, kRows); ++r) {
            uint32_t* c = reinterpret_cast<uint32_t*>(a.g.pool + page * ((int64_t)a.g.bs * kHeadDim) +
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
    int64_t page = 0;
    if (!page_of(a.g, p, a.status, page)) return;
    const int sub = lane / LPR, col = (lane % LPR) * V;
    const float s = __ldg(a.g.scales + page);
    const uint8_t* src = a.g.pool + page * ((int64_t)a.g.bs * kHeadDim) + (int64_t)p.first * kHeadDim + col;
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

int64_t grid_of(const Fp8Geometry& g, const Fp8Batch& b) {
    const int64_t warps = (fp8_units(b.num_tokens, b.batch, g.bs, 2) * g.hkv * 2) << (g.bs_shift - 4);
    return (warps + kWarps - 1) / kWarps;
}

}  // namespace

bool fp8_rows_count(const Fp8Geometry& g, const Fp8Batch& b) { return grid_of(g, b) < (1 << 28); }

int launch_fp8_write(const Fp8WriteArgs& a, void* stream) {
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int shift = a.g.bs_shift - 4;
    const dim3 grid((unsigned)grid_of(a.g, a.b)), block(kWarps * 32);
    if (a.dtype == TQ_F32) return (int)launch_programmatic(fp8_write_kernel<float>, grid, block, 0, s, a, shift);
    if (a.dtype == TQ_BF16) return (int)launch_programmatic(fp8_write_kernel<__nv_bfloat16>, grid, block, 0, s, a, shift);
    return (int)launch_programmatic(fp8_write_kernel<__half>, grid, block, 0, s, a, shift);
}

int launch_fp8_read(const Fp8ReadArgs& a, void* stream) {
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int shift = a.g.bs_shift - 4;
    const dim3 grid((unsigned)grid_of(a.g, a.b)), block(kWarps * 32);
    if (a.dtype == TQ_F32) return (int)launch_programmatic(fp8_read_kernel<float>, grid, block, 0, s, a, shift);
    if (a.dtype == TQ_BF16) return (int)launch_programmatic(fp8_read_kernel<__nv_bfloat16>, grid, block, 0, s, a, shift);
    return (int)launch_programmatic(fp8_read_kernel<__half>, grid, block, 0, s, a, shift);
}

}  // namespace tq
