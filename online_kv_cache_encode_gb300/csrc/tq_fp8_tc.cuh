// Tensor-core and TMA building blocks of the 8-bit cache's attention kernels.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "tq_fp8.cuh"
#include "tq_tcgen05.cuh"

namespace tq {

__device__ __forceinline__ void mma_f8_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// kind::f8f6f4, e4m3 x e4m3 -> fp32, M = 128; bits 15 and 16 read A and B MN-major
__device__ constexpr uint32_t idesc_f8(int n, bool mn) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | (8u << 24) | (mn ? (3u << 15) : 0u);
}
// Rows of 128 bytes in the 128-byte swizzle, 8-row groups `sbo` bytes apart: K-major as they are, or read MN-major,
// where 128 e4m3 values fill the one atom along M (its leading offset is not used).
__device__ __forceinline__ uint64_t desc_rows(uint32_t saddr, uint32_t sbo) { return tc::smem_desc_sw128(saddr, sbo); }
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* map, int row, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(map), "r"(0), "r"(row), "r"(bar)
        : "memory");
}
// Whether the phase of the given parity is over; does not wait.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ float redux_max(float x) {  // NaN is ignored
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}
// C columns of the thread's tensor-memory lane; the registers hold them after tmem_ready.
template <int C>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t* r) {
    if constexpr (C == 4)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
    else if constexpr (C == 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(addr) : "memory");
    else
        for (int i = 0; i < C; i += 8) tmem_ld<8>(addr + i, r + i);
}
template <int C>
__device__ __forceinline__ void tmem_ready(uint32_t* r) {  // registers are defined from here on
    tc::wait_ld();
#pragma unroll
    for (int i = 0; i < C; i += 4) asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]));
}
// Two 16-bit elements of a word as floats, and back (nearest, ties to even).
template <typename T>
__device__ __forceinline__ float2 two_floats(uint32_t w) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    else
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack_two(float lo, float hi) {
    uint32_t r;
    if constexpr (std::is_same<T, __nv_bfloat16>::value) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Query rows of 128 elements in terms of e4m3: x 2^-e = h1 + h2 + .., with e the exponent that puts the row's largest
// element into (224, 448].  LANES lanes hold a row, W words of two elements each (the whole warp calls it: 32 lanes a
// row or 16, two rows at once), and R such rows go through every step together: one at a time its chain of shuffles
// and conversions took 400 cycles.  The remainders are exact in fp16, whose 11 bits hold what 16-bit inputs have
// (elements below 2^-24 / 448 of the row's largest vanish).
template <typename T, int LANES, int R>
struct Fp8Split {
    static constexpr int W = 64 / LANES;
    uint32_t y[R][W];
    int e[R];
    bool odd[R];  // an element that is not finite
    __device__ __forceinline__ explicit Fp8Split(const uint32_t (&raw)[R][W]) {
        uint32_t top[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            uint32_t m2 = raw[r][0] & 0x7FFF7FFFu;  // magnitudes order as their bits do
#pragma unroll
            for (int i = 1; i < W; ++i) m2 = __vmaxu2(m2, raw[r][i] & 0x7FFF7FFFu);
            top[r] = max(m2 & 0xFFFFu, m2 >> 16);
        }
        if constexpr (LANES == 32) {
#pragma unroll
            for (int r = 0; r < R; ++r) top[r] = __reduce_max_sync(0xFFFFFFFFu, top[r]);
        } else {
#pragma unroll
            for (int o = LANES / 2; o; o >>= 1)
#pragma unroll
                for (int r = 0; r < R; ++r) top[r] = max(top[r], __shfl_xor_sync(0xFFFFFFFFu, top[r], o));
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            odd[r] = top[r] >= (std::is_same<T, __nv_bfloat16>::value ? 0x7F80u : 0x7C00u);
            e[r] = odd[r] ? 0 : fp8_exponent(two_floats<T>(top[r]).x);
            const float inv = fp8_pow2(-e[r]);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float2 a = two_floats<T>(raw[r][i]);
                y[r][i] = pack_two<__half>(a.x * inv, a.y * inv);
            }
        }
    }
    // The next term's codes, four to a word; what remains is multiplied by UP (a pair of fp16 powers of two, or 0: by 1).
    template <uint32_t UP>
    __device__ __forceinline__ void term(uint32_t (&w)[R][W / 2]) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < W; i += 2) {
                const uint32_t lo = half2_to_fp8(y[r][i]), hi = half2_to_fp8(y[r][i + 1]);
                w[r][i / 2] = lo | (hi << 16);
                y[r][i] = rest<UP>(y[r][i], fp8_to_half2(lo));
                y[r][i + 1] = rest<UP>(y[r][i + 1], fp8_to_half2(hi));
            }
    }
    // What a product with row r's terms is multiplied with; NaN makes the row NaN.
    __device__ __forceinline__ float factor(int r, float scale) const { return odd[r] ? NAN : scale * fp8_pow2(e[r]); }

  private:
    static __device__ __forceinline__ uint32_t half2_to_fp8(uint32_t h) {
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
        return r;
    }
    template <uint32_t UP>
    static __device__ __forceinline__ uint32_t rest(uint32_t x, uint32_t h) {
        uint32_t r;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(h));
        if constexpr (UP != 0) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(UP));
        return r;
    }
};

}  // namespace tq
