// Device helpers of the 8-bit paged cache.
#pragma once

#include "tq_decode_impl.cuh"
#include "tq_fp8.h"

namespace tq {

// 2^e for -126 <= e <= 127, and the exponent of a power of two.
__device__ __forceinline__ float fp8_pow2(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ int fp8_exp_of(float s) { return ((__float_as_int(s) >> 23) & 0xFF) - 127; }

// The least e >= kFp8MinExp with amax <= 448 * 2^e, for a finite amax >= 0:
// amax = 1.f * 2^x against 448 = 1.75 * 2^8.
__device__ __forceinline__ int fp8_exponent(float amax) {
    const int bits = __float_as_int(amax);
    const int e = (bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000 ? 1 : 0);
    return e < kFp8MinExp ? kFp8MinExp : e;
}

// Two fp32 values to two e4m3 codes (nearest, ties to even; lo in the low byte).
__device__ __forceinline__ uint32_t fp8_cvt2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two e4m3 codes (low 16 bits) to two fp16 values; exact.
__device__ __forceinline__ uint32_t fp8_to_half2(uint32_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
    return r;
}
__device__ __forceinline__ float2 fp8_to_float2(uint32_t codes) {
    const uint32_t h = fp8_to_half2(codes);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ int fp8_clamp_cu(const int32_t* cu, int i, int64_t num_tokens) {
    const int v = __ldg(cu + i);
    return v < 0 ? 0 : (v > num_tokens ? (int)num_tokens : v);
}

// Work units of a ragged batch, without a prefix sum: sequence b owns the unit
// numbers from base(b) = cu[b] / step + extra * b up to base(b + 1).  With
// extra = 1 that is enough for the ceil(n / step) pieces of its n rows counted
// from its first, with extra = 2 for the blocks of `step` positions that they
// touch, wherever they start; the rest of its numbers stay idle.
__host__ __device__ __forceinline__ int64_t fp8_units(int64_t num_tokens, int batch, int step, int extra) {
    return num_tokens / step + (int64_t)extra * batch;
}

// The sequence of a unit (the last b with base(b) <= unit), its packed rows and first position.
struct Fp8Seq {
    int b, row0, n, start;
    int64_t base;
};
// Probes 32 places at a time; in the last round the lanes hold 32 neighbours, and what else is wanted of the sequence
// has been read with them: one round trip to memory for up to 32 sequences, two for 1024.  The whole warp calls it.
__device__ __forceinline__ Fp8Seq fp8_seq_of_unit(const Fp8Batch& t, int64_t unit, int step, int extra) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = t.batch;
    while (hi - lo > 32) {
        const int jump = (hi - lo + 31) >> 5, i = lo + lane * jump;
        const bool in = lane == 0 || (i < hi && fp8_clamp_cu(t.cu, i, t.num_tokens) / step + (int64_t)extra * i <= unit);
        lo += (31 - __clz((int)__ballot_sync(0xFFFFFFFFu, in))) * jump;
        hi = min(hi, lo + jump);
    }
    const int i = min(lo + lane, t.batch - 1);
    const int c0 = fp8_clamp_cu(t.cu, i, t.num_tokens), c1 = fp8_clamp_cu(t.cu, i + 1, t.num_tokens), st = __ldg(t.start + i);
    const int64_t base = c0 / step + (int64_t)extra * i;
    const unsigned in = __ballot_sync(0xFFFFFFFFu, lane == 0 || (lo + lane < hi && base <= unit));
    const int l = 31 - __clz((int)in);
    Fp8Seq s;
    s.b = lo + l;
    s.row0 = __shfl_sync(0xFFFFFFFFu, c0, l);
    s.n = __shfl_sync(0xFFFFFFFFu, c1, l) - s.row0;
    s.start = __shfl_sync(0xFFFFFFFFu, st, l);
    s.base = __shfl_sync(0xFFFFFFFFu, base, l);
    return s;
}

}  // namespace tq
