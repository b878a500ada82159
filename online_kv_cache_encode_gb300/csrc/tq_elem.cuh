// 16-byte pieces of a row in each element type.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace tq {
namespace {

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

}  // namespace
}  // namespace tq
