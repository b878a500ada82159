// Rotary positions on pieces of a row.
//
// A head's first `rot` dims are pairs (a, b), rotated by the position's angles:
//   a' = a c - b s,   b' = b c + a s,   c = m cos(p f_j), s = m sin(p f_j),
// with c and s from a table that was computed in 64 bits (an angle of position 10^5 in 32 bits is off by 2^-7).
// Products and sums are rounded one by one, so that the result does not depend on how a compiler contracts them
// and a rotated key has the same codes wherever it is rotated.
#pragma once

#include "tq_elem.cuh"
#include "tq_rotary.h"

namespace tq {
namespace {

__device__ __forceinline__ void rotate_pair(float& a, float& b, float c, float s) {
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = x;
}

// A lane's two 16-byte pieces of a row of `pieces` pieces, of V elements each: lane l of the pieces / 2 that share a row.
// In the half layout piece j meets its partner j + rot / 2 in one lane; everything else goes in the row's order.
template <int V>
struct RotaryLane {
    int c0, c1;    // the pieces
    int at;        // cosines of the first piece's pairs start there (half: of both pieces')
    int at1;       // of the second's (interleaved)
    bool on0, on1; // whether they are rotated
    __device__ __forceinline__ RotaryLane(const RotaryTable& r, int l, int pieces) {
        if (r.interleaved) {
            c0 = l;
            c1 = l + pieces / 2;
            on0 = c0 * V < r.rot;
            on1 = c1 * V < r.rot;
            at = c0 * (V / 2);
            at1 = c1 * (V / 2);
        } else {
            const int half = r.rot / (2 * V);
            on0 = on1 = l < half;
            c0 = on0 ? l : 2 * l;
            c1 = on0 ? l + half : 2 * l + 1;
            at = at1 = l * V;
        }
    }
};

// The cosines and sines of a lane's pairs at one position (table row `row`): V of each, whichever the layout.
template <int V>
struct RotaryAngles {
    float c[V], s[V];
    __device__ __forceinline__ void load(const RotaryTable& r, const RotaryLane<V>& l, const float* row, bool transpose) {
        const float* sines = row + r.rot / 2;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            c[i] = 1.f;
            s[i] = 0.f;
        }
        if (r.interleaved) {
            if (l.on0) get<V / 2>(row + l.at, sines + l.at, c, s);
            if (l.on1) get<V / 2>(row + l.at1, sines + l.at1, c + V / 2, s + V / 2);
        } else if (l.on0) {
            get<V>(row + l.at, sines + l.at, c, s);
        }
        if (transpose)
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] = -s[i];
    }

  private:
    template <int N>
    static __device__ __forceinline__ void get(const float* pc, const float* ps, float* c, float* s) {
        if constexpr (N >= 4) {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const float4 a = __ldg(reinterpret_cast<const float4*>(pc + i)), b = __ldg(reinterpret_cast<const float4*>(ps + i));
                c[i] = a.x; c[i + 1] = a.y; c[i + 2] = a.z; c[i + 3] = a.w;
                s[i] = b.x; s[i + 1] = b.y; s[i + 2] = b.z; s[i + 3] = b.w;
            }
        } else {
            const float2 a = __ldg(reinterpret_cast<const float2*>(pc)), b = __ldg(reinterpret_cast<const float2*>(ps));
            c[0] = a.x; c[1] = a.y;
            s[0] = b.x; s[1] = b.y;
        }
    }
};

// Rotates a lane's two pieces x, y.
template <int V>
__device__ __forceinline__ void rotate_pieces(const RotaryTable& r, const RotaryLane<V>& l, const RotaryAngles<V>& t, float (&x)[V],
                                              float (&y)[V]) {
    if (r.interleaved) {
        if (l.on0)
#pragma unroll
            for (int i = 0; i < V; i += 2) rotate_pair(x[i], x[i + 1], t.c[i / 2], t.s[i / 2]);
        if (l.on1)
#pragma unroll
            for (int i = 0; i < V; i += 2) rotate_pair(y[i], y[i + 1], t.c[V / 2 + i / 2], t.s[V / 2 + i / 2]);
    } else if (l.on0) {
#pragma unroll
        for (int i = 0; i < V; ++i) rotate_pair(x[i], y[i], t.c[i], t.s[i]);
    }
}

constexpr int kRotaryRows = 4;  // pairs of pieces of a token that a lane has in flight

// One token's rows of `heads` heads by one warp: x and out point at its first head.  `row`: the position's table row.
// WIDE: the lanes of a row divide the warp, so that a lane has the same pairs in every head.
template <typename T, bool WIDE>
__device__ __forceinline__ void rotate_heads(const RotaryTable& r, const float* row, bool transpose, const T* x, int64_t x_head,
                                             T* out, int64_t out_head, int heads, int d) {
    using E = Elem<T>;
    constexpr int V = E::V;
    const int lane = threadIdx.x & 31, pieces = d / V, per = pieces / 2, items = heads * per;
    RotaryLane<V> l(r, lane % per, pieces);
    RotaryAngles<V> t;
    if constexpr (WIDE) t.load(r, l, row, transpose);
    const bool same = x == out;
    for (int i0 = lane; i0 < items; i0 += 32 * kRotaryRows) {
        uint4 raw[kRotaryRows][2];
#pragma unroll
        for (int k = 0; k < kRotaryRows; ++k) {
            const int i = i0 + 32 * k, h = i / per;
            if constexpr (!WIDE) l = RotaryLane<V>(r, i % per, pieces);
            raw[k][0] = raw[k][1] = make_uint4(0, 0, 0, 0);
            if (i < items) {
                const T* p = x + h * x_head;
                if (l.on0 || !same) raw[k][0] = *reinterpret_cast<const uint4*>(p + l.c0 * V);
                if (l.on1 || !same) raw[k][1] = *reinterpret_cast<const uint4*>(p + l.c1 * V);
            }
        }
#pragma unroll
        for (int k = 0; k < kRotaryRows; ++k) {
            const int i = i0 + 32 * k, h = i / per;
            if (i >= items) break;
            if constexpr (!WIDE) {
                l = RotaryLane<V>(r, i % per, pieces);
                t.load(r, l, row, transpose);
            }
            T* p = out + h * out_head;
            if (l.on0 || l.on1) {
                float a[V], b[V];
                E::get(raw[k][0], a);
                E::get(raw[k][1], b);
                rotate_pieces<V>(r, l, t, a, b);
                if (l.on0) raw[k][0] = E::put(a);
                if (l.on1) raw[k][1] = E::put(b);
            }
            if (l.on0 || !same) *reinterpret_cast<uint4*>(p + l.c0 * V) = raw[k][0];
            if (l.on1 || !same) *reinterpret_cast<uint4*>(p + l.c1 * V) = raw[k][1];
        }
    }
}

}  // namespace
}  // namespace tq
