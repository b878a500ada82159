// Rotary positions on pieces of a row.
//
// A head's first `rot` dims are pairs (a, b), rotated by the position's angles:
//   a' = a c - b s,   b' = b c + a s,   c = m cos(p f_j), s = m sin(p f_j),
// with c and s from a table that was computed in 64 bits (an angle of position 10^5 in 32 bits is off by 2^-7).
// Products and sums are rounded one by one, so that the result does not depend on how a compiler contracts them
// and a rotated key has the same codes wherever it is rotated.
#pragma once

#include "tq_device.cuh"
#include "tq_elem.cuh"
#include "tq_rotary.h"

namespace tq {
namespace {

// A lane's two 16-byte pieces of a row of `pieces` pieces, of V elements each: lane l of the pieces / 2 that share a row.
// In the half layout piece j meets its partner j + rot / 2 in one lane; everything else goes in the row's order.
template <int V, bool INTER>
struct RotaryLane {
    int c0, c1;    // the pieces
    int at, at1;   // where the cosines of their pairs start (half layout: of both at `at`)
    bool on0, on1; // whether they are rotated
    __device__ __forceinline__ RotaryLane(const RotaryTable& r, int l, int pieces) {
        if constexpr (INTER) {
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

// Two pieces as pairs of neighbouring elements, for the two-wide fp32 instructions.
template <int V>
struct RotaryPieces {
    uint64_t x[V / 2], y[V / 2];
    template <typename E>
    __device__ __forceinline__ void get(const uint4& a, const uint4& b) {
        float u[V], v[V];
        E::get(a, u);
        E::get(b, v);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            x[i] = f2_pack(u[2 * i], u[2 * i + 1]);
            y[i] = f2_pack(v[2 * i], v[2 * i + 1]);
        }
    }
};

// The cosines and sines of a lane's pairs at one position, V of each: of the one set that both pieces share (half layout),
// or of the first piece's pairs and then the second's.
template <int V, bool INTER>
struct RotaryAngles {
    uint64_t c[V / 2], s[V / 2];
    __device__ __forceinline__ void load(const RotaryTable& r, const RotaryLane<V, INTER>& l, const float* row) {
        const float* sines = row + r.rot / 2;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) c[i] = s[i] = 0;
        if constexpr (INTER) {
            if (l.on0) get<V / 4>(row + l.at, c), get<V / 4>(sines + l.at, s);
            if (l.on1) get<V / 4>(row + l.at1, c + V / 4), get<V / 4>(sines + l.at1, s + V / 4);
        } else if (l.on0) {
            get<V / 2>(row + l.at, c);
            get<V / 2>(sines + l.at, s);
        }
    }
    __device__ __forceinline__ void transpose() {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) s[i] ^= 0x8000000080000000ull;
    }
    __device__ __forceinline__ void rotate(const RotaryLane<V, INTER>& l, RotaryPieces<V>& p) const {
        if constexpr (INTER) {
            if (l.on0) turn(p.x, 0);
            if (l.on1) turn(p.y, V / 2);
        } else if (l.on0) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const uint64_t x = p.x[i], y = p.y[i];
                p.x[i] = sum<-1>(f2_mul(x, c[i]), f2_mul(y, s[i]));
                p.y[i] = sum<1>(f2_mul(y, c[i]), f2_mul(x, s[i]));
            }
        }
    }

  private:
    // (a two-wide sum of two-wide products gets contracted, the products' roundings with it; this one does not)
    template <int SIGN>
    static __device__ __forceinline__ uint64_t sum(uint64_t a, uint64_t b) {
        float u[2], v[2];
        f2_unpack(a, u[0], u[1]);
        f2_unpack(b, v[0], v[1]);
        return SIGN < 0 ? f2_pack(__fsub_rn(u[0], v[0]), __fsub_rn(u[1], v[1])) : f2_pack(__fadd_rn(u[0], v[0]), __fadd_rn(u[1], v[1]));
    }
    template <int N>
    static __device__ __forceinline__ void get(const float* p, uint64_t* to) {
        if constexpr (N >= 2) {
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const ulonglong2 a = __ldg(reinterpret_cast<const ulonglong2*>(p + 2 * i));
                to[i] = a.x;
                to[i + 1] = a.y;
            }
        } else {
            to[0] = __ldg(reinterpret_cast<const unsigned long long*>(p));
        }
    }
    // pairs (a, b) of one piece, whose angles start at `from`: (a c, b c) + (b (-s), a s)
    __device__ __forceinline__ void turn(uint64_t (&p)[V / 2], int from) const {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            float a, b, c2[2], s2[2];
            f2_unpack(p[i], a, b);
            f2_unpack(c[(from + i) / 2], c2[0], c2[1]);
            f2_unpack(s[(from + i) / 2], s2[0], s2[1]);
            const float cc = c2[i % 2], ss = s2[i % 2];
            p[i] = sum<1>(f2_mul(p[i], f2_pack(cc, cc)), f2_mul(f2_pack(b, a), f2_pack(-ss, ss)));
        }
    }
};

// One token's rows of `heads` heads by one warp: x and out point at its first head.  `row`: the position's table row.
// WIDE: the lanes of a row divide the warp, so that a lane has the same pairs in every head.  ROWS: pairs of pieces that a
// lane has in flight.
template <typename T, bool INTER, bool WIDE, int ROWS>
__device__ __forceinline__ void rotate_heads(const RotaryTable& r, const float* row, bool transpose, const T* x, int64_t x_head,
                                             T* out, int64_t out_head, int heads, int d) {
    using E = Elem<T>;
    constexpr int V = E::V;
    const int lane = threadIdx.x & 31, pieces = d / V, per = pieces / 2;
    const bool same = x == out;
    RotaryAngles<V, INTER> t;
    auto angles = [&](const RotaryLane<V, INTER>& l) {
        t.load(r, l, row);
        if (transpose) t.transpose();
    };
    auto load = [&](const RotaryLane<V, INTER>& l, const T* p, uint4 (&raw)[2]) {
        if (l.on0 || !same) raw[0] = __ldcs(reinterpret_cast<const uint4*>(p + l.c0 * V));
        if (l.on1 || !same) raw[1] = __ldcs(reinterpret_cast<const uint4*>(p + l.c1 * V));
    };
    auto store = [&](const RotaryLane<V, INTER>& l, T* p, uint4 (&raw)[2]) {
        if (l.on0 || l.on1) {
            RotaryPieces<V> w;
            w.template get<E>(raw[0], raw[1]);
            t.rotate(l, w);
            float a[V], b[V];
#pragma unroll
            for (int n = 0; n < V / 2; ++n) {
                f2_unpack(w.x[n], a[2 * n], a[2 * n + 1]);
                f2_unpack(w.y[n], b[2 * n], b[2 * n + 1]);
            }
            if (l.on0) raw[0] = E::put(a);
            if (l.on1) raw[1] = E::put(b);
        }
        if (l.on0 || !same) __stcs(reinterpret_cast<uint4*>(p + l.c0 * V), raw[0]);
        if (l.on1 || !same) __stcs(reinterpret_cast<uint4*>(p + l.c1 * V), raw[1]);
    };
    if constexpr (WIDE) {
        const RotaryLane<V, INTER> l(r, lane % per, pieces);
        const int step = 32 / per;  // heads of a warp's step
        angles(l);
        int h = lane / per;
        x += h * x_head;
        out += h * out_head;
        for (; h < heads; h += ROWS * step) {
            uint4 raw[ROWS][2];
#pragma unroll
            for (int k = 0; k < ROWS; ++k)
                if (h + k * step < heads) load(l, x + k * step * x_head, raw[k]);
#pragma unroll
            for (int k = 0; k < ROWS; ++k)
                if (h + k * step < heads) store(l, out + k * step * out_head, raw[k]);
            x += ROWS * step * x_head;
            out += ROWS * step * out_head;
        }
    } else {
        for (int i = lane; i < heads * per; i += 32) {
            const int h = i / per;
            const RotaryLane<V, INTER> l(r, i - h * per, pieces);
            uint4 raw[2];
            load(l, x + h * x_head, raw);
            angles(l);
            store(l, out + h * out_head, raw);
        }
    }
}

}  // namespace
}  // namespace tq
