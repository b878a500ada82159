// Appending to the 8-bit paged cache with the position rotation on the way:
// keys are rotated in fp32 registers and quantised from there (by the rule of the
// plain write: the block's least power-of-two scale, or its present one where that is
// larger), values are quantised as they are, and the step's queries are rotated by the
// same launch.
//
// Against rotating first and writing after, the keys are read once and not written in
// between, and not rounded to their 16-bit type before they are rounded to e4m3.  The
// floor is the rows in (2 T hkv d elements, T hq d of queries), the codes and the
// rotated queries out, and a table row of 4 rot bytes a position.
//
// One warp owns 16 tokens of one (block, head, side), a whole block goes to neighbouring
// warps of one CTA; CTAs behind those take the queries, a warp one token and 16 heads.
#include <cuda_runtime.h>

#include "tq_fp8_rows.cuh"
#include "tq_rotary.cuh"

namespace tq {
namespace {

constexpr int kAppendHeads = 16;  // query heads of a warp

template <typename T>
__device__ __forceinline__ void append_queries(const Fp8AppendArgs& a, int64_t item) {
    const int parts = (a.hq + kAppendHeads - 1) / kAppendHeads;
    const int64_t token = item / parts;
    if (token >= a.b.num_tokens) return;
    const Fp8Seq s = fp8_seq_of_unit(a.b, token, 1, 0);
    const int64_t i = token - s.row0;
    if (i < 0 || i >= s.n || s.start < 0) return;  // (a negative start: its rows are not touched)
    const int64_t p = a.positions ? (int64_t)__ldg(a.positions + token) : (int64_t)s.start + i;
    if (p < 0 || p >= a.r.positions) {
        if ((threadIdx.x & 31) == 0) flag(a.status, TQ_FLAG_BAD_SLOT);
        return;
    }
    const int h0 = (int)(item - token * parts) * kAppendHeads;
    rotate_heads<T, true>(a.r, a.r.table + p * a.r.rot, false, static_cast<const T*>(a.q) + token * a.q_token + h0 * a.q_head, a.q_head,
                          static_cast<T*>(a.q_out) + token * a.out_token + h0 * a.out_head, a.out_head, min(kAppendHeads, a.hq - h0),
                          kHeadDim);
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32, 2) fp8_append_kernel(const Fp8AppendArgs a, int wpb_shift, int64_t kv_grid) {
    using E = Elem<T>;
    constexpr int V = E::V, P = kHeadDim / V, LPR = P / 2, RPI = 32 / LPR, IT = kRows / RPI;
    __shared__ float tops[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    if (blockIdx.x >= kv_grid) {
        append_queries<T>(a, ((int64_t)blockIdx.x - kv_grid) * kWarps + warp);
        return;
    }
    const Place p = find_place(a.g, a.b, (int64_t)blockIdx.x * kWarps + warp, wpb_shift, a.status);
    const int sub = lane / LPR;
    const RotaryLane<V> l(a.r, lane % LPR, P);
    const int64_t step = p.side ? a.v_token : a.k_token;
    const T* src = static_cast<const T*>(p.side ? a.V : a.K) + p.row0 * step + p.head * (p.side ? a.v_head : a.k_head);
    // the rows are on their way before the block's id is looked at
    uint4 raw[IT][2];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int r = i * RPI + sub, t = p.first + r;
        raw[i][0] = raw[i][1] = make_uint4(0, 0, 0, 0);
        if (t >= p.lo && t < p.hi) {
            raw[i][0] = __ldcs(reinterpret_cast<const uint4*>(src + r * step + l.c0 * V));
            raw[i][1] = __ldcs(reinterpret_cast<const uint4*>(src + r * step + l.c1 * V));
        }
    }
    int64_t page = 0;
    const bool there = page_of(a.g, p, a.status, page);
    // the block's scale as earlier tokens left it
    const int e_old = there && p.lo > 0 ? fp8_exp_of(a.g.scales[page]) : kFp8MinExp;
    float x[IT][2][V];
    float top = 0.f;
    bool odd = false;  // an inf or a NaN among the new rows: the maximum of the others
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int r = i * RPI + sub, t = p.first + r;
        E::get(raw[i][0], x[i][0]);
        E::get(raw[i][1], x[i][1]);
        if (p.side == 0 && t >= p.lo && t < p.hi) {
            const int64_t row = p.row0 + r;
            // (row0 counts from the warp's first token: start + (row - cu) is the position)
            const int64_t at = a.positions ? (int64_t)__ldg(a.positions + row) : p.pos + r;
            if (at >= 0 && at < a.r.positions) {
                RotaryAngles<V> ang;
                ang.load(a.r, l, a.r.table + at * a.r.rot, false);
                rotate_pieces<V>(a.r, l, ang, x[i][0], x[i][1]);
            } else {
                flag(a.status, TQ_FLAG_BAD_SLOT);
#pragma unroll
                for (int k = 0; k < V; ++k) x[i][0][k] = x[i][1][k] = 0.f;
            }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const bool fin = finite(x[i][s][k]);
                odd |= !fin;
                top = fmaxf(top, fin ? fabsf(x[i][s][k]) : 0.f);
            }
    }
    top = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top)));  // magnitudes order as their bits do
    if (__any_sync(0xFFFFFFFFu, odd) && lane == 0) flag(a.status, TQ_FLAG_NONFINITE);
    if (wpb_shift) {  // the block's warps are neighbours of one CTA
        if (lane == 0) tops[warp] = top;
        __syncthreads();
        for (int w = 0; w < 1 << wpb_shift; ++w) top = fmaxf(top, tops[(warp >> wpb_shift << wpb_shift) + w]);
    }
    if (!there) return;
    const int e = max(fp8_exponent(top), e_old);
    if (p.first == 0 && lane == 0) a.g.scales[page] = fp8_pow2(e);
    const float inv = fp8_pow2(-e);
    uint8_t* dst = a.g.pool + page * ((int64_t)a.g.bs * kHeadDim) + (int64_t)p.first * kHeadDim;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int r = i * RPI + sub, t = p.first + r;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            uint32_t w[V / 4];
#pragma unroll
            for (int k = 0; k < V; k += 4) {
                float y[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    y[n] = x[i][s][k + n] * inv;
                    y[n] = y[n] != y[n] ? 0.f : y[n];  // NaN is stored as 0
                }
                w[k / 4] = fp8_cvt2(y[0], y[1]) | (fp8_cvt2(y[2], y[3]) << 16);
            }
            if (t >= p.lo && t < p.hi) {
                uint8_t* to = dst + r * kHeadDim + (s ? l.c1 : l.c0) * V;
                if constexpr (V == 8) *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[V / 4 - 1]);
                else *reinterpret_cast<uint32_t*>(to) = w[0];
            }
        }
    }
    if (p.lo > p.first && e > e_old) move_codes(a.g.pool + page * ((int64_t)a.g.bs * kHeadDim) + (int64_t)p.first * kHeadDim,
                                                min(p.lo - p.first, kRows), e_old - e);
}

template <typename T>
int launch(const Fp8AppendArgs& a, cudaStream_t s) {
    const int64_t kv = fp8_row_grid(a.g, a.b);
    const int64_t q = a.q ? (a.b.num_tokens * ((a.hq + kAppendHeads - 1) / kAppendHeads) + kWarps - 1) / kWarps : 0;
    return (int)launch_programmatic(fp8_append_kernel<T>, dim3((unsigned)(kv + q)), dim3(kWarps * 32), 0, s, a, a.g.bs_shift - 4, kv);
}

}  // namespace

bool fp8_append_counts(const Fp8Geometry& g, const Fp8Batch& b, int hq) {
    return fp8_rows_count(g, b) && b.num_tokens * ((hq + kAppendHeads - 1) / kAppendHeads) / kWarps < (1 << 28);
}

int launch_fp8_append(const Fp8AppendArgs& a, void* stream) {
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (a.dtype == TQ_F32) return launch<float>(a, s);
    return a.dtype == TQ_BF16 ? launch<__nv_bfloat16>(a, s) : launch<__half>(a, s);
}

}  // namespace tq
