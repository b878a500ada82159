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
// A warp owns 16 tokens of one (block, head), keys and values, a whole block goes to
// neighbouring warps of one CTA.  One CTA an SM goes through a run of them, so that the
// rows of the next item are on their way while this one's are worked on, and what the
// heads of a block share is looked up once.  CTAs behind those take the queries, a warp
// one token and 16 heads.
#include <cuda_runtime.h>

#include <type_traits>

#include "tq_fp8_rows.cuh"
#include "tq_rotary.cuh"

namespace tq {
namespace {

constexpr int kAppendHeads = 16;   // query heads of a warp
constexpr int kAppendWarps = 16;

template <typename T, bool INTER>
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
    rotate_heads<T, INTER, true, 4>(a.r, a.r.table + p * a.r.rot, false, static_cast<const T*>(a.q) + token * a.q_token + h0 * a.q_head, a.q_head,
                          static_cast<T*>(a.q_out) + token * a.out_token + h0 * a.out_head, a.out_head, min(kAppendHeads, a.hq - h0),
                          kHeadDim);
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN where either is one
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ void copy_async(uint32_t smem, const void* p, bool in) {  // 16 bytes, or zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(p), "r"(in ? 16 : 0) : "memory");
}

// V neighbouring fp32 values to codes.  ODD: an infinity or a NaN may be among them; NaN is stored as 0.
template <int V, bool ODD>
__device__ __forceinline__ void store_codes(uint8_t* to, const uint64_t (&x)[V / 2], float inv) {
    const uint64_t i2 = f2_pack(inv, inv);
    uint32_t o[V / 4];
#pragma unroll
    for (int k = 0; k < V / 4; ++k) {
        float u[4];
        f2_unpack(f2_mul(x[2 * k], i2), u[0], u[1]);
        f2_unpack(f2_mul(x[2 * k + 1], i2), u[2], u[3]);
        if constexpr (ODD)
#pragma unroll
            for (int n = 0; n < 4; ++n) u[n] = u[n] != u[n] ? 0.f : u[n];
        o[k] = fp8_cvt2(u[0], u[1]) | (fp8_cvt2(u[2], u[3]) << 16);
    }
    if constexpr (V == 8) *reinterpret_cast<uint2*>(to) = make_uint2(o[0], o[V / 4 - 1]);
    else *reinterpret_cast<uint32_t*>(to) = o[0];
}

// Shared memory of a warp, rows in the type they came in: keys, whose place is free once they are rotated, and two places
// of values.
template <typename T>
constexpr int kStageBytes = kRows * kHeadDim * (int)sizeof(T);
template <typename T>
constexpr int kAppendCtaWarps = sizeof(T) == 4 ? kAppendWarps / 2 : kAppendWarps;  // (fp32 rows: 8 warps, 192 KB all the same)

// What bounds it is instructions as much as bytes (a rotated and coded element is 8 of them).  32K x 8 heads of bf16: a
// warp a side and an item, two CTAs an SM, 87 us; keys rotated a second time instead of held in registers, three CTAs an
// SM, 62; a warp for both sides 56, all of these without the next item's rows on their way; with them 40 (4.6 TB/s, issue
// active 36 % with 16 warps an SM; the codes of 33 MB stay in L2).  fp32 rows, 8 warps of 156 registers: 70, 0.76 of the
// copy's rate.  With the queries of 64 heads 230, of 32 136: CTAs of queries have an SM to themselves, one at a time, as the
// launch gives them the others' shared memory; a call without queries and one of the rotation take 220 and 133.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kAppendCtaWarps<T> * 32, 1) fp8_append_kernel(const Fp8AppendArgs a, int wpb_shift, uint32_t items, uint32_t kv_grid) {
    using E = Elem<T>;
    constexpr int V = E::V, P = kHeadDim / V, LPR = P / 2, RPI = 32 / LPR, IT = kRows / RPI, W = kAppendCtaWarps<T>;
    extern __shared__ uint4 staged[];  // [warps][3][16 rows][P]
    __shared__ uint32_t tops[2][2][W];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    if (blockIdx.x >= kv_grid) {
        append_queries<T, INTER>(a, ((int64_t)blockIdx.x - kv_grid) * W + warp);
        return;
    }
    // this group of warps' run of items (unit, head), and its warp's tokens of every block
    const int group = warp >> wpb_shift, groups = W >> wpb_shift, first = (warp & ((1 << wpb_shift) - 1)) * kRows;
    const uint64_t g0 = (uint64_t)blockIdx.x * groups + group, all = (uint64_t)kv_grid * groups;
    const uint32_t i0 = (uint32_t)(items * g0 / all), i1 = (uint32_t)(items * (g0 + 1) / all);
    const int sub = lane / LPR;
    const RotaryLane<V, INTER> l(a.r, lane % LPR, P);
    uint4* const mine = staged + warp * (3 * kRows * P);
    // The next item: its block's place, and of the rows the positions (lane r holds row r's; -1: not a new row, or one
    // outside the table, whose key is a row of zeros).
    Place p;
    uint32_t unit = 0xFFFFFFFFu;
    int at = -1;
    unsigned kin = 0, vin = 0;
    auto look_up = [&](uint32_t item) {
        const uint32_t u = item / (uint32_t)a.g.hkv;
        if (u != unit) {
            unit = u;
            p = place_of_unit(a.g, a.b, u, first, a.status);
            const int t = first + (lane & 15);
            const bool in = t >= p.lo && t < p.hi;
            at = -1;
            if (in) {
                const int64_t pos = a.positions ? (int64_t)__ldg(a.positions + p.row0 + (lane & 15)) : p.pos + (lane & 15);
                if (pos >= 0 && pos < a.r.positions) at = (int)pos;
                else flag(a.status, TQ_FLAG_BAD_SLOT);
            }
            kin = __ballot_sync(0xFFFFFFFFu, at >= 0);
            vin = __ballot_sync(0xFFFFFFFFu, in);
            at = max(at, 0);
        }
        p.head = (int)(item - u * (uint32_t)a.g.hkv);
    };
    auto issue = [&](int buffer) {  // the rows (rows of zeros: nothing is read)
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            constexpr int RPC = 32 / P;  // rows of a warp's copy
            const int64_t step = side ? a.v_token : a.k_token;
            const T* src = static_cast<const T*>(side ? a.V : a.K) + (p.row0 + lane / P) * step + p.head * (side ? a.v_head : a.k_head) +
                           (lane % P) * V;
            const uint32_t to = smem_u32(mine + (side ? 1 + buffer : 0) * kRows * P + lane);
            const unsigned in = side ? vin : kin;
            if (in == 0xFFFFFFFFu) {
#pragma unroll
                for (int i = 0; i < kRows / RPC; ++i) {
                    copy_async(to + i * 512, src, true);
                    src += RPC * step;
                }
            } else {
#pragma unroll
                for (int i = 0; i < kRows / RPC; ++i) {
                    const bool on = (in >> (i * RPC + lane / P)) & 1;
                    copy_async(to + i * 512, on ? src : a.K, on);
                    src += RPC * step;
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    // the largest finite magnitude of a row, where there is an infinity or a NaN
    auto finite_top = [&](const RotaryPieces<V>& w, float m) {
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
            float u[4];
            f2_unpack(w.x[k], u[0], u[1]);
            f2_unpack(w.y[k], u[2], u[3]);
            for (int n = 0; n < 4; ++n) m = fmaxf(m, finite(u[n]) ? fabsf(u[n]) : 0.f);
        }
        return m;
    };
    if (i0 < i1) {
        look_up(i0);
        issue(0);
    }
    for (uint32_t item = i0; item < i1; ++item) {
        const int buffer = (item - i0) & 1;
        const uint4* const keys = mine + sub * P;
        const uint4* const values = mine + ((1 + buffer) * kRows + sub) * P;
        auto value = [&](int i, RotaryPieces<V>& w) { w.template get<E>(values[i * RPI * P + l.c0], values[i * RPI * P + l.c1]); };
        int64_t page = 0;
        const bool there = page_of(a.g, p, a.status, page);
        const int held = p.lo;  // the block holds that many earlier positions of the sequence
        const unsigned rows = vin;
        // the block's scales as they left them
        float2 old = make_float2(0.f, 0.f);
        if (there && held > 0) old = *reinterpret_cast<const float2*>(a.g.scales + page);
        // ---- the block's maxima: magnitudes order as their bits do, infinities and NaN above all ----
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        RotaryPieces<V> key[IT];
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            RotaryAngles<V, INTER> t;
            t.load(a.r, l, a.r.table + (int64_t)__shfl_sync(0xFFFFFFFFu, at, i * RPI + sub) * a.r.rot);
            key[i].template get<E>(keys[i * RPI * P + l.c0], keys[i * RPI * P + l.c1]);
            t.rotate(l, key[i]);
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
                float u, v;
                f2_unpack(key[i].x[k], u, v);
                m = max_nan(max_nan(m, fabsf(u)), fabsf(v));
                f2_unpack(key[i].y[k], u, v);
                m = max_nan(max_nan(m, fabsf(u)), fabsf(v));
            }
        }
        // the keys' place and the other values' are free: the next item's rows
        __syncwarp();
        if (item + 1 < i1) {
            look_up(item + 1);
            issue(buffer ^ 1);
        } else {
            asm volatile("cp.async.commit_group;\n\tcp.async.commit_group;" ::: "memory");
        }
        uint32_t ktop = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m));
        const bool kodd = ktop >= 0x7F800000u;
        if (kodd) {
            m = 0.f;
#pragma unroll
            for (int i = 0; i < IT; ++i) m = finite_top(key[i], m);
            ktop = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m));
        }
        asm volatile("cp.async.wait_group 2;" ::: "memory");
        __syncwarp();
        uint32_t vm = 0;
#pragma unroll
        for (int i = 0; i < IT; ++i) vm = E::top(values[i * RPI * P + l.c1], E::top(values[i * RPI * P + l.c0], vm));
        vm = __reduce_max_sync(0xFFFFFFFFu, E::join(vm));
        const bool vodd = vm >= E::kInf;
        uint32_t vtop = __float_as_uint(E::value(vm));
        if (vodd) {
            m = 0.f;
#pragma unroll 1
            for (int i = 0; i < IT; ++i) {
                RotaryPieces<V> w;
                value(i, w);
                m = finite_top(w, m);
            }
            vtop = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m));
        }
        if ((kodd || vodd) && lane == 0) flag(a.status, TQ_FLAG_NONFINITE);
        if (wpb_shift) {  // the block's warps, on a barrier of their own
            if (lane == 0) {
                tops[buffer][0][warp] = ktop;
                tops[buffer][1][warp] = vtop;
            }
            asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 << wpb_shift) : "memory");
            for (int w = 0; w < 1 << wpb_shift; ++w) {
                ktop = max(ktop, tops[buffer][0][(group << wpb_shift) + w]);
                vtop = max(vtop, tops[buffer][1][(group << wpb_shift) + w]);
            }
        }
        if (!there) continue;  // (the same in all the block's warps)
        // ---- the codes ----
        const int ke_old = held > 0 ? fp8_exp_of(old.x) : kFp8MinExp, ve_old = held > 0 ? fp8_exp_of(old.y) : kFp8MinExp;
        const int ke = max(fp8_exponent(__uint_as_float(ktop)), ke_old), ve = max(fp8_exponent(__uint_as_float(vtop)), ve_old);
        if (first == 0 && lane == 0) *reinterpret_cast<float2*>(a.g.scales + page) = make_float2(fp8_pow2(ke), fp8_pow2(ve));
        const int64_t side = (int64_t)a.g.bs * kHeadDim;
        uint8_t* const kdst = a.g.pool + page * side + (int64_t)first * kHeadDim;
        const float kinv = fp8_pow2(-ke), vinv = fp8_pow2(-ve);
        auto codes = [&](auto odd) {
            uint8_t* to = kdst + sub * kHeadDim;
            unsigned in = rows >> sub;
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                RotaryPieces<V> w;
                value(i, w);
                if (in & 1) {
                    store_codes<V, odd.value>(to + l.c0 * V, key[i].x, kinv);
                    store_codes<V, odd.value>(to + l.c1 * V, key[i].y, kinv);
                    store_codes<V, odd.value>(to + side + l.c0 * V, w.x, vinv);
                    store_codes<V, odd.value>(to + side + l.c1 * V, w.y, vinv);
                }
                in >>= RPI;
                to += RPI * kHeadDim;
            }
        };
        if (kodd || vodd) codes(std::true_type{});
        else codes(std::false_type{});
        if (held > first) {  // earlier rows move to a larger scale
            if (ke > ke_old) move_codes(kdst, min(held - first, kRows), ke_old - ke);
            if (ve > ve_old) move_codes(kdst + side, min(held - first, kRows), ve_old - ve);
        }
        __syncwarp();  // (the values' place is written again two items on)
    }
}

// Items (unit, head) of a launch.
int64_t append_items(const Fp8Geometry& g, const Fp8Batch& b) { return fp8_units(b.num_tokens, b.batch, g.bs, 2) * g.hkv; }

template <typename T, bool INTER>
int launch(const Fp8AppendArgs& a, cudaStream_t s) {
    auto kern = fp8_append_kernel<T, INTER>;
    constexpr int W = kAppendCtaWarps<T>, smem = W * 3 * kStageBytes<T>;
    static int done[64] = {};
    const cudaError_t e = ensure_smem_limit(kern, smem, done);
    if (e != cudaSuccess) return (int)e;
    const int shift = a.g.bs_shift - 4;
    const int64_t items = append_items(a.g, a.b), ctas = (items + (W >> shift) - 1) / (W >> shift);
    const int64_t kv = ctas < a.g.num_sms ? ctas : a.g.num_sms;
    const int64_t q = a.q ? (a.b.num_tokens * ((a.hq + kAppendHeads - 1) / kAppendHeads) + W - 1) / W : 0;
    return (int)launch_programmatic(kern, dim3((unsigned)(kv + q)), dim3(W * 32), (size_t)smem, s, a, shift, (uint32_t)items, (uint32_t)kv);
}
template <typename T>
int launch(const Fp8AppendArgs& a, cudaStream_t s) {
    return a.r.interleaved ? launch<T, true>(a, s) : launch<T, false>(a, s);
}

}  // namespace

bool fp8_append_counts(const Fp8Geometry& g, const Fp8Batch& b, int hq) {
    return append_items(g, b) < (1 << 30) && b.num_tokens * ((hq + kAppendHeads - 1) / kAppendHeads) < (1 << 30);
}

int launch_fp8_append(const Fp8AppendArgs& a, void* stream) {
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (a.dtype == TQ_F32) return launch<float>(a, s);
    return a.dtype == TQ_BF16 ? launch<__nv_bfloat16>(a, s) : launch<__half>(a, s);
}

}  // namespace tq
