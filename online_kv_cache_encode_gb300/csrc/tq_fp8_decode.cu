// Attention of one query token per sequence over the 8-bit paged cache, on the
// fp8 tensor cores.
//
// The codes go from the pool to the tensor cores as they are.  For a tile of
// 256 tokens of one KV head and up to 16 of its query heads (GP of them):
//   S^T [tokens x N] = K . Q^T      K: codes, token rows of 128 bytes (K-major)
//   O^T [128 dims x N] = V^T . P^T  V: the same rows read MN-major
// with fp8 operands, fp32 accumulation.  A query row and a softmax weight are
// split into NT terms of e4m3, x = h1 + h2 / 16 + h3 / 256, each a column of its
// own (N = NT * GP, padded to 16), so nothing shares a range with anything:
// 2 terms hold a bf16 query exactly (8 significant bits, to 2^-22 of the row's
// largest element) and a weight to 2^-8, the rounding of a bf16 output; fp16
// takes 3 terms, 2^-12.  Each tile's weights are exponentials against the
// tile's own maximum, so the tokens behind one that dominates a long context
// keep their relative precision; the tile's output leaves tensor memory and is
// joined in fp32 registers against the running maximum.  Key scales multiply
// the scores, value scales the weights (both powers of two).
//
// What bounds it is the cache's bytes: the tensor work of a tile is about 500
// cycles and its softmax about as much, against 2850 cycles that HBM needs for
// its 64 KB on one of 152 SMs.  Hence one CTA per SM, a ring of three 64 KB
// stages filled by TMA (pages land in the 128-byte swizzle that both readings
// of a row share), and the flat list of all (sequence, head, tile) cut into
// equal runs, whatever the lengths are.  An item (sequence, head) that lies in
// one run is written directly; otherwise each run leaves a partial (max, sum,
// accumulator) and the last run to arrive joins them in their order, so results
// do not depend on timing.
//
// Warps: 0-7 softmax and accumulation (thread = token of the tile for the
// scores, = dim for the output, the two warpgroups taking half of the columns
// each), 8 TMA, 9 MMA, 10 queries, 11 scales.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <type_traits>

#include "tq_fp8.cuh"
#include "tq_tcgen05.cuh"

namespace tq {
namespace {

constexpr int kTile = 256;            // tokens of a tile
constexpr int kStages = 3;
constexpr int kSide = kTile * kHeadDim;   // bytes of a tile's keys (or values)
constexpr int kPagesMax = kTile / 16;
constexpr int kDecWarps = 12;
constexpr int kDecThreads = kDecWarps * 32;
constexpr float kPScale = 256.f;      // weights are coded as p * 2^8 <= 256

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
// Rows of 128 bytes in the 128-byte swizzle read MN-major: 8-row groups 1 KB apart along K.
__device__ __forceinline__ uint64_t desc_sw128_mn(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (64ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* map, int row, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(map), "r"(0), "r"(row), "r"(bar)
        : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Floats in the order of signed integers.
__device__ __forceinline__ int order_key(float x) {
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float order_val(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7FFFFFFF)); }

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
__device__ __forceinline__ void soft_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Reduces C values of every lane over the warp; lane l gets the result of value l % C.
template <int C, bool MAX>
__device__ __forceinline__ float reduce_lanes(float (&v)[C]) {
    const int lane = threadIdx.x & 31;
    auto op = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
#pragma unroll
    for (int w = C / 2; w >= 1; w /= 2) {  // halve the values, keep those of this lane's half
        const bool up = lane & w;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float mine = up ? v[i + w] : v[i], other = up ? v[i] : v[i + w];
            v[i] = op(mine, __shfl_xor_sync(0xFFFFFFFFu, other, w));
        }
    }
    float x = v[0];
#pragma unroll
    for (int w = C; w < 32; w *= 2) x = op(x, __shfl_xor_sync(0xFFFFFFFFu, x, w));
    return x;
}

// A run of tiles in the flat list (sequence, head part, tile).
struct Walk {
    int b, hs, ti, nt, len;
};

template <int NT, int GP>
struct DecLayout {
    static constexpr int N = (NT * GP + 15) / 16 * 16;
    static constexpr int QB = N <= 32 ? 2 : 1;              // query buffers
    static constexpr int p_bytes = N / 16 * kTile * 16;     // one weight buffer: planes of [token][16 columns]
    static constexpr int q_bytes = N * kHeadDim;
    static constexpr int p = kStages * 2 * kSide;
    static constexpr int q = p + 2 * p_bytes;
    static constexpr int meta = q + QB * q_bytes;           // per stage: key scales, relative value scales [16 each]
    static constexpr int okm = meta + kStages * 2 * kPagesMax * 4;  // per stage: pages there, largest value exponent
    static constexpr int mult = okm + kStages * 8;          // per query buffer: [GP]
    static constexpr int top = mult + QB * GP * 4;          // [3][GP] maxima as ordered ints
    static constexpr int sums = top + 3 * GP * 4;           // [8 warps][GP]
    static constexpr int bars = (sums + 8 * GP * 4 + 7) / 8 * 8;
    static constexpr int nbars = 2 * kStages + 6 + 2 * QB + 1;
    static constexpr int misc = bars + 8 * nbars;           // tmem address, last-arrival word
    static constexpr int total = misc + 16;
    static constexpr int smem = total + 1024;               // the base is rounded up to 1 KB
    static constexpr int tmem = 6 * N <= 128 ? 128 : 6 * N <= 256 ? 256 : 512;
    static_assert(smem <= kSmemLimit, "decode does not fit in shared memory");
};

constexpr int kPartFloats = 16 * kHeadDim + 32;  // a partial: accumulators [GP][128], (max, sum) [GP]

struct DecArgs {
    Fp8AttnArgs a;
    int nsub;             // parts of GP query heads per KV head
    unsigned* counters;   // [batch * hkv * nsub]
    float* partials;      // [grid][2][kPartFloats]
    long long stall_cycles;
};

template <typename T, int NT, int GP>
__global__ void __launch_bounds__(kDecThreads, 1)
fp8_decode_kernel(const DecArgs A, const __grid_constant__ CUtensorMap map) {
    using L = DecLayout<NT, GP>;
    constexpr int N = L::N;
    extern __shared__ uint8_t raw[];
    uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(sm);
    const Fp8Geometry& g = A.a.g;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto bar = [&](int i) { return sb + L::bars + 8 * i; };
    constexpr int bFull = 0, bEmpty = kStages, bS = 2 * kStages, bP = bS + 2, bO = bP + 2, bQ = bO + 2, bQe = bQ + L::QB,
                  bNever = bQe + L::QB;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(bar(bFull + i), 2);
            mbar_init(bar(bEmpty + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(bS + i), 1);
            mbar_init(bar(bP + i), 8);
            mbar_init(bar(bO + i), 1);
        }
        for (int i = 0; i < L::QB; ++i) {
            mbar_init(bar(bQ + i), 1);
            mbar_init(bar(bQe + i), 2);
        }
        mbar_init(bar(bNever), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) tc::tmem_alloc<L::tmem>(sb + L::misc);
    int* top_s = reinterpret_cast<int*>(sm + L::top);
    for (int i = tid; i < 3 * GP; i += kDecThreads) top_s[i] = INT_MIN;
    // columns behind NT * GP: query rows and weights of zero, never written again
    for (int i = tid; i < L::QB * L::q_bytes / 4; i += kDecThreads) reinterpret_cast<uint32_t*>(sm + L::q)[i] = 0;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + L::misc);
    grid_dependency_wait();
    grid_launch_dependents();

    // ---- this CTA's run of tiles ----
    const int HS = g.hkv * A.nsub, B = A.a.b.batch;
    const int cap = (int)min((int64_t)A.a.b.max_blocks * g.bs, (int64_t)0x7FFFFF00);
    auto length = [&](int b) {
        const int n = __ldg(A.a.lens + b);
        return n < 0 ? 0 : min(n, cap);
    };
    auto tiles = [&](int len) { return max(1, (len + kTile - 1) / kTile); };  // an empty sequence has one, all masked
    int64_t total = 0;
    for (int b = lane; b < B; b += 32) total += tiles(length(b));
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
    total *= HS;
    const int64_t runs = min((int64_t)gridDim.x, total);
    const int64_t t0 = (int64_t)blockIdx.x * total / runs, t1 = ((int64_t)blockIdx.x + 1) * total / runs;
    const bool work = (int64_t)blockIdx.x < runs;
    Walk w0{0, 0, 0, 1, 0};
    if (work) {  // the sequence that tile t0 lies in
        int64_t before = 0;
        for (int b0 = 0;; b0 += 32) {
            const int b = b0 + lane;
            const int n = b < B ? tiles(length(b)) : 0;
            int64_t inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                if (lane >= o) inc += y;
            }
            const unsigned past = __ballot_sync(0xFFFFFFFFu, (before + inc) * HS > t0);
            if (past || b0 + 32 >= B) {
                const int l = past ? __ffs((int)past) - 1 : 31;
                w0.b = b0 + l;
                w0.nt = __shfl_sync(0xFFFFFFFFu, n, l);
                before += __shfl_sync(0xFFFFFFFFu, inc, l) - w0.nt;
                break;
            }
            before += __shfl_sync(0xFFFFFFFFu, inc, 31);
        }
        w0.len = length(w0.b);
        const int64_t rem = t0 - before * HS;
        w0.hs = (int)(rem / w0.nt);
        w0.ti = (int)(rem - (int64_t)w0.hs * w0.nt);
    }
    auto next_item = [&](Walk& w) {
        w.ti = 0;
        if (++w.hs == HS) {
            w.hs = 0;
            if (++w.b < B) {
                w.len = length(w.b);
                w.nt = tiles(w.len);
            }
        }
    };
    bool bad = false;  // a bounded wait of this thread gave up: it waits no more
    auto wait = [&](int i, uint32_t parity) {
        if (!bad && !mbar_wait(bar(i), parity)) bad = true;
    };
    const int PT = kTile >> g.bs_shift;  // pages of a tile
    // block id of page `pg` of the tile, or -1
    auto page_id = [&](const Walk& w, int pg) {
        const int64_t i = (int64_t)w.ti * PT + pg;
        if (pg >= PT || (i << g.bs_shift) >= w.len) return -1;
        const int id = __ldg(A.a.b.block_table + (int64_t)w.b * A.a.b.max_blocks + i);
        return id >= 0 && id < g.num_blocks ? id : -2;
    };

    if (!work) {
        // fewer tiles than CTAs
    } else if (warp == 8) {
        // ================= TMA: lanes 0-15 the pages of even tiles, 16-31 of odd ones =================
        const int half = lane >> 4, pg = lane & 15;
        const uint32_t bytes = (uint32_t)g.bs * kHeadDim;
        asm volatile("fence.proxy.async.global;" ::: "memory");  // the codes were written by ordinary stores
        Walk w = w0;
        int64_t t = t0;
        auto advance = [&]() {
            if (++w.ti == w.nt) next_item(w);
            ++t;
        };
        if (half) advance();
        int id = t < t1 ? page_id(w, pg) : -1;
        const int n = (int)(t1 - t0);
        for (int u = 0; u < n; u += 2) {
            const int now = id, h = w.hs / A.nsub;
            if (now == -2) flag(A.a.status, TQ_FLAG_BAD_SLOT);
            if (pg == 0 && t < t1 && w.ti == 0 && w.hs == 0) {
                const int raw_len = __ldg(A.a.lens + w.b);
                if (raw_len < 0 || raw_len > cap) flag(A.a.status, TQ_FLAG_BAD_SLOT);
            }
            advance();
            advance();
            id = t < t1 ? page_id(w, pg) : -1;  // of two tiles on, while this one's copies are issued
            for (int k = 0; k < 2 && u + k < n; ++k) {
                const int st = (u + k) % kStages, ph = (u + k) / kStages;
                if (ph > 0) wait(bEmpty + st, (ph - 1) & 1);
                const unsigned there = __ballot_sync(0xFFFFFFFFu, half == k && now >= 0);
                if (lane == 0) mbar_arrive_tx(bar(bFull + st), (uint32_t)__popc(there) * 2 * bytes);
                __syncwarp();
                if (half == k && now >= 0) {
                    const int row = (int)((((int64_t)now * g.hkv + h) * 2) << g.bs_shift);
                    const uint32_t dst = sb + st * 2 * kSide + pg * bytes;
                    tma_page(dst, &map, row, bar(bFull + st));
                    tma_page(dst + kSide, &map, row + g.bs, bar(bFull + st));
                }
            }
        }
        // copies may be in flight where a wait gave up: they end (again with a limit) before the memory is given back
        for (int u = max(0, n - kStages); u < n; ++u) mbar_wait(bar(bFull + u % kStages), (u / kStages) & 1);
    } else if (warp == 11) {
        // ================= scales of the pages =================
        Walk w = w0;
        const int n = (int)(t1 - t0);
        for (int u = 0; u < n; ++u) {
            const int st = u % kStages, ph = u / kStages;
            const int id = lane < 16 ? page_id(w, lane) : -1;
            float2 s = make_float2(0.f, 0.f);
            if (id >= 0) s = __ldg(reinterpret_cast<const float2*>(g.scales + ((int64_t)id * g.hkv + w.hs / A.nsub) * 2));
            int e = id >= 0 ? fp8_exp_of(s.y) : -1000;
            int emax = e;
#pragma unroll
            for (int o = 8; o; o >>= 1) emax = max(emax, __shfl_xor_sync(0xFFFFFFFFu, emax, o));
            const unsigned there = __ballot_sync(0xFFFFFFFFu, id >= 0);
            if (ph > 0) wait(bEmpty + st, (ph - 1) & 1);
            float* m = reinterpret_cast<float*>(sm + L::meta) + st * 2 * kPagesMax;
            if (lane < 16) {
                m[lane] = s.x;
                m[16 + lane] = id >= 0 && e - emax > -126 ? fp8_pow2(e - emax) : 0.f;
            }
            if (lane == 0) {
                int* o = reinterpret_cast<int*>(sm + L::okm) + 2 * st;
                o[0] = (int)there;
                o[1] = there ? emax : 0;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(bFull + st));
            if (++w.ti == w.nt) next_item(w);
        }
    } else if (warp == 10) {
        // ================= queries: NT terms of e4m3, rows in the 128-byte swizzle =================
        Walk w = w0;
        int64_t t = t0;
        for (int i = 0; t < t1; ++i) {
            const int qb = i % L::QB, use = i / L::QB;
            const int h = w.hs / A.nsub, sub = w.hs - h * A.nsub;
            const int count = min(GP, A.a.group - sub * GP);
            const T* q = static_cast<const T*>(A.a.q) + w.b * A.a.q_token +
                         ((int64_t)h * A.a.group + sub * GP) * A.a.q_head + 4 * lane;
            uint2 rawq[GP];
#pragma unroll
            for (int r = 0; r < GP; ++r)
                rawq[r] = r < count ? __ldg(reinterpret_cast<const uint2*>(q + r * A.a.q_head)) : make_uint2(0, 0);
            if (use > 0) wait(bQe + qb, (use - 1) & 1);
            float* mult = reinterpret_cast<float*>(sm + L::mult) + qb * GP;
#pragma unroll
            for (int r = 0; r < GP; ++r) {
                float x[4];
                load4(&rawq[r], std::is_same<T, __nv_bfloat16>::value ? TQ_BF16 : TQ_F16, 0, x);
                float top = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
                const bool odd = !(fabsf(x[0]) < INFINITY && fabsf(x[1]) < INFINITY && fabsf(x[2]) < INFINITY &&
                                   fabsf(x[3]) < INFINITY);
#pragma unroll
                for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                const bool row_odd = __any_sync(0xFFFFFFFFu, odd);
                const int e = row_odd ? 0 : fp8_exponent(top);
                const float inv = fp8_pow2(-e);
#pragma unroll
                for (int k = 0; k < 4; ++k) x[k] *= inv;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int n = j * GP + r;
                    const uint32_t lo = fp8_cvt2(x[0], x[1]), hi = fp8_cvt2(x[2], x[3]);
                    *reinterpret_cast<uint32_t*>(sm + L::q + qb * L::q_bytes + n * 128 + (((lane >> 2) ^ (n & 7)) << 4) +
                                                 (lane & 3) * 4) = lo | (hi << 16);
                    const float2 a = fp8_to_float2(lo), c = fp8_to_float2(hi);
                    x[0] = (x[0] - a.x) * 16.f;
                    x[1] = (x[1] - a.y) * 16.f;
                    x[2] = (x[2] - c.x) * 16.f;
                    x[3] = (x[3] - c.y) * 16.f;
                }
                // a query that is not finite makes its own row NaN
                if (lane == 0) mult[r] = row_odd ? NAN : A.a.sm_scale_log2 * fp8_pow2(e);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(bQ + qb));
            t += min((int64_t)(w.nt - w.ti), t1 - t);
            next_item(w);
        }
    } else if (warp == 9) {
        // ================= MMA =================
        if (lane == 0) {
            Walk w = w0;
            int64_t t = t0;
            int u = 0;
            auto values = [&](int v) {
                const int st = v % kStages;
                wait(bP + (v & 1), (v >> 1) & 1);
                tc::fence_after_sync();
                const uint32_t sv = sb + st * 2 * kSide + kSide, sp = sb + L::p + (v & 1) * L::p_bytes;
#pragma unroll
                for (int k = 0; k < kTile / 32; ++k)
                    mma_f8_ss(tmem + 4 * N + (v & 1) * N, desc_sw128_mn(sv + 4096 * k), tc::smem_desc(sp + 512 * k, 128, kTile * 16),
                              idesc_f8(N, true), k > 0);
                tc::commit(bar(bO + (v & 1)));
                tc::commit(bar(bEmpty + st));
            };
            for (int i = 0; t < t1; ++i) {
                const int qb = i % L::QB;
                const int n = (int)min((int64_t)(w.nt - w.ti), t1 - t);
                wait(bQ + qb, (i / L::QB) & 1);
                const uint32_t sq = sb + L::q + qb * L::q_bytes;
                for (int j = 0; j < n; ++j, ++u) {
                    const int st = u % kStages;
                    wait(bFull + st, (u / kStages) & 1);
                    tc::fence_after_sync();
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_f8_ss(tmem + ((u & 1) * 2 + m) * N,
                                      tc::smem_desc_sw128(sb + st * 2 * kSide + m * (kSide / 2) + 32 * k, 1024),
                                      tc::smem_desc_sw128(sq + 32 * k, 1024), idesc_f8(N, false), k > 0);
                    tc::commit(bar(bS + (u & 1)));
                    if (j == n - 1) tc::commit(bar(bQe + qb));
                    if (j > 0) values(u - 1);
                }
                values(u - 1);  // the item's last: its output is drained before the next one's scores
                t += n;
                next_item(w);
            }
        }
        __syncwarp();
    } else {
        // ================= softmax and accumulation =================
        constexpr int H = GP / 2;  // accumulator columns of a thread
        const int wg = warp >> 2, quad = warp & 3;
        const uint32_t my = tmem + ((uint32_t)(quad * 32) << 16);
        const int tok = tid;                // token of the tile
        const int dim = quad * 32 + lane;   // output dim
        int* last_s = reinterpret_cast<int*>(sm + L::misc + 8);
        float* sums_s = reinterpret_cast<float*>(sm + L::sums);
        bool empty = false;  // test hook: this CTA's partials are empty
        if (A.stall_cycles > 0 && (blockIdx.x & 1)) {
            empty = !mbar_wait_for(bar(bNever), 0, A.stall_cycles);
            if (empty && tid == 0) flag(A.a.status, TQ_FLAG_TIMEOUT);
        }
        Walk w = w0;
        int64_t t = t0;
        int u = 0;
        for (int i = 0; t < t1; ++i) {
            const int qb = i % L::QB;
            const int n = (int)min((int64_t)(w.nt - w.ti), t1 - t);
            float m[GP], sum[GP], acc[H], mult[GP], pa[H], pb[H];
#pragma unroll
            for (int k = 0; k < GP; ++k) {
                m[k] = -INFINITY;
                sum[k] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < H; ++k) acc[k] = 0.f;
            auto take_output = [&](int v) {  // acc = acc * pa + O(v) * pb
                wait(bO + (v & 1), (v >> 1) & 1);
                tc::fence_after_sync();
                __syncwarp();
                uint32_t o[NT * H];
#pragma unroll
                for (int j = 0; j < NT; ++j) tmem_ld<H>(my + 4 * N + (v & 1) * N + j * GP + wg * H, o + j * H);
                tmem_ready<NT * H>(o);
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    float x = __uint_as_float(o[(NT - 1) * H + k]);
#pragma unroll
                    for (int j = NT - 2; j >= 0; --j) x = fmaf(x, 0.0625f, __uint_as_float(o[j * H + k]));
                    acc[k] = fmaf(acc[k], pa[k], x * pb[k]);
                }
            };
            wait(bQ + qb, (i / L::QB) & 1);
#pragma unroll
            for (int k = 0; k < GP; ++k) mult[k] = reinterpret_cast<const float*>(sm + L::mult)[qb * GP + k];
            for (int j = 0; j < n; ++j, ++u) {
                const int st = u % kStages;
                wait(bFull + st, (u / kStages) & 1);
                const float* me = reinterpret_cast<const float*>(sm + L::meta) + st * 2 * kPagesMax;
                const int* okm = reinterpret_cast<const int*>(sm + L::okm) + 2 * st;
                const int pg = tok >> g.bs_shift;
                const bool there = ((okm[0] >> pg) & 1) && (w.ti + j) * kTile + tok < w.len;
                const float ks = me[pg], vr = me[16 + pg], vscale = fp8_pow2(okm[1]);
                wait(bS + (u & 1), (u >> 1) & 1);
                tc::fence_after_sync();
                __syncwarp();
                uint32_t s[N];
                tmem_ld<NT * GP>(my + ((u & 1) * 2 + wg) * N, s);
                tmem_ready<NT * GP>(s);
                float l[GP], x[GP];
#pragma unroll
                for (int k = 0; k < GP; ++k) {
                    float y = __uint_as_float(s[(NT - 1) * GP + k]);
#pragma unroll
                    for (int q = NT - 2; q >= 0; --q) y = fmaf(y, 0.0625f, __uint_as_float(s[q * GP + k]));
                    l[k] = there ? y * (mult[k] * ks) : -INFINITY;
                    x[k] = l[k];
                }
                // the tile's maximum of every column
                const float best = reduce_lanes<GP, true>(x);
                int* top = top_s + (u % 3) * GP;
                if (lane < GP) atomicMax(top + lane, order_key(best));
                if (!there) {  // a weight of zero against whatever the slot holds
                    const uint32_t v = sb + st * 2 * kSide + kSide + tok * kHeadDim;
#pragma unroll
                    for (int c = 0; c < 8; ++c) asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v + 16 * c), "r"(0) : "memory");
                }
                soft_barrier();
                // for the tile after the next: its last readers have passed this barrier, its writers come after the next
                if (tid < GP) top_s[((u + 2) % 3) * GP + tid] = INT_MIN;
                if (j == 0 && tid == 0) mbar_arrive(bar(bQe + qb));  // everybody has read the multipliers
                float na[H], nb[H];
#pragma unroll
                for (int k = 0; k < GP; ++k) {
                    const float mt = order_val(top[k]);
                    const float mn = fmaxf(m[k], mt), ref = mn == -INFINITY ? 0.f : mn;
                    const float al = ex2(m[k] - ref), be = ex2(mt - ref);
                    m[k] = mn;
                    const float p = ex2(l[k] - (mt == -INFINITY ? 0.f : mt));
                    sum[k] = fmaf(sum[k], al, p * be);
                    x[k] = there ? p * (vr * kPScale) : 0.f;
                    if (k / H == 0 && wg == 0) {
                        na[k % H] = al;
                        nb[k % H] = be * (1.f / kPScale) * vscale;
                    }
                    if (k / H == 1 && wg == 1) {
                        na[k % H] = al;
                        nb[k % H] = be * (1.f / kPScale) * vscale;
                    }
                }
                // the weights' terms: byte n of the token's 16-column rows
                uint32_t word[N / 4];
#pragma unroll
                for (int k = 0; k < N / 4; ++k) word[k] = 0;
#pragma unroll
                for (int q = 0; q < NT; ++q)
#pragma unroll
                    for (int k = 0; k < GP; k += 4) {
                        const uint32_t lo = fp8_cvt2(x[k], x[k + 1]), hi = fp8_cvt2(x[k + 2], x[k + 3]);
                        word[(q * GP + k) / 4] = lo | (hi << 16);
                        if (q + 1 < NT) {
                            const float2 a = fp8_to_float2(lo), c = fp8_to_float2(hi);
                            x[k] = (x[k] - a.x) * 16.f;
                            x[k + 1] = (x[k + 1] - a.y) * 16.f;
                            x[k + 2] = (x[k + 2] - c.x) * 16.f;
                            x[k + 3] = (x[k + 3] - c.y) * 16.f;
                        }
                    }
                const uint32_t sp = sb + L::p + (u & 1) * L::p_bytes + tok * 16;
#pragma unroll
                for (int k = 0; k < N / 16; ++k)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(sp + k * kTile * 16), "r"(word[4 * k]),
                                 "r"(word[4 * k + 1]), "r"(word[4 * k + 2]), "r"(word[4 * k + 3])
                                 : "memory");
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(bP + (u & 1)));
                if (j > 0) take_output(u - 1);
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    pa[k] = na[k];
                    pb[k] = nb[k];
                }
            }
            take_output(u - 1);
            // ---- the item's end ----
            const float part_sum = reduce_lanes<GP, false>(sum);
            if (lane < GP) sums_s[warp * GP + lane] = part_sum;
            soft_barrier();
            float tot[H];
#pragma unroll
            for (int k = 0; k < H; ++k) {
                tot[k] = 0.f;
#pragma unroll
                for (int y = 0; y < 8; ++y) tot[k] += sums_s[y * GP + wg * H + k];
            }
            if (bad && !empty) {
                flag(A.a.status, TQ_FLAG_TIMEOUT);
                empty = true;
            }
            const int h = w.hs / A.nsub, sub = w.hs - h * A.nsub;
            const int count = min(GP, A.a.group - sub * GP);
            const int64_t row0 = (int64_t)w.b * A.a.hq + (int64_t)h * A.a.group + sub * GP;
            T* out = static_cast<T*>(A.a.out) + row0 * kHeadDim;
            const int64_t a0 = t - w.ti, a1 = a0 + w.nt;  // the item's tiles in the flat list
            if (a0 >= t0 && a1 <= t1) {
#pragma unroll
                for (int k = 0; k < H; ++k)
                    if (wg * H + k < count && !empty)
                        out[(wg * H + k) * kHeadDim + dim] = (T)(tot[k] == 0.f ? 0.f : acc[k] / tot[k]);
                soft_barrier();
            } else {
                float* part = A.partials + ((int64_t)blockIdx.x * 2 + (a0 >= t0 ? 1 : 0)) * kPartFloats;
                float mm[H];
#pragma unroll
                for (int k = 0; k < H; ++k) mm[k] = wg ? m[H + k] : m[k];
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    part[(wg * H + k) * kHeadDim + dim] = empty ? 0.f : acc[k];
                    if (dim == 0) {
                        part[16 * kHeadDim + 2 * (wg * H + k)] = empty ? -INFINITY : mm[k];
                        part[16 * kHeadDim + 2 * (wg * H + k) + 1] = empty ? 0.f : tot[k];
                    }
                }
                const int c0 = (int)(((a0 + 1) * runs - 1) / total), c1 = (int)((a1 * runs - 1) / total);
                __threadfence();
                soft_barrier();
                if (tid == 0) {
                    unsigned* c = A.counters + (int64_t)w.b * HS + w.hs;
                    const unsigned before = atomicAdd(c, 1u);
                    const bool last = before == (unsigned)(c1 - c0);
                    if (last) *c = 0u;
                    *last_s = last;
                    __threadfence();
                }
                soft_barrier();
                if (*last_s) {
                    // join the runs' partials in their order, one warp per query row
                    for (int r = warp; r < count; r += 8) {
                        auto of = [&](int c) {
                            return A.partials + ((int64_t)c * 2 + (c == c0 ? 1 : 0)) * kPartFloats;
                        };
                        float mx = -INFINITY;
                        for (int c = c0 + lane; c <= c1; c += 32) mx = fmaxf(mx, __ldcg(of(c) + 16 * kHeadDim + 2 * r));
#pragma unroll
                        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
                        const float ref = mx == -INFINITY ? 0.f : mx;
                        float4 o4 = make_float4(0.f, 0.f, 0.f, 0.f);
                        float all = 0.f;
                        for (int cb = c0; cb <= c1; cb += 32) {
                            float wt = 0.f, sl = 0.f;
                            if (cb + lane <= c1) {
                                const float* ml = of(cb + lane) + 16 * kHeadDim + 2 * r;
                                wt = ex2(__ldcg(ml) - ref);
                                sl = __ldcg(ml + 1) * wt;
                            }
                            const int nc = min(32, c1 - cb + 1);
#pragma unroll 8
                            for (int c = 0; c < nc; ++c) {
                                const float f = __shfl_sync(0xFFFFFFFFu, wt, c);
                                all += __shfl_sync(0xFFFFFFFFu, sl, c);
                                const float4 v = __ldcg(reinterpret_cast<const float4*>(of(cb + c) + r * kHeadDim) + lane);
                                o4.x = fmaf(v.x, f, o4.x);
                                o4.y = fmaf(v.y, f, o4.y);
                                o4.z = fmaf(v.z, f, o4.z);
                                o4.w = fmaf(v.w, f, o4.w);
                            }
                        }
                        const float inv = all == 0.f ? 0.f : 1.f / all;
                        T y[4] = {(T)(o4.x * inv), (T)(o4.y * inv), (T)(o4.z * inv), (T)(o4.w * inv)};
                        *reinterpret_cast<uint2*>(out + r * kHeadDim + 4 * lane) = *reinterpret_cast<const uint2*>(y);
                    }
                }
                soft_barrier();
            }
            t += n;
            next_item(w);
        }
    }
    if (bad && lane == 0) flag(A.a.status, TQ_FLAG_TIMEOUT);
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 9) {
        tc::fence_after_sync();
        tc::tmem_dealloc<L::tmem>(tmem);
    }
}

template <typename T, int NT, int GP>
int launch(const DecArgs& d, const CUtensorMap& map, int grid, cudaStream_t s) {
    auto kern = fp8_decode_kernel<T, NT, GP>;
    static int done[64] = {};
    const cudaError_t e = ensure_smem_limit(kern, DecLayout<NT, GP>::smem, done);
    if (e != cudaSuccess) return (int)e;
    return (int)launch_programmatic(kern, dim3((unsigned)grid), dim3(kDecThreads), (size_t)DecLayout<NT, GP>::smem, s, d, map);
}

// Query heads go in parts of 8 or 16 columns: 8 where they suffice (fewer exponentials per token).
int part_of(int group) { return group <= 8 ? 8 : 16; }

size_t counter_bytes(int batch, int hkv, int group) {
    const int gp = part_of(group);
    return ((size_t)batch * hkv * ((group + gp - 1) / gp) * sizeof(unsigned) + 255) / 256 * 256;
}

}  // namespace

size_t fp8_decode_workspace(const Fp8Geometry& g, int batch, int group) {
    return counter_bytes(batch, g.hkv, group) + (size_t)(g.num_sms > 0 ? g.num_sms : 1) * 2 * kPartFloats * sizeof(float);
}

int launch_fp8_decode(const Fp8AttnArgs& a, const CUtensorMap& map, void* workspace, void* stream) {
    DecArgs d{};
    d.a = a;
    const int gp = part_of(a.group);
    d.nsub = (a.group + gp - 1) / gp;
    d.counters = static_cast<unsigned*>(workspace);
    d.partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + counter_bytes(a.b.batch, a.g.hkv, a.group));
    d.stall_cycles = test_stall_cycles();
    const int64_t most = (int64_t)a.b.batch * a.g.hkv * d.nsub * (((int64_t)a.b.max_blocks * a.g.bs + kTile - 1) / kTile);
    const int grid = (int)(most < a.g.num_sms ? most : a.g.num_sms);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (a.dtype == TQ_BF16)
        return gp == 8 ? launch<__nv_bfloat16, 2, 8>(d, map, grid, s) : launch<__nv_bfloat16, 2, 16>(d, map, grid, s);
    return gp == 8 ? launch<__half, 3, 8>(d, map, grid, s) : launch<__half, 3, 16>(d, map, grid, s);
}

}  // namespace tq
