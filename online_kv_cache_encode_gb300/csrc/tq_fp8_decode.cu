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
// takes 3 terms, 2^-12 (tiles whose value scales lie far apart are weighed in
// fp32 instead).  Key scales multiply the scores, value scales the
// weights (both powers of two).  The weights of a tile are taken against a
// reference near its own maximum, not the running one, and a tile's output
// leaves tensor memory and is joined in fp32 registers: the tokens behind one
// that dominates a long context keep the bits of their weights.
//
// What bounds it is the cache's bytes: the tensor work of a tile is about 500
// cycles and its softmax 1000, against 2850 cycles that HBM needs for its 64 KB
// on one of 152 SMs.  Hence one CTA per SM, a ring of three 64 KB stages filled
// by TMA (pages land in the 128-byte swizzle that both readings of a row
// share), and the flat list of all (sequence, head, tile) cut into equal runs,
// whatever the lengths are.  An item (sequence, head) that lies in one run is
// written directly; otherwise each run leaves a partial (reference, sum,
// accumulator) and the last run to arrive joins them in their order, so results
// do not depend on timing.  64 sequences of 1K-16K tokens, 8 KV heads: 192 us,
// 0.84 of HBM; 32K tokens, 8 heads: 22 us, of which 13 stream (0.75).
//
// Warps: 0-7 softmax and accumulation (thread = token of the tile for the
// scores, = dim for the output, the two warpgroups taking half of the columns
// each), 8 and 10 TMA, 9 MMA, 11 queries and scales.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>

#include "tq_fp8.cuh"
#include "tq_fp8_tc.cuh"

namespace tq {
namespace {

constexpr int kTile = 256;            // tokens of a tile
constexpr int kStages = 3;
constexpr int kSide = kTile * kHeadDim;   // bytes of a tile's keys (or values)
constexpr int kPagesMax = kTile / 16;
constexpr int kDecWarps = 12;
constexpr int kDecThreads = kDecWarps * 32;
constexpr float kPScale = 256.f;      // weights are coded as p * 2^8 <= 430 (e4m3's largest value is 448)
constexpr int kWideSpread = 6;        // octaves between a tile's value scales beyond which it is weighed in fp32
constexpr int kLeastValueExp = -98;   // blocks below hold values under 2^-89 only: they make no tile wide

__device__ __forceinline__ void soft_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// The same, and whether `x` holds in any of the 256 threads: one answer for all, whatever each of them has read.
__device__ __forceinline__ bool soft_barrier_or(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

// Sums C values of every lane over the warp; lane l gets the sum of value l % C.
template <int C>
__device__ __forceinline__ float sum_lanes(float (&v)[C]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int w = C / 2; w >= 1; w /= 2) {  // halve the values, keep those of this lane's half
        const bool up = lane & w;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float mine = up ? v[i + w] : v[i], other = up ? v[i] : v[i + w];
            v[i] = mine + __shfl_xor_sync(0xFFFFFFFFu, other, w);
        }
    }
    float x = v[0];
#pragma unroll
    for (int w = C; w < 32; w *= 2) x += __shfl_xor_sync(0xFFFFFFFFu, x, w);
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
    static constexpr int meta = q + QB * q_bytes;           // per stage: key scales, relative value scales (wide: exponents - 20) [16 each]
    static constexpr int okm = meta + kStages * 2 * kPagesMax * 4;  // per stage: pages there (bit 31: wide), largest value exponent
    static constexpr int mult = okm + kStages * 8;          // per query buffer: [GP]
    static constexpr int top = (mult + QB * GP * 4 + 15) / 16 * 16;  // [2][8 warps][GP] maxima
    static constexpr int sums = top + 2 * 8 * GP * 4;       // [8 warps][GP]
    static constexpr int bars = sums + 8 * GP * 4;
    static constexpr int nbars = 3 * kStages + 6 + 2 * QB + 1;
    static constexpr int misc = bars + 8 * nbars;           // tmem address, last-arrival word
    static constexpr int total = misc + 16;
    static constexpr int smem = total + 1024;               // the base is rounded up to 1 KB
    static constexpr int tmem = 6 * N <= 128 ? 128 : 6 * N <= 256 ? 256 : 512;
    static_assert(p % 1024 == 0 && q % 1024 == 0 && q_bytes % 1024 == 0, "swizzled rows and 16-byte pieces");
    static_assert(meta % 16 == 0 && top % 16 == 0 && bars % 8 == 0 && misc % 8 == 0, "vector accesses");
    static_assert(smem <= kSmemLimit, "decode does not fit in shared memory");
    static_assert(2 * p_bytes >= kTile * GP * 4, "a wide tile's fp32 weights take both weight buffers");
};

constexpr int kPartFloats = 16 * kHeadDim + 32;  // a partial: accumulators [GP][128], (max, sum) [GP]

struct DecArgs {
    Fp8AttnArgs a;
    int nsub;             // parts of GP query heads per KV head
    unsigned* counters;   // [batch * hkv * nsub]
    float* partials;      // [grid][2][kPartFloats]
    long long stall_cycles;
};

template <typename T, int NT, int GP, bool PAIRED>
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
    // a tile landed, its stage free again, its scales stored; scores, weights and outputs of a tile; queries stored,
    // and read; one that nothing arrives on (the wait-timeout test hook)
    constexpr int bF = 0, bE = kStages, bM = 2 * kStages, bS = 3 * kStages, bP = bS + 2, bO = bP + 2, bQ = bO + 2,
                  bQe = bQ + L::QB, bNever = bQe + L::QB;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(bar(bF + i), 2);
            mbar_init(bar(bE + i), 1);
            mbar_init(bar(bM + i), 1);
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
    if (warp == 8 && lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(&map) : "memory");
    if (warp == 9) tc::tmem_alloc<L::tmem>(sb + L::misc);
    float* top_s = reinterpret_cast<float*>(sm + L::top);
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
    // totals stay below 2^31 (the host checks the largest possible)
    const int len0 = lane < B ? length(lane) : 0;  // of the first 32 sequences, read once
    int total = lane < B ? tiles(len0) : 0;
    for (int b = lane + 32; b < B; b += 32) total += tiles(length(b));
    total = __reduce_add_sync(0xFFFFFFFFu, total) * HS;
    const int runs = min((int)gridDim.x, total), cta = (int)blockIdx.x;
    const int each = total / runs, more = total - each * runs;  // the first `more` runs have a tile more
    const int t0 = cta * each + min(cta, more), t1 = t0 + each + (cta < more ? 1 : 0);
    auto run_of = [&](int t) { return t < more * (each + 1) ? t / (each + 1) : more + (t - more * (each + 1)) / each; };
    const bool work = cta < runs;
    Walk w0{0, 0, 0, 1, 0};
    if (work) {  // the sequence that tile t0 lies in
        int before = 0;
        for (int b0 = 0;; b0 += 32) {
            const int b = b0 + lane, len = b0 == 0 ? len0 : b < B ? length(b) : 0;
            const int n = b < B ? tiles(len) : 0;
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                if (lane >= o) inc += y;
            }
            const unsigned past = __ballot_sync(0xFFFFFFFFu, (before + inc) * HS > t0);
            if (past || b0 + 32 >= B) {
                const int l = past ? __ffs((int)past) - 1 : 31;
                w0.b = b0 + l;
                w0.nt = __shfl_sync(0xFFFFFFFFu, n, l);
                w0.len = __shfl_sync(0xFFFFFFFFu, len, l);
                before += __shfl_sync(0xFFFFFFFFu, inc, l) - w0.nt;
                break;
            }
            before += __shfl_sync(0xFFFFFFFFu, inc, 31);
        }
        const int rem = t0 - before * HS;
        w0.hs = rem / w0.nt;
        w0.ti = rem - w0.hs * w0.nt;
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
    // A stage.  With blocks of 16 tokens (PAIRED) a page's keys and values, 4 KB that lie together in the pool, come in one
    // copy, page by page: the tensor cores then take the 8-row groups 4 KB apart, the first halves of the 16 pages
    // and then the second ones, and the tile's tokens go in that order everywhere.  Larger blocks have copies of 4 KB
    // and more for each side: all keys, then all values.  (A copy costs about 75 cycles to issue: 32 of them a tile
    // took as long as the tile's bytes.)
    constexpr uint32_t sbo = PAIRED ? 4096 : 1024;
    constexpr uint32_t k_half = PAIRED ? 1024 : kSide / 2, v_base = PAIRED ? 2048 : kSide;
    // block id of page `pg` of the tile, or -1
    auto page_id = [&](const Walk& w, int pg) {
        const int64_t i = (int64_t)w.ti * PT + pg;
        if (pg >= PT || (i << g.bs_shift) >= w.len) return -1;
        const int id = __ldg(A.a.b.block_table + (int64_t)w.b * A.a.b.max_blocks + i);
        return id >= 0 && id < g.num_blocks ? id : -2;
    };

    if (!work) {
        // fewer tiles than CTAs
    } else if (warp == 8 || warp == 10) {
        // ================= TMA: a quarter of the lanes per tile, a lane per copy =================
        const int quarter = lane >> 3, second = warp == 10;
        const int pg = (lane & 7) + (PAIRED && second ? 8 : 0);
        const uint32_t bytes = PAIRED ? 4096 : (uint32_t)g.bs * kHeadDim;
        const uint32_t at = (uint32_t)pg * bytes + (!PAIRED && second ? kSide : 0);
        asm volatile("fence.proxy.async.global;" ::: "memory");  // the codes were written by ordinary stores
        Walk w = w0;
        int t = t0;
        auto advance = [&](int k) {
            for (; k > 0; --k, ++t)
                if (++w.ti == w.nt) next_item(w);
        };
        advance(quarter);
        int id = t < t1 ? page_id(w, pg) : -1;
        const int n = t1 - t0;
        int sent = 0;  // tiles whose copies are issued: none after a wait that gave up
        for (int u = 0; u < n && !bad; u += 4) {
            const int now = id, h = w.hs / A.nsub, b = w.b;
            const bool first = t < t1 && w.ti == 0 && w.hs == 0;
            advance(4);
            id = t < t1 ? page_id(w, pg) : -1;  // of four tiles on, while these ones' copies are issued
            const int row = (int)((((int64_t)max(now, 0) * g.hkv + h) * 2 + (!PAIRED && second)) << g.bs_shift);
            for (int k = 0; k < 4 && u + k < n; ++k) {
                const int st = (u + k) % kStages, ph = (u + k) / kStages;
                const unsigned there = __ballot_sync(0xFFFFFFFFu, quarter == k && now >= 0);
                if (ph > 0) {
                    wait(bE + st, (ph - 1) & 1);
                    bad = __any_sync(0xFFFFFFFFu, bad);
                    if (bad) break;
                }
                sent = u + k + 1;
                if (lane == 0) mbar_arrive_tx(bar(bF + st), (uint32_t)__popc(there) * bytes);
                __syncwarp();
                if (quarter == k && now >= 0) tma_page(sb + st * 2 * kSide + at, &map, row, bar(bF + st));
            }
            if (now == -2) flag(A.a.status, TQ_FLAG_BAD_SLOT);
            if (pg == 0 && !second && first) {
                const int given = __ldg(A.a.lens + b);
                if (given < 0 || given > cap) flag(A.a.status, TQ_FLAG_BAD_SLOT);
            }
        }
        // copies may be in flight where a wait gave up: they end (again with a limit) before the memory is given back
        for (int u = max(0, sent - kStages); u < sent; ++u) mbar_wait(bar(bF + u % kStages), (u / kStages) & 1);
    } else if (warp == 11) {
        // ================= queries and scales =================
        Walk w = w0;
        const int n = t1 - t0;
        bool fresh = true;  // tile u is the item's first here
        for (int u = 0, i = -1; u < n; ++u) {
            const int st = u % kStages, ph = u / kStages;
            const int h = w.hs / A.nsub, sub = w.hs - h * A.nsub;
            const int id = lane < 16 ? page_id(w, lane) : -1;
            float2 s = make_float2(0.f, 0.f);
            if (id >= 0) s = __ldg(reinterpret_cast<const float2*>(g.scales + ((int64_t)id * g.hkv + h) * 2));
            if (fresh) {  // the item's queries: NT terms of e4m3, rows in the 128-byte swizzle
                ++i;
                const int qb = i % L::QB, use = i / L::QB;
                const int count = min(GP, A.a.group - sub * GP);
                const T* q = static_cast<const T*>(A.a.q) + w.b * A.a.q_token +
                             ((int64_t)h * A.a.group + sub * GP) * A.a.q_head + 4 * lane;
                uint32_t rawq[GP][2];
#pragma unroll
                for (int r = 0; r < GP; ++r) {
                    const uint2 v = r < count ? __ldg(reinterpret_cast<const uint2*>(q + r * A.a.q_head)) : make_uint2(0, 0);
                    rawq[r][0] = v.x;
                    rawq[r][1] = v.y;
                }
                if (use > 0) wait(bQe + qb, (use - 1) & 1);
                float* mult = reinterpret_cast<float*>(sm + L::mult) + qb * GP;
                Fp8Split<T, 32, GP> split(rawq);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    uint32_t code[GP][1];
                    split.template term<0x4C004C00u>(code);  // the terms 1/16 apart
#pragma unroll
                    for (int r = 0; r < GP; ++r) {
                        const int c = j * GP + r;
                        *reinterpret_cast<uint32_t*>(sm + L::q + qb * L::q_bytes + c * 128 + (((lane >> 2) ^ (c & 7)) << 4) +
                                                     (lane & 3) * 4) = code[r][0];
                    }
                }
                float factors = 0.f;  // a query that is not finite makes its own row NaN
#pragma unroll
                for (int r = 0; r < GP; ++r) factors = lane == r ? split.factor(r, A.a.sm_scale_log2) : factors;
                if (lane < GP) mult[lane] = factors;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(bQ + qb));
            }
            const int e = id >= 0 ? fp8_exp_of(s.y) : -1000;
            int emax = e, emin = e >= kLeastValueExp ? e : 1000;
#pragma unroll
            for (int o = 8; o; o >>= 1) {  // (lanes 0-15 hold the blocks)
                emax = max(emax, __shfl_xor_sync(0xFFFFFFFFu, emax, o));
                emin = min(emin, __shfl_xor_sync(0xFFFFFFFFu, emin, o));
            }
            const unsigned there = __ballot_sync(0xFFFFFFFFu, id >= 0);
            const bool wide = emax - emin > kWideSpread;  // (without such blocks emin > emax)
            if (ph > 0) wait(bE + st, (ph - 1) & 1);
            float* m = reinterpret_cast<float*>(sm + L::meta) + st * 2 * kPagesMax;
            if (lane < 16) {
                m[lane] = s.x;
                m[16 + lane] = id < 0 ? 0.f : wide ? (float)(e - 20) : e - emax < -100 ? 0.f : fp8_pow2(e - emax);
            }
            if (lane == 0) {
                int* o = reinterpret_cast<int*>(sm + L::okm) + 2 * st;
                o[0] = (int)(there | (wide ? 0x80000000u : 0u));
                o[1] = there ? emax : 0;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(bM + st));
            fresh = w.ti + 1 == w.nt;
            if (fresh) next_item(w);
            else ++w.ti;
        }
    } else if (warp == 9) {
        // ================= MMA =================
        // Scores of tile u and values of tile v are issued as their operands come: with the cache in HBM the weights
        // of a tile are ready before the next tile's keys are, with the cache in L2 the other way round.  Scores run
        // at most one tile ahead (their buffer's last reader has stored the weights of tile u - 2).  The warp stays
        // together and one lane issues, so that descriptors live in uniform registers.
        Walk w = w0;
        const int n = t1 - t0;
        int u = 0, v = 0;
        uint32_t su = 0, pu = 0, sv = 0, qb = 0, pq = 0;  // stage and parity of tile u, stage of v, buffer and parity of Q
        bool fresh = true;                                // tile u is the item's first here
        long long since = clock64();
        const uint64_t d_rows = desc_rows(sb, sbo), d_q = desc_rows(sb + L::q, 1024),
                       d_p = tc::smem_desc(sb + L::p, 128, kTile * 16);
        const bool issues = elect_one();
        while (v < n && !bad) {
            bool did = false;
            if (v < u && __all_sync(0xFFFFFFFFu, mbar_test(bar(bP + (v & 1)), (v >> 1) & 1))) {
                tc::fence_after_sync();
                const uint64_t a = d_rows + (sv * 2 * kSide + v_base) / 16, p = d_p + (v & 1) * (L::p_bytes / 16);
                const uint32_t d = tmem + 4 * N + (v & 1) * N;
                if (issues) {
#pragma unroll
                    for (int k = 0; k < kTile / 32; ++k)
                        mma_f8_ss(d, a + (PAIRED ? (k >> 2) * 1024 + (k & 3) * 16384 : k * 4096) / 16, p + 32 * k,
                                  idesc_f8(N, true), k > 0);
                    tc::commit(bar(bO + (v & 1)));
                    tc::commit(bar(bE + sv));
                }
                __syncwarp();
                ++v;
                sv = sv + 1 == kStages ? 0 : sv + 1;
                did = true;
            }
            if (u < n && u <= v + 1 && (!fresh || __all_sync(0xFFFFFFFFu, mbar_test(bar(bQ + qb), pq))) &&
                __all_sync(0xFFFFFFFFu, mbar_test(bar(bF + su), pu))) {
                tc::fence_after_sync();
                const uint64_t q = d_q + qb * (L::q_bytes / 16), a = d_rows + su * 2 * kSide / 16;
                const uint32_t d = tmem + (u & 1) * 2 * N;
                fresh = w.ti + 1 == w.nt;
                const bool last = fresh || u + 1 == n;
                if (issues) {
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_f8_ss(d + m * N, a + (m * k_half + 32 * k) / 16, q + 2 * k, idesc_f8(N, false), k > 0);
                    tc::commit(bar(bS + (u & 1)));
                    if (last) tc::commit(bar(bQe + qb));
                }
                __syncwarp();
                ++u;
                if (++su == kStages) {
                    su = 0;
                    pu ^= 1;
                }
                if (fresh) {
                    next_item(w);
                    if (++qb == L::QB) {
                        qb = 0;
                        pq ^= 1;
                    }
                } else {
                    ++w.ti;
                }
                did = true;
            }
            if (did) since = clock64();
            else if (__any_sync(0xFFFFFFFFu, clock64() - since > kWaitCycles)) bad = true;
        }
        // products may be in flight where a wait gave up: they too end before the memory is given back
        if (u > 0) mbar_wait(bar(bS + ((u - 1) & 1)), ((u - 1) >> 1) & 1);
        if (v > 0) mbar_wait(bar(bO + ((v - 1) & 1)), ((v - 1) >> 1) & 1);
        __syncwarp();
    } else {
        // ================= softmax and accumulation =================
        constexpr int H = GP / 2;  // accumulator columns of a thread
        const int wg = warp >> 2, quad = warp & 3;
        const uint32_t my = tmem + ((uint32_t)(quad * 32) << 16);
        const int row = tid & 127;
        const int pg = PAIRED ? row >> 3 : tid >> g.bs_shift;                    // the thread's token: its page,
        const int tok = PAIRED ? pg * 16 + wg * 8 + (row & 7) : tid;             // its place in the tile,
        const uint32_t v_row = PAIRED ? pg * 4096 + 2048 + (wg * 8 + (row & 7)) * 128 : kSide + tid * 128;  // its values
        const int dim = quad * 32 + lane;   // output dim
        int* last_s = reinterpret_cast<int*>(sm + L::misc + 8);
        float* sums_s = reinterpret_cast<float*>(sm + L::sums);
        bool empty = false;  // test hook: this CTA's partials are empty
        if (A.stall_cycles > 0 && (blockIdx.x & 1)) {
            empty = !mbar_wait_for(bar(bNever), 0, A.stall_cycles);
            if (empty && tid == 0) flag(A.a.status, TQ_FLAG_TIMEOUT);
        }
        // Weights are 2^(l - ref) against a reference `ref` for each column that moves only when the tile's maximum
        // leaves [ref - 6, ref + 3/4]: then it goes to 1.5 above that maximum, though not further than 18.5 below the
        // running one.  So 2^8 times a weight stays below 448, a tile far below the running maximum keeps the bits of
        // its own weights, and what still lies deeper (2^-14 of a weight unit, 2^-40 of the largest weight) does not
        // count.  Lane l watches columns 2 (l % (GP / 2)) and the next; sums and accumulators follow the reference,
        // the latter held 2^-20 small, so that its largest fall leaves them where they would be without it.
        constexpr int LP = GP / 2;
        const int mine = lane % LP;
        Walk w = w0;
        int t = t0;
        int u = 0;
        for (int i = 0; t < t1; ++i) {
            const int qb = i % L::QB;
            const int n = min(w.nt - w.ti, t1 - t);
            float ref[GP], sum[GP], acc[H], mult[GP], fac[H], vs = 0.f;
            float lref[2] = {0.f, 0.f}, lrun[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < GP; ++k) ref[k] = sum[k] = 0.f;
#pragma unroll
            for (int k = 0; k < H; ++k) acc[k] = 0.f;
            auto take_output = [&](int v) {  // acc += O(v) * vs
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
                    acc[k] = fmaf(x, vs, acc[k]);
                }
            };
            wait(bQ + qb, (i / L::QB) & 1);
#pragma unroll
            for (int k = 0; k < GP; ++k) mult[k] = reinterpret_cast<const float*>(sm + L::mult)[qb * GP + k];
            for (int j = 0; j < n; ++j, ++u) {
                const int st = u % kStages;
                wait(bM + st, (u / kStages) & 1);
                const float* me = reinterpret_cast<const float*>(sm + L::meta) + st * 2 * kPagesMax;
                const int* okm = reinterpret_cast<const int*>(sm + L::okm) + 2 * st;
                const bool there = ((okm[0] >> pg) & 1) && (w.ti + j) * kTile + tok < w.len;
                const float ks = me[pg], vr = me[16 + pg] * kPScale;
                const float vs_new = fp8_pow2(okm[1]) * (1.f / kPScale / 1048576.f);
                wait(bS + (u & 1), (u >> 1) & 1);
                tc::fence_after_sync();
                __syncwarp();
                uint32_t s[N];
                tmem_ld<NT * GP>(my + ((u & 1) * 2 + wg) * N, s);
                tmem_ready<NT * GP>(s);
                float l[GP];
                float* top = top_s + (u & 1) * 8 * GP;
                {
                    const uint64_t k16 = f2_pack(0.0625f, 0.0625f), ks2 = f2_pack(ks, ks);
#pragma unroll
                    for (int k = 0; k < GP; k += 2) {
                        uint64_t y = f2_pack(__uint_as_float(s[(NT - 1) * GP + k]), __uint_as_float(s[(NT - 1) * GP + k + 1]));
#pragma unroll
                        for (int q = NT - 2; q >= 0; --q)
                            y = f2_fma(y, k16, f2_pack(__uint_as_float(s[q * GP + k]), __uint_as_float(s[q * GP + k + 1])));
                        f2_unpack(f2_mul(y, f2_mul(f2_pack(mult[k], mult[k + 1]), ks2)), l[k], l[k + 1]);
                    }
                }
                if (!there)
#pragma unroll
                    for (int k = 0; k < GP; ++k) l[k] = -INFINITY;
                // the tile's maximum of every column
                float best[GP];
#pragma unroll
                for (int k = 0; k < GP; ++k) best[k] = redux_max(l[k]);
                if (lane == 0)
#pragma unroll
                    for (int k = 0; k < GP; k += 4)
                        *reinterpret_cast<float4*>(top + warp * GP + k) = make_float4(best[k], best[k + 1], best[k + 2], best[k + 3]);
                // (warps whose bounded waits gave up may have read other words, and all have to take the same barriers)
                const bool wide = soft_barrier_or(okm[0] < 0);
                if (j == 0 && tid == 0) mbar_arrive(bar(bQe + qb));  // everybody has read the multipliers
                float2 tile = make_float2(-INFINITY, -INFINITY);
#pragma unroll
                for (int y = 0; y < 8 * LP / 32; ++y) {
                    const float2 x = *reinterpret_cast<const float2*>(top + (lane / LP + y * (32 / LP)) * GP + 2 * mine);
                    tile.x = fmaxf(tile.x, x.x);
                    tile.y = fmaxf(tile.y, x.y);
                }
#pragma unroll
                for (int o = LP; o < 32; o <<= 1) {
                    tile.x = fmaxf(tile.x, __shfl_xor_sync(0xFFFFFFFFu, tile.x, o));
                    tile.y = fmaxf(tile.y, __shfl_xor_sync(0xFFFFFFFFu, tile.y, o));
                }
                lrun[0] = fmaxf(lrun[0], tile.x);
                lrun[1] = fmaxf(lrun[1], tile.y);
                const float to0 = fmaxf(tile.x + 1.5f, lrun[0] - 18.5f), to1 = fmaxf(tile.y + 1.5f, lrun[1] - 18.5f);
                const bool move0 = tile.x > lref[0] + 0.75f || (tile.x < lref[0] - 6.f && to0 < lref[0]);
                const bool move1 = tile.y > lref[1] + 0.75f || (tile.y < lref[1] - 6.f && to1 < lref[1]);
                // the same in every warp; a column without tokens (its maximum is -inf) stays
                const bool moved = __any_sync(0xFFFFFFFFu, (move0 && to0 > -INFINITY) || (move1 && to1 > -INFINITY));
                if (moved) {
                    if (move0 && to0 > -INFINITY) lref[0] = to0;
                    if (move1 && to1 > -INFINITY) lref[1] = to1;
#pragma unroll
                    for (int k = 0; k < GP; ++k) {
                        const float to = __shfl_sync(0xFFFFFFFFu, lref[k & 1], k >> 1);
                        // (before the column's first token there is nothing to scale: any finite factor does)
                        const float f = ex2(fminf(ref[k] - to, 100.f));
                        ref[k] = to;
                        sum[k] *= f;
                        if (k / H == wg) fac[k % H] = f;
                    }
                }
                float x[GP];
                {
                    const uint64_t vr2 = f2_pack(vr, vr);
#pragma unroll
                    for (int k = 0; k < GP; k += 2) {
                        float a, b;
                        f2_unpack(f2_sub(f2_pack(l[k], l[k + 1]), f2_pack(ref[k], ref[k + 1])), a, b);
                        a = ex2(a);
                        b = ex2(b);
                        const uint64_t p = f2_pack(a, b);
                        f2_unpack(f2_add(f2_pack(sum[k], sum[k + 1]), p), sum[k], sum[k + 1]);
                        f2_unpack(f2_mul(p, vr2), x[k], x[k + 1]);
                    }
                }
                auto clear_row = [&] {  // the token's weights are 0, but its slot may hold NaN codes
                    wait(bF + st, (u / kStages) & 1);
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(sb + st * 2 * kSide + v_row + 16 * c), "r"(0)
                                     : "memory");
                };
                if (wide) {
                    // Value scales far apart: in a column's fp8 weights a block with a large scale would take the range of
                    // the others, also in the dims where its codes are 0 and only the others count.  So the tile is weighed
                    // in fp32, with every token's weight times its scale (2^-20 of it, as the accumulators are) whatever
                    // the others' are.  64 sequences of 8192 tokens, 8 KV heads: 546 us with every tile like that, 182 with
                    // none (the loop's loads bound it: 757 with 4 tokens at a time instead of 16).  The weights go through
                    // both weight buffers, which the tensor cores have left once the last output is there.
                    if (j > 0) take_output(u - 1);
                    if (moved)
#pragma unroll
                        for (int k = 0; k < H; ++k) acc[k] *= fac[k];
                    float* wt = reinterpret_cast<float*>(sm + L::p);
                    const float er = me[16 + pg];
#pragma unroll
                    for (int k = 0; k < GP; k += 4)
                        *reinterpret_cast<float4*>(wt + tid * GP + k) =
                            make_float4(ex2((l[k] - ref[k]) + er), ex2((l[k + 1] - ref[k + 1]) + er),
                                        ex2((l[k + 2] - ref[k + 2]) + er), ex2((l[k + 3] - ref[k + 3]) + er));
                    if (there) wait(bF + st, (u / kStages) & 1);
                    else clear_row();
                    soft_barrier();
                    float add[H];
#pragma unroll
                    for (int k = 0; k < H; ++k) add[k] = 0.f;
#pragma unroll 16
                    for (int y = 0; y < kTile; ++y) {
                        const int at = PAIRED ? ((y & 127) >> 3) * 4096 + 2048 + ((y >> 7) * 8 + (y & 7)) * 128 : kSide + y * 128;
                        const float c = fp8_to_float2(sm[st * 2 * kSide + at + (((dim >> 4) ^ (y & 7)) << 4) + (dim & 15)]).x;
#pragma unroll
                        for (int k = 0; k < H; k += 4) {
                            const float4 f = *reinterpret_cast<const float4*>(wt + y * GP + wg * H + k);
                            add[k] = fmaf(f.x, c, add[k]);
                            add[k + 1] = fmaf(f.y, c, add[k + 1]);
                            add[k + 2] = fmaf(f.z, c, add[k + 2]);
                            add[k + 3] = fmaf(f.w, c, add[k + 3]);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < H; ++k) acc[k] += add[k];
#pragma unroll
                    for (int k = 0; k < GP; ++k) x[k] = 0.f;  // (for the tensor cores, whose output then adds nothing)
                    soft_barrier();
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
                        if (q + 1 < NT) {  // (x - h) * 16 = 16 x - 16 h, both exact
                            const uint64_t m16 = f2_pack(-16.f, -16.f), p16 = f2_pack(16.f, 16.f);
                            const float2 a = fp8_to_float2(lo), c = fp8_to_float2(hi);
                            f2_unpack(f2_fma(f2_pack(a.x, a.y), m16, f2_mul(f2_pack(x[k], x[k + 1]), p16)), x[k], x[k + 1]);
                            f2_unpack(f2_fma(f2_pack(c.x, c.y), m16, f2_mul(f2_pack(x[k + 2], x[k + 3]), p16)), x[k + 2], x[k + 3]);
                        }
                    }
                const uint32_t sp = sb + L::p + (u & 1) * L::p_bytes + tid * 16;
#pragma unroll
                for (int k = 0; k < N / 16; ++k)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(sp + k * kTile * 16), "r"(word[4 * k]),
                                 "r"(word[4 * k + 1]), "r"(word[4 * k + 2]), "r"(word[4 * k + 3])
                                 : "memory");
                if (!there && !wide) clear_row();
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(bP + (u & 1)));
                if (!wide) {
                    if (j > 0) take_output(u - 1);
                    if (moved)
#pragma unroll
                        for (int k = 0; k < H; ++k) acc[k] *= fac[k];
                }
                vs = vs_new;
            }
            // ---- the item's end ----
            const float part_sum = sum_lanes<GP>(sum);
            take_output(u - 1);  // (with its wait every warp is past the last tile's use of sums_s)
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
            const int a0 = t - w.ti, a1 = a0 + w.nt;  // the item's tiles in the flat list
            if (a0 >= t0 && a1 <= t1) {
#pragma unroll
                for (int k = 0; k < H; ++k)
                    if (wg * H + k < count && !empty)
                        out[(wg * H + k) * kHeadDim + dim] = (T)(tot[k] == 0.f ? 0.f : acc[k] * (1048576.f / tot[k]));
                soft_barrier();
            } else {
                float* part = A.partials + ((int64_t)blockIdx.x * 2 + (a0 >= t0 ? 1 : 0)) * kPartFloats;
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    part[(wg * H + k) * kHeadDim + dim] = empty ? 0.f : acc[k];
                    if (dim == 0) {  // (a column without tokens has a sum of 0: its reference does not count)
                        part[16 * kHeadDim + 2 * (wg * H + k)] = empty || tot[k] == 0.f ? -INFINITY : wg ? ref[H + k] : ref[k];
                        part[16 * kHeadDim + 2 * (wg * H + k) + 1] = empty ? 0.f : tot[k];
                    }
                }
                const int c0 = run_of(a0), c1 = run_of(a1 - 1);
                soft_barrier();
                if (tid == 0) {
                    // releases what the CTA stored before the barrier, acquires what the others did
                    unsigned* c = A.counters + (int64_t)w.b * HS + w.hs;
                    unsigned before;
                    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(c) : "memory");
                    const bool last = before == (unsigned)(c1 - c0);
                    if (last) *c = 0u;
                    *last_s = last;
                }
                soft_barrier();
                if (*last_s) {
                    // join the runs' partials in their order, one warp per query row: lane c holds the weight of run c
                    auto of = [&](int c) { return A.partials + ((int64_t)c * 2 + (c == c0 ? 1 : 0)) * kPartFloats; };
                    for (int r = warp; r < count; r += 8) {
                        float mx = -INFINITY, all = 0.f;
                        float4 o4 = make_float4(0.f, 0.f, 0.f, 0.f);
                        constexpr int kJoin = 24;  // runs at a time: all their loads in flight (a head's 19 to 20 runs at 8 heads)
                        for (int cb = c0; cb <= c1; cb += kJoin) {
                            const int nc = min(kJoin, c1 - cb + 1);
                            float2 ml = make_float2(-INFINITY, 0.f);
                            if (lane < nc) ml = __ldcg(reinterpret_cast<const float2*>(of(cb + lane) + 16 * kHeadDim) + r);
                            float4 v[kJoin];
#pragma unroll
                            for (int c = 0; c < kJoin; ++c)
                                v[c] = c < nc ? __ldcg(reinterpret_cast<const float4*>(of(cb + c) + r * kHeadDim) + lane)
                                              : make_float4(0.f, 0.f, 0.f, 0.f);
                            const float mn = fmaxf(mx, redux_max(ml.x)), ref = mn == -INFINITY ? 0.f : mn, al = ex2(mx - ref);
                            const float wt = ex2(ml.x - ref);
                            float sl = ml.y * wt;
                            mx = mn;
#pragma unroll
                            for (int o = 16; o; o >>= 1) sl += __shfl_xor_sync(0xFFFFFFFFu, sl, o);
                            all = fmaf(all, al, sl);
                            o4.x *= al;
                            o4.y *= al;
                            o4.z *= al;
                            o4.w *= al;
#pragma unroll
                            for (int c = 0; c < kJoin; ++c) {
                                const float f = __shfl_sync(0xFFFFFFFFu, wt, c);
                                o4.x = fmaf(v[c].x, f, o4.x);
                                o4.y = fmaf(v[c].y, f, o4.y);
                                o4.z = fmaf(v[c].z, f, o4.z);
                                o4.w = fmaf(v[c].w, f, o4.w);
                            }
                        }
                        const float inv = all == 0.f ? 0.f : 1048576.f / all;
                        *reinterpret_cast<uint2*>(out + r * kHeadDim + 4 * lane) =
                            make_uint2(pack_two<T>(o4.x * inv, o4.y * inv), pack_two<T>(o4.z * inv, o4.w * inv));
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

template <typename T, int NT, int GP, bool PAIRED>
int launch(const DecArgs& d, const CUtensorMap& map, int grid, cudaStream_t s) {
    auto kern = fp8_decode_kernel<T, NT, GP, PAIRED>;
    static int done[64] = {};
    const cudaError_t e = ensure_smem_limit(kern, DecLayout<NT, GP>::smem, done);
    if (e != cudaSuccess) return (int)e;
    return (int)launch_programmatic(kern, dim3((unsigned)grid), dim3(kDecThreads), (size_t)DecLayout<NT, GP>::smem, s, d, map);
}

// Query heads go in parts of 8 or 16 columns: 8 where they suffice (fewer exponentials per token).
int part_of(int group) { return group <= 8 ? 8 : 16; }

// The workspace: the partials, whose size does not depend on the call, and the counters behind them, so that calls of
// all shapes find every counter at zero where an earlier one left it.
size_t partial_bytes(const Fp8Geometry& g) {
    return ((size_t)(g.num_sms > 0 ? g.num_sms : 1) * 2 * kPartFloats * sizeof(float) + 255) / 256 * 256;
}
size_t counter_bytes(int batch, int hkv, int group) {
    const int gp = part_of(group);
    return ((size_t)batch * hkv * ((group + gp - 1) / gp) * sizeof(unsigned) + 255) / 256 * 256;
}

int64_t most_tiles(const Fp8Geometry& g, int batch, int group, int max_blocks) {
    const int gp = part_of(group);
    const int64_t items = (int64_t)batch * g.hkv * ((group + gp - 1) / gp), per = ((int64_t)max_blocks * g.bs + kTile - 1) / kTile;
    return items > INT_MAX ? INT64_MAX : items * per;
}

}  // namespace

bool fp8_decode_counts(const Fp8Geometry& g, int batch, int group, int max_blocks) {
    return most_tiles(g, batch, group, max_blocks) < INT_MAX;
}

size_t fp8_decode_workspace(const Fp8Geometry& g, int batch, int group) {
    return partial_bytes(g) + counter_bytes(batch, g.hkv, group);
}

size_t fp8_decode_counters_at(const Fp8Geometry& g) { return partial_bytes(g); }

int launch_fp8_decode(const Fp8AttnArgs& a, const CUtensorMap& map, void* workspace, void* stream) {
    DecArgs d{};
    d.a = a;
    const int gp = part_of(a.group);
    d.nsub = (a.group + gp - 1) / gp;
    d.partials = static_cast<float*>(workspace);
    d.counters = reinterpret_cast<unsigned*>(static_cast<char*>(workspace) + partial_bytes(a.g));
    d.stall_cycles = test_stall_cycles();
    const int64_t most = most_tiles(a.g, a.b.batch, a.group, a.b.max_blocks);
    const int grid = (int)(most < a.g.num_sms ? most : a.g.num_sms);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool paired = a.g.bs == 16;
    if (a.dtype == TQ_BF16) {
        if (gp == 8) return paired ? launch<__nv_bfloat16, 2, 8, true>(d, map, grid, s) : launch<__nv_bfloat16, 2, 8, false>(d, map, grid, s);
        return paired ? launch<__nv_bfloat16, 2, 16, true>(d, map, grid, s) : launch<__nv_bfloat16, 2, 16, false>(d, map, grid, s);
    }
    if (gp == 8) return paired ? launch<__half, 3, 8, true>(d, map, grid, s) : launch<__half, 3, 8, false>(d, map, grid, s);
    return paired ? launch<__half, 3, 16, true>(d, map, grid, s) : launch<__half, 3, 16, false>(d, map, grid, s);
}

}  // namespace tq
