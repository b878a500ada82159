// Causal attention of a ragged batch's new tokens over the 8-bit paged cache,
// on the tensor cores.
//
// A unit is 256 query rows of one sequence and KV head (row = token * group +
// query head in the group), two tiles A and B of 128 rows; a CTA takes a unit,
// or one of its splits over the tokens, 128 tokens a step:
//   S [128 rows x 128 tokens] = Q . K^T    kind::f8f6f4
//   O [128 rows x 128 dims]  += P . V      kind::f16 with bf16 operands
// K goes to the tensor cores as its codes.  A query row is split into e4m3
// terms that add up in one accumulator, x = h1 + h2 (+ h3), scaled so that its
// largest element lies in (224, 448]: 2 terms are a bf16 query's 8 bits (3 an
// fp16 one's 11), down to steps of 2^-9, 2^-17.8 of the row's largest element.
// Two passes of fp8 cost what one of bf16 does, and K needs no conversion.
// V's codes times their block's scale are exact in bf16, and bf16 weights keep
// their relative precision at any size, so a weight far below a dominating one
// (or on a block with a small scale) counts with its own bits; fp8 weights in
// one accumulator would not do that.  Weights round to bf16 (2^-8) for bf16
// queries; fp16 ones add the remainder as a second bf16 operand (2^-16).
//
// Bounds, per 128 tokens and 256 rows: tensor cores 1024 (QK, 2 terms) + 1024
// (PV) cycles, exponentials 1024 at 32 a cycle, shared memory about 2200 (both
// operands of QK, V's conversion).  Hence two row tiles that take turns: the
// tensor cores work on one while the softmax of the other runs, and both use
// the same K and V.
//
// Warps: 0-3 softmax of A, 4-7 of B (thread = row), 8-11 V's conversion (these
// twelve split the queries first), 12 TMA, 13 MMA, 14 scales.  Tensor memory:
// S_A, S_B (their weights overwrite them), O_A, O_B, 128 columns each.  O is
// rescaled in place where a row's reference rises, which hardly happens after
// the first step.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>

#include "tq_fp8.cuh"
#include "tq_fp8_tc.cuh"

namespace tq {
namespace {

constexpr int kRowsPerTile = 128;
constexpr int kUnitRows = 256;
constexpr int kTok = 128;                    // tokens of a step
constexpr int kThreads = 512;
constexpr int kMetaRing = 4;
constexpr int kSoftRegs = 184, kOtherRegs = 72;  // of the two softmax warpgroups and the two others, out of 128 each
constexpr float kHeadroom = 24.f;

template <int NT>
struct PreLayout {
    static constexpr int KS = NT == 2 ? 3 : 2;          // stages of keys
    static constexpr int q = 0;                         // [2 tiles][NT][128 rows][128 B], 128-byte swizzle
    static constexpr int k = q + 2 * NT * 16384;        // [KS][128 tokens][128 B], 128-byte swizzle
    static constexpr int v = k + KS * 16384;            // [2][128 tokens][128 B] codes, 128-byte swizzle
    static constexpr int vb = v + 2 * 16384;            // [2] bf16 operand: 8 x 8 core matrices, MN-major
    static constexpr int meta = vb + 2 * 32768;         // [ring]: key scales [8], value scales [8] of 16 tokens each
    static constexpr int okm = meta + kMetaRing * 64;   // [ring]: groups of 16 tokens that are there
    static constexpr int bars = okm + kMetaRing * 4;
    static constexpr int nbars = 2 + 2 * KS + 4 + 4 + 6 + 2 * kMetaRing + 1;
    static constexpr int misc = bars + nbars * 8;       // tensor memory's address; the first token with a NaN in any dim
    static constexpr int mult = misc + 16;              // [256] rows' score multipliers
    static constexpr int nan = mult + 256 * 4;          // [128 dims] the first token of this split whose value is a NaN there
    static constexpr int total = nan + kHeadDim * 4;
    static constexpr int smem = total + 1008;           // the base is rounded up to 1 KB, from 16 bytes at least
    static_assert(k % 1024 == 0 && v % 1024 == 0 && vb % 1024 == 0 && meta % 16 == 0 && bars % 8 == 0, "alignment");
    static_assert(smem <= kSmemLimit, "prefill does not fit in shared memory");
};
// V's operand: 8 tokens x 8 dims core matrices of 128 bytes, token groups 128 bytes apart, dim groups 2048; the dims of
// every four in the order 0, 2, 1, 3, as a word of codes is taken apart with the fewest instructions
constexpr uint32_t kVLbo = 128, kVSbo = 2048;

struct PreArgs {
    Fp8AttnArgs a;
    int tpt;              // tokens of a row tile: 128 / group
    int splits;
    float* partials;      // [units][hkv][splits][256][128], unnormalised (splits > 1)
    float2* ml;           // [units][hkv][splits][256] (maximum, sum)
    long long stall_cycles;
};

// A unit: its sequence, packed rows and positions.
struct Unit {
    int b, n, first;   // sequence, its new tokens, the unit's first among them
    int64_t row0;      // packed row of the sequence's first new token
    int start;         // its position (a negative one is flagged, its rows attend to nothing)
    bool live;
};
__device__ __forceinline__ Unit find_unit(const Fp8Batch& b, int u, int step) {
    Unit x;
    const Fp8Seq s = fp8_seq_of_unit(b, u, step, 1);
    x.b = s.b;
    x.n = s.n;
    x.row0 = s.row0;
    const int64_t first = ((int64_t)u - s.base) * step;
    x.live = first >= 0 && first < x.n;
    x.first = x.live ? (int)first : 0;
    x.start = s.start;
    return x;
}

__device__ __forceinline__ void pre_sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Eight columns of tensor memory.
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Notes the codes of NaN among the 32 tokens of a step that converter `cw` has: in `first` the first token of each dim that
// holds one, in `any` of all dims, counted from the split's first token (t0 is the step's).  Rare, and out of line: inlined
// it made the loop that calls it slower (a chunk of 4096 at 12288: 1368 us against 1345).
__device__ __noinline__ void note_nan(const uint8_t* codes, const int* exps, int* first, int* any, int cw, int t0) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int i = lane; i < 32 * kHeadDim; i += 32) {
        const int t = cw * 32 + (i >> 7), d = i & 127;
        const uint8_t code = codes[t * 128 + (((d >> 4) ^ (t & 7)) << 4) + (d & 15)];
        if ((code & 127) == 127 && exps[t >> 4] != INT_MIN) {
            atomicMin(first + d, t0 + t);
            atomicMin(any, t0 + t);
        }
    }
}

template <typename T, int NT, int NP>  // NP: bf16 operands of the weights
__global__ void __launch_bounds__(kThreads, 1) fp8_prefill_kernel(const PreArgs A, const __grid_constant__ CUtensorMap map) {
    using L = PreLayout<NT>;
    extern __shared__ uint8_t raw[];
    uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(sm);
    const Fp8Geometry& g = A.a.g;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto bar = [&](int i) { return sb + L::bars + 8 * i; };
    // queries of a tile stored; keys landed, free; codes of values landed, free; operand of values stored, free;
    // scores, weights and output of a row tile; scales stored, free; one that nothing arrives on
    constexpr int bQ = 0, bK = 2, bKe = bK + L::KS, bV = bKe + L::KS, bVe = bV + 2, bB = bVe + 2, bBe = bB + 2, bS = bBe + 2,
                  bP = bS + 2, bO = bP + 2, bM = bO + 2, bMe = bM + kMetaRing, bNever = bMe + kMetaRing;
    static_assert(bNever + 1 == L::nbars, "barriers");

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(bQ + i), 6);
            mbar_init(bar(bV + i), 1);
            mbar_init(bar(bVe + i), 4);
            mbar_init(bar(bB + i), 4);
            mbar_init(bar(bBe + i), 1);
            mbar_init(bar(bS + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(bP + i), 4);
            mbar_init(bar(bO + i), 1);
        }
        for (int i = 0; i < L::KS; ++i) {
            mbar_init(bar(bK + i), 1);
            mbar_init(bar(bKe + i), 1);
        }
        for (int i = 0; i < kMetaRing; ++i) {
            mbar_init(bar(bM + i), 1);
            mbar_init(bar(bMe + i), 1);
        }
        mbar_init(bar(bNever), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    int* nan_s = reinterpret_cast<int*>(sm + L::nan);
    int* any_nan = reinterpret_cast<int*>(sm + L::misc + 4);
    if (tid < kHeadDim) nan_s[tid] = INT_MAX;
    if (tid == kHeadDim) *any_nan = INT_MAX;
    if (warp == 12 && lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(&map) : "memory");
    if (warp == 13) tc::tmem_alloc<512>(sb + L::misc);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + L::misc);
    // (The next grid is not let in early: CTAs that wait for this one's end cost it more than their start takes, 117 us
    // against 106 for a ragged fp16 batch of 300 units called again and again, 76 against 72 for 64 tokens at 32704.)
    grid_dependency_wait();

    // ---- the unit, its row tiles and this split's tokens ----
    // heads and splits run fastest; the units go from the last back, as those attend to the most tokens
    const int split = blockIdx.x % A.splits, uh = blockIdx.x / A.splits;
    const int h = uh % g.hkv;
    const int u_all = (int)(gridDim.x / A.splits / g.hkv);
    const int unit = u_all - 1 - uh / g.hkv;
    const Unit U = find_unit(A.a.b, unit, 2 * A.tpt);
    const int G = A.a.group;
    const int64_t cap = (int64_t)A.a.b.max_blocks * g.bs;
    // tokens that a row tile's last row sees, and how many steps that takes
    auto steps_of = [&](int x) {
        const int t0 = U.first + x * A.tpt;
        if (!U.live || t0 >= U.n) return 0;
        const int64_t end = U.start < 0 ? 0 : min((int64_t)U.start + min(U.n, t0 + A.tpt), cap);
        return max(1, (int)((end + kTok - 1) / kTok));
    };
    const int nA = steps_of(0), nB = steps_of(1), nt = max(nA, nB);
    // (fewer than 2^25 steps and at most 64 splits)
    const int s0 = (int)((uint32_t)nt * split / A.splits), s1 = (int)((uint32_t)nt * (split + 1) / A.splits);
    const int cnt = s1 - s0;
    const int cA = min(max(nA - s0, 0), cnt), cB = min(max(nB - s0, 0), cnt);

    bool bad = false;
    auto wait = [&](int i, uint32_t parity) {
        if (!bad && !mbar_wait(bar(i), parity)) bad = true;
    };
    // id of the block that holds tokens 16 j .. of step u, or -1 (past the end) or -2 (not in the pool)
    auto block_of = [&](int u, int j) {
        const int64_t p = (int64_t)(s0 + u) * kTok + 16 * j;
        const int64_t end = min((int64_t)U.start + min(U.n, U.first + 2 * A.tpt), cap);
        if (U.start < 0 || p >= end) return -1;
        const int id = __ldg(A.a.b.block_table + (int64_t)U.b * A.a.b.max_blocks + (p >> g.bs_shift));
        return id >= 0 && id < g.num_blocks ? id : -2;
    };

    if (U.live && warp < 12) {
        // The tiles' queries in e4m3 terms, 24 rows a softmax warp and 16 a converter, before the registers are shared
        // out: two rows at a time (half a warp each, 8 elements a lane), all loads in flight at once.  The split then goes
        // through them by shifting, in a loop small enough for a cold instruction cache.
        const bool soft = warp < 8;
        const int x = soft ? warp >> 2 : (warp - 8) >> 1;
        const int base = soft ? (warp & 3) * 24 : 96 + (warp & 1) * 16, pairs = soft ? 12 : 8;
        if ((x ? cB : cA) > 0) {
            float* mult_s = reinterpret_cast<float*>(sm + L::mult) + x * 128;
            const int sub = lane >> 4, col = lane & 15, first_row = base + sub;
            int row_tok = U.first + x * A.tpt + first_row / G, row_g = first_row % G;
            constexpr int kBatch = 4;
            uint4 raw_q[12];
#pragma unroll
            for (int i = 0; i < 12; ++i) {
                const bool in = i < pairs && first_row + 2 * i < A.tpt * G && row_tok < U.n;
                const T* q = static_cast<const T*>(A.a.q) + (U.row0 + row_tok) * A.a.q_token +
                             ((int64_t)h * G + row_g) * A.a.q_head + 8 * col;
                raw_q[i] = in ? __ldg(reinterpret_cast<const uint4*>(q)) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (++row_g == G) {
                        row_g = 0;
                        ++row_tok;
                    }
            }
#pragma unroll 1
            for (int r0 = first_row; r0 < base + 2 * pairs; r0 += 2 * kBatch) {
                uint32_t words[kBatch][4];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    words[i][0] = raw_q[i].x;
                    words[i][1] = raw_q[i].y;
                    words[i][2] = raw_q[i].z;
                    words[i][3] = raw_q[i].w;
                }
                Fp8Split<T, 16, kBatch> split(words);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    uint32_t code[kBatch][2];
                    split.template term<0>(code);
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const int row = r0 + 2 * i;
                        *reinterpret_cast<uint2*>(sm + L::q + (x * NT + j) * 16384 + row * 128 + (((col >> 1) ^ (row & 7)) << 4) +
                                                  (col & 1) * 8) = make_uint2(code[i][0], code[i][1]);
                    }
                }
                float factors = 0.f;  // a query that is not finite makes its own row NaN
#pragma unroll
                for (int i = 0; i < kBatch; ++i) factors = col == i ? split.factor(i, A.a.sm_scale_log2) : factors;
                if (col < kBatch) mult_s[r0 + 2 * col] = factors;
#pragma unroll
                for (int i = 0; i + kBatch < 12; ++i) raw_q[i] = raw_q[i + kBatch];
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(bQ + x));
        }
        __syncwarp();
    }
    if (!U.live) {
        // no such unit
    } else if (warp < 8) {
        // ================= softmax: thread = query row =================
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        const int x = warp >> 2, quad = warp & 3;      // row tile, lane quarter
        const int r = quad * 32 + lane;
        const int tok = U.first + x * A.tpt + r / G;   // new token of the sequence
        const bool there = r < A.tpt * G && tok < U.n;
        const int steps = x ? cB : cA;
        // the last token that the row sees, and the tile's first row, counted from this split's first token
        auto relative = [&](int t) {
            return (int)max((int64_t)-1, min((int64_t)U.start + t - (int64_t)s0 * kTok, (int64_t)cnt * kTok - 1));
        };
        const int pos = relative(tok), pos0 = relative(U.first + x * A.tpt);
        const uint32_t my = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t tS = my + x * 128, tO = my + 256 + x * 128;
        float* mult_s = reinterpret_cast<float*>(sm + L::mult) + x * 128;
        bool empty = false;
        if (A.stall_cycles > 0 && (split & 1)) {
            empty = !mbar_wait_for(bar(bNever), 0, A.stall_cycles);
            if (empty && r == 0) flag(A.a.status, TQ_FLAG_TIMEOUT);
        }
        if (steps > 0) wait(bQ + x, 0);
        __syncwarp();
        const float mult = steps > 0 ? mult_s[r] : 0.f;
        // the row's place in the output waits there meanwhile: registers are what the loop lacks
        reinterpret_cast<int*>(mult_s)[r] = there ? (int)(U.row0 + tok) : -1;
        // Weights are 2^(l - m) against a reference m that is put 2^24 above the row's maximum and raised again only when
        // the 128 weights of a step add up to more than 128 (some weight is above 1 then; where it is not raised each is at
        // most 128): bf16 and fp32 keep their precision at any size, the sum is needed anyway, and no maximum is formed
        // otherwise (which took a fifth of the step).  The scores are still in tensor memory then, and the step is weighed again.  A row that has seen no
        // token yet has no reference.
        float m = there ? -INFINITY : 0.f;
        uint64_t acc = f2_pack(0.f, 0.f);
        for (int u = 0; u < steps; ++u) {
            const int mi = u % kMetaRing;
            wait(bM + mi, (u / kMetaRing) & 1);
            const int ok = *reinterpret_cast<const int*>(sm + L::okm + mi * 4);
            const float* ks = reinterpret_cast<const float*>(sm + L::meta + mi * 64);
            auto factor = [&](int j) {  // of tokens 16 j .. (a masked score of -inf stays one; NaN stays NaN)
                const float y = ks[j] * mult;
                return y < 1e-37f ? 1e-37f : y;
            };
            const int limit = pos - u * kTok;  // the row sees tokens 0 .. limit of the tile
            const bool masked = ok != 0xFF || u * kTok + kTok - 1 > pos0;  // a mask begins here, or a block is missing
            wait(bS + x, u & 1);
            tc::fence_after_sync();
            __syncwarp();
            constexpr int kLo = NP == 2 ? 64 : 1;
            auto load = [&](uint32_t (&s)[128]) {
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 4; ++c) tc::ld_32x32b_x32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * c));
                tc::wait_ld();
#pragma unroll
                for (int c = 0; c < 4; ++c) tc::reg_fence(*reinterpret_cast<uint32_t(*)[32]>(s + 32 * c));
                if (masked) {
#pragma unroll
                    for (int j = 0; j < 128; ++j)
                        if (j > limit || !((ok >> (j >> 4)) & 1)) s[j] = 0xFF800000u;
                }
            };
            auto raise = [&](const uint32_t (&s)[128]) {
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < 8; ++j) {  // the scales are positive: maximum first, scale after
                    float y = -INFINITY;
#pragma unroll
                    for (int k = 0; k < 16; ++k) y = fmaxf(y, __uint_as_float(s[16 * j + k]));
                    mx = fmaxf(mx, y == -INFINITY ? y : y * factor(j));
                }
                const bool rise = mx > m;
                const float fac = rise ? ex2(m - (mx + kHeadroom)) : 1.f;
                if (rise) m = mx + kHeadroom;
                acc = f2_mul(acc, f2_pack(fac, fac));
                if (u > 0 && __any_sync(0xFFFFFFFFu, rise)) {
                    wait(bO + x, (u - 1) & 1);  // the output of the step before is complete
                    tc::fence_after_sync();
                    __syncwarp();
#pragma unroll 1
                    for (int c = 0; c < 16; ++c) {
                        uint32_t o[8];
                        tmem_ld<8>(tO + 8 * c, o);
                        tmem_ready<8>(o);
#pragma unroll
                        for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * fac);
                        tmem_st8(tO + 8 * c, o);
                    }
                    tc::wait_st();
                }
            };
            // the scores' weights, packed into the first half of s (their remainders into lo), and their sum
            auto weigh = [&](uint32_t (&s)[128], uint32_t (&lo)[kLo]) {
                const float ref = m == -INFINITY ? 0.f : m;
                const uint64_t neg = f2_pack(-ref, -ref);
                uint64_t part = f2_pack(0.f, 0.f), part2 = part;
                uint64_t f2;
#pragma unroll
                for (int j = 0; j < 128; j += 2) {
                    if (j % 16 == 0) {
                        const float y = factor(j >> 4);
                        f2 = f2_pack(y, y);
                    }
                    float a, b;
                    // a masked score is -inf: its product with a positive scale too
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), f2, neg), a, b);
                    a = ex2(a);
                    b = ex2(b);
                    if (j & 2) part = f2_add(part, f2_pack(a, b));
                    else part2 = f2_add(part2, f2_pack(a, b));
                    s[j / 2] = pack_bf16(a, b);
                    if constexpr (NP == 2)
                        lo[j / 2] = pack_bf16(a - __uint_as_float(s[j / 2] << 16), b - __uint_as_float(s[j / 2] & 0xFFFF0000u));
                }
                return f2_add(part, part2);
            };
            auto store = [&](uint32_t (&s)[128], uint32_t (&lo)[kLo]) {
                __syncwarp();
                tc::st_32x32b_x32(tS, *reinterpret_cast<uint32_t(*)[32]>(s));
                tc::st_32x32b_x32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
                if constexpr (NP == 2) {
                    tc::st_32x32b_x32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(lo));
                    tc::st_32x32b_x32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(lo + 32));
                }
                tc::wait_st();
            };
            bool again = __any_sync(0xFFFFFFFFu, m == -INFINITY);
            if (!again) {
                uint32_t s[128], lo[kLo];
                load(s);
                const uint64_t part = weigh(s, lo);
                float a, b;
                f2_unpack(part, a, b);
                again = __any_sync(0xFFFFFFFFu, a + b > 128.f);
                if (!again) {
                    acc = f2_add(acc, part);
                    store(s, lo);
                }
            }
            if (again) {  // the scores are still in tensor memory
                uint32_t s[128], lo[kLo];
                load(s);
                raise(s);
                acc = f2_add(acc, weigh(s, lo));
                store(s, lo);
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(bP + x));
        }
        // ---- the rows' end ----
        if (bad && !empty) {
            flag(A.a.status, TQ_FLAG_TIMEOUT);
            empty = true;
        }
        float sum;
        {
            float a, b;
            f2_unpack(acc, a, b);
            sum = a + b;
        }
        if (steps > 0) {
            wait(bO + x, (steps - 1) & 1);
            tc::fence_after_sync();
            __syncwarp();
        }
        const int row = reinterpret_cast<const int*>(mult_s)[r];
        int cta;
        asm volatile("mov.u32 %0, %%ctaid.x;" : "=r"(cta));  // (read again, not held)
        const int uh2 = cta / A.splits, h2 = uh2 % A.a.g.hkv;
        // A thread has a row of its own in tensor memory; rows of 16-byte pieces leave through shared memory (the place
        // of the tile's queries, whose last reader is done), so that a store takes two rows and not 32 pieces 4 KB apart
        // (which cost 4000 cycles of the unit's end).
        const uint32_t stage = sb + L::q + x * NT * 16384 + quad * 8192;
        auto leave = [&](char* mine) {  // 256 bytes of every row to `mine` of its thread (null: nowhere)
            __syncwarp();
#pragma unroll (NT == 2 ? 4 : 1)
            for (int i = 0; i < 16; ++i) {
                const int from = 2 * i + (lane >> 4);
                const uint64_t to = __shfl_sync(0xFFFFFFFFu, (unsigned long long)mine, from);
                const uint4 v = lds128(stage + from * 256 + (((lane & 15) ^ (from & 7)) << 4));
                if (to) *reinterpret_cast<uint4*>(to + 16 * (lane & 15)) = v;
            }
            __syncwarp();
        };
        auto piece = [&](int i) { return stage + lane * 256 + ((i ^ (lane & 7)) << 4); };
        auto swap_dims = [](uint32_t (&o)[16]) {  // the columns are dims 0, 2, 1, 3 of every four
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const uint32_t y = o[i + 1];
                o[i + 1] = o[i + 2];
                o[i + 2] = y;
            }
        };
        // a dim is NaN from the first token on that has a NaN there: in the staged rows, dims d0 .. of `size` bytes
        auto spoil = [&](int d0, int n, int size) {
#pragma unroll 1
            for (int d = *any_nan <= pos ? 0 : n; d < n; ++d)
                if (nan_s[d0 + d] <= pos) {
                    const uint32_t at = piece(d * size >> 4) + (d * size & 15);
                    if (size == 2) asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((unsigned short)0x7FFF) : "memory");
                    else asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(0x7FFFFFFF) : "memory");
                }
        };
        if (A.splits == 1) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            T* out = static_cast<T*>(A.a.out) + ((int64_t)row * A.a.hq + (int64_t)h2 * A.a.group + r % A.a.group) * kHeadDim;
            if (steps > 0) {
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                    uint32_t o[16];
                    tmem_ld<16>(tO + 16 * c, o);
                    tmem_ready<16>(o);
                    swap_dims(o);
                    uint32_t w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        w[i] = sum == 0.f ? 0u : pack_two<T>(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
                    pre_sts128(piece(2 * c), w[0], w[1], w[2], w[3]);
                    pre_sts128(piece(2 * c + 1), w[4], w[5], w[6], w[7]);
                }
                spoil(0, kHeadDim, 2);
                leave(row >= 0 && !empty ? reinterpret_cast<char*>(out) : nullptr);
            }
        } else {
            const int u_all2 = (int)(gridDim.x / A.splits / A.a.g.hkv);
            const int64_t slot = ((int64_t)(u_all2 - 1 - uh2 / A.a.g.hkv) * A.a.g.hkv + h2) * A.splits + cta % A.splits;
            const int64_t at = slot * kUnitRows + x * kRowsPerTile + r;
            const bool none = steps == 0 || empty || sum == 0.f;
            A.ml[at] = make_float2(none ? -INFINITY : m, none ? 0.f : sum);
            char* part = row >= 0 && !none ? reinterpret_cast<char*>(A.partials + at * kHeadDim) : nullptr;
            if (steps > 0)
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t o[16];
                        tmem_ld<16>(tO + 64 * half + 16 * c, o);
                        tmem_ready<16>(o);
                        swap_dims(o);
#pragma unroll
                        for (int i = 0; i < 4; ++i) pre_sts128(piece(4 * c + i), o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                    spoil(64 * half, 64, 4);
                    leave(part ? part + 256 * half : nullptr);
                }
        }
    } else if (warp < 12) {
        // ================= V: codes to bf16, times the block's scale =================
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        const int cw = warp - 8;
        for (int u = 0; u < cnt; ++u) {
            const int b = u & 1, mi = u % kMetaRing;
            wait(bM + mi, (u / kMetaRing) & 1);
            wait(bV + b, (u >> 1) & 1);
            if (u > 1) wait(bBe + b, ((u - 2) >> 1) & 1);
            const int* vs = reinterpret_cast<const int*>(sm + L::meta + mi * 64 + 32);
            const uint32_t src = sb + L::v + b * 16384, dst = sb + L::vb + b * 32768;
            uint32_t most = 0;  // largest magnitudes, in either half: a NaN's is 0x7F0
            // a warp converts 32 tokens: 8 of them by 4 pieces of 16 codes at a time (unrolled by measurement: twice is 2 %
            // faster than once with two query terms, 4 % slower with three)
#pragma unroll (NT == 2 ? 2 : 1)
            for (int i = 0; i < 8; ++i) {
                const int t = cw * 32 + (i >> 1) * 8 + (lane & 7), c = (i & 1) * 4 + (lane >> 3);
                const uint4 v4 = lds128(src + t * 128 + ((c ^ (t & 7)) << 4));
                const uint32_t w[4] = {v4.x, v4.y, v4.z, v4.w};
                const int e = vs[t >> 4];  // exponent of the value scale, or INT_MIN where there is no block
                // e4m3's fields moved into bf16's read as the value times 2^-120 (subnormals too)
                const int e1 = min(e + 120, 127);
                const uint32_t f1 = e == INT_MIN ? 0u : (uint32_t)(e1 + 127 > 254 ? 254 : e1 + 127) << 7;
                const uint32_t m1 = f1 | (f1 << 16);
                uint32_t o[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    // dims 0 and 2, 1 and 3 of the word's four: the operand's columns hold them in that order
                    const uint32_t even = (w[k] << 4) & 0x07F007F0u, odd = (w[k] >> 4) & 0x07F007F0u;
                    o[2 * k] = mul_bf16x2(((w[k] << 8) & 0x80008000u) | even, m1);
                    o[2 * k + 1] = mul_bf16x2((w[k] & 0x80008000u) | odd, m1);
                    most = __vimax3_u16x2(most, even, odd);
                }
                if (e > 7) {  // 2^(e + 120) is past bf16's range: the rest in a second product
                    const uint32_t f2 = (uint32_t)(e - 7 + 127) << 7, m2 = f2 | (f2 << 16);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        // codes of 256 and more times 2^120 are past bf16: its largest value instead, as an infinity would
                        // reach the rows that do not see the token (0 * inf is NaN)
                        o[k] = mul_bf16x2(o[k], m2);
                        o[k] = (o[k] & 0x80008000u) | __vminu2(o[k] & 0x7FFF7FFFu, 0x7F7F7F7Fu);
                    }
                }
                const uint32_t at = dst + (2 * c) * kVSbo + (t >> 3) * kVLbo + (t & 7) * 16;
                pre_sts128(at, o[0], o[1], o[2], o[3]);
                pre_sts128(at + kVSbo, o[4], o[5], o[6], o[7]);
            }
            // A NaN (0x7F or 0xFF: tq_fp8_write stores none, but a pool may come from elsewhere) is 480 in the operand, which
            // does no harm to the rows that do not see it; the rows' end makes it NaN for those that do.
            if (__any_sync(0xFFFFFFFFu, (most & 0xFFFFu) == 0x7F0u || (most >> 16) == 0x7F0u))
                note_nan(sm + L::v + b * 16384, vs, nan_s, any_nan, cw, u * kTok);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(bB + b));
                mbar_arrive(bar(bVe + b));
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 12) {
            // ================= TMA: lanes 0-7 the blocks' keys, 8-15 their values =================
            const int pages = kTok >> g.bs_shift, pg = lane & 7, side = (lane >> 3) & 1;
            const uint32_t bytes = (uint32_t)g.bs * kHeadDim;
            asm volatile("fence.proxy.async.global;" ::: "memory");  // the codes were written by ordinary stores
            const bool mine = lane < 16 && pg < pages;
            const int per = g.bs >> 4;  // groups of 16 tokens in a block
            int id = mine && cnt > 0 ? block_of(0, pg * per) : -1;
            int sent = 0;  // steps whose copies are issued: none behind one whose wait gave up
            for (int u = 0; u < cnt; ++u) {
                const int now = id;
                id = mine && u + 1 < cnt ? block_of(u + 1, pg * per) : -1;
                const int row = (int)((((int64_t)max(now, 0) * g.hkv + h) * 2 + side) << g.bs_shift);
                const unsigned kmask = __ballot_sync(0xFFFFFFFFu, now >= 0 && side == 0), vmask = __ballot_sync(0xFFFFFFFFu, now >= 0 && side == 1);
                const int ks = u % L::KS;
                if (u >= L::KS) wait(bKe + ks, (u / L::KS - 1) & 1);
                if (lane == 0) mbar_arrive_tx(bar(bK + ks), (uint32_t)__popc(kmask) * bytes);
                __syncwarp();
                if (now >= 0 && side == 0) tma_page(sb + L::k + ks * 16384 + pg * bytes, &map, row, bar(bK + ks));
                if (u > 1) wait(bVe + (u & 1), ((u - 2) >> 1) & 1);
                sent = u + 1;
                if (lane == 0) mbar_arrive_tx(bar(bV + (u & 1)), (uint32_t)__popc(vmask) * bytes);
                __syncwarp();
                if (now >= 0 && side == 1) tma_page(sb + L::v + (u & 1) * 16384 + pg * bytes, &map, row, bar(bV + (u & 1)));
                if (now == -2) flag(A.a.status, TQ_FLAG_BAD_SLOT);
                if (u > 1 && __any_sync(0xFFFFFFFFu, bad)) break;
            }
            if (lane == 0 && (U.start < 0 || (int64_t)U.start + min(U.n, U.first + 2 * A.tpt) > cap)) flag(A.a.status, TQ_FLAG_BAD_SLOT);
            // copies may be in flight where a wait gave up: they end (again with a limit) before the memory is given back
            for (int u = max(0, sent - L::KS); u < sent; ++u) mbar_wait(bar(bK + u % L::KS), (u / L::KS) & 1);
            for (int u = max(0, sent - 2); u < sent; ++u) mbar_wait(bar(bV + (u & 1)), (u >> 1) & 1);
        } else if (warp == 14) {
            // ================= scales of every 16 tokens =================
            for (int u = 0; u < cnt; ++u) {
                const int mi = u % kMetaRing;
                const int id = lane < 8 ? block_of(u, lane) : -1;
                float2 s = make_float2(0.f, 0.f);
                if (id >= 0) s = __ldg(reinterpret_cast<const float2*>(g.scales + ((int64_t)id * g.hkv + h) * 2));
                const unsigned ok = __ballot_sync(0xFFFFFFFFu, id >= 0);
                if (u >= kMetaRing) wait(bMe + mi, (u / kMetaRing - 1) & 1);
                if (lane < 8) {
                    // where there is no block any positive scale does: the scores are masked
                    reinterpret_cast<float*>(sm + L::meta + mi * 64)[lane] = id >= 0 ? s.x : 1.f;
                    reinterpret_cast<int*>(sm + L::meta + mi * 64 + 32)[lane] = id >= 0 ? fp8_exp_of(s.y) : INT_MIN;
                }
                if (lane == 0) *reinterpret_cast<int*>(sm + L::okm + mi * 4) = (int)ok;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(bM + mi));
            }
        } else if (warp == 13) {
            // ================= MMA: QK A(u), PV B(u - 1), QK B(u), PV A(u) =================
            const bool issues = elect_one();
            const uint64_t d_q = desc_rows(sb + L::q, 1024), d_k = desc_rows(sb + L::k, 1024),
                           d_v = tc::smem_desc(sb + L::vb, kVLbo, kVSbo);
            constexpr uint32_t idesc_v = tc::idesc_bf16_f32(128, 128) | (1u << 16);
            auto scores = [&](int x, int ks) {
                tc::fence_after_sync();
                if (issues) {
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_f8_ss(tmem + x * 128, d_q + (x * NT + j) * 1024 + 2 * k, d_k + ks * 1024 + 2 * k, idesc_f8(128, false),
                                      j > 0 || k > 0);
                    tc::commit(bar(bS + x));
                }
                __syncwarp();
            };
            auto values = [&](int x, int u) {
                wait(bB + (u & 1), (u >> 1) & 1);
                wait(bP + x, u & 1);
                __syncwarp();
                tc::fence_after_sync();
                if (issues) {
#pragma unroll
                    for (int j = 0; j < NP; ++j)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            tc::mma_f16_ts(tmem + 256 + x * 128, tmem + x * 128 + 64 * j + 8 * k, d_v + (u & 1) * 2048 + 16 * k, idesc_v,
                                           u > 0 || j > 0 || k > 0);
                    tc::commit(bar(bO + x));
                }
                __syncwarp();
            };
            auto release = [&](int u) {  // both tiles' values of step u are issued
                if (issues) {
                    tc::commit(bar(bBe + (u & 1)));
                    tc::commit(bar(bMe + u % kMetaRing));
                }
                __syncwarp();
            };
            if (cA > 0) wait(bQ, 0);
            if (cB > 0) wait(bQ + 1, 0);
            for (int u = 0; u < cnt; ++u) {
                const int ks = u % L::KS;
                wait(bK + ks, (u / L::KS) & 1);
                __syncwarp();
                if (u < cA) scores(0, ks);
                if (u > 0) {
                    if (u - 1 < cB) values(1, u - 1);
                    release(u - 1);
                }
                if (u < cB) scores(1, ks);
                if (issues) tc::commit(bar(bKe + ks));
                __syncwarp();
                if (u < cA) values(0, u);
            }
            if (cnt > 0) {
                if (cnt - 1 < cB) values(1, cnt - 1);
                release(cnt - 1);
                // products may be in flight where a wait gave up: they too end before the memory is given back
                mbar_wait(bar(bBe + ((cnt - 1) & 1)), ((cnt - 1) >> 1) & 1);
            }
        }
    }
    if (bad && lane == 0) flag(A.a.status, TQ_FLAG_TIMEOUT);
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 13) {
        tc::fence_after_sync();
        tc::tmem_dealloc<512>(tmem);
    }
}

// Joins the splits of every row, one warp per row, in their order.
template <typename T>
__global__ void __launch_bounds__(256) fp8_prefill_join_kernel(const PreArgs A) {
    const int lane = threadIdx.x & 31;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int r = (int)(item % kUnitRows);
    const int64_t uh = item / kUnitRows;
    const int h = (int)(uh % A.a.g.hkv), unit = (int)(uh / A.a.g.hkv);
    if (unit >= fp8_units(A.a.b.num_tokens, A.a.b.batch, 2 * A.tpt, 1)) return;
    // the partials first: where they lie does not depend on the sequence (rows that do not exist are read, not used)
    const int64_t at = uh * A.splits * kUnitRows + r;
    float4 o4 = make_float4(0.f, 0.f, 0.f, 0.f);
    float all = 0.f, mx = -INFINITY;
    for (int s0 = 0; s0 < A.splits; s0 += 16) {
        const int n = min(16, A.splits - s0);
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < n) ml = A.ml[at + (int64_t)(s0 + lane) * kUnitRows];
        float4 v[16];
#pragma unroll
        for (int s = 0; s < 16; ++s)
            v[s] = s < n ? *(reinterpret_cast<const float4*>(A.partials + (at + (int64_t)(s0 + s) * kUnitRows) * kHeadDim) + lane)
                         : make_float4(0.f, 0.f, 0.f, 0.f);
        const float top = fmaxf(mx, redux_max(ml.x));
        const float ref = top == -INFINITY ? 0.f : top, fac = ex2(mx - ref);
        mx = top;
        all *= fac;
        o4.x *= fac;
        o4.y *= fac;
        o4.z *= fac;
        o4.w *= fac;
        const float w = ex2(ml.x - ref);
#pragma unroll
        for (int s = 0; s < 16; ++s) {
            const float ws = __shfl_sync(0xFFFFFFFFu, w, s), sum = __shfl_sync(0xFFFFFFFFu, ml.y, s);
            if (sum == 0.f) continue;  // nothing there, and nothing stored
            all = fmaf(sum, ws, all);
            o4.x = fmaf(v[s].x, ws, o4.x);
            o4.y = fmaf(v[s].y, ws, o4.y);
            o4.z = fmaf(v[s].z, ws, o4.z);
            o4.w = fmaf(v[s].w, ws, o4.w);
        }
    }
    const Unit U = find_unit(A.a.b, unit, 2 * A.tpt);
    const int x = r / kRowsPerTile, rr = r % kRowsPerTile, G = A.a.group;
    const int tok = U.first + x * A.tpt + rr / G;
    if (!U.live || rr >= A.tpt * G || tok >= U.n) return;
    const float inv = all == 0.f ? 0.f : 1.f / all;
    T* out = static_cast<T*>(A.a.out) + ((U.row0 + tok) * A.a.hq + (int64_t)h * G + rr % G) * kHeadDim;
    *(reinterpret_cast<uint2*>(out) + lane) = make_uint2(pack_two<T>(o4.x * inv, o4.y * inv), pack_two<T>(o4.z * inv, o4.w * inv));
}

int tokens_per_tile(int group) { return kRowsPerTile / group; }

// Splits over the tokens, where the units alone leave SMs idle.
int splits_of(const Fp8Geometry& g, int64_t num_tokens, int batch, int group) {
    const int step = 2 * tokens_per_tile(group);
    const int64_t units = ((num_tokens + step - 1) / step + (batch - 1) / 2) * g.hkv;  // about as many as there are
    const int64_t s = (g.num_sms > 0 ? g.num_sms : 1) / units;
    return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

template <typename T, int NT, int NP>
int launch(const PreArgs& p, const CUtensorMap& map, int64_t units, cudaStream_t s) {
    auto kern = fp8_prefill_kernel<T, NT, NP>;
    static int done[64] = {};
    cudaError_t e = ensure_smem_limit(kern, PreLayout<NT>::smem, done);
    if (e != cudaSuccess) return (int)e;
    // the warpgroups share out the registers that the block is launched with: a build that gave it fewer would wait for
    // the rest without end
    static const bool enough = [&] {
        cudaFuncAttributes f;
        return cudaFuncGetAttributes(&f, kern) == cudaSuccess && (f.numRegs + 7) / 8 * 8 * 2 >= kSoftRegs + kOtherRegs;
    }();
    if (!enough) return (int)cudaErrorInvalidConfiguration;
    e = launch_programmatic(kern, dim3((unsigned)(units * p.a.g.hkv * p.splits)), dim3(kThreads), (size_t)PreLayout<NT>::smem, s, p, map);
    if (e != cudaSuccess || p.splits == 1) return (int)e;
    return (int)launch_programmatic(fp8_prefill_join_kernel<T>, dim3((unsigned)(units * p.a.g.hkv * (kUnitRows / 8))), dim3(256), 0, s, p);
}

}  // namespace

bool fp8_prefill_counts(const Fp8Geometry& g, int64_t num_tokens, int batch, int group) {
    return fp8_units(num_tokens, batch, 2 * tokens_per_tile(group), 1) * g.hkv * (kUnitRows / 8) < INT_MAX;
}

size_t fp8_prefill_workspace(const Fp8Geometry& g, int64_t num_tokens, int batch, int group) {
    const int splits = splits_of(g, num_tokens, batch, group);
    if (splits == 1) return 256;
    const size_t rows = (size_t)fp8_units(num_tokens, batch, 2 * tokens_per_tile(group), 1) * g.hkv * splits * kUnitRows;
    return rows * (kHeadDim * sizeof(float) + sizeof(float2));
}

int launch_fp8_prefill(const Fp8AttnArgs& a, const CUtensorMap& map, void* workspace, void* stream) {
    PreArgs p{};
    p.a = a;
    p.tpt = tokens_per_tile(a.group);
    p.splits = splits_of(a.g, a.b.num_tokens, a.b.batch, a.group);
    const int64_t units = fp8_units(a.b.num_tokens, a.b.batch, 2 * p.tpt, 1);
    p.partials = static_cast<float*>(workspace);
    p.ml = reinterpret_cast<float2*>(p.partials + (size_t)units * a.g.hkv * p.splits * kUnitRows * kHeadDim);
    p.stall_cycles = test_stall_cycles();
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return a.dtype == TQ_BF16 ? launch<__nv_bfloat16, 2, 1>(p, map, units, s) : launch<__half, 3, 2>(p, map, units, s);
}

}  // namespace tq
