// Attention of trees of drafted tokens over the 8-bit paged cache, on the
// tensor cores.
//
// Node i of a sequence attends over the prefix (positions before `start`) and over
// the nodes j with bit j in its row of a mask:
//   out_i = sum_t w_t V_t / sum_t w_t,  w_t = exp(s_t - m),  t < start or bit (t - start) of mask_i
//   S [128 rows x 128 tokens] = Q . K^T    kind::f8f6f4, the query in two or three e4m3 terms, K as its codes
//   O [128 rows x 128 dims]  += P . V      kind::f16, weights as bf16 and their remainders as bf16, V's codes times
//                                          their scale converted to bf16
// The operands are those of the causal kernel for chunks; what differs is that all rows of a tree see the
// whole prefix, that there are few of them, and that bf16 queries' weights keep their remainders too: a
// weight rounded to 8 bits puts three times the output's own rounding into rows whose values cancel.
//
// A unit is up to 256 query rows of one sequence and KV head (row = token * group + query
// head in the group): one row tile of 128 where that is enough (16 nodes of 8 query
// heads), else two that see the same tokens.  A turn is one row tile over one tile of 128
// tokens, and the tensor cores work on the scores of the next turn or two while the
// softmax of this one runs.  Eight warps share it, each half of them (a thread a row) with
// every other turn: with two row tiles a half has one of them, with one the halves take
// every other token tile of the same rows and hand the output's reference on.  References are
// whole numbers, so that what was weighed against another one follows by a power of two.
// Against all eight warps on every turn (64 tokens a thread, a barrier a turn; bf16 weights
// without remainders): 64 trees of 16 nodes over up to 16K tokens 286 -> 264 us, one of 64 behind
// 32K 85 -> 89 (two row tiles: a half waits longer for its next scores), one of 7 over 1K 17.8 ->
// 18.1; fp16, with remainders: 8 of 33 over windows of 4096 57 -> 55.
//
// With the remainders the same cases take 300, 106, 20.5 and 55 us; errors against 64 bits go from
// 0.0023, 0.0023 and 0.0041 of the output to 0.0016, 0.0016 and 0.0018, which is its rounding.
//
// What bounds it: the chains between the warps.  A turn of one row tile has 1536 tensor
// cycles (1792 with fp16 queries), 512 of exponentials and about 1650 of shared memory
// (the operands of the scores 512 and of the values 512, copies 256, V's conversion 384), a tile
// of tokens 1430 of HBM for its 32 KB on one of 152 SMs, and it takes 2700 (the tensor pipe is
// active in 58 % of the cycles; 41 % where two row tiles share a tile): V's conversion by
// four warps 1480 and its waits for codes and a free operand, the issue of products and the
// waits between them.
//
// The flat list of all token tiles (sequence, unit, head, tile) is cut into equal runs, one
// CTA each, whatever the lengths are; a unit counts kUnitCost more, for its start and end.
// A unit that lies in one run is written directly; otherwise each run leaves a partial
// (maximum, sum, output), which a second launch joins in their order, so results do not
// depend on timing.
//
// Warps: 0-7 softmax and output, 8-11 V's conversion, 12 TMA of the keys, 13 MMA, 14 the
// list of items, the scales and TMA of the values, 15 the next unit's queries.  Tensor memory,
// in parts of 128 columns: one row tile: three of scores (their weights overwrite them), one
// of output; two: two of scores, two of outputs.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>

#include "tq_fp8.cuh"
#include "tq_fp8_tc.cuh"

namespace tq {
namespace {

constexpr int kRowsPerTile = 128;
constexpr int kUnitRows = 256;
constexpr int kTok = 128;   // tokens of a tile
constexpr int kThreads = 512;
constexpr int kNanRing = 3;
constexpr int kUseRing = 8;
constexpr int kSoftRegs = 144, kOtherRegs = 112;  // of the two softmax warpgroups and the two others, out of 128 each
constexpr float kHeadroom = 24.f;

// What a run has of a unit.  Warp 14 goes through the list and leaves a record of every item, which all warps read.  A record
// is written again IR items on, when the softmax warps, the last to need it, are done with it: the copy of the values of a
// tile waits for the conversion of the tile VS before it, that one for the output of the tile two before it, and that for the
// softmax warps' weights, which they form when they are done with the item before; every item has a tile at least.
struct Item {
    int b, n, row0, start;   // the sequence, its nodes, packed row of the first, its position (negative: they see nothing)
    int end;                 // the tokens that there are: start + n, at most what the block table holds
    int first;               // the unit's first node
    int head;
    int tile0, tiles;        // the tokens' tiles of this run
    int flags;               // below
    int runs;                // of a unit that begins here and goes on: how many
    int unused;
};
constexpr int kOne = 1, kLast = 2, kWhole = 4, kBegins = 8;  // one row tile; the run's last; all of the unit; its first tile
constexpr int kAhead = 16;  // warp 15 prepares its queries

// A unit's start and end in turns of one row tile, for the length of the runs.
constexpr int kUnitCost = 8;

template <int NT>
struct TreeLayout {
    static constexpr int KS = 2;                        // stages of keys
    static constexpr int VS = NT == 2 ? 3 : 2;          // of codes of values: the wait for a copy and its conversion take longer than two turns
    static constexpr int IR = NT == 2 ? 8 : 6;          // records of the list: VS + 4 at least, see above
    static constexpr int MR = NT == 2 ? 8 : 6;          // tiles of scales: the same waits free them, VS + 3 at least
    static constexpr bool ahead = NT == 2;              // there is room for the next unit's queries
    static constexpr int q = 0;                         // [2 tiles][NT][128 rows][128 B], 128-byte swizzle
    static constexpr int k = q + 2 * NT * 16384;        // [KS][128 tokens][128 B], 128-byte swizzle
    static constexpr int v = k + KS * 16384;            // [VS][128 tokens][128 B] codes, 128-byte swizzle
    static constexpr int vb = v + VS * 16384;           // [2] bf16 operand: 8 x 8 core matrices, MN-major
    static constexpr int meta = vb + 2 * 32768;         // [ring]: key scales [8], value exponents [8] of 16 tokens each
    static constexpr int okm = meta + MR * 64;          // [ring]: groups of 16 tokens that are there
    static constexpr int items = okm + MR * 4;          // [ring] of Item
    static constexpr int bars = items + IR * (int)sizeof(Item);
    static constexpr int nbars = 2 + KS + 2 * VS + 2 + 12 + MR + 1 + IR + 2 + (ahead ? kUseRing : 0);
    static constexpr int misc = bars + nbars * 8;       // tensor memory's address; the first token with a NaN in any dim [ring]
    static constexpr int mult = (misc + 16 + 15) / 16 * 16;  // [2][128] rows' score multipliers
    static constexpr int swap = ahead ? mult + 1024 : mult;  // [2][128] what the two threads of a row exchange
    static constexpr int total = swap + 1024;
    static constexpr int smem = total + 1008;           // the base is rounded up to 1 KB, from 16 bytes at least
    static_assert(KS == 2 && MR >= VS + 3 && IR >= VS + 4 && IR <= kUseRing, "rings");
    static_assert(k % 1024 == 0 && v % 1024 == 0 && vb % 1024 == 0 && meta % 16 == 0 && bars % 8 == 0 && mult % 16 == 0, "alignment");
    static_assert(smem <= kSmemLimit, "tree attention does not fit in shared memory");
};
// V's operand: 8 tokens x 8 dims core matrices of 128 bytes, token groups 128 bytes apart, dim groups 2048; the dims of
// every four in the order 0, 2, 1, 3, as a word of codes is taken apart with the fewest instructions
constexpr uint32_t kVLbo = 128, kVSbo = 2048;

struct TreeArgs {
    Fp8AttnArgs a;
    int tpt;             // nodes of a row tile: 128 / group
    float* partials;     // [runs][2][256][128], unnormalised: of a unit that began before the run, and of one that goes on behind it
    float2* ml;          // [runs][2][256] (maximum, sum)
    int4* joins;         // [runs]: of the unit that begins in the run and goes on: runs (0: none), packed row, nodes, head
    int* nan;            // [runs][ring][128 dims]: the first position of the item whose value is a NaN there
    long long stall_cycles;
};

__device__ __forceinline__ int tiles_of(int end) { return max(1, (end + kTok - 1) / kTok); }  // (no tokens: one, all masked)

// A sequence's part of the list: `full` units of two row tiles, and one more of one where the rest fits it.  Of one head a
// unit takes as many places as it has turns, and kUnitCost.
struct Shape {
    int full, left, tiles, size_full, size_left;
    __device__ __forceinline__ Shape(int n, int end, int tpt) {
        full = n / (2 * tpt);
        left = n - full * 2 * tpt;
        if (left > tpt) {
            ++full;
            left = 0;
        }
        tiles = tiles_of(end);
        size_full = 2 * tiles + kUnitCost;
        size_left = left ? tiles + kUnitCost : 0;
    }
    __device__ __forceinline__ int size() const { return full * size_full + size_left; }
};
// Where a place of the list lies: the unit and head of its sequence, and the place in it.
struct Spot {
    int unit, head, at, size;
    bool one;
    __device__ __forceinline__ Spot(const Shape& sh, int rest, int hkv) {
        const int of_full = sh.full * sh.size_full * hkv;
        one = rest >= of_full;
        size = one ? sh.size_left : sh.size_full;
        if (one) rest -= of_full;
        unit = one ? sh.full : rest / (size * hkv);
        if (!one) rest -= unit * size * hkv;
        head = rest / size;
        at = rest - head * size;
    }
};
// The unit's tiles that lie before a place of it: places are its cost first, then one a tile (two: the first counts).
__device__ __forceinline__ int tiles_before(int at, bool one) {
    return at <= kUnitCost ? 0 : one ? at - kUnitCost : (at - kUnitCost + 1) / 2;
}
// Runs are no shorter, so that one inside a unit has a tile of it at least.
constexpr int kLeastRun = kUnitCost + 4;

// 32 bits of a row's mask: of nodes first .. first + 31 of its sequence's n (those before node 0 are the prefix, which every
// row sees).
__device__ __forceinline__ uint32_t seen_nodes(const uint64_t* mask, int words, int first, int n) {
    if (first <= -32) return 0xFFFFFFFFu;
    const int at = max(first, 0), w = at >> 6, sh = at & 63;
    uint64_t x = w < words ? __ldg(mask + w) >> sh : 0;
    if (sh > 32 && w + 1 < words) x |= __ldg(mask + w + 1) << (64 - sh);
    const int left = n - at;
    uint32_t bits = left <= 0 ? 0u : left >= 32 ? (uint32_t)x : (uint32_t)x & ((1u << left) - 1);
    if (first < 0) bits = (bits << -first) | ((1u << -first) - 1);
    return bits;
}

// Notes the codes of NaN among the 32 tokens of a tile that converter `cw` has: in `first` (global memory) the first position
// of each dim that holds one, in `any` of all dims.  p0: the tile's first position.  Rare, and out of line.
__device__ __noinline__ void note_nan(const uint8_t* codes, const int* exps, int* first, int* any, int cw, int p0, int end) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int i = lane; i < 32 * kHeadDim; i += 32) {
        const int t = cw * 32 + (i >> 7), d = i & 127;
        const uint8_t code = codes[t * 128 + (((d >> 4) ^ (t & 7)) << 4) + (d & 15)];
        if ((code & 127) == 127 && exps[t >> 4] != INT_MIN && p0 + t < end) {
            atomicMin(first + d, p0 + t);
            atomicMin(any, p0 + t);
        }
    }
    __threadfence_block();
}

// A bounded wait in few instructions (the waits are many, and what the warps execute together has to fit the SM's
// instruction cache): `tries` tries that sleep for about 4 us each where nothing arrives (7885 cycles measured), so a second.
constexpr int kTries = 1 << 18;
__device__ __forceinline__ bool wait_tries(uint32_t bar, uint32_t parity, int tries) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .s32 n;\n mov.s32 n, %3;\n"
        "WAIT: mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n"
        " @p bra DONE;\n sub.s32 n, n, 1;\n setp.gt.s32 q, n, 0;\n @q bra WAIT;\n"
        "DONE: selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(tries)
        : "memory");
    return ok != 0;
}

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

// A batch of query rows in e4m3 terms: K pairs of rows of a tile, half a warp a row, 8 elements a lane; the lane's first row
// is `row`.
template <typename T, int NT, int K>
__device__ __forceinline__ void store_terms(const uint4 (&raw)[K], uint8_t* place, float* mult, int row, int col, float scale) {
    uint32_t words[K][4];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        words[k][0] = raw[k].x;
        words[k][1] = raw[k].y;
        words[k][2] = raw[k].z;
        words[k][3] = raw[k].w;
    }
    Fp8Split<T, 16, K> split(words);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        uint32_t code[K][2];
        split.template term<0>(code);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int r = row + 2 * k;
            *reinterpret_cast<uint2*>(place + j * 16384 + r * 128 + (((col >> 1) ^ (r & 7)) << 4) + (col & 1) * 8) = make_uint2(code[k][0], code[k][1]);
        }
    }
    float factors = 0.f;  // a query that is not finite makes its own row NaN
#pragma unroll
    for (int k = 0; k < K; ++k) factors = col == k ? split.factor(k, scale) : factors;
    if (col < K) mult[row + 2 * col] = factors;
}

template <typename T, int NT>
__global__ void __launch_bounds__(kThreads, 1) fp8_tree_kernel(const TreeArgs A, const __grid_constant__ CUtensorMap map) {
    using L = TreeLayout<NT>;
    extern __shared__ uint8_t raw[];
    uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(sm);
    const Fp8Geometry& g = A.a.g;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto bar = [&](int i) { return sb + L::bars + 8 * i; };
    // queries stored by the softmax warps, by warp 15; keys landed; codes of values landed, free; operand of values stored;
    // scores, weights and output of a turn [4]; scales stored; outputs read; an item's record; all products done; one that
    // nothing arrives on; an item's queries are in use [8].  (The scores of the tile two before free a place of keys, its
    // output one of the operands: no turn four later can be done by then, so the rings of 4 tell them apart.)
    constexpr int bQ = 0, bQa = 1, bK = 2, bV = bK + L::KS, bVe = bV + L::VS, bB = bVe + L::VS,
                  bS = bB + 2, bP = bS + 4, bO = bP + 4, bM = bO + 4, bOe = bM + L::MR, bR = bOe + 1,
                  bEnd = bR + L::IR, bNever = bEnd + 1, bQu = bNever + 1;
    static_assert(bQu + (L::ahead ? kUseRing : 0) == L::nbars, "barriers");

    if (tid == 0) {
        mbar_init(bar(bQ), 8);
        mbar_init(bar(bQa), 1);
        for (int i = 0; i < (L::ahead ? kUseRing : 0); ++i) mbar_init(bar(bQu + i), 10);  // softmax, MMA, and warp 15 has the record
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(bB + i), 4);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(bS + i), 1);
            mbar_init(bar(bP + i), 4);
            mbar_init(bar(bO + i), 1);
        }
        for (int i = 0; i < L::VS; ++i) {
            mbar_init(bar(bV + i), 1);
            mbar_init(bar(bVe + i), 4);
        }
        for (int i = 0; i < L::KS; ++i) {
            mbar_init(bar(bK + i), 1);
        }
        for (int i = 0; i < L::MR; ++i) {
            mbar_init(bar(bM + i), 1);
        }
        for (int i = 0; i < L::IR; ++i) mbar_init(bar(bR + i), 1);
        mbar_init(bar(bOe), 8);
        mbar_init(bar(bEnd), 1);
        mbar_init(bar(bNever), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    int* any_nan = reinterpret_cast<int*>(sm + L::misc + 4);
    if (tid < kNanRing) any_nan[tid] = INT_MAX;
    if (warp == 12 && lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(&map) : "memory");
    if (warp == 13) tc::tmem_alloc<512>(sb + L::misc);
    grid_dependency_wait();
    int* const nan_g = A.nan + (int64_t)blockIdx.x * kNanRing * kHeadDim;
    if (tid < kNanRing * kHeadDim) nan_g[tid] = INT_MAX;

    // ---- this CTA's run of the list: the places of all sequences are added up by all threads ----
    const int B = A.a.b.batch, G = A.a.group;
    const int cap = (int)min((int64_t)A.a.b.max_blocks * g.bs, (int64_t)0x7FFFFF00);
    auto nodes_of = [&](int b, int& row0, int& start, int& end) {
        row0 = fp8_clamp_cu(A.a.b.cu, b, A.a.b.num_tokens);
        const int n = max(0, fp8_clamp_cu(A.a.b.cu, b + 1, A.a.b.num_tokens) - row0);
        start = __ldg(A.a.b.start + b);
        end = start < 0 ? 0 : (int)min((int64_t)start + n, (int64_t)cap);
        return n;
    };
    auto places_of = [&](int b) {
        int row0, start, end;
        const int n = b < B ? nodes_of(b, row0, start, end) : 0;
        return n ? Shape(n, end, A.tpt).size() * g.hkv : 0;
    };
    int* scan = reinterpret_cast<int*>(sm + L::mult);  // [16 warps]; the run's first sequence, the places before it, a sum
    // (The host's limit keeps the places below 2^31 - 1, but cu_tokens that fall and rise again count tokens more than once.)
    auto add = [](int x, int y) { return (int)min((uint32_t)x + (uint32_t)y, (uint32_t)INT_MAX); };
    // inclusive sum over the CTA, and the total
    auto sum_up = [&](int x, int& total) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x = add(x, y);
        }
        __syncthreads();
        if (lane == 31) scan[warp] = x;
        __syncthreads();
        int before = 0;
        total = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            before = add(before, w < warp ? scan[w] : 0);
            total = add(total, scan[w]);
        }
        return add(x, before);
    };
    int total = 0, mine = 0, upto = 0, first_part = 0;  // (the first 512 sequences' are kept)
    for (int b0 = 0; b0 < B; b0 += kThreads) {
        const int x = places_of(b0 + tid);
        int part;
        const int inc = sum_up(x, part);
        if (b0 == 0) {
            mine = x;
            upto = inc;
            first_part = part;
        }
        total = add(total, part);
    }
    if (total == INT_MAX) {
        if (blockIdx.x == 0 && tid == 0) flag(A.a.status, TQ_FLAG_BAD_SLOT);
        total = 0;
    }
    const int runs = min((int)gridDim.x, max(1, total / kLeastRun)), cta = (int)blockIdx.x;
    const int each = total / runs, more = total - each * runs;  // the first `more` runs have a place more
    const int t0 = cta * each + min(cta, more), t1 = t0 + each + (cta < more ? 1 : 0);
    auto run_of = [&](int t) { return t < more * (each + 1) ? t / (each + 1) : more + (t - more * (each + 1)) / each; };
    bool work = cta < runs && total > 0;
    int b_first = 0, rest = 0;  // the sequence that the run begins in, and where
    if (work) {
        int base = 0;
        for (int b0 = 0; b0 < B; b0 += kThreads) {
            int x = mine, inc = upto, part = first_part;
            if (b0 > 0) {
                x = places_of(b0 + tid);
                inc = sum_up(x, part);
            }
            if (x > 0 && base + inc > t0 && base + inc - x <= t0) {
                scan[16] = b0 + tid;
                scan[17] = t0 - (base + inc - x);
            }
            base += part;
            if (base > t0) break;  // (the same in all threads)
        }
        __syncthreads();
        b_first = scan[16];
        rest = scan[17];
        // a run may lie in what units cost, and have no tiles
        int row0, start, end;
        const int n = nodes_of(b_first, row0, start, end);
        const Spot sp(Shape(n, end, A.tpt), rest, g.hkv);
        const int len = t1 - t0, at1 = min(sp.size, sp.at + len);
        work = tiles_before(at1, sp.one) > tiles_before(sp.at, sp.one) || sp.at + len - sp.size > kUnitCost;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + L::misc);

    bool bad = false;  // a bounded wait of this thread gave up: it waits no more
    auto wait = [&](int i, uint32_t parity) {
        if (!bad && !wait_tries(bar(i), parity, kTries)) bad = true;
    };
    const Item* ring = reinterpret_cast<const Item*>(sm + L::items);
    // The record of the CTA's i-th item, or null where a wait gave up.
    auto record = [&](int i) -> const Item* {
        wait(bR + i % L::IR, (i / L::IR) & 1);
        return __any_sync(0xFFFFFFFFu, bad) ? nullptr : ring + i % L::IR;
    };
    // id of the block that holds tokens 16 j .. of a tile, or -1 (past the end) or -2 (not in the pool)
    auto block_of = [&](int b, int end, int tile, int j) {
        const int p = tile * kTok + 16 * j;
        if (p >= end) return -1;
        const int id = __ldg(A.a.b.block_table + (int64_t)b * A.a.b.max_blocks + (p >> g.bs_shift));
        return id >= 0 && id < g.num_blocks ? id : -2;
    };
    // Where an item's queries and outputs are: of one row tile the places take turns, so that the next item's can be stored.
    auto place_of = [&](const Item* it, int i) { return L::ahead && (it->flags & kOne) ? i & 1 : 0; };

    if (!work) {
        if (tid == 0) A.joins[cta] = make_int4(0, 0, 0, 0);
    } else if (warp < 8) {
        // ================= queries, softmax, a thread a row in every other turn, and output, two threads a row =================
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        const int half = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t my = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        float* const mult_s = reinterpret_cast<float*>(sm + L::mult);
        float* const swap_s = reinterpret_cast<float*>(sm + L::swap);
        // what the thread of the row in the other half has for x
        auto exchange = [&](float x) {
            swap_s[half * 128 + r] = x;
            soft_barrier();
            return swap_s[(half ^ 1) * 128 + r];
        };
        bool empty = false;  // test hook: this CTA's partials are empty
        if (A.stall_cycles > 0 && (blockIdx.x & 1)) {
            empty = !mbar_wait_for(bar(bNever), 0, A.stall_cycles);
            if (empty && tid == 0) flag(A.a.status, TQ_FLAG_TIMEOUT);
        }
        if (tid == 0) A.joins[cta] = make_int4(0, 0, 0, 0);
        int tile = 0, turn = 0, asked = 0, ahead = 0;  // of the CTA so far: tiles, turns, items with queries stored here and by warp 15
        for (int i = 0;; ++i) {
            // These eight warps meet at barriers, so all of them have to go through the same items, also after a wait that
            // gave up.  Warp 14 leaves no record behind a wait of its own that did, and has left each of its records long
            // before these warps come to it: with four times its limit either all of them find one or none does.
            if (!wait_tries(bar(bR + i % L::IR), (i / L::IR) & 1, 4 * kTries)) {
                bad = true;
                break;
            }
            __syncwarp();
            const Item* it = ring + i % L::IR;
            const bool one = it->flags & kOne;
            const int place = place_of(it, i);
            if (it->flags & kAhead) {
                wait(bQa, ahead++ & 1);
            } else {
                // The queries in e4m3 terms, two rows at a time (half a warp each), 16 rows of either tile a warp
                const int sub = lane >> 4, col = lane & 15, first_row = warp * 16 + sub;
                const int left = it->n - it->first;  // nodes from the unit's first on
                const T* q0 = static_cast<const T*>(A.a.q) + (int64_t)(it->row0 + it->first) * A.a.q_token + (int64_t)it->head * G * A.a.q_head + 8 * col;
                int node = first_row / G, gr = first_row % G;
                uint4 raw_q[16];  // the first tile's rows, and the second's
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const T* q = q0 + (int64_t)node * A.a.q_token + (int64_t)gr * A.a.q_head;
                    const bool in = first_row + 2 * k < A.tpt * G;
                    raw_q[k] = in && node < left ? __ldg(reinterpret_cast<const uint4*>(q)) : make_uint4(0, 0, 0, 0);
                    raw_q[8 + k] = in && !one && node + A.tpt < left ? __ldg(reinterpret_cast<const uint4*>(q + (int64_t)A.tpt * A.a.q_token)) : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        if (++gr == G) {
                            gr = 0;
                            ++node;
                        }
                }
#pragma unroll 1
                for (int k = 0; k < (one ? 2 : 4); ++k) {
                    uint4 four[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) four[y] = raw_q[y];
#pragma unroll
                    for (int y = 0; y < 12; ++y) raw_q[y] = raw_q[y + 4];
                    const int x = k >> 1;
                    // (rows without a node are not stored: whatever lies there reaches no other row)
                    if (warp * 16 + 8 * (k & 1) >= min(A.tpt, left - x * A.tpt) * G) continue;
                    store_terms<T, NT, 4>(four, sm + L::q + (place + x) * NT * 16384, mult_s + (place + x) * 128, first_row + 8 * (k & 1), col, A.a.sm_scale_log2);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(bQ));
                wait(bQ, asked++ & 1);
            }
            __syncwarp();
            if (L::ahead && lane == 0) mbar_arrive(bar(bQu + i % kUseRing));
            // Each half of these warps takes every other turn, a thread a row: with two row tiles its own, with one of the same
            // rows, whose output they share.
            const int mine = one ? 0 : half;
            const float factor = mult_s[(place + mine) * 128 + r];
            // A query that is not finite has a factor of NaN. Its row goes along with another one, so that masked scores stay
            // -inf, and its sum becomes NaN at the item's end if it has seen anything.
            const bool odd = factor != factor;
            const float mult = odd ? 1.f : factor;
            int node = it->first + mine * A.tpt + r / G;  // -1: there is none
            if (r >= A.tpt * G || node >= it->n) node = -1;
            // Warps without a node among their rows only meet the others: what lies in their rows reaches no other row.
            const bool live = __any_sync(0xFFFFFFFFu, node >= 0);
            // Weights are 2^(l - m) against a reference m, a whole number, that is put 2^24 above the row's maximum and raised again
            // only when 32 weights add up to more than 32 (some weight is above 1 then): bf16 and fp32 keep their precision at
            // any size, the sum is needed anyway, and no maximum is formed otherwise.  What was weighed before follows by a power of
            // two, exactly.  A row that has seen no token yet has no reference.
            float m = -INFINITY, sum = 0.f;
            soft_barrier();  // the factors are read: their place may be written again
            const int tiles = it->tiles, turns = one ? tiles : 2 * tiles;
            // multiplies 8 columns of pairs of weights by a power of two
            auto scale_weights = [&](uint32_t at, float by) {
                uint32_t p = pack_bf16(by, by), y[8];
                __syncwarp();
                tmem_ld<8>(at, y);
                tmem_ready<8>(y);
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] = mul_bf16x2(y[k], p);
                tmem_st8(at, y);
            };
            for (int u = half; u < turns; u += 2) {
                const int now = turn + u, tu = one ? u : u >> 1, mi = (tile + tu) % L::MR;
                const uint32_t tS = my + (one ? u % 3 : u & 1) * 128, tO = my + (one ? 384 : 256 + 128 * half);
                wait(bM + mi, ((tile + tu) / L::MR) & 1);
                const int ok = *reinterpret_cast<const int*>(sm + L::okm + mi * 4);
                const float* ks = reinterpret_cast<const float*>(sm + L::meta + mi * 64);
                // the node that the tile's first token is: the masks begin behind the prefix
                const int node0 = (it->tile0 + tu) * kTok - it->start;
                wait(bS + (now & 3), (now >> 2) & 1);
                tc::fence_after_sync();
                __syncwarp();
                if (live) {
                    // Everything goes through tensor memory in loops that are not unrolled, the weights into the place of their
                    // scores: with a turn's tokens in straight line, warps waited for instructions more than for anything else.
                    if (ok != 0xFF || node0 + kTok > 0) {
                        uint32_t bits = 0;
#pragma unroll 1
                        for (int c = 0; c < 8; ++c) {  // 16 tokens, of a block
                            if (c & 1) bits >>= 16;
                            else bits = node >= 0 && it->start >= 0
                                            ? seen_nodes(A.a.mask + (int64_t)(it->row0 + node) * A.a.words, A.a.words, node0 + 16 * c, it->n) : 0u;
                            const uint32_t see = (ok >> c) & 1 ? bits : 0u;
                            uint32_t y[16];
                            __syncwarp();
                            tmem_ld<16>(tS + 16 * c, y);
                            tmem_ready<16>(y);
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                if (!((see >> k) & 1)) y[k] = 0xFF800000u;
                            tmem_st8(tS + 16 * c, *reinterpret_cast<uint32_t(*)[8]>(y));
                            tmem_st8(tS + 16 * c + 8, *reinterpret_cast<uint32_t(*)[8]>(y + 8));
                        }
                        tc::wait_st();
                    }
#pragma unroll 1
                    for (int c = 0, tried = 0; c < 4;) {  // 32 tokens; once more with a new reference
                        uint32_t y[32], lo[16];
                        __syncwarp();
                        tc::ld_32x32b_x32(tS + 32 * c, y);
                        // (a masked score of -inf stays one with a positive factor; NaN stays NaN)
                        float f[2] = {ks[2 * c] * mult, ks[2 * c + 1] * mult};
                        f[0] = f[0] < 1e-37f ? 1e-37f : f[0];
                        f[1] = f[1] < 1e-37f ? 1e-37f : f[1];
                        const float ref = m == -INFINITY ? 0.f : m;
                        const uint64_t neg = f2_pack(-ref, -ref), f0 = f2_pack(f[0], f[0]), f1 = f2_pack(f[1], f[1]);
                        uint64_t part = f2_pack(0.f, 0.f), part2 = part;
                        tc::wait_ld();
                        tc::reg_fence(y);
                        uint32_t w[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            float a, b;
                            f2_unpack(f2_fma(f2_pack(__uint_as_float(y[2 * k]), __uint_as_float(y[2 * k + 1])), k < 8 ? f0 : f1, neg), a, b);
                            a = ex2(a);
                            b = ex2(b);
                            if (k & 1) part = f2_add(part, f2_pack(a, b));
                            else part2 = f2_add(part2, f2_pack(a, b));
                            w[k] = pack_bf16(a, b);
                            lo[k] = pack_bf16(a - __uint_as_float(w[k] << 16), b - __uint_as_float(w[k] & 0xFFFF0000u));
                        }
                        float a, b;
                        f2_unpack(f2_add(part, part2), a, b);
                        a += b;
                        if (!tried && __any_sync(0xFFFFFFFFu, node >= 0 && (a > 32.f || m == -INFINITY))) {
                            tried = 1;
                            // a new reference; the scores are still there
                            float mx = -INFINITY;
#pragma unroll
                            for (int k = 0; k < 32; ++k) {
                                uint32_t z = y[k];
                                if (__uint_as_float(z) != -INFINITY) mx = fmaxf(mx, __uint_as_float(z) * f[k >> 4]);
                            }
                            float by = 1.f;
                            if (mx > m) {
                                const float to = ceilf(mx) + kHeadroom;
                                by = ex2(m - to);
                                m = to;
                            }
                            sum *= by;
                            tc::wait_st();  // the weights of the chunks before, which are read again
#pragma unroll 1
                            for (int k = 0; k < c; ++k)
                                for (int z = 0; z < 4; ++z) scale_weights(tS + 32 * k + 8 * z, by);
                            tc::wait_st();
                            continue;
                        }
                        sum += a;
                        tc::st_32x32b_x16(tS + 32 * c, w);
                        tc::st_32x32b_x16(tS + 32 * c + 16, lo);
                        ++c;
                        tried = 0;
                    }
                    tc::wait_st();
                }
                // The output's reference is the one of the turn before it: with one row tile the other half's.
                const bool follows = one ? u > 0 : u > 1;
                if (one && follows) wait(bP + ((now - 1) & 3), ((now - 1) >> 2) & 1);
                __syncwarp();
                if (live && follows) {
                    const float before = swap_s[mine * 128 + r];
                    if (__any_sync(0xFFFFFFFFu, before != m)) {
                        const float to = fmaxf(before, m);
                        const float by_w = to == m ? 1.f : ex2(m - to), by_o = to == before ? 1.f : ex2(before - to);
                        m = to;
                        sum *= by_w;
                        if (__any_sync(0xFFFFFFFFu, by_w != 1.f)) {
#pragma unroll 1
                            for (int k = 0; k < 4; ++k)
                                for (int z = 0; z < 4; ++z) scale_weights(tS + 32 * k + 8 * z, by_w);
                        }
                        if (__any_sync(0xFFFFFFFFu, by_o != 1.f)) {
                            const int last = now - (one ? 1 : 2);
                            wait(bO + (last & 3), (last >> 2) & 1);
                            tc::fence_after_sync();
                            __syncwarp();
#pragma unroll 1
                            for (int c = 0; c < 16; ++c) {
                                uint32_t o[8];
                                tmem_ld<8>(tO + 8 * c, o);
                                tmem_ready<8>(o);
#pragma unroll
                                for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * by_o);
                                tmem_st8(tO + 8 * c, o);
                            }
                        }
                        tc::wait_st();
                    }
                }
                swap_s[mine * 128 + r] = m;
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(bP + (now & 3)));
            }
            turn += turns;
            // ---- the item's end ----
            tile += tiles;
            for (int k = 1; k <= (one ? 1 : 2); ++k) {
                wait(bO + ((turn - k) & 3), ((turn - k) >> 2) & 1);
                __syncwarp();
            }
            tc::fence_after_sync();
            if (odd && sum != 0.f) sum = NAN;
            // With one row tile both halves have sums of the same rows, and the output has the last turn's reference.
            soft_barrier();
            const float last_m = one ? swap_s[r] : m;
            soft_barrier();
            if (one) sum = sum == 0.f ? 0.f : sum * ex2(m - last_m);
            m = last_m;
            if (bad && !empty) {
                flag(A.a.status, TQ_FLAG_TIMEOUT);
                empty = true;
            }
            const bool whole = it->flags & kWhole;
            const int64_t slot = (int64_t)cta * 2 + (it->flags & kBegins ? 1 : 0);
            const int nan_slot = i % kNanRing;
            const bool nan_here = any_nan[nan_slot] != INT_MAX;
#pragma unroll 1
            for (int x = 0; x < (one ? 1 : 2); ++x) {
                const uint32_t tO = my + (one ? 384 : 256 + 128 * x) + 64 * half;
                // sums and references: of either half's turns, or of the half that has the tile
                const float other = exchange(sum);
                soft_barrier();
                const float other_m = exchange(m);
                const float all = one ? sum + other : half == x ? sum : other, ref = one || half == x ? m : other_m;
                const int node_x = it->first + x * A.tpt + r / G, row_node = r < A.tpt * G && node_x < it->n ? node_x : -1;
                const bool live_x = __any_sync(0xFFFFFFFFu, row_node >= 0);
                const bool none = all == 0.f;
                const float inv = whole && !none ? 1.f / all : 1.f;
                if (!whole && half == 0)
                    A.ml[slot * kUnitRows + x * 128 + r] = make_float2(none || empty ? -INFINITY : ref, none || empty ? 0.f : all);
                // A dim is NaN in the rows that see a token with a NaN there: all, where the first such position is in the prefix.
                auto sees_nan = [&](int d) -> bool {
                    const int at = __ldcg(nan_g + nan_slot * kHeadDim + d);
                    if (row_node < 0 || at == INT_MAX) return false;
                    if (at < it->start) return true;
                    const int last = min(it->end, (it->tile0 + tiles) * kTok);
                    for (int p = at; p < last; ++p) {
                        if (!(seen_nodes(A.a.mask + (int64_t)(it->row0 + row_node) * A.a.words, A.a.words, p - it->start, it->n) & 1)) continue;
                        const int id = __ldg(A.a.b.block_table + (int64_t)it->b * A.a.b.max_blocks + (p >> g.bs_shift));
                        if (id < 0 || id >= g.num_blocks) continue;
                        const int64_t row = ((((int64_t)id * g.hkv + it->head) * 2 + 1) << g.bs_shift) + (p & (g.bs - 1));
                        if ((__ldg(g.pool + row * kHeadDim + d) & 127) == 127) return true;
                    }
                    return false;
                };
                // Rows leave through shared memory (the place of the queries, whose last reader is done), 256 bytes of every row
                // at a time, so that a store takes two rows and not 32 pieces: whole ones of 16-bit elements at once, fp32 ones of
                // a partial first one thread's 64 dims and then the other's.
                const uint32_t at = sb + L::q + (place + x) * NT * 16384;
                auto piece = [&](int k) { return at + r * 256 + ((k ^ (lane & 7)) << 4); };
#pragma unroll 1
                for (int pass = 0; pass < (whole ? 1 : 2); ++pass) {
                    if (live_x && (whole || pass == half)) {
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t o[16];
                            __syncwarp();
                            tmem_ld<16>(tO + 16 * c, o);
                            tmem_ready<16>(o);
                            float y[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k)  // the columns are dims 0, 2, 1, 3 of every four
                                y[k] = none ? 0.f : __uint_as_float(o[(k & ~3) | ((k & 1) << 1) | ((k >> 1) & 1)]) * inv;
                            if (nan_here)
                                for (int k = 0; k < 16; ++k)
                                    if (sees_nan(64 * half + 16 * c + k))
#pragma unroll
                                        for (int z = 0; z < 16; ++z) y[z] = z == k ? NAN : y[z];
                            if (whole) {
                                uint32_t w[8];
#pragma unroll
                                for (int k = 0; k < 8; ++k) w[k] = pack_two<T>(y[2 * k], y[2 * k + 1]);
                                pre_sts128(piece(8 * half + 2 * c), w[0], w[1], w[2], w[3]);
                                pre_sts128(piece(8 * half + 2 * c + 1), w[4], w[5], w[6], w[7]);
                            } else {
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    pre_sts128(piece(4 * c + k), __float_as_uint(y[4 * k]), __float_as_uint(y[4 * k + 1]), __float_as_uint(y[4 * k + 2]),
                                               __float_as_uint(y[4 * k + 3]));
                            }
                        }
                    }
                    if (x == (one ? 0 : 1) && pass == (whole ? 0 : 1)) {  // the last reading of outputs
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(bOe));
                    }
                    soft_barrier();
                    // 16 rows a warp, of those that have a node
                    int row = warp * 16 + (lane >> 4), gr = row % G;
                    const int rows = min(A.tpt, it->n - it->first - x * A.tpt) * G;
                    char* to = whole ? reinterpret_cast<char*>(static_cast<T*>(A.a.out) + ((int64_t)(it->row0 + it->first + x * A.tpt + row / G) * A.a.hq +
                                                                                           (int64_t)it->head * G + gr) * kHeadDim)
                                     : reinterpret_cast<char*>(A.partials + (slot * kUnitRows + x * 128 + row) * kHeadDim + 64 * pass);
                    const int64_t step = kHeadDim * (whole ? (int)sizeof(T) : 4), wrap = whole ? (int64_t)(A.a.hq - G) * step : 0;
                    to += 16 * (lane & 15);
#pragma unroll 2
                    for (int k = 0; k < 8; ++k, row += 2) {
                        if (row >= rows || (whole && empty)) break;
                        *reinterpret_cast<uint4*>(to) = lds128(at + row * 256 + (((lane & 15) ^ (row & 7)) << 4));
                        for (int z = 0; z < 2; ++z) {
                            to += step;
                            if (++gr == G) {
                                gr = 0;
                                to += wrap;
                            }
                        }
                    }
                    if (!whole && pass == 0) soft_barrier();  // the place is free for the other half
                }
            }
            if (!whole && tid == 0 && (it->flags & kBegins)) A.joins[cta] = make_int4(it->runs, it->row0 + it->first, it->n - it->first, it->head);
            const bool last = it->flags & kLast;
            // the places are free for the next queries; the notes are written again three items on
            if (soft_barrier_or(nan_here)) {
                if (half == 0) nan_g[nan_slot * kHeadDim + r] = INT_MAX;
                __threadfence_block();
                if (tid == 0) any_nan[nan_slot] = INT_MAX;
            }
            if (last) break;
        }
    } else if (warp < 12) {
        // ================= V: codes to bf16, times the block's scale =================
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        const int cw = warp - 8;
        int t = 0, turn = 0, last1 = 0, last2 = 0;  // last turns of the two tiles before
        for (int i = 0;; ++i) {
            const Item* it = record(i);
            if (!it) break;
            const int per_tile = it->flags & kOne ? 1 : 2;
            const int p_item = it->tile0 * kTok, end = it->end, last = it->flags & kLast, t_item = t, t_end = t + it->tiles;
            for (; t < t_end; ++t) {
                const int b = t & 1, vi = t % L::VS, mi = t % L::MR;
                wait(bV + vi, (t / L::VS) & 1);  // (warp 14 has written the scales before it arrives there)
                if (t > 1) wait(bO + (last2 & 3), (last2 >> 2) & 1);
                last2 = last1;
                last1 = (turn += per_tile) - 1;
                const int* vs = reinterpret_cast<const int*>(sm + L::meta + mi * 64 + 32);
                // A warp converts 32 tokens, of two groups of 16 with a scale each: 8 of them by 4 pieces of 16 codes at a
                // time.  What a lane reads and writes differs by constants from one time to the next.  (Unrolled by 8 it is slower, as all
                // that makes the loops longer than the SM's instruction cache.)
                const uint32_t src = sb + L::v + vi * 16384 + (cw * 32 + (lane & 7)) * 128, piece0 = ((lane >> 3) ^ (lane & 7)) << 4;
                const uint32_t dst = sb + L::vb + b * 32768 + (lane >> 3) * 2 * kVSbo + cw * 4 * kVLbo + (lane & 7) * 16;
                uint32_t most = 0;  // largest magnitudes, in either half: a NaN's is 0x7F0
                auto piece = [&](int k8) { return lds128(src + (k8 >> 1) * 1024 + (piece0 ^ ((k8 & 1) << 6))); };
                uint4 next = piece(0);  // read one ahead
                const int2 e2 = *reinterpret_cast<const int2*>(vs + 2 * cw);  // exponents of the value scales, or INT_MIN where there is no block
                // e4m3's fields moved into bf16's read as the value times 2^-120 (subnormals too)
                auto scale_of = [](int e) {
                    const uint32_t f = e == INT_MIN ? 0u : (uint32_t)(min(e + 120, 127) + 127) << 7;
                    return f | (f << 16);
                };
                uint32_t m1 = scale_of(e2.x);
                const uint32_t m1b = scale_of(e2.y);
                const bool large = max(e2.x, e2.y) > 7;  // 2^(e + 120) is past bf16's range: the rest in a second product
#pragma unroll 2
                for (int k8 = 0; k8 < 8; ++k8) {
                    const uint32_t w[4] = {next.x, next.y, next.z, next.w};
                    next = piece((k8 + 1) & 7);
                    uint32_t o[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // dims 0 and 2, 1 and 3 of the word's four: the operand's columns hold them in that order
                        const uint32_t even = (w[k] << 4) & 0x07F007F0u, odd = (w[k] >> 4) & 0x07F007F0u;
                        o[2 * k] = mul_bf16x2(((w[k] << 8) & 0x80008000u) | even, m1);
                        o[2 * k + 1] = mul_bf16x2((w[k] & 0x80008000u) | odd, m1);
                        most = __vimax3_u16x2(most, even, odd);
                    }
                    if (large) {
                        const int e = k8 < 4 ? e2.x : e2.y;
                        const uint32_t f2 = (uint32_t)((e > 7 ? e - 7 : 0) + 127) << 7, m2 = f2 | (f2 << 16);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            // codes of 256 and more times 2^120 are past bf16: its largest value instead, as an infinity would
                            // reach the rows that do not see the token (0 * inf is NaN)
                            o[k] = mul_bf16x2(o[k], m2);
                            o[k] = (o[k] & 0x80008000u) | __vminu2(o[k] & 0x7FFF7FFFu, 0x7F7F7F7Fu);
                        }
                    }
                    const uint32_t at = dst + (k8 & 1) * 8 * kVSbo + (k8 >> 1) * kVLbo;
                    pre_sts128(at, o[0], o[1], o[2], o[3]);
                    pre_sts128(at + kVSbo, o[4], o[5], o[6], o[7]);
                    if (k8 == 3) m1 = m1b;
                }
                // A NaN (0x7F or 0xFF: a pool may come from elsewhere) is 480 in the operand, which does no harm to the rows
                // that do not see it; the item's end makes it NaN for those that do.
                if (__any_sync(0xFFFFFFFFu, (most & 0xFFFFu) == 0x7F0u || (most >> 16) == 0x7F0u))
                    note_nan(sm + L::v + vi * 16384, vs, nan_g + (i % kNanRing) * kHeadDim, any_nan + i % kNanRing, cw, p_item + (t - t_item) * kTok, end);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(bB + b));
                    mbar_arrive(bar(bVe + vi));
                }
            }
            if (last || __any_sync(0xFFFFFFFFu, bad)) break;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 12) {
            // ================= TMA of the keys, a lane a block =================
            const int pages = kTok >> g.bs_shift;
            const uint32_t bytes = (uint32_t)g.bs * kHeadDim;
            asm volatile("fence.proxy.async.global;" ::: "memory");  // the codes were written by ordinary stores
            const int per = g.bs >> 4;  // groups of 16 tokens in a block
            int t = 0, sent = 0;  // tiles whose copies are issued: none behind one whose wait gave up
            int turn = 0, last1 = 0, last2 = 0;  // last turns of the two tiles before
            for (int i = 0; !__any_sync(0xFFFFFFFFu, bad); ++i) {
                const Item* it = record(i);
                if (!it) break;
                const int b = it->b, end = it->end, h = it->head, tile0 = it->tile0, tiles = it->tiles, last = it->flags & kLast, per_tile = it->flags & kOne ? 1 : 2;
                if (lane == 0 && (it->start < 0 || end < (int64_t)it->start + it->n)) flag(A.a.status, TQ_FLAG_BAD_SLOT);
                int id = lane < pages ? block_of(b, end, tile0, lane * per) : -1;
                for (int u = 0; u < tiles; ++u, ++t) {
                    const int now = id, ks = t % L::KS;
                    id = lane < pages && u + 1 < tiles ? block_of(b, end, tile0 + u + 1, lane * per) : -1;
                    const unsigned there = __ballot_sync(0xFFFFFFFFu, now >= 0);
                    if (t >= L::KS) wait(bS + (last2 & 3), (last2 >> 2) & 1);
                    last2 = last1;
                    last1 = (turn += per_tile) - 1;
                    if (__any_sync(0xFFFFFFFFu, bad)) break;
                    sent = t + 1;
                    if (lane == 0) mbar_arrive_tx(bar(bK + ks), (uint32_t)__popc(there) * bytes);
                    __syncwarp();
                    if (now >= 0) tma_page(sb + L::k + ks * 16384 + lane * bytes, &map, (int)((((int64_t)now * g.hkv + h) * 2) << g.bs_shift), bar(bK + ks));
                    if (now == -2) flag(A.a.status, TQ_FLAG_BAD_SLOT);
                }
                if (last) break;
            }
            // copies may be in flight where a wait gave up: they end (again with a limit) before the memory is given back
            for (int u = max(0, sent - L::KS); u < sent; ++u) wait_tries(bar(bK + u % L::KS), (u / L::KS) & 1, kTries);
        } else if (warp == 14) {
            // ================= the list of items, the scales of every 16 tokens, and TMA of the values =================
            // (Keys and values have a warp each: the scores run ahead of the values, and their keys' copies must not wait for
            // a place of values.)
            const uint32_t bytes = (uint32_t)g.bs * kHeadDim;
            const int per = g.bs >> 4;  // groups of 16 tokens in a block
            asm volatile("fence.proxy.async.global;" ::: "memory");
            int sent = 0;
            int b = b_first, row0, start, end, n = nodes_of(b, row0, start, end);
            Shape sh(n, end, A.tpt);
            Spot sp(sh, rest, g.hkv);
            int to_go = t1 - t0, t = 0;  // places of the run from the spot on
            bool was_one = false;
            for (int i = 0; to_go > 0 && !__any_sync(0xFFFFFFFFu, bad);) {
                const int at1 = min(sp.size, sp.at + to_go), tile0 = tiles_before(sp.at, sp.one), tiles = tiles_before(at1, sp.one) - tile0;
                to_go -= at1 - sp.at;
                if (tiles > 0) {
                    // (warp 15 has read what is written over)
                    if (L::ahead && i >= L::IR) wait(bQu + (i - L::IR) % kUseRing, ((i - L::IR) / kUseRing) & 1);
                    if (__any_sync(0xFFFFFFFFu, bad)) break;
                    if (lane == 0) {
                        Item* it = reinterpret_cast<Item*>(sm + L::items) + i % L::IR;
                        it->b = b;
                        it->n = n;
                        it->row0 = row0;
                        it->start = start;
                        it->end = end;
                        it->first = sp.unit * 2 * A.tpt;
                        it->head = sp.head;
                        it->tile0 = tile0;
                        it->tiles = tiles;
                        it->flags = (sp.one ? kOne : 0) | (to_go <= kUnitCost ? kLast : 0) | (tile0 == 0 && tiles == sh.tiles ? kWhole : 0) |
                                    (tile0 == 0 ? kBegins : 0) | (L::ahead && sp.one && was_one ? kAhead : 0);
                        it->runs = run_of(t1 - to_go - at1 + sp.size - (sp.one ? 1 : 2)) - cta + 1;  // (up to the one with its last tile)
                        mbar_arrive(bar(bR + i % L::IR));
                    }
                    __syncwarp();
                    was_one = sp.one;
                    ++i;
                    auto scales_of = [&](int id) {
                        return id >= 0 ? __ldg(reinterpret_cast<const float2*>(g.scales + ((int64_t)id * g.hkv + sp.head) * 2)) : make_float2(0.f, 0.f);
                    };
                    // block ids are read two tiles ahead, scales one
                    int id = lane < 8 ? block_of(b, end, tile0, lane) : -1, id1 = lane < 8 && tiles > 1 ? block_of(b, end, tile0 + 1, lane) : -1;
                    float2 sc = scales_of(id);
                    for (int u = 0; u < tiles; ++u, ++t) {
                        const int mi = t % L::MR, vs = t % L::VS;
                        const int id2 = lane < 8 && u + 2 < tiles ? block_of(b, end, tile0 + u + 2, lane) : -1;
                        const float2 sc1 = scales_of(id1);
                        const unsigned ok = __ballot_sync(0xFFFFFFFFu, id >= 0);
                        if (__any_sync(0xFFFFFFFFu, bad)) break;
                        if (lane < 8) {
                            // where there is no block any positive scale does: the scores are masked
                            reinterpret_cast<float*>(sm + L::meta + mi * 64)[lane] = id >= 0 ? sc.x : 1.f;
                            reinterpret_cast<int*>(sm + L::meta + mi * 64 + 32)[lane] = id >= 0 ? fp8_exp_of(sc.y) : INT_MIN;
                        }
                        if (lane == 0) *reinterpret_cast<int*>(sm + L::okm + mi * 4) = (int)ok;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(bM + mi));
                        if (t >= L::VS) wait(bVe + vs, (t / L::VS - 1) & 1);
                        if (__any_sync(0xFFFFFFFFu, bad)) break;
                        sent = t + 1;
                        const bool mine_pg = id >= 0 && lane % per == 0;
                        const unsigned there = __ballot_sync(0xFFFFFFFFu, mine_pg);
                        if (lane == 0) mbar_arrive_tx(bar(bV + vs), (uint32_t)__popc(there) * bytes);
                        __syncwarp();
                        if (mine_pg)
                            tma_page(sb + L::v + vs * 16384 + lane * 16 * kHeadDim, &map, (int)((((int64_t)id * g.hkv + sp.head) * 2 + 1) << g.bs_shift), bar(bV + vs));
                        id = id1;
                        id1 = id2;
                        sc = sc1;
                    }
                }
                if (to_go <= kUnitCost) break;
                // the next unit, or the next sequence that has nodes (32 are looked at together)
                sp.at = 0;
                if (++sp.head == g.hkv) {
                    sp.head = 0;
                    ++sp.unit;
                    if (sp.unit > sh.full || (sp.unit == sh.full && !sh.left)) {
                        sp.unit = 0;
                        bool found = false;
                        for (++b;; b += 32) {
                            const int c = min(b + lane, B - 1);
                            int r0, st, en;
                            const int nn = nodes_of(c, r0, st, en);
                            const unsigned has = __ballot_sync(0xFFFFFFFFu, b + lane < B && nn > 0);
                            if (has || b + 32 >= B) {
                                const int l = has ? __ffs((int)has) - 1 : 0;
                                found = has;
                                b = min(b + l, B - 1);
                                n = __shfl_sync(0xFFFFFFFFu, nn, l);
                                row0 = __shfl_sync(0xFFFFFFFFu, r0, l);
                                start = __shfl_sync(0xFFFFFFFFu, st, l);
                                end = __shfl_sync(0xFFFFFFFFu, en, l);
                                break;
                            }
                        }
                        if (!found) break;  // (the inputs have changed since they were added up: the others' waits give up)
                        sh = Shape(n, end, A.tpt);
                    }
                    sp.one = sp.unit == sh.full;
                    sp.size = sp.one ? sh.size_left : sh.size_full;
                }
            }
            for (int u = max(0, sent - L::VS); u < sent; ++u) wait_tries(bar(bV + u % L::VS), (u / L::VS) & 1, kTries);  // (as above)
        } else if (warp == 13) {
            // ================= MMA =================
            // (Votes and reductions make what the loops turn on uniform: the descriptors then stay in uniform registers.)
            const bool issues = elect_one();
            const uint64_t d_q = desc_rows(sb + L::q, 1024), d_k = desc_rows(sb + L::k, 1024),
                           d_v = tc::smem_desc(sb + L::vb, kVLbo, kVSbo);
            constexpr uint32_t idesc_v = tc::idesc_bf16_f32(128, 128) | (1u << 16);
            int t = 0, turn = 0, asked = 0, ahead = 0;  // of the CTA: tiles, turns, items with queries from either side
            for (int i = 0; !__any_sync(0xFFFFFFFFu, bad); ++i) {
                const Item* it = record(i);
                if (!it) break;
                const int flags = __reduce_or_sync(0xFFFFFFFFu, it->flags), tiles = __reduce_max_sync(0xFFFFFFFFu, it->tiles);
                const int place = L::ahead && (flags & kOne) ? i & 1 : 0;
                if (flags & kAhead) wait(bQa, ahead++ & 1);
                else wait(bQ, asked++ & 1);
                if (L::ahead && lane == 0) mbar_arrive(bar(bQu + i % kUseRing));
                __syncwarp();
                const bool one = flags & kOne;
                const int turns = one ? tiles : 2 * tiles, deep = one ? 2 : 1;  // scores run that far ahead
                // scores of turn u: row tile u & 1 where there are two
                auto scores = [&](int u) {
                    const int x = one ? 0 : u & 1, tu = t + (one ? u : u >> 1), ks = tu % L::KS;
                    wait(bK + ks, (tu / L::KS) & 1);
                    __syncwarp();
                    tc::fence_after_sync();
                    if (issues) {
                        const uint64_t q = d_q + (place + x) * NT * 1024, kk = d_k + ks * 1024;
                        const uint32_t d = tmem + (one ? u % 3 : u & 1) * 128;
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int k = 0; k < 4; ++k) mma_f8_ss(d, q + j * 1024 + 2 * k, kk + 2 * k, idesc_f8(128, false), j > 0 || k > 0);
                        tc::commit(bar(bS + ((turn + u) & 3)));
                    }
                    __syncwarp();
                };
                for (int u = 0; u < min(deep, turns); ++u) scores(u);
                for (int u = 0; u < turns; ++u) {
                    // (the third part of tensor memory is an output of an item with two row tiles)
                    if (u == 0 && i > 0) wait(bOe, (i - 1) & 1);  // the last item's outputs are read
                    if (u + deep < turns) scores(u + deep);
                    const int x = one ? 0 : u & 1, tu = t + (one ? u : u >> 1), vb = tu & 1;
                    wait(bB + vb, (tu >> 1) & 1);
                    wait(bP + ((turn + u) & 3), ((turn + u) >> 2) & 1);
                    __syncwarp();
                    tc::fence_after_sync();
                    if (issues) {
                        const uint32_t s = tmem + (one ? u % 3 : u & 1) * 128, d = tmem + (one ? 384 : 256 + 128 * x);
                        const uint64_t v = d_v + vb * 2048;
#pragma unroll
                        for (int j = 0; j < 2; ++j)  // the weights, their remainders
#pragma unroll
                            for (int k = 0; k < 8; ++k) tc::mma_f16_ts(d, s + 32 * (k >> 1) + 8 * (k & 1) + 16 * j, v + 16 * k, idesc_v, u > x || j > 0 || k > 0);
                        tc::commit(bar(bO + ((turn + u) & 3)));
                    }
                    __syncwarp();
                    if (__any_sync(0xFFFFFFFFu, bad)) break;
                }
                t += tiles;
                turn += turns;
                if (flags & kLast) break;
            }
            // products may be in flight where a wait gave up: they end (again with a limit) before the memory is given back
            if (issues) tc::commit(bar(bEnd));
            __syncwarp();
            wait_tries(bar(bEnd), 0, kTries);
        } else if constexpr (L::ahead) {
            // ================= the next unit's queries, while this one's turns run =================
            // (Its place was the last but one's, which is done with once all softmax warps have this one's queries.)
            const int sub = lane >> 4, col = lane & 15;
            for (int i = 0;; ++i) {
                const Item* it = record(i);
                if (!it) break;
                const int flags = it->flags;
                if (flags & kAhead) {
                    wait(bQu + (i - 1) % kUseRing, ((i - 1) / kUseRing) & 1);
                    if (__any_sync(0xFFFFFFFFu, bad)) break;
                    const int place = place_of(it, i), left = it->n - it->first;
                    const T* q0 = static_cast<const T*>(A.a.q) + (int64_t)(it->row0 + it->first) * A.a.q_token + (int64_t)it->head * G * A.a.q_head + 8 * col;
                    int node = sub / G, gr = sub % G;
                    auto load = [&](int row, uint4 (&to)[4]) {  // rows row, row + 2 ..
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const bool in = row + 2 * k < A.tpt * G && node < left;
                            to[k] = in ? __ldg(reinterpret_cast<const uint4*>(q0 + (int64_t)node * A.a.q_token + (int64_t)gr * A.a.q_head)) : make_uint4(0, 0, 0, 0);
#pragma unroll
                            for (int y = 0; y < 2; ++y)
                                if (++gr == G) {
                                    gr = 0;
                                    ++node;
                                }
                        }
                    };
                    uint4 now[4], next[4];
                    load(sub, now);
#pragma unroll 1
                    for (int row = sub; row - sub < min(A.tpt, left) * G; row += 8) {
                        load(row + 8, next);
                        store_terms<T, NT, 4>(now, sm + L::q + place * NT * 16384, reinterpret_cast<float*>(sm + L::mult) + place * 128, row, col, A.a.sm_scale_log2);
#pragma unroll
                        for (int k = 0; k < 4; ++k) now[k] = next[k];
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(bQa));
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(bQu + i % kUseRing));
                if (flags & kLast) break;
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

// Joins the runs of every unit that was cut, in their order, one warp per row: block (run, 8 of its 256 rows).
template <typename T>
__global__ void __launch_bounds__(256) fp8_tree_join_kernel(const TreeArgs A) {
    const int lane = threadIdx.x & 31;
    grid_dependency_wait();
    grid_launch_dependents();
    const int c0 = blockIdx.x / (kUnitRows / 8), r = (int)(blockIdx.x % (kUnitRows / 8)) * 8 + (threadIdx.x >> 5);
    const int4 j = A.joins[c0];
    const int G = A.a.group, x = r / kRowsPerTile, rr = r % kRowsPerTile, node = x * A.tpt + rr / G;
    if (rr >= A.tpt * G || node >= j.z || j.x == 0) return;
    auto of = [&](int c) { return ((int64_t)(c0 + c) * 2 + (c == 0 ? 1 : 0)) * kUnitRows + r; };
    float4 o4 = make_float4(0.f, 0.f, 0.f, 0.f);
    float all = 0.f, mx = -INFINITY;
    for (int s0 = 0; s0 < j.x; s0 += 16) {
        const int n = min(16, j.x - s0);
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < n) ml = A.ml[of(s0 + lane)];
        float4 v[16];
#pragma unroll
        for (int s = 0; s < 16; ++s)
            v[s] = s < n ? *(reinterpret_cast<const float4*>(A.partials + of(s0 + s) * kHeadDim) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
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
            if (sum == 0.f) continue;  // nothing there
            all = fmaf(sum, ws, all);
            o4.x = fmaf(v[s].x, ws, o4.x);
            o4.y = fmaf(v[s].y, ws, o4.y);
            o4.z = fmaf(v[s].z, ws, o4.z);
            o4.w = fmaf(v[s].w, ws, o4.w);
        }
    }
    const float inv = all == 0.f ? 0.f : 1.f / all;
    T* out = static_cast<T*>(A.a.out) + ((int64_t)(j.y + node) * A.a.hq + (int64_t)j.w * G + rr % G) * kHeadDim;
    *(reinterpret_cast<uint2*>(out) + lane) = make_uint2(pack_two<T>(o4.x * inv, o4.y * inv), pack_two<T>(o4.z * inv, o4.w * inv));
}

int tokens_per_tile(int group) { return kRowsPerTile / group; }

// At least as many places as the list can have.
int64_t most_places(const Fp8Geometry& g, int64_t num_tokens, int batch, int group, int max_blocks) {
    const int64_t units = (num_tokens / (2 * tokens_per_tile(group)) + batch) * g.hkv;
    const int64_t size = 2 * (((int64_t)max_blocks * g.bs + kTok - 1) / kTok + 1) + kUnitCost;
    return units > INT_MAX || size > INT_MAX ? INT64_MAX : units * size;
}

int runs_of(const Fp8Geometry& g) { return g.num_sms > 0 ? g.num_sms : 1; }

template <typename T, int NT>
int launch(const TreeArgs& p, const CUtensorMap& map, int grid, cudaStream_t s) {
    auto kern = fp8_tree_kernel<T, NT>;
    static int done[64] = {};
    cudaError_t e = ensure_smem_limit(kern, TreeLayout<NT>::smem, done);
    if (e != cudaSuccess) return (int)e;
    // the warpgroups share out the registers that the block is launched with: a build that gave it fewer would wait for
    // the rest without end
    static const bool enough = [&] {
        cudaFuncAttributes f;
        return cudaFuncGetAttributes(&f, kern) == cudaSuccess && (f.numRegs + 7) / 8 * 8 * 2 >= kSoftRegs + kOtherRegs;
    }();
    if (!enough) return (int)cudaErrorInvalidConfiguration;
    e = launch_programmatic(kern, dim3((unsigned)grid), dim3(kThreads), (size_t)TreeLayout<NT>::smem, s, p, map);
    if (e != cudaSuccess) return (int)e;
    return (int)launch_programmatic(fp8_tree_join_kernel<T>, dim3((unsigned)(grid * (kUnitRows / 8))), dim3(256), 0, s, p);
}

}  // namespace

bool fp8_tree_counts(const Fp8Geometry& g, int64_t num_tokens, int batch, int group, int max_blocks) {
    return most_places(g, num_tokens, batch, group, max_blocks) < INT_MAX;
}

// Partials, their maxima and sums, what is to be joined, the NaN notes: of the same size for every call.
size_t fp8_tree_workspace(const Fp8Geometry& g) {
    return (size_t)runs_of(g) * (2 * kUnitRows * (kHeadDim * sizeof(float) + sizeof(float2)) + sizeof(int4) + kNanRing * kHeadDim * sizeof(int));
}

int launch_fp8_tree(const Fp8AttnArgs& a, const CUtensorMap& map, void* workspace, void* stream) {
    TreeArgs p{};
    p.a = a;
    p.tpt = tokens_per_tile(a.group);
    const int runs = runs_of(a.g);
    p.partials = static_cast<float*>(workspace);
    p.ml = reinterpret_cast<float2*>(p.partials + (size_t)runs * 2 * kUnitRows * kHeadDim);
    p.joins = reinterpret_cast<int4*>(p.ml + (size_t)runs * 2 * kUnitRows);
    p.nan = reinterpret_cast<int*>(p.joins + runs);
    p.stall_cycles = test_stall_cycles();
    const int64_t most = most_places(a.g, a.b.num_tokens, a.b.batch, a.group, a.b.max_blocks);
    const int grid = (int)(most / kLeastRun < runs ? most / kLeastRun < 1 ? 1 : most / kLeastRun : runs);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return a.dtype == TQ_BF16 ? launch<__nv_bfloat16, 2>(p, map, grid, s) : launch<__half, 3>(p, map, grid, s);
}

}  // namespace tq
