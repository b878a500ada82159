// Internal declarations of the 8-bit paged cache (e4m3 codes, one power-of-two
// scale per block, KV head and side).
#pragma once

#include <cuda.h>

#include <cstdint>

#include "tq_internal.h"
#include "tq_rotary.h"

namespace tq {

constexpr int kFp8MinExp = -120;   // exponent of the scale of a block of zeros
constexpr int kFp8MaxGroup = 128;  // query heads per KV head

// Pool: codes [num_blocks][hkv][2: K, V][bs][128], scales [num_blocks][hkv][2].
struct Fp8Geometry {
    uint8_t* pool;
    float* scales;
    int64_t num_blocks;
    int hkv;
    int bs;        // tokens of a block: 16, 32, 64 or 128
    int bs_shift;  // log2(bs)
    int num_sms;
};

// The tokens of a ragged batch: sequence b's rows cu[b] .. cu[b + 1] - 1 of the
// packed tensors are its positions start[b] ..; block_table [batch][max_blocks].
struct Fp8Batch {
    int batch;
    int64_t num_tokens;  // rows of the packed tensors
    const int32_t* cu;
    const int32_t* start;
    const int32_t* block_table;
    int max_blocks;
};

struct Fp8WriteArgs {
    Fp8Geometry g;
    Fp8Batch b;
    const void* K;
    const void* V;
    int dtype;
    int64_t k_token, k_head, v_token, v_head;  // strides in elements
    int32_t* status;
};
struct Fp8ReadArgs {
    Fp8Geometry g;
    Fp8Batch b;
    void* K;
    void* V;
    int dtype;
    int32_t* status;
};
struct Fp8AppendArgs {
    Fp8Geometry g;
    Fp8Batch b;
    const void* K;
    const void* V;
    const void* q;  // null: no queries
    void* q_out;
    int dtype;
    int64_t k_token, k_head, v_token, v_head, q_token, q_head, out_token, out_head;  // strides in elements
    int hq;
    RotaryTable r;
    const int32_t* positions;  // of every packed row; null: start + its place in the sequence
    int32_t* status;
};
struct Fp8KeepArgs {
    Fp8Geometry g;
    Fp8Batch b;            // of the kept rows
    const int32_t* kept;   // row r of a sequence is what was at position start + kept[r]
    int32_t* status;
};
struct Fp8AttnArgs {
    Fp8Geometry g;
    Fp8Batch b;
    const int32_t* lens;  // decode: one query row per sequence at position lens[b] - 1
    const void* q;
    int dtype;
    int64_t q_token, q_head;  // strides in elements
    int hq, group;
    const uint64_t* mask;  // trees: of every packed row `words` words, bit j: it sees row j of its sequence
    int words;
    float sm_scale_log2;
    void* out;  // [rows][hq][128], q's type
    int32_t* status;
};

bool fp8_rows_count(const Fp8Geometry& g, const Fp8Batch& b);  // work items are counted in 32 bits
int launch_fp8_write(const Fp8WriteArgs& a, void* stream);
int launch_fp8_read(const Fp8ReadArgs& a, void* stream);
bool fp8_append_counts(const Fp8Geometry& g, const Fp8Batch& b, int hq);
int launch_fp8_append(const Fp8AppendArgs& a, void* stream);
bool fp8_keep_counts(const Fp8Geometry& g, int batch);
int launch_fp8_keep(const Fp8KeepArgs& a, void* stream);
// The pool as rows of 128 codes: the tensor map whose boxes have `rows` of them.
bool fp8_tensor_map(CUtensorMap* map, const Fp8Geometry& g, int rows);
bool fp8_decode_counts(const Fp8Geometry& g, int batch, int group, int max_blocks);  // tiles are counted in 32 bits
size_t fp8_decode_workspace(const Fp8Geometry& g, int batch, int group);
size_t fp8_decode_counters_at(const Fp8Geometry& g);  // the workspace's part that has to be zero starts there
int launch_fp8_decode(const Fp8AttnArgs& a, const CUtensorMap& map, void* workspace, void* stream);
bool fp8_prefill_counts(const Fp8Geometry& g, int64_t num_tokens, int batch, int group);  // the grid fits 32 bits
size_t fp8_prefill_workspace(const Fp8Geometry& g, int64_t num_tokens, int batch, int group);
int launch_fp8_prefill(const Fp8AttnArgs& a, const CUtensorMap& map, void* workspace, void* stream);
bool fp8_tree_counts(const Fp8Geometry& g, int64_t num_tokens, int batch, int group, int max_blocks);  // steps are counted in 32 bits
size_t fp8_tree_workspace(const Fp8Geometry& g);
int launch_fp8_tree(const Fp8AttnArgs& a, const CUtensorMap& map, void* workspace, void* stream);

}  // namespace tq

struct tq_fp8_cache {
    tq::Fp8Geometry g;
    int device;       // -1: made without one
    CUtensorMap map;   // boxes of a block's keys or values of one head; with blocks of 16 tokens of both
    CUtensorMap side;  // boxes of a block's keys or values
};
