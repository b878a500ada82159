// Host side of the 8-bit paged cache: argument checks, the cache descriptor
// and the calls that launch its kernels.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <new>

#include "tq_fp8.h"

namespace {

using namespace tq;

tq_status fail(tq_status s, const char* what) {
    set_error("%s", what);
    return s;
}

tq_status cuda_fail(cudaError_t e, const char* what) {
    set_error("%s: %s", what, cudaGetErrorString(e));
    return TQ_ERR_CUDA;
}

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// Strided rows of 128 elements: every row on a 16-byte boundary.
bool bad_rows(const void* p, int64_t token, int64_t head, int64_t elem) {
    return misaligned(p, 16) || token < 0 || head < 0 || token * elem % 16 || head * elem % 16;
}

tq_status check_device(const tq_fp8_cache* c) {
    int dev = -1;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev != c->device) return fail(TQ_ERR_INVALID_ARG, "the current device is not the cache's");
    return TQ_OK;
}

// The arguments that the ragged calls share.
tq_status check_batch(const tq_fp8_cache* c, int64_t num_tokens, int batch, const int32_t* cu, const int32_t* start,
                      const int32_t* block_table, int max_blocks) {
    if (!c) return fail(TQ_ERR_INVALID_ARG, "cache is NULL");
    if (num_tokens < 0 || num_tokens > INT_MAX || batch < 0) return fail(TQ_ERR_INVALID_ARG, "bad num_tokens or batch");
    if (num_tokens == 0 || batch == 0) return TQ_OK;
    if (!cu || !start || !block_table)
        return fail(TQ_ERR_INVALID_ARG, "cu_tokens, start and block_table must be non-NULL");
    if (max_blocks <= 0) return fail(TQ_ERR_INVALID_ARG, "max_blocks_per_seq must be positive");
    return TQ_OK;
}

bool known(tq_dtype t) { return t == TQ_F32 || t == TQ_BF16 || t == TQ_F16; }

Fp8Batch make_batch(int64_t num_tokens, int batch, const int32_t* cu, const int32_t* start, const int32_t* block_table,
                    int max_blocks) {
    Fp8Batch b;
    b.batch = batch;
    b.num_tokens = num_tokens;
    b.cu = cu;
    b.start = start;
    b.block_table = block_table;
    b.max_blocks = max_blocks;
    return b;
}

// The arguments that both attention calls share, once the batch is known to be non-empty.
tq_status check_attn(const tq_fp8_cache* c, const void* q, tq_dtype dtype, int64_t q_token, int64_t q_head, int hq,
                     float sm_scale, const void* out, const void* workspace, size_t workspace_bytes, size_t need) {
    if (hq <= 0 || hq % c->g.hkv) return fail(TQ_ERR_INVALID_ARG, "num_q_heads must be a multiple of num_kv_heads");
    if (hq / c->g.hkv > kFp8MaxGroup) return fail(TQ_ERR_UNSUPPORTED, "more than 128 query heads per KV head");
    if (dtype == TQ_F32) return fail(TQ_ERR_UNSUPPORTED, "queries must be bf16 or fp16");
    if (dtype != TQ_BF16 && dtype != TQ_F16) return fail(TQ_ERR_INVALID_ARG, "bad dtype");
    if (!q || !out || !workspace) return fail(TQ_ERR_INVALID_ARG, "q, out and workspace must be non-NULL");
    if (bad_rows(q, q_token, q_head, 2)) return fail(TQ_ERR_INVALID_ARG, "q's rows must be 16-byte aligned");
    if (misaligned(out, 16)) return fail(TQ_ERR_INVALID_ARG, "out must be 16-byte aligned");
    if (misaligned(workspace, 256)) return fail(TQ_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (!(sm_scale > 0.0f) || !std::isfinite(sm_scale)) return fail(TQ_ERR_INVALID_ARG, "sm_scale must be positive");
    if (workspace_bytes < need) {
        set_error("workspace has %zu bytes, needs %zu", workspace_bytes, need);
        return TQ_ERR_WORKSPACE;
    }
    return TQ_OK;
}

}  // namespace

namespace tq {

bool fp8_tensor_map(CUtensorMap* map, const Fp8Geometry& g, int rows) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fn)
        return false;
    const cuuint64_t dims[2] = {(cuuint64_t)kHeadDim, (cuuint64_t)g.num_blocks * g.hkv * 2 * g.bs};
    const cuuint64_t strides[1] = {(cuuint64_t)kHeadDim};
    const cuuint32_t box[2] = {(cuuint32_t)kHeadDim, (cuuint32_t)rows};
    const cuuint32_t estr[2] = {1, 1};
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn)(
               map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, g.pool, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tq

extern "C" {

TQ_API tq_status tq_fp8_cache_create(void* pool, float* scales, int64_t num_blocks, int block_size, int num_kv_heads,
                                     int d, tq_fp8_cache** out) {
    if (!out) return fail(TQ_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    if (!pool || !scales) return fail(TQ_ERR_INVALID_ARG, "pool and scales must be non-NULL");
    if (misaligned(pool, 16) || misaligned(scales, 16))
        return fail(TQ_ERR_INVALID_ARG, "pool and scales must be 16-byte aligned");
    if (num_blocks <= 0 || num_kv_heads <= 0 || block_size <= 0 || d <= 0)
        return fail(TQ_ERR_INVALID_ARG, "sizes must be positive");
    if (d != kHeadDim) return fail(TQ_ERR_UNSUPPORTED, "head dim must be 128");
    if (block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128)
        return fail(TQ_ERR_UNSUPPORTED, "block_size must be 16, 32, 64 or 128");
    // rows of the pool are numbered in 32 bits
    if (num_kv_heads > 65536 || num_blocks > (int64_t)INT_MAX / (2 * (int64_t)block_size * num_kv_heads))
        return fail(TQ_ERR_UNSUPPORTED, "the pool has more than 2^31 rows of 128 codes");
    tq_fp8_cache* c = new (std::nothrow) tq_fp8_cache();
    if (!c) return fail(TQ_ERR_INVALID_ARG, "out of host memory");
    c->g.pool = static_cast<uint8_t*>(pool);
    c->g.scales = scales;
    c->g.num_blocks = num_blocks;
    c->g.hkv = num_kv_heads;
    c->g.bs = block_size;
    while ((1 << c->g.bs_shift) < block_size) ++c->g.bs_shift;
    // without a device the descriptor is made all the same, and the calls that launch refuse
    if (cudaGetDevice(&c->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&c->g.num_sms, cudaDevAttrMultiProcessorCount, c->device) != cudaSuccess) {
        cudaGetLastError();
        c->device = -1;
        c->g.num_sms = 0;
    } else if (!fp8_tensor_map(&c->map, c->g, block_size == 16 ? 32 : block_size) || !fp8_tensor_map(&c->side, c->g, block_size)) {
        delete c;
        return fail(TQ_ERR_CUDA, "making the pool's tensor map failed");
    }
    *out = c;
    return TQ_OK;
}

TQ_API void tq_fp8_cache_free(tq_fp8_cache* c) { delete c; }

TQ_API tq_status tq_fp8_write(const tq_fp8_cache* c, const void* K, const void* V, tq_dtype dtype,
                              int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                              int64_t v_head_stride, int64_t num_tokens, int batch, const int32_t* cu_tokens,
                              const int32_t* start, const int32_t* block_table, int max_blocks_per_seq,
                              int32_t* dev_status, void* stream) {
    tq_status st = check_batch(c, num_tokens, batch, cu_tokens, start, block_table, max_blocks_per_seq);
    if (st != TQ_OK || num_tokens == 0 || batch == 0) return st;
    if (!known(dtype)) return fail(TQ_ERR_INVALID_ARG, "bad dtype");
    if (!K || !V) return fail(TQ_ERR_INVALID_ARG, "K and V must be non-NULL");
    const int64_t elem = dtype == TQ_F32 ? 4 : 2;
    if (bad_rows(K, k_token_stride, k_head_stride, elem) || bad_rows(V, v_token_stride, v_head_stride, elem))
        return fail(TQ_ERR_INVALID_ARG, "the rows of K and V must be 16-byte aligned");
    Fp8WriteArgs a{};
    a.g = c->g;
    a.b = make_batch(num_tokens, batch, cu_tokens, start, block_table, max_blocks_per_seq);
    if (!fp8_rows_count(a.g, a.b)) return fail(TQ_ERR_UNSUPPORTED, "more rows than a launch holds");
    if ((st = check_device(c)) != TQ_OK) return st;
    a.K = K;
    a.V = V;
    a.dtype = (int)dtype;
    a.k_token = k_token_stride;
    a.k_head = k_head_stride;
    a.v_token = v_token_stride;
    a.v_head = v_head_stride;
    a.status = dev_status;
    const int e = launch_fp8_write(a, stream);
    return e ? cuda_fail((cudaError_t)e, "write launch") : TQ_OK;
}

TQ_API tq_status tq_fp8_read(const tq_fp8_cache* c, void* K, void* V, tq_dtype dtype, int64_t num_tokens, int batch,
                             const int32_t* cu_tokens, const int32_t* start, const int32_t* block_table,
                             int max_blocks_per_seq, int32_t* dev_status, void* stream) {
    tq_status st = check_batch(c, num_tokens, batch, cu_tokens, start, block_table, max_blocks_per_seq);
    if (st != TQ_OK || num_tokens == 0 || batch == 0) return st;
    if (!known(dtype)) return fail(TQ_ERR_INVALID_ARG, "bad dtype");
    if (!K || !V) return fail(TQ_ERR_INVALID_ARG, "K and V must be non-NULL");
    if (misaligned(K, 16) || misaligned(V, 16)) return fail(TQ_ERR_INVALID_ARG, "K and V must be 16-byte aligned");
    Fp8ReadArgs a{};
    a.g = c->g;
    a.b = make_batch(num_tokens, batch, cu_tokens, start, block_table, max_blocks_per_seq);
    if (!fp8_rows_count(a.g, a.b)) return fail(TQ_ERR_UNSUPPORTED, "more rows than a launch holds");
    if ((st = check_device(c)) != TQ_OK) return st;
    a.K = K;
    a.V = V;
    a.dtype = (int)dtype;
    a.status = dev_status;
    const int e = launch_fp8_read(a, stream);
    return e ? cuda_fail((cudaError_t)e, "read launch") : TQ_OK;
}

TQ_API tq_status tq_fp8_append(const tq_fp8_cache* c, const void* K, const void* V, tq_dtype dtype, int64_t k_token_stride,
                               int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride, const void* q,
                               int64_t q_token_stride, int64_t q_head_stride, int num_q_heads, void* q_out,
                               int64_t out_token_stride, int64_t out_head_stride, int64_t num_tokens, int batch,
                               const int32_t* cu_tokens, const int32_t* start, const int32_t* block_table, int max_blocks_per_seq,
                               const int32_t* positions, const float* table, int64_t num_positions, int rot,
                               tq_rotary_layout layout, int32_t* dev_status, void* stream) {
    tq_status st = check_batch(c, num_tokens, batch, cu_tokens, start, block_table, max_blocks_per_seq);
    if (st != TQ_OK) return st;
    bool unsupported;
    const char* fault = rotary_table_fault(table, num_positions, rot, (int)layout, &unsupported);
    if (fault) return fail(unsupported ? TQ_ERR_UNSUPPORTED : TQ_ERR_INVALID_ARG, fault);
    if (rot > kHeadDim) return fail(TQ_ERR_INVALID_ARG, "more rotated dims than a head has");
    if (!known(dtype)) return fail(TQ_ERR_INVALID_ARG, "bad dtype");
    if (num_tokens == 0 || batch == 0) return TQ_OK;
    if (!K || !V) return fail(TQ_ERR_INVALID_ARG, "K and V must be non-NULL");
    const int64_t elem = dtype == TQ_F32 ? 4 : 2;
    if (bad_rows(K, k_token_stride, k_head_stride, elem) || bad_rows(V, v_token_stride, v_head_stride, elem))
        return fail(TQ_ERR_INVALID_ARG, "the rows of K and V must be 16-byte aligned");
    if (q) {
        if (num_q_heads <= 0 || !q_out) return fail(TQ_ERR_INVALID_ARG, "queries need num_q_heads and q_out");
        if (bad_rows(q, q_token_stride, q_head_stride, elem) || bad_rows(q_out, out_token_stride, out_head_stride, elem))
            return fail(TQ_ERR_INVALID_ARG, "the rows of q and q_out must be 16-byte aligned");
        if (const char* f = rotary_rows_fault(q, q_token_stride, q_head_stride, q_out, out_token_stride, out_head_stride, num_tokens,
                                              num_q_heads, kHeadDim, (int)elem))
            return fail(TQ_ERR_INVALID_ARG, f);
    }
    Fp8AppendArgs a{};
    a.g = c->g;
    a.b = make_batch(num_tokens, batch, cu_tokens, start, block_table, max_blocks_per_seq);
    if (!fp8_append_counts(a.g, a.b, q ? num_q_heads : 0)) return fail(TQ_ERR_UNSUPPORTED, "more rows than a launch holds");
    if ((st = check_device(c)) != TQ_OK) return st;
    a.K = K;
    a.V = V;
    a.q = q;
    a.q_out = q_out;
    a.dtype = (int)dtype;
    a.k_token = k_token_stride;
    a.k_head = k_head_stride;
    a.v_token = v_token_stride;
    a.v_head = v_head_stride;
    a.q_token = q_token_stride;
    a.q_head = q_head_stride;
    a.out_token = out_token_stride;
    a.out_head = out_head_stride;
    a.hq = q ? num_q_heads : 0;
    a.r.table = table;
    a.r.positions = num_positions;
    a.r.rot = rot;
    a.r.interleaved = layout == TQ_ROTARY_INTERLEAVED;
    a.positions = positions;
    a.status = dev_status;
    const int e = launch_fp8_append(a, stream);
    return e ? cuda_fail((cudaError_t)e, "append launch") : TQ_OK;
}

TQ_API tq_status tq_fp8_keep(const tq_fp8_cache* c, int64_t num_kept, int batch, const int32_t* cu_kept, const int32_t* kept,
                             const int32_t* start, const int32_t* block_table, int max_blocks_per_seq, int32_t* dev_status,
                             void* stream) {
    tq_status st = check_batch(c, num_kept, batch, cu_kept, start, block_table, max_blocks_per_seq);
    if (st != TQ_OK || num_kept == 0 || batch == 0) return st;
    if (!kept) return fail(TQ_ERR_INVALID_ARG, "kept must be non-NULL");
    if (!fp8_keep_counts(c->g, batch)) return fail(TQ_ERR_UNSUPPORTED, "more sequences than a launch holds");
    if ((st = check_device(c)) != TQ_OK) return st;
    Fp8KeepArgs a{};
    a.g = c->g;
    a.b = make_batch(num_kept, batch, cu_kept, start, block_table, max_blocks_per_seq);
    a.kept = kept;
    a.status = dev_status;
    const int e = launch_fp8_keep(a, stream);
    return e ? cuda_fail((cudaError_t)e, "keep launch") : TQ_OK;
}

TQ_API size_t tq_fp8_decode_workspace_bytes(const tq_fp8_cache* c, int batch, int num_q_heads) {
    if (!c || batch <= 0 || num_q_heads <= 0 || num_q_heads % c->g.hkv) return 0;
    return fp8_decode_workspace(c->g, batch, num_q_heads / c->g.hkv);
}

TQ_API size_t tq_fp8_decode_counters_offset(const tq_fp8_cache* c) { return c ? fp8_decode_counters_at(c->g) : 0; }

TQ_API tq_status tq_fp8_decode_attention(const tq_fp8_cache* c, const void* q, tq_dtype dtype, int64_t q_seq_stride,
                                         int64_t q_head_stride, int batch, int num_q_heads, const int32_t* block_table,
                                         int max_blocks_per_seq, const int32_t* lens, float sm_scale, void* out,
                                         void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
    if (!c) return fail(TQ_ERR_INVALID_ARG, "cache is NULL");
    if (batch < 0) return fail(TQ_ERR_INVALID_ARG, "batch < 0");
    if (batch == 0) return TQ_OK;
    if (!block_table || !lens) return fail(TQ_ERR_INVALID_ARG, "block_table and lens must be non-NULL");
    if (max_blocks_per_seq <= 0) return fail(TQ_ERR_INVALID_ARG, "max_blocks_per_seq must be positive");
    tq_status st = check_attn(c, q, dtype, q_seq_stride, q_head_stride, num_q_heads, sm_scale, out, workspace,
                              workspace_bytes, tq_fp8_decode_workspace_bytes(c, batch, num_q_heads));
    if (st != TQ_OK) return st;
    if (!fp8_decode_counts(c->g, batch, num_q_heads / c->g.hkv, max_blocks_per_seq))
        return fail(TQ_ERR_UNSUPPORTED, "batch, heads and block table make 2^31 tiles or more");
    if ((st = check_device(c)) != TQ_OK) return st;
    Fp8AttnArgs a{};
    a.g = c->g;
    a.b = make_batch(batch, batch, nullptr, nullptr, block_table, max_blocks_per_seq);
    a.lens = lens;
    a.q = q;
    a.dtype = (int)dtype;
    a.q_token = q_seq_stride;
    a.q_head = q_head_stride;
    a.hq = num_q_heads;
    a.group = num_q_heads / c->g.hkv;
    a.sm_scale_log2 = sm_scale * 1.4426950408889634f;
    a.out = out;
    a.status = dev_status;
    const int e = launch_fp8_decode(a, c->map, workspace, stream);
    return e ? cuda_fail((cudaError_t)e, "decode launch") : TQ_OK;
}

TQ_API size_t tq_fp8_prefill_workspace_bytes(const tq_fp8_cache* c, int64_t num_tokens, int batch, int num_q_heads) {
    if (!c || num_tokens <= 0 || num_tokens > INT_MAX || batch <= 0 || num_q_heads <= 0 || num_q_heads % c->g.hkv || num_q_heads / c->g.hkv > kFp8MaxGroup)
        return 0;
    return fp8_prefill_workspace(c->g, num_tokens, batch, num_q_heads / c->g.hkv);
}

TQ_API tq_status tq_fp8_prefill_attention(const tq_fp8_cache* c, const void* q, tq_dtype dtype, int64_t q_token_stride,
                                          int64_t q_head_stride, int64_t num_tokens, int batch, int num_q_heads,
                                          const int32_t* cu_tokens, const int32_t* start, const int32_t* block_table,
                                          int max_blocks_per_seq, float sm_scale, void* out, void* workspace,
                                          size_t workspace_bytes, int32_t* dev_status, void* stream) {
    tq_status st = check_batch(c, num_tokens, batch, cu_tokens, start, block_table, max_blocks_per_seq);
    if (st != TQ_OK || num_tokens == 0 || batch == 0) return st;
    st = check_attn(c, q, dtype, q_token_stride, q_head_stride, num_q_heads, sm_scale, out, workspace, workspace_bytes,
                    tq_fp8_prefill_workspace_bytes(c, num_tokens, batch, num_q_heads));
    if (st != TQ_OK) return st;
    if (!fp8_prefill_counts(c->g, num_tokens, batch, num_q_heads / c->g.hkv))
        return fail(TQ_ERR_UNSUPPORTED, "more query rows than a launch holds");
    if ((st = check_device(c)) != TQ_OK) return st;
    Fp8AttnArgs a{};
    a.g = c->g;
    a.b = make_batch(num_tokens, batch, cu_tokens, start, block_table, max_blocks_per_seq);
    a.q = q;
    a.dtype = (int)dtype;
    a.q_token = q_token_stride;
    a.q_head = q_head_stride;
    a.hq = num_q_heads;
    a.group = num_q_heads / c->g.hkv;
    a.sm_scale_log2 = sm_scale * 1.4426950408889634f;
    a.out = out;
    a.status = dev_status;
    const int e = launch_fp8_prefill(a, c->side, workspace, stream);
    return e ? cuda_fail((cudaError_t)e, "prefill launch") : TQ_OK;
}

TQ_API size_t tq_fp8_tree_workspace_bytes(const tq_fp8_cache* c, int64_t num_tokens, int batch, int num_q_heads) {
    if (!c || num_tokens <= 0 || num_tokens > INT_MAX || batch <= 0 || num_q_heads <= 0 || num_q_heads % c->g.hkv || num_q_heads / c->g.hkv > kFp8MaxGroup)
        return 0;
    return fp8_tree_workspace(c->g);
}

TQ_API tq_status tq_fp8_tree_attention(const tq_fp8_cache* c, const void* q, tq_dtype dtype, int64_t q_token_stride,
                                       int64_t q_head_stride, int64_t num_tokens, int batch, int num_q_heads,
                                       const int32_t* cu_tokens, const int32_t* start, const int32_t* block_table,
                                       int max_blocks_per_seq, const uint64_t* mask, int mask_words, float sm_scale, void* out,
                                       void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
    tq_status st = check_batch(c, num_tokens, batch, cu_tokens, start, block_table, max_blocks_per_seq);
    if (st != TQ_OK || num_tokens == 0 || batch == 0) return st;
    st = check_attn(c, q, dtype, q_token_stride, q_head_stride, num_q_heads, sm_scale, out, workspace, workspace_bytes,
                    tq_fp8_tree_workspace_bytes(c, num_tokens, batch, num_q_heads));
    if (st != TQ_OK) return st;
    if (!mask || misaligned(mask, 8)) return fail(TQ_ERR_INVALID_ARG, "mask must be non-NULL and 8-byte aligned");
    if (mask_words <= 0) return fail(TQ_ERR_INVALID_ARG, "mask_words must be positive");
    if (!fp8_tree_counts(c->g, num_tokens, batch, num_q_heads / c->g.hkv, max_blocks_per_seq))
        return fail(TQ_ERR_UNSUPPORTED, "tokens, heads and block table make 2^31 steps or more");
    if ((st = check_device(c)) != TQ_OK) return st;
    Fp8AttnArgs a{};
    a.g = c->g;
    a.b = make_batch(num_tokens, batch, cu_tokens, start, block_table, max_blocks_per_seq);
    a.q = q;
    a.dtype = (int)dtype;
    a.q_token = q_token_stride;
    a.q_head = q_head_stride;
    a.hq = num_q_heads;
    a.group = num_q_heads / c->g.hkv;
    a.mask = mask;
    a.words = mask_words;
    a.sm_scale_log2 = sm_scale * 1.4426950408889634f;
    a.out = out;
    a.status = dev_status;
    const int e = launch_fp8_tree(a, c->side, workspace, stream);
    return e ? cuda_fail((cudaError_t)e, "tree attention launch") : TQ_OK;
}

}  // extern "C"
