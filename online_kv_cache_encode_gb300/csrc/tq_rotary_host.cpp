// Host side of the rotary positions: frequencies, argument checks and the calls that launch the kernels.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "tq_rotary.h"

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

// a * b + c for non-negative numbers, or -1 where it passes 2^62.
int64_t mul_add(int64_t a, int64_t b, int64_t c) {
    const __int128 x = (__int128)a * b + c;
    return x > ((__int128)1 << 62) ? -1 : (int64_t)x;
}

// Elements from the first to behind the last of rows [tokens][heads][d], or -1.
int64_t span(int64_t tokens, int heads, int d, int64_t token, int64_t head) {
    const int64_t h = mul_add(heads - 1, head, d);
    return h < 0 ? -1 : mul_add(tokens - 1, token, h);
}

}  // namespace

namespace tq {

const char* rotary_table_fault(const float* table, int64_t positions, int rot, int layout, bool* unsupported) {
    *unsupported = false;
    if (!table || misaligned(table, 16)) return "the table must be non-NULL and 16-byte aligned";
    if (positions <= 0) return "the table's positions must be positive";
    if (rot <= 0) return "the rotated dims must be positive";
    if (layout != TQ_ROTARY_HALF && layout != TQ_ROTARY_INTERLEAVED) return "bad layout";
    *unsupported = true;
    if (rot % 16 || rot > kRotaryMaxDim) return "the rotated dims must be a multiple of 16, at most 256";
    if (positions > INT_MAX) return "more than 2^31 - 1 positions";
    return nullptr;
}

const char* rotary_rows_fault(const void* x, int64_t x_token, int64_t x_head, const void* out, int64_t out_token, int64_t out_head,
                              int64_t tokens, int heads, int d, int elem) {
    const int64_t nx = span(tokens, heads, d, x_token, x_head), no = span(tokens, heads, d, out_token, out_head);
    if (nx < 0 || no < 0) return "strides past the address space";
    // output rows apart from one another: the heads of a token together, or the tokens of a head
    const bool heads_in = (heads == 1 || out_head >= d) && (tokens == 1 || out_token >= (heads - 1) * out_head + d);
    const bool tokens_in = (tokens == 1 || out_token >= d) && (heads == 1 || out_head >= (tokens - 1) * out_token + d);
    if (!heads_in && !tokens_in) return "the output's rows overlap";
    const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(out);
    const bool in_place = a == b && (tokens == 1 || x_token == out_token) && (heads == 1 || x_head == out_head);
    if (!in_place && a < b + (uintptr_t)no * elem && b < a + (uintptr_t)nx * elem)
        return "input and output overlap without being the same";
    return nullptr;
}

}  // namespace tq

extern "C" {

TQ_API tq_status tq_rotary_frequencies(int rot, double base, tq_rotary_scaling scaling, double factor, double original_positions,
                                       double low_turns, double high_turns, double* out) {
    if (!out) return fail(TQ_ERR_INVALID_ARG, "out is NULL");
    if (rot <= 0 || rot % 2) return fail(TQ_ERR_INVALID_ARG, "the rotated dims must be positive and even");
    if (!(base > 0.0) || !std::isfinite(base)) return fail(TQ_ERR_INVALID_ARG, "base must be positive");
    if (scaling != TQ_ROTARY_PLAIN && scaling != TQ_ROTARY_LINEAR && scaling != TQ_ROTARY_BASE && scaling != TQ_ROTARY_PARTS)
        return fail(TQ_ERR_INVALID_ARG, "bad scaling");
    if (scaling != TQ_ROTARY_PLAIN && (!(factor > 0.0) || !std::isfinite(factor)))
        return fail(TQ_ERR_INVALID_ARG, "factor must be positive");
    if (scaling == TQ_ROTARY_BASE && rot <= 2) return fail(TQ_ERR_INVALID_ARG, "a scaled base needs more than 2 rotated dims");
    if (scaling == TQ_ROTARY_PARTS && (!(original_positions > 0.0) || !std::isfinite(original_positions) || !(low_turns < high_turns) ||
                                       !std::isfinite(low_turns) || !std::isfinite(high_turns)))
        return fail(TQ_ERR_INVALID_ARG, "original_positions must be positive and low_turns below high_turns");
    if (scaling == TQ_ROTARY_BASE) base *= std::pow(factor, (double)rot / (rot - 2));
    for (int j = 0; j < rot / 2; ++j) {
        double f = std::pow(base, -2.0 * j / rot);
        if (scaling == TQ_ROTARY_LINEAR) f /= factor;
        if (scaling == TQ_ROTARY_PARTS) {
            const double turns = original_positions * f / (2.0 * 3.14159265358979323846);
            double keep = (turns - low_turns) / (high_turns - low_turns);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            f = (1.0 - keep) * f / factor + keep * f;
        }
        out[j] = f;
    }
    return TQ_OK;
}

TQ_API tq_status tq_rotary_table(const double* frequencies, int rot, double magnitude, int64_t num_positions, float* table,
                                 void* stream) {
    bool unsupported;
    if (!frequencies) return fail(TQ_ERR_INVALID_ARG, "frequencies is NULL");
    const char* fault = rotary_table_fault(table, num_positions, rot, TQ_ROTARY_HALF, &unsupported);
    if (fault) return fail(unsupported ? TQ_ERR_UNSUPPORTED : TQ_ERR_INVALID_ARG, fault);
    if (!(magnitude > 0.0) || !std::isfinite(magnitude)) return fail(TQ_ERR_INVALID_ARG, "magnitude must be positive");
    for (int j = 0; j < rot / 2; ++j)
        if (!std::isfinite(frequencies[j])) return fail(TQ_ERR_INVALID_ARG, "a frequency is not finite");
    const int e = launch_rotary_table(frequencies, rot, magnitude, num_positions, table, stream);
    return e ? cuda_fail((cudaError_t)e, "rotary table launch") : TQ_OK;
}

TQ_API tq_status tq_rotary(const void* x, tq_dtype dtype, int64_t x_token_stride, int64_t x_head_stride, int64_t num_tokens,
                           int num_heads, int d, const int32_t* positions, const float* table, int64_t num_positions, int rot,
                           tq_rotary_layout layout, int transpose, void* out, int64_t out_token_stride, int64_t out_head_stride,
                           int32_t* dev_status, void* stream) {
    if (num_tokens < 0 || num_heads < 0 || d <= 0) return fail(TQ_ERR_INVALID_ARG, "bad num_tokens, num_heads or d");
    bool unsupported;
    const char* fault = rotary_table_fault(table, num_positions, rot, (int)layout, &unsupported);
    if (fault) return fail(unsupported ? TQ_ERR_UNSUPPORTED : TQ_ERR_INVALID_ARG, fault);
    if (rot > d) return fail(TQ_ERR_INVALID_ARG, "more rotated dims than a head has");
    if (d % 16 || d > 4096) return fail(TQ_ERR_UNSUPPORTED, "the head dim must be a multiple of 16, at most 4096");
    if (dtype != TQ_F32 && dtype != TQ_BF16 && dtype != TQ_F16) return fail(TQ_ERR_INVALID_ARG, "bad dtype");
    if (num_tokens == 0 || num_heads == 0) return TQ_OK;
    if (!x || !out || !positions) return fail(TQ_ERR_INVALID_ARG, "x, positions and out must be non-NULL");
    const int64_t elem = dtype == TQ_F32 ? 4 : 2;
    auto bad_rows = [&](const void* p, int64_t token, int64_t head) {
        return misaligned(p, 16) || token < 0 || head < 0 || token > INT64_MAX / 4 || head > INT64_MAX / 4 || token * elem % 16 ||
               head * elem % 16;
    };
    if (bad_rows(x, x_token_stride, x_head_stride) || bad_rows(out, out_token_stride, out_head_stride))
        return fail(TQ_ERR_INVALID_ARG, "the rows of x and out must be 16-byte aligned");
    fault = rotary_rows_fault(x, x_token_stride, x_head_stride, out, out_token_stride, out_head_stride, num_tokens, num_heads, d, (int)elem);
    if (fault) return fail(TQ_ERR_INVALID_ARG, fault);
    if (!rotary_counts(num_tokens, num_heads)) return fail(TQ_ERR_UNSUPPORTED, "more rows than a launch holds");
    RotaryArgs r{};
    r.r.table = table;
    r.r.positions = num_positions;
    r.r.rot = rot;
    r.r.interleaved = layout == TQ_ROTARY_INTERLEAVED;
    r.x = x;
    r.out = out;
    r.dtype = (int)dtype;
    r.x_token = x_token_stride;
    r.x_head = x_head_stride;
    r.out_token = out_token_stride;
    r.out_head = out_head_stride;
    r.tokens = num_tokens;
    r.heads = num_heads;
    r.d = d;
    r.positions = positions;
    r.transpose = transpose;
    r.status = dev_status;
    const int e = launch_rotary(r, stream);
    return e ? cuda_fail((cudaError_t)e, "rotary launch") : TQ_OK;
}

}  // extern "C"
