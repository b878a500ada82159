// Internal declarations of the rotary positions.
#pragma once

#include <cstdint>

#include "tq_internal.h"

namespace tq {

// Cosines and sines of every position: [positions][2][rot / 2] fp32.
struct RotaryTable {
    const float* table;
    int64_t positions;
    int rot;          // rotated dims of a head, its first ones: a multiple of 16
    int interleaved;  // pairs (2 j, 2 j + 1), else (j, j + rot / 2)
};

// x, out: [tokens][heads][d], strides in elements.
struct RotaryArgs {
    RotaryTable r;
    const void* x;
    void* out;
    int dtype;
    int64_t x_token, x_head, out_token, out_head;
    int64_t tokens;
    int heads, d;
    const int32_t* positions;  // [tokens]
    int transpose;
    int32_t* status;
};

constexpr int kRotaryMaxDim = 256;  // rotated dims: the frequencies travel as kernel arguments

bool rotary_counts(int64_t tokens, int heads);  // the grid fits 32 bits
int launch_rotary(const RotaryArgs& a, void* stream);
int launch_rotary_table(const double* frequencies, int rot, double magnitude, int64_t positions, float* table, void* stream);

// What is wrong with a table's arguments (and whether that is a limit: *unsupported), or NULL.
const char* rotary_table_fault(const float* table, int64_t positions, int rot, int layout, bool* unsupported);
// What is wrong with rows that are rotated from x to out (strides in elements): output rows that overlap one another or,
// without being the same rows, the input.  NULL: nothing.
const char* rotary_rows_fault(const void* x, int64_t x_token, int64_t x_head, const void* out, int64_t out_token, int64_t out_head,
                              int64_t tokens, int heads, int d, int elem);

}  // namespace tq
