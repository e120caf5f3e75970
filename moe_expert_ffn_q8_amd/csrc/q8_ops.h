// q8_ops.h -- host-side declarations of the operators around the products of a
// token step: embedding rows, norm rows, sampling (launchers called by
// abi_ops.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q8 {

// Table formats of the embedding lookup beyond q8_type.
enum { kTableQ8_0 = 16, kTableR8 = 17 };

// Embedding rows, already validated.
struct EmbedArgs {
    const void *table;
    const float *table_scale;     // int8 tables
    const int32_t *tokens;
    void *y;
    int64_t row_bytes;            // of a table row (not R8)
    int64_t y_stride;             // elements
    int64_t m, n;
    int k;
    int table_type, y_type;       // q8_type or kTable*; Q8_T_F32, Q8_T_F16, Q8_T_BF16
    float scale;
};

int launch_embed(const EmbedArgs &a, hipStream_t stream);

// Norm rows, already validated: residual null: y = norm(x); else the residual
// stream's update and the next norm.  Strides in elements.
struct NormArgs {
    const void *x, *residual, *gate;
    void *residual_out, *y;
    const float *post_weight, *post_bias, *weight, *bias;
    float *y_scale;               // int8 y
    int64_t x_stride, r_stride, ro_stride, gate_stride, y_stride;
    int64_t m;
    int n;
    int x_type, r_type, gate_type, y_type;
    float residual_scale, eps;
    int layer, post;
};

int launch_norm(const NormArgs &a, hipStream_t stream);

// Sampling, already validated.
struct SampleArgs {
    const void *logits;
    const float *u, *temperature, *top_p, *min_p;   // the last three may be null
    const int32_t *top_k;                           // may be null
    int32_t *ids, *kept;
    float *logprob;
    int64_t row_stride;           // elements
    int64_t m, n_vocab;
    int type;
};

constexpr int64_t kSampleMaxVocab = (int64_t)1 << 24;
constexpr int64_t kSampleMaxRows = (int64_t)1 << 23;
size_t sample_ws_bytes(int64_t m, int64_t n_vocab);
int launch_sample(const SampleArgs &a, void *ws, hipStream_t stream);

}  // namespace q8
