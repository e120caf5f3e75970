// q8_i8.h -- host-side declarations of the 8-bit products with token and
// channel scales and of the log probabilities (launchers called by abi_i8.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q8 {

// Exact int32 sums: 2^14 (= 128 * 128) * k < 2^31.
constexpr int64_t kI8MaxK = 131040;
// Tile rows are addressed with 32-bit byte offsets: 256 rows of at most 4 MiB.
constexpr int64_t kI8MaxRowBytes = (int64_t)1 << 22;
constexpr int64_t kI8MaxRows = (int64_t)1 << 27;
constexpr int64_t kI8MaxOutputs = (int64_t)1 << 36;

// One product, already validated.  x: codes with x_scale per row.
struct I8Args {
    const int8_t *x;
    const float *x_scale;
    const int8_t *w;
    const float *w_scale;
    const float *bias;        // or null; not used by the gated form
    void *y;
    int64_t x_stride, w_stride;   // bytes
    int64_t y_stride;             // elements
    int64_t n, k, m;              // n: output columns (n_ff in the gated form)
    int y_type;                   // Q8_T_F32, Q8_T_F16, Q8_T_BF16
};

// Rows of k values of `type` to codes and scales.
int launch_i8_quantize(const void *x, int type, int64_t x_stride, int8_t *q, int64_t q_stride,
                       float *scale, int64_t n_rows, int64_t k, hipStream_t stream);

// Few token rows or few outputs (i8_stream_ok), weights streamed once for at
// most 64 rows.  With xf the token rows are taken as given (xf_type, Q8_T_I8
// included; bytes per row xf_stride) where i8_inline_ok, and a.x is not read.
bool i8_stream_ok(const I8Args &a, bool gated);
bool i8_inline_ok(const I8Args &a, bool gated);
int launch_i8_stream(const I8Args &a, const void *xf, int xf_type, int64_t xf_stride, bool gated,
                     hipStream_t stream);

// Many token rows, on tiles of both operands (i8_gemm_form: which, as Q8V_I8_*).
int i8_gemm_form(const I8Args &a, bool gated);
int launch_i8_gemm(const I8Args &a, bool gated, hipStream_t stream);

// Log probabilities, already validated.
struct LogprobArgs {
    const void *logits;
    const int32_t *tokens;
    float *logprob, *lse, *entropy;
    int32_t *top_ids;
    float *top_logprobs;
    int64_t row_stride;           // elements
    int64_t m, n_vocab;
    int n_given, n_top, type;
};

constexpr int kLogprobMaxTop = 64;
size_t logprob_ws_bytes(int64_t m, int64_t n_vocab, int64_t n_top);   // for up to m rows
size_t logprob_ws_needed(int64_t m, int64_t n_vocab, int64_t n_top);  // by a call of m
int launch_logprob(const LogprobArgs &a, void *ws, hipStream_t stream);

}  // namespace q8
