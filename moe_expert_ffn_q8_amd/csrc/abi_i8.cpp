// abi_i8.cpp -- the extern "C" entry points of the 8-bit products with token
// and channel scales and of the log probabilities (see include/q8moe.h).
//
// As in abi.cpp every argument is checked on the host before any HIP call, and
// nothing here allocates, frees or synchronizes.
#include "q8moe.h"

#include "q8_i8.h"

namespace {

inline bool aligned(const void *p, uintptr_t a) { return (((uintptr_t)p) % a) == 0; }

inline int hip_status(int rc) { return rc == 0 ? Q8_OK : (rc < 0 ? rc : Q8_E_HIP); }

inline bool float_type(int t) { return t == Q8_T_F32 || t == Q8_T_F16 || t == Q8_T_BF16; }

inline int64_t type_bytes(int t) { return t == Q8_T_F32 ? 4 : t == Q8_T_I8 ? 1 : 2; }

inline int64_t up16(int64_t v) { return (v + 15) / 16 * 16; }

int check_i8_k(int64_t k)
{
    if (k <= 0 || k % 32 != 0) return Q8_E_SHAPE;
    return k > q8::kI8MaxK ? Q8_E_UNSUPPORTED : Q8_OK;
}

// Rows of k elements of `bytes` bytes at a 16-byte aligned base: the stride
// (elements) of a single row is not read and is taken as k.
int check_rows(const void *p, int64_t &stride, int64_t rows, int64_t k, int64_t bytes)
{
    if (rows <= 1) stride = k;
    if (stride < k) return Q8_E_SHAPE;
    if (!aligned(p, 16) || stride * bytes % 16 != 0) return Q8_E_ALIGN;
    return stride > q8::kI8MaxRowBytes / bytes ? Q8_E_UNSUPPORTED : Q8_OK;
}

int i8_product(const void *x, int x_type, int64_t x_row_stride, const float *x_scale,
               const int8_t *w, int64_t w_row_stride, const float *w_scale, const float *bias,
               void *y, int y_type, int64_t y_row_stride, int64_t n, int64_t k, int64_t m,
               bool gated, void *ws, size_t ws_bytes, void *stream)
{
    if (int rc = check_i8_k(k)) return rc;
    if (n < 0 || m < 0) return Q8_E_SHAPE;
    if (!float_type(y_type) || (x_type != Q8_T_I8 && !float_type(x_type))) return Q8_E_UNSUPPORTED;
    if (n > q8::kI8MaxRows || m > q8::kI8MaxRows || (m > 0 && n > q8::kI8MaxOutputs / m))
        return Q8_E_UNSUPPORTED;
    if (n == 0 || m == 0) return Q8_OK;
    const bool codes = x_type == Q8_T_I8;
    if (!x || !w || !w_scale || !y || (codes && !x_scale)) return Q8_E_NULL;
    const int64_t w_rows = gated ? 2 * n : n;
    if (int rc = check_rows(x, x_row_stride, m, k, type_bytes(x_type))) return rc;
    if (int rc = check_rows(w, w_row_stride, w_rows, k, 1)) return rc;
    if (m == 1) y_row_stride = n;
    if (y_row_stride < n) return Q8_E_SHAPE;
    if (!aligned(y, type_bytes(y_type)) || !aligned(w_scale, 4) || (codes && !aligned(x_scale, 4)) ||
        (bias && !aligned(bias, 4)))
        return Q8_E_ALIGN;
    const hipStream_t st = (hipStream_t)stream;
    q8::I8Args a;
    a.w = w; a.w_scale = w_scale; a.bias = bias; a.y = y;
    a.w_stride = w_row_stride; a.y_stride = y_row_stride;
    a.n = n; a.k = k; a.m = m; a.y_type = y_type;
    if (!codes && (!ws || ws_bytes < i8_workspace_bytes(m, k))) return Q8_E_WORKSPACE;
    if (!codes && !aligned(ws, 256)) return Q8_E_ALIGN;
    a.x = (const int8_t *)x; a.x_scale = x_scale; a.x_stride = x_row_stride;
    if (q8::i8_inline_ok(a, gated))
        return hip_status(q8::launch_i8_stream(a, x, x_type, x_row_stride * type_bytes(x_type),
                                               gated, st));
    if (!codes) {
        // workspace: m rows of codes, then m scales
        int8_t *q = (int8_t *)ws;
        float *s = (float *)(q + m * up16(k));
        if (int rc = q8::launch_i8_quantize(x, x_type, x_row_stride, q, up16(k), s, m, k, st))
            return hip_status(rc);
        a.x = q; a.x_scale = s; a.x_stride = up16(k);
    }
    return hip_status(q8::i8_stream_ok(a, gated)
                          ? q8::launch_i8_stream(a, nullptr, Q8_T_I8, 0, gated, st)
                          : q8::launch_i8_gemm(a, gated, st));
}

}  // namespace

extern "C" {

int i8_quantize_rows(const void *x, int x_type, int64_t x_row_stride, int8_t *q,
                     int64_t q_row_stride, float *scale, int64_t n_rows, int64_t k, void *stream)
{
    if (int rc = check_i8_k(k)) return rc;
    if (n_rows < 0) return Q8_E_SHAPE;
    if (!float_type(x_type) || n_rows > q8::kI8MaxRows) return Q8_E_UNSUPPORTED;
    if (n_rows == 0) return Q8_OK;
    if (!x || !q || !scale) return Q8_E_NULL;
    if (int rc = check_rows(x, x_row_stride, n_rows, k, type_bytes(x_type))) return rc;
    if (int rc = check_rows(q, q_row_stride, n_rows, k, 1)) return rc;
    if (!aligned(scale, 4)) return Q8_E_ALIGN;
    return hip_status(q8::launch_i8_quantize(x, x_type, x_row_stride, q, q_row_stride, scale,
                                             n_rows, k, (hipStream_t)stream));
}

size_t i8_workspace_bytes(int64_t m, int64_t k)
{
    if (check_i8_k(k) || m < 0 || m > q8::kI8MaxRows) return 0;
    const size_t b = (size_t)(m > 0 ? m : 1) * (up16(k) + 4);
    return (b + 255) / 256 * 256;
}

int i8_matmul(const void *x, int x_type, int64_t x_row_stride, const float *x_scale,
              const int8_t *w, int64_t w_row_stride, const float *w_scale, const float *bias,
              void *y, int y_type, int64_t y_row_stride, int64_t n, int64_t k, int64_t m,
              void *ws, size_t ws_bytes, void *stream)
{
    return i8_product(x, x_type, x_row_stride, x_scale, w, w_row_stride, w_scale, bias, y, y_type,
                      y_row_stride, n, k, m, false, ws, ws_bytes, stream);
}

int i8_up_gate_swiglu(const void *x, int x_type, int64_t x_row_stride, const float *x_scale,
                      const int8_t *w, int64_t w_row_stride, const float *w_scale, void *h,
                      int h_type, int64_t h_row_stride, int64_t n_ff, int64_t k, int64_t m,
                      void *ws, size_t ws_bytes, void *stream)
{
    return i8_product(x, x_type, x_row_stride, x_scale, w, w_row_stride, w_scale, nullptr, h,
                      h_type, h_row_stride, n_ff, k, m, true, ws, ws_bytes, stream);
}

int q8v_i8_form(int64_t n, int64_t k, int64_t m, int gated)
{
    if (int rc = check_i8_k(k)) return rc;
    if (n <= 0 || m <= 0) return Q8_E_SHAPE;
    if (n > q8::kI8MaxRows || m > q8::kI8MaxRows || n > q8::kI8MaxOutputs / m)
        return Q8_E_UNSUPPORTED;
    q8::I8Args a = {};
    a.n = n; a.k = k; a.m = m;
    if (q8::i8_inline_ok(a, gated != 0)) return Q8V_I8_STREAM_INLINE;
    if (q8::i8_stream_ok(a, gated != 0)) return Q8V_I8_STREAM;
    return q8::i8_gemm_form(a, gated != 0);
}

static int check_logprob_sizes(int64_t m, int64_t n_vocab, int64_t n_top)
{
    if (m < 0 || n_vocab <= 0 || n_top < 0 || n_top > n_vocab) return Q8_E_SHAPE;
    if (n_top > q8::kLogprobMaxTop || n_vocab > ((int64_t)1 << 30) || m > ((int64_t)1 << 24))
        return Q8_E_UNSUPPORTED;
    return Q8_OK;
}

static constexpr size_t kWsLeast = 256;

size_t logprob_workspace_bytes(int64_t m, int64_t n_vocab, int64_t n_top)
{
    if (check_logprob_sizes(m, n_vocab, n_top)) return 0;
    const size_t b = q8::logprob_ws_bytes(m, n_vocab, n_top);
    return b < kWsLeast ? kWsLeast : (b + 255) / 256 * 256;
}

int logprob_rows(const void *logits, int type, int64_t row_stride, const int32_t *tokens,
                 int64_t n_given, float *logprob, float *lse, float *entropy, int32_t *top_ids,
                 float *top_logprobs, int64_t m, int64_t n_vocab, int64_t n_top, void *ws,
                 size_t ws_bytes, void *stream)
{
    if (int rc = check_logprob_sizes(m, n_vocab, n_top)) return rc;
    if (n_given < 0) return Q8_E_SHAPE;
    if (n_given > 1024 || !float_type(type)) return Q8_E_UNSUPPORTED;
    if (m == 0) return Q8_OK;
    if (!logits || (n_given > 0 && (!tokens || !logprob)) ||
        (n_top > 0 && (!top_ids || !top_logprobs)))
        return Q8_E_NULL;
    if (m == 1) row_stride = n_vocab;
    if (row_stride < n_vocab) return Q8_E_SHAPE;
    if (!aligned(logits, type_bytes(type)) || (n_given > 0 && (!aligned(tokens, 4) || !aligned(logprob, 4))) ||
        (n_top > 0 && (!aligned(top_ids, 4) || !aligned(top_logprobs, 4))) ||
        (lse && !aligned(lse, 4)) || (entropy && !aligned(entropy, 4)))
        return Q8_E_ALIGN;
    if (!ws || ws_bytes < kWsLeast || ws_bytes < q8::logprob_ws_needed(m, n_vocab, n_top))
        return Q8_E_WORKSPACE;
    if (!aligned(ws, 256)) return Q8_E_ALIGN;
    q8::LogprobArgs a;
    a.logits = logits; a.tokens = tokens; a.logprob = logprob; a.lse = lse; a.entropy = entropy;
    a.top_ids = top_ids; a.top_logprobs = top_logprobs; a.row_stride = row_stride;
    a.m = m; a.n_vocab = n_vocab; a.n_given = (int)n_given; a.n_top = (int)n_top; a.type = type;
    return hip_status(q8::launch_logprob(a, ws, (hipStream_t)stream));
}

}  // extern "C"
