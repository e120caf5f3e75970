// abi_ops.cpp -- the extern "C" entry points of the operators around the
// products of a token step: embedding rows, norm rows, sampling (see
// include/q8moe.h).
//
// As in abi.cpp every argument is checked on the host before any HIP call, and
// nothing here allocates, frees or synchronizes.
#include "q8moe.h"

#include <math.h>

#include "q8_ops.h"

namespace {

inline bool aligned(const void *p, uintptr_t a) { return (((uintptr_t)p) % a) == 0; }

inline int hip_status(int rc) { return rc == 0 ? Q8_OK : (rc < 0 ? rc : Q8_E_HIP); }

inline bool float_type(int t) { return t == Q8_T_F32 || t == Q8_T_F16 || t == Q8_T_BF16; }

inline int64_t type_bytes(int t) { return t == Q8_T_F32 ? 4 : t == Q8_T_I8 ? 1 : 2; }

constexpr int64_t kMaxRows = (int64_t)1 << 27;
constexpr int64_t kMaxStride = (int64_t)1 << 32;      // elements: byte offsets of rows fit 64 bits
constexpr int64_t kMaxEmbedK = (int64_t)1 << 20;
constexpr int64_t kMaxNormN = 65536;

// The stride of rows of n elements at an element-aligned base (that of a single
// row is not read and taken as n).
int check_stride(const void *p, int64_t &stride, int64_t rows, int64_t n, int type)
{
    if (rows <= 1) stride = n;
    if (stride < n) return Q8_E_SHAPE;
    if (!aligned(p, type_bytes(type))) return Q8_E_ALIGN;
    return stride > kMaxStride ? Q8_E_UNSUPPORTED : Q8_OK;
}

int embed_sizes(int64_t m, int64_t n, int64_t k, int y_type, bool blocks)
{
    if (m < 0 || n <= 0 || k <= 0 || (blocks && k % 32 != 0)) return Q8_E_SHAPE;
    if (!float_type(y_type) || m > kMaxRows || n > (((int64_t)1 << 31) - 1) || k > kMaxEmbedK)
        return Q8_E_UNSUPPORTED;
    return Q8_OK;
}

int embed(q8::EmbedArgs &a, const void *table, const int32_t *tokens, float scale, void *y, int y_type,
          int64_t y_row_stride, int64_t m, int64_t n, int64_t k, void *stream)
{
    if (!aligned(tokens, 4)) return Q8_E_ALIGN;
    if (int rc = check_stride(y, y_row_stride, m, k, y_type)) return rc;
    a.table = table; a.tokens = tokens; a.scale = scale; a.y = y; a.y_type = y_type;
    a.y_stride = y_row_stride; a.m = m; a.n = n; a.k = (int)k;
    return hip_status(q8::launch_embed(a, (hipStream_t)stream));
}

// The rows of x, and of y as floats or codes; y_scale goes with codes.
int check_norm(q8::NormArgs &a, int64_t m, int64_t n)
{
    if (m < 0 || n <= 0 || (a.y_type == Q8_T_I8 && n % 32 != 0)) return Q8_E_SHAPE;
    if (!float_type(a.x_type) || (a.y_type != Q8_T_I8 && !float_type(a.y_type)) || n > kMaxNormN ||
        m > kMaxRows || !(a.eps >= 0.0f) || isinf(a.eps))
        return Q8_E_UNSUPPORTED;
    return Q8_OK;
}

int check_norm_pointers(q8::NormArgs &a, int64_t m, int64_t n)
{
    const bool codes = a.y_type == Q8_T_I8;
    if (!a.x || !a.weight || !a.y || (codes && !a.y_scale)) return Q8_E_NULL;
    if (int rc = check_stride(a.x, a.x_stride, m, n, a.x_type)) return rc;
    if (int rc = check_stride(a.y, a.y_stride, m, n, a.y_type)) return rc;
    if (codes && (!aligned(a.y, 16) || a.y_stride % 16 != 0 || !aligned(a.y_scale, 4))) return Q8_E_ALIGN;
    if (!aligned(a.weight, 4) || !aligned(a.bias, 4)) return Q8_E_ALIGN;
    a.m = m;
    a.n = (int)n;
    return Q8_OK;
}

int check_sample_sizes(int64_t m, int64_t n_vocab)
{
    if (m < 0 || n_vocab <= 0) return Q8_E_SHAPE;
    return n_vocab > q8::kSampleMaxVocab || m > q8::kSampleMaxRows ? Q8_E_UNSUPPORTED : Q8_OK;
}

}  // namespace

extern "C" {

int embed_rows(const void *table, int table_type, int64_t table_row_stride, const float *table_scale,
               const int32_t *tokens, float scale, void *y, int y_type, int64_t y_row_stride, int64_t m,
               int64_t n, int64_t k, void *stream)
{
    const bool codes = table_type == Q8_T_I8;
    if (!codes && !float_type(table_type)) return Q8_E_UNSUPPORTED;
    if (int rc = embed_sizes(m, n, k, y_type, codes)) return rc;
    if (m == 0) return Q8_OK;
    if (!table || !tokens || !y || (codes && !table_scale)) return Q8_E_NULL;
    if (int rc = check_stride(table, table_row_stride, n, k, table_type)) return rc;
    if (codes && (!aligned(table, 16) || table_row_stride % 16 != 0 || !aligned(table_scale, 4)))
        return Q8_E_ALIGN;
    q8::EmbedArgs a = {};
    a.table_type = table_type; a.table_scale = table_scale;
    a.row_bytes = table_row_stride * type_bytes(table_type);
    return embed(a, table, tokens, scale, y, y_type, y_row_stride, m, n, k, stream);
}

int q8_0_embed_rows(const void *w, int r8, const int32_t *tokens, float scale, void *y, int y_type,
                    int64_t y_row_stride, int64_t m, int64_t n, int64_t k, void *stream)
{
    if (int rc = embed_sizes(m, n, k, y_type, true)) return rc;
    if (m == 0) return Q8_OK;
    if (!w || !tokens || !y) return Q8_E_NULL;
    if (!aligned(w, 16)) return Q8_E_ALIGN;
    q8::EmbedArgs a = {};
    a.table_type = r8 ? q8::kTableR8 : q8::kTableQ8_0;
    a.row_bytes = k / 32 * (int64_t)sizeof(q8_0_block);
    return embed(a, w, tokens, scale, y, y_type, y_row_stride, m, n, k, stream);
}

int norm_rows(const void *x, int x_type, int64_t x_row_stride, const float *weight, const float *bias,
              float eps, int layer, void *y, int y_type, int64_t y_row_stride, float *y_scale, int64_t m,
              int64_t n, void *stream)
{
    q8::NormArgs a = {};
    a.x = x; a.x_type = x_type; a.x_stride = x_row_stride; a.weight = weight; a.bias = bias;
    a.eps = eps; a.layer = layer != 0;
    a.y = y; a.y_type = y_type; a.y_stride = y_row_stride; a.y_scale = y_scale;
    if (int rc = check_norm(a, m, n)) return rc;
    if (m == 0) return Q8_OK;
    if (int rc = check_norm_pointers(a, m, n)) return rc;
    return hip_status(q8::launch_norm(a, (hipStream_t)stream));
}

int residual_norm_rows(const residual_norm_desc *d, int64_t m, int64_t n, void *stream)
{
    if (!d) return Q8_E_NULL;
    q8::NormArgs a = {};
    a.x = d->x; a.x_type = d->x_type; a.x_stride = d->x_row_stride;
    a.weight = d->weight; a.bias = d->bias; a.eps = d->eps; a.layer = d->layer != 0;
    a.y = d->y; a.y_type = d->y_type; a.y_stride = d->y_row_stride; a.y_scale = d->y_scale;
    if (int rc = check_norm(a, m, n)) return rc;
    if (!float_type(d->residual_type) || (d->gate && !float_type(d->gate_type))) return Q8_E_UNSUPPORTED;
    if (m == 0) return Q8_OK;
    if (!d->residual || !d->residual_out || (d->post_bias && !d->post_weight)) return Q8_E_NULL;
    if (int rc = check_norm_pointers(a, m, n)) return rc;
    a.residual = d->residual; a.r_type = d->residual_type; a.r_stride = d->residual_row_stride;
    a.residual_out = d->residual_out; a.ro_stride = d->residual_out_row_stride;
    if (int rc = check_stride(a.residual, a.r_stride, m, n, a.r_type)) return rc;
    if (int rc = check_stride(a.residual_out, a.ro_stride, m, n, a.r_type)) return rc;
    if (d->gate) {
        a.gate = d->gate; a.gate_type = d->gate_type; a.gate_stride = d->gate_row_stride;
        if (!aligned(a.gate, type_bytes(a.gate_type))) return Q8_E_ALIGN;
        if (a.gate_stride != 0)                    // 0: one row of gates for all
            if (int rc = check_stride(a.gate, a.gate_stride, m, n, a.gate_type)) return rc;
    }
    if (!aligned(d->post_weight, 4) || !aligned(d->post_bias, 4)) return Q8_E_ALIGN;
    a.post_weight = d->post_weight; a.post_bias = d->post_bias; a.post = d->post_weight != nullptr;
    a.residual_scale = d->residual_scale;
    return hip_status(q8::launch_norm(a, (hipStream_t)stream));
}

size_t sample_workspace_bytes(int64_t m, int64_t n_vocab)
{
    if (check_sample_sizes(m, n_vocab)) return 0;
    return (q8::sample_ws_bytes(m, n_vocab) + 255) / 256 * 256;
}

int sample_rows(const void *logits, int type, int64_t row_stride, const float *u, const float *temperature,
                const int32_t *top_k, const float *top_p, const float *min_p, int32_t *ids, float *logprob,
                int32_t *kept, int64_t m, int64_t n_vocab, void *ws, size_t ws_bytes, void *stream)
{
    if (int rc = check_sample_sizes(m, n_vocab)) return rc;
    if (!float_type(type)) return Q8_E_UNSUPPORTED;
    if (m == 0) return Q8_OK;
    if (!logits || !u || !ids || !logprob || !kept) return Q8_E_NULL;
    if (int rc = check_stride(logits, row_stride, m, n_vocab, type)) return rc;
    const void *vectors[] = {u, temperature, top_k, top_p, min_p, ids, logprob, kept};
    for (const void *p : vectors)
        if (!aligned(p, 4)) return Q8_E_ALIGN;
    if (!ws || ws_bytes < sample_workspace_bytes(m, n_vocab)) return Q8_E_WORKSPACE;
    if (!aligned(ws, 256)) return Q8_E_ALIGN;
    q8::SampleArgs a;
    a.logits = logits; a.type = type; a.row_stride = row_stride; a.u = u; a.temperature = temperature;
    a.top_k = top_k; a.top_p = top_p; a.min_p = min_p; a.ids = ids; a.logprob = logprob; a.kept = kept;
    a.m = m; a.n_vocab = n_vocab;
    return hip_status(q8::launch_sample(a, ws, (hipStream_t)stream));
}

}  // extern "C"
