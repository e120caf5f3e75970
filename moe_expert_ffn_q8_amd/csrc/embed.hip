// embed.hip -- rows of an embedding table by token, scaled: fp32, binary16,
// bfloat16, int8 codes with a scale per row, Q8_0 rows and the R8 layout of
// them.
//
// A gather: HBM bounds it for many tokens (16384 x 4096 int8 to bfloat16: 43.7 us,
// 4.3 TB/s of what it must move, 38 at the rate of a copy), the launch and two
// round trips (token, row) for few (1.8 us).  Work goes by the 16 bytes of an output: a lane reads
// what these need, 4 or 8 values, and stores them at once.  A value is formed
// in fp32: code * scale of its block or row, then the lookup's scale, each
// product rounded, then once to the output's type.
#include "i8_device.h"
#include "q8_ops.h"

namespace q8 {

namespace {

typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef u32x2 __attribute__((aligned(2))) u32x2_any;
typedef uint32_t __attribute__((aligned(2))) u32_any;

// int8 codes of a dword as fp32.
__device__ __forceinline__ void codes4(uint32_t c, float *v)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = (float)(int8_t)(c >> (8 * j));
}

// V consecutive values of float type T from element alignment.
template <int T, int V>
__device__ __forceinline__ void load_floats(const uint8_t *p, float (&v)[V])
{
    constexpr int kBytes = V * (T == Q8_T_F32 ? 4 : 2);
    if constexpr (kBytes == 8) {
        const u32x2 r = *(const u32x2_any *)p;
        float w[8];
        unpack16<T>((u32x4){r.x, r.y, 0u, 0u}, w);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = w[j];
    } else {
        constexpr int N = kVec<T>;
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) {
            float w[N];
            unpack16<T>(*(const u32x4_any *)(p + 16 * i), w);
#pragma unroll
            for (int j = 0; j < N; ++j) v[i * N + j] = w[j];
        }
    }
}

// Values e .. e + V - 1 of row `tok` (all inside the row).
template <int TT, int V>
__device__ __forceinline__ void table_values(const EmbedArgs &a, int64_t tok, int e, float (&v)[V])
{
    const uint8_t *t = (const uint8_t *)a.table;
    if constexpr (TT == kTableQ8_0 || TT == kTableR8 || TT == Q8_T_I8) {
        const uint8_t *codes;
        float s;
        if constexpr (TT == Q8_T_I8) {
            codes = t + tok * a.row_bytes + e;
            s = a.table_scale[tok];
        } else if constexpr (TT == kTableQ8_0) {
            const uint8_t *b = t + tok * a.row_bytes + e / 32 * kBlockBytes;
            s = half_bits_to_float(load_u16(b));
            codes = b + 2 + e % 32;
        } else {
            const int nb = a.k / 32;
            const uint8_t *g = t + (tok >> 3) * (272 * (int64_t)nb);
            const int at = 8 * (e / 32) + (int)(tok & 7);
            s = half_bits_to_float(load_u16(g + 2 * at));
            codes = g + 16 * nb + 32 * (int64_t)at + e % 32;
        }
        if constexpr (V == 8) {
            const u32x2 c = *(const u32x2_any *)codes;
            codes4(c.x, v);
            codes4(c.y, v + 4);
        } else
            codes4(*(const u32_any *)codes, v);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] *= s;
    } else
        load_floats<TT, V>(t + tok * a.row_bytes + (int64_t)e * (TT == Q8_T_F32 ? 4 : 2), v);
}

// 256 threads: `lanes` (a power of two) per row, 256 / lanes rows.
template <int TT, int YT>
__global__ __launch_bounds__(256) void embed_kernel(const EmbedArgs a, int lanes_log2, int64_t row0)
{
    constexpr int V = kVec<YT>, kES = YT == Q8_T_F32 ? 4 : 2;
    const int lanes = 1 << lanes_log2;
    const int64_t row = row0 + (int64_t)blockIdx.x * (256 >> lanes_log2) + (threadIdx.x >> lanes_log2);
    if (row >= a.m) return;
    const int64_t tok = a.tokens[row];
    const bool real = tok >= 0 && tok < a.n;
    uint8_t *y = (uint8_t *)a.y + row * a.y_stride * kES;
#pragma unroll 4
    for (int e = (threadIdx.x & (lanes - 1)) * V; e < a.k; e += lanes * V) {
        float v[V];
        const int left = a.k - e;
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = __builtin_nanf("");
        if (real) {
            if (left >= V)
                table_values<TT, V>(a, tok, e, v);
            else if constexpr (TT == Q8_T_F32 || TT == Q8_T_F16 || TT == Q8_T_BF16) {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (j < left)
                        v[j] = (float)((const typename Elem<TT>::type *)((const uint8_t *)a.table +
                                                                         tok * a.row_bytes))[e + j];
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] *= a.scale;
        store16<YT, false>(y + (int64_t)e * kES, pack_vec<YT>(v), left);
    }
}

template <int TT, int YT>
int launch(const EmbedArgs &a, hipStream_t stream)
{
    int lg = 8;
    while (lg > 3 && (kVec<YT> << (lg - 1)) >= a.k) --lg;
    const int64_t per = 256 >> lg;
    // (2^32 threads bound a launch)
    const int64_t most = per << 23;
    for (int64_t r = 0; r < a.m; r += most) {
        const int64_t rows = a.m - r < most ? a.m - r : most;
        hipLaunchKernelGGL((embed_kernel<TT, YT>), dim3((unsigned)((rows + per - 1) / per)), dim3(256), 0,
                           stream, a, lg, r);
        if (hipGetLastError() != hipSuccess) return -6;
    }
    return 0;
}

template <int TT>
int launch_table(const EmbedArgs &a, hipStream_t stream)
{
    return a.y_type == Q8_T_F32   ? launch<TT, Q8_T_F32>(a, stream)
           : a.y_type == Q8_T_F16 ? launch<TT, Q8_T_F16>(a, stream)
                                  : launch<TT, Q8_T_BF16>(a, stream);
}

}  // namespace

int launch_embed(const EmbedArgs &a, hipStream_t stream)
{
    switch (a.table_type) {
    case Q8_T_F32: return launch_table<Q8_T_F32>(a, stream);
    case Q8_T_F16: return launch_table<Q8_T_F16>(a, stream);
    case Q8_T_BF16: return launch_table<Q8_T_BF16>(a, stream);
    case Q8_T_I8: return launch_table<Q8_T_I8>(a, stream);
    case kTableQ8_0: return launch_table<kTableQ8_0>(a, stream);
    default: return launch_table<kTableR8>(a, stream);
    }
}

}  // namespace q8
