// i8_quantize.hip -- rows of fp32, binary16 or bfloat16 values to int8 codes
// with one fp32 scale per row (the rule: q8moe.h; the arithmetic: i8_device.h).
//
// HBM bounds it for many rows, the launch and two memory round trips for few.
// A row of up to 16 KB is held in registers between finding its largest |x| and
// coding it, so it is read once; the tail of a longer one is read again, from
// L2.  Many rows of up to 4 KB go to a wave each (four per workgroup, no
// barrier).  14336 x 4096 fp32: 51 us, 5.75 TB/s; 512 x 4096 bfloat16: 3.7 us.
#include "i8_device.h"
#include "q8_i8.h"

namespace q8 {

namespace {

constexpr int kHold = 4;      // 16-byte pieces per thread held in registers

// ROW: threads per row, 64 or 256.
template <int T, int ROW>
__global__ __launch_bounds__(256) void i8_quantize_kernel(const uint8_t *__restrict__ x,
                                                          int64_t x_bytes, int8_t *__restrict__ q,
                                                          int64_t q_stride,
                                                          float *__restrict__ scale, int64_t rows,
                                                          int k)
{
    __shared__ uint32_t part[4];
    constexpr int V = kVec<T>;
    const int t = threadIdx.x % ROW;
    const int64_t row = (int64_t)blockIdx.x * (256 / ROW) + threadIdx.x / ROW;
    if (ROW == 64 && row >= rows) return;
    const u32x4 *src = (const u32x4 *)(x + row * x_bytes);
    const int pieces = k / V;
    u32x4 held[kHold];
#pragma unroll
    for (int u = 0; u < kHold; ++u) {
        held[u] = (u32x4){0u, 0u, 0u, 0u};
        if (t + ROW * u < pieces) held[u] = __builtin_nontemporal_load(src + t + ROW * u);
    }
    uint32_t a = 0;
    auto largest = [&](u32x4 r) {
        float v[V];
        unpack16<T>(r, v);
#pragma unroll
        for (int j = 0; j < V; ++j) a = max(a, abs_bits(v[j]));
    };
#pragma unroll
    for (int u = 0; u < kHold; ++u) largest(held[u]);
    for (int i = t + ROW * kHold; i < pieces; i += ROW) largest(src[i]);
#pragma unroll
    for (int d = 32; d; d >>= 1) a = max(a, (uint32_t)__shfl_xor((int)a, d));
    if (ROW > 64) {
        if ((t & 63) == 0) part[t >> 6] = a;
        __syncthreads();
        a = max(max(part[0], part[1]), max(part[2], part[3]));
    }
    const float s = row_scale(a);
    if (t == 0) scale[row] = s;
    const RowCoder rc(s);
    auto code = [&](u32x4 r, int i) {
        float v[V];
        unpack16<T>(r, v);
        int8_t *to = q + row * q_stride + (int64_t)i * V;
        if constexpr (V == 4)
            *(uint32_t *)to = rc.code4(v);
        else
            *(u32x2 *)to = (u32x2){rc.code4(v), rc.code4(v + 4)};
    };
#pragma unroll
    for (int u = 0; u < kHold; ++u)
        if (t + ROW * u < pieces) code(held[u], t + ROW * u);
    for (int i = t + ROW * kHold; i < pieces; i += ROW) code(src[i], i);
}

template <int T>
int launch_type(const uint8_t *x, int64_t x_bytes, int8_t *q, int64_t q_stride, float *scale,
                int64_t rows, int64_t k, hipStream_t stream)
{
    // (48 x 2048 binary16: 3.6 us by waves, 3.0 by workgroups; 2048 x 256: 2.7 and 3.1)
    if (k / kVec<T> <= 64 * kHold && rows >= 1024)
        hipLaunchKernelGGL((i8_quantize_kernel<T, 64>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0,
                           stream, x, x_bytes, q, q_stride, scale, rows, (int)k);
    else
        hipLaunchKernelGGL((i8_quantize_kernel<T, 256>), dim3((unsigned)rows), dim3(256), 0, stream, x,
                           x_bytes, q, q_stride, scale, rows, (int)k);
    return hipGetLastError() == hipSuccess ? 0 : -6;
}

}  // namespace

int launch_i8_quantize(const void *x, int type, int64_t x_stride, int8_t *q, int64_t q_stride,
                       float *scale, int64_t n_rows, int64_t k, hipStream_t stream)
{
    const uint8_t *p = (const uint8_t *)x;
    // (2^32 threads bound a launch)
    for (int64_t r = 0; r < n_rows; r += 1 << 23) {
        const int64_t n = n_rows - r < (1 << 23) ? n_rows - r : 1 << 23;
        const int64_t es = type == Q8_T_F32 ? 4 : 2;
        const uint8_t *px = p + r * x_stride * es;
        int8_t *pq = q + r * q_stride;
        const int rc = type == Q8_T_F32
                           ? launch_type<Q8_T_F32>(px, x_stride * 4, pq, q_stride, scale + r, n, k, stream)
                       : type == Q8_T_F16
                           ? launch_type<Q8_T_F16>(px, x_stride * 2, pq, q_stride, scale + r, n, k, stream)
                           : launch_type<Q8_T_BF16>(px, x_stride * 2, pq, q_stride, scale + r, n, k, stream);
        if (rc) return rc;
    }
    return 0;
}

}  // namespace q8
