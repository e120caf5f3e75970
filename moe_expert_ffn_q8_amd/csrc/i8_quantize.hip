// i8_quantize.hip -- rows of fp32, binary16 or bfloat16 values to int8 codes
// with one fp32 scale per row (the rule: q8moe.h; the arithmetic: i8_device.h).
//
// One workgroup per row: the largest |x| over the row, then the codes.
#include "i8_device.h"
#include "q8_i8.h"

namespace q8 {

namespace {

constexpr int kThreads = 256;

template <int T>
__global__ __launch_bounds__(kThreads) void i8_quantize_kernel(const uint8_t *__restrict__ x,
                                                               int64_t x_bytes,
                                                               int8_t *__restrict__ q,
                                                               int64_t q_stride,
                                                               float *__restrict__ scale, int k)
{
    __shared__ uint32_t part[kThreads / 64];
    constexpr int V = kVec<T>;
    const int64_t row = blockIdx.x;
    const u32x4 *src = (const u32x4 *)(x + row * x_bytes);
    const int chunks = k / V;
    uint32_t a = 0;
    for (int i = threadIdx.x; i < chunks; i += kThreads) {
        float v[V];
        unpack16<T>(src[i], v);
#pragma unroll
        for (int j = 0; j < V; ++j) a = max(a, abs_bits(v[j]));
    }
    for (int d = 32; d; d >>= 1) a = max(a, (uint32_t)__shfl_xor((int)a, d));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = a;
    __syncthreads();
    for (int i = 0; i < kThreads / 64; ++i) a = max(a, part[i]);
    const float s = row_scale(a);
    if (threadIdx.x == 0) scale[row] = s;
    const RowCoder rc(s);
    for (int i = threadIdx.x; i < chunks; i += kThreads) {
        float v[V];
        unpack16<T>(src[i], v);
        uint32_t w[V / 4];
#pragma unroll
        for (int j = 0; j < V / 4; ++j)
            w[j] = rc.code4(v + 4 * j);
#pragma unroll
        for (int j = 0; j < V / 4; ++j) *(uint32_t *)(q + row * q_stride + (int64_t)i * V + 4 * j) = w[j];
    }
}

}  // namespace

int launch_i8_quantize(const void *x, int type, int64_t x_stride, int8_t *q, int64_t q_stride,
                       float *scale, int64_t n_rows, int64_t k, hipStream_t stream)
{
    const dim3 grid((unsigned)n_rows), block(kThreads);
    const uint8_t *p = (const uint8_t *)x;
    if (type == Q8_T_F32)
        hipLaunchKernelGGL(i8_quantize_kernel<Q8_T_F32>, grid, block, 0, stream, p, x_stride * 4, q,
                           q_stride, scale, (int)k);
    else if (type == Q8_T_F16)
        hipLaunchKernelGGL(i8_quantize_kernel<Q8_T_F16>, grid, block, 0, stream, p, x_stride * 2, q,
                           q_stride, scale, (int)k);
    else
        hipLaunchKernelGGL(i8_quantize_kernel<Q8_T_BF16>, grid, block, 0, stream, p, x_stride * 2, q,
                           q_stride, scale, (int)k);
    return hipGetLastError() == hipSuccess ? 0 : -6;
}

}  // namespace q8
