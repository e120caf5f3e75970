// i8_gemm.hip -- the 8-bit products with token and channel scales: Y[m][n] from
// codes X[m][k] and W[n][k], and the gated form.
//
// Each output is an exact int32 sum over k, rescaled once.  A workgroup
// computes a 64 x 64 tile (in the gated form 64 tokens x 32 gate rows and the
// 32 up rows that belong to them), 4 x 4 outputs per thread, v_dot4 over
// 32-byte slices of k staged in LDS.
#include "i8_device.h"
#include "q8_i8.h"

namespace q8 {

namespace {

constexpr int kT = 64, kStep = 32, kPad = 36;

template <int YT, bool GATED>
__global__ __launch_bounds__(256) void i8_tile_kernel(const I8Args a, int tiles_n)
{
    __shared__ __align__(16) uint8_t sx[kT * kPad];
    __shared__ __align__(16) uint8_t sw[kT * kPad];
    constexpr int kCols = GATED ? kT / 2 : kT;
    const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * kT;
    const int64_t n0 = (int64_t)(blockIdx.x % tiles_n) * kCols;
    const int tid = threadIdx.x, tr = tid >> 4, tc = tid & 15;
    int acc[4][4] = {};
    // thread tid stages 8 bytes of row tid/4 of each operand
    const int r = tid >> 2, c = 8 * (tid & 3);
    const int64_t xr = min(m0 + r, a.m - 1);
    const int64_t wc = min(n0 + r % kCols, a.n - 1) + (GATED && r >= kCols ? a.n : 0);
    for (int64_t k0 = 0; k0 < a.k; k0 += kStep) {
        const u32x2 vx = *(const u32x2 *)(a.x + xr * a.x_stride + k0 + c);
        const u32x2 vw = *(const u32x2 *)(a.w + wc * a.w_stride + k0 + c);
        __syncthreads();
        ((uint32_t *)(sx + r * kPad + c))[0] = vx.x;
        ((uint32_t *)(sx + r * kPad + c))[1] = vx.y;
        ((uint32_t *)(sw + r * kPad + c))[0] = vw.x;
        ((uint32_t *)(sw + r * kPad + c))[1] = vw.y;
        __syncthreads();
#pragma unroll
        for (int d = 0; d < kStep / 4; ++d) {
            uint32_t x[4], w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = *(const uint32_t *)(sx + (tr + 16 * i) * kPad + 4 * d);
                w[i] = *(const uint32_t *)(sw + (tc + 16 * i) * kPad + 4 * d);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = sdot4(x[i], w[j], acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t t = m0 + tr + 16 * i;
        if (t >= a.m) continue;
        const float s = a.x_scale[t];
#pragma unroll
        for (int j = 0; j < (GATED ? 2 : 4); ++j) {
            const int64_t n = n0 + tc + 16 * j;
            if (n >= a.n) continue;
            float v;
            if (GATED)
                v = silu_mul(i8_rescale(acc[i][j], s, a.w_scale[n]),
                             i8_rescale(acc[i][j + 2], s, a.w_scale[a.n + n]));
            else
                v = a.bias ? i8_rescale(acc[i][j], s, a.w_scale[n], a.bias[n])
                           : i8_rescale(acc[i][j], s, a.w_scale[n]);
            store_out<YT>(a.y, t * a.y_stride + n, v);
        }
    }
}

template <int YT>
int launch_type(const I8Args &a, bool gated, hipStream_t stream)
{
    const int64_t cols = gated ? kT / 2 : kT;
    const int64_t tn = (a.n + cols - 1) / cols, tm = (a.m + kT - 1) / kT;
    if (tn * tm >= ((int64_t)1 << 24)) return Q8_E_UNSUPPORTED;
    const dim3 grid((unsigned)(tn * tm)), block(256);
    if (gated)
        hipLaunchKernelGGL((i8_tile_kernel<YT, true>), grid, block, 0, stream, a, (int)tn);
    else
        hipLaunchKernelGGL((i8_tile_kernel<YT, false>), grid, block, 0, stream, a, (int)tn);
    return hipGetLastError() == hipSuccess ? 0 : -6;
}

}  // namespace

int launch_i8_product(const I8Args &a, bool gated, hipStream_t stream)
{
    if (a.y_type == Q8_T_F32) return launch_type<Q8_T_F32>(a, gated, stream);
    if (a.y_type == Q8_T_F16) return launch_type<Q8_T_F16>(a, gated, stream);
    return launch_type<Q8_T_BF16>(a, gated, stream);
}

}  // namespace q8
