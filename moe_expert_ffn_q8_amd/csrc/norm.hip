// norm.hip -- norms of rows: of a tensor, or of a residual stream that takes a
// block's output first, to floats or to int8 codes with a scale per row.
//
//   a  = x, or its norm with post_weight (and post_bias)
//   r' = round(gate * a + residual_scale * r)      stored, and what comes next reads it
//   y  = round(norm(r') * weight + bias), or codes of the fp32 y by the row rule
//   norm(v) = (v - mean) / sqrt(var + eps), or v / sqrt(mean of v^2 + eps)
//
// Everything between the roundings is in 64 bits: fp64 multiply-adds issue at
// the rate of fp32 ones here and HBM bounds the kernel, and a code of the row
// rule, which turns at a border, then does not hang on the order of a sum.
//
// A row lies in the registers of one wave or workgroup, 8 values a piece, so
// every tensor is read and written once.
#include "i8_device.h"
#include "q8_ops.h"

namespace q8 {

namespace {

typedef u32x4 __attribute__((aligned(2))) u32x4_any;

constexpr int kPiece = 8;

// Values i .. i + 7 of a row of `type` (the first `left` of them; 0 beyond).
__device__ __forceinline__ void load8(const void *row, int type, int64_t i, int left,
                                      float (&v)[kPiece])
{
    if (left >= kPiece) {
        if (type == Q8_T_F32) {
            const u32x4_any *p = (const u32x4_any *)((const float *)row + i);
            float a[4], b[4];
            unpack16<Q8_T_F32>(p[0], a);
            unpack16<Q8_T_F32>(p[1], b);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = a[j];
                v[4 + j] = b[j];
            }
        } else {
            const u32x4 r = *(const u32x4_any *)((const uint16_t *)row + i);
            if (type == Q8_T_F16)
                unpack16<Q8_T_F16>(r, v);
            else
                unpack16<Q8_T_BF16>(r, v);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < kPiece; ++j) {
        v[j] = 0.0f;
        if (j < left)
            v[j] = type == Q8_T_F32   ? ((const float *)row)[i + j]
                   : type == Q8_T_F16 ? (float)((const _Float16 *)row)[i + j]
                                      : (float)((const __bf16 *)row)[i + j];
    }
}

__device__ __forceinline__ void store8(void *row, int type, int64_t i, int left,
                                       const float (&v)[kPiece])
{
    if (type == Q8_T_F32) {
        uint8_t *p = (uint8_t *)((float *)row + i);
        const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
        store16<Q8_T_F32, false>(p, pack_vec<Q8_T_F32>(lo), left);
        if (left > 4) store16<Q8_T_F32, false>(p + 16, pack_vec<Q8_T_F32>(hi), left - 4);
    } else if (type == Q8_T_F16)
        store16<Q8_T_F16, false>((uint8_t *)((uint16_t *)row + i), pack_vec<Q8_T_F16>(v), left);
    else
        store16<Q8_T_BF16, false>((uint8_t *)((uint16_t *)row + i), pack_vec<Q8_T_BF16>(v), left);
}

// fp32 values as the type holds them.
__device__ __forceinline__ float as_stored(float v, int type)
{
    if (type == Q8_T_F32) return v;
    return type == Q8_T_F16 ? (float)round_out<Q8_T_F16>(v) : (float)round_out<Q8_T_BF16>(v);
}

// The sum over a row's threads, the same bits in all of them (the order is
// fixed).  `part` is free again after the next one.
template <int ROW>
__device__ __forceinline__ double row_sum(double s, double *part)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
    if constexpr (ROW > 64) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
        __syncthreads();
        s = 0.0;
#pragma unroll
        for (int w = 0; w < ROW / 64; ++w) s += part[w];
    }
    return s;
}

// ROW threads per row, P pieces of 8 values each.
template <int ROW, int P>
__global__ __launch_bounds__(ROW == 1024 ? 1024 : 256) void norm_kernel(const NormArgs a, int64_t row0)
{
    __shared__ double part[4][ROW / 64];
    __shared__ uint32_t part_max[ROW / 64];
    const int t = threadIdx.x % ROW;
    const int64_t row = row0 + (ROW == 64 ? (int64_t)blockIdx.x * 4 + threadIdx.x / 64 : blockIdx.x);
    if (ROW == 64 && row >= a.m) return;
    const int n = a.n;
    auto bytes = [](int type) { return type == Q8_T_F32 ? 4 : type == Q8_T_I8 ? 1 : 2; };
    const uint8_t *x = (const uint8_t *)a.x + row * a.x_stride * bytes(a.x_type);

    float v[P][kPiece];
#pragma unroll
    for (int p = 0; p < P; ++p) load8(x, a.x_type, (t + ROW * p) * kPiece, n - (t + ROW * p) * kPiece, v[p]);

    // mean and 1 / sqrt(mean square + eps) of the row held
    double mean = 0.0, rstd;
    auto stats = [&](double *p0, double *p1) {
        if (a.layer) {
            double s = 0.0;
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int j = 0; j < kPiece; ++j) s += (double)v[p][j];
            mean = row_sum<ROW>(s, p0) / n;
        }
        double s = 0.0;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int left = n - (t + ROW * p) * kPiece;
#pragma unroll
            for (int j = 0; j < kPiece; ++j) {
                const double d = (double)v[p][j] - mean;
                if (!a.layer || j < left) s = fma(d, d, s);
            }
        }
        rstd = 1.0 / sqrt(row_sum<ROW>(s, p1) / n + (double)a.eps);
    };

    if (a.residual) {
        if (a.post) stats(part[0], part[1]);
        const uint8_t *r = (const uint8_t *)a.residual + row * a.r_stride * bytes(a.r_type);
        const uint8_t *g = (const uint8_t *)a.gate + row * a.gate_stride * bytes(a.gate_type);
        uint8_t *ro = (uint8_t *)a.residual_out + row * a.ro_stride * bytes(a.r_type);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int i = (t + ROW * p) * kPiece, left = n - i;
            if (left <= 0) continue;
            float rv[kPiece], gv[kPiece], wv[kPiece], bv[kPiece];
            load8(r, a.r_type, i, left, rv);
            if (a.gate) load8(g, a.gate_type, i, left, gv);
            if (a.post) load8(a.post_weight, Q8_T_F32, i, left, wv);
            if (a.post_bias) load8(a.post_bias, Q8_T_F32, i, left, bv);
#pragma unroll
            for (int j = 0; j < kPiece; ++j) {
                double y = v[p][j];
                if (a.post) {
                    y = (y - mean) * rstd * (double)wv[j];
                    if (a.post_bias) y += (double)bv[j];
                }
                if (a.gate) y *= (double)gv[j];
                v[p][j] = as_stored((float)fma((double)a.residual_scale, (double)rv[j], y), a.r_type);
                if (j >= left) v[p][j] = 0.0f;
            }
            store8(ro, a.r_type, i, left, v[p]);
        }
    }

    stats(part[2], part[3]);
    const bool codes = a.y_type == Q8_T_I8;
    uint8_t *y = (uint8_t *)a.y + row * a.y_stride * bytes(a.y_type);
    uint32_t amax = 0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int i = (t + ROW * p) * kPiece, left = n - i;
        if (left <= 0) continue;
        float wv[kPiece], bv[kPiece];
        load8(a.weight, Q8_T_F32, i, left, wv);
        if (a.bias) load8(a.bias, Q8_T_F32, i, left, bv);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) {
            double o = ((double)v[p][j] - mean) * rstd * (double)wv[j];
            if (a.bias) o += (double)bv[j];
            v[p][j] = (float)o;
            if (j < left) amax = max(amax, abs_bits(v[p][j]));
        }
        if (!codes) store8(y, a.y_type, i, left, v[p]);
    }
    if (!codes) return;
#pragma unroll
    for (int d = 32; d; d >>= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, d));
    if constexpr (ROW > 64) {
        if ((threadIdx.x & 63) == 0) part_max[threadIdx.x >> 6] = amax;
        __syncthreads();
        amax = 0;
#pragma unroll
        for (int w = 0; w < ROW / 64; ++w) amax = max(amax, part_max[w]);
    }
    const float s = row_scale(amax);
    if (t == 0) a.y_scale[row] = s;
    const RowCoder rc(s);
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int i = (t + ROW * p) * kPiece;       // (n is a multiple of 32)
        if (i < n) *(u32x2 *)(y + i) = (u32x2){rc.code4(v[p]), rc.code4(v[p] + 4)};
    }
}

template <int ROW, int P>
int launch(const NormArgs &a, hipStream_t stream)
{
    constexpr int64_t per = ROW == 64 ? 4 : 1, most = per << (ROW == 1024 ? 21 : 23);
    // (2^32 threads bound a launch)
    for (int64_t r = 0; r < a.m; r += most) {
        const int64_t rows = a.m - r < most ? a.m - r : most;
        hipLaunchKernelGGL((norm_kernel<ROW, P>), dim3((unsigned)((rows + per - 1) / per)),
                           dim3(ROW == 1024 ? 1024 : 256), 0, stream, a, r);
        if (hipGetLastError() != hipSuccess) return -6;
    }
    return 0;
}

}  // namespace

int launch_norm(const NormArgs &a, hipStream_t stream)
{
    const int n = a.n;
    if (n <= 512) return launch<64, 1>(a, stream);
    if (n <= 1024) return launch<64, 2>(a, stream);
    if (n <= 2048) return launch<256, 1>(a, stream);
    if (n <= 4096) return launch<256, 2>(a, stream);
    if (n <= 8192) return launch<256, 4>(a, stream);
    if (n <= 16384) return launch<256, 8>(a, stream);
    if (n <= 32768) return launch<1024, 4>(a, stream);
    return launch<1024, 8>(a, stream);
}

}  // namespace q8
