// norm.hip -- norms of rows: of a tensor, or of a residual stream that takes a
// block's output first, to floats or to int8 codes with a scale per row.
//
//   a  = x, or its norm with post_weight (and post_bias)
//   r' = round(gate * a + residual_scale * r)      stored, and what comes next reads it
//   y  = round(norm(r') * weight + bias), or codes of the fp32 y by the row rule
//   norm(v) = (v - mean) / sqrt(var + eps), or v / sqrt(mean of v^2 + eps)
//
// Two arithmetics.  Where any row is fp32 or codes come out, everything between the
// roundings is in 64 bits: a code of the row rule turns at a border, and then
// does not hang on the order of a sum.  Where all rows are 16-bit floats it is
// in 32 bits, with means and sums over threads in 64: conversions to and from 64
// bits issue at a quarter of the rate of other instructions, and everything in 64
// would bound the kernel (16384 x 4096 bfloat16 181 us; the squares alone 173).
// There v - mean is (v - p) - q with p the mean in 32 bits and q its rest, two
// roundings of about the result's size wherever the mean and the largest values
// lie; squares that 32 bits do not hold are summed again in 64, and a row whose
// root or differences may leave 32 bits is normed in 64, or scaled.
//
// HBM bounds it: a row lies in the registers of one wave or workgroup, 8 values a
// piece, so every tensor is read and written once; where rows are many a
// workgroup takes several, keeps the weights and has the next row's loads on
// their way (16384 x 4096 bfloat16, residual, mean and bias: 133 to 137 us, 3.9 to 4.0
// TB/s, 79 to 81% of a copy; 257 x 4096 with a norm after the block and gates, to codes:
// 10.6 us, a chain of loads, three reductions and stores; 16384 x 4096 with residual to
// codes 162 to 168 us, from fp32 to fp32 213 to 235).
#include <type_traits>

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
        store16<Q8_T_F16, true>((uint8_t *)((uint16_t *)row + i), pack_vec<Q8_T_F16>(v), left);
    else
        store16<Q8_T_BF16, true>((uint8_t *)((uint16_t *)row + i), pack_vec<Q8_T_BF16>(v), left);
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

__device__ __forceinline__ int type_bytes(int type) { return type == Q8_T_F32 ? 4 : type == Q8_T_I8 ? 1 : 2; }

// A piece as loaded, of 16-bit values (HALF) or of any type.
template <bool HALF>
struct Piece {
    float v[kPiece];
    __device__ __forceinline__ void load(const void *row, int type, int64_t i, int left) { load8(row, type, i, left, v); }
    __device__ __forceinline__ void get(int, float (&to)[kPiece]) const
    {
#pragma unroll
        for (int j = 0; j < kPiece; ++j) to[j] = v[j];
    }
};
template <>
struct Piece<true> {
    u32x4 raw;
    __device__ __forceinline__ void load(const void *row, int, int64_t i, int left)
    {
        const uint8_t *p = (const uint8_t *)row + 2 * i;                   // (either 16-bit type)
        raw = left >= kPiece ? __builtin_nontemporal_load((const u32x4_any *)p) : load16<Q8_T_BF16>(p, left);
    }
    __device__ __forceinline__ void get(int type, float (&to)[kPiece]) const
    {
        if (type == Q8_T_F16)
            unpack16<Q8_T_F16>(raw, to);
        else
            unpack16<Q8_T_BF16>(raw, to);
    }
};

// ROW threads per row, P pieces of 8 values each.  HALF: x, the residual and
// gates by row are of 16-bit types.
template <int ROW, int P, bool WIDE, bool HALF>
__global__ __launch_bounds__(ROW > 256 ? ROW : 256) void norm_kernel(const NormArgs a)
{
    typedef typename std::conditional<WIDE, double, float>::type R;
    constexpr bool FEW = P <= (HALF ? 4 : 2);   // a row's loads all at once
    constexpr bool AHEAD = FEW && HALF;         // and the next row's before its work
    // Rows far from 1 in code of their own: for few pieces no product for the others
    // (16384 x 4096 137 us, with one 142), for many registers count (4096 x 14336
    // with a norm after the block 188 apart, 164 with the product)
    constexpr bool APART = !WIDE && P <= 2;
    constexpr int kPer = ROW == 64 ? 4 : 1, K = FEW ? P : 1;
    __shared__ double part[2][4][ROW / 64];
    __shared__ uint32_t part_max[2][ROW / 64];
    const int t = threadIdx.x % ROW, n = a.n;
    const double inv_n = 1.0 / n;
    int begin;                             // of this thread's values
    auto at = [&](int p) { return begin + ROW * p * kPiece; };
    const bool gate_row = a.gate && a.gate_stride != 0;
    float w[K][kPiece] = {}, pw[K][kPiece] = {};
    bool first = true;
    int odd = 0;                           // LDS of one row and the next
    Piece<HALF> xs[P], rs[K], gs[K];
    auto load_row = [&](int64_t row) {
        const uint8_t *x = (const uint8_t *)a.x + row * a.x_stride * type_bytes(a.x_type);
        const uint8_t *r = (const uint8_t *)a.residual + row * a.r_stride * type_bytes(a.r_type);
        const uint8_t *g = (const uint8_t *)a.gate + row * a.gate_stride * type_bytes(a.gate_type);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int i = at(p), left = n - i;
            xs[p].load(x, a.x_type, i, left);
            if (FEW && a.residual) rs[p].load(r, a.r_type, i, left);
            if (FEW && gate_row) gs[p].load(g, a.gate_type, i, left);
        }
    };
    for (int64_t row = (int64_t)blockIdx.x * kPer + threadIdx.x / ROW; row < a.m;
         row += (int64_t)gridDim.x * kPer, odd ^= 1) {
        // (formed in every turn: addresses and converted weights carried over the
        // loop would take the registers of several waves)
        begin = t * kPiece;
        asm volatile("" : "+v"(begin));
#pragma unroll
        for (int p = 0; p < K; ++p)
#pragma unroll
            for (int j = 0; j < kPiece; ++j) asm volatile("" : "+v"(w[p][j]), "+v"(pw[p][j]));
        const uint8_t *r = (const uint8_t *)a.residual + row * a.r_stride * type_bytes(a.r_type);
        const uint8_t *g = (const uint8_t *)a.gate + row * a.gate_stride * type_bytes(a.gate_type);
        float v[P][kPiece];
        if (!AHEAD || first) load_row(row);
        if (FEW && first) {                // (kept where rows are many)
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int i = at(p), left = n - i;
                if (a.post) load8(a.post_weight, Q8_T_F32, i, left, pw[p]);
                load8(a.weight, Q8_T_F32, i, left, w[p]);
            }
            first = false;
        }
#pragma unroll
        for (int p = 0; p < P; ++p) xs[p].get(a.x_type, v[p]);
        Piece<HALF> rn[K], gn[K];
        if (AHEAD) {                       // the next row's streams are on their way during this one's work
#pragma unroll
            for (int p = 0; p < K; ++p) {
                rn[p] = rs[p];
                gn[p] = gs[p];
            }
            const int64_t next = row + (int64_t)gridDim.x * kPer;
            if (next < a.m) load_row(next);
        }
        // the row held as (lift v - pivot) - middle, and 1 / (lift sqrt(mean square +
        // eps)).  far: a row whose differences or root may leave 32 bits; it is normed in
        // 64 bits (APART), or has a power of two as its lift, which is 1 else
        R lift = 1, pivot = 0, middle = 0, rstd;
        double mean = 0.0, root = 0.0;
        bool far = false;
        auto centred = [&](float x, R by) { return a.layer ? fma((R)x, by, -pivot) - middle : (R)x * by; };
        auto normed = [&](float x, auto apart) -> R {
            if constexpr (decltype(apart)::value) return (R)(((double)x - mean) * root);
            return centred(x, WIDE || APART ? (R)1 : lift) * rstd;
        };
        auto each_kind = [&](auto f) {
            if (APART && far)
                f(std::integral_constant<bool, APART>());
            else
                f(std::false_type());
        };
        auto stats = [&](double *p0, double *p1) {
            lift = 1;
            if (a.layer) {
                double s = 0.0;
#pragma unroll
                for (int p = 0; p < P; ++p)
#pragma unroll
                    for (int j = 0; j < kPiece; ++j) s += (double)v[p][j];     // (0 beyond the row)
                mean = row_sum<ROW>(s, p0) * inv_n;
                pivot = (R)mean;
                middle = (R)(mean - (double)pivot);                            // (0 where R is double)
            }
            R s = 0;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int left = n - at(p);
#pragma unroll
                for (int j = 0; j < kPiece; ++j) {
                    const R d = j < left ? centred(v[p][j], (R)1) : (R)0;
                    s = fma(d, d, s);
                }
            }
            double sum = (double)s;
            if (!WIDE && begin < n && !(s > 1e-30f && s < 3e38f)) {    // squares, or differences, that 32 bits do not hold
                sum = 0.0;
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const int left = n - at(p);
#pragma unroll
                    for (int j = 0; j < kPiece; ++j) {
                        float x = v[p][j];
                        asm("" : "+v"(x));                 // (not the values converted above: registers)
                        const double d = j < left ? (double)x - mean : 0.0;
                        sum = fma(d, d, sum);
                    }
                }
            }
            const double square = row_sum<ROW>(sum, p1) * inv_n + (double)a.eps;
            far = false;
            if (!WIDE && square > 1e-30 && square < 1e37) {
                rstd = __builtin_amdgcn_rsqf((float)square);
                return;
            }
            root = 1.0 / sqrt(square);
            far = !WIDE && wave_uniform(root > 1e36 || root < 1e-36);
            if (far && !APART) {
                lift = root > 1e36 ? (R)0x1p64 : (R)0x1p-64;
                mean *= (double)lift;
                root /= (double)lift;
                pivot = (R)mean;
                middle = (R)(mean - (double)pivot);
            }
            rstd = (R)root;
        };

        if (a.residual) {
            if (a.post) stats(part[odd][0], part[odd][1]);
            uint8_t *ro = (uint8_t *)a.residual_out + row * a.ro_stride * type_bytes(a.r_type);
            auto update = [&](auto apart) {
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const int i = at(p), left = n - i, k = FEW ? p : 0;
                    if (left <= 0) continue;
                    float rv[kPiece], gv[kPiece], pb[kPiece];
                    if (!FEW || decltype(apart)::value) __builtin_amdgcn_sched_barrier(0);   // (one piece at a time: registers)
                    if (!FEW) {
                        rs[0].load(r, a.r_type, i, left);
                        if (gate_row) gs[0].load(g, a.gate_type, i, left);
                        if (a.post) load8(a.post_weight, Q8_T_F32, i, left, pw[0]);
                    }
                    (AHEAD ? rn : rs)[k].get(a.r_type, rv);
                    if (gate_row) (AHEAD ? gn : gs)[k].get(a.gate_type, gv);
                    else if (a.gate) load8(a.gate, a.gate_type, i, left, gv);
                    if (a.post_bias) load8(a.post_bias, Q8_T_F32, i, left, pb);
#pragma unroll
                    for (int j = 0; j < kPiece; ++j) {
                        R y = (R)v[p][j];
                        if (a.post) {
                            y = normed(v[p][j], apart) * (R)pw[k][j];
                            if (a.post_bias) y += (R)pb[j];
                        }
                        if (a.gate) y *= (R)gv[j];
                        v[p][j] = as_stored((float)fma((R)a.residual_scale, (R)rv[j], y), a.r_type);
                        if (j >= left) v[p][j] = 0.0f;
                    }
                    store8(ro, a.r_type, i, left, v[p]);
                }
            };
            each_kind(update);
        }

        stats(part[odd][2], part[odd][3]);
        const bool codes = a.y_type == Q8_T_I8;
        uint8_t *y = (uint8_t *)a.y + row * a.y_stride * type_bytes(a.y_type);
        uint32_t amax = 0;
        auto finish = [&](auto apart) {
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int i = at(p), left = n - i, k = FEW ? p : 0;
                if (left <= 0) continue;
                float b[kPiece];
                if (!FEW || decltype(apart)::value) __builtin_amdgcn_sched_barrier(0);
                if (!FEW) {
                    load8(a.weight, Q8_T_F32, i, left, w[0]);
                }
                if (a.bias) load8(a.bias, Q8_T_F32, i, left, b);
#pragma unroll
                for (int j = 0; j < kPiece; ++j) {
                    R o = normed(v[p][j], apart) * (R)w[k][j];
                    if (a.bias) o += (R)b[j];
                    v[p][j] = (float)o;
                    if (j < left) amax = max(amax, abs_bits(v[p][j]));
                }
                if (!WIDE || !codes) store8(y, a.y_type, i, left, v[p]);
            }
        };
        each_kind(finish);
        if (!WIDE || !codes) continue;
#pragma unroll
        for (int d = 32; d; d >>= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, d));
        if constexpr (ROW > 64) {
            if ((threadIdx.x & 63) == 0) part_max[odd][threadIdx.x >> 6] = amax;
            __syncthreads();
            amax = 0;
#pragma unroll
            for (int k = 0; k < ROW / 64; ++k) amax = max(amax, part_max[odd][k]);
        }
        const float s = row_scale(amax);
        if (t == 0) a.y_scale[row] = s;
        const RowCoder rc(s);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int i = at(p);            // (n is a multiple of 32)
            if (i < n) *(u32x2 *)(y + i) = (u32x2){rc.code4(v[p]), rc.code4(v[p] + 4)};
        }
    }
}

// Workgroups: one per row (four rows, by waves), or as many as the device holds,
// which then take several (16384 x 4096 bfloat16: 133 us, with twice or two
// thirds as many 144 and 169).
template <int ROW, int P, bool WIDE, bool HALF>
int launch(const NormArgs &a, hipStream_t stream)
{
    constexpr int64_t per = ROW == 64 ? 4 : 1, threads = ROW > 256 ? ROW : 256;
    static const int resident = [] {
        int n = 0;
        const hipError_t e = hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, norm_kernel<ROW, P, WIDE, HALF>,
                                                                          (int)threads, 0);
        return 256 * (e == hipSuccess && n > 0 ? n : 1);       // (256 CUs)
    }();
    const int64_t groups = (a.m + per - 1) / per;
    hipLaunchKernelGGL((norm_kernel<ROW, P, WIDE, HALF>), dim3((unsigned)(groups < resident ? groups : resident)),
                       dim3((unsigned)threads), 0, stream, a);
    return hipGetLastError() == hipSuccess ? 0 : -6;
}

template <int ROW, int P>
int launch_shape(const NormArgs &a, hipStream_t stream)
{
    auto half = [](int type) { return type == Q8_T_F16 || type == Q8_T_BF16; };
    const bool halves = half(a.x_type) && (!a.residual || half(a.r_type)) &&
                        (!a.gate || a.gate_stride == 0 || half(a.gate_type));
    if (!halves) return launch<ROW, P, true, false>(a, stream);
    return half(a.y_type) ? launch<ROW, P, false, true>(a, stream) : launch<ROW, P, true, true>(a, stream);
}

}  // namespace

int launch_norm(const NormArgs &a, hipStream_t stream)
{
    const int n = a.n;
    if (n <= 512) return launch_shape<64, 1>(a, stream);
    if (n <= 1024) return launch_shape<64, 2>(a, stream);
    if (n <= 2048) return launch_shape<256, 1>(a, stream);
    if (n <= 4096) return launch_shape<256, 2>(a, stream);
    if (n <= 8192) return launch_shape<512, 2>(a, stream);
    if (n <= 16384) return launch_shape<512, 4>(a, stream);
    if (n <= 32768) return launch_shape<512, 8>(a, stream);
    return launch_shape<512, 16>(a, stream);
}

}  // namespace q8
