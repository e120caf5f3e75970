// i8_stream.hip -- the 8-bit products with token and channel scales for few
// token rows (decode, small batches), where HBM bounds the kernel, and for
// small matrices, where the length of k does: no workgroup waits for another
// and its waves walk interleaved parts of k.  262144 x 2048 at one token: 78 us,
// 6.9 TB/s; 14336 x 4096 at 13 tokens 12.7 us, of which 59 MB are 8.4; 768 x 768
// from fp32 3.4 us in a graph, nearly all of it the launch and two round trips.
//
// Work decomposition:
//  * Workgroup = 4 or 8 waves, 16*NI weight rows x 16*MT tokens, all of k: the
//    waves take the 128-byte steps of k in turn (so a row's bytes are read in
//    runs of 512 or 1024) and their int32 sums are joined in LDS at the end.
//  * Each wave has a ring of stages of its own in LDS: the weight rows (and
//    token rows) of a step are copied straight there (16-byte buffer loads in
//    LDS DMA mode, 8 rows x 128 bytes each), so loads in flight cost no
//    registers, and a wave waits for its own loads only: no barrier until the
//    end.  Chunk c of a staged row is at slot c ^ ((row/2) % 8): the 16-byte
//    fragment reads of 16 rows fall on all 64 banks once.
//  * v_mfma_i32_16x16x64_i8: A = 16 weight rows, B = 16 tokens (rows past m
//    are zeros); a lane ends up with 4 consecutive outputs of one token.
//  * XL: the token rows are few values, quantized (or copied) by every
//    workgroup into LDS while its first weights are in flight: one launch.
#include "i8_device.h"
#include "q8_i8.h"

namespace q8 {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

constexpr int kStep = 128;
constexpr int kOut = 0x7fffff00;  // an offset past every resource: reads zero
// XL: values of all token rows together, in the kernels of one workgroup per CU
// and in those of many (NI = 4; more there would leave room for one per CU, and
// 262144 x 2048 at one token would take 98 us for 80).
template <int NI> constexpr int kXlValues = NI == 4 ? 8192 : 16384;
constexpr int kXlRows = 4;

struct StreamArgs {
    I8Args a;
    const void *xf;               // XL: the token rows as given
    int64_t xf_stride;            // bytes
};

// Barrier of LDS traffic only: the loads in flight to the ring are not waited
// for (a __syncthreads would).
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The token rows as 16-byte pieces, `per` of them a row; thread t has pieces
// t + 64 kWaves u.
template <int XT, int kWaves, int kValues>
struct Rows {
    static constexpr int kBytes = XT == Q8_T_F32 ? 4 : XT == Q8_T_I8 ? 1 : 2;
    static constexpr int kN = kValues * kBytes / 16 / (64 * kWaves);
    static_assert(kN > 0, "at least a piece per thread");
    u32x4 r[kN];
    int row[kN], at[kN];                   // kXlRows past the last piece

    __device__ __forceinline__ void load(const StreamArgs &p, int per)
    {
        const int m = (int)p.a.m;
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
            (void *)p.xf, 0, (m - 1) * (int)p.xf_stride + 16 * per, kBufferWord3);
#pragma unroll
        for (int u = 0; u < kN; ++u) {
            if (64 * kWaves * u >= m * per) break;
            const int i = threadIdx.x + 64 * kWaves * u;
            row[u] = i >= m * per ? kXlRows : (i >= per) + (i >= 2 * per) + (i >= 3 * per);
            at[u] = i - row[u] * per;
            const int off = row[u] < kXlRows ? row[u] * (int)p.xf_stride + 16 * at[u] : kOut;
            r[u] = __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0);
        }
    }

    // codes to xs [m][k], scales to scale (those of i8_quantize_rows; codes
    // are copied, with the scales they came with)
    __device__ __forceinline__ void store(const StreamArgs &p, int per, uint8_t *xs, float *scale,
                                          uint32_t (*amax)[kXlRows])
    {
        const int m = (int)p.a.m;
        if constexpr (XT == Q8_T_I8) {
#pragma unroll
            for (int u = 0; u < kN; ++u) {
                if (64 * kWaves * u >= m * per) break;
                if (row[u] < kXlRows) *(u32x4 *)(xs + 16 * (row[u] * per + at[u])) = r[u];
            }
            if (threadIdx.x < p.a.m) scale[threadIdx.x] = p.a.x_scale[threadIdx.x];
        } else {
            constexpr int V = kVec<XT>;
            uint32_t b[kXlRows] = {};
#pragma unroll
            for (int u = 0; u < kN; ++u) {
                if (64 * kWaves * u >= m * per) break;
                float v[V];
                unpack16<XT>(r[u], v);
                uint32_t c = 0;
#pragma unroll
                for (int j = 0; j < V; ++j) c = max(c, abs_bits(v[j]));
#pragma unroll
                for (int t = 0; t < kXlRows; ++t) b[t] = max(b[t], row[u] == t ? c : 0u);
            }
#pragma unroll
            for (int t = 0; t < kXlRows; ++t) {
                if (t >= m) break;
#pragma unroll
                for (int d = 32; d; d >>= 1) b[t] = max(b[t], (uint32_t)__shfl_xor((int)b[t], d));
                if ((threadIdx.x & 63) == 0) amax[threadIdx.x >> 6][t] = b[t];
            }
            lds_barrier();
            auto of_row = [&](int t) {
                uint32_t c = amax[0][t];
#pragma unroll
                for (int w = 1; w < kWaves; ++w) c = max(c, amax[w][t]);
                return row_scale(c);
            };
            if (threadIdx.x < m) scale[threadIdx.x] = of_row(threadIdx.x);
#pragma unroll
            for (int u = 0; u < kN; ++u) {
                if (64 * kWaves * u >= m * per) break;
                if (row[u] == kXlRows) continue;
                const RowCoder rc(of_row(row[u]));
                float v[V];
                unpack16<XT>(r[u], v);
                uint8_t *to = xs + V * (row[u] * per + at[u]);
                if constexpr (V == 4)
                    *(uint32_t *)to = rc.code4(v);
                else
                    *(u32x2 *)to = (u32x2){rc.code4(v), rc.code4(v + 4)};
            }
        }
    }
};

template <int kWaves, int kValues>
struct Rows<-1, kWaves, kValues> {
    __device__ __forceinline__ void load(const StreamArgs &, int) {}
    __device__ __forceinline__ void store(const StreamArgs &, int, uint8_t *, float *,
                                          uint32_t (*)[kXlRows]) {}
};

// NI: 16-row weight tiles (in the gated form NI/2 of gate rows, then NI/2 of
// the up rows of the same outputs).  MT: 16-token tiles.
// XT: the type of token rows taken as given (XL), or -1.  EPI: y = act(value) +
// residual.
template <int NI, int MT, int kWaves, int XT, bool GATED, bool EPI>
__global__ __launch_bounds__(64 * kWaves) void i8_stream_kernel(const StreamArgs p)
{
    constexpr bool XL = XT >= 0;
    constexpr int kRowsX = XL ? 0 : 16 * MT;
    constexpr int kRows = 16 * NI + kRowsX;
    constexpr int kStage = kRows * kStep;
    constexpr int kLoads = kRows / 8;                    // DMA instructions per stage
    constexpr int kOuts = 16 * (GATED ? NI / 2 : NI);    // outputs per tile
    static_assert(!XL || MT == 1, "few rows");
    __shared__ __align__(16) uint8_t ring0[kWaves][kStage];
    __shared__ __align__(16) uint8_t ring1[kWaves][kStage];
    __shared__ __align__(16) uint8_t xs[XL ? kXlValues<NI> : 16];
    __shared__ float xl_scale[kXlRows];
    __shared__ uint32_t xl_amax[kWaves][kXlRows];

    const I8Args &a = p.a;
    const int wave = wave_uniform((int)(threadIdx.x >> 6));
    const int lane = threadIdx.x & 63;
    const int lr = lane >> 3;
    const int grp = lane >> 4, li = lane & 15;
    const int k = (int)a.k, m = (int)min(a.m - (int64_t)blockIdx.y * 16 * MT, (int64_t)16 * MT);
    const int64_t n0 = (int64_t)blockIdx.x * kOuts, m0 = (int64_t)blockIdx.y * 16 * MT;
    const int w_rows = (int)min((int64_t)kOuts, a.n - n0);
    const int w_stride = (int)a.w_stride, x_stride = (int)a.x_stride;
    const int8_t *w_gate = a.w + n0 * a.w_stride;
    const int8_t *w_up = GATED ? w_gate + a.n * a.w_stride : w_gate;
    const int8_t *x = a.x + m0 * a.x_stride;
    const int w_bytes = (w_rows - 1) * w_stride + k;

    // steps wave, wave + kWaves, ...; a step past the end loads zeros, so every
    // wave has the same number of loads in flight
    auto issue = [&](int it, uint8_t *s) {
        const int st = it * kWaves + wave;
        const __amdgpu_buffer_rsrc_t rg =
            __builtin_amdgcn_make_buffer_rsrc((void *)w_gate, 0, w_bytes, kBufferWord3);
        const __amdgpu_buffer_rsrc_t ru =
            __builtin_amdgcn_make_buffer_rsrc((void *)w_up, 0, w_bytes, kBufferWord3);
#pragma unroll
        for (int f = 0; f < kLoads; ++f) {
            const int row = 8 * f + lr;                          // staged row
            const int off = st * kStep + 16 * ((lane & 7) ^ ((4 * f + (lr >> 1)) & 7));
            auto *dst = (__attribute__((address_space(3))) void *)(s + 1024 * f);
            if (8 * f < 16 * NI) {
                const int half = GATED && 8 * f >= 8 * NI;
                const int wr = row - (half ? 8 * NI : 0);
                const int o = off < k && wr < w_rows ? wr * w_stride + off : kOut;
                if (half)
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(ru, dst, 16, o, 0, 0, kCacheNT);
                else
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(rg, dst, 16, o, 0, 0, kCacheNT);
            } else {
                const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
                    (void *)x, 0, (m - 1) * x_stride + k, kBufferWord3);
                const int xr = row - 16 * NI;
                const int o = off < k && xr < m ? xr * x_stride + off : kOut;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, dst, 16, o, 0, 0, 0);
            }
        }
    };

    v4i acc[NI][MT];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = (v4i){0, 0, 0, 0};

    const int its = (k + kStep * kWaves - 1) / (kStep * kWaves);
    const int swz = (li >> 1) & 7;
    auto body = [&](int it, uint8_t *s) {
        // the next stage may still be in flight
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoads) : "memory");
        const int st = it * kWaves + wave;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const int c = 16 * ((4 * ks + grp) ^ swz);
            v4i w[NI], b[MT];
#pragma unroll
            for (int i = 0; i < NI; ++i) w[i] = *(const v4i *)(s + (16 * i + li) * kStep + c);
            if (XL) {
                // (columns past m are not used, bytes past k meet zeros of w)
                const int o = min(st * kStep + 16 * (4 * ks + grp), k - 16);
                b[0] = *(const v4i *)(xs + (li < m ? li * k : 0) + o);
            } else {
#pragma unroll
                for (int j = 0; j < MT; ++j)
                    b[j] = *(const v4i *)(s + (16 * NI + 16 * j + li) * kStep + c);
            }
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int j = 0; j < MT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[i], b[j], acc[i][j], 0, 0, 0);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the stage is read
        issue(it + 2, s);
    };

    // the scales this lane needs at the end: tiles wave, wave + kWaves, ...
    constexpr int kTiles = NI * MT;
    constexpr int kDone = GATED ? kTiles / 2 : kTiles;
    constexpr int kMine = (kDone + kWaves - 1) / kWaves;
    float s_gate[kMine][4], s_up[kMine][4], s_x[kMine], bias[kMine][4], res[kMine][4];
#pragma unroll
    for (int o = 0; o < kMine; ++o) {
        const int tile = min(o * kWaves + wave, kDone - 1);
        const int i = tile / MT, j = tile - i * MT;
        const int64_t t = m0 + min(16 * j + li, m - 1);
        s_x[o] = XL ? 0.0f : a.x_scale[t];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t n = min(n0 + 16 * i + 4 * grp + r, a.n - 1);
            s_gate[o][r] = a.w_scale[n];
            s_up[o][r] = GATED ? a.w_scale[a.n + n] : 0.0f;
            bias[o][r] = !GATED && a.bias ? a.bias[n] : 0.0f;
            if (EPI) res[o][r] = a.residual ? load_in(a.residual, a.y_type, t * a.r_stride + n) : 0.0f;
        }
    }
    const int per = k * (XT == Q8_T_F32 ? 4 : XT == Q8_T_I8 ? 1 : 2) / 16;
    Rows<XT, kWaves, kXlValues<NI>> rows;
    rows.load(p, per);
    issue(0, ring0[wave]);
    issue(1, ring1[wave]);
    if (XL) {
        rows.store(p, per, xs, xl_scale, xl_amax);
        lds_barrier();
    }
    // whole turns of the ring: stages past the end hold zeros
    for (int it = 0; it < its; it += 2) {
        body(it, ring0[wave]);
        body(it + 1, ring1[wave]);
    }

    // join the waves' sums: each wave its own ring slot, then wave w finishes
    // tiles w, w + kWaves, ...  (zeros still in flight to the ring land first)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    v4i *join = (v4i *)ring0;                              // [kWaves][kTiles][64]
    static_assert(kWaves * kTiles * 64 * 16 <= (int)sizeof(ring0), "join fits");
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) join[(wave * kTiles + i * MT + j) * 64 + lane] = acc[i][j];
    __syncthreads();
#pragma unroll
    for (int o = 0; o < kMine; ++o) {
        const int tile = o * kWaves + wave;
        if (kDone % kWaves != 0 && tile >= kDone) break;
        v4i s = join[tile * 64 + lane], u = s;
        if (GATED) u = join[(tile + kDone) * 64 + lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) {
            s += join[(w * kTiles + tile) * 64 + lane];
            if (GATED) u += join[(w * kTiles + tile + kDone) * 64 + lane];
        }
        const int i = tile / MT, j = tile - i * MT;
        const int tr = 16 * j + li;
        if (tr >= m) continue;
        const float sx = XL ? xl_scale[min(tr, kXlRows - 1)] : s_x[o];
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (GATED)
                v[r] = silu_mul(i8_rescale(s[r], sx, s_gate[o][r]), i8_rescale(u[r], sx, s_up[o][r]));
            else
                v[r] = a.bias ? i8_rescale(s[r], sx, s_gate[o][r], bias[o][r])
                              : i8_rescale(s[r], sx, s_gate[o][r]);
            if (EPI) {
                v[r] = activate(a.act, v[r]);
                if (a.residual) v[r] += res[o][r];
            }
        }
        const int64_t n = n0 + 16 * i + 4 * grp, at = (m0 + tr) * a.y_stride + n;
        const int left = (int)min((int64_t)4, a.n - n);
        if (a.y_type == Q8_T_F32)
            store_run<Q8_T_F32>(a.y, at, v, left);
        else if (a.y_type == Q8_T_F16)
            store_run<Q8_T_F16>(a.y, at, v, left);
        else
            store_run<Q8_T_BF16>(a.y, at, v, left);
    }
}

int64_t workgroups(const I8Args &a, bool gated, int ni, int mt)
{
    const int64_t outs = 16 * (gated ? ni / 2 : ni);
    return (a.n + outs - 1) / outs * ((a.m + 16 * mt - 1) / (16 * mt));
}

template <int NI, int MT, int NW, int XT>
int launch(const StreamArgs &p, bool gated, hipStream_t stream)
{
    const int64_t by = (p.a.m + 16 * MT - 1) / (16 * MT), bx = workgroups(p.a, gated, NI, MT) / by;
    if (bx >= (1 << 24)) return Q8_E_UNSUPPORTED;
    const dim3 grid((unsigned)bx, (unsigned)by);
    bool done = false;
    if constexpr (NI > 1)            // (shape() gives the gated form two rows of tiles)
        if (gated) {
            hipLaunchKernelGGL((i8_stream_kernel<NI, MT, NW, XT, true, false>), grid, dim3(64 * NW), 0, stream, p);
            done = true;
        }
    if (!done && p.a.epilogue)
        hipLaunchKernelGGL((i8_stream_kernel<NI, MT, NW, XT, false, true>), grid, dim3(64 * NW), 0, stream, p);
    else if (!done)
        hipLaunchKernelGGL((i8_stream_kernel<NI, MT, NW, XT, false, false>), grid, dim3(64 * NW), 0, stream, p);
    return hipGetLastError() == hipSuccess ? 0 : -6;
}

// The smallest workgroups of which the device needs at most one per CU are the
// fastest (a workgroup's time grows with its rows: at k = 4096, in 4 waves,
// 7.6 us for 32 weight rows x 16 tokens, 8.4 for 32 x 32, 10.6 for 32 x 64,
// 14.1 for 64 x 64); 0 where even 64 x 64 ones are more.
struct Shape {
    int ni, mt;
};

Shape shape(const I8Args &a, bool gated)
{
    const Shape s[5] = {{1, 1}, {2, 1}, {2, 2}, {2, 4}, {4, 4}};
    for (int i = gated ? 1 : 0; i < 5; ++i)
        if ((i < 2 || 8 * s[i].mt < a.m) && workgroups(a, gated, s[i].ni, s[i].mt) <= 256) return s[i];
    return {0, 0};
}

// Waves of the small shapes.  A turn of the ring is two steps per wave, 1024
// values of k in 4 waves: past that 8 waves take half the turns (1 x 4096 x 4096
// 7.5 -> 6.0 us, 1 x 8192 x 2048 11.8 -> 8.3, 16 x 8192 x 1024 13.5 -> 11.3),
// up to it they only join more sums (1 x 768 x 2 x 2048 gated 4.0 -> 4.7).
template <int NI, int MT, int XT>
int launch_small(const StreamArgs &p, bool gated, hipStream_t stream)
{
    return p.a.k > 2 * 4 * kStep ? launch<NI, MT, 8, XT>(p, gated, stream)
                                 : launch<NI, MT, 4, XT>(p, gated, stream);
}

template <int XT>
int launch_rows(const StreamArgs &p, bool gated, hipStream_t stream)
{
    const int ni = shape(p.a, gated).ni;
    if (ni == 1) return launch_small<1, 1, XT>(p, gated, stream);
    return ni ? launch_small<2, 1, XT>(p, gated, stream) : launch<4, 1, 4, XT>(p, gated, stream);
}

}  // namespace

bool i8_stream_ok(const I8Args &a, bool gated) { return a.m <= 64 || shape(a, gated).ni != 0; }

// (graph times with 16384 values against a quantizer launch: 1 x 14336 x 4096
// bfloat16 13.8 and 16.8 us, fp32 15.0 and 19.2, 2 x 8192 x 2048 9.4 and 10.4, but
// 4 x 4096 x 2048 fp32 9.4 and 8.0)
bool i8_inline_ok(const I8Args &a, bool gated)
{
    const int64_t values = a.m <= 2 && shape(a, gated).ni ? kXlValues<1> : kXlValues<4>;
    return a.m <= kXlRows && a.m * a.k <= values;
}

int launch_i8_stream(const I8Args &a, const void *xf, int xf_type, int64_t xf_stride, bool gated,
                     hipStream_t stream)
{
    StreamArgs p;
    p.a = a;
    p.xf = xf; p.xf_stride = xf_stride;
    if (xf && xf_type == Q8_T_F32) return launch_rows<Q8_T_F32>(p, gated, stream);
    if (xf && xf_type == Q8_T_F16) return launch_rows<Q8_T_F16>(p, gated, stream);
    if (xf && xf_type == Q8_T_BF16) return launch_rows<Q8_T_BF16>(p, gated, stream);
    if (xf) return launch_rows<Q8_T_I8>(p, gated, stream);
    const Shape s = shape(a, gated);
    if (s.ni == 1) return launch_small<1, 1, -1>(p, gated, stream);
    if (s.mt == 1) return launch_small<2, 1, -1>(p, gated, stream);
    if (s.mt == 2) return launch_small<2, 2, -1>(p, gated, stream);
    if (s.ni == 2) return launch<2, 4, 4, -1>(p, gated, stream);
    // HBM bounds it: 64 weight rows, all tokens at once where they are 64 or fewer
    if (a.m <= 16) return launch<4, 1, 4, -1>(p, gated, stream);
    if (a.m <= 32) return launch<4, 2, 4, -1>(p, gated, stream);
    return launch<4, 4, 4, -1>(p, gated, stream);
}

}  // namespace q8
