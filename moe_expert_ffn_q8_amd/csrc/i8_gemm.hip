// i8_gemm.hip -- the 8-bit products with token and channel scales for many
// token rows, on the gfx950 int8 matrix cores: Y[m][n] from codes X[m][k] and
// W[n][k], and the gated form.
//
// One scale per row and per column leaves the int32 sums in the matrix core
// over all of k: 32 v_mfma_i32_32x32x32_i8 per 128 bytes of k and wave tile, no
// rescale between them, one rescale per output at the end.  Bound by the
// matrix cores.
//
// Work decomposition:
//  * Workgroup = WN x WM waves, tile TN weight rows x TM tokens; a wave
//    computes NI x MI tiles of 32 x 32.  In the gated form half of a wave's
//    weight rows are gate rows and the other half the up rows of the same
//    outputs, so that silu(g) * u is formed in registers.
//  * k is walked in steps of 128 bytes.  A step of both operands goes straight
//    from HBM to LDS (16-byte buffer loads in LDS DMA mode; rows past m or n
//    and bytes past k read as zero), double-buffered: the loads of step s + 2
//    go out when the last fragments of step s are in registers and have a
//    whole step to land.
//  * A staged row is 128 bytes, its 16-byte chunk c at slot c ^ ((row/2) % 8):
//    the 16-byte fragment reads of 16 consecutive rows then fall on all 64
//    banks once, and the swizzle costs nothing (the DMA's LDS side is linear,
//    the lanes' global addresses carry it).
//  * Matrix operands: A = weight rows, B = tokens, so that a lane's results
//    are runs of 4 consecutive outputs of one token.
//  * Workgroups are dealt to the 8 XCDs round robin; each XCD takes a
//    contiguous run of tiles, up to 8 token tiles of one weight tile next to
//    each other, so that an XCD's L2 serves both operands' reuse.
#include "i8_device.h"
#include "q8_i8.h"

namespace q8 {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

constexpr int kStep = 128;        // bytes of k per step
constexpr int kGroupM = 8;        // token tiles next to each other
constexpr int kOut = 0x7fffff00;  // an offset past every resource: reads zero

struct TileGrid {
    int tiles_n, tiles_m;
};

template <int TN, int TM, int WN, int WM, int YT, bool GATED>
__global__ __launch_bounds__(64 * WN * WM, 2) void i8_gemm_kernel(const I8Args a, const TileGrid g)
{
    constexpr int kWaves = WN * WM;
    constexpr int NI = TN / WN / 32, MI = TM / WM / 32;
    constexpr int kLoadsW = TN / 8 / kWaves, kLoadsX = TM / 8 / kWaves;
    constexpr int kCols = GATED ? TN / 2 : TN;          // outputs per tile
    constexpr int kWaveCols = kCols / WN;
    static_assert(TN % (8 * kWaves) == 0 && TM % (8 * kWaves) == 0, "whole loads per wave");
    static_assert(!GATED || NI % 2 == 0, "gate and up halves");
    __shared__ __align__(16) uint8_t stage0[(TN + TM) * kStep];
    __shared__ __align__(16) uint8_t stage1[(TN + TM) * kStep];

    const int wave = wave_uniform((int)(threadIdx.x >> 6));
    const int lane = threadIdx.x & 63;
    const int wn = wave / WM, wm = wave % WM;
    const int h = lane >> 5, li = lane & 31;

    // this workgroup's tile
    const int nwg = g.tiles_n * g.tiles_m;
    const int xcd = blockIdx.x & 7, per = nwg >> 3, rest = nwg & 7;
    const int work = xcd * per + min(xcd, rest) + (blockIdx.x >> 3);
    const int group = work / (kGroupM * g.tiles_n);
    const int gm = min(kGroupM, g.tiles_m - group * kGroupM);
    const int in = work - group * kGroupM * g.tiles_n;
    const int64_t n0 = (int64_t)(in / gm) * kCols;
    const int64_t m0 = (int64_t)(group * kGroupM + in % gm) * TM;

    // operand rows of the tile
    const int k = (int)a.k;
    const int w_rows = (int)min((int64_t)kCols, a.n - n0), x_rows = (int)min((int64_t)TM, a.m - m0);
    const int w_stride = (int)a.w_stride, x_stride = (int)a.x_stride;
    const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(a.x + m0 * a.x_stride), 0, (x_rows - 1) * x_stride + k, kBufferWord3);
    const int8_t *w_base[kLoadsW];     // (no array of resources: the host pass has no such type)
    int voff[kLoadsW + kLoadsX];
    // load u of a wave: staged rows 8f .. 8f+7, f = wave + kWaves * u
    const int lr = lane >> 3;
    const int chunk = (lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7);   // (8f + lr)/2 % 8
    static_assert(kWaves % 2 == 0, "the chunk of a lane is the same for every load");
#pragma unroll
    for (int u = 0; u < kLoadsW; ++u) {
        const int b = 8 * (wave + kWaves * u);          // of TN; 32-row groups are uniform
        int row = b;
        const int8_t *base = a.w + n0 * a.w_stride;
        if (GATED) {
            const int grp = b / 32 % NI, half = grp / (NI / 2);
            row = b / (32 * NI) * kWaveCols + 32 * (grp % (NI / 2)) + b % 32;
            if (half) base += a.n * a.w_stride;
        }
        w_base[u] = base;
        voff[u] = row + lr < w_rows ? (row + lr) * w_stride + 16 * chunk : kOut;
    }
#pragma unroll
    for (int u = 0; u < kLoadsX; ++u) {
        const int row = 8 * (wave + kWaves * u) + lr;
        voff[kLoadsW + u] = row < x_rows ? row * x_stride + 16 * chunk : kOut;
    }

    auto issue = [&](int st, uint8_t *s) {
        const bool in_k = 16 * chunk < k - st * kStep;
        const int so = st * kStep;
#pragma unroll
        for (int u = 0; u < kLoadsW + kLoadsX; ++u) {
            const int off = in_k ? voff[u] : kOut;
            const int f = u < kLoadsW ? wave + kWaves * u : TN / 8 + wave + kWaves * (u - kLoadsW);
            auto *dst = (__attribute__((address_space(3))) void *)(s + 1024 * f);
            if (u < kLoadsW) {
                const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
                    (void *)w_base[u], 0, (w_rows - 1) * w_stride + k, kBufferWord3);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, dst, 16, off, so, 0, 0);
            } else
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, dst, 16, off, so, 0, 0);
        }
    };

    v16i acc[NI][MI];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < MI; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

    struct Frag {
        v4i w[NI], x[MI];
    };
    // 32 bytes of k (k-group s of the step): lane = row li, bytes 16h .. 16h+15
    const int row_w = (wn * NI * 32 + li) * kStep, row_x = (TN + wm * MI * 32 + li) * kStep;
    const int swz = (li >> 1) & 7;
    auto load = [&](const uint8_t *s, int ks, Frag &f) {
        const int c = 16 * ((2 * ks + h) ^ swz);
#pragma unroll
        for (int i = 0; i < NI; ++i) f.w[i] = *(const v4i *)(s + row_w + c + i * 32 * kStep);
#pragma unroll
        for (int j = 0; j < MI; ++j) f.x[j] = *(const v4i *)(s + row_x + c + j * 32 * kStep);
    };
    auto mul = [&](const Frag &f) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < MI; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.w[i], f.x[j], acc[i][j], 0, 0, 0);
    };
    auto landed = [&]() {
        __builtin_amdgcn_s_waitcnt(0x3f70);    // vmcnt(0): this wave's loads are in LDS
        __syncthreads();
    };

    const int steps = (k + kStep - 1) / kStep;
    Frag f0, f1;
    issue(0, stage0);
    if (steps > 1) issue(1, stage1);
    landed();
    load(stage0, 0, f0);
    auto body = [&](int st, uint8_t *cur, const uint8_t *next) {
        load(cur, 1, f1);
        mul(f0);
        load(cur, 2, f0);
        mul(f1);
        load(cur, 3, f1);
        mul(f0);
        landed();                              // and every wave is done reading cur
        if (st + 2 < steps) issue(st + 2, cur);
        if (st + 1 < steps) load(next, 0, f0);
        mul(f1);
    };
    for (int st = 0; st < steps; st += 2) {
        body(st, stage0, stage1);
        if (st + 1 < steps) body(st + 1, stage1, stage0);
    }

    // result r of a lane: weight row 8(r/4) + 4h + r%4 of its tile, token li
#pragma unroll
    for (int j = 0; j < MI; ++j) {
        const int64_t t = m0 + (wm * MI + j) * 32 + li;
        if (t >= a.m) continue;
        const float sx = a.x_scale[t];
#pragma unroll
        for (int i = 0; i < (GATED ? NI / 2 : NI); ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int64_t n = n0 + wn * kWaveCols + 32 * i + 8 * (r / 4) + 4 * h + r % 4;
                if (n >= a.n) continue;
                float v;
                if (GATED)
                    v = silu_mul(i8_rescale(acc[i][j][r], sx, a.w_scale[n]),
                                 i8_rescale(acc[i + NI / 2][j][r], sx, a.w_scale[a.n + n]));
                else
                    v = a.bias ? i8_rescale(acc[i][j][r], sx, a.w_scale[n], a.bias[n])
                               : i8_rescale(acc[i][j][r], sx, a.w_scale[n]);
                store_out<YT>(a.y, t * a.y_stride + n, v);
            }
    }
}

template <int TN, int TM, int WN, int WM, int YT, bool GATED>
int launch_tiles(const I8Args &a, hipStream_t stream)
{
    const int64_t cols = GATED ? TN / 2 : TN;
    const int64_t tn = (a.n + cols - 1) / cols, tm = (a.m + TM - 1) / TM;
    if (tn * tm >= ((int64_t)1 << 22)) return Q8_E_UNSUPPORTED;
    hipLaunchKernelGGL((i8_gemm_kernel<TN, TM, WN, WM, YT, GATED>), dim3((unsigned)(tn * tm)),
                       dim3(64 * WN * WM), 0, stream, a, (TileGrid{(int)tn, (int)tm}));
    return hipGetLastError() == hipSuccess ? 0 : -6;
}

template <int YT, bool GATED>
int launch_form(const I8Args &a, hipStream_t stream)
{
    const int64_t cols = GATED ? 128 : 256;
    if ((a.n + cols - 1) / cols * ((a.m + 255) / 256) >= 256)
        return launch_tiles<256, 256, 4, 2, YT, GATED>(a, stream);
    return launch_tiles<128, 128, 2, 2, YT, GATED>(a, stream);
}

template <int YT>
int launch_type(const I8Args &a, bool gated, hipStream_t stream)
{
    return gated ? launch_form<YT, true>(a, stream) : launch_form<YT, false>(a, stream);
}

}  // namespace

int launch_i8_gemm(const I8Args &a, bool gated, hipStream_t stream)
{
    if (a.y_type == Q8_T_F32) return launch_type<Q8_T_F32>(a, gated, stream);
    if (a.y_type == Q8_T_F16) return launch_type<Q8_T_F16>(a, gated, stream);
    return launch_type<Q8_T_BF16>(a, gated, stream);
}

}  // namespace q8
