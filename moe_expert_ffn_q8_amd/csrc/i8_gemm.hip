// i8_gemm.hip -- the 8-bit products with token and channel scales for many
// token rows, on the gfx950 int8 matrix cores: Y[m][n] from codes X[m][k] and
// W[n][k], and the gated form.
//
// One scale per row and per column leaves the int32 sums in the matrix core
// over all of k: 32 v_mfma_i32_32x32x32_i8 per 128 bytes of k and wave tile, no
// rescale between them, one rescale per output at the end.  Bound by the
// matrix cores, and they by power on codes that are not mostly zeros: 8192^3
// 441 us, 2.5 POPS; gated 2048 x 4096 x 2*14336 206 to 221 us, 2.2 to 2.3 POPS at
// 1.8 GHz; 512 x 4096 x 14336 30 to 32 us on part of the device.  With few steps
// the start and end of each tile are most of the time: 333 x 768 x 50257 25 to 29
// us, of which the outputs are 10.  A long k with few outputs leaves CUs idle (k
// is not split but in the narrow kernel): 512 x 14336 x 4096 53 to 68 us.
//
// Work decomposition:
//  * Workgroup = WN x WM waves, tile TN weight rows x TM tokens; a wave
//    computes NI x MI tiles of 32 x 32.  In the gated form half of a wave's
//    weight rows are gate rows and the other half the up rows of the same
//    outputs, so that silu(g) * u is formed in registers.
//  * k is walked in steps of 128 bytes.  A step of both operands goes straight
//    from HBM to LDS (16-byte buffer loads in LDS DMA mode; rows past m or n
//    and bytes past k read as zero): three stages for the weights, which come
//    from HBM, two for the tokens, which the XCD's L2 holds, 160 KB at
//    256 x 256.  A stage is refilled as soon as its last fragments are in
//    registers.  (Steps of 64 bytes allow five stages, but such half-line rows
//    reach LDS at 58 GB/s per CU against 123: 264 us for the gated
//    2048 x 4096 x 2*14336.)
//  * A staged row is 128 bytes, its 16-byte chunk c at slot c ^ ((row/2) % 8):
//    the 16-byte fragment reads of 16 consecutive rows then fall on all 64
//    banks once, and the swizzle costs nothing (the DMA's LDS side is linear,
//    the lanes' global addresses carry it).
//  * The fragments of the next 32 bytes of k are read between the matrix
//    instructions of these, one read after each.
//  * Matrix operands: A = weight rows, B = tokens, so that a lane's results
//    are runs of 4 consecutive outputs of one token.
//  * Workgroups are dealt to the 8 XCDs round robin; each XCD takes a
//    contiguous run of tiles, up to 4 token tiles of one weight tile next to
//    each other, so that an XCD's L2 serves both operands' reuse.
//  * Large tiles where they fill the device, 128 x 128 ones elsewhere (rule and
//    figures: plan).
#include <type_traits>

#include "i8_device.h"
#include "q8_i8.h"

namespace q8 {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

constexpr int kStep = 128;        // bytes of k per step
constexpr int kGroupM = 4;        // token tiles next to each other (8, 16: 1 to 2% slower)
constexpr int kOut = 0x7ff00000;  // an offset past every resource: reads zero

// One tile: outputs n0 .. (TN of them, TN/2 gated), tokens m0 .. m0 + TM - 1.
// w0 .. x1: the stages, separate LDS objects, so that a fragment read waits for
// its own stage's loads only.  STREAM: outputs are written past the caches.  EPI:
// y = act(value) + residual.  KS 2: two groups of WN x WM waves take half of k each,
// in stages of their own (the second behind the first's), and join their sums.
template <int TN, int TM, int WN, int WM, int YT, bool GATED, bool STREAM, bool EPI, int KS = 1>
__device__ __forceinline__ void i8_tile(const I8Args &a, int64_t n0, int64_t m0, uint8_t *w0,
                                        uint8_t *w1, uint8_t *w2, uint8_t *x0, uint8_t *x1)
{
    constexpr int kWaves = WN * WM;
    constexpr int NI = TN / WN / 32, MI = TM / WM / 32;
    constexpr int kLoadsW = TN / 8 / kWaves, kLoadsX = TM / 8 / kWaves;
    constexpr int kCols = GATED ? TN / 2 : TN;          // outputs per tile
    constexpr int kWaveCols = kCols / WN;
    static_assert(TN % (8 * kWaves) == 0 && TM % (8 * kWaves) == 0, "whole loads per wave");
    static_assert(kWaves % 2 == 0, "the chunk of a lane is the same for every load");
    static_assert(!GATED || NI % 2 == 0, "gate and up halves");

    const int wave_all = wave_uniform((int)(threadIdx.x >> 6));
    const int part = KS == 1 ? 0 : wave_all / kWaves, wave = KS == 1 ? wave_all : wave_all % kWaves;
    const int lane = threadIdx.x & 63;
    const int wn = wave / WM, wm = wave % WM;
    const int h = lane >> 5, li = lane & 31;

    // operand rows of the tile; bytes k_begin .. k_begin + k - 1 of them
    const int k_first = KS == 1 ? (int)a.k : ((int)a.k / 2 + kStep - 1) / kStep * kStep;
    const int k_begin = part ? k_first : 0, k = part ? (int)a.k - k_first : k_first;
    if constexpr (KS > 1) {
        w0 += part * TN * kStep; w1 += part * TN * kStep; w2 += part * TN * kStep;
        x0 += part * TM * kStep; x1 += part * TM * kStep;
    }
    const int w_rows = (int)min((int64_t)kCols, a.n - n0), x_rows = (int)min((int64_t)TM, a.m - m0);
    const int w_stride = (int)a.w_stride, x_stride = (int)a.x_stride;
    const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(a.x + m0 * a.x_stride + k_begin), 0, (x_rows - 1) * x_stride + k, kBufferWord3);
    const int8_t *w_base[kLoadsW];     // (no array of resources: the host pass has no such type)
    int voff[kLoadsW + kLoadsX];
    // load u of a wave: staged rows 8f .. 8f+7, f = wave + kWaves * u
    const int lr = lane >> 3;
    const int chunk = (lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7);   // (8f + lr)/2 % 8
#pragma unroll
    for (int u = 0; u < kLoadsW; ++u) {
        const int b = 8 * (wave + kWaves * u);          // of TN; 32-row groups are uniform
        int row = b;
        const int8_t *base = a.w + n0 * a.w_stride + k_begin;
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

    auto issue_w = [&](int st, uint8_t *s) {
        const bool in_k = 16 * chunk < k - st * kStep;
        const int so = min(st * kStep, k);       // (kOut + so stays below 2^31)
#pragma unroll
        for (int u = 0; u < kLoadsW; ++u) {
            const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
                (void *)w_base[u], 0, (w_rows - 1) * w_stride + k, kBufferWord3);
            auto *dst = (__attribute__((address_space(3))) void *)(s + 1024 * (wave + kWaves * u));
            const int off = in_k ? voff[u] : kOut;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, dst, 16, off, so, 0, 0);
        }
    };
    auto issue_x = [&](int st, uint8_t *s) {
        const bool in_k = 16 * chunk < k - st * kStep;
        const int so = min(st * kStep, k);       // (kOut + so stays below 2^31)
#pragma unroll
        for (int u = 0; u < kLoadsX; ++u) {
            auto *dst = (__attribute__((address_space(3))) void *)(s + 1024 * (wave + kWaves * u));
            const int off = in_k ? voff[kLoadsW + u] : kOut;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, dst, 16, off, so, 0, 0);
        }
    };

    // what the outputs need: one weight row's scale and bias per thread, the
    // scales of the lane's tokens
    const int tid = KS == 1 ? (int)threadIdx.x : (int)threadIdx.x % (64 * kWaves);
    float w_scale = 0.0f, w_bias = 0.0f, s_x[MI];
    static_assert(TN <= 64 * kWaves, "a thread per weight row");
    if (tid < TN) {
        const int grp = tid / 32 % NI;
        const int64_t col = n0 + (!GATED ? tid
                                         : tid / (32 * NI) * kWaveCols +
                                               32 * (grp % (NI / 2 + !GATED)) + tid % 32);
        if (col < a.n) {
            w_scale = a.w_scale[GATED && grp >= NI / 2 ? a.n + col : col];
            if (!GATED && a.bias) w_bias = a.bias[col];
        }
    }
#pragma unroll
    for (int j = 0; j < MI; ++j)
        s_x[j] = a.x_scale[min(m0 + (wm * MI + j) * 32 + li, a.m - 1)];

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
    // 32 bytes of k (group ks of the step): lane = row li, bytes 16h .. 16h+15
    const int row_w = (wn * NI * 32 + li) * kStep, row_x = (wm * MI * 32 + li) * kStep;
    const int swz = (li >> 1) & 7;
    auto load = [&](const uint8_t *sw, const uint8_t *sx, int ks, Frag &f) {
        const int c = 16 * ((2 * ks + h) ^ swz);
#pragma unroll
        for (int i = 0; i < NI; ++i) f.w[i] = *(const v4i *)(sw + row_w + c + i * 32 * kStep);
#pragma unroll
        for (int j = 0; j < MI; ++j) f.x[j] = *(const v4i *)(sx + row_x + c + j * 32 * kStep);
    };
    auto mul = [&](const Frag &f) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < MI; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.w[i], f.x[j], acc[i][j], 0, 0, 0);
    };
    // the order of the instructions since the last mark: a fragment read after
    // each of the first matrix instructions
    auto interleave = [&]() {
        constexpr int kPairs = NI + MI;
        static_assert(kPairs <= NI * MI, "a matrix instruction for each read");
#pragma unroll
        for (int z = 0; z < kPairs; ++z) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        }
        if constexpr (NI * MI > kPairs) __builtin_amdgcn_sched_group_barrier(0x008, NI * MI - kPairs, 0);
        __builtin_amdgcn_sched_barrier(0);
    };
    // this wave's loads of the next stage have landed (but not the weights of the
    // one after it) and its reads of this one are done; then every wave's (a
    // __syncthreads would wait for all loads)
    auto next_stage = [&]() {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kLoadsW) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };

    const int steps = (k_first + kStep - 1) / kStep;     // (as many for either part: the barriers are shared)
    Frag f0, f1;
    issue_w(0, w0);
    issue_x(0, x0);
    issue_w(1, w1);
    issue_x(1, x1);
    issue_w(2, w2);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * kLoadsW + kLoadsX) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    load(w0, x0, 0, f0);
    // a step past the end loads zeros, so that every wait count is exact
    auto body = [&](int st, uint8_t *wc, const uint8_t *wnext, uint8_t *xc, const uint8_t *xnext) {
        load(wc, xc, 1, f1);
        mul(f0);
        interleave();
        load(wc, xc, 2, f0);
        mul(f1);
        interleave();
        load(wc, xc, 3, f1);
        mul(f0);
        interleave();
        next_stage();
        load(wnext, xnext, 0, f0);
        issue_x(st + 2, xc);
        issue_w(st + 3, wc);
        mul(f1);
        interleave();
    };
    int st = 0;
    for (; st + 6 <= steps; st += 6) {
        body(st, w0, w1, x0, x1);
        body(st + 1, w1, w2, x1, x0);
        body(st + 2, w2, w0, x0, x1);
        body(st + 3, w0, w1, x1, x0);
        body(st + 4, w1, w2, x0, x1);
        body(st + 5, w2, w0, x1, x0);
    }
    if (st < steps) body(st, w0, w1, x0, x1);
    if (st + 1 < steps) body(st + 1, w1, w2, x1, x0);
    if (st + 2 < steps) body(st + 2, w2, w0, x0, x1);
    if (st + 3 < steps) body(st + 3, w0, w1, x1, x0);
    if (st + 4 < steps) body(st + 4, w1, w2, x0, x1);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // (zeros still on their way to LDS)
    if constexpr (KS > 1) {
        static_assert(KS == 2 && kWaves == 2 && NI * MI * 4 * 1024 <= TN * kStep, "a stage of the second part per wave");
        __syncthreads();
        const int over = part ? 0 : TN * kStep;        // the second part's stages
        v4i *sums = (v4i *)((wave ? w1 : w0) + over);
        if (part)
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int j = 0; j < MI; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        sums[((i * MI + j) * 4 + q) * 64 + lane] = (v4i){acc[i][j][4 * q], acc[i][j][4 * q + 1],
                                                                        acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        __syncthreads();
        if (!part)
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int j = 0; j < MI; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const v4i s = sums[((i * MI + j) * 4 + q) * 64 + lane];
                        acc[i][j][4 * q] += s.x;
                        acc[i][j][4 * q + 1] += s.y;
                        acc[i][j][4 * q + 2] += s.z;
                        acc[i][j][4 * q + 3] += s.w;
                    }
    }

    // Outputs.  Result r of a lane: weight row 8(r/4) + 4h + r%4 of its tile,
    // token li.  The tile's scales (and bias) go to LDS, and every wave turns its
    // results round there, 32 tokens x 128 bytes at a time (swizzled as above), so
    // that a token's outputs leave as runs of 16-byte stores.
    __syncthreads();                           // every wave is done with the stages
    float *scales = (float *)w2;               // [TN], then bias [TN]
    if (tid < TN) {
        scales[tid] = w_scale;
        if (!GATED) scales[TN + tid] = w_bias;
    }
    __syncthreads();
    if (KS > 1 && part) return;
    constexpr int kES = YT == Q8_T_F32 ? 4 : 2;
    constexpr int kOutTiles = GATED ? NI / 2 : NI;
    constexpr int kPass = kOutTiles < 4 / kES ? kOutTiles : 4 / kES;    // tiles side by side
    constexpr int kChunks = kPass * 32 * kES / 16;                      // 16-byte pieces a row
    constexpr int kPerX = TM * kStep / 4096, kPerW = TN * kStep / 4096; // waves per stage
    static_assert(kWaves <= 2 * kPerX + kPerW && 2 * 4 <= kStep, "fits");
    uint8_t *turn = wave < kPerX ? x0 + wave * 4096
                    : wave < 2 * kPerX ? x1 + (wave - kPerX) * 4096 : w0 + (wave - 2 * kPerX) * 4096;
    // a lane's place in the wave's outputs: row o_row (+ 64 / kChunks per store),
    // 16 bytes from column o_col on
    const int o_row = lane / kChunks, o_col = lane % kChunks * (16 / kES);
    const int rows_left = x_rows - wm * MI * 32 - o_row, cols_left = w_rows - wn * kWaveCols - o_col;
    const int64_t y_bytes = a.y_stride * kES;
    uint8_t *y = (uint8_t *)a.y + (m0 + wm * MI * 32 + o_row) * y_bytes + (n0 + wn * kWaveCols + o_col) * kES;
    auto outputs = [&](auto with_bias) {
        constexpr bool biased = decltype(with_bias)::value;
#pragma unroll
        for (int j = 0; j < MI; ++j) {
#pragma unroll
            for (int i0 = 0; i0 < kOutTiles; i0 += kPass) {
#pragma unroll
                for (int ip = 0; ip < kPass; ++ip)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int i = i0 + ip, row = (wn * NI + i) * 32 + 8 * q + 4 * h;
                        const float4 sg = *(const float4 *)(scales + row);
                        float4 su = sg, sb = sg;
                        if (GATED) su = *(const float4 *)(scales + row + NI / 2 * 32);
                        if (!GATED) sb = *(const float4 *)(scales + TN + row);
                        const float g4[4] = {sg.x, sg.y, sg.z, sg.w}, u4[4] = {su.x, su.y, su.z, su.w},
                                    b4[4] = {sb.x, sb.y, sb.z, sb.w};
                        float v[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int s = acc[i][j][4 * q + r];
                            if (GATED)
                                v[r] = silu_mul(
                                    i8_rescale(s, s_x[j], g4[r]),
                                    i8_rescale(acc[GATED ? i + NI / 2 : i][j][4 * q + r], s_x[j], u4[r]));
                            else
                                v[r] = biased ? i8_rescale(s, s_x[j], g4[r], b4[r])
                                              : i8_rescale(s, s_x[j], g4[r]);
                        }
                        if (YT == Q8_T_F32)
                            *(float4 *)(turn + li * 128 + 16 * ((2 * q + h) ^ ((li >> 1) & 7))) =
                                make_float4(v[0], v[1], v[2], v[3]);
                        else
                            *(u32x2 *)(turn + li * 128 + 16 * ((4 * ip + q) ^ ((li >> 1) & 7)) + 8 * h) =
                                (u32x2){pack2<YT>(v[0], v[1]), pack2<YT>(v[2], v[3])};
                    }
                wave_lds_sync();
#pragma unroll
                for (int e = 0; e < kChunks / 2; ++e) {
                    const int up = e * (64 / kChunks), row = up + o_row, c = lane % kChunks;
                    const u32x4 o = *(const u32x4 *)(turn + row * 128 + 16 * (c ^ ((row >> 1) & 7)));
                    if (32 * j + up < rows_left && 32 * i0 < cols_left)
                        store16<YT, STREAM>(y + (32 * j + up) * y_bytes + 32 * i0 * kES, o,
                                            cols_left - 32 * i0);
                }
                wave_lds_sync();
            }
        }
    };
    if constexpr (EPI) {
        // fp32 values through LDS 32 columns at a time: the residual is added, and
        // the sum rounded, where a lane holds 16 bytes of outputs
        constexpr int V = 16 / kES, kRow = 32 / V, kTurns = 32 * kRow / 64;   // 16-byte pieces a row
        const int e_row = lane / kRow, e_col = lane % kRow * V;
        const int e_rows = x_rows - wm * MI * 32 - e_row, e_cols = w_rows - wn * kWaveCols - e_col;
        uint8_t *ye = (uint8_t *)a.y + (m0 + wm * MI * 32 + e_row) * y_bytes + (n0 + wn * kWaveCols + e_col) * kES;
        const int64_t r_bytes = a.r_stride * kES;
        const uint8_t *re = (const uint8_t *)a.residual + (m0 + wm * MI * 32 + e_row) * r_bytes +
                            (n0 + wn * kWaveCols + e_col) * kES;
#pragma unroll
        for (int j = 0; j < MI; ++j) {
#pragma unroll
            for (int i = 0; i < kOutTiles; ++i) {
                u32x4 res[kTurns];
#pragma unroll
                for (int e = 0; e < kTurns; ++e) {
                    const int up = e * (64 / kRow);
                    res[e] = (u32x4){0u, 0u, 0u, 0u};
                    if (a.residual && 32 * j + up < e_rows && 32 * i < e_cols)
                        res[e] = load16<YT>(re + (32 * j + up) * r_bytes + 32 * i * kES, e_cols - 32 * i);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int row = (wn * NI + i) * 32 + 8 * q + 4 * h;
                    const float4 sg = *(const float4 *)(scales + row), sb = *(const float4 *)(scales + TN + row);
                    const float g4[4] = {sg.x, sg.y, sg.z, sg.w}, b4[4] = {sb.x, sb.y, sb.z, sb.w};
                    float v[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int s = acc[i][j][4 * q + r];
                        v[r] = a.bias ? i8_rescale(s, s_x[j], g4[r], b4[r]) : i8_rescale(s, s_x[j], g4[r]);
                    }
                    *(float4 *)(turn + li * 128 + 16 * ((2 * q + h) ^ ((li >> 1) & 7))) =
                        make_float4(v[0], v[1], v[2], v[3]);
                }
                // (by a loop over what the lane has just written: the activations' code
                // 16 times in each turn would keep these loops from being unrolled, and
                // the sums, then indexed by variables, in memory)
                if (a.act != Q8_ACT_NONE)
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        float4 *o = (float4 *)(turn + li * 128 + 16 * ((2 * q + h) ^ ((li >> 1) & 7)));
                        float v[4] = {o->x, o->y, o->z, o->w};
                        activate_run<4>(a.act, v);
                        *o = make_float4(v[0], v[1], v[2], v[3]);
                    }
                wave_lds_sync();
#pragma unroll
                for (int e = 0; e < kTurns; ++e) {
                    const int up = e * (64 / kRow), row = up + e_row;
                    float v[V], r[V];
#pragma unroll
                    for (int c = 0; c < V / 4; ++c) {
                        const float4 o = *(const float4 *)(turn + row * 128 + 16 * ((e_col / 4 + c) ^ ((row >> 1) & 7)));
                        v[4 * c] = o.x; v[4 * c + 1] = o.y; v[4 * c + 2] = o.z; v[4 * c + 3] = o.w;
                    }
                    if (a.residual) {
                        unpack16<YT>(res[e], r);
#pragma unroll
                        for (int c = 0; c < V; ++c) v[c] += r[c];
                    }
                    if (32 * j + up < e_rows && 32 * i < e_cols)
                        store16<YT, STREAM>(ye + (32 * j + up) * y_bytes + 32 * i * kES, pack_vec<YT>(v),
                                            e_cols - 32 * i);
                }
                wave_lds_sync();
            }
        }
    } else if (!GATED && a.bias)
        outputs(std::integral_constant<bool, !GATED>());
    else
        outputs(std::integral_constant<bool, false>());
}

// Tiles in work order: up to kGroupM token tiles of one weight tile next to
// each other.
struct TileGrid {
    int tiles_n, tiles_m;
    int whole;                   // LARGE: tiles computed whole, the others in two halves

    __device__ __forceinline__ void at(int work, int &tn, int &tm) const
    {
        const int group = work / (kGroupM * tiles_n);
        const int gm = min(kGroupM, tiles_m - group * kGroupM);
        const int in = work - group * kGroupM * tiles_n;
        tn = in / gm;
        tm = group * kGroupM + in % gm;
    }
};

// Item b of n, dealt round robin to the 8 XCDs, as a run of items per XCD.
__device__ __forceinline__ int xcd_run(int b, int n)
{
    const int xcd = b & 7, per = n >> 3, rest = n & 7;
    return xcd * per + min(xcd, rest) + (b >> 3);
}

// 256 x 256, one workgroup of 8 waves per CU: 2.5 POPS where all CUs have work.
// The last tiles, where they would occupy half of the CUs or fewer, are
// computed as halves of 128 tokens, on twice as many CUs.
template <int YT, bool GATED, bool STREAM, bool EPI>
__global__ __launch_bounds__(512, 2) void i8_large_kernel(const I8Args a, const TileGrid g)
{
    __shared__ __align__(16) uint8_t w0[256 * kStep];
    __shared__ __align__(16) uint8_t w1[256 * kStep];
    __shared__ __align__(16) uint8_t w2[256 * kStep];
    __shared__ __align__(16) uint8_t x0[256 * kStep];
    __shared__ __align__(16) uint8_t x1[256 * kStep];
    constexpr int kCols = GATED ? 128 : 256;
    const int b = blockIdx.x;
    int tn, tm;
    if (b < g.whole) {
        g.at(xcd_run(b, g.whole), tn, tm);
        i8_tile<256, 256, 4, 2, YT, GATED, STREAM, EPI>(a, (int64_t)tn * kCols, (int64_t)tm * 256, w0,
                                                        w1, w2, x0, x1);
    } else {
        const int half = xcd_run(b - g.whole, 2 * (g.tiles_n * g.tiles_m - g.whole));
        g.at(g.whole + half / 2, tn, tm);
        const int64_t m0 = (int64_t)tm * 256 + 128 * (half & 1);
        if (m0 < a.m)
            i8_tile<256, 128, 4, 2, YT, GATED, STREAM, EPI>(a, (int64_t)tn * kCols, m0, w0, w1, w2, x0, x1);
    }
}

// 128 x 128, two workgroups of 4 waves per CU.
template <int YT, bool GATED, bool STREAM, bool EPI>
__global__ __launch_bounds__(256, 2) void i8_medium_kernel(const I8Args a, const TileGrid g)
{
    __shared__ __align__(16) uint8_t w0[128 * kStep];
    __shared__ __align__(16) uint8_t w1[128 * kStep];
    __shared__ __align__(16) uint8_t w2[128 * kStep];
    __shared__ __align__(16) uint8_t x0[128 * kStep];
    __shared__ __align__(16) uint8_t x1[128 * kStep];
    int tn, tm;
    g.at(xcd_run(blockIdx.x, g.tiles_n * g.tiles_m), tn, tm);
    i8_tile<128, 128, 2, 2, YT, GATED, STREAM, EPI>(a, (int64_t)tn * (GATED ? 64 : 128), (int64_t)tm * 128,
                                               w0, w1, w2, x0, x1);
}

// 128 x 64 by two pairs of waves, each over half of k, with an epilogue only: for
// products with few outputs and a long k, whose tiles of 128 x 128 would leave half
// of the CUs without one and are bound by the round trip of each of their steps.
template <int YT, bool STREAM>
__global__ __launch_bounds__(256) void i8_narrow_kernel(const I8Args a, const TileGrid g)
{
    __shared__ __align__(16) uint8_t w0[2 * 128 * kStep];
    __shared__ __align__(16) uint8_t w1[2 * 128 * kStep];
    __shared__ __align__(16) uint8_t w2[2 * 128 * kStep];
    __shared__ __align__(16) uint8_t x0[2 * 64 * kStep];
    __shared__ __align__(16) uint8_t x1[2 * 64 * kStep];
    int tn, tm;
    g.at(xcd_run(blockIdx.x, g.tiles_n * g.tiles_m), tn, tm);
    i8_tile<128, 64, 2, 1, YT, false, STREAM, true, 2>(a, (int64_t)tn * 128, (int64_t)tm * 64, w0, w1, w2, x0, x1);
}

TileGrid tile_grid(const I8Args &a, bool gated, int tile)
{
    const int64_t cols = gated ? tile / 2 : tile;
    const int64_t tn = (a.n + cols - 1) / cols, tm = (a.m + tile - 1) / tile;
    // (2^36 outputs are fewer than 2^24 tiles, and those below 2^32 threads)
    if (tn * tm >= ((int64_t)1 << 24)) return {0, 0, 0};
    return {(int)tn, (int)tm, (int)(tn * tm)};
}

// The tiles of a product: large ones (large.whole of them whole), or medium
// ones, or none (more than a launch takes).
struct Plan {
    bool large;
    TileGrid grid;
};

Plan plan(const I8Args &a, bool gated)
{
    TileGrid large = tile_grid(a, gated, 256);
    const TileGrid medium = tile_grid(a, gated, 128);
    const int tiles = large.tiles_n * large.tiles_m, mtiles = medium.tiles_n * medium.tiles_m;
    if (!mtiles) return {false, medium};
    // Rounds of the device's 256 CUs at the times of one round, in us at
    // k = 4096: 56 for 256 tiles of 256 x 256, 36 for 256 halves, 37 for 512
    // tiles of 128 x 128, 25 for 256 of them.  (Full rounds: one that is half
    // full is quicker, 128 tiles of 128 x 128 take 19 us at k = 4096 and 15 to 19
    // per 4096 at k = 14336, which the rule does not know.)
    const int rest = tiles % 256;
    const int cost_large = tiles / 256 * 56 + (rest == 0 ? 0 : rest <= 128 ? 36 : 56);
    const int cost_medium = mtiles <= 256 ? 25 : (mtiles + 511) / 512 * 37;
    if (cost_large > cost_medium) return {false, medium};
    if (rest <= 128) large.whole -= rest;
    return {true, large};
}

// Whether a product with an epilogue goes to the narrow kernel.  512 x k x 4096 on
// tiles of 128 x 128 and on halves of k, us: k = 14336 54.1 and 40.8, 4096 18.6 and 16.7,
// 2048 11.7 and 10.1, 1536 9.8 and 9.0, 1024 8.6 and 8.5, 768 7.9 and 8.1; 300 x 256 x 4096
// 6.3 and 6.7.
bool halves_of_k(const I8Args &a, const Plan &p)
{
    return a.epilogue && !p.large && p.grid.tiles_n * p.grid.tiles_m <= 128 && a.k >= 1024;
}

template <int YT, bool GATED, bool STREAM, bool EPI>
int launch_form(const I8Args &a, hipStream_t stream)
{
    const Plan p = plan(a, GATED);
    const int tiles = p.grid.tiles_n * p.grid.tiles_m;
    if (!tiles) return Q8_E_UNSUPPORTED;
    if constexpr (EPI)
        if (halves_of_k(a, p)) {
            const TileGrid g = {p.grid.tiles_n, (int)((a.m + 63) / 64), 0};
            hipLaunchKernelGGL((i8_narrow_kernel<YT, STREAM>), dim3((unsigned)(g.tiles_n * g.tiles_m)), dim3(256), 0,
                               stream, a, g);
            return hipGetLastError() == hipSuccess ? 0 : -6;
        }
    if (p.large)
        hipLaunchKernelGGL((i8_large_kernel<YT, GATED, STREAM, EPI>), dim3((unsigned)(2 * tiles - p.grid.whole)),
                           dim3(512), 0, stream, a, p.grid);
    else
        hipLaunchKernelGGL((i8_medium_kernel<YT, GATED, STREAM, EPI>), dim3((unsigned)tiles), dim3(256), 0, stream,
                           a, p.grid);
    return hipGetLastError() == hipSuccess ? 0 : -6;
}

// 16-bit rows that start on cache lines are written past the caches (gated 2048 x
// 4096 x 2*14336: 211 against 216 us, 384 x 768 x 50176: 25 and 36 us); other
// rows would leave parts of lines (333 x 768 x 50257: 28 against 26 us in
// binary16, 57 against 38 in fp32), and fp32 gains nothing (233 against 239 us
// without at 4096 x 8192 x 8192).
template <int YT>
int launch_type(const I8Args &a, bool gated, hipStream_t stream)
{
    if constexpr (YT != Q8_T_F32)
        if (a.y_stride * 2 % 128 == 0 && (uintptr_t)a.y % 128 == 0)
            return gated        ? launch_form<YT, true, true, false>(a, stream)
                   : a.epilogue ? launch_form<YT, false, true, true>(a, stream)
                                : launch_form<YT, false, true, false>(a, stream);
    return gated        ? launch_form<YT, true, false, false>(a, stream)
           : a.epilogue ? launch_form<YT, false, false, true>(a, stream)
                        : launch_form<YT, false, false, false>(a, stream);
}

}  // namespace

int i8_gemm_form(const I8Args &a, bool gated)
{
    const Plan p = plan(a, gated);
    const int tiles = p.grid.tiles_n * p.grid.tiles_m;
    if (halves_of_k(a, p)) return Q8V_I8_TILES_K_HALVES;
    if (!p.large) return Q8V_I8_TILES_128;
    return p.grid.whole == tiles ? Q8V_I8_TILES_256 : p.grid.whole ? Q8V_I8_TILES_256_SOME_HALVES
                                                                   : Q8V_I8_TILES_256_HALVES;
}

int launch_i8_gemm(const I8Args &a, bool gated, hipStream_t stream)
{
    if (a.y_type == Q8_T_F32) return launch_type<Q8_T_F32>(a, gated, stream);
    if (a.y_type == Q8_T_F16) return launch_type<Q8_T_F16>(a, gated, stream);
    return launch_type<Q8_T_BF16>(a, gated, stream);
}

}  // namespace q8
