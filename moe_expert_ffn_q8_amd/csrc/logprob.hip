// logprob.hip -- log probabilities of given tokens, log sum exp, entropy and the
// largest logits of each row, in one pass over the logits.
//
// A workgroup takes a row, or a part of one where there are few rows; the parts
// are joined by a second launch.  Every lane keeps a running (reference r, S =
// sum 2^(x L - r L), W = sum 2^(x L - r L) (x L - r L)), L = log2 e, over 16-byte
// loads, four in flight; per logit that is a fused multiply-add, an exponential,
// two sums and a comparison.
//
// The largest n_top logits: every wave keeps candidates of its own, (value,
// lowest index first) as one 64-bit key, in LDS, and the key that a logit has to
// pass.  After turns 1, 2, 4, 8, ... the workgroup sets a common bound: the
// n_top-th largest of the maxima so far of 64 or 256 groups of its lanes, which
// n_top logits reach and few more, so few logits ever get in.  When a wave's
// 128 places are full, each candidate counts the larger ones (its rank) and the
// first n_top stay.  Most 16-byte groups are dismissed by their maximum, which
// the sums need anyway.
//
// Bounds: HBM for long rows without a list (512 x 262144 bfloat16 42 us, 6.4
// TB/s).  With one, 7 vector instructions per logit and 900 per wave for a list of
// 20 keep the vector pipe busy half of the time; what the other half waits for
// (the bound's barriers, exponentials, loads) was not separated (1021 x 50257
// bfloat16 24 to 25 us, 4.2 TB/s; 21 us without the list).  For few rows the chain
// of launch, loads and joins (1 x 32000 8 us).
#include <type_traits>

#include "i8_device.h"
#include "q8_i8.h"

namespace q8 {

namespace {

constexpr float kL2E = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
constexpr int kPlaces = 128;      // candidates per wave
constexpr int kMaxParts = 64;
constexpr int kShortTop = 24;     // alternatives of a short list
constexpr int kLoads = 4;         // 16-byte loads per lane and turn

// r: the largest logit seen, kLow at least.  The terms are formed beside the
// rounded product r L, which up to |r| = 2^24 is within 1 of r L, so that S counts
// each largest logit as 1/2 to 2; the rounding grows with r, and beside a
// reference of -2.5e9 (a mask of -1e9 over a temperature of 0.4) the terms would be
// 2^110 and W overflow.  A mask below kLow adds nothing, and a row whose maximum
// is not between kLow and -kLow is left to slow_stat.
constexpr float kLow = -0x1p24f;

struct Stat {
    float r, s, w;
};

__device__ __forceinline__ Stat stat_zero() { return {kLow, 0.0f, 0.0f}; }

// Both references as the rounded products that the terms were formed with (a
// fused multiply-add would put the rounding of r L into every move).
__device__ __forceinline__ void stat_move(Stat &a, float r)
{
    float d;
    {
#pragma clang fp contract(off)
        const float old2 = a.r * kL2E, new2 = r * kL2E;
        d = old2 - new2;
    }
    d = fmaxf(d, -1e30f);
    const float f = __builtin_amdgcn_exp2f(d);
    a.w = fmaf(a.s, d, a.w) * f;
    a.s *= f;
    a.r = r;
}

// One term; r2 = the reference's product, a.r the reference.  LOW: x may be so
// low that d is -infinity; else that makes w a NaN (0 * infinity).
template <bool LOW>
__device__ __forceinline__ void stat_add(Stat &a, float x, float r2)
{
    const float d = fmaf(x, kL2E, -r2);
    const float e = __builtin_amdgcn_exp2f(d);
    a.s += e;
    a.w = fmaf(e, LOW ? fmaxf(d, -1e30f) : d, a.w);
}

// A reduction over the wave's lanes by data-parallel-primitive moves (in rows
// of 16, then across them), the result in every lane.
template <int Ctrl, int RowMask>
__device__ __forceinline__ float dpp(float id, float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
        __builtin_bit_cast(int, id), __builtin_bit_cast(int, v), Ctrl, RowMask, 0xf, false));
}

template <bool MAX>
__device__ __forceinline__ float wave_reduce(float v)
{
    const float id = MAX ? -INFINITY : 0.0f;
    auto op = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
    v = op(v, dpp<0x111, 0xf>(id, v));         // row_shr:1
    v = op(v, dpp<0x112, 0xf>(id, v));         // row_shr:2
    v = op(v, dpp<0x114, 0xf>(id, v));         // row_shr:4
    v = op(v, dpp<0x118, 0xf>(id, v));         // row_shr:8
    v = op(v, dpp<0x142, 0xa>(id, v));         // row_bcast:15
    v = op(v, dpp<0x143, 0xc>(id, v));         // row_bcast:31
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

__device__ __forceinline__ Stat wave_join(Stat st)
{
    stat_move(st, wave_reduce<true>(st.r));
    return {st.r, wave_reduce<false>(st.s), wave_reduce<false>(st.w)};
}

// Order of the top list: larger value first, then lower index; NaN last.  No
// key of a logit is 0.
__device__ __forceinline__ uint32_t value_key(float x)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);       // -0 -> +0
    const uint32_t key = (u >> 31) ? ~u : (u | 0x80000000u);
    return x != x ? 0u : key;
}

__device__ __forceinline__ uint64_t order_key(float x, uint32_t i)
{
    return ((uint64_t)value_key(x) << 32) | (uint32_t)~i;
}

__device__ __forceinline__ float key_value(uint64_t key)
{
    const uint32_t k = (uint32_t)(key >> 32);
    if (k == 0) return __builtin_nanf("");
    return __builtin_bit_cast(float, (k >> 31) ? (k & 0x7fffffffu) : ~k);
}

__device__ __forceinline__ int key_index(uint64_t key) { return (int)~(uint32_t)key; }

// Moves within rows of 16 lanes.
template <int Ctrl>
__device__ __forceinline__ uint32_t row_move(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, Ctrl, 0xf, 0xf, false);
}

// The n-th largest of 64 keys, one per lane, its low half cut (0: fewer than n
// keys are not 0).
__device__ __forceinline__ uint32_t nth_key(uint32_t key, int n)
{
    uint32_t t = 0;
    for (int b = 31; b >= 16; --b) {
        const uint32_t c = t | (1u << b);
        if (__popcll(__ballot(key >= c)) >= n) t = c;
    }
    return t;
}

// The same of 256 keys, four per lane.
__device__ __forceinline__ uint32_t nth_key(u32x4 key, int n)
{
    uint32_t t = 0;
    for (int b = 31; b >= 16; --b) {
        const uint32_t c = t | (1u << b);
        if (__popcll(__ballot(key.x >= c)) + __popcll(__ballot(key.y >= c)) +
                __popcll(__ballot(key.z >= c)) + __popcll(__ballot(key.w >= c)) >= n)
            t = c;
    }
    return t;
}

// f(rank, key) for the first n of `count` different keys in LDS (0: none), by
// a whole workgroup: eight lanes count the larger ones of each, two at a time
// (what lies behind the last key, of an even number of places, is not counted).
template <class F>
__device__ __forceinline__ void by_rank(const uint64_t *keys, int count, int n, int threads, F f)
{
    const int sub = threadIdx.x & 7;
    for (int c0 = 0; c0 < count; c0 += threads / 8) {
        const int c = c0 + (threadIdx.x >> 3);
        const uint64_t k = c < count ? keys[c] : 0;
        int rank = 0;
#pragma unroll 4
        for (int j = 2 * sub; j < count; j += 16) {
            const ulonglong2 o = *(const ulonglong2 *)(keys + j);
            rank += o.x > k;
            rank += j + 1 < count && o.y > k;
        }
        rank += (int)row_move<0xb1>((uint32_t)rank);     // quad_perm:[1,0,3,2]
        rank += (int)row_move<0x4e>((uint32_t)rank);     // quad_perm:[2,3,0,1]
        rank += (int)row_move<0x141>((uint32_t)rank);    // row_half_mirror
        if (sub == 0 && k != 0 && rank < n) f(rank, k);
    }
}

// One wave's candidates.  thr: what a key has to exceed; least: a value below
// which no logit can (-infinity: all have to be looked at).
struct Top {
    uint64_t *place;              // [kPlaces]
    uint64_t thr;
    float least;
    int count, n;

    __device__ __forceinline__ void init(uint64_t *p, int n_top)
    {
        place = p;
        n = n_top;
        count = 0;
        set(0);
    }
    __device__ __forceinline__ void set(uint64_t t)
    {
        thr = t;
        least = (t >> 32) > 0x007fffffu ? key_value(t) : -INFINITY;
    }
    // Ranks; the first n stay, in order.
    __device__ __forceinline__ void compact(int lane)
    {
        if (lane < 8 && count + lane < kPlaces) place[count + lane] = 0;     // read by eights
        wave_lds_sync();
        const uint64_t k0 = lane < count ? place[lane] : 0;
        const uint64_t k1 = 64 + lane < count ? place[64 + lane] : 0;
        int r0 = 0, r1 = 0;
        for (int i = 0; i < count; i += 8)
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const ulonglong2 o = *(const ulonglong2 *)(place + i + j);
                r0 += (o.x > k0) + (o.y > k0);
                r1 += (o.x > k1) + (o.y > k1);
            }
        wave_lds_sync();
        if (lane < count && r0 < n) place[r0] = k0;
        if (64 + lane < count && r1 < n) place[r1] = k1;
        wave_lds_sync();
        if (count >= n) {
            count = n;
            const uint64_t t = place[n - 1];
            set(((uint64_t)(uint32_t)wave_uniform((int)(t >> 32)) << 32) |
                (uint32_t)wave_uniform((int)(uint32_t)t));
        }
    }
    // One logit per lane (all lanes of the wave call).
    __device__ __forceinline__ void offer(float x, uint32_t i, bool real, int lane)
    {
        const uint64_t key = order_key(x, i);
        uint64_t in = __ballot(real && key > thr);
        if (!in) return;
        if (count + __popcll(in) > kPlaces) {
            compact(lane);
            in = __ballot(real && key > thr);
        }
        if (in >> lane & 1)
            place[count + __builtin_amdgcn_mbcnt_hi((uint32_t)(in >> 32),
                                                    __builtin_amdgcn_mbcnt_lo((uint32_t)in, 0))] = key;
        count += __popcll(in);
    }
};

// Vectors with a logit that may get in, of one wave: a lane per logit looks at
// them when there are 64 logits together.
constexpr int kPend = 64 + 16;
template <int T>
struct Pending {
    static constexpr int V = kVec<T>, kBatch = 64 / V;
    u32x4 *vec;                   // [kPend]
    int *at;
    int count;

    __device__ __forceinline__ void init(u32x4 *v, int *i)
    {
        vec = v;
        at = i;
        count = 0;
    }
    // vectors count .. count + n - 1, n <= kBatch
    __device__ __forceinline__ void look(int n, int begin, Top &top, int lane) const
    {
        typedef typename Elem<T>::type E;
        const int p = count + lane / V, j = lane % V;
        const bool real = lane / V < n;
        const float x = real ? (float)((const E *)(vec + p))[j] : -INFINITY;
        top.offer(x, (uint32_t)(begin + (real ? at[p] : 0) * V + j), real, lane);
    }
    __device__ __forceinline__ void push(uint64_t in, u32x4 raw, int v, int begin, Top &top, int lane)
    {
        if (in >> lane & 1) {
            const int p = count + __builtin_amdgcn_mbcnt_hi((uint32_t)(in >> 32),
                                                            __builtin_amdgcn_mbcnt_lo((uint32_t)in, 0));
            vec[p] = raw;
            at[p] = v;
        }
        count += __popcll(in);
        wave_lds_sync();
        while (count >= kBatch) {
            count -= kBatch;
            look(kBatch, begin, top, lane);
        }
        wave_lds_sync();
    }
    __device__ __forceinline__ void flush(int begin, Top &top, int lane)
    {
        const int n = count;
        count = 0;
        if (n) look(n, begin, top, lane);
    }
};

struct Work {
    Stat *stats;                  // [m][parts]
    uint64_t *tops;               // [m][parts][n_top], 0 where a part has fewer
    int parts;
    int part_len;                 // logits, a multiple of 8
};

template <int T>
__device__ __forceinline__ float logit(const LogprobArgs &a, int64_t row, int64_t i)
{
    return (float)((const typename Elem<T>::type *)a.logits)[row * a.row_stride + i];
}

// The 16 bytes that unpack16 took the values from.
template <int T>
__device__ __forceinline__ u32x4 repack16(const float (&v)[kVec<T>])
{
    uint32_t d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (T == Q8_T_F32)
            d[i] = __builtin_bit_cast(uint32_t, v[i]);
        else if constexpr (T == Q8_T_F16)
            d[i] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v[2 * i]) |
                   (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v[2 * i + 1]) << 16;
        else
            d[i] = __builtin_bit_cast(uint32_t, v[2 * i]) >> 16 |
                   (__builtin_bit_cast(uint32_t, v[2 * i + 1]) & 0xffff0000u);
    }
    return (u32x4){d[0], d[1], d[2], d[3]};
}

// Values joined to (r, S, W) as differences from the largest, r = -infinity at
// first; bad counts NaN and +infinity.
__device__ __forceinline__ void slow_move(Stat &st, float r)       // r >= st.r
{
    const float d = r > st.r ? fmaxf((st.r - r) * kL2E, -1e30f) : 0.0f;
    const float f = __builtin_amdgcn_exp2f(d);
    st = {r, st.s * f, fmaf(st.s, d, st.w) * f};
}

template <int N>
__device__ __forceinline__ void slow_add(Stat &st, float &bad, const float (&x)[N])
{
    float r = st.r;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        bad += x[j] != x[j] || x[j] == INFINITY ? 1.0f : 0.0f;
        r = fmaxf(r, x[j]);
    }
    if (r == -INFINITY) return;
    slow_move(st, r);
    float s = 0.0f, w = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float d = fmaxf((x[j] - r) * kL2E, -1e30f);
        const float e = __builtin_amdgcn_exp2f(d);
        s += e;
        w = fmaf(e, d, w);
    }
    st.s += s;
    st.w += w;
}

// (r, S, W) of a whole row by one workgroup without the products x L, for the
// rows where those are too coarse or nothing is finite: a maximum of 2^24 or
// more, of either sign (masks throughout among them), -infinity throughout, NaN,
// +infinity.  r is then the row's maximum, S = 0 only if it is -infinity.  (Four
// such rows among 512 x 262144 bfloat16: 41 -> 68 us.)
template <int T>
__device__ Stat slow_stat(const LogprobArgs &a, int64_t row, Stat *part, int waves)
{
    typedef typename Elem<T>::type E;
    constexpr int V = kVec<T>;
    const int tid = threadIdx.x, n = 64 * waves;
    Stat st = {-INFINITY, 0.0f, 0.0f};
    float bad = 0.0f;
    // (vectors and the logits beside them as in logprob_kernel)
    const E *x0 = (const E *)a.logits + row * a.row_stride;
    const int len = (int)a.n_vocab;
    const int head = min((int)((-(uintptr_t)x0 & 15) / sizeof(E)), len);
    const int vecs = (len - head) / V, tail = len - head - vecs * V;
    const u32x4 *xv = (const u32x4 *)(x0 + head);
    for (int v = tid; v < vecs; v += kLoads * n) {
        u32x4 raw[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) raw[u] = xv[min(v + u * n, vecs - 1)];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            float x[V];
            unpack16<T>(raw[u], x);
            if (v + u * n < vecs) slow_add(st, bad, x);
        }
    }
    if (tid < head + tail) {
        const float x[1] = {(float)x0[tid < head ? tid : tid + vecs * V]};
        slow_add(st, bad, x);
    }
    float r = st.r;
    for (int d = 32; d; d >>= 1) {
        r = fmaxf(r, __shfl_xor(r, d));
        bad += __shfl_xor(bad, d);
    }
    __syncthreads();                                 // (`part` has been read)
    if ((tid & 63) == 0) part[tid >> 6] = {r, bad, 0.0f};
    __syncthreads();
    bad = 0.0f;
    for (int w = 0; w < waves; ++w) {
        r = fmaxf(r, part[w].r);
        bad += part[w].s;
    }
    __syncthreads();
    if (bad > 0.0f) return {r, __builtin_nanf(""), 0.0f};
    if (r == -INFINITY) return {r, 0.0f, 0.0f};
    slow_move(st, r);
    for (int d = 32; d; d >>= 1) {
        st.s += __shfl_xor(st.s, d);
        st.w += __shfl_xor(st.w, d);
    }
    if ((tid & 63) == 0) part[tid >> 6] = st;
    __syncthreads();
    st = {r, 0.0f, 0.0f};
    for (int w = 0; w < waves; ++w) {
        st.s += part[w].s;
        st.w += part[w].w;
    }
    return st;
}

// The given token that a thread writes, read before it is needed.
struct Given {
    int token;
    float x;
};

template <int T>
__device__ __forceinline__ Given given(const LogprobArgs &a, int64_t row, int i)
{
    Given g = {-1, 0.0f};
    if (i < a.n_given) {
        g.token = a.tokens[row * a.n_given + i];
        if (g.token >= 0 && g.token < a.n_vocab) g.x = logit<T>(a, row, g.token);
    }
    return g;
}

// Outputs of a row from its (r, S, W), the same in every thread; `tops` are
// `count` candidates in LDS, n_top of them the answer; g: token threadIdx.x.
template <int T>
__device__ __forceinline__ void finish(const LogprobArgs &a, int64_t row, Stat st, Stat *part,
                                       int waves, const uint64_t *tops, int count, Given g)
{
    const int tid = threadIdx.x, threads = 64 * waves;
    float shift = 0.0f;                          // r L as rounded, minus r L
    if (st.r > kLow && st.r < -kLow && st.s > 0.0f)    // (not with a NaN)
        shift = fmaf(-st.r, kL2E, st.r * kL2E);
    else
        st = slow_stat<T>(a, row, part, waves);
    const bool empty = st.s == 0.0f;
    const float l2 = log2f(st.s);
    // (the roundings of a row with one likely token leave neither log sum exp
    // below its logit nor the entropy below 0; NaN stays)
    float lse = empty ? -INFINITY : st.r + (l2 + shift) * kLn2;
    if (lse < st.r) lse = st.r;
    float entropy = empty ? 0.0f : (l2 - st.w / st.s) * kLn2;
    if (entropy < 0.0f) entropy = 0.0f;
    if (tid == 0) {
        if (a.lse) a.lse[row] = lse;
        if (a.entropy) a.entropy[row] = entropy;
    }
    auto lp = [&](float x) { return empty ? lse : x - lse; };
    for (int i = tid; i < a.n_given; i += threads) {
        if (i != tid) g = given<T>(a, row, i);
        a.logprob[row * a.n_given + i] =
            g.token >= 0 && g.token < a.n_vocab ? lp(g.x) : __builtin_nanf("");
    }
    by_rank(tops, count, a.n_top, threads, [&](int rank, uint64_t k) {
        a.top_ids[row * a.n_top + rank] = key_index(k);
        a.top_logprobs[row * a.n_top + rank] = lp(key_value(k));
    });
}

template <int T, int W, bool TOP>
__global__ __launch_bounds__(64 * W) void logprob_kernel(const LogprobArgs a, const Work wk)
{
    typedef typename Elem<T>::type E;
    constexpr int V = kVec<T>;
    static_assert(W == 4 || W == 16, "256 lanes, or quads of them");
    __shared__ Stat part[W];
    __shared__ __align__(16) uint64_t places[TOP ? W : 1][TOP ? kPlaces : 2];
    __shared__ __align__(16) uint64_t merged[TOP ? W * kLogprobMaxTop : 2];
    __shared__ __align__(16) u32x4 pend_v[TOP ? W : 1][TOP ? kPend : 1];
    __shared__ int pend_i[TOP ? W : 1][TOP ? kPend : 1];
    __shared__ __align__(16) uint32_t bounds[2][256];
    __shared__ int counts[W];
    const int64_t row = blockIdx.y;
    const int lane = threadIdx.x & 63, wave = wave_uniform((int)(threadIdx.x >> 6));
    const int begin = blockIdx.x * wk.part_len;
    const int len = min(wk.part_len, (int)a.n_vocab - begin);
    const E *x0 = (const E *)a.logits + row * a.row_stride + begin;
    // whole 16-byte vectors from the first aligned one; the logits before and
    // after them (up to 14) are taken one per lane at the end
    const int head = min((int)((-(uintptr_t)x0 & 15) / sizeof(E)), len);
    const E *x = x0 + head;
    const int vecs = (len - head) / V, tail = len - head - vecs * V;

    Stat st = stat_zero();
    Top top;
    Pending<T> pend;
    if (TOP) {
        top.init(places[wave], a.n_top);
        pend.init(pend_v[wave], pend_i[wave]);
    }
    // a turn: kLoads x 64 vectors per wave, 64 of each wave in turn, so that a
    // short row or last turn is spread over the waves; every wave makes the same
    // number of turns
    constexpr int kPart = 64 * W, kTurn = kPart * kLoads;
    u32x4 raw[kLoads];
    auto fetch = [&](int v0) {
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            // past the end the last vector again, dismissed below
            const int v = min(v0 + kPart * u + lane, vecs - 1);
            raw[u] = __builtin_nontemporal_load((const u32x4 *)(x + (int64_t)v * V));
        }
    };
    const int edge_i = lane < head ? lane : lane + vecs * V;
    const float edge = lane < head + tail && wave == W - 1 ? (float)x0[edge_i] : -INFINITY;
    if (vecs > 0) fetch(64 * wave);
    Given g = {-1, 0.0f};
    if (wk.parts == 1) g = given<T>(a, row, threadIdx.x);
    float lane_max = __builtin_nanf("");
    bool low = false;                  // this wave has met a logit of -infinity or near
    for (int it = 0; it * kTurn < vecs; ++it) {
        const int v0 = it * kTurn + 64 * wave, left = vecs - v0;
        float xv[kLoads][V], best[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            unpack16<T>(raw[u], xv[u]);
            best[u] = -INFINITY;
        }
        if ((it + 1) * kTurn < vecs) fetch(v0 + kTurn);    // lands during this turn
        const bool full = left >= kPart * (kLoads - 1) + 64;
        if (!full) {
            // no terms: lower than any reference, and d stays finite
#pragma unroll
            for (int u = 0; u < kLoads; ++u)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (kPart * u + lane >= left) xv[u][j] = -2e38f;
        }
        if (left > 0) {
            float r = st.r;
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                best[u] = xv[u][0];
#pragma unroll
                for (int j = 1; j < V; ++j) best[u] = fmaxf(best[u], xv[u][j]);
                r = fmaxf(r, best[u]);
            }
            stat_move(st, r);
            const float r2 = r * kL2E;
            auto terms = [&](auto with_low) {
                Stat t = {r, 0.0f, 0.0f};
#pragma unroll
                for (int u = 0; u < kLoads; ++u) {
                    if (kPart * u >= left) break;
#pragma unroll
                    for (int j = 0; j < V; ++j) stat_add<decltype(with_low)::value>(t, xv[u][j], r2);
                }
                return t;
            };
            // without the clamp of every term, 32 of 220 instructions, until a
            // sum says that it is needed
            Stat t;
            if (!low) {
                t = terms(std::false_type());
                low = __ballot(t.w != t.w) != 0;
            }
            if (low) t = terms(std::true_type());
            // (a turn's terms in a sum of their own: equal terms round to one
            // side, and 1024 of them in one chain put the log sum exp of 262144
            // logits 1.2e-5 off; now 7e-7)
            st.s += t.s;
            st.w += t.w;
        }
        if (TOP) {
            if (full) {
#pragma unroll
                for (int u = 0; u < kLoads; ++u) lane_max = fmaxf(lane_max, best[u]);
            } else {
#pragma unroll
                for (int u = 0; u < kLoads; ++u)
                    lane_max = fmaxf(lane_max, kPart * u + lane < left ? best[u] : __builtin_nanf(""));
            }
            if ((it & (it + 1)) == 0) {            // turns 1, 2, 4, 8, ...
                uint32_t mine = value_key(lane_max);
                if (W == 16) {                     // 256 quads
                    mine = max(mine, row_move<0xb1>(mine));
                    mine = max(mine, row_move<0x4e>(mine));
                }
                // (a wave is at most one barrier ahead: two sets are enough)
                uint32_t *set = bounds[__builtin_popcount(it) & 1];
                if (W == 4 || lane % 4 == 0) set[threadIdx.x / (W / 4)] = mine;
                __syncthreads();
                // (64 groups do for a short list: 20 of them let in 24 logits
                // where 20 of 256 let in 21, at a quarter of the work: 2048 x
                // 32000 bfloat16 with a list of 20 34.9 -> 31.0 us)
                const u32x4 four = {set[lane], set[64 + lane], set[128 + lane], set[192 + lane]};
                const uint32_t all = a.n_top <= kShortTop
                                         ? nth_key(max(max(four.x, four.y), max(four.z, four.w)), a.n_top)
                                         : nth_key(four, a.n_top);
                const uint64_t t = ((uint64_t)all << 32) - 1;
                if (all && t > top.thr) top.set(t);
            }
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const int v = v0 + kPart * u + lane;
                uint64_t in = __ballot(!(best[u] < top.least));
                if (!full) in &= __ballot(v < vecs);
                if (in) pend.push(in, repack16<T>(xv[u]), v, begin + head, top, lane);
            }
        }
    }
    if (TOP) pend.flush(begin + head, top, lane);
    if (head + tail && wave == W - 1) {
        const float r = fmaxf(st.r, edge);
        stat_move(st, r);
        stat_add<true>(st, edge, r * kL2E);
        if (TOP) top.offer(edge, (uint32_t)(begin + edge_i), lane < head + tail, lane);
    }

    st = wave_join(st);
    if (lane == 0) part[wave] = st;
    if (TOP) {
        if (top.count > kLogprobMaxTop) top.compact(lane);       // what `merged` has room for
        wave_lds_sync();
        if (lane == 0) counts[wave] = top.count;
    }
    __syncthreads();
    int count = 0;
    if (TOP) {
        // the waves' candidates behind each other
        int at = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w == wave) at = count;
            count += counts[w];
        }
        for (int i = lane; i < top.count; i += 64) merged[at + i] = top.place[i];
    }
    st = stat_zero();
    if (lane < W) st = part[lane];
    st = wave_join(st);
    __syncthreads();
    if (wk.parts == 1) {
        finish<T>(a, row, st, part, W, merged, count, g);
        return;
    }
    const int64_t slot = row * wk.parts + blockIdx.x;
    if (threadIdx.x == 0) wk.stats[slot] = st;
    if (TOP) {
        // the part's list: its entries by rank, 0 behind them
        uint64_t *out = wk.tops + slot * a.n_top;
        const int have = min(len, a.n_top);
        for (int i = threadIdx.x; i < a.n_top; i += 64 * W)
            if (i >= have) out[i] = 0;
        by_rank(merged, count, a.n_top, 64 * W, [&](int rank, uint64_t k) { out[rank] = k; });
    }
}

// The parts of a row.
template <int T>
__global__ __launch_bounds__(256) void logprob_join_kernel(const LogprobArgs a, const Work wk)
{
    __shared__ Stat part[4];
    __shared__ __align__(16) uint64_t keys[kMaxParts * kLogprobMaxTop];
    __shared__ int count;
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63;
    const Given g = given<T>(a, row, tid);
    Stat st = stat_zero();
    if (lane < wk.parts) st = wk.stats[row * wk.parts + lane];
    const uint64_t *tops = wk.tops + row * wk.parts * a.n_top;
    uint64_t k[kMaxParts / 4];
    const int total = wk.parts * a.n_top;
    // (n_top <= 64: at most kMaxParts / 4 keys per thread)
#pragma unroll
    for (int i = 0; i < kMaxParts / 4; ++i) {
        if (256 * i >= total) break;
        k[i] = tid + 256 * i < total ? tops[tid + 256 * i] : 0;
    }
    // A bound: with r = n_top / parts, the (n_top / r)-th largest of the parts'
    // r-th entries (n_top keys reach it).
    uint32_t t = 0;
    if (a.n_top > 0) {
        const int each = (a.n_top + wk.parts - 1) / wk.parts;
        const uint32_t v = lane < wk.parts ? (uint32_t)(tops[lane * a.n_top + each - 1] >> 32) : 0;
        t = nth_key(v, (a.n_top + each - 1) / each);
        if (tid == 0) count = 0;
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kMaxParts / 4; ++i) {
        if (256 * i >= total) break;
        if (k[i] != 0 && (uint32_t)(k[i] >> 32) >= t) keys[atomicAdd(&count, 1)] = k[i];
    }
    st = wave_join(st);
    __syncthreads();
    finish<T>(a, row, st, part, 4, keys, a.n_top > 0 ? count : 0, g);
}

// How a call is cut: waves per workgroup and parts per row.
struct Cut {
    int waves, parts, part_len;
};

Cut cut(int64_t m, int64_t v)
{
    Cut c;
    // 1024 workgroups of 4 waves fill the device; from 512 rows on a second
    // launch costs more than it gives (512 x 262144 bf16: 42 us in one, 46 in
    // two parts; 300 rows: 37 and 33 us)
    int64_t parts = m >= 512 ? 1 : 1024 / (m > 0 ? m : 1);
    if (parts > v / 16384) parts = v / 16384;
    if (parts > kMaxParts) parts = kMaxParts;
    if (parts < 1) parts = 1;
    // fewer workgroups than CUs: more waves each
    c.waves = m * parts < 256 && v > 8192 ? 16 : 4;
    const int64_t len = ((v + parts - 1) / parts + 7) / 8 * 8;
    c.part_len = (int)len;
    c.parts = (int)((v + len - 1) / len);
    return c;
}

template <int T>
void launch_part(const LogprobArgs &a, const Work &w, const Cut &c, hipStream_t stream)
{
    const dim3 grid((unsigned)c.parts, (unsigned)a.m), block(64 * c.waves);
    if (c.waves == 4 && a.n_top)
        hipLaunchKernelGGL((logprob_kernel<T, 4, true>), grid, block, 0, stream, a, w);
    else if (c.waves == 4)
        hipLaunchKernelGGL((logprob_kernel<T, 4, false>), grid, block, 0, stream, a, w);
    else if (a.n_top)
        hipLaunchKernelGGL((logprob_kernel<T, 16, true>), grid, block, 0, stream, a, w);
    else
        hipLaunchKernelGGL((logprob_kernel<T, 16, false>), grid, block, 0, stream, a, w);
}

template <int T>
int launch_type(const LogprobArgs &a, void *ws, hipStream_t stream)
{
    const Cut c = cut(a.m, a.n_vocab);
    Work wk;
    wk.parts = c.parts;
    wk.part_len = c.part_len;
    wk.tops = (uint64_t *)ws;
    wk.stats = (Stat *)(wk.tops + a.m * c.parts * a.n_top);
    // rows are the grid's second axis: at most 65535 a launch
    for (int64_t r0 = 0; r0 < a.m; r0 += 65535) {
        const int64_t rows = a.m - r0 < 65535 ? a.m - r0 : 65535;
        LogprobArgs b = a;
        Work w = wk;
        const int64_t es = T == Q8_T_F32 ? 4 : 2;
        b.logits = (const uint8_t *)a.logits + r0 * a.row_stride * es;
        if (a.n_given) { b.tokens += r0 * a.n_given; b.logprob += r0 * a.n_given; }
        if (a.lse) b.lse += r0;
        if (a.entropy) b.entropy += r0;
        if (a.n_top) { b.top_ids += r0 * a.n_top; b.top_logprobs += r0 * a.n_top; }
        b.m = rows;
        w.tops += r0 * c.parts * a.n_top;
        w.stats += r0 * c.parts;
        launch_part<T>(b, w, c, stream);
        if (c.parts > 1)
            hipLaunchKernelGGL(logprob_join_kernel<T>, dim3((unsigned)rows), dim3(256), 0, stream, b, w);
    }
    return hipGetLastError() == hipSuccess ? 0 : -6;
}

}  // namespace

size_t logprob_ws_needed(int64_t m, int64_t n_vocab, int64_t n_top)
{
    const Cut c = cut(m, n_vocab);
    return c.parts == 1 ? 0 : (size_t)m * c.parts * (8 * n_top + sizeof(Stat));
}

// What any call of up to m rows needs: rows are in most parts when they are
// few, and never in more than 1024 parts together (cut).
size_t logprob_ws_bytes(int64_t m, int64_t n_vocab, int64_t n_top)
{
    const int64_t parts = cut(1, n_vocab).parts;
    if (parts == 1) return 0;
    const int64_t all = m < 1024 / parts ? m * parts : 1024;
    return (size_t)all * (8 * n_top + sizeof(Stat));
}

int launch_logprob(const LogprobArgs &a, void *ws, hipStream_t stream)
{
    if (a.type == Q8_T_F32) return launch_type<Q8_T_F32>(a, ws, stream);
    if (a.type == Q8_T_F16) return launch_type<Q8_T_F16>(a, ws, stream);
    return launch_type<Q8_T_BF16>(a, ws, stream);
}

}  // namespace q8
