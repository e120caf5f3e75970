// logprob.hip -- log probabilities of given tokens, log sum exp, entropy and the
// largest logits of each row.
//
// One workgroup per row.  One pass keeps the running maximum M, S = sum
// exp(x - M) and W = sum exp(x - M)(x - M); the top list is found one entry at
// a time, each the largest (value, lowest index) below the last.
#include "i8_device.h"
#include "q8_i8.h"

namespace q8 {

namespace {

constexpr int kThreads = 256;

// Running (M, S, W).  M starts at the lowest finite value, so that x - M never
// is infinity minus infinity for a row's -infinities; a NaN or +infinity makes
// S NaN and stays.
struct Stat {
    float m, s, w;
};

__device__ __forceinline__ Stat stat_zero() { return {-3.402823466e38f, 0.0f, 0.0f}; }

// The clamp keeps 0 * -infinity out of W; exp of it is 0 all the same.
__device__ __forceinline__ float floor_d(float d) { return fmaxf(d, -1e30f); }

__device__ __forceinline__ void stat_rescale(Stat &a, float m)
{
    const float d = floor_d(a.m - m), f = __expf(d);
    a.w = (a.w + a.s * d) * f;
    a.s *= f;
    a.m = m;
}

__device__ __forceinline__ void stat_add(Stat &a, float x)
{
    if (x > a.m) stat_rescale(a, x);
    const float d = x - a.m, e = __expf(d);
    a.s += e;
    a.w = fmaf(e, floor_d(d), a.w);
}

__device__ __forceinline__ Stat stat_join(Stat a, Stat b)
{
    const float m = fmaxf(a.m, b.m);
    stat_rescale(a, m);
    stat_rescale(b, m);
    return {m, a.s + b.s, a.w + b.w};
}

// Order of the top list: larger value first, then lower index; NaN last.
__device__ __forceinline__ uint64_t order_key(float x, uint32_t i)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);       // -0 -> +0
    uint32_t key = (u >> 31) ? ~u : (u | 0x80000000u);
    if (x != x) key = 0;
    return ((uint64_t)key << 32) | (uint32_t)~i;
}

template <int T>
__global__ __launch_bounds__(kThreads) void logprob_kernel(const LogprobArgs a)
{
    typedef typename Elem<T>::type E;
    __shared__ Stat stats[kThreads / 64];
    __shared__ uint64_t best[kThreads / 64];
    __shared__ float result;
    const int64_t row = blockIdx.x;
    const E *x = (const E *)a.logits + row * a.row_stride;
    const int v = (int)a.n_vocab;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    Stat st = stat_zero();
    for (int i = tid; i < v; i += kThreads) stat_add(st, (float)x[i]);
    for (int d = 32; d; d >>= 1)
        st = stat_join(st, {__shfl_xor(st.m, d), __shfl_xor(st.s, d), __shfl_xor(st.w, d)});
    if (lane == 0) stats[wave] = st;
    __syncthreads();
    if (tid == 0) {
        for (int i = 1; i < kThreads / 64; ++i) st = stat_join(st, stats[i]);
        const bool empty = st.s == 0.0f;
        const float ls = logf(st.s);
        const float lse = empty ? -INFINITY : st.m + ls;
        if (a.lse) a.lse[row] = lse;
        if (a.entropy) a.entropy[row] = empty ? 0.0f : ls - st.w / st.s;
        result = lse;
    }
    __syncthreads();
    const float lse = result;
    // x - lse, with -infinity where the whole row is
    auto lp = [&](float xv) { return lse == -INFINITY ? lse : xv - lse; };
    for (int i = tid; i < a.n_given; i += kThreads) {
        const int tok = a.tokens[row * a.n_given + i];
        a.logprob[row * a.n_given + i] =
            tok >= 0 && tok < v ? lp((float)x[tok]) : __builtin_nanf("");
    }
    uint64_t last = ~(uint64_t)0;
    for (int n = 0; n < a.n_top; ++n) {
        uint64_t b = 0;
        for (int i = tid; i < v; i += kThreads) {
            const uint64_t key = order_key((float)x[i], i);
            if (key < last && key > b) b = key;
        }
        for (int d = 32; d; d >>= 1) {
            const uint64_t o = (uint64_t)__shfl_xor((long long)b, d);
            b = o > b ? o : b;
        }
        if (lane == 0) best[wave] = b;
        __syncthreads();
        for (int i = 0; i < kThreads / 64; ++i) b = best[i] > b ? best[i] : b;
        __syncthreads();
        last = b;
        if (tid == 0) {
            const uint32_t id = ~(uint32_t)b;
            a.top_ids[row * a.n_top + n] = (int)id;
            a.top_logprobs[row * a.n_top + n] = lp((float)x[id]);
        }
    }
}

}  // namespace

size_t logprob_ws_bytes(int64_t, int64_t, int64_t) { return 0; }

int launch_logprob(const LogprobArgs &a, void *, hipStream_t stream)
{
    const dim3 grid((unsigned)a.m), block(kThreads);
    if (a.type == Q8_T_F32)
        hipLaunchKernelGGL(logprob_kernel<Q8_T_F32>, grid, block, 0, stream, a);
    else if (a.type == Q8_T_F16)
        hipLaunchKernelGGL(logprob_kernel<Q8_T_F16>, grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL(logprob_kernel<Q8_T_BF16>, grid, block, 0, stream, a);
    return hipGetLastError() == hipSuccess ? 0 : -6;
}

}  // namespace q8
