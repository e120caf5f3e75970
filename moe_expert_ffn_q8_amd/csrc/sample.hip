// sample.hip -- one token per row of logits: temperature, top-k, top-p, min-p
// and a draw from a given random number.
//
// A row's tokens are taken in the order (value descending, index ascending).
// Each filter keeps a head of that order, so what is kept is the shortest head,
// and the drawn token is the first at which the running mass passes u times the
// head's mass: every question is "where does the running count (or mass) reach
// a target", and a histogram over the values answers it without a sort.
//
// Weights exp((x - M) / T) are formed in 64 bits and summed as whole numbers of
// 2^-52 of the largest (coarser where a row's sum S would pass 2^62): sums are
// exact, whatever their order, and a border of top-p or of the random number
// falls between tokens as it does in 64 bits.
#include "i8_device.h"
#include "q8_ops.h"

namespace q8 {

namespace {

typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef unsigned long long u64;

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBins = 2048;       // two per thread
constexpr float kReach = 64.0f;   // the first histogram covers weights down to 2^-64

// 2^t for t <= 0, off by 1.5e-14 at most: 2^r on [-1/2, 1/2] as a polynomial of
// degree 9 that is 1 at 0 (the coefficients by the exchange algorithm).
__device__ __forceinline__ double exp2_64(double t)
{
    t = fmax(t, -1100.0);
    const double n = rint(t), r = t - n;
    double p = 0x1.b3de7e08233fap-24;
    p = fma(p, r, 0x1.63e6984270859p-20);
    p = fma(p, r, 0x1.ffce2f62db0e4p-17);
    p = fma(p, r, 0x1.430897f140f61p-13);
    p = fma(p, r, 0x1.5d87fd93b0878p-10);
    p = fma(p, r, 0x1.3b2ab7241364fp-7);
    p = fma(p, r, 0x1.c6b08d70c8658p-5);
    p = fma(p, r, 0x1.ebfbdff81bdf6p-3);
    p = fma(p, r, 0x1.62e42fefa37d2p-1);
    p = fma(p, r, 1.0);
    return __builtin_amdgcn_ldexp(p, (int)n);
}

// Order of the values: larger ones have larger keys; -0 as +0.
__device__ __forceinline__ uint32_t value_key(float x)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k)
{
    return __builtin_bit_cast(float, (k >> 31) ? (k & 0x7fffffffu) : ~k);
}

constexpr uint32_t kLeastKey = 0x00800000u;       // of the lowest finite value

// What the weights of a row are formed with.
struct Weights {
    float top;                    // M
    double scale;                 // log2(e) / T
    int bits;                     // a unit is 2^-bits
    double unit;                  // 2^(52 - bits): added, leaves whole units
    __device__ __forceinline__ double t(float x) const { return ((double)x - (double)top) * scale; }
    __device__ __forceinline__ u64 units(float x) const
    {
        return __builtin_bit_cast(u64, exp2_64(t(x)) + unit) - __builtin_bit_cast(u64, unit);
    }
};

struct Head {                     // tokens at the head of the order
    uint32_t count;
    u64 mass;
};

// Sums over the workgroup, in every thread; the order is fixed.
template <class N>
__device__ N block_sum(N v, u64 *part)
{
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = __builtin_bit_cast(u64, v);
    __syncthreads();
    v = 0;
    for (int w = 0; w < kWaves; ++w) v += __builtin_bit_cast(N, part[w]);
    return v;
}

// f(value, index) for every logit of the row.
template <int T, class F>
__device__ __forceinline__ void each(const SampleArgs &a, int64_t row, F f)
{
    typedef typename Elem<T>::type E;
    constexpr int V = kVec<T>;
    const E *x = (const E *)a.logits + row * a.row_stride;
    const int len = (int)a.n_vocab, vecs = len / V;
    for (int v = threadIdx.x; v < vecs; v += kThreads) {
        float y[V];
        unpack16<T>(*(const u32x4_any *)(x + v * V), y);
#pragma unroll
        for (int j = 0; j < V; ++j) f(y[j], v * V + j);
    }
    const int i = vecs * V + threadIdx.x;
    if (i < len) f((float)x[i], i);
}

// Histogram of one stretch of the order.
struct Bins {
    uint32_t count[kBins];
    u64 mass[kBins];
};

struct Shared {
    Bins first, next;             // of the whole row; of one of its bins and less
    u64 part[kWaves];
    Head wave[kWaves];
    Head before;                  // the answer of find()
    int bin;
    uint32_t key, lowest;
    int index;
};

__device__ __forceinline__ void clear(Bins &b)
{
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
        b.count[i] = 0;
        b.mass[i] = 0;
    }
}

// The first bin at which the head `before` and the bins so far reach the target
// (by count, or by mass), and the head before that bin.
__device__ void find(Shared &s, const Bins &b, Head before, bool by_mass, u64 target)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    __syncthreads();              // the last answer has been read, the histogram is whole
    const Head h0 = {b.count[2 * tid], b.mass[2 * tid]};
    const Head h1 = {b.count[2 * tid + 1], b.mass[2 * tid + 1]};
    Head sum = {h0.count + h1.count, h0.mass + h1.mass};
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t c = __shfl_up(sum.count, d);
        const u64 m = __shfl_up(sum.mass, d);
        if (lane >= d) {
            sum.count += c;
            sum.mass += m;
        }
    }
    if (lane == 63) s.wave[wave] = sum;
    if (tid == 0) s.bin = 0;
    __syncthreads();
    for (int w = 0; w < wave; ++w) {
        before.count += s.wave[w].count;
        before.mass += s.wave[w].mass;
    }
    before.count += sum.count - h0.count - h1.count;
    before.mass += sum.mass - h0.mass - h1.mass;
    auto reaches = [&](const Head &h) { return by_mass ? h.mass >= target : h.count >= target; };
    const Head mid = {before.count + h0.count, before.mass + h0.mass};
    const Head end = {mid.count + h1.count, mid.mass + h1.mass};
    if (!reaches(before)) {
        if (reaches(mid)) {
            s.bin = 2 * tid;
            s.before = before;
        } else if (reaches(end)) {
            s.bin = 2 * tid + 1;
            s.before = mid;
        }
    }
    __syncthreads();
}

// Where the order reaches a target: the value there, how many of its equals are
// needed, and the head up to and with them.
struct Place {
    uint32_t key, equals;
    Head head;
};

template <int T>
__device__ Place locate(const SampleArgs &a, int64_t row, const Weights &w, float bin_scale, Shared &s,
                        bool by_mass, u64 target)
{
    find(s, s.first, {0, 0}, by_mass, target);
    const int first = s.bin;
    Head before = s.before;
    // keys that the bin may hold, a bin's width to spare on either side
    auto bound = [&](double d) { return value_key((float)((double)w.top - d / (double)bin_scale)); };
    uint32_t hi = first <= 0 ? value_key(w.top) : min(value_key(w.top), bound(first - 1.0));
    uint32_t lo = first == kBins - 1 || bin_scale == 0.0f ? kLeastKey : max(kLeastKey, bound(first + 2.0));
    while (lo != hi) {            // 11 bits of the key a turn: three at most
        const int shift = max(0, 32 - __clz(hi - lo) - 11);
        __syncthreads();
        clear(s.next);
        __syncthreads();
        each<T>(a, row, [&](float x, int) {
            const uint32_t k = value_key(x);
            if (k < lo || k > hi) return;
            if ((int)fminf((w.top - x) * bin_scale, (float)(kBins - 1)) != first) return;
            atomicAdd(&s.next.count[(hi - k) >> shift], 1u);
            atomicAdd(&s.next.mass[(hi - k) >> shift], w.units(x));
        });
        find(s, s.next, before, by_mass, target);
        before = s.before;
        const uint32_t top = hi - ((uint32_t)s.bin << shift);
        lo = max(lo, top - ((1u << shift) - 1));
        hi = top;
    }
    const u64 one = w.units(key_value(hi));
    Place p;
    p.key = hi;
    p.equals = by_mass ? (uint32_t)((target - before.mass + one - 1) / one) : (uint32_t)(target - before.count);
    p.head = {before.count + p.equals, before.mass + p.equals * one};
    return p;
}

// Index of the nth (from 1) logit of the row that has this key.
template <int T>
__device__ int nth_equal(const SampleArgs &a, int64_t row, uint32_t key, uint32_t nth, Shared &s)
{
    typedef typename Elem<T>::type E;
    const E *x = (const E *)a.logits + row * a.row_stride;
    const int len = (int)a.n_vocab, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t before = 0;
    if (threadIdx.x == 0) s.index = 0;
    for (int i0 = 0; i0 < len; i0 += kThreads) {
        const int i = i0 + threadIdx.x;
        const bool eq = i < len && value_key((float)x[i]) == key;
        const u64 in = __ballot(eq);
        __syncthreads();
        if (lane == 0) s.part[wave] = __popcll(in);
        __syncthreads();
        uint32_t rank = before + __popcll(in & ((1ull << lane) - 1)), all = 0;
        for (int w = 0; w < kWaves; ++w) {
            if (w < wave) rank += (uint32_t)s.part[w];
            all += (uint32_t)s.part[w];
        }
        if (eq && rank + 1 == nth) s.index = i;
        before += all;
        if (before >= nth) break;
    }
    __syncthreads();
    return s.index;
}

// One workgroup per row, the row read again for every step.
template <int T>
__global__ __launch_bounds__(kThreads) void sample_kernel(const SampleArgs a)
{
    __shared__ Shared s;
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;

    // the largest logit, how many there are, and what makes the row no distribution
    uint32_t best = 0, finite = 0, bad = 0;
    each<T>(a, row, [&](float x, int) {
        bad |= x != x || x == INFINITY;
        finite += x > -INFINITY;
        best = max(best, value_key(x));
    });
    for (int d = 32; d; d >>= 1) best = max(best, __shfl_xor(best, d));
    if (tid == 0) s.key = 0;
    finite = (uint32_t)block_sum((u64)finite, s.part);
    bad = (uint32_t)block_sum((u64)bad, s.part);
    if ((tid & 63) == 0) atomicMax(&s.key, best);
    __syncthreads();
    best = s.key;
    if (bad || !finite) {
        if (tid == 0) {
            a.ids[row] = -1;
            a.kept[row] = 0;
            a.logprob[row] = bad ? __builtin_nanf("") : -INFINITY;
        }
        return;
    }

    const float temp = a.temperature ? a.temperature[row] : 1.0f;
    if (!(temp > 0.0f)) {                      // the largest logit, the first of equals
        const int i = nth_equal<T>(a, row, best, 1, s);
        if (tid == 0) {
            a.ids[row] = i;
            a.kept[row] = 1;
            a.logprob[row] = 0.0f;
        }
        return;
    }
    Weights w;
    w.top = key_value(best);
    w.scale = 1.4426950408889634074 / (double)temp;
    double total = 0.0;
    each<T>(a, row, [&](float x, int) { total += x > -INFINITY ? exp2_64(w.t(x)) : 0.0; });
    total = block_sum(total, s.part);
    w.bits = min(52, 61 - __builtin_amdgcn_frexp_exp(total));
    w.unit = __builtin_amdgcn_ldexp(1.0, 52 - w.bits);
    const float bin_scale = (float)fmin(w.scale * ((kBins - 1) / kReach), 1e30);
    const double min_p = a.min_p ? (double)a.min_p[row] : 0.0;
    const double least = min_p > 0.0 ? fmin(log2(min_p), 0.0) : -INFINITY;

    clear(s.first);
    __syncthreads();
    Head floor_ = {0, 0};                      // the tokens that min-p keeps
    each<T>(a, row, [&](float x, int) {
        if (!(x > -INFINITY)) return;
        const int b = (int)fminf((w.top - x) * bin_scale, (float)(kBins - 1));
        const u64 m = w.units(x);
        atomicAdd(&s.first.count[b], 1u);
        atomicAdd(&s.first.mass[b], m);
        if (w.t(x) >= least) {
            ++floor_.count;
            floor_.mass += m;
        }
    });
    floor_.count = (uint32_t)block_sum((u64)floor_.count, s.part);
    floor_.mass = block_sum(floor_.mass, s.part);

    Head head = {finite, 0};
    head.mass = block_sum(s.first.mass[tid] + s.first.mass[tid + kThreads], s.part);
    const int32_t k = a.top_k ? a.top_k[row] : 0;
    if (k > 0 && (uint32_t)k < finite) head = locate<T>(a, row, w, bin_scale, s, false, (u64)k).head;
    const float p = a.top_p ? a.top_p[row] : 1.0f;
    if (p < 1.0f) {
        const u64 target = (u64)ceil(fmax((double)p, 0.0) * (double)head.mass);
        head = locate<T>(a, row, w, bin_scale, s, true, target > 0 ? target : 1).head;
    }
    if (floor_.count < head.count) head = floor_;
    const float u = a.u[row];
    u64 target = (u64)((u > 0.0f ? (double)u : 0.0) * (double)head.mass) + 1;
    if (!(u < 1.0f) || target > head.mass) target = u != u ? 1 : head.mass;
    const Place at = locate<T>(a, row, w, bin_scale, s, true, target);
    const int i = nth_equal<T>(a, row, at.key, at.equals, s);
    if (tid == 0) {
        a.ids[row] = i;
        a.kept[row] = (int32_t)head.count;
        const double lp = (w.t(key_value(at.key)) - (log2((double)head.mass) - w.bits)) * 0.693147180559945309417;
        a.logprob[row] = (float)fmin(lp, 0.0);
    }
}

}  // namespace

size_t sample_ws_bytes(int64_t, int64_t) { return 256; }

int launch_sample(const SampleArgs &a, void *, hipStream_t stream)
{
    if (a.type == Q8_T_F32)
        hipLaunchKernelGGL((sample_kernel<Q8_T_F32>), dim3((unsigned)a.m), dim3(kThreads), 0, stream, a);
    else if (a.type == Q8_T_F16)
        hipLaunchKernelGGL((sample_kernel<Q8_T_F16>), dim3((unsigned)a.m), dim3(kThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((sample_kernel<Q8_T_BF16>), dim3((unsigned)a.m), dim3(kThreads), 0, stream, a);
    return hipGetLastError() == hipSuccess ? 0 : -6;
}

}  // namespace q8
