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
//
// The logits are read once.  A workgroup holds a row, or a part of one, in its
// registers, sums its weights where a filter needs the sum, and lists the logits
// that reach a bound: that many of its lanes' maxima do.  The list is a head of
// the row's order (down to the largest bound of its parts), and where the
// answers lie in it, as they do for most rows, it alone is looked at further.
// Else (a target beyond the list, many equal logits) the row is read again, once
// per 11 bits of each answer.
#include "i8_device.h"
#include "order_device.h"
#include "q8_ops.h"

namespace q8 {

namespace {

typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef unsigned long long u64;

constexpr float kReach = 64.0f;   // a histogram by value covers weights down to 2^-64
constexpr int kPlaces = 128;      // listed logits per wave of a part

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

constexpr uint32_t kLeastKey = 0x00800000u;       // value_key of the lowest finite value
constexpr uint32_t kNoBound = 0xffffffffu;        // of a part that has no list

__device__ __forceinline__ float value_of(uint32_t key) { return key_value((uint64_t)key << 32); }

// A row's settings, as they are applied.
struct Settings {
    float u;
    double scale;                 // log2(e) / T; 0: the largest logit
    uint32_t top_k;               // 0: all
    double top_p;                 // 1: all
    double least;                 // log2(min_p); -infinity: all
    bool greedy;

    __device__ __forceinline__ Settings(const SampleArgs &a, int64_t row)
    {
        const float temp = a.temperature ? a.temperature[row] : 1.0f;
        const int32_t k = a.top_k ? a.top_k[row] : 0;
        const float p = a.top_p ? a.top_p[row] : 1.0f;
        const float m = a.min_p ? a.min_p[row] : 0.0f;
        u = a.u[row];
        greedy = !(temp > 0.0f);
        scale = greedy ? 0.0 : 1.4426950408889634074 / (double)temp;
        top_k = k > 0 ? (uint32_t)k : 0u;
        top_p = p < 1.0f ? fmax((double)p, 0.0) : 1.0;
        least = m > 0.0f ? fmin(log2((double)m), 0.0) : -INFINITY;
    }
    // whether the mass of the whole row is asked for (where k does not reach
    // all finite logits, that of its head is)
    __device__ __forceinline__ bool needs_sum() const { return !greedy && top_k == 0; }
};

// What the weights of a row are formed with.
struct Weights {
    float top;                    // M
    double scale;
    int bits;                     // a unit is 2^-bits
    double unit;                  // 2^(52 - bits): added, leaves whole units

    // sum: what the weights' sum is below, or twice that
    __device__ __forceinline__ Weights(float top, double scale, double sum) : top(top), scale(scale)
    {
        bits = min(52, 61 - __builtin_amdgcn_frexp_exp(sum));
        unit = __builtin_amdgcn_ldexp(1.0, 52 - bits);
    }
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

// ---------------------------------------------------------------------------
// By a workgroup of NT threads.

template <int NT>
struct __align__(16) Shared {
    static constexpr int kBins = 2 * NT;               // of a histogram of the row
    static constexpr int kBinBits = NT == 1024 ? 11 : 9;
    static constexpr int kList = 4 * NT;               // logits of a list
    static constexpr int kMembers = NT;                // of one bin of a list
    static_assert(NT == 1024 || NT == 256, "bins by powers of two");
    union {
        uint32_t keys[256];
        struct {
            u64 list[kList], mass[NT], member_key[kMembers], member_mass[kMembers];
            uint32_t count[NT];
        };
        struct {                  // of the whole row; of one of its bins and less
            u64 first_mass[kBins], next_mass[kBins];
            uint32_t first_count[kBins], next_count[kBins];
        };
    };
    u64 part[NT / 64];
    Head wave[NT / 64];
    Head before;                  // the answers of find() and list_locate()
    u64 key;
    int bin, index, members, listed;
};

// Sums over the workgroup, in every thread; the order is fixed.
template <int NT, class N>
__device__ __forceinline__ N block_sum(N v, u64 *part)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = __builtin_bit_cast(u64, v);
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) v += __builtin_bit_cast(N, part[w]);
    return v;
}

// f(value, index) for every logit of the row, from memory.
template <int T, int NT, class F>
__device__ __forceinline__ void each(const SampleArgs &a, int64_t row, F f)
{
    typedef typename Elem<T>::type E;
    constexpr int V = kVec<T>;
    const E *x = (const E *)a.logits + row * a.row_stride;
    const int len = (int)a.n_vocab, vecs = len / V;
    for (int v = threadIdx.x; v < vecs; v += NT) {
        float y[V];
        unpack16<T>(*(const u32x4_any *)(x + v * V), y);
#pragma unroll
        for (int j = 0; j < V; ++j) f(y[j], v * V + j);
    }
    const int i = vecs * V + threadIdx.x;
    if (i < len) f((float)x[i], i);
}

// The running head before bins own (of this thread), given that before all bins.
template <int NT>
__device__ __forceinline__ Head scan(Shared<NT> &s, Head before, Head own)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    Head sum = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t c = __shfl_up(sum.count, d);
        const u64 m = __shfl_up(sum.mass, d);
        if (lane >= d) {
            sum.count += c;
            sum.mass += m;
        }
    }
    if (lane == 63) s.wave[wave] = sum;
    __syncthreads();
    for (int w = 0; w < wave; ++w) {
        before.count += s.wave[w].count;
        before.mass += s.wave[w].mass;
    }
    return {before.count + sum.count - own.count, before.mass + sum.mass - own.mass};
}

__device__ __forceinline__ bool reaches(const Head &h, bool by_mass, u64 target)
{
    return by_mass ? h.mass >= target : h.count >= target;
}

// The first bin at which the head `before` and the bins so far reach the target
// (by count, or by mass), and the head before that bin.
template <int NT>
__device__ void find(Shared<NT> &s, const uint32_t *count, const u64 *mass, Head before, bool by_mass,
                     u64 target)
{
    constexpr int N = Shared<NT>::kBins / NT;
    __syncthreads();              // the last answer has been read, the histogram is whole
    Head own = {0, 0};
    for (int i = 0; i < N; ++i) {
        own.count += count[N * threadIdx.x + i];
        own.mass += mass[N * threadIdx.x + i];
    }
    if (threadIdx.x == 0) s.bin = 0;
    Head h = scan<NT>(s, before, own);
    for (int i = 0; i < N; ++i) {
        const Head next = {h.count + count[N * threadIdx.x + i], h.mass + mass[N * threadIdx.x + i]};
        if (!reaches(h, by_mass, target) && reaches(next, by_mass, target)) {
            s.bin = N * threadIdx.x + i;
            s.before = h;
        }
        h = next;
    }
    __syncthreads();
}

// Where the order reaches a target: the value there, how many of its equals are
// needed, and the head up to and with them.
struct Place {
    uint32_t key, equals;
    Head head;
};

template <int T, int NT>
__device__ Place locate(const SampleArgs &a, int64_t row, const Weights &w, float bin_scale, Shared<NT> &s,
                        bool by_mass, u64 target)
{
    constexpr int kBins = Shared<NT>::kBins;
    find<NT>(s, s.first_count, s.first_mass, {0, 0}, by_mass, target);
    const int first = s.bin;
    Head before = s.before;
    // keys that the bin may hold, a bin's width to spare on either side
    auto bound = [&](double d) { return value_key((float)((double)w.top - d / (double)bin_scale)); };
    uint32_t hi = first <= 0 ? value_key(w.top) : min(value_key(w.top), bound(first - 1.0));
    uint32_t lo = first == kBins - 1 || bin_scale == 0.0f ? kLeastKey : max(kLeastKey, bound(first + 2.0));
    while (lo != hi) {            // kBinBits of the key a turn
        const int shift = max(0, 32 - __clz(hi - lo) - Shared<NT>::kBinBits);
        __syncthreads();
        for (int i = threadIdx.x; i < kBins; i += NT) {
            s.next_count[i] = 0;
            s.next_mass[i] = 0;
        }
        __syncthreads();
        each<T, NT>(a, row, [&](float x, int) {
            const uint32_t k = value_key(x);
            if (k < lo || k > hi) return;
            if ((int)fminf((w.top - x) * bin_scale, (float)(kBins - 1)) != first) return;
            atomicAdd(&s.next_count[(hi - k) >> shift], 1u);
            atomicAdd(&s.next_mass[(hi - k) >> shift], w.units(x));
        });
        find<NT>(s, s.next_count, s.next_mass, before, by_mass, target);
        before = s.before;
        const uint32_t top = hi - ((uint32_t)s.bin << shift);
        lo = max(lo, top - ((1u << shift) - 1));
        hi = top;
    }
    const u64 one = w.units(value_of(hi));
    Place p;
    p.key = hi;
    p.equals = by_mass ? (uint32_t)((target - before.mass + one - 1) / one) : (uint32_t)(target - before.count);
    p.head = {before.count + p.equals, before.mass + p.equals * one};
    return p;
}

// Index of the nth (from 1) logit of the row that has this key.
template <int T, int NT>
__device__ int nth_equal(const SampleArgs &a, int64_t row, uint32_t key, uint32_t nth, Shared<NT> &s)
{
    typedef typename Elem<T>::type E;
    const E *x = (const E *)a.logits + row * a.row_stride;
    const int len = (int)a.n_vocab, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t before = 0;
    if (threadIdx.x == 0) s.index = 0;
    for (int i0 = 0; i0 < len; i0 += NT) {
        const int i = i0 + threadIdx.x;
        const bool eq = i < len && value_key((float)x[i]) == key;
        const u64 in = __ballot(eq);
        __syncthreads();
        if (lane == 0) s.part[wave] = __popcll(in);
        __syncthreads();
        uint32_t rank = before + __popcll(in & ((1ull << lane) - 1)), all = 0;
        for (int w = 0; w < NT / 64; ++w) {
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

__device__ __forceinline__ u64 mass_target(double share, u64 mass)
{
    const u64 t = (u64)ceil(share * (double)mass);
    return t > 0 ? t : 1;
}

// The mass that the drawn token is the first to reach.
__device__ __forceinline__ u64 draw_target(float u, u64 mass)
{
    if (u >= 1.0f) return mass;
    const u64 t = (u64)((u > 0.0f ? (double)u : 0.0) * (double)mass) + 1;     // (NaN as 0)
    return t < mass ? t : mass;
}

__device__ __forceinline__ void answer(const SampleArgs &a, int64_t row, const Weights &w, uint32_t key,
                                       int index, const Head &head)
{
    a.ids[row] = index;
    a.kept[row] = (int32_t)head.count;
    const double lp = (w.t(value_of(key)) - (log2((double)head.mass) - w.bits)) * 0.693147180559945309417;
    a.logprob[row] = (float)fmin(lp, 0.0);
}

// What every answer of a row starts from.
struct Row {
    float top;                    // the largest logit
    uint32_t finite, bad;         // how many are finite; whether one is NaN or +infinity
    double sum;                   // of the weights, where the settings need it
    uint32_t bound;               // the list has all logits with keys from here on
    int listed;
};

// Rows that no list answers: the row is read again for every step.
template <int T, int NT>
__device__ void whole_row(const SampleArgs &a, int64_t row, const Settings &set, const Row &r, Shared<NT> &s)
{
    if (set.greedy) {
        const int i = nth_equal<T, NT>(a, row, value_key(r.top), 1, s);
        if (threadIdx.x == 0) {
            a.ids[row] = i;
            a.kept[row] = 1;
            a.logprob[row] = 0.0f;
        }
        return;
    }
    constexpr int kBins = Shared<NT>::kBins;
    double sum = r.sum;
    if (!set.needs_sum()) {
        const Weights w(r.top, set.scale, 1.0);
        sum = 0.0;
        each<T, NT>(a, row, [&](float x, int) { sum += exp2_64(w.t(x)); });
        sum = block_sum<NT>(sum, s.part);
    }
    const Weights w(r.top, set.scale, sum);
    const float bin_scale = (float)fmin(w.scale * ((kBins - 1) / kReach), 1e30);
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += NT) {
        s.first_count[i] = 0;
        s.first_mass[i] = 0;
    }
    __syncthreads();
    Head least = {0, 0};                       // the tokens that min-p keeps
    each<T, NT>(a, row, [&](float x, int) {
        if (!(x > -INFINITY)) return;
        const int b = (int)fminf((w.top - x) * bin_scale, (float)(kBins - 1));
        const u64 m = w.units(x);
        atomicAdd(&s.first_count[b], 1u);
        atomicAdd(&s.first_mass[b], m);
        if (w.t(x) >= set.least) {
            ++least.count;
            least.mass += m;
        }
    });
    least.count = (uint32_t)block_sum<NT>((u64)least.count, s.part);
    least.mass = block_sum<NT>(least.mass, s.part);
    Head head = {r.finite, 0};
    for (int i = threadIdx.x; i < kBins; i += NT) head.mass += s.first_mass[i];
    head.mass = block_sum<NT>(head.mass, s.part);
    if (set.top_k > 0 && set.top_k < r.finite)
        head = locate<T, NT>(a, row, w, bin_scale, s, false, set.top_k).head;
    if (set.top_p < 1.0)
        head = locate<T, NT>(a, row, w, bin_scale, s, true, mass_target(set.top_p, head.mass)).head;
    if (least.count < head.count) head = least;
    const Place at = locate<T, NT>(a, row, w, bin_scale, s, true, draw_target(set.u, head.mass));
    const int i = nth_equal<T, NT>(a, row, at.key, at.equals, s);
    if (threadIdx.x == 0) answer(a, row, w, at.key, i, head);
}

// ---------------------------------------------------------------------------
// The list of a row, in s.list.

// Where the list reaches a target: its key and the head up to and with it in
// s.key and s.before.  h: the head before the thread's bin; own: the bin's.
// False: too many logits in that bin.
template <int NT, int N>
__device__ bool list_locate(Shared<NT> &s, const Head &h, const Head &own, const u64 (&key)[N],
                            const u64 (&mass)[N], const int (&bin)[N], bool by_mass, u64 target)
{
    __syncthreads();
    if (threadIdx.x == 0) s.members = 0;
    const Head next = {h.count + own.count, h.mass + own.mass};
    if (!reaches(h, by_mass, target) && reaches(next, by_mass, target)) {
        s.bin = threadIdx.x;
        s.before = h;
    }
    __syncthreads();
    const int b = s.bin;
    const Head before = s.before;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (bin[i] == b) {
            const int at = atomicAdd(&s.members, 1);
            if (at < Shared<NT>::kMembers) {
                s.member_key[at] = key[i];
                s.member_mass[at] = mass[i];
            }
        }
    __syncthreads();
    const int n = s.members;
    if (n > Shared<NT>::kMembers) return false;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (bin[i] == b) {
            Head ahead = before;
            for (int j = 0; j < n; ++j)
                if (s.member_key[j] > key[i]) {
                    ++ahead.count;
                    ahead.mass += s.member_mass[j];
                }
            const Head with = {ahead.count + 1, ahead.mass + mass[i]};
            if (!reaches(ahead, by_mass, target) && reaches(with, by_mass, target)) {
                s.key = key[i];
                s.before = with;
            }
        }
    __syncthreads();
    return true;
}

// The row's answers from its list; false where they do not lie in it.
template <int NT>
__device__ bool from_list(const SampleArgs &a, int64_t row, const Settings &set, const Row &r, Shared<NT> &s)
{
    constexpr int kList = Shared<NT>::kList, N = kList / NT;
    const int tid = threadIdx.x, n = r.listed;
    if (n == 0 || n > kList) return false;
    const bool all = (uint32_t)n == r.finite;
    if (set.top_k > 0 && set.top_k < r.finite && set.top_k > (uint32_t)n) return false;
    if (set.greedy) {                          // the largest key
        u64 best = 0;
        for (int i = tid; i < n; i += NT) best = max(best, s.list[i]);
#pragma unroll
        for (int d = 32; d; d >>= 1) best = max(best, (u64)__shfl_xor(best, d));
        if ((tid & 63) == 0) s.part[tid >> 6] = best;
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < NT / 64; ++w) best = max(best, s.part[w]);
            a.ids[row] = key_index(best);
            a.kept[row] = 1;
            a.logprob[row] = 0.0f;
        }
        return true;
    }
    const float low = value_of(r.bound);
    const Weights w(r.top, set.scale, set.needs_sum() ? r.sum : (double)n);
    // bins by value, a bin per thread, down to the bound or to weights of 2^-64
    const float reach = fminf(r.top - low, (float)(kReach / set.scale));
    const float bin_scale = fminf((float)(NT - 1) / reach, 1e30f);
    s.count[tid] = 0;
    s.mass[tid] = 0;
    __syncthreads();
    u64 key[N], mass[N];
    int bin[N];
    Head least = {0, 0};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        bin[i] = -1;
        key[i] = mass[i] = 0;
        if (tid + i * NT < n) {
            key[i] = s.list[tid + i * NT];
            const float x = key_value(key[i]);
            mass[i] = w.units(x);
            bin[i] = (int)fminf((w.top - x) * bin_scale, (float)(NT - 1));
            atomicAdd(&s.count[bin[i]], 1u);
            atomicAdd(&s.mass[bin[i]], mass[i]);
            if (w.t(x) >= set.least) {
                ++least.count;
                least.mass += mass[i];
            }
        }
    }
    __syncthreads();
    const Head own = {s.count[tid], s.mass[tid]};
    const Head h = scan<NT>(s, {0, 0}, own);
    if (tid == NT - 1) s.before = {0, h.mass + own.mass};
    __syncthreads();
    const u64 listed_mass = s.before.mass;
    Head head = {r.finite, listed_mass};
    if (!all && set.needs_sum()) head.mass = (u64)(r.sum * __builtin_amdgcn_ldexp(1.0, w.bits));
    if (set.top_k > 0 && set.top_k < r.finite) {
        if (!list_locate<NT, N>(s, h, own, key, mass, bin, false, set.top_k)) return false;
        head = s.before;
    } else if (!all && !set.needs_sum())
        return false;                          // top-k of more than there are
    if (set.top_p < 1.0) {
        const u64 target = mass_target(set.top_p, head.mass);
        if (target > listed_mass || !list_locate<NT, N>(s, h, own, key, mass, bin, true, target)) return false;
        head = s.before;
    }
    if (set.least > -INFINITY) {
        // the tokens that min-p keeps are all listed, or all that is listed is among them
        if (all || w.t(low) < set.least) {
            least.count = (uint32_t)block_sum<NT>((u64)least.count, s.part);
            least.mass = block_sum<NT>(least.mass, s.part);
            if (least.count < head.count) head = least;
        } else if (head.count > (uint32_t)n)
            return false;
    }
    const u64 target = draw_target(set.u, head.mass);
    if (target > listed_mass || !list_locate<NT, N>(s, h, own, key, mass, bin, true, target)) return false;
    if (tid == 0) answer(a, row, w, (uint32_t)(s.key >> 32), key_index(s.key), head);
    return true;
}

template <int T, int NT>
__device__ void row_answers(const SampleArgs &a, int64_t row, const Settings &set, const Row &r, Shared<NT> &s)
{
    if (r.bad || !r.finite) {
        if (threadIdx.x == 0) {
            a.ids[row] = -1;
            a.kept[row] = 0;
            a.logprob[row] = r.bad ? __builtin_nanf("") : -INFINITY;
        }
        return;
    }
    if (from_list<NT>(a, row, set, r, s)) return;
    __syncthreads();
    whole_row<T, NT>(a, row, set, r, s);
}

// ---------------------------------------------------------------------------
// Logits in registers: `E` of them a thread, of a stretch of a row.

template <int T, int NT, int E>
struct Held {
    static constexpr int V = kVec<T>, N = E / V;
    u32x4 raw[N];
    int begin;                    // index of the stretch in its row

    // logits begin .. begin + len - 1; those beyond are -infinity
    __device__ __forceinline__ void load(const SampleArgs &a, int64_t row, int first, int len)
    {
        typedef typename Elem<T>::type El;
        begin = first;
        const El *x = (const El *)a.logits + row * a.row_stride + first;
        const uint32_t none = T == Q8_T_F32 ? 0xff800000u : T == Q8_T_F16 ? 0xfc00fc00u : 0xff80ff80u;
#pragma unroll
        for (int v = 0; v < N; ++v) {
            const int i = (threadIdx.x + v * NT) * V;
            if (i + V <= len)
                raw[v] = *(const u32x4_any *)(x + i);
            else {
                raw[v] = (u32x4){none, none, none, none};
                if (i < len) {
                    float y[V];
#pragma unroll
                    for (int j = 0; j < V; ++j) y[j] = i + j < len ? (float)x[i + j] : -INFINITY;
                    raw[v] = pack_vec<T>(y);
                }
            }
        }
    }
    template <class F>
    __device__ __forceinline__ void each(F f) const
    {
#pragma unroll
        for (int v = 0; v < N; ++v) {
            float y[V];
            unpack16<T>(raw[v], y);
#pragma unroll
            for (int j = 0; j < V; ++j) f(y[j], begin + (int)(threadIdx.x + v * NT) * V + j);
        }
    }
};

// The largest logit of the stretch and of this thread, how many are finite and
// whether one is NaN or +infinity, and the weights' sum beside the largest.
struct Stretch {
    float top, own_top;
    uint32_t finite, bad;
    double sum;
};

template <int T, int NT, int E>
__device__ Stretch stretch(const Held<T, NT, E> &x, const Settings &set, int len, u64 *part)
{
    Stretch r = {-INFINITY, -INFINITY, 0, 0, 0.0};
    float lowest = INFINITY;
    bool bad = false;
    x.each([&](float v, int) {
        r.own_top = fmaxf(r.own_top, v);
        lowest = fminf(lowest, v);
        bad |= v != v;
    });
    bad |= r.own_top == INFINITY;
    uint32_t finite = 0;
    if (lowest == -INFINITY) x.each([&](float v, int) { finite += v > -INFINITY; });
    else finite = E;
    r.top = r.own_top;
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        r.top = fmaxf(r.top, __shfl_xor(r.top, d));
        finite += __shfl_xor(finite, d);
    }
    const u64 any = __ballot(bad);
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
        part[wave] = (u64)__builtin_bit_cast(uint32_t, r.top) << 32 | finite << 1 | (any != 0);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        r.top = fmaxf(r.top, __builtin_bit_cast(float, (uint32_t)(part[w] >> 32)));
        r.finite += (uint32_t)part[w] >> 1;
        r.bad |= (uint32_t)part[w] & 1;
    }
    if (set.needs_sum() && r.top > -INFINITY && !r.bad) {
        // (the difference first: v * scale - top * scale would round masks near the
        // type's lowest value apart)
        const double top = r.top;
        double sum = 0.0;
        x.each([&](float v, int) { sum += exp2_64(((double)v - top) * set.scale); });
        r.sum = block_sum<NT>(sum, part);
    }
    return r;
}

// A key that `rank` or more logits of the workgroup reach: that of the rank-th
// of 256 groups' maxima, its low half cut.
template <int NT>
__device__ uint32_t list_bound(float own_top, int rank, uint32_t *keys)
{
    uint32_t k = value_key(own_top);
    if constexpr (NT == 1024) {
        k = max(k, (uint32_t)__shfl_xor((int)k, 1));
        k = max(k, (uint32_t)__shfl_xor((int)k, 2));
        if ((threadIdx.x & 3) == 0) keys[threadIdx.x >> 2] = k;
    } else
        keys[threadIdx.x] = k;
    __syncthreads();
    return max(nth_key(((const u32x4 *)keys)[threadIdx.x & 63], rank), kLeastKey);
}

// ---------------------------------------------------------------------------
// A row per workgroup.
template <int T, int NT, int E>
__global__ __launch_bounds__(NT) void sample_row_kernel(const SampleArgs a)
{
    __shared__ Shared<NT> s;
    const int64_t row = blockIdx.x;
    const int len = (int)a.n_vocab, lane = threadIdx.x & 63;
    Held<T, NT, E> x;
    x.load(a, row, 0, len);
    const Settings set(a, row);
    if (threadIdx.x == 0) s.listed = 0;
    const Stretch st = stretch<T, NT, E>(x, set, len, s.part);
    Row r;
    r.top = st.top; r.finite = st.finite; r.bad = st.bad; r.sum = st.sum;
    r.bound = list_bound<NT>(st.own_top, 128, s.keys);
    __syncthreads();              // (the list lies where the keys were)
    const float low = value_of(r.bound);
    x.each([&](float v, int i) {
        const u64 in = __ballot(v >= low);
        if (!in) return;
        int at = 0;
        if (lane == 0) at = atomicAdd(&s.listed, (int)__popcll(in));
        at = wave_uniform(at) + __builtin_amdgcn_mbcnt_hi((uint32_t)(in >> 32),
                                                          __builtin_amdgcn_mbcnt_lo((uint32_t)in, 0));
        if (v >= low && at < Shared<NT>::kList) s.list[at] = order_key(v, (uint32_t)i);
    });
    __syncthreads();
    r.listed = s.listed;
    row_answers<T, NT>(a, row, set, r, s);
}

// A part of a row per workgroup, and the join of a row's parts.
constexpr int kPartWaves = 4, kPartThreads = 64 * kPartWaves;

struct PartOut {
    double sum;
    float top;
    uint32_t bound, finite, bad;
    int listed[kPartWaves];
};

struct Work {
    PartOut *parts;               // [m][parts]
    u64 *lists;                   // [m][parts][kPartWaves][kPlaces]
    int n_parts, rank;
};

template <int T, int E>
__global__ __launch_bounds__(kPartThreads) void sample_part_kernel(const SampleArgs a, const Work w)
{
    __shared__ u64 part[kPartWaves];
    __shared__ __align__(16) uint32_t keys[256];
    __shared__ PartOut out;
    const int64_t row = blockIdx.y;
    const int wave = wave_uniform((int)(threadIdx.x >> 6));
    const int first = blockIdx.x * kPartThreads * E, len = min(kPartThreads * E, (int)a.n_vocab - first);
    Held<T, kPartThreads, E> x;
    x.load(a, row, first, len);
    const Settings set(a, row);
    const Stretch st = stretch<T, kPartThreads, E>(x, set, len, part);
    uint32_t bound = list_bound<kPartThreads>(st.own_top, w.rank, keys);
    const float low = value_of(bound);
    const int64_t at = row * w.n_parts + blockIdx.x;
    u64 *list = w.lists + (at * kPartWaves + wave) * kPlaces;
    int listed = 0;
    x.each([&](float v, int i) {
        const u64 in = __ballot(v >= low);
        if (!in) return;
        const int p = listed + __builtin_amdgcn_mbcnt_hi((uint32_t)(in >> 32),
                                                         __builtin_amdgcn_mbcnt_lo((uint32_t)in, 0));
        if (v >= low && p < kPlaces) list[p] = order_key(v, (uint32_t)i);
        listed += __popcll(in);
    });
    if ((threadIdx.x & 63) == 0) out.listed[wave] = listed;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kPartWaves; ++i)
            if (out.listed[i] > kPlaces) bound = kNoBound;
        out.sum = st.sum; out.top = st.top; out.bound = bound; out.finite = st.finite; out.bad = st.bad;
        w.parts[at] = out;
    }
}

template <int T>
__global__ __launch_bounds__(1024) void sample_join_kernel(const SampleArgs a, const Work w)
{
    constexpr int NT = 1024;
    __shared__ Shared<NT> s;
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const Settings set(a, row);
    const PartOut *parts = w.parts + row * w.n_parts;
    PartOut p;
    p.top = -INFINITY; p.bound = 0; p.finite = 0; p.bad = 0; p.sum = 0.0;
    if (tid < w.n_parts) p = parts[tid];
    if (tid == 0) s.listed = 0;
    Row r;
    // (the largest of the keys; a row that is all -infinity has the key of that)
    u64 best = (u64)value_key(p.top) << 32 | p.bound;
    uint32_t top = (uint32_t)(best >> 32), bound = (uint32_t)best;
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        top = max(top, (uint32_t)__shfl_xor((int)top, d));
        bound = max(bound, (uint32_t)__shfl_xor((int)bound, d));
    }
    if (lane == 0) s.part[wave] = (u64)top << 32 | bound;
    __syncthreads();
    for (int i = 0; i < NT / 64; ++i) {
        top = max(top, (uint32_t)(s.part[i] >> 32));
        bound = max(bound, (uint32_t)s.part[i]);
    }
    r.top = value_of(top);
    r.bound = bound;
    const u64 counts = block_sum<NT>((u64)p.bad << 32 | p.finite, s.part);
    r.finite = (uint32_t)counts;
    r.bad = (uint32_t)(counts >> 32);
    r.sum = 0.0;
    if (set.needs_sum() && !r.bad && r.finite)
        r.sum = block_sum<NT>(p.sum > 0.0 ? p.sum * exp2_64(((double)p.top - (double)r.top) * set.scale) : 0.0,
                              s.part);
    if (r.bound != kNoBound) {
        const u64 *lists = w.lists + row * w.n_parts * (kPartWaves * kPlaces);
        for (int l = wave; l < w.n_parts * kPartWaves; l += NT / 64) {
            const int n = parts[l / kPartWaves].listed[l % kPartWaves];
            for (int i = lane; i - lane < n; i += 64) {
                const u64 key = i < n ? lists[l * kPlaces + i] : 0;
                const bool real = (uint32_t)(key >> 32) >= r.bound && i < n;
                const u64 in = __ballot(real);
                int at = 0;
                if (lane == 0) at = atomicAdd(&s.listed, (int)__popcll(in));
                at = wave_uniform(at) + __builtin_amdgcn_mbcnt_hi((uint32_t)(in >> 32),
                                                                  __builtin_amdgcn_mbcnt_lo((uint32_t)in, 0));
                if (real && at < Shared<NT>::kList) s.list[at] = key;
            }
        }
    }
    __syncthreads();
    r.listed = s.listed;
    row_answers<T, NT>(a, row, set, r, s);
}

// Rows of up to 65536 logits are held whole; longer ones in parts.
constexpr int kPartLogits = 16384;

int64_t n_parts(int64_t n_vocab)
{
    return n_vocab <= 65536 ? 0 : (n_vocab + kPartLogits - 1) / kPartLogits;
}

constexpr int64_t kPartBytes = sizeof(PartOut) + sizeof(u64) * kPartWaves * kPlaces;

template <int T, int NT, int E>
int launch_row(const SampleArgs &a, hipStream_t stream)
{
    // (2^32 threads bound a launch)
    constexpr int64_t most = (int64_t)1 << 21;
    for (int64_t i = 0; i < a.m; i += most) {
        SampleArgs b = a;
        b.m = a.m - i < most ? a.m - i : most;
        b.logits = (const uint8_t *)a.logits + i * a.row_stride * (T == Q8_T_F32 ? 4 : 2);
        b.u += i; b.ids += i; b.logprob += i; b.kept += i;
        if (b.temperature) b.temperature += i;
        if (b.top_k) b.top_k += i;
        if (b.top_p) b.top_p += i;
        if (b.min_p) b.min_p += i;
        hipLaunchKernelGGL((sample_row_kernel<T, NT, E>), dim3((unsigned)b.m), dim3(NT), 0, stream, b);
        if (hipGetLastError() != hipSuccess) return -6;
    }
    return 0;
}

template <int T>
int launch_parts(const SampleArgs &a, void *ws, hipStream_t stream)
{
    const int64_t parts = n_parts(a.n_vocab);
    // (65535 rows bound a grid's second dimension)
    constexpr int64_t most = 65535;
    for (int64_t i = 0; i < a.m; i += most) {
        SampleArgs b = a;
        b.m = a.m - i < most ? a.m - i : most;
        b.logits = (const uint8_t *)a.logits + i * a.row_stride * (T == Q8_T_F32 ? 4 : 2);
        b.u += i; b.ids += i; b.logprob += i; b.kept += i;
        if (b.temperature) b.temperature += i;
        if (b.top_k) b.top_k += i;
        if (b.top_p) b.top_p += i;
        if (b.min_p) b.min_p += i;
        Work w;
        w.lists = (u64 *)ws;
        w.parts = (PartOut *)(w.lists + b.m * parts * (kPartWaves * kPlaces));
        w.n_parts = (int)parts;
        const int64_t rank = 2048 / parts;
        w.rank = (int)(rank < 32 ? 32 : rank > 128 ? 128 : rank);
        hipLaunchKernelGGL((sample_part_kernel<T, kPartLogits / kPartThreads>), dim3((unsigned)parts, (unsigned)b.m),
                           dim3(kPartThreads), 0, stream, b, w);
        if (hipGetLastError() != hipSuccess) return -6;
        hipLaunchKernelGGL((sample_join_kernel<T>), dim3((unsigned)b.m), dim3(1024), 0, stream, b, w);
        if (hipGetLastError() != hipSuccess) return -6;
    }
    return 0;
}

template <int T>
int launch_type(const SampleArgs &a, void *ws, hipStream_t stream)
{
    if (n_parts(a.n_vocab)) return launch_parts<T>(a, ws, stream);
    if (a.n_vocab <= 4096) return launch_row<T, 256, 16>(a, stream);
    if (a.n_vocab <= 16384) return launch_row<T, 1024, 16>(a, stream);
    if (a.n_vocab <= 32768) return launch_row<T, 1024, 32>(a, stream);
    return launch_row<T, 1024, 64>(a, stream);
}

}  // namespace

size_t sample_ws_bytes(int64_t m, int64_t n_vocab)
{
    const int64_t rows = m < 65535 ? m : 65535, parts = n_parts(n_vocab);
    const int64_t b = rows * parts * kPartBytes;
    return (size_t)(b > 256 ? b : 256);
}

int launch_sample(const SampleArgs &a, void *ws, hipStream_t stream)
{
    if (a.type == Q8_T_F32) return launch_type<Q8_T_F32>(a, ws, stream);
    if (a.type == Q8_T_F16) return launch_type<Q8_T_F16>(a, ws, stream);
    return launch_type<Q8_T_BF16>(a, ws, stream);
}

}  // namespace q8
