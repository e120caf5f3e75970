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
// falls between tokens as it does in 64 bits.  The mass of a row that nothing cuts
// is, where its list answers it, the 64-bit floating-point sum instead, whose
// order is fixed (its parts have no common unit before the largest is known).
//
// The logits are read once.  A workgroup takes a short row, a wave a part of a long
// one, sums its weights where a filter needs the sum, and lists the logits that
// reach a bound: as many lanes' maxima do as are wanted.  The list is a head of
// the row's order (down to the largest bound of its parts), and where the answers
// lie in it, as they do for most rows, it alone is looked at further.  The other
// rows (a head that goes beyond the list, many equal logits) are read again: for a
// histogram of all their weights, by many workgroups where calls are large, and
// for the logits of each bin that holds an answer.
//
// A sum in 64 bits costs 20 vector instructions a logit, one in 32 bits 7.  For
// top-p the latter is enough where the answer is the same over the range of its
// error; the few rows where it is not are read again.
//
// Bounds: vector instructions for many long rows (512 x 262144 bfloat16, top-p:
// parts 59 us, of which the pipe is busy 75%, join 12; HBM's floor 38); else the
// chain of launches, round trips and barriers: 1 x 32000 5.9 + 11.5 us, 8 x 262144
// 6.6 + 13, 333 x 50257 with settings of their own 20 + 13, and 7 + 26 where a row
// is read again.  These times are those of likely tokens all over the vocabulary and
// masks of -infinity: a part that holds most of them, or one whose mask is finite and
// leaves it fewer tokens than its list asks for, sends the row to be read again.
#include "i8_device.h"
#include "order_device.h"
#include "q8_ops.h"

namespace q8 {

namespace {

typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef unsigned long long u64;

constexpr float kReach = 64.0f;   // a histogram by value covers weights down to 2^-64
constexpr int kPlaces = 128;      // listed logits of a part
constexpr int kRank = 128;        // how many maxima reach a list's bound, of 256: at most

// 2^t for t <= 0 (2^-1000 below -1000), off by 1.55e-14 at most: 2^r on [-1/2, 1/2]
// as a polynomial of degree 9 that is 1 at 0 (the coefficients by the exchange
// algorithm; 1.513e-14, the rest its roundings).  The nearest whole number comes from a sum with 1.5 * 2^52, whose
// low bits hold it: the conversions, rounding and scaling instructions of fp64
// issue at a quarter of the rate of its sums and products.
__device__ __forceinline__ double exp2_64(double t)
{
    constexpr double kWhole = 0x1.8p52;
    t = fmax(t, -1000.0);
    const double y = t + kWhole, r = t - (y - kWhole);
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
    const u32x2 n = __builtin_bit_cast(u32x2, y), v = __builtin_bit_cast(u32x2, p);
    return __builtin_bit_cast(double, (u32x2){v.x, v.y + (n.x << 20)});
}

constexpr uint32_t kLeastKey = 0x00800000u;       // value_key of the lowest finite value
constexpr uint32_t kNoBound = 0xffffffffu;        // of a part that has no list

__device__ __forceinline__ float value_of(uint32_t key) { return key_value((uint64_t)key << 32); }

// Half of how far x lies below `top` (finite values: the whole distance may pass
// fp32's range, as between masks of either sign), in one rounding.
__device__ __forceinline__ float half_below(float top, float x) { return fmaf(-0.5f, x, 0.5f * top); }

// The bin of x in a histogram by value.
__device__ __forceinline__ int value_bin(float top, float x, float bin_scale, int bins)
{
    return (int)fminf(half_below(top, x) * (2.0f * bin_scale), (float)(bins - 1));
}

// A row's settings, as they are applied.
struct Settings {
    float u;
    double scale;                 // log2(e) / T; 0: the largest logit
    uint32_t top_k;               // 0: all
    double top_p;                 // 1: all
    float min_p;                  // 0: all
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
        min_p = m > 0.0f ? m : 0.0f;
    }
    // the least distance to the largest logit that min-p keeps, in powers of two
    __device__ __forceinline__ double least() const
    {
        return min_p > 0.0f ? fmin(log2((double)min_p), 0.0) : -INFINITY;
    }
    // The sum of a row's weights: not needed where a head of the order is cut
    // without it; in 32 bits for a share of it; in 64 bits as the mass of a row
    // that nothing cuts (and where a scale does not fit 32 bits).
    enum Sum { kNone, kRough, kFull };
    __device__ __forceinline__ Sum sum() const
    {
        if (greedy || top_k > 0 || (top_p >= 1.0 && min_p > 0.0f)) return kNone;
        return top_p < 1.0 && scale > 1e-30 && scale < 1e30 ? kRough : kFull;
    }
};

// How far a rough sum may be off, relative: with |t| the distance to the largest
// logit in powers of two, a term carries 2 2^-24 ln 2 |t| (the scale, the fused
// product) and 2^-23 (the exponential); over a part of up to 2^13 logits beside
// its largest the weights' mean of |t| is below 9 (n - 1 terms at s = 10 make the
// most of (n - 1) s 2^-s / (1 + (n - 1) 2^-s)); the sums of 8 add 3 2^-24, the
// rounding of the product with the largest logit, at most 2^-4, taken out by a
// factor, 2^-23 and 2^-28: 1.2e-6 in all.
constexpr double kRoughError = 0x1p-19;

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
    __device__ __forceinline__ u64 units_at(double t) const
    {
        return __builtin_bit_cast(u64, exp2_64(t) + unit) - __builtin_bit_cast(u64, unit);
    }
    __device__ __forceinline__ u64 units(float x) const { return units_at(t(x)); }
};

struct Head {                     // tokens at the head of the order
    uint32_t count;
    u64 mass;
};

// ---------------------------------------------------------------------------
// By a workgroup of NT threads.

template <int NT>
struct __align__(16) Shared {
    static constexpr int kBins = 4 * NT;               // of a histogram of the row
    static constexpr int kBinBits = NT == 512 ? 11 : 10;
    static constexpr int kList = 8 * NT;               // logits of a list
    static constexpr int kMembers = 2 * NT;            // of one bin of a list
    static_assert(kBins == 1 << kBinBits, "bins by powers of two");
    union {
        uint32_t keys[256];
        struct {                  // a list, in bins by value
            u64 list[kList], mass[NT], member_key[kMembers], member_mass[kMembers];
            uint32_t count[NT];
        };
        struct {                  // a histogram of part of the row
            u64 next_mass[kBins];
            uint32_t next_count[kBins];
        };
    };
    u64 first_mass[kBins];        // of the whole row
    uint32_t first_count[kBins];
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
    constexpr int V = kVec<T>, kAhead = 4;
    const E *x = (const E *)a.logits + row * a.row_stride;
    const int len = (int)a.n_vocab, vecs = len / V;
    for (int v = threadIdx.x; v < vecs; v += kAhead * NT) {
        u32x4 raw[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) raw[u] = *(const u32x4_any *)(x + min(v + u * NT, vecs - 1) * V);
#pragma unroll 1
        for (int u = 0; u < kAhead; ++u) {
            if (v + u * NT >= vecs) break;
            float y[V];
            unpack16<T>(raw[0], y);
            raw[0] = raw[1]; raw[1] = raw[2]; raw[2] = raw[3];
#pragma unroll
            for (int j = 0; j < V; ++j) f(y[j], (v + u * NT) * V + j);
        }
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
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        const Head o = s.wave[w];
        before.count += w < wave ? o.count : 0u;
        before.mass += w < wave ? o.mass : 0ull;
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

__device__ __forceinline__ u64 mass_target(double share, double mass)
{
    const u64 t = (u64)ceil(share * mass);
    return t > 0 ? t : 1;
}

// The mass that the drawn token is the first to reach.
__device__ __forceinline__ u64 draw_target(float u, u64 mass)
{
    if (u >= 1.0f) return mass;
    return min((u64)((u > 0.0f ? (double)u : 0.0) * (double)mass) + 1, mass);   // (NaN as 0)
}

__device__ __forceinline__ void answer(const SampleArgs &a, int64_t row, const Weights &w, u64 key,
                                       const Head &head)
{
    a.ids[row] = key_index(key);
    a.kept[row] = (int32_t)head.count;
    const double lp = (w.t(key_value(key)) - (log2((double)head.mass) - w.bits)) * 0.693147180559945309417;
    a.logprob[row] = (float)fmin(lp, 0.0);
}

__device__ __forceinline__ void greedy_answer(const SampleArgs &a, int64_t row, int index)
{
    a.ids[row] = index;
    a.kept[row] = 1;
    a.logprob[row] = 0.0f;
}

// What every answer of a row starts from.
struct Row {
    float top;                    // the largest logit
    uint32_t finite, bad;         // how many are finite; whether one is NaN or +infinity
    double sum;                   // of the weights, as the settings have it
    uint32_t bound;               // the list has all logits with keys from here on
    int listed;
};

// ---------------------------------------------------------------------------
// The logits of a list, some per thread, in bins by value: a bin per thread.
template <int NT>
struct Listed {
    static constexpr int N = Shared<NT>::kList / NT;
    u64 key[N], mass[N];
    int bin[N];
    Head h, own;                  // the head before this thread's bin; the bin
    u64 end;                      // the mass of the head with the whole list

    __device__ __forceinline__ void take(Shared<NT> &s, int n)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = threadIdx.x + i * NT;
            key[i] = at < n ? s.list[at] : 0;
        }
    }
    // high, low: no listed value is outside; before: the head before the list
    __device__ void sort(Shared<NT> &s, const Weights &w, float high, float low, Head before)
    {
        const float reach = fminf(half_below(high, low), (float)(0.5 * kReach / w.scale));
        const float bin_scale = fminf((float)(NT - 1) / reach, 1e30f);      // of half distances
        __syncthreads();
        s.count[threadIdx.x] = 0;
        s.mass[threadIdx.x] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            bin[i] = -1;
            mass[i] = 0;
            if (key[i]) {
                const float x = key_value(key[i]);
                mass[i] = w.units(x);
                bin[i] = (int)fminf(half_below(high, x) * bin_scale, (float)(NT - 1));
                atomicAdd(&s.count[bin[i]], 1u);
                atomicAdd(&s.mass[bin[i]], mass[i]);
            }
        }
        __syncthreads();
        own = {s.count[threadIdx.x], s.mass[threadIdx.x]};
        h = scan<NT>(s, before, own);
        if (threadIdx.x == NT - 1) s.before = {0, h.mass + own.mass};
        __syncthreads();
        end = s.before.mass;
    }
    // Where the order reaches a target: its key and the head up to and with it in
    // s.key and s.before.  False: not in the list, or too many logits in a bin.
    __device__ bool locate(Shared<NT> &s, bool by_mass, u64 target) const
    {
        if (by_mass && target > end) return false;
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
        // eight lanes to a member count what is ahead of it
        const int sub = threadIdx.x & 7;
        for (int c = threadIdx.x >> 3; c < n; c += NT / 8) {
            const u64 k = s.member_key[c];
            Head ahead = {0, 0};
            for (int j = sub; j < n; j += 8)
                if (s.member_key[j] > k) {
                    ++ahead.count;
                    ahead.mass += s.member_mass[j];
                }
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) {
                ahead.count += __shfl_xor(ahead.count, d);
                ahead.mass += __shfl_xor(ahead.mass, d);
            }
            ahead.count += before.count;
            ahead.mass += before.mass;
            const Head with = {ahead.count + 1, ahead.mass + s.member_mass[c]};
            if (sub == 0 && !reaches(ahead, by_mass, target) && reaches(with, by_mass, target)) {
                s.key = k;
                s.before = with;
            }
        }
        __syncthreads();
        return true;
    }
    // The listed tokens that min-p keeps.
    __device__ Head least(Shared<NT> &s, const Weights &w, double least) const
    {
        Head l = {0, 0};
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (key[i] && w.t(key_value(key[i])) >= least) {
                ++l.count;
                l.mass += mass[i];
            }
        l.count = (uint32_t)block_sum<NT>((u64)l.count, s.part);
        l.mass = block_sum<NT>(l.mass, s.part);
        return l;
    }
};

// The row's answers from its list; false where they do not lie in it.  sum: what
// r.sum is.
template <int NT>
__device__ __forceinline__ bool from_list(const SampleArgs &a, int64_t row, const Settings &set, const Row &r,
                                          Settings::Sum sum, Shared<NT> &s, Listed<NT> &l)
{
    const int tid = threadIdx.x, n = r.listed;
    const bool all = (uint32_t)n == r.finite, cut = set.top_k > 0 && set.top_k < r.finite;
    if (cut && set.top_k > (uint32_t)n) return false;
    if (set.greedy) {                          // the largest key
        u64 best = 0;
#pragma unroll
        for (int i = 0; i < Listed<NT>::N; ++i) best = max(best, l.key[i]);
#pragma unroll
        for (int d = 32; d; d >>= 1) best = max(best, (u64)__shfl_xor(best, d));
        if ((tid & 63) == 0) s.part[tid >> 6] = best;
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < NT / 64; ++w) best = max(best, s.part[w]);
            greedy_answer(a, row, key_index(best));
        }
        return true;
    }
    const float low = value_of(r.bound);
    const Weights w(r.top, set.scale, sum != Settings::kNone ? r.sum : (double)n);
    l.sort(s, w, r.top, low, {0, 0});
    // the head so far, the mass that shares are of and how far it may be off
    Head head = {r.finite, l.end};
    double mass = (double)l.end, off = 0.0;
    bool whole = !all;                         // the head goes beyond the list
    if (!all && sum != Settings::kNone) {
        mass = r.sum * __builtin_amdgcn_ldexp(1.0, w.bits);
        head.mass = (u64)mass;
        off = sum == Settings::kRough ? kRoughError : 0.0;
    }
#pragma unroll 1
    for (int step = 0; step < 3; ++step) {     // top-k, top-p, the draw
        u64 target = set.top_k;
        if (step == 0 && !cut) continue;
        if (step == 1) {
            if (set.top_p >= 1.0) continue;
            if (whole && sum == Settings::kNone) return false;      // (top-k of all there are)
            target = mass_target(set.top_p, mass * (1.0 - off));
        }
        if (step == 2) {
            // the tokens that min-p keeps are all listed, or all that is listed is among them
            const double reach = set.least();
            if (set.min_p > 0.0f && (all || w.t(low) < reach)) {
                const Head least = l.least(s, w, reach);
                if (least.count < head.count) {
                    head = least;
                    whole = false;
                }
            }
            // (the last token that has mass is that of the whole units)
            if (whole && (sum != Settings::kFull || set.u >= 1.0f)) return false;
            target = draw_target(set.u, head.mass);
        }
        if (!l.locate(s, step > 0, target)) return false;
        if (step == 2) break;
        head = s.before;
        if (step == 1 && head.mass < mass_target(set.top_p, mass * (1.0 + off))) return false;
        mass = (double)head.mass;
        off = 0.0;
        whole = false;
    }
    if (tid == 0) answer(a, row, w, s.key, head);
    return true;
}

// ---------------------------------------------------------------------------
// Rows that the list does not answer.

// Index of the nth (from 1) logit of the row that has this key: the waves count
// a stretch each, and the one that has it looks for it.
template <int T, int NT>
__device__ int nth_equal(const SampleArgs &a, int64_t row, uint32_t key, uint32_t nth, Shared<NT> &s)
{
    typedef typename Elem<T>::type E;
    const E *x = (const E *)a.logits + row * a.row_stride;
    const int len = (int)a.n_vocab, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int per = ((len + NT - 1) / NT) * 64, begin = min(wave * per, len), end = min(begin + per, len);
    uint32_t count = 0;
#pragma unroll 8
    for (int i = begin + lane; i < end; i += 64) count += value_key((float)x[i]) == key;
#pragma unroll
    for (int d = 32; d; d >>= 1) count += __shfl_xor(count, d);
    __syncthreads();
    if (threadIdx.x == 0) s.index = 0;
    if (lane == 0) s.part[wave] = count;
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < wave; ++w) before += (uint32_t)s.part[w];
    if (before < nth && nth <= before + count)
        for (int i0 = begin; i0 < end; i0 += 64) {
            const bool eq = i0 + lane < end && value_key((float)x[i0 + lane]) == key;
            const u64 in = __ballot(eq);
            if (eq && before + __popcll(in & ((1ull << lane) - 1)) + 1 == nth) s.index = i0 + lane;
            before += __popcll(in);
            if (before >= nth) break;
        }
    __syncthreads();
    return s.index;
}

// Where the order reaches a target, from the row: the key with its index in s.key
// (`index`), and the head up to and with it, returned.  known: the row's list,
// which has all keys from `known_from` on.
template <int T, int NT>
__device__ __forceinline__ Head locate(const SampleArgs &a, int64_t row, const Weights &w, float bin_scale,
                                       Shared<NT> &s, const Listed<NT> &known, uint32_t known_from,
                                       bool by_mass, u64 target, bool index)
{
    constexpr int kBins = Shared<NT>::kBins;
    find<NT>(s, s.first_count, s.first_mass, {0, 0}, by_mass, target);
    const int first = s.bin;
    uint32_t count = s.first_count[first];
    Head before = s.before;
    // keys that the bin may hold, a bin's width to spare on either side (a logit of the
    // bin lies between the bounds, so that lo <= hi, and every turn below shortens them)
    auto bound = [&](double d) { return value_key((float)((double)w.top - d / (double)bin_scale)); };
    uint32_t hi = first <= 0 ? value_key(w.top) : min(value_key(w.top), bound(first - 1.0));
    uint32_t lo = first == kBins - 1 || bin_scale == 0.0f ? kLeastKey : max(kLeastKey, bound(first + 2.0));
    auto inside = [&](float x, uint32_t k) {
        return k >= lo && k <= hi && value_bin(w.top, x, bin_scale, kBins) == first;
    };
    while (lo < hi) {
        __syncthreads();
        if (count <= Shared<NT>::kList) {      // its logits as a list
            if (threadIdx.x == 0) s.listed = 0;
            __syncthreads();
            const float low = value_of(lo), high = value_of(hi);
            auto take = [&](float x, int i) {
                if (!(x >= low && x <= high)) return;
                const u64 key = order_key(x, (uint32_t)i);
                if (!inside(x, (uint32_t)(key >> 32))) return;
                const int at = atomicAdd(&s.listed, 1);
                if (at < Shared<NT>::kList) s.list[at] = key;
            };
            if (lo >= known_from) {
                for (int i = 0; i < Listed<NT>::N; ++i)
                    if (known.key[i]) take(key_value(known.key[i]), key_index(known.key[i]));
            } else
                each<T, NT>(a, row, take);
            __syncthreads();
            Listed<NT> l;
            l.take(s, min(s.listed, Shared<NT>::kList));
            l.sort(s, w, value_of(hi), value_of(lo), before);
            if (l.locate(s, by_mass, target)) return s.before;
            __syncthreads();
            count = Shared<NT>::kList + 1;
        }
        // else in bins by key, kBinBits of it a turn
        const int shift = max(0, 32 - __clz(hi - lo) - Shared<NT>::kBinBits);
        for (int i = threadIdx.x; i < kBins; i += NT) {
            s.next_count[i] = 0;
            s.next_mass[i] = 0;
        }
        __syncthreads();
        each<T, NT>(a, row, [&](float x, int) {
            const uint32_t k = value_key(x);
            if (!inside(x, k)) return;
            atomicAdd(&s.next_count[(hi - k) >> shift], 1u);
            atomicAdd(&s.next_mass[(hi - k) >> shift], w.units(x));
        });
        find<NT>(s, s.next_count, s.next_mass, before, by_mass, target);
        before = s.before;
        count = s.next_count[s.bin];
        const uint32_t top = hi - ((uint32_t)s.bin << shift);
        lo = max(lo, top - ((1u << shift) - 1));
        hi = top;
    }
    const u64 one = w.units(value_of(hi));
    const uint32_t equals = by_mass ? (uint32_t)((target - before.mass + one - 1) / one)
                                    : (uint32_t)(target - before.count);
    if (index) {
        const int i = nth_equal<T, NT>(a, row, hi, equals, s);
        if (threadIdx.x == 0) s.key = order_key(value_of(hi), (uint32_t)i);
    }
    return {before.count + equals, before.mass + equals * one};
}

// The histogram of a row by value.
__device__ __forceinline__ float row_bin_scale(const Weights &w, int bins)
{
    return (float)fmin(w.scale * ((bins - 1) / kReach), 1e30);
}

template <int BINS>
struct RowBins {
    const Weights &w;
    float bin_scale;
    double least;
    Head kept;                    // the tokens that min-p keeps, of this thread
    __device__ __forceinline__ RowBins(const Weights &w, double least)
        : w(w), bin_scale(row_bin_scale(w, BINS)), least(least), kept({0, 0})
    {
    }
    __device__ __forceinline__ void add(float x, uint32_t *count, u64 *mass)
    {
        if (!(x > -INFINITY)) return;
        const int b = value_bin(w.top, x, bin_scale, BINS);
        const double t = w.t(x);
        const u64 m = w.units_at(t);
        atomicAdd(&count[b], 1u);
        atomicAdd(&mass[b], m);
        if (t >= least) {
            ++kept.count;
            kept.mass += m;
        }
    }
};

// The row's answers from its histogram (s.first_*) and the row.  least: the
// tokens that min-p keeps; l has all the row's keys from known_from on.
template <int T, int NT>
__device__ __forceinline__ void from_bins(const SampleArgs &a, int64_t row, const Settings &set, uint32_t finite,
                                          const Weights &w, Head least, Shared<NT> &s, const Listed<NT> &l,
                                          uint32_t known_from)
{
    constexpr int kBins = Shared<NT>::kBins;
    Head head = {finite, 0};
    for (int i = threadIdx.x; i < kBins; i += NT) head.mass += s.first_mass[i];
    head.mass = block_sum<NT>(head.mass, s.part);
#pragma unroll 1
    for (int step = 0; step < 3; ++step) {     // top-k, top-p, the draw
        u64 target = set.top_k;
        if (step == 0 && (set.top_k == 0 || set.top_k >= finite)) continue;
        if (step == 1) {
            if (set.top_p >= 1.0) continue;
            target = mass_target(set.top_p, (double)head.mass);
        }
        if (step == 2) {
            if (least.count < head.count) head = least;
            target = draw_target(set.u, head.mass);
        }
        const Head h = locate<T, NT>(a, row, w, row_bin_scale(w, kBins), s, l, known_from, step > 0, target,
                                     step == 2);
        if (step < 2) head = h;
    }
    if (threadIdx.x == 0) answer(a, row, w, s.key, head);
}

// What the units of a row are set by: its sum as far as known, else a bound (no
// weight beyond the list is above the bound's).
__device__ __forceinline__ double units_sum(const Settings &set, const Row &r)
{
    if (set.sum() != Settings::kNone) return r.sum;
    if (r.bound == kNoBound) return (double)r.finite;
    const double t = ((double)value_of(r.bound) - (double)r.top) * set.scale;
    return (double)r.listed + (double)(r.finite - (uint32_t)r.listed) * exp2_64(t);
}

// The row's answers from the row itself.
template <int T, int NT>
__device__ __forceinline__ void from_row(const SampleArgs &a, int64_t row, const Settings &set, const Row &r,
                                         Shared<NT> &s, const Listed<NT> &l, uint32_t known_from)
{
    constexpr int kBins = Shared<NT>::kBins;
    if (set.greedy) {
        const int i = nth_equal<T, NT>(a, row, value_key(r.top), 1, s);
        if (threadIdx.x == 0) greedy_answer(a, row, i);
        return;
    }
    const Weights w(r.top, set.scale, units_sum(set, r));
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += NT) {
        s.first_count[i] = 0;
        s.first_mass[i] = 0;
    }
    __syncthreads();
    RowBins<kBins> bins(w, set.least());
    each<T, NT>(a, row, [&](float x, int) { bins.add(x, s.first_count, s.first_mass); });
    Head least;
    least.count = (uint32_t)block_sum<NT>((u64)bins.kept.count, s.part);
    least.mass = block_sum<NT>(bins.kept.mass, s.part);
    from_bins<T, NT>(a, row, set, r.finite, w, least, s, l, known_from);
}

// A row without a distribution: true, and its answers are written.
__device__ __forceinline__ bool no_row(const SampleArgs &a, int64_t row, const Row &r)
{
    if (!r.bad && r.finite) return false;
    if (threadIdx.x == 0) {
        a.ids[row] = -1;
        a.kept[row] = 0;
        a.logprob[row] = r.bad ? __builtin_nanf("") : -INFINITY;
    }
    return true;
}

// ---------------------------------------------------------------------------
// A stretch of a row, VECS vectors of 16 bytes a thread, in LDS, where each thread
// keeps its own: loops over them stay rolled and take few registers.  What is
// left after the last whole vector is one logit a thread.
template <int T, int NT, int VECS>
struct Held {
    static constexpr int V = kVec<T>, kLogits = VECS * V * NT;
    u32x4 *lds;                   // [VECS][NT]
    u32x4 raw[VECS];              // on their way
    float most[VECS];             // the largest logit of each vector
    float extra;
    int begin, extra_at;          // indices in the row

    // logits first .. first + len - 1 of the row
    __device__ __forceinline__ void load(const SampleArgs &a, int64_t row, int first, int len)
    {
        typedef typename Elem<T>::type El;
        const uint32_t none = T == Q8_T_F32 ? 0xff800000u : T == Q8_T_F16 ? 0xfc00fc00u : 0xff80ff80u;
        const El *p = (const El *)a.logits + row * a.row_stride + first;
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            const int i = (threadIdx.x + v * NT) * V;
            raw[v] = (u32x4){none, none, none, none};
            if (i + V <= len) raw[v] = *(const u32x4_any *)(p + i);
        }
        const int left = len / V * V + threadIdx.x;
        begin = first;
        extra_at = first + left;
        extra = left < len ? (float)p[left] : -INFINITY;
    }

    // f(value, index); beyond the stretch -infinity
    template <class F>
    __device__ __forceinline__ void each(F f) const
    {
#pragma unroll 1
        for (int v = 0; v < VECS; ++v) {
            float y[V];
            unpack16<T>(lds[v * NT + threadIdx.x], y);
            const int i = begin + (int)(threadIdx.x + v * NT) * V;
#pragma unroll
            for (int j = 0; j < V; ++j) f(y[j], i + j);
        }
        f(extra, extra_at);
    }
};

// The largest logit of the stretch and of this thread, how many are finite and
// whether one is NaN or +infinity, and the weights' sum beside the largest.
struct Stretch {
    float top, own_top;
    uint32_t finite, bad;
    double sum;
};

// The logits loaded go to LDS; their statistics.  (The maximum that NaN passes
// through: one instruction for two logits, without a comparison for NaN.)
template <int T, int NT, int VECS>
__device__ __forceinline__ Stretch stretch(const Settings &set, Held<T, NT, VECS> &x, u64 *part)
{
    constexpr int V = kVec<T>;
    auto larger = [](float p, float q) { return __builtin_elementwise_maximum(p, q); };
    Stretch r = {-INFINITY, x.extra, 0, 0, 0.0};
    float lowest = INFINITY;      // of this thread's vectors
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
        float y[V];
        x.lds[v * NT + threadIdx.x] = x.raw[v];
        unpack16<T>(x.raw[v], y);
        x.most[v] = larger(y[0], y[1]);
        lowest = fminf(fminf(y[0], y[1]), lowest);
#pragma unroll
        for (int j = 2; j < V; j += 2) {
            x.most[v] = larger(larger(y[j], y[j + 1]), x.most[v]);
            lowest = fminf(fminf(y[j], y[j + 1]), lowest);
        }
        r.own_top = larger(r.own_top, x.most[v]);
        __builtin_amdgcn_sched_barrier(0);
    }
    const bool bad = !(r.own_top < INFINITY);
    // (counted where a vector holds -infinity, banned or beyond the stretch)
    uint32_t finite = 0;
    if (lowest == -INFINITY) x.each([&](float v, int) { finite += v > -INFINITY; });
    else finite = VECS * V + (x.extra > -INFINITY);
    r.top = r.own_top;
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        r.top = fmaxf(r.top, __shfl_xor(r.top, d));
        finite += __shfl_xor(finite, d);
    }
    const u64 any = __ballot(bad);
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
        part[wave] = (u64)__builtin_bit_cast(uint32_t, r.top) << 32 | finite << 1 | (any != 0);   // (finite < 2^13)
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        r.top = fmaxf(r.top, __builtin_bit_cast(float, (uint32_t)(part[w] >> 32)));
        r.finite += (uint32_t)part[w] >> 1;
        r.bad |= (uint32_t)part[w] & 1;
    }
    const Settings::Sum kind = set.sum();
    if (kind == Settings::kNone || r.top == -INFINITY || r.bad) return r;
    double sum = 0.0;
    const float scale = (float)set.scale, off = r.top * scale;
    if (kind == Settings::kRough && fabsf(off) < 0x1p20f) {
        // 2^(v scale - off), a fused product each; what off was rounded by is a
        // factor of the sum
#pragma unroll 2
        for (int v = 0; v < VECS; ++v) {
            float y[V];
            unpack16<T>(x.lds[v * NT + threadIdx.x], y);
#pragma unroll
            for (int j = 0; j < V; ++j) y[j] = __builtin_amdgcn_exp2f(fmaf(y[j], scale, -off));
#pragma unroll
            for (int d = 1; d < V; d *= 2)
#pragma unroll
                for (int j = 0; j < V; j += 2 * d) y[j] += y[j + d];
            sum += (double)y[0];
        }
        sum += (double)__builtin_amdgcn_exp2f(fmaf(x.extra, scale, -off));
        sum *= (double)__builtin_amdgcn_exp2f((float)((double)off - (double)r.top * (double)scale));
    } else {
        // (the difference first: v * scale - top * scale would round masks near the
        // type's lowest value apart)
        const double top = r.top;
        x.each([&](float v, int) { sum += exp2_64(((double)v - top) * set.scale); });
    }
    r.sum = block_sum<NT>(sum, part);
    return r;
}

// A key that `rank` or more logits of a workgroup of 64 or 256 reach: that of the
// rank-th of its threads' maxima, its low half cut.
__device__ __forceinline__ uint32_t list_bound(float own_top, int rank)
{
    return max(nth_key(value_key(own_top), rank), kLeastKey);
}

__device__ __forceinline__ uint32_t list_bound(float own_top, int rank, uint32_t *keys)
{
    keys[threadIdx.x] = value_key(own_top);
    __syncthreads();
    return max(nth_key(((const u32x4 *)keys)[threadIdx.x & 63], rank), kLeastKey);
}

constexpr int kJoinThreads = 256;     // of a short row, and of a join

// The logits of a stretch from `low` on as keys to list(place, key), where they
// are `most` or fewer; returns how many they are.  Few vectors have any: the
// largest logit of each says which.
template <int T, int NT, int VECS, class F>
__device__ __forceinline__ int list_stretch(const Held<T, NT, VECS> &x, float low, int most, u64 *part, F list)
{
    constexpr int V = kVec<T>;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t hits = 0;            // a bit per vector
#pragma unroll
    for (int v = 0; v < VECS; ++v) hits |= x.most[v] >= low ? 1u << v : 0u;
    if constexpr (NT == 64) {     // by ballots, the lanes' next vectors together
        int n = 0;
        auto offer = [&](bool in, float y, int i) {
            const uint64_t all = __ballot(in);
            if (!all) return;
            const int to = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(all >> 32),
                                                         __builtin_amdgcn_mbcnt_lo((uint32_t)all, 0));
            if (in && to < most) list(to, order_key(y, (uint32_t)i));
            n += __popcll(all);
        };
        for (; __ballot(hits != 0); hits &= hits - 1) {
            const int v = hits ? __builtin_ctz(hits) : 0, i = x.begin + (int)(threadIdx.x + v * NT) * V;
            float y[V];
            unpack16<T>(x.lds[v * NT + threadIdx.x], y);
#pragma unroll
            for (int j = 0; j < V; ++j) offer(hits != 0 && y[j] >= low, y[j], i + j);
        }
        offer(x.extra >= low, x.extra, x.extra_at);
        return n;
    }
    auto each_hit = [&](auto f) {
        for (uint32_t h = hits; h; h &= h - 1) {
            const int v = __builtin_ctz(h), i = x.begin + (int)(threadIdx.x + v * NT) * V;
            float y[V];
            unpack16<T>(x.lds[v * NT + threadIdx.x], y);
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (y[j] >= low) f(y[j], i + j);
        }
        if (x.extra >= low) f(x.extra, x.extra_at);
    };
    int at = 0;
    each_hit([&](float, int) { ++at; });
    const int mine = at;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int c = __shfl_up(at, d);
        if (lane >= d) at += c;
    }
    if (lane == 63) part[wave] = (u64)at;
    __syncthreads();
    at -= mine;
    int all = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        if (w < wave) at += (int)part[w];
        all += (int)part[w];
    }
    __syncthreads();
    if (all <= most) each_hit([&](float y, int i) { list(at++, order_key(y, (uint32_t)i)); });
    return all;
}

// ---------------------------------------------------------------------------
// Short rows: one per workgroup.
constexpr int kShortVecs = 4;

template <int T>
__global__ __launch_bounds__(kJoinThreads) void sample_row_kernel(const SampleArgs a)
{
    constexpr int NT = kJoinThreads;
    __shared__ Shared<NT> s;
    __shared__ u32x4 held[kShortVecs * NT];
    const int64_t row = blockIdx.x;
    const Settings set(a, row);
    Held<T, NT, kShortVecs> x;
    x.lds = held;
    x.load(a, row, 0, (int)a.n_vocab);
    const Stretch st = stretch<T, NT, kShortVecs>(set, x, s.part);
    Row r = {st.top, st.finite, st.bad, st.sum, 0, 0};
    if (no_row(a, row, r)) return;
#pragma unroll 1
    for (int rank = kRank; rank > 0; rank /= 4) {       // (a smaller one where the list is full)
        r.bound = list_bound(st.own_top, rank, s.keys);
        __syncthreads();          // (the list lies where the keys were)
        r.listed = list_stretch<T, NT, kShortVecs>(x, value_of(r.bound), Shared<NT>::kList, s.part,
                                       [&](int at, u64 key) { s.list[at] = key; });
        if (r.listed <= Shared<NT>::kList) break;
        __syncthreads();
    }
    __syncthreads();
    Listed<NT> l;
    const bool listed = r.listed > 0 && r.listed <= Shared<NT>::kList;
    l.take(s, listed ? r.listed : 0);
    if (listed && from_list<NT>(a, row, set, r, set.sum(), s, l)) return;
    __syncthreads();
    if (!listed) r.bound = kNoBound;
    from_row<T, NT>(a, row, set, r, s, l, r.bound);
}

// ---------------------------------------------------------------------------
// Longer rows: a part of one per workgroup, the join of its parts, and for the
// rows that their lists do not answer a histogram by parts and its reading.

struct PartOut {
    double sum;
    float top;
    uint32_t bound, finite, bad;
    int listed;
};

constexpr int kAgainThreads = 512;
constexpr int kRowBins = Shared<kAgainThreads>::kBins, kRowList = Shared<kJoinThreads>::kList;

// A row that is read again.
struct Again {
    u64 mass[kRowBins], list[kRowList], least_mass, all_mass;
    uint32_t count[kRowBins], least_count;
    int row;
    Row r;
};

struct Work {
    PartOut *parts;               // [m][parts]
    u64 *lists;                   // [m][parts][kPlaces]
    Again *again;                 // [m], the first *n_again of them
    int *n_again;
    int n_parts, part_len, rank;
};

// A part is a wave's, without barriers.  What is done once a part (statistics,
// bound, list) is 400 instructions, against 7 a logit; twice the vectors would
// halve that share but leave nine waves to a CU (512 x 262144, with a pass that
// counted the logits: 90 us against 72; parts by four waves of as many vectors 89 to
// 150).
constexpr int kPartThreads = 64, kPartVecs = 8;

template <int T>
__global__ __launch_bounds__(kPartThreads) void sample_part_kernel(const SampleArgs a, const Work w)
{
    constexpr int NT = kPartThreads;
    __shared__ u32x4 held[kPartVecs * NT];
    __shared__ u64 part[NT / 64];
    const int64_t row = blockIdx.y, at = row * w.n_parts + blockIdx.x;
    const int first = blockIdx.x * w.part_len;
    if (at == 0 && threadIdx.x == 0) *w.n_again = 0;
    Held<T, NT, kPartVecs> x;
    x.lds = held;
    x.load(a, row, first, min(w.part_len, (int)a.n_vocab - first));
    const Settings set(a, row);
    const Stretch st = stretch<T, NT, kPartVecs>(set, x, part);
    PartOut out = {st.sum, st.top, kNoBound, st.finite, st.bad, 0};
#pragma unroll 1
    for (int rank = w.rank; rank > 0; rank /= 4) {      // (a smaller one where the list is full)
        const uint32_t bound = list_bound(st.own_top, rank);
        const int n = list_stretch<T, NT, kPartVecs>(x, value_of(bound), kPlaces, part,
                                                     [&](int i, u64 key) { w.lists[at * kPlaces + i] = key; });
        if (n <= kPlaces) {
            out.bound = bound;
            out.listed = n;
            break;
        }
    }
    if (threadIdx.x == 0) w.parts[at] = out;
}

// INLINE: rows that the list does not answer are read here.
template <int T, bool INLINE>
__global__ __launch_bounds__(kJoinThreads) void sample_join_kernel(const SampleArgs a, const Work w)
{
    constexpr int NT = kJoinThreads, kWaves = NT / 64, kRound = 5;
    __shared__ Shared<NT> s;
    __shared__ int ends[NT + 1];
    const int half = w.n_parts > 1 ? 1 << (31 - __clz(min(w.n_parts, NT) - 1)) : 1;     // of a power of two of parts
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, wave = wave_uniform(tid >> 6), lane = tid & 63;
    const PartOut *parts = w.parts + row * w.n_parts;
    PartOut p = {0.0, -INFINITY, 0, 0, 0, 0};           // this thread's first part
    if (tid < w.n_parts) p = parts[tid];
    const Settings set(a, row);
    if (tid == 0) s.listed = 0;
    Row r;
    // (by the keys; a row that is all -infinity has the key of that)
    uint32_t top = 0, bound = 0;
    u64 counts = 0;
    for (int i = tid; i < w.n_parts; i += NT) {
        const PartOut o = i == tid ? p : parts[i];
        top = max(top, value_key(o.top));
        bound = max(bound, o.bound);
        counts += (u64)o.bad << 32 | o.finite;
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        top = max(top, (uint32_t)__shfl_xor((int)top, d));
        bound = max(bound, (uint32_t)__shfl_xor((int)bound, d));
        counts += __shfl_xor(counts, d);
    }
    if (lane == 0) {
        s.part[wave] = (u64)top << 32 | bound;
        s.list[wave] = counts;
    }
    __syncthreads();
    counts = 0;
    for (int i = 0; i < kWaves; ++i) {
        top = max(top, (uint32_t)(s.part[i] >> 32));
        bound = max(bound, (uint32_t)s.part[i]);
        counts += s.list[i];
    }
    r.top = value_of(top);
    r.bound = bound;
    r.finite = (uint32_t)counts;
    r.bad = (uint32_t)(counts >> 32);
    r.sum = 0.0;
    if (no_row(a, row, r)) return;
    __syncthreads();
    for (int l0 = 0; l0 < w.n_parts && r.bound != kNoBound; l0 += NT) {
        // NT lists at a time, one after another as one run of logits
        int end = l0 + tid < w.n_parts ? (l0 == 0 ? p.listed : parts[l0 + tid].listed) : 0;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int c = __shfl_up(end, d);
            if (lane >= d) end += c;
        }
        if (lane == 63) s.wave[wave].count = (uint32_t)end;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWaves; ++i) end += i < wave ? (int)s.wave[i].count : 0;
        ends[tid + 1] = end;
        if (tid == 0) ends[0] = 0;
        __syncthreads();
        const int n = ends[NT];
        const u64 *lists = w.lists + (row * w.n_parts + l0) * kPlaces;
        for (int e0 = 0; e0 < n; e0 += kRound * NT) {
            // the last list that begins at e or before, for each of a thread's places
            int l[kRound];
            u64 key[kRound];
#pragma unroll
            for (int u = 0; u < kRound; ++u) l[u] = 0;
#pragma unroll 1
            for (int d = l0 + NT < w.n_parts ? NT / 2 : half; d; d >>= 1)
#pragma unroll
                for (int u = 0; u < kRound; ++u) l[u] += ends[l[u] + d] <= min(e0 + u * NT + tid, n - 1) ? d : 0;
            // (all lanes load, so that no branch keeps one load from the next)
#pragma unroll
            for (int u = 0; u < kRound; ++u) {
                key[u] = lists[(int64_t)l[u] * kPlaces + min(e0 + u * NT + tid, n - 1) - ends[l[u]]];
            }
            int some = 0, at = 0;
#pragma unroll
            for (int u = 0; u < kRound; ++u) {
                const bool in = e0 + u * NT + tid < n && (uint32_t)(key[u] >> 32) >= r.bound;
                key[u] = in ? key[u] : 0;
                some += __popcll(__ballot(in));
            }
            if (lane == 0) at = atomicAdd(&s.listed, some);
            at = wave_uniform(at);
#pragma unroll
            for (int u = 0; u < kRound; ++u) {
                const uint64_t all = __ballot(key[u] != 0);
                const int to = at + __builtin_amdgcn_mbcnt_hi((uint32_t)(all >> 32),
                                                              __builtin_amdgcn_mbcnt_lo((uint32_t)all, 0));
                if (key[u] != 0 && to < kRowList) s.list[to] = key[u];
                at += __popcll(all);
            }
        }
        __syncthreads();
    }
    if (set.sum() != Settings::kNone) {
        double sum = 0.0;
        for (int i = tid; i < w.n_parts; i += NT) {
            const double some = i == tid ? p.sum : parts[i].sum;
            const float beside = i == tid ? p.top : parts[i].top;
            if (some > 0.0) sum += some * exp2_64(((double)beside - (double)r.top) * set.scale);
        }
        r.sum = block_sum<NT>(sum, s.part);
    }
    __syncthreads();
    r.listed = s.listed;
    Listed<NT> l;
    const bool listed = r.listed > 0 && r.listed <= kRowList;
    l.take(s, listed ? r.listed : 0);
    if (listed && from_list<NT>(a, row, set, r, set.sum(), s, l)) return;
    __syncthreads();
    if (!listed) {
        r.bound = kNoBound;
        r.listed = 0;
    }
    if constexpr (INLINE)
        from_row<T, NT>(a, row, set, r, s, l, r.bound);
    else {
        if (tid == 0) s.index = atomicAdd(w.n_again, 1);
        __syncthreads();
        Again &g = w.again[s.index];
        for (int i = tid; i < kRowBins; i += NT) {
            g.mass[i] = 0;
            g.count[i] = 0;
        }
        for (int i = 0; i < Listed<NT>::N; ++i) g.list[tid + i * NT] = l.key[i];
        if (tid == 0) {
            g.least_mass = 0;
            g.all_mass = 0;
            g.least_count = 0;
            g.row = (int)row;
            g.r = r;
        }
    }
}

constexpr int kAgainGroups = 1024, kAgainLogits = 4096;

// Histograms of the rows that are read again, by parts.
template <int T>
__global__ __launch_bounds__(256) void sample_bins_kernel(const SampleArgs a, const Work w)
{
    typedef typename Elem<T>::type E;
    constexpr int NT = 256, V = kVec<T>;
    __shared__ uint32_t count[kRowBins];
    __shared__ u64 mass[kRowBins];
    __shared__ u64 part[NT / 64];
    const int tid = threadIdx.x;
    const int per_row = ((int)a.n_vocab + kAgainLogits - 1) / kAgainLogits;
    const int64_t items = (int64_t)*w.n_again * per_row;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        Again &g = w.again[item / per_row];
        const int64_t row = g.row;
        const int first = (int)(item % per_row) * kAgainLogits, len = min(kAgainLogits, (int)a.n_vocab - first);
        const Settings set(a, row);
        if (set.greedy) continue;
        const Row r = g.r;
        const Weights weights(r.top, set.scale, units_sum(set, r));
        for (int i = tid; i < kRowBins; i += NT) {
            count[i] = 0;
            mass[i] = 0;
        }
        __syncthreads();
        RowBins<kRowBins> bins(weights, set.least());
        const E *x = (const E *)a.logits + row * a.row_stride + first;
        const int vecs = len / V;
        for (int v = tid; v < vecs; v += NT) {
            float y[V];
            unpack16<T>(*(const u32x4_any *)(x + v * V), y);
#pragma unroll
            for (int j = 0; j < V; ++j) bins.add(y[j], count, mass);
        }
        if (vecs * V + tid < len) bins.add((float)x[vecs * V + tid], count, mass);
        const u64 least_count = block_sum<NT>((u64)bins.kept.count, part);
        const u64 least_mass = block_sum<NT>(bins.kept.mass, part);
        // (whole numbers: the order of the sums does not matter)
        u64 all = 0;
        for (int i = tid; i < kRowBins; i += NT)
            if (count[i]) {
                atomicAdd(&g.count[i], count[i]);
                atomicAdd(&g.mass[i], mass[i]);
                all += mass[i];
            }
        all = block_sum<NT>(all, part);
        if (tid == 0) {
            atomicAdd(&g.least_count, (uint32_t)least_count);
            atomicAdd(&g.least_mass, least_mass);
            atomicAdd(&g.all_mass, all);
        }
        __syncthreads();
    }
}

// Their answers.
template <int T>
__global__ __launch_bounds__(kAgainThreads) void sample_again_kernel(const SampleArgs a, const Work w)
{
    constexpr int NT = kAgainThreads;
    __shared__ Shared<NT> s;
    const int tid = threadIdx.x, n = *w.n_again;
    for (int item = blockIdx.x; item < n; item += gridDim.x) {
        const Again &g = w.again[item];
        const int64_t row = g.row;
        const Settings set(a, row);
        const Row r = g.r;
        __syncthreads();
        if (set.greedy) {
            const int i = nth_equal<T, NT>(a, row, value_key(r.top), 1, s);
            if (tid == 0) greedy_answer(a, row, i);
            continue;
        }
        Listed<NT> l;
#pragma unroll
        for (int i = 0; i < Listed<NT>::N; ++i) l.key[i] = i < kRowList / NT ? g.list[tid + i * NT] : 0;
        const Weights weights(r.top, set.scale, units_sum(set, r));
        if (r.listed && set.sum() == Settings::kRough) {
            Row known = r;                     // the list again, with the sum as it is
            known.sum = (double)g.all_mass * __builtin_amdgcn_ldexp(1.0, -weights.bits);
            if (from_list<NT>(a, row, set, known, Settings::kFull, s, l)) continue;
            __syncthreads();
        }
        for (int i = tid; i < kRowBins; i += NT) {
            s.first_count[i] = g.count[i];
            s.first_mass[i] = g.mass[i];
        }
        __syncthreads();
        from_bins<T, NT>(a, row, set, r.finite, weights, {g.least_count, g.least_mass}, s, l, r.bound);
    }
}

constexpr int kShortRow = Held<Q8_T_F32, kJoinThreads, kShortVecs>::kLogits;   // logits of a row that one workgroup takes
// Calls of up to so many logits read rows again in their join: two launches fewer
// (1 x 32000 17.7 us against 20.5), but one workgroup for all of it (333 x 50257 with
// such rows 89 against 69).
constexpr int64_t kInline = 1 << 18;
constexpr int kGroupRows = 2048;     // rows that share a workspace's turn

template <int T>
constexpr int kPartMost = Held<T, kPartThreads, kPartVecs>::kLogits;

int64_t n_parts(int64_t n_vocab, int64_t most) { return (n_vocab + most - 1) / most; }

constexpr int64_t kPartBytes = sizeof(PartOut) + sizeof(u64) * kPlaces;

SampleArgs rows_of(const SampleArgs &a, int64_t from, int64_t most)
{
    SampleArgs b = a;
    b.m = a.m - from < most ? a.m - from : most;
    b.logits = (const uint8_t *)a.logits + from * a.row_stride * (a.type == Q8_T_F32 ? 4 : 2);
    b.u += from; b.ids += from; b.logprob += from; b.kept += from;
    if (b.temperature) b.temperature += from;
    if (b.top_k) b.top_k += from;
    if (b.top_p) b.top_p += from;
    if (b.min_p) b.min_p += from;
    return b;
}

bool launched() { return hipGetLastError() == hipSuccess; }

template <int T>
int launch_parts(const SampleArgs &a, void *ws, hipStream_t stream)
{
    for (int64_t i = 0; i < a.m; i += kGroupRows) {
        const SampleArgs b = rows_of(a, i, kGroupRows);
        const int64_t parts = n_parts(a.n_vocab, kPartMost<T>);
        const bool again = a.m * a.n_vocab > kInline;
        Work w;
        w.n_again = (int *)ws;
        w.lists = (u64 *)((uint8_t *)ws + 256);
        w.parts = (PartOut *)(w.lists + b.m * parts * kPlaces);
        w.again = (Again *)(w.parts + b.m * parts);
        w.n_parts = (int)parts;
        w.part_len = (int)((a.n_vocab + 8 * parts - 1) / (8 * parts) * 8);
        w.rank = parts > 64 ? 12 : parts > 16 ? 768 / (int)parts : 48;
        hipLaunchKernelGGL((sample_part_kernel<T>), dim3((unsigned)parts, (unsigned)b.m), dim3(kPartThreads), 0,
                           stream, b, w);
        if (!launched()) return -6;
        if (!again) {
            hipLaunchKernelGGL((sample_join_kernel<T, true>), dim3((unsigned)b.m), dim3(kJoinThreads), 0, stream, b,
                               w);
            if (!launched()) return -6;
            continue;
        }
        hipLaunchKernelGGL((sample_join_kernel<T, false>), dim3((unsigned)b.m), dim3(kJoinThreads), 0, stream, b, w);
        if (!launched()) return -6;
        hipLaunchKernelGGL((sample_bins_kernel<T>), dim3(kAgainGroups), dim3(256), 0, stream, b, w);
        if (!launched()) return -6;
        hipLaunchKernelGGL((sample_again_kernel<T>), dim3((unsigned)(b.m < 256 ? b.m : 256)),
                           dim3(kAgainThreads), 0,
                           stream, b, w);
        if (!launched()) return -6;
    }
    return 0;
}

template <int T>
int launch_type(const SampleArgs &a, void *ws, hipStream_t stream)
{
    if (a.n_vocab > kShortRow) return launch_parts<T>(a, ws, stream);
    // (2^32 threads bound a launch)
    constexpr int64_t most = (int64_t)1 << 23;
    for (int64_t i = 0; i < a.m; i += most) {
        const SampleArgs b = rows_of(a, i, most);
        hipLaunchKernelGGL((sample_row_kernel<T>), dim3((unsigned)b.m), dim3(kJoinThreads), 0, stream, b);
        if (!launched()) return -6;
    }
    return 0;
}

}  // namespace

// Enough for any call of up to m rows of up to n_vocab logits, of any type.
size_t sample_ws_bytes(int64_t m, int64_t n_vocab)
{
    if (n_vocab <= kShortRow || m == 0) return 256;
    const int64_t rows = m < kGroupRows ? m : kGroupRows;
    const int64_t parts = rows * n_parts(n_vocab, kPartMost<Q8_T_F32>);      // (the most of any type)
    return 256 + (size_t)(parts * kPartBytes + rows * (int64_t)sizeof(Again));
}

int launch_sample(const SampleArgs &a, void *ws, hipStream_t stream)
{
    if (a.type == Q8_T_F32) return launch_type<Q8_T_F32>(a, ws, stream);
    if (a.type == Q8_T_F16) return launch_type<Q8_T_F16>(a, ws, stream);
    return launch_type<Q8_T_BF16>(a, ws, stream);
}

}  // namespace q8
