// sample.hip -- temperature, top-k, top-p and min-p over a row of logits: the token that a
// given random number draws, and the distribution that is left.
//
// The entries are taken in the order of falling logits (equal ones: the lowest index first) with
// the weights w = exp((l - max) / temperature).  Every filter keeps a prefix of that order: the
// first k; those before which less than p of the weight (of the first k) has passed; those with
// w >= min_p.  The token is the first at which the running weight exceeds u times the weight
// that is kept, so the draw too is a place in that order.  No sort is needed for it:
// a histogram of the distance from the maximum (kBuckets steps over at most 32 nats) gives the
// bucket of each place, and only that bucket's entries are ordered, by counting.
// A bucket of more entries than kList (ties) is cut further by digits of (logit, index).
//
// Weights are formed in 64 bits and added as whole numbers in steps of 2^-43 of the largest: sums
// of 2^20 of them fit 63 bits, no order of additions changes them, and the choice agrees with
// one made in 64-bit floating point but at a border nearer than some 10^-12.
//
// One workgroup takes a row and reads it once for the maximum and once for each place looked for.
#include "common.h"
#include "kernels.h"
#include "norm_rows.h"

namespace prism {

namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBuckets = 2048, kList = 1024, kIndexBits = 20, kDigitBits = 11;
static_assert(kSampleMaxVocab == 1 << kIndexBits, "an index fills the order's low bits");
static_assert(kBuckets == 2 * kThreads && kBuckets == 1 << kDigitBits, "two buckets a thread; a digit fills them");
constexpr double kOne = 8796093022208.;                      // 2^43, the weight of the maximum

// Counts and weights of 2048 buckets; after scan() the sums up to and with each.
struct Hist {
    uint64_t mass[kBuckets];
    uint32_t count[kBuckets];
};
struct List {
    uint64_t order[kList], weight[kList];
};

struct Shared {
    Hist h;
    union {
        Hist digits;
        List list;
    } x;
    double table[32];                                        // 2^(i / 32)
    uint64_t wave_mass[kWaves], found_order, found_mass, base_mass;
    uint32_t wave_count[kWaves], base_count, number;
    float wave_max[kWaves], wave_min[kWaves];
    int wave_arg[kWaves], at;
};

// What a row is measured by.
struct Row {
    float max, step;                                         // step: buckets per unit of l
    double c;                                                // 32 log2 e / temperature
};

// l as a whole number that rises with it (+0 and -0 the same).
__device__ __forceinline__ uint32_t key_of(float l)
{
    const uint32_t b = __float_as_uint(l + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

// The place of an entry in the order: falling logit, then rising index.
__device__ __forceinline__ uint64_t order_of(float l, int index)
{
    return (uint64_t)~key_of(l) << kIndexBits | (uint32_t)index;
}
__device__ __forceinline__ float logit_of(uint64_t order) { return of_key(~(uint32_t)(order >> kIndexBits)); }

__device__ __forceinline__ int bucket_of(const Row& r, float l)
{
    return (int)fminf((r.max - l) * r.step, (float)(kBuckets - 1));
}

// exp((l - max) / temperature): 2^(n / 32) from the table, and the rest of the exponent, at most
// ln 2 / 64, by its series to the fifth power (2 10^-15).
__device__ __forceinline__ double weight_of(const Row& r, const double* table, float l)
{
    const double y = fmax(((double)l - (double)r.max) * r.c, -32. * 1100.), n = rint(y);
    const double t = (y - n) * 0.021660849392498290;         // ln 2 / 32
    double s = __builtin_fma(t, 1. / 120, 1. / 24);
    s = __builtin_fma(s, t, 1. / 6);
    s = __builtin_fma(s, t, 0.5);
    s = __builtin_fma(s, t, 1.);
    s = __builtin_fma(s, t, 1.);
    const int i = (int)n;
    return ldexp(table[i & 31] * s, i >> 5);
}
__device__ __forceinline__ uint64_t steps_of(double w)
{
    return (uint64_t)__double_as_longlong(__builtin_fma(w, kOne, 4503599627370496.)) & 0xfffffffffffffull;   // + 2^52
}

// Entries of a row as they are weighed: NaN counts as -infinity; beside +infinity nothing else counts.
__device__ __forceinline__ float entry(float l) { return l > -__builtin_inff() ? l : -__builtin_inff(); }
__device__ __forceinline__ float entry(float l, bool infinite)
{
    l = entry(l);
    return !infinite ? l : l == __builtin_inff() ? 0.f : -__builtin_inff();
}

// f(l, index) for every element of a row, which may begin at any element's address.
template <typename T, typename F> __device__ __forceinline__ void each(const T* row, int vocab, F f)
{
    constexpr int VE = Vec16<T>::N;
    const int whole = vocab / VE * VE;
    for (int at = threadIdx.x * VE; at < whole; at += kThreads * VE) {
        const rows::AtElement a = *reinterpret_cast<const rows::AtElement*>(row + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 2) {
                f(__uint_as_float(a[i] << 16), at + 2 * i);
                f(__uint_as_float(a[i] & 0xffff0000u), at + 2 * i + 1);
            } else {
                f(__uint_as_float(a[i]), at + i);
            }
        }
    }
    if (whole + (int)threadIdx.x < vocab)
        f(to_f32(row[whole + threadIdx.x]), whole + threadIdx.x);
}

__device__ __forceinline__ void clear(Hist& h)
{
    for (int i = threadIdx.x; i < kBuckets; i += kThreads) {
        h.mass[i] = 0;
        h.count[i] = 0;
    }
}

// Sums up to and with each bucket.
__device__ void scan(Hist& h, Shared& s)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    __syncthreads();
    uint64_t m0 = h.mass[2 * tid], m = m0 + h.mass[2 * tid + 1];
    uint32_t c0 = h.count[2 * tid], c = c0 + h.count[2 * tid + 1];
    const uint64_t m_own = m;
    const uint32_t c_own = c;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint64_t mu = __shfl_up(m, d);
        const uint32_t cu = __shfl_up(c, d);
        if (lane >= d) {
            m += mu;
            c += cu;
        }
    }
    if (lane == 63) {
        s.wave_mass[wave] = m;
        s.wave_count[wave] = c;
    }
    __syncthreads();
    for (int w = 0; w < wave; ++w) {
        m += s.wave_mass[w];
        c += s.wave_count[w];
    }
    h.mass[2 * tid] = m - m_own + m0;
    h.mass[2 * tid + 1] = m;
    h.count[2 * tid] = c - c_own + c0;
    h.count[2 * tid + 1] = c;
    __syncthreads();
}

// The places that are looked for in the order.
enum Place {
    kCount,                                                  // the goal-th entry
    kReach,                                                  // the entry with which the weight reaches the goal
    kPass,                                                   // the entry with which the weight exceeds the goal
    kUpTo                                                    // the entry that has the goal for its place
};

// Whether a step from (count, mass) before it by (dc, dm) takes in the place.
template <Place P>
__device__ __forceinline__ bool takes(uint64_t goal, uint64_t mass, uint64_t dm, uint32_t count, uint32_t dc)
{
    if (P == kCount)
        return count < goal && goal <= (uint64_t)count + dc;
    if (P == kReach)
        return mass < goal && goal <= mass + dm;
    return mass <= goal && goal < mass + dm;
}

// The bucket of a scanned histogram that takes in the place, and what is before it.  For kUpTo
// it is the bucket `given`.
template <Place P> __device__ __forceinline__ void find_bucket(const Hist& h, Shared& s, uint64_t goal, int given, uint64_t mass0, uint32_t count0)
{
    for (int b = threadIdx.x; b < kBuckets; b += kThreads) {
        const uint64_t before = b ? h.mass[b - 1] : 0;
        const uint32_t cb = b ? h.count[b - 1] : 0;
        const bool hit = P == kUpTo ? b == given
                                    : takes<P>(goal, mass0 + before, h.mass[b] - before, count0 + cb, h.count[b] - cb);
        if (hit) {
            s.at = b;
            s.base_mass = mass0 + before;
            s.base_count = count0 + cb;
            s.number = h.count[b] - cb;
        }
    }
    __syncthreads();
}

// The place's entry, in s.found_order, and the weight up to and with it, in s.found_mass.  For kUpTo:
// the weight of the entries whose place is at most `goal`, which lies in bucket `given`.
template <Place P, typename T>
__device__ void find(const T* row, int vocab, bool infinite, const Row& r, Shared& s, uint64_t goal, int given)
{
    const int tid = threadIdx.x;
    if (tid == 0)
        s.number = 0;
    __syncthreads();
    find_bucket<P>(s.h, s, goal, given, 0, 0);
    const int bucket = s.at;
    uint64_t prefix = 0;
    int shift = 32 + kIndexBits;
    auto in = [&](float l, uint64_t order) { return bucket_of(r, l) == bucket && order >> shift == prefix; };
    while (s.number > kList) {                               // shift is 0 at the latest when one entry is left
        const int next = shift > kDigitBits ? shift - kDigitBits : 0;
        const uint64_t mass0 = s.base_mass;
        const uint32_t count0 = s.base_count;
        clear(s.x.digits);
        __syncthreads();
        each(row, vocab, [&](float raw, int i) {
            const float l = entry(raw, infinite);
            if (l > -__builtin_inff()) {
                const uint64_t order = order_of(l, i);
                if (in(l, order)) {
                    const int d = (int)(order >> next) & ((1 << (shift - next)) - 1);
                    atomicAdd(&s.x.digits.count[d], 1u);
                    atomicAdd((unsigned long long*)&s.x.digits.mass[d], (unsigned long long)steps_of(weight_of(r, s.table, l)));
                }
            }
        });
        scan(s.x.digits, s);
        find_bucket<P>(s.x.digits, s, goal, (int)(goal >> next) & ((1 << (shift - next)) - 1), mass0, count0);
        prefix = prefix << (shift - next) | (uint32_t)s.at;
        shift = next;
    }
    const uint64_t mass0 = s.base_mass;
    const uint32_t count0 = s.base_count;
    __syncthreads();
    if (tid == 0) {
        s.number = 0;
        s.found_mass = mass0;
    }
    __syncthreads();
    each(row, vocab, [&](float raw, int i) {
        const float l = entry(raw, infinite);
        if (l > -__builtin_inff()) {
            const uint64_t order = order_of(l, i);
            if (in(l, order)) {
                const uint32_t at = atomicAdd(&s.number, 1u);
                if (at < kList) {                            // always: the histogram counted them
                    s.x.list.order[at] = order;
                    s.x.list.weight[at] = steps_of(weight_of(r, s.table, l));
                }
            }
        }
    });
    __syncthreads();
    const int n = min((int)s.number, kList);
    if (tid < n) {
        const uint64_t mine = s.x.list.order[tid], w = s.x.list.weight[tid];
        if (P == kUpTo) {
            if (mine <= goal)
                atomicAdd((unsigned long long*)&s.found_mass, (unsigned long long)w);
        } else {
            uint64_t mass = mass0;
            uint32_t count = count0;
            for (int i = 0; i < n; ++i) {
                const bool before = s.x.list.order[i] < mine;
                mass += before ? s.x.list.weight[i] : 0;
                count += before;
            }
            if (takes<P>(goal, mass, w, count, 1)) {
                s.found_order = mine;
                s.found_mass = mass + w;
            }
        }
    }
    __syncthreads();
}

}  // namespace

template <typename T>
__global__ __launch_bounds__(kThreads) void sample_kernel(const T* __restrict__ logits, int64_t stride, int vocab,
                                                          const float* __restrict__ temperature,
                                                          const int32_t* __restrict__ top_k,
                                                          const float* __restrict__ top_p,
                                                          const float* __restrict__ min_p, const float* __restrict__ u,
                                                          int32_t* __restrict__ tokens, float* __restrict__ probs)
{
    __shared__ Shared s;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t n = blockIdx.x;
    const T* row = logits + n * stride;
    float* out = probs ? probs + n * vocab : nullptr;
    const float t = temperature ? temperature[n] : 1.f;
    const float inf = __builtin_inff();

    // the largest entry (the first of equal ones) and the smallest
    float hi = -inf, lo = inf;
    int arg = INT32_MAX;
    each(row, vocab, [&](float raw, int i) {
        const float l = entry(raw);
        if (l > hi || (l == hi && i < arg)) {
            hi = l;
            arg = i;
        }
        if (l > -inf)
            lo = fminf(lo, l);
    });
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const float h2 = __shfl_xor(hi, m), l2 = __shfl_xor(lo, m);
        const int a2 = __shfl_xor(arg, m);
        if (h2 > hi || (h2 == hi && a2 < arg)) {
            hi = h2;
            arg = a2;
        }
        lo = fminf(lo, l2);
    }
    if (lane == 0) {
        s.wave_max[wave] = hi;
        s.wave_min[wave] = lo;
        s.wave_arg[wave] = arg;
    }
    if (tid < 32)
        s.table[tid] = exp2(tid / 32.);
    clear(s.h);
    __syncthreads();
    for (int w = 0; w < kWaves; ++w) {
        const float h2 = s.wave_max[w];
        if (h2 > hi || (h2 == hi && s.wave_arg[w] < arg)) {
            hi = h2;
            arg = s.wave_arg[w];
        }
        lo = fminf(lo, s.wave_min[w]);
    }
    const bool none = hi == -inf;
    if (none || !(t > 0.f)) {                                // nothing to draw from, or the largest is taken
        if (tokens && tid == 0)
            tokens[n] = none ? -1 : arg;
        if (out)
            for (int i = tid; i < vocab; i += kThreads)
                out[i] = !none && i == arg ? 1.f : 0.f;
        return;
    }
    const bool infinite = hi == inf;
    Row r;
    r.max = infinite ? 0.f : hi;
    const float span = fminf(infinite ? 0.f : hi - lo, 32.f * t);
    r.step = span > 0.f ? fminf((kBuckets - 1) / span, 3e38f) : 0.f;
    r.c = 46.166241308446828384 / (double)t;                 // 32 log2 e

    each(row, vocab, [&](float raw, int i) {
        const float l = entry(raw, infinite);
        if (l > -inf) {
            const int b = bucket_of(r, l);
            atomicAdd(&s.h.count[b], 1u);
            atomicAdd((unsigned long long*)&s.h.mass[b], (unsigned long long)steps_of(weight_of(r, s.table, l)));
        }
    });
    scan(s.h, s);

    uint64_t cut = ~0ull;                                    // the last place that is kept
    uint64_t total = s.h.mass[kBuckets - 1];
    const int k = top_k ? top_k[n] : 0;
    if (k > 0 && (uint32_t)k < s.h.count[kBuckets - 1]) {
        find<kCount>(row, vocab, infinite, r, s, (uint64_t)k, 0);
        cut = s.found_order;
        total = s.found_mass;
    }
    const float p = top_p ? top_p[n] : 1.f;
    const uint64_t whole = total;
    if (p < 1.f) {
        const uint64_t goal = (uint64_t)fmax(ceil((double)p * (double)whole), 1.);
        find<kReach>(row, vocab, infinite, r, s, goal, 0);
        cut = s.found_order;
        total = s.found_mass;
    }
    const float mp = min_p && min_p[n] > 0.f ? fminf(min_p[n], 1.f) : 0.f;       // NaN: off
    if (mp > 0.f) {
        // the smallest logit whose weight is at least mp
        const double least = log((double)mp), back = 1. / (double)t;
        float l = (float)((double)r.max + least * (double)t);
        auto heavy = [&](float v) { return ((double)v - (double)r.max) * back >= least; };
        for (int i = 0; i < 4 && !heavy(l); ++i)
            l = of_key(key_of(l) + 1);
        for (int i = 0; i < 4 && heavy(of_key(key_of(l) - 1)); ++i)
            l = of_key(key_of(l) - 1);
        if (l > (infinite ? 0.f : lo)) {
            const uint64_t last = order_of(l, kSampleMaxVocab - 1);
            if (last < cut) {
                find<kUpTo>(row, vocab, infinite, r, s, last, bucket_of(r, l));
                cut = last;
                total = s.found_mass;
            }
        }
    }
    if (out) {
        const double share = 1. / ((double)total / kOne);
        each(row, vocab, [&](float raw, int i) {
            const float l = entry(raw, infinite);
            out[i] = l > -inf && order_of(l, i) <= cut ? (float)(weight_of(r, s.table, l) * share) : 0.f;
        });
    }
    if (tokens) {
        const float x = u[n];
        const double at = x >= 1.f ? 1. - 5.9604644775390625e-8 : x > 0.f ? (double)x : 0.;      // below 1 by an fp32 half step
        find<kPass>(row, vocab, infinite, r, s, (uint64_t)(at * (double)total), 0);
        if (tid == 0)
            tokens[n] = (int32_t)(s.found_order & (kSampleMaxVocab - 1));
    }
}

bool sample_fits(int64_t rows, int) { return rows <= UINT32_MAX / kThreads; }

size_t sample_workspace_bytes(int64_t, int) { return 0; }

template <typename T> static hipError_t launch_T(const SampleArgs& p, hipStream_t stream)
{
    if (p.rows == 0)
        return hipSuccess;
    hipLaunchKernelGGL((sample_kernel<T>), dim3((unsigned)p.rows), dim3(kThreads), 0, stream, (const T*)p.logits,
                       p.stride, p.vocab, p.temperature, p.top_k, p.top_p, p.min_p, p.u, p.tokens, p.probs);
    return hipGetLastError();
}

hipError_t launch_sample(const SampleArgs& p, hipStream_t stream)
{
    return p.bf16 ? launch_T<uint16_t>(p, stream) : launch_T<float>(p, stream);
}

}  // namespace prism
