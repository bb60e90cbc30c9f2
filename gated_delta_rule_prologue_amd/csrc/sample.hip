// sample.hip -- temperature, top-k, top-p and min-p over a row of logits: the token that a
// given random number draws, and the distribution that is left.
//
// The entries are taken in the order of falling logits (equal ones: the lowest index first) with
// the weights w = exp((l - max) / temperature).  Every filter keeps a prefix of that order: the
// first k; those before which less than p of the weight (of the first k) has passed; those with
// w >= min_p.  The token is the first at which the running weight exceeds u times the weight
// that is kept, so the draw too is a place in that order.  No sort of the row is needed for it:
// a histogram of the distance from the maximum (768 buckets over 16 nats, 256 over what is
// behind, or 1024 over less) bounds the weight before each place, and so the few buckets in
// which each can lie; only their entries are collected, and the places are looked up one after
// the other: up to 64 entries by one wavefront, up to 1024 by the workgroup.
// More entries in those buckets (ties, places in the last bucket) are cut further by digits of
// (logit, index).
//
// Weights are formed in 64 bits and added as whole numbers in steps of 2^-43 of the largest: sums
// of 2^20 of them fit 64 bits and no order of additions changes them.  A weight is off by half a step at most,
// a sum over V entries by V 2^-44 of the largest weight (7 10^-9 at 128,000, 6 10^-8, as u's own steps, at 2^20; met
// only where entries are alike and so rounded alike, entries below 2^-44 count as none).  The choice is that of exact
// sums but at a border nearer than twice that.
//
// Bound by a chain of dependent passes where there are few rows (maximum, histogram, its sums,
// collection, lookup: 1 to 7 us each), by the instructions of the weights (some 30 an entry, a third of
// them 64-bit) and one compute unit's reads of a row where there are many; reading the logits once
// would take a tenth to a third of it.  A row of up to 32,768 entries stays in the registers of one
// workgroup for all passes, so they are one launch: 1 row of 32,000 16 us, 64 19 us, 256 in bf16
// 23 us.  Longer rows are read again by each pass, and while they are few they are cut into chunks,
// one workgroup each, with a launch for the maximum, the histograms, the collection and the choice
// (and one for the distribution): 64 rows of 128,000 43 us; 256 rows, whole, 81 us;
// beyond 288 rows by half as many lanes a row: 320 distributions of 50,001 81 us.
#include <type_traits>

#include "common.h"
#include "kernels.h"
#include "norm_rows.h"

namespace prism {

namespace {

constexpr int kBuckets = 1024, kLast = kBuckets - 1, kList = 1024, kIndexBits = 20, kDigitBits = 10;
static_assert(kSampleMaxVocab == 1 << kIndexBits, "an index fills the order's low bits");
static_assert(kBuckets == 1 << kDigitBits, "a digit fills the buckets");
constexpr double kOne = 8796093022208.;                      // 2^43, the weight of the maximum
constexpr float kNats = 16.f;                                // that the first kNear buckets cover
constexpr int kNear = 768;
constexpr uint64_t kNowhere = ~0ull;

__device__ __forceinline__ float infinity() { return __builtin_inff(); }

// Counts and weights of the buckets; after scan() the sums up to and with each.
struct Hist {
    uint64_t mass[kBuckets];
    uint32_t count[kBuckets];
    __device__ __forceinline__ uint64_t mass_before(int b) const { return b ? mass[b - 1] : 0; }
    __device__ __forceinline__ uint32_t count_before(int b) const { return b ? count[b - 1] : 0; }
};

// What a row is measured by.
struct Scale {
    float max, min;
    float step, far_step, far_from;                          // buckets per unit of l, near and far, where they meet
    double c, top, least;                                    // 32 log2 e / temperature; max; l - max of a weight of 2^-45
};

// What is asked of a row.
struct Wish {
    float t, p, m;                                           // m: 0 is off
    double at;                                               // u as the nearest below 1
    int k;                                                   // 0 is off
    bool draw;
};

// What a row's histogram says of it: which filters cut it (min_p's place, or kNowhere), and the ranges of buckets in
// which the places lie, as bounds on height_of.
struct Plan {
    uint64_t m_order;
    int k, p, m;                                             // k, p: whether they are in force; m: its bucket, or -1
    int ranges;
    float from[4], to[4];
    float middle[4], reach[4];                               // all of a range is this near to its middle, and little else
};

struct Choice {
    uint64_t cut, total;                                     // the last place that is kept, the weight up to it; 0: none was found
    int token;
};

struct Shared {
    Hist h;
    union {
        Hist digits;
        struct {
            uint64_t order[kList], mass[kList];
        } list;
    } x;
    double table[32];                                        // 2^(i / 32)
    uint64_t wave_mass[16], found_order, found_mass, base_mass;
    uint64_t place_order[3], place_mass[3];                  // top-k's, top-p's and the draw's in the sorted list
    Plan plan;
    Choice choice;
    uint32_t wave_count[16], base_count, number;
    uint32_t first[kBuckets];                                // where a bucket begins in the sorted list
    float wave_max[16], wave_min[16];
    int at;
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

// A bucket and a fraction, rising as l falls: near the maximum d * step, from where the far buckets begin on the
// smaller of both lines.
__device__ __forceinline__ float height_of(const Scale& r, float l)
{
    const float d = r.max - l;
    return fminf(fminf(d * r.step, __builtin_fmaf(d, r.far_step, r.far_from)), (float)kLast);
}
__device__ __forceinline__ int bucket_of(const Scale& r, float l) { return (int)height_of(r, l); }

// The constants of the weights' arithmetic, held in registers: as literals each would be moved into the accumulator
// of its product first.
struct Constants {
    double whole, c4, c3, c2, c1, one, steps;
    __device__ __forceinline__ Constants()
        : whole(6755399441055744.),                          // 1.5 * 2^52: a sum's low word is its whole part
          c4(9.17256270182464329e-9), c3(1.69385097243718201e-6), c2(2.34596198202246789e-4),
          c1(2.16608493924982909e-2),                        // powers of ln 2 / 32 over 4!, 3!, 2!, 1!
          one(1.), steps(4503599627370496.)                  // 2^52: the steps are the sum's mantissa
    {
        asm volatile("" : "+v"(whole), "+v"(c4), "+v"(c3), "+v"(c2), "+v"(c1), "+v"(one), "+v"(steps));
    }
};

// exp(d / temperature): 2^(n / 32) from the table, and the rest of the exponent, at most
// ln 2 / 64, by its series to the fourth power (10^-12).
__device__ __forceinline__ double series_of(const Constants& k, const Scale& r, double d, int& n)
{
    const double m = __builtin_fma(d, r.c, k.whole);
    const double t = __builtin_fma(d, r.c, -(m - k.whole));
    double s = __builtin_fma(t, k.c4, k.c3);
    s = __builtin_fma(s, t, k.c2);
    s = __builtin_fma(s, t, k.c1);
    n = (int)__double_as_longlong(m);
    return __builtin_fma(s, t, k.one);
}
__device__ __forceinline__ double power_of(const double* table, int n, int add)
{
    const double t = table[n & 31];
    return __hiloint2double(__double2hiint(t) + (((n >> 5) + add) << 20), __double2loint(t));
}
// In steps of 2^-43: what is below the scale's least has a quarter of one.
__device__ __forceinline__ uint64_t steps_of(const Constants& k, const Scale& r, const double* table, float l)
{
    int n;
    double d = (double)l - r.top;
    // an instruction: the compiler would keep a second, quieted copy of the scale's least beside it
    asm("v_max_f64 %0, %0, %1" : "+v"(d) : "v"(r.least));
    const double s = series_of(k, r, d, n);
    const double w = __builtin_fma(power_of(table, n, 43), s, k.steps);
    return (uint64_t)(uint32_t)(__double2hiint(w) & 0xfffff) << 32 | (uint32_t)__double2loint(w);
}
__device__ __forceinline__ uint64_t steps_of(const Scale& r, const double* table, float l)
{
    return steps_of(Constants(), r, table, l);
}
// For fp32, whose least value is 2^-149: at least 2^-151.
__device__ __forceinline__ double weight_of(const Constants& k, const Scale& r, const double* table, float l)
{
    int n;
    const double s = series_of(k, r, fmax((double)l - r.top, r.least * (151. / 45.)), n);
    return power_of(table, n, 0) * s;
}

// Whether an entry counts, by its bits: the compiler takes a float comparison of what entry() has selected back to the
// value before the selection, and lets NaN through.
__device__ __forceinline__ bool live_entry(float l) { return __float_as_uint(l) != 0xff800000u; }

// Entries of a row as they are weighed: NaN counts as -infinity; beside +infinity nothing else counts.
__device__ __forceinline__ float entry(float l) { return l > -infinity() ? l : -infinity(); }
__device__ __forceinline__ float entry(float l, bool infinite)
{
    l = entry(l);
    return !infinite ? l : l == infinity() ? 0.f : -infinity();
}

// The elements from `first` to `end` of a row that are read again each time they are gone over.  A row may begin at
// any element's address.
template <typename T, int THREADS_> struct Streamed {
    static constexpr int THREADS = THREADS_;
    // vectors in flight (256 rows of 128,000 fp32: one 86 us, two 84, four 84; 128 of 50,001 in bf16: 35.5, 36.6, 39)
    static constexpr int AHEAD = sizeof(T) == 2 ? 1 : 2;
    const T* row;
    int first, end;
    bool infinite;                                           // entries of +infinity are all that counts
    __device__ __forceinline__ void load() { infinite = false; }
    __device__ __forceinline__ void settle() {}
    __device__ __forceinline__ void only_infinite() { infinite = true; }
    // f(vector, index of its first element) for every whole vector, AHEAD of them on their way to a lane
    template <typename F> __device__ __forceinline__ void vectors(int whole, F f) const
    {
        constexpr int VE = Vec16<T>::N, STEP = THREADS * VE;
        auto load = [&](int at) {                            // behind the last one that again
            return *reinterpret_cast<const rows::AtElement*>(row + (at < whole ? at : whole - VE));
        };
        int at = first + threadIdx.x * VE;
        if (at >= whole)
            return;
        rows::AtElement a[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            a[u] = load(at + u * STEP);
        for (; at < whole; at += AHEAD * STEP)
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const rows::AtElement x = a[u];
                a[u] = load(at + (u + AHEAD) * STEP);
                if (at + u * STEP < whole)
                    f(x, at + u * STEP);
            }
    }
    // f(entry, index) for every element, spread over the workgroup
    template <typename F> __device__ __forceinline__ void each(F f) const
    {
        constexpr int VE = Vec16<T>::N;
        const int whole = first + (end - first) / VE * VE;
        vectors(whole, [&](const rows::AtElement& a, int at) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 2) {
                    f(entry(__uint_as_float(a[i] << 16), infinite), at + 2 * i);
                    f(entry(__uint_as_float(a[i] & 0xffff0000u), infinite), at + 2 * i + 1);
                } else {
                    f(entry(__uint_as_float(a[i]), infinite), at + i);
                }
            }
        });
        if (whole + (int)threadIdx.x < end)
            f(entry(to_f32(row[whole + threadIdx.x]), infinite), whole + threadIdx.x);
    }
    // f(entries, index of the first) for every four, -infinity behind the last
    template <typename F> __device__ __forceinline__ void each4(F f) const
    {
        constexpr int VE = Vec16<T>::N;
        const int whole = first + (end - first) / VE * VE;
        vectors(whole, [&](const rows::AtElement& a, int at) {
#pragma unroll
            for (int j = 0; j < VE / 4; ++j) {
                float l[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (sizeof(T) == 2)
                        l[i] = entry(__uint_as_float(i % 2 ? a[2 * j + i / 2] & 0xffff0000u : a[2 * j + i / 2] << 16), infinite);
                    else
                        l[i] = entry(__uint_as_float(a[i]), infinite);
                }
                f(l, at + 4 * j);
            }
        });
        const int at = whole + 4 * (int)threadIdx.x;
        if (at < end) {
            float l[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                l[i] = at + i < end ? entry(to_f32(row[at + i]), infinite) : -infinity();
            f(l, at);
        }
    }
};

// Those that stay in the workgroup's registers, PER elements a thread; what is behind them reads as -infinity.
template <typename T, int THREADS_, int PER_> struct Held {
    static constexpr int THREADS = THREADS_, PER = PER_, VE = Vec16<T>::N, W = PER * (int)sizeof(T) / 4;
    const T* row;
    int first, end;
    uint32_t x[W];
    __device__ __forceinline__ int index(int vec) const { return first + (vec * THREADS + (int)threadIdx.x) * VE; }
    __device__ __forceinline__ void load()
    {
        constexpr uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
#pragma unroll
        for (int v = 0; v < W / 4; ++v) {
            rows::AtElement a = {none, none, none, none};
            if (index(v) + VE <= end)
                a = *reinterpret_cast<const rows::AtElement*>(row + index(v));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[4 * v + i] = a[i];
        }
        if ((end - first) % VE) {                            // the last vector, element by element
#pragma unroll
            for (int v = 0; v < W / 4; ++v)
                if (index(v) < end && index(v) + VE > end) {
#pragma unroll
                    for (int i = 0; i < VE; ++i)
                        if (index(v) + i < end) {
                            if constexpr (sizeof(T) == 2) {
                                const uint32_t half = row[index(v) + i];
                                x[4 * v + i / 2] = i % 2 ? (x[4 * v + i / 2] & 0xffffu) | half << 16
                                                         : (x[4 * v + i / 2] & 0xffff0000u) | half;
                            } else {
                                x[4 * v + i] = __float_as_uint(row[index(v) + i]);
                            }
                        }
                }
        }
    }
    __device__ __forceinline__ void settle()                 // once they are there
    {
        change([](float l) { return entry(l); });
    }
    template <typename F> __device__ __forceinline__ void each(F f) const
    {
#pragma unroll
        for (int v = 0; v < W / 4; ++v) {
            const int at = index(v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t a = x[4 * v + i];
                if constexpr (sizeof(T) == 2) {
                    asm volatile("" : "+v"(a));              // the halves are not kept beside the words
                    f(__uint_as_float(a << 16), at + 2 * i);
                    f(__uint_as_float(a & 0xffff0000u), at + 2 * i + 1);
                } else {
                    f(__uint_as_float(a), at + i);
                }
            }
        }
    }
    // f(entries, index of the first) for every four
    template <typename F> __device__ __forceinline__ void each4(F f) const
    {
#pragma unroll
        for (int v = 0; v < W / 4; ++v) {
            const int at = index(v);
#pragma unroll
            for (int j = 0; j < VE / 4; ++j) {
                float l[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (sizeof(T) == 2) {
                        uint32_t a = x[4 * v + 2 * j + i / 2];
                        asm volatile("" : "+v"(a));
                        l[i] = __uint_as_float(i % 2 ? a & 0xffff0000u : a << 16);
                    } else {
                        l[i] = __uint_as_float(x[4 * v + i]);
                    }
                }
                f(l, at + 4 * j);
            }
        }
    }
    template <typename F> __device__ __forceinline__ void change(F f)
    {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if constexpr (sizeof(T) == 2)
                x[i] = __float_as_uint(f(__uint_as_float(x[i] << 16))) >> 16 |
                       __float_as_uint(f(__uint_as_float(x[i] & 0xffff0000u)));
            else
                x[i] = __float_as_uint(f(__uint_as_float(x[i])));
        }
    }
    __device__ __forceinline__ void only_infinite()
    {
        change([](float l) { return entry(l, true); });
    }
};

template <int THREADS> __device__ __forceinline__ void clear(Hist& h)
{
    for (int i = threadIdx.x; i < kBuckets; i += THREADS) {
        h.mass[i] = 0;
        h.count[i] = 0;
    }
}

// Sums over the lanes up to and with each, in registers: shifts by 1, 2, 4, 8 within rows of 16 lanes, then the
// rows' last lanes to the rows behind them.
template <int CTRL, int ROWS> __device__ __forceinline__ uint32_t moved(uint32_t x)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS> __device__ __forceinline__ uint64_t moved(uint64_t x)
{
    return (uint64_t)moved<CTRL, ROWS>((uint32_t)(x >> 32)) << 32 | moved<CTRL, ROWS>((uint32_t)x);
}
template <typename N> __device__ __forceinline__ N row_scan(N x)         // of 16 lanes
{
    x += moved<0x111, 0xF>(x);
    x += moved<0x112, 0xF>(x);
    x += moved<0x114, 0xF>(x);
    return x + moved<0x118, 0xF>(x);
}
template <typename N> __device__ __forceinline__ N lane_scan(N x)
{
    x = row_scan(x);
    x += moved<0x142, 0xA>(x);
    return x + moved<0x143, 0xC>(x);
}
__device__ __forceinline__ uint32_t at_lane(uint32_t x, int lane) { return __builtin_amdgcn_readlane(x, lane); }
__device__ __forceinline__ uint64_t at_lane(uint64_t x, int lane)
{
    return (uint64_t)at_lane((uint32_t)(x >> 32), lane) << 32 | at_lane((uint32_t)x, lane);
}

// Sums up to and with each bucket.
template <int THREADS> __device__ __forceinline__ void scan(Hist& h, Shared& s)
{
    constexpr int PER = kBuckets / THREADS, WAVES = THREADS / 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    __syncthreads();
    uint64_t m[PER], mt = 0;
    uint32_t c[PER], ct = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        m[i] = mt += h.mass[PER * tid + i];
        c[i] = ct += h.count[PER * tid + i];
    }
    const uint64_t m_own = mt;
    const uint32_t c_own = ct;
    mt = lane_scan(mt);
    ct = lane_scan(ct);
    if (lane == 63) {
        s.wave_mass[wave] = mt;
        s.wave_count[wave] = ct;
    }
    __syncthreads();
    static_assert(WAVES <= 16, "the wavefronts before this one in a row of lanes");
    mt += at_lane(row_scan(lane < wave ? s.wave_mass[lane] : 0), 15) - m_own;
    ct += at_lane(row_scan(lane < wave ? s.wave_count[lane] : 0), 15) - c_own;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        h.mass[PER * tid + i] = mt + m[i];
        h.count[PER * tid + i] = ct + c[i];
    }
    __syncthreads();
}

// The largest value of the lanes, in registers.
template <int CTRL, int ROWS> __device__ __forceinline__ float max_moved(float x)
{
    return fmaxf(x, __uint_as_float(__builtin_amdgcn_update_dpp(__float_as_uint(x), __float_as_uint(x), CTRL, ROWS, 0xF, false)));
}
__device__ __forceinline__ float lane_max(float x)
{
    x = max_moved<0x111, 0xF>(x);
    x = max_moved<0x112, 0xF>(x);
    x = max_moved<0x114, 0xF>(x);
    x = max_moved<0x118, 0xF>(x);
    x = max_moved<0x142, 0xA>(x);
    x = max_moved<0x143, 0xC>(x);
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), 63));
}

// The largest and smallest entry, over the workgroup.
template <int THREADS> __device__ __forceinline__ void reduce(float& hi, float& lo, Shared& s)
{
    constexpr int WAVES = THREADS / 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    hi = lane_max(hi);
    lo = -lane_max(-lo);
    if (lane == 0) {
        s.wave_max[wave] = hi;
        s.wave_min[wave] = lo;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        hi = fmaxf(hi, s.wave_max[w]);
        lo = fminf(lo, s.wave_min[w]);
    }
    __syncthreads();
}

// An instruction each: the compiler would first make quiet the NaN that entries are not.
__device__ __forceinline__ float larger(float a, float b)
{
    asm("v_max_f32 %0, %1, %0" : "+v"(a) : "v"(b));
    return a;
}
__device__ __forceinline__ float smaller(float a, float b)
{
    asm("v_min_f32 %0, %1, %0" : "+v"(a) : "v"(b));
    return a;
}

// The largest entry (-infinity: there is none) and the smallest that counts.
template <typename Source> __device__ __forceinline__ void extremes(const Source& row, float& hi, float& lo)
{
    hi = -infinity();
    lo = infinity();
    row.each([&](float l, int) {
        hi = larger(hi, l);
        lo = smaller(lo, live_entry(l) ? l : infinity());
    });
}

// The lowest index of an entry that equals hi.
template <typename Source> __device__ __forceinline__ int index_of(const Source& row, float hi, Shared& s)
{
    if (threadIdx.x == 0)
        s.at = INT32_MAX;
    __syncthreads();
    int arg = INT32_MAX;
    row.each([&](float l, int i) { arg = l == hi && i < arg ? i : arg; });
    if (arg != INT32_MAX)
        atomicMin(&s.at, arg);
    __syncthreads();
    return s.at;
}

__device__ __forceinline__ Scale scale_of(float hi, float lo, float t)
{
    Scale r;
    const bool infinite = hi == infinity();
    r.max = infinite ? 0.f : hi;
    r.min = infinite ? 0.f : lo;
    // a difference beyond fp32 counts as its largest number (both lines keep a slope, entries that far down share the
    // last bucket), and no slope exceeds 2^125, so that logit_at can invert both
    const float range = fminf(r.max - r.min, 3.402823466e38f), near = kNats * t;
    constexpr float steepest = 4.253529587e37f;
    if (range * ((float)kNear / kLast) > near) {             // the far buckets are the wider ones
        r.step = fminf(kNear / near, steepest);
        r.far_step = fminf((kLast - kNear) / (range - near), steepest);
        r.far_from = kNear - near * r.far_step;
    } else {
        r.step = range > 0.f ? fminf(kLast / range, steepest) : 0.f;
        r.far_step = r.step;
        r.far_from = (float)kLast;
    }
    const double t64 = fmin((double)t, 1e300);               // an infinite one leaves -infinity no weight either
    r.c = 46.166241308446828384 / t64;                       // 32 log2 e
    r.top = r.max;
    r.least = -31.191623125197541 * t64;                     // 45 ln 2
    return r;
}

struct Settings {
    int64_t stride;
    int vocab, chunk, chunks;
    const float* temperature;
    const int32_t* top_k;
    const float *top_p, *min_p, *u;
    int32_t* tokens;
    float* probs;
};

__device__ __forceinline__ Wish wish_of(const Settings& a, int64_t n)
{
    Wish w;
    w.t = a.temperature ? a.temperature[n] : 1.f;
    w.p = a.top_p ? a.top_p[n] : 1.f;
    w.m = a.min_p && a.min_p[n] > 0.f ? fminf(a.min_p[n], 1.f) : 0.f;     // NaN: off
    const int k = a.top_k ? a.top_k[n] : 0;
    w.k = k > 0 && k < a.vocab ? k : 0;
    w.draw = a.tokens != nullptr;
    const float u = w.draw ? a.u[n] : 0.f;
    w.at = u >= 1.f ? 1. - 5.9604644775390625e-8 : u > 0.f ? (double)u : 0.;         // below 1 by an fp32 half step
    return w;
}

// The entries into a cleared histogram.
template <typename Source>
__device__ __forceinline__ void fill(const Source& row, const Scale& r, bool counted, Shared& s)
{
    const Constants k;
    row.each4([&](const float(&l)[4], int) {
        int b[4];
        uint64_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            b[e] = bucket_of(r, l[e]);
            w[e] = steps_of(k, r, s.table, l[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (w[e])
                atomicAdd((unsigned long long*)&s.h.mass[b[e]], (unsigned long long)w[e]);
        if (counted)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (live_entry(l[e]))
                    atomicAdd(&s.h.count[b[e]], 1u);
    });
}

__device__ __forceinline__ void start_table(Shared& s)
{
    if (threadIdx.x < 32)
        s.table[threadIdx.x] = exp2(threadIdx.x / 32.);
}

// The places that are looked for in the order.
enum Place {
    kCount,                                                  // the goal-th entry
    kReach,                                                  // the entry with which the weight reaches the goal
    kPass,                                                   // the entry with which the weight exceeds the goal
    kUpTo                                                    // the entry that has the goal for its place
};

// Whether a step from (count, mass) before it by (dc, dm) takes in the place.
__device__ __forceinline__ bool takes(Place place, uint64_t goal, uint64_t mass, uint64_t dm, uint32_t count, uint32_t dc)
{
    if (place == kCount)
        return count < goal && goal <= (uint64_t)count + dc;
    if (place == kReach)
        return mass < goal && goal <= mass + dm;
    return mass <= goal && goal < mass + dm;
}

// The goals of top-p and of the draw for a weight that is left.
__device__ __forceinline__ uint64_t reach_goal(float p, uint64_t total)
{
    return (uint64_t)fmax(ceil((double)p * (double)total), 1.);
}
__device__ __forceinline__ uint64_t pass_goal(double at, uint64_t total) { return (uint64_t)(at * (double)total); }

// min_p's place: behind the smallest logit whose weight is at least m.  False where that keeps every entry.
__device__ __forceinline__ bool least_place(const Scale& r, const Wish& w, uint64_t& order, int& bucket)
{
    const double least = log((double)w.m), back = 1. / (double)w.t;
    float l = (float)((double)r.max + least * (double)w.t);
    auto heavy = [&](float v) { return ((double)v - (double)r.max) * back >= least; };
    for (int i = 0; i < 4 && !heavy(l); ++i)
        l = of_key(key_of(l) + 1);
    for (int i = 0; i < 4 && heavy(of_key(key_of(l) - 1)); ++i)
        l = of_key(key_of(l) - 1);
    order = order_of(l, kSampleMaxVocab - 1);
    bucket = bucket_of(r, l);
    return l > r.min;
}

// The first bucket whose sum takes in the goal, by one wavefront: of every sixteenth, then of the sixteen before it.
__device__ __forceinline__ int first_bucket(const Hist& h, Place place, uint64_t goal)
{
    const int lane = threadIdx.x & 63;
    auto reached = [&](int b) {
        return place == kCount ? h.count[b] >= goal : place == kReach ? h.mass[b] >= goal : h.mass[b] > goal;
    };
    const uint64_t coarse = __ballot(reached(16 * lane + 15));
    const int from = coarse ? 16 * (__ffsll((unsigned long long)coarse) - 1) : kBuckets - 16;
    const uint64_t fine = __ballot(reached(from + (lane & 15)));
    return fine ? from + __ffsll((unsigned long long)fine) - 1 : kLast;
}

// The logit at a height, off to the given side by its rounding; where all have one height that side's infinity.
__device__ __forceinline__ float logit_at(const Scale& r, float height, float side)
{
    float d = height * __builtin_amdgcn_rcpf(r.step);
    if (r.far_step > 0.f)
        d = fmaxf(d, (height - r.far_from) * __builtin_amdgcn_rcpf(r.far_step));
    const float l = r.max - d + side * 4.7683716e-7f * (fabsf(r.max) + fabsf(d));     // 2^-21
    return r.step > 0.f && fabsf(l) < infinity() ? l : side * infinity();
}

// Each filter leaves a weight between two sums of buckets; so each goal, and the bucket of each place, lies between
// two others.  By the first wavefront, into s.plan.
__device__ __forceinline__ void make_plan(const Hist& h, const Scale& r, const Wish& w, Shared& s)
{
    if (threadIdx.x < 64) {
        int from[4], to[4], n = 0;
        Plan q;
        uint64_t lo = h.mass[kLast], hi = lo;                // the weight that is left
        q.k = w.k > 0 && (uint32_t)w.k < h.count[kLast];
        q.p = w.p < 1.f;
        q.m = -1;
        q.m_order = kNowhere;
        if (q.k) {
            const int b = first_bucket(h, kCount, w.k);
            lo = h.mass_before(b);
            hi = h.mass[b];
            from[0] = to[0] = b;
            n = 1;
        }
        if (q.p) {
            const uint64_t least = reach_goal(w.p, lo);
            const int f = first_bucket(h, kReach, least), t = first_bucket(h, kReach, reach_goal(w.p, hi));
            lo = least;
            hi = h.mass[t] < hi ? h.mass[t] : hi;
            from[n] = f;
            to[n++] = t;
        }
        uint64_t order;
        int bucket;
        if (w.m > 0.f && least_place(r, w, order, bucket)) {
            q.m = bucket;
            q.m_order = order;
            lo = h.mass_before(bucket) < lo ? h.mass_before(bucket) : lo;
            hi = h.mass[bucket] < hi ? h.mass[bucket] : hi;
            from[n] = to[n] = bucket;
            ++n;
        }
        if (w.draw) {
            from[n] = first_bucket(h, kPass, pass_goal(w.at, lo));
            to[n] = first_bucket(h, kPass, pass_goal(w.at, hi));
            ++n;
        }
        if (threadIdx.x == 0) {
            // overlapping ranges become one: an entry is collected once
            int m = 0;
            for (int i = 0; i < n; ++i) {
                int f = from[i], t = to[i];
                for (int j = 0; j < m;)
                    if (from[j] <= t && to[j] >= f) {
                        f = from[j] < f ? from[j] : f;
                        t = to[j] > t ? to[j] : t;
                        --m;
                        from[j] = from[m];
                        to[j] = to[m];
                        j = 0;
                    } else {
                        ++j;
                    }
                from[m] = f;
                to[m++] = t;
            }
            q.ranges = m;
            for (int i = 0; i < 4; ++i) {
                q.from[i] = i < m ? (float)from[i] : infinity();
                q.to[i] = i < m ? (float)(to[i] + 1) : -infinity();
            }
            s.plan = q;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (threadIdx.x < 4) {                               // a hundredth of a bucket wider than the range: heights
            const int i = threadIdx.x;                       // up to 1024 and their inverses are off by 2^-11 at most
            const float f = s.plan.from[i], t = s.plan.to[i];
            const float high = fminf(logit_at(r, f - 0.01f, 1.f), r.max);
            const float low = t < (float)kBuckets ? fmaxf(logit_at(r, t + 0.01f, -1.f), r.min) : r.min;
            const float off = 2.3841858e-7f * (fabsf(high) + fabsf(low)) + 1.175494351e-38f;     // 2^-22: their own roundings
            s.plan.middle[i] = f < t ? 0.5f * high + 0.5f * low : 0.f;
            s.plan.reach[i] = f < t ? 0.5f * high - 0.5f * low + off : -infinity();
        }
    }
    __syncthreads();
}

// The entries for which in(l, i) holds, into the list (in any order); s.number of them.  beyond(l) is positive for none
// of these, and for most others.
template <typename Source, typename G, typename F>
__device__ __forceinline__ void gather(const Source& row, Shared& s, G beyond, F in)
{
    if (threadIdx.x == 0)
        s.number = 0;
    __syncthreads();
    row.each4([&](const float(&l)[4], int i) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            x[e] = beyond(l[e]);
        if (fminf(fminf(x[0], x[1]), fminf(x[2], x[3])) <= 0.f) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (x[e] <= 0.f && in(l[e], i + e)) {
                    const uint32_t at = atomicAdd(&s.number, 1u);
                    if (at < kList)
                        s.x.list.order[at] = order_of(l[e], i + e);
                }
        }
    });
    __syncthreads();
}

// Those of the plan's ranges.
template <typename Source> __device__ __forceinline__ void gather_plan(const Source& row, const Scale& r, Shared& s)
{
    const Plan q = s.plan;
    const bool more = __builtin_amdgcn_readfirstlane(q.ranges) > 2;
    // no lane masks for each entry: the scalar unit's operations on them would be half of the work
    auto beyond = [&](float l) {
        float x = fminf(fabsf(l - q.middle[0]) - q.reach[0], fabsf(l - q.middle[1]) - q.reach[1]);
        if (more)
            x = fminf(fminf(x, fabsf(l - q.middle[2]) - q.reach[2]), fabsf(l - q.middle[3]) - q.reach[3]);
        return x;
    };
    gather(row, s, beyond, [&](float l, int) {
        const float f = height_of(r, l);
        bool hit = false;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            hit |= f >= q.from[i] && f < q.to[i];
        return hit && live_entry(l);
    });
}

// The value of the lane that differs in the bit FAR (1 to 32), in registers where there is an instruction for it.
template <int FAR> __device__ __forceinline__ uint32_t other(uint32_t x)
{
    if constexpr (FAR == 1)
        return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, false);
    else if constexpr (FAR == 2)
        return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, false);
    else if constexpr (FAR == 8)
        return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x128, 0xF, 0xF, false);
    else if constexpr (FAR == 4 || FAR == 16)
        return (uint32_t)__builtin_amdgcn_ds_swizzle((int)x, FAR << 10 | 0x1F);
    else {
        const auto both = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        return threadIdx.x & 32 ? both[0] : both[1];
    }
}
template <int FAR> __device__ __forceinline__ uint64_t other(uint64_t x)
{
    return (uint64_t)other<FAR>((uint32_t)(x >> 32)) << 32 | other<FAR>((uint32_t)x);
}

// A step of a bitonic sort within wavefronts: entry i of runs of `run`.
template <int FAR> __device__ __forceinline__ uint64_t exchanged(uint64_t x, int i, int run)
{
    const uint64_t y = other<FAR>(x);
    const bool up = ((i & run) == 0) == ((i & FAR) == 0);    // the smaller one is kept here
    return (x < y) == up ? x : y;
}
// All steps within a wavefront of the stage that makes runs of `run`.
template <typename F> __device__ __forceinline__ void near_steps(int run, F step)
{
    if (run > 32) step(std::integral_constant<int, 32>{});
    if (run > 16) step(std::integral_constant<int, 16>{});
    if (run > 8) step(std::integral_constant<int, 8>{});
    if (run > 4) step(std::integral_constant<int, 4>{});
    if (run > 2) step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 1>{});
}

// The places looked up one after the other among the s.number <= 64 entries of the list.  What is before an entry is
// found by comparing it with the others of its bucket or, from 9 entries on, by sorting them and adding up (40 entries:
// 3800 cycles by sorting, 9600 by comparing; 10: 3800 and 4200; 3: 2700 by comparing).  By the first wavefront, into
// s.choice.
__device__ __forceinline__ void choose_few(const Hist& h, const Scale& r, const Wish& w, Shared& s)
{
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x, n = (int)s.number;
        const Plan q = s.plan;
        const bool there = lane < n;
        uint64_t x = there ? s.x.list.order[lane] : kNowhere;
        if (n > 8)
            for (int run = 2; run <= 64; run *= 2)
                near_steps(run, [&](auto far) { x = exchanged<decltype(far)::value>(x, lane, run); });
        const int bucket = there ? bucket_of(r, logit_of(x)) : -1;
        const uint64_t own = there ? steps_of(r, s.table, logit_of(x)) : 0;
        uint64_t mass = there ? h.mass_before(bucket) : 0;
        uint32_t count = there ? h.count_before(bucket) : 0;
        if (n > 8) {
            const uint64_t sum = lane_scan(own) - own;
            const int previous = __shfl_up(bucket, 1);       // by all lanes
            const uint64_t firsts = __ballot(lane == 0 || previous != bucket) & (~0ull >> (63 - lane));
            const int at = 63 - __clzll((long long)firsts);  // the bucket's first lane
            mass += sum - ((uint64_t)(uint32_t)__shfl((int)(sum >> 32), at) << 32 | (uint32_t)__shfl((int)sum, at));
            count += lane - at;
        } else {
            for (int i = 0; i < n; ++i) {
                const bool before = at_lane(x, i) < x && (int)at_lane((uint32_t)bucket, i) == bucket;
                mass += before ? at_lane(own, i) : 0;
                count += before;
            }
        }
        Choice c = {kNowhere, h.mass[kLast], -1};
        bool missed = false;
        auto look = [&](Place place, uint64_t goal) {
            const uint64_t hit = __ballot(there && takes(place, goal, mass, own, count, 1));
            const int at = hit ? __ffsll((unsigned long long)hit) - 1 : 0;
            missed |= hit == 0;
            c.cut = at_lane(x, at);
            c.total = at_lane(mass + own, at);
        };
        if (q.k)
            look(kCount, w.k);
        if (q.p)
            look(kReach, reach_goal(w.p, c.total));
        if (q.m >= 0 && q.m_order < c.cut) {                 // with the entries of its bucket that are not behind it
            c.total = h.mass_before(q.m) + at_lane(lane_scan(there && bucket == q.m && x <= q.m_order ? own : (uint64_t)0), 63);
            c.cut = q.m_order;
        }
        if (w.draw) {
            const uint64_t hit = __ballot(there && takes(kPass, pass_goal(w.at, c.total), mass, own, count, 1));
            missed |= hit == 0;
            c.token = (int)(at_lane(x, hit ? __ffsll((unsigned long long)hit) - 1 : 0) & (kSampleMaxVocab - 1));
        }
        if (missed)
            c.total = 0;
        if (lane == 0)
            s.choice = c;
    }
    __syncthreads();
}

// The same with the list sorted (bitonic: within wavefronts by exchanged registers).
template <int THREADS>
__device__ __forceinline__ void choose_sorted(const Hist& h, const Scale& r, const Wish& w, Shared& s)
{
    constexpr int PER = kList / THREADS;                     // entries j * THREADS + tid of a thread
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = (int)s.number;
    const Plan q = s.plan;
    int size = 64;
    while (size < n)
        size *= 2;
    uint64_t x[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j)
        x[j] = j * THREADS + tid < n ? s.x.list.order[j * THREADS + tid] : kNowhere;
    if (tid < 3)
        s.place_mass[tid] = 0;
    for (int run = 2; run <= size; run *= 2) {
        for (int far = run / 2; far >= 64; far /= 2) {       // another wavefront's
            __syncthreads();
#pragma unroll
            for (int j = 0; j < PER; ++j)
                s.x.list.order[j * THREADS + tid] = x[j];
            __syncthreads();
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int i = j * THREADS + tid;
                const uint64_t y = s.x.list.order[i ^ far];
                const bool up = ((i & run) == 0) == ((i & far) == 0);
                x[j] = (x[j] < y) == up ? x[j] : y;
            }
        }
        if (wave * 64 < size)
            near_steps(run, [&](auto far) {
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    x[j] = exchanged<decltype(far)::value>(x[j], j * THREADS + tid, run);
            });
    }
    __syncthreads();
    // weights, and their sums in the order of the list
    uint64_t own[PER], sum[PER];
    int bucket[PER];
    uint64_t before = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = j * THREADS + tid;
        const bool there = i < n;
        const float l = there ? logit_of(x[j]) : r.max;
        bucket[j] = there ? bucket_of(r, l) : kLast;
        own[j] = there ? steps_of(r, s.table, l) : 0;
        sum[j] = lane_scan(own[j]);
        if (lane == 63)
            s.wave_mass[wave] = sum[j];
        if (there)
            s.x.list.order[i] = x[j];
        __syncthreads();
        uint64_t all = 0;
#pragma unroll
        for (int v = 0; v < THREADS / 64; ++v) {
            sum[j] += v < wave ? s.wave_mass[v] : 0;
            all += s.wave_mass[v];
        }
        sum[j] += before;
        before += all;
        __syncthreads();
    }
    // a bucket's first entry leaves its place and the sum before it
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = j * THREADS + tid;
        if (i < n && (i == 0 || bucket_of(r, logit_of(s.x.list.order[i - 1])) != bucket[j])) {
            s.first[bucket[j]] = i;
            s.x.list.mass[i] = sum[j] - own[j];
        }
    }
    __syncthreads();
    uint64_t mass[PER];
    uint32_t count[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = j * THREADS + tid;
        mass[j] = count[j] = 0;
        if (i < n) {
            const int f = s.first[bucket[j]];
            mass[j] = h.mass_before(bucket[j]) + (sum[j] - own[j] - s.x.list.mass[f]);
            count[j] = h.count_before(bucket[j]) + (uint32_t)(i - f);
        }
    }
    Choice c = {kNowhere, h.mass[kLast], -1};
    bool missed = false;
    auto look = [&](int which, Place place, uint64_t goal) {
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (j * THREADS + tid < n && takes(place, goal, mass[j], own[j], count[j], 1)) {
                s.place_order[which] = x[j];
                s.place_mass[which] = mass[j] + own[j];
            }
        __syncthreads();
        missed |= s.place_mass[which] == 0;
    };
    if (q.k) {
        look(0, kCount, w.k);
        c.cut = s.place_order[0];
        c.total = s.place_mass[0];
    }
    if (q.p) {
        look(1, kReach, reach_goal(w.p, c.total));
        c.cut = s.place_order[1];
        c.total = s.place_mass[1];
    }
    if (q.m >= 0 && q.m_order < c.cut) {                     // up to the last entry of its bucket that is not behind it
        __syncthreads();
        if (tid == 0)
            s.found_mass = h.mass_before(q.m);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (j * THREADS + tid < n && bucket[j] == q.m && x[j] <= q.m_order)
                atomicMax((unsigned long long*)&s.found_mass, (unsigned long long)(mass[j] + own[j]));
        __syncthreads();
        c.cut = q.m_order;
        c.total = s.found_mass;
    }
    if (w.draw) {
        look(2, kPass, pass_goal(w.at, c.total));
        c.token = (int)(s.place_order[2] & (kSampleMaxVocab - 1));
    }
    if (missed)
        c.total = 0;
    if (tid == 0)
        s.choice = c;
    __syncthreads();
}

// The bucket of a scanned histogram that takes in the place, and what is before it.  For kUpTo
// it is the bucket `given`.
template <int THREADS>
__device__ __forceinline__ void find_bucket(const Hist& h, Shared& s, Place place, uint64_t goal, int given,
                                            uint64_t mass0, uint32_t count0)
{
    for (int b = threadIdx.x; b < kBuckets; b += THREADS) {
        const uint64_t m0 = h.mass_before(b);
        const uint32_t c0 = h.count_before(b);
        if (place == kUpTo ? b == given : takes(place, goal, mass0 + m0, h.mass[b] - m0, count0 + c0, h.count[b] - c0)) {
            s.at = b;
            s.base_mass = mass0 + m0;
            s.base_count = count0 + c0;
        }
    }
    __syncthreads();
}

// One place after the other, where the list cannot hold the entries of all: its bucket's entries are cut by digits of
// the order until kList are left, and compared with each other.  s.found_order is the place's entry and
// s.found_mass the weight up to and with it; for kUpTo the weight of the entries whose place is at most `goal`, which
// lies in bucket `given`.
template <typename Source>
__device__ __forceinline__ void find(const Source& row, const Scale& r, Shared& s, Place place, uint64_t goal, int given)
{
    constexpr int THREADS = Source::THREADS;
    const int tid = threadIdx.x;
    find_bucket<THREADS>(s.h, s, place, goal, given, 0, 0);
    const int bucket = s.at;
    uint64_t prefix = 0;
    int shift = 32 + kIndexBits;
    auto in = [&](float l, int i) {
        return live_entry(l) && bucket_of(r, l) == bucket && order_of(l, i) >> shift == prefix;
    };
    const auto any = [](float) { return 0.f; };
    gather(row, s, any, in);
#pragma unroll 1
    while (s.number > kList) {                               // at shift 0 one entry is left
        const int next = shift > kDigitBits ? shift - kDigitBits : 0, mask = (1 << (shift - next)) - 1;
        const uint64_t mass0 = s.base_mass;
        const uint32_t count0 = s.base_count;
        clear<THREADS>(s.x.digits);
        __syncthreads();
        row.each([&](float l, int i) {
            if (in(l, i)) {
                const int d = (int)(order_of(l, i) >> next) & mask;
                atomicAdd(&s.x.digits.count[d], 1u);
                atomicAdd((unsigned long long*)&s.x.digits.mass[d], (unsigned long long)steps_of(r, s.table, l));
            }
        });
        scan<THREADS>(s.x.digits, s);
        find_bucket<THREADS>(s.x.digits, s, place, goal, (int)(goal >> next) & mask, mass0, count0);
        prefix = prefix << (shift - next) | (uint32_t)s.at;
        shift = next;
        gather(row, s, any, in);
    }
    const uint64_t mass0 = s.base_mass;
    const uint32_t count0 = s.base_count;
    const int n = (int)s.number;
    for (int j = tid; j < n; j += THREADS)
        s.x.list.mass[j] = steps_of(r, s.table, logit_of(s.x.list.order[j]));
    if (tid == 0)
        s.found_mass = mass0;
    __syncthreads();
    for (int j = tid; j < n; j += THREADS) {
        const uint64_t mine = s.x.list.order[j], w = s.x.list.mass[j];
        if (place == kUpTo) {
            if (mine <= goal)
                atomicAdd((unsigned long long*)&s.found_mass, (unsigned long long)w);
        } else {
            uint64_t mass = mass0;
            uint32_t count = count0;
            for (int i = 0; i < n; ++i) {
                const bool before = s.x.list.order[i] < mine;
                mass += before ? s.x.list.mass[i] : 0;
                count += before;
            }
            if (takes(place, goal, mass, w, count, 1)) {
                s.found_order = mine;
                s.found_mass = mass + w;
            }
        }
    }
    __syncthreads();
}

template <typename Source>
__device__ __forceinline__ void choose_slowly(const Source& row, const Scale& r, const Wish& w, Shared& s)
{
    const Plan q = s.plan;
    Choice c = {kNowhere, s.h.mass[kLast], -1};
#pragma unroll 1
    for (int step = 0; step < 4; ++step) {
        Place place = kPass;
        uint64_t goal = 0;
        if (step == 0) {
            if (!q.k)
                continue;
            place = kCount;
            goal = w.k;
        } else if (step == 1) {
            if (!q.p)
                continue;
            place = kReach;
            goal = reach_goal(w.p, c.total);
        } else if (step == 2) {
            if (q.m < 0 || q.m_order >= c.cut)
                continue;
            place = kUpTo;
            goal = q.m_order;
        } else {
            if (!w.draw)
                continue;
            goal = pass_goal(w.at, c.total);
        }
        find(row, r, s, place, goal, q.m);
        if (step < 3) {
            c.cut = place == kUpTo ? goal : s.found_order;
            c.total = s.found_mass;
        } else {
            c.token = (int)(s.found_order & (kSampleMaxVocab - 1));
        }
        __syncthreads();
    }
    if (threadIdx.x == 0)
        s.choice = c;
    __syncthreads();
}

// The choice from a scanned histogram, a plan and the list.  Rows that the list does not hold are read again, and so are
// those where a place is not found in it, which the histogram alone then finds: no token is made up.
template <typename Source>
__device__ __forceinline__ void choose(const Source& again, const Scale& r, const Wish& w, Shared& s)
{
    const uint32_t number = s.number;
    if (number <= 64)
        choose_few(s.h, r, w, s);
    else if (number <= kList)
        choose_sorted<Source::THREADS>(s.h, r, w, s);
    if (number > kList || s.choice.total == 0)
        choose_slowly(again, r, w, s);
}

// The probability of an entry after the cut, in the share that the kept weight has of it.
__device__ __forceinline__ float probability(const Constants& k, const Scale& r, const double* table, const Choice& c,
                                             double share, float l, int i)
{
    return live_entry(l) && order_of(l, i) <= c.cut ? (float)(weight_of(k, r, table, l) * share) : 0.f;
}

// The distribution that is left of the entries.
template <typename Source>
__device__ __forceinline__ void put_probs(const Source& row, const Scale& r, const Shared& s, const Choice& c, float* out)
{
    const double share = kOne / (double)c.total;
    const Constants k;
    row.each4([&](const float(&l)[4], int i) {
        rows::AtElement a;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            a[e] = __float_as_uint(probability(k, r, s.table, c, share, l[e], i + e));
        if (i + 4 <= row.end) {
            *reinterpret_cast<rows::AtElement*>(out + i) = a;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e < row.end)
                    out[i + e] = __uint_as_float(a[e]);
        }
    });
}

}  // namespace

// A row of logits by one workgroup.
template <typename T, typename Source>
__global__ __launch_bounds__(Source::THREADS) void sample_row_kernel(const T* __restrict__ logits, Settings a)
{
    constexpr int THREADS = Source::THREADS;
    __shared__ Shared s;
    const int tid = threadIdx.x, vocab = a.vocab;
    const int64_t n = blockIdx.x;
    Source row;
    row.row = logits + n * a.stride;
    row.first = 0;
    row.end = vocab;
    const Wish w = wish_of(a, n);
    row.load();
    start_table(s);                                          // while they are on their way
    clear<THREADS>(s.h);
    row.settle();
    float* out = a.probs ? a.probs + n * vocab : nullptr;
    float hi, lo;
    extremes(row, hi, lo);
    reduce<THREADS>(hi, lo, s);
    if (!live_entry(hi) || !(w.t > 0.f)) {                         // nothing to draw from, or the largest is taken
        const int arg = !live_entry(hi) ? -1 : index_of(row, hi, s);
        if (a.tokens && tid == 0)
            a.tokens[n] = arg;
        if (out)
            for (int i = tid; i < vocab; i += THREADS)
                out[i] = i == arg ? 1.f : 0.f;
        return;
    }
    const Scale r = scale_of(hi, lo, w.t);
    Streamed<T, THREADS> again = {row.row, 0, vocab, false};
    if (hi == infinity()) {                                  // nothing else counts
        row.only_infinite();
        again.only_infinite();
    }
    fill(row, r, w.k > 0, s);
    scan<THREADS>(s.h, s);
    make_plan(s.h, r, w, s);
    gather_plan(row, r, s);
    choose(again, r, w, s);
    const Choice c = s.choice;
    if (a.tokens && tid == 0)
        a.tokens[n] = c.token;
    if (out)                                                 // read again, so that no registers are held for it
        put_probs(again, r, s, c, out);
}

// ---- rows cut into chunks

// What is left of a row between the launches.
struct Parts {
    float *hi, *lo;                                          // [rows][chunks]
    uint32_t* number;                                        // [rows][chunks]: entries in the chunk's list
    uint64_t* mass;                                          // [rows][chunks][kBuckets], then of the row [rows][kBuckets]
    uint32_t* count;
    uint64_t* list;                                          // [rows][chunks][kList]
    Plan* plan;                                              // [rows]
    Choice* choice;
};

namespace {

template <typename Source, typename T>
__device__ __forceinline__ Source chunk_of(const T* logits, const Settings& a, int64_t n, int chunk)
{
    Source row;
    row.row = logits + n * a.stride;
    row.first = chunk * a.chunk;
    row.end = a.vocab - row.first < a.chunk ? a.vocab : row.first + a.chunk;
    row.load();
    return row;                                              // to be settled
}

// The row's extremes from its chunks'.
__device__ __forceinline__ void row_extremes(const Parts& x, const Settings& a, int64_t n, float& hi, float& lo)
{
    hi = -infinity();
    lo = infinity();
    for (int c = 0; c < a.chunks; ++c) {
        hi = fmaxf(hi, x.hi[n * a.chunks + c]);
        lo = fminf(lo, x.lo[n * a.chunks + c]);
    }
}

// A row's scanned histogram from its chunks'.
template <int THREADS>
__device__ __forceinline__ void sum_chunks(const Parts& x, const Settings& a, int64_t n, bool counted, Shared& s)
{
    constexpr int PER = kBuckets / THREADS;
    const int64_t from = n * a.chunks * kBuckets;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = i * THREADS + threadIdx.x;
        uint64_t m = 0;
        uint32_t c = 0;
#pragma unroll 8
        for (int j = 0; j < a.chunks; ++j) {
            m += x.mass[from + (int64_t)j * kBuckets + b];
            if (counted)
                c += x.count[from + (int64_t)j * kBuckets + b];
        }
        s.h.mass[b] = m;
        s.h.count[b] = c;
    }
    scan<THREADS>(s.h, s);
}

}  // namespace

template <typename T, typename Source>
__global__ __launch_bounds__(Source::THREADS) void sample_max_kernel(const T* __restrict__ logits, Settings a, Parts x)
{
    __shared__ Shared s;
    const int64_t n = blockIdx.x / a.chunks;
    const int chunk = blockIdx.x % a.chunks;
    Source row = chunk_of<Source>(logits, a, n, chunk);
    row.settle();
    float hi, lo;
    extremes(row, hi, lo);
    reduce<Source::THREADS>(hi, lo, s);
    if (threadIdx.x == 0) {
        x.hi[blockIdx.x] = hi;
        x.lo[blockIdx.x] = lo;
    }
}

template <typename T, typename Source>
__global__ __launch_bounds__(Source::THREADS) void sample_hist_kernel(const T* __restrict__ logits, Settings a, Parts x)
{
    constexpr int THREADS = Source::THREADS;
    __shared__ Shared s;
    const int64_t n = blockIdx.x / a.chunks;
    Source row = chunk_of<Source>(logits, a, n, blockIdx.x % a.chunks);
    const Wish w = wish_of(a, n);
    float hi, lo;
    row_extremes(x, a, n, hi, lo);
    if (!live_entry(hi) || !(w.t > 0.f))
        return;
    start_table(s);
    clear<THREADS>(s.h);
    row.settle();
    __syncthreads();
    const Scale r = scale_of(hi, lo, w.t);
    if (hi == infinity())
        row.only_infinite();
    fill(row, r, w.k > 0, s);
    __syncthreads();
    const int64_t to = (int64_t)blockIdx.x * kBuckets;
    for (int b = threadIdx.x; b < kBuckets; b += THREADS) {
        x.mass[to + b] = s.h.mass[b];
        if (w.k > 0)
            x.count[to + b] = s.h.count[b];
    }
}

template <typename T, typename Source>
__global__ __launch_bounds__(Source::THREADS) void sample_gather_kernel(const T* __restrict__ logits, Settings a, Parts x)
{
    constexpr int THREADS = Source::THREADS;
    __shared__ Shared s;
    const int64_t n = blockIdx.x / a.chunks;
    const int chunk = blockIdx.x % a.chunks, tid = threadIdx.x;
    Source row = chunk_of<Source>(logits, a, n, chunk);
    const Wish w = wish_of(a, n);
    float hi, lo;
    row_extremes(x, a, n, hi, lo);
    if (!live_entry(hi) || !(w.t > 0.f)) {                   // in place of a list: where the maximum is first
        row.settle();
        const int arg = !live_entry(hi) ? INT32_MAX : index_of(row, hi, s);
        if (tid == 0)
            x.number[blockIdx.x] = (uint32_t)arg;
        return;
    }
    const Scale r = scale_of(hi, lo, w.t);
    sum_chunks<THREADS>(x, a, n, w.k > 0, s);
    make_plan(s.h, r, w, s);
    row.settle();
    if (hi == infinity())
        row.only_infinite();
    if (chunk == 0) {
        const int64_t to = ((int64_t)gridDim.x + n) * kBuckets;
        for (int b = tid; b < kBuckets; b += THREADS) {
            x.mass[to + b] = s.h.mass[b];
            x.count[to + b] = s.h.count[b];
        }
        if (tid == 0)
            x.plan[n] = s.plan;
    }
    gather_plan(row, r, s);
    if (tid == 0)
        x.number[blockIdx.x] = s.number;
    const int here = s.number < kList ? (int)s.number : kList;
    for (int j = tid; j < here; j += THREADS)
        x.list[(int64_t)blockIdx.x * kList + j] = s.x.list.order[j];
}

template <typename T>
__global__ __launch_bounds__(1024) void sample_choose_kernel(const T* __restrict__ logits, Settings a, Parts x)
{
    constexpr int THREADS = 1024;
    __shared__ Shared s;
    const int64_t n = blockIdx.x, rows = gridDim.x;
    const int tid = threadIdx.x;
    const Wish w = wish_of(a, n);
    float hi, lo;
    row_extremes(x, a, n, hi, lo);
    if (!live_entry(hi) || !(w.t > 0.f)) {
        int arg = INT32_MAX;
        for (int c = 0; c < a.chunks; ++c) {
            const int i = (int)x.number[n * a.chunks + c];
            arg = i < arg ? i : arg;
        }
        if (tid == 0) {
            if (a.tokens)
                a.tokens[n] = !live_entry(hi) ? -1 : arg;
            x.choice[n].token = !live_entry(hi) ? -1 : arg;
        }
        return;
    }
    const Scale r = scale_of(hi, lo, w.t);
    start_table(s);
    const int64_t from = (rows * a.chunks + n) * kBuckets;
    for (int b = tid; b < kBuckets; b += THREADS) {
        s.h.mass[b] = x.mass[from + b];
        s.h.count[b] = x.count[from + b];
    }
    uint32_t all = 0;                                        // chunks * vocab at most
    for (int c = 0; c < a.chunks; ++c) {
        const uint32_t here = x.number[n * a.chunks + c];
        if (here <= kList && all + here <= kList && (uint32_t)tid >= all && (uint32_t)tid < all + here)
            s.x.list.order[tid] = x.list[(n * a.chunks + c) * kList + tid - all];
        all += here;
    }
    if (tid == 0) {
        s.plan = x.plan[n];
        s.number = all;
    }
    __syncthreads();
    Streamed<T, THREADS> again = {logits + n * a.stride, 0, a.vocab, hi == infinity()};
    choose(again, r, w, s);
    if (tid == 0) {
        if (a.tokens)
            a.tokens[n] = s.choice.token;
        x.choice[n] = s.choice;
    }
}

template <typename T, typename Source>
__global__ __launch_bounds__(Source::THREADS) void sample_probs_kernel(const T* __restrict__ logits, Settings a, Parts x)
{
    __shared__ Shared s;
    const int64_t n = blockIdx.x / a.chunks;
    Source row = chunk_of<Source>(logits, a, n, blockIdx.x % a.chunks);
    row.settle();
    const Wish w = wish_of(a, n);
    float hi, lo;
    row_extremes(x, a, n, hi, lo);
    const Choice c = x.choice[n];
    float* out = a.probs + n * a.vocab;
    if (!live_entry(hi) || !(w.t > 0.f)) {
        row.each([&](float, int i) {
            if (i < a.vocab)
                out[i] = i == c.token ? 1.f : 0.f;
        });
        return;
    }
    start_table(s);
    __syncthreads();
    const Scale r = scale_of(hi, lo, w.t);
    if (hi == infinity())
        row.only_infinite();
    put_probs(row, r, s, c, out);
}

namespace {

struct Cut {
    int chunk, chunks;                                       // chunks 0: whole rows
};
// Rows are cut where one workgroup would have to read them again and again, and few of them would leave most compute
// units idle; into chunks of 16,384 where that takes no second round of workgroups.  us, fp32, whole rows, chunks of
// 16,384, of 32,768: 1 of 128,000 56, 22, 27; 64 of 128,000 76, 62, 49; 64 of 50,001 38 and 35, 96 of them 38 and 41;
// 128 of 128,000 79 and 100; 16 of 33,000 22 and 25; 8 of 32,000, which fit the registers, 22 and 32 (later steps took
// as much from both sides).  Rows longer than 128,000 go by the same limit, unmeasured against whole rows.
Cut cut_of(int64_t rows, int vocab)
{
    if (rows > 80 || vocab <= 40 * 1024)
        return {0, 0};
    constexpr int small = 1024 * 16, large = 1024 * 32;
    const int few = (vocab + small - 1) / small;
    if (rows * few <= 256)
        return {small, few};
    return {large, (vocab + large - 1) / large};
}

// The parts laid out one after the other, 256 bytes apart at least; returns the bytes.
size_t lay_out(int64_t rows, const Cut& c, char* at, Parts& x)
{
    size_t used = 0;
    auto take = [&](auto*& p, size_t count) {
        p = (typename std::remove_reference<decltype(p)>::type)(at + used);
        used += (count * sizeof(*p) + 255) / 256 * 256;
    };
    const size_t all = (size_t)rows * c.chunks;
    take(x.hi, all);
    take(x.lo, all);
    take(x.number, all);
    take(x.mass, (all + rows) * kBuckets);
    take(x.count, (all + rows) * kBuckets);
    take(x.list, all * kList);
    take(x.plan, rows);
    take(x.choice, rows);
    return used;
}

}  // namespace

bool sample_fits(int64_t rows) { return rows <= UINT32_MAX / 1024; }

size_t sample_workspace_bytes(int64_t rows, int vocab)
{
    const Cut c = cut_of(rows, vocab);
    Parts x;
    return c.chunks ? lay_out(rows, c, nullptr, x) : 0;
}

static Settings settings_of(const SampleArgs& p, const Cut& c)
{
    return {p.stride, p.vocab, c.chunk, c.chunks, p.temperature, p.top_k, p.top_p, p.min_p, p.u, p.tokens, p.probs};
}

template <typename T, typename Source> static hipError_t launch_rows(const SampleArgs& p, hipStream_t stream)
{
    hipLaunchKernelGGL((sample_row_kernel<T, Source>), dim3((unsigned)p.rows), dim3(Source::THREADS), 0, stream,
                       (const T*)p.logits, settings_of(p, {}));
    return hipGetLastError();
}

template <typename T, typename Source> static hipError_t launch_chunks(const SampleArgs& p, const Cut& c, hipStream_t stream)
{
    const Settings a = settings_of(p, c);
    Parts x;
    lay_out(p.rows, c, (char*)p.ws, x);
    const dim3 grid((unsigned)(p.rows * c.chunks)), block(Source::THREADS);
    const T* l = (const T*)p.logits;
    hipError_t e = hipSuccess;
    auto next = [&](auto kernel, dim3 g, dim3 b) {
        if (e == hipSuccess) {
            hipLaunchKernelGGL(kernel, g, b, 0, stream, l, a, x);
            e = hipGetLastError();
        }
    };
    next(sample_max_kernel<T, Source>, grid, block);
    next(sample_hist_kernel<T, Source>, grid, block);
    next(sample_gather_kernel<T, Source>, grid, block);
    next(sample_choose_kernel<T>, dim3((unsigned)p.rows), dim3(1024));
    if (p.probs)
        next(sample_probs_kernel<T, Source>, grid, block);
    return e;
}

template <typename T> static hipError_t launch_T(const SampleArgs& p, hipStream_t stream)
{
    if (p.rows == 0)
        return hipSuccess;
    const Cut c = cut_of(p.rows, p.vocab);
    if (c.chunks > 0) {
        if (c.chunk == 1024 * 16) return launch_chunks<T, Held<T, 1024, 16>>(p, c, stream);
        return launch_chunks<T, Held<T, 1024, 32>>(p, c, stream);
    }
    if (p.vocab <= 256 * 8) return launch_rows<T, Held<T, 256, 8>>(p, stream);
    if (p.vocab <= 256 * 32) return launch_rows<T, Held<T, 256, 32>>(p, stream);
    // More rows than one workgroup on each compute unit: two smaller ones there overlap each other's waits.  us, with 1024
    // and with 512 lanes: 320 of 50,001 with distributions 89 and 81, 2000 of 128,000 in bf16 466 and 402, 1000 of 9000 48
    // and 30, 4000 of 32,000 in bf16 271 and 222; 260 of 50,001 45 and 48, 512 of 32,000 42 and 43.
    if (p.rows > (p.vocab > 1024 * 16 && p.vocab <= 1024 * 32 ? 512 : 288))
        return launch_rows<T, Streamed<T, 512>>(p, stream);
    if (p.vocab <= 1024 * 16) return launch_rows<T, Held<T, 1024, 16>>(p, stream);
    if (p.vocab <= 1024 * 32) return launch_rows<T, Held<T, 1024, 32>>(p, stream);
    return launch_rows<T, Streamed<T, 1024>>(p, stream);
}

hipError_t launch_sample(const SampleArgs& p, hipStream_t stream)
{
    return p.bf16 ? launch_T<uint16_t>(p, stream) : launch_T<float>(p, stream);
}

}  // namespace prism
