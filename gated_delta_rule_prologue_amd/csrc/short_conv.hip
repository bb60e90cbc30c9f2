// short_conv.hip -- causal depthwise convolution over packed sequences, in front of the
// memory-writing operator: with K taps w[c][m], tap K - 1 on the token itself,
//   s_t = bias + sum_m w[m] x[t - K + 1 + m],   y_t = act(s_t)   (per channel),
// rows in front of a sequence being its history (or zero), act = silu or none.
// Gradients: ds = dy act'(s),
//   dx_t = sum_m w[m] ds[t + K - 1 - m]   (rows of the same sequence),
//   dw[m] = sum_t ds_t x[t - K + 1 + m],   dbias = sum_t ds_t,
//   dhist[m] = sum_{p <= m} w[m - p] ds_p   (the sequence's first rows p).
//
// Bound by HBM: 2 streams forward, 3 backward, 2 K + 6 to 6 K + 14 operations an element.  A
// lane owns 16 bytes of channels (8 beyond 4 taps, whose windows would not fit the
// registers) and walks a run of tokens with the last K - 1 rows in registers, so every row
// is read once but for the K - 1 rows in front of each run.  Batches of rows that lie in one
// sequence for the whole wavefront run without a look at the offsets, the next batch's loads in
// flight; the others, at a sequence's ends, row by row.  16,384 x 2304: bf16 37 us forward and 62 backward (151 and
// 227 MB), fp32 65 and 102 (302 and 453 MB); times here are of graphs over four sets of inputs.
#include <type_traits>

#include "activation.h"
#include "common.h"
#include "kernels.h"
#include "norm_rows.h"

namespace prism {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;                                    // rows in flight per lane

// VE elements of channels at any element's address.
template <typename T, int VE> struct Group {
    static constexpr int D = VE * (int)sizeof(T) / 4;        // dwords
    typedef uint32_t Access __attribute__((ext_vector_type(D), aligned(2)));
    struct Raw { uint32_t d[D]; };

    static __device__ __forceinline__ Raw load(const T* p)
    {
        const Access a = *reinterpret_cast<const Access*>(p);
        Raw r;
#pragma unroll
        for (int i = 0; i < D; ++i)
            r.d[i] = a[i];
        return r;
    }
    static __device__ __forceinline__ void store(T* p, const Raw& r)
    {
        Access a;
#pragma unroll
        for (int i = 0; i < D; ++i)
            a[i] = r.d[i];
        *reinterpret_cast<Access*>(p) = a;
    }
    // The first `n` elements at p; zeros behind them.
    static __device__ __forceinline__ Raw load(const T* p, int n)
    {
        if (n >= VE)
            return load(p);
        T e[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i)
            e[i] = i < n ? p[i] : T(0);
        return __builtin_bit_cast(Raw, e);
    }
    static __device__ __forceinline__ void store(T* p, int n, const Raw& r)
    {
        if (n >= VE)
            return store(p, r);
        T e[VE];
        __builtin_memcpy(e, &r, sizeof r);
#pragma unroll
        for (int i = 0; i < VE; ++i)
            if (i < n)
                p[i] = e[i];
    }
    template <bool FEW> static __device__ __forceinline__ Raw load_if(const T* p, int n)
    {
        if constexpr (FEW)
            return load(p, n);
        else
            return load(p);
    }
    template <bool FEW> static __device__ __forceinline__ void store_if(T* p, int n, const Raw& r)
    {
        if constexpr (FEW)
            store(p, n, r);
        else
            store(p, r);
    }
    static __device__ __forceinline__ void unpack(const Raw& r, float* out)
    {
#pragma unroll
        for (int i = 0; i < D; ++i) {
            if constexpr (sizeof(T) == 2) {
                out[2 * i] = __uint_as_float(r.d[i] << 16);
                out[2 * i + 1] = __uint_as_float(r.d[i] & 0xffff0000u);
            } else {
                out[i] = __uint_as_float(r.d[i]);
            }
        }
    }
    static __device__ __forceinline__ Raw pack(const float* in)
    {
        Raw r;
#pragma unroll
        for (int i = 0; i < D; ++i) {
            if constexpr (sizeof(T) == 2)
                r.d[i] = pack_bf16x2(in[2 * i], in[2 * i + 1]);
            else
                r.d[i] = __float_as_uint(in[i]);
        }
        return r;
    }
};

// What a walk over tokens is compiled for: its activation, or rows shorter than a lane's vector (kFew),
// which are read element by element and whose activation is looked at as they go.
enum Mode { kPlain, kSilu, kFew };
template <Mode MODE> __device__ __forceinline__ bool with_silu(bool silu) { return MODE == kFew ? silu : MODE == kSilu; }

// The taps of a lane's channels, w[c][m] with m running fastest.
template <typename T, int K, int VE>
__device__ __forceinline__ void load_taps(const T* w, const T* bias, int c0, int n, float (&wv)[K][VE], float (&bv)[VE])
{
    typedef Group<T, VE> G;
    float flat[K * VE];
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int left = n * K - i * VE;
        G::unpack(G::load(w + (int64_t)c0 * K + i * VE, left < 0 ? 0 : left), flat + i * VE);
    }
#pragma unroll
    for (int m = 0; m < K; ++m)
#pragma unroll
        for (int e = 0; e < VE; ++e)
            wv[m][e] = flat[e * K + m];
#pragma unroll
    for (int e = 0; e < VE; ++e)
        bv[e] = 0.f;
    if (bias)
        G::unpack(G::load(bias + c0, n), bv);
}

// The sequence that holds a token, and where it begins and ends.
struct Cursor {
    int n, start, end;

    // The last sequence that begins at or before t (none is empty among those that hold t);
    // n == n_seqs for a token behind the last sequence.
    __device__ __forceinline__ void find(const int32_t* cu, int n_seqs, int t, int from)
    {
        int lo = from, hi = n_seqs;                          // cu[lo] <= t, the answer is in lo..hi
        while (lo < hi) {
            const int mid = lo + (hi - lo + 1) / 2;
            if (cu[mid] <= t)
                lo = mid;
            else
                hi = mid - 1;
        }
        n = lo;
        start = cu[n];
        end = n < n_seqs ? cu[n + 1] : INT32_MAX;
    }
};

// The K - 1 rows in front of token t: the sequence's own, then its history's last.
template <typename T, int K, int VE, bool FEW = true, int N>
__device__ __forceinline__ void load_window(const T* x, int64_t ldx, const T* hist, const Cursor& at, int t, int c0,
                                            int C, int n, float (&win)[N][VE])
{
    typedef Group<T, VE> G;
#pragma unroll
    for (int m = 0; m < K - 1; ++m) {
        const int row = t - (K - 1) + m;
#pragma unroll
        for (int e = 0; e < VE; ++e)
            win[m][e] = 0.f;
        if (row >= at.start && row >= 0)
            G::unpack(G::template load_if<FEW>(x + row * ldx + c0, n), win[m]);
        else if (hist)
            G::unpack(G::template load_if<FEW>(hist + ((int64_t)at.n * (K - 1) + (K - 1) + (row - at.start)) * C + c0, n), win[m]);
    }
}

// s of the row in win[K - 1] and the K - 1 before it.
template <int K, int VE>
__device__ __forceinline__ void convolve(const float (&wv)[K][VE], const float (&bv)[VE], const float (&win)[K][VE],
                                         float (&s)[VE])
{
#pragma unroll
    for (int e = 0; e < VE; ++e) {
        s[e] = bv[e];
#pragma unroll
        for (int m = 0; m < K; ++m)
            s[e] = __builtin_fmaf(wv[m][e], win[m][e], s[e]);
    }
}

// silu and its slope.  bf16's rounding leaves room for the short forms: s = 1 / (1 + e^-z), slope
// s (1 + z (1 - s)), off by |z| 2^-24 of 1 where the gate is open; fp32 takes the forms without the
// difference.
template <typename T> __device__ __forceinline__ float silu(float z)
{
    if constexpr (sizeof(T) == 2)
        return z * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
    float slope;
    return gate_act<T, 0>(z, slope);
}
template <typename T> __device__ __forceinline__ float silu_slope(float z)
{
    if constexpr (sizeof(T) == 2) {
        const float s = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
        return s * __builtin_fmaf(z, 1.f - s, 1.f);
    }
    float slope;
    gate_act<T, 0>(z, slope);
    return slope;
}

// The last K - 1 of K - 1 + by rows become the first.
template <int K, int VE, int N> __device__ __forceinline__ void advance(float (&win)[N][VE], int by)
{
#pragma unroll
    for (int m = 0; m + 1 < K; ++m)
#pragma unroll
        for (int e = 0; e < VE; ++e)
            win[m][e] = win[m + by][e];
}

// The histories to carry on: the last K - 1 rows of [history; sequence].  A lane reads all of its
// channels before it writes any: hist_out may be hist.
template <typename T, int K, int VE>
__device__ __forceinline__ void carry_history(const T* x, int64_t ldx, const T* hist, const int32_t* cu, int n_seqs, int C,
                                              int64_t id, T* hist_out)
{
    typedef Group<T, VE> G;
    const int groups = (C + VE - 1) / VE;
    const int64_t n = id / groups;
    if (n >= n_seqs)
        return;
    const int c0 = (int)(id % groups) * VE, cn = C - c0 < VE ? C - c0 : VE;
    const int start = cu[n], len = cu[n + 1] - start;
    typename G::Raw raw[K];
#pragma unroll
    for (int m = 0; m < K - 1; ++m) {
        const int row = len - (K - 1) + m;
        if (row >= 0)
            raw[m] = G::load(x + ((int64_t)start + row) * ldx + c0, cn);
        else if (hist)
            raw[m] = G::load(hist + (n * (K - 1) + len + m) * C + c0, cn);
        else
            raw[m] = {};
    }
#pragma unroll
    for (int m = 0; m < K - 1; ++m)
        G::store(hist_out + (n * (K - 1) + m) * C + c0, cn, raw[m]);
}

// A workgroup is LV lanes of channel groups by 256 / LV runs of tokens.  Where the channels do not
// fill the last vector it begins that much earlier: its lane forms some channels a second time, and
// stores the same values.
struct Where {
    int c0, n, group, groups, chunk, block;                  // n <= 0: a lane without channels
    __device__ Where(int C, int VE, int lv_bits, int chunks)
    {
        const int lv = 1 << lv_bits;
        chunk = blockIdx.x % chunks;
        block = blockIdx.x / chunks;
        group = threadIdx.x >> lv_bits;
        groups = kThreads >> lv_bits;
        c0 = (chunk * lv + (threadIdx.x & (lv - 1))) * VE;
        n = C - c0 < VE ? C - c0 : VE;
        if (n > 0 && n < VE && C >= VE) {
            c0 = C - VE;
            n = VE;
        }
    }
};

}  // namespace

template <typename T, int K, int VE, Mode MODE>
__global__ __launch_bounds__(kThreads) void short_conv_kernel(
    const T* __restrict__ x, int64_t ldx, const T* __restrict__ w, const T* __restrict__ bias,
    const T* __restrict__ hist, const int32_t* __restrict__ cu, bool act, int n_seqs, int tokens, int C, int lv_bits,
    int chunks, int run, int walks, bool clear, T* __restrict__ y, T* __restrict__ hist_out)
{
    constexpr bool FEW = MODE == kFew;
    typedef Group<T, VE> G;
    if constexpr (K > 1)
        if ((int)blockIdx.x >= walks) {                      // the workgroups behind those that walk
            carry_history<T, K, VE>(x, ldx, hist, cu, n_seqs, C, (int64_t)(blockIdx.x - walks) * kThreads + threadIdx.x,
                                    hist_out);
            return;
        }
    const Where me(C, VE, lv_bits, chunks);
    const int64_t first = ((int64_t)me.block * me.groups + me.group) * run;
    if (me.n <= 0 || first >= tokens)
        return;
    const int t0 = (int)first, t1 = tokens - t0 < run ? tokens : t0 + run;
    const T* col = x + me.c0;
    T* out = y + me.c0;
    float wv[K][VE], bv[VE], win[K - 1 + kBatch][VE];        // the rows before a batch, then its own
    auto one = [&](int at, int64_t t) {                      // y of row t, which is win[at]
        float s[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            s[e] = bv[e];
#pragma unroll
            for (int m = 0; m < K; ++m)
                s[e] = __builtin_fmaf(wv[m][e], win[at - (K - 1) + m][e], s[e]);
            if (with_silu<MODE>(act))
                s[e] = silu<T>(s[e]);
        }
        G::template store_if<FEW>(out + t * C, me.n, G::pack(s));
    };
    // rows do not wait for the cursor: those in front of the run are on their way while it searches
    typename G::Raw raw[kBatch], past[K];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
        raw[i] = G::template load_if<FEW>(col + (int64_t)(t0 + i < t1 ? t0 + i : t1 - 1) * ldx, me.n);
#pragma unroll
    for (int m = 0; m < K - 1; ++m)
        past[m] = G::template load_if<FEW>(col + (int64_t)(t0 - (K - 1) + m > 0 ? t0 - (K - 1) + m : 0) * ldx, me.n);
    load_taps<T, K, VE>(w, bias, me.c0, me.n, wv, bv);
    Cursor at;
    at.find(cu, n_seqs, t0, 0);
    if (clear) {                                             // rows behind the last sequence, which the walk leaves alone
#pragma unroll 1
        for (int t = t0 > cu[n_seqs] ? t0 : cu[n_seqs]; t < t1; ++t)
            G::template store_if<FEW>(out + (int64_t)t * C, me.n, typename G::Raw{});
    }
    if (at.n >= n_seqs)
        return;
    if (t0 - (K - 1) >= at.start) {
#pragma unroll
        for (int m = 0; m < K - 1; ++m)
            G::unpack(past[m], win[m]);
    } else {
        load_window<T, K, VE, FEW>(x, ldx, hist, at, t0, me.c0, C, me.n, win);
    }
    for (int tb = t0; tb < t1;) {
        const int whole = t1 < at.end ? t1 : at.end;         // batches up to here are rows of one sequence
        bool ok = __all(tb + kBatch <= whole);
        if (ok) {
            if (tb != t0) {
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    raw[i] = G::template load_if<FEW>(col + (int64_t)(tb + i) * ldx, me.n);
            }
            do {
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    G::unpack(raw[i], win[K - 1 + i]);
                ok = __all(tb + 2 * kBatch <= whole);
                if (ok) {
#pragma unroll
                    for (int i = 0; i < kBatch; ++i)
                        raw[i] = G::template load_if<FEW>(col + (int64_t)(tb + kBatch + i) * ldx, me.n);
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    one(K - 1 + i, tb + i);
                advance<K, VE>(win, kBatch);
                tb += kBatch;
            } while (ok);
            continue;
        }
#pragma unroll 1
        for (int end = tb + kBatch; tb < end; ++tb) {
            if (tb >= t1)
                return;
            if (tb >= at.end) {
                at.find(cu, n_seqs, tb, at.n + 1);
                if (at.n >= n_seqs)
                    return;
                load_window<T, K, VE, FEW>(x, ldx, hist, at, tb, me.c0, C, me.n, win);
            }
            G::unpack(G::template load_if<FEW>(col + (int64_t)tb * ldx, me.n), win[K - 1]);
            one(K - 1, tb);
            advance<K, VE>(win, 1);
        }
    }
}

template <typename T, int K, int VE>
__global__ __launch_bounds__(kThreads) void short_conv_hist_kernel(const T* x, int64_t ldx, const T* hist,
                                                                   const int32_t* cu, int n_seqs, int C, T* hist_out)
{
    carry_history<T, K, VE>(x, ldx, hist, cu, n_seqs, C, (int64_t)blockIdx.x * kThreads + threadIdx.x, hist_out);
}

// One token a sequence.  hist_out may be hist, as above.
template <typename T, int K, int VE>
__global__ __launch_bounds__(kThreads) void short_conv_step_kernel(const T* __restrict__ x, int64_t ldx,
                                                                   const T* __restrict__ w, const T* __restrict__ bias,
                                                                   const T* hist, bool silu_on, int n_seqs, int C, int groups,
                                                                   T* __restrict__ y, T* hist_out)
{
    typedef Group<T, VE> G;
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t n = id / groups;
    if (n >= n_seqs)
        return;
    const int c0 = (int)(id % groups) * VE, cn = C - c0 < VE ? C - c0 : VE;
    typename G::Raw raw[K];
#pragma unroll
    for (int m = 0; m + 1 < K; ++m)
        raw[m] = G::load(hist + (n * (K - 1) + m) * C + c0, cn);
    raw[K - 1] = G::load(x + n * ldx + c0, cn);
    float wv[K][VE], bv[VE], win[K][VE], s[VE];
    load_taps<T, K, VE>(w, bias, c0, cn, wv, bv);
#pragma unroll
    for (int m = 0; m < K; ++m)
        G::unpack(raw[m], win[m]);
    convolve<K, VE>(wv, bv, win, s);
    if (silu_on) {
#pragma unroll
        for (int e = 0; e < VE; ++e)
            s[e] = silu<T>(s[e]);
    }
    G::store(y + n * C + c0, cn, G::pack(s));
#pragma unroll
    for (int m = 0; m + 1 < K; ++m)
        G::store(hist_out + (n * (K - 1) + m) * C + c0, cn, raw[m + 1]);
}

// Rows whose terms of dw and dbias a lane adds up in turn, before they join its sums of the stretches before: so the
// rounding errors grow with 256 and a run's 256ths, not with a run.
constexpr int kStretch = 256;

// dx, and the workgroup's part of dw and dbias: part [block][C * K | C].
template <typename T, int K, int VE, Mode MODE>
__global__ __launch_bounds__(kThreads) void short_conv_bwd_kernel(
    const T* __restrict__ x, int64_t ldx, const T* __restrict__ w, const T* __restrict__ bias,
    const T* __restrict__ hist, const int32_t* __restrict__ cu, const T* __restrict__ dy, bool act, bool bias_grad,
    int n_seqs, int tokens, int C, int lv_bits, int chunks, int run, T* __restrict__ dx, float* __restrict__ part)
{
    constexpr bool FEW = MODE == kFew;
    typedef Group<T, VE> G;
    extern __shared__ float buf[];                           // [groups][lv][VE]; before that, in runs beyond a stretch,
                                                             // the lanes' sums [K + 1][VE][kThreads]
    const Where me(C, VE, lv_bits, chunks);
    const int total = cu[n_seqs] < tokens ? cu[n_seqs] : tokens;
    float acc[K + 1][VE], wv[K][VE], bv[VE];
#pragma unroll
    for (int m = 0; m <= K; ++m)
#pragma unroll
        for (int e = 0; e < VE; ++e)
            acc[m][e] = 0.f;
    load_taps<T, K, VE>(w, bias, me.c0, me.n < 0 ? 0 : me.n, wv, bv);
    const T *col = x + me.c0, *dcol = dy + me.c0;
    T* out_col = dx + me.c0;
    float win[K - 1 + kBatch][VE], dsw[K - 1 + kBatch][VE];  // rows of x and ds before a batch, then its own
    // ds of the row in win[at], from its dy in dsw[at]
    auto slope = [&](int at) {
        if (with_silu<MODE>(act)) {
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                float s = bv[e];
#pragma unroll
                for (int m = 0; m < K; ++m)
                    s = __builtin_fmaf(wv[m][e], win[at - (K - 1) + m][e], s);
                dsw[at][e] *= silu_slope<T>(s);
            }
        }
    };
    auto weigh = [&](int at) {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
#pragma unroll
            for (int m = 0; m < K; ++m)
                acc[m][e] = __builtin_fmaf(dsw[at][e], win[at - (K - 1) + m][e], acc[m][e]);
        }
    };
    const int64_t first = ((int64_t)me.block * me.groups + me.group) * run;
    if (me.n > 0 && first < tokens) {
        const int t0 = (int)first, t1 = tokens - t0 < run ? tokens : t0 + run;
        const int last = t1 - 1 + (K - 1);               // the last row whose ds reaches this run's dx
        Cursor at, out;                                  // of the row whose ds is formed, and of the one whose dx is
        at.find(cu, n_seqs, t0, 0);
        out = at;
        if (at.n < n_seqs)
            load_window<T, K, VE, FEW>(x, ldx, hist, at, t0, me.c0, C, me.n, win);
        // All lanes of a wavefront are as far in their runs, `done` rows.  A batch is plain where its
        // rows, and those before them whose dx it completes, are of one sequence.
        const int whole = at.n < n_seqs ? (at.end < total ? at.end : total) : 0;
        int until = whole - t0, from = 0;                // in rows of the run
        for (int done = 0; done <= run - 1 + (K - 1);) {
            if (done > 0 && done % kStretch == 0)
#pragma unroll
                for (int m = 0; m <= K; ++m)
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        float* sum = buf + (m * VE + e) * kThreads + threadIdx.x;
                        *sum = done == kStretch ? acc[m][e] : *sum + acc[m][e];
                        acc[m][e] = 0.f;
                    }
            auto plain = [&](int d) { return __all(d + kBatch <= until && (d == 0 || d - (K - 1) >= from)); };
            if (plain(done)) {
                typename G::Raw xr[kBatch], dr[kBatch];
                const T *xp = col + (int64_t)(t0 + done) * ldx, *dp = dcol + (int64_t)(t0 + done) * C;
                T* op = out_col + ((int64_t)(t0 + done) - (K - 1)) * C;
                auto fetch = [&]() {
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        xr[i] = G::template load_if<FEW>(xp + i * ldx, me.n);
                        dr[i] = G::template load_if<FEW>(dp + (int64_t)i * C, me.n);
                    }
                    xp += kBatch * ldx;
                    dp += (int64_t)kBatch * C;
                };
                fetch();
                bool more;
                do {
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        G::unpack(xr[i], win[K - 1 + i]);
                        G::unpack(dr[i], dsw[K - 1 + i]);
                    }
                    more = done + kBatch <= run - 1 + (K - 1) && (done + kBatch) % kStretch != 0 && plain(done + kBatch);
                    if (more)
                        fetch();
#pragma unroll
                    for (int i = 0; i < kBatch; ++i)
                        slope(K - 1 + i);
                    if (done < run) {                    // run is a multiple of kBatch; the rows behind it are another's
#pragma unroll
                        for (int i = 0; i < kBatch; ++i)
                            weigh(K - 1 + i);
                        if (bias_grad)
#pragma unroll
                            for (int i = 0; i < kBatch; ++i)
#pragma unroll
                                for (int e = 0; e < VE; ++e)
                                    acc[K][e] += dsw[K - 1 + i][e];
                    }
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        if (done + i < K - 1 || done + i >= run + K - 1)
                            continue;
                        float d[VE];
#pragma unroll
                        for (int e = 0; e < VE; ++e) {
                            d[e] = wv[K - 1][e] * dsw[i][e];
#pragma unroll
                            for (int j = 1; j < K; ++j)
                                d[e] = __builtin_fmaf(wv[K - 1 - j][e], dsw[i + j][e], d[e]);
                        }
                        G::template store_if<FEW>(op + (int64_t)i * C, me.n, G::pack(d));
                    }
                    advance<K, VE>(win, kBatch);
                    advance<K, VE>(dsw, kBatch);
                    op += (int64_t)kBatch * C;
                    done += kBatch;
                } while (more);
                continue;
            }
#pragma unroll 1
            for (int i = 0; i < kBatch; ++i, ++done) {
                const int t = t0 + done, o = t - (K - 1);
                if (t > last)
                    continue;
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    dsw[K - 1][e] = 0.f;
                if (t < total) {
                    if (t >= at.end) {
                        at.find(cu, n_seqs, t, at.n + 1);
                        load_window<T, K, VE, FEW>(x, ldx, hist, at, t, me.c0, C, me.n, win);
                        from = at.start - t0;
                        until = (at.end < total ? at.end : total) - t0;
                    }
                    G::unpack(G::template load_if<FEW>(col + (int64_t)t * ldx, me.n), win[K - 1]);
                    G::unpack(G::template load_if<FEW>(dcol + (int64_t)t * C, me.n), dsw[K - 1]);
                    slope(K - 1);
                    if (t < t1) {
                        weigh(K - 1);
#pragma unroll
                        for (int e = 0; e < VE; ++e)
                            acc[K][e] += dsw[K - 1][e];
                    }
                    advance<K, VE>(win, 1);
                }
                if (o >= t0) {
                    if (o >= out.end)
                        out.find(cu, n_seqs, o, out.n + 1);
                    float d[VE];
                    const int reach = out.n < n_seqs ? out.end - o : 0;      // rows of the sequence from o on
#pragma unroll
                    for (int e = 0; e < VE; ++e)
                        d[e] = 0.f;
#pragma unroll
                    for (int j = 0; j < K; ++j)
                        if (j < reach) {
#pragma unroll
                            for (int e = 0; e < VE; ++e)
                                d[e] = __builtin_fmaf(wv[K - 1 - j][e], dsw[j][e], d[e]);
                        }
                    G::template store_if<FEW>(out_col + (int64_t)o * C, me.n, G::pack(d));
                }
                advance<K, VE>(dsw, 1);
            }
        }
        if (run - 1 + (K - 1) >= kStretch)
#pragma unroll
            for (int m = 0; m <= K; ++m)
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    acc[m][e] += buf[(m * VE + e) * kThreads + threadIdx.x];
    }
    // the groups' sums, added in their order; a row of the partials is [C][K], then [C]
    const int lv = 1 << lv_bits, cols = lv * VE, base = me.chunk * cols;
    float* row = part + (int64_t)me.block * C * (K + 1);
#pragma unroll
    for (int m = 0; m <= K; ++m) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < VE; ++e)
            if (me.n > 0 && me.c0 + e >= base)
                buf[me.group * cols + me.c0 + e - base] = acc[m][e];
        __syncthreads();
        for (int c = threadIdx.x; c < cols && base + c < C; c += kThreads) {
            float t = 0.f;
            for (int g = 0; g < me.groups; ++g)
                t += buf[g * cols + c];
            row[m < K ? (int64_t)(base + c) * K + m : (int64_t)C * K + base + c] = t;
        }
    }
}

// dhist from the sequence's first K - 1 rows.
template <typename T, int K, int VE>
__global__ __launch_bounds__(kThreads) void short_conv_dhist_kernel(
    const T* __restrict__ x, int64_t ldx, const T* __restrict__ w, const T* __restrict__ bias,
    const T* __restrict__ hist, const int32_t* __restrict__ cu, const T* __restrict__ dy, bool silu_on, int n_seqs, int C, int groups,
    T* __restrict__ dhist)
{
    typedef Group<T, VE> G;
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t n = id / groups;
    if (n >= n_seqs)
        return;
    const int c0 = (int)(id % groups) * VE, cn = C - c0 < VE ? C - c0 : VE;
    Cursor at;
    at.n = (int)n;
    at.start = cu[n];
    at.end = cu[n + 1];
    const int len = at.end - at.start;
    float wv[K][VE], bv[VE], win[K][VE], s[VE], ds[VE], dh[K][VE];
    load_taps<T, K, VE>(w, bias, c0, cn, wv, bv);
    load_window<T, K, VE>(x, ldx, hist, at, at.start, c0, C, cn, win);
#pragma unroll
    for (int m = 0; m < K; ++m)
#pragma unroll
        for (int e = 0; e < VE; ++e)
            dh[m][e] = 0.f;
#pragma unroll
    for (int p = 0; p < K - 1; ++p)
        if (p < len) {
            const int64_t t = at.start + p;
            G::unpack(G::load(x + t * ldx + c0, cn), win[K - 1]);
            G::unpack(G::load(dy + t * C + c0, cn), ds);
            if (silu_on) {
                convolve<K, VE>(wv, bv, win, s);
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    ds[e] *= silu_slope<T>(s[e]);
            }
            advance<K, VE>(win, 1);
#pragma unroll
            for (int m = p; m < K - 1; ++m)
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    dh[m][e] = __builtin_fmaf(wv[m - p][e], ds[e], dh[m][e]);
        }
#pragma unroll
    for (int m = 0; m < K - 1; ++m)
        G::store(dhist + (n * (K - 1) + m) * C + c0, cn, G::pack(dh[m]));
}

namespace {

// Elements of channels a lane holds: 16 bytes, 8 beyond 4 taps (histories of 111,600 x 1536 in 133 us,
// with 8 bytes 140).
constexpr int lane_channels(int elem_bytes, int taps) { return (taps > 4 ? 8 : 16) / elem_bytes; }
// The backward's: its windows are twice as many and the sums of the weights' gradients join them, so 8
// bytes, 4 beyond 4 taps (16 bytes leave one wavefront a SIMD: 287 instead of 229 us for those
// histories; 4 bytes 235).
constexpr int lane_channels_bwd(int elem_bytes, int taps) { return taps > 4 && elem_bytes == 2 ? 2 : 8 / elem_bytes; }

// Lanes (a power of two, as bits) that a workgroup lays along the channels: 64, or fewer where
// they would leave more lanes idle.
int lane_bits(int groups)
{
    int best = 3, waste = INT32_MAX;
    for (int b = 3; b <= 6; ++b) {
        const int padded = (groups + (1 << b) - 1) >> b << b;
        if (padded - groups <= waste) {
            waste = padded - groups;
            best = b;
        }
    }
    return best;
}

struct Plan {
    int ve, groups, lv_bits, chunks, per_block;              // per_block: runs side by side in a workgroup
    Plan(int channels, int ve_)
    {
        ve = ve_;
        groups = (channels + ve - 1) / ve;
        lv_bits = lane_bits(groups);
        chunks = (groups + (1 << lv_bits) - 1) >> lv_bits;
        per_block = kThreads >> lv_bits;
    }
};

// Tokens of a run: so many that all runs make up one round of `blocks` workgroups, within limits.
int run_of(int tokens, const Plan& plan, int blocks, int least, int most)
{
    const int64_t lanes = (int64_t)(blocks > plan.chunks ? blocks / plan.chunks : 1) * plan.per_block;
    const int64_t run = (((int64_t)tokens + lanes - 1) / lanes + kBatch - 1) / kBatch * kBatch;
    return (int)(run < least ? least : run > most ? most : run);
}
// Forward: short runs spread few tokens over the compute units (512 tokens of 2304: 4.0 us in runs of 4, 6.8 in
// runs of 16); of many the workgroups of several rounds keep to neighbouring rows (histories: runs of 16
// 133 us, of 32 138).
int fwd_run(int tokens, const Plan& plan) { return run_of(tokens, plan, 1536, 4, 16); }
// Backward: two workgroups a compute unit, one run a lane (histories: 230 us; runs of 64 in turn 234, three
// workgroups 248).
int bwd_run(int tokens, const Plan& plan) { return run_of(tokens, plan, kConvBwdBlocks, 16, INT32_MAX / 2); }

template <Mode M> struct ModeTag { static constexpr Mode mode = M; };
template <typename Fn> hipError_t with_mode(bool few, bool silu, Fn&& fn)
{
    return few ? fn(ModeTag<kFew>{}) : silu ? fn(ModeTag<kSilu>{}) : fn(ModeTag<kPlain>{});
}

template <typename Fn> hipError_t with_taps(int taps, Fn&& fn)
{
    switch (taps) {
    case 1: return fn(std::integral_constant<int, 1>{});
    case 2: return fn(std::integral_constant<int, 2>{});
    case 3: return fn(std::integral_constant<int, 3>{});
    case 4: return fn(std::integral_constant<int, 4>{});
    case 5: return fn(std::integral_constant<int, 5>{});
    case 6: return fn(std::integral_constant<int, 6>{});
    case 7: return fn(std::integral_constant<int, 7>{});
    case 8: return fn(std::integral_constant<int, 8>{});
    }
    return hipErrorInvalidValue;
}

unsigned blocks_of(int64_t items) { return (unsigned)((items + kThreads - 1) / kThreads); }

template <typename T> hipError_t fwd(const ShortConvArgs& p, hipStream_t stream)
{
    return with_taps(p.taps, [&](auto taps) -> hipError_t {
        constexpr int K = decltype(taps)::value, VE = lane_channels(sizeof(T), K);
        const Plan plan(p.channels, VE);
        const unsigned carry = K > 1 && p.hist_out ? blocks_of((int64_t)p.n_seqs * plan.groups) : 0;
        const bool apart = p.hist_out != p.hist;             // else the walk reads what the histories overwrite
        const int run = fwd_run(p.total_tokens, plan);
        const int64_t runs = ((int64_t)p.total_tokens + run - 1) / run;
        const unsigned walks = (unsigned)((runs + plan.per_block - 1) / plan.per_block * plan.chunks);
        const unsigned blocks = walks + (apart ? carry : 0);
        hipError_t e = hipSuccess;
        if (blocks > 0)
            e = with_mode(p.channels < VE, p.silu, [&](auto mode) -> hipError_t {
                hipLaunchKernelGGL((short_conv_kernel<T, K, VE, decltype(mode)::mode>), dim3(blocks), dim3(kThreads), 0,
                                   stream, (const T*)p.x, p.x_stride, (const T*)p.w, (const T*)p.bias,
                                   (const T*)p.hist, p.cu_seqlens, p.silu, p.n_seqs, p.total_tokens, p.channels,
                                   plan.lv_bits, plan.chunks, run, (int)walks, p.clear_behind, (T*)p.y, (T*)p.hist_out);
                return hipGetLastError();
            });
        if constexpr (K > 1)
            if (e == hipSuccess && carry > 0 && !apart) {
                hipLaunchKernelGGL((short_conv_hist_kernel<T, K, VE>), dim3(carry), dim3(kThreads), 0, stream,
                                   (const T*)p.x, p.x_stride, (const T*)p.hist, p.cu_seqlens, p.n_seqs, p.channels,
                                   (T*)p.hist_out);
                e = hipGetLastError();
            }
        return e;
    });
}

template <typename T> hipError_t step(const ShortConvArgs& p, hipStream_t stream)
{
    return with_taps(p.taps, [&](auto taps) -> hipError_t {
        constexpr int K = decltype(taps)::value, VE = lane_channels(sizeof(T), K);
        const Plan plan(p.channels, VE);
        hipLaunchKernelGGL((short_conv_step_kernel<T, K, VE>), dim3(blocks_of((int64_t)p.n_seqs * plan.groups)),
                           dim3(kThreads), 0, stream, (const T*)p.x, p.x_stride, (const T*)p.w, (const T*)p.bias,
                           (const T*)p.hist, p.silu, p.n_seqs, p.channels, plan.groups, (T*)p.y, (T*)p.hist_out);
        return hipGetLastError();
    });
}

template <typename T> hipError_t bwd(const ShortConvArgs& p, hipStream_t stream)
{
    return with_taps(p.taps, [&](auto taps) -> hipError_t {
        constexpr int K = decltype(taps)::value, VE = lane_channels_bwd(sizeof(T), K), VH = lane_channels(sizeof(T), K);
        const Plan plan(p.channels, VE);
        const int nb = short_conv_bwd_blocks(p.total_tokens, p.channels, p.bf16, K);
        const int run = bwd_run(p.total_tokens, plan);
        const size_t sums = run - 1 + (K - 1) >= kStretch ? K + 1 : 1;
        hipError_t e = with_mode(p.channels < VE, p.silu, [&](auto mode) -> hipError_t {
            hipLaunchKernelGGL((short_conv_bwd_kernel<T, K, VE, decltype(mode)::mode>), dim3((unsigned)nb * plan.chunks),
                               dim3(kThreads), sums * kThreads * VE * sizeof(float), stream, (const T*)p.x, p.x_stride,
                               (const T*)p.w, (const T*)p.bias, (const T*)p.hist, p.cu_seqlens, (const T*)p.dy, p.silu,
                               p.dbias != nullptr, p.n_seqs, p.total_tokens, p.channels, plan.lv_bits, plan.chunks,
                               run, (T*)p.dx, p.ws);
            return hipGetLastError();
        });
        if (e != hipSuccess)
            return e;
        e = rows::launch_sum_partials(p.ws, nb, p.channels * (K + 1), p.channels * K, p.dw, p.dbias, stream);
        if (e != hipSuccess)
            return e;
        if constexpr (K > 1)
            if (p.dhist) {
                const int groups = (p.channels + VH - 1) / VH;
                hipLaunchKernelGGL((short_conv_dhist_kernel<T, K, VH>),
                                   dim3(blocks_of((int64_t)p.n_seqs * groups)), dim3(kThreads), 0, stream,
                                   (const T*)p.x, p.x_stride, (const T*)p.w, (const T*)p.bias, (const T*)p.hist,
                                   p.cu_seqlens, (const T*)p.dy, p.silu, p.n_seqs, p.channels, groups, (T*)p.dhist);
                return hipGetLastError();
            }
        return hipSuccess;
    });
}

}  // namespace

int64_t short_conv_blocks(int total_tokens, int n_seqs, int channels, bool bf16, int taps)
{
    const Plan plan(channels, lane_channels(bf16 ? 2 : 4, taps));
    const int run = fwd_run(total_tokens, plan);
    const int64_t runs = ((int64_t)total_tokens + run - 1) / run;
    const int64_t walk = (runs + plan.per_block - 1) / plan.per_block * plan.chunks;
    const int64_t hist = ((int64_t)n_seqs * plan.groups + kThreads - 1) / kThreads;
    return walk + hist;
}

int short_conv_bwd_blocks(int total_tokens, int channels, bool bf16, int taps)
{
    const Plan plan(channels, lane_channels_bwd(bf16 ? 2 : 4, taps));
    const int run = bwd_run(total_tokens, plan);
    const int64_t runs = ((int64_t)total_tokens + run - 1) / run;
    const int64_t want = (runs + plan.per_block - 1) / plan.per_block;
    return (int)(want < 1 ? 1 : want);
}

hipError_t launch_short_conv(const ShortConvArgs& p, hipStream_t stream)
{
    return p.bf16 ? fwd<uint16_t>(p, stream) : fwd<float>(p, stream);
}

hipError_t launch_short_conv_step(const ShortConvArgs& p, hipStream_t stream)
{
    return p.bf16 ? step<uint16_t>(p, stream) : step<float>(p, stream);
}

hipError_t launch_short_conv_bwd(const ShortConvArgs& p, hipStream_t stream)
{
    return p.bf16 ? bwd<uint16_t>(p, stream) : bwd<float>(p, stream);
}

}  // namespace prism
