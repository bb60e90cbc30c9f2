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
// is read once but for the K - 1 rows in front of each run.
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

    // `n` elements at p (VE but in a row's last group); zeros behind them.
    static __device__ __forceinline__ Raw load(const T* p, int n)
    {
        Raw r;
        if (n >= VE) {
            const Access a = *reinterpret_cast<const Access*>(p);
#pragma unroll
            for (int i = 0; i < D; ++i)
                r.d[i] = a[i];
        } else {
            T e[VE];
#pragma unroll
            for (int i = 0; i < VE; ++i)
                e[i] = i < n ? p[i] : T(0);
            r = __builtin_bit_cast(Raw, e);
        }
        return r;
    }
    static __device__ __forceinline__ void store(T* p, int n, const Raw& r)
    {
        if (n >= VE) {
            Access a;
#pragma unroll
            for (int i = 0; i < D; ++i)
                a[i] = r.d[i];
            *reinterpret_cast<Access*>(p) = a;
        } else {
            T e[VE];
            __builtin_memcpy(e, &r, sizeof r);
#pragma unroll
            for (int i = 0; i < VE; ++i)
                if (i < n)
                    p[i] = e[i];
        }
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
template <typename T, int K, int VE>
__device__ __forceinline__ void load_window(const T* x, int64_t ldx, const T* hist, const Cursor& at, int t, int c0,
                                            int C, int n, float (&win)[K][VE])
{
    typedef Group<T, VE> G;
#pragma unroll
    for (int m = 0; m < K - 1; ++m) {
        const int row = t - (K - 1) + m;
#pragma unroll
        for (int e = 0; e < VE; ++e)
            win[m][e] = 0.f;
        if (row >= at.start && row >= 0)
            G::unpack(G::load(x + row * ldx + c0, n), win[m]);
        else if (hist)
            G::unpack(G::load(hist + ((int64_t)at.n * (K - 1) + (K - 1) + (row - at.start)) * C + c0, n), win[m]);
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

template <int K, int VE> __device__ __forceinline__ void shift(float (&win)[K][VE])
{
#pragma unroll
    for (int m = 0; m + 1 < K; ++m)
#pragma unroll
        for (int e = 0; e < VE; ++e)
            win[m][e] = win[m + 1][e];
}

// A workgroup is LV lanes of channel groups by 256 / LV runs of tokens.
struct Where {
    int c0, n, group, groups, chunk, block, blocks;
    __device__ Where(int C, int VE, int lv_bits, int chunks)
    {
        const int lv = 1 << lv_bits;
        chunk = blockIdx.x % chunks;
        block = blockIdx.x / chunks;
        blocks = gridDim.x / chunks;
        group = threadIdx.x >> lv_bits;
        groups = kThreads >> lv_bits;
        c0 = (chunk * lv + (threadIdx.x & (lv - 1))) * VE;
        n = C - c0 < VE ? C - c0 : VE;
    }
};

}  // namespace

template <typename T, int K, int VE, bool SILU>
__global__ __launch_bounds__(kThreads) void short_conv_kernel(
    const T* __restrict__ x, int64_t ldx, const T* __restrict__ w, const T* __restrict__ bias,
    const T* __restrict__ hist, const int32_t* __restrict__ cu, int n_seqs, int tokens, int C, int lv_bits, int chunks,
    int run, T* __restrict__ y)
{
    typedef Group<T, VE> G;
    const Where me(C, VE, lv_bits, chunks);
    const int64_t first = ((int64_t)me.block * me.groups + me.group) * run;
    if (me.n <= 0 || first >= tokens)
        return;
    const int t0 = (int)first, t1 = tokens - t0 < run ? tokens : t0 + run;
    Cursor at;
    at.find(cu, n_seqs, t0, 0);
    if (at.n >= n_seqs)
        return;                                              // rows behind the last sequence are left alone
    float wv[K][VE], bv[VE], win[K][VE], s[VE];
    load_taps<T, K, VE>(w, bias, me.c0, me.n, wv, bv);
    load_window<T, K, VE>(x, ldx, hist, at, t0, me.c0, C, me.n, win);
    for (int tb = t0; tb < t1; tb += kBatch) {
        typename G::Raw raw[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            raw[i] = G::load(x + (int64_t)(tb + i < t1 ? tb + i : t1 - 1) * ldx + me.c0, me.n);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int t = tb + i;
            if (t >= t1)
                return;
            if (t >= at.end) {
                at.find(cu, n_seqs, t, at.n + 1);
                if (at.n >= n_seqs)
                    return;
                load_window<T, K, VE>(x, ldx, hist, at, t, me.c0, C, me.n, win);
            }
            G::unpack(raw[i], win[K - 1]);
            convolve<K, VE>(wv, bv, win, s);
            if (SILU) {
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    float slope;
                    s[e] = gate_act<T, 0>(s[e], slope);
                }
            }
            G::store(y + (int64_t)t * C + me.c0, me.n, G::pack(s));
            shift<K, VE>(win);
        }
    }
}

// The histories to carry on: the last K - 1 rows of [history; sequence].  A lane reads all of its
// channels before it writes any: hist_out may be hist.
template <typename T, int K, int VE>
__global__ __launch_bounds__(kThreads) void short_conv_hist_kernel(const T* x, int64_t ldx, const T* hist,
                                                                   const int32_t* cu, int n_seqs, int C, int groups,
                                                                   T* hist_out)
{
    typedef Group<T, VE> G;
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t n = id / groups;
    if (n >= n_seqs)
        return;
    const int c0 = (int)(id % groups) * VE, cn = C - c0 < VE ? C - c0 : VE;
    const int start = cu[n], len = cu[n + 1] - start;
    typename G::Raw raw[K - 1];
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

// One token a sequence.  hist_out may be hist, as above.
template <typename T, int K, int VE, bool SILU>
__global__ __launch_bounds__(kThreads) void short_conv_step_kernel(const T* __restrict__ x, int64_t ldx,
                                                                   const T* __restrict__ w, const T* __restrict__ bias,
                                                                   const T* hist, int n_seqs, int C, int groups,
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
    if (SILU) {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            float slope;
            s[e] = gate_act<T, 0>(s[e], slope);
        }
    }
    G::store(y + n * C + c0, cn, G::pack(s));
#pragma unroll
    for (int m = 0; m + 1 < K; ++m)
        G::store(hist_out + (n * (K - 1) + m) * C + c0, cn, raw[m + 1]);
}

// dx, and the workgroup's part of dw and dbias: part [block][C * K | C].
template <typename T, int K, int VE, bool SILU>
__global__ __launch_bounds__(kThreads) void short_conv_bwd_kernel(
    const T* __restrict__ x, int64_t ldx, const T* __restrict__ w, const T* __restrict__ bias,
    const T* __restrict__ hist, const int32_t* __restrict__ cu, const T* __restrict__ dy, int n_seqs, int tokens, int C,
    int lv_bits, int chunks, int run, T* __restrict__ dx, float* __restrict__ part)
{
    typedef Group<T, VE> G;
    extern __shared__ float buf[];                           // [groups][lv][VE]
    const Where me(C, VE, lv_bits, chunks);
    const int total = cu[n_seqs];
    float acc[K + 1][VE];
#pragma unroll
    for (int m = 0; m <= K; ++m)
#pragma unroll
        for (int e = 0; e < VE; ++e)
            acc[m][e] = 0.f;
    float wv[K][VE], bv[VE];
    load_taps<T, K, VE>(w, bias, me.c0, me.n < 0 ? 0 : me.n, wv, bv);
    const int64_t runs = ((int64_t)tokens + run - 1) / run;
    if (me.n > 0)
        for (int64_t r = (int64_t)me.block * me.groups + me.group; r < runs; r += (int64_t)me.blocks * me.groups) {
            const int t0 = (int)(r * run), t1 = tokens - t0 < run ? tokens : t0 + run;
            Cursor at, out;                                  // of the row whose ds is formed, and of the one whose dx is
            at.find(cu, n_seqs, t0, 0);
            out = at;
            float win[K][VE], dsw[K][VE];
            if (at.n < n_seqs)
                load_window<T, K, VE>(x, ldx, hist, at, t0, me.c0, C, me.n, win);
            const int last = t1 - 1 + (K - 1);               // the last row whose ds reaches this run's dx
            for (int tb = t0; tb <= last; tb += kBatch) {
                typename G::Raw xr[kBatch], dr[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int64_t row = tb + i < tokens ? tb + i : tokens - 1;
                    xr[i] = G::load(x + row * ldx + me.c0, me.n);
                    dr[i] = G::load(dy + row * C + me.c0, me.n);
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int t = tb + i, o = t - (K - 1);
                    if (t > last)
                        break;
                    float ds[VE];
#pragma unroll
                    for (int e = 0; e < VE; ++e)
                        ds[e] = 0.f;
                    if (t < total && t < tokens) {
                        if (t >= at.end) {
                            at.find(cu, n_seqs, t, at.n + 1);
                            load_window<T, K, VE>(x, ldx, hist, at, t, me.c0, C, me.n, win);
                        }
                        float s[VE];
                        G::unpack(xr[i], win[K - 1]);
                        G::unpack(dr[i], ds);
                        if (SILU) {
                            convolve<K, VE>(wv, bv, win, s);
#pragma unroll
                            for (int e = 0; e < VE; ++e) {
                                float slope;
                                gate_act<T, 0>(s[e], slope);
                                ds[e] *= slope;
                            }
                        }
                        if (t < t1) {
#pragma unroll
                            for (int e = 0; e < VE; ++e) {
#pragma unroll
                                for (int m = 0; m < K; ++m)
                                    acc[m][e] = __builtin_fmaf(ds[e], win[m][e], acc[m][e]);
                                acc[K][e] += ds[e];
                            }
                        }
                        shift<K, VE>(win);
                    }
#pragma unroll
                    for (int e = 0; e < VE; ++e)
                        dsw[K - 1][e] = ds[e];
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
                        G::store(dx + (int64_t)o * C + me.c0, me.n, G::pack(d));
                    }
                    shift<K, VE>(dsw);
                }
            }
        }
    // the groups' sums, added in their order; a row of the partials is [C][K], then [C]
    const int lv = 1 << lv_bits, cols = lv * VE, base = me.chunk * cols;
    float* row = part + (int64_t)me.block * C * (K + 1);
#pragma unroll
    for (int m = 0; m <= K; ++m) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < VE; ++e)
            buf[me.group * cols + (threadIdx.x & (lv - 1)) * VE + e] = acc[m][e];
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += kThreads) {
            float t = 0.f;
            for (int g = 0; g < me.groups; ++g)
                t += buf[g * cols + c];
            if (base + c < C)
                row[m < K ? (int64_t)(base + c) * K + m : (int64_t)C * K + base + c] = t;
        }
    }
}

// dhist from the sequence's first K - 1 rows.
template <typename T, int K, int VE, bool SILU>
__global__ __launch_bounds__(kThreads) void short_conv_dhist_kernel(
    const T* __restrict__ x, int64_t ldx, const T* __restrict__ w, const T* __restrict__ bias,
    const T* __restrict__ hist, const int32_t* __restrict__ cu, const T* __restrict__ dy, int n_seqs, int C, int groups,
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
            if (SILU) {
                convolve<K, VE>(wv, bv, win, s);
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    float slope;
                    gate_act<T, 0>(s[e], slope);
                    ds[e] *= slope;
                }
            }
            shift<K, VE>(win);
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

// Elements of channels a lane holds: 16 bytes, 8 beyond 4 taps.
int lane_channels(bool bf16, int taps) { return (bf16 ? 8 : 4) / (taps > 4 ? 2 : 1); }

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
    Plan(bool bf16, int channels, int taps)
    {
        ve = lane_channels(bf16, taps);
        groups = (channels + ve - 1) / ve;
        lv_bits = lane_bits(groups);
        chunks = (groups + (1 << lv_bits) - 1) >> lv_bits;
        per_block = kThreads >> lv_bits;
    }
};

constexpr int kRun = 32, kBwdRun = 64;

template <typename T, bool SILU, typename Fn> hipError_t with_taps(int taps, Fn&& fn)
{
    constexpr int VE = 16 / (int)sizeof(T);
    switch (taps) {
    case 1: return fn(std::integral_constant<int, 1>{}, std::integral_constant<int, VE>{});
    case 2: return fn(std::integral_constant<int, 2>{}, std::integral_constant<int, VE>{});
    case 3: return fn(std::integral_constant<int, 3>{}, std::integral_constant<int, VE>{});
    case 4: return fn(std::integral_constant<int, 4>{}, std::integral_constant<int, VE>{});
    case 5: return fn(std::integral_constant<int, 5>{}, std::integral_constant<int, VE / 2>{});
    case 6: return fn(std::integral_constant<int, 6>{}, std::integral_constant<int, VE / 2>{});
    case 7: return fn(std::integral_constant<int, 7>{}, std::integral_constant<int, VE / 2>{});
    case 8: return fn(std::integral_constant<int, 8>{}, std::integral_constant<int, VE / 2>{});
    }
    return hipErrorInvalidValue;
}

unsigned blocks_of(int64_t items) { return (unsigned)((items + kThreads - 1) / kThreads); }

template <typename T, bool SILU> hipError_t fwd(const ShortConvArgs& p, hipStream_t stream)
{
    return with_taps<T, SILU>(p.taps, [&](auto taps, auto ve) -> hipError_t {
        constexpr int K = decltype(taps)::value, VE = decltype(ve)::value;
        const Plan plan(p.bf16, p.channels, K);
        if (p.total_tokens > 0) {
            const int64_t runs = ((int64_t)p.total_tokens + kRun - 1) / kRun;
            const int64_t nb = (runs + plan.per_block - 1) / plan.per_block;
            hipLaunchKernelGGL((short_conv_kernel<T, K, VE, SILU>), dim3((unsigned)(nb * plan.chunks)), dim3(kThreads),
                               0, stream, (const T*)p.x, p.x_stride, (const T*)p.w, (const T*)p.bias, (const T*)p.hist,
                               p.cu_seqlens, p.n_seqs, p.total_tokens, p.channels, plan.lv_bits, plan.chunks, kRun,
                               (T*)p.y);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess)
                return e;
        }
        if constexpr (K > 1)
            if (p.hist_out) {
                hipLaunchKernelGGL((short_conv_hist_kernel<T, K, VE>), dim3(blocks_of((int64_t)p.n_seqs * plan.groups)),
                                   dim3(kThreads), 0, stream, (const T*)p.x, p.x_stride, (const T*)p.hist, p.cu_seqlens,
                                   p.n_seqs, p.channels, plan.groups, (T*)p.hist_out);
                return hipGetLastError();
            }
        return hipSuccess;
    });
}

template <typename T, bool SILU> hipError_t step(const ShortConvArgs& p, hipStream_t stream)
{
    return with_taps<T, SILU>(p.taps, [&](auto taps, auto ve) -> hipError_t {
        constexpr int K = decltype(taps)::value, VE = decltype(ve)::value;
        const Plan plan(p.bf16, p.channels, K);
        hipLaunchKernelGGL((short_conv_step_kernel<T, K, VE, SILU>), dim3(blocks_of((int64_t)p.n_seqs * plan.groups)),
                           dim3(kThreads), 0, stream, (const T*)p.x, p.x_stride, (const T*)p.w, (const T*)p.bias,
                           (const T*)p.hist, p.n_seqs, p.channels, plan.groups, (T*)p.y, (T*)p.hist_out);
        return hipGetLastError();
    });
}

template <typename T, bool SILU> hipError_t bwd(const ShortConvArgs& p, hipStream_t stream)
{
    return with_taps<T, SILU>(p.taps, [&](auto taps, auto ve) -> hipError_t {
        constexpr int K = decltype(taps)::value, VE = decltype(ve)::value;
        const Plan plan(p.bf16, p.channels, K);
        const int nb = short_conv_bwd_blocks(p.total_tokens, p.channels, p.bf16, K);
        hipLaunchKernelGGL((short_conv_bwd_kernel<T, K, VE, SILU>), dim3((unsigned)nb * plan.chunks), dim3(kThreads),
                           kThreads * VE * sizeof(float), stream, (const T*)p.x, p.x_stride, (const T*)p.w,
                           (const T*)p.bias, (const T*)p.hist, p.cu_seqlens, (const T*)p.dy, p.n_seqs, p.total_tokens,
                           p.channels, plan.lv_bits, plan.chunks, kBwdRun, (T*)p.dx, p.ws);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        e = rows::launch_sum_partials(p.ws, nb, p.channels * (K + 1), p.channels * K, p.dw, p.dbias, stream);
        if (e != hipSuccess)
            return e;
        if constexpr (K > 1)
            if (p.dhist) {
                hipLaunchKernelGGL((short_conv_dhist_kernel<T, K, VE, SILU>),
                                   dim3(blocks_of((int64_t)p.n_seqs * plan.groups)), dim3(kThreads), 0, stream,
                                   (const T*)p.x, p.x_stride, (const T*)p.w, (const T*)p.bias, (const T*)p.hist,
                                   p.cu_seqlens, (const T*)p.dy, p.n_seqs, p.channels, plan.groups, (T*)p.dhist);
                return hipGetLastError();
            }
        return hipSuccess;
    });
}

}  // namespace

int64_t short_conv_blocks(int total_tokens, int n_seqs, int channels, bool bf16, int taps)
{
    const Plan plan(bf16, channels, taps);
    const int64_t runs = ((int64_t)total_tokens + kRun - 1) / kRun;
    const int64_t walk = (runs + plan.per_block - 1) / plan.per_block * plan.chunks;
    const int64_t hist = ((int64_t)n_seqs * plan.groups + kThreads - 1) / kThreads;
    return walk > hist ? walk : hist;
}

int short_conv_bwd_blocks(int total_tokens, int channels, bool bf16, int taps)
{
    const Plan plan(bf16, channels, taps);
    const int64_t runs = ((int64_t)total_tokens + kBwdRun - 1) / kBwdRun;
    const int64_t want = (runs + plan.per_block - 1) / plan.per_block;
    const int64_t cap = plan.chunks < kConvBwdBlocks ? kConvBwdBlocks / plan.chunks : 1;
    return (int)(want < 1 ? 1 : want < cap ? want : cap);
}

hipError_t launch_short_conv(const ShortConvArgs& p, hipStream_t stream)
{
    if (p.bf16)
        return p.silu ? fwd<uint16_t, true>(p, stream) : fwd<uint16_t, false>(p, stream);
    return p.silu ? fwd<float, true>(p, stream) : fwd<float, false>(p, stream);
}

hipError_t launch_short_conv_step(const ShortConvArgs& p, hipStream_t stream)
{
    if (p.bf16)
        return p.silu ? step<uint16_t, true>(p, stream) : step<uint16_t, false>(p, stream);
    return p.silu ? step<float, true>(p, stream) : step<float, false>(p, stream);
}

hipError_t launch_short_conv_bwd(const ShortConvArgs& p, hipStream_t stream)
{
    if (p.bf16)
        return p.silu ? bwd<uint16_t, true>(p, stream) : bwd<uint16_t, false>(p, stream);
    return p.silu ? bwd<float, true>(p, stream) : bwd<float, false>(p, stream);
}

}  // namespace prism
