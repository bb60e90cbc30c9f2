// qk_norm.hip -- the queries and keys that enter the memory-writing operator: every head's
// row of d elements is normalised, weighted and rotated by its token's position,
//   xh = x rstd,   rstd = 1 / sqrt(mean(x^2) + eps) (rms), 1 / sqrt(sum(x^2) + eps) (l2) or 1,
//   y = R(position * freqs) (xh w),
// where R turns the pairs of the first `rot` elements: (i, i + rot / 2) in the half layout,
// (2 i, 2 i + 1) in the interleaved one.  Gradients: e = R^T dy,
//   dw = sum e xh,   dx = rstd (e w - xh c sum(e w xh)),   c = 1 / d (rms), 1 (l2), 0 (none).
//
// Angles: the product of an int32 position and an fp32 frequency is exact to 2^-53 in 64
// bits; its whole turns are dropped there, and sine and cosine are taken in 32 bits of what is
// left, so far positions lose nothing.  A workgroup forms the cosines and sines of its tokens
// once, in LDS, for all heads.
//
// Bound by HBM (2 streams forward, 3 backward).  A lane holds pairs of 16-byte vectors of a
// row, the two that rotate with each other in the half layout, so a row needs width / 16
// lanes in bf16 (width / 8 in fp32) and the rotation stays in a lane.  Rows that do not
// fill whole vectors (and rotations that do not fill whole pairs of them) take a wavefront
// and single elements.
#include "common.h"
#include "kernels.h"
#include "norm_rows.h"

namespace prism {

namespace {

constexpr int kThreads = 256;

// The elements of a row that a lane holds: NP pairs of vectors of VE elements.
template <typename T, int VE_, int LANES_, int NP_> struct Shape {
    typedef T elem;
    static constexpr int VE = VE_, LANES = LANES_, NP = NP_;
    static constexpr int GROUPS = kThreads / LANES;
    static constexpr int E = 2 * VE * NP;
};

// Where a pair of vectors lies in the row, and how it turns.
struct Pair {
    int a, b;                                                // first elements; -1: none
    int freq;                                                // first frequency, of a's elements; -1: a does not turn
    int freq_b;                                              // interleaved vectors: of b's elements; -1: none
};

// Pair j of a row.  The half layout's first pairs are vectors that turn with each other; all
// other vectors follow in their order, two a pair.
template <typename S> __device__ __forceinline__ Pair pair_at(int j, int width, int rot, bool interleaved)
{
    constexpr int VE = S::VE;
    Pair p;
    if (!interleaved || VE == 1) {
        const int turning = rot / 2 / VE;
        if (j < turning) {
            p.a = interleaved ? 2 * j : j * VE;
            p.b = interleaved ? 2 * j + 1 : j * VE + rot / 2;
            p.freq = j * VE;
        } else {
            p.a = rot + (j - turning) * 2 * VE;
            p.b = p.a + VE;
            p.freq = -1;
        }
        p.freq_b = -1;
    } else {
        p.a = j * 2 * VE;
        p.b = p.a + VE;
        p.freq = p.a < rot ? p.a / 2 : -1;
        p.freq_b = p.b < rot ? p.b / 2 : -1;
    }
    if (p.a >= width)
        p.a = -1;
    if (p.b >= width)
        p.b = -1;
    return p;
}

template <typename T, int VE> __device__ __forceinline__ void load_vec(const T* p, float* out)
{
    if constexpr (VE == 1) {
        out[0] = to_f32(*p);
    } else {
        const rows::AtElement a = *reinterpret_cast<const rows::AtElement*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 2) {
                out[2 * i] = __uint_as_float(a[i] << 16);
                out[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
            } else {
                out[i] = __uint_as_float(a[i]);
            }
        }
    }
}

template <typename T, int VE> __device__ __forceinline__ void store_vec(T* p, const float* in)
{
    if constexpr (VE == 1) {
        *p = from_f32<T>(in[0]);
    } else {
        alignas(16) T e[VE];
        Vec16<T>::store(e, in);
        const uint4 x = *reinterpret_cast<const uint4*>(e);
        *reinterpret_cast<rows::AtElement*>(p) = rows::AtElement{x.x, x.y, x.z, x.w};
    }
}

template <typename S> __device__ __forceinline__ void load_row(const typename S::elem* row, const Pair (&at)[S::NP], float (&x)[S::E])
{
    constexpr int VE = S::VE;
#pragma unroll
    for (int i = 0; i < S::NP; ++i) {
#pragma unroll
        for (int e = 0; e < 2 * VE; ++e)
            x[i * 2 * VE + e] = 0.f;
        if (at[i].a >= 0)
            load_vec<typename S::elem, VE>(row + at[i].a, x + i * 2 * VE);
        if (at[i].b >= 0)
            load_vec<typename S::elem, VE>(row + at[i].b, x + i * 2 * VE + VE);
    }
}

template <typename S> __device__ __forceinline__ void store_row(typename S::elem* row, const Pair (&at)[S::NP], const float (&x)[S::E])
{
    constexpr int VE = S::VE;
#pragma unroll
    for (int i = 0; i < S::NP; ++i) {
        if (at[i].a >= 0)
            store_vec<typename S::elem, VE>(row + at[i].a, x + i * 2 * VE);
        if (at[i].b >= 0)
            store_vec<typename S::elem, VE>(row + at[i].b, x + i * 2 * VE + VE);
    }
}

// The row turned (BACK: turned back) by the cosines and sines cs[frequency].
template <typename S, bool BACK>
__device__ __forceinline__ void turn(const float2* cs, const Pair (&at)[S::NP], bool interleaved, float (&x)[S::E])
{
    constexpr int VE = S::VE;
    auto one = [](float2 c, float& a, float& b) {
        const float s = BACK ? -c.y : c.y, u = a;
        a = u * c.x - b * s;
        b = b * c.x + u * s;
    };
#pragma unroll
    for (int i = 0; i < S::NP; ++i) {
        float* v = x + i * 2 * VE;
        if (VE > 1 && interleaved) {
            if (at[i].freq >= 0)
#pragma unroll
                for (int e = 0; e < VE / 2; ++e)
                    one(cs[at[i].freq + e], v[2 * e], v[2 * e + 1]);
            if (at[i].freq_b >= 0)
#pragma unroll
                for (int e = 0; e < VE / 2; ++e)
                    one(cs[at[i].freq_b + e], v[VE + 2 * e], v[VE + 2 * e + 1]);
        } else if (at[i].freq >= 0) {
#pragma unroll
            for (int e = 0; e < VE; ++e)
                one(cs[at[i].freq + e], v[e], v[VE + e]);
        }
    }
}

// cs[token][frequency] for `count` tokens from the one at `positions` on.
__device__ __forceinline__ void fill_angles(const int32_t* positions, const float* freqs, int count, int half,
                                            float scale, float2* cs)
{
    for (int i = threadIdx.x; i < count * half; i += kThreads) {
        const double turns = (double)positions[i / half] * (double)freqs[i % half] * 0.15915494309189533577;
        float s, c;
        sincospif((float)(2. * (turns - rint(turns))), &s, &c);
        cs[i] = make_float2(c * scale, s * scale);
    }
}

struct RowArgs {
    int64_t tokens;
    int heads[2];
    int width, rot, norm, tile;                              // tile: tokens a workgroup takes at once
    bool interleaved;
    float eps, rot_scale;
    int64_t stride[2], head_stride[2];
    const int32_t* positions;
    const float* freqs;
};

__device__ __forceinline__ float rstd_of(float ss, const RowArgs& p)
{
    return p.norm == 0 ? 1.f : rsqrtf((p.norm == 1 ? ss / (float)p.width : ss) + p.eps);
}

template <typename S> __device__ __forceinline__ void pairs_of(const RowArgs& p, Pair (&at)[S::NP])
{
#pragma unroll
    for (int i = 0; i < S::NP; ++i)
        at[i] = pair_at<S>(threadIdx.x % S::LANES + i * S::LANES, p.width, p.rot, p.interleaved);
}

}  // namespace

template <typename S>
__global__ __launch_bounds__(kThreads) void qk_norm_kernel(RowArgs p, const typename S::elem* xq, const typename S::elem* xk,
                                                           const typename S::elem* wq, const typename S::elem* wk,
                                                           typename S::elem* yq, typename S::elem* yk)
{
    extern __shared__ float2 cs[];
    const int64_t first = (int64_t)blockIdx.x * p.tile;
    const int count = p.tokens - first < p.tile ? (int)(p.tokens - first) : p.tile;
    const int half = p.rot / 2, group = threadIdx.x / S::LANES;
    Pair at[S::NP];
    pairs_of<S>(p, at);
    if (half) {
        fill_angles(p.positions + first, p.freqs, count, half, p.rot_scale, cs);
        __syncthreads();
    }
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const int heads = p.heads[which];
        const typename S::elem* w = which ? wk : wq;
        float wv[S::E];
        if (heads && w)
            load_row<S>(w, at, wv);
        for (int r = group; r < count * heads; r += S::GROUPS) {
            const int t = r / heads, h = r % heads;
            const typename S::elem* x = (which ? xk : xq) + (first + t) * p.stride[which] + h * p.head_stride[which];
            float v[S::E], ss[1] = {0.f};
            load_row<S>(x, at, v);
            if (p.norm) {
#pragma unroll
                for (int e = 0; e < S::E; ++e)
                    ss[0] += v[e] * v[e];
                rows::group_sum<S::LANES>(ss, nullptr, 0);
            }
            const float rstd = rstd_of(ss[0], p);
#pragma unroll
            for (int e = 0; e < S::E; ++e)
                v[e] = w ? v[e] * rstd * wv[e] : v[e] * rstd;
            if (half)
                turn<S, false>(cs + t * half, at, p.interleaved, v);
            store_row<S>((which ? yk : yq) + ((first + t) * heads + h) * p.width, at, v);
        }
    }
}

// part [block][width of dwq | width of dwk, where there is a k]
template <typename S>
__global__ __launch_bounds__(kThreads) void qk_norm_bwd_kernel(RowArgs p, const typename S::elem* xq, const typename S::elem* xk,
                                                               const typename S::elem* wq, const typename S::elem* wk,
                                                               const typename S::elem* dyq, const typename S::elem* dyk,
                                                               typename S::elem* dxq, typename S::elem* dxk, float* part)
{
    extern __shared__ float2 cs[];                           // the angles, then the sums of dw
    const int half = p.rot / 2, group = threadIdx.x / S::LANES;
    Pair at[S::NP];
    pairs_of<S>(p, at);
    float acc[2][S::E];
#pragma unroll
    for (int e = 0; e < S::E; ++e)
        acc[0][e] = acc[1][e] = 0.f;
    const float share = p.norm == 1 ? 1.f / (float)p.width : p.norm == 2 ? 1.f : 0.f;
    for (int64_t first = (int64_t)blockIdx.x * p.tile; first < p.tokens; first += (int64_t)gridDim.x * p.tile) {
        const int count = p.tokens - first < p.tile ? (int)(p.tokens - first) : p.tile;
        if (half) {
            __syncthreads();
            fill_angles(p.positions + first, p.freqs, count, half, p.rot_scale, cs);
            __syncthreads();
        }
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const int heads = p.heads[which];
            const typename S::elem* w = which ? wk : wq;
            float wv[S::E];
            if (heads && w)
                load_row<S>(w, at, wv);
            for (int r = group; r < count * heads; r += S::GROUPS) {
                const int t = r / heads, h = r % heads;
                const typename S::elem* x = (which ? xk : xq) + (first + t) * p.stride[which] + h * p.head_stride[which];
                const int64_t row = ((first + t) * heads + h) * p.width;
                float v[S::E], d[S::E], ss[2] = {0.f, 0.f};
                load_row<S>(x, at, v);
                load_row<S>((which ? dyk : dyq) + row, at, d);
                if (half)
                    turn<S, true>(cs + t * half, at, p.interleaved, d);
#pragma unroll
                for (int e = 0; e < S::E; ++e) {
                    ss[0] += v[e] * v[e];
                    ss[1] += (w ? d[e] * wv[e] : d[e]) * v[e];
                }
                if (p.norm)
                    rows::group_sum<S::LANES>(ss, nullptr, 0);
                const float rstd = rstd_of(ss[0], p), mean = ss[1] * rstd * share;
#pragma unroll
                for (int e = 0; e < S::E; ++e) {
                    const float xh = v[e] * rstd;
                    const float ew = w ? d[e] * wv[e] : d[e];
                    if (w)
                        acc[which][e] += d[e] * xh;
                    v[e] = p.norm ? rstd * (ew - xh * mean) : ew;
                }
                store_row<S>((which ? dxk : dxq) + row, at, v);
            }
        }
    }
    if (!part)
        return;
    float* buf = reinterpret_cast<float*>(cs);               // [group][width], the groups added in their order
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (!p.heads[which])
            continue;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < S::NP; ++i)
#pragma unroll
            for (int e = 0; e < S::VE; ++e) {
                if (at[i].a >= 0)
                    buf[group * p.width + at[i].a + e] = acc[which][i * 2 * S::VE + e];
                if (at[i].b >= 0)
                    buf[group * p.width + at[i].b + e] = acc[which][i * 2 * S::VE + S::VE + e];
            }
        __syncthreads();
        for (int c = threadIdx.x; c < p.width; c += kThreads) {
            float t = 0.f;
            for (int g = 0; g < S::GROUPS; ++g)
                t += buf[g * p.width + c];
            part[((int64_t)blockIdx.x * (p.heads[1] ? 2 : 1) + which) * p.width + c] = t;
        }
    }
}

namespace {

template <typename S> struct Tag { typedef S type; };

// Whole vectors where they fill the row and the rotation's pairs; else single elements.
template <typename T, typename Fn> hipError_t with_shape(const QkNormArgs& p, Fn&& fn)
{
    constexpr int VE = Vec16<T>::N;
    const bool whole = p.width % VE == 0 && p.rot % (p.interleaved ? VE : 2 * VE) == 0;
    if (!whole)
        return fn(Tag<Shape<T, 1, 64, kQkMaxWidth / 128>>{});
    const int pairs = (p.width / VE + 1) / 2;
    if (pairs <= 4) return fn(Tag<Shape<T, VE, 4, 1>>{});
    if (pairs <= 8) return fn(Tag<Shape<T, VE, 8, 1>>{});
    if (pairs <= 16) return fn(Tag<Shape<T, VE, 16, 1>>{});
    if (pairs <= 32) return fn(Tag<Shape<T, VE, 32, 1>>{});
    return fn(Tag<Shape<T, VE, 64, 1>>{});
}

RowArgs row_args(const QkNormArgs& p, int tile)
{
    RowArgs r;
    r.tokens = p.tokens;
    r.width = p.width;
    r.rot = p.rot;
    r.norm = p.norm;
    r.tile = tile;
    r.interleaved = p.interleaved;
    r.eps = p.eps;
    r.rot_scale = p.rot_scale;
    for (int i = 0; i < 2; ++i) {
        r.heads[i] = p.heads[i];
        r.stride[i] = p.stride[i];
        r.head_stride[i] = p.head_stride[i];
    }
    r.positions = p.positions;
    r.freqs = p.freqs;
    return r;
}

// Tokens a workgroup takes at once: 8, or fewer where that leaves compute units without work.
int tile_of(int64_t tokens) { return tokens >= 8192 ? 8 : tokens >= 2048 ? 4 : 1; }

template <typename T> hipError_t fwd(const QkNormArgs& p, hipStream_t stream)
{
    if (p.tokens == 0)
        return hipSuccess;
    return with_shape<T>(p, [&](auto tag) -> hipError_t {
        typedef typename decltype(tag)::type S;
        const int tile = tile_of(p.tokens);
        hipLaunchKernelGGL((qk_norm_kernel<S>), dim3((unsigned)((p.tokens + tile - 1) / tile)), dim3(kThreads),
                           (size_t)tile * (p.rot / 2) * sizeof(float2), stream, row_args(p, tile), (const T*)p.x[0],
                           (const T*)p.x[1], (const T*)p.w[0], (const T*)p.w[1], (T*)p.y[0], (T*)p.y[1]);
        return hipGetLastError();
    });
}

template <typename T> hipError_t bwd(const QkNormArgs& p, hipStream_t stream)
{
    const bool weights = p.dw[0];                            // of q and k, or of neither
    if (p.tokens == 0 && !weights)
        return hipSuccess;
    const int nb = qk_norm_bwd_blocks(p.tokens);
    const hipError_t e = with_shape<T>(p, [&](auto tag) -> hipError_t {
        typedef typename decltype(tag)::type S;
        const int tile = tile_of(p.tokens);
        const size_t angles = (size_t)tile * (p.rot / 2) * sizeof(float2);
        const size_t sums = weights ? (size_t)S::GROUPS * p.width * sizeof(float) : 0;
        hipLaunchKernelGGL((qk_norm_bwd_kernel<S>), dim3(nb), dim3(kThreads), angles > sums ? angles : sums, stream,
                           row_args(p, tile), (const T*)p.x[0], (const T*)p.x[1], (const T*)p.w[0], (const T*)p.w[1],
                           (const T*)p.dy[0], (const T*)p.dy[1], (T*)p.dx[0], (T*)p.dx[1], weights ? p.ws : nullptr);
        return hipGetLastError();
    });
    if (e != hipSuccess || !weights)
        return e;
    return rows::launch_sum_partials(p.ws, nb, p.heads[1] ? 2 * p.width : p.width, p.width, p.dw[0], p.dw[1], stream);
}

}  // namespace

int qk_norm_bwd_blocks(int64_t tokens)
{
    const int tile = tile_of(tokens);
    const int64_t want = (tokens + tile - 1) / tile;
    return (int)(want < 1 ? 1 : want < kQkBwdBlocks ? want : kQkBwdBlocks);
}

hipError_t launch_qk_norm(const QkNormArgs& p, hipStream_t stream)
{
    return p.bf16 ? fwd<uint16_t>(p, stream) : fwd<float>(p, stream);
}

hipError_t launch_qk_norm_bwd(const QkNormArgs& p, hipStream_t stream)
{
    return p.bf16 ? bwd<uint16_t>(p, stream) : bwd<float>(p, stream);
}

}  // namespace prism
