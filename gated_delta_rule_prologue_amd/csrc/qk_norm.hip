// qk_norm.hip -- the queries and keys that enter the memory-writing operator: every head's
// row of d elements is normalised, weighted and rotated by its token's position,
//   xh = x rstd,   rstd = 1 / sqrt(mean(x^2) + eps) (rms), 1 / sqrt(sum(x^2) + eps) (l2) or 1,
//   y = R(position * freqs) (xh w),
// where R turns the pairs of the first `rot` elements: (i, i + rot / 2) in the half layout,
// (2 i, 2 i + 1) in the interleaved one.  Gradients: e = R^T dy,
//   dw = sum e xh,   dx = rstd (e w - xh c sum(e w xh)),   c = 1 / d (rms), 1 (l2), 0 (none).
//
// Angles: the product of an int32 position and an fp32 frequency is right to 2^-53 in 64
// bits; its whole turns are dropped there, and sine and cosine are formed in 32 bits from what is
// left.  At a frequency of one that is less than fp32's half step up to positions of 2^28, and 2.4 10^-7 at 2^31.
//
// Bound by HBM (2 streams forward, 3 backward).  A lane holds pairs of 16-byte vectors of a
// row, the two that rotate with each other in the half layout, so a row needs width / 16
// lanes in bf16 (width / 8 in fp32), the rotation stays in a lane, and a lane keeps to the same
// frequencies.  Forward a workgroup takes all rows of a few tokens, q's and k's, on angles that it
// forms once in LDS while the first rows are on their way (16,384 tokens of 6 + 6 heads of 128
// bf16: 25 us, 4.0 TB/s, in a graph over four sets of inputs, 21 us eager over three, which leave more of them in the
// Infinity Cache; a plain copy of as many bytes 20 us).  Backward a group of lanes takes
// the heads of one token on angles in its registers, and sums the weights' gradients there: no
// barrier but for their last sums, which a second launch joins (the same sizes 37 us, 4.1 TB/s,
// 34 without weights; eager 34).  Other times here are of such graphs too.  Rows that do not fill whole vectors (and rotations that do not fill whole
// pairs of them) take single elements, a wavefront a row beyond 32 of them.
#include "common.h"
#include "kernels.h"
#include "norm_rows.h"

namespace prism {

namespace {

constexpr int kThreads = 256;
// Rows whose terms of a weight's gradient a lane adds up in turn, at most, before they join its sum of the stretches
// before in LDS: so the rounding errors grow with 256 and a lane's 256ths of the rows, not with its rows.
constexpr int kStretch = 256;
// The elements of a row that a lane holds: NP pairs of vectors of VE elements.
template <typename T, bool INTERLEAVED_, int VE_, int LANES_, int NP_> struct Shape {
    typedef T elem;
    static constexpr bool INTERLEAVED = INTERLEAVED_;
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

// Pair j of a row.  The half layout's first pairs are vectors that turn with each other; of the other
// vectors the first half goes with the second, so that neighbouring lanes read neighbouring vectors.
template <typename S> __device__ __forceinline__ Pair pair_at(int j, int width, int rot)
{
    constexpr int VE = S::VE;
    constexpr bool interleaved = S::INTERLEAVED, inside = interleaved && VE > 1;     // inside: pairs lie within a vector
    const int turning = inside ? 0 : rot / 2 / VE, rest = inside ? 0 : rot;
    Pair p;
    if (j < turning) {
        p.a = interleaved ? 2 * j : j * VE;
        p.b = interleaved ? 2 * j + 1 : j * VE + rot / 2;
        p.freq = j * VE;
        p.freq_b = -1;
        return p;
    }
    const int half = ((width - rest) / VE + 1) / 2;
    p.a = j - turning < half ? rest + (j - turning) * VE : width;
    p.b = p.a + half * VE;
    p.freq = inside && p.a < rot ? p.a / 2 : -1;
    p.freq_b = inside && p.b < rot ? p.b / 2 : -1;
    if (p.a >= width)
        p.a = -1;
    if (p.b >= width)
        p.b = -1;
    return p;
}

// A branch that all lanes take alike, kept as one instead of selections.
__device__ __forceinline__ void apart() { asm volatile(""); }

// VE elements as they are stored, and as numbers.
template <typename T, int VE> struct RawVec {
    rows::AtElement v;
    __device__ __forceinline__ void clear() { v = rows::AtElement{0, 0, 0, 0}; }
    __device__ __forceinline__ void load(const T* p) { v = *reinterpret_cast<const rows::AtElement*>(p); }
    __device__ __forceinline__ void unpack(float* out) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 2) {
                out[2 * i] = __uint_as_float(v[i] << 16);
                out[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
            } else {
                out[i] = __uint_as_float(v[i]);
            }
        }
    }
};
template <typename T> struct RawVec<T, 1> {
    T v;
    __device__ __forceinline__ void clear() { v = T(0); }
    __device__ __forceinline__ void load(const T* p) { v = *p; }
    __device__ __forceinline__ void unpack(float* out) const { out[0] = to_f32(v); }
};

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

// A row as it is stored.  Lanes keep the zeros they begin with in place of vectors that they have not.
template <typename S> struct RawRow {
    typedef typename S::elem T;
    RawVec<T, S::VE> a[S::NP], b[S::NP];
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < S::NP; ++i) {
            a[i].clear();
            b[i].clear();
        }
    }
    __device__ __forceinline__ void load(const T* row, const Pair (&at)[S::NP])
    {
#pragma unroll
        for (int i = 0; i < S::NP; ++i) {
            if (at[i].a >= 0)
                a[i].load(row + at[i].a);
            if (at[i].b >= 0)
                b[i].load(row + at[i].b);
        }
    }
    __device__ __forceinline__ void unpack(float (&x)[S::E]) const
    {
#pragma unroll
        for (int i = 0; i < S::NP; ++i) {
            a[i].unpack(x + i * 2 * S::VE);
            b[i].unpack(x + i * 2 * S::VE + S::VE);
        }
    }
};

template <typename S>
__device__ __forceinline__ void store_row(typename S::elem* row, const Pair (&at)[S::NP], const float (&x)[S::E])
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

// Cosine and sine of a * b quarter turns, by series in what is left of the angle beyond the nearest one, r quarter
// turns (|r| <= 1/2, so at most pi / 4; up to the 9th and 10th power: 2 10^-9 and less), which then trade places
// and signs.  Adding 1.5 * 2^52 leaves the number of quarter turns in the sum's low word.
__device__ __forceinline__ void cos_sin(double a64, double b64, float scale, float& c, float& s)
{
    const double m = __builtin_fma(a64, b64, 6755399441055744.), n = m - 6755399441055744.;
    const float r = (float)__builtin_fma(a64, b64, -n), y = r * r;
    // the series' coefficients times powers of pi / 2
    float a = __builtin_fmaf(y, 1.6044118478735982e-4f, -4.6817541353186881e-3f);
    a = __builtin_fmaf(a, y, 7.9692626246167045e-2f);
    a = __builtin_fmaf(a, y, -6.4596409750624625e-1f);
    a = __builtin_fmaf(a, y, 1.5707963267948966f);
    const float sx = a * r;
    float b = __builtin_fmaf(y, -2.5202042373060605e-5f, 9.1926027483942658e-4f);
    b = __builtin_fmaf(b, y, -2.0863480763352961e-2f);
    b = __builtin_fmaf(b, y, 2.5366950790104802e-1f);
    b = __builtin_fmaf(b, y, -1.2337005501361698f);
    const float cx = __builtin_fmaf(b, y, 1.f);
    const uint32_t k = (uint32_t)__double_as_longlong(m);    // sin: sx, cx, -sx, -cx for k = 0, 1, 2, 3 (mod 4)
    s = scale * __uint_as_float(__float_as_uint(k & 1 ? cx : sx) ^ (k & 2) << 30);
    c = scale * __uint_as_float(__float_as_uint(k & 1 ? sx : cx) ^ ((k + 1) & 2) << 30);
}
constexpr double kQuarterTurns = 0.63661977236758134308;     // in one radian: 2 / pi

// The row turned, or (BACK) turned back, by the cosines and sines cs(f, i): of frequency f, the i-th that the lane
// needs.  Vectors that turn with each other have one frequency an element, vectors that hold whole pairs one for
// two: VE a pair of vectors.
template <typename S, bool BACK, typename F>
__device__ __forceinline__ void turn(const Pair (&at)[S::NP], float (&x)[S::E], F cs)
{
    constexpr int VE = S::VE, H = VE / 2;
    auto one = [&](int f, int i, float& a, float& b) {
        const float2 t = cs(f, i);
        const float sn = BACK ? -t.y : t.y, u = a;
        a = u * t.x - b * sn;
        b = b * t.x + u * sn;
    };
#pragma unroll
    for (int i = 0; i < S::NP; ++i) {
        float* v = x + i * 2 * VE;
        if constexpr (S::INTERLEAVED && VE > 1) {
            if (at[i].freq >= 0)
#pragma unroll
                for (int e = 0; e < H; ++e)
                    one(at[i].freq + e, i * VE + e, v[2 * e], v[2 * e + 1]);
            if (at[i].freq_b >= 0)
#pragma unroll
                for (int e = 0; e < H; ++e)
                    one(at[i].freq_b + e, i * VE + H + e, v[VE + 2 * e], v[VE + 2 * e + 1]);
        } else if (at[i].freq >= 0) {
#pragma unroll
            for (int e = 0; e < VE; ++e)
                one(at[i].freq + e, i * VE + e, v[e], v[VE + e]);
        }
    }
}

// Forward: the angles of a workgroup's tokens in LDS, cs[token][frequency], for all heads of q and k.  A thread
// keeps to one frequency.
__device__ __forceinline__ void fill_angles(const int32_t* positions, const float* freqs, int count, int half,
                                            float scale, float2* cs)
{
    const int step = kThreads / half, t0 = threadIdx.x / half, i = threadIdx.x - t0 * half;
    if (t0 >= step)
        return;
    const double freq = (double)freqs[i] * kQuarterTurns;
    for (int t = t0; t < count; t += step) {
        float c, s;
        cos_sin(positions[t], freq, scale, c, s);
        cs[t * half + i] = make_float2(c, s);
    }
}

// Backward: those of a lane's pairs, in its registers.
template <typename S> struct Angles {
    static constexpr int N = S::NP * S::VE, H = S::VE / 2;
    float freq[N], c[N], s[N];

    __device__ __forceinline__ void load(const float* freqs, const Pair (&at)[S::NP])
    {
#pragma unroll
        for (int i = 0; i < S::NP; ++i)
#pragma unroll
            for (int e = 0; e < S::VE; ++e) {
                const bool second = S::INTERLEAVED && S::VE > 1 && e >= H;
                const int f = second ? at[i].freq_b : at[i].freq;
                freq[i * S::VE + e] = f >= 0 ? freqs[f + (second ? e - H : e)] : 0.f;
            }
    }
    __device__ __forceinline__ void at(int position, float scale)
    {
        const double turns = (double)position * kQuarterTurns;
#pragma unroll
        for (int i = 0; i < N; ++i)
            cos_sin(turns, freq[i], scale, c[i], s[i]);
    }
};

// One of q and k.
template <typename T> struct Side {
    const T *x, *w, *dy;                                     // w may be null
    T* y;                                                    // y, or dx
    uint32_t stride, head_stride;
    int heads, blocks;
    int tile;                                                // forward: tokens of a workgroup
    float inv_heads;
    int part, parts;                                         // backward: a group of lanes takes `part` heads of a token

    // Row r of a tile's, token by token: its token (r < 2^17, so the rounded quotient of r + 1/2 stays off whole
    // numbers) and its head.
    __device__ __forceinline__ void place(int r, int& t, int& h) const
    {
        t = (int)(((float)r + 0.5f) * inv_heads);
        h = r - t * heads;
    }
    // The row of head h of the t-th token from x on.
    __device__ __forceinline__ const T* row(const T* from, int t, int h) const
    {
        return from + ((uint64_t)(uint32_t)t * stride + (uint64_t)(uint32_t)h * head_stride);
    }
};

struct RowArgs {
    int64_t tokens;
    int width, rot, norm;
    float eps, share, rot_scale;                             // share: 1 / width (rms), 1 (l2), 0
    const int32_t* positions;
    const float* freqs;
};

// Sums over the LANES lanes of a group, in registers up to 16 lanes: neighbours, pairs, then the mirrored
// half of 8 and of 16.
template <int CTRL> __device__ __forceinline__ float add_dpp(float x)
{
    return x + __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(x), CTRL, 0xF, 0xF, false));
}
template <int LANES, int N> __device__ __forceinline__ void lane_sum(float (&s)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        s[i] = add_dpp<0xB1>(s[i]);
        s[i] = add_dpp<0x4E>(s[i]);
        if (LANES >= 8)
            s[i] = add_dpp<0x141>(s[i]);
        if (LANES >= 16)
            s[i] = add_dpp<0x140>(s[i]);
        if (LANES >= 32)
            s[i] += __shfl_xor(s[i], 16);
        if (LANES >= 64)
            s[i] += __shfl_xor(s[i], 32);
    }
}

template <typename S> __device__ __forceinline__ void pairs_of(const RowArgs& p, Pair (&at)[S::NP])
{
#pragma unroll
    for (int i = 0; i < S::NP; ++i)
        at[i] = pair_at<S>(threadIdx.x % S::LANES + i * S::LANES, p.width, p.rot);
}

// The weights, or ones.
template <typename S>
__device__ __forceinline__ void weights_of(const typename S::elem* w, const Pair (&at)[S::NP], float (&wv)[S::E])
{
#pragma unroll
    for (int e = 0; e < S::E; ++e)
        wv[e] = 1.f;
    if (w) {
        RawRow<S> raw;
        raw.clear();
        raw.load(w, at);
        raw.unpack(wv);
    }
}

}  // namespace

// The rows of one side of the tokens from `first` on; `angles`: they are formed first.
template <typename S>
__device__ __forceinline__ void norm_rows(const RowArgs& p, const Side<typename S::elem>& me, const Pair (&at)[S::NP],
                                          int64_t first, int count, bool angles, float2* cs)
{
    const int half = p.rot / 2, rows = count * me.heads;
    const typename S::elem* x = me.x + first * me.stride;
    typename S::elem* y = me.y + first * me.heads * p.width;
    float wv[S::E];
    weights_of<S>(me.w, at, wv);
    RawRow<S> raw;
    raw.clear();
    for (int r = threadIdx.x / S::LANES;; r += S::GROUPS) {
        int t, h;
        me.place(r < rows ? r : rows - 1, t, h);
        raw.load(me.row(x, t, h), at);
        if (angles) {                                        // while the first rows are on their way
            fill_angles(p.positions + first, p.freqs, count, half, p.rot_scale, cs);
            lds_barrier();
            angles = false;
        }
        if (r >= rows)
            break;
        float v[S::E];
        raw.unpack(v);
        if (p.norm) {
            apart();
            float ss[1] = {0.f};
#pragma unroll
            for (int e = 0; e < S::E; ++e)
                ss[0] = __builtin_fmaf(v[e], v[e], ss[0]);
            lane_sum<S::LANES>(ss);
            const float rstd = rsqrtf(__builtin_fmaf(ss[0], p.share, p.eps));
#pragma unroll
            for (int e = 0; e < S::E; ++e)
                v[e] *= rstd;
        }
        if (me.w) {
            apart();
#pragma unroll
            for (int e = 0; e < S::E; ++e)
                v[e] *= wv[e];
        }
        if (half)
            turn<S, false>(at, v, [&](int f, int) { return cs[t * half + f]; });
        store_row<S>(y + (uint32_t)r * (uint32_t)p.width, at, v);
    }
}

// q's workgroups, then k's; with `both` q's take k's rows of their tokens too, on the same angles.
template <typename S>
__global__ __launch_bounds__(kThreads) void qk_norm_kernel(RowArgs p, Side<typename S::elem> q, Side<typename S::elem> k,
                                                           bool both)
{
    extern __shared__ float2 cs[];
    const bool second = (int)blockIdx.x >= q.blocks;
    const int tile = second ? k.tile : q.tile;
    const int64_t first = (int64_t)(blockIdx.x - (second ? q.blocks : 0)) * tile;
    const int count = p.tokens - first < tile ? (int)(p.tokens - first) : tile;
    Pair at[S::NP];
    pairs_of<S>(p, at);
#pragma unroll 1
    for (int side = second; side <= (second || both); ++side)
        norm_rows<S>(p, side ? k : q, at, first, count, p.rot > 0 && side == second, cs);
}

// part [block][width of dwq | width of dwk, where there is a k]
template <typename S>
__global__ __launch_bounds__(kThreads) void qk_norm_bwd_kernel(RowArgs p, Side<typename S::elem> q, Side<typename S::elem> k,
                                                               float* part)
{
    typedef typename S::elem T;
    extern __shared__ float buf[];                           // with `part`: [group][width]
    const bool second = (int)blockIdx.x >= q.blocks;
    const Side<T> me = second ? k : q;
    const int block = blockIdx.x - (second ? q.blocks : 0), group = threadIdx.x / S::LANES;
    Pair at[S::NP];
    pairs_of<S>(p, at);
    float acc[S::E], wv[S::E];
#pragma unroll
    for (int e = 0; e < S::E; ++e)
        acc[e] = 0.f;
    weights_of<S>(me.w, at, wv);
    Angles<S> angles;
    if (p.rot)
        angles.load(p.freqs, at);
    // the lane's own places in LDS: the sums of its stretches
    auto join = [&](bool first) {
#pragma unroll
        for (int i = 0; i < S::NP; ++i)
#pragma unroll
            for (int e = 0; e < S::VE; ++e) {
                float* to = buf + opaque(group * p.width) + e;       // no registers for its addresses
                const int a = i * 2 * S::VE + e, b = a + S::VE;
                if (at[i].a >= 0)
                    to[at[i].a] = first ? acc[a] : to[at[i].a] + acc[a];
                if (at[i].b >= 0)
                    to[at[i].b] = first ? acc[b] : to[at[i].b] + acc[b];
                acc[a] = acc[b] = 0.f;
            }
    };
    const int every = kStretch / me.part;                    // tokens of a stretch, or parts of them
    int done = 0;
    const int64_t units = p.tokens * me.parts;
    RawRow<S> raw, raw_d;
    raw.clear();
    raw_d.clear();
    for (int64_t unit = (int64_t)block * S::GROUPS + group; unit < units; unit += (int64_t)me.blocks * S::GROUPS) {
        const int64_t t = unit / me.parts;
        const int h0 = (int)(unit - t * me.parts) * me.part, h1 = h0 + me.part < me.heads ? h0 + me.part : me.heads;
        const T *x = me.row(me.x + t * me.stride, 0, h0), *dy = me.dy + (t * me.heads + h0) * p.width;
        T* dx = me.y + (t * me.heads + h0) * p.width;
        raw.load(x, at);
        raw_d.load(dy, at);
        if (p.rot)                                           // while the first rows are on their way
            angles.at(p.positions[t], p.rot_scale);
        for (int h = h0; h < h1; ++h, dx += p.width) {
            float v[S::E], d[S::E];
            raw.unpack(v);
            raw_d.unpack(d);
            x += me.head_stride;
            dy += p.width;
            if (h + 1 < h1) {
                raw.load(x, at);
                raw_d.load(dy, at);
            }
            if (p.rot)
                turn<S, true>(at, d, [&](int, int n) { return make_float2(angles.c[n], angles.s[n]); });
            if (p.norm) {
                apart();
                float ss[2] = {0.f, 0.f};
#pragma unroll
                for (int e = 0; e < S::E; ++e) {
                    ss[0] = __builtin_fmaf(v[e], v[e], ss[0]);
                    ss[1] = __builtin_fmaf(d[e] * wv[e], v[e], ss[1]);
                }
                lane_sum<S::LANES>(ss);
                const float rstd = rsqrtf(__builtin_fmaf(ss[0], p.share, p.eps));
                const float mean = ss[1] * rstd * p.share;
#pragma unroll
                for (int e = 0; e < S::E; ++e) {
                    const float xh = v[e] * rstd;
                    acc[e] = __builtin_fmaf(d[e], xh, acc[e]);
                    v[e] = rstd * __builtin_fmaf(-xh, mean, d[e] * wv[e]);
                }
            } else {
                apart();
#pragma unroll
                for (int e = 0; e < S::E; ++e) {
                    acc[e] = __builtin_fmaf(d[e], v[e], acc[e]);
                    v[e] = d[e] * wv[e];
                }
            }
            store_row<S>(dx, at, v);
        }
        if (part && ++done % every == 0)
            join(done == every);
    }
    if (!part)
        return;
    // the groups' sums, added in their order; the lane has had a stretch if it has had its every-th unit
    join((int64_t)(every - 1) * me.blocks * S::GROUPS + (int64_t)block * S::GROUPS + group >= units);
    __syncthreads();
    for (int c = threadIdx.x; c < p.width; c += kThreads) {
        float t = 0.f;
        for (int g = 0; g < S::GROUPS; ++g)
            t += buf[g * p.width + c];
        part[((int64_t)block * (k.heads ? 2 : 1) + second) * p.width + c] = t;
    }
}

namespace {

template <typename S> struct Tag { typedef S type; };

// Whole vectors where they fill the row and the rotation's pairs; else single elements.
template <typename T, bool IL, typename Fn> hipError_t with_layout(const QkNormArgs& p, Fn&& fn)
{
    constexpr int VE = Vec16<T>::N;
    if (p.width % VE || p.rot % (IL ? VE : 2 * VE)) {
        if (p.width <= 32) return fn(Tag<Shape<T, IL, 1, 16, 1>>{});
        if (p.width <= 128) return fn(Tag<Shape<T, IL, 1, 64, 1>>{});
        if (p.width <= 256) return fn(Tag<Shape<T, IL, 1, 64, 2>>{});
        return fn(Tag<Shape<T, IL, 1, 64, 4>>{});
    }
    const int pairs = (p.width / VE + 1) / 2;
    if (pairs <= 4) return fn(Tag<Shape<T, IL, VE, 4, 1>>{});
    if (pairs <= 8) return fn(Tag<Shape<T, IL, VE, 8, 1>>{});
    if (pairs <= 16) return fn(Tag<Shape<T, IL, VE, 16, 1>>{});
    if (pairs <= 32) return fn(Tag<Shape<T, IL, VE, 32, 1>>{});
    return fn(Tag<Shape<T, IL, VE, 64, 1>>{});
}

template <typename T, typename Fn> hipError_t with_shape(const QkNormArgs& p, Fn&& fn)
{
    return p.interleaved && p.rot > 0 ? with_layout<T, true>(p, fn) : with_layout<T, false>(p, fn);
}

RowArgs row_args(const QkNormArgs& p)
{
    RowArgs r;
    r.tokens = p.tokens;
    r.width = p.width;
    r.rot = p.rot;
    r.norm = p.norm;
    r.eps = p.eps;
    r.share = p.norm == 1 ? 1.f / (float)p.width : p.norm == 2 ? 1.f : 0.f;
    r.rot_scale = p.rot_scale;
    r.positions = p.positions;
    r.freqs = p.freqs;
    return r;
}

template <typename S> Side<typename S::elem> side_of(const QkNormArgs& p, int i, bool bwd)
{
    typedef typename S::elem T;
    Side<T> s = {};
    s.heads = p.heads[i];
    if (s.heads == 0)
        return s;
    s.x = (const T*)p.x[i];
    s.w = (const T*)p.w[i];
    s.dy = (const T*)p.dy[i];
    s.y = (T*)(bwd ? p.dx[i] : p.y[i]);
    s.stride = (uint32_t)p.stride[i];
    s.head_stride = (uint32_t)p.head_stride[i];
    s.inv_heads = 1.f / s.heads;
    // forward: tokens that fill a workgroup's rows once (angles of at most 32 KB; twice: LM layer 26.8 instead of
    // 25.2 us), or fewer where that leaves compute units without work
    s.tile = S::GROUPS / s.heads;
    if (p.rot > 0 && s.tile > 8192 / p.rot)
        s.tile = 8192 / p.rot;
    while (s.tile > 1 && p.tokens / s.tile < 512)
        s.tile /= 2;
    if (s.tile < 1)
        s.tile = 1;
    // backward: all heads of a token on the same angles (those of a stretch), or fewer where that leaves SIMDs without a wavefront
    for (s.part = s.heads < kStretch ? s.heads : kStretch;; s.part = (s.part + 1) / 2) {
        s.parts = (s.heads + s.part - 1) / s.part;
        if (s.part == 1 || p.tokens * s.parts * S::LANES >= 1024 * 64)
            break;
    }
    const int64_t want = bwd ? (p.tokens * s.parts + S::GROUPS - 1) / S::GROUPS : (p.tokens + s.tile - 1) / s.tile;
    s.blocks = (int)(want < 1 ? 1 : want);
    return s;
}

template <typename T> hipError_t fwd(const QkNormArgs& p, hipStream_t stream)
{
    if (p.tokens == 0)
        return hipSuccess;
    return with_shape<T>(p, [&](auto tag) -> hipError_t {
        typedef typename decltype(tag)::type S;
        const Side<T> q = side_of<S>(p, 0, false), k = side_of<S>(p, 1, false);
        // few tokens: k's rows on other compute units rather than behind q's (LM layer 28.8 us with its angles formed twice)
        const bool both = k.heads > 0 && p.tokens >= 2048 && (int64_t)q.tile * k.heads <= 1 << 17;         // place()
        const int tile = both || q.tile > k.tile ? q.tile : k.tile;
        hipLaunchKernelGGL((qk_norm_kernel<S>), dim3((unsigned)q.blocks + (both ? 0 : k.blocks)), dim3(kThreads),
                           (size_t)tile * (p.rot / 2) * sizeof(float2), stream, row_args(p), q, k, both);
        return hipGetLastError();
    });
}

template <typename T> hipError_t bwd(const QkNormArgs& p, hipStream_t stream)
{
    const bool weights = p.dw[0];                            // of q and k, or of neither
    if (p.tokens == 0 && !weights)
        return hipSuccess;
    int nb = 0;
    const hipError_t e = with_shape<T>(p, [&](auto tag) -> hipError_t {
        typedef typename decltype(tag)::type S;
        Side<T> q = side_of<S>(p, 0, true), k = side_of<S>(p, 1, true);
        if (weights) {                                       // as many workgroups each: their partial sums lie side by side
            // fewer where a wavefront holds several rows, more where its lanes hold but a pair each (LM layer: 256 of them
            // 36.9, 512 39.1 us; 4096 tokens of 4 + 4 heads of 256 in fp32: 256 25.5, 512 28.2 us; 20,000 of 5 + 1 of 75:
            // 512 57, 1024 39 us; 4096 of 6 + 6 of 130 in bf16: 512 24.3, 1024 26.3 us)
            const int most = q.blocks > k.blocks ? q.blocks : k.blocks, all = qk_norm_bwd_blocks(p.tokens);
            const int limit = S::GROUPS >= 8 ? kQkBwdBlocks / 4 : S::E > 2 ? kQkBwdBlocks / 2 : kQkBwdBlocks;
            const int cap = all < limit ? all : limit;
            q.blocks = most < cap ? most : cap;
            k.blocks = k.heads ? q.blocks : 0;
        }
        nb = q.blocks;
        hipLaunchKernelGGL((qk_norm_bwd_kernel<S>), dim3((unsigned)q.blocks + k.blocks), dim3(kThreads),
                           weights ? (size_t)S::GROUPS * p.width * sizeof(float) : 0, stream, row_args(p), q, k,
                           weights ? p.ws : nullptr);
        return hipGetLastError();
    });
    if (e != hipSuccess || !weights)
        return e;
    return rows::launch_sum_partials(p.ws, nb, p.heads[1] ? 2 * p.width : p.width, p.width, p.dw[0], p.dw[1], stream);
}

}  // namespace

// Workgroups of q, and of k, in a backward pass that sums weights' gradients, at most.
int qk_norm_bwd_blocks(int64_t tokens)
{
    return (int)(tokens < 1 ? 1 : tokens < kQkBwdBlocks ? tokens : kQkBwdBlocks);
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
