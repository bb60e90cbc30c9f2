// norm_gate.hip -- what follows the memory-writing operator in a layer: every
// head's output row o (width elements) is normalised, weighted and multiplied
// by its gate z,
//   y = o rstd w act(z),   rstd = 1 / sqrt(mean(o^2) + eps),
// act = silu or sigmoid, and the gradients: with oh = o rstd, e = dy act(z) w,
//   do = rstd (e - oh mean(e oh)),   dz = dy oh w act'(z),   dw = sum dy act(z) oh.
// w is one row for all heads, or one a head; dw is summed accordingly.
//
// Bound by HBM (3 streams forward, 5 backward, up to some 40 operations an
// element).  A head's row is a few hundred bytes, held by 8 to 64 lanes, so a
// wavefront works on several rows at once and the row sums stay within it.
// With a weight a head a workgroup keeps to one head (w and the column sums
// stay in its registers); its rows are then H rows apart, each of them at least
// a whole 64-byte segment at the operator's widths.  Forward of 65,536 tokens x 16 heads
// x 128 in bf16: 805 MB in 161 us, 5.0 TB/s (a copy of a gigabyte: 5.2); backward of
// 65,536 tokens x 4 heads x 64: 168 MB in 36 us, 4.7 TB/s, of which the second
// launch takes 4.  In fp32 65,536 x 4 x 128 takes 80 us forward and 124 us backward.  Outputs may be the inputs' own buffers.
#include "common.h"
#include "kernels.h"
#include "norm_rows.h"

namespace prism {

using rows::group_sum;

// e^-a for a >= 0 (a NaN stays one).  exp2 of the rounded product a log2 e is off by up to 64
// half steps of fp32 at a = 80.  That is nothing beside bf16's own rounding (2^-18 of the value
// against 2^-8); in fp32 it is 2^n 2^f with n + f = -a log2 e, |f| <= 1/2 and log2 e in two
// parts, so that f is rounded once and the error does not grow with a.
template <typename T> __device__ __forceinline__ float exp_minus(float a)
{
    if constexpr (sizeof(T) == 2)
        return __builtin_amdgcn_exp2f(a * -1.44269504088896341f);
    const float n = fmaxf(rintf(a * -1.44269504088896341f), -200.f);     // beyond it f takes the rest, and e^-a is zero
    const float f = __builtin_fmaf(a, -1.925962991e-8f, __builtin_fmaf(a, -1.44269502162933350f, -n));
    return ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
}

// act(z) and act'(z): s = 1 / (1 + e^-z) and c = 1 - s = 1 / (1 + e^z), both formed from
// e^-|z| <= 1 (a difference 1 - s would lose c of open gates: 6 % at z = 16, all of it from 18 on);
// silu = z s, silu' = s (1 + z c)
template <typename T, int GATE> __device__ __forceinline__ float gate_act(float z, float& slope)
{
    const float e = exp_minus<T>(fabsf(z)), d = __builtin_amdgcn_rcpf(1.f + e);
    const float s = z < 0.f ? e * d : d, c = z < 0.f ? d : e * d;
    if (GATE == 0) {
        slope = s * (1.f + z * c);
        return z * s;
    }
    slope = s * c;
    return s;
}

template <typename S, int GATE>
__global__ __launch_bounds__(S::THREADS) void norm_gate_kernel(
    const typename S::elem* o, const typename S::elem* z, const typename S::elem* w, float eps,
    int64_t tokens, int heads, int width, typename S::elem* y)
{
    __shared__ float red[2 * S::THREADS / 64];
    const int e = blockIdx.x % heads, tb = blockIdx.x / heads, nt = gridDim.x / heads;
    const int64_t first = (int64_t)tb * S::GROUPS + threadIdx.x / S::LANES;
    const S sh(threadIdx.x % S::LANES, width);
    float wv[S::E];
    sh.load_weight(w + (int64_t)e * width, wv);
    const float inv = 1.f / (float)width;
    int phase = 0;
    for (int64_t t = first; t < tokens; t += (int64_t)nt * S::GROUPS) {
        const int64_t at = (t * heads + e) * width, room = (tokens * heads - (t * heads + e)) * width;
        typename S::Raw orr, zr;
        sh.load(o + at, room, orr);
        sh.load(z + at, room, zr);
        float ov[S::E], zv[S::E];
        S::unpack(orr, ov);
        S::unpack(zr, zv);
        float ss[1] = {0.f};
#pragma unroll
        for (int c = 0; c < S::E; ++c)
            ss[0] += ov[c] * ov[c];
        group_sum<S::LANES>(ss, red, phase);
        phase ^= 1;
        const float rstd = rsqrtf(ss[0] * inv + eps);
#pragma unroll
        for (int c = 0; c < S::E; ++c) {
            float slope;
            ov[c] = ov[c] * rstd * wv[c] * gate_act<typename S::elem, GATE>(zv[c], slope);
        }
        sh.store(y + at, ov);
    }
}

template <typename S, int GATE>
__global__ __launch_bounds__(S::THREADS) void norm_gate_bwd_kernel(
    const typename S::elem* o, const typename S::elem* z, const typename S::elem* w, float eps,
    const typename S::elem* dy, int64_t tokens, int heads, int width, typename S::elem* d_o,
    typename S::elem* dz, float* part)
{
    __shared__ float red[2 * 2 * S::THREADS / 64];
    extern __shared__ float buf[];
    const int e = blockIdx.x % heads, tb = blockIdx.x / heads, nt = gridDim.x / heads;
    const int64_t first = (int64_t)tb * S::GROUPS + threadIdx.x / S::LANES;
    const S sh(threadIdx.x % S::LANES, width);
    float wv[S::E], aw[S::E];
    sh.load_weight(w + (int64_t)e * width, wv);
#pragma unroll
    for (int c = 0; c < S::E; ++c)
        aw[c] = 0.f;
    const float inv = 1.f / (float)width;
    int phase = 0;
    for (int64_t t = first; t < tokens; t += (int64_t)nt * S::GROUPS) {
        const int64_t at = (t * heads + e) * width, room = (tokens * heads - (t * heads + e)) * width;
        typename S::Raw orr, zr, dyr;
        sh.load(o + at, room, orr);
        sh.load(z + at, room, zr);
        sh.load(dy + at, room, dyr);
        float ov[S::E], zv[S::E], dv[S::E];
        S::unpack(orr, ov);
        S::unpack(zr, zv);
        S::unpack(dyr, dv);
        float ss[2] = {0.f, 0.f};
#pragma unroll
        for (int c = 0; c < S::E; ++c) {
            float slope;
            const float act = gate_act<typename S::elem, GATE>(zv[c], slope);
            zv[c] = dv[c] * wv[c] * slope * ov[c];       // dz, but for rstd
            dv[c] *= act;                                // dy act(z)
            ss[0] += ov[c] * ov[c];
            ss[1] += dv[c] * wv[c] * ov[c];
        }
        group_sum<S::LANES>(ss, red, phase);
        phase ^= 1;
        const float rstd = rsqrtf(ss[0] * inv + eps);
        const float mean = ss[1] * inv * rstd;           // mean(e oh)
#pragma unroll
        for (int c = 0; c < S::E; ++c) {
            const float oh = ov[c] * rstd;
            aw[c] += dv[c] * oh;
            ov[c] = rstd * (dv[c] * wv[c] - oh * mean);
            zv[c] *= rstd;
        }
        sh.store(d_o + at, ov);
        sh.store(dz + at, zv);
    }
    rows::store_partial(sh, aw, buf, part + ((int64_t)tb * heads + e) * width);
}

// Two workgroups a compute unit over all heads (65,536 tokens of 4 heads of 64, bf16: 256,
// 512, 768, 1024 workgroups 50.8, 37.5, 39.4, 41.1 us).
int norm_gate_bwd_blocks(int64_t tokens, int heads)
{
    const int64_t cap = heads < kNormBwdBlocks ? kNormBwdBlocks / heads : 1;
    return (int)(tokens < 1 ? 1 : tokens < cap ? tokens : cap);
}

template <typename T, int GATE> static hipError_t launch_fwd(const NormGateArgs& p, hipStream_t stream)
{
    if (p.tokens == 0)
        return hipSuccess;
    return rows::with_shape<T>(p.width, [&](auto tag) -> hipError_t {
        typedef typename decltype(tag)::type S;
        if constexpr (S::LANES <= 64) {                  // width <= kNormGateMaxWidth
            const int64_t want = (p.tokens + S::GROUPS - 1) / S::GROUPS;
            const int64_t cap = p.heads < 2048 ? 2048 / p.heads : 1;
            const int64_t nt = want < cap ? want : cap;
            hipLaunchKernelGGL((norm_gate_kernel<S, GATE>), dim3((unsigned)(nt * p.heads)), dim3(S::THREADS), 0,
                               stream, (const T*)p.o, (const T*)p.z, (const T*)p.w, p.eps, p.tokens, p.heads,
                               p.width, (T*)p.y);
            return hipGetLastError();
        }
        return hipErrorInvalidValue;
    });
}

template <typename T, int GATE> static hipError_t launch_bwd_t(const NormGateArgs& p, hipStream_t stream)
{
    const int nt = norm_gate_bwd_blocks(p.tokens, p.heads);
    const hipError_t e = rows::with_shape<T>(p.width, [&](auto tag) -> hipError_t {
        typedef typename decltype(tag)::type S;
        if constexpr (S::LANES <= 64) {
            hipLaunchKernelGGL((norm_gate_bwd_kernel<S, GATE>), dim3((unsigned)nt * p.heads), dim3(S::THREADS),
                               S::PARTIAL_LDS, stream, (const T*)p.o, (const T*)p.z,
                               (const T*)p.w, p.eps, (const T*)p.dy, p.tokens, p.heads, p.width, (T*)p.d_o,
                               (T*)p.dz, p.ws);
            return hipGetLastError();
        }
        return hipErrorInvalidValue;
    });
    if (e != hipSuccess)
        return e;
    const int cols = p.heads * p.width;
    return rows::launch_sum_partials(p.ws, nt, cols, cols, p.dw, nullptr, stream);
}

template <typename T> static hipError_t launch_T(const NormGateArgs& p, bool bwd, hipStream_t stream)
{
    if (bwd)
        return p.gate == 0 ? launch_bwd_t<T, 0>(p, stream) : launch_bwd_t<T, 1>(p, stream);
    return p.gate == 0 ? launch_fwd<T, 0>(p, stream) : launch_fwd<T, 1>(p, stream);
}

hipError_t launch_norm_gate(const NormGateArgs& p, hipStream_t stream)
{
    return p.bf16 ? launch_T<uint16_t>(p, false, stream) : launch_T<float>(p, false, stream);
}

hipError_t launch_norm_gate_bwd(const NormGateArgs& p, hipStream_t stream)
{
    return p.bf16 ? launch_T<uint16_t>(p, true, stream) : launch_T<float>(p, true, stream);
}

}  // namespace prism
