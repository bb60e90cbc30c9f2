// norm_residual.hip -- the step between two blocks of a layer stack: the block's
// output y joins the residual stream x, scaled per channel, and the sum is
// normalised for the next block,
//   r = x + s * y,   n = r rstd w,   rstd = 1 / sqrt(mean(r^2) + eps),
// and its gradients.  With e = dn * w, rh = r rstd and dr the gradient that
// arrives on the residual stream itself:
//   t  = dL/dr = rstd (e - rh mean(e rh)) + dr
//   dx = t,  dy = s t,  ds = sum_rows t y,  dw = sum_rows dn rh.
// mean(e rh) = rstd mean(e r), so both row sums (r^2 and e r) are taken in one
// pass over the row.
//
// Bound by HBM: every element is read and written once, at 6 to 14 operations.  Backward
// of 16,384 rows of 768 in bf16 with scale: 151 MB in 32 us, 4.7 TB/s, of which the
// second launch takes 4; 4,099 rows of 1,001 in fp32, forward, 11.5 us; a decode
// step's 8 rows, 5.8 us, a launch and one read after another.
// A row stays in registers between the sum and the scaling; w and s stay in
// registers over all rows of a workgroup, and so do the column sums of the
// backward, which leave one fp32 partial row per workgroup (no atomics: the
// second pass adds the partials in a fixed order).
// n is formed from the fp32 sum, before r is rounded for storage: one rounding
// per output.  Outputs may be the inputs' own buffers: a lane has read its
// elements of a row before it stores them, and no other lane touches them.
#include "common.h"
#include "kernels.h"
#include "norm_rows.h"

namespace prism {

using rows::group_sum;

template <typename S>
__global__ __launch_bounds__(S::THREADS) void norm_residual_kernel(
    const typename S::elem* x, const typename S::elem* y, const typename S::elem* scale,
    const typename S::elem* w, float eps, int64_t n_rows, int width, typename S::elem* r_out,
    typename S::elem* n_out)
{
    __shared__ float red[2 * S::THREADS / 64];
    const int64_t first = (int64_t)blockIdx.x * S::GROUPS + threadIdx.x / S::LANES;
    const S sh(threadIdx.x % S::LANES, width);
    float wv[S::E], sv[S::E];
    sh.load_weight(w, wv);
    if (scale)
        sh.load_weight(scale, sv);
    const float inv = 1.f / (float)width;
    const int64_t step = (int64_t)gridDim.x * S::GROUPS;
    int phase = 0;
    for (int64_t i = first; i < n_rows; i += step) {
        const int64_t at = i * width, room = (n_rows - i) * width;
        typename S::Raw xr, yr;
        sh.load(x + at, room, xr);
        if (y)
            sh.load(y + at, room, yr);
        float r[S::E];
        S::unpack(xr, r);
        if (y) {
            float yv[S::E];
            S::unpack(yr, yv);
#pragma unroll
            for (int c = 0; c < S::E; ++c)
                r[c] += scale ? sv[c] * yv[c] : yv[c];
        }
        float ss[1] = {0.f};
#pragma unroll
        for (int c = 0; c < S::E; ++c)
            ss[0] += r[c] * r[c];
        group_sum<S::LANES>(ss, red, phase);
        phase ^= 1;
        const float rstd = rsqrtf(ss[0] * inv + eps);
        if (r_out)
            sh.store(r_out + at, r);
#pragma unroll
        for (int c = 0; c < S::E; ++c)
            r[c] *= rstd * wv[c];
        sh.store(n_out + at, r);
    }
}

template <typename S>
__global__ __launch_bounds__(S::THREADS) void norm_residual_bwd_kernel(
    const typename S::elem* r, const typename S::elem* y, const typename S::elem* scale,
    const typename S::elem* w, float eps, const typename S::elem* dn, const typename S::elem* dr,
    int64_t n_rows, int width, typename S::elem* dx, typename S::elem* dy, float* part, bool want_scale)
{
    __shared__ float red[2 * 2 * S::THREADS / 64];
    extern __shared__ float buf[];
    const int64_t first = (int64_t)blockIdx.x * S::GROUPS + threadIdx.x / S::LANES;
    const S sh(threadIdx.x % S::LANES, width);
    float wv[S::E], sv[S::E], aw[S::E], as[S::E];
    sh.load_weight(w, wv);
    if (scale)
        sh.load_weight(scale, sv);
#pragma unroll
    for (int c = 0; c < S::E; ++c)
        aw[c] = as[c] = 0.f;
    const float inv = 1.f / (float)width;
    const int64_t step = (int64_t)gridDim.x * S::GROUPS;
    int phase = 0;
    for (int64_t i = first; i < n_rows; i += step) {
        const int64_t at = i * width, room = (n_rows - i) * width;
        typename S::Raw rr, dnr, drr, yr;
        sh.load(r + at, room, rr);
        sh.load(dn + at, room, dnr);
        if (dr)
            sh.load(dr + at, room, drr);
        if (want_scale)
            sh.load(y + at, room, yr);
        float rv[S::E], dv[S::E];
        S::unpack(rr, rv);
        S::unpack(dnr, dv);
        float ss[2] = {0.f, 0.f};
#pragma unroll
        for (int c = 0; c < S::E; ++c) {
            ss[0] += rv[c] * rv[c];
            ss[1] += dv[c] * wv[c] * rv[c];
        }
        group_sum<S::LANES>(ss, red, phase);
        phase ^= 1;
        const float rstd = rsqrtf(ss[0] * inv + eps);
        const float mean = ss[1] * inv * rstd;           // mean(e rh)
        float t[S::E];
#pragma unroll
        for (int c = 0; c < S::E; ++c) {
            const float rh = rv[c] * rstd;
            aw[c] += dv[c] * rh;
            t[c] = rstd * (dv[c] * wv[c] - rh * mean);
        }
        if (dr) {
            S::unpack(drr, dv);
#pragma unroll
            for (int c = 0; c < S::E; ++c)
                t[c] += dv[c];
        }
        if (want_scale) {
            S::unpack(yr, dv);
#pragma unroll
            for (int c = 0; c < S::E; ++c)
                as[c] += t[c] * dv[c];
        }
        sh.store(dx + at, t);
        if (dy) {
            if (scale)
#pragma unroll
                for (int c = 0; c < S::E; ++c)
                    t[c] *= sv[c];
            sh.store(dy + at, t);
        }
    }
    const int cols = want_scale ? 2 * width : width;
    float* out = part + (int64_t)blockIdx.x * cols;
    rows::store_partial(sh, aw, buf, out);
    if (want_scale)
        rows::store_partial(sh, as, buf, out + width);
}

namespace rows {

__global__ __launch_bounds__(kPartCols* kPartSlices) void sum_partials_kernel(const float* part, int nb,
                                                                           int cols, int split, float* out0,
                                                                           float* out1)
{
    __shared__ float s[kPartSlices][kPartCols + 1];
    const int ci = threadIdx.x % kPartCols, slice = threadIdx.x / kPartCols;
    const int c = blockIdx.x * kPartCols + ci;
    float t = 0.f;
    if (c < cols)
#pragma unroll 4
        for (int i = slice; i < nb; i += kPartSlices)
            t += part[(int64_t)i * cols + c];
    s[slice][ci] = t;
    __syncthreads();
#pragma unroll
    for (int m = kPartSlices / 2; m > 0; m >>= 1) {
        if (slice < m)
            s[slice][ci] += s[slice + m][ci];
        __syncthreads();
    }
    if (slice == 0 && c < cols) {
        if (c < split)
            out0[c] = s[0][ci];
        else
            out1[c - split] = s[0][ci];
    }
}

hipError_t launch_sum_partials(const float* part, int nb, int cols, int split, float* out0, float* out1,
                               hipStream_t stream)
{
    hipLaunchKernelGGL(sum_partials_kernel, dim3((cols + kPartCols - 1) / kPartCols),
                       dim3(kPartCols * kPartSlices), 0, stream, part, nb, cols, split, out0, out1);
    return hipGetLastError();
}

}  // namespace rows

// Two workgroups a compute unit, and half as many of the wide rows' twice as large ones:
// more leave more partials to add, fewer leave memory idle (16,384 rows of 768, bf16: 256,
// 512, 768, 1024 workgroups 40.3, 36.7, 38.7, 40.5 us; 4096 rows of 8192: 95.6, 107,
// 123, 137 us).
int norm_residual_bwd_blocks(int64_t n_rows, int width)
{
    const int64_t cap = width > 4096 ? kNormBwdBlocks / 2 : kNormBwdBlocks;
    return (int)(n_rows < 1 ? 1 : n_rows < cap ? n_rows : cap);
}

template <typename T> static hipError_t launch_fwd(const NormResidualArgs& p, hipStream_t stream)
{
    if (p.rows == 0)
        return hipSuccess;
    return rows::with_shape<T>(p.width, [&](auto tag) -> hipError_t {
        typedef typename decltype(tag)::type S;
        const int64_t want = (p.rows + S::GROUPS - 1) / S::GROUPS, cap = 2048 * 256 / S::THREADS;
        hipLaunchKernelGGL((norm_residual_kernel<S>), dim3((unsigned)(want < cap ? want : cap)),
                           dim3(S::THREADS), 0, stream, (const T*)p.x, (const T*)p.y, (const T*)p.scale,
                           (const T*)p.w, p.eps, p.rows, p.width, (T*)p.r, (T*)p.n);
        return hipGetLastError();
    });
}

template <typename T> static hipError_t launch_bwd_t(const NormResidualArgs& p, hipStream_t stream)
{
    const int nb = norm_residual_bwd_blocks(p.rows, p.width);
    const bool ws = p.dscale != nullptr;
    const hipError_t e = rows::with_shape<T>(p.width, [&](auto tag) -> hipError_t {
        typedef typename decltype(tag)::type S;
        hipLaunchKernelGGL((norm_residual_bwd_kernel<S>), dim3(nb), dim3(S::THREADS),
                           S::PARTIAL_LDS, stream, (const T*)p.r, (const T*)p.y,
                           (const T*)p.scale, (const T*)p.w, p.eps, (const T*)p.dn, (const T*)p.dr, p.rows,
                           p.width, (T*)p.dx, (T*)p.dy, p.ws, ws);
        return hipGetLastError();
    });
    if (e != hipSuccess)
        return e;
    return rows::launch_sum_partials(p.ws, nb, ws ? 2 * p.width : p.width, p.width, p.dw, p.dscale, stream);
}

hipError_t launch_norm_residual(const NormResidualArgs& p, hipStream_t stream)
{
    return p.bf16 ? launch_fwd<uint16_t>(p, stream) : launch_fwd<float>(p, stream);
}

hipError_t launch_norm_residual_bwd(const NormResidualArgs& p, hipStream_t stream)
{
    return p.bf16 ? launch_bwd_t<uint16_t>(p, stream) : launch_bwd_t<float>(p, stream);
}

}  // namespace prism
