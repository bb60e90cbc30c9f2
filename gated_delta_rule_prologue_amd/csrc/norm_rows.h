// norm_rows.h -- rows of a matrix held in registers by groups of lanes: the
// loads, stores and row sums shared by the residual norm and the gated norm
// (norm_residual.hip, norm_gate.hip).
//
// A group of LANES lanes owns one row at a time and keeps it in registers, so
// a row is read once whatever is computed from it; lane l holds the vectors
// l, l + LANES, ... (NV of them), so that every access of a group is
// contiguous.  Rows whose width fills whole 16-byte vectors are read in those
// (every row then starts at a 16-byte address); other widths element by
// element, since their rows start anywhere.
#pragma once

#include <type_traits>

#include "common.h"

namespace prism {
namespace rows {

template <typename T, bool VECTOR, int LANES_, int NV_> struct Shape {
    typedef T elem;
    static constexpr int LANES = LANES_;
    static constexpr int NV = NV_;
    static constexpr int VE = VECTOR ? Vec16<T>::N : 1;        // elements per access
    static constexpr int E = NV * VE;                          // elements per lane
    static constexpr int THREADS = LANES > 64 ? LANES : 256;
    static constexpr int GROUPS = THREADS / LANES;             // rows in flight per workgroup

    static constexpr size_t PARTIAL_LDS = GROUPS > 1 ? (size_t)THREADS * E * sizeof(float) : 0;

    typedef typename std::conditional<VECTOR, uint4, T>::type access;
    struct Raw { access v[NV]; };

    __device__ static int col(int j, int lane) { return (j * LANES + lane) * VE; }

    // elements past the width read as zero
    __device__ static void load(const T* row, int lane, int width, Raw& x)
    {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            x.v[j] = access{};
            if (col(j, lane) < width)
                x.v[j] = *reinterpret_cast<const access*>(row + col(j, lane));
        }
    }
    __device__ static void unpack(const Raw& x, float* out)
    {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (!VECTOR) {
                out[j] = to_f32(x.v[j]);
            } else if constexpr (sizeof(T) == 2) {
                const uint32_t w[4] = {x.v[j].x, x.v[j].y, x.v[j].z, x.v[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    out[j * VE + 2 * i] = __uint_as_float(w[i] << 16);
                    out[j * VE + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                }
            } else {
                out[j * VE] = __uint_as_float(x.v[j].x);
                out[j * VE + 1] = __uint_as_float(x.v[j].y);
                out[j * VE + 2] = __uint_as_float(x.v[j].z);
                out[j * VE + 3] = __uint_as_float(x.v[j].w);
            }
        }
    }
    __device__ static void load_f32(const T* row, int lane, int width, float* out)
    {
        Raw x;
        load(row, lane, width, x);
        unpack(x, out);
    }
    __device__ static void store(T* row, int lane, int width, const float* in)
    {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (col(j, lane) < width) {
                if constexpr (VECTOR)
                    Vec16<T>::store(row + col(j, lane), in + j * VE);
                else
                    row[col(j, lane)] = from_f32<T>(in[j]);
            }
    }
};

// Sums over the LANES lanes of a group, of one or two values; every lane gets
// them.  Groups of at most a wavefront exchange registers; larger ones are the
// whole workgroup and go through LDS, in the half of `red` that `phase` names:
// with the halves taken in turn one barrier per sum is enough, since a
// wavefront that writes a half again has passed the barrier of the other half,
// which every reader of the first reached after reading it.
template <int LANES, int N>
__device__ __forceinline__ void group_sum(float (&s)[N], float* red, int phase)
{
    constexpr int LW = LANES < 64 ? LANES : 64;
#pragma unroll
    for (int m = LW / 2; m > 0; m >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i)
            s[i] += __shfl_xor(s[i], m, LW);
    if constexpr (LANES > 64) {
        constexpr int NW = LANES / 64;
        float* r = red + phase * N * NW;
        const int wave = threadIdx.x / 64;
        if (threadIdx.x % 64 == 0)
#pragma unroll
            for (int i = 0; i < N; ++i)
                r[i * NW + wave] = s[i];
        lds_barrier();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float t = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w)
                t += r[i * NW + w];
            s[i] = t;
        }
    }
}

// Per-lane column sums of the groups of one workgroup, added up in the order
// of the groups and stored as fp32 at out[0..width) (one workgroup's partial).
// `buf` holds PARTIAL_LDS bytes; every thread of the workgroup calls it.
template <typename S>
__device__ __forceinline__ void store_partial(const float* acc, float* buf, int lane, int group, int width,
                                              float* out)
{
    if constexpr (S::GROUPS == 1) {
#pragma unroll
        for (int j = 0; j < S::NV; ++j)
#pragma unroll
            for (int i = 0; i < S::VE; ++i)
                if (S::col(j, lane) + i < width)
                    out[S::col(j, lane) + i] = acc[j * S::VE + i];
    } else {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < S::NV; ++j)
#pragma unroll
            for (int i = 0; i < S::VE; ++i)
                buf[group * S::LANES * S::E + S::col(j, lane) + i] = acc[j * S::VE + i];
        __syncthreads();
        for (int c = threadIdx.x; c < width; c += S::THREADS) {
            float t = 0.f;
#pragma unroll
            for (int g = 0; g < S::GROUPS; ++g)
                t += buf[g * S::LANES * S::E + c];
            out[c] = t;
        }
    }
}

// The shape for a width, handed to `fn` as a value of its Shape type.  A lane
// holds at most 16 elements (the backward keeps up to seven such arrays in
// registers); a row takes the fewest lanes that this allows, up to a wavefront,
// so that narrow rows (one head) leave no lane idle and need no LDS; wider rows
// take a whole workgroup.
template <typename T, typename Fn> hipError_t with_shape(int width, Fn&& fn)
{
    constexpr int VE = Vec16<T>::N, NV = 16 / VE;
    if (width % VE == 0) {
        const int nv = width / VE;
        if (nv <= 8) return fn(Shape<T, true, 8, 1>{});
        if (nv <= 16) return fn(Shape<T, true, 16, 1>{});
        if (nv <= 32) return fn(Shape<T, true, 32, 1>{});
        if (nv <= 64) return fn(Shape<T, true, 64, 1>{});
        if (nv <= 128) return fn(Shape<T, true, 64, 2>{});
        if constexpr (NV == 4) {
            if (nv <= 192) return fn(Shape<T, true, 64, 3>{});
            if (nv <= 256) return fn(Shape<T, true, 64, 4>{});
        }
        if (nv <= 128 * NV) return fn(Shape<T, true, 128, NV>{});
        if (nv <= 256 * NV) return fn(Shape<T, true, 256, NV>{});
        return fn(Shape<T, true, 512, NV>{});
    }
    if (width <= 8) return fn(Shape<T, false, 8, 1>{});
    if (width <= 64) return fn(Shape<T, false, 64, 1>{});
    if (width <= 256) return fn(Shape<T, false, 64, 4>{});
    if (width <= 1024) return fn(Shape<T, false, 64, 16>{});
    if (width <= 4096) return fn(Shape<T, false, 256, 16>{});
    return fn(Shape<T, false, 512, 16>{});
}

// out[c] = the sum over the nb rows of part [nb][cols], fp32: the second pass
// over the workgroups' partials.  Columns before `split` go to out0, the others
// to out1.  One workgroup per 16 columns; 64 threads a column take every 64th
// row each, then add up in a fixed order, so the result does not depend on
// timing.
constexpr int kPartCols = 16, kPartSlices = 64;

hipError_t launch_sum_partials(const float* part, int nb, int cols, int split, float* out0, float* out1,
                               hipStream_t stream);

}  // namespace rows
}  // namespace prism
