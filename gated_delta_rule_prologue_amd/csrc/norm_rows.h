// norm_rows.h -- rows of a matrix held in registers by groups of lanes: the
// loads, stores and row sums shared by the residual norm and the gated norm
// (norm_residual.hip, norm_gate.hip).
//
// A group of LANES lanes owns one row at a time and keeps it in registers, so
// a row is read once whatever is computed from it; lane l holds the 16-byte vectors
// l, l + LANES, ... (NV of them), so that every access of a group is contiguous.
// A row whose width does not fill whole vectors (kRagged) starts at any element's
// address; its vectors are read and written there all the same (global accesses of 16
// bytes need no alignment in the mode that the HSA runtime sets).  Its last vector also
// covers elements of the next rows, which are cleared after the load and left alone by
// the store (element by element there); where that vector would reach past the end of
// the tensor, the tensor's last 16 bytes are read and shifted into place.  Rows shorter
// than a vector (kShort) are read element by element.
#pragma once

#include <type_traits>

#include "common.h"

namespace prism {
namespace rows {

// 16 bytes at a 16-byte address, and at any element's.
typedef uint32_t Aligned __attribute__((ext_vector_type(4)));
typedef uint32_t AtElement __attribute__((ext_vector_type(4), aligned(2)));

enum Kind { kWhole, kRagged, kShort };

template <typename T, Kind KIND, int LANES_, int NV_> struct Shape {
    typedef T elem;
    static constexpr bool RAGGED = KIND != kWhole;
    static constexpr int LANES = LANES_;
    static constexpr int NV = NV_;
    static constexpr int VE = Vec16<T>::N;                     // elements per access
    static constexpr int E = NV * VE;                          // elements per lane
    static constexpr int THREADS = LANES > 64 ? LANES : 256;
    static constexpr int GROUPS = THREADS / LANES;             // rows in flight per workgroup
    static constexpr size_t PARTIAL_LDS = GROUPS > 1 ? (size_t)THREADS * E * sizeof(float) : 0;

    struct Raw { uint4 v[NV]; };

    typedef typename std::conditional<KIND == kWhole, Aligned, AtElement>::type Access;

    int lane, width;
    Raw mask;                                                  // kRagged: the bits of the row's elements

    __device__ Shape(int lane_, int width_) : lane(lane_), width(width_)
    {
        if constexpr (KIND == kRagged) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                uint32_t m[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    constexpr int P = VE / 4;                  // elements per dword
                    m[i] = 0;
#pragma unroll
                    for (int x = 0; x < P; ++x)
                        if (col(j) + i * P + x < width)
                            m[i] |= P == 1 ? 0xffffffffu : 0xffffu << (16 * x);
                }
                mask.v[j] = make_uint4(m[0], m[1], m[2], m[3]);
            }
        }
    }
    __device__ int col(int j) const { return (j * LANES + lane) * VE; }

    // A row of the tensor, of which `room` elements are left from the row's start on; elements
    // outside the row read as zero.
    __device__ void load(const T* row, int64_t room, Raw& x) const
    {
        if constexpr (KIND == kWhole) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                x.v[j] = make_uint4(0, 0, 0, 0);
                if (col(j) < width)
                    x.v[j] = *reinterpret_cast<const uint4*>(row + col(j));
            }
        } else if constexpr (KIND == kShort) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                alignas(16) T e[VE];
#pragma unroll
                for (int i = 0; i < VE; ++i)
                    e[i] = col(j) + i < width ? row[col(j) + i] : T(0);
                x.v[j] = *reinterpret_cast<const uint4*>(e);
            }
        } else {
            // the last vector that the row has and the tensor fills; lanes beyond read that one
            const int own = (width - 1) / VE * VE;
            const int last = room < own + VE ? (int)room - VE : own;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = col(j);
                const Access a = *reinterpret_cast<const Access*>(row + (c < last ? c : last));
                x.v[j] = make_uint4(a[0], a[1], a[2], a[3]);
            }
            if (last < own) {                                  // the tensor's last rows
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int by = col(j) - last;
                    if (by > 0 && by < VE) {
                        const unsigned __int128 bits = __builtin_bit_cast(unsigned __int128, x.v[j]);
                        x.v[j] = __builtin_bit_cast(uint4, bits >> (by * (int)sizeof(T) * 8));
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                x.v[j].x &= mask.v[j].x;
                x.v[j].y &= mask.v[j].y;
                x.v[j].z &= mask.v[j].z;
                x.v[j].w &= mask.v[j].w;
            }
        }
    }
    __device__ static void unpack(const Raw& x, float* out)
    {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t w[4] = {x.v[j].x, x.v[j].y, x.v[j].z, x.v[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 2) {
                    out[j * VE + 2 * i] = __uint_as_float(w[i] << 16);
                    out[j * VE + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                } else {
                    out[j * VE + i] = __uint_as_float(w[i]);
                }
            }
        }
    }
    // A vector of weights [width], on its own.
    __device__ void load_weight(const T* w, float* out) const
    {
        Raw x;
        load(w, width, x);
        unpack(x, out);
    }
    __device__ void store(T* row, const float* in) const
    {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = RAGGED ? (j * LANES + opaque(lane)) * VE : col(j);
            if (c >= width)
                continue;
            if (!RAGGED || c + VE <= width) {
                alignas(16) T e[VE];
                Vec16<T>::store(e, in + j * VE);
                const uint4 x = *reinterpret_cast<const uint4*>(e);
                *reinterpret_cast<Access*>(row + c) = Access{x.x, x.y, x.z, x.w};
            } else {
#pragma unroll
                for (int i = 0; i < VE - 1; ++i)
                    if (c + i < width)
                        row[c + i] = from_f32<T>(in[j * VE + i]);
            }
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
template <typename S> __device__ __forceinline__ void store_partial(const S& s, const float* acc, float* buf, float* out)
{
    if constexpr (S::GROUPS == 1) {
#pragma unroll
        for (int j = 0; j < S::NV; ++j)
#pragma unroll
            for (int i = 0; i < S::VE; ++i)
                if (s.col(j) + i < s.width)
                    out[s.col(j) + i] = acc[j * S::VE + i];
    } else {
        constexpr int COLS = S::LANES * S::E;
        const int group = threadIdx.x / S::LANES;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < S::NV; ++j)
#pragma unroll
            for (int i = 0; i < S::VE; ++i)
                buf[group * COLS + s.col(j) + i] = acc[j * S::VE + i];
        __syncthreads();
        for (int c = threadIdx.x; c < s.width; c += S::THREADS) {
            float t = 0.f;
#pragma unroll
            for (int g = 0; g < S::GROUPS; ++g)
                t += buf[g * COLS + c];
            out[c] = t;
        }
    }
}

// The shape for a width, handed to `fn` as its type (in a Tag).  A lane
// holds at most 16 elements (the backward keeps up to seven such arrays in
// registers); a row takes the fewest lanes that this allows, up to a wavefront,
// so that narrow rows (one head) leave no lane idle and need no LDS; wider rows
// take a whole workgroup.
template <typename S> struct Tag { typedef S type; };

template <typename T, Kind KIND, typename Fn> hipError_t pick_shape(int nv, Fn&& fn)
{
    constexpr int NV = 16 / Vec16<T>::N;
    if (nv <= 8) return fn(Tag<Shape<T, KIND, 8, 1>>{});
    if (nv <= 16) return fn(Tag<Shape<T, KIND, 16, 1>>{});
    if (nv <= 32) return fn(Tag<Shape<T, KIND, 32, 1>>{});
    if (nv <= 64) return fn(Tag<Shape<T, KIND, 64, 1>>{});
    if (nv <= 128) return fn(Tag<Shape<T, KIND, 64, 2>>{});
    if constexpr (NV == 4) {
        if (nv <= 192) return fn(Tag<Shape<T, KIND, 64, 3>>{});
        if (nv <= 256) return fn(Tag<Shape<T, KIND, 64, 4>>{});
    }
    if (nv <= 128 * NV) return fn(Tag<Shape<T, KIND, 128, NV>>{});
    if (nv <= 256 * NV) return fn(Tag<Shape<T, KIND, 256, NV>>{});
    return fn(Tag<Shape<T, KIND, 512, NV>>{});
}

template <typename T, typename Fn> hipError_t with_shape(int width, Fn&& fn)
{
    constexpr int VE = Vec16<T>::N;
    if (width % VE == 0)
        return pick_shape<T, kWhole>(width / VE, fn);
    if (width < VE)
        return fn(Tag<Shape<T, kShort, 8, 1>>{});
    return pick_shape<T, kRagged>((width + VE - 1) / VE, fn);
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
