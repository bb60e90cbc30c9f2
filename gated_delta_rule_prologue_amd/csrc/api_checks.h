// api_checks.h -- the argument checks shared by the C ABI's entry points.
#pragma once

#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include <hip/hip_runtime.h>

#include "prism.h"

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

bool dims_ok(const prism_dims* d)
{
    return d && d->n_seqs >= 1 && d->total_tokens >= 0 && d->heads >= 1 && d->dk >= 1 &&
           d->dv >= 1 && (d->dtype == PRISM_F32 || d->dtype == PRISM_BF16);
}

size_t elem_bytes(const prism_dims* d) { return d->dtype == PRISM_BF16 ? 2 : 4; }

// Pointer must be non-null and 16-byte aligned.
bool ptr_ok(const void* p) { return p && aligned16(p); }

// Per-token arrays may be NULL when there are no tokens at all.
bool tok_ok(const prism_dims* d, const void* p)
{
    return d->total_tokens == 0 ? aligned16(p) : ptr_ok(p);
}

// Optional pointer: null, or 16-byte aligned.
bool opt_ok(const void* p) { return aligned16(p); }

bool residual_ok(int r) { return r == PRISM_RESIDUAL_LINEAR || r == PRISM_RESIDUAL_GELU; }

prism_status from_hip(hipError_t e) { return e == hipSuccess ? PRISM_OK : PRISM_EHIP; }

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

bool eps_ok(float eps) { return eps >= 0.f && isfinite(eps); }

// Strided inputs may begin at any element's address.
bool elem_ok(const void* p, int dtype) { return p && ((uintptr_t)p & (dtype == PRISM_BF16 ? 1u : 3u)) == 0; }

// The bytes of an array that a call reads or writes; `either`: its whole buffer may be
// input and output at once.
struct Region {
    const void* p;
    int64_t bytes;
    bool either = false;
};

// No output shares a byte with an input or another output, but for buffers that may be both.
bool apart(std::initializer_list<Region> outs, std::initializer_list<Region> ins)
{
    auto meet = [](const Region& x, const Region& y) {
        return x.p && y.p && x.bytes > 0 && y.bytes > 0 && (uintptr_t)x.p < (uintptr_t)y.p + y.bytes &&
               (uintptr_t)y.p < (uintptr_t)x.p + x.bytes;
    };
    for (const Region* o = outs.begin(); o != outs.end(); ++o) {
        for (const Region* x = o + 1; x != outs.end(); ++x)
            if (meet(*o, *x))
                return false;
        for (const Region& x : ins)
            if (meet(*o, x) && !(o->either && x.either && o->p == x.p && o->bytes == x.bytes))
                return false;
    }
    return true;
}

int64_t size_of(int dtype) { return dtype == PRISM_BF16 ? 2 : 4; }

// A launch holds less than 2^32 threads in a dimension of its grid.
bool grid_ok(int64_t blocks, int64_t threads) { return blocks <= UINT32_MAX / threads; }

}  // namespace
