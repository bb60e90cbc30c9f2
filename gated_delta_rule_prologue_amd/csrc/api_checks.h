// api_checks.h -- the argument checks shared by the C ABI's entry points.
#pragma once

#include <stddef.h>
#include <stdint.h>

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

}  // namespace
