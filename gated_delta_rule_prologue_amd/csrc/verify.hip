// verify.hip -- which drafted tokens are kept, and the token that follows them
// (speculative decoding with given random numbers).
//
// Sequence n fed the packed tokens c0..c1-1: the last token it already had,
// then the drafted ones.  Row t of p (and of q) is the target's (the draft
// model's) distribution of the token after token t.  The drafted token x_t,
// t = c0+1.., is kept while
//   u_accept[t] q[t-1, x_t] < p[t-1, x_t]        (q = 1 at x_t without a draft row)
// and every one before it was; n_accept counts the fed tokens that stay, the
// first among them.  The next token is drawn from row t* = c0 + n_accept - 1:
//   w_j = max(p_j - q_j, 0) after a rejection (without q: p_j, but 0 at the rejected
//   token), p_j after the last token;
//   next = the smallest j with w_j > 0 and w_0 + .. + w_j > u_sample (w_0 + .. ),
// so that the kept tokens and the next one together are distributed as the
// target's.  Weights that are not positive and finite count as none; rows of w
// without weight fall back to p, rows of p without weight to token -1.
//
// Products and sums are in 64 bits: u q of two 24-bit values and p - q are then
// exact (or 2^-53 off where exponents differ widely), and sums of 10^5 weights
// hold 2^-50, so the choice does not depend on the order of the additions but
// at a border that near.
//
// Bound by HBM: one row of p and one of q a sequence.  The row is cut into
// chunks of kChunk elements, one workgroup each, so that a single sequence too
// is read by many compute units; the second launch finds the chunk in which the
// sum passes the threshold and walks that one alone.
#include "common.h"
#include "kernels.h"

namespace prism {

namespace {

constexpr int kThreads = 256, kPer = 16, kChunk = kThreads * kPer;

__device__ __forceinline__ double weight_of(double w) { return w > 0. && w < __builtin_inf() ? w : 0.; }

__device__ __forceinline__ double shfl_xor_f64(double x, int m)
{
    const uint64_t b = __double_as_longlong(x);
    const uint32_t lo = __shfl_xor((uint32_t)b, m), hi = __shfl_xor((uint32_t)(b >> 32), m);
    return __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo));
}

__device__ __forceinline__ double shfl_up_f64(double x, int d)
{
    const uint64_t b = __double_as_longlong(x);
    const uint32_t lo = __shfl_up((uint32_t)b, d), hi = __shfl_up((uint32_t)(b >> 32), d);
    return __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo));
}

// Fed tokens that stay, of the len >= 1 at c0; every lane of a wavefront gets
// the count (64 tokens are tested at once).
template <typename T>
__device__ __forceinline__ int kept_tokens(const T* p, const T* q, const int32_t* tokens, const float* u,
                                           int64_t c0, int len, int vocab, int lane)
{
    for (int i = 1; i < len; i += 64) {
        const int t = i + lane;
        bool ok = true;
        if (t < len) {
            const int x = tokens[c0 + t];
            ok = false;
            if (x >= 0 && x < vocab) {
                const int64_t at = (c0 + t - 1) * vocab + x;
                const double px = to_f32(p[at]), qx = q ? to_f32(q[at]) : 1.f;
                ok = (double)u[c0 + t] * qx < px;
            }
        }
        const uint64_t bad = ~__ballot(ok);
        if (bad)
            return i + __ffsll((unsigned long long)bad) - 1;
    }
    return len;
}

// p and w of element i of the row
template <typename T>
__device__ __forceinline__ void weights(T praw, T qraw, bool rejected, bool has_q, bool is_token, double& pw,
                                        double& w)
{
    const double p = to_f32(praw);
    pw = weight_of(p);
    w = pw;
    if (rejected)
        w = has_q ? weight_of(p - (double)to_f32(qraw)) : is_token ? 0. : pw;
}

}  // namespace

// sums [n][chunk][2]: the weights of the chunk, and its p
template <typename T, bool VECTOR>
__global__ __launch_bounds__(kThreads) void verify_sum_kernel(
    const T* __restrict__ p, const T* __restrict__ q, const int32_t* __restrict__ tokens,
    const int32_t* __restrict__ cu, const float* __restrict__ u_accept, int vocab, int chunks,
    int32_t* __restrict__ n_accept, double* __restrict__ sums)
{
    constexpr int VE = VECTOR ? Vec16<T>::N : 1;
    __shared__ double red[2][kThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t n = blockIdx.x / chunks;
    const int chunk = blockIdx.x % chunks;
    const int64_t c0 = cu[n];
    const int len = cu[n + 1] - (int)c0;
    if (len <= 0) {
        if (chunk == 0 && tid == 0)
            n_accept[n] = 0;
        return;
    }
    const int kept = kept_tokens(p, q, tokens, u_accept, c0, len, vocab, lane);
    if (chunk == 0 && tid == 0)
        n_accept[n] = kept;
    const bool rejected = kept < len;
    const int token = rejected ? tokens[c0 + kept] : -1;
    const int64_t row = (c0 + kept - 1) * vocab;
    const bool use_q = rejected && q;

    double sw = 0., sp = 0.;
#pragma unroll
    for (int i = 0; i < kPer / VE; ++i) {
        const int at = chunk * kChunk + (i * kThreads + tid) * VE;
        if (at < vocab) {
            alignas(16) T pv[VE], qv[VE] = {};
            if constexpr (VECTOR) {
                *reinterpret_cast<uint4*>(pv) = *reinterpret_cast<const uint4*>(p + row + at);
                if (use_q)
                    *reinterpret_cast<uint4*>(qv) = *reinterpret_cast<const uint4*>(q + row + at);
            } else {
                pv[0] = p[row + at];
                if (use_q)
                    qv[0] = q[row + at];
            }
#pragma unroll
            for (int x = 0; x < VE; ++x) {
                double pw, w;
                weights(pv[x], qv[x], rejected, q != nullptr, at + x == token, pw, w);
                sw += w;
                sp += pw;
            }
        }
    }
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) {
        sw += shfl_xor_f64(sw, m);
        sp += shfl_xor_f64(sp, m);
    }
    if (lane == 0) {
        red[0][wave] = sw;
        red[1][wave] = sp;
    }
    __syncthreads();
    if (tid < 2) {
        double t = 0.;
        for (int i = 0; i < kThreads / 64; ++i)
            t += red[tid][i];
        sums[(n * chunks + chunk) * 2 + tid] = t;
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void verify_pick_kernel(
    const T* __restrict__ p, const T* __restrict__ q, const int32_t* __restrict__ tokens,
    const int32_t* __restrict__ cu, const float* __restrict__ u_sample, int vocab, int chunks,
    const int32_t* __restrict__ n_accept, const double* __restrict__ sums, int32_t* __restrict__ next_token)
{
    __shared__ double scan[kThreads / 64];
    __shared__ int found[kThreads / 64], last[kThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = blockIdx.x;
    const int64_t c0 = cu[n];
    const int len = cu[n + 1] - (int)c0;
    if (len <= 0) {
        if (tid == 0)
            next_token[n] = -1;
        return;
    }
    const int kept = n_accept[n];
    const double* sn = sums + (int64_t)n * chunks * 2;
    // every wavefront for itself: the totals, then the chunk that passes the threshold
    double tw = 0., tp = 0.;
    for (int c = lane; c < chunks; c += 64) {
        tw += sn[2 * c];
        tp += sn[2 * c + 1];
    }
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) {
        tw += shfl_xor_f64(tw, m);
        tp += shfl_xor_f64(tp, m);
    }
    const bool rejected = kept < len && tw > 0.;         // else the weights are p itself
    const double total = rejected ? tw : tp;
    if (!(total > 0.)) {
        if (tid == 0)
            next_token[n] = -1;
        return;
    }
    const double goal = (double)u_sample[n] * total;
    const int which = rejected ? 0 : 1;
    int chunk = -1, tail = 0;                            // tail: the last chunk with weight
    double before = 0., run = 0.;
    for (int cb = 0; cb < chunks && chunk < 0; cb += 64) {
        const int c = cb + lane;
        const double x = c < chunks ? sn[2 * c + which] : 0.;
        double inc = x;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const double y = shfl_up_f64(inc, d);
            inc += lane >= d ? y : 0.;
        }
        const uint64_t some = __ballot(x > 0.);
        const uint64_t pass = __ballot(x > 0. && run + inc > goal);
        if (some)
            tail = cb + 63 - __clzll((long long)some);
        if (pass) {
            const int at = __ffsll((unsigned long long)pass) - 1;
            chunk = cb + at;
            const double prev = shfl_up_f64(inc, 1);
            const uint64_t bits = __double_as_longlong(run + (lane > 0 ? prev : 0.));
            before = __longlong_as_double(
                (int64_t)((uint64_t)(uint32_t)__shfl((uint32_t)(bits >> 32), at) << 32 |
                          (uint32_t)__shfl((uint32_t)bits, at)));
        } else {
            const uint64_t bits = __double_as_longlong(run + inc);
            run = __longlong_as_double(
                (int64_t)((uint64_t)(uint32_t)__shfl((uint32_t)(bits >> 32), 63) << 32 |
                          (uint32_t)__shfl((uint32_t)bits, 63)));
        }
    }
    const bool passed = chunk >= 0;
    if (!passed)                                         // u_sample near 1 or out of range: the last weight
        chunk = tail;

    // the chunk: thread t holds its elements kPer t .. kPer t + kPer - 1
    const int64_t row = (c0 + kept - 1) * vocab;
    const int token = rejected ? tokens[c0 + kept] : -1;
    const int at = chunk * kChunk + tid * kPer;
    double w[kPer], mine = 0.;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        w[i] = 0.;
        if (at + i < vocab) {
            double pw, ww;
            const T qv = rejected && q ? q[row + at + i] : T(0);
            weights(p[row + at + i], qv, rejected, q != nullptr, at + i == token, pw, ww);
            w[i] = ww;
        }
        mine += w[i];
    }
    double inc = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double y = shfl_up_f64(inc, d);
        inc += lane >= d ? y : 0.;
    }
    if (lane == 63)
        scan[wave] = inc;
    __syncthreads();
    double c = before + (inc - mine);
    for (int i = 0; i < wave; ++i)
        c += scan[i];
    int hit = 0x7fffffff, final_one = -1;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        c += w[i];
        if (w[i] > 0.) {
            final_one = at + i;
            if (passed && hit == 0x7fffffff && c > goal)
                hit = at + i;
        }
    }
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) {
        hit = min(hit, __shfl_xor(hit, m));
        final_one = max(final_one, __shfl_xor(final_one, m));
    }
    if (lane == 0) {
        found[wave] = hit;
        last[wave] = final_one;
    }
    __syncthreads();
    if (tid == 0) {
        for (int i = 1; i < kThreads / 64; ++i) {
            hit = min(hit, found[i]);
            final_one = max(final_one, last[i]);
        }
        // a threshold within rounding of the chunk's end takes the chunk's last weight
        next_token[n] = hit != 0x7fffffff ? hit : final_one;
    }
}

int verify_chunks(int vocab) { return (int)(((int64_t)vocab + kChunk - 1) / kChunk); }

size_t verify_workspace_bytes(int n_seqs, int vocab)
{
    return (size_t)n_seqs * verify_chunks(vocab) * 2 * sizeof(double);
}

template <typename T> static hipError_t launch_T(const VerifyArgs& p, hipStream_t stream)
{
    const int chunks = verify_chunks(p.vocab);
    const dim3 grid((unsigned)((int64_t)chunks * p.n_seqs));
    double* sums = (double*)p.ws;
    if (p.vocab % Vec16<T>::N == 0)                      // every row then starts at a 16-byte address
        hipLaunchKernelGGL((verify_sum_kernel<T, true>), grid, dim3(kThreads), 0, stream, (const T*)p.p,
                           (const T*)p.q, p.tokens, p.cu_seqlens, p.u_accept, p.vocab, chunks, p.n_accept, sums);
    else
        hipLaunchKernelGGL((verify_sum_kernel<T, false>), grid, dim3(kThreads), 0, stream, (const T*)p.p,
                           (const T*)p.q, p.tokens, p.cu_seqlens, p.u_accept, p.vocab, chunks, p.n_accept, sums);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL((verify_pick_kernel<T>), dim3(p.n_seqs), dim3(kThreads), 0, stream, (const T*)p.p,
                       (const T*)p.q, p.tokens, p.cu_seqlens, p.u_sample, p.vocab, chunks, p.n_accept, sums,
                       p.next_token);
    return hipGetLastError();
}

hipError_t launch_verify(const VerifyArgs& p, hipStream_t stream)
{
    return p.bf16 ? launch_T<uint16_t>(p, stream) : launch_T<float>(p, stream);
}

}  // namespace prism
