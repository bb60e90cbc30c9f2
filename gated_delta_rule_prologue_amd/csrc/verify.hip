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
// Bound by HBM where there are many sequences: one row of p and one of q a sequence; by
// a chain of four dependent reads (offsets, tokens, their probabilities, the row) where
// there are few.  A large row is cut into chunks of kChunk elements, one workgroup each,
// so that a single sequence too is read by many compute units; the second launch finds
// the chunk in which the sum passes the threshold and walks that one alone.  A small
// row takes one workgroup and one launch.  The sums over lanes stay in registers (DPP
// moves of both halves: through LDS exchanges one sequence of 32,000 entries took 12.2
// instead of 9.0 us).  64 sequences of 128,000 entries in fp32, p and q: 65.5 MB in
// 12.5 us of the first launch (5.2 TB/s) and 4.7 of the second, whose start overlaps the first's
// end where calls follow each other (15 us a call); in bf16 9.7 and 4.6 us.
#include "common.h"
#include "kernels.h"

namespace prism {

namespace {

constexpr int kThreads = 256, kPer = 16, kChunk = kThreads * kPer;

__device__ __forceinline__ double weight_of(double w) { return w > 0. && w < __builtin_inf() ? w : 0.; }

// The value of lane `at` (the same for the whole wavefront).
__device__ __forceinline__ double lane_f64(double x, int at)
{
    const uint64_t b = __double_as_longlong(x);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)b, at), hi = __builtin_amdgcn_readlane((uint32_t)(b >> 32), at);
    return __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo));
}

// x plus the value a DPP move brings from another lane (zero where there is none).
template <int CTRL, int ROWS> __device__ __forceinline__ double add_dpp(double x)
{
    const uint64_t b = __double_as_longlong(x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0u, (uint32_t)b, CTRL, ROWS, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0u, (uint32_t)(b >> 32), CTRL, ROWS, 0xF, false);
    return x + __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo));
}

// Inclusive sums over the lanes, within registers: shifts by 1, 2, 4, 8 within rows of 16
// lanes, then the rows' last lanes to the rows behind them.
__device__ __forceinline__ double inclusive_sum(double x)
{
    x = add_dpp<0x111, 0xF>(x);
    x = add_dpp<0x112, 0xF>(x);
    x = add_dpp<0x114, 0xF>(x);
    x = add_dpp<0x118, 0xF>(x);
    x = add_dpp<0x142, 0xA>(x);
    return add_dpp<0x143, 0xC>(x);
}
__device__ __forceinline__ double wave_sum(double x) { return lane_f64(inclusive_sum(x), 63); }

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

// The first of `count` pieces (weight(c) each) at which the running sum exceeds `goal`, and the
// sum before it; -1 if there is none.  `tail`: the last piece with weight.  A wavefront
// works together, 64 pieces at a time.
template <typename F>
__device__ __forceinline__ void find_passing(int count, double goal, int lane, F weight, int& piece, int& tail,
                                             double& before)
{
    double run = 0.;
    for (int cb = 0; cb < count && piece < 0; cb += 64) {
        const int c = cb + lane;
        const double x = c < count ? weight(c) : 0.;
        const double inc = inclusive_sum(x);
        const uint64_t some = __ballot(x > 0.);
        const uint64_t pass = __ballot(x > 0. && run + inc > goal);
        if (some)
            tail = cb + 63 - __clzll((long long)some);
        if (pass) {
            const int at = __ffsll((unsigned long long)pass) - 1;
            piece = cb + at;
            before = at > 0 ? run + lane_f64(inc, at - 1) : run;
        } else {
            run += lane_f64(inc, 63);
        }
    }
}

// A row may start at any element's address (an odd vocabulary), so it is cut from the
// 16-byte address at or below its start: `at` counts from there, less that offset, and
// is negative in front of the row.  Whole vectors inside the row are read as such, the
// two that it only partly fills element by element (zeros outside).
template <typename T> __device__ __forceinline__ int row_offset(int64_t row) { return (int)(row % Vec16<T>::N); }

template <typename T> __device__ __forceinline__ void load_vector(const T* row, int at, int vocab, T* out)
{
    constexpr int VE = Vec16<T>::N;
    if (at >= 0 && at + VE <= vocab) {
        *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(row + at);
    } else {
#pragma unroll
        for (int x = 0; x < VE; ++x)
            out[x] = at + x >= 0 && at + x < vocab ? row[at + x] : T(0);
    }
}

// add(p, q, at) for every vector of a piece: vectors first, first + STRIDE, .. (kPer elements a
// lane), all read before the first is added.  `inside`: the piece lies within the row.
// Otherwise vectors that the row does not fill are read from its first whole one and
// zeroed, and what it holds of them is read element by element (two vectors a row).
template <typename T, int STRIDE, typename F>
__device__ __forceinline__ void read_piece(const T* prow, const T* qrow, bool use_q, bool inside, int first, int off,
                                           int vocab, F add)
{
    constexpr int VE = Vec16<T>::N, NV = kPer / VE;
    alignas(16) T pv[kPer], qv[kPer] = {};
    auto vec = [](const T* at) { return *reinterpret_cast<const uint4*>(at); };
    if (inside) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            *reinterpret_cast<uint4*>(pv + i * VE) = vec(prow + first + i * STRIDE);
            if (use_q)
                *reinterpret_cast<uint4*>(qv + i * VE) = vec(qrow + first + i * STRIDE);
        }
    } else if (vocab >= 2 * VE) {
        const int whole = off ? VE - off : 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = first + i * STRIDE;
            const bool in = at >= 0 && at + VE <= vocab;
            uint4 x = vec(prow + (in ? at : whole)), y = make_uint4(0, 0, 0, 0);
            if (use_q)
                y = vec(qrow + (in ? at : whole));
            *reinterpret_cast<uint4*>(pv + i * VE) = in ? x : make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(qv + i * VE) = in ? y : make_uint4(0, 0, 0, 0);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (inside || vocab >= 2 * VE)
            add(pv + i * VE, qv + i * VE, first + i * STRIDE);
    if (!inside) {
#pragma unroll 1
        for (int i = 0; i < NV; ++i) {
            const int at = first + i * STRIDE;
            const bool part = at > -VE && at < vocab && (at < 0 || at + VE > vocab);
            if (part || (vocab < 2 * VE && at > -VE && at < vocab)) {
                alignas(16) T x[VE], y[VE] = {};
                load_vector(prow, at, vocab, x);
                if (use_q)
                    load_vector(qrow, at, vocab, y);
                add(x, y, at);
            }
        }
    }
}

// The weights of elements at .. at + kPer - 1 of a row (p, less q if it is given, zero at
// `token`), looked at one by one; returns their sum.
template <typename T>
__device__ __forceinline__ double load_weights(const T* p, const T* q, int token, int at, int vocab, double (&w)[kPer])
{
    alignas(16) T pv[kPer], qv[kPer] = {};
#pragma unroll
    for (int i = 0; i < kPer; i += Vec16<T>::N) {
        load_vector(p, at + i, vocab, pv + i);
        if (q)
            load_vector(q, at + i, vocab, qv + i);
    }
    double sum = 0.;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        w[i] = weight_of((double)to_f32(pv[i]) - (double)to_f32(qv[i]));
        if (token >= 0 && at + i == token)
            w[i] = 0.;
        sum += w[i];
    }
    return sum;
}

// The wavefront's first element (kPer a lane, from `at`) with weight at which the running sum
// from c exceeds the goal, and its last one with weight; -1 for none.
__device__ __forceinline__ void pick_element(const double (&w)[kPer], double goal, double c, int at, int& hit, int& end)
{
    int h = -1, l = -1;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        c += w[i];
        if (w[i] > 0.) {
            l = at + i;
            if (h < 0 && c > goal)
                h = at + i;
        }
    }
    const uint64_t hits = __ballot(h >= 0), some = __ballot(l >= 0);
    hit = hits ? __builtin_amdgcn_readlane(h, __ffsll((unsigned long long)hits) - 1) : -1;
    end = some ? __builtin_amdgcn_readlane(l, 63 - __clzll((long long)some)) : -1;
}

}  // namespace

// sums [n][chunk][2]: the weights of the chunk, and its p
template <typename T>
__global__ __launch_bounds__(kThreads) void verify_sum_kernel(
    const T* __restrict__ p, const T* __restrict__ q, const int32_t* __restrict__ tokens,
    const int32_t* __restrict__ cu, const float* __restrict__ u_accept, int vocab, int chunks,
    int32_t* __restrict__ n_accept, double* __restrict__ sums)
{
    constexpr int VE = Vec16<T>::N;
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
    const bool use_q = rejected && q;
    const int token = rejected && !q ? tokens[c0 + kept] : -1;
    const int64_t row = (c0 + kept - 1) * vocab;

    double sw = 0., sp = 0.;
    const int off = row_offset<T>(row), first = chunk * kChunk + tid * VE - off;
    auto add = [&](const T* pv, const T* qv, int at) {
#pragma unroll
        for (int x = 0; x < VE; ++x) {
            const double pw = weight_of(to_f32(pv[x]));
            sp += pw;
            if (use_q)
                sw += weight_of((double)to_f32(pv[x]) - (double)to_f32(qv[x]));
            else
                sw += token >= 0 && at + x == token ? 0. : pw;
        }
    };
    read_piece<T, kThreads * VE>(p + row, q + row, use_q, chunk * kChunk >= off && (chunk + 1) * kChunk - off <= vocab,
                                 first, off, vocab, add);
    sw = wave_sum(sw);
    sp = wave_sum(sp);
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
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t n = blockIdx.x;
    const int64_t c0 = cu[n];
    const int len = cu[n + 1] - (int)c0;
    if (len <= 0) {
        if (tid == 0)
            next_token[n] = -1;
        return;
    }
    const int kept = n_accept[n];
    const double* sn = sums + n * chunks * 2;
    // every wavefront for itself: the totals, then the chunk that passes the threshold
    double tw = 0., tp = 0.;
    for (int c = lane; c < chunks; c += 64) {
        tw += sn[2 * c];
        tp += sn[2 * c + 1];
    }
    tw = wave_sum(tw);
    tp = wave_sum(tp);
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
    double before = 0.;
    find_passing(chunks, goal, lane, [&](int c) { return sn[2 * c + which]; }, chunk, tail, before);
    const bool passed = chunk >= 0;
    if (!passed)                                         // u_sample near 1 or out of range: the last weight
        chunk = tail;

    // the chunk: thread t holds kPer consecutive elements
    __shared__ double scan[kThreads / 64];
    __shared__ int found[kThreads / 64], last[kThreads / 64];
    const int64_t row = (c0 + kept - 1) * vocab;
    const int token = rejected && !q ? tokens[c0 + kept] : -1;
    const int at = chunk * kChunk + tid * kPer - row_offset<T>(row);
    double w[kPer];
    const double mine = load_weights<T>(p + row, rejected && q ? q + row : nullptr, token, at, vocab, w);
    const double inc = inclusive_sum(mine);
    if (lane == 63)
        scan[wave] = inc;
    __syncthreads();
    double c = before + (inc - mine);
    for (int i = 0; i < wave; ++i)
        c += scan[i];
    int hit, end;
    pick_element(w, passed ? goal : __builtin_inf(), c, at, hit, end);
    if (lane == 0) {
        found[wave] = hit;
        last[wave] = end;
    }
    __syncthreads();
    if (tid == 0) {
        for (int i = kThreads / 64 - 1; i >= 0; --i) {
            hit = found[i] >= 0 ? found[i] : hit;
            end = max(end, last[i]);
        }
        // a threshold within rounding of the chunk's end takes the chunk's last weight
        next_token[n] = hit >= 0 ? hit : end;
    }
}

// One workgroup a sequence, in one launch: the row's sums by pieces of kPiece elements (a
// wavefront each) in LDS, then the piece in which the threshold is passed, walked by
// one wavefront.  The fast sum takes max(w, 0), which drops negative weights and NaN;
// an infinite weight shows in its total, and then (as where the total is empty) the
// sums are taken again with every weight looked at.
constexpr int kRowThreads = 1024, kPiece = 64 * kPer;

template <typename T>
__global__ __launch_bounds__(kRowThreads) void verify_row_kernel(
    const T* __restrict__ p, const T* __restrict__ q, const int32_t* __restrict__ tokens,
    const int32_t* __restrict__ cu, const float* __restrict__ u_accept, const float* __restrict__ u_sample, int vocab,
    int32_t* __restrict__ n_accept, int32_t* __restrict__ next_token)
{
    constexpr int VE = Vec16<T>::N, WAVES = kRowThreads / 64;
    extern __shared__ double sums[];                     // a piece's weight
    __shared__ double total_of[WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t n = blockIdx.x;
    const int64_t c0 = cu[n];
    const int len = cu[n + 1] - (int)c0;
    if (len <= 0) {
        if (tid == 0) {
            n_accept[n] = 0;
            next_token[n] = -1;
        }
        return;
    }
    const int kept = kept_tokens(p, q, tokens, u_accept, c0, len, vocab, lane);
    if (tid == 0)
        n_accept[n] = kept;
    const int64_t row = (c0 + kept - 1) * vocab;
    const T *prow = p + row, *qrow = q + row;
    const int off = row_offset<T>(row), pieces = (vocab + off + kPiece - 1) / kPiece;

    // 0: max(w, 0); 1: w, every weight looked at; 2: p, likewise
    bool rejected = kept < len;
    double total = 0.;
    for (int mode = 0; mode < 3; ++mode) {
        if (mode == 2)
            rejected = false;
        const int token = rejected && !q ? tokens[c0 + kept] : -1;
        double mine = 0.;
        for (int pc = wave; pc < pieces; pc += WAVES) {
            double acc = 0.;
            const int first = pc * kPiece + lane * VE - off;
            auto add = [&](const T* pv, const T* qv, int at) {
#pragma unroll
                for (int x = 0; x < VE; ++x) {
                    double w = to_f32(pv[x]);
                    if (rejected && q)
                        w -= (double)to_f32(qv[x]);
                    w = fmax(w, 0.);
                    if (mode > 0)
                        w = weight_of(w);
                    if (token >= 0 && at + x == token)
                        w = 0.;
                    acc += w;
                }
            };
            read_piece<T, 64 * VE>(prow, qrow, rejected && q, pc * kPiece >= off && (pc + 1) * kPiece - off <= vocab,
                                   first, off, vocab, add);
            acc = wave_sum(acc);
            if (lane == 0)
                sums[pc] = acc;
            mine += acc;
        }
        if (lane == 0)
            total_of[wave] = mine;
        __syncthreads();
        total = 0.;
        for (int i = 0; i < WAVES; ++i)
            total += total_of[i];
        if (total > 0. && total < __builtin_inf())
            break;
        if (!rejected && mode > 0)
            break;
        __syncthreads();
    }
    if (wave > 0)
        return;
    if (!(total > 0.)) {
        if (lane == 0)
            next_token[n] = -1;
        return;
    }
    const double goal = (double)u_sample[n] * total;
    int piece = -1, tail = 0;                            // tail: the last piece with weight
    double before = 0.;
    find_passing(pieces, goal, lane, [&](int c) { return sums[c]; }, piece, tail, before);
    const bool passed = piece >= 0;
    if (!passed)                                         // u_sample near 1 or out of range: the last weight
        piece = tail;
    // lane l holds kPer consecutive elements of the piece
    const int token = rejected && !q ? tokens[c0 + kept] : -1;
    const int at = piece * kPiece + lane * kPer - off;
    double w[kPer];
    const double mine = load_weights<T>(prow, rejected && q ? qrow : nullptr, token, at, vocab, w);
    int hit, end;
    pick_element(w, passed ? goal : __builtin_inf(), before + (inclusive_sum(mine) - mine), at, hit, end);
    // a threshold within rounding of the piece's end takes the piece's last weight
    if (lane == 0)
        next_token[n] = hit >= 0 ? hit : end;
}

// chunks of a row, whatever its offset
int verify_chunks(int vocab) { return (int)(((int64_t)vocab + 7 + kChunk - 1) / kChunk); }

// One launch up to this vocabulary, two beyond (see verify_row_kernel).  One sequence of
// 5 tokens, fp32, one launch against two: 8.9 against 8.0 us at 32,000 entries on the
// GPU, but 9.0 against 9.9 us with the host's part, and 5.5 against 7.5 us at 4,096;
// 26 against 8.2 us at 128,000, where one compute unit alone reads the row.  256
// sequences of 32,000: 17.8 against 19.6 us.
constexpr int kRowVocab = 32768;

bool verify_in_rows(int vocab) { return vocab <= kRowVocab; }

size_t verify_workspace_bytes(int n_seqs, int vocab)
{
    return verify_in_rows(vocab) ? 0 : (size_t)n_seqs * verify_chunks(vocab) * 2 * sizeof(double);
}

template <typename T> static hipError_t launch_T(const VerifyArgs& p, hipStream_t stream)
{
    if (verify_in_rows(p.vocab)) {
        const size_t lds = (((size_t)p.vocab + 7 + kPiece - 1) / kPiece) * sizeof(double);
        hipLaunchKernelGGL((verify_row_kernel<T>), dim3(p.n_seqs), dim3(kRowThreads), lds, stream, (const T*)p.p,
                           (const T*)p.q, p.tokens, p.cu_seqlens, p.u_accept, p.u_sample, p.vocab, p.n_accept,
                           p.next_token);
        return hipGetLastError();
    }
    const int chunks = verify_chunks(p.vocab);
    double* sums = (double*)p.ws;
    hipLaunchKernelGGL((verify_sum_kernel<T>), dim3((unsigned)((int64_t)chunks * p.n_seqs)), dim3(kThreads), 0, stream,
                       (const T*)p.p, (const T*)p.q, p.tokens, p.cu_seqlens, p.u_accept, p.vocab, chunks, p.n_accept,
                       sums);
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
