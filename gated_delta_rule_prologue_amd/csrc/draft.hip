// draft.hip -- the operator over the few drafted tokens of every sequence, from
// a carried state that stays as it is, and the state's move by the tokens that
// were kept (speculative decoding: a recurrent state cannot be rolled back, so
// it is only moved once it is known how far).
//
// Per (sequence, head) chain and drafted tokens t = 0..M-1 (at most 16 at a
// time; more are walked in blocks of 16), with S the carried state and
//   kw_t = the write key of the operator (ShortConv anchor, residual chain),
//   p_t  = S_{t-1}^T k_t,
//   S_t  = g_t (S_{t-1} - b_t k_t p_t^T) + kw_t v_t^T,   o_t = S_t^T q_t:
// unrolled over the block, with rho(i, j) = prod_{l=j+1..i} g_l and gamma_i the
// product of the gates 0..i,
//   S_i  = gamma_i S - sum_{j<=i} rho(i, j) g_j b_j k_j p_j^T + sum_{j<=i} rho(i, j) kw_j v_j^T
// so that P (the rows p_t) solves a unit lower triangular system:
//   (I + A) P = diag(gamma_{i-1}) K S + B V
//   O         = diag(gamma_i) Q S - C P + E V
//   A_ij = rho(i-1, j) g_j b_j <k_j, k_i>, B_ij = rho(i-1, j) <kw_j, k_i>   (j < i)
//   C_ij = rho(i, j) g_j b_j <k_j, q_i>,   E_ij = rho(i, j) <kw_j, q_i>     (j <= i)
// The products of gates are formed directly (never a quotient), so a gate of
// exactly zero is served.  kw and p are left as records, in fp32, from which
// the commit moves the state by m kept tokens without solving anything:
//   S' = gamma_{m-1} S + sum_{j<m} k_j x_j^T + kw_j y_j^T,
//   x_j = -rho(m-1, j) g_j b_j p_j,  y_j = rho(m-1, j) v_j.
// PRISM pages: WeChat ICML 2026 summary, sections 核心迭代形式, 消除 Token 间串行
// and 消除 Step 间串行; gist.science summary of arXiv 2602.10796, section 2.1
// (S_t = S_{t-1} A_t + B_t: moving by any prefix is exact).
//
// Bound by HBM: the fp32 state is read once (and written once by the commit);
// the products cost 4 M dk dv flops a chain, which run on the fp32 matrix
// instructions (16x16x4) under the loads of other workgroups.
//
// Layout.  One workgroup per chain, one wavefront per 32 value columns, the
// state in registers: lane (kq, j) = (lane / 16, lane % 16) holds rows
// 16 R + 4 kq + r and the columns 2 j, 2 j + 1 of its wavefront, so a row of
// the tile is read in 128-byte pieces.  That is the accumulator layout of a
// 16x16 tile and, register r taken as one 16x16x4 step whose contraction index
// kq names row 4 kq + r, the second operand's too: S enters K S and receives
// K^T X with no exchange between lanes.  The first operand of step r then
// wants channel 4 kq + r, so one 16-byte LDS read serves four steps.  The same
// holds for P, which comes out of one product and enters the next.
// Token t sits in tile row 4 (t % 4) + t / 4: step r of a contraction over
// tokens covers tokens 4 r .. 4 r + 3, so steps beyond the last token are left
// out.
#include "common.h"
#include "kernels.h"

namespace prism {

namespace {

constexpr int kBlock = 16;                       // tokens per pass, at most
constexpr float kLarge = 1073741824.f;           // 2^30

__device__ __forceinline__ f32x4_t mfma4(float a, float b, f32x4_t c)
{
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// tile row of a token and back (its own inverse)
__device__ __forceinline__ int slot_of(int t) { return 4 * (t & 3) + (t >> 2); }

__device__ __forceinline__ float2 load2(const uint16_t* p)
{
    const uint32_t x = *reinterpret_cast<const uint32_t*>(p);
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
__device__ __forceinline__ float2 load2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ void store2(uint16_t* p, float a, float b)
{
    *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(a, b);
}
__device__ __forceinline__ void store2(float* p, float a, float b)
{
    *reinterpret_cast<float2*>(p) = make_float2(a, b);
}

typedef __attribute__((ext_vector_type(2))) float f32x2_t;

// S += K^T X + KW^T Y of one block, with the rows of K and KW (fp32, [slot][LD]) in LDS; `steps` = ceil(tokens / 4)
template <int RT, int LD>
__device__ __forceinline__ void add_tokens(f32x4_t (&s)[RT][2], const float* sK, const float* sKW, int steps,
                                           int kq, int j, const f32x4_t (&x)[2],
                                           const f32x4_t (&y)[2])
{
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        if (r < steps) {
#pragma unroll
            for (int R = 0; R < RT; ++R) {
                const int at = (4 * kq + r) * LD + 16 * R + j;
                const float ka = sK[at], kwa = sKW[at];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    s[R][c] = mfma4(ka, x[c][r], s[R][c]);
                    s[R][c] = mfma4(kwa, y[c][r], s[R][c]);
                }
            }
        }
    }
}

}  // namespace

template <typename T, int DK, int DV>
__global__ __launch_bounds__(2 * DV) void draft_kernel(
    const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, const T* __restrict__ u,
    const T* __restrict__ a, const T* __restrict__ h, const T* __restrict__ g, const T* __restrict__ b,
    const T* __restrict__ conv_w, const int32_t* __restrict__ cu, int H, int L, bool gelu,
    const float* __restrict__ S, const T* __restrict__ k_hist, T* __restrict__ o, float* __restrict__ kw_out,
    float* __restrict__ p_out)
{
    constexpr int NTH = 2 * DV, W = NTH / 64, RT = DK / 16, LD = DK + 4;
    constexpr int VE = Vec16<T>::N, CG = DK / VE;        // channels per access, accesses per row
    __shared__ __align__(16) float sK[kBlock * LD], sQ[kBlock * LD], sKW[kBlock * LD];
    __shared__ __align__(16) float sM[4][16][20];        // A (then its inverse), B, -C, E by tile row
    __shared__ __align__(16) float sG[kBlock];
    __shared__ float sB[kBlock], sRho[kBlock][kBlock + 1], sGam[kBlock + 1];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, kq = lane >> 4, j = lane & 15;
    const int64_t chain = blockIdx.x;
    const int e = (int)(chain % H);
    const int64_t n = chain / H;
    const int64_t c0 = cu[n];
    const int len = cu[n + 1] - (int)c0;
    if (len <= 0)
        return;

    f32x4_t s[RT][2];
    const float* Sc = S + chain * DK * DV + 32 * wave + 2 * j;
#pragma unroll
    for (int R = 0; R < RT; ++R)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const f32x2_t x = __builtin_nontemporal_load(
                reinterpret_cast<const f32x2_t*>(Sc + (16 * R + 4 * kq + r) * DV));
            s[R][0][r] = x[0];
            s[R][1][r] = x[1];
        }

    // A token's zeros in the triangular matrices would turn an infinity or a NaN
    // of a later token into a NaN of its own, so a sequence with a value beyond
    // kLarge (whose products may overflow too) takes its tokens one at a time.
    int cap = kBlock;
    for (int base = 0; base < len;) {
        const int m = len - base < cap ? len - base : cap;
        const int steps = (m + 3) >> 2;
        bool tame = true;
        if (base > 0)
            __syncthreads();                             // the block before is done with the LDS
        if (tid < kBlock) {
            const bool on = tid < m;
            const int64_t at = (c0 + base + tid) * H + e;
            const float gt = on ? to_f32(g[at]) : 1.f, bt = on ? to_f32(b[at]) : 0.f;
            sG[tid] = gt;
            sB[tid] = bt;
            tame = fabsf(gt) <= kLarge && fabsf(bt) <= kLarge;
        }
        // write keys: one thread per (token, VE channels)
        for (int i = tid; i < kBlock * CG; i += NTH) {
            const int t = i / CG, ch = (i % CG) * VE, to = slot_of(t) * LD + ch;
            float kt[VE], qt[VE], acc[VE];
#pragma unroll
            for (int x = 0; x < VE; ++x)
                kt[x] = qt[x] = acc[x] = 0.f;
            if (t < m) {
                const int64_t row = (c0 + base + t) * H + e;
                Vec16<T>::load(k + row * DK + ch, kt);
                Vec16<T>::load(q + row * DK + ch, qt);
                float past[3][VE], w[4 * VE];
#pragma unroll
                for (int d = 1; d <= 3; ++d) {
                    const int pos = base + t - d;
                    Vec16<T>::load(pos >= 0 ? k + (row - (int64_t)d * H) * DK + ch
                                            : k_hist + (chain * 3 + 3 + pos) * DK + ch, past[d - 1]);
                }
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    Vec16<T>::load(conv_w + ((int64_t)e * DK + ch) * 4 + x * VE, w + x * VE);
                const float bt = to_f32(b[row]);
                float r[VE];
#pragma unroll
                for (int x = 0; x < VE; ++x) {
                    r[x] = w[4 * x + 3] * kt[x] + w[4 * x + 2] * past[0][x] + w[4 * x + 1] * past[1][x] +
                           w[4 * x] * past[2][x];
                    acc[x] = bt * kt[x];
                }
                const int64_t lev = row * (L - 1) * DK + ch;
#pragma unroll 2
                for (int l = 0; l < L - 1; ++l) {
                    float av[VE], uv[VE], hv[VE];
                    Vec16<T>::load(a + lev + (int64_t)l * DK, av);
                    Vec16<T>::load(u + lev + (int64_t)l * DK, uv);
                    const bool more = l < L - 2;
                    if (more)
                        Vec16<T>::load(h + lev + (int64_t)l * DK, hv);
#pragma unroll
                    for (int x = 0; x < VE; ++x) {
                        acc[x] += av[x] * r[x] * uv[x];
                        if (more)
                            r[x] = gelu ? r[x] - av[x] * gelu_as(hv[x] * r[x]) : r[x] * (1.f - av[x] * hv[x]);
                    }
                }
#pragma unroll
                for (int x = 0; x < VE; x += 4)
                    *reinterpret_cast<f32x4_t*>(kw_out + row * DK + ch + x) =
                        f32x4_t{acc[x], acc[x + 1], acc[x + 2], acc[x + 3]};
            }
#pragma unroll
            for (int x = 0; x < VE; x += 4) {
                *reinterpret_cast<f32x4_t*>(sK + to + x) = f32x4_t{kt[x], kt[x + 1], kt[x + 2], kt[x + 3]};
                *reinterpret_cast<f32x4_t*>(sQ + to + x) = f32x4_t{qt[x], qt[x + 1], qt[x + 2], qt[x + 3]};
                *reinterpret_cast<f32x4_t*>(sKW + to + x) = f32x4_t{acc[x], acc[x + 1], acc[x + 2], acc[x + 3]};
            }
#pragma unroll
            for (int x = 0; x < VE; ++x)
                tame = tame && fabsf(kt[x]) <= kLarge && fabsf(acc[x]) <= kLarge;
        }
        // value rows: register r holds token 4 r + kq, both columns
        f32x4_t vv[2] = {};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = 4 * r + kq;
            if (t < m) {
                const float2 x = load2(v + ((c0 + base + t) * H + e) * DV + 32 * wave + 2 * j);
                vv[0][r] = x.x;
                vv[1][r] = x.y;
                tame = tame && fabsf(x.x) <= kLarge && fabsf(x.y) <= kLarge;
            }
        }
        if (__syncthreads_or(!tame) && cap > 1) {
            cap = 1;
            continue;
        }
        // products of gates: thread t takes column t of rho
        if (tid < kBlock) {
            float gg[kBlock], x = 1.f, gam = 1.f;
#pragma unroll
            for (int i = 0; i < kBlock; i += 4)
                *reinterpret_cast<f32x4_t*>(gg + i) = *reinterpret_cast<const f32x4_t*>(sG + i);
#pragma unroll
            for (int i = 0; i < kBlock; ++i) {
                x = i > tid ? x * gg[i] : 1.f;
                gam = i < tid ? gam * gg[i] : gam;
                sRho[i][tid] = x;                        // rho(i, tid); 1 up to i = tid
            }
            sGam[tid] = gam;                             // the product of the gates before tid
            if (tid == kBlock - 1)
                sGam[kBlock] = gam * gg[kBlock - 1];
        }
        __syncthreads();
        // the four products of tokens with tokens, 4 / W of them a wavefront
#pragma unroll
        for (int x = 0; x < 4 / W; ++x) {
            const int mat = wave + x * W;                // K K^T, K KW^T, Q K^T, Q KW^T
            const float* pa = (mat < 2 ? sK : sQ) + j * LD + 4 * kq;
            const float* pb = (mat & 1 ? sKW : sK) + j * LD + 4 * kq;
            f32x4_t d0 = {}, d1 = {};
#pragma unroll
            for (int R = 0; R < RT; ++R) {
                const f32x4_t fa = *reinterpret_cast<const f32x4_t*>(pa + 16 * R);
                const f32x4_t fb = *reinterpret_cast<const f32x4_t*>(pb + 16 * R);
                d0 = mfma4(fa[0], fb[0], d0);
                d1 = mfma4(fa[1], fb[1], d1);
                d0 = mfma4(fa[2], fb[2], d0);
                d1 = mfma4(fa[3], fb[3], d1);
            }
            d0 += d1;
            const int tj = slot_of(j);
            const float gb = sG[tj] * sB[tj];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int ti = 4 * r + kq;               // the token of tile row 4 kq + r
                float x = 0.f;                           // selected, not scaled: later tokens may be infinite
                if (mat < 2 && tj < ti && ti < m)
                    x = sRho[ti - 1][tj] * (mat == 0 ? gb : 1.f) * d0[r];
                if (mat >= 2 && tj <= ti && ti < m)
                    x = sRho[ti][tj] * (mat == 2 ? -gb : 1.f) * d0[r];
                sM[mat][4 * kq + r][j] = x;
            }
        }
        __syncthreads();
        // (I + A)^-1, one column a lane, by substitution over the tokens
        if (tid < kBlock) {
            float col[kBlock];
#pragma unroll
            for (int i = 0; i < kBlock; ++i) {
                float row[kBlock];                       // A's row of token i, by tile column
#pragma unroll
                for (int l = 0; l < kBlock; l += 4)
                    *reinterpret_cast<f32x4_t*>(row + l) =
                        *reinterpret_cast<const f32x4_t*>(&sM[0][slot_of(i)][l]);
                float x = i == tid ? 1.f : 0.f;
#pragma unroll
                for (int l = 0; l < i; ++l)
                    x -= row[slot_of(l)] * col[l];
                col[i] = x;
            }
            __builtin_amdgcn_wave_barrier();             // every lane has read A
#pragma unroll
            for (int i = 0; i < kBlock; ++i)
                sM[0][slot_of(i)][slot_of(tid)] = col[i];
        }
        // K S and Q S
        f32x4_t ks[2] = {}, qs[2] = {};
#pragma unroll
        for (int R = 0; R < RT; ++R) {
            const f32x4_t fk = *reinterpret_cast<const f32x4_t*>(sK + j * LD + 16 * R + 4 * kq);
            const f32x4_t fq = *reinterpret_cast<const f32x4_t*>(sQ + j * LD + 16 * R + 4 * kq);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    ks[c] = mfma4(fk[r], s[R][c][r], ks[c]);
                    qs[c] = mfma4(fq[r], s[R][c][r], qs[c]);
                }
        }
        __syncthreads();
        f32x4_t pp[2] = {};
        {
            const f32x4_t fb = *reinterpret_cast<const f32x4_t*>(&sM[1][j][4 * kq]);
            const f32x4_t ft = *reinterpret_cast<const f32x4_t*>(&sM[0][j][4 * kq]);
            const f32x4_t fc = *reinterpret_cast<const f32x4_t*>(&sM[2][j][4 * kq]);
            const f32x4_t fe = *reinterpret_cast<const f32x4_t*>(&sM[3][j][4 * kq]);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    ks[c][r] *= sGam[4 * r + kq];
                    qs[c][r] *= sGam[4 * r + kq + 1];
                }
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (r < steps)
                        ks[c] = mfma4(fb[r], vv[c][r], ks[c]);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (r < steps)
                        pp[c] = mfma4(ft[r], ks[c][r], pp[c]);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (r < steps) {
                        qs[c] = mfma4(fc[r], pp[c][r], qs[c]);
                        qs[c] = mfma4(fe[r], vv[c][r], qs[c]);
                    }
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = 4 * r + kq;
            if (t < m) {
                const int64_t at = ((c0 + base + t) * H + e) * DV + 32 * wave + 2 * j;
                store2(o + at, qs[0][r], qs[1][r]);
                store2(p_out + at, pp[0][r], pp[1][r]);
            }
        }
        if (base + m < len) {                            // the state enters the next block
            const float gam = sGam[kBlock];
            f32x4_t x[2], y[2];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = 4 * r + kq;
                const float rho = sRho[kBlock - 1][t], gb = -rho * sG[t] * sB[t];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    x[c][r] = t < m ? gb * pp[c][r] : 0.f;
                    y[c][r] = rho * vv[c][r];
                }
            }
#pragma unroll
            for (int R = 0; R < RT; ++R)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    s[R][c] *= gam;
            add_tokens<RT, LD>(s, sK, sKW, steps, kq, j, x, y);
        }
        base += m;
    }
}

// S_out and hist_out may be S and hist: a thread has read what it overwrites.
// blockIdx.y is a band of DK / gridDim.y state rows.
template <typename T, int DK, int DV, int ROWS>
__global__ __launch_bounds__(2 * DV) void commit_kernel(
    const T* __restrict__ k, const T* __restrict__ v, const T* __restrict__ g, const T* __restrict__ b,
    const int32_t* __restrict__ cu, const int32_t* __restrict__ n_accept, int H,
    const float* __restrict__ kw, const float* __restrict__ p, const float* S, const T* hist, float* S_out,
    T* hist_out)
{
    constexpr int NTH = 2 * DV, RT = ROWS / 16, LD = ROWS + 4;
    constexpr int VE = Vec16<T>::N;
    __shared__ __align__(16) float sK[kBlock * LD], sKW[kBlock * LD];
    __shared__ float sG[kBlock], sB[kBlock], sRho[kBlock + 1];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, kq = lane >> 4, j = lane & 15;
    const int64_t chain = blockIdx.x;
    const int e = (int)(chain % H), row0 = blockIdx.y * ROWS;
    const int64_t n = chain / H;
    const int64_t c0 = cu[n];
    int len = cu[n + 1] - (int)c0;
    const int acc = n_accept[n];
    len = acc < len ? acc : len;                         // the tokens kept
    len = len < 0 ? 0 : len;
    if (len == 0 && S_out == S && hist_out == hist)
        return;

    f32x4_t s[RT][2];
    const int64_t at0 = (chain * DK + row0) * DV + 32 * wave + 2 * j;
#pragma unroll
    for (int R = 0; R < RT; ++R)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const f32x2_t x = __builtin_nontemporal_load(
                reinterpret_cast<const f32x2_t*>(S + at0 + (16 * R + 4 * kq + r) * DV));
            s[R][0][r] = x[0];
            s[R][1][r] = x[1];
        }
    // the history's move: the last three of (history, kept tokens)
    if (blockIdx.y == 0 && tid < DK) {
        T x[3];
#pragma unroll
        for (int d = 0; d < 3; ++d) {
            const int pos = len - 3 + d;                 // position of the row, from the first new token
            x[d] = pos >= 0 ? k[((c0 + pos) * H + e) * DK + tid] : hist[(chain * 3 + 3 + pos) * DK + tid];
        }
#pragma unroll
        for (int d = 0; d < 3; ++d)
            hist_out[(chain * 3 + d) * DK + tid] = x[d];
    }

    for (int base = 0; base < len; base += kBlock) {
        const int m = len - base < kBlock ? len - base : kBlock;
        const int steps = (m + 3) >> 2;
        if (base > 0)
            __syncthreads();
        if (tid < kBlock) {
            const bool on = tid < m;
            const int64_t at = (c0 + base + tid) * H + e;
            sG[tid] = on ? to_f32(g[at]) : 1.f;
            sB[tid] = on ? to_f32(b[at]) : 0.f;
        }
        for (int i = tid; i < 4 * steps * (ROWS / VE); i += NTH) {
            const int t = i / (ROWS / VE), ch = (i % (ROWS / VE)) * VE, to = slot_of(t) * LD + ch;
            float kt[VE], wt[VE];
#pragma unroll
            for (int x = 0; x < VE; ++x)
                kt[x] = wt[x] = 0.f;
            if (t < m) {
                const int64_t at = ((c0 + base + t) * H + e) * DK + row0 + ch;
                Vec16<T>::load(k + at, kt);
#pragma unroll
                for (int x = 0; x < VE; x += 4)
                    Vec16<float>::load(kw + at + x, wt + x);
            }
#pragma unroll
            for (int x = 0; x < VE; x += 4) {
                *reinterpret_cast<f32x4_t*>(sK + to + x) = f32x4_t{kt[x], kt[x + 1], kt[x + 2], kt[x + 3]};
                *reinterpret_cast<f32x4_t*>(sKW + to + x) = f32x4_t{wt[x], wt[x + 1], wt[x + 2], wt[x + 3]};
            }
        }
        f32x4_t x[2] = {}, y[2] = {};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = 4 * r + kq;
            if (t < m) {
                const int64_t at = ((c0 + base + t) * H + e) * DV + 32 * wave + 2 * j;
                const float2 pv = load2(p + at), vv = load2(v + at);
                x[0][r] = pv.x; x[1][r] = pv.y;
                y[0][r] = vv.x; y[1][r] = vv.y;
            }
        }
        __syncthreads();
        if (tid <= kBlock) {                             // the product of the gates tid..m-1
            float f = 1.f;
            for (int i = tid; i < kBlock; ++i)
                f *= sG[i];
            sRho[tid] = f;
        }
        __syncthreads();
        const float gam = sRho[0];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = 4 * r + kq;
            const float fx = -sRho[t] * sB[t], fy = sRho[t + 1];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                x[c][r] *= fx;
                y[c][r] *= fy;
            }
        }
#pragma unroll
        for (int R = 0; R < RT; ++R)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                s[R][c] *= gam;
        add_tokens<RT, LD>(s, sK, sKW, steps, kq, j, x, y);
    }
#pragma unroll
    for (int R = 0; R < RT; ++R)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const f32x2_t x = {s[R][0][r], s[R][1][r]};
            __builtin_nontemporal_store(
                x, reinterpret_cast<f32x2_t*>(S_out + at0 + (16 * R + 4 * kq + r) * DV));
        }
}

template <typename T, int DK, int DV>
static hipError_t launch_draft_t(const DraftArgs& p, hipStream_t stream)
{
    hipLaunchKernelGGL((draft_kernel<T, DK, DV>), dim3((unsigned)((int64_t)p.n_seqs * p.heads)), dim3(2 * DV), 0,
                       stream, (const T*)p.q, (const T*)p.k, (const T*)p.v, (const T*)p.u, (const T*)p.a,
                       (const T*)p.h, (const T*)p.g, (const T*)p.b, (const T*)p.conv_w, p.cu_seqlens, p.heads,
                       p.L, p.gelu, p.S, (const T*)p.k_hist, (T*)p.o, p.kw, p.p);
    return hipGetLastError();
}

template <typename T, int DK, int DV>
static hipError_t launch_commit_t(const DraftArgs& p, hipStream_t stream)
{
    hipLaunchKernelGGL((commit_kernel<T, DK, DV, DK>), dim3((unsigned)((int64_t)p.n_seqs * p.heads)),
                       dim3(2 * DV), 0, stream, (const T*)p.k, (const T*)p.v, (const T*)p.g, (const T*)p.b,
                       p.cu_seqlens, p.n_accept, p.heads, p.kw, p.p, p.S, (const T*)p.k_hist, p.S_out,
                       (T*)p.k_hist_out);
    return hipGetLastError();
}

template <typename T> static hipError_t launch_T(const DraftArgs& p, bool commit, hipStream_t s)
{
    if (p.dk == 64 && p.dv == 64)
        return commit ? launch_commit_t<T, 64, 64>(p, s) : launch_draft_t<T, 64, 64>(p, s);
    if (p.dk == 64 && p.dv == 128)
        return commit ? launch_commit_t<T, 64, 128>(p, s) : launch_draft_t<T, 64, 128>(p, s);
    if (p.dk == 128 && p.dv == 64)
        return commit ? launch_commit_t<T, 128, 64>(p, s) : launch_draft_t<T, 128, 64>(p, s);
    return commit ? launch_commit_t<T, 128, 128>(p, s) : launch_draft_t<T, 128, 128>(p, s);
}

hipError_t launch_draft(const DraftArgs& p, hipStream_t stream)
{
    if (!decode_supported(p.dk, p.dv) || p.L < 1)
        return hipErrorInvalidValue;
    return p.bf16 ? launch_T<uint16_t>(p, false, stream) : launch_T<float>(p, false, stream);
}

hipError_t launch_commit(const DraftArgs& p, hipStream_t stream)
{
    if (!decode_supported(p.dk, p.dv))
        return hipErrorInvalidValue;
    return p.bf16 ? launch_T<uint16_t>(p, true, stream) : launch_T<float>(p, true, stream);
}

}  // namespace prism
