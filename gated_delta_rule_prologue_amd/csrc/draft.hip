// draft.hip -- the operator over the few drafted tokens of every sequence, from
// a carried state that stays as it is, and the state's move by the tokens that
// were kept (speculative decoding: a recurrent state cannot be rolled back, so
// it is only moved once it is known how far).
//
// Per (sequence, head) chain and drafted tokens t = 0..M-1 (at most 8 at a
// time; more are walked in blocks of 8), with S the carried state and
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
// With T = (I + A)^-1 and the rows of K and Q stacked,
//   [XP; XO] = [gamma K S; gamma Q S] + [B; E] V,   [P; O] = [0; XO] + W XP,   W = [T; -C T]:
// a row of Q is added to its own output and enters no product with the others', whose zeros
// would make a query that is not finite a NaN of every token.
// The products of gates are formed directly (never a quotient), so a gate of
// exactly zero is served.  A token's p and o depend on the tokens up to it alone, also where later
// ones hold infinities or NaN, or overflow: what a later token makes of a matrix is in its own
// row, and where a triangular matrix meets rows that are not finite (XP, V), its zeros are
// left out by selection instead of multiplied.  kw and p are left as records, in fp32, from which
// the commit moves the state by m kept tokens without solving anything:
//   S' = gamma_{m-1} S + sum_{j<m} k_j x_j^T + kw_j y_j^T,
//   x_j = -rho(m-1, j) g_j b_j p_j,  y_j = rho(m-1, j) v_j.
// PRISM pages: WeChat ICML 2026 summary, sections 核心迭代形式, 消除 Token 间串行
// and 消除 Step 间串行; gist.science summary of arXiv 2602.10796, section 2.1
// (S_t = S_{t-1} A_t + B_t: moving by any prefix is exact).
//
// Bounds.  The least traffic is the fp32 state, read once (and written once by the
// commit), and the tokens' rows; the products cost 4 M dk dv flops a chain and run on the
// fp32 matrix instructions (16x16x4) under the loads of other workgroups.  The commit
// keeps to that: 256 sequences x 6 heads, dk = dv = 128, 5 of 8 tokens kept at the mean,
// 210 MB in 41 us, 5.1 TB/s.  The draft of one pass is two or three
// dependent reads, a barrier, the small matrices and the products, and a batch of 1500 to 4000 chains is
// only two rounds of the workgroups that the registers let run at a time (up to 128 a lane
// and four wavefronts a SIMD in bf16 and at L = 1; 129 to 159 and three in fp32 with levels, and in bf16
// with the GELU chain beyond L = 4), so that loads and products of one round overlap in part: the same
// batch, 1 to 8 tokens, 131 MB in 29.4 us, 4.5 TB/s; 512 x 8 heads of 64 x 64 with
// L = 8, 37 us for 8 tokens (5.1 TB/s) and 66 us for 9, whose second pass reads the
// state again; 8 x 6 heads of 5 tokens, 7.1 us (a launch alone: 3.8).  In fp32 those two batches
// take 32 us (156 MB, 4.9 TB/s) and 57 us (297 MB, 5.2 TB/s) for up to 8 tokens.
// Long sequences are walked all the same, with the square of the passes: 32 x 8
// heads (64 x 64) take 8.5, 94, 1380 and 23,000 us for 8, 64, 256 and 1024 tokens.
//
// Layout.  One workgroup per chain, one wavefront per 32 value columns; of the
// state, lane (kq, j) = (lane / 16, lane % 16) takes rows 16 R + 4 kq + r and the
// columns 2 j, 2 j + 1 of its wavefront, so a row of the tile is read in 128-byte
// pieces.  That is the accumulator layout of a 16x16 tile and, register r taken as one
// 16x16x4 step whose contraction index kq names row 4 kq + r, the second operand's
// too: S enters [K; Q] S and receives [K; KW]^T [X; Y] with no exchange between lanes.
// The first operand of step r then wants channel 4 kq + r, so one 16-byte LDS read
// serves four steps.  The same holds for XP, which comes out of one product and
// enters the next.
// The commit holds the state in registers (64 a lane at 128 x 128).  The draft streams
// it through the products instead, four tiles in flight, and reads it again in each
// pass, where the tokens of earlier passes enter by 16x16 products of the rows: with the
// state kept in registers 256 x 6 heads took 44 us instead of 35 (fewer workgroups at
// a time).
// Eight tokens fill a 16-row tile with K over Q, and one 16x16 product of
// [K; Q] with [K; KW] gives the dot products of all four triangular matrices (16 tokens a
// pass, with a tile each for K and Q and barriers between the small matrices: 512 x 8
// heads 77 us instead of 45).
// Token t sits in row 4 (t % 2) + t / 2 of its half: step r of a contraction over
// tokens covers tokens 2 r and 2 r + 1, so steps beyond the last token are left out.
// The write keys are formed by the whole workgroup (one thread per token and
// four channels, every load of it issued before the state's and before the first
// wait).  After a barrier one wavefront forms the small matrices, while the others
// go on to the state's product; after a second one all take them from LDS (each
// wavefront for itself: 512 x 8 heads 40.8 instead of 38.8 us, 256 x 6 heads 32.6
// instead of 31.4; the work given to another wavefront from chain to chain: 38.4 and 32.4).
// kw and p stay in fp32, as in the single-token step, so that the commit loses nothing;
// o is rounded once, from fp32.
#include "common.h"
#include "kernels.h"
#include "prism.h"

namespace prism {

namespace {

constexpr int kBlock = 8;                        // tokens per pass, at most

__device__ __forceinline__ f32x4_t mfma4(float a, float b, f32x4_t c)
{
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// row of a token within its half of a tile, and back
__device__ __forceinline__ int slot_of(int t) { return 4 * (t & 1) + (t >> 1); }
__device__ __forceinline__ int token_of(int s) { return 2 * (s & 3) + (s >> 2); }

typedef __attribute__((ext_vector_type(2))) float f32x2_t;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2_t;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;

// Device memory read and written at 32-bit byte offsets a lane from a base that is
// the same for the whole wavefront (a buffer resource in scalar registers), bounded:
// reads past the end give zeros, writes there are dropped, so tokens past the last
// need no branch.
struct Span {
    __amdgpu_buffer_rsrc_t r;
    __device__ Span(const void* p, int64_t bytes)
        : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000))
    {
    }
};

// One, two and four elements of the storage type: raw, and as fp32.
template <typename T> struct Elems;
template <> struct Elems<uint16_t> {
    typedef u32x2_t raw4;
    typedef uint32_t raw2;
    typedef uint16_t raw1;
    template <int AUX = 0> __device__ static raw4 load4(const Span& b, uint32_t at)
    {
        return __builtin_bit_cast(raw4, __builtin_amdgcn_raw_buffer_load_b64(b.r, at, 0, AUX));
    }
    __device__ static raw2 load2(const Span& b, uint32_t at) { return __builtin_amdgcn_raw_buffer_load_b32(b.r, at, 0, 0); }
    __device__ static raw1 load1(const Span& b, uint32_t at) { return __builtin_amdgcn_raw_buffer_load_b16(b.r, at, 0, 0); }
    __device__ static f32x4_t f32(raw4 x)
    {
        return {__uint_as_float(x[0] << 16), __uint_as_float(x[0] & 0xffff0000u), __uint_as_float(x[1] << 16),
                __uint_as_float(x[1] & 0xffff0000u)};
    }
    __device__ static f32x2_t f32(raw2 x) { return {__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)}; }
    __device__ static float f32(raw1 x) { return bf16_to_f32(x); }
    __device__ static void store1(uint16_t* to, float x) { *to = f32_to_bf16(x); }
    __device__ static void store2(const Span& b, uint32_t at, float x, float y)
    {
        __builtin_amdgcn_raw_buffer_store_b32(pack_bf16x2(x, y), b.r, at, 0, 0);
    }
};
template <> struct Elems<float> {
    typedef u32x4_t raw4;
    typedef u32x2_t raw2;
    typedef uint32_t raw1;
    template <int AUX = 0> __device__ static raw4 load4(const Span& b, uint32_t at)
    {
        return __builtin_bit_cast(raw4, __builtin_amdgcn_raw_buffer_load_b128(b.r, at, 0, AUX));
    }
    template <int AUX = 0> __device__ static raw2 load2(const Span& b, uint32_t at)
    {
        return __builtin_bit_cast(raw2, __builtin_amdgcn_raw_buffer_load_b64(b.r, at, 0, AUX));
    }
    __device__ static raw1 load1(const Span& b, uint32_t at) { return __builtin_amdgcn_raw_buffer_load_b32(b.r, at, 0, 0); }
    __device__ static f32x4_t f32(raw4 x) { return __builtin_bit_cast(f32x4_t, x); }
    __device__ static f32x2_t f32(raw2 x) { return __builtin_bit_cast(f32x2_t, x); }
    __device__ static float f32(raw1 x) { return __uint_as_float(x); }
    __device__ static void store1(float* to, float x) { *to = x; }
    __device__ static void store2(const Span& b, uint32_t at, float x, float y)
    {
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2_t, f32x2_t{x, y}), b.r, at, 0, 0);
    }
    __device__ static void store4(const Span& b, uint32_t at, f32x4_t x)
    {
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, x), b.r, at, 0, 0);
    }
};
typedef Elems<float> E32;
constexpr int kOnce = 2;                         // nontemporal: read once per call
constexpr uint32_t kOutside = 0xffffff00u;       // an offset past any span

// LDS that only this wavefront uses: what its lanes have stored is there for its loads
// (no instruction: the LDS serves a wavefront in order).
__device__ __forceinline__ void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local"); }

__device__ __forceinline__ float lane_value(float x, int lane)
{
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), lane));
}

// The factors of p (rows kq < 2) and v in [X; Y] of up to 8 tokens whose gates lane t
// holds (1 and 0 past the last): -between rho(last, t) g_t b_t and between rho(last, t).
// Returns between times all their gates.
__device__ __forceinline__ float scale_tokens(float gl, float bl, int kq, float between, float (&f)[4])
{
    float after = between;                               // times the product of the gates after t
#pragma unroll
    for (int t = kBlock - 1; t >= 0; --t) {
        const float y = after;
        after *= lane_value(gl, t);
        const float x = -after * lane_value(bl, t);
        f[t >> 1] = (t & 1) == 1 || (kq & 1) == 0 ? (kq < 2 ? x : y) : f[t >> 1];
    }
    return after;
}

// Whether every lane's values are finite: 0 x is zero for them, and NaN for an infinity or a NaN.
__device__ __forceinline__ bool all_finite(const f32x4_t (&x)[2])
{
    float z[2] = {0.f, 0.f};
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 2; ++c)
            z[c] = __builtin_fmaf(x[c][r], 0.f, z[c]);
    return __ballot(z[0] + z[1] != 0.f) == 0;
}

// y += M x for a matrix M (16 rows, columns `at` .. at + 7, rows and columns in slots) that is
// triangular in the tokens, and the tokens' values x (token 2 r + kq in register r of lanes
// kq < 2): as the matrix product, but M's zeros are left out instead of multiplied, which an
// x that is not finite would turn into NaN of earlier tokens.  A row takes the tokens up to its
// own; with STRICT a row of K (kq < 2) takes those before it.
template <bool STRICT>
__device__ __forceinline__ void add_triangular(f32x4_t (&y)[2], const float (*M)[20], int at, const f32x4_t (&x)[2],
                                               int kq, int j)
{
    const bool own_even = !STRICT || kq != 0, own_odd = STRICT ? kq == 3 : (kq & 1) == 1;
#pragma unroll
    for (int t = 0; t < kBlock; ++t) {
        float xt[2];
#pragma unroll
        for (int c = 0; c < 2; ++c)
            xt[c] = __int_as_float(__builtin_amdgcn_ds_bpermute(4 * ((t & 1) * 16 + j), __float_as_int(x[c][t >> 1])));
#pragma unroll
        for (int r = t >> 1; r < 4; ++r) {               // row 4 kq + r: token 2 r + kq % 2
            const float w = M[4 * kq + r][at + slot_of(t)];
            const bool in = t < 2 * r || (t == 2 * r ? own_even : own_odd);
#pragma unroll
            for (int c = 0; c < 2; ++c)
                y[c][r] = in ? y[c][r] + w * xt[c] : y[c][r];
        }
    }
}

// S <- gam S + [K; KW]^T [X; Y] for the rows of [K; KW] in LDS (fp32, 16 rows of
// LD); xy is [X; Y] as a tile; `steps` = ceil(tokens / 2)
template <int RT, int LD>
__device__ __forceinline__ void add_tokens(f32x4_t (&s)[RT][2], float gam, const float* rows, int steps, int kq,
                                           int j, const f32x4_t (&xy)[2])
{
#pragma unroll
    for (int R = 0; R < RT; ++R)
#pragma unroll
        for (int c = 0; c < 2; ++c)
            s[R][c] *= gam;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        if (r < steps) {
#pragma unroll
            for (int R = 0; R < RT; ++R) {
                const float x = rows[(4 * kq + r) * LD + 16 * R + j];
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    s[R][c] = mfma4(x, xy[c][r], s[R][c]);
            }
        }
    }
}

}  // namespace

// The arrays of a chain's tokens base .. base + m - 1 (m <= 8), at their head's rows.
template <typename T, int DK, int DV> struct Pass {
    Span k, q, v, g, b, kw, p;
    uint32_t krow, vrow, grow;                           // bytes from token to token
    __device__ Pass(const T* k_, const T* q_, const T* v_, const T* g_, const T* b_, float* kw_, float* p_, int64_t at,
                    int m, int H, int e)
        : k(k_ + (at * H + e) * DK, bytes(m, H, DK, sizeof(T))), q(q_ + (at * H + e) * DK, bytes(m, H, DK, sizeof(T))),
          v(v_ + (at * H + e) * DV, bytes(m, H, DV, sizeof(T))), g(g_ + at * H + e, bytes(m, H, 1, sizeof(T))),
          b(b_ + at * H + e, bytes(m, H, 1, sizeof(T))), kw(kw_ + (at * H + e) * DK, bytes(m, H, DK, 4)),
          p(p_ + (at * H + e) * DV, bytes(m, H, DV, 4)), krow(H * DK), vrow(H * DV), grow(H)
    {
    }
    // up to the end of the last token's row
    __device__ static int64_t bytes(int m, int H, int width, int size) { return ((int64_t)(m - 1) * H + 1) * width * size; }
};

// The write key of one token (in a pass that starts at token `base` of its sequence) in
// four channels, to its record in fp32; zeros past the pass.  LEV levels of u, a, h
// are loaded at a time (LEV = 0: L = 1), every load issued before the first use.
template <typename T, int DK, int DV, int LEV, bool GELU> struct WriteKey {
    typedef Elems<T> X;
    typedef typename X::raw4 raw4;
    static constexpr int LV = LEV > 0 ? LEV : 1, ES = sizeof(T);
    const Pass<T, DK, DV>& ps;
    Span u, a, h, past, hist, w;
    int base, L;

    __device__ WriteKey(const Pass<T, DK, DV>& ps_, const T* k_, const T* u_, const T* a_, const T* h_, const T* conv_w,
                        const T* k_hist, int64_t chain, int64_t c0, int base_, int m, int H, int e, int L_)
        : ps(ps_), u(u_ + lev(c0 + base_, H, e, L_), lev_bytes(m, H, L_)),
          a(a_ + lev(c0 + base_, H, e, L_), lev_bytes(m, H, L_)), h(h_ + lev(c0 + base_, H, e, L_), lev_bytes(m, H, L_)),
          // the rows before a token: of the sequence, or (for its first three) carried
          past(k_ + ((c0 + (base_ > 3 ? base_ - 3 : 0)) * H + e) * DK,
               ps_.bytes(m + (base_ > 3 ? 3 : base_), H, DK, ES)),
          hist(k_hist + chain * 3 * DK, base_ == 0 ? 3 * DK * ES : 0), w(conv_w + (int64_t)e * DK * 4, DK * 4 * ES),
          base(base_), L(L_)
    {
    }
    __device__ static int64_t lev(int64_t at, int H, int e, int L) { return (at * H + e) * (L - 1) * DK; }
    __device__ static int64_t lev_bytes(int m, int H, int L) { return Pass<T, DK, DV>::bytes(m, H, (L - 1) * DK, ES); }

    raw4 ar[LV], ur[LV], hr[LV], pr[3], hi[3], wr[4], kr;
    typename X::raw1 br;
    __device__ void fetch_levels(uint32_t t, uint32_t ch, int l0)
    {
        const uint32_t at = (t * ps.krow * (L - 1) + ch) * ES;
#pragma unroll
        for (int l = 0; l < LEV; ++l) {                  // past the last level: zeros, which change no finite sum
            const uint32_t la = l0 + l < L - 1 ? at + (l0 + l) * DK * ES : kOutside;
            ar[l] = X::template load4<kOnce>(a, la);
            ur[l] = X::template load4<kOnce>(u, la);
            hr[l] = X::template load4<kOnce>(h, l0 + l < L - 2 ? la : kOutside);
        }
    }
    __device__ void fetch_taps(uint32_t t, uint32_t ch)
    {
        kr = X::load4(ps.k, (t * ps.krow + ch) * ES);
#pragma unroll
        for (int d = 1; d <= 3; ++d) {
            const uint32_t row = base > 3 ? t + 3 - d : t + base - d;    // wraps past the end below the first row
            pr[d - 1] = X::load4(past, (row * ps.krow + ch) * ES);
            hi[d - 1] = X::load4(hist, ((t + 3 - d) * DK + ch) * ES);    // empty but for the first pass
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
            wr[x] = X::load4(w, (ch + x) * 4 * ES);
        br = X::load1(ps.b, t * ps.grow * ES);
    }
    __device__ void fetch(uint32_t t, uint32_t ch)
    {
        fetch_levels(t, ch, 0);
        fetch_taps(t, ch);
    }
    // the ShortConv anchor r and b k
    __device__ void start(f32x4_t& kt, f32x4_t& r, f32x4_t& acc)
    {
        kt = X::f32(kr);
        f32x4_t x[3];
#pragma unroll
        for (int d = 0; d < 3; ++d)                      // one of the two is zero
            x[d] = X::f32(pr[d] | hi[d]);
        const float bt = X::f32(br);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const f32x4_t wc = X::f32(wr[c]);
            r[c] = wc[3] * kt[c] + wc[2] * x[0][c] + wc[1] * x[1][c] + wc[0] * x[2][c];
            acc[c] = bt * kt[c];
        }
    }
    __device__ f32x4_t form(uint32_t t, uint32_t ch, f32x4_t& kt)
    {
        f32x4_t r, acc;
        start(kt, r, acc);
        for (int l0 = 0; LEV > 0 && l0 < L - 1; l0 += LV) {
            if (l0 > 0)
                fetch_levels(t, ch, l0);
#pragma unroll
            for (int l = 0; l < LEV; ++l) {              // r (1 - a h) = r - (a r) h
                const f32x4_t av = X::f32(ar[l]), uv = X::f32(ur[l]), hv = X::f32(hr[l]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float ar_c = av[c] * r[c];
                    acc[c] += ar_c * uv[c];
                    r[c] -= GELU ? av[c] * gelu_as(hv[c] * r[c]) : ar_c * hv[c];
                }
            }
        }
        if (LEV > 0 && !(acc[0] * 0.f + acc[1] * 0.f + acc[2] * 0.f + acc[3] * 0.f == 0.f))
            acc = form_by_level(t, ch);
        E32::store4(ps.kw, (t * ps.krow + ch) * 4, acc);
        return acc;
    }
    // The same where it is not finite: level by level as the recurrence has it, so that an infinite r is
    // neither met by the zeros past the last level nor taken from itself
    __device__ f32x4_t form_by_level(uint32_t t, uint32_t ch)
    {
        f32x4_t kt, r, acc;
        fetch_taps(t, ch);
        start(kt, r, acc);
#pragma unroll 1
        for (int l = 0; l < L - 1; ++l) {
            const uint32_t at = ((t * ps.krow * (L - 1) + ch) + l * DK) * ES;
            const f32x4_t av = X::f32(X::load4(a, at)), uv = X::f32(X::load4(u, at)), hv = X::f32(X::load4(h, at));
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                acc[c] += av[c] * r[c] * uv[c];
                if (l < L - 2)
                    r[c] = GELU ? r[c] - av[c] * gelu_as(hv[c] * r[c]) : r[c] * (1.f - av[c] * hv[c]);
            }
        }
        return acc;
    }
};

// The draft kernel's arguments, read from the kernel's argument segment where they are used:
// held in scalar registers over the pass loop (30 of them beside the buffer resources)
// they were spilled into vector lanes, as 10 to 23 scalars of the instances with levels still are.
template <typename T> struct DraftPointers {
    const T *q, *k, *v, *u, *a, *h, *g, *b, *conv_w;
    const int32_t* cu;
    const float* S;
    const T* k_hist;
    T* o;
    float *kw, *p;
    int H, L;
};
template <typename T> using Segment = const __attribute__((address_space(4))) DraftPointers<T>*;

// The same scalar value, not known to the compiler: loads from an address, and what derives
// from a number, are not moved to where it came from.
template <typename P> __device__ __forceinline__ P again(P p)
{
    asm volatile("" : "+s"(p));
    return p;
}

template <typename T, int DK, int DV, int LEV, bool GELU>
__global__ __launch_bounds__(2 * DV, 3) void draft_kernel(DraftPointers<T>)
{
    typedef Elems<T> X;
    constexpr int NTH = 2 * DV, W = NTH / 64, RT = DK / 16, LD = DK + 4, CG = DK / 4, ES = sizeof(T);
    constexpr int ITEMS = (kBlock * CG + NTH - 1) / NTH;         // pieces of the tile rows a thread stages
    // rows 0..7 Q, 8..15 K, 16..23 KW: rows 8.. are [K; KW], row (i + 8) % 16 of [K; Q] is i
    __shared__ __align__(16) float sRows[24 * LD];
    __shared__ __align__(16) float sM[2][16][20];        // [A B; C E], then W
    __shared__ __align__(16) float sGam[16];             // the gates before a row of K, up to a row of Q
    __shared__ __align__(16) float sD[W][16][20];        // a wavefront's dot products with earlier tokens

    const Segment<T> in = (Segment<T>)__builtin_amdgcn_kernarg_segment_ptr();
    const int heads = in->H, levels = in->L;
    const int64_t chain = blockIdx.x;
    const int e = (int)(chain % heads);
    const int64_t n = chain / heads;

    // the state is streamed: tiles R .. R + PRE - 1 in flight, rows 16 R + 4 kq + r, two
    // columns a lane; the first EARLY are on their way before the sequence is looked up
    // (fewer where the write key's loads need the registers)
    constexpr int PRE = RT < 4 ? RT : 4, EARLY = LEV > 3 ? PRE / 2 : PRE;
    const Span state(in->S + chain * DK * DV, DK * DV * 4);
    E32::raw2 s[PRE][4];
    auto fetch_state = [&](int R, int tid) {
        const int at = ((tid & 48) / 4 * DV + 32 * (tid >> 6) + 2 * (tid & 15)) * 4;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            s[R % PRE][r] = E32::template load2<kOnce>(state, at + (16 * R + r) * DV * 4);
    };
#pragma unroll
    for (int R = 0; R < EARLY; ++R)
        fetch_state(R, threadIdx.x);

    const int64_t c0 = in->cu[n];
    const int len = in->cu[n + 1] - (int)c0;
    if (len <= 0)
        return;
    if (len > PRISM_MAX_DRAFT) {                         // not served
        for (int64_t i = threadIdx.x; i < (int64_t)len * DK; i += NTH)
            in->kw[((c0 + i / DK) * heads + e) * DK + i % DK] = __builtin_nanf("");
        for (int64_t i = threadIdx.x; i < (int64_t)len * DV; i += NTH) {
            in->p[((c0 + i / DV) * heads + e) * DV + i % DV] = __builtin_nanf("");
            X::store1(in->o + ((c0 + i / DV) * heads + e) * DV + i % DV, __builtin_nanf(""));
        }
        return;
    }

    for (int base = 0, m; base < len; base += m) {
        // what derives from the sizes is formed in each pass: kept over them it is spilled
        const int H = again(heads), L = again(levels);
        __builtin_assume(LEV == 0 || L > 1);             // as launched: no branch parts a token's loads
        const int tid = opaque(threadIdx.x), lane = tid & 63, kq = lane >> 4, j = lane & 15;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), col = 32 * wave + 2 * j;
        m = len - base < kBlock ? len - base : kBlock;
        const int steps = (m + 1) >> 1;
        const Segment<T> ap = again(in);
        const Pass<T, DK, DV> ps(ap->k, ap->q, ap->v, ap->g, ap->b, ap->kw, ap->p, c0 + base, m, H, e);
        const bool staged = again(base) > 0;             // whether the write keys are formed
        if (staged)
            __syncthreads();                             // the pass before is done with the LDS; kw and p are written
        // gates (lane t holds token t's) and value rows: register r holds row 4 (kq % 2) + r, token
        // 2 r + kq % 2, in both halves
        const typename X::raw1 gr = X::load1(ps.g, (lane & 7) * ps.grow * ES),
                               br = X::load1(ps.b, (lane & 7) * ps.grow * ES);
        typename X::raw2 vr[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
            vr[r] = X::load2(ps.v, ((2 * r + (kq & 1)) * ps.vrow + col) * ES);
#pragma unroll
        for (int x = 0; x < ITEMS; ++x) {
            const int i = tid + x * NTH, t = i / CG, ch = (i % CG) * 4;
            f32x4_t kt = {}, wt = {};
            const typename X::raw4 qr = X::load4(ps.q, (t * ps.krow + ch) * ES);
            if (LEV > 0 && t >= m) {
                // no token: zero rows without the chain (4 of 8 tokens, L = 8: 3 % less time; at
                // L = 1, where there is none, the branch costs 4 %)
            } else if (!staged) {
                WriteKey<T, DK, DV, LEV, GELU> key(ps, ap->k, ap->u, ap->a, ap->h, ap->conv_w, ap->k_hist, chain, c0,
                                                     base, m, H, e, L);
                key.fetch(t, ch);
                wt = key.form(t, ch, kt);
            } else {
                kt = X::f32(X::load4(ps.k, (t * ps.krow + ch) * ES));
                wt = E32::f32(E32::load4(ps.kw, (t * ps.krow + ch) * 4));
            }
            if (kBlock * CG >= NTH || t < kBlock) {
                float* to = sRows + slot_of(t) * LD + ch;
                *reinterpret_cast<f32x4_t*>(to) = X::f32(qr);
                *reinterpret_cast<f32x4_t*>(to + 8 * LD) = kt;
                *reinterpret_cast<f32x4_t*>(to + 16 * LD) = wt;
            }
        }
        if (!staged) {
            for (int at = kBlock; at < len; at += kBlock) {
                const int mt = len - at < kBlock ? len - at : kBlock;
                const Segment<T> al = again(in);
                const Pass<T, DK, DV> later(al->k, al->q, al->v, al->g, al->b, al->kw, al->p, c0 + at, mt, H, e);
                WriteKey<T, DK, DV, LEV, GELU> key(later, al->k, al->u, al->a, al->h, al->conv_w, al->k_hist, chain, c0,
                                                   at, mt, H, e, L);
#pragma unroll 1
                for (int i = opaque(tid); i < mt * CG; i += NTH) {
                    f32x4_t kt;
                    key.fetch(i / CG, (i % CG) * 4);
                    key.form(i / CG, (i % CG) * 4, kt);
                }
            }
        }
#pragma unroll
        for (int R = 0; R < PRE; ++R)
            if (staged || R >= EARLY)
                fetch_state(R, tid);
        const float gl = (lane & 7) < m ? X::f32(gr) : 1.f, bl = X::f32(br);
        f32x4_t vv[2];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const f32x2_t x = X::f32(vr[r]);
            vv[0][r] = x[0];
            vv[1][r] = x[1];
        }
        lds_barrier();                                   // the state's loads stay in flight
        const float* pa = sRows + ((j + 8) & 15) * LD + 4 * kq;      // row j of [K; Q]
        float(*M0)[20] = sM[0], (*M1)[20] = sM[1];
        if (wave == 0) {                                 // the small matrices, while the others go on to the state
            float gg[kBlock], bb[kBlock];
#pragma unroll
            for (int t = 0; t < kBlock; ++t) {
                gg[t] = lane_value(gl, t);
                bb[t] = lane_value(bl, t);
            }
            // [K; Q] [K; KW]^T
            f32x4_t d0 = {}, d1 = {};
            const float* pb = sRows + (j + 8) * LD + 4 * kq;             // row j of [K; KW]
#pragma unroll
            for (int R = 0; R < RT; ++R) {
                const f32x4_t fa = *reinterpret_cast<const f32x4_t*>(pa + 16 * R);
                const f32x4_t fb = *reinterpret_cast<const f32x4_t*>(pb + 16 * R);
                d0 = mfma4(fa[0], fb[0], d0);
                d1 = mfma4(fa[1], fb[1], d1);
                d0 = mfma4(fa[2], fb[2], d0);
                d1 = mfma4(fa[3], fb[3], d1);
                if (R % 4 == 3)
                    __builtin_amdgcn_sched_barrier(0);       // not all the LDS reads at once: registers
            }
            d0 += d1;
            // element (i, j): token ti of row i against token tj of column j, times the gates
            // between them: for a row of K those before ti, for a row of Q those up to ti
            const int tj = token_of(j & 7);
            float rho[4] = {}, gam[4] = {}, run = 0.f, all = 1.f, own = 0.f;
#pragma unroll
            for (int t = 0; t < kBlock; ++t) {
                const float before = all, upto = run;        // products of the gates before t; from tj + 1 before t
                all *= gg[t];
                run = t == tj ? 1.f : run * gg[t];           // 0 before tj, rho(t, tj) from there on
                own = t == tj ? gg[t] * bb[t] : own;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (t == 2 * r + (kq & 1)) {
                        rho[r] = kq < 2 ? upto : run;
                        gam[r] = kq < 2 ? before : all;
                    }
            }
            __builtin_amdgcn_sched_barrier(0);
            if (j == 0)
                *reinterpret_cast<f32x4_t*>(sGam + 4 * kq) = f32x4_t{gam[0], gam[1], gam[2], gam[3]};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int ti = 2 * r + (kq & 1);
                float x = 0.f;                               // selected, not scaled: see above
                if (ti < m && (kq < 2 ? tj < ti : tj <= ti))
                    x = rho[r] * (j < 8 ? own : 1.f) * d0[r];
                M0[4 * kq + r][j] = x;
            }
            wave_fence();
            // T by substitution, column tj' = slot lane % 8 on every group of 8 lanes; row lane / 8 of
            // T and of -C T is kept
            {
                const int c = lane & 7, gr = lane >> 3;
                float tc[kBlock];                            // T's column, by token
#pragma unroll
                for (int i = 0; i < kBlock; ++i) {
                    float x = token_of(c) == i ? 1.f : 0.f;
                    const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(&M0[slot_of(i)][0]);
                    const f32x4_t hi = *reinterpret_cast<const f32x4_t*>(&M0[slot_of(i)][4]);
#pragma unroll
                    for (int l = 0; l < i; ++l)
                        x -= ((l & 1) ? hi[l >> 1] : lo[l >> 1]) * tc[l];
                    tc[i] = x;
                    if (i % 4 == 3)
                        __builtin_amdgcn_sched_barrier(0);
                }
                const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(&M0[8 + gr][0]);
                const f32x4_t hi = *reinterpret_cast<const f32x4_t*>(&M0[8 + gr][4]);
                const int own = token_of(gr);
                float ct = 0.f, tt = 0.f;
#pragma unroll
                for (int l = 0; l < kBlock; ++l) {           // C's zeros left out: later rows of T may not be finite
                    ct = l <= own ? ct - ((l & 1) ? hi[l >> 1] : lo[l >> 1]) * tc[l] : ct;
                    tt = slot_of(l) == gr ? tc[l] : tt;
                }
                M1[gr][c] = tt;
                M1[8 + gr][c] = ct;
                M1[gr][8 + c] = M1[8 + gr][8 + c] = 0.f;     // what the lanes of Q's rows read
            }
            wave_fence();
            __builtin_amdgcn_sched_barrier(0);
        }
        // [K; Q] S
        f32x4_t x[2] = {};
#pragma unroll
        for (int R = 0; R < RT; ++R) {
            const f32x4_t fa = *reinterpret_cast<const f32x4_t*>(pa + 16 * R);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    x[c] = mfma4(fa[r], __uint_as_float(s[R % PRE][r][c]), x[c]);
            if (R + PRE < RT)
                fetch_state(R + PRE, tid);
            if (R % 4 == 3)
                __builtin_amdgcn_sched_barrier(0);
        }
        lds_barrier();
        // columns 8.. of the first matrix ([B; E]; the second half of vv repeats the first), and W,
        // zeros for the rows of Q
        const f32x4_t fv = *reinterpret_cast<const f32x4_t*>(&M0[j][8 + 4 * (kq & 1)]);
        const f32x4_t fw = *reinterpret_cast<const f32x4_t*>(&M1[j][4 * kq]);
        const f32x4_t gam = *reinterpret_cast<const f32x4_t*>(sGam + 4 * kq);
        if (base > 0) {
            // the tokens of earlier passes, 8 at a time from the latest: their part of the state
            // is [K'; KW']^T [X'; Y'], so that they add ([K; Q] [K'; KW']^T) [X'; Y'] of 16x16
            f32x4_t z[2] = {};
            float between = 1.f;                         // the product of the gates from here to this pass
            for (int cb = base - kBlock; cb >= 0; cb -= kBlock) {
                const int lane = opaque(threadIdx.x) & 63, kq = lane >> 4, j = lane & 15;
                const float* pa = sRows + ((j + 8) & 15) * LD + 4 * kq;
                const Segment<T> ac = again(in);
                const Pass<T, DK, DV> pc(ac->k, ac->q, ac->v, ac->g, ac->b, ac->kw, ac->p, c0 + cb, again(kBlock), H, e);
                const float gc = X::f32(X::load1(pc.g, (lane & 7) * pc.grow * ES));
                const float bc = X::f32(X::load1(pc.b, (lane & 7) * pc.grow * ES));
                f32x4_t xy[2], d = {};
#pragma unroll
                for (int r = 0; r < 4; ++r) {            // p: what this lane has stored itself
                    const uint32_t at = (2 * r + (kq & 1)) * pc.vrow + col;
                    const f32x2_t y = kq < 2 ? E32::f32(E32::load2(pc.p, at * 4)) : X::f32(X::load2(pc.v, at * ES));
                    xy[0][r] = y[0];
                    xy[1][r] = y[1];
                }
                const uint32_t row = token_of(j & 7) * pc.krow + 4 * kq;
#pragma unroll
                for (int R = 0; R < RT; ++R) {
                    const f32x4_t fa = *reinterpret_cast<const f32x4_t*>(pa + 16 * R);
                    const f32x4_t fb = j < 8 ? X::f32(X::load4(pc.k, (row + 16 * R) * ES))
                                             : E32::f32(E32::load4(pc.kw, (row + 16 * R) * 4));
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        d = mfma4(fa[r], fb[r], d);
                    if (R % 2 == 1)
                        __builtin_amdgcn_sched_barrier(0);
                }
                float f[4];
                between = scale_tokens(gc, bc, kq, between, f);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    xy[0][r] *= f[r];
                    xy[1][r] *= f[r];
                    sD[wave][4 * kq + r][j] = d[r];
                }
                wave_fence();
                const f32x4_t fd = *reinterpret_cast<const f32x4_t*>(&sD[wave][j][4 * kq]);
                wave_fence();
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        z[c] = mfma4(fd[r], xy[c][r], z[c]);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c)
                x[c] = between * x[c] + z[c];
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r)                  // rows past the tokens stay out of the next product
                x[c][r] = 2 * r + (kq & 1) < m ? gam[r] * x[c][r] : 0.f;
        if (!all_finite(vv)) {
            add_triangular<true>(x, M0, 8, vv, kq, j);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (r < steps)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        x[c] = mfma4(kq < 2 ? fv[r] : 0.f, vv[c][r], x[c]);
        }
        f32x4_t y[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {                // Q's rows: to their outputs alone
                y[c][r] = kq < 2 ? 0.f : x[c][r];
                x[c][r] = kq < 2 ? x[c][r] : 0.f;
            }
        }
        // an infinity or a NaN of a token's row of XP (its key's, or an overflow) is not its
        // predecessors'
        if (!all_finite(x)) {
            add_triangular<false>(y, M1, 0, x, kq, j);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (r < steps)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        y[c] = mfma4(fw[r], x[c][r], y[c]);
        }
        const Span out(again(in)->o + ((c0 + base) * H + e) * DV, ps.bytes(m, H, DV, ES));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint32_t at = (2 * r + (kq & 1)) * ps.vrow + col;
            if (kq < 2)
                E32::store2(ps.p, at * 4, y[0][r], y[1][r]);
            else
                X::store2(out, at * ES, y[0][r], y[1][r]);
        }
    }
}

// S_out and hist_out may be S and hist: a thread has read what it overwrites.
// blockIdx.y is a band of ROWS state rows.
template <typename T, int DK, int DV, int ROWS>
__global__ __launch_bounds__(2 * DV, 4) void commit_kernel(
    const T* __restrict__ k, const T* __restrict__ v, const T* __restrict__ g, const T* __restrict__ b,
    const int32_t* __restrict__ cu, const int32_t* __restrict__ n_accept, int H,
    const float* __restrict__ kw, const float* __restrict__ p, const float* S, const T* hist, float* S_out,
    T* hist_out)
{
    typedef Elems<T> X;
    constexpr int NTH = 2 * DV, RT = ROWS / 16, LD = ROWS + 4, CG = ROWS / 4, ES = sizeof(T);
    __shared__ __align__(16) float sRows[16 * LD];       // rows of K, then of KW

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
    const int col = 32 * wave + 2 * j;
    const Span from(S + (chain * DK + row0) * DV, ROWS * DV * 4), to(S_out + (chain * DK + row0) * DV, ROWS * DV * 4);
    const uint32_t sat = (4 * kq * DV + col) * 4;
#pragma unroll
    for (int R = 0; R < RT; ++R)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const f32x2_t x = E32::f32(E32::template load2<kOnce>(from, sat + (16 * R + r) * DV * 4));
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
        const int steps = (m + 1) >> 1;
        const Pass<T, DK, DV> ps(k, k, v, g, b, const_cast<float*>(kw), const_cast<float*>(p), c0 + base, m, H, e);
        if (base > 0)
            __syncthreads();                             // the pass before is done with the LDS
        for (int i = tid; i < 2 * steps * CG; i += NTH) {
            const int t = i / CG, ch = (i % CG) * 4;
            const uint32_t at = t * ps.krow + row0 + ch;
            float* row = sRows + slot_of(t) * LD + ch;
            const f32x4_t kt = X::f32(X::load4(ps.k, at * ES)), wt = E32::f32(E32::load4(ps.kw, at * 4));
            *reinterpret_cast<f32x4_t*>(row) = kt;
            *reinterpret_cast<f32x4_t*>(row + 8 * LD) = wt;
        }
        const float gl = (lane & 7) < m ? X::f32(X::load1(ps.g, (lane & 7) * ps.grow * ES)) : 1.f;
        const float bl = X::f32(X::load1(ps.b, (lane & 7) * ps.grow * ES));
        f32x4_t xy[2];                                   // p over v
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint32_t at = (2 * r + (kq & 1)) * ps.vrow + col;
            const f32x2_t x = kq < 2 ? E32::f32(E32::load2(ps.p, at * 4)) : X::f32(X::load2(ps.v, at * ES));
            xy[0][r] = x[0];
            xy[1][r] = x[1];
        }
        __syncthreads();
        float f[4];
        const float after = scale_tokens(gl, bl, kq, 1.f, f);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            xy[0][r] *= f[r];
            xy[1][r] *= f[r];
        }
        add_tokens<RT, LD>(s, after, sRows, steps, kq, j, xy);
    }
#pragma unroll
    for (int R = 0; R < RT; ++R)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            __builtin_amdgcn_raw_buffer_store_b64(
                __builtin_bit_cast(u32x2_t, f32x2_t{s[R][0][r], s[R][1][r]}), to.r, sat + (16 * R + r) * DV * 4, 0, kOnce);
}

template <typename T, int DK, int DV, int LEV, bool GELU>
static hipError_t launch_draft_lev(const DraftArgs& p, hipStream_t stream)
{
    const DraftPointers<T> in = {(const T*)p.q, (const T*)p.k, (const T*)p.v, (const T*)p.u, (const T*)p.a,
                                 (const T*)p.h, (const T*)p.g, (const T*)p.b, (const T*)p.conv_w, p.cu_seqlens,
                                 p.S, (const T*)p.k_hist, (T*)p.o, p.kw, p.p, p.heads, p.L};
    hipLaunchKernelGGL((draft_kernel<T, DK, DV, LEV, GELU>), dim3((unsigned)((int64_t)p.n_seqs * p.heads)), dim3(2 * DV),
                       0, stream, in);
    return hipGetLastError();
}

// Levels loaded at a time: all of them up to L = 4 and (bf16) up to L = 8, seven at a
// time beyond; fp32 takes three at a time, whose loads fill as many registers.  The
// two chains are the same up to L = 2.
template <typename T, int DK, int DV>
static hipError_t launch_draft_t(const DraftArgs& p, hipStream_t stream)
{
    if (p.L == 1)
        return launch_draft_lev<T, DK, DV, 0, false>(p, stream);
    const bool gelu = p.gelu && p.L > 2;
    if constexpr (sizeof(T) == 2) {
        if (p.L > 4)
            return gelu ? launch_draft_lev<T, DK, DV, 7, true>(p, stream)
                        : launch_draft_lev<T, DK, DV, 7, false>(p, stream);
    }
    return gelu ? launch_draft_lev<T, DK, DV, 3, true>(p, stream) : launch_draft_lev<T, DK, DV, 3, false>(p, stream);
}

template <typename T, int DK, int DV, int ROWS>
static hipError_t launch_commit_rows(const DraftArgs& p, hipStream_t stream)
{
    hipLaunchKernelGGL((commit_kernel<T, DK, DV, ROWS>), dim3((unsigned)((int64_t)p.n_seqs * p.heads), DK / ROWS),
                       dim3(2 * DV), 0, stream, (const T*)p.k, (const T*)p.v, (const T*)p.g, (const T*)p.b,
                       p.cu_seqlens, p.n_accept, p.heads, p.kw, p.p, p.S, (const T*)p.k_hist, p.S_out,
                       (T*)p.k_hist_out);
    return hipGetLastError();
}

// A chain's rows are apart in the commit, so few chains are cut into bands of 32 rows that
// run side by side: 48 chains of 128 x 128 take 4.6 instead of 7.0 us, 192 take 7.0
// instead of 7.7; with 384 the two are equal (11.3 us), and 1536 take 44.5 instead of
// 43.5, the tokens' rows of p and v being read by every band.
template <typename T, int DK, int DV>
static hipError_t launch_commit_t(const DraftArgs& p, hipStream_t stream)
{
    return (int64_t)p.n_seqs * p.heads <= 256 ? launch_commit_rows<T, DK, DV, 32>(p, stream)
                                               : launch_commit_rows<T, DK, DV, DK>(p, stream);
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
