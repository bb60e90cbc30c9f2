// layer_api.hip -- C ABI of the layer operators around the memory-writing
// operator (declared in include/prism.h): the norms before and after it, the
// decoding of drafted tokens, its commit and the verification.  Argument
// checks and launches on the caller's stream.
#include <math.h>

#include <initializer_list>

#include "api_checks.h"
#include "kernels.h"
#include "prism.h"

namespace {

bool norm_dims_ok(const prism_norm_dims* d)
{
    return d && d->rows >= 0 && d->heads >= 1 && d->width >= 1 && d->rows % d->heads == 0 &&
           d->rows <= INT64_MAX / 16 / d->width && (int64_t)d->heads * d->width <= INT32_MAX &&
           (d->dtype == PRISM_F32 || d->dtype == PRISM_BF16);
}

// Row arrays may be null when there are no rows.
bool row_ok(const prism_norm_dims* d, const void* p) { return d->rows == 0 ? aligned16(p) : ptr_ok(p); }

bool eps_ok(float eps) { return eps >= 0.f && isfinite(eps); }

bool gate_ok(int gate) { return gate == PRISM_GATE_SILU || gate == PRISM_GATE_SIGMOID; }

bool verify_dims_ok(const prism_verify_dims* d)
{
    return d && d->n_seqs >= 1 && d->total_tokens >= 0 && d->vocab >= 1 &&
           (d->dtype == PRISM_F32 || d->dtype == PRISM_BF16);
}

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

// The kernels of drafted tokens reach 8 tokens and the three rows before them from one
// base with 32-bit offsets.
bool draft_shape_ok(const prism_dims* d, int64_t levels)
{
    const int64_t row = d->dk * levels > d->dv ? d->dk * levels : d->dv;
    return prism::decode_supported(d->dk, d->dv) && (int64_t)d->heads * row * 11 * 4 <= INT32_MAX &&
           grid_ok((int64_t)d->n_seqs * d->heads, 2 * d->dv);
}

}  // namespace

extern "C" {

size_t prism_norm_workspace_bytes(const prism_norm_dims* d)
{
    if (!norm_dims_ok(d))
        return 0;
    // the larger of the two backwards: dw and dscale of a single weight row, or
    // dw of `heads` rows
    const size_t gate = (size_t)prism::norm_gate_bwd_blocks(d->rows / d->heads, d->heads) * d->heads;
    const size_t res = 2 * (size_t)prism::norm_residual_bwd_blocks(d->rows, d->width);
    return round256((gate > res ? gate : res) * d->width * sizeof(float));
}

prism_status prism_norm_residual(const prism_norm_dims* d, const void* x, const void* y, const void* scale,
                                 const void* w, float eps, void* r, void* n, void* stream)
{
    if (!norm_dims_ok(d) || d->heads != 1 || !eps_ok(eps))
        return PRISM_EINVAL;
    if (!row_ok(d, x) || !opt_ok(y) || !opt_ok(scale) || !ptr_ok(w) || !opt_ok(r) || !row_ok(d, n))
        return PRISM_EINVAL;
    if (d->rows > 0 && ((scale && !y) || (y && !r)))
        return PRISM_EINVAL;
    if (d->width > prism::kNormMaxWidth)
        return PRISM_EUNSUPPORTED;
    const int64_t all = d->rows * d->width * size_of(d->dtype), row = d->width * size_of(d->dtype);
    if (!apart({{r, all, true}, {n, all, true}}, {{x, all, true}, {y, all, true}, {scale, row}, {w, row}}))
        return PRISM_EINVAL;
    prism::NormResidualArgs p = {};
    p.bf16 = d->dtype == PRISM_BF16;
    p.rows = d->rows;
    p.width = d->width;
    p.eps = eps;
    p.x = x; p.y = y; p.scale = scale; p.w = w;
    p.r = r;
    p.n = n;
    return from_hip(prism::launch_norm_residual(p, (hipStream_t)stream));
}

prism_status prism_norm_residual_bwd(const prism_norm_dims* d, const void* r, const void* y,
                                     const void* scale, const void* w, float eps, const void* dn,
                                     const void* dr, void* dx, void* dy, float* dw, float* dscale,
                                     void* workspace, size_t workspace_bytes, void* stream)
{
    if (!norm_dims_ok(d) || d->heads != 1 || !eps_ok(eps))
        return PRISM_EINVAL;
    if (!row_ok(d, r) || !opt_ok(y) || !opt_ok(scale) || !ptr_ok(w) || !row_ok(d, dn) || !opt_ok(dr) ||
        !row_ok(d, dx) || !opt_ok(dy) || !ptr_ok(dw) || !opt_ok(dscale) || !ptr_ok(workspace))
        return PRISM_EINVAL;
    if (dscale && (!scale || (!y && d->rows > 0)))
        return PRISM_EINVAL;
    if (d->width > prism::kNormMaxWidth)
        return PRISM_EUNSUPPORTED;
    const int64_t need = prism_norm_workspace_bytes(d);
    if (workspace_bytes < (size_t)need)
        return PRISM_EINVAL;
    const int64_t all = d->rows * d->width * size_of(d->dtype), row = d->width * size_of(d->dtype);
    if (!apart({{dx, all, true}, {dy, all, true}, {dw, d->width * 4}, {dscale, d->width * 4}, {workspace, need}},
               {{r, all, true}, {y, all, true}, {dn, all, true}, {dr, all, true}, {scale, row}, {w, row}}))
        return PRISM_EINVAL;
    prism::NormResidualArgs p = {};
    p.bf16 = d->dtype == PRISM_BF16;
    p.rows = d->rows;
    p.width = d->width;
    p.eps = eps;
    p.y = y; p.scale = scale; p.w = w;
    p.r = const_cast<void*>(r);
    p.dn = dn; p.dr = dr;
    p.dx = dx; p.dy = dy;
    p.dw = dw;
    p.dscale = dscale;
    p.ws = (float*)workspace;
    return from_hip(prism::launch_norm_residual_bwd(p, (hipStream_t)stream));
}

prism_status prism_norm_gate(const prism_norm_dims* d, const void* o, const void* z, const void* w,
                             float eps, int gate, void* y, void* stream)
{
    if (!norm_dims_ok(d) || !eps_ok(eps) || !gate_ok(gate))
        return PRISM_EINVAL;
    if (!row_ok(d, o) || !row_ok(d, z) || !ptr_ok(w) || !row_ok(d, y))
        return PRISM_EINVAL;
    if (d->width > prism::kNormGateMaxWidth || d->heads > prism::kNormGateMaxHeads)
        return PRISM_EUNSUPPORTED;
    const int64_t es = size_of(d->dtype), all = d->rows * d->width * es;
    if (!apart({{y, all, true}}, {{o, all, true}, {z, all, true}, {w, (int64_t)d->heads * d->width * es}}))
        return PRISM_EINVAL;
    prism::NormGateArgs p = {};
    p.bf16 = d->dtype == PRISM_BF16;
    p.gate = gate;
    p.tokens = d->rows / d->heads;
    p.heads = d->heads;
    p.width = d->width;
    p.eps = eps;
    p.o = o; p.z = z; p.w = w;
    p.y = y;
    return from_hip(prism::launch_norm_gate(p, (hipStream_t)stream));
}

prism_status prism_norm_gate_bwd(const prism_norm_dims* d, const void* o, const void* z, const void* w,
                                 float eps, int gate, const void* dy, void* d_o, void* dz, float* dw,
                                 void* workspace, size_t workspace_bytes, void* stream)
{
    if (!norm_dims_ok(d) || !eps_ok(eps) || !gate_ok(gate))
        return PRISM_EINVAL;
    if (!row_ok(d, o) || !row_ok(d, z) || !ptr_ok(w) || !row_ok(d, dy) || !row_ok(d, d_o) || !row_ok(d, dz) ||
        !ptr_ok(dw) || !ptr_ok(workspace))
        return PRISM_EINVAL;
    if (d->width > prism::kNormGateMaxWidth || d->heads > prism::kNormGateMaxHeads)
        return PRISM_EUNSUPPORTED;
    const int64_t need = prism_norm_workspace_bytes(d);
    if (workspace_bytes < (size_t)need)
        return PRISM_EINVAL;
    const int64_t es = size_of(d->dtype), all = d->rows * d->width * es, nw = (int64_t)d->heads * d->width;
    if (!apart({{d_o, all, true}, {dz, all, true}, {dw, nw * 4}, {workspace, need}},
               {{o, all, true}, {z, all, true}, {dy, all, true}, {w, nw * es}}))
        return PRISM_EINVAL;
    prism::NormGateArgs p = {};
    p.bf16 = d->dtype == PRISM_BF16;
    p.gate = gate;
    p.tokens = d->rows / d->heads;
    p.heads = d->heads;
    p.width = d->width;
    p.eps = eps;
    p.o = o; p.z = z; p.w = w;
    p.dy = dy;
    p.d_o = d_o;
    p.dz = dz;
    p.dw = dw;
    p.ws = (float*)workspace;
    return from_hip(prism::launch_norm_gate_bwd(p, (hipStream_t)stream));
}

prism_status prism_decode_draft(const prism_dims* d, const void* q, const void* k, const void* v,
                                const void* u, const void* g, const void* b, const void* a, const void* h,
                                const void* conv_w, const int32_t* cu_seqlens, int L, int residual,
                                const float* S, const void* k_hist, void* o, float* kw, float* p_rec,
                                void* stream)
{
    if (!dims_ok(d) || L < 1 || L > PRISM_MAX_LEVELS || !residual_ok(residual))
        return PRISM_EINVAL;
    if (!tok_ok(d, q) || !tok_ok(d, k) || !tok_ok(d, v) || !tok_ok(d, g) || !tok_ok(d, b) || !ptr_ok(conv_w) ||
        !ptr_ok(cu_seqlens) || !ptr_ok(S) || !ptr_ok(k_hist) || !tok_ok(d, o) || !tok_ok(d, kw) ||
        !tok_ok(d, p_rec))
        return PRISM_EINVAL;
    if (L > 1 && (!tok_ok(d, u) || !tok_ok(d, a) || !tok_ok(d, h)))
        return PRISM_EINVAL;
    if (!draft_shape_ok(d, L > 1 ? L - 1 : 1) || d->total_tokens > (int64_t)d->n_seqs * PRISM_MAX_DRAFT)
        return PRISM_EUNSUPPORTED;
    const int64_t es = size_of(d->dtype), th = (int64_t)d->total_tokens * d->heads, nh = (int64_t)d->n_seqs * d->heads;
    const int64_t lev = L > 1 ? th * (L - 1) * d->dk * es : 0;
    if (!apart({{o, th * d->dv * es}, {kw, th * d->dk * 4}, {p_rec, th * d->dv * 4}},
               {{q, th * d->dk * es}, {k, th * d->dk * es}, {v, th * d->dv * es}, {u, lev}, {a, lev}, {h, lev},
                {g, th * es}, {b, th * es}, {conv_w, (int64_t)d->heads * d->dk * 4 * es},
                {cu_seqlens, ((int64_t)d->n_seqs + 1) * 4}, {S, nh * d->dk * d->dv * 4}, {k_hist, nh * 3 * d->dk * es}}))
        return PRISM_EINVAL;
    if (d->total_tokens == 0)
        return PRISM_OK;
    prism::DraftArgs p;
    p.bf16 = d->dtype == PRISM_BF16;
    p.n_seqs = d->n_seqs;
    p.heads = d->heads;
    p.dk = d->dk;
    p.dv = d->dv;
    p.L = L;
    p.gelu = residual == PRISM_RESIDUAL_GELU;
    p.q = q; p.k = k; p.v = v; p.u = u; p.a = a; p.h = h; p.g = g; p.b = b;
    p.conv_w = conv_w;
    p.cu_seqlens = cu_seqlens;
    p.S = S;
    p.k_hist = k_hist;
    p.o = o;
    p.kw = kw;
    p.p = p_rec;
    return from_hip(prism::launch_draft(p, (hipStream_t)stream));
}

prism_status prism_decode_commit(const prism_dims* d, const void* k, const void* v, const void* g,
                                 const void* b, const int32_t* cu_seqlens, const int32_t* n_accept,
                                 const float* kw, const float* p_rec, const float* S, const void* k_hist,
                                 float* S_out, void* k_hist_out, void* stream)
{
    if (!dims_ok(d))
        return PRISM_EINVAL;
    if (!tok_ok(d, k) || !tok_ok(d, v) || !tok_ok(d, g) || !tok_ok(d, b) || !ptr_ok(cu_seqlens) ||
        !ptr_ok(n_accept) || !tok_ok(d, kw) || !tok_ok(d, p_rec) || !ptr_ok(S) || !ptr_ok(k_hist) ||
        !ptr_ok(S_out) || !ptr_ok(k_hist_out))
        return PRISM_EINVAL;
    if (!draft_shape_ok(d, 1))
        return PRISM_EUNSUPPORTED;
    const int64_t es = size_of(d->dtype), th = (int64_t)d->total_tokens * d->heads, nh = (int64_t)d->n_seqs * d->heads;
    const int64_t state = nh * d->dk * d->dv * 4, hist = nh * 3 * d->dk * es;
    if (!apart({{S_out, state, true}, {k_hist_out, hist, true}},
               {{S, state, true}, {k_hist, hist, true}, {k, th * d->dk * es}, {v, th * d->dv * es}, {g, th * es},
                {b, th * es}, {kw, th * d->dk * 4}, {p_rec, th * d->dv * 4}, {n_accept, (int64_t)d->n_seqs * 4},
                {cu_seqlens, ((int64_t)d->n_seqs + 1) * 4}}))
        return PRISM_EINVAL;
    prism::DraftArgs p;
    p.bf16 = d->dtype == PRISM_BF16;
    p.n_seqs = d->n_seqs;
    p.heads = d->heads;
    p.dk = d->dk;
    p.dv = d->dv;
    p.k = k; p.v = v; p.g = g; p.b = b;
    p.cu_seqlens = cu_seqlens;
    p.S = S;
    p.k_hist = k_hist;
    p.kw = const_cast<float*>(kw);
    p.p = const_cast<float*>(p_rec);
    p.n_accept = n_accept;
    p.S_out = S_out;
    p.k_hist_out = k_hist_out;
    return from_hip(prism::launch_commit(p, (hipStream_t)stream));
}

size_t prism_verify_workspace_bytes(const prism_verify_dims* d)
{
    return verify_dims_ok(d) ? round256(prism::verify_workspace_bytes(d->n_seqs, d->vocab)) : 0;
}

prism_status prism_verify_draft(const prism_verify_dims* d, const void* p, const void* q,
                                const int32_t* tokens, const int32_t* cu_seqlens, const float* u_accept,
                                const float* u_sample, int32_t* n_accept, int32_t* next_token,
                                void* workspace, size_t workspace_bytes, void* stream)
{
    if (!verify_dims_ok(d))
        return PRISM_EINVAL;
    const bool none = d->total_tokens == 0;              // then the per-token arrays may be null
    if (!(none ? aligned16(p) : ptr_ok(p)) || !opt_ok(q) || !(none ? aligned16(tokens) : ptr_ok(tokens)) ||
        !ptr_ok(cu_seqlens) || !(none ? aligned16(u_accept) : ptr_ok(u_accept)) || !ptr_ok(u_sample) ||
        !ptr_ok(n_accept) || !ptr_ok(next_token))
        return PRISM_EINVAL;
    const size_t need = prism_verify_workspace_bytes(d);
    if (need > 0 ? !ptr_ok(workspace) || workspace_bytes < need : !opt_ok(workspace))
        return PRISM_EINVAL;
    if (d->vocab > (1 << 28) || !grid_ok((int64_t)d->n_seqs * prism::verify_chunks(d->vocab), 1024))
        return PRISM_EUNSUPPORTED;
    const int64_t rows = (int64_t)d->total_tokens * d->vocab * size_of(d->dtype), each = (int64_t)d->n_seqs * 4;
    if (!apart({{n_accept, each}, {next_token, each}, {workspace, (int64_t)need}},
               {{p, rows}, {q, rows}, {tokens, (int64_t)d->total_tokens * 4}, {u_accept, (int64_t)d->total_tokens * 4},
                {u_sample, each}, {cu_seqlens, each + 4}}))
        return PRISM_EINVAL;
    prism::VerifyArgs a;
    a.bf16 = d->dtype == PRISM_BF16;
    a.n_seqs = d->n_seqs;
    a.total_tokens = d->total_tokens;
    a.vocab = d->vocab;
    a.p = p; a.q = q;
    a.tokens = tokens;
    a.cu_seqlens = cu_seqlens;
    a.u_accept = u_accept;
    a.u_sample = u_sample;
    a.n_accept = n_accept;
    a.next_token = next_token;
    a.ws = workspace;
    return from_hip(prism::launch_verify(a, (hipStream_t)stream));
}

}  // extern "C"
