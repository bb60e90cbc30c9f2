// stack_api.hip -- C ABI of the operators in front of the memory-writing operator and behind
// the model's last product (declared in include/prism.h): the short convolution, the norm and
// rotation of queries and keys, the choice of a token.  Argument checks and launches on the
// caller's stream.
#include "api_checks.h"
#include "kernels.h"
#include "prism.h"

namespace {

bool dtype_ok(int dtype) { return dtype == PRISM_F32 || dtype == PRISM_BF16; }

// Elements from the first to the last of `count` rows of `width`, `stride` apart.
int64_t extent(int64_t count, int64_t stride, int64_t width) { return count > 0 ? (count - 1) * stride + width : 0; }

// A stride whose rows stay within 2^59 elements.
bool stride_ok(int64_t count, int64_t stride)
{
    return stride >= 0 && (count < 2 || stride <= ((int64_t)1 << 59) / (count - 1));
}

bool conv_dims_ok(const prism_conv_dims* d)
{
    return d && d->n_seqs >= 1 && d->total_tokens >= 0 && d->channels >= 1 && d->taps >= 1 &&
           d->taps <= PRISM_MAX_TAPS && dtype_ok(d->dtype) && stride_ok(d->total_tokens, d->x_stride);
}

bool act_ok(int a) { return a == PRISM_ACT_NONE || a == PRISM_ACT_SILU; }

bool conv_fits(const prism_conv_dims* d)
{
    return d->channels <= 1 << 22 && d->total_tokens <= 1 << 30 &&
           grid_ok(prism::short_conv_blocks(d->total_tokens, d->n_seqs, d->channels, d->dtype == PRISM_BF16, d->taps), 256);
}

struct ConvSizes {
    int64_t x, y, w, c, hist, cu;
    explicit ConvSizes(const prism_conv_dims* d)
    {
        const int64_t es = size_of(d->dtype), C = d->channels;
        x = extent(d->total_tokens, d->x_stride, C) * es;
        y = (int64_t)d->total_tokens * C * es;
        w = C * d->taps * es;
        c = C * es;
        hist = (int64_t)d->n_seqs * (d->taps - 1) * C * es;
        cu = ((int64_t)d->n_seqs + 1) * 4;
    }
};

prism::ShortConvArgs conv_args(const prism_conv_dims* d, const void* x, const void* w, const void* bias,
                               const void* hist, const int32_t* cu, int activation)
{
    prism::ShortConvArgs p = {};
    p.bf16 = d->dtype == PRISM_BF16;
    p.silu = activation == PRISM_ACT_SILU;
    p.n_seqs = d->n_seqs;
    p.total_tokens = d->total_tokens;
    p.channels = d->channels;
    p.taps = d->taps;
    p.x_stride = d->x_stride;
    p.x = x; p.w = w; p.bias = bias;
    p.hist = d->taps > 1 ? hist : nullptr;
    p.cu_seqlens = cu;
    return p;
}

bool qk_dims_ok(const prism_qk_dims* d)
{
    return d && d->tokens >= 0 && d->tokens <= (int64_t)1 << 40 && d->heads_q >= 1 && d->heads_k >= 0 && d->width >= 1 &&
           d->rot >= 0 && d->rot % 2 == 0 && d->rot <= d->width && dtype_ok(d->dtype) &&
           stride_ok(d->tokens, d->q_stride) && stride_ok(d->heads_q, d->q_head_stride) &&
           stride_ok(d->tokens, d->k_stride) && stride_ok(d->heads_k, d->k_head_stride);
}

bool qk_fits(const prism_qk_dims* d)
{
    const auto near = [](int64_t stride) { return stride <= UINT32_MAX; };
    return d->width <= prism::kQkMaxWidth && d->heads_q <= 65535 && d->heads_k <= 65535 && near(d->q_stride) &&
           near(d->q_head_stride) && near(d->k_stride) && near(d->k_head_stride) && grid_ok(2 * d->tokens, 256);
}

struct QkSizes {
    int64_t in[2], out[2], w;
    bool dense[2];
    explicit QkSizes(const prism_qk_dims* d)
    {
        const int64_t es = size_of(d->dtype), heads[2] = {d->heads_q, d->heads_k};
        const int64_t st[2] = {d->q_stride, d->k_stride}, hs[2] = {d->q_head_stride, d->k_head_stride};
        for (int i = 0; i < 2; ++i) {
            in[i] = d->tokens > 0 && heads[i] > 0 ? extent(d->tokens, st[i], extent(heads[i], hs[i], d->width)) * es : 0;
            out[i] = d->tokens * heads[i] * d->width * es;
            dense[i] = (heads[i] < 2 || hs[i] == d->width) && (d->tokens < 2 || st[i] == heads[i] * d->width);
        }
        w = d->width * es;
    }
};

// The checks that both passes share.
prism_status qk_check(const prism_qk_dims* d, const void* q, const void* k, const void* wq, const void* wk, int norm,
                      float eps, const int32_t* positions, const float* freqs, int layout)
{
    if (!qk_dims_ok(d) || !eps_ok(eps) || norm < PRISM_QK_NONE || norm > PRISM_QK_L2 ||
        (layout != PRISM_ROT_HALF && layout != PRISM_ROT_INTERLEAVED))
        return PRISM_EINVAL;
    if (d->heads_k > 0 ? !wq != !wk : k || wk)
        return PRISM_EINVAL;
    if (!opt_ok(wq) || !opt_ok(wk) || !opt_ok(positions) || !opt_ok(freqs) || (d->rot > 0 && !freqs))
        return PRISM_EINVAL;
    if (d->tokens > 0 && (!elem_ok(q, d->dtype) || (d->heads_k > 0 && !elem_ok(k, d->dtype)) || (d->rot > 0 && !positions)))
        return PRISM_EINVAL;
    return qk_fits(d) ? PRISM_OK : PRISM_EUNSUPPORTED;
}

prism::QkNormArgs qk_args(const prism_qk_dims* d, const void* q, const void* k, const void* wq, const void* wk,
                          int norm, float eps, const int32_t* positions, const float* freqs, int layout, float rot_scale)
{
    prism::QkNormArgs p = {};
    p.bf16 = d->dtype == PRISM_BF16;
    p.norm = norm;
    p.interleaved = layout == PRISM_ROT_INTERLEAVED;
    p.tokens = d->tokens;
    p.heads[0] = d->heads_q; p.heads[1] = d->heads_k;
    p.width = d->width;
    p.rot = d->rot;
    p.eps = eps;
    p.rot_scale = rot_scale;
    p.stride[0] = d->q_stride; p.stride[1] = d->k_stride;
    p.head_stride[0] = d->q_head_stride; p.head_stride[1] = d->k_head_stride;
    p.x[0] = q; p.x[1] = k;
    p.w[0] = wq; p.w[1] = wk;
    p.positions = positions;
    p.freqs = freqs;
    return p;
}

bool sample_dims_ok(const prism_sample_dims* d)
{
    return d && d->rows >= 0 && d->rows <= (int64_t)1 << 40 && d->vocab >= 1 && dtype_ok(d->dtype) &&
           stride_ok(d->rows, d->stride);
}

bool sample_fits(const prism_sample_dims* d)
{
    return d->vocab <= PRISM_MAX_SAMPLE_VOCAB && prism::sample_fits(d->rows);
}

}  // namespace

extern "C" {

size_t prism_conv_workspace_bytes(const prism_conv_dims* d)
{
    if (!conv_dims_ok(d) || !conv_fits(d))
        return 0;
    const int nb = prism::short_conv_bwd_blocks(d->total_tokens, d->channels, d->dtype == PRISM_BF16, d->taps);
    return round256((size_t)nb * d->channels * (d->taps + 1) * sizeof(float));
}

prism_status prism_short_conv_ex(const prism_conv_dims* d, const void* x, const void* w, const void* bias,
                                 const void* hist, const int32_t* cu_seqlens, int activation, int clear_behind, void* y,
                                 void* hist_out, void* stream)
{
    if (!conv_dims_ok(d) || !act_ok(activation) || clear_behind < 0 || clear_behind > 1)
        return PRISM_EINVAL;
    if (!ptr_ok(w) || !opt_ok(bias) || !opt_ok(hist) || !ptr_ok(cu_seqlens) || !opt_ok(y) || !opt_ok(hist_out))
        return PRISM_EINVAL;
    if (d->total_tokens > 0 && (!elem_ok(x, d->dtype) || !y))
        return PRISM_EINVAL;
    if (!conv_fits(d))
        return PRISM_EUNSUPPORTED;
    const ConvSizes z(d);
    if (!apart({{y, z.y}, {hist_out, z.hist, true}},
               {{x, z.x}, {w, z.w}, {bias, z.c}, {hist, z.hist, true}, {cu_seqlens, z.cu}}))
        return PRISM_EINVAL;
    prism::ShortConvArgs p = conv_args(d, x, w, bias, hist, cu_seqlens, activation);
    p.y = y;
    p.hist_out = hist_out;
    p.clear_behind = clear_behind;
    return from_hip(prism::launch_short_conv(p, (hipStream_t)stream));
}

prism_status prism_short_conv(const prism_conv_dims* d, const void* x, const void* w, const void* bias,
                              const void* hist, const int32_t* cu_seqlens, int activation, void* y, void* hist_out,
                              void* stream)
{
    return prism_short_conv_ex(d, x, w, bias, hist, cu_seqlens, activation, 0, y, hist_out, stream);
}

prism_status prism_short_conv_step(const prism_conv_dims* d, const void* x, const void* w, const void* bias,
                                   const void* hist, int activation, void* y, void* hist_out, void* stream)
{
    if (!conv_dims_ok(d) || !act_ok(activation) || d->total_tokens != d->n_seqs)
        return PRISM_EINVAL;
    if (!elem_ok(x, d->dtype) || !ptr_ok(w) || !opt_ok(bias) || !ptr_ok(y) || !opt_ok(hist) || !opt_ok(hist_out))
        return PRISM_EINVAL;
    if (d->taps > 1 && (!hist || !hist_out))
        return PRISM_EINVAL;
    if (!conv_fits(d))
        return PRISM_EUNSUPPORTED;
    const ConvSizes z(d);
    if (!apart({{y, z.y}, {hist_out, z.hist, true}}, {{x, z.x}, {w, z.w}, {bias, z.c}, {hist, z.hist, true}}))
        return PRISM_EINVAL;
    prism::ShortConvArgs p = conv_args(d, x, w, bias, hist, nullptr, activation);
    p.y = y;
    p.hist_out = hist_out;
    return from_hip(prism::launch_short_conv_step(p, (hipStream_t)stream));
}

prism_status prism_short_conv_bwd(const prism_conv_dims* d, const void* x, const void* w, const void* bias,
                                  const void* hist, const int32_t* cu_seqlens, int activation, const void* dy,
                                  void* dx, float* dw, float* dbias, void* dhist, void* workspace,
                                  size_t workspace_bytes, void* stream)
{
    if (!conv_dims_ok(d) || !act_ok(activation))
        return PRISM_EINVAL;
    if (!ptr_ok(w) || !opt_ok(bias) || !opt_ok(hist) || !ptr_ok(cu_seqlens) || !opt_ok(dy) || !opt_ok(dx) ||
        !ptr_ok(dw) || !opt_ok(dbias) || !opt_ok(dhist))
        return PRISM_EINVAL;
    if (d->total_tokens > 0 && (!elem_ok(x, d->dtype) || !dy || !dx))
        return PRISM_EINVAL;
    if (!conv_fits(d))
        return PRISM_EUNSUPPORTED;
    const size_t need = prism_conv_workspace_bytes(d);
    if (!ptr_ok(workspace) || workspace_bytes < need)
        return PRISM_EINVAL;
    const ConvSizes z(d);
    const int64_t C = d->channels;
    if (!apart({{dx, z.y}, {dw, C * d->taps * 4}, {dbias, C * 4}, {dhist, z.hist}, {workspace, (int64_t)need}},
               {{x, z.x}, {w, z.w}, {bias, z.c}, {hist, z.hist}, {cu_seqlens, z.cu}, {dy, z.y}}))
        return PRISM_EINVAL;
    prism::ShortConvArgs p = conv_args(d, x, w, bias, hist, cu_seqlens, activation);
    p.dy = dy;
    p.dx = dx;
    p.dw = dw;
    p.dbias = dbias;
    p.dhist = dhist;
    p.ws = (float*)workspace;
    return from_hip(prism::launch_short_conv_bwd(p, (hipStream_t)stream));
}

size_t prism_qk_workspace_bytes(const prism_qk_dims* d)
{
    if (!qk_dims_ok(d) || !qk_fits(d))
        return 0;
    return round256((size_t)prism::qk_norm_bwd_blocks(d->tokens) * (d->heads_k > 0 ? 2 : 1) * d->width * sizeof(float));
}

prism_status prism_qk_norm(const prism_qk_dims* d, const void* q, const void* k, const void* wq, const void* wk,
                           int norm, float eps, const int32_t* positions, const float* freqs, int layout,
                           float rot_scale, void* q_out, void* k_out, void* stream)
{
    const prism_status s = qk_check(d, q, k, wq, wk, norm, eps, positions, freqs, layout);
    if (s != PRISM_OK)
        return s;
    if (!opt_ok(q_out) || !opt_ok(k_out) || (d->tokens > 0 && (!q_out || (d->heads_k > 0 && !k_out))))
        return PRISM_EINVAL;
    const QkSizes z(d);
    if (!apart({{q_out, z.out[0], true}, {k_out, z.out[1], true}},
               {{q, z.in[0], z.dense[0]}, {k, z.in[1], z.dense[1]}, {wq, z.w}, {wk, z.w}, {positions, d->tokens * 4},
                {freqs, (int64_t)d->rot / 2 * 4}}) ||
        (q_out && q_out == k) || (k_out && k_out == q))
        return PRISM_EINVAL;
    prism::QkNormArgs p = qk_args(d, q, k, wq, wk, norm, eps, positions, freqs, layout, rot_scale);
    p.y[0] = q_out;
    p.y[1] = k_out;
    return from_hip(prism::launch_qk_norm(p, (hipStream_t)stream));
}

prism_status prism_qk_norm_bwd(const prism_qk_dims* d, const void* q, const void* k, const void* wq, const void* wk,
                               int norm, float eps, const int32_t* positions, const float* freqs, int layout,
                               float rot_scale, const void* dq_out, const void* dk_out, void* dq, void* dk, float* dwq,
                               float* dwk, void* workspace, size_t workspace_bytes, void* stream)
{
    const prism_status s = qk_check(d, q, k, wq, wk, norm, eps, positions, freqs, layout);
    if (s != PRISM_OK)
        return s;
    const bool has_k = d->heads_k > 0;
    if (!opt_ok(dq_out) || !opt_ok(dk_out) || !opt_ok(dq) || !opt_ok(dk) || !opt_ok(dwq) || !opt_ok(dwk))
        return PRISM_EINVAL;
    if (d->tokens > 0 && (!dq_out || !dq || (has_k && (!dk_out || !dk))))
        return PRISM_EINVAL;
    if (!dwq != !wq || !dwk != !wk)
        return PRISM_EINVAL;
    const size_t need = prism_qk_workspace_bytes(d);
    if (wq ? !ptr_ok(workspace) || workspace_bytes < need : !opt_ok(workspace))
        return PRISM_EINVAL;
    const QkSizes z(d);
    if (!apart({{dq, z.out[0], true}, {dk, z.out[1], true}, {dwq, (int64_t)d->width * 4}, {dwk, (int64_t)d->width * 4},
                {workspace, wq ? (int64_t)need : 0}},
               {{q, z.in[0]}, {k, z.in[1]}, {wq, z.w}, {wk, z.w}, {positions, d->tokens * 4},
                {freqs, (int64_t)d->rot / 2 * 4}, {dq_out, z.out[0], true}, {dk_out, z.out[1], true}}) ||
        (dq && dq == dk_out) || (dk && dk == dq_out))
        return PRISM_EINVAL;
    prism::QkNormArgs p = qk_args(d, q, k, wq, wk, norm, eps, positions, freqs, layout, rot_scale);
    p.dy[0] = dq_out; p.dy[1] = dk_out;
    p.dx[0] = dq; p.dx[1] = dk;
    p.dw[0] = dwq; p.dw[1] = dwk;
    p.ws = (float*)workspace;
    return from_hip(prism::launch_qk_norm_bwd(p, (hipStream_t)stream));
}

size_t prism_sample_workspace_bytes(const prism_sample_dims* d)
{
    return sample_dims_ok(d) && sample_fits(d) ? round256(prism::sample_workspace_bytes(d->rows, d->vocab)) : 0;
}

prism_status prism_sample(const prism_sample_dims* d, const void* logits, const float* temperature,
                          const int32_t* top_k, const float* top_p, const float* min_p, const float* u,
                          int32_t* tokens, float* probs, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!sample_dims_ok(d))
        return PRISM_EINVAL;
    if (!opt_ok(temperature) || !opt_ok(top_k) || !opt_ok(top_p) || !opt_ok(min_p) || !opt_ok(u) || !opt_ok(tokens) ||
        !opt_ok(probs))
        return PRISM_EINVAL;
    if (d->rows > 0 && (!elem_ok(logits, d->dtype) || (!tokens && !probs) || (tokens && !u)))
        return PRISM_EINVAL;
    if (!sample_fits(d))
        return PRISM_EUNSUPPORTED;
    const size_t need = prism_sample_workspace_bytes(d);
    if (need > 0 ? !ptr_ok(workspace) || workspace_bytes < need : !opt_ok(workspace))
        return PRISM_EINVAL;
    const int64_t each = d->rows * 4;
    if (!apart({{tokens, each}, {probs, each * d->vocab}, {workspace, (int64_t)need}},
               {{logits, extent(d->rows, d->stride, d->vocab) * size_of(d->dtype)}, {temperature, each}, {top_k, each},
                {top_p, each}, {min_p, each}, {u, each}}))
        return PRISM_EINVAL;
    prism::SampleArgs p = {};
    p.bf16 = d->dtype == PRISM_BF16;
    p.rows = d->rows;
    p.vocab = d->vocab;
    p.stride = d->stride;
    p.logits = logits;
    p.temperature = temperature;
    p.top_k = top_k;
    p.top_p = top_p; p.min_p = min_p;
    p.u = u;
    p.tokens = tokens;
    p.probs = probs;
    p.ws = workspace;
    return from_hip(prism::launch_sample(p, (hipStream_t)stream));
}

}  // extern "C"
