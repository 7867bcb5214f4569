// kda_layer_api.cu -- extern "C" boundary of the layer around the recurrences (selective scan,
// short convolution with a bias and its backward, residual norms): host-side validation and
// dispatch. Nothing here allocates device memory or synchronises.
#include <stdint.h>

#include "kda_layer.cuh"

namespace {

bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <typename... P> bool aligned16(const P *...p) { return (aligned(p, 16) && ...); }
template <typename... P> bool aligned4(const P *...p) { return (aligned(p, 4) && ...); }

bool known_dtype(kda_dtype t) { return t == KDA_DTYPE_F32 || t == KDA_DTYPE_BF16; }

// Sizes that every selective scan call shares; `rows` is the number of tokens.
kda_status check_ssm_sizes(int32_t num_seqs, int64_t rows, int32_t channels, int32_t states, int32_t groups) {
    if (num_seqs < 1 || num_seqs > 65535 || rows < 0) return KDA_ERR_INVALID_ARG;
    if (channels < 1 || groups < 1 || states < 1) return KDA_ERR_INVALID_ARG;
    if (channels % groups || channels / groups % 8) return KDA_ERR_UNSUPPORTED;
    if (states != 8 && states != 16 && states != 32 && states != 64 && states != 128) return KDA_ERR_UNSUPPORTED;
    if (rows > INT32_MAX || channels > 65536) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}
kda_status check_ssm(const kda_ssm *p, int32_t num_seqs, int64_t rows, kda_dtype dtype, uint32_t flags) {
    if (!p || !known_dtype(dtype) || (flags & ~(uint32_t)KDA_FLAG_SOFTPLUS)) return KDA_ERR_INVALID_ARG;
    if (kda_status rc = check_ssm_sizes(num_seqs, rows, p->channels, p->states, p->groups); rc != KDA_OK) return rc;
    if (!p->A) return KDA_ERR_INVALID_ARG;
    if (!aligned16(p->A) || !aligned4(p->D, p->dt_bias)) return KDA_ERR_MISALIGNED;
    return KDA_OK;
}

kda::SsmArgs ssm_args(const void *x, const void *dt, const void *B, const void *C, const void *z, const kda_ssm *p,
                      int32_t N, int64_t total, uint32_t flags) {
    kda::SsmArgs a{};
    a.x = x; a.dt = dt; a.B = B; a.C = C; a.z = z;
    a.A = p->A; a.D = p->D; a.dt_bias = p->dt_bias;
    a.N = N; a.total = total;
    a.channels = p->channels; a.states = p->states; a.groups = p->groups;
    a.softplus = (flags & KDA_FLAG_SOFTPLUS) != 0;
    return a;
}

// What every short convolution call shares.
kda_status check_conv(const kda_short_conv *conv, const float *bias, int32_t num_seqs, int64_t rows, int32_t channels,
                      kda_dtype dtype) {
    if (!conv || num_seqs < 1 || rows < 0 || channels < 8 || channels % 8 || !known_dtype(dtype)) return KDA_ERR_INVALID_ARG;
    if (conv->width < 1 || conv->width > KDA_MAX_CONV_WIDTH) return KDA_ERR_UNSUPPORTED;
    if (num_seqs > 65535 || rows > INT32_MAX || channels > (1 << 20)) return KDA_ERR_UNSUPPORTED;
    if (rows > 0 && !conv->weight) return KDA_ERR_INVALID_ARG;
    if (!aligned16(conv->state_in, conv->state_out) || !aligned4(conv->weight, bias)) return KDA_ERR_MISALIGNED;
    return KDA_OK;
}

kda::ConvArgs conv_args(const void *x, void *y, const kda_short_conv *conv, const float *bias, const int32_t *cu,
                        int32_t N, int64_t total, int32_t C) {
    kda::ConvArgs a{};
    a.x = x; a.y = y; a.w = conv->weight; a.bias = bias;
    a.state_in = conv->state_in; a.state_out = conv->state_out;
    a.cu = cu; a.N = N; a.total = total; a.C = C; a.W = conv->width;
    return a;
}

bool overlap(const void *p, size_t np, const void *q, size_t nq) {  // p's np bytes and q's nq bytes
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + nq && b < a + np;
}
size_t size_of(kda_dtype t) { return t == KDA_DTYPE_BF16 ? 2 : 4; }

kda_status check_norm(const kda_residual_norm_args *a) {
    if (!a || a->rows < 0 || a->D < 8 || a->D % 8 || !known_dtype(a->dtype) || !known_dtype(a->res_dtype)) return KDA_ERR_INVALID_ARG;
    if (!(a->eps > 0.f)) return KDA_ERR_INVALID_ARG;
    if (a->D > KDA_MAX_NORM_CHANNELS || a->rows > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (a->res_dtype != a->dtype && a->res_dtype != KDA_DTYPE_F32) return KDA_ERR_UNSUPPORTED;
    if (a->rows > 0 && !a->y) return KDA_ERR_INVALID_ARG;
    if (!aligned16(a->y, a->r, a->gate, a->w_post, a->scale, a->w_pre)) return KDA_ERR_MISALIGNED;
    return KDA_OK;
}
kda::NormArgs norm_args(const kda_residual_norm_args *p) {
    kda::NormArgs a{};
    a.y = p->y; a.r = p->r; a.gate = p->gate;
    a.w_post = p->w_post; a.scale = p->scale; a.w_pre = p->w_pre;
    a.res_scale = p->res_scale; a.eps = p->eps;
    a.rows = p->rows; a.D = p->D;
    a.res_bf16 = p->res_dtype == KDA_DTYPE_BF16;
    return a;
}

kda_status done(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

}  // namespace

extern "C" {

size_t kda_ssm_tile_states_size(int32_t num_seqs, int64_t total_tokens, int32_t channels, int32_t states) {
    if (num_seqs < 1 || total_tokens < 0 || channels < 1 || states < 1) return 0;
    return (size_t)kda::ssm_tile0(total_tokens, num_seqs) * channels * states * sizeof(float);
}

size_t kda_ssm_prefill_workspace_size(int32_t num_seqs, int64_t total_tokens, int32_t channels, int32_t states,
                                      int32_t groups) {
    if (check_ssm_sizes(num_seqs, total_tokens, channels, states, groups) != KDA_OK) return 0;
    return kda::ssm_prefill_workspace(total_tokens, num_seqs, channels, states, groups);
}

int64_t kda_ssm_prefill_launches(int32_t num_seqs, int64_t total_tokens, int32_t channels, int32_t states,
                                 int32_t groups) {
    if (check_ssm_sizes(num_seqs, total_tokens, channels, states, groups) != KDA_OK) return -1;
    return kda::ssm_prefill_launches(total_tokens, num_seqs, channels, states, groups);
}

kda_status kda_ssm_prefill(const void *x, const void *dt, const void *B, const void *C, const void *z, const kda_ssm *ssm,
                           const float *S0, const int32_t *cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                           kda_dtype dtype, uint32_t flags, void *y, float *S_T, float *tile_states, void *workspace,
                           size_t workspace_bytes, kda_stream_t stream) {
    if (kda_status rc = check_ssm(ssm, num_seqs, total_tokens, dtype, flags); rc != KDA_OK) return rc;
    if (!cu_seqlens && num_seqs != 1) return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0 && (!x || !dt || !B || !C || !y)) return KDA_ERR_INVALID_ARG;
    const size_t need = kda::ssm_prefill_workspace(total_tokens, num_seqs, ssm->channels, ssm->states, ssm->groups);
    if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    if (!aligned16(x, dt, B, C, z, S0, cu_seqlens, y, S_T, tile_states, workspace)) return KDA_ERR_MISALIGNED;
    kda::SsmArgs a = ssm_args(x, dt, B, C, z, ssm, num_seqs, total_tokens, flags);
    a.S0 = S0; a.cu = cu_seqlens; a.y = y; a.S_T = S_T; a.tiles = tile_states;
    return done(kda::ssm_prefill(a, workspace, dtype == KDA_DTYPE_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_ssm_step(const void *x, const void *dt, const void *B, const void *C, const void *z, const kda_ssm *ssm,
                        float *S, int32_t N, kda_dtype dtype, uint32_t flags, void *y, kda_stream_t stream) {
    if (N < 1) return KDA_ERR_INVALID_ARG;
    if (kda_status rc = check_ssm(ssm, 1, N, dtype, flags); rc != KDA_OK) return rc;
    if (!x || !dt || !B || !C || !S || !y) return KDA_ERR_INVALID_ARG;
    if (!aligned16(x, dt, B, C, z, S, y)) return KDA_ERR_MISALIGNED;
    kda::SsmArgs a = ssm_args(x, dt, B, C, z, ssm, N, N, flags);
    a.S_T = S; a.y = y;
    return done(kda::ssm_step(a, dtype == KDA_DTYPE_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_ssm_backward_workspace_size(int32_t num_seqs, int64_t total_tokens, int32_t channels, int32_t states,
                                       int32_t groups) {
    if (check_ssm_sizes(num_seqs, total_tokens, channels, states, groups) != KDA_OK) return 0;
    return kda::ssm_backward_workspace(total_tokens, num_seqs, channels, states, groups);
}

kda_status kda_ssm_backward(const void *x, const void *dt, const void *B, const void *C, const void *z,
                            const kda_ssm *ssm, const float *S0, const int32_t *cu_seqlens, int32_t num_seqs,
                            int64_t total_tokens, kda_dtype dtype, uint32_t flags, const float *tile_states,
                            const void *dy, const float *dS_T, const kda_ssm_grads *grads, void *workspace,
                            size_t workspace_bytes, kda_stream_t stream) {
    if (kda_status rc = check_ssm(ssm, num_seqs, total_tokens, dtype, flags); rc != KDA_OK) return rc;
    if (!grads || !grads->dA || (!cu_seqlens && num_seqs != 1)) return KDA_ERR_INVALID_ARG;
    const kda_ssm_grads &o = *grads;
    if (total_tokens > 0 && (!x || !dt || !B || !C || !dy || !tile_states || !o.dx || !o.ddt || !o.dB || !o.dC ||
                             (z != nullptr) != (o.dz != nullptr)))
        return KDA_ERR_INVALID_ARG;
    const size_t need = kda::ssm_backward_workspace(total_tokens, num_seqs, ssm->channels, ssm->states, ssm->groups);
    if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
    if (!aligned16(x, dt, B, C, z, S0, cu_seqlens, tile_states, dy, dS_T, workspace) ||
        !aligned16(o.dx, o.ddt, o.dB, o.dC, o.dz, o.dA, o.dS0) || !aligned4(o.dD, o.ddt_bias))
        return KDA_ERR_MISALIGNED;
    kda::SsmBackwardArgs g{};
    g.f = ssm_args(x, dt, B, C, z, ssm, num_seqs, total_tokens, flags);
    g.f.S0 = S0; g.f.cu = cu_seqlens;
    g.f.tiles = const_cast<float *>(tile_states);
    g.dy = dy; g.dS_T = dS_T;
    g.dx = o.dx; g.ddt = o.ddt; g.dB = o.dB; g.dC = o.dC; g.dz = o.dz;
    g.dA = o.dA; g.dD = o.dD; g.ddt_bias = o.ddt_bias; g.dS0 = o.dS0;
    g.ws = workspace;
    return done(kda::ssm_backward(g, dtype == KDA_DTYPE_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_short_conv_swish_ex(const void *x, void *y, const kda_short_conv *conv, const float *bias,
                                   const int32_t *cu_seqlens, int32_t num_seqs, int64_t total_tokens, int32_t channels,
                                   kda_dtype dtype, kda_stream_t stream) {
    if (kda_status rc = check_conv(conv, bias, num_seqs, total_tokens, channels, dtype); rc != KDA_OK) return rc;
    if (!cu_seqlens && num_seqs != 1) return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0 && (!x || !y)) return KDA_ERR_INVALID_ARG;
    if (!aligned16(x, y, cu_seqlens)) return KDA_ERR_MISALIGNED;
    const size_t bytes = (size_t)total_tokens * channels * size_of(dtype);
    if (total_tokens > 0 && overlap(x, bytes, y, bytes)) return KDA_ERR_INVALID_ARG;
    return done(kda::conv_bias(conv_args(x, y, conv, bias, cu_seqlens, num_seqs, total_tokens, channels),
                               dtype == KDA_DTYPE_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_short_conv_step(const void *x, void *y, const kda_short_conv *conv, const float *bias, int32_t N,
                               int32_t channels, kda_dtype dtype, kda_stream_t stream) {
    if (N < 1) return KDA_ERR_INVALID_ARG;
    if (kda_status rc = check_conv(conv, bias, 1, N, channels, dtype); rc != KDA_OK) return rc;
    if (!x || !y || (conv->width > 1 && !conv->state_out)) return KDA_ERR_INVALID_ARG;
    if (!aligned16(x, y)) return KDA_ERR_MISALIGNED;
    const size_t bytes = (size_t)N * channels * size_of(dtype);
    if (overlap(x, bytes, y, bytes)) return KDA_ERR_INVALID_ARG;
    if (conv->width > 1) {  // the window is shifted while x is read and y is written
        const size_t state = (conv->width - 1) * bytes;
        if (overlap(x, bytes, conv->state_out, state) || overlap(y, bytes, conv->state_out, state)) return KDA_ERR_INVALID_ARG;
    }
    return done(kda::conv_step(conv_args(x, y, conv, bias, nullptr, N, N, channels), dtype == KDA_DTYPE_BF16,
                               reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_short_conv_backward_workspace_size(int64_t total_tokens, int32_t channels, int32_t width) {
    if (total_tokens < 0 || channels < 8 || channels % 8 || width < 1 || width > KDA_MAX_CONV_WIDTH) return 0;
    return kda::conv_backward_workspace(total_tokens, channels, width);
}

kda_status kda_short_conv_backward(const void *x, const kda_short_conv *conv, const float *bias,
                                   const int32_t *cu_seqlens, int32_t num_seqs, int64_t total_tokens, int32_t channels,
                                   kda_dtype dtype, const void *dy, kda_dtype dy_dtype, float *dx, float *dweight,
                                   float *dbias, float *dstate, void *workspace, size_t workspace_bytes,
                                   kda_stream_t stream) {
    if (kda_status rc = check_conv(conv, bias, num_seqs, total_tokens, channels, dtype); rc != KDA_OK) return rc;
    if (!cu_seqlens && num_seqs != 1) return KDA_ERR_INVALID_ARG;
    if (!known_dtype(dy_dtype) || !dweight || (total_tokens > 0 && (!x || !dy || !dx))) return KDA_ERR_INVALID_ARG;
    if (dy_dtype != dtype && dy_dtype != KDA_DTYPE_F32) return KDA_ERR_UNSUPPORTED;
    const size_t need = kda::conv_backward_workspace(total_tokens, channels, conv->width);
    if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    if (!aligned16(x, dy, dx, dstate, workspace, cu_seqlens) || !aligned4(dweight, dbias)) return KDA_ERR_MISALIGNED;
    if (total_tokens > 0) {  // a run of tokens reads the rows around it: dx in their place would change them
        const size_t n = (size_t)total_tokens * channels;
        if (overlap(dx, n * sizeof(float), x, n * size_of(dtype)) || overlap(dx, n * sizeof(float), dy, n * size_of(dy_dtype)))
            return KDA_ERR_INVALID_ARG;
    }
    kda::ConvBackwardArgs p{};
    p.f = conv_args(x, nullptr, conv, bias, cu_seqlens, num_seqs, total_tokens, channels);
    p.dy = dy; p.dy_bf16 = dy_dtype == KDA_DTYPE_BF16;
    p.dx = dx; p.dw = dweight; p.dbias = dbias; p.dstate = dstate; p.ws = workspace;
    return done(kda::conv_backward(p, dtype == KDA_DTYPE_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_residual_norm(const kda_residual_norm_args *args, void *x, void *r_out, kda_stream_t stream) {
    if (kda_status rc = check_norm(args); rc != KDA_OK) return rc;
    if ((x != nullptr) != (args->w_pre != nullptr) && args->rows > 0) return KDA_ERR_INVALID_ARG;
    if (args->rows > 0 && !r_out) return KDA_ERR_INVALID_ARG;
    if (!aligned16(x, r_out)) return KDA_ERR_MISALIGNED;
    kda::NormArgs a = norm_args(args);
    a.x = x; a.r_out = r_out;
    return done(kda::residual_norm(a, args->dtype == KDA_DTYPE_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_residual_norm_backward_workspace_size(int64_t rows, int32_t D) {
    if (rows < 0 || D < 8 || D % 8 || D > KDA_MAX_NORM_CHANNELS) return 0;
    return kda::residual_norm_backward_workspace(rows, D);
}

kda_status kda_residual_norm_backward(const kda_residual_norm_args *args, const void *dx, const float *dr_out, float *dy,
                                      float *dr, float *dgate, float *dw_post, float *dscale, float *dw_pre,
                                      void *workspace, size_t workspace_bytes, kda_stream_t stream) {
    if (kda_status rc = check_norm(args); rc != KDA_OK) return rc;
    if (args->rows > 0 && (!dy || (dx != nullptr) != (args->w_pre != nullptr) ||
                           (dgate != nullptr) != (args->gate != nullptr)))
        return KDA_ERR_INVALID_ARG;
    if ((dw_post && !args->w_post) || (dscale && !args->scale) || (dw_pre && !args->w_pre)) return KDA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < kda::residual_norm_backward_workspace(args->rows, args->D)) return KDA_ERR_WORKSPACE;
    if (!aligned16(dx, dr_out, dy, dr, dgate, dw_post, dscale, dw_pre, workspace)) return KDA_ERR_MISALIGNED;
    kda::NormBackwardArgs p{};
    p.f = norm_args(args);
    p.dx = dx; p.dr_out = dr_out;
    p.dy = dy; p.dr = dr; p.dgate = dgate; p.dw_post = dw_post; p.dscale = dscale; p.dw_pre = dw_pre;
    p.ws = workspace;
    return done(kda::residual_norm_backward(p, args->dtype == KDA_DTYPE_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
