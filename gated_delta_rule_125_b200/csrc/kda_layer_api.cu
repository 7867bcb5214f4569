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
    if (rows > 0 && !p->A) return KDA_ERR_INVALID_ARG;
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

kda_status done(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

}  // namespace

extern "C" {

size_t kda_ssm_tile_states_size(int64_t total_tokens, int32_t channels, int32_t states) {
    if (total_tokens < 0 || channels < 1 || states < 1) return 0;
    return (size_t)((total_tokens + kda::kSsmTile - 1) / kda::kSsmTile) * channels * states * sizeof(float);
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
    if (!grads || !ssm->A || !grads->dA || (!cu_seqlens && num_seqs != 1)) return KDA_ERR_INVALID_ARG;
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

}  // extern "C"
