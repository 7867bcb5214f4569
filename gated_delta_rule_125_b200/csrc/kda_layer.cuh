// kda_layer.cuh -- declarations and element helpers shared by the kernels of the layer
// around the recurrences: the selective scan, the short convolution with a bias and its
// backward, the residual norms.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda.h"

namespace kda {

// ------------------------------------------------------------ element helpers ----

// Eight consecutive channels as they lie in memory (one 16-byte vector of bf16, two of fp32).
template <typename T> struct Pack8;
template <> struct Pack8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void load_stream(const __nv_bfloat16 *p) { u = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        u = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint4 *>(p) = u; }
    __device__ __forceinline__ void store_stream(__nv_bfloat16 *p) const { __stcs(reinterpret_cast<uint4 *>(p), u); }
};
template <> struct Pack8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void load_stream(const float *p) {
        a = __ldcs(reinterpret_cast<const float4 *>(p));
        b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    __device__ __forceinline__ void set(const float (&x)[8]) {
        a = make_float4(x[0], x[1], x[2], x[3]);
        b = make_float4(x[4], x[5], x[6], x[7]);
    }
    __device__ __forceinline__ void store(float *p) const {
        reinterpret_cast<float4 *>(p)[0] = a;
        reinterpret_cast<float4 *>(p)[1] = b;
    }
    __device__ __forceinline__ void store_stream(float *p) const {
        __stcs(reinterpret_cast<float4 *>(p), a);
        __stcs(reinterpret_cast<float4 *>(p) + 1, b);
    }
};

__device__ __forceinline__ float exp2_approx(float x) {  // relative error about 2^-22
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / (1 + e^-v): for very negative v, e^-v = inf and the quotient is 0.
__device__ __forceinline__ float sigmoid_f(float v) { return __fdividef(1.f, 1.f + expf(-v)); }
__device__ __forceinline__ float silu_f(float v) { return v * sigmoid_f(v); }

// log(1 + e^v) = max(v, 0) + log1p(e^-|v|), with log1p(u) = 2 atanh(s), s = u / (2 + u) <= 1/3, by the
// series of atanh (the first term left out is s^17 / 17 < 5e-10 of s): small results keep their
// relative accuracy, which a logarithm of 1 + u would lose (a step delta of 0.001 is log(1.001)).
__device__ __forceinline__ float softplus_f(float v) {
    const float u = expf(-fabsf(v));
    const float s = __fdividef(u, 2.f + u), w = s * s;
    float p = fmaf(w, 1.f / 15.f, 1.f / 13.f);
    p = fmaf(w, p, 1.f / 11.f);
    p = fmaf(w, p, 1.f / 9.f);
    p = fmaf(w, p, 1.f / 7.f);
    p = fmaf(w, p, 1.f / 5.f);
    p = fmaf(w, p, 1.f / 3.f);
    p = fmaf(w, p, 1.f);
    return fmaf(2.f * s, p, fmaxf(v, 0.f));
}

template <bool V> struct Bool {
    static constexpr bool value = V;
};

// Two fp32 lanes in one instruction (fma.rn.f32x2 and friends of sm_100): half the issue slots.
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack(F2 p, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v));
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// ------------------------------------------------------------- selective scan ----

constexpr int kSsmTile = 128;  // tokens of a tile (KDA_SSM_TILE)

struct SsmArgs {
    const void *x, *dt, *B, *C, *z;  // io dtype; z may be nullptr
    const float *A, *D, *dt_bias;    // [channels][states]; D, dt_bias [channels] or nullptr
    const float *S0;                 // [N][channels][states] or nullptr
    const int32_t *cu;               // [N + 1] or nullptr (one sequence)
    int N;
    int64_t total;
    int channels, states, groups;
    bool softplus;
    void *y;
    float *S_T;    // may be nullptr
    float *tiles;  // [ceil(total / kSsmTile)][channels][states]: states before each tile, or nullptr
};
cudaError_t ssm_prefill(const SsmArgs &a, bool bf16, cudaStream_t st);
// One token of each of N sequences: x, dt, z, y [N][channels], B, C [N][groups][states]; a.S_T in place.
cudaError_t ssm_step(const SsmArgs &a, bool bf16, cudaStream_t st);

struct SsmBackwardArgs {
    SsmArgs f;  // the forward's inputs; f.tiles as the forward wrote it; f.y, f.S_T unused
    const void *dy;     // [T][channels] io dtype
    const float *dS_T;  // [N][channels][states] or nullptr
    float *dx, *ddt, *dB, *dC, *dz;  // [T][..]; dz nullptr without z
    float *dA, *dD, *ddt_bias;       // dD, ddt_bias may be nullptr
    float *dS0;                      // may be nullptr
    void *ws;
};
size_t ssm_backward_workspace(int64_t total, int N, int channels, int states, int groups);
cudaError_t ssm_backward(const SsmBackwardArgs &b, bool bf16, cudaStream_t st);

// Sequences of the packed axis dealt to R ranges of whole sequences: range r holds those whose first
// token lies in [r T / R, (r + 1) T / R) (the last range also the empty ones behind the last token).
struct SsmRange {
    int s0, s1;      // sequences [s0, s1)
    int64_t t0, t1;  // their tokens
};
__device__ __forceinline__ int lower_bound_cu(const int32_t *cu, int N, int64_t t) {  // first s with cu[s] >= t
    int lo = 0, hi = N;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] >= t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}
__device__ __forceinline__ SsmRange ssm_range(const int32_t *cu, int N, int64_t total, int r, int R) {
    SsmRange g;
    if (!cu) return SsmRange{0, 1, 0, total};
    g.s0 = r == 0 ? 0 : lower_bound_cu(cu, N, total * r / R);
    g.s1 = r == R - 1 ? N : lower_bound_cu(cu, N, total * (r + 1) / R);
    g.t0 = cu[g.s0];
    g.t1 = cu[g.s1];
    return g;
}

// ---------------------------------------------------------- short convolution ----

struct ConvArgs {
    const void *x;        // [T][C]
    void *y;              // [T][C]
    const float *w;       // [C][W]
    const float *bias;    // [C] or nullptr
    const void *state_in; // [N][W-1][C] or nullptr
    void *state_out;      // [N][W-1][C] or nullptr
    const int32_t *cu;
    int N;
    int64_t total;
    int C, W;
};
cudaError_t conv_bias(const ConvArgs &a, bool bf16, cudaStream_t st);
cudaError_t conv_step(const ConvArgs &a, bool bf16, cudaStream_t st);  // total = N, state_out in place

struct ConvBackwardArgs {
    ConvArgs f;  // y, state_out unused
    const void *dy;
    bool dy_bf16;
    float *dx, *dw, *dbias, *dstate;  // dbias, dstate may be nullptr
    void *ws;
};
size_t conv_backward_workspace(int64_t total, int C, int W);
cudaError_t conv_backward(const ConvBackwardArgs &b, bool bf16, cudaStream_t st);

// ------------------------------------------------------------- residual norms ----

struct NormArgs {
    const void *y, *r, *gate;  // gate may be nullptr
    const float *w_post, *scale, *w_pre;  // w_post, scale may be nullptr
    float res_scale, eps;
    int64_t rows;
    int D;
    bool res_bf16;
    void *x, *r_out;
};
cudaError_t residual_norm(const NormArgs &a, bool bf16, cudaStream_t st);

struct NormBackwardArgs {
    NormArgs f;  // x, r_out unused
    const void *dx;
    const float *dr_out;  // may be nullptr
    float *dy, *dr, *dgate, *dw_post, *dscale, *dw_pre;
    void *ws;
};
size_t residual_norm_backward_workspace(int64_t rows, int D);
cudaError_t residual_norm_backward(const NormBackwardArgs &b, bool bf16, cudaStream_t st);

}  // namespace kda
