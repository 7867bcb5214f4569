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

// Four consecutive channels likewise.
template <typename T> struct Pack4;
template <> struct Pack4<__nv_bfloat16> {
    uint2 u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void zero() { u = make_uint2(0, 0); }
    __device__ __forceinline__ void get(float (&x)[4]) const {
        x[0] = __uint_as_float(u.x << 16), x[1] = __uint_as_float(u.x & 0xFFFF0000u);
        x[2] = __uint_as_float(u.y << 16), x[3] = __uint_as_float(u.y & 0xFFFF0000u);
    }
    __device__ __forceinline__ void set(const float (&x)[4]) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
        u = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint2 *>(p) = u; }
    __device__ __forceinline__ void store_stream(__nv_bfloat16 *p) const { __stcs(reinterpret_cast<uint2 *>(p), u); }
};
template <> struct Pack4<float> {
    float4 a;
    __device__ __forceinline__ void load(const float *p) { a = *reinterpret_cast<const float4 *>(p); }
    __device__ __forceinline__ void zero() { a = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&x)[4]) const { x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w; }
    __device__ __forceinline__ void set(const float (&x)[4]) { a = make_float4(x[0], x[1], x[2], x[3]); }
    __device__ __forceinline__ void store(float *p) const { *reinterpret_cast<float4 *>(p) = a; }
    __device__ __forceinline__ void store_stream(float *p) const { __stcs(reinterpret_cast<float4 *>(p), a); }
};
template <typename T, int V> struct PackOf;
template <typename T> struct PackOf<T, 8> { using type = Pack8<T>; };
template <typename T> struct PackOf<T, 4> { using type = Pack4<T>; };
template <typename T, int V> using Pack = typename PackOf<T, V>::type;  // V channels

// Copies 16 bytes to shared memory in the background (zeros where `on` is false).
__device__ __forceinline__ void copy16(void *to, const void *from, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from),
                 "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_end_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() {  // until at most the N last groups are in flight
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Four channels likewise (`to`: a place that only this thread reads).
template <typename P, typename T> __device__ __forceinline__ void copy_pack(P *to, const T *from) {
    static_assert(sizeof(P) == 8 || sizeof(P) == 16, "bytes");
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
    if constexpr (sizeof(P) == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(at), "l"(from) : "memory");
    else asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
}
// Eight channels by copy16, to a place that only this thread reads.
template <typename T> __device__ __forceinline__ void copy8(Pack8<T> *to, const T *from, bool on) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(Pack8<T>) / 16; ++i)
        copy16(reinterpret_cast<char *>(to) + 16 * i, reinterpret_cast<const char *>(from) + (on ? 16 * i : 0), on);
}

__device__ __forceinline__ float exp2_approx(float x) {  // relative error about 2^-22
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float kLog2e = 1.4426950408889634f;

// e^v as 2^(v log2 e): relative error about 2^-22 + |v| 2^-24.
__device__ __forceinline__ float exp_f(float v) { return exp2_approx(v * kLog2e); }
__device__ __forceinline__ float rcp_approx(float x) {  // relative error about 2^-23; 0 for an infinite x
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / (1 + e^-v): for very negative v, e^-v = inf and the quotient is 0.
__device__ __forceinline__ float sigmoid_f(float v) { return rcp_approx(1.f + exp_f(-v)); }
__device__ __forceinline__ float silu_f(float v) { return v * sigmoid_f(v); }

// log(1 + e^v) = max(v, 0) + log1p(e^-|v|), with log1p(u) = 2 atanh(s), s = u / (2 + u) <= 1/3: small
// results keep their relative accuracy, which a logarithm of 1 + u would lose (a step delta of 0.001 is
// log(1.001)). atanh(s) / s is taken as the polynomial of degree 4 in s^2 that interpolates it at the
// five Chebyshev points of [0, 1/9] (error below 2e-8).
__device__ __forceinline__ float softplus_f(float v) {
    const float u = exp_f(-fabsf(v));
    const float s = u * rcp_approx(2.f + u), w = s * s;
    float p = fmaf(w, 0.1407888979f, 0.1398257911f);
    p = fmaf(w, p, 0.2001229823f);
    p = fmaf(w, p, 0.3333316147f);
    p = fmaf(w, p, 1.f);
    return fmaf(2.f * s, p, fmaxf(v, 0.f));
}

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
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}


__device__ __forceinline__ F2 exp2_pair(F2 x) {
    float a, b;
    unpack(x, a, b);
    return f2(exp2_approx(a), exp2_approx(b));
}

// ------------------------------------------------------------- selective scan ----

constexpr int kSsmTile = 128;  // tokens of a tile (KDA_SSM_TILE)

// First tile of sequence s, which starts at token b: its ceil(length / kSsmTile) tiles fit before the next
// sequence's, and total / kSsmTile + N hold them all.
__host__ __device__ __forceinline__ int64_t ssm_tile0(int64_t b, int s) { return b / kSsmTile + s; }

// B and C of a token in shared memory, by pairs of states: (B, C) of bf16 as they came, two pairs to 16
// bytes, or (B, B, C, C) of fp32. Lane q of a channel owns the pairs q NP .. q NP + NP - 1.
template <typename T, int NP, int LPC> struct SsmWeights;
template <int NP, int LPC> struct SsmWeights<__nv_bfloat16, NP, LPC> {
    static constexpr int kWords = 2 * NP * LPC;  // of a token
    static __device__ __forceinline__ F2 wide(uint32_t w) { return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
    // the states 8 j .. 8 j + 7
    static __device__ __forceinline__ void put(float *row, int j, const Pack8<__nv_bfloat16> &b, const Pack8<__nv_bfloat16> &c) {
        uint4 *to = reinterpret_cast<uint4 *>(row);
        auto at = [](int pair) { return NP == 1 ? pair / 2 : pair % NP / 2 * LPC + pair / NP; };
        to[at(4 * j)] = make_uint4(b.u.x, c.u.x, b.u.y, c.u.y);
        to[at(4 * j + 2)] = make_uint4(b.u.z, c.u.z, b.u.w, c.u.w);
    }
    static __device__ __forceinline__ void get(const float *row, int q, F2 (&b)[NP], F2 (&c)[NP]) {
        if constexpr (NP == 1) {
            const uint2 w = reinterpret_cast<const uint2 *>(row)[q];
            b[0] = wide(w.x), c[0] = wide(w.y);
        } else {
#pragma unroll
            for (int v = 0; v < NP / 2; ++v) {
                const uint4 w = reinterpret_cast<const uint4 *>(row)[v * LPC + q];
                b[2 * v] = wide(w.x), c[2 * v] = wide(w.y);
                b[2 * v + 1] = wide(w.z), c[2 * v + 1] = wide(w.w);
            }
        }
    }
};
template <int NP, int LPC> struct SsmWeights<float, NP, LPC> {
    static constexpr int kWords = 4 * NP * LPC;
    static __device__ __forceinline__ void put(float *row, int j, const Pack8<float> &b, const Pack8<float> &c) {
        float v[8], w[8];
        b.get(v);
        c.get(w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int pair = 4 * j + i;
            reinterpret_cast<float4 *>(row)[pair % NP * LPC + pair / NP] = make_float4(v[2 * i], v[2 * i + 1], w[2 * i], w[2 * i + 1]);
        }
    }
    static __device__ __forceinline__ void get(const float *row, int q, F2 (&b)[NP], F2 (&c)[NP]) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const float4 g = reinterpret_cast<const float4 *>(row)[p * LPC + q];
            b[p] = f2(g.x, g.y), c[p] = f2(g.z, g.w);
        }
    }
};

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
    float *tiles;  // [total / kSsmTile + N][channels][states]: states before each tile (ssm_tile0), or nullptr
};
size_t ssm_prefill_workspace(int64_t total, int N, int channels, int states, int groups);
int ssm_prefill_launches(int64_t total, int N, int channels, int states, int groups);
cudaError_t ssm_prefill(const SsmArgs &a, void *ws, bool bf16, cudaStream_t st);
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
