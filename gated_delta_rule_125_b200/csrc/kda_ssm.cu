// kda_ssm.cu -- the selective state space scan: packed prompts (ssm_prefill_kernel) and one
// token of each sequence (ssm_step_kernel).
//
//     delta = softplus(dt + dt_bias),  a_t = e^(delta_t A),  h_t = a_t h_(t-1) + delta_t x_t B_t,
//     y_t = (sum_n C_t h_t + D x_t) silu(z_t)                per channel d and state n.
//
// Prompts. The recurrence is diagonal: per (token, channel, state) one exponential, three
// multiply-adds and two multiplies, nothing a matrix instruction could take (the decay differs
// per channel AND state). With 16 states the exponentials bound it: 16 per clock and SM.
//
// A CTA owns CB channels and walks the tokens of its sequences in tiles of 128, TL lanes of K
// consecutive tokens per channel (K TL = 128). Per state n a thread forms its K decays and inputs
// once, in registers; folds them from a zero state; the TL lanes of a channel combine their
// (decay product, end state) pairs by a shuffle scan; and each thread replays its tokens from the
// state before them. So the time axis is parallel inside a tile and every exponential is taken
// once: a split of the time axis into independent pieces would take each twice. The decay product
// of a lane is one exponential of the sum of its steps, not a product of K roundings.
//
// Memory: x, dt, z and y move once, as 16-byte vectors of 8 channels; delta and delta x go through
// shared memory as fp32 [channel][token] (four tokens per load; a pad of 4 words per lane keeps the
// lanes on different banks). B and C of a tile are transposed into shared memory as fp32
// [state][token], 16 states at a time. The next tile's rows are loaded before the current tile is
// worked on.
//
// Sequence edges inside a tile: the first token of a sequence has its decay replaced by 0 after
// its own initial state went through it, so a tile may hold the end of one sequence, some short
// ones and the start of another. Only tiles that hold an edge run that variant of the loop.
#include "kda_layer.cuh"

namespace kda {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kNB = 16;  // states of B and C held in shared memory at a time

template <int K, int TL> struct Lay {
    static constexpr int kPad = K + 4;          // words per lane segment: 16-byte loads of all lanes hit different banks
    static constexpr int kRow = TL * kPad;      // words per row of 128 tokens
    static __device__ __forceinline__ int at(int t) { return t + (t / K) * 4; }
};

size_t prefill_smem(int CB, int row, int states) {
    return ((size_t)2 * CB * row + 16 + 2 * kNB * row + (size_t)2 * CB * states + 2 * kSsmTile) * 4;
}

template <typename T, int CB, int K, int TL>
__global__ void __launch_bounds__(CB *TL)
ssm_prefill_kernel(const SsmArgs a, const int bpg, const int R) {
    using L = Lay<K, TL>;
    constexpr int kRow = L::kRow;
    constexpr int NT = CB * TL;
    constexpr int U = kSsmTile * (CB / 8) / NT;   // (token, 8 channels) pieces per thread
    constexpr int UB = kSsmTile * (kNB / 8) / NT; // (token, 8 states) pieces per thread
    static_assert(K * TL == kSsmTile && U * NT == kSsmTile * (CB / 8) && UB * NT == kSsmTile * (kNB / 8), "shape");
    extern __shared__ float4 smem4[];
    float *sDt = reinterpret_cast<float *>(smem4);   // [CB][kRow] (8 channels, then 16 words, so that two pieces
    float *sDx = sDt + CB * kRow + 8;                //  of a row do not meet on a bank)
    float *sB = sDx + CB * kRow + 8;                 // [kNB][kRow]
    float *sC = sB + kNB * kRow;
    const int n = a.states;
    float *sA = sC + kNB * kRow;                     // [CB][n], times log2 e
    float *sH = sA + CB * n;                         // [CB][n], states before the tile
    int *sFirst = reinterpret_cast<int *>(sH + CB * n);  // [128] sequence whose first token this is, or -1
    int *sLast = sFirst + kSsmTile;
    __shared__ int sNext;

    const int tid = threadIdx.x, j = tid % TL, c = tid / TL;
    const int cpg = a.channels / a.groups;
    const int grp = blockIdx.x / bpg, cb = (blockIdx.x % bpg) * CB;  // channel block inside the group
    const int d0 = grp * cpg + cb;
    const int nc = min(CB, cpg - cb);  // channels of this block (a multiple of 8)
    const T *x = static_cast<const T *>(a.x) + d0, *dt = static_cast<const T *>(a.dt) + d0;
    const T *z = a.z ? static_cast<const T *>(a.z) + d0 : nullptr;
    T *y = static_cast<T *>(a.y) + d0;
    const size_t ldx = a.channels, ldb = (size_t)a.groups * n;
    const T *Bp = static_cast<const T *>(a.B) + (size_t)grp * n, *Cp = static_cast<const T *>(a.C) + (size_t)grp * n;

    const SsmRange rg = ssm_range(a.cu, a.N, a.total, blockIdx.y, R);
    const size_t nstate = (size_t)a.channels * n;
    // sequences without tokens keep their initial state
    if (a.S_T) {
        for (int s = rg.s0; s < rg.s1; ++s) {
            if ((a.cu ? (int64_t)a.cu[s + 1] - a.cu[s] : a.total) > 0) continue;
            for (int i = tid; i < nc * n; i += NT) {
                const size_t at = s * nstate + (size_t)d0 * n + i;
                a.S_T[at] = a.S0 ? a.S0[at] : 0.f;
            }
        }
    }
    if (rg.t1 <= rg.t0) return;
    for (int i = tid; i < CB * n; i += NT) {
        sA[i] = i < nc * n ? a.A[(size_t)d0 * n + i] * kLog2e : 0.f;
        sH[i] = 0.f;
    }
    for (int i = tid; i < 2 * kSsmTile; i += NT) sFirst[i] = -1;
    if (tid == 0) sNext = rg.s0;

    Pack8<T> rx[U], rd[U], rb[UB], rc[UB];
    auto load_rows = [&](int64_t t0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = tid + u * NT, c8 = (p / kSsmTile) * 8;
            const int64_t t = t0 + p % kSsmTile;
            if (t >= rg.t0 && t < rg.t1 && c8 < nc) {
                rx[u].load(x + t * ldx + c8);
                rd[u].load(dt + t * ldx + c8);
            } else {
                rx[u].zero();
                rd[u].zero();
            }
        }
    };
    auto load_bc = [&](int64_t t0, int nb) {
#pragma unroll
        for (int u = 0; u < UB; ++u) {
            const int p = tid + u * NT, n8 = nb + (p / kSsmTile) * 8;
            const int64_t t = t0 + p % kSsmTile;
            if (t >= rg.t0 && t < rg.t1 && n8 < n) {
                rb[u].load(Bp + t * ldb + n8);
                rc[u].load(Cp + t * ldb + n8);
            } else {
                rb[u].zero();
                rc[u].zero();
            }
        }
    };
    auto store_bc = [&]() {
#pragma unroll
        for (int u = 0; u < UB; ++u) {
            const int p = tid + u * NT, n8 = (p / kSsmTile) * 8, at = L::at(p % kSsmTile);
            float v[8];
            rb[u].get(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sB[(n8 + i) * kRow + at] = v[i];
            rc[u].get(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sC[(n8 + i) * kRow + at] = v[i];
        }
    };
    auto row = [&](int ch) { return ch * kRow + (ch / 8) * 8; };

    const int64_t tile0 = rg.t0 / kSsmTile, tile1 = (rg.t1 + kSsmTile - 1) / kSsmTile;
    load_rows(tile0 * kSsmTile);
    load_bc(tile0 * kSsmTile, 0);
    for (int64_t tile = tile0; tile < tile1; ++tile) {
        const int64_t t0 = tile * kSsmTile;
        const int64_t tb = max(t0, rg.t0), te = min(t0 + kSsmTile, rg.t1);
        __syncthreads();  // the previous tile's y and marks have been read
        const int s_from = sNext;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = tid + u * NT, c8 = (p / kSsmTile) * 8, at = L::at(p % kSsmTile);
            const int64_t t = t0 + p % kSsmTile;
            const bool in = t >= tb && t < te && c8 < nc;
            float v[8], w[8];
            rd[u].get(v);
            rx[u].get(w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float dl = 0.f;
                if (in) {
                    dl = v[i] + (a.dt_bias ? a.dt_bias[d0 + c8 + i] : 0.f);
                    if (a.softplus) dl = softplus_f(dl);
                }
                sDt[row(c8 + i) + at] = dl;
                sDx[row(c8 + i) + at] = dl * w[i];
            }
        }
        store_bc();
        if (a.tiles && t0 >= rg.t0)
            for (int i = tid; i < nc * n; i += NT) a.tiles[(size_t)tile * nstate + (size_t)d0 * n + i] = sH[i];
        bool edge = false;
        int next = s_from;
        if (a.cu) {
            for (int s = s_from + tid; s < rg.s1; s += NT) {
                const int64_t b = a.cu[s], e = a.cu[s + 1];
                if (b >= te) break;
                if (e <= te) next = s + 1;
                if (e <= b) continue;
                if (b >= tb) sFirst[b - t0] = s, edge = true;
                if (e <= te) sLast[e - 1 - t0] = s, edge = true;
            }
        } else if (tid == 0) {
            if (tb == 0) sFirst[0] = 0, edge = true;
            if (te == a.total) sLast[te - 1 - t0] = 0, edge = true;
        }
        edge = __syncthreads_or(edge);
        if (next > s_from) atomicMax(&sNext, next);
        if (tile + 1 < tile1) load_rows(t0 + kSsmTile);
        if (n > kNB) load_bc(t0, kNB);
        else if (tile + 1 < tile1) load_bc(t0 + kSsmTile, 0);

        F2 dl[K / 2], dx[K / 2], yv[K / 2];
        float sum = 0.f;
        {
            const float *pd = sDt + row(c) + j * L::kPad, *px = sDx + row(c) + j * L::kPad;
#pragma unroll
            for (int k = 0; k < K; k += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(pd + k);
                const float4 w = *reinterpret_cast<const float4 *>(px + k);
                dl[k / 2] = f2(v.x, v.y);
                dl[k / 2 + 1] = f2(v.z, v.w);
                dx[k / 2] = f2(w.x, w.y);
                dx[k / 2 + 1] = f2(w.z, w.w);
                sum += (v.x + v.y) + (v.z + v.w);
                yv[k / 2] = yv[k / 2 + 1] = f2(0.f, 0.f);
            }
        }
        uint32_t first = 0, last = 0;
        if (edge) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                first |= (sFirst[j * K + k] >= 0 ? 1u : 0u) << k;
                last |= (sLast[j * K + k] >= 0 ? 1u : 0u) << k;
            }
        }

        auto states = [&](auto marked, int nb, int cnt) {
            constexpr bool kMarked = decltype(marked)::value;
            for (int i = 0; i < cnt; ++i) {
                const float A2 = sA[c * n + nb + i], carry = sH[c * n + nb + i];
                const float *pb = sB + i * kRow + j * L::kPad, *pc = sC + i * kRow + j * L::kPad;
                float av[K], bv[K];
                const F2 A22 = f2(A2, A2);
#pragma unroll
                for (int k = 0; k < K; k += 4) {
                    const float4 b = *reinterpret_cast<const float4 *>(pb + k);
                    float u0, u1;
                    unpack(mul2(dl[k / 2], A22), u0, u1);
                    av[k] = exp2_approx(u0);
                    av[k + 1] = exp2_approx(u1);
                    unpack(mul2(dl[k / 2 + 1], A22), u0, u1);
                    av[k + 2] = exp2_approx(u0);
                    av[k + 3] = exp2_approx(u1);
                    unpack(mul2(dx[k / 2], f2(b.x, b.y)), bv[k], bv[k + 1]);
                    unpack(mul2(dx[k / 2 + 1], f2(b.z, b.w)), bv[k + 2], bv[k + 3]);
                }
                float ap = exp2_approx(sum * A2);
                if constexpr (kMarked) {
                    if (first) {
                        ap = 0.f;
#pragma unroll
                        for (int k = 0; k < K; ++k)
                            if (first >> k & 1) {
                                if (a.S0 && c < nc)
                                    bv[k] = fmaf(av[k], a.S0[sFirst[j * K + k] * nstate + (size_t)(d0 + c) * n + nb + i], bv[k]);
                                av[k] = 0.f;
                            }
                    }
                }
                float e = bv[0];
#pragma unroll
                for (int k = 1; k < K; ++k) e = fmaf(av[k], e, bv[k]);
                if (j == 0) e = fmaf(ap, carry, e);
#pragma unroll
                for (int s = 1; s < TL; s <<= 1) {
                    const float eo = __shfl_up_sync(0xffffffffu, e, s, TL), ao = __shfl_up_sync(0xffffffffu, ap, s, TL);
                    if (j >= s) {
                        e = fmaf(ap, eo, e);
                        ap *= ao;
                    }
                }
                float h = __shfl_up_sync(0xffffffffu, e, 1, TL);
                if (j == 0) h = carry;
                if (j == TL - 1) sH[c * n + nb + i] = e;
#pragma unroll
                for (int k = 0; k < K; k += 4) {
                    const float4 cc = *reinterpret_cast<const float4 *>(pc + k);
#pragma unroll
                    for (int m = 0; m < 4; ++m) bv[k + m] = h = fmaf(av[k + m], h, bv[k + m]);
                    yv[k / 2] = fma2(f2(cc.x, cc.y), f2(bv[k], bv[k + 1]), yv[k / 2]);
                    yv[k / 2 + 1] = fma2(f2(cc.z, cc.w), f2(bv[k + 2], bv[k + 3]), yv[k / 2 + 1]);
                }
                if constexpr (kMarked) {
                    if (last && a.S_T && c < nc) {
#pragma unroll
                        for (int k = 0; k < K; ++k)
                            if (last >> k & 1) a.S_T[sLast[j * K + k] * nstate + (size_t)(d0 + c) * n + nb + i] = bv[k];
                    }
                }
            }
        };
        for (int nb = 0; nb < n; nb += kNB) {
            if (nb) {
                __syncthreads();
                store_bc();
                __syncthreads();
                if (nb + kNB < n) load_bc(t0, nb + kNB);
                else if (tile + 1 < tile1) load_bc(t0 + kSsmTile, 0);
            }
            const int cnt = min(kNB, n - nb);
            if (edge) states(Bool<true>{}, nb, cnt);
            else states(Bool<false>{}, nb, cnt);
        }
        {  // y over this thread's own delta segment
            float *py = sDt + row(c) + j * L::kPad;
#pragma unroll
            for (int k = 0; k < K; k += 4) {
                float4 v;
                unpack(yv[k / 2], v.x, v.y);
                unpack(yv[k / 2 + 1], v.z, v.w);
                *reinterpret_cast<float4 *>(py + k) = v;
            }
        }
        __syncthreads();
        if (edge)
            for (int i = tid; i < 2 * kSsmTile; i += NT) sFirst[i] = -1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = tid + u * NT, c8 = (p / kSsmTile) * 8, at = L::at(p % kSsmTile);
            const int64_t t = t0 + p % kSsmTile;
            if (t < tb || t >= te || c8 >= nc) continue;
            Pack8<T> q;
            float xv[8], v[8];
            q.load(x + t * ldx + c8);
            q.get(xv);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fmaf(a.D ? a.D[d0 + c8 + i] : 0.f, xv[i], sDt[row(c8 + i) + at]);
            if (z) {
                q.load_stream(z + t * ldx + c8);
                q.get(xv);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= silu_f(xv[i]);
            }
            q.set(v);
            q.store_stream(y + t * ldx + c8);
        }
    }
}

template <typename T, int CB, int K, int TL>
cudaError_t launch_prefill(const SsmArgs &a, int R, cudaStream_t st) {
    const int cpg = a.channels / a.groups, bpg = (cpg + CB - 1) / CB;
    const size_t smem = prefill_smem(CB, Lay<K, TL>::kRow, a.states);
    auto kern = ssm_prefill_kernel<T, CB, K, TL>;
    if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem); e != cudaSuccess)
        return e;
    kern<<<dim3(bpg * a.groups, R), CB * TL, smem, st>>>(a, bpg, R);
    return cudaGetLastError();
}

template <typename T>
cudaError_t prefill_t(const SsmArgs &a, cudaStream_t st) {
    const int cpg = a.channels / a.groups;
    const int64_t wide = (int64_t)a.groups * ((cpg + 15) / 16);
    const int64_t most = (a.total + kSsmTile - 1) / kSsmTile;
    const int R = (int)max((int64_t)1, min((int64_t)a.N, min(most, (148 * 8 + wide - 1) / wide)));
    if (wide * R >= 148) return launch_prefill<T, 16, 8, 16>(a, R, st);
    return launch_prefill<T, 8, 8, 16>(a, R, st);
}

}  // namespace

cudaError_t ssm_prefill(const SsmArgs &a, bool bf16, cudaStream_t st) {
    return bf16 ? prefill_t<__nv_bfloat16>(a, st) : prefill_t<float>(a, st);
}

// ------------------------------------------------------------------- one token ----
//
// Bound by the fp32 state, read and written once (8 bytes per channel and state against 2 of
// arithmetic). A warp owns CPW consecutive channels (their A stays in registers) and walks the
// sequences; a lane holds U 4-state vectors of them, n / 4 lanes to a channel, so every access is
// a run of 16-byte vectors. The per-channel work (softplus, gate) is done by one lane per channel
// and handed over by shuffles; C h is summed over a channel's lanes by shuffles.
namespace {

constexpr int kStepThreads = 128;

template <typename T, int NS>
__global__ void __launch_bounds__(kStepThreads)
ssm_step_kernel(const SsmArgs a) {
    constexpr int LPC = NS / 4;                 // lanes of a channel
    constexpr int G = 32 / LPC;                 // channels of one pass over the lanes
    constexpr int U = LPC == 2 ? 2 : 4;         // passes
    constexpr int CPW = U * G;                  // channels of a warp (at most 32)
    const int lane = threadIdx.x & 31, warp = (blockIdx.x * kStepThreads + threadIdx.x) >> 5;
    const int D = a.channels, base = warp * CPW;
    if (base >= D) return;
    const int cpg = D / a.groups, q = lane % LPC;
    const T *x = static_cast<const T *>(a.x), *dt = static_cast<const T *>(a.dt), *z = static_cast<const T *>(a.z);
    const T *B = static_cast<const T *>(a.B), *C = static_cast<const T *>(a.C);
    T *y = static_cast<T *>(a.y);
    float4 A[U];
    int bc[U];  // offset of this lane's states in a row of B and C
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int d = base + u * G + lane / LPC;
        on[u] = d < D;
        A[u] = on[u] ? *reinterpret_cast<const float4 *>(a.A + (size_t)d * NS + 4 * q) : make_float4(0.f, 0.f, 0.f, 0.f);
        A[u].x *= kLog2e; A[u].y *= kLog2e; A[u].z *= kLog2e; A[u].w *= kLog2e;
        bc[u] = on[u] ? (d / cpg) * NS + 4 * q : 0;
    }
    const int dl_ch = base + lane;  // the channel of this lane's scalar work
    const bool mine = lane < CPW && dl_ch < D;
    const float bias = mine && a.dt_bias ? a.dt_bias[dl_ch] : 0.f, skip = mine && a.D ? a.D[dl_ch] : 0.f;

    auto load4 = [](const T *p) {
        if constexpr (sizeof(T) == 2) {
            const uint2 w = *reinterpret_cast<const uint2 *>(p);
            return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                               __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
        } else {
            return *reinterpret_cast<const float4 *>(p);
        }
    };
    for (int s = blockIdx.y; s < a.N; s += gridDim.y) {
        float4 h[U];
        float *S = a.S_T + ((size_t)s * D + base) * NS;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (on[u]) h[u] = __ldcs(reinterpret_cast<const float4 *>(S) + u * 32 + lane);
        const size_t row = (size_t)s * D;
        float xv = 0.f, dv = 0.f, zv = 0.f;
        if (mine) {
            xv = static_cast<float>(x[row + dl_ch]);
            dv = static_cast<float>(dt[row + dl_ch]) + bias;
            if (z) zv = static_cast<float>(z[row + dl_ch]);
            if (a.softplus) dv = softplus_f(dv);
        }
        const float dxv = dv * xv;
        float out = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float4 b = load4(B + (size_t)s * a.groups * NS + bc[u]), c = load4(C + (size_t)s * a.groups * NS + bc[u]);
            const float dl = __shfl_sync(0xffffffffu, dv, u * G + lane / LPC);
            const float dx = __shfl_sync(0xffffffffu, dxv, u * G + lane / LPC);
            float sum = 0.f;
            if (on[u]) {
                h[u].x = fmaf(exp2_approx(dl * A[u].x), h[u].x, dx * b.x);
                h[u].y = fmaf(exp2_approx(dl * A[u].y), h[u].y, dx * b.y);
                h[u].z = fmaf(exp2_approx(dl * A[u].z), h[u].z, dx * b.z);
                h[u].w = fmaf(exp2_approx(dl * A[u].w), h[u].w, dx * b.w);
                __stcs(reinterpret_cast<float4 *>(S) + u * 32 + lane, h[u]);
                sum = fmaf(c.x, h[u].x, c.y * h[u].y) + fmaf(c.z, h[u].z, c.w * h[u].w);
            }
#pragma unroll
            for (int m = 1; m < LPC; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
            const float got = __shfl_sync(0xffffffffu, sum, (lane % G) * LPC);
            if (lane / G == u) out = got;
        }
        if (mine) {
            out = fmaf(skip, xv, out);
            if (z) out *= silu_f(zv);
            y[row + dl_ch] = static_cast<T>(out);
        }
    }
}

template <typename T, int NS>
cudaError_t launch_step(const SsmArgs &a, cudaStream_t st) {
    constexpr int U = NS == 8 ? 2 : 4, CPW = U * 32 / (NS / 4);
    const int64_t warps = (a.channels + CPW - 1) / CPW;
    const unsigned gx = (unsigned)((warps * 32 + kStepThreads - 1) / kStepThreads);
    // about eight warps in flight per SM quarter; a warp then walks the rest of the sequences
    const unsigned gy = (unsigned)max((int64_t)1, min((int64_t)a.N, (int64_t)(148 * 8 + gx - 1) / gx));
    ssm_step_kernel<T, NS><<<dim3(gx, gy), kStepThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t step_t(const SsmArgs &a, cudaStream_t st) {
    switch (a.states) {
    case 8: return launch_step<T, 8>(a, st);
    case 16: return launch_step<T, 16>(a, st);
    case 32: return launch_step<T, 32>(a, st);
    case 64: return launch_step<T, 64>(a, st);
    case 128: return launch_step<T, 128>(a, st);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t ssm_step(const SsmArgs &a, bool bf16, cudaStream_t st) {
    return bf16 ? step_t<__nv_bfloat16>(a, st) : step_t<float>(a, st);
}

}  // namespace kda
