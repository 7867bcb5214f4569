// kda_ssm_backward.cu -- gradients of the selective state space scan.
//
// With e = dy silu(z) (dy without a gate), y' the output before the gate, and
// G_t = dL/dh_t = C_t e_t + a_(t+1) G_(t+1) (plus dS_T at a sequence's last token), p_t = G_t a_t h_(t-1):
//
//     dz = dy y' silu'(z)                     dD = sum_t e x
//     dC_t[n] = sum_d e h                     dB_t[n] = sum_d G delta x
//     dA = sum_t p delta                      dx = delta sum_n G B + D e
//     ddelta = sum_n A p + x sum_n G B        ddt = ddelta sigmoid(dt + dt_bias)
//     ddt_bias = sum_t ddt                    dS0 = a_0 G_0.
//
// A CTA owns CB channels of one sequence (LPC lanes per channel, NS states each, as the forward) and
// walks its tokens backwards in blocks of 128, from the state before each block that the forward
// saved. It first folds the block forwards, keeping the state before each group of UG tokens; then,
// group by group from the end, it forms the group's decays and states again in registers and runs the
// reverse recurrence over them. So each exponential is taken twice and no state goes to memory. A block's
// rows (x, dt, dy, z) are loaded together, the next block's on their way to the L2 cache meanwhile; B and C
// are loaded a stage of up to 32 tokens ahead.
// (h_t - delta x B in place of a h_(t-1) would save a product, and its relative accuracy.)
//
// Sums over the states (three per token and channel) are a reduce-scatter of shuffles over a
// channel's lanes. Sums over the channels (dB, dC) are one over the lanes of the same states, then the
// CTA's warps through shared memory, then its partial sums go to the workspace and ssm_sum_kernel adds
// them in a fixed order: no atomics, the same bits every time.
//
// Measured, 4096 tokens (the longest sequence 2853) x 4096 channels x 16 states, bf16 with a gate: 694 us
// with 24 more for the sums over the channels. Two warps per SM quarter (221 registers) issue in 52 % of the
// clocks; the shared memory's pipe is 56 % busy, half of that with shuffles. What it replaced: every load
// waited for where it is used 735 us, with B and C expanded to fp32 in shared memory; three CTAs to an SM
// (registers capped without spills) 790 us, as the longest sequence's chain then gets a third of an SM (8
// sequences of 512 tokens, which balance: 734 us with two CTAs, 703 us with three). At 32 and at 128 states the
// states before the groups take 64 and 80 KB of shared memory (127 to 131 KB in all), so that only one CTA fits an
// SM there; the sizes above were measured at 16 states.
#include "kda_layer.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;

// 2^x for two x, more exactly than the hardware's near x = 0: x = i + r, 2^r = 1 + r q(r) with q the
// polynomial of degree 4 that interpolates (2^r - 1) / r at the five Chebyshev points of [-1/2, 1/2]
// (error below 2.1e-7 of the result, and of x itself for small x: a slow decay keeps its rate over a
// long chain). Adding 1.5 2^23 rounds x to the integer i in the low bits. The gradients' own chain
// takes this one: with the hardware's exponential the gradient of S0 after 500 tokens was off by 1.0e-6
// of its norm, with this one by 4e-7, what rounding the chain leaves.
__device__ __forceinline__ F2 exp2_poly2(F2 x) {
    float a, b;
    unpack(x, a, b);
    x = f2(fminf(fmaxf(a, -126.f), 127.f), fminf(fmaxf(b, -126.f), 127.f));
    const F2 t = add2(x, f2(12582912.f, 12582912.f)), i = add2(t, f2(-12582912.f, -12582912.f));
    const F2 r = fma2(i, f2(-1.f, -1.f), x);
    F2 q = fma2(r, f2(0.00133813021f, 0.00133813021f), f2(0.00966636837f, 0.00966636837f));
    q = fma2(r, q, f2(0.0555038117f, 0.0555038117f));
    q = fma2(r, q, f2(0.240223497f, 0.240223497f));
    q = fma2(r, q, f2(0.693147182f, 0.693147182f));
    q = fma2(r, q, f2(1.f, 1.f));
    float t0, t1, q0, q1;
    unpack(t, t0, t1);
    unpack(q, q0, q1);
    return f2(__int_as_float(__float_as_int(q0) + (__float_as_int(t0) << 23)),
              __int_as_float(__float_as_int(q1) + (__float_as_int(t1) << 23)));
}

template <typename T, int NS, int LPC> struct BackMem {
    static constexpr int N_ = NS * LPC, CB = kThreads / LPC;
    static constexpr int UG = 16 / NS;                       // tokens of a group: 16 (token, state) values per lane
    static constexpr int BT = 512 / N_ > 32 ? 32 : 512 / N_; // tokens of B and C staged at a time
    static constexpr int EB = NS >= 8 ? 32 : kSsmTile;       // tokens whose groups' states fit shared memory
    static constexpr int kX = CB * 4 + 4;
    static_assert(EB % BT == 0 && BT % UG == 0 && kSsmTile % BT == 0, "groups");
    // Where token v of the staged ones has its sums: two warps' parts of 16 states in a row of banks belong to the tokens
    // v and v + 2 (written) or v and v + 1 (read).
    static __host__ __device__ constexpr int slot(int v) { return N_ == 16 ? v ^ (v >> 1 & 1) : v; }
    float sX[kSsmTile * kX];                         // (delta, delta x, e, -), then (sum A p, sum G B, sum C h, -)
    using W = SsmWeights<T, NS / 2, LPC>;
    float sBC[BT * W::kWords];                       // B and C
    float sPar[2][CB];                               // dt_bias, D
    float sAcc[2][kThreads][8];                      // dD, ddt_bias: a thread's sums over the tokens of its pieces
    float sRed[2][kWarps][BT * N_];                  // a warp's sums over its channels: dB, dC
    unsigned long long sEnt[EB / UG][NS / 2][kThreads];        // the state before each group
    unsigned long long sTop[EB < kSsmTile ? kSsmTile / EB : 1][NS / 2][kThreads];  // and before each EB tokens
};

template <typename T, int NS, int LPC>
__global__ void __launch_bounds__(kThreads, 2)
ssm_backward_kernel(const SsmBackwardArgs g, const int nblk, const int bpg, float *__restrict__ pB, float *__restrict__ pC,
                    float *__restrict__ pA, float *__restrict__ pD, float *__restrict__ pbias) {
    using M = BackMem<T, NS, LPC>;
    using W = typename M::W;
    constexpr int N_ = M::N_, NP = NS / 2, CB = M::CB, UG = M::UG, BT = M::BT, EB = M::EB, kX = M::kX, G_ = 32 / LPC;
    constexpr int PIECES = kSsmTile * CB / 8 / kThreads;    // (token, 8 channels) pieces per thread of a block
    extern __shared__ __align__(16) char smem_raw[];
    M &sm = *reinterpret_cast<M *>(smem_raw);
    const SsmArgs &a = g.f;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, q = tid % LPC, ch = tid / LPC;
    const int blk = blockIdx.x % nblk, s = blockIdx.x / nblk;
    const int64_t b = a.cu ? a.cu[s] : 0, e = a.cu ? a.cu[s + 1] : a.total;

    const int cpg = a.channels / a.groups, grp = blk / bpg, c0 = (blk % bpg) * CB;
    const int nc = min(CB, cpg - c0), d0 = grp * cpg + c0;
    const bool on = ch < nc;
    const size_t ldx = a.channels, nstate = (size_t)a.channels * N_, own = (size_t)(d0 + (on ? ch : 0)) * N_ + q * NS;
    int base = 0;  // the first of the 16 values whose sums over the warp's channels this lane ends up with
#pragma unroll
    for (int m = G_ / 2, n = 8; m > 0; m >>= 1, n >>= 1) base += lane / LPC & m ? n : 0;
    const int red0 = M::slot(base / NS) * N_ + q * NS + base % NS, red1 = M::slot(base / NS + 1) * N_ + q * NS + base % NS;
    F2 A2[NP], A1[NP], r[NP];  // A log2 e, A, the gradient a_(t+1) G_(t+1) that comes in
    F2 dA[NP], blockA[NP];     // dA of the blocks done, of this one (added group by group: short sums keep their bits)
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const float2 v = *reinterpret_cast<const float2 *>(a.A + own + 2 * p);
        A1[p] = f2(v.x, v.y);
        A2[p] = f2(v.x * kLog2e, v.y * kLog2e);
        r[p] = dA[p] = blockA[p] = f2(0.f, 0.f);
        if (g.dS_T && on) r[p].v = *reinterpret_cast<const unsigned long long *>(g.dS_T + s * nstate + own + 2 * p);
    }
    const T *x = static_cast<const T *>(a.x) + d0, *dt = static_cast<const T *>(a.dt) + d0;
    const T *z = a.z ? static_cast<const T *>(a.z) + d0 : nullptr, *dy = static_cast<const T *>(g.dy) + d0;
    const size_t ldb = (size_t)a.groups * N_;
    const T *Bp = static_cast<const T *>(a.B) + (size_t)grp * N_, *Cp = static_cast<const T *>(a.C) + (size_t)grp * N_;

    // this thread's pieces: channels pc .. pc + 7 of tokens pt, pt + kThreads * 8 / CB, ...
    constexpr int TS = kThreads * 8 / CB;
    const int pt = tid % TS, pc = tid / TS * 8;
    const bool pon = pc < nc;
    // dt_bias and D by channel, and each thread's sums for dD and ddt_bias, kept out of the registers that the chain needs
    if (tid < CB) {
        sm.sPar[0][tid] = tid < nc && a.dt_bias ? a.dt_bias[d0 + tid] : 0.f;
        sm.sPar[1][tid] = tid < nc && a.D ? a.D[d0 + tid] : 0.f;
    }
    Pack8<float> zero;
    zero.zero();
#pragma unroll
    for (int o = 0; o < 2; ++o) zero.store(sm.sAcc[o][tid]);

    // x, dt, dy, z of J of this thread's pieces (zeros behind the last token)
    constexpr int J = PIECES < 2 ? 1 : 2;
    Pack8<T> rows[J][4];
    auto load_rows = [&](int64_t t0, int len, int u0) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int t = pt + (u0 + j) * TS;
#pragma unroll
            for (int i = 0; i < 4; ++i) rows[j][i].zero();
            if (!pon || t >= len) continue;
            const size_t at = (t0 + t) * ldx + pc;
            rows[j][0].load(dt + at);
            rows[j][1].load(x + at);
            rows[j][2].load(dy + at);
            if (z) rows[j][3].load(z + at);
        }
    };

    constexpr int PK = (BT * N_ / 8 + kThreads - 1) / kThreads;
    Pack8<T> nB[PK], nC[PK];  // the next stage's B and C,
    int have = kSsmTile;      // of the tokens from this one on (none: kSsmTile)
    for (int64_t k = (e - b + kSsmTile - 1) / kSsmTile - 1; k >= 0; --k, have += kSsmTile) {
        const int64_t t0 = b + k * kSsmTile;
        const int len = (int)min((int64_t)kSsmTile, e - t0);
        F2 h[NP];
        {
            const float *from = k == 0 ? a.S0 ? a.S0 + s * nstate : nullptr : a.tiles + (ssm_tile0(b, s) + k) * nstate;
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                h[p] = f2(0.f, 0.f);
                if (from) h[p].v = *reinterpret_cast<const unsigned long long *>(from + own + 2 * p);
            }
        }
        load_rows(t0, len, 0);
        if (k > 0) {  // the next block's rows into the L2 cache
#pragma unroll
            for (int u = 0; u < PIECES; ++u) {
                const size_t at = (t0 - kSsmTile + pt + u * TS) * ldx + pc;
                if (!pon) break;
                asm volatile("prefetch.global.L2 [%0];" ::"l"(dt + at));
                asm volatile("prefetch.global.L2 [%0];" ::"l"(x + at));
                asm volatile("prefetch.global.L2 [%0];" ::"l"(dy + at));
                if (z) asm volatile("prefetch.global.L2 [%0];" ::"l"(z + at));
            }
        }
        __syncthreads();  // the block before has been read out
#pragma unroll 1
        for (int u0 = 0; u0 < PIECES; u0 += J) {
            if (u0) load_rows(t0, len, u0);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int t = pt + (u0 + j) * TS;
                if (t >= (len + UG - 1) / UG * UG) break;
                float dl[8], xv[8], ev[8];
                rows[j][0].get(dl);
                rows[j][1].get(xv);
                rows[j][2].get(ev);
                if (pon && t < len) {
                    float bias[8];
                    Pack8<float> par;
                    par.load(sm.sPar[0] + pc);
                    par.get(bias);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        dl[i] += bias[i];
                        if (a.softplus) dl[i] = softplus_f(dl[i]);
                    }
                    if (z) {
                        float zv[8];
                        rows[j][3].get(zv);
#pragma unroll
                        for (int i = 0; i < 8; ++i) ev[i] *= silu_f(zv[i]);
                    }
                    // exp2_poly2's limits turn a NaN into a number: a step that is none goes into the chain here instead
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (dl[i] != dl[i]) ev[i] = dl[i];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<float4 *>(sm.sX + t * kX + (pc + i) * 4) = make_float4(dl[i], dl[i] * xv[i], ev[i], 0.f);
            }
        }
        // B and C of the tokens v0 .. v0 + BT - 1 of this block (of the next one, where v0 < 0), zeros behind the last:
        // loaded while the stage before is worked on, then put down
        auto fetch = [&](int v0) {
            if (t0 + v0 < b) return;
            have = v0;
#pragma unroll
            for (int i = 0; i < PK; ++i) {
                const int p = tid + i * kThreads, t = v0 + p / (N_ / 8);
                nB[i].zero(), nC[i].zero();
                if (p < BT * N_ / 8 && t < len) {
                    const size_t at = (size_t)(t0 + t) * ldb + (p % (N_ / 8)) * 8;
                    nB[i].load(Bp + at);
                    nC[i].load(Cp + at);
                }
            }
        };
        auto stage = [&](int v0) {
            if (have != v0) fetch(v0);
#pragma unroll
            for (int i = 0; i < PK; ++i) {
                const int p = tid + i * kThreads;
                if (p >= BT * N_ / 8) break;
                W::put(sm.sBC + p / (N_ / 8) * W::kWords, p % (N_ / 8), nB[i], nC[i]);
            }
        };
        auto behind = [&](int v0, int ta) { return v0 - BT >= ta ? v0 - BT : ta > 0 ? ta - EB : -kSsmTile; };  // the reverse order

        // forwards over the tokens [ta, tb); `keep`: the state before each group
        auto fold = [&](int ta, int tb, bool keep) {
#pragma unroll 1
            for (int v0 = ta; v0 < tb; v0 += BT) {
                __syncthreads();
                stage(v0);
                fetch(v0 + BT < tb || !keep ? v0 + BT : behind(v0, ta));
                __syncthreads();
#pragma unroll 1
                for (int v = 0; v < BT && v0 + v < tb; v += UG) {
                    F2 av[UG][NP], bv[UG][NP];
#pragma unroll
                    for (int u = 0; u < UG; ++u) {
                        const float2 w = *reinterpret_cast<const float2 *>(sm.sX + (v0 + v + u) * kX + ch * 4);
                        F2 Cv[NP];
                        W::get(sm.sBC + (v + u) * W::kWords, q, bv[u], Cv);
#pragma unroll
                        for (int p = 0; p < NP; ++p) {
                            av[u][p] = exp2_pair(mul2(f2(w.x, w.x), A2[p]));
                            bv[u][p] = mul2(f2(w.y, w.y), bv[u][p]);
                        }
                    }
                    if (keep) {
#pragma unroll
                        for (int p = 0; p < NP; ++p) sm.sEnt[(v0 - ta + v) / UG][p][tid] = h[p].v;
                    }
#pragma unroll
                    for (int u = 0; u < UG; ++u)
#pragma unroll
                        for (int p = 0; p < NP; ++p) h[p] = fma2(av[u][p], h[p], bv[u][p]);
                }
            }
        };
        if constexpr (EB < kSsmTile) {
            for (int ta = 0; ta < len; ta += EB) {
#pragma unroll
                for (int p = 0; p < NP; ++p) sm.sTop[ta / EB][p][tid] = h[p].v;
                if (ta + EB < len) fold(ta, ta + EB, false);
            }
        }
#pragma unroll 1
        for (int ta = (len - 1) / EB * EB; ta >= 0; ta -= EB) {
        if constexpr (EB < kSsmTile) {
#pragma unroll
            for (int p = 0; p < NP; ++p) h[p].v = sm.sTop[ta / EB][p][tid];
        }
        const int tb = min(ta + EB, len), subs = (tb + BT - 1) / BT;
        fold(ta, tb, true);
        // backwards, group by group
#pragma unroll 1
        for (int sb = subs - 1; sb >= ta / BT; --sb) {
            if (sb != subs - 1) {  // (the last one is still staged)
                stage(sb * BT);
                fetch(behind(sb * BT, ta));
                __syncthreads();
            }
            const int groups = min((len - sb * BT + UG - 1) / UG, BT / UG);
#pragma unroll 1
            for (int v = (groups - 1) * UG; v >= 0; v -= UG) {
                const int t = sb * BT + v;
                F2 av[UG][NP], ah[UG][NP], bv[UG][NP], vB[UG][NP], vC[UG][NP];
                float4 w[UG];
                F2 groupA[NP];
                float sq[UG], ss[UG], sy[UG];
#pragma unroll
                for (int u = 0; u < UG; ++u) {
                    w[u] = *reinterpret_cast<const float4 *>(sm.sX + (t + u) * kX + ch * 4);
                    F2 Cv[NP];
                    W::get(sm.sBC + (v + u) * W::kWords, q, bv[u], Cv);
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        av[u][p] = exp2_poly2(mul2(f2(w[u].x, w[u].x), A2[p]));
                        bv[u][p] = mul2(f2(w[u].y, w[u].y), bv[u][p]);
                    }
                }
#pragma unroll
                for (int p = 0; p < NP; ++p) h[p].v = sm.sEnt[(t - ta) / UG][p][tid];
#pragma unroll
                for (int u = 0; u < UG; ++u)
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        ah[u][p] = mul2(av[u][p], h[p]);
                        h[p] = add2(ah[u][p], bv[u][p]);
                    }
#pragma unroll
                for (int u = UG - 1; u >= 0; --u) {
                    const F2 dl = f2(w[u].x, w[u].x), dx = f2(w[u].y, w[u].y), ev = f2(w[u].z, w[u].z);
                    F2 tq = f2(0.f, 0.f), ts = tq, ty = tq, Bv[NP], Cv[NP];
                    W::get(sm.sBC + (v + u) * W::kWords, q, Bv, Cv);
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        const F2 hv = add2(ah[u][p], bv[u][p]);
                        const F2 Gv = fma2(Cv[p], ev, r[p]);
                        const F2 pv = mul2(Gv, ah[u][p]);
                        ty = p ? fma2(Cv[p], hv, ty) : mul2(Cv[p], hv);
                        tq = p ? fma2(A1[p], pv, tq) : mul2(A1[p], pv);
                        ts = p ? fma2(Bv[p], Gv, ts) : mul2(Bv[p], Gv);
                        groupA[p] = u == UG - 1 ? mul2(pv, dl) : fma2(pv, dl, groupA[p]);
                        vB[u][p] = mul2(Gv, dx);
                        vC[u][p] = mul2(hv, ev);
                        r[p] = mul2(av[u][p], Gv);
                    }
                    float lo, hi;
                    unpack(tq, lo, hi);
                    sq[u] = lo + hi;
                    unpack(ts, lo, hi);
                    ss[u] = lo + hi;
                    unpack(ty, lo, hi);
                    sy[u] = lo + hi;
                }
#pragma unroll
                for (int p = 0; p < NP; ++p) blockA[p] = add2(blockA[p], groupA[p]);
                // over the channel's lanes: lane q keeps the tokens u = q mod UG
#pragma unroll
                for (int m = LPC / 2; m > 0; m >>= 1) {
#pragma unroll
                    for (int u = 0; u < UG; ++u) {
                        if (m >= UG) {
                            sq[u] += __shfl_xor_sync(0xffffffffu, sq[u], m);
                            ss[u] += __shfl_xor_sync(0xffffffffu, ss[u], m);
                            sy[u] += __shfl_xor_sync(0xffffffffu, sy[u], m);
                            continue;
                        }
                        if (u & m || u % LPC >= 2 * m) continue;
                        const bool up = q & m;
                        float give = up ? sq[u] : sq[u + m], keep = up ? sq[u + m] : sq[u];
                        sq[u] = keep + __shfl_xor_sync(0xffffffffu, give, m);
                        give = up ? ss[u] : ss[u + m], keep = up ? ss[u + m] : ss[u];
                        ss[u] = keep + __shfl_xor_sync(0xffffffffu, give, m);
                        give = up ? sy[u] : sy[u + m], keep = up ? sy[u + m] : sy[u];
                        sy[u] = keep + __shfl_xor_sync(0xffffffffu, give, m);
                    }
                }
                constexpr int STEP = LPC < UG ? LPC : UG;  // a lane's tokens lie this far apart
#pragma unroll
                for (int u = 0; u < UG; u += STEP)
                    if (LPC <= UG || q < UG)
                        *reinterpret_cast<float4 *>(sm.sX + (t + u + q % STEP) * kX + ch * 4) = make_float4(sq[u], ss[u], sy[u], 0.f);
                // over the warp's channels: 16 values of dB and of dC, dealt to the lanes of the same states
                float f[2][16];
#pragma unroll
                for (int u = 0; u < UG; ++u)
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        unpack(vB[u][p], f[0][u * NS + 2 * p], f[0][u * NS + 2 * p + 1]);
                        unpack(vC[u][p], f[1][u * NS + 2 * p], f[1][u * NS + 2 * p + 1]);
                    }
                const int c = lane / LPC;  // channel in the warp
#pragma unroll
                for (int m = G_ / 2, n = 8; m > 0; m >>= 1, n >>= 1) {
                    const bool up = c & m;
#pragma unroll
                    for (int o = 0; o < 2; ++o)
#pragma unroll
                        for (int i = 0; i < n; ++i) {
                            const float give = up ? f[o][i] : f[o][i + n], keep = up ? f[o][i + n] : f[o][i];
                            f[o][i] = keep + __shfl_xor_sync(0xffffffffu, give, m * LPC);
                        }
                }
#pragma unroll
                for (int i = 0; i < 16 / G_; i += NS < 4 ? NS : 4) {
                    const int at = v * N_ + (i / NS % 2 ? red1 : red0) + i / NS / 2 * 2 * N_ + i % NS;
#pragma unroll
                    for (int o = 0; o < 2; ++o) {
                        float *to = sm.sRed[o][warp] + at;
                        if constexpr (NS == 2) *reinterpret_cast<float2 *>(to) = make_float2(f[o][i], f[o][i + 1]);
                        else *reinterpret_cast<float4 *>(to) = make_float4(f[o][i], f[o][i + 1], f[o][i + 2], f[o][i + 3]);
                    }
                }
            }
            __syncthreads();
            for (int i = tid; i < groups * UG * N_; i += kThreads) {
                const int t = sb * BT + i / N_;
                if (t >= len) break;
                const int from = M::slot(i / N_) * N_ + i % N_;
                float vb = 0.f, vc = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) vb += sm.sRed[0][w][from], vc += sm.sRed[1][w][from];
                const size_t at = ((size_t)blk * a.total + t0 + t) * N_ + i % N_;
                pB[at] = vb;
                pC[at] = vc;
            }
            if (sb > ta / BT) __syncthreads();
        }
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            dA[p] = add2(dA[p], blockA[p]);
            blockA[p] = f2(0.f, 0.f);
        }
        load_rows(t0, len, 0);
        __syncthreads();
        // the rows' gradients
#pragma unroll 1
        for (int u0 = 0; u0 < PIECES; u0 += J) {
            if (u0) load_rows(t0, len, u0);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int t = pt + (u0 + j) * TS;
                if (!pon || t >= len) break;
                const size_t at = (t0 + t) * ldx + pc;
                float dtv[8], xv[8], dyv[8], o0[8], o1[8], o2[8], zv[8], bias[8], skip[8], dD[8], db[8];
                Pack8<float> w;
                w.load(sm.sPar[0] + pc);
                w.get(bias);
                w.load(sm.sPar[1] + pc);
                w.get(skip);
                w.load(sm.sAcc[0][tid]);
                w.get(dD);
                w.load(sm.sAcc[1][tid]);
                w.get(db);
                rows[j][0].get(dtv);
                rows[j][1].get(xv);
                rows[j][2].get(dyv);
                rows[j][3].get(zv);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 w = *reinterpret_cast<const float4 *>(sm.sX + t * kX + (pc + i) * 4);
                    const float raw = dtv[i] + bias[i], dl = a.softplus ? softplus_f(raw) : raw;
                    float ev = dyv[i];
                    if (z) {
                        const float sg = sigmoid_f(zv[i]);
                        o2[i] = dyv[i] * fmaf(skip[i], xv[i], w.z) * sg * fmaf(zv[i], 1.f - sg, 1.f);
                        ev *= zv[i] * sg;
                    }
                    o0[i] = fmaf(dl, w.y, skip[i] * ev);
                    const float dd = fmaf(xv[i], w.y, w.x);
                    o1[i] = a.softplus ? dd * sigmoid_f(raw) : dd;
                    dD[i] = fmaf(ev, xv[i], dD[i]);
                    db[i] += o1[i];
                }
                w.set(dD);
                w.store(sm.sAcc[0][tid]);
                w.set(db);
                w.store(sm.sAcc[1][tid]);
                const size_t to = at + d0;
                w.set(o0);
                w.store_stream(g.dx + to);
                w.set(o1);
                w.store_stream(g.ddt + to);
                if (z) {
                    w.set(o2);
                    w.store_stream(g.dz + to);
                }
            }
        }
    }
    if (on) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            *reinterpret_cast<unsigned long long *>(pA + s * nstate + own + 2 * p) = dA[p].v;
            if (g.dS0) *reinterpret_cast<unsigned long long *>(g.dS0 + s * nstate + own + 2 * p) = r[p].v;
        }
    }
    // dD, ddt_bias: the sums of the threads that share 8 channels, in the order of their tokens
    __syncthreads();
    for (int i = tid; i < 2 * nc; i += kThreads) {
        const int c = i % nc;
        float v = 0.f;
        for (int t = 0; t < TS; ++t) v += sm.sAcc[i / nc][c / 8 * TS + t][c % 8];
        (i < nc ? pD : pbias)[(size_t)s * ldx + d0 + c] = v;
    }
}

// dB, dC: the channel blocks' partial sums of each group, added by kSumLanes threads per value and then
// over those, in order.
constexpr int kSumLanes = 8;
__global__ void __launch_bounds__(256)
ssm_sum_kernel(const SsmArgs a, const int bpg, const float *__restrict__ pB, const float *__restrict__ pC,
               float *__restrict__ dB, float *__restrict__ dC) {
    __shared__ float4 red[kSumLanes][32];
    const int n4 = a.states / 4, lane = threadIdx.x / 32, me = threadIdx.x % 32;
    const int64_t i = (int64_t)blockIdx.x * 32 + me;
    const int64_t rows = a.cu ? a.cu[a.N] : a.total;
    const bool on = i < rows * a.groups * n4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) {
        const int64_t t = i / (a.groups * n4);
        const int grp = (int)(i / n4 % a.groups), j = (int)(i % n4);
        const float4 *from = reinterpret_cast<const float4 *>(blockIdx.y ? pC : pB) + ((size_t)grp * bpg * a.total + t) * n4 + j;
        const size_t ld = (size_t)a.total * n4;
#pragma unroll 8
        for (int k = lane; k < bpg; k += kSumLanes) {
            const float4 w = __ldcs(from + k * ld);
            v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
        }
    }
    red[lane][me] = v;
    __syncthreads();
    if (lane || !on) return;
#pragma unroll
    for (int k = 1; k < kSumLanes; ++k) {
        const float4 w = red[k][me];
        v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
    }
    reinterpret_cast<float4 *>(blockIdx.y ? dC : dB)[i] = v;
}

// dA, dD, ddt_bias: over the sequences. One thread per value of [dA | dD | ddt_bias].
__global__ void __launch_bounds__(256)
ssm_param_kernel(const int N, const int channels, const int states, const float *__restrict__ pA, const float *__restrict__ pD,
                 const float *__restrict__ pbias, float *__restrict__ dA, float *__restrict__ dD, float *__restrict__ dbias) {
    const int64_t nA = (int64_t)channels * states;
    int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const float *from = pA;
    float *to = dA;
    int64_t ld = nA;
    if (i >= nA) {
        const bool second = i >= nA + channels;
        i -= second ? nA + channels : nA;
        if (i >= channels) return;
        from = second ? pbias : pD;
        to = second ? dbias : dD;
        ld = channels;
    }
    if (!to) return;
    float v = 0.f;
    for (int s0 = 0; s0 < N; s0 += 64) {  // 64 at a time: short sums keep their bits
        float part = 0.f;
        const int s1 = min(s0 + 64, N);
#pragma unroll 8
        for (int s = s0; s < s1; ++s) part += from[s * ld + i];
        v += part;
    }
    to[i] = v;
}

int back_lanes(int states) { return states == 8 ? 4 : states <= 32 ? 8 : 16; }
int back_blocks(int channels, int groups, int states) {  // per group
    const int CB = kThreads / back_lanes(states);
    return (channels / groups + CB - 1) / CB;
}

template <typename T, int NS, int LPC>
cudaError_t launch_back(const SsmBackwardArgs &g, cudaStream_t st) {
    const SsmArgs &a = g.f;
    const int bpg = back_blocks(a.channels, a.groups, a.states), nblk = bpg * a.groups;
    const size_t rows = (size_t)nblk * a.total * a.states, nA = (size_t)a.N * a.channels * a.states;
    float *pB = static_cast<float *>(g.ws), *pC = pB + rows, *pA = pC + rows, *pD = pA + nA, *pb = pD + (size_t)a.N * a.channels;
    auto kern = ssm_backward_kernel<T, NS, LPC>;
    constexpr int bytes = sizeof(BackMem<T, NS, LPC>);
    if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); e != cudaSuccess) return e;
    kern<<<(unsigned)((int64_t)a.N * nblk), kThreads, bytes, st>>>(g, nblk, bpg, pB, pC, pA, pD, pb);
    if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    if (a.total > 0) {
        const int64_t n = a.total * a.groups * (a.states / 4);
        ssm_sum_kernel<<<dim3((unsigned)((n + 31) / 32), 2), 256, 0, st>>>(a, bpg, pB, pC, g.dB, g.dC);
        if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    }
    const int64_t n = (int64_t)a.channels * (a.states + 2);
    ssm_param_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(a.N, a.channels, a.states, pA, pD, pb, g.dA, g.dD, g.ddt_bias);
    return cudaGetLastError();
}

template <typename T>
cudaError_t back_t(const SsmBackwardArgs &g, cudaStream_t st) {
    switch (g.f.states) {
    case 8: return launch_back<T, 2, 4>(g, st);
    case 16: return launch_back<T, 2, 8>(g, st);
    case 32: return launch_back<T, 4, 8>(g, st);
    case 64: return launch_back<T, 4, 16>(g, st);
    case 128: return launch_back<T, 8, 16>(g, st);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

size_t ssm_backward_workspace(int64_t total, int N, int channels, int states, int groups) {
    const size_t nblk = (size_t)back_blocks(channels, groups, states) * groups;
    return (2 * nblk * total * states + (size_t)N * channels * (states + 2)) * sizeof(float);
}

cudaError_t ssm_backward(const SsmBackwardArgs &g, bool bf16, cudaStream_t st) {
    return bf16 ? back_t<__nv_bfloat16>(g, st) : back_t<float>(g, st);
}

}  // namespace kda
