// kda_ssm.cu -- the selective state space scan: packed prompts (ssm_scan_kernel) and one token of each
// sequence (ssm_step_kernel).
//
//     delta = softplus(dt + dt_bias),  a_t = e^(delta_t A),  h_t = a_t h_(t-1) + delta_t x_t B_t,
//     y_t = (sum_n C_t h_t + D x_t) silu(z_t)                per channel d and state n.
//
// Prompts. The recurrence is diagonal: per (token, channel, state) one exponential, two products and
// two multiply-adds, nothing a matrix instruction could take (the decay differs per channel AND
// state). With 16 states the exponentials bound it (16 per clock and SM: 8 clocks of a quarter SM for
// a warp's 32; a quarter more for softplus and gate), before memory does (x, dt, z, y move once).
//
// LPC lanes share a channel, NS states each, kept in registers as packed pairs (products and
// multiply-adds two at a time), and walk the tokens of one sequence. Nothing but the chain of
// multiply-adds waits for the token before: a batch's loads, products and exponentials are issued
// before the steps of the batch in front of it. Sums over a channel's lanes are a reduce-scatter of
// shuffles. Half of a CTA's warps do that; the other half do the work per (token, channel) for 32
// tokens at a time, 8 channels (a 16-byte vector of bf16) per thread: softplus and the products before
// the scan (tile i + 1 while the scan walks tile i), skip, gate and store after it (tile i - 1). They also
// copy x, dt, z, B and C two tiles ahead (cp.async, each thread to its own place) and lay B and C out for
// the scan, whose loads from shared memory are what counts: a lane takes (delta, delta x) of two tokens in
// one load, and B and C of bf16 inputs as they came (with both expanded to fp32 and each of delta, delta x
// stored twice, ready for packed arithmetic, the loads kept shared memory 83 % busy: 363 us, not 323).
//
// Where the channels leave most SMs idle the time axis is cut: one pass folds each segment from a zero
// state into its end state and the sum of its steps (the decay of a whole segment is e^(A sum delta),
// one exponential), ssm_join_kernel chains those, and the full pass starts each segment from its true
// state. That takes the exponentials twice.
//
// Measured, 8192 tokens x 4096 channels x 16 states, bf16 with a gate: 323 us (0.83 TB/s; floors 41 us of
// bytes, 145 us of exponentials: one warp of scan per SM quarter waits for its own chain; with two CTAs to
// an SM the exponentials are at 71 % of their rate). What it replaced, before those loads: no split of the
// warps, time axis cut, 409 us; the time axis parallel inside a tile, lanes combining (decay product, end
// state) pairs by a shuffle scan, 525 us.
#include "kda_layer.cuh"

namespace kda {
namespace {

constexpr int kScanThreads = 128;

// What a batch of SU tokens needs that no state enters: decays, inputs, read-out weights of a lane's
// states. w = (delta, delta x) of a token and of the one behind it, bc the rows of B and C.
template <typename T, int SU, int NP, int LPC> struct Batch {
    F2 e[SU][NP], in[SU][NP], c[SU][NP];
    __device__ __forceinline__ void load(const F2 (&A)[NP], const float *sX, int ldw, const float *sBC, int t, int q) {
        using W = SsmWeights<T, NP, LPC>;
        F2 dl[SU];
        float2 w[SU];
#pragma unroll
        for (int u = 0; u < SU; ++u) {
            const float *from = sX + (t + u) / 2 * ldw;
            if (SU % 2) {
                w[u] = reinterpret_cast<const float2 *>(from)[(t + u) % 2];
            } else if (u % 2 == 0) {
                const float4 v = *reinterpret_cast<const float4 *>(from);
                w[u] = make_float2(v.x, v.y), w[u + (SU > 1)] = make_float2(v.z, v.w);
            }
        }
#pragma unroll
        for (int u = 0; u < SU; ++u) {
            dl[u] = f2(w[u].x, w[u].x);
            W::get(sBC + (t + u) * W::kWords, q, in[u], c[u]);
#pragma unroll
            for (int p = 0; p < NP; ++p) in[u][p] = mul2(f2(w[u].y, w[u].y), in[u][p]);
        }
#pragma unroll
        for (int u = 0; u < SU; ++u)
#pragma unroll
            for (int p = 0; p < NP; ++p) e[u][p] = exp2_pair(mul2(dl[u], A[p]));
    }
    // the batch's steps; out = the lane's part of sum C h
    template <bool READ> __device__ __forceinline__ void step(F2 (&h)[NP], int u, float &out) const {
        F2 acc;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            h[p] = fma2(e[u][p], h[p], in[u][p]);
            if (READ) acc = p ? fma2(c[u][p], h[p], acc) : mul2(c[u][p], h[p]);
        }
        if (READ) {
            float lo, hi;
            unpack(acc, lo, hi);
            out = lo + hi;
        }
    }
};

// Segment `slot` of the packed sequences: sequence s owns the slots from cu[s] / L + s on (its
// ceil(length / L) segments fit before the next sequence's; the rest stay empty).
struct Segment {
    int s, seg, len;
    int64_t t0;   // first token
    int64_t end;  // slot of the sequence's last segment
    bool last;
};
__device__ __forceinline__ Segment segment_of(const int32_t *cu, int N, int64_t total, int64_t slot, int L) {
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] / L + (int64_t)mid <= slot) lo = mid;
        else hi = mid - 1;
    }
    const int64_t b = cu ? cu[lo] : 0, e = cu ? cu[lo + 1] : total;
    Segment g;
    g.s = lo;
    g.seg = (int)(slot - (b / L + lo));
    g.t0 = b + (int64_t)g.seg * L;
    const int64_t left = e - g.t0;
    g.len = (int)min((int64_t)L, left);
    g.end = slot - g.seg + (e - b + L - 1) / L - 1;
    g.last = left <= L;
    if (left <= 0 && !(g.seg == 0 && left == 0)) g.s = -1;  // an empty slot
    return g;
}

enum { kFull, kSave, kFold };  // y and final states; tile states too; only the segments' ends

// Shared memory of a CTA, and the sizes that follow from the lanes per channel. Two tiles at a time: the
// scan threads walk one while the others write the next and read the last one out.
constexpr int TT = 32;  // tokens of a tile
template <typename T, int NS, int LPC, int MODE> struct ScanMem {
    static constexpr int N_ = NS * LPC, CB = kScanThreads / LPC;  // states; channels of a CTA
    static constexpr int UT = LPC > 8 ? LPC : 8;        // tokens of a group
    static constexpr int ROWS = TT * CB / 8, PR = (ROWS + kScanThreads - 1) / kScanThreads;      // pieces of 8 channels; per thread
    static constexpr int PIECES = TT * N_ / 8, PK = (PIECES + kScanThreads - 1) / kScanThreads;  // pieces of 8 states of B (C); per thread
    using W = SsmWeights<T, NS / 2, LPC>;
    static constexpr int kX = CB * 4 + 4, kY = CB + 4;  // words per two tokens, per token (padded: threads of consecutive tokens write)
    float sX[2][TT / 2 * kX];     // (delta, delta x) of two tokens
    float sY[2][TT * kY];         // sum C h
    float sBC[2][TT * W::kWords]; // B and C
    Pack8<T> sRow[3][MODE == kFold ? 2 : 3][PR][kScanThreads];  // x, dt, z of three tiles: each thread's own pieces
    Pack8<T> sRaw[MODE == kFold ? 1 : 2][PK][kScanThreads];     // B and C of the next tile likewise
};

template <typename T, int NS, int LPC, int MODE>
__global__ void __launch_bounds__(2 * kScanThreads, 2)
ssm_scan_kernel(const SsmArgs a, const int nblk, const int bpg, const int L, float *__restrict__ seg_state,
                float *__restrict__ seg_step) {
    using M = ScanMem<T, NS, LPC, MODE>;
    constexpr int N_ = M::N_, NP = NS / 2, CB = M::CB, UT = M::UT, PR = M::PR, PK = M::PK;
    constexpr int kX = M::kX, kY = M::kY, SU = NP < 8 ? 8 / NP : 1;  // tokens of a batch: 8 pairs of states
    extern __shared__ __align__(16) char smem_raw[];
    M &sm = *reinterpret_cast<M *>(smem_raw);
    const int tid = threadIdx.x % kScanThreads;
    const int blk = blockIdx.x % nblk;
    const int64_t slot = blockIdx.x / nblk;
    const Segment g = segment_of(a.cu, a.N, a.total, slot, L);
    if (g.s < 0 || (MODE == kFold && g.last)) return;
    const int64_t b = g.t0;
    const int len = g.len, tiles = (len + TT - 1) / TT;

    const int cpg = a.channels / a.groups, grp = blk / bpg, c0 = (blk % bpg) * CB;
    const int nc = min(CB, cpg - c0);  // channels of this block (a multiple of 8)
    const int d0 = grp * cpg + c0;
    const size_t ldx = a.channels, nstate = (size_t)a.channels * N_;

    if (threadIdx.x >= kScanThreads) {
        // ---- rows: copied ahead, made into steps and inputs before the scan, into outputs after it ----
        const size_t ldb = (size_t)a.groups * N_;
        const T *px = static_cast<const T *>(a.x) + b * ldx + d0, *pd = static_cast<const T *>(a.dt) + b * ldx + d0;
        const T *pz = a.z ? static_cast<const T *>(a.z) + b * ldx + d0 : nullptr;
        T *py = static_cast<T *>(a.y) + b * ldx + d0;
        const T *Bp = static_cast<const T *>(a.B) + b * ldb + (size_t)grp * N_, *Cp = static_cast<const T *>(a.C) + b * ldb + (size_t)grp * N_;
        float bias[PR][8], skip[PR][8];
        bool mine[PR];
#pragma unroll
        for (int u = 0; u < PR; ++u) {
            const int p = tid + u * kScanThreads, c = p / TT * 8;
            mine[u] = p < M::ROWS && c < nc;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                bias[u][i] = mine[u] && a.dt_bias ? a.dt_bias[d0 + c + i] : 0.f;
                skip[u][i] = mine[u] && a.D ? a.D[d0 + c + i] : 0.f;
            }
        }
        auto copy_ahead = [&](int tile) {
#pragma unroll
            for (int u = 0; u < PR; ++u) {
                const int p = tid + u * kScanThreads, t = tile * TT + p % TT;
                const bool in = mine[u] && t < len;
                const size_t at = in ? t * ldx + p / TT * 8 : 0;
                copy8(&sm.sRow[tile % 3][0][u][tid], px + at, in);
                copy8(&sm.sRow[tile % 3][1][u][tid], pd + at, in);
                if constexpr (MODE != kFold) {
                    if (pz) copy8(&sm.sRow[tile % 3][2][u][tid], pz + at, in);
                }
            }
#pragma unroll
            for (int u = 0; u < PK; ++u) {
                const int p = tid + u * kScanThreads, t = tile * TT + p / (N_ / 8);
                const bool in = p < M::PIECES && t < len;
                const size_t at = in ? t * ldb + (p % (N_ / 8)) * 8 : 0;
                copy8(&sm.sRaw[0][u][tid], Bp + at, in);
                if constexpr (MODE != kFold) copy8(&sm.sRaw[1][u][tid], Cp + at, in);
            }
            copies_end_group();
        };
        auto before = [&](int tile) {
            copies_wait<0>();
            float *sX = sm.sX[tile & 1];
#pragma unroll
            for (int u = 0; u < PR; ++u) {
                const int p = tid + u * kScanThreads, t = p % TT;
                if (p >= M::ROWS) break;
                float xv[8], dl[8];
                sm.sRow[tile % 3][0][u][tid].get(xv);
                sm.sRow[tile % 3][1][u][tid].get(dl);
#pragma unroll
                for (int i = 0; i < 8; ++i) dl[i] += bias[u][i];
                if (a.softplus) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) dl[i] = softplus_f(dl[i]);
                }
                const bool in = tile * TT + t < len;  // no step behind the last token
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float v = in ? dl[i] : 0.f, w = v * xv[i];
                    *reinterpret_cast<float2 *>(sX + t / 2 * kX + (p / TT * 8 + i) * 4 + t % 2 * 2) = make_float2(v, w);
                }
            }
#pragma unroll
            for (int u = 0; u < PK; ++u) {
                const int p = tid + u * kScanThreads;
                if (p >= M::PIECES) break;
                M::W::put(sm.sBC[tile & 1] + p / (N_ / 8) * M::W::kWords, p % (N_ / 8), sm.sRaw[0][u][tid],
                          sm.sRaw[MODE == kFold ? 0 : 1][u][tid]);  // (the fold has no use for C)
            }
        };
        auto after = [&](int tile) {
            if constexpr (MODE != kFold) {
                const float *sY = sm.sY[tile & 1];
#pragma unroll
                for (int u = 0; u < PR; ++u) {
                    const int p = tid + u * kScanThreads, t = p % TT, c = p / TT * 8;
                    if (!mine[u] || tile * TT + t >= len) continue;
                    float o[8], xv[8], zv[8];
                    sm.sRow[tile % 3][0][u][tid].get(xv);
                    sm.sRow[tile % 3][2][u][tid].get(zv);
#pragma unroll
                    for (int i = 0; i < 8; i += 4) {
                        const float4 v = *reinterpret_cast<const float4 *>(sY + t * kY + c + i);
                        o[i] = v.x, o[i + 1] = v.y, o[i + 2] = v.z, o[i + 3] = v.w;
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        o[i] = fmaf(skip[u][i], xv[i], o[i]);
                        if (pz) o[i] *= silu_f(zv[i]);
                    }
                    Pack8<T> w;
                    w.set(o);
                    w.store_stream(py + (size_t)(tile * TT + t) * ldx + c);
                }
            }
        };
        if (tiles) {
            copy_ahead(0);
            before(0);
            if (tiles > 1) copy_ahead(1);
        }
        __syncthreads();
        for (int i = 0; i < tiles; ++i) {
            if (i) after(i - 1);
            if (i + 1 < tiles) {
                before(i + 1);
                if (i + 2 < tiles) copy_ahead(i + 2);
            }
            __syncthreads();
        }
        if (tiles) after(tiles - 1);
        return;
    }

    // ---- the scan ----
    const int q = tid % LPC, ch = tid / LPC;
    const bool on = ch < nc;
    const size_t own = (size_t)(d0 + (on ? ch : 0)) * N_ + q * NS;
    F2 A[NP], h[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const float2 v = *reinterpret_cast<const float2 *>(a.A + own + 2 * p);
        A[p] = f2(v.x * kLog2e, v.y * kLog2e);
        h[p] = f2(0.f, 0.f);
        // A sequence in several segments: the last one may write S_T over S0 before the first one reads it, so the
        // fold keeps S0 in the last segment's slot, which has no use for its own end state.
        const float *from = g.seg ? MODE == kFold ? nullptr : seg_state + (slot - 1) * nstate
                            : !a.S0 ? nullptr
                            : MODE == kFold || g.last ? a.S0 + g.s * nstate : seg_state + g.end * nstate;
        if (from) h[p].v = *reinterpret_cast<const unsigned long long *>(from + own + 2 * p);
    }
    auto put = [&](float *to) {
        if (!on) return;
#pragma unroll
        for (int p = 0; p < NP; ++p) *reinterpret_cast<unsigned long long *>(to + own + 2 * p) = h[p].v;
    };
    if (MODE == kFold && g.seg == 0) put(seg_state + g.end * nstate);
    float sum = 0.f;  // of the steps (kFold)
    __syncthreads();
    for (int tile = 0; tile < tiles; ++tile) {
        const float *sX = sm.sX[tile & 1] + ch * 4;
        float *sY = sm.sY[tile & 1];
        if (MODE == kSave && tile % (kSsmTile / TT) == 0)
            put(a.tiles + (ssm_tile0(b - (int64_t)g.seg * L, g.s) + (g.seg * (int64_t)L + tile * TT) / kSsmTile) * nstate);
        // The next batch's loads, products and exponentials stand before the current one's steps: they fill the
        // time that its chain of multiply-adds and its shuffles wait.
        Batch<T, SU, NP, LPC> bt[2];
        bt[0].load(A, sX, kX, sm.sBC[tile & 1], 0, q);
#pragma unroll
        for (int tok = 0; tok < TT; tok += UT) {  // (behind the last token: no steps, nothing stored)
            float out[UT];
#pragma unroll
            for (int u0 = 0; u0 < UT; u0 += SU) {
                const int k = (tok + u0) / SU, next = tok + u0 + SU;
                if (next < TT) bt[(k + 1) & 1].load(A, sX, kX, sm.sBC[tile & 1], next, q);
#pragma unroll
                for (int i = 0; i < SU; ++i) {
                    const int u = u0 + i;
                    bt[k & 1].template step<MODE != kFold>(h, i, out[u]);
                    if (MODE == kFold) sum += sX[(tok + u) / 2 * kX + (tok + u) % 2 * 2];
                }
            }
            if (MODE == kFold) continue;
            // sums over the channel's lanes: lane q keeps the tokens u = q mod LPC
#pragma unroll
            for (int m = LPC / 2; m > 0; m >>= 1) {
#pragma unroll
                for (int u = 0; u < UT; ++u) {
                    if (u & m || u % LPC >= 2 * m) continue;
                    const float give = q & m ? out[u] : out[u + m], keep = q & m ? out[u + m] : out[u];
                    out[u] = keep + __shfl_xor_sync(0xffffffffu, give, m);
                }
            }
#pragma unroll
            for (int k = 0; k < UT / LPC; ++k) sY[(tok + k * LPC + q) * kY + ch] = out[k * LPC];
        }
        __syncthreads();
    }
    if (MODE == kFold) {
        put(seg_state + slot * nstate);
        if (on && q == 0) seg_step[slot * ldx + d0 + ch] = sum;
    } else if (g.last && a.S_T) {
        put(a.S_T + g.s * nstate);
    }
}

// True states at the segments' ends: seg_state[k] += e^(A sum delta_k) seg_state[k - 1] along a sequence.
__global__ void __launch_bounds__(kScanThreads)
ssm_join_kernel(const SsmArgs a, const int L, float *__restrict__ seg_state, const float *__restrict__ seg_step) {
    const size_t nstate = (size_t)a.channels * a.states;
    const size_t i = ((size_t)blockIdx.x * kScanThreads + threadIdx.x) * 4;
    const int s = blockIdx.y;
    if (i >= nstate) return;
    const int64_t b = a.cu ? a.cu[s] : 0, e = a.cu ? a.cu[s + 1] : a.total;
    const int64_t slot = b / L + s;
    const int inner = (int)((e - b + L - 1) / L) - 1;  // segments that another one follows
    if (inner < 2) return;
    const int d = (int)(i / a.states);
    float4 A = *reinterpret_cast<const float4 *>(a.A + i);
    A.x *= kLog2e; A.y *= kLog2e; A.z *= kLog2e; A.w *= kLog2e;
    float4 h = *reinterpret_cast<const float4 *>(seg_state + slot * nstate + i);
    constexpr int P = 4;  // segments loaded ahead
    for (int k0 = 1; k0 < inner; k0 += P) {
        float4 v[P];
        float w[P];
#pragma unroll
        for (int k = 0; k < P; ++k)
            if (k0 + k < inner) {
                v[k] = *reinterpret_cast<const float4 *>(seg_state + (slot + k0 + k) * nstate + i);
                w[k] = seg_step[(slot + k0 + k) * a.channels + d];
            }
#pragma unroll
        for (int k = 0; k < P; ++k)
            if (k0 + k < inner) {
                h.x = fmaf(exp2_approx(A.x * w[k]), h.x, v[k].x);
                h.y = fmaf(exp2_approx(A.y * w[k]), h.y, v[k].y);
                h.z = fmaf(exp2_approx(A.z * w[k]), h.z, v[k].z);
                h.w = fmaf(exp2_approx(A.w * w[k]), h.w, v[k].w);
                *reinterpret_cast<float4 *>(seg_state + (slot + k0 + k) * nstate + i) = h;
            }
    }
}

// How the lanes and the time axis are dealt out.
constexpr int kMinSegment = 256;
// Lanes of a channel (in turn on one GPU). 16 states: four lanes 324 us for 8192 tokens of 4096 channels, eight
// 356 us (fewer shuffles against more warps). 64 states: eight lanes 156 us for 6151 tokens of 1024 channels in 16
// sequences, sixteen 179 us.
constexpr int lanes_of(int states) { return states <= 16 ? 4 : 8; }
struct Cut {
    int L;  // tokens of a segment
    int nblk, bpg;
    int64_t slots;
    bool split;
};
// The time axis is cut where the sequences' channels give a CTA to fewer than half of the SMs: a cut takes
// the exponentials twice (8192 tokens of 4096 channels, 128 CTAs: 324 us uncut, 424 us in four segments).
// The rule counts sequences, not their tokens: a batch of one long prompt and many short ones of few channels
// stays uncut.
Cut cut_of(int64_t total, int N, int channels, int states, int groups) {
    const int CB = kScanThreads / lanes_of(states);
    Cut c;
    c.bpg = (channels / groups + CB - 1) / CB;
    c.nblk = c.bpg * groups;
    int64_t L = total;
    if ((int64_t)N * c.nblk * 2 <= 148) {
        const int64_t segs = 148 / c.nblk;  // of all sequences
        L = max(((total + segs - 1) / segs + kSsmTile - 1) / kSsmTile * kSsmTile, (int64_t)kMinSegment);
    }
    c.split = L < total;
    c.L = (int)max(min(L, total), (int64_t)1);
    c.slots = total / c.L + N;
    return c;
}

template <typename T, int NS, int LPC, int MODE>
cudaError_t launch_mode(const SsmArgs &a, const Cut &c, unsigned grid, float *state, float *step, cudaStream_t st) {
    auto kern = ssm_scan_kernel<T, NS, LPC, MODE>;
    constexpr int bytes = sizeof(ScanMem<T, NS, LPC, MODE>);
    if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); e != cudaSuccess) return e;
    kern<<<grid, 2 * kScanThreads, bytes, st>>>(a, c.nblk, c.bpg, c.L, state, step);
    return cudaGetLastError();
}

template <typename T, int NS, int LPC>
cudaError_t launch_scan(const SsmArgs &a, const Cut &c, void *ws, cudaStream_t st) {
    float *state = static_cast<float *>(ws), *step = state + (size_t)c.slots * a.channels * a.states;
    const unsigned grid = (unsigned)(c.slots * c.nblk);
    if (c.split) {
        if (cudaError_t e = launch_mode<T, NS, LPC, kFold>(a, c, grid, state, step, st); e != cudaSuccess) return e;
        const unsigned gx = (unsigned)(((size_t)a.channels * a.states / 4 + kScanThreads - 1) / kScanThreads);
        if (a.total > 2 * (int64_t)c.L) ssm_join_kernel<<<dim3(gx, a.N), kScanThreads, 0, st>>>(a, c.L, state, step);
    }
    return a.tiles ? launch_mode<T, NS, LPC, kSave>(a, c, grid, state, step, st)
                   : launch_mode<T, NS, LPC, kFull>(a, c, grid, state, step, st);
}

template <typename T>
cudaError_t prefill_t(const SsmArgs &a, void *ws, cudaStream_t st) {
    const Cut c = cut_of(a.total, a.N, a.channels, a.states, a.groups);
    switch (a.states) {
    case 8: return launch_scan<T, 2, 4>(a, c, ws, st);
    case 16: return launch_scan<T, 4, 4>(a, c, ws, st);
    case 32: return launch_scan<T, 4, 8>(a, c, ws, st);
    case 64: return launch_scan<T, 8, 8>(a, c, ws, st);
    case 128: return launch_scan<T, 16, 8>(a, c, ws, st);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

size_t ssm_prefill_workspace(int64_t total, int N, int channels, int states, int groups) {
    const Cut c = cut_of(total, N, channels, states, groups);
    return c.split ? ((size_t)c.slots * channels * (states + 1) * sizeof(float) + 15) / 16 * 16 : 0;
}

int ssm_prefill_launches(int64_t total, int N, int channels, int states, int groups) {
    const Cut c = cut_of(total, N, channels, states, groups);
    return c.split ? total > 2 * (int64_t)c.L ? 3 : 2 : 1;
}

cudaError_t ssm_prefill(const SsmArgs &a, void *ws, bool bf16, cudaStream_t st) {
    return bf16 ? prefill_t<__nv_bfloat16>(a, ws, st) : prefill_t<float>(a, ws, st);
}

// ------------------------------------------------------------------- one token ----
//
// Bound by the fp32 state, read and written once (8 bytes per channel and state against 2 of
// arithmetic). A warp owns CPW consecutive channels (their A stays in registers) and walks the
// sequences; a lane holds U 4-state vectors of them, n / 4 lanes to a channel, so every access is
// a run of 16-byte vectors. The per-channel work (softplus, gate) is done by one lane per channel
// and handed over by shuffles; C h is summed over a channel's lanes by shuffles. Measured, 256 sequences
// x 4096 channels x 16 states in bf16 (143 MB): 28 to 31 us, 70 to 77 % of the copy rate. Six CTAs to an SM cap
// the registers at 80: 20 to 36 bytes a thread spill at 16 to 128 states.
namespace {

constexpr int kStepThreads = 128, kStepPerSm = 6;

template <typename T, int NS>
__global__ void __launch_bounds__(kStepThreads, kStepPerSm)
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
    float4 nh[U];
    auto load_state = [&](int s) {
        const float4 *S = reinterpret_cast<const float4 *>(a.S_T + ((size_t)s * D + base) * NS);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (on[u] && s < a.N) nh[u] = __ldcs(S + u * 32 + lane);
    };
    load_state(blockIdx.y);
    for (int s = blockIdx.y; s < a.N; s += gridDim.y) {
        float4 h[U];
        float *S = a.S_T + ((size_t)s * D + base) * NS;
#pragma unroll
        for (int u = 0; u < U; ++u) h[u] = nh[u];
        load_state(s + gridDim.y);
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
    // six CTAs to an SM, all at once: a warp walks the rest of the sequences, the next one's state loaded ahead
    const unsigned gy = (unsigned)max((int64_t)1, min((int64_t)a.N, (int64_t)(148 * kStepPerSm) / gx));
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
