// kda_conv_layer.cu -- the short convolution + Swish with a bias, for one token of each sequence, and
// its gradients:
//
//     v_t[c] = bias[c] + sum_j w[c][j] x_(t-W+1+j)[c],   y = v sigmoid(v),
//     g = dy sigmoid(v) (1 + v (1 - sigmoid(v))),
//     dx_t = sum_j w[j] g_(t+W-1-j) (tokens of the same sequence),  dw[j] = sum_t g_t x_(t-W+1+j),  dbias = sum g,
//
// rows before a sequence's first token being its initial state (which gets dx's share as dstate).
//
// All of it is bound by memory: x (and dy) read once, y (dx) written once. A thread owns 4 consecutive
// channels of a run of consecutive tokens and keeps the window in registers (8 channels halve the loads and
// double the registers: 117 us against 85 us for an earlier backward of 8192 tokens x 4096 channels, W = 4).
// It loads some rows ahead, so that bytes are in flight: the forward (32 us for that size, 64 % of the copy rate;
// it waits for those loads, its schedulers issue in 56 % of the clocks, its exponentials and reciprocals run at 49 %
// of their rate) to registers, the backward, which has none left, to shared memory (60 us with an fp32 dy, 85 % of
// the copy rate; to registers and none further ahead 85 us). The rows around its run that its window needs are its
// neighbours' too and come from the L2 cache.
#include <type_traits>

#include "kda_layer.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;

// The last s with cu[s] <= t: the sequence of token t (t < cu[N]; the empty ones before it are skipped).
__device__ __forceinline__ int sequence_of(const int32_t *cu, int N, int64_t t) {
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Row `pos` of a sequence that starts at token b (pos < 0: from its initial state, or zero).
template <int W, typename P, typename T>
__device__ __forceinline__ void window_row(P &r, const T *x, const T *state, int64_t b, int64_t pos, int s, int C) {
    if (pos >= 0) r.load(x + (size_t)(b + pos) * C);
    else if (state) r.load(state + ((size_t)s * (W - 1) + (W - 1 + pos)) * C);
    else r.zero();
}
template <int W, int V, typename T>
__device__ __forceinline__ void window_row(float (&v)[V], const T *x, const T *state, int64_t b, int64_t pos, int s, int C) {
    Pack<T, V> r;
    window_row<W>(r, x, state, b, pos, s, C);
    r.get(v);
}

// The taps of V channels lie together: loads of 16 bytes where w allows them.
template <int W, int V> __device__ __forceinline__ void load_taps(const float *w, int c0, float (&tap)[W][V]) {
    const float *from = w + (size_t)c0 * W;
    float v[V * W];
    if ((reinterpret_cast<uintptr_t>(w) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < V * W / 4; ++i) *reinterpret_cast<float4 *>(v + 4 * i) = reinterpret_cast<const float4 *>(from)[i];
    } else {
#pragma unroll
        for (int i = 0; i < V * W; ++i) v[i] = from[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) tap[j][i] = v[i * W + j];
}

template <int V> __device__ __forceinline__ void load_bias(const float *bias, int c0, float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = bias ? bias[c0 + i] : 0.f;
}

// ---- prompts ----

constexpr int kRun = 32, kVec = 4;                         // tokens and channels of a thread's run
constexpr int ahead(int W) { return W > 4 ? 1 : 4; }       // rows loaded together (wide windows take the registers)
constexpr int ring(int W) { return W > 4 ? 8 : 2; }        // such groups in the backward's ring (three: 62 us, not 60)

template <int W, int V, typename T>
__global__ void __launch_bounds__(kThreads)
conv_bias_kernel(const ConvArgs a) {
    constexpr int kAhead = ahead(W);
    const int nv = a.C / V;
    const int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x, t0 = g / nv * kRun;
    const int c0 = (int)(g % nv) * V;
    const int64_t rows = a.cu ? a.cu[a.N] : a.total;
    if (t0 >= rows) return;
    const T *x = static_cast<const T *>(a.x) + c0;
    const T *st = a.state_in ? static_cast<const T *>(a.state_in) + c0 : nullptr;
    T *y = static_cast<T *>(a.y) + c0;
    float tap[W][V], bias[V];
    load_taps<W, V>(a.w, c0, tap);
    load_bias(a.bias, c0, bias);
    int s = a.cu ? sequence_of(a.cu, a.N, t0) : 0;
    int64_t b = a.cu ? a.cu[s] : 0, e = a.cu ? a.cu[s + 1] : a.total;
    const int64_t t1 = min(t0 + kRun, rows);
    float win[W][V];  // win[W - 1]: the current row
    auto fill = [&](int64_t t) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) window_row<W, V>(win[j], x, st, b, t - b - (W - 1) + j, s, a.C);
    };
    fill(t0);
    // n tokens of the current sequence from t on (`whole`: kAhead of them)
    auto tokens = [&](auto whole, int64_t t, int n) {
        constexpr bool kWhole = decltype(whole)::value;
        const T *px = x + (size_t)t * a.C;
        T *py = y + (size_t)t * a.C;
        Pack<T, V> next[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k, px += a.C)
            if (kWhole || k < n) next[k].load(px);
#pragma unroll
        for (int k = 0; k < kAhead; ++k, py += a.C) {
            if (!kWhole && k >= n) break;
            next[k].get(win[W - 1]);
            float v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = bias[i];
#pragma unroll
            for (int j = 0; j < W; ++j) {
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = fmaf(tap[j][i], win[j][i], v[i]);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = silu_f(v[i]);
            Pack<T, V> o;
            o.set(v);
            o.store_stream(py);
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) win[j][i] = win[j + 1][i];
        }
    };
    for (int64_t t = t0; t < t1;) {
        if (t == e) {  // the next sequence (skipping the empty ones)
            do {
                ++s;
                b = a.cu[s];
                e = a.cu[s + 1];
            } while (e == b);
            fill(t);
        }
        const int n = (int)min((int64_t)kAhead, min(t1, e) - t);
        if (n == kAhead) tokens(std::true_type{}, t, n);
        else tokens(std::false_type{}, t, n);
        t += n;
    }
}

// Each sequence's last W - 1 raw rows (a thread reads all of its rows before it writes: in place is safe).
template <int W, typename T>
__global__ void __launch_bounds__(kThreads)
conv_last_kernel(const ConvArgs a) {
    if constexpr (W > 1) {
        const int nv = a.C / 8;
        const int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x;
        if (g >= (int64_t)a.N * nv) return;
        const int s = (int)(g / nv), c0 = (int)(g % nv) * 8;
        const int64_t b = a.cu ? a.cu[s] : 0, e = a.cu ? a.cu[s + 1] : a.total;
        const T *x = static_cast<const T *>(a.x) + c0;
        const T *st = a.state_in ? static_cast<const T *>(a.state_in) + c0 : nullptr;
        T *to = static_cast<T *>(a.state_out) + c0;
        Pack8<T> r[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) window_row<W>(r[j], x, st, b, e - b - (W - 1) + j, s, a.C);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) r[j].store(to + ((size_t)s * (W - 1) + j) * a.C);
    }
}

// ---- one token of each sequence: window = state and the new row, the state shifted in place ----

template <int W, typename T>
__global__ void __launch_bounds__(kThreads)
conv_step_kernel(const ConvArgs a) {
    const int nv = a.C / 8, v0 = blockIdx.x * kThreads + threadIdx.x;
    if (v0 >= nv) return;
    const int c0 = v0 * 8;
    const T *x = static_cast<const T *>(a.x) + c0;
    T *st = static_cast<T *>(a.state_out) + c0, *y = static_cast<T *>(a.y) + c0;
    float tap[W][8], bias[8];
    load_taps<W, 8>(a.w, c0, tap);
    load_bias(a.bias, c0, bias);
    for (int64_t s = blockIdx.y; s < a.N; s += gridDim.y) {
        Pack8<T> win[W];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) win[j].load(st + ((size_t)s * (W - 1) + j) * a.C);
        win[W - 1].load(x + (size_t)s * a.C);
        float v[8], r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = bias[i];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            win[j].get(r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fmaf(tap[j][i], r[i], v[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = silu_f(v[i]);
        Pack8<T> o;
        o.set(v);
        o.store(y + (size_t)s * a.C);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) win[j + 1].store(st + ((size_t)s * (W - 1) + j) * a.C);
    }
}

// ---- gradients ----
//
// A thread's run takes the g of its tokens and of the W - 1 behind them (which the
// next run forms too) and writes its dx. Its sums for dw and dbias go to the workspace, a row per run,
// and conv_sum_kernel adds the runs in order. A sequence's dstate is written by the thread of its first
// token, which holds the g of its first W - 1 tokens.

// Long runs cost less (a row of partial sums each, W - 1 tokens formed twice), short ones fill the GPU: runs
// that give every lane of four CTAs per SM one each, or as many each as keep them at 128 tokens (whose sums
// keep their bits), and at least 32 tokens (8192 tokens x 4096 channels: runs of 128, 64 of 74, 67 us).
int back_run(int64_t total, int C) {
    const int64_t lanes = max((int64_t)148 * 4 * kThreads * kVec / C, (int64_t)1);
    const int64_t runs = max((total + 128 * lanes - 1) / (128 * lanes), (int64_t)1) * lanes;
    return (int)max(((total + runs - 1) / runs + 3) / 4 * 4, (int64_t)32);
}

template <int W, int V, typename T, typename TG>
__global__ void __launch_bounds__(kThreads, W <= 4 ? 4 : 1)
conv_backward_kernel(const ConvBackwardArgs p, float *__restrict__ part, const int run_len) {
    constexpr int kAhead = ahead(W), kRing = ring(W);
    const ConvArgs &a = p.f;
    const int nv = a.C / V;
    const int64_t gid = (int64_t)blockIdx.x * kThreads + threadIdx.x, run = gid / nv, t0 = run * run_len;
    if (t0 >= a.total) return;
    const int c0 = (int)(gid % nv) * V;
    const int64_t rows = a.cu ? a.cu[a.N] : a.total;
    const T *x = static_cast<const T *>(a.x) + c0;
    const T *st = a.state_in ? static_cast<const T *>(a.state_in) + c0 : nullptr;
    const TG *dy = static_cast<const TG *>(p.dy) + c0;
    __shared__ Pack<T, V> ring_x[kRing * kAhead][kThreads];
    __shared__ Pack<TG, V> ring_dy[kRing * kAhead][kThreads];
    float tap[W][V], bias[V], dw[W][V], db[V];
    load_taps<W, V>(a.w, c0, tap);
    load_bias(a.bias, c0, bias);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = 0.f;
    }
    if (t0 < rows) {
        int s = a.cu ? sequence_of(a.cu, a.N, t0) : 0;
        int64_t b = a.cu ? a.cu[s] : 0, e = a.cu ? a.cu[s + 1] : a.total;
        const int64_t t1 = min(t0 + run_len, rows), tl = min(t1 + W - 1, rows);  // the run, and what its dx needs
        float win[W][V];
        float acc[W][V];  // acc[j]: dx of row t - (W - 1) + j, so far
        auto start = [&](int64_t t) {  // the window of token t of the current sequence, nothing summed yet
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                window_row<W, V>(win[j], x, st, b, t - b - (W - 1) + j, s, a.C);
#pragma unroll
                for (int i = 0; i < V; ++i) acc[j][i] = 0.f;
            }
        };
        auto flush = [&](int64_t t, int j) {  // acc[j], of row t, is complete: dx, or a row of the initial state
            Pack<float, V> o;
            o.set(acc[j]);
            if (t >= b) {
                if (t >= t0 && t < t1) o.store_stream(p.dx + (size_t)t * a.C + c0);
            } else if (p.dstate && t0 <= b) {
                o.store(p.dstate + ((size_t)s * (W - 1) + (t - b + W - 1)) * a.C + c0);
            }
        };
        // x and dy come through a ring of kRing groups of kAhead rows, each thread's its own (no barrier)
        auto copy = [&](int64_t t, int at) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (t + k >= tl) break;
                copy_pack(&ring_x[at + k][threadIdx.x], x + (size_t)(t + k) * a.C);
                copy_pack(&ring_dy[at + k][threadIdx.x], dy + (size_t)(t + k) * a.C);
            }
            copies_end_group();
        };
#pragma unroll
        for (int i = 0; i < kRing - 1; ++i) copy(t0 + i * kAhead, i * kAhead);
        int head = 0;  // the current group's place
        start(t0);
        // n tokens of the current sequence from t on, in one group, the rows from `at` on of the ring (`inner`: kAhead of
        // them, in the run, and so are the rows whose dx they complete)
        auto tokens = [&](auto inner, int64_t t, int n, int at) {
            constexpr bool kInner = decltype(inner)::value;
            float *pd = p.dx + (size_t)(t - (W - 1)) * a.C + c0;
#pragma unroll
            for (int k = 0; k < kAhead; ++k, pd += a.C) {
                if (!kInner && k >= n) break;
                ring_x[at + k][threadIdx.x].get(win[W - 1]);
                float v[V], g[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    v[i] = bias[i];
                    acc[W - 1][i] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < W; ++j) {
#pragma unroll
                    for (int i = 0; i < V; ++i) v[i] = fmaf(tap[j][i], win[j][i], v[i]);
                }
                ring_dy[at + k][threadIdx.x].get(g);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float sg = sigmoid_f(v[i]);
                    g[i] *= sg * fmaf(v[i], 1.f - sg, 1.f);
                }
#pragma unroll
                for (int j = 0; j < W; ++j)
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[j][i] = fmaf(tap[j][i], g[i], acc[j][i]);
                if (kInner || t + k < t1) {
#pragma unroll
                    for (int i = 0; i < V; ++i) db[i] += g[i];
#pragma unroll
                    for (int j = 0; j < W; ++j) {
#pragma unroll
                        for (int i = 0; i < V; ++i) dw[j][i] = fmaf(g[i], win[j][i], dw[j][i]);
                    }
                }
                if (kInner) {
                    Pack<float, V> o;
                    o.set(acc[0]);
                    o.store_stream(pd);
                } else {
                    flush(t + k - (W - 1), 0);
                }
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        win[j][i] = win[j + 1][i];
                        acc[j][i] = acc[j + 1][i];
                    }
            }
        };
        for (int64_t t = t0; t < tl;) {
            if (t == e) {  // the next sequence: what the last rows of this one have is all they get
#pragma unroll
                for (int j = 0; j < W - 1; ++j) flush(e - (W - 1) + j, j);
                if (t >= t1) {
                    e = -1;
                    break;
                }
                do {
                    ++s;
                    b = a.cu[s];
                    e = a.cu[s + 1];
                } while (e == b);
                start(t);
            }
            const int in = (int)(t - t0) % kAhead;
            if (in == 0) {
                copy(t + (kRing - 1) * kAhead, (head + (kRing - 1) * kAhead) % (kRing * kAhead));
                copies_wait<kRing - 1>();
            }
            const int n = (int)min((int64_t)(kAhead - in), min(tl, e) - t);
            if (n == kAhead && t - (W - 1) >= max(b, t0) && t + kAhead <= t1) tokens(std::true_type{}, t, n, head);
            else tokens(std::false_type{}, t, n, head + in);
            t += n;
            if (in + n == kAhead) head = (head + kAhead) % (kRing * kAhead);
        }
        copies_wait<0>();
        if (e >= 0) {  // what is left: rows up to the last of the run (complete: their sequence, or the rows, end here)
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
                if (tl == e || tl - (W - 1) + j < t1) flush(tl - (W - 1) + j, j);
        }
    }
    float *to = part + (size_t)run * (W + 1) * a.C + c0;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        Pack<float, V> o;
        if (j < W) o.set(dw[j < W ? j : 0]);
        else o.set(db);
        o.store(to + (size_t)j * a.C);
    }
}

// dw [C][W], dbias [C]: the runs' sums, added in order by kSumLanes threads per value and then over those.
constexpr int kSumLanes = 8;
__global__ void __launch_bounds__(256)
conv_sum_kernel(const float *__restrict__ part, const int64_t runs, const int C, const int W, float *__restrict__ dw,
                float *__restrict__ dbias) {
    __shared__ float red[kSumLanes][32];
    const int c = blockIdx.x * 32 + threadIdx.x % 32, lane = threadIdx.x / 32, j = blockIdx.y;
    float v = 0.f;
    if (c < C) {
#pragma unroll 4
        for (int64_t r = lane; r < runs; r += kSumLanes) v += part[((size_t)r * (W + 1) + j) * C + c];
    }
    red[lane][threadIdx.x % 32] = v;
    __syncthreads();
    if (lane || c >= C) return;
#pragma unroll
    for (int k = 1; k < kSumLanes; ++k) v += red[k][threadIdx.x];
    if (j < W) dw[(size_t)c * W + j] = v;
    else if (dbias) dbias[c] = v;
}

// A sequence without tokens passes nothing on to its initial state.
template <int W>
__global__ void __launch_bounds__(kThreads)
conv_empty_kernel(const int32_t *cu, const int64_t total, float *dstate, const int C) {
    const int s = blockIdx.y;
    const int64_t len = cu ? (int64_t)cu[s + 1] - cu[s] : total;
    if (len > 0) return;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i < (int64_t)(W - 1) * C / 4)
        reinterpret_cast<float4 *>(dstate + (size_t)s * (W - 1) * C)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}

unsigned blocks(int64_t n) { return (unsigned)((n + kThreads - 1) / kThreads); }

template <int W, typename T> cudaError_t launch_bias(const ConvArgs &a, cudaStream_t st) {
    const int nv = a.C / 8;
    if (a.total > 0) conv_bias_kernel<W, kVec, T><<<blocks((a.total + kRun - 1) / kRun * (a.C / kVec)), kThreads, 0, st>>>(a);
    if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    if (W > 1 && a.state_out) conv_last_kernel<W, T><<<blocks((int64_t)a.N * nv), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <int W, typename T> cudaError_t launch_step(const ConvArgs &a, cudaStream_t st) {
    const unsigned gx = blocks(a.C / 8);
    const unsigned gy = (unsigned)max(1, min(a.N, (int)((148 * 2 + gx - 1) / gx)));
    conv_step_kernel<W, T><<<dim3(gx, gy), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <int W, typename T, typename TG> cudaError_t launch_back(const ConvBackwardArgs &p, cudaStream_t st) {
    const ConvArgs &a = p.f;
    const int run = back_run(a.total, a.C);
    const int64_t runs = (a.total + run - 1) / run;
    float *part = static_cast<float *>(p.ws);
    if (runs > 0) conv_backward_kernel<W, kVec, T, TG><<<blocks(runs * (a.C / kVec)), kThreads, 0, st>>>(p, part, run);
    if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    conv_sum_kernel<<<dim3((a.C + 31) / 32, W + 1), 256, 0, st>>>(part, runs, a.C, W, p.dw, p.dbias);
    if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    if (W > 1 && p.dstate && (a.cu || a.total == 0))
        conv_empty_kernel<W><<<dim3(blocks((int64_t)(W - 1) * a.C / 4), a.N), kThreads, 0, st>>>(a.cu, a.total, p.dstate, a.C);
    return cudaGetLastError();
}

template <typename F> cudaError_t by_width(int W, F f) {
    switch (W) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 3: return f(std::integral_constant<int, 3>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 5: return f(std::integral_constant<int, 5>{});
    case 6: return f(std::integral_constant<int, 6>{});
    case 7: return f(std::integral_constant<int, 7>{});
    case 8: return f(std::integral_constant<int, 8>{});
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t conv_bias(const ConvArgs &a, bool bf16, cudaStream_t st) {
    return by_width(a.W, [&](auto w) {
        return bf16 ? launch_bias<w.value, __nv_bfloat16>(a, st) : launch_bias<w.value, float>(a, st);
    });
}

cudaError_t conv_step(const ConvArgs &a, bool bf16, cudaStream_t st) {
    return by_width(a.W, [&](auto w) {
        return bf16 ? launch_step<w.value, __nv_bfloat16>(a, st) : launch_step<w.value, float>(a, st);
    });
}

size_t conv_backward_workspace(int64_t total, int C, int W) {
    const int run = back_run(total, C);
    return (size_t)((total + run - 1) / run) * (W + 1) * C * sizeof(float);
}

cudaError_t conv_backward(const ConvBackwardArgs &p, bool bf16, cudaStream_t st) {
    return by_width(p.f.W, [&](auto w) {
        if (!bf16) return launch_back<w.value, float, float>(p, st);
        return p.dy_bf16 ? launch_back<w.value, __nv_bfloat16, __nv_bfloat16>(p, st)
                         : launch_back<w.value, __nv_bfloat16, float>(p, st);
    });
}

}  // namespace kda
