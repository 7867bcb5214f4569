// kda_residual_norm.cu -- what stands between two blocks of a layer stack, in one pass over the rows:
//
//     u = RMSNorm(y) w_post,   r' = a r + s sigmoid(g) u,   x = RMSNorm(r') w_pre
//
// (the norm after a block, its gate and residual scale, the residual stream, the norm before the next
// block), and its gradients: with rs1 = 1 / rms(y), rs2 = 1 / rms(r'), and row means <.>,
//
//     d = dr' + rs2 (w_pre dx - rs2^2 r' <w_pre dx r'>),   dr = a d,          dw_pre = sum dx rs2 r'
//     dscale = sum d sigmoid(g) u,   dg = d s u sigmoid(g) (1 - sigmoid(g)),  f = d s sigmoid(g)
//     dw_post = sum f rs1 y,         dy = rs1 (w_post f - rs1^2 y <w_post f y>).
//
// Bound by memory: every row is read once and stays in registers through its two (three) row sums. A
// CTA takes a row at a time, one vector of 8 channels per thread (two above 4096 channels), and loads the
// next row before it works on the current one. The column sums of the backward stay in shared memory, each
// thread's its own, over all of its CTA's rows; one partial row per CTA goes to the workspace and
// norm_sum_kernel adds them in order.
#include "kda_layer.cuh"

namespace kda {
namespace {

constexpr int kMaxThreads = 512;

// Sums of N values over the CTA, the same in every thread. Two calls in a row use different `slot`s.
template <int N> __device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[2][kMaxThreads / 32], int slot) {
    const int warps = blockDim.x / 32, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
    if (warps == 1) return;
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) red[slot][i][warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float t = lane < warps ? red[slot][i][lane] : 0.f;
#pragma unroll
        for (int m = kMaxThreads / 64; m > 0; m >>= 1) t += __shfl_xor_sync(0xffffffffu, t, m);
        v[i] = __shfl_sync(0xffffffffu, t, 0);
    }
}

__device__ __forceinline__ void load_weights(const float *w, int c, float (&v)[8], float none) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = none;
    if (w) {
        const float4 a = *reinterpret_cast<const float4 *>(w + c), b = *reinterpret_cast<const float4 *>(w + c + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}

// One row's inputs as loaded.
template <typename T, typename R, int V> struct Row {
    Pack8<T> y[V], g[V];
    Pack8<R> r[V];
    __device__ __forceinline__ void load(const NormArgs &a, int64_t row) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (threadIdx.x + k * blockDim.x) * 8;
            y[k].zero(), g[k].zero(), r[k].zero();
            if (c >= a.D || row >= a.rows) continue;
            const size_t at = (size_t)row * a.D + c;
            y[k].load_stream(static_cast<const T *>(a.y) + at);
            if (a.gate) g[k].load_stream(static_cast<const T *>(a.gate) + at);
            if (a.r) r[k].load_stream(static_cast<const R *>(a.r) + at);
        }
    }
    __device__ __forceinline__ float squares() const {  // this thread's part of the row's sum of y^2
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            float v[8];
            y[k].get(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(v[i], v[i], s);
        }
        return s;
    }
};

template <typename T, typename R, int V, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == kMaxThreads ? 1 : 3)
norm_kernel(const NormArgs a) {
    constexpr bool kAhead = THREADS < kMaxThreads;  // (two vectors in each of 512 threads leave no registers for a row ahead)
    __shared__ float red[2][2][kMaxThreads / 32];
    const float inv = 1.f / a.D;
    Row<T, R, V> next;
    if (kAhead) next.load(a, blockIdx.x);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        if (!kAhead) next.load(a, row);
        const Row<T, R, V> in = next;
        if (kAhead) next.load(a, row + gridDim.x);
        float out[V][8], sum[1] = {0.f};
        if (a.w_post) {
            sum[0] = in.squares();
            row_sums(sum, red, 0);
        }
        const float rs1 = rsqrtf(fmaf(sum[0], inv, a.eps));
        sum[0] = 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (threadIdx.x + k * blockDim.x) * 8, cc = min(c, a.D - 8);
            float y[8], g[8], r[8], w[8], s[8];
            in.y[k].get(y);
            in.r[k].get(r);
            load_weights(a.scale, cc, s, 1.f);
            if (a.w_post) {
                load_weights(a.w_post, cc, w, 1.f);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] *= rs1 * w[i];
            }
            if (a.gate) {
                in.g[k].get(g);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] *= sigmoid_f(g[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                out[k][i] = c < a.D ? fmaf(a.res_scale, r[i], s[i] * y[i]) : 0.f;
                sum[0] = fmaf(out[k][i], out[k][i], sum[0]);
            }
            if (c < a.D) {
                Pack8<R> o;
                o.set(out[k]);
                o.store_stream(static_cast<R *>(a.r_out) + (size_t)row * a.D + c);
            }
        }
        if (!a.w_pre) {
            if (a.w_post) __syncthreads();  // the next row's sum takes the slot that this row's readers may still read
            continue;
        }
        row_sums(sum, red, 1);
        const float rs2 = rsqrtf(fmaf(sum[0], inv, a.eps));
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (threadIdx.x + k * blockDim.x) * 8;
            if (c >= a.D) continue;
            float w[8], v[8];
            load_weights(a.w_pre, c, w, 1.f);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = out[k][i] * rs2 * w[i];
            Pack8<T> o;
            o.set(v);
            o.store_stream(static_cast<T *>(a.x) + (size_t)row * a.D + c);
        }
        // (without w_post the next row's sum takes the same slot: its writers have to wait for the readers)
        if (!a.w_post) __syncthreads();
    }
}

template <typename T, typename R, int V>
__global__ void __launch_bounds__(kMaxThreads)
norm_backward_kernel(const NormBackwardArgs p, float *__restrict__ part) {
    const NormArgs &a = p.f;
    __shared__ float red[3][2][kMaxThreads / 32];
    const float inv = 1.f / a.D;
    // this thread's column sums (w_post, scale, w_pre) lie in shared memory: the registers hold its weights (V = 1)
    extern __shared__ __align__(16) char smem_raw[];
    float4 *mine = reinterpret_cast<float4 *>(smem_raw) + threadIdx.x;
    auto sum_of = [&](int j, int k, int half) -> float4 & { return mine[((j * V + k) * 2 + half) * blockDim.x]; };
    auto add = [&](int j, int k, const float (&x)[8], const float (&y)[8]) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float4 v = sum_of(j, k, half);
            v.x = fmaf(x[4 * half], y[4 * half], v.x), v.y = fmaf(x[4 * half + 1], y[4 * half + 1], v.y);
            v.z = fmaf(x[4 * half + 2], y[4 * half + 2], v.z), v.w = fmaf(x[4 * half + 3], y[4 * half + 3], v.w);
            sum_of(j, k, half) = v;
        }
    };
    float wr[V == 1 ? 3 : 1][8];
#pragma unroll
    for (int k = 0; k < 6 * V; ++k) mine[k * blockDim.x] = make_float4(0.f, 0.f, 0.f, 0.f);
    if constexpr (V == 1) {
        const int cc = min((int)threadIdx.x * 8, a.D - 8);
        load_weights(a.scale, cc, wr[0], 1.f);
        load_weights(a.w_post, cc, wr[1], 1.f);
        load_weights(a.w_pre, cc, wr[2], 0.f);
    }
    auto weights = [&](int cc, float (&s)[8], float (&w)[8], float (&q)[8]) {
        if constexpr (V == 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = wr[0][i], w[i] = wr[1][i], q[i] = wr[2][i];
        } else {
            load_weights(a.scale, cc, s, 1.f);
            load_weights(a.w_post, cc, w, 1.f);
            load_weights(a.w_pre, cc, q, 0.f);
        }
    };
    Row<T, R, V> next;
    Pack8<T> ndx[V];
    Pack8<float> ndr[V];
    auto load = [&](int64_t row) {
        next.load(a, row);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (threadIdx.x + k * blockDim.x) * 8;
            ndx[k].zero(), ndr[k].zero();
            if (c >= a.D || row >= a.rows) continue;
            const size_t at = (size_t)row * a.D + c;
            if (p.dx) ndx[k].load_stream(static_cast<const T *>(p.dx) + at);
            if (p.dr_out) ndr[k].load_stream(p.dr_out + at);
        }
    };
    float y2[1] = {0.f};
    if (V == 1) {
        load(blockIdx.x);
        if (a.w_post) {
            y2[0] = next.squares();
            row_sums(y2, red, 0);
        }
    }
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        if (V > 1) load(row);
        const Row<T, R, V> in = next;
        float d[V][8], h[V][8];  // dr', w_pre dx
#pragma unroll
        for (int k = 0; k < V; ++k) {
            ndr[k].get(d[k]);
            ndx[k].get(h[k]);
        }
        if (V == 1) load(row + gridDim.x);
        if (V > 1 && a.w_post) {
            y2[0] = in.squares();
            row_sums(y2, red, 0);
        }
        const float rs1 = rsqrtf(fmaf(y2[0], inv, a.eps));
        float two[2] = {0.f, 0.f}, out[V][8];  // sums of r'^2 and w_pre dx r'
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (threadIdx.x + k * blockDim.x) * 8, cc = min(c, a.D - 8);
            float y[8], g[8], r[8], w[8], s[8], q[8];
            in.y[k].get(y);
            in.g[k].get(g);
            in.r[k].get(r);
            weights(cc, s, w, q);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float u = y[i];
                if (a.w_post) u *= rs1 * w[i];
                if (a.gate) u *= sigmoid_f(g[i]);
                out[k][i] = c < a.D ? fmaf(a.res_scale, r[i], s[i] * u) : 0.f;
                two[0] = fmaf(out[k][i], out[k][i], two[0]);
                two[1] = fmaf(h[k][i] * q[i], out[k][i], two[1]);
            }
        }
        float rs2 = 0.f, mean = 0.f;
        if (a.w_pre) {
            row_sums(two, red, 1);
            rs2 = rsqrtf(fmaf(two[0], inv, a.eps));
            mean = two[1] * inv * rs2 * rs2;
        }
        float sum[2] = {0.f, 0.f};  // of w_post f y; of the next row's y^2 (V = 1), one exchange for both
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (threadIdx.x + k * blockDim.x) * 8, cc = min(c, a.D - 8);
            const bool on = c < a.D;
            const size_t at = (size_t)row * a.D + c;
            float y[8], g[8], w[8], s[8], q[8], o[8], e[8];
            in.y[k].get(y);
            in.g[k].get(g);
            weights(cc, s, w, q);
            if (a.w_pre) {  // without it d = dr', whatever r' holds (0 times an infinite r' would be a NaN)
#pragma unroll
                for (int i = 0; i < 8; ++i) e[i] = out[k][i] * rs2;
                add(2, k, h[k], e);
#pragma unroll
                for (int i = 0; i < 8; ++i) d[k][i] = fmaf(rs2, fmaf(-out[k][i], mean, h[k][i] * q[i]), d[k][i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = a.res_scale * d[k][i];
            Pack8<float> v;
            if (on && p.dr) {
                v.set(o);
                v.store_stream(p.dr + at);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float u = a.w_post ? y[i] * rs1 * w[i] : y[i];
                const float m = a.gate ? sigmoid_f(g[i]) : 1.f;
                e[i] = m * u;
                out[k][i] = d[k][i];
                const float ds = d[k][i] * s[i];
                o[i] = ds * u * m * (1.f - m);
                const float f = ds * m;
                h[k][i] = f;
                d[k][i] = a.w_post ? f * w[i] : f;  // w_post f
                sum[0] = fmaf(d[k][i], y[i], sum[0]);
            }
            add(1, k, out[k], e);
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = y[i] * rs1;
            add(0, k, h[k], e);
            if (on && a.gate) {
                v.set(o);
                v.store_stream(p.dgate + at);
            }
        }
        float back = 0.f;
        if (a.w_post) {
            if (V == 1) sum[1] = next.squares();
            row_sums(sum, red, 2);
            back = sum[0] * inv * rs1 * rs1;
            if (V == 1) y2[0] = sum[1];
            if (!a.w_pre) __syncthreads();  // (the next row's sums take the same slot)
        } else {
            __syncthreads();  // the next row's sum takes the slot that this row's readers may still read
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (threadIdx.x + k * blockDim.x) * 8;
            if (c >= a.D) continue;
            float y[8], o[8];
            in.y[k].get(y);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = a.w_post ? rs1 * fmaf(-y[i], back, d[k][i]) : d[k][i];
            Pack8<float> v;
            v.set(o);
            v.store_stream(p.dy + (size_t)row * a.D + c);
        }
    }
    // this CTA's column sums: [w_post | scale | w_pre]
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int c = (threadIdx.x + k * blockDim.x) * 8;
        if (c >= a.D) continue;
        float *to = part + (size_t)blockIdx.x * 3 * a.D + c;
#pragma unroll
        for (int j = 0; j < 3; ++j)
#pragma unroll
            for (int half = 0; half < 2; ++half) *reinterpret_cast<float4 *>(to + j * a.D + 4 * half) = sum_of(j, k, half);
    }
}

// Column sums: the CTAs' partial rows, added by kLanes threads per column and then over those, in order.
constexpr int kLanes = 8;
__global__ void __launch_bounds__(256)
norm_sum_kernel(const float *__restrict__ part, const int n, const int D, float *__restrict__ d0, float *__restrict__ d1,
                float *__restrict__ d2) {
    __shared__ float red[kLanes][32];
    const int c = blockIdx.x * 32 + threadIdx.x % 32, lane = threadIdx.x / 32, j = blockIdx.y;
    float *to = j == 0 ? d0 : j == 1 ? d1 : d2;
    if (!to) return;
    float v = 0.f;
    if (c < D) {
#pragma unroll 4
        for (int r = lane; r < n; r += kLanes) v += part[((size_t)r * 3 + j) * D + c];
    }
    red[lane][threadIdx.x % 32] = v;
    __syncthreads();
    if (lane || c >= D) return;
#pragma unroll
    for (int k = 1; k < kLanes; ++k) v += red[k][threadIdx.x];
    to[c] = v;
}

// Threads of a CTA, at most `most`, one vector of 8 channels each (two above that).
int threads_of(int D, int most) { return min(most, (D / 8 + 31) / 32 * 32); }
// CTAs: enough rows in flight on every SM (a row of `most` threads, or several of fewer).
int64_t ctas_of(int64_t rows, int threads, int most, int per_sm) {
    return max((int64_t)1, min(rows, (int64_t)148 * per_sm * (most / threads)));
}

// Forward: 256 threads of up to two vectors, three CTAs to an SM, up to 4096 channels (61 us for 8192 rows
// of 4096 bf16 channels with a gate, 83 % of the copy rate; 512 threads of one vector, two CTAs: 70 us). Three CTAs
// cap the registers at 80: from 2056 channels on 40 bytes a thread spill with an fp32 stream, 232 in all fp32.
template <typename T, typename R> cudaError_t launch(const NormArgs &a, cudaStream_t st) {
    if (a.rows == 0) return cudaSuccess;
    if (a.D <= 4096) {
        const int nt = threads_of(a.D, 256);
        const unsigned grid = (unsigned)ctas_of(a.rows, nt, 256, 3);
        if (a.D <= 2048) norm_kernel<T, R, 1, 256><<<grid, nt, 0, st>>>(a);
        else norm_kernel<T, R, 2, 256><<<grid, nt, 0, st>>>(a);
    } else {
        norm_kernel<T, R, 2, kMaxThreads><<<(unsigned)ctas_of(a.rows, kMaxThreads, kMaxThreads, 1), kMaxThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}

// Backward: 512 threads, one vector each up to 4096 channels, one CTA to an SM: 165 us for 8191 rows of 4096
// channels, its stream in fp32, 81 % of the copy rate. With the column sums in registers and the weights read
// again for every row 218 us (256 threads of two vectors, two CTAs: 236 us); with the sum of y^2 exchanged by
// itself, not together with the row before's last sum, 181 us. (The forward, three CTAs to an SM, loses by
// that: 63 us against 60, it waits for the next row's loads.)
unsigned back_ctas(int64_t rows, int D) {
    return (unsigned)ctas_of(rows, threads_of(D, kMaxThreads), kMaxThreads, 1);
}
template <typename T, typename R> cudaError_t launch_back(const NormBackwardArgs &p, cudaStream_t st) {
    const NormArgs &a = p.f;
    const int nt = threads_of(a.D, kMaxThreads);
    const unsigned grid = back_ctas(a.rows, a.D);
    float *part = static_cast<float *>(p.ws);
    auto kern = a.D <= 8 * kMaxThreads ? norm_backward_kernel<T, R, 1> : norm_backward_kernel<T, R, 2>;
    const int bytes = 3 * 2 * (int)sizeof(float4) * nt * (a.D <= 8 * kMaxThreads ? 1 : 2);
    if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); e != cudaSuccess) return e;
    kern<<<grid, nt, bytes, st>>>(p, part);
    if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    if (p.dw_post || p.dscale || p.dw_pre)
        norm_sum_kernel<<<dim3((a.D + 31) / 32, 3), 256, 0, st>>>(part, (int)grid, a.D, p.dw_post, p.dscale, p.dw_pre);
    return cudaGetLastError();
}

}  // namespace

cudaError_t residual_norm(const NormArgs &a, bool bf16, cudaStream_t st) {
    if (!bf16) return launch<float, float>(a, st);
    return a.res_bf16 ? launch<__nv_bfloat16, __nv_bfloat16>(a, st) : launch<__nv_bfloat16, float>(a, st);
}

size_t residual_norm_backward_workspace(int64_t rows, int D) {
    return (size_t)back_ctas(rows, D) * 3 * D * sizeof(float);
}

cudaError_t residual_norm_backward(const NormBackwardArgs &p, bool bf16, cudaStream_t st) {
    if (!bf16) return launch_back<float, float>(p, st);
    return p.f.res_bf16 ? launch_back<__nv_bfloat16, __nv_bfloat16>(p, st) : launch_back<__nv_bfloat16, float>(p, st);
}

}  // namespace kda
