// short_conv.hip -- the short causal convolution in front of an attention block
// (gfx950): per channel c of a sequence,
//   z_t = bias[c] + sum_j weight[c, j] x_{t - W + 1 + j},  y_t = act(z_t),
// act none or silu; in front of a sequence stand the W - 1 rows of its state.
// Gradients, with dz_t = dy_t act'(z_t) and the state's rows as x before token 0:
//   dx_t = sum_j weight[c, j] dz_{t + W - 1 - j},  dbias = sum dz,
//   dweight[c, j] = sum dz_t x_{t - W + 1 + j}.
//
// Bound by HBM.  A wave has a strip of tokens and 16 bytes of channels a lane, so
// that a sequence's boundary is the same for all its lanes: the window of the last
// W - 1 tokens and the gradients of the last W - 1 slide through registers.
#include "block_device.h"

namespace kda {

namespace {

constexpr int SC_WAVES = 4;
constexpr int SC_THREADS = 64 * SC_WAVES;
constexpr int SC_STRIP = 32;  // tokens of a wave

__device__ __forceinline__ int clamp_tok(int v, int T) { return min(max(v, 0), T); }

// The sequence that a strip's token belongs to: tokens [s, e) of its row of the batch.
struct Seq {
    int n, s, e;
    // the last sequence that begins at or before t (an empty one at T if none does)
    __device__ __forceinline__ void find(const ConvArgs& a, int b, int t) {
        if (!a.cu) {
            n = b;
            s = 0;
            e = a.T;
            return;
        }
        int lo = 0, hi = a.N;
        while (lo < hi) {
            const int mid = lo + (hi - lo) / 2;
            if (clamp_tok(a.cu[mid], a.T) <= t) lo = mid + 1;
            else hi = mid;
        }
        set(a, lo - 1);
    }
    __device__ __forceinline__ void set(const ConvArgs& a, int i) {
        n = i;
        s = i < 0 ? -1 : i < a.N ? clamp_tok(a.cu[i], a.T) : a.T;
        e = i < 0 ? -1 : i < a.N ? max(clamp_tok(a.cu[i + 1], a.T), s) : a.T;
    }
    // the sequence that begins at or behind e
    __device__ __forceinline__ void next(const ConvArgs& a, int t) {
        if (!a.cu) return;
        while (n < a.N && e <= t) set(a, n + 1);
    }
};

// act and its slope at z
template <bool SLOPE>
__device__ __forceinline__ float act(bool silu, float z, float& slope) {
    slope = 1.f;
    if (!silu) return z;
    const BlockSigmoid g(z);
    if (SLOPE) slope = g.s * (1.f + z * g.rest);
    return z * g.s;
}

}  // namespace

// row j of the window in front of token t of sequence q: x_{t - W + 1 + j}
template <class T, int W>
__device__ __forceinline__ void window_row(const ConvArgs& a, const Seq& q, int64_t row0, int t, int j, int c,
                                           float* f) {
    const int at = t - (W - 1) + j;
    if (at >= q.s) Slice<T>::load(a.x, (row0 + at) * a.C + c, f);
    else if (a.h0) Slice<T>::load(a.h0, ((int64_t)q.n * (W - 1) + (t - q.s + j)) * a.C + c, f);
    else {
#pragma unroll
        for (int v = 0; v < Slice<T>::N; ++v) f[v] = 0.f;
    }
}

template <class T, int W>
__global__ __launch_bounds__(SC_THREADS) void short_conv_fwd_kernel(ConvArgs a) {
    constexpr int V = Slice<T>::N, CB = 64 * V;
    const int blocks = (a.C + CB - 1) / CB;
    const int64_t wg = (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int per_row = (a.T + SC_STRIP - 1) / SC_STRIP;
    const int64_t strip = wg / blocks * SC_WAVES + w;
    const int b = (int)(strip / max(per_row, 1));
    if (b >= a.B || per_row == 0) return;
    const int c = ((int)(wg % blocks) * 64 + (threadIdx.x & 63)) * V;
    if (c >= a.C) return;
    const int t0 = (int)(strip % per_row) * SC_STRIP, t1 = min(t0 + SC_STRIP, a.T);
    const int64_t row0 = (int64_t)b * a.T;
    float wt[W][V], bias[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        bias[v] = a.bias ? a.bias[c + v] : 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) wt[j][v] = a.weight[(int64_t)(c + v) * W + j];
    }
    Seq q;
    q.find(a, b, t0);
    float win[W][V];
    if (t0 > q.s && t0 < q.e) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) window_row<T, W>(a, q, row0, t0, j, c, win[j]);
    }
    for (int t = t0; t < t1; ++t) {
        if (t >= q.e) q.next(a, t);
        if (t == q.s) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) window_row<T, W>(a, q, row0, t, j, c, win[j]);
        }
        float y[V];
        if (t >= q.s && t < q.e) {
            Slice<T>::load(a.x, (row0 + t) * a.C + c, win[W - 1]);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float z = bias[v], slope;
#pragma unroll
                for (int j = 0; j < W; ++j) z = fmaf(wt[j][v], win[j][v], z);
                y[v] = act<false>(a.silu, z, slope);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) win[j][v] = win[j + 1][v];
            }
            if (a.h_final && t == q.e - 1) {
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
                    Slice<T>::store(a.h_final, ((int64_t)q.n * (W - 1) + j) * a.C + c, win[j]);
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) y[v] = 0.f;
        }
        Slice<T>::store(a.y, (row0 + t) * a.C + c, y);
    }
}

template <class T, int W>
__global__ __launch_bounds__(SC_THREADS) void short_conv_bwd_kernel(ConvArgs a) {
    constexpr int V = Slice<T>::N, CB = 64 * V;
    __shared__ float red[SC_WAVES][W + 1][V][64];
    const int blocks = (a.C + CB - 1) / CB;
    const int64_t wg = (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
    const int64_t group = wg / blocks;
    if (group >= a.groups) return;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int per_row = (a.T + SC_STRIP - 1) / SC_STRIP;
    const int64_t strip = group * SC_WAVES + w;
    const int b = (int)(strip / per_row);
    const int c = ((int)(wg % blocks) * 64 + lane) * V;
    float dw[W + 1][V];
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) dw[j][v] = 0.f;
    if (b < a.B && c < a.C) {
        const int t0 = (int)(strip % per_row) * SC_STRIP, t1 = min(t0 + SC_STRIP, a.T);
        const int64_t row0 = (int64_t)b * a.T;
        float wt[W][V], bias[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            bias[v] = a.bias ? a.bias[c + v] : 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) wt[j][v] = a.weight[(int64_t)(c + v) * W + j];
        }
        Seq q;
        q.find(a, b, t0);
        float win[W][V], acc[W][V];  // acc[k]: the gradient of x_{t - k} so far
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) acc[k][v] = 0.f;
        // the gradient of place p of the sequence: a token's, or a row of its state's
        const auto emit = [&](int p, const float* f) {
            if (p >= q.s) {
                if (p >= t0 && p < t1) Slice<T>::store(a.dx, (row0 + p) * a.C + c, f);
            } else if (a.dh0 && q.s >= t0 && q.s < t1) {
                Slice<T>::store(a.dh0, ((int64_t)q.n * (W - 1) + (W - 1 + p - q.s)) * a.C + c, f);
            }
        };
        if (t0 > q.s && t0 < q.e) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) window_row<T, W>(a, q, row0, t0, j, c, win[j]);
        }
        const int end = min(t1 + W - 1, a.T);
        for (int t = t0; t < end; ++t) {
            if (t >= q.e) q.next(a, t);
            if (t == q.s) {
#pragma unroll
                for (int j = 0; j < W - 1; ++j) window_row<T, W>(a, q, row0, t, j, c, win[j]);
            }
            if (t < q.s || t >= q.e) {
                if (t < t1) {
                    const float zero[V] = {};
                    Slice<T>::store(a.dx, (row0 + t) * a.C + c, zero);
                }
                continue;
            }
            float dz[V];
            Slice<T>::load(a.x, (row0 + t) * a.C + c, win[W - 1]);
            Slice<T>::load(a.dy, (row0 + t) * a.C + c, dz);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float z = bias[v], slope;
#pragma unroll
                for (int j = 0; j < W; ++j) z = fmaf(wt[j][v], win[j][v], z);
                act<true>(a.silu, z, slope);
                dz[v] *= slope;
                if (t < t1) {
#pragma unroll
                    for (int j = 0; j < W; ++j) dw[j][v] = fmaf(dz[v], win[j][v], dw[j][v]);
                    dw[W][v] += dz[v];
                }
#pragma unroll
                for (int k = 0; k < W; ++k) acc[k][v] = fmaf(wt[W - 1 - k][v], dz[v], acc[k][v]);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) win[j][v] = win[j + 1][v];
            }
            emit(t - (W - 1), acc[W - 1]);
#pragma unroll
            for (int v = 0; v < V; ++v) {
#pragma unroll
                for (int k = W - 1; k > 0; --k) acc[k][v] = acc[k - 1][v];
                acc[0][v] = 0.f;
            }
            if (t == q.e - 1) {
                // the last places, and what comes back through the state left behind
#pragma unroll
                for (int k = W - 1; k > 0; --k) {
                    if (a.d_final) {
                        float df[V];
                        Slice<T>::load(a.d_final, ((int64_t)q.n * (W - 1) + (W - 1 - k)) * a.C + c, df);
#pragma unroll
                        for (int v = 0; v < V; ++v) acc[k][v] += df[v];
                    }
                    emit(t + 1 - k, acc[k]);
#pragma unroll
                    for (int v = 0; v < V; ++v) acc[k][v] = 0.f;
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) red[w][j][v][lane] = dw[j][v];
    __syncthreads();
    for (int i = threadIdx.x; i < (W + 1) * CB; i += SC_THREADS) {
        const int j = i / CB, l = i % CB / V, v = i % V, ch = (int)(wg % blocks) * CB + i % CB;
        if (ch >= a.C) continue;
        float s = 0.f;
        for (int k = 0; k < SC_WAVES; ++k) s += red[k][j][v][l];
        a.part[(group * (W + 1) + j) * a.C + ch] = s;
    }
}

// a workgroup for 8 channels of a tap's (or the bias's) gradient
template <int W>
__global__ __launch_bounds__(256) void short_conv_sum_kernel(ConvArgs a) {
    const int j = blockIdx.x % (W + 1), c = blockIdx.x / (W + 1) * 8 + threadIdx.x % 8;
    if (j == W && !a.dbias) return;
    const double s = sum_columns(a.part + (int64_t)j * a.C + c, a.groups, (int64_t)(W + 1) * a.C);
    if (threadIdx.x < 8) (j < W ? a.dweight + (int64_t)c * W + j : a.dbias + c)[0] = (float)s;
}

// dst = src (or zeros) for the sequences without a token: a workgroup a sequence
__global__ __launch_bounds__(256) void short_conv_empty_kernel(const int32_t* cu, int32_t T, int32_t N, int64_t words,
                                                               const uint32_t* src, uint32_t* dst) {
    const int64_t n = (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
    if (n >= N) return;
    if (T > 0 && (!cu || clamp_tok(cu[n + 1], T) > clamp_tok(cu[n], T))) return;
    for (int64_t i = threadIdx.x; i < words; i += 256) dst[n * words + i] = src ? src[n * words + i] : 0;
}

template <class T, int W>
__global__ __launch_bounds__(256) void short_conv_decode_kernel(ConvDecodeArgs a) {
    constexpr int V = Slice<T>::N;
    const int64_t per_row = a.C / V;
    const int64_t i = ((int64_t)blockIdx.z * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
    if (i >= a.N * per_row) return;
    const int64_t n = i / per_row;
    const int c = (int)(i % per_row) * V;
    float win[W][V], y[V];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) Slice<T>::load(a.state_in, (n * (W - 1) + j) * a.C + c, win[j]);
    Slice<T>::load(a.x, n * a.C + c, win[W - 1]);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float z = a.bias ? a.bias[c + v] : 0.f, slope;
#pragma unroll
        for (int j = 0; j < W; ++j) z = fmaf(a.weight[(int64_t)(c + v) * W + j], win[j][v], z);
        y[v] = act<false>(a.silu, z, slope);
    }
    Slice<T>::store(a.y, n * a.C + c, y);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) Slice<T>::store(a.state_out, (n * (W - 1) + j) * a.C + c, win[j + 1]);
}

namespace {

template <class F>
void by_taps(int W, bool fp32, F&& f) {
    const auto with = [&](auto w) { fp32 ? f(float{}, w) : f(uint16_t{}, w); };
    switch (W) {
        case 2: return with(std::integral_constant<int, 2>{});
        case 3: return with(std::integral_constant<int, 3>{});
        default: return with(std::integral_constant<int, 4>{});
    }
}

template <class T>
int64_t channel_blocks(int32_t C) {
    return (C + 64 * Slice<T>::N - 1) / (64 * Slice<T>::N);
}

// copies of the state for sequences without a token
void launch_empty(const ConvArgs& a, int W, bool fp32, const void* src, void* dst, hipStream_t stream) {
    if (!dst || (!a.cu && a.T > 0)) return;
    const int64_t words = (int64_t)(W - 1) * a.C / (fp32 ? 1 : 2);
    hipLaunchKernelGGL(short_conv_empty_kernel, wide_grid(a.N, 256), dim3(256), 0, stream, a.cu, a.T, a.N, words,
                       static_cast<const uint32_t*>(src), static_cast<uint32_t*>(dst));
}

}  // namespace

int64_t short_conv_groups(int32_t B, int32_t T) {
    const int64_t strips = (int64_t)B * ((T + SC_STRIP - 1) / SC_STRIP);
    return (strips + SC_WAVES - 1) / SC_WAVES;
}

void launch_short_conv_fwd(const ConvArgs& a, int W, bool fp32, hipStream_t stream) {
    launch_empty(a, W, fp32, a.h0, a.h_final, stream);
    if (a.T == 0) return;
    by_taps(W, fp32, [&](auto t, auto w) {
        using T = decltype(t);
        hipLaunchKernelGGL((short_conv_fwd_kernel<T, decltype(w)::value>),
                           wide_grid(short_conv_groups(a.B, a.T) * channel_blocks<T>(a.C), SC_THREADS),
                           dim3(SC_THREADS), 0, stream, a);
    });
}

void launch_short_conv_bwd(const ConvArgs& a, int W, bool fp32, hipStream_t stream) {
    launch_empty(a, W, fp32, a.d_final, a.dh0, stream);
    by_taps(W, fp32, [&](auto t, auto w) {
        using T = decltype(t);
        constexpr int TAPS = decltype(w)::value;
        if (a.T > 0)
            hipLaunchKernelGGL((short_conv_bwd_kernel<T, TAPS>),
                               wide_grid(a.groups * channel_blocks<T>(a.C), SC_THREADS), dim3(SC_THREADS), 0, stream,
                               a);
        hipLaunchKernelGGL(short_conv_sum_kernel<TAPS>, dim3((unsigned)(a.C / 8 * (TAPS + 1))), dim3(256), 0, stream,
                           a);
    });
}

void launch_short_conv_decode(const ConvDecodeArgs& a, int W, bool fp32, hipStream_t stream) {
    by_taps(W, fp32, [&](auto t, auto w) {
        using T = decltype(t);
        const int64_t lanes = (int64_t)a.N * (a.C / Slice<T>::N);
        hipLaunchKernelGGL((short_conv_decode_kernel<T, decltype(w)::value>), wide_grid((lanes + 255) / 256, 256),
                           dim3(256), 0, stream, a);
    });
}

}  // namespace kda
