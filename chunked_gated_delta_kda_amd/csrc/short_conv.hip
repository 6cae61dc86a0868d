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
// W - 1 tokens and the gradients of the last W - 1 slide through registers, while the
// loads of the next eight tokens are under way.
#include "block_device.h"

namespace kda {

namespace {

constexpr int SC_WAVES = 4;
constexpr int SC_THREADS = 64 * SC_WAVES;
#ifndef SC_FWD_BATCH
#define SC_FWD_BATCH 8
#define SC_BWD_BATCH 4
#define SC_FWD_WORDS 4
#define SC_BWD_WORDS 2
#endif
template <class T>
using FwdSlice = Slice<T, SC_FWD_WORDS>;
template <class T>
using BwdSlice = Slice<T, SC_BWD_WORDS>;

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
template <class S, int W>
__device__ __forceinline__ void window_row(const ConvArgs& a, const Seq& q, int64_t row0, int t, int j, int c,
                                           float* f) {
    const int at = t - (W - 1) + j;
    if (at >= q.s) S::load(a.x, (row0 + at) * a.C + c, f);
    else if (a.h0) S::load(a.h0, ((int64_t)q.n * (W - 1) + (t - q.s + j)) * a.C + c, f);
    else {
#pragma unroll
        for (int v = 0; v < S::N; ++v) f[v] = 0.f;
    }
}

// Workgroup n of those behind the strips: dst = src (or zeros), the rows of a state, where
// sequence n has no token.
template <class T>
__device__ __forceinline__ void copy_empty(const ConvArgs& a, int64_t n, int rows, const void* src, void* dst) {
    if (!dst || n >= a.N) return;
    if (a.T > 0 && (!a.cu || clamp_tok(a.cu[n + 1], a.T) > clamp_tok(a.cu[n], a.T))) return;
    const int64_t words = (int64_t)rows * a.C / Word<T>::N;
    for (int64_t i = threadIdx.x; i < words; i += SC_THREADS)
        static_cast<uint32_t*>(dst)[n * words + i] = src ? static_cast<const uint32_t*>(src)[n * words + i] : 0;
}

// the loads of n tokens from t on (those from `end` on are of the last one before)
template <class S, int n>
__device__ __forceinline__ void fetch(const void* p, int64_t row0, int t, int end, int C, int c,
                                      typename S::raw (&r)[n]) {
#pragma unroll
    for (int i = 0; i < n; ++i) r[i] = S::load(p, (row0 + min(t + i, end - 1)) * C + c);
}

template <class T, int W>
__global__ __launch_bounds__(SC_THREADS) void short_conv_fwd_kernel(ConvArgs a) {
    typedef FwdSlice<T> S;
    constexpr int V = S::N, CB = 64 * V;
    const int blocks = (a.C + CB - 1) / CB;
    const int64_t wg = (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
    if (wg >= a.groups * blocks) return copy_empty<T>(a, wg - a.groups * blocks, W - 1, a.h0, a.h_final);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int per_row = (a.T + a.strip - 1) / a.strip;
    const int64_t strip = wg / blocks * SC_WAVES + w;
    const int b = (int)(strip / per_row);
    const int c = ((int)(wg % blocks) * 64 + (threadIdx.x & 63)) * V;
    if (b >= a.B || c >= a.C) return;
    const int t0 = (int)(strip % per_row) * a.strip, t1 = min(t0 + a.strip, a.T);
    const int64_t row0 = (int64_t)b * a.T;
    typename S::raw next[SC_FWD_BATCH];
    fetch<S>(a.x, row0, t0, t1, a.C, c, next);
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
        for (int j = 0; j < W - 1; ++j) window_row<S, W>(a, q, row0, t0, j, c, win[j]);
    }
    for (int tb = t0; tb < t1; tb += SC_FWD_BATCH) {
        typename S::raw rx[SC_FWD_BATCH];
#pragma unroll
        for (int i = 0; i < SC_FWD_BATCH; ++i) rx[i] = next[i];
        if (tb + SC_FWD_BATCH < t1) fetch<S>(a.x, row0, tb + SC_FWD_BATCH, t1, a.C, c, next);
#pragma unroll
        for (int i = 0; i < SC_FWD_BATCH; ++i) {
            const int t = tb + i;
            if (t >= t1) break;
            if (t >= q.e) q.next(a, t);
            if (t == q.s) {
#pragma unroll
                for (int j = 0; j < W - 1; ++j) window_row<S, W>(a, q, row0, t, j, c, win[j]);
            }
            float y[V];
            if (t >= q.s && t < q.e) {
                S::unpack(rx[i], win[W - 1]);
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
                        S::store(a.h_final, ((int64_t)q.n * (W - 1) + j) * a.C + c, win[j]);
                }
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) y[v] = 0.f;
            }
            S::store(a.y, (row0 + t) * a.C + c, y);
        }
    }
}

template <class T, int W>
__global__ __launch_bounds__(SC_THREADS) void short_conv_bwd_kernel(ConvArgs a) {
    typedef BwdSlice<T> S;
    constexpr int V = S::N, CB = 64 * V;
    __shared__ float red[SC_WAVES][W + 1][V][64];
    const int blocks = (a.C + CB - 1) / CB;
    const int64_t wg = (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
    const int64_t group = wg / blocks;
    if (group >= a.groups) return copy_empty<T>(a, wg - a.groups * blocks, W - 1, a.d_final, a.dh0);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int per_row = (a.T + a.strip - 1) / a.strip;
    const int64_t strip = group * SC_WAVES + w;
    const int b = (int)(strip / per_row);
    const int c = ((int)(wg % blocks) * 64 + lane) * V;
    float dw[W + 1][V];
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) dw[j][v] = 0.f;
    if (b < a.B && c < a.C) {
        const int t0 = (int)(strip % per_row) * a.strip, t1 = min(t0 + a.strip, a.T);
        const int64_t row0 = (int64_t)b * a.T;
        const int end = min(t1 + W - 1, a.T);
        typename S::raw next_x[SC_BWD_BATCH], next_y[SC_BWD_BATCH];
        fetch<S>(a.x, row0, t0, end, a.C, c, next_x);
        fetch<S>(a.dy, row0, t0, end, a.C, c, next_y);
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
                if (p >= t0 && p < t1) S::store(a.dx, (row0 + p) * a.C + c, f);
            } else if (a.dh0 && q.s >= t0 && q.s < t1) {
                S::store(a.dh0, ((int64_t)q.n * (W - 1) + (W - 1 + p - q.s)) * a.C + c, f);
            }
        };
        if (t0 > q.s && t0 < q.e) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) window_row<S, W>(a, q, row0, t0, j, c, win[j]);
        }
        for (int tb = t0; tb < end; tb += SC_BWD_BATCH) {
            typename S::raw rx[SC_BWD_BATCH], ry[SC_BWD_BATCH];
#pragma unroll
            for (int i = 0; i < SC_BWD_BATCH; ++i) {
                rx[i] = next_x[i];
                ry[i] = next_y[i];
            }
            if (tb + SC_BWD_BATCH < end) {
                fetch<S>(a.x, row0, tb + SC_BWD_BATCH, end, a.C, c, next_x);
                fetch<S>(a.dy, row0, tb + SC_BWD_BATCH, end, a.C, c, next_y);
            }
#pragma unroll
            for (int i = 0; i < SC_BWD_BATCH; ++i) {
                const int t = tb + i;
                if (t >= end) break;
                if (t >= q.e) q.next(a, t);
                if (t == q.s) {
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) window_row<S, W>(a, q, row0, t, j, c, win[j]);
                }
                if (t < q.s || t >= q.e) {
                    if (t < t1) {
                        const float zero[V] = {};
                        S::store(a.dx, (row0 + t) * a.C + c, zero);
                    }
                    continue;
                }
                float dz[V];
                S::unpack(rx[i], win[W - 1]);
                S::unpack(ry[i], dz);
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
                            S::load(a.d_final, ((int64_t)q.n * (W - 1) + (W - 1 - k)) * a.C + c, df);
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

// a workgroup for 32 channels of a tap's (or the bias's) gradient
template <int W>
__global__ __launch_bounds__(256) void short_conv_sum_kernel(ConvArgs a) {
    const int j = blockIdx.x % (W + 1), c = blockIdx.x / (W + 1) * 32 + threadIdx.x % 32;
    if (j == W && !a.dbias) return;
    const double s =
        sum_columns(a.part + (int64_t)j * a.C + min(c, a.C - 1), a.groups, (int64_t)(W + 1) * a.C);
    if (threadIdx.x < 32 && c < a.C) (j < W ? a.dweight + (int64_t)c * W + j : a.dbias + c)[0] = (float)s;
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

template <class S>
int64_t channel_blocks(int32_t C) {
    return (C + 64 * S::N - 1) / (64 * S::N);
}

// Tokens of a strip: 32, or 16 where that leaves fewer than eight waves to a CU.
#ifndef SC_LONG
#define SC_LONG 32
#define SC_SHORT 16
#endif
int strip_of(int32_t B, int32_t T, int64_t blocks) {
    return (int64_t)B * ((T + SC_LONG - 1) / SC_LONG) * blocks < 8 * 256 ? SC_SHORT : SC_LONG;
}

int64_t groups_of(int32_t B, int32_t T, int strip) {
    const int64_t strips = (int64_t)B * ((T + strip - 1) / strip);
    return (strips + SC_WAVES - 1) / SC_WAVES;
}

// strips, and the sequences that may be empty behind them
template <class S>
dim3 grid_of(ConvArgs& a, const void* state) {
    const int64_t blocks = channel_blocks<S>(a.C);
    a.strip = strip_of(a.B, a.T, blocks);
    a.groups = groups_of(a.B, a.T, a.strip);
    return wide_grid(a.groups * blocks + (state && (a.cu || a.T == 0) ? a.N : 0), SC_THREADS);
}

}  // namespace

int64_t short_conv_groups(int32_t B, int32_t T, int32_t C, bool fp32) {
    return groups_of(
        B, T, strip_of(B, T, fp32 ? channel_blocks<BwdSlice<float>>(C) : channel_blocks<BwdSlice<uint16_t>>(C)));
}

void launch_short_conv_fwd(const ConvArgs& args, int W, bool fp32, hipStream_t stream) {
    ConvArgs a = args;
    if (a.T == 0 && !a.h_final) return;
    by_taps(W, fp32, [&](auto t, auto w) {
        using T = decltype(t);
        const dim3 grid = grid_of<FwdSlice<T>>(a, a.h_final);
        hipLaunchKernelGGL((short_conv_fwd_kernel<T, decltype(w)::value>), grid, dim3(SC_THREADS), 0, stream, a);
    });
}

void launch_short_conv_bwd(const ConvArgs& args, int W, bool fp32, hipStream_t stream) {
    ConvArgs a = args;
    by_taps(W, fp32, [&](auto t, auto w) {
        using T = decltype(t);
        constexpr int TAPS = decltype(w)::value;
        const dim3 grid = grid_of<BwdSlice<T>>(a, a.dh0);
        if (a.T > 0 || a.dh0)
            hipLaunchKernelGGL((short_conv_bwd_kernel<T, TAPS>), grid, dim3(SC_THREADS), 0, stream, a);
        hipLaunchKernelGGL(short_conv_sum_kernel<TAPS>, dim3((unsigned)((a.C + 31) / 32 * (TAPS + 1))), dim3(256), 0,
                           stream, a);
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
