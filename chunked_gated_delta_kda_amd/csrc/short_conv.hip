// short_conv.hip -- the short causal convolution in front of an attention block
// (gfx950): per channel c of a sequence,
//   z_t = bias[c] + sum_j weight[c, j] x_{t - W + 1 + j},  y_t = act(z_t),
// act none or silu; in front of a sequence stand the W - 1 rows of its state.
// Gradients, with dz_t = dy_t act'(z_t) and the state's rows as x before token 0:
//   dx_t = sum_j weight[c, j] dz_{t + W - 1 - j},  dbias = sum dz,
//   dweight[c, j] = sum dz_t x_{t - W + 1 + j}.
//
// Bound by HBM.  A wave has a strip of tokens and two channels a lane, so that a
// sequence's boundary is the same for all its lanes: the last W - 1 tokens and their
// gradients slide through registers, while the loads of the next four tokens are
// under way.  (Four and eight channels a lane leave too few waves, and in the
// gradients too few registers: with the gates of the time, 4096 tokens of 4096 bf16
// channels took 34 us with two, 42 with four, 56 with eight.)  The arithmetic is not far
// behind: a gradient is some 40 instructions a channel, which the VALU is active for in 84%
// of the cycles.
// Measured (bf16, 4 taps, silu): 35862 packed tokens of 12288 channels 334 us, 5.3 TB/s;
// 2 x 2048 tokens of 4096 channels 14.3 us, 4.7 TB/s, their gradients 25.8 us with the sums
// over strips, 3.9 TB/s.
#include "block_device.h"

namespace kda {

namespace {

constexpr int SC_WAVES = 4;
constexpr int SC_THREADS = 64 * SC_WAVES;
constexpr int SC_BATCH = 4;  // tokens whose loads are under way together; divides a strip

template <class T>
using Pair = Slice<T, sizeof(T) / 2>;  // two channels

__device__ __forceinline__ int clamp_tok(int v, int T) { return min(max(v, 0), T); }

// The sequence that a strip's token belongs to: tokens [s, e) of its row of the batch.
struct Seq {
    int n, s, e;
    // The last sequence that begins at or before t (-1: none does), 64 candidates at a time:
    // all lanes of the wave have to be there.
    __device__ __forceinline__ void find(const ConvArgs& a, int b, int t) {
        if (!a.cu) {
            n = b;
            s = 0;
            e = a.T;
            return;
        }
        search(a, t, 6);
    }
    // (2^w candidates: as many of the wave's lanes, from the first, are there; w > 0)
    __device__ __forceinline__ void search(const ConvArgs& a, int t, int w) {
        const int lane = threadIdx.x & 63;
        uint32_t lo = 0, count = a.N, step;  // (N + 63 may pass 31 bits)
        do {
            step = (count + (1u << w) - 1) >> w;
            const uint32_t i = lane * step;
            const int before =
                __popcll(__ballot(i < count && clamp_tok(a.cu[min(lo + i, (uint32_t)a.N)], a.T) <= t));
            if (before == 0) return set(a, -1);
            lo += (before - 1) * step;
            count = min(step, count - (before - 1) * step);
        } while (step > 1);
        set(a, (int)lo);
    }
    __device__ __forceinline__ void set(const ConvArgs& a, int i) {
        n = i;
        s = i < 0 ? -1 : i < a.N ? clamp_tok(a.cu[i], a.T) : a.T;
        e = i < 0 ? -1 : i < a.N ? max(clamp_tok(a.cu[i + 1], a.T), s) : a.T;
    }
    // The next sequence that has a token, t or one behind it.  Where the one behind this has
    // none it is searched for: offsets that repeat by the thousand (a batch padded to a fixed
    // number of sequences) are passed in a few steps, not one by one.
    __device__ __forceinline__ void next(const ConvArgs& a, int t) {
        if (!a.cu || n >= a.N) return;
        set(a, n + 1);
        if (n >= a.N || e > t) return;
        search(a, t, 31 - __builtin_clz(__popcll(__ballot(true))));  // (channels come in eights)
        if (e <= t) set(a, n + 1);
    }
};

// act and its slope
template <bool SILU>
__device__ __forceinline__ float act(float z) {
    return SILU ? z * BlockSigmoid(z).s : z;
}
template <bool SILU>
__device__ __forceinline__ float slope(float z) {
    if (!SILU) return 1.f;
    const BlockSigmoid g(z);
    return fmaf(z, g.side, g.s);
}

}  // namespace

// The block of channels of workgroup wg, of those of a group of strips.  Workgroups go to
// the XCDs one after the other: where the number of blocks is a multiple of 8, the eight
// change places from one group to the next, or an XCD would read the same columns of every
// row, which share few of its L2's channels (35862 packed tokens of 12288 channels 334 us,
// 345 without; 32768 of 4096 100 and 105).
__device__ __forceinline__ uint32_t column_of(uint32_t wg, uint32_t blocks) {
    const uint32_t c = wg % blocks;
    return blocks % 8 ? c : (c & ~7u) + ((c + wg / blocks) & 7);
}

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

// Four tokens that are all inside of one sequence, not its last among them, are straight
// code over what was loaded ahead; the others go one by one, with loads of their own.
template <class T, int W, bool SILU>
__global__ __launch_bounds__(SC_THREADS) void short_conv_fwd_kernel(ConvArgs a) {
    typedef Pair<T> S;
    constexpr int V = S::N, CB = 64 * V;
    const uint32_t blocks = (a.C + CB - 1) / CB;
    const uint32_t wg = blockIdx.z * gridDim.x + blockIdx.x;
    if (wg >= a.groups * blocks) return copy_empty<T>(a, wg - a.groups * blocks, W - 1, a.h0, a.h_final);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t per_row = (a.T + a.strip - 1) / a.strip, strip = wg / blocks * SC_WAVES + w;
    const int b = strip / max(per_row, 1u);
    const int c = ((int)column_of(wg, blocks) * 64 + (threadIdx.x & 63)) * V;
    if (b >= a.B) return;
    const int t0 = strip % per_row * a.strip, t1 = min(t0 + a.strip, a.T);
    Seq q;
    q.find(a, b, t0);
    if (c >= a.C) return;
    const int64_t row0 = (int64_t)b * a.T;
    typename S::raw next[SC_BATCH];
    fetch<S>(a.x, row0, t0, t1, a.C, c, next);
    float wt[W][V], bias[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        bias[v] = a.bias ? a.bias[c + v] : 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) wt[j][v] = a.weight[(int64_t)(c + v) * W + j];
    }
    float win[W - 1][V];  // x of the W - 1 tokens before
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) win[j][v] = 0.f;
    if (t0 > q.s && t0 < q.e) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) window_row<S, W>(a, q, row0, t0, j, c, win[j]);
    }
    for (int tb = t0; tb < t1; tb += SC_BATCH) {
        typename S::raw rx[SC_BATCH];
#pragma unroll
        for (int i = 0; i < SC_BATCH; ++i) rx[i] = next[i];
        if (tb + SC_BATCH < t1) fetch<S>(a.x, row0, tb + SC_BATCH, t1, a.C, c, next);
        if (tb > q.s && tb + SC_BATCH < q.e && tb + SC_BATCH <= t1) {
            float x[SC_BATCH + W - 1][V];
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) x[j][v] = win[j][v];
#pragma unroll
            for (int i = 0; i < SC_BATCH; ++i) S::unpack(rx[i], x[W - 1 + i]);
#pragma unroll
            for (int i = 0; i < SC_BATCH; ++i) {
                float y[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float z = bias[v];
#pragma unroll
                    for (int j = 0; j < W; ++j) z = fmaf(wt[j][v], x[i + j][v], z);
                    y[v] = act<SILU>(z);
                }
                S::store(a.y, (row0 + tb + i) * a.C + c, y);
            }
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) win[j][v] = x[SC_BATCH + j][v];
            continue;
        }
        for (int t = tb; t < min(tb + SC_BATCH, t1); ++t) {
            if (t >= q.e) q.next(a, t);
            if (t == q.s) {
#pragma unroll
                for (int j = 0; j < W - 1; ++j) window_row<S, W>(a, q, row0, t, j, c, win[j]);
            }
            float y[V];
            if (t >= q.s && t < q.e) {
                float x[V];
                S::load(a.x, (row0 + t) * a.C + c, x);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float z = bias[v];
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) z = fmaf(wt[j][v], win[j][v], z);
                    y[v] = act<SILU>(fmaf(wt[W - 1][v], x[v], z));
#pragma unroll
                    for (int j = 0; j < W - 2; ++j) win[j][v] = win[j + 1][v];
                    win[W - 2][v] = x[v];
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

template <class T, int W, bool SILU>
__global__ __launch_bounds__(SC_THREADS, 4) void short_conv_bwd_kernel(ConvArgs a) {
    typedef Pair<T> S;
    constexpr int V = S::N, CB = 64 * V;
    __shared__ float red[SC_WAVES][W + 1][V][64];
    const uint32_t blocks = (a.C + CB - 1) / CB;
    const uint32_t wg = blockIdx.z * gridDim.x + blockIdx.x, group = wg / blocks;
    if (group >= a.groups) return copy_empty<T>(a, wg - a.groups * blocks, W - 1, a.d_final, a.dh0);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const uint32_t per_row = (a.T + a.strip - 1) / a.strip, strip = group * SC_WAVES + w;
    const int b = strip / max(per_row, 1u);
    const int c = ((int)column_of(wg, blocks) * 64 + lane) * V;
    float dw[W + 1][V];
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) dw[j][v] = 0.f;
    const int t0 = strip % max(per_row, 1u) * a.strip, t1 = min(t0 + a.strip, a.T);
    Seq q;
    if (b < a.B) q.find(a, b, t0);
    if (b < a.B && c < a.C) {
        const int64_t row0 = (int64_t)b * a.T;
        const int end = min(t1 + W - 1, a.T);
        typename S::raw next_x[SC_BATCH], next_y[SC_BATCH];
        fetch<S>(a.x, row0, t0, end, a.C, c, next_x);
        fetch<S>(a.dy, row0, t0, end, a.C, c, next_y);
        float wt[W][V], bias[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            bias[v] = a.bias ? a.bias[c + v] : 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) wt[j][v] = a.weight[(int64_t)(c + v) * W + j];
        }
        // of the W - 1 tokens before: x, and the gradient of x so far
        float win[W - 1][V], pend[W - 1][V];
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) win[j][v] = pend[j][v] = 0.f;
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
        for (int tb = t0; tb < end; tb += SC_BATCH) {
            typename S::raw rx[SC_BATCH], ry[SC_BATCH];
#pragma unroll
            for (int i = 0; i < SC_BATCH; ++i) {
                rx[i] = next_x[i];
                ry[i] = next_y[i];
            }
            if (tb + SC_BATCH < end) {
                fetch<S>(a.x, row0, tb + SC_BATCH, end, a.C, c, next_x);
                fetch<S>(a.dy, row0, tb + SC_BATCH, end, a.C, c, next_y);
            }
            // (a batch behind the strip may have tokens from `end` on: their part is of
            // places that are not this strip's)
            if (tb >= q.s + W && tb + SC_BATCH < q.e && (tb >= t1 || tb + SC_BATCH <= t1)) {
                float x[SC_BATCH + W - 1][V], dx[SC_BATCH + W - 1][V], dz[SC_BATCH][V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) {
                        x[j][v] = win[j][v];
                        dx[j][v] = pend[j][v];
                    }
#pragma unroll
                    for (int j = W - 1; j < SC_BATCH + W - 1; ++j) dx[j][v] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < SC_BATCH; ++i) {
                    S::unpack(rx[i], x[W - 1 + i]);
                    S::unpack(ry[i], dz[i]);
                }
#pragma unroll
                for (int i = 0; i < SC_BATCH; ++i) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        float z = bias[v];
#pragma unroll
                        for (int j = 0; j < W; ++j) z = fmaf(wt[j][v], x[i + j][v], z);
                        dz[i][v] *= slope<SILU>(z);
#pragma unroll
                        for (int j = 0; j < W; ++j) dx[i + j][v] = fmaf(wt[j][v], dz[i][v], dx[i + j][v]);
                    }
                }
#pragma unroll
                for (int i = 0; i < SC_BATCH; ++i) {
                    const int p = tb + i - (W - 1);
                    if (p >= t0 && p < t1) S::store(a.dx, (row0 + p) * a.C + c, dx[i]);
                }
                if (tb < t1) {
#pragma unroll
                    for (int i = 0; i < SC_BATCH; ++i)
#pragma unroll
                        for (int v = 0; v < V; ++v) {
#pragma unroll
                            for (int j = 0; j < W; ++j) dw[j][v] = fmaf(dz[i][v], x[i + j][v], dw[j][v]);
                            dw[W][v] += dz[i][v];
                        }
                }
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        win[j][v] = x[SC_BATCH + j][v];
                        pend[j][v] = dx[SC_BATCH + j][v];
                    }
                continue;
            }
            for (int t = tb; t < min(tb + SC_BATCH, end); ++t) {
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
                float x[V], dz[V], done[V];
                S::load(a.x, (row0 + t) * a.C + c, x);
                S::load(a.dy, (row0 + t) * a.C + c, dz);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float z = bias[v];
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) z = fmaf(wt[j][v], win[j][v], z);
                    dz[v] *= slope<SILU>(fmaf(wt[W - 1][v], x[v], z));
                    if (t < t1) {
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) dw[j][v] = fmaf(dz[v], win[j][v], dw[j][v]);
                        dw[W - 1][v] = fmaf(dz[v], x[v], dw[W - 1][v]);
                        dw[W][v] += dz[v];
                    }
                    done[v] = fmaf(wt[0][v], dz[v], pend[0][v]);
#pragma unroll
                    for (int j = 0; j < W - 2; ++j) {
                        win[j][v] = win[j + 1][v];
                        pend[j][v] = fmaf(wt[j + 1][v], dz[v], pend[j + 1][v]);
                    }
                    win[W - 2][v] = x[v];
                    pend[W - 2][v] = wt[W - 1][v] * dz[v];
                }
                emit(t - (W - 1), done);
                if (t == q.e - 1) {
                    // the last places, and what comes back through the state left behind
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) {
                        if (a.d_final) {
                            float df[V];
                            S::load(a.d_final, ((int64_t)q.n * (W - 1) + j) * a.C + c, df);
#pragma unroll
                            for (int v = 0; v < V; ++v) pend[j][v] += df[v];
                        }
                        emit(t + 1 - (W - 1) + j, pend[j]);
#pragma unroll
                        for (int v = 0; v < V; ++v) pend[j][v] = 0.f;
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
        const int j = i / CB, l = i % CB / V, v = i % V, ch = (int)column_of(wg, blocks) * CB + i % CB;
        if (ch >= a.C) continue;
        float s = 0.f;
        for (int k = 0; k < SC_WAVES; ++k) s += red[k][j][v][l];
        a.part[((int64_t)group * (W + 1) + j) * a.C + ch] = s;
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

// One token: two channels of SC_SEQS sequences a lane, so that the taps are read once for
// them (64 sequences of 12288 channels: 4.3 us, 6.6 with eight channels of one).
constexpr int SC_SEQS = 4;

template <class T, int W, bool SILU>
__global__ __launch_bounds__(256) void short_conv_decode_kernel(ConvDecodeArgs a) {
    typedef Pair<T> S;
    constexpr int V = S::N;
    const uint32_t per_row = a.C / V;
    const int64_t i = ((int64_t)blockIdx.z * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
    const int64_t n0 = i / per_row * SC_SEQS;
    if (n0 >= a.N) return;
    const int c = (int)(i % per_row) * V;
    typename S::raw row[SC_SEQS][W];
#pragma unroll
    for (int k = 0; k < SC_SEQS; ++k) {
        const int64_t n = min(n0 + k, (int64_t)a.N - 1);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) row[k][j] = S::load(a.state_in, (n * (W - 1) + j) * a.C + c);
        row[k][W - 1] = S::load(a.x, n * a.C + c);
    }
    float wt[V][W], bias[V] = {};
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < W; ++j) wt[v][j] = a.weight[(int64_t)(c + v) * W + j];
    if (a.bias) {
#pragma unroll
        for (int v = 0; v < V; ++v) bias[v] = a.bias[c + v];
    }
#pragma unroll
    for (int k = 0; k < SC_SEQS; ++k) {
        const int64_t n = n0 + k;
        if (n >= a.N) break;
        float x[W][V], y[V];
#pragma unroll
        for (int j = 0; j < W; ++j) S::unpack(row[k][j], x[j]);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float z = bias[v];
#pragma unroll
            for (int j = 0; j < W; ++j) z = fmaf(wt[v][j], x[j][v], z);
            y[v] = act<SILU>(z);
        }
        S::store(a.y, n * a.C + c, y);
        typename S::raw* out = reinterpret_cast<typename S::raw*>(static_cast<T*>(a.state_out) + n * (W - 1) * a.C + c);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) out[(int64_t)j * per_row] = row[k][j + 1];
    }
}

namespace {

template <class F>
void by_taps(int W, bool fp32, bool silu, F&& f) {
    const auto with = [&](auto w) {
        const auto type = [&](auto s) { fp32 ? f(float{}, w, s) : f(uint16_t{}, w, s); };
        silu ? type(std::true_type{}) : type(std::false_type{});
    };
    switch (W) {
        case 2: return with(std::integral_constant<int, 2>{});
        case 3: return with(std::integral_constant<int, 3>{});
        default: return with(std::integral_constant<int, 4>{});
    }
}

// Tokens of a strip, 16 or 32.  The gradients read W - 1 tokens more than a strip has, and
// leave a row of sums for four strips; bf16 calls that fill the GPU with strips of 32 gain
// by them (32768 tokens of 4096 channels: 173 us, 194 with 16; 2048 tokens: 22.6 and 21.5),
// fp32 calls do not (338 and 309), nor does the forward pass (109 and 106).
int strip_of(int32_t B, int32_t T, int64_t blocks, bool fp32, bool backward) {
    return backward && !fp32 && (int64_t)B * ((T + 31) / 32) * blocks >= 16 * 256 ? 32 : 16;
}

int64_t channel_blocks(int32_t C) { return (C + 127) / 128; }

int64_t groups_of(int32_t B, int32_t T, int strip) {
    const int64_t strips = (int64_t)B * (((int64_t)T + strip - 1) / strip);
    return (strips + SC_WAVES - 1) / SC_WAVES;
}

// strips, and the sequences that may be empty behind them
dim3 grid_of(ConvArgs& a, bool fp32, bool backward, const void* state) {
    const int64_t blocks = channel_blocks(a.C);
    a.strip = strip_of(a.B, a.T, blocks, fp32, backward);
    a.groups = (uint32_t)groups_of(a.B, a.T, a.strip);
    return wide_grid(a.groups * blocks + (state && (a.cu || a.T == 0) ? a.N : 0), SC_THREADS);
}

}  // namespace

int64_t short_conv_groups(int32_t B, int32_t T, int32_t C, bool fp32) {
    return groups_of(B, T, strip_of(B, T, channel_blocks(C), fp32, true));
}

int64_t short_conv_workgroups(int32_t B, int32_t T, int32_t C, int32_t N) {
    return groups_of(B, T, 16) * channel_blocks(C) + N;
}

void launch_short_conv_fwd(const ConvArgs& args, int W, bool fp32, hipStream_t stream) {
    ConvArgs a = args;
    if (a.T == 0 && !a.h_final) return;
    const dim3 grid = grid_of(a, fp32, false, a.h_final);
    by_taps(W, fp32, a.silu, [&](auto t, auto w, auto silu) {
        hipLaunchKernelGGL((short_conv_fwd_kernel<decltype(t), decltype(w)::value, decltype(silu)::value>), grid,
                           dim3(SC_THREADS), 0, stream, a);
    });
}

void launch_short_conv_bwd(const ConvArgs& args, int W, bool fp32, hipStream_t stream) {
    ConvArgs a = args;
    const dim3 grid = grid_of(a, fp32, true, a.dh0);
    by_taps(W, fp32, a.silu, [&](auto t, auto w, auto silu) {
        constexpr int TAPS = decltype(w)::value;
        if (a.T > 0 || a.dh0)
            hipLaunchKernelGGL((short_conv_bwd_kernel<decltype(t), TAPS, decltype(silu)::value>), grid,
                               dim3(SC_THREADS), 0, stream, a);
        hipLaunchKernelGGL(short_conv_sum_kernel<TAPS>, dim3((unsigned)((a.C + 31) / 32 * (TAPS + 1))), dim3(256), 0,
                           stream, a);
    });
}

void launch_short_conv_decode(const ConvDecodeArgs& a, int W, bool fp32, hipStream_t stream) {
    const int64_t lanes = ((int64_t)a.N + SC_SEQS - 1) / SC_SEQS * (a.C / 2);
    by_taps(W, fp32, a.silu, [&](auto t, auto w, auto silu) {
        hipLaunchKernelGGL((short_conv_decode_kernel<decltype(t), decltype(w)::value, decltype(silu)::value>),
                           wide_grid((lanes + 255) / 256, 256), dim3(256), 0, stream, a);
    });
}

}  // namespace kda
