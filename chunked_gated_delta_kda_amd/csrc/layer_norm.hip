// layer_norm.hip -- the norm in front of an attention block, with the skip's
// addition before it (gfx950).  Per row of D channels:
//   u = x + residual (rounded to the rows' type, and handed on),
//   n = (u - mean(u)) rho,  rho = (mean((u - mean(u))^2) + eps)^(-1/2),
//   y = n weight + bias.
// Gradients, with t = dy weight:
//   du = rho (t - mean(t) - n mean(t n)) + dsum,
//   dweight = sum over rows of dy n,  dbias = sum over rows of dy.
//
// Bound by HBM: a row is read once and stays in the registers of the lanes that
// share it, 16 bytes a lane at a time.  The squares are those of the differences
// from the mean, and what the mean's own rounding leaves in them is taken out
// (c = mean(u - mean)), so a row far from zero keeps its digits.  All arithmetic
// is fp32; each output is rounded once.  The backward kernel's workgroups walk
// over the rows and keep their lanes' channels of dweight and dbias in registers;
// a second kernel adds the workgroups' sums in a fixed order, in 64 bits.
#include "block_device.h"

namespace kda {

namespace {

constexpr int LN_THREADS = 256;  // of a workgroup whose rows are a wave's or less
constexpr int LN_GROUPS = 1024;  // most workgroups of the backward kernel

// Sums of n values over the L lanes (or threads, from 256 on) that share a row.
template <int L, int n>
__device__ __forceinline__ void row_sums(float (&v)[n]) {
#pragma unroll
    for (int m = 1; m < (L < 64 ? L : 64); m <<= 1)
#pragma unroll
        for (int i = 0; i < n; ++i) v[i] += __shfl_xor(v[i], m);
    if constexpr (L > 64) {
        constexpr int WAVES = L / 64;
        __shared__ float red[n][WAVES];
        __syncthreads();
        if (threadIdx.x % 64 == 0)
#pragma unroll
            for (int i = 0; i < n; ++i) red[i][threadIdx.x / 64] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < n; ++i) {
            v[i] = 0.f;
            for (int w = 0; w < WAVES; ++w) v[i] += red[i][w];
        }
    }
}

template <int L>
__device__ __forceinline__ float row_max(float m) {
#pragma unroll
    for (int k = 1; k < (L < 64 ? L : 64); k <<= 1) m = fmaxf(m, __shfl_xor(m, k));
    if constexpr (L > 64) {
        __shared__ float red[L / 64];
        __syncthreads();
        if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = m;
        __syncthreads();
        for (int w = 0; w < L / 64; ++w) m = fmaxf(m, red[w]);
    }
    return m;
}

// what a row is normalised by
struct Stats {
    float mean, rest, rho, scale;  // n = ((u scale - mean) - rest) rho
};

// Power of two for a row whose squares, plus eps, or whose sum leave fp32's range, though
// the norm is of the size of one: it brings the larger of the row's largest value and
// sqrt(eps) to 1 .. 2.  1 for a row of zeros without eps and for one with an infinity or
// a NaN.
__device__ __forceinline__ float row_scale(float m) {
    if (!(m > 0.f && m <= 0x1.fffffep127f)) return 1.f;
    return ldexpf(1.f, min(max(-ilogbf(m), -126), 126));
}

template <int L, int M>
__device__ __forceinline__ Stats row_stats(float (&u)[M], int count, int D, float eps) {
    Stats s;
    s.scale = 1.f;
    const float inv = 1.f / (float)D;
    for (;;) {
        float one[1] = {0.f};
#pragma unroll
        for (int i = 0; i < M; ++i) one[0] += u[i];  // (zeros behind the row's end)
        row_sums<L, 1>(one);
        s.mean = one[0] * inv;
        float two[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const float d = i < count ? u[i] - s.mean : 0.f;
            two[0] += d;
            two[1] = fmaf(d, d, two[1]);
        }
        row_sums<L, 2>(two);
        s.rest = two[0] * inv;
        float var = fmaf(-s.rest, s.rest, two[1] * inv);
        var = (var < 0.f ? 0.f : var) + eps * s.scale * s.scale;  // (a NaN stays)
        s.rho = 1.f / sqrtf(var);
        if (s.scale != 1.f || (var >= 0x1p-100f && var <= 0x1p100f)) return s;
        float m = sqrtf(eps);
#pragma unroll
        for (int i = 0; i < M; ++i) m = fmaxf(m, fabsf(u[i]));
        s.scale = row_scale(row_max<L>(m));
        if (s.scale == 1.f) return s;
#pragma unroll
        for (int i = 0; i < M; ++i) u[i] *= s.scale;
    }
}

}  // namespace

// K slices of a row in each of its L lanes
template <class T, int L, int K>
__global__ __launch_bounds__(L > LN_THREADS ? L : LN_THREADS) void layer_norm_fwd_kernel(LayerNormArgs a) {
    constexpr int V = Slice<T>::N, THREADS = L > LN_THREADS ? L : LN_THREADS, RPW = THREADS / L;
    const int l = threadIdx.x % L;
    const int64_t row = ((int64_t)blockIdx.z * gridDim.x + blockIdx.x) * RPW + threadIdx.x / L;
    if (row >= a.rows) return;  // (all lanes of a row together)
    const int64_t at = row * a.D;
    float u[K * V];
    int count = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * L + l) * V;
        if (c < a.D) {
            Slice<T>::load(a.x, at + c, u + k * V);
            if (a.res) {
                float r[V];
                Slice<T>::load(a.res, at + c, r);
#pragma unroll
                for (int v = 0; v < V; ++v) r[v] += u[k * V + v];
                Slice<T>::store(a.sum, at + c, r);
                Slice<T>::round(r, u + k * V);
            }
            count = (k + 1) * V;
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) u[k * V + v] = 0.f;
        }
    }
    const Stats s = row_stats<L, K * V>(u, count, a.D, a.eps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * L + l) * V;
        if (c < a.D) {
            float y[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float n = ((u[k * V + v] - s.mean) - s.rest) * s.rho;
                y[v] = fmaf(n, a.weight[c + v], a.bias ? a.bias[c + v] : 0.f);
            }
            Slice<T>::store(a.y, at + c, y);
        }
    }
}

template <class T, int L, int K>
__global__ __launch_bounds__(L > LN_THREADS ? L : LN_THREADS) void layer_norm_bwd_kernel(LayerNormArgs a) {
    constexpr int V = Slice<T>::N, THREADS = L > LN_THREADS ? L : LN_THREADS, RPW = THREADS / L;
    const int l = threadIdx.x % L;
    float dw[K * V], db[K * V];
#pragma unroll
    for (int i = 0; i < K * V; ++i) dw[i] = db[i] = 0.f;
    const float inv = 1.f / (float)a.D;
    for (int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / L; row < a.rows; row += (int64_t)a.groups * RPW) {
        const int64_t at = row * a.D;
        float u[K * V], dy[K * V];
        int count = 0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + l) * V;
            if (c < a.D) {
                Slice<T>::load(a.x, at + c, u + k * V);
                Slice<T>::load(a.dy, at + c, dy + k * V);
                count = (k + 1) * V;
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) u[k * V + v] = dy[k * V + v] = 0.f;
            }
        }
        const Stats s = row_stats<L, K * V>(u, count, a.D, a.eps);
        float two[2] = {0.f, 0.f};  // sums of t and t n
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + l) * V;
            if (c < a.D) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int i = k * V + v;
                    u[i] = ((u[i] - s.mean) - s.rest) * s.rho;
                    dw[i] = fmaf(dy[i], u[i], dw[i]);
                    db[i] += dy[i];
                    dy[i] *= a.weight[c + v];
                    two[0] += dy[i];
                    two[1] = fmaf(dy[i], u[i], two[1]);
                }
            }
        }
        row_sums<L, 2>(two);
        const float mt = two[0] * inv, mtn = two[1] * inv, rho = s.rho;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + l) * V;
            if (c < a.D) {
                float dx[V], ds[V];
                if (a.dsum) Slice<T>::load(a.dsum, at + c, ds);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int i = k * V + v;
                    dx[v] = rho * (dy[i] - mt - u[i] * mtn) * s.scale;
                    if (a.dsum) dx[v] += ds[v];
                }
                Slice<T>::store(a.dx, at + c, dx);
            }
        }
    }
    // the workgroup's sums: rows side by side are added through LDS
    if constexpr (RPW == 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + l) * V;
            if (c < a.D) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    a.part[((int64_t)blockIdx.x * 2) * a.D + c + v] = dw[k * V + v];
                    a.part[((int64_t)blockIdx.x * 2 + 1) * a.D + c + v] = db[k * V + v];
                }
            }
        }
    } else {
        __shared__ float red[THREADS][V + 1];
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                __syncthreads();
#pragma unroll
                for (int v = 0; v < V; ++v) red[threadIdx.x][v] = which ? db[k * V + v] : dw[k * V + v];
                __syncthreads();
                for (int i = threadIdx.x; i < L * V; i += THREADS) {
                    const int c = k * L * V + i;
                    if (c >= a.D) break;
                    float sum = 0.f;
                    for (int r = 0; r < RPW; ++r) sum += red[r * L + i / V][i % V];
                    a.part[((int64_t)blockIdx.x * 2 + which) * a.D + c] = sum;
                }
            }
        }
    }
}

// a workgroup for 8 channels of dweight or dbias
__global__ __launch_bounds__(256) void layer_norm_sum_kernel(LayerNormArgs a) {
    const int which = blockIdx.x % 2, c = blockIdx.x / 2 * 8 + threadIdx.x % 8;
    if (which && !a.dbias) return;
    const double s = sum_columns(a.part + (int64_t)which * a.D + c, a.groups, (int64_t)2 * a.D);
    if (threadIdx.x < 8) (which ? a.dbias : a.dweight)[c] = (float)s;
}

namespace {

// Lanes of a row and slices in each: the fewest lanes up to a wave, then two and four
// slices a lane, then more waves.
template <class F>
void by_row(int slices, F&& f) {
    using std::integral_constant;
    if (slices <= 8) f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
    else if (slices <= 16) f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
    else if (slices <= 32) f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
    else if (slices <= 64) f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else if (slices <= 128) f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    else if (slices <= 256) f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
    else if (slices <= 512) f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
    else if (slices <= 1024) f(integral_constant<int, 256>{}, integral_constant<int, 4>{});
    else if (slices <= 2048) f(integral_constant<int, 512>{}, integral_constant<int, 4>{});
    else f(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
}

template <class F>
void by_type_and_row(bool fp32, int32_t D, F&& f) {
    if (fp32) by_row(D / Slice<float>::N, [&](auto l, auto k) { f(float{}, l, k); });
    else by_row(D / Slice<uint16_t>::N, [&](auto l, auto k) { f(uint16_t{}, l, k); });
}

constexpr int threads_of(int L) { return L > LN_THREADS ? L : LN_THREADS; }

}  // namespace

int32_t layer_norm_groups(int64_t rows, int32_t D, bool fp32) {
    int64_t g = 1;
    by_type_and_row(fp32, D, [&](auto, auto l, auto) {
        constexpr int per = threads_of(decltype(l)::value) / decltype(l)::value;
        g = (rows + per - 1) / per;
    });
    return (int32_t)(g < 1 ? 1 : g > LN_GROUPS ? LN_GROUPS : g);
}

void launch_layer_norm_fwd(const LayerNormArgs& a, bool fp32, hipStream_t stream) {
    by_type_and_row(fp32, a.D, [&](auto t, auto l, auto k) {
        constexpr int L = decltype(l)::value, THREADS = threads_of(L), RPW = THREADS / L;
        hipLaunchKernelGGL((layer_norm_fwd_kernel<decltype(t), L, decltype(k)::value>),
                           wide_grid((a.rows + RPW - 1) / RPW, THREADS), dim3(THREADS), 0, stream, a);
    });
}

void launch_layer_norm_bwd(const LayerNormArgs& a, bool fp32, hipStream_t stream) {
    by_type_and_row(fp32, a.D, [&](auto t, auto l, auto k) {
        constexpr int L = decltype(l)::value;
        hipLaunchKernelGGL((layer_norm_bwd_kernel<decltype(t), L, decltype(k)::value>), dim3((unsigned)a.groups),
                           dim3(threads_of(L)), 0, stream, a);
    });
    hipLaunchKernelGGL(layer_norm_sum_kernel, dim3((unsigned)(a.D / 4)), dim3(256), 0, stream, a);
}

}  // namespace kda
