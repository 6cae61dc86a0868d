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
// over the rows and keep their lanes' channels of dweight and dbias in registers, 64
// rows at a time in fp32 (LN_CHAIN) and more of them in 64 bits in LDS; a second kernel
// adds the workgroups' sums in a fixed order, in 64 bits.
// Measured (16384 x 4096 bf16, calls of one kind): forward with a residual 101 us, 5.3 TB/s,
// gradients with the launch behind 113 us, 4.8 TB/s; one behind the other, in a trace, 93,
// 123 and 5 us.  3001 x 1000 fp32: forward 7.7 us, gradients 13.6 and their sum 4.0 (its 24
// MB are in flight for too short a time: six rows a workgroup, one after the other).
#include <algorithm>

#include "block_device.h"

namespace kda {

namespace {

constexpr int LN_THREADS = 256;  // of a workgroup whose rows are a wave's or less

// Sums of n values over the L lanes (or threads, from 256 on) that share a row.  `red`
// belongs to this one sum: another's barrier stands between two uses of it.
template <int L, int n>
__device__ __forceinline__ void row_sums(float (&v)[n], float (*red)[16]) {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = lane_sum<(L < 64 ? L : 64)>(v[i]);
    if constexpr (L > 64) {
        constexpr int WAVES = L / 64;
        if (threadIdx.x % 64 == 0) {
#pragma unroll
            for (int i = 0; i < n; ++i) red[i][threadIdx.x / 64] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < n; ++i) {
            v[i] = 0.f;
#pragma unroll
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
    __shared__ float red_one[1][16], red_two[2][16];
    Stats s;
    s.scale = 1.f;
    const float inv = 1.f / (float)D;
    for (;;) {
        float one[1] = {0.f};
#pragma unroll
        for (int i = 0; i < M; ++i) one[0] += u[i];  // (zeros behind the row's end)
        row_sums<L, 1>(one, red_one);
        s.mean = one[0] * inv;
        float two[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const float d = i < count ? u[i] - s.mean : 0.f;
            two[0] += d;
            two[1] = fmaf(d, d, two[1]);
        }
        row_sums<L, 2>(two, red_two);
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

// The weights of a lane's slices of V channels: in registers, or read again for every row
// (from L2) where a lane has more than 16 channels, or a workgroup of 1024 threads leaves it
// 128 registers.
template <int K, int V, bool KEEP>
struct Weights {
    float w[KEEP ? K * V : 1];
    const float* p;
    __device__ __forceinline__ explicit Weights(const float* q) : p(q) {}
    __device__ __forceinline__ void read(int c, float* f) const {
        typedef float four __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
        for (int v = 0; v < V; v += 4) {
            const four q = *reinterpret_cast<const four*>(p + c + v);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[v + e] = q[e];
        }
    }
    // slice k, which begins at channel c
    __device__ __forceinline__ void keep(int k, int c, bool there) {
        if constexpr (KEEP) {
            if (there && p) {
                read(c, w + k * V);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) w[k * V + v] = 0.f;
            }
        }
    }
    // (the compiler would read them ahead of the rows, and spill them)
    __device__ __forceinline__ void next_row() {
        if constexpr (!KEEP) asm volatile("" : "+s"(p));
    }
    __device__ __forceinline__ void get(int k, int c, float* f) const {
        if constexpr (KEEP) {
#pragma unroll
            for (int v = 0; v < V; ++v) f[v] = w[k * V + v];
        } else if (p) {
            read(c, f);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) f[v] = 0.f;
        }
    }
};

// K slices of a row in each of its L lanes, the workgroup's rows one after the other.  The
// next row's loads are under way while this one is summed.
template <class T, int L, int K>
__global__ __launch_bounds__(L > LN_THREADS ? L : LN_THREADS) void layer_norm_fwd_kernel(LayerNormArgs a) {
    constexpr int V = Slice<T>::N, THREADS = L > LN_THREADS ? L : LN_THREADS, RPW = THREADS / L;
    constexpr bool KEEP = K * V <= 16 && THREADS < 1024;
    const int l = threadIdx.x % L;
    Weights<K, V, KEEP> wt(a.weight), bias(a.bias);
    int count = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * L + l) * V;
        if (c < a.D) count = (k + 1) * V;
        wt.keep(k, c, c < a.D);
        bias.keep(k, c, c < a.D);
    }
    const int64_t step = (int64_t)a.groups * RPW;
    int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / L;
    u32x4 rx[K], rr[K];
    const auto fetch = [&](int64_t r) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + l) * V;
            if (c < a.D) {
                rx[k] = Slice<T>::load(a.x, r * a.D + c);
                if (a.res) rr[k] = Slice<T>::load(a.res, r * a.D + c);
            }
        }
    };
    if (row < a.rows) fetch(row);
    for (; row < a.rows; row += step) {
        const int64_t at = row * a.D;
        float u[K * V];
        wt.next_row();
        bias.next_row();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + l) * V;
            if (c < a.D) {
                Slice<T>::unpack(rx[k], u + k * V);
                if (a.res) {
                    float r[V];
                    Slice<T>::unpack(rr[k], r);
#pragma unroll
                    for (int v = 0; v < V; ++v) r[v] += u[k * V + v];
                    Slice<T>::store(a.sum, at + c, r);
                    Slice<T>::round(r, u + k * V);
                }
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) u[k * V + v] = 0.f;
            }
        }
        if (row + step < a.rows) fetch(row + step);
        const Stats s = row_stats<L, K * V>(u, count, a.D, a.eps);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + l) * V;
            if (c < a.D) {
                float y[V], q[V], d[V];
                wt.get(k, c, q);
                bias.get(k, c, d);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    y[v] = fmaf(((u[k * V + v] - s.mean) - s.rest) * s.rho, q[v], d[v]);
                Slice<T>::store(a.y, at + c, y);
            }
        }
    }
}

// Rows that a lane adds in fp32, one after the other: 64 roundings of a sum and those of
// the rows side by side (32) and of what is left in part stay below 2^-17 of the terms'
// sizes.  More rows go on in 64 bits, in LDS (LONG), where a workgroup's sums fit there
// (131072 x 4096 bf16 with the forward pass: 1609 us, 1607 in fp32 alone).  Wider rows have
// more workgroups instead, which leave more of part to write and to add (65536 x 16384 bf16:
// 3402 us, 3360).
constexpr int LN_CHAIN = 64;
constexpr bool long_in_lds(int values, int threads) { return values * threads <= 8192; }  // (128 KB)

// (In workgroups of 1024 threads the next row's loads do not fit beside the sums.)
template <class T, int L, int K, bool LONG>
__global__ __launch_bounds__(L > LN_THREADS ? L : LN_THREADS) void layer_norm_bwd_kernel(LayerNormArgs a) {
    constexpr int V = Slice<T>::N, THREADS = L > LN_THREADS ? L : LN_THREADS, RPW = THREADS / L;
    constexpr bool KEEP = K * V <= 16 && THREADS < 1024, AHEAD = THREADS < 1024;
    __shared__ float red_t[2][16];
    __shared__ double before[2][LONG ? K * V : 1][LONG ? THREADS : 1];  // (a thread's own)
    const int l = threadIdx.x % L;
    int left = LN_CHAIN;
    float dw[K * V], db[K * V];
    Weights<K, V, KEEP> wt(a.weight);
    int count = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * L + l) * V;
        if (c < a.D) count = (k + 1) * V;
        wt.keep(k, c, c < a.D);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            dw[k * V + v] = db[k * V + v] = 0.f;
            if constexpr (LONG) before[0][k * V + v][threadIdx.x] = before[1][k * V + v][threadIdx.x] = 0.0;
        }
    }
    const float inv = 1.f / (float)a.D;
    const int64_t step = (int64_t)a.groups * RPW;
    int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / L;
    u32x4 rx[K], ry[K], rs[K];
    const auto fetch = [&](int64_t r) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + l) * V;
            if (c < a.D) {
                rx[k] = Slice<T>::load(a.x, r * a.D + c);
                ry[k] = Slice<T>::load(a.dy, r * a.D + c);
                if (AHEAD && a.dsum) rs[k] = Slice<T>::load(a.dsum, r * a.D + c);
            }
        }
    };
    if (AHEAD && row < a.rows) fetch(row);
    for (; row < a.rows; row += step) {
        const int64_t at = row * a.D;
        float u[K * V];
        u32x4 gy[K], gs[K];
        if (!AHEAD) fetch(row);
        wt.next_row();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + l) * V;
            if (c < a.D) {
                Slice<T>::unpack(rx[k], u + k * V);
                gy[k] = ry[k];
                if (a.dsum) gs[k] = rs[k];
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) u[k * V + v] = 0.f;
            }
        }
        if (AHEAD && row + step < a.rows) fetch(row + step);
        const Stats s = row_stats<L, K * V>(u, count, a.D, a.eps);
        float two[2] = {0.f, 0.f};  // sums of t = dy weight and of t n
        float t[KEEP ? K * V : 1];  // (kept, too, where the weights are)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + l) * V;
            if (c < a.D) {
                float dy[V], q[V];
                Slice<T>::unpack(gy[k], dy);
                wt.get(k, c, q);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int i = k * V + v;
                    u[i] = ((u[i] - s.mean) - s.rest) * s.rho;
                    dw[i] = fmaf(dy[v], u[i], dw[i]);
                    db[i] += dy[v];
                    dy[v] *= q[v];
                    two[0] += dy[v];
                    two[1] = fmaf(dy[v], u[i], two[1]);
                    if constexpr (KEEP) t[i] = dy[v];
                }
            }
        }
        row_sums<L, 2>(two, red_t);
        const float mt = two[0] * inv, mtn = two[1] * inv, rho = s.rho;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + l) * V;
            if (c < a.D) {
                float dx[V], dy[V], q[V], d[V];
                if constexpr (!KEEP) {
                    Slice<T>::unpack(gy[k], dy);
                    wt.get(k, c, q);
                }
                if (a.dsum) {
                    if (!AHEAD) gs[k] = Slice<T>::load(a.dsum, at + c);
                    Slice<T>::unpack(gs[k], d);
                }
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int i = k * V + v;
                    if constexpr (KEEP) dx[v] = rho * (t[i] - mt - u[i] * mtn) * s.scale;
                    else dx[v] = rho * (dy[v] * q[v] - mt - u[i] * mtn) * s.scale;
                    if (a.dsum) dx[v] += d[v];
                }
                Slice<T>::store(a.dx, at + c, dx);
            }
        }
        if constexpr (LONG) {
            if (--left == 0) {
                left = LN_CHAIN;
#pragma unroll
                for (int i = 0; i < K * V; ++i) {
                    before[0][i][threadIdx.x] += dw[i];
                    before[1][i][threadIdx.x] += db[i];
                    dw[i] = db[i] = 0.f;
                }
            }
        }
    }
    if constexpr (LONG) {
#pragma unroll
        for (int i = 0; i < K * V; ++i) {
            dw[i] = (float)(before[0][i][threadIdx.x] + dw[i]);
            db[i] = (float)(before[1][i][threadIdx.x] + db[i]);
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

// a workgroup for 32 channels of dweight or dbias
__global__ __launch_bounds__(256) void layer_norm_sum_kernel(LayerNormArgs a) {
    const int which = blockIdx.x % 2, c = blockIdx.x / 2 * 32 + threadIdx.x % 32;
    if (which && !a.dbias) return;
    const double s = sum_columns(a.part + (int64_t)which * a.D + min(c, a.D - 1), a.groups, (int64_t)2 * a.D);
    if (threadIdx.x < 32 && c < a.D) (which ? a.dbias : a.dweight)[c] = (float)s;
}

namespace {

// Lanes of a row and slices in each: the fewest lanes up to a wave, then two slices a lane,
// then more waves.  (256 slices in one wave, four a lane, need no barrier but registers:
// gradients of 3001 x 1000 fp32 21.1 us, 17.5 in four waves; 16384 x 2048 bf16 73 and 66.)
template <class T, class F>
void by_row(int32_t D, F&& rows) {
    using std::integral_constant;
    const int slices = D / Slice<T>::N;
    const auto f = [&](auto l, auto k) { rows(T{}, l, k); };
    if (slices <= 8) f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
    else if (slices <= 16) f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
    else if (slices <= 32) f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
    else if (slices <= 64) f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else if (slices <= 128) f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    else if (slices <= 256) f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
    else if (slices <= 512) f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
    else if (slices <= 1024) f(integral_constant<int, 512>{}, integral_constant<int, 2>{});
    else if (slices <= 2048) f(integral_constant<int, 512>{}, integral_constant<int, 4>{});
    else if constexpr (sizeof(T) == 4) f(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
}

template <class F>
void by_type_and_row(bool fp32, int32_t D, F&& f) {
    if (fp32) by_row<float>(D, f);
    else by_row<uint16_t>(D, f);
}

constexpr int threads_of(int L) { return L > LN_THREADS ? L : LN_THREADS; }

// Workgroups: as many as are in flight at once, `waves` waves of them on each CU, for every
// width and type by what one size took.  (16384 x 4096 bf16: forward 101 us, 125 with 8 and 105 with 32 waves; gradients 114 us,
// 167 with 4 and 137 with 16, which leave twice the sums to add.)
constexpr int LN_FWD_WAVES = 16, LN_BWD_WAVES = 8;

int32_t groups_of(int64_t rows, int32_t D, bool fp32, int waves, bool backward) {
    int64_t g = 1;
    by_type_and_row(fp32, D, [&](auto t, auto l, auto k) {
        constexpr int L = decltype(l)::value, per = threads_of(L) / L;
        g = std::min<int64_t>((rows + per - 1) / per, std::max(1, waves * 64 / threads_of(L)) * 256);
        if (backward && !long_in_lds(decltype(k)::value * Slice<decltype(t)>::N, threads_of(L)))
            g = std::max(g, (rows + LN_CHAIN * per - 1) / (LN_CHAIN * per));
    });
    return (int32_t)std::max<int64_t>(g, 1);
}

}  // namespace

int32_t layer_norm_groups(int64_t rows, int32_t D, bool fp32) { return groups_of(rows, D, fp32, LN_BWD_WAVES, true); }

void launch_layer_norm_fwd(const LayerNormArgs& args, bool fp32, hipStream_t stream) {
    LayerNormArgs a = args;
    a.groups = groups_of(a.rows, a.D, fp32, LN_FWD_WAVES, false);
    by_type_and_row(fp32, a.D, [&](auto t, auto l, auto k) {
        constexpr int L = decltype(l)::value;
        hipLaunchKernelGGL((layer_norm_fwd_kernel<decltype(t), L, decltype(k)::value>), dim3((unsigned)a.groups),
                           dim3(threads_of(L)), 0, stream, a);
    });
}

void launch_layer_norm_bwd(const LayerNormArgs& a, bool fp32, hipStream_t stream) {
    by_type_and_row(fp32, a.D, [&](auto t, auto l, auto k) {
        constexpr int L = decltype(l)::value, K = decltype(k)::value, threads = threads_of(L);
        const dim3 grid((unsigned)a.groups);
        if constexpr (long_in_lds(K * Slice<decltype(t)>::N, threads)) {
            if (a.rows > (int64_t)a.groups * (threads / L) * LN_CHAIN) {
                hipLaunchKernelGGL((layer_norm_bwd_kernel<decltype(t), L, K, true>), grid, dim3(threads), 0, stream, a);
                return;
            }
        }
        hipLaunchKernelGGL((layer_norm_bwd_kernel<decltype(t), L, K, false>), grid, dim3(threads), 0, stream, a);
    });
    hipLaunchKernelGGL(layer_norm_sum_kernel, dim3((unsigned)((a.D + 31) / 32 * 2)), dim3(256), 0, stream, a);
}

}  // namespace kda
