// gated_norm.hip -- the norm behind an attention block, with the block's skip
// before it and its gate after it (gfx950).  Per row of D channels, head h:
//   u = x + res_scale[h] res,  n = u (mean(u^2) + eps)^(-1/2),
//   y = n weight act(gate),    act = sigmoid or silu.
// Gradients, with p = dy weight act(gate) and rho = (mean(u^2) + eps)^(-1/2):
//   du = rho (p - n mean(p n)),  dx = du,  dres = res_scale du,
//   dres_scale[h] = sum over tokens and channels of du res,
//   dgate = dy n weight act'(gate),  dweight = sum over rows of dy n act(gate).
//
// Bound by HBM: every row is read and written once.  A row is held by the
// smallest power of two of lanes that covers it with eight channels each (16
// lanes at D = 128), so its sums are a few lane exchanges.  All arithmetic is
// fp32; each output is rounded once.  The backward kernel's workgroups walk
// over the rows and keep their lanes' channels of dweight in registers; each
// leaves one row of sums, and a second kernel adds them in a fixed order, in
// 64 bits, so gradients are the same from call to call.
//
// 4096 tokens, 32 heads of 128, a gate: forward 23 us (101 MB, 4.4 TB/s), backward
// 37 us (168 MB, 4.6 TB/s; 36 without row_scale) and 4.7 us for the sums.  2048
// workgroups instead of 1024 make the backward kernel 9 us slower, a row's loads ahead of
// the row before change nothing.
#include "kda_common.h"
#include "la_launch.h"

namespace kda {

namespace {

constexpr int GN_THREADS = 256;
constexpr int GN_GROUPS = 1024;  // most workgroups of the backward kernel

__device__ __forceinline__ void to_float8(bf16x8 v, float* f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (float)v[e];
}
__device__ __forceinline__ void load8(const uint16_t* p, float* f) {
    to_float8(*reinterpret_cast<const bf16x8*>(p), f);
}
__device__ __forceinline__ void store8(uint16_t* p, const float* f) {
    bf16x8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (bf16)f[e];
    *reinterpret_cast<bf16x8*>(p) = v;
}

// sum over the L lanes that hold a row
template <int L>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int m = 1; m < L; m <<= 1) v += __shfl_xor(v, m);
    return v;
}

// Power of two that a row is multiplied by where the mean of its squares, plus eps, is
// not within 2^-100 .. 2^100: there the squares (or rho^2 in the gradients) leave fp32's
// range, though the norm is of the size of one.  It brings the larger of the row's
// largest value and sqrt(eps) to 1 .. 2.  1 for the other rows, for a row of zeros
// without eps and for one with an infinity or a NaN.
template <int L>
__device__ __forceinline__ float row_scale(const float (&u)[8], float mean, float eps) {
    if (mean >= 0x1p-100f && mean <= 0x1p100f) return 1.f;
    float m = sqrtf(eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(u[e]));
#pragma unroll
    for (int k = 1; k < L; k <<= 1) m = fmaxf(m, __shfl_xor(m, k));
    if (!(m > 0.f && m <= 0x1.fffffep127f)) return 1.f;
    return ldexpf(1.f, min(max(-ilogbf(m), -126), 126));
}

// A gate's sigmoid 1 / (1 + e^-z) as e^min(z, 0) / (1 + e^-|z|): to a few ulps where it
// is normal, and subnormal below z = -87 (e^-z would be infinite there, and the gate
// closed too early).  `rest` is 1 - s, which a difference would round away where the gate
// is open; the slope is their product.
struct Sigmoid {
    float s, rest;
    __device__ __forceinline__ explicit Sigmoid(float z) {
        const float e = expf(-fabsf(z)), r = 1.f / (1.f + e);
        s = z < 0.f ? e * r : r;
        rest = z < 0.f ? r : e * r;
    }
};

}  // namespace

template <int L>
__global__ __launch_bounds__(GN_THREADS) void gated_norm_fwd_kernel(GatedNormArgs a) {
    constexpr int RPW = GN_THREADS / L;  // rows per workgroup
    const int l = threadIdx.x % L, c = 8 * l;
    const int64_t row = ((int64_t)blockIdx.z * gridDim.x + blockIdx.x) * RPW + threadIdx.x / L;
    if (row >= a.rows) return;  // (all lanes of a row together)
    const bool in = c < a.D;
    const int64_t at = row * a.D + c;
    float u[8] = {}, z[8], w[8];
    if (in) {
        load8(a.x + at, u);
        if (a.res) {
            float res[8];
            load8(a.res + at, res);
            const float rs = a.res_scale[row % a.H];
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = fmaf(rs, res[e], u[e]);
        }
        if (a.gate) load8(a.gate + at, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = a.weight[c + e];
    }
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(u[e], u[e], ss);
    float mean = row_sum<L>(ss) / (float)a.D + a.eps;
    const float scale = row_scale<L>(u, mean, a.eps);
    if (scale != 1.f) {
        ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            u[e] *= scale;
            ss = fmaf(u[e], u[e], ss);
        }
        mean = row_sum<L>(ss) / (float)a.D + a.eps * scale * scale;
    }
    const float rho = 1.f / sqrtf(mean);
    if (!in) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        u[e] *= rho * w[e];
        if (a.gate) {
            const float s = Sigmoid(z[e]).s;
            u[e] *= a.silu ? z[e] * s : s;
        }
    }
    store8(a.y + at, u);
}

template <int L>
__global__ __launch_bounds__(GN_THREADS) void gated_norm_bwd_kernel(GatedNormArgs a) {
    constexpr int RPW = GN_THREADS / L;
    __shared__ float red[GN_THREADS][9];
    const int l = threadIdx.x % L, c = 8 * l;
    const bool in = c < a.D;
    float w[8] = {}, dw[8] = {};
    if (in) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = a.weight[c + e];
    }
    const float inv_d = 1.f / (float)a.D;
    for (int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / L; row < a.rows; row += (int64_t)a.groups * RPW) {
        const int64_t at = row * a.D + c;
        float u[8] = {}, z[8] = {}, dy[8] = {}, res[8] = {};
        float rs = 0.f;
        if (in) {
            load8(a.x + at, u);
            load8(a.dy + at, dy);
            if (a.gate) load8(a.gate + at, z);
            if (a.res) {
                load8(a.res + at, res);
                rs = a.res_scale[row % a.H];
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = fmaf(rs, res[e], u[e]);
            }
        }
        float ss = 0.f, pu = 0.f;
        float act[8], slope[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            act[e] = 1.f;
            slope[e] = 0.f;
            if (a.gate) {
                const Sigmoid g(z[e]);
                act[e] = a.silu ? z[e] * g.s : g.s;
                slope[e] = a.silu ? g.s * (1.f + z[e] * g.rest) : g.s * g.rest;
            }
            ss = fmaf(u[e], u[e], ss);
            pu = fmaf(dy[e] * w[e] * act[e], u[e], pu);
        }
        ss = row_sum<L>(ss);
        pu = row_sum<L>(pu);
        float mean = ss * inv_d + a.eps;
        const float scale = row_scale<L>(u, mean, a.eps);
        if (scale != 1.f) {
            ss = pu = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                u[e] *= scale;
                ss = fmaf(u[e], u[e], ss);
                pu = fmaf(dy[e] * w[e] * act[e], u[e], pu);
            }
            ss = row_sum<L>(ss);
            pu = row_sum<L>(pu);
            mean = ss * inv_d + a.eps * scale * scale;
        }
        const float rho = 1.f / sqrtf(mean);
        const float back = rho * rho * pu * inv_d;  // rho mean(p n), n = u rho
        float dx[8], dz[8], ds = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float n = u[e] * rho, t = dy[e] * n;
            dx[e] = rho * (dy[e] * w[e] * act[e] - u[e] * back) * scale;
            dz[e] = t * w[e] * slope[e];
            dw[e] = fmaf(t, act[e], dw[e]);
            ds = fmaf(dx[e], res[e], ds);
        }
        if (in) {
            store8(a.dx + at, dx);
            if (a.gate) store8(a.dgate + at, dz);
            if (a.res) {
#pragma unroll
                for (int e = 0; e < 8; ++e) dx[e] *= rs;
                store8(a.dres + at, dx);
            }
        }
        if (a.res) {
            ds = row_sum<L>(ds);
            if (l == 0) a.row_ds[row] = ds;
        }
    }
    // the workgroup's sum for each channel
#pragma unroll
    for (int e = 0; e < 8; ++e) red[threadIdx.x][e] = dw[e];
    __syncthreads();
    for (int d = threadIdx.x; d < a.D; d += GN_THREADS) {
        float s = 0.f;
        for (int i = 0; i < RPW; ++i) s += red[i * L + d / 8][d % 8];
        a.part_w[(int64_t)blockIdx.x * a.D + d] = s;
    }
}

// sum of n values, `step` apart, 32 loads in flight at a time
__device__ __forceinline__ double sum_strided(const float* p, int64_t n, int64_t step) {
    double s = 0.0;
    for (int64_t i = 0; i < n; i += 32) {
        float v[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = p[(i + k < n ? i + k : n - 1) * step];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < 32; ++k) s += i + k < n ? v[k] : 0.f;
    }
    return s;
}

// dweight and dres_scale from the partial sums: workgroup b < D / 8 adds
// channels 8 b .. 8 b + 7 over the groups, the others one head's rows.  The latency
// of its loads bounds it: 11.5 us with one in flight, 4.6 with 32.
__global__ __launch_bounds__(GN_THREADS) void gated_norm_sum_kernel(GatedNormArgs a) {
    __shared__ double red[GN_THREADS];
    const int tid = threadIdx.x, wb = a.D / 8;
    const int64_t wg = (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
    if (wg >= (int64_t)wb + a.H) return;
    double s = 0.0;
    const bool weight = wg < wb;
    const int h = (int)(wg - wb);
    if (weight) {
        const int first = tid / 8, step = GN_THREADS / 8;
        s = sum_strided(a.part_w + (int64_t)first * a.D + 8 * wg + tid % 8,
                        ((int64_t)a.groups - first + step - 1) / step, (int64_t)step * a.D);
    } else {
        s = sum_strided(a.row_ds + (int64_t)tid * a.H + h, (a.rows / a.H - tid + GN_THREADS - 1) / GN_THREADS,
                        (int64_t)GN_THREADS * a.H);
    }
    red[tid] = s;
    __syncthreads();
    const int keep = weight ? 8 : 1;
    for (int m = GN_THREADS / 2; m >= keep; m >>= 1) {
        if (tid < m) red[tid] += red[tid + m];
        __syncthreads();
    }
    if (tid < keep) {
        if (weight) a.dweight[8 * wg + tid] = (float)red[tid];
        else a.dres_scale[h] = (float)red[0];
    }
}

namespace {

int row_lanes(int32_t D) {
    int l = 1;
    while (8 * l < D) l *= 2;
    return l;
}

template <class F>
void by_lanes(int l, F&& f) {
    switch (l) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        case 4: return f(std::integral_constant<int, 4>{});
        case 8: return f(std::integral_constant<int, 8>{});
        case 16: return f(std::integral_constant<int, 16>{});
        case 32: return f(std::integral_constant<int, 32>{});
        default: return f(std::integral_constant<int, 64>{});
    }
}

}  // namespace

int32_t gated_norm_groups(int64_t rows, int32_t D) {
    const int64_t per = GN_THREADS / row_lanes(D);
    const int64_t g = (rows + per - 1) / per;
    return (int32_t)(g < 1 ? 1 : g > GN_GROUPS ? GN_GROUPS : g);
}

void launch_gated_norm_fwd(const GatedNormArgs& a, hipStream_t stream) {
    by_lanes(row_lanes(a.D), [&](auto l) {
        constexpr int L = decltype(l)::value;
        constexpr int RPW = GN_THREADS / L;
        hipLaunchKernelGGL((gated_norm_fwd_kernel<L>), wide_grid((a.rows + RPW - 1) / RPW, GN_THREADS), dim3(GN_THREADS),
                           0, stream, a);
    });
}

void launch_gated_norm_bwd(const GatedNormArgs& a, hipStream_t stream) {
    by_lanes(row_lanes(a.D), [&](auto l) {
        hipLaunchKernelGGL((gated_norm_bwd_kernel<decltype(l)::value>), dim3((unsigned)a.groups), dim3(GN_THREADS), 0,
                           stream, a);
    });
    hipLaunchKernelGGL(gated_norm_sum_kernel, wide_grid(a.D / 8 + (a.res_scale ? (int64_t)a.H : 0), GN_THREADS),
                       dim3(GN_THREADS), 0, stream, a);
}

}  // namespace kda
