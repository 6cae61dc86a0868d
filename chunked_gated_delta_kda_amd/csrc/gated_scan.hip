// gated_scan.hip -- the gated linear recurrence over channels (gfx950): per
// channel c of a sequence, with the decay gate of KDA and a gate on the input,
//   L_t = exp(A_log[c]) softplus(g_t + dt_bias[c]),  a_t = exp(-L_t),
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t,  o_t = h_t.
// Gradients, with e_t = dL/dh_t = do_t + a_{t+1} e_{t+1}, m = sqrt(1 - a^2),
// s = sigmoid(i), p_t = dL/dL_t = a e (a s x / m - h_{t-1}):
//   dx = e m s,  di = e m x s (1 - s),  dg = p exp(A_log) sigmoid(g + dt_bias),
//   dA_log = sum p L,  ddt_bias = sum dg,  dh0 = a_0 e_0.
//
// A wave has 64 words of a token row (128 bf16 channels, 64 of fp32) for 16
// tokens, a workgroup eight such waves one behind the other: a tile of 128
// tokens.  Every wave scans its own tokens from a zero state, keeping the state
// and the product of the decays at each; the eight pairs (product, state) are
// joined through LDS, and each output is then one fused multiply-add from the
// state that enters the wave.  Gradients run the same way from the last token
// to the first; the states they need are scanned again from the state that the
// forward pass kept at the head of each tile.
#include "block_device.h"

namespace kda {

namespace {

constexpr int GS_WAVES = 8;
constexpr int GS_STEPS = GS_TILE / GS_WAVES;  // tokens of a wave
constexpr int GS_THREADS = 64 * GS_WAVES;
static_assert(GS_STEPS == 16, "marks are 16-bit masks");

// The decay's gate for one element.  e = exp(-|z|), r = 1 / (1 + e) give
// softplus(z) = max(z, 0) + log(1 + e) and sigmoid(z) = r or e r.  1 + e rounds
// what a slow channel's decay is made of away: the lost part (e - (u - 1)) comes
// back to first order.
struct Decay {
    float L, a, sig;
    __device__ __forceinline__ Decay(float z, float amount) {
        const float e = __builtin_amdgcn_exp2f(-LOG2E * fabsf(z));
        const float u = 1.f + e, r = __builtin_amdgcn_rcpf(u);
        const float log1p = fmaf(__builtin_amdgcn_logf(u), LN2, (e - (u - 1.f)) * r);
        L = amount * (fmaxf(z, 0.f) + log1p);
        a = __builtin_amdgcn_exp2f(-LOG2E * L);
        sig = z < 0.f ? e * r : r;
    }
};

// 1 - a^2 = 1 - exp(-2 L): by its series where a^2 is close to one (the next term is
// below 2^-26 of it), else from a.
__device__ __forceinline__ float one_minus_square(float L, float a) {
    const float t = 2.f * L;
    float s = 1.f / 5040.f;
    s = fmaf(s, -t, 1.f / 720.f);
    s = fmaf(s, -t, 1.f / 120.f);
    s = fmaf(s, -t, 1.f / 24.f);
    s = fmaf(s, -t, 1.f / 6.f);
    s = fmaf(s, -t, 0.5f);
    s = fmaf(s, -t, 1.f);
    return t < 0.25f ? s * t : fmaf(-a, a, 1.f);
}

// A gate on the input: s and s (1 - s).
struct InputGate {
    float s, slope;
    __device__ __forceinline__ explicit InputGate(float i) {
        const float e = __builtin_amdgcn_exp2f(-LOG2E * fabsf(i)), r = __builtin_amdgcn_rcpf(1.f + e);
        s = i < 0.f ? e * r : r;
        slope = e * r * r;
    }
};

// (product, sum) applied to a state: behind a product of zero nothing of the state is
// left, not even an infinity or a NaN of another sequence
__device__ __forceinline__ float carry(float prod, float sum, float h) { return prod == 0.f ? sum : fmaf(prod, h, sum); }

__device__ __forceinline__ int clamp_to(int v, int T) { return min(max(v, 0), T); }

// What a wave knows of its place: its channels and, of a packed batch, its tokens.
struct Marks {
    uint32_t start, in, last;
    __device__ __forceinline__ Marks() {}
    __device__ __forceinline__ explicit Marks(uint2 m) : start(m.x & 0xffffu), in(m.x >> 16), last(m.y) {}
};

}  // namespace

// Of a packed batch: which sequence each token belongs to, which tokens begin and end one.
__global__ __launch_bounds__(256) void gated_scan_marks_kernel(ScanArgs a) {
    const int64_t t64 = ((int64_t)blockIdx.z * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
    const int64_t padded = ((int64_t)a.T + 15) / 16 * 16;
    if (t64 >= padded) return;  // (whole groups of 16 lanes)
    const int t = (int)t64;
    int lo = 0, hi = a.N;
    while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        if (clamp_to(a.cu[mid], a.T) <= t) lo = mid + 1;
        else hi = mid;
    }
    const int n = lo - 1;
    bool in = false, start = false, last = false;
    if (n >= 0 && t < a.T) {
        const int s = clamp_to(a.cu[n], a.T), e = clamp_to(a.cu[n + 1], a.T);
        in = t < e;
        start = in && t == s;
        last = in && t == e - 1;
    }
    a.seq[t] = max(n, 0);
    const int sh = threadIdx.x & 48;
    const uint32_t bs = (uint32_t)(__ballot(start) >> sh) & 0xffffu, bi = (uint32_t)(__ballot(in) >> sh) & 0xffffu,
                   bl = (uint32_t)(__ballot(last) >> sh) & 0xffffu;
    if (threadIdx.x % 16 == 0) a.marks[t / 16] = make_uint2(bs | bi << 16, bl);
}

// dst = src (or zeros) for the sequences without a token: a workgroup a sequence.
__global__ __launch_bounds__(256) void gated_scan_empty_kernel(const int32_t* cu, int32_t T, int32_t N, int32_t C,
                                                               const float* src, float* dst) {
    const int64_t n = (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
    if (n >= N) return;
    if (T > 0 && (!cu || clamp_to(cu[n + 1], T) > clamp_to(cu[n], T))) return;
    for (int c = threadIdx.x; c < C; c += 256) dst[n * C + c] = src ? src[n * C + c] : 0.f;
}

template <class T, bool PACKED>
__global__ __launch_bounds__(GS_THREADS) void gated_scan_fwd_kernel(ScanArgs a) {
    constexpr int V = Word<T>::N, CB = 64 * V;
    __shared__ float s_prod[GS_WAVES][CB], s_sum[GS_WAVES][CB], s_carry[CB];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int blocks = (a.C + CB - 1) / CB;
    const int64_t chain = (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
    if (chain >= (int64_t)a.B * blocks) return;
    const int b = (int)(chain / blocks), cb = (int)(chain % blocks);
    const int own = cb * CB + lane * V;
    const bool active = own < a.C;
    const int c = active ? own : a.C - V;
    float bias[V], amount[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        bias[v] = a.dt_bias[c + v];
        amount[v] = expf(a.A_log[c + v]);
        if (w == 0) s_carry[lane * V + v] = !PACKED && a.h0 ? a.h0[(int64_t)b * a.C + c + v] : 0.f;
    }
    const int64_t row_words = a.C / V;
    const int at = c / V;
    for (int k = 0; k < a.tiles; ++k) {
        const int t0 = k * GS_TILE + w * GS_STEPS;
        uint32_t rx[GS_STEPS], rg[GS_STEPS], ri[GS_STEPS];
#pragma unroll
        for (int t = 0; t < GS_STEPS; ++t) {
            const int64_t row = ((int64_t)b * a.T + min(t0 + t, a.T - 1)) * row_words;
            rx[t] = (static_cast<const uint32_t*>(a.x) + row)[at];
            rg[t] = (static_cast<const uint32_t*>(a.g) + row)[at];
            ri[t] = (static_cast<const uint32_t*>(a.gate) + row)[at];
        }
        Marks m;
        if constexpr (PACKED) m = Marks(t0 < a.T ? a.marks[t0 / 16] : make_uint2(0, 0));
        float prod[GS_STEPS][V], sum[GS_STEPS][V];
        float p[V], h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            p[v] = 1.f;
            h[v] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < GS_STEPS; ++t) {
            float x[V], g[V], i[V];
            Word<T>::get(rx[t], x);
            Word<T>::get(rg[t], g);
            Word<T>::get(ri[t], i);
            const bool there = PACKED ? (m.in >> t & 1) : t0 + t < a.T;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Decay d(g[v] + bias[v], amount[v]);
                const float in = __builtin_amdgcn_sqrtf(one_minus_square(d.L, d.a)) * InputGate(i[v]).s * x[v];
                if constexpr (PACKED) {
                    if (m.start >> t & 1) {
                        const float h0 = a.h0 ? a.h0[(int64_t)a.seq[t0 + t] * a.C + c + v] : 0.f;
                        p[v] = 0.f;
                        h[v] = fmaf(d.a, h0, in);
                    } else {
                        p[v] = there ? p[v] * d.a : 0.f;
                        h[v] = there ? fmaf(d.a, h[v], in) : 0.f;
                    }
                } else {
                    p[v] = there ? p[v] * d.a : p[v];
                    h[v] = there ? fmaf(d.a, h[v], in) : h[v];
                }
                prod[t][v] = p[v];
                sum[t][v] = h[v];
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s_prod[w][lane * V + v] = p[v];
            s_sum[w][lane * V + v] = h[v];
        }
        __syncthreads();
        float enter[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            enter[v] = s_carry[lane * V + v];
            if (a.states && w == 0 && active) a.states[((int64_t)b * a.tiles + k) * a.C + c + v] = enter[v];
            for (int j = 0; j < w; ++j) enter[v] = carry(s_prod[j][lane * V + v], s_sum[j][lane * V + v], enter[v]);
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (w == GS_WAVES - 1) s_carry[lane * V + v] = carry(p[v], h[v], enter[v]);
#pragma unroll
        for (int t = 0; t < GS_STEPS; ++t) {
            if (t0 + t >= a.T || !active) break;
            float o[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if constexpr (PACKED) o[v] = m.in >> t & 1 ? carry(prod[t][v], sum[t][v], enter[v]) : 0.f;
                else o[v] = fmaf(prod[t][v], enter[v], sum[t][v]);
            }
            if constexpr (PACKED) {
                if (a.h_final && m.last >> t & 1) {
#pragma unroll
                    for (int v = 0; v < V; ++v) a.h_final[(int64_t)a.seq[t0 + t] * a.C + c + v] = o[v];
                }
            }
            (static_cast<uint32_t*>(a.o) + ((int64_t)b * a.T + t0 + t) * row_words)[at] = Word<T>::put(o);
        }
    }
    if (!PACKED && a.h_final) {
        __syncthreads();
        if (w == 0 && active) {
#pragma unroll
            for (int v = 0; v < V; ++v) a.h_final[(int64_t)b * a.C + c + v] = s_carry[lane * V + v];
        }
    }
}

template <class T, bool PACKED>
__global__ __launch_bounds__(GS_THREADS) void gated_scan_bwd_kernel(ScanArgs a) {
    constexpr int V = Word<T>::N, CB = 64 * V;
    __shared__ float s_prod[GS_WAVES][CB], s_sum[GS_WAVES][CB];    // states, forwards
    __shared__ float s_bprod[GS_WAVES][CB], s_bsum[GS_WAVES][CB];  // gradients, backwards
    __shared__ float s_carry[CB];
    __shared__ float s_dA[GS_WAVES][CB], s_db[GS_WAVES][CB];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int blocks = (a.C + CB - 1) / CB;
    const int64_t chain = (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
    if (chain >= (int64_t)a.B * blocks) return;
    const int b = (int)(chain / blocks), cb = (int)(chain % blocks);
    const int own = cb * CB + lane * V;
    const bool active = own < a.C;
    const int c = active ? own : a.C - V;
    float bias[V], amount[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        bias[v] = a.dt_bias[c + v];
        amount[v] = expf(a.A_log[c + v]);
        if (w == 0) s_carry[lane * V + v] = !PACKED && a.d_final ? a.d_final[(int64_t)b * a.C + c + v] : 0.f;
    }
    const int64_t row_words = a.C / V;
    const int at = c / V;
    for (int k = a.tiles - 1; k >= 0; --k) {
        const int t0 = k * GS_TILE + w * GS_STEPS;
        uint32_t rx[GS_STEPS], rg[GS_STEPS], ri[GS_STEPS], rd[GS_STEPS];
#pragma unroll
        for (int t = 0; t < GS_STEPS; ++t) {
            const int64_t row = ((int64_t)b * a.T + min(t0 + t, a.T - 1)) * row_words;
            rx[t] = (static_cast<const uint32_t*>(a.x) + row)[at];
            rg[t] = (static_cast<const uint32_t*>(a.g) + row)[at];
            ri[t] = (static_cast<const uint32_t*>(a.gate) + row)[at];
            rd[t] = (static_cast<const uint32_t*>(a.d_o) + row)[at];
        }
        Marks m;
        if constexpr (PACKED) m = Marks(t0 < a.T ? a.marks[t0 / 16] : make_uint2(0, 0));
        float dec[GS_STEPS][V];
        float p[V], h[V], q[V], e[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            p[v] = q[v] = 1.f;
            h[v] = e[v] = 0.f;
        }
        // states from zero
#pragma unroll
        for (int t = 0; t < GS_STEPS; ++t) {
            float x[V], g[V], i[V];
            Word<T>::get(rx[t], x);
            Word<T>::get(rg[t], g);
            Word<T>::get(ri[t], i);
            const bool there = PACKED ? (m.in >> t & 1) : t0 + t < a.T;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Decay d(g[v] + bias[v], amount[v]);
                const float in = __builtin_amdgcn_sqrtf(one_minus_square(d.L, d.a)) * InputGate(i[v]).s * x[v];
                if constexpr (PACKED) {
                    if (m.start >> t & 1) {
                        const float h0 = a.h0 ? a.h0[(int64_t)a.seq[t0 + t] * a.C + c + v] : 0.f;
                        p[v] = 0.f;
                        h[v] = fmaf(d.a, h0, in);
                    } else {
                        p[v] = there ? p[v] * d.a : 0.f;
                        h[v] = there ? fmaf(d.a, h[v], in) : 0.f;
                    }
                } else {
                    p[v] = there ? p[v] * d.a : p[v];
                    h[v] = there ? fmaf(d.a, h[v], in) : h[v];
                }
                dec[t][v] = d.a;
            }
        }
        // gradients of the states, from zero, last token first: what reaches the state
        // before a token is a (do + what reaches its own)
#pragma unroll
        for (int t = GS_STEPS - 1; t >= 0; --t) {
            float d[V];
            Word<T>::get(rd[t], d);
            const bool there = PACKED ? (m.in >> t & 1) : t0 + t < a.T;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if constexpr (PACKED) {
                    if (m.last >> t & 1) {
                        const float df = a.d_final ? a.d_final[(int64_t)a.seq[t0 + t] * a.C + c + v] : 0.f;
                        q[v] = 0.f;
                        e[v] = dec[t][v] * (d[v] + df);
                    } else {
                        q[v] = there ? q[v] * dec[t][v] : 0.f;
                        e[v] = there ? dec[t][v] * (d[v] + e[v]) : 0.f;
                    }
                } else {
                    q[v] = there ? q[v] * dec[t][v] : q[v];
                    e[v] = there ? dec[t][v] * (d[v] + e[v]) : e[v];
                }
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s_prod[w][lane * V + v] = p[v];
            s_sum[w][lane * V + v] = h[v];
            s_bprod[w][lane * V + v] = q[v];
            s_bsum[w][lane * V + v] = e[v];
        }
        __syncthreads();
        float enter[V], back[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            enter[v] = a.states[((int64_t)b * a.tiles + k) * a.C + c + v];
            back[v] = s_carry[lane * V + v];
            for (int j = 0; j < w; ++j) enter[v] = carry(s_prod[j][lane * V + v], s_sum[j][lane * V + v], enter[v]);
            for (int j = GS_WAVES - 1; j > w; --j)
                back[v] = carry(s_bprod[j][lane * V + v], s_bsum[j][lane * V + v], back[v]);
        }
        __syncthreads();
        // the state before each token
        float prev[GS_STEPS][V];
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = enter[v];
#pragma unroll
        for (int t = 0; t < GS_STEPS; ++t) {
            float x[V], g[V], i[V];
            Word<T>::get(rx[t], x);
            Word<T>::get(rg[t], g);
            Word<T>::get(ri[t], i);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if constexpr (PACKED) {
                    if (m.start >> t & 1) h[v] = a.h0 ? a.h0[(int64_t)a.seq[t0 + t] * a.C + c + v] : 0.f;
                }
                const Decay d(g[v] + bias[v], amount[v]);
                const float in = __builtin_amdgcn_sqrtf(one_minus_square(d.L, d.a)) * InputGate(i[v]).s * x[v];
                prev[t][v] = h[v];
                h[v] = fmaf(d.a, h[v], in);
            }
        }
        float dA[V], db[V];
#pragma unroll
        for (int v = 0; v < V; ++v) dA[v] = db[v] = 0.f;
#pragma unroll
        for (int t = GS_STEPS - 1; t >= 0; --t) {
            float x[V], g[V], i[V], d_o[V], dx[V], dg[V], di[V];
            Word<T>::get(rx[t], x);
            Word<T>::get(rg[t], g);
            Word<T>::get(ri[t], i);
            Word<T>::get(rd[t], d_o);
            const bool there = PACKED ? (m.in >> t & 1) : t0 + t < a.T;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if constexpr (PACKED) {
                    if (m.last >> t & 1) back[v] = a.d_final ? a.d_final[(int64_t)a.seq[t0 + t] * a.C + c + v] : 0.f;
                }
                const Decay d(g[v] + bias[v], amount[v]);
                const InputGate ig(i[v]);
                const float m2 = one_minus_square(d.L, d.a);
                // (no decay at all: nothing of the input enters, and nothing comes back)
                const float inv = m2 > 0.f ? __builtin_amdgcn_rsqf(m2) : 0.f;
                const float root = m2 * inv;
                const float et = d_o[v] + back[v];
                const float pt = d.a * et * (d.a * ig.s * x[v] * inv - prev[t][v]);
                dx[v] = et * root * ig.s;
                di[v] = et * root * x[v] * ig.slope;
                dg[v] = pt * amount[v] * d.sig;
                if (there) {
                    dA[v] = fmaf(pt, d.L, dA[v]);
                    db[v] += dg[v];
                    back[v] = d.a * et;
                } else {
                    dx[v] = di[v] = dg[v] = 0.f;
                }
                if constexpr (PACKED) {
                    if (a.dh0 && active && m.start >> t & 1)
                        a.dh0[(int64_t)a.seq[t0 + t] * a.C + c + v] = back[v];
                }
            }
            if (active && t0 + t < a.T) {
                const int64_t row = ((int64_t)b * a.T + t0 + t) * row_words;
                (static_cast<uint32_t*>(a.dx) + row)[at] = Word<T>::put(dx);
                (static_cast<uint32_t*>(a.dg) + row)[at] = Word<T>::put(dg);
                (static_cast<uint32_t*>(a.dgate) + row)[at] = Word<T>::put(di);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s_dA[w][lane * V + v] = dA[v];
            s_db[w][lane * V + v] = db[v];
            if (w == 0) s_carry[lane * V + v] = back[v];
        }
        __syncthreads();
        if (w < 2 && active) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float s = 0.f;
                for (int j = 0; j < GS_WAVES; ++j) s += w ? s_db[j][lane * V + v] : s_dA[j][lane * V + v];
                a.part[(((int64_t)b * a.tiles + k) * 2 + w) * a.C + c + v] = s;
            }
        }
    }
    if (!PACKED && a.dh0) {
        if (w == 0 && active) {
#pragma unroll
            for (int v = 0; v < V; ++v) a.dh0[(int64_t)b * a.C + c + v] = s_carry[lane * V + v];
        }
    }
}

// dA_log and ddt_bias from the tiles' sums, in a fixed order and in 64 bits: a workgroup
// for 8 channels of one of them
__global__ __launch_bounds__(256) void gated_scan_sum_kernel(ScanArgs a) {
    const int which = blockIdx.x % 2, c = blockIdx.x / 2 * 8 + threadIdx.x % 8;
    const double s = sum_columns(a.part + (int64_t)which * a.C + c, (int64_t)a.B * a.tiles, (int64_t)2 * a.C);
    if (threadIdx.x < 8) (which ? a.ddt_bias : a.dA_log)[c] = (float)s;
}

// One token: 4 words of a row a lane.
template <class T>
__global__ __launch_bounds__(256) void gated_scan_decode_kernel(ScanDecodeArgs a) {
    constexpr int V = Word<T>::N;
    const int64_t word = ((int64_t)blockIdx.z * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
    const int64_t row_words = a.C / V;
    if (word >= a.N * row_words) return;
    const int c = (int)(word % row_words) * V;
    float x[V], g[V], i[V], o[V];
    Word<T>::get(static_cast<const uint32_t*>(a.x)[word], x);
    Word<T>::get(static_cast<const uint32_t*>(a.g)[word], g);
    Word<T>::get(static_cast<const uint32_t*>(a.gate)[word], i);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const Decay d(g[v] + a.dt_bias[c + v], expf(a.A_log[c + v]));
        const float in = __builtin_amdgcn_sqrtf(one_minus_square(d.L, d.a)) * InputGate(i[v]).s * x[v];
        o[v] = a.state_in ? fmaf(d.a, a.state_in[word * V + v], in) : in;
        a.state_out[word * V + v] = o[v];
    }
    static_cast<uint32_t*>(a.o)[word] = Word<T>::put(o);
}

namespace {

void launch_marks(const ScanArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL(gated_scan_marks_kernel, wide_grid(((int64_t)a.T + 255) / 256, 256), dim3(256), 0, stream, a);
}

void launch_empty(const ScanArgs& a, const float* src, float* dst, hipStream_t stream) {
    hipLaunchKernelGGL(gated_scan_empty_kernel, wide_grid(a.N, 256), dim3(256), 0, stream, a.cu, a.T, a.N, a.C, src,
                       dst);
}

template <class F>
void by_type(bool fp32, bool packed, F&& f) {
    if (fp32) packed ? f(float{}, std::true_type{}) : f(float{}, std::false_type{});
    else packed ? f(uint16_t{}, std::true_type{}) : f(uint16_t{}, std::false_type{});
}

}  // namespace

void launch_gated_scan_fwd(const ScanArgs& a, bool fp32, hipStream_t stream) {
    if (a.h_final && (a.cu || a.T == 0)) launch_empty(a, a.h0, a.h_final, stream);
    if (a.T == 0) return;
    if (a.cu) launch_marks(a, stream);
    by_type(fp32, a.cu != nullptr, [&](auto t, auto packed) {
        using T = decltype(t);
        constexpr int CB = 64 * Word<T>::N;
        hipLaunchKernelGGL((gated_scan_fwd_kernel<T, decltype(packed)::value>),
                           wide_grid((int64_t)a.B * ((a.C + CB - 1) / CB), GS_THREADS), dim3(GS_THREADS), 0, stream, a);
    });
}

void launch_gated_scan_bwd(const ScanArgs& a, bool fp32, hipStream_t stream) {
    if (a.dh0 && (a.cu || a.T == 0)) launch_empty(a, a.d_final, a.dh0, stream);
    if (a.T > 0) {
        if (a.cu) launch_marks(a, stream);
        by_type(fp32, a.cu != nullptr, [&](auto t, auto packed) {
            using T = decltype(t);
            constexpr int CB = 64 * Word<T>::N;
            hipLaunchKernelGGL((gated_scan_bwd_kernel<T, decltype(packed)::value>),
                               wide_grid((int64_t)a.B * ((a.C + CB - 1) / CB), GS_THREADS), dim3(GS_THREADS), 0,
                               stream, a);
        });
    }
    hipLaunchKernelGGL(gated_scan_sum_kernel, dim3((unsigned)(a.C / 4)), dim3(256), 0, stream, a);
}

void launch_gated_scan_decode(const ScanDecodeArgs& a, bool fp32, hipStream_t stream) {
    const int64_t words = (int64_t)a.N * a.C / (fp32 ? 1 : 2);
    const dim3 grid = wide_grid((words + 255) / 256, 256);
    if (fp32) hipLaunchKernelGGL(gated_scan_decode_kernel<float>, grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL(gated_scan_decode_kernel<uint16_t>, grid, dim3(256), 0, stream, a);
}

}  // namespace kda
