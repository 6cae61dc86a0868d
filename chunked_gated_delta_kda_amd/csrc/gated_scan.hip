// gated_scan.hip -- the gated linear recurrence over channels (gfx950): per
// channel c of a sequence, with the decay gate of KDA and a gate on the input,
//   L_t = exp(A_log[c]) softplus(g_t + dt_bias[c]),  a_t = exp(-L_t),
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t,  o_t = h_t.
// Gradients, with e_t = dL/dh_t = do_t + a_{t+1} e_{t+1}, m = sqrt(1 - a^2),
// s = sigmoid(i), p_t = dL/dL_t = a e (a s x / m - h_{t-1}):
//   dx = e m s,  di = e m x s (1 - s),  dg = p exp(A_log) sigmoid(g + dt_bias),
//   dA_log = sum p L,  ddt_bias = sum dg,  dh0 = a_0 e_0.
//
// One pass over the data.  A wave has 64 words of a token row (128 bf16 channels,
// 64 of fp32) for 16 tokens, a workgroup eight such waves one behind the other: a
// tile of 128 tokens.  Every wave scans its own tokens from a zero state, keeping
// the state and the product of the decays at each; the eight pairs (product,
// state) are joined through LDS, the tiles of a chain through memory
// (enter_tile), and each output is then one fused multiply-add from the state that
// enters the wave.  Gradients run the same way from the last token to the first,
// in tiles of 64 tokens; the states they need are scanned again from those that
// the forward pass kept at the head of each.
#include "block_device.h"

namespace kda {

namespace {

constexpr int GS_WAVES = 8;
constexpr int GS_THREADS = 64 * GS_WAVES;
constexpr int TICKET_WORDS = GS_TICKET_BYTES / 4;
constexpr int FWD_STEPS = 16, BWD_STEPS = 8;  // tokens of a wave
constexpr int FWD_TILE = GS_WAVES * FWD_STEPS, BWD_TILE = GS_WAVES * BWD_STEPS;
static_assert(BWD_TILE == GS_STATES && FWD_TILE == 2 * GS_STATES, "the states kept are those entering a BWD_TILE");

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
__device__ __forceinline__ float join(float prod, float before) { return prod == 0.f ? 0.f : prod * before; }

__host__ __device__ __forceinline__ int tiles_of(int T, int tile) { return (int)(((int64_t)T + tile - 1) / tile); }
__device__ __forceinline__ int clamp_to(int v, int T) { return min(max(v, 0), T); }

// What a tile makes of the state that enters it, as one 64-bit word that the tiles behind
// it read while it runs: (product, sum), or (0, state left behind) once that is known.
// One atomic word needs no order of stores; EMPTY is a product that no tile has.
constexpr uint64_t EMPTY = ~0ull;

__device__ __forceinline__ void post(uint64_t* p, float prod, float sum) {
    const uint32_t lo = prod != prod ? 0x7fc00000u : __float_as_uint(prod);
    __hip_atomic_store(p, (uint64_t)__float_as_uint(sum) << 32 | lo, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float word_prod(uint64_t w) { return __uint_as_float((uint32_t)w); }
__device__ __forceinline__ float word_sum(uint64_t w) { return __uint_as_float((uint32_t)(w >> 32)); }

// Waits until the tiles back, back + GS_WAVES, ... (n of them) before the one that posts at
// `own` have posted, and tile `state` before it even knows the state behind it.  The number
// of looks is bounded all the same: a workspace that someone else writes to gives NaN, not
// a hang.
template <int V, int n>
__device__ __forceinline__ void await_words(const uint64_t* own, int64_t step, int order, int back, int state,
                                            int lane, uint64_t (*look)[64 * V]) {
    uint64_t word[n][V];
    for (int looks = 0;; ++looks) {
#pragma unroll
        for (int i = 0; i < n; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v)
                word[i][v] = __hip_atomic_load(own + v - (1 + min(back + i * GS_WAVES, order - 1)) * step,
                                               __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        bool ready = true;
#pragma unroll
        for (int i = 0; i < n; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v)
                ready = ready && (back + i * GS_WAVES == state ? word_prod(word[i][v]) == 0.f
                                                              : (uint32_t)word[i][v] != (uint32_t)EMPTY);
        if (__all(ready)) break;
        if (looks == 1 << 20) {
#pragma unroll
            for (int i = 0; i < n; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) word[i][v] = 0x7fc00000ull << 32;
            break;
        }
        __builtin_amdgcn_s_sleep(1);
    }
#pragma unroll
    for (int i = 0; i < n; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) look[back + i * GS_WAVES][lane * V + v] = word[i][v];
}

// The state that enters tile `order` of a chain (0: `first`), whose own product and sum
// are (prod, sum) in the last wave.  The words of the eight tiles before this one are
// looked at first, one by each wave; where none is a state in all channels, those of the
// next 24, of which the oldest is waited for until it is one.  Folded from the oldest on,
// this is the same sum in the same order whatever each tile had posted by then: bits do
// not depend on time.  A tile waits only for tiles whose tickets were drawn before
// its own: those run already, and wait for earlier ones in turn.
constexpr int NEAR = GS_WAVES, FAR = 4 * GS_WAVES;

template <int V>
__device__ __forceinline__ void enter_tile(const ScanArgs& a, int tiles, int order, int64_t column, bool active, int w, int lane,
                                           const float (&prod)[V], const float (&sum)[V], const float (&first)[V],
                                           uint64_t (*look)[64 * V], float (&in)[V]) {
    const int64_t step = (int64_t)a.B * a.C;
    uint64_t* own = a.words + order * step + column;
    const bool poster = w == GS_WAVES - 1 && active;
    if (order == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) in[v] = first[v];
    } else {
        if (poster) {
#pragma unroll
            for (int v = 0; v < V; ++v) post(own + v, prod[v], sum[v]);
        }
        const auto fold = [&](int from) {
            for (int j = from; j >= 0; --j) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const uint64_t t = look[j][lane * V + v];
                    in[v] = carry(word_prod(t), word_sum(t), in[v]);
                }
            }
        };
        await_words<V, 1>(own, step, order, w, a.far ? -1 : NEAR - 1, lane, look);
        __syncthreads();
        int from = min(order, NEAR) - 1;
        if (a.far && order > NEAR) {
            bool state = true;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                bool some = false;
#pragma unroll
                for (int j = 0; j < NEAR; ++j) some = some || word_prod(look[j][lane * V + v]) == 0.f;
                state = state && some;
            }
            if (!__all(state)) {  // (the same words in every wave)
                await_words<V, FAR / NEAR - 1>(own, step, order, w + NEAR, FAR - 1, lane, look);
                __syncthreads();
                from = min(order, FAR) - 1;
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) in[v] = 0.f;
        fold(from);
    }
    if (poster && order + 1 < tiles) {
#pragma unroll
        for (int v = 0; v < V; ++v) post(own + v, 0.f, carry(prod[v], sum[v], in[v]));
    }
}

// The compiler takes v for another value from here on (and computes from it anew).
__device__ __forceinline__ void forget(uint32_t& v) { asm volatile("" : "+v"(v)); }

// What a wave knows of its place: its channels and, of a packed batch, its tokens.
struct Marks {
    uint32_t start, in, last;
    __device__ __forceinline__ Marks() {}
    // those from token t0 on (a multiple of 8)
    __device__ __forceinline__ Marks(const ScanArgs& a, int t0) : start(0), in(0), last(0) {
        if (t0 >= a.T) return;
        const uint2 m = a.marks[t0 / 16];
        start = uniform((m.x & 0xffffu) >> t0 % 16);
        in = uniform((m.x >> 16) >> t0 % 16);
        last = uniform(m.y >> t0 % 16);
    }
    static __device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }
};

}  // namespace

// What a pass needs before it: words that are empty and tickets that are not drawn; of a packed batch
// which sequence each token belongs to and which tokens begin and end one; and for the
// sequences without a token, the state behind them (dst = src, or zeros).  Workgroups
// [0, fill) have the words, the next `marks` the tokens, the others a sequence each.
struct PrepareArgs {
    ScanArgs a;
    int64_t fill, marks;
    int64_t n_words, n_tickets;
    const float* src;
    float* dst;
};

__global__ __launch_bounds__(256) void gated_scan_prepare_kernel(PrepareArgs q) {
    const ScanArgs& a = q.a;
    int64_t wg = (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
    if (wg < q.fill) {
        // (8 words a thread, 2 at a time; their number is a multiple of 8.  There are more
        // threads than tickets.)
        const int64_t first = wg * 2048 + threadIdx.x * 2;
        if (wg * 256 + threadIdx.x < q.n_tickets) a.tickets[(wg * 256 + threadIdx.x) * TICKET_WORDS] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (first + i * 512 < q.n_words)
                *reinterpret_cast<u32x4*>(a.words + first + i * 512) = u32x4{~0u, ~0u, ~0u, ~0u};
        return;
    }
    wg -= q.fill;
    if (wg < q.marks) {
        const int64_t t64 = wg * 256 + threadIdx.x;
        if (t64 >= ((int64_t)a.T + 15) / 16 * 16) return;  // (whole groups of 16 lanes)
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
        const uint32_t bs = (uint32_t)(__ballot(start) >> sh) & 0xffffu,
                       bi = (uint32_t)(__ballot(in) >> sh) & 0xffffu, bl = (uint32_t)(__ballot(last) >> sh) & 0xffffu;
        if (threadIdx.x % 16 == 0) a.marks[t / 16] = make_uint2(bs | bi << 16, bl);
        return;
    }
    const int64_t n = wg - q.marks;
    if (!q.dst || n >= a.N) return;
    if (a.T > 0 && clamp_to(a.cu[n + 1], a.T) > clamp_to(a.cu[n], a.T)) return;
    for (int c = threadIdx.x; c < a.C; c += 256) q.dst[n * a.C + c] = q.src ? q.src[n * a.C + c] : 0.f;
}

// The tile that this workgroup takes.  A counter has the tiles of a.beside chains (a row of
// the batch and a block of channels) side by side, in the order of time; workgroup i draws
// from counter i % counters, as many from each as it has tiles.
struct Place {
    int64_t chain;
    int order;
    __device__ __forceinline__ Place(const ScanArgs& a, int tiles, int64_t chains) {
        __shared__ uint32_t ticket;
        const int64_t wg = (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
        if (tiles == 1 || wg >= chains * tiles) {
            chain = wg % chains;
            order = (int)(wg / chains);
            return;
        }
        const int64_t counters = chains / a.beside, counter = wg % counters;
        if (threadIdx.x == 0) ticket = atomicAdd(a.tickets + counter * TICKET_WORDS, 1u);
        __syncthreads();
        chain = counter * a.beside + ticket % a.beside;
        order = ticket / a.beside;
    }
};

template <class T, bool PACKED>
__global__ __launch_bounds__(GS_THREADS, 4) void gated_scan_fwd_kernel(ScanArgs a) {
    constexpr int V = Word<T>::N, CB = 64 * V;
    __shared__ float s_prod[GS_WAVES][CB], s_sum[GS_WAVES][CB];
    __shared__ uint64_t look[FAR][CB];
    const int tiles = tiles_of(a.T, FWD_TILE);
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int blocks = (a.C + CB - 1) / CB;
    const Place place(a, tiles, (int64_t)a.B * blocks);
    const int k = place.order, b = (int)(place.chain / blocks), cb = (int)(place.chain % blocks);
    if (k >= tiles) return;
    const int own = cb * CB + lane * V;
    const bool active = own < a.C;
    const int c = active ? own : a.C - V;
    float bias[V], amount[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        bias[v] = a.dt_bias[c + v];
        amount[v] = expf(a.A_log[c + v]);
    }
    const int64_t row_words = a.C / V;
    const int at = c / V;
    const int t0 = k * FWD_TILE + w * FWD_STEPS;
    uint32_t rx[FWD_STEPS], rg[FWD_STEPS], ri[FWD_STEPS];
#pragma unroll
    for (int t = 0; t < FWD_STEPS; ++t) {
        const int64_t row = ((int64_t)b * a.T + min(t0 + t, a.T - 1)) * row_words;
        rx[t] = (static_cast<const uint32_t*>(a.x) + row)[at];
        rg[t] = (static_cast<const uint32_t*>(a.g) + row)[at];
        ri[t] = (static_cast<const uint32_t*>(a.gate) + row)[at];
    }
    Marks m;
    if constexpr (PACKED) m = Marks(a, t0);
    float prod[FWD_STEPS][V], sum[FWD_STEPS][V];
    float p[V], h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        p[v] = 1.f;
        h[v] = 0.f;
    }
#pragma unroll
    for (int t = 0; t < FWD_STEPS; ++t) {
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
    // what the waves before this one make of the tile's state; the last wave's is the tile's
    float bp[V], bs[V], first[V], in[V], enter[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        bp[v] = 1.f;
        bs[v] = 0.f;
        for (int j = 0; j < w; ++j) {
            bs[v] = carry(s_prod[j][lane * V + v], s_sum[j][lane * V + v], bs[v]);
            bp[v] = join(s_prod[j][lane * V + v], bp[v]);
        }
        first[v] = k == 0 && !PACKED && a.h0 ? a.h0[(int64_t)b * a.C + c + v] : 0.f;
        h[v] = carry(p[v], h[v], bs[v]);
        p[v] = join(p[v], bp[v]);
    }
    enter_tile<V>(a, tiles, k, (int64_t)b * a.C + c, active, w, lane, p, h, first, look, in);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        enter[v] = carry(bp[v], bs[v], in[v]);
        if (w % (GS_WAVES / 2) == 0 && a.states && active && t0 < a.T)
            a.states[((int64_t)b * a.n_states + t0 / GS_STATES) * a.C + c + v] = enter[v];
        if (!PACKED && w == GS_WAVES - 1 && a.h_final && k == tiles - 1 && active)
            a.h_final[(int64_t)b * a.C + c + v] = carry(p[v], h[v], in[v]);
    }
#pragma unroll
    for (int t = 0; t < FWD_STEPS; ++t) {
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

template <class T, bool PACKED>
__global__ __launch_bounds__(GS_THREADS, 4) void gated_scan_bwd_kernel(ScanArgs a) {
    constexpr int V = Word<T>::N, CB = 64 * V;
    __shared__ float s_prod[GS_WAVES][CB], s_sum[GS_WAVES][CB];    // states, forwards
    __shared__ float s_bprod[GS_WAVES][CB], s_bsum[GS_WAVES][CB];  // gradients, backwards
    __shared__ uint64_t look[FAR][CB];
    const int tiles = tiles_of(a.T, BWD_TILE);
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int blocks = (a.C + CB - 1) / CB;
    const Place place(a, tiles, (int64_t)a.B * blocks);
    const int order = place.order, k = tiles - 1 - order;
    const int b = (int)(place.chain / blocks), cb = (int)(place.chain % blocks);
    if (k < 0) return;
    const int own = cb * CB + lane * V;
    const bool active = own < a.C;
    const int c = active ? own : a.C - V;
    const int64_t row_words = a.C / V;
    const int at = c / V;
    const int t0 = k * BWD_TILE + w * BWD_STEPS;
    float bias[V], amount[V], enter[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        bias[v] = a.dt_bias[c + v];
        amount[v] = expf(a.A_log[c + v]);
        enter[v] = a.states[((int64_t)b * a.n_states + k) * a.C + c + v];
    }
    Marks m;
    if constexpr (PACKED) m = Marks(a, t0);
    const auto there = [&](int t) { return PACKED ? (m.in >> t & 1) != 0 : t0 + t < a.T; };
    float dec[BWD_STEPS][V], prev[BWD_STEPS][V];
    float p[V], h[V], q[V], e[V];
    uint32_t rx[BWD_STEPS], rg[BWD_STEPS], ri[BWD_STEPS], rd[BWD_STEPS];
#pragma unroll
    for (int t = 0; t < BWD_STEPS; ++t) {
        const int64_t row = ((int64_t)b * a.T + min(t0 + t, a.T - 1)) * row_words;
        rx[t] = (static_cast<const uint32_t*>(a.x) + row)[at];
        rg[t] = (static_cast<const uint32_t*>(a.g) + row)[at];
        ri[t] = (static_cast<const uint32_t*>(a.gate) + row)[at];
    }
#pragma unroll
    for (int t = 0; t < BWD_STEPS; ++t) {
        const int64_t row = ((int64_t)b * a.T + min(t0 + t, a.T - 1)) * row_words;
        rd[t] = (static_cast<const uint32_t*>(a.d_o) + row)[at];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        p[v] = q[v] = 1.f;
        h[v] = e[v] = 0.f;
    }
    // states from zero
#pragma unroll
    for (int t = 0; t < BWD_STEPS; ++t) {
        float x[V], g[V], i[V];
        Word<T>::get(rx[t], x);
        Word<T>::get(rg[t], g);
        Word<T>::get(ri[t], i);
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
                    p[v] = there(t) ? p[v] * d.a : 0.f;
                    h[v] = there(t) ? fmaf(d.a, h[v], in) : 0.f;
                }
            } else {
                p[v] = there(t) ? p[v] * d.a : p[v];
                h[v] = there(t) ? fmaf(d.a, h[v], in) : h[v];
            }
            dec[t][v] = d.a;
            prev[t][v] = h[v];
        }
    }
    // gradients of the states, from zero, last token first: what reaches the state
    // before a token is a (do + what reaches its own)
#pragma unroll
    for (int t = BWD_STEPS - 1; t >= 0; --t) {
        float d[V];
        Word<T>::get(rd[t], d);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if constexpr (PACKED) {
                if (m.last >> t & 1) {
                    const float df = a.d_final ? a.d_final[(int64_t)a.seq[t0 + t] * a.C + c + v] : 0.f;
                    q[v] = 0.f;
                    e[v] = dec[t][v] * (d[v] + df);
                } else {
                    q[v] = there(t) ? q[v] * dec[t][v] : 0.f;
                    e[v] = there(t) ? dec[t][v] * (d[v] + e[v]) : 0.f;
                }
            } else {
                q[v] = there(t) ? q[v] * dec[t][v] : q[v];
                e[v] = there(t) ? dec[t][v] * (d[v] + e[v]) : e[v];
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
    // (the wave that posts a tile's word is the last: it folds all waves' gradients, the
    // others those behind them)
    float bp[V], bs[V], tp[V], ts[V], first[V], in[V], back[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        for (int j = 0; j < w; ++j) enter[v] = carry(s_prod[j][lane * V + v], s_sum[j][lane * V + v], enter[v]);
        bp[v] = tp[v] = 1.f;
        bs[v] = ts[v] = 0.f;
        for (int j = GS_WAVES - 1; j > w; --j) {
            bs[v] = carry(s_bprod[j][lane * V + v], s_bsum[j][lane * V + v], bs[v]);
            bp[v] = join(s_bprod[j][lane * V + v], bp[v]);
        }
        if (w == GS_WAVES - 1) {
            for (int j = GS_WAVES - 1; j >= 0; --j) {
                ts[v] = carry(s_bprod[j][lane * V + v], s_bsum[j][lane * V + v], ts[v]);
                tp[v] = join(s_bprod[j][lane * V + v], tp[v]);
            }
        }
        first[v] = order == 0 && !PACKED && a.d_final ? a.d_final[(int64_t)b * a.C + c + v] : 0.f;
    }
    enter_tile<V>(a, tiles, order, (int64_t)b * a.C + c, active, w, lane, tp, ts, first, look, in);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        back[v] = carry(bp[v], bs[v], in[v]);
        if (!PACKED && w == GS_WAVES - 1 && a.dh0 && k == 0 && active)
            a.dh0[(int64_t)b * a.C + c + v] = carry(tp[v], ts[v], in[v]);
    }
    // the state before each token, from what a zero state left after it
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float prod = 1.f, before = enter[v];
#pragma unroll
        for (int t = 0; t < BWD_STEPS; ++t) {
            const float after = prev[t][v];
            prev[t][v] = before;
            if constexpr (PACKED) {
                if (m.start >> t & 1) {
                    prev[t][v] = a.h0 ? a.h0[(int64_t)a.seq[t0 + t] * a.C + c + v] : 0.f;
                    prod = 0.f;
                }
            }
            prod *= dec[t][v];
            before = carry(prod, after, enter[v]);
        }
    }
    float dA[V], db[V];
#pragma unroll
    for (int v = 0; v < V; ++v) dA[v] = db[v] = 0.f;
    // the gates are computed again: kept, they would take the registers of a second
    // workgroup
#pragma unroll
    for (int t = 0; t < BWD_STEPS; ++t) {
        forget(rx[t]);
        forget(rg[t]);
        forget(ri[t]);
        forget(rd[t]);
    }
#pragma unroll
    for (int t = BWD_STEPS - 1; t >= 0; --t) {
        float x[V], g[V], i[V], d_o[V], dx[V], dg[V], di[V];
        Word<T>::get(rx[t], x);
        Word<T>::get(rg[t], g);
        Word<T>::get(ri[t], i);
        Word<T>::get(rd[t], d_o);
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
            if (there(t)) {
                dA[v] = fmaf(pt, d.L, dA[v]);
                db[v] += dg[v];
                back[v] = d.a * et;
            } else {
                dx[v] = di[v] = dg[v] = 0.f;
            }
            if constexpr (PACKED) {
                if (a.dh0 && active && m.start >> t & 1) a.dh0[(int64_t)a.seq[t0 + t] * a.C + c + v] = back[v];
            }
        }
        if (active && t0 + t < a.T) {
            const int64_t row = ((int64_t)b * a.T + t0 + t) * row_words;
            (static_cast<uint32_t*>(a.dx) + row)[at] = Word<T>::put(dx);
            (static_cast<uint32_t*>(a.dg) + row)[at] = Word<T>::put(dg);
            (static_cast<uint32_t*>(a.dgate) + row)[at] = Word<T>::put(di);
        }
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) {
        s_prod[w][lane * V + v] = dA[v];
        s_sum[w][lane * V + v] = db[v];
    }
    __syncthreads();
    if (w < 2 && active) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float s = 0.f;
            for (int j = 0; j < GS_WAVES; ++j) s += w ? s_sum[j][lane * V + v] : s_prod[j][lane * V + v];
            a.part[(((int64_t)b * tiles + k) * 2 + w) * a.C + c + v] = s;
        }
    }
}

// dA_log and ddt_bias from the tiles' sums: a workgroup for 32 channels of one of them
__global__ __launch_bounds__(256) void gated_scan_sum_kernel(ScanArgs a) {
    const int which = blockIdx.x % 2, c = blockIdx.x / 2 * 32 + threadIdx.x % 32;
    const double s = sum_columns(a.part + (int64_t)which * a.C + min(c, a.C - 1), (int64_t)a.B * a.n_states,
                                 (int64_t)2 * a.C);
    if (threadIdx.x < 32 && c < a.C) (which ? a.ddt_bias : a.dA_log)[c] = (float)s;
}

// One token: a word of a row a lane.
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

int64_t chains_of(const ScanArgs& a, bool fp32) {
    const int per = 64 * (fp32 ? Word<float>::N : Word<uint16_t>::N);
    return (int64_t)a.B * ((a.C + per - 1) / per);
}

void launch_prepare(const ScanArgs& a, int tiles, int64_t chains, const float* src, float* dst, hipStream_t stream) {
    PrepareArgs q{};
    q.a = a;
    q.n_words = tiles > 1 ? (int64_t)tiles * a.B * a.C : 0;
    q.n_tickets = tiles > 1 ? chains / a.beside : 0;
    q.fill = (q.n_words + 2047) / 2048;
    q.marks = a.cu ? ((int64_t)a.T + 255) / 256 : 0;
    q.src = src;
    q.dst = a.cu || a.T == 0 ? dst : nullptr;
    const int64_t groups = q.fill + q.marks + (q.dst ? a.N : 0);
    if (groups) hipLaunchKernelGGL(gated_scan_prepare_kernel, wide_grid(groups, 256), dim3(256), 0, stream, q);
}

#ifndef FAR_GROUPS
#define FAR_GROUPS GS_MAX_COUNTERS
#define OWN_GROUPS GS_MAX_COUNTERS
#endif
int64_t set_chains(ScanArgs& a, int tiles, bool fp32) {
    const int64_t chains = chains_of(a, fp32);
    a.far = chains * tiles <= FAR_GROUPS;
    a.beside = chains * tiles <= OWN_GROUPS ? 1 : (int32_t)chains;
    return chains;
}

template <class F>
void by_type(bool fp32, bool packed, F&& f) {
    if (fp32) packed ? f(float{}, std::true_type{}) : f(float{}, std::false_type{});
    else packed ? f(uint16_t{}, std::true_type{}) : f(uint16_t{}, std::false_type{});
}

}  // namespace

void launch_gated_scan_fwd(const ScanArgs& args, bool fp32, hipStream_t stream) {
    ScanArgs a = args;
    const int tiles = tiles_of(a.T, FWD_TILE);
    const int64_t chains = set_chains(a, tiles, fp32);
    launch_prepare(a, tiles, chains, a.h0, a.h_final, stream);
    if (a.T == 0) return;
    by_type(fp32, a.cu != nullptr, [&](auto t, auto packed) {
        using T = decltype(t);
        hipLaunchKernelGGL((gated_scan_fwd_kernel<T, decltype(packed)::value>),
                           wide_grid(chains * tiles, GS_THREADS), dim3(GS_THREADS), 0,
                           stream, a);
    });
}

void launch_gated_scan_bwd(const ScanArgs& args, bool fp32, hipStream_t stream) {
    ScanArgs a = args;
    const int tiles = tiles_of(a.T, BWD_TILE);
    const int64_t chains = set_chains(a, tiles, fp32);
    launch_prepare(a, tiles, chains, a.d_final, a.dh0, stream);
    if (a.T > 0) {
        by_type(fp32, a.cu != nullptr, [&](auto t, auto packed) {
            using T = decltype(t);
                hipLaunchKernelGGL((gated_scan_bwd_kernel<T, decltype(packed)::value>),
                               wide_grid(chains * tiles, GS_THREADS),
                               dim3(GS_THREADS), 0, stream, a);
        });
    }
    hipLaunchKernelGGL(gated_scan_sum_kernel, dim3((unsigned)((a.C + 31) / 32 * 2)), dim3(256), 0, stream, a);
}

void launch_gated_scan_decode(const ScanDecodeArgs& a, bool fp32, hipStream_t stream) {
    const int64_t words = (int64_t)a.N * a.C / (fp32 ? 1 : 2);
    const dim3 grid = wide_grid((words + 255) / 256, 256);
    if (fp32) hipLaunchKernelGGL(gated_scan_decode_kernel<float>, grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL(gated_scan_decode_kernel<uint16_t>, grid, dim3(256), 0, stream, a);
}

}  // namespace kda
