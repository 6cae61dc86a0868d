// gated_scan.hip -- the gated linear recurrence over channels (gfx950): per
// channel c of a sequence, with the decay gate of KDA (no lower bound) and a gate on the input,
//   L_t = exp(A_log[c]) softplus(g_t + dt_bias[c]),  a_t = exp(-L_t),
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t,  o_t = h_t.
// Gradients, with e_t = dL/dh_t = do_t + a_{t+1} e_{t+1}, m = sqrt(1 - a^2),
// s = sigmoid(i), p_t = dL/dL_t = a e (a s x / m - h_{t-1}):
//   dx = e m s,  di = e m x s (1 - s),  dg = p exp(A_log) sigmoid(g + dt_bias),
//   dA_log = sum p L,  ddt_bias = sum dg,  dh0 = a_0 e_0.
//
// One pass over the data, bound by HBM.  A lane has a channel of 16 tokens of a row
// (gradients: 8), a workgroup eight such waves one behind the other: a tile of 64
// channels and 128 tokens (64).  Every wave scans its own tokens from a zero state,
// keeping the state and the product of the decays at each; the eight pairs (product,
// state) are joined through LDS, the tiles of a chain through memory (enter_tile), and
// each output is then one fused multiply-add from the state that enters the wave.
// Gradients run the same way from the last token to the first, in tiles of half the
// tokens, since a token has twice the values to keep; the states they need are scanned
// again from those that the forward pass kept of every eighth token.  One channel a lane
// keeps a forward wave within 64 registers, so that eight fit on a SIMD; two channels a
// lane (rows of 256 bytes) are slower: 131072 x 2048 bf16 tokens took 501 us with two when
// they took 468 with one, 571 and 448 with eight tokens a wave, and the gradients of
// 2 x 2048 x 4096 the same to 1%.  Tiles of 256 tokens halve what tiles exchange, and end
// later: 443 and 448 us, packed prompts 268 and 254.
// Measured (bf16): 131072 x 2048 454 us, 4.7 TB/s; 2 x 2048 x 4096 with the states kept
// 37 us, 3.8 TB/s; their gradients 59 us with the launches before and behind, 4.1 TB/s;
// those of 16384 x 4096 220 us, 4.4 TB/s.
// What bounds the long call is the memory, with the arithmetic close behind: a kernel that
// only moves such rows reaches 4.7 TB/s (of 256 bytes: 5.1), and the VALU is active for 91%
// of the cycles (2 x 2048 x 4096: 72%, its gradients 83%; there the workgroups that run together
// load, compute and store at the same time).  The gradients lose 13 us to three launches.
#include <cfloat>

#include "block_device.h"

namespace kda {

namespace {

constexpr int GS_WAVES = 8;
constexpr int GS_THREADS = 64 * GS_WAVES;
constexpr int TICKET_WORDS = GS_TICKET_BYTES / 4;
constexpr int FWD_STEPS = 16, BWD_STEPS = 8;  // tokens of a wave
constexpr int FWD_TILE = GS_WAVES * FWD_STEPS, BWD_TILE = GS_WAVES * BWD_STEPS;
static_assert(BWD_STEPS == GS_STATES && FWD_STEPS == 2 * GS_STATES, "the states kept are those entering BWD_STEPS tokens");
static_assert(BWD_TILE == GS_TILE, "the smallest tile");

// The decay's gate for one element, in powers of two: L = amount softplus(z) log2(e) and
// a = 2^-L.  With y = z log2(e) and e = 2^-|y|, softplus(z) log2(e) = max(y, 0) +
// log2(1 + e).  1 + e rounds away what a slow channel's decay is made of: the lost part
// e - (u - 1), below 2^-24, comes back (it would have to be divided by u: what that leaves
// out is 2^-24 of the logarithm).
struct Decay {
    float y, log, L, a;
    __device__ __forceinline__ Decay(float z, float amount) {
        y = LOG2E * z;
        const float e = __builtin_amdgcn_exp2f(-fabsf(y)), u = 1.f + e;
        log = fmaf(e - (u - 1.f), LOG2E, __builtin_amdgcn_logf(u));
        L = amount * (fmaxf(y, 0.f) + log);
        a = __builtin_amdgcn_exp2f(-L);
    }
    // 1 - a^2 = 1 - 2^-2L: where a^2 is close to one by a polynomial for (1 - 2^-2L) / L,
    // L <= 0.18 (1e-8 of it at most, fitted to the function), else from a
    __device__ __forceinline__ float one_minus_square() const {
        float s = 0.038452982902526855f;
        s = fmaf(s, L, -0.15323370695114136f);
        s = fmaf(s, L, 0.44399064779281616f);
        s = fmaf(s, L, -0.9609050750732422f);
        s = fmaf(s, L, 1.3862943649291992f);
        return L < 0.18f ? s * L : fmaf(-a, a, 1.f);
    }
    // sigmoid(z) = 2^(y - softplus(z) log2(e))
    __device__ __forceinline__ float sigmoid() const { return __builtin_amdgcn_exp2f(fminf(y, 0.f) - log); }
};

// sigmoid(z), which counts as zero below 2^-126
__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-LOG2E * z));
}

// A gate on the input: s and s (1 - s).
struct InputGate {
    float s, slope;
    __device__ __forceinline__ explicit InputGate(float i) {
        const float e = __builtin_amdgcn_exp2f(-LOG2E * fabsf(i)), r = __builtin_amdgcn_rcpf(1.f + e), er = e * r;
        s = i < 0.f ? er : r;
        slope = er * r;
    }
};

// The product of what is cut off from the state before it, by a sequence's beginning: minus
// zero, which stays itself under products of decays.  (Decays that underflow leave plus zero,
// and a NaN or an infinity of their own sequence goes on.)
constexpr float CUT = -0.f;
__device__ __forceinline__ bool is_cut(float prod) { return __float_as_uint(prod) == 0x80000000u; }

// (product, sum) applied to a state: behind a cut nothing of the state is left, not even an
// infinity or a NaN of another sequence.  (cuts: whether the product may be one.)
template <bool cuts = true>
__device__ __forceinline__ float carry(float prod, float sum, float h) {
    return cuts && is_cut(prod) ? sum : fmaf(prod, h, sum);
}
template <bool cuts = true>
__device__ __forceinline__ float join(float prod, float before) {
    return cuts && is_cut(prod) ? CUT : prod * before;
}

__host__ __device__ __forceinline__ int tiles_of(int T, int tile) { return (int)(((int64_t)T + tile - 1) / tile); }
__device__ __forceinline__ int clamp_to(int v, int T) { return min(max(v, 0), T); }

// What a tile makes of the state that enters it, as one 64-bit word that the tiles behind
// it read while it runs: (product, sum), or (CUT, state left behind) once that is known.
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
// of looks is bounded all the same: words or counters that something else writes to while
// the kernel runs give NaN or outputs that are not written, not a hang.  (A packed batch's
// marks and sequences, in the same workspace, are indexes, and are trusted.)
template <int n>
__device__ __forceinline__ void await_words(const uint64_t* own, int64_t step, int order, int back, int state,
                                            int lane, uint64_t (*look)[64]) {
    uint64_t word[n];
    for (int looks = 0;; ++looks) {
#pragma unroll
        for (int i = 0; i < n; ++i)
            word[i] = __hip_atomic_load(own - (1 + min(back + i * GS_WAVES, order - 1)) * step, __ATOMIC_RELAXED,
                                        __HIP_MEMORY_SCOPE_AGENT);
        bool ready = true;
#pragma unroll
        for (int i = 0; i < n; ++i)
            ready = ready && (back + i * GS_WAVES == state ? is_cut(word_prod(word[i]))
                                                          : (uint32_t)word[i] != (uint32_t)EMPTY);
        if (__all(ready)) break;
        if (looks == 1 << 20) {
#pragma unroll
            for (int i = 0; i < n; ++i) word[i] = 0x7fc00000ull << 32 | 0x80000000u;  // (NaN, cut off)
            break;
        }
        __builtin_amdgcn_s_sleep(1);
    }
#pragma unroll
    for (int i = 0; i < n; ++i) look[back + i * GS_WAVES][lane] = word[i];
}

// The state that enters tile `order` of a chain (0: `first`), whose own product and sum
// are (prod, sum) in the last wave.  The words of the eight tiles before this one are
// looked at first, one by each wave, and the oldest is waited for until it is a state; with
// few chains (far), where none of the eight is a state in all channels, those of the next
// 24, of which the oldest is waited for.  Folded from the oldest on, this is the same sum in
// the same order whatever each tile had posted by then: bits do not depend on time.  A tile
// waits only for tiles whose tickets were drawn before its own: those run already, and wait
// for earlier ones in turn.
constexpr int NEAR = GS_WAVES, FAR = 4 * GS_WAVES;

template <bool far>
__device__ __forceinline__ float enter_tile(const ScanArgs& a, int tiles, int order, int64_t column, bool active,
                                            int w, int lane, float prod, float sum, float first,
                                            uint64_t (*look)[64]) {
    const int64_t step = (int64_t)a.B * a.C;
    uint64_t* own = a.words + order * step + column;
    const bool poster = w == GS_WAVES - 1 && active;
    float in = first;
    if (order > 0) {
        if (poster) post(own, prod, sum);
        await_words<1>(own, step, order, w, far ? -1 : NEAR - 1, lane, look);
        __syncthreads();
        int from = min(order, NEAR) - 1;
        if (far && order > NEAR) {
            bool state = false;
#pragma unroll
            for (int j = 0; j < NEAR; ++j) state = state || is_cut(word_prod(look[j][lane]));
            if (!__all(state)) {  // (the same words in every wave)
                await_words<FAR / NEAR - 1>(own, step, order, w + NEAR, FAR - 1, lane, look);
                __syncthreads();
                from = min(order, FAR) - 1;
            }
        }
        in = 0.f;
        for (int j = from; j >= 0; --j) {
            const uint64_t t = look[j][lane];
            in = carry(word_prod(t), word_sum(t), in);
        }
    }
    if (poster && order + 1 < tiles) post(own, CUT, carry(prod, sum, in));
    return in;
}

// Of a packed batch, what a wave knows of its tokens: which begin a sequence, belong to
// one, end one.
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

// Rows of tokens from t0 on, one after the other: the offset in bytes of each from the
// head of a token tensor, the last row's again behind it.
struct RowWalk {
    int64_t at;
    int left;
    uint32_t stride;
    __device__ __forceinline__ RowWalk(const ScanArgs& a, int b, int t0, uint32_t row_bytes)
        : at(((int64_t)b * a.T + min(t0, a.T - 1)) * row_bytes), left(a.T - 1 - t0), stride(row_bytes) {}
    __device__ __forceinline__ void next() { at += left-- > 0 ? stride : 0u; }
};

// The same with a lane's channel, for stores and for the gradients' loads: offsets in bytes
// from `head`, which is the same for all lanes, so that an access takes one 32-bit addition
// for all tensors of a row (gradients of 16384 x 4096 bf16: 212 us; 219 for the stores
// alone, 226 without).  Loads of a packed batch are slower for it (15605 x 4096: 254 us, 230
// for the stores alone, 234 without), and the forward pass, whose loads the compiler spreads
// over the arithmetic to hold 64 registers, would spill.
struct Rows {
    int64_t head;
    int last;
    uint32_t stride, lane;
    __device__ __forceinline__ Rows(const ScanArgs& a, int b, int t0, uint32_t row_bytes, uint32_t lane_bytes)
        : head(((int64_t)b * a.T + min(t0, a.T - 1)) * row_bytes), last(max(a.T - 1 - t0, 0)), stride(row_bytes),
          lane(lane_bytes) {}
    __device__ __forceinline__ uint32_t at(int i) const {
        uint32_t o = lane + (uint32_t)min(i, last) * stride;
        asm volatile("" : "+v"(o));  // (or it would be made part of 64-bit sums, or kept)
        return o;
    }
};
// A channel of a token tensor: its bits, in a register of their own (held as 16 bits, the
// compiler puts two into one as they arrive, and waits for it: 8% slower), and its value.
template <class T>
__device__ __forceinline__ uint32_t load_bits(const void* p, int64_t head, uint32_t at) {
    const T v = *reinterpret_cast<const T*>(static_cast<const char*>(p) + head + at);
    if constexpr (sizeof(T) == 2) return v;
    else return __float_as_uint(v);
}
template <class T>
__device__ __forceinline__ float value(uint32_t bits) {
    return __uint_as_float(sizeof(T) == 2 ? bits << 16 : bits);
}
template <class T>
__device__ __forceinline__ void store_one(void* p, int64_t head, uint32_t at, float f) {
    T* to = reinterpret_cast<T*>(static_cast<char*>(p) + head + at);
    if constexpr (sizeof(T) == 2) *to = __builtin_bit_cast(uint16_t, (bf16)f);
    else *to = f;
}

}  // namespace

// What a pass needs before it: words that are empty and tickets that are not drawn; of a
// packed batch which sequence each token belongs to and which tokens begin and end one; and
// for the sequences without a token, the state behind them (dst = src, or zeros).
// Workgroups [0, fill) have the words, the next `marks` the tokens, the others a sequence
// each.
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

// The tile that this workgroup takes: of a chain (a row of the batch and a block of
// channels) the next in the order of time, by the chain's counter, so that the tiles that it
// waits for run already, whatever the order in which workgroups start.  Workgroups go to the
// chains one after the other, as many to each as it has tiles.  They also go to the XCDs one
// after the other: where the number of chains is a multiple of 8, the eight change places
// from one round to the next, or an XCD would read the same columns of every row, which
// share few of its L2's channels (131072 x 2048 454 us, 543 without; 32768 x 1024 66 and
// 76).  One counter for all chains deals them out well enough, but is a queue: 467 and 75
// us, and 2048 x 4096 32 us, not 22.
struct Place {
    uint32_t chain, order;
    // lds: a place for the ticket, written to only behind the next barrier
    __device__ __forceinline__ Place(const ScanArgs& a, uint32_t tiles, uint32_t chains, void* lds) {
        uint32_t* ticket = static_cast<uint32_t*>(lds);
        const uint32_t wg = blockIdx.z * gridDim.x + blockIdx.x;  // (fewer than 2^31 have a tile)
        order = wg / chains;
        chain = wg % chains;
        if (tiles == 1 || !is_tile(order, tiles)) return;
        if (chains % 8 == 0) chain = (chain & ~7u) + ((chain + order) & 7);
        if (threadIdx.x == 0) *ticket = atomicAdd(a.tickets + (int64_t)chain * TICKET_WORDS, 1u);
        __syncthreads();
        order = __builtin_amdgcn_readfirstlane(*ticket);
    }
};

// WAVES: 8, or 16 where that makes a row one tile (then nothing is posted).
template <class T, bool PACKED, bool far, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 8) void gated_scan_fwd_kernel(ScanArgs a) {
    constexpr int TILE = WAVES * FWD_STEPS;
    __shared__ float s_prod[WAVES][64], s_sum[WAVES][64];
    __shared__ uint64_t look[far ? FAR : NEAR][64];
    const int tiles = tiles_of(a.T, TILE);
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t blocks = (a.C + 63) / 64;
    const Place place(a, tiles, a.B * blocks, look);
    if (!is_tile(place.order, tiles)) return;
    const int k = place.order, b = place.chain / blocks, own = place.chain % blocks * 64 + lane;
    const bool active = own < a.C;
    const uint32_t c = active ? own : a.C - 1;
    const uint32_t row_bytes = a.C * (uint32_t)sizeof(T), lane_bytes = c * (uint32_t)sizeof(T);
    const int t0 = k * TILE + w * FWD_STEPS;
    uint32_t rx[FWD_STEPS], rg[FWD_STEPS], ri[FWD_STEPS];
    {
        RowWalk row(a, b, t0, row_bytes);
#pragma unroll
        for (int t = 0; t < FWD_STEPS; ++t, row.next()) {
            rx[t] = load_bits<T>(a.x, row.at, lane_bytes);
            rg[t] = load_bits<T>(a.g, row.at, lane_bytes);
            ri[t] = load_bits<T>(a.gate, row.at, lane_bytes);
        }
    }
    const float bias = a.dt_bias[c], amount = expf(a.A_log[c]);
    Marks m;
    if constexpr (PACKED) m = Marks(a, t0);
    // tokens that do not go on from the one before, and those behind the first such one
    const uint32_t fresh = PACKED ? m.start | ~m.in : 0u;
    const auto after_fresh = [&](int t) { return (fresh & ((2u << t) - 1)) != 0; };
    // the sequence of token t, which has one, and its state
    const auto sequence = [&](int t) { return (int64_t)(int)Marks::uniform(a.seq[t0 + t]); };
    const auto state_of = [&](const float* p, int t) { return p ? p[sequence(t) * a.C + c] : 0.f; };
    float prod[FWD_STEPS], sum[FWD_STEPS];
    float p = 1.f, h = 0.f;
    // (rows behind the last token of a batch of fixed length only follow: what is made of
    // them goes nowhere)
#pragma unroll
    for (int t = 0; t < FWD_STEPS; ++t) {
        const Decay d(value<T>(rg[t]) + bias, amount);
        const float in = __builtin_amdgcn_sqrtf(d.one_minus_square()) * sigmoid(value<T>(ri[t])) * value<T>(rx[t]);
        if (PACKED && fresh >> t & 1) {
            p = CUT;
            h = m.start >> t & 1 ? fmaf(d.a, state_of(a.h0, t), in) : 0.f;
        } else {
            p *= d.a;
            h = fmaf(d.a, h, in);
        }
        prod[t] = p;
        sum[t] = h;
    }
    // behind a fresh token nothing of the state before it is left, whatever it and the
    // decays are
    if (PACKED && after_fresh(FWD_STEPS - 1)) p = CUT;
    s_prod[w][lane] = p;
    s_sum[w][lane] = h;
    __syncthreads();
    // what the waves before this one make of the tile's state; the last wave's is the tile's
    float bp = 1.f, bs = 0.f;
    for (int j = 0; j < w; ++j) {
        bs = carry<PACKED>(s_prod[j][lane], s_sum[j][lane], bs);
        bp = join<PACKED>(s_prod[j][lane], bp);
    }
    const float first = k == 0 && !PACKED && a.h0 ? a.h0[(int64_t)b * a.C + c] : 0.f;
    float in = first;
    if constexpr (WAVES == GS_WAVES) {
            in = enter_tile<far>(a, tiles, k, (int64_t)b * a.C + c, active, w, lane, join(p, bp), carry(p, h, bs), first, look);
    }
    if (!active) return;
    const float enter = carry<PACKED>(bp, bs, in);
    float* states = a.states ? a.states + ((int64_t)b * a.n_states + t0 / GS_STATES) * a.C + c : nullptr;
    if (states && t0 < a.T) states[0] = enter;
    const Rows rows(a, b, t0, row_bytes, lane_bytes);
#pragma unroll
    for (int t = 0; t < FWD_STEPS; ++t) {
        if (t0 + t >= a.T) break;
        const float o = PACKED && after_fresh(t) ? sum[t] : fmaf(prod[t], enter, sum[t]);
        if (PACKED ? m.last >> t & 1 : t0 + t == a.T - 1) {
            if (a.h_final) a.h_final[(PACKED ? sequence(t) : (int64_t)b) * a.C + c] = o;
        }
        if (t == GS_STATES - 1 && states && t0 + GS_STATES < a.T) states[a.C] = o;
        store_one<T>(a.o, rows.head, rows.at(t), o);
    }
}

// A wave knows the state that enters its eight tokens, and so everything but the gradients
// that come back to them: what each gradient is of those is made ready before they are
// known, and there is little to do behind enter_tile.  A wave waits between its loads and
// its stores, so that many of them are needed: two of the factors wait in LDS, and the decays
// are formed again behind it, for 64 registers and four workgroups on a CU (16384 x 4096
// bf16, before Rows: 230 us; 246 with all factors in registers, three workgroups; 267 with
// the decays, too, two).  Looking far takes 12 KB more of LDS, and leaves three.
template <class T, bool PACKED, bool far>
__global__ __launch_bounds__(GS_THREADS, far ? 6 : 8) void gated_scan_bwd_kernel(ScanArgs a) {
    __shared__ float s_prod[GS_WAVES][64], s_sum[GS_WAVES][64];
    __shared__ uint64_t look[far ? FAR : NEAR][64];
    __shared__ float2 park[BWD_STEPS][GS_THREADS];
    const int tiles = tiles_of(a.T, BWD_TILE);
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t blocks = (a.C + 63) / 64;
    const Place place(a, tiles, a.B * blocks, look);
    if (!is_tile(place.order, tiles)) return;
    const int order = place.order, k = tiles - 1 - order;
    const int b = place.chain / blocks, own = place.chain % blocks * 64 + lane;
    const bool active = own < a.C;
    const uint32_t c = active ? own : a.C - 1;
    const uint32_t row_bytes = a.C * (uint32_t)sizeof(T), lane_bytes = c * (uint32_t)sizeof(T);
    const int t0 = k * BWD_TILE + w * BWD_STEPS;
    uint32_t rx[BWD_STEPS], rg[BWD_STEPS], ri[BWD_STEPS], rd[BWD_STEPS];
    const Rows rows(a, b, t0, row_bytes, lane_bytes);
    const auto load = [&](int t, int64_t row, uint32_t at) {
        rx[t] = load_bits<T>(a.x, row, at);
        rg[t] = load_bits<T>(a.g, row, at);
        ri[t] = load_bits<T>(a.gate, row, at);
        rd[t] = load_bits<T>(a.d_o, row, at);
    };
    RowWalk row(a, b, t0, row_bytes);
#pragma unroll
    for (int t = 0; t < BWD_STEPS; ++t, row.next()) {
        if constexpr (PACKED) load(t, row.at, lane_bytes);
        else load(t, rows.head, rows.at(t));
    }
    // (A bias of +infinity by a number: beside a gate of -infinity, below, it would be a NaN.
    // g + FLT_MAX forgets everything, too, but for a g of -FLT_MAX itself.)
    const float dt_bias = a.dt_bias[c], bias = dt_bias > FLT_MAX ? FLT_MAX : dt_bias;
    const float amount = expf(a.A_log[c]);
    // (tokens behind the last one have none, and need none)
    float h = a.states[((int64_t)b * a.n_states + min(t0 / GS_STATES, a.n_states - 1)) * a.C + c];
    Marks m;
    if constexpr (PACKED) m = Marks(a, t0);
    const uint32_t ended = PACKED ? m.last | ~m.in : 0u;  // nothing comes back from the token behind
    const auto sequence = [&](int t) { return (int64_t)(int)Marks::uniform(a.seq[t0 + t]); };
    const auto state_of = [&](const float* p, int t) { return p ? p[sequence(t) * a.C + c] : 0.f; };
    if constexpr (!PACKED) {
        // rows behind the last token: no decay (g = -infinity) and no gradient, so that
        // what comes back passes them
#pragma unroll
        for (int t = 0; t < BWD_STEPS; ++t) {
            if (t0 + t >= a.T) {
                rg[t] = sizeof(T) == 2 ? 0xff80u : 0xff800000u;
                rd[t] = 0;
            }
        }
    }
    // With e the gradient of h_t: dx = e fx, di = e fi, dL/dL_t = (a e) fp, and
    // dg = (a e) fp fg
    float dec[BWD_STEPS], L[BWD_STEPS], fp[BWD_STEPS], fg[BWD_STEPS];
#pragma unroll
    for (int t = 0; t < BWD_STEPS; ++t) {
        const float z = value<T>(rg[t]) + bias, x = value<T>(rx[t]);
        const Decay d(z, amount);
        const InputGate ig(value<T>(ri[t]));
        const float root = __builtin_amdgcn_sqrtf(d.one_minus_square());
        if (PACKED && (m.start >> t & 1)) h = state_of(a.h0, t);
        dec[t] = d.a;
        L[t] = d.L;
        const float fx = root * ig.s;
        park[t][threadIdx.x] = make_float2(fx, root * x * ig.slope);
        // (no decay at all: nothing of the input enters, and sigmoid(z) is zero)
        fp[t] = fmaf(d.a * ig.s * x, root == 0.f ? 0.f : __builtin_amdgcn_rcpf(root), -h);
        fg[t] = amount * d.sigmoid();
        h = fmaf(d.a, h, fx * x);
        // (here, and not where they are used: what they are made of would stay in registers)
        asm volatile("" : "+v"(fp[t]), "+v"(fg[t]));
    }
    // gradients of the states, from zero, last token first: what reaches the state before a
    // token is a (do + what reaches its own)
    float q = 1.f, e = 0.f;
#pragma unroll
    for (int t = BWD_STEPS - 1; t >= 0; --t) {
        if (PACKED && ended >> t & 1) {
            q = CUT;
            e = m.last >> t & 1 ? dec[t] * (value<T>(rd[t]) + state_of(a.d_final, t)) : 0.f;
        } else {
            q *= dec[t];
            e = dec[t] * (value<T>(rd[t]) + e);
        }
    }
    if (PACKED && (ended & ((1u << BWD_STEPS) - 1))) q = CUT;
    s_prod[w][lane] = q;
    s_sum[w][lane] = e;
    __syncthreads();
    // (the wave that posts a tile's word is the last: it folds all waves' gradients, the
    // others those behind them)
    float bp = 1.f, bs = 0.f;
    const int until = w == GS_WAVES - 1 ? 0 : w + 1;
    for (int j = GS_WAVES - 1; j >= until; --j) {
        bs = carry<PACKED>(s_prod[j][lane], s_sum[j][lane], bs);
        bp = join<PACKED>(s_prod[j][lane], bp);
    }
    const float first = order == 0 && !PACKED && a.d_final ? a.d_final[(int64_t)b * a.C + c] : 0.f;
    const float in = enter_tile<far>(a, tiles, order, (int64_t)b * a.C + c, active, w, lane, bp, bs, first, look);
    float back = in;
    if (w < GS_WAVES - 1) back = carry<PACKED>(bp, bs, in);
    else if (!PACKED && a.dh0 && k == 0 && active) a.dh0[(int64_t)b * a.C + c] = carry<PACKED>(bp, bs, in);
    float dA = 0.f, db = 0.f;
#pragma unroll
    for (int t = BWD_STEPS - 1; t >= 0; --t) {
        float dx = 0.f, dg = 0.f, di = 0.f;
        if (PACKED && m.last >> t & 1) back = state_of(a.d_final, t);
        if (!PACKED || m.in >> t & 1) {
            const float et = value<T>(rd[t]) + back;
            asm volatile("" : "+v"(L[t]));  // (or the decay of before would be kept)
            back = __builtin_amdgcn_exp2f(-L[t]) * et;
            const float pt = back * fp[t];
            const float2 f = park[t][threadIdx.x];
            dx = et * f.x;
            di = et * f.y;
            dg = pt * fg[t];
            // (A row behind the last token counts for nothing, however large what passes it.  An
            // L of infinity is a decay of zero: its part is zero, not 0 * inf.)
            if (PACKED || t0 + t < a.T) {
                dA = fmaf(pt, __builtin_amdgcn_fmed3f(L[t], 0.f, FLT_MAX), dA);
                db += dg;
            }
        }
        if (PACKED && a.dh0 && active && m.start >> t & 1) a.dh0[sequence(t) * a.C + c] = back;
        if (active && t0 + t < a.T) {
            const uint32_t at = rows.at(t);
            store_one<T>(a.dx, rows.head, at, dx);
            store_one<T>(a.dg, rows.head, at, dg);
            store_one<T>(a.dgate, rows.head, at, di);
        }
    }
    __syncthreads();
    s_prod[w][lane] = LN2 * dA;
    s_sum[w][lane] = db;
    __syncthreads();
    if (w < 2 && active) {
        float s = 0.f;
        for (int j = 0; j < GS_WAVES; ++j) s += w ? s_sum[j][lane] : s_prod[j][lane];
        a.part[(((int64_t)b * tiles + k) * 2 + w) * a.C + c] = s;
    }
}

// dA_log and ddt_bias from the tiles' sums: a workgroup for 32 channels of one of them
__global__ __launch_bounds__(256) void gated_scan_sum_kernel(ScanArgs a) {
    const int which = blockIdx.x % 2, c = blockIdx.x / 2 * 32 + threadIdx.x % 32;
    const double s = sum_columns(a.part + (int64_t)which * a.C + min(c, a.C - 1), (int64_t)a.B * tiles_of(a.T, BWD_TILE),
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
        const float in = __builtin_amdgcn_sqrtf(d.one_minus_square()) * sigmoid(i[v]) * x[v];
        o[v] = a.state_in ? fmaf(d.a, a.state_in[word * V + v], in) : in;
        a.state_out[word * V + v] = o[v];
    }
    static_cast<uint32_t*>(a.o)[word] = Word<T>::put(o);
}

namespace {

void launch_prepare(const ScanArgs& a, int tiles, int64_t chains, const float* src, float* dst, hipStream_t stream) {
    PrepareArgs q{};
    q.a = a;
    q.n_words = tiles > 1 ? (int64_t)tiles * a.B * a.C : 0;
    q.n_tickets = tiles > 1 ? chains : 0;
    q.fill = (q.n_words + 2047) / 2048;
    q.marks = a.cu ? ((int64_t)a.T + 255) / 256 : 0;
    q.src = src;
    q.dst = a.cu || a.T == 0 ? dst : nullptr;
    const int64_t groups = q.fill + q.marks + (q.dst ? a.N : 0);
    if (groups) hipLaunchKernelGGL(gated_scan_prepare_kernel, wide_grid(groups, 256), dim3(256), 0, stream, q);
}

// Few chains are short of tiles that can end, and a tile looks far; with more of them the
// words that it reads cost more (bf16, 131072 x 512, 8 chains: forward 138 us, 176 without,
// gradients 301 and 359; 65536 x 640, 10 chains: 89 and 103, 196 and 206; 32768 x 768, 12
// chains: 57 and 61, 123 and 118; 16384 x 1024: 39 and 38, 79 and 67).  All of these are
// rows of one length; packed batches go by the same number.
constexpr int64_t FAR_CHAINS = 10;

int64_t chains_of(const ScanArgs& a) { return (int64_t)a.B * ((a.C + 63) / 64); }

template <class F>
void by_type(bool fp32, bool packed, bool far, F&& f) {
    const auto with = [&](auto t) {
        const auto looks = [&](auto p) { far ? f(t, p, std::true_type{}) : f(t, p, std::false_type{}); };
        packed ? looks(std::true_type{}) : looks(std::false_type{});
    };
    fp32 ? with(float{}) : with(uint16_t{});
}

}  // namespace

void launch_gated_scan_fwd(const ScanArgs& a, bool fp32, hipStream_t stream) {
    // Rows of 129 to 256 tokens in one tile of sixteen waves need no words, and so no
    // launch before this one (256 tokens of 256 channels: 11.0 us a call, 15.6 in two tiles).
    const bool one = !a.cu && a.T > FWD_TILE && a.T <= GS_ONE_TILE;
    const int tiles = one ? 1 : tiles_of(a.T, FWD_TILE);
    const int64_t chains = chains_of(a);
    launch_prepare(a, tiles, chains, a.h0, a.h_final, stream);
    if (a.T == 0) return;
    by_type(fp32, a.cu != nullptr, !one && chains <= FAR_CHAINS, [&](auto t, auto packed, auto far) {
        using T = decltype(t);
        constexpr bool PACKED = decltype(packed)::value, LOOKS = decltype(far)::value;
        if constexpr (!PACKED && !LOOKS) {
            constexpr int WAVES = GS_ONE_TILE / FWD_STEPS;
            if (one) {
                hipLaunchKernelGGL((gated_scan_fwd_kernel<T, false, false, WAVES>), wide_grid(chains, 64 * WAVES),
                                   dim3(64 * WAVES), 0, stream, a);
                return;
            }
        }
        hipLaunchKernelGGL((gated_scan_fwd_kernel<T, PACKED, LOOKS, GS_WAVES>), wide_grid(chains * tiles, GS_THREADS),
                           dim3(GS_THREADS), 0, stream, a);
    });
}

void launch_gated_scan_bwd(const ScanArgs& a, bool fp32, hipStream_t stream) {
    const int tiles = tiles_of(a.T, BWD_TILE);
    const int64_t chains = chains_of(a);
    launch_prepare(a, tiles, chains, a.d_final, a.dh0, stream);
    if (a.T > 0) {
        by_type(fp32, a.cu != nullptr, chains <= FAR_CHAINS, [&](auto t, auto packed, auto far) {
            using T = decltype(t);
            hipLaunchKernelGGL((gated_scan_bwd_kernel<T, decltype(packed)::value, decltype(far)::value>),
                               wide_grid(chains * tiles, GS_THREADS), dim3(GS_THREADS), 0, stream, a);
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
