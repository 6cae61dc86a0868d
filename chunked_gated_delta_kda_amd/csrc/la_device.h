// la_device.h -- what the two chunked linear-attention kernels (la_chunk.hip,
// la_narrow.hip) share: segments, tiles in LDS and the order of instructions.
#pragma once

#include "kda_common.h"
#include "la_launch.h"

namespace kda {

namespace {

constexpr int LC = LA_CHUNK;

// the type's lowest log decay that matters: exp(-200) is zero in fp32 twice over
constexpr float LOG_DECAY_FLOOR = -200.f;

__device__ __forceinline__ float head_log_decay(const float* p, int h) {
    const float v = p[h];
    return v < LOG_DECAY_FLOOR ? LOG_DECAY_FLOOR : v;  // keeps a NaN
}

// a segment: tokens t0 .. t0 + len of sequence n, positions p0 .. p1
struct Seg {
    int n;
    int t0, len;
    int p0, p1;
};

__device__ __forceinline__ int clamp_tok(const LaSeqs& s, int v) { return min(max(v, 0), s.T); }

// The segment of a slot; false if the slot holds none.  Offsets are clamped
// to the batch, so an array that is not what it should be gives wrong
// results, never an access out of bounds.
__device__ __forceinline__ bool find_seg(const LaSeqs& s, int slot, Seg& g) {
    int seg;
    if (!s.cu) {
        g.n = slot / s.seg_per_seq;
        seg = slot % s.seg_per_seq;
        g.t0 = g.n * s.T;
        g.len = s.T;
    } else {
        int n = slot;
        seg = 0;
        if (s.by_length) {
            // whole sequences, at most 64: the longest first, so that none begins when
            // the others are done.  Lane i has sequence i, and counts those before it.
            const int lane = threadIdx.x & 63;
            const int i = min(lane, s.n_seqs - 1);
            const int len = lane < s.n_seqs ? max(clamp_tok(s, s.cu[i + 1]) - clamp_tok(s, s.cu[i]), 0) : -1;
            int before = 0;
            for (int j = 0; j < s.n_seqs; ++j) {
                const int other = __builtin_amdgcn_readlane(len, j);
                before += other > len || (other == len && j < lane);
            }
            n = min(__ffsll((unsigned long long)__ballot(lane < s.n_seqs && before == slot)) - 1, s.n_seqs - 1);
            n = max(n, 0);
        }
        if (s.seg_tokens) {
            // the last sequence whose first slot is not behind this one: 64
            // candidates at a time
            const int lane = threadIdx.x & 63;
            int lo = 0, cnt = s.n_seqs;
            for (;;) {
                const int step = (cnt + 63) / 64;
                const int i = lo + lane * step;
                const bool le = lane * step < cnt &&
                                clamp_tok(s, s.cu[min(i, s.n_seqs)]) / s.seg_tokens + i <= slot;
                const int k = __popcll(__ballot(le)) - 1;
                if (k < 0) return false;
                lo += k * step;
                if (step == 1) break;
                cnt = min(step, cnt - k * step);
            }
            n = lo;
            seg = slot - (clamp_tok(s, s.cu[n]) / s.seg_tokens + n);
        }
        g.n = n;
        g.t0 = clamp_tok(s, s.cu[n]);
        g.len = max(clamp_tok(s, s.cu[n + 1]) - g.t0, 0);
    }
    if (!s.seg_tokens) {
        g.p0 = 0;
        g.p1 = g.len;
        return true;
    }
    if (seg > 0 && (int64_t)seg * s.seg_tokens >= g.len) return false;
    g.p0 = seg * s.seg_tokens;
    g.p1 = g.p0 + min(g.len - g.p0, s.seg_tokens);
    return true;
}

// Operand that contracts over tokens: lane (r, g) receives rows 4 g .. 4 g + 3,
// column tile_channel(t, r) of 16 rows of an LDS tile, by one transposing read
// (ds_read_b64_tr_b16): in each group of 16 lanes, lane r fetches four
// consecutive columns of row 4 g + r / 4, those that lanes 4 (r % 4) .. + 3
// receive.
__device__ __forceinline__ bf16x4 read_t(const bf16* p) {
    typedef __attribute__((address_space(3))) short4_t* lds_short4;
    return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4)p));
}

// the two bf16 values of a word
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ bf16x8 join(bf16x4 a, bf16x4 b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Nothing is moved across by the compiler.
#define FENCE __builtin_amdgcn_sched_barrier(0)

// v is computed by here (the compiler places a computation at its use, else).
template <typename T>
__device__ __forceinline__ void pin(T& v) { asm volatile("" : "+v"(v)); }

// Waits until the products issued before are done (64 cycles).  The compiler
// keeps the wait states between a product and the first reader of its result,
// but not where the reader begins a block that other paths enter too: there it
// was seen to leave them out, and the reader took two registers of four too
// early.
__device__ __forceinline__ void settle() {
    FENCE;
    asm volatile("s_nop 15");
    FENCE;
}

// An x, y or z tile holds its rows of D columns without padding; 16-byte unit u of
// row m sits at unit u ^ swizzle(m).  Sixteen rows of one unit (the products that
// contract over channels) then lie in sixteen different units, and the four rows of
// a transposing read in four different 64-byte blocks.
template <int D>
__device__ __forceinline__ int swizzle(int m) {
    return D == 128 ? 4 * (m & 3) + ((m >> 2) & 3) : 4 * ((m >> 1) & 1) + ((m >> 2) & 3);
}

// Rows channel .. channel + 3 of a column of a state that enters (`row` elements
// apart; a transposed state's are neighbours).
__device__ __forceinline__ floatx4 load_state(const float* column, int channel, int row) {
    if (row == 1) return *reinterpret_cast<const floatx4*>(column + channel);
    floatx4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = column[(channel + i) * row];
    return v;
}

// The decay of a chunk, a^64, lies between two neighbouring floats: `below`, and the
// next, which is taken in a part `above` of the chunks.  So the product of any number
// of chunks' decays stays within a rounding of a power of a, where one float's own
// rounding would add up over thousands of chunks.
struct ChunkDecay {
    float below, above, carry;
    __device__ __forceinline__ explicit ChunkDecay(float ld) {
        const double whole = exp((double)ld * LC);
        below = (float)whole;
        if (below > whole) below = __uint_as_float(__float_as_uint(below) - 1);
        const float next = __uint_as_float(__float_as_uint(below) + 1);
        above = (float)((whole - below) / ((double)next - below));
        carry = 0.f;
    }
    __device__ __forceinline__ float step() {
        carry += above;
        const bool up = carry >= 1.f;
        if (up) carry -= 1.f;
        return __uint_as_float(__float_as_uint(below) + up);
    }
};

// Two decayed z as bf16 terms: eight bits of the 24 each, cut off, so that three add
// up to the value exactly (a rounding conversion issues at a quarter of the rate).
// Takes the next term off v0 and v1.
__device__ __forceinline__ uint32_t take_term(float& v0, float& v1) {
    const uint32_t term = __builtin_amdgcn_perm(__float_as_uint(v1), __float_as_uint(v0), 0x07060302u);
    v0 -= __uint_as_float(__float_as_uint(v0) & 0xffff0000u);
    v1 -= __uint_as_float(__float_as_uint(v1) & 0xffff0000u);
    return term;
}
// (the rounded product, not contracted into the differences: where la_chunk.hip takes
// three terms too, the two kernels give the same bits)
__device__ __forceinline__ float decayed(float z, float w) {
#pragma clang fp contract(off)
    return z * w;
}

}  // namespace

}  // namespace kda
