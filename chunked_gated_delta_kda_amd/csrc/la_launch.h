// la_launch.h -- host-side launch interface of the linear-attention and gated
// norm kernels (la_chunk.hip, la_decode.hip, gated_norm.hip) for the C-ABI
// layer (la_api.hip).  Pointers are device pointers; bf16 tensors are passed
// as uint16_t bit patterns.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

constexpr int LA_CHUNK = 64;  // tokens per chunk

// A grid of at least `groups` workgroups of `threads` threads over x and z, y as given:
// HIP launches fewer than 2^32 work items in a dimension, and a grid beyond that was
// seen to wrap without an error.  Workgroup z * gridDim.x + x; those from `groups` on
// have no work.
inline dim3 wide_grid(int64_t groups, int threads, unsigned y = 1) {
    const int64_t most = ((int64_t)1 << 31) / threads;
    const int64_t z = (groups + most - 1) / most;
    return dim3((unsigned)((groups + z - 1) / z), y, (unsigned)z);
}

// One chunked pass over the tokens of a batch (la_chunk.hip):
//   O_p = x_scale a^(p+1-late) S_in^T x_p + in_scale sum_{j<=p} a^(p-j) (x_p . y_j) z_j
//   S_out = a^n S_in + z_scale sum_j a^(n-1-j+late) y_j z_j^T
// over the positions p of a segment, with S [D1, D2].  The forward pass and
// the three gradients are passes of this form (late = 1 where it runs in
// reverse).
struct LaPass {
    const uint16_t* x;     // [tokens, H, D1] bf16 (null for a pass over states only)
    const uint16_t* y;     // [tokens, H, D1] bf16
    const uint16_t* z;     // [tokens, H, D2] bf16
    uint16_t* o;           // [tokens, H, D2] bf16 (null for a pass over states only)
    const float* s_in;     // entering states, fp32, or null (zeros)
    float* s_out;          // states left behind, fp32, or null (not written)
    int32_t s_in_slots;    // s_in holds one state per segment slot (else per sequence)
    int32_t s_out_slots;   // s_out: one per slot, of all segments but a sequence's last
                           // (else one per sequence, of its last segment)
    int32_t D1, D2;        // 64 or 128 each
    int32_t row, col;      // element (d1, d2) of a state sits at row * d1 + col * d2
    int32_t reverse;       // positions run from the last token to the first, late = 1
    float in_scale, x_scale, z_scale;
};

// Sequences and segments.  Fixed length: sequence n is tokens [n T, (n+1) T),
// in seg_per_seq segments, slot n seg_per_seq + s.  Packed: sequence n is
// tokens [cu[n], cu[n+1]), its segment s is slot cu[n] / seg_tokens + n + s
// (distinct for all sequences, since floor(a + b) >= floor(a) + ceil(b) - 1);
// whole sequences (seg_tokens 0): slot n.
struct LaSeqs {
    const int32_t* cu;     // null: fixed length
    int32_t n_seqs;
    int32_t T;             // tokens of a sequence (fixed) or of the batch (packed)
    int32_t H;
    int32_t seg_tokens;    // positions per segment (a multiple of LA_CHUNK), 0: whole
    int32_t seg_per_seq;   // fixed length only
    int32_t n_slots;
    int32_t by_length;     // packed whole sequences: slot i is the i-th longest
};

struct LaArgs {
    LaPass pass[3];
    LaSeqs s;
    const float* log_decay;  // [H] fp32
};

struct LaScanArgs {
    LaSeqs s;
    const float* log_decay;
    const float* init[2];  // [n_seqs, H, elems] or null: the state entering a sequence
    float* state[2];       // [n_slots, H, elems]: in, what each segment adds to a zero
                           // state (not read for the last); out, the state entering it
    int32_t elems;         // K * V
    int32_t n_dirs;
};

struct LaDecodeArgs {
    const uint16_t* q;         // [pairs, K] bf16 (pairs = N * H, head fastest)
    const uint16_t* k;         // [pairs, K] bf16
    const uint16_t* v;         // [pairs, V] bf16
    const float* log_decay;    // [H] fp32
    const float* state_in;     // [pairs, K, V] fp32 or null (zeros)
    float* state_out;          // [pairs, K, V] fp32 (may equal state_in)
    uint16_t* o;               // [pairs, V] bf16
    float scale;
    int32_t H;
    int32_t V;
    int32_t n_pairs;
};

struct GatedNormArgs {
    const uint16_t* x;         // [rows, D] bf16 (rows = tokens * H, head fastest)
    const uint16_t* gate;      // [rows, D] bf16 or null (no gate)
    const float* weight;       // [D] fp32
    const uint16_t* res;       // [rows, D] bf16 or null
    const float* res_scale;    // [H] fp32 or null (no residual)
    float eps;
    int32_t silu;              // the gate's activation: silu (1) or sigmoid (0)
    int32_t H;
    int32_t D;
    int64_t rows;
    uint16_t* y;               // forward: [rows, D]
    const uint16_t* dy;        // backward from here on: [rows, D]
    uint16_t* dx;              // [rows, D]
    uint16_t* dgate;           // [rows, D] (with gate)
    uint16_t* dres;            // [rows, D] (with res)
    float* dweight;            // [D]
    float* dres_scale;         // [H] (with res)
    float* part_w;             // [groups, D]: a workgroup's sums for dweight
    float* row_ds;             // [rows]: a row's sum for dres_scale (with res)
    int32_t groups;
};

// Passes [0, n) of a, of one D1 x D2, or of both 64 x 128 and 128 x 64; states: no
// outputs (x and o null), one D1 x D2.
void launch_la_chunk(const LaArgs& a, int n, bool states, hipStream_t stream);
// The same for whole sequences, in workgroups of a few columns (la_narrow.hip).
void launch_la_narrow(const LaArgs& a, int n, hipStream_t stream);
// workgroups of a pass there
int64_t la_narrow_groups(int64_t pairs, int cols);
void launch_la_scan(const LaScanArgs& a, hipStream_t stream);
void launch_la_decode(const LaDecodeArgs& a, int K, hipStream_t stream);
void launch_gated_norm_fwd(const GatedNormArgs& a, hipStream_t stream);
void launch_gated_norm_bwd(const GatedNormArgs& a, hipStream_t stream);
// workgroups of the backward kernel, each leaving one [D] row in part_w
int32_t gated_norm_groups(int64_t rows, int32_t D);

}  // namespace kda
