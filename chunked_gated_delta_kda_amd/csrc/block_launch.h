// block_launch.h -- host-side launch interface of what stands around an
// attention block (gated_scan.hip, short_conv.hip, layer_norm.hip) for the
// C-ABI layer (block_api.hip).  Pointers are device pointers; token tensors are
// bf16 or fp32, as the call's dtype says, everything else fp32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "la_launch.h"

namespace kda {

// The recurrence's tiles are 128 tokens of a row of the batch in the forward pass and 64
// in the backward pass; the forward pass keeps the state that enters every 8th token.
constexpr int GS_TILE = 64;
constexpr int GS_STATES = 8;
constexpr int GS_ONE_TILE = 256;  // most tokens of a row that the forward pass has as one tile
constexpr int GS_TICKET_BYTES = 64;  // counters do not share a line

// Whether a chain of so many tiles has one of this number, which is a counter's: compared
// without a sign, since a counter that something else wrote to may hold anything, and a
// negative tile would be read and written in front of every array.
__host__ __device__ constexpr bool is_tile(uint32_t number, int32_t tiles) { return number < (uint32_t)tiles; }

struct ScanArgs {
    const void* x;          // [B, T, C] tokens
    const void* g;          // [B, T, C] tokens
    const void* gate;       // [B, T, C] tokens
    const float* A_log;     // [C]
    const float* dt_bias;   // [C]
    const float* h0;        // [N, C] or null
    float* h_final;         // [N, C] or null
    const int32_t* cu;      // [N + 1] or null (fixed length, N = B)
    int32_t B, T, C, N;
    int32_t n_states;       // of a row of the batch
    void* o;                // [B, T, C] tokens
    float* states;          // [B, n_states, C] (forward: or null)
    // what the tiles of a chain post for those behind them, and counters of tiles taken
    // (neither is used where a row is one tile)
    uint64_t* words;        // [tiles, B, C]
    uint32_t* tickets;      // a counter for each chain, GS_TICKET_BYTES apart
    // packed batches: per 16 tokens, whether each begins a sequence,
    // belongs to one, ends one; per token, which
    uint2* marks;           // [ceil(T / 16)]
    int32_t* seq;           // [16 * ceil(T / 16)]
    // backward
    const void* d_o;        // [B, T, C] tokens
    const float* d_final;   // [N, C] or null
    void* dx;               // [B, T, C] tokens
    void* dg;
    void* dgate;
    float* dA_log;          // [C]
    float* ddt_bias;        // [C]
    float* dh0;             // [N, C] or null
    float* part;            // [B, tiles, 2, C]: a tile's sums for dA_log and ddt_bias
};

struct ScanDecodeArgs {
    const void* x;          // [N, C] tokens
    const void* g;
    const void* gate;
    const float* A_log;
    const float* dt_bias;
    const float* state_in;  // [N, C] or null (zeros)
    float* state_out;       // [N, C] (may equal state_in)
    void* o;
    int32_t N, C;
};

struct ConvArgs {
    const void* x;          // [B, T, C] tokens
    const float* weight;    // [C, W]
    const float* bias;      // [C] or null
    const void* h0;         // [N, W - 1, C] tokens or null
    void* h_final;          // [N, W - 1, C] tokens or null
    const int32_t* cu;
    int32_t B, T, C, N;
    int32_t silu;
    void* y;                // [B, T, C] tokens
    // backward
    const void* dy;
    const void* d_final;    // [N, W - 1, C] tokens or null
    void* dx;
    void* dh0;              // [N, W - 1, C] tokens or null
    float* dweight;         // [C, W]
    float* dbias;           // [C] or null
    float* part;            // [groups, W + 1, C]: a workgroup's sums
    uint32_t groups;        // workgroups of strips (of a block of channels), and a strip's tokens
    int32_t strip;
};

struct ConvDecodeArgs {
    const void* x;          // [N, C] tokens
    const float* weight;
    const float* bias;
    const void* state_in;   // [N, W - 1, C] tokens
    void* state_out;        // (may equal state_in)
    void* y;
    int32_t N, C;
    int32_t silu;
};

struct LayerNormArgs {
    const void* x;          // [rows, D] tokens (backward: the sum that was normalised)
    const void* res;        // [rows, D] tokens or null
    const float* weight;    // [D]
    const float* bias;      // [D] or null
    float eps;
    int32_t D;
    int64_t rows;
    void* y;                // [rows, D] tokens
    void* sum;              // [rows, D] tokens (with res)
    // backward
    const void* dy;
    const void* dsum;       // [rows, D] tokens or null
    void* dx;
    float* dweight;         // [D]
    float* dbias;           // [D] or null
    float* part;            // [groups, 2, D]
    int32_t groups;
};

// fp32: token tensors are fp32 (else bf16)
void launch_gated_scan_fwd(const ScanArgs& a, bool fp32, hipStream_t stream);
void launch_gated_scan_bwd(const ScanArgs& a, bool fp32, hipStream_t stream);
void launch_gated_scan_decode(const ScanDecodeArgs& a, bool fp32, hipStream_t stream);
// W: 2, 3 or 4 taps
void launch_short_conv_fwd(const ConvArgs& a, int W, bool fp32, hipStream_t stream);
void launch_short_conv_bwd(const ConvArgs& a, int W, bool fp32, hipStream_t stream);
void launch_short_conv_decode(const ConvDecodeArgs& a, int W, bool fp32, hipStream_t stream);
// rows of sums that the convolution's backward kernel leaves in part
int64_t short_conv_groups(int32_t B, int32_t T, int32_t C, bool fp32);
// most workgroups of its kernels (counted in 32 bits)
int64_t short_conv_workgroups(int32_t B, int32_t T, int32_t C, int32_t N);
void launch_layer_norm_fwd(const LayerNormArgs& a, bool fp32, hipStream_t stream);
void launch_layer_norm_bwd(const LayerNormArgs& a, bool fp32, hipStream_t stream);
// workgroups of the norm's backward kernel, each leaving a row of sums in part
int32_t layer_norm_groups(int64_t rows, int32_t D, bool fp32);

}  // namespace kda
