// la_decode.hip -- one step of linear attention with a decay for each head per
// sequence (gfx950): the single-token form of la_chunk.hip's recurrence,
//   S' = a S + k v^T,   o = scale S'^T q,   a = exp(log_decay[h]).
//
// Bound by HBM: the state is read and written once (8 K V bytes a pair): 64
// sequences of 32 heads of 128 x 128 (268 MB) take 52 us, 5.1 TB/s.  One
// workgroup per (sequence, head, 64 value columns); thread (rg, cq) owns rows
// RPT rg .. RPT rg + RPT - 1 and columns 4 cq .. 4 cq + 3 of the block, so a
// row of the block is 16 threads x 16 bytes.  The sum over rows for o goes
// through LDS.  The decay is applied as S + (a - 1) S where a is near one: the
// rounding of a would add up over the tokens.
#include "kda_common.h"
#include "la_launch.h"

namespace kda {

namespace {

constexpr int LD_COLS = 64;
constexpr int LD_CQ = LD_COLS / 4;
constexpr int LD_THREADS = 256;
constexpr int LD_RG = LD_THREADS / LD_CQ;

}  // namespace

template <int K>
__global__ __launch_bounds__(LD_THREADS) void la_decode_kernel(LaDecodeArgs a) {
    constexpr int RPT = K / LD_RG;
    __shared__ floatx4 red[LD_RG][LD_CQ];
    const int vb = a.V / LD_COLS;
    const uint32_t wg = blockIdx.z * gridDim.x + blockIdx.x;
    if (wg / vb >= (uint32_t)a.n_pairs) return;
    const int pair = wg / vb, h = pair % a.H;
    const int tid = threadIdx.x, cq = tid % LD_CQ, rg = tid / LD_CQ;
    const int r0 = RPT * rg, c0 = (int)(wg % vb) * LD_COLS + 4 * cq;
    const int64_t base = (int64_t)pair * K * a.V + (int64_t)r0 * a.V + c0;

    floatx4 S[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i)
        S[i] = a.state_in ? *reinterpret_cast<const floatx4*>(a.state_in + base + (int64_t)i * a.V)
                          : floatx4{0.f, 0.f, 0.f, 0.f};
    const float raw = a.log_decay[h];
    const float ld = raw < -200.f ? -200.f : raw;  // keeps a NaN
    const bool near = ld > -0.6f;
    const float s0 = near ? 1.f : 0.f, s1 = near ? expm1f(ld) : expf(ld);
    const bf16x4 vb4 = *reinterpret_cast<const bf16x4*>(a.v + (int64_t)pair * a.V + c0);
    const bf16* q = reinterpret_cast<const bf16*>(a.q) + (int64_t)pair * K + r0;
    const bf16* k = reinterpret_cast<const bf16*>(a.k) + (int64_t)pair * K + r0;

    floatx4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const float kv = (float)k[i], qv = (float)q[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            S[i][e] = fmaf(S[i][e], s1, S[i][e] * s0) + kv * (float)vb4[e];
            o[e] = fmaf(S[i][e], qv, o[e]);
        }
        *reinterpret_cast<floatx4*>(a.state_out + base + (int64_t)i * a.V) = S[i];
    }
    red[rg][cq] = o;
    __syncthreads();
    if (rg == 0) {
#pragma unroll
        for (int j = 1; j < LD_RG; ++j) o += red[j][cq];
        *reinterpret_cast<bf16x4*>(a.o + (int64_t)pair * a.V + c0) = to_bf16x4(o * a.scale);
    }
}

void launch_la_decode(const LaDecodeArgs& a, int K, hipStream_t stream) {
    const dim3 grid = wide_grid((int64_t)a.n_pairs * (a.V / LD_COLS), LD_THREADS);
    if (K == 128) hipLaunchKernelGGL((la_decode_kernel<128>), grid, dim3(LD_THREADS), 0, stream, a);
    else hipLaunchKernelGGL((la_decode_kernel<64>), grid, dim3(LD_THREADS), 0, stream, a);
}

}  // namespace kda
