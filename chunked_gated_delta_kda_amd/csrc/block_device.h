// block_device.h -- what the kernels around an attention block share: token
// types, the gate's functions and sums over rows of partial sums.
#pragma once

#include "block_launch.h"
#include "kda_common.h"

namespace kda {

namespace {

// One 4-byte word of a token tensor: two bf16 channels or one fp32 channel.
template <class T>
struct Word;
template <>
struct Word<uint16_t> {
    static constexpr int N = 2;
    static __device__ __forceinline__ void get(uint32_t w, float* f) {
        f[0] = __uint_as_float(w << 16);
        f[1] = __uint_as_float(w & 0xffff0000u);
    }
    static __device__ __forceinline__ uint32_t put(const float* f) {
        typedef __attribute__((ext_vector_type(2))) __bf16 pair;
        pair p;
        p[0] = (__bf16)f[0];
        p[1] = (__bf16)f[1];
        return __builtin_bit_cast(uint32_t, p);
    }
};
template <>
struct Word<float> {
    static constexpr int N = 1;
    static __device__ __forceinline__ void get(uint32_t w, float* f) { f[0] = __uint_as_float(w); }
    static __device__ __forceinline__ uint32_t put(const float* f) { return __float_as_uint(f[0]); }
};

// A sigmoid s = 1 / (1 + e^-z) as e^min(z, 0) / (1 + e^-|z|), to a few ulps where it is
// normal, and subnormal below z = -87: 2^t by the hardware is not, the square of 2^(t / 2)
// is.  `side` is s (1 - s).  For a NaN both are NaN.
struct BlockSigmoid {
    float s, side;
    __device__ __forceinline__ explicit BlockSigmoid(float z) {
        const float h = __builtin_amdgcn_exp2f(-0.5f * LOG2E * fabsf(z)), e = h * h;
        const float r = __builtin_amdgcn_rcpf(1.f + e), er = e * r;
        s = z < 0.f ? er : r;
        side = er * r;
    }
};

// adds b values at a time to s, while there are any (all: while there are b)
template <int b, bool all>
__device__ __forceinline__ void add_batches(const float* p, int64_t& i, int64_t n, int64_t step, double& s) {
    for (; all ? i + b <= n : i < n; i += b) {
        float v[b];
#pragma unroll
        for (int k = 0; k < b; ++k) v[k] = p[(all || i + k < n ? i + k : n - 1) * step];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < b; ++k) s += all || i + k < n ? v[k] : 0.f;
    }
}

// sum of n values, `step` apart: 32 loads in flight at a time, 4 where fewer are left (the
// convolution's gradients of 2 x 2048 x 4096 end with sums over 32 rows, 4 for a thread: a
// call took 30.9 us with 32 loads there, too, and 28.7 with these)
__device__ __forceinline__ double sum_strided(const float* p, int64_t n, int64_t step) {
    double s = 0.0;
    int64_t i = 0;
    add_batches<32, true>(p, i, n, step, s);
    add_batches<4, false>(p, i, n, step, s);
    return s;
}

// A workgroup of 256 threads adds 32 columns of n rows, `step` apart, in a fixed order and
// in 64 bits: thread i has column i % 32 (where p points) and every 8th row.  Returns the
// sum of the thread's column.  (512 threads: the same to 1%.)
__device__ __forceinline__ double sum_columns(const float* p, int64_t n, int64_t step) {
    __shared__ double red[8][32];
    const int col = threadIdx.x % 32, first = threadIdx.x / 32;
    red[first][col] = sum_strided(p + first * step, (n - first + 7) / 8, 8 * step);
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += red[i][col];
    return s;
}

// the sum of both of v's lanes in each pair of lanes that differ in bit `m` (a power of
// two), where the lower bits' sums are done
template <int m>
__device__ __forceinline__ float add_across(float v) {
    const int w = __float_as_int(v);
    if constexpr (m == 1) return v + __int_as_float(__builtin_amdgcn_update_dpp(0, w, 0xB1, 0xf, 0xf, true));
    else if constexpr (m == 2) return v + __int_as_float(__builtin_amdgcn_update_dpp(0, w, 0x4E, 0xf, 0xf, true));
    else if constexpr (m == 4) return v + __int_as_float(__builtin_amdgcn_update_dpp(0, w, 0x141, 0xf, 0xf, true));
    else if constexpr (m == 8) return v + __int_as_float(__builtin_amdgcn_update_dpp(0, w, 0x140, 0xf, 0xf, true));
    else if constexpr (m == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(w, w, false, false);
        return __int_as_float(r[0]) + __int_as_float(r[1]);
    } else {
        const auto r = __builtin_amdgcn_permlane32_swap(w, w, false, false);
        return __int_as_float(r[0]) + __int_as_float(r[1]);
    }
}

// the sum over L lanes that stand together, in each of them
template <int L>
__device__ __forceinline__ float lane_sum(float v) {
    if constexpr (L > 1) v = add_across<1>(v);
    if constexpr (L > 2) v = add_across<2>(v);
    if constexpr (L > 4) v = add_across<4>(v);
    if constexpr (L > 8) v = add_across<8>(v);
    if constexpr (L > 16) v = add_across<16>(v);
    if constexpr (L > 32) v = add_across<32>(v);
    return v;
}

// R words of a token row (4, 8 or 16 bytes): 2 R bf16 channels or R fp32 channels
template <class T, int R = 4>
struct Slice {
    static constexpr int W = Word<T>::N, N = R * W;
    typedef __attribute__((ext_vector_type(R))) unsigned int raw;
    static __device__ __forceinline__ raw load(const void* p, int64_t at) {
        return *reinterpret_cast<const raw*>(static_cast<const T*>(p) + at);
    }
    static __device__ __forceinline__ void load(const void* p, int64_t at, float* f) { unpack(load(p, at), f); }
    static __device__ __forceinline__ void unpack(raw v, float* f) {
#pragma unroll
        for (int i = 0; i < R; ++i) Word<T>::get(v[i], f + W * i);
    }
    static __device__ __forceinline__ void store(void* p, int64_t at, const float* f) {
        raw v;
#pragma unroll
        for (int i = 0; i < R; ++i) v[i] = Word<T>::put(f + W * i);
        *reinterpret_cast<raw*>(static_cast<T*>(p) + at) = v;
    }
    // f as it is when stored
    static __device__ __forceinline__ void round(const float* f, float* r) {
#pragma unroll
        for (int i = 0; i < R; ++i) Word<T>::get(Word<T>::put(f + W * i), r + W * i);
    }
};

}  // namespace

}  // namespace kda
