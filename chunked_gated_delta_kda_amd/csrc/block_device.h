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

// A sigmoid 1 / (1 + e^-z) as e^min(z, 0) / (1 + e^-|z|): to a few ulps where it is
// normal, and subnormal below z = -87.  `rest` is 1 - s.
struct BlockSigmoid {
    float s, rest;
    __device__ __forceinline__ explicit BlockSigmoid(float z) {
        const float e = expf(-fabsf(z)), r = 1.f / (1.f + e);
        s = z < 0.f ? e * r : r;
        rest = z < 0.f ? r : e * r;
    }
};

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

// A workgroup of 256 threads adds 8 columns of n rows, `step` apart, in a fixed order and
// in 64 bits: thread i has column i % 8 (where p points) and every 32nd row; threads 0 to
// 7 return the sums.
__device__ __forceinline__ double sum_columns(const float* p, int64_t n, int64_t step) {
    __shared__ double red[256];
    const int tid = threadIdx.x, first = tid / 8;
    red[tid] = sum_strided(p + first * step, (n - first + 31) / 32, 32 * step);
    __syncthreads();
    for (int m = 128; m >= 8; m >>= 1) {
        if (tid < m) red[tid] += red[tid + m];
        __syncthreads();
    }
    return red[tid % 8];
}

// 16 bytes of a token tensor: eight bf16 channels or four fp32 channels
template <class T>
struct Slice {
    static constexpr int W = Word<T>::N, N = 4 * W;
    static __device__ __forceinline__ void load(const void* p, int64_t at, float* f) {
        unpack(*reinterpret_cast<const u32x4*>(static_cast<const T*>(p) + at), f);
    }
    static __device__ __forceinline__ void unpack(u32x4 v, float* f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) Word<T>::get(v[i], f + W * i);
    }
    static __device__ __forceinline__ void store(void* p, int64_t at, const float* f) {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = Word<T>::put(f + W * i);
        *reinterpret_cast<u32x4*>(static_cast<T*>(p) + at) = v;
    }
    // f as it is when stored
    static __device__ __forceinline__ void round(const float* f, float* r) {
#pragma unroll
        for (int i = 0; i < 4; ++i) Word<T>::get(Word<T>::put(f + W * i), r + W * i);
    }
};

}  // namespace

}  // namespace kda
