// rowio.cuh -- a lane's share of a row of fp32 or bf16 values, held as read
// (packed) until it is used, and the sums over lanes and blocks.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace so {

using bf16 = __nv_bfloat16;

// Two fp32 values worked on by one instruction.
struct F2 {
    uint64_t q;
    __device__ __forceinline__ static F2 of(float lo, float hi)
    {
        F2 r;
        asm("mov.b64 %0, {%1, %2};" : "=l"(r.q) : "f"(lo), "f"(hi));
        return r;
    }
    __device__ __forceinline__ static F2 both(float a) { return of(a, a); }
    __device__ __forceinline__ float lo() const
    {
        return __uint_as_float(static_cast<uint32_t>(q));
    }
    __device__ __forceinline__ float hi() const
    {
        return __uint_as_float(static_cast<uint32_t>(q >> 32));
    }
    __device__ __forceinline__ float sum() const { return lo() + hi(); }
};
__device__ __forceinline__ F2 operator+(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.q) : "l"(a.q), "l"(b.q));
    return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.q) : "l"(a.q), "l"(b.q));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.q) : "l"(a.q), "l"(b.q), "l"(c.q));
    return r;
}

// V consecutive values as they lie in memory.  V = 1 reads any element; V > 1
// needs the address aligned to min(16, V * sizeof) bytes.
template <class T, int V> struct Pack;

template <> struct Pack<float, 1> {
    float a;
    __device__ __forceinline__ void load(const float* p) { a = *p; }
    __device__ __forceinline__ void zero() { a = 0.0f; }
    __device__ __forceinline__ void get(float (&x)[1]) const { x[0] = a; }
    __device__ __forceinline__ static void put(float* p, const float (&x)[1]) { *p = x[0]; }
};
template <> struct Pack<float, 2> {
    float2 a;
    __device__ __forceinline__ void load(const float* p) { a = *reinterpret_cast<const float2*>(p); }
    __device__ __forceinline__ void zero() { a = make_float2(0.0f, 0.0f); }
    __device__ __forceinline__ void get(float (&x)[2]) const { x[0] = a.x, x[1] = a.y; }
    __device__ __forceinline__ static void put(float* p, const float (&x)[2]) { *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]); }
};
template <> struct Pack<float, 4> {
    float4 a;
    __device__ __forceinline__ void load(const float* p) { a = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void zero() { a = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    __device__ __forceinline__ void get(float (&x)[4]) const { x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w; }
    __device__ __forceinline__ static void put(float* p, const float (&x)[4])
    {
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    }
};
template <> struct Pack<float, 8> {
    Pack<float, 4> lo, hi;
    __device__ __forceinline__ void load(const float* p) { lo.load(p), hi.load(p + 4); }
    __device__ __forceinline__ void zero() { lo.zero(), hi.zero(); }
    __device__ __forceinline__ void get(float (&x)[8]) const
    {
        x[0] = lo.a.x, x[1] = lo.a.y, x[2] = lo.a.z, x[3] = lo.a.w;
        x[4] = hi.a.x, x[5] = hi.a.y, x[6] = hi.a.z, x[7] = hi.a.w;
    }
    __device__ __forceinline__ static void put(float* p, const float (&x)[8])
    {
        reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
};
template <> struct Pack<bf16, 1> {
    bf16 a;
    __device__ __forceinline__ void load(const bf16* p) { a = *p; }
    __device__ __forceinline__ void zero() { a = __float2bfloat16_rn(0.0f); }
    __device__ __forceinline__ void get(float (&x)[1]) const { x[0] = __bfloat162float(a); }
    __device__ __forceinline__ static void put(bf16* p, const float (&x)[1]) { *p = __float2bfloat16_rn(x[0]); }
};
template <> struct Pack<bf16, 2> {
    uint32_t a;
    __device__ __forceinline__ void load(const bf16* p) { a = *reinterpret_cast<const uint32_t*>(p); }
    __device__ __forceinline__ void zero() { a = 0u; }
    __device__ __forceinline__ void get(float (&x)[2]) const { x[0] = __uint_as_float(a << 16), x[1] = __uint_as_float(a & 0xffff0000u); }
    __device__ __forceinline__ static void put(bf16* p, const float (&x)[2]) { *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x[0], x[1]); }
};
template <> struct Pack<bf16, 8> {
    uint4 a;
    __device__ __forceinline__ void load(const bf16* p) { a = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float (&x)[8]) const
    {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ static void put(bf16* p, const float (&x)[8])
    {
        uint4 a;
        uint32_t* w = reinterpret_cast<uint32_t*>(&a);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 q = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&q);
        }
        *reinterpret_cast<uint4*>(p) = a;
    }
};

// Sums of N values over a group of G lanes (a power of two, 1 to 32), by butterflies.
template <int N>
__device__ __forceinline__ void lanes_sum(float (&x)[N], int G)
{
    if (G == 32) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(kFull, x[i], d);
    } else {
        for (int d = G >> 1; d > 0; d >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(kFull, x[i], d);
    }
}

// Sums of N values over a block of `threads` threads (a power of two).  By butterflies: within a warp,
// then over the warps' sums in `tmp` (2 * 32 * N words, the half `half` used by turns: the
// barrier of the next call is what frees it), so every lane holds the same bits.  (The
// warps' sums one after the other took 0.2 us more for 8 warps.)
template <int N>
__device__ __forceinline__ void block_sum(float (&x)[N], int threads, float* tmp, int half)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(kFull, x[i], d);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = threads >> 5;
    float* t = tmp + half * 32 * N;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) t[i * 32 + warp] = x[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = t[i * 32 + (lane & (warps - 1))];
    for (int d = warps >> 1; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(kFull, x[i], d);
}

}  // namespace so
