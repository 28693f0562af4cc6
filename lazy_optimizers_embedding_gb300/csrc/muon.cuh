// muon.cuh -- what the Newton-Schulz kernels share: the update's values, their
// split into f16 parts, and the interface between the general path (muon.cu) and the
// one for matrices that a cluster's shared memory holds (muon_small.cu).
#pragma once

#include <cuda_fp16.h>

#include "rowio.cuh"
#include "tensor.cuh"

namespace so {

constexpr float kScale = 16384.0f;              // 2^14: X, A and B are held times this
constexpr float kInvScale = 1.0f / 16384.0f;
constexpr int kMuonBlock = 256;

// Whether a Muon step takes place, a word of the workspace that one block settles for all (k_muon_norm
// clears it): the caller's error word may be set at any moment, by another stream that shares it, and a
// step that part of its blocks had left out would have moved the buffer without the weights, or
// half of either.
constexpr uint32_t kUndecided = 0, kGo = 1, kStop = 2;

// By one thread of a block.
__device__ __forceinline__ bool step_goes(uint32_t* verdict, const int32_t* d_err)
{
    const uint32_t mine = read_error(d_err) != 0 ? kStop : kGo;
    uint32_t v = ld_volatile(verdict);
    if (v == kUndecided) v = atomicCAS(verdict, kUndecided, mine);
    return (v == kUndecided ? mine : v) == kGo;
}

// u of one call: given, or the momentum's.
struct Update {
    const void* g;      // u itself, or the gradient
    int g_bf16;
    const float* buf;   // momentum buffer, nullptr: u = g
    float momentum;
    int nesterov;
};

// E values of u from element i on (E = 1, or 4 or 8 by 16-byte accesses, 8-byte ones of 4 bf16), and
// the new buffer's.
template <int E>
__device__ __forceinline__ void read_u(const Update& U, int64_t i, float (&u)[E], float (&nb)[E])
{
    float g[E], b[E];
    if (U.g_bf16) {
        const bf16* at = static_cast<const bf16*>(U.g) + i;
        if constexpr (E == 4) {
            const uint2 q = *reinterpret_cast<const uint2*>(at);
            g[0] = __uint_as_float(q.x << 16), g[1] = __uint_as_float(q.x & 0xffff0000u);
            g[2] = __uint_as_float(q.y << 16), g[3] = __uint_as_float(q.y & 0xffff0000u);
        } else {
            Pack<bf16, E> q;
            q.load(at);
            q.get(g);
        }
    } else {
        Pack<float, E> q;
        q.load(static_cast<const float*>(U.g) + i);
        q.get(g);
    }
    if (U.buf) {
        Pack<float, E> q;
        q.load(U.buf + i);
        q.get(b);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
        nb[e] = U.buf ? fmaf(U.momentum, b[e], g[e]) : 0.0f;
        u[e] = U.buf == nullptr ? g[e] : U.nesterov ? fmaf(U.momentum, nb[e], g[e]) : nb[e];
    }
}

// Four values of u from element i on, those below `left` (the others 0), and the new buffer's.
template <bool kVec>
__device__ __forceinline__ void read_u4(const Update& U, int64_t i, int left, float (&u)[4], float (&nb)[4])
{
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = nb[e] = 0.0f;
    if (kVec) {
        if (left > 0) read_u<4>(U, i, u, nb);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left) {
                float u1[1], b1[1];
                read_u<1>(U, i + e, u1, b1);
                u[e] = u1[0], nb[e] = b1[0];
            }
    }
}

// v as hi + lo f16, four at a time.
__device__ __forceinline__ void split4(__half* hi, __half* lo, const float (&v)[4])
{
    __half2 h[2], l[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        h[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        const float2 f = __half22float2(h[i]);
        l[i] = __floats2half2_rn(v[2 * i] - f.x, v[2 * i + 1] - f.y);
    }
    *reinterpret_cast<uint2*>(hi) = *reinterpret_cast<const uint2*>(h);
    if (lo) *reinterpret_cast<uint2*>(lo) = *reinterpret_cast<const uint2*>(l);
}

__device__ __forceinline__ void unpack8(uint4 a, float (&x)[8])
{
    const __half2* h = reinterpret_cast<const __half2*>(&a);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(h[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// Squares leave fp32 below about 1e-38, so a matrix whose squares sum to less than kSmallSquares (a norm
// below 2^-40) is summed again with its values times kRaise, which the smallest fp32 value's
// square survives too.
constexpr float kSmallSquares = 0x1p-80f;
constexpr float kRaise = 0x1p100f;

// The scale of one matrix from its `parts` sums of squares (x, and raised y where x is small), by a block of
// kThreads threads (`tmp`: 64 words).  Negative: of raised values, 2^14 / (|u| kRaise + eps kRaise), for x_of; a
// matrix of zeros has scale 0, whatever eps.  fp32: in fp64 the root and quotient alone held a block for 4 us.
template <int kThreads>
__device__ __forceinline__ float start_scale(const float2* part, int parts, float eps, float eps_raised, float* tmp)
{
    float s[2] = {0.0f, 0.0f};
    for (int i = threadIdx.x; i < parts; i += kThreads) {
        const float2 q = part[i];
        s[0] += q.x, s[1] += q.y;
    }
    block_sum<2>(s, kThreads, tmp, 0);
    const bool small = s[0] < kSmallSquares;   // both sums at once: a branch between two kept a block 2 us longer
    const float sum = small ? s[1] : s[0];
    return sum != 0.0f ? (small ? -kScale : kScale) / (sqrtf(sum) + (small ? eps_raised : eps)) : 0.0f;
}
// X's value of u.
__device__ __forceinline__ float x_of(float u, float scale) { return (scale < 0.0f ? u * -kRaise : u) * scale; }

// Whether the matrices take the cluster path, and that path, once the sums of squares are on
// their way (`vec`: 16-byte accesses of the update).
bool muon_fits_cluster(int64_t batch, int64_t m, int64_t n);
cudaError_t muon_cluster(const MuonParams& M, const Update& U, const float2* part, int parts, uint32_t* verdict,
                         bool vec, cudaStream_t s);

}  // namespace so
