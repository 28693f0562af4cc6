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

// u of one call: given, or the momentum's.
struct Update {
    const void* g;      // u itself, or the gradient
    int g_bf16;
    const float* buf;   // momentum buffer, nullptr: u = g
    float momentum;
    int nesterov;
};

// Four values of u from element i on (those below `left`), and the new buffer's.
template <bool kVec>
__device__ __forceinline__ void read_u4(const Update& U, int64_t i, int left, float (&u)[4], float (&nb)[4])
{
    float g[4] = {0.0f, 0.0f, 0.0f, 0.0f}, b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (kVec) {
        if (left > 0) {
            if (U.g_bf16) {
                const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const bf16*>(U.g) + i);
                g[0] = __uint_as_float(q.x << 16), g[1] = __uint_as_float(q.x & 0xffff0000u);
                g[2] = __uint_as_float(q.y << 16), g[3] = __uint_as_float(q.y & 0xffff0000u);
            } else {
                Pack<float, 4> q;
                q.load(static_cast<const float*>(U.g) + i);
                q.get(g);
            }
            if (U.buf) {
                Pack<float, 4> q;
                q.load(U.buf + i);
                q.get(b);
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left) {
                g[e] = U.g_bf16 ? __bfloat162float(static_cast<const bf16*>(U.g)[i + e]) : static_cast<const float*>(U.g)[i + e];
                if (U.buf) b[e] = U.buf[i + e];
            }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        nb[e] = fmaf(U.momentum, b[e], g[e]);
        u[e] = U.buf == nullptr ? g[e] : U.nesterov ? fmaf(U.momentum, nb[e], g[e]) : nb[e];
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

// Scale of one matrix from its `parts` sums of squares, by a block of kMuonBlock threads.
__device__ __forceinline__ float start_scale(const float* part, int64_t parts, float eps, double* sums)
{
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < parts; i += kMuonBlock) s += part[i];
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = s;
    __syncthreads();
    s = sums[0];
    for (int w = 1; w < kMuonBlock / 32; ++w) s += sums[w];
    return static_cast<float>(static_cast<double>(kScale) / (sqrt(s) + static_cast<double>(eps)));
}

// Whether the matrices take the cluster path, and that path, once the sums of squares are on
// their way (`vec`: 16-byte accesses of the update).
bool muon_fits_cluster(int64_t batch, int64_t m, int64_t n);
cudaError_t muon_cluster(const MuonParams& M, const Update& U, const float* part, int64_t parts, bool vec,
                         cudaStream_t s);

}  // namespace so
