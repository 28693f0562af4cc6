// route.cu -- the k experts of every token from its scores, and the scores' gradient.
//
// A warp has a token's row in registers, up to 32 scores a lane.  Most of them never come near: the k-th
// largest of the lanes' own largest (different ones) is a bound from below, and the few that reach it (8 of
// 256: 10 on the average) go to a lane each by way of shared memory, which counts those that stand before its
// own: larger ones, and equals of a lower index.  (131072 rows of 256, 8 picks, are bound by instructions: k rounds of a
// maximum over all scores 99 us; bitonic sorts of the lanes' largest and of the candidates 64 us; the least of 8 groups of lanes
// as the bound, which 19 reach, 66 us.)  Where more than 32 reach the bound, equals most of them, k rounds over all
// scores remain.  Softmax sums are fp32.
#include <algorithm>
#include <cfloat>

#include "profile.cuh"
#include "rowio.cuh"

namespace so {

namespace {

constexpr int kRouteBlock = 256;

__device__ __forceinline__ float warp_max(float x)
{
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float exp_of(float x)   // of the terms of a sum
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}

// Where a lane's value v lies in the row: accesses of W values by neighbouring lanes.
template <int W>
__device__ __forceinline__ int index_of(int v, int lane) { return v / W * 32 * W + lane * W + v % W; }

template <class T, int V, int W>
__device__ __forceinline__ void read_row(const T* row, int experts, int lane, float (&x)[V])
{
#pragma unroll
    for (int v = 0; v < V; v += W) {
        const int i = index_of<W>(v, lane);
        float y[W];
        if (i < experts) {
            Pack<T, W> q;
            q.load(row + i);
            q.get(y);
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e) y[e] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < W; ++e) x[v + e] = y[e];
    }
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(kFull, x, d);
    return x;
}

// A score and its index as one whole number: larger scores above smaller ones, -0 as 0, of equals the lower index above.
__device__ __forceinline__ uint64_t key_of(float x, int index)
{
    const uint32_t u = __float_as_uint(x + 0.0f);
    return static_cast<uint64_t>(u & 0x80000000u ? ~u : u | 0x80000000u) << 32 | ~static_cast<uint32_t>(index);
}

// A lane's largest score, NaN where there is one.
template <int V>
__device__ __forceinline__ float lane_max(const float (&x)[V])
{
    float m = x[0];
#pragma unroll
    for (int v = 1; v < V; ++v) asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(m), "f"(x[v]));
    return m;
}

template <class T, int V, int W>
__global__ void __launch_bounds__(kRouteBlock) k_route(const T* __restrict__ logits, int64_t n, int experts, int k, int renormalize,
                                                       int64_t* __restrict__ expert, float* __restrict__ weights, int32_t* d_err)
{
    pdl_wait();
    __shared__ uint64_t near[kRouteBlock / 32][32];   // a row's candidates
    const int lane = threadIdx.x & 31;
    uint64_t* mine = near[threadIdx.x >> 5];
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kRouteBlock / 32);
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * (kRouteBlock / 32) + (threadIdx.x >> 5); row < n; row += step) {
        float x[V];
        read_row<T, V, W>(logits + row * experts, experts, lane, x);
        const float best = lane_max(x);
        const bool odd = __any_sync(kFull, !(best < INFINITY));
        if (odd && lane == 0) set_error(d_err, SPARSE_ERR_NON_FINITE);
        int count = 0, place = 32, at = -1;   // candidates; which pick this lane's is, and its index
        float high = -INFINITY, pick = -INFINITY;
        if (!odd) {
            float bound = best, left = best;
            for (int j = 0; j < k; ++j) {
                bound = warp_max(left);
                if (j == 0) high = bound;
                if (left == bound) left = -INFINITY;
            }
            bound = fmaxf(bound, -FLT_MAX);   // -inf is no candidate
            int own = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) own += x[v] >= bound ? 1 : 0;
            int to = own;
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const int y = __shfl_up_sync(kFull, to, s);
                if (lane >= s) to += y;
            }
            count = __shfl_sync(kFull, to, 31);
            to -= own;
            if (count <= 32) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (x[v] >= bound) mine[to++] = static_cast<uint64_t>(__float_as_uint(x[v])) << 32 | static_cast<uint32_t>(index_of<W>(v, lane));
                __syncwarp();
                const uint64_t raw = lane < count ? mine[lane] : 0u;
                const uint64_t key = key_of(__uint_as_float(static_cast<uint32_t>(raw >> 32)), static_cast<int>(raw));
                mine[lane] = key;
                __syncwarp();
                int before = 0;
#pragma unroll 4
                for (int c = 0; c < count; ++c) before += mine[c] > key ? 1 : 0;
                if (lane < count && before < k) {
                    pick = __uint_as_float(static_cast<uint32_t>(raw >> 32));
                    at = static_cast<int>(raw);
                    place = before;
                }
                __syncwarp();
            }
        }
        if (count > 32) {                                     // many equals
            float y[V];
#pragma unroll
            for (int v = 0; v < V; ++v) y[v] = x[v];
            count = 0;
            for (int j = 0; j < k; ++j) {
                const float top = warp_max(lane_max(y));
                if (top == -INFINITY) break;
                uint32_t first = 0xffffffffu;
#pragma unroll
                for (int v = V - 1; v >= 0; --v)
                    if (y[v] == top) first = index_of<W>(v, lane);
                const uint32_t taken = __reduce_min_sync(kFull, first);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (static_cast<uint32_t>(index_of<W>(v, lane)) == taken) y[v] = -INFINITY;
                if (lane == j) pick = top, at = static_cast<int>(taken), place = j;
                ++count;
            }
        }
        if (lane >= count) place = lane;                      // picks that there are none for
        const float w = at >= 0 ? expf(pick - high) : 0.0f;
        float total = w;
        if (!renormalize) {
            total = 0.0f;
            if (high > -INFINITY)
#pragma unroll
                for (int v = 0; v < V; ++v) total += exp_of(x[v] - high);
        }
        total = warp_sum(total);
        if (place < k) {
            expert[row * k + place] = at;
            weights[row * k + place] = at >= 0 ? __fdividef(w, total) : 0.0f;
        }
    }
}

// A row's picks go to their places by way of shared memory (zeros but for them), so that it leaves in whole
// accesses.
template <class T, int V, int W>
__global__ void __launch_bounds__(kRouteBlock) k_route_grad(const float* __restrict__ dweights, const T* __restrict__ logits,
                                                            int64_t n, int experts, int k, int renormalize,
                                                            const int64_t* __restrict__ expert, const float* __restrict__ weights,
                                                            T* __restrict__ dlogits, int32_t* d_err)
{
    pdl_wait();
    __shared__ __align__(16) float places[kRouteBlock / 32][32 * V];
    const int lane = threadIdx.x & 31;
    float* mine = places[threadIdx.x >> 5];
    for (int i = lane; i < 32 * V; i += 32) mine[i] = 0.0f;
    __syncwarp();
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kRouteBlock / 32);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (kRouteBlock / 32) + (threadIdx.x >> 5);
    int64_t at = -1, next_at = -1;
    float w = 0.0f, g = 0.0f, next_w = 0.0f, next_g = 0.0f;
    auto fetch = [&](int64_t row) {   // a row ahead
        if (lane >= k || row >= n) return;
        next_at = expert[row * k + lane];
        next_w = weights[row * k + lane];
        next_g = dweights[row * k + lane];
    };
    fetch(first);
    for (int64_t row = first; row < n; row += step) {
        at = next_at, w = next_w, g = next_g;
        fetch(row + step);
        if (at < -1 || at >= experts) {
            set_error(d_err, SPARSE_ERR_INDEX_OUT_OF_RANGE);
            at = -1;
        }
        if (at < 0) w = g = 0.0f;   // whatever stands there
        const float s = warp_sum(w * g);
        if (at >= 0) mine[at] = renormalize ? w * (g - s) : w * g;
        __syncwarp();
        float x[V];
        if (renormalize) {
#pragma unroll
            for (int v = 0; v < V; ++v) x[v] = 0.0f;
        } else {
            read_row<T, V, W>(logits + row * experts, experts, lane, x);
            const float high = warp_max(lane_max(x));
            bool odd = false;
#pragma unroll
            for (int v = 0; v < V; ++v) odd |= !(x[v] < INFINITY);
            if (__any_sync(kFull, odd) && lane == 0) set_error(d_err, SPARSE_ERR_NON_FINITE);
            const bool some = high > -INFINITY;
            float total = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                x[v] = some ? exp_of(x[v] - high) : 0.0f;
                total += x[v];
            }
            total = warp_sum(total);
            const float scale = some ? -s / total : 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) x[v] *= scale;
        }
        T* to = dlogits + row * experts;
#pragma unroll
        for (int v = 0; v < V; v += W) {
            const int i = index_of<W>(v, lane);
            float y[W];
#pragma unroll
            for (int e = 0; e < W; ++e) y[e] = x[v + e] + mine[i + e];
            if (i < experts) Pack<T, W>::put(to + i, y);
        }
        __syncwarp();
        if (at >= 0) mine[at] = 0.0f;
        __syncwarp();
    }
}

// Calls f with the values a lane has (a power of two that holds the row) and those of an access.
template <class T, class F>
cudaError_t by_shape(int64_t experts, bool vec, F f)
{
    constexpr int W = 16 / sizeof(T);
    if (vec) {
        if (experts <= 32 * W) return f(std::integral_constant<int, W>(), std::integral_constant<int, W>());
        if (experts <= 64 * W) return f(std::integral_constant<int, 2 * W>(), std::integral_constant<int, W>());
        if (experts <= 128 * W) return f(std::integral_constant<int, 4 * W>(), std::integral_constant<int, W>());
        if constexpr (W == 4) return f(std::integral_constant<int, 8 * W>(), std::integral_constant<int, W>());
    }
    using One = std::integral_constant<int, 1>;
    if (experts <= 32) return f(One(), One());
    if (experts <= 64) return f(std::integral_constant<int, 2>(), One());
    if (experts <= 128) return f(std::integral_constant<int, 4>(), One());
    if (experts <= 256) return f(std::integral_constant<int, 8>(), One());
    if (experts <= 512) return f(std::integral_constant<int, 16>(), One());
    return f(std::integral_constant<int, 32>(), One());
}

dim3 grid_of(int64_t n)
{
    return dim3(static_cast<unsigned>(std::min<int64_t>((n + kRouteBlock / 32 - 1) / (kRouteBlock / 32), int64_t(32) * num_sms())));
}

template <class T>
bool whole_accesses(const void* a, const void* b, int64_t experts)
{
    return experts % (16 / sizeof(T)) == 0 && ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 15) == 0;
}

template <class T>
cudaError_t route_of(const T* logits, int64_t n, int64_t experts, int k, int renormalize, int64_t* expert, float* weights,
                     int32_t* d_err, cudaStream_t s)
{
    SO_PROFILE("expert_route", s);
    return by_shape<T>(experts, whole_accesses<T>(logits, nullptr, experts), [&](auto v, auto w) {
        return launch(k_route<T, decltype(v)::value, decltype(w)::value>, grid_of(n), dim3(kRouteBlock), s, logits, n,
                      static_cast<int>(experts), k, renormalize, expert, weights, d_err);
    });
}

template <class T>
cudaError_t route_grad_of(const float* dweights, const T* logits, int64_t n, int64_t experts, int k, int renormalize,
                          const int64_t* expert, const float* weights, T* dlogits, int32_t* d_err, cudaStream_t s)
{
    SO_PROFILE("expert_route_grad", s);
    return by_shape<T>(experts, whole_accesses<T>(logits, dlogits, experts), [&](auto v, auto w) {
        return launch(k_route_grad<T, decltype(v)::value, decltype(w)::value>, grid_of(n), dim3(kRouteBlock), s, dweights, logits,
                      n, static_cast<int>(experts), k, renormalize, expert, weights, dlogits, d_err);
    });
}

}  // namespace

cudaError_t expert_route(const void* logits, int is_bf16, int64_t n, int64_t experts, int k, int renormalize, int64_t* expert,
                         float* weights, int32_t* d_err, cudaStream_t s)
{
    return is_bf16 ? route_of(static_cast<const bf16*>(logits), n, experts, k, renormalize, expert, weights, d_err, s)
                   : route_of(static_cast<const float*>(logits), n, experts, k, renormalize, expert, weights, d_err, s);
}

cudaError_t expert_route_grad(const float* dweights, const void* logits, int is_bf16, int64_t n, int64_t experts, int k,
                              int renormalize, const int64_t* expert, const float* weights, void* dlogits, int32_t* d_err,
                              cudaStream_t s)
{
    return is_bf16 ? route_grad_of(dweights, static_cast<const bf16*>(logits), n, experts, k, renormalize, expert, weights,
                                   static_cast<bf16*>(dlogits), d_err, s)
                   : route_grad_of(dweights, static_cast<const float*>(logits), n, experts, k, renormalize, expert, weights,
                                   static_cast<float*>(dlogits), d_err, s);
}

}  // namespace so
