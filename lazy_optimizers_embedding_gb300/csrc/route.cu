// route.cu -- the k experts of every token from its scores, and the scores' gradient.
//
// A warp has a token's row in registers, up to 32 scores a lane, as integers of the same order.  A round
// takes the largest that is left: every lane's own largest, the warp's by one reduction, of equals
// the lowest index by another; lane j keeps pick j.  Softmax sums are fp32.
#include <algorithm>

#include "profile.cuh"
#include "rowio.cuh"

namespace so {

namespace {

constexpr int kRouteBlock = 256;
constexpr uint32_t kNone = 0x007fffffu;   // the key of -inf; NaN and +inf are no scores

// Whole numbers in the order of the floats, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

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

template <class T, int V, int W>
__global__ void __launch_bounds__(kRouteBlock) k_route(const T* __restrict__ logits, int64_t n, int experts, int k, int renormalize,
                                                       int64_t* __restrict__ expert, float* __restrict__ weights, int32_t* d_err)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kRouteBlock / 32);
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * (kRouteBlock / 32) + (threadIdx.x >> 5); row < n; row += step) {
        float x[V];
        read_row<T, V, W>(logits + row * experts, experts, lane, x);
        bool odd = false;
        uint32_t key[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            odd |= !(x[v] < INFINITY);
            key[v] = key_of(x[v]);
        }
        odd = __any_sync(kFull, odd);
        if (odd && lane == 0) set_error(d_err, SPARSE_ERR_NON_FINITE);
        uint32_t first = 0, mine = kNone;   // the first pick's key, and this lane's pick's
        int at = -1;
        for (int j = 0; j < k && !odd; ++j) {
            uint32_t best = kNone;
            int where = 0;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (key[v] > best) best = key[v], where = v;   // of a lane's equals the first
            const uint32_t top = __reduce_max_sync(kFull, best);
            if (top == kNone) break;                           // nothing but -inf is left
            const uint32_t place = best == top ? index_of<W>(where, lane) : 0xffffffffu;
            const uint32_t pick = __reduce_min_sync(kFull, place);
            if (place == pick)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (v == where) key[v] = 0u;
            if (j == 0) first = top;
            if (lane == j) mine = top, at = static_cast<int>(pick);
        }
        const float high = first ? of_key(first) : 0.0f;
        const float w = at >= 0 ? expf(of_key(mine) - high) : 0.0f;
        float total = 0.0f;
        if (renormalize) {
            total = w;
        } else if (first) {
#pragma unroll
            for (int v = 0; v < V; ++v) total += expf(x[v] - high);
        }
        total = warp_sum(total);
        if (lane < k) {
            expert[row * k + lane] = at;
            weights[row * k + lane] = at >= 0 ? w / total : 0.0f;
        }
    }
}

// A row's gradient is written without its picks' share, zeros or -p s, and then the picks over it.
template <class T, int V, int W>
__global__ void __launch_bounds__(kRouteBlock) k_route_grad(const float* __restrict__ dweights, const T* __restrict__ logits,
                                                            int64_t n, int experts, int k, int renormalize,
                                                            const int64_t* __restrict__ expert, const float* __restrict__ weights,
                                                            T* __restrict__ dlogits, int32_t* d_err)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kRouteBlock / 32);
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * (kRouteBlock / 32) + (threadIdx.x >> 5); row < n; row += step) {
        int64_t at = -1;
        float w = 0.0f, g = 0.0f;
        if (lane < k) {
            at = expert[row * k + lane];
            if (at < -1 || at >= experts) {
                set_error(d_err, SPARSE_ERR_INDEX_OUT_OF_RANGE);
                at = -1;
            }
            if (at >= 0) w = weights[row * k + lane], g = dweights[row * k + lane];   // the others' are not looked at
        }
        const float s = warp_sum(w * g);
        T* to = dlogits + row * experts;
        float x[V];
        if (renormalize) {
#pragma unroll
            for (int v = 0; v < V; ++v) x[v] = 0.0f;
        } else {
            read_row<T, V, W>(logits + row * experts, experts, lane, x);
            float high = -INFINITY;
            bool odd = false;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                high = fmaxf(high, x[v]);
                odd |= !(x[v] < INFINITY);
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) high = fmaxf(high, __shfl_xor_sync(kFull, high, d));
            if (__any_sync(kFull, odd) && lane == 0) set_error(d_err, SPARSE_ERR_NON_FINITE);
            const bool some = high > -INFINITY;
            float total = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                x[v] = some ? expf(x[v] - high) : 0.0f;
                total += x[v];
            }
            total = warp_sum(total);
            const float scale = some ? -s / total : 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) x[v] *= scale;
        }
#pragma unroll
        for (int v = 0; v < V; v += W) {
            const int i = index_of<W>(v, lane);
            float y[W];
#pragma unroll
            for (int e = 0; e < W; ++e) y[e] = x[v + e];
            if (i < experts) Pack<T, W>::put(to + i, y);
        }
        __syncwarp();
        if (at >= 0) {
            const float y[1] = {w * (g - s)};
            Pack<T, 1>::put(to + at, y);
        }
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
