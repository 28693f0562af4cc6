// layer_norm.cu -- layer norm of dense rows or of looked-up table rows, and its
// backward pass with the sums of the scale's and shift's gradients over all rows.
//
//   mu = sum(x) / c, var = sum((x - mu)^2) / c, rstd = 1 / sqrt(var + eps)
//   xhat = (x - mu) rstd, y = xhat gamma + beta
//   h = dy gamma, dx = rstd (h - mean(h) - xhat mean(h xhat))
//   dgamma = sum over rows of dy xhat, dbeta = sum over rows of dy
//
// A group of G lanes holds one row in registers, kLane values a lane (G is the
// least power of two with G * kLane >= c, at most kMaxGroup), so a row is read once
// for both statistics (and, going back, for both row sums and dx).  A group
// walks rows at the grid's stride and requests its next row before it works on
// the present one; gamma, beta and the column sums stay in its registers.  The
// column sums are joined over the block's groups in shared memory, over the
// blocks by a second kernel, in fixed orders: equal inputs give equal bits.
// Wider rows are walked in passes over the row (k_ln_wide, k_ln_grad_wide,
// k_ln_cols).  All statistics and sums are fp32.
#include <algorithm>
#include <type_traits>

#include "profile.cuh"
#include "rowio.cuh"

namespace so {

namespace {

constexpr int kLane = 16;          // row values a lane holds
constexpr int kMaxGroup = 512;     // lanes of a group at most: rows of up to 8192 columns
constexpr int kLnBlock = 256;      // threads of a block whose groups are no wider
constexpr int64_t kLnParts = 1024; // blocks of the backward kernel at most, hence partial column sums

// The lookup: row i of x, or nullptr where idx is out of range.
template <class X>
__device__ __forceinline__ const X* ln_row(const X* x, int64_t r, int64_t c, const int64_t* idx, int64_t i)
{
    if (idx == nullptr) return x + i * c;
    const int64_t k = idx[i];
    return (k >= 0 && k < r) ? x + k * c : nullptr;
}

template <class T, int V, int NV>
__device__ __forceinline__ void ln_load(Pack<T, V> (&p)[NV], const T* row, int64_t c, int G, int gl)
{
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int64_t col = static_cast<int64_t>(k * G + gl) * V;
        if (row != nullptr && col < c)
            p[k].load(row + col);
        else
            p[k].zero();
    }
}

template <int V, int NV>
__device__ __forceinline__ void ln_load_vec(float (&g)[NV][V], const float* v, float none, int64_t c, int G, int gl)
{
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int64_t col = static_cast<int64_t>(k * G + gl) * V + e;
            g[k][e] = (v != nullptr && col < c) ? v[col] : none;
        }
}

template <class X, class Y, int V>
__global__ void __launch_bounds__(kMaxGroup) k_ln(const X* __restrict__ x, int64_t r, int64_t c,
                                                  const int64_t* __restrict__ idx, int64_t n,
                                                  const float* __restrict__ gamma, const float* __restrict__ beta,
                                                  float eps, Y* __restrict__ y, float* __restrict__ mean,
                                                  float* __restrict__ rstd, int G, int32_t* d_err)
{
    pdl_wait();   // writes caller outputs: dependents start after this grid exits
    constexpr int NV = kLane / V;
    __shared__ float tmp[2 * 32];
    const int gl = threadIdx.x & (G - 1);
    const int groups = blockDim.x / G;
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
    const float inv_c = 1.0f / static_cast<float>(c);
    float g[NV][V], b[NV][V];
    ln_load_vec<V, NV>(g, gamma, 1.0f, c, G, gl);
    ln_load_vec<V, NV>(b, beta, 0.0f, c, G, gl);

    int64_t base = static_cast<int64_t>(blockIdx.x) * groups;   // the block's first row: its trips are block-uniform
    const int sub = threadIdx.x / G;
    Pack<X, V> cur[NV];
    const X* row = base + sub < n ? ln_row(x, r, c, idx, base + sub) : nullptr;
    ln_load(cur, row, c, G, gl);
    for (; base < n; base += step) {
        const int64_t i = base + sub;
        const X* now = row;
        Pack<X, V> next[NV];
        row = i + step < n ? ln_row(x, r, c, idx, i + step) : nullptr;
        ln_load(next, row, c, G, gl);

        float v[NV][V], s[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            cur[k].get(v[k]);
#pragma unroll
            for (int e = 0; e < V; ++e) s[0] += v[k][e];
        }
        group_sum<1>(s, G, tmp, 0);
        const float mu = s[0] * inv_c;
        s[0] = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int64_t col = static_cast<int64_t>(k * G + gl) * V + e;
                v[k][e] -= mu;
                if (col < c) s[0] = fmaf(v[k][e], v[k][e], s[0]);
            }
        group_sum<1>(s, G, tmp, 1);
        const float rs = 1.0f / sqrtf(fmaf(s[0], inv_c, eps));
        if (now != nullptr) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int64_t col = static_cast<int64_t>(k * G + gl) * V;
#pragma unroll
                for (int e = 0; e < V; ++e) v[k][e] = fmaf(v[k][e] * rs, g[k][e], b[k][e]);
                if (col < c) Pack<Y, V>::put(y + i * c + col, v[k]);
            }
            if (gl == 0) {
                if (mean) mean[i] = mu;
                if (rstd) rstd[i] = rs;
            }
        } else if (i < n && gl == 0) {
            set_error(d_err, SPARSE_ERR_INDEX_OUT_OF_RANGE);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) cur[k] = next[k];
    }
}

// Rows wider than a group holds: one block a row, three passes over it (sum,
// squares about the mean, output); the second and third find the row in L2.
template <class X, class Y>
__global__ void __launch_bounds__(kMaxGroup) k_ln_wide(const X* __restrict__ x, int64_t r, int64_t c,
                                                       const int64_t* __restrict__ idx, int64_t n,
                                                       const float* __restrict__ gamma, const float* __restrict__ beta,
                                                       float eps, Y* __restrict__ y, float* __restrict__ mean,
                                                       float* __restrict__ rstd, int32_t* d_err)
{
    pdl_wait();
    __shared__ float tmp[2 * 32];
    const float inv_c = 1.0f / static_cast<float>(c);
    for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
        const X* row = ln_row(x, r, c, idx, i);
        if (row == nullptr) {   // the same for the whole block
            if (threadIdx.x == 0) set_error(d_err, SPARSE_ERR_INDEX_OUT_OF_RANGE);
            continue;
        }
        float s[1] = {0.0f};
        for (int64_t j = threadIdx.x; j < c; j += kMaxGroup) s[0] += static_cast<float>(row[j]);
        group_sum<1>(s, kMaxGroup, tmp, 0);
        const float mu = s[0] * inv_c;
        s[0] = 0.0f;
        for (int64_t j = threadIdx.x; j < c; j += kMaxGroup) {
            const float d = static_cast<float>(row[j]) - mu;
            s[0] = fmaf(d, d, s[0]);
        }
        group_sum<1>(s, kMaxGroup, tmp, 1);
        const float rs = 1.0f / sqrtf(fmaf(s[0], inv_c, eps));
        for (int64_t j = threadIdx.x; j < c; j += kMaxGroup) {
            const float d = (static_cast<float>(row[j]) - mu) * rs;
            y[i * c + j] = static_cast<Y>(fmaf(d, gamma ? gamma[j] : 1.0f, beta ? beta[j] : 0.0f));
        }
        if (threadIdx.x == 0) {
            if (mean) mean[i] = mu;
            if (rstd) rstd[i] = rs;
        }
    }
}

template <class X, class Y, int V>
__global__ void __launch_bounds__(kMaxGroup) k_ln_grad(const Y* __restrict__ dy, const X* __restrict__ x, int64_t r,
                                                       int64_t c, const int64_t* __restrict__ idx, int64_t n,
                                                       const float* __restrict__ gamma,
                                                       const float* __restrict__ mean, const float* __restrict__ rstd,
                                                       X* __restrict__ dx, float* __restrict__ part, int want, int G,
                                                       int32_t* d_err)
{
    pdl_wait();
    constexpr int NV = kLane / V;
    __shared__ float tmp[2 * 32 * 2];
    extern __shared__ float cols[];   // [groups][2][c]: the groups' column sums
    const int gl = threadIdx.x & (G - 1);
    const int groups = blockDim.x / G;
    const int sub = threadIdx.x / G;
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
    const float inv_c = 1.0f / static_cast<float>(c);
    float g[NV][V], sg[NV][V], sb[NV][V];
    ln_load_vec<V, NV>(g, gamma, 1.0f, c, G, gl);
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) sg[k][e] = sb[k][e] = 0.0f;

    int64_t base = static_cast<int64_t>(blockIdx.x) * groups;
    int half = 0;
    Pack<X, V> cx[NV];
    Pack<Y, V> cy[NV];
    const X* row = base + sub < n ? ln_row(x, r, c, idx, base + sub) : nullptr;
    ln_load(cx, row, c, G, gl);
    ln_load(cy, row ? dy + (base + sub) * c : nullptr, c, G, gl);
    float mu = row ? mean[base + sub] : 0.0f, rs = row ? rstd[base + sub] : 0.0f;
    for (; base < n; base += step) {
        const int64_t i = base + sub, j = i + step;
        const X* now = row;
        Pack<X, V> nx[NV];
        Pack<Y, V> ny[NV];
        row = j < n ? ln_row(x, r, c, idx, j) : nullptr;
        ln_load(nx, row, c, G, gl);
        ln_load(ny, row ? dy + j * c : nullptr, c, G, gl);
        const float nmu = row ? mean[j] : 0.0f, nrs = row ? rstd[j] : 0.0f;

        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float xv[V], dv[V];
            cx[k].get(xv);
            cy[k].get(dv);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float xh = (xv[e] - mu) * rs;
                const float h = dv[e] * g[k][e];   // 0 beyond the row: dy is 0 there
                s[0] += h;
                s[1] = fmaf(h, xh, s[1]);
                sg[k][e] = fmaf(dv[e], xh, sg[k][e]);
                sb[k][e] += dv[e];
            }
        }
        group_sum<2>(s, G, tmp, half);
        half ^= 1;
        const float a = s[0] * inv_c, b = s[1] * inv_c;
        if (now != nullptr) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int64_t col = static_cast<int64_t>(k * G + gl) * V;
                float xv[V], dv[V];
                cx[k].get(xv);
                cy[k].get(dv);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float xh = (xv[e] - mu) * rs;
                    xv[e] = rs * (fmaf(dv[e], g[k][e], -a) - xh * b);
                }
                if (col < c) Pack<X, V>::put(dx + i * c + col, xv);
            }
        } else if (i < n && gl == 0) {
            set_error(d_err, SPARSE_ERR_INDEX_OUT_OF_RANGE);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) cx[k] = nx[k], cy[k] = ny[k];
        mu = nmu, rs = nrs;
    }
    if (!want) return;

    float* mine = part + static_cast<int64_t>(blockIdx.x) * 2 * c;
    float* to = groups > 1 ? cols + static_cast<int64_t>(sub) * 2 * c : mine;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int64_t col = static_cast<int64_t>(k * G + gl) * V + e;
            if (col < c) to[col] = sg[k][e], to[c + col] = sb[k][e];
        }
    if (groups == 1) return;
    __syncthreads();
    for (int64_t q = threadIdx.x; q < 2 * c; q += blockDim.x) {
        float s = 0.0f;
        for (int u = 0; u < groups; ++u) s += cols[static_cast<int64_t>(u) * 2 * c + q];
        mine[q] = s;
    }
}

// Rows wider than a group holds: the row sums and dx by one block a row, the
// column sums apart (k_ln_cols).
template <class X, class Y>
__global__ void __launch_bounds__(kMaxGroup) k_ln_grad_wide(const Y* __restrict__ dy, const X* __restrict__ x,
                                                            int64_t r, int64_t c, const int64_t* __restrict__ idx,
                                                            int64_t n, const float* __restrict__ gamma,
                                                            const float* __restrict__ mean,
                                                            const float* __restrict__ rstd, X* __restrict__ dx,
                                                            int32_t* d_err)
{
    pdl_wait();
    __shared__ float tmp[2 * 32 * 2];
    const float inv_c = 1.0f / static_cast<float>(c);
    int half = 0;
    for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
        const X* row = ln_row(x, r, c, idx, i);
        if (row == nullptr) {
            if (threadIdx.x == 0) set_error(d_err, SPARSE_ERR_INDEX_OUT_OF_RANGE);
            continue;
        }
        const float mu = mean[i], rs = rstd[i];
        float s[2] = {0.0f, 0.0f};
        for (int64_t j = threadIdx.x; j < c; j += kMaxGroup) {
            const float h = static_cast<float>(dy[i * c + j]) * (gamma ? gamma[j] : 1.0f);
            s[0] += h;
            s[1] = fmaf(h, (static_cast<float>(row[j]) - mu) * rs, s[1]);
        }
        group_sum<2>(s, kMaxGroup, tmp, half);
        half ^= 1;
        const float a = s[0] * inv_c, b = s[1] * inv_c;
        for (int64_t j = threadIdx.x; j < c; j += kMaxGroup) {
            const float h = static_cast<float>(dy[i * c + j]) * (gamma ? gamma[j] : 1.0f);
            dx[i * c + j] = static_cast<X>(rs * (h - a - (static_cast<float>(row[j]) - mu) * rs * b));
        }
    }
}

// Column sums of one slab of rows (blockIdx.y) into its partial.
template <class X, class Y>
__global__ void __launch_bounds__(kLnBlock) k_ln_cols(const Y* __restrict__ dy, const X* __restrict__ x, int64_t r,
                                                      int64_t c, const int64_t* __restrict__ idx, int64_t n,
                                                      const float* __restrict__ mean, const float* __restrict__ rstd,
                                                      float* __restrict__ part)
{
    pdl_wait();
    const int64_t j = static_cast<int64_t>(blockIdx.x) * kLnBlock + threadIdx.x;
    if (j >= c) return;
    const int64_t per = (n + gridDim.y - 1) / gridDim.y;
    const int64_t i0 = per * blockIdx.y, i1 = i0 + per < n ? i0 + per : n;
    float sg = 0.0f, sb = 0.0f;
    for (int64_t i = i0; i < i1; ++i) {
        const X* row = ln_row(x, r, c, idx, i);
        if (row == nullptr) continue;
        const float d = static_cast<float>(dy[i * c + j]);
        sg = fmaf(d, (static_cast<float>(row[j]) - mean[i]) * rstd[i], sg);
        sb += d;
    }
    part[(static_cast<int64_t>(blockIdx.y) * 2) * c + j] = sg;
    part[(static_cast<int64_t>(blockIdx.y) * 2 + 1) * c + j] = sb;
}

// dgamma[c], dbeta[c] = sums of `parts` partials [2][c], each 32 columns' by one
// block: warp w sums partials w, w + 8, ... of its lane's column, then the warps'
// sums are added in order.
__global__ void __launch_bounds__(kLnBlock) k_ln_join(const float* __restrict__ part, int64_t parts, int64_t c,
                                                      float* __restrict__ dgamma, float* __restrict__ dbeta)
{
    pdl_wait();   // writes caller outputs
    __shared__ float t[kLnBlock / 32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t q = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float s = 0.0f;
    if (q < 2 * c)
#pragma unroll 4
        for (int64_t p = warp; p < parts; p += kLnBlock / 32) s += part[p * 2 * c + q];
    t[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && q < 2 * c) {
#pragma unroll
        for (int w = 1; w < kLnBlock / 32; ++w) s += t[w][lane];
        float* out = q < c ? dgamma : dbeta;
        if (out) out[q < c ? q : q - c] = s;
    }
}

int group_of(int64_t c)
{
    int G = 1;
    while (static_cast<int64_t>(G) * kLane < c) G *= 2;
    return G;
}

template <class K>
int resident(K kernel, int threads, size_t smem)
{
    int o = 0;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&o, kernel, threads, smem);
    return std::max(o, 1);
}

template <class X, class Y, int V>
cudaError_t run_ln(const void* x, int64_t r, int64_t c, const int64_t* idx, int64_t n, const float* gamma,
                   const float* beta, float eps, void* y, float* mean, float* rstd, int32_t* d_err, cudaStream_t s)
{
    SO_PROFILE("layer_norm", s);
    if (c > static_cast<int64_t>(kMaxGroup) * kLane) {
        const int blocks = static_cast<int>(std::min<int64_t>(n, 4 * num_sms()));
        return launch(k_ln_wide<X, Y>, dim3(blocks), dim3(kMaxGroup), s, static_cast<const X*>(x), r, c, idx, n, gamma,
                      beta, eps, static_cast<Y*>(y), mean, rstd, d_err);
    }
    const int G = group_of(c), threads = std::max(kLnBlock, G), groups = threads / G;
    const int blocks = static_cast<int>(std::min<int64_t>(
        (n + groups - 1) / groups, static_cast<int64_t>(resident(k_ln<X, Y, V>, threads, 0)) * num_sms()));
    return launch(k_ln<X, Y, V>, dim3(blocks), dim3(threads), s, static_cast<const X*>(x), r, c, idx, n, gamma, beta,
                  eps, static_cast<Y*>(y), mean, rstd, G, d_err);
}

// Partial column sums that a backward pass may write.
int64_t grad_parts(int64_t n, int64_t c)
{
    if (c > static_cast<int64_t>(kMaxGroup) * kLane) return std::min<int64_t>(64, std::max<int64_t>(1, n / 64));
    const int G = group_of(c), groups = std::max(kLnBlock, G) / G;
    return std::min<int64_t>((n + groups - 1) / groups, kLnParts);
}

template <class X, class Y, int V>
cudaError_t run_ln_grad(const void* dy, const void* x, int64_t r, int64_t c, const int64_t* idx, int64_t n,
                        const float* gamma, const float* mean, const float* rstd, void* dx, float* dgamma,
                        float* dbeta, float* part, int32_t* d_err, cudaStream_t s)
{
    const bool want = dgamma != nullptr || dbeta != nullptr;
    int64_t parts = n > 0 ? grad_parts(n, c) : 0;
    cudaError_t e = cudaSuccess;
    if (n > 0) {
        SO_PROFILE("layer_norm_grad", s);
        if (c > static_cast<int64_t>(kMaxGroup) * kLane) {
            const int blocks = static_cast<int>(std::min<int64_t>(n, 4 * num_sms()));
            e = launch(k_ln_grad_wide<X, Y>, dim3(blocks), dim3(kMaxGroup), s, static_cast<const Y*>(dy),
                       static_cast<const X*>(x), r, c, idx, n, gamma, mean, rstd, static_cast<X*>(dx), d_err);
            if (e == cudaSuccess && want)
                e = launch(k_ln_cols<X, Y>, dim3(static_cast<unsigned>((c + kLnBlock - 1) / kLnBlock),
                                                 static_cast<unsigned>(parts)),
                           dim3(kLnBlock), s, static_cast<const Y*>(dy), static_cast<const X*>(x), r, c, idx, n, mean,
                           rstd, part);
        } else {
            const int G = group_of(c), threads = std::max(kLnBlock, G), groups = threads / G;
            const size_t smem = groups > 1 ? sizeof(float) * 2 * c * groups : 0;
            parts = std::min<int64_t>(parts, static_cast<int64_t>(resident(k_ln_grad<X, Y, V>, threads, smem)) *
                                                 num_sms());
            e = launch_smem(k_ln_grad<X, Y, V>, dim3(static_cast<unsigned>(parts)), dim3(threads), smem, s,
                            static_cast<const Y*>(dy), static_cast<const X*>(x), r, c, idx, n, gamma, mean, rstd,
                            static_cast<X*>(dx), part, want ? 1 : 0, G, d_err);
        }
    }
    if (e != cudaSuccess || !want) return e;
    SO_PROFILE("layer_norm_grad_join", s);
    return launch(k_ln_join, dim3(static_cast<unsigned>((2 * c + 31) / 32)), dim3(kLnBlock), s,
                  static_cast<const float*>(part), parts, c, dgamma, dbeta);
}

}  // namespace

int64_t layer_norm_parts(int64_t n, int64_t c) { return grad_parts(n, c); }

cudaError_t layer_norm(const void* x, int x_bf16, int64_t r, int64_t c, const int64_t* idx, int64_t n,
                       const float* gamma, const float* beta, float eps, void* y, int y_bf16, int vec, float* mean,
                       float* rstd, int32_t* d_err, cudaStream_t s)
{
    if (!x_bf16 && !y_bf16)
        return vec ? run_ln<float, float, 4>(x, r, c, idx, n, gamma, beta, eps, y, mean, rstd, d_err, s)
                   : run_ln<float, float, 1>(x, r, c, idx, n, gamma, beta, eps, y, mean, rstd, d_err, s);
    if (!x_bf16)
        return vec ? run_ln<float, bf16, 8>(x, r, c, idx, n, gamma, beta, eps, y, mean, rstd, d_err, s)
                   : run_ln<float, bf16, 1>(x, r, c, idx, n, gamma, beta, eps, y, mean, rstd, d_err, s);
    return vec ? run_ln<bf16, bf16, 8>(x, r, c, idx, n, gamma, beta, eps, y, mean, rstd, d_err, s)
               : run_ln<bf16, bf16, 1>(x, r, c, idx, n, gamma, beta, eps, y, mean, rstd, d_err, s);
}

cudaError_t layer_norm_grad(const void* dy, int y_bf16, const void* x, int x_bf16, int64_t r, int64_t c,
                            const int64_t* idx, int64_t n, const float* gamma, const float* mean, const float* rstd,
                            void* dx, float* dgamma, float* dbeta, float* part, int vec, int32_t* d_err,
                            cudaStream_t s)
{
    if (!x_bf16 && !y_bf16)
        return vec ? run_ln_grad<float, float, 4>(dy, x, r, c, idx, n, gamma, mean, rstd, dx, dgamma, dbeta, part, d_err, s)
                   : run_ln_grad<float, float, 1>(dy, x, r, c, idx, n, gamma, mean, rstd, dx, dgamma, dbeta, part, d_err, s);
    if (!x_bf16)
        return vec ? run_ln_grad<float, bf16, 8>(dy, x, r, c, idx, n, gamma, mean, rstd, dx, dgamma, dbeta, part, d_err, s)
                   : run_ln_grad<float, bf16, 1>(dy, x, r, c, idx, n, gamma, mean, rstd, dx, dgamma, dbeta, part, d_err, s);
    return vec ? run_ln_grad<bf16, bf16, 8>(dy, x, r, c, idx, n, gamma, mean, rstd, dx, dgamma, dbeta, part, d_err, s)
               : run_ln_grad<bf16, bf16, 1>(dy, x, r, c, idx, n, gamma, mean, rstd, dx, dgamma, dbeta, part, d_err, s);
}

}  // namespace so
