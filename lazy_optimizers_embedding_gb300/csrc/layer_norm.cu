// layer_norm.cu -- layer norm of dense rows or of looked-up table rows, and its
// backward pass with the sums of the scale's and shift's gradients over all rows.
//
//   mu = sum(x) / c, var = sum((x - mu)^2) / c, rstd = 1 / sqrt(var + eps)
//   xhat = (x - mu) rstd, y = xhat gamma + beta
//   h = dy gamma, dx = rstd (h - mean(h) - xhat mean(h xhat))
//   dgamma = sum over rows of dy xhat, dbeta = sum over rows of dy
//
// Both directions are bound by memory as long as few instructions go to a value, so
// what a row costs once (addresses, butterflies, a root and a quotient) is spread
// over many values a lane.
//
// Forward, a group of G lanes, a warp at most, holds a row of up to 1024 packed columns (or
// an odd one of less than 1 KB) in registers, 32 values a lane, with its whole share of the
// row in flight at once; gamma and beta lie in shared memory.  Backward the lanes also
// carry the column sums, so a lane has 8 or 16 columns and a row up to 512 lanes.
// Longer and odd rows pass through a ring in shared memory (k_ln_ring,
// k_ln_grad_ring).  The column sums are joined over the block's groups in shared
// memory, over the blocks by k_ln_join, in fixed orders: equal inputs give equal bits.
// Wider rows yet are walked in passes over the row, held in shared memory where they fit
// (k_ln_wide, k_ln_grad_wide, k_ln_cols).  All statistics and sums are fp32.
//
// Measured, 16384 x 4096 bf16: forward 48 us (268 MB, 5.6 TB/s), backward 76 us with the
// join (403 MB, 5.3 TB/s).  262144 rows of 128 fp32 columns looked up in a 10M-row
// table: forward 36 us, backward 66 us.
#include <algorithm>
#include <atomic>

#include "profile.cuh"
#include "rowio.cuh"
#include "tensor.cuh"

namespace so {

namespace {

constexpr size_t kRingSmem = 200 * 1024;   // dynamic shared memory that a launch has at most
constexpr int kLnBlock = 256;           // threads of a block (of the groups that are no wider)
constexpr int kMaxBackGroup = 512;      // backward: lanes of a group at most
constexpr int64_t kLnParts = 1024;      // blocks of the backward kernel at most, hence partial column sums
constexpr int64_t kMaxBackward = int64_t(kMaxBackGroup) * 16;   // columns of the kernel that holds rows

// The lookup: row i of x, or nullptr where idx is out of range or i past the last row.
template <class X>
__device__ __forceinline__ const X* ln_row(const X* x, int64_t r, int64_t c, const int64_t* idx, int64_t i, int64_t n)
{
    if (i >= n) return nullptr;
    if (idx == nullptr) return x + i * c;
    const int64_t k = idx[i];
    return (k >= 0 && k < r) ? x + k * c : nullptr;
}

// Lane gl holds the accesses k G + gl of V columns each, k < NV; those past the row are
// zero (kEven: none is, below `used`), and k from `used` on are past every lane's, so
// they are skipped.
template <bool kEven, class T, int V, int NV>
__device__ __forceinline__ void ln_load(Pack<T, V> (&p)[NV], const T* row, int c, int G, int gl, int used)
{
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        p[k].zero();
        if (k < used && row != nullptr && (kEven || (k * G + gl) * V < c)) p[k].load(row + (k * G + gl) * V);
    }
}

// An access as pairs of values (one value: its pair's other is 0).
template <int V> constexpr int kPairs = V == 1 ? 1 : V / 2;
template <class T, int V>
__device__ __forceinline__ void ln_pairs(F2 (&v)[kPairs<V>], const Pack<T, V>& p)
{
    float x[V];
    p.get(x);
    if constexpr (V == 1) {
        v[0] = F2::of(x[0], 0.0f);
    } else {
#pragma unroll
        for (int e = 0; e < V; e += 2) v[e / 2] = F2::of(x[e], x[e + 1]);
    }
}
template <class T, int V>
__device__ __forceinline__ void ln_put(T* to, const F2 (&v)[kPairs<V>])
{
    float x[V];
    if constexpr (V == 1) {
        x[0] = v[0].lo();
    } else {
#pragma unroll
        for (int e = 0; e < V; e += 2) x[e] = v[e / 2].lo(), x[e + 1] = v[e / 2].hi();
    }
    Pack<T, V>::put(to, x);
}

// A vector over the columns in shared memory as its lanes read it: 16-byte pieces (or 8, 4) of
// an access lie G apart, so neighbouring lanes read neighbouring pieces.
template <int V>
__device__ __forceinline__ int ln_slot(int k, int e, int G, int gl)
{
    constexpr int W = V < 4 ? V : 4;
    return ((k * (V / W) + e / W) * G + gl) * W + e % W;
}
template <int V>
__device__ __forceinline__ void ln_stage(float* to, const float* v, float none, int c, int G, int threads)
{
    if ((G & (G - 1)) != 0) {   // the one group of its block
        for (int k = 0; k * G * V < c; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int col = (k * G + static_cast<int>(threadIdx.x)) * V + e;
                to[ln_slot<V>(k, e, G, threadIdx.x)] = v != nullptr && col < c ? v[col] : none;
            }
        return;
    }
    const int step = 31 - __clz(G * V), gmask = G - 1;
    for (int q = threadIdx.x; q < ((c + G * V - 1) >> step << step); q += threads)
        to[ln_slot<V>(q >> step, q % V, G, q / V & gmask)] = v != nullptr && q < c ? v[q] : none;
}
template <int V>
__device__ __forceinline__ void ln_staged(F2 (&g)[kPairs<V>], const float* from, int k, int G, int gl)
{
    if constexpr (V == 1) {
        g[0] = F2::of(from[ln_slot<V>(k, 0, G, gl)], 0.0f);
    } else if constexpr (V == 2) {
        const float2 q = *reinterpret_cast<const float2*>(from + ln_slot<V>(k, 0, G, gl));
        g[0] = F2::of(q.x, q.y);
    } else {
#pragma unroll
        for (int e = 0; e < V; e += 4) {
            const float4 q = *reinterpret_cast<const float4*>(from + ln_slot<V>(k, e, G, gl));
            g[e / 2] = F2::of(q.x, q.y), g[e / 2 + 1] = F2::of(q.z, q.w);
        }
    }
}

template <class X, class Y, int V, int L, bool kEven>
__global__ void __launch_bounds__(kLnBlock, 4)
    k_ln(const X* __restrict__ x, int64_t r, int c, const int64_t* __restrict__ idx, int64_t n,
         const float* __restrict__ gamma, const float* __restrict__ beta, float eps, Y* __restrict__ y,
         float* __restrict__ mean, float* __restrict__ rstd, int G, int32_t* d_err)
{
    pdl_wait();   // writes caller outputs: dependents start after this grid exits
    constexpr int NV = L / V, NP = kPairs<V>;
    extern __shared__ float4 stage[];
    const int gl = threadIdx.x & (G - 1), sub = threadIdx.x / G, groups = blockDim.x / G;
    const int used = (c + G * V - 1) / (G * V);
    float* sg = reinterpret_cast<float*>(stage);
    float* sb = sg + used * G * V;
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
    const float inv_c = 1.0f / static_cast<float>(c);
    bool staged = false;

    for (int64_t base = static_cast<int64_t>(blockIdx.x) * groups; base < n; base += step) {   // block-uniform trips
        const int64_t i = base + sub;
        const X* row = ln_row(x, r, c, idx, i, n);
        F2 v[NV][NP], s2 = F2::both(0.0f);
        {
            Pack<X, V> p[NV];
            ln_load<kEven>(p, row, c, G, gl, used);
            if (!staged) {   // while the first rows are on their way
                ln_stage<V>(sg, gamma, 1.0f, c, G, blockDim.x);
                ln_stage<V>(sb, beta, 0.0f, c, G, blockDim.x);
                __syncthreads();
                staged = true;
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                ln_pairs<X, V>(v[k], p[k]);
#pragma unroll
                for (int e = 0; e < NP; ++e) s2 = s2 + v[k][e];
            }
        }
        float s[1] = {s2.sum()};
        lanes_sum<1>(s, G);
        const float mu = s[0] * inv_c;
        s2 = F2::both(0.0f);
        const F2 off = V == 1 ? F2::of(-mu, 0.0f) : F2::both(-mu), none = F2::both(0.0f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const F2 o = k < used && (kEven || (k * G + gl) * V < c) ? off : none;   // what is past the row stays 0
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                v[k][e] = v[k][e] + o;
                s2 = fma2(v[k][e], v[k][e], s2);
            }
        }
        s[0] = s2.sum();
        lanes_sum<1>(s, G);
        const float rs = rsqrtf(fmaf(s[0], inv_c, eps));   // within 2 ulp
        if (row != nullptr) {
            Y* to = y + i * c;
            const F2 rs2 = F2::both(rs);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (k < used && (kEven || (k * G + gl) * V < c)) {
                    F2 g[NP], b[NP];
                    ln_staged<V>(g, sg, k, G, gl);
                    ln_staged<V>(b, sb, k, G, gl);
#pragma unroll
                    for (int e = 0; e < NP; ++e) g[e] = fma2(v[k][e] * rs2, g[e], b[e]);
                    ln_put<Y, V>(to + (k * G + gl) * V, g);
                }
            }
            if (gl == 0) {
                if (mean) mean[i] = mu;
                if (rstd) rstd[i] = rs;
            }
        } else if (i < n && gl == 0) {
            set_error(d_err, SPARSE_ERR_INDEX_OUT_OF_RANGE);
        }
    }
}

// V values of a vector over the columns, from column j on; quad: 16-byte accesses.
template <int V>
__device__ __forceinline__ void ln_vector(float (&g)[V], const float* from, int64_t j, float none, bool quad)
{
    if constexpr (V > 1) {
        if (from != nullptr && quad) {
            Pack<float, V> p;
            p.load(from + j);
            p.get(g);
            return;
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) g[e] = from != nullptr ? from[j + e] : none;
}

// Rows wider than a group or the ring holds: R rows a block at a time, three passes over them (sum, squares
// about the mean, output).  kHeld: the first pass leaves them in shared memory as read, every thread
// its own accesses, so no one waits for another's; wider rows yet are read three times.  (4096 x
// 16384 bf16: 59 us against 98.7 us with single values and three reads.)
template <class X, class Y, int V, int R, bool kHeld>
__global__ void __launch_bounds__(kMaxBackGroup, V < 4 && !kHeld ? 4 : 2) k_ln_wide(const X* __restrict__ x, int64_t r, int64_t c,
                                                          const int64_t* __restrict__ idx, int64_t n,
                                                          const float* __restrict__ gamma, const float* __restrict__ beta,
                                                          int quad, float eps, Y* __restrict__ y, float* __restrict__ mean,
                                                          float* __restrict__ rstd, int32_t* d_err)
{
    pdl_wait();
    __shared__ float tmp[2 * 32 * R];
    extern __shared__ float4 stage[];
    X* held = reinterpret_cast<X*>(stage);
    const float inv_c = 1.0f / static_cast<float>(c);
    const int64_t j0 = static_cast<int64_t>(threadIdx.x) * V, step = static_cast<int64_t>(kMaxBackGroup) * V;
    for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * R; i0 < n; i0 += static_cast<int64_t>(gridDim.x) * R) {
        const X* row[R];
        float s[R], mu[R], rs[R];
#pragma unroll
        for (int u = 0; u < R; ++u) {   // the same for the whole block
            row[u] = ln_row(x, r, c, idx, i0 + u, n);
            if (row[u] == nullptr && i0 + u < n && threadIdx.x == 0) set_error(d_err, SPARSE_ERR_INDEX_OUT_OF_RANGE);
            s[u] = 0.0f;
        }
#pragma unroll 4
        for (int64_t j = j0; j < c; j += step)
#pragma unroll
            for (int u = 0; u < R; ++u)
                if (row[u] != nullptr) {
                    Pack<X, V> p;
                    float v[V];
                    p.load(row[u] + j);
                    if (kHeld) *reinterpret_cast<Pack<X, V>*>(held + u * c + j) = p;
                    p.get(v);
#pragma unroll
                    for (int e = 0; e < V; ++e) s[u] += v[e];
                }
        block_sum<R>(s, kMaxBackGroup, tmp, 0);
#pragma unroll
        for (int u = 0; u < R; ++u) mu[u] = s[u] * inv_c, s[u] = 0.0f;
#pragma unroll 4
        for (int64_t j = j0; j < c; j += step)
#pragma unroll
            for (int u = 0; u < R; ++u)
                if (row[u] != nullptr) {
                    Pack<X, V> p;
                    float v[V];
                    p.load((kHeld ? held + u * c : row[u]) + j);
                    p.get(v);
#pragma unroll
                    for (int e = 0; e < V; ++e) s[u] = fmaf(v[e] - mu[u], v[e] - mu[u], s[u]);
                }
        block_sum<R>(s, kMaxBackGroup, tmp, 1);
#pragma unroll
        for (int u = 0; u < R; ++u) rs[u] = 1.0f / sqrtf(fmaf(s[u], inv_c, eps));
#pragma unroll 2
        for (int64_t j = j0; j < c; j += step) {
            float g[V], b[V];
            ln_vector<V>(g, gamma, j, 1.0f, quad);
            ln_vector<V>(b, beta, j, 0.0f, quad);
#pragma unroll
            for (int u = 0; u < R; ++u)
                if (row[u] != nullptr) {
                    Pack<X, V> p;
                    float v[V];
                    p.load((kHeld ? held + u * c : row[u]) + j);
                    p.get(v);
#pragma unroll
                    for (int e = 0; e < V; ++e) v[e] = fmaf((v[e] - mu[u]) * rs[u], g[e], b[e]);
                    Pack<Y, V>::put(y + (i0 + u) * c + j, v);
                }
        }
        if (threadIdx.x == 0)
#pragma unroll
            for (int u = 0; u < R; ++u)
                if (row[u] != nullptr) {
                    if (mean) mean[i0 + u] = mu[u];
                    if (rstd) rstd[i0 + u] = rs[u];
                }
    }
}

// Sums of N values (1, 2 or 4) over a group of W warps (up to 16, from warp `first` on): the
// first butterfly steps halve the values a lane carries instead of carrying all of
// them through, then N lanes' sums of every warp meet in `tmp` (32 N words).
// The group's block meets at named barrier 1, `threads` of it (other warps of the block do not).
template <int N>
__device__ __forceinline__ void warps_sum(float (&x)[N], int W, int first, float* tmp, int threads)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kPer = 32 / N;   // lanes that end with one value's sum
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = x[i];
#pragma unroll
    for (int h = N / 2, d = 16; h > 0; h >>= 1, d >>= 1) {
        const bool up = lane & d;
#pragma unroll
        for (int i = 0; i < h; ++i) {
            const float give = up ? v[i] : v[i + h];
            v[i] = (up ? v[i + h] : v[i]) + __shfl_xor_sync(kFull, give, d);
        }
    }
#pragma unroll
    for (int d = kPer / 2; d > 0; d >>= 1) v[0] += __shfl_xor_sync(kFull, v[0], d);
    const int mine = lane / kPer, at = lane % kPer;   // the value this lane has now
    if (at == 0) tmp[mine * 32 + warp] = v[0];
    asm volatile("barrier.cta.sync 1, %0;" ::"r"(threads) : "memory");
    const float* t = tmp + mine * 32 + first;
    v[0] = at < W ? t[at] : 0.0f;
    if (kPer < 16 && at + kPer < W) v[0] += t[at + kPer];
#pragma unroll
    for (int d = kPer / 2; d > 0; d >>= 1) v[0] += __shfl_xor_sync(kFull, v[0], d);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __shfl_sync(kFull, v[0], i * kPer);
}

// xhat of two values.  fp32: (x - mean) rstd, whose difference is as good as the mean; x rstd - mean rstd would be
// off by a rounding of mean rstd, far more than xhat's own where the mean is far above the spread.  bf16 values lie 2^-8
// of themselves apart, so there that rounding is 2^-15 of the row's largest xhat at most (unless the row is
// constant), and the form takes one instruction less (24480 x 1208: 48 against 51 us).
template <class X>
__device__ __forceinline__ float ln_off(float mean, float rs) { return sizeof(X) == 2 ? -mean * rs : -mean; }
template <class X>
__device__ __forceinline__ F2 ln_xhat(F2 x, F2 off, F2 rs) { return sizeof(X) == 2 ? fma2(x, rs, off) : (x + off) * rs; }

template <class X, class Y, int V, int L, int R, bool kEven>
__global__ void __launch_bounds__(kMaxBackGroup, 1)
    k_ln_grad(const Y* __restrict__ dy, const X* __restrict__ x, int64_t r, int c, const int64_t* __restrict__ idx, int64_t n,
              const float* __restrict__ gamma, const float* __restrict__ mean, const float* __restrict__ rstd,
              X* __restrict__ dx, float* __restrict__ part, int want, int G, int32_t* d_err)
{
    pdl_wait();
    constexpr int NV = L / V, NP = kPairs<V>;
    __shared__ float tmp[2][2 * R * 32];
    extern __shared__ float4 stage[];   // gamma; then [groups][2][c], the groups' column sums
    float* sgamma = reinterpret_cast<float*>(stage);
    const int groups = blockDim.x / G, sub = groups == 1 ? 0 : threadIdx.x / G, gl = threadIdx.x - sub * G;
    const int used = (c + G * V - 1) / (G * V);
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
    const float inv_c = 1.0f / static_cast<float>(c);
    F2 sg[NV][NP], sb[NV][NP];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < NP; ++e) sg[k][e] = sb[k][e] = F2::both(0.0f);
    bool staged = false;
    int half = 0;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * groups; base < n; base += R * step) {   // block-uniform trips
        Pack<X, V> px[R][NV];
        Pack<Y, V> py[R][NV];
        float rs[R], off[R], s[2 * R];
        bool found[R];
#pragma unroll
        for (int u = 0; u < R; ++u) {
            const int64_t i = base + sub + u * step;
            const X* row = ln_row(x, r, c, idx, i, n);
            found[u] = row != nullptr;
            ln_load<kEven>(px[u], row, c, G, gl, used);
            ln_load<kEven>(py[u], row ? dy + i * c : nullptr, c, G, gl, used);
            rs[u] = row ? rstd[i] : 0.0f;
            off[u] = row ? ln_off<X>(mean[i], rs[u]) : 0.0f;
            if (row == nullptr && i < n && gl == 0) set_error(d_err, SPARSE_ERR_INDEX_OUT_OF_RANGE);
        }
        if (!staged) {
            ln_stage<V>(sgamma, gamma, 1.0f, c, G, blockDim.x);
            __syncthreads();
            staged = true;
        }
        F2 s0[R], s1[R];
#pragma unroll
        for (int u = 0; u < R; ++u) s0[u] = s1[u] = F2::both(0.0f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (k < used) {
                F2 g[NP];
                ln_staged<V>(g, sgamma, k, G, gl);
#pragma unroll
                for (int u = 0; u < R; ++u) {
                    F2 xv[NP], dv[NP];
                    ln_pairs<X, V>(xv, px[u][k]);
                    ln_pairs<Y, V>(dv, py[u][k]);
                    const F2 rs2 = F2::both(rs[u]), off2 = F2::both(off[u]);
#pragma unroll
                    for (int e = 0; e < NP; ++e) {
                        const F2 xh = ln_xhat<X>(xv[e], off2, rs2);
                        const F2 h = dv[e] * g[e];   // 0 beyond the row: dy is 0 there
                        s0[u] = s0[u] + h;
                        s1[u] = fma2(h, xh, s1[u]);
                        sg[k][e] = fma2(dv[e], xh, sg[k][e]);
                        sb[k][e] = sb[k][e] + dv[e];
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < R; ++u) s[2 * u] = s0[u].sum(), s[2 * u + 1] = s1[u].sum();
        if (G > 32) {
            warps_sum<2 * R>(s, G >> 5, sub * (G >> 5), tmp[half], blockDim.x);
            half ^= 1;
        } else {
            lanes_sum<2 * R>(s, G);
        }
#pragma unroll
        for (int u = 0; u < R; ++u) {
            if (!found[u]) continue;
            // dx = rs h - rs a - xhat rs b
            const F2 rs2 = F2::both(rs[u]), off2 = F2::both(off[u]);
            const F2 a = F2::both(-rs[u] * (s[2 * u] * inv_c)), b = F2::both(-rs[u] * (s[2 * u + 1] * inv_c));
            X* to = dx + (base + sub + u * step) * c;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (k < used && (kEven || (k * G + gl) * V < c)) {
                    F2 xv[NP], dv[NP], g[NP];
                    ln_pairs<X, V>(xv, px[u][k]);
                    ln_pairs<Y, V>(dv, py[u][k]);
                    ln_staged<V>(g, sgamma, k, G, gl);
#pragma unroll
                    for (int e = 0; e < NP; ++e)
                        xv[e] = fma2(ln_xhat<X>(xv[e], off2, rs2), b, fma2(dv[e] * g[e], rs2, a));
                    ln_put<X, V>(to + (k * G + gl) * V, xv);
                }
            }
        }
    }
    if (!want) return;

    float* mine = part + static_cast<int64_t>(blockIdx.x) * 2 * c;
    float* cols = sgamma;
    if (groups > 1) __syncthreads();   // gamma has been read
    float* to = groups > 1 ? cols + sub * 2 * c : mine;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int col = (k * G + gl) * V;
        if (col < c) {
            ln_put<float, V>(to + col, sg[k]);
            ln_put<float, V>(to + c + col, sb[k]);
        }
    }
    if (groups == 1) return;
    __syncthreads();
    for (int q = threadIdx.x; q < 2 * c; q += blockDim.x) {
        float s = 0.0f;
        for (int u = 0; u < groups; ++u) s += cols[u * 2 * c + q];
        mine[q] = s;
    }
}

// ------------------------------------------------------------- long rows
// Longer rows pass through a ring in shared memory (ring_shape says which): a warp of its own requests
// whole rows (bulk copies) some rounds ahead, so what is in flight costs no register, and
// the block's G other lanes hold 16 columns each, gamma, beta or the column sums in
// registers.  (Requested by a lane that also works on rows, every row waited for it.)
constexpr int kRingLane = 16, kRingRows = 2, kBackRows = 1, kRingStages = 4;   // rows of a round; stages at most
__host__ __device__ constexpr int ring_rows(bool back) { return back ? kBackRows : kRingRows; }

// A row's bytes in the ring: those of its 16-byte lines (up to 15 before it and after it).
__host__ __device__ constexpr uint32_t ring_bytes(int64_t c, int size) { return static_cast<uint32_t>((c * size + 15) / 16 * 16 + 16); }

// The 16-byte lines of a row of c values that lie within its array [base, base + total).  Where the
// row's first or last line reaches out of the array, its values there go to the ring (`to`: the
// row's first line) one by one.
struct Lines {
    uintptr_t lo, hi;
};
template <class T>
__device__ __forceinline__ Lines ring_lines(uint8_t* to, const T* row, int c, const T* base, int64_t total)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(row), e = a + static_cast<uintptr_t>(c) * sizeof(T);
    const uintptr_t first = a & ~static_cast<uintptr_t>(15);
    uintptr_t lo = first, hi = (e + 15) & ~static_cast<uintptr_t>(15);
    if (lo < reinterpret_cast<uintptr_t>(base)) {
        lo += 16;
        for (uintptr_t q = a; q < lo && q < e; q += sizeof(T))
            *reinterpret_cast<T*>(to + (q - first)) = *reinterpret_cast<const T*>(q);
    }
    if (hi > reinterpret_cast<uintptr_t>(base + total)) {
        hi -= 16;
        for (uintptr_t q = hi > a ? hi : a; q < e; q += sizeof(T))
            *reinterpret_cast<T*>(to + (q - first)) = *reinterpret_cast<const T*>(q);
    }
    return {lo, hi > lo ? hi : lo};
}
__device__ __forceinline__ void ring_copy(uint8_t* to, const void* row, Lines l, uint32_t bar)
{
    const uintptr_t first = reinterpret_cast<uintptr_t>(row) & ~static_cast<uintptr_t>(15);
    if (l.hi > l.lo)
        bulk_load(smem_addr(to + (l.lo - first)), reinterpret_cast<const void*>(l.lo), static_cast<uint32_t>(l.hi - l.lo), bar);
}

// A lane's 16 values of a row in the ring, pairs in the order of its accesses; zeros past
// the row.
template <class T, int V, bool kEven>
__device__ __forceinline__ void ring_get(F2 (&v)[kRingLane / 2], const uint8_t* row, int c, int G, int gl, int used)
{
    if constexpr (V == 1) {
        const T* t = reinterpret_cast<const T*>(row);
#pragma unroll
        for (int k = 0; k < kRingLane; k += 2) {
            const int a = k * G + gl, b = a + G;
            v[k / 2] = F2::of(a < c ? static_cast<float>(t[a]) : 0.0f, b < c ? static_cast<float>(t[b]) : 0.0f);
        }
    } else {
#pragma unroll
        for (int k = 0; k < kRingLane / V; ++k) {
            Pack<T, V> p;
            p.zero();
            const int col = (k * G + gl) * V;
            if (k < used && (kEven || col < c)) p.load(reinterpret_cast<const T*>(row) + col);
            F2 x[V / 2];
            ln_pairs<T, V>(x, p);
#pragma unroll
            for (int e = 0; e < V / 2; ++e) v[k * (V / 2) + e] = x[e];
        }
    }
}
template <class T, int V, bool kEven>
__device__ __forceinline__ void ring_put(T* row, const F2 (&v)[kRingLane / 2], int c, int G, int gl, int used)
{
    if constexpr (V == 1) {
#pragma unroll
        for (int k = 0; k < kRingLane; k += 2) {
            const int a = k * G + gl, b = a + G;
            if (a < c) row[a] = static_cast<T>(v[k / 2].lo());
            if (b < c) row[b] = static_cast<T>(v[k / 2].hi());
        }
    } else {
#pragma unroll
        for (int k = 0; k < kRingLane / V; ++k) {
            const int col = (k * G + gl) * V;
            F2 x[V / 2];
#pragma unroll
            for (int e = 0; e < V / 2; ++e) x[e] = v[k * (V / 2) + e];
            if (k < used && (kEven || col < c)) ln_put<T, V>(row + col, x);
        }
    }
}
// The same lane's values of a vector over the columns (`none` where there is no vector).
template <int V>
__device__ __forceinline__ void ring_vector(F2 (&v)[kRingLane / 2], const float* from, float none, int c, int G, int gl)
{
    float x[kRingLane];
#pragma unroll
    for (int k = 0; k < kRingLane; ++k) {
        const int col = V == 1 ? k * G + gl : (k / V * G + gl) * V + k % V;
        x[k] = from == nullptr ? none : col < c ? from[col] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < kRingLane; k += 2) v[k / 2] = F2::of(x[k], x[k + 1]);
}

// And of one staged in shared memory.
template <int V>
__device__ __forceinline__ void ring_staged(F2 (&v)[kRingLane / 2], const float* from, int G, int gl, int used)
{
    if constexpr (V == 1) {
#pragma unroll
        for (int k = 0; k < kRingLane; k += 2)
            v[k / 2] = F2::of(k < used ? from[k * G + gl] : 0.0f, k + 1 < used ? from[(k + 1) * G + gl] : 0.0f);
    } else {
#pragma unroll
        for (int k = 0; k < kRingLane / V; ++k) {
            F2 x[V / 2];
#pragma unroll
            for (int e = 0; e < V / 2; ++e) x[e] = F2::both(0.0f);
            if (k < used) ln_staged<V>(x, from, k, G, gl);
#pragma unroll
            for (int e = 0; e < V / 2; ++e) v[k * (V / 2) + e] = x[e];
        }
    }
}

// Bytes of dynamic shared memory: the ring's rounds of kRingRows rows (kBack: of x and dy).
template <class X, class Y, bool kBack>
__host__ __device__ constexpr uint32_t ring_round(int64_t c)
{
    return ring_rows(kBack) * (ring_bytes(c, sizeof(X)) + (kBack ? ring_bytes(c, sizeof(Y)) : 0));
}

struct Ring {
    uint64_t full[kRingStages], empty[kRingStages];
    int found[kRingStages][kRingRows];   // 0: no row; else 1 + x's offset within its first line
    float tmp[2][2 * kRingRows * 32];
    int dead;
};

// Round `it` of rows into stage `stage`, by the requesting lane.
template <class X, class Y, bool kBack>
__device__ __forceinline__ void ring_fill(Ring& S, uint8_t* data, int64_t it, int stage, const X* x, int64_t r, int c,
                                          const int64_t* idx, int64_t n, const Y* dy, int32_t* d_err)
{
    constexpr int R = ring_rows(kBack);
    const int64_t i0 = (it * gridDim.x + blockIdx.x) * R;
    if (i0 >= n) return;
    const uint32_t bar = smem_addr(&S.full[stage]), xb = ring_bytes(c, sizeof(X)), yb = kBack ? ring_bytes(c, sizeof(Y)) : 0;
    uint8_t* to = data + stage * ring_round<X, Y, kBack>(c);
    const X* row[R];
    Lines xl[R], yl[R];
    uint32_t bytes = 0;
#pragma unroll
    for (int u = 0; u < R; ++u) {
        row[u] = ln_row(x, r, c, idx, i0 + u, n);
        S.found[stage][u] = row[u] ? 1 + static_cast<int>(reinterpret_cast<uintptr_t>(row[u]) & 15u) : 0;
        if (row[u] != nullptr) {
            xl[u] = ring_lines(to + u * (xb + yb), row[u], c, x, r * c);
            bytes += static_cast<uint32_t>(xl[u].hi - xl[u].lo);
            if (kBack) {
                yl[u] = ring_lines(to + u * (xb + yb) + xb, dy + (i0 + u) * c, c, dy, n * c);
                bytes += static_cast<uint32_t>(yl[u].hi - yl[u].lo);
            }
        } else if (i0 + u < n) {
            set_error(d_err, SPARSE_ERR_INDEX_OUT_OF_RANGE);
        }
    }
    fence_async_proxy();
    mbar_expect(bar, bytes);   // the round's one arrival
#pragma unroll
    for (int u = 0; u < R; ++u)
        if (row[u] != nullptr) {
            ring_copy(to + u * (xb + yb), row[u], xl[u], bar);
            if (kBack) ring_copy(to + u * (xb + yb) + xb, dy + (i0 + u) * c, yl[u], bar);
        }
}

// The requesting warp's part: every round of the block, a stage once all `warps` others have read it.
template <class X, class Y, bool kBack>
__device__ __forceinline__ void ring_requests(Ring& S, uint8_t* data, int stages, const X* x, int64_t r, int c, const int64_t* idx,
                                              int64_t n, const Y* dy, int32_t* d_err)
{
    if ((threadIdx.x & 31) != 0) return;
    int stage = 0;
    uint32_t parity = 1;
    int64_t it = 0;
    for (; (it * gridDim.x + blockIdx.x) * ring_rows(kBack) < n; ++it) {
        if (!mbar_wait(smem_addr(&S.empty[stage]), parity, &S.dead)) break;
        ring_fill<X, Y, kBack>(S, data, it, stage, x, r, c, idx, n, dy, d_err);
        if (it == 0)
            for (int s = 1; s < kRingStages; ++s) S.found[s][0] = S.found[s][kRingRows - 1] = 0;   // what a wait that runs out, two seconds on, finds
        if (++stage == stages) stage = 0, parity ^= 1u;
    }
    // The copies land before this warp, and so the block, leaves, also where a wait ran out (two seconds at most).
    const uint64_t t0 = now_ns();
    for (int s = 0; s < stages; ++s)
        if (s < stage || it >= stages)
            while (!mbar_try(smem_addr(&S.full[s]), s < stage ? parity ^ 1u : parity) && now_ns() - t0 < 2000000000ull) {
            }
    if (S.dead) set_error(d_err, SPARSE_ERR_INTERNAL);
}
__device__ __forceinline__ void ring_init(Ring& S, int G)
{
    if (threadIdx.x == 0) {
        S.dead = 0;
        for (int s = 0; s < kRingStages; ++s) mbar_init(smem_addr(&S.full[s]), 1), mbar_init(smem_addr(&S.empty[s]), G / 32);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
}

template <class X, class Y, int V, bool kEven, int kT>
__global__ void __launch_bounds__(kT + 32, kT <= 256 ? 2 : 1)
    k_ln_ring(const X* __restrict__ x, int64_t r, int c, const int64_t* __restrict__ idx, int64_t n,
              const float* __restrict__ gamma, const float* __restrict__ beta, float eps, Y* __restrict__ y,
              float* __restrict__ mean, float* __restrict__ rstd, int stages, int32_t* d_err)
{
    pdl_wait();   // writes caller outputs
    constexpr int R = kRingRows, N = kRingLane / 2;
    __shared__ Ring S;
    extern __shared__ __align__(16) uint8_t data[];
    const int G = blockDim.x - 32, gl = threadIdx.x;
    const int used = (c + G * V - 1) / (G * V);
    const uint32_t round = ring_round<X, Y, false>(c), bytes = ring_bytes(c, sizeof(X));
    const float inv_c = 1.0f / static_cast<float>(c);
    ring_init(S, G);
    if (gl >= G) {
        ring_requests<X, Y, false>(S, data, stages, x, r, c, idx, n, static_cast<const Y*>(nullptr), d_err);
        return;
    }
    F2 g[N], b[N];
    ring_vector<V>(g, gamma, 1.0f, c, G, gl);
    ring_vector<V>(b, beta, 0.0f, c, G, gl);
    int stage = 0;
    uint32_t parity = 0;
    for (int64_t it = 0;; ++it) {
        const int64_t i0 = (it * gridDim.x + blockIdx.x) * R;
        if (i0 >= n) break;
        mbar_wait(smem_addr(&S.full[stage]), parity, &S.dead);
        const uint8_t* at = data + stage * round;
        F2 v[R][N];
        float s[R];
        bool found[R];
#pragma unroll
        for (int u = 0; u < R; ++u) {
            found[u] = S.found[stage][u] != 0;
            const int skew = V < 4 && found[u] ? S.found[stage][u] - 1 : 0;
            ring_get<X, V, kEven>(v[u], at + u * bytes + skew, c, G, gl, used);
            F2 t = v[u][0];
#pragma unroll
            for (int e = 1; e < N; ++e) t = t + v[u][e];
            s[u] = found[u] ? t.sum() : 0.0f;
        }
        __syncwarp();
        if ((gl & 31) == 0) mbar_arrive(smem_addr(&S.empty[stage]));   // the warp has read the stage
        warps_sum<R>(s, G >> 5, 0, S.tmp[0], G);
        float mu[R];
#pragma unroll
        for (int u = 0; u < R; ++u) {
            mu[u] = s[u] * inv_c;
            const F2 off = F2::both(-mu[u]);
            F2 t = F2::both(0.0f);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int k = V == 1 ? 2 * e : 2 * e / V, col = V == 1 ? k * G + gl : (k * G + gl) * V;
                if (V == 1)   // what is past the row stays 0
                    v[u][e] = v[u][e] + F2::of(col < c ? -mu[u] : 0.0f, col + G < c ? -mu[u] : 0.0f);
                else if (k < used && (kEven || col < c))
                    v[u][e] = v[u][e] + off;
                t = fma2(v[u][e], v[u][e], t);
            }
            s[u] = t.sum();
        }
        warps_sum<R>(s, G >> 5, 0, S.tmp[1], G);
#pragma unroll
        for (int u = 0; u < R; ++u) {
            if (!found[u]) continue;
            const float rs = rsqrtf(fmaf(s[u], inv_c, eps));   // within 2 ulp
            const F2 rs2 = F2::both(rs);
#pragma unroll
            for (int e = 0; e < N; ++e) v[u][e] = fma2(v[u][e] * rs2, g[e], b[e]);
            ring_put<Y, V, kEven>(y + (i0 + u) * c, v[u], c, G, gl, used);
            if (gl == 0) {
                if (mean) mean[i0 + u] = mu[u];
                if (rstd) rstd[i0 + u] = rs;
            }
        }
        if (++stage == stages) stage = 0, parity ^= 1u;
    }
    if (gl == 0 && S.dead) set_error(d_err, SPARSE_ERR_INTERNAL);   // its own wait ran out
}

template <class X, class Y, int V, bool kEven, int kT>
__global__ void __launch_bounds__(kT + 32, kT <= 256 ? 2 : 1)
    k_ln_grad_ring(const Y* __restrict__ dy, const X* __restrict__ x, int64_t r, int c, const int64_t* __restrict__ idx,
                   int64_t n, const float* __restrict__ gamma, const float* __restrict__ mean,
                   const float* __restrict__ rstd, X* __restrict__ dx, float* __restrict__ part, int want, int stages, int32_t* d_err)
{
    pdl_wait();
    constexpr int R = kBackRows, N = kRingLane / 2;
    __shared__ Ring S;
    extern __shared__ __align__(16) uint8_t data[];
    const int G = blockDim.x - 32, gl = threadIdx.x;
    const int used = (c + G * V - 1) / (G * V);
    const uint32_t round = ring_round<X, Y, true>(c), xb = ring_bytes(c, sizeof(X)), yb = ring_bytes(c, sizeof(Y));
    const float inv_c = 1.0f / static_cast<float>(c);
    float* sgamma = reinterpret_cast<float*>(data + stages * round);   // (in registers it made the sums spill)
    if (gl < G) ln_stage<V>(sgamma, gamma, 1.0f, c, G, G);
    ring_init(S, G);
    if (gl >= G) {
        ring_requests<X, Y, true>(S, data, stages, x, r, c, idx, n, dy, d_err);
        return;
    }
    F2 sg[N], sb[N];
#pragma unroll
    for (int e = 0; e < N; ++e) sg[e] = sb[e] = F2::both(0.0f);
    // a round's statistics are read a round ahead
    float next_rs[R], next_mu[R];
    auto statistics = [&](int64_t it) {
#pragma unroll
        for (int u = 0; u < R; ++u) {
            const int64_t i = (it * gridDim.x + blockIdx.x) * R + u;
            next_rs[u] = i < n ? rstd[i] : 0.0f;
            next_mu[u] = i < n ? mean[i] : 0.0f;
        }
    };
    statistics(0);
    int stage = 0;
    uint32_t parity = 0;
    for (int64_t it = 0;; ++it) {
        const int64_t i0 = (it * gridDim.x + blockIdx.x) * R;
        if (i0 >= n) break;
        float rs[R], off[R], s[2 * R];
#pragma unroll
        for (int u = 0; u < R; ++u) rs[u] = next_rs[u], off[u] = ln_off<X>(next_mu[u], next_rs[u]);
        statistics(it + 1);
        mbar_wait(smem_addr(&S.full[stage]), parity, &S.dead);
        const uint8_t* at = data + stage * round;
        F2 xh[R][N], h[R][N];
        bool found[R];
#pragma unroll
        for (int u = 0; u < R; ++u) {
            found[u] = S.found[stage][u] != 0;
            s[2 * u] = s[2 * u + 1] = 0.0f;
            if (!found[u]) continue;   // the same for the whole block
            const int xs = V < 4 ? S.found[stage][u] - 1 : 0;
            const int ys = V < 4 ? static_cast<int>(reinterpret_cast<uintptr_t>(dy + (i0 + u) * c) & 15u) : 0;
            ring_get<X, V, kEven>(xh[u], at + u * (xb + yb) + xs, c, G, gl, used);
            ring_get<Y, V, kEven>(h[u], at + u * (xb + yb) + xb + ys, c, G, gl, used);
            const F2 rs2 = F2::both(rs[u]), off2 = F2::both(off[u]);
            F2 s0 = F2::both(0.0f), s1 = s0, g[N];
            ring_staged<V>(g, sgamma, G, gl, used);
#pragma unroll
            for (int e = 0; e < N; ++e) {   // dy is 0 past the row, so nothing there counts
                xh[u][e] = ln_xhat<X>(xh[u][e], off2, rs2);
                sg[e] = fma2(h[u][e], xh[u][e], sg[e]);
                sb[e] = sb[e] + h[u][e];
                h[u][e] = h[u][e] * g[e];
                s0 = s0 + h[u][e];
                s1 = fma2(h[u][e], xh[u][e], s1);
            }
            s[2 * u] = s0.sum(), s[2 * u + 1] = s1.sum();
        }
        __syncwarp();
        if ((gl & 31) == 0) mbar_arrive(smem_addr(&S.empty[stage]));   // the warp has read the stage
        warps_sum<2 * R>(s, G >> 5, 0, S.tmp[it & 1], G);
#pragma unroll
        for (int u = 0; u < R; ++u) {
            if (!found[u]) continue;
            // dx = rs h - rs a - xhat rs b
            const F2 rs2 = F2::both(rs[u]);
            const F2 a = F2::both(-rs[u] * (s[2 * u] * inv_c)), b = F2::both(-rs[u] * (s[2 * u + 1] * inv_c));
#pragma unroll
            for (int e = 0; e < N; ++e) h[u][e] = fma2(xh[u][e], b, fma2(h[u][e], rs2, a));
            ring_put<X, V, kEven>(dx + (i0 + u) * c, h[u], c, G, gl, used);
        }
        if (++stage == stages) stage = 0, parity ^= 1u;
    }
    if (gl == 0 && S.dead) set_error(d_err, SPARSE_ERR_INTERNAL);   // its own wait ran out
    if (!want) return;
    float* mine = part + static_cast<int64_t>(blockIdx.x) * 2 * c;
    if constexpr (V > 1) {   // whole accesses (a value at a time 64 x 8192 bf16 took 22 us and not 10)
        ring_put<float, V, false>(mine, sg, c, G, gl, used);
        ring_put<float, V, false>(mine + c, sb, c, G, gl, used);
    } else {
#pragma unroll
        for (int k = 0; k < kRingLane; ++k) {
            const int col = k * G + gl;
            if (col < c) {
                mine[col] = k % 2 ? sg[k / 2].hi() : sg[k / 2].lo();
                mine[c + col] = k % 2 ? sb[k / 2].hi() : sb[k / 2].lo();
            }
        }
    }
}

// Rows wider than a group or the ring holds: the row sums and dx by one block a row, which holds x and dy in
// shared memory as k_ln_wide holds x; the column sums apart (k_ln_cols).  (4096 x 16384 bf16, all
// three kernels: 149 us against 259.5 us with single values.)
template <class X, class Y, int V, bool kHeld>
__global__ void __launch_bounds__(kMaxBackGroup, V < 4 && !kHeld ? 4 : 2) k_ln_grad_wide(const Y* __restrict__ dy, const X* __restrict__ x,
                                                               int64_t r, int64_t c, const int64_t* __restrict__ idx,
                                                               int64_t n, const float* __restrict__ gamma, int quad,
                                                               const float* __restrict__ mean,
                                                               const float* __restrict__ rstd, X* __restrict__ dx,
                                                               int32_t* d_err)
{
    pdl_wait();
    __shared__ float tmp[2 * 32 * 2];
    extern __shared__ float4 stage[];
    X* held_x = reinterpret_cast<X*>(stage);
    Y* held_y = reinterpret_cast<Y*>(reinterpret_cast<uint8_t*>(stage) + (c * static_cast<int64_t>(sizeof(X)) + 15) / 16 * 16);
    const float inv_c = 1.0f / static_cast<float>(c);
    const int64_t j0 = static_cast<int64_t>(threadIdx.x) * V, step = static_cast<int64_t>(kMaxBackGroup) * V;
    int half = 0;
    for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
        const X* row = ln_row(x, r, c, idx, i, n);
        if (row == nullptr) {   // the same for the whole block
            if (threadIdx.x == 0) set_error(d_err, SPARSE_ERR_INDEX_OUT_OF_RANGE);
            continue;
        }
        const Y* from = dy + i * c;
        const float mu = mean[i], rs = rstd[i];
        float s[2] = {0.0f, 0.0f};
#pragma unroll 4
        for (int64_t j = j0; j < c; j += step) {
            Pack<X, V> p;
            Pack<Y, V> q;
            float v[V], d[V], g[V];
            p.load(row + j);
            q.load(from + j);
            ln_vector<V>(g, gamma, j, 1.0f, quad);
            if (kHeld) {
                *reinterpret_cast<Pack<X, V>*>(held_x + j) = p;
                *reinterpret_cast<Pack<Y, V>*>(held_y + j) = q;
            }
            p.get(v);
            q.get(d);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float h = d[e] * g[e];
                s[0] += h;
                s[1] = fmaf(h, (v[e] - mu) * rs, s[1]);
            }
        }
        block_sum<2>(s, kMaxBackGroup, tmp, half);
        half ^= 1;
        const float a = s[0] * inv_c, b = s[1] * inv_c;
#pragma unroll 2
        for (int64_t j = j0; j < c; j += step) {
            Pack<X, V> p;
            Pack<Y, V> q;
            float v[V], d[V], g[V];
            p.load((kHeld ? held_x : row) + j);
            q.load((kHeld ? held_y : from) + j);
            ln_vector<V>(g, gamma, j, 1.0f, quad);
            p.get(v);
            q.get(d);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = rs * (d[e] * g[e] - a - (v[e] - mu) * rs * b);
            Pack<X, V>::put(dx + i * c + j, v);
        }
    }
}

// Column sums of one slab of rows (blockIdx.y) into its partial, V columns a thread.
template <class X, class Y, int V>
__global__ void __launch_bounds__(kLnBlock) k_ln_cols(const Y* __restrict__ dy, const X* __restrict__ x, int64_t r,
                                                      int64_t c, const int64_t* __restrict__ idx, int64_t n,
                                                      const float* __restrict__ mean, const float* __restrict__ rstd,
                                                      float* __restrict__ part)
{
    pdl_wait();
    const int64_t j = (static_cast<int64_t>(blockIdx.x) * kLnBlock + threadIdx.x) * V;
    if (j >= c) return;
    const int64_t per = (n + gridDim.y - 1) / gridDim.y;
    const int64_t i0 = per * blockIdx.y, i1 = i0 + per < n ? i0 + per : n;
    float sg[V], sb[V];
#pragma unroll
    for (int e = 0; e < V; ++e) sg[e] = sb[e] = 0.0f;
    constexpr int R = 4;   // rows requested at once
    for (int64_t i = i0; i < i1; i += R) {
        Pack<X, V> p[R];
        Pack<Y, V> q[R];
        float mu[R], rs[R];
#pragma unroll
        for (int u = 0; u < R; ++u) {
            const X* row = i + u < i1 ? ln_row(x, r, c, idx, i + u, n) : nullptr;
            p[u].zero();
            q[u].zero();   // a row that is not there adds nothing
            mu[u] = rs[u] = 0.0f;
            if (row != nullptr) {
                p[u].load(row + j);
                q[u].load(dy + (i + u) * c + j);
                mu[u] = mean[i + u], rs[u] = rstd[i + u];
            }
        }
#pragma unroll
        for (int u = 0; u < R; ++u) {
            float v[V], d[V];
            p[u].get(v);
            q[u].get(d);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                sg[e] = fmaf(d[e], (v[e] - mu[u]) * rs[u], sg[e]);
                sb[e] += d[e];
            }
        }
    }
    float* to = part + static_cast<int64_t>(blockIdx.y) * 2 * c + j;
    Pack<float, V>::put(to, sg);
    Pack<float, V>::put(to + c, sb);
}

// dgamma[c], dbeta[c] = sums of `parts` partials [2][c], each 32 columns' by one
// block: of its W warps (a power of two up to 32), warp w sums partials w, w + W, ... of its
// lane's column, then the warps' sums are added in order.
__global__ void __launch_bounds__(1024) k_ln_join(const float* __restrict__ part, int64_t parts, int64_t c,
                                                  float* __restrict__ dgamma, float* __restrict__ dbeta)
{
    pdl_wait();   // writes caller outputs
    __shared__ float t[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
    const int64_t q = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float s = 0.0f;
    if (q < 2 * c)
        for (int64_t p0 = warp; p0 < parts; p0 += W * 16) {   // 16 requests at once
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = p0 + W * i < parts ? part[(p0 + W * i) * 2 * c + q] : 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) s += v[i];
        }
    t[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && q < 2 * c) {
        for (int w = 1; w < W; ++w) s += t[w][lane];
        float* out = q < c ? dgamma : dbeta;
        if (out) out[q < c ? q : q - c] = s;
    }
}

// Lanes of a group that hold `lane` values each: the least power of two that has the row.
int lanes_of(int64_t c, int lane)
{
    int G = 1;
    while (static_cast<int64_t>(G) * lane < c) G *= 2;
    return G;
}
// The same for a group that may be a block of its own: whole warps then (4744 fp32 columns by 297 lanes, 320
// of them and not 512).
int lanes_of_block(int64_t c, int lane, int least)
{
    const int G = lanes_of(c, lane);
    return G < least ? G : std::max<int>(least, static_cast<int>((c + lane - 1) / lane + 31) / 32 * 32);
}
// Resident blocks of a kernel that groups of G lanes share (G sets its threads and, at most, its
// shared memory).
constexpr int kGroupKinds = 5 + kMaxBackGroup / 32 + 1;
template <class K>
int resident(std::atomic<int> (&known)[kGroupKinds], K kernel, int G, int threads, size_t smem)
{
    int i = 0;   // of G: powers of two to 32, multiples of 32 past it
    while (i < 5 && (1 << i) < G) ++i;
    i += (G - 1) / 32;
    int o = known[i].load(std::memory_order_relaxed);
    if (o == 0) {
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&o, kernel, threads, smem);
        o = std::max(o, 1);
        known[i].store(o, std::memory_order_relaxed);
    }
    return o;
}

struct Forward {
    const void* x;
    int64_t r, c;
    const int64_t* idx;
    int64_t n;
    const float *gamma, *beta;
    float eps;
    void* y;
    float *mean, *rstd;
    int32_t* d_err;
    cudaStream_t s;
};

template <class X, class Y, int V, int L, bool kEven>
cudaError_t run_ln_lane(const Forward& F)
{
    auto* kernel = k_ln<X, Y, V, L, kEven>;
    const int G = lanes_of(F.c, L), groups = kLnBlock / G;
    const int64_t row = (F.c + G * V - 1) / (G * V) * (G * V);
    static std::atomic<int> known[kGroupKinds];
    const int blocks = static_cast<int>(std::min<int64_t>(
        (F.n + groups - 1) / groups,
        static_cast<int64_t>(resident(known, kernel, G, kLnBlock, sizeof(float) * 2 * L * G)) * num_sms()));
    return launch_smem(kernel, dim3(blocks), dim3(kLnBlock), sizeof(float) * 2 * row, F.s, static_cast<const X*>(F.x), F.r,
                       static_cast<int>(F.c), F.idx, F.n, F.gamma, F.beta, F.eps, static_cast<Y*>(F.y), F.mean, F.rstd, G,
                       F.d_err);
}

// The ring of a row length: lanes, stages and shared memory; no stages where the registers alone
// measured faster, rows are longer than its lanes hold, or two rounds do not fit.
//   Single values (odd rows): from 1 KB (5000 x 601 fp32: 8.6 against 12.5 us forward, 18 against
//   30 back; 5000 x 1111: 12 against 21, 23 against 48).
//   Packed, forward: rows that registers would spread over several warps, from 1025 columns
//   (65536 x 2048 bf16: 84 against 95 us, 16 x 4096: 3.2 against 4.5; 65536 x 1024: 54 against 44).
//   Packed, back: long rows with a bf16 side, where there are 16 Mi values of them (bf16 16384 x 2048: 46
//   against 56 us, 4096 x 8192: 55 against 66, 4096 x 4096: 31.5 against 32.7, but 4096 x 2048: 18.7
//   against 17.1, 1000 x 8192: 23 against 21; fp32 and bf16 16384 x 2560: 73 against 114); of fp32
//   alone, whose registers hold half as many rows, those past 4096 columns (8192 x 5120: 98 against 134)
//   or that leave over a quarter of the registers' lanes idle (24480 x 1208: 80 against 94; but
//   20000 x 1536: 83 against 82, 8192 x 4096: 121 against 79).
constexpr int64_t kRingBack = 16 << 20;
struct RingShape {
    int G, stages;
    size_t smem;
};
template <class X, class Y, int V, bool kBack>
RingShape ring_shape(int64_t c, int64_t n)
{
    RingShape s{lanes_of_block(std::max<int64_t>(c, 64 * kRingLane), kRingLane, 64), 0, 0};
    const bool faster = V < 4 ? c * static_cast<int64_t>(sizeof(X)) >= 1024
                        : kBack ? c > 1024 && n * c >= kRingBack &&
                                      (sizeof(X) == 2 || sizeof(Y) == 2 || c > 4096 || c < 12 * lanes_of(c, 16))
                                : c > 1024;
    if (!faster || c > static_cast<int64_t>(kMaxBackGroup) * kRingLane) return s;
    const size_t round = ring_round<X, Y, kBack>(c);
    s.stages = static_cast<int>(std::min<size_t>(kRingStages, std::max<size_t>(2, 100 * 1024 / round)));
    s.smem = s.stages * round + (kBack ? sizeof(float) * s.G * kRingLane : 0);   // and gamma
    if (s.smem > kRingSmem) s.stages = 0;
    return s;
}
// Blocks of a ring kernel that an SM holds: its registers' limit, and the shared memory's.
template <class K>
int ring_blocks(std::atomic<int> (&known)[kGroupKinds], K kernel, const RingShape& s)
{
    return static_cast<int>(std::max<size_t>(1, std::min<size_t>(resident(known, kernel, s.G, s.G + 32, 0), 227 * 1024 / (s.smem + sizeof(Ring) + 1024))));
}

template <class X, class Y, int V, bool kEven, int kT>
cudaError_t run_ln_ring(const Forward& F, const RingShape& g)
{
    auto* kernel = k_ln_ring<X, Y, V, kEven, kT>;
    cudaError_t e = allow_smem(kernel, g.smem, kRingSmem);
    if (e != cudaSuccess) return e;
    static std::atomic<int> known[kGroupKinds];
    const int64_t blocks = std::min<int64_t>((F.n + kRingRows - 1) / kRingRows,
                                             static_cast<int64_t>(ring_blocks(known, kernel, g)) * num_sms());
    return launch_smem(kernel, dim3(static_cast<unsigned>(blocks)), dim3(g.G + 32), g.smem, F.s, static_cast<const X*>(F.x), F.r,
                       static_cast<int>(F.c), F.idx, F.n, F.gamma, F.beta, F.eps, static_cast<Y*>(F.y), F.mean, F.rstd,
                       g.stages, F.d_err);
}

// Blocks that the GPU holds at once (few calls have rows this wide: asked every time).
template <class K>
int64_t wide_blocks(K kernel, size_t smem)
{
    int o = 0;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&o, kernel, kMaxBackGroup, smem);
    return static_cast<int64_t>(std::max(o, 1)) * num_sms();
}

bool quads(const float* a, const float* b) { return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 15u) == 0; }

template <class X, class Y, int V, int R, bool kHeld>
cudaError_t run_ln_wide(const Forward& F, size_t smem)
{
    auto* kernel = k_ln_wide<X, Y, V, R, kHeld>;
    const cudaError_t e = allow_smem(kernel, smem, kRingSmem);
    if (e != cudaSuccess) return e;
    const int64_t blocks = std::min<int64_t>((F.n + R - 1) / R, wide_blocks(kernel, smem));
    return launch_smem(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kMaxBackGroup), smem, F.s, static_cast<const X*>(F.x),
                       F.r, F.c, F.idx, F.n, F.gamma, F.beta, static_cast<int>(quads(F.gamma, F.beta)), F.eps,
                       static_cast<Y*>(F.y), F.mean, F.rstd, F.d_err);
}

template <class X, class Y, int V>
cudaError_t run_ln(const Forward& F)
{
    const RingShape g = ring_shape<X, Y, V, false>(F.c, F.n);
    if (g.stages) {
        SO_PROFILE("layer_norm_ring", F.s);
        const bool even = V > 1 && F.c % (g.G * V) == 0;
        if (g.G <= 256) return even ? run_ln_ring<X, Y, V, (V > 1), 256>(F, g) : run_ln_ring<X, Y, V, false, 256>(F, g);
        return even ? run_ln_ring<X, Y, V, (V > 1), 512>(F, g) : run_ln_ring<X, Y, V, false, 512>(F, g);
    }
    constexpr int L = V == 1 ? 16 : 32;   // values a lane holds (single ones take two registers each)
    if (F.c <= 32 * L) {   // what the ring leaves of the rows that it could hold: a warp has a row at most
        SO_PROFILE("layer_norm", F.s);
        if (V > 1 && F.c % (lanes_of(F.c, L) * V) == 0) return run_ln_lane<X, Y, V, L, (V > 1)>(F);
        return run_ln_lane<X, Y, V, L, false>(F);
    }
    SO_PROFILE("layer_norm_wide", F.s);
    // two rows share gamma and beta where they leave room for two blocks an SM and the rows go round
    const size_t row = (static_cast<size_t>(F.c) * sizeof(X) + 15) / 16 * 16;
    const bool held = row <= kRingSmem && !(V * sizeof(X) == 2);   // (two bytes at a time they cost more than they save)
    if (!held) return run_ln_wide<X, Y, V, 1, false>(F, 0);
    if (2 * row <= kRingSmem / 2 && F.n >= 4 * static_cast<int64_t>(num_sms())) return run_ln_wide<X, Y, V, 2, true>(F, 2 * row);
    return run_ln_wide<X, Y, V, 1, true>(F, row);
}

// Partial column sums that a backward pass may write, whatever its accesses.
int64_t grad_parts(int64_t n, int64_t c)
{
    if (c > kMaxBackward) return std::min<int64_t>(64, std::max<int64_t>(1, n / 16));
    const int64_t groups = c * 2 >= 1024 ? 1 : std::max(1, kLnBlock / lanes_of(c, 8));   // the fewest
    return std::min<int64_t>((n + groups - 1) / groups, kLnParts);
}

struct Backward {
    const void *dy, *x;
    int64_t r, c;
    const int64_t* idx;
    int64_t n;
    const float *gamma, *mean, *rstd;
    void* dx;
    float *dgamma, *dbeta, *part;
    int32_t* d_err;
    cudaStream_t s;
};

// Blocks of a backward pass at most: four rounds of rows each once half the SMs have one (a block
// costs its column sums' way to memory and back).
int64_t back_blocks(int64_t n, int64_t rows)
{
    const int64_t rounds = (n + rows - 1) / rows;
    return std::max<int64_t>(std::min<int64_t>(rounds, num_sms() / 2), (rounds + 3) / 4);
}

template <class X, class Y, int V, int L, int R, bool kEven>
cudaError_t run_grad_lane(const Backward& B, int want, int64_t& parts)
{
    auto* kernel = k_ln_grad<X, Y, V, L, R, kEven>;
    const int G = lanes_of_block(B.c, L, kLnBlock), threads = std::max(kLnBlock, G), groups = threads / G;
    const size_t smem = sizeof(float) * L * (groups > 1 ? 2 * threads : G);   // column sums, or gamma
    static std::atomic<int> known[kGroupKinds];
    parts = std::min<int64_t>(std::min<int64_t>(parts, back_blocks(B.n, groups)),
                              static_cast<int64_t>(resident(known, kernel, G, threads, smem)) * num_sms());
    return launch_smem(kernel, dim3(static_cast<unsigned>(parts)), dim3(threads), smem, B.s, static_cast<const Y*>(B.dy),
                       static_cast<const X*>(B.x), B.r, static_cast<int>(B.c), B.idx, B.n, B.gamma, B.mean, B.rstd,
                       static_cast<X*>(B.dx), B.part, want, G, B.d_err);
}

template <class X, class Y, int V, bool kEven, int kT>
cudaError_t run_grad_ring(const Backward& B, const RingShape& g, int want, int64_t& parts)
{
    auto* kernel = k_ln_grad_ring<X, Y, V, kEven, kT>;
    cudaError_t e = allow_smem(kernel, g.smem, kRingSmem);
    if (e != cudaSuccess) return e;
    static std::atomic<int> known[kGroupKinds];
    parts = std::min<int64_t>(std::min<int64_t>(parts, back_blocks(B.n, kBackRows)),
                              static_cast<int64_t>(ring_blocks(known, kernel, g)) * num_sms());
    return launch_smem(kernel, dim3(static_cast<unsigned>(parts)), dim3(g.G + 32), g.smem, B.s, static_cast<const Y*>(B.dy),
                       static_cast<const X*>(B.x), B.r, static_cast<int>(B.c), B.idx, B.n, B.gamma, B.mean, B.rstd,
                       static_cast<X*>(B.dx), B.part, want, g.stages, B.d_err);
}

template <class X, class Y, int V, bool kHeld>
cudaError_t run_grad_wide(const Backward& B, size_t smem)
{
    auto* kernel = k_ln_grad_wide<X, Y, V, kHeld>;
    const cudaError_t e = allow_smem(kernel, smem, kRingSmem);
    if (e != cudaSuccess) return e;
    return launch_smem(kernel, dim3(static_cast<unsigned>(std::min<int64_t>(B.n, wide_blocks(kernel, smem)))), dim3(kMaxBackGroup), smem,
                       B.s, static_cast<const Y*>(B.dy), static_cast<const X*>(B.x), B.r, B.c, B.idx, B.n, B.gamma,
                       static_cast<int>(quads(B.gamma, nullptr)), B.mean, B.rstd, static_cast<X*>(B.dx), B.d_err);
}

template <class X, class Y, int V>
cudaError_t run_ln_grad(const Backward& B)
{
    const bool want = B.dgamma != nullptr || B.dbeta != nullptr;
    int64_t parts = B.n > 0 ? grad_parts(B.n, B.c) : 0;
    cudaError_t e = cudaSuccess;
    if (B.n > 0) {
        if (B.c > kMaxBackward) {
            SO_PROFILE("layer_norm_grad_wide", B.s);
            const size_t smem = ((static_cast<size_t>(B.c) * sizeof(X) + 15) / 16 + (static_cast<size_t>(B.c) * sizeof(Y) + 15) / 16) * 16;
            e = smem <= kRingSmem && !(V * sizeof(X) == 2) ? run_grad_wide<X, Y, V, true>(B, smem) : run_grad_wide<X, Y, V, false>(B, 0);
            if (e == cudaSuccess && want)
                e = launch(k_ln_cols<X, Y, V>, dim3(static_cast<unsigned>((B.c / V + kLnBlock - 1) / kLnBlock),
                                                    static_cast<unsigned>(parts)),
                           dim3(kLnBlock), B.s, static_cast<const Y*>(B.dy), static_cast<const X*>(B.x), B.r, B.c, B.idx,
                           B.n, B.mean, B.rstd, B.part);
        } else if (const RingShape g = ring_shape<X, Y, V, true>(B.c, B.n); g.stages) {
            SO_PROFILE("layer_norm_grad_ring", B.s);
            const bool even = V > 1 && B.c % (g.G * V) == 0;
            if (g.G <= 256)
                e = even ? run_grad_ring<X, Y, V, (V > 1), 256>(B, g, want, parts) : run_grad_ring<X, Y, V, false, 256>(B, g, want, parts);
            else
                e = even ? run_grad_ring<X, Y, V, (V > 1), 512>(B, g, want, parts) : run_grad_ring<X, Y, V, false, 512>(B, g, want, parts);
        } else {
            SO_PROFILE("layer_norm_grad", B.s);
            if constexpr (V < 4) {   // rows of less than 1 KB
                e = run_grad_lane<X, Y, V, 8, 1, false>(B, want, parts);
            } else {
                // two rows at a time where a lane's shares of both leave it the registers
                constexpr int R = sizeof(X) == 2 ? 2 : 1;
                e = B.c % (lanes_of_block(B.c, 16, kLnBlock) * V) == 0 ? run_grad_lane<X, Y, V, 16, R, true>(B, want, parts)
                                                                       : run_grad_lane<X, Y, V, 16, R, false>(B, want, parts);
            }
        }
    }
    if (e != cudaSuccess || !want) return e;
    SO_PROFILE("layer_norm_grad_join", B.s);
    int threads = 64;   // of a block: about 8 partials a warp, so that more columns' blocks fit beside one another
    while (threads < 1024 && threads / 32 * 8 < parts) threads *= 2;
    return launch(k_ln_join, dim3(static_cast<unsigned>((2 * B.c + 31) / 32)), dim3(threads), B.s,
                  static_cast<const float*>(B.part), parts, B.c, B.dgamma, B.dbeta);
}

}  // namespace

int64_t layer_norm_parts(int64_t n, int64_t c) { return grad_parts(n, c); }

cudaError_t layer_norm(const void* x, int x_bf16, int64_t r, int64_t c, const int64_t* idx, int64_t n,
                       const float* gamma, const float* beta, float eps, void* y, int y_bf16, int vec, float* mean,
                       float* rstd, int32_t* d_err, cudaStream_t s)
{
    const Forward F{x, r, c, idx, n, gamma, beta, eps, y, mean, rstd, d_err, s};
    if (!x_bf16 && !y_bf16) return vec > 2 ? run_ln<float, float, 4>(F) : vec ? run_ln<float, float, 2>(F) : run_ln<float, float, 1>(F);
    if (!x_bf16) return vec > 2 ? run_ln<float, bf16, 8>(F) : vec ? run_ln<float, bf16, 2>(F) : run_ln<float, bf16, 1>(F);
    return vec > 2 ? run_ln<bf16, bf16, 8>(F) : vec ? run_ln<bf16, bf16, 2>(F) : run_ln<bf16, bf16, 1>(F);
}

cudaError_t layer_norm_grad(const void* dy, int y_bf16, const void* x, int x_bf16, int64_t r, int64_t c,
                            const int64_t* idx, int64_t n, const float* gamma, const float* mean, const float* rstd,
                            void* dx, float* dgamma, float* dbeta, float* part, int vec, int32_t* d_err,
                            cudaStream_t s)
{
    const Backward B{dy, x, r, c, idx, n, gamma, mean, rstd, dx, dgamma, dbeta, part, d_err, s};
    if (!x_bf16 && !y_bf16) return vec > 2 ? run_ln_grad<float, float, 4>(B) : vec ? run_ln_grad<float, float, 2>(B) : run_ln_grad<float, float, 1>(B);
    if (!x_bf16) return vec > 2 ? run_ln_grad<float, bf16, 8>(B) : vec ? run_ln_grad<float, bf16, 2>(B) : run_ln_grad<float, bf16, 1>(B);
    return vec > 2 ? run_ln_grad<bf16, bf16, 8>(B) : vec ? run_ln_grad<bf16, bf16, 2>(B) : run_ln_grad<bf16, bf16, 1>(B);
}

}  // namespace so
