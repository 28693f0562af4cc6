// expert.cu -- tokens sorted by expert and back.
//
// n tokens name k experts each (int64 [n, k]; -1: this slot goes nowhere).  The
// slots s = t*k + j are sorted stably by expert; pos[s] is a slot's sorted place,
// src[p] the slot at a sorted place, offsets[e] the first place of expert e.
//   dispatch  xs[pos[t, j]] = x[t], and zeros in the places past offsets[experts]
//   combine   y[t] = sum_j w[t, j] ys[pos[t, j]]
//   its gradient  dys[pos[t, j]] = w[t, j] dy[t], zeros past the end;
//                 dw[t, j] = <dy[t], ys[pos[t, j]]>
// and dispatch's gradient is combine without weights.
//
// Sort: counting, in at most kSortBlocks contiguous tiles.  k_expert_count
// counts every tile's experts, k_expert_scan turns each expert's column of tile
// counts into a running sum, k_expert_place ranks the slots: a warp owns a
// contiguous run of its tile and walks it 32 slots at a time; each lane ORs its
// bit into the warp's word of its expert, so the bits below its own are the
// slots of the same expert before it.  Up to kOneBlock slots the last kernel
// alone does it all.  Only whole numbers are added, so the result is exact and
// the same on every run.
//
// Rows: a group of G lanes owns a token and walks the columns G * V at a time
// (16-byte accesses where the rows allow them), so each x or dy row is read once
// for all its slots.  Weighted sums and dot products are fp32, in slot order
// and in lane order.
#include <algorithm>

#include "profile.cuh"
#include "rowio.cuh"

namespace so {

namespace {

constexpr int kExBlock = 256;
constexpr int kExWarps = kExBlock / 32;
constexpr int64_t kExTile = 1024;     // slots of a tile at least
constexpr int64_t kSortBlocks = 512;  // tiles at most
constexpr int64_t kOneBlock = 4096;   // slots that one block sorts alone

struct SortShape {
    int64_t tile;
    int blocks;
};

SortShape sort_shape(int64_t slots)
{
    if (slots <= kOneBlock) return {std::max<int64_t>(kExBlock, (slots + kExBlock - 1) / kExBlock * kExBlock), 1};
    const int64_t per = (slots + kSortBlocks - 1) / kSortBlocks;
    const int64_t tile = std::max(kExTile, (per + kExBlock - 1) / kExBlock * kExBlock);
    return {tile, static_cast<int>((slots + tile - 1) / tile)};
}

// A slot's expert, or -1 where it goes nowhere; a bad one is reported.
__device__ __forceinline__ int slot_expert(const int64_t* expert, int64_t s, int experts, int32_t* d_err)
{
    const int64_t e = expert[s];
    if (e >= 0 && e < experts) return static_cast<int>(e);
    if (e != -1) set_error(d_err, SPARSE_ERR_INDEX_OUT_OF_RANGE);
    return -1;
}

__global__ void __launch_bounds__(kExBlock) k_expert_count(const int64_t* __restrict__ expert, int64_t slots,
                                                           int experts, int64_t tile, uint32_t* __restrict__ counts,
                                                           int32_t* d_err)
{
    pdl_enter();   // writes the workspace and the error word only
    extern __shared__ uint32_t sh[];
    for (int e = threadIdx.x; e < experts; e += kExBlock) sh[e] = 0;
    __syncthreads();
    const int64_t s0 = tile * blockIdx.x, s1 = min(s0 + tile, slots);
#pragma unroll 4
    for (int64_t s = s0 + threadIdx.x; s < s1; s += kExBlock) {
        const int e = slot_expert(expert, s, experts, d_err);
        if (e >= 0) atomicAdd(&sh[e], 1u);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < experts; e += kExBlock)
        counts[static_cast<int64_t>(e) * gridDim.x + blockIdx.x] = sh[e];
}

// One warp an expert: counts[e][*] to the sums of the tiles before, totals[e].
__global__ void __launch_bounds__(kExBlock) k_expert_scan(uint32_t* __restrict__ counts, int experts, int tiles,
                                                          uint32_t* __restrict__ totals)
{
    pdl_enter();   // writes the workspace only
    const int lane = threadIdx.x & 31;
    const int e = blockIdx.x * kExWarps + (threadIdx.x >> 5);
    if (e >= experts) return;
    uint32_t* row = counts + static_cast<int64_t>(e) * tiles;
    uint32_t run = 0;
    for (int b = 0; b < tiles; b += 32) {
        const uint32_t v = b + lane < tiles ? row[b + lane] : 0u;
        const uint32_t incl = warp_incl_scan(v, lane);
        if (b + lane < tiles) row[b + lane] = run + incl - v;
        run += __shfl_sync(kFull, incl, 31);
    }
    if (lane == 0) totals[e] = run;
}

// counts, totals: nullptr where one block has all slots.
__global__ void __launch_bounds__(kExBlock) k_expert_place(const int64_t* __restrict__ expert, int64_t slots,
                                                           int experts, int64_t tile,
                                                           const uint32_t* __restrict__ counts,
                                                           const uint32_t* __restrict__ totals,
                                                           int64_t* __restrict__ offsets, int32_t* __restrict__ src,
                                                           int32_t* __restrict__ pos, int32_t* d_err)
{
    pdl_wait();   // writes caller outputs
    extern __shared__ uint32_t sh[];
    uint32_t* cnt = sh;                              // [kExWarps][experts]: the warps' counts, then next places
    uint32_t* bits = sh + kExWarps * experts;        // [kExWarps][experts]: lanes of the present 32 slots
    __shared__ uint32_t scan[kExWarps + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int q = threadIdx.x; q < 2 * kExWarps * experts; q += kExBlock) sh[q] = 0;
    __syncthreads();

    const int64_t s0 = tile * blockIdx.x, s1 = min(s0 + tile, slots);
    const int64_t w0 = min(s0 + tile / kExWarps * warp, s1), w1 = min(w0 + tile / kExWarps, s1);
    uint32_t* mine = cnt + warp * experts;
    uint32_t* word = bits + warp * experts;
#pragma unroll 4
    for (int64_t s = w0 + lane; s < w1; s += 32) {
        const int e = slot_expert(expert, s, experts, d_err);
        if (e >= 0) atomicAdd(&mine[e], 1u);
    }
    __syncthreads();

    // first places: experts before this one, tiles before this one, warps before this one
    uint32_t run = 0;
    for (int e0 = 0; e0 < experts; e0 += kExBlock) {
        const int e = e0 + threadIdx.x;
        uint32_t all = 0;
        if (e < experts) {
            if (totals != nullptr)
                all = totals[e];
            else
                for (int w = 0; w < kExWarps; ++w) all += cnt[w * experts + e];
        }
        uint32_t sum;
        const uint32_t before = run + block_excl_scan(all, scan, &sum);
        run += sum;
        if (e < experts) {
            if (blockIdx.x == 0) offsets[e] = before;
            uint32_t at = before + (counts ? counts[static_cast<int64_t>(e) * gridDim.x + blockIdx.x] : 0u);
            for (int w = 0; w < kExWarps; ++w) {
                const uint32_t v = cnt[w * experts + e];
                cnt[w * experts + e] = at;
                at += v;
            }
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) offsets[experts] = run;
    __syncthreads();

    for (int64_t s = w0; s < w1; s += 32) {
        const bool in = s + lane < w1;
        const int e = in ? slot_expert(expert, s + lane, experts, d_err) : -1;
        if (e >= 0) atomicOr(&word[e], 1u << lane);
        __syncwarp();
        const uint32_t same = e >= 0 ? word[e] : 0u;
        const uint32_t first = e >= 0 ? mine[e] : 0u;
        __syncwarp();
        if (e >= 0) {
            const int rank = __popc(same & ((1u << lane) - 1u));
            const int32_t p = static_cast<int32_t>(first) + rank;
            pos[s + lane] = p;
            if (src) src[p] = static_cast<int32_t>(s + lane);
            if (rank == 0) {
                word[e] = 0u;
                mine[e] = first + __popc(same);
            }
        } else if (in) {
            pos[s + lane] = -1;
        }
        __syncwarp();
    }
    if (src)
        for (int64_t p = run + static_cast<int64_t>(blockIdx.x) * kExBlock + threadIdx.x; p < slots;
             p += static_cast<int64_t>(gridDim.x) * kExBlock)
            src[p] = -1;
}

// A slot's place, or -1 where it has none; one outside the sorted rows is reported.
__device__ __forceinline__ int64_t slot_place(const int32_t* pos, int64_t s, int64_t slots, int32_t* d_err)
{
    const int32_t p = pos[s];
    if (p >= 0 && p < slots) return p;
    if (p != -1) set_error(d_err, SPARSE_ERR_INDEX_OUT_OF_RANGE);
    return -1;
}

// Zeros in the sorted rows that no slot has, from offsets[experts] on.
template <class T, int V>
__device__ __forceinline__ void clear_tail(T* rows, int c, int64_t slots, const int64_t* end, int G, int gl,
                                           int64_t first, int64_t step)
{
    Pack<T, V> zero;
    zero.zero();
    float z[V];
    zero.get(z);
    const int64_t p0 = *end < 0 ? 0 : *end;
    for (int64_t p = p0 + first; p < slots; p += step) {
        T* row = rows + p * c;
        for (int col = gl * V; col < c; col += G * V) Pack<T, V>::put(row + col, z);
    }
}

// Rows are copied as units U (16 bytes where the rows allow it): cu units a row.
template <class U>
__global__ void __launch_bounds__(kExBlock) k_expert_dispatch(const U* __restrict__ x, int64_t n, int k, int cu,
                                                              const int32_t* __restrict__ pos,
                                                              const int64_t* __restrict__ end, U* __restrict__ xs,
                                                              int G, int32_t* d_err)
{
    pdl_wait();   // writes a caller output
    constexpr int R = 4;   // units a lane requests at once
    const int gl = threadIdx.x & (G - 1);
    const int64_t group = static_cast<int64_t>(blockIdx.x) * (kExBlock / G) + threadIdx.x / G;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kExBlock / G);
    const int64_t slots = n * k;
    for (int64_t t = group; t < n; t += step) {
        const U* from = x + t * cu;
        for (int c0 = gl; c0 < cu; c0 += G * R) {
            U v[R];
#pragma unroll
            for (int q = 0; q < R; ++q)
                if (c0 + q * G < cu) v[q] = from[c0 + q * G];
            for (int j = 0; j < k; ++j) {
                const int64_t p = slot_place(pos, t * k + j, slots, d_err);
                if (p < 0) continue;
                U* to = xs + p * cu;
#pragma unroll
                for (int q = 0; q < R; ++q)
                    if (c0 + q * G < cu) to[c0 + q * G] = v[q];
            }
        }
    }
    const U zero{};
    const int64_t p0 = *end < 0 ? 0 : *end;
    for (int64_t p = p0 + group; p < slots; p += step) {
        U* to = xs + p * cu;
        for (int col = gl; col < cu; col += G) to[col] = zero;
    }
}

// J slots' rows by their first access, nullptr where a slot has none.
template <class T, int J>
__device__ __forceinline__ void slot_rows(const T* (&row)[J], const T* rows, int64_t c, const int32_t* pos, int64_t t, int k,
                                          int j0, int64_t slots, int32_t* d_err)
{
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int64_t p = j0 + j < k ? slot_place(pos, t * k + j0 + j, slots, d_err) : -1;
        row[j] = p >= 0 ? rows + p * c : nullptr;
    }
}

// A lane holds R accesses of its token's sum while the slots' rows go by, J at a time.
template <class T, int V>
__global__ void __launch_bounds__(kExBlock) k_expert_combine(const T* __restrict__ ys, int64_t n, int k, int c,
                                                             const int32_t* __restrict__ pos,
                                                             const float* __restrict__ w, T* __restrict__ y, int G,
                                                             int32_t* d_err)
{
    pdl_wait();   // writes a caller output
    constexpr int J = 4, R = V == 1 ? 4 : 1;
    const int gl = threadIdx.x & (G - 1);
    const int64_t group = static_cast<int64_t>(blockIdx.x) * (kExBlock / G) + threadIdx.x / G;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kExBlock / G);
    const int64_t slots = n * k;
    for (int64_t t = group; t < n; t += step)
        for (int c0 = gl * V; c0 < c; c0 += G * V * R) {
            float a[R][V];
#pragma unroll
            for (int q = 0; q < R; ++q)
#pragma unroll
                for (int e = 0; e < V; ++e) a[q][e] = 0.0f;
            for (int j0 = 0; j0 < k; j0 += J) {
                const T* row[J];
                slot_rows(row, ys, c, pos, t, k, j0, slots, d_err);
                Pack<T, V> r[J][R];
                float wj[J];
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    wj[j] = row[j] && w ? w[t * k + j0 + j] : 1.0f;
#pragma unroll
                    for (int q = 0; q < R; ++q)
                        if (row[j] && c0 + q * G * V < c) r[j][q].load(row[j] + c0 + q * G * V);
                }
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (row[j])
#pragma unroll
                        for (int q = 0; q < R; ++q) {
                            float v[V];
                            r[j][q].get(v);
#pragma unroll
                            for (int e = 0; e < V; ++e) a[q][e] = fmaf(wj[j], v[e], a[q][e]);
                        }
            }
            T* to = y + t * c;
#pragma unroll
            for (int q = 0; q < R; ++q)
                if (c0 + q * G * V < c) Pack<T, V>::put(to + c0 + q * G * V, a[q]);
        }
}

template <class T, int V>
__global__ void __launch_bounds__(kExBlock) k_expert_grad(const T* __restrict__ dy, const T* __restrict__ ys, int64_t n,
                                                          int k, int c, const int32_t* __restrict__ pos,
                                                          const int64_t* __restrict__ end,
                                                          const float* __restrict__ w, T* __restrict__ dys,
                                                          float* __restrict__ dw, int G, int32_t* d_err)
{
    pdl_wait();   // writes caller outputs
    constexpr int J = 4, R = V == 1 ? 4 : 1;
    __shared__ float tmp[2 * 32 * J];
    const int gl = threadIdx.x & (G - 1);
    const int groups = kExBlock / G, sub = threadIdx.x / G;
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
    const int64_t slots = n * k;
    int half = 0;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * groups; base < n; base += step) {   // block-uniform trips
        const int64_t t = base + sub;
        const T* from = dy + t * c;
        for (int j0 = 0; j0 < k; j0 += J) {
            const T* row[J];
            slot_rows(row, ys, c, pos, t < n ? t : 0, t < n ? k : 0, j0, slots, d_err);
            float wj[J], dot[J];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                wj[j] = row[j] && w ? w[t * k + j0 + j] : 1.0f;
                dot[j] = 0.0f;
            }
            if (t < n)
                for (int c0 = gl * V; c0 < c; c0 += G * V * R) {
                    Pack<T, V> d[R], r[J][R];
#pragma unroll
                    for (int q = 0; q < R; ++q)
                        if (c0 + q * G * V < c) {
                            d[q].load(from + c0 + q * G * V);
#pragma unroll
                            for (int j = 0; j < J; ++j)
                                if (row[j]) r[j][q].load(row[j] + c0 + q * G * V);
                        }
#pragma unroll
                    for (int q = 0; q < R; ++q)
                        if (c0 + q * G * V < c) {
                            float dv[V];
                            d[q].get(dv);
#pragma unroll
                            for (int j = 0; j < J; ++j)
                                if (row[j]) {
                                    float v[V];
                                    r[j][q].get(v);
#pragma unroll
                                    for (int e = 0; e < V; ++e) {
                                        dot[j] = fmaf(dv[e], v[e], dot[j]);
                                        v[e] = wj[j] * dv[e];
                                    }
                                    Pack<T, V>::put(dys + (row[j] - ys) + c0 + q * G * V, v);
                                }
                        }
                }
            if (dw == nullptr) continue;
            group_sum<J>(dot, G, tmp, half);
            half ^= 1;
            if (t < n && gl == 0)
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (j0 + j < k) dw[t * k + j0 + j] = row[j] ? dot[j] : 0.0f;
        }
    }
    clear_tail<T, V>(dys, c, slots, end, G, gl, static_cast<int64_t>(blockIdx.x) * groups + sub, step);
}

// Lanes of a group: a power of two, `per` accesses of a row each where it is wide enough.
int lanes_for(int64_t accesses, int per)
{
    int G = 1;
    while (G < kExBlock && static_cast<int64_t>(G) * per < accesses) G *= 2;
    return G;
}

// Resident blocks of a row kernel at most.
template <class K>
int resident(K kernel)
{
    int o = 0;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&o, kernel, kExBlock, 0);
    return std::max(o, 1);
}

int row_blocks(int most, int64_t rows, int G)
{
    const int64_t groups = kExBlock / G;
    return static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>((rows + groups - 1) / groups, static_cast<int64_t>(most) * num_sms())));
}

size_t place_smem(int64_t experts) { return sizeof(uint32_t) * static_cast<size_t>(2 * kExWarps * experts); }

}  // namespace

size_t expert_ws_bytes(int64_t slots, int64_t experts)
{
    const SortShape S = sort_shape(slots);
    return sizeof(uint32_t) * static_cast<size_t>(experts) * static_cast<size_t>(S.blocks + 1);
}

cudaError_t expert_sort(const int64_t* expert, int64_t slots, int64_t experts, int64_t* offsets, int32_t* src,
                        int32_t* pos, void* ws, int32_t* d_err, cudaStream_t s)
{
    const SortShape S = sort_shape(slots);
    uint32_t* counts = S.blocks > 1 ? static_cast<uint32_t*>(ws) : nullptr;
    uint32_t* totals = S.blocks > 1 ? counts + experts * S.blocks : nullptr;
    const int E = static_cast<int>(experts);
    cudaError_t e = cudaSuccess;
    if (S.blocks > 1) {
        {
            SO_PROFILE("expert_count", s);
            e = launch_smem(k_expert_count, dim3(S.blocks), dim3(kExBlock), sizeof(uint32_t) * experts, s, expert,
                            slots, E, S.tile, counts, d_err);
        }
        if (e != cudaSuccess) return e;
        SO_PROFILE("expert_scan", s);
        e = launch(k_expert_scan, dim3((E + kExWarps - 1) / kExWarps), dim3(kExBlock), s, counts, E, S.blocks, totals);
        if (e != cudaSuccess) return e;
    }
    const size_t smem = place_smem(experts);
    if (smem > 48 * 1024) {
        e = cudaFuncSetAttribute(k_expert_place, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    SO_PROFILE("expert_place", s);
    return launch_smem(k_expert_place, dim3(S.blocks), dim3(kExBlock), smem, s, expert, slots, E, S.tile,
                       static_cast<const uint32_t*>(counts), static_cast<const uint32_t*>(totals), offsets, src, pos,
                       d_err);
}

template <class U>
static cudaError_t run_dispatch(const void* x, int64_t n, int64_t k, int64_t cu, const int32_t* pos,
                                const int64_t* end, void* xs, int32_t* d_err, cudaStream_t s)
{
    const int G = lanes_for(cu, 4);
    static const int most = resident(k_expert_dispatch<U>);
    SO_PROFILE("expert_dispatch", s);
    return launch(k_expert_dispatch<U>, dim3(row_blocks(most, n, G)), dim3(kExBlock), s,
                  static_cast<const U*>(x), n, static_cast<int>(k), static_cast<int>(cu), pos, end, static_cast<U*>(xs), G, d_err);
}

cudaError_t expert_dispatch(const void* x, int is_bf16, int64_t n, int64_t k, int64_t c, const int32_t* pos,
                            const int64_t* end, void* xs, int vec, int32_t* d_err, cudaStream_t s)
{
    const int64_t bytes = c * (is_bf16 ? 2 : 4);
    if (vec) return run_dispatch<uint4>(x, n, k, bytes / 16, pos, end, xs, d_err, s);
    if (!is_bf16) return run_dispatch<uint32_t>(x, n, k, c, pos, end, xs, d_err, s);
    return run_dispatch<uint16_t>(x, n, k, c, pos, end, xs, d_err, s);
}

template <class T, int V>
static cudaError_t run_combine(const void* ys, int64_t n, int64_t k, int64_t c, const int32_t* pos, const float* w,
                               void* y, int32_t* d_err, cudaStream_t s)
{
    const int G = lanes_for(c / V, V == 1 ? 4 : 1);
    static const int most = resident(k_expert_combine<T, V>);
    SO_PROFILE("expert_combine", s);
    return launch(k_expert_combine<T, V>, dim3(row_blocks(most, n, G)), dim3(kExBlock), s,
                  static_cast<const T*>(ys), n, static_cast<int>(k), static_cast<int>(c), pos, w, static_cast<T*>(y), G, d_err);
}

cudaError_t expert_combine(const void* ys, int is_bf16, int64_t n, int64_t k, int64_t c, const int32_t* pos,
                           const float* w, void* y, int vec, int32_t* d_err, cudaStream_t s)
{
    if (is_bf16)
        return vec ? run_combine<bf16, 8>(ys, n, k, c, pos, w, y, d_err, s)
                   : run_combine<bf16, 1>(ys, n, k, c, pos, w, y, d_err, s);
    return vec ? run_combine<float, 4>(ys, n, k, c, pos, w, y, d_err, s)
               : run_combine<float, 1>(ys, n, k, c, pos, w, y, d_err, s);
}

template <class T, int V>
static cudaError_t run_grad(const void* dy, const void* ys, int64_t n, int64_t k, int64_t c, const int32_t* pos,
                            const int64_t* end, const float* w, void* dys, float* dw, int32_t* d_err, cudaStream_t s)
{
    const int G = lanes_for(c / V, V == 1 ? 4 : 1);
    static const int most = resident(k_expert_grad<T, V>);
    SO_PROFILE("expert_combine_grad", s);
    return launch(k_expert_grad<T, V>, dim3(row_blocks(most, n, G)), dim3(kExBlock), s,
                  static_cast<const T*>(dy), static_cast<const T*>(ys), n, static_cast<int>(k), static_cast<int>(c), pos, end, w, static_cast<T*>(dys), dw,
                  G, d_err);
}

cudaError_t expert_combine_grad(const void* dy, const void* ys, int is_bf16, int64_t n, int64_t k, int64_t c,
                                const int32_t* pos, const int64_t* end, const float* w, void* dys, float* dw, int vec,
                                int32_t* d_err, cudaStream_t s)
{
    if (is_bf16)
        return vec ? run_grad<bf16, 8>(dy, ys, n, k, c, pos, end, w, dys, dw, d_err, s)
                   : run_grad<bf16, 1>(dy, ys, n, k, c, pos, end, w, dys, dw, d_err, s);
    return vec ? run_grad<float, 4>(dy, ys, n, k, c, pos, end, w, dys, dw, d_err, s)
               : run_grad<float, 1>(dy, ys, n, k, c, pos, end, w, dys, dw, d_err, s);
}

}  // namespace so
