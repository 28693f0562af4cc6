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
// Sort: counting.  A warp owns a contiguous run of slots and walks it 32 at a time; each
// lane ORs its bit into the warp's word of its expert, so the bits below its own are
// the slots of the same expert before it.  Up to kClusterSlots slots one cluster of
// up to 8 blocks does it all in one launch (k_expert_sort: the blocks read one another's
// counts from shared memory; 16384 slots of 64 experts 4.6 us, and 8 more, which take
// three launches, 6.4).  More take contiguous tiles: k_expert_count counts every
// tile's experts, k_expert_scan turns each expert's column of tile counts into a
// running sum, k_expert_sort places.  Only whole numbers are added, so the result is
// exact and the same on every run.
//
// Rows: a group of G lanes owns a token and walks the columns G * V at a time
// (16-byte accesses where the rows allow them), so each x or dy row is read once
// for all its slots.  Weighted sums and dot products are fp32, in slot order
// and in lane order.
#include <algorithm>

#include "profile.cuh"
#include "rowio.cuh"
#include "tensor.cuh"

namespace so {

namespace {

constexpr int kExBlock = 256;
constexpr int kExWarps = kExBlock / 32;
constexpr int64_t kExTile = 1024;          // slots of a tile at least
constexpr int64_t kSortBlocks = 512;       // tiles at most
constexpr int64_t kClusterSlots = 16384;   // slots that one cluster sorts
constexpr size_t kSortSmem = 160 * 1024;   // dynamic shared memory of k_expert_sort at most
constexpr int kHeld = 4;                   // rows of 32 slots whose experts a warp keeps between its two passes

// Blocks of `threads` threads (kernel k_expert_sort), each with `tile` slots; one cluster of them or
// many with counts in the workspace.
struct SortShape {
    int64_t tile;
    int blocks, threads;
    bool cluster;
};

size_t sort_smem(int threads, int64_t experts) { return sizeof(uint32_t) * static_cast<size_t>((2 * (threads / 32) + 1) * experts); }

SortShape sort_shape(int64_t slots, int64_t experts)
{
    // as many warps as have kHeld rows of 32 slots, and as their counts leave room for
    auto threads_for = [&](int64_t tile) {
        int t = 64;
        while (t < 1024 && t * kHeld < tile && sort_smem(2 * t, experts) <= kSortSmem) t *= 2;
        return t;
    };
    if (slots <= kClusterSlots) {
        int blocks = 1;
        while (blocks < 8 && slots > 2048 * blocks) blocks *= 2;
        const int64_t tile = (slots + blocks - 1) / blocks;
        return {tile, blocks, threads_for(tile), true};
    }
    const int64_t tile = std::max(kExTile, (slots + kSortBlocks - 1) / kSortBlocks);
    return {tile, static_cast<int>((slots + tile - 1) / tile), threads_for(tile), false};
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

// Exclusive scan of one value a thread over the block; *total: the block's sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* tmp, uint32_t* total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const uint32_t incl = warp_incl_scan(x, lane);
    if (lane == 31) tmp[warp] = incl;
    __syncthreads();
    const uint32_t w = lane < warps ? tmp[lane] : 0u;
    const uint32_t wi = warp_incl_scan(w, lane);
    const uint32_t before = __shfl_sync(kFull, wi - w, warp);
    *total = __shfl_sync(kFull, wi, 31);
    __syncthreads();
    return before + incl - x;
}

// counts, totals: of every tile, where the tiles are not one cluster's (else nullptr).
__global__ void __launch_bounds__(1024) k_expert_sort(const int64_t* __restrict__ expert, int64_t slots, int experts,
                                                      int64_t tile, const uint32_t* __restrict__ counts,
                                                      const uint32_t* __restrict__ totals,
                                                      int64_t* __restrict__ offsets, int32_t* __restrict__ src,
                                                      int32_t* __restrict__ pos, int32_t* d_err)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, threads = blockDim.x, warps = threads >> 5;
    extern __shared__ uint32_t sh[];
    uint32_t* cnt = sh;                          // [warps][experts]: the warps' counts, then next places
    uint32_t* bits = sh + warps * experts;       // [warps][experts]: lanes of the present 32 slots
    uint32_t* mine_all = bits + warps * experts; // [experts]: the block's counts, for its cluster
    __shared__ uint32_t scan[32];
    for (int q = threadIdx.x; q < 2 * warps * experts; q += threads) sh[q] = 0;
    pdl_wait();   // writes caller outputs
    __syncthreads();

    const int64_t s0 = min(tile * blockIdx.x, slots), s1 = min(s0 + tile, slots);
    const int64_t run_len = ((tile + warps - 1) / warps + 31) / 32 * 32;
    const int64_t w0 = min(s0 + run_len * warp, s1), w1 = min(w0 + run_len, s1);
    uint32_t* mine = cnt + warp * experts;
    uint32_t* word = bits + warp * experts;
    int held[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int64_t s = w0 + 32 * i + lane;
        held[i] = s < w1 ? slot_expert(expert, s, experts, d_err) : -1;
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        if (held[i] >= 0) atomicAdd(&mine[held[i]], 1u);
    for (int64_t s = w0 + 32 * kHeld + lane; s < w1; s += 32) {
        const int e = slot_expert(expert, s, experts, d_err);
        if (e >= 0) atomicAdd(&mine[e], 1u);
    }
    __syncthreads();
    const bool cluster = counts == nullptr && gridDim.x > 1;
    const int rank = cluster ? static_cast<int>(cluster_rank()) : 0;
    if (counts == nullptr) {
        for (int e = threadIdx.x; e < experts; e += threads) {
            uint32_t v = 0;
            for (int w = 0; w < warps; ++w) v += cnt[w * experts + e];
            mine_all[e] = v;
        }
        if (cluster) cluster_sync();   // alone, a lane reads the counts that it wrote
    }

    // first places: experts before this one, tiles before this one, warps before this one
    uint32_t run = 0;
    for (int e0 = 0; e0 < experts; e0 += threads) {
        const int e = e0 + threadIdx.x;
        uint32_t all = 0, tiles_before = 0;
        if (e < experts) {
            if (counts != nullptr) {
                all = totals[e];
                tiles_before = counts[static_cast<int64_t>(e) * gridDim.x + blockIdx.x];
            } else if (!cluster) {
                all = mine_all[e];
            } else {
                for (int r = 0; r < static_cast<int>(gridDim.x); ++r) {
                    const uint32_t v = lds_cluster_u32(cluster_addr(smem_addr(mine_all + e), r));
                    all += v;
                    tiles_before += r < rank ? v : 0u;
                }
            }
        }
        uint32_t sum;
        const uint32_t before = run + block_scan(all, scan, &sum);
        run += sum;
        if (e < experts) {
            if (blockIdx.x == 0) offsets[e] = before;
            uint32_t at = before + tiles_before;
            for (int w = 0; w < warps; ++w) {
                const uint32_t v = cnt[w * experts + e];
                cnt[w * experts + e] = at;
                at += v;
            }
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) offsets[experts] = run;
    if (cluster)
        cluster_sync();   // every block has read the others' counts
    else
        __syncthreads();

    auto place = [&](int64_t s, int e) {   // 32 slots from s on, this lane's of expert e
        const bool in = s + lane < w1;
        if (e >= 0) atomicOr(&word[e], 1u << lane);
        __syncwarp();
        const uint32_t same = e >= 0 ? word[e] : 0u;
        const uint32_t first = e >= 0 ? mine[e] : 0u;
        __syncwarp();
        if (e >= 0) {
            const int rank_of = __popc(same & ((1u << lane) - 1u));
            const int32_t p = static_cast<int32_t>(first) + rank_of;
            pos[s + lane] = p;
            if (src) src[p] = static_cast<int32_t>(s + lane);
            if (rank_of == 0) {
                word[e] = 0u;
                mine[e] = first + __popc(same);
            }
        } else if (in) {
            pos[s + lane] = -1;
        }
        __syncwarp();
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        if (w0 + 32 * i < w1) place(w0 + 32 * i, held[i]);
    for (int64_t s = w0 + 32 * kHeld; s < w1; s += 32)
        place(s, s + lane < w1 ? slot_expert(expert, s + lane, experts, d_err) : -1);
    if (src)
        for (int64_t p = run + static_cast<int64_t>(blockIdx.x) * threads + threadIdx.x; p < slots;
             p += static_cast<int64_t>(gridDim.x) * threads)
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
template <class T, int V, int J>
__global__ void __launch_bounds__(kExBlock) k_expert_combine(const T* __restrict__ ys, int64_t n, int k, int c,
                                                             const int32_t* __restrict__ pos,
                                                             const float* __restrict__ w, T* __restrict__ y, int G,
                                                             int32_t* d_err)
{
    pdl_wait();   // writes a caller output
    constexpr int R = V < 4 ? 4 : 2;
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

// A warp has one token: it holds 32 R accesses of dy while the rows of up to kMany slots go by, J
// at a time, and carries those slots' dot products along.
template <class T, int V, bool kWeights>
__global__ void __launch_bounds__(kExBlock) k_expert_grad(const T* __restrict__ dy, const T* __restrict__ ys, int64_t n,
                                                          int k, int c, const int32_t* __restrict__ pos,
                                                          const int64_t* __restrict__ end,
                                                          const float* __restrict__ w, T* __restrict__ dys,
                                                          float* __restrict__ dw, int32_t* d_err)
{
    pdl_wait();   // writes caller outputs
    // Six narrow accesses were the fastest of 4, 6 and 8 in 17 of 20 shapes (26775 x 8 x 393 bf16: 106, 92 and 106 us;
    // 5000 x 4 x 1333 fp32: 52, 44 and 51); 8, a block an SM less, where a few tokens more than the GPU has warps
    // make another round of six (4167 x 6 x 1081 fp32: 50 and 46 us, 2000 x 8 x 5001: 133 and 122).
    constexpr int J = 2, R = V < 4 ? 6 : 4, kMany = 8;
    const int lane = threadIdx.x & 31;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kExWarps + (threadIdx.x >> 5);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kExWarps;
    const int64_t slots = n * k;
    for (int64_t t = first; t < n; t += step) {
        const T* from = dy + t * c;
        for (int j0 = 0; j0 < k; j0 += kMany) {
            int place[kMany];
            float wj[kMany], dot[kMany];
#pragma unroll
            for (int j = 0; j < kMany; ++j) {
                place[j] = j0 + j < k ? static_cast<int>(slot_place(pos, t * k + j0 + j, slots, d_err)) : -1;
                wj[j] = kWeights && place[j] >= 0 ? w[t * k + j0 + j] : 1.0f;
                dot[j] = 0.0f;
            }
            for (int c0 = 0; c0 < c; c0 += 32 * V * R) {
                Pack<T, V> d[R];
#pragma unroll
                for (int q = 0; q < R; ++q) {
                    d[q].zero();
                    const int col = c0 + (q * 32 + lane) * V;
                    if (col < c) d[q].load(from + col);
                }
#pragma unroll
                for (int j1 = 0; j1 < kMany; j1 += J) {
                    if (j0 + j1 >= k) break;
                    Pack<T, V> r[J][R];
#pragma unroll
                    for (int j = 0; j < J; ++j)
#pragma unroll
                        for (int q = 0; q < R; ++q) {
                            const int col = c0 + (q * 32 + lane) * V;
                            if (place[j1 + j] >= 0 && col < c) r[j][q].load(ys + static_cast<int64_t>(place[j1 + j]) * c + col);
                        }
#pragma unroll
                    for (int j = 0; j < J; ++j)
                        if (place[j1 + j] >= 0) {
                            T* to = dys + static_cast<int64_t>(place[j1 + j]) * c;
#pragma unroll
                            for (int q = 0; q < R; ++q) {
                                const int col = c0 + (q * 32 + lane) * V;
                                if (col < c) {
                                    float dv[V], v[V];
                                    d[q].get(dv);
                                    r[j][q].get(v);
#pragma unroll
                                    for (int e = 0; e < V; ++e) {
                                        dot[j1 + j] = fmaf(dv[e], v[e], dot[j1 + j]);
                                        v[e] = wj[j1 + j] * dv[e];
                                    }
                                    Pack<T, V>::put(to + col, v);
                                }
                            }
                        }
                }
            }
            if (dw == nullptr) continue;
            // eight sums by butterflies that halve what a lane carries: lane 4 j ends with slot j's
#pragma unroll
            for (int h = kMany / 2, s = 16; h > 0; h >>= 1, s >>= 1) {
                const bool up = lane & s;
#pragma unroll
                for (int i = 0; i < h; ++i) {
                    const float give = up ? dot[i] : dot[i + h];
                    dot[i] = (up ? dot[i + h] : dot[i]) + __shfl_xor_sync(kFull, give, s);
                }
            }
            dot[0] += __shfl_xor_sync(kFull, dot[0], 2);
            dot[0] += __shfl_xor_sync(kFull, dot[0], 1);
            const int j = lane / 4;
            if (lane % 4 == 0 && j0 + j < k) dw[t * k + j0 + j] = dot[0];   // 0 for a slot that goes nowhere
        }
    }
    clear_tail<T, V>(dys, c, slots, end, 32, lane, first, step);
}

// Lanes of a group: a power of two that walks a row of `accesses`, `per` a lane at a time, in at most
// four rounds with the fewest idle lanes; of equals the widest.  (3001 x 3 x 515 fp32: 64 lanes; 8,
// which leave fewer idle but read 32 bytes at a time, took the whole there-and-back from 46 to 77 us.)
int lanes_for(int64_t accesses, int per)
{
    int best = kExBlock;
    int64_t least = INT64_MAX;
    for (int G = kExBlock; G >= 1; G /= 2) {
        const int64_t rounds = (accesses + static_cast<int64_t>(G) * per - 1) / (static_cast<int64_t>(G) * per);
        if (rounds > 4) break;
        if (rounds * G < least) best = G, least = rounds * G;
    }
    return best;
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

}  // namespace

// (A cluster uses none; a size of its own keeps a caller's pointer from being null.)
size_t expert_ws_bytes(int64_t slots, int64_t experts)
{
    const SortShape S = sort_shape(slots, experts);
    return S.cluster ? 256 : sizeof(uint32_t) * static_cast<size_t>(experts) * static_cast<size_t>(S.blocks + 1);
}

cudaError_t expert_sort(const int64_t* expert, int64_t slots, int64_t experts, int64_t* offsets, int32_t* src,
                        int32_t* pos, void* ws, int32_t* d_err, cudaStream_t s)
{
    const SortShape S = sort_shape(slots, experts);
    uint32_t* counts = S.cluster ? nullptr : static_cast<uint32_t*>(ws);
    uint32_t* totals = S.cluster ? nullptr : counts + experts * S.blocks;
    const int E = static_cast<int>(experts);
    if (!S.cluster) {
        cudaError_t e;
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
    const cudaError_t ready = allow_smem(k_expert_sort, sort_smem(S.threads, experts), kSortSmem);
    if (ready != cudaSuccess) return ready;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(S.blocks);
    cfg.blockDim = dim3(S.threads);
    cfg.dynamicSmemBytes = sort_smem(S.threads, experts);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = S.cluster ? S.blocks : 1;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    SO_PROFILE("expert_sort", s);
    return cudaLaunchKernelEx(&cfg, k_expert_sort, expert, slots, E, S.tile, static_cast<const uint32_t*>(counts),
                              static_cast<const uint32_t*>(totals), offsets, src, pos, d_err);
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
    if (vec > 2) return run_dispatch<uint4>(x, n, k, bytes / 16, pos, end, xs, d_err, s);
    if (vec && !is_bf16) return run_dispatch<uint2>(x, n, k, bytes / 8, pos, end, xs, d_err, s);
    if (vec) return run_dispatch<uint32_t>(x, n, k, bytes / 4, pos, end, xs, d_err, s);
    if (!is_bf16) return run_dispatch<uint32_t>(x, n, k, c, pos, end, xs, d_err, s);
    return run_dispatch<uint16_t>(x, n, k, c, pos, end, xs, d_err, s);
}

template <class T, int V, int J>
static cudaError_t run_combine_j(const void* ys, int64_t n, int64_t k, int64_t c, const int32_t* pos, const float* w,
                                 void* y, int32_t* d_err, cudaStream_t s)
{
    const int G = lanes_for(c / V, V < 4 ? 4 : 2);
    static const int most = resident(k_expert_combine<T, V, J>);
    SO_PROFILE("expert_combine", s);
    return launch(k_expert_combine<T, V, J>, dim3(row_blocks(most, n, G)), dim3(kExBlock), s,
                  static_cast<const T*>(ys), n, static_cast<int>(k), static_cast<int>(c), pos, w, static_cast<T*>(y), G, d_err);
}
// As many slots' rows at a time as tokens have, up to four (25986 x 1 x 269 bf16: 13.7 us, by four 23.6; 32768 x 2 x 4096 bf16 121, by four 139).
template <class T, int V>
static cudaError_t run_combine(const void* ys, int64_t n, int64_t k, int64_t c, const int32_t* pos, const float* w,
                               void* y, int32_t* d_err, cudaStream_t s)
{
    if (k == 1) return run_combine_j<T, V, 1>(ys, n, k, c, pos, w, y, d_err, s);
    if (k == 2) return run_combine_j<T, V, 2>(ys, n, k, c, pos, w, y, d_err, s);
    return run_combine_j<T, V, 4>(ys, n, k, c, pos, w, y, d_err, s);
}

cudaError_t expert_combine(const void* ys, int is_bf16, int64_t n, int64_t k, int64_t c, const int32_t* pos,
                           const float* w, void* y, int vec, int32_t* d_err, cudaStream_t s)
{
    if (is_bf16)
        return vec > 2 ? run_combine<bf16, 8>(ys, n, k, c, pos, w, y, d_err, s)
               : vec   ? run_combine<bf16, 2>(ys, n, k, c, pos, w, y, d_err, s)
                       : run_combine<bf16, 1>(ys, n, k, c, pos, w, y, d_err, s);
    return vec > 2 ? run_combine<float, 4>(ys, n, k, c, pos, w, y, d_err, s)
           : vec   ? run_combine<float, 2>(ys, n, k, c, pos, w, y, d_err, s)
                   : run_combine<float, 1>(ys, n, k, c, pos, w, y, d_err, s);
}

template <class T, int V, bool kWeights>
static cudaError_t run_grad_w(const void* dy, const void* ys, int64_t n, int64_t k, int64_t c, const int32_t* pos,
                              const int64_t* end, const float* w, void* dys, float* dw, int32_t* d_err, cudaStream_t s)
{
    static const int most = resident(k_expert_grad<T, V, kWeights>);
    SO_PROFILE("expert_combine_grad", s);
    return launch(k_expert_grad<T, V, kWeights>, dim3(row_blocks(most, n, 32)), dim3(kExBlock), s,
                  static_cast<const T*>(dy), static_cast<const T*>(ys), n, static_cast<int>(k), static_cast<int>(c), pos, end, w,
                  static_cast<T*>(dys), dw, d_err);
}
template <class T, int V>
static cudaError_t run_grad(const void* dy, const void* ys, int64_t n, int64_t k, int64_t c, const int32_t* pos,
                            const int64_t* end, const float* w, void* dys, float* dw, int32_t* d_err, cudaStream_t s)
{
    return w ? run_grad_w<T, V, true>(dy, ys, n, k, c, pos, end, w, dys, dw, d_err, s)
             : run_grad_w<T, V, false>(dy, ys, n, k, c, pos, end, w, dys, dw, d_err, s);
}

cudaError_t expert_combine_grad(const void* dy, const void* ys, int is_bf16, int64_t n, int64_t k, int64_t c,
                                const int32_t* pos, const int64_t* end, const float* w, void* dys, float* dw, int vec,
                                int32_t* d_err, cudaStream_t s)
{
    if (is_bf16)
        return vec > 2 ? run_grad<bf16, 8>(dy, ys, n, k, c, pos, end, w, dys, dw, d_err, s)
               : vec   ? run_grad<bf16, 2>(dy, ys, n, k, c, pos, end, w, dys, dw, d_err, s)
                       : run_grad<bf16, 1>(dy, ys, n, k, c, pos, end, w, dys, dw, d_err, s);
    return vec > 2 ? run_grad<float, 4>(dy, ys, n, k, c, pos, end, w, dys, dw, d_err, s)
           : vec   ? run_grad<float, 2>(dy, ys, n, k, c, pos, end, w, dys, dw, d_err, s)
                   : run_grad<float, 1>(dy, ys, n, k, c, pos, end, w, dys, dw, d_err, s);
}

}  // namespace so
