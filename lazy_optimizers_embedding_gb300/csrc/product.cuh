// product.cuh -- the matrix products of the experts' operators and of the loss over a
// table's rows, on the tcgen05 unit: one persistent kernel in four forms.
//
// D = A B with A's rows M in tensor memory's lanes, B's columns N along its columns and fp32 sums:
//   kRows     M: columns of a group's matrix, N: rows of the group, K: the other side of the matrix.
//             D is the result transposed, so a warp's lanes write neighbours of one row, whatever
//             its alignment, and a group of any number of rows has tiles of just that width
//             (N is chosen tile by tile).
//   kWeights  M, N: columns of two arrays of rows, K: the rows of a group.  Rows behind the group's last
//             in its last 64 belong to the next group: they are cleared in shared memory, in both
//             operands, before the product reads them.
//   kScore    M: tokens, N: a table's rows, K: their columns.  D is not stored: a lane keeps its token's
//             running maximum and sum of exponentials over the tiles of an item.
//   kSlope    the same product; the loss's slope in every score leaves as bf16.
//
// Operands are bf16.  fp32 values come as three bf16 parts (v = hi + mid + lo to 2^-26), and a product is
// the six of nine that reach 2^-24: hi hi in one accumulator, hi mid, mid hi, mid mid, hi lo and lo hi, all
// below 2^-8 of it, in another.  The unit rounds every sum towards zero (about 2^-24 of the
// running sum each time): where an fp32 result asks for it (kDrain, and always with six
// products) the sums of every 512 K values, 32 a time, are added up by the epilogue in registers, to nearest.
#pragma once

#include <algorithm>

#include "profile.cuh"
#include "rowio.cuh"
#include "tensor.cuh"

namespace so {

enum Form { kRows, kWeights, kScore, kSlope };

constexpr int kPM = 128, kPK = 64;                    // rows of a block's tile; K values of a stage (128 bytes)
constexpr int kPBox = 64;                             // rows of one copied box: 64 x 128 bytes
constexpr uint32_t kPBoxBytes = kPBox * kPK * 2;
constexpr int kMaxGroups = 1024;
constexpr int kMaxSorted = 256;                       // groups that kWeights takes by their length (each block ranks them: 0.5 us)
constexpr int64_t kSms = 152;                         // what tiles and parts, and so workspaces, are planned for, whatever the device of a size query
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct ProductMaps {
    CUtensorMap a, b;
};

struct ProductArgs {
    int32_t rows;            // kRows, kWeights: rows over all groups; else tokens
    int32_t m, n, k;         // extents of M, N (not kRows) and K (not kWeights)
    int32_t m_tiles, n_tiles;
    int32_t width;           // columns of a tile at most, a multiple of 32
    int32_t groups, splits;  // parts of K, each with a result of its own, `slab` values apart
    const int64_t* offsets;  // rows of the groups; nullptr: all rows, one group
    // kRows, kWeights
    void* out;
    const float* add;        // fp32, laid out as the result: added to it (nullptr: nothing)
    int64_t slab;
    int32_t ld;              // values of a row of the result
    float* unit;             // kSlope with one part: written, see common_unit; else, where given, what results are multiplied by
    int32_t out_bf16, clear; // clear: zeros in the rows behind the last group
    // kScore, kSlope
    const int64_t* target;
    int32_t run;             // kScore: tiles of an item
    int32_t v, v0;           // the table's rows; kSlope: the first column's
    float2* part;            // kScore: [items of a row of items x groups of warps][rows], maximum and sum
    float* hit;              // kScore: score of the target
    const float *lse, *dloss;
    bf16* slope;             // kSlope: [parts][rows][ld]
    int64_t slope_part;
    int32_t release;         // writes workspace only
    int32_t* d_err;
};

template <int kForm_, bool kAmn_, bool kBmn_, int kPair_, int P_, bool kDrain_>
struct ProductShape {
    static constexpr int kForm = kForm_, kPair = kPair_, P = P_;
    static constexpr bool kAmn = kAmn_, kBmn = kBmn_;
    static constexpr bool kGrouped = kForm == kRows || kForm == kWeights;
    static constexpr int kParts = P == 6 ? 3 : 1;
    static constexpr int BN = P == 6 ? 128 : 256, TM = kPM * kPair;
    static constexpr uint32_t kA = kPM / kPBox * kPBoxBytes, kB = BN / kPair / kPBox * kPBoxBytes;
    static constexpr uint32_t kStage = kParts * (kA + kB);
    static constexpr bool kSum = P == 6 || kDrain_;
    // groups of four warps that finish tiles: some columns each where sums are in registers, else pieces of 32 in turn
    static constexpr int kCols = 64;
    static constexpr int kWarpGroups = kSum ? BN / kCols : kForm == kSlope ? 4 : 2;
    static constexpr int kThreads = 96 + kWarpGroups * 128;               // copy warp, product warp, clearing warp
    static constexpr int kStages = static_cast<int>((kGrouped ? 220 * 1024 : 225 * 1024) / kStage);
    static constexpr uint32_t kSmem = kStages * kStage + 1024;            // + alignment
    static constexpr int kAccCols = P == 6 ? 2 * BN : BN, kAccs = 2;
    static constexpr int kChunk = kSum ? 8 : INT32_MAX;                   // stages of an accumulator's turn
    static_assert(kStages >= 2 && kAccs * kAccCols == 512, "shape");
};

struct Tile {
    int e, split;            // group (kScore: item of its row of items) and part of K
    int m0, n0;              // first row of M (of the pair's) and column of N (kRows: row of the result)
    int valid, N;            // columns that count, and that the product has
    int k0, len;             // kWeights: the group's first row and rows
    int c0, c1;              // stages of K
};

__device__ __forceinline__ int up32(int x) { return (x + 31) & ~31; }

__device__ __forceinline__ bool sorted_groups(const ProductArgs& Q) { return Q.groups > 1 && Q.groups <= kMaxSorted; }

// Items of a launch (kRows: known once the groups' rows are).  All counts of items stay below 2^31 (see the entry points' limits).
template <class S>
__device__ __forceinline__ int items_of(const ProductArgs& Q, const uint32_t* start)
{
    if (S::kForm == kRows) return static_cast<int>(start[Q.groups]) * Q.splits;
    if (S::kForm == kWeights) return Q.groups * Q.m_tiles * Q.n_tiles * Q.splits;
    if (S::kForm == kScore) return (Q.n_tiles + Q.run - 1) / Q.run * Q.m_tiles;
    return Q.n_tiles * Q.m_tiles;
}

// Item t, at its first tile; `count` tiles.  The experts' tiles of a column of M follow one another (they share A), the
// score's token blocks of some columns do (they share the table's rows).
template <class S>
__device__ __forceinline__ Tile item_of(const ProductArgs& Q, const int* begin, const uint32_t* start, const uint16_t* order, int t, int& count)
{
    Tile T{};
    count = 1;
    if (S::kForm == kRows) {
        uint32_t u = t;
        if (Q.splits > 1) {
            u /= Q.splits;
            T.split = t - static_cast<int>(u) * Q.splits;
        }
        int lo = 0, hi = Q.groups;             // start[lo] <= u < start[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (start[mid] <= u)
                lo = mid;
            else
                hi = mid;
        }
        T.e = lo;
        const int rows = begin[T.e + 1] - begin[T.e], r = static_cast<int>(u - start[lo]);
        const int tiles = (rows + Q.width - 1) / Q.width;
        const int w = up32((rows + tiles - 1) / tiles);        // equal tiles; the last has a row at least
        const int across = r / tiles, i = r - across * tiles;
        T.m0 = across * S::TM;
        T.n0 = begin[T.e] + i * w;
        T.valid = min(w, rows - i * w);
        T.c1 = (Q.k + kPK - 1) / kPK;
    } else if (S::kForm == kWeights) {
        uint32_t u = t;
        if (Q.splits > 1) {
            u /= Q.splits;
            T.split = t - static_cast<int>(u) * Q.splits;
        }
        const uint32_t v = u / Q.m_tiles;
        T.m0 = static_cast<int>(u - v * Q.m_tiles) * S::TM;
        T.e = static_cast<int>(v / Q.n_tiles);
        T.n0 = static_cast<int>(v - T.e * Q.n_tiles) * Q.width;
        if (sorted_groups(Q)) T.e = order[T.e];
        T.valid = min(Q.width, Q.n - T.n0);
        T.k0 = begin[T.e];
        T.len = begin[T.e + 1] - T.k0;
        T.c1 = (T.len + kPK - 1) / kPK;
    } else {
        const uint32_t across = static_cast<uint32_t>(t) / Q.m_tiles;
        T.m0 = (t - static_cast<int>(across) * Q.m_tiles) * S::TM;
        if (S::kForm == kScore) {
            T.n0 = static_cast<int>(across) * Q.run * Q.width;
            count = min(Q.run, Q.n_tiles - static_cast<int>(across) * Q.run);
            T.e = static_cast<int>(across);
        } else {
            T.n0 = static_cast<int>(across) * Q.width;
        }
        T.valid = min(Q.width, Q.n - T.n0);
        T.c1 = (Q.k + kPK - 1) / kPK;
    }
    if (S::kGrouped && Q.splits > 1) {   // chunks shared out, the first parts one more
        const int each = T.c1 / Q.splits, more = T.c1 - each * Q.splits;
        T.c0 = T.split * each + min(T.split, more);
        T.c1 = T.c0 + each + (T.split < more ? 1 : 0);
    }
    T.N = up32(T.valid);
    return T;
}
// The item's next tile (kScore: the next columns).
__device__ __forceinline__ void next_tile(const ProductArgs& Q, Tile& T)
{
    T.n0 += Q.width;
    T.valid = min(Q.width, Q.n - T.n0);
    T.N = up32(T.valid);
}

__device__ __forceinline__ float exp2_fast(float x)   // 2 ulp
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b)
{
    const __nv_bfloat162 q = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&q);
}
__device__ __forceinline__ float2 pair_floats(uint32_t q)
{
    return make_float2(__uint_as_float(q << 16), __uint_as_float(q & 0xffff0000u));
}

// A lane's row f of M in 32 columns: neighbours of one row of the result in a warp's lanes.
template <class S>
__device__ __forceinline__ void put_columns(const ProductArgs& Q, const Tile& T, int f, int col, const float (&v)[32])
{
    if (f >= Q.m) return;
    const int have = T.valid - col;
    const int64_t row = S::kForm == kRows ? T.n0 + col : static_cast<int64_t>(T.e) * Q.n + T.n0 + col;
    const int64_t at = row * Q.ld + f + T.split * Q.slab;
    float x[32];
    const float unit = Q.unit != nullptr ? *Q.unit : 1.0f;
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = v[e] * unit;
    if (Q.add != nullptr)
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if (e < have) x[e] += Q.add[at + static_cast<int64_t>(e) * Q.ld];
    if (Q.out_bf16) {
        bf16* to = static_cast<bf16*>(Q.out) + at;
#pragma unroll
        for (int e = 0; e < 32; ++e, to += Q.ld)
            if (e < have) *to = __float2bfloat16_rn(x[e]);
    } else {
        float* to = static_cast<float*>(Q.out) + at;
#pragma unroll
        for (int e = 0; e < 32; ++e, to += Q.ld)
            if (e < have) *to = x[e];
    }
}

// Slopes that leave as bf16 are first divided by this, the significand (1 to 2) of the first dloss of a token that counts (among 1024), and the products
// with them multiplied by it.  Where all tokens have one dloss, as under a mean, a token's largest slope is then a
// power of two less a probability; as dloss itself it would be rounded the same way for every token, by up to 2^-8 of all results.
// By a warp.
__device__ __forceinline__ float common_unit(const float* dloss, const int64_t* target, int n, int lane)
{
    if (dloss == nullptr) return 1.0f;
    for (int i0 = 0; i0 < min(n, 1024); i0 += 32) {
        const int i = i0 + lane;
        float d = 0.0f;
        if (i < n && target[i] >= 0) d = dloss[i];
        const uint32_t votes = __ballot_sync(kFull, d != 0.0f && isfinite(d));
        if (votes != 0) {
            d = __shfl_sync(kFull, d, __ffs(votes) - 1);
            return __uint_as_float((__float_as_uint(d) & 0x007fffffu) | 0x3f800000u);
        }
    }
    return 1.0f;
}

// The slopes of a lane's token in 32 of the table's rows: dloss (softmax - [target]).
template <class S>
__device__ __forceinline__ void put_slopes(const ProductArgs& Q, const Tile& T, int row, int col, float lse2, float scale, int target,
                                           const float (&v)[32])
{
    const int c0 = T.n0 + col, left = Q.n - c0;
    if (row >= Q.rows || left <= 0) return;
    float x[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = exp2_fast(fmaf(v[e], kLog2e, -lse2));
    const int hit = target - Q.v0 - c0;
    if (static_cast<uint32_t>(hit) < 32u)
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if (e == hit) x[e] -= 1.0f;
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = target >= 0 ? x[e] * scale : 0.0f;   // a token without one leaves nothing, whatever its scores
    bf16* to = Q.slope + static_cast<int64_t>(row) * Q.ld + c0;
#pragma unroll
    for (int p = 0; p < S::kParts; ++p) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            uint32_t u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float &a = x[q * 16 + 2 * e], &b = x[q * 16 + 2 * e + 1];
                u[e] = bf16_pair(a, b);
                if (p + 1 < S::kParts) {
                    const float2 h = pair_floats(u[e]);
                    a -= h.x, b -= h.y;
                }
            }
            if (q * 16 < left) stg256(to + p * Q.slope_part + q * 16, u);   // rows are padded to 16
        }
    }
}

// 32 more scores of a lane's token: running maximum and sum.
__device__ __forceinline__ void take_scores(const ProductArgs& Q, const Tile& T, int row, int col, int target, float& top, float& sum,
                                            float (&z)[32])
{
    const int c0 = T.n0 + col, left = Q.n - c0;
    if (left <= 0) return;
    if (left < 32)
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if (e >= left) z[e] = -INFINITY;
    const int hit = target - c0;
    if (static_cast<uint32_t>(hit) < 32u) {
        float mine = 0.0f;
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if (e == hit) mine = z[e];
        Q.hit[row] = mine;
    }
    float t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] = fmaxf(z[e], z[e + 4]);
#pragma unroll
    for (int e = 8; e < 32; ++e) t[e & 3] = fmaxf(t[e & 3], z[e]);
    const float high = fmaxf(top, fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])));
    const float base = high == -INFINITY ? 0.0f : high * kLog2e;   // nothing but -inf so far: sums of 0
    float s[4] = {sum * exp2_fast(fmaf(top, kLog2e, -base)), 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 32; ++e) s[e & 3] += exp2_fast(fmaf(z[e], kLog2e, -base));
    sum = (s[0] + s[1]) + (s[2] + s[3]);
    top = high;
}

// Zeros in `count` values from `at` on, by all finishing warps of the grid.
template <class T>
__device__ __forceinline__ void clear_values(T* at, int64_t count, int64_t first, int64_t step)
{
    const int64_t head = min(count, static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(at) & 15)) & 15) / static_cast<int64_t>(sizeof(T)));
    constexpr int V = 16 / sizeof(T);
    const int64_t body = (count - head) / V;
    uint4* v = reinterpret_cast<uint4*>(at + head);
    for (int64_t i = first; i < body; i += step) v[i] = make_uint4(0, 0, 0, 0);
    for (int64_t i = first; i < head; i += step) at[i] = T(0.0f);
    for (int64_t i = head + body * V + first; i < count; i += step) at[i] = T(0.0f);
}

// One block an SM (or one pair of blocks on two), items in turn: warp 0 copies boxes of 64 K values of A and B
// into a ring of stages, warp 1 (of the pair's first block) issues the products into one of two
// accumulators, warp 2 clears what lies behind a group's last row, groups of four warps finish the other
// accumulator.  In shared memory every box has 64 rows of 128 bytes, 16-byte pieces permuted by
// row (the copies' 128-byte swizzle).
template <class S>
__global__ void __launch_bounds__(S::kThreads, 1) k_product(const __grid_constant__ ProductMaps maps, const ProductArgs Q)
{
    constexpr int kForm = S::kForm, kPair = S::kPair, kStages = S::kStages, P = S::P;
    constexpr bool kAmn = S::kAmn, kBmn = S::kBmn;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[3 * kStages + 2 * S::kAccs + 1];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int dead;
    __shared__ int begin[S::kGrouped ? kMaxGroups + 1 : 1];
    __shared__ uint32_t start[kForm == kRows ? kMaxGroups + 1 : 1];   // first item of the groups
    __shared__ uint16_t order[kForm == kWeights ? kMaxSorted : 1];    // the groups by length
    const uint32_t data = (smem_addr(raw) + 1023u) & ~1023u;
    const uint32_t full = smem_addr(bars), empty = full + 8 * kStages, tfull = empty + 8 * kStages,
                   tempty = tfull + 8 * S::kAccs, drain = tempty + 8 * S::kAccs, fix = drain + 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = kPair == 2 ? static_cast<int>(cluster_rank()) : 0;
    const int first = blockIdx.x / kPair, step = gridDim.x / kPair;

    if (threadIdx.x == 32) {   // while the kernel before ends
        tma_prefetch(&maps.a);
        tma_prefetch(&maps.b);
    }
    if (threadIdx.x == 0) {
        dead = 0;
        // (kWeights: each block of a pair says so when its boxes are requested, or cleared and there)
        for (int s = 0; s < kStages; ++s) mbar_init(full + 8 * s, kForm == kWeights ? kPair : 1), mbar_init(empty + 8 * s, 1);
        for (int s = 0; s < S::kAccs; ++s) mbar_init(tfull + 8 * s, 1), mbar_init(tempty + 8 * s, 4 * S::kWarpGroups * kPair);
        for (int s = 0; s < kStages; ++s) mbar_init(fix + 8 * s, 1);
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<kPair>(&tmem_slot, 512);
    tc_fence_before();
    if (kPair == 2)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_wait();
    if (Q.release) pdl_release();   // after this block's allocation, so that no later block can hold what it waits for
    fence_async_proxy();            // the kernels before wrote with ordinary stores

    bool sound = true;
    if (S::kGrouped) {
        if (Q.offsets != nullptr) {
            bool wrong = false;
            for (int e = threadIdx.x; e <= Q.groups; e += S::kThreads) {
                const int64_t o = Q.offsets[e], before = e > 0 ? Q.offsets[e - 1] : 0;
                wrong |= o < before || o > Q.rows || (e == 0 && o != 0);
                begin[e] = static_cast<int>(o);
            }
            sound = __syncthreads_or(wrong) == 0;
            if (!sound && blockIdx.x == 0 && threadIdx.x == 0) set_error(Q.d_err, SPARSE_ERR_INDEX_OUT_OF_RANGE);
        } else {
            if (threadIdx.x == 0) begin[0] = 0, begin[1] = Q.rows;
            __syncthreads();
        }
        // Items go to the blocks in turn: with the longest groups first neighbours are alike and the blocks' sums even out (16384 x 8 rows
        // among 128 experts of uneven favour: 448 against 402 us).  kRows' tiles differ by their width alone, and took longer that way (304
        // against 285 us there).
        if (kForm == kWeights && sound && sorted_groups(Q)) {
            for (int e = threadIdx.x; e < Q.groups; e += S::kThreads) {
                const int mine = begin[e + 1] - begin[e];
                int rank = 0;
                for (int f = 0; f < Q.groups; ++f) {
                    const int rows = begin[f + 1] - begin[f];
                    rank += rows > mine || (rows == mine && f < e) ? 1 : 0;
                }
                order[rank] = static_cast<uint16_t>(e);
            }
            __syncthreads();
        }
        if (kForm == kRows && sound) {
            if (warp == 0) {
                uint32_t base = 0;
                for (int e0 = 0; e0 < Q.groups; e0 += 32) {
                    const int e = e0 + lane;
                    const uint32_t mine = e < Q.groups ? static_cast<uint32_t>((begin[e + 1] - begin[e] + Q.width - 1) / Q.width * Q.m_tiles) : 0u;
                    const uint32_t incl = warp_incl_scan(mine, lane);
                    if (e < Q.groups) start[e] = base + incl - mine;
                    base += __shfl_sync(kFull, incl, 31);
                }
                if (lane == 0) start[Q.groups] = base;
            }
            __syncthreads();
        }
    }
    const int items = sound ? items_of<S>(Q, start) : 0;

    if (warp == 0) {
        if (elect_one()) {
            uint32_t it = 0, fixed = 0, turn = 0;   // stages; those that warp 2 has had at all, and (parity) how often
            for (int t = first; t < items; t += step) {
                int count;
                Tile T = item_of<S>(Q, begin, start, order, t, count);
                for (int j = 0; j < count; ++j, next_tile(Q, T)) {
                    const int boxes = (T.N / kPair + kPBox - 1) / kPBox;
                    const uint32_t bytes = S::kParts * (S::kA + boxes * kPBoxBytes);
                    const int m0 = T.m0 + rank * kPM, n0 = T.n0 + rank * (T.N / kPair);
                    for (int c = T.c0; c < T.c1; ++c, ++it) {
                        const uint32_t s = it % kStages;
                        if (!mbar_wait(empty + 8 * s, (it / kStages & 1) ^ 1, &dead)) goto copied;
                        const bool tail = kForm == kWeights && (c + 1) * kPK > T.len;   // goes by way of warp 2
                        const uint32_t there = kPair == 2 ? cluster_addr(full + 8 * s, 0) : full + 8 * s;
                        const uint32_t bar = tail ? fix + 8 * s : there;
                        if (tail)
                            mbar_expect(bar, bytes), fixed |= 1u << s, turn ^= 1u << s;
                        else if (rank == 0)
                            mbar_expect(full + 8 * s, kPair * bytes);
                        else if (kForm == kWeights)
                            mbar_arrive_relaxed(there);
                        uint32_t at = data + s * S::kStage;
                        const int kk = kForm == kWeights ? T.k0 + c * kPK : c * kPK;
                        auto load = [&](const CUtensorMap* map, int x, int y, int z) {
                            if (tail)
                                tma_load<1>(at, map, bar, x, y, z);
                            else
                                tma_load<kPair>(at, map, bar, x, y, z);
                            at += kPBoxBytes;
                        };
#pragma unroll
                        for (int p = 0; p < S::kParts; ++p) {
                            const int z = kForm == kRows ? p * Q.groups + T.e : p;
#pragma unroll
                            for (int q = 0; q < kPM / kPBox; ++q) {
                                if (kAmn)
                                    load(&maps.a, m0 + q * kPBox, kk, z);
                                else
                                    load(&maps.a, kk, m0 + q * kPBox, z);
                            }
                        }
#pragma unroll
                        for (int p = 0; p < S::kParts; ++p) {
                            at = data + s * S::kStage + S::kParts * S::kA + p * S::kB;
                            for (int q = 0; q < boxes; ++q) {
                                if (kBmn)
                                    load(&maps.b, n0 + q * kPBox, kk, p);
                                else
                                    load(&maps.b, kk, n0 + q * kPBox, p);
                            }
                        }
                    }
                }
            }
        copied:
            if (dead) {   // copies in flight land before the blocks leave
                volatile int none = 0;
                for (uint32_t s = 0; s < static_cast<uint32_t>(kStages) && s < it; ++s) {
                    const uint32_t last = (it - 1 - s) / kStages * kStages + s;   // the stage's last use
                    if (rank == 0) mbar_wait(full + 8 * s, last / kStages & 1, &none);
                    if (fixed >> s & 1) mbar_wait(fix + 8 * s, (turn >> s & 1) ^ 1, &none);
                }
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            constexpr uint32_t idesc = mma_desc_bf16(S::TM, kAmn, kBmn);
            uint32_t it = 0, done = 0;   // stages, accumulators used
            bool ok = true;
            for (int t = first; ok && t < items; t += step) {
                int count;
                Tile T = item_of<S>(Q, begin, start, order, t, count);
                for (int j = 0; ok && j < count; ++j, next_tile(Q, T)) {
                    const uint32_t what = idesc | static_cast<uint32_t>(T.N >> 3) << 17;
                    for (int c = T.c0; ok && c < T.c1; ++done) {
                        const uint32_t acc = done % S::kAccs;
                        if (!(ok = mbar_wait(tempty + 8 * acc, (done / S::kAccs & 1) ^ 1, &dead))) break;
                        tc_fence_after();
                        const uint32_t d = tmem + acc * S::kAccCols;
                        for (int part = 0; part < S::kChunk && c < T.c1; ++part, ++c, ++it) {
                            const uint32_t s = it % kStages;
                            if (!(ok = mbar_wait(full + 8 * s, it / kStages & 1, &dead))) break;
                            if (kForm == kWeights && kPair == 2 && (c + 1) * kPK > T.len)
                                mbar_acquire_cluster(full + 8 * s, it / kStages & 1);   // the other block's warp 2 cleared rows
                            tc_fence_after();
                            const uint32_t a = data + s * S::kStage, b = a + S::kParts * S::kA;
                            // 16 K values: 32 bytes along a K-major row, two 8-row groups of an MN-major block
                            const int steps = kForm == kWeights ? min(kPK / 16, (T.len - c * kPK + 15) / 16) : kPK / 16;
#pragma unroll
                            for (int k = 0; k < kPK / 16; ++k) {
                                if (kForm == kWeights && k >= steps) break;
                                const uint32_t ak = a + (kAmn ? k * 2048 : k * 32), bk = b + (kBmn ? k * 2048 : k * 32);
                                auto da = [&](int p) { return smem_desc(ak + p * S::kA, kAmn ? kPBoxBytes : 16, 1024); };
                                auto db = [&](int p) { return smem_desc(bk + p * S::kB, kBmn ? kPBoxBytes : 16, 1024); };
                                const bool more = part + k > 0;
                                tc_mma_f16<kPair>(d, da(0), db(0), what, more);
                                if (P == 6) {
                                    tc_mma_f16<kPair>(d + S::BN, da(0), db(2), what, more);
                                    tc_mma_f16<kPair>(d + S::BN, da(2), db(0), what, true);
                                    tc_mma_f16<kPair>(d + S::BN, da(1), db(1), what, true);
                                    tc_mma_f16<kPair>(d + S::BN, da(0), db(1), what, true);
                                    tc_mma_f16<kPair>(d + S::BN, da(1), db(0), what, true);
                                }
                            }
                            tc_commit<kPair>(empty + 8 * s);
                        }
                        if (ok) tc_commit<kPair>(tfull + 8 * acc);
                    }
                }
            }
            if (dead) {   // products in flight finish before the blocks leave
                volatile int none = 0;
                tc_commit<kPair>(drain);
                mbar_wait(drain, 0, &none);
            }
        }
    } else if (warp == 2) {
        if (kForm == kWeights) {
            uint32_t it = 0, turn = 0;
            bool ok = true;
            for (int t = first; ok && t < items; t += step) {
                int count;
                const Tile T = item_of<S>(Q, begin, start, order, t, count);
                it += T.c1 - T.c0;
                if (T.c1 == T.c0 || T.c1 * kPK <= T.len) continue;   // no last stage, or a whole one
                const uint32_t s = (it - 1) % kStages;
                ok = __all_sync(kFull, mbar_wait(fix + 8 * s, turn >> s & 1, &dead));
                turn ^= 1u << s;
                if (!ok) break;
                const int from = T.len - (T.c1 - 1) * kPK, to = (from + 15) & ~15;   // the product reads 16 rows at a time
                const int boxes = (T.N / kPair + kPBox - 1) / kPBox;
                const uint32_t at = data + s * S::kStage;
                for (int p = 0; p < S::kParts; ++p)
                    for (int q = 0; q < kPM / kPBox + boxes; ++q) {
                        const uint32_t box = q < kPM / kPBox ? at + p * S::kA + q * kPBoxBytes
                                                             : at + S::kParts * S::kA + p * S::kB + (q - kPM / kPBox) * kPBoxBytes;
                        for (int i = from * 8 + lane; i < to * 8; i += 32) sts128(box + i * 16, make_uint4(0, 0, 0, 0));
                    }
                fence_async_proxy();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(kPair == 2 ? cluster_addr(full + 8 * s, 0) : full + 8 * s);
            }
        }
    } else {
        constexpr int kWarpGroups = S::kWarpGroups;
        const int group = (warp - 3) >> 2, id = 1 + group;
        const int rowl = (warp & 3) * 32 + lane;   // the tensor memory lanes this warp can read
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        if (kForm == kRows && Q.clear && sound) {
            const int64_t from = static_cast<int64_t>(begin[Q.groups]) * Q.ld, count = static_cast<int64_t>(Q.rows) * Q.ld - from;
            const int64_t mine = static_cast<int64_t>(blockIdx.x) * (S::kThreads - 96) + threadIdx.x - 96,
                          all = static_cast<int64_t>(gridDim.x) * (S::kThreads - 96);
            if (Q.out_bf16)
                clear_values(static_cast<bf16*>(Q.out) + from, count, mine, all);
            else
                clear_values(static_cast<float*>(Q.out) + from, count, mine, all);
        }
        float unit = 1.0f;
        if (kForm == kSlope && S::kParts == 1) {
            unit = common_unit(Q.dloss, Q.target, Q.rows, lane);
            if (blockIdx.x == 0 && threadIdx.x == 96) *Q.unit = unit;
        }
        uint32_t done = 0;
        bool ok = true;
        auto leave = [&](uint32_t acc) {   // this warp has read all of the accumulator that it wants
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_near(kPair == 2 ? cluster_addr(tempty + 8 * acc, 0) : tempty + 8 * acc);
        };
        for (int t = first; ok && t < items; t += step) {
            int count;
            Tile T = item_of<S>(Q, begin, start, order, t, count);
            const int f = T.m0 + rank * kPM + rowl;
            float top = -INFINITY, total = 0.0f;      // kScore
            float lse2 = 0.0f, scale = 0.0f;          // kSlope
            int target = -1, row = 0;
            for (int j = 0; ok && j < count; ++j, next_tile(Q, T)) {
                if (!S::kGrouped && j == 0) {
                    row = f;
                    if (row < Q.rows) {
                        const int64_t g = Q.target[row];
                        if (g < -1 || g >= Q.v) set_error(Q.d_err, SPARSE_ERR_INDEX_OUT_OF_RANGE);
                        target = g < 0 || g >= Q.v ? -1 : static_cast<int>(g);
                        if (kForm == kSlope) {
                            lse2 = Q.lse[row] * kLog2e;
                            scale = Q.dloss ? __fdiv_rn(Q.dloss[row], unit) : 1.0f;
                        }
                    }
                }
                if (S::kSum) {
                    constexpr int kCols = S::kCols;
                    float sum[kCols / 32][32];
                    if (P == 1 || T.c0 == T.c1)   // (with one product first values in their place cost 500 bytes of spills)
#pragma unroll
                        for (int q = 0; q < kCols; ++q) sum[q / 32][q % 32] = 0.0f;
#pragma unroll 1
                    for (int c = T.c0; c < T.c1; c += min(S::kChunk, T.c1 - c), ++done) {
                        const uint32_t acc = done % S::kAccs;
                        if (!(ok = all_of(id, 128, mbar_wait(tfull + 8 * acc, done / S::kAccs & 1, &dead)))) break;
                        tc_fence_after();
                        if (group * kCols < T.N) {
#pragma unroll
                            for (int q = 0; q < kCols / 16; ++q) {
                                const uint32_t from = lanes + acc * S::kAccCols + group * kCols + q * 16;
                                float v[16];
                                if constexpr (P == 6) {
                                    float x[16];
                                    tmem_load16(from, from + S::BN, v, x);
#pragma unroll
                                    for (int e = 0; e < 16; ++e) v[e] += x[e];
                                } else {
                                    tmem_load16(from, v);
                                }
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    float& to = sum[q / 2][q % 2 * 16 + e];
                                    to = P == 6 && c == T.c0 ? v[e] : to + v[e];
                                }
                            }
                        }
                        leave(acc);
                    }
                    if (!ok) break;
#pragma unroll
                    for (int q = 0; q < kCols / 32; ++q) {
                        const int col = group * kCols + q * 32;
                        if (col >= T.valid) break;
                        if (kForm == kScore)
                            take_scores(Q, T, row, col, target, top, total, sum[q]);
                        else if (kForm == kSlope)
                            put_slopes<S>(Q, T, row, col, lse2, scale, target, sum[q]);
                        else
                            put_columns<S>(Q, T, f, col, sum[q]);
                    }
                } else {
                    const bool some = T.c1 > T.c0;
                    const uint32_t acc = done % S::kAccs;
                    if (some) {
                        if (!(ok = all_of(id, 128, mbar_wait(tfull + 8 * acc, done / S::kAccs & 1, &dead)))) break;
                        tc_fence_after();
                        ++done;
                    }
                    for (int col = group * 32; col < T.valid; col += kWarpGroups * 32) {
                        float v[32];
                        if (some)
                            tmem_load32(lanes + acc * S::kAccCols + col, v);
                        else
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = 0.0f;
                        if (some && col + kWarpGroups * 32 >= T.valid) leave(acc);   // the last piece: the accumulator is free
                        if (kForm == kScore)
                            take_scores(Q, T, row, col, target, top, total, v);
                        else if (kForm == kSlope)
                            put_slopes<S>(Q, T, row, col, lse2, scale, target, v);
                        else
                            put_columns<S>(Q, T, f, col, v);
                    }
                    if (some && group * 32 >= T.valid) leave(acc);
                }
            }
            if (kForm == kScore && ok && row < Q.rows)
                Q.part[static_cast<int64_t>(T.e * kWarpGroups + group) * Q.rows + row] = make_float2(top, total);
        }
    }
    __syncwarp();
    tc_fence_before();
    if (kPair == 2)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    if (dead && threadIdx.x == 0) set_error(Q.d_err, SPARSE_ERR_INTERNAL);
    if (warp == 1) tmem_free<kPair>(tmem, 512);
}

// -------------------------------------------------------------------- host
// Boxes of 64 rows x 64 values of `batch` matrices of rows x cols bf16 values, rows `ld` and matrices `step` values apart;
// zeros beyond.
inline bool encode_bf16(CUtensorMap* map, const void* at, int64_t rows, int64_t cols, int64_t ld, int64_t batch, int64_t step)
{
    const cuuint64_t dim[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(batch)};
    const cuuint64_t stride[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(step) * 2};
    const cuuint32_t box[3] = {kPK, kPBox, 1}, each[3] = {1, 1, 1};
    return tensor_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(at), dim, stride, box, each,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What a stage of a tile of w columns takes, in cycles: 128 rows x w x 64 products an SM at 4096 a cycle, or its boxes from L2
// at about 80 bytes a cycle and SM, whichever is longer.
template <class S>
int64_t stage_cycles(int64_t w)
{
    return std::max<int64_t>(2 * w * S::P, S::kParts * (kPM + w / S::kPair) * 128 / 80);
}

// `items` at most, each a block's (a pair's) at a time.
template <class S>
cudaError_t run_product(const char* name, const ProductMaps& maps, const ProductArgs& Q, int64_t items, cudaStream_t s)
{
    auto* kernel = k_product<S>;
    const cudaError_t ready = allow_smem(kernel, S::kSmem, S::kSmem);
    if (ready != cudaSuccess) return ready;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(items, num_sms() / S::kPair)) * S::kPair));
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = S::kPair;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    SO_PROFILE(name, s);
    return cudaLaunchKernelEx(&cfg, kernel, maps, Q);
}

// An operand: bf16 values as they lie in memory, or `parts` bf16 arrays in the workspace.
struct Operand {
    const void* at;
    int64_t rows, cols, ld;   // of one matrix
    int64_t batch;            // matrices
    int parts;
    int64_t step = 0;         // values between matrices, where they do not follow one another
    bool map(CUtensorMap* m) const { return encode_bf16(m, at, rows, cols, ld, batch * parts, step > 0 ? step : rows * ld); }
};

// Rows of an array copied into the workspace start on 128-byte lines, so that boxes read whole ones; short ones on 16 bytes.
inline int64_t packed_ld(int64_t cols) { return cols >= 256 ? (cols + 63) / 64 * 64 : (cols + 7) / 8 * 8; }

// One array to be packed: rows x cols values, fp32 into three parts or bf16 into one with aligned rows.
// With offsets the rows are those of matrices of `each` rows, and a matrix whose group has no rows is left out.  With targets a
// row whose target is none of v rows is zeros, whatever lies there.
struct Pack1 {
    const void* from;
    bf16* to;
    int64_t rows, cols, ld;
    const int64_t* offsets = nullptr;
    int64_t each = 1;
    const int64_t* target = nullptr;
    int64_t v = 0;
};
// The tokens' numbers for the loss's gradient: lse log2(e), dloss (over the unit, where one is asked for) and target, 0 and -1 for
// a token that does not count and behind the last (vocab_back.cu).
struct TokenRows {
    const float *lse, *dloss;
    const int64_t* target;
    int n, padded, v;
    float4* out;
    float* unit;
    int32_t* d_err;
};
__device__ __forceinline__ void put_token(const TokenRows& R, int i, float unit)
{
    if (i >= R.padded) return;
    float4 q = make_float4(0.0f, 0.0f, __int_as_float(-1), 0.0f);
    if (i < R.n) {
        const int64_t g = R.target[i];
        if (g < -1 || g >= R.v) set_error(R.d_err, SPARSE_ERR_INDEX_OUT_OF_RANGE);
        if (g >= 0 && g < R.v)
            q = make_float4(R.lse[i] * kLog2e, R.dloss ? __fdiv_rn(R.dloss[i], unit) : 1.0f, __int_as_float(static_cast<int>(g)), 0.0f);
    }
    R.out[i] = q;
}

// Up to two arrays in one launch (either's rows may be 0), and the tokens' numbers and their unit (padded may be 0).
cudaError_t pack(const Pack1& a, const Pack1& b, const TokenRows& tokens, int is_bf16, cudaStream_t s);

// rows x cols fp32 sums of `slabs` arrays, in order; rows from *end on (end given) are zeros.
struct Join {
    const float* from;
    int slabs;
    int64_t slab, rows, cols;
    const int64_t* end;
};
cudaError_t join_slabs(const Join& J, void* out, int out_bf16, cudaStream_t s);
cudaError_t join_two(const Join& a, void* out_a, const Join& b, void* out_b, int out_bf16, cudaStream_t s);

// The product of rows with their group's matrix, and of two arrays of rows (product_rows.cu, product_weights.cu): fills in the rest of Q
// (extents, tiles); `pieces`: sums are added to what `out` (fp32 slabs) holds.
struct RowsProduct {
    Operand a, b;            // the matrices [groups], K x M (MN-major A) or M x K; the rows [rows, K]
    int a_mn;
    int64_t rows, m, k;
    int groups;
    const int64_t* offsets;
    int splits;
    void* out;
    int out_bf16, add, clear, release;
    float* unit;
    int32_t* d_err;
};
int rows_splits(int64_t rows, int64_t m, int64_t k, int64_t groups, int parts);
cudaError_t rows_product(const RowsProduct& R, cudaStream_t s);

struct WeightsProduct {
    Operand a, b;            // rows x M, rows x N
    int64_t rows, m, n;
    int groups;
    const int64_t* offsets;
    int splits;
    void* out;               // [groups, n, m]
    int out_bf16, release;
    float* unit;
    int32_t* d_err;
};
int weights_splits(int64_t rows, int64_t m, int64_t n, int64_t groups, int parts);
cudaError_t weights_product(const WeightsProduct& R, cudaStream_t s);

}  // namespace so
