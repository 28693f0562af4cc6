// muon.cu -- an update orthogonalised by Newton-Schulz products, and the Muon step
// that applies it.
//
// For each r x c matrix u of a batch, with X of m = min(r, c) rows and n = max(r, c)
// columns (u or its transpose):
//   X = u / (|u|_F + eps), then `steps` times
//   A = X X^T, B = b A + c A^2, X = a X + B X
// drives every singular value of X towards 1 (a fixed polynomial in each of them).
//
// Matrix products run on the tcgen05 unit with f16 operands and fp32 accumulators.
// f16, because its 11-bit significand is eight times finer than bf16's and its
// range suffices: singular values stay below kMaxSigma, so X, A and B, scaled by
// kScale, stay below 65504, and what is below the normal range there is below
// 2^-28 of the scale.  Every matrix is held as hi = f16(v), lo = f16(v - hi):
//   products = 3  hi hi + hi lo + lo hi: 22 bits, as accurate as fp32 products;
//   products = 1  hi hi.  A is used as rounded in both b A and c A^2 (the
//                 polynomial of a nearby A: its error near singular value 1 is
//                 half that of b A exact, c A^2 rounded), and X's lo part is added,
//                 times a, in every step but the last (there the small singular
//                 values, tripled by a step, would drown in the rounding of the
//                 large ones: 2e-2 of a low-rank matrix; in the last step X as
//                 rounded is the better polynomial).  In a 64-bit simulation (more than 128 rows) at
//                 most 1.7e-3 of the result's norm over flat, decaying and low-rank spectra and 2.5e-3
//                 for rank one, about what rounding it to bf16 costs.
//                 B is formed with a on its diagonal, so that B X holds a X.
// (With three products a X is added in the epilogue: in the tensor unit's sums, which
// round towards zero, it cost a low-rank matrix 4e-5.  Simulated as above: 5e-7 flat, 6.5e-6 low rank, 3.6e-5
// for rank one, where fp32 products give 1e-4.)
#include <algorithm>

#include "muon.cuh"
#include "profile.cuh"

namespace so {

namespace {

constexpr int kBM = 128, kBK = 64;              // rows of a block's tile; K values of a stage (128 bytes)
constexpr int kBox = 64;                        // rows of one copied box: 64 x 128 bytes
constexpr uint32_t kBoxBytes = kBox * kBK * 2;
constexpr int kSub = 64;                        // columns the epilogue finishes at a time
constexpr int kGroup = 128;                     // threads of an epilogue group
constexpr int64_t kNormParts = 1024;            // partial sums of squares of a matrix at most

// ------------------------------------------------------------------- start
// Sums of squares of one matrix's pieces, where they are small (a matrix of zeros among them) also of the
// values times kRaise; a sum that is not finite is reported before anything is written.  E: values
// of an access.
template <int E>
__global__ void __launch_bounds__(kMuonBlock) k_muon_norm(Update U, int64_t size, int parts, float2* __restrict__ part,
                                                          uint32_t* verdict, int32_t* d_err)
{
    pdl_enter();   // writes the workspace and the error word only
    if (blockIdx.x == 0 && threadIdx.x == 0) *verdict = kUndecided;
    __shared__ float tmp[2 * 32];
    const int mat = static_cast<int>(blockIdx.x) / parts, p = static_cast<int>(blockIdx.x) % parts;
    const int64_t base = mat * size, step = static_cast<int64_t>(parts) * kMuonBlock * E;
    const int64_t first = (static_cast<int64_t>(p) * kMuonBlock + threadIdx.x) * E;
    constexpr int R = E == 1 ? 8 : 4;   // accesses a lane requests at once
    float s[1] = {0.0f}, raised[1] = {0.0f};
    for (int64_t i = first; i < size; i += R * step) {
        float u[R][E], nb[E];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            if (i + q * step < size)
                read_u<E>(U, base + i + q * step, u[q], nb);
            else
#pragma unroll
                for (int e = 0; e < E; ++e) u[q][e] = 0.0f;
        }
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
            for (int e = 0; e < E; ++e) s[0] = fmaf(u[q][e], u[q][e], s[0]);
    }
    block_sum<1>(s, kMuonBlock, tmp, 0);
    if (s[0] < kSmallSquares) {   // the same for the whole block
#pragma unroll 1
        for (int64_t i = first; i < size; i += step) {
            float u[E], nb[E];
            read_u<E>(U, base + i, u, nb);
#pragma unroll
            for (int e = 0; e < E; ++e) raised[0] = fmaf(u[e] * kRaise, u[e] * kRaise, raised[0]);
        }
        block_sum<1>(raised, kMuonBlock, tmp, 1);
    }
    if (threadIdx.x == 0) {
        part[blockIdx.x] = make_float2(s[0], raised[0]);
        if (!isfinite(s[0] * static_cast<float>(parts))) set_error(d_err, SPARSE_ERR_NON_FINITE);   // nor may the whole overflow
    }
}

// X = u / (|u| + eps), scaled and split, and the new momentum buffer, where X lies as u does (wide,
// whole 16-byte accesses): `pieces` blocks a matrix, 8 accesses of 8 values a thread (fewer, larger
// blocks are busy for less time with the scale, which each works out: 16 x 768 x 2048 bf16, 150 MB, 31
// us; 4 accesses 36 us, 32 accesses 33 us).
__global__ void __launch_bounds__(kMuonBlock) k_muon_start_flat(Update U, float* __restrict__ buf, int64_t size, int pieces,
                                                                const float2* __restrict__ part, int parts, float eps, float eps_raised,
                                                                __half* __restrict__ hi, __half* __restrict__ lo,
                                                                int c, int64_t ldn, uint32_t* verdict, const int32_t* d_err)
{
    pdl_enter();   // writes the workspace and optimizer state only
    __shared__ float sums[2 * 32];
    __shared__ bool goes;
    if (threadIdx.x == kMuonBlock - 1) goes = buf == nullptr || step_goes(verdict, d_err);
    const int mat = static_cast<int>(blockIdx.x) / pieces, p = static_cast<int>(blockIdx.x) % pieces;
    const int64_t base = mat * size, step = static_cast<int64_t>(pieces) * kMuonBlock * 8;
    const int64_t rows = size / c;
    float scale = 0.0f;
    bool scaled = false;
    for (int64_t i = (static_cast<int64_t>(p) * kMuonBlock + threadIdx.x) * 8; i - threadIdx.x * 8 < size; i += step) {
        float u[8], nb[8];
        if (i < size) read_u<8>(U, base + i, u, nb);
        if (!scaled) {   // while those are on their way
            scaled = true;
            scale = start_scale<kMuonBlock>(part + static_cast<int64_t>(mat) * parts, parts, eps, eps_raised, sums);
            if (!goes) return;   // (start_scale's barrier lies between)
        }
        if (i >= size) continue;
        if (buf) Pack<float, 8>::put(buf + base + i, nb);
        const int64_t to = ldn == c ? base + i : (mat * rows + i / c) * ldn + i % c;
        uint4 h, l;
        __half2* hh = reinterpret_cast<__half2*>(&h);
        __half2* ll = reinterpret_cast<__half2*>(&l);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float a = x_of(u[2 * e], scale), b = x_of(u[2 * e + 1], scale);
            hh[e] = __floats2half2_rn(a, b);
            const float2 f = __half22float2(hh[e]);
            ll[e] = __floats2half2_rn(a - f.x, b - f.y);
        }
        *reinterpret_cast<uint4*>(hi + to) = h;
        if (lo) *reinterpret_cast<uint4*>(lo + to) = l;
    }
}

// X = u / (|u| + eps), scaled and split, transposed where u is tall; the new momentum
// buffer.  One 64 x 64 tile of u at a time, four values a thread.  (Five blocks an SM: with four the 640 tiles of
// 2501 x 1003 go round twice, 12 us and not 10.)
template <bool kVec>
__global__ void __launch_bounds__(kMuonBlock, 5) k_muon_start(Update U, float* __restrict__ buf, int64_t r, int64_t c,
                                                           int tiles_c, int tiles, int ntiles,
                                                           const float2* __restrict__ part, int parts, float eps, float eps_raised,
                                                           __half* __restrict__ hi, __half* __restrict__ lo,
                                                           int64_t ldn, int tall, uint32_t* verdict, const int32_t* d_err)
{
    pdl_enter();   // writes the workspace and optimizer state only
    __shared__ float tile[64][65];
    __shared__ float sums[2 * 32];
    __shared__ bool goes;
    if (threadIdx.x == kMuonBlock - 1) goes = buf == nullptr || step_goes(verdict, d_err);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t m = tall ? c : r;
    int64_t have = -1;
    float scale = 0.0f;
    // neighbouring tiles by one block: few matrices, whose scales it has to work out
    const int t1 = static_cast<int>(static_cast<int64_t>(ntiles) * (blockIdx.x + 1) / gridDim.x);
    for (int t = static_cast<int>(static_cast<int64_t>(ntiles) * blockIdx.x / gridDim.x); t < t1; ++t) {
        const int64_t mat = t / tiles;
        const int q = t % tiles;
        const int64_t r0 = q / tiles_c * 64, c0 = q % tiles_c * 64;
        if (mat != have) {
            if (have >= 0) __syncthreads();   // the last sums have been read
            scale = start_scale<kMuonBlock>(part + mat * parts, parts, eps, eps_raised, sums);
            have = mat;
            if (!goes) return;   // (start_scale's barrier lies between)
        }
        float u[4][4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int64_t row = r0 + ty + 16 * y, col = c0 + 4 * tx;
            const int64_t i = (mat * r + row) * c + col;
            const int left = row < r ? static_cast<int>(max(min(c - col, static_cast<int64_t>(4)), static_cast<int64_t>(0))) : 0;
            float nb[4];
            read_u4<kVec>(U, i, left, u[y], nb);
            if (buf) {
                if (kVec) {
                    if (left > 0) Pack<float, 4>::put(buf + i, nb);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e < left) buf[i + e] = nb[e];
                }
            }
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int64_t row = r0 + ty + 16 * y, col = c0 + 4 * tx;
#pragma unroll
            for (int e = 0; e < 4; ++e) u[y][e] = x_of(u[y][e], scale);
            if (tall) {
#pragma unroll
                for (int e = 0; e < 4; ++e) tile[ty + 16 * y][4 * tx + e] = u[y][e];
            } else if (row < r && col < c) {   // rows of X are padded to a multiple of 8 values
                const int64_t at = (mat * m + row) * ldn + col;
                split4(hi + at, lo ? lo + at : nullptr, u[y]);
            }
        }
        if (tall) {
            __syncthreads();
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int64_t row = c0 + ty + 16 * y, col = r0 + 4 * tx;
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = tile[4 * tx + e][ty + 16 * y];
                if (row < c && col < r) {
                    const int64_t at = (mat * m + row) * ldn + col;
                    split4(hi + at, lo ? lo + at : nullptr, v);
                }
            }
            __syncthreads();
        }
    }
}

// ---------------------------------------------------------------- products
enum Kind { kGram, kPoly, kUpdate, kFinal };

struct Maps {
    CUtensorMap ahi, alo, bhi, blo;   // operands
    CUtensorMap rhi, rlo;             // added term
    CUtensorMap whi, wlo;             // result
};

struct Product {
    int64_t m, n, k;        // result m x n, inner dimension k
    int64_t tiles;          // of one matrix
    int64_t all;            // of the batch
    int cols_of_tiles;      // tiles of a row of tiles (not the symmetric kinds)
    float add, mul;         // result = add * term + mul * product, and
    float diag;             // (kPoly) this on the diagonal
    int rlo, wlo;           // the term has, the result gets, a lo part
    // kFinal: the update applied or stored, r x c (transposed where tall)
    void* out;
    float* w;
    int out_bf16, tall;
    int pairs;              // rows of an even number of values, out aligned to two of them
    float decay, lr;
    uint32_t* verdict;      // of a Muon step, else nullptr
    int32_t* d_err;
};

// kPair blocks (a cluster) share a tile of 128 kPair rows x BN columns, or kSplit blocks have a part of
// the inner dimension of one tile each; P products; G epilogue groups.
template <int kKind, int kPair, int kSplit, int BN, int P, int G>
struct Shape {
    static constexpr bool kSym = kKind == kGram || kKind == kPoly;
    static constexpr uint32_t kA = kBM / kBox * kBoxBytes;                 // one f16 part of A in a stage
    static constexpr uint32_t kB = BN / kPair / kBox * kBoxBytes;
    static constexpr int kParts = P == 3 ? 2 : 1;
    static constexpr uint32_t kStage = kParts * (kA + kB);
    // Epilogue: groups of 4 warps, each with a set of its own for 64 columns of a tile: hi and lo
    // (128 x 64 each; one product's symmetric results: hi and its mirror image).
    static constexpr uint32_t kSubBytes = kBM / kBox * kBoxBytes;
    static constexpr int kGroups = G;
    static constexpr int kThreads = 64 + kGroups * kGroup;                 // copy warp, product warp, groups
    static constexpr uint32_t kSet = 2 * kSubBytes;
    static constexpr int kStages = static_cast<int>((224 * 1024 - kGroups * kSet) / kStage);
    static constexpr uint32_t kSmem = kStages * kStage + kGroups * kSet + 1024;   // + alignment
    // Accumulators in tensor memory.  The unit rounds every sum towards zero: with three products and one
    // accumulator the 940 sums of K = 5000 were off by 6e-5 of the result.  So three products have two
    // accumulators, hi hi and (2^-11 of it) hi lo + lo hi, and every kChunk stages, 32 sums of hi hi, a
    // drift below 1e-6, the epilogue adds them to its own fp32 sums, which round to nearest.  (One
    // accumulator read every 24 sums: 403 against 353 us at 2501 x 1003.)  With one product f16's own roundings are
    // 1e-3 and more, and the drift is K 2^-28: nothing at 128000 columns (200 x 131072 off by 1.0e-3 with and
    // without it), as much again and more at 2^20 (140 rows: 4.0e-3).
    static constexpr int kAccCols = P == 3 ? 2 * BN : BN;
    static constexpr int kAccs = 512 / kAccCols < 2 ? 1 : P == 3 ? 512 / kAccCols : 2;
    static constexpr int kChunk = P == 3 ? 8 : INT32_MAX;
    // Split tiles: a block is given one tile, and sums of 64 columns (fp32) from the kSplit - 1 others of its
    // cluster come to where its stages were.
    static constexpr uint32_t kSums = kBM * kSub * 4;
    static_assert(kSplit == 1 || (kPair == 1 && BN / kSub == G && kSplit >= G && (kSplit - 1) * kSums <= kStages * kStage), "split");
    static_assert(BN / kPair % kBox == 0 && kStages >= 2 && kAccs * kAccCols <= 512, "shape");
};

// Tile t of a matrix: its first row (of the pair's) and column.  Symmetric results need
// the tiles that reach the diagonal or lie below it: row of tiles i of TM rows has
// (TM i + TM - 1) / BN + 1 of them.
template <int TM, int BN, bool kSym>
__device__ __forceinline__ void tile_at(const Product& Q, int64_t t, int& mat, int& row0, int& col0)
{
    const int64_t z = t / Q.tiles;
    int q = static_cast<int>(t - z * Q.tiles);
    mat = static_cast<int>(z);
    if (kSym) {
        int i = 0;
        for (;; ++i) {
            const int w = (i * TM + TM - 1) / BN + 1;
            if (q < w) break;
            q -= w;
        }
        row0 = i * TM;
        col0 = q * BN;
    } else {
        row0 = q / Q.cols_of_tiles * TM;
        col0 = q % Q.cols_of_tiles * BN;
    }
}

// Where column `col` of a row's 64 fp32 results lies in a set: the first four of each eight in the
// hi part's 16 bytes of those columns, the others in the lo part's.
__device__ __forceinline__ uint32_t result_at(int row, int col)
{
    return ((col >> 2) & 1) * (kBM / kBox * kBoxBytes) + (row >> 6) * kBoxBytes + (row & 63) * 128 +
           (((col >> 3) ^ (row & 7)) << 4) + (col & 3) * 4;
}

// A warp's 32 rows (from `rowl` of the tile on) of 64 columns of the update from a set to where they
// belong, row by row.
__device__ __forceinline__ void put_rows(const Product& Q, uint32_t set, int rowl, int64_t mat, int row0, int col0, int lane)
{
    const int rows = min(32, static_cast<int>(Q.m) - row0);
    const int64_t c = Q.n;
    const int64_t at = (mat * Q.m + row0) * c + col0;
    if (Q.w == nullptr && Q.out_bf16 && Q.pairs) {   // two neighbours a lane
        if (col0 + 2 * lane >= c) return;
#pragma unroll 4
        for (int r = 0; r < rows; ++r) {
            const uint32_t from = set + result_at(rowl + r, 2 * lane);
            *reinterpret_cast<__nv_bfloat162*>(static_cast<bf16*>(Q.out) + at + r * c + 2 * lane) =
                __floats2bfloat162_rn(lds32(from), lds32(from + 4));
        }
        return;
    }
    bool in[2];
    in[0] = col0 + lane < c;
    in[1] = col0 + 32 + lane < c;
    for (int r0 = 0; r0 < rows; r0 += 4) {
        float v[4][2], w[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = r0 + i, col = lane + 32 * h;
                v[i][h] = lds32(set + result_at(rowl + r, col));
                w[i][h] = Q.w && in[h] && r < rows ? Q.w[at + r * c + col] : 0.0f;
            }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = r0 + i;
                if (!in[h] || r >= rows) continue;
                const int64_t o = at + r * c + lane + 32 * h;
                if (Q.w)
                    Q.w[o] = fmaf(Q.decay, w[i][h], -Q.lr * v[i][h]);
                else if (Q.out_bf16)
                    static_cast<bf16*>(Q.out)[o] = __float2bfloat16_rn(v[i][h]);
                else
                    static_cast<float*>(Q.out)[o] = v[i][h];
            }
    }
}

// Eight columns of the transposed update: a lane's row of X is a column there, so a warp
// writes 32 neighbours.
__device__ __forceinline__ void put_columns(const Product& Q, int64_t mat, int row, int col, const float (&v)[8])
{
    if (row >= Q.m) return;
    const int64_t at = (mat * Q.n + col) * Q.m + row;
    const int left = static_cast<int>(min(Q.n - col, static_cast<int64_t>(8)));
    float w[8];
    if (Q.w)
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = e < left ? Q.w[at + e * Q.m] : 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (e >= left) continue;
        const int64_t o = at + e * Q.m;
        if (Q.w)
            Q.w[o] = fmaf(Q.decay, w[e], -Q.lr * v[e]);
        else if (Q.out_bf16)
            static_cast<bf16*>(Q.out)[o] = __float2bfloat16_rn(v[e]);
        else
            static_cast<float*>(Q.out)[o] = v[e];
    }
}

// Eight columns of a lane's row (piece `p` of its 64) into the mirror image's 128 x 64 part: a column
// is a 128-byte row of the box that has this lane's 64 rows.
__device__ __forceinline__ void put_image(uint32_t part, int rowl, int p, uint4 v)
{
    const uint32_t box = part + (rowl >> 6) * kBoxBytes + (rowl & 7) * 2;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int y = p * 8 + e;
        sts16(box + y * 128 + ((((rowl & 63) >> 3) ^ (y & 7)) << 4), reinterpret_cast<const uint16_t*>(&v)[e]);
    }
}

// One block an SM (or one pair of blocks on two), tiles in turn: warp 0 copies A and B
// boxes of 64 K values into a ring of stages, warp 1 (of the pair's first block) issues
// the products into one of the accumulators, groups of four warps finish others, each
// 64 columns at a time: the added term arrives in the group's set in shared memory by
// tensor copies, the result replaces it there and leaves the same way, so every access
// of the matrices is whole lines.  The groups take the pieces in turn, so one computes
// while the others' copies are on their way.  A is K-major; B is K-major too (rows of
// the symmetric factor) or, for B X, MN-major (X as it lies).  In shared memory every
// box has 64 rows of 128 bytes, 16-byte pieces permuted by row (the copies' 128-byte
// swizzle).
template <int kKind, int kPair, int kSplit, int BN, int P, int G>
__global__ void __launch_bounds__(Shape<kKind, kPair, kSplit, BN, P, G>::kThreads, 1)
    k_muon_product(const __grid_constant__ Maps maps, const Product Q)
{
    using S = Shape<kKind, kPair, kSplit, BN, P, G>;
    constexpr bool kSym = S::kSym, kBmn = !S::kSym,
                   kTerm = kKind == kPoly || kKind == kUpdate || (kKind == kFinal && P == 3);
    constexpr bool kSum = P == 3 || kSplit > 1;   // the epilogue sums in registers, piece g of a tile by group g
    constexpr int kStages = S::kStages, TM = kBM * kPair;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[2 * kStages + 2 * S::kAccs + 1 + S::kGroups];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int dead;
    const uint32_t data = (smem_addr(raw) + 1023u) & ~1023u;
    const uint32_t sets = data + kStages * S::kStage;
    const uint32_t full = smem_addr(bars), empty = full + 8 * kStages, tfull = empty + 8 * kStages,
                   tempty = tfull + 8 * S::kAccs, drain = tempty + 8 * S::kAccs, term = drain + 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = kPair == 2 ? static_cast<int>(cluster_rank()) : 0;
    const int64_t first = blockIdx.x / (kPair * kSplit), step = gridDim.x / (kPair * kSplit);
    const int part_of_k = kSplit > 1 ? static_cast<int>(cluster_rank()) : 0;

    if (threadIdx.x == 32) {   // while the kernel before ends
        tma_prefetch(&maps.ahi);
        tma_prefetch(&maps.bhi);
        if (kTerm) tma_prefetch(&maps.rhi);
        if (kKind != kFinal) tma_prefetch(&maps.whi);
    }
    if (threadIdx.x == 0) {
        dead = 0;
        for (int s = 0; s < kStages; ++s) mbar_init(full + 8 * s, 1), mbar_init(empty + 8 * s, 1);
        for (int s = 0; s < S::kAccs; ++s) mbar_init(tfull + 8 * s, 1), mbar_init(tempty + 8 * s, 4 * S::kGroups * kPair);
        mbar_init(drain, 1);
        for (int s = 0; s < S::kGroups; ++s) mbar_init(term + 8 * s, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<kPair>(&tmem_slot, S::kAccs * S::kAccCols);
    tc_fence_before();
    if (kPair == 2)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_wait();
    if (kKind != kFinal) pdl_release();   // workspace only; after this block's allocation, so that no later block can hold what it waits for
    fence_async_proxy();                  // the first kernels wrote with ordinary stores

    // this block's stages of the inner dimension
    const int all_chunks = static_cast<int>((Q.k + kBK - 1) / kBK);
    const int begin = all_chunks * part_of_k / kSplit, chunks = all_chunks * (part_of_k + 1) / kSplit;
    if (warp == 0) {
        if (elect_one()) {
            uint32_t it = 0;
            for (int64_t t = first; t < Q.all; t += step) {
                int mat, row0, col0;
                tile_at<TM, BN, kSym>(Q, t, mat, row0, col0);
                row0 += rank * kBM;
                col0 += rank * (BN / kPair);
                for (int c = begin; c < chunks; ++c, ++it) {
                    const uint32_t s = it % kStages;
                    if (!mbar_wait(empty + 8 * s, (it / kStages & 1) ^ 1, &dead)) goto copied;
                    const uint32_t bar = kPair == 2 ? cluster_addr(full + 8 * s, 0) : full + 8 * s;
                    uint32_t at = data + s * S::kStage;
                    if (rank == 0) mbar_expect(full + 8 * s, kPair * S::kStage);
#pragma unroll
                    for (int p = 0; p < S::kParts; ++p)
#pragma unroll
                        for (int q = 0; q < kBM / kBox; ++q, at += kBoxBytes)
                            tma_load<kPair>(at, p ? &maps.alo : &maps.ahi, bar, c * kBK, row0 + q * kBox, mat);
#pragma unroll
                    for (int p = 0; p < S::kParts; ++p)
#pragma unroll
                        for (int q = 0; q < BN / kPair / kBox; ++q, at += kBoxBytes) {
                            if (kBmn)
                                tma_load<kPair>(at, p ? &maps.blo : &maps.bhi, bar, col0 + q * kBox, c * kBK, mat);
                            else
                                tma_load<kPair>(at, p ? &maps.blo : &maps.bhi, bar, c * kBK, col0 + q * kBox, mat);
                        }
                }
            }
        copied:
            if (dead && rank == 0) {   // copies in flight land before the blocks leave
                volatile int none = 0;
                for (uint32_t s = 0; s < static_cast<uint32_t>(kStages) && s < it; ++s) {
                    const uint32_t last = (it - 1 - s) / kStages * kStages + s;   // the stage's last use
                    mbar_wait(full + 8 * s, last / kStages & 1, &none);
                }
            }
        }
        if (kSplit > 1) {   // as the epilogue's
            __syncwarp();
            cluster_sync();
            cluster_sync();
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            constexpr uint32_t idesc = mma_desc_f16(TM, BN, kBmn);
            uint32_t it = 0, done = 0;   // stages, accumulators used
            bool ok = true;
            for (int64_t t = first; ok && t < Q.all; t += step)
                for (int c = begin; ok && c < chunks; ++done) {
                    const uint32_t acc = done % S::kAccs;
                    if (!(ok = mbar_wait(tempty + 8 * acc, (done / S::kAccs & 1) ^ 1, &dead))) break;
                    tc_fence_after();
                    const uint32_t d = tmem + acc * S::kAccCols;
                    for (int part = 0; part < S::kChunk && c < chunks; ++part, ++c, ++it) {
                        const uint32_t s = it % kStages;
                        if (!(ok = mbar_wait(full + 8 * s, it / kStages & 1, &dead))) break;
                        tc_fence_after();
                        const uint32_t a = data + s * S::kStage, b = a + S::kParts * S::kA;
#pragma unroll
                        for (int k = 0; k < kBK / 16; ++k) {
                            // 16 K values: 32 bytes along a K-major row, two 8-row groups of an MN-major block
                            const uint32_t ak = k * 32, bk = kBmn ? k * 2048 : k * 32;
                            const uint32_t lead = kBmn ? kBoxBytes : 16;
                            const uint64_t ah = smem_desc(a + ak, 16, 1024), bh = smem_desc(b + bk, lead, 1024);
                            tc_mma_f16<kPair>(d, ah, bh, idesc, part + k > 0);
                            if (P == 3) {
                                const uint64_t al = smem_desc(a + S::kA + ak, 16, 1024);
                                const uint64_t bl = smem_desc(b + S::kB + bk, lead, 1024);
                                tc_mma_f16<kPair>(d + BN, ah, bl, idesc, part + k > 0);
                                tc_mma_f16<kPair>(d + BN, al, bh, idesc, true);
                            }
                        }
                        tc_commit<kPair>(empty + 8 * s);
                    }
                    if (ok) tc_commit<kPair>(tfull + 8 * acc);
                }
            if (dead) {   // products in flight finish before the blocks leave
                volatile int none = 0;
                tc_commit<kPair>(drain);
                mbar_wait(drain, 0, &none);
            }
        }
        if (kSplit > 1) {
            __syncwarp();
            cluster_sync();
            cluster_sync();
        }
    } else {
        constexpr int kGroups = S::kGroups;
        const int group = (warp - 2) >> 2, id = 1 + group;
        const int rowl = (warp & 3) * 32 + lane;   // the tensor memory lanes this warp can read
        const int xr = rowl & 7;
        const uint32_t mine = (rowl >> 6) * kBoxBytes + (rowl & 63) * 128;   // this lane's row of a 128 x 64 part
        const bool head = warp == 2 + 4 * group && lane == 0;                // issues the group's copies
        const bool blocked = kKind == kFinal && Q.w != nullptr && ld_volatile(Q.verdict) != kGo;
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t at = sets + group * S::kSet, bar = term + 8 * group;
        // A tile's 64-column pieces that are wanted: inside the matrix, not above the diagonal.  They go
        // to the groups in turn, `before` counting the earlier tiles' (three products: piece g to group g).
        int mat = 0, row0 = 0, col0 = 0, pieces = 0, before = 0;
        auto plan = [&](int64_t t) {
            before = (before + pieces) % kGroups;
            pieces = 0;
            if (t >= Q.all) return;
            tile_at<TM, BN, kSym>(Q, t, mat, row0, col0);
            row0 += rank * kBM;
            const int cols = kSym ? min(row0 + kBM, static_cast<int>(Q.m)) : static_cast<int>(Q.n);
            pieces = row0 < Q.m ? max(0, min(BN / kSub, (cols - col0 + kSub - 1) / kSub)) : 0;
        };
        // (split tiles: piece g is finished by block g of the cluster)
        auto first_piece = [&] {
            return kSum ? (kSplit == 1 || part_of_k == group ? group : BN) : (group - before + kGroups) % kGroups;
        };
        // The term of piece j into the set, once nothing leaves from there any more.
        auto fetch = [&](int j) {
            tma_store_read<0>();
            mbar_expect(bar, S::kSubBytes * (Q.rlo ? 2 : 1));
            for (int q = 0; q < kBM / kBox; ++q) {
                tma_load<1>(at + q * kBoxBytes, &maps.rhi, bar, col0 + j * kSub, row0 + q * kBox, mat);
                if (Q.rlo) tma_load<1>(at + S::kSubBytes + q * kBoxBytes, &maps.rlo, bar, col0 + j * kSub, row0 + q * kBox, mat);
            }
        };
        uint32_t done = 0, terms = 0;   // accumulators, terms used
        bool ok = true;
        plan(first);
        if (kTerm && head && first_piece() < pieces) fetch(first_piece());
        for (int64_t t = first; ok && t < Q.all; t += step) {
            float sum[kSum ? 2 : 1][32];
            uint32_t acc = done % S::kAccs;
            if (kSum) {
#pragma unroll
                for (int q = 0; q < 64; ++q) sum[kSum ? q / 32 : 0][q % 32] = 0.0f;
#pragma unroll 1
                for (int c = begin; c < chunks; c += min(S::kChunk, chunks - c), ++done) {
                    acc = done % S::kAccs;
                    if (!(ok = all_of(id, kGroup, mbar_wait(tfull + 8 * acc, done / S::kAccs & 1, &dead)))) break;
                    tc_fence_after();
                    if (group * kSub < BN) {
#pragma unroll
                        for (int q = 0; q < (kSum ? 4 : 0); ++q) {
                            const uint32_t from = lanes + acc * S::kAccCols + group * kSub + q * 16;
                            float v[16], x[16];
                            tmem_load16(from, P == 3 ? from + BN : from, v, x);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                if (P == 3) v[e] += x[e];
                                sum[kSum ? q / 2 : 0][q % 2 * 16 + e] += v[e];
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(kPair == 2 ? cluster_addr(tempty + 8 * acc, 0) : tempty + 8 * acc);
                }
            } else {
                ok = all_of(id, kGroup, mbar_wait(tfull + 8 * acc, done / S::kAccs & 1, &dead));
                tc_fence_after();
                ++done;
            }
            if (kSplit > 1) {
                // Sums go to the block that finishes their piece, four columns of 32 rows at a time, once its
                // products have been through its stages, and are added there in block order.
                const uint32_t to = (part_of_k < group ? part_of_k : part_of_k - 1) * S::kSums + rowl * 16;
                __syncwarp();
                cluster_sync();
                if (ok && part_of_k != group) {
                    const uint32_t there = cluster_addr(data + to, group);
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        sts128_cluster(there + q * kBM * 16, make_uint4(__float_as_uint(sum[kSum ? q / 8 : 0][q % 8 * 4]),
                                                                        __float_as_uint(sum[kSum ? q / 8 : 0][q % 8 * 4 + 1]),
                                                                        __float_as_uint(sum[kSum ? q / 8 : 0][q % 8 * 4 + 2]),
                                                                        __float_as_uint(sum[kSum ? q / 8 : 0][q % 8 * 4 + 3])));
                }
                cluster_sync();
                if (ok && part_of_k == group)
                    for (int r = 0; r + 1 < kSplit; ++r)
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            const uint4 v = lds128(data + r * S::kSums + rowl * 16 + q * kBM * 16);
                            sum[kSum ? q / 8 : 0][q % 8 * 4] += __uint_as_float(v.x);
                            sum[kSum ? q / 8 : 0][q % 8 * 4 + 1] += __uint_as_float(v.y);
                            sum[kSum ? q / 8 : 0][q % 8 * 4 + 2] += __uint_as_float(v.z);
                            sum[kSum ? q / 8 : 0][q % 8 * 4 + 3] += __uint_as_float(v.w);
                        }
            }
            if (!ok) break;
            for (int j = first_piece(); j < pieces; j += kGroups) {
                const int col = col0 + j * kSub;
                const bool more = j + kGroups < pieces;
                if (kTerm) {
                    ok = all_of(id, kGroup, mbar_wait(bar, terms & 1, &dead));
                    if (!ok) break;
                    ++terms;
                } else if (kKind != kFinal) {
                    if (head) tma_store_read<0>();   // the set's last results have left
                    all_of(id, kGroup, true);
                }
                const bool image = kSym && col + kSub <= row0;   // wholly below the diagonal block
                uint4 khi[P == 3 && kSym ? 8 : 1], klo[P == 3 && kSym ? 8 : 1];   // kept for the image
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float v[32];
                    if (kSum) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = sum[kSum ? h : 0][e];
                    } else {
                        tmem_load32(lanes + acc * S::kAccCols + j * kSub + h * 32, v);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t piece = ((h * 4 + q) ^ xr) << 4;
                        float x[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = Q.mul * v[q * 8 + e];
                        if (kTerm) {
                            float r[8];
                            unpack8(lds128(at + mine + piece), r);
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] = fmaf(Q.add, r[e], x[e]);
                            if (Q.rlo) {
                                unpack8(lds128(at + S::kSubBytes + mine + piece), r);
#pragma unroll
                                for (int e = 0; e < 8; ++e) x[e] = fmaf(Q.add, r[e], x[e]);
                            }
                        }
                        if (kKind == kPoly && P == 1 && !image) {
                            const int e0 = row0 + rowl - (col + h * 32 + q * 8);
                            if (e0 >= 0 && e0 < 8)
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    if (e == e0) x[e] += Q.diag;
                        }
                        if (kKind == kFinal) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] *= kInvScale;
                            if (Q.tall) {
                                if (!blocked) put_columns(Q, mat, row0 + rowl, col + h * 32 + q * 8, x);
                            } else {   // see result_at
                                sts128(at + mine + piece, make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]),
                                                                     __float_as_uint(x[2]), __float_as_uint(x[3])));
                                sts128(at + S::kSubBytes + mine + piece, make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]),
                                                                                    __float_as_uint(x[6]), __float_as_uint(x[7])));
                            }
                            continue;
                        }
                        uint4 hi, lo;
                        __half2* hh = reinterpret_cast<__half2*>(&hi);
                        __half2* ll = reinterpret_cast<__half2*>(&lo);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            hh[e] = __floats2half2_rn(x[2 * e], x[2 * e + 1]);
                            const float2 f = __half22float2(hh[e]);
                            ll[e] = __floats2half2_rn(x[2 * e] - f.x, x[2 * e + 1] - f.y);
                        }
                        sts128(at + mine + piece, hi);
                        if ((P == 3 || !kSym) && Q.wlo) sts128(at + S::kSubBytes + mine + piece, lo);
                        if (P == 3 && kSym) khi[h * 4 + q] = hi, klo[h * 4 + q] = lo;
                        if (P == 1 && image) put_image(at + S::kSubBytes, rowl, h * 4 + q, hi);
                    }
                }
                if (kKind == kFinal) {   // a warp's rows are its own affair
                    __syncwarp();
                    if (!Q.tall && !blocked && row0 + (warp & 3) * 32 < Q.m)
                        put_rows(Q, at, (warp & 3) * 32, mat, row0 + (warp & 3) * 32, col, lane);
                    __syncwarp();
                    if (kTerm) {
                        fence_async_proxy();
                        all_of(id, kGroup, true);   // every warp is done with the set
                        if (head && more) fetch(j + kGroups);
                    }
                    continue;
                }
                fence_async_proxy();
                all_of(id, kGroup, true);
                if (head) {
                    for (int q = 0; q < kBM / kBox; ++q) {
                        tma_store(&maps.whi, at + q * kBoxBytes, col, row0 + q * kBox, mat);
                        if (Q.wlo) tma_store(&maps.wlo, at + S::kSubBytes + q * kBoxBytes, col, row0 + q * kBox, mat);
                        if (P == 1 && image) tma_store(&maps.whi, at + S::kSubBytes + q * kBoxBytes, row0 + q * kBox, col, mat);
                    }
                    tma_store_commit();
                }
                if (P == 3 && image) {
                    // hi and lo fill the set: the image follows when they have left, or (a split tile, the
                    // block's only one) goes by way of the stages, whose sums every warp has read
                    const uint32_t by = kSplit > 1 ? data : at;
                    if (kSplit == 1) {
                        if (head) tma_store_read<0>();
                        all_of(id, kGroup, true);
                    }
#pragma unroll
                    for (int p = 0; p < (P == 3 && kSym ? 8 : 0); ++p) {
                        put_image(by, rowl, p, khi[p]);
                        put_image(by + S::kSubBytes, rowl, p, klo[p]);
                    }
                    fence_async_proxy();
                    all_of(id, kGroup, true);
                    if (head) {
                        for (int q = 0; q < kBM / kBox; ++q) {
                            tma_store(&maps.whi, by + q * kBoxBytes, row0 + q * kBox, col, mat);
                            tma_store(&maps.wlo, by + S::kSubBytes + q * kBoxBytes, row0 + q * kBox, col, mat);
                        }
                        tma_store_commit();
                    }
                }
                if (kTerm && head && more) fetch(j + kGroups);
            }
            if (!ok) break;
            if (!kSum) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(kPair == 2 ? cluster_addr(tempty + 8 * acc, 0) : tempty + 8 * acc);
            }
            plan(t + step);
            if (kTerm && head && first_piece() < pieces) fetch(first_piece());
        }
        if (head) {
            tma_store_done();
            if (kTerm && dead) {   // a term that is on its way lands before the block leaves
                volatile int none = 0;
                mbar_wait(bar, terms & 1, &none);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    if (kPair == 2)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    if (dead && threadIdx.x == 0) {
        if (Q.verdict != nullptr) *Q.verdict = kStop;   // no weights from what this product has not finished
        set_error(Q.d_err, SPARSE_ERR_INTERNAL);
    }
    if (warp == 1) tmem_free<kPair>(tmem, S::kAccs * S::kAccCols);
}

// -------------------------------------------------------------------- host
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder()
{
    static const EncodeTiled f = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult how;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &how) != cudaSuccess ||
            how != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return f;
}

// Boxes of 64 rows x 64 values of a batch of rows x cols f16 matrices; zeros beyond.
bool encode(CUtensorMap* map, const __half* at, int64_t rows, int64_t cols, int64_t ld, int64_t batch)
{
    const cuuint64_t dim[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(batch)};
    const cuuint64_t stride[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(ld * rows) * 2};
    const cuuint32_t box[3] = {kBK, kBox, 1}, step[3] = {1, 1, 1};
    return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half*>(at), dim, stride, box, step,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

struct Layout {
    int64_t m, n, ldm, ldn;
    int parts, products;
    size_t part, verdict, x[2][2], a[2], b[2], total;   // [.][0] hi, [.][1] lo
};

// Matrices of at most 128 rows (columns) have three products whatever was asked for: with one, the few
// roundings that a small matrix averages over are off by up to 2.2e-3 of its norm, and its time is
// that of the launches and phases.
Layout muon_layout(int64_t batch, int64_t r, int64_t c, int asked)
{
    Layout L{};
    L.m = std::min(r, c);
    const int products = L.products = L.m <= 128 ? 3 : asked;
    L.n = std::max(r, c);
    L.ldm = up(L.m, 64);   // rows start on 128-byte lines: copies of boxes read whole ones
    L.ldn = up(L.n, 64);
    L.parts = static_cast<int>(std::min<int64_t>(kNormParts, std::max<int64_t>(1, r * c / 8192)));
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t p = at;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    L.part = take(sizeof(float2) * static_cast<size_t>(batch * L.parts));
    L.verdict = take(sizeof(uint32_t));
    for (int i = 0; i < 2; ++i)
        for (int h = 0; h < 2; ++h) L.x[i][h] = take(2 * static_cast<size_t>(batch * L.m * L.ldn));
    for (int h = 0; h < 2; ++h) {
        const bool needed = h == 0 || products == 3;
        L.a[h] = needed ? take(2 * static_cast<size_t>(batch * L.m * L.ldm)) : 0;
        L.b[h] = needed ? take(2 * static_cast<size_t>(batch * L.m * L.ldm)) : 0;
    }
    L.total = at;
    return L;
}

int64_t tiles_of(int64_t m, int64_t n, int tm, int bn, bool sym)
{
    if (!sym) return (m + tm - 1) / tm * ((n + bn - 1) / bn);
    int64_t t = 0;
    for (int64_t i = 0; i * tm < m; ++i) t += (i * tm + tm - 1) / bn + 1;
    return t;
}

template <int kKind, int kPair, int kSplit, int BN, int P, int G>
cudaError_t run_product(const char* name, const Maps& maps, Product Q, int64_t batch, cudaStream_t s)
{
    using S = Shape<kKind, kPair, kSplit, BN, P, G>;
    auto* kernel = k_muon_product<kKind, kPair, kSplit, BN, P, G>;
    constexpr int kCluster = kPair * kSplit;
    Q.tiles = tiles_of(Q.m, Q.n, kBM * kPair, BN, S::kSym);
    Q.all = Q.tiles * batch;
    Q.cols_of_tiles = static_cast<int>((Q.n + BN - 1) / BN);
    const cudaError_t ready = allow_smem(kernel, S::kSmem, S::kSmem);
    if (ready != cudaSuccess) return ready;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((kSplit > 1 ? Q.all : std::min<int64_t>(Q.all, num_sms() / kPair)) * kCluster));
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    SO_PROFILE(name, s);
    return cudaLaunchKernelEx(&cfg, kernel, maps, Q);
}

// What a shape's tiles take, in cycles: rounds over the GPU times the stages of a tile.  A stage needs
// 128 x BN x 64 x P products at 4096 a cycle and SM, and its boxes from L2 at about 80 bytes a cycle and
// SM, whichever is longer.  Split tiles have one round, and hand their sums over in about 6000 cycles.
template <int kKind, int kPair, int kSplit, int BN, int P>
int64_t shape_cost(const Product& Q, int64_t batch)
{
    using S = Shape<kKind, kPair, kSplit, BN, P, BN == 64 ? 1 : 2>;
    const int64_t units = num_sms() / (kPair * kSplit);
    const int64_t tiles = tiles_of(Q.m, Q.n, kBM * kPair, BN, S::kSym) * batch;
    const int64_t chunks = (Q.k + kBK - 1) / kBK;
    if (kSplit > 1 && (tiles > units || chunks < 2 * kSplit)) return INT64_MAX;
    return (tiles + units - 1) / units * ((chunks + kSplit - 1) / kSplit) * std::max<int64_t>(2 * BN * P, S::kStage / 80) +
           (kSplit > 1 ? 6000 : 0);
}

template <int kKind, int P>
cudaError_t run_kind(const char* name, const Maps& maps, const Product& Q, int64_t batch, cudaStream_t s)
{
    constexpr int kWide = P == 1 ? 256 : 128;
    const int64_t wide = P == 1 ? shape_cost<kKind, 2, 1, kWide, P>(Q, batch) : INT64_MAX;
    const int64_t pair = shape_cost<kKind, 2, 1, 128, P>(Q, batch), one = shape_cost<kKind, 1, 1, 128, P>(Q, batch),
                  half = shape_cost<kKind, 1, 1, 64, P>(Q, batch), two = shape_cost<kKind, 1, 2, 128, P>(Q, batch),
                  four = shape_cost<kKind, 1, 4, 128, P>(Q, batch);
    const int64_t least = std::min(std::min(std::min(wide, pair), std::min(one, half)), std::min(two, four));
    if (wide == least || pair == least) {
        // a short product's tile is finished in less time than two groups take over its results; a
        // long one's fares better with a fifth stage in place of the third group's set
        // (256 wide, K = 768: 58 against 70 us, K = 4096: 118 against 108; 128 wide, 16 of K = 768:
        // 20.9 against 22.9 us)
        const bool brief = P == 1 && Q.k < 1024;
        constexpr int kBrief = P == 1 ? 3 : 2;
        if (wide == least)
            return brief ? run_product<kKind, 2, 1, kWide, P, kBrief>(name, maps, Q, batch, s)
                         : run_product<kKind, 2, 1, kWide, P, 2>(name, maps, Q, batch, s);
        return brief ? run_product<kKind, 2, 1, 128, P, kBrief>(name, maps, Q, batch, s)
                     : run_product<kKind, 2, 1, 128, P, 2>(name, maps, Q, batch, s);
    }
    if (one == least) return run_product<kKind, 1, 1, 128, P, 2>(name, maps, Q, batch, s);
    if (half == least) return run_product<kKind, 1, 1, 64, P, 1>(name, maps, Q, batch, s);
    if (two == least) return run_product<kKind, 1, 2, 128, P, 2>(name, maps, Q, batch, s);
    return run_product<kKind, 1, 4, 128, P, 2>(name, maps, Q, batch, s);
}

template <int P>
cudaError_t run_steps(const Layout& L, const MuonParams& M, uint8_t* ws, cudaStream_t s)
{
    auto half = [&](size_t at) { return reinterpret_cast<__half*>(ws + at); };
    CUtensorMap mx[2][2], ma[2], mb[2];
    for (int h = 0; h < (P == 3 ? 2 : 1); ++h) {
        for (int i = 0; i < 2; ++i)
            if (!encode(&mx[i][h], half(L.x[i][h]), L.m, L.n, L.ldn, M.batch)) return cudaErrorUnknown;
        if (!encode(&ma[h], half(L.a[h]), L.m, L.m, L.ldm, M.batch)) return cudaErrorUnknown;
        if (!encode(&mb[h], half(L.b[h]), L.m, L.m, L.ldm, M.batch)) return cudaErrorUnknown;
    }
    constexpr int l = P == 3 ? 1 : 0;   // without lo parts the maps of hi stand in, unread
    if (P == 1)
        for (int i = 0; i < 2; ++i)
            if (!encode(&mx[i][1], half(L.x[i][1]), L.m, L.n, L.ldn, M.batch)) return cudaErrorUnknown;
    for (int step = 0; step < M.steps; ++step) {
        const int in = step & 1, out = in ^ 1;
        Product Q{};
        Q.verdict = M.w != nullptr ? reinterpret_cast<uint32_t*>(ws + L.verdict) : nullptr;
        Q.d_err = M.d_err;
        Q.m = Q.n = L.m;
        Q.k = L.n;
        Q.mul = kInvScale;
        Q.wlo = P == 3;
        cudaError_t e = run_kind<kGram, P>("muon_gram",
                                           Maps{mx[in][0], mx[in][l], mx[in][0], mx[in][l], ma[0], ma[l], ma[0], ma[l]},
                                           Q, M.batch, s);
        if (e != cudaSuccess) return e;

        Q.k = L.m;
        Q.add = M.b;
        Q.mul = M.c * kInvScale;
        Q.diag = P == 1 ? M.a * kScale : 0.0f;
        Q.rlo = P == 3;
        e = run_kind<kPoly, P>("muon_poly", Maps{ma[0], ma[l], ma[0], ma[l], ma[0], ma[l], mb[0], mb[l]}, Q, M.batch, s);
        if (e != cudaSuccess) return e;

        const bool last = step + 1 == M.steps;
        Q.n = L.n;
        Q.add = M.a;
        Q.mul = kInvScale;
        Q.rlo = P == 3;
        Q.wlo = P == 3 || step + 2 < M.steps;
        // the term: X, or with one product (a lies on B's diagonal) its lo part in every step but the last
        const CUtensorMap &term = P == 3 ? mx[in][0] : mx[in][1];
        const Maps maps{mb[0], mb[l], mx[in][0], mx[in][l], term, mx[in][1], mx[out][0], mx[out][1]};
        if (last) {
            Q.out = M.out;
            Q.w = M.w;
            Q.out_bf16 = M.out_bf16;
            Q.tall = M.r > M.cols;
            Q.pairs = M.cols % 2 == 0 && reinterpret_cast<uintptr_t>(M.out) % 4 == 0;
            Q.decay = M.decay;
            Q.lr = M.lr;
            e = run_kind<kFinal, P>("muon_final", maps, Q, M.batch, s);
        } else {
            e = run_kind<kUpdate, P>("muon_update", maps, Q, M.batch, s);
        }
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

size_t muon_ws_bytes(int64_t batch, int64_t r, int64_t c, int products) { return muon_layout(batch, r, c, products).total; }

cudaError_t muon(const MuonParams& M, void* ws, cudaStream_t s)
{
    if (encoder() == nullptr) return cudaErrorNotSupported;
    const Layout L = muon_layout(M.batch, M.r, M.cols, M.products);
    uint8_t* base = static_cast<uint8_t*>(ws);
    float2* part = reinterpret_cast<float2*>(base + L.part);
    uint32_t* verdict = reinterpret_cast<uint32_t*>(base + L.verdict);
    const Update U{M.g, M.g_bf16, M.buf, M.momentum, M.nesterov};
    const int64_t size = M.r * M.cols;
    cudaError_t e;
    // values of an access: rows, and so matrices, of a multiple of them, arrays aligned to match
    const uintptr_t bits = reinterpret_cast<uintptr_t>(M.buf) | reinterpret_cast<uintptr_t>(M.g);
    const int values = M.cols % 8 == 0 && bits % 16 == 0 ? 8 : M.cols % 4 == 0 && bits % (M.g_bf16 && !M.buf ? 8 : 16) == 0 ? 4 : 1;
    {
        SO_PROFILE("muon_norm", s);
        e = launch(values == 8 ? k_muon_norm<8> : values == 4 ? k_muon_norm<4> : k_muon_norm<1>,
                   dim3(static_cast<unsigned>(M.batch * L.parts)), dim3(kMuonBlock), s, U, size, L.parts, part, verdict, M.d_err);
    }
    if (e != cudaSuccess) return e;
    if (muon_fits_cluster(M.batch, L.m, L.n)) return muon_cluster(M, U, part, L.parts, verdict, values > 1, s);
    {
        const bool lo = L.products == 3 || M.steps > 1;
        __half* xhi = reinterpret_cast<__half*>(base + L.x[0][0]);
        __half* xlo = lo ? reinterpret_cast<__half*>(base + L.x[0][1]) : nullptr;
        SO_PROFILE("muon_start", s);
        if (values == 8 && M.r <= M.cols) {
            const int pieces = static_cast<int>(std::max<int64_t>(1, size / (kMuonBlock * 8 * 8)));
            e = launch(k_muon_start_flat, dim3(static_cast<unsigned>(M.batch * pieces)), dim3(kMuonBlock), s, U, M.buf, size,
                       pieces, static_cast<const float2*>(part), L.parts, M.eps, M.eps_raised, xhi, xlo, static_cast<int>(M.cols), L.ldn, verdict,
                       static_cast<const int32_t*>(M.d_err));
        } else {
            const int64_t tc = (M.cols + 63) / 64, tiles = (M.r + 63) / 64 * tc, all = tiles * M.batch;
            e = launch(values > 1 ? k_muon_start<true> : k_muon_start<false>,
                       dim3(static_cast<unsigned>(std::min<int64_t>(all, 8 * num_sms()))), dim3(kMuonBlock), s, U, M.buf,
                       M.r, M.cols, static_cast<int>(tc), static_cast<int>(tiles), static_cast<int>(all),
                       static_cast<const float2*>(part), L.parts, M.eps, M.eps_raised, xhi, xlo, L.ldn, M.r > M.cols ? 1 : 0, verdict,
                       static_cast<const int32_t*>(M.d_err));
        }
    }
    if (e != cudaSuccess) return e;
    return L.products == 3 ? run_steps<3>(L, M, base, s) : run_steps<1>(L, M, base, s);
}

}  // namespace so
