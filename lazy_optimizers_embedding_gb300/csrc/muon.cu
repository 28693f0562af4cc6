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
//                 half that of b A exact, c A^2 rounded), and X keeps its lo in
//                 a X in every step but the last (there the small singular
//                 values, tripled by a step, would drown in the rounding of the
//                 large ones; in the last step X as rounded in both terms is the
//                 better polynomial).  About 2e-3 of the result's norm, which is
//                 what rounding it to bf16 costs too.
#include <cuda_fp16.h>

#include <algorithm>

#include "profile.cuh"
#include "rowio.cuh"
#include "tensor.cuh"

namespace so {

namespace {

constexpr float kScale = 16384.0f;              // 2^14
constexpr float kInvScale = 1.0f / 16384.0f;
constexpr int kBM = 128, kBK = 64;              // tile rows; K values of a stage (128 bytes)
constexpr int kBox = 64;                        // rows of one copied box: 64 x 128 bytes
constexpr uint32_t kBoxBytes = kBox * kBK * 2;
constexpr int kThreads = 192;                   // copy warp, product warp, 4 epilogue warps
constexpr int kMuonBlock = 256;
constexpr int kNormParts = 64;                  // partial sums of squares of a matrix at most

// ------------------------------------------------------------------- start
// u of one call: given, or the momentum's.
struct Update {
    const void* g;      // u itself, or the gradient
    int g_bf16;
    const float* buf;   // momentum buffer, nullptr: u = g
    float momentum;
    int nesterov;
};

__device__ __forceinline__ float read_g(const Update& U, int64_t i)
{
    return U.g_bf16 ? __bfloat162float(static_cast<const bf16*>(U.g)[i]) : static_cast<const float*>(U.g)[i];
}
__device__ __forceinline__ float read_u(const Update& U, int64_t i, float& nb)
{
    const float g = read_g(U, i);
    if (U.buf == nullptr) return g;
    nb = fmaf(U.momentum, U.buf[i], g);
    return U.nesterov ? fmaf(U.momentum, nb, g) : nb;
}

// Sums of squares of one matrix's pieces; a sum that is not finite is reported
// before anything is written.
__global__ void __launch_bounds__(kMuonBlock) k_muon_norm(Update U, int64_t size, int parts, float* __restrict__ part,
                                                          int32_t* d_err)
{
    pdl_enter();   // writes the workspace and the error word only
    __shared__ float tmp[2 * 32];
    const int64_t mat = blockIdx.x / parts;
    const int p = static_cast<int>(blockIdx.x % parts);
    const int64_t base = mat * size;
    float s[1] = {0.0f}, nb;
#pragma unroll 4
    for (int64_t i = static_cast<int64_t>(p) * kMuonBlock + threadIdx.x; i < size;
         i += static_cast<int64_t>(parts) * kMuonBlock) {
        const float u = read_u(U, base + i, nb);
        s[0] = fmaf(u, u, s[0]);
    }
    group_sum<1>(s, kMuonBlock, tmp, 0);
    if (threadIdx.x == 0) {
        part[blockIdx.x] = s[0];
        if (!isfinite(s[0])) set_error(d_err, SPARSE_ERR_NON_FINITE);
    }
}

__device__ __forceinline__ void split_store(__half* hi, __half* lo, int64_t at, float v)
{
    const __half h = __float2half_rn(v);
    hi[at] = h;
    if (lo) lo[at] = __float2half_rn(v - __half2float(h));
}

// X = u / (|u| + eps), scaled and split, transposed where u is tall; the new momentum
// buffer.  One 32 x 32 tile of u at a time.
__global__ void __launch_bounds__(kMuonBlock) k_muon_start(Update U, float* __restrict__ buf, int64_t r, int64_t c,
                                                           int64_t tiles_c, int64_t tiles, int64_t ntiles,
                                                           const float* __restrict__ part, int parts, float eps,
                                                           __half* __restrict__ hi, __half* __restrict__ lo,
                                                           int64_t ldn, int tall, const int32_t* d_err)
{
    pdl_enter();   // writes the workspace and optimizer state only
    __shared__ float tile[32][33];
    __shared__ float s_scale;
    if (buf != nullptr && read_error(d_err) != 0) return;   // set before this kernel: the same for every block
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t m = tall ? c : r;
    int64_t have = -1;
    for (int64_t t = blockIdx.x; t < ntiles; t += gridDim.x) {
        const int64_t mat = t / tiles, q = t % tiles;
        const int64_t r0 = q / tiles_c * 32, c0 = q % tiles_c * 32;
        if (mat != have) {
            __syncthreads();
            if (ty == 0) {
                double s = 0.0;
                for (int i = tx; i < parts; i += 32) s += part[mat * parts + i];
                for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
                if (tx == 0) s_scale = static_cast<float>(static_cast<double>(kScale) / (sqrt(s) + static_cast<double>(eps)));
            }
            __syncthreads();
            have = mat;
        }
        const float scale = s_scale;
#pragma unroll
        for (int y = ty; y < 32; y += 8) {
            const int64_t row = r0 + y, col = c0 + tx;
            float v = 0.0f;
            if (row < r && col < c) {
                const int64_t i = (mat * r + row) * c + col;
                float nb = 0.0f;
                v = read_u(U, i, nb) * scale;
                if (buf) buf[i] = nb;
                if (!tall) split_store(hi, lo, (mat * m + row) * ldn + col, v);
            }
            if (tall) tile[y][tx] = v;
        }
        if (tall) {
            __syncthreads();
#pragma unroll
            for (int y = ty; y < 32; y += 8) {
                const int64_t row = c0 + y, col = r0 + tx;
                if (row < c && col < r) split_store(hi, lo, (mat * m + row) * ldn + col, tile[tx][y]);
            }
            __syncthreads();
        }
    }
}

// ---------------------------------------------------------------- products
enum Kind { kGram, kPoly, kUpdate, kFinal };

struct Product {
    int64_t m, n, k;        // result m x n, inner dimension k
    int64_t ld;             // of result and added term
    int64_t tiles;          // of one matrix
    int64_t all;            // of the batch
    int cols_of_tiles;      // tiles of a row of tiles (not the symmetric kinds)
    float add, mul;         // result = add * term + mul * product
    const __half *rhi, *rlo;    // term (rlo may be nullptr)
    __half *whi, *wlo;          // result (wlo may be nullptr)
    // kFinal: the update applied or stored, r x c (transposed where tall)
    void* out;
    float* w;
    int out_bf16, tall, vec;
    float decay, lr;
    int32_t* d_err;
};

struct Maps {
    CUtensorMap ahi, alo, bhi, blo;
};

template <int BN, int P>
struct Shape {
    static constexpr uint32_t kA = kBM / kBox * kBoxBytes;        // one f16 part of A in a stage
    static constexpr uint32_t kB = BN / kBox * kBoxBytes;
    static constexpr int kParts = P == 3 ? 2 : 1;
    static constexpr uint32_t kStage = kParts * (kA + kB);
    static constexpr int kStages = (200 * 1024) / kStage;
    static constexpr uint32_t kSmem = kStages * kStage + 1024;    // + alignment
    static constexpr int kAccs = P == 3 ? 512 / BN : 2;           // accumulators in tensor memory
    // Stages that one accumulator sums.  The unit rounds every sum towards zero: with three products
    // the 940 sums of K = 5000 were off by 6e-5 of the result, so every 24 sums (128 K values, a
    // drift below 1e-6) the epilogue adds the accumulator to its own fp32 sums, which round to nearest.
    // Against f16 operands alone (one product) the drift does not count.
    static constexpr int kChunk = P == 3 ? 2 : INT32_MAX;
};

// Tile t of a matrix.  Symmetric results need the tiles that reach the diagonal or
// lie below it: row of tiles i has (128 i + 127) / BN + 1 of them.
template <int BN, bool kSym>
__device__ __forceinline__ void tile_at(const Product& Q, int64_t t, int64_t& mat, int64_t& row0, int64_t& col0)
{
    mat = t / Q.tiles;
    int64_t q = t - mat * Q.tiles;
    if (kSym) {
        int64_t i = 0;
        for (;; ++i) {
            const int64_t w = (i * kBM + kBM - 1) / BN + 1;
            if (q < w) break;
            q -= w;
        }
        row0 = i * kBM;
        col0 = q * BN;
    } else {
        row0 = q / Q.cols_of_tiles * kBM;
        col0 = q % Q.cols_of_tiles * BN;
    }
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

// Eight consecutive results of one row.
template <int kKind>
__device__ __forceinline__ void finish8(const Product& Q, int64_t mat, int64_t row, int64_t col, const float* acc)
{
    constexpr bool kSym = kKind == kGram || kKind == kPoly;
    if (row >= Q.m || col >= Q.n || (kSym && col > row)) return;
    const int64_t at = (mat * Q.m + row) * Q.ld + col;   // ld and col are multiples of 8: 16-byte aligned, within the row
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = Q.mul * acc[e];
    if (kKind != kGram) {
        float x[8];
        unpack8(*reinterpret_cast<const uint4*>(Q.rhi + at), x);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf(Q.add, x[e], v[e]);
        if (Q.rlo) {
            unpack8(*reinterpret_cast<const uint4*>(Q.rlo + at), x);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = fmaf(Q.add, x[e], v[e]);
        }
    }
    if (kKind == kFinal) {
        const int64_t r = Q.tall ? Q.n : Q.m, c = Q.tall ? Q.m : Q.n;
        for (int e = 0; e < 8; ++e) {
            if (col + e >= Q.n) break;
            const int64_t o = mat * r * c + (Q.tall ? (col + e) * c + row : row * c + col + e);
            const float x = v[e] * kInvScale;
            if (Q.w)
                Q.w[o] = fmaf(Q.decay, Q.w[o], -Q.lr * x);
            else if (Q.out_bf16)
                static_cast<bf16*>(Q.out)[o] = __float2bfloat16_rn(x);
            else
                static_cast<float*>(Q.out)[o] = x;
        }
        return;
    }
    uint4 hi, lo;
    __half* h = reinterpret_cast<__half*>(&hi);
    __half* l = reinterpret_cast<__half*>(&lo);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        h[e] = __float2half_rn(v[e]);
        l[e] = __float2half_rn(v[e] - __half2float(h[e]));
    }
    if (!kSym) {
        *reinterpret_cast<uint4*>(Q.whi + at) = hi;
        if (Q.wlo) *reinterpret_cast<uint4*>(Q.wlo + at) = lo;
        return;
    }
    // the element and its mirror image; across the diagonal nothing (its mirror image is written)
    if (col + 8 <= row + 1 && col + 8 <= Q.n) {
        *reinterpret_cast<uint4*>(Q.whi + at) = hi;
        if (Q.wlo) *reinterpret_cast<uint4*>(Q.wlo + at) = lo;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (col + e <= row) {
                Q.whi[at + e] = h[e];
                if (Q.wlo) Q.wlo[at + e] = l[e];
            }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (col + e < row) {
            const int64_t mt = (mat * Q.m + col + e) * Q.ld + row;
            Q.whi[mt] = h[e];
            if (Q.wlo) Q.wlo[mt] = l[e];
        }
}

// One block an SM, tiles of 128 x BN in turn: warp 0 copies A and B boxes of 64 K
// values into a ring of stages, warp 1 issues the products into one of two
// accumulators, warps 2 to 5 finish the other.  A is K-major; B is K-major too
// (rows of the symmetric factor) or, for B X, MN-major (X as it lies).
template <int kKind, int BN, int P>
__global__ void __launch_bounds__(kThreads, 1) k_muon_product(const __grid_constant__ Maps maps, const Product Q)
{
    using S = Shape<BN, P>;
    constexpr bool kSym = kKind == kGram || kKind == kPoly;
    constexpr bool kBmn = !kSym;
    constexpr int kStages = S::kStages;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[2 * kStages + 2 * S::kAccs + 1];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int dead;
    const uint32_t data = (smem_addr(raw) + 1023u) & ~1023u;
    const uint32_t full = smem_addr(bars), empty = full + 8 * kStages, tfull = empty + 8 * kStages, tempty = tfull + 8 * S::kAccs,
                   drain = tempty + 8 * S::kAccs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        dead = 0;
        for (int s = 0; s < kStages; ++s) mbar_init(full + 8 * s, 1), mbar_init(empty + 8 * s, 1);
        for (int s = 0; s < S::kAccs; ++s) mbar_init(tfull + 8 * s, 1), mbar_init(tempty + 8 * s, 128);
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc(&tmem_slot, S::kAccs * BN);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_wait();
    if (kKind != kFinal) pdl_release();   // workspace only; after this block's allocation, so that no later block can hold what it waits for
    fence_async_proxy();                  // the kernels before wrote with ordinary stores

    const int chunks = static_cast<int>((Q.k + kBK - 1) / kBK);
    if (warp == 0) {
        if (elect_one()) {
            tma_prefetch(&maps.ahi);
            tma_prefetch(&maps.bhi);
            uint32_t it = 0;
            for (int64_t t = blockIdx.x; t < Q.all; t += gridDim.x) {
                int64_t mat, row0, col0;
                tile_at<BN, kSym>(Q, t, mat, row0, col0);
                const int z = static_cast<int>(mat), y = static_cast<int>(row0), x = static_cast<int>(col0);
                for (int c = 0; c < chunks; ++c, ++it) {
                    const uint32_t s = it % kStages;
                    if (!mbar_wait(empty + 8 * s, (it / kStages & 1) ^ 1, &dead)) goto copied;
                    const uint32_t bar = full + 8 * s;
                    uint32_t at = data + s * S::kStage;
                    mbar_expect(bar, S::kStage);
#pragma unroll
                    for (int p = 0; p < S::kParts; ++p)
#pragma unroll
                        for (int q = 0; q < kBM / kBox; ++q, at += kBoxBytes)
                            tma_load(at, p ? &maps.alo : &maps.ahi, bar, c * kBK, y + q * kBox, z);
#pragma unroll
                    for (int p = 0; p < S::kParts; ++p)
#pragma unroll
                        for (int q = 0; q < BN / kBox; ++q, at += kBoxBytes) {
                            if (kBmn)
                                tma_load(at, p ? &maps.blo : &maps.bhi, bar, x + q * kBox, c * kBK, z);
                            else
                                tma_load(at, p ? &maps.blo : &maps.bhi, bar, c * kBK, x + q * kBox, z);
                        }
                }
            }
        copied:
            if (dead) {   // copies in flight land before the block leaves
                volatile int none = 0;
                for (uint32_t s = 0; s < static_cast<uint32_t>(kStages) && s < it; ++s) {
                    const uint32_t last = (it - 1 - s) / kStages * kStages + s;   // the stage's last use
                    if (last < it) mbar_wait(full + 8 * s, last / kStages & 1, &none);
                }
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {
            constexpr uint32_t idesc = mma_desc_f16(kBM, BN, kBmn);
            uint32_t it = 0, done = 0;   // stages, accumulators used
            bool ok = true;
            for (int64_t t = blockIdx.x; ok && t < Q.all; t += gridDim.x)
                for (int c = 0; ok && c < chunks; ++done) {
                    const uint32_t acc = done % S::kAccs;
                    if (!(ok = mbar_wait(tempty + 8 * acc, (done / S::kAccs & 1) ^ 1, &dead))) break;
                    tc_fence_after();
                    const uint32_t d = tmem + acc * BN;
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
                            tc_mma_f16(d, ah, bh, idesc, part + k > 0);
                            if (P == 3) {
                                const uint64_t al = smem_desc(a + S::kA + ak, 16, 1024);
                                const uint64_t bl = smem_desc(b + S::kB + bk, lead, 1024);
                                tc_mma_f16(d, ah, bl, idesc, true);
                                tc_mma_f16(d, al, bh, idesc, true);
                            }
                        }
                        tc_commit(empty + 8 * s);
                    }
                    if (ok) tc_commit(tfull + 8 * acc);
                }
            if (dead) {   // products in flight finish before the block leaves
                volatile int none = 0;
                tc_commit(drain);
                mbar_wait(drain, 0, &none);
            }
        }
    } else {
        const int quarter = warp & 3;   // the tensor memory lanes this warp can read
        const bool blocked = kKind == kFinal && Q.w != nullptr && read_error(Q.d_err) != 0;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        uint32_t done = 0;
        bool ok = true;
        for (int64_t t = blockIdx.x; ok && t < Q.all; t += gridDim.x) {
            int64_t mat, row0, col0;
            tile_at<BN, kSym>(Q, t, mat, row0, col0);
            const int64_t row = row0 + quarter * 32 + lane;
            float sum[P == 3 ? BN / 32 : 1][32];
            for (int c = 0; c < chunks; c += S::kChunk, ++done) {
                const uint32_t acc = done % S::kAccs;
                if (!(ok = __all_sync(kFull, mbar_wait(tfull + 8 * acc, done / S::kAccs & 1, &dead)))) break;
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < BN / 32; ++q) {
                    float v[32];
                    tmem_load32(lanes + acc * BN + q * 32, v);
                    if (P == 3) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) sum[q % (P == 3 ? BN / 32 : 1)][e] = c ? sum[q % (P == 3 ? BN / 32 : 1)][e] + v[e] : v[e];
                    } else if (!blocked) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) finish8<kKind>(Q, mat, row, col0 + q * 32 + e, v + e);
                    }
                }
                tc_fence_before();
                mbar_arrive(tempty + 8 * acc);
                if (P != 3) {
                    ++done;
                    break;   // one accumulator holds the tile
                }
            }
            if (P == 3 && ok && !blocked)
#pragma unroll
                for (int q = 0; q < BN / 32; ++q)
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        finish8<kKind>(Q, mat, row, col0 + q * 32 + e, sum[q % (P == 3 ? BN / 32 : 1)] + e);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (dead && threadIdx.x == 0) set_error(Q.d_err, SPARSE_ERR_INTERNAL);
    if (warp == 1) tmem_free(tmem, S::kAccs * BN);
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
    int parts;
    size_t part, x[2][2], a[2], b[2], total;   // [.][0] hi, [.][1] lo
};

Layout muon_layout(int64_t batch, int64_t r, int64_t c, int products)
{
    Layout L{};
    L.m = std::min(r, c);
    L.n = std::max(r, c);
    L.ldm = up(L.m, 8);
    L.ldn = up(L.n, 8);
    L.parts = static_cast<int>(std::min<int64_t>(kNormParts, std::max<int64_t>(1, r * c / 8192)));
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t p = at;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    L.part = take(sizeof(float) * static_cast<size_t>(batch * L.parts));
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

int64_t tiles_of(int64_t m, int64_t n, int bn, bool sym)
{
    if (!sym) return (m + kBM - 1) / kBM * ((n + bn - 1) / bn);
    int64_t t = 0;
    for (int64_t i = 0; i * kBM < m; ++i) t += (i * kBM + kBM - 1) / bn + 1;
    return t;
}

template <int kKind, int BN, int P>
cudaError_t run_product(const char* name, const Maps& maps, Product Q, int64_t batch, cudaStream_t s)
{
    constexpr bool kSym = kKind == kGram || kKind == kPoly;
    using S = Shape<BN, P>;
    Q.tiles = tiles_of(Q.m, Q.n, BN, kSym);
    Q.all = Q.tiles * batch;
    Q.cols_of_tiles = static_cast<int>((Q.n + BN - 1) / BN);
    const cudaError_t e = cudaFuncSetAttribute(k_muon_product<kKind, BN, P>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(S::kSmem));
    if (e != cudaSuccess) return e;
    const int blocks = static_cast<int>(std::min<int64_t>(Q.all, num_sms()));
    SO_PROFILE(name, s);
    return launch_smem(k_muon_product<kKind, BN, P>, dim3(blocks), dim3(kThreads), S::kSmem, s, maps, Q);
}

template <int kKind, int P>
cudaError_t run_kind(const char* name, const Maps& maps, const Product& Q, int64_t batch, cudaStream_t s)
{
    return run_product<kKind, 128, P>(name, maps, Q, batch, s);
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
    for (int step = 0; step < M.steps; ++step) {
        const int in = step & 1, out = in ^ 1;
        Product Q{};
        Q.d_err = M.d_err;
        Q.m = Q.n = L.m;
        Q.ld = L.ldm;
        Q.k = L.n;
        Q.mul = kInvScale;
        Q.whi = half(L.a[0]);
        Q.wlo = P == 3 ? half(L.a[1]) : nullptr;
        cudaError_t e = run_kind<kGram, P>("muon_gram", Maps{mx[in][0], mx[in][l], mx[in][0], mx[in][l]}, Q, M.batch, s);
        if (e != cudaSuccess) return e;

        Q.k = L.m;
        Q.add = M.b;
        Q.mul = M.c * kInvScale;
        Q.rhi = half(L.a[0]);
        Q.rlo = P == 3 ? half(L.a[1]) : nullptr;
        Q.whi = half(L.b[0]);
        Q.wlo = P == 3 ? half(L.b[1]) : nullptr;
        e = run_kind<kPoly, P>("muon_poly", Maps{ma[0], ma[l], ma[0], ma[l]}, Q, M.batch, s);
        if (e != cudaSuccess) return e;

        const bool last = step + 1 == M.steps;
        Q.n = L.n;
        Q.ld = L.ldn;
        Q.add = M.a;
        Q.mul = kInvScale;
        Q.rhi = half(L.x[in][0]);
        Q.rlo = P == 3 || !last ? half(L.x[in][1]) : nullptr;
        Q.whi = half(L.x[out][0]);
        Q.wlo = P == 3 || step + 2 < M.steps ? half(L.x[out][1]) : nullptr;
        const Maps maps{mb[0], mb[l], mx[in][0], mx[in][l]};
        if (last) {
            Q.out = M.out;
            Q.w = M.w;
            Q.out_bf16 = M.out_bf16;
            Q.tall = M.r > M.cols;
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
    float* part = reinterpret_cast<float*>(base + L.part);
    const Update U{M.g, M.g_bf16, M.buf, M.momentum, M.nesterov};
    const int64_t size = M.r * M.cols;
    cudaError_t e;
    {
        SO_PROFILE("muon_norm", s);
        e = launch(k_muon_norm, dim3(static_cast<unsigned>(M.batch * L.parts)), dim3(kMuonBlock), s, U, size, L.parts,
                   part, M.d_err);
    }
    if (e != cudaSuccess) return e;
    {
        const int64_t tc = (M.cols + 31) / 32, tiles = (M.r + 31) / 32 * tc, all = tiles * M.batch;
        const bool lo = M.products == 3 || M.steps > 1;
        SO_PROFILE("muon_start", s);
        e = launch(k_muon_start, dim3(static_cast<unsigned>(std::min<int64_t>(all, 8 * num_sms()))), dim3(kMuonBlock), s,
                   U, M.buf, M.r, M.cols, tc, tiles, all, static_cast<const float*>(part), L.parts, M.eps,
                   reinterpret_cast<__half*>(base + L.x[0][0]),
                   lo ? reinterpret_cast<__half*>(base + L.x[0][1]) : static_cast<__half*>(nullptr), L.ldn,
                   M.r > M.cols ? 1 : 0, static_cast<const int32_t*>(M.d_err));
    }
    if (e != cudaSuccess) return e;
    return M.products == 3 ? run_steps<3>(L, M, base, s) : run_steps<1>(L, M, base, s);
}

}  // namespace so
