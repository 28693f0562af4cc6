// muon_small.cu -- Newton-Schulz for matrices of at most 128 rows (columns, where
// tall) whose X a cluster's shared memory holds: all steps in one launch.
//
// A cluster of up to 8 blocks has one matrix; each block keeps some columns of X, hi and lo f16, and
// the whole of A and B (three products: the time is mostly that of the phases, 35 us for 64 x 128
// with one or three).  It has room for 128 rows of 256 columns; of a matrix of at most 64 (32) rows it
// keeps two (four) times as many, in parts that lie below one another: the products of parts with
// themselves then add up to A's share, and B, once for every part on the diagonal, serves them
// all.  A step is
//   A's share of the columns   X_s X_s^T, the shares summed over the cluster (and the parts) through
//                              shared memory, in the same order on every block
//   A A                        by every block
//   B X_s                      by every block, in place
// hi + lo is X to 22.6 bits, and the roundings of small singular values' directions grow with these,
// 484 times in five steps.  Where few rows share them (at most 16) they are most of the result's
// error (3 x 8190, singular values 1 to e^-9: 2.1e-5, fp32 products 1.4e-5), so there what hi + lo
// leave of X is kept too, a byte of three bits and an exponent, and a X has all of it (1.6e-5; it costs a
// sixth of the time).
// One copy of X serves both products: boxes of 64 columns, 128 rows of 128 bytes, are
// K-major for X X^T and MN-major for B X.  Products of one hi and one lo part, 2^-11
// of the others, have an accumulator of their own, so that the tensor unit's
// rounding towards zero is one of K / 16 sums and not of three times as many.
//
// Of a step's time at 64 x 128 (3 us) most is latency: products 0.9 us, barriers 0.6 us, tensor memory
// reads and f16 splits the rest.  At 128 x 256 (7 us) the three products of one SM take 4 us.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include <cuda_fp8.h>

#include "muon.cuh"
#include "profile.cuh"

namespace so {

namespace {

constexpr int kRows = 128;                       // rows of X, A and B held, zeros past the matrix's
constexpr int kSlice = 256;                      // columns of X a block holds at most
constexpr uint32_t kBlockBytes = kRows * 128;    // 64 columns of 128 rows
constexpr uint32_t kXBytes = kSlice / 64 * kBlockBytes, kSquareBytes = kRows / 64 * kBlockBytes;
constexpr int kRestRows = 16;                     // rows up to which X has rests (below)
constexpr uint32_t kRestBytes = kRows * kSlice;
constexpr uint32_t kSmallSmem = 2 * kXBytes + 2 * kSquareBytes + 1024;   // and kRestBytes
constexpr float kRestScale = 16384.0f;           // what hi + lo leave of 65504 is below 2^-8
constexpr int kMaxCluster = 8;
constexpr int kBlockThreads = 512, kWarps = kBlockThreads / 32;   // four warps for every 32 rows, a quarter of the columns each
constexpr uint32_t kGramCol = 0, kCrossCol = 128, kUpdateCol = 256, kTmemCols = 512;

// Byte of element (row, col) in an array of 64-column blocks, 16-byte pieces permuted by row.
__device__ __forceinline__ uint32_t place(int row, int col)
{
    return (col >> 6) * kBlockBytes + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4) + (col & 7) * 2;
}

// And in the array of what hi and lo leave, a byte each: 64-column blocks, 8-byte pieces permuted by row pair.
__device__ __forceinline__ uint32_t rest_place(int row, int col)
{
    return (col >> 6) * (kRows * 64) + row * 64 + ((((col & 63) >> 3) ^ (row >> 1 & 7)) << 3) + (col & 7);
}
// Two values' rests as bytes, and back.
__device__ __forceinline__ uint16_t rest_of(float a, float b)
{
    return __nv_cvt_float2_to_fp8x2(make_float2(a * kRestScale, b * kRestScale), __NV_SATFINITE, __NV_E5M2);
}
__device__ __forceinline__ float2 rest_values(uint16_t q)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(q, __NV_E5M2);
    const float2 f = __half22float2(__half2(h));
    return make_float2(f.x * (1.0f / kRestScale), f.y * (1.0f / kRestScale));
}

__device__ __forceinline__ float4 lds_cluster(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// Eight values as hi and lo f16 to shared memory, and what these leave.
template <bool kRest>
__device__ __forceinline__ void split8(uint32_t hi_at, uint32_t lo_at, uint32_t rest_at, const float (&x)[8])
{
    uint16_t rest[4];
    uint4 hi, lo;
    __half2* hh = reinterpret_cast<__half2*>(&hi);
    __half2* ll = reinterpret_cast<__half2*>(&lo);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        hh[e] = __floats2half2_rn(x[2 * e], x[2 * e + 1]);
        const float2 f = __half22float2(hh[e]);
        ll[e] = __floats2half2_rn(x[2 * e] - f.x, x[2 * e + 1] - f.y);
        if (kRest) {
            const float2 l = __half22float2(ll[e]);
            rest[e] = rest_of(x[2 * e] - f.x - l.x, x[2 * e + 1] - f.y - l.y);
        }
    }
    sts128(hi_at, hi);
    sts128(lo_at, lo);
    if (kRest) sts64(rest_at, rest[0] | static_cast<uint32_t>(rest[1]) << 16, rest[2] | static_cast<uint32_t>(rest[3]) << 16);
}

__device__ __forceinline__ uint16_t bits_of(__half h) { return __half_as_ushort(h); }

__device__ __forceinline__ __half lds_half(uint32_t a)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return __ushort_as_half(v);
}

struct Small {
    int64_t size;        // of a matrix
    int m, n;            // X: m x n
    int fold;            // parts of a block's columns that lie below one another, 128 / fold rows each
    int slice;           // columns of a part, a multiple of 64
    int tall, steps;
    float a, b, c, eps, eps_raised;
    const float2* part;
    int parts;
    float* buf;
    void* out;
    int out_bf16, vec;   // vec: rows of a multiple of four values, out (w) aligned to four of them
    float* w;
    float decay, lr;
    uint32_t* verdict;   // of a Muon step
    int32_t* d_err;
};

// kLayout: one part, several, or (at most kRestRows rows) with rests.
enum Layout { kOnePart, kParts, kRests };
template <bool kVec, Layout kLayout>
__global__ void __launch_bounds__(kBlockThreads, 1) k_muon_cluster(const Update U, const Small Q, int blocks)
{
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bar_mem[2];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int dead;
    __shared__ bool goes;
    __shared__ float sums[2 * 32];
    const uint32_t xhi = (smem_addr(raw) + 1023u) & ~1023u, xlo = xhi + kXBytes, shi = xlo + kXBytes, slo = shi + kSquareBytes, xrest = slo + kSquareBytes;
    const uint32_t bar = smem_addr(bar_mem);
    constexpr bool kRest = kLayout == kRests;
    const int fold = kLayout == kOnePart ? 1 : Q.fold;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t mat = blockIdx.x / blocks;
    const int rank = static_cast<int>(blockIdx.x % blocks);
    const int col0 = rank * fold * Q.slice, cols = max(0, min(fold * Q.slice, Q.n - col0));   // this block's columns of X
    const int side = fold == 1 && Q.m <= 64 ? 64 : 128;   // of A and B, in the products
    const int part_rows = kRows / fold;
    auto held = [&](int& r, int& c) {   // where row r, column c of the block's columns lies
        int h = 0;
        if (fold > 1) h = (c >= Q.slice) + (c >= 2 * Q.slice) + (c >= 3 * Q.slice);
        r += h * part_rows, c -= h * Q.slice;
    };

    if (threadIdx.x == 0) {
        dead = 0;
        mbar_init(bar, 1), mbar_init(bar + 8, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tmem_alloc<1>(&tmem_slot, kTmemCols);
    for (uint32_t i = threadIdx.x * 16; i < 2 * kXBytes; i += kBlockThreads * 16) sts128(xhi + i, make_uint4(0u, 0u, 0u, 0u));
    for (uint32_t i = threadIdx.x * 16; i < (kRest ? kRestBytes : 0u); i += kBlockThreads * 16) sts128(xrest + i, make_uint4(0u, 0u, 0u, 0u));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_wait();   // writes a caller output: dependents start after this grid exits
    if (threadIdx.x == kBlockThreads - 1) goes = Q.w == nullptr || step_goes(Q.verdict, Q.d_err);   // (one that reads no sums)

    // X of the slice, scaled and split; the new momentum buffer
    const float scale = start_scale<kBlockThreads>(Q.part + mat * Q.parts, Q.parts, Q.eps, Q.eps_raised, sums);
    const bool blocked = !goes;   // (start_scale's barrier lies between)
    const int64_t base = mat * Q.size;
    // Groups of lanes take u's rows (X's, or its columns where u is tall), a lane four values at a time: a
    // whole warp, or as many lanes as such a row has use for.
    const int outer = Q.tall ? cols : Q.m, inner = Q.tall ? Q.m : cols;
    int lanes_of_row = 32;
    while (lanes_of_row > 1 && lanes_of_row * 2 >= inner) lanes_of_row /= 2;
    const int groups = kBlockThreads / lanes_of_row, group = threadIdx.x / lanes_of_row, k0 = threadIdx.x % lanes_of_row * 4;
    auto value_at = [&](int o, int k) {
        return base + (Q.tall ? static_cast<int64_t>(col0 + o) * Q.m + k : static_cast<int64_t>(o) * Q.n + col0 + k);
    };
    constexpr int kRowsAtOnce = 4;
    if (!blocked)
        for (int k = k0; k < inner; k += lanes_of_row * 4)
            for (int o0 = group; o0 < outer; o0 += groups * kRowsAtOnce) {
                float u[kRowsAtOnce][4], nb[kRowsAtOnce][4];
                const int left = min(4, inner - k);
#pragma unroll
                for (int i = 0; i < kRowsAtOnce; ++i) {
                    const int o = o0 + i * groups;
                    if (o < outer) read_u4<kVec>(U, value_at(o, k), left, u[i], nb[i]);
                }
#pragma unroll
                for (int i = 0; i < kRowsAtOnce; ++i) {
                    const int o = o0 + i * groups;
                    if (o >= outer) continue;
                    if (Q.buf) {
                        const int64_t at = value_at(o, k);
                        if (kVec) {
                            Pack<float, 4>::put(Q.buf + at, nb[i]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (e < left) Q.buf[at + e] = nb[i][e];
                        }
                    }
                    uint16_t h[4], l[4], rest[2];
                    float left_over[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {   // 0 past `left`
                        const float v = x_of(u[i][e], scale);
                        const __half q = __float2half_rn(v), ql = __float2half_rn(v - __half2float(q));
                        h[e] = bits_of(q), l[e] = bits_of(ql);
                        left_over[e] = v - __half2float(q) - __half2float(ql);
                    }
                    if (kRest) rest[0] = rest_of(left_over[0], left_over[1]), rest[1] = rest_of(left_over[2], left_over[3]);
                    int y = Q.tall ? k : o, x = Q.tall ? o : k;
                    held(y, x);
                    if (Q.tall) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (e < left) {
                                sts16(xhi + place(y + e, x), h[e]), sts16(xlo + place(y + e, x), l[e]);
                                if (kRest) sts8(xrest + rest_place(y + e, x), rest[e / 2] >> e % 2 * 8);
                            }
                    } else {
                        const uint32_t p = place(y, x);   // four columns of one 16-byte piece
                        sts64(xhi + p, h[0] | static_cast<uint32_t>(h[1]) << 16, h[2] | static_cast<uint32_t>(h[3]) << 16);
                        sts64(xlo + p, l[0] | static_cast<uint32_t>(l[1]) << 16, l[2] | static_cast<uint32_t>(l[3]) << 16);
                        if (kRest) sts32(xrest + rest_place(y, x), rest[0] | static_cast<uint32_t>(rest[1]) << 16);
                    }
                }
            }

    // this warp's share of an accumulator: 32 rows, a quarter of the columns
    const int row = (warp & 3) * 32 + lane, quarter = warp >> 2;
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const bool rows_used = (warp & 3) * 32 % part_rows < Q.m;
    // Of the parts' products only those of a part with itself are A's; a warp's 32 x 32 are or are not.
    const bool own_part = fold == 1 || (warp & 3) * 32 / part_rows == quarter * 32 / part_rows;
    uint32_t phase = 0;
    auto products_done = [&] {   // of the phase's MMAs, by every thread
        mbar_wait(bar, phase & 1, &dead);
        ++phase;
        __syncwarp();
        tc_fence_after();
    };
    auto operands_done = [&] {   // written by every thread, for the MMAs
        fence_async_proxy();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    };
    // 64-value blocks of K: hi hi into `d`, hi lo + lo hi into `x` (the same accumulator where d == x).
    // Operands K-major, B MN-major where kMn (a K value 128 bytes on).
    const uint64_t dxh = smem_desc(xhi, 16, 1024), dxl = smem_desc(xlo, 16, 1024);
    const uint64_t dsh = smem_desc(shi, 16, 1024), dsl = smem_desc(slo, 16, 1024);
    const uint64_t mxh = smem_desc(xhi, kBlockBytes, 1024), mxl = smem_desc(xlo, kBlockBytes, 1024);
    auto issue = [&](auto mn, uint32_t d, uint32_t x, uint32_t idesc, uint64_t ah, uint64_t al, uint64_t bh, uint64_t bl,
                     int blocks_of_k) {
        constexpr bool kMn = decltype(mn)::value;
        for (int k = 0; k < blocks_of_k; ++k) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint64_t a = q * 2, b = kMn ? q * 128 : q * 2;   // 16 K values, in 16-byte units
                tc_mma_f16<1>(tmem + d, ah + a, bh + b, idesc, k + q > 0);
                tc_mma_f16<1>(tmem + x, ah + a, bl + b, idesc, d == x || k + q > 0);
                tc_mma_f16<1>(tmem + x, al + a, bh + b, idesc, true);
            }
            ah += kBlockBytes / 16, al += kBlockBytes / 16;
            bh += kMn ? 512 : kBlockBytes / 16, bl += kMn ? 512 : kBlockBytes / 16;
        }
        tc_commit<1>(bar);
    };
    const uint32_t square = mma_desc_f16(kRows, side, false), update = mma_desc_f16(kRows, Q.slice, true);

    for (int step = 0; step < Q.steps; ++step) {
        // ---- A
        operands_done();
        if (warp == 0 && elect_one()) {
            issue(std::false_type{}, kGramCol, kCrossCol, square, dxh, dxl, dxh, dxl, Q.slice / 64);
        }
        products_done();
        const int per = side / 4;              // columns of A this warp has: 16 or 32
        float av[32];
        if (rows_used && own_part)
#pragma unroll
            for (int q = 0; q < 2; ++q)
                if (q * 16 < per) {
                    float v[16], x[16];
                    tmem_load16(lanes + kGramCol + quarter * per + q * 16, lanes + kCrossCol + quarter * per + q * 16, v, x);
#pragma unroll
                    for (int e = 0; e < 16; ++e) av[q * 16 + e] = v[e] + x[e];
                }
        if (blocks > 1 || fold > 1) {
            // The shares of the blocks' parts, fp32, where A will be: rows of rows_of / 4 16-byte pieces, permuted
            // by row.  Block r sums the r-th share of the pieces over the cluster, in the order of parts
            // and blocks, in place (no other block reads that share), then every block fetches the others'
            // sums, neighbouring lanes neighbouring pieces.  (Every block reading every share in its own
            // rows' order, 16 bytes of 32 rows at a time, took 130 us a step at 128 x 2048.)
            const int rows_of = fold == 1 ? side : part_rows;
            const int quads = rows_of / 4, all = quads * rows_of, mine = all / blocks, shift = 31 - __clz(mine);   // powers of two
            const int r0 = fold == 1 ? row : row % part_rows, q0 = fold == 1 ? quarter * (per / 4) : quarter * 32 % part_rows / 4;
            const uint32_t part_at = fold == 1 ? 0u : static_cast<uint32_t>(row / part_rows * all * 16);
            auto quad = [&](int q) { return shi + static_cast<uint32_t>(r0 * quads + ((q0 + q) ^ (r0 & 7))) * 16; };
            if (rows_used && own_part)
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (q * 4 < per)
                        sts128(quad(q) + part_at, make_uint4(__float_as_uint(av[4 * q]), __float_as_uint(av[4 * q + 1]),
                                                   __float_as_uint(av[4 * q + 2]), __float_as_uint(av[4 * q + 3])));
            cluster_sync();
            const int used = min(rows_of, (Q.m + 31) / 32 * 32) * quads;   // pieces of rows that the warps wrote
            for (int f = rank * mine + threadIdx.x; f < (rank + 1) * mine && f < used; f += kBlockThreads) {
                float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (int h = 0; h < fold; ++h) {
                    float4 v[kMaxCluster];
#pragma unroll
                    for (int r = 0; r < kMaxCluster; ++r)
                        if (r < blocks) v[r] = lds_cluster(cluster_addr(shi + (h * all + f) * 16, r));
#pragma unroll
                    for (int r = 0; r < kMaxCluster; ++r)
                        if (r < blocks) t.x += v[r].x, t.y += v[r].y, t.z += v[r].z, t.w += v[r].w;
                }
                sts128(shi + f * 16, make_uint4(__float_as_uint(t.x), __float_as_uint(t.y), __float_as_uint(t.z), __float_as_uint(t.w)));
            }
            cluster_sync();
            for (int f0 = threadIdx.x; f0 < used; f0 += 8 * kBlockThreads) {
                float4 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int f = f0 + i * kBlockThreads;
                    if (f < used && f >> shift != rank) v[i] = lds_cluster(cluster_addr(shi + f * 16, f >> shift));
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int f = f0 + i * kBlockThreads;
                    if (f < used && f >> shift != rank)
                        sts128(shi + f * 16, make_uint4(__float_as_uint(v[i].x), __float_as_uint(v[i].y), __float_as_uint(v[i].z),
                                                        __float_as_uint(v[i].w)));
                }
            }
            cluster_sync();   // the block has all sums, and no block reads another's any more
            if (rows_used && own_part)
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (q * 4 < per) {
                        const uint4 f = lds128(quad(q));
                        av[4 * q] = __uint_as_float(f.x), av[4 * q + 1] = __uint_as_float(f.y);
                        av[4 * q + 2] = __uint_as_float(f.z), av[4 * q + 3] = __uint_as_float(f.w);
                    }
            __syncthreads();
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (q * 8 < per) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = av[8 * q + e] = rows_used && own_part ? av[8 * q + e] * kInvScale : 0.0f;
                const uint32_t p = place(row, quarter * per + q * 8);
                split8<false>(shi + p, slo + p, 0u, x);   // zeros in the rows past the matrix's
            }
        operands_done();

        // ---- A A, and B in A's place
        if (warp == 0 && elect_one()) {
            issue(std::false_type{}, kGramCol, kCrossCol, square, dsh, dsl, dsh, dsl, side / 64);
        }
        products_done();
        if (rows_used)
#pragma unroll
            for (int q = 0; q < 2; ++q)
                if (q * 16 < per) {
                    float v[16], y[16];
                    tmem_load16(lanes + kGramCol + quarter * per + q * 16, lanes + kCrossCol + quarter * per + q * 16, v, y);
#pragma unroll
                    for (int p8 = 0; p8 < 2; ++p8) {
                        float x[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int i = p8 * 8 + e;
                            x[e] = fmaf(Q.b, av[q * 16 + i], Q.c * kInvScale * (v[i] + y[i]));
                        }
                        const uint32_t p = place(row, quarter * per + q * 16 + p8 * 8);
                        split8<false>(shi + p, slo + p, 0u, x);
                    }
                }
        operands_done();

        // ---- B X, and the new X in its place
        if (warp == 0 && elect_one()) {
            issue(std::true_type{}, kUpdateCol, kUpdateCol, update, dsh, dsl, mxh, mxl, side / 64);
        }
        products_done();
        if (rows_used)
            for (int q = quarter; q < Q.slice / 32; q += 4) {
                float v[32];
                tmem_load32(lanes + kUpdateCol + q * 32, v);
#pragma unroll
                for (int p8 = 0; p8 < 4; ++p8) {
                    const uint32_t p = place(row, q * 32 + p8 * 8);
                    const uint32_t at = xrest + rest_place(row, q * 32 + p8 * 8);
                    float x[8], l[8];
                    unpack8(lds128(xhi + p), x);
                    unpack8(lds128(xlo + p), l);
                    if (kRest) {
                        const uint2 rest = lds64(at);
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            const float2 t = rest_values(static_cast<uint16_t>((e < 4 ? rest.x : rest.y) >> e % 4 * 8));
                            l[e] += t.x, l[e + 1] += t.y;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = fmaf(Q.a, x[e] + l[e], kInvScale * v[p8 * 8 + e]);
                    split8<kRest>(xhi + p, xlo + p, at, x);
                }
            }
    }
    __syncthreads();

    // the update, as u came
    if (!blocked && !dead)
        for (int k = k0; k < inner; k += lanes_of_row * 4)
            for (int o0 = group; o0 < outer; o0 += groups * kRowsAtOnce) {
                const int left = min(4, inner - k);
                float w[kRowsAtOnce][4];
                if (Q.w)
#pragma unroll
                    for (int i = 0; i < kRowsAtOnce; ++i) {
                        const int o = o0 + i * groups;
                        if (o >= outer) continue;
                        const float* from = Q.w + value_at(o, k);
                        if (Q.vec) {
                            Pack<float, 4> q;
                            q.load(from);
                            q.get(w[i]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e) w[i][e] = e < left ? from[e] : 0.0f;
                        }
                    }
#pragma unroll
                for (int i = 0; i < kRowsAtOnce; ++i) {
                    const int o = o0 + i * groups;
                    if (o >= outer) continue;
                    float x[4];
                    if (Q.tall) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            int y = k + min(e, left - 1), c = o;
                            held(y, c);
                            const uint32_t p = place(y, c);
                            x[e] = __half2float(lds_half(xhi + p)) + __half2float(lds_half(xlo + p));
                        }
                    } else {
                        int y = o, c = k;
                        held(y, c);
                        const uint32_t p = place(y, c);
                        const uint2 h = lds64(xhi + p), l = lds64(xlo + p);
                        const float2 h0 = __half22float2(*reinterpret_cast<const __half2*>(&h.x)), h1 = __half22float2(*reinterpret_cast<const __half2*>(&h.y));
                        const float2 l0 = __half22float2(*reinterpret_cast<const __half2*>(&l.x)), l1 = __half22float2(*reinterpret_cast<const __half2*>(&l.y));
                        x[0] = h0.x + l0.x, x[1] = h0.y + l0.y, x[2] = h1.x + l1.x, x[3] = h1.y + l1.y;
                    }
                    const int64_t at = value_at(o, k);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[e] *= kInvScale;
                        if (Q.w) x[e] = fmaf(Q.decay, w[i][e], -Q.lr * x[e]);
                    }
                    float* to = Q.w ? Q.w : static_cast<float*>(Q.out);
                    if (Q.out_bf16) {
                        bf16* out = static_cast<bf16*>(Q.out) + at;
                        if (Q.vec) {
                            const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
                            *reinterpret_cast<uint2*>(out) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (e < left) out[e] = __float2bfloat16_rn(x[e]);
                        }
                    } else if (Q.vec) {
                        Pack<float, 4>::put(to + at, x);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (e < left) to[at + e] = x[e];
                    }
                }
            }
    if (dead && threadIdx.x == 0) set_error(Q.d_err, SPARSE_ERR_INTERNAL);
    if (warp == 0 && dead && elect_one()) {   // products in flight finish before their memory is given back
        const uint32_t drain = smem_addr(bar_mem + 1);   // (by mbar_wait here the kernel's registers spilled)
        tc_commit<1>(drain);
        for (const uint64_t t0 = now_ns(); !mbar_try(drain, 0) && now_ns() - t0 < 2000000000ull;) {
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_free<1>(tmem, kTmemCols);
}

// Clusters of `blocks` blocks that the GPU holds at once.
int clusters_at_once(int blocks)
{
    static std::atomic<int> known[kMaxCluster + 1];
    int n = known[blocks].load(std::memory_order_relaxed);
    if (n == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(blocks);
        cfg.blockDim = dim3(kBlockThreads);
        cfg.dynamicSmemBytes = kSmallSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = blocks;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (allow_smem((k_muon_cluster<true, kOnePart>), kSmallSmem, kSmallSmem) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, (k_muon_cluster<true, kOnePart>), &cfg) != cudaSuccess) n = 0;
        n = std::max(n, 1);
        known[blocks].store(n, std::memory_order_relaxed);
    }
    return n;
}

// How a matrix is laid out over a cluster, and what the batch then takes, in tenths of a microsecond.
struct Fold {
    int fold, blocks, slice;
    int64_t cost;
};

// The cheapest layout (fold 0: none has room).  One round of clusters takes, measured at five steps:
//   m <= 64, one part a block   26 us (64 columns), 30 (128), 40 (256); 12 more where blocks exchange sums
//   m > 64                      38, 41 and 54 us; 24 more
//   several parts a block       50, 57 and 74 us, sums over parts included
// and about 2 us more for every doubling of the blocks past two.  (300 x (32 x 512): 117 us in four
// parts of a block, 198 in two blocks; 32 x 512 alone: 57 and 50, and 37 in eight blocks.)
Fold fold_of(int64_t batch, int64_t m, int64_t n)
{
    Fold best{0, 0, 0, INT64_MAX};
    for (int fold = 1; fold <= 4 && m <= kRows / fold; fold *= 2)
        for (int blocks = 1; blocks <= kMaxCluster; blocks *= 2) {
            const int64_t parts = static_cast<int64_t>(fold) * blocks, slice = ((n + parts - 1) / parts + 63) / 64 * 64;
            if (slice > kSlice || parts / 2 * slice >= n) continue;   // no room, or half as many would do
            const int64_t more = slice / 64 - 1;   // 64 columns each
            int64_t round;
            if (fold > 1) round = 500 + 50 * more + 10 * more * more;
            else if (m > 64) round = 380 + 20 * more + 10 * more * more + (blocks > 1 ? 240 : 0);
            else round = 260 + 35 * more + 4 * more * more + (blocks > 1 ? 120 : 0);
            for (int b = 4; b <= blocks; b *= 2) round += 20;
            const int64_t at_once = clusters_at_once(blocks), cost = (batch + at_once - 1) / at_once * round;
            if (cost < best.cost) best = {fold, blocks, static_cast<int>(slice), cost};
        }
    return best;
}

}  // namespace

// Where the cheapest layout beats the general path, whose launches take 85 us and 1.6 us (2.9 with more than
// 64 rows) for every 1000 columns: 64 x 128 fp32 29 us against 91, 30 x 8192 80 against 193, 11 x (64 x
// 4000) 80 against 199, 300 x (32 x 512) 117 against 311; but 48 x (48 x 3195), four rounds, 385
// against 336.
bool muon_fits_cluster(int64_t batch, int64_t m, int64_t n)
{
    if (m > kRows || n > static_cast<int64_t>(kMaxCluster) * kSlice * 4) return false;
    const Fold f = fold_of(batch, m, n);
    return f.fold > 0 && f.cost < 850 + batch * n * (m > 64 ? 29 : 16) / 1000;
}

cudaError_t muon_cluster(const MuonParams& M, const Update& U, const float2* part, int parts, uint32_t* verdict, bool vec,
                         cudaStream_t s)
{
    Small Q{};
    Q.size = M.r * M.cols;
    Q.tall = M.r > M.cols;
    Q.m = static_cast<int>(std::min(M.r, M.cols));
    Q.n = static_cast<int>(std::max(M.r, M.cols));
    const Fold F = fold_of(M.batch, Q.m, Q.n);
    const int blocks = F.blocks;
    Q.fold = F.fold;
    Q.slice = F.slice;
    Q.steps = M.steps;
    Q.a = M.a, Q.b = M.b, Q.c = M.c, Q.eps = M.eps, Q.eps_raised = M.eps_raised;
    Q.part = part;
    Q.parts = parts;
    Q.buf = M.buf;
    Q.out = M.out;
    Q.out_bf16 = M.w == nullptr && M.out_bf16;
    Q.vec = M.cols % 4 == 0 && (reinterpret_cast<uintptr_t>(M.w) | reinterpret_cast<uintptr_t>(M.out)) % (Q.out_bf16 ? 8 : 16) == 0;
    Q.w = M.w;
    Q.decay = M.decay;
    Q.lr = M.lr;
    Q.verdict = verdict;
    Q.d_err = M.d_err;
    auto* kernel = Q.m <= kRestRows ? (vec ? k_muon_cluster<true, kRests> : k_muon_cluster<false, kRests>)
                   : F.fold > 1     ? (vec ? k_muon_cluster<true, kParts> : k_muon_cluster<false, kParts>)
                                    : (vec ? k_muon_cluster<true, kOnePart> : k_muon_cluster<false, kOnePart>);
    const uint32_t smem = kSmallSmem + (Q.m <= kRestRows ? kRestBytes : 0);   // (what is not asked for is cache)
    const cudaError_t ready = allow_smem(kernel, smem, smem);
    if (ready != cudaSuccess) return ready;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(M.batch * blocks));
    cfg.blockDim = dim3(kBlockThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = blocks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    SO_PROFILE("muon_cluster", s);
    return cudaLaunchKernelEx(&cfg, kernel, U, Q, blocks);
}

}  // namespace so
