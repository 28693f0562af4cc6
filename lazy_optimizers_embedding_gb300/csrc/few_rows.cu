// few_rows.cu -- see few_rows.cuh.  All three are bound by the matrices' bytes; sums are fp32 products and sums in a fixed order.
#include "few_rows.cuh"

namespace so {

namespace {

constexpr int kFewBlock = 256, kFewWarps = kFewBlock / 32;
constexpr int kR = 16;                 // rows at a time at most
constexpr int kOut = 0, kScores = 1, kSlopes = 2;   // what becomes of dot products: results, running sums, the loss's slopes
constexpr int kDotTile = 128;          // rows of a matrix of a block: 16 a warp
constexpr int kDotChunk = 1024;        // columns of x in shared memory
constexpr int kCols = 128;             // columns of a block of sums or outer products, four a lane

int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a; }

// Rows t0 to t1 by passes of 16, 8 or 4, the fewest that hold what is left: 16 are bound by instructions (the scores of 1, 4, 8 and 16 tokens
// against 1M x 64: 54, 53, 75 and 123 us, by passes of 16 124).
template <class F>
__device__ __forceinline__ void by_rows(int64_t t0, int64_t t1, F pass)
{
    for (int64_t t = t0; t < t1; t += kR)
        if (t1 - t <= 4)
            pass(std::integral_constant<int, 4>(), t);
        else if (t1 - t <= 8)
            pass(std::integral_constant<int, 8>(), t);
        else
            pass(std::integral_constant<int, kR>(), t);
}

// A group's rows; none, and the error, where the offsets are no offsets.
__device__ __forceinline__ void rows_of(const int64_t* offsets, int e, int64_t n, int32_t* d_err, int64_t& t0, int64_t& t1)
{
    t0 = 0, t1 = n;
    if (offsets == nullptr) return;
    t0 = offsets[e], t1 = offsets[e + 1];
    if (t0 < 0 || t1 < t0 || t1 > n || (e == 0 && t0 != 0)) {
        if (threadIdx.x == 0) set_error(d_err, SPARSE_ERR_INDEX_OUT_OF_RANGE);
        t0 = t1 = 0;
    }
}

// Four values of a row: neighbours by one access (kVec), or every L-th from `i` on, zeros past the row's end.
template <bool kVec, int L>
__device__ __forceinline__ void four(const float* row, int64_t i, int64_t end, float (&v)[4])
{
    if (kVec) {
        Pack<float, 4> q;
        q.zero();
        if (i < end) q.load(row + i);
        q.get(v);
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = i + q * L < end ? row[i + q * L] : 0.0f;
    }
}

// ------------------------------------------------------------- dot products
// Eight lanes have a row of the matrix, 128 bytes at a time, a warp 4 sets of 4 rows; x comes from shared memory, where the
// four rows' lanes read the same places.  A lane's 4 R sums (4 rows, R tokens) are then added up over the eight lanes by halves:
// after three exchanges a lane has a row's sums for half of the tokens.
// kRows: of the one group of the loss's forms, 0 where groups differ.
template <bool kVec, int kMode, int kRows>
__global__ void __launch_bounds__(kFewBlock, 2) k_few_dots(const FewDots D, int tiles, int chunk)
{
    pdl_wait();
    if (kMode != kOut) pdl_release();        // writes the workspace and the error word
    extern __shared__ float xs[];            // [kR][chunk + 4]
    __shared__ int targets[kR];
    __shared__ float2 numbers[kR];           // lse and dloss
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l8 = lane & 7, rowl = lane >> 3;
    const int ld = chunk + 4;
    const bool b2 = lane & 4, b1 = lane & 2, b0 = lane & 1;
    const int set = (b2 ? 2 : 0) + (b1 ? 1 : 0);   // what a lane has after the exchanges
    const int64_t all = static_cast<int64_t>(D.groups) * tiles;
    if (kMode == kOut) {                     // zeros behind the last group
        const int64_t end = min(max(D.offsets[D.groups], static_cast<int64_t>(0)), D.n);
        for (int64_t i = end * D.m + static_cast<int64_t>(blockIdx.x) * kFewBlock + threadIdx.x; i < D.n * D.m; i += static_cast<int64_t>(gridDim.x) * kFewBlock)
            D.out[i] = 0.0f;
    }
    constexpr int kEach = kRows > 0 ? kRows / 2 : 1;   // tokens of a lane
    float top[kEach], sum[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) top[i] = -INFINITY, sum[i] = 0.0f;
    if (kMode != kOut) {
        if (threadIdx.x < kR) {
            const int64_t t = threadIdx.x, g = t < D.n ? D.target[t] : -1;
            if (g < -1 || g >= D.m) set_error(D.d_err, SPARSE_ERR_INDEX_OUT_OF_RANGE);
            targets[t] = g < 0 || g >= D.m ? -1 : static_cast<int>(g);
            if (kMode == kSlopes && targets[t] >= 0) numbers[t] = make_float2(D.lse[t], D.dloss ? D.dloss[t] : 1.0f);
        }
        __syncthreads();
    }
    int64_t held_t = -1, held_k = -1;        // which part of x shared memory has
    for (int64_t tile = blockIdx.x; tile < all; tile += gridDim.x) {
        const int e = static_cast<int>(tile / tiles);
        const int64_t m0 = (tile - static_cast<int64_t>(e) * tiles) * kDotTile + warp * 16;
        int64_t t0, t1;
        rows_of(D.offsets, e, D.n, D.d_err, t0, t1);
        const float* rows[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) rows[s] = D.w + (e * D.m + min(m0 + s * 4 + rowl, D.m - 1)) * D.k;
        auto pass = [&](auto size, int64_t t) {
            constexpr int R = decltype(size)::value;
            const int r0 = b0 ? R / 2 : 0;
            float acc[4 * R];
#pragma unroll
            for (int i = 0; i < 4 * R; ++i) acc[i] = 0.0f;
            for (int64_t k0 = 0; k0 < D.k; k0 += chunk) {
                const int64_t kend = min(D.k, k0 + chunk);
                if (held_t != t || held_k != k0) {
                    __syncthreads();
                    for (int r = warp; r < R; r += kFewWarps)
                        for (int i = lane; i < chunk; i += 32)
                            xs[r * ld + i] = t + r < t1 && k0 + i < D.k ? D.x[(t + r) * D.k + k0 + i] : 0.0f;
                    __syncthreads();
                    held_t = t, held_k = k0;
                }
#pragma unroll 2
                for (int64_t k = k0; k < kend; k += 32) {
                    float v[4][4];
                    const int64_t at = k + (kVec ? 4 * l8 : l8);
#pragma unroll
                    for (int s = 0; s < 4; ++s) four<kVec, 8>(rows[s], at, kend, v[s]);
                    const float* xr = xs + (at - k0);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        float u[4];
                        if (kVec) {
                            const float4 q = *reinterpret_cast<const float4*>(xr + r * ld);
                            u[0] = q.x, u[1] = q.y, u[2] = q.z, u[3] = q.w;
                        } else {
#pragma unroll
                            for (int q = 0; q < 4; ++q) u[q] = xr[r * ld + 8 * q];
                        }
#pragma unroll
                        for (int s = 0; s < 4; ++s)
#pragma unroll
                            for (int q = 0; q < 4; ++q) acc[s * R + r] = fmaf(v[s][q], u[q], acc[s * R + r]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 2 * R; ++i) {
                const float keep = b2 ? acc[i + 2 * R] : acc[i], give = b2 ? acc[i] : acc[i + 2 * R];
                acc[i] = keep + __shfl_xor_sync(kFull, give, 4);
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float keep = b1 ? acc[i + R] : acc[i], give = b1 ? acc[i] : acc[i + R];
                acc[i] = keep + __shfl_xor_sync(kFull, give, 2);
            }
#pragma unroll
            for (int i = 0; i < R / 2; ++i) {
                const float keep = b0 ? acc[i + R / 2] : acc[i], give = b0 ? acc[i] : acc[i + R / 2];
                acc[i] = keep + __shfl_xor_sync(kFull, give, 1);
            }
            const int64_t row = m0 + set * 4 + rowl;
            if (row >= D.m) return;
#pragma unroll
            for (int i = 0; i < R / 2; ++i) {
                if constexpr (kMode == kScores) {
                    const float high = fmaxf(top[i], acc[i]), base = high == -INFINITY ? 0.0f : high * kLog2e;
                    sum[i] = sum[i] * exp2_fast(fmaf(top[i], kLog2e, -base)) + exp2_fast(fmaf(acc[i], kLog2e, -base));
                    top[i] = high;
                    if (targets[r0 + i] == row) D.hit[r0 + i] = acc[i];
                } else if constexpr (kMode == kSlopes) {
                    const int q = r0 + i, target = targets[q];
                    const float2 u = numbers[q];
                    const float p = exp2_fast((acc[i] - u.x) * kLog2e) - (target == row ? 1.0f : 0.0f);
                    if (q < D.n) D.out[q * D.m + row] = target >= 0 ? p * u.y : 0.0f;
                } else if (t + r0 + i < t1) {
                    D.out[(t + r0 + i) * D.m + row] = acc[i];
                }
            }
        };
        if constexpr (kRows > 0)
            pass(std::integral_constant<int, kRows>(), t0);
        else
            by_rows(t0, t1, pass);
    }
    if (kMode == kScores) {                  // over the lanes that have the same tokens
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            for (int d = 2; d < 32; d <<= 1) {
                const float t = __shfl_xor_sync(kFull, top[i], d), u = __shfl_xor_sync(kFull, sum[i], d);
                const float high = fmaxf(top[i], t), base = high == -INFINITY ? 0.0f : high;
                sum[i] = sum[i] * exp2_fast((top[i] - base) * kLog2e) + u * exp2_fast((t - base) * kLog2e);
                top[i] = high;
            }
            const int t = (b0 ? kEach : 0) + i;
            if ((lane >> 1) == 0 && t < D.n)
                D.part[(static_cast<int64_t>(blockIdx.x) * kFewWarps + warp) * D.n + t] = make_float2(top[i], sum[i]);
        }
    }
}

// ---------------------------------------------------------------- weighted sums
// A warp has every eighth four of the matrix's rows, a lane four of 128 columns and 16 tokens' sums of them; x comes from shared
// memory by broadcasts of four tokens.  The warps' sums are added up in order.  Where there are at most 64 columns half a warp is a team with rows
// of its own (1M x 64 and a token, dx with the slopes: 173 us, by whole warps 217).
template <bool kVec, bool kNarrow>
__global__ void __launch_bounds__(kFewBlock, 2) k_few_sums(const FewSums D, int tiles)
{
    pdl_enter();   // writes the workspace and the error word
    constexpr int L = kNarrow ? 16 : 32, kTeams = kFewBlock / L, kWide = 4 * L;
    extern __shared__ float smem[];          // [256][kR] of x, then the teams' sums [kTeams][kR][kWide]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, team = threadIdx.x / L, l = threadIdx.x % L;
    const int64_t all = static_cast<int64_t>(D.groups) * tiles * D.splits;
    for (int64_t item = blockIdx.x; item < all; item += gridDim.x) {
        const int split = static_cast<int>(item % D.splits);
        const int64_t u = item / D.splits;
        const int e = static_cast<int>(u / tiles);
        const int64_t c0 = (u - static_cast<int64_t>(e) * tiles) * kWide;
        const int64_t ka = D.k * split / D.splits, kb = D.k * (split + 1) / D.splits;
        const int64_t col = c0 + (kVec ? 4 * l : l);
        int64_t t0, t1;
        rows_of(D.offsets, e, D.n, D.d_err, t0, t1);
        auto pass = [&](auto size, int64_t t) {
            constexpr int R = decltype(size)::value;
            float acc[R][4];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[r][q] = 0.0f;
            for (int64_t kc = ka; kc < kb; kc += 256) {
                __syncthreads();
                for (int r = warp; r < R; r += kFewWarps)
                    for (int i = lane; i < 256; i += 32)
                        smem[i * R + r] = t + r < t1 && kc + i < kb ? D.x[(t + r) * D.k + kc + i] : 0.0f;
                __syncthreads();
#pragma unroll (R <= 8 ? 2 : 1)
                for (int i0 = team * 4; i0 < 256 && kc + i0 < kb; i0 += 4 * kTeams) {
                    float v[4][4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int64_t k = kc + i0 + j;
                        if (k < kb)
                            four<kVec, L>(D.w + (e * D.k + k) * D.m, col, D.m, v[j]);
                        else
                            v[j][0] = v[j][1] = v[j][2] = v[j][3] = 0.0f;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int r = 0; r < R; r += 4) {
                            const float4 q = *reinterpret_cast<const float4*>(smem + (i0 + j) * R + r);
                            const float f[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int p = 0; p < 4; ++p) acc[r + i][p] = fmaf(f[i], v[j][p], acc[r + i][p]);
                        }
                }
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int q = 0; q < 4; ++q) smem[(team * R + r) * kWide + (kVec ? 4 * l + q : l + L * q)] = acc[r][q];
            __syncthreads();
            for (int i = threadIdx.x; i < R * kWide; i += kFewBlock) {
                const int r = i / kWide, c = i % kWide;
                float s = 0.0f;
#pragma unroll
                for (int p = 0; p < kTeams; ++p) s += smem[(p * R + r) * kWide + c];
                if (t + r < t1 && c0 + c < D.m) D.slabs[(split * D.n + t + r) * D.m + c0 + c] = s;
            }
        };
        by_rows(t0, t1, pass);
    }
}

// --------------------------------------------------------------- outer products
// A warp has 8 rows of 128 columns of the result; the tokens go by one after the other.
template <bool kVec>
__global__ void __launch_bounds__(kFewBlock) k_few_outer(const FewOuter D, int64_t tiles_a, int tiles_b)
{
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t all = D.groups * tiles_a * tiles_b;
    for (int64_t item = blockIdx.x; item < all; item += gridDim.x) {
        const int64_t u = item / tiles_b;
        const int e = static_cast<int>(u / tiles_a);
        const int64_t a0 = (u - e * tiles_a) * 64 + warp * 8, col = (item - u * tiles_b) * kCols + (kVec ? 4 * lane : lane);
        int64_t t0, t1;
        rows_of(D.offsets, e, D.n, D.d_err, t0, t1);
        const int have = static_cast<int>(min(D.a - a0, static_cast<int64_t>(8)));
        if (have <= 0) continue;
        float acc[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[i][q] = 0.0f;
#pragma unroll 2
        for (int64_t t = t0; t < t1; ++t) {
            if (D.target != nullptr && (D.target[t] < 0 || D.target[t] >= D.a)) continue;   // whatever lies in the row
            float v[4];
            four<kVec, 32>(D.y + t * D.b, col, D.b, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float f = i < have ? D.x[t * D.a + a0 + i] : 0.0f;
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[i][q] = fmaf(f, v[q], acc[i][q]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= have) continue;
            float* to = D.out + (e * D.a + a0 + i) * D.b + col;
            if (kVec) {
                if (col < D.b) Pack<float, 4>::put(to, acc[i]);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (col + 32 * q < D.b) to[32 * q] = acc[i][q];
            }
        }
    }
}

bool whole(const void* p, int64_t cols) { return cols % 4 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Blocks that the matrices' rows are shared out to: two an SM.
int64_t dot_blocks(int64_t tiles) { return std::min<int64_t>(tiles, 2 * kSms); }

}  // namespace

int few_dot_slots(int64_t m) { return static_cast<int>(dot_blocks(up(m, kDotTile)) * kFewWarps); }

cudaError_t few_dots(const FewDots& D, cudaStream_t s)
{
    const int64_t tiles = up(D.m, kDotTile);
    const int chunk = static_cast<int>(std::min<int64_t>(kDotChunk, up(D.k, 32) * 32));
    const size_t smem = sizeof(float) * kR * (chunk + 4), most = sizeof(float) * kR * (kDotChunk + 4);
    const int64_t blocks = D.target == nullptr ? std::min<int64_t>(tiles * D.groups, 4 * kSms) : dot_blocks(tiles);
    SO_PROFILE("few_dots", s);
    auto go = [&](auto* kernel) {
        const cudaError_t e = allow_smem(kernel, smem, most);
        return e != cudaSuccess ? e
                                : launch_smem(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kFewBlock), smem, s, D, static_cast<int>(tiles), chunk);
    };
    const bool vec = whole(D.w, D.k);
    auto loss = [&](auto rows) {
        constexpr int R = decltype(rows)::value;
        if (D.part != nullptr) return vec ? go(k_few_dots<true, kScores, R>) : go(k_few_dots<false, kScores, R>);
        if constexpr (R <= kFewGrad) return vec ? go(k_few_dots<true, kSlopes, R>) : go(k_few_dots<false, kSlopes, R>);
        return cudaErrorInvalidValue;
    };
    if (D.target == nullptr) return vec ? go(k_few_dots<true, kOut, 0>) : go(k_few_dots<false, kOut, 0>);
    if (D.n <= 4) return loss(std::integral_constant<int, 4>());
    return D.n <= 8 ? loss(std::integral_constant<int, 8>()) : loss(std::integral_constant<int, kR>());
}

int few_sums_splits(int64_t n, int64_t m, int64_t k, int64_t groups)
{
    const int64_t tiles = std::min(n, groups) * up(m, kCols);
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({up(3 * kSms, tiles), up(k, 256), 512})));
}

cudaError_t few_sums(const FewSums& D, cudaStream_t s)
{
    const bool narrow = D.m <= kCols / 2;
    const int tiles = static_cast<int>(up(D.m, kCols));
    const size_t smem = sizeof(float) * kFewWarps * kR * kCols;
    const int64_t blocks = std::min<int64_t>(static_cast<int64_t>(D.groups) * tiles * D.splits, 64 * kSms);
    SO_PROFILE("few_sums", s);
    auto go = [&](auto* kernel) {
        const cudaError_t e = allow_smem(kernel, smem, smem);
        return e != cudaSuccess ? e : launch_smem(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kFewBlock), smem, s, D, tiles);
    };
    if (narrow) return whole(D.w, D.m) ? go(k_few_sums<true, true>) : go(k_few_sums<false, true>);
    return whole(D.w, D.m) ? go(k_few_sums<true, false>) : go(k_few_sums<false, false>);
}

cudaError_t few_outer(const FewOuter& D, cudaStream_t s)
{
    const int64_t tiles_a = up(D.a, 64);
    const int tiles_b = static_cast<int>(up(D.b, kCols));
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(tiles_a * tiles_b * D.groups, 64 * kSms)));
    SO_PROFILE("few_outer", s);
    auto go = [&](auto* kernel) { return launch(kernel, grid, dim3(kFewBlock), s, D, tiles_a, tiles_b); };
    return whole(D.y, D.b) && whole(D.out, D.b) ? go(k_few_outer<true>) : go(k_few_outer<false>);
}

}  // namespace so
