// product_rows.cu -- rows by the matrix of their group, what packs operands for the
// products, and what joins the sums of a long inner dimension's parts.
#include "product.cuh"

namespace so {

namespace {

constexpr int kPackBlock = 256;

// Eight values from `from` on, those below `left`.  (Pairs of values by neighbouring lanes: 45 against 41 us at 9003 x 515 and 19055 x 771
// fp32, the stores being four times as many.)
template <class T, bool kVec>
__device__ __forceinline__ void read8(const T* from, int64_t left, float (&x)[8])
{
    if (kVec) {
        Pack<T, 8> q;
        q.load(from);
        q.get(x);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            Pack<T, 1> q;
            float one[1];
            q.zero();
            if (e < left) q.load(from + e);
            q.get(one);
            x[e] = one[0];
        }
    }
}

// A part of v: its bf16, one that stays finite where v is (values above bf16's largest, which would round to
// infinity, are cut off; what is left goes to the next part).
__device__ __forceinline__ float part_of(float v)
{
    const float h = __bfloat162float(__float2bfloat16_rn(v));
    return isinf(h) && isfinite(v) ? __uint_as_float(__float_as_uint(v) & 0xffff0000u) : h;
}

template <class T, bool kVec>
__device__ __forceinline__ void pack_rows(const Pack1& A, int64_t warp, int64_t warps, int lane)
{
    constexpr int kParts = sizeof(T) == 4 ? 3 : 1;
    const int64_t lanes = (A.cols + 7) / 8;
    const int G = lanes > 16 ? 32 : lanes > 8 ? 16 : lanes > 4 ? 8 : lanes > 2 ? 4 : static_cast<int>(lanes);
    const int each = 32 / G;                              // rows of a warp at a time
    const int64_t size = A.rows * A.ld;
    for (int64_t r = warp * each + lane / G; r < A.rows; r += warps * each) {
        if (A.offsets != nullptr) {     // 10 bytes a value for nothing
            const int64_t g = r / A.each;
            if (A.offsets[g] == A.offsets[g + 1]) continue;
        }
        bool none = false;
        if (A.target != nullptr) {
            const int64_t g = A.target[r];
            none = g < 0 || g >= A.v;
        }
        for (int64_t i = lane % G * 8; i < A.cols; i += G * 8) {
            float x[8];
            read8<T, kVec>(static_cast<const T*>(A.from) + r * A.cols + i, A.cols - i, x);
            if (none)
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = 0.0f;
            bf16* to = A.to + r * A.ld + i;
            if (kParts == 1) {
                Pack<bf16, 8>::put(to, x);
                continue;
            }
            bool plain = true;   // nothing that is not finite, or not as bf16
#pragma unroll
            for (int e = 0; e < 8; ++e) plain = plain && fabsf(x[e]) <= 3.38e38f;
            if (plain) {         // (with every value looked at for itself: 42 us and not 34 at 7200 x 515 and 19055 x 771)
#pragma unroll
                for (int p = 0; p < kParts; ++p) {
                    uint4 w;
                    uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        u[e] = bf16_pair(x[2 * e], x[2 * e + 1]);
                        const float2 h = pair_floats(u[e]);
                        x[2 * e] -= h.x, x[2 * e + 1] -= h.y;
                    }
                    *reinterpret_cast<uint4*>(to + p * size) = w;
                }
                continue;
            }
#pragma unroll
            for (int p = 0; p < kParts; ++p) {
                float h[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    h[e] = part_of(x[e]);
                    x[e] = isfinite(h[e]) ? x[e] - h[e] : 0.0f;   // an infinity or NaN is all in the first part
                }
                Pack<bf16, 8>::put(to + p * size, h);
            }
        }
    }
}

// Rows of one or two arrays as bf16 with aligned rows: fp32 in three parts, hi = bf16(v), mid = bf16(v - hi), lo = what
// those leave (2^-26 of v at most).  Bound by memory: 4 bytes in, 6 out.
template <class T, bool kVec>
__global__ void __launch_bounds__(kPackBlock) k_pack(const Pack1 A, const Pack1 B, const TokenRows R, int blocks_a, int blocks_b)
{
    pdl_enter();   // writes the workspace and the error word
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, per = kPackBlock / 32, block = blockIdx.x;
    if (block < blocks_a)
        pack_rows<T, kVec>(A, static_cast<int64_t>(block) * per + w, static_cast<int64_t>(blocks_a) * per, lane);
    else if (block < blocks_a + blocks_b)
        pack_rows<T, kVec>(B, static_cast<int64_t>(block - blocks_a) * per + w, static_cast<int64_t>(blocks_b) * per, lane);
    else {
        const float unit = R.unit != nullptr ? common_unit(R.dloss, R.target, R.n, lane) : 1.0f;
        if (R.unit != nullptr && block == blocks_a + blocks_b && threadIdx.x == 0) *R.unit = unit;
        put_token(R, (block - blocks_a - blocks_b) * kPackBlock + static_cast<int>(threadIdx.x), unit);
    }
}

// Sums of slabs in order, four neighbours a thread.
template <class T, bool kVec>
__device__ __forceinline__ void join_rows(const Join& J, T* __restrict__ out, int block, int blocks)
{
    const int64_t groups = (J.cols + 3) / 4, count = J.rows * groups;
    const int64_t live = J.end ? min(max(*J.end, static_cast<int64_t>(0)), J.rows) : J.rows;
    for (int64_t i = static_cast<int64_t>(block) * 256 + threadIdx.x; i < count; i += static_cast<int64_t>(blocks) * 256) {
        const int64_t row = (count >> 32) == 0 ? static_cast<uint32_t>(i) / static_cast<uint32_t>(groups) : i / groups;
        const int col = static_cast<int>(i - row * groups) * 4, left = static_cast<int>(min(J.cols - col, static_cast<int64_t>(4)));
        const int64_t at = row * J.cols + col;
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (row < live) {
#pragma unroll 4
            for (int q = 0; q < J.slabs; ++q) {
                float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if (kVec) {
                    Pack<float, 4> k;
                    k.load(J.from + q * J.slab + at);
                    k.get(v);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e < left) v[e] = J.from[q * J.slab + at + e];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) s[e] += v[e];
            }
        }
        if (kVec && sizeof(T) == 4) {
            Pack<float, 4>::put(reinterpret_cast<float*>(out) + at, s);
        } else if (kVec) {
            uint2 w;
            w.x = bf16_pair(s[0], s[1]);
            w.y = bf16_pair(s[2], s[3]);
            *reinterpret_cast<uint2*>(out + at) = w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < left) out[at + e] = T(s[e]);
        }
    }
}

// Of one or two arrays in one launch.
template <class T, bool kVec>
__global__ void __launch_bounds__(256) k_join_slabs(const Join A, T* a, const Join B, T* b, int blocks_a)
{
    pdl_wait();
    if (static_cast<int>(blockIdx.x) < blocks_a)
        join_rows<T, kVec>(A, a, blockIdx.x, blocks_a);
    else
        join_rows<T, kVec>(B, b, static_cast<int>(blockIdx.x) - blocks_a, static_cast<int>(gridDim.x) - blocks_a);
}

int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a; }

// Pairs of blocks take 256 rows of M: not where those would leave much of a tile empty, nor where
// there are fewer tiles than pairs.
bool wants_pair(int64_t m, int64_t tiles_of_128)
{
    return up(m, 256) * 2 <= up(m, 128) + up(m, 128) / 4 && tiles_of_128 >= kSms;
}

// Tiles at most: every group may end in a part of one.
int64_t row_tiles(int64_t rows, int64_t groups, int64_t width) { return groups == 1 ? up(rows, width) : rows / width + std::min(rows, groups); }

template <class S>
cudaError_t rows_form(const RowsProduct& R, cudaStream_t s)
{
    ProductMaps maps;
    if (!R.a.map(&maps.a) || !R.b.map(&maps.b)) return cudaErrorInvalidValue;
    ProductArgs Q{};
    Q.rows = static_cast<int32_t>(R.rows);
    Q.m = static_cast<int32_t>(R.m);
    Q.k = static_cast<int32_t>(R.k);
    Q.m_tiles = static_cast<int32_t>(up(R.m, S::TM));
    Q.width = S::BN;
    const int64_t units = kSms / S::kPair;
    if (R.groups == 1) {   // the width whose rounds over the GPU take least; a stage: see stage_cycles
        int64_t best = INT64_MAX;
        for (int w = S::BN; w >= 64; w -= 32) {
            const int64_t cost = up(up(R.rows, w) * Q.m_tiles * R.splits, units) * stage_cycles<S>(w);
            if (cost < best) best = cost, Q.width = w;
        }
    }
    Q.groups = R.groups;
    Q.splits = R.splits;
    Q.offsets = R.offsets;
    Q.out = R.out;
    Q.add = R.add ? static_cast<const float*>(R.out) : nullptr;
    Q.slab = R.rows * R.m;
    Q.ld = static_cast<int32_t>(R.m);
    Q.out_bf16 = R.out_bf16;
    Q.clear = R.clear;
    Q.release = R.release;
    Q.unit = R.unit;
    Q.d_err = R.d_err;
    return run_product<S>("rows_product", maps, Q, row_tiles(R.rows, R.groups, Q.width) * Q.m_tiles * R.splits, s);
}

}  // namespace

cudaError_t pack(const Pack1& a, const Pack1& b, const TokenRows& tokens, int is_bf16, cudaStream_t s)
{
    auto blocks = [](const Pack1& p) { return std::min<int64_t>(8 * num_sms(), up(p.rows * up(p.ld, 8), 8 * kPackBlock)); };
    const int64_t na = blocks(a), nb = blocks(b), nt = up(tokens.padded, kPackBlock);
    if (na + nb + nt == 0) return cudaSuccess;
    const int v = is_bf16 ? 8 : 4;
    auto fits = [&](const Pack1& p) {
        return p.rows == 0 || (p.cols % 8 == 0 && reinterpret_cast<uintptr_t>(p.from) % (is_bf16 ? 2 * v : 4 * v) == 0);
    };
    const bool vec = fits(a) && fits(b);
    auto go = [&](auto* kernel) {
        return launch(kernel, dim3(static_cast<unsigned>(na + nb + nt)), dim3(kPackBlock), s, a, b, tokens, static_cast<int>(na),
                      static_cast<int>(nb));
    };
    SO_PROFILE("pack", s);
    if (is_bf16) return vec ? go(k_pack<bf16, true>) : go(k_pack<bf16, false>);
    return vec ? go(k_pack<float, true>) : go(k_pack<float, false>);
}

cudaError_t join_two(const Join& a, void* out_a, const Join& b, void* out_b, int out_bf16, cudaStream_t s)
{
    auto blocks = [](const Join& J) { return J.rows > 0 ? std::max<int64_t>(1, std::min<int64_t>(8 * num_sms(), up(J.rows * up(J.cols, 4), 256))) : 0; };
    const int64_t na = blocks(a), nb = blocks(b);
    // the slabs lie in the workspace
    const bool vec = a.cols % 4 == 0 && b.cols % 4 == 0 && ((reinterpret_cast<uintptr_t>(out_a) | reinterpret_cast<uintptr_t>(out_b)) & 15) == 0;
    SO_PROFILE("join_slabs", s);
    auto go = [&](auto* kernel, auto* one, auto* two) {
        return launch(kernel, dim3(static_cast<unsigned>(na + nb)), dim3(256), s, a, one, b, two, static_cast<int>(na));
    };
    if (out_bf16) return go(vec ? k_join_slabs<bf16, true> : k_join_slabs<bf16, false>, static_cast<bf16*>(out_a), static_cast<bf16*>(out_b));
    return go(vec ? k_join_slabs<float, true> : k_join_slabs<float, false>, static_cast<float*>(out_a), static_cast<float*>(out_b));
}

cudaError_t join_slabs(const Join& J, void* out, int out_bf16, cudaStream_t s) { return join_two(J, out, Join{}, nullptr, out_bf16, s); }

int rows_splits(int64_t rows, int64_t m, int64_t k, int64_t groups, int parts)
{
    const int64_t width = parts == 3 ? 128 : 256;
    const int64_t tiles = row_tiles(rows, groups, width) * up(m, 128);
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({kSms / std::max<int64_t>(tiles, 1), up(k, kPK) / 4, 64})));
}

cudaError_t rows_product(const RowsProduct& R, cudaStream_t s)
{
    const int64_t width = R.b.parts == 3 ? 128 : 256;
    const bool pair = R.splits == 1 && wants_pair(R.m, row_tiles(R.rows, R.groups, width) * up(R.m, 128));
    if (R.b.parts == 3) {
        if (R.a_mn)
            return pair ? rows_form<ProductShape<kRows, true, false, 2, 6, false>>(R, s)
                        : rows_form<ProductShape<kRows, true, false, 1, 6, false>>(R, s);
        return pair ? rows_form<ProductShape<kRows, false, false, 2, 6, false>>(R, s)
                    : rows_form<ProductShape<kRows, false, false, 1, 6, false>>(R, s);
    }
    if (R.a_mn)
        return pair ? rows_form<ProductShape<kRows, true, false, 2, 1, false>>(R, s)
                    : rows_form<ProductShape<kRows, true, false, 1, 1, false>>(R, s);
    return pair ? rows_form<ProductShape<kRows, false, false, 2, 1, false>>(R, s)
                : rows_form<ProductShape<kRows, false, false, 1, 1, false>>(R, s);
}

}  // namespace so
