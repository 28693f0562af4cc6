// vocab_back.cu -- the gradient of the loss over a table's rows for narrow rows (at
// most 128 columns), in one launch and without the slopes in memory.
//
//   S = own other^T, G = dloss (exp(S - lse) - [target]), D += G other
//
// An item has 128 rows of its own, tokens (D is their dx) or rows of the table (their dW, G then
// transposed), and goes through rows of the other kind, TN at a time.  Scores come from the tensor unit
// into tensor memory, a warp's lanes have a row each, and their slopes go back to where the scores
// were, as bf16 parts: the A operand of the second product, whose B operand is the other rows' tile
// once more, read as it lies but MN-major.  So memory holds the rows and results alone: with the slopes
// written out (vocab_loss.cu) 2048 x 1M fp32 scores of 64 columns moved 37 GB.
// Two pairs of groups of four warps have every second tile each, a group half of its scores, so that one pair's
// exponentials run beside the other's and both beside the products (one group a tile: 4.9 ms there, the tensor
// unit 55 % active); a fifth (and for 128 columns a sixth) empties D into fp32 sums, which round to nearest,
// every 512 (1024) K values.
#include "product.cuh"
#include "vocab_back.cuh"

namespace so {

namespace {

constexpr int kOwn = 128;                 // rows of an item

template <int P_, int C_>
struct BackShape {
    static constexpr int P = P_, C = C_, kParts = P == 6 ? 3 : 1;
    static constexpr int TN = P == 6 ? 64 : 128;                           // rows of the other kind in a tile
    static constexpr int kBlocks = C / 64;                                 // of 64 columns
    // In shared memory: blocks of 64 columns, in each its parts, in each all rows.  So the first two parts of the other rows are
    // one operand of 2 TN rows.
    static constexpr uint32_t kOwnPart = kOwn * 128, kOtherPart = TN * 128;
    static constexpr uint32_t kOwnBytes = kBlocks * kParts * kOwnPart, kOtherBytes = kBlocks * kParts * kOtherPart;
    static constexpr uint32_t kStage = kOtherBytes + 2048;                 // and the tokens' numbers, 16 bytes each
    static constexpr int kOwns = kOwnBytes <= 48 * 1024 ? 2 : 1;
    static constexpr int kFit = static_cast<int>((224 * 1024 - kOwns * kOwnBytes) / kStage);
    static constexpr int kStages = kFit < 8 ? kFit : 8;
    static constexpr uint32_t kSmem = kOwns * kOwnBytes + kStages * kStage + 1024;
    static constexpr int kSums = C / 64;                                   // groups of warps that empty D, 64 columns each
    static constexpr int kThreads = 64 + (4 + kSums) * 128;
    static constexpr int kScoreCols = kParts > 1 ? 2 * TN : TN;            // = 128: hi and lo sums of TN scores, or one
    static constexpr bool kWide = kParts > 1 && C == 64;                   // three accumulators of D, by the order of their products
    static constexpr int kSumCols = kWide ? 3 * C : kParts > 1 ? 2 * C : C;
    static constexpr int kBufs = (512 - kSumCols) / kScoreCols;            // tiles whose scores or slopes are there at a time: 2 or 3
    static constexpr int kD = kBufs * kScoreCols;                          // D's first column
    static constexpr int kChunk = 8;                                       // tiles of D between two emptyings
    static_assert(kStages >= 2 && kBufs >= 2, "shape");
};

// An item: which rows are its own and which of the other kind it goes through.
struct Item {
    bool tokens;
    int own0, split;
    int j0, j1;              // tiles of the other kind
};

template <class S>
__device__ __forceinline__ Item item_of(const BackArgs& Q, int t)
{
    Item I;
    I.tokens = t < Q.dx_items;
    const int u = I.tokens ? t : t - Q.dx_items;
    const int splits = I.tokens ? Q.dx_splits : Q.dw_splits;
    const int own = u / splits;
    I.split = u - own * splits;
    I.own0 = own * kOwn;
    const int tiles = ((I.tokens ? Q.v : Q.n) + S::TN - 1) / S::TN, each = tiles / splits, more = tiles - each * splits;
    I.j0 = I.split * each + min(I.split, more);   // the first parts have one more
    I.j1 = I.j0 + each + (I.split < more ? 1 : 0);
    return I;
}

struct Maps {
    CUtensorMap x, w;
};

template <class S>
__global__ void __launch_bounds__(S::kThreads, 1) k_loss_back(const __grid_constant__ Maps maps, const BackArgs Q)
{
    constexpr int P = S::P, C = S::C, TN = S::TN, kStages = S::kStages, kParts = S::kParts;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[2 * kStages + 2 * S::kOwns + 2 * S::kBufs + 3];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int dead;
    const uint32_t data = (smem_addr(raw) + 1023u) & ~1023u;
    const uint32_t owns = data, stages = data + S::kOwns * S::kOwnBytes;
    const uint32_t full = smem_addr(bars), empty = full + 8 * kStages, own_full = empty + 8 * kStages, own_empty = own_full + 8 * S::kOwns,
                   scored = own_empty + 8 * S::kOwns, sloped = scored + 8 * S::kBufs, summed = sloped + 8 * S::kBufs, emptied = summed + 8, drain = emptied + 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = blockIdx.x, step = gridDim.x, items = Q.dx_items + Q.dw_items;

    if (threadIdx.x == 32) {   // while the kernel before ends
        tma_prefetch(&maps.x);
        tma_prefetch(&maps.w);
    }
    if (threadIdx.x == 0) {
        dead = 0;
        for (int s = 0; s < kStages; ++s) mbar_init(full + 8 * s, 1), mbar_init(empty + 8 * s, 1);
        for (int s = 0; s < S::kOwns; ++s) mbar_init(own_full + 8 * s, 1), mbar_init(own_empty + 8 * s, 1);
        for (int s = 0; s < S::kBufs; ++s) mbar_init(scored + 8 * s, 1), mbar_init(sloped + 8 * s, 8);
        mbar_init(summed, 1);
        mbar_init(emptied, 4 * S::kSums);
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<1>(&tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_wait();
    if (Q.release) pdl_release();   // after this block's allocation, so that no later block can hold what it waits for
    fence_async_proxy();   // the kernels before wrote with ordinary stores

    if (warp == 0) {
        if (elect_one()) {
            uint32_t it = 0, owned = 0;
            for (int t = first; t < items; t += step, ++owned) {
                const Item I = item_of<S>(Q, t);
                const CUtensorMap *own = I.tokens ? &maps.x : &maps.w, *other = I.tokens ? &maps.w : &maps.x;
                const uint32_t o = owned % S::kOwns;
                if (!mbar_wait(own_empty + 8 * o, (owned / S::kOwns & 1) ^ 1, &dead)) goto copied;
                mbar_expect(own_full + 8 * o, S::kOwnBytes);
#pragma unroll 1
                for (int q = 0; q < kParts * S::kBlocks * (kOwn / 64); ++q)
                    tma_load<1>(owns + o * S::kOwnBytes + q * kPBoxBytes, own, own_full + 8 * o, q / (kOwn / 64 * kParts) * 64,
                                I.own0 + q % (kOwn / 64) * 64, q / (kOwn / 64) % kParts);
#pragma unroll 1
                for (int j = I.j0; j < I.j1; ++j, ++it) {
                    const uint32_t s = it % kStages, at = stages + s * S::kStage;
                    if (!mbar_wait(empty + 8 * s, (it / kStages & 1) ^ 1, &dead)) {
                        ++owned;
                        goto copied;
                    }
                    mbar_expect(full + 8 * s, S::kOtherBytes + (I.tokens ? 0 : TN * 16));
#pragma unroll 1
                    for (int q = 0; q < kParts * S::kBlocks * (TN / 64); ++q)
                        tma_load<1>(at + q * kPBoxBytes, other, full + 8 * s, q / (TN / 64 * kParts) * 64, j * TN + q % (TN / 64) * 64,
                                    q / (TN / 64) % kParts);
                    if (!I.tokens) bulk_load(at + S::kOtherBytes, Q.tokens + static_cast<int64_t>(j) * TN, TN * 16, full + 8 * s);
                }
            }
        copied:
            if (dead) {   // copies in flight land before the block leaves
                volatile int none = 0;
                for (uint32_t s = 0; s < static_cast<uint32_t>(kStages) && s < it; ++s)
                    mbar_wait(full + 8 * s, ((it - 1 - s) / kStages) & 1, &none);
                for (uint32_t o = 0; o < static_cast<uint32_t>(S::kOwns) && o < owned; ++o)
                    mbar_wait(own_full + 8 * o, ((owned - 1 - o) / S::kOwns) & 1, &none);
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {
            constexpr uint32_t score_desc = mma_desc_bf16(kOwn, false, false) | static_cast<uint32_t>(TN >> 3) << 17;
            constexpr uint32_t score_desc2 = mma_desc_bf16(kOwn, false, false) | static_cast<uint32_t>(2 * TN >> 3) << 17;
            constexpr uint32_t sum_desc = mma_desc_bf16(kOwn, false, true) | static_cast<uint32_t>(C >> 3) << 17;
            constexpr uint32_t sum_desc2 = mma_desc_bf16(kOwn, false, true) | static_cast<uint32_t>(2 * C >> 3) << 17;
            constexpr uint32_t sum_desc3 = mma_desc_bf16(kOwn, false, true) | static_cast<uint32_t>(3 * C >> 3) << 17;
            // Scores of tile it, the next, are asked for as soon as its rows are there and the slopes of tile it - kBufs have been used, the
            // second product of tile back_it when its slopes are there, whichever is first: with two stages the
            // rows of the next tile come only after a second product (128 fp32 columns in fixed order: 6350 cycles a tile of 3840 of products).
            uint32_t it = 0, back_it = 0, owned = 0, chunks = 0;
            uint32_t place = 0, ends = 0;            // of the next second product: its place in its item; tiles (by buffer) that end theirs
            int t = first, j = 0;
            Item I{};
            bool fresh_item = true;
            uint64_t since = 0;
            uint32_t spins = 0;
            while (t < items || back_it < it) {
                bool done_something = false;
                if (t < items && it - back_it < S::kBufs) {
                    if (fresh_item) {
                        I = item_of<S>(Q, t);
                        j = I.j0;
                        fresh_item = false;
                    }
                    const uint32_t o = owned % S::kOwns, s = it % kStages, b = it % S::kBufs;
                    if (mbar_test(full + 8 * s, it / kStages & 1) && (j > I.j0 || mbar_test(own_full + 8 * o, owned / S::kOwns & 1))) {
                        tc_fence_after();
                        // (the slopes that were here have been read: products are carried out in the order of their issue)
                        const uint32_t d = tmem + b * S::kScoreCols;
                        const uint64_t mine = smem_desc(owns + o * S::kOwnBytes, 16, 1024), rows = smem_desc(stages + s * S::kStage, 16, 1024);
                        constexpr uint64_t kMine = S::kOwnPart / 16, kPart = S::kOtherPart / 16;   // so many 16 bytes on
#pragma unroll
                        for (int k = 0; k < C / 16; ++k) {
                            const uint64_t m = mine + (k / 4) * (kParts * kMine) + (k % 4) * 2, r = rows + (k / 4) * (kParts * kPart) + (k % 4) * 2;
                            if (P == 6) {
                                tc_mma_f16<1>(d, m, r, score_desc2, k > 0);   // hi hi, and hi mid among the lo sums behind them
                                tc_mma_f16<1>(d + TN, m, r + 2 * kPart, score_desc, true);
                                tc_mma_f16<1>(d + TN, m + 2 * kMine, r, score_desc, true);
                                tc_mma_f16<1>(d + TN, m + kMine, r + kPart, score_desc, true);
                                tc_mma_f16<1>(d + TN, m + kMine, r, score_desc, true);
                            } else {
                                tc_mma_f16<1>(d, m, r, score_desc, k > 0);
                            }
                        }
                        tc_commit<1>(scored + 8 * b);
                        const bool end = j + 1 == I.j1;
                        ends = (ends & ~(1u << b)) | static_cast<uint32_t>(end) << b;
                        ++it;
                        ++j;
                        if (end) {
                            tc_commit<1>(own_empty + 8 * o);
                            ++owned;
                            t += step;
                            fresh_item = true;
                        }
                        done_something = true;
                    }
                }
                if (back_it < it && (it - back_it == S::kBufs || t >= items || !done_something)) {
                    const uint32_t b = back_it % S::kBufs, s = back_it % kStages;
                    const bool fresh = place % S::kChunk == 0;
                    if (mbar_test(sloped + 8 * b, back_it / S::kBufs & 1) && (!fresh || mbar_test(emptied, (chunks & 1) ^ 1))) {
                        tc_fence_after();
                        const uint32_t g = tmem + b * S::kScoreCols, d = tmem + S::kD;
                        const uint64_t rows = smem_desc(stages + s * S::kStage, C == 64 ? TN * 128 : kParts * TN * 128, 1024);
                        constexpr uint64_t kPart = S::kOtherPart / 16;
#pragma unroll
                        for (int k = 0; k < TN / 16; ++k) {
                            const bool more = !fresh || k > 0;
                            const uint32_t a = g + (P == 6 ? k / 2 * 32 + k % 2 * 8 : k / 4 * 64 + k % 4 * 8);   // see the slopes' places below
                            const uint64_t r = rows + k * (2048 / 16);
                            // The parts lie side by side as D's sums do.  Fetching A bounds a product of few columns: 64 take about as long as
                            // 128, 57 cycles with A in shared memory. (Three accumulators of scores and two of D, 12 and 20 products a tile of
                            // 64 and not 20 and 12: 555 against 477 us for dx at 2048 x 64 x 200000; three of both do not fit.)
                            if (S::kWide) {
                                tc_mma_f16_tmem(d, a, r, sum_desc3, more);
                                tc_mma_f16_tmem(d + C, a + TN, r, sum_desc2, true);
                                tc_mma_f16_tmem(d + 2 * C, a + 16, r, sum_desc, true);
                                continue;
                            }
                            tc_mma_f16_tmem(d, a, r, sum_desc, more);
                            if (P == 6) {
                                tc_mma_f16_tmem(d + C, a, r + kPart, sum_desc, more);
                                tc_mma_f16_tmem(d + C, a, r + 2 * kPart, sum_desc, true);
                                tc_mma_f16_tmem(d + C, a + 16, r, sum_desc, true);
                                tc_mma_f16_tmem(d + C, a + TN, r + kPart, sum_desc, true);
                                tc_mma_f16_tmem(d + C, a + TN, r, sum_desc, true);
                            }
                        }
                        tc_commit<1>(empty + 8 * s);
                        const bool end = ends >> b & 1;
                        if (end || place % S::kChunk == S::kChunk - 1) {
                            tc_commit<1>(summed);
                            ++chunks;
                        }
                        place = end ? 0 : place + 1;
                        ++back_it;
                        done_something = true;
                    }
                }
                if (done_something) {
                    spins = 0;
                } else if ((++spins & 63) == 0) {   // bounded as mbar_wait is
                    if (dead) break;
                    if (spins == 64)
                        since = now_ns();
                    else if (now_ns() - since > 2000000000ull) {
                        dead = 1;
                        break;
                    }
                }
            }
            if (dead) {   // products in flight finish before the block leaves
                volatile int none = 0;
                tc_commit<1>(drain);
                mbar_wait(drain, 0, &none);
            }
        }
    } else if (warp < 18) {
        const int group = (warp - 2) >> 2, pair = group >> 1, half = group & 1, id = 1 + group;
        constexpr int kHalf = TN / 2, kOnce = P == 6 ? 16 : 32;   // scores of a group, and those it reads at a time
        const int rowl = (warp & 3) * 32 + lane;
        uint32_t it = 0;
        bool ok = true;
        for (int t = first; ok && t < items; t += step) {
            const Item I = item_of<S>(Q, t);
            const int row = I.own0 + rowl;
            float4 mine = make_float4(0.0f, 0.0f, __int_as_float(-1), 0.0f);
            if (I.tokens && row < Q.n) mine = Q.tokens[row];
            const int target = __float_as_int(mine.z);
            for (int j = I.j0; ok && j < I.j1; ++j, ++it) {
                if ((it & 1) != static_cast<uint32_t>(pair)) continue;
                const uint32_t s = it % kStages, buf = it % S::kBufs;
                const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + buf * S::kScoreCols + half * kHalf;
                if (!(ok = all_of(id, 128, mbar_wait(scored + 8 * buf, it / S::kBufs & 1, &dead)))) break;
                tc_fence_after();
                const uint32_t numbers = stages + s * S::kStage + S::kOtherBytes + half * kHalf * 16;
                const int c0 = j * TN + half * kHalf;
                const int left = I.tokens ? Q.v - c0 : kHalf;   // columns that are rows of the table
                if (!I.tokens && !(ok = all_of(id, 128, mbar_wait(full + 8 * s, it / kStages & 1, &dead)))) break;   // the numbers
                uint32_t last[kParts > 1 ? kHalf / 2 : 1];   // the third part, whose place is free last
#pragma unroll
                for (int q = 0; q < kHalf / kOnce; ++q) {
                    float z[kOnce];
                    if constexpr (P == 6) {
                        float x[kOnce];
                        tmem_load16(lanes + q * 16, lanes + TN + q * 16, z, x);
#pragma unroll
                        for (int e = 0; e < kOnce; ++e) z[e] += x[e];
                    } else {
                        tmem_load32(lanes + q * 32, z);
                    }
                    if (I.tokens) {
#pragma unroll
                        for (int e = 0; e < kOnce; ++e) z[e] = exp2_fast(fmaf(z[e], kLog2e, -mine.x));
                        const int hit = target - (c0 + q * kOnce);
                        if (static_cast<uint32_t>(hit) < static_cast<uint32_t>(kOnce))
#pragma unroll
                            for (int e = 0; e < kOnce; ++e)
                                if (e == hit) z[e] -= 1.0f;
#pragma unroll
                        for (int e = 0; e < kOnce; ++e) z[e] = target >= 0 ? z[e] * mine.y : 0.0f;
                        if (q * kOnce + kOnce > left)
#pragma unroll
                            for (int e = 0; e < kOnce; ++e)
                                if (q * kOnce + e >= left) z[e] = 0.0f;
                    } else {
#pragma unroll
                        for (int e = 0; e < kOnce; ++e) {
                            const uint4 u = lds128(numbers + (q * kOnce + e) * 16);
                            const int other = static_cast<int>(u.z);
                            float p = exp2_fast(fmaf(z[e], kLog2e, -__uint_as_float(u.x)));
                            if (other == row) p -= 1.0f;
                            z[e] = other >= 0 ? p * __uint_as_float(u.y) : 0.0f;
                        }
                    }
                    // A K step's 16 slopes are 8 columns a part, where this group's scores were that it has read: the first part
                    // from its first score's column on, the second among its lo sums, the third behind the first.
#pragma unroll
                    for (int h = 0; h < kOnce / 16; ++h) {
                        uint32_t r[8];
#pragma unroll
                        for (int p = 0; p < kParts; ++p) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                float &a = z[h * 16 + 2 * e], &b = z[h * 16 + 2 * e + 1];
                                r[e] = bf16_pair(a, b);
                                if (p + 1 < kParts) {
                                    const float2 f = pair_floats(r[e]);
                                    a -= f.x, b -= f.y;
                                }
                                if (p == 2) last[kParts > 1 ? q * 8 + e : 0] = r[e];
                            }
                            if (p < 2) tmem_store8(lanes + (p == 1 ? TN : 0) + (q * kOnce / 16 + h) * 8, r);
                        }
                    }
                }
                if (kParts > 1)
#pragma unroll
                    for (int q = 0; q < (kParts > 1 ? kHalf / 16 : 0); ++q) {
                        uint32_t r[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) r[e] = last[kParts > 1 ? q * 8 + e : 0];
                        tmem_store8(lanes + 16 + q * 8, r);
                    }
                tmem_store_done();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(sloped + 8 * buf);
            }
        }
    } else {
        const int group = (warp - 18) >> 2, id = 5 + group;
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + S::kD + group * 64;
        uint32_t chunks = 0;
        bool ok = true;
        for (int t = first; ok && t < items; t += step) {
            const Item I = item_of<S>(Q, t);
            float sum[2][32];
#pragma unroll
            for (int q = 0; q < 64; ++q) sum[q / 32][q % 32] = 0.0f;
#pragma unroll 1
            for (int j = I.j0; j < I.j1; j += min(S::kChunk, I.j1 - j), ++chunks) {
                if (!(ok = all_of(id, 128, mbar_wait(summed, chunks & 1, &dead)))) break;
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v[16];
                    if constexpr (P == 6) {
                        float x[16];
                        tmem_load16(lanes + q * 16, lanes + C + q * 16, v, x);
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] += x[e];
                        if constexpr (S::kWide) {
                            tmem_load16(lanes + 2 * C + q * 16, x);
#pragma unroll
                            for (int e = 0; e < 16; ++e) v[e] += x[e];
                        }
                    } else {
                        tmem_load16(lanes + q * 16, v);
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) sum[q / 2][q % 2 * 16 + e] += v[e];
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(emptied);
            }
            if (!ok) break;
            const int row = I.own0 + (warp & 3) * 32 + lane;
            if (row >= (I.tokens ? Q.n : Q.v)) continue;
            const int64_t rows = I.tokens ? Q.n : Q.v;
            const bool slabs = (I.tokens ? Q.dx_splits : Q.dw_splits) > 1;
            if (kParts == 1) {
                const float unit = *Q.unit;
#pragma unroll
                for (int q = 0; q < 64; ++q) sum[q / 32][q % 32] *= unit;
            }
            void* out = I.tokens ? Q.dx : Q.dw;
            const int64_t at = ((slabs ? I.split * rows : 0) + row) * Q.c + group * 64;
            const int left = Q.c - group * 64;
            const bool narrow = !slabs && Q.out_bf16;
            if (left >= 64 && (reinterpret_cast<uintptr_t>(out) + at * (narrow ? 2 : 4)) % 16 == 0) {
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = sum[q / 4][q % 4 * 8 + e];
                    if (narrow)
                        Pack<bf16, 8>::put(static_cast<bf16*>(out) + at + q * 8, v);
                    else
                        Pack<float, 8>::put(static_cast<float*>(out) + at + q * 8, v);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 64; ++e) {
                    if (e >= left) break;
                    if (narrow)
                        static_cast<bf16*>(out)[at + e] = __float2bfloat16_rn(sum[e / 32][e % 32]);
                    else
                        static_cast<float*>(out)[at + e] = sum[e / 32][e % 32];
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (dead && threadIdx.x == 0) set_error(Q.d_err, SPARSE_ERR_INTERNAL);
    if (warp == 1) tmem_free<1>(tmem, 512);
}

int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a; }

// Parts that the other rows are cut into, for tokens and for the table's rows: those that take least, in 64ths of a tile's time. An item's
// own rows, its first scores and its sums take about 3 tiles' time, a part's sums are written and read again.
void back_splits(int64_t n, int64_t v, int64_t tile, int& tokens, int& rows)
{
    const int64_t units = kSms, own_n = up(n, kOwn), own_v = up(v, kOwn), tiles_v = up(v, tile), tiles_n = up(n, tile);
    int64_t least = INT64_MAX;
    tokens = rows = 1;
    for (int64_t a = 1; a <= 64 && a <= tiles_v; ++a)
        for (int64_t b = 1; b <= 8 && b <= tiles_n; ++b) {
            const int64_t la = up(tiles_v, a) + 3, lb = up(tiles_n, b) + 3, items_a = own_n * a, items_b = own_v * b;
            const int64_t ra = items_a % units, rb = items_b % units;
            const int64_t whole = items_a / units * la + items_b / units * lb;   // rounds that fill the GPU
            const int64_t end = ra + rb <= units ? std::max(ra > 0 ? la : 0, rb > 0 ? lb : 0) : la + lb;
            const int64_t joined = (a > 1 ? a * own_n : 0) + (b > 1 ? b * own_v : 0);
            const int64_t cost = 64 * (whole + end) + 16 * joined / units;
            if (cost < least) least = cost, tokens = static_cast<int>(a), rows = static_cast<int>(b);
        }
}

template <class S>
cudaError_t run_back(const Maps& maps, const BackArgs& Q, cudaStream_t s)
{
    auto* kernel = k_loss_back<S>;
    const cudaError_t ready = allow_smem(kernel, S::kSmem, S::kSmem);
    if (ready != cudaSuccess) return ready;
    const int64_t grid = std::min<int64_t>(num_sms(), Q.dx_items + Q.dw_items);
    SO_PROFILE("vocab_back", s);
    return launch_smem(kernel, dim3(static_cast<unsigned>(grid)), dim3(S::kThreads), S::kSmem, s, maps, Q);
}

}  // namespace

BackPlan back_plan(bool f32, int64_t n, int64_t c, int64_t v)
{
    BackPlan B{};
    const int64_t tile = f32 ? 64 : 128;
    back_splits(n, v, tile, B.dx_splits, B.dw_splits);
    B.tokens = up(n, 128) * 128;
    return B;
}

cudaError_t loss_back(const CUtensorMap& x, const CUtensorMap& w, bool f32, BackArgs Q, cudaStream_t s)
{
    const Maps maps{x, w};
    Q.dx_items = Q.dx != nullptr ? static_cast<int32_t>(up(Q.n, kOwn)) * Q.dx_splits : 0;
    Q.dw_items = Q.dw != nullptr ? static_cast<int32_t>(up(Q.v, kOwn)) * Q.dw_splits : 0;
    if (f32) return Q.c <= 64 ? run_back<BackShape<6, 64>>(maps, Q, s) : run_back<BackShape<6, 128>>(maps, Q, s);
    return Q.c <= 64 ? run_back<BackShape<1, 64>>(maps, Q, s) : run_back<BackShape<1, 128>>(maps, Q, s);
}

}  // namespace so
