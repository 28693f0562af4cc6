// vocab_loss.cu -- softmax cross entropy of n tokens against all rows of a table, and
// its gradient, without the n x v scores.
//
//   z = x W^T, lse = log sum exp z, loss = lse - z[target]
//   G = dloss (exp(z - lse) - [target]), dx = G W, dW = G^T x
//
// Forward, a product whose epilogue keeps a running maximum and sum of exponentials for every token (a lane
// has a token, so nothing is exchanged) over the tiles of an item: some hundred of the table's rows
// for 256 tokens; a second launch joins the items.  Scores stay in tensor memory and registers.
// Backward, the scores are made again for a piece of the table at a time, and their slopes G kept as
// bf16 (fp32 operands: three bf16 parts): G and the piece's rows make the piece's share of dx, which is summed
// in fp32 over the pieces, G and x the piece's rows of dW, complete.  A piece is as wide as kSlopeBytes allows.
#include "product.cuh"
#include "few_rows.cuh"
#include "vocab_back.cuh"

namespace so {

namespace {

// Groups of warps of a score's tile, each with running sums of its own.
constexpr int score_groups(bool f32)
{
    return f32 ? ProductShape<kScore, false, false, 2, 6, false>::kWarpGroups : ProductShape<kScore, false, false, 2, 1, true>::kWarpGroups;
}
constexpr size_t kSlopeBytes = size_t(256) << 20;   // G of one piece, all parts

int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a; }

struct Grid {
    int width, run, items;   // columns of a tile, tiles of an item, items in a row of them
    bool pair;
};

// Tiles of the scores: the width and run whose rounds over the GPU take least, in cycles.  A tile takes its stages (2 cycles a column and
// product, or the boxes' way from L2), 1500 at least, which is the epilogue's; an item 2000 more, for its tokens' numbers and its running sums, which the
// second launch reads at 3400 bytes a cycle.  (A run of one tile: 1.44 against 1.10 ms at 2048 x 64 x 1M fp32, and 94 us of that launch.)
Grid score_grid(int64_t n, int64_t c, int64_t v, int parts, bool runs)
{
    Grid g{};
    g.pair = n > 128;
    const int most = parts == 3 ? 128 : 256, products = parts == 3 ? 6 : 1;
    const int64_t units = kSms / (g.pair ? 2 : 1), m_tiles = up(n, g.pair ? 256 : 128), chunks = up(c, kPK);
    int64_t best = INT64_MAX;
    for (int w = most; w >= most / 2; w -= 32) {
        const int64_t stage = std::max<int64_t>(2 * w * products, parts * (kPM + w / (g.pair ? 2 : 1)) * 128 / 80);
        const int64_t tile = std::max<int64_t>(chunks * stage, 1500);
        for (int run = runs ? 32 : 1; run >= 1; run /= 2) {
            const int64_t items = up(up(v, w), run);
            const int64_t cost = up(items * m_tiles, units) * (run * tile + 2000) + (runs ? items * n * 32 / 3400 : 0);
            if (cost < best) best = cost, g.width = w, g.run = run, g.items = static_cast<int>(items);
        }
    }
    return g;
}

// The items' sums of R tokens a block: 1024 / R threads a token have some of them each, and are joined in shared memory, a warp a
// token.  Few tokens have few to a block: 16 tokens against 100000 rows of 2048 bf16 take 71 us in all with 4 to a block, 77.5 with 32, and
// 82.6 with a block of 128 threads each, small enough to be on an SM beside a block of the scores.
template <int R>
__global__ void __launch_bounds__(1024) k_loss_join(const float2* __restrict__ part, int slots, const float* __restrict__ hit,
                                                        const int64_t* __restrict__ target, int64_t n, float* __restrict__ loss,
                                                        float* __restrict__ lse)
{
    pdl_wait();
    constexpr int kEach = 1024 / R;              // threads of a token: 32 or more
    __shared__ float2 sums[R][kEach + 1];
    const int token = threadIdx.x % R, mine = threadIdx.x / R;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * R + token;
    float top = -INFINITY, sum = 0.0f;
    auto add = [&](float t, float u) {
        const float high = fmaxf(top, t), base = high == -INFINITY ? 0.0f : high;
        sum = sum * exp2_fast((top - base) * kLog2e) + u * exp2_fast((t - base) * kLog2e);
        top = high;
    };
    if (row < n)
#pragma unroll 4
        for (int s = mine; s < slots; s += kEach) {
            const float2 q = part[static_cast<int64_t>(s) * n + row];
            add(q.x, q.y);
        }
    sums[token][mine] = make_float2(top, sum);
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp >= R) return;
    top = -INFINITY, sum = 0.0f;
    for (int i = lane; i < kEach; i += 32) add(sums[warp][i].x, sums[warp][i].y);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float t = __shfl_xor_sync(kFull, top, d), u = __shfl_xor_sync(kFull, sum, d);
        add(t, u);
    }
    const int64_t to = static_cast<int64_t>(blockIdx.x) * R + warp;
    if (lane == 0 && to < n) {
        const float l = top + logf(sum);
        lse[to] = l;
        loss[to] = target[to] < 0 ? 0.0f : l - hit[to];
    }
}

struct Layout {
    int parts;
    bool pack_x, pack_w;
    int64_t ldx, ldw;        // of the packed arrays, or c
    Grid score, slope;
    int64_t piece, pieces, ldg;
    int dx_splits, dw_splits;
    bool dx_slabs, dw_slabs;
    bool narrow;             // the gradient in one launch (vocab_back.cu)
    bool few;                // few fp32 tokens: see few_rows.cuh
    int slots;               // running sums of a token
    BackPlan back;
    size_t x, w, part, hit, g, dx, dw, tokens, unit, total;
};

Layout layout(bool f32, int64_t n, int64_t c, int64_t v, bool grad, bool x_aligned, bool w_aligned)
{
    Layout L{};
    L.parts = f32 ? 3 : 1;
    L.pack_x = f32 || c % 8 != 0 || !x_aligned || grad;   // the gradient reads zeros for a token that does not count: 0 times NaN is NaN
    L.pack_w = f32 || c % 8 != 0 || !w_aligned;
    L.ldx = L.pack_x ? packed_ld(c) : c;
    L.ldw = L.pack_w ? packed_ld(c) : c;
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t p = at;
        at += (static_cast<size_t>(bytes) + 255) / 256 * 256;
        return p;
    };
    if (f32 && !grad && n <= kFewTokens) {
        L.few = true;
        L.slots = few_dot_slots(v);
        L.part = take(static_cast<int64_t>(sizeof(float2)) * L.slots * n);
        L.hit = take(4 * n);
        L.total = std::max<size_t>(at, 256);
        return L;
    }
    if (f32 && grad && n <= kFewGrad) {
        L.few = true;
        L.g = take(4 * n * v);
        L.dx_splits = few_sums_splits(n, c, v, 1);
        L.dx = take(4 * L.dx_splits * n * c);
        L.total = at;
        return L;
    }
    if (L.pack_x) L.x = take(2 * L.parts * n * L.ldx);
    if (L.pack_w) L.w = take(2 * L.parts * v * L.ldw);
    if (!grad) {
        L.score = score_grid(n, c, v, L.parts, true);
        L.slots = L.score.items * score_groups(f32);
        L.part = take(static_cast<int64_t>(sizeof(float2)) * L.slots * n);
        L.hit = take(static_cast<int64_t>(sizeof(float)) * n);
    } else if (c <= kBackCols) {
        L.narrow = true;
        L.back = back_plan(f32, n, c, v);
        L.dx_splits = L.back.dx_splits;
        L.dw_splits = L.back.dw_splits;
        L.dx_slabs = L.dx_splits > 1;
        L.dw_slabs = L.dw_splits > 1;
        if (!f32) L.unit = take(4);
        L.tokens = take(static_cast<int64_t>(sizeof(float4)) * L.back.tokens);
        if (L.dx_slabs) L.dx = take(4 * L.dx_splits * n * c);
        if (L.dw_slabs) L.dw = take(4 * L.dw_splits * v * c);
    } else {
        const int64_t most = std::max<int64_t>(256, static_cast<int64_t>(kSlopeBytes) / (2 * L.parts * n) / 256 * 256);
        L.pieces = up(v, most);
        L.piece = up(up(v, L.pieces), 256) * 256;
        L.pieces = up(v, L.piece);
        L.ldg = std::min(L.piece, up(v, 16) * 16);   // rows of whole 32-byte accesses
        L.slope = score_grid(n, c, L.piece, L.parts, false);
        L.g = take(2 * L.parts * n * L.ldg);
        L.dx_splits = rows_splits(n, c, L.piece, 1, L.parts);
        L.dx_slabs = L.pieces > 1 || L.dx_splits > 1;
        if (!f32) L.unit = take(4);
        if (L.dx_slabs) L.dx = take(4 * L.dx_splits * n * c);
        L.dw_splits = weights_splits(n, c, L.piece, 1, L.parts);
        L.dw_slabs = L.dw_splits > 1;
        if (L.dw_slabs) L.dw = take(4 * L.dw_splits * L.piece * c);
    }
    L.total = std::max<size_t>(at, 256);
    return L;
}

template <int kForm, int P, bool kDrain>
cudaError_t run_scores(const char* name, bool pair, const ProductMaps& maps, ProductArgs Q, int64_t across, cudaStream_t s)
{
    Q.m_tiles = static_cast<int32_t>(up(Q.rows, pair ? 256 : 128));
    return pair ? run_product<ProductShape<kForm, false, false, 2, P, kDrain>>(name, maps, Q, across * Q.m_tiles, s)
                : run_product<ProductShape<kForm, false, false, 1, P, kDrain>>(name, maps, Q, across * Q.m_tiles, s);
}

// x and w as the products read them, for the gradient with the tokens' numbers.
cudaError_t prepare(const Layout& L, const VocabLoss& V, bool grad, uint8_t* ws, const void*& x, const void*& w, const TokenRows& tokens,
                    cudaStream_t s)
{
    x = L.pack_x ? ws + L.x : V.x;
    w = L.pack_w ? ws + L.w : V.w;
    if (!L.pack_x && !L.pack_w) return cudaSuccess;
    return pack(Pack1{V.x, reinterpret_cast<bf16*>(ws + L.x), L.pack_x ? V.n : 0, V.c, L.ldx, nullptr, 1, grad ? V.target : nullptr, V.v},
                Pack1{V.w, reinterpret_cast<bf16*>(ws + L.w), L.pack_w ? V.v : 0, V.c, L.ldw}, tokens, !V.f32, s);
}

bool aligned(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

size_t vocab_loss_ws_bytes(int f32, int64_t n, int64_t c, int64_t v, int grad, int is_aligned)
{
    return layout(f32, n, c, v, grad, is_aligned, is_aligned).total;
}

size_t vocab_loss_ws_bytes(const VocabLoss& V, int grad)
{
    return layout(V.f32, V.n, V.c, V.v, grad, aligned(V.x), aligned(V.w)).total;
}

static cudaError_t join_scores(const VocabLoss& V, const Layout& L, const float2* part, const float* hit, cudaStream_t s)
{
    SO_PROFILE("vocab_join", s);
    auto join = [&](auto* kernel, int rows) {
        return launch(kernel, dim3(static_cast<unsigned>(up(V.n, rows))), dim3(1024), s, part, L.slots, hit, V.target, V.n, V.loss, V.lse);
    };
    return V.n <= 4 * kSms ? join(k_loss_join<4>, 4) : join(k_loss_join<32>, 32);
}

cudaError_t vocab_loss(const VocabLoss& V, void* workspace, cudaStream_t s)
{
    if (tensor_encoder() == nullptr) return cudaErrorNotSupported;
    const Layout L = layout(V.f32, V.n, V.c, V.v, false, aligned(V.x), aligned(V.w));
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    if (L.few) {
        FewDots D{};
        D.x = static_cast<const float*>(V.x);
        D.w = static_cast<const float*>(V.w);
        D.n = V.n;
        D.m = V.v;
        D.k = V.c;
        D.groups = 1;
        D.target = V.target;
        D.d_err = V.d_err;
        D.part = reinterpret_cast<float2*>(ws + L.part);
        D.hit = reinterpret_cast<float*>(ws + L.hit);
        const cudaError_t e = few_dots(D, s);
        return e != cudaSuccess ? e : join_scores(V, L, D.part, D.hit, s);
    }
    const void *x, *w;
    cudaError_t e = prepare(L, V, false, ws, x, w, TokenRows{}, s);
    if (e != cudaSuccess) return e;
    ProductMaps maps;
    if (!Operand{x, V.n, V.c, L.ldx, 1, L.parts}.map(&maps.a) || !Operand{w, V.v, V.c, L.ldw, 1, L.parts}.map(&maps.b))
        return cudaErrorInvalidValue;
    ProductArgs Q{};
    Q.rows = static_cast<int32_t>(V.n);
    Q.m = Q.rows;
    Q.n = Q.v = static_cast<int32_t>(V.v);
    Q.k = static_cast<int32_t>(V.c);
    Q.width = L.score.width;
    Q.run = L.score.run;
    Q.n_tiles = static_cast<int32_t>(up(V.v, Q.width));
    Q.target = V.target;
    Q.part = reinterpret_cast<float2*>(ws + L.part);
    Q.hit = reinterpret_cast<float*>(ws + L.hit);
    Q.release = 1;
    Q.d_err = V.d_err;
    e = V.f32 ? run_scores<kScore, 6, false>("vocab_score", L.score.pair, maps, Q, L.score.items, s)
              : run_scores<kScore, 1, true>("vocab_score", L.score.pair, maps, Q, L.score.items, s);
    if (e != cudaSuccess) return e;
    return join_scores(V, L, Q.part, Q.hit, s);
}

// Rows of at most kBackCols columns.
static cudaError_t narrow_grad(const VocabLoss& V, const Layout& L, const void* x, const void* w, uint8_t* ws, cudaStream_t s)
{
    CUtensorMap mx, mw;
    if (!Operand{x, V.n, V.c, L.ldx, 1, L.parts}.map(&mx) || !Operand{w, V.v, V.c, L.ldw, 1, L.parts}.map(&mw))
        return cudaErrorInvalidValue;
    BackArgs Q{};
    Q.n = static_cast<int32_t>(V.n);
    Q.c = static_cast<int32_t>(V.c);
    Q.v = static_cast<int32_t>(V.v);
    Q.tokens = reinterpret_cast<const float4*>(ws + L.tokens);
    Q.dx = V.dx == nullptr ? nullptr : L.dx_slabs ? static_cast<void*>(ws + L.dx) : V.dx;
    Q.dw = V.dw == nullptr ? nullptr : L.dw_slabs ? static_cast<void*>(ws + L.dw) : V.dw;
    Q.dx_splits = L.dx_splits;
    Q.dw_splits = L.dw_splits;
    Q.out_bf16 = !V.f32;
    Q.unit = V.f32 ? nullptr : reinterpret_cast<const float*>(ws + L.unit);
    Q.release = (V.dx == nullptr || L.dx_slabs) && (V.dw == nullptr || L.dw_slabs);
    Q.d_err = V.d_err;
    const cudaError_t e = loss_back(mx, mw, V.f32, Q, s);
    Join dx{}, dw{};
    if (V.dx != nullptr && L.dx_slabs) dx = Join{reinterpret_cast<const float*>(ws + L.dx), L.dx_splits, V.n * V.c, V.n, V.c};
    if (V.dw != nullptr && L.dw_slabs) dw = Join{reinterpret_cast<const float*>(ws + L.dw), L.dw_splits, V.v * V.c, V.v, V.c};
    if (e != cudaSuccess || dx.rows + dw.rows == 0) return e;
    return dx.rows > 0 ? join_two(dx, V.dx, dw, V.dw, !V.f32, s) : join_slabs(dw, V.dw, !V.f32, s);
}

// Few fp32 tokens: the slopes in fp32, then the sums of the table's rows and the outer products, each a pass over the table.
static cudaError_t few_loss_grad(const VocabLoss& V, const Layout& L, uint8_t* ws, cudaStream_t s)
{
    float *g = reinterpret_cast<float*>(ws + L.g), *slabs = reinterpret_cast<float*>(ws + L.dx);
    FewDots D{};
    D.x = static_cast<const float*>(V.x);
    D.w = static_cast<const float*>(V.w);
    D.n = V.n;
    D.m = V.v;
    D.k = V.c;
    D.groups = 1;
    D.out = g;
    D.target = V.target;
    D.lse = V.lse;
    D.dloss = V.dloss;
    D.d_err = V.d_err;
    cudaError_t e = few_dots(D, s);
    if (e == cudaSuccess && V.dw != nullptr)
        e = few_outer(FewOuter{g, D.x, V.n, V.v, V.c, 1, nullptr, static_cast<float*>(V.dw), V.target, V.d_err}, s);
    if (e == cudaSuccess && V.dx != nullptr) {
        e = few_sums(FewSums{g, D.w, V.n, V.c, V.v, 1, nullptr, L.dx_splits, slabs, V.d_err}, s);
        if (e == cudaSuccess) e = join_slabs(Join{slabs, L.dx_splits, V.n * V.c, V.n, V.c}, V.dx, 0, s);
    }
    return e;
}

cudaError_t vocab_loss_grad(const VocabLoss& V, void* workspace, cudaStream_t s)
{
    if (tensor_encoder() == nullptr) return cudaErrorNotSupported;
    const Layout L = layout(V.f32, V.n, V.c, V.v, true, aligned(V.x), aligned(V.w));
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    if (L.few) return few_loss_grad(V, L, ws, s);
    const void *x, *w;
    TokenRows tokens{};
    if (L.narrow) {
        tokens = TokenRows{V.lse, V.dloss, V.target, static_cast<int>(V.n), static_cast<int>(L.back.tokens), static_cast<int>(V.v),
                           reinterpret_cast<float4*>(ws + L.tokens), V.f32 ? nullptr : reinterpret_cast<float*>(ws + L.unit), V.d_err};
    }
    cudaError_t e = prepare(L, V, true, ws, x, w, tokens, s);
    if (e == cudaSuccess && L.narrow) return narrow_grad(V, L, x, w, ws, s);
    const int64_t row = 2 * L.ldw;   // bytes of one part's row
    for (int64_t p = 0; p < L.pieces && e == cudaSuccess; ++p) {
        const int64_t v0 = p * L.piece, wide = std::min(L.piece, V.v - v0);
        ProductMaps maps;
        const Operand piece{static_cast<const uint8_t*>(w) + v0 * row, wide, V.c, L.ldw, 1, L.parts, V.v * L.ldw};
        if (!Operand{x, V.n, V.c, L.ldx, 1, L.parts}.map(&maps.a) || !piece.map(&maps.b)) return cudaErrorInvalidValue;
        ProductArgs Q{};
        Q.rows = static_cast<int32_t>(V.n);
        Q.m = Q.rows;
        Q.n = static_cast<int32_t>(wide);
        Q.v = static_cast<int32_t>(V.v);
        Q.v0 = static_cast<int32_t>(v0);
        Q.k = static_cast<int32_t>(V.c);
        Q.width = L.slope.width;
        Q.n_tiles = static_cast<int32_t>(up(wide, Q.width));
        Q.target = V.target;
        Q.lse = V.lse;
        Q.dloss = V.dloss;
        Q.slope = reinterpret_cast<bf16*>(ws + L.g);
        Q.slope_part = V.n * L.ldg;
        Q.unit = V.f32 ? nullptr : reinterpret_cast<float*>(ws + L.unit);
        Q.ld = static_cast<int32_t>(L.ldg);
        Q.release = 1;
        Q.d_err = V.d_err;
        e = V.f32 ? run_scores<kSlope, 6, false>("vocab_slope", L.slope.pair, maps, Q, Q.n_tiles, s)
                  : run_scores<kSlope, 1, false>("vocab_slope", L.slope.pair, maps, Q, Q.n_tiles, s);
        if (e == cudaSuccess && V.dx != nullptr) {
            RowsProduct R{};
            R.a = piece;
            R.b = Operand{ws + L.g, V.n, wide, L.ldg, 1, L.parts};
            R.a_mn = 1;
            R.rows = V.n;
            R.m = V.c;
            R.k = wide;
            R.groups = 1;
            R.splits = L.dx_splits;
            R.out = L.dx_slabs ? static_cast<void*>(ws + L.dx) : V.dx;
            R.out_bf16 = !L.dx_slabs && !V.f32;
            R.add = p > 0;
            R.release = L.dx_slabs;
            R.unit = Q.unit;
            R.d_err = V.d_err;
            e = rows_product(R, s);
        }
        if (e == cudaSuccess && V.dw != nullptr) {
            uint8_t* to = static_cast<uint8_t*>(V.dw) + v0 * V.c * (V.f32 ? 4 : 2);
            WeightsProduct R{};
            R.a = Operand{x, V.n, V.c, L.ldx, 1, L.parts};
            R.b = Operand{ws + L.g, V.n, wide, L.ldg, 1, L.parts};
            R.rows = V.n;
            R.m = V.c;
            R.n = wide;
            R.groups = 1;
            R.splits = L.dw_splits;
            R.out = L.dw_slabs ? static_cast<void*>(ws + L.dw) : to;
            R.out_bf16 = !L.dw_slabs && !V.f32;
            R.release = L.dw_slabs;
            R.unit = Q.unit;
            R.d_err = V.d_err;
            e = weights_product(R, s);
            if (e == cudaSuccess && L.dw_slabs)
                e = join_slabs(Join{reinterpret_cast<const float*>(ws + L.dw), L.dw_splits, wide * V.c, wide, V.c}, to, !V.f32, s);
        }
    }
    if (e == cudaSuccess && V.dx != nullptr && L.dx_slabs)
        e = join_slabs(Join{reinterpret_cast<const float*>(ws + L.dx), L.dx_splits, V.n * V.c, V.n, V.c}, V.dx, !V.f32, s);
    return e;
}

}  // namespace so
