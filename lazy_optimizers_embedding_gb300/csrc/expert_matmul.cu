// expert_matmul.cu -- the products of every expert's rows with its matrix, and the
// gradient of the matrices: which arrays are packed, where the workspace's parts lie.
#include "few_rows.cuh"

namespace so {

namespace {

bool aligned(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// An operand as the product reads it: as it lies, or packed into the workspace at `at`.
struct Placed {
    bool packed;
    int64_t ld;
    size_t bytes;
};
Placed place(bool f32, int64_t rows, int64_t cols, bool is_aligned)
{
    const bool packed = f32 || cols % 8 != 0 || !is_aligned;
    const int64_t ld = packed ? packed_ld(cols) : cols;
    return {packed, ld, packed ? (static_cast<size_t>(2 * (f32 ? 3 : 1) * rows * ld) + 255) / 256 * 256 : 0};
}

struct Layout {
    Placed p, q;             // rows and matrices; rows and their gradients
    bool few;                // few fp32 rows: see few_rows.cuh
    int splits;
    size_t q_at, slabs, total;
};

Layout product_layout(bool f32, int64_t n, int64_t a, int64_t b, int64_t experts, int transpose, bool x_aligned, bool w_aligned)
{
    Layout L{};
    const int64_t k = transpose ? b : a, m = transpose ? a : b;
    L.p = place(f32, n, k, x_aligned);
    L.q = place(f32, experts * a, b, w_aligned);
    if (f32 && few_rows(n, experts)) {
        L.few = true;
        L.splits = transpose ? 0 : few_sums_splits(n, m, k, experts);
        L.total = std::max<size_t>(256, sizeof(float) * L.splits * n * m);
        return L;
    }
    L.splits = rows_splits(n, m, k, experts, f32 ? 3 : 1);
    L.q_at = L.p.bytes;
    L.slabs = L.q_at + L.q.bytes;
    L.total = std::max<size_t>(256, L.slabs + (L.splits > 1 ? sizeof(float) * L.splits * n * m : 0));
    return L;
}

Layout grad_layout(bool f32, int64_t n, int64_t a, int64_t b, int64_t experts, bool x_aligned, bool dy_aligned)
{
    Layout L{};
    L.p = place(f32, n, a, x_aligned);
    L.q = place(f32, n, b, dy_aligned);
    if (f32 && few_rows(n, experts)) {
        L.few = true;
        L.total = 256;
        return L;
    }
    L.splits = weights_splits(n, b, a, experts, f32 ? 3 : 1);
    L.q_at = L.p.bytes;
    L.slabs = L.q_at + L.q.bytes;
    L.total = std::max<size_t>(256, L.slabs + (L.splits > 1 ? sizeof(float) * L.splits * experts * a * b : 0));
    return L;
}

// Packs what has to be (of q, matrices of `each` rows, those of groups with rows); p and q as the product reads them.
cudaError_t prepare(const Layout& L, bool f32, const void*& p, int64_t p_rows, int64_t p_cols, const void*& q, int64_t q_rows,
                    int64_t q_cols, const int64_t* offsets, int64_t each, uint8_t* ws, cudaStream_t s)
{
    const Pack1 first{p, reinterpret_cast<bf16*>(ws), L.p.packed ? p_rows : 0, p_cols, L.p.ld};
    const Pack1 second{q, reinterpret_cast<bf16*>(ws + L.q_at), L.q.packed ? q_rows : 0, q_cols, L.q.ld, offsets, each};
    if (L.p.packed) p = first.to;
    if (L.q.packed) q = second.to;
    return L.p.packed || L.q.packed ? pack(first, second, TokenRows{}, !f32, s) : cudaSuccess;
}

}  // namespace

size_t expert_matmul_ws_bytes(int f32, int64_t n, int64_t a, int64_t b, int64_t experts, int is_aligned)
{
    return std::max({product_layout(f32, n, a, b, experts, 0, is_aligned, is_aligned).total,
                     product_layout(f32, n, a, b, experts, 1, is_aligned, is_aligned).total,
                     grad_layout(f32, n, a, b, experts, is_aligned, is_aligned).total});
}

size_t expert_matmul_ws_bytes(const ExpertMatmul& M)
{
    return M.dy != nullptr ? grad_layout(M.f32, M.n, M.a, M.b, M.experts, aligned(M.x), aligned(M.dy)).total
                           : product_layout(M.f32, M.n, M.a, M.b, M.experts, M.transpose, aligned(M.x), aligned(M.w)).total;
}

cudaError_t expert_matmul(const ExpertMatmul& M, void* workspace, cudaStream_t s)
{
    if (tensor_encoder() == nullptr) return cudaErrorNotSupported;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const Layout L = product_layout(M.f32, M.n, M.a, M.b, M.experts, M.transpose, aligned(M.x), aligned(M.w));
    const int64_t k = M.transpose ? M.b : M.a, m = M.transpose ? M.a : M.b;
    const int parts = M.f32 ? 3 : 1;
    if (L.few && M.transpose) {
        FewDots D{};
        D.x = static_cast<const float*>(M.x);
        D.w = static_cast<const float*>(M.w);
        D.n = M.n;
        D.m = m;
        D.k = k;
        D.groups = static_cast<int>(M.experts);
        D.offsets = M.offsets;
        D.out = static_cast<float*>(M.out);
        D.d_err = M.d_err;
        return few_dots(D, s);
    }
    if (L.few) {
        float* slabs = reinterpret_cast<float*>(ws);
        const cudaError_t e = few_sums(FewSums{static_cast<const float*>(M.x), static_cast<const float*>(M.w), M.n, m, k,
                                               static_cast<int>(M.experts), M.offsets, L.splits, slabs, M.d_err}, s);
        if (e != cudaSuccess) return e;
        return join_slabs(Join{slabs, L.splits, M.n * m, M.n, m, M.offsets + M.experts}, M.out, !M.f32, s);
    }
    const void *x = M.x, *w = M.w;
    cudaError_t e = prepare(L, M.f32, x, M.n, k, w, M.experts * M.a, M.b, M.offsets, M.a, ws, s);
    if (e != cudaSuccess) return e;
    RowsProduct R{};
    R.a = Operand{w, M.a, M.b, L.q.ld, M.experts, parts};
    R.b = Operand{x, M.n, k, L.p.ld, 1, parts};
    R.a_mn = !M.transpose;
    R.rows = M.n;
    R.m = m;
    R.k = k;
    R.groups = static_cast<int>(M.experts);
    R.offsets = M.offsets;
    R.splits = L.splits;
    const bool slabs = L.splits > 1;
    R.out = slabs ? static_cast<void*>(ws + L.slabs) : M.out;
    R.out_bf16 = !slabs && !M.f32;
    R.clear = !slabs;
    R.release = slabs;
    R.d_err = M.d_err;
    e = rows_product(R, s);
    if (e != cudaSuccess || !slabs) return e;
    return join_slabs(Join{reinterpret_cast<const float*>(ws + L.slabs), L.splits, M.n * m, M.n, m, M.offsets + M.experts}, M.out,
                      !M.f32, s);
}

cudaError_t expert_matmul_grad(const ExpertMatmul& M, void* workspace, cudaStream_t s)
{
    if (tensor_encoder() == nullptr) return cudaErrorNotSupported;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const Layout L = grad_layout(M.f32, M.n, M.a, M.b, M.experts, aligned(M.x), aligned(M.dy));
    const int parts = M.f32 ? 3 : 1;
    if (L.few)
        return few_outer(FewOuter{static_cast<const float*>(M.x), static_cast<const float*>(M.dy), M.n, M.a, M.b,
                                  static_cast<int>(M.experts), M.offsets, static_cast<float*>(M.out), nullptr, M.d_err}, s);
    const void *x = M.x, *dy = M.dy;
    cudaError_t e = prepare(L, M.f32, x, M.n, M.a, dy, M.n, M.b, nullptr, 1, ws, s);
    if (e != cudaSuccess) return e;
    WeightsProduct R{};
    R.a = Operand{dy, M.n, M.b, L.q.ld, 1, parts};
    R.b = Operand{x, M.n, M.a, L.p.ld, 1, parts};
    R.rows = M.n;
    R.m = M.b;
    R.n = M.a;
    R.groups = static_cast<int>(M.experts);
    R.offsets = M.offsets;
    R.splits = L.splits;
    const bool slabs = L.splits > 1;
    R.out = slabs ? static_cast<void*>(ws + L.slabs) : M.out;
    R.out_bf16 = !slabs && M.out_bf16;
    R.release = slabs;
    R.d_err = M.d_err;
    e = weights_product(R, s);
    if (e != cudaSuccess || !slabs) return e;
    const int64_t rows = M.experts * M.a;
    return join_slabs(Join{reinterpret_cast<const float*>(ws + L.slabs), L.splits, rows * M.b, rows, M.b}, M.out, M.out_bf16, s);
}

}  // namespace so
