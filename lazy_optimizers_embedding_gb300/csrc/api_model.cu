// api_model.cu -- the extern "C" entry points of the operators around the table
// step (declared in include/sparseopt.h): argument validation, workspace
// carving and the choice of 16-byte accesses.  No host synchronisation.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "common.cuh"

namespace {

using namespace so;

bool ws_ok(const void* ws, size_t have, size_t need)
{
    return ws != nullptr && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0 && have >= need;
}

bool valid_type(sparse_dtype_t t) { return t == SPARSE_F32 || t == SPARSE_BF16; }

bool is_bf16(sparse_dtype_t t) { return t == SPARSE_BF16; }

// An eps as fp32: one above 0 stays there (a row without spread has xhat = 0 with any but 0), a large one finite.
float small_eps(double eps)
{
    return eps > 0.0 ? static_cast<float>(std::clamp(eps, static_cast<double>(FLT_TRUE_MIN), static_cast<double>(FLT_MAX))) : 0.0f;
}

sparse_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? SPARSE_OK : SPARSE_ERR_CUDA; }

// n rows of c values, with n * c within int64 (and far from its end).
bool valid_rows(int64_t n, int64_t c) { return n >= 0 && c >= 1 && (n == 0 || c <= (INT64_MAX >> 4) / n); }

// Layer norm's rows: x [r, c], n of them looked up, or the first n without idx.
bool valid_norm(const void* x, sparse_dtype_t x_type, int64_t r, int64_t c, const int64_t* idx, int64_t n,
                sparse_dtype_t y_type, const int32_t* d_err)
{
    return valid_type(x_type) && valid_type(y_type) && !(is_bf16(x_type) && !is_bf16(y_type)) && valid_rows(r, c) &&
           valid_rows(n, c) && c <= INT32_MAX && (idx != nullptr || n <= r) && (n == 0 || x != nullptr) &&
           d_err != nullptr;
}

// Values of an access to rows of c values in all these arrays: those of 16 bytes (of two accesses to an fp32
// array beside a bf16 one), two, or 0 for single ones.
int access(int64_t c, bool any_bf16, const void* a, bool a_bf16, const void* b, bool b_bf16, const void* d, bool d_bf16)
{
    auto fits = [&](const void* p, bool bf16, int64_t v) {
        return reinterpret_cast<uintptr_t>(p) % std::min<uintptr_t>(16, static_cast<uintptr_t>(v * (bf16 ? 2 : 4))) == 0;
    };
    for (int v : {any_bf16 ? 8 : 4, 2})
        if (c % v == 0 && fits(a, a_bf16, v) && fits(b, b_bf16, v) && fits(d, d_bf16, v)) return v;
    return 0;
}

bool valid_expert(sparse_dtype_t type, int64_t n, int64_t k, int64_t c, const int32_t* d_err)
{
    return valid_type(type) && n >= 0 && k >= 1 && (n == 0 || k <= INT32_MAX / n) && valid_rows(n * k, c) &&
           c <= kMaxExpertCols && d_err != nullptr;
}

bool valid_route(sparse_dtype_t type, int64_t n, int64_t experts, int64_t k, const int32_t* d_err)
{
    return valid_type(type) && n >= 0 && experts >= 1 && experts <= kMaxExperts && k >= 1 && k <= experts && k <= 32 &&
           valid_rows(n, experts) && d_err != nullptr;
}

// Sizes that the tensor copies can address, and whose tiles (64 x 128 scores at least) are fewer than 2^31.
constexpr int64_t kMaxRows = INT32_MAX - 1024;   // 32-bit rows, a tile past the last included
constexpr int64_t kMaxCols = int64_t(1) << 20, kMaxValues = int64_t(1) << 37, kMaxScores = int64_t(1) << 43;

bool valid_matmul(sparse_dtype_t type, int64_t n, int64_t a, int64_t b, int64_t experts)
{
    return valid_type(type) && n >= 0 && n <= kMaxRows && a >= 1 && a <= kMaxCols && b >= 1 && b <= kMaxCols &&
           experts >= 1 && experts <= kMaxExperts && n <= kMaxValues / std::max(a, b) && experts * a <= kMaxValues / b;
}

bool valid_loss(sparse_dtype_t type, int64_t n, int64_t c, int64_t v)
{
    return valid_type(type) && n >= 0 && n <= (1 << 30) && c >= 1 && c <= kMaxCols && v >= 1 && v <= (1 << 30) &&
           n <= kMaxValues / c && v <= kMaxValues / c && n <= kMaxScores / v;
}

// Newton-Schulz keeps X, A = X X^T and B = b A + c A^2, with and without a on its
// diagonal, as f16 values times 2^14: their singular values have to stay below
// 65504 / 2^14 with 2 % to spare.  Bounded step by step, X's from [0, 1] on (all that a
// matrix of Frobenius norm at most 1 can have): with l = x^2 at most h^2, the largest
// of |b l + c l^2|, |a + b l + c l^2| and |x (a + b l + c l^2)| is at an end of [0, h]
// or where a derivative is 0.
constexpr double kMaxNs = 3.9;

bool valid_ns(const sparse_ns_config_t& c)
{
    if (!std::isfinite(c.a) || !std::isfinite(c.b) || !std::isfinite(c.c) || !(c.eps >= 0.0) || !std::isfinite(c.eps) ||
        c.steps < 1 || c.steps > 64 || (c.products != 1 && c.products != 3))
        return false;
    // l of the extrema of b l + c l^2, and of x (a + b x^2 + c x^4); the ends
    double at[5] = {0.0, 0.0, 0.0, 0.0, 0.0};   // [4]: the end 0
    if (c.c != 0.0) {
        at[0] = -c.b / (2.0 * c.c);
        const double d = 9.0 * c.b * c.b - 20.0 * c.a * c.c;
        if (d >= 0.0) {
            at[1] = (-3.0 * c.b + std::sqrt(d)) / (10.0 * c.c);
            at[2] = (-3.0 * c.b - std::sqrt(d)) / (10.0 * c.c);
        }
    } else if (c.b != 0.0) {
        at[1] = -c.a / (3.0 * c.b);
    }
    double h = 1.0;
    for (int s = 0; s < c.steps; ++s) {
        const double top = h * h;
        double next = 0.0;
        at[3] = top;
        for (double l : at) {
            if (!(l >= 0.0 && l <= top)) continue;
            const double p = c.b * l + c.c * l * l, x = std::sqrt(l) * (c.a + p);
            if (!(std::fabs(p) <= kMaxNs && std::fabs(c.a + p) <= kMaxNs)) return false;
            next = std::fmax(next, std::fabs(x));
        }
        if (!(top <= kMaxNs && next <= kMaxNs)) return false;
        h = next;
    }
    return true;
}

// A batch of r x c matrices whose sizes the tensor copies can address.
bool valid_batch(int64_t batch, int64_t r, int64_t c)
{
    return batch >= 0 && batch <= (1 << 24) && r >= 1 && c >= 1 && r <= (1 << 20) && c <= (1 << 20) &&
           (batch == 0 || r * c <= (int64_t(1) << 36) / batch);
}

so::MuonParams muon_params(int64_t batch, int64_t r, int64_t c, const sparse_ns_config_t& ns, int32_t* d_err)
{
    so::MuonParams M{};
    M.batch = batch;
    M.r = r;
    M.cols = c;
    M.a = static_cast<float>(ns.a);
    M.b = static_cast<float>(ns.b);
    M.c = static_cast<float>(ns.c);
    M.eps = small_eps(ns.eps);
    M.eps_raised = small_eps(ns.eps * 0x1p100);
    M.steps = ns.steps;
    M.products = ns.products;
    M.d_err = d_err;
    return M;
}

}  // namespace

extern "C" {

size_t sparse_layer_norm_workspace_size(int64_t n, int64_t c)
{
    if (!valid_rows(n, c)) return 0;
    return sizeof(float) * 2 * static_cast<size_t>(c) * static_cast<size_t>(layer_norm_parts(n, c));
}

sparse_status_t sparse_layer_norm(const void* x, sparse_dtype_t x_type, int64_t r, int64_t c, const int64_t* idx,
                                  int64_t n, const float* gamma, const float* beta, double eps, void* y,
                                  sparse_dtype_t y_type, float* mean, float* rstd, int32_t* d_err, cudaStream_t stream)
{
    if (!valid_norm(x, x_type, r, c, idx, n, y_type, d_err) || !(eps >= 0.0) || !std::isfinite(eps))
        return SPARSE_ERR_INVALID_ARG;
    if (n == 0) return SPARSE_OK;
    if (y == nullptr) return SPARSE_ERR_INVALID_ARG;
    const bool xb = is_bf16(x_type), yb = is_bf16(y_type);
    const int vec = access(c, xb || yb, x, xb, y, yb, y, yb);
    return from_cuda(layer_norm(x, is_bf16(x_type), r, c, idx, n, gamma, beta, small_eps(eps), y,
                                is_bf16(y_type), vec, mean, rstd, d_err, stream));
}

sparse_status_t sparse_layer_norm_grad(const void* dy, sparse_dtype_t y_type, const void* x, sparse_dtype_t x_type,
                                       int64_t r, int64_t c, const int64_t* idx, int64_t n, const float* gamma,
                                       const float* mean, const float* rstd, void* dx, float* dgamma, float* dbeta,
                                       void* ws, size_t ws_bytes, int32_t* d_err, cudaStream_t stream)
{
    if (!valid_norm(x, x_type, r, c, idx, n, y_type, d_err)) return SPARSE_ERR_INVALID_ARG;
    if (n > 0 && (dy == nullptr || mean == nullptr || rstd == nullptr || dx == nullptr)) return SPARSE_ERR_INVALID_ARG;
    if ((dgamma != nullptr || dbeta != nullptr) && n > 0 &&
        !ws_ok(ws, ws_bytes, sparse_layer_norm_workspace_size(n, c)))
        return SPARSE_ERR_WORKSPACE;
    const bool xb = is_bf16(x_type), yb = is_bf16(y_type);
    const int vec = access(c, xb || yb, x, xb, dy, yb, dx, xb);
    return from_cuda(layer_norm_grad(dy, is_bf16(y_type), x, is_bf16(x_type), r, c, idx, n, gamma, mean, rstd, dx,
                                     dgamma, dbeta, static_cast<float*>(ws), vec, d_err, stream));
}

size_t sparse_expert_workspace_size(int64_t n, int64_t k, int64_t experts)
{
    if (n < 0 || k < 1 || (n > 0 && k > INT32_MAX / n) || experts < 1 || experts > kMaxExperts) return 0;
    return expert_ws_bytes(n * k, experts);
}

sparse_status_t sparse_expert_sort(const int64_t* expert, int64_t n, int64_t k, int64_t experts, int64_t* offsets,
                                   int32_t* src, int32_t* pos, void* ws, size_t ws_bytes, int32_t* d_err,
                                   cudaStream_t stream)
{
    if (!valid_expert(SPARSE_F32, n, k, 1, d_err) || experts < 1 || experts > kMaxExperts || offsets == nullptr)
        return SPARSE_ERR_INVALID_ARG;
    if (n > 0 && (expert == nullptr || pos == nullptr)) return SPARSE_ERR_INVALID_ARG;
    if (n == 0)
        return from_cuda(cudaMemsetAsync(offsets, 0, sizeof(int64_t) * static_cast<size_t>(experts + 1), stream));
    if (!ws_ok(ws, ws_bytes, sparse_expert_workspace_size(n, k, experts))) return SPARSE_ERR_WORKSPACE;
    return from_cuda(expert_sort(expert, n * k, experts, offsets, src, pos, ws, d_err, stream));
}

sparse_status_t sparse_expert_dispatch(const void* x, sparse_dtype_t type, int64_t n, int64_t k, int64_t c,
                                       const int32_t* pos, const int64_t* offsets, int64_t experts, void* xs,
                                       int32_t* d_err, cudaStream_t stream)
{
    if (!valid_expert(type, n, k, c, d_err) || experts < 1 || experts > kMaxExperts) return SPARSE_ERR_INVALID_ARG;
    if (n == 0) return SPARSE_OK;
    if (x == nullptr || pos == nullptr || offsets == nullptr || xs == nullptr) return SPARSE_ERR_INVALID_ARG;
    const bool b = is_bf16(type);
    const int vec = access(c, b, x, b, xs, b, xs, b);
    return from_cuda(expert_dispatch(x, is_bf16(type), n, k, c, pos, offsets + experts, xs, vec, d_err, stream));
}

sparse_status_t sparse_expert_combine(const void* ys, sparse_dtype_t type, int64_t n, int64_t k, int64_t c,
                                      const int32_t* pos, const float* weights, void* y, int32_t* d_err,
                                      cudaStream_t stream)
{
    if (!valid_expert(type, n, k, c, d_err)) return SPARSE_ERR_INVALID_ARG;
    if (n == 0) return SPARSE_OK;
    if (ys == nullptr || pos == nullptr || y == nullptr) return SPARSE_ERR_INVALID_ARG;
    const bool b = is_bf16(type);
    const int vec = access(c, b, ys, b, y, b, y, b);
    return from_cuda(expert_combine(ys, is_bf16(type), n, k, c, pos, weights, y, vec, d_err, stream));
}

sparse_status_t sparse_expert_combine_grad(const void* dy, const void* ys, sparse_dtype_t type, int64_t n, int64_t k,
                                           int64_t c, const int32_t* pos, const int64_t* offsets, int64_t experts,
                                           const float* weights, void* dys, float* dweights, int32_t* d_err,
                                           cudaStream_t stream)
{
    if (!valid_expert(type, n, k, c, d_err) || experts < 1 || experts > kMaxExperts) return SPARSE_ERR_INVALID_ARG;
    if (n == 0) return SPARSE_OK;
    if (dy == nullptr || ys == nullptr || pos == nullptr || offsets == nullptr || dys == nullptr)
        return SPARSE_ERR_INVALID_ARG;
    const bool b = is_bf16(type);
    const int vec = access(c, b, dy, b, ys, b, dys, b);
    return from_cuda(expert_combine_grad(dy, ys, is_bf16(type), n, k, c, pos, offsets + experts, weights, dys,
                                         dweights, vec, d_err, stream));
}

sparse_status_t sparse_expert_route(const void* logits, sparse_dtype_t type, int64_t n, int64_t experts, int64_t k,
                                    int renormalize, int64_t* expert, float* weights, int32_t* d_err, cudaStream_t stream)
{
    if (!valid_route(type, n, experts, k, d_err)) return SPARSE_ERR_INVALID_ARG;
    if (n == 0) return SPARSE_OK;
    if (logits == nullptr || expert == nullptr || weights == nullptr) return SPARSE_ERR_INVALID_ARG;
    return from_cuda(expert_route(logits, is_bf16(type), n, experts, static_cast<int>(k), renormalize != 0, expert, weights,
                                  d_err, stream));
}

sparse_status_t sparse_expert_route_grad(const float* dweights, const void* logits, sparse_dtype_t type, int64_t n,
                                         int64_t experts, int64_t k, int renormalize, const int64_t* expert,
                                         const float* weights, void* dlogits, int32_t* d_err, cudaStream_t stream)
{
    if (!valid_route(type, n, experts, k, d_err)) return SPARSE_ERR_INVALID_ARG;
    if (n == 0) return SPARSE_OK;
    if (dweights == nullptr || (logits == nullptr && renormalize == 0) || expert == nullptr || weights == nullptr ||
        dlogits == nullptr)
        return SPARSE_ERR_INVALID_ARG;
    return from_cuda(expert_route_grad(dweights, logits, is_bf16(type), n, experts, static_cast<int>(k), renormalize != 0,
                                       expert, weights, dlogits, d_err, stream));
}

size_t sparse_expert_matmul_workspace_size(sparse_dtype_t type, int64_t n, int64_t a, int64_t b, int64_t experts, int aligned)
{
    if (!valid_matmul(type, n, a, b, experts)) return 0;
    return n > 0 ? expert_matmul_ws_bytes(!is_bf16(type), n, a, b, experts, aligned != 0) : 256;
}

sparse_status_t sparse_expert_matmul(const void* x, const void* w, sparse_dtype_t type, int64_t n, int64_t a, int64_t b,
                                     int transpose, const int64_t* offsets, int64_t experts, void* y, void* ws,
                                     size_t ws_bytes, int32_t* d_err, cudaStream_t stream)
{
    if (!valid_matmul(type, n, a, b, experts) || d_err == nullptr) return SPARSE_ERR_INVALID_ARG;
    if (n == 0) return SPARSE_OK;
    if (x == nullptr || w == nullptr || offsets == nullptr || y == nullptr) return SPARSE_ERR_INVALID_ARG;
    ExpertMatmul M{};
    M.x = x;
    M.w = w;
    M.f32 = !is_bf16(type);
    M.transpose = transpose != 0;
    M.n = n;
    M.a = a;
    M.b = b;
    M.experts = experts;
    M.offsets = offsets;
    M.out = y;
    M.d_err = d_err;
    if (!ws_ok(ws, ws_bytes, expert_matmul_ws_bytes(M))) return SPARSE_ERR_WORKSPACE;
    return from_cuda(expert_matmul(M, ws, stream));
}

sparse_status_t sparse_expert_matmul_grad(const void* x, const void* dy, sparse_dtype_t type, int64_t n, int64_t a,
                                          int64_t b, const int64_t* offsets, int64_t experts, void* dw,
                                          sparse_dtype_t dw_type, void* ws, size_t ws_bytes, int32_t* d_err,
                                          cudaStream_t stream)
{
    if (!valid_matmul(type, n, a, b, experts) || !valid_type(dw_type) || (is_bf16(dw_type) && !is_bf16(type)) ||
        dw == nullptr || d_err == nullptr)
        return SPARSE_ERR_INVALID_ARG;
    if (n == 0)
        return from_cuda(cudaMemsetAsync(dw, 0, static_cast<size_t>(experts * a * b) * (is_bf16(dw_type) ? 2 : 4), stream));
    if (x == nullptr || dy == nullptr || offsets == nullptr) return SPARSE_ERR_INVALID_ARG;
    ExpertMatmul M{};
    M.x = x;
    M.dy = dy;
    M.f32 = !is_bf16(type);
    M.out_bf16 = is_bf16(dw_type);
    M.n = n;
    M.a = a;
    M.b = b;
    M.experts = experts;
    M.offsets = offsets;
    M.out = dw;
    M.d_err = d_err;
    if (!ws_ok(ws, ws_bytes, expert_matmul_ws_bytes(M))) return SPARSE_ERR_WORKSPACE;
    return from_cuda(expert_matmul_grad(M, ws, stream));
}

size_t sparse_vocab_loss_workspace_size(sparse_dtype_t type, int64_t n, int64_t c, int64_t v, int grad, int aligned)
{
    if (!valid_loss(type, n, c, v)) return 0;
    if (n == 0) return 256;
    const size_t forward = vocab_loss_ws_bytes(!is_bf16(type), n, c, v, 0, aligned != 0);
    return grad ? std::max(forward, vocab_loss_ws_bytes(!is_bf16(type), n, c, v, 1, aligned != 0)) : forward;
}

sparse_status_t sparse_vocab_loss(const void* x, const void* w, sparse_dtype_t type, int64_t n, int64_t c, int64_t v,
                                  const int64_t* target, float* loss, float* lse, void* ws, size_t ws_bytes,
                                  int32_t* d_err, cudaStream_t stream)
{
    if (!valid_loss(type, n, c, v) || d_err == nullptr) return SPARSE_ERR_INVALID_ARG;
    if (n == 0) return SPARSE_OK;
    if (x == nullptr || w == nullptr || target == nullptr || loss == nullptr || lse == nullptr) return SPARSE_ERR_INVALID_ARG;
    VocabLoss V{};
    V.x = x;
    V.w = w;
    V.f32 = !is_bf16(type);
    V.n = n;
    V.c = c;
    V.v = v;
    V.target = target;
    V.loss = loss;
    V.lse = lse;
    V.d_err = d_err;
    if (!ws_ok(ws, ws_bytes, vocab_loss_ws_bytes(V, 0))) return SPARSE_ERR_WORKSPACE;
    return from_cuda(vocab_loss(V, ws, stream));
}

sparse_status_t sparse_vocab_loss_grad(const float* dloss, const void* x, const void* w, sparse_dtype_t type, int64_t n,
                                       int64_t c, int64_t v, const int64_t* target, const float* lse, void* dx, void* dw,
                                       void* ws, size_t ws_bytes, int32_t* d_err, cudaStream_t stream)
{
    if (!valid_loss(type, n, c, v) || d_err == nullptr) return SPARSE_ERR_INVALID_ARG;
    if (n == 0)   // no token: no gradient
        return dw == nullptr ? SPARSE_OK
                             : from_cuda(cudaMemsetAsync(dw, 0, static_cast<size_t>(v * c) * (is_bf16(type) ? 2 : 4), stream));
    if (x == nullptr || w == nullptr || target == nullptr || lse == nullptr) return SPARSE_ERR_INVALID_ARG;
    if (dx == nullptr && dw == nullptr) return SPARSE_OK;
    VocabLoss V{};
    V.x = x;
    V.w = w;
    V.f32 = !is_bf16(type);
    V.n = n;
    V.c = c;
    V.v = v;
    V.target = target;
    V.lse = const_cast<float*>(lse);
    V.dloss = dloss;
    V.dx = dx;
    V.dw = dw;
    V.d_err = d_err;
    if (!ws_ok(ws, ws_bytes, vocab_loss_ws_bytes(V, 1))) return SPARSE_ERR_WORKSPACE;
    return from_cuda(vocab_loss_grad(V, ws, stream));
}

size_t sparse_muon_workspace_size(int64_t batch, int64_t r, int64_t c, int products)
{
    if (!valid_batch(batch, r, c) || (products != 1 && products != 3)) return 0;
    return batch > 0 ? muon_ws_bytes(batch, r, c, products) : 0;
}

sparse_status_t sparse_orthogonalize(const void* u, sparse_dtype_t u_type, int64_t batch, int64_t r, int64_t c,
                                     sparse_ns_config_t cfg, void* out, sparse_dtype_t out_type, void* ws,
                                     size_t ws_bytes, int32_t* d_err, cudaStream_t stream)
{
    if (!valid_type(u_type) || !valid_type(out_type) || !valid_batch(batch, r, c) || !valid_ns(cfg) || d_err == nullptr)
        return SPARSE_ERR_INVALID_ARG;
    if (batch == 0) return SPARSE_OK;
    if (u == nullptr || out == nullptr) return SPARSE_ERR_INVALID_ARG;
    if (!ws_ok(ws, ws_bytes, muon_ws_bytes(batch, r, c, cfg.products))) return SPARSE_ERR_WORKSPACE;
    MuonParams M = muon_params(batch, r, c, cfg, d_err);
    M.g = u;
    M.g_bf16 = is_bf16(u_type);
    M.out = out;
    M.out_bf16 = is_bf16(out_type);
    return from_cuda(muon(M, ws, stream));
}

sparse_status_t sparse_muon_step(float* w, float* buf, const void* g, sparse_dtype_t g_type, int64_t batch, int64_t r,
                                 int64_t c, sparse_muon_config_t cfg, void* ws, size_t ws_bytes, int32_t* d_err,
                                 cudaStream_t stream)
{
    if (!valid_type(g_type) || !valid_batch(batch, r, c) || !valid_ns(cfg.ns) || d_err == nullptr ||
        !std::isfinite(cfg.lr) || !std::isfinite(cfg.scale) || !std::isfinite(cfg.momentum) || cfg.momentum < 0.0 ||
        !std::isfinite(cfg.weight_decay) || cfg.weight_decay < 0.0)
        return SPARSE_ERR_INVALID_ARG;
    if (batch == 0) return SPARSE_OK;
    if (w == nullptr || buf == nullptr || g == nullptr) return SPARSE_ERR_INVALID_ARG;
    if (!ws_ok(ws, ws_bytes, muon_ws_bytes(batch, r, c, cfg.ns.products))) return SPARSE_ERR_WORKSPACE;
    MuonParams M = muon_params(batch, r, c, cfg.ns, d_err);
    M.g = g;
    M.g_bf16 = is_bf16(g_type);
    M.buf = buf;
    M.momentum = static_cast<float>(cfg.momentum);
    M.nesterov = cfg.nesterov != 0;
    M.w = w;
    M.decay = static_cast<float>(1.0 - cfg.lr * cfg.weight_decay);
    M.lr = static_cast<float>(cfg.lr * cfg.scale);
    return from_cuda(muon(M, ws, stream));
}

}  // extern "C"
