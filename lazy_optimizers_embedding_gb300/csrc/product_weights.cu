// product_weights.cu -- the gradients of the groups' matrices: the product of two
// arrays of rows over each group's rows.
#include "product.cuh"

namespace so {

namespace {

int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a; }

template <class S>
cudaError_t weights_form(const WeightsProduct& R, cudaStream_t s)
{
    ProductMaps maps;
    if (!R.a.map(&maps.a) || !R.b.map(&maps.b)) return cudaErrorInvalidValue;
    ProductArgs Q{};
    Q.rows = static_cast<int32_t>(R.rows);
    Q.m = static_cast<int32_t>(R.m);
    Q.n = static_cast<int32_t>(R.n);
    Q.m_tiles = static_cast<int32_t>(up(R.m, S::TM));
    Q.n_tiles = static_cast<int32_t>(up(R.n, S::BN));
    Q.width = static_cast<int32_t>(up(up(R.n, Q.n_tiles), 32) * 32);   // equal tiles
    Q.groups = R.groups;
    Q.splits = R.splits;
    Q.offsets = R.offsets;
    Q.out = R.out;
    Q.slab = static_cast<int64_t>(R.groups) * R.n * R.m;
    Q.ld = static_cast<int32_t>(R.m);
    Q.out_bf16 = R.out_bf16;
    Q.release = R.release;
    Q.unit = R.unit;
    Q.d_err = R.d_err;
    return run_product<S>("weights_product", maps, Q, static_cast<int64_t>(Q.m_tiles) * Q.n_tiles * R.groups * R.splits, s);
}

}  // namespace

int weights_splits(int64_t rows, int64_t m, int64_t n, int64_t groups, int parts)
{
    const int64_t tiles = groups * up(m, 128) * up(n, parts == 3 ? 128 : 256);
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({kSms / tiles, rows / groups / (4 * kPK), 64})));
}

cudaError_t weights_product(const WeightsProduct& R, cudaStream_t s)
{
    // pairs of blocks: see rows_product
    const int64_t tiles = R.groups * up(R.m, 128) * up(R.n, R.b.parts == 3 ? 128 : 256);
    const bool pair = R.splits == 1 && up(R.m, 256) * 2 <= up(R.m, 128) + up(R.m, 128) / 4 && tiles >= kSms;
    if (R.b.parts == 3)
        return pair ? weights_form<ProductShape<kWeights, true, true, 2, 6, false>>(R, s)
                    : weights_form<ProductShape<kWeights, true, true, 1, 6, false>>(R, s);
    if (R.out_bf16)
        return pair ? weights_form<ProductShape<kWeights, true, true, 2, 1, false>>(R, s)
                    : weights_form<ProductShape<kWeights, true, true, 1, 1, false>>(R, s);
    return pair ? weights_form<ProductShape<kWeights, true, true, 2, 1, true>>(R, s)
                : weights_form<ProductShape<kWeights, true, true, 1, 1, true>>(R, s);
}

}  // namespace so
