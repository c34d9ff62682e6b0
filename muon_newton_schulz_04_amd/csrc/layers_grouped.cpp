// C ABI of the linear layers of a mixture of experts (include/libmuon.h): argument
// checks, the choice of tile, and the launches on the caller's stream.

#include "layer_checks.hpp"

using namespace muon::checks;

namespace {

muon_status check_grouped(const muon_grouped* d) {
    if (!d) return fail(MUON_E_INVALID_ARG, "null descriptor");
    if (d->dtype != MUON_TYPE_BF16 && d->dtype != MUON_TYPE_FP16)
        return fail(MUON_E_INVALID_ARG, "grouped linear: dtype must be bf16 or fp16");
    if (d->weight_layout != MUON_WEIGHT_IN_OUT && d->weight_layout != MUON_WEIGHT_OUT_IN)
        return fail(MUON_E_INVALID_ARG, "grouped linear: bad weight_layout");
    if (d->rows < 0 || d->rows >= kMaxRows) return fail(MUON_E_SHAPE, "grouped linear: rows must be in [0, 2^24)");
    if (d->experts < 1 || d->experts > 65536)
        return fail(MUON_E_SHAPE, "grouped linear: experts must be in [1, 2^16]");
    if (d->in_features < 8 || d->in_features > kMaxCols || d->out_features < 8 || d->out_features > kMaxCols)
        return fail(MUON_E_SHAPE, "grouped linear: features must be in [8, 2^21]");
    const bool io = d->weight_layout == MUON_WEIGHT_IN_OUT;
    const int64_t r = io ? d->in_features : d->out_features, c = io ? d->out_features : d->in_features;
    TRY(check_ld(d->ld_x, d->in_features, "ld_x"));
    TRY(check_ld(d->ld_w, c, "ld_w"));
    TRY(check_ld(d->ld_y, d->out_features, "ld_y"));
    const int64_t least = (r - 1) * stride_of(d->ld_w, c) + c;
    if (d->stride_w != 0 && (d->stride_w < least || d->stride_w > (int64_t)1 << 42))
        return fail(MUON_E_LAYOUT, "stride_w must be 0 or from a weight's extent to 2^42");
    return MUON_OK;
}

// The weights (or their gradients) as one run of elements, and the elements from one
// to the next.
int64_t weight_step(const muon_grouped& d) {
    const bool io = d.weight_layout == MUON_WEIGHT_IN_OUT;
    const int64_t r = io ? d.in_features : d.out_features, c = io ? d.out_features : d.in_features;
    return d.stride_w ? d.stride_w : r * stride_of(d.ld_w, c);
}
Tensor weights_of(const muon_grouped& d, const void* p, int size) {
    const bool io = d.weight_layout == MUON_WEIGHT_IN_OUT;
    const int64_t r = io ? d.in_features : d.out_features, c = io ? d.out_features : d.in_features;
    const int64_t n = (d.experts - 1) * weight_step(d) + (r - 1) * stride_of(d.ld_w, c) + c;
    return {p, 1, n, n, size};
}
Tensor rows_of(const muon_grouped& d, const void* p, int64_t cols, int64_t ld) {
    return {p, d.rows, cols, stride_of(ld, cols), 2};
}

// Rows that start 16-byte aligned and are whole chunks of 8; else the small tile reads
// them through registers.
bool whole_chunks(const void* p, int64_t ld, int64_t cols) { return aligned16(p, ld, 2) && cols % 8 == 0; }

// The tiles of the forward pass and the input gradient, by prices fitted to times
// measured over 24 shapes and every tile (rows, experts, in, out; bf16, us, small, small
// in groups, square, square in groups, tall): 48, 16, 768, 1536 8.9, 11.8, 13.0, 12.0,
// 17.5; 2, 16, 6400, 1600 29, 21, 64, 47, 84 (blocks of 16 rows 13.2); 4099, 8, 1536,
// 768 25, 31, 22, 19, 28; 4096, 8, 1600, 1600 45, 59, 28, 38, 30; 32768, 16, 1600, 1600
// 301, 381, 184, 253, 161.
constexpr TileCost kRowTiles[] = {{muon::TILE_TALL, 256, 128, 6.0, 0.82, 1.65, 5.0, 512},
                                  {muon::TILE_SQUARE, 128, 128, 5.0, 0.65, 0.95, 3.0, 512},
                                  {muon::TILE_SQUARE_GROUPS, 128, 128, 5.5, 0.52, 0.75, 3.0, 256},
                                  {muon::TILE_SMALL, 64, 64, 4.0, 0.26, 0.48, 1.0, 512},
                                  {muon::TILE_SMALL_GROUPS, 64, 64, 5.0, 0.18, 0.33, 2.0, 256}};
// The weight gradient's, over 18 shapes, 3 tiles and 1 to 32 pieces of each expert's rows;
// rows, experts, in, out; us whole and in the best of the pieces (small, square, tall):
// 32768, 16, 1600, 1600 351, 253, 227; 32768, 2, 2048, 800 269 and 260, 293 and 174, 394
// and 167; 32768, 4, 768, 768 92 and 92, 166 and 87, 209 and 95; 32768, 4, 256, 128 60 and
// 19, 121 and 22, 164 and 25; 4099, 8, 1536, 768 40, 36, 39.
constexpr TileCost kWeightTiles[] = {{muon::TILE_TALL, 256, 128, 10.0, 0.83, 1.47, 0.0, 512},
                                     {muon::TILE_SQUARE, 128, 128, 8.0, 0.64, 0.85, 0.0, 512},
                                     {muon::TILE_SMALL, 64, 64, 8.0, 0.23, 0.31, 0.65, 512}};

int64_t up_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct GroupedPlan {
    muon::TileKind tile;
    int rows, cols;
    int pieces = 1;  // of each expert's rows (weight gradient)
};

// Workgroups of the forward pass and the input gradient: every expert with rows may end
// inside a tile.
int64_t most_blocks(int64_t rows, int64_t experts, int64_t tall) {
    return (rows < experts ? rows : experts) + rows / tall;
}
int64_t rows_grid(const GroupedPlan& p, int64_t rows, int64_t experts, int64_t N) {
    return most_blocks(rows, experts, p.rows) * up_div(N, p.cols);
}

// A launch has fewer than 2^32 threads.
bool fits(int64_t grid, muon::TileKind tile) {
    const bool two = tile != muon::TILE_TALL && tile != muon::TILE_SQUARE && tile != muon::TILE_SMALL;
    return grid < (int64_t)1 << (two ? 23 : 24);
}

// How many blocks of `tall` rows the groups are, as far as the host can tell: half a
// block more for each group that has rows.
double expected_blocks(int64_t rows, int64_t experts, int64_t tall) {
    const double some = (double)(rows < experts ? rows : experts), n = (double)rows / (double)tall + 0.5 * some;
    return std::ceil(n > some ? n : some);
}

// rows 0: no tile's workgroups fit one launch
GroupedPlan rows_plan(int64_t rows, int64_t experts, int64_t N, int64_t K, bool b_kc) {
    const double slices = (double)up_div(K, muon::kGemmSlice);
    GroupedPlan best{};
    double least = 1e300;
    for (const TileCost& c : kRowTiles) {
        const GroupedPlan p{c.kind, c.rows, c.cols};
        if (!fits(rows_grid(p, rows, experts, N), c.kind)) continue;
        const double t = tile_price(c, expected_blocks(rows, experts, c.rows) * (double)up_div(N, c.cols), slices);
        if (t >= least) continue;
        least = t;
        best = p;
    }
    // blocks of few rows: rounds of 256 workgroups, each a wait of its own
    const bool one = rows <= 16 * experts;
    const int cols = b_kc ? 16 : 32, tall = one ? 16 : 32;
    const double wgs = expected_blocks(rows, experts, tall) * (double)up_div(N, cols);
    const double t = 4.0 + std::ceil(wgs / 256) * (b_kc ? 2.2 + 0.038 * slices : 2.6 + 0.08 * slices);
    const GroupedPlan few{one ? muon::TILE_FEW16 : muon::TILE_FEW32, tall, cols};
    return t < least && fits(rows_grid(few, rows, experts, N), few.tile) ? few : best;
}

// The workgroups of a weight gradient: an expert's tiles, in runs of one length for each
// of the 8 XCDs, for each piece of its rows.
int64_t weight_grid(const GroupedPlan& p, int64_t experts, int64_t M, int64_t N) {
    return experts * p.pieces * (up_div(up_div(M, p.rows) * up_div(N, p.cols), 8) * 8);
}

// Few tiles of long sums leave CUs idle: then each expert's rows are cut into pieces,
// whose sums meet in a second kernel (its launch, and each piece's sums once written
// and read). rows 0: no tile's workgroups fit one launch.
GroupedPlan weight_plan(int64_t rows, int64_t experts, int64_t M, int64_t N, bool raw) {
    // the longest of the sums, where some experts have half as much again as the mean
    const double all = 1.5 * (double)rows / (double)experts / muon::kGemmSlice;
    const double out = (double)experts * (double)M * (double)N;
    GroupedPlan best{};
    double least = 1e300;
    for (int pieces = 1; pieces == 1 || (pieces <= 64 && all >= 8.0 * pieces); pieces *= 2)
        for (const TileCost& c : kWeightTiles) {
            if (raw && c.kind != muon::TILE_SMALL) continue;
            const GroupedPlan p{c.kind, c.rows, c.cols, pieces};
            const int64_t grid = weight_grid(p, experts, M, N);
            if (!fits(grid, c.kind)) continue;
            if (pieces > 1 && (grid >= (int64_t)1 << 22 || M * N >= (int64_t)1 << 31)) continue;
            double t = tile_price(c, (double)(experts * pieces * up_div(M, c.rows) * up_div(N, c.cols)), 1.0 + all / pieces);
            if (pieces > 1) t += 3.3 + out * (2 * pieces + 1) * 4e-6 / 4.9;
            if (t >= least) continue;
            least = t;
            best = p;
        }
    return best;
}

struct WeightLayout {
    bool io, raw;  // weight_layout; operands read as they are
    int64_t M, N;  // an expert's gradient
    GroupedPlan plan;
    int64_t ld_part;
    size_t part, need;  // bytes of the pieces' sums, with those of their bias sums
};
WeightLayout weight_layout(const muon_grouped& d, const void* x, const void* dy) {
    WeightLayout w{};
    w.io = d.weight_layout == MUON_WEIGHT_IN_OUT;
    w.M = w.io ? d.in_features : d.out_features;
    w.N = w.io ? d.out_features : d.in_features;
    const int64_t ld_x = stride_of(d.ld_x, d.in_features), ld_y = stride_of(d.ld_y, d.out_features);
    w.raw = d.rows > 0 && (!whole_chunks(x, ld_x, d.in_features) || !whole_chunks(dy, ld_y, d.out_features));
    w.plan = weight_plan(d.rows, d.experts, w.M, w.N, w.raw);
    w.ld_part = (w.N + 3) / 4 * 4;
    if (w.plan.pieces > 1) {
        const size_t each = (size_t)w.plan.pieces * (size_t)d.experts;
        w.part = up256(each * (size_t)(w.M * w.ld_part) * 4);
        w.need = w.part + up256(each * (size_t)d.out_features * 4);
    }
    return w;
}

muon_status too_large() { return fail(MUON_E_SHAPE, "grouped linear: output too large"); }

// forward and grad input
muon_status run_grouped(const muon_grouped* d, bool fwd, const void* a, const void* w, const int32_t* offsets,
                        const muon_epilogue* e, void* y, void* stream) {
    TRY(check_grouped(d));
    const int64_t N = fwd ? d->out_features : d->in_features, K = fwd ? d->in_features : d->out_features;
    const muon_epilogue none{};
    if (!e) e = &none;
    TRY(check_epilogue(fwd, N, *e));
    if (d->rows == 0) return MUON_OK;
    if (!a || !w || !offsets || !y) return fail(MUON_E_INVALID_ARG, "null tensor");
    if (!fwd && e->activation != MUON_ACT_NONE && !e->z)
        return fail(MUON_E_INVALID_ARG, "grad input: an activation needs its pre-activation z");
    const Tensor A = rows_of(*d, a, K, fwd ? d->ld_x : d->ld_y), W = weights_of(*d, w, 2);
    const Outputs o = outputs_of(fwd, d->rows, N, fwd ? d->ld_y : d->ld_x, *e, y);
    const Tensor &Y = o.y, &R = o.add, &Z = o.z;
    const Tensor Bi{e->bias, 1, d->experts * N, d->experts * N, 4}, Of{offsets, 1, d->experts + 1, d->experts + 1, 4};
    for (const Tensor& t : {A, W, Y, R, Z}) TRY(check_align(t.p, 2, "a 16-bit tensor"));
    TRY(check_align(e->bias, 4, "bias"));
    TRY(check_align(offsets, 4, "offsets"));
    TRY(check_disjoint(Y, {A, W, Z, Bi, Of}));
    TRY(check_add(Y, R));
    if (fwd) TRY(check_disjoint(Z, {A, W, R, Bi, Of}));
    // B's k index is contiguous where its rows are output features
    const bool b_kc = fwd == (d->weight_layout == MUON_WEIGHT_OUT_IN);
    const int64_t wc = d->weight_layout == MUON_WEIGHT_IN_OUT ? d->out_features : d->in_features;
    const int64_t ld_w = stride_of(d->ld_w, wc), step = weight_step(*d);
    const bool raw = !whole_chunks(a, A.ld, K) || !whole_chunks(w, ld_w, wc) || step % 8 != 0;
    const GroupedPlan plan = raw ? GroupedPlan{muon::TILE_SMALL, 64, 64} : rows_plan(d->rows, d->experts, N, K, b_kc);
    if (plan.rows == 0 || !fits(rows_grid(plan, d->rows, d->experts, N), plan.tile)) return too_large();
    muon::GroupedArgs p{};
    p.a = a;
    p.b = w;
    p.offsets = offsets;
    p.stride_w = step;
    p.ld_a = (int)A.ld;
    p.ld_b = (int)ld_w;
    p.rows = (int)d->rows;
    p.experts = (int)d->experts;
    p.N = (int)N;
    p.K = (int)K;
    p.tiles_n = (int)up_div(N, plan.cols);
    p.epi = epilogue_args(fwd, *e, o);
    p.tiles_m = (int)most_blocks(d->rows, d->experts, plan.rows);
    const int64_t grid = rows_grid(plan, d->rows, d->experts, N);
    TRY(check_device());
    return hip_status(muon::launch_grouped(p, plan.tile, raw, b_kc, d->dtype, (unsigned)grid,
                                           static_cast<hipStream_t>(stream)),
                      "grouped product kernel");
}

}  // namespace

extern "C" {

muon_status muon_grouped_linear_forward(const muon_grouped* d, const void* x, const void* w, const int32_t* offsets,
                                        const muon_epilogue* e, void* y, void* stream) {
    return guarded([&]() { return run_grouped(d, true, x, w, offsets, e, y, stream); });
}

muon_status muon_grouped_linear_grad_input(const muon_grouped* d, const void* dy, const void* w, const int32_t* offsets,
                                           const muon_epilogue* e, void* dx, void* stream) {
    return guarded([&]() { return run_grouped(d, false, dy, w, offsets, e, dx, stream); });
}

muon_status muon_grouped_linear_workspace_bytes(const muon_grouped* d, const void* x, const void* dy,
                                                size_t* out_bytes) {
    return guarded([&]() -> muon_status {
        if (!out_bytes) return fail(MUON_E_INVALID_ARG, "null out_bytes");
        TRY(check_grouped(d));
        *out_bytes = weight_layout(*d, x, dy).need;
        return MUON_OK;
    });
}

muon_status muon_grouped_linear_grad_weight(const muon_grouped* d, const void* x, const void* dy,
                                            const int32_t* offsets, float* dw, float* dbias, int32_t accumulate,
                                            void* workspace, size_t ws_bytes, void* stream) {
    return guarded([&]() -> muon_status {
        TRY(check_grouped(d));
        if (!dw || !offsets || (d->rows > 0 && (!x || !dy))) return fail(MUON_E_INVALID_ARG, "null tensor");
        const WeightLayout lay = weight_layout(*d, x, dy);
        const bool io = lay.io;
        const Tensor X = rows_of(*d, x, d->in_features, d->ld_x), Y = rows_of(*d, dy, d->out_features, d->ld_y);
        const Tensor W = weights_of(*d, dw, 4), Bi{dbias, 1, d->experts * d->out_features, d->experts * d->out_features, 4};
        const Tensor Of{offsets, 1, d->experts + 1, d->experts + 1, 4};
        TRY(check_align(x, 2, "x"));
        TRY(check_align(dy, 2, "dy"));
        TRY(check_align(dw, 4, "dw"));
        TRY(check_align(dbias, 4, "dbias"));
        TRY(check_align(offsets, 4, "offsets"));
        TRY(check_disjoint(W, {X, Y, Bi, Of}));
        TRY(check_disjoint(Bi, {X, Y, Of}));
        const Tensor &A = io ? X : Y, &B = io ? Y : X;
        const GroupedPlan& plan = lay.plan;
        if (plan.rows == 0) return too_large();
        const int64_t grid = weight_grid(plan, d->experts, lay.M, lay.N);
        TRY(check_workspace(workspace, ws_bytes, lay.need));
        const Tensor K{workspace, 1, (int64_t)lay.need, (int64_t)lay.need, 1};
        TRY(check_disjoint(K, {X, Y, W, Bi, Of}));
        muon::GroupedArgs p{};
        p.a = A.p;
        p.b = B.p;
        p.offsets = offsets;
        p.stride_w = weight_step(*d);
        p.sums = dbias;
        p.ld_a = (int)A.ld;
        p.ld_b = (int)B.ld;
        p.rows = (int)d->rows;
        p.experts = (int)d->experts;
        p.M = (int)A.cols;
        p.N = (int)B.cols;
        p.tiles_m = (int)up_div(A.cols, plan.rows);
        p.tiles_n = (int)up_div(B.cols, plan.cols);
        p.epi.mode = muon::EPI_GRAD_WEIGHT;
        p.epi.y = dw;
        p.epi.ld_y = (int)stride_of(d->ld_w, io ? d->out_features : d->in_features);
        const bool cut = plan.pieces > 1;
        p.epi.accumulate = accumulate != 0 && !cut;
        p.pieces = plan.pieces;
        p.ld_part = (int)lay.ld_part;
        const int ld_w = p.epi.ld_y;
        if (cut) {
            p.part = static_cast<float*>(workspace);
            p.part_sums = reinterpret_cast<float*>(static_cast<char*>(workspace) + lay.part);
            p.epi.ld_y = p.ld_part;
        }
        TRY(check_device());
        // dy is the second operand of an [in, out] gradient, else the first
        const int sum = !dbias ? 0 : io ? 1 : 2;
        hipStream_t st = static_cast<hipStream_t>(stream);
        TRY(hip_status(muon::launch_grouped_weight(p, plan.tile, lay.raw, d->dtype, sum, (unsigned)grid, st),
                       "grouped weight gradient kernel"));
        if (!cut) return MUON_OK;
        p.epi.accumulate = accumulate != 0;
        p.epi.ld_y = ld_w;
        return hip_status(muon::launch_grouped_join(p, dbias ? (int)d->out_features : 0, st),
                          "grouped weight gradient sums");
    });
}

}  // extern "C"
