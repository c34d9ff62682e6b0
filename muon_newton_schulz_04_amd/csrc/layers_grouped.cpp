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

// rows of a tile for `rows` rows of `experts` groups
int rows_tile(int64_t rows, int64_t experts, int64_t N) {
    const int64_t each = (rows + experts - 1) / experts;
    if (rows <= 16) return 16;
    if (each <= 16) return 32;
    const int64_t cols = (N + 127) / 128;
    if (each >= 384 && rows / 256 * cols >= 400) return 256;
    if (each >= 96 && rows / 128 * cols >= 200) return 128;
    return 64;
}

int weight_tile(int64_t rows, int64_t experts, int64_t M, int64_t N) {
    const int64_t cols = (N + 127) / 128;
    if (experts * ((M + 255) / 256) * cols >= 400 && M > 128) return 256;
    if (experts * ((M + 127) / 128) * cols >= 200) return 128;
    return 64;
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
    const int tile = raw ? 64 : rows_tile(d->rows, d->experts, N);
    const int tile_n = tile <= 32 ? (b_kc ? 16 : 32) : tile == 64 ? 64 : 128;
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
    p.tiles_n = (int)((N + tile_n - 1) / tile_n);
    p.epi = epilogue_args(fwd, *e, o);
    // every expert with rows may end inside a tile
    const int64_t most = (d->rows < d->experts ? d->rows : d->experts) + d->rows / tile, grid = most * p.tiles_n;
    if (grid >= (int64_t)1 << 22) return too_large();
    TRY(check_device());
    return hip_status(muon::launch_grouped(p, tile, raw, b_kc, d->dtype, (unsigned)grid, static_cast<hipStream_t>(stream)),
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

muon_status muon_grouped_linear_grad_weight(const muon_grouped* d, const void* x, const void* dy,
                                            const int32_t* offsets, float* dw, float* dbias, int32_t accumulate,
                                            void* stream) {
    return guarded([&]() -> muon_status {
        TRY(check_grouped(d));
        if (!dw || !offsets || (d->rows > 0 && (!x || !dy))) return fail(MUON_E_INVALID_ARG, "null tensor");
        const bool io = d->weight_layout == MUON_WEIGHT_IN_OUT;
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
        const bool raw = d->rows > 0 && (!whole_chunks(A.p, A.ld, A.cols) || !whole_chunks(B.p, B.ld, B.cols));
        const int tile = raw ? 64 : weight_tile(d->rows, d->experts, A.cols, B.cols);
        const int tile_n = tile == 64 ? 64 : 128;
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
        p.tiles_m = (int)((A.cols + tile - 1) / tile);
        p.tiles_n = (int)((B.cols + tile_n - 1) / tile_n);
        p.epi.mode = muon::EPI_GRAD_WEIGHT;
        p.epi.y = dw;
        p.epi.ld_y = (int)stride_of(d->ld_w, io ? d->out_features : d->in_features);
        p.epi.accumulate = accumulate != 0;
        const int64_t grid = d->experts * p.tiles_m * p.tiles_n;
        if (grid >= (int64_t)1 << 22) return too_large();
        TRY(check_device());
        // dy is the second operand of an [in, out] gradient, else the first
        const int sum = !dbias ? 0 : io ? 1 : 2;
        return hip_status(muon::launch_grouped_weight(p, tile, raw, d->dtype, sum, (unsigned)grid,
                                                      static_cast<hipStream_t>(stream)),
                          "grouped weight gradient kernel");
    });
}

}  // extern "C"
