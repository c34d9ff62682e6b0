// C ABI of the layer operators on 8-bit floating point with a float32 scale for each
// block of 128 (include/libmuon.h), and of the root-mean-square norm that can write
// it: argument checks and the launches on the caller's stream.

#include "layer_checks.hpp"

using namespace muon::checks;

namespace {

constexpr int64_t kBlock = muon::kScaleBlock;
int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }
int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

int size_of(int32_t dtype) { return dtype == MUON_TYPE_FP32 ? 4 : 2; }

muon_status check_type(int32_t dtype) {
    if (dtype < MUON_TYPE_BF16 || dtype > MUON_TYPE_FP32)
        return fail(MUON_E_INVALID_ARG, "dtype must be bf16, fp16 or fp32");
    return MUON_OK;
}

muon_status check_sizes(int64_t rows, int64_t cols) {
    if (rows < 0 || rows >= kMaxRows) return fail(MUON_E_SHAPE, "rows must be in [0, 2^24)");
    if (cols < 1 || cols > kMaxCols) return fail(MUON_E_SHAPE, "cols must be in [1, 2^21]");
    return MUON_OK;
}

// The data of an 8-bit matrix [rows, cols], each row with what follows it up to the
// next multiple of 16, and its scales.
Tensor data_of(const muon_eight& q, int64_t rows, int64_t cols) {
    return {q.data, rows, up16(cols), stride_of(q.ld, up16(cols)), 1};
}
Tensor scales_of(const muon_eight& q, int64_t a, int64_t b) { return {q.scale, 1, a * b, a * b, 4}; }

muon_status check_eight(const muon_eight& q, int64_t cols, bool weight) {
    if (q.format != MUON_EIGHT_E4M3 && (weight || q.format != MUON_EIGHT_E5M2))
        return fail(MUON_E_INVALID_ARG, weight ? "8-bit weights are E4M3" : "unknown 8-bit format");
    if (q.reserved != 0) return fail(MUON_E_INVALID_ARG, "8-bit matrix: reserved must be 0");
    if (!q.data || !q.scale) return fail(MUON_E_INVALID_ARG, "null 8-bit data or scales");
    if ((uintptr_t)q.data % 16 != 0 || q.ld % 16 != 0 || (q.ld != 0 && (q.ld < cols || q.ld > kMaxCols)))
        return fail(MUON_E_LAYOUT,
                    "8-bit rows must start 16-byte aligned: data and ld (0, or from the row length to 2^21)");
    return check_align(q.scale, 4, "scale");
}

muon_status check_rms(const muon_rmsnorm* d) {
    if (!d) return fail(MUON_E_INVALID_ARG, "null descriptor");
    TRY(check_type(d->dtype));
    TRY(check_sizes(d->rows, d->cols));
    if (!(d->eps >= 0.f) || !std::isfinite(d->eps))
        return fail(MUON_E_INVALID_ARG, "rmsnorm: eps must be finite and not negative");
    TRY(check_ld(d->ld_x, d->cols, "ld_x"));
    TRY(check_ld(d->ld_add, d->cols, "ld_add"));
    TRY(check_ld(d->ld_sum, d->cols, "ld_sum"));
    TRY(check_ld(d->ld_y, d->cols, "ld_y"));
    return check_ld(d->ld_dx, d->cols, "ld_dx");
}

size_t rms_workspace(const muon_rmsnorm& d) {
    return up256((size_t)muon::rms_backward_blocks(d.rows, d.cols, d.dtype) * (size_t)d.cols * 4);
}

// The tile of an 8-bit product: blocks of few rows while there are no more of them than
// CUs (64 rows, 6400 -> 1600 6.7 us, in 64 x 64 tiles 13.6; 1600 -> 6400, which has more,
// 13.6 and 7.2), else by prices fitted to times measured over 22 shapes and every tile
// (bf16 output; us, small, small in groups, square, square in groups, tall):
// 512 x 6400 x 1600 32, 19, 54, 39, 60; 1024 x 1600 x 1600 10.9, 14.5, 14.4, 13.4, 21.7;
// 2048 x 6400 x 1600 64, 68, 54, 39, 60; 4096 x 1600 x 1600 31, 44, 18.4, 26, 22; 4096 x
// 1600 x 6400 123, 173, 70, 92, 59.
constexpr TileCost kScaledTiles[] = {{muon::TILE_TALL, 256, 128, 6.0, 1.15, 2.3, 5.0, 512},
                                     {muon::TILE_SQUARE, 128, 128, 5.5, 0.8, 1.15, 3.0, 512},
                                     {muon::TILE_SQUARE_GROUPS, 128, 128, 6.0, 0.62, 1.0, 3.0, 256},
                                     {muon::TILE_SMALL, 64, 64, 4.5, 0.42, 0.55, 1.0, 512},
                                     {muon::TILE_SMALL_GROUPS, 64, 64, 6.0, 0.23, 0.33, 2.0, 256}};

struct ScaledPlan {
    muon::TileKind tile;
    int64_t tiles_m, tiles_n;
};
ScaledPlan scaled_plan(int64_t M, int64_t N, int64_t K) {
    if (M <= 16) return {muon::TILE_FEW16, 1, (N + 15) / 16};
    const int64_t blocks = (M + 31) / 32, few = blocks * ((N + 15) / 16);
    if (blocks == 1 || few <= 256) return {muon::TILE_FEW32, blocks, (N + 15) / 16};
    ScaledPlan best{};
    double least = 1e300;
    for (const TileCost& c : kScaledTiles) {
        const int64_t m = (M + c.rows - 1) / c.rows, n = (N + c.cols - 1) / c.cols;
        const double t = tile_price(c, (double)(m * n), (double)blocks_of(K));
        if (t >= least) continue;
        least = t;
        best = {c.kind, m, n};
    }
    return best;
}

// forward (X [tokens, in], W [out, in]) and grad input (dY [tokens, out], W [in, out])
muon_status run_scaled(const muon_linear* d, bool fwd, const muon_eight* a, const muon_eight* w,
                       const muon_epilogue* e, void* y, void* stream) {
    if (!d) return fail(MUON_E_INVALID_ARG, "null descriptor");
    if (d->dtype != MUON_TYPE_BF16 && d->dtype != MUON_TYPE_FP16)
        return fail(MUON_E_INVALID_ARG, "8-bit linear: dtype (of the output) must be bf16 or fp16");
    if (d->weight_layout != (fwd ? MUON_WEIGHT_OUT_IN : MUON_WEIGHT_IN_OUT))
        return fail(MUON_E_INVALID_ARG, fwd ? "8-bit linear forward: the weight is [out, in]"
                                            : "8-bit linear grad input: the weight is [in, out]");
    if (d->tokens < 0 || d->tokens >= kMaxRows) return fail(MUON_E_SHAPE, "8-bit linear: tokens must be in [0, 2^24)");
    if (d->in_features < 1 || d->in_features > kMaxCols || d->out_features < 1 || d->out_features > kMaxCols)
        return fail(MUON_E_SHAPE, "8-bit linear: features must be in [1, 2^21]");
    if (d->ld_w != 0 || (fwd ? d->ld_x : d->ld_y) != 0)
        return fail(MUON_E_LAYOUT, "8-bit linear: the operands' strides are their own, not the descriptor's");
    const int64_t M = d->tokens, N = fwd ? d->out_features : d->in_features, K = fwd ? d->in_features : d->out_features;
    const int64_t ld_out = fwd ? d->ld_y : d->ld_x;
    TRY(check_ld(ld_out, N, fwd ? "ld_y" : "ld_x"));
    const muon_epilogue none{};
    if (!e) e = &none;
    TRY(check_epilogue(fwd, N, *e));
    if (M == 0) return MUON_OK;
    if (!a || !w || !y) return fail(MUON_E_INVALID_ARG, "null tensor");
    if (!fwd && e->activation != MUON_ACT_NONE && !e->z)
        return fail(MUON_E_INVALID_ARG, "grad input: an activation needs its pre-activation z");
    TRY(check_eight(*a, K, false));
    TRY(check_eight(*w, K, true));
    if (((M + 127) / 128) * ((N + 127) / 128) >= (int64_t)1 << 21)
        return fail(MUON_E_SHAPE, "8-bit linear: output too large");
    const Outputs o = outputs_of(fwd, M, N, ld_out, *e, y);
    const Tensor &Y = o.y, &R = o.add, &Z = o.z;
    const Tensor Bi{e->bias, 1, N, N, 4};
    const Tensor A = data_of(*a, M, K), SA = scales_of(*a, blocks_of(K), M), W = data_of(*w, N, K),
                 SW = scales_of(*w, blocks_of(N), blocks_of(K));
    for (const Tensor& t : {Y, R, Z}) TRY(check_align(t.p, 2, "a 16-bit tensor"));
    TRY(check_align(e->bias, 4, "bias"));
    TRY(check_disjoint(Y, {A, SA, W, SW, Z, Bi}));
    TRY(check_add(Y, R));
    if (fwd) TRY(check_disjoint(Z, {A, SA, W, SW, R, Bi}));
    TRY(check_device());
    const ScaledPlan plan = scaled_plan(M, N, K);
    muon::ScaledArgs p{};
    muon::GemmArgs& g = p.g;
    g.a = a->data;
    g.b = w->data;
    g.ld_a = (int)A.ld;
    g.ld_b = (int)W.ld;
    g.M = (int)M;
    g.N = (int)N;
    g.K = (int)K;
    g.tiles_m = (int)plan.tiles_m;
    g.tiles_n = (int)plan.tiles_n;
    g.slices = (int)blocks_of(K);
    g.epi = epilogue_args(fwd, *e, o);
    p.scale_x = a->scale;
    p.scale_w = w->scale;
    return hip_status(muon::launch_scaled(p, plan.tile, d->dtype, a->format, static_cast<hipStream_t>(stream)),
                      "8-bit product kernel");
}

}  // namespace

extern "C" {

muon_status muon_rmsnorm_forward(const muon_rmsnorm* d, const void* x, const void* residual, const float* weight,
                                 void* sum, void* y, const muon_eight* q, float* rstd, void* stream) {
    return guarded([&]() -> muon_status {
        TRY(check_rms(d));
        if (!y && !q && d->rows > 0) return fail(MUON_E_INVALID_ARG, "rmsnorm: y and q are both null");
        if (d->rows == 0) return MUON_OK;
        if (!x || !rstd || !residual != !sum)
            return fail(MUON_E_INVALID_ARG, "null tensor (a residual and its sum come together)");
        const int size = size_of(d->dtype);
        const int64_t m = d->rows, n = d->cols;
        const Tensor X{x, m, n, stride_of(d->ld_x, n), size}, A{residual, m, n, stride_of(d->ld_add, n), size},
            S{sum, m, n, stride_of(d->ld_sum, n), size}, Y{y, m, n, stride_of(d->ld_y, n), size};
        const Tensor W{weight, 1, n, n, 4}, T{rstd, 1, m, m, 4};
        Tensor Q{}, QS{};
        if (q) {
            TRY(check_eight(*q, n, false));
            Q = data_of(*q, m, n);
            QS = scales_of(*q, blocks_of(n), m);
        }
        for (const Tensor& t : {X, A, S, Y}) TRY(check_align(t.p, size, "x, residual, sum or y"));
        for (const Tensor& t : {W, T}) TRY(check_align(t.p, 4, "a float32 tensor"));
        // a row's x and residual are read before its sum is stored, by the same lanes
        TRY(check_disjoint(S, {Y, W, T, Q, QS}));
        for (const Tensor& t : {X, A})
            if (!same_tensor(S, t)) TRY(check_disjoint(S, {t}));
        TRY(check_disjoint(Y, {X, A, W, T, Q, QS}));
        TRY(check_disjoint(T, {X, A, W, Q, QS}));
        TRY(check_disjoint(Q, {X, A, W, QS}));
        TRY(check_disjoint(QS, {X, A, W}));
        TRY(check_device());
        const muon::RmsForward k{x, residual, weight, sum, y, q ? q->data : nullptr, q ? q->scale : nullptr, rstd,
                                 (int)m, (int)n, (int)X.ld, (int)A.ld, (int)S.ld, (int)Y.ld, (int)Q.ld, d->eps};
        return hip_status(muon::launch_rms_forward(k, d->dtype, q ? q->format : muon::EIGHT_NONE,
                                                   static_cast<hipStream_t>(stream)),
                          "rms norm kernel");
    });
}

muon_status muon_rmsnorm_workspace_bytes(const muon_rmsnorm* d, size_t* out_bytes) {
    return guarded([&]() -> muon_status {
        if (!out_bytes) return fail(MUON_E_INVALID_ARG, "null out_bytes");
        TRY(check_rms(d));
        *out_bytes = rms_workspace(*d);
        return MUON_OK;
    });
}

muon_status muon_rmsnorm_backward(const muon_rmsnorm* d, const void* dy, const void* x, const float* weight,
                                  const float* rstd, const void* add, void* dx, float* dweight, int32_t accumulate,
                                  void* workspace, size_t ws_bytes, void* stream) {
    return guarded([&]() -> muon_status {
        TRY(check_rms(d));
        if (d->rows > 0 && (!dy || !x || !rstd || !dx)) return fail(MUON_E_INVALID_ARG, "null tensor");
        const int size = size_of(d->dtype);
        const int64_t m = d->rows, n = d->cols;
        const Tensor DY{dy, m, n, stride_of(d->ld_y, n), size}, X{x, m, n, stride_of(d->ld_x, n), size},
            DX{dx, m, n, stride_of(d->ld_dx, n), size}, R{add, m, n, stride_of(d->ld_add, n), size};
        const Tensor W{weight, 1, n, n, 4}, DW{dweight, 1, n, n, 4}, T{rstd, 1, m, m, 4};
        for (const Tensor& t : {DY, X, DX, R}) TRY(check_align(t.p, size, "dy, x, dx or add"));
        for (const Tensor& t : {W, DW, T}) TRY(check_align(t.p, 4, "a float32 tensor"));
        const size_t need = dweight ? rms_workspace(*d) : 0;
        TRY(check_workspace(workspace, ws_bytes, need));
        const Tensor K{workspace, 1, (int64_t)need, (int64_t)need, 1};
        TRY(check_disjoint(DX, {DY, X, W, DW, T, K}));
        TRY(check_add(DX, R));
        TRY(check_disjoint(DW, {DY, X, R, W, T, K}));
        TRY(check_disjoint(K, {DY, X, R, W, T}));
        if (m == 0 && (!dweight || accumulate)) return MUON_OK;
        TRY(check_device());
        const int blocks = muon::rms_backward_blocks(m, n, d->dtype);
        float* part = dweight ? static_cast<float*>(workspace) : nullptr;
        hipStream_t st = static_cast<hipStream_t>(stream);
        if (m > 0) {
            const muon::RmsBackward k{dy, x, weight, rstd, add, dx, part, (int)m, (int)n, (int)X.ld, (int)DY.ld,
                                      (int)DX.ld, (int)R.ld, blocks};
            TRY(hip_status(muon::launch_rms_backward(k, d->dtype, st), "rms norm gradient kernels"));
        }
        if (!dweight) return MUON_OK;
        const muon::RmsSums k{part, dweight, (int)n, blocks, accumulate != 0};
        return hip_status(muon::launch_rms_sums(k, st), "rms norm gradient sums");
    });
}

muon_status muon_quantize(int64_t rows, int64_t cols, int64_t ld_x, int32_t dtype, const void* x, const muon_eight* q,
                          void* stream) {
    return guarded([&]() -> muon_status {
        TRY(check_type(dtype));
        TRY(check_sizes(rows, cols));
        TRY(check_ld(ld_x, cols, "ld_x"));
        if (rows == 0) return MUON_OK;
        if (!x || !q) return fail(MUON_E_INVALID_ARG, "null tensor");
        TRY(check_eight(*q, cols, false));
        const int size = size_of(dtype);
        TRY(check_align(x, size, "x"));
        // four segments of 512 columns a workgroup of 256 threads, fewer than 2^32 a launch
        if (rows * ((cols + 511) / 512) > ((int64_t)1 << 26) - 4)
            return fail(MUON_E_SHAPE, "quantize: rows times cols too large");
        const Tensor X{x, rows, cols, stride_of(ld_x, cols), size}, Q = data_of(*q, rows, cols),
                     S = scales_of(*q, blocks_of(cols), rows);
        TRY(check_disjoint(Q, {X, S}));
        TRY(check_disjoint(S, {X}));
        TRY(check_device());
        const muon::Quantize k{x, q->data, q->scale, (int)rows, (int)cols, (int)X.ld, (int)Q.ld};
        return hip_status(muon::launch_quantize(k, dtype, q->format, static_cast<hipStream_t>(stream)),
                          "quantize kernel");
    });
}

muon_status muon_quantize_weight(int64_t rows, int64_t cols, int64_t ld_w, int32_t dtype, const void* w,
                                 const muon_eight* q, const muon_eight* q_t, void* stream) {
    return guarded([&]() -> muon_status {
        TRY(check_type(dtype));
        if (rows < 1 || rows > kMaxCols || cols < 1 || cols > kMaxCols)
            return fail(MUON_E_SHAPE, "quantize weight: rows and cols must be in [1, 2^21]");
        TRY(check_ld(ld_w, cols, "ld_w"));
        if (!w || (!q && !q_t)) return fail(MUON_E_INVALID_ARG, "null tensor");
        if (blocks_of(rows) * blocks_of(cols) >= (int64_t)1 << 23)
            return fail(MUON_E_SHAPE, "quantize weight: rows times cols too large");
        const int size = size_of(dtype);
        TRY(check_align(w, size, "w"));
        const Tensor W{w, rows, cols, stride_of(ld_w, cols), size};
        Tensor Q{}, S{}, QT{}, ST{};
        if (q) {
            TRY(check_eight(*q, cols, true));
            Q = data_of(*q, rows, cols);
            S = scales_of(*q, blocks_of(rows), blocks_of(cols));
        }
        if (q_t) {
            TRY(check_eight(*q_t, rows, true));
            QT = data_of(*q_t, cols, rows);
            ST = scales_of(*q_t, blocks_of(rows), blocks_of(cols));
        }
        TRY(check_disjoint(Q, {W, S, QT, ST}));
        TRY(check_disjoint(S, {W, QT, ST}));
        TRY(check_disjoint(QT, {W, ST}));
        TRY(check_disjoint(ST, {W}));
        TRY(check_device());
        const muon::QuantizeWeight k{w, q ? q->data : nullptr, q ? q->scale : nullptr, q_t ? q_t->data : nullptr,
                                     q_t ? q_t->scale : nullptr, (int)rows, (int)cols, (int)W.ld, (int)Q.ld,
                                     (int)QT.ld};
        return hip_status(muon::launch_quantize_weight(k, dtype, static_cast<hipStream_t>(stream)),
                          "quantize weight kernel");
    });
}

muon_status muon_linear_scaled_forward(const muon_linear* d, const muon_eight* x, const muon_eight* w,
                                       const muon_epilogue* e, void* y, void* stream) {
    return guarded([&]() { return run_scaled(d, true, x, w, e, y, stream); });
}

muon_status muon_linear_scaled_grad_input(const muon_linear* d, const muon_eight* dy, const muon_eight* w,
                                          const muon_epilogue* e, void* dx, void* stream) {
    return guarded([&]() { return run_scaled(d, false, dy, w, e, dx, stream); });
}

}  // extern "C"
