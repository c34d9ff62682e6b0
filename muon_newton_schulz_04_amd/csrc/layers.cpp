// C ABI of the layer operators (include/libmuon.h): argument checks, operand
// packing and workspace layout, the choice of tile and K split, and the
// launches on the caller's stream.

#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstring>
#include <exception>
#include <new>
#include <string>

#include "../../include/libmuon.h"
#include "layers.hpp"

namespace {

thread_local std::string g_error;

muon_status fail(muon_status s, const char* msg) noexcept {
    try {
        g_error = msg;
    } catch (...) {
    }
    return s;
}

// No exception crosses the ABI.
template <typename F>
muon_status guarded(F&& body) noexcept {
    try {
        return body();
    } catch (const std::bad_alloc&) {
        return fail(MUON_E_HOST, "out of host memory");
    } catch (const std::exception& ex) {
        return fail(MUON_E_HOST, ex.what());
    } catch (...) {
        return fail(MUON_E_HOST, "unknown exception");
    }
}

muon_status hip_status(hipError_t e, const char* where) {
    if (e == hipSuccess) return MUON_OK;
    return fail(MUON_E_HIP, (std::string(where) + ": " + hipGetErrorString(e)).c_str());
}

// The current device must be a gfx950; asked once per device.
muon_status check_device() {
    constexpr int kMax = 64;
    static std::atomic<int> known[kMax];
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) {
        (void)hipGetLastError();
        return fail(MUON_E_NO_DEVICE, "no HIP device");
    }
    if (dev < kMax && known[dev].load(std::memory_order_relaxed) == 1) return MUON_OK;
    hipDeviceProp_t prop;
    hipError_t e = hipGetDeviceProperties(&prop, dev);
    if (e != hipSuccess) return hip_status(e, "hipGetDeviceProperties");
    if (std::strncmp(prop.gcnArchName, "gfx950", 6) != 0)
        return fail(MUON_E_NO_DEVICE, (std::string("device is ") + prop.gcnArchName + ", need gfx950").c_str());
    if (dev < kMax) known[dev].store(1, std::memory_order_relaxed);
    return MUON_OK;
}

constexpr int64_t kMaxRows = (int64_t)1 << 24;
constexpr int64_t kMaxCols = (int64_t)1 << 21;

// A [rows, cols] tensor with a row stride, and the bytes from its first to
// its last element.
struct Tensor {
    const void* p;
    int64_t rows, cols, ld;
    int size;
    int64_t bytes() const { return rows == 0 ? 0 : ((rows - 1) * ld + cols) * size; }
};

bool overlap(const Tensor& a, const Tensor& b) {
    const int64_t na = a.bytes(), nb = b.bytes();
    if (!a.p || !b.p || na == 0 || nb == 0) return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    if (x >= y + (uintptr_t)nb || y >= x + (uintptr_t)na) return false;
    // column ranges of one buffer's rows may lie side by side
    const uintptr_t pitch = (uintptr_t)(a.ld * a.size), ca = (uintptr_t)(a.cols * a.size),
                    cb = (uintptr_t)(b.cols * b.size);
    if (pitch != (uintptr_t)(b.ld * b.size)) return true;
    const uintptr_t d = x >= y ? (x - y) % pitch : (pitch - (y - x) % pitch) % pitch;  // a's column in b's rows
    return !(d >= cb && d + ca <= pitch);
}

bool same_tensor(const Tensor& a, const Tensor& b) { return a.p == b.p && (a.ld == b.ld || a.rows <= 1); }

// `out` against inputs, other outputs and the workspace
muon_status check_disjoint(const Tensor& out, std::initializer_list<Tensor> others) {
    for (const Tensor& o : others)
        if (overlap(out, o)) return fail(MUON_E_INVALID_ARG, "an output overlaps another tensor or the workspace");
    return MUON_OK;
}

// ... and against the tensor added to it, which it may replace. (An operand at
// that address is check_disjoint's: others still read it while `out` is stored.)
muon_status check_add(const Tensor& out, const Tensor& add) {
    return same_tensor(out, add) ? MUON_OK : check_disjoint(out, {add});
}

muon_status check_align(const void* p, int size, const char* what) {
    if ((uintptr_t)p % (uintptr_t)size == 0) return MUON_OK;
    return fail(MUON_E_LAYOUT, (std::string(what) + " is not aligned to its element size").c_str());
}

muon_status check_ld(int64_t ld, int64_t cols, const char* what) {
    if (ld == 0 || (ld >= cols && ld <= kMaxCols)) return MUON_OK;
    return fail(MUON_E_LAYOUT, (std::string(what) + " must be 0 or from the row length to 2^21").c_str());
}

muon_status check_workspace(const void* ws, size_t have, size_t need) {
    if (need == 0) return MUON_OK;
    if (!ws) return fail(MUON_E_WORKSPACE, "null workspace");
    if ((uintptr_t)ws % 256 != 0) return fail(MUON_E_WORKSPACE, "workspace not 256-byte aligned");
    if (have < need)
        return fail(MUON_E_WORKSPACE, ("workspace too small: need " + std::to_string(need) + " bytes").c_str());
    return MUON_OK;
}

#define TRY(expr)                          \
    do {                                   \
        const muon_status s_ = (expr);     \
        if (s_ != MUON_OK) return s_;      \
    } while (0)

bool aligned16(const void* p, int64_t ld, int size) { return (uintptr_t)p % 16 == 0 && ld * size % 16 == 0; }
int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

muon_status check_linear(const muon_linear* d) {
    if (!d) return fail(MUON_E_INVALID_ARG, "null descriptor");
    if (d->dtype != MUON_TYPE_BF16 && d->dtype != MUON_TYPE_FP16)
        return fail(MUON_E_INVALID_ARG, "linear: dtype must be bf16 or fp16");
    if (d->weight_layout != MUON_WEIGHT_IN_OUT && d->weight_layout != MUON_WEIGHT_OUT_IN)
        return fail(MUON_E_INVALID_ARG, "linear: bad weight_layout");
    if (d->tokens < 0 || d->tokens >= kMaxRows) return fail(MUON_E_SHAPE, "linear: tokens must be in [0, 2^24)");
    if (d->in_features < 1 || d->in_features > kMaxCols || d->out_features < 1 || d->out_features > kMaxCols)
        return fail(MUON_E_SHAPE, "linear: features must be in [1, 2^21]");
    TRY(check_ld(d->ld_x, d->in_features, "ld_x"));
    TRY(check_ld(d->ld_w, d->weight_layout == MUON_WEIGHT_IN_OUT ? d->out_features : d->in_features, "ld_w"));
    TRY(check_ld(d->ld_y, d->out_features, "ld_y"));
    return MUON_OK;
}

Tensor tensor_x(const muon_linear& d, const void* p) {
    return {p, d.tokens, d.in_features, d.ld_x ? d.ld_x : d.in_features, 2};
}
Tensor tensor_y(const muon_linear& d, const void* p) {
    return {p, d.tokens, d.out_features, d.ld_y ? d.ld_y : d.out_features, 2};
}
Tensor tensor_w(const muon_linear& d, const void* p, int size) {
    const bool io = d.weight_layout == MUON_WEIGHT_IN_OUT;
    const int64_t r = io ? d.in_features : d.out_features, c = io ? d.out_features : d.in_features;
    return {p, r, c, d.ld_w ? d.ld_w : c, size};
}

// How an M x N x K product is cut: the tile, how many tiles run whole, and in
// how many K pieces the others go. Each candidate is priced in clocks (2.4 GHz)
// with constants fitted to times measured over 26 shapes, three tiles and up to
// 24 pieces; the choice was within 5% of the best at all but two. In us, tall
// (256 x 128), square (128) and small (64) tiles: 4096 x 1600 x 1600 32.5, 36.6,
// -; 2048 x 1600 x 1600 31.2, 19.3, 23.4; 1024 x 1600 x 1600 29, 19.7, 12.9;
// 2051 x 768 x 768 20.9, 13.7, 9.0; the 6400 x 1600 weight gradient over 8192
// tokens 154 with pieces beside whole tiles, 192 without.
muon::GemmPlan choose_plan(int64_t M, int64_t N, int64_t K) {
    int64_t slices = (K + muon::kGemmSlice - 1) / muon::kGemmSlice;
    if (slices < 1) slices = 1;
    // per tile: a slice of a workgroup alone on its CU and beside a second one
    // (a 128 x 128 one fills its CU: the second runs after it), what a
    // workgroup does besides and another round of workgroups, and the chip
    struct Tile {
        int m, n;
        double alone, beside, fixed, next, chip;
        int64_t round;
    };
    static const Tile tiles_of[] = {{256, 128, 2200, 3700, 23000, 5000, 8.0, 512},
                                    {128, 128, 1140, 2280, 18000, 12000, 5.5, 256},
                                    {64, 64, 600, 900, 9500, 9000, 2.0, 512}};
    muon::GemmPlan best{};
    double best_t = 1e300;
    for (const Tile& T : tiles_of) {
        const int64_t tiles_m = (M + T.m - 1) / T.m, tiles_n = (N + T.n - 1) / T.n, tiles = tiles_m * tiles_n;
        const double chip = (double)tiles * (double)slices * T.chip;
        auto rounds = [&](int64_t wgs, double per) {
            const int64_t rest = wgs % 512;
            return T.fixed + T.next * (double)((wgs - 1) / T.round) +
                   per * ((double)(wgs / 512) * T.beside + (rest == 0 ? 0.0 : rest > 256 ? T.beside : T.alone));
        };
        auto consider = [&](double t, int64_t whole, int64_t splits, int64_t per) {
            if (t < chip) t = chip;
            if (whole < tiles)
                t += 8.0 * (double)((tiles - whole) * splits) * (double)((M < T.m ? M : T.m) * T.n) / 1700.0 + 11000.0;
            if (t >= best_t) return;
            best_t = t;
            best = {T.m, T.n, (int)tiles_m, (int)tiles_n, (int)slices, (int)whole, (int)splits, (int)per};
        };
        consider(rounds(tiles, (double)slices), tiles, 1, slices);
        for (int64_t s = 2; s <= 64 && s <= slices; ++s) {
            const int64_t per = (slices + s - 1) / s;
            if ((slices + per - 1) / per != s) continue;  // every piece has work
            if (tiles * s <= 1024) consider(rounds(tiles * s, (double)per), 0, s, per);
            // one tall tile a CU and the rest of a round in pieces beside them
            const int64_t rest = tiles % 512 - 256, n = (rest * s + 255) / 256;
            if (T.m == 256 && rest > 0 && n * per <= slices)
                consider(T.fixed + (double)(tiles / 512 * slices + n * per) * T.beside +
                             (double)(slices - n * per) * T.alone,
                         tiles - rest, s, per);
        }
    }
    return best;
}

// One product: operands, where packed copies and partial sums go, and the plan.
struct Product {
    int64_t M, N, K;
    Tensor a, b;
    bool a_kc, b_kc;  // k is the contiguous index
    bool pack_a, pack_b;
    bool raw;  // the small tiles read rows as they are
    muon::GemmPlan plan;
    size_t off_a, off_b, off_part, off_sums, bytes;
};

bool needs_pack(const Tensor& t) { return t.rows > 0 && (!aligned16(t.p, t.ld, 2) || t.cols % 8 != 0); }

muon_status plan_product(const muon_linear& d, int op, const void* pa, const void* pb, bool dbias, Product* P) {
    const bool io = d.weight_layout == MUON_WEIGHT_IN_OUT;
    if (op == MUON_LINEAR_FORWARD) {
        *P = {d.tokens, d.out_features, d.in_features, tensor_x(d, pa), tensor_w(d, pb, 2), true, !io};
    } else if (op == MUON_LINEAR_GRAD_INPUT) {
        *P = {d.tokens, d.in_features, d.out_features, tensor_y(d, pa), tensor_w(d, pb, 2), true, io};
    } else {
        const Tensor x = tensor_x(d, pa), dy = tensor_y(d, pb);
        if (io)
            *P = {d.in_features, d.out_features, d.tokens, x, dy, false, false};
        else
            *P = {d.out_features, d.in_features, d.tokens, dy, x, false, false};
    }
    P->pack_a = needs_pack(P->a);
    P->pack_b = needs_pack(P->b);
    // launches hold fewer than 2^32 threads
    if (((P->M + 127) / 128) * ((P->N + 127) / 128) >= (int64_t)1 << 21)
        return fail(MUON_E_SHAPE, "linear: output too large");
    // Copies to aligned rows are a launch of their own, 3 to 6 us of the chip
    // and 3 of the host, which only the larger tiles' loads need (us, copied and
    // as they are: 60 x 333 x 257 14.3, 8.3; 999 x 1001 x 777 14.8, 10.6; 1024 x
    // 1601 x 1599 26.7, 20.7; weight gradient 4099 x 1001 x 1003 31.5, 29.0; with
    // 128 x 128 tiles, that of 2048 x 1601 x 1599 31.5, 37.6). So few tokens on
    // such rows leave their own kernel, too (1 x 1001 x 777 13.0, 9.6; 24 x 6401 x
    // 1599 29.6, 14.6; 8 x 1600 x 50257 127, 32).
    const bool few = op != MUON_LINEAR_GRAD_WEIGHT && P->M <= muon::kSkinnyRows;
    const bool can = (P->pack_a || P->pack_b) && P->a.cols >= 8 && P->b.cols >= 8;
    if (!few || can) P->plan = choose_plan(P->M, P->N, P->K);
    P->raw = can && P->plan.tile_m == 64;
    if (few && !P->raw)
        P->plan = {0, 0, 0, 0, (int)((P->K + muon::kGemmSlice - 1) / muon::kGemmSlice), 0, 0, 0};
    if (P->raw) P->pack_a = P->pack_b = false;
    size_t o = 0;
    P->off_a = o;
    if (P->pack_a) o = up256(o + (size_t)P->a.rows * up8(P->a.cols) * 2);
    P->off_b = o;
    if (P->pack_b) o = up256(o + (size_t)P->b.rows * up8(P->b.cols) * 2);
    const muon::GemmPlan& G = P->plan;
    const size_t pieces = (size_t)(G.tiles_m * G.tiles_n - G.whole) * (size_t)G.splits;
    P->off_part = o;
    o = up256(o + pieces * (size_t)(G.tile_m * G.tile_n) * 4);
    P->off_sums = o;
    if (dbias) o = up256(o + pieces * 256 * 4);
    P->bytes = o;
    return MUON_OK;
}

// sums (bias gradient) and sum: see GemmArgs and launch_gemm
muon_status run_product(Product& P, int dtype, muon::Epilogue& E, float* sums, int sum, char* ws, hipStream_t st) {
    muon::PackArgs packs[2];
    int n = 0;
    for (int k = 0; k < 2; ++k) {
        Tensor& t = k ? P.b : P.a;
        if (!(k ? P.pack_b : P.pack_a)) continue;
        char* dst = ws + (k ? P.off_b : P.off_a);
        packs[n++] = {t.p, dst, (int)t.ld, (int)t.rows, (int)t.cols, (int)(up8(t.cols) / 8)};
        t.p = dst;
        t.ld = up8(t.cols);
    }
    if (n) TRY(hip_status(muon::launch_pack(packs, n, st), "pack kernel"));
    const muon::GemmPlan& G = P.plan;
    if (G.tile_m == 0) {
        const muon::SkinnyArgs k{P.a.p, P.b.p, (int)P.a.ld, (int)P.b.ld, (int)P.M, (int)P.N, (int)P.K, G.slices, E};
        return hip_status(muon::launch_skinny(k, P.b_kc, dtype, st), "product kernel");
    }
    muon::GemmArgs g{};
    g.a = P.a.p;
    g.b = P.b.p;
    g.ld_a = (int)P.a.ld;
    g.ld_b = (int)P.b.ld;
    g.M = (int)P.M;
    g.N = (int)P.N;
    g.K = (int)P.K;
    g.tiles_m = G.tiles_m;
    g.tiles_n = G.tiles_n;
    g.slices = G.slices;
    g.whole = G.whole;
    g.splits = G.splits;
    g.per = G.per;
    g.partial = reinterpret_cast<float*>(ws + P.off_part);
    g.sums = sums;
    g.sum_part = reinterpret_cast<float*>(ws + P.off_sums);
    g.epi = E;
    TRY(hip_status(muon::launch_gemm(g, G.tile_m, P.raw, P.a_kc, P.b_kc, dtype, sum, st), "product kernel"));
    if (G.whole < G.tiles_m * G.tiles_n) TRY(hip_status(muon::launch_gemm_join(g, G.tile_m, dtype, sum, st), "join kernel"));
    return MUON_OK;
}

muon_status check_epilogue(const muon_linear& d, int op, const muon_epilogue& e) {
    const bool fwd = op == MUON_LINEAR_FORWARD;
    const int64_t cols = fwd ? d.out_features : d.in_features;
    if (e.activation < MUON_ACT_NONE || e.activation > MUON_ACT_SILU)
        return fail(MUON_E_INVALID_ARG, "epilogue: unknown activation");
    if (e.reserved != 0) return fail(MUON_E_INVALID_ARG, "epilogue: reserved must be 0");
    if (!fwd && e.bias) return fail(MUON_E_INVALID_ARG, "grad input: takes no bias");
    TRY(check_ld(e.ld_add, cols, "ld_add"));
    return check_ld(e.ld_z, cols, "ld_z");
}

// What a product's epilogue reads and writes (e NULL: only the output).
struct Outputs {
    Tensor y, add, z;
};

Outputs outputs_of(const muon_linear& d, int op, const muon_epilogue* e, const void* y) {
    const bool fwd = op == MUON_LINEAR_FORWARD;
    const int64_t cols = fwd ? d.out_features : d.in_features;
    Outputs o{fwd ? tensor_y(d, y) : tensor_x(d, y), {}, {}};
    if (!e) return o;
    o.add = {e->add, d.tokens, cols, e->ld_add ? e->ld_add : cols, 2};
    // the way back reads z only for an activation
    if (fwd || e->activation != MUON_ACT_NONE) o.z = {e->z, d.tokens, cols, e->ld_z ? e->ld_z : cols, 2};
    return o;
}

// forward and grad input
muon_status run_layer(const muon_linear* d, int op, const void* a, const void* w, const muon_epilogue* e, void* y,
                      void* ws, size_t ws_bytes, void* stream) {
    TRY(check_linear(d));
    const bool fwd = op == MUON_LINEAR_FORWARD;
    muon_epilogue none{};
    if (!e) e = &none;
    TRY(check_epilogue(*d, op, *e));
    if (d->tokens == 0) return MUON_OK;
    if (!a || !w || !y) return fail(MUON_E_INVALID_ARG, "null tensor");
    if (!fwd && e->activation != MUON_ACT_NONE && !e->z)
        return fail(MUON_E_INVALID_ARG, "grad input: an activation needs its pre-activation z");
    const Tensor A = fwd ? tensor_x(*d, a) : tensor_y(*d, a), W = tensor_w(*d, w, 2);
    const Outputs o = outputs_of(*d, op, e, y);
    const Tensor &Y = o.y, &R = o.add, &Z = o.z;
    const Tensor Bi{e->bias, 1, d->out_features, d->out_features, 4};
    for (const Tensor& t : {A, W, Y, R, Z}) TRY(check_align(t.p, 2, "a 16-bit tensor"));
    TRY(check_align(e->bias, 4, "bias"));
    Product P;
    TRY(plan_product(*d, op, a, w, false, &P));
    TRY(check_workspace(ws, ws_bytes, P.bytes));
    const Tensor S{ws, 1, (int64_t)P.bytes, (int64_t)P.bytes, 1};
    TRY(check_disjoint(Y, {A, W, Z, Bi, S}));
    TRY(check_add(Y, R));
    if (fwd) TRY(check_disjoint(Z, {A, W, R, Bi, S}));
    for (const Tensor& t : {A, W, R, Z, Bi})
        if (overlap(S, t)) return fail(MUON_E_INVALID_ARG, "the workspace overlaps a tensor");
    TRY(check_device());
    muon::Epilogue E{};
    E.mode = fwd ? muon::EPI_FORWARD : muon::EPI_GRAD_INPUT;
    E.act = (int8_t)e->activation;
    E.bias = e->bias;
    E.add = e->add;
    E.z = e->z && Z.p ? e->z : nullptr;
    E.y = y;
    E.ld_add = (int)R.ld;
    E.ld_z = (int)Z.ld;
    E.ld_y = (int)Y.ld;
    return run_product(P, d->dtype, E, nullptr, 0, static_cast<char*>(ws), static_cast<hipStream_t>(stream));
}

muon_status check_norm(const muon_layernorm* d) {
    if (!d) return fail(MUON_E_INVALID_ARG, "null descriptor");
    if (d->dtype < MUON_TYPE_BF16 || d->dtype > MUON_TYPE_FP32)
        return fail(MUON_E_INVALID_ARG, "layernorm: dtype must be bf16, fp16 or fp32");
    if (d->rows < 0 || d->rows >= kMaxRows) return fail(MUON_E_SHAPE, "layernorm: rows must be in [0, 2^24)");
    if (d->cols < 1 || d->cols > kMaxCols) return fail(MUON_E_SHAPE, "layernorm: cols must be in [1, 2^21]");
    if (!(d->eps >= 0.f) || !std::isfinite(d->eps))
        return fail(MUON_E_INVALID_ARG, "layernorm: eps must be finite and not negative");
    TRY(check_ld(d->ld_x, d->cols, "ld_x"));
    TRY(check_ld(d->ld_y, d->cols, "ld_y"));
    TRY(check_ld(d->ld_dx, d->cols, "ld_dx"));
    TRY(check_ld(d->ld_add, d->cols, "ld_add"));
    return MUON_OK;
}

int64_t stride_of(int64_t ld, int64_t cols) { return ld ? ld : cols; }

size_t norm_workspace(const muon_layernorm& d) {
    return up256((size_t)muon::norm_backward_blocks(d.rows, d.cols, d.dtype) * 2 * (size_t)d.cols * 4);
}

}  // namespace

extern "C" {

const char* muon_op_last_error(void) { return g_error.c_str(); }

muon_status muon_linear_workspace_bytes(const muon_linear* d, int32_t op, const void* a, const void* b,
                                        size_t* out_bytes) {
    return guarded([&]() -> muon_status {
        if (!out_bytes) return fail(MUON_E_INVALID_ARG, "null out_bytes");
        TRY(check_linear(d));
        if (op < MUON_LINEAR_FORWARD || op > MUON_LINEAR_GRAD_WEIGHT)
            return fail(MUON_E_INVALID_ARG, "unknown linear operation");
        *out_bytes = 0;
        if (d->tokens == 0 && op != MUON_LINEAR_GRAD_WEIGHT) return MUON_OK;
        Product P;
        TRY(plan_product(*d, op, a, b, op == MUON_LINEAR_GRAD_WEIGHT, &P));
        *out_bytes = P.bytes;
        return MUON_OK;
    });
}

muon_status muon_linear_forward(const muon_linear* d, const void* x, const void* w, const muon_epilogue* e, void* y,
                                void* workspace, size_t ws_bytes, void* stream) {
    return guarded([&]() { return run_layer(d, MUON_LINEAR_FORWARD, x, w, e, y, workspace, ws_bytes, stream); });
}

muon_status muon_linear_grad_input(const muon_linear* d, const void* dy, const void* w, const muon_epilogue* e,
                                   void* dx, void* workspace, size_t ws_bytes, void* stream) {
    return guarded([&]() { return run_layer(d, MUON_LINEAR_GRAD_INPUT, dy, w, e, dx, workspace, ws_bytes, stream); });
}

muon_status muon_linear_grad_weight(const muon_linear* d, const void* x, const void* dy, float* dw, float* dbias,
                                    int32_t accumulate, void* workspace, size_t ws_bytes, void* stream) {
    return guarded([&]() -> muon_status {
        TRY(check_linear(d));
        if (!dw || (d->tokens > 0 && (!x || !dy))) return fail(MUON_E_INVALID_ARG, "null tensor");
        const Tensor X = tensor_x(*d, x), Y = tensor_y(*d, dy), W = tensor_w(*d, dw, 4);
        const Tensor Bi{dbias, 1, d->out_features, d->out_features, 4};
        TRY(check_align(x, 2, "x"));
        TRY(check_align(dy, 2, "dy"));
        TRY(check_align(dw, 4, "dw"));
        TRY(check_align(dbias, 4, "dbias"));
        Product P;
        TRY(plan_product(*d, MUON_LINEAR_GRAD_WEIGHT, x, dy, dbias != nullptr, &P));
        TRY(check_workspace(workspace, ws_bytes, P.bytes));
        const Tensor S{workspace, 1, (int64_t)P.bytes, (int64_t)P.bytes, 1};
        TRY(check_disjoint(W, {X, Y, Bi, S}));
        TRY(check_disjoint(Bi, {X, Y, S}));
        if (overlap(S, X) || overlap(S, Y)) return fail(MUON_E_INVALID_ARG, "the workspace overlaps a tensor");
        TRY(check_device());
        char* ws = static_cast<char*>(workspace);
        hipStream_t st = static_cast<hipStream_t>(stream);
        muon::Epilogue E{};
        E.mode = muon::EPI_GRAD_WEIGHT;
        E.y = dw;
        E.ld_y = (int)W.ld;
        E.accumulate = accumulate != 0;
        // dy is the second operand of an [in, out] gradient, else the first
        const int sum = !dbias ? 0 : d->weight_layout == MUON_WEIGHT_IN_OUT ? 1 : 2;
        return run_product(P, d->dtype, E, dbias, sum, ws, st);
    });
}

muon_status muon_layernorm_forward(const muon_layernorm* d, const void* x, const float* weight, const float* bias,
                                   void* y, float* mean, float* rstd, void* stream) {
    return guarded([&]() -> muon_status {
        TRY(check_norm(d));
        if (d->rows == 0) return MUON_OK;
        if (!x || !y || !mean || !rstd) return fail(MUON_E_INVALID_ARG, "null tensor");
        const int size = d->dtype == MUON_TYPE_FP32 ? 4 : 2;
        const Tensor X{x, d->rows, d->cols, stride_of(d->ld_x, d->cols), size},
            Y{y, d->rows, d->cols, stride_of(d->ld_y, d->cols), size};
        const Tensor W{weight, 1, d->cols, d->cols, 4}, Bi{bias, 1, d->cols, d->cols, 4};
        const Tensor M{mean, 1, d->rows, d->rows, 4}, S{rstd, 1, d->rows, d->rows, 4};
        for (const Tensor& t : {X, Y}) TRY(check_align(t.p, size, "x or y"));
        for (const Tensor& t : {W, Bi, M, S}) TRY(check_align(t.p, 4, "a float32 tensor"));
        TRY(check_disjoint(Y, {X, W, Bi, M, S}));
        TRY(check_disjoint(M, {X, W, Bi, S}));
        TRY(check_disjoint(S, {X, W, Bi}));
        TRY(check_device());
        const muon::NormForward n{x,  weight, bias, y, mean, rstd, (int)d->rows, (int)d->cols, (int)X.ld, (int)Y.ld,
                                  d->eps};
        return hip_status(muon::launch_norm_forward(n, d->dtype, static_cast<hipStream_t>(stream)),
                          "layer norm kernel");
    });
}

muon_status muon_layernorm_workspace_bytes(const muon_layernorm* d, size_t* out_bytes) {
    return guarded([&]() -> muon_status {
        if (!out_bytes) return fail(MUON_E_INVALID_ARG, "null out_bytes");
        TRY(check_norm(d));
        *out_bytes = norm_workspace(*d);
        return MUON_OK;
    });
}

muon_status muon_layernorm_backward(const muon_layernorm* d, const void* dy, const void* x, const float* weight,
                                    const float* mean, const float* rstd, const void* add, void* dx, float* dweight,
                                    float* dbias, int32_t accumulate, void* workspace, size_t ws_bytes, void* stream) {
    return guarded([&]() -> muon_status {
        TRY(check_norm(d));
        if (d->rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return fail(MUON_E_INVALID_ARG, "null tensor");
        const int size = d->dtype == MUON_TYPE_FP32 ? 4 : 2;
        const Tensor DY{dy, d->rows, d->cols, stride_of(d->ld_y, d->cols), size},
            X{x, d->rows, d->cols, stride_of(d->ld_x, d->cols), size},
            DX{dx, d->rows, d->cols, stride_of(d->ld_dx, d->cols), size},
            R{add, d->rows, d->cols, stride_of(d->ld_add, d->cols), size};
        const Tensor W{weight, 1, d->cols, d->cols, 4}, DW{dweight, 1, d->cols, d->cols, 4},
            DB{dbias, 1, d->cols, d->cols, 4};
        const Tensor M{mean, 1, d->rows, d->rows, 4}, S{rstd, 1, d->rows, d->rows, 4};
        for (const Tensor& t : {DY, X, DX, R}) TRY(check_align(t.p, size, "dy, x, dx or add"));
        for (const Tensor& t : {W, DW, DB, M, S}) TRY(check_align(t.p, 4, "a float32 tensor"));
        const bool sums = dweight || dbias;
        const size_t need = sums ? norm_workspace(*d) : 0;
        TRY(check_workspace(workspace, ws_bytes, need));
        const Tensor K{workspace, 1, (int64_t)need, (int64_t)need, 1};
        TRY(check_disjoint(DX, {DY, X, W, DW, DB, M, S, K}));
        TRY(check_add(DX, R));
        TRY(check_disjoint(DW, {DY, X, R, W, DB, M, S, K}));
        TRY(check_disjoint(DB, {DY, X, R, W, M, S, K}));
        TRY(check_disjoint(K, {DY, X, R, W, M, S}));
        if (d->rows == 0 && (!sums || accumulate)) return MUON_OK;
        TRY(check_device());
        const int blocks = muon::norm_backward_blocks(d->rows, d->cols, d->dtype);
        float* part = sums ? static_cast<float*>(workspace) : nullptr;
        hipStream_t st = static_cast<hipStream_t>(stream);
        if (d->rows > 0) {
            const muon::NormBackward n{dy, x, weight, mean, rstd, add, dx, part, (int)d->rows, (int)d->cols, (int)X.ld,
                                       (int)DY.ld, (int)DX.ld, (int)R.ld, blocks};
            TRY(hip_status(muon::launch_norm_backward(n, d->dtype, st), "layer norm gradient kernels"));
        }
        if (!sums) return MUON_OK;
        const muon::NormSums k{part, dweight, dbias, (int)d->cols, blocks, accumulate != 0};
        return hip_status(muon::launch_norm_sums(k, st), "layer norm gradient sums");
    });
}

}  // extern "C"
