// Host side of the layer operators' C calls, shared by their entry points:
// errors and their text, exceptions kept inside, the device check, and the
// checks of tensors, strides and workspaces.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstring>
#include <exception>
#include <initializer_list>
#include <new>
#include <string>

#include "../../include/libmuon.h"
#include "layers.hpp"

namespace muon {
namespace checks {

// Keeps the message for muon_op_last_error; returns s.
muon_status fail(muon_status s, const char* msg) noexcept;

// No exception crosses the ABI.
template <typename F>
inline muon_status guarded(F&& body) noexcept {
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

inline muon_status hip_status(hipError_t e, const char* where) {
    if (e == hipSuccess) return MUON_OK;
    return fail(MUON_E_HIP, (std::string(where) + ": " + hipGetErrorString(e)).c_str());
}

// The current device must be a gfx950; asked once per device.
inline muon_status check_device() {
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

inline bool overlap(const Tensor& a, const Tensor& b) {
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

inline bool same_tensor(const Tensor& a, const Tensor& b) { return a.p == b.p && (a.ld == b.ld || a.rows <= 1); }

// `out` against inputs, other outputs and the workspace
inline muon_status check_disjoint(const Tensor& out, std::initializer_list<Tensor> others) {
    for (const Tensor& o : others)
        if (overlap(out, o)) return fail(MUON_E_INVALID_ARG, "an output overlaps another tensor or the workspace");
    return MUON_OK;
}

// ... and against the tensor added to it, which it may replace. (An operand at
// that address is check_disjoint's: others still read it while `out` is stored.)
inline muon_status check_add(const Tensor& out, const Tensor& add) {
    return same_tensor(out, add) ? MUON_OK : check_disjoint(out, {add});
}

inline muon_status check_align(const void* p, int size, const char* what) {
    if ((uintptr_t)p % (uintptr_t)size == 0) return MUON_OK;
    return fail(MUON_E_LAYOUT, (std::string(what) + " is not aligned to its element size").c_str());
}

inline muon_status check_ld(int64_t ld, int64_t cols, const char* what) {
    if (ld == 0 || (ld >= cols && ld <= kMaxCols)) return MUON_OK;
    return fail(MUON_E_LAYOUT, (std::string(what) + " must be 0 or from the row length to 2^21").c_str());
}

inline muon_status check_workspace(const void* ws, size_t have, size_t need) {
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

inline bool aligned16(const void* p, int64_t ld, int size) { return (uintptr_t)p % 16 == 0 && ld * size % 16 == 0; }
inline int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }
inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

inline int64_t stride_of(int64_t ld, int64_t cols) { return ld ? ld : cols; }

// A product's epilogue: forward (cols: out features) or input gradient (in features).
inline muon_status check_epilogue(bool fwd, int64_t cols, const muon_epilogue& e) {
    if (e.activation < MUON_ACT_NONE || e.activation > MUON_ACT_SILU)
        return fail(MUON_E_INVALID_ARG, "epilogue: unknown activation");
    if (e.reserved != 0) return fail(MUON_E_INVALID_ARG, "epilogue: reserved must be 0");
    if (!fwd && e.bias) return fail(MUON_E_INVALID_ARG, "grad input: takes no bias");
    TRY(check_ld(e.ld_add, cols, "ld_add"));
    return check_ld(e.ld_z, cols, "ld_z");
}

// What it reads and writes.
struct Outputs {
    Tensor y, add, z;
};

inline Outputs outputs_of(bool fwd, int64_t rows, int64_t cols, int64_t ld, const muon_epilogue& e, const void* y) {
    Outputs o{{y, rows, cols, stride_of(ld, cols), 2}, {e.add, rows, cols, stride_of(e.ld_add, cols), 2}, {}};
    // the way back reads z only for an activation
    if (fwd || e.activation != MUON_ACT_NONE) o.z = {e.z, rows, cols, stride_of(e.ld_z, cols), 2};
    return o;
}

inline Epilogue epilogue_args(bool fwd, const muon_epilogue& e, const Outputs& o) {
    Epilogue E{};
    E.mode = fwd ? EPI_FORWARD : EPI_GRAD_INPUT;
    E.act = (int8_t)e.activation;
    E.bias = e.bias;
    E.add = e.add;
    E.z = e.z && o.z.p ? e.z : nullptr;
    E.y = const_cast<void*>(o.y.p);
    E.ld_add = (int)o.add.ld;
    E.ld_z = (int)o.z.ld;
    E.ld_y = (int)o.y.ld;
    return E;
}

// What a product takes on one kind of tile, in microseconds: all but its slices, a
// slice's worth of a workgroup alone on its CU and of a CU that holds all it can, and
// each further round of workgroups.
struct TileCost {
    TileKind kind;
    int rows, cols;
    double fixed, alone, beside, next;
    int places;  // workgroups that the chip holds: 512, or 256 for those that fill their CU
};

inline double tile_price(const TileCost& c, double tiles, double slices) {
    const double full = std::floor(tiles / c.places), rest = tiles - full * c.places;
    const double more = rest > 256 ? c.alone + (c.beside - c.alone) * (rest - 256) / 256 : rest > 0 ? c.alone : 0;
    return c.fixed + c.next * std::ceil(tiles / c.places - 1) + slices * (full * c.beside + more);
}

}  // namespace checks
}  // namespace muon
