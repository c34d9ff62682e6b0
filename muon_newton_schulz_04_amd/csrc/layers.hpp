// Internal interface of the layer operators: the linear layer (matrix product
// with bias, activation and residual in its epilogue, and its gradients) and
// layer norm. Plain data shared by the host entry points and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {

// What the epilogue of a product does with its fp32 accumulators.
enum EpiMode {
    EPI_FORWARD = 0,     // y = act(v + bias) + add; z = v + bias if asked
    EPI_GRAD_INPUT = 1,  // y = v act'(z) + add
    EPI_GRAD_WEIGHT = 2  // w (+)= v, float32
};

// (The arguments of kernels are kept small: a launch costs the host 2.7 us with
// 8 bytes of them and 3.7 us with 216.)
struct Epilogue {
    const float* bias;  // [N] or null
    const void* add;    // [M, N] of the 16-bit type, or null
    void* z;            // forward: written if not null; grad input: read if act != none
    void* y;            // 16-bit output, or float32 for the weight gradient
    int32_t ld_add, ld_z, ld_y;
    int8_t mode, act;
    int8_t accumulate;  // weight gradient: add to what is there
};

// C[M, N] = sum_k A(m, k) B(k, n) over 16-bit operands, each stored with its k
// index contiguous ([M, K], [N, K]) or its other index contiguous ([K, M],
// [K, N]). Every operand's rows start 16-byte aligned and hold a multiple of
// 8 elements (others are packed first, zero-padded to the next multiple), or,
// for a raw product (64 x 64 tiles), start anywhere and hold 8 or more.
struct GemmArgs {
    const void* a;
    const void* b;
    int32_t ld_a, ld_b;  // elements
    int32_t M, N, K;
    int32_t tiles_m, tiles_n;
    // K is `slices` slices of kGemmSlice. The first `whole` tiles (a multiple
    // of 8, or all) are one workgroup each, which finishes them; the others
    // are `splits` pieces of `per` slices each, whose sums meet in the
    // workspace: piece p belongs to tile whole + p % (tiles - whole).
    int32_t slices, whole, splits, per;
    float* partial;   // piece p: [tile_m][tile_n] at index p
    float* sums;      // bias gradient, or null
    float* sum_part;  // its pieces: 256 floats at index p
    Epilogue epi;
};

constexpr int kGemmSlice = 64;  // K per pipeline stage
constexpr int kSkinnyRows = 32;

struct GemmPlan {
    int tile_m, tile_n;  // 256 x 128, 128 x 128 or 64 x 64; 0: the kernel for up to kSkinnyRows rows of A
    int tiles_m, tiles_n, slices, whole, splits, per;
};

// sum: the bias gradient is the sums over k of neither (0), B's (1) or A's (2) rows
hipError_t launch_gemm(const GemmArgs& g, int tile_m, bool raw, bool a_kc, bool b_kc, int dtype, int sum,
                       hipStream_t st);
hipError_t launch_gemm_join(const GemmArgs& g, int tile_m, int dtype, int sum, hipStream_t st);
// M <= kSkinnyRows, A k-contiguous
struct SkinnyArgs {
    const void* a;
    const void* b;
    int32_t ld_a, ld_b;
    int32_t M, N, K, slices;
    Epilogue epi;
};
hipError_t launch_skinny(const SkinnyArgs& g, bool b_kc, int dtype, hipStream_t st);
// dst [rows, 8 chunks] <- src [rows, cols] of 16-bit elements with row stride
// ld, zero-padded; n (1 or 2) of them in a launch
struct PackArgs {
    const void* src;
    void* dst;
    int32_t ld, rows, cols, chunks;
};
hipError_t launch_pack(const PackArgs* p, int n, hipStream_t st);

struct NormForward {
    const void* x;
    const float* weight;
    const float* bias;
    void* y;
    float* mean;
    float* rstd;
    int32_t rows, cols, ld_x, ld_y;
    float eps;
};

struct NormBackward {
    const void* dy;
    const void* x;
    const float* weight;
    const float* mean;
    const float* rstd;
    const void* add;
    void* dx;
    float* part;  // [blocks][2][cols], or null: no column sums
    int32_t rows, cols, ld_x, ld_y, ld_dx, ld_r, blocks;
};

// what the column sums of NormBackward's workgroups become
struct NormSums {
    const float* part;
    float* dweight;
    float* dbias;
    int32_t cols, blocks, accumulate;
};

int norm_backward_blocks(int64_t rows, int64_t cols, int dtype);
hipError_t launch_norm_forward(const NormForward& n, int dtype, hipStream_t st);
hipError_t launch_norm_backward(const NormBackward& n, int dtype, hipStream_t st);
hipError_t launch_norm_sums(const NormSums& n, hipStream_t st);

}  // namespace muon
