// The linear layer's products on gfx950: C[M, N] = sum_k A(m, k) B(k, n) over
// bf16 or fp16 operands with fp32 accumulation, and an epilogue on the fp32
// sums that is rounded once (see Epilogue).
//
//  * One kernel for the three products of a layer (forward, input gradient,
//    weight gradient, in either weight layout): each operand may have its k
//    index contiguous (AKC, BKC) or its other index; the latter are read from
//    LDS with the transposing read.
//  * A workgroup of 4 waves computes a 256 x 128, 128 x 128 or 64 x 64 tile, each
//    wave a quarter of it, in blocks of 32x32x16 matrix instructions. K goes by
//    in slices of 64 that direct-to-LDS loads bring in, 128 bytes of a row at
//    a time where k is contiguous: L2 serves whole lines, and slices of 32
//    took two requests for each (16384 x 1600 x 6400: 356 us, against 319).
//    Loads past K, past a piece's end or past the matrix go out with an offset
//    beyond the buffer resource's range and land as zeros, so the loop has no
//    tail and reads nothing outside the operands.
//  * The tall tile keeps two slices of A and one of B in LDS (80 KB) and the B
//    fragments of its slice in registers, so that two workgroups share a CU:
//    one multiplies while the other is in its prologue or epilogue (one 256 x
//    256 workgroup per CU: 593 us with the epilogue of c_fc, against 335).
//    Bound by LDS and power: both workgroups' fragment reads and incoming
//    slices are 140 bytes a clock at the matrix peak, of the 128 that LDS
//    gives, and the matrix unit is busy 72% of the clocks, at 1.5 GHz (8192^3:
//    1.26 PFLOP/s on random numbers, 1.76 on zeros). A longer way for B's loads,
//    loads and reads spread over the matrix instructions, and wave priorities
//    changed nothing.
//  * The square tiles keep a ring of four slices of both operands (128 and 64
//    KB): they are for products that do not fill the chip, whose time is the
//    latency of a few loads.
//  * Tiles that a round of the chip leaves over go in K pieces beside whole
//    ones: each piece leaves fp32 sums in the workspace and a second kernel adds
//    them in order and does the epilogue (the same bits every run).
//  * Rows off 16-byte borders go through registers for the small tile
//    (RawOperand) and are packed first for the others.
//  * Up to 32 rows of A, unless through registers, have a kernel of their own
//    (k_skinny).

#include "gemm_device.hpp"

namespace muon {

namespace {

template <typename T, int TM, int TN, bool AKC, bool BKC, int SUM, bool RAW>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(TM == 128 ? 1 : 2, TM == 128 ? 1 : 2))) void
k_gemm(const GemmArgs g) {
    __shared__ __attribute__((aligned(16))) char smem[GemmShape<T, TM, TN, AKC, BKC, RAW>::SMEM];
    // a whole tile, or piece number `piece` (-1: none): all split tiles' first
    // K runs come before their second ones, so that pieces running at the same
    // time share operand panels
    const int b = blockIdx.x;
    int tile, piece = -1, s0 = 0, nk = g.slices;
    if (b < g.whole) {
        tile = per_xcd(b, g.whole);
    } else {
        const int split = g.tiles_m * g.tiles_n - g.whole;
        piece = per_xcd(b - g.whole, gridDim.x - g.whole);
        tile = g.whole + piece % split;
        s0 = piece / split * g.per;
        nk = g.slices - s0 < g.per ? g.slices - s0 : g.per;
    }
    int ti, tj;
    tile_at(g, tile, ti, tj);
    gemm_tile<T, TM, TN, AKC, BKC, SUM, RAW>(g, smem, ti, tj, piece, s0, nk);
}

// The pieces of each split tile added in order, then the epilogue: GS
// neighbouring lanes share a chunk of 8 outputs, each adding a run of pieces.
template <typename T, int TM, int TN, int GS, int SUM>
__global__ __launch_bounds__(256) void k_gemm_join(const GemmArgs g) {
    constexpr int PER = 256 / GS;                 // chunks a block takes
    constexpr int BLOCKS = TM * (TN / 8) / PER;   // blocks per tile
    const int t = blockIdx.x / BLOCKS, sub = blockIdx.x % BLOCKS;
    const int split = g.tiles_m * g.tiles_n - g.whole;
    int ti, tj;
    tile_at(g, g.whole + t, ti, tj);
    if (SUM != 0 && sub == 0 && (SUM == 1 ? ti == tj % g.tiles_m : tj == ti % g.tiles_n)) {
        const int at = threadIdx.x, n = (SUM == 1 ? tj * TN : ti * TM) + at;
        if (at < (SUM == 1 ? TN : TM) && n < (SUM == 1 ? g.N : g.M)) {
            float v = 0.f;
            for (int s = 0; s < g.splits; ++s) v += g.sum_part[((int64_t)s * split + t) * 256 + at];
            g.sums[n] = g.epi.accumulate ? g.sums[n] + v : v;
        }
    }
    const int id = sub * PER + threadIdx.x / GS, part = threadIdx.x % GS;
    const int64_t row = (int64_t)ti * TM + id / (TN / 8);
    const int col = tj * TN + id % (TN / 8) * 8;
    if (row >= g.M || col >= g.N) return;  // all GS lanes of a chunk alike
    const int run = (g.splits + GS - 1) / GS;
    const int sa = part * run, sb = sa + run < g.splits ? sa + run : g.splits;
    const float* p = g.partial + (int64_t)t * (TM * TN) + id * 8;
    const int64_t stride = (int64_t)split * (TM * TN);
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = sa; s < sb; ++s) {
        float u[8];
        load8(p + s * stride, 8, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += u[e];
    }
    if constexpr (GS > 1) {
#pragma unroll
        for (int off = 1; off < GS; off <<= 1)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += __shfl_xor(v[e], off, 64);
        if (part) return;
    }
    const int left = g.N - col;
    float bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (g.epi.bias) load8(g.epi.bias + col, left, bias);
    u32x4 in = {0, 0, 0, 0}, in2 = in;
    if (left >= 8) {
        in = first8<T>(g.epi, row, col, LaneAt());
        if (has_second(g.epi)) in2 = second8<T>(g.epi, row, col, LaneAt());
    }
    finish8<T>(g.epi, row, col, LaneAt(), left, v, bias, in, in2);
}

// B's columns over the XCDs as the tiles are (per_xcd).
template <typename T, bool BKC, int MT>
__global__ __launch_bounds__(512) void k_skinny(const SkinnyArgs g) {
    __shared__ __attribute__((aligned(16))) char smem[SkinnyShape<BKC, MT>::SMEM];
    skinny_tile<T, BKC, MT>(g, smem, per_xcd(blockIdx.x, gridDim.x) * SkinnyShape<BKC, MT>::TNS);
}

// Rows of any alignment and length to 16-byte aligned, zero-padded ones: a
// wave a row, a 16-byte chunk a lane; one operand or both in a launch.
__global__ __launch_bounds__(256) void k_pack(const PackArgs a, const PackArgs b) {
    const PackArgs& p = blockIdx.y ? b : a;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= p.rows) return;
    const uint16_t* s = static_cast<const uint16_t*>(p.src) + row * p.ld;
    u32x4* d = static_cast<u32x4*>(p.dst) + row * p.chunks;
    for (int k = threadIdx.x & 63; k < p.chunks; k += 64) {
        const int c = k * 8;
        if (c + 8 <= p.cols) {
            d[k] = *reinterpret_cast<const u32x4_mem*>(s + c);
        } else {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = c + e < p.cols ? s[c + e] : 0u;
            d[k] = u32x4{w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16};
        }
    }
}

template <typename T, int TM, int TN, bool RAW>
hipError_t gemm_t(const GemmArgs& g, bool a_kc, bool b_kc, int sum, hipStream_t st) {
    const int wgs = g.whole + (g.tiles_m * g.tiles_n - g.whole) * g.splits;
    if (a_kc && b_kc)
        k_gemm<T, TM, TN, true, true, 0, RAW><<<wgs, 256, 0, st>>>(g);
    else if (a_kc)
        k_gemm<T, TM, TN, true, false, 0, RAW><<<wgs, 256, 0, st>>>(g);
    else if (sum == 0)
        k_gemm<T, TM, TN, false, false, 0, RAW><<<wgs, 256, 0, st>>>(g);
    else if (sum == 1)
        k_gemm<T, TM, TN, false, false, 1, RAW><<<wgs, 256, 0, st>>>(g);
    else
        k_gemm<T, TM, TN, false, false, 2, RAW><<<wgs, 256, 0, st>>>(g);
    return hipGetLastError();
}

template <typename T, int MT>
hipError_t skinny_t(const SkinnyArgs& g, bool b_kc, hipStream_t st) {
    if (b_kc)
        k_skinny<T, true, MT><<<(g.N + 15) / 16, 512, 0, st>>>(g);
    else
        k_skinny<T, false, MT><<<(g.N + 31) / 32, 512, 0, st>>>(g);
    return hipGetLastError();
}

template <typename T, int TM, int TN, int GS>
void join_gs(const GemmArgs& g, int sum, hipStream_t st) {
    const int grid = (g.tiles_m * g.tiles_n - g.whole) * (TM * (TN / 8) * GS / 256);
    if (sum == 0)
        k_gemm_join<T, TM, TN, GS, 0><<<grid, 256, 0, st>>>(g);
    else if (sum == 1)
        k_gemm_join<T, TM, TN, GS, 1><<<grid, 256, 0, st>>>(g);
    else
        k_gemm_join<T, TM, TN, GS, 2><<<grid, 256, 0, st>>>(g);
}
template <typename T, int TM, int TN>
hipError_t join_t(const GemmArgs& g, int sum, hipStream_t st) {
    // four lanes a chunk for eight pieces or more
    if (g.splits >= 8)
        join_gs<T, TM, TN, 4>(g, sum, st);
    else
        join_gs<T, TM, TN, 1>(g, sum, st);
    return hipGetLastError();
}

template <typename T>
hipError_t gemm_tile(const GemmArgs& g, int tile_m, bool raw, bool a_kc, bool b_kc, int sum, hipStream_t st) {
    return tile_m == 256   ? gemm_t<T, 256, 128, false>(g, a_kc, b_kc, sum, st)
           : tile_m == 128 ? gemm_t<T, 128, 128, false>(g, a_kc, b_kc, sum, st)
           : raw           ? gemm_t<T, 64, 64, true>(g, a_kc, b_kc, sum, st)
                           : gemm_t<T, 64, 64, false>(g, a_kc, b_kc, sum, st);
}
template <typename T>
hipError_t join_tile(const GemmArgs& g, int tile_m, int sum, hipStream_t st) {
    return tile_m == 256   ? join_t<T, 256, 128>(g, sum, st)
           : tile_m == 128 ? join_t<T, 128, 128>(g, sum, st)
                           : join_t<T, 64, 64>(g, sum, st);
}

}  // namespace

hipError_t launch_gemm(const GemmArgs& g, int tile_m, bool raw, bool a_kc, bool b_kc, int dtype, int sum,
                       hipStream_t st) {
    return dtype == 0 ? gemm_tile<bf16>(g, tile_m, raw, a_kc, b_kc, sum, st)
                      : gemm_tile<f16>(g, tile_m, raw, a_kc, b_kc, sum, st);
}

hipError_t launch_gemm_join(const GemmArgs& g, int tile_m, int dtype, int sum, hipStream_t st) {
    return dtype == 0 ? join_tile<bf16>(g, tile_m, sum, st) : join_tile<f16>(g, tile_m, sum, st);
}

hipError_t launch_skinny(const SkinnyArgs& g, bool b_kc, int dtype, hipStream_t st) {
    if (dtype == 0) return g.M <= 16 ? skinny_t<bf16, 1>(g, b_kc, st) : skinny_t<bf16, 2>(g, b_kc, st);
    return g.M <= 16 ? skinny_t<f16, 1>(g, b_kc, st) : skinny_t<f16, 2>(g, b_kc, st);
}

hipError_t launch_pack(const PackArgs* p, int n, hipStream_t st) {
    const int rows = p[0].rows > p[n - 1].rows ? p[0].rows : p[n - 1].rows;
    if (rows == 0) return hipSuccess;
    k_pack<<<dim3(((unsigned)rows + 3) / 4, (unsigned)n), 256, 0, st>>>(p[0], p[n - 1]);
    return hipGetLastError();
}

}  // namespace muon
