// The linear layers of a mixture of experts on gfx950: rows lie grouped by expert,
// expert e's from offsets[e] to offsets[e + 1], each group with a weight of its own.
// The tiles and their products are the linear layer's (gemm_device.hpp); what is
// here is which tile a workgroup takes.
//
//  * The offsets are read on the device, so that no launch waits for the router and
//    a captured graph serves any of its choices. The grid is what the rows and
//    experts can need at most; a workgroup finds its tile by a prefix sum over the
//    experts' tile counts (64 experts a turn, a lane each), and one past the last
//    tile ends at once.
//  * Offsets are taken within [0, rows] and as ascending, whatever they hold: no
//    read or write leaves the tensors.
//  * Forward and input gradient: the tiles of all experts are one list, which each
//    XCD takes a contiguous run of, so that an expert's weight is read into few L2s.
//    Few rows an expert go through the kernel for few rows, whose list is of blocks
//    of 16 or 32 rows.
//  * Weight gradient: an expert's rows are the sum's index; an expert without rows
//    gets zeros (or keeps what it has, when accumulating). Few tiles of long sums are
//    cut into pieces of the experts' rows, whose sums a second kernel adds in order
//    (32768 rows of 2 experts, 2048 -> 800: 270 us whole in the best of the tiles, 167
//    in 4 pieces; 128 -> 128 101 and 20 in 32).
//
// Measured, 32768 rows of 16 experts, 1600 -> 1600, bf16, inputs that no cache holds:
// forward 181 to 191 us, by the box (the linear layer on one weight of that size 182, a library's 209; with
// inputs in cache 158), weight gradient added to what is there 235 to 246 (stored 215, of equal
// groups 205; the linear layer's one gradient 190): 16 times the float32 output and the
// ends of 16 sums. The matrix unit is busy 46% and 38% of the clocks. Two rows of two
// experts, 1600 -> 6400, 9.7 us a call: 41 MB of weights and one launch.
// Rows off 16-byte borders, or of features that are no multiple of 8, go through registers
// in 64 x 64 tiles whatever the size. Equal groups, the same inputs each call, forward, input and
// weight gradient: 1600 -> 1600 186, 167 and 202 us, 1600 -> 1601 365, 445 and 404,
// 1601 -> 1601 465, 467 and 497; two rows of 1600 -> 6400 11 and 10, of 1601 -> 6401 16
// and 47.

#include "gemm_device.hpp"

namespace muon {

namespace {

struct Group {
    int begin, end;
};
__device__ __forceinline__ Group group_of(const int32_t* __restrict__ offsets, int rows, int e) {
    int a = offsets[e], b = offsets[e + 1];
    a = a < 0 ? 0 : a < rows ? a : rows;
    b = b < a ? a : b < rows ? b : rows;
    return {a, b};
}

template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_plus(int v) {
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
// The sum of the lanes up to and with this one.
__device__ __forceinline__ int wave_prefix(int v) {
    v = dpp_plus<0x111, 0xf>(v);  // row_shr 1, 2, 4, 8
    v = dpp_plus<0x112, 0xf>(v);
    v = dpp_plus<0x114, 0xf>(v);
    v = dpp_plus<0x118, 0xf>(v);
    v = dpp_plus<0x142, 0xa>(v);  // row_bcast 15 into rows 1, 3
    v = dpp_plus<0x143, 0xc>(v);  // row_bcast 31 into rows 2, 3
    return v;
}

// A block of TM rows of one expert.
struct Block {
    int expert, begin, end, ti;
};

// The list of the experts' blocks of TM rows: their number, and the at(total)-th of
// them. False: there is none for this workgroup.
template <int TM, typename F>
__device__ __forceinline__ bool find_block(const GroupedArgs& p, Block& out, F&& at) {
    const int lane = threadIdx.x & 63;
    // the first 64 experts' counts stay for the second turn, when there are no more
    int total = 0, run = 0;
    Group q{0, 0};
    for (int e0 = 0; e0 < p.experts; e0 += 64) {
        const int e = e0 + lane;
        q = e < p.experts ? group_of(p.offsets, p.rows, e) : Group{0, 0};
        run = wave_prefix((q.end - q.begin + TM - 1) / TM);
        // offsets that repeat rows may count more blocks than there are workgroups for, and
        // their sum would pass 32 bits
        total += __builtin_amdgcn_readlane(run, 63);
        total = total < p.tiles_m ? total : p.tiles_m;
    }
    int t = at(total);
    if (t < 0) return false;
    for (int e0 = 0; e0 < p.experts; e0 += 64) {
        const int e = e0 + lane;
        if (p.experts > 64) {
            q = e < p.experts ? group_of(p.offsets, p.rows, e) : Group{0, 0};
            run = wave_prefix((q.end - q.begin + TM - 1) / TM);
        }
        const int here = __builtin_amdgcn_readlane(run, 63);
        if (t < here) {
            const int l = __builtin_ctzll(__ballot(run > t));
            out.begin = __builtin_amdgcn_readlane(q.begin, l);
            out.end = __builtin_amdgcn_readlane(q.end, l);
            out.expert = e0 + l;
            out.ti = t - (__builtin_amdgcn_readlane(run, l) - (out.end - out.begin + TM - 1) / TM);
            return true;
        }
        t -= here;
    }
    return false;
}

// The expert with the r-th most rows (of equal ones the first), and its rows; of more
// than 64 experts, which are not ranked, the r-th.
__device__ __forceinline__ int ranked(const GroupedArgs& p, int r, int& begin, int& end) {
    const int lane = threadIdx.x & 63;
    int e = r;
    if (p.experts <= 64) {
        const Group q = lane < p.experts ? group_of(p.offsets, p.rows, lane) : Group{0, -1};
        const int n = q.end - q.begin;
        int before = 0;
        for (int k = 0; k < p.experts; ++k) {
            const int m = __builtin_amdgcn_readlane(n, k);
            before += m > n || (m == n && k < lane) ? 1 : 0;
        }
        e = __builtin_ctzll(__ballot(before == r));
        begin = __builtin_amdgcn_readlane(q.begin, e);
        end = __builtin_amdgcn_readlane(q.end, e);
    } else {
        const Group q = group_of(p.offsets, p.rows, e);
        begin = __builtin_amdgcn_readfirstlane(q.begin);
        end = __builtin_amdgcn_readfirstlane(q.end);
    }
    return e;
}

// The epilogue of one expert's rows, whose first is row `begin`.
template <typename T>
__device__ __forceinline__ Epilogue epilogue_of(const Epilogue& e, const Block& b, int n) {
    Epilogue r = e;
    auto down = [&](const void* t, int ld) { return static_cast<const T*>(t) + (int64_t)b.begin * ld; };
    r.y = const_cast<T*>(down(e.y, e.ld_y));
    if (e.z) r.z = const_cast<T*>(down(e.z, e.ld_z));
    if (e.add) r.add = down(e.add, e.ld_add);
    if (e.bias) r.bias = e.bias + (int64_t)b.expert * n;
    return r;
}

// STAGES: buffers of the square tiles' rings. Two for 128 x 128, so that two
// workgroups fit a CU, four for 64 x 64. KG: groups of waves that share the sum.
template <typename T, int TM, int TN, int STAGES, int KG, bool BKC, bool RAW, int MODE>
__global__ __launch_bounds__(256 * KG) __attribute__((amdgpu_waves_per_eu(2))) void k_grouped(
    const GroupedArgs p) {
    __shared__ __attribute__((aligned(16))) char smem[GemmShape<T, TM, TN, true, BKC, RAW, STAGES, KG>::SMEM];
    Block b;
    int tj = 0;
    const bool some = find_block<TM>(p, b, [&](int total) {
        GemmArgs order{};
        order.tiles_m = total;
        order.tiles_n = p.tiles_n;
        const int tiles = total * p.tiles_n;
        if ((int)blockIdx.x >= tiles) return -1;
        int ti;
        tile_at(order, per_xcd(blockIdx.x, tiles), ti, tj);
        return ti;
    });
    if (!some) return;
    GemmArgs g{};
    g.a = static_cast<const T*>(p.a) + (int64_t)b.begin * p.ld_a;
    g.b = static_cast<const T*>(p.b) + b.expert * p.stride_w;
    g.ld_a = p.ld_a;
    g.ld_b = p.ld_b;
    g.M = b.end - b.begin;
    g.N = p.N;
    g.K = p.K;
    g.slices = (p.K + BK - 1) / BK;
    g.epi = epilogue_of<T>(p.epi, b, p.N);
    gemm_tile<T, TM, TN, true, BKC, 0, RAW, STAGES, KG, MODE>(g, smem, b.ti, tj, -1, 0, g.slices);
}

template <typename T, bool BKC, int MT>
__global__ __launch_bounds__(512) void k_grouped_few(const GroupedArgs p) {
    using Shape = SkinnyShape<BKC, MT>;
    __shared__ __attribute__((aligned(16))) char smem[Shape::SMEM];
    Block b;
    int j0 = 0;
    const bool some = find_block<16 * MT>(p, b, [&](int total) {
        const int tiles = total * p.tiles_n;
        if ((int)blockIdx.x >= tiles) return -1;
        const int l = per_xcd(blockIdx.x, tiles);
        j0 = l % p.tiles_n * Shape::TNS;
        return l / p.tiles_n;
    });
    if (!some) return;
    b.begin += b.ti * 16 * MT;
    SkinnyArgs g{};
    g.a = static_cast<const T*>(p.a) + (int64_t)b.begin * p.ld_a;
    g.b = static_cast<const T*>(p.b) + b.expert * p.stride_w;
    g.ld_a = p.ld_a;
    g.ld_b = p.ld_b;
    g.M = b.end - b.begin < 16 * MT ? b.end - b.begin : 16 * MT;
    g.N = p.N;
    g.K = p.K;
    g.slices = (p.K + BK - 1) / BK;
    g.epi = epilogue_of<T>(p.epi, b, p.N);
    skinny_tile<T, BKC, MT>(g, smem, j0);
}

// Rows of each piece of an expert's (the last may be shorter): whole slices, and a
// number that the kernel and the join both come to.
__device__ __forceinline__ int piece_rows(int rows, int pieces) {
    return ((rows + BK - 1) / BK + pieces - 1) / pieces * BK;
}

template <typename T, int TM, int TN, int STAGES, int SUM, bool RAW>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) void k_grouped_weight(const GroupedArgs p) {
    __shared__ __attribute__((aligned(16))) char smem[GemmShape<T, TM, TN, false, false, RAW, STAGES>::SMEM];
    // Each expert's tiles are shared by all XCDs, a contiguous run each, and the experts
    // come by their rows, most first: their sums are unlike long, and one XCD with the
    // longest, or a long one begun last, would keep the others waiting.
    const int per = p.tiles_m * p.tiles_n, run = (per + 7) >> 3;
    const int r = blockIdx.x / (8 * run), i = blockIdx.x - r * 8 * run;
    const int l = ((i + r) & 7) * run + (i >> 3);
    if (l >= per) return;
    int begin, end;
    const int turn = r / p.pieces, piece = r - turn * p.pieces;
    const int e = ranked(p, turn, begin, end);
    GemmArgs g{};
    g.epi = p.epi;
    if (p.pieces > 1) {
        const int rows = piece_rows(end - begin, p.pieces);
        begin += piece * rows;
        end = end - begin < rows ? end : begin + rows;
        if (begin >= end) return;  // no such piece, which the join knows
        const int64_t at = (int64_t)piece * p.experts + e;
        g.epi.y = p.part + at * p.M * p.ld_part;
        if (SUM) g.sums = p.part_sums + at * (SUM == 1 ? p.N : p.M);
    } else {
        g.epi.y = static_cast<float*>(p.epi.y) + e * p.stride_w;
        if (SUM) g.sums = p.sums + (int64_t)e * (SUM == 1 ? p.N : p.M);
    }
    g.a = static_cast<const T*>(p.a) + (int64_t)begin * p.ld_a;
    g.b = static_cast<const T*>(p.b) + (int64_t)begin * p.ld_b;
    g.ld_a = p.ld_a;
    g.ld_b = p.ld_b;
    g.M = p.M;
    g.N = p.N;
    g.K = end - begin;
    g.tiles_m = p.tiles_m;
    g.tiles_n = p.tiles_n;
    g.slices = (g.K + BK - 1) / BK;
    int ti, tj;
    tile_at(g, l, ti, tj);
    gemm_tile<T, TM, TN, false, false, SUM, RAW, STAGES, 1, EPI_GRAD_WEIGHT>(g, smem, ti, tj, -1, 0, g.slices);
}

// One expert's gradient (blockIdx.y) from its pieces, an element a thread, and behind it
// the bias's: the loads of 8 pieces are on the way at once, and small gradients still
// make enough workgroups.
__global__ __launch_bounds__(256) void k_grouped_join(const GroupedArgs p, const int sums) {
    const int e = blockIdx.y;
    const uint32_t total = (uint32_t)p.M * (uint32_t)p.N, i = blockIdx.x * 256u + threadIdx.x;
    if (i >= total + (uint32_t)sums) return;
    const Group q = group_of(p.offsets, p.rows, e);
    const int rows = q.end - q.begin, tall = piece_rows(rows, p.pieces);
    const int live = rows ? (rows + tall - 1) / tall : 0;
    const float* from;
    float* to;
    int64_t step;
    if (i < total) {
        const uint32_t m = i / (uint32_t)p.N, n = i - m * (uint32_t)p.N;
        step = (int64_t)p.experts * p.M * p.ld_part;
        from = p.part + ((int64_t)e * p.M + m) * p.ld_part + n;
        to = static_cast<float*>(p.epi.y) + e * p.stride_w + (int64_t)m * p.epi.ld_y + n;
    } else {
        step = (int64_t)p.experts * sums;
        from = p.part_sums + (int64_t)e * sums + (i - total);
        to = p.sums + (int64_t)e * sums + (i - total);
    }
    const float old = p.epi.accumulate ? *to : 0.f;
    float s = 0.f;
#pragma unroll 8
    for (int t = 0; t < live; ++t) s += from[t * step];
    *to = p.epi.accumulate ? old + s : s;
}

template <typename T, int TM, int TN, int STAGES, int KG, bool RAW, int MODE>
void rows_tile(const GroupedArgs& p, bool b_kc, unsigned grid, hipStream_t st) {
    if (b_kc)
        k_grouped<T, TM, TN, STAGES, KG, true, RAW, MODE><<<grid, 256 * KG, 0, st>>>(p);
    else
        k_grouped<T, TM, TN, STAGES, KG, false, RAW, MODE><<<grid, 256 * KG, 0, st>>>(p);
}
template <typename T, int MODE>
void rows_mode(const GroupedArgs& p, TileKind tile, bool raw, bool b_kc, unsigned grid, hipStream_t st) {
    if (raw)
        rows_tile<T, 64, 64, 2, 1, true, MODE>(p, b_kc, grid, st);
    else if (tile == TILE_TALL)
        rows_tile<T, 256, 128, 2, 1, false, MODE>(p, b_kc, grid, st);
    else if (tile == TILE_SQUARE)
        rows_tile<T, 128, 128, 2, 1, false, MODE>(p, b_kc, grid, st);
    else if (tile == TILE_SQUARE_GROUPS)
        rows_tile<T, 128, 128, 2, 2, false, MODE>(p, b_kc, grid, st);
    else if (tile == TILE_SMALL)
        rows_tile<T, 64, 64, 4, 1, false, MODE>(p, b_kc, grid, st);
    else
        rows_tile<T, 64, 64, 4, 2, false, MODE>(p, b_kc, grid, st);
}
template <typename T, int MT>
void few_tile(const GroupedArgs& p, bool b_kc, unsigned grid, hipStream_t st) {
    if (b_kc)
        k_grouped_few<T, true, MT><<<grid, 512, 0, st>>>(p);
    else
        k_grouped_few<T, false, MT><<<grid, 512, 0, st>>>(p);
}
template <typename T>
hipError_t rows_t(const GroupedArgs& p, TileKind tile, bool raw, bool b_kc, unsigned grid, hipStream_t st) {
    if (tile == TILE_FEW16)
        few_tile<T, 1>(p, b_kc, grid, st);
    else if (tile == TILE_FEW32)
        few_tile<T, 2>(p, b_kc, grid, st);
    else if (p.epi.mode == EPI_FORWARD)
        rows_mode<T, EPI_FORWARD>(p, tile, raw, b_kc, grid, st);
    else
        rows_mode<T, EPI_GRAD_INPUT>(p, tile, raw, b_kc, grid, st);
    return hipGetLastError();
}

template <typename T, int TM, int TN, int STAGES, bool RAW>
void weight_tile(const GroupedArgs& p, int sum, unsigned grid, hipStream_t st) {
    if (sum == 0)
        k_grouped_weight<T, TM, TN, STAGES, 0, RAW><<<grid, 256, 0, st>>>(p);
    else if (sum == 1)
        k_grouped_weight<T, TM, TN, STAGES, 1, RAW><<<grid, 256, 0, st>>>(p);
    else
        k_grouped_weight<T, TM, TN, STAGES, 2, RAW><<<grid, 256, 0, st>>>(p);
}
template <typename T>
hipError_t weight_t(const GroupedArgs& p, TileKind tile, bool raw, int sum, unsigned grid, hipStream_t st) {
    if (raw)
        weight_tile<T, 64, 64, 2, true>(p, sum, grid, st);
    else if (tile == TILE_TALL)
        weight_tile<T, 256, 128, 2, false>(p, sum, grid, st);
    else if (tile == TILE_SQUARE)
        weight_tile<T, 128, 128, 2, false>(p, sum, grid, st);
    else
        weight_tile<T, 64, 64, 4, false>(p, sum, grid, st);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped(const GroupedArgs& p, TileKind tile, bool raw, bool b_kc, int dtype, unsigned grid,
                          hipStream_t st) {
    return dtype == 0 ? rows_t<bf16>(p, tile, raw, b_kc, grid, st) : rows_t<f16>(p, tile, raw, b_kc, grid, st);
}

hipError_t launch_grouped_join(const GroupedArgs& p, int sums, hipStream_t st) {
    const dim3 grid((unsigned)(((int64_t)p.M * p.N + sums + 255) / 256), (unsigned)p.experts);
    k_grouped_join<<<grid, 256, 0, st>>>(p, sums);
    return hipGetLastError();
}

hipError_t launch_grouped_weight(const GroupedArgs& p, TileKind tile, bool raw, int dtype, int sum, unsigned grid,
                                 hipStream_t st) {
    return dtype == 0 ? weight_t<bf16>(p, tile, raw, sum, grid, st) : weight_t<f16>(p, tile, raw, sum, grid, st);
}

}  // namespace muon
