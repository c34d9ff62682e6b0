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
//    gets zeros (or keeps what it has, when accumulating).

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
__global__ __launch_bounds__(256 * KG) __attribute__((amdgpu_waves_per_eu(KG > 2 ? KG : 2))) void k_grouped(
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

template <typename T, int TM, int TN, int STAGES, int KG, int SUM, bool RAW>
__global__ __launch_bounds__(256 * KG) __attribute__((amdgpu_waves_per_eu(KG > 2 ? KG : 2))) void k_grouped_weight(
    const GroupedArgs p) {
    __shared__ __attribute__((aligned(16))) char smem[GemmShape<T, TM, TN, false, false, RAW, STAGES, KG>::SMEM];
    // Each expert's tiles are shared by all XCDs, a contiguous run each, and the experts
    // come by their rows, most first: their sums are unlike long, and one XCD with the
    // longest, or a long one begun last, would keep the others waiting.
    const int per = p.tiles_m * p.tiles_n, run = (per + 7) >> 3;
    const int r = blockIdx.x / (8 * run), i = blockIdx.x - r * 8 * run;
    const int l = ((i + r) & 7) * run + (i >> 3);
    if (l >= per) return;
    int begin, end;
    const int e = ranked(p, r, begin, end);
    GemmArgs g{};
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
    g.epi = p.epi;
    g.epi.y = static_cast<float*>(p.epi.y) + e * p.stride_w;
    if (SUM) g.sums = p.sums + (int64_t)e * (SUM == 1 ? p.N : p.M);
    int ti, tj;
    tile_at(g, l, ti, tj);
    gemm_tile<T, TM, TN, false, false, SUM, RAW, STAGES, KG, EPI_GRAD_WEIGHT>(g, smem, ti, tj, -1, 0, g.slices);
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

template <typename T, int TM, int TN, int STAGES, int KG, bool RAW>
void weight_tile(const GroupedArgs& p, int sum, unsigned grid, hipStream_t st) {
    if (sum == 0)
        k_grouped_weight<T, TM, TN, STAGES, KG, 0, RAW><<<grid, 256 * KG, 0, st>>>(p);
    else if (sum == 1)
        k_grouped_weight<T, TM, TN, STAGES, KG, 1, RAW><<<grid, 256 * KG, 0, st>>>(p);
    else
        k_grouped_weight<T, TM, TN, STAGES, KG, 2, RAW><<<grid, 256 * KG, 0, st>>>(p);
}
template <typename T>
hipError_t weight_t(const GroupedArgs& p, TileKind tile, bool raw, int sum, unsigned grid, hipStream_t st) {
    if (raw)
        weight_tile<T, 64, 64, 2, 1, true>(p, sum, grid, st);
    else if (tile == TILE_TALL)
        weight_tile<T, 256, 128, 2, 1, false>(p, sum, grid, st);
    else if (tile == TILE_SQUARE)
        weight_tile<T, 128, 128, 2, 1, false>(p, sum, grid, st);
    else if (tile == TILE_SMALL)
        weight_tile<T, 64, 64, 4, 1, false>(p, sum, grid, st);
    else
        weight_tile<T, 64, 64, 2, 4, false>(p, sum, grid, st);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped(const GroupedArgs& p, TileKind tile, bool raw, bool b_kc, int dtype, unsigned grid,
                          hipStream_t st) {
    return dtype == 0 ? rows_t<bf16>(p, tile, raw, b_kc, grid, st) : rows_t<f16>(p, tile, raw, b_kc, grid, st);
}

hipError_t launch_grouped_weight(const GroupedArgs& p, TileKind tile, bool raw, int dtype, int sum, unsigned grid,
                                 hipStream_t st) {
    return dtype == 0 ? weight_t<bf16>(p, tile, raw, sum, grid, st) : weight_t<f16>(p, tile, raw, sum, grid, st);
}

}  // namespace muon
