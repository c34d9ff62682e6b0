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

#include "layer_device.hpp"

namespace muon {

namespace {

constexpr int BK = kGemmSlice;
constexpr int NKS = BK / 16;       // k16 steps of a slice
constexpr int KROWB = 2 * BK;      // bytes of a row of a k-contiguous tile
constexpr uint32_t OUT = 0x80000000u;  // an offset beyond every resource's range

template <typename T>
__device__ __forceinline__ f32x16 mfma(typename V8<T>::type a, typename V8<T>::type b, f32x16 c);
template <>
__device__ __forceinline__ f32x16 mfma<bf16>(bf16x8 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x16 mfma<f16>(f16x8 a, f16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// s_waitcnt vmcnt(n), the other counters left alone
template <int N>
__device__ __forceinline__ void wait_vm() {
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
}

// 16 bytes per lane, global -> LDS: lane i lands at lds + 16 i (a wave-uniform
// LDS address, passed in M0, which the asm sets right before the load: see
// dma16, whose conditions hold here too).
__device__ __forceinline__ void load_lds(u32x4 r, uint32_t lds, uint32_t voff, uint32_t soff) {
    asm volatile("s_mov_b32 m0, %3\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                 :
                 : "v"(voff), "s"(r), "s"(soff), "s"(__builtin_amdgcn_readfirstlane(lds)));
}

// How one operand's tile is loaded and read. KC: TILE rows of 128 bytes (whole
// cache lines), chunk c (16 bytes) of row r stored at c ^ ((r >> 1) & 7), so
// that the 16 rows of a phase of ds_read_b128 fall in 16 distinct 16-byte
// slots. Otherwise BK rows of 2 TILE bytes, chunk c of row r at c ^ (4 (r & 3))
// (128-byte rows: c ^ (4 (r >> 1 & 1))), so that the 4 rows x 64 bytes of a
// half-wave's transposing read fall in 4 distinct 64-byte windows.
template <typename T, int TILE, bool KC>
struct Operand {
    static constexpr int BYTES = TILE * BK * 2;
    static constexpr int NLD = BYTES / 4096;  // load instructions a wave issues per slice
    static constexpr int BLK = TILE / 64;     // 32-wide fragment blocks of a wave
    static __device__ __forceinline__ int turn(int row) { return 4 * (TILE == 64 ? row >> 1 & 1 : row & 3); }
    u32x4 r;           // KC: the tile's rows; else the slice's
    uint32_t range;    // bytes of a whole slice's resource (not KC)
    uint32_t tail;     // bytes of the last row (not KC)
    uint32_t rowb;     // row stride in bytes
    uint32_t soff;     // KC: byte offset of the next slice to load
    int left;          // k values from the next slice to load to the split's end
    int kch;           // KC: the lane's first k within a slice
    uint32_t off[NLD];
    uint32_t lds_row;  // wave's first LDS byte of a load instruction
    int rd[4];         // fragment read offsets: KC one per k16 step, else one per block

    __device__ __forceinline__ void init(const void* p, int ld, int i0, int n, int kp, int kb, int kend, int wave,
                                         int lane, int wblk) {
        rowb = (uint32_t)ld * 2u;
        left = kend - kb;
        if constexpr (KC) {
            // 8 rows of 8 chunks per instruction
            const int rows = n - i0 < TILE ? n - i0 : TILE;
            r = rsrc(static_cast<const char*>(p) + (int64_t)i0 * rowb, (uint32_t)(rows - 1) * rowb + (uint32_t)kp * 2u);
            soff = (uint32_t)kb * 2u;
            const int row0 = wave * 8 + (lane >> 3);
            const int c = (lane & 7) ^ ((row0 >> 1) & 7);
            kch = c * 8;
#pragma unroll
            for (int q = 0; q < NLD; ++q) {
                const int row = row0 + q * 32;
                off[q] = row < rows ? (uint32_t)row * rowb + (uint32_t)c * 16u : OUT;
            }
            lds_row = wave * 8 * KROWB;
            const int l32 = lane & 31, hi = lane >> 5;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                rd[ks] = (wblk * (TILE / 2) + l32) * KROWB + 16 * ((2 * ks + hi) ^ ((l32 >> 1) & 7));
        } else {
            constexpr int XCH = TILE / 8;  // chunks of a row
            constexpr int RPI = 64 / XCH;  // rows per instruction
            const int cols = n - i0 < TILE ? n - i0 : TILE;
            tail = (uint32_t)cols * 2u;
            range = (uint32_t)(BK - 1) * rowb + tail;
            r = rsrc(static_cast<const char*>(p) + (int64_t)kb * rowb + (int64_t)i0 * 2, 0u);
            const int row0 = wave * RPI + lane / XCH;
            const int c = (lane % XCH) ^ turn(row0);
#pragma unroll
            for (int q = 0; q < NLD; ++q)
                off[q] = c * 8 < cols ? (uint32_t)(row0 + q * 4 * RPI) * rowb + (uint32_t)c * 16u : OUT;
            lds_row = wave * 1024;
            const int g = lane >> 4, s = lane & 15;
            const int row = 8 * (g >> 1) + (s >> 2);
#pragma unroll
            for (int f = 0; f < BLK; ++f) {
                const int e = wblk * (TILE / 2) + 32 * f + 16 * (g & 1) + 4 * (s & 3);
                rd[f] = row * (2 * TILE) + 16 * ((e >> 3) ^ turn(row)) + 2 * (e & 7);
            }
        }
    }

    // issue the next slice's loads to LDS address S
    __device__ __forceinline__ void load(uint32_t S) {
        if constexpr (KC) {
            const uint32_t dead = kch < left ? 0u : OUT;  // chunks past the end of k
            const uint32_t so = left > 0 ? soff : 0u;
#pragma unroll
            for (int q = 0; q < NLD; ++q) load_lds(r, S + lds_row + q * 4096, off[q] | dead, so);
            soff += 2 * BK;
        } else {
            r[2] = left >= BK ? range : left > 0 ? (uint32_t)(left - 1) * rowb + tail : 0u;
#pragma unroll
            for (int q = 0; q < NLD; ++q) load_lds(r, S + lds_row + q * 4096, off[q], 0u);
            const uint64_t base = (((uint64_t)r[1] << 32) | r[0]) + (uint64_t)BK * rowb;
            r[0] = (uint32_t)base;
            r[1] = (uint32_t)(base >> 32) & 0xffffu;
        }
        left -= BK;
    }
    // fragment block f of k16 step ks
    __device__ __forceinline__ typename V8<T>::type read(const char* S, int ks, int f) const {
        if constexpr (KC) {
            return *reinterpret_cast<const typename V8<T>::type*>(S + rd[ks] + f * 32 * KROWB);
        } else {
            const bf16x4 lo = tr_read(S + rd[f] + (16 * ks) * (2 * TILE));
            const bf16x4 up = tr_read(S + rd[f] + (16 * ks + 4) * (2 * TILE));
            return __builtin_bit_cast(typename V8<T>::type, __builtin_shufflevector(lo, up, 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }
};

// An operand whose rows start anywhere and end anywhere (8 elements at least),
// through registers: 16 bytes a lane, then to where Operand's loads put them. In
// the last slice, a chunk that would pass its row's end holds the row's last 8
// elements, which are moved down on the way to LDS, and zeros fill the k values
// past the end; in the others it reads on, up to 7 elements towards the next row
// (moved down there too, the tiles at the edge were the last to end: weight
// gradient of 999 x 1001 x 777 15.5 us). A tile's rows or columns past the
// matrix hold anything: nothing of their products is stored.
template <typename T, int TILE, bool KC>
struct RawOperand : Operand<T, TILE, KC> {
    using Base = Operand<T, TILE, KC>;
    static constexpr int NLD = Base::NLD;
    static constexpr int STEP = KC ? 32 : 32 * 64 / TILE;  // rows from one chunk of a lane to its next
    const char* p;             // KC: the tile's first row; else the next slice's (from the end on the last one's)
    uint32_t roff[NLD];        // byte offsets of the lane's rows
    uint32_t col, whole;       // not KC: byte offsets of the lane's chunk, and of one that is wholly in its row
    int row, at, end;          // the lane's first row; KC: its chunk's first k in a slice, and one past the last k
    int over;                  // not KC: elements from `whole` to the chunk
    int put_left;              // k values from the next slice to put to the end

    __device__ __forceinline__ void init(const void* src, int stride, int i0, int n, int kb, int kend, int wave,
                                         int lane, int wblk) {
        Base::init(src, stride, i0, n, 0, kb, kend, wave, lane, wblk);
        put_left = this->left;
        end = kend;
        p = static_cast<const char*>(src) + (int64_t)(KC ? i0 : kb) * this->rowb;
        if constexpr (KC) {
            row = wave * 8 + (lane >> 3);
            at = this->kch;
        } else {
            constexpr int XCH = TILE / 8;
            row = wave * (64 / XCH) + lane / XCH;
            const int c = i0 + 8 * ((lane % XCH) ^ Base::turn(row));
            over = c + 8 > n && c < n ? c + 8 - n : 0;
            whole = 2u * (uint32_t)(c + 8 <= n ? c : n - 8);
            col = c < n ? 2u * (uint32_t)c : whole;
        }
#pragma unroll
        for (int q = 0; q < NLD; ++q) {
            int r = row + q * STEP;
            if (KC && r > n - i0 - 1) r = n - i0 - 1;
            roff[q] = (uint32_t)r * this->rowb;
        }
    }
    // the next slice's chunks
    __device__ __forceinline__ void fetch(u32x4 (&v)[NLD]) {
        const int left = this->left;
        uint32_t o, last = ~0u;
        if constexpr (KC) {
            const int k = end - left + at;
            o = 2u * (uint32_t)(k < end - 8 ? k : end - 8);
        } else {
            const int rows = left < 1 ? 1 : left < BK ? left : BK;
            last = (uint32_t)(rows - 1) * this->rowb;
            o = left > BK ? col : whole;
        }
#pragma unroll
        for (int q = 0; q < NLD; ++q)
            v[q] = *reinterpret_cast<const u32x4_mem*>(p + ((roff[q] < last ? roff[q] : last) + o));
        if (!KC) p += left > BK ? (int64_t)BK * this->rowb : 0;
        this->left -= BK;
    }
    // fetched chunks to LDS
    __device__ __forceinline__ void put(char* S, int lane, u32x4 (&v)[NLD]) {
        if (put_left <= BK) {
            const int o = KC ? at + 8 - put_left : over;
#pragma unroll
            for (int q = 0; q < NLD; ++q) {
                const unsigned __int128 w = __builtin_bit_cast(unsigned __int128, v[q]);
                if (o > 0) v[q] = __builtin_bit_cast(u32x4, o < 8 ? w >> (16 * o) : (unsigned __int128)0);
                if (!KC && row + q * STEP >= put_left) v[q] = u32x4{0, 0, 0, 0};
            }
        }
#pragma unroll
        for (int q = 0; q < NLD; ++q) *reinterpret_cast<u32x4*>(S + this->lds_row + q * 4096 + lane * 16) = v[q];
        put_left -= BK;
    }
};

// Workgroups go round-robin over the 8 XCDs: of `total` of them, each XCD takes
// one contiguous run of the logical order, so what it works on at once shares
// operand panels in its L2.
__device__ __forceinline__ int per_xcd(int b, int total) {
    const int x = b & 7, i = b >> 3, q = total >> 3, r = total & 7;
    return x * q + (x < r ? x : r) + i;
}

// Tile l in the order of groups of kGroup tile rows that walk along the columns.
constexpr int kGroup = 4;
__device__ __forceinline__ void tile_at(const GemmArgs& g, int l, int& ti, int& tj) {
    const int per = kGroup * g.tiles_n;
    const int grp = l / per;
    const int rows = g.tiles_m - grp * kGroup < kGroup ? g.tiles_m - grp * kGroup : kGroup;
    l -= grp * per;
    ti = grp * kGroup + l % rows;
    tj = l / rows;
}

// v + the sum of a fragment's 8 elements
__device__ __forceinline__ float add8(bf16x8 f, float v) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 one = {(bf16)1.f, (bf16)1.f};
#pragma unroll
    for (int e = 0; e < 4; ++e) v = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{f[2 * e], f[2 * e + 1]}, one, v, false);
    return v;
}
__device__ __forceinline__ float add8(f16x8 f, float v) {
    typedef f16 f16x2 __attribute__((ext_vector_type(2)));
    const f16x2 one = {(f16)1.f, (f16)1.f};
#pragma unroll
    for (int e = 0; e < 4; ++e) v = __builtin_amdgcn_fdot2(f16x2{f[2 * e], f[2 * e + 1]}, one, v, false);
    return v;
}

// SUM: also the sums over k of the B (1) or A (2) operand's rows, for the bias
// gradient: two-element dot products with 1 on the fragments in registers, in
// the shadow of the matrix instructions. RAW: operands as RawOperand has them.
template <typename T, int TM, int TN, bool AKC, bool BKC, int SUM, bool RAW>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(TM == 128 ? 1 : 2, TM == 128 ? 1 : 2))) void
k_gemm(const GemmArgs g) {
    using OA = std::conditional_t<RAW, RawOperand<T, TM, AKC>, Operand<T, TM, AKC>>;
    using OB = std::conditional_t<RAW, RawOperand<T, TN, BKC>, Operand<T, TN, BKC>>;
    constexpr int WM = TM / 2, WN = TN / 2;   // a wave's block
    constexpr int FRI = WM / 32, FRJ = WN / 32;
    constexpr int SROW = WN * 4 + 16;  // bytes of a staged epilogue row
    // the tall tile: two A buffers and one B buffer, so that two workgroups fit
    // a CU; the square tiles, for products too small to fill the chip, whose
    // time is load latency: a ring of four buffers of both
    constexpr bool RING = TM <= 128;
    constexpr int STAGE = OA::BYTES + OB::BYTES;
    constexpr int SMEM = RAW ? 2 * STAGE : RING ? 4 * STAGE : OA::BYTES + STAGE;
    static_assert(4 * 32 * SROW <= SMEM, "epilogue staging");
    __shared__ __attribute__((aligned(16))) char smem[SMEM];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wi = wave >> 1, wj = wave & 1;
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
    // a k-contiguous operand's rows go on to the next multiple of 8 (zeros), the
    // rows of the others likewise
    const int kp = (g.K + 7) & ~7, kmax = (AKC || BKC) && !RAW ? kp : g.K;
    int ti, tj;
    tile_at(g, tile, ti, tj);
    const int i0 = ti * TM, j0 = tj * TN;
    const int kb = s0 * BK;
    int ke = kb + nk * BK;
    ke = ke < kmax ? ke : kmax;

    OA A;
    OB B;
    if constexpr (RAW) {
        A.init(g.a, g.ld_a, i0, g.M, kb, ke, wave, lane, wi);
        B.init(g.b, g.ld_b, j0, g.N, kb, ke, wave, lane, wj);
    } else {
        A.init(g.a, g.ld_a, i0, AKC ? g.M : (g.M + 7) & ~7, kp, kb, AKC ? ke : (ke < g.K ? ke : g.K), wave, lane, wi);
        B.init(g.b, g.ld_b, j0, BKC ? g.N : (g.N + 7) & ~7, kp, kb, BKC ? ke : (ke < g.K ? ke : g.K), wave, lane, wj);
    }

    f32x16 acc[FRI][FRJ];
#pragma unroll
    for (int a = 0; a < FRI; ++a)
#pragma unroll
        for (int b = 0; b < FRJ; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.f;

    typename V8<T>::type pf[2][FRI], qf[NKS][FRJ];
    auto read_a = [&](const char* S, int ks) {
#pragma unroll
        for (int f = 0; f < FRI; ++f) pf[ks & 1][f] = A.read(S, ks, f);
    };
    auto read_b = [&](const char* S, int ks) {
#pragma unroll
        for (int f = 0; f < FRJ; ++f) qf[ks][f] = B.read(S, ks, f);
    };
    auto products = [&](int ks, int f0, int f1) {
#pragma unroll
        for (int fi = f0; fi < f1; ++fi)
#pragma unroll
            for (int fj = 0; fj < FRJ; ++fj) acc[fi][fj] = mfma<T>(qf[ks][fj], pf[ks & 1][fi], acc[fi][fj]);
    };
    constexpr int RA = (AKC ? 1 : 2) * FRI, RB = (BKC ? 1 : 2) * FRJ;  // LDS reads of a k16 step
    // M matrix instructions with N LDS reads spread over them
    auto interleave = [&](auto n_c, auto m_c) {
        constexpr int N = decltype(n_c)::value, M = decltype(m_c)::value;
        static_for<0, M>([&](auto i_c) {
            constexpr int I = decltype(i_c)::value;
            constexpr int R = N * (I + 1) / M - N * I / M;
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            if constexpr (R > 0) __builtin_amdgcn_sched_group_barrier(0x100, R, 0);
        });
    };
    constexpr int NSUM = SUM == 1 ? FRJ : SUM == 2 ? FRI : 1;
    float sums[NSUM];
#pragma unroll
    for (int f = 0; f < NSUM; ++f) sums[f] = 0.f;
    // the rows of A are twice a wave's columns of B, and their sums cost twice as
    // much: the two waves that hold the same rows take two k16 steps each (the
    // [out, in] gradient of 16384 x 1600 x 6400: 345 us, against 368)
    auto add_sums = [&](int ks) {
        if (SUM == 2 && (ks >= 2) != (wj == 1)) return;
#pragma unroll
        for (int f = 0; f < NSUM; ++f) {
            if constexpr (SUM == 1) sums[f] = add8(qf[ks][f], sums[f]);
            if constexpr (SUM == 2) sums[f] = add8(pf[ks & 1][f], sums[f]);
        }
    };
    using CM = std::integral_constant<int, FRI * FRJ>;
    using CH = std::integral_constant<int, FRI * FRJ / 2>;

    const uint32_t lds0 = (uint32_t)(uintptr_t)(LDS_AS char*)smem;
    if constexpr (RAW) {
        // two slices in LDS, the three after the current one in registers or
        // on their way there
        u32x4 ra[3][OA::NLD], rb[3][OB::NLD];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            A.fetch(ra[k]);
            B.fetch(rb[k]);
        }
        A.put(smem, lane, ra[0]);
        B.put(smem + OA::BYTES, lane, rb[0]);
        __syncthreads();
        read_b(smem + OA::BYTES, 0);
        read_a(smem, 0);
        // slice kt: the one three on goes into registers F (kt's own were put in
        // the slice before), the next one's P into LDS, where every wave had
        // read slice kt - 1 before the last barrier
        auto slice = [&](int kt, auto f_c, auto p_c) __attribute__((always_inline)) {
            constexpr int F = decltype(f_c)::value, P = decltype(p_c)::value;
            char* const S = smem + (kt & 1) * STAGE;
            char* const N = smem + (~kt & 1) * STAGE;
            A.fetch(ra[F]);
            B.fetch(rb[F]);
            __builtin_amdgcn_sched_barrier(0);
            static_for<0, NKS>([&](auto k_c) {
                constexpr int KS = decltype(k_c)::value;
                if constexpr (KS + 1 < NKS) {
                    read_b(S + OA::BYTES, KS + 1);
                    read_a(S, KS + 1);
                }
                products(KS, 0, FRI);
                add_sums(KS);
                if constexpr (KS == 0) {
                    A.put(N, lane, ra[P]);
                    B.put(N + OA::BYTES, lane, rb[P]);
                }
            });
            __syncthreads();
            read_b(N + OA::BYTES, 0);
            read_a(N, 0);
        };
        using I0 = std::integral_constant<int, 0>;
        using I1 = std::integral_constant<int, 1>;
        using I2 = std::integral_constant<int, 2>;
        for (int kt = 0; kt < nk; kt += 3) {
            slice(kt, I0{}, I1{});
            if (kt + 1 == nk) break;
            slice(kt + 1, I1{}, I2{});
            if (kt + 2 == nk) break;
            slice(kt + 2, I2{}, I0{});
        }
    } else if constexpr (!RING) {
        char* const SB = smem + 2 * OA::BYTES;
        A.load(lds0);
        B.load(lds0 + 2 * OA::BYTES);
        wait_vm0();
        __syncthreads();
        read_b(SB, 0);
        read_a(smem, 0);
        // One slice: its A tile in S (its B tile in SB), the next slice's A
        // tile coming into N. The loads are invisible to the compiler; the
        // waits and barriers here order them.
        auto slice = [&](const char* __restrict__ S, const char* __restrict__ N, const char* __restrict__ Q,
                         uint32_t ldsN) __attribute__((always_inline)) {
            A.load(ldsN);  // every wave had read this buffer before the last barrier
            __builtin_amdgcn_sched_barrier(0);
            read_b(Q, 1);
            read_b(Q, 2);
            read_b(Q, 3);
            read_a(S, 1);
            products(0, 0, FRI);
            add_sums(0);
            interleave(std::integral_constant<int, 3 * RB + RA>{}, CM{});
            __builtin_amdgcn_sched_barrier(0);
            __syncthreads();  // every wave holds the slice's B fragments
            B.load(lds0 + 2 * OA::BYTES);
            __builtin_amdgcn_sched_barrier(0);
            read_a(S, 2);
            products(1, 0, FRI);
            add_sums(1);
            interleave(std::integral_constant<int, RA>{}, CM{});
            read_a(S, 3);
            products(2, 0, FRI);
            add_sums(2);
            interleave(std::integral_constant<int, RA>{}, CM{});
            products(3, 0, FRI / 2);
            add_sums(3);
            __builtin_amdgcn_sched_barrier(0);
            wait_vm0();  // the next slice has landed
            __syncthreads();
            read_b(Q, 0);
            read_a(N, 0);
            products(3, FRI / 2, FRI);
            interleave(std::integral_constant<int, RA + RB>{}, CH{});
        };
        for (int kt = 0; kt < nk; kt += 2) {
            slice(smem, smem + OA::BYTES, SB, lds0 + OA::BYTES);
            if (kt + 1 < nk) slice(smem + OA::BYTES, smem, SB, lds0);
        }
    } else {
        constexpr int NLD = OA::NLD + OB::NLD;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            A.load(lds0 + k * STAGE);
            B.load(lds0 + k * STAGE + OA::BYTES);
        }
        wait_vm<2 * NLD>();
        __syncthreads();
        read_b(smem + OA::BYTES, 0);
        read_a(smem, 0);
        // S: this slice, N: the next, ldsF: the buffer of the one before,
        // which every wave had read before the last barrier
        auto slice = [&](const char* __restrict__ S, const char* __restrict__ N, uint32_t ldsF)
                         __attribute__((always_inline)) {
            A.load(ldsF);
            B.load(ldsF + OA::BYTES);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int ks = 0; ks < NKS - 1; ++ks) {
                read_b(S + OA::BYTES, ks + 1);
                read_a(S, ks + 1);
                products(ks, 0, FRI);
                add_sums(ks);
                interleave(std::integral_constant<int, RA + RB>{}, CM{});
            }
            products(NKS - 1, 0, FRI / 2);
            add_sums(NKS - 1);
            __builtin_amdgcn_sched_barrier(0);
            wait_vm<2 * NLD>();  // the next slice has landed
            __syncthreads();
            read_b(N + OA::BYTES, 0);
            read_a(N, 0);
            products(NKS - 1, FRI / 2, FRI);
            interleave(std::integral_constant<int, RA + RB>{}, CH{});
        };
        for (int kt = 0; kt < nk; ++kt)
            slice(smem + (kt & 3) * STAGE, smem + ((kt + 1) & 3) * STAGE, lds0 + ((kt + 3) & 3) * STAGE);
        wait_vm0();  // the loads past the end
    }
    __syncthreads();

    // ---- epilogue: lane holds C[i][j .. j+3], i = l32, j = 8 g + 4 hi; each
    // wave stages 32 rows at a time in its own LDS region and leaves with 8
    // consecutive columns a lane. What the epilogue reads for a block of 32
    // rows goes out two blocks ahead, before the stores of the blocks between,
    // which it would otherwise wait for (loads and stores retire in order). ----
    char* W = smem + wave * 32 * SROW;
    const int l32 = lane & 31, hi = lane >> 5;
    constexpr int CPR = WN / 8;      // chunks of 8 per staged row
    constexpr int RPI = 64 / CPR;    // rows per pass of the wave
    constexpr int NP = 32 / RPI;     // passes per block
    const int ch = lane % CPR, rr = lane / CPR;
    const int col = j0 + wj * WN + ch * 8;
    const bool inside = col < g.N;
    // columns of the lane's chunk: 8, or fewer at the edge
    const int ncol = g.N - col >= 8 ? 8 : g.N - col;
    // lanes without a whole chunk fetch their row's first one, unused (rows of
    // less than one fetch nothing)
    const int row0 = i0 + wi * WM + rr;
    const LaneAt at(g.epi, rr, ch * 8);
    const int wcol = j0 + wj * WN;  // the wave's first column
    // a tile at the matrix's edge
    const bool edge = i0 + TM > g.M || j0 + TN > g.N;
    const int64_t ccol = inside && ncol == 8 ? col : 0;
    const bool direct = piece < 0;
    float* const part = g.partial + (int64_t)piece * (TM * TN);
    float bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (direct && g.epi.bias && inside) load8(g.epi.bias + col, ncol, bias);
    // this block's first8, the next one's, and the one's after that or, where
    // there is one, this block's second8
    u32x4 in0[NP], in1[NP], in2[NP];
    const bool ahead = direct && g.N >= 8, second = ahead && has_second(g.epi);
    auto fetch = [&](int fi, u32x4(&x)[NP]) {
#pragma unroll
        for (int it = 0; it < NP; ++it) {
            const int row = row0 + 32 * fi + it * RPI;
            x[it] = edge ? first8<T>(g.epi, row < g.M ? row : g.M - 1, ccol, LaneAt())
                         : first8<T>(g.epi, row - rr, wcol, at);
        }
    };
    if (ahead) {
        fetch(0, in0);
        if (FRI > 1) fetch(1, in1);
    }
#pragma unroll 1
    for (int fi = 0; fi < FRI; ++fi) {
        static_for<0, FRI>([&](auto f_c) {
            constexpr int F = decltype(f_c)::value;
            if (fi == F) {
#pragma unroll
                for (int fj = 0; fj < FRJ; ++fj)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        f32x4 v;
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = acc[F][fj][4 * q + e];
                        *reinterpret_cast<f32x4*>(W + l32 * SROW + 4 * (32 * fj + 8 * q + 4 * hi)) = v;
                    }
            }
        });
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (second) {
#pragma unroll
            for (int it = 0; it < NP; ++it) {
                const int row = row0 + 32 * fi + it * RPI;
                in2[it] = edge ? second8<T>(g.epi, row < g.M ? row : g.M - 1, ccol, LaneAt())
                               : second8<T>(g.epi, row - rr, wcol, at);
            }
        } else if (ahead && fi + 2 < FRI) {
            fetch(fi + 2, in2);
        }
#pragma unroll
        for (int it = 0; it < NP; ++it) {
            const int row = row0 + 32 * fi + it * RPI;
            const f32x4* s = reinterpret_cast<const f32x4*>(W + (it * RPI + rr) * SROW + 32 * ch);
            const f32x4 lo = s[0], up = s[1];
            if (row < g.M && inside) {
                if (direct) {
                    float v[8] = {lo[0], lo[1], lo[2], lo[3], up[0], up[1], up[2], up[3]};
                    finish8<T>(g.epi, row - rr, wcol, at, ncol, v, bias, in0[it], in2[it]);
                } else {
                    float* p = part + (row - i0) * TN + (col - j0);
                    *reinterpret_cast<f32x4*>(p) = lo;
                    *reinterpret_cast<f32x4*>(p + 4) = up;
                }
            }
        }
#pragma unroll
        for (int it = 0; it < NP; ++it) {
            in0[it] = in1[it];
            in1[it] = in2[it];
        }
        if (second && fi + 2 < FRI) fetch(fi + 2, in1);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    if constexpr (SUM != 0) {
        // the bias gradient: one tile of each row or column of tiles, spread
        // over them
        float* const half = reinterpret_cast<float*>(smem);
        if constexpr (SUM == 2) {
            __syncthreads();  // the staged rows have been read
#pragma unroll
            for (int f = 0; f < NSUM; ++f) {
                sums[f] += __shfl_xor(sums[f], 32, 64);
                if (wj == 1 && hi == 0) half[wi * WM + 32 * f + l32] = sums[f];
            }
            __syncthreads();
        }
        const bool mine = SUM == 1 ? ti == tj % g.tiles_m && wi == 0 : tj == ti % g.tiles_n && wj == 0;
        if (mine) {
            const int at = (SUM == 1 ? wj * WN : wi * WM) + l32;
            const int n = (SUM == 1 ? j0 : i0) + at, end = SUM == 1 ? g.N : g.M;
            float old[NSUM];
#pragma unroll
            for (int f = 0; f < NSUM; ++f) {
                old[f] = 0.f;
                if (direct && g.epi.accumulate && n + 32 * f < end) old[f] = g.sums[n + 32 * f];
            }
#pragma unroll
            for (int f = 0; f < NSUM; ++f) {
                const float s = SUM == 1 ? sums[f] + __shfl_xor(sums[f], 32, 64) : sums[f] + half[at + 32 * f];
                if (hi == 0 && n + 32 * f < end) {
                    if (direct)
                        g.sums[n + 32 * f] = old[f] + s;
                    else
                        g.sum_part[(int64_t)piece * 256 + at + 32 * f] = s;
                }
            }
        }
    }
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

template <typename T>
__device__ __forceinline__ f32x4 mfma16(typename V8<T>::type a, typename V8<T>::type b, f32x4 c);
template <>
__device__ __forceinline__ f32x4 mfma16<bf16>(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x4 mfma16<f16>(f16x8 a, f16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Few rows of A (up to 16 MT tokens) against all of B, one launch: bound by
// reading B once. A workgroup of 8 waves takes 16 columns of a k-contiguous B
// or 32 of the other and all of K; the waves take its slices of 64 in turn,
// each through a ring of its own in LDS (no barriers: a wave waits for its own
// loads), 16 to 18 KB a wave on the way. Their sums meet in LDS, in wave order.
template <typename T, bool BKC, int MT>
__global__ __launch_bounds__(512) void k_skinny(const SkinnyArgs g) {
    constexpr int TNS = BKC ? 16 : 32;       // columns
    constexpr int WB = TNS * 128;            // bytes of a slice of B
    constexpr int XB = MT * 2048;            // and of A
    constexpr int STAGE = WB + XB;
    constexpr int NI = STAGE / 1024;         // load instructions per slice
    constexpr int R = BKC && MT == 1 ? 4 : BKC || MT == 1 ? 3 : 2;  // slices in a wave's ring
    __shared__ __attribute__((aligned(16))) char smem[8 * R * STAGE];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int j0 = per_xcd(blockIdx.x, gridDim.x) * TNS;
    const int kp = (g.K + 7) & ~7;
    char* const ring = smem + wave * R * STAGE;
    const uint32_t lring = (uint32_t)(uintptr_t)(LDS_AS char*)ring;

    // B, k-contiguous: 8 rows (columns of C) of 8 chunks per instruction, chunk
    // c of row r at c ^ (r & 7); else 16 rows (k) of 4 chunks, chunk c of row r
    // at c ^ (2 (r >> 3 & 1)). A: 8 rows of 8 chunks, as the former.
    const uint32_t rowb = (uint32_t)g.ld_b * 2u, rowa = (uint32_t)g.ld_a * 2u;
    const int r8 = lane >> 3, c8 = (lane & 7) ^ (r8 & 7);
    uint32_t offw[WB / 1024], offx[XB / 1024];
    u32x4 rw, rx;
    uint32_t tail = 0;
    const int rows = g.N - j0 < TNS ? g.N - j0 : TNS;
    if constexpr (BKC) {
#pragma unroll
        for (int q = 0; q < WB / 1024; ++q)
            offw[q] = r8 + 8 * q < rows ? (uint32_t)(r8 + 8 * q) * rowb + (uint32_t)c8 * 16u : OUT;
        rw = rsrc(static_cast<const char*>(g.b) + (int64_t)j0 * rowb, (uint32_t)(rows - 1) * rowb + (uint32_t)kp * 2u);
    } else {
        const int r4 = lane >> 2, c4 = (lane & 3) ^ (2 * (r4 >> 3 & 1));
        const int np = (g.N + 7) & ~7, cols = np - j0 < TNS ? np - j0 : TNS;
        tail = (uint32_t)cols * 2u;
#pragma unroll
        for (int q = 0; q < WB / 1024; ++q)
            offw[q] = c4 * 8 < cols ? (uint32_t)(r4 + 16 * q) * rowb + (uint32_t)c4 * 16u : OUT;
        rw = rsrc(g.b, 0u);
    }
#pragma unroll
    for (int q = 0; q < XB / 1024; ++q)
        offx[q] = r8 + 8 * q < g.M ? (uint32_t)(r8 + 8 * q) * rowa + (uint32_t)c8 * 16u : OUT;
    rx = rsrc(g.a, (uint32_t)(g.M - 1) * rowa + (uint32_t)kp * 2u);

    auto load = [&](int slice, uint32_t dst) {
        const int k0 = slice * BK;
        const uint32_t so = k0 < kp ? (uint32_t)k0 * 2u : 0u;
        const uint32_t dead = c8 * 8 < kp - k0 ? 0u : OUT;
        if constexpr (BKC) {
#pragma unroll
            for (int q = 0; q < WB / 1024; ++q) load_lds(rw, dst + q * 1024, offw[q] | dead, so);
        } else {
            const int left = g.K - k0;
            const u32x4 r = rsrc(static_cast<const char*>(g.b) + (left > 0 ? (int64_t)k0 * rowb : 0) + (int64_t)j0 * 2,
                                 left >= BK ? (uint32_t)(BK - 1) * rowb + tail
                                            : left > 0 ? (uint32_t)(left - 1) * rowb + tail : 0u);
#pragma unroll
            for (int q = 0; q < WB / 1024; ++q) load_lds(r, dst + q * 1024, offw[q], 0u);
        }
#pragma unroll
        for (int q = 0; q < XB / 1024; ++q) load_lds(rx, dst + WB + q * 1024, offx[q] | dead, so);
    };

    f32x4 acc[TNS / 16][MT];
#pragma unroll
    for (int a = 0; a < TNS / 16; ++a)
#pragma unroll
        for (int b = 0; b < MT; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int l16 = lane & 15, g16 = lane >> 4;
    const int mine = (g.slices - wave + 7) / 8;  // slices wave, wave + 8, ...
#pragma unroll
    for (int k = 0; k < R - 1; ++k) load(wave + 8 * k, lring + k * STAGE);
    int at = 0;
    for (int i = 0; i < mine; ++i) {
        // the buffer read last turn takes the slice R - 1 ahead: its reads have
        // returned (their products were issued), and none moves across here
        int to = at + R - 1;
        if (to >= R) to -= R;
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        load(wave + 8 * (i + R - 1), lring + to * STAGE);
        wait_vm<(R - 1) * NI>();
        asm volatile("" ::: "memory");
        const char* S = ring + at * STAGE;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            typename V8<T>::type wf[TNS / 16], xf[MT];
#pragma unroll
            for (int h = 0; h < TNS / 16; ++h) {
                if constexpr (BKC) {
                    wf[h] = *reinterpret_cast<const typename V8<T>::type*>(S + l16 * 128 + 16 * ((4 * ks + g16) ^ (l16 & 7)));
                } else {
                    const int row = 32 * ks + 8 * g16 + (l16 >> 2);
                    const char* p = S + row * 64 + 32 * (h ^ (g16 & 1)) + 8 * (l16 & 3);
                    const bf16x4 lo = tr_read(p), up = tr_read(p + 4 * 64);
                    wf[h] = __builtin_bit_cast(typename V8<T>::type, __builtin_shufflevector(lo, up, 0, 1, 2, 3, 4, 5, 6, 7));
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
                xf[m] = *reinterpret_cast<const typename V8<T>::type*>(S + WB + (m * 16 + l16) * 128 +
                                                                       16 * ((4 * ks + g16) ^ (l16 & 7)));
#pragma unroll
            for (int h = 0; h < TNS / 16; ++h)
#pragma unroll
                for (int m = 0; m < MT; ++m) acc[h][m] = mfma16<T>(wf[h], xf[m], acc[h][m]);
        }
        at = at + 1 == R ? 0 : at + 1;
    }
    wait_vm0();  // the loads past the end
    asm volatile("" ::: "memory");

    // lane holds C[token l16 + 16 m][column 16 h + 4 g16 .. +3]; each wave's
    // [16 MT][TNS] sums go into its own ring
    float* const own = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int h = 0; h < TNS / 16; ++h)
#pragma unroll
        for (int m = 0; m < MT; ++m)
            *reinterpret_cast<f32x4*>(own + (m * 16 + l16) * TNS + 16 * h + 4 * g16) = acc[h][m];
    __syncthreads();
    const int row = threadIdx.x / (TNS / 8), c = threadIdx.x % (TNS / 8) * 8;
    const int col = j0 + c, left = g.N - col;
    if (row >= g.M || left <= 0) return;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        const f32x4* p = reinterpret_cast<const f32x4*>(smem + w * R * STAGE + (row * TNS + c) * 4);
        const f32x4 lo = p[0], up = p[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] += lo[e];
            v[4 + e] += up[e];
        }
    }
    float bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (g.epi.bias) load8(g.epi.bias + col, left, bias);
    u32x4 in = {0, 0, 0, 0}, in2 = in;
    if (left >= 8) {
        in = first8<T>(g.epi, row, col, LaneAt());
        if (has_second(g.epi)) in2 = second8<T>(g.epi, row, col, LaneAt());
    }
    finish8<T>(g.epi, row, col, LaneAt(), left, v, bias, in, in2);
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
