// The parts of a product's kernel that its forms share: how an operand's slices are
// loaded and read, the order of tiles, one tile's product over a run of slices,
// and its epilogue.
#pragma once

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

    // issue the next slice's loads to LDS address S; the one after is STEP further
    template <int STEP = 1>
    __device__ __forceinline__ void load(uint32_t S) {
        if constexpr (KC) {
            const uint32_t dead = kch < left ? 0u : OUT;  // chunks past the end of k
            const uint32_t so = left > 0 ? soff : 0u;
#pragma unroll
            for (int q = 0; q < NLD; ++q) load_lds(r, S + lds_row + q * 4096, off[q] | dead, so);
            soff += 2 * BK * STEP;
        } else {
            r[2] = left >= BK ? range : left > 0 ? (uint32_t)(left - 1) * rowb + tail : 0u;
#pragma unroll
            for (int q = 0; q < NLD; ++q) load_lds(r, S + lds_row + q * 4096, off[q], 0u);
            const uint64_t base = (((uint64_t)r[1] << 32) | r[0]) + (uint64_t)(BK * STEP) * rowb;
            r[0] = (uint32_t)base;
            r[1] = (uint32_t)(base >> 32) & 0xffffu;
        }
        left -= BK * STEP;
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

// What a tile's epilogue stages through: a wave's 32 rows of WN sums.
template <int WN>
constexpr int kStagedRow = WN * 4 + 16;

// The epilogue of a tile of TM x TN from row i0 and column j0 on, each of four waves
// holding the sums of a quarter of it. Each wave stages 32 rows at a time in its own
// LDS region and leaves with 8 consecutive columns a lane. What the epilogue reads
// for a block of 32 rows goes out two blocks ahead, before the stores of the blocks
// between, which it would otherwise wait for (loads and stores retire in order).
// piece: where the sums of a K piece go instead, -1 for a whole tile.
// stage(f, W): writes the sums of the wave's rows 32 f .. 32 f + 31 to W.
template <typename T, int TM, int TN, typename STAGE>
__device__ __forceinline__ void tile_epilogue(const GemmArgs& g, char* smem, int i0, int j0, int piece, int lane,
                                              int wave, STAGE&& stage) {
    constexpr int WM = TM / 2, WN = TN / 2;   // a wave's block
    constexpr int FRI = WM / 32;
    constexpr int SROW = kStagedRow<WN>;
    const int wi = wave >> 1, wj = wave & 1;
    char* W = smem + wave * 32 * SROW;
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
                stage(f_c, W);
                // unlike in each branch: the compiler would else merge them to one
                // that picks its sums by address, out of registers
                asm volatile("" ::"n"(F));
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
}

// The same for a whole tile of a known MODE: what a block of 32 rows needs is decided
// once for its passes, whose reads, activations and stores then go out together
// (chunk by chunk, with every mode's branches in each, a 256 x 128 tile's epilogue took
// 20000 clocks without any input or activation).
template <int MODE, typename T, int TM, int TN, typename STAGE>
__device__ __forceinline__ void whole_epilogue(const GemmArgs& g, char* smem, int i0, int j0, int lane, int wave,
                                               STAGE&& stage) {
    using U = std::conditional_t<MODE == EPI_GRAD_WEIGHT, float, T>;
    constexpr int WM = TM / 2, WN = TN / 2;   // a wave's block
    constexpr int FRI = WM / 32;
    constexpr int SROW = kStagedRow<WN>;
    constexpr int CPR = WN / 8;      // chunks of 8 per staged row
    constexpr int RPI = 64 / CPR;    // rows per pass of the wave
    constexpr int NP = 32 / RPI;     // passes per block
    constexpr int PG = TM == 256 && NP > 2 ? 2 : NP;  // of them at a time, beside the tall tile's sums
    const Epilogue& E = g.epi;
    const int wi = wave >> 1, wj = wave & 1;
    char* W = smem + wave * 32 * SROW;
    const int ch = lane % CPR, rr = lane / CPR;
    const int wrow = i0 + wi * WM, wcol = j0 + wj * WN;  // the wave's first row and column
    const int col = wcol + ch * 8;
    const bool inside = col < g.N;
    const int ncol = g.N - col >= 8 ? 8 : g.N - col;  // of the lane's chunk: fewer at the edge
    const bool edge = i0 + TM > g.M || j0 + TN > g.N;
    const int act = E.act;
    // what is read: on the way back through an activation z first, then add
    const bool slope = MODE == EPI_GRAD_INPUT && act != ACT_NONE;
    const U* const p1 = MODE == EPI_GRAD_WEIGHT ? (E.accumulate ? static_cast<const U*>(E.y) : nullptr)
                                                : static_cast<const U*>(slope ? E.z : E.add);
    const U* const p2 = slope ? static_cast<const U*>(E.add) : nullptr;
    const int ld1 = MODE == EPI_GRAD_WEIGHT ? E.ld_y : slope ? E.ld_z : E.ld_add, ld2 = E.ld_add;
    const int lane1 = rr * ld1 + ch * 8, lane2 = rr * ld2 + ch * 8;
    auto row_of = [&](int fi, int it) { return wrow + 32 * fi + it * RPI; };
    // the lane's chunk of pass `it`; lanes without a whole one have their row's first
    // (rows of less than one read nothing ahead)
    auto chunk = [&](const U* p, int ld, int ln, int fi, int it) {
        if (!edge) return p + ((int64_t)row_of(fi, it) * ld + wcol) + ln;
        const int row = row_of(fi, it) + rr;
        return p + ((int64_t)(row < g.M ? row : g.M - 1) * ld + (inside && ncol == 8 ? col : 0));
    };
    typedef u32x4 Chunk[sizeof(U) / 2];
    auto fetch = [&](const U* p, int ld, int ln, int fi, Chunk(&x)[NP]) {
#pragma unroll
        for (int it = 0; it < NP; ++it) {
            const u32x4_mem* q = reinterpret_cast<const u32x4_mem*>(chunk(p, ld, ln, fi, it));
#pragma unroll
            for (int k = 0; k < (int)sizeof(U) / 2; ++k) x[it][k] = __builtin_nontemporal_load(q + k);
        }
    };
    // the chunk's values, from what was fetched or, of fewer than 8, in place
    auto widen = [&](const Chunk& x, const U* p, int ld, int fi, int it, float* t) {
        if (edge && ncol < 8) {
            const int row = row_of(fi, it) + rr;
            float u[8];
            load8(p + ((int64_t)(row < g.M ? row : g.M - 1) * ld + col), ncol, u);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = u[e];
        } else if constexpr (sizeof(U) == 2) {
            const typename V8<T>::type u = __builtin_bit_cast(typename V8<T>::type, x[0]);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = (float)u[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = __uint_as_float(x[e / 4][e % 4]);
        }
    };
    auto put = [&](U* p, int ld, int fi, int from, const float (&v)[8 * PG]) {
        const int ln = rr * ld + ch * 8;
#pragma unroll
        for (int k = 0; k < PG; ++k) {
            const int it = from + k;
            float u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = v[8 * k + e];
            if (!edge)
                stream8(p + ((int64_t)row_of(fi, it) * ld + wcol) + ln, 8, u);
            else if (inside && row_of(fi, it) + rr < g.M)
                stream8(p + ((int64_t)(row_of(fi, it) + rr) * ld + col), ncol, u);
        }
    };
    float bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (MODE == EPI_FORWARD && E.bias && inside) load8(E.bias + col, ncol, bias);
    // inputs of this block and of the next one, which go out before this one's stores
    Chunk a0[NP], a1[NP], b0[NP];
    const bool ahead = p1 && g.N >= 8, second = p2 && g.N >= 8;
    if (ahead) fetch(p1, ld1, lane1, 0, a0);
#pragma unroll 1
    for (int fi = 0; fi < FRI; ++fi) {
        static_for<0, FRI>([&](auto f_c) {
            constexpr int F = decltype(f_c)::value;
            if (fi == F) {
                stage(f_c, W);
                asm volatile("" ::"n"(F));  // as in tile_epilogue
            }
        });
        if (second) fetch(p2, ld2, lane2, fi, b0);
        if (ahead && fi + 1 < FRI) fetch(p1, ld1, lane1, fi + 1, a1);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        static_for<0, NP / PG>([&](auto p_c) {
            constexpr int from = decltype(p_c)::value * PG;
            float v[8 * PG];
#pragma unroll
            for (int k = 0; k < PG; ++k) {
                const f32x4* s = reinterpret_cast<const f32x4*>(W + ((from + k) * RPI + rr) * SROW + 32 * ch);
                const f32x4 lo = s[0], up = s[1];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[8 * k + e] = lo[e];
                    v[8 * k + 4 + e] = up[e];
                }
            }
            if constexpr (MODE == EPI_FORWARD) {
#pragma unroll
                for (int n = 0; n < 8 * PG; ++n) v[n] += bias[n & 7];
                if (E.z) put(static_cast<U*>(E.z), E.ld_z, fi, from, v);
                act_values(act, v);
            }
            if (p1) {
                float t[8 * PG];
#pragma unroll
                for (int k = 0; k < PG; ++k) widen(a0[from + k], p1, ld1, fi, from + k, t + 8 * k);
                if (slope) {
                    act_slopes(act, t);
#pragma unroll
                    for (int n = 0; n < 8 * PG; ++n) v[n] *= t[n];
                    if (p2) {
#pragma unroll
                        for (int k = 0; k < PG; ++k) widen(b0[from + k], p2, ld2, fi, from + k, t + 8 * k);
                    }
                }
                if (!slope || p2) {
#pragma unroll
                    for (int n = 0; n < 8 * PG; ++n) v[n] += t[n];
                }
            }
            put(static_cast<U*>(E.y), E.ld_y, fi, from, v);
        });
        if (p1) {
#pragma unroll
            for (int it = 0; it < NP; ++it)
#pragma unroll
                for (int k = 0; k < (int)sizeof(U) / 2; ++k) a0[it][k] = a1[it][k];
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// LDS of a tile's product
template <typename T, int TM, int TN, bool AKC, bool BKC, bool RAW, int STAGES = 4, int KG = 1>
struct GemmShape {
    using OA = std::conditional_t<RAW, RawOperand<T, TM, AKC>, Operand<T, TM, AKC>>;
    using OB = std::conditional_t<RAW, RawOperand<T, TN, BKC>, Operand<T, TN, BKC>>;
    static constexpr int WM = TM / 2, WN = TN / 2;   // a wave's block
    static constexpr int FRI = WM / 32, FRJ = WN / 32;
    // the tall tile: two A buffers and one B buffer, so that two workgroups fit
    // a CU; the square tiles, for products too small to fill the chip, whose
    // time is load latency: a ring of four (STAGES) buffers of both
    static constexpr bool RING = TM <= 128;
    static constexpr int STAGE = OA::BYTES + OB::BYTES;
    static constexpr int SMEM = RAW ? 2 * STAGE : RING ? KG * STAGES * STAGE : OA::BYTES + STAGE;
    // the sums of the groups of waves but the first, behind the epilogue's staging
    static constexpr int MEET = (4 * 32 * kStagedRow<WN> + 1023) / 1024 * 1024;
    static_assert(4 * 32 * kStagedRow<WN> <= SMEM, "epilogue staging");
    static_assert(KG == 1 || (RING && !RAW && MEET + (KG - 1) * TM * TN * 4 <= SMEM), "groups of waves");
};

// SUM: also the sums over k of the B (1) or A (2) operand's rows, for the bias
// gradient: two-element dot products with 1 on the fragments in registers, in
// the shadow of the matrix instructions. RAW: operands as RawOperand has them.
// The tile (ti, tj)'s product over nk slices from s0 on, and its epilogue. KG groups of
// 4 waves take the slices in turn, each through a ring of its own, where a few tiles
// leave most of the chip idle and a slice is the latency of its reads and products one
// after the other; their sums meet in LDS, in the groups' order. MODE: the epilogue's,
// where it is known (and the tile whole).
template <typename T, int TM, int TN, bool AKC, bool BKC, int SUM, bool RAW, int STAGES = 4, int KG = 1,
          int MODE = -1>
__device__ __forceinline__ void gemm_tile(const GemmArgs& g, char* smem, int ti, int tj, int piece, int s0, int nk) {
    using Shape = GemmShape<T, TM, TN, AKC, BKC, RAW, STAGES, KG>;
    using OA = typename Shape::OA;
    using OB = typename Shape::OB;
    constexpr int WM = Shape::WM, WN = Shape::WN, FRI = Shape::FRI, FRJ = Shape::FRJ, STAGE = Shape::STAGE;
    constexpr bool RING = Shape::RING;
    static_assert(KG == 1 || SUM == 0, "the groups' sums over k do not meet");
    const int tid = KG > 1 ? threadIdx.x & 255 : threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int grp = KG > 1 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 8) : 0;
    const int wi = wave >> 1, wj = wave & 1;
    // a k-contiguous operand's rows go on to the next multiple of 8 (zeros), the
    // rows of the others likewise
    const int kp = (g.K + 7) & ~7, kmax = (AKC || BKC) && !RAW ? kp : g.K;
    const int i0 = ti * TM, j0 = tj * TN;
    const int kb = (s0 + grp) * BK;
    int ke = s0 * BK + nk * BK;
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

    char* const ring = smem + grp * STAGES * STAGE;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(LDS_AS char*)ring;
    if constexpr (RAW) {
        if (nk > 0) {  // else there may be no row to read
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
        static_assert((STAGES & (STAGES - 1)) == 0, "a ring's index");
        constexpr int NLD = OA::NLD + OB::NLD;
#pragma unroll
        for (int k = 0; k < STAGES - 1; ++k) {
            A.template load<KG>(lds0 + k * STAGE);
            B.template load<KG>(lds0 + k * STAGE + OA::BYTES);
        }
        wait_vm<(STAGES - 2) * NLD>();
        __syncthreads();
        read_b(ring + OA::BYTES, 0);
        read_a(ring, 0);
        // S: this slice, N: the next, ldsF: the buffer of the one before,
        // which every wave had read before the last barrier
        auto slice = [&](const char* __restrict__ S, const char* __restrict__ N, uint32_t ldsF)
                         __attribute__((always_inline)) {
            A.template load<KG>(ldsF);
            B.template load<KG>(ldsF + OA::BYTES);
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
            wait_vm<(STAGES - 2) * NLD>();  // the next slice has landed
            __syncthreads();
            read_b(N + OA::BYTES, 0);
            read_a(N, 0);
            products(NKS - 1, FRI / 2, FRI);
            interleave(std::integral_constant<int, RA + RB>{}, CH{});
        };
        const int turns = (nk + KG - 1) / KG;  // past the end, zeros are added
        for (int kt = 0; kt < turns; ++kt)
            slice(ring + (kt & (STAGES - 1)) * STAGE, ring + ((kt + 1) & (STAGES - 1)) * STAGE,
                  lds0 + ((kt - 1) & (STAGES - 1)) * STAGE);
        wait_vm0();  // the loads past the end
    }
    __syncthreads();
    if constexpr (KG > 1) {
        char* const meet = smem + Shape::MEET;
        auto place = [&](int group, int n) {
            return reinterpret_cast<f32x4*>(meet + (((group - 1) * FRI * FRJ * 4 + n) * 256 + tid) * 16);
        };
        if (grp > 0) {
            static_for<0, FRI * FRJ * 4>([&](auto n_c) {
                constexpr int n = decltype(n_c)::value;
                const f32x16& a = acc[n / (4 * FRJ)][n / 4 % FRJ];
                *place(grp, n) = f32x4{a[4 * (n & 3)], a[4 * (n & 3) + 1], a[4 * (n & 3) + 2], a[4 * (n & 3) + 3]};
            });
        }
        __syncthreads();
        if (grp == 0) static_for<0, FRI * FRJ * 4>([&](auto n_c) {
            constexpr int n = decltype(n_c)::value;
            f32x16& a = acc[n / (4 * FRJ)][n / 4 % FRJ];
#pragma unroll
            for (int k = 1; k < KG; ++k) {
                const f32x4 v = *place(k, n);
#pragma unroll
                for (int e = 0; e < 4; ++e) a[4 * (n & 3) + e] += v[e];
            }
        });
    }

    auto stage = [&](auto f_c, char* W) {
        constexpr int F = decltype(f_c)::value;
        const int l32 = lane & 31, hi = lane >> 5;
#pragma unroll
        for (int fj = 0; fj < FRJ; ++fj)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                f32x4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = acc[F][fj][4 * q + e];
                *reinterpret_cast<f32x4*>(W + l32 * kStagedRow<WN> + 4 * (32 * fj + 8 * q + 4 * hi)) = v;
            }
    };
    if constexpr (MODE < 0)
        tile_epilogue<T, TM, TN>(g, smem, i0, j0, piece, lane, wave, stage);
    else if (grp == 0)
        whole_epilogue<MODE, T, TM, TN>(g, smem, i0, j0, lane, wave, stage);
    if constexpr (SUM != 0) {
        const int l32 = lane & 31, hi = lane >> 5;
        const bool direct = piece < 0;
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

// The epilogue of few rows, `rows` of them from row i0 on: a workgroup's 8 waves have left
// their sums [rows][TNS] in LDS, `stride` bytes apart, which are added in wave order.
template <typename T, int TNS>
__device__ __forceinline__ void few_epilogue(const Epilogue& epi, int i0, int rows, int N, const char* smem, int stride,
                                             int j0) {
    const int row = threadIdx.x / (TNS / 8), c = threadIdx.x % (TNS / 8) * 8;
    const int col = j0 + c, left = N - col;
    if (row >= rows || left <= 0) return;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        const f32x4* p = reinterpret_cast<const f32x4*>(smem + w * stride + (row * TNS + c) * 4);
        const f32x4 lo = p[0], up = p[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] += lo[e];
            v[4 + e] += up[e];
        }
    }
    float bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (epi.bias) load8(epi.bias + col, left, bias);
    u32x4 in = {0, 0, 0, 0}, in2 = in;
    if (left >= 8) {
        in = first8<T>(epi, i0 + row, col, LaneAt());
        if (has_second(epi)) in2 = second8<T>(epi, i0 + row, col, LaneAt());
    }
    finish8<T>(epi, i0 + row, col, LaneAt(), left, v, bias, in, in2);
}

// LDS of a workgroup for few rows
template <bool BKC, int MT>
struct SkinnyShape {
    static constexpr int TNS = BKC ? 16 : 32;       // columns
    static constexpr int WB = TNS * 128;            // bytes of a slice of B
    static constexpr int XB = MT * 2048;            // and of A
    static constexpr int STAGE = WB + XB;
    static constexpr int NI = STAGE / 1024;         // load instructions per slice
    static constexpr int R = BKC && MT == 1 ? 4 : BKC || MT == 1 ? 3 : 2;  // slices in a wave's ring
    static constexpr int SMEM = 8 * R * STAGE;
};

// Few rows of A (up to 16 MT tokens) against all of B, one launch: bound by
// reading B once. A workgroup of 8 waves takes 16 columns of a k-contiguous B
// or 32 of the other and all of K; the waves take its slices of 64 in turn,
// each through a ring of its own in LDS (no barriers: a wave waits for its own
// loads), 16 to 18 KB a wave on the way. Their sums meet in LDS, in wave order.
// j0: the workgroup's first column.
template <typename T, bool BKC, int MT>
__device__ __forceinline__ void skinny_tile(const SkinnyArgs& g, char* smem, int j0) {
    using Shape = SkinnyShape<BKC, MT>;
    constexpr int TNS = Shape::TNS, WB = Shape::WB, XB = Shape::XB, STAGE = Shape::STAGE, NI = Shape::NI, R = Shape::R;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
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
    few_epilogue<T, TNS>(g.epi, 0, g.M, g.N, smem, R * STAGE, j0);
}

}  // namespace

}  // namespace muon
