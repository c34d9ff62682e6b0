// The linear layer's product on 8-bit floating point operands with a float32 scale
// for each block of 128, on gfx950:
//   C[m, n] = sum over blocks b of sx[b, m] sw[n / 128, b] sum over k in b of X[m, k] W[n, k],
// both operands k-contiguous, fp32 sums, the linear layer's epilogue.
//
//  * A slice of K is a block: 128 bytes of a row, the same bytes as a slice of 64
//    16-bit elements, so that loads to LDS and reads from it are the linear layer's
//    (Operand). The matrix instruction's k order does not matter as long as both
//    operands have the same.
//  * A block's products are summed by the matrix unit from 0, and its sum times its
//    scale is added to the accumulator: one vector instruction for 64 outputs of a
//    block (each an fma, rounded once), half of the matrix unit's time, and beside
//    it where another fragment's products run. Tokens are the lanes' index of the
//    result, so that a lane has one scale per fragment; a tile's columns lie in one
//    block of the weight, whose scale is the same for all lanes.
//  * The matrix unit's sums: it adds the products of 8 consecutive bytes in fixed point,
//    cut off 13 bits below the power of two of the largest, and such groups in about
//    float32. A group is so off by less than 7 2^-13 of its largest product. Products of
//    8-bit operands have few bits there: for operands of random sign the error of a whole
//    result is 2^-12 of it at most in root mean square (2 10^-4 measured), beside 2^-5 and
//    more that the operands' own rounding cost. Where the large products of a group
//    cancel, what is left may be what was cut, and no relative bound holds.
//  * Rows start 16-byte aligned. Where K is no multiple of 16, the bytes past it in
//    the last 16 are cleared in LDS, whatever they hold.
//
// What bounds it: 8192^3 492 us (2.23 PFLOP/s; a library product with one scale for a
// whole matrix, which adds nothing per block, 2.55 to 2.88). The matrix unit is busy 51% of
// the clocks, the vector unit 41%: the scales' fmas cost 15 to 20% (without them 2.52
// PFLOP/s), the barriers and LDS reads the rest: a slice begins with its first fragments'
// reads, while none of the wave's products runs. 16384 x 1600 -> 6400 with bias, GELU and
// kept pre-activation 219 to 228 us, by the box: 13 blocks of K a tile, then 64 KB of activations each, two
// outputs; the matrix unit is busy 33%. The library's bare product takes 196.
// Tried: 32 x 32 x 64 instructions (half the reads, but 16 registers a block sum: 802 us
// for 8192^3 against 525 then); a 256 x 256 tile of 128 x 128 a wave (more than the 256
// registers that fmas can take, so moves for the others: 705 against 512); rings of 8
// half slices; the CU's second workgroup begun late: no gain. Rows of K that are no
// multiple of 128 bytes share cache lines: K = 1600 220 us, 1664 204, which is why the
// Python layer lays out rows of many in whole lines.

#include "eight_device.hpp"
#include "gemm_device.hpp"

namespace muon {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// The products of a whole block. W's fragment first: lanes of the result are X's rows.
template <int F>
__device__ __forceinline__ f32x4 mfma_eight(i32x8 w, i32x8 x) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, f32x4{0.f, 0.f, 0.f, 0.f}, 0, F, 0, 0, 0, 0);
}

// Clears what lies past K in the last 16 bytes of each of `rows` rows of a slice.
template <int ROWS>
__device__ __forceinline__ void clear_tail(char* S, int k, int tid) {
    const int c = (k & 127) >> 4, keep = k & 15;
    for (int r = tid; r < ROWS; r += 256) {
        u32x4* p = reinterpret_cast<u32x4*>(S + r * KROWB + 16 * (c ^ ((r >> 1) & 7)));
        const unsigned __int128 mask = ((unsigned __int128)1 << (8 * keep)) - 1;
        *p = __builtin_bit_cast(u32x4, __builtin_bit_cast(unsigned __int128, *p) & mask);
    }
}

// 4 bytes per lane, global -> LDS: as load_lds.
__device__ __forceinline__ void load_lds4(u32x4 r, uint32_t lds, uint32_t voff, uint32_t soff) {
    asm volatile("s_mov_b32 m0, %3\n\tbuffer_load_dword %0, %1, %2 offen lds"
                 :
                 : "v"(voff), "s"(r), "s"(soff), "s"(__builtin_amdgcn_readfirstlane(lds)));
}

// KG groups of 4 waves take the slices in turn, as in gemm_tile.
template <typename T, int TM, int TN, int STAGES, int KG, int F, int MODE>
__global__ __launch_bounds__(256 * KG) __attribute__((amdgpu_waves_per_eu(KG > 2 ? KG : 2))) void k_scaled(
    const ScaledArgs p) {
    using OA = Operand<bf16, TM, true>;
    using OB = Operand<bf16, TN, true>;
    constexpr int WM = TM / 2, WN = TN / 2;   // a wave's block
    constexpr int FRI = WM / 16, FRJ = WN / 16;
    constexpr bool RING = TM <= 128;
    // a ring's buffer: the slices of both operands, and each wave's scales of X's rows
    constexpr int STAGE = OA::BYTES + OB::BYTES + (RING ? 1024 : 0);
    constexpr int MEET = (4 * 32 * kStagedRow<WN> + 1023) / 1024 * 1024;  // the groups' sums, behind the staging
    constexpr int SMEM = RING ? KG * STAGES * STAGE : OA::BYTES + STAGE;
    static_assert(KG == 1 || (RING && MEET + (KG - 1) * TM * TN * 4 <= SMEM), "groups of waves");
    __shared__ __attribute__((aligned(16))) char smem[SMEM];
    const GemmArgs& g = p.g;
    const int tid = KG > 1 ? threadIdx.x & 255 : threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int grp = KG > 1 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 8) : 0;
    const int wi = wave >> 1, wj = wave & 1;
    int ti, tj;
    tile_at(g, per_xcd(blockIdx.x, gridDim.x), ti, tj);
    const int i0 = ti * TM, j0 = tj * TN;
    const int nk = g.slices;
    // K in pairs of bytes, to the end of the last 16
    const int kp = ((g.K + 15) & ~15) / 2;
    const bool tail = (g.K & 15) != 0;

    OA A;
    OB B;
    A.init(g.a, g.ld_a / 2, i0, g.M, kp, grp * BK, kp, wave, lane, wi);
    B.init(g.b, g.ld_b / 2, j0, g.N, kp, grp * BK, kp, wave, lane, wj);

    f32x4 acc[FRI][FRJ];
#pragma unroll
    for (int a = 0; a < FRI; ++a)
#pragma unroll
        for (int b = 0; b < FRJ; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};

    // scales: X's of the lane's rows (0 past the last one), W's of the tile's block
    // of columns
    const float* const sw = p.scale_w + (int64_t)(j0 >> 7) * nk;
    const int l16 = lane & 15, g16 = lane >> 4;
    float raw[FRI], sc[FRI];
    // tall tile: to registers, a slice ahead, under the wait for the slice itself
    auto fetch_scales = [&](int kt) {
        const auto r = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<float*>(p.scale_x + (int64_t)(kt < nk ? kt : nk - 1) * g.M), 0, g.M * 4, 0x00020000);
#pragma unroll
        for (int f = 0; f < FRI; ++f)
            raw[f] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, (i0 + wi * WM + l16 + 16 * f) * 4, 0, 0));
    };
    // W's of 64 blocks at a time, one a lane (a scalar load for each slice is one
    // latency for each slice)
    float sw64 = sw[lane < nk ? lane : nk - 1];
    auto take_scales = [&](int kt) {
        if (kt > 63 && (kt & 63) < KG) sw64 = sw[(kt & ~63) + lane < nk ? (kt & ~63) + lane : nk - 1];
        const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sw64), kt & 63));
#pragma unroll
        for (int f = 0; f < FRI; ++f) sc[f] = raw[f] * w;
    };

    // A fragment is 16 rows of a slice: the lane's are chunks g16 and g16 + 4 of row l16
    i32x8 qf[FRJ], pf[2];
    const int turn = (l16 >> 1) & 7;
    const int rd0 = l16 * KROWB + 16 * (g16 ^ turn), rd1 = l16 * KROWB + 16 * ((g16 + 4) ^ turn);
    auto frag = [&](const char* S) {
        const u32x4 lo = *reinterpret_cast<const u32x4*>(S + rd0), up = *reinterpret_cast<const u32x4*>(S + rd1);
        return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)up[0], (int)up[1], (int)up[2], (int)up[3]};
    };
    auto read_b = [&](const char* S) {
#pragma unroll
        for (int f = 0; f < FRJ; ++f) qf[f] = frag(S + (wj * WN + 16 * f) * KROWB);
    };
    auto read_a = [&](const char* S, auto f_c) {
        constexpr int f = decltype(f_c)::value;
        pf[f & 1] = frag(S + (wi * WM + 16 * f) * KROWB);
    };
    // Pair n of fragments (row n / FRJ, column n % FRJ): its block sum, and what
    // becomes of the one DIST before it, whose matrix instruction has ended.
    constexpr int PAIRS = FRI * FRJ, DIST = 2;
    f32x4 t[DIST + 1];
    auto collect = [&](auto n_c) {
        constexpr int n = decltype(n_c)::value;
        const float s = sc[n / FRJ];
        f32x4& a = acc[n / FRJ][n % FRJ];
        a = __builtin_elementwise_fma(t[n % (DIST + 1)], f32x4{s, s, s, s}, a);
        asm volatile("" : "+v"(a));  // here, and not sunk behind a later branch with every block sum kept
    };
    // pairs FROM .. TO - 1 of the slice in S, whose first row of A has been read
    auto products = [&](const char* S, auto from_c, auto to_c) {
        static_for<decltype(from_c)::value, decltype(to_c)::value>([&](auto n_c) {
            constexpr int n = decltype(n_c)::value, f = n / FRJ;
            if constexpr (n % FRJ == 0 && f + 1 < FRI) read_a(S, std::integral_constant<int, f + 1>{});
            t[n % (DIST + 1)] = mfma_eight<F>(qf[n % FRJ], pf[f & 1]);
            if constexpr (n >= DIST) collect(std::integral_constant<int, n - DIST>{});
            __builtin_amdgcn_sched_barrier(0);
        });
        if constexpr (decltype(to_c)::value == PAIRS)
            static_for<(PAIRS > DIST ? PAIRS - DIST : 0), PAIRS>([&](auto n_c) { collect(n_c); });
    };

    char* const ring = smem + grp * STAGES * STAGE;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(LDS_AS char*)ring;
    if constexpr (!RING) {
        char* const SB = smem + 2 * OA::BYTES;
        fetch_scales(0);
        A.load(lds0);
        B.load(lds0 + 2 * OA::BYTES);
        wait_vm0();
        take_scales(0);
        __syncthreads();
        if (tail && nk == 1) {
            clear_tail<TM>(smem, g.K, tid);
            clear_tail<TN>(SB, g.K, tid);
            __syncthreads();
        }
        // One slice: its A tile in S (its B tile in SB), the next slice's A tile
        // coming into N, at address ldsN. The loads are invisible to the compiler;
        // the waits and barriers here order them.
        auto slice = [&](int kt, const char* __restrict__ S, char* __restrict__ N, const char* __restrict__ Q,
                         uint32_t ldsN) __attribute__((always_inline)) {
            fetch_scales(kt + 1);
            A.load(ldsN);  // every wave had read this buffer before the last barrier
            __builtin_amdgcn_sched_barrier(0);
            read_b(Q);
            read_a(S, std::integral_constant<int, 0>{});
            products(S, std::integral_constant<int, 0>{}, std::integral_constant<int, FRJ>{});
            __syncthreads();  // every wave holds the slice's B fragments
            B.load(lds0 + 2 * OA::BYTES);
            __builtin_amdgcn_sched_barrier(0);
            products(S, std::integral_constant<int, FRJ>{}, std::integral_constant<int, PAIRS>{});
            __builtin_amdgcn_sched_barrier(0);
            wait_vm0();  // the next slice has landed
            take_scales(kt + 1);
            __syncthreads();
            if (tail && kt + 2 == nk) {
                clear_tail<TM>(N, g.K, tid);
                clear_tail<TN>(SB, g.K, tid);
                __syncthreads();
            }
        };
        // (one copy of the slice: with one for each buffer, as the linear layer has, the
        // sums' registers had to be the same at two exits, and spilled)
        for (int kt = 0; kt < nk; ++kt) {
            const int o = (kt & 1) * OA::BYTES, n = OA::BYTES - o;
            slice(kt, smem + o, smem + n, SB, lds0 + n);
        }
    } else {
        // Scales go the way of the operands: into registers, the compiler's wait for
        // them would be one for every load in flight (2048 x 6400 x 1600 43.7 us).
        constexpr int NLD = OA::NLD + OB::NLD + 1;
        const uint32_t at = lane < WM && i0 + wi * WM + lane < g.M ? 4u * (uint32_t)(i0 + wi * WM + lane) : OUT;
        int next = grp;  // the next slice to load
        auto load = [&](uint32_t buf) {
            A.template load<KG>(buf);
            B.template load<KG>(buf + OA::BYTES);
            const float* s = p.scale_x + (int64_t)(next < nk ? next : nk - 1) * g.M;
            load_lds4(rsrc(s, (uint32_t)g.M * 4u), buf + OA::BYTES + OB::BYTES + wave * 256, at, 0u);
            next += KG;
        };
#pragma unroll
        for (int k = 0; k < STAGES - 1; ++k) load(lds0 + k * STAGE);
        const int turns = (nk + KG - 1) / KG;  // past the end, zeros are added
        for (int t = 0; t < turns; ++t) {
            const int kt = grp + KG * t;
            char* const S = ring + (t & (STAGES - 1)) * STAGE;
            wait_vm<(STAGES - 2) * NLD>();  // this slice has landed
            __syncthreads();
            if (tail && t + 1 == turns) {
                if (kt + 1 == nk) {
                    clear_tail<TM>(S, g.K, tid);
                    clear_tail<TN>(S + OA::BYTES, g.K, tid);
                }
                __syncthreads();
            }
            // into the buffer of the slice before, which every wave had read
            // before the barrier
            load(lds0 + ((t - 1) & (STAGES - 1)) * STAGE);
            __builtin_amdgcn_sched_barrier(0);
            read_b(S + OA::BYTES);
            read_a(S, std::integral_constant<int, 0>{});
            const float* own = reinterpret_cast<const float*>(S + OA::BYTES + OB::BYTES + wave * 256);
#pragma unroll
            for (int f = 0; f < FRI; ++f) raw[f] = own[16 * f + l16];
            take_scales(kt);
            products(S, std::integral_constant<int, 0>{}, std::integral_constant<int, PAIRS>{});
        }
        wait_vm0();  // the loads past the end
    }
    __syncthreads();
    if constexpr (KG > 1) {
        auto place = [&](int group, int n) {
            return reinterpret_cast<f32x4*>(smem + MEET + (((group - 1) * FRI * FRJ + n) * 256 + tid) * 16);
        };
        if (grp > 0) static_for<0, PAIRS>([&](auto n_c) {
            constexpr int n = decltype(n_c)::value;
            *place(grp, n) = acc[n / FRJ][n % FRJ];
        });
        __syncthreads();
        if (grp > 0) return;
        static_for<0, PAIRS>([&](auto n_c) {
            constexpr int n = decltype(n_c)::value;
#pragma unroll
            for (int k = 1; k < KG; ++k) acc[n / FRJ][n % FRJ] += *place(k, n);
        });
    }
    // lane holds C[i][j .. j + 3] of a fragment, i = l16, j = 4 g16
    whole_epilogue<MODE, T, TM, TN>(g, smem, i0, j0, lane, wave, [&](auto f_c, char* W) {
        constexpr int R = 2 * decltype(f_c)::value;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int b = 0; b < FRJ; ++b)
                *reinterpret_cast<f32x4*>(W + (16 * a + l16) * kStagedRow<WN> + 4 * (16 * b + 4 * g16)) = acc[R + a][b];
    });
}

// Few rows of X, in blocks of 16 MT, against all of W: bound by reading W once (a block
// of rows each, and it is in cache for the next one). A workgroup of 8 waves takes a
// block's 16 columns and all of K; the waves take its slices in turn, each through a
// ring of its own in LDS (a wave waits for its own loads, X's scales among them). Their
// sums meet in LDS, in wave order. One row, 1600 -> 6400: 7.8 us, of which the 10 MB of
// W are 2. The rest is a launch, and two rounds of workgroups (400 of them, and 136 KB of
// LDS lets one run on a CU) that each wait for W's scales, then for their first slice.
template <typename T, int MT, int F>
__global__ __launch_bounds__(512) void k_scaled_few(const ScaledArgs p) {
    constexpr int WB = 2048, XB = MT * 2048;      // bytes of a slice of W, of X
    constexpr int STAGE = WB + XB + 256;          // and its scales
    constexpr int NI = (WB + XB) / 1024 + 1;      // load instructions per slice
    constexpr int R = MT == 1 ? 4 : 3;            // slices in a wave's ring
    __shared__ __attribute__((aligned(16))) char smem[8 * R * STAGE];
    const GemmArgs& g = p.g;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    // the row blocks of 16 columns follow one another, for the same XCD
    const int l = per_xcd(blockIdx.x, gridDim.x);
    const int j0 = l / g.tiles_m * 16, i0 = (l - l / g.tiles_m * g.tiles_m) * 16 * MT;
    const int here = g.M - i0 < 16 * MT ? g.M - i0 : 16 * MT;  // rows
    const int kp = (g.K + 15) & ~15;
    char* const ring = smem + wave * R * STAGE;
    const uint32_t lring = (uint32_t)(uintptr_t)(LDS_AS char*)ring;
    // 8 rows of 8 chunks per instruction, chunk c of row r at c ^ (r & 7)
    const uint32_t rowa = (uint32_t)g.ld_a, rowb = (uint32_t)g.ld_b;
    const int r8 = lane >> 3, c8 = (lane & 7) ^ (r8 & 7);
    const int rows = g.N - j0 < 16 ? g.N - j0 : 16;
    uint32_t offw[WB / 1024], offx[XB / 1024];
#pragma unroll
    for (int q = 0; q < WB / 1024; ++q)
        offw[q] = r8 + 8 * q < rows ? (uint32_t)(r8 + 8 * q) * rowb + (uint32_t)c8 * 16u : OUT;
#pragma unroll
    for (int q = 0; q < XB / 1024; ++q)
        offx[q] = r8 + 8 * q < here ? (uint32_t)(r8 + 8 * q) * rowa + (uint32_t)c8 * 16u : OUT;
    const uint32_t offs = lane < here ? 4u * (uint32_t)lane : OUT;
    const u32x4 rw = rsrc(static_cast<const char*>(g.b) + (int64_t)j0 * rowb, (uint32_t)(rows - 1) * rowb + (uint32_t)kp);
    const u32x4 rx = rsrc(static_cast<const char*>(g.a) + (int64_t)i0 * rowa, (uint32_t)(here - 1) * rowa + (uint32_t)kp);
    const float* const sw = p.scale_w + (int64_t)(j0 >> 7) * g.slices;
    auto load = [&](int slice, uint32_t dst) {
        const int k0 = slice * 128;
        const uint32_t so = k0 < kp ? (uint32_t)k0 : 0u, dead = c8 * 16 < kp - k0 ? 0u : OUT;
#pragma unroll
        for (int q = 0; q < WB / 1024; ++q) load_lds(rw, dst + q * 1024, offw[q] | dead, so);
#pragma unroll
        for (int q = 0; q < XB / 1024; ++q) load_lds(rx, dst + WB + q * 1024, offx[q] | dead, so);
        const float* sx = p.scale_x + (int64_t)(slice < g.slices ? slice : g.slices - 1) * g.M + i0;
        load_lds4(rsrc(sx, 4u * (uint32_t)here), dst + WB + XB, offs, 0u);
    };
    f32x4 acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int l16 = lane & 15, g16 = lane >> 4;
    const int rd0 = l16 * 128 + 16 * (g16 ^ (l16 & 7)), rd1 = l16 * 128 + 16 * ((g16 + 4) ^ (l16 & 7));
    auto frag = [&](const char* S) {
        const u32x4 lo = *reinterpret_cast<const u32x4*>(S + rd0), up = *reinterpret_cast<const u32x4*>(S + rd1);
        return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)up[0], (int)up[1], (int)up[2], (int)up[3]};
    };
    const int mine = (g.slices - wave + 7) / 8;  // slices wave, wave + 8, ...
    int at = 0;
    // W's scales of the wave's next 64 slices, one a lane, which come before its loads
    auto scales64 = [&](int i) {
        const int b = wave + 8 * (i + lane);
        return sw[b < g.slices ? b : g.slices - 1];
    };
    float sw64 = scales64(0);
    asm volatile("" : "+v"(sw64));
#pragma unroll
    for (int k = 0; k < R - 1; ++k) load(wave + 8 * k, lring + k * STAGE);
    for (int i = 0; i < mine; ++i) {
        if ((i & 63) == 0 && i) sw64 = scales64(i);
        // the buffer read last turn takes the slice R - 1 ahead: its reads have
        // returned (their products were issued), and none moves across here
        int to = at + R - 1;
        if (to >= R) to -= R;
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        load(wave + 8 * (i + R - 1), lring + to * STAGE);
        wait_vm<(R - 1) * NI>();
        asm volatile("" ::: "memory");
        char* S = ring + at * STAGE;
        const int slice = wave + 8 * i;
        if ((g.K & 15) && slice + 1 == g.slices && lane < 16 + 16 * MT) {
            // what lies past K in the last 16 bytes of the lane's row
            u32x4* q = reinterpret_cast<u32x4*>(S + lane * 128 + 16 * (((g.K & 127) >> 4) ^ (lane & 7)));
            const unsigned __int128 mask = ((unsigned __int128)1 << (8 * (g.K & 15))) - 1;
            *q = __builtin_bit_cast(u32x4, __builtin_bit_cast(unsigned __int128, *q) & mask);
        }
        const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sw64), i & 63));
        const i32x8 wf = frag(S);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const float s = reinterpret_cast<const float*>(S + WB + XB)[16 * m + l16] * w;
            const f32x4 t = mfma_eight<F>(wf, frag(S + WB + m * 2048));
            acc[m] = __builtin_elementwise_fma(t, f32x4{s, s, s, s}, acc[m]);
        }
        at = at + 1 == R ? 0 : at + 1;
    }
    wait_vm0();  // the loads past the end
    asm volatile("" ::: "memory");
    // lane holds C[token l16 + 16 m][column 4 g16 .. +3]
    float* const own = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int m = 0; m < MT; ++m) *reinterpret_cast<f32x4*>(own + (m * 16 + l16) * 16 + 4 * g16) = acc[m];
    __syncthreads();
    few_epilogue<T, 16>(g.epi, i0, here, g.N, smem, R * STAGE, j0);
}

template <typename T, int F, int MODE>
void scaled_tiles(const ScaledArgs& p, TileKind tile, unsigned grid, hipStream_t st) {
    if (tile == TILE_TALL)
        k_scaled<T, 256, 128, 2, 1, F, MODE><<<grid, 256, 0, st>>>(p);
    else if (tile == TILE_SQUARE)
        k_scaled<T, 128, 128, 2, 1, F, MODE><<<grid, 256, 0, st>>>(p);
    else if (tile == TILE_SQUARE_GROUPS)
        k_scaled<T, 128, 128, 2, 2, F, MODE><<<grid, 512, 0, st>>>(p);
    else if (tile == TILE_SMALL)
        k_scaled<T, 64, 64, 4, 1, F, MODE><<<grid, 256, 0, st>>>(p);
    else
        k_scaled<T, 64, 64, 2, 4, F, MODE><<<grid, 1024, 0, st>>>(p);
}
template <typename T, int F>
hipError_t scaled_t(const ScaledArgs& p, TileKind tile, hipStream_t st) {
    const unsigned grid = (unsigned)(p.g.tiles_m * p.g.tiles_n);
    if (tile == TILE_FEW16)
        k_scaled_few<T, 1, F><<<grid, 512, 0, st>>>(p);
    else if (tile == TILE_FEW32)
        k_scaled_few<T, 2, F><<<grid, 512, 0, st>>>(p);
    else if (p.g.epi.mode == EPI_FORWARD)
        scaled_tiles<T, F, EPI_FORWARD>(p, tile, grid, st);
    else
        scaled_tiles<T, F, EPI_GRAD_INPUT>(p, tile, grid, st);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_scaled(const ScaledArgs& p, TileKind tile, int dtype, int format, hipStream_t st) {
    if (dtype == 0)
        return format == EIGHT_E4M3 ? scaled_t<bf16, EIGHT_E4M3>(p, tile, st) : scaled_t<bf16, EIGHT_E5M2>(p, tile, st);
    return format == EIGHT_E4M3 ? scaled_t<f16, EIGHT_E4M3>(p, tile, st) : scaled_t<f16, EIGHT_E5M2>(p, tile, st);
}

}  // namespace muon
