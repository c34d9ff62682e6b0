// Matrices to 8-bit floating point with a float32 scale for each block of 128, on
// gfx950. Bound by HBM: each element is read once and written once (a weight in
// both orders twice, from one read). 2051 x 6400 bf16 9.1 us a call (39 MB), 1600 x 6400
// float32 in both orders 12.5 (61 MB, 4.9 TB/s; a copy of 2 GiB 4.9).
//
//  * Rows (activations, gradients): a block is 128 columns of a row, 16
//    neighbouring lanes of a wave; a wave takes 512 columns of a row at a time.
//  * Weights: a block is 128 x 128, one workgroup, in registers between its
//    maximum and its outputs: a thread holds 8 x 8, which it rounds two at a time
//    along the columns for the one order and along the rows for the other, so that
//    neither has to be taken apart again. The other order's rows meet in LDS and
//    leave as 128 consecutive bytes.

#include "eight_device.hpp"

namespace muon {

namespace {

// (One segment of 512 columns a wave: with four, their loads all on the way before the
// first is used, 2051 x 6400 bf16 took 11.3 us against 9.3.)
template <typename T, int F>
__global__ __launch_bounds__(256) void k_quantize(const Quantize a) {
    const int lane = threadIdx.x & 63;
    const int segs = (a.cols + 511) >> 9;
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t row = unit / segs;
    if (row >= a.rows) return;
    const int c = (int)(unit - row * segs) * 512 + lane * 8, left = a.cols - c;
    float v[8];
    load8(static_cast<const T*>(a.x) + row * a.ld_x + c, left, v);
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = umax(m, magnitude(v[e]));
    const ScaleOf<F, T> s(max16(m));
    s.scale8(v, left);
    // rows go on with zeros to the next multiple of 16
    if (left > 0 || (left > -8 && (c & 8)))
        *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.q) + row * a.ld_q + c) = pack8<F>(v);
    if ((lane & 15) == 0 && left > 0) a.scale[(int64_t)(c >> 7) * a.rows + row] = s.scale;
}

template <typename T>
__global__ __launch_bounds__(256) void k_quantize_weight(const QuantizeWeight a) {
    constexpr int F = EIGHT_E4M3;
    // Bytes of a row in LDS. Neighbouring lanes write 8 rows apart, 272 banks, so that 16 of
    // them begin at 4 of the 64 (any pitch of whole 8 bytes puts them on 4 at most): 74% of
    // the LDS-active clocks are conflicts, 1 us of a CU's, beside the wait for HBM.
    constexpr int PITCH = 136;
    __shared__ __attribute__((aligned(16))) uint8_t turn[128 * PITCH];
    __shared__ uint32_t red[4];
    const int tid = threadIdx.x;
    const int c8 = (tid & 15) * 8, r8 = (tid >> 4) * 8;  // the thread's 8 x 8
    const int row0 = blockIdx.y * 128, col0 = blockIdx.x * 128;
    const int left = a.cols - col0 - c8, down = a.rows - row0 - r8;
    float v[8][8];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        load8(static_cast<const T*>(a.w) + (int64_t)(row0 + r8 + j) * a.ld_w + col0 + c8, j < down ? left : 0, v[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = umax(m, magnitude(v[j][e]));
    }
    m = max16(m);
    m = umax(m, (uint32_t)__shfl_xor((int)m, 16, 64));
    m = umax(m, (uint32_t)__shfl_xor((int)m, 32, 64));
    if ((tid & 63) == 0) red[tid >> 6] = m;
    __syncthreads();
    const ScaleOf<F, T> s(umax(umax(red[0], red[1]), umax(red[2], red[3])));
    // values past an edge are 0, and stay 0 beside a NaN
#pragma unroll
    for (int j = 0; j < 8; ++j) s.scale8(v[j], j < down ? left : 0);
    const int rb = blockIdx.y, cb = blockIdx.x;
    if (a.q) {
        // rows go on with zeros to the next multiple of 16
        if (left > 0 || (left > -8 && (c8 & 8))) {
            uint8_t* q = static_cast<uint8_t*>(a.q) + (int64_t)(row0 + r8) * a.ld_q + col0 + c8;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < down) *reinterpret_cast<u32x2*>(q + (int64_t)j * a.ld_q) = pack8<F>(v[j]);
        }
        if (tid == 0) a.scale[(int64_t)rb * gridDim.x + cb] = s.scale;
    }
    if (a.qt) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const u32x2 t = {pack4<F>(v[0][e], v[1][e], v[2][e], v[3][e]), pack4<F>(v[4][e], v[5][e], v[6][e], v[7][e])};
            *reinterpret_cast<u32x2*>(turn + (c8 + e) * PITCH + r8) = t;
        }
        __syncthreads();
        // 8 threads a row of the other order, 16 bytes each
        const int r = tid >> 3, b = (tid & 7) * 16;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int row = r + 32 * k;
            if (col0 + row < a.cols && row0 + b < a.rows) {
                const u32x2 lo = *reinterpret_cast<const u32x2*>(turn + row * PITCH + b),
                            up = *reinterpret_cast<const u32x2*>(turn + row * PITCH + b + 8);
                *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(a.qt) + (int64_t)(col0 + row) * a.ld_qt + row0 + b) =
                    u32x4{lo[0], lo[1], up[0], up[1]};
            }
        }
        if (tid == 0) a.scale_t[(int64_t)cb * gridDim.y + rb] = s.scale;
    }
}

template <typename T>
void quantize_t(const Quantize& a, int format, hipStream_t st) {
    const int64_t units = (int64_t)a.rows * ((a.cols + 511) / 512);
    const unsigned g = (unsigned)((units + 3) / 4);
    if (format == EIGHT_E4M3)
        k_quantize<T, EIGHT_E4M3><<<g, 256, 0, st>>>(a);
    else
        k_quantize<T, EIGHT_E5M2><<<g, 256, 0, st>>>(a);
}

}  // namespace

hipError_t launch_quantize(const Quantize& a, int dtype, int format, hipStream_t st) {
    if (dtype == 0)
        quantize_t<bf16>(a, format, st);
    else if (dtype == 1)
        quantize_t<f16>(a, format, st);
    else
        quantize_t<float>(a, format, st);
    return hipGetLastError();
}

hipError_t launch_quantize_weight(const QuantizeWeight& a, int dtype, hipStream_t st) {
    const dim3 g((unsigned)((a.cols + 127) / 128), (unsigned)((a.rows + 127) / 128));
    if (dtype == 0)
        k_quantize_weight<bf16><<<g, 256, 0, st>>>(a);
    else if (dtype == 1)
        k_quantize_weight<f16><<<g, 256, 0, st>>>(a);
    else
        k_quantize_weight<float><<<g, 256, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace muon
