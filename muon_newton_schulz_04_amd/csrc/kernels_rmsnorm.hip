// Root-mean-square norm over rows, forward (with the residual's addition before
// it and an output in 8 bits beside or instead of its own type) and backward, on
// gfx950. Bound by HBM: forward reads x and the residual once and writes their
// sum and the outputs once, backward reads dy, x (and the residual's gradient)
// once and writes dx once.
//
//  * The sum of x and the residual is rounded to their type, as the residual
//    stream that goes on, and the norm is taken of what was stored: the backward
//    pass has those very numbers.
//  * A row lives in registers between its sum and its output, in chunks of 8
//    consecutive elements a lane, as in the layer norm: 16 neighbouring lanes
//    hold the 128 columns that share a scale, whose largest magnitude is four
//    DPP rotations away. What is rounded to 8 bits is the float32 output, not its
//    rounding to the row's type.
//  * Rows of more than kBlockCols columns are read twice (the second time from
//    cache as far as it holds them).
//  * The weight's gradient: each wave keeps the sums of dy xhat of its own columns
//    in registers over all the rows it goes through, a workgroup writes one
//    partial row, and a second kernel adds the partial rows in order.
//
// Measured, inputs in turn that no cache holds (a copy of 2 GiB reaches 4.9 TB/s on the
// same box): 16384 x 1600 bf16, residual, 8-bit output 37.1 us a call (184 MB, 5.0 TB/s);
// its backward with the residual's gradient 45 (210 MB; the pass 40, the join of 768
// partial rows 4). One row takes 4 us, the call 13 on the host. Nontemporal
// loads of x and the residual: no difference.

#include "eight_device.hpp"
#include "norm_device.hpp"

namespace muon {

namespace {

// The longest rows that live in registers: 32 elements a lane of 4 waves.
constexpr int kBlockCols = 8192;

// What a lane does with its chunk of 8 outputs t from column c on, `left` of which
// exist (the others are 0): y, and the 8-bit form with its scale. All 16 lanes of
// a block call it together.
template <typename T, int F>
__device__ __forceinline__ void emit(const RmsForward& n, int64_t row, int c, int left, const float (&t)[8]) {
    if (n.y && left > 0) stream8(static_cast<T*>(n.y) + row * n.ld_y + c, left, t);
    if constexpr (F != EIGHT_NONE) {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = umax(m, magnitude(t[e]));
        const ScaleOf<F, float> s(max16(m));
        // rows go on with zeros to the next multiple of 16
        if (left > -8 && (left > 0 || (c & 8))) {
            float u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = t[e];
            s.scale8(u, left);
            const u32x2 q = pack8<F>(u);
            __builtin_nontemporal_store(q, reinterpret_cast<u32x2*>(static_cast<uint8_t*>(n.q) + row * n.ld_q + c));
        }
        if ((c & 127) == 0 && left > 0) n.scale[(int64_t)(c >> 7) * n.rows + row] = s.scale;
    }
}

// ADD: the residual is added first
template <typename T, int NCH, int WPR, bool VEC, bool ADD, int F>
__global__ __launch_bounds__(256) void k_rms_forward(const RmsForward n) {
    __shared__ float red[8];
    constexpr int LPR = 64 * WPR;  // lanes per row
    const int lane = threadIdx.x % LPR;
    const int64_t row = (int64_t)blockIdx.x * (4 / WPR) + threadIdx.x / LPR;
    if (row >= n.rows) return;  // a whole wave (WPR = 1) or never (WPR = 4)
    const T* x = static_cast<const T*>(n.x) + row * n.ld_x;
    const T* add = static_cast<const T*>(n.add) + row * n.ld_add;
    T* sum = static_cast<T*>(n.sum) + row * n.ld_sum;
    Raw<T> v[NCH], r[ADD ? NCH : 1];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = (i * LPR + lane) * 8;
        v[i].template load<VEC>(x + c, n.cols - c);
        if constexpr (ADD) r[i].template load<VEC>(add + c, n.cols - c);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        if constexpr (ADD) {
            const int c = (i * LPR + lane) * 8, left = n.cols - c;
            float t[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = v[i].get(e) + r[i].get(e);
            v[i].put(t);
            if (left > 0) {
                if (VEC || left >= 8) {
                    v[i].store(sum + c);
                } else {
                    for (int e = 0; e < left; ++e) sum[c + e] = (T)t[e];
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = v[i].get(e);
            s = fmaf(d, d, s);
        }
    }
    const float rstd = 1.f / sqrtf(row_sum<WPR>(s, red) * (1.f / (float)n.cols) + n.eps);
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = (i * LPR + lane) * 8, left = n.cols - c;
        float t[8], w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = v[i].get(e) * rstd;
        if (n.weight) {
            load8(n.weight + c, left, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] *= w[e];
        }
        emit<T, F>(n, row, c, left, t);
    }
    if (lane == 0) n.rstd[row] = rstd;
}

// Rows of any length, one workgroup each: each lane reads again what it stored.
template <typename T, bool ADD, int F>
__global__ __launch_bounds__(256) void k_rms_forward_wide(const RmsForward n) {
    __shared__ float red[8];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(n.x) + row * n.ld_x;
    const T* add = static_cast<const T*>(n.add) + row * n.ld_add;
    T* sum = static_cast<T*>(n.sum) + row * n.ld_sum;
    float s = 0.f;
    for (int c = threadIdx.x * 8; c < n.cols; c += 2048) {
        const int left = n.cols - c;
        float v[8], r[8];
        load8(x + c, left, v);
        if constexpr (ADD) {
            load8(add + c, left, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (float)(T)(v[e] + r[e]);
            store8(sum + c, left, v);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(v[e], v[e], s);
    }
    const float rstd = 1.f / sqrtf(row_sum<4>(s, red) * (1.f / (float)n.cols) + n.eps);
    for (int b = 0; b < n.cols; b += 2048) {
        const int c = b + threadIdx.x * 8, left = n.cols - c;
        float t[8], w[8];
        load8((ADD ? sum : x) + c, left, t);
        if (n.weight) load8(n.weight + c, left, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            t[e] *= rstd;
            if (n.weight) t[e] *= w[e];
        }
        emit<T, F>(n, row, c, left, t);
    }
    if (threadIdx.x == 0) n.rstd[row] = rstd;
}

// dx = rstd (g - xhat mean(g xhat)) + add with g = dy w, and the workgroup's sums
// of dy xhat per column. WPR waves share a row, and go through their rows with the
// next row's x, dy and add on the way in. VEC: rows are whole chunks.
template <typename T, int NCH, int WPR, bool VEC>
__global__ __launch_bounds__(WPR == 8 ? 512 : 256) __attribute__((amdgpu_waves_per_eu(2))) void k_rms_backward(
    const RmsBackward n) {
    constexpr int LPR = 64 * WPR;
    constexpr int WAVES = WPR == 8 ? 8 : 4;
    constexpr int RPB = WAVES / WPR;  // rows a workgroup works on at once
    constexpr int CW = NCH * LPR * 8;
    __shared__ float red[2][2 * WAVES];
    __shared__ float col[RPB > 1 ? RPB / 2 * CW : 1];
    const int lane = threadIdx.x % LPR;
    const float inv = 1.f / (float)n.cols;
    float w[NCH][8], dw[NCH][8];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = (i * LPR + lane) * 8;
        if (n.weight) {
            load8(n.weight + c, n.cols - c, w[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[i][e] = 1.f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
    }
    struct Row {
        Raw<T> x[NCH], dy[NCH], add[NCH];
        float rstd;
    };
    auto fetch = [&](Row& r, int64_t row) {
        const T* x = static_cast<const T*>(n.x) + row * n.ld_x;
        const T* dy = static_cast<const T*>(n.dy) + row * n.ld_y;
        const T* add = static_cast<const T*>(n.add) + row * n.ld_add;
        r.rstd = n.rstd[row];
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = (i * LPR + lane) * 8;
            r.x[i].template load<VEC>(x + c, n.cols - c);
            r.dy[i].template load<VEC>(dy + c, n.cols - c);
            if (n.add) r.add[i].template load<VEC>(add + c, n.cols - c);
        }
    };
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR;
    Row cur, nxt;
    if (row < n.rows) fetch(cur, row);
    // the same number of turns for every wave
    const int64_t turns = (n.rows + step - 1) / step;
    for (int64_t t = 0; t < turns; ++t, row += step) {
        const bool live = row < n.rows;
        if (row + step < n.rows) fetch(nxt, row + step);
        const float rstd = cur.rstd;
        // x and dy are 0 past the row's end, which adds nothing to any sum
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            if (!live) break;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xh = cur.x[i].get(e) * rstd, d = cur.dy[i].get(e);
                dw[i][e] = fmaf(d, xh, dw[i][e]);
                s = fmaf(d * w[i][e], xh, s);
            }
        }
        s = row_sum<WPR>(s, red[t & 1]) * inv;
        T* dx = static_cast<T*>(n.dx) + row * n.ld_dx;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = (i * LPR + lane) * 8;
            const int left = n.cols - c;
            if (left <= 0 || !live) continue;
            cur.x[i].renew();
            cur.dy[i].renew();
            float t[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xh = cur.x[i].get(e) * rstd;
                t[e] = (cur.dy[i].get(e) * w[i][e] - xh * s) * rstd;
            }
            if (n.add) {
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] += cur.add[i].get(e);
            }
            store8(dx + c, VEC ? 8 : left, t);
        }
        cur = nxt;
    }
    if (!n.part) return;
    float* part = n.part + (int64_t)blockIdx.x * n.cols;
    if constexpr (RPB > 1) {
        // the sums of waves that hold the same columns, halved each time, in
        // fixed order
        const int grp = threadIdx.x / LPR;
#pragma unroll
        for (int half = RPB / 2; half >= 1; half /= 2) {
            if (grp >= half && grp < 2 * half) {
                float* o = col + (grp - half) * CW;
#pragma unroll
                for (int i = 0; i < NCH; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[(i * LPR + lane) * 8 + e] = dw[i][e];
            }
            __syncthreads();
            if (grp < half) {
                const float* o = col + grp * CW;
#pragma unroll
                for (int i = 0; i < NCH; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) dw[i][e] += o[(i * LPR + lane) * 8 + e];
            }
            __syncthreads();
        }
        if (grp != 0) return;
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = (i * LPR + lane) * 8;
        if (c < n.cols) store8(part + c, n.cols - c, dw[i]);
    }
}

// dx of rows of any length, one workgroup each.
template <typename T>
__global__ __launch_bounds__(256) void k_rms_backward_wide(const RmsBackward n) {
    __shared__ float red[8];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(n.x) + row * n.ld_x;
    const T* dy = static_cast<const T*>(n.dy) + row * n.ld_y;
    const float rstd = n.rstd[row];
    float s = 0.f;
    auto chunk = [&](int c, float (&xh)[8], float (&g)[8]) {
        const int left = n.cols - c;
        float w[8];
        load8(x + c, left, xh);
        load8(dy + c, left, g);
        if (n.weight) load8(n.weight + c, left, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            xh[e] *= rstd;
            if (n.weight) g[e] *= w[e];
        }
    };
    for (int c = threadIdx.x * 8; c < n.cols; c += 2048) {
        float xh[8], g[8];
        chunk(c, xh, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(g[e], xh[e], s);
    }
    s = row_sum<4>(s, red) * (1.f / (float)n.cols);
    T* dx = static_cast<T*>(n.dx) + row * n.ld_dx;
    const T* add = n.add ? static_cast<const T*>(n.add) + row * n.ld_add : nullptr;
    for (int c = threadIdx.x * 8; c < n.cols; c += 2048) {
        float xh[8], g[8], a[8];
        chunk(c, xh, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = (g[e] - xh[e] * s) * rstd;
        if (add) {
            load8(add + c, n.cols - c, a);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] += a[e];
        }
        store8(dx + c, n.cols - c, g);
    }
}

// The column sums for rows of any length: 256 columns (32 lanes x 8) of every
// n.blocks-th group of 8 rows.
template <typename T>
__global__ __launch_bounds__(256) void k_rms_columns(const RmsBackward n) {
    __shared__ float red[8][32][9];
    const int lane = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int c = blockIdx.x * 256 + lane * 8;
    float dw[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[e] = 0.f;
    if (c < n.cols) {
        for (int64_t r = (int64_t)blockIdx.y * 8 + rl; r < n.rows; r += (int64_t)n.blocks * 8) {
            float x[8], g[8];
            load8(static_cast<const T*>(n.x) + r * n.ld_x + c, n.cols - c, x);
            load8(static_cast<const T*>(n.dy) + r * n.ld_y + c, n.cols - c, g);
            const float rstd = n.rstd[r];
#pragma unroll
            for (int e = 0; e < 8; ++e) dw[e] = fmaf(g[e], x[e] * rstd, dw[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) red[rl][lane][e] = dw[e];
    __syncthreads();
    const int l = threadIdx.x >> 3, e = threadIdx.x & 7;
    const int cc = blockIdx.x * 256 + l * 8 + e;
    if (cc >= n.cols) return;
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) s += red[r][l][e];
    n.part[(int64_t)blockIdx.y * n.cols + cc] = s;
}

// dweight (+)= the partial rows: 32 columns a workgroup, each of its 32 half waves
// a run of the rows, added in order.
__global__ __launch_bounds__(1024) void k_rms_join(const RmsSums n) {
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, half = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    const int per = (n.blocks + 31) / 32;
    const int b1 = (half + 1) * per < n.blocks ? (half + 1) * per : n.blocks;
    float s = 0.f;
    if (c < n.cols) {
#pragma unroll 8
        for (int b = half * per; b < b1; ++b) s += n.part[(int64_t)b * n.cols + c];
    }
    red[half][lane] = s;
    __syncthreads();
    if (half == 0 && c < n.cols) {
        s = red[0][lane];
#pragma unroll
        for (int w = 1; w < 32; ++w) s += red[w][lane];
        n.dweight[c] = n.accumulate ? n.dweight[c] + s : s;
    }
}

template <typename T, bool VEC, bool ADD, int F>
void forward_rows(const RmsForward& n, hipStream_t st) {
    const unsigned g4 = ((unsigned)n.rows + 3) / 4, g1 = (unsigned)n.rows;
    if (n.cols <= 512)
        k_rms_forward<T, 1, 1, VEC, ADD, F><<<g4, 256, 0, st>>>(n);
    else if (n.cols <= 1024)
        k_rms_forward<T, 2, 1, VEC, ADD, F><<<g4, 256, 0, st>>>(n);
    else if (n.cols <= 2048)
        k_rms_forward<T, 4, 1, VEC, ADD, F><<<g4, 256, 0, st>>>(n);
    else if (n.cols <= 4096)
        k_rms_forward<T, 2, 4, VEC, ADD, F><<<g1, 256, 0, st>>>(n);
    else if (n.cols <= kBlockCols)
        k_rms_forward<T, 4, 4, VEC, ADD, F><<<g1, 256, 0, st>>>(n);
    else
        k_rms_forward_wide<T, ADD, F><<<g1, 256, 0, st>>>(n);
}

template <typename T, bool ADD, int F>
void forward_v(const RmsForward& n, hipStream_t st) {
    if (n.cols % 8 == 0)
        forward_rows<T, true, ADD, F>(n, st);
    else
        forward_rows<T, false, ADD, F>(n, st);
}
template <typename T, int F>
void forward_a(const RmsForward& n, hipStream_t st) {
    if (n.add)
        forward_v<T, true, F>(n, st);
    else
        forward_v<T, false, F>(n, st);
}
template <typename T>
hipError_t forward_t(const RmsForward& n, int format, hipStream_t st) {
    if (format == EIGHT_NONE)
        forward_a<T, EIGHT_NONE>(n, st);
    else if (format == EIGHT_E4M3)
        forward_a<T, EIGHT_E4M3>(n, st);
    else
        forward_a<T, EIGHT_E5M2>(n, st);
    return hipGetLastError();
}

template <typename T, bool VEC>
void backward_rows(const RmsBackward& n, hipStream_t st) {
    const unsigned b = (unsigned)n.blocks;
    if (n.cols <= 512)
        k_rms_backward<T, 1, 1, VEC><<<b, 256, 0, st>>>(n);
    else if (n.cols <= 1024)
        k_rms_backward<T, 2, 1, VEC><<<b, 256, 0, st>>>(n);
    else if (n.cols <= 2048)
        k_rms_backward<T, 2, 2, VEC><<<b, 256, 0, st>>>(n);
    else if (n.cols <= 4096)
        k_rms_backward<T, 2, 4, VEC><<<b, 256, 0, st>>>(n);
    else
        k_rms_backward<T, 2, 8, VEC><<<b, 512, 0, st>>>(n);
}

template <typename T>
hipError_t backward_t(const RmsBackward& n, hipStream_t st) {
    if (n.cols > kBlockCols) {
        if (n.part) {
            k_rms_columns<T><<<dim3((unsigned)((n.cols + 255) / 256), (unsigned)n.blocks), 256, 0, st>>>(n);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        k_rms_backward_wide<T><<<(unsigned)n.rows, 256, 0, st>>>(n);
    } else if (n.cols % 8 == 0) {
        backward_rows<T, true>(n, st);
    } else {
        backward_rows<T, false>(n, st);
    }
    return hipGetLastError();
}

}  // namespace

// Workgroups of the backward pass, each with a partial row: two or three a CU, and at
// least 8 rows each, so that a row's next one is on the way while it is summed. A call in
// us, in 256, 512, 768 and 1024 workgroups: 16384 x 1600 bf16 66, 49, 45, 46; 16384 x
// 1001 bf16 75, 47, 40, 51; 16384 x 1600 float32 90, 80, 84, 91; 8192 x 6400 bf16 (8 waves
// a workgroup) 95, 83, 95, 89.
int rms_backward_blocks(int64_t rows, int64_t cols, int dtype) {
    if (rows == 0) return 0;
    const int64_t b = cols <= kBlockCols ? rows / 8 : rows / 64;
    const int64_t most = cols > kBlockCols ? 64 : cols > 4096 || dtype == 2 ? 512 : 768;
    return (int)(b < 1 ? 1 : b < most ? b : most);
}

hipError_t launch_rms_forward(const RmsForward& n, int dtype, int format, hipStream_t st) {
    return dtype == 0   ? forward_t<bf16>(n, format, st)
           : dtype == 1 ? forward_t<f16>(n, format, st)
                        : forward_t<float>(n, format, st);
}

hipError_t launch_rms_backward(const RmsBackward& n, int dtype, hipStream_t st) {
    return dtype == 0 ? backward_t<bf16>(n, st) : dtype == 1 ? backward_t<f16>(n, st) : backward_t<float>(n, st);
}

hipError_t launch_rms_sums(const RmsSums& n, hipStream_t st) {
    k_rms_join<<<(unsigned)((n.cols + 31) / 32), 1024, 0, st>>>(n);
    return hipGetLastError();
}

}  // namespace muon
