// Layer norm over rows, forward and backward, on gfx950. Bound by HBM: the
// forward pass reads x once and writes y once, the backward pass reads dy, x
// (and the residual's gradient) once and writes dx once.
//
//  * A row lives in registers between its sums and its output: one wave holds
//    a row of up to 2048 columns (4 rows a workgroup), a workgroup of 4 waves
//    one of up to 8192, in chunks of 8 consecutive elements a lane. Longer rows
//    are read again from cache (k_norm_*_wide).
//  * Statistics in fp32, centred: the mean first, then the squares of x - mean
//    (both from registers), so that a mean far from 0 costs no digits.
//  * Weight gradients: a wave keeps the sums of dy xhat and dy of its own
//    columns in registers over all the rows it goes through, the workgroup
//    adds its waves' sums in wave order through LDS and writes one partial
//    row, and a second kernel adds the partial rows in order (no atomics: the
//    same bits every run).

#include "layer_device.hpp"

namespace muon {

namespace {

// Sum over the lanes that share a row: a wave (WPR = 1) or the workgroup.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
    if constexpr (WPR == 1)
        return wave_sum(v);
    else
        return block_sum_256(v, red);
}

// Two sums at once.
template <int WPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float* red) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        a += __shfl_xor(a, off, 64);
        b += __shfl_xor(b, off, 64);
    }
    if constexpr (WPR > 1) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        __syncthreads();
        if (lane == 0) {
            red[wave] = a;
            red[4 + wave] = b;
        }
        __syncthreads();
        a = ((red[0] + red[1]) + red[2]) + red[3];
        b = ((red[4] + red[5]) + red[6]) + red[7];
    }
}

template <typename T, int NCH, int WPR>
__global__ __launch_bounds__(256) void k_norm_forward(const NormArgs n) {
    __shared__ float red[8];
    constexpr int LPR = 64 * WPR;  // lanes per row
    const int lane = threadIdx.x % LPR;
    const int64_t row = (int64_t)blockIdx.x * (4 / WPR) + threadIdx.x / LPR;
    if (row >= n.rows) return;  // a whole wave (WPR = 1) or never (WPR = 4)
    const T* x = static_cast<const T*>(n.x) + row * n.ld_x;
    T* y = static_cast<T*>(n.y) + row * n.ld_y;
    const float inv = 1.f / (float)n.cols;
    float v[NCH][8];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = (i * LPR + lane) * 8;
        load8(x + c, n.cols - c, n.vec, v[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v[i][e];
    }
    const float mean = row_sum<WPR>(s, red) * inv;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int left = n.cols - (i * LPR + lane) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[i][e] = e < left ? v[i][e] - mean : 0.f;
            q = fmaf(v[i][e], v[i][e], q);
        }
    }
    const float rstd = 1.f / sqrtf(row_sum<WPR>(q, red) * inv + n.eps);
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = (i * LPR + lane) * 8;
        const int left = n.cols - c;
        if (left <= 0) continue;
        float w[8], b[8];
        if (n.weight) load8(n.weight + c, left, n.vec_w, w);
        if (n.bias) load8(n.bias + c, left, n.vec_w, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float t = v[i][e] * rstd;
            if (n.weight) t *= w[e];
            if (n.bias) t += b[e];
            v[i][e] = t;
        }
        store8(y + c, left, n.vec, v[i]);
    }
    if (lane == 0) {
        n.mean[row] = mean;
        n.rstd[row] = rstd;
    }
}

// Rows of any length, one workgroup each, read three times (twice from cache).
template <typename T>
__global__ __launch_bounds__(256) void k_norm_forward_wide(const NormArgs n) {
    __shared__ float red[8];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(n.x) + row * n.ld_x;
    T* y = static_cast<T*>(n.y) + row * n.ld_y;
    const float inv = 1.f / (float)n.cols;
    float s = 0.f;
    for (int c = threadIdx.x * 8; c < n.cols; c += 2048) {
        float v[8];
        load8(x + c, n.cols - c, n.vec, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v[e];
    }
    const float mean = block_sum_256(s, red) * inv;
    float q = 0.f;
    for (int c = threadIdx.x * 8; c < n.cols; c += 2048) {
        float v[8];
        load8(x + c, n.cols - c, n.vec, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = c + e < n.cols ? v[e] - mean : 0.f;
            q = fmaf(d, d, q);
        }
    }
    const float rstd = 1.f / sqrtf(block_sum_256(q, red) * inv + n.eps);
    for (int c = threadIdx.x * 8; c < n.cols; c += 2048) {
        const int left = n.cols - c;
        float v[8], w[8], b[8];
        load8(x + c, left, n.vec, v);
        if (n.weight) load8(n.weight + c, left, n.vec_w, w);
        if (n.bias) load8(n.bias + c, left, n.vec_w, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] = (v[e] - mean) * rstd;
            if (n.weight) v[e] *= w[e];
            if (n.bias) v[e] += b[e];
        }
        store8(y + c, left, n.vec, v);
    }
    if (threadIdx.x == 0) {
        n.mean[row] = mean;
        n.rstd[row] = rstd;
    }
}

// dx = rstd (g - mean(g) - xhat mean(g xhat)) + add with g = dy w, and the
// workgroup's sums of dy xhat and dy per column.
template <typename T, int NCH, int WPR>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) void k_norm_backward(const NormArgs n) {
    constexpr int LPR = 64 * WPR;
    constexpr int RPB = 4 / WPR;  // rows a workgroup works on at once
    __shared__ float red[8];
    __shared__ float col[WPR == 1 ? 2 * NCH * 512 : 1];
    const int lane = threadIdx.x % LPR;
    const float inv = 1.f / (float)n.cols;
    float w[NCH][8], dw[NCH][8], db[NCH][8];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = (i * LPR + lane) * 8;
        if (n.weight) {
            load8(n.weight + c, n.cols - c, n.vec_w, w[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[i][e] = 1.f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = db[i][e] = 0.f;
    }
    const int64_t step = (int64_t)gridDim.x * RPB;
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR; row < n.rows; row += step) {
        const T* x = static_cast<const T*>(n.x) + row * n.ld_x;
        const T* dy = static_cast<const T*>(n.dy) + row * n.ld_y;
        const float mean = n.mean[row], rstd = n.rstd[row];
        float xh[NCH][8], g[NCH][8];
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = (i * LPR + lane) * 8;
            load8(x + c, n.cols - c, n.vec, xh[i]);
            load8(dy + c, n.cols - c, n.vec, g[i]);
        }
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            // columns past the row's end have dy = 0, so they add nothing to any sum
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xh[i][e] = (xh[i][e] - mean) * rstd;
                dw[i][e] = fmaf(g[i][e], xh[i][e], dw[i][e]);
                db[i][e] += g[i][e];
                g[i][e] *= w[i][e];
                s0 += g[i][e];
                s1 = fmaf(g[i][e], xh[i][e], s1);
            }
        }
        row_sum2<WPR>(s0, s1, red);
        s0 *= inv;
        s1 *= inv;
        T* dx = static_cast<T*>(n.dx) + row * n.ld_dx;
        const T* add = n.add ? static_cast<const T*>(n.add) + row * n.ld_r : nullptr;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = (i * LPR + lane) * 8;
            const int left = n.cols - c;
            if (left <= 0) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) g[i][e] = (g[i][e] - fmaf(xh[i][e], s1, s0)) * rstd;
            if (add) {
                float a[8];
                load8(add + c, left, n.vec, a);
#pragma unroll
                for (int e = 0; e < 8; ++e) g[i][e] += a[e];
            }
            store8(dx + c, left, n.vec, g[i]);
        }
    }
    if (!n.part) return;
    float* part = n.part + (int64_t)blockIdx.x * 2 * n.cols;
    if constexpr (WPR == 1) {
        // the four waves' sums, added in wave order
        constexpr int CW = NCH * 512;
        for (int wv = 0; wv < 4; ++wv) {
            if ((threadIdx.x >> 6) == wv) {
#pragma unroll
                for (int i = 0; i < NCH; ++i) {
                    const int c = (i * 64 + lane) * 8;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        col[c + e] = (wv ? col[c + e] : 0.f) + dw[i][e];
                        col[CW + c + e] = (wv ? col[CW + c + e] : 0.f) + db[i][e];
                    }
                }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < n.cols; c += 256) {
            part[c] = col[c];
            part[n.cols + c] = col[CW + c];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = (i * LPR + lane) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < n.cols) {
                    part[c + e] = dw[i][e];
                    part[n.cols + c + e] = db[i][e];
                }
        }
    }
}

// dx of rows of any length, one workgroup each.
template <typename T>
__global__ __launch_bounds__(256) void k_norm_backward_wide(const NormArgs n) {
    __shared__ float red[8];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(n.x) + row * n.ld_x;
    const T* dy = static_cast<const T*>(n.dy) + row * n.ld_y;
    const float mean = n.mean[row], rstd = n.rstd[row], inv = 1.f / (float)n.cols;
    float s0 = 0.f, s1 = 0.f;
    auto chunk = [&](int c, float (&xh)[8], float (&g)[8]) {
        const int left = n.cols - c;
        float w[8];
        load8(x + c, left, n.vec, xh);
        load8(dy + c, left, n.vec, g);
        if (n.weight) load8(n.weight + c, left, n.vec_w, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            xh[e] = (xh[e] - mean) * rstd;
            if (n.weight) g[e] *= w[e];
        }
    };
    for (int c = threadIdx.x * 8; c < n.cols; c += 2048) {
        float xh[8], g[8];
        chunk(c, xh, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            s0 += g[e];
            s1 = fmaf(g[e], xh[e], s1);
        }
    }
    row_sum2<4>(s0, s1, red);
    s0 *= inv;
    s1 *= inv;
    T* dx = static_cast<T*>(n.dx) + row * n.ld_dx;
    const T* add = n.add ? static_cast<const T*>(n.add) + row * n.ld_r : nullptr;
    for (int c = threadIdx.x * 8; c < n.cols; c += 2048) {
        float xh[8], g[8], a[8];
        chunk(c, xh, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = (g[e] - fmaf(xh[e], s1, s0)) * rstd;
        if (add) {
            load8(add + c, n.cols - c, n.vec, a);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] += a[e];
        }
        store8(dx + c, n.cols - c, n.vec, g);
    }
}

// The column sums for rows of any length: 256 columns (32 lanes x 8) of every
// n.blocks-th group of 8 rows.
template <typename T>
__global__ __launch_bounds__(256) void k_norm_columns(const NormArgs n) {
    __shared__ float red[2][8][32][9];
    const int lane = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int c = blockIdx.x * 256 + lane * 8;
    float dw[8], db[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[e] = db[e] = 0.f;
    if (c < n.cols) {
        for (int64_t r = (int64_t)blockIdx.y * 8 + rl; r < n.rows; r += (int64_t)n.blocks * 8) {
            float x[8], g[8];
            load8(static_cast<const T*>(n.x) + r * n.ld_x + c, n.cols - c, n.vec, x);
            load8(static_cast<const T*>(n.dy) + r * n.ld_y + c, n.cols - c, n.vec, g);
            const float mean = n.mean[r], rstd = n.rstd[r];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dw[e] = fmaf(g[e], (x[e] - mean) * rstd, dw[e]);
                db[e] += g[e];
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        red[0][rl][lane][e] = dw[e];
        red[1][rl][lane][e] = db[e];
    }
    __syncthreads();
    const int l = threadIdx.x >> 3, e = threadIdx.x & 7;
    const int cc = blockIdx.x * 256 + l * 8 + e;
    if (cc >= n.cols) return;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < 8; ++r) s += red[k][r][l][e];
        n.part[((int64_t)blockIdx.y * 2 + k) * n.cols + cc] = s;
    }
}

// dweight, dbias (+)= the partial rows, added in order: 64 columns a
// workgroup, each wave a quarter of the partial rows.
__global__ __launch_bounds__(256) void k_norm_join(const NormArgs n) {
    __shared__ float red[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    float* out = blockIdx.y ? n.dbias : n.dweight;
    if (!out) return;
    const int per = (n.blocks + 3) / 4;
    const int b1 = (wave + 1) * per < n.blocks ? (wave + 1) * per : n.blocks;
    float s = 0.f;
    if (c < n.cols) {
#pragma unroll 8
        for (int b = wave * per; b < b1; ++b) s += n.part[((int64_t)b * 2 + blockIdx.y) * n.cols + c];
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < n.cols) {
        s = ((red[0][lane] + red[1][lane]) + red[2][lane]) + red[3][lane];
        out[c] = n.accumulate ? out[c] + s : s;
    }
}

constexpr int kWaveCols = 2048;   // a wave's registers hold a row
constexpr int kBlockCols = 8192;  // a workgroup's do

template <typename T>
hipError_t forward_t(const NormArgs& n, hipStream_t st) {
    if (n.rows == 0) return hipSuccess;
    const unsigned g4 = (unsigned)((n.rows + 3) / 4), g1 = (unsigned)n.rows;
    if (n.cols <= 512)
        k_norm_forward<T, 1, 1><<<g4, 256, 0, st>>>(n);
    else if (n.cols <= 1024)
        k_norm_forward<T, 2, 1><<<g4, 256, 0, st>>>(n);
    else if (n.cols <= kWaveCols)
        k_norm_forward<T, 4, 1><<<g4, 256, 0, st>>>(n);
    else if (n.cols <= 4096)
        k_norm_forward<T, 2, 4><<<g1, 256, 0, st>>>(n);
    else if (n.cols <= kBlockCols)
        k_norm_forward<T, 4, 4><<<g1, 256, 0, st>>>(n);
    else
        k_norm_forward_wide<T><<<g1, 256, 0, st>>>(n);
    return hipGetLastError();
}

template <typename T>
hipError_t backward_t(const NormArgs& n, hipStream_t st) {
    hipError_t e = hipSuccess;
    if (n.rows > 0) {
        const unsigned b = (unsigned)n.blocks;
        if (n.cols <= 512) {
            k_norm_backward<T, 1, 1><<<b, 256, 0, st>>>(n);
        } else if (n.cols <= 1024) {
            k_norm_backward<T, 2, 1><<<b, 256, 0, st>>>(n);
        } else if (n.cols <= kWaveCols) {
            k_norm_backward<T, 4, 1><<<b, 256, 0, st>>>(n);
        } else if (n.cols <= 4096) {
            k_norm_backward<T, 2, 4><<<b, 256, 0, st>>>(n);
        } else if (n.cols <= kBlockCols) {
            k_norm_backward<T, 4, 4><<<b, 256, 0, st>>>(n);
        } else {
            if (n.part) {
                k_norm_columns<T><<<dim3((unsigned)((n.cols + 255) / 256), b), 256, 0, st>>>(n);
                e = hipGetLastError();
                if (e != hipSuccess) return e;
            }
            k_norm_backward_wide<T><<<(unsigned)n.rows, 256, 0, st>>>(n);
        }
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (n.dweight || n.dbias) {
        k_norm_join<<<dim3((unsigned)((n.cols + 63) / 64), 2), 256, 0, st>>>(n);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace

// Workgroups of the backward pass (each leaves one partial row of column
// sums): up to 512, two for every CU, one row (or 4, a wave each) at a time.
int norm_backward_blocks(int64_t rows, int64_t cols) {
    int64_t b;
    if (cols <= kWaveCols)
        b = (rows + 3) / 4;
    else if (cols <= kBlockCols)
        b = rows;
    else
        b = (rows + 63) / 64;
    const int64_t most = cols <= kBlockCols ? 512 : 64;
    return (int)(b < most ? b : most);
}

hipError_t launch_norm_forward(const NormArgs& n, int dtype, hipStream_t st) {
    return dtype == 0 ? forward_t<bf16>(n, st) : dtype == 1 ? forward_t<f16>(n, st) : forward_t<float>(n, st);
}

hipError_t launch_norm_backward(const NormArgs& n, int dtype, hipStream_t st) {
    return dtype == 0 ? backward_t<bf16>(n, st) : dtype == 1 ? backward_t<f16>(n, st) : backward_t<float>(n, st);
}

}  // namespace muon
