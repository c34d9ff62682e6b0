// Layer norm over rows, forward and backward, on gfx950. Bound by HBM: the
// forward pass reads x once and writes y once, the backward pass reads dy, x
// (and the residual's gradient) once and writes dx once.
//
//  * A row lives in registers between its sums and its output, in chunks of 8
//    consecutive elements a lane: forward one wave holds a row of up to 2048
//    columns and four one of up to 8192; backward, which also holds dy and the
//    next row, one wave 1024, two 2048, four 4096 and eight 8192. Longer rows are
//    read again (k_norm_*_wide): from cache as far as it holds them (bf16, 4096 x
//    8192 and x 8200: forward 23 and 43 us, backward 62 and 105).
//  * Statistics in fp32, centred: the mean first, then the squares of x - mean
//    (both from registers). Where the mean is far from 0 against the spread, what
//    its rounding left in x - mean is taken off too (row_is_far).
//  * Weight gradients: a wave keeps the sums of dy xhat and dy of its own
//    columns in registers over all the rows it goes through, the workgroup
//    adds its waves' sums in wave order through LDS and writes one partial
//    row, and a second kernel adds the partial rows in order (no atomics: the
//    same bits every run).

#include "norm_device.hpp"

namespace muon {

namespace {

// The first mean of a row of up to 8192 columns is off by up to about 46 2^-24 of
// its mean |x| (a lane's strand and the joins), which counts in xhat times mean
// |x| / spread: at most 190 2^-24 up to a mean of four times the spread, and
// without bound beyond (a constant row of 1e5 came out as +-1). Rows beyond take
// one more sum, of x - mean (16384 x 1600 bf16 19.6 -> 19.8 us; taken for every
// row it cost all of them 20.5). q: the mean square of x - mean. No NaN is far,
// nor a row whose squares overflow.
__device__ __forceinline__ bool row_is_far(float mean, float q) { return mean * mean > 16.f * q; }
// r: the mean of x - mean. xhat = (x - mean) rstd + off.
struct Stats {
    float mean, rstd, off;
};
__device__ __forceinline__ Stats row_stats(float mean, float r, float q, float eps) {
    const float var = q - r * r;
    const float rstd = 1.f / sqrtf((var < 0.f ? 0.f : var) + eps);  // a NaN stays one
    return {mean + r, rstd, -r * rstd};
}

// 16-bit rows of up to 2048 columns within 64 registers, 8 waves a SIMD (with 66,
// 16384 x 1601 bf16 25.0 us, against 24.2).
template <typename T, int NCH, int WPR, bool VEC>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(sizeof(T) == 2 && WPR == 1 ? 8 : 1))) void
k_norm_forward(const NormForward n) {
    __shared__ float red[16];
    constexpr int LPR = 64 * WPR;  // lanes per row
    const int lane = threadIdx.x % LPR;
    const int64_t row = (int64_t)blockIdx.x * (4 / WPR) + threadIdx.x / LPR;
    if (row >= n.rows) return;  // a whole wave (WPR = 1) or never (WPR = 4)
    const T* x = static_cast<const T*>(n.x) + row * n.ld_x;
    T* y = static_cast<T*>(n.y) + row * n.ld_y;
    const float inv = 1.f / (float)n.cols;
    Raw<T> v[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = (i * LPR + lane) * 8;
        v[i].template load<VEC>(x + c, n.cols - c);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v[i].get(e);
    const float mean = row_sum<WPR>(s, red) * inv;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int left = n.cols - (i * LPR + lane) * 8;
        if (VEC ? left > 0 : left >= 8) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = v[i].get(e) - mean;
                q = fmaf(d, d, q);
            }
        } else if (!VEC) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = e < left ? v[i].get(e) - mean : 0.f;
                q = fmaf(d, d, q);
            }
        }
    }
    q = row_sum<WPR>(q, red + 8) * inv;
    float r = 0.f;
    if (row_is_far(mean, q)) {  // for all lanes of the row alike
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int left = n.cols - (i * LPR + lane) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) r += (VEC ? left > 0 : e < left) ? v[i].get(e) - mean : 0.f;
        }
        r = row_sum<WPR>(r, red) * inv;
    }
    const Stats st = row_stats(mean, r, q, n.eps);
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = (i * LPR + lane) * 8;
        const int left = n.cols - c;
        if (left <= 0) continue;
        float t[8], u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = (v[i].get(e) - mean) * st.rstd;
        if (st.off != 0.f) {
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] += st.off;
        }
        if (n.weight) {
            load8(n.weight + c, left, u);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] *= u[e];
        }
        if (n.bias) {
            load8(n.bias + c, left, u);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] += u[e];
        }
        stream8(y + c, VEC ? 8 : left, t);
    }
    if (lane == 0) {
        n.mean[row] = st.mean;
        n.rstd[row] = st.rstd;
    }
}

// Rows of any length, one workgroup each, read three times (twice from cache).
template <typename T>
__global__ __launch_bounds__(256) void k_norm_forward_wide(const NormForward n) {
    __shared__ float red[16];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(n.x) + row * n.ld_x;
    T* y = static_cast<T*>(n.y) + row * n.ld_y;
    const float inv = 1.f / (float)n.cols;
    float s = 0.f;
    for (int c = threadIdx.x * 8; c < n.cols; c += 2048) {
        float v[8];
        load8(x + c, n.cols - c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v[e];
    }
    const float mean = row_sum<4>(s, red) * inv;
    // the reads take the time here, and strands are longer: every row takes the
    // sum that row_is_far asks for, unless its squares overflow
    float q = 0.f, r = 0.f;
    for (int c = threadIdx.x * 8; c < n.cols; c += 2048) {
        float v[8];
        load8(x + c, n.cols - c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = c + e < n.cols ? v[e] - mean : 0.f;
            r += d;
            q = fmaf(d, d, q);
        }
    }
    row_sum2<4>(r, q, red + 8);
    q *= inv;
    r = q < __builtin_inff() ? r * inv : 0.f;
    const Stats st = row_stats(mean, r, q, n.eps);
    for (int c = threadIdx.x * 8; c < n.cols; c += 2048) {
        const int left = n.cols - c;
        float v[8], w[8], b[8];
        load8(x + c, left, v);
        if (n.weight) load8(n.weight + c, left, w);
        if (n.bias) load8(n.bias + c, left, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] = fmaf(v[e] - mean, st.rstd, st.off);
            if (n.weight) v[e] *= w[e];
            if (n.bias) v[e] += b[e];
        }
        store8(y + c, left, v);
    }
    if (threadIdx.x == 0) {
        n.mean[row] = st.mean;
        n.rstd[row] = st.rstd;
    }
}

// dx = rstd (g - mean(g) - xhat mean(g xhat)) + add with g = dy w, and the
// workgroup's sums of dy xhat and dy per column. WPR waves share a row, and go
// through their rows with the next row's x, dy and add on the way in; these
// stay as loaded and are widened twice, so that a lane of two chunks leaves
// room for them at two or three waves a SIMD (four chunks a lane, one wave a
// row of 2048, spilled: 90 us at 16384 x 1600 bf16, against 52 without the
// next row on the way). VEC: rows are whole chunks.
template <typename T, int NCH, int WPR, bool VEC>
__global__ __launch_bounds__(WPR == 8 ? 512 : 256) __attribute__((amdgpu_waves_per_eu(2))) void k_norm_backward(
    const NormBackward n) {
    constexpr int LPR = 64 * WPR;
    constexpr int WAVES = WPR == 8 ? 8 : 4;
    constexpr int RPB = WAVES / WPR;  // rows a workgroup works on at once
    constexpr int CW = NCH * LPR * 8;
    __shared__ float red[2][2 * WAVES];
    __shared__ float col[RPB > 1 ? RPB / 2 * 2 * CW : 1];
    const int lane = threadIdx.x % LPR;
    const float inv = 1.f / (float)n.cols;
    float w[NCH][8], dw[NCH][8], db[NCH][8];
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
        for (int e = 0; e < 8; ++e) dw[i][e] = db[i][e] = 0.f;
    }
    struct Row {
        Raw<T> x[NCH], dy[NCH], add[NCH];
        float mean, rstd;
    };
    auto fetch = [&](Row& r, int64_t row) {
        const T* x = static_cast<const T*>(n.x) + row * n.ld_x;
        const T* dy = static_cast<const T*>(n.dy) + row * n.ld_y;
        const T* add = static_cast<const T*>(n.add) + row * n.ld_r;
        r.mean = n.mean[row];
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
    // the same number of turns for every wave: with no row left, dy and so
    // every sum is left as it is
    const int64_t turns = (n.rows + step - 1) / step;
    for (int64_t t = 0; t < turns; ++t, row += step) {
        const bool live = row < n.rows;
        if (row + step < n.rows) fetch(nxt, row + step);
        const float rstd = cur.rstd, shift = -cur.mean;
        // x and dy are 0 past the row's end, which adds nothing to any sum as long
        // as the xhat there, -mean rstd, is finite. For an all but constant row far
        // from 0 it is not: the row's first element takes the place of x then. (A
        // masked second copy of the sums, or loads that always put an element of
        // the row there, take more registers: 16384 x 1601 bf16 87 us, against 79)
        if (live && !(fabsf(shift * rstd) < __builtin_inff())) {
            const T first = static_cast<const T*>(n.x)[row * n.ld_x];
#pragma unroll
            for (int i = 0; i < NCH; ++i) cur.x[i].fill(n.cols - (i * LPR + lane) * 8, first);
        }
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            if (!live) break;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xh = (cur.x[i].get(e) + shift) * rstd, d = cur.dy[i].get(e);
                dw[i][e] = fmaf(d, xh, dw[i][e]);
                db[i][e] += d;
                const float g = d * w[i][e];
                s0 += g;
                s1 = fmaf(g, xh, s1);
            }
        }
        row_sum2<WPR>(s0, s1, red[t & 1]);
        s0 *= inv;
        s1 *= inv;
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
                const float xh = (cur.x[i].get(e) + shift) * rstd;
                t[e] = (cur.dy[i].get(e) * w[i][e] - fmaf(xh, s1, s0)) * rstd;
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
    float* part = n.part + (int64_t)blockIdx.x * 2 * n.cols;
    if constexpr (RPB > 1) {
        // the sums of waves that hold the same columns, halved each time, in
        // fixed order
        const int grp = threadIdx.x / LPR;
#pragma unroll
        for (int half = RPB / 2; half >= 1; half /= 2) {
            if (grp >= half && grp < 2 * half) {
                float* o = col + (grp - half) * 2 * CW;
#pragma unroll
                for (int i = 0; i < NCH; ++i) {
                    const int c = (i * LPR + lane) * 8;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        o[c + e] = dw[i][e];
                        o[CW + c + e] = db[i][e];
                    }
                }
            }
            __syncthreads();
            if (grp < half) {
                const float* o = col + grp * 2 * CW;
#pragma unroll
                for (int i = 0; i < NCH; ++i) {
                    const int c = (i * LPR + lane) * 8;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        dw[i][e] += o[c + e];
                        db[i][e] += o[CW + c + e];
                    }
                }
            }
            __syncthreads();
        }
        if (grp != 0) return;
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = (i * LPR + lane) * 8;
        if (c < n.cols) {
            store8(part + c, n.cols - c, dw[i]);
            store8(part + n.cols + c, n.cols - c, db[i]);
        }
    }
}

// dx of rows of any length, one workgroup each.
template <typename T>
__global__ __launch_bounds__(256) void k_norm_backward_wide(const NormBackward n) {
    __shared__ float red[8];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(n.x) + row * n.ld_x;
    const T* dy = static_cast<const T*>(n.dy) + row * n.ld_y;
    const float mean = n.mean[row], rstd = n.rstd[row], inv = 1.f / (float)n.cols;
    float s0 = 0.f, s1 = 0.f;
    auto chunk = [&](int c, float (&xh)[8], float (&g)[8]) {
        const int left = n.cols - c;
        float w[8];
        load8(x + c, left, xh);
        load8(dy + c, left, g);
        if (n.weight) load8(n.weight + c, left, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            xh[e] = (e < left ? xh[e] - mean : 0.f) * rstd;  // 0 past the row's end, where g is
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
__global__ __launch_bounds__(256) void k_norm_columns(const NormBackward n) {
    __shared__ float red[2][8][32][9];
    const int lane = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int c = blockIdx.x * 256 + lane * 8;
    float dw[8], db[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[e] = db[e] = 0.f;
    if (c < n.cols) {
        for (int64_t r = (int64_t)blockIdx.y * 8 + rl; r < n.rows; r += (int64_t)n.blocks * 8) {
            float x[8], g[8];
            load8(static_cast<const T*>(n.x) + r * n.ld_x + c, n.cols - c, x);
            load8(static_cast<const T*>(n.dy) + r * n.ld_y + c, n.cols - c, g);
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

// dweight, dbias (+)= the partial rows: 64 columns a workgroup, each of its 16
// waves a run of the rows, added in order.
__global__ __launch_bounds__(1024) void k_norm_join(const NormSums n) {
    __shared__ float red[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    float* out = blockIdx.y ? n.dbias : n.dweight;
    if (!out) return;
    const int per = (n.blocks + 15) / 16;
    const int b1 = (wave + 1) * per < n.blocks ? (wave + 1) * per : n.blocks;
    float s = 0.f;
    if (c < n.cols) {
#pragma unroll 16
        for (int b = wave * per; b < b1; ++b) s += n.part[((int64_t)b * 2 + blockIdx.y) * n.cols + c];
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < n.cols) {
        s = red[0][lane];
#pragma unroll
        for (int w = 1; w < 16; ++w) s += red[w][lane];
        out[c] = n.accumulate ? out[c] + s : s;
    }
}

constexpr int kBlockCols = 8192;  // longest rows that live in registers

template <typename T, bool VEC>
void forward_rows(const NormForward& n, hipStream_t st) {
    const unsigned g4 = ((unsigned)n.rows + 3) / 4, g1 = (unsigned)n.rows;
    if (n.cols <= 512)
        k_norm_forward<T, 1, 1, VEC><<<g4, 256, 0, st>>>(n);
    else if (n.cols <= 1024)
        k_norm_forward<T, 2, 1, VEC><<<g4, 256, 0, st>>>(n);
    else if (n.cols <= 2048)
        k_norm_forward<T, 4, 1, VEC><<<g4, 256, 0, st>>>(n);
    else if (n.cols <= 4096)
        k_norm_forward<T, 2, 4, VEC><<<g1, 256, 0, st>>>(n);
    else
        k_norm_forward<T, 4, 4, VEC><<<g1, 256, 0, st>>>(n);
}

template <typename T, bool VEC>
void backward_rows(const NormBackward& n, hipStream_t st) {
    const unsigned b = (unsigned)n.blocks;
    if (n.cols <= 512)
        k_norm_backward<T, 1, 1, VEC><<<b, 256, 0, st>>>(n);
    else if (n.cols <= 1024)
        k_norm_backward<T, 2, 1, VEC><<<b, 256, 0, st>>>(n);
    else if (n.cols <= 2048)
        k_norm_backward<T, 2, 2, VEC><<<b, 256, 0, st>>>(n);
    else if (n.cols <= 4096)
        k_norm_backward<T, 2, 4, VEC><<<b, 256, 0, st>>>(n);
    else
        k_norm_backward<T, 2, 8, VEC><<<b, 512, 0, st>>>(n);
}

template <typename T>
hipError_t forward_t(const NormForward& n, hipStream_t st) {
    if (n.cols > kBlockCols)
        k_norm_forward_wide<T><<<(unsigned)n.rows, 256, 0, st>>>(n);
    else if (n.cols % 8 == 0)
        forward_rows<T, true>(n, st);
    else
        forward_rows<T, false>(n, st);
    return hipGetLastError();
}

template <typename T>
hipError_t backward_t(const NormBackward& n, hipStream_t st) {
    if (n.cols > kBlockCols) {
        if (n.part) {
            k_norm_columns<T><<<dim3((unsigned)((n.cols + 255) / 256), (unsigned)n.blocks), 256, 0, st>>>(n);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        k_norm_backward_wide<T><<<(unsigned)n.rows, 256, 0, st>>>(n);
    } else if (n.cols % 8 == 0) {
        backward_rows<T, true>(n, st);
    } else {
        backward_rows<T, false>(n, st);
    }
    return hipGetLastError();
}

}  // namespace

// Workgroups of the backward pass (each leaves one partial row of column sums),
// of at least 8 rows. More of them hide more latency as long as all run at once,
// but each brings a row to the join. us of both at 16384 rows with at most 512,
// 768, 1024 and 1536: bf16 x 1600 42.6, 40.5, 47.6, 46.8; x 512 17.2, 17.9, 18.7,
// 21.2; x 4096 84, 87, 92, 95; bf16 x 1601 79, 102, 85, 92; fp32 x 1600 63, 74,
// 69, 73; x 512 24.8, 26.9, 28.8, 30.9. So three a CU for 16-bit rows of whole
// chunks and two for the others, whose registers leave room for no more (rows of
// up to 512 columns do, without a gain); beyond 4096 columns one of 8 waves. For
// rows longer than registers hold, runs of at least 64 rows.
int norm_backward_blocks(int64_t rows, int64_t cols, int dtype) {
    if (rows == 0) return 0;
    const int64_t b = cols <= kBlockCols ? rows / 8 : rows / 64;
    const int64_t most = cols > kBlockCols ? 64 : cols > 4096 ? 256 : dtype != 2 && cols % 8 == 0 ? 768 : 512;
    return (int)(b < 1 ? 1 : b < most ? b : most);
}

hipError_t launch_norm_forward(const NormForward& n, int dtype, hipStream_t st) {
    return dtype == 0 ? forward_t<bf16>(n, st) : dtype == 1 ? forward_t<f16>(n, st) : forward_t<float>(n, st);
}

hipError_t launch_norm_backward(const NormBackward& n, int dtype, hipStream_t st) {
    return dtype == 0 ? backward_t<bf16>(n, st) : dtype == 1 ? backward_t<f16>(n, st) : backward_t<float>(n, st);
}

hipError_t launch_norm_sums(const NormSums& n, hipStream_t st) {
    k_norm_join<<<dim3((unsigned)((n.cols + 63) / 64), 2), 1024, 0, st>>>(n);
    return hipGetLastError();
}

}  // namespace muon
