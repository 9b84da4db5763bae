// Layer norm, forward and backward.
//
//   mu = mean(x), var = mean((x - mu)^2), rstd = 1 / sqrt(var + eps)
//   xh = (x - mu) rstd,  y = xh w + b
//   g = dy w,  dx = rstd (g - mean(g) - xh mean(g xh))
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Both passes are bound by memory: x is read once and y written once, x and
// dy read once and dx written once.  A row stays in registers between the
// statistics and their use, packed as it came.  Statistics and sums are
// fp32; the variance is that of the centred values (no difference of
// squares), and the only roundings to fewer bits are those of y and dx.
#include <algorithm>

#include "elem.cuh"

namespace moe {
namespace {

constexpr int kMaxCols = 16384;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the row's threads: a warp, or the whole CTA (every thread gets
// it; `red` holds 32 floats and is not used again before the next barrier).
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* red) {
    v = warp_sum(v);
    if (WARP) return v;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return warp_sum(lane < warps ? red[lane] : 0.0f);
}

// A row per warp (WARP) or per CTA; a thread holds CH chunks of E columns.
template <class T, int E, int CH, bool WARP>
__global__ void __launch_bounds__(WARP ? 128 : 1024) layernorm_forward_kernel(const T* __restrict__ x, int64_t rows, int cols,
                                         const float* __restrict__ weight,
                                         const float* __restrict__ bias, float eps,
                                         T* __restrict__ y, float* __restrict__ mean,
                                         float* __restrict__ rstd) {
    __shared__ float red[2][32];
    const int tpr = WARP ? 32 : int(blockDim.x);
    const int t = WARP ? int(threadIdx.x & 31) : int(threadIdx.x);
    const int64_t row =
        WARP ? int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : int64_t(blockIdx.x);
    if (WARP && row >= rows) return;  // whole warps
    const T* xr = x + row * cols;
    Raw<T, E> v[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = (t + j * tpr) * E;
        v[j] = c < cols ? raw_load<T, E>(xr + c) : raw_zero<T, E>();
    }
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        float f[E];
        raw_floats(v[j], f);
#pragma unroll
        for (int i = 0; i < E; ++i) s += f[i];
    }
    const float mu = row_sum<WARP>(s, red[0]) / float(cols);
    float s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        if ((t + j * tpr) * E < cols) {
            float f[E];
            raw_floats(v[j], f);
#pragma unroll
            for (int i = 0; i < E; ++i) s2 = fmaf(f[i] - mu, f[i] - mu, s2);
        }
    }
    const float r = 1.0f / sqrtf(row_sum<WARP>(s2, red[1]) / float(cols) + eps);
    if (t == 0) {
        if (mean) mean[row] = mu;
        if (rstd) rstd[row] = r;
    }
    T* yr = y + row * cols;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = (t + j * tpr) * E;
        if (c < cols) {
            float f[E], w[E], b[E];
            raw_floats(v[j], f);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                w[i] = 1.0f;
                b[i] = 0.0f;
            }
            if (weight) raw_floats(raw_load<float, E>(weight + c), w);
            if (bias) raw_floats(raw_load<float, E>(bias + c), b);
#pragma unroll
            for (int i = 0; i < E; ++i) f[i] = fmaf((f[i] - mu) * r, w[i], b[i]);
            store_floats(yr + c, f);
        }
    }
}

// Rows r, r + gridDim.x, ... of a CTA: a thread keeps its CH chunks' columns
// through all of them, so dw and db gather in registers; one row of partial
// sums per CTA goes to the workspace, where the next kernel adds them in a
// fixed order.
template <class T, class X, int E, int CH>
__global__ void __launch_bounds__(1024) layernorm_backward_kernel(const T* __restrict__ dy, const X* __restrict__ x,
                                          const float* __restrict__ x_scales, int64_t rows,
                                          int cols, int64_t x_pitch,
                                          const float* __restrict__ weight,
                                          const float* __restrict__ mean,
                                          const float* __restrict__ rstd, T* __restrict__ dx,
                                          float* __restrict__ part) {
    __shared__ float red[2][2][32];
    const int t = threadIdx.x, tpr = blockDim.x;
    float dw[CH * E], db[CH * E];
#pragma unroll
    for (int i = 0; i < CH * E; ++i) dw[i] = db[i] = 0.0f;
    int par = 0;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, par ^= 1) {
        const float mu = mean[row], rs = rstd[row];
        float xh[CH * E], g[CH * E];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = (t + j * tpr) * E;
            float xv[E], dv[E], w[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                xv[i] = mu;
                dv[i] = 0.0f;
                w[i] = 1.0f;
            }
            if (c < cols) {
                raw_floats(raw_load<X, E>(x + row * x_pitch + c), xv);
                if constexpr (sizeof(X) == 1) {
                    const float sc = x_scales[int64_t(c / kTile) * rows + row];
#pragma unroll
                    for (int i = 0; i < E; ++i) xv[i] *= sc;
                }
                raw_floats(raw_load<T, E>(dy + row * cols + c), dv);
                if (weight) raw_floats(raw_load<float, E>(weight + c), w);
            }
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float h = (xv[i] - mu) * rs, gv = dv[i] * w[i];
                xh[j * E + i] = h;
                g[j * E + i] = gv;
                s1 += gv;
                s2 = fmaf(gv, h, s2);
                db[j * E + i] += dv[i];
                dw[j * E + i] = fmaf(dv[i], h, dw[j * E + i]);
            }
        }
        // both sums behind one barrier; the other parity's slots are read
        // until the barrier after it
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        const int warps = blockDim.x >> 5, lane = t & 31;
        if (lane == 0) {
            red[par][0][t >> 5] = s1;
            red[par][1][t >> 5] = s2;
        }
        __syncthreads();
        const float m1 = warp_sum(lane < warps ? red[par][0][lane] : 0.0f) / float(cols);
        const float m2 = warp_sum(lane < warps ? red[par][1][lane] : 0.0f) / float(cols);
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = (t + j * tpr) * E;
            if (c < cols) {
                float o[E];
#pragma unroll
                for (int i = 0; i < E; ++i)
                    o[i] = rs * (g[j * E + i] - m1 - xh[j * E + i] * m2);
                store_floats(dx + row * cols + c, o);
            }
        }
    }
    if (!part) return;
    float* p = part + int64_t(blockIdx.x) * 2 * cols;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = (t + j * tpr) * E;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (c + i < cols) {
                p[c + i] = dw[j * E + i];
                p[cols + c + i] = db[j * E + i];
            }
        }
    }
}

// Column sums of the partial rows [n][2 cols]: a CTA per 32 columns, its 8
// warps take every eighth row, then their sums are added in order.
__global__ void __launch_bounds__(256) layernorm_sum_kernel(const float* __restrict__ part, int n,
                                                            int cols, float* __restrict__ dweight,
                                                            float* __restrict__ dbias) {
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float a = 0.0f;
    if (c < 2 * cols)
#pragma unroll 4
        for (int i = warp; i < n; i += 8) a += part[int64_t(i) * 2 * cols + c];
    s[warp][lane] = a;
    __syncthreads();
    if (warp == 0 && c < 2 * cols) {
#pragma unroll
        for (int i = 1; i < 8; ++i) a += s[i][lane];
        if (c < cols) {
            if (dweight) dweight[c] = a;
        } else if (dbias) {
            dbias[c - cols] = a;
        }
    }
}

int backward_ctas(int64_t rows) { return int(std::min<int64_t>(rows, sm_count())); }

template <class T, int E, int CH>
int forward_launch(bool warp, int threads, const void* x, int64_t rows, int cols,
                   const float* w, const float* b, float eps, void* y, float* mean, float* rstd,
                   cudaStream_t st) {
    const T* xp = static_cast<const T*>(x);
    T* yp = static_cast<T*>(y);
    if (warp)
        layernorm_forward_kernel<T, E, CH, true><<<int((rows + 3) / 4), 128, 0, st>>>(
            xp, rows, cols, w, b, eps, yp, mean, rstd);
    else
        layernorm_forward_kernel<T, E, CH, false><<<int(rows), threads, 0, st>>>(
            xp, rows, cols, w, b, eps, yp, mean, rstd);
    return check_launch();
}

int round_threads(int chunks, int ch) { return ((chunks + ch - 1) / ch + 31) / 32 * 32; }

template <class T>
int forward_any(bool vec, const void* x, int64_t rows, int cols, const float* w, const float* b,
                float eps, void* y, float* mean, float* rstd, cudaStream_t st) {
    if (vec) {
        const int chunks = cols / 8;
        if (chunks <= 64)
            return forward_launch<T, 8, 2>(true, 0, x, rows, cols, w, b, eps, y, mean, rstd, st);
        if (chunks <= 128)
            return forward_launch<T, 8, 4>(true, 0, x, rows, cols, w, b, eps, y, mean, rstd, st);
        return forward_launch<T, 8, 4>(false, round_threads(chunks, 4), x, rows, cols, w, b, eps,
                                       y, mean, rstd, st);
    }
    if (cols <= 256)
        return forward_launch<T, 1, 8>(true, 0, x, rows, cols, w, b, eps, y, mean, rstd, st);
    if (cols <= 8192)
        return forward_launch<T, 1, 8>(false, round_threads(cols, 8), x, rows, cols, w, b, eps, y,
                                       mean, rstd, st);
    return forward_launch<T, 1, 16>(false, round_threads(cols, 16), x, rows, cols, w, b, eps, y,
                                    mean, rstd, st);
}

struct BwdArgs {
    const void* dy;
    const void* x;
    const float* x_scales;
    int64_t rows;
    int cols;
    int64_t x_pitch;
    const float* weight;
    const float* mean;
    const float* rstd;
    void* dx;
    float* part;
};

template <class T, class X, int E, int CH>
int backward_launch(const BwdArgs& a, int threads, cudaStream_t st) {
    layernorm_backward_kernel<T, X, E, CH><<<backward_ctas(a.rows), threads, 0, st>>>(
        static_cast<const T*>(a.dy), static_cast<const X*>(a.x), a.x_scales, a.rows, a.cols,
        a.x_pitch, a.weight, a.mean, a.rstd, static_cast<T*>(a.dx), a.part);
    return check_launch();
}

template <class T, class X>
int backward_any(bool vec, const BwdArgs& a, cudaStream_t st) {
    if (vec) {
        const int chunks = a.cols / 8;
        if (chunks <= 1024) return backward_launch<T, X, 8, 1>(a, round_threads(chunks, 1), st);
        return backward_launch<T, X, 8, 2>(a, round_threads(chunks, 2), st);
    }
    if (a.cols <= 4096) return backward_launch<T, X, 1, 4>(a, round_threads(a.cols, 4), st);
    return backward_launch<T, X, 1, 16>(a, round_threads(a.cols, 16), st);
}

template <class T>
int backward_typed(int x_type, int type, bool vec, const BwdArgs& a, cudaStream_t st) {
    if (x_type == type) return backward_any<T, T>(vec, a, st);
    if (x_type == MOE_T_CKPT) return backward_any<T, e4m3_t>(vec, a, st);
    if constexpr (sizeof(T) == 4) {
        if (x_type == MOE_T_BF16) return backward_any<T, bf16_t>(vec, a, st);
        if (x_type == MOE_T_F16) return backward_any<T, f16_t>(vec, a, st);
    }
    return MOE_ERR_ARG;
}

size_t backward_ws(int64_t rows, int cols) {
    return size_t(std::min<int64_t>(rows, sm_count())) * 2 * size_t(cols) * sizeof(float);
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t type_size(int type) { return type == MOE_T_F32 ? 4 : type == MOE_T_CKPT ? 1 : 2; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" MOE_API int moe_layernorm_forward(const void* x, int type, int64_t rows, int cols,
                                             const float* weight, const float* bias, float eps,
                                             void* y, float* mean, float* rstd, int* dev_status,
                                             void* stream) {
    (void)dev_status;
    if (!plain_type(type)) return MOE_ERR_ARG;
    if (rows < 0 || rows > INT32_MAX || cols < 1 || cols > kMaxCols) return MOE_ERR_SHAPE;
    if (!(eps >= 0.0f)) return MOE_ERR_ARG;
    if (rows == 0) return MOE_OK;
    if (!x || !y) return MOE_ERR_NULL;
    const size_t es = type_size(type);
    if (!aligned(x, es) || !aligned(y, es) || !aligned(weight, 4) || !aligned(bias, 4))
        return MOE_ERR_ALIGN;
    if (!device_is_sm100()) return MOE_ERR_DEVICE;
    const bool vec = cols % 8 == 0 && aligned16(x) && aligned16(y) && aligned16(weight) &&
                     aligned16(bias);
    cudaStream_t st = as_stream(stream);
    if (type == MOE_T_F32)
        return forward_any<float>(vec, x, rows, cols, weight, bias, eps, y, mean, rstd, st);
    if (type == MOE_T_BF16)
        return forward_any<bf16_t>(vec, x, rows, cols, weight, bias, eps, y, mean, rstd, st);
    return forward_any<f16_t>(vec, x, rows, cols, weight, bias, eps, y, mean, rstd, st);
}

extern "C" MOE_API size_t moe_layernorm_backward_workspace_size(int64_t rows, int cols) {
    if (rows < 0 || rows > INT32_MAX || cols < 1 || cols > kMaxCols) return 0;
    return backward_ws(rows, cols);
}

extern "C" MOE_API int moe_layernorm_backward(const void* dy, int type, const void* x, int x_type,
                                              const float* x_scales, int64_t rows, int cols,
                                              const float* weight, const float* mean,
                                              const float* rstd, void* dx, float* dweight,
                                              float* dbias, void* ws, size_t ws_bytes,
                                              int* dev_status, void* stream) {
    (void)dev_status;
    if (!plain_type(type)) return MOE_ERR_ARG;
    if (x_type != type && x_type != MOE_T_CKPT &&
        !(type == MOE_T_F32 && (x_type == MOE_T_BF16 || x_type == MOE_T_F16)))
        return MOE_ERR_ARG;
    if (rows < 0 || rows > INT32_MAX || cols < 1 || cols > kMaxCols) return MOE_ERR_SHAPE;
    cudaStream_t st = as_stream(stream);
    if (rows == 0) {
        // no rows: the parameters' gradients are empty sums
        for (float* g : {dweight, dbias})
            if (g && cudaMemsetAsync(g, 0, sizeof(float) * size_t(cols), st) != cudaSuccess)
                return MOE_ERR_CUDA;
        return MOE_OK;
    }
    if (!dy || !x || !mean || !rstd || !dx) return MOE_ERR_NULL;
    if (x_type == MOE_T_CKPT && !x_scales) return MOE_ERR_NULL;
    const size_t es = type_size(type);
    if (!aligned(dy, es) || !aligned(dx, es) || !aligned(weight, 4) || !aligned(x, type_size(x_type)))
        return MOE_ERR_ALIGN;
    if (x_type == MOE_T_CKPT && !aligned16(x)) return MOE_ERR_ALIGN;
    const bool sums = dweight || dbias;
    if (sums && (!ws || ws_bytes < backward_ws(rows, cols))) return MOE_ERR_WORKSPACE;
    if (sums && !aligned16(ws)) return MOE_ERR_ALIGN;
    if (!device_is_sm100()) return MOE_ERR_DEVICE;
    const bool vec = cols % 8 == 0 && aligned16(dy) && aligned16(x) && aligned16(dx) &&
                     aligned16(weight);
    BwdArgs a{dy, x, x_scales, rows, cols, x_type == MOE_T_CKPT ? ckpt_row_bytes(cols) : cols,
              weight, mean, rstd, dx, sums ? static_cast<float*>(ws) : nullptr};
    int rc = type == MOE_T_F32    ? backward_typed<float>(x_type, type, vec, a, st)
             : type == MOE_T_BF16 ? backward_typed<bf16_t>(x_type, type, vec, a, st)
                                  : backward_typed<f16_t>(x_type, type, vec, a, st);
    if (rc != MOE_OK || !sums) return rc;
    layernorm_sum_kernel<<<(2 * cols + 31) / 32, 256, 0, st>>>(a.part, backward_ctas(rows), cols,
                                                               dweight, dbias);
    return check_launch();
}
