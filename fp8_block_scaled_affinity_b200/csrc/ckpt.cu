// Activation checkpoints in 8 bits: a matrix kept between the forward and
// the backward pass as E4M3 codes with one fp32 scale per 1x128 tile of a
// row: scale = amax / 448, code = E4M3(v (448 / amax)), kept_scale's rule.  Codes lie in [rows, cols rounded up to 128] bytes, so a
// tile is one 128-byte line; scales in [tiles, rows], the layout the grouped
// GEMM reads.
//
// All passes here are bound by memory: each value is read once, each code
// written once.
#include <algorithm>

#include "elem.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kStripRows = 32;  // rows of a CTA: one 128-byte line of scales per tile

// ----------------------------------------------------------------- pack
// A CTA takes 32 rows x ST tiles; a warp 4 rows.  16 lanes hold a tile, 8
// columns each, so an amax is four shuffles.  The scales of the strip go
// through shared memory: 32 rows of a tile are one line in [tiles, rows].
constexpr int kPackTiles = 4;

template <class T, bool VEC>
__global__ void __launch_bounds__(kThreads) ckpt_pack_kernel(const T* __restrict__ x, int64_t rows,
                                                             int64_t cols, int64_t pitch,
                                                             uint8_t* __restrict__ q,
                                                             float* __restrict__ scales) {
    __shared__ float sc[kPackTiles][kStripRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane & 15, half = lane >> 4;
    const int64_t tiles = pitch / kTile;
    const int64_t row0 = int64_t(blockIdx.x) * kStripRows;
    const int64_t tile0 = int64_t(blockIdx.y) * kPackTiles;
    constexpr int RW = kStripRows / (kThreads / 32);  // rows of a warp
    Raw<T, 8> v[RW][kPackTiles / 2];
#pragma unroll
    for (int r = 0; r < RW; ++r) {
        const int64_t row = row0 + warp * RW + r;
#pragma unroll
        for (int j = 0; j < kPackTiles / 2; ++j) {
            const int64_t c = (tile0 + 2 * j + half) * kTile + 8 * sub;
            if (VEC) {
                v[r][j] = row < rows && c < cols ? raw_load<T, 8>(x + row * cols + c)
                                                 : raw_zero<T, 8>();
            } else {
                T e[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    e[i] = row < rows && c + i < cols ? x[row * cols + c + i] : T(0.0f);
                memcpy(&v[r][j], e, sizeof(e));
            }
        }
    }
#pragma unroll
    for (int r = 0; r < RW; ++r) {
        const int64_t row = row0 + warp * RW + r;
#pragma unroll
        for (int j = 0; j < kPackTiles / 2; ++j) {
            const int64_t tile = tile0 + 2 * j + half;
            float f[8];
            raw_floats(v[r][j], f);
            float amax = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1)
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            float scale, inv;
            kept_scale(amax, scale, inv);
            uint32_t w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t lo = e4m3x2(__fmul_rn(f[4 * i], inv), __fmul_rn(f[4 * i + 1], inv));
                const uint32_t hi =
                    e4m3x2(__fmul_rn(f[4 * i + 2], inv), __fmul_rn(f[4 * i + 3], inv));
                w[i] = lo | (hi << 16);
            }
            if (row < rows && tile < tiles)
                *reinterpret_cast<uint2*>(q + row * pitch + tile * kTile + 8 * sub) =
                    make_uint2(w[0], w[1]);
            if (sub == 0) sc[2 * j + half][warp * RW + r] = scale;
        }
    }
    __syncthreads();
    if (warp < kPackTiles) {
        const int64_t tile = tile0 + warp, row = row0 + lane;
        if (tile < tiles && row < rows) scales[tile * rows + row] = sc[warp][lane];
    }
}

// --------------------------------------------------------------- unpack
// A thread takes 8 columns of UR rows: 8 codes in, 8 values out.
constexpr int UR = 4;

template <class T, bool VEC>
__global__ void __launch_bounds__(kThreads) ckpt_unpack_kernel(const uint8_t* __restrict__ q,
                                                               const float* __restrict__ scales,
                                                               int64_t rows, int64_t cols,
                                                               int64_t pitch, T* __restrict__ y) {
    const int64_t chunks = (cols + 7) / 8;
    const int64_t strips = (rows + UR - 1) / UR;
    const int64_t u = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (u >= strips * chunks) return;
    const int64_t strip = u / chunks;
    const int64_t c = (u - strip * chunks) * 8;
    Raw<e4m3_t, 8> v[UR];
    float s[UR];
#pragma unroll
    for (int r = 0; r < UR; ++r) {
        const int64_t row = strip * UR + r;
        v[r] = raw_zero<e4m3_t, 8>();
        s[r] = 0.0f;
        if (row < rows) {
            v[r] = raw_load<e4m3_t, 8>(reinterpret_cast<const e4m3_t*>(q) + row * pitch + c);
            s[r] = __ldg(scales + c / kTile * rows + row);
        }
    }
#pragma unroll
    for (int r = 0; r < UR; ++r) {
        const int64_t row = strip * UR + r;
        if (row >= rows) break;
        float f[8];
        raw_floats(v[r], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= s[r];
        if (VEC) {
            store_floats(y + row * cols + c, f);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < cols) elem_store(y + row * cols + c + i, f[i]);
        }
    }
}

// ------------------------------------- SwiGLU backward from a checkpoint
// da = dh c s (1 + a (1 - s)), dc = dh a s with s = sigmoid(a), from dh
// (fp32) and the kept [a | c]; the row [da | dc] quantised in 1x128 tiles.
// A CTA takes 32 rows of one 128-feature tile of a and of c: 16 lanes hold a
// row's tile, 8 features each, so da's and dc's amax are four shuffles.
// Scales of the strip, read and written, go through shared memory as lines.
__global__ void __launch_bounds__(kThreads) swiglu_backward_ckpt_kernel(
    const float* __restrict__ dh, const uint8_t* __restrict__ ac,
    const float* __restrict__ ac_scales, int64_t rows, int I, int64_t rows_total,
    uint8_t* __restrict__ q, float* __restrict__ qs) {
    __shared__ float sin[2][kStripRows], sout[2][kStripRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane & 15, half = lane >> 4;
    const int nt = I / kTile;
    const int tile = blockIdx.x % nt;
    const int64_t row0 = int64_t(blockIdx.x / nt) * kStripRows;
    if (warp < 2) {
        const int64_t row = row0 + lane;
        sin[warp][lane] =
            row < rows ? ac_scales[int64_t(warp * nt + tile) * rows_total + row] : 0.0f;
    }
    constexpr int RW = kStripRows / (kThreads / 32) / 2;  // row pairs of a warp
    Raw<float, 8> hv[RW];
    Raw<e4m3_t, 8> av[RW], cv[RW];
    const int f0 = tile * kTile + 8 * sub;
#pragma unroll
    for (int r = 0; r < RW; ++r) {
        const int64_t row = row0 + (warp * RW + r) * 2 + half;
        hv[r] = raw_zero<float, 8>();
        av[r] = cv[r] = raw_zero<e4m3_t, 8>();
        if (row < rows) {
            const e4m3_t* acr = reinterpret_cast<const e4m3_t*>(ac) + row * 2 * I + f0;
            hv[r] = raw_load<float, 8>(dh + row * I + f0);
            av[r] = raw_load<e4m3_t, 8>(acr);
            cv[r] = raw_load<e4m3_t, 8>(acr + I);
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RW; ++r) {
        const int lr = (warp * RW + r) * 2 + half;
        const int64_t row = row0 + lr;
        const float sa = sin[0][lr], sc = sin[1][lr];
        float h[8], a[8], c[8];
        raw_floats(hv[r], h);
        raw_floats(av[r], a);
        raw_floats(cv[r], c);
        float ma = 0.0f, mc = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = a[i] * sa;
            const float sg = __fdividef(1.0f, 1.0f + __expf(-x));
            const float hs = h[i] * sg;
            a[i] = hs * (c[i] * sc) * fmaf(x, 1.0f - sg, 1.0f);
            c[i] = hs * x;
            ma = fmaxf(ma, fabsf(a[i]));
            mc = fmaxf(mc, fabsf(c[i]));
        }
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) {
            ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, o));
            mc = fmaxf(mc, __shfl_xor_sync(0xffffffffu, mc, o));
        }
        float s0, i0, s1, i1;
        scale_from_amax(ma, s0, i0);
        scale_from_amax(mc, s1, i1);
        uint32_t wa[2], wc[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            wa[i] = e4m3x2(__fmul_rn(a[4 * i], i0), __fmul_rn(a[4 * i + 1], i0)) |
                    (uint32_t(e4m3x2(__fmul_rn(a[4 * i + 2], i0), __fmul_rn(a[4 * i + 3], i0)))
                     << 16);
            wc[i] = e4m3x2(__fmul_rn(c[4 * i], i1), __fmul_rn(c[4 * i + 1], i1)) |
                    (uint32_t(e4m3x2(__fmul_rn(c[4 * i + 2], i1), __fmul_rn(c[4 * i + 3], i1)))
                     << 16);
        }
        if (row < rows) {
            uint8_t* o = q + row * 2 * I + f0;
            *reinterpret_cast<uint2*>(o) = make_uint2(wa[0], wa[1]);
            *reinterpret_cast<uint2*>(o + I) = make_uint2(wc[0], wc[1]);
        }
        if (sub == 0) {
            sout[0][lr] = s0;
            sout[1][lr] = s1;
        }
    }
    __syncthreads();
    if (warp < 2) {
        const int64_t row = row0 + lane;
        if (row < rows) qs[int64_t(warp * nt + tile) * rows_total + row] = sout[warp][lane];
    }
}

template <class T>
int pack_any(const void* x, int64_t rows, int64_t cols, uint8_t* q, float* scales,
             cudaStream_t st) {
    const int64_t pitch = ckpt_row_bytes(cols);
    const int64_t gx = (rows + kStripRows - 1) / kStripRows;
    const int64_t gy = (pitch / kTile + kPackTiles - 1) / kPackTiles;
    if (gx > INT32_MAX || gy > 65535) return MOE_ERR_SHAPE;
    const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
    const T* xp = static_cast<const T*>(x);
    if (cols % 8 == 0 && aligned16(x))
        ckpt_pack_kernel<T, true><<<grid, kThreads, 0, st>>>(xp, rows, cols, pitch, q, scales);
    else
        ckpt_pack_kernel<T, false><<<grid, kThreads, 0, st>>>(xp, rows, cols, pitch, q, scales);
    return check_launch();
}

template <class T>
int unpack_any(const uint8_t* q, const float* scales, int64_t rows, int64_t cols, void* y,
               cudaStream_t st) {
    const int64_t units = (rows + UR - 1) / UR * ((cols + 7) / 8);
    const int64_t grid = (units + kThreads - 1) / kThreads;
    if (grid > INT32_MAX) return MOE_ERR_SHAPE;
    T* yp = static_cast<T*>(y);
    if (cols % 8 == 0 && aligned16(y))
        ckpt_unpack_kernel<T, true><<<unsigned(grid), kThreads, 0, st>>>(
            q, scales, rows, cols, ckpt_row_bytes(cols), yp);
    else
        ckpt_unpack_kernel<T, false><<<unsigned(grid), kThreads, 0, st>>>(
            q, scales, rows, cols, ckpt_row_bytes(cols), yp);
    return check_launch();
}

bool elem_aligned(const void* p, int type) {
    return (reinterpret_cast<uintptr_t>(p) & (type == MOE_T_F32 ? 3 : 1)) == 0;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" MOE_API int64_t moe_ckpt_row_bytes(int64_t cols) {
    return cols < 0 || cols > INT32_MAX ? -1 : ckpt_row_bytes(cols);
}

extern "C" MOE_API int moe_ckpt_pack(const void* x, int type, int64_t rows, int64_t cols,
                                     uint8_t* q, float* scales, int* dev_status, void* stream) {
    (void)dev_status;
    if (!plain_type(type)) return MOE_ERR_ARG;
    if (rows < 0 || rows > INT32_MAX || cols < 0 || cols > INT32_MAX) return MOE_ERR_SHAPE;
    if (rows == 0 || cols == 0) return MOE_OK;
    if (!x || !q || !scales) return MOE_ERR_NULL;
    if (!aligned16(q) || !elem_aligned(x, type)) return MOE_ERR_ALIGN;
    if (!device_is_sm100()) return MOE_ERR_DEVICE;
    cudaStream_t st = as_stream(stream);
    if (type == MOE_T_F32) return pack_any<float>(x, rows, cols, q, scales, st);
    if (type == MOE_T_BF16) return pack_any<bf16_t>(x, rows, cols, q, scales, st);
    return pack_any<f16_t>(x, rows, cols, q, scales, st);
}

extern "C" MOE_API int moe_ckpt_unpack(const uint8_t* q, const float* scales, int64_t rows,
                                       int64_t cols, void* y, int type, int* dev_status,
                                       void* stream) {
    (void)dev_status;
    if (!plain_type(type)) return MOE_ERR_ARG;
    if (rows < 0 || rows > INT32_MAX || cols < 0 || cols > INT32_MAX) return MOE_ERR_SHAPE;
    if (rows == 0 || cols == 0) return MOE_OK;
    if (!q || !scales || !y) return MOE_ERR_NULL;
    if (!aligned16(q) || !elem_aligned(y, type)) return MOE_ERR_ALIGN;
    if (!device_is_sm100()) return MOE_ERR_DEVICE;
    cudaStream_t st = as_stream(stream);
    if (type == MOE_T_F32) return unpack_any<float>(q, scales, rows, cols, y, st);
    if (type == MOE_T_BF16) return unpack_any<bf16_t>(q, scales, rows, cols, y, st);
    return unpack_any<f16_t>(q, scales, rows, cols, y, st);
}

extern "C" MOE_API int moe_swiglu_backward_quant_ckpt(const float* dh, const uint8_t* ac_q,
                                                      const float* ac_scales, int64_t rows,
                                                      int inter, int64_t rows_total, uint8_t* q,
                                                      float* q_scales, int* dev_status,
                                                      void* stream) {
    (void)dev_status;
    if (rows < 0 || inter <= 0 || inter % 128 || rows_total < rows) return MOE_ERR_SHAPE;
    if (rows == 0) return MOE_OK;
    if (!dh || !ac_q || !ac_scales || !q || !q_scales) return MOE_ERR_NULL;
    if (!aligned16(dh) || !aligned16(ac_q) || !aligned16(q)) return MOE_ERR_ALIGN;
    const int64_t grid = (rows + kStripRows - 1) / kStripRows * (inter / kTile);
    if (grid > INT32_MAX) return MOE_ERR_SHAPE;
    if (!device_is_sm100()) return MOE_ERR_DEVICE;
    swiglu_backward_ckpt_kernel<<<unsigned(grid), kThreads, 0, as_stream(stream)>>>(
        dh, ac_q, ac_scales, rows, inter, rows_total, q, q_scales);
    return check_launch();
}
