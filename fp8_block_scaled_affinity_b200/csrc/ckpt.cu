// Activation checkpoints in 8 bits: a matrix kept between the forward and
// the backward pass as E4M3 codes with one fp32 scale per 1x128 tile of a
// row: scale = amax / 448, code = E4M3(v (448 / amax)), kept_scale's rule.
// Codes lie in [rows, cols rounded up to 128] bytes, so a tile is one 128-byte
// line; scales in [tiles, rows], the layout the grouped GEMM reads.
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
// A thread takes 4 columns of UR rows: 4 codes in, 4 values out, so that a
// warp's stores are whole lines in every type (with 8 columns its fp32 stores
// are halves of twice as many: 261 us for 36864 rows of 7168).
constexpr int UR = 4;

template <class T, bool VEC>
__global__ void __launch_bounds__(kThreads) ckpt_unpack_kernel(const uint8_t* __restrict__ q,
                                                               const float* __restrict__ scales,
                                                               int64_t rows, int64_t cols,
                                                               int64_t pitch, T* __restrict__ y) {
    const int64_t c = (int64_t(blockIdx.y) * kThreads + threadIdx.x) * 4;
    if (c >= cols) return;
    const int64_t row0 = int64_t(blockIdx.x) * UR;
    const int n = int(min(int64_t(UR), rows - row0));
    uint32_t v[UR];
    float s[UR];
#pragma unroll
    for (int r = 0; r < UR; ++r) {
        v[r] = 0u;
        s[r] = 0.0f;
        if (r < n) {
            v[r] = __ldcs(reinterpret_cast<const uint32_t*>(q + (row0 + r) * pitch + c));
            s[r] = __ldg(scales + c / kTile * rows + row0 + r);
        }
    }
#pragma unroll
    for (int r = 0; r < UR; ++r) {
        if (r >= n) break;
        float2 f[2] = {e4m3x2_to_float2(uint16_t(v[r] & 0xFFFFu)),
                       e4m3x2_to_float2(uint16_t(v[r] >> 16))};
        f[0] = mul2(f[0], both(s[r]));
        f[1] = mul2(f[1], both(s[r]));
        T* o = y + (row0 + r) * cols + c;
        if (VEC) {
            store_pairs(o, f);
        } else {
            const float g[4] = {f[0].x, f[0].y, f[1].x, f[1].y};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c + i < cols) elem_store(o + i, g[i]);
        }
    }
}

// 1 / e of two numbers from 1 to infinity: the hardware's approximation (one
// step of fp32) and one of Newton's steps, r + r (1 - e r), on both at once:
// __frcp_rn's result for each of the 2^23 mantissas up to 2^126, and 0 where
// that is subnormal.  (36864 rows of I = 2048: 118.6 us; with __frcp_rn 130.9,
// with __fdividef, two steps off at most, 116.8.)  e = inf: r = 0, and the NaN
// of inf * 0 becomes a finite number.
__device__ __forceinline__ float2 reciprocal2(float2 e) {
    float2 r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
    float2 t = fma2(mul2(e, both(-1.0f)), r, both(1.0f));
    t = make_float2(fmaxf(t.x, -1.0f), fmaxf(t.y, -1.0f));
    return fma2(r, t, r);
}

// ------------------------------------- SwiGLU backward from a checkpoint
// da = dh c s (1 + a (1 - s)), dc = dh a s with s = sigmoid(a), from dh
// (fp32) and the kept [a | c]; the row [da | dc] quantised in 1x128 tiles.  The
// products are taken in the order of the same step from fp32 a and c, so that
// both give the same bits from the same values.
// A CTA takes 32 rows of one 128-feature tile of a and of c, a warp a row at
// a time, 4 features a lane (whole lines of dh), four rows' loads in flight.
// Scales of the strip, read and written, go through shared memory as lines.
// Close to both limits: per 8 bytes a feature about 25 instructions.
__global__ void __launch_bounds__(kThreads) swiglu_backward_ckpt_kernel(
    const float* __restrict__ dh, const uint8_t* __restrict__ ac,
    const float* __restrict__ ac_scales, int64_t rows, int I, int64_t rows_total,
    uint8_t* __restrict__ q, float* __restrict__ qs) {
    __shared__ float sin[2][kStripRows], sout[2][kStripRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nt = I / kTile;
    const int tile = blockIdx.x % nt;
    const int64_t row0 = int64_t(blockIdx.x / nt) * kStripRows;
    const int n = int(min(int64_t(kStripRows), rows - row0));
    constexpr int RW = kStripRows / (kThreads / 32);  // rows of a warp
    float4 hv[RW];
    uint32_t av[RW], cv[RW];
    const int f0 = tile * kTile + 4 * lane;
#pragma unroll
    for (int r = 0; r < RW; ++r) {
        const int lr = warp * RW + r;
        hv[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        av[r] = cv[r] = 0u;
        if (lr < n) {
            const uint8_t* acr = ac + (row0 + lr) * 2 * I + f0;
            hv[r] = __ldcs(reinterpret_cast<const float4*>(dh + (row0 + lr) * I + f0));
            av[r] = __ldcs(reinterpret_cast<const uint32_t*>(acr));
            cv[r] = __ldcs(reinterpret_cast<const uint32_t*>(acr + I));
        }
    }
    if (warp < 2)
        sin[warp][lane] =
            lane < n ? ac_scales[int64_t(warp * nt + tile) * rows_total + row0 + lane] : 0.0f;
    __syncthreads();
    float2 da[RW][2], dc[RW][2];
    float amax = 0.0f;  // lane 2 r: da's of row r, lane 2 r + 1: dc's
#pragma unroll
    for (int r = 0; r < RW; ++r) {
        const int lr = warp * RW + r;
        const float2 sa = both(sin[0][lr]), sc = both(sin[1][lr]);
        const float2 h[2] = {make_float2(hv[r].x, hv[r].y), make_float2(hv[r].z, hv[r].w)};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 a = mul2(e4m3x2_to_float2(uint16_t(av[r] >> (16 * i))), sa);
            const float2 c = mul2(e4m3x2_to_float2(uint16_t(cv[r] >> (16 * i))), sc);
            const float2 e = add2(make_float2(__expf(-a.x), __expf(-a.y)), both(1.0f));
            const float2 s = reciprocal2(e);
            const float2 t = fma2(a, fma2(s, both(-1.0f), both(1.0f)), both(1.0f));
            da[r][i] = mul2(mul2(mul2(h[i], c), s), t);
            dc[r][i] = mul2(mul2(h[i], a), s);
        }
        float ma = 0.0f, mc = 0.0f;  // (a NaN is no maximum)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            ma = fmaxf(fmaxf(ma, fabsf(da[r][i].x)), fabsf(da[r][i].y));
            mc = fmaxf(fmaxf(mc, fabsf(dc[r][i].x)), fabsf(dc[r][i].y));
        }
        // the warp's maxima: as integers, whose order is that of |v|
        const uint32_t wa = __reduce_max_sync(0xffffffffu, __float_as_uint(ma));
        const uint32_t wc = __reduce_max_sync(0xffffffffu, __float_as_uint(mc));
        if (lane == 2 * r) amax = __uint_as_float(wa);
        if (lane == 2 * r + 1) amax = __uint_as_float(wc);
    }
    // the divisions of all the warp's tiles at once, a tile a lane
    float scale, inv;
    scale_from_amax(kept_amax(amax), scale, inv);
    if (lane < 2 * RW) sout[lane & 1][warp * RW + (lane >> 1)] = scale;
#pragma unroll
    for (int r = 0; r < RW; ++r) {
        const int lr = warp * RW + r;
        const float2 i0 = both(__shfl_sync(0xffffffffu, inv, 2 * r));
        const float2 i1 = both(__shfl_sync(0xffffffffu, inv, 2 * r + 1));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            da[r][i] = mul2(da[r][i], i0);
            dc[r][i] = mul2(dc[r][i], i1);
        }
        if (lr < n) {
            uint8_t* o = q + (row0 + lr) * 2 * I + f0;
            __stcs(reinterpret_cast<uint32_t*>(o),
                   e4m3x2(da[r][0].x, da[r][0].y) |
                       (uint32_t(e4m3x2(da[r][1].x, da[r][1].y)) << 16));
            __stcs(reinterpret_cast<uint32_t*>(o + I),
                   e4m3x2(dc[r][0].x, dc[r][0].y) |
                       (uint32_t(e4m3x2(dc[r][1].x, dc[r][1].y)) << 16));
        }
    }
    __syncthreads();
    if (warp < 2 && lane < n)
        qs[int64_t(warp * nt + tile) * rows_total + row0 + lane] = sout[warp][lane];
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
    const int64_t gx = (rows + UR - 1) / UR;
    const int64_t gy = (cols + 4 * kThreads - 1) / (4 * kThreads);
    if (gy > 65535) return MOE_ERR_SHAPE;
    const dim3 grid{unsigned(gx), unsigned(gy)};
    // a CTA no wider than the row
    const int threads = int(std::min<int64_t>(kThreads, ((cols + 3) / 4 + 31) / 32 * 32));
    T* yp = static_cast<T*>(y);
    if (cols % 4 == 0 && aligned16(y))
        ckpt_unpack_kernel<T, true><<<grid, threads, 0, st>>>(q, scales, rows, cols,
                                                              ckpt_row_bytes(cols), yp);
    else
        ckpt_unpack_kernel<T, false><<<grid, threads, 0, st>>>(q, scales, rows, cols,
                                                               ckpt_row_bytes(cols), yp);
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
