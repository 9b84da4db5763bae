// Element types of the layer norm, the 8-bit checkpoints and the dense gated
// feed-forward block: 8 consecutive elements as fp32 values, from and to
// memory.  Every conversion down rounds once, to nearest even.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {

using bf16_t = __nv_bfloat16;
using f16_t = __half;
struct e4m3_t {  // code of a checkpoint (its tile's scale is kept apart)
    uint8_t code;
};

constexpr int kTile = 128;  // columns of a checkpoint tile
inline int64_t ckpt_row_bytes(int64_t cols) { return (cols + kTile - 1) / kTile * kTile; }
inline int64_t ckpt_tiles(int64_t cols) { return (cols + kTile - 1) / kTile; }

// true for the type codes of plain elements
inline bool plain_type(int type) {
    return type == MOE_T_F32 || type == MOE_T_BF16 || type == MOE_T_F16;
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t codes) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(codes));
    return __half22float2(*reinterpret_cast<__half2*>(&h2));
}
__device__ __forceinline__ float e4m3_to_float(uint8_t code) {
    return e4m3x2_to_float2(uint16_t(code)).x;
}

// Two fp32 values in one instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(r))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(r))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(r))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
          "l"(reinterpret_cast<uint64_t&>(c)));
    return r;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Scale rule of the checkpoints: scale = fp32(amax / 448), inverse =
// fp32(448 fp32(1 / amax)), both 1 for a tile of zeros.  (The online
// quantisers round 448 / amax once; here one reciprocal and one product are
// enough, and a code differs only where its value lies within an fp32
// rounding of the border between two codes.)  448 / amax passes the fp32 range
// below 1.32e-36, where zeros would become 0 * inf: such an amax counts as
// 2^-119 (1.5e-36), whose inverse is exact and whose scale is subnormal with 22
// bits, and the tile's values keep what E4M3 has down to 2^-10 of that scale.
constexpr float kLeastAmax = 0x1p-119f;
__device__ __forceinline__ float kept_amax(float amax) {
    return amax == 0.0f ? 0.0f : fmaxf(amax, kLeastAmax);
}
__device__ __forceinline__ void kept_scale(float amax, float& scale, float& inv) {
    if (amax == 0.0f) {
        scale = 1.0f;
        inv = 1.0f;
    } else {
        amax = fmaxf(amax, kLeastAmax);
        scale = __fdiv_rn(amax, 448.0f);
        inv = __fmul_rn(__frcp_rn(amax), 448.0f);
    }
}

// Raw storage of 8 or 4 elements (or of one, for rows that are not aligned),
// kept packed until it is used.
template <class T, int E> struct Raw;
template <> struct Raw<float, 8> { float4 a, b; };
template <> struct Raw<bf16_t, 8> { uint4 a; };
template <> struct Raw<f16_t, 8> { uint4 a; };
template <> struct Raw<e4m3_t, 8> { uint2 a; };
template <> struct Raw<float, 4> { float4 a; };
template <> struct Raw<bf16_t, 4> { uint2 a; };
template <> struct Raw<f16_t, 4> { uint2 a; };
template <class T> struct Raw<T, 1> { T a; };

template <class T, int E>
__device__ __forceinline__ Raw<T, E> raw_load(const T* p) {
    Raw<T, E> r;
    if constexpr (E == 1) {
        r.a = *p;
    } else if constexpr (E == 4) {
        if constexpr (sizeof(T) == 4) r.a = __ldg(reinterpret_cast<const float4*>(p));
        else r.a = __ldg(reinterpret_cast<const uint2*>(p));
    } else if constexpr (sizeof(T) == 4) {
        r.a = __ldg(reinterpret_cast<const float4*>(p));
        r.b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    } else if constexpr (sizeof(T) == 2) {
        r.a = __ldg(reinterpret_cast<const uint4*>(p));
    } else {
        r.a = __ldg(reinterpret_cast<const uint2*>(p));
    }
    return r;
}

// The same of data read once, which is not kept in L1 before what is read
// again; and stores of data that this kernel does not read.
template <class T, int E>
__device__ __forceinline__ Raw<T, E> raw_load_once(const T* p) {
    Raw<T, E> r;
    if constexpr (E == 4) {
        if constexpr (sizeof(T) == 4) r.a = __ldcs(reinterpret_cast<const float4*>(p));
        else r.a = __ldcs(reinterpret_cast<const uint2*>(p));
    } else {
        r = raw_load<T, E>(p);
    }
    return r;
}

template <class T, int E>
__device__ __forceinline__ Raw<T, E> raw_zero() {
    Raw<T, E> r;
    memset(&r, 0, sizeof(r));
    return r;
}

__device__ __forceinline__ void unpack2f(bf16_t, uint32_t w, float& a, float& b) {
    a = bf16_lo(w);
    b = bf16_hi(w);
}
__device__ __forceinline__ void unpack2f(f16_t, uint32_t w, float& a, float& b) {
    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&w));
    a = f.x;
    b = f.y;
}
__device__ __forceinline__ uint32_t pack2t(bf16_t, float a, float b) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2t(f16_t, float a, float b) {
    __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ void raw_floats(const Raw<float, 8>& r, float (&f)[8]) {
    f[0] = r.a.x; f[1] = r.a.y; f[2] = r.a.z; f[3] = r.a.w;
    f[4] = r.b.x; f[5] = r.b.y; f[6] = r.b.z; f[7] = r.b.w;
}
template <class T>
__device__ __forceinline__ void raw_floats(const Raw<T, 8>& r, float (&f)[8]) {
    if constexpr (sizeof(T) == 1) {
        const uint32_t w[2] = {r.a.x, r.a.y};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 lo = e4m3x2_to_float2(uint16_t(w[i] & 0xFFFFu));
            const float2 hi = e4m3x2_to_float2(uint16_t(w[i] >> 16));
            f[4 * i] = lo.x; f[4 * i + 1] = lo.y; f[4 * i + 2] = hi.x; f[4 * i + 3] = hi.y;
        }
    } else {
        unpack2f(T(), r.a.x, f[0], f[1]);
        unpack2f(T(), r.a.y, f[2], f[3]);
        unpack2f(T(), r.a.z, f[4], f[5]);
        unpack2f(T(), r.a.w, f[6], f[7]);
    }
}
__device__ __forceinline__ float elem_float(float v) { return v; }
__device__ __forceinline__ float elem_float(bf16_t v) { return __bfloat162float(v); }
__device__ __forceinline__ float elem_float(f16_t v) { return __half2float(v); }
__device__ __forceinline__ float elem_float(e4m3_t v) { return e4m3_to_float(v.code); }
template <class T>
__device__ __forceinline__ void raw_floats(const Raw<T, 1>& r, float (&f)[1]) {
    f[0] = elem_float(r.a);
}

__device__ __forceinline__ void elem_store(float* p, float v) { *p = v; }
__device__ __forceinline__ void elem_store(bf16_t* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void elem_store(f16_t* p, float v) { *p = __float2half_rn(v); }

template <class T>
__device__ __forceinline__ void store_floats(T* p, const float (&f)[1]) {
    elem_store(p, f[0]);
}
template <class T>
__device__ __forceinline__ void store_floats(T* p, const float (&f)[8]) {
    if constexpr (sizeof(T) == 4) {
        float4* o = reinterpret_cast<float4*>(p);
        o[0] = make_float4(f[0], f[1], f[2], f[3]);
        o[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        *reinterpret_cast<uint4*>(p) =
            make_uint4(pack2t(T(), f[0], f[1]), pack2t(T(), f[2], f[3]), pack2t(T(), f[4], f[5]),
                       pack2t(T(), f[6], f[7]));
    }
}

// Pairs of 4 elements, or one element and a zero.
__device__ __forceinline__ void raw_pairs(const Raw<float, 4>& r, float2 (&f)[2]) {
    f[0] = make_float2(r.a.x, r.a.y);
    f[1] = make_float2(r.a.z, r.a.w);
}
template <class T>
__device__ __forceinline__ void raw_pairs(const Raw<T, 4>& r, float2 (&f)[2]) {
    unpack2f(T(), r.a.x, f[0].x, f[0].y);
    unpack2f(T(), r.a.y, f[1].x, f[1].y);
}
template <class T>
__device__ __forceinline__ void raw_pairs(const Raw<T, 1>& r, float2 (&f)[1]) {
    f[0] = make_float2(elem_float(r.a), 0.0f);
}
template <class T>
__device__ __forceinline__ void store_pairs(T* p, const float2 (&f)[2]) {
    if constexpr (sizeof(T) == 4)
        __stcs(reinterpret_cast<float4*>(p), make_float4(f[0].x, f[0].y, f[1].x, f[1].y));
    else
        __stcs(reinterpret_cast<uint2*>(p),
               make_uint2(pack2t(T(), f[0].x, f[0].y), pack2t(T(), f[1].x, f[1].y)));
}
template <class T>
__device__ __forceinline__ void store_pairs(T* p, const float2 (&f)[1]) {
    elem_store(p, f[0].x);
}

}  // namespace moe
