// Layer norm, forward and backward.
//
//   mu = mean(x), var = mean((x - mu)^2), rstd = 1 / sqrt(var + eps)
//   xh = (x - mu) rstd,  y = xh w + b
//   g = dy w,  dx = rstd (g - mean(g) - xh mean(g xh))
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Both passes are bound by memory: x is read once and y written once, x and
// dy read once and dx written once.  A row stays in registers between the
// statistics and their use.  Statistics and sums are fp32; the variance is
// that of the centred values (no difference of squares), and the only
// roundings to fewer bits are those of y and dx.
//
// In the forward pass a CTA or a warp takes one row, and many rows share an
// SM.  The backward pass keeps the sums of dw and db in registers, so a CTA
// walks rows, its threads on the same columns through all of them; those
// registers leave room for one wide row at a time on an SM, whose loads and
// barrier nothing else hides.  So rows are streamed: several ahead are copied
// into shared memory in bulk, which goes on whatever the threads wait for
// (4096 rows of 7168 kept in 8 bits: 53 us, against 73 us with each row loaded
// when its turn comes; 47 us since the partial sums leave 16 bytes a lane, 48
// since xh is a difference first).
// Rows that are no multiple of 16 bytes are copied from the 16-byte boundary
// before them, and read an element at a time.
#include <algorithm>

#include "elem.cuh"
#include "tc.cuh"

namespace moe {
namespace {

constexpr int kMaxCols = 16384;
// CTAs of the forward pass on an SM, and their threads
template <int CTAS> constexpr int kForwardThreads = CTAS == 2 ? 512 : 256;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the row's threads: a warp, or the whole CTA (every thread gets
// it; `red` is not used again before the next barrier).
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* red) {
    v = warp_sum(v);
    if (WARP) return v;
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < warps ? red[lane] : 0.0f);
}

// E values of w from column c, or `none` without w.
template <int E>
__device__ __forceinline__ void load_pairs(float2 (&f)[E == 4 ? 2 : 1], const float* w, int c,
                                           float none) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < (E == 4 ? 2 : 1); ++i) f[i] = both(none);
    } else if constexpr (E == 4) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(w + c));
        f[0] = make_float2(q.x, q.y);
        f[1] = make_float2(q.z, q.w);
    } else {
        f[0] = both(__ldg(w + c));
    }
}

// A row per warp (WARP) or per CTA; a thread holds CH chunks of E columns,
// packed as they came.  What hides the time of a row's loads and barriers is
// other rows: CTAS of them on an SM.  Chunks are 4 elements, so that a warp's
// loads of the fp32 weights are whole lines: with 8 they are halves of twice as
// many, and 57 KB of weights a row of 7168 through L1 take longer than the row
// (16384 rows of bf16: 114 us, with chunks of 4 93 us).  Rows pass L1 by, where
// the weights stay (90 us: 5.2 TB/s).
template <class T, int E, int CH, bool WARP, int CTAS>
__global__ void __launch_bounds__(WARP ? 128 : CTAS > 1 ? kForwardThreads<CTAS> : 1024, CTAS)
    layernorm_forward_kernel(const T* __restrict__ x, int64_t rows, int cols,
                             const float* __restrict__ weight, const float* __restrict__ bias,
                             float eps, T* __restrict__ y, float* __restrict__ mean,
                             float* __restrict__ rstd) {
    __shared__ float red[2][32];
    const int tpr = WARP ? 32 : int(blockDim.x);
    const int t = WARP ? int(threadIdx.x & 31) : int(threadIdx.x);
    const int64_t row =
        WARP ? int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : int64_t(blockIdx.x);
    if (WARP && row >= rows) return;  // whole warps
    constexpr int H = E == 4 ? 2 : 1;  // pairs of a chunk
    const T* xr = x + row * cols;
    Raw<T, E> v[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = (t + j * tpr) * E;
        v[j] = c < cols ? raw_load_once<T, E>(xr + c) : raw_zero<T, E>();
    }
    float2 s = both(0.0f);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        float2 f[H];
        raw_pairs(v[j], f);
#pragma unroll
        for (int i = 0; i < H; ++i) s = add2(s, f[i]);
    }
    const float inv_cols = 1.0f / float(cols);
    const float mu = row_sum<WARP>(s.x + s.y, red[0]) * inv_cols;
    s = both(0.0f);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        if ((t + j * tpr) * E < cols) {
            float2 f[H];
            raw_pairs(v[j], f);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const float2 d = add2(f[i], both(-mu));
                if (E == 1) s.x = fmaf(d.x, d.x, s.x);
                else s = fma2(d, d, s);
            }
        }
    }
    // (rsqrtf is within two steps of fp32)
    const float rs = rsqrtf(row_sum<WARP>(s.x + s.y, red[1]) * inv_cols + eps);
    if (t == 0) {
        if (mean) mean[row] = mu;
        if (rstd) rstd[row] = rs;
    }
    T* yr = y + row * cols;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = (t + j * tpr) * E;
        if (c < cols) {
            float2 f[H], w[H], b[H];
            load_pairs<E>(w, weight, c, 1.0f);
            load_pairs<E>(b, bias, c, 0.0f);
            raw_pairs(v[j], f);
#pragma unroll
            for (int i = 0; i < H; ++i)
                f[i] = fma2(mul2(add2(f[i], both(-mu)), both(rs)), w[i], b[i]);
            store_pairs(yr + c, f);
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
            float xv[E], dv[E], w[E], sc = 1.0f;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                xv[i] = mu;
                dv[i] = 0.0f;
                w[i] = 1.0f;
            }
            if (c < cols) {
                raw_floats(raw_load<X, E>(x + row * x_pitch + c), xv);
                if constexpr (sizeof(X) == 1) sc = x_scales[int64_t(c / kTile) * rows + row];
                raw_floats(raw_load<T, E>(dy + row * cols + c), dv);
                if (weight) raw_floats(raw_load<float, E>(weight + c), w);
            }
#pragma unroll
            for (int i = 0; i < E; ++i) {
                // (the difference rounded once; columns that are not there: 0)
                const float h = fmaf(xv[i], sc, -mu) * rs, gv = dv[i] * w[i];
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
        if (c < cols) {
            float a[E], b[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                a[i] = dw[j * E + i];
                b[i] = db[j * E + i];
            }
            store_floats(p + c, a);
            store_floats(p + cols + c, b);
        }
    }
}

// ------------------------------------------------------- streamed rows
constexpr int kMaxAhead = 8;
constexpr int kPerThread = 16;        // columns of a thread
constexpr int kStreamThreads = 512;   // of a CTA, so columns up to 8192
constexpr int kMaxCtas = 8;           // of an SM
constexpr int kSmBytes = 200 * 1024;  // shared memory of an SM for rows
constexpr int kSlotPad = 32;          // a row's 16-byte boundaries, before and after

// A matrix whose rows are copied into shared memory.
struct Rows {
    const char* base;    // 16-byte aligned
    int64_t pitch;       // bytes from row to row
    int64_t total;       // bytes of the matrix, rounded down to 16
    int bytes;           // of a row
};
// Bytes of row r that a copy brings: [first, last) from base.
__device__ __forceinline__ void row_range(const Rows& m, int64_t r, int64_t& first, int64_t& last) {
    const int64_t b = r * m.pitch;
    first = b & ~int64_t(15);
    last = min((b + m.bytes + 15) & ~int64_t(15), m.total);
}
__device__ __forceinline__ uint32_t row_copy(const Rows& m, int64_t r, uint32_t dst,
                                             uint32_t bar) {
    int64_t first, last;
    row_range(m, r, first, last);
    const uint32_t n = uint32_t(last - first);
    if (n == 0) return 0;  // a matrix of under 16 bytes from here on
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(dst),
        "l"(m.base + first), "r"(n), "r"(bar)
        : "memory");
    return n;
}
__device__ __forceinline__ uint32_t row_bytes(const Rows& m, int64_t r) {
    int64_t first, last;
    row_range(m, r, first, last);
    return uint32_t(last - first);
}
// A row in its slot: E elements from column c.  Rows of whole 16 bytes (E = 8)
// start where the slot does; the others at their place in 16 bytes, and the
// last elements of a matrix that ends inside 16 bytes are not in the slot
// (`have` columns are).
template <class T, int E>
struct RowView {
    const T* at;       // column 0 in the slot
    const T* memory;   // and in the matrix
    int have;
    __device__ __forceinline__ RowView(const Rows& m, int64_t row, const char* slot, int cols) {
        at = reinterpret_cast<const T*>(slot);
        if constexpr (E == 1) {
            const int64_t b = row * m.pitch;
            at = reinterpret_cast<const T*>(slot + int(b & 15));
            memory = reinterpret_cast<const T*>(m.base + b);
            have = int(min(int64_t(cols), (m.total - b) / int64_t(sizeof(T))));
        }
    }
    __device__ __forceinline__ void get(int c, float (&f)[E]) const {
        if constexpr (E == 8) {
            const T* p = at + c;
            Raw<T, 8> v;
            if constexpr (sizeof(T) == 4) {
                v.a = reinterpret_cast<const float4*>(p)[0];
                v.b = reinterpret_cast<const float4*>(p)[1];
            } else if constexpr (sizeof(T) == 2) {
                v.a = *reinterpret_cast<const uint4*>(p);
            } else {
                v.a = *reinterpret_cast<const uint2*>(p);
            }
            raw_floats(v, f);
        } else {
            f[0] = elem_float(c < have ? at[c] : memory[c]);
        }
    }
};

struct Stream {
    int slot;        // bytes of a row's place
    int ahead;       // rows copied ahead
    int* dev_status;
    uint64_t wait_limit_ns;
    int fault;       // FaultKind
};
struct StreamState {
    uint64_t full[kMaxAhead];
    int abort_flag;
};
// The slot of a CTA's next row, and the phase of its barrier.
struct Turn {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int ahead) {
        if (++slot == ahead) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// 16 columns a thread in chunks of E: chunk j starts at column (t + j tpr) E.
// Bound by the instructions of a row and the walk from one barrier to the next,
// not by memory: 48 us for 4096 rows of 7168 kept in 8 bits, which read and
// write 150 MB (23 us).  With 8 columns and twice the threads 60 us, where this
// form took 53 us (its partial sums were stored 4 bytes a lane then: 6 us).
template <class T, class X, int E>
__global__ void __launch_bounds__(kStreamThreads)
    layernorm_backward_stream(const Rows dy, const Rows x, const float* __restrict__ x_scales,
                              int64_t rows, int cols, const float* __restrict__ weight,
                              const float* __restrict__ mean, const float* __restrict__ rstd,
                              T* __restrict__ dx, float* __restrict__ part, const Stream st,
                              int x_slot) {
    constexpr bool KEPT = sizeof(X) == 1;
    constexpr int CH = kPerThread / E, P = kPerThread / 2;
    constexpr int kScales = kStreamThreads * kPerThread / kTile;  // tiles of a row, 64
    extern __shared__ __align__(128) char slots[];
    __shared__ StreamState ss;
    __shared__ __align__(16) float2 red[2][kStreamThreads / 32];  // (s1, s2) of each warp
    __shared__ float scale_s[2][KEPT ? kScales : 1];
    const int t = threadIdx.x, tpr = blockDim.x;
    const int64_t G = gridDim.x;
    auto issue = [&](int64_t row, int slot) {
        if (row >= rows || (st.fault == kFaultNormRows && row == blockIdx.x)) return;
        const uint32_t bar = tc::smem_u32(&ss.full[slot]);
        const uint32_t dst = tc::smem_u32(slots + slot * st.slot);
        tc::mbar_arrive_expect_tx(bar, row_bytes(x, row) + row_bytes(dy, row));
        row_copy(x, row, dst, bar);
        row_copy(dy, row, dst + x_slot, bar);
    };
    if (t == 0) {
        for (int i = 0; i < st.ahead; ++i) tc::mbar_init(tc::smem_u32(&ss.full[i]), 1);
        ss.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        for (int i = 0; i < st.ahead; ++i) issue(blockIdx.x + int64_t(i) * G, i);
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // a row's statistics and tile scales are fetched a row (two rows) ahead;
    // there are more threads than tiles
    const int tiles = (cols + kTile - 1) / kTile;
    int64_t row = blockIdx.x;
    float scale_next = 0.0f;
    if (KEPT && t < tiles) {
        scale_s[0][t] = x_scales[int64_t(t) * rows + row];
        if (row + G < rows) scale_next = x_scales[int64_t(t) * rows + row + G];
    }
    if (t < 2 * (kStreamThreads / 32)) red[0][t] = both(0.0f);  // of warps that are not there
    float mu = mean[row], rs = rstd[row];
    float2 w[P], dw[P], db[P];
#pragma unroll
    for (int k = 0; k < P; ++k) dw[k] = db[k] = both(0.0f);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = (t + j * tpr) * E;
        float wv[E];
#pragma unroll
        for (int e = 0; e < E; ++e) wv[e] = 1.0f;
        if (c < cols && weight) raw_floats(raw_load<float, E>(weight + c), wv);
#pragma unroll
        for (int e = 0; e < E; ++e) reinterpret_cast<float*>(w)[j * E + e] = wv[e];
    }
    __syncthreads();
    const float inv_cols = 1.0f / float(cols);
    const int lane = t & 31;
    T* dxr = dx + row * cols;
    const int64_t dx_step = G * cols;
    const int64_t far = int64_t(st.ahead) * G;
    Turn turn;
    int par = 0;
    for (; row < rows; row += G, dxr += dx_step, turn.next(st.ahead), par ^= 1) {
        const char* slot = slots + turn.slot * st.slot;
        const int64_t after = row + G;
        float mu_next = 0.0f, rs_next = 0.0f;
        if (after < rows) {
            mu_next = mean[after];
            rs_next = rstd[after];
        }
        const bool ok = tc::mbar_wait(tc::smem_u32(&ss.full[turn.slot]), turn.phase,
                                      &ss.abort_flag, st.dev_status, st.wait_limit_ns);
        float2 xh[P], g[P];
        float* const xf = reinterpret_cast<float*>(xh);
        float* const gf = reinterpret_cast<float*>(g);
        const RowView<X, E> xr(x, row, slot, cols);
        const RowView<T, E> dr(dy, row, slot + x_slot, cols);
        // xh = (x - mu) rstd, the difference first (of a kept value: code times
        // scale less mu, rounded once), so that xh's error is relative to xh
        // however far the row lies from zero
        const float2 minus_mu = both(-mu);
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = (t + j * tpr) * E;
            float xv[E], dv[E];
#pragma unroll
            for (int e = 0; e < E; ++e) xv[e] = dv[e] = 0.0f;
            float sc = 1.0f;
            if (c < cols) {
                xr.get(c, xv);
                dr.get(c, dv);
                if (KEPT) sc = scale_s[par][c / kTile];
            }
            // (no columns: dy 0 keeps them out of every sum)
            if constexpr (E == 8) {
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const float2 x2 = make_float2(xv[e], xv[e + 1]);
                    xh[(j * E + e) / 2] =
                        mul2(KEPT ? fma2(x2, both(sc), minus_mu) : add2(x2, minus_mu), both(rs));
                }
            } else {
                xf[j] = fmaf(xv[0], sc, -mu) * rs;
            }
#pragma unroll
            for (int e = 0; e < E; ++e) gf[j * E + e] = dv[e];
        }
        float2 s1 = both(0.0f), s2 = both(0.0f);
#pragma unroll
        for (int k = 0; k < P; ++k) {
            db[k] = add2(db[k], g[k]);
            dw[k] = fma2(g[k], xh[k], dw[k]);
            g[k] = mul2(g[k], w[k]);
            s1 = add2(s1, g[k]);
            s2 = fma2(g[k], xh[k], s2);
        }
        // both sums behind one barrier; the other parity's places are read
        // until the barrier after it
        float2 s = make_float2(s1.x + s1.y, s2.x + s2.y);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1)
            s = add2(s, make_float2(__shfl_xor_sync(0xffffffffu, s.x, o),
                                    __shfl_xor_sync(0xffffffffu, s.y, o)));
        if (lane == 0) red[par][t >> 5] = s;
        if (KEPT && t < tiles) {
            scale_s[par ^ 1][t] = scale_next;
            if (after + G < rows) scale_next = x_scales[int64_t(t) * rows + after + G];
        }
        if (__syncthreads_or(!ok)) break;
        if (t == 0) issue(row + far, turn.slot);  // everyone has read the slot
        // every thread adds up the warps' sums: eight broadcast loads take less
        // time than shuffles
        const float4* rp = reinterpret_cast<const float4*>(red[par]);
        float2 q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 u = rp[2 * i], v = rp[2 * i + 1];
            q[i] = add2(add2(make_float2(u.x, u.y), make_float2(u.z, u.w)),
                        add2(make_float2(v.x, v.y), make_float2(v.z, v.w)));
        }
        s = mul2(add2(add2(q[0], q[1]), add2(q[2], q[3])), both(-inv_cols * rs));
        // dx = rstd (g - m1 - xh m2)
#pragma unroll
        for (int k = 0; k < P; ++k)
            g[k] = fma2(g[k], both(rs), fma2(xh[k], both(s.y), both(s.x)));
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = (t + j * tpr) * E;
            if (c < cols) {
                float o[E];
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = gf[j * E + e];
                store_floats(dxr + c, o);
            }
        }
        mu = mu_next;
        rs = rs_next;
    }
    if (ss.abort_flag && t == 0)  // copies in flight land before the CTA leaves
        for (int k = 0; k < st.ahead; ++k, row += G, turn.next(st.ahead))
            if (row < rows)
                tc::mbar_quiesce(tc::smem_u32(&ss.full[turn.slot]), turn.phase, nullptr,
                                 tc::quiesce_ns(st.wait_limit_ns));
    if (!part) return;
    float* p = part + int64_t(blockIdx.x) * 2 * cols;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = (t + j * tpr) * E;
        if (c < cols) {
            float a[E], b[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                a[e] = reinterpret_cast<float*>(dw)[j * E + e];
                b[e] = reinterpret_cast<float*>(db)[j * E + e];
            }
            store_floats(p + c, a);
            store_floats(p + cols + c, b);
        }
    }
}

// A value that the kernel before this one writes: a plain load that the
// compiler leaves behind the wait, where one through a const __restrict__
// pointer counts as read-only for the whole kernel.
__device__ __forceinline__ float load_written(const float* p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
    return v;
}

// Column sums of the partial rows [n][2 cols]: a CTA per 32 columns, its 32
// warps take every 32nd row, then their sums are added in order.
__global__ void __launch_bounds__(1024) layernorm_sum_kernel(const float* part, int n, int cols,
                                                             float* __restrict__ dweight,
                                                             float* __restrict__ dbias) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float a = 0.0f;
    // (launched while the rows are still being walked)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (c < 2 * cols)
#pragma unroll 8
        for (int i = warp; i < n; i += 32) a += load_written(part + int64_t(i) * 2 * cols + c);
    s[warp][lane] = a;
    __syncthreads();
    // warp w adds up column w of the 32: lanes are the warps' sums
    a = warp_sum(s[lane][warp]);
    const int col = blockIdx.x * 32 + warp;
    if (lane == 0 && col < 2 * cols) {
        if (col < cols) {
            if (dweight) dweight[col] = a;
        } else if (dbias) {
            dbias[col - cols] = a;
        }
    }
}

int stream_threads(int cols) { return ((cols + kPerThread - 1) / kPerThread + 31) / 32 * 32; }

// CTAs of the backward pass: what an SM holds (512 threads of 128 registers),
// and no more than leave three rows to each (a CTA's partial sums are written
// and read once, as much as one or two rows; 1001 fp32 rows of 1477: 11.3 us,
// 12.6 with four rows, 11.6 with two; 1001 bf16 rows of 1480: 8.5, 9.4, 9.9).
int backward_per_sm(int cols) {
    return std::max(1, std::min(kMaxCtas, kStreamThreads / stream_threads(cols)));
}
int backward_ctas(int64_t rows, int cols) {
    const int64_t most = int64_t(sm_count()) * backward_per_sm(cols);
    return int(std::min(rows, std::min(most, std::max<int64_t>(sm_count(), rows / 3))));
}

// Rows ahead for `ctas` CTAs an SM and rows of `slot` bytes: two at least
// (two fp32 rows of 8192 columns and their gradients are 131 KB).
int rows_ahead(int slot, int ctas) {
    return std::max(2, std::min(kMaxAhead, kSmBytes / ctas / slot));
}
int slot_bytes(int64_t row) { return int((row + 15) / 16 * 16 + kSlotPad); }
Rows make_rows(const void* p, int64_t rows, int64_t pitch, int64_t bytes) {
    return Rows{static_cast<const char*>(p), pitch, rows * pitch / 16 * 16, int(bytes)};
}
// Leave for a launch of any size, never for this call's alone: the limit is the
// device's, and another thread may be between its own and its launch.
constexpr int kStreamSmem = std::max(kSmBytes, 2 * (2 * kPerThread * kStreamThreads * 4 + 2 * kSlotPad));
template <class K>
bool allow_smem(K kernel) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamSmem) ==
           cudaSuccess;
}
int round_threads(int chunks, int ch) { return ((chunks + ch - 1) / ch + 31) / 32 * 32; }

template <class T>
int forward_any(bool vec, const void* x, int64_t rows, int cols, const float* w, const float* b,
                float eps, void* y, float* mean, float* rstd, cudaStream_t st) {
    auto go = [&](auto kernel, int grid, int threads) {
        kernel<<<grid, threads, 0, st>>>(static_cast<const T*>(x), rows, cols, w, b, eps,
                                         static_cast<T*>(y), mean, rstd);
        return check_launch();
    };
    const int warps = int((rows + 3) / 4), n = int(rows);
    if (vec) {
        const int chunks = cols / 4;
        if (chunks <= 128) return go(layernorm_forward_kernel<T, 4, 4, true, 1>, warps, 128);
        if (chunks <= 256) return go(layernorm_forward_kernel<T, 4, 8, true, 1>, warps, 128);
        // rows of fp32 take twice the registers: 16 columns a thread (4096 rows
        // of 7168: 38.6 us, with 32 41.3 us; bf16 the other way, 104 and 93 us)
        if (chunks > 2048)
            return go(layernorm_forward_kernel<T, 4, 8, false, 1>, n, round_threads(chunks, 8));
        if constexpr (sizeof(T) == 4)
            return go(layernorm_forward_kernel<T, 4, 4, false, 2>, n, round_threads(chunks, 4));
        else
            return go(layernorm_forward_kernel<T, 4, 8, false, 5>, n, round_threads(chunks, 8));
    }
    if (cols <= 256) return go(layernorm_forward_kernel<T, 1, 8, true, 1>, warps, 128);
    if (cols <= 4096)
        return go(layernorm_forward_kernel<T, 1, 16, false, 4>, n, round_threads(cols, 16));
    return go(layernorm_forward_kernel<T, 1, 16, false, 1>, n, round_threads(cols, 16));
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
    int* dev_status;
};

template <class T, class X, int E, int CH>
int backward_launch(const BwdArgs& a, int threads, cudaStream_t st) {
    layernorm_backward_kernel<T, X, E, CH><<<backward_ctas(a.rows, a.cols), threads, 0, st>>>(
        static_cast<const T*>(a.dy), static_cast<const X*>(a.x), a.x_scales, a.rows, a.cols,
        a.x_pitch, a.weight, a.mean, a.rstd, static_cast<T*>(a.dx), a.part);
    return check_launch();
}

template <class T, class X, int E>
int backward_stream(const BwdArgs& a, int x_slot, const Stream& s, cudaStream_t st) {
    const int bytes = s.slot * s.ahead;
    if (!allow_smem(layernorm_backward_stream<T, X, E>)) return cuda_failed();
    const int64_t row = int64_t(a.cols) * int64_t(sizeof(T));
    layernorm_backward_stream<T, X, E>
        <<<backward_ctas(a.rows, a.cols), stream_threads(a.cols), bytes, st>>>(
            make_rows(a.dy, a.rows, row, row),
            make_rows(a.x, a.rows, a.x_pitch * int64_t(sizeof(X)),
                      int64_t(a.cols) * int64_t(sizeof(X))),
            a.x_scales, a.rows, a.cols, a.weight, a.mean, a.rstd, static_cast<T*>(a.dx), a.part, s,
            x_slot);
    return check_launch();
}

template <class T, class X>
int backward_any(bool vec, const BwdArgs& a, cudaStream_t st) {
    if (a.cols <= kPerThread * kStreamThreads && aligned16(a.dy) && aligned16(a.x)) {
        const int x_slot = slot_bytes(int64_t(a.cols) * int64_t(sizeof(X)));
        Stream s;
        s.slot = x_slot + slot_bytes(int64_t(a.cols) * int64_t(sizeof(T)));
        s.ahead = rows_ahead(s.slot, backward_per_sm(a.cols));
        s.dev_status = a.dev_status;
        s.wait_limit_ns = wait_limit_ns();
        s.fault = fault_injection();
        return vec ? backward_stream<T, X, 8>(a, x_slot, s, st)
                   : backward_stream<T, X, 1>(a, x_slot, s, st);
    }
    if (vec) return backward_launch<T, X, 8, 2>(a, round_threads(a.cols / 8, 2), st);
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
    return size_t(backward_ctas(rows, cols)) * 2 * size_t(cols) * sizeof(float);
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
    if (!aligned(x, es) || !aligned(y, es) || !aligned(weight, 4) || !aligned(bias, 4) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return MOE_ERR_ALIGN;
    if (!device_is_sm100()) return MOE_ERR_DEVICE;
    const bool vec = cols % 4 == 0 && aligned16(x) && aligned16(y) && aligned16(weight) &&
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
                return cuda_failed();
        return MOE_OK;
    }
    if (!dy || !x || !mean || !rstd || !dx) return MOE_ERR_NULL;
    if (x_type == MOE_T_CKPT && !x_scales) return MOE_ERR_NULL;
    const size_t es = type_size(type);
    if (!aligned(dy, es) || !aligned(dx, es) || !aligned(weight, 4) ||
        !aligned(x, type_size(x_type)) || !aligned(x_scales, 4) || !aligned(mean, 4) ||
        !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(dbias, 4))
        return MOE_ERR_ALIGN;
    if (x_type == MOE_T_CKPT && !aligned16(x)) return MOE_ERR_ALIGN;
    const bool sums = dweight || dbias;
    if (sums && (!ws || ws_bytes < backward_ws(rows, cols))) return MOE_ERR_WORKSPACE;
    if (sums && !aligned16(ws)) return MOE_ERR_ALIGN;
    if (!device_is_sm100()) return MOE_ERR_DEVICE;
    const bool vec = cols % 8 == 0 && aligned16(dy) && aligned16(x) && aligned16(dx) &&
                     aligned16(weight);
    BwdArgs a{dy, x, x_scales, rows, cols, x_type == MOE_T_CKPT ? ckpt_row_bytes(cols) : cols,
              weight, mean, rstd, dx, sums ? static_cast<float*>(ws) : nullptr, dev_status};
    int rc = type == MOE_T_F32    ? backward_typed<float>(x_type, type, vec, a, st)
             : type == MOE_T_BF16 ? backward_typed<bf16_t>(x_type, type, vec, a, st)
                                  : backward_typed<f16_t>(x_type, type, vec, a, st);
    if (rc != MOE_OK || !sums) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((2 * cols + 31) / 32), 1, 1);
    cfg.blockDim = dim3(1024, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, layernorm_sum_kernel, static_cast<const float*>(a.part),
                           backward_ctas(rows, cols), cols, dweight, dbias) != cudaSuccess)
        return cuda_failed();
    return check_launch();
}
