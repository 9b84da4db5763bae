// Dense gated feed-forward block in 16 bits (bf16 or fp16), forward and
// backward, on tcgen05.
//
//   a = x W1^T, c = x W3^T, h = silu(a) c, y = h W2^T
//   dh = dy W2, s = sigmoid(a), da = dh c s (1 + a (1 - s)), dc = dh a s
//   dx = da W1 + dc W3, dW13 = [da | dc]^T x, dW2 = dy^T h
//
// Every product runs through one kernel: CTA pairs (cta_group::2) of 256 x
// (up to 256) output tiles, 64 K elements a stage, six stages fed by TMA,
// the fp32 accumulator in TMEM twice, so that a tile's epilogue runs under
// the next tile's products.  An operand whose K runs along its rows in
// memory (W2 and W13 in the backward pass, all operands of the weight
// gradients) is read as it lies, as an MN-major tile: nothing is transposed
// in memory.  The epilogues are the element-wise steps:
//   kGated     a and c of the same 128 (or 64) features lie in one tile (one
//              CTA of the pair loads their rows of W1, the other those of W3):
//              h, and where asked a and c kept for the backward pass, in 8
//              bits (1x128 tiles) or in 16;
//   kBackward  dh stays in TMEM: da, dc and h from it and the kept a, c;
//   kPlain     the product.
// dx, dW13 and dW2 do not depend on one another and are one launch over one
// list of tiles, so that the last round of tiles is left part empty once and
// not three times.
//
// Few tokens leave most pairs without a tile, and one token's work is reading
// the weights once.  There the operands change places (few_kernel): 128 rows
// of weights are the M side, up to 256 tokens the N side, and a cluster of up
// to eight CTAs splits K, so that every SM streams weights; the partial sums
// meet in shared memory across the cluster, in a fixed order.  One to four
// tokens are matrix-vector products on the CUDA cores (vec_kernel).  In both
// forms the second product's kernel starts under the first's end and fetches
// weights before it waits for h.
//
// Accumulators are fp32.  h and [da | dc] are rounded to the operands' type
// between two products (the tensor cores take 16-bit operands); everything
// else is rounded once, on output.  Bound by the tensor cores for hundreds of
// tokens and more.
#include <cuda.h>

#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "elem.cuh"
#include "tc_pair.cuh"

namespace moe {

// 2D map over [rows, cols] with a row pitch in bytes, any element type and
// box (defined with the grouped GEMM).
bool make_map_2d(CUtensorMap* m, CUtensorMapDataType type, const void* base, uint64_t rows,
                 uint64_t cols, uint64_t pitch_bytes, uint32_t box_rows,
                 uint32_t box_cols, CUtensorMapSwizzle swizzle, CUtensorMapL2promotion promote);

namespace {

using namespace tc;

enum Epilogue { kPlain = 0, kGated = 1, kBackward = 2 };
enum Kept { kKeptNone = 0, kKept8 = 1, kKept16 = 2 };

constexpr int kThreads = 384;
constexpr int kStages = 6;
constexpr int kTileM = 256;               // rows of a pair's tile, 128 a CTA
constexpr int kTileK = 64;                // K elements of a stage
constexpr int kOperandBytes = 128 * 128;  // 128 rows of 64 16-bit elements
constexpr int kPieceBytes = 64 * 128;     // MN-major piece: 64 K x 64 elements
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kEpiWarps = 8;
constexpr int kChunk = 32;                // output columns of one epilogue step
constexpr int kBoxBytes = 32 * 64;        // 32 rows x 32 16-bit elements
constexpr int kMaxProblems = 3;
constexpr int kGroupM = 8;                // row tiles walked together

struct Problem {
    CUtensorMap a, b, out;
    int m, n;                // output rows and columns
    int nkb;                 // stages of K
    int nt;                  // tile columns (multiple of 32, at most 256); kGated: of a and of c, nt / 2
                             // features
    int tiles_m, tiles_n;
    int first;               // index of its first tile in the launch's list
    int a_mn, b_mn;          // operand's K runs along its rows in memory
};

struct Args {
    Problem p[kMaxProblems];
    CUtensorMap o1, o2;      // kGated 16-bit a, c; kBackward dc, h
    int n_problems;
    int tiles;
    int inter;
    int64_t rows;            // tokens
    void* ac;                // kept a, c
    float* ac_scales;
    int wait_first;          // 1: operands come from the kernel before this one
    int* dev_status;
    uint64_t wait_limit_ns;
    int fault;               // FaultKind
};

struct Shared {
    uint64_t full[kStages];
    uint64_t empty[kStages];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t drain;
    PairState ps;
    uint32_t tmem_base;
    uint32_t issued[4];      // the leader's: steps that each of the pair's producers has loaded
};

template <int EPI>
struct Cfg {
    static constexpr int kBoxes = EPI == kGated ? 1 : 2;  // parked boxes per epilogue warp
    static constexpr int kParkBytes = kEpiWarps * kBoxes * kBoxBytes;
    // kGated: amax of a and c, [tile parity][column half][a, c][row]
    static constexpr int kRedBytes = EPI == kGated ? 2 * 2 * 2 * 128 * 4 : 0;
    static constexpr size_t kSmem =
        size_t(kStages) * kStageBytes + kParkBytes + kRedBytes + sizeof(Shared) + 1024;
};
static_assert(Cfg<kPlain>::kSmem <= 232448 && Cfg<kGated>::kSmem <= 232448 &&
                  Cfg<kBackward>::kSmem <= 232448,
              "dynamic shared memory above the sm_100 limit per CTA");

struct Tile {
    int p;       // problem
    int m0, n0;  // first row; first column (kGated: first feature)
};

// Tiles of a problem in groups of kGroupM row tiles, rows fastest: the tiles
// that run side by side share few operand tiles, which stay in L2.
template <int EPI>
__device__ __forceinline__ Tile decode_for(const Args& a, int t) {
    Tile r;
    r.p = 0;
    while (r.p + 1 < a.n_problems && t >= a.p[r.p + 1].first) ++r.p;
    const Problem& p = a.p[r.p];
    t -= p.first;
    const int per_group = kGroupM * p.tiles_n;
    const int g = t / per_group;
    const int in_g = t - g * per_group;
    const int gm = min(kGroupM, p.tiles_m - g * kGroupM);
    r.m0 = (g * kGroupM + in_g % gm) * kTileM;
    r.n0 = (in_g / gm) * (EPI == kGated ? p.nt / 2 : p.nt);
    return r;
}

// ------------------------------------------------ TMA producers (warps 0 and 2)
// Warp 0 loads A and announces the stage's bytes, warp 2 loads B.
template <int EPI, bool IS_A>
__device__ __forceinline__ void producer(const Args& a, uint8_t* smem, Shared* ss, int rank,
                                         int unit, int units) {
    const bool lead = elect_one();
    // the leader's barrier of stage 0
    const uint32_t bar0 = uniform(mapa(smem_u32(&ss->full[0]), 0));
    uint32_t s = 0, par = 1, issued = 0;
    bool ok = true;
    for (int t = unit; ok && t < a.tiles; t += units) {
        const Tile w = decode_for<EPI>(a, t);
        const Problem& p = a.p[w.p];
        const int half = p.nt / 2;
        // this CTA's rows of A; and of B: half the tile's columns, or the
        // features' rows of W1 (rank 0) and of W3 (rank 1)
        const int first =
            IS_A ? w.m0 + 128 * rank : w.n0 + rank * (EPI == kGated ? a.inter : half);
        const CUtensorMap* map = IS_A ? &p.a : &p.b;
        const int mn = IS_A ? p.a_mn : p.b_mn;
        const int b_pieces = (half + 63) / 64;
        const int pieces = IS_A ? 2 : b_pieces;
        const uint32_t tx = 2 * (kOperandBytes + (p.b_mn ? b_pieces * kPieceBytes : half * 128));
        const int nkb = p.nkb;
        for (int kb = 0; kb < nkb; ++kb) {
            ok = pair_wait(smem_u32(&ss->empty[s]), par, &ss->ps, a.dev_status);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            const uint32_t dst =
                smem_u32(smem) + s * uint32_t(kStageBytes) + (IS_A ? 0u : uint32_t(kOperandBytes));
            const uint32_t bar = bar0 + 8 * s;
            const int k0 = kb * kTileK;
            const bool withheld =
                IS_A && rank == 0 && a.fault == kFaultFfnProducer && issued == 0;
            if (lead && !withheld) {
                if (IS_A && rank == 0) mbar_arrive_expect_tx(smem_u32(&ss->full[s]), tx);
                if (mn) {
                    pair_tma_load_2d(dst, map, bar, first, k0);
                    if (pieces > 1) pair_tma_load_2d(dst + kPieceBytes, map, bar, first + 64, k0);
                } else {
                    pair_tma_load_2d(dst, map, bar, k0, first);
                }
            }
            ++issued;
            if (++s == kStages) {
                s = 0;
                par ^= 1u;
            }
        }
    }
    if (lead) st_cluster(mapa(smem_u32(&ss->issued[2 * rank + (IS_A ? 0 : 1)]), 0), issued);
    __syncwarp();
}

// ------------------------------------------------ MMA issuer (warp 1 of the leader)
template <int EPI, bool BF16>
__device__ __forceinline__ void issuer(const Args& a, uint8_t* smem, Shared* ss,
                                       uint32_t tmem_base, int unit, int units) {
    const bool lead = elect_one();
    uint32_t s = 0, par = 0, n = 0;
    bool ok = true;
    const uint64_t desc0 = sw128_desc16(smem_u32(smem), kPieceBytes);
    for (int t = unit; ok && t < a.tiles; t += units, ++n) {
        const Tile w = decode_for<EPI>(a, t);
        const Problem& p = a.p[w.p];
        const uint32_t idesc = idesc_f16(BF16, p.a_mn, p.b_mn, kTileM, p.nt);
        // bytes per 16 K elements, in descriptor units of 16
        const uint32_t a_step = p.a_mn ? 2048 / 16 : 32 / 16;
        const uint32_t b_step = p.b_mn ? 2048 / 16 : 32 / 16;
        const uint32_t d = tmem_base + (n & 1) * 256;
        const int nkb = p.nkb;
        ok = pair_wait(smem_u32(&ss->tempty[n & 1]), ((n >> 1) & 1u) ^ 1u, &ss->ps, a.dev_status);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        fence_after();
        for (int kb = 0; kb < nkb; ++kb) {
            ok = pair_wait(smem_u32(&ss->full[s]), par, &ss->ps, a.dev_status);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            fence_after();
            const uint64_t ad = desc0 + s * uint32_t(kStageBytes / 16);
            const uint64_t bd = ad + kOperandBytes / 16;
            if (lead) {
#pragma unroll
                for (int kk = 0; kk < kTileK / 16; ++kk)
                    pair_mma_f16(d, ad + kk * a_step, bd + kk * b_step, idesc,
                                 (kb | kk) ? 1u : 0u);
                pair_commit_both(smem_u32(&ss->empty[s]));
            }
            __syncwarp();
            if (++s == kStages) {
                s = 0;
                par ^= 1u;
            }
        }
        if (ok && lead) pair_commit_both(smem_u32(&ss->tfull[n & 1]));
        __syncwarp();
    }
    if (lead) {
        // every MMA has completed once this fires (after an abort too)
        pair_commit(smem_u32(&ss->drain));
        mbar_quiesce(smem_u32(&ss->drain), 0, nullptr, quiesce_ns(ss->ps.wait_limit));
    }
    __syncwarp();
}

// ------------------------------------------------ epilogue (warps 4-11)
// One 32-column step of a warp's 32 rows: rounded to T, parked in the 64-byte
// swizzle of the output map (16-byte piece j of row r at j ^ (r / 2 % 4)) and
// handed to the TMA engine, which clips rows and columns past the end.
template <class T, int BOXES>
__device__ __forceinline__ void put32(const float (&v)[32], char* park, int& box,
                                      const CUtensorMap* map, int x, int y, bool any) {
    const int lane = threadIdx.x & 31;
    char* const b = park + box * kBoxBytes;
    box = box + 1 == BOXES ? 0 : box + 1;
    if (lane == 0) bulk_wait_read<BOXES - 1>();
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4*>(b + lane * 64 + ((j ^ ((lane >> 1) & 3)) * 16)) = make_uint4(
            pack2t(T(), v[8 * j], v[8 * j + 1]), pack2t(T(), v[8 * j + 2], v[8 * j + 3]),
            pack2t(T(), v[8 * j + 4], v[8 * j + 5]), pack2t(T(), v[8 * j + 6], v[8 * j + 7]));
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
        if (any) tma_store_2d(map, smem_u32(b), x, y);
        bulk_commit();
    }
}

// sigmoid from the fast exponential and reciprocal (about 1e-6 relative, where
// what follows is rounded to 16 bits: 5e-4 in fp16, 4e-3 in bf16; e^-a = inf
// gives 0)
__device__ __forceinline__ float sigmoid_fast(float a) {
    return __fdividef(1.0f, 1.0f + __expf(-a));
}

// da, dc and h of one feature from dh and the kept a and c.
__device__ __forceinline__ void gated_backward(float dh, float a, float c, float& da, float& dc,
                                               float& h) {
    const float s = sigmoid_fast(a);
    const float as = a * s, ds = dh * s;
    h = as * c;
    dc = dh * as;
    da = ds * c * fmaf(a, 1.0f - s, 1.0f);
}

// 4 values -> their codes
__device__ __forceinline__ uint32_t codes4(const float* v, float inv) {
    return e4m3x2(__fmul_rn(v[0], inv), __fmul_rn(v[1], inv)) |
           (uint32_t(e4m3x2(__fmul_rn(v[2], inv), __fmul_rn(v[3], inv))) << 16);
}

// 32 values -> 32 codes at q (32-byte aligned)
__device__ __forceinline__ void put_codes(uint8_t* q, const float (&v)[32], float inv) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = codes4(v + 16 * j + 4 * i, inv);
        reinterpret_cast<uint4*>(q)[j] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// A step's kept a and c of one row, as they lie in memory.
template <int KEPT>
struct KeptRaw {
    uint4 a[KEPT == kKept8 ? 2 : 4], c[KEPT == kKept8 ? 2 : 4];
    float sa, sc;
};
template <int KEPT>
__device__ __forceinline__ KeptRaw<KEPT> load_kept(const Args& a, int64_t row, int f) {
    KeptRaw<KEPT> k;
    memset(&k, 0, sizeof(k));
    if (row < a.rows && f < a.inter) {
        if constexpr (KEPT == kKept8) {
            const int64_t wide = (a.inter + kTile - 1) / kTile * kTile;
            const uint8_t* q = static_cast<const uint8_t*>(a.ac) + row * 2 * wide + f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                k.a[j] = __ldg(reinterpret_cast<const uint4*>(q) + j);
                k.c[j] = __ldg(reinterpret_cast<const uint4*>(q + wide) + j);
            }
            k.sa = __ldg(a.ac_scales + int64_t(f / kTile) * a.rows + row);
            k.sc = __ldg(a.ac_scales + (wide / kTile + f / kTile) * a.rows + row);
        } else {
            const uint16_t* q = static_cast<const uint16_t*>(a.ac) + row * 2 * a.inter + f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (f + 8 * j < a.inter) {
                    k.a[j] = __ldg(reinterpret_cast<const uint4*>(q) + j);
                    k.c[j] = __ldg(reinterpret_cast<const uint4*>(q + a.inter) + j);
                }
        }
    }
    return k;
}
// Values 8 j .. 8 j + 7 of a step.
template <class T, int KEPT>
__device__ __forceinline__ void kept_floats(const uint4* q, int j, float s, float (&f)[8]) {
    if constexpr (KEPT == kKept8) {
        const uint4 w = q[j / 2];
        Raw<e4m3_t, 8> r;
        r.a = j & 1 ? make_uint2(w.z, w.w) : make_uint2(w.x, w.y);
        raw_floats(r, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= s;
    } else {
        Raw<T, 8> r;
        r.a = q[j];
        raw_floats(r, f);
    }
}

template <int EPI, int KEPT, class T>
__device__ __forceinline__ void epilogue(const Args& a, Shared* ss, char* park_area, float* red,
                                         uint32_t tmem_base, int rank, int unit, int units) {
    constexpr int BOXES = Cfg<EPI>::kBoxes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane_addr = tmem_base + (uint32_t(q * 32) << 16);
    char* const park = park_area + (warp - 4) * (BOXES * kBoxBytes);
    int box = 0;
    uint32_t n = 0;
    for (int t = unit; t < a.tiles; t += units, ++n) {
        const Tile w = decode_for<EPI>(a, t);
        const Problem& p = a.p[w.p];
        const int y0 = w.m0 + 128 * rank + 32 * q;
        const int64_t row = y0 + lane;
        const bool rows_any = y0 < p.m;
        constexpr int RAW = KEPT == kKept16 ? kKept16 : kKept8;
        KeptRaw<RAW> kept;
        if constexpr (EPI == kBackward) kept = load_kept<RAW>(a, row, w.n0 + kChunk * half);
        bool ok = true;
        if (lane == 0)
            ok = pair_wait(smem_u32(&ss->tfull[n & 1]), (n >> 1) & 1u, &ss->ps, a.dev_status);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        // all epilogue warps agree on whether to go on
        if (named_bar_or(2, kEpiWarps * 32,
                         !ok || *reinterpret_cast<volatile int*>(&ss->ps.abort_flag)))
            break;
        fence_after();
        const uint32_t tm = lane_addr + (n & 1) * 256;
        if constexpr (EPI == kPlain) {
            for (int ch = half; ch < p.nt / kChunk; ch += 2) {
                uint32_t v[32];
                tmem_ld32(tm + ch * kChunk, v);
                float f[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
                const int x = w.n0 + ch * kChunk;
                put32<T, BOXES>(f, park, box, &p.out, x, y0, rows_any && x < p.n);
            }
        } else if constexpr (EPI == kGated) {
            float ia = 1.0f, ic = 1.0f;
            const int64_t wide = (a.inter + kTile - 1) / kTile * kTile;
            if constexpr (KEPT == kKept8) {
                // a first look at the tile for the 1x128 scales of a and c;
                // each warp sees 64 of the 128 features, its partner the rest
                float ma = 0.0f, mc = 0.0f;
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
                    const int col = 64 * half + kChunk * ch;
                    uint32_t va[32], vc[32];
                    tmem_ld32(tm + col, va);
                    tmem_ld32(tm + 128 + col, vc);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (w.n0 + col + (i & ~7) < a.inter) {  // 8 features exist together
                            ma = fmaxf(ma, fabsf(__uint_as_float(va[i])));
                            mc = fmaxf(mc, fabsf(__uint_as_float(vc[i])));
                        }
                }
                float* const r = red + (n & 1) * 512 + q * 32 + lane;
                r[half * 256] = ma;
                r[half * 256 + 128] = mc;
                named_bar(1, kEpiWarps * 32);
                ma = fmaxf(ma, r[(half ^ 1) * 256]);
                mc = fmaxf(mc, r[(half ^ 1) * 256 + 128]);
                float sa, sc;
                kept_scale(ma, sa, ia);
                kept_scale(mc, sc, ic);
                if (half == 0 && row < a.rows) {
                    a.ac_scales[int64_t(w.n0 / kTile) * a.rows + row] = sa;
                    a.ac_scales[(wide / kTile + w.n0 / kTile) * a.rows + row] = sc;
                }
            }
            const int features = p.nt / 2;
#pragma unroll 1
            for (int col = features / 2 * half; col < features / 2 * (half + 1); col += kChunk) {
                const int x = w.n0 + col;
                uint32_t va[32], vc[32];
                tmem_ld32(tm + col, va);
                tmem_ld32(tm + features + col, vc);
                float fa[32], fc[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    fa[i] = __uint_as_float(va[i]);
                    fc[i] = __uint_as_float(vc[i]);
                }
                if constexpr (KEPT == kKept8) {
                    if (row < a.rows) {
                        // columns past the last feature (rows of W3 for a) are kept as zeros
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (x + (i & ~7) >= a.inter) fa[i] = fc[i] = 0.0f;
                        uint8_t* o = static_cast<uint8_t*>(a.ac) + row * 2 * wide + x;
                        put_codes(o, fa, ia);
                        put_codes(o + wide, fc, ic);
                    }
                } else if constexpr (KEPT == kKept16) {
                    put32<T, BOXES>(fa, park, box, &a.o1, x, y0, rows_any && x < a.inter);
                    put32<T, BOXES>(fc, park, box, &a.o2, x, y0, rows_any && x < a.inter);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) fa[i] = fa[i] * sigmoid_fast(fa[i]) * fc[i];
                put32<T, BOXES>(fa, park, box, &p.out, x, y0, rows_any && x < a.inter);
            }
        } else {
            for (int ch = half; ch < p.nt / kChunk; ch += 2) {
                const int x = w.n0 + ch * kChunk;
                uint32_t v[32];
                tmem_ld32(tm + ch * kChunk, v);
                const int after = ch + 2 < p.nt / kChunk ? x + 2 * kChunk : a.inter;
                const KeptRaw<RAW> next = load_kept<RAW>(a, row, after);
                float da[32], dc[32], h[32];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float ka[8], kc[8];
                    kept_floats<T, KEPT>(kept.a, j, kept.sa, ka);
                    kept_floats<T, KEPT>(kept.c, j, kept.sc, kc);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        gated_backward(__uint_as_float(v[8 * j + i]), ka[i], kc[i], da[8 * j + i],
                                       dc[8 * j + i], h[8 * j + i]);
                }
                const bool any = rows_any && x < a.inter;
                put32<T, BOXES>(da, park, box, &p.out, x, y0, any);
                put32<T, BOXES>(dc, park, box, &a.o1, x, y0, any);
                put32<T, BOXES>(h, park, box, &a.o2, x, y0, any);
                kept = next;
            }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa(smem_u32(&ss->tempty[n & 1]), 0));
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
    fence_before();
}

template <int EPI, int KEPT, class T>
__global__ void __launch_bounds__(kThreads, 1) ffn_kernel(const __grid_constant__ Args a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    char* park = reinterpret_cast<char*>(smem + kStages * kStageBytes);
    float* red = reinterpret_cast<float*>(park + Cfg<EPI>::kParkBytes);
    Shared* ss = reinterpret_cast<Shared*>(park + Cfg<EPI>::kParkBytes + Cfg<EPI>::kRedBytes);
    const int warp = int(uniform(threadIdx.x >> 5));
    const int rank = int(blockIdx.x & 1);  // clusters are pairs along x
    const int unit = int(blockIdx.x >> 1), units = int(gridDim.x >> 1);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&ss->full[s]), 1);
            mbar_init(smem_u32(&ss->empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&ss->tfull[b]), 1);
            mbar_init(smem_u32(&ss->tempty[b]), 2 * kEpiWarps);
        }
        mbar_init(smem_u32(&ss->drain), 1);
        ss->ps.wait_limit = a.wait_limit_ns;
        ss->ps.abort_flag = 0;
        ss->ps.peer_abort = mapa(smem_u32(&ss->ps.abort_flag), uint32_t(rank ^ 1));
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) pair_tmem_alloc(smem_u32(&ss->tmem_base));
    if (threadIdx.x >= 96 && threadIdx.x < 96 + 2 * a.n_problems) {
        const Problem& p = a.p[(threadIdx.x - 96) >> 1];
        prefetch_map(threadIdx.x & 1 ? &p.b : &p.a);
    }
    fence_before();
    __syncthreads();
    cluster_sync();  // the peer's barriers exist before anyone signals them
    fence_after();
    // The next launch may set itself up as this one's CTAs leave; its loads
    // and stores wait for this grid's end.
    launch_dependents();
    if (a.wait_first) wait_dependencies();
    const uint32_t tmem_base = uniform(ss->tmem_base);
    if (warp == 0)
        producer<EPI, true>(a, smem, ss, rank, unit, units);
    else if (warp == 2)
        producer<EPI, false>(a, smem, ss, rank, unit, units);
    else if (warp == 1 && rank == 0)
        issuer<EPI, std::is_same<T, bf16_t>::value>(a, smem, ss, tmem_base, unit, units);
    else if (warp >= 4)
        epilogue<EPI, KEPT, T>(a, ss, park, red, tmem_base, rank, unit, units);
    __syncthreads();
    // neither CTA leaves while the other may still signal its barriers or
    // the leader's MMAs may still read its shared memory
    cluster_sync();
    // Given up (both CTAs' flags are raised together, and by nobody any more):
    // loads of either CTA may be in flight, whichever wait ran out.  The
    // barriers they arrive on are the leader's.
    if (*reinterpret_cast<volatile int*>(&ss->ps.abort_flag)) {
        if (rank == 0 && threadIdx.x == 0) {
            const volatile uint32_t* n = ss->issued;
            ring_quiesce(ss->full, kStages, max(max(n[0], n[1]), max(n[2], n[3])),
                         ss->ps.wait_limit);
        }
        __syncwarp();
        cluster_sync();
    }
    if (warp == 1) {
        fence_after();
        pair_tmem_free(tmem_base);
    }
}

// ================================================== few tokens: split K
// out[t, r] = sum_k W[r, k] x[t, k] for 128 rows r of W a CTA: W is the M side
// of the MMA (a row per TMEM lane), nt tokens the N side.
//   kFewPlain     the product
//   kFewTurned    the same with W as [k, r] in memory, read as it lies (dx)
//   kFewGated     64 rows of W1 in lanes 0-63 and the same 64 of W3 in lanes
//                 64-127: h
//   kFewKept      the same, and a and c kept; two CTAs of the cluster have the
//                 128 features of a tile between them
//   kFewBackward  W2 as [k, r]: dh, and from it and the kept a, c: da, dc, h
//   warp 0 TMA producer, warp 1 MMA issuer, warps 2-9 move the accumulator
//   into shared memory (over the stages, all consumed by then); then every
//   CTA of the cluster adds up its share of the tokens, ranks in order.
constexpr int kFewThreads = 320;
constexpr int kFewMaxStages = 12;
constexpr int kFewRing1 = 200 * 1024;  // stages of a CTA alone on its SM,
constexpr int kFewRing2 = 106 * 1024;  // and of two on one
constexpr int kFewShared = 64;         // tokens up to which two share an SM
constexpr int kFewMaxTokens = 256;  // N side of one tile
constexpr int kFewMaxSplit = 8;     // portable cluster size

enum FewMode { kFewPlain, kFewTurned, kFewGated, kFewKept, kFewBackward };
constexpr bool few_gated(int mode) { return mode == kFewGated || mode == kFewKept; }
constexpr bool few_turned(int mode) { return mode == kFewTurned || mode == kFewBackward; }

struct FewArgs {
    CUtensorMap w, x;
    void* out;      // kFewBackward: [da | dc]
    void* h;        // kFewBackward
    void* ac;       // kFewKept (out), kFewBackward (in)
    float* ac_scales;
    int kept;
    int rows;       // output columns (W2's rows, or features)
    int pitch;      // of out
    int w3;         // GATED: first row of W3
    int64_t tokens;
    int nt;         // tokens of a tile, a multiple of 16
    int nkb;
    int ring;       // bytes of the stages
    int stages;
    int wait_first; // 1: x comes from the kernel before this one
    int* dev_status;
    uint64_t wait_limit_ns;
    int fault;      // FaultKind
};

struct FewShared {
    uint64_t full[kFewMaxStages];
    uint64_t empty[kFewMaxStages];
    uint64_t done;
    uint32_t tmem_base;
    int abort_flag;
};
constexpr size_t few_smem(int ring) { return size_t(ring) + sizeof(FewShared) + 1024; }
static_assert(kFewMaxTokens * 128 * 4 <= kFewRing1 && kFewShared * 128 * 4 <= kFewRing2,
              "the partial sums lie over the stages");
static_assert(few_smem(kFewRing1) <= 232448 && 2 * (few_smem(kFewRing2) + 1024) <= 233472,
              "shared memory of an SM");

// Two neighbouring features' kept a and c of one token.
template <class T>
struct KeptPair {
    uint32_t a, c;
    float sa, sc;
    __device__ __forceinline__ void load(const FewArgs& g, int64_t t, int f) {
        a = c = 0u;
        sa = sc = 0.0f;
        if (f >= g.rows) return;
        if (g.kept == kKept8) {
            const int64_t wide = (g.rows + kTile - 1) / kTile * kTile;
            const uint8_t* q = static_cast<const uint8_t*>(g.ac) + t * 2 * wide + f;
            a = __ldg(reinterpret_cast<const uint16_t*>(q));
            c = __ldg(reinterpret_cast<const uint16_t*>(q + wide));
            sa = __ldg(g.ac_scales + int64_t(f / kTile) * g.tokens + t);
            sc = __ldg(g.ac_scales + (wide / kTile + f / kTile) * g.tokens + t);
        } else {
            const T* q = static_cast<const T*>(g.ac) + t * 2 * g.rows + f;
            a = __ldg(reinterpret_cast<const uint32_t*>(q));
            c = __ldg(reinterpret_cast<const uint32_t*>(q + g.rows));
        }
    }
    __device__ __forceinline__ void get(const FewArgs& g, float2& va, float2& vc) const {
        if (g.kept == kKept8) {
            va = mul2(e4m3x2_to_float2(uint16_t(a)), both(sa));
            vc = mul2(e4m3x2_to_float2(uint16_t(c)), both(sc));
        } else {
            unpack2f(T(), a, va.x, va.y);
            unpack2f(T(), c, vc.x, vc.y);
        }
    }
};

// The sums of this CTA's share of the tile over the cluster's partial sums,
// ranks in order, and the output.  A warp takes 64 columns of a token at a
// time, two a lane; eight ranks' loads, or several tokens' of fewer ranks, are
// in flight together.
template <int MODE, class T, int SPLIT>
__device__ __forceinline__ void few_sum(const FewArgs& a, uint32_t part, int rank, int wt,
                                        int64_t t0) {
    constexpr bool GATED = few_gated(MODE);
    constexpr int kBatch = 8 / SPLIT;
    constexpr int kSteps = GATED ? 1 : 2;  // pieces of 64 output columns
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int step = SPLIT * (kFewThreads / 32);
    const int items = int(min(int64_t(a.nt), a.tokens - t0)) * kSteps;  // (token, piece)
    T* const out = static_cast<T*>(a.out);
    uint32_t at[SPLIT];
#pragma unroll
    for (int k = 0; k < SPLIT; ++k) at[k] = mapa(part, k) + uint32_t(lane) * 8u;
    for (int i0 = rank + SPLIT * warp; i0 < items; i0 += kBatch * step) {
        float2 v[kBatch][SPLIT], u[kBatch][SPLIT];
        KeptPair<T> kept[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = i0 + j * step;
            if (i < items) {
                if constexpr (MODE == kFewBackward)
                    kept[j].load(a, t0 + i / kSteps, wt * 128 + 64 * (i % kSteps) + 2 * lane);
                const uint32_t off = uint32_t((i / kSteps) * 128 + 64 * (i % kSteps)) * 4u;
#pragma unroll
                for (int k = 0; k < SPLIT; ++k) {
                    v[j][k] = ld_cluster2(at[k] + off);
                    if (GATED) u[j][k] = ld_cluster2(at[k] + off + 256u);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = i0 + j * step;
            const int r = wt * (64 * kSteps) + 64 * (i % kSteps) + 2 * lane;
            if (i < items && r < a.rows) {  // an even number: both columns exist
                float2 s = v[j][0];
#pragma unroll
                for (int k = 1; k < SPLIT; ++k) {
                    s.x += v[j][k].x;
                    s.y += v[j][k].y;
                }
                if (GATED) {
                    float2 c = u[j][0];
#pragma unroll
                    for (int k = 1; k < SPLIT; ++k) {
                        c.x += u[j][k].x;
                        c.y += u[j][k].y;
                    }
                    s.x = s.x * sigmoid_fast(s.x) * c.x;
                    s.y = s.y * sigmoid_fast(s.y) * c.y;
                }
                T* const o = out + (t0 + i / kSteps) * a.pitch + r;
                if constexpr (MODE == kFewBackward) {
                    float2 ka, kc, da, dc, h;
                    kept[j].get(a, ka, kc);
                    gated_backward(s.x, ka.x, kc.x, da.x, dc.x, h.x);
                    gated_backward(s.y, ka.y, kc.y, da.y, dc.y, h.y);
                    s = da;
                    *reinterpret_cast<uint32_t*>(o + a.rows) = pack2t(T(), dc.x, dc.y);
                    *reinterpret_cast<uint32_t*>(static_cast<T*>(a.h) +
                                                 (t0 + i / kSteps) * a.rows + r) =
                        pack2t(T(), h.x, h.y);
                }
                *reinterpret_cast<uint32_t*>(o) = pack2t(T(), s.x, s.y);
            }
        }
    }
}

// The same for kFewKept: a warp takes the 128 features of a token, four a
// lane, from the two CTAs that have them (even and odd ranks), and keeps a
// and c as the pairs' epilogue does.
template <class T, int SPLIT>
__device__ __forceinline__ void few_keep(const FewArgs& a, uint32_t part, int rank, int tile,
                                         int64_t t0) {
    constexpr int kBatch = 4 / SPLIT;
    constexpr int step = 2 * SPLIT * (kFewThreads / 32);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int items = int(min(int64_t(a.nt), a.tokens - t0));
    const int f = tile * kTile + 4 * lane;
    const bool have = f < a.rows;  // a multiple of 8: four features exist together
    const int64_t wide = (a.rows + kTile - 1) / kTile * kTile;
    T* const out = static_cast<T*>(a.out);
    uint32_t at[SPLIT];
#pragma unroll
    for (int k = 0; k < SPLIT; ++k)
        at[k] = mapa(part, 2 * k + (lane >> 4)) + uint32_t(lane & 15) * 16u;
    for (int i0 = rank + 2 * SPLIT * warp; i0 < items; i0 += kBatch * step) {
        float4 v[kBatch][SPLIT], u[kBatch][SPLIT];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = i0 + j * step;
            if (i < items) {
#pragma unroll
                for (int k = 0; k < SPLIT; ++k) {
                    v[j][k] = ld_cluster4(at[k] + uint32_t(i) * 512u);
                    u[j][k] = ld_cluster4(at[k] + uint32_t(i) * 512u + 256u);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = i0 + j * step;
            if (i >= items) break;
            float s[4] = {v[j][0].x, v[j][0].y, v[j][0].z, v[j][0].w};
            float c[4] = {u[j][0].x, u[j][0].y, u[j][0].z, u[j][0].w};
#pragma unroll
            for (int k = 1; k < SPLIT; ++k) {
                s[0] += v[j][k].x, s[1] += v[j][k].y, s[2] += v[j][k].z, s[3] += v[j][k].w;
                c[0] += u[j][k].x, c[1] += u[j][k].y, c[2] += u[j][k].z, c[3] += u[j][k].w;
            }
            const int64_t t = t0 + i;
            if (a.kept == kKept8) {
                float ma = 0.0f, mc = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // columns past the last feature (rows of W3 for a) are kept as zeros
                    if (!have) s[e] = c[e] = 0.0f;
                    ma = fmaxf(ma, fabsf(s[e]));
                    mc = fmaxf(mc, fabsf(c[e]));
                }
                // as integers, whose order is that of values that are not negative
                ma = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(ma)));
                mc = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mc)));
                float sa, sc, ia, ic;
                kept_scale(ma, sa, ia);
                kept_scale(mc, sc, ic);
                uint8_t* const q = static_cast<uint8_t*>(a.ac) + t * 2 * wide + f;
                *reinterpret_cast<uint32_t*>(q) = codes4(s, ia);
                *reinterpret_cast<uint32_t*>(q + wide) = codes4(c, ic);
                if (lane == 0) {
                    a.ac_scales[int64_t(tile) * a.tokens + t] = sa;
                    a.ac_scales[(wide / kTile + tile) * a.tokens + t] = sc;
                }
            } else if (have) {
                T* const q = static_cast<T*>(a.ac) + t * 2 * a.rows + f;
                *reinterpret_cast<uint2*>(q) =
                    make_uint2(pack2t(T(), s[0], s[1]), pack2t(T(), s[2], s[3]));
                *reinterpret_cast<uint2*>(q + a.rows) =
                    make_uint2(pack2t(T(), c[0], c[1]), pack2t(T(), c[2], c[3]));
            }
            if (have) {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[e] = s[e] * sigmoid_fast(s[e]) * c[e];
                *reinterpret_cast<uint2*>(out + t * a.rows + f) =
                    make_uint2(pack2t(T(), s[0], s[1]), pack2t(T(), s[2], s[3]));
            }
        }
    }
}

template <int MODE, class T>
__global__ void __launch_bounds__(kFewThreads, 1) few_kernel(const __grid_constant__ FewArgs a) {
    constexpr bool GATED = few_gated(MODE), MN = few_turned(MODE), KEPT = MODE == kFewKept;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    FewShared* ss = reinterpret_cast<FewShared*>(smem + a.ring);
    const int warp = int(uniform(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    // the cluster is the x row of the grid
    const int rank = blockIdx.x, split = KEPT ? gridDim.x / 2 : gridDim.x;
    const int kr = KEPT ? rank / 2 : rank;
    const int wt = KEPT ? 2 * blockIdx.y + (rank & 1) : blockIdx.y;
    const int64_t t0 = int64_t(blockIdx.z) * a.nt;
    // this CTA's part of K
    const int kb0 = int(int64_t(a.nkb) * kr / split);
    const int n = int(int64_t(a.nkb) * (kr + 1) / split) - kb0;
    const uint32_t cols = a.nt <= 32 ? 32 : a.nt <= 64 ? 64 : a.nt <= 128 ? 128 : 256;
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(smem_u32(&ss->full[s]), 1);
            mbar_init(smem_u32(&ss->empty[s]), 1);
        }
        mbar_init(smem_u32(&ss->done), 1);
        ss->abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc(smem_u32(&ss->tmem_base), cols);
    if (warp == 2 && lane == 0) {
        prefetch_map(&a.w);
        prefetch_map(&a.x);
    }
    fence_before();
    __syncthreads();
    fence_after();
    launch_dependents();
    const uint32_t tmem = uniform(ss->tmem_base);
    const int stage_bytes = kOperandBytes + a.nt * 128;
    bool ok = true;
    int loaded = 0;  // steps that warp 0 has loaded
    if (warp == 0) {
        const bool lead = elect_one();
        const int w0 = wt * (GATED ? 64 : 128);
        auto load_w = [&](int i, int s) {
            if (i == 0 && a.fault == kFaultFfnProducer) return;
            const int k0 = (kb0 + i) * kTileK;
            const uint32_t bar = smem_u32(&ss->full[s]);
            const uint32_t dst = smem_u32(smem) + s * stage_bytes;
            mbar_arrive_expect_tx(bar, uint32_t(stage_bytes));
            if (MN) {
                tma_load_2d(dst, &a.w, bar, w0, k0);
                tma_load_2d(dst + kPieceBytes, &a.w, bar, w0 + 64, k0);
            } else {
                tma_load_2d(dst, &a.w, bar, k0, w0);
                if (GATED) tma_load_2d(dst + kOperandBytes / 2, &a.w, bar, k0, a.w3 + w0);
            }
        };
        auto load_x = [&](int i, int s) {
            if (i == 0 && a.fault == kFaultFfnProducer) return;
            tma_load_2d(smem_u32(smem) + s * stage_bytes + kOperandBytes, &a.x,
                        smem_u32(&ss->full[s]), (kb0 + i) * kTileK, int(t0));
        };
        // the first stages: weights before the wait, tokens after it
        const int first = min(n, a.stages);
        if (lead)
            for (int i = 0; i < first; ++i) load_w(i, i);
        if (a.wait_first) wait_dependencies();
        if (lead)
            for (int i = 0; i < first; ++i) load_x(i, i);
        __syncwarp();
        int i = first, s = 0;
        uint32_t par = 0;
        for (; i < n; ++i) {
            ok = mbar_wait(smem_u32(&ss->empty[s]), par, &ss->abort_flag, a.dev_status,
                           a.wait_limit_ns);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            if (lead) {
                load_w(i, s);
                load_x(i, s);
            }
            __syncwarp();
            if (++s == a.stages) {
                s = 0;
                par ^= 1u;
            }
        }
        loaded = i;
    } else if (warp == 1) {
        const bool lead = elect_one();
        // (the limit of its waits does not run while the kernel before this one does)
        if (a.wait_first) wait_dependencies();
        const uint32_t idesc = idesc_f16(std::is_same<T, bf16_t>::value, MN, 0, 128, a.nt);
        constexpr uint32_t w_step = MN ? 2048 / 16 : 32 / 16;  // as in the pairs' issuer
        const uint64_t desc0 = sw128_desc16(smem_u32(smem), kPieceBytes);
        int s = 0;
        uint32_t par = 0;
        for (int i = 0; i < n; ++i) {
            ok = mbar_wait(smem_u32(&ss->full[s]), par, &ss->abort_flag, a.dev_status,
                           a.wait_limit_ns);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            fence_after();
            const uint64_t ad = desc0 + uint32_t(s * (stage_bytes / 16));
            const uint64_t bd = ad + kOperandBytes / 16;
            if (lead) {
#pragma unroll
                for (int kk = 0; kk < kTileK / 16; ++kk)
                    mma_f16(tmem, ad + w_step * kk, bd + 2 * kk, idesc, (i | kk) ? 1u : 0u);
                commit(smem_u32(&ss->empty[s]));
            }
            __syncwarp();
            if (++s == a.stages) {
                s = 0;
                par ^= 1u;
            }
        }
        if (lead) {
            commit(smem_u32(&ss->done));
            mbar_quiesce(smem_u32(&ss->done), 0, nullptr, quiesce_ns(a.wait_limit_ns));
        }
    }
    __syncwarp();
    // the products are done (warp 1 has waited for them), or given up
    const bool bad = __syncthreads_or(!ok || *reinterpret_cast<volatile int*>(&ss->abort_flag));
    fence_after();
    // given up, whoever's wait ran out: loads may be in flight into the stages,
    // over which no sums are laid then
    if (bad && warp == 0) {
        if (lane == 0)
            ring_quiesce(ss->full, uint32_t(a.stages), uint32_t(loaded), a.wait_limit_ns);
        __syncwarp();
    }
    float* part = reinterpret_cast<float*>(smem);  // [nt][128]
    if (warp >= 2 && !bad) {
        const int q = warp & 3;  // the quarter of the lanes it may read
        for (int c = warp < 6 ? 0 : 16; c < a.nt; c += 32) {
            uint32_t v[16];
            if (n > 0) {
                tmem_ld16(tmem + (uint32_t(q * 32) << 16) + c, v);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = 0u;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) part[(c + i) * 128 + q * 32 + lane] = __uint_as_float(v[i]);
        }
        fence_before();
    }
    cluster_sync();  // every CTA's partial sums are in place
    if (!bad) {
        if constexpr (KEPT) {
            if (split == 1) few_keep<T, 1>(a, smem_u32(part), rank, blockIdx.y, t0);
            else if (split == 2) few_keep<T, 2>(a, smem_u32(part), rank, blockIdx.y, t0);
            else few_keep<T, 4>(a, smem_u32(part), rank, blockIdx.y, t0);
        } else {
            if (split == 1) few_sum<MODE, T, 1>(a, smem_u32(part), rank, wt, t0);
            else if (split == 2) few_sum<MODE, T, 2>(a, smem_u32(part), rank, wt, t0);
            else if (split == 4) few_sum<MODE, T, 4>(a, smem_u32(part), rank, wt, t0);
            else few_sum<MODE, T, 8>(a, smem_u32(part), rank, wt, t0);
        }
    }
    cluster_sync();  // nobody's partial sums are read any more
    if (warp == 1) {
        fence_after();
        tmem_free(tmem, cols);
    }
}

// ================================================== one to four tokens
// Matrix-vector products on the CUDA cores: reading the weights once is all
// the work there is, and plain 16-byte loads of whole rows, many in flight in
// every warp, start and end sooner than a pipeline of tiles.  A warp takes a
// part of one output's K (GATED: of the feature's rows of W1 and of W3): 256
// elements a step, kVecSteps steps' weights in flight; tokens come through L1.
// Four warps a CTA; `parts` warps share an output and meet in shared memory.
constexpr int kVecWarps = 4;
constexpr int kVecSteps = 4;
constexpr int kVecTokens = 4;

template <class T>
__device__ __forceinline__ uint4 ld_plain(const T* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

template <bool GATED, int TOK, class T>
__global__ void __launch_bounds__(kVecWarps * 32)
    vec_kernel(const T* __restrict__ w, const T* x, T* __restrict__ out, int tokens, int rows,
               int K, int parts, int wait_first) {
    constexpr int R = GATED ? 2 : 1;
    __shared__ float part[kVecWarps][R * TOK];
    launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.x * (kVecWarps / parts) + warp / parts;
    const bool have = row < rows;
    const int steps = (K + 255) / 256;
    const int s0 = steps * (warp % parts) / parts, s1 = steps * (warp % parts + 1) / parts;
    const T* wr[R];
#pragma unroll
    for (int r = 0; r < R; ++r) wr[r] = w + (int64_t(have ? row : 0) + int64_t(r) * rows) * K;
    float acc[R][TOK];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < TOK; ++t) acc[r][t] = 0.0f;
    for (int b = s0; b < s1; b += kVecSteps) {
        uint4 v[R][kVecSteps];
#pragma unroll
        for (int i = 0; i < kVecSteps; ++i) {
            const int k = (b + i) * 256 + lane * 8;
#pragma unroll
            for (int r = 0; r < R; ++r)
                v[r][i] = b + i < s1 && k < K && have
                              ? __ldcs(reinterpret_cast<const uint4*>(wr[r] + k))
                              : make_uint4(0u, 0u, 0u, 0u);
        }
        // the first weights are on their way before the values they wait for
        if (wait_first && b == s0) wait_dependencies();
#pragma unroll
        for (int i = 0; i < kVecSteps; ++i) {
            const int k = (b + i) * 256 + lane * 8;
            if (b + i < s1 && k < K) {
                float wf[R][8];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    Raw<T, 8> raw;
                    raw.a = v[r][i];
                    raw_floats(raw, wf[r]);
                }
#pragma unroll
                for (int t = 0; t < TOK; ++t) {
                    if (TOK == 1 || t < tokens) {
                        Raw<T, 8> raw;
                        raw.a = ld_plain(x + int64_t(t) * K + k);
                        float xf[8];
                        raw_floats(raw, xf);
#pragma unroll
                        for (int r = 0; r < R; ++r)
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                acc[r][t] = fmaf(wf[r][e], xf[e], acc[r][t]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < TOK; ++t) {
            float a = acc[r][t];
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
            if (lane == 0) part[warp][r * TOK + t] = a;
        }
    __syncthreads();
    if (have && warp % parts == 0 && lane < TOK && lane < tokens) {
        float a = 0.0f, c = 0.0f;
        for (int p = 0; p < parts; ++p) {
            a += part[warp + p][lane];
            if (GATED) c += part[warp + p][TOK * (R - 1) + lane];
        }
        if (GATED) a = a * sigmoid_fast(a) * c;
        elem_store(out + int64_t(lane) * rows + row, a);
    }
}

// -------------------------------------------------------------------- host
// CTA pairs the device holds at once (cached per device).
template <int EPI, int KEPT, class T>
int pair_units(cudaLaunchConfig_t& cfg) {
    static int cache[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (cudaFuncSetAttribute(ffn_kernel<EPI, KEPT, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(Cfg<EPI>::kSmem)) != cudaSuccess)
        return 0;
    if (cache[dev] == 0) {
        int n = 0;
        cfg.gridDim = dim3(unsigned(2 * (sm_count() / 2)), 1, 1);
        if (cudaOccupancyMaxActiveClusters(&n, ffn_kernel<EPI, KEPT, T>, &cfg) != cudaSuccess)
            return 0;
        cache[dev] = std::min(n, sm_count() / 2);
    }
    return cache[dev];
}

template <int EPI, int KEPT, class T>
int launch(Args& a, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = Cfg<EPI>::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int units = pair_units<EPI, KEPT, T>(cfg);
    if (units < 1) return cuda_failed();
    if (a.wait_first) cfg.numAttrs = 2;
    cfg.gridDim = dim3(unsigned(2 * std::min(units, a.tiles)), 1, 1);
    if (cudaLaunchKernelEx(&cfg, ffn_kernel<EPI, KEPT, T>, a) != cudaSuccess) return cuda_failed();
    return check_launch();
}

struct Maker {
    CUtensorMapDataType type;
    bool ok = true;
    // operand: K-major box of `rows` rows x 64 K, or MN-major box of 64 K
    // rows x 64 elements
    void operand(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int box_rows) {
        ok = ok && make_map_2d(m, type, base, uint64_t(rows), uint64_t(cols),
                               uint64_t(cols) * 2, uint32_t(box_rows), 64,
                               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
    }
    // output: boxes of 32 rows x 32 columns of a [rows, cols] part of rows
    // `pitch` elements long
    void output(CUtensorMap* m, void* base, int64_t rows, int64_t cols, int64_t pitch) {
        ok = ok && make_map_2d(m, type, base, uint64_t(rows), uint64_t(cols),
                               uint64_t(pitch) * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B,
                               CU_TENSOR_MAP_L2_PROMOTION_NONE);
    }
};

// The columns of a launch's pair tiles, and about how long it takes, in SM
// clocks.  A stage of 64 K elements takes the MMA 2 clocks a column, and 100
// more; a column of the epilogue costs `epilogue` clocks after the last tile,
// and under the next tile's products no tile of kPlain takes less than 1200 and
// 11 a column (the weight gradients of 16 tokens of d = 7168, inter = 2048: 24 us
// in columns of 256, 29 of 128, 40 of 64); starting and ending take 5500; and
// no launch ends before its longest tile.  So
// few tiles are cut narrow (256 tokens, d = 512, inter = 256: dy W2 14 us in one
// tile of 256 columns, 9 us in four of 64), and many take the width whose
// rounds over the pairs waste least (4096 x 7168 on 74 pairs: 7 rounds of 256
// columns, or 7 of 224: 85 and 80 us).  An MN-major B comes in pieces of 64
// columns for each half tile: 256 or 128 there, 64 with half of each piece
// unused (13 tiles of 160 instead of 8 of 256: 110 us for 95).
struct PairPlan {
    int nt = 0;
    int64_t clocks = INT64_MAX;
};
struct Extent {
    int64_t m, n;
    int nkb;
};
constexpr int64_t kLaunchClocks = 5500;
constexpr int kPlainClocks = 8, kGatedClocks = 16, kBackwardClocks = 66;
PairPlan pair_plan(const Extent* e, int count, int epilogue, std::initializer_list<int> widths) {
    const int pairs = std::max(1, sm_count() / 2);
    PairPlan best;
    for (int nt : widths) {
        int64_t tiles = 0, main = 0, longest = 0;
        for (int i = 0; i < count; ++i) {
            const int64_t t = (e[i].m + kTileM - 1) / kTileM * ((e[i].n + nt - 1) / nt);
            tiles += t;
            main += t * e[i].nkb * (2 * nt + 100);
            if (t > 0) longest = std::max<int64_t>(longest, e[i].nkb * (2 * nt + 100));
        }
        if (tiles == 0) return PairPlan{256, 0};
        main /= tiles;  // of an average tile
        const int64_t last = int64_t(epilogue) * nt;
        const int64_t least = epilogue == kPlainClocks ? 1200 + 11 * nt : last;
        const int64_t more = (tiles + pairs - 1) / pairs - 1;  // rounds over the pairs after the first
        const int64_t clocks =
            kLaunchClocks + std::max(longest, main + more * std::max(main, least)) + last;
        if (clocks < best.clocks) {
            best.nt = nt;
            best.clocks = clocks;
        }
    }
    return best;
}

// out [m, n] = A B^T over k: A is [m, k] in memory, or [k, m] (a_mn); B is
// [n, k], or [k, n] (b_mn).
void product(Args& a, Maker& mk, const void* A, bool a_mn, const void* B, bool b_mn, void* out,
             int64_t m, int64_t n, int64_t k, int nt) {
    Problem& p = a.p[a.n_problems++];
    p.m = int(m);
    p.n = int(n);
    p.nkb = int((k + kTileK - 1) / kTileK);
    p.nt = nt;
    p.tiles_m = int((m + kTileM - 1) / kTileM);
    p.tiles_n = int((n + nt - 1) / nt);
    p.first = a.tiles;
    p.a_mn = a_mn;
    p.b_mn = b_mn;
    a.tiles += p.tiles_m * p.tiles_n;
    if (a_mn) mk.operand(&p.a, A, k, m, 64);
    else mk.operand(&p.a, A, m, k, 128);
    if (b_mn) mk.operand(&p.b, B, k, n, 64);
    else mk.operand(&p.b, B, n, k, nt / 2);
    mk.output(&p.out, out, m, n, n);
}

Args make_args(int64_t T, int inter, int* dev_status) {
    Args a = {};
    a.rows = T;
    a.inter = inter;
    a.dev_status = dev_status;
    a.wait_limit_ns = wait_limit_ns();
    a.fault = fault_injection();
    return a;
}

// How a product with few tokens is laid out, and about how long it takes, in
// SM clocks fitted to 12 sizes from 16 to 1024 tokens, d and inter from 512 to
// 7168 and 256 to 2048: for 64 K elements 3 clocks a token (the MMA's 2, and
// the stage's bytes), 128 at least; starting, filling the pipeline, adding up
// and writing, 7000 and 30 a token.
struct FewPlan {
    int tiles_t, tiles_w, nt, split, ring;
    int64_t clocks;
};
FewPlan few_tiles(int mode, int64_t T, int tiles_t, int rows, int nkb) {
    const int rows_per_tile = few_gated(mode) ? 64 : 128;
    const int max_split = mode == kFewKept ? kFewMaxSplit / 2 : kFewMaxSplit;
    FewPlan p;
    p.tiles_t = tiles_t;
    p.nt = int(((T + p.tiles_t - 1) / p.tiles_t + 15) / 16 * 16);
    p.tiles_w = (rows + rows_per_tile - 1) / rows_per_tile;
    if (mode == kFewKept) p.tiles_w += p.tiles_w & 1;
    const int64_t tiles = int64_t(p.tiles_t) * p.tiles_w;
    const int sms = sm_count();
    // Up to 64 tokens two CTAs share an SM, so that one fetches while the
    // other adds up, and the next product's start under this one: K is split
    // until there are more CTAs than SMs (one token of d = 7168, inter = 2048:
    // 22.9 us against 28.7 us with one CTA an SM).  Wider stages leave room
    // for one: split until three quarters of the SMs have a CTA, and into
    // clusters of eight only up to there (500 tokens, dy W2 of d = 2048, inter =
    // 512: 16 such clusters do not find room at once and take 14.9 us, 32 with
    // half an SM a CTA 9.6).
    const bool two = p.nt <= kFewShared;
    p.ring = two ? kFewRing2 : kFewRing1;
    p.split = 1;
    const int pair = mode == kFewKept ? 2 : 1;
    auto room = [&](int split) {
        return two || pair * split < 8 || tiles * split * 4 <= 3 * int64_t(sms);
    };
    while (p.split < max_split && tiles * p.split * 4 < int64_t(sms) * (two ? 4 : 3) &&
           nkb >= 8 * p.split && room(2 * p.split))
        p.split *= 2;
    // Two on an SM take turns at its operands, and only a quarter longer before
    // and after them (64 tokens, d = 7168, inter = 2048 forward: 25.9 us, h W2^T
    // in pairs 28.3; 256 tokens, d = 4096, inter = 1024: 20.7 us in tiles of 64
    // tokens, two an SM, and 19.4 in tiles of 128).
    const int64_t ctas = tiles * p.split, at_once = int64_t(sms) * (two ? 2 : 1);
    const int64_t k = (nkb + p.split - 1) / p.split * std::max(3 * p.nt, 128);
    const int64_t rest = 7000 + 30 * p.nt;
    p.clocks = (ctas + at_once - 1) / at_once *
               (two && ctas > sms ? 2 * k + rest * 5 / 4 : k + rest);
    return p;
}
// As few tiles of tokens as there can be, or two, four or eight times as many,
// whose sums are sooner added up.
FewPlan few_plan(int mode, int64_t T, int rows, int nkb) {
    const int least = int((T + kFewMaxTokens - 1) / kFewMaxTokens);
    FewPlan best = few_tiles(mode, T, least, rows, nkb);
    for (int k = 2; k <= 8 && T >= 32 * int64_t(k) * least; k *= 2) {
        const FewPlan p = few_tiles(mode, T, k * least, rows, nkb);
        if (p.clocks < best.clocks) best = p;
    }
    return best;
}
// Whether a plan beats pairs: only where tiles of 256 x 256 leave pairs idle,
// and then by the two estimates.  (Forward that keeps a and c, and backward: 48
// tokens, d = 1032, inter = 328 24.8 us, all in pairs 31.6; 300 tokens, d = 4104,
// inter = 136 41 and 75 us; 16 tokens, d = 7168, inter = 2048 87 and 118 us.)
bool few_better(const FewPlan& p, int64_t m, int64_t n, const PairPlan& pair) {
    return (m + kTileM - 1) / kTileM * ((n + 255) / 256) < sm_count() / 2 &&
           p.clocks < pair.clocks;
}

template <bool GATED, int TOK, class T>
int launch_vec_tok(const void* w, const void* x, void* out, int tokens, int rows, int K, bool after,
                   cudaStream_t st) {
    // Warps per output: as many as leave every warp one batch of steps, so
    // that there are enough CTAs to even out over the SMs.
    const int steps = (K + 255) / 256;
    const int parts = steps > 2 * kVecSteps ? 4 : steps > kVecSteps ? 2 : 1;
    const int per = kVecWarps / parts;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((rows + per - 1) / per), 1, 1);
    cfg.blockDim = dim3(kVecWarps * 32, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = after ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, vec_kernel<GATED, TOK, T>, static_cast<const T*>(w),
                           static_cast<const T*>(x), static_cast<T*>(out), tokens, rows, K, parts,
                           int(after)) != cudaSuccess)
        return cuda_failed();
    return check_launch();
}
template <bool GATED, class T>
int launch_vec(const void* w, const void* x, void* out, int tokens, int rows, int K, bool after,
               cudaStream_t st) {
    return tokens == 1   ? launch_vec_tok<GATED, 1, T>(w, x, out, tokens, rows, K, after, st)
           : tokens == 2 ? launch_vec_tok<GATED, 2, T>(w, x, out, tokens, rows, K, after, st)
                         : launch_vec_tok<GATED, 4, T>(w, x, out, tokens, rows, K, after, st);
}

// kept, ac, ac_scales, h: kFewKept and kFewBackward.
struct FewKept {
    void* ac;
    float* ac_scales;
    int kept;
    void* h;
};
template <int MODE, class T>
int launch_few(Maker& mk, const FewPlan& p, const void* w, const void* x, void* out, int64_t tokens,
               int rows, int K, const FewKept& kept, int* dev_status, bool after,
               cudaStream_t st) {
    FewArgs a = {};
    if (few_turned(MODE)) mk.operand(&a.w, w, K, rows, 64);
    else mk.operand(&a.w, w, few_gated(MODE) ? 2 * int64_t(rows) : rows, K, few_gated(MODE) ? 64 : 128);
    mk.operand(&a.x, x, tokens, K, p.nt);
    if (!mk.ok) return MOE_ERR_CUDA;
    a.out = out;
    a.h = kept.h;
    a.ac = kept.ac;
    a.ac_scales = kept.ac_scales;
    a.kept = kept.kept;
    a.rows = rows;
    a.pitch = MODE == kFewBackward ? 2 * rows : rows;
    a.w3 = rows;
    a.tokens = tokens;
    a.nt = p.nt;
    a.nkb = (K + kTileK - 1) / kTileK;
    a.ring = p.ring;
    a.stages = std::min(kFewMaxStages, p.ring / (kOperandBytes + p.nt * 128));
    a.wait_first = after;
    a.dev_status = dev_status;
    a.wait_limit_ns = wait_limit_ns();
    a.fault = fault_injection();
    // (leave for either ring, whichever this call takes: the limit is the
    // device's, and another thread may be between its own and its launch)
    if (cudaFuncSetAttribute(few_kernel<MODE, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(few_smem(kFewRing1))) != cudaSuccess)
        return cuda_failed();
    const int pair = MODE == kFewKept ? 2 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(pair * p.split), unsigned(p.tiles_w / pair), unsigned(p.tiles_t));
    cfg.blockDim = dim3(kFewThreads, 1, 1);
    cfg.dynamicSmemBytes = few_smem(p.ring);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cfg.gridDim.x;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = after ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, few_kernel<MODE, T>, a) != cudaSuccess) return cuda_failed();
    return check_launch();
}

template <class T>
int forward(Maker mk, const void* x, const void* w13, const void* w2, int64_t rows, int d, int I,
            void* h, void* y, void* ac, int kept, float* ac_scales, int* dev_status,
            cudaStream_t st) {
    int rc;
    // One token, or a few with few weights (a token's multiplications cost as
    // much time as its weights' bytes: 2 and 4 tokens of 88 MB of weights take
    // 25 and 36 us as vectors and 23 us as tiles, of 0.8 MB 3.4 and 9.3 us).
    if (kept == kKeptNone && (rows == 1 || (rows <= kVecTokens &&
                                            rows * 6 * int64_t(d) * I <= 100000000))) {
        rc = launch_vec<true, T>(w13, x, h, int(rows), I, d, false, st);
        return rc != MOE_OK ? rc : launch_vec<false, T>(w2, h, y, int(rows), d, I, true, st);
    }
    const int kd = (d + kTileK - 1) / kTileK, ki = (I + kTileK - 1) / kTileK;
    // few tokens: whichever way takes fewer clocks.  (One token, d = 7168,
    // inter = 2048: 70 us in pairs of CTAs.)  a and c are kept in 8 bits from
    // tiles that see 128 features together.
    const Extent ea = {rows, 2 * int64_t(I), kd}, eb = {rows, d, ki};
    const PairPlan pa = kept == kKept8 ? pair_plan(&ea, 1, kGatedClocks, {256})
                                       : pair_plan(&ea, 1, kGatedClocks, {256, 128});
    const PairPlan pb = pair_plan(&eb, 1, kPlainClocks, {256, 224, 192, 160, 128, 96, 64});
    const FewPlan fa = few_plan(kept == kKeptNone ? kFewGated : kFewKept, rows, I, kd);
    const FewPlan fb = few_plan(kFewPlain, rows, d, ki);
    const bool few_a = few_better(fa, rows, 2 * int64_t(I), pa);
    const bool few_b = few_better(fb, rows, d, pb);
    if (few_a) {
        rc = kept == kKeptNone
                 ? launch_few<kFewGated, T>(mk, fa, w13, x, h, rows, I, d, {}, dev_status, false, st)
                 : launch_few<kFewKept, T>(mk, fa, w13, x, h, rows, I, d, {ac, ac_scales, kept, nullptr},
                                           dev_status, false, st);
    } else {
        Args a = make_args(rows, I, dev_status);
        product(a, mk, x, false, w13, false, h, rows, 2 * int64_t(I), d, pa.nt);
        // the gated tile: nt / 2 features of W1 and of W3
        Problem& p = a.p[0];
        p.n = I;
        p.tiles_n = (I + pa.nt / 2 - 1) / (pa.nt / 2);
        a.tiles = p.tiles_m * p.tiles_n;
        mk.output(&p.out, h, rows, I, I);
        a.ac = ac;
        a.ac_scales = ac_scales;
        if (kept == kKept16) {
            mk.output(&a.o1, ac, rows, I, 2 * int64_t(I));
            mk.output(&a.o2, static_cast<uint16_t*>(ac) + I, rows, I, 2 * int64_t(I));
        }
        if (!mk.ok) return MOE_ERR_CUDA;
        rc = kept == kKept8    ? launch<kGated, kKept8, T>(a, st)
             : kept == kKept16 ? launch<kGated, kKept16, T>(a, st)
                               : launch<kGated, kKeptNone, T>(a, st);
    }
    if (rc != MOE_OK) return rc;
    // (laid out while the first product is on its way)
    if (few_b) return launch_few<kFewPlain, T>(mk, fb, w2, h, y, rows, d, I, {}, dev_status, true, st);
    Args b = make_args(rows, I, dev_status);
    product(b, mk, h, false, w2, false, y, rows, d, I, pb.nt);
    b.wait_first = 1;
    return mk.ok ? launch<kPlain, kKeptNone, T>(b, st) : MOE_ERR_CUDA;
}

template <class T>
int backward(Maker mk, const void* dy, const void* x, const void* w13, const void* w2, void* ac,
             int kept, float* ac_scales, int64_t rows, int d, int I, void* dac, void* h, void* dx,
             void* dw13, void* dw2, int* dev_status, cudaStream_t st) {
    const int kd = (d + kTileK - 1) / kTileK, kt = int((rows + kTileK - 1) / kTileK);
    const int k2 = (2 * I + kTileK - 1) / kTileK;
    // dy W2 and its element-wise step, and dx, with few tokens: as in the
    // forward pass.  (dx costs a launch of its own then; the choice does not
    // depend on what else is wanted, so neither do its bits.)
    const Extent ea = {rows, I, kd}, ex = {rows, d, k2};
    const PairPlan pa = pair_plan(&ea, 1, kBackwardClocks, {256, 128, 64});
    const PairPlan px = pair_plan(&ex, 1, kPlainClocks, {256, 128, 64});
    const FewPlan fa = few_plan(kFewBackward, rows, I, kd);
    FewPlan fx = few_plan(kFewTurned, rows, d, k2);
    fx.clocks += kLaunchClocks;
    const bool few_x = dx && few_better(fx, rows, d, px);
    int rc;
    if (few_better(fa, rows, I, pa)) {
        rc = launch_few<kFewBackward, T>(mk, fa, w2, dy, dac, rows, I, d,
                                         {ac, ac_scales, kept, h}, dev_status, false, st);
    } else {
        Args a = make_args(rows, I, dev_status);
        a.ac = ac;
        a.ac_scales = ac_scales;
        product(a, mk, dy, false, w2, true, h, rows, I, d, pa.nt);
        mk.output(&a.p[0].out, dac, rows, I, 2 * int64_t(I));
        mk.output(&a.o1, static_cast<uint16_t*>(dac) + I, rows, I, 2 * int64_t(I));
        mk.output(&a.o2, h, rows, I, I);
        if (!mk.ok) return MOE_ERR_CUDA;
        rc = kept == kKept8 ? launch<kBackward, kKept8, T>(a, st)
                            : launch<kBackward, kKept16, T>(a, st);
    }
    if (rc == MOE_OK && few_x)
        rc = launch_few<kFewTurned, T>(mk, fx, w13, dac, dx, rows, d, 2 * I, {}, dev_status, true,
                                       st);
    if (rc != MOE_OK) return rc;
    Args b = make_args(rows, I, dev_status);
    const Extent eb[3] = {{dx && !few_x ? rows : 0, d, k2},
                          {dw13 ? 2 * int64_t(I) : 0, d, kt},
                          {dw2 ? d : 0, I, kt}};
    const int nt = pair_plan(eb, 3, kPlainClocks, {256, 128, 64}).nt;
    if (dx && !few_x) product(b, mk, dac, false, w13, true, dx, rows, d, 2 * int64_t(I), nt);
    if (dw13) product(b, mk, dac, true, x, true, dw13, 2 * int64_t(I), d, rows, nt);
    if (dw2) product(b, mk, dy, true, h, true, dw2, d, I, rows, nt);
    b.wait_first = 1;
    if (!mk.ok) return MOE_ERR_CUDA;
    return b.n_problems == 0 ? MOE_OK : launch<kPlain, kKeptNone, T>(b, st);
}

int check_sizes(int type, int64_t T, int d, int inter) {
    if (type != MOE_T_BF16 && type != MOE_T_F16) return MOE_ERR_ARG;
    if (T < 0 || T > (1 << 24) || d < 8 || d % 8 || inter < 8 || inter % 8 || d > (1 << 20) ||
        inter > (1 << 20))
        return MOE_ERR_SHAPE;
    // 2^30 output tiles of 256 x 128 are more than any of these sizes gives
    return MOE_OK;
}

Maker maker(int type) {
    return Maker{type == MOE_T_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT16};
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" MOE_API int moe_ffn_forward(const void* x, const void* w13, const void* w2, int type,
                                       int64_t T, int d, int inter, void* h, void* y, void* ac,
                                       int ac_type, float* ac_scales, int* dev_status,
                                       void* stream) {
    int rc = check_sizes(type, T, d, inter);
    if (rc != MOE_OK) return rc;
    if (ac && ac_type != MOE_T_CKPT && ac_type != type) return MOE_ERR_ARG;
    if (T == 0) return MOE_OK;
    if (!x || !w13 || !w2 || !h || !y) return MOE_ERR_NULL;
    const int kept = !ac ? kKeptNone : ac_type == MOE_T_CKPT ? kKept8 : kKept16;
    if (kept == kKept8 && !ac_scales) return MOE_ERR_NULL;
    if (!aligned16(x) || !aligned16(w13) || !aligned16(w2) || !aligned16(h) || !aligned16(y) ||
        !aligned16(ac))
        return MOE_ERR_ALIGN;
    if (!device_is_sm100()) return MOE_ERR_DEVICE;
    cudaStream_t st = as_stream(stream);
    return type == MOE_T_BF16
               ? forward<bf16_t>(maker(type), x, w13, w2, T, d, inter, h, y, ac, kept, ac_scales,
                                 dev_status, st)
               : forward<f16_t>(maker(type), x, w13, w2, T, d, inter, h, y, ac, kept, ac_scales,
                                dev_status, st);
}

extern "C" MOE_API int moe_ffn_backward(const void* dy, const void* x, const void* w13,
                                        const void* w2, const void* ac, int ac_type,
                                        const float* ac_scales, int type, int64_t T, int d,
                                        int inter, void* dac, void* h, void* dx, void* dw13,
                                        void* dw2, int* dev_status, void* stream) {
    int rc = check_sizes(type, T, d, inter);
    if (rc != MOE_OK) return rc;
    if (ac_type != MOE_T_CKPT && ac_type != type) return MOE_ERR_ARG;
    cudaStream_t st = as_stream(stream);
    if (T == 0) {
        // no tokens: the weights' gradients are empty sums
        const size_t n = size_t(d) * size_t(inter) * 2;
        if ((dw13 && cudaMemsetAsync(dw13, 0, 2 * n, st) != cudaSuccess) ||
            (dw2 && cudaMemsetAsync(dw2, 0, n, st) != cudaSuccess))
            return cuda_failed();
        return MOE_OK;
    }
    if (!dy || !w2 || !ac || !dac || !h || (dx && !w13) || (dw13 && !x)) return MOE_ERR_NULL;
    const int kept = ac_type == MOE_T_CKPT ? kKept8 : kKept16;
    if (kept == kKept8 && !ac_scales) return MOE_ERR_NULL;
    const void* all[] = {dy, x, w13, w2, ac, dac, h, dx, dw13, dw2};
    for (const void* p : all)
        if (!aligned16(p)) return MOE_ERR_ALIGN;
    if (!device_is_sm100()) return MOE_ERR_DEVICE;
    return type == MOE_T_BF16
               ? backward<bf16_t>(maker(type), dy, x, w13, w2, const_cast<void*>(ac), kept,
                                  const_cast<float*>(ac_scales), T, d, inter, dac, h, dx, dw13,
                                  dw2, dev_status, st)
               : backward<f16_t>(maker(type), dy, x, w13, w2, const_cast<void*>(ac), kept,
                                 const_cast<float*>(ac_scales), T, d, inter, dac, h, dx, dw13, dw2,
                                 dev_status, st);
}
