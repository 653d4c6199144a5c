// Kernels of the e4m3 operators with a scale for each block of 128: the
// quantiser and the matrix product.
#pragma once

#include "fp8_device.hpp"

namespace fp8dev {

constexpr int kScaleBlock = 128;  // columns (and weight rows) that share a scale

// ---------------------------------------------------------------------------
// quantiser
//
//   scale = max(amax / 448, 2^-126),   q = e4m3(x · (1/scale))
//
// The division and the reciprocal are IEEE fp32, so the values are the same
// whatever computes the formula; the product is rounded to fp32 and then to
// e4m3.  A block that holds an infinity or NaN gets that as its scale.
// ---------------------------------------------------------------------------

// Eight consecutive elements of a row, widened to fp32; those from `n` on
// read as zero and are not touched.
template <class D>
__device__ __forceinline__ void load8(const typename D::storage* p, int n, float (&v)[8]) {
    if (n >= 8) {
        if constexpr (D::bytes == 4) {
            const quad a = *reinterpret_cast<const quad_any*>(p);
            const quad b = *reinterpret_cast<const quad_any*>(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = gemvdev::f32_of(a[i]);
                v[4 + i] = gemvdev::f32_of(b[i]);
            }
        } else {
            const quad a = *reinterpret_cast<const quad_any*>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = widen(D{}, (uint16_t)(a[i] & 0xffffu));
                v[2 * i + 1] = widen(D{}, (uint16_t)(a[i] >> 16));
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? widen(D{}, p[i]) : 0.0f;
}

__device__ __forceinline__ void store8(uint8_t* p, int n, u32x2 w) {
    if (n >= 8) {
        *reinterpret_cast<u32x2_any*>(p) = w;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
}

__device__ __forceinline__ float scale_of(uint32_t amax_bits) {
    const float s = __builtin_bit_cast(float, amax_bits) / kE4m3Max;
    return s < kSmallestScale ? kSmallestScale : s;  // NaN stays
}

// One scale per row and 128 columns.  16 lanes hold a block, 8 elements
// each, so a wavefront takes 512 consecutive columns of a row, reads each
// element once and keeps it in registers until its block's maximum is known.
// Bound by memory: 4096 x 14336 bf16 33.3 us, 5.4 TB/s read and written (a large
// copy reaches 4.8); 16 x 4096 fp32 is one launch's latency, 2.5 us.
constexpr int kQuantWaves = 4;
template <class D>
__global__ __launch_bounds__(kQuantWaves * 64) void fp8_quantise_rows_kernel(
    const typename D::storage* X, int64_t ldx, uint8_t* Q, int64_t ldq, float* scale, int64_t lds,
    int64_t units, int units_per_row, int K) {
    const int64_t unit = (int64_t)blockIdx.x * kQuantWaves + (threadIdx.x >> 6);
    if (unit >= units) return;
    const int lane = threadIdx.x & 63;
    const int64_t row = unit / units_per_row;
    const int64_t col = (unit - row * units_per_row) * 512 + lane * 8;
    const int n = (int)(K - col);
    float v[8];
    load8<D>(X + row * ldx + col, n, v);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_u32(m, magnitude(v[i]));
    const float s = scale_of(row_max16(m));
    const float inv = 1.0f / s;
    u32x2 w;
    w[0] = to_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    w[1] = to_e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
    if (n > 0) {
        store8(Q + row * ldq + col, n, w);
        if ((lane & 15) == 0) scale[row * lds + col / kScaleBlock] = s;
    }
}

// One scale per 128 rows and 128 columns: a workgroup holds the block in
// registers, 16 lanes a row, and reduces its maximum through LDS.  Bound by
// memory as well: 3045 x 3463 fp32 12.0 us, where the bytes take 11.1 at a large
// copy's rate.
constexpr int kTileWaves = 8;
template <class D>
__global__ __launch_bounds__(kTileWaves * 64) void fp8_quantise_tile_kernel(
    const typename D::storage* X, int64_t ldx, uint8_t* Q, int64_t ldq, float* scale, int64_t lds,
    int rows, int K) {
    constexpr int kPerLane = kScaleBlock / (kTileWaves * 4);
    __shared__ uint32_t part[kTileWaves];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int col = (int)blockIdx.x * kScaleBlock + (lane & 15) * 8;
    const int row0 = (int)blockIdx.y * kScaleBlock + wave * 4 + (lane >> 4);
    const int n = K - col;
    float v[kPerLane][8];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
        const int row = row0 + j * kTileWaves * 4;
        load8<D>(X + (int64_t)row * ldx + col, row < rows ? n : 0, v[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max_u32(m, magnitude(v[j][i]));
    }
    m = wave_max(m);
    if (lane == 0) part[wave] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kTileWaves; ++w) m = max_u32(m, part[w]);
    const float s = scale_of(m);
    const float inv = 1.0f / s;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
        const int row = row0 + j * kTileWaves * 4;
        u32x2 w;
        w[0] = to_e4m3x4(v[j][0] * inv, v[j][1] * inv, v[j][2] * inv, v[j][3] * inv);
        w[1] = to_e4m3x4(v[j][4] * inv, v[j][5] * inv, v[j][6] * inv, v[j][7] * inv);
        if (row < rows && n > 0) store8(Q + (int64_t)row * ldq + col, n, w);
    }
    if (threadIdx.x == 0) scale[(int64_t)blockIdx.y * lds + blockIdx.x] = s;
}

// ---------------------------------------------------------------------------
// product   Y[t,m] = Σ_b sx[t,b]·sw[m/128,b]·Σ_{k in block b} W[m,k]·X[t,k] + bias[m]
//
// A block's 128 products are taken by the matrix cores in one of two ways.
// Exactly: as 16×16×32 fp16 steps on exactly widened values; measured, the sum
// is then within 4e-8 of Σ|products|.  Or as one 16×16×128 e4m3 step, half the
// matrix-core cycles and no conversions.  The e4m3 steps (the 16×16×32 ones
// too) align each 8 products to the largest of them and cut what lies 2^-13
// below it: the sum is within 7·2^-13 of Σ|products| whatever they are, and
// measured within 2^-15 of it on random data (a relative error of 1.5e-5 of the
// results, where fp16's rounding is 2e-4 and bf16's 1.7e-3).  So they are taken
// for fp16 and bf16 results of many tokens, where the matrix cores are the
// bound, and never for fp32 results.
//
// A is 16 rows of W, B 16 tokens of X.  The order of the products is free as
// long as A and B agree, so lane l takes row (or token) l % 16 and the bytes
// 16·(l/16) .. +15 and 64 + 16·(l/16) .. +15 of the block: one load instruction
// then covers 64 consecutive bytes of each row.  The block's sum starts from
// zero; it is scaled and added in fp32.
// ---------------------------------------------------------------------------

// 8 e4m3 bytes as fp16, exactly.
__device__ __forceinline__ quad widen8(int lo, int hi) {
    return quad{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true))};
}

struct Wide {
    quad step[4];
};
__device__ __forceinline__ Wide widen32(i32x8 v) {
    Wide w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w.step[i] = widen8(v[2 * i], v[2 * i + 1]);
    return w;
}
__device__ __forceinline__ f32x4 mma_block(const Wide& a, const Wide& b) {
    f32x4 d{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i) d = gemvdev::mma_16x16x32(TF16{}, a.step[i], b.step[i], d);
    return d;
}

__device__ __forceinline__ i32x8 join(quad lo, quad hi) {
    i32x8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[i] = (int)lo[i];
        r[4 + i] = (int)hi[i];
    }
    return r;
}

// The lane's 32 bytes of a block that starts at column k of the row at p.
__device__ __forceinline__ i32x8 load_block(const uint8_t* p, int k, int group, int K) {
    const uint8_t* at = p + k + 16 * group;
    if (K - k >= kScaleBlock)
        return join(*reinterpret_cast<const quad_any*>(at),
                    *reinterpret_cast<const quad_any*>(at + 64));
    return join(load_end(p, (int64_t)k + 16 * group, K), load_end(p, (int64_t)k + 16 * group + 64, K));
}

// Four neighbouring results of a token, from row m on, at any alignment.
template <class O>
__device__ __forceinline__ void store_row4(void* Y, int64_t at, int m, int M, f32x4 v) {
    typename O::storage* y = static_cast<typename O::storage*>(Y) + at + m;
    if (m + 4 <= M) {
        struct __attribute__((packed, aligned(O::bytes))) Four {
            typename O::storage v[4];
        };
        *reinterpret_cast<Four*>(y) = Four{{narrow(O{}, v[0]), narrow(O{}, v[1]), narrow(O{}, v[2]), narrow(O{}, v[3])}};
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (m + e < M) y[e] = narrow(O{}, v[e]);
}

// Few tokens of few rows: 16 rows of W by 16 tokens to a workgroup; its
// wavefronts take the scale blocks in turn, U at a time with all their loads in
// flight, and add their sums in LDS, in a fixed order.  W is loaded through the
// caches: several token tiles read it again (past them 30 x 1024 x 11008 takes
// 14.6 us against 13.3, 4000 x 16 x 11008 17.4 against 13.0), and a single one
// loses nothing by it (1 x 4096 x 4096 6.2 and 5.8).  Bound by latency: of W
// from memory, 1 x 1024 x 4096 takes 5.1 us, of which its 4 MiB are 0.9; 16 x
// 4096 x 4096 7.8.
template <class O, int W, int U>
__global__ __launch_bounds__(W * 64) void fp8_few_kernel(
    const uint8_t* A, int64_t lda, const float* as, int64_t ldas, const uint8_t* X, int64_t ldx,
    const float* xs, int64_t ldxs, const float* bias, void* Y, int64_t ldy, int M, int K, int T, int) {
    __shared__ f32x4 part[W][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int r = lane & 15, group = lane >> 4;
    const int row0 = (int)blockIdx.x * 16, t0 = (int)blockIdx.y * 16;
    const int blocks = K / kScaleBlock + (K % kScaleBlock != 0);
    const int whole = K / kScaleBlock;  // blocks that have all their columns
    // rows and tokens past the end repeat the last one; their results are not stored
    const uint8_t* a = A + (int64_t)(row0 + r < M ? row0 + r : M - 1) * lda;
    const float* asr = as + (int64_t)(row0 / kScaleBlock) * ldas;
    const int64_t token = t0 + r < T ? t0 + r : T - 1;
    const uint8_t* x = X + token * ldx;
    const float* xsr = xs + token * ldxs;
    f32x4 acc{0.0f, 0.0f, 0.0f, 0.0f};
    const auto add = [&](i32x8 af, i32x8 xf, float by) {
        const f32x4 d = mma_block(widen32(af), widen32(xf));
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(d[e], by, acc[e]);
    };
    int b = wave;
    for (; b + (U - 1) * W < whole; b += U * W) {
        i32x8 af[U], xf[U];
        float s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = (int64_t)(b + u * W) * kScaleBlock + 16 * group;
            af[u] = join(*reinterpret_cast<const quad_any*>(a + k), *reinterpret_cast<const quad_any*>(a + k + 64));
            xf[u] = join(*reinterpret_cast<const quad_any*>(x + k), *reinterpret_cast<const quad_any*>(x + k + 64));
            s[u] = asr[b + u * W] * xsr[b + u * W];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) add(af[u], xf[u], s[u]);
    }
    for (; b < blocks; b += W)
        add(load_block(a, b * kScaleBlock, group, K), load_block(x, b * kScaleBlock, group, K), asr[b] * xsr[b]);
    part[wave][lane] = acc;
    __syncthreads();
    if (threadIdx.x >= 64) return;
    f32x4 v = part[0][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) v += part[w][lane];
    const int m = row0 + 4 * group;
    if (t0 + r >= T || m >= M) return;
    if (bias)
#pragma unroll
        for (int n = 0; n < 4; ++n) v[n] += bias[m + n < M ? m + n : M - 1];
    store_row4<O>(Y, (int64_t)(t0 + r) * ldy, m, M, v);
}

// ---------------------------------------------------------------------------
// product over many tokens: tiles staged in LDS
//
// A workgroup of eight wavefronts takes BM rows of W by BN tokens, a wavefront
// WM by WN of them, one scale block at a time.  The bytes go from memory to LDS
// without passing through registers, STAGES - 1 blocks ahead of the products.
//
// Two wavefronts share a SIMD, one of each half of the workgroup, and the
// halves work in opposite phases: while one reads its operands of a block from
// LDS, the other multiplies, and at the barrier they change over.  (With both
// in the same phase the LDS, the matrix cores and the vector ALUs, which scale
// each block's sum, waited for each other in turn.)
//
// DIRECT, for aligned rows of whole 16-byte pieces; anything else passes
// through registers, one block ahead: 2000 x 4096 x 4112 bf16 50 us, 2000 x 4096
// x 4100 86.
//
// 4096 x 14336 x 4096 bf16 takes 266 to 286 us from box to box (1.7 to 1.8
// PFLOP/s; the library's largest product of e4m3 without block scales reaches
// 2.6): bound by LDS, whose reads and writes of a step take about 1000 cycles by
// their bytes, its matrix-core work 860, and by scaling each block's sum on the
// vector ALUs.  The
// larger 256 x 128 tile in one workgroup a compute unit measured the same.
//
// LDS.  A stage holds the rows' 128 bytes one behind the other in eight
// 16-byte slots; slot s of row r holds piece s ^ (r % 8), so that the 8 lanes
// of a read that want the same piece of 8 neighbouring rows find it in 8
// different slots (a memory-to-LDS load writes its 64 lanes' pieces in lane
// order, so the swizzle is in the lanes' addresses).
// ---------------------------------------------------------------------------

// The wavefront's lanes' 16-byte pieces (or words) at base + offset, written
// to LDS from `lds` on in lane order (base and lds uniform).  The caller waits
// (wait_loads): written as instructions, because the compiler, which cannot
// tell the stages apart, would wait for all of them before it reads any.
// There is no register result.  m0, which takes the LDS address, is declared as
// written; the compiler warns that it keeps that register to itself and will not
// preserve it, which nothing here asks for.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_load16(const uint8_t* base, uint32_t offset, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(offset), "s"(base)
                 : "m0", "memory");
}
__device__ __forceinline__ void lds_load4(const float* base, uint32_t offset, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
                 :
                 : "s"(lds), "v"(offset), "s"(base)
                 : "m0", "memory");
}
#pragma clang diagnostic pop
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); }
// Nothing moves across a change of phase.
__device__ __forceinline__ void change_over() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ f32x4 mma_16x16x128(i32x8 a, i32x8 b) {
    const f32x4 zero{0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}

// An operand of a block as its matrix-core steps take it.
template <bool EXACT>
struct Operand;
template <>
struct Operand<true> {
    Wide v;
    __device__ __forceinline__ static Operand of(i32x8 x) { return Operand{widen32(x)}; }
};
template <>
struct Operand<false> {
    i32x8 v;
    __device__ __forceinline__ static Operand of(i32x8 x) { return Operand{x}; }
};
__device__ __forceinline__ f32x4 block_sum(const Operand<true>& a, const Operand<true>& b) {
    return mma_block(a.v, b.v);
}
__device__ __forceinline__ f32x4 block_sum(const Operand<false>& a, const Operand<false>& b) {
    return mma_16x16x128(a.v, b.v);
}

// The 16-byte piece at byte `piece` of block b of a row of K bytes, from any
// address; what lies behind the row reads as zero.
__device__ __forceinline__ quad piece_of(const uint8_t* row, int b, int piece, int K) {
    const int64_t at = (int64_t)b * kScaleBlock + piece;
    // (uniform)
    if (K - b * kScaleBlock >= kScaleBlock) return *reinterpret_cast<const quad_any*>(row + at);
    return load_end(row, at, K);
}

// A last block of fewer columns, in whole pieces, loaded straight into LDS: the
// lanes of the pieces behind the row load the block's first piece again, and X's
// copies are made zero as they are read.  (W's need not be: a NaN among them
// is also in its own place in that row, whose results it makes NaN there.)
__device__ __forceinline__ void blank_behind(i32x8& x, int group, int columns) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = 16 * group < columns ? x[i] : 0;
        x[4 + i] = 16 * (group + 4) < columns ? x[4 + i] : 0;
    }
}

template <int BM_, int BN_, int WM_, int WN_, int STAGES_, int GROUP_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, STAGES = STAGES_, GROUP = GROUP_;
    static constexpr int kWaves = BM / WM * (BN / WN);
    static constexpr int kRows = BM + BN;                      // rows of a stage
    static constexpr int kStageBytes = kRows * kScaleBlock;
    static constexpr int kLoads = kRows / 8 / kWaves;          // 1 KiB loads of a wavefront per stage
    static constexpr int kInFlight = (STAGES - 2) * kLoads;
    // Scales lie behind the stages, those of kSpan blocks at a time and twice:
    // the tokens', then the rows' (one for each 128), 8 lines to a load.
    static constexpr int kSpan = 8;
    static constexpr int kScaleLoads = BN / 8 + 1;
    // the same number for every wavefront: spare ones repeat the last
    static constexpr int kScaleEach = (kScaleLoads + kWaves - 1) / kWaves;
    static constexpr int kScaleBytes = kScaleLoads * 256;
    static constexpr int kLds = STAGES * kStageBytes + 2 * kScaleBytes;
    // wavefronts of a SIMD: two for each workgroup whose LDS fits a compute unit
    static constexpr int kOccupancy = 2 * (160 * 1024 / kLds) < 4 ? 2 * (160 * 1024 / kLds) : 4;
    static_assert(kWaves == 8 && kRows % (8 * kWaves) == 0 && BM <= 8 * kScaleBlock, "whole loads");
};

template <class O, class C, bool EXACT, bool DIRECT>
__global__ __launch_bounds__(C::kWaves * 64, DIRECT ? C::kOccupancy : 2) void fp8_tile_kernel(
    const uint8_t* A, int64_t lda, const float* as, int64_t ldas, const uint8_t* X, int64_t ldx,
    const float* xs, int64_t ldxs, const float* bias, void* Y, int64_t ldy, int M, int K, int T,
    int row_tiles) {
    constexpr int NM = C::WM / 16, NN = C::WN / 16;
    extern __shared__ __align__(16) uint8_t lds[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int r = lane & 15, g = lane >> 4;
    // the workgroups that share a chiplet's cache (every eighth) take
    // neighbouring tiles: GROUP row tiles by the tokens, one token tile after the other
    const int tiles = gridDim.x;
    const int per = tiles / 8, id = blockIdx.x;
    const int tile = id < per * 8 ? id % 8 * per + id / 8 : id;
    const int token_tiles = tiles / row_tiles;
    const int first_row = tile / (C::GROUP * token_tiles) * C::GROUP;
    const int in_group = tile - first_row * token_tiles;
    const int rows = row_tiles - first_row < C::GROUP ? row_tiles - first_row : C::GROUP;
    const int row0 = (first_row + in_group % rows) * C::BM, t0 = in_group / rows * C::BN;
    const int wm = wave % (C::BM / C::WM) * C::WM, wn = wave / (C::BM / C::WM) * C::WN;
    const int blocks = K / kScaleBlock + (K % kScaleBlock != 0);
    // what the wavefront loads of each stage: 8 rows at a time, of W or of X,
    // a lane a piece; rows past the end repeat the last one
    const int in = lane >> 3, piece = 16 * ((lane & 7) ^ in);
    const uint8_t* base[C::kLoads];
    int64_t offset[C::kLoads];  // the lane's, of its row
#pragma unroll
    for (int i = 0; i < C::kLoads; ++i) {
        const int row = (wave + i * C::kWaves) * 8;
        const bool of_w = row < C::BM;
        const int last = of_w ? M - 1 : T - 1;
        int first = of_w ? row0 + row : t0 + row - C::BM;
        first = first < last ? first : last;
        offset[i] = (in < last - first ? in : last - first) * (of_w ? lda : ldx);
        base[i] = of_w ? A + (int64_t)first * lda : X + (int64_t)first * ldx;
    }
    // ... and which scales: eight lines of eight blocks, block b of line n in
    // place b ^ (n / 8 % 2), so that 16 neighbouring lines lie in 16 banks
    const float* sbase[C::kScaleEach];
    int sleft[C::kScaleEach];  // lines behind the first of the eight
    uint32_t spitch[C::kScaleEach], sto[C::kScaleEach];
#pragma unroll
    for (int i = 0; i < C::kScaleEach; ++i) {
        const int n = wave + i * C::kWaves < C::kScaleLoads ? wave + i * C::kWaves : C::kScaleLoads - 1;
        sto[i] = n * 256;
        const bool of_x = n < C::BN / 8;
        const int last = of_x ? T - 1 : (M - 1) / kScaleBlock;
        int first = of_x ? t0 + n * 8 : row0 / kScaleBlock;
        first = first < last ? first : last;
        sbase[i] = of_x ? xs + (int64_t)first * ldxs : as + (int64_t)first * ldas;
        sleft[i] = last - first;
        spitch[i] = (uint32_t)(of_x ? ldxs : ldas);
    }
    const uint32_t lds_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    // Straight into LDS (DIRECT: whole, aligned pieces) ...
    const int tail = K % kScaleBlock, tail_block = tail ? blocks - 1 : -1;
    uint32_t from[DIRECT ? C::kLoads : 1];
    if constexpr (DIRECT)
#pragma unroll
        for (int i = 0; i < C::kLoads; ++i) from[i] = (uint32_t)offset[i] + piece;
    auto stage = [&](int to, int b) {
        const uint32_t at = lds_at + to * C::kStageBytes;
        if (b == tail_block) {  // once: what follows is that block again
            const int l = worked_out_here(lane);
            const int own = 16 * ((l & 7) ^ (l >> 3));
            const uint32_t back = own >= tail ? own : 0;
#pragma unroll
            for (int i = 0; i < C::kLoads; ++i) from[i] -= back;
        }
        const int64_t column = (int64_t)(b < blocks ? b : blocks - 1) * kScaleBlock;
#pragma unroll
        for (int i = 0; i < C::kLoads; ++i)
            lds_load16(base[i] + column, from[i], at + (wave + i * C::kWaves) * 1024);
    };
    // ... or through registers: fetched when a stage becomes free, written to it
    // at the end of the next phase.
    quad held[DIRECT ? 1 : C::kLoads];
    auto fetch = [&](int b) {
#pragma unroll
        for (int i = 0; i < C::kLoads; ++i) held[i] = piece_of(base[i] + offset[i], b, piece, K);
    };
    auto commit = [&](int to) {
        if constexpr (!DIRECT) {
#pragma unroll
            for (int i = 0; i < C::kLoads; ++i)
                *reinterpret_cast<quad*>(lds + to * C::kStageBytes + (wave + i * C::kWaves) * 1024 + lane * 16) = held[i];
            wait_lds();
        }
    };
    auto stage_scales = [&](int span) {
        const uint32_t at = lds_at + C::STAGES * C::kStageBytes + (span & 1) * C::kScaleBytes;
        const int l = worked_out_here(lane), line = l >> 3;
#pragma unroll
        for (int i = 0; i < C::kScaleEach; ++i) {
            const int swap = sto[i] / 256 & 1;  // line n / 8 of the load is n: all its lines share it
            const int b = span * C::kSpan + ((l & 7) ^ swap);
            lds_load4(sbase[i], ((line < sleft[i] ? line : sleft[i]) * spitch[i] + (b < blocks ? b : blocks - 1)) * 4,
                      at + sto[i]);
        }
    };

    f32x4 acc[NM][NN];
#pragma unroll
    for (int i = 0; i < NM; ++i)
#pragma unroll
        for (int j = 0; j < NN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int lo = r * kScaleBlock + 16 * (g ^ (r & 7));
    const int hi = r * kScaleBlock + 16 * ((g + 4) ^ (r & 7));
    i32x8 xf[NN], af[NM];
    float st[NN];
    auto read = [&](int b) {
        const uint8_t* at = lds + b % C::STAGES * C::kStageBytes;
        const uint8_t* a = at + wm * kScaleBlock;
        const uint8_t* x = at + (C::BM + wn) * kScaleBlock;
        const float* s = reinterpret_cast<const float*>(
            lds + C::STAGES * C::kStageBytes + (b / C::kSpan & 1) * C::kScaleBytes);
        const int span_at = b % C::kSpan;
#pragma unroll
        for (int j = 0; j < NN; ++j)
            xf[j] = join(*reinterpret_cast<const quad*>(x + 16 * j * kScaleBlock + lo),
                         *reinterpret_cast<const quad*>(x + 16 * j * kScaleBlock + hi));
#pragma unroll
        for (int i = 0; i < NM; ++i)
            af[i] = join(*reinterpret_cast<const quad*>(a + 16 * i * kScaleBlock + lo),
                         *reinterpret_cast<const quad*>(a + 16 * i * kScaleBlock + hi));
        if (DIRECT && b == tail_block)
#pragma unroll
            for (int j = 0; j < NN; ++j) blank_behind(xf[j], g, tail);
        const float sa = s[(C::BN + wm / kScaleBlock) * C::kSpan + (span_at ^ (C::BN / 8 & 1))];
#pragma unroll
        for (int j = 0; j < NN; ++j) st[j] = sa * s[(wn + 16 * j + r) * C::kSpan + (span_at ^ (r >> 3))];
    };
    auto multiply = [&]() {
        // a sum is scaled and added while the kLag next ones are multiplied
        constexpr int kLag = 3;
        f32x4 d[kLag + 1];
        Operand<EXACT> xo[NN];
#pragma unroll
        for (int j = 0; j < NN; ++j) xo[j] = Operand<EXACT>::of(xf[j]);
        Operand<EXACT> ao;
#pragma unroll
        for (int n = 0; n < NM * NN + kLag; ++n) {
            if (n < NM * NN) {
                if (n % NN == 0) ao = Operand<EXACT>::of(af[n / NN]);
                d[n % (kLag + 1)] = block_sum(ao, xo[n % NN]);
            }
            if (n >= kLag) {
                const int p = n - kLag, i = p / NN, j = p % NN;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[i][j][e] = __builtin_fmaf(d[p % (kLag + 1)][e], st[j], acc[i][j][e]);
            }
        }
        if constexpr (!EXACT) {
#pragma unroll
            for (int n = 0; n < NM * NN + kLag; ++n) {
                if (n < NM * NN) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                if (n >= kLag) __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
            }
        }
    };

    // Phase 2b: the first half reads block b, the second multiplies block
    // b - 1; phase 2b + 1: the first half multiplies block b, the second reads
    // it.  In phase 2b every wavefront loads block b - 1 + STAGES into the stage
    // that block b - 1 has left; before phase 2b block b has landed.  Past the
    // last block the last is loaded again, into stages that nothing reads any
    // more: every wavefront always waits for the same count.
    const int half = wave >> 2;
    // The scales of a span are loaded a block after the span before it began,
    // when nothing reads the span before that any more.
    auto load = [&](int b) {
        if constexpr (DIRECT)
            stage(b % C::STAGES, b);
        else
            fetch(b < blocks ? b : blocks - 1);
        const int at = b + 1 - C::STAGES;
        if (at % C::kSpan == 1) stage_scales(at / C::kSpan + 1);
    };
    // loads that may be in flight when a block must have landed (the scales of
    // the next span may be: they are wanted blocks later)
    constexpr int kInFlight = DIRECT ? C::kInFlight : 0;
    stage_scales(0);
#pragma unroll
    for (int b = 0; b < C::STAGES - 1; ++b) {
        load(b);
        commit(b);
    }
    wait_loads<kInFlight>();
    change_over();
    if (half == 0) {
        for (int b = 0; b < blocks; ++b) {
            load(b + C::STAGES - 1);
            read(b);
            wait_lds();
            change_over();
            __builtin_amdgcn_s_setprio(1);
            multiply();
            __builtin_amdgcn_s_setprio(0);
            commit((b + C::STAGES - 1) % C::STAGES);
            wait_loads<kInFlight>();
            change_over();
        }
        change_over();
    } else {
        load(C::STAGES - 1);
        change_over();
        for (int b = 0; b < blocks; ++b) {
            read(b);
            wait_lds();
            commit((b + C::STAGES - 1) % C::STAGES);
            wait_loads<kInFlight>();
            change_over();
            load(b + C::STAGES);
            __builtin_amdgcn_s_setprio(1);
            multiply();
            __builtin_amdgcn_s_setprio(0);
            change_over();
        }
    }
    // The results go through LDS, so that a token's BM values are stored as
    // one piece (straight from the registers they would be 32-byte pieces).
    wait_loads<0>();
    change_over();
    using S = typename O::storage;
    constexpr int kPitch = C::BM * O::bytes + 16;
    static_assert(C::BN * kPitch <= C::kLds, "the results fit the stages");
#pragma unroll
    for (int i = 0; i < NM; ++i) {
        const int m = wm + 16 * i + 4 * g;
        f32x4 add{0.0f, 0.0f, 0.0f, 0.0f};
        if (bias)
#pragma unroll
            for (int e = 0; e < 4; ++e) add[e] = bias[row0 + m + e < M ? row0 + m + e : M - 1];
#pragma unroll
        for (int j = 0; j < NN; ++j) {
            const f32x4 v = acc[i][j] + add;
            struct alignas(4 * O::bytes) Four {
                S v[4];
            };
            *reinterpret_cast<Four*>(lds + (wn + 16 * j + r) * kPitch + m * O::bytes) =
                Four{{narrow(O{}, v[0]), narrow(O{}, v[1]), narrow(O{}, v[2]), narrow(O{}, v[3])}};
        }
    }
    __syncthreads();
    constexpr int kPer = 16 / O::bytes, kAcross = C::BM / kPer;  // a lane's values, the lanes of a token
    const int m = threadIdx.x % kAcross * kPer;
    const int left_m = M - row0 - m;
    for (int t = threadIdx.x / kAcross; t < C::BN && t0 + t < T; t += C::kWaves * 64 / kAcross) {
        const uint8_t* from = lds + t * kPitch + m * O::bytes;
        S* to = static_cast<S*>(Y) + (int64_t)(t0 + t) * ldy + row0 + m;
        if (left_m >= kPer)
            *reinterpret_cast<quad_any*>(to) = *reinterpret_cast<const quad*>(from);
        else
            for (int e = 0; e < kPer && e < left_m; ++e) to[e] = reinterpret_cast<const S*>(from)[e];
    }
}

// ---------------------------------------------------------------------------
// product with few tiles: K split within the workgroup
//
// With few tiles, or few tokens, a compute unit has one workgroup and a step is
// bound by its latencies, not by its work; so four groups of four wavefronts
// take four scale blocks of the same BM rows by BN tokens in one step, a fourth
// of the steps, STAGES - 1 steps of bytes are in flight, and the groups join their
// sums in LDS, in a fixed order.
//
// 16 x 14336 x 4096 takes 11.6 us, which is W's bytes at 5.1 TB/s.  250 x 4096 x
// 11008 takes 28.7 us (787 TFLOP/s): bound by LDS, which
// a tile of 64 x 64 fills twice and reads a third more often for a product than one
// of 128 x 128, and by the latency between two barriers.
// ---------------------------------------------------------------------------
template <int BM_, int BN_, int STAGES_>
struct Split {
    static constexpr int BM = BM_, BN = BN_, STAGES = STAGES_, KS = 4, kWaves = 4 * KS;
    static constexpr int kAcross = BN >= 64 ? 2 : 1;              // wavefronts of a group across the tokens
    static constexpr int NM = BM / 16 / (4 / kAcross), NN = BN / 16 / kAcross;
    static constexpr int kBlockBytes = (BM + BN) * kScaleBlock;   // of one group
    // 1 KiB loads of a wavefront per step: of W, and of X (where those are
    // fewer than the wavefronts, the spare ones repeat the last)
    static constexpr int kLoadsW = BM / 32, kLoadsX = (BN / 8 + 3) / 4;
    // scales of a step: a line of KS blocks for each token, then one for the rows
    static constexpr int kScaleLoads = BN / 16 + 1;
    static constexpr int kStageBytes = KS * kBlockBytes + kScaleLoads * 256;
    static constexpr int kInFlight = (STAGES - 2) * (kLoadsW + kLoadsX + 1);
    static constexpr int kPitch = BM + 4;                         // of a token's sums, in fp32
    static constexpr int kLds = STAGES * kStageBytes;
    static_assert(BM % 64 == 0 && BN % 16 == 0 && kScaleLoads <= kWaves, "whole loads");
    static_assert(KS * BN * kPitch * 4 <= kLds && kLds <= 160 * 1024, "the sums fit the stages");
};

template <class O, class C, bool EXACT, bool DIRECT>
__global__ __launch_bounds__(C::kWaves * 64) void fp8_split_kernel(
    const uint8_t* A, int64_t lda, const float* as, int64_t ldas, const uint8_t* X, int64_t ldx,
    const float* xs, int64_t ldxs, const float* bias, void* Y, int64_t ldy, int M, int K, int T,
    int row_tiles) {
    extern __shared__ __align__(16) uint8_t lds[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int ks = wave >> 2, member = wave & 3;
    const int wm = member / C::kAcross * 16 * C::NM, wn = member % C::kAcross * 16 * C::NN;
    const int r = lane & 15, g = lane >> 4;
    // neighbours of a chiplet take the same rows of W with all the tokens
    const int tiles = gridDim.x, per = tiles / 8, id = blockIdx.x;
    const int tile = id < per * 8 ? id % 8 * per + id / 8 : id;
    const int token_tiles = tiles / row_tiles;
    const int row0 = tile / token_tiles * C::BM, t0 = tile % token_tiles * C::BN;
    const int blocks = K / kScaleBlock + (K % kScaleBlock != 0);

    // what the wavefront loads of each step: 8 rows at a time, of W, then of X
    constexpr int kLoads = C::kLoadsW + C::kLoadsX;
    const int in = lane >> 3, piece = 16 * ((lane & 7) ^ in);
    const auto first_row = [&](int i) {  // of load i, among the BM + BN
        if (i < C::kLoadsW) return (member + i * 4) * 8;
        const int n = member + (i - C::kLoadsW) * 4;
        return C::BM + (n < C::BN / 8 ? n : C::BN / 8 - 1) * 8;
    };
    const uint8_t* base[kLoads];
    int line[kLoads];  // the lane's, behind the first
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int row = first_row(i);
        const bool of_w = i < C::kLoadsW;
        const int last = of_w ? M - 1 : T - 1;
        int first = of_w ? row0 + row : t0 + row - C::BM;
        first = first < last ? first : last;
        base[i] = of_w ? A + (int64_t)first * lda : X + (int64_t)first * ldx;
        line[i] = in < last - first ? in : last - first;
    }
    const int sn = wave < C::kScaleLoads ? wave : C::kScaleLoads - 1;
    const float* sbase;
    uint32_t soffset;
    {
        const bool of_x = sn < C::BN / 16;
        const int last = of_x ? T - 1 : (M - 1) / kScaleBlock;
        int first = of_x ? t0 + sn * 16 : row0 / kScaleBlock;
        first = first < last ? first : last;
        const int line = lane >> 2;
        sbase = of_x ? xs + (int64_t)first * ldxs : as + (int64_t)first * ldas;
        soffset = (uint32_t)(line < last - first ? line : last - first) * (uint32_t)(of_x ? ldxs : ldas);
    }
    const uint32_t lds_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    const int tail = K % kScaleBlock, tail_block = tail ? blocks - 1 : -1;
    const uint32_t back = tail && piece >= tail ? piece : 0;
    // Straight into LDS (DIRECT: whole, aligned pieces), or through registers, written to the stage at
    // the end of the step.  Past the last block the last is loaded again, into
    // places that nothing reads: every wavefront always waits for the same count.
    quad held[DIRECT ? 1 : kLoads];
    auto stage = [&](int n, int to) {
        int b = n * C::KS + ks;
        b = b < blocks ? b : blocks - 1;
        const uint32_t own = b == tail_block ? piece - back : piece;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if constexpr (DIRECT)
                lds_load16(base[i] + (int64_t)b * kScaleBlock,
                           line[i] * (uint32_t)(i < C::kLoadsW ? lda : ldx) + own,
                           lds_at + to * C::kStageBytes + ks * C::kBlockBytes + first_row(i) * kScaleBlock);
            else
                held[i] = piece_of(base[i] + line[i] * (i < C::kLoadsW ? lda : ldx), b, piece, K);
        const int sb = n * C::KS + (lane & 3);
        lds_load4(sbase, (soffset + (sb < blocks ? sb : blocks - 1)) * 4,
                  lds_at + to * C::kStageBytes + C::KS * C::kBlockBytes + sn * 256);
    };
    auto commit = [&](int to) {
        if constexpr (!DIRECT) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                *reinterpret_cast<quad*>(lds + to * C::kStageBytes + ks * C::kBlockBytes +
                                         first_row(i) * kScaleBlock + lane * 16) = held[i];
            wait_lds();
        }
    };
    constexpr int kInFlight = DIRECT ? C::kInFlight : 0;

    f32x4 acc[C::NM][C::NN];
#pragma unroll
    for (int i = 0; i < C::NM; ++i)
#pragma unroll
        for (int j = 0; j < C::NN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int lo = r * kScaleBlock + 16 * (g ^ (r & 7));
    const int hi = r * kScaleBlock + 16 * ((g + 4) ^ (r & 7));
    const int steps = (blocks + C::KS - 1) / C::KS;
    auto product_of = [&](int b, int from) {
        const uint8_t* at = lds + from * C::kStageBytes;
        const uint8_t* a = at + ks * C::kBlockBytes + wm * kScaleBlock;
        const uint8_t* x = at + ks * C::kBlockBytes + (C::BM + wn) * kScaleBlock;
        const float* s = reinterpret_cast<const float*>(at + C::KS * C::kBlockBytes);
        Operand<EXACT> xo[C::NN];
        float st[C::NN];
        const float sa = s[(C::BN + wm / kScaleBlock) * C::KS + ks];
#pragma unroll
        for (int j = 0; j < C::NN; ++j) {
            i32x8 xf = join(*reinterpret_cast<const quad*>(x + 16 * j * kScaleBlock + lo),
                            *reinterpret_cast<const quad*>(x + 16 * j * kScaleBlock + hi));
            if (DIRECT && b == tail_block) blank_behind(xf, g, tail);
            xo[j] = Operand<EXACT>::of(xf);
            st[j] = sa * s[(wn + 16 * j + r) * C::KS + ks];
        }
#pragma unroll
        for (int i = 0; i < C::NM; ++i) {
            const Operand<EXACT> ao =
                Operand<EXACT>::of(join(*reinterpret_cast<const quad*>(a + 16 * i * kScaleBlock + lo),
                                        *reinterpret_cast<const quad*>(a + 16 * i * kScaleBlock + hi)));
#pragma unroll
            for (int j = 0; j < C::NN; ++j) {
                const f32x4 d = block_sum(ao, xo[j]);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(d[e], st[j], acc[i][j][e]);
            }
        }
    };
#pragma unroll
    for (int n = 0; n < C::STAGES - 1; ++n) {
        stage(n, n);
        commit(n);
    }
    int now = 0, next = C::STAGES - 1;
    for (int n = 0; n < steps; ++n) {
        wait_loads<kInFlight>();
        change_over();
        stage(n + C::STAGES - 1, next);
        if (n * C::KS + ks < blocks) product_of(n * C::KS + ks, now);
        commit(next);
        next = now;
        now = now + 1 == C::STAGES ? 0 : now + 1;
    }
    wait_loads<0>();
    change_over();
    // join: a token's BM values in a line, the groups' one behind the other
    float* sums = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int i = 0; i < C::NM; ++i)
#pragma unroll
        for (int j = 0; j < C::NN; ++j)
            *reinterpret_cast<f32x4*>(sums + (ks * C::BN + wn + 16 * j + r) * C::kPitch + wm + 16 * i + 4 * g) = acc[i][j];
    __syncthreads();
    constexpr int kLine = C::BM / 4;  // lanes of a token
    for (int e = threadIdx.x; e < C::BN * kLine; e += C::kWaves * 64) {
        const int t = e / kLine, m = e % kLine * 4;
        if (t0 + t >= T || row0 + m >= M) continue;
        f32x4 v = *reinterpret_cast<const f32x4*>(sums + t * C::kPitch + m);
#pragma unroll
        for (int k = 1; k < C::KS; ++k) v += *reinterpret_cast<const f32x4*>(sums + (k * C::BN + t) * C::kPitch + m);
        if (bias)
#pragma unroll
            for (int n = 0; n < 4; ++n) v[n] += bias[row0 + m + n < M ? row0 + m + n : M - 1];
        store_row4<O>(Y, (int64_t)(t0 + t) * ldy, row0 + m, M, v);
    }
}

}  // namespace fp8dev
