// Kernels of the products with 4-bit weights and group scales.
//
//   Y[t,m] = Σ_g scale[m,g]·Σ_{k in g} (q[m,k] - zero[m,g])·X[t,k] + bias[m]
//
// q - zero is a whole number of at most 8 bits, so fp16 and bf16 hold it, and
// the matrix cores' products with X are exact; a group's products are summed
// in fp32 and its sum is scaled and added in fp32.  fp32 vectors go to the
// matrix cores as three bf16 parts that add up to them exactly.
#pragma once

#include "fp8_device.hpp"
#include "fp8_kernels.hpp"
#include "q4_plan.hpp"

namespace q4dev {

using fp8dev::bf16x2;
using fp8dev::f16x2;
using fp8dev::f32x4;
using fp8dev::quad;
using fp8dev::quad_any;
using fp8dev::TBF16;
using fp8dev::TF16;
using fp8dev::TF32;
using fp8dev::u32x2;
using fp8dev::widen;

using q4plan::kChunk;
constexpr int kNoZero = 8;  // the zero of weights without zeros

struct Product {
    const uint8_t* Q;
    int64_t ldq;
    const void* scale;
    int64_t lds;
    const uint8_t* zero;         // without zeros: bytes that may be read in their place, ...
    int64_t ldz;
    uint32_t zero_mask, no_zero;  // ... of which this mask leaves nothing, and kNoZero in each byte
    const void* X;
    int64_t ldx;
    const float* bias;           // or NULL
    void* Y;
    int64_t ldy;
    int y_type;                  // gemv_dtype_t
    int M, K, T;
};

// The type that X meets the weights in, and in how many parts.
template <class T>
struct Operand {
    using type = T;
    static constexpr int parts = 1;
};
template <>
struct Operand<TF32> {
    using type = TBF16;
    static constexpr int parts = 3;
};

// ---------------------------------------------------------------------------
// weights
//
// A word holds eight columns, the first in its lowest four bits.  Shifted right
// by 4·i its two halves' lowest bits are columns i and i + 4, so the eight
// values come out as the pairs (0,4), (1,5), (2,6), (3,7); X is taken in the same
// order.  With 1024's exponent around them the four bits are the fp16 number
// 1024 + q, from which 1024 + zero is taken exactly.
// ---------------------------------------------------------------------------

// 1024 + zero: for fp16 twice in a word, for bf16 as an fp32 number.
__device__ __forceinline__ uint32_t offset_of(TF16, uint32_t zero) { return zero * 0x10001u + 0x64006400u; }
__device__ __forceinline__ float offset_of(TBF16, uint32_t zero) { return (float)zero + 1024.0f; }

// The four bits' place in both halves and 1024's exponent; the latter stays in a
// vector register, so that one instruction masks and sets (an instruction of three
// operands takes no constant of 32 bits and one scalar register).
__device__ __forceinline__ uint32_t pair_of(uint32_t w, int i, uint32_t exponent) {
    return ((w >> (4 * i)) & 0x000f000fu) | exponent;
}
__device__ __forceinline__ uint32_t exponent_of_1024() {
    uint32_t e = 0x64006400u;
    asm("" : "+v"(e));
    return e;
}
// A half of a pair of fp16 values minus an fp32 number.
template <int HALF>
__device__ __forceinline__ float half_minus(uint32_t pair, float b) {
    float d;
    if constexpr (HALF == 0)
        asm("v_fma_mix_f32 %0, %1, 1.0, -%2 op_sel_hi:[1,0,0]" : "=v"(d) : "v"(pair), "v"(b));
    else
        asm("v_fma_mix_f32 %0, %1, 1.0, -%2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(d) : "v"(pair), "v"(b));
    return d;
}
__device__ __forceinline__ quad values8(TF16, uint32_t w, uint32_t offset, uint32_t exponent) {
    quad v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, pair_of(w, i, exponent)) -
                                                __builtin_bit_cast(f16x2, offset));
    return v;
}
__device__ __forceinline__ quad values8(TBF16, uint32_t w, float offset, uint32_t exponent) {
    quad v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t p = pair_of(w, i, exponent);
        const uint32_t a = __builtin_bit_cast(uint32_t, half_minus<0>(p, offset));
        const uint32_t b = __builtin_bit_cast(uint32_t, half_minus<1>(p, offset));
        v[i] = __builtin_amdgcn_perm(b, a, 0x07060302u);  // their upper halves: whole numbers of 8 bits
    }
    return v;
}

// A lane's 16 bytes of a row are columns 32·g .. 32·g+31 of the chunk (g =
// lane / 16); the matrix cores want columns 32·j + 8·g .. +7 at step j, so the
// four words are transposed among the four groups of lanes.
__device__ __forceinline__ quad transposed(quad w) {
    auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return quad{c[0], c[1], d[0], d[1]};
}

// ---------------------------------------------------------------------------
// vectors
// ---------------------------------------------------------------------------

template <class T>
struct Vec8 {  // eight columns of a vector, as the matrix cores take them
    quad part[Operand<T>::parts];
};

// Pairs (0,4), (1,5), (2,6), (3,7) of eight 16-bit values in order.
__device__ __forceinline__ quad in_order(quad v) {
    return quad{__builtin_amdgcn_perm(v[2], v[0], 0x05040100u), __builtin_amdgcn_perm(v[2], v[0], 0x07060302u),
                __builtin_amdgcn_perm(v[3], v[1], 0x05040100u), __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)};
}
template <class T>
__device__ __forceinline__ Vec8<T> operand_of(T, quad v) {
    return Vec8<T>{{in_order(v)}};
}
// An fp32 value is the sum of its first 8 bits, the next 8 and the last 8: cut
// off, not rounded, so each part is exact and none overflows.  An infinity or
// NaN is its first part alone.
__device__ __forceinline__ Vec8<TF32> operand_of(TF32, quad lo, quad hi) {
    uint32_t p[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t bits = i < 4 ? lo[i] : hi[i - 4];
        const bool finite = (bits & 0x7f800000u) != 0x7f800000u;
        // (a NaN may have all its bits in the lower half)
        const uint32_t first = finite ? bits : bits | ((bits & 0xffffu) ? 0x10000u : 0u);
        const float rest = finite ? gemvdev::f32_of(bits) - gemvdev::f32_of(bits & 0xffff0000u) : 0.0f;
        const uint32_t second = __builtin_bit_cast(uint32_t, rest);
        const float last = rest - gemvdev::f32_of(second & 0xffff0000u);
        p[0][i] = first;
        p[1][i] = second;
        p[2][i] = __builtin_bit_cast(uint32_t, last);
    }
    Vec8<TF32> v;
#pragma unroll
    for (int n = 0; n < 3; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) v.part[n][i] = __builtin_amdgcn_perm(p[n][i + 4], p[n][i], 0x07060302u);
    return v;
}

// A uniform address that the compiler keeps in scalar registers: loads add the lanes'
// 32-bit offsets to it, where it would else keep a 64-bit address for each of them.
// (It names global memory: loads from anywhere are counted as LDS's too, and every
// wait for LDS would be one for them.)
using global_bytes = const uint8_t __attribute__((address_space(1)))*;
__device__ __forceinline__ global_bytes scalar_here(const uint8_t* p) {
    global_bytes g = (global_bytes)p;
    asm volatile("" : "+s"(g));
    return g;
}
using global_quad = const quad_any __attribute__((address_space(1)))*;
__device__ __forceinline__ uint32_t offset_here(uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
}

// 16 bytes at byte `at` of a row of `bytes` (at least 16), in one load: near the
// row's end the last 16, moved down; what lies behind reads as zero.
__device__ __forceinline__ quad load_end(const uint8_t* row, int64_t at, int64_t bytes) {
    const int64_t from = at < bytes - 16 ? at : bytes - 16;
    const int64_t by = at - from;
    const int down = by < 16 ? (int)by : 16;
    quad v = *reinterpret_cast<const quad_any*>(row + from);
    if (down & 4) v = quad{v[1], v[2], v[3], 0u};
    if (down & 8) v = quad{v[2], v[3], 0u, 0u};
    if (down & 16) v = quad{0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __builtin_amdgcn_alignbyte(i < 3 ? v[i + 1] : 0u, v[i], down & 3);
    return v;
}

// What a lane loads of a vector for one matrix-core step: columns k .. k+7;
// those from K on read as zero and are not touched.  Rows are of 32 columns at least.
template <class T>
struct Raw8 {
    quad v[T::bytes / 2];
};
template <class T>
__device__ __forceinline__ Raw8<T> load_vec(const typename T::storage* x, int64_t k, bool whole, int K) {
    Raw8<T> r;
    if (whole) {
#pragma unroll
        for (int i = 0; i < T::bytes / 2; ++i)
            r.v[i] = *reinterpret_cast<const quad_any*>(x + k + i * (16 / T::bytes));
    } else {
#pragma unroll
        for (int i = 0; i < T::bytes / 2; ++i)
            r.v[i] = load_end(reinterpret_cast<const uint8_t*>(x), k * T::bytes + 16 * i, (int64_t)K * T::bytes);
    }
    return r;
}
template <class T>
__device__ __forceinline__ Vec8<T> operand_of(const Raw8<T>& r) {
    if constexpr (T::bytes == 4)
        return operand_of(T{}, r.v[0], r.v[1]);
    else
        return operand_of(T{}, r.v[0]);
}

// Scales and zeros of U neighbouring chunks of a row as they lie in memory (G:
// columns of a group over kBlock, as a power of two); those of groups behind the row's last
// are 0.
// N bytes from p on as they are: a number of the narrow type where N is 2 (widened
// right behind the load, it would be waited for there), else words.
template <int N>
struct Narrow {
    using type = uint32_t;
};
template <>
struct Narrow<2> {
    using type = uint16_t;
};
template <int N>
__device__ __forceinline__ void load_words(global_bytes p, typename Narrow<N>::type (&v)[(N + 3) / 4]) {
    if constexpr (N == 1) {
        v[0] = *p;
        return;
    }
    typedef typename Narrow<N>::type Word;
    typedef Word Words __attribute__((ext_vector_type((N + 3) / 4), aligned(1)));
    const Words w = *(const Words __attribute__((address_space(1)))*)p;
#pragma unroll
    for (int i = 0; i < (N + 3) / 4; ++i) v[i] = w[i];
}
template <class T, int G, int U>
struct RawScales {
    static constexpr int N = 4 * U >> G, kWords = (N * T::bytes + 3) / 4, kZeros = (N + 3) / 4;
    typename Narrow<N * T::bytes>::type s[kWords];
    typename Narrow<N>::type z[kZeros];

    // of step j (0 .. 4·U-1)
    __device__ __forceinline__ float scale(int j) const {
        const int i = j >> G;
        if constexpr (T::bytes == 4) return gemvdev::f32_of(s[i]);
        return widen(T{}, (uint16_t)(s[i >> 1] >> (16 * (i & 1))));
    }
    __device__ __forceinline__ uint32_t zero(const Product& p, int j) const {
        const int i = j >> G;
        return (((uint32_t)z[i >> 2] & p.zero_mask) | p.no_zero) >> (8 * (i & 3)) & 0xffu;
    }
    template <class MT>
    __device__ __forceinline__ auto offset(const Product& p, int j) const {
        return offset_of(MT{}, zero(p, j));
    }
};
template <class T, int G, int U>
__device__ __forceinline__ RawScales<T, G, U> load_scales(const Product& p, int64_t m, int chunk, bool whole) {
    using R = RawScales<T, G, U>;
    using S = typename T::storage;
    const int g0 = 4 * chunk >> G;
    const S* s = static_cast<const S*>(p.scale) + m * p.lds + g0;
    const uint8_t* z = p.zero + m * p.ldz + g0;
    R r;
    if (whole) {
        load_words<R::N * T::bytes>((global_bytes)s, r.s);
        load_words<R::N>((global_bytes)z, r.z);
        return r;
    }
#pragma unroll
    for (int i = 0; i < R::kWords; ++i) r.s[i] = 0;
#pragma unroll
    for (int i = 0; i < R::kZeros; ++i) r.z[i] = 0;
    const int left = q4plan::groups_of(p.K, G) - g0;  // groups from g0 on
#pragma unroll
    for (int i = 0; i < R::N; ++i) {
        const int at = i < left ? i : left - 1;  // (those behind repeat the last, and become 0)
        if constexpr (T::bytes == 4) {
            const uint32_t v = __builtin_bit_cast(uint32_t, s[at]);
            r.s[i] = i < left ? v : 0u;
        } else {
            const uint32_t v = s[at];
            r.s[i >> 1] = (typename Narrow<R::N * 2>::type)(r.s[i >> 1] | (i < left ? v : 0u) << (16 * (i & 1)));
        }
        r.z[i >> 2] = (typename Narrow<R::N>::type)(r.z[i >> 2] | (uint32_t)z[at] << (8 * (i & 3)));
    }
    return r;
}

template <class O>
__device__ __forceinline__ void put(const Product& p, int64_t at, float v) {
    static_cast<typename O::storage*>(p.Y)[at] = fp8dev::narrow(O{}, v);
}
// f with the type of Y.
template <class F>
__device__ __forceinline__ void with_type(const Product& p, F f) {
    if (p.y_type == 0)
        f(TF32{});
    else if (p.y_type == 1)
        f(TF16{});
    else
        f(TBF16{});
}
__device__ __forceinline__ void store(const Product& p, int t, int m, float v) {
    const int64_t at = t * p.ldy + m;
    if (p.y_type == 0)
        put<TF32>(p, at, v);
    else if (p.y_type == 1)
        put<TF16>(p, at, v);
    else
        put<TBF16>(p, at, v);
}

// Rows of fewer columns than one matrix-core step (and the empty sum): a thread a
// result.
template <class T>
__global__ __launch_bounds__(256) void q4_short_kernel(Product p) {
    const int64_t t = blockIdx.y;
    const int m = (int)(blockIdx.x * 256 + threadIdx.x);
    if (m >= p.M) return;
    float v = 0.0f;
    if (p.K > 0) {
        const uint8_t* q = p.Q + m * p.ldq;
        const typename T::storage* x = static_cast<const typename T::storage*>(p.X) + t * p.ldx;
        const float zero = (float)(((p.zero[m * p.ldz] & p.zero_mask) | p.no_zero) & 0xffu);
        for (int k = 0; k < p.K; ++k) v = __builtin_fmaf((float)(q[k >> 1] >> (4 * (k & 1)) & 15) - zero, widen(T{}, x[k]), v);
        v *= widen(T{}, static_cast<const typename T::storage*>(p.scale)[m * p.lds]);
    }
    if (p.bias) v += p.bias[m];
    store(p, (int)t, m, v);
}

// The products of one chunk: acc += scale·(w·x) for each group, which takes one,
// two or four steps.
template <class MT, int G, int RT, int NT, int PARTS, class S, class X>
__device__ __forceinline__ void multiply(const Product& p, f32x4 (&acc)[RT][NT], const quad (&w)[RT], const S (&scales)[RT], int first,
                                         X&& x_of) {
    constexpr int kSteps = 1 << G;
    const uint32_t exponent = exponent_of_1024();
#pragma unroll
    for (int j0 = 0; j0 < 4; j0 += kSteps) {
        f32x4 d[RT][NT];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int j = j0 + s;
            quad b[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i) b[i] = values8(MT{}, w[i][j], scales[i].template offset<MT>(p, first + j), exponent);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const auto v = x_of(n, j);
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    if (s == 0) d[i][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int e = 0; e < PARTS; ++e) d[i][n] = gemvdev::mma_16x16x32(MT{}, v.part[e], b[i], d[i][n]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const float by = scales[i].scale(first + j0);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][n][e] = __builtin_fmaf(d[i][n][e], by, acc[i][n][e]);
        }
    }
}

// Few vectors: a workgroup takes 16·RT rows by 16·NT vectors; its W wavefronts
// take U neighbouring chunks of 128 columns in turn, the next ones' weights and
// scales in flight while those at hand are multiplied, and add their sums in LDS,
// in a fixed order.  A lane has row (and vector) lane % 16.
//
// STAGED (where the vectors fit): they are brought to LDS once for the workgroup, in
// the order that the weights come out in; an fp32 vector as three, of its parts,
// whose sums are added at the end.
//
// Bound by the latency of this mapping, not by memory: nearly all of a wavefront's share is
// one batch with nothing in flight behind it, so a call is a launch, a load and a join.
// 1 x 4096 x 4096 fp16 4.6 us (1.9 TB/s), 16 x 14336 x 4096 bf16 12.5 (2.5), fp32 1 x 4096
// x 11008 with groups of 32 10.9 (2.7).  With weights that no cache holds the int8 rows of
// gemv_q8 read twice the bytes of 1 x 14336 x 4096 in 11.0 us, where this takes 12.4.
// A lane's 16 bytes are in another row than its neighbours', which costs the first
// cache four accesses for one; loaded one behind the other and passed on through LDS
// they take a quarter of the accesses and the same time or more (16 x 14336: 13.8).
// X of 16 vectors staged whole, as the fp32 parts are, leaves one workgroup to a compute
// unit (19.7).
template <class T, int G, int RT, int NT, int W, int U, bool STAGED>
__global__ __launch_bounds__(W * 64) void q4_few_kernel(Product p) {
    using MT = typename Operand<T>::type;
    constexpr int PER = STAGED ? Operand<T>::parts : 1, PARTS = STAGED ? 1 : Operand<T>::parts;
    static_assert(!STAGED || NT == 1, "one tile of vectors or parts");
    extern __shared__ __align__(16) uint8_t lds[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int r = lane & 15, g = lane >> 4;
    const int row0 = (int)blockIdx.x * 16 * RT, t0 = (int)blockIdx.y * 16 * NT;
    const int chunks = p.K / kChunk + (p.K % kChunk != 0), whole = p.K / kChunk;
    // rows and vectors past the end repeat the last one; their results are not stored
    int64_t m[RT];
    const uint8_t* q[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        m[i] = row0 + 16 * i + r < p.M ? row0 + 16 * i + r : p.M - 1;
        q[i] = p.Q + m[i] * p.ldq + 16 * g;
    }
    const typename T::storage* x[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int t = t0 + 16 * n + r;
        x[n] = static_cast<const typename T::storage*>(p.X) + (t < p.T ? t : p.T - 1) * p.ldx;
    }
    f32x4 acc[RT][NT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[i][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    struct Batch {
        quad w[U][RT];
        RawScales<T, G, U> s[RT];
        Raw8<T> x[STAGED ? 1 : U][NT][4];
    };
    const auto load_x = [&](Raw8<T> (&to)[NT][4], int c, bool all) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) to[n][j] = load_vec<T>(x[n], (int64_t)c * kChunk + 32 * j + 8 * g, all, p.K);
    };
    const auto load = [&](Batch& to, int c) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < RT; ++i)
                to.w[u][i] = *reinterpret_cast<const quad_any*>(q[i] + (int64_t)(c + u) * (kChunk / 2));
#pragma unroll
        for (int i = 0; i < RT; ++i) to.s[i] = load_scales<T, G, U>(p, m[i], c, true);
        if constexpr (!STAGED)
#pragma unroll
            for (int u = 0; u < U; ++u) load_x(to.x[u], c + u, true);
    };
    // a vector's (or part's) line in LDS: whole chunks and 16 bytes, so that lines
    // start in other banks
    const int pitch = STAGED ? chunks * kChunk * 2 + 16 : 0;
    const uint8_t* line = lds + (r < PER * p.T ? r : PER * p.T - 1) * pitch + 16 * g;
    struct Parts {
        quad part[PARTS];
    };
    // the products of chunk c of the U that start at its batch's first
    const auto chunk = [&](quad (&w)[RT], const auto (&scales)[RT], const Raw8<T> (&raw)[NT][4], int u, int c) {
#pragma unroll
        for (int i = 0; i < RT; ++i) w[i] = transposed(w[i]);
        multiply<MT, G, RT, NT, PARTS>(p, acc, w, scales, 4 * u, [&](int n, int j) {
            Parts v;
            if constexpr (STAGED) {
                v.part[0] = *reinterpret_cast<const quad*>(line + c * 256 + 64 * j);
            } else {
                const Vec8<T> full = operand_of<T>(raw[n][j]);
#pragma unroll
                for (int e = 0; e < PARTS; ++e) v.part[e] = full.part[e];
            }
            return v;
        });
    };
    const auto work = [&](Batch& b, int c) {
#pragma unroll
        for (int u = 0; u < U; ++u) chunk(b.w[u], b.s, b.x[STAGED ? 0 : u], u, c + u);
    };
    int c = wave * U;
    Batch batch;
    const bool any = c + U <= whole;
    if (any) load(batch, c);
    if constexpr (STAGED) {
        const int pieces = chunks * 16;
        for (int at = threadIdx.x; at < p.T * pieces; at += W * 64) {
            const int t = at / pieces, piece = at - t * pieces;
            const Vec8<T> v = operand_of<T>(load_vec<T>(static_cast<const typename T::storage*>(p.X) + t * p.ldx,
                                                        piece * 8, p.K % kChunk == 0, p.K));
#pragma unroll
            for (int e = 0; e < PER; ++e)
                *reinterpret_cast<quad*>(lds + (t * PER + e) * pitch + piece * 16) = v.part[e];
        }
        __syncthreads();
    }
    if (any) {
        while (true) {
            work(batch, c);
            c += W * U;
            if (c + U > whole) break;
            load(batch, c);
        }
    }
    // the last columns: fewer chunks than U, the last of fewer columns
    for (int u = 0; u < U && c + u < chunks; ++u) {
        const int64_t row_bytes = p.K / 2 + (p.K & 1);
        quad w[RT];
        RawScales<T, G, 1> s[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            w[i] = load_end(p.Q + m[i] * p.ldq, (int64_t)(c + u) * (kChunk / 2) + 16 * g, row_bytes);
            s[i] = load_scales<T, G, 1>(p, m[i], c + u, false);
        }
        Raw8<T> raw[NT][4];
        if constexpr (!STAGED) load_x(raw, c + u, false);
        chunk(w, s, raw, 0, c + u);
    }
    // join: of the tile's 256 sums a thread takes one, vector e / 16, row e % 16
    if constexpr (STAGED) __syncthreads();  // (the sums lie where the vectors did)
    f32x4(*part)[64] = reinterpret_cast<f32x4(*)[64]>(lds);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n) part[(i * NT + n) * W + wave][lane] = acc[i][n];
    __syncthreads();
    for (int at = threadIdx.x; at < RT * NT * 256; at += W * 64) {
        const int tile = at >> 8, i = tile / NT, n = tile - i * NT;
        const int tt = at >> 4 & 15, rr = at & 15;
        const int t = t0 + 16 * n + tt, row = row0 + 16 * i + rr;
        if (PER * tt > 16 - PER || t >= p.T || row >= p.M) continue;
        float v = 0.0f;
#pragma unroll
        for (int a = 0; a < PER; ++a) {
            const int from = PER * tt + a;
#pragma unroll
            for (int k = 0; k < W; ++k) v += part[tile * W + k][(from >> 2) * 16 + rr][from & 3];
        }
        if (p.bias) v += p.bias[row];
        store(p, t, row, v);
    }
}

// ---------------------------------------------------------------------------
// many vectors: X through LDS
//
// A workgroup takes 16·RT·W rows by 16·NT vectors, a wavefront 16·RT rows of its
// own by all the vectors, so no weight is widened twice.  A chunk of 128 columns
// of X lies in LDS in the order that the weights' values come out in, its parts one
// behind the other; the next chunk's X and weights are loaded into registers
// meanwhile.
//
// LDS.  A vector's 256 bytes of a chunk are 16 slots; slot s holds piece
// s ^ (vector % 16), so that 16 lanes that want the same piece of 16 neighbouring
// vectors find it in 16 different slots.
//
// Bound by the vector ALUs (widening a weight for 128 vectors, and an fp32 multiply-add
// for each sum and group), which the matrix cores wait for: 500 x 4096 x 4096, 64 x 64,
// 42 us (390 TFLOP/s); 2000 x 14336 x 4096, 128 x 128, 388 (605).
// ---------------------------------------------------------------------------
template <class T, int G, int RT, int NT, int W>
__global__ __launch_bounds__(W * 64, 2) void q4_tile_kernel(Product p, int row_tiles) {
    using MT = typename Operand<T>::type;
    using R = RawScales<T, G, 1>;
    constexpr int PARTS = Operand<T>::parts, BN = 16 * NT, BM = 16 * RT * W;
    constexpr int kPieces = BN * 16 / (W * 64);       // of X, for each thread and chunk
    constexpr int kPart = BN * 256, kStage = PARTS * kPart;
    static_assert(BN * 16 % (W * 64) == 0 && W * 4 % 16 == 0,
                  "whole pieces, which lie in the same slot of their vectors for each thread");
    extern __shared__ __align__(16) uint8_t lds[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int r = lane & 15, g = lane >> 4;
    // the workgroups that share a chiplet's cache (every eighth) take
    // neighbouring tiles: all the vectors of a row tile, then the next
    const int tiles = gridDim.x, per = tiles / 8, id = blockIdx.x;
    const int tile = id < per * 8 ? id % 8 * per + id / 8 : id;
    const int token_tiles = tiles / row_tiles;
    const int row0 = tile / token_tiles * BM, t0 = tile % token_tiles * BN;
    const int chunks = p.K / kChunk + (p.K % kChunk != 0);
    const int row_bytes = p.K / 2 + (p.K & 1);
    // rows and vectors past the end repeat the last one; their results are not stored.
    // Places are 32-bit offsets from the tile's first row or vector.
    const int64_t first_row = row0 + wave * RT * 16 < p.M ? row0 + wave * RT * 16 : p.M - 1;
    uint32_t q_at[RT], s_at[RT], z_at[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int left = p.M - 1 - (int)first_row;
        const uint32_t n = 16 * i + r < left ? 16 * i + r : left;
        q_at[i] = n * (uint32_t)p.ldq + 16 * g;
        s_at[i] = n * (uint32_t)p.lds * T::bytes;
        z_at[i] = n * (uint32_t)p.ldz;
    }
    const uint8_t* q0 = p.Q + first_row * p.ldq;
    const uint8_t* s0 = static_cast<const uint8_t*>(p.scale) + first_row * p.lds * T::bytes;
    const uint8_t* z0 = p.zero + first_row * p.ldz;
    const uint8_t* x0 = static_cast<const uint8_t*>(p.X) + t0 * p.ldx * T::bytes;
    const int piece = threadIdx.x & 15, first = threadIdx.x >> 4;
    const int to = first * 256 + 16 * (piece ^ (first & 15));

    Raw8<T> ahead[kPieces];
    quad next[RT];
    R then[RT];
    const auto fetch = [&](int c) {
        const global_bytes xc = scalar_here(x0 + (int64_t)c * (kChunk * T::bytes));
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int t = first + i * (W * 4), last = p.T - 1 - t0;
            const uint32_t at = (uint32_t)(t < last ? t : last) * ((uint32_t)p.ldx * T::bytes) + piece * 8 * T::bytes;
#pragma unroll
            for (int h = 0; h < T::bytes / 2; ++h) ahead[i].v[h] = *(global_quad)(xc + offset_here(at + 16 * h));
        }
        const int g0 = 4 * c >> G;
        const global_bytes qc = scalar_here(q0 + (int64_t)c * (kChunk / 2));
        const global_bytes sc = scalar_here(s0 + (int64_t)g0 * T::bytes);
        const global_bytes zc = scalar_here(z0 + g0);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            next[i] = *(global_quad)(qc + offset_here(q_at[i]));
            R raw;
            load_words<R::N * T::bytes>(sc + offset_here(s_at[i]), raw.s);
            load_words<R::N>(zc + offset_here(z_at[i]), raw.z);
            then[i] = raw;
        }
    };
    // the last chunk, where it has fewer columns
    const auto fetch_end = [&](int c) {
        const int id = fp8dev::worked_out_here(threadIdx.x);
        const int64_t k = (int64_t)c * (kChunk * T::bytes);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int t = t0 + (id >> 4) + i * (W * 4);
            const uint8_t* row = static_cast<const uint8_t*>(p.X) + (t < p.T ? t : p.T - 1) * p.ldx * T::bytes;
#pragma unroll
            for (int h = 0; h < T::bytes / 2; ++h)
                ahead[i].v[h] = load_end(row, k + (id & 15) * 8 * T::bytes + 16 * h, (int64_t)p.K * T::bytes);
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int row = row0 + ((id >> 6) * RT + i) * 16 + (id & 15);
            const int64_t m = row < p.M ? row : p.M - 1;
            next[i] = load_end(p.Q + m * p.ldq, (int64_t)c * (kChunk / 2) + 16 * ((id & 63) >> 4), row_bytes);
            then[i] = load_scales<T, G, 1>(p, m, c, false);
        }
    };
    const auto put_x = [&](int c) {
        uint8_t* stage = lds + (c & 1) * kStage;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const Vec8<T> v = operand_of<T>(ahead[i]);
#pragma unroll
            for (int e = 0; e < PARTS; ++e)
                *reinterpret_cast<quad*>(stage + e * kPart + to + i * (W * 4 * 256)) = v.part[e];
        }
    };
    f32x4 acc[RT][NT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[i][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int whole = p.K / kChunk;
    if (whole > 0)
        fetch(0);
    else
        fetch_end(0);
    put_x(0);
    __syncthreads();
    const uint32_t exponent = exponent_of_1024();
    for (int c = 0; c < chunks; ++c) {
        quad w[RT];
        R s[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            w[i] = transposed(next[i]);
            s[i] = then[i];
        }
        if (c + 1 < whole) fetch(c + 1);
        const uint8_t* stage = lds + (c & 1) * kStage + r * 256;
        // a group's steps, two at most (of 128 columns in two halves, whose scales are alike)
        constexpr int kSteps = G == 0 ? 1 : 2;
#pragma unroll
        for (int j0 = 0; j0 < 4; j0 += kSteps) {
            __builtin_amdgcn_sched_barrier(0);
            quad b[RT][kSteps];
            float by[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                by[i] = s[i].scale(j0);
#pragma unroll
                for (int e = 0; e < kSteps; ++e) b[i][e] = values8(MT{}, w[i][j0 + e], s[i].template offset<MT>(p, j0 + e), exponent);
            }
            // a vector tile's operands are read while the one before is multiplied, whose
            // sums are scaled while the next one is
            struct Tile {
                quad v[kSteps][PARTS];
            } v[2];
            f32x4 d[2][RT];
            const auto read = [&](int n, Tile& to) {
#pragma unroll
                for (int e = 0; e < kSteps; ++e)
#pragma unroll
                    for (int a = 0; a < PARTS; ++a)
                        to.v[e][a] = *reinterpret_cast<const quad*>(stage + a * kPart + n * 4096 +
                                                                    16 * ((4 * (j0 + e) + g) ^ r));
            };
            read(0, v[0]);
#pragma unroll
            for (int n = 0; n <= NT; ++n) {
                __builtin_amdgcn_sched_barrier(0);
                if (n + 1 < NT) read(n + 1, v[(n + 1) & 1]);
                if (n < NT) {
#pragma unroll
                    for (int e = 0; e < kSteps; ++e)
#pragma unroll
                        for (int a = 0; a < PARTS; ++a)
#pragma unroll
                            for (int i = 0; i < RT; ++i) {
                                if (e + a == 0) d[n & 1][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                                d[n & 1][i] = gemvdev::mma_16x16x32(MT{}, v[n & 1].v[e][a], b[i][e], d[n & 1][i]);
                            }
                }
                if (n > 0)
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[i][n - 1][e] = __builtin_fmaf(d[(n - 1) & 1][i][e], by[i], acc[i][n - 1][e]);
                        // (here, and not where the chunk ends: the sums would all wait in registers)
                        asm volatile("" : "+v"(acc[i][n - 1]));
                    }
                if (n > 0 && n < NT) {
                    constexpr int kProducts = RT * kSteps * PARTS, kEach = (4 * RT + kProducts - 1) / kProducts;
#pragma unroll
                    for (int i = 0; i < kProducts; ++i) {
                        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                        __builtin_amdgcn_sched_group_barrier(0x002, kEach, 0);
                    }
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        if (c + 1 < chunks) {
            if (c + 1 >= whole) fetch_end(c + 1);
            put_x(c + 1);
        }
        __syncthreads();
    }
    with_type(p, [&](auto type) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int row = row0 + (wave * RT + i) * 16 + r;
            if (row >= p.M) continue;
            const float add = p.bias ? p.bias[row] : 0.0f;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = t0 + 16 * n + 4 * g + e;
                    if (t < p.T) put<decltype(type)>(p, t * p.ldy + row, acc[i][n][e] + add);
                }
        }
    });
}

// ---------------------------------------------------------------------------
// very many vectors: X straight into LDS
//
// As above, but a wavefront takes 16·RT rows with RT = 4, so that what it reads of X
// from LDS serves twice as many products, and X and W go to LDS without passing
// registers, which hold the sums (whole chunks and aligned pieces only).  X then lies
// there in its own order, and the weights come out in that.  A row's scale and
// zero are loaded by one lane and passed to the four that want them.
//
// Two workgroups of four wavefronts share a compute unit, each with its own
// barriers: while one widens, the other multiplies (one workgroup of eight, whose
// wavefronts all wait for the slowest at each chunk: 322 us and 319, with a third fewer
// wavefront cycles spent waiting).  X's two stages and the one of W, which is in
// registers before the next is brought, are 80 KiB, half of a unit's LDS.
//
// 2000 x 14336 x 4096, groups of 64: 284 us, 827 TFLOP/s (the library's product of
// bf16 weights, with nothing to widen or scale: 202).  The vector ALUs issue 5.4 instructions
// to a product (2.4 widen, 2 scale), 66 % of the issue slots and 41 % of the matrix
// cores' cycles are taken, and the clock falls as either rises: 2.06 GHz here, 1.97 with 112
// vectors to a tile, whose rounds come out even.
//
// With groups of 128 a chunk has one scale, and the order in which its columns are
// taken is free: step j takes columns 32·g + 8·j .. +7 from the lanes' group g,
// those that the lane has loaded.
// ---------------------------------------------------------------------------

// Eight columns in their order.  fp16: a value between zero bytes is q·2^-24, and
// times 2^15 less zero·2^-9 all exact: the weights in units of 2^9, which the scale
// takes (kUnit).
template <class MT>
constexpr float kUnit = 1.0f;
template <>
constexpr float kUnit<TF16> = 512.0f;
__device__ __forceinline__ uint32_t ordered_offset_of(TF16, uint32_t zero) {
    const _Float16 z = (_Float16)((float)zero * -0x1p-9f);
    return __builtin_bit_cast(uint32_t, f16x2{z, z});
}
__device__ __forceinline__ float ordered_offset_of(TBF16, uint32_t zero) { return offset_of(TBF16{}, zero); }
__device__ __forceinline__ quad ordered8(TF16, uint32_t w, uint32_t offset, uint32_t) {
    const uint32_t even = w & 0x0f0f0f0fu, odd = w >> 4 & 0x0f0f0f0fu;
    const f16x2 by{(_Float16)0x1p15f, (_Float16)0x1p15f};
    quad v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t pair = __builtin_amdgcn_perm(odd, even, 0x0c040c00u + 0x00010001u * i);
        v[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(f16x2, pair), by,
                                                                      __builtin_bit_cast(f16x2, offset)));
    }
    return v;
}
__device__ __forceinline__ quad ordered8(TBF16, uint32_t w, float offset, uint32_t exponent) {
    uint32_t a[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t p = pair_of(w, i, exponent);
        a[i] = __builtin_bit_cast(uint32_t, half_minus<0>(p, offset));
        a[i + 4] = __builtin_bit_cast(uint32_t, half_minus<1>(p, offset));
    }
    quad v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __builtin_amdgcn_perm(a[2 * i + 1], a[2 * i], 0x07060302u);
    return v;
}

template <class T, int G, int RT, int NT, int W>
__global__ __launch_bounds__(W * 64, 2) void q4_wide_kernel(Product p, int row_tiles) {
    using R = RawScales<T, G, 1>;
    constexpr int BN = 16 * NT, BM = 16 * RT * W, kStage = BN * 256;
    constexpr int kLoads = BN * 16 / (W * 64);  // of X, for each wavefront and chunk
    static_assert(BN * 16 % (W * 64) == 0 && RT == 4, "whole loads, and a lane for each row of a wavefront");
    extern __shared__ __align__(16) uint8_t lds[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int r = lane & 15, g = lane >> 4;
    const int tiles = gridDim.x, per = tiles / 8, id = blockIdx.x;
    const int tile = id < per * 8 ? id % 8 * per + id / 8 : id;
    const int token_tiles = tiles / row_tiles;
    const int row0 = tile / token_tiles * BM, t0 = tile % token_tiles * BN;
    const int chunks = p.K / kChunk;
    const int64_t first_row = row0 + wave * RT * 16 < p.M ? row0 + wave * RT * 16 : p.M - 1;
    const int left = p.M - 1 - (int)first_row;
    const uint32_t own = lane < left ? lane : left;
    const uint32_t s_at = own * (uint32_t)p.lds * T::bytes, z_at = own * (uint32_t)p.ldz;
    const uint8_t* q0 = p.Q + first_row * p.ldq;
    const uint8_t* s0 = static_cast<const uint8_t*>(p.scale) + first_row * p.lds * T::bytes;
    const uint8_t* z0 = p.zero + first_row * p.ldz;
    const uint8_t* x0 = static_cast<const uint8_t*>(p.X) + t0 * p.ldx * T::bytes;
    // load i of a wavefront brings four vectors; a lane's slot is lane % 16, the piece
    // there the slot ^ the vector's last four bits.  Of W it brings 16 rows of four
    // pieces.
    uint32_t x_at[kLoads], q_at[RT];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int t = (i * W + wave) * 4 + g, last = p.T - 1 - t0;
        x_at[i] = (uint32_t)(t < last ? t : last) * (uint32_t)(p.ldx * T::bytes) + 16 * (r ^ (t & 15));
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int n = 16 * i + (lane >> 2);
        q_at[i] = (uint32_t)(n < left ? n : left) * (uint32_t)p.ldq + 16 * ((lane ^ (lane >> 3)) & 3);
    }
    const uint32_t lds_at = (uint32_t)(uintptr_t)lds;
    const uint32_t own_rows = 2 * kStage + wave * (RT * 1024);
    R then;
    const auto fetch_x = [&](int c) {
        const uint8_t* xc = x0 + (int64_t)c * (kChunk * T::bytes);
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            fp8dev::lds_load16(xc, x_at[i], lds_at + (c & 1) * kStage + (i * W + wave) * 1024);
    };
    const auto fetch_w = [&](int c) {
        const uint8_t* qc = q0 + (int64_t)c * (kChunk / 2);
#pragma unroll
        for (int i = 0; i < RT; ++i) fp8dev::lds_load16(qc, q_at[i], lds_at + own_rows + i * 1024);
        const int g0 = 4 * c >> G;
        load_words<R::N * T::bytes>(scalar_here(s0 + (int64_t)g0 * T::bytes) + offset_here(s_at), then.s);
        load_words<R::N>(scalar_here(z0 + g0) + offset_here(z_at), then.z);
    };
    f32x4 acc[RT][NT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[i][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    fetch_x(0);
    fetch_w(0);
    const uint32_t exponent = exponent_of_1024();
    constexpr int kSteps = G == 0 ? 1 : 2;
    for (int c = 0; c < chunks; ++c) {
        const uint8_t* stage = lds + (c & 1) * kStage;
        fp8dev::wait_loads<0>();
        quad w[RT];
        R s[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            w[i] = *reinterpret_cast<const quad*>(lds + own_rows + i * 1024 + r * 64 + 16 * (g ^ (r >> 1 & 3)));
            const int from = 4 * (16 * i + r);
#pragma unroll
            for (int e = 0; e < R::kWords; ++e) s[i].s[e] = __builtin_amdgcn_ds_bpermute(from, then.s[e]);
#pragma unroll
            for (int e = 0; e < R::kZeros; ++e) s[i].z[e] = __builtin_amdgcn_ds_bpermute(from, then.z[e]);
        }
        fp8dev::change_over();
        if (c + 1 < chunks) fetch_x(c + 1);
        stage += r * 256;
        if constexpr (G < 2) {
#pragma unroll
            for (int i = 0; i < RT; ++i) w[i] = transposed(w[i]);
        }
#pragma unroll
        for (int j0 = 0; j0 < 4; j0 += kSteps) {
            __builtin_amdgcn_sched_barrier(0);
            quad b[RT][kSteps];
            float by[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                by[i] = s[i].scale(j0) * kUnit<T>;
                const auto offset = ordered_offset_of(T{}, s[i].zero(p, j0));
#pragma unroll
                for (int e = 0; e < kSteps; ++e) b[i][e] = ordered8(T{}, w[i][j0 + e], offset, exponent);
            }
            if (j0 == 0 && c + 1 < chunks) {  // (the rows are in registers)
                __builtin_amdgcn_sched_barrier(0);
                fp8dev::wait_lds();
                fetch_w(c + 1);
            }
            quad v[2][kSteps];
            f32x4 d[2][RT];
            const auto read = [&](int n, quad (&to)[kSteps]) {
#pragma unroll
                for (int e = 0; e < kSteps; ++e) {
                    const int piece = G == 2 ? 4 * g + j0 + e : 4 * (j0 + e) + g;
                    to[e] = *reinterpret_cast<const quad*>(stage + n * 4096 + 16 * (piece ^ r));
                }
            };
            read(0, v[0]);
#pragma unroll
            for (int n = 0; n <= NT; ++n) {
                __builtin_amdgcn_sched_barrier(0);
                if (n + 1 < NT) read(n + 1, v[(n + 1) & 1]);
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    if (n > 0) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[i][n - 1][e] = __builtin_fmaf(d[(n - 1) & 1][i][e], by[i], acc[i][n - 1][e]);
                        asm volatile("" : "+v"(acc[i][n - 1]));
                    }
                    if (n < NT) {
                        d[n & 1][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int e = 0; e < kSteps; ++e)
                            d[n & 1][i] = gemvdev::mma_16x16x32(T{}, v[n & 1][e], b[i][e], d[n & 1][i]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    fp8dev::wait_loads<0>();
    with_type(p, [&](auto type) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int row = row0 + (wave * RT + i) * 16 + r;
            if (row >= p.M) continue;
            const float add = p.bias ? p.bias[row] : 0.0f;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = t0 + 16 * n + 4 * g + e;
                    if (t < p.T) put<decltype(type)>(p, t * p.ldy + row, acc[i][n][e] + add);
                }
        }
    });
}

}  // namespace q4dev
