// Kernels of the paged 8-bit key/value cache: the append and the attention
// over it.
//
// The cache.  A page holds page_size tokens of every head, in blocks of 16
// tokens of one head.  K keeps a token's dim values together, [token][dim];
// V keeps the 16 tokens of one dim together, [block][dim][16 tokens]: both
// products of the attention then read the bytes of a matrix-core operand with
// 16-byte loads, straight from memory to registers (below).  A block has one
// fp32 scale for its keys and one for its values.
#pragma once

#include "fp8_device.hpp"
#include "kv_plan.hpp"

namespace kvdev {

using fp8dev::f32x4;
using fp8dev::max_u32;
using fp8dev::quad;
using fp8dev::quad_any;
using fp8dev::TBF16;
using fp8dev::TF16;
using fp8dev::TF32;
using fp8dev::widen;

using kvplan::kBlock;

// The two 8-bit formats: the largest magnitude that a scale maps to.
struct Int8 {
    static constexpr float qmax = 127.0f;
};
struct E4m3 {
    static constexpr float qmax = 448.0f;
};

struct Cache {
    uint8_t* k;
    uint8_t* v;
    float* k_scale;
    float* v_scale;
    int heads;
    int pages;
    int per_page_log2;  // blocks of a page, as a power of two
};

// A batch's layout: sequence b has seq_lens[b] tokens, of which the last
// starts[b+1] - starts[b] (one, where starts is NULL) are the rows of this
// call; its blocks lie in the pages of row b of the table.
struct Batch {
    const int* table;
    int64_t table_pitch;
    int table_width;
    const int* lens;
    const int* starts;
    int count;
    int total;  // rows of the call
};

__device__ __forceinline__ int start_of(const Batch& q, int b) {
    return q.starts ? q.starts[b] : b;
}

// The page that holds a block of sequence b, or -1 where the table has none
// (past its width, or an entry that is no page).
__device__ __forceinline__ int page_of(const Batch& q, const Cache& c, int b, int block) {
    const int i = block >> c.per_page_log2;
    if (i >= q.table_width) return -1;
    const int page = q.table[(int64_t)b * q.table_pitch + i];
    return page >= 0 && page < c.pages ? page : -1;
}

// Index of a block of a head among all blocks of the cache.
__device__ __forceinline__ int64_t block_index(const Cache& c, int page, int head, int block) {
    return (((int64_t)page * c.heads + head) << c.per_page_log2) +
           (block & ((1 << c.per_page_log2) - 1));
}

// The item that a flattened index names: each sequence owns
// floor(starts[b+1]·n/d) - floor(starts[b]·n/d) + extra places from
// floor(starts[b]·n/d) + extra·b on, enough for what it needs whatever the
// starts, so the grid needs no count from the device.
__device__ __forceinline__ int64_t first_place(const Batch& q, int b, int64_t n, int64_t d, int extra) {
    return (int64_t)start_of(q, b) * n / d + (int64_t)extra * b;
}
// Every lane of the wavefront takes part: the last 64 candidates are looked at
// side by side.
__device__ __forceinline__ int sequence_of(const Batch& q, int64_t place, int64_t n, int64_t d, int extra) {
    int lo = 0, hi = q.count;  // the last b in [lo, hi) whose first place is at most `place`
    while (hi - lo > 64) {
        const int mid = (lo + hi) >> 1;
        if (first_place(q, mid, n, d, extra) <= place)
            lo = mid;
        else
            hi = mid;
    }
    const int b = lo + (int)(threadIdx.x & 63);
    const uint64_t before = __ballot(b < hi && first_place(q, b < hi ? b : lo, n, d, extra) <= place);
    const int found = lo + __popcll(before) - 1;
    return found < lo ? lo : found;
}

// ---------------------------------------------------------------------------
// append
//
// The scale of a block is the smallest power of two s >= 2^-126 with
// amax <= qmax·s over its new values, or the scale of the tokens that stay
// where that is larger.  Where it grows over the tokens that stay, they are
// rounded again; by powers of two that is exact in e4m3 (but for subnormals).
// ---------------------------------------------------------------------------

// Smallest power of two s with amax <= qmax·s, from amax's bits; NaN for an
// infinity or NaN.  qmax is 127 = (127/64)·2^6 or 448 = 1.75·2^8: with amax =
// f·2^e, 1 <= f < 2, s is 2^(e-6) or 2^(e-8), or twice that where f is above.
template <class F>
__device__ __forceinline__ float block_scale(uint32_t amax) {
    if (amax >= 0x7f800000u) return __builtin_nanf("");
    constexpr bool e4m3 = F::qmax == 448.0f;
    constexpr int shift = e4m3 ? 8 : 6;
    constexpr uint32_t limit = e4m3 ? 0x600000u : 0x7e0000u;  // mantissa bits of 1.75 and of 127/64
    int e = (int)(amax >> 23) - shift + ((amax & 0x7fffffu) > limit ? 1 : 0);
    if (e < 1) e = 1;
    return __builtin_bit_cast(float, (uint32_t)e << 23);
}

// A value over its scale, rounded to the nearest that 8 bits hold.
__device__ __forceinline__ uint32_t round8(Int8, float v) {
    v = __builtin_rintf(fminf(fmaxf(v, -127.0f), 127.0f));
    return (uint32_t)(int)v & 0xffu;
}
__device__ __forceinline__ uint32_t round8(E4m3, float v) {
    v = fminf(fmaxf(v, -448.0f), 448.0f);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false) & 0xffu;
}
// 16 values over their scale, in the order of their bytes.
template <class F>
__device__ __forceinline__ quad pack16(F, const float (&x)[16], float inv) {
    quad w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = fminf(fmaxf(x[4 * i + e] * inv, -F::qmax), F::qmax);
        if constexpr (F::qmax == 448.0f) {
            w[i] = fp8dev::to_e4m3x4(v[0], v[1], v[2], v[3]);
        } else {
            w[i] = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[i] |= ((uint32_t)(int)__builtin_rintf(v[e]) & 0xffu) << (8 * e);
        }
    }
    return w;
}
__device__ __forceinline__ float value8(Int8, uint32_t byte) { return (float)(int)(int8_t)byte; }
__device__ __forceinline__ float value8(E4m3, uint32_t byte) {
    return __builtin_amdgcn_cvt_f32_fp8((int)byte, 0);
}

// N consecutive elements from p on, widened to fp32.
template <class D, int N>
__device__ __forceinline__ void load_run(const typename D::storage* p, float (&v)[N]) {
    using S = typename D::storage;
    struct __attribute__((packed, aligned(D::bytes))) Run {
        S v[N];
    };
    const Run r = *reinterpret_cast<const Run*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = widen(D{}, r.v[i]);
}

// The lowest n of 16 bits, n clamped to 0..16.
__device__ __forceinline__ uint32_t low_bits(int64_t n) {
    return n <= 0 ? 0u : n >= 16 ? 0xffffu : (1u << (int)n) - 1;
}

// One wavefront per block of one head's keys or values.  16-byte piece p of
// the block is 16 dims of a token (K) or the 16 tokens of a dim (V); a lane
// holds K's pieces lane, lane + 64, ... and V's pieces of DIM / 64 neighbouring
// dims, so that both read runs of elements.  The values are asked for before
// the page, which they do not need.  Bound by latency for single tokens (64
// sequences, 8 heads of 128: 5.8 us, of which the bytes are 0.14) and by that and memory
// for prompts (14.4 us against 9.9 at a large copy's rate, the vector ALUs busy for a
// third of it); one wavefront to a
// workgroup, because blocks share nothing.
template <class D, class F, int DIM>
__global__ __launch_bounds__(64) void kv_append_kernel(Cache c, Batch q,
                                                       const typename D::storage* K, int64_t ldk,
                                                       const typename D::storage* V, int64_t ldv) {
    constexpr int kPieces = DIM / 64;  // of a lane: kBlock·DIM / 16 / 64
    const int lane = threadIdx.x;
    const int head = (int)blockIdx.y;
    const bool values = blockIdx.z != 0;
    const int64_t place = blockIdx.x;
    int b;
    int64_t ahead;  // blocks of the sequence's new tokens before this one
    if (q.starts == nullptr) {
        b = (int)place;
        ahead = 0;
    } else {
        b = sequence_of(q, place, 1, kBlock, 2);
        ahead = place - first_place(q, b, 1, kBlock, 2);
    }
    const int start = start_of(q, b), stop = start_of(q, b + 1);
    const int len = q.lens[b];
    const int64_t first = (int64_t)len - ((int64_t)stop - start);  // position of the first new token
    const int64_t at = ((first > 0 ? first : 0) / kBlock + ahead) * kBlock;  // ... of the block's token 0
    if (ahead < 0 || at >= len || stop <= start) return;
    const int64_t row0 = start + at - first;                       // its row
    // tokens of the block that stay, and those that this call brings
    const uint32_t stay = low_bits(first - at);
    const uint32_t fresh = low_bits(len - at) & ~stay & low_bits(q.total - row0) & ~low_bits(-row0);
    if (fresh == 0) return;
    float x[kPieces][16];
    if (values) {
        const typename D::storage* p = V + row0 * ldv + (int64_t)head * DIM + lane * kPieces;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float run[kPieces] = {};
            if (fresh >> i & 1) load_run<D, kPieces>(p + i * ldv, run);
#pragma unroll
            for (int j = 0; j < kPieces; ++j) x[j][i] = run[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const int piece = lane + 64 * j, token = piece / (DIM / 16), dim = piece % (DIM / 16) * 16;
#pragma unroll
            for (int i = 0; i < 16; ++i) x[j][i] = 0.0f;
            if (fresh >> token & 1) load_run<D, 16>(K + (row0 + token) * ldk + (int64_t)head * DIM + dim, x[j]);
        }
    }
    const int block = (int)(at / kBlock);
    const int page = page_of(q, c, b, block);
    if (page < 0) return;
    const int64_t index = block_index(c, page, head, block);
    uint8_t* held = (values ? c.v : c.k) + index * (kBlock * DIM);
    float* scale = (values ? c.v_scale : c.k_scale) + index;
    const float old = stay != 0 ? *scale : 0.0f;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kPieces; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) m = max_u32(m, fp8dev::magnitude(x[j][i]));
    const float need = block_scale<F>(fp8dev::wave_max(m));
    float s = need, ratio = 1.0f;
    if (stay != 0) {
        if (!(old <= need)) s = old;  // the larger, and NaN once either is
        if (need != need) s = need;
        ratio = old / s;
    }
    const float inv = 1.0f / s;
    const bool bad = s != s;  // the bytes of a block with no scale are zero
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        const int piece = values ? lane * kPieces + j : lane + 64 * j;
        const int token = piece / (DIM / 16);
        const uint32_t put = values ? fresh : (fresh >> token & 1 ? 0xffffu : 0u);
        const uint32_t keep = values ? stay : (stay >> token & 1 ? 0xffffu : 0u);
        if (put == 0 && (keep == 0 || ratio == 1.0f)) continue;
        quad* to = reinterpret_cast<quad*>(held) + piece;
        if (put == 0xffffu && !bad) {
            *to = pack16(F{}, x[j], inv);
            continue;
        }
        quad w = put == 0xffffu ? quad{0u, 0u, 0u, 0u} : *to;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t was = w[i >> 2] >> (8 * (i & 3)) & 0xffu;
            uint32_t now = was;
            if (put >> i & 1)
                now = bad ? 0u : round8(F{}, x[j][i] * inv);
            else if ((keep >> i & 1) && ratio != 1.0f)
                now = bad ? 0u : round8(F{}, value8(F{}, was) * ratio);
            w[i >> 2] = (w[i >> 2] & ~(0xffu << (8 * (i & 3)))) | now << (8 * (i & 3));
        }
        *to = w;
    }
    if (lane == 0) *scale = s;
}

// ---------------------------------------------------------------------------
// attention
//
//   O[i,h] = Σ_j softmax_j(c·Q[i,h]·K[j]) V[j],   j visible to row i
//
// One pass over the tokens with the running maximum m and sum l of the
// softmax.  A wavefront takes 16·RT rows (a row is a token's query head; the
// query heads that share a K/V head are neighbouring rows, so each byte of
// the cache is read once for all of them) and walks chunks of 64 tokens, four
// cache blocks.
//
// Both products are taken transposed, S^T = K·Q^T and O^T = V^T·P^T, with
// 16×16×32 matrix-core steps, so that a lane holds one query row (lane % 16)
// throughout: of S^T and P^T the 16 tokens of block lane / 16, of O^T four
// dims of each 16.  The result of the first product is laid out exactly as
// the operand of the second, because the order in which a step takes its
// tokens is free: row 4·g + i of the t-th K tile is token 4·t + i of block g,
// and a lane's 16-byte piece of V is the 16 tokens of one dim of block g.
// Nothing passes through LDS or between lanes but the row maximum (once a
// chunk) and the row sum (once at the end).
//
// Single tokens are bound by memory: one sequence of 131071 tokens 50.7 us with
// its join (5.3 TB/s), 64 sequences of up to 8192 115 us (4.8 TB/s), 4 with a
// window of 512 10.6 us, which is latency.  Prompts are bound by the vector ALUs,
// which widen K and V for every 32 rows and take 7 to 8 instructions to each
// matrix-core one: 2160 tokens over contexts of up to 4096, 32 heads, 161 to 164
// us, 655 TFLOP/s.  (Wider row tiles would share the widening, but 32 rows of dim
// 128 fill 237 registers as it is.)
//
// K and V are widened exactly (e4m3 and int8 both fit fp16 and bf16); a
// block's scales are one number a lane: K's multiplies S in fp32, V's
// multiplies P.  K meets Q in Q's type, P meets V in fp16 (11 bits, where bf16
// keeps 8), whatever Q is: a term, P times its block's V scale, is held in a
// unit of its row, a power of two that follows the row's largest term: at most 2^-6
// of it when it is set, and set anew once a term passes 2^14 units.  So terms keep
// fp16's 11 bits down to 2^-20 of the row's largest, and below that are within half of fp16's
// smallest step, 2^-31 of it (the sum l counts P in fp32).  The unit follows the
// terms and not the V scales alone: a block with a large scale and no weight
// would push the terms that matter out of fp16's range.
// ---------------------------------------------------------------------------

using fp8dev::bf16x2;
using fp8dev::f16x2;

__device__ __forceinline__ uint32_t pack(TF16, float a, float b) {
    const f16x2 p{(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, p);
}
__device__ __forceinline__ uint32_t pack(TBF16, float a, float b) {
    const bf16x2 p{(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, p);
}

// Two bytes of a word (the low or the high pair) widened to a pair of T.
template <bool HIGH>
__device__ __forceinline__ uint32_t widen_pair(E4m3, TF16, uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HIGH));
}
template <bool HIGH>
__device__ __forceinline__ uint32_t widen_pair(E4m3, TBF16, uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HIGH));
}
template <bool HIGH, class T>
__device__ __forceinline__ uint32_t widen_pair(Int8, T, uint32_t w) {
    return pack(T{}, gemvdev::q8_at(w, HIGH ? 2 : 0), gemvdev::q8_at(w, HIGH ? 3 : 1));
}
// 8 bytes to the 8 values of a matrix-core operand.
template <class F, class T>
__device__ __forceinline__ quad widen8(uint32_t lo, uint32_t hi) {
    return quad{widen_pair<false>(F{}, T{}, lo), widen_pair<true>(F{}, T{}, lo),
                widen_pair<false>(F{}, T{}, hi), widen_pair<true>(F{}, T{}, hi)};
}

// The bytes of a piece of V whose tokens are among the block's first n.
__device__ __forceinline__ quad first_bytes(quad v, int n) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int k = n - 4 * w;
        v[w] = k >= 4 ? v[w] : k <= 0 ? 0u : v[w] & ((1u << (8 * k)) - 1);
    }
    return v;
}

__device__ __forceinline__ float max_of_groups(float v) {  // over the four 16-lane groups
    const unsigned u = __builtin_bit_cast(unsigned, v);
    auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = fmaxf(gemvdev::f32_of(r[0]), gemvdev::f32_of(r[1]));
    const unsigned w = __builtin_bit_cast(unsigned, v);
    r = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    return fmaxf(gemvdev::f32_of(r[0]), gemvdev::f32_of(r[1]));
}
__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, gemvdev::dpp<gemvdev::kDppSwapAdjacent>(v));
    v = fmaxf(v, gemvdev::dpp<gemvdev::kDppSwapPairs>(v));
    v = fmaxf(v, gemvdev::dpp<gemvdev::kDppHalfRowMirror>(v));
    v = fmaxf(v, gemvdev::dpp<gemvdev::kDppRowMirror>(v));
    return max_of_groups(v);
}
__device__ __forceinline__ float sum_of_groups(float v) {
    return gemvdev::half_pair_sum32(gemvdev::row_pair_sum16(v));
}

// 16 bytes of the cache; ONCE: as a rule nothing reads them again in this call
// (wavefronts share their rows, and there are seldom more of them to a K/V head than
// one workgroup takes), so they go past the caches (nontemporal; 7 % of one long
// sequence's time).
template <bool ONCE>
__device__ __forceinline__ quad load_once(const uint8_t* p) {
    if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const quad*>(p));
    return *reinterpret_cast<const quad*>(p);
}

// A row that has seen nothing keeps its base at -inf; its exponents are taken
// against 0.
__device__ __forceinline__ float finite_base(float m) { return m == -__builtin_inff() ? 0.0f : m; }
// A row's unit in its largest term when it is set, and the largest term in that
// unit that it is kept for (fp16 ends at 2^16; the factor of 4 is for terms past
// 2^127, which a caller's scales can make).
constexpr float kUnitOfLargest = 0x1p-6f, kMostUnits = 0x1p14f;
// The power of two at or below v, 2^-126 at least, and the reciprocal of one up to 2^126.
__device__ __forceinline__ float unit_of(float v) {
    return gemvdev::f32_of(__builtin_bit_cast(uint32_t, fmaxf(v, fp8dev::kSmallestScale)) & 0x7f800000u);
}
__device__ __forceinline__ float inverse(float unit) {
    return gemvdev::f32_of(0x7f000000u - __builtin_bit_cast(uint32_t, unit));
}

using kvplan::kChunk;
using kvplan::kMaxSplits;
using kvplan::kOwnWaves;
using kvplan::kShareWaves;
using kvplan::Span;
template <int WS>
constexpr int kWavesOf = WS == 1 ? kOwnWaves : WS;

// The first n of a block's 16 tokens, as bits.
__device__ __forceinline__ uint32_t first_bits(int n) {
    n = n < 0 ? 0 : n > kBlock ? kBlock : n;
    return (1u << n) - 1;
}

struct Attend {
    Cache cache;
    Batch batch;
    const uint16_t* Q;
    int64_t ldq;
    uint16_t* O;
    int64_t ldo;
    int group;          // query heads that share a K/V head
    float scale;        // |softmax scale| · log2(e)
    uint32_t q_sign;    // sign bits of two values of Q, set where the scale is negative
    int window, sinks;  // window 0: none
    int capacity;       // tokens that a row of the table can hold
    int splits;         // workgroups that share a row tile's tokens, ...
    int split_chunks;   // ... each so many chunks of them; splits > 1:
    int rows;           // rows of a place that can be there
    float* partial;     // see partial_at
    int shared;         // chunks that the batch shares and another launch takes (0: none):
                        // then the results are partial ones, whatever the splits
    float slack;        // of the rows over shared tokens, see slack_of
};

// How far a row's largest score, as a power of two, may pass the base of its
// exponents before that follows: prompts, whose vector ALUs are the bound, save
// the rescaling (2160 tokens over up to 4096, 164 us against 175 with 0; 942 over 4000
// shared ones 166 and 175); single
// tokens take the same time with 0 (1 x 131071 51.3 and 51.5), and the largest
// weight is then 1, which fp16 holds exactly (4 with a window of 512, fp16
// results: error 2.15e-4 against 2.21e-4, of which the result's rounding is 2.06e-4).
// Shared tokens are weighed as the call without them would weigh them.
constexpr float kPromptSlack = 8.0f;
template <int WS, bool SHARED>
__device__ __forceinline__ float slack_of(const Attend& p) {
    return SHARED ? p.slack : WS == 1 ? kPromptSlack : 0.0f;
}

// What a row tile sees of the sequence's tokens.
__device__ __forceinline__ Span span_of(const Attend& p, int min_pos, int max_pos, int len) {
    return kvplan::span_of(p.window, p.sinks, p.capacity, min_pos, max_pos, len, p.shared);
}

// Rows of a sequence that a workgroup takes: from row r0 on.
struct Tile {
    int b;       // the sequence
    int start;   // its first row of the call
    int first;   // the position of that row's token
    int len;     // tokens of the sequence
    int rows;    // its rows times the query heads of a K/V head
    int r0;
};
template <int R>
__device__ __forceinline__ bool tile_of(const Attend& p, int64_t place, Tile& t) {
    const Batch& q = p.batch;
    int64_t r0;
    bool from_last = false;
    if (q.starts == nullptr) {  // one token each: so many places for its heads
        const int each = (p.group + R - 1) / R;
        t.b = (int)(place / each);
        r0 = (place - (int64_t)t.b * each) * R;
    } else {
        t.b = sequence_of(q, place, p.group, R, 1);
        r0 = (place - first_place(q, t.b, p.group, R, 1)) * R;
        from_last = true;
    }
    t.start = start_of(q, t.b);
    const int stop = start_of(q, t.b + 1);
    // rows outside the call's are not there, whatever the starts say
    if (t.start < 0 || stop > q.total || stop <= t.start) return false;
    t.len = q.lens[t.b];
    t.first = (int)((int64_t)t.len - (stop - t.start));
    t.rows = (stop - t.start) * p.group;
    // a prompt's last rows see the most tokens: those workgroups start first
    // (two 2048-token prompts 172 us in ascending order, 142 in this one)
    if (from_last) r0 = (t.rows - 1) / R * R - r0;
    t.r0 = (int)r0;
    return r0 >= 0 && r0 < t.rows;
}

// Where all sequences share their first tokens: the rows of the whole batch, over
// the first sequence's pages.
template <int R>
__device__ __forceinline__ bool shared_tile_of(const Attend& p, int64_t place, Tile& t) {
    const Batch& q = p.batch;
    int rows = start_of(q, q.count);
    rows = rows < q.total ? rows : q.total;
    t.b = t.start = t.first = 0;
    t.len = p.capacity;
    t.rows = rows * p.group;
    const int64_t r0 = place * R;
    t.r0 = (int)r0;
    return r0 < t.rows;
}
// The position of a row of the call in its sequence, or -1 where it has none.
__device__ __forceinline__ int position_of(const Batch& q, int row) {
    int lo = row, hi = row + 1;
    if (q.starts != nullptr) {
        lo = 0;
        hi = q.count;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (q.starts[mid] <= row)
                lo = mid;
            else
                hi = mid;
        }
    }
    const int start = start_of(q, lo), stop = start_of(q, lo + 1);
    if (row < start || row >= stop || stop > q.total) return -1;
    const int64_t pos = (int64_t)q.lens[lo] - (stop - row);
    return pos < 0 ? -1 : (int)pos;
}
__device__ __forceinline__ int wave_max_int(int v) {  // of numbers from -1 on
    return (int)fp8dev::wave_max((uint32_t)(v + 1)) - 1;
}

// splits > 1: each split of a place and head leaves p.rows rows, each as the result
// over its own tokens, and their m and l: first all (m, l), then all rows.
struct Partial {
    float* ml;
    float* rows;
};
template <int DIM>
__device__ __forceinline__ Partial partial_at(const Attend& p, int64_t places, int64_t part) {
    const int64_t rows = places * p.cache.heads * p.splits * p.rows;
    return Partial{p.partial + part * p.rows * 2, p.partial + kvplan::stats_floats(rows) + part * p.rows * DIM};
}

// WS > 1: the workgroup's wavefronts take the chunks of one row tile in turn
// and join in LDS.  WS = 1: each wavefront has a row tile of its own.  SHARED: the
// rows of all sequences over the p.capacity tokens that they share; the results
// are partial ones.
template <class T, class F, int DIM, int RT, int WS, bool SHARED>
__device__ __forceinline__ void attend_part(const Attend& p, int64_t places, int64_t workgroup) {
    constexpr int kRows = 16 * RT;                              // rows of a wavefront
    constexpr int kGroupRows = WS == 1 ? kOwnWaves * kRows : kRows;
    constexpr int kSteps = DIM / 32;                            // K·Q^T steps
    constexpr int kTiles = DIM / 16;                            // 16-dim tiles of O^T
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int n = lane & 15, g = lane >> 4;
    const Cache& c = p.cache;
    // heads fastest: neighbouring workgroups, which go to different chiplets,
    // share no K or V; then the splits
    int64_t at = workgroup;
    const int head = (int)(at % c.heads);
    at /= c.heads;
    // (the places of shared tokens before their splits: they read the same bytes)
    const int64_t outer = SHARED ? places : p.splits;
    const int split = (int)(SHARED ? at / outer : at % outer);
    const int64_t place = SHARED ? at % outer : at / outer;
    Tile t;
    if (!(SHARED ? shared_tile_of<kGroupRows>(p, place, t) : tile_of<kGroupRows>(p, place, t))) return;
    const int r0 = t.r0 + (WS == 1 ? wave * kRows : 0);
    if (WS == 1 && r0 >= t.rows) return;
    const int last = (r0 + kRows < t.rows ? r0 + kRows : t.rows) - 1;
    int min_pos = t.first + r0 / p.group, max_pos = t.first + last / p.group;
    int pos[RT];  // the lane's row of each 16: its position (-1: none)
    if constexpr (SHARED) {
        int most = -1, most_left = -1;  // 0x7fffffff less the position
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int r = r0 + 16 * i + n;
            pos[i] = r <= last ? position_of(p.batch, r / p.group) : -1;
            most = pos[i] > most ? pos[i] : most;
            const int left = pos[i] < 0 ? -1 : 0x7ffffffe - pos[i];
            most_left = left > most_left ? left : most_left;
        }
        max_pos = __builtin_amdgcn_readfirstlane(wave_max_int(most));
        min_pos = 0x7ffffffe - __builtin_amdgcn_readfirstlane(wave_max_int(most_left));
        min_pos = max_pos < 0 ? -1 : min_pos;
        // (what lies behind the last token that a row sees need not have been written: a
        // byte there may be NaN, which no weight of 0 takes away)
        t.len = max_pos + 1 < t.len ? max_pos + 1 : t.len;
    }
    const Span span = span_of(p, min_pos, max_pos, t.len);
    const int begin = p.splits == 1 ? 0 : split * p.split_chunks;
    int end = p.splits == 1 ? span.count() : begin + p.split_chunks;
    end = end < span.count() ? end : span.count();
    if (!SHARED && split > 0 && begin >= end) return;  // (the whole workgroup: the splits are cut for all its rows alike)

    // ... and its Q
    // (two tiles' Q does not fit the registers beside the rest: it stays in LDS)
    constexpr bool kQInLds = RT > 1;
    // (wavefronts that share their rows write the same)
    constexpr int kCopies = kQInLds && !SHARED ? kWavesOf<WS> : 1;
    __shared__ quad q_lds[kCopies][kQInLds ? RT : 1][kQInLds ? kSteps : 1][64];
    const int copy = kCopies > 1 ? wave : 0;
    int64_t row[RT];     // row of the call
    int qhead[RT];
    quad q[RT][kSteps];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int r = r0 + 16 * i + n;
        const int rr = r <= last ? r : last;
        const int token = rr / p.group;
        if (!SHARED) pos[i] = r <= last ? t.first + token : -1;
        row[i] = (int64_t)t.start + token;
        qhead[i] = head * p.group + (rr - token * p.group);
        const uint16_t* src = p.Q + row[i] * p.ldq + (int64_t)qhead[i] * DIM + 16 * g;
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
            q[i][s] = *reinterpret_cast<const quad_any*>(src + 64 * (s >> 1) + 8 * (s & 1)) ^ p.q_sign;
        if constexpr (kQInLds)  // read back by the lane that wrote it
#pragma unroll
            for (int s = 0; s < kSteps; ++s) q_lds[copy][i][s][lane] = q[i][s];
    }
    const auto q_of = [&](int i, int s) {
        if constexpr (kQInLds) return q_lds[copy][i][s][lane];
        return q[i][s];
    };

    f32x4 o[RT][kTiles];
    float m[RT], l[RT];
    // the unit of the row's terms, relative to the base m of its exponents: o is in it
    float unit[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        unit[i] = fp8dev::kSmallestScale;
        m[i] = -__builtin_inff();
        l[i] = 0.0f;
#pragma unroll
        for (int u = 0; u < kTiles; ++u) o[i][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // Of a chunk's four blocks, the lane reads K from block n / 4 and V from
    // block g.  A block's page is looked up two chunks ahead.  With one row
    // tile a chunk's bytes are loaded while the chunk before it is worked on,
    // into registers of their own (single tokens wait for memory, and a wave's 16
    // KiB in flight are what hides it); with two, or dim 256, there is room for one
    // chunk, and its K is loaded behind the first product of the chunk before, its V behind
    // the second.  (With eight wavefronts, which have few chunks each, the plain
    // step beats the pair: 12.2 us against 12.9 for 4 sequences with a window
    // of 512; it is half the code.)
    constexpr bool kAhead = RT == 1 && DIM <= 128 && WS <= 4;
    // The table's entries as they are: what they are worth is looked at when
    // they are used, so that the lookup never waits for the loads before it.
    struct Where {
        int kpage, vpage;
    };
    const int* table = p.batch.table + (int64_t)t.b * p.batch.table_pitch;
    auto entry_of = [&](int block) {
        const int i = block >> c.per_page_log2;
        return table[i < p.batch.table_width ? i : p.batch.table_width - 1];
    };
    auto look_up = [&](int it) {
        const int chunk = span.chunk(it);
        return Where{entry_of(4 * chunk + (n >> 2)), entry_of(4 * chunk + g)};
    };
    // the page in an entry for a block, or -1 where the block is not there
    auto page_in = [&](int entry, int block) {
        const bool there = (unsigned)entry < (unsigned)c.pages && block * kBlock < t.len &&
                           block >> c.per_page_log2 < p.batch.table_width;
        return there ? entry : -1;
    };
    struct Bytes {
        quad k[4][DIM / 64], v[kTiles];
        float kscale, vscale;
    };
    auto load_k = [&](int it, const Where& w, Bytes& to) {
        const int kb = 4 * span.chunk(it) + (n >> 2);
        const int page = page_in(w.kpage, kb);
        const uint8_t* kp = c.k + block_index(c, page < 0 ? 0 : page, head, kb) * (kBlock * DIM) +
                            (n & 3) * DIM + 16 * g;
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int h = 0; h < DIM / 64; ++h)
                to.k[tt][h] = load_once<(WS > 1 && !SHARED)>(kp + 4 * tt * DIM + 64 * h);
    };
    auto load_v = [&](int it, const Where& w, Bytes& to) {
        const int vb = 4 * span.chunk(it) + g;
        const int page = page_in(w.vpage, vb);
        const int64_t vi = block_index(c, page < 0 ? 0 : page, head, vb);
        to.kscale = c.k_scale[vi];
        to.vscale = c.v_scale[vi];
        const uint8_t* vp = c.v + vi * (kBlock * DIM) + n * kBlock;
#pragma unroll
        for (int u = 0; u < kTiles; ++u) to.v[u] = load_once<(WS > 1 && !SHARED)>(vp + 16 * u * kBlock);
    };

    int it = begin + (WS == 1 ? 0 : wave);
    Bytes first, second;
    Where now{-1, -1}, next{-1, -1};
    if (it < end) {
        now = look_up(it);
        load_k(it, now, first);
        load_v(it, now, first);
        if (it + WS < end) next = look_up(it + WS);
    }
    auto step = [&](Bytes& in, Bytes& ahead) {
        const bool more = it + WS < end;
        const Where then = next;
        if (kAhead && more) {
            load_k(it + WS, then, ahead);
            load_v(it + WS, then, ahead);
            if (it + 2 * WS < end) next = look_up(it + 2 * WS);
        }
        const int chunk = span.chunk(it);
        const int vb = 4 * chunk + g;
        // tokens of block g that are there
        const bool held = page_in(now.vpage, vb) >= 0;
        int there = held ? t.len - vb * kBlock : 0;
        there = there < 0 ? 0 : there > kBlock ? kBlock : there;
        const int lo = chunk * kChunk, hi = lo + kChunk - 1;
        const bool whole = __all(there == kBlock) && hi <= min_pos &&
                           (p.window == 0 || max_pos - lo < p.window || hi < p.sinks);

        // a wavefront that has products goes before one that weighs, whose vector
        // instructions fit between (prompts up to 4 %)
        if constexpr (WS == 1) __builtin_amdgcn_s_setprio(1);
        f32x4 s[RT][4];
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
#pragma unroll
            for (int i = 0; i < RT; ++i) s[i][tt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int st = 0; st < kSteps; ++st) {
                const quad& w = in.k[tt][st >> 1];
                const quad a = widen8<F, T>(w[2 * (st & 1)], w[2 * (st & 1) + 1]);
#pragma unroll
                for (int i = 0; i < RT; ++i) s[i][tt] = gemvdev::mma_16x16x32(T{}, a, q_of(i, st), s[i][tt]);
            }
            // (else all of K is widened first, and two row tiles run out of registers)
            if (RT > 1 && tt == 1) __builtin_amdgcn_sched_barrier(0);
        }
        if (!kAhead && more) {
            load_k(it + WS, then, ahead);
            if (it + 2 * WS < end) next = look_up(it + 2 * WS);
        }
        if constexpr (WS == 1) __builtin_amdgcn_s_setprio(0);
        // a block's keys have one scale, so the largest score of the lane's 16
        // is the largest product times it (a scale is not negative; a negative
        // softmax scale has been given to Q)
        const float ks = in.kscale * p.scale;
        const float vs = held ? in.vscale : 0.0f;
        const bool finite = vs < __builtin_inff();
        const float vfinite = finite ? vs : 0.0f;

        quad pb[RT][2];
        const auto weigh = [&](auto all_seen) {
            constexpr bool WHOLE = decltype(all_seen)::value;
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                uint32_t sees = 0xffffu;  // tokens of block g that the lane's row sees
                if constexpr (!WHOLE) {
                    const int j = vb * kBlock;
                    sees = first_bits(there) & first_bits(pos[i] + 1 - j);
                    if (p.window > 0 && pos[i] >= p.window)
                        sees &= ~first_bits(pos[i] - p.window + 1 - j) | first_bits(p.sinks - j);
#pragma unroll
                    for (int e = 0; e < kBlock; ++e)
                        if (!(sees >> e & 1)) s[i][e >> 2][e & 3] = -__builtin_inff();
                }
                float top = s[i][0][0];
#pragma unroll
                for (int e = 1; e < kBlock; ++e) top = fmaxf(top, s[i][e >> 2][e & 3]);
                // (a lane that sees nothing has top = -inf; ks = 0 would make that a NaN)
                top = WHOLE || sees != 0 ? top * ks : -__builtin_inff();
                // the base of the exponents follows the maximum only where that
                // has grown past it by the slack: then most chunks leave it, and o and
                // l with it, as they are, and no weight passes 2^slack
                const float most = max_of_groups(top);
                const bool higher = most > m[i] + slack_of<WS, SHARED>(p);
                const float to = higher ? most : m[i];
                const float base = finite_base(to);
                // the largest term of the lane's block (a scale that is not finite
                // makes the row NaN by itself)
                const float own = __builtin_amdgcn_exp2f(top - base) * vfinite;
                if (__any(higher || own * (1.0f / kMostUnits) > unit[i])) {
                    // (only the rows whose own it is change: a row's bits do not
                    // depend on what its neighbours see)
                    const float term = max_of_groups(own);
                    const bool grows = higher || term > unit[i] * kMostUnits;
                    const float down = __builtin_amdgcn_exp2f(m[i] - base);
                    l[i] *= down;  // (1 where the base stays)
                    const float kept = unit[i] * down;
                    if (grows) unit[i] = unit_of(fmaxf(fminf(term, 0x1p127f) * kUnitOfLargest, kept));
                    const float by = grows ? kept * inverse(unit[i]) : 1.0f;
#pragma unroll
                    for (int u = 0; u < kTiles; ++u) o[i][u] *= by;
                    m[i] = to;
                }
                // (a scale so far above the unit that their ratio overflows meets
                // weights of next to nothing only)
                const float by = finite ? fminf(vfinite * inverse(unit[i]), 0x1p127f) : vs;
                float sum = 0.0f;
#pragma unroll
                for (int e = 0; e < kBlock; ++e) {
                    float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][e >> 2][e & 3], ks, -base));
                    // a hidden token's weight is zero whatever its block's scales
                    if (!WHOLE && !(sees >> e & 1)) x = 0.0f;
                    sum += x;
                    x *= by;
                    if (!WHOLE && !(sees >> e & 1)) x = 0.0f;
                    s[i][e >> 2][e & 3] = x;
                }
                l[i] += sum;
#pragma unroll
                for (int tt = 0; tt < 4; ++tt) {
                    pb[i][tt >> 1][2 * (tt & 1)] = pack(TF16{}, s[i][tt][0], s[i][tt][1]);
                    pb[i][tt >> 1][2 * (tt & 1) + 1] = pack(TF16{}, s[i][tt][2], s[i][tt][3]);
                }
            }
        };
        // (heads of 256 always take the masks, which they have the time for: with both
        // forms their registers do not hold everything)
        if (whole && DIM <= 128)
            weigh(std::true_type{});
        else
            weigh(std::false_type{});
        if (!whole) {
#pragma unroll
            for (int u = 0; u < kTiles; ++u) in.v[u] = first_bytes(in.v[u], there);
        }
        if constexpr (WS == 1) __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int u = 0; u < kTiles; ++u) {
            const quad a0 = widen8<F, TF16>(in.v[u][0], in.v[u][1]), a1 = widen8<F, TF16>(in.v[u][2], in.v[u][3]);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                o[i][u] = gemvdev::mma_16x16x32(TF16{}, a0, pb[i][0], o[i][u]);
                o[i][u] = gemvdev::mma_16x16x32(TF16{}, a1, pb[i][1], o[i][u]);
            }
        }
        if constexpr (WS == 1) __builtin_amdgcn_s_setprio(0);
        now = then;
        it += WS;
        if (!kAhead && more) load_v(it, now, ahead);
    };
    while (it < end) {
        step(first, kAhead ? second : first);
        if (!kAhead) continue;
        if (it >= end) break;
        step(second, first);
    }

#pragma unroll
    for (int i = 0; i < RT; ++i) l[i] = sum_of_groups(l[i]);
    if constexpr (WS > 1) {
        // the upper half of the wavefronts joins the lower, and so on
        __shared__ f32x4 rows[WS / 2][RT][kTiles][64];
        __shared__ float stat[WS / 2][RT][3][64];
#pragma unroll
        for (int round = WS / 2; round >= 1; round /= 2) {
            const int slot = wave - round;
            if (round < WS / 2) __syncthreads();
            if (slot >= 0 && slot < round) {
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    stat[slot][i][0][lane] = m[i];
                    stat[slot][i][1][lane] = l[i];
                    stat[slot][i][2][lane] = unit[i];
#pragma unroll
                    for (int u = 0; u < kTiles; ++u) rows[slot][i][u][lane] = o[i][u];
                }
            }
            __syncthreads();
            if (wave < round) {
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const float m2 = stat[wave][i][0][lane];
                    const float top = fmaxf(m[i], m2), base = finite_base(top);
                    const float a = __builtin_amdgcn_exp2f(m[i] - base);
                    const float b = __builtin_amdgcn_exp2f(m2 - base);
                    m[i] = top;
                    l[i] = l[i] * a + stat[wave][i][1][lane] * b;
                    const float own = unit[i] * a, other = stat[wave][i][2][lane] * b;
                    unit[i] = unit_of(fmaxf(own, other));
                    const float in = inverse(unit[i]), by = own * in, by2 = other * in;
#pragma unroll
                    for (int u = 0; u < kTiles; ++u) o[i][u] = o[i][u] * by + rows[wave][i][u][lane] * by2;
                }
            }
        }
        if (wave != 0) return;
    }

    // (a row without a position sees nothing, but min_pos is that of the rows that have
    // one, and the chunks before it were taken without masks for all rows of the tile; the
    // join leaves out what a sum of 0 stands beside)
    if constexpr (SHARED) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            if (pos[i] >= 0) continue;
            m[i] = -__builtin_inff();
            l[i] = 0.0f;
        }
    }
    // (the unit over the sum before o meets either: the result is within V's
    // range, o in V's unit need not be)
    float result[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) result[i] = l[i] == 0.0f ? 0.0f : unit[i] * (1.0f / l[i]);
    if (!SHARED && p.splits == 1 && p.shared == 0) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            if (r0 + 16 * i + n > last) continue;
            uint16_t* dst = p.O + row[i] * p.ldo + (int64_t)qhead[i] * DIM + 4 * g;
#pragma unroll
            for (int u = 0; u < kTiles; ++u) {
                const f32x4 x = o[i][u] * result[i];
                fp8dev::u32x2 w;
                w[0] = pack(T{}, x[0], x[1]);
                w[1] = pack(T{}, x[2], x[3]);
                *reinterpret_cast<fp8dev::u32x2_any*>(dst + 16 * u) = w;
            }
        }
        return;
    }
    const Partial out = partial_at<DIM>(p, places, (place * c.heads + head) * p.splits + split);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        if (r0 + 16 * i + n > last) continue;
        const int r = r0 - t.r0 + 16 * i + n;
        if (g == 0) {
            out.ml[2 * r] = m[i];
            out.ml[2 * r + 1] = l[i];
        }
#pragma unroll
        for (int u = 0; u < kTiles; ++u)
            *reinterpret_cast<f32x4*>(out.rows + (int64_t)r * DIM + 16 * u + 4 * g) = o[i][u] * result[i];
    }
}

template <class T, class F, int DIM, int RT, int WS>
__global__ __launch_bounds__(kWavesOf<WS> * 64, DIM <= 128 ? 2 : 1) void kv_attend_kernel(Attend p, int64_t places) {
    attend_part<T, F, DIM, RT, WS, false>(p, places, blockIdx.x);
}

// The rows of all sequences over their shared tokens in the first workgroups, then
// each sequence's rows over its own (own_places: 0 where another launch has these):
// one launch, whose second part starts as the first runs out (4 sequences of up to
// 100 tokens behind 2000: 19.3 us in two, 13.0 in one; 64 of up to 1000 behind 8192: 49
// and 48, the shared ones in 512 workgroups.  In turns, the longer workgroups of the first part end late: 16 behind 65536
// take 68 us instead of 55).
//
// Every 32 rows (16 of dim 256) widen all of the shared K and V for themselves.  So the
// shared part is bound by the vector ALUs and by what two wavefronts a SIMD leave
// unhidden of the steps' latency: 942 tokens of 32 heads over 4000 151 us, 410 TFLOP/s, 64 % of the
// cycles with a vector or matrix instruction; 64 and 16 single tokens, whose shared workgroups
// have a few steps each, 37 and 51 us with their own tokens.  K brought straight to
// LDS a chunk ahead, and Q in registers then, change nothing or cost 9 %; wavefronts with rows of their
// own, which do not fit the registers with masks and without, likewise.
template <class T, class F, int DIM, int RT>
__global__ __launch_bounds__(kShareWaves * 64, DIM <= 128 ? 2 : 1) void kv_attend_shared_kernel(
    Attend s, int64_t shared_places, Attend p, int64_t own_places) {
    const int64_t shared_groups = shared_places * s.cache.heads * s.splits;
    if (blockIdx.x < shared_groups)
        attend_part<T, F, DIM, RT, kShareWaves, true>(s, shared_places, blockIdx.x);
    else
        attend_part<T, F, DIM, 1, kShareWaves, false>(p, own_places, blockIdx.x - shared_groups);
}

// Joins the few splits of rows, their own and those of the shared tokens `s`, a
// wavefront for four neighbouring rows: sixteen lanes a row have a split's
// maximum and sum each, then a lane has DIM / 64 values of each row, and the rows' loads
// are in flight together.  (With a workgroup to each row, the 40096 rows of twelve prompts
// took 120 us.)
constexpr int kFewSplits = 16, kJoinRows = 4;
template <class T, int DIM, int R, int RW>
__global__ __launch_bounds__(kShareWaves * 64) void kv_join_rows_kernel(Attend p, int64_t places, Attend s,
                                                                        int64_t shared_places) {
    constexpr int kPer = DIM / 64;
    typedef float piece __attribute__((ext_vector_type(kPer)));
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const Cache& c = p.cache;
    const int64_t place = blockIdx.x / c.heads;
    const int head = (int)(blockIdx.x - place * c.heads);
    Tile t;
    const int r = ((int)blockIdx.y * kShareWaves + wave) * kJoinRows;  // (all of one wavefront's RW rows)
    if (!tile_of<R>(p, place, t) || r >= p.rows || t.r0 + r >= t.rows) return;
    int rows = t.rows - t.r0 - r;
    rows = rows < p.rows - r ? rows : p.rows - r;
    rows = rows < kJoinRows ? rows : kJoinRows;
    const int r0 = t.r0 + r / RW * RW, last = (r0 + RW < t.rows ? r0 + RW : t.rows) - 1;
    const int chunks = span_of(p, t.first + r0 / p.group, t.first + last / p.group, t.len).count();
    int splits = chunks > p.split_chunks ? (chunks + p.split_chunks - 1) / p.split_chunks : 1;
    splits = splits < p.splits ? splits : p.splits;
    const int all = splits + s.splits;
    const Partial in = partial_at<DIM>(p, places, (place * c.heads + head) * p.splits);
    // row j's place in the call, and among the rows over the shared tokens
    const auto token_of = [&](int j) { return (t.r0 + r + j) / p.group; };
    const auto shared_row = [&](int j) {
        const int token = token_of(j);
        return (t.start + token) * p.group + (t.r0 + r + j - token * p.group);
    };
    const auto shared_at = [&](int row) {
        return partial_at<DIM>(s, shared_places, ((int64_t)(row / s.rows) * c.heads + head) * s.splits);
    };
    const int j = lane >> 4, i = lane & 15;
    float m = -__builtin_inff(), ls = 0.0f;
    if (j < rows && i < all) {
        const int row = shared_row(j);
        const float* ml = i < splits ? in.ml + (i * p.rows + r + j) * 2
                                     : shared_at(row).ml + ((i - splits) * s.rows + row % s.rows) * 2;
        m = ml[0];
        ls = ml[1];
    }
    float top = m;
    top = fmaxf(top, gemvdev::dpp<gemvdev::kDppSwapAdjacent>(top));
    top = fmaxf(top, gemvdev::dpp<gemvdev::kDppSwapPairs>(top));
    top = fmaxf(top, gemvdev::dpp<gemvdev::kDppHalfRowMirror>(top));
    top = fmaxf(top, gemvdev::dpp<gemvdev::kDppRowMirror>(top));
    const float l = ls == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(m - finite_base(top)) * ls;
    const float sum = gemvdev::segment_sum<16>(l);
    // (over the sum before they meet the rows: a result is within V's range, its
    // multiple need not be; a split in which the row sees nothing adds nothing,
    // whatever its row holds)
    const float weight = ls == 0.0f ? -1.0f : l * (sum == 0.0f ? 0.0f : 1.0f / sum);
    const float* own[kJoinRows];
    const float* also[kJoinRows];
    piece o[kJoinRows];
#pragma unroll
    for (int k = 0; k < kJoinRows; ++k) {
        const int n = k < rows ? k : rows - 1;  // (those that are not there repeat the last, and are not stored)
        const int row = shared_row(n);
        own[k] = in.rows + (int64_t)(r + n) * DIM + lane * kPer;
        also[k] = shared_at(row).rows + (int64_t)(row % s.rows) * DIM + lane * kPer;
        o[k] = 0.0f;
    }
    for (int n = 0; n < all; ++n) {
        piece x[kJoinRows];
#pragma unroll
        for (int k = 0; k < kJoinRows; ++k)
            x[k] = *reinterpret_cast<const piece*>(n < splits ? own[k] + (int64_t)n * p.rows * DIM
                                                              : also[k] + (int64_t)(n - splits) * s.rows * DIM);
#pragma unroll
        for (int k = 0; k < kJoinRows; ++k) {
            const float w = gemvdev::f32_of(__builtin_amdgcn_readlane(__builtin_bit_cast(uint32_t, weight), 16 * k + n));
            if (w != -1.0f) o[k] += x[k] * w;
        }
    }
#pragma unroll
    for (int k = 0; k < kJoinRows; ++k) {
        if (k >= rows) break;
        const int token = token_of(k);
        uint16_t* dst = p.O + ((int64_t)t.start + token) * p.ldo +
                        (int64_t)(head * p.group + (t.r0 + r + k - token * p.group)) * DIM + lane * kPer;
#pragma unroll
        for (int d = 0; d < kPer; ++d) dst[d] = fp8dev::narrow(T{}, o[k][d]);
    }
}

// Joins the splits of a row, a workgroup a row (R: rows of a place, RW: of one
// of its wavefronts): the splits' maxima and sums give each its weight, then the
// wavefronts add the weighted rows in turn and join in LDS, in a fixed order.
// SHARED: behind its own splits come those of the shared tokens, `s`.
// Bound by latency: 4.5 us for 32 rows of 64 splits, 7.0 for 2048 rows of up to 11.
template <class T, int DIM, int R, int RW, bool SHARED = false>
__global__ __launch_bounds__(kShareWaves * 64) void kv_join_kernel(Attend p, int64_t places, Attend s,
                                                                   int64_t shared_places) {
    constexpr int kPer = DIM / 64;
    __shared__ float weight[kMaxSplits * (SHARED ? 2 : 1)];
    __shared__ float part[kShareWaves][DIM];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const Cache& c = p.cache;
    const int64_t place = blockIdx.x / c.heads;
    const int head = (int)(blockIdx.x - place * c.heads);
    Tile t;
    const int r = blockIdx.y;
    if (!tile_of<R>(p, place, t) || t.r0 + r >= t.rows) return;
    const int token = (t.r0 + r) / p.group;
    const int in_group = t.r0 + r - token * p.group;
    // the splits that its wavefront's rows have (split 0 always leaves its rows)
    const int r0 = t.r0 + r / RW * RW, last = (r0 + RW < t.rows ? r0 + RW : t.rows) - 1;
    const int chunks = span_of(p, t.first + r0 / p.group, t.first + last / p.group, t.len).count();
    int splits = chunks > p.split_chunks ? (chunks + p.split_chunks - 1) / p.split_chunks : 1;
    splits = splits < p.splits ? splits : p.splits;  // (the partial results end there)
    const Partial in = partial_at<DIM>(p, places, (place * c.heads + head) * p.splits);
    // the row's place among the rows over the shared tokens
    Partial also{};
    int shared_r = 0, all = splits;
    if constexpr (SHARED) {
        const int row = (t.start + token) * p.group + in_group;
        shared_r = row % s.rows;
        also = partial_at<DIM>(s, shared_places, ((int64_t)(row / s.rows) * c.heads + head) * s.splits);
        all += s.splits;
    }
    const auto ml_of = [&](int i) {
        if (!SHARED || i < splits) return in.ml + (i * p.rows + r) * 2;
        return also.ml + ((i - splits) * s.rows + shared_r) * 2;
    };
    // every wavefront reduces the maxima and sums for itself
    float top = -__builtin_inff();
    for (int i = lane; i < all; i += 64) top = fmaxf(top, ml_of(i)[0]);
    const float base = finite_base(wave_max(top));
    float l = 0.0f;
    for (int i = lane; i < all; i += 64) {
        const float ls = ml_of(i)[1];
        // a split in which the row sees nothing adds nothing, whatever its row holds
        const float w = ls == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(ml_of(i)[0] - base) * ls;
        l += w;
        if (wave == 0) weight[i] = ls == 0.0f ? -1.0f : w;
    }
    l = gemvdev::segment_sum<64>(l);
    // (over the sum before they meet the rows: a result is within V's range, its
    // multiple need not be)
    const float by = l == 0.0f ? 0.0f : 1.0f / l;
    if (wave == 0)
        for (int i = lane; i < all; i += 64)
            if (weight[i] != -1.0f) weight[i] *= by;
    __syncthreads();
    float o[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = 0.0f;
    const auto add = [&](int i, const float* row) {
        const float w = weight[i];
#pragma unroll
        for (int d = 0; d < kPer; ++d) {
            const float x = row[d * 64 + lane];
            o[d] += w == -1.0f ? 0.0f : x * w;
        }
    };
#pragma unroll 8
    for (int i = wave; i < splits; i += kShareWaves) add(i, in.rows + ((int64_t)i * p.rows + r) * DIM);
    if constexpr (SHARED) {
#pragma unroll 8
        for (int i = wave; i < s.splits; i += kShareWaves)
            add(splits + i, also.rows + ((int64_t)i * s.rows + shared_r) * DIM);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) part[wave][i * 64 + lane] = o[i];
    __syncthreads();
    uint16_t* dst = p.O + ((int64_t)t.start + token) * p.ldo + (int64_t)(head * p.group + in_group) * DIM;
    for (int d = threadIdx.x; d < DIM; d += kShareWaves * 64) {
        float v = part[0][d];
#pragma unroll
        for (int w = 1; w < kShareWaves; ++w) v += part[w][d];
        dst[d] = fp8dev::narrow(T{}, v);
    }
}

}  // namespace kvdev
