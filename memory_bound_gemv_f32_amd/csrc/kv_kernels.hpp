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

namespace kvdev {

using fp8dev::f32x4;
using fp8dev::max_u32;
using fp8dev::quad;
using fp8dev::quad_any;
using fp8dev::TBF16;
using fp8dev::TF16;
using fp8dev::TF32;
using fp8dev::widen;

constexpr int kBlock = 16;  // tokens that share a scale

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
__device__ __forceinline__ int sequence_of(const Batch& q, int64_t place, int64_t n, int64_t d, int extra) {
    int lo = 0, hi = q.count - 1;  // the last b whose first place is at most `place`
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first_place(q, mid, n, d, extra) <= place)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
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
__device__ __forceinline__ float value8(Int8, uint32_t byte) { return (float)(int)(int8_t)byte; }
__device__ __forceinline__ float value8(E4m3, uint32_t byte) {
    return __builtin_amdgcn_cvt_f32_fp8((int)byte, 0);
}

// 16 elements from p on, `step` apart, of which bit i of `take` says whether
// element i is there.
template <class D>
__device__ __forceinline__ void load16(const typename D::storage* p, int64_t step, uint32_t take,
                                       float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = take >> i & 1 ? widen(D{}, p[i * step]) : 0.0f;
}

// One wavefront per block of one head's keys or values.  16-byte piece p of
// the block is 16 dims of a token (K) or the 16 tokens of a dim (V); a lane
// holds pieces lane, lane + 64, ...
template <class D, class F, int DIM>
__global__ __launch_bounds__(64) void kv_append_kernel(Cache c, Batch q,
                                                       const typename D::storage* K, int64_t ldk,
                                                       const typename D::storage* V, int64_t ldv) {
    constexpr int kPieces = DIM / 64;  // of a lane: kBlock·DIM / 16 / 64
    const int lane = threadIdx.x;
    const int head = (int)blockIdx.y;
    const bool values = blockIdx.z != 0;
    const int64_t place = blockIdx.x;
    const int b = sequence_of(q, place, 1, kBlock, 2);
    const int start = start_of(q, b), stop = start_of(q, b + 1);
    const int len = q.lens[b];
    const int64_t first = (int64_t)len - ((int64_t)stop - start);  // position of the first new token
    const int64_t block64 = (first > 0 ? first : 0) / kBlock + place - first_place(q, b, 1, kBlock, 2);
    if (block64 < 0 || block64 * kBlock >= len || stop <= start) return;
    const int block = (int)block64;
    const int page = page_of(q, c, b, block);
    if (page < 0) return;
    const int64_t index = block_index(c, page, head, block);
    uint8_t* held = (values ? c.v : c.k) + index * (kBlock * DIM);
    float* scale = (values ? c.v_scale : c.k_scale) + index;
    // tokens of the block that this call brings, and those that stay
    uint32_t fresh = 0, stay = 0;
    for (int i = 0; i < kBlock; ++i) {
        const int64_t pos = (int64_t)block * kBlock + i;
        const int64_t row = start + pos - first;
        if (pos < first)
            stay |= 1u << i;
        else if (pos < len && row >= 0 && row < q.total)
            fresh |= 1u << i;
    }
    if (fresh == 0) return;
    const int64_t row0 = start + (int64_t)block * kBlock - first;  // the row of the block's token 0
    float x[kPieces][16];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        const int piece = lane + 64 * j;
        if (values) {
            const int dim = piece;
            load16<D>(V + row0 * ldv + (int64_t)head * DIM + dim, ldv, fresh, x[j]);
        } else {
            const int token = piece / (DIM / 16), dim = piece % (DIM / 16) * 16;
            load16<D>(K + (row0 + token) * ldk + (int64_t)head * DIM + dim, 1,
                      fresh >> token & 1 ? 0xffffu : 0u, x[j]);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) m = max_u32(m, fp8dev::magnitude(x[j][i]));
    }
    const float need = block_scale<F>(fp8dev::wave_max(m));
    float s = need, ratio = 1.0f;
    if (stay != 0) {
        const float old = *scale;
        if (!(old <= need)) s = old;  // the larger, and NaN once either is
        if (need != need) s = need;
        ratio = old / s;
    }
    const float inv = 1.0f / s;
    const bool bad = s != s;  // the bytes of a block with no scale are zero
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        const int piece = lane + 64 * j;
        const int token = piece / (DIM / 16);
        const uint32_t put = values ? fresh : (fresh >> token & 1 ? 0xffffu : 0u);
        const uint32_t keep = values ? stay : (stay >> token & 1 ? 0xffffu : 0u);
        if (put == 0 && (keep == 0 || ratio == 1.0f)) continue;
        quad* at = reinterpret_cast<quad*>(held) + piece;
        quad w = put == 0xffffu ? quad{0u, 0u, 0u, 0u} : *at;
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
        *at = w;
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
// K and V are widened exactly (e4m3 and int8 both fit fp16 and bf16); a
// block's scales are one number a lane: K's multiplies S in fp32, V's
// multiplies P.  P is rounded to Q's type; relative to the largest V scale
// seen so far, so that it stays at most 1 and fp16 does not underflow.
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
__device__ __forceinline__ float sum_of_groups(float v) {
    return gemvdev::half_pair_sum32(gemvdev::row_pair_sum16(v));
}

constexpr int kChunk = 64;    // tokens of a step: four blocks
constexpr int kAttWaves = 4;  // wavefronts of a workgroup

struct Attend {
    Cache cache;
    Batch batch;
    const uint16_t* Q;
    int64_t ldq;
    uint16_t* O;
    int64_t ldo;
    int group;          // query heads that share a K/V head
    float scale;        // softmax scale · log2(e)
    int window, sinks;  // window 0: none
    int capacity;       // tokens that a row of the table can hold
    int splits;         // workgroups that share a row tile's tokens
    float* partial;     // splits > 1: see partial_at
};

// What a row tile sees: chunks [0, first) hold the first tokens that stay
// visible, [low, high) the window (or everything up to the last row).
struct Span {
    int first, low, high;
    __device__ __forceinline__ int count() const { return first + high - low; }
    __device__ __forceinline__ int chunk(int i) const { return i < first ? i : i - first + low; }
};
__device__ __forceinline__ Span span_of(const Attend& p, int min_pos, int max_pos, int len) {
    int end = max_pos + 1 < len ? max_pos + 1 : len;
    end = end < p.capacity ? end : p.capacity;
    Span s;
    s.high = end > 0 ? (end + kChunk - 1) / kChunk : 0;
    s.low = 0;
    s.first = 0;
    if (p.window > 0 && min_pos >= p.window) {
        s.low = (min_pos - p.window + 1) / kChunk;
        const int sinks = (p.sinks + (kChunk - 1)) / kChunk;
        s.first = sinks < s.low ? sinks : s.low;
    }
    if (s.low > s.high) s.low = s.high;
    return s;
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
    t.b = sequence_of(q, place, p.group, R, 1);
    const int64_t r0 = (place - first_place(q, t.b, p.group, R, 1)) * R;
    t.start = start_of(q, t.b);
    const int stop = start_of(q, t.b + 1);
    // rows outside the call's are not there, whatever the starts say
    if (t.start < 0 || stop > q.total || stop <= t.start) return false;
    t.len = q.lens[t.b];
    t.first = (int)((int64_t)t.len - (stop - t.start));
    t.rows = (stop - t.start) * p.group;
    t.r0 = (int)r0;
    return r0 >= 0 && r0 < t.rows;
}

// splits > 1: each split leaves its unnormalised row and the row's m and l,
// for rows of a place, a head and a split: first all (m, l), then all rows.
struct Partial {
    float* ml;
    float* rows;
};
template <int R, int DIM>
__device__ __forceinline__ Partial partial_at(const Attend& p, int64_t places, int64_t part) {
    const int64_t parts = places * p.cache.heads * p.splits;
    return Partial{p.partial + part * R * 2, p.partial + parts * R * 2 + part * R * DIM};
}

// WS = 4: the workgroup's wavefronts take the chunks of one row tile in turn
// and join in LDS.  WS = 1: each wavefront has a row tile of its own.
template <class T, class F, int DIM, int RT, int WS>
__global__ __launch_bounds__(kAttWaves * 64) void kv_attend_kernel(Attend p, int64_t places) {
    constexpr int kRows = 16 * RT;                              // rows of a wavefront
    constexpr int kGroupRows = WS == 1 ? kAttWaves * kRows : kRows;
    constexpr int kSteps = DIM / 32;                            // K·Q^T steps
    constexpr int kTiles = DIM / 16;                            // 16-dim tiles of O^T
    constexpr bool kRelative = std::is_same<T, TF16>::value;    // P over the largest V scale
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int n = lane & 15, g = lane >> 4;
    const Cache& c = p.cache;
    // heads fastest: neighbouring workgroups, which go to different chiplets,
    // share no K or V; then the splits; the last rows, which see the most, first
    int64_t at = blockIdx.x;
    const int head = (int)(at % c.heads);
    at /= c.heads;
    const int split = (int)(at % p.splits);
    const int64_t place = places - 1 - at / p.splits;
    Tile t;
    if (!tile_of<kGroupRows>(p, place, t)) return;
    const int r0 = t.r0 + (WS == 1 ? wave * kRows : 0);
    if (WS == 1 && r0 >= t.rows) return;
    const int last = (r0 + kRows < t.rows ? r0 + kRows : t.rows) - 1;
    const int min_pos = t.first + r0 / p.group, max_pos = t.first + last / p.group;
    const Span span = span_of(p, min_pos, max_pos, t.len);
    const int per_split = (span.count() + p.splits - 1) / p.splits;
    const int begin = split * per_split;
    const int end = begin + per_split < span.count() ? begin + per_split : span.count();

    // the lane's row of each 16: its position (-1: none) and its Q
    int pos[RT];
    int64_t row[RT];     // row of the call
    int qhead[RT];
    quad q[RT][kSteps];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int r = r0 + 16 * i + n;
        const int rr = r <= last ? r : last;
        const int token = rr / p.group;
        pos[i] = r <= last ? t.first + token : -1;
        row[i] = (int64_t)t.start + token;
        qhead[i] = head * p.group + (rr - token * p.group);
        const uint16_t* src = p.Q + row[i] * p.ldq + (int64_t)qhead[i] * DIM + 16 * g;
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
            q[i][s] = *reinterpret_cast<const quad_any*>(src + 64 * (s >> 1) + 8 * (s & 1));
    }

    f32x4 o[RT][kTiles];
    float m[RT], l[RT];
    float vref = kRelative ? 0.0f : 1.0f;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        m[i] = -__builtin_inff();
        l[i] = 0.0f;
#pragma unroll
        for (int u = 0; u < kTiles; ++u) o[i][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    for (int it = begin + (WS == 1 ? 0 : wave); it < end; it += WS) {
        const int chunk = span.chunk(it);
        // of the four blocks, the lane reads K from block n / 4 and V from block g
        const int kb = 4 * chunk + (n >> 2), vb = 4 * chunk + g;
        int kpage = kb * kBlock < t.len ? page_of(p.batch, c, t.b, kb) : -1;
        int vpage = vb * kBlock < t.len ? page_of(p.batch, c, t.b, vb) : -1;
        const int64_t ki = block_index(c, kpage < 0 ? 0 : kpage, head, kb);
        const int64_t vi = block_index(c, vpage < 0 ? 0 : vpage, head, vb);
        const uint8_t* kp = c.k + ki * (kBlock * DIM) + (n & 3) * DIM + 16 * g;
        const uint8_t* vp = c.v + vi * (kBlock * DIM) + n * kBlock;
        quad k[4][DIM / 64], v[kTiles];
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int h = 0; h < DIM / 64; ++h)
                k[tt][h] = *reinterpret_cast<const quad*>(kp + 4 * tt * DIM + 64 * h);
#pragma unroll
        for (int u = 0; u < kTiles; ++u) v[u] = *reinterpret_cast<const quad*>(vp + 16 * u * kBlock);
        const float ks = c.k_scale[vi] * p.scale;
        float vs = vpage < 0 ? 0.0f : c.v_scale[vi];
        // tokens of block g that are there
        int there = vpage < 0 ? 0 : t.len - vb * kBlock;
        there = there < 0 ? 0 : there > kBlock ? kBlock : there;
        const int lo = chunk * kChunk, hi = lo + kChunk - 1;
        const bool whole = __all(there == kBlock) && hi <= min_pos &&
                           (p.window == 0 || max_pos - lo < p.window || hi < p.sinks);
        if (!whole) {
#pragma unroll
            for (int u = 0; u < kTiles; ++u) v[u] = first_bytes(v[u], there);
        }
        if (kRelative) {
            const float top = max_of_groups(vs);
            if (__any(top > vref)) {
                const float down = vref / top;
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int u = 0; u < kTiles; ++u) o[i][u] *= down;
                vref = top;
            }
            vs = vref > 0.0f ? vs / vref : vs;
        }

        quad pb[RT][2];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            f32x4 s[4];
#pragma unroll
            for (int tt = 0; tt < 4; ++tt) {
                s[tt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int st = 0; st < kSteps; ++st) {
                    const quad& w = k[tt][st >> 1];
                    const quad a = widen8<F, T>(w[2 * (st & 1)], w[2 * (st & 1) + 1]);
                    s[tt] = gemvdev::mma_16x16x32(T{}, a, q[i][st], s[tt]);
                }
            }
            // tokens of block g that the lane's row sees
            uint32_t sees = 0xffffu;
            if (!whole) {
                sees = 0;
#pragma unroll
                for (int off = 0; off < kBlock; ++off) {
                    const int j = vb * kBlock + off;
                    if (off < there && j <= pos[i] &&
                        (p.window == 0 || pos[i] - j < p.window || j < p.sinks))
                        sees |= 1u << off;
                }
            }
            float top = -__builtin_inff();
#pragma unroll
            for (int tt = 0; tt < 4; ++tt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = s[tt][e] * ks;
                    s[tt][e] = sees >> (4 * tt + e) & 1 ? x : -__builtin_inff();
                    top = fmaxf(top, s[tt][e]);
                }
            top = fmaxf(m[i], max_of_groups(top));
            // a row that has seen nothing yet keeps its maximum at -inf; its
            // exponents are taken against 0
            const float base = top == -__builtin_inff() ? 0.0f : top;
            if (__any(top != m[i])) {
                const float down = __builtin_amdgcn_exp2f(m[i] - base);
                l[i] *= down;
#pragma unroll
                for (int u = 0; u < kTiles; ++u) o[i][u] *= down;
                m[i] = top;
            }
#pragma unroll
            for (int tt = 0; tt < 4; ++tt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = __builtin_amdgcn_exp2f(s[tt][e] - base);
                    l[i] += x;
                    // a hidden token's weight is zero whatever its block's scale
                    s[tt][e] = sees >> (4 * tt + e) & 1 ? x * vs : 0.0f;
                }
                pb[i][tt >> 1][2 * (tt & 1)] = pack(T{}, s[tt][0], s[tt][1]);
                pb[i][tt >> 1][2 * (tt & 1) + 1] = pack(T{}, s[tt][2], s[tt][3]);
            }
        }
#pragma unroll
        for (int u = 0; u < kTiles; ++u) {
            const quad a0 = widen8<F, T>(v[u][0], v[u][1]), a1 = widen8<F, T>(v[u][2], v[u][3]);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                o[i][u] = gemvdev::mma_16x16x32(T{}, a0, pb[i][0], o[i][u]);
                o[i][u] = gemvdev::mma_16x16x32(T{}, a1, pb[i][1], o[i][u]);
            }
        }
    }

#pragma unroll
    for (int i = 0; i < RT; ++i) {
        l[i] = sum_of_groups(l[i]);
        if (kRelative)
#pragma unroll
            for (int u = 0; u < kTiles; ++u) o[i][u] *= vref;
    }
    if constexpr (WS > 1) {
        // wavefronts 2 and 3 join 0 and 1, then 1 joins 0
        __shared__ f32x4 rows[2][RT][kTiles][64];
        __shared__ float stat[2][RT][2][64];
#pragma unroll
        for (int round = 2; round >= 1; --round) {
            const int slot = wave - round;
            if (round == 1) __syncthreads();
            if (slot >= 0 && slot < round) {
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    stat[slot][i][0][lane] = m[i];
                    stat[slot][i][1][lane] = l[i];
#pragma unroll
                    for (int u = 0; u < kTiles; ++u) rows[slot][i][u][lane] = o[i][u];
                }
            }
            __syncthreads();
            if (wave < round) {
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const float m2 = stat[wave][i][0][lane];
                    const float top = fmaxf(m[i], m2);
                    const float base = top == -__builtin_inff() ? 0.0f : top;
                    const float a = __builtin_amdgcn_exp2f(m[i] - base);
                    const float b = __builtin_amdgcn_exp2f(m2 - base);
                    m[i] = top;
                    l[i] = l[i] * a + stat[wave][i][1][lane] * b;
#pragma unroll
                    for (int u = 0; u < kTiles; ++u) o[i][u] = o[i][u] * a + rows[wave][i][u][lane] * b;
                }
            }
        }
        if (wave != 0) return;
    }

    if (p.splits == 1) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            if (r0 + 16 * i + n > last) continue;
            const float by = l[i] == 0.0f ? 0.0f : 1.0f / l[i];
            uint16_t* dst = p.O + row[i] * p.ldo + (int64_t)qhead[i] * DIM + 4 * g;
#pragma unroll
            for (int u = 0; u < kTiles; ++u) {
                const f32x4 x = o[i][u] * by;
                fp8dev::u32x2 w;
                w[0] = pack(T{}, x[0], x[1]);
                w[1] = pack(T{}, x[2], x[3]);
                *reinterpret_cast<fp8dev::u32x2_any*>(dst + 16 * u) = w;
            }
        }
        return;
    }
    const Partial out = partial_at<kGroupRows, DIM>(
        p, places, (place * c.heads + head) * p.splits + split);
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
            *reinterpret_cast<f32x4*>(out.rows + (int64_t)r * DIM + 16 * u + 4 * g) = o[i][u];
    }
}

// Joins the splits of each row: a wavefront a row.
template <class T, int DIM, int R>
__global__ __launch_bounds__(kAttWaves * 64) void kv_join_kernel(Attend p, int64_t places) {
    constexpr int kPer = DIM / 64;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const Cache& c = p.cache;
    const int64_t place = blockIdx.x / c.heads;
    const int head = (int)(blockIdx.x - place * c.heads);
    Tile t;
    if (!tile_of<R>(p, place, t)) return;
    for (int r = (int)blockIdx.y * kAttWaves + wave; r < R && t.r0 + r < t.rows; r += kAttWaves * gridDim.y) {
        float m = -__builtin_inff(), l = 0.0f, o[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[i] = 0.0f;
        for (int s = 0; s < p.splits; ++s) {
            const Partial in = partial_at<R, DIM>(p, places, (place * c.heads + head) * p.splits + s);
            const float m2 = in.ml[2 * r], l2 = in.ml[2 * r + 1];
            if (l2 == 0.0f) continue;
            const float top = fmaxf(m, m2);
            const float base = top == -__builtin_inff() ? 0.0f : top;
            const float a = __builtin_amdgcn_exp2f(m - base), b = __builtin_amdgcn_exp2f(m2 - base);
            m = top;
            l = l * a + l2 * b;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                o[i] = o[i] * a + in.rows[(int64_t)r * DIM + i * 64 + lane] * b;
        }
        const float by = l == 0.0f ? 0.0f : 1.0f / l;
        const int token = (t.r0 + r) / p.group;
        uint16_t* dst = p.O + ((int64_t)t.start + token) * p.ldo +
                        (int64_t)(head * p.group + (t.r0 + r - token * p.group)) * DIM;
#pragma unroll
        for (int i = 0; i < kPer; ++i) dst[i * 64 + lane] = fp8dev::narrow(T{}, o[i] * by);
    }
}

}  // namespace kvdev
