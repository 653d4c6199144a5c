// How the attention over the paged 8-bit cache is cut into work: which chunks
// of tokens a row tile walks, which rows a workgroup takes, and how many
// workgroups share a row tile's tokens.
//
// Pure C++ (no HIP headers): the launcher sizes the grid and the workspace with
// these functions and the kernels walk with them, so that the two can be held
// against each other on a machine without a GPU.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace kvplan {

constexpr int kBlock = 16;       // tokens that share a scale
constexpr int kChunk = 64;       // tokens of a step: four blocks
constexpr int kMaxSplits = 512;  // workgroups that share a row tile's tokens, at most
// Wavefronts of a workgroup: 4 or 8 that share their rows, or 2 with rows of their
// own (4 of those would read the same bytes more often from the same cache, but
// leave fewer and longer workgroups: 176 us against 183 for four prompts of up to 1024 tokens).
constexpr int kShareWaves = 4, kOwnWaves = 2;

// What a row tile sees: chunks [0, first) hold the first tokens that stay
// visible, [low, high) the window (or everything up to the last row).
struct Span {
    int first, low, high;
    constexpr int count() const { return first + high - low; }
    constexpr int chunk(int i) const { return i < first ? i : i - first + low; }
};
// Of rows at positions min_pos to max_pos of a sequence of len tokens, whose row
// of the table can hold `capacity` of them: tokens past that are not there, so
// no chunk lies past it, whatever the length says, and there are no more chunks
// than map_attend counts.
constexpr Span span_of(int window, int sinks, int capacity, int min_pos, int max_pos, int len) {
    int end = max_pos + 1 < len ? max_pos + 1 : len;
    end = end < capacity ? end : capacity;
    Span s{0, 0, 0};
    s.high = end > 0 ? (end - 1) / kChunk + 1 : 0;
    if (window > 0 && min_pos >= window) {
        s.low = (min_pos - window + 1) / kChunk;
        if (s.low > s.high) s.low = s.high;
        const int in_sinks = sinks / kChunk + (sinks % kChunk != 0);
        s.first = in_sinks < s.low ? in_sinks : s.low;
    }
    return s;
}

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How an attention call is mapped: the rows of a workgroup, whether its
// wavefronts share them, and how many workgroups share a row tile's tokens.
struct Mapping {
    int row_tiles;     // 16-row tiles of a wavefront
    int waves_share;   // 4 or 8: so many wavefronts take the chunks of the same rows in turn; 1: own rows each
    int group_rows;    // rows of a workgroup
    int place_rows;    // rows of it that can be there
    int splits, split_chunks;
    int64_t places;
};

// A split is a workgroup's work.  Where all of it fits the 512 slots (two
// workgroups for each compute unit) in splits of at most 32 chunks (2048 tokens),
// that many, of at least 8 (less is mostly start-up); else splits of 12, short
// enough that the last round of workgroups is not long.  Measured, us: one
// sequence of 131071 tokens, 8 heads: 59 | 58 | 54 | 56 | 51 with splits of 8 | 12
// | 16 | 24 | 32; 64 sequences of up to 8192: 127 | 113 | 120 | 114 | 137.  The
// longest contexts and largest batches get longer ones, so that the workspace
// stays at 8192 workgroups' rows.  Wavefronts with rows of their own (prompts) have
// many rows, whose partial results cost a write and a read each, so they are split
// only into one round of workgroups, four of theirs to a compute unit (256 tokens over 16384,
// 32 heads: 154 us in splits of 12, 126 in one round; 9 x 29 over up to 42563, 5
// heads: 83 and 54), and not at all once a quarter of that has a workgroup.
constexpr int64_t kOwnSlots = 1024, kLeastLongSplit = 4;
constexpr int64_t kMostTiles = 0x7fffffff;
constexpr int64_t kLeastSplit = 8, kOneRoundSplit = 32, kSplit = 12, kSlots = 512, kMostWorkgroups = 8192;

inline Mapping map_attend(int q_heads, int heads, int dim, int rows, int sequences, bool one_each, int64_t capacity,
                   int window, int sinks) {
    Mapping m;
    const int group = q_heads / heads;
    const int64_t per_sequence = one_each ? group : ceil_div((int64_t)rows * group, sequences);
    m.waves_share = per_sequence <= 32 ? 4 : 1;
    m.row_tiles = per_sequence <= 16 || dim > 128 ? 1 : 2;  // (two of dim 256 would not fit the registers)
    m.group_rows = 16 * m.row_tiles * (m.waves_share == 1 ? kOwnWaves : 1);
    m.places = one_each ? sequences * ceil_div(group, m.group_rows)
                        : (int64_t)rows * group / m.group_rows + sequences;
    m.place_rows = one_each && group < m.group_rows ? group : m.group_rows;
    // chunks that a row tile can see
    int64_t chunks = ceil_div(capacity, kChunk);
    if (window > 0) {
        const int64_t tokens = ceil_div(m.group_rows, group) + 1;
        const int64_t in_window = ceil_div((int64_t)window + tokens, kChunk) + 1 +
                                  ceil_div(sinks, kChunk);
        if (in_window < chunks) chunks = in_window;
    }
    if (m.places * heads > kMostTiles) {  // (launchable refuses it; the products below would overflow)
        m.splits = 1;
        m.split_chunks = (int)chunks;
        return m;
    }
    const int64_t all = m.places * heads * chunks;
    const bool own = m.waves_share == 1;
    // (a chunk of dim 256 takes long: 1 x 28767 tokens, one head, 23.6 us in splits of
    // 8 chunks, 19.5 of 4; 4 x 4000, 4 heads, 20.8 and 16.6)
    const int64_t least = own || dim > 128 ? kLeastLongSplit : kLeastSplit;
    int64_t each = ceil_div(all, own ? kOwnSlots : kSlots);
    each = !own && each > kOneRoundSplit ? kSplit : each < least ? least : each;
    if (each < ceil_div(all, kMostWorkgroups)) each = ceil_div(all, kMostWorkgroups);
    if (each < ceil_div(chunks, kMaxSplits)) each = ceil_div(chunks, kMaxSplits);
    // (a single split would save little)
    if (chunks < 2 * (own ? kLeastLongSplit : kLeastSplit) || (own && m.places * heads >= kOwnSlots / 4)) each = chunks;
    m.splits = each > 0 ? (int)ceil_div(chunks, each) : 1;
    if (m.splits < 1) m.splits = 1;
    m.split_chunks = (int)each;
    // No more than a workgroup for each compute unit, and latency is all: eight
    // wavefronts (of dim 256 too large for the registers) halve the chunks that wait
    // for each other (4 sequences, window 512: 13.8 us with four, 12.2 with eight;
    // 4 x 4000 tokens, in two launches: 13.7 and 13.2).
    if (dim <= 128 && m.waves_share == 4 && m.row_tiles == 1 && each > 4 &&
        m.places * heads * m.splits <= kSlots / 2)
        m.waves_share = 8;
    return m;
}

// Wavefronts of a workgroup of the attention, and whether its launch and the
// join's hold all their workgroups and threads.
constexpr int waves_of(const Mapping& m) { return m.waves_share == 1 ? kOwnWaves : m.waves_share; }
constexpr bool launchable(const Mapping& m, int heads) {
    const int64_t tiles = m.places * heads, most = 0xffffffff;
    return tiles <= kMostTiles && tiles * m.splits <= kMostTiles && tiles * m.splits * waves_of(m) * 64 <= most &&
           (m.splits == 1 || tiles * kShareWaves * 64 <= most);
}

// The workspace holds so many partial rows' maxima and sums, then the rows, which
// are stored in 16-byte pieces: the first part in floats.
constexpr int64_t stats_floats(int64_t rows) { return (rows * 2 + 3) / 4 * 4; }

inline size_t workspace_of(const Mapping& m, int heads, int dim) {
    if (m.splits == 1) return 0;
    const int64_t rows = m.places * heads * m.splits * m.place_rows;
    return (size_t)(stats_floats(rows) + rows * dim) * sizeof(float);
}

inline int64_t capacity_of(int64_t table_width, int page_size) {
    const int64_t n = table_width * page_size;
    return n < 0x7fffffff ? n : 0x7fffffff;
}

}  // namespace kvplan
