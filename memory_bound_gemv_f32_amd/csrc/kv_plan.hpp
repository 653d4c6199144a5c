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
    int skip = 0;  // so many of these are left out: those that the batch shares
    constexpr int count() const { return first + high - low - skip; }
    constexpr int chunk(int i) const { return i + skip < first ? i + skip : i + skip - first + low; }
};
// Of rows at positions min_pos to max_pos of a sequence of len tokens, whose row
// of the table can hold `capacity` of them: tokens past that are not there, so
// no chunk lies past it, whatever the length says, and there are no more chunks
// than map_attend counts.  Chunks before `from` are left out.
constexpr Span span_of(int window, int sinks, int capacity, int min_pos, int max_pos, int len, int from = 0) {
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
    const int in_window = from < s.low ? 0 : from < s.high ? from - s.low : s.high - s.low;
    s.skip = from < s.first ? from : s.first + in_window;
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

// Cuts a mapping's chunks into splits; where they fit `slots` in splits of at most
// one_round, so.
inline void cut(Mapping& m, int heads, int dim, int64_t chunks, int64_t slots = kSlots,
                int64_t one_round = kOneRoundSplit) {
    if (m.places * heads > kMostTiles) {  // (launchable refuses it; the products below would overflow)
        m.splits = 1;
        m.split_chunks = (int)chunks;
        return;
    }
    const int64_t all = m.places * heads * chunks;
    const bool own = m.waves_share == 1;
    // (a chunk of dim 256 takes long: 1 x 28767 tokens, one head, 23.6 us in splits of
    // 8 chunks, 19.5 of 4; 4 x 4000, 4 heads, 20.8 and 16.6)
    const int64_t least = own || dim > 128 ? kLeastLongSplit : kLeastSplit;
    int64_t each = ceil_div(all, own ? kOwnSlots : slots);
    each = !own && each > one_round ? kSplit : each < least ? least : each;
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
}

// (skip: chunks at the start of the sequences that are left out)
inline Mapping map_attend(int q_heads, int heads, int dim, int rows, int sequences, bool one_each, int64_t capacity,
                          int window, int sinks, int skip = 0) {
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
    int64_t chunks = ceil_div(capacity, kChunk) - skip;
    if (window > 0) {
        const int64_t tokens = ceil_div(m.group_rows, group) + 1;
        const int64_t in_window = ceil_div((int64_t)window + tokens, kChunk) + 1 +
                                  ceil_div(sinks, kChunk);
        if (in_window < chunks) chunks = in_window;
    }
    cut(m, heads, dim, chunks);
    return m;
}

// The rows of the whole batch over `chunks` chunks that all its sequences share.  Their
// splits are alike, and each leaves a partial result of all rows, so they are one
// round of workgroups, however long (16384 tokens, 8 heads of 4 query heads, with own
// tokens up to 1000, us with splits of 12 past 32 chunks and without: 96 sequences 110
// and 86, 300 sequences 312 and 226).  many_own: the sequences' own tokens have a
// workgroup for every other slot; then the shared ones leave them these, while their
// splits stay at 32 chunks or less (64 sequences: 4096 tokens 44 and 42, 8192 48 and 40; 16384, of
// 64 chunks, 64 and 77).
inline Mapping map_shared(int q_heads, int heads, int dim, int rows, int64_t chunks, bool many_own) {
    Mapping m;
    const int64_t all_rows = (int64_t)rows * (q_heads / heads);
    m.waves_share = 4;
    m.row_tiles = all_rows <= 16 || dim > 128 ? 1 : 2;
    m.group_rows = 16 * m.row_tiles;
    m.places = ceil_div(all_rows, m.group_rows);
    m.place_rows = all_rows < m.group_rows ? (int)all_rows : m.group_rows;
    const bool half = many_own && m.places * heads <= kSlots / 2 * kOneRoundSplit / (chunks > 0 ? chunks : 1);
    cut(m, heads, dim, chunks, half ? kSlots / 2 : kSlots, chunks);
    m.waves_share = 4;  // (one kernel takes them and the sequences' own tokens)
    // Many rows fill the GPU by themselves, and every split costs a start and an end of
    // its own, and a write and a read of all rows (3768 rows, 8 heads, over 4000 tokens:
    // 158 us, and in two splits 177).
    if (m.places * heads >= kSlots) {
        m.splits = 1;
        m.split_chunks = (int)chunks;
    }
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

inline size_t partials_of(const Mapping& m, int heads, int dim) {
    const int64_t rows = m.places * heads * m.splits * m.place_rows;
    return (size_t)(stats_floats(rows) + rows * dim) * sizeof(float);
}
inline size_t workspace_of(const Mapping& m, int heads, int dim) {
    return m.splits == 1 ? 0 : partials_of(m, heads, dim);
}

inline int64_t capacity_of(int64_t table_width, int page_size) {
    const int64_t n = table_width * page_size;
    return n < 0x7fffffff ? n : 0x7fffffff;
}

// A call whose sequences share their first tokens: `chunks` chunks of them are
// taken for all rows together and the rest for each sequence as ever; 0: that
// would gain nothing, and `own` takes all.
struct SharedMapping {
    int chunks;
    Mapping shared, own;
};
// Taken together the shared tokens cost a join, and save reading them for each
// sequence: from 16 MiB a byte of each key and value and sequence on.  Measured, us
// without and with, 8 heads of 128, single tokens: 4 sequences behind 2048 12.5 and
// 12.7, behind 4096 16.8 and 13.0; 8 behind 1024 12.3 and 14.9, behind 2048 16.5 and 15.3;
// 64 behind 256 13.3 and 16.9, behind 512 17.7 and 16.5; of 256, 4 behind 2048 23.2 and 15.0.
// Prompts, whose rows fill the matrix cores by themselves, gain where the sequences
// are many: 4 of up to 60 tokens behind 4096 51 and 57, 12 behind 1024 54 and 62, behind 4096
// 169 and 118; 8 of up to 150 behind 4096 177 and 133.  Of shared tokens that a window
// hides in part each sequence reads the rest only, and at another place: it takes eight
// times as many of these (64 single tokens behind 4096, windows of 512 17 and 24, of 1024 22
// and 26, of 2048 44 and 27; 64 prompts of up to 60, of 1024 108 and 143, of 2048 182 and
// 186, of 4096 behind 16384 331 and 273).
//
// Prompts that fill the GPU by themselves widen no less behind shared tokens (both ways
// for each 32 rows), and lose a partial result of each row, written and read.  The plain call
// takes a step for each 1024 of its workgroups or part of them, this one grows with the rows,
// so they are taken together up to three quarters of the first step; behind many
// tokens, where the join is little, always; and behind fewer where each prompt has at most
// two workgroups' rows, which it seldom fills.  Measured, us without and with, e4m3, dim 128:
// 16 prompts of 4 query heads, 600 | 700 | 800 | 1000 | 1150 | 1600 | 4200 workgroups, behind
// 4096 200 and 148 | 193 and 168 | 190 and 191 | 190 and 222 | 185 and 246 | 352 and 361 | 827
// and 964, behind 8192 385 and 240 | 363 and 278 | 363 and 321 | 364 and 374 | 362 and 423 | 672
// and 618 | 1606 and 1646; 64 of 512 tokens behind 1024 1012 and 1763.  Of 34 | 48 | 63 | 98 |
// 116 rows, 256 or 64 of them, behind 4096 465 and 285 | 470 and 371 | 595 and 501 | 298 and
// 221 | 298 and 247, behind 1024 139 and 144 | 143 and 181 | 192 and 246.  (Of dim 256 the same
// within a fifth either way.)
constexpr int64_t kWorthSharing = 1 << 24, kManySequences = 8, kManyTokens = 1 << 15, kHidden = 8;
constexpr int64_t kFewWorkgroups = kOwnSlots * 3 / 4, kLong = 4096, kVeryLong = 8192;
// plain: the mapping of the call without shared tokens
constexpr bool worth_sharing(const Mapping& plain, int heads, int dim, int sequences, bool one_each, int64_t shared,
                             int64_t seen, int64_t rows_each) {
    if (sequences < 2 || shared < kChunk) return false;
    if (!one_each && sequences < kManySequences) return false;
    if (plain.waves_share == 1 && plain.places * heads > kFewWorkgroups &&
        shared < (rows_each > 2 * plain.group_rows ? kVeryLong : kLong))
        return false;
    const int64_t tokens = seen < shared ? sequences * seen / kHidden : sequences * shared;
    return tokens >= (rows_each > 32 ? kManyTokens : kWorthSharing / ((int64_t)heads * dim));
}
inline SharedMapping map_both(int q_heads, int heads, int dim, int rows, int sequences, bool one_each,
                              int64_t capacity, int window, int sinks, int shared) {
    SharedMapping s{};
    const int64_t there = shared < capacity ? shared : capacity;
    const int64_t group = q_heads / heads;
    const int64_t rows_each = one_each ? group : sequences > 0 ? ceil_div(rows * group, sequences) : 0;
    const int64_t seen = window > 0 ? (int64_t)window + sinks : there;
    s.own = map_attend(q_heads, heads, dim, rows, sequences, one_each, capacity, window, sinks);
    if (!worth_sharing(s.own, heads, dim, sequences, one_each, there, seen, rows_each)) return s;
    s.chunks = (int)(there / kChunk);
    s.own = map_attend(q_heads, heads, dim, rows, sequences, one_each, capacity, window, sinks, s.chunks);
    if (s.own.waves_share == 8) s.own.waves_share = 4;  // (as the shared tokens' wavefronts)
    const bool many_own = s.own.waves_share == 4 && s.own.places * heads * s.own.splits >= kSlots / 2;
    s.shared = map_shared(q_heads, heads, dim, rows, s.chunks, many_own);
    return s;
}
// Whether one launch takes both parts, and whether the launches hold them and their join.
constexpr bool together(const SharedMapping& s) { return s.own.waves_share == 4 && s.own.row_tiles == 1; }
constexpr bool launchable(const SharedMapping& s, int heads) {
    return launchable(s.own, heads) &&
           (s.chunks == 0 || (launchable(s.shared, heads) &&
                              (s.own.places * s.own.splits + s.shared.places * s.shared.splits) * heads *
                                      kShareWaves * 64 <= 0xffffffff));
}
inline size_t workspace_of(const SharedMapping& s, int heads, int dim) {
    return s.chunks == 0 ? workspace_of(s.own, heads, dim)
                         : partials_of(s.own, heads, dim) + partials_of(s.shared, heads, dim);
}
// The mapping of a call: shared tokens are taken together where that pays and fits.
// Both parts leave partial results of all rows, where the plain call leaves those of few or
// none, so theirs are 1 GiB at most (8192 single tokens of 32 query heads of 256 take half
// of it); and what the plain call's launches hold is never refused.
constexpr size_t kMostShared = (size_t)1 << 30;
inline SharedMapping map_call(int q_heads, int heads, int dim, int rows, int sequences, bool one_each,
                              int64_t capacity, int window, int sinks, int shared) {
    const SharedMapping s = map_both(q_heads, heads, dim, rows, sequences, one_each, capacity, window, sinks, shared);
    if (s.chunks == 0 || (launchable(s, heads) && workspace_of(s, heads, dim) <= kMostShared)) return s;
    return map_both(q_heads, heads, dim, rows, sequences, one_each, capacity, window, sinks, 0);
}

}  // namespace kvplan
