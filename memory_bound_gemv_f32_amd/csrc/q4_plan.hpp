// Sizes of the products with 4-bit weights, and which kernel takes which call.
//
// Pure C++ (no HIP headers): the launcher chooses and the kernels count with these
// functions, and a machine without a GPU can hold them against their meaning.
#pragma once

#include <stdint.h>

namespace q4plan {

constexpr int kChunk = 128;  // columns of a step: 16 bytes to a lane
constexpr int kBlock = 32;   // columns of a matrix-core step
constexpr int kLeastColumns = 32;  // of every kernel but kShort's

// Of one launch: rows and vectors.
constexpr int kMostRows = 1 << 20, kMostTokens = 1 << 15;

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Groups of kBlock << log2 columns in a row of K, the last of them maybe shorter (K up
// to an int's end: nothing may be added to it).
constexpr int groups_of(int K, int log2) {
    const int blocks = K / kBlock + (K % kBlock != 0);
    return (blocks >> log2) + ((blocks & ((1 << log2) - 1)) != 0);
}

// LDS that the vectors of a call take, in `parts` parts each.
constexpr int64_t staged_bytes(int parts, int K, int T) {
    return parts * (int64_t)T * (ceil_div(K, kChunk) * kChunk * 2 + 16);
}

// Which kernel takes a call.  Few vectors read W straight into registers, in as many rows to a
// workgroup as leave two of them to a compute unit at most (X, which each
// of them reads whole, is what wider row tiles save: of more than 8 vectors they are wide as soon as
// most units have one); past that the tiles, whose X goes
// through LDS.  Measured, us at vectors x rows x K, bf16, groups of 128 (16 rows | 32
// rows | 64 rows | tile of 64 x 64):
//   1 x 4096 x 4096        5.7 |  7.2 | 11.6 | 29.8
//   1 x 14336 x 4096      13.3 | 11.5 | 12.1
//   8 x 14336 x 4096      17.4 | 12.9 | 12.6
//   16 x 4096 x 4096       7.8 |  9.0 | 12.5 | 30.1
//   16 x 14336 x 4096     22.5 | 15.4 | 13.0 | 30.2
//   24 x 14336 x 4096          | 25.6 | 23.6 | 30.6
//   64 x 14336 x 4096          | 47.2 | 45.9 | 32.1
//   128 x 4096 x 4096          | 28.3 | 24.5 | 31.2
//   256 x 4096 x 4096          | 52.9 | 45.7 | 31.4
// and of tiles 64 x 64 | 128 x 128 through registers | 256 x 64 | 256 x 112 | 256 x
// 128 straight into LDS, where every unit's first tile takes some 18 us, and each
// 5.5 us for 16 vectors and 25 besides:
//   512 x 4096 x 4096     42.5 |  86.9 |  60.1 |  81.0 |  88.5
//   1024 x 4096 x 4096    82.1 |  92.7 |  66.4 |  84.3 |  90.1
//   2000 x 4096 x 4096   163.2 | 113.7 | 102.7 | 126.4 |  95.9
//   512 x 14336 x 4096   132.0 | 111.6 |  99.5 | 125.6 |  94.4
//   1024 x 14336 x 4096  246.6 | 206.8 | 180.4 | 192.3 | 143.4
//   2000 x 14336 x 4096  503.1 | 388.1 | 314.0 | 267.3 | 276.6
enum Family {
    kShort,    // rows of fewer columns than a matrix-core step
    kStaged,   // few vectors in parts, brought to LDS
    kFew16,    // few vectors, 16 | 32 | 64 rows to a workgroup
    kFew32,
    kFew64,
    kTile64,   // X through LDS, 64 x 64
    kTile128,  // 128 rows x 128 vectors; in parts 192 x 64
    kWide64,   // X straight into LDS, 256 rows x 64 | 112 | 128 vectors
    kWide112,
    kWide128,
};
constexpr int64_t kUnits = 256, kEnoughTiles = 384;
constexpr int64_t kMostStaged = 150 * 1024;  // bytes of LDS for vectors
constexpr int kMostOffset = 1 << 22;         // pitch with which a tile's rows are 32-bit offsets apart
// parts: of a vector's value, 1 or 3.  far: a pitch of kMostOffset or more.  whole: all chunks
// of columns are whole, and all 16-byte pieces of them aligned.
constexpr Family family_of(int parts, int M, int K, int T, bool far, bool whole) {
    if (K < kLeastColumns) return kShort;
    // (1 x 4096 x 11008: 11.1 us; with the parts cut by every wavefront for itself 17)
    if (parts > 1 && parts * T <= 16 && staged_bytes(parts, K, T) <= kMostStaged) return kStaged;
    const int64_t tokens = ceil_div(T, 16);
    if (ceil_div(M, 16) * tokens <= kUnits) return kFew16;
    const bool wide_rows = parts == 1 && T > 8 && 4 * ceil_div(M, 64) * tokens >= 3 * kUnits;
    if (!wide_rows && ceil_div(M, 32) * tokens < 2 * kUnits) return kFew32;
    if (far || ceil_div(M, 64) * tokens <= 2 * kUnits) return kFew64;
    if (parts == 1) {
        if (ceil_div(M, 64) * ceil_div(T, 64) <= 2 * kUnits) return kTile64;
        if (whole) {
            // a compute unit's tiles, and what one of them takes
            const auto cost = [&](int nt) { return ceil_div(ceil_div(M, 256) * ceil_div(T, 16 * nt), kUnits) * (2 * nt + 9); };
            if (cost(8) <= cost(7) && cost(8) <= cost(4)) return kWide128;
            return cost(7) <= cost(4) ? kWide112 : kWide64;
        }
    }
    return ceil_div(M, 128) * ceil_div(T, 128) < kEnoughTiles ? kTile64 : kTile128;
}

}  // namespace q4plan
