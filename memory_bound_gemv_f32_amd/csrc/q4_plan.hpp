// Sizes of the products with 4-bit weights.
//
// Pure C++ (no HIP headers): the kernels count with these functions, and a machine
// without a GPU can hold them against their meaning.
#pragma once

#include <stdint.h>

namespace q4plan {

constexpr int kChunk = 128;  // columns of a step: 16 bytes to a lane
constexpr int kBlock = 32;   // columns of a matrix-core step

// Groups of kBlock << log2 columns in a row of K, the last of them maybe shorter (K up
// to an int's end: nothing may be added to it).
constexpr int groups_of(int K, int log2) {
    const int blocks = K / kBlock + (K % kBlock != 0);
    return (blocks >> log2) + ((blocks & ((1 << log2) - 1)) != 0);
}

}  // namespace q4plan
