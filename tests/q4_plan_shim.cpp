// Host build of the sizes of the products with 4-bit weights for the CPU tests.
#include "../memory_bound_gemv_f32_amd/csrc/q4_plan.hpp"

extern "C" int shim_groups_of(int K, int log2) { return q4plan::groups_of(K, log2); }
