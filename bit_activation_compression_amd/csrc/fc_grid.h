// Grids of the kernels with one workgroup for little data: a launch counts its
// threads along x in 32 bits, so their workgroups lie in rows of 2^20 (x) along y.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fc {

constexpr int kGridRow = 20;

__device__ __forceinline__ uint64_t grid_index() {
    return (uint64_t)__builtin_amdgcn_workgroup_id_y() << kGridRow | __builtin_amdgcn_workgroup_id_x();
}

inline dim3 grid_of_blocks(uint64_t blocks) {
    const uint64_t row = uint64_t(1) << kGridRow;
    return blocks <= row ? dim3((unsigned)blocks) : dim3((unsigned)row, (unsigned)((blocks + row - 1) / row));
}

}  // namespace fc
