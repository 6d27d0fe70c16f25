// Grids: the device's compute units, and rows of workgroups for the layer
// operators (include/fc/layer.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace fc {

// Kernels with one workgroup for little data: a launch counts its threads along
// x in 32 bits, so their workgroups lie in rows of 2^20 (x) along y.
constexpr int kGridRow = 20;

__device__ __forceinline__ uint64_t grid_index() {
    return (uint64_t)__builtin_amdgcn_workgroup_id_y() << kGridRow | __builtin_amdgcn_workgroup_id_x();
}

inline dim3 grid_of_blocks(uint64_t blocks) {
    const uint64_t row = uint64_t(1) << kGridRow;
    return blocks <= row ? dim3((unsigned)blocks) : dim3((unsigned)row, (unsigned)((blocks + row - 1) / row));
}

// Whether a launch of `blocks` workgroups along x counts its threads in 32 bits: what is
// past that is not refused by the runtime, a launch of 2^32 + n threads runs n of them.
inline bool launch_fits(uint64_t blocks, unsigned threads) {
    return blocks != 0 && blocks <= 0xFFFFFFFFull / threads;
}

// run(first value, values) for n values in pieces of at most `most`, but at least `unit`,
// which every piece but the last is a multiple of.
template <class Run>
hipError_t in_pieces(uint64_t n, uint64_t most, uint64_t unit, Run &&run) {
    const uint64_t piece = most > unit ? most / unit * unit : unit;
    for (uint64_t at = 0; at < n; at += piece) {
        const hipError_t err = run(at, n - at < piece ? n - at : piece);
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

// Compute units of the current device (persistent kernels have a workgroup or
// two on each), looked up once per device. The cache is atomic: calls from
// several host threads may fill it at once (with the same value).
inline int compute_units() {
    static std::atomic<int> cached[64] = {};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return -1;
    int n = cached[dev].load(std::memory_order_relaxed);
    if (n <= 0) {
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
            n <= 0)
            return -1;
        cached[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

}  // namespace fc
