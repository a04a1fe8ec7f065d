// gemm_tile.hpp -- what the kernels of 256 x 256 tiles share: LDS DMA, waits and
// barriers, the block order, the device's compute units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace fp4dev {

typedef __attribute__((address_space(3))) void lds_void_t;

constexpr int kXcds = 8;

// s_waitcnt immediate: vmcnt(n) with lgkmcnt(0).
constexpr int wait_vm_lgkm0(int n) { return (n & 15) | ((n >> 4) << 14) | 0x0070; }

// Workgroup barrier without the workgroup-scope release fence of
// __syncthreads(), which would wait for every outstanding LDS DMA: the caller
// has already waited (s_waitcnt) for exactly the DMA the barrier publishes.
// The wavefront-scope fences emit no code; they keep the compiler from moving
// memory accesses across the barrier.
__device__ __forceinline__ void barrier_after_wait() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Wave-wide DMA: each lane's 16 (or 4) bytes at (voff + soff) of the buffer
// go to LDS at lds_dst + 16 (or 4) * lane; lds_dst must be wave-uniform.
__device__ __forceinline__ void dma16_to_lds(__amdgpu_buffer_rsrc_t rsrc, void* lds_dst,
                                             uint32_t voff, int soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void_t*)lds_dst, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void dma4_to_lds(__amdgpu_buffer_rsrc_t rsrc, void* lds_dst,
                                            uint32_t voff, int soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void_t*)lds_dst, 4, voff, soff, 0, 0);
}

// Maps the hardware block index to a (tile_m, tile_n) pair: XCD-contiguous
// runs of logical tiles, grouped GM tile-rows at a time.
template <int GM>
__device__ __forceinline__ void tile_of_block(int b, int nb, int tm, int tn, int& tile_m, int& tile_n) {
    const int xcd = b % kXcds, idx = b / kXcds;
    const int full = nb / kXcds, rem = nb % kXcds;
    const int t = xcd * full + (xcd < rem ? xcd : rem) + idx;
    const int per_group = GM * tn;
    const int group = t / per_group, first_m = group * GM;
    const int gm = (tm - first_m) < GM ? (tm - first_m) : GM;
    const int r = t - group * per_group;
    tile_m = first_m + r % gm;
    tile_n = r / gm;
}

// Compute units of each device, queried once per device (concurrent first
// calls may both query; they store the same value).
inline int cu_count() {
    static std::atomic<int> counts[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    int n = counts[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
            n = 256;
        counts[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

// Tile-rows per group of the block order (each XCD runs 32 tiles at a time):
// groups of 2 to 4 rows measured best on the gate/up and q_proj shapes.
constexpr int kGroupRows = 4;

}  // namespace fp4dev
