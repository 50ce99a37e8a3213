// Device helpers shared by the 8-bit tile kernels: explicit waits, LDS DMA, the
// order of the tiles.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace svdq {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef unsigned int u32;
typedef u32 u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) void glb_void;

constexpr int kXcds = 8;
constexpr int kBandM = 4;

// wait until at most n vector-memory operations of this wave are outstanding
// and all of its LDS operations are done
template <int n>
__device__ __forceinline__ void wait_vm_lds() {
  static_assert(n >= 0 && n < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((n & 0xF) | (0x7 << 4) | ((n >> 4) << 14));
}

// workgroup barrier without the memory fences of __syncthreads (the waits it
// needs are explicit); the empty asm keeps LDS accesses on their side
__device__ __forceinline__ void barrier() {
  __asm__ volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  __asm__ volatile("" ::: "memory");
}

__device__ __forceinline__ void dma16(const void* gptr, uint8_t* lds_wave_base) {
  __builtin_amdgcn_global_load_lds((glb_void*)gptr, (lds_void*)lds_wave_base, 16, 0, 0);
}

// Workgroup id -> (tile_m, tile_n).  Workgroups go round-robin over the 8
// XCDs (id % 8), each with its own L2; the ids of one XCD take one contiguous
// chunk of the tile list, ordered in bands of kBandM tile rows, so the
// workgroups an XCD runs together share few weight and token tiles.
__device__ __forceinline__ void tile_of(int bid, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int T = tiles_m * tiles_n;
  const int x = bid % kXcds;
  const int i = bid / kXcds;
  const int per = T / kXcds, rem = T % kXcds;
  const int t = x * per + min(x, rem) + i;
  const int band = t / (kBandM * tiles_n);
  const int first = band * kBandM;
  const int rows = min(tiles_m - first, kBandM);
  const int in = t - band * kBandM * tiles_n;
  tm = first + in % rows;
  tn = in / rows;
}

}  // namespace svdq
