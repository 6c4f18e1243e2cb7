// Thread-block cluster helpers: rank, barrier, and reads of another CTA's
// shared memory (select.cu, sparse_decode.cu).
#pragma once

#include <atomic>
#include <cstdint>

#include "common.cuh"

namespace pkv {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Every thread of every CTA of the cluster arrives and waits: writes to
// shared memory before it are visible to the cluster after it.  It cannot be
// bounded; callers reach it on every path.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Its two halves: work on memory that no other CTA touches may stand between.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Shared-memory address of this CTA's `addr` in the CTA of rank `rank`.
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void red_cluster_add(uint32_t addr, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v)
               : "memory");
}
__device__ __forceinline__ void red_cluster_min(uint32_t addr, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.min.u32 [%0], %1;" ::"r"(addr), "r"(v)
               : "memory");
}
__device__ __forceinline__ void red_cluster_max(uint32_t addr, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(addr), "r"(v)
               : "memory");
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  return __uint_as_float(ld_cluster_u32(addr));
}

// Launch `kern` on `s` as clusters of `cluster` CTAs along x (grid.x a
// multiple of it) and as a programmatic dependent of the work before it.
// Dynamic shared memory that passes 48 KB with the kernel's own has to be
// allowed before (allow_shared).
struct ClusterLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  ClusterLaunch(dim3 grid, dim3 block, size_t smem, unsigned cluster, cudaStream_t s) {
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
};

template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                            unsigned cluster, cudaStream_t s, Args... args) {
  ClusterLaunch l(grid, block, smem, cluster, s);
  return cudaLaunchKernelEx(&l.cfg, kern, static_cast<KArgs>(args)...);
}

// Facts of the current device, asked of it once and kept by the caller, in a
// word for each device (of kDevices) that starts as 0.

// Allow the kernel's launches up to `smem` bytes of dynamic shared memory:
// always the same number, so that calls of several threads agree.
template <typename... KArgs>
cudaError_t allow_shared(void (*kern)(KArgs...), size_t smem, std::atomic<int>& done) {
  if (done.load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) done.store(1, std::memory_order_release);
  return e;
}

// The clusters of `cluster` CTAs that the device holds at once.  (Its parts
// differ in SMs, and a cluster lies in one: 15 clusters of 8 CTAs fit on 152 SMs.)
template <typename... KArgs>
cudaError_t clusters_held(void (*kern)(KArgs...), int threads, size_t smem, unsigned cluster,
                          std::atomic<int>& known, int* n) {
  int k = known.load(std::memory_order_relaxed);
  if (k == 0) {
    ClusterLaunch l(dim3(cluster), dim3(threads), smem, cluster, nullptr);
    int held = 0;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&held, kern, &l.cfg);
    if (e != cudaSuccess) return e;
    k = held + 1;
    known.store(k, std::memory_order_relaxed);
  }
  *n = k - 1;
  return cudaSuccess;
}

}  // namespace pkv
