// cache_ops.h -- internal launch interface of the serving operators' kernels (the
// public C ABI is include/attn_cache.h).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/attn_cache.h"

namespace attn {

// Where a kernel found its input inconsistent: the site byte of the device error word
// (code 1 = ATTN_ERR_INVALID_ARG below it).  The attention kernels use 1..31.
enum CacheSite : int {
  kSiteSlot = 32,     // slot number out of range, or named twice
  kSiteLength,        // lens / cu_q / new_lens inconsistent
  kSitePage,          // page number out of range, or a reference count below zero
  kSitePath,          // accepted path not increasing or outside the drafted tokens
  kSiteCopyOverlap    // a copied page is also written
};

__device__ __forceinline__ void record_invalid(int* err, int site) {
  if (err) atomicCAS(err, 0, 1 | (site << 8));
}

// The serving operators follow one another on a stream in kernels of a few microseconds.  Each is
// launched as a programmatic dependent of the kernel before it; before it touches memory it waits
// until that one, whatever it was, has completed (and with it everything earlier on the stream).
// At its own entry it lets the next one launch (but for the rotary kernel, whose many
// blocks the next one's would keep from the SMs).  What the kernel before may have written is read
// past L1 or by plain loads, never through the read-only path.
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The blocks in clusters of `cluster` (a part of the grid's x).
template <typename... P, typename... A>
cudaError_t launch_clusters_after(void (*kernel)(P...), int cluster, dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                                  A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
  if (e != cudaSuccess) cudaGetLastError();  // reported here, not by a later call
  return e;
}

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A&&... args) {
  return launch_clusters_after(kernel, 1, grid, block, smem, st, args...);
}

constexpr int kMaxSequences = 1024;  // of a packed batch

struct RopeArgs {
  attn_rope_plan_t plan;  // plan.turns null: nothing is rotated
  attn_rows_t t[3];       // q, k (attn_rope: count of them; append: q, k, v)
  int inverse, d, B, N, tokens;
  const int32_t* cu;
  const int32_t* positions;
  // append only
  attn_cache_t cache;
  int layer;
  const int32_t* slots;
  int* err;
};
cudaError_t launch_rope(const RopeArgs& a, attn_type_t type, int sms, cudaStream_t st);
cudaError_t launch_append(const RopeArgs& a, int sms, cudaStream_t st);

cudaError_t launch_alloc(const attn_cache_t& c, const int32_t* slots, const int32_t* want, int n,
                         int32_t* granted, int* err, cudaStream_t st);
cudaError_t launch_free(const attn_cache_t& c, const int32_t* slots, int n, int* err, cudaStream_t st);
cudaError_t launch_fork(const attn_cache_t& c, const int32_t* src, const int32_t* dst, int n,
                        int32_t* granted, void* ws, int* err, cudaStream_t st);
cudaError_t launch_copy(const attn_cache_t& c, const int32_t* src, const int32_t* dst, int n, int* err,
                        cudaStream_t st);
cudaError_t launch_compact(const attn_cache_t& c, const int32_t* cu_q, const int32_t* path, int width,
                           const int32_t* accepted, const int32_t* slots, int B, int* err,
                           cudaStream_t st);

struct TreeArgs {
  attn_cache_t cache;
  int layer;
  const void* q;
  void* o;
  float* lse;
  int Hq, B, T;
  const int32_t* cu;
  const int32_t* slots;
  const uint8_t* mask;
  int mask_width;
  float scale;
  void* ws;
  int* err;
};
size_t tree_workspace(int d);
// ATTN_ERR_UNSUPPORTED: too many tiles for 32-bit counting; ATTN_ERR_CUDA: a tensor map was
// rejected; otherwise *cuda is the launches' result.
attn_status_t launch_tree(const TreeArgs& a, int sms, cudaStream_t st, cudaError_t* cuda);

}  // namespace attn
