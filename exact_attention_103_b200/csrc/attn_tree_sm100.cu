// attn_tree_sm100.cu -- exact attention of new tokens over the paged cache.
//
// One warp per (token, query head): keys one by one, each lane holding d / 32 values of the
// head, with the running maximum and sum of the softmax in fp32.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "cache_ops.h"

namespace attn {
namespace {

template <int D, bool F8>
__global__ void __launch_bounds__(128) tree_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int E = D / 32;
  const attn_cache_t& c = a.cache;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (w >= static_cast<int64_t>(a.T) * a.Hq) return;
  const int t = static_cast<int>(w / a.Hq), h = static_cast<int>(w % a.Hq);
  int b = -1;
  for (int i = 0; i < a.B; ++i)
    if (a.cu[i] <= t && t < a.cu[i + 1]) b = i;
  if (b < 0) return;
  const int n = a.cu[b + 1] - a.cu[b], local = t - a.cu[b];
  const int slot = a.slots ? a.slots[b] : b;
  if (slot < 0 || slot >= c.slots) {
    record_invalid(a.err, kSiteSlot);
    return;
  }
  const int len = c.lens[slot];
  if (len < n || len > static_cast<int64_t>(c.max_pages) * c.page_size || (a.mask && n > a.mask_width)) {
    record_invalid(a.err, kSiteLength);
    return;
  }
  const int hk = h / (a.Hq / c.heads);
  float q[E], o[E] = {};
  for (int e = 0; e < E; ++e)
    q[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[(static_cast<int64_t>(t) * a.Hq + h) * D + lane * E + e]);
  const float ks = F8 ? c.k_scale : 1.f, vs = F8 ? c.v_scale : 1.f;
  auto value = [&](const void* base, int64_t at) -> float {
    if constexpr (F8) return static_cast<float>(static_cast<const __nv_fp8_e4m3*>(base)[at]);
    else return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at]);
  };
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < len; ++j) {
    const int jl = j - (len - n);
    if (jl >= 0 && (a.mask ? a.mask[static_cast<int64_t>(t) * a.mask_width + jl] == 0 : jl > local)) continue;
    const int page = c.page_table[static_cast<int64_t>(slot) * c.max_pages + j / c.page_size];
    if (page < 0 || page >= c.pages) {
      record_invalid(a.err, kSitePage);
      return;
    }
    const int64_t at = (((static_cast<int64_t>(a.layer) * c.pages + page) * c.page_size + j % c.page_size) * c.heads + hk) * D + lane * E;
    float s = 0.f;
    for (int e = 0; e < E; ++e) s += q[e] * value(c.k, at + e);
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= a.scale * ks;
    const float top = fmaxf(m, s);
    const float old = m == -INFINITY ? 0.f : expf(m - top), p = expf(s - top);
    m = top;
    l = l * old + p;
    for (int e = 0; e < E; ++e) o[e] = o[e] * old + p * value(c.v, at + e);
  }
  for (int e = 0; e < E; ++e)
    static_cast<__nv_bfloat16*>(a.o)[(static_cast<int64_t>(t) * a.Hq + h) * D + lane * E + e] = __float2bfloat16(l > 0.f ? o[e] / l * vs : 0.f);
  if (lane == 0) a.lse[static_cast<int64_t>(h) * a.T + t] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t tree_workspace(int) { return 0; }

cudaError_t launch_tree(const TreeArgs& a, int, cudaStream_t st) {
  const int64_t warps = static_cast<int64_t>(a.T) * a.Hq;
  const unsigned grid = static_cast<unsigned>((warps + 3) / 4);
  if (a.cache.d == 128) {
    if (a.cache.e4m3) tree_kernel<128, true><<<grid, 128, 0, st>>>(a);
    else tree_kernel<128, false><<<grid, 128, 0, st>>>(a);
  } else {
    if (a.cache.e4m3) tree_kernel<64, true><<<grid, 128, 0, st>>>(a);
    else tree_kernel<64, false><<<grid, 128, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace attn
