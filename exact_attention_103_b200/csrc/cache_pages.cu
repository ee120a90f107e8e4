// cache_pages.cu -- the pages of the key/value cache: handing out, sharing, copying,
// moving together and releasing them (include/attn_cache.h).
//
// The state is a table of page numbers per slot, a length per slot and a reference
// count per page.  Free pages are those with count 0, handed out lowest number first in
// the order of the requests, so results never depend on timing.  All of it is
// integer bookkeeping of a few kilobytes, bound by latency; the copies are bound by HBM.
#include <climits>
#include <cstring>
#include <cuda_runtime.h>

#include "cache_ops.h"

namespace attn {
namespace {

constexpr int kBlock = 1024;     // the one block that hands out pages
constexpr int kPagesPerThread = 16;

__device__ __forceinline__ int pages_of(int tokens, int page_size) {
  return static_cast<int>((static_cast<int64_t>(tokens) + page_size - 1) / page_size);
}

// Exclusive prefix sum of one value per thread of the block, and the block's total.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* warp_sums, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    T s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T n = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += n;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  const T before = warp ? warp_sums[warp - 1] : 0;
  total = warp_sums[31];
  __syncthreads();
  return before + incl - v;
}

__device__ __forceinline__ int64_t row_bytes(const attn_cache_t& c) {
  return static_cast<int64_t>(c.heads) * c.d * (c.e4m3 ? 1 : 2);
}
// K (kv = 0) or V of layer l, row `row` of its pages.
__device__ __forceinline__ uint8_t* cache_row(const attn_cache_t& c, int l, int kv, int64_t row) {
  return static_cast<uint8_t*>(kv ? c.v : c.k) +
         (static_cast<int64_t>(l) * c.pages * c.page_size + row) * row_bytes(c);
}

// Copies `bytes` (a multiple of 16), 16 per thread (t of `threads`) and step, U of them in flight.
template <int U>
__device__ __forceinline__ void copy_bytes(const uint8_t* src, uint8_t* dst, int64_t bytes, int t, int threads) {
  const uint4* s = reinterpret_cast<const uint4*>(src);
  uint4* d = reinterpret_cast<uint4*>(dst);
  const int64_t n = bytes / 16;
  int64_t i = t;
  for (; i + (U - 1) * threads < n; i += U * threads) {
    uint4 w[U];
#pragma unroll
    for (int k = 0; k < U; ++k) w[k] = __ldcg(s + i + k * threads);
#pragma unroll
    for (int k = 0; k < U; ++k) d[i + k * threads] = w[k];
  }
  for (; i < n; i += threads) d[i] = __ldcg(s + i);
}

// One fork, decided by the first kernel and carried out by the second.
struct alignas(16) ForkItem {
  int src, dst, len;  // len 0: nothing to do
  int fresh;          // page of the copied tail (len % page_size != 0)
};

// Grants requests for pages.  alloc: slot a[i] grows to b[i] tokens.  FORK: slot a[i]
// is forked into slot b[i] (the pages of its full part and the copies follow in
// fork_kernel).  A slot that grows inside a page which another slot holds too (compaction cut it back
// there) gets a page of its own in its place, one page more, whose tokens this block copies itself, at one SM's
// rate (44 tokens of 8 heads of 128 in 32 layers 129 us): blocks for it would cost every other call.  Shared memory: owner (first request that names a slot), upto (pages
// needed by requests 0..i), have, slot, shared_page.  One block, bound by its round trips to memory: the requests
// and the first 16384 reference counts, the lengths, the stores.  Measured (B200, in a graph): freeing
// and granting 128 slots of a pool of 65536 pages 9.4 us, a grant that finds nothing to do 4.2 us, one
// that grows 64 slots inside their last pages 3.4 us (two round trips of it to look whether they are shared).
template <bool FORK>
__global__ void __launch_bounds__(kBlock, 1) grant_kernel(const attn_cache_t c, const int32_t* a, const int32_t* b, int n,
                                                          int32_t* granted, ForkItem* items, int* err) {
  extern __shared__ int64_t shared[];
  __shared__ int64_t need_sums[32];
  __shared__ int page_sums[32];
  int64_t* upto = shared;  // [n] in 64 bits: each request may ask for as many pages as a table row has entries
  int* owner = reinterpret_cast<int*>(upto + n);  // [slots]
  int* have = owner + c.slots;  // [n] pages held before (-1: refused)
  int* slot = have + n;         // [n] the slot that is written
  int* shared_page = slot + n;  // [n] alloc: the page whose tokens are copied (-1: none)
  const int tid = threadIdx.x;
  const int32_t* target = FORK ? b : a;  // the slot that is written
  let_next_launch();
  for (int s = tid; s < c.slots; s += kBlock) owner[s] = INT_MAX;
  wait_for_previous();
  // The first stretch of reference counts is on its way while the requests are read.
  const bool wide = (reinterpret_cast<uintptr_t>(c.refs) & 15) == 0;
  auto free_pages = [&](int p0) -> unsigned {  // bit k: page p0 + k is free
    unsigned bits = 0;
    if (wide && p0 + kPagesPerThread <= c.pages) {
      int4 w[kPagesPerThread / 4];
#pragma unroll
      for (int k = 0; k < kPagesPerThread / 4; ++k) w[k] = __ldcg(reinterpret_cast<const int4*>(c.refs + p0) + k);
#pragma unroll
      for (int k = 0; k < kPagesPerThread / 4; ++k)
        bits |= ((w[k].x == 0) | ((w[k].y == 0) << 1) | ((w[k].z == 0) << 2) | ((w[k].w == 0) << 3)) << (4 * k);
    } else {
      for (int k = 0; k < kPagesPerThread; ++k)
        if (p0 + k < c.pages && __ldcg(c.refs + p0 + k) == 0) bits |= 1u << k;
    }
    return bits;
  };
  unsigned bits = free_pages(tid * kPagesPerThread);
  // Each thread takes consecutive requests, so that the prefix sum follows their order.
  const int per = (n + kBlock - 1) / kBlock;
  const int i0 = min(tid * per, n), i1 = min(i0 + per, n);
  __syncthreads();
  for (int i = i0; i < i1; ++i) {
    const int s = slot[i] = __ldcg(target + i);
    if (s >= 0 && s < c.slots) atomicMin(&owner[s], i);
  }
  __syncthreads();
  int64_t sum = 0;
  for (int i = i0; i < i1; ++i) {
    const int s = slot[i];
    bool ok = s >= 0 && s < c.slots && owner[s] == i;
    int site = kSiteSlot, need = 0, held = 0;
    [[maybe_unused]] int alone = -1;
    if (FORK) {
      const int from = __ldcg(a + i);
      ok = ok && from >= 0 && from < c.slots && from != s;
      if (ok) {
        const int len = __ldcg(c.lens + from), there = __ldcg(c.lens + s);
        site = kSiteLength;
        ok = there == 0 && len >= 0 && len <= static_cast<int64_t>(c.max_pages) * c.page_size;
        if (ok) {
          need = (len & (c.page_size - 1)) ? 1 : 0;
          items[i].len = len;
        }
      }
    } else if (ok) {
      const int len = __ldcg(c.lens + s), want = __ldcg(b + i);
      site = kSiteLength;
      ok = len >= 0 && want >= len && want <= static_cast<int64_t>(c.max_pages) * c.page_size;
      if (ok) {
        held = pages_of(len, c.page_size);
        need = pages_of(want, c.page_size) - held;
        if (want > len && (len & (c.page_size - 1))) {
          const int last = __ldcg(c.page_table + static_cast<int64_t>(s) * c.max_pages + held - 1);
          if (last < 0 || last >= c.pages) {
            ok = false;
            site = kSitePage;
            need = 0;
          } else if (__ldcg(c.refs + last) > 1) {
            alone = last;
            --held;
            ++need;
          }
        }
      }
    }
    if (!ok) record_invalid(err, site);
    have[i] = ok ? held : -1;
    if (!FORK) shared_page[i] = alone;
    sum += need;
    upto[i] = sum;  // within the thread; the threads before are added below
  }
  int64_t total;
  const int64_t before = block_scan(sum, need_sums, total);
  for (int i = i0; i < i1; ++i) upto[i] += before;
  __syncthreads();
  // The free pages, lowest first: each thread counts its pages of a stretch, a
  // prefix sum ranks them, and page number `rank` goes to the request it falls into.
  int found = 0;
  for (int base = 0; base < c.pages && found < total; base += kBlock * kPagesPerThread) {
    const int p0 = base + tid * kPagesPerThread;
    int here;
    int rank = found + block_scan(__popc(bits), page_sums, here);
    unsigned next = 0;  // the next stretch loads behind this one's work
    if (found + here < total && p0 + kBlock * kPagesPerThread < c.pages) next = free_pages(p0 + kBlock * kPagesPerThread);
    int lo = 0;  // the first request with upto > rank: searched once, then followed
    if (bits && rank < total) {
      int hi = n - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (upto[mid] > rank) hi = mid; else lo = mid + 1;
      }
    }
    for (; bits && rank < total; ++rank, bits &= bits - 1) {
      const int page = p0 + __ffs(bits) - 1;
      while (upto[lo] <= rank) ++lo;
      c.refs[page] = 1;
      if (FORK) {
        items[lo].fresh = page;
      } else {
        const int k = have[lo] + static_cast<int>(rank - (lo ? upto[lo - 1] : 0));
        c.page_table[static_cast<int64_t>(slot[lo]) * c.max_pages + k] = page;
      }
    }
    found += here;
    bits = next;
  }
  __syncthreads();
  bool copies = false;
  for (int i = i0; i < i1; ++i) {
    const int64_t first = i ? upto[i - 1] : 0, need = upto[i] - first;
    bool ok = have[i] >= 0;
    const int s = slot[i];
    if (ok && need > 0 && upto[i] > found) {
      ok = false;
      // What it did get goes back (a fork needs one page: it got none).
      for (int k = 0; !FORK && k < found - first; ++k) {
        int32_t* e = c.page_table + static_cast<int64_t>(s) * c.max_pages + have[i] + k;
        c.refs[__ldcg(e)] = 0;
        *e = -1;
      }
      if (!FORK && shared_page[i] >= 0) {
        c.page_table[static_cast<int64_t>(s) * c.max_pages + have[i]] = shared_page[i];
        shared_page[i] = -1;
      }
    }
    granted[i] = ok;
    if (FORK) {
      items[i].src = __ldcg(a + i);
      items[i].dst = s;
      if (!ok) items[i].len = 0;
      else c.lens[s] = items[i].len;
    } else if (ok) {
      if (shared_page[i] >= 0) {
        copies = true;
        atomicSub(c.refs + shared_page[i], 1);
        have[i] = __ldcg(c.page_table + static_cast<int64_t>(s) * c.max_pages + have[i]);  // the new page
        slot[i] = __ldcg(c.lens + s) & (c.page_size - 1);                                 // its tokens
      }
      c.lens[s] = __ldcg(b + i);
    }
  }
  if (FORK || !__syncthreads_or(copies)) return;
  for (int i = 0; i < n; ++i) {
    if (shared_page[i] < 0) continue;
    const int64_t from = static_cast<int64_t>(shared_page[i]) * c.page_size, to = static_cast<int64_t>(have[i]) * c.page_size;
    // a warp per layer and K or V
    for (int y = tid >> 5; y < 2 * c.layers; y += kBlock / 32)
      copy_bytes<8>(cache_row(c, y >> 1, y & 1, from), cache_row(c, y >> 1, y & 1, to), slot[i] * row_bytes(c), tid & 31, 32);
  }
}

// Block (i, 0) writes the table row and references of fork i; block (i, 1 + y) copies
// the tail's tokens of one layer's K or V.  A second launch, as the copies need blocks on every SM:
// 48 forks of 8 layers (with the freeing of their slots before) 15 us, 27 MB of them copies.  A source with
// a page out of range is found here, where its row is read: block (i, 0) takes the grant back.
__global__ void fork_kernel(const attn_cache_t c, const ForkItem* items, int32_t* granted, int* err) {
  let_next_launch();
  wait_for_previous();
  const int4 w = __ldcg(reinterpret_cast<const int4*>(items + blockIdx.x));
  ForkItem it;
  memcpy(&it, &w, sizeof(it));
  if (it.len <= 0) return;
  const int full = it.len / c.page_size, part = it.len & (c.page_size - 1);
  const int32_t* from = c.page_table + static_cast<int64_t>(it.src) * c.max_pages;
  if (blockIdx.y == 0) {
    int32_t* to = c.page_table + static_cast<int64_t>(it.dst) * c.max_pages;
    bool bad = false;
    for (int m = threadIdx.x; m < full + (part ? 1 : 0); m += blockDim.x) {
      const int p = __ldcg(from + m);
      bad |= p < 0 || p >= c.pages;
    }
    if (__syncthreads_or(bad)) {
      if (threadIdx.x == 0) {
        record_invalid(err, kSitePage);
        granted[blockIdx.x] = 0;
        c.lens[it.dst] = 0;
        if (part) c.refs[it.fresh] = 0;
      }
      return;
    }
    for (int m = threadIdx.x; m < full; m += blockDim.x) {
      const int p = __ldcg(from + m);
      atomicAdd(c.refs + p, 1);
      to[m] = p;
    }
    if (part && threadIdx.x == 0) to[full] = it.fresh;
    return;
  }
  if (!part) return;
  const int old = __ldcg(from + full);
  if (old < 0 || old >= c.pages) return;
  const int y = blockIdx.y - 1;
  copy_bytes<4>(cache_row(c, y >> 1, y & 1, static_cast<int64_t>(old) * c.page_size),
                cache_row(c, y >> 1, y & 1, static_cast<int64_t>(it.fresh) * c.page_size), part * row_bytes(c), threadIdx.x, blockDim.x);
}

__device__ __forceinline__ void drop(const attn_cache_t& c, int page, int* err) {
  if (page < 0 || page >= c.pages) {
    record_invalid(err, kSitePage);
  } else if (atomicSub(c.refs + page, 1) <= 0) {
    atomicAdd(c.refs + page, 1);
    record_invalid(err, kSitePage);
  }
}

// Takes a reference from entries [m0, m1) of a slot's table row and clears them: thread t of n.
__device__ __forceinline__ void release(const attn_cache_t& c, int slot, int m0, int m1, int t, int n, int* err) {
  int32_t* row = c.page_table + static_cast<int64_t>(slot) * c.max_pages;
  for (int m = m0 + t; m < m1; m += n) {
    const int p = __ldcg(row + m);
    row[m] = -1;
    drop(c, p, err);
  }
}

__global__ void free_kernel(const attn_cache_t c, const int32_t* slots, int* err) {
  __shared__ int len;
  let_next_launch();
  wait_for_previous();
  const int slot = __ldcg(slots + blockIdx.x);
  if (slot < 0 || slot >= c.slots) {
    if (threadIdx.x == 0) record_invalid(err, kSiteSlot);
    return;
  }
  // The first entries of the row load beside the length.
  int32_t* row = c.page_table + static_cast<int64_t>(slot) * c.max_pages;
  const int m = threadIdx.x;
  const int p = m < c.max_pages ? __ldcg(row + m) : 0;
  if (threadIdx.x == 0) len = atomicExch(c.lens + slot, 0);  // named twice: the second finds 0
  __syncthreads();
  if (len <= 0) return;
  const int count = min(pages_of(len, c.page_size), c.max_pages);
  if (m < count) {
    row[m] = -1;
    drop(c, p, err);
  }
  release(c, slot, blockDim.x, count, threadIdx.x, blockDim.x, err);
}

__global__ void copy_kernel(const attn_cache_t c, const int32_t* src, const int32_t* dst, int n, int chunks, int* err) {
  let_next_launch();
  wait_for_previous();
  const int i = blockIdx.x;
  const int from = __ldcg(src + i), to = __ldcg(dst + i);
  if (from < 0 || from >= c.pages || to < 0 || to >= c.pages) {
    if (threadIdx.x == 0) record_invalid(err, kSitePage);
    return;
  }
  if (from == to) return;
  bool later = false, written = false;
  for (int j = threadIdx.x; j < n; j += blockDim.x) {
    const int o = __ldcg(dst + j);
    const bool moves = __ldcg(src + j) != o;  // a page copied onto itself is not written
    later |= moves && j > i && o == to;
    written |= moves && o == from;
  }
  later = __syncthreads_or(later);
  written = __syncthreads_or(written);
  if (written && threadIdx.x == 0) record_invalid(err, kSiteCopyOverlap);
  if (later || written) return;
  const int64_t bytes = row_bytes(c) * c.page_size, part = bytes / chunks;
  for (int y = blockIdx.y; y < c.layers * 2 * chunks; y += gridDim.y) {
    const int lk = y / chunks, ch = y - lk * chunks;
    copy_bytes<4>(cache_row(c, lk >> 1, lk & 1, static_cast<int64_t>(from) * c.page_size) + ch * part,
                  cache_row(c, lk >> 1, lk & 1, static_cast<int64_t>(to) * c.page_size) + ch * part, part, threadIdx.x, blockDim.x);
  }
}

// What compact does with sequence b.  Both of its kernels decide it, from the same lengths, tables and
// reference counts: neither changes any of them before every sequence has been decided.
struct Kept {
  int slot, base, len, count;
};
// The share of thread t of n in the checks of sequence b: 0, or the site of what is wrong.
__device__ __forceinline__ int check_kept(const attn_cache_t& c, const int32_t* cu_q, const int32_t* path, int width,
                                          const int32_t* accepted, const int32_t* slots, int b, int t, int n, Kept& k) {
  k.slot = slots ? __ldcg(slots + b) : b;
  k.len = k.base = k.count = 0;
  if (k.slot < 0 || k.slot >= c.slots) return kSiteSlot;
  const int drafted = __ldcg(cu_q + b + 1) - __ldcg(cu_q + b);
  k.len = __ldcg(c.lens + k.slot);
  k.count = __ldcg(accepted + b);
  k.base = k.len - drafted;
  int bad = 0;
  if (drafted < 0 || k.base < 0 || k.len > static_cast<int64_t>(c.max_pages) * c.page_size) return kSiteLength;
  if (k.count < 0 || k.count > drafted || k.count > width) return kSitePath;
  const int32_t* row = path + static_cast<int64_t>(b) * width;
  for (int i = t; i < k.count; i += n) {
    const int p = row[i];  // by way of L1: read again for the moves
    if (p < i || p >= drafted || p <= (i ? row[i - 1] : -1)) {  // increasing from 0 on, so never below i
      bad = kSitePath;
    } else if (p != i) {  // a token moves: from a page of the cache, to one that no other slot holds
      const int32_t* table = c.page_table + static_cast<int64_t>(k.slot) * c.max_pages;
      const int from = __ldcg(table + (k.base + p) / c.page_size), to = __ldcg(table + (k.base + i) / c.page_size);
      if (from < 0 || from >= c.pages || to < 0 || to >= c.pages || __ldcg(c.refs + to) != 1) bad = kSitePage;
    }
  }
  for (int j = t; slots && j < b; j += n)
    if (__ldcg(slots + j) == k.slot) bad = kSiteSlot;
  return bad;
}

constexpr int kMoves = 128;  // moves whose rows are looked up together

// Block (b, layer and K/V, columns): moves the accepted tokens' rows.  A thread owns 16
// bytes of the row and takes the moves in order.  Move i reads position path[i] >= i and
// writes position i, so no later move reads what an earlier one wrote: the reads of 8
// moves may go before their writes.  The release is a launch of its own, as the blocks of all layers
// read the table.  64 trees, 8 layers, with the grant before: 18.4 us, bound by latency.
__global__ void compact_kernel(const attn_cache_t c, const int32_t* cu_q, const int32_t* path, int width,
                               const int32_t* accepted, const int32_t* slots) {
  __shared__ int64_t from[kMoves], to[kMoves];
  let_next_launch();
  wait_for_previous();
  const int b = blockIdx.x;
  Kept k;
  const int bad = check_kept(c, cu_q, path, width, accepted, slots, b, threadIdx.x, blockDim.x, k);  // cut_kernel reports it
  if (__syncthreads_or(bad)) return;
  const int l = blockIdx.y >> 1, kv = blockIdx.y & 1;
  const int64_t rb = row_bytes(c);
  const int64_t col = (static_cast<int64_t>(blockIdx.z) * blockDim.x + threadIdx.x) * 16;
  uint8_t* base = cache_row(c, l, kv, 0) + col;
  const int32_t* row = c.page_table + static_cast<int64_t>(k.slot) * c.max_pages;
  for (int m0 = 0; m0 < k.count; m0 += kMoves) {
    const int m = min(kMoves, k.count - m0);
    __syncthreads();
    for (int i = threadIdx.x; i < m; i += blockDim.x) {
      const int x = k.base + path[static_cast<int64_t>(b) * width + m0 + i], y = k.base + m0 + i;
      // the pages of tokens that move have been checked
      from[i] = x == y ? -1 : static_cast<int64_t>(__ldcg(row + x / c.page_size)) * c.page_size + (x & (c.page_size - 1));
      to[i] = static_cast<int64_t>(__ldcg(row + y / c.page_size)) * c.page_size + (y & (c.page_size - 1));
    }
    __syncthreads();
    if (col >= rb) continue;
    for (int i = 0; i < m; i += 8) {
      uint4 w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j < m && from[i + j] >= 0) w[j] = __ldcg(reinterpret_cast<const uint4*>(base + from[i + j] * rb));
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j < m && from[i + j] >= 0) *reinterpret_cast<uint4*>(base + to[i + j] * rb) = w[j];
    }
  }
}

// A warp per sequence, in one cluster of blocks: releasing pages changes the reference counts that other
// sequences' checks read (two slots that share a page may be in one call), so the first page is
// released when all sequences have been decided.
constexpr int kCutWarps = 32, kCutBlocks = 8, kCutEach = kMaxSequences / (kCutWarps * kCutBlocks);
__global__ void __launch_bounds__(kCutWarps * 32) cut_kernel(const attn_cache_t c, const int32_t* cu_q, const int32_t* path,
                                                            int width, const int32_t* accepted, const int32_t* slots, int B,
                                                            int* err) {
  __shared__ Kept kept[kCutWarps][kCutEach];
  let_next_launch();
  wait_for_previous();  // the moves have read the table
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int n = 0;
  for (int b = blockIdx.x * kCutWarps + warp; b < B; b += gridDim.x * kCutWarps, ++n) {
    Kept k;
    const int bad = check_kept(c, cu_q, path, width, accepted, slots, b, lane, 32, k);
    if (bad) record_invalid(err, bad);
    if (__any_sync(0xffffffffu, bad)) k.slot = -1;
    if (lane == 0) kept[warp][n] = k;
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  for (int i = 0; i < n; ++i) {
    const Kept k = kept[warp][i];
    if (k.slot < 0) continue;
    if (lane == 0) c.lens[k.slot] = k.base + k.count;
    release(c, k.slot, pages_of(k.base + k.count, c.page_size), pages_of(k.len, c.page_size), lane, 32, err);
  }
}

}  // namespace

// The lists of grant_kernel, one of slots and those of requests, are raised to the most that any call needs
// (8192 of each), never to this call's own size, which another thread's smaller call would lower again
// before the launch.
static cudaError_t grant_smem(const void* kern, size_t smem) {
  constexpr int most = 8192 * (sizeof(int64_t) + 4 * sizeof(int));
  return smem > 40 * 1024 ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most) : cudaSuccess;
}

cudaError_t launch_alloc(const attn_cache_t& c, const int32_t* slots, const int32_t* want, int n, int32_t* granted,
                         int* err, cudaStream_t st) {
  const size_t smem = (static_cast<size_t>(c.slots) + 3 * n) * sizeof(int) + n * sizeof(int64_t);
  const cudaError_t e = grant_smem(reinterpret_cast<const void*>(grant_kernel<false>), smem);
  if (e != cudaSuccess) return e;
  return launch_after(grant_kernel<false>, 1, kBlock, smem, st, c, slots, want, n, granted, static_cast<ForkItem*>(nullptr), err);
}

cudaError_t launch_free(const attn_cache_t& c, const int32_t* slots, int n, int* err, cudaStream_t st) {
  return launch_after(free_kernel, n, 128, 0, st, c, slots, err);
}

cudaError_t launch_fork(const attn_cache_t& c, const int32_t* src, const int32_t* dst, int n, int32_t* granted,
                        void* ws, int* err, cudaStream_t st) {
  const size_t smem = (static_cast<size_t>(c.slots) + 2 * n) * sizeof(int) + n * sizeof(int64_t);
  cudaError_t e = grant_smem(reinterpret_cast<const void*>(grant_kernel<true>), smem);
  if (e != cudaSuccess) return e;
  ForkItem* items = static_cast<ForkItem*>(ws);
  e = launch_after(grant_kernel<true>, 1, kBlock, smem, st, c, src, dst, n, granted, items, err);
  if (e != cudaSuccess) return e;
  return launch_after(fork_kernel, dim3(n, 1 + 2 * c.layers), 256, 0, st, c, items, granted, err);
}

cudaError_t launch_copy(const attn_cache_t& c, const int32_t* src, const int32_t* dst, int n, int* err, cudaStream_t st) {
  // A block reads the whole list of destinations, so there are no more blocks than fill
  // the device: about 4096, in pieces of at least 4 KB (page_size >= 16 rows of 64 bytes
  // or more divide evenly into the powers of two used here).
  const int64_t bytes = static_cast<int64_t>(c.heads) * c.d * (c.e4m3 ? 1 : 2) * c.page_size;
  int chunks = 1;
  while (chunks < 16 && bytes / (2 * chunks) >= 4096 && static_cast<int64_t>(n) * c.layers * 2 * chunks < 4096) chunks *= 2;
  int parts = 4096 / n;
  if (parts > c.layers * 2 * chunks) parts = c.layers * 2 * chunks;
  if (parts < 1) parts = 1;
  return launch_after(copy_kernel, dim3(n, parts), 256, 0, st, c, src, dst, n, chunks, err);
}

cudaError_t launch_compact(const attn_cache_t& c, const int32_t* cu_q, const int32_t* path, int width,
                           const int32_t* accepted, const int32_t* slots, int B, int* err, cudaStream_t st) {
  const int64_t words = static_cast<int64_t>(c.heads) * c.d * (c.e4m3 ? 1 : 2) / 16;
  const int threads = words >= 256 ? 256 : static_cast<int>((words + 31) / 32 * 32);
  const int z = static_cast<int>((words + threads - 1) / threads);
  const cudaError_t e = launch_after(compact_kernel, dim3(B, 2 * c.layers, z), threads, 0, st, c, cu_q, path, width, accepted, slots);
  if (e != cudaSuccess) return e;
  int blocks = 1;  // of the cluster: a power of two
  while (blocks < kCutBlocks && blocks * kCutWarps < B) blocks *= 2;
  return launch_clusters_after(cut_kernel, blocks, blocks, kCutWarps * 32, 0, st, c, cu_q, path, width, accepted, slots, B, err);
}

}  // namespace attn
