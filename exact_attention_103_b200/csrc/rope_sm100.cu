// rope_sm100.cu -- rotary positions: q and k rotated in one launch (forward, and by the
// negative angles the gradient), and the serving form that also writes k and v into the
// pages of the cache.
//
// A pair (a, b) at position p turns by p * f:  (a cos - b sin, b cos + a sin) * amplitude.
// The angle as a fraction of a turn is p * turns modulo 2^64 in integer arithmetic: exact
// at every position, where an fp32 product would have lost the fraction by p = 2^24.
// Its upper 32 bits go to sincospif (angle error below 1e-7).  The arithmetic is fp32; each
// result is rounded once to its type.
//
// Bound by HBM: every value is read once and written once.  A block takes a few whole
// tokens, so that one table of their sines (in shared memory) serves all their heads, and
// moves 16 values of one head per thread and step with 16-byte accesses.  Measured (B200, a call with cold inputs /
// a replayed graph): 2 x 8192 tokens, 16 + 16 heads, d 128, bf16: 48.3 / 46.8 us, 85% / 88% of the copy rate; a
// packed batch of 16 sequences of 512 to 16384 tokens, half of each head rotated: 210 / 198 us, 89% / 94%.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "cache_ops.h"

namespace attn {
namespace {

constexpr int kThreads = 128;        // rope; 256 took 48 and 202 us for the two above
constexpr int kAppendThreads = 256;  // append
constexpr int kAhead = 2;            // append: rows whose loads go together (1: 10.9, 3: 12.0 us for the trees)
constexpr int kMaxTok = 16;
constexpr int kPitch = 20;  // floats of a table chunk: 8 (cos, sin) pairs, padded so that 8
                            // neighbouring chunks read as 16-byte words meet no bank twice

__device__ __forceinline__ void widen(uint4 w, float (&x)[8]) {  // 8 bf16
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(v[i] << 16);
    x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
  }
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = __ldcg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[8]) {
  widen(*reinterpret_cast<const uint4*>(p), x);
}
template <>
__device__ __forceinline__ void load8<__half>(const __half* p, float (&x)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    v[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(v[0], v[1], v[2], v[3]);
}
template <>
__device__ __forceinline__ void store8<__half>(__half* p, const float (&x)[8]) {
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    v[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(v[0], v[1], v[2], v[3]);
}

// 8 values as E4M3 bytes (nearest even, saturating).
__device__ __forceinline__ void store8_e4m3(uint8_t* p, const float (&x)[8]) {
  uint32_t v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint16_t lo, hi;  // cvt packs its first source into the upper byte
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[4 * i + 1]), "f"(x[4 * i]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[4 * i + 3]), "f"(x[4 * i + 2]));
    v[i] = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  }
  *reinterpret_cast<uint2*>(p) = make_uint2(v[0], v[1]);
}

// The sequence of packed token t: cu[b] <= t < cu[b + 1] (cu non-decreasing); -1 if none.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, int t) {
  if (B == 0 || t < cu[0] || t >= cu[B]) return -1;
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid + 1] > t) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// What a block knows of one of its tokens.
struct Token {
  int live;       // 0: left alone
  int pos;        // rotary position
  int64_t b, n;   // batch and token index of the row strides
  int64_t row;    // append: row of the cache (page * page_size + offset); -1: none
};

// 16 values of a head: chunk u of a rotated head is pairs 8u..8u+7 (values 8u.. and
// dim/2 + 8u.., or 16u.. when interleaved); behind `dim` values 16u.. pass through.
struct Unit {
  int first, second;  // offsets of its two groups of 8
  bool turn;
};
__device__ __forceinline__ Unit unit_at(int u, int dim, bool inter) {
  Unit k;
  k.turn = 16 * u < dim;
  k.first = (k.turn && !inter) ? 8 * u : 16 * u;
  k.second = (k.turn && !inter) ? dim / 2 + 8 * u : 16 * u + 8;
  return k;
}

__device__ __forceinline__ void turn(float (&x)[8], float (&y)[8], const float* cs, bool inter) {
  float c[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 w = reinterpret_cast<const float4*>(cs)[i];
    c[4 * i] = w.x; c[4 * i + 1] = w.y; c[4 * i + 2] = w.z; c[4 * i + 3] = w.w;
  }
  if (inter) {  // x holds pairs 0..3 of the chunk, y pairs 4..7
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1], e = y[2 * i], f = y[2 * i + 1];
      x[2 * i] = a * c[2 * i] - b * c[2 * i + 1];
      x[2 * i + 1] = b * c[2 * i] + a * c[2 * i + 1];
      y[2 * i] = e * c[8 + 2 * i] - f * c[9 + 2 * i];
      y[2 * i + 1] = f * c[8 + 2 * i] + e * c[9 + 2 * i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[i], b = y[i];
      x[i] = a * c[2 * i] - b * c[2 * i + 1];
      y[i] = b * c[2 * i] + a * c[2 * i + 1];
    }
  }
}

// The sines of a block's tokens, one chunk of 8 pairs behind the other.
__device__ __forceinline__ void fill_table(float* table, const Token* tok, int ntok, const RopeArgs& a, int threads) {
  const int half = a.plan.dim / 2;
  const float sign = a.inverse ? -1.f : 1.f;
  for (int i = threadIdx.x; i < ntok * half; i += threads) {
    const int k = i / half, f = i - k * half;
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(tok[k].pos)) * a.plan.turns[f];
    const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(half_turns, &s, &c);
    float* out = table + (k * (half / 8) + (f >> 3)) * kPitch + 2 * (f & 7);
    out[0] = c * a.plan.amplitude;
    out[1] = s * a.plan.amplitude * sign;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a, int per_block, int count) {
  extern __shared__ float table[];
  __shared__ Token tok[kMaxTok];
  wait_for_previous();
  const int t0 = blockIdx.x * per_block;
  const int ntok = min(per_block, a.tokens - t0);
  if (threadIdx.x < ntok) {
    const int t = t0 + threadIdx.x;
    Token k;
    k.live = 1;
    k.b = 0;
    k.n = t;
    if (a.cu == nullptr) {
      k.b = t / a.N;
      k.n = t - k.b * a.N;
    }
    k.pos = static_cast<int>(k.n);
    if (a.positions) {
      k.pos = __ldcg(a.positions + t);
    } else if (a.cu) {
      const int b = sequence_of(a.cu, a.B, t);
      k.live = b >= 0;
      if (b >= 0) k.pos = t - __ldcg(a.cu + b);
    }
    tok[threadIdx.x] = k;
  }
  __syncthreads();
  fill_table(table, tok, ntok, a, kThreads);
  __syncthreads();
  const int units = a.d / 16, heads = a.t[0].heads + (count > 1 ? a.t[1].heads : 0);
  const int lanes = kThreads / units;  // rows in flight; threads behind lanes * units idle
  const int u = threadIdx.x % units;
  if (static_cast<int>(threadIdx.x) >= lanes * units) return;
  const Unit k = unit_at(u, a.plan.dim, a.plan.interleaved);
  for (int r = threadIdx.x / units; r < ntok * heads; r += lanes) {
    const int ti = r / heads;
    int h = r - ti * heads;
    const bool second = h >= a.t[0].heads;
    if (second) h -= a.t[0].heads;
    const attn_rows_t& w = a.t[second ? 1 : 0];
    const Token& tk = tok[ti];
    if (!tk.live) continue;
    const T* src = static_cast<const T*>(w.src) + tk.b * w.src_batch + tk.n * w.src_token + h * w.src_head;
    T* dst = static_cast<T*>(w.dst) + tk.b * w.dst_batch + tk.n * w.dst_token + h * w.dst_head;
    if (!k.turn && src == dst) continue;  // in place: what passes through stays
    float x[8], y[8];
    load8<T>(src + k.first, x);
    load8<T>(src + k.second, y);
    if (k.turn) turn(x, y, table + (ti * (a.plan.dim / 16) + u) * kPitch, a.plan.interleaved);
    store8<T>(dst + k.first, x);
    store8<T>(dst + k.second, y);
  }
}

// Append: rows of q, k, v of each token, in that order (none of a token that has no row in the cache).  Rotated keys and the values go to
// the token's row of the cache.  A step of decoding has few tokens, so what counts is the
// chain of loads behind one another: offsets, slots and the first rows come together
// (each block takes all offsets and slots into shared memory), then lengths, then pages.
// The rows of all tokens are dealt evenly to one wave of blocks.  Measured: 48 single tokens of 32 +
// 8 + 8 heads 3.9 us; 32 trees of 61 tokens into an E4M3 cache 11.4 us (31 MB: 4.8 at the copy
// rate, the rest is that chain).
template <bool F8>
__global__ void __launch_bounds__(kAppendThreads, 4) append_kernel(const __grid_constant__ RopeArgs a, int per_block) {
  extern __shared__ float table[];
  __shared__ Token tok[kMaxTok];
  __shared__ int cu[kMaxSequences + 1], slots[kMaxSequences];
  __shared__ int again[kMaxTok];  // the token's slot is named by an earlier sequence too
  using T = __nv_bfloat16;
  let_next_launch();
  const attn_cache_t& c = a.cache;
  const int hq = a.t[0].heads, hk = c.heads, heads = hq + 2 * hk;
  const int64_t rows = static_cast<int64_t>(a.tokens) * heads, row0 = static_cast<int64_t>(blockIdx.x) * per_block;
  const int t0 = static_cast<int>(row0 / heads);
  const int r0 = static_cast<int>(row0 - static_cast<int64_t>(t0) * heads);  // rows count from token t0's first
  const int r1 = r0 + static_cast<int>(min(static_cast<int64_t>(per_block), rows - row0));
  const int ntok = (r1 + heads - 1) / heads;
  const bool rotate = a.plan.turns != nullptr;
  const int units = a.d / 16, lanes = kAppendThreads / units;
  const int u = threadIdx.x % units;
  const Unit turned = unit_at(u, rotate ? a.plan.dim : 0, a.plan.interleaved);
  const Unit plain = unit_at(u, 0, false);
  struct Row {
    int ti, which, h;
  };
  auto row_at = [&](int r) {
    Row k;
    k.ti = r / heads;
    const int hh = r - k.ti * heads;
    k.which = hh < hq ? 0 : hh < hq + hk ? 1 : 2;
    k.h = k.which == 0 ? hh : k.which == 1 ? hh - hq : hh - hq - hk;
    return k;
  };
  uint4 raw[kAhead][2];  // the next rows' values
  auto fetch = [&](int r) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i, r += lanes) {
      if (r >= r1) break;
      const Row k = row_at(r);
      const attn_rows_t& w = a.t[k.which];
      const Unit& n = k.which == 2 ? plain : turned;
      const T* src = static_cast<const T*>(w.src) + static_cast<int64_t>(t0 + k.ti) * w.src_token + k.h * w.src_head;
      raw[i][0] = *reinterpret_cast<const uint4*>(src + n.first);
      raw[i][1] = *reinterpret_cast<const uint4*>(src + n.second);
    }
  };
  wait_for_previous();
  int r = r0 + static_cast<int>(threadIdx.x) / units;
  fetch(r);
  for (int b = threadIdx.x; b <= a.B; b += kAppendThreads) {
    cu[b] = __ldcg(a.cu + b);
    if (b < a.B) slots[b] = a.slots ? __ldcg(a.slots + b) : b;
  }
  if (threadIdx.x < kMaxTok) again[threadIdx.x] = 0;
  __syncthreads();
  if (threadIdx.x < ntok) {
    const int t = t0 + threadIdx.x;
    Token k;
    k.b = 0;
    k.n = t;
    k.row = -1;
    k.pos = 0;
    const int b = sequence_of(cu, a.B, t);
    k.live = b >= 0;
    if (b >= 0) {
      k.b = b;
      const int slot = slots[b];
      const int first = cu[b], n = cu[b + 1] - first;
      if (a.positions) k.pos = __ldcg(a.positions + t);
      if (slot < 0 || slot >= c.slots) {
        record_invalid(a.err, kSiteSlot);
      } else {
        const int len = __ldcg(c.lens + slot);
        const int64_t p = static_cast<int64_t>(len) - n + (t - first);
        if (t < first || t - first >= n || len < n ||
            len > static_cast<int64_t>(c.max_pages) * c.page_size) {
          record_invalid(a.err, kSiteLength);
        } else {
          const int in_page = static_cast<int>(p) & (c.page_size - 1);
          const int page = __ldcg(c.page_table + static_cast<int64_t>(slot) * c.max_pages + p / c.page_size);
          if (page < 0 || page >= c.pages) record_invalid(a.err, kSitePage);
          else k.row = static_cast<int64_t>(page) * c.page_size + in_page;
          if (!a.positions) k.pos = static_cast<int>(p);
        }
      }
    }
    tok[threadIdx.x] = k;
  }
  __syncthreads();
  if (a.slots) {
    // Two sequences with one slot would write the same rows: the first one counts.
    for (int i = 0; i < ntok; ++i) {
      if (!tok[i].live) continue;
      const int b = static_cast<int>(tok[i].b), slot = slots[b];
      if (i > 0 && tok[i - 1].live && tok[i - 1].b == b) continue;  // seen with its first token
      for (int j = threadIdx.x; j < b; j += kAppendThreads)
        if (slots[j] == slot && cu[j + 1] > cu[j])
          for (int x = i; x < ntok && tok[x].live && tok[x].b == b; ++x) again[x] = 1;
    }
  }
  if (rotate) fill_table(table, tok, ntok, a, kAppendThreads);
  __syncthreads();
  if (threadIdx.x < ntok && again[threadIdx.x]) record_invalid(a.err, kSiteSlot);
  const int64_t cache_row = static_cast<int64_t>(hk) * a.d;
  const int64_t layer0 = static_cast<int64_t>(a.layer) * c.pages * c.page_size;
  while (r < r1) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i, r += lanes) {
      if (r >= r1) break;
      const Row row = row_at(r);
      const Token& tk = tok[row.ti];
      if (tk.row < 0 || again[row.ti]) continue;  // of no sequence, or of one that cannot be appended
      const Unit& k = row.which == 2 ? plain : turned;
      float x[8], y[8];
      widen(raw[i][0], x);
      widen(raw[i][1], y);
      if (k.turn) turn(x, y, table + (row.ti * (a.plan.dim / 16) + u) * kPitch, a.plan.interleaved);
      if (row.which == 0) {
        const attn_rows_t& w = a.t[0];
        T* dst = static_cast<T*>(w.dst) + tk.n * w.dst_token + row.h * w.dst_head;
        store8<T>(dst + k.first, x);
        store8<T>(dst + k.second, y);
        continue;
      }
      void* base = row.which == 1 ? c.k : c.v;
      const int64_t at = (layer0 + tk.row) * cache_row + row.h * a.d;
      if constexpr (F8) {
        const float scale = row.which == 1 ? c.k_scale : c.v_scale;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = __fdiv_rn(x[i], scale);
          y[i] = __fdiv_rn(y[i], scale);
        }
        store8_e4m3(static_cast<uint8_t*>(base) + at + k.first, x);
        store8_e4m3(static_cast<uint8_t*>(base) + at + k.second, y);
      } else {
        store8<T>(static_cast<T*>(base) + at + k.first, x);
        store8<T>(static_cast<T*>(base) + at + k.second, y);
      }
    }
    fetch(r);
  }
}

// rope: tokens of a block: enough rows for eight steps of a block (four: 207 us for the packed batch,
// sixteen: 54 for the dense one), fewer when that would leave SMs without a block.
int tokens_per_block(int tokens, int rows_per_token, int d, int sms) {
  const int lanes = kThreads / (d / 16);
  int per = 8 * lanes / rows_per_token;
  if (per > tokens / (2 * sms)) per = tokens / (2 * sms);
  return per < 1 ? 1 : per > kMaxTok ? kMaxTok : per;
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, attn_type_t type, int sms, cudaStream_t st) {
  const int count = a.t[1].heads > 0 ? 2 : 1;
  const int per = tokens_per_block(a.tokens, a.t[0].heads + a.t[1].heads, a.d, sms);
  const int grid = (a.tokens + per - 1) / per;
  const size_t smem = static_cast<size_t>(per) * (a.plan.dim / 16) * kPitch * sizeof(float);
  if (type == ATTN_FP32) return launch_after(rope_kernel<float>, grid, kThreads, smem, st, a, per, count);
  if (type == ATTN_FP16) return launch_after(rope_kernel<__half>, grid, kThreads, smem, st, a, per, count);
  return launch_after(rope_kernel<__nv_bfloat16>, grid, kThreads, smem, st, a, per, count);
}

cudaError_t launch_append(const RopeArgs& a, int sms, cudaStream_t st) {
  // Rows of a block: one wave of four blocks on an SM, in whole steps; no more tokens than a
  // block keeps (its first and last may be parts).
  const int heads = a.t[0].heads + 2 * a.cache.heads;
  const int64_t lanes = kAppendThreads / (a.d / 16), rows = static_cast<int64_t>(a.tokens) * heads;
  int64_t per = (rows + 4 * sms - 1) / (4 * sms);
  per = (per + lanes - 1) / lanes * lanes;
  const int64_t most = static_cast<int64_t>(kMaxTok - 1) * heads;
  if (per > most) per = most;
  if (per > 8 * lanes) per = 8 * lanes;
  const int64_t grid = (rows + per - 1) / per;
  const int64_t ntok = (per + heads - 2) / heads + 1;
  const size_t smem = a.plan.turns ? static_cast<size_t>(ntok) * (a.plan.dim / 16) * kPitch * sizeof(float) : 0;
  return launch_after(a.cache.e4m3 ? append_kernel<true> : append_kernel<false>, static_cast<unsigned>(grid), kAppendThreads,
                      smem, st, a, static_cast<int>(per));
}

}  // namespace attn
