// attn_tree_sm100.cu -- exact attention of each sequence's newest (drafted) tokens over
// the paged cache, for B200 (sm_100a): tree_kernel, and combine_kernel for the rows whose keys
// were split over several CTAs.
//
// The mathematics is the forward kernel's (attn_fwd_sm100.cu): O = sum_j 2^(x_j - m) v_j /
// sum_j 2^(x_j - m), x = scale log2(e) q.k, one pass over the keys with a running
// maximum m per row, rescaled only when it grows by more than tau.
//
// What bounds it: a cache is read once per step, 2 d values per (token, cache head), for
// 4 d flops per query row: below about 128 query rows per cache head the copies from HBM bound
// it, above the tensor cores.  Hence:
//  - The query heads that share a cache head, and all drafted tokens, are packed into the rows
//    of one item: row r of a 128-row tile is token r / G, head r % G of the group (G = Hq /
//    heads), so K and V are read once for all of them.
//  - Work is dealt in equal costs: the 128-key tiles of all (sequence, cache head, row pair)
//    items form one list, and CTA c of the grid takes the c-th equal part.  One long
//    sequence fills every SM as well as many short ones do.  A part that begins or ends
//    inside an item leaves its rows' unnormalised O (fp32), maximum and sum in the workspace; a
//    CTA leaves at most two of those.  combine_kernel joins them in a fixed order.
//  - An item of up to 128 rows gives each of the two softmax warpgroups (streams, with an O of
//    their own in TMEM, joined at the end) one half of every key tile, so that one's softmax
//    overlaps the other's products.  An item of 129 to 256 rows gives each its own 128 rows of every
//    key tile.
//  - Few rows leave most threads of a row-per-thread softmax idle: up to 32 rows the scores are
//    computed transposed, a key per thread (swapped items).
//
// E4M3 caches: the keys and values go to the tensor cores as they are (kind::f8f6f4), and the
// other operand of each product is a sum of 8-bit terms that keeps bf16's precision.  A bf16 query
// scaled by a power of two (its row's largest value in [128, 256)) is hi + lo, two E4M3 terms, to
// 2^-17 of the row's largest value.  P~ needs E4M3's precision over far more than its range, as many small
// weights beside a large one may hold most of a row: it is rounded to fp16 and split into three E5M2
// terms (3 bits each), off by 2^-9 of itself or 2^-28 of the row's reference.  (Two E4M3 terms lost
// every weight below 2^-14 of the reference: of a row with one key 10 nats above the others, up to 57% of O.)  A term
// costs one more product, at twice bf16's rate; up to 64 rows the first two are rows of one product (duo
// items) and up to 32 all of them are columns of one (swapped items).
//
// Warp roles (384 threads): 0-3 and 4-7 softmax, correction and epilogue of streams 0 and 1;
// 8 and 10 TMA producers of K (and q) and of V; 9 (TMEM owner) and 11 issue S and P~V.  The softmax
// warps write an E4M3 cache's split queries.  Every wait is bounded; on expiry the CTA stops, drains its
// copies and products, frees TMEM and returns.
//
// Measured (B200, Hq 32, 8 cache heads, d 128, us of a call with cold inputs / of a replayed graph; share of the
// copies' time at the measured bandwidth): 64 ragged contexts of 512 to 8192, one token, bf16: 145 / 145
// (86%).  Two contexts of 131072, 64 rows, E4M3: 172 / 143 (46% / 55%; per key tile the chain S -> softmax -> P~V
// -> next S, and 1.2 times the cache's bytes are read: rows of 128 bytes, fetched in pairs).  A call of little work:
// 15 / 12, two launches and about seven round trips to memory behind one another.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "attn_internal.h"
#include "cache_ops.h"
#include "cache_ptx.cuh"

namespace attn {
namespace {

constexpr int kThreads = 384;
constexpr int kBM = 128;  // rows of a tile
constexpr int kBN = 128;  // keys of a tile
constexpr float kLn2 = 0.693147180559945309f;
constexpr uint64_t kTimeoutNs = 2000000000ull;

enum TreeSite : int {  // wait sites of the device error word (16..30)
  kSiteTQFull = 16, kSiteTQEmpty, kSiteTKvFull, kSiteTKvEmpty, kSiteTSFull, kSiteTPFull, kSiteTOFull, kSiteTMerge,
  kSiteTDrain, kSiteTPvDone, kSiteTSFree,
  kSiteTItems
};
__host__ __device__ constexpr int timeout_code(int site) { return 4 | (site << 8); }

// Items of at most this many rows compute transposed scores.  Measured (64 sequences of 2000 tokens, 32 rows,
// us, transposed and not): bf16 d 128 133, 141, d 64 99, 111; E4M3 d 128 129, 143, d 64 102, 109.  64 rows (8
// sequences of 8192 tokens, bf16 / E4M3 while that had two terms of P~): 80 / 81 transposed, 73 / 68 as one row
// tile, where every row has a thread and its reference stays in a register.
constexpr int kSwapped = 32;
// E4M3 items above that and up to 64 rows: see Seg::duo.  Measured (two contexts of 131072, 64 rows,
// us): 188 with every term as a product of its own, 168; d 64 170, 140.
constexpr int kDuo = 64;
constexpr int kMinPart = 7;  // no CTA takes less of the list: the longest tile

struct TreeParams {
  __nv_bfloat16* o;
  float* lse;
  const __nv_bfloat16* q;
  const int32_t *cu, *slots, *page_table, *lens;
  const uint8_t* mask;
  int mask_width;
  int Hq, heads, G, B, T;
  int nslots, max_pages, pages, page_shift;
  int layer_row;   // first row of the layer in the tensor maps
  int rows;        // rows of the tensor maps: a copy from there on gives zeros
  int box_rows;    // rows of one K/V copy: min(page size, 128)
  int tpt;         // tokens of a 128-row tile: 128 / G
  int tpt32;       // tokens of a swapped item's copy of q: kSwapped / G
  uint32_t inv_g;  // ceil(2^32 / G): rows up to 2^24 are divided by its high product; 0: G = 1
  float scale_log2, o_scale, tau, p_shift;
  float* part;     // [grid][2][D / 4][256][4] unnormalised O: four columns of neighbouring rows
                   // lie together, as the lanes that write and join them are neighbouring rows
  float2* stat;    // [grid][2][256] (maximum in log2 units, sum; sum -1: a page was out of range)
  int4* head;      // [grid] the item whose first tiles this CTA left unfinished
  int* err;
};

// head[c]: x = row of q of its first token (-1: none), y = cache head, z = tokens, w = last CTA.

template <int D, bool F8>
struct Layout {
  static constexpr int ESZ = F8 ? 1 : 2;
  static constexpr int ROWB = D * ESZ < 128 ? D * ESZ : 128;  // bytes of a row in one swizzled chunk
  static constexpr int NCHUNK = D * ESZ / ROWB;
  static constexpr int CHUNK = kBM * ROWB;
  static constexpr int TILE = NCHUNK * CHUNK;
  static constexpr int CELEMS = ROWB / ESZ;  // values of a row in a chunk
  static constexpr int KSTEP = 32 / ESZ;     // values of a K step of the products
  // Two rings, K's slots first: each has one producer and one consumer that take its slots in
  // order, so that no role is ever a whole round ahead of a barrier's parity.
  static constexpr int NRING = TILE >= 32768 ? 2 : 4;
  static constexpr int NSTAGE = 2 * NRING;
  static constexpr int QTILE = F8 ? 2 * TILE : TILE;  // E4M3: hi, then lo
  static constexpr int Q_OFF = 0;
  static constexpr int KV_OFF = 2 * QTILE;
  // P~ of swapped items, [128 keys][128 bytes] per stream.  With d = 128 it lies where a tile of q
  // keeps rows that swapped items do not have: see p_row.
  static constexpr int P_OFF = KV_OFF + NSTAGE * TILE;
  static constexpr int ML_OFF = P_OFF + (D == 64 ? 2 * 16384 : 0);  // float2 [2][128]: (m, l) of the two streams
  static constexpr int QS_OFF = ML_OFF + 2 * kBM * 8;  // float [2][128]: factors of the scores (split queries)
  // swapped items, per stream: -m_ref + p_shift, rescale factors, m_ref, (row sums by warp, then the
  // weights of the streams): float [64] each, the last [4][64]; then four vote flags
  static constexpr int SW_OFF = QS_OFF + 2 * kBM * 4;
  static constexpr int SW_STREAM = 7 * 64 + 4;
  static constexpr int BAR_OFF = SW_OFF + 2 * SW_STREAM * 4;
  // SFULL, PFULL, PVDONE: one per S buffer; DRAIN: one per issuing warp
  // The W forms are those of swapped items, one per stream; WG: the four warps of a stream.
  static constexpr int B_QFULL = 0, B_QEMPTY = 2, B_SFULL = 4, B_PFULL = 8, B_PVDONE = 12, B_OFULL = 16, B_ML = 17,
                       B_EPI = 18, B_DRAIN = 19, B_WSFULL = 21, B_WSFREE = 23, B_WPFULL = 25, B_WPVDONE = 27, B_WG = 29,
                       B_KVFULL = 31, B_KVEMPTY = B_KVFULL + NSTAGE, NBARS = B_KVEMPTY + NSTAGE;
  static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;
  static constexpr int TABLE_OFF = MISC_OFF + 128;
  // Cost of a key tile with one and with two row tiles, and of beginning an item (its mask, queries
  // and epilogue), in units of about 1000 to 1300 cycles, as homogeneous batches and then mixed ones
  // measured.  With an item at 12, 20, 28 (bf16 d 128, us): 256 single tokens over 50 to 2000 167, 157,
  // 161; 16 trees of 48 tokens 118, 113, 113; 128 single tokens over 100 to 4000 112, 115, 120.  At 8, 10, 12
  // (bf16 d 64): 158, 152, 150; 154, 152, 149; 111, 110, 103; 64 single tokens over 512 to 8192 96, 97, 100.  At
  // 16, 20, 24 (E4M3, d 128 / d 64): 184, 186, 184 / 158, 160, 158; 201, 195, 192 / 162, 166, 168; 120, 125, 123 / 104,
  // 104, 102; 64 single tokens 104, 104, 106 / 83, 84, 84.
  static constexpr int COST_ONE = !F8 && D == 128 ? 4 : 2, COST_PAIR = !F8 && D == 128 ? 7 : 4,
                       COST_ITEM = F8 || D == 128 ? 20 : 10;
  static constexpr int P_TERMS = F8 ? 3 : 1;  // products that P~V is the sum of
  static constexpr int TM_S = 0, TM_O0 = 256, TM_O1 = 384;  // S: four buffers of 64 columns
  // Row `key` of stream s's P~ (a swapped item's), from the shared-memory base.
  __host__ __device__ static constexpr int p_row(int s, int key) {
    return D == 64 ? P_OFF + s * 16384 + key * 128
           : F8    ? Q_OFF + s * QTILE + TILE + key * 128
                   : Q_OFF + s * QTILE + (key >> 6) * CHUNK + 64 * 128 + (key & 63) * 128;
  }
};

__device__ __forceinline__ int token_of(int row, const TreeParams& p) {  // row / G
  return p.inv_g ? static_cast<int>(__umulhi(static_cast<uint32_t>(row), p.inv_g)) : row;
}
__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// One CTA's stretch of an item: key tiles [j0, j1) of kvt (none if j0 >= j1).
struct Seg {
  int h, tok0, nt;        // cache head; first token (of the sequence) and number of tokens
  int n, ctx, len, slot;  // the sequence: drafted tokens, context, tokens in the cache, slot
  int q0;                 // its first row of q
  int j0, j1, kvt;
  int begin, next;        // where the item begins in the list, and the next stretch
  bool two;               // more than one row tile
  bool swapped;           // at most kSwapped rows, all of the sequence's
  // E4M3, at most kDuo rows: two terms of a split operand are rows of one product, hi of row i
  // in lane 32 (i / 16) + i % 16, lo 16 lanes behind; two threads of the warp share the row.  The third
  // term of P~ is a product of its own, with zeros in the lo rows.
  bool duo;
};

// The list of work, decoded alike by every role: items (sequence, cache head, row pair) one
// behind the other: the cost of beginning it, then each key tile as long as its cost (`one` or
// `pair` of row tiles).  A tile belongs to the CTA whose part holds its first unit; parts are no
// shorter than the longest tile, so a part among an item's tiles holds one of them.  Tables in
// shared memory, per sequence: cum (cost before it), its cost per cache head, first row of q, slot,
// tokens in the cache.  The decoding stands before every item's products, so it divides by constants or
// by way of a reciprocal.
template <int one, int pair, int item>
struct List {
  const int *cum, *per, *cu, *slot, *len;
  int B, G, tpt;
  bool masked, split;

  // Key tiles of row pair rt of a sequence: without a mask its last token sees no further
  // than itself.
  __device__ __forceinline__ int tiles(int n, int length, int rt) const {
    const int end = masked ? n : min((rt + 1) * 2 * tpt, n);
    return (length - n + end + kBN - 1) / kBN;
  }
  __device__ __forceinline__ int cost(int n, int rt) const { return n - rt * 2 * tpt > tpt ? pair : one; }
  __device__ __forceinline__ Seg at(int x, int end) const {
    int lo = 0, hi = B - 1;  // the sequence with cum[b] <= x < cum[b + 1]
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (cum[mid + 1] > x) hi = mid; else lo = mid + 1;
    }
    Seg s;
    s.q0 = cu[lo];
    s.n = cu[lo + 1] - s.q0;
    s.slot = slot[lo];
    s.len = len[lo];
    s.ctx = s.len - s.n;
    const int per_head = per[lo];
    int r = x - cum[lo];
    s.h = static_cast<int>(__fdividef(static_cast<float>(r), static_cast<float>(per_head)));  // off by one at most
    if (s.h * per_head > r) --s.h;
    else if ((s.h + 1) * per_head <= r) ++s.h;
    r -= s.h * per_head;
    int rt = 0, kv = tiles(s.n, s.len, 0), w = cost(s.n, 0);
    while (r >= item + kv * w) {
      r -= item + kv * w;
      ++rt;
      kv = tiles(s.n, s.len, rt);
      w = cost(s.n, rt);
    }
    s.tok0 = rt * 2 * tpt;
    s.nt = min(2 * tpt, s.n - s.tok0);
    s.two = s.nt > tpt;
    // Not the last few rows of a long chunk: changing the kind of item between its row pairs costs
    // more than it gains (10 chunks of about 260 tokens: 78 against 70 us).
    s.swapped = s.nt * G <= kSwapped && rt == 0;
    s.duo = split && !s.swapped && s.nt * G <= kDuo;
    s.kvt = kv;
    s.begin = x - r;
    s.next = min(end, s.begin + item + kv * w);
    const int a = max(0, r - item), b = max(0, s.next - s.begin - item);
    s.j0 = s.two ? ceil_div(a, pair) : ceil_div(a, one);
    s.j1 = s.two ? ceil_div(b, pair) : ceil_div(b, one);
    return s;
  }
};

// The products run as units of 64 keys, in rounds of one unit for each stream, S(v) two rounds
// ahead of P~V(v); round v's S (then P~) lie in buffers 2 (v % 2) and the next one, so that a
// stream finds its next S computed while it works on one.  Two row tiles: both streams take the
// same half tile, two rounds a tile; one: stream s takes half s, a round a tile, so that a tile's slot
// is soon free again.  A second half that lies behind the sequence's end is left out.
struct Unit {
  int j, half;  // tile (from j0) and half
  bool live;
};
__device__ __forceinline__ bool full_tile(const Seg& it, int j) { return it.len - (it.j0 + j) * kBN > kBN / 2; }
__device__ __forceinline__ Unit unit_at(const Seg& it, int v, int s) {
  Unit x;
  x.half = it.two ? v & 1 : s;
  x.j = it.two ? v >> 1 : v;
  x.live = x.half == 0 || full_tile(it, x.j);
  return x;
}
__device__ __forceinline__ int rounds_of(const Seg& it) { return (it.two ? 2 : 1) * (it.j1 - it.j0); }

__device__ __forceinline__ bool drain_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > limit_ns) return false;
  }
  return true;
}

constexpr uint32_t kE5m2A = 1u << 7, kE5m2B = 1u << 10;  // instruction descriptor: that operand is E5M2, not E4M3
constexpr uint32_t kLoLanes = 16u << 16;  // from the hi rows of a duo item to its lo rows, as a TMEM address

// Rows of a swapped item's products.
__device__ __forceinline__ int swapped_rows(int rows) { return rows <= 16 ? 16 : 32; }

// Maximum over the warp, by the integer order of floats (negative ones with their bits reversed).
__device__ __forceinline__ float warp_max(float x) {
  int i = __float_as_int(x);
  i ^= (i >> 31) & 0x7fffffff;
  i = __reduce_max_sync(0xffffffffu, i);
  return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
}

// The scores of a swapped item's key: N columns in one load.
template <int N>
__device__ __forceinline__ void load_scores(uint32_t at, float (&x)[N]) {
  uint32_t w[N];
  if constexpr (N == 32) tmem_ld_x32(at, w);
  else tmem_ld_x16(at, w);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = __uint_as_float(w[i]);
}

// Weight of a part with maximum x and sum l beside a joint maximum m.  A part that saw nothing has none;
// one whose sum is not a number (then its maximum may be anything, as maxima pass over NaN) is kept, so
// that the row's sum is none either.
__device__ __forceinline__ float part_weight(float x, float l, float m) {
  return x == -INFINITY && l == 0.f ? 0.f : fast_exp2(x - m);
}
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.f ? 0.f : 1.f / l; }  // 0: a row that sees nothing
__device__ __forceinline__ float natural_lse(float m, float l, float p_shift) {
  return l == 0.f ? -INFINITY : (m + __log2f(l) - p_shift) * kLn2;
}

// Bits [0, k) of word g of a 128-bit set of columns.
__device__ __forceinline__ uint32_t below(int k, int g) {
  k -= 32 * g;
  return k <= 0 ? 0u : k >= 32 ? ~0u : (1u << k) - 1u;
}

template <int D, bool F8>
__global__ void __launch_bounds__(kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_q32,
                const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                const __grid_constant__ TreeParams p) {
  using Lay = Layout<D, F8>;
  constexpr int NS = Lay::NSTAGE, NR = Lay::NRING;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sb + Lay::BAR_OFF + 8 * i; };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + Lay::MISC_OFF);
  // misc[0] TMEM base, misc[1] abort flag, misc[2] items finished, misc[3] items whose K copies have all
  // been issued, misc[4..16) sums of the warps, misc[16..32) page out of range in item i (% 16)
  int* tab = reinterpret_cast<int*>(smem + Lay::TABLE_OFF);
  int *t_cum = tab, *t_cu = t_cum + p.B + 1, *t_slot = t_cu + p.B + 1, *t_len = t_slot + p.B, *t_per = t_len + p.B;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  let_next_launch();
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(Lay::B_QFULL + s), F8 ? 8 : 1);  // E4M3: written by the softmax warps
      mbar_init(bar(Lay::B_QEMPTY + s), 1);
      mbar_init(bar(Lay::B_DRAIN + s), 1);
      mbar_init(bar(Lay::B_WSFULL + s), 1);
      mbar_init(bar(Lay::B_WSFREE + s), 4);
      mbar_init(bar(Lay::B_WPFULL + s), 4);
      mbar_init(bar(Lay::B_WPVDONE + s), 1);
      mbar_init(bar(Lay::B_WG + s), 4);
      int* votes = reinterpret_cast<int*>(smem + Lay::SW_OFF) + s * Lay::SW_STREAM + 7 * 64;
      for (int i = 0; i < 4; ++i) votes[i] = 0;
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(Lay::B_SFULL + i), 1);
      mbar_init(bar(Lay::B_PFULL + i), 4);
      mbar_init(bar(Lay::B_PVDONE + i), 1);
    }
    mbar_init(bar(Lay::B_OFULL), 1);
    mbar_init(bar(Lay::B_ML), 8);
    mbar_init(bar(Lay::B_EPI), 8);
    for (int i = 0; i < NS; ++i) {
      mbar_init(bar(Lay::B_KVFULL + i), 1);
      mbar_init(bar(Lay::B_KVEMPTY + i), 1);
    }
    misc[1] = misc[2] = misc[3] = 0u;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(sb + Lay::MISC_OFF, 512);
    tmem_relinquish();
  }
  wait_for_previous();
  // The page table's lines on their way while the list is built (as many as there are threads).
  {
    const int lines = (p.max_pages + 31) >> 5;
    const int b = static_cast<int>(threadIdx.x) / lines;
    if (b < p.B) {
      const int slot = p.slots ? __ldcg(p.slots + b) : b;
      if (slot >= 0 && slot < p.nslots)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.page_table + static_cast<int64_t>(slot) * p.max_pages +
                                                      32 * (static_cast<int>(threadIdx.x) - b * lines)));
    }
  }
  List<Lay::COST_ONE, Lay::COST_PAIR, Lay::COST_ITEM> list;
  list.cum = t_cum;
  list.per = t_per;
  list.cu = t_cu;
  list.slot = t_slot;
  list.len = t_len;
  list.B = p.B;
  list.G = p.G;
  list.tpt = p.tpt;
  list.masked = p.mask != nullptr;
  list.split = F8;
  {
    // The tiles of each sequence and their prefix sum; a thread takes consecutive sequences.
    const int per = ceil_div(p.B, kThreads);
    const int b0 = min(static_cast<int>(threadIdx.x) * per, p.B), b1 = min(b0 + per, p.B);
    int sum = 0, broken = 0;
    for (int b = b0; b < b1; ++b) {
      const int first = __ldcg(p.cu + b), n = __ldcg(p.cu + b + 1) - first;
      const int slot = p.slots ? __ldcg(p.slots + b) : b;
      int len = 0, work = 0;
      if (n < 0 || first < 0 || n > p.T - first) {
        broken = 1;  // nothing of the batch can be told apart
      } else if (n != 0) {
        int bad = 0;
        if (slot < 0 || slot >= p.nslots) {
          bad = kSiteSlot;
        } else {
          len = __ldcg(p.lens + slot);
          if (len < n || len > (static_cast<int64_t>(p.max_pages) << p.page_shift) || (p.mask && n > p.mask_width))
            bad = kSiteLength;
        }
        if (bad) {
          record_invalid(p.err, bad);
        } else {
          for (int rt = 0; rt * 2 * p.tpt < n; ++rt) work += Lay::COST_ITEM + list.tiles(n, len, rt) * list.cost(n, rt);
          t_per[b] = work;
          work *= p.heads;
        }
      }
      t_cu[b] = first;
      t_slot[b] = slot;
      t_len[b] = len;
      sum += work;
      t_cum[b + 1] = sum;
    }
    if (threadIdx.x == 0) {
      t_cum[0] = 0;
      t_cu[p.B] = __ldcg(p.cu + p.B);
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) misc[4 + warp] = static_cast<uint32_t>(incl);
    if (__syncthreads_or(broken)) {
      if (threadIdx.x == 0) record_invalid(p.err, kSiteLength);
      for (int b = b0; b < b1; ++b) t_cum[b + 1] = 0;
      if (lane == 0) misc[4 + warp] = 0u;
      incl = sum = 0;
      __syncthreads();
    }
    int before = incl - sum;
    for (int w = 0; w < warp; ++w) before += static_cast<int>(misc[4 + w]);
    for (int b = b0; b < b1; ++b) t_cum[b + 1] += before;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const int total = t_cum[p.B];
  // CTAs with work; a part holds at least one tile
  const int ctas = total > 0 ? max(1, min(static_cast<int>(gridDim.x), total / kMinPart)) : 0;
  const int cta = static_cast<int>(blockIdx.x);
  const int x0 = cta < ctas ? static_cast<int>(static_cast<int64_t>(cta) * total / ctas) : 0;
  const int x1 = cta < ctas ? static_cast<int>(static_cast<int64_t>(cta + 1) * total / ctas) : 0;
  WaitCtl wc;
  wc.abort = reinterpret_cast<volatile uint32_t*>(misc + 1);
  wc.err = p.err;
  wc.limit_ns = kTimeoutNs;
  auto wait = [&](int b, uint32_t parity, int site) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(bar(b), parity, wc, timeout_code(site)));
  };

  // Until misc[word] has counted this CTA's first k items.  A count, not a barrier's phase: the waiting
  // role may be several items ahead.
  auto wait_count = [&](int word, int k) -> bool {
    const uint32_t at = sb + Lay::MISC_OFF + 4 * word;
    uint64_t t0 = 0;
    bool good = true;
    while (true) {
      uint32_t done;
      asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(done) : "r"(at) : "memory");
      if (static_cast<int>(done) >= k) break;
      if (t0 == 0) t0 = global_timer_ns();  // not before it is needed: reading the timer is slow
      if (*wc.abort) good = false;
      if (good && global_timer_ns() - t0 > wc.limit_ns) {
        *wc.abort = 1u;
        if (wc.err) atomicCAS(wc.err, 0, timeout_code(kSiteTItems));
        good = false;
      }
      if (!good) break;
    }
    return __all_sync(0xffffffffu, good);
  };
  auto wait_items = [&](int k) -> bool { return wait_count(2, k); };
  auto count_items = [&](int word, int k) {
    asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(sb + Lay::MISC_OFF + 4 * word), "r"(k) : "memory");
  };
  // Pages out of range, found by the producer of K for item i: nothing of such an item is written.  That
  // producer is at most 9 items ahead of the softmax warps' epilogue: the S of two items fit in TMEM beside the
  // one they are at, the K ring holds four tiles more, and one waits for its slot.
  volatile uint32_t* bad_page = misc + 16;
  // E4M3: softmax warp w writes its eighth of an item's queries, from q slot nq on: each row is
  // scaled by the power of two that brings its largest value into [128, 256), hi = E4M3(x), lo =
  // E4M3(x - hi).  A row is held by D / 8 lanes, 8 values each; a warp's rows are 8 kRows apart.
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  auto load_q = [&](const Seg& it, int r) -> uint4 {
    const int t = token_of(r, p);
    const __nv_bfloat16* q = p.q + (static_cast<int64_t>(it.q0 + it.tok0) * p.Hq + it.h * p.G) * D + 8 * (lane % kLanes);
    if (r >= it.nt * p.G) return make_uint4(0, 0, 0, 0);
    return __ldcg(reinterpret_cast<const uint4*>(q + (static_cast<int64_t>(t) * (p.Hq - p.G) + r) * D));
  };
  auto split_row = [&](const Seg& it, int nq, int r, const uint4& x) {
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
    const int c = lane % kLanes, rows = it.nt * p.G, tile_rows = p.tpt * p.G;
    float v[8];
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(u[e] << 16);
      v[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
      top = fmaxf(top, fmaxf(fabsf(v[2 * e]), fabsf(v[2 * e + 1])));
    }
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // 2^(7 - exponent of top): exact, clamped so that both it and its inverse are normal
    int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
    e = max(-100, min(e, 120));
    const float up = __uint_as_float(static_cast<uint32_t>(127 + 7 - e) << 23);
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      hi[y] = lo[y] = 0;
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const float a = v[4 * y + 2 * z] * up, b = v[4 * y + 2 * z + 1] * up;
        float ha, hb;
        upper4_x2(ha, hb, a, b);
        hi[y] |= pack_e4m3x2(ha, hb) << (16 * z);
        lo[y] |= pack_e4m3x2(a - ha, b - hb) << (16 * z);
      }
    }
    if (r < rows) {
      const int tile = r >= tile_rows, rt = r - tile * tile_rows, slot = (nq + tile) & 1;
      uint8_t* base = smem + Lay::Q_OFF + slot * Lay::QTILE;
      if (c == 0)
        reinterpret_cast<float*>(smem + Lay::QS_OFF)[slot * kBM + rt] =
            p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - 7 + e) << 23);
      // 16-byte units of a row are permuted as the copies' swizzle does.  A swapped item's
      // lo rows follow its hi rows: both are columns of one product.
      auto at = [&](int row) {
        return Lay::ROWB == 128 ? row * 128 + (((c >> 1) ^ (row & 7)) << 4) + (c & 1) * 8
                                : row * 64 + (((c >> 1) ^ ((row >> 1) & 3)) << 4) + (c & 1) * 8;
      };
      const int row = it.duo ? 32 * (rt >> 4) + (rt & 15) : rt;
      uint8_t* lo_at = it.swapped ? base + at(rt + swapped_rows(rows)) : it.duo ? base + at(row + 16) : base + Lay::TILE + at(rt);
      *reinterpret_cast<uint2*>(base + at(row)) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(lo_at) = make_uint2(lo[0], lo[1]);
    }
  };
  auto split_done = [&](const Seg& it, int nq) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(bar(Lay::B_QFULL + (nq & 1)));
      if (it.two) mbar_arrive(bar(Lay::B_QFULL + ((nq + 1) & 1)));
    }
  };
  // Eight rows' loads are in flight: they queue behind the copies of K and V, which have begun.  The
  // loop is not unrolled, as its code runs cold at the head of an item, where fetching it is what counts.
  auto split_q = [&](const Seg& it, int nq, int w8) -> bool {
    constexpr int U = 8;
    int r = w8 * kRows + lane / kLanes;
    uint4 w[U];
#pragma unroll
    for (int i = 0; i < U; ++i) w[i] = load_q(it, r + 8 * kRows * i);
    for (int k = 0; k < (it.two ? 2 : 1); ++k)
      if (nq + k >= 2 && !wait(Lay::B_QEMPTY + ((nq + k) & 1), (((nq + k) >> 1) - 1) & 1, kSiteTQEmpty)) return false;
#pragma unroll 1
    for (; __any_sync(0xffffffffu, r < it.nt * p.G); r += 8 * kRows) {
      const uint4 x = w[0];
#pragma unroll
      for (int i = 0; i + 1 < U; ++i) w[i] = w[i + 1];
      w[U - 1] = load_q(it, r + 8 * kRows * U);
      split_row(it, nq, r, x);
    }
    split_done(it, nq);
    return true;
  };

  // Producers: K (and q) by one warp, V by another.
  auto produce = [&](auto keys) {
    constexpr bool is_k = decltype(keys)::value;
    if (elect_one()) {
      if (is_k && !F8) tma_prefetch_map(&tm_q);
      tma_prefetch_map(is_k ? &tm_k : &tm_v);
    }
    __syncwarp();
    const uint64_t pol = l2_policy_evict_normal();
    uint32_t n = 0;  // tiles copied
    int nq = 0, items = 0;
    bool ok = true, was_swapped = false;
    // A tile is copied in boxes of box_rows keys, box i by lane i; per_tile is a power of two.
    const int per_tile = kBN / p.box_rows;
    const int box_bytes = p.box_rows * Lay::ROWB * Lay::NCHUNK;
    const uint32_t lane_dst = sb + Lay::KV_OFF + (is_k ? 0 : NR * Lay::TILE) + lane * p.box_rows * Lay::ROWB;
    const int in_page = (1 << p.page_shift) - 1;
    for (int x = x0; x < x1 && ok;) {
      const Seg it = list.at(x, x1);
      x = it.next;
      if (it.j0 >= it.j1) continue;
      // The pages of 32 boxes, one per lane, and of the next 32.
      const int32_t* row = p.page_table + static_cast<int64_t>(it.slot) * p.max_pages;
      const int first = it.j0 * kBN, end = min(it.len, it.j1 * kBN);
      auto pages_from = [&](int pos) -> int {
        pos += lane * p.box_rows;
        return pos < end ? __ldcg(row + (pos >> p.page_shift)) : 0;
      };
      int win = 0, win_next = pages_from(first), from = 32;  // from: the next box's lane in win
      int pos = first, next_win = first;
      if (!F8 && is_k) {
        // A swapped item's P~ lies in the tiles of q: they are whole again when its products are done.
        if (was_swapped && !it.swapped) ok = wait_items(items);
        for (int k = 0; k < (it.two ? 2 : 1) && ok; ++k, ++nq) {
          const int slot = nq & 1;
          if (nq >= 2) ok = wait(Lay::B_QEMPTY + slot, ((nq >> 1) - 1) & 1, kSiteTQEmpty);
          if (!ok) break;
          if (elect_one()) {
            const int tokens = it.swapped ? p.tpt32 : p.tpt;
            mbar_arrive_expect_tx(bar(Lay::B_QFULL + slot), Lay::NCHUNK * tokens * p.G * Lay::ROWB);
#pragma unroll
            for (int c = 0; c < Lay::NCHUNK; ++c)
              tma_load_4d(sb + Lay::Q_OFF + slot * Lay::QTILE + c * Lay::CHUNK, it.swapped ? &tm_q32 : &tm_q,
                          bar(Lay::B_QFULL + slot), c * Lay::CELEMS, 0, it.h, it.q0 + it.tok0 + k * p.tpt, pol);
          }
          __syncwarp();
        }
        if (!ok) break;
      }
      was_swapped = it.swapped;
      bool out_of_range = false;
      for (int j = it.j0; j < it.j1; ++j, ++n, pos += kBN, from += per_tile) {
        if (from == 32) {
          from = 0;
          win = win_next;
          next_win += 32 * p.box_rows;
          win_next = pages_from(next_win);
        }
        const uint32_t slot = n % NR, full = bar(Lay::B_KVFULL + (is_k ? 0 : NR)) + 8 * slot;
        const int page = __shfl_sync(0xffffffffu, win, from + (lane & (per_tile - 1)));
        const int mine = pos + lane * p.box_rows;
        const bool copies = lane < per_tile && mine < it.len;
        int at = p.rows;
        if (static_cast<unsigned>(page) < static_cast<unsigned>(p.pages)) at = p.layer_row + (page << p.page_shift) + (mine & in_page);
        else if (copies) out_of_range = true;
        const int boxes = min(per_tile, (it.len - pos + p.box_rows - 1) / p.box_rows);
        if (n >= static_cast<uint32_t>(NR)) {
          ok = wait(Lay::B_KVEMPTY + (is_k ? 0 : NR) + slot, ((n / NR) - 1) & 1u, kSiteTKvEmpty);
          if (!ok) break;
        }
        if (lane == 0) mbar_arrive_expect_tx(full, boxes * box_bytes);
        __syncwarp();
        if (copies) {
#pragma unroll
          for (int c = 0; c < Lay::NCHUNK; ++c)
            tma_load_3d(lane_dst + slot * Lay::TILE + c * Lay::CHUNK, is_k ? &tm_k : &tm_v, full, c * Lay::CELEMS, it.h, at, pol);
        }
        __syncwarp();
      }
      if (is_k) {
        out_of_range = __any_sync(0xffffffffu, out_of_range);
        if (lane == 0) {
          if (out_of_range) record_invalid(p.err, kSitePage);
          bad_page[items & 15] = out_of_range;
          count_items(3, items + 1);
        }
      }
      ++items;
    }
    // This warp's copies have landed before the CTA may exit.
    for (uint32_t i = n > static_cast<uint32_t>(NR) ? n - NR : 0u; i < n; ++i)
      drain_wait(bar(Lay::B_KVFULL + i % NR + (is_k ? 0 : NR)), (i / NR) & 1u, kDrainLimitNs);
    if (!F8 && is_k) {
      for (int i = nq > 2 ? nq - 2 : 0; i < nq; ++i) drain_wait(bar(Lay::B_QFULL + (i & 1)), (i >> 1) & 1, kDrainLimitNs);
    }
  };

  // 4 x 32 x (168 - 120) registers released by warpgroup 2, 8 x 32 x (192 - 168) taken.
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;\n" ::: "memory");
    // ------------------------------------------------------------ softmax
    // Stream s = warp / 4; warp w owns TMEM lanes 32(w%4)..+31, one row per thread.
    const int s = warp >> 2, wq = warp & 3;
    const int r = wq * 32 + lane;
    const uint32_t lane_bits = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t t_o = tmem + lane_bits + (s ? Lay::TM_O1 : Lay::TM_O0);
    float2* ml = reinterpret_cast<float2*>(smem + Lay::ML_OFF);
    uint32_t phases = 0;  // bit u & 3: phase of that buffer's next use
    uint32_t o_phase = 0, m_phase = 0, e_phase = 0;
    int nq = 0;  // row tiles of q taken so far
    int items = 0;
    auto finished = [&]() {
      ++items;
      if (threadIdx.x == 0) count_items(2, items);
    };
    uint32_t w_s_phase = 0, w_pv = 0, w_wg = 0, votes = 0;  // swapped items; w_pv: P~ handed over
    // An item of few rows, scores transposed: a thread holds one key of the tile and all
    // rows, so all four warps of the stream share the exponentials, however few rows there are.
    // P~ (rows side by side) goes to shared memory as the second operand of O^T += V^T P~^T.  The
    // maximum of a row is over lanes and warps: it is taken for the stream's first tile, and again
    // only when some score exceeds its row's reference by more than tau (a vote of the four warps).
    // Unrolled for 16 or 32 rows: the code of a tile is run straight through, and fetching it
    // costs more than computing it when rows that do not exist are jumped over.
    // `behind` runs when the stream's last P~ has been handed over.
    auto swapped_item = [&](const Seg& it, int nq_item, auto blocks, auto behind) -> bool {
      constexpr int NCH = decltype(blocks)::value, N = 16 * NCH;
      const int nj = it.j1 - it.j0, rows = it.nt * p.G;
      const int key = r;
      float* st = reinterpret_cast<float*>(smem + Lay::SW_OFF) + s * Lay::SW_STREAM;
      float *nm = st, *al = st + 64, *mr = st + 128, *wm = st + 192;
      volatile int* vote = reinterpret_cast<volatile int*>(st + 448);
      [[maybe_unused]] const float* qs = reinterpret_cast<const float*>(smem + Lay::QS_OFF) + (nq_item & 1) * kBM;
      const uint32_t t_s = tmem + lane_bits + Lay::TM_S + 128 * s;
      auto meet = [&]() -> bool {  // the stream's four warps
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Lay::B_WG + s));
        const bool good = wait(Lay::B_WG + s, w_wg & 1u, kSiteTMerge);
        w_wg ^= 1u;
        return good;
      };
      float l[N];
#pragma unroll
      for (int i = 0; i < N; ++i) l[i] = 0.f;
      bool first = true;
      for (int j = s; j < nj; j += 2) {
        if (!wait(Lay::B_WSFULL + s, w_s_phase, kSiteTSFull)) return false;
        w_s_phase ^= 1u;
        tc_fence_after();
        float x[N];
        load_scores(t_s, x);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Lay::B_WSFREE + s));
        // Rows that see this key.
        const int pos = (it.j0 + j) * kBN + key, jl = pos - it.ctx;
        uint32_t vis[2] = {below(rows, 0), below(rows, 1)};
        const bool part = (it.j0 + j + 1) * kBN > it.ctx;
        if (part && jl >= 0) {
          uint32_t see[2] = {0u, 0u};
          if (pos < it.len) {
            if (p.mask == nullptr) {
              const int from = max(0, jl - it.tok0) * p.G;  // tokens from jl on
              see[0] = ~below(from, 0);
              see[1] = ~below(from, 1);
            } else {
              const uint8_t* m = p.mask + static_cast<int64_t>(it.q0 + it.tok0) * p.mask_width + jl;
#pragma unroll 4
              for (int t2 = 0; t2 < it.nt; ++t2)
                if (m[static_cast<int64_t>(t2) * p.mask_width] != 0) {
                  see[0] |= below((t2 + 1) * p.G, 0) & ~below(t2 * p.G, 0);
                  see[1] |= below((t2 + 1) * p.G, 1) & ~below(t2 * p.G, 1);
                }
            }
          }
          vis[0] &= see[0];
          vis[1] &= see[1];
        }
        // x = scale s - reference (log2 units, times 2^p_shift); the first tile has no reference yet
#pragma unroll
        for (int c = 0; c < 4 * NCH; ++c) {
          const float4 n4 = first ? make_float4(0.f, 0.f, 0.f, 0.f) : reinterpret_cast<const float4*>(nm)[c];
          if constexpr (F8) {
            const float4 s4 = reinterpret_cast<const float4*>(qs)[c];
            ffma2_vv(x[4 * c], x[4 * c + 1], x[4 * c], x[4 * c + 1], s4.x, s4.y, n4.x, n4.y);
            ffma2_vv(x[4 * c + 2], x[4 * c + 3], x[4 * c + 2], x[4 * c + 3], s4.z, s4.w, n4.z, n4.w);
          } else {
            ffma2_bv(x[4 * c], x[4 * c + 1], x[4 * c], x[4 * c + 1], p.scale_log2, n4.x, n4.y);
            ffma2_bv(x[4 * c + 2], x[4 * c + 3], x[4 * c + 2], x[4 * c + 3], p.scale_log2, n4.z, n4.w);
          }
        }
        if (part || rows != N) {
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (!((vis[i >> 5] >> (i & 31)) & 1u)) x[i] = -INFINITY;
        }
        bool renew = first;
        if (!first) {
          float top = x[0];
#pragma unroll
          for (int i = 1; i + 1 < N; i += 2) top = fmax3(top, x[i], x[i + 1]);
          top = fmaxf(top, x[N - 1]);
          const bool over = __any_sync(0xffffffffu, top > p.tau + p.p_shift);
          if (over && lane == 0) vote[votes & 3] = 1;
          if (!meet()) return false;
          renew = vote[votes & 3] != 0;
          if (wq == 0 && lane == 0) vote[(votes + 2) & 3] = 0;  // read by all before the last meeting
          ++votes;
        }
        // P~ of the stream's last tile has been multiplied: O is whole, its place is free
        if (w_pv > 0 && !wait(Lay::B_WPVDONE + s, (w_pv - 1) & 1u, kSiteTPvDone)) return false;
        tc_fence_after();
        if (renew) {
          float keep[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float y = warp_max(x[i]);  // relative to the reference so far
            if (lane == (i & 31)) keep[i >> 5] = y;
          }
          wm[wq * 64 + lane] = keep[0];
          wm[wq * 64 + 32 + lane] = keep[1];
          if (!meet()) return false;
          if (key < 64) {
            // the tile's maximum relative to nm, the row's reference and its new one
            const float rel = fmaxf(fmaxf(wm[key], wm[64 + key]), fmaxf(wm[128 + key], wm[192 + key]));
            const float was = first ? 0.f : nm[key], old = first ? -INFINITY : mr[key];
            const float m = rel - was;
            const float now = (old == -INFINITY || m - old > p.tau) ? m : old;
            const float next = (now == -INFINITY ? 0.f : -now) + p.p_shift;
            al[key] = old == -INFINITY ? 1.f : fast_exp2(old - now);  // a row without keys so far has O = 0
            mr[key] = now;
            nm[key] = next;
            wm[key] = next - was;  // what the scores move by (the other warps' maxima have been read)
          }
          if (!meet()) return false;
#pragma unroll
          for (int i = 0; i < N; ++i) x[i] += wm[i];
          if (!first) {
#pragma unroll
            for (int i = 0; i < N; ++i) l[i] *= al[i];
#pragma unroll 1
            for (int c = 0; c < NCH; ++c) {
#pragma unroll
              for (int term = 0; term < Lay::P_TERMS; ++term) {
                uint32_t w[16];
                const uint32_t at = t_o + N * term + 16 * c;
                tmem_ld_x16(at, w);
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * al[16 * c + i]);
                tmem_st_x16(at, w);
              }
            }
            tmem_st_wait();
          }
        }
        first = false;
        uint8_t* prow = smem + Lay::p_row(s, key);
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          {
            float e[16];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              e[i] = fast_exp2(x[16 * c + i]);
              e[i + 1] = fast_exp2(x[16 * c + i + 1]);
              fadd2_acc(l[16 * c + i], l[16 * c + i + 1], e[i], e[i + 1]);
            }
            // 16-byte units of a key's row, permuted as the descriptors' 128-byte swizzle
            if constexpr (F8) {
              uint32_t t[3][4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                split_e5m2x4(e[4 * i], e[4 * i + 1], e[4 * i + 2], e[4 * i + 3], t[0][i], t[1][i], t[2][i]);
#pragma unroll
              for (int k = 0; k < 3; ++k)
                *reinterpret_cast<uint4*>(prow + (((NCH * k + c) ^ (key & 7)) << 4)) = make_uint4(t[k][0], t[k][1], t[k][2], t[k][3]);
            } else {
#pragma unroll
              for (int k = 0; k < 2; ++k)
                *reinterpret_cast<uint4*>(prow + (((2 * c + k) ^ (key & 7)) << 4)) =
                    make_uint4(pack_bf16x2(e[8 * k], e[8 * k + 1]), pack_bf16x2(e[8 * k + 2], e[8 * k + 3]),
                               pack_bf16x2(e[8 * k + 4], e[8 * k + 5]), pack_bf16x2(e[8 * k + 6], e[8 * k + 7]));
            }
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Lay::B_WPFULL + s));
        ++w_pv;
      }
      if (!behind()) return false;
      // Row sums over the keys (lanes, then warps): each step adds a lane's other half of the rows, so
      // that a lane ends with row lane % N.
      {
        float v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = l[i];
#pragma unroll
        for (int o = N / 2; o; o >>= 1) {
#pragma unroll
          for (int i = 0; i < o; ++i) {
            const bool up = (lane & o) != 0;
            const float give = up ? v[i] : v[i + o], have = up ? v[i + o] : v[i];
            v[i] = have + __shfl_xor_sync(0xffffffffu, give, o);
          }
        }
        if constexpr (N == 16) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 16);
        wm[wq * 64 + lane] = v[0];
      }
      if (first && key < 64) mr[key] = -INFINITY;  // no tile for this stream
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(Lay::B_ML));
      if (!wait(Lay::B_ML, m_phase, kSiteTMerge)) return false;
      m_phase ^= 1u;
      if (!wait_count(3, items + 1)) return false;
      const bool bad = bad_page[items & 15] != 0;
      const bool whole = it.j0 == 0 && it.j1 == it.kvt;
      const int64_t slot = static_cast<int64_t>(cta) * 2 + (it.j0 == 0 ? 1 : 0);
      if (key < rows) {
        // Both streams' state of row `key`; weights of their O, into nm and al of this stream.
        const float* f = reinterpret_cast<const float*>(smem + Lay::SW_OFF);
        float m2[2], l2[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float* g2 = f + i * Lay::SW_STREAM;
          m2[i] = g2[128 + key];
          l2[i] = (g2[192 + key] + g2[256 + key]) + (g2[320 + key] + g2[384 + key]);
        }
        const float m = fmaxf(m2[0], m2[1]);
        const float w0 = part_weight(m2[0], l2[0], m), w1 = part_weight(m2[1], l2[1], m);
        const float sum = l2[0] * w0 + l2[1] * w1;
        const float f0 = whole ? inverse_sum(sum) * p.o_scale : 1.f;
        nm[key] = w0 * f0;
        al[key] = w1 * f0;
        if (s == 0) {
          const int t2 = token_of(key, p), g2 = key - t2 * p.G;
          if (!whole)
            p.stat[slot * (2 * kBM) + key] = make_float2(m, bad ? -1.f : sum);
          else if (!bad)
            p.lse[static_cast<int64_t>(it.h * p.G + g2) * p.T + it.q0 + it.tok0 + t2] = natural_lse(m, sum, p.p_shift);
        }
      }
      if (!meet()) return false;
      if (!wait(Lay::B_OFULL, o_phase, kSiteTOFull)) return false;
      o_phase ^= 1u;
      tc_fence_after();
      // O^T: lane = dimension; this warpgroup takes every other group of 4 rows.
      if (wq * 32 < D) {
        const uint32_t t0 = tmem + lane_bits + Lay::TM_O0, t1 = tmem + lane_bits + Lay::TM_O1;
        for (int c = 4 * s; c < rows; c += 8) {
          float v[4] = {0.f, 0.f, 0.f, 0.f};
          auto add = [&](uint32_t at, const float* weight) {
            uint32_t w[8];
            tmem_ld_x8(at + c, w);  // of the 8 columns from there (there are that many) the first 4
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = fmaf(__uint_as_float(w[i]), weight[c + i], v[i]);
          };
#pragma unroll
          for (int term = 0; term < Lay::P_TERMS; ++term) {
            add(t0 + N * term, nm);
            if (nj > 1) add(t1 + N * term, al);
          }
          int t2 = token_of(c, p), g2 = c - t2 * p.G;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = c + i;
            if (row < rows && !bad) {
              if (whole)
                p.o[(static_cast<int64_t>(it.q0 + it.tok0 + t2) * p.Hq + it.h * p.G + g2) * D + key] = __float2bfloat16(v[i]);
              else
                p.part[((slot * (D / 4) + (key >> 2)) * (2 * kBM) + row) * 4 + (key & 3)] = v[i];
            }
            if (++g2 == p.G) ++t2, g2 = 0;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(Lay::B_EPI));
      if (!wait(Lay::B_EPI, e_phase, kSiteTMerge)) return false;
      e_phase ^= 1u;
      return true;
    };
    bool ok = true;
    [[maybe_unused]] bool split = false;  // the item's queries have been written already
    if (threadIdx.x == 0) p.head[cta] = make_int4(-1, 0, 0, 0);
    for (int x = x0; x < x1 && ok;) {
      const Seg it = list.at(x, x1);
      x = it.next;
      if (it.j0 >= it.j1) continue;
      if (threadIdx.x == 0 && it.j0 == 0 && it.j1 < it.kvt) {
        // The item's first tiles without its last: the CTA whose part holds the first unit of the item's last tile
        const int64_t end = it.begin + Lay::COST_ITEM + (it.kvt - 1) * (it.two ? Lay::COST_PAIR : Lay::COST_ONE);
        int last = static_cast<int>(end * ctas / total);
        while (static_cast<int64_t>(last + 1) * total / ctas <= end) ++last;
        while (static_cast<int64_t>(last) * total / ctas > end) --last;
        p.head[cta] = make_int4(it.q0 + it.tok0, it.h, it.nt, last);
      }
      const int first = it.two ? s * p.tpt : 0;  // this stream's first token of the item
      const int mine = it.two ? (s ? it.nt - p.tpt : p.tpt) : it.nt;
      // The warp's rows of the tile, this thread's row of it, and that row's token.
      const int row_n = it.duo ? 16 : 32, row0 = wq * row_n, rr = row0 + (lane & (row_n - 1));
      const int tl = token_of(rr, p);
      const int tok = it.tok0 + first + tl;  // of the sequence
      const bool valid = tl < mine;
      const bool busy = row0 < mine * p.G;   // the warp has a valid row
      float sl = p.scale_log2;
      if constexpr (F8) {
        if (!split) ok = split_q(it, nq, warp);
        split = false;
        if (!ok) break;
        // every warp has written its rows' scales
        const int mine_q = nq + (it.two ? s : 0);
        ok = wait(Lay::B_QFULL + (mine_q & 1), (mine_q >> 1) & 1, kSiteTQFull);
        if (!ok) break;
        sl = reinterpret_cast<const float*>(smem + Lay::QS_OFF)[(mine_q & 1) * kBM + rr];
      }
      if (p.mask != nullptr && it.j1 * kBN > it.ctx) {
        // The mask rows of this warp's tokens will be needed for the last tiles.
        const int t0 = it.swapped ? 0 : token_of(row0, p), t1 = it.swapped ? it.nt - 1 : min(token_of(row0 + row_n - 1, p), mine - 1);
        const uint8_t* rows = p.mask + static_cast<int64_t>(it.q0 + it.tok0 + first + t0) * p.mask_width;
        for (int i = lane * 128; i < (t1 - t0 + 1) * p.mask_width; i += 32 * 128)
          asm volatile("prefetch.global.L1 [%0];" ::"l"(rows + i));
      }
      if (it.swapped) {
        const int width = swapped_rows(it.nt * p.G);
        // E4M3, d 128: the next item's queries load beside this one's tiles, and are written before its
        // epilogue (the other q slot, whose rows a swapped item's P~ leaves alone).  64 single tokens
        // over 512 to 8192: 109 -> 105 us; with d 64, whose tiles are half as long, 85 -> 94.
        Seg nx = it;
        uint4 w[2];
        const int qr = warp * kRows + lane / kLanes;
        if constexpr (F8 && D == 128) {
          if (x < x1) nx = list.at(x, x1);
          split = x < x1 && nx.swapped && nx.j0 < nx.j1;
          if (split) {
            w[0] = load_q(nx, qr);
            w[1] = load_q(nx, qr + 8 * kRows);
          }
        }
        auto behind = [&]() -> bool {
          if constexpr (F8 && D == 128) {
            if (split) {
              const int n = nq + 1;
              if (n >= 2 && !wait(Lay::B_QEMPTY + (n & 1), ((n >> 1) - 1) & 1, kSiteTQEmpty)) return false;
#pragma unroll 1
              for (int i = 0; i < 2; ++i) {
                split_row(nx, n, qr + 8 * kRows * i, i ? w[1] : w[0]);
              }
              split_done(nx, n);
            }
          }
          return true;
        };
        ok = width == 16 ? swapped_item(it, nq, std::integral_constant<int, 1>{}, behind)
                         : swapped_item(it, nq, std::integral_constant<int, 2>{}, behind);
        if (!ok) break;
        ++nq;
        finished();
        continue;
      }
      nq += it.two ? 2 : 1;
      float m_ref = -INFINITY, l = 0.f;
      bool any = false;
      int last_buf = 0;  // buffer of the stream's last unit
      const int rounds = rounds_of(it);
      // W threads share a row, 64 / W keys of a unit each.
      auto attend = [&](auto threads) -> bool {
        constexpr int W = decltype(threads)::value, NC = 64 / W;
        for (int v = 0; v < rounds; ++v) {
          const Unit un = unit_at(it, v, s);
          if (!un.live) continue;
          const int buf = 2 * (v & 1) + s;
          const uint32_t t_s = tmem + lane_bits + Lay::TM_S + 64 * buf;
          if (!wait(Lay::B_SFULL + buf, (phases >> buf) & 1u, kSiteTSFull)) return false;
          phases ^= 1u << buf;
          tc_fence_after();
          auto release = [&]() {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(Lay::B_PFULL + buf));
          };
          const bool again = any;  // O holds something
          any = true;
          if (!busy) {  // nothing to compute: the rows of P~ that stay behind are never read
            release();
            last_buf = buf;
            continue;
          }
          uint32_t sa[NC];
          if constexpr (W == 1) {
            tmem_ld_x64(t_s, sa);
          } else {
            uint32_t lo[NC];
            tmem_ld_duo_both(t_s, sa, lo);
#pragma unroll
            for (int c = 0; c < NC; ++c) sa[c] = __float_as_uint(__uint_as_float(sa[c]) + __uint_as_float(lo[c]));
          }
          const int kb = (it.j0 + un.j) * kBN + 64 * un.half;
          if (kb + 64 > it.ctx) {  // the half tile holds drafted tokens, or ends behind them
            uint32_t vis[2];
            if (p.mask == nullptr) {
#pragma unroll
              for (int c = 0; c < 2; ++c) vis[c] = below(it.ctx + tok + 1 - kb, c);
            } else {
#pragma unroll
              for (int c = 0; c < 2; ++c) vis[c] = below(it.ctx - kb, c);
              // The mask rows of the warp's tokens, 32 columns per load, 8 tokens at a time.
              const int t_lo = token_of(row0, p), t_hi = min(token_of(row0 + row_n - 1, p), mine - 1);
              const uint8_t* rows = p.mask + static_cast<int64_t>(it.q0 + it.tok0 + first) * p.mask_width;
              const int col = kb + lane - it.ctx;
              for (int t0 = t_lo; t0 <= t_hi; t0 += 8) {
                uint8_t w[8][2];
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                  for (int c = 0; c < 2; ++c) {
                    const int jl = col + 32 * c;
                    w[i][c] = (t0 + i <= t_hi && jl >= 0 && jl < it.n)
                                  ? rows[static_cast<int64_t>(t0 + i) * p.mask_width + jl]
                                  : 0;
                  }
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                  for (int c = 0; c < 2; ++c) {
                    const uint32_t bits = __ballot_sync(0xffffffffu, w[i][c] != 0);
                    if (t0 + i == tl) vis[c] |= bits;
                  }
              }
            }
            if (W == 2 && lane >= 16) vis[0] = vis[1];
#pragma unroll
            for (int c = 0; c < NC; ++c)
              if (!((vis[c >> 5] >> (c & 31)) & 1u)) sa[c] = __float_as_uint(-INFINITY);
          }
          float m4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            m4[i] = fmax3(__uint_as_float(sa[i]), __uint_as_float(sa[i + 4]), __uint_as_float(sa[i + 8]));
#pragma unroll
          for (int c = 12; c < NC - 4; c += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              m4[i] = fmax3(m4[i], __uint_as_float(sa[c + i]), __uint_as_float(sa[c + 4 + i]));
#pragma unroll
          for (int i = 0; i < 4; ++i) m4[i] = fmaxf(m4[i], __uint_as_float(sa[NC - 4 + i]));
          float m_tile = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
          if constexpr (W == 2) m_tile = fmaxf(m_tile, __shfl_xor_sync(0xffffffffu, m_tile, 16));
          m_tile *= sl;
          bool need = false;
          float alpha = 1.f;
          if (m_ref == -INFINITY) {  // the first keys that this row sees
            m_ref = m_tile;
          } else if (m_tile - m_ref > p.tau) {
            need = valid;
            alpha = fast_exp2(m_ref - m_tile);
            m_ref = m_tile;
            l *= alpha;
          }
          float nm = m_ref == -INFINITY ? 0.f : -m_ref;
          if constexpr (F8) nm += p.p_shift;
          float ls[4] = {0.f, 0.f, 0.f, 0.f};
          auto exps = [&](int c, float& a, float& e) {  // column pair c (keys 2c, 2c + 1)
            ffma2_bc(a, e, __uint_as_float(sa[2 * c]), __uint_as_float(sa[2 * c + 1]), sl, nm);
            a = fast_exp2(a);
            e = fast_exp2(e);
            if (c & 1) fadd2_acc(ls[2], ls[3], a, e);
            else fadd2_acc(ls[0], ls[1], a, e);
          };
          if constexpr (!F8) {
            uint32_t pk[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              float a, e;
              exps(c, a, e);
              pk[c] = pack_bf16x2(a, e);
            }
            tmem_st_x32(t_s, pk);
          } else {
            uint32_t t1[NC / 4], t2[NC / 4], t3[NC / 4];
#pragma unroll
            for (int c = 0; c < NC / 4; ++c) {
              float e[4];
              exps(2 * c, e[0], e[1]);
              exps(2 * c + 1, e[2], e[3]);
              split_e5m2x4(e[0], e[1], e[2], e[3], t1[c], t2[c], t3[c]);
            }
            if constexpr (W == 1) {
              tmem_st_x16(t_s, t1);
              tmem_st_x16(t_s + 16, t2);
              tmem_st_x16(t_s + 32, t3);
            } else {
              const uint32_t none[NC / 4] = {};
              tmem_st_duo(t_s, t1);
              tmem_st_duo(t_s + kLoLanes, t2);
              tmem_st_duo(t_s + 16, t3);
              tmem_st_duo(t_s + 16 + kLoLanes, none);
            }
          }
          if (again && __any_sync(0xffffffffu, need)) {
            // the stream's last P~V has to be in O before O is rescaled
            if (!wait(Lay::B_PVDONE + last_buf, ((phases >> last_buf) & 1u) ^ 1u, kSiteTPvDone)) return false;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t ov[32];
              tmem_ld_x32(t_o + 32 * c, ov);
#pragma unroll
              for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
              tmem_st_x32(t_o + 32 * c, ov);
            }
          }
          last_buf = buf;
          release();
          l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
        }
        if constexpr (W == 2) l += __shfl_xor_sync(0xffffffffu, l, 16);
        return true;
      };
      if constexpr (F8) {
        ok = it.duo ? attend(std::integral_constant<int, 2>{}) : attend(std::integral_constant<int, 1>{});
      } else {
        ok = attend(std::integral_constant<int, 1>{});
      }
      if (!ok) break;
      // ---------------------------------------------------------- epilogue
      // Two row tiles: each warpgroup writes its own rows.  One: the streams' O are joined, and
      // each warpgroup writes half the columns.
      float a0 = 1.f, a1 = 0.f;  // weights of this stream's O and the other's
      if (!it.two) {
        ml[s * kBM + r] = make_float2(m_ref, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Lay::B_ML));
        ok = wait(Lay::B_ML, m_phase, kSiteTMerge);
        if (!ok) break;
        m_phase ^= 1u;
        const float2 other = ml[(s ^ 1) * kBM + r];
        const float m = fmaxf(m_ref, other.x);
        a0 = part_weight(m_ref, l, m);
        a1 = part_weight(other.x, other.y, m);
        l = l * a0 + other.y * a1;
        m_ref = m;
      }
      ok = wait(Lay::B_OFULL, o_phase, kSiteTOFull);
      if (!ok) break;
      o_phase ^= 1u;
      tc_fence_after();
      ok = wait_count(3, items + 1);
      if (!ok) break;
      const bool bad = bad_page[items & 15] != 0;
      const bool whole = it.j0 == 0 && it.j1 == it.kvt;
      if (busy) {
        const int g = rr - tl * p.G;
        const int64_t row = static_cast<int64_t>(it.q0 + tok) * p.Hq + it.h * p.G + g;
        const int64_t slot = static_cast<int64_t>(cta) * 2 + (it.j0 == 0 ? 1 : 0);
        const int slot_row = (it.two ? s * kBM : 0) + rr;
        float4* part = reinterpret_cast<float4*>(p.part) + slot * (2 * kBM) * (D / 4) + slot_row;
        const float inv = inverse_sum(l) * p.o_scale;
        // Columns of this warpgroup; a stream that took no tile has nothing in its O.
        const int c_lo = it.two ? 0 : s * (D / 64), c_hi = it.two ? D / 32 : (s + 1) * (D / 64);
        const bool use_own = any, use_other = !it.two && (s != 0 || it.j1 - it.j0 > 1 || full_tile(it, 0));
        const uint32_t t_x = tmem + lane_bits + (s ? Lay::TM_O0 : Lay::TM_O1);
        auto write = [&](auto threads) {
          constexpr int W = decltype(threads)::value, NV = 32 / W;  // columns of a thread, of 32
          const int mine_at = W == 2 ? lane & 16 : 0;
          for (int c = c_lo; c < c_hi; ++c) {
            uint32_t ov[NV];
            float v[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] = 0.f;
            auto add = [&](uint32_t at, float weight) {
              if constexpr (W == 1) tmem_ld_x32(at + 32 * c, ov);
              else tmem_ld_duo(at + 32 * c, ov);
              // weight 0 also where the stream's O was never a number
              if (weight != 0.f) {
#pragma unroll
                for (int i = 0; i < NV; ++i) v[i] = fmaf(__uint_as_float(ov[i]), weight, v[i]);
              }
            };
#pragma unroll
            for (int term = 0; term < W; ++term) {
              if (use_own) add(t_o + term * kLoLanes, a0);
              if (use_other) add(t_x + term * kLoLanes, a1);
            }
            if (valid && whole && !bad) {
              uint4* dst = reinterpret_cast<uint4*>(p.o + row * D + 32 * c + mine_at);
#pragma unroll
              for (int i = 0; i < NV / 8; ++i)
                dst[i] = make_uint4(pack_bf16x2(v[8 * i] * inv, v[8 * i + 1] * inv),
                                    pack_bf16x2(v[8 * i + 2] * inv, v[8 * i + 3] * inv),
                                    pack_bf16x2(v[8 * i + 4] * inv, v[8 * i + 5] * inv),
                                    pack_bf16x2(v[8 * i + 6] * inv, v[8 * i + 7] * inv));
            } else if (valid && !bad) {
              float4* dst = part + (c * 8 + mine_at / 4) * (2 * kBM);
#pragma unroll
              for (int i = 0; i < NV / 4; ++i)
                dst[i * (2 * kBM)] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            }
            __syncwarp();
          }
        };
        if constexpr (F8) {
          if (it.duo) write(std::integral_constant<int, 2>{});
          else write(std::integral_constant<int, 1>{});
        } else {
          write(std::integral_constant<int, 1>{});
        }
        if (valid && (it.two || s == 0) && !(it.duo && lane >= 16)) {
          if (!whole)
            p.stat[slot * (2 * kBM) + slot_row] = make_float2(m_ref, bad ? -1.f : l);
          else if (!bad)
            p.lse[static_cast<int64_t>(it.h * p.G + g) * p.T + it.q0 + tok] = natural_lse(m_ref, l, p.p_shift);
        }
      }
      // The next item's P~V may write either O only when both warpgroups have read them, and
      // neither warpgroup runs an item ahead of the other.
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(Lay::B_EPI));
      ok = wait(Lay::B_EPI, e_phase, kSiteTMerge);
      e_phase ^= 1u;
      finished();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;\n" ::: "memory");
    if (warp == 8) {
      produce(std::true_type{});
    } else if (warp == 10) {
      produce(std::false_type{});
    } else {
      // ------------------------------------------------- products: S (9), P~V (11)
      // Two warps issue them, so that one's waits run beside the other's products: a lone
      // issuer spent as long waiting as the products took.
      constexpr int kHalf = kBN / 2;
      constexpr bool SW64 = Lay::ROWB == 64;
      uint32_t n_ld = 0, phases = 0, used = 0;  // bit b: phase of S buffer b, and whether it was used
      uint32_t w_phase = 0, w_used = 0;         // the same for the streams of swapped items
      int nq = 0, items = 0;
      bool ok = true, was_swapped = false;
      // Rows of a V tile from the sequence's end to the end of the last K step: whatever the
      // page holds there must not meet the zero weights.
      auto clear_rows = [&](uint32_t slot, int from, int to) {
        if (from >= to) return;
        constexpr int U = Lay::ROWB / 16;
        const int units = (to - from) * U;
        uint8_t* at = smem + Lay::KV_OFF + slot * Lay::TILE + from * Lay::ROWB;
        for (int i = lane; i < units * Lay::NCHUNK; i += 32) {
          const int c = i / units, w = i - c * units;
          *reinterpret_cast<uint4*>(at + c * Lay::CHUNK + w * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      };
      for (int x = x0; x < x1 && ok;) {
        const Seg it = list.at(x, x1);
        x = it.next;
        if (it.j0 >= it.j1) continue;
        const int nj = it.j1 - it.j0;
        // TMEM changes hands between swapped and other items when the products are done.
        if (warp == 9 && items > 0 && was_swapped != it.swapped) ok = wait_items(items);
        if (!ok) break;
        was_swapped = it.swapped;
        ++items;
        if (it.swapped) {
          // S^T = K Q^T (128 keys x N rows) and O^T += V^T P~^T (d x N), N the item's rows rounded up.
          // Split operands: S sums both terms of q; O has 3 N columns, N for each term of P~.  d = 64: V's 64
          // rows twice (LBO 0).
          const uint32_t N = static_cast<uint32_t>(swapped_rows(it.nt * p.G));
          if (warp == 9) {
            const uint32_t idesc = (F8 ? idesc_e4m3_f32(kBM, 0, 0, 0) : idesc_bf16_f32(kBM, 0, 0, 0)) | ((N >> 3) << 17);
            const uint32_t lo = N * Lay::ROWB;  // the lo rows of split queries
            auto desc = [&](uint32_t a) { return SW64 ? sdesc_sw64(a, 16, 512) : sdesc_sw128(a, 16, 1024); };
            ok = wait(Lay::B_QFULL + (nq & 1), (nq >> 1) & 1, kSiteTQFull);
            const uint64_t dq = desc(sb + Lay::Q_OFF + (nq & 1) * Lay::QTILE);
            for (int j = 0; j < nj && ok; ++j) {
              const int s = j & 1;
              const uint32_t n = n_ld + j, slot = n % NR;
              ok = wait(Lay::B_KVFULL + slot, (n / NR) & 1u, kSiteTKvFull);
              if (ok && ((w_used >> s) & 1u)) {  // the stream has read its last scores
                ok = wait(Lay::B_WSFREE + s, (w_phase >> s) & 1u, kSiteTSFree);
                w_phase ^= 1u << s;
              }
              if (!ok) break;
              w_used |= 1u << s;
              tc_fence_after();
              const uint64_t dk = desc(sb + Lay::KV_OFF + slot * Lay::TILE);
              const uint32_t tS = tmem + Lay::TM_S + 128 * s;
              if (elect_one()) {
                constexpr int PER = Lay::ROWB / 32;
#pragma unroll
                for (int kk = 0; kk < D / Lay::KSTEP; ++kk) {
                  const uint32_t off = (kk / PER) * Lay::CHUNK + (kk % PER) * 32;
                  if constexpr (F8) {
                    mma_ss_f8(tS, desc_add(dk, off), desc_add(dq, off), idesc, kk > 0);
                    mma_ss_f8(tS, desc_add(dk, off), desc_add(dq, off + lo), idesc, 1u);
                  } else {
                    mma_ss(tS, desc_add(dk, off), desc_add(dq, off), idesc, kk > 0);
                  }
                }
                tc_commit(bar(Lay::B_WSFULL + s));
                tc_commit(bar(Lay::B_KVEMPTY + slot));
                if (j == nj - 1) tc_commit(bar(Lay::B_QEMPTY + (nq & 1)));
              }
              __syncwarp();
            }
          } else {
            const uint32_t idesc = (F8 ? idesc_e4m3_f32(kBM, 0, 1, 1) | kE5m2B : idesc_bf16_f32(kBM, 0, 1, 1)) | ((Lay::P_TERMS * N >> 3) << 17);
            constexpr int NK = kBN / Lay::KSTEP;
            constexpr int LBO = D == 64 ? 0 : Lay::CHUNK;
            for (int j = 0; j < nj && ok; ++j) {
              const int s = j & 1;
              const uint32_t n = n_ld + j, slot = NR + n % NR;
              const int left = it.len - (it.j0 + j) * kBN;
              const int steps = min(NK, ceil_div(left, Lay::KSTEP));
              ok = wait(Lay::B_KVFULL + slot, (n / NR) & 1u, kSiteTKvFull);
              if (!ok) break;
              clear_rows(slot, left, steps * Lay::KSTEP);
              ok = wait(Lay::B_WPFULL + s, (w_phase >> s) & 1u, kSiteTPFull);
              if (!ok) break;
              w_phase ^= 1u << s;
              tc_fence_after();
              const uint32_t tO = tmem + (s ? Lay::TM_O1 : Lay::TM_O0);
              const uint32_t vbase = sb + Lay::KV_OFF + slot * Lay::TILE;
              const uint64_t dv0 = SW64 ? sdesc_sw64(vbase, LBO, 512) : sdesc_sw128(vbase, LBO, 1024);
              const uint32_t more = j >= 2 ? 1u : 0u;
              if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < NK; ++kk) {
                  if (kk >= steps) continue;
                  const uint64_t dv = desc_add(dv0, kk * Lay::KSTEP * Lay::ROWB);
                  const uint64_t dp = sdesc_sw128(sb + Lay::p_row(s, kk * Lay::KSTEP), 16, 1024);
                  if constexpr (F8) mma_ss_f8(tO, dv, dp, idesc, kk > 0 ? 1u : more);
                  else mma_ss(tO, dv, dp, idesc, kk > 0 ? 1u : more);
                }
                tc_commit(bar(Lay::B_WPVDONE + s));
                tc_commit(bar(Lay::B_KVEMPTY + slot));
                if (j == nj - 1) tc_commit(bar(Lay::B_OFULL));
              }
              __syncwarp();
            }
          }
          if (!ok) break;
          n_ld += nj;
          ++nq;
          continue;
        }
        const int rounds = rounds_of(it);
        if (warp == 9) {
          constexpr uint32_t idesc = F8 ? idesc_e4m3_f32(kBM, kHalf, 0, 0) : idesc_bf16_f32(kBM, kHalf, 0, 0);
          constexpr uint32_t idesc_tile = F8 ? idesc_e4m3_f32(kBM, kBN, 0, 0) : idesc_bf16_f32(kBM, kBN, 0, 0);
          auto desc = [&](uint32_t a) { return SW64 ? sdesc_sw64(a, 16, 512) : sdesc_sw128(a, 16, 1024); };
          for (int k = 0; k < (it.two ? 2 : 1) && ok; ++k)
            ok = wait(Lay::B_QFULL + ((nq + k) & 1), ((nq + k) >> 1) & 1, kSiteTQFull);
          const uint64_t dq0 = desc(sb + Lay::Q_OFF + (nq & 1) * Lay::QTILE);
          const uint64_t dq1 = it.two ? desc(sb + Lay::Q_OFF + ((nq + 1) & 1) * Lay::QTILE) : dq0;
          // A round: one set of waits, then the products of both streams.
          for (int v = 0; v < rounds && ok; ++v) {
            const Unit u0 = unit_at(it, v, 0), u1 = unit_at(it, v, 1);
            if (!u0.live) continue;
            const uint32_t n = n_ld + u0.j, slot = n % NR;
            const bool full = full_tile(it, u0.j);
            if (u0.half == 0) ok = wait(Lay::B_KVFULL + slot, (n / NR) & 1u, kSiteTKvFull);
            const int b0 = 2 * (v & 1), b1 = b0 + 1;
            // the buffers' last P~ have been multiplied
            if (ok && ((used >> b0) & 1u)) {
              ok = wait(Lay::B_PVDONE + b0, (phases >> b0) & 1u, kSiteTPvDone);
              phases ^= 1u << b0;
            }
            if (ok && u1.live && ((used >> b1) & 1u)) {
              ok = wait(Lay::B_PVDONE + b1, (phases >> b1) & 1u, kSiteTPvDone);
              phases ^= 1u << b1;
            }
            if (!ok) break;
            used |= (u1.live ? 3u : 1u) << b0;
            tc_fence_after();
            const uint32_t kbase = sb + Lay::KV_OFF + slot * Lay::TILE;
            const uint64_t dk0 = desc(kbase + u0.half * kHalf * Lay::ROWB), dk1 = desc(kbase + u1.half * kHalf * Lay::ROWB);
            const uint32_t tS = tmem + Lay::TM_S + 64 * b0;
            const bool tile_ends = !it.two || u0.half == 1 || !full;
            if (elect_one()) {
              auto products = [&](uint32_t d, uint64_t dq, uint64_t dk, uint32_t shape, auto terms) {
                constexpr int PER = Lay::ROWB / 32;  // K steps of a chunk
#pragma unroll
                for (int term = 0; term < decltype(terms)::value; ++term) {
#pragma unroll
                  for (int kk = 0; kk < D / Lay::KSTEP; ++kk) {
                    const uint32_t off = (kk / PER) * Lay::CHUNK + (kk % PER) * 32;
                    const uint32_t acc = (term > 0 || kk > 0) ? 1u : 0u;
                    if constexpr (F8) mma_ss_f8(d, desc_add(dq, off + term * Lay::TILE), desc_add(dk, off), shape, acc);
                    else mma_ss(d, desc_add(dq, off), desc_add(dk, off), shape, acc);
                  }
                }
              };
              // One row tile: both units' S are the product with the whole tile, which reads q once
              // (63 cycles a step for 128 keys, 2 x 48 for two halves).
              constexpr std::integral_constant<int, 1> one_term{};
              constexpr std::integral_constant<int, F8 ? 2 : 1> all_terms{};
              if (it.two || !u1.live) {
                if (F8 && it.duo) products(tS, dq0, dk0, idesc, one_term);
                else products(tS, dq0, dk0, idesc, all_terms);
                tc_commit(bar(Lay::B_SFULL + b0));
                if (u1.live) {
                  products(tS + 64, dq1, dk1, idesc, all_terms);
                  tc_commit(bar(Lay::B_SFULL + b1));
                }
              } else {
                if (F8 && it.duo) products(tS, dq0, dk0, idesc_tile, one_term);
                else products(tS, dq0, dk0, idesc_tile, all_terms);
                tc_commit(bar(Lay::B_SFULL + b0));
                tc_commit(bar(Lay::B_SFULL + b1));
              }
              if (tile_ends) tc_commit(bar(Lay::B_KVEMPTY + slot));
              if (tile_ends && u0.j == nj - 1) {  // q is free after the item's last S
                tc_commit(bar(Lay::B_QEMPTY + (nq & 1)));
                if (it.two) tc_commit(bar(Lay::B_QEMPTY + ((nq + 1) & 1)));
              }
            }
            __syncwarp();
          }
          if (!ok) break;
        } else {
          constexpr uint32_t idesc = F8 ? idesc_e4m3_f32(kBM, D, 0, 1) | kE5m2A : idesc_bf16_f32(kBM, D, 0, 1);
          constexpr int NK = kHalf / Lay::KSTEP;
          for (int v = 0; v < rounds && ok; ++v) {
            for (int s = 0; s < 2; ++s) {
              const Unit un = unit_at(it, v, s);
              if (!un.live) continue;
              const int buf = 2 * (v & 1) + s;
              const uint32_t n = n_ld + un.j, slot = NR + n % NR;
              const bool full = full_tile(it, un.j);
              const int left = it.len - (it.j0 + un.j) * kBN - un.half * kHalf;  // keys of the half inside the sequence, or more
              const int steps = min(NK, ceil_div(left, Lay::KSTEP));
              if (s == 0 && un.half == 0) {
                ok = wait(Lay::B_KVFULL + slot, (n / NR) & 1u, kSiteTKvFull);
                if (!ok) break;
              }
              if (!it.two || s == 0) clear_rows(slot, un.half * kHalf + left, un.half * kHalf + steps * Lay::KSTEP);
              ok = wait(Lay::B_PFULL + buf, (phases >> buf) & 1u, kSiteTPFull);
              if (!ok) break;
              phases ^= 1u << buf;
              tc_fence_after();
              const uint32_t tP = tmem + Lay::TM_S + 64 * buf, tO = tmem + (s ? Lay::TM_O1 : Lay::TM_O0);
              const uint32_t more = v > 0 ? 1u : 0u;  // not the stream's first product
              const uint32_t vbase = sb + Lay::KV_OFF + slot * Lay::TILE + un.half * kHalf * Lay::ROWB;
              const uint64_t dv0 = SW64 ? sdesc_sw64(vbase, Lay::CHUNK, 512) : sdesc_sw128(vbase, Lay::CHUNK, 1024);
              const bool tile_ends = it.two ? s == 1 && (un.half == 1 || !full) : s == 1 || !full;
              if (elect_one()) {
                auto product = [&](int kk, auto terms) {
                  const uint64_t dv = desc_add(dv0, kk * Lay::KSTEP * Lay::ROWB);
                  const uint32_t acc = kk > 0 ? 1u : more;
                  if constexpr (F8) {
#pragma unroll
                    for (int term = 0; term < decltype(terms)::value; ++term)
                      mma_ts_f8(tO, tP + 16 * term + kk * 8, dv, idesc, term > 0 ? 1u : acc);
                  } else {
                    mma_ts(tO, tP + kk * 8, dv, idesc, acc);
                  }
                };
                if (F8 && it.duo) {
#pragma unroll
                  for (int kk = 0; kk < NK; ++kk)
                    if (kk < steps) product(kk, std::integral_constant<int, 2>{});
                } else {
#pragma unroll
                  for (int kk = 0; kk < NK; ++kk)
                    if (kk < steps) product(kk, std::integral_constant<int, 3>{});
                }
                tc_commit(bar(Lay::B_PVDONE + buf));
                if (tile_ends) tc_commit(bar(Lay::B_KVEMPTY + slot));
                if (tile_ends && un.j == nj - 1) tc_commit(bar(Lay::B_OFULL));
              }
              __syncwarp();
            }
          }
          if (!ok) break;
        }
        n_ld += nj;
        nq += it.two ? 2 : 1;
      }
      // Every product issued by this warp completes before TMEM is freed.
      const int db = Lay::B_DRAIN + (warp == 9 ? 0 : 1);
      if (elect_one()) tc_commit(bar(db));
      __syncwarp();
      if (!__all_sync(0xffffffffu, drain_wait(bar(db), 0u, kDrainLimitNs)) && lane == 0 && p.err)
        atomicCAS(p.err, 0, timeout_code(kSiteTDrain));
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// Joins the parts of the items that were split: CTA c's second slot holds the first part, the
// first slots of CTAs c + 1 .. last the others, in the order of the keys.  A thread joins four
// columns of a row, eight parts at a time.
template <int D>
__global__ void __launch_bounds__(128) combine_kernel(const __grid_constant__ TreeParams p) {
  let_next_launch();
  wait_for_previous();
  const int c = blockIdx.x;
  const int4 hd = p.head[c];
  if (hd.x < 0) return;
  const int rows = hd.z * p.G;
  const int i = blockIdx.y * 128 + threadIdx.x;
  const int col = i / rows, j = i - col * rows;  // columns 4 col.., row j: token j / G, head j % G
  if (col >= D / 4) return;
  const int t = token_of(j, p), g = j - t * p.G;
  const int tile = t / p.tpt;
  const int r = tile * kBM + (t - tile * p.tpt) * p.G + g;
  const int parts = hd.w - c + 1;
  constexpr int N = 8;
  float m = -INFINITY, l = 0.f, acc[4] = {};
  bool bad = false;
  for (int k0 = 0; k0 < parts; k0 += N) {
    float2 st[N];
    float4 v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      st[k] = make_float2(-INFINITY, 0.f);
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k0 + k < parts) {
        const int64_t slot = static_cast<int64_t>(c + k0 + k) * 2 + (k0 + k == 0 ? 1 : 0);
        st[k] = p.stat[slot * (2 * kBM) + r];
        v[k] = reinterpret_cast<const float4*>(p.part)[(slot * (D / 4) + col) * (2 * kBM) + r];
      }
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      top = fmaxf(top, st[k].x);
      bad |= st[k].y < 0.f;
    }
    const float old = m == top ? 1.f : fast_exp2(m - top);
    m = top;
    l *= old;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] *= old;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float w = part_weight(st[k].x, st[k].y, m);
      if (w == 0.f && st[k].y == st[k].y) continue;
      l = fmaf(w, st[k].y, l);
      acc[0] = fmaf(w, v[k].x, acc[0]);
      acc[1] = fmaf(w, v[k].y, acc[1]);
      acc[2] = fmaf(w, v[k].z, acc[2]);
      acc[3] = fmaf(w, v[k].w, acc[3]);
    }
  }
  if (bad) return;
  const float inv = inverse_sum(l) * p.o_scale;
  const int64_t row = static_cast<int64_t>(hd.x + t) * p.Hq + hd.y * p.G + g;
  *reinterpret_cast<uint2*>(p.o + row * D + 4 * col) =
      make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  if (col == 0)
    p.lse[static_cast<int64_t>(hd.y * p.G + g) * p.T + hd.x + t] = natural_lse(m, l, p.p_shift);
}

constexpr int kMaxSmem = 232448;
constexpr int kMaxGrid = 160;  // CTAs the workspace has room for (148 SMs)

template <int D, bool F8>
cudaError_t launch_t(const CUtensorMap& tq, const CUtensorMap& tq32, const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p, int grid,
                     int rows, cudaStream_t st) {
  using Lay = Layout<D, F8>;
  auto kern = tree_kernel<D, F8>;
  const int smem = 1024 + Lay::TABLE_OFF + (5 * p.B + 2) * 4;
  static_assert(1024 + Lay::TABLE_OFF + (5 * 1024 + 2) * 4 <= kMaxSmem, "tables of 1024 sequences fit");
  // Once per device: the call costs the host more than a tensor map does.
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!((ready.load(std::memory_order_acquire) >> dev) & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  e = launch_after(kern, grid, kThreads, smem, st, tq, tq32, tk, tv, p);
  if (e != cudaSuccess) return e;
  return launch_after(combine_kernel<D>, dim3(grid, (rows * (D / 4) + 127) / 128), 128, 0, st, p);
}

}  // namespace

// Parts, statistics and heads, each 256-byte aligned.
size_t tree_workspace(int d) {
  return static_cast<size_t>(kMaxGrid) * 2 * 256 * (d * sizeof(float) + sizeof(float2)) + kMaxGrid * 64;
}

attn_status_t launch_tree(const TreeArgs& a, int sms, cudaStream_t st, cudaError_t* cuda) {
  const attn_cache_t& c = a.cache;
  *cuda = cudaSuccess;
  TreeParams p = {};
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.cu = a.cu;
  p.slots = a.slots;
  p.page_table = c.page_table;
  p.lens = c.lens;
  p.mask = a.mask;
  p.mask_width = a.mask_width;
  p.Hq = a.Hq;
  p.heads = c.heads;
  p.G = a.Hq / c.heads;
  p.B = a.B;
  p.T = a.T;
  p.nslots = c.slots;
  p.max_pages = c.max_pages;
  p.pages = c.pages;
  while ((1 << p.page_shift) < c.page_size) ++p.page_shift;
  p.layer_row = a.layer * c.pages * c.page_size;
  p.rows = c.layers * c.pages * c.page_size;
  p.box_rows = c.page_size < kBN ? c.page_size : kBN;
  p.tpt = kBM / p.G;
  p.inv_g = p.G > 1 ? 0xffffffffu / p.G + 1 : 0u;
  p.tpt32 = kSwapped / p.G;
  const bool f8 = c.e4m3 != 0;
  p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634 * (f8 ? static_cast<double>(c.k_scale) : 1.0));
  p.o_scale = f8 ? c.v_scale : 1.f;
  // P~ <= 2^tau; on the E4M3 path it carries 2^p_shift, so that at most 2^15 of fp16's 65504 and E5M2's
  // 57344 is reached, and the terms' smallest half step, 2^-17, is 2^-28 of the row's reference.  tau 4
  // rather than 2: a maximum of 64 rows grew by 2 in most tiles (a rescale each), by 4 in few.
  p.tau = f8 ? 4.f : 8.f;
  p.p_shift = f8 ? 11.f : 0.f;
  p.err = a.err;
  char* ws = static_cast<char*>(a.ws);
  p.part = reinterpret_cast<float*>(ws);
  ws += static_cast<size_t>(kMaxGrid) * 2 * 256 * c.d * sizeof(float);
  p.stat = reinterpret_cast<float2*>(ws);
  ws += static_cast<size_t>(kMaxGrid) * 2 * 256 * sizeof(float2);
  p.head = reinterpret_cast<int4*>(ws);
  // At most one item more per sequence than full row pairs, and no more tiles than the tables
  // describe.
  const int64_t items = (static_cast<int64_t>(a.B) + a.T / (2 * p.tpt)) * c.heads;
  const int64_t tiles = (static_cast<int64_t>(c.max_pages) * c.page_size + kBN - 1) / kBN;
  if (items > INT32_MAX / (7 * tiles + 20)) return ATTN_ERR_UNSUPPORTED;  // a tile costs at most 7, an item 20
  int grid = static_cast<int>(items * tiles < sms ? items * tiles : sms);
  if (grid > kMaxGrid) grid = kMaxGrid;
  const int rows = (a.T < 2 * p.tpt ? a.T : 2 * p.tpt) * p.G;
  // {d, heads, rows} of K and V, one box per page (or 128 rows of it); q as {d, G, heads, T}.
  const int esz = f8 ? 1 : 2, elems = (c.d * esz < 128 ? c.d : 128 / esz);
  CUtensorMap tq = {}, tq32 = {}, tk, tv;
  const uint64_t kvd[3] = {static_cast<uint64_t>(c.d), static_cast<uint64_t>(c.heads),
                           static_cast<uint64_t>(c.layers) * c.pages * c.page_size};
  const uint64_t kvs[2] = {static_cast<uint64_t>(c.d) * esz, static_cast<uint64_t>(c.heads) * c.d * esz};
  const uint32_t kvb[3] = {static_cast<uint32_t>(elems), 1, static_cast<uint32_t>(p.box_rows)};
  const int swizzle = elems * esz;
  bool ok = attn_internal::make_tensor_map(&tk, c.k, esz, 3, kvd, kvs, kvb, swizzle) &&
            attn_internal::make_tensor_map(&tv, c.v, esz, 3, kvd, kvs, kvb, swizzle);
  if (ok && !f8) {
    const uint64_t qd[4] = {static_cast<uint64_t>(c.d), static_cast<uint64_t>(p.G), static_cast<uint64_t>(c.heads),
                            static_cast<uint64_t>(a.T)};
    const uint64_t qs[3] = {static_cast<uint64_t>(c.d) * 2, static_cast<uint64_t>(p.G) * c.d * 2,
                            static_cast<uint64_t>(a.Hq) * c.d * 2};
    const uint32_t qb[4] = {64, static_cast<uint32_t>(p.G), 1, static_cast<uint32_t>(p.tpt)};
    ok = attn_internal::make_tensor_map(&tq, a.q, 2, 4, qd, qs, qb, 128);
    if (ok && p.tpt32 > 0) {
      const uint32_t q32[4] = {64, static_cast<uint32_t>(p.G), 1, static_cast<uint32_t>(p.tpt32)};
      ok = attn_internal::make_tensor_map(&tq32, a.q, 2, 4, qd, qs, q32, 128);
    }
  }
  if (!ok) return ATTN_ERR_CUDA;
  if (c.d == 128) *cuda = f8 ? launch_t<128, true>(tq, tq32, tk, tv, p, grid, rows, st) : launch_t<128, false>(tq, tq32, tk, tv, p, grid, rows, st);
  else *cuda = f8 ? launch_t<64, true>(tq, tq32, tk, tv, p, grid, rows, st) : launch_t<64, false>(tq, tq32, tk, tv, p, grid, rows, st);
  return ATTN_OK;
}

}  // namespace attn
