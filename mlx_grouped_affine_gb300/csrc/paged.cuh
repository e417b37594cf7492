// Shared by the paged-attention kernels: the call's arguments, how its work is
// cut over the blocks, and how a row's partial results join.
//
// Work.  Queries of one request and one kv head are rows r = i * G + g (i the
// new token, g the query head inside its group of G), so that a tile of rows
// shares every K and V tile it reads.  An item is (request, kv head, TQ
// consecutive new tokens): it walks the key tiles (KT keys each) that any of
// its rows may see.  (A group of more heads than a tile has rows is cut into
// S slices of Gs heads, each walked as a kv head of its own.)  All items' key
// tiles, in order, form one line; an item counts item_cost units for its start
// and end, then one for each tile, W in all, and block c of `parts` takes units
// [c W / parts, (c + 1) W / parts).
// Every block therefore does the same work whatever the requests' lengths are,
// and at most parts - 1 items are cut.  A cut item's pieces leave their running
// maximum, sum and unnormalised output in the workspace, and a second kernel
// joins them in block order (so results repeat bit for bit).
//
// Softmax over a line of keys in pieces: with m = max s, l = sum 2^(s - m) and
// o = sum 2^(s - m) v over each piece, pieces a and b join as
// m = max(ma, mb), l = la 2^(ma - m) + lb 2^(mb - m), and o the same way;
// scores carry scale * log2(e), so the natural-log statistic is
// lse = (m + log2 l) ln 2.
#pragma once
#include <algorithm>

#include "common.cuh"

namespace qmm {
namespace paged {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -INFINITY;
constexpr int kMaxBlocks = 512;  // of an attention launch: descriptors in the workspace

struct AttnArgs {
  const void *q;
  int64_t q_stride;            // elements between tokens; head h at h * D
  const void *k, *v;
  int64_t page_stride, head_stride, token_stride;  // elements
  const int *table;            // [B, width] page ids
  int64_t table_stride;
  const int *starts, *seq;     // [B + 1], [B]
  void *out;
  int64_t out_stride;
  float *lse;                  // [T, Hq] or null
  float *ws;                   // partial rows of cut items
  int *desc;                   // [blocks][8]: the cut item each block continues
  unsigned *err;
  uint32_t spin_limit;
  int page, num_pages;
  int T, B, Hq, Hkv, G, D;
  int S, Gs, heads;            // each group of G heads in S slices of Gs; heads = Hkv * S
  int TQ;                      // new tokens of an item
  int TH;                      // new tokens of 128 of its rows (TQ where it has no more)
  int max_keys;                // width * page, at most 2^31 - 1
  int causal, window;          // window 0: none
  float scale_log2;            // scale * log2(e)
  int min_rows, max_rows;      // requests of another row count are left to the other kernel
  int item_cost;               // units of an item beside its tiles
};

// A request as the kernels use it: lengths clamped so that nothing that the
// arrays hold leads outside the tensors.
struct Request {
  int first, n, len;  // first token, new tokens, keys
};

__device__ __forceinline__ Request request_of(const AttnArgs &a, int b) {
  Request r;
  const int s0 = max(0, min(__ldg(a.starts + b), a.T));
  const int s1 = max(s0, min(__ldg(a.starts + b + 1), a.T));
  r.first = s0;
  r.n = s1 - s0;
  r.len = max(0, min(__ldg(a.seq + b), a.max_keys));
  const int64_t rows = static_cast<int64_t>(r.n) * a.G;
  if (rows < a.min_rows || rows > a.max_rows) r.n = 0;
  return r;
}

// Keys [lo, hi) that the row of new token i sees: its position is
// p = len - n + i; causal rows see keys up to p, a window the last `window`
// of them.  lo >= hi for a row that sees nothing.  hi may be 2^31 - 1 and a tile then
// ends at 2^31: bounds are compared by differences, which an int holds.
struct Span {
  int lo, hi;
};
__device__ __forceinline__ Span span_of(const AttnArgs &a, const Request &r, int i) {
  const int64_t p = static_cast<int64_t>(r.len) - r.n + i;
  int64_t hi = r.len, lo = 0;
  if (a.causal) hi = min(hi, p + 1);
  if (a.window) lo = max(lo, p - a.window + 1);
  Span s;
  s.hi = static_cast<int>(max(hi, int64_t(0)));
  s.lo = static_cast<int>(min(lo, static_cast<int64_t>(a.max_keys)));
  return s;
}

// The keys that any row of item qt (TQ tokens) sees, and its key tiles: at
// least one, so that an item that sees nothing still writes its rows.
struct ItemTiles {
  int lo, hi, tile0, tiles;
};
template <int KT>
__device__ __forceinline__ ItemTiles item_tiles(const AttnArgs &a, const Request &r, int qt) {
  const int i0 = qt * a.TQ, i1 = min(r.n, i0 + a.TQ) - 1;
  ItemTiles t;
  t.lo = span_of(a, r, i0).lo;
  t.hi = span_of(a, r, i1).hi;
  if (t.lo >= t.hi) {
    t.lo = t.hi = 0;
    t.tile0 = 0;
    t.tiles = 1;
  } else {
    t.tile0 = t.lo / KT;
    t.tiles = (t.hi - 1) / KT + 1 - t.tile0;
  }
  return t;
}

__device__ __forceinline__ int items_of(const AttnArgs &a, const Request &r) {
  return (r.n + a.TQ - 1) / a.TQ;
}

// Where a block is in the line of tiles.
struct Cursor {
  Request r;
  int b, h, qt;       // item
  int lo, hi;         // keys of the item
  int tile0, tiles;   // key tiles of the item
  int at;             // next tile of the item, from 0
  int left;           // units left for the block
};

template <int KT>
__device__ __forceinline__ void cursor_item(const AttnArgs &a, Cursor &c) {
  const ItemTiles t = item_tiles<KT>(a, c.r, c.qt);
  c.lo = t.lo;
  c.hi = t.hi;
  c.tile0 = t.tile0;
  c.tiles = t.tiles;
}

// On to the next item, whose start takes item_cost units (only when units are
// left for the block, so one exists; the bound on b stops a block whose lengths
// changed under it).
template <int KT>
__device__ __forceinline__ void cursor_next(const AttnArgs &a, Cursor &c) {
  c.at = 0;
  if (++c.qt >= items_of(a, c.r)) {
    c.qt = 0;
    if (++c.h >= a.heads) {
      c.h = 0;
      do {
        if (++c.b >= a.B) {
          c.left = 0;
          return;
        }
        c.r = request_of(a, c.b);
      } while (c.r.n == 0);
    }
  }
  cursor_item<KT>(a, c);
  c.left = max(c.left - a.item_cost, 0);
}

// The cursor's item from its unit u on, with `left` units from there.  (u is one of
// the item's; the bound holds a block whose lengths changed under it.)
template <int KT>
__device__ __forceinline__ void cursor_start(const AttnArgs &a, Cursor &c, int u, long long left) {
  cursor_item<KT>(a, c);
  const int skip = max(a.item_cost - u, 0);
  c.at = min(max(u - a.item_cost, 0), c.tiles - 1);
  c.left = static_cast<int>(max(left - skip, 0ll));
}

// x * y / z, in 32 bits where the product fits (a 64-bit division costs several
// times as much and stands in every block's start).
__device__ __forceinline__ long long mul_div(long long x, long long y, long long z) {
  const unsigned long long p = static_cast<unsigned long long>(x) * y;
  if ((p | z) >> 32 == 0) return static_cast<unsigned>(p) / static_cast<unsigned>(z);
  return static_cast<long long>(p / static_cast<unsigned long long>(z));
}

template <int NT>
struct PlanScratch {
  long long warp_sum[NT / 32];
  long long found_before, found_tiles;  // tiles before the found request, and its own
  int found;
  unsigned marks[NT / 32];
  Cursor cursor;
};

// Inclusive block scan of one value a thread; also the block's total.
template <int NT>
__device__ __forceinline__ long long block_scan(long long v, PlanScratch<NT> &s, long long *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  __syncthreads();
  if (lane == 31) s.warp_sum[warp] = v;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const long long x = s.warp_sum[w];
    if (w < warp) before += x;
    all += x;
  }
  *total = all;
  return before + v;
}

// Units of one head slice of request r: every step-th item from `from` on.
template <int KT>
__device__ __forceinline__ long long head_tiles(const AttnArgs &a, const Request &r, int from, int step) {
  long long n = 0;
  const int items = items_of(a, r);
  for (int q = from; q < items; q += step) n += item_tiles<KT>(a, r, q).tiles + a.item_cost;
  return n;
}

constexpr int kOwnItems = 4;  // items a thread counts alone; longer requests are counted by the block

// Tiles of the requests [base, base + NT), one a thread.
template <int NT, int KT>
__device__ long long request_tiles(const AttnArgs &a, int base, PlanScratch<NT> &s) {
  const int b = base + threadIdx.x;
  long long mine = 0;
  bool big = false;
  if (b < a.B) {
    const Request r = request_of(a, b);
    big = items_of(a, r) > kOwnItems;
    if (!big) mine = head_tiles<KT>(a, r, 0, 1) * a.heads;
  }
  if (!__syncthreads_or(big)) return mine;
  // Long requests one after another, their items spread over the block.
  const unsigned m = __ballot_sync(0xffffffffu, big);
  if ((threadIdx.x & 31) == 0) s.marks[threadIdx.x >> 5] = m;
  __syncthreads();
  for (int w = 0; w < NT / 32; ++w) {
    for (unsigned bits = s.marks[w]; bits; bits &= bits - 1) {
      const int owner = 32 * w + __ffs(bits) - 1;
      const Request r = request_of(a, base + owner);
      long long total;
      block_scan<NT>(head_tiles<KT>(a, r, threadIdx.x, NT), s, &total);
      if (threadIdx.x == owner) mine = total * a.heads;
    }
  }
  return mine;
}

// The cut item that block `part` continues, for the joining kernel: request,
// head, item, the blocks that hold the item's first and last tiles, and the
// request's first token and count (block
// p holds unit g when p W / parts <= g, so p = ((g + 1) parts - 1) / W).
__device__ __forceinline__ void leave_desc(const AttnArgs &a, const Cursor &c, int part, long long t0,
                                           long long parts, long long W) {
  int *d = a.desc + 8 * part;
  if (c.at == 0 || c.left == 0) {
    d[0] = -1;
    return;
  }
  const long long g0 = t0 - c.at, g1 = g0 + c.tiles - 1;  // units of its first and last tiles
  d[0] = c.b;
  d[1] = c.h;
  d[2] = c.qt;
  d[3] = static_cast<int>(mul_div((g0 + 1) * parts - 1, 1, W));
  d[4] = static_cast<int>(mul_div((g1 + 1) * parts - 1, 1, W));
  d[5] = c.r.first;
  d[6] = c.r.n;
}

// The block's place in the line: its cursor and how many tiles it has (0: none).
// Called by all NT threads of block `part` of `blocks`.  Also leaves in
// desc[part] the cut item that the block continues.
template <int NT, int KT>
__device__ Cursor plan_block(const AttnArgs &a, int part, int blocks, PlanScratch<NT> &s) {
  if (threadIdx.x == 0) s.found = -1;
  // Total, keeping the first chunk's sums.
  long long W = 0, total, kept = 0, kept_incl = 0, kept_total = 0;
  for (int base = 0; base < a.B; base += NT) {
    const long long mine = request_tiles<NT, KT>(a, base, s);
    const long long incl = block_scan<NT>(mine, s, &total);
    if (base == 0) {
      kept = mine;
      kept_incl = incl;
      kept_total = total;
    }
    W += total;
  }
  const long long parts = min(W, static_cast<long long>(blocks));
  Cursor c;
  c.left = 0;
  if (part >= parts) {
    if (threadIdx.x == 0) a.desc[8 * part] = -1;
    return c;
  }
  const long long t0 = mul_div(part, W, parts), t1 = mul_div(part + 1, W, parts);
  // The request that holds tile t0.
  long long before = 0;
  for (int base = 0; base < a.B; base += NT) {
    long long mine = kept, incl = kept_incl;
    total = kept_total;
    if (base != 0) {
      mine = request_tiles<NT, KT>(a, base, s);
      incl = block_scan<NT>(mine, s, &total) + before;
    }
    if (t0 < incl && t0 >= incl - mine) {
      s.found = base + threadIdx.x;
      s.found_before = incl - mine;
      s.found_tiles = mine;
    }
    before += total;
    if (before > t0) break;
  }
  __syncthreads();
  const int b = s.found;
  if (b < 0) {  // only if the lengths changed while the kernel ran
    if (threadIdx.x == 0) a.desc[8 * part] = -1;
    return c;
  }
  const long long in_request = t0 - s.found_before;
  const Request r = request_of(a, b);
  // The head (all head slices of a request have the same tiles), then the item.
  const long long per_head = mul_div(s.found_tiles, 1, a.heads);
  const int h = static_cast<int>(mul_div(in_request, 1, per_head));
  const long long in_head = in_request - h * per_head;
  const int items = items_of(a, r);
  int at = static_cast<int>(in_head);  // its unit of the item
  c.qt = 0;
  if (items > 1) {
    before = 0;
    if (threadIdx.x == 0) s.cursor.qt = s.cursor.at = 0;
    for (int base = 0; base < items; base += NT) {
      const int q = base + threadIdx.x;
      const long long mine = q < items ? item_tiles<KT>(a, r, q).tiles + a.item_cost : 0;
      const long long incl = block_scan<NT>(mine, s, &total) + before;
      if (in_head < incl && in_head >= incl - mine) {
        s.cursor.qt = q;
        s.cursor.at = static_cast<int>(in_head - (incl - mine));
      }
      before += total;
      if (before > in_head) break;
    }
    __syncthreads();
    c.qt = s.cursor.qt;
    at = s.cursor.at;
  }
  c.r = r;
  c.b = b;
  c.h = h;
  cursor_start<KT>(a, c, at, t1 - t0);
  if (threadIdx.x == 0) leave_desc(a, c, part, t0, parts, W);
  return c;
}

// Row r of item (h, qt): its new token in the request and its query head;
// false for a row past the item's tokens or past the group's heads.  (An item of
// 256 rows is two of 128, each with TH tokens of its own.)
__device__ __forceinline__ bool row_of(const AttnArgs &a, const Request &r, int h, int qt, int row,
                                       int *i, int *head) {
  const int in = row & 127, t = in / a.Gs, g = (h % a.S) * a.Gs + (in - t * a.Gs);
  *i = qt * a.TQ + (row >> 7) * a.TH + t;
  *head = (h / a.S) * a.G + g;
  return t < a.TH && *i < r.n && g < a.G;
}

// ------------------------------------------------------------ elements ----

struct ElemF32 {};

template <typename E>
struct Elem {
  using type = uint16_t;
  // The sign, and the lowest bit of the exponent, in each element of a word.
  static constexpr uint32_t kSign = 0x80008000u, kExponent = E::kF16 ? 0x04000400u : 0x00800080u;
  __device__ static __forceinline__ float to_f32(uint16_t v) { return E::to_f32(v); }
  __device__ static __forceinline__ uint16_t from_f32(float v) { return E::from_f32(v); }
};
template <>
struct Elem<ElemF32> {
  using type = float;
  static constexpr uint32_t kSign = 0x80000000u, kExponent = 0x00800000u;
  __device__ static __forceinline__ float to_f32(float v) { return v; }
  __device__ static __forceinline__ float from_f32(float v) { return v; }
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Element offset of key j of request b's head h, or -1 where the table holds
// no page of the pool (the key then reads as zero and the index bit is set).
__device__ __forceinline__ int64_t key_offset(const AttnArgs &a, int b, int h, int j) {
  const int pg = j / a.page, row = j - pg * a.page;
  const int id = __ldg(a.table + b * a.table_stride + pg);
  if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.num_pages)) {
    atomicOr(a.err, kErrIndexBit);
    return -1;
  }
  return id * a.page_stride + row * a.token_stride + h * a.head_stride;
}

// ------------------------------------------------ K and V to shared memory ----
// Tiles in shared memory are 64-column chunks of 128-byte rows, whose 16-byte
// pieces are swizzled by the row: piece x of row r at position x ^ (r % 8).
//
// The unit of a copy is a block of 8 keys.  Where the page size is a multiple of
// 8 a block lies in one page, so that its address is looked up once (one lane a
// block, long before the copy) and a lane's rows follow by adding the row
// stride: cp.async at 12 cycles an instruction of a warp, 43 bytes a cycle of one
// warp and 53 of two.  (A shuffled address for every row: 31 cycles.  TMA boxes
// of a page's rows: 45 cycles a box and 3.5 a 128-byte row, 20 bytes a cycle at
// 16-row pages.)  Rows that hold no key of the item are written as zeros.  At
// other page sizes every row is looked up when it is copied.

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

// A block as one lane looked it up: `how` 0 no key of the item, 1 one page, 2 row
// by row; its table entry and its first row in the page.
struct Block {
  int how, id, row;
};
__device__ __forceinline__ Block look_up(const AttnArgs &a, int b, int key, int lo, int hi) {
  Block x{0, 0, 0};
  if (lo - key >= 8 || key >= hi) return x;
  x.how = 2;
  if (a.page % 8 == 0) {
    x.how = 1;
    const int pg = key / a.page;
    x.row = key - pg * a.page;
    x.id = __ldg(a.table + b * a.table_stride + pg);
  }
  return x;
}

// Element offset of the block's first row in the pool; -1 none, -2 row by row.
__device__ __forceinline__ int64_t block_offset(const AttnArgs &a, const Block &x, int kv) {
  if (x.how != 1) return x.how == 0 ? -1 : -2;
  if (static_cast<unsigned>(x.id) >= static_cast<unsigned>(a.num_pages)) {
    atomicOr(a.err, kErrIndexBit);
    return -1;
  }
  return x.id * a.page_stride + x.row * a.token_stride + kv * a.head_stride;
}

// Where a lane's 16 bytes of a block's rows lie, from the block's place in the
// first chunk: instruction i covers 32 / (DP / 8) rows.
template <int DP>
struct Copier {
  static constexpr int CH = DP / 8, RPI = 32 / CH, N = 8 / RPI;
  uint32_t at[N];
  uint32_t bytes;  // 16, or 0 for columns past the head
  int first, col;
  __device__ __forceinline__ Copier(int D, uint32_t chunk) {
    const int lane = threadIdx.x & 31, ch = lane % CH;
    first = lane / CH;
    col = ch * 8;
    bytes = col < D ? 16u : 0u;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = first + i * RPI;
      at[i] = (ch >> 3) * chunk + r * 128 + (((ch & 7) ^ r) << 4);
    }
  }
  // One block of one pool; off is the same in all lanes.
  __device__ __forceinline__ void copy(const AttnArgs &a, const void *pool, int64_t off, uint32_t dst, int b,
                                       int kv, int key, int lo, int hi) const {
    const uint16_t *src = static_cast<const uint16_t *>(pool) + col;
    if (off >= 0 && key >= lo && hi - key >= 8) {
      src += off + first * a.token_stride;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        cp_async16(dst + at[i], src, bytes);
        src += RPI * a.token_stride;
      }
    } else if (off >= -1) {  // rows [lo, hi) of the block's keys, or none
      src += max(off, int64_t(0)) + first * a.token_stride;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int k = key + first + i * RPI;
        cp_async16(dst + at[i], src, off >= 0 && k >= lo && k < hi ? bytes : 0u);
        src += RPI * a.token_stride;
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < N; ++i) {
        const int k = key + first + i * RPI;
        const int64_t o = k >= lo && k < hi ? key_offset(a, b, kv, k) : -1;
        uint32_t x = at[0];
#pragma unroll
        for (int y = 1; y < N; ++y) x = i == y ? at[y] : x;
        cp_async16(dst + x, src + max(o, int64_t(0)), o >= 0 ? bytes : 0u);
      }
    }
  }
};

// Whether a key that row i does not see, but that its item's tiles hold for other rows
// (at most the item's tokens at either end of the row's keys), has a V that is not
// finite: an element's exponent has all bits set, so that one more at its lowest bit
// carries into the sign's place.  By one warp, a key a lane.  Small, because the size of
// code that a kernel seldom reaches shows in its time: three long requests take 37 us,
// with this loop four times unrolled and plain tests 40.
template <typename E>
__device__ __forceinline__ bool unseen_not_finite(const AttnArgs &a, const Request &r, const Span &s, int b, int h,
                                                  int i) {
  using T = typename Elem<E>::type;
  constexpr uint32_t kSign = Elem<E>::kSign, kOne = Elem<E>::kExponent;
  const int i0 = i / a.TQ * a.TQ, i1 = min(r.n - i0, a.TQ) - 1 + i0;
  const int lo = span_of(a, r, i0).lo, before = max(s.lo - lo, 0), after = max(span_of(a, r, i1).hi - s.hi, 0);
  uint32_t bad = 0;
  for (int x = threadIdx.x & 31; x < before + after; x += 32) {
    const int64_t off = key_offset(a, b, h, x < before ? lo + x : s.hi + (x - before));
    if (off < 0) continue;
    const uint4 *v = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.v) + off);
#pragma unroll 1
    for (int d = 0; d < a.D; d += 16 / sizeof(T)) {
      const uint4 w = *v++;
      bad |= ((w.x & ~kSign) + kOne) | ((w.y & ~kSign) + kOne) | ((w.z & ~kSign) + kOne) | ((w.w & ~kSign) + kOne);
    }
  }
  return __any_sync(0xffffffffu, bad & kSign);
}

// Columns [d0, d1) of an output row by one warp, from the keys it sees alone.  The
// tiled kernels multiply masked keys by weight zero, which is no longer nothing when
// such a key's V is not finite; a row that came out non-finite for that is done again
// here, where a key that the row does not see is never read.  That takes about a
// microsecond a key, so it is left out where the row is non-finite of itself:
// callers do so where its sum of weights is not finite (it has the keys that the row
// sees alone, so one of their scores is not and the row is NaN either way), and here
// where no unseen key's V is to blame.
template <typename E>
__device__ __noinline__ void row_alone(const AttnArgs &a, int b, int head, int i, int d0, int d1) {
  using T = typename Elem<E>::type;
  const int lane = threadIdx.x & 31;
  const int h = head / a.G;
  const Request r = request_of(a, b);
  const Span s = span_of(a, r, i);
  if (!unseen_not_finite<E>(a, r, s, b, h, i)) return;
  const int64_t token = r.first + i;
  const T *q = static_cast<const T *>(a.q) + token * a.q_stride + static_cast<int64_t>(head) * a.D;
  float o[8], qv[8];
  const int n = (a.D + 31) / 32;
#pragma unroll
  for (int d = 0; d < 8; ++d) {
    o[d] = 0.f;
    qv[d] = d < n && lane + 32 * d < a.D ? Elem<E>::to_f32(q[lane + 32 * d]) : 0.f;
  }
  float m = kNegInf, l = 0.f;
  for (int j = s.lo; j < s.hi; ++j) {
    const int64_t off = key_offset(a, b, h, j);
    const T *k = static_cast<const T *>(a.k) + off, *v = static_cast<const T *>(a.v) + off;
    float dot = 0.f;
#pragma unroll
    for (int d = 0; d < 8; ++d)
      if (off >= 0 && d < n && lane + 32 * d < a.D) dot += qv[d] * Elem<E>::to_f32(k[lane + 32 * d]);
#pragma unroll
    for (int x = 16; x; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
    const float sc = dot * a.scale_log2;
    const float mn = fmaxf(m, sc);
    const float base = mn == kNegInf ? 0.f : mn;
    const float f = exp2f(m - base);
    // NaN scores must stay NaN: fmaxf drops them, the exponential keeps them.
    const float p = exp2f(sc - base);
    m = mn;
    l = l * f + p;
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      const float vv = off >= 0 && d < n && lane + 32 * d < a.D ? Elem<E>::to_f32(v[lane + 32 * d]) : 0.f;
      o[d] = o[d] * f + p * vv;
    }
  }
  T *out = static_cast<T *>(a.out) + token * a.out_stride + static_cast<int64_t>(head) * a.D;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int d = 0; d < 8; ++d)
    if (lane + 32 * d >= d0 && lane + 32 * d < d1) out[lane + 32 * d] = Elem<E>::from_f32(o[d] * inv);
}

// A piece of a cut item in the workspace: R rows of DP sums, their maxima and
// their sums of weights.  A block leaves at most two: the item it continues
// (slot 2 c) and the item it begins and does not end (slot 2 c + 1).
template <int R, int DP>
__device__ __forceinline__ float *slot_of(const AttnArgs &a, int block, int begins) {
  return a.ws + (2 * static_cast<int64_t>(block) + begins) * (R * (DP + 2));
}

// Joins the pieces of each cut item.  An item in P pieces is continued by P - 1
// blocks of the attention kernel, and the blocks here of the same numbers, R / 64
// of each (one at least), share its R x DP sums: whatever P and R are, a block
// reads about 64 x DP of them.  While it has few, up to 16 lanes share a column's
// pieces (their reads are in flight together) and join in lane order; else a
// thread has whole columns, four at a time.  The order of the sums is fixed by P
// alone.  (6 items of 51 pieces took 27 us with a warp per row; 64 items of 256
// rows in two or three pieces took 46 us with a block for all of an item's rows.)
// Two blocks an SM (64 registers), so that the blocks of all cut items run at once:
// at 70 registers and one block five fp32 requests take 52.7 us in place of 50.4.
constexpr int kJoinThreads = 512;
constexpr int kJoinLanes = 16;

// Weights that a block keeps: rows it touches x pieces.
template <int R>
constexpr int join_weights(int blocks) { return 2 * R + 3 * blocks; }

template <typename E, int R, int DP>
__global__ void __launch_bounds__(kJoinThreads, 2) join_kernel(const __grid_constant__ AttnArgs a) {
  using T = typename Elem<E>::type;
  extern __shared__ float weight[];  // [rows][P]
  __shared__ float4 sums[kJoinThreads];
  __shared__ unsigned bad_rows[(R + 31) / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_wait();
  const int4 *d = reinterpret_cast<const int4 *>(a.desc + 8 * (blockIdx.x + 1));
  const int4 d0 = d[0], d1 = d[1];
  const int b = d0.x, h = d0.y, qt = d0.z, first = d0.w, last = d1.x;
  if (b < 0) return;
  const Request r{d1.y, d1.z, 0};
  const int P = last - first + 1;
  const int me = (blockIdx.x - first) * gridDim.y + blockIdx.y, all = (P - 1) * gridDim.y;
  constexpr int U = R * DP / 4, UR = DP / 4;  // float4 sums of an item, of a row
  const int u0 = static_cast<int>(static_cast<unsigned>(me * U) / static_cast<unsigned>(all));
  const int u1 = static_cast<int>(static_cast<unsigned>((me + 1) * U) / static_cast<unsigned>(all));
  if (u0 >= u1) return;  // more blocks than sums
  const int row0 = u0 / UR, rows = (u1 - 1) / UR + 1 - row0;
  const int lanes = max(1, min(min(P, kJoinLanes), kJoinThreads / (u1 - u0))), cols = kJoinThreads / lanes;
  const int tc = tid % cols, j = tid / cols;
  // The first columns' sums, in flight while the weights are worked out.
  constexpr int kAhead = 4;
  float4 early[kAhead];
  {
    const int u = min(u0 + tc, u1 - 1), row = u / UR, col = (u - row * UR) * 4;
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int p = j + x * lanes;
      if (lanes > 1 && j < lanes && p < P)
        early[x] = *reinterpret_cast<const float4 *>(slot_of<R, DP>(a, first + p, p == 0) + row * DP + col);
    }
  }
  if (tid < (R + 31) / 32) bad_rows[tid] = 0;
  // A warp per row: the row's maximum and sum, then each piece's share.
  for (int x = warp; x < rows; x += kJoinThreads / 32) {
    int i, head;
    if (!row_of(a, r, h, qt, row0 + x, &i, &head)) continue;
    float m = kNegInf, l = 0.f;
    float l0 = 0.f;  // the sum of the lane's first piece, read beside its maximum
    for (int p = lane; p < P; p += 32) {
      const float *s = slot_of<R, DP>(a, first + p, p == 0) + R * DP + row0 + x;
      const float v = s[0];
      if (p == lane) l0 = s[R];
      weight[x * P + p] = v;
      m = fmaxf(m, v);
    }
#pragma unroll
    for (int y = 16; y; y >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, y));
    const float base = m == kNegInf ? 0.f : m;
    for (int p = lane; p < P; p += 32) {
      const float w = exp2f(weight[x * P + p] - base);
      l += w * (p == lane ? l0 : slot_of<R, DP>(a, first + p, p == 0)[R * DP + R + row0 + x]);
      weight[x * P + p] = w;
    }
#pragma unroll
    for (int y = 16; y; y >>= 1) l += __shfl_xor_sync(0xffffffffu, l, y);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int p = lane; p < P; p += 32) weight[x * P + p] *= inv;
    if (lane == 0 && a.lse && (row0 + x) * UR >= u0)
      a.lse[(static_cast<int64_t>(r.first) + i) * a.Hq + head] = (m + log2f(l)) * kLn2;
  }
  __syncthreads();
  auto write = [&](int row, int col, const float4 &o) {
    int i, head;
    if (col >= a.D || !row_of(a, r, h, qt, row, &i, &head)) return;
    T *out = static_cast<T *>(a.out) + (static_cast<int64_t>(r.first) + i) * a.out_stride +
             static_cast<int64_t>(head) * a.D + col;
    out[0] = Elem<E>::from_f32(o.x);
    out[1] = Elem<E>::from_f32(o.y);
    out[2] = Elem<E>::from_f32(o.z);
    out[3] = Elem<E>::from_f32(o.w);
    if (!(isfinite(o.x) && isfinite(o.y) && isfinite(o.z) && isfinite(o.w)))
      atomicOr(&bad_rows[row / 32], 1u << (row & 31));
  };
  if (lanes == 1) {
    constexpr int kCols = 4;
    for (int c0 = u0 + tid; c0 < u1; c0 += kCols * kJoinThreads) {
      float4 o[kCols];
#pragma unroll
      for (int x = 0; x < kCols; ++x) o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int p = 0; p < P; ++p) {
        const float *s = slot_of<R, DP>(a, first + p, p == 0);
        float4 v[kCols];
#pragma unroll
        for (int x = 0; x < kCols; ++x)
          v[x] = *reinterpret_cast<const float4 *>(s + 4 * min(c0 + x * kJoinThreads, u1 - 1));
#pragma unroll
        for (int x = 0; x < kCols; ++x) {
          const float w = weight[(min(c0 + x * kJoinThreads, u1 - 1) / UR - row0) * P + p];
          o[x].x += w * v[x].x;
          o[x].y += w * v[x].y;
          o[x].z += w * v[x].z;
          o[x].w += w * v[x].w;
        }
      }
#pragma unroll
      for (int x = 0; x < kCols; ++x) {
        const int u = c0 + x * kJoinThreads;
        if (u < u1) write(u / UR, u % UR * 4, o[x]);
      }
    }
  }
#pragma unroll 1
  for (int c0 = u0; lanes > 1 && c0 < u1; c0 += cols) {
    const int u = c0 + tc;
    const int row = u / UR, col = (u - row * UR) * 4;
    const bool live = u < u1 && j < lanes;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
      const float *w = weight + (row - row0) * P;
      if (c0 != u0) {
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
          const int p = j + x * lanes;
          if (p < P)
            early[x] = *reinterpret_cast<const float4 *>(slot_of<R, DP>(a, first + p, p == 0) + row * DP + col);
        }
      }
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        const int p = j + x * lanes;
        if (p < P) {
          o.x += w[p] * early[x].x;
          o.y += w[p] * early[x].y;
          o.z += w[p] * early[x].z;
          o.w += w[p] * early[x].w;
        }
      }
#pragma unroll 4
      for (int p = j + kAhead * lanes; p < P; p += lanes) {
        const float4 x = *reinterpret_cast<const float4 *>(slot_of<R, DP>(a, first + p, p == 0) + row * DP + col);
        o.x += w[p] * x.x;
        o.y += w[p] * x.y;
        o.z += w[p] * x.z;
        o.w += w[p] * x.w;
      }
    }
    __syncthreads();
    sums[tid] = o;
    __syncthreads();
    if (live && j == 0) {
      for (int y = 1; y < lanes; ++y) {
        const float4 x = sums[y * cols + tid];
        o.x += x.x;
        o.y += x.y;
        o.z += x.z;
        o.w += x.w;
      }
      write(row, col, o);
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int x = warp; x < rows; x += kJoinThreads / 32) {
    const int row = row0 + x;
    if (isnan(weight[x * P])) continue;  // the row's sum is not finite
    if (!(bad_rows[row / 32] >> (row & 31) & 1u)) continue;
    int i, head;
    if (!row_of(a, r, h, qt, row, &i, &head)) continue;
    // This block's columns of the row.
    const int from = max(u0, row * UR), to = min(u1, (row + 1) * UR);
    row_alone<E>(a, b, head, i, 4 * (from - row * UR), min(a.D, 4 * (to - row * UR)));
  }
}

// After the attention kernel on the same stream; starts early and waits.
template <typename E, int R, int DP>
cudaError_t launch_join(const AttnArgs &a, int blocks, cudaStream_t stream) {
  if (blocks < 2) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks - 1, R > 64 ? R / 64 : 1);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = sizeof(float) * join_weights<R>(blocks);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<E, R, DP>, a);
}

}  // namespace paged

namespace paged {
// Map of the queries (columns, heads, tokens) with boxes of 64 x Gs x TH.
cudaError_t query_map(const AttnArgs &a, int type, CUtensorMap *q);
// Map of the K pool (columns, rows of a page, heads, pages) with boxes of 64
// columns x `rows` rows.
cudaError_t key_map(const AttnArgs &a, int type, int rows, CUtensorMap *k);
}  // namespace paged

// paged_tiles.cu: fp32, and 16-bit types with heads above 128, on the CUDA cores.
cudaError_t launch_attention_tiles(paged::AttnArgs a, int type, size_t ws_bytes, cudaStream_t stream);
// paged_decode.cu: 16-bit types, heads of at most 128, few rows per kv head.
cudaError_t launch_attention_decode(const paged::AttnArgs &a, int type, size_t ws_bytes, cudaStream_t stream);
// paged_prefill.cu: 16-bit types, heads of at most 128, a positive scale, many
// rows per kv head (tcgen05).
cudaError_t launch_attention_prefill(const paged::AttnArgs &a, int type, size_t ws_bytes, cudaStream_t stream);

}  // namespace qmm
