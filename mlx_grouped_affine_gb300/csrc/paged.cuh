// Shared by the paged-attention kernels: the call's arguments, how its work is
// cut over the blocks, and how a row's partial results join.
//
// Work.  Queries of one request and one kv head are rows r = i * G + g (i the
// new token, g the query head inside its group of G), so that a tile of rows
// shares every K and V tile it reads.  An item is (request, kv head, TQ
// consecutive new tokens): it walks the key tiles (KT keys each) that any of
// its rows may see.  (A group of more heads than a tile has rows is cut into
// S slices of Gs heads, each walked as a kv head of its own.)  All items' key tiles, in order, form one line of W tiles;
// block c of `parts` takes tiles [c W / parts, (c + 1) W / parts).  Every
// block therefore does the same work whatever the requests' lengths are, and
// at most parts - 1 items are cut.  A cut item's pieces leave their running
// maximum, sum and unnormalised output in the workspace, and a second kernel
// joins them in block order (so results repeat bit for bit).
//
// Softmax over a line of keys in pieces: with m = max s, l = sum 2^(s - m) and
// o = sum 2^(s - m) v over each piece, pieces a and b join as
// m = max(ma, mb), l = la 2^(ma - m) + lb 2^(mb - m), and o the same way;
// scores carry scale * log2(e), so the natural-log statistic is
// lse = (m + log2 l) ln 2.
#pragma once
#include "common.cuh"

namespace qmm {
namespace paged {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -INFINITY;

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
  int TQ;                      // new tokens of an item: rows TQ * Gs
  int max_keys;                // width * page, at most 2^31 - 1
  int causal, window;          // window 0: none
  float scale_log2;            // scale * log2(e)
  int min_rows, max_rows;      // requests of another row count are left to the other kernel
  int min_tiles;               // least key tiles worth a block of their own
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
// of them.  lo >= hi for a row that sees nothing.
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
  int left;           // tiles left for the block
};

template <int KT>
__device__ __forceinline__ void cursor_item(const AttnArgs &a, Cursor &c) {
  const ItemTiles t = item_tiles<KT>(a, c.r, c.qt);
  c.lo = t.lo;
  c.hi = t.hi;
  c.tile0 = t.tile0;
  c.tiles = t.tiles;
}

// On to the next item (only when tiles are left for the block, so one exists;
// the bound on b stops a block whose lengths changed under it).
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
}

template <int NT>
struct PlanScratch {
  long long warp_sum[NT / 32];
  long long total;
  long long found_before;  // tiles before the found element
  int found;
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

// Tiles of one head slice of request r: every step-th item from `from` on.
template <int KT>
__device__ __forceinline__ long long head_tiles(const AttnArgs &a, const Request &r, int from, int step) {
  long long n = 0;
  const int items = items_of(a, r);
  for (int q = from; q < items; q += step) n += item_tiles<KT>(a, r, q).tiles;
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
  // Long requests one after another, their items spread over the block.
  __shared__ unsigned marks[NT / 32];
  const unsigned m = __ballot_sync(0xffffffffu, big);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) marks[threadIdx.x >> 5] = m;
  __syncthreads();
  for (int w = 0; w < NT / 32; ++w) {
    for (unsigned bits = marks[w]; bits; bits &= bits - 1) {
      const int owner = 32 * w + __ffs(bits) - 1;
      const Request r = request_of(a, base + owner);
      long long total;
      block_scan<NT>(head_tiles<KT>(a, r, threadIdx.x, NT), s, &total);
      if (threadIdx.x == owner) mine = total * a.heads;
    }
  }
  return mine;
}

// The block's place in the line: its cursor and how many tiles it has (0: none).
// Called by all NT threads of block `part` of `blocks`.  Also leaves in
// desc[part] the cut item that the block continues, for the joining kernel.
template <int NT, int KT>
__device__ Cursor plan_block(const AttnArgs &a, int part, int blocks, PlanScratch<NT> &s) {
  // Total, keeping the first chunk's counts.
  long long W = 0, total;
  long long kept = 0;
  for (int base = 0; base < a.B; base += NT) {
    const long long mine = request_tiles<NT, KT>(a, base, s);
    if (base == 0) kept = mine;
    block_scan<NT>(mine, s, &total);
    W += total;
  }
  long long parts = (W + a.min_tiles - 1) / a.min_tiles;
  if (parts > blocks) parts = blocks;
  Cursor c;
  c.left = 0;
  if (part >= parts) {
    if (threadIdx.x == 0) a.desc[8 * part] = -1;
    return c;
  }
  const long long t0 = part * W / parts, t1 = (part + 1) * W / parts;
  // The request that holds tile t0.
  long long before = 0;
  __syncthreads();
  if (threadIdx.x == 0) s.found = -1;
  for (int base = 0; base < a.B; base += NT) {
    const long long mine = base == 0 ? kept : request_tiles<NT, KT>(a, base, s);
    const long long incl = block_scan<NT>(mine, s, &total) + before;
    if (t0 < incl && t0 >= incl - mine) {
      s.found = base + threadIdx.x;
      s.found_before = incl - mine;
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
  // The head (all heads of a request have the same tiles), then the item.
  block_scan<NT>(head_tiles<KT>(a, r, threadIdx.x, NT), s, &total);
  const int h = static_cast<int>(in_request / total);
  const long long in_head = in_request - h * total;
  before = 0;
  const int items = items_of(a, r);
  __syncthreads();
  for (int base = 0; base < items; base += NT) {
    const int q = base + threadIdx.x;
    const long long mine = q < items ? item_tiles<KT>(a, r, q).tiles : 0;
    const long long incl = block_scan<NT>(mine, s, &total) + before;
    if (in_head < incl && in_head >= incl - mine) {
      s.cursor.qt = q;
      s.cursor.at = static_cast<int>(in_head - (incl - mine));
    }
    before += total;
    if (before > in_head) break;
  }
  __syncthreads();
  c.r = r;
  c.b = b;
  c.h = h;
  c.qt = s.cursor.qt;
  c.at = s.cursor.at;
  c.left = static_cast<int>(t1 - t0);
  cursor_item<KT>(a, c);
  if (threadIdx.x == 0) {
    int *d = a.desc + 8 * part;
    if (c.at == 0) {
      d[0] = -1;
    } else {
      // The blocks that hold the item's first and last tiles: block p holds
      // tile g when p W / parts <= g, so p = ((g + 1) parts - 1) / W.
      const long long g0 = t0 - c.at, g1 = g0 + c.tiles - 1;
      d[0] = c.b;
      d[1] = c.h;
      d[2] = c.qt;
      d[3] = static_cast<int>(((g0 + 1) * parts - 1) / W);
      d[4] = static_cast<int>(((g1 + 1) * parts - 1) / W);
    }
  }
  return c;
}

// Row r of item (h, qt): its new token in the request and its query head;
// false for a row past the item's tokens or past the group's heads.
__device__ __forceinline__ bool row_of(const AttnArgs &a, const Request &r, int h, int qt, int row,
                                       int *i, int *head) {
  const int t = row / a.Gs, g = (h % a.S) * a.Gs + (row - t * a.Gs);
  *i = qt * a.TQ + t;
  *head = (h / a.S) * a.G + g;
  return t < a.TQ && *i < r.n && g < a.G;
}

// ------------------------------------------------------------ elements ----

struct ElemF32 {};

template <typename E>
struct Elem {
  using type = uint16_t;
  __device__ static __forceinline__ float to_f32(uint16_t v) { return E::to_f32(v); }
  __device__ static __forceinline__ uint16_t from_f32(float v) { return E::from_f32(v); }
};
template <>
struct Elem<ElemF32> {
  using type = float;
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

// One output row by one warp, from the keys it sees alone.  The tiled kernels
// multiply masked keys by weight zero, which is no longer nothing when such a
// key's V is not finite; a row that came out non-finite is done again here,
// where a key that the row does not see is never read.
template <typename E>
__device__ __noinline__ void row_alone(const AttnArgs &a, int b, int head, int i) {
  using T = typename Elem<E>::type;
  const int lane = threadIdx.x & 31;
  const Request r = request_of(a, b);
  const Span s = span_of(a, r, i);
  const int64_t token = r.first + i;
  const int h = head / a.G;
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
    if (d < n && lane + 32 * d < a.D) out[lane + 32 * d] = Elem<E>::from_f32(o[d] * inv);
}

// A piece of a cut item in the workspace: R rows of DP sums, their maxima and
// their sums of weights.  A block leaves at most two: the item it continues
// (slot 2 c) and the item it begins and does not end (slot 2 c + 1).
template <int R, int DP>
__device__ __forceinline__ float *slot_of(const AttnArgs &a, int block, int begins) {
  return a.ws + (2 * static_cast<int64_t>(block) + begins) * (R * (DP + 2));
}

// Joins the pieces of each cut item, in block order.  Block (c, y) has 16 rows
// of the item that attention block c continues, when c is the first to
// continue it.  Bytes: each piece read once; a warp per row, 16 bytes a lane.
template <typename E, int R, int DP>
__global__ void __launch_bounds__(128) join_kernel(AttnArgs a) {
  using T = typename Elem<E>::type;
  griddep_wait();
  const int c = blockIdx.x + 1;
  const int *d = a.desc + 8 * c;
  const int b = d[0];
  if (b < 0 || d[3] != c - 1) return;
  const int h = d[1], qt = d[2], first = d[3], last = d[4];
  const Request r = request_of(a, b);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int V = (DP + 127) / 128;  // float4s a lane
  for (int row = blockIdx.y * 16 + warp; row < min(R, (static_cast<int>(blockIdx.y) + 1) * 16); row += 4) {
    int i, head;
    if (!row_of(a, r, h, qt, row, &i, &head)) continue;
    float m = kNegInf;
    for (int p = first + lane; p <= last; p += 32)
      m = fmaxf(m, slot_of<R, DP>(a, p, p == first)[R * DP + row]);
#pragma unroll
    for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    const float base = m == kNegInf ? 0.f : m;
    float l = 0.f;
    float4 o[V];
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = first; p0 <= last; p0 += 32) {
      float w = 0.f, wl = 0.f;
      if (p0 + lane <= last) {
        const float *s = slot_of<R, DP>(a, p0 + lane, p0 + lane == first) + R * DP + row;
        w = exp2f(s[0] - base);
        wl = w * s[R];
      }
      const int n = min(32, last - p0 + 1);
#pragma unroll 4
      for (int p = 0; p < n; ++p) {
        const float wp = __shfl_sync(0xffffffffu, w, p);
        l += __shfl_sync(0xffffffffu, wl, p);
        const float *s = slot_of<R, DP>(a, p0 + p, p0 + p == first) + row * DP;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (128 * j + 4 * lane < DP) {
            const float4 x = *reinterpret_cast<const float4 *>(s + 128 * j + 4 * lane);
            o[j].x += wp * x.x;
            o[j].y += wp * x.y;
            o[j].z += wp * x.z;
            o[j].w += wp * x.w;
          }
        }
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T *out = static_cast<T *>(a.out) + (static_cast<int64_t>(r.first) + i) * a.out_stride +
             static_cast<int64_t>(head) * a.D;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = 128 * j + 4 * lane;
      const float y[4] = {o[j].x * inv, o[j].y * inv, o[j].z * inv, o[j].w * inv};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (col < a.D) {
          out[col + e] = Elem<E>::from_f32(y[e]);
          bad |= !isfinite(y[e]);
        }
      }
    }
    if (lane == 0 && a.lse)
      a.lse[(static_cast<int64_t>(r.first) + i) * a.Hq + head] = (m + log2f(l)) * kLn2;
    if (__any_sync(0xffffffffu, bad)) {
      __syncwarp();
      row_alone<E>(a, b, head, i);
    }
  }
}

// After the attention kernel on the same stream; starts early and waits.
template <typename E, int R, int DP>
cudaError_t launch_join(const AttnArgs &a, int blocks, cudaStream_t stream) {
  if (blocks < 2) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks - 1, (R + 15) / 16);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<E, R, DP>, a);
}

}  // namespace paged

// paged_tiles.cu: every type and head size on the CUDA cores.
cudaError_t launch_attention_tiles(paged::AttnArgs a, int type, size_t ws_bytes, cudaStream_t stream);
// paged_decode.cu: 16-bit types, heads of at most 128, few rows per kv head.
cudaError_t launch_attention_decode(const paged::AttnArgs &a, int type, size_t ws_bytes, cudaStream_t stream);

}  // namespace qmm
