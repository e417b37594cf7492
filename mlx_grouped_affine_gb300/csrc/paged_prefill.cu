// Paged attention for many query rows per kv head (prompts, chunks of prompts)
// on the sm_103a tensor cores.
//
// Per key tile of 128 keys, 256 query rows and heads of D: 4 * 128 * 256 * D
// flops and 128 * 256 exponentials, against 512 D bytes of K and V: the tensor
// pipe and the exponentials bound it.  One persistent block per SM; its item is
// two halves of 128 rows (rows are (token, head of the group) pairs, so every
// row of an item shares its K and V).  For each half h and key tile j
//   S_h = Q_h K_j^T     tcgen05.mma, 128 x 128 fp32 in TMEM
//   P_h = 2^(S_h - m)   a row per thread; 16-bit P over S_h in TMEM
//   O_h += P_h V_j      tcgen05.mma with P from TMEM, 128 x D fp32 in TMEM
// and the halves take turns: while one is in its softmax the other has the
// tensor pipe.  Roles:
//   warps 0-3, 4-7  softmax and output of half 0, 1 (thread = row = TMEM lane)
//   warp 8          TMA: Q, and a ring of K and V tiles, a box of a page's rows
//                   at a time, lanes in parallel
//   warp 9          issues the MMAs (one lane); owns the TMEM allocation
// The running maximum moves lazily: P is relative to a row maximum m that is
// only raised, and O and the row sum rescaled, when a score exceeds it by more
// than 2^8 (P stays below 256, exact in both types' range; the result is the
// same because O and the sum share m).
//
// Waits are bounded; one that runs out sets the error word and an abort flag
// that stops every role, and the block still drains its copies and MMAs.
//
// Shared tiles are 64-column chunks of 128-byte rows, 128-byte swizzled; K and
// Q chunks are K-major operands (8-row groups 1024 bytes apart), V chunks
// MN-major ones (atoms of 64 columns x 8 keys).
//
// The last page's rows past the request's end are stale: P is zero there, but
// zero times a stale infinity is not nothing.  The box that holds the end is
// therefore loaded shift rows early, so that it ends with the last key: the
// rows before a page's first read as zero, rows of the page before the box are
// the request's own.  The box's columns of S move with it, and the mask knows.
#include "paged.cuh"

namespace qmm {
namespace paged {
namespace {

constexpr int R = 256, KT = 128, kSoftmaxWarps = 8, NT = 32 * (kSoftmaxWarps + 2);
constexpr float kLazy = 8.f;  // log2 by which scores may exceed the row's reference

template <int DP>
struct Tile {
  static constexpr uint32_t CHUNK = 128 * 128;          // 128 rows of 64 columns
  static constexpr uint32_t TILE = CHUNK * (DP / 64);   // Q half, K or V tile
  static constexpr int SLOTS = DP == 128 ? 5 : 8;
  static constexpr uint32_t O0 = 256;                   // TMEM: S_0 at 0, S_1 at 128, O_0, O_1
};

struct Barriers {
  uint64_t q_full, q_empty, kv_full[8], kv_empty[8], s_full[2], p_ready[2], o_full[2], o_empty[2], mma_done;
  uint32_t tmem_base;
  int abort;
};

template <int DP>
constexpr size_t smem_bytes() {
  return 2 * Tile<DP>::TILE + Tile<DP>::SLOTS * Tile<DP>::TILE + sizeof(Barriers);
}

// ------------------------------------------------------------- PTX glue ----

// Whole-warp bounded wait; false when it ran out or another role gave up.
__device__ __forceinline__ bool wait_warp(uint64_t *b, uint32_t parity, volatile int *abort, unsigned *err,
                                       uint32_t limit) {
  uint32_t spins = 0;
  while (true) {
    if (__all_sync(0xffffffffu, mbar_try_wait(b, parity))) return true;
    if ((++spins & 255u) == 0 || spins >= limit) {
      int stop = *abort;
      if (!stop && spins >= limit) {
        stop = 1;
        *abort = 1;
        atomicOr(err, kErrTimeoutBit);
      }
      if (__any_sync(0xffffffffu, stop)) return false;
    }
  }
}

__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

// Descriptor of a 128-byte swizzled operand (start, leading and stride byte
// offsets in units of 16, version 1, swizzle mode 2).  K-major: 8-row groups
// 1024 bytes apart.  MN-major: atoms 16384 bytes apart along N (a 64-column
// chunk of 128 keys), 1024 along K.
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, uint32_t lead) {
  uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(lead >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// kind::f16, fp32 accumulator, M = 128; B transposed (MN-major) for V.
template <typename E, int N, bool BMN>
__host__ __device__ constexpr uint32_t idesc() {
  return (1u << 4) | (E::kF16 ? 0u : (1u << 7) | (1u << 10)) | (BMN ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}

template <uint32_t IDESC>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(IDESC), "r"(acc)
      : "memory");
}
template <uint32_t IDESC>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(IDESC), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
      : "memory");
}


// 32 columns of this warp's 32 TMEM lanes; no wait.
template <int O, int N>
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float (&f)[N]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(f[O]), "=f"(f[O + 1]), "=f"(f[O + 2]), "=f"(f[O + 3]), "=f"(f[O + 4]), "=f"(f[O + 5]),
        "=f"(f[O + 6]), "=f"(f[O + 7]), "=f"(f[O + 8]), "=f"(f[O + 9]), "=f"(f[O + 10]), "=f"(f[O + 11]),
        "=f"(f[O + 12]), "=f"(f[O + 13]), "=f"(f[O + 14]), "=f"(f[O + 15]), "=f"(f[O + 16]), "=f"(f[O + 17]),
        "=f"(f[O + 18]), "=f"(f[O + 19]), "=f"(f[O + 20]), "=f"(f[O + 21]), "=f"(f[O + 22]), "=f"(f[O + 23]),
        "=f"(f[O + 24]), "=f"(f[O + 25]), "=f"(f[O + 26]), "=f"(f[O + 27]), "=f"(f[O + 28]), "=f"(f[O + 29]),
        "=f"(f[O + 30]), "=f"(f[O + 31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]),
      "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}
// 16 columns times f, in place.
__device__ __forceinline__ void tmem_scale16(uint32_t addr, float f) {
  float o[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(o[0]), "=f"(o[1]), "=f"(o[2]), "=f"(o[3]), "=f"(o[4]), "=f"(o[5]), "=f"(o[6]), "=f"(o[7]),
        "=f"(o[8]), "=f"(o[9]), "=f"(o[10]), "=f"(o[11]), "=f"(o[12]), "=f"(o[13]), "=f"(o[14]), "=f"(o[15])
      : "r"(addr));
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] *= f;
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"f"(
          o[0]),
      "f"(o[1]), "f"(o[2]), "f"(o[3]), "f"(o[4]), "f"(o[5]), "f"(o[6]), "f"(o[7]), "f"(o[8]), "f"(o[9]),
      "f"(o[10]), "f"(o[11]), "f"(o[12]), "f"(o[13]), "f"(o[14]), "f"(o[15]), "r"(addr)
      : "memory");
}

// ---------------------------------------------------------------- pieces ----

// Key tiles of a piece [t0, t1) that half h's rows see; from == to: none.
struct Tiles {
  int from, to;
};
__device__ __forceinline__ Tiles half_tiles(const AttnArgs &a, const Cursor &c, int h, int t0, int t1) {
  const int i0 = c.qt * a.TQ + h * a.TH;
  Tiles t{t0, t0};
  if (i0 >= c.r.n) return t;
  const int lo = span_of(a, c.r, i0).lo, hi = span_of(a, c.r, min(c.r.n, i0 + a.TH) - 1).hi;
  if (lo >= hi) return t;
  const int from = max(t0, lo / KT), to = min(t1, (hi - 1) / KT + 1);
  if (from < to) t = Tiles{from, to};
  return t;
}

// The next piece of the block: the cursor's item from tile t0 to t1, the
// tiles of each half, and those that either needs.
struct Piece {
  int t0, t1;
  Tiles half[2], any;
  bool whole;
};
__device__ __forceinline__ Piece piece_of(const AttnArgs &a, const Cursor &c) {
  Piece p;
  const int n = min(c.left, c.tiles - c.at);
  p.t0 = c.tile0 + c.at;
  p.t1 = p.t0 + n;
  p.whole = c.at == 0 && n == c.tiles;
  p.half[0] = half_tiles(a, c, 0, p.t0, p.t1);
  p.half[1] = half_tiles(a, c, 1, p.t0, p.t1);
  const bool e0 = p.half[0].from == p.half[0].to, e1 = p.half[1].from == p.half[1].to;
  p.any.from = e0 ? p.half[1].from : e1 ? p.half[0].from : min(p.half[0].from, p.half[1].from);
  p.any.to = e0 ? p.half[1].to : e1 ? p.half[0].to : max(p.half[0].to, p.half[1].to);
  return p;
}
__device__ __forceinline__ void piece_done(const AttnArgs &a, Cursor &c, const Piece &p) {
  c.left -= p.t1 - p.t0;
  if (c.left > 0) cursor_next<KT>(a, c);
}

// ----------------------------------------------------------------- roles ----

template <int DP>
__device__ void load_role(const AttnArgs &a, Cursor c, const CUtensorMap *qmap, const CUtensorMap *kmap,
                          const CUtensorMap *vmap, int box, uint8_t *sq, uint8_t *skv, Barriers *bars) {
  using X = Tile<DP>;
  const int lane = threadIdx.x & 31;
  volatile int *abort = &bars->abort;
  const int boxes = KT / box;  // 1 to 128 a tile, four a lane at most
  uint32_t count = 0, q_count = 0;  // tiles and Qs loaded
  bool ok = true;
  while (ok && c.left > 0) {
    const Piece p = piece_of(a, c);
    if (p.any.from < p.any.to) {
      // Q of both halves, once the previous one has been multiplied.
      ok = wait_warp(&bars->q_empty, (q_count & 1) ^ 1u, abort, a.err, a.spin_limit);
      if (!ok) break;
      if (lane == 0) {
        const uint32_t rows = a.Gs * a.TH;
        mbar_expect_tx(&bars->q_full, 2 * (DP / 64) * rows * 128);
        const int head = (c.h / a.S) * a.G + (c.h % a.S) * a.Gs;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int x = 0; x < DP / 64; ++x)
            tma_box(smem_u32(sq + h * X::TILE + x * X::CHUNK), qmap, 64 * x, head,
                    c.r.first + c.qt * a.TQ + h * a.TH, 0, &bars->q_full);
      }
      __syncwarp();
      ++q_count;
      const int kv = c.h / a.S;
      int id[4], row[4];
      auto look = [&](int tile) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int bx = lane + 32 * x, key = tile * KT + bx * box;
          id[x] = 0;
          row[x] = -KT;  // no key of the item in the box
          if (bx < boxes && tile < p.any.to && key + box > c.lo && key < c.hi) {
            const int pg = key / a.page;
            id[x] = __ldg(a.table + c.b * a.table_stride + pg);
            // The box that holds the request's end ends with its last key.
            row[x] = key - pg * a.page - max(0, key + box - c.r.len);
          }
        }
      };
      look(p.any.from);
      for (int j = p.any.from; ok && j < p.any.to; ++j) {
        int page[4], at[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const bool known = static_cast<unsigned>(id[x]) < static_cast<unsigned>(a.num_pages);
          if (row[x] > -KT && !known) atomicOr(a.err, kErrIndexBit);
          // Past the pool's end: reads as zeros.
          page[x] = row[x] > -KT && known ? id[x] : a.num_pages;
          at[x] = row[x] > -KT ? row[x] : 0;
        }
        look(j + 1);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const uint32_t slot = count % X::SLOTS, round = count / X::SLOTS;
          ok = wait_warp(&bars->kv_empty[slot], (round & 1) ^ 1u, abort, a.err, a.spin_limit);
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(&bars->kv_full[slot], X::TILE);
          __syncwarp();
          const uint32_t dst = smem_u32(skv + slot * X::TILE);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int bx = lane + 32 * x;
            if (bx < boxes) {
#pragma unroll
              for (int y = 0; y < DP / 64; ++y)
                tma_box(dst + y * X::CHUNK + bx * box * 128, v ? vmap : kmap, 64 * y, at[x], kv, page[x],
                         &bars->kv_full[slot]);
            }
          }
          __syncwarp();
          ++count;
        }
      }
    }
    if (ok) piece_done(a, c, p);
  }
  // Stopped early: the copies in flight land before the block ends (bounded).
  if (!ok) {
    if (q_count) {
      for (uint32_t s = 0; s < kDefaultWaitLimit; ++s)
        if (__all_sync(0xffffffffu, mbar_try_wait(&bars->q_full, (q_count - 1) & 1))) break;
    }
    for (uint32_t n = count > X::SLOTS ? count - X::SLOTS : 0; n < count; ++n) {
      for (uint32_t s = 0; s < kDefaultWaitLimit; ++s)
        if (__all_sync(0xffffffffu, mbar_try_wait(&bars->kv_full[n % X::SLOTS], (n / X::SLOTS) & 1))) break;
    }
  }
}

template <typename E, int DP>
__device__ void mma_role(const AttnArgs &a, Cursor c, uint8_t *sq, uint8_t *skv, Barriers *bars, uint32_t tmem) {
  using X = Tile<DP>;
  const int lane = threadIdx.x & 31;
  volatile int *abort = &bars->abort;
  uint32_t count = 0, q_count = 0;         // K/V tiles and Qs consumed
  uint32_t p_count[2] = {0, 0}, o_count[2] = {0, 0};
  bool ok = true;
  auto full = [&](uint32_t n) {
    return wait_warp(&bars->kv_full[n % X::SLOTS], (n / X::SLOTS) & 1, abort, a.err, a.spin_limit);
  };
  while (ok && c.left > 0) {
    const Piece p = piece_of(a, c);
    if (p.any.from < p.any.to) {
      ok = wait_warp(&bars->q_full, q_count & 1, abort, a.err, a.spin_limit);
      ++q_count;
      // Step j: the products of tile j - 1 with V, then of tile j with Q.  Tile j's
      // K is number count + 2 (j - from) of the ring, its V the next.
      for (int j = p.any.from; ok && j <= p.any.to; ++j) {
        const uint32_t kn = count + 2 * (j - p.any.from), vn = kn - 1;
        if (j < p.any.to) ok = full(kn);
        if (ok && j > p.any.from) ok = full(vn);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!ok) break;
          if (j > p.half[h].from && j <= p.half[h].to) {
            const bool first = j - 1 == p.half[h].from;
            // The previous piece's output has left O_h.
            if (first) {
              ok = wait_warp(&bars->o_empty[h], (o_count[h] & 1) ^ 1u, abort, a.err, a.spin_limit);
              ++o_count[h];
            }
            ok = ok && wait_warp(&bars->p_ready[h], p_count[h] & 1, abort, a.err, a.spin_limit);
            if (!ok) break;
            ++p_count[h];
            tc_fence_after();
            if (lane == 0) {
              const uint32_t v = smem_u32(skv + vn % X::SLOTS * X::TILE);
              const uint32_t o = tmem + X::O0 + h * DP, pa = tmem + 128 * h;
#pragma unroll
              for (int k = 0; k < KT / 16; ++k)
                mma_ts<idesc<E, DP, true>()>(o, pa + 8 * k, smem_desc(v + 2048 * k, X::CHUNK), !first || k);
              if (j == p.half[h].to) mma_commit(&bars->o_full[h]);
            }
            __syncwarp();
          }
          if (j >= p.half[h].from && j < p.half[h].to) {
            if (lane == 0) {
              const uint32_t q = smem_u32(sq + h * X::TILE), k = smem_u32(skv + kn % X::SLOTS * X::TILE);
#pragma unroll
              for (int x = 0; x < DP / 16; ++x) {
                const uint32_t at = (x >> 2) * X::CHUNK + (x & 3) * 32;
                mma_ss<idesc<E, KT, false>()>(tmem + 128 * h, smem_desc(q + at, 16), smem_desc(k + at, 16), x != 0);
              }
              mma_commit(&bars->s_full[h]);
            }
            __syncwarp();
          }
        }
        if (!ok) break;
        if (lane == 0) {
          if (j > p.any.from) mma_commit(&bars->kv_empty[vn % X::SLOTS]);
          if (j < p.any.to) mma_commit(&bars->kv_empty[kn % X::SLOTS]);
          if (j == p.any.to - 1) mma_commit(&bars->q_empty);
        }
        __syncwarp();
      }
      count += 2 * (p.any.to - p.any.from);
    }
    if (ok) piece_done(a, c, p);
  }
  // Every MMA retires before the block frees its TMEM.
  if (lane == 0) mma_commit(&bars->mma_done);
  __syncwarp();
  for (uint32_t s = 0; s < kDefaultWaitLimit; ++s)
    if (__all_sync(0xffffffffu, mbar_try_wait(&bars->mma_done, 0))) break;
}

// Bits [from, to) of a word whose bit 0 is column `base`.
__device__ __forceinline__ uint32_t bits_of(int from, int to, int base) {
  const int lo = max(from - base, 0), hi = min(to - base, 32);
  if (lo >= hi) return 0u;
  return (hi == 32 ? 0xFFFFFFFFu : (1u << hi) - 1u) & ~((1u << lo) - 1u);
}

template <typename E, int DP>
__device__ void softmax_role(const AttnArgs &a, Cursor c, int box, Barriers *bars, uint32_t tmem) {
  using X = Tile<DP>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = warp >> 2;
  const int row = threadIdx.x;  // of the item; also half * 128 + TMEM lane
  const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
  const uint32_t ts = tmem + 128 * h + lanes, to = tmem + X::O0 + h * DP + lanes;
  volatile int *abort = &bars->abort;
  uint32_t s_count = 0, o_count = 0;
  bool continues = c.at != 0;
  while (c.left > 0) {
    const Piece p = piece_of(a, c);
    int i, head;
    const bool live = row_of(a, c.r, c.h, c.qt, row, &i, &head);
    const Span span = live ? span_of(a, c.r, i) : Span{0, 0};
    // Keys that every live row of the warp sees.
    int deep_lo = live ? span.lo : 0, deep_hi = live ? span.hi : 0x7FFFFFFF;
#pragma unroll
    for (int x = 16; x; x >>= 1) {
      deep_lo = max(deep_lo, __shfl_xor_sync(0xffffffffu, deep_lo, x));
      deep_hi = min(deep_hi, __shfl_xor_sync(0xffffffffu, deep_hi, x));
    }
    float m = kNegInf, l = 0.f;
    for (int j = p.half[h].from; j < p.half[h].to; ++j) {
      if (!wait_warp(&bars->s_full[h], s_count & 1, abort, a.err, a.spin_limit)) return;
      ++s_count;
      tc_fence_after();
      float s[KT];
      tmem_ld32<0>(ts, s);
      tmem_ld32<32>(ts + 32, s);
      tmem_ld32<64>(ts + 64, s);
      tmem_ld32<96>(ts + 96, s);
      tmem_wait_ld();
      const int key0 = j * KT;
      if (key0 < deep_lo || key0 + KT > deep_hi) {
        // The row's columns: keys [lo, hi); from the box that holds the request's
        // end on, columns are `shift` past their keys.
        const int tail = c.r.len % box, shift = tail ? box - tail : 0;
        const int edge = shift ? c.r.len - tail - key0 : KT;  // that box's first column
        const int lo = span.lo - key0, hi = span.hi - key0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t seen = bits_of(lo, min(hi, edge), 32 * w);
          if (shift) seen |= bits_of(max(lo, edge) + shift, hi + shift, 32 * w);
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (!(seen >> x & 1u)) s[32 * w + x] = kNegInf;
        }
      }
      float top = s[0];
#pragma unroll
      for (int x = 1; x < KT; ++x) top = fmaxf(top, s[x]);
      top *= a.scale_log2;
      // Raise the reference when a score is far above it (and in the first tile).
      if (__any_sync(0xffffffffu, top > m + kLazy)) {
        const float up = fmaxf(m, top);
        const float f = exp2_fast(m - (up == kNegInf ? 0.f : up));
        m = up;
        l *= f;
        if (j > p.half[h].from) {
          // O_h is complete up to the previous tile: S_h was committed after it.
#pragma unroll 1
          for (int x = 0; x < DP / 16; ++x) tmem_scale16(to + 16 * x, f);
        }
      }
      const float base = m == kNegInf ? 0.f : -m;
      float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        uint32_t pk[32];
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          const float e0 = exp2_fast(fmaf(s[64 * y + 2 * x], a.scale_log2, base));
          const float e1 = exp2_fast(fmaf(s[64 * y + 2 * x + 1], a.scale_log2, base));
          sum0 += e0;
          sum1 += e1;
          pk[x] = E::pack2(e0, e1);  // rounded once to the element type for the product with V
        }
        tmem_st32(ts + 32 * y, pk);
      }
      l += sum0 + sum1;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->p_ready[h]);
    }
    // The piece's rows: to the output, or to the workspace when the item is cut.
    const bool any = p.half[h].from < p.half[h].to;
    if (any) {
      if (!wait_warp(&bars->o_full[h], o_count & 1, abort, a.err, a.spin_limit)) return;
      ++o_count;
      tc_fence_after();
    }
    const float inv = !p.whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
    const int64_t token = static_cast<int64_t>(c.r.first) + i;
    uint16_t *out = static_cast<uint16_t *>(a.out) + token * a.out_stride + static_cast<int64_t>(head) * a.D;
    float *piece = slot_of<R, DP>(a, blockIdx.x, !continues);
    bool bad = false;
#pragma unroll
    for (int x = 0; x < DP / 32; ++x) {
      float o[32];
      if (any) {
        tmem_ld32<0>(to + 32 * x, o);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int y = 0; y < 32; ++y) o[y] = 0.f;
      }
#pragma unroll
      for (int y = 0; y < 32; ++y) {
        o[y] = any ? o[y] * inv : 0.f;
        bad |= !isfinite(o[y]);
      }
      if (!p.whole) {
#pragma unroll
        for (int y = 0; y < 32; y += 4)
          *reinterpret_cast<float4 *>(piece + row * DP + 32 * x + y) = make_float4(o[y], o[y + 1], o[y + 2], o[y + 3]);
      } else if (live) {
#pragma unroll
        for (int y = 0; y < 32; y += 8)
          if (32 * x + y < a.D)
            *reinterpret_cast<uint4 *>(out + 32 * x + y) =
                make_uint4(E::pack2(o[y], o[y + 1]), E::pack2(o[y + 2], o[y + 3]), E::pack2(o[y + 4], o[y + 5]),
                           E::pack2(o[y + 6], o[y + 7]));
      }
    }
    if (any) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->o_empty[h]);
    }
    if (!p.whole) {
      piece[R * DP + row] = m;
      piece[R * DP + R + row] = l;
    } else if (live && a.lse) {
      a.lse[token * a.Hq + head] = (m + log2f(l)) * kLn2;
    }
    unsigned votes = __ballot_sync(0xffffffffu, bad && live && p.whole);
    if (votes) {
      __syncwarp();
      for (; votes; votes &= votes - 1) {
        const int x = __ffs(votes) - 1;
        row_alone<E>(a, c.b, __shfl_sync(0xffffffffu, head, x), __shfl_sync(0xffffffffu, i, x), 0, a.D);
      }
    }
    continues = false;
    piece_done(a, c, p);
  }
}

template <typename E, int DP>
__global__ void __launch_bounds__(NT, 1)
prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
               const __grid_constant__ CUtensorMap vmap, AttnArgs a, int box) {
  using X = Tile<DP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sq = smem, *skv = smem + 2 * X::TILE;
  Barriers *bars = reinterpret_cast<Barriers *>(skv + X::SLOTS * X::TILE);
  const int warp = threadIdx.x >> 5;
  static_assert(sizeof(PlanScratch<NT>) <= X::TILE, "the plan's scratch lies in the ring");
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&qmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 1);
    for (int i = 0; i < X::SLOTS; ++i) {
      mbar_init(&bars->kv_full[i], 1);
      mbar_init(&bars->kv_empty[i], 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&bars->s_full[h], 1);
      mbar_init(&bars->p_ready[h], 4);
      mbar_init(&bars->o_full[h], 1);
      mbar_init(&bars->o_empty[h], 4);
    }
    mbar_init(&bars->mma_done, 1);
    bars->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  const Cursor c = plan_block<NT, KT>(a, blockIdx.x, gridDim.x, *reinterpret_cast<PlanScratch<NT> *>(skv));
  if (c.left <= 0) return;
  if (a.Gs * a.TH < 128) {
    // Rows of Q that no load writes: zeros, so that they multiply as such.
    for (uint32_t x = threadIdx.x * 16; x < 2 * X::TILE; x += NT * 16)
      *reinterpret_cast<uint4 *>(sq + x) = make_uint4(0, 0, 0, 0);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  if (warp == kSoftmaxWarps + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&bars->tmem_base)),
                 "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp < kSoftmaxWarps) {
    softmax_role<E, DP>(a, c, box, bars, tmem);
  } else {
    if (warp == kSoftmaxWarps) load_role<DP>(a, c, &qmap, &kmap, &vmap, box, sq, skv, bars);
    else if (warp == kSoftmaxWarps + 1) mma_role<E, DP>(a, c, sq, skv, bars, tmem);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kSoftmaxWarps + 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
  }
}

template <typename E, int DP>
cudaError_t launch_t(AttnArgs a, size_t ws_bytes, cudaStream_t stream) {
  a.S = (a.G + 127) / 128;
  a.Gs = (a.G + a.S - 1) / a.S;
  a.heads = a.Hkv * a.S;
  a.TH = 128 / a.Gs;
  a.TQ = 2 * a.TH;
  a.min_tiles = 1;
  const int box = box_rows(a.page, KT);
  const int type = E::kF16 ? kTypeF16 : kTypeBF16;
  CUtensorMap q, k, v;
  cudaError_t e = pool_maps(a, type, box, &k, &v);
  if (e == cudaSuccess) e = query_map(a, type, &q);
  if (e != cudaSuccess) return e;
  constexpr size_t smem = smem_bytes<DP>();
  e = ensure_smem_limit<prefill_kernel<E, DP>>(smem);
  if (e != cudaSuccess) return e;
  int blocks = sm_count();
  const size_t per_block = 2 * sizeof(float) * R * (DP + 2);
  blocks = static_cast<int>(std::min<size_t>(std::min(blocks, kMaxBlocks), ws_bytes / per_block));
  prefill_kernel<E, DP><<<blocks, NT, smem, stream>>>(q, k, v, a, box);
  const cudaError_t le = cudaGetLastError();
  return le != cudaSuccess ? le : launch_join<E, R, DP>(a, blocks, stream);
}

template <typename E>
cudaError_t launch_e(const AttnArgs &a, size_t ws_bytes, cudaStream_t stream) {
  return a.D <= 64 ? launch_t<E, 64>(a, ws_bytes, stream) : launch_t<E, 128>(a, ws_bytes, stream);
}

}  // namespace
}  // namespace paged

cudaError_t launch_attention_prefill(const paged::AttnArgs &a, int type, size_t ws_bytes, cudaStream_t stream) {
  return type == kTypeF16 ? paged::launch_e<ElemF16>(a, ws_bytes, stream)
                          : paged::launch_e<ElemBF16>(a, ws_bytes, stream);
}

}  // namespace qmm
