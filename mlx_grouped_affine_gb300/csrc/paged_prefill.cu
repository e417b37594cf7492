// Paged attention for many query rows per kv head (prompts, chunks of prompts)
// on the sm_103a tensor cores.
//
// Per key tile of 128 keys, 256 query rows and heads of D: 4 * 128 * 256 * D
// flops and 128 * 256 exponentials, against 512 D bytes of K and V: the tensor
// pipe bounds it (2048 cycles a tile at D = 128; the exponentials take 1024 of
// the special-function units' cycles).  One persistent block per SM; its item is
// two halves of 128 rows (rows are (token, head of the group) pairs, so every
// row of an item shares its K and V).  For each half h and key tile j
//   S_h = Q_h K_j^T     tcgen05.mma, 128 x 128 fp32 in TMEM
//   P_h = 2^(S_h - m)   16-bit P over S_h in TMEM
//   O_h += P_h V_j      tcgen05.mma with P from TMEM, 128 x D fp32 in TMEM
// S_h, P_h and O_h of a half follow one another, so the halves take turns:
// while one is in its softmax the other has the tensor pipe.  One warp issues
// for both, in turns, which keeps them out of step (with an issuer each they
// fell into step: both softmaxes, then both products, 5400 cycles a tile).  A
// half's softmax has two threads a row, 64 columns each: with one thread a row
// its latency (1600 cycles) stood above what the other half's products hide.
// Roles:
//   warps 0-7, 8-15  softmax and output of half 0, 1: warp w has TMEM lanes
//                    32 (w % 4) on and columns 64 (w / 4 % 2) on of S
//   warp 16          issues the MMAs (one lane); owns the TMEM allocation
//   warp 17          Q and K by TMA, K a box of a page's rows at a time
//   warps 18, 19     V by cp.async
// K and V share a ring of tiles.  Each way of loading alone is too slow beside
// the tensor cores' own reads of shared memory: TMA boxes of 16 rows move 20
// bytes a cycle (3300 cycles for the 64 KB of a tile), and cp.async from three
// warps, 50 bytes a cycle on an idle SM, 15 here.  V goes the way that can write
// zeros for single rows (below); a stale row of K only makes scores that are
// masked.
// The running maximum moves lazily: P is relative to a row maximum m that is
// only raised, and O and the row sum rescaled, when a score exceeds it by more
// than 2^8 (P stays below 256; the result is the same because O and the sum share
// m).  For fp16 m is raised to 2^7 below the maximum, so that P reaches 2^15, half of
// the type's range, and keeps all bits down to 2^-21 of the row's largest weight.  The
// products in P's exponents are exact and m is rounded, 2^-24 of it: in fp16 with scores
// of 2^20 and more m is the maximum itself, so that P is 2^that at most.
//
// Measured (32 heads over 8 of 128, bf16): 512 tokens over 32000 keys 220 us,
// 1.23 PFLOP/s, 0.64 of the measured bf16 rate (as called 228 us, 0.62); causal prompts
// of 2000 to 8192 tokens 615 to 628 us, 0.63 to 0.65 (622 to 646, 0.61 to 0.64).  The
// tensor pipe is busy 61 % of the time: its products read 192 KB of shared memory a
// tile, 64 KB more are written by the loads, and 256 KB at 128 bytes a cycle take the
// 2048 cycles that the products alone would.  Beside that the chunk reads K and V from
// HBM 7.5 times (its items are at different keys at one time): 4.8 TB/s, 0.71 of the
// copy rate.  Heads of 72 to 120 are padded to 128 in products and loads and take the
// time of 128 (prompts with heads of 80 and 96: 607 and 608 us).
//
// Waits are bounded; one that runs out sets the error word and an abort flag
// that stops every role, and the block still drains its copies and MMAs.  The
// two warps of a row meet at a hardware barrier every tile, which is not
// bounded: a warp that gave up goes on to meet its partner, tile by tile, and
// does nothing else.
//
// Shared tiles are 64-column chunks of 128-byte rows, 128-byte swizzled; K and
// Q chunks are K-major operands (8-row groups 1024 bytes apart), V chunks
// MN-major ones (atoms of 64 columns x 8 keys).
//
// Rows of a tile that hold no key of the item are written as zeros: P is zero
// there, but zero times a stale infinity of the last page is not nothing.
#include "paged.cuh"

namespace qmm {
namespace paged {
namespace {

constexpr int R = 256, KT = 128, kSoftmaxWarps = 16, kValueWarps = 2;
constexpr int NT = 32 * (kSoftmaxWarps + 2 + kValueWarps);
constexpr uint32_t kDrainPolls = 1u << 14;  // for copies under way after a wait ran out: milliseconds
constexpr int KC = KT / 2;    // columns of S a softmax thread has
// log2 by which scores exceed the row's reference when it is set, and beyond that
// before it is set again; in fp16 both nothing for scores from kHuge on.
template <typename E>
constexpr float kRaise = E::kF16 ? 7.f : 0.f;
constexpr float kLazy = 8.f, kHuge = 0x1p20f;

template <int DP>
struct Tile {
  static constexpr uint32_t CHUNK = 128 * 128;          // 128 rows of 64 columns
  static constexpr uint32_t TILE = CHUNK * (DP / 64);   // Q half, K or V tile
  static constexpr int SLOTS = DP == 128 ? 5 : 8;
  static_assert(SLOTS + 1 <= 16, "a step's barrier is free when its turn comes again");
  static constexpr uint32_t O0 = 256;                   // TMEM: S_0 at 0, S_1 at 128, O_0, O_1
};

// Barriers of the loads of a step.  A step has one load at least, so no more
// steps are under way than the ring has slots, and one.
constexpr int kSteps = 16;

struct Barriers {
  uint64_t q_full, q_empty, kv_full[kSteps], kv_empty[8], s_full[2], p_ready[2], o_full[2], o_empty[2], mma_done;
  uint32_t tmem_base;
  int abort, redo;
  Cursor start;                           // the block's
  Cursor cursor[kSoftmaxWarps / 2];       // of a pair of softmax warps
  float exchange[kSoftmaxWarps][32];      // between its two warps
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
// offsets in units of 16, version 1, swizzle mode 2): its low word holds the
// start and the leading offset, its high word is the same for all.  K-major:
// 8-row groups 1024 bytes apart.  MN-major: atoms 16384 bytes apart along N (a
// 64-column chunk of 128 keys), 1024 along K.
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t lead) {
  return (saddr >> 4) | (lead >> 4) << 16;
}
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;

// One lane of the warp, the same at every call; the warp is converged.
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
  return yes != 0;
}

// kind::f16, fp32 accumulator, M = 128; B transposed (MN-major) for V.
template <typename E, int N, bool BMN>
__host__ __device__ constexpr uint32_t idesc() {
  return (1u << 4) | (E::kF16 ? 0u : (1u << 7) | (1u << 10)) | (BMN ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}

template <uint32_t IDESC>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\t"
      "mov.b64 b, {%2, %5};\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "n"(IDESC), "r"(acc), "n"(kDescHigh)
      : "memory");
}
template <uint32_t IDESC>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "n"(IDESC), "r"(acc), "n"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
      : "memory");
}


// 32 columns of this warp's 32 TMEM lanes into f[O], ..; no wait.
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
// Two fp32 operations an instruction: (x0, x1) * k + c, and (s0, s1) += (x0, x1).
__device__ __forceinline__ void fma2(float x0, float x1, float k, float c, float &y0, float &y1) {
  asm("{\n\t.reg .b64 x, k, c, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 k, {%4, %4};\n\tmov.b64 c, {%5, %5};\n\t"
      "fma.rn.f32x2 y, x, k, c;\n\tmov.b64 {%0, %1}, y;\n\t}"
      : "=f"(y0), "=f"(y1)
      : "f"(x0), "f"(x1), "f"(k), "f"(c));
}
__device__ __forceinline__ void add2(float &s0, float &s1, float x0, float x1) {
  asm("{\n\t.reg .b64 s, x;\n\tmov.b64 s, {%0, %1};\n\tmov.b64 x, {%2, %3};\n\tadd.rn.f32x2 s, s, x;\n\t"
      "mov.b64 {%0, %1}, s;\n\t}"
      : "+f"(s0), "+f"(s1)
      : "f"(x0), "f"(x1));
}

// The two warps of a row meet (64 threads at hardware barrier `id`); whether
// any of their threads said yes.
__device__ __forceinline__ bool meet_any(int id, bool yes) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.aligned.pred q, %2, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(static_cast<uint32_t>(yes)), "r"(id)
      : "memory");
  return any != 0;
}
__device__ __forceinline__ void meet(int id) {
  asm volatile("barrier.cta.sync.aligned %0, 64;" ::"r"(id) : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t addr, float (&o)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(o[0]), "=f"(o[1]), "=f"(o[2]), "=f"(o[3]), "=f"(o[4]), "=f"(o[5]), "=f"(o[6]), "=f"(o[7]),
        "=f"(o[8]), "=f"(o[9]), "=f"(o[10]), "=f"(o[11]), "=f"(o[12]), "=f"(o[13]), "=f"(o[14]), "=f"(o[15])
      : "r"(addr));
}
// 16 columns times f, in place.
__device__ __forceinline__ void tmem_scale16(uint32_t addr, float f) {
  float o[16];
  tmem_ld16(addr, o);
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

// 32 bytes to global memory, 32-byte aligned.
__device__ __forceinline__ void store32(void *p, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e,
                                        uint32_t f, uint32_t g, uint32_t h) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a), "r"(b), "r"(c), "r"(d),
               "r"(e), "r"(f), "r"(g), "r"(h)
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

// A box of the queries' tensor map (columns, heads, tokens, one).  What lies
// outside reads as zeros; the first coordinate is a multiple of 64.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w,
                                        uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// This thread's arrival at the barrier once all its copies so far have landed.
__device__ __forceinline__ void arrive_landed(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Step j of a piece needs V of tile j - 1 and K of tile j (the first only K, the
// last only V).  The ring's slots take K and V of a tile in turn: tile j of a
// piece that begins with load n has K in load n + 2 (j - from), V in the next.  A
// step's barrier counts an arrival of every thread of the K warp and of the V
// warps, made when the thread's copies have landed, so that no load waits for
// another.  (The issuer of the MMAs fences the copies that are generic writes
// for the tensor cores.)
template <int DP>
__device__ __forceinline__ bool slot_free(const AttnArgs &a, uint32_t n, Barriers *bars) {
  using X = Tile<DP>;
  return wait_warp(&bars->kv_empty[n % X::SLOTS], (n / X::SLOTS & 1) ^ 1u, &bars->abort, a.err, a.spin_limit);
}

// `box` rows of a TMA box of K; 0: K by cp.async too (pages not of 8 rows).
template <int DP>
__device__ void key_role(const AttnArgs &a, Cursor c, const CUtensorMap *qmap, const CUtensorMap *kmap, int box,
                         uint8_t *sq, uint8_t *skv, Barriers *bars) {
  using X = Tile<DP>;
  const int lane = threadIdx.x & 31;
  const Copier<DP> copier(a.D, X::CHUNK);
  uint32_t load = 0, steps = 0, q_count = 0;
  bool ok = true;
  while (ok && c.left > 0) {
    const Piece p = piece_of(a, c);
    if (p.any.from < p.any.to) {
      const int kv = c.h / a.S;
      // Lane l looks up box (block) l of the next tile.
      const int rows = box ? box : 8;
      Block next;
      auto look = [&](int tile) {
        next = Block{0, 0, 0};
        if (rows * lane >= KT || tile >= p.any.to) return;
        const int key = tile * KT + rows * lane;
        if (!box) {
          next = look_up(a, c.b, key, c.lo, c.hi);
        } else if (c.lo - key < rows && key < c.hi) {
          const int pg = key / a.page;
          next = Block{1, __ldg(a.table + c.b * a.table_stride + pg), key - pg * a.page};
        }
      };
      look(p.any.from);
      // Q of both halves, once the previous one has been multiplied.
      ok = wait_warp(&bars->q_empty, (q_count & 1) ^ 1u, &bars->abort, a.err, a.spin_limit);
      if (!ok) break;
      if (lane == 0) {
        mbar_expect_tx(&bars->q_full, 2 * (DP / 64) * a.Gs * a.TH * 128);
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
      for (int j = p.any.from; ok && j < p.any.to; ++j, ++steps) {
        uint64_t *bar = &bars->kv_full[steps % kSteps];
        const Block mine = next;
        look(j + 1);
        ok = slot_free<DP>(a, load, bars);
        if (!ok) break;
        const uint32_t dst = smem_u32(skv + load % X::SLOTS * X::TILE);
        if (box) {
          // A page past the pool's end, and boxes without a key, read as zeros.
          const bool known = static_cast<unsigned>(mine.id) < static_cast<unsigned>(a.num_pages);
          if (mine.how && !known) atomicOr(a.err, kErrIndexBit);
          if (lane == 0) mbar_expect_tx(bar, X::TILE);
          __syncwarp();
          if (lane * box < KT) {
#pragma unroll
            for (int x = 0; x < DP / 64; ++x)
              tma_box(dst + x * X::CHUNK + lane * box * 128, kmap, 64 * x, mine.row, kv,
                      mine.how && known ? mine.id : a.num_pages, bar);
          }
          if (lane != 0) mbar_arrive(bar);
        } else {
          const int64_t off = block_offset(a, mine, kv);
#pragma unroll 1
          for (int x = 0; x < KT / 8; ++x)
            copier.copy(a, a.k, __shfl_sync(0xffffffffu, off, x), dst + 1024 * x, c.b, kv, j * KT + 8 * x, c.lo, c.hi);
          arrive_landed(bar);
        }
        load += 2;
      }
      if (ok) mbar_arrive(&bars->kv_full[steps++ % kSteps]);  // no K in the last step
    }
    if (ok) piece_done(a, c, p);
  }
  // No copy outlives the warp's part, whichever role stopped early: where every load fits the
  // ring, this one's only waits are met.  Stopped early, the barriers of the steps under way may
  // lack other warps' arrivals: the waits are short.
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (q_count) {
    for (uint32_t x = 0; x < kDrainPolls; ++x)
      if (__all_sync(0xffffffffu, mbar_try_wait(&bars->q_full, (q_count - 1) & 1))) break;
  }
  for (uint32_t n = steps > X::SLOTS ? steps - X::SLOTS : 0; n < steps; ++n) {
    for (uint32_t x = 0; x < kDrainPolls; ++x)
      if (__all_sync(0xffffffffu, mbar_try_wait(&bars->kv_full[n % kSteps], (n / kSteps) & 1))) break;
  }
}

// V: warp w has blocks w, w + 2, .. of a tile's 16 and looks them up a tile ahead.
template <int DP>
__device__ void value_role(const AttnArgs &a, Cursor c, int w, uint8_t *skv, Barriers *bars) {
  using X = Tile<DP>;
  const int lane = threadIdx.x & 31;
  const Copier<DP> copier(a.D, X::CHUNK);
  uint32_t load = 1, steps = 0;
  bool ok = true;
  while (ok && c.left > 0) {
    const Piece p = piece_of(a, c);
    if (p.any.from < p.any.to) {
      const int kv = c.h / a.S;
      Block next;
      auto look = [&](int tile) {
        next = Block{0, 0, 0};
        if (lane < KT / 8 && tile < p.any.to) next = look_up(a, c.b, tile * KT + 8 * lane, c.lo, c.hi);
      };
      look(p.any.from);
      mbar_arrive(&bars->kv_full[steps++ % kSteps]);  // no V in the first step
      for (int j = p.any.from; ok && j < p.any.to; ++j, ++steps) {
        uint64_t *bar = &bars->kv_full[steps % kSteps];
        const int64_t off = block_offset(a, next, kv);
        look(j + 1);
        ok = slot_free<DP>(a, load, bars);
        if (!ok) break;
        const uint32_t dst = smem_u32(skv + load % X::SLOTS * X::TILE);
#pragma unroll 2
        for (int x = w; x < KT / 8; x += kValueWarps)
          copier.copy(a, a.v, __shfl_sync(0xffffffffu, off, x), dst + 1024 * x, c.b, kv, j * KT + 8 * x, c.lo, c.hi);
        arrive_landed(bar);
        load += 2;
      }
    }
    if (ok) piece_done(a, c, p);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");  // no copy outlives the warp's part
}

// By one thread: a vote of the warp after every wait would cost as much again.
template <typename E, int DP>
__device__ void mma_role(const AttnArgs &a, Cursor c, uint8_t *sq, uint8_t *skv, Barriers *bars, uint32_t tmem) {
  using X = Tile<DP>;
  volatile int *abort = &bars->abort;
  uint32_t steps = 0, q_count = 0, slot = 0;  // as the loads count them
  uint32_t p_count[2] = {0, 0}, o_count[2] = {0, 0};
  const uint32_t q = desc_low(smem_u32(sq), 16);
  const uint32_t ring_k = desc_low(smem_u32(skv), 16), ring_v = desc_low(smem_u32(skv), X::CHUNK);
  bool ok = true;
  while (ok && c.left > 0) {
    const Piece p = piece_of(a, c);
    if (p.any.from < p.any.to) {
      ok = wait_warp(&bars->q_full, q_count & 1, abort, a.err, a.spin_limit);
      ++q_count;
      for (int j = p.any.from; ok && j <= p.any.to; ++j, ++steps) {
        ok = wait_warp(&bars->kv_full[steps % kSteps], (steps / kSteps) & 1, abort, a.err, a.spin_limit);
        if (!ok) break;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        const bool has_v = j > p.any.from, has_k = j < p.any.to;
        const uint32_t vs = slot, ks = has_v ? (slot + 1 == X::SLOTS ? 0 : slot + 1) : slot;
        slot = has_k ? (ks + 1 == X::SLOTS ? 0 : ks + 1) : ks;
        const uint32_t v = ring_v + vs * (X::TILE >> 4), k = ring_k + ks * (X::TILE >> 4);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool pv = j > p.half[h].from && j <= p.half[h].to, qk = j >= p.half[h].from && j < p.half[h].to;
          const bool first = j - 1 == p.half[h].from;
          if (pv) {
            // The previous piece's output has left O_h; P_h is there.
            if (first && !(ok = wait_warp(&bars->o_empty[h], (o_count[h]++ & 1) ^ 1u, abort, a.err, a.spin_limit)))
              break;
            if (!(ok = wait_warp(&bars->p_ready[h], p_count[h]++ & 1, abort, a.err, a.spin_limit))) break;
            tc_fence_after();
          }
          if (elect_one()) {
            if (pv) {
#pragma unroll
              for (int x = 0; x < KT / 16; ++x)
                mma_ts<idesc<E, DP, true>()>(tmem + X::O0 + h * DP, tmem + 128 * h + KC * (x >> 2) + 8 * (x & 3),
                                             v + 128 * x, !first || x);
              if (j == p.half[h].to) mma_commit(&bars->o_full[h]);
            }
            if (h == 1 && has_v) mma_commit(&bars->kv_empty[vs]);
            if (qk) {
#pragma unroll
              for (int x = 0; x < DP / 16; ++x) {
                const uint32_t at = (x >> 2) * (X::CHUNK >> 4) + (x & 3) * 2;
                mma_ss<idesc<E, KT, false>()>(tmem + 128 * h, q + h * (X::TILE >> 4) + at, k + at, x != 0);
              }
              mma_commit(&bars->s_full[h]);
            }
            if (h == 1) {
              if (has_k) mma_commit(&bars->kv_empty[ks]);
              if (j == p.any.to - 1) mma_commit(&bars->q_empty);
            }
          }
          __syncwarp();
        }
      }
    }
    if (ok) piece_done(a, c, p);
  }
  // Every MMA retires before the block frees its TMEM.
  if (elect_one()) mma_commit(&bars->mma_done);
  __syncwarp();
  for (uint32_t x = 0; x < kDefaultWaitLimit; ++x)
    if (__all_sync(0xffffffffu, mbar_try_wait(&bars->mma_done, 0))) break;
}

// Columns of a row that it does not see become -infinity: the row sees keys
// [span.lo, span.hi), and its 32 columns are keys key0 on.
__device__ __forceinline__ void hide(float (&s)[32], const Span &span, int key0) {
  const int lo = max(span.lo - key0, 0), hi = min(span.hi - key0, 32);
  const uint32_t seen = lo >= hi ? 0u : (hi == 32 ? 0xFFFFFFFFu : (1u << hi) - 1u) & ~((1u << lo) - 1u);
#pragma unroll
  for (int x = 0; x < 32; ++x)
    if (!(seen >> x & 1u)) s[x] = kNegInf;
}

__device__ __forceinline__ float chunk_top(const float (&s)[32]) {
  float t[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
  for (int x = 4; x < 32; x += 8)
#pragma unroll
    for (int y = 0; y < 4; ++y) t[y] = fmaxf(t[y], x + 4 < 32 ? fmaxf(s[x + y], s[x + 4 + y]) : s[x + y]);
  return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
}

// Weights 2^(s * scale + base) of 32 columns, rounded once to the element type
// for the product with V, into 16 columns of TMEM, and their sums before that.
template <typename E>
__device__ __forceinline__ void weights(const float (&s)[32], float scale, float base, float (&sums)[2],
                                        uint32_t addr) {
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    uint32_t pk[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      float e0, e1;
      fma2(s[16 * y + 2 * x], s[16 * y + 2 * x + 1], scale, base, e0, e1);
      e0 = exp2_fast(e0);
      e1 = exp2_fast(e1);
      add2(sums[0], sums[1], e0, e1);
      pk[x] = E::pack2(e0, e1);
    }
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(pk[0]), "r"(pk[1]),
                 "r"(pk[2]), "r"(pk[3]), "r"(pk[4]), "r"(pk[5]), "r"(pk[6]), "r"(pk[7]), "r"(addr + 8 * y)
                 : "memory");
  }
}

// The rows that the block wrote whole, once more where one is not finite.  Called
// after everything else, when some thread saw such a value in a row whose sum is
// finite, so that the tile loop makes no calls.
template <typename E>
__device__ __noinline__ void redo_rows(const AttnArgs &a, Cursor c) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  while (c.left > 0) {
    const Piece p = piece_of(a, c);
    for (int row = warp; p.whole && row < R; row += NT / 32) {
      int i, head;
      if (!row_of(a, c.r, c.h, c.qt, row, &i, &head)) continue;
      const uint16_t *out = static_cast<const uint16_t *>(a.out) +
                            (static_cast<int64_t>(c.r.first) + i) * a.out_stride + static_cast<int64_t>(head) * a.D;
      bool bad = false;
      for (int d = lane; d < a.D; d += 32) bad |= !isfinite(E::to_f32(out[d]));
      if (__any_sync(0xffffffffu, bad)) row_alone<E>(a, c.b, head, i, 0, a.D);
    }
    piece_done(a, c, p);
  }
}

template <typename E, int DP>
__device__ void softmax_role(const AttnArgs &a, Barriers *bars, uint32_t tmem) {
  using X = Tile<DP>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = warp >> 3, part = warp >> 2 & 1;
  const int pair = warp >> 3 << 2 | (warp & 3), meeting = 1 + pair;
  const int row = 128 * h + 32 * (warp & 3) + lane;  // of the item; its TMEM lane in the half
  const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
  const uint32_t ts = tmem + 128 * h + KC * part + lanes;            // its columns of S; P in the first half
  const uint32_t to = tmem + X::O0 + h * DP + DP / 2 * part + lanes;  // of O
  volatile int *abort = &bars->abort;
  // The cursor stays in shared memory between pieces, out of the registers.
  Cursor *cursor = &bars->cursor[pair];
  uint32_t s_count = 0, o_count = 0;
  bool continues = cursor->at != 0, dead = false;
  while (cursor->left > 0) {
    int from, to_tile;
    Span span{0, 0};
    int deep_lo = 0, deep_hi = 0x7FFFFFFF;  // keys that every live row of the warp sees
    {
      const Cursor c = *cursor;
      const Piece p = piece_of(a, c);
      int i, head;
      if (row_of(a, c.r, c.h, c.qt, row, &i, &head)) {
        span = span_of(a, c.r, i);
        deep_lo = span.lo;
        deep_hi = span.hi;
      }
      from = h ? p.half[1].from : p.half[0].from;
      to_tile = h ? p.half[1].to : p.half[0].to;
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) {
      deep_lo = max(deep_lo, __shfl_xor_sync(0xffffffffu, deep_lo, x));
      deep_hi = min(deep_hi, __shfl_xor_sync(0xffffffffu, deep_hi, x));
    }
    float m = kNegInf, l = 0.f;
    for (int j = from; j < to_tile; ++j) {
      dead = dead || !wait_warp(&bars->s_full[h], s_count & 1, abort, a.err, a.spin_limit);
      ++s_count;
      const bool deep = j * KT >= deep_lo && deep_hi - j * KT >= KT;
      float s[32], top = kNegInf;
      if (!dead) {
        tc_fence_after();
        tmem_ld32<0>(ts + 32, s);
        tmem_wait_ld();
        if (!deep) hide(s, span, j * KT + KC * part + 32);
        top = chunk_top(s);
        tmem_ld32<0>(ts, s);
        tmem_wait_ld();
        if (!deep) hide(s, span, j * KT + KC * part);
        top = fmaxf(top, chunk_top(s)) * a.scale_log2;
      }
      // Raise the reference when a score is far above it (and in the first tile).
      if (meet_any(meeting, !dead && top > m + (!E::kF16 || fabsf(top) < kHuge ? kRaise<E> + kLazy : 0.f))) {
        bars->exchange[warp][lane] = top;
        meet(meeting);
        const float most = fmaxf(top, bars->exchange[warp ^ 4][lane]);
        const float up = fmaxf(m, E::kF16 && fabsf(most) < kHuge ? most - kRaise<E> : most);
        const float f = exp2_fast(m - (up == kNegInf ? 0.f : up));
        m = up;
        l *= f;
        if (j > from && !dead) {
          // O_h is complete up to the previous tile: S_h was committed after it.
#pragma unroll 1
          for (int x = 0; x < DP / 32; ++x) tmem_scale16(to + 16 * x, f);
        }
      }
      if (dead) continue;
      const float base = m == kNegInf ? 0.f : -m;
      float sums[2] = {0.f, 0.f};
      weights<E>(s, a.scale_log2, base, sums, ts);
      tmem_ld32<0>(ts + 32, s);
      tmem_wait_ld();
      if (!deep) hide(s, span, j * KT + KC * part + 32);
      weights<E>(s, a.scale_log2, base, sums, ts + 16);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->p_ready[h]);
      l += sums[0] + sums[1];
    }

    if (from < to_tile) {
      dead = dead || !wait_warp(&bars->o_full[h], o_count & 1, abort, a.err, a.spin_limit);
      ++o_count;
      bars->exchange[warp][lane] = l;
      meet(meeting);
      l += bars->exchange[warp ^ 4][lane];
    }
    if (!dead) {
      // The row's part: to the output, or to the workspace when the item is cut.
      const Cursor c = *cursor;
      const bool any = from < to_tile, whole = c.at == 0 && c.left >= c.tiles;
      int i, head;
      const bool live = row_of(a, c.r, c.h, c.qt, row, &i, &head);
      const float inv = !any ? 0.f : !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
      const int64_t token = static_cast<int64_t>(c.r.first) + i;
      float *piece = slot_of<R, DP>(a, blockIdx.x, !continues);
      if (part == 0) {
        if (!whole) {
          piece[R * DP + row] = m;
          piece[R * DP + R + row] = l;
        } else if (live && a.lse) {
          a.lse[token * a.Hq + head] = (m + log2f(l)) * kLn2;
        }
      }
      piece += row * DP + DP / 2 * part;
      uint16_t *out = static_cast<uint16_t *>(a.out) + token * a.out_stride + static_cast<int64_t>(head) * a.D +
                      DP / 2 * part;
      const int cols = a.D - DP / 2 * part;  // of the head from this part on
      // A row's stores are whole 32-byte sectors where rows and heads allow it: a
      // warp's store touches 32 rows, and each is a trip of its own.
      const bool wide = ((reinterpret_cast<uintptr_t>(a.out) | a.out_stride * 2 | a.D * 2) & 31) == 0;
      bool bad = false;
      tc_fence_after();
#pragma unroll 1
      for (int x = 0; x < DP / 2; x += 16) {
        float o[16];
        tmem_ld16(to + x, o);
        tmem_wait_ld();
#pragma unroll
        for (int y = 0; y < 16; ++y) {
          o[y] = any ? o[y] * inv : 0.f;  // without a tile O_h holds whatever was there
          bad |= !isfinite(o[y]);
        }
        if (!whole) {
#pragma unroll
          for (int y = 0; y < 16; y += 8)
            store32(piece + x + y, __float_as_uint(o[y]), __float_as_uint(o[y + 1]), __float_as_uint(o[y + 2]),
                    __float_as_uint(o[y + 3]), __float_as_uint(o[y + 4]), __float_as_uint(o[y + 5]),
                    __float_as_uint(o[y + 6]), __float_as_uint(o[y + 7]));
        } else if (live) {
          uint32_t u[8];
#pragma unroll
          for (int y = 0; y < 8; ++y) u[y] = E::pack2(o[2 * y], o[2 * y + 1]);
          if (wide) {
            if (x < cols) store32(out + x, u[0], u[1], u[2], u[3], u[4], u[5], u[6], u[7]);
          } else {
            if (x < cols) *reinterpret_cast<uint4 *>(out + x) = make_uint4(u[0], u[1], u[2], u[3]);
            if (x + 8 < cols) *reinterpret_cast<uint4 *>(out + x + 8) = make_uint4(u[4], u[5], u[6], u[7]);
          }
        }
      }
      if (any) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->o_empty[h]);
      }
      if (bad && live && whole && isfinite(l)) bars->redo = 1;
    }
    continues = false;
    // Both warps have read the cursor; one moves it on.
    meet(meeting);
    if (part == 0) {
      Cursor c = *cursor;
      __syncwarp();
      piece_done(a, c, piece_of(a, c));
      if (lane == 0) *cursor = c;
    }
    meet(meeting);
  }
}

template <typename E, int DP>
__global__ void __launch_bounds__(NT, 1)
prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
               const __grid_constant__ AttnArgs a, int box) {
  using X = Tile<DP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sq = smem, *skv = smem + 2 * X::TILE;
  Barriers *bars = reinterpret_cast<Barriers *>(skv + X::SLOTS * X::TILE);
  const int warp = threadIdx.x >> 5;
  static_assert(sizeof(PlanScratch<NT>) <= X::TILE, "the plan's scratch lies in the ring");
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&qmap) : "memory");
    if (box) asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 1);
    for (int i = 0; i < kSteps; ++i) mbar_init(&bars->kv_full[i], 32 * (1 + kValueWarps));
    for (int i = 0; i < X::SLOTS; ++i) mbar_init(&bars->kv_empty[i], 1);
    for (int h = 0; h < 2; ++h) {
      mbar_init(&bars->s_full[h], 1);
      mbar_init(&bars->p_ready[h], 8);
      mbar_init(&bars->o_full[h], 1);
      mbar_init(&bars->o_empty[h], 8);
    }
    mbar_init(&bars->mma_done, 1);
    bars->abort = bars->redo = 0;
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
  if (warp == kSoftmaxWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&bars->tmem_base)),
                 "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (threadIdx.x == 0) bars->start = c;
  if (warp < kSoftmaxWarps && (threadIdx.x & 31) == 0 && !(warp & 4)) bars->cursor[warp >> 3 << 2 | (warp & 3)] = c;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp < kSoftmaxWarps) softmax_role<E, DP>(a, bars, tmem);
  else if (warp == kSoftmaxWarps) mma_role<E, DP>(a, c, sq, skv, bars, tmem);
  else if (warp == kSoftmaxWarps + 1) key_role<DP>(a, c, &qmap, &kmap, box, sq, skv, bars);
  else value_role<DP>(a, c, warp - kSoftmaxWarps - 2, skv, bars);

  tc_fence_before();
  __syncthreads();
  if (warp == kSoftmaxWarps) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
  }
  if (bars->redo && !bars->abort) redo_rows<E>(a, bars->start);
}

template <typename E, int DP>
cudaError_t launch_t(AttnArgs a, size_t ws_bytes, cudaStream_t stream) {
  a.S = (a.G + 127) / 128;
  a.Gs = (a.G + a.S - 1) / a.S;
  a.heads = a.Hkv * a.S;
  a.TH = 128 / a.Gs;
  a.TQ = 2 * a.TH;
  // An item's first products and its output, in key tiles.  Measured at 0 / 3 / 6:
  // three causal prompts of 2000 to 8192 tokens 690 / 618 / 626 and 699 / 628 / 625 us.
  a.item_cost = 3;
  // Rows of a TMA box of K: the largest power of two that divides the page.
  int box = 0;
  if (a.page % 8 == 0)
    for (box = 8; box < KT && a.page % (2 * box) == 0;) box *= 2;
  const int type = E::kF16 ? kTypeF16 : kTypeBF16;
  CUtensorMap q, k;
  cudaError_t e = query_map(a, type, &q);
  if (e == cudaSuccess) e = box ? key_map(a, type, box, &k) : (k = q, cudaSuccess);
  if (e != cudaSuccess) return e;
  constexpr size_t smem = smem_bytes<DP>();
  e = ensure_smem_limit<prefill_kernel<E, DP>>(smem);
  if (e != cudaSuccess) return e;
  int blocks = sm_count();
  const size_t per_block = 2 * sizeof(float) * R * (DP + 2);
  blocks = static_cast<int>(std::min<size_t>(std::min(blocks, kMaxBlocks), ws_bytes / per_block));
  prefill_kernel<E, DP><<<blocks, NT, smem, stream>>>(q, k, a, box);
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
