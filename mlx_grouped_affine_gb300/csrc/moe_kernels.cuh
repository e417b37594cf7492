// Kernels of qmm_moe_experts and qmm_moe_layer, instantiated per code width by
// moe_bits_*.cu.
//
// With w = s c + b per group of G codes, a row's product with x over one group is
// s * sum(c x) + b * sum(x).  Codes are exact in bf16, so sum(c x) and sum(x) run on the
// tensor cores (mma.sync m16n8k16, fp32 sums) and s and b are applied to them in fp32: no
// weight is ever rounded, and s and b cost two multiply-adds per group and output instead
// of one per code.  x goes in as bf16: as it stands where it is bf16, else as a sum of two
// (fp16) or three (fp32) bf16 planes that hold it exactly, one product each.
//
// The weights that the routing asks for are streamed once; everything else (x, h, scales'
// sectors) stays in L1 or L2.  Bound by instructions and their latency: 211 per 64 columns of
// 32 rows (72 spread 4-bit codes and scale them, 12 are products, 16 apply scales), at half of the
// issue slots with the 16 warps an SM that registers allow.  16 tokens of 8 of 64 experts, 2048 x
// 1024 at 4 bits, 84.2 us (gate and up 46, down 43), 0.35 of HBM; 16 tokens of 2 of 8, 4096 x
// 14336, 269 us, 0.43.  A warp works on its own: 32 weight rows (two 16-row tiles of
// the MMA, sharing the x operand) and a range of chunks of 128 or 256 columns.  A chunk's
// codes come by TMA, a box of 16 rows per tile, into a ring of the warp's own, so that loads
// in flight cost no registers and need no block barrier.  (Copies by the lanes themselves
// touch eight rows an instruction and were held up at one cache line a cycle: 2500 cycles
// for 2048 codes a warp.)  8 slots fill the MMA's columns, and so many of an expert are taken
// per pass over its weights.  (16 a pass halve the passes of experts with more than 8 slots, but
// their registers cost all others: 48 tokens of 4 of 32 experts in fp32 76 us against 56.)
#pragma once
#include "common.cuh"

namespace qmm {

constexpr int kMoeThreads = 256, kMoeWarps = kMoeThreads / 32;
constexpr int kMoePass = 8;       // slots of an expert per pass over its weights
constexpr int kMoeMaxCluster = 8;

struct MoePlan;

// What the kernels share of a call.
struct MoeArgs {
  Routing route;
  ExpertWeights w;
  const uint16_t *x;    // bf16 planes [planes][tokens][hidden]
  int64_t x_plane;      // elements between planes of x
  int x_planes;
  uint16_t *h;          // silu(gate) * up: bf16 planes [h_planes][slots][inner]
  int64_t h_plane;
  int h_planes;
  int tokens;
  void *y;
  int y_type;
  const MoePlan *plan;
  unsigned *err;
  uint32_t wait_limit;
  uint32_t code_scale;  // kCodeScale
};

// ------------------------------------------------------------- the plan ----
// Which slots (token * top_k + place) go to which expert (moe_experts.cu works it out).  A
// unit is an expert with up to kMoePass of its slots; an expert's units follow one another,
// its slots are in order, and experts come in the order of their first slots.
// Three tables side by side, an entry of each per slot: units, slots unit by unit, slots.
struct alignas(16) MoeEntry {
  short unit_expert, unit_first, unit_count;  // of unit i; first in the second table
  short listed, token;                        // the slot at place i, and its token
  short slot_unit;                            // of slot i: unit * kMoePass + place in it; -1: no part in y
  float slot_weight;
};
struct MoePlan {
  alignas(16) int units;
  MoeEntry entries[kMoeMaxSlots];
};

// The block's copy.  (From L2: a kernel launched early must not trust its L1.)
__device__ __forceinline__ int read_plan(const MoePlan *from, MoeEntry *to, int slots) {
  for (int i = threadIdx.x; i < slots; i += kMoeThreads)
    reinterpret_cast<uint4 *>(to)[i] = __ldcg(reinterpret_cast<const uint4 *>(&from->entries[i]));
  const int units = __ldcg(&from->units);
  __syncthreads();
  return units;
}

// ------------------------------------------------------------ the codes ----

// A lane's part of a group: the G / 4 codes [t G / 4, (t + 1) G / 4) for lane 4 g + t, so
// that the four lanes of an MMA row are in one group.
template <int BITS, int G>
struct Run {
  static constexpr int kCodes = G / 4;
  static constexpr int kBits = kCodes * BITS;
  static constexpr bool kWhole = kBits % 32 == 0;  // whole words, else shifted into place
  static constexpr int words() {
    int n = 0;
    for (int t = 0; t < 4; ++t) {
      const int w = (t * kBits % 32 + kBits + 31) / 32;
      n = w > n ? w : n;
    }
    return n;
  }
  static constexpr int kWords = words();
  // Words read at once: as many as the run's alignment (its own size) allows.
  static constexpr int kPiece = !kWhole ? 1 : kWords % 4 == 0 ? 4 : kWords % 2 == 0 ? 2 : 1;
  // Codes j and j + half of a word share a register (one mask for both) where a word holds
  // whole codes; otherwise neighbours do.
  static constexpr bool kSplit = kWhole && (BITS == 2 || BITS == 4 || BITS == 8);
  static constexpr int kSub = kCodes < 16 ? kCodes : 16;  // codes spread at a time
  // A chunk: what a warp's ring holds per stage of each row, at most 128 bytes.
  static constexpr int kChunk = BITS <= 4 ? 256 : 128;
  static constexpr int kSteps = kChunk / G;
  static constexpr int kRowBytes = kChunk * BITS / 8;
  static constexpr int kStageBytes = 2 * 16 * kRowBytes;
  static constexpr int kDepth = kStageBytes > 2560 ? 2 : 4;
  // A warp's part of the ring: its stages, then a chunk's scales as every lane reads them.
  static constexpr int kWarpBytes = kDepth * kStageBytes + (kSteps * 256 + 1023) / 1024 * 1024;
  static constexpr CUtensorMapSwizzle kSwizzle = kRowBytes == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                                 : kRowBytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                                   : CU_TENSOR_MAP_SWIZZLE_NONE;
  // TMA swaps 16-byte units of a box's rows so that rows start in other banks: byte `off`
  // of row r is at r * kRowBytes + (off ^ swap(r)), the same for r + 8.
  __device__ static __forceinline__ uint32_t swap(uint32_t r) {
    return kRowBytes == 128 ? (r & 7u) << 4 : kRowBytes == 64 ? (r >> 1 & 3u) << 4 : 0u;
  }
};

// Codes as bf16 pairs, each code * 2^-15.  A bf16 pattern P <= 0xFF is worth P * 2^-133, so a
// code at bit o of an otherwise clear half reads as c * 2^(o - 133), and times 2^(118 - o) it is
// exact and normal; sum(x) is taken times 2^-15 too, and the sums times 2^15 at the end.  Not
// multiplied as it stands, with the powers of two in x: the tensor cores line products up by
// their factors' exponents, and an unnormalised code costs the sum up to 7 of its last bits
// (1e-5 of the outputs' norm; the few x instead of the many codes saved 5 % of the time).
// 2^-15, so that 128 codes of 8 bits do not take a sum beyond its x: x as large as fp32 holds
// goes in, and sums keep all their bits down to x of 2^-110.
// The factors come with the call's arguments: constants would be put into a register again
// for every product (32 instructions a group).
constexpr uint32_t kCodeScale = 0x7A807A80u;  // 2^118, twice
constexpr uint32_t kOnes = 0x38003800u;       // 2^-15, twice
constexpr float kUnscale = 32768.0f;
template <int BITS>
struct Factors {
  static constexpr int kCount = BITS == 8 ? 1 : BITS == 4 ? 2 : BITS == 2 ? 4 : 1;
  uint32_t v[kCount];  // (2^(118 - o), 2^(118 - o)) for o = 0, BITS, 2 BITS ..
  __device__ __forceinline__ explicit Factors(uint32_t code_scale) {
#pragma unroll
    for (int i = 0; i < kCount; ++i) v[i] = code_scale - (static_cast<uint32_t>(i * BITS) << 7) * 0x00010001u;
  }
};

template <int BITS, int G>
__device__ __forceinline__ void spread_codes(const uint32_t *v, int sub, const Factors<BITS> &f,
                                             uint32_t (&p)[Run<BITS, G>::kSub / 2]) {
  using R = Run<BITS, G>;
  if constexpr (R::kSplit) {
    constexpr int kHalf = 16 / BITS, kPerSub = R::kSub * BITS / 32;
    constexpr uint32_t kMask = ((1u << BITS) - 1u) * 0x00010001u;
#pragma unroll
    for (int i = 0; i < kPerSub; ++i) {
      const uint32_t w = v[sub * kPerSub + i];
#pragma unroll
      for (int j = 0; j < kHalf; ++j) {
        const int o = j * BITS % 8, sh = j * BITS - o;
        p[i * kHalf + j] = bf16x2_fma((w >> sh) & (kMask << o), f.v[o / BITS], 0x80008000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < R::kSub / 2; ++i)
      p[i] = bf16x2_fma(pair_at<BITS>(v, sub * R::kSub + 2 * i), f.v[0], 0x80008000u);
  }
}

// x of those codes, in the same pairs.
template <int BITS, int G>
__device__ __forceinline__ void pair_x(const uint16_t *x, uint32_t (&p)[Run<BITS, G>::kSub / 2]) {
  using R = Run<BITS, G>;
  uint32_t n[R::kSub / 2];
#pragma unroll
  for (int i = 0; i < R::kSub / 8; ++i) {
    const uint4 u = *reinterpret_cast<const uint4 *>(x + 8 * i);
    n[4 * i] = u.x, n[4 * i + 1] = u.y, n[4 * i + 2] = u.z, n[4 * i + 3] = u.w;
  }
  if constexpr (R::kSplit) {
    constexpr int kHalf = 16 / BITS;
#pragma unroll
    for (int i = 0; i < R::kSub / 2; ++i) {
      const int word = i / kHalf, j = i % kHalf, at = word * kHalf + j / 2;
      p[i] = prmt(n[at], n[at + kHalf / 2], j & 1 ? 0x7632u : 0x5410u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < R::kSub / 2; ++i) p[i] = n[i];
  }
}

// ------------------------------------------------------------- the ring ----

template <int N, int OFF>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t *v) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4 + %5];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(a), "n"(OFF));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2 + %3];" : "=r"(v[0]), "=r"(v[1]) : "r"(a), "n"(OFF));
  else
    asm volatile("ld.shared.u32 %0, [%1 + %2];" : "=r"(v[0]) : "r"(a), "n"(OFF));
}

// Scales and biases of a chunk, of the row that this lane stands for: row g + 8 (t % 2) of
// tile t / 2 for lane 4 g + t.  16-bit types are kept in pairs.
template <int STEPS>
struct Scales {
  static constexpr int kPairs = (STEPS + 1) / 2;
  uint32_t s[STEPS], b[STEPS];

  template <int N>
  __device__ static __forceinline__ void load_words(const void *p, uint32_t *v) {
    if constexpr (N == 4) {
      const uint4 u = __ldg(static_cast<const uint4 *>(p));
      v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
    } else if constexpr (N == 2) {
      const uint2 u = __ldg(static_cast<const uint2 *>(p));
      v[0] = u.x, v[1] = u.y;
    } else {
      v[0] = __ldg(static_cast<const uint32_t *>(p));
    }
  }
  // As fp32 pairs (s, b) to `to`, [step][lane's row]: what every lane of the rows reads.
  __device__ static __forceinline__ void put(uint32_t at, float fs, float fb) {
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(fs), "f"(fb) : "memory");
  }
  __device__ __forceinline__ void spread(uint32_t at, int type) const {
    if (type == kTypeBF16) {
#pragma unroll
      for (int i = 0; i < STEPS; ++i)
        put(at + i * 256, __uint_as_float(i & 1 ? s[i / 2] & 0xFFFF0000u : s[i / 2] << 16),
            __uint_as_float(i & 1 ? b[i / 2] & 0xFFFF0000u : b[i / 2] << 16));
    } else if (type == kTypeF16) {
#pragma unroll
      for (int i = 0; i < STEPS; ++i)
        put(at + i * 256, ElemF16::to_f32(s[i / 2] >> (16 * (i & 1)) & 0xFFFFu), ElemF16::to_f32(b[i / 2] >> (16 * (i & 1)) & 0xFFFFu));
    } else {
#pragma unroll
      for (int i = 0; i < STEPS; ++i) put(at + i * 256, __uint_as_float(s[i]), __uint_as_float(b[i]));
    }
  }
  // From ps and pb on, `count` groups of them.  `whole`: 16-bit types, rows of whole chunks
  // (which are then aligned, as every row is).
  __device__ __forceinline__ void load(const char *ps, const char *pb, int type, bool whole, int count) {
    if (STEPS > 1 && whole) {
      load_words<kPairs>(ps, s);
      load_words<kPairs>(pb, b);
    } else {
      load_some(ps, pb, type, count);
    }
  }
  __device__ __forceinline__ void load_some(const char *ps, const char *pb, int type, int count) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i) s[i] = b[i] = 0;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      if (i >= count) break;
      if (type == kTypeF32) {
        s[i] = __ldg(reinterpret_cast<const uint32_t *>(ps) + i);
        b[i] = __ldg(reinterpret_cast<const uint32_t *>(pb) + i);
      } else {
        s[i / 2] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t *>(ps) + i)) << (16 * (i % 2));
        b[i / 2] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t *>(pb) + i)) << (16 * (i % 2));
      }
    }
  }
};

// The MMA's columns: rows of x (or h) of up to 8 slots, lane 4 g + t reading column g.
// Columns without a slot repeat the first: nothing looks at their sums.
struct Columns {
  const uint16_t *x;  // this lane's column, at its run
  int planes;
  int64_t plane;
};

// d = a b (FIRST) or d += a b.
template <bool FIRST>
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (FIRST)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The products of up to 16 codes a lane with one plane of x.
template <int BITS, int G, bool FIRST>
__device__ __forceinline__ void multiply(const uint32_t (&code)[4][Run<BITS, G>::kSub / 2],
                                         const uint32_t (&x)[Run<BITS, G>::kSub / 2], float (&part)[2][4], float (&ones)[4]) {
  using R = Run<BITS, G>;
#pragma unroll
  for (int m = 0; m < R::kSub / 4; ++m) {
    if (FIRST && m == 0) {
#pragma unroll
      for (int tile = 0; tile < 2; ++tile)
        mma_bf16<true>(part[tile], code[2 * tile][0], code[2 * tile + 1][0], code[2 * tile][1], code[2 * tile + 1][1], x[0], x[1]);
      mma_bf16<true>(ones, kOnes, kOnes, kOnes, kOnes, x[0], x[1]);
    } else {
#pragma unroll
      for (int tile = 0; tile < 2; ++tile)
        mma_bf16<false>(part[tile], code[2 * tile][2 * m], code[2 * tile + 1][2 * m], code[2 * tile][2 * m + 1],
                        code[2 * tile + 1][2 * m + 1], x[2 * m], x[2 * m + 1]);
      mma_bf16<false>(ones, kOnes, kOnes, kOnes, kOnes, x[2 * m], x[2 * m + 1]);
    }
  }
}

// One chunk of 32 rows: acc[2 q + column] += s sum(c x) + b sum(x) over its `count`
// groups, q = 2 tile + row half; `at` is the chunk's first column, `scales` where its scales
// were spread.  Not unrolled over groups: the warps share an instruction cache that the body
// must not outgrow.
template <int BITS, int G>
__device__ __forceinline__ void consume(uint32_t stage, int lane, const Columns &c, int at, int count,
                                        uint32_t scales, const Factors<BITS> &f, float (&acc)[8]) {
  using R = Run<BITS, G>;
  const int g = lane / 4, t = lane % 4;
  const uint32_t rows = stage + g * R::kRowBytes, flip = (t * R::kBits / 32 * 4) ^ R::swap(g);
  const uint16_t *px = c.x + at;
  uint32_t sb = scales + g * 8;
  count = min(count, R::kSteps);
#pragma unroll 1
  for (int step = 0; step < count; ++step, sb += 256) {
    float part[2][4], ones[4];
    uint32_t v[4][R::kWords + 1];
#pragma unroll
    for (int i = 0; i < R::kWords; i += R::kPiece) {
      // (a row's 16-byte units keep their order where nothing is swapped)
      const uint32_t off = step * (G * BITS / 8) + 4 * i;
      const uint32_t from = rows + (R::kSwizzle == CU_TENSOR_MAP_SWIZZLE_NONE ? off + flip : R::kWhole ? off ^ flip
                                        : ((off + t * R::kBits / 32 * 4) ^ R::swap(g)));
      lds_words<R::kPiece, 0>(from, &v[0][i]);
      lds_words<R::kPiece, 8 * R::kRowBytes>(from, &v[1][i]);
      lds_words<R::kPiece, 16 * R::kRowBytes>(from, &v[2][i]);
      lds_words<R::kPiece, 24 * R::kRowBytes>(from, &v[3][i]);
    }
    if constexpr (!R::kWhole) {
      const uint32_t sh = t * R::kBits % 32;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[q][R::kWords] = 0;
#pragma unroll
        for (int i = 0; i < R::kWords; ++i) v[q][i] = __funnelshift_r(v[q][i], v[q][i + 1], sh);
      }
    }
#pragma unroll
    for (int sub = 0; sub < R::kCodes / R::kSub; ++sub) {
      uint32_t x[R::kSub / 2];  // loaded ahead of the codes' instructions
      pair_x<BITS, G>(px + sub * R::kSub, x);
      uint32_t code[4][R::kSub / 2];
#pragma unroll
      for (int q = 0; q < 4; ++q) spread_codes<BITS, G>(v[q], sub, f, code[q]);
      if (c.planes < 3) {
        if (sub == 0) multiply<BITS, G, true>(code, x, part, ones);
        else multiply<BITS, G, false>(code, x, part, ones);
        if (c.planes == 2) {
          pair_x<BITS, G>(px + sub * R::kSub + c.plane, x);
          multiply<BITS, G, false>(code, x, part, ones);
        }
      } else {
        // fp32: the smallest part of x first, the tensor cores cut what they add to a large sum.
        if (sub == 0)
#pragma unroll
          for (int i = 0; i < 4; ++i) part[0][i] = part[1][i] = ones[i] = 0.0f;
#pragma unroll 1
        for (int plane = 2; plane >= 0; --plane) {
          pair_x<BITS, G>(px + sub * R::kSub + plane * c.plane, x);
          multiply<BITS, G, false>(code, x, part, ones);
        }
      }
    }
    px += G;
    uint32_t both[4][2];
    lds_words<2, 0>(sb, both[0]);
    lds_words<2, 64>(sb, both[1]);
    lds_words<2, 128>(sb, both[2]);
    lds_words<2, 192>(sb, both[3]);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float s = __uint_as_float(both[q][0]), b = __uint_as_float(both[q][1]);
#pragma unroll
      for (int i = 0; i < 2; ++i) acc[2 * q + i] = fmaf(s, part[q / 2][2 * (q % 2) + i], fmaf(b, ones[i], acc[2 * q + i]));
    }
  }
}

// Brings a chunk of x of the unit's slots into L1 ahead of its use: a 4-byte copy of each
// 32-byte sector to a place that nothing reads.
template <int CHUNK, bool TOKENS>
__device__ __forceinline__ void touch_x(uint32_t scratch, const uint16_t *x, int64_t plane, int planes, const MoeEntry *slots,
                                        int count, int width, int chunk, int lane) {
  constexpr int kSectors = CHUNK / 16;
  const int all = count * kSectors;
  for (int p = 0; p < planes; ++p) {
    for (int i = lane; i < all; i += 32) {
      const int row = TOKENS ? slots[i / kSectors].token : slots[i / kSectors].listed, at = chunk * CHUNK + i % kSectors * 16;
      const uint16_t *from = x + p * plane + static_cast<int64_t>(row) * width + at;
      if (at < width)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(scratch + 4 * lane), "l"(from) : "memory");
    }
  }
}

// A weight whose boxes are loaded.  Rows that are no multiple of 16 bytes long (hidden or
// inner times bits no multiple of 128, which 4 and 8 bits never are) are out of TMA's reach:
// the warp then copies its chunks itself, as it comes to them.
struct Source {
  const CUtensorMap *map;
  const uint32_t *w;  // where the warp copies, else null
  int words;          // of a row
};

// A warp's ring of chunks.
template <int BITS, int G>
struct Ring {
  using R = Run<BITS, G>;
  uint32_t base;
  uint64_t *bars;
  int lane, in, out;
  uint32_t parity;   // of the stage to read next
  int flying;        // chunks issued and not yet waited for

  __device__ __forceinline__ void init(unsigned char *stages, uint64_t *barriers, int warp, int lane_) {
    base = smem_u32(stages) + warp * R::kWarpBytes;
    bars = barriers + warp * R::kDepth;
    lane = lane_;
    in = out = flying = 0;
    parity = 0;
    if (lane == 0) {
      for (int i = 0; i < R::kDepth; ++i) mbar_init(&bars[i], 1);
      asm volatile("fence.mbarrier_init.release.cluster;\n\tfence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncwarp();
  }
  // Chunk `chunk` of the 16 rows at y0 of map0 and at y1 of map1.
  __device__ __forceinline__ void issue(const Source &s0, const Source &s1, int y0, int y1, int chunk) {
    const uint32_t st = base + in * R::kStageBytes;
    constexpr int kRowWords = R::kRowBytes / 4;
    if (BITS != 4 && BITS != 8 && s0.w) {
      for (int i = lane; i < 32 * kRowWords; i += 32) {
        const int row = i / kRowWords, at = i - row * kRowWords, word = chunk * kRowWords + at;
        const uint32_t *p = (row < 16 ? s0.w : s1.w) + static_cast<int64_t>((row < 16 ? y0 : y1) + row % 16) * s0.words;
        const uint32_t v = word < s0.words ? __ldg(p + word) : 0u;
        const uint32_t to = st + row / 16 * (R::kStageBytes / 2) + (row % 16) * R::kRowBytes + ((4 * at) ^ R::swap(row));
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(to), "r"(v) : "memory");
      }
    } else if (lane == 0) {
      mbar_expect_tx(&bars[in], R::kStageBytes);
      tma_load_2d(st, s0.map, chunk * kRowWords, y0, &bars[in]);
      tma_load_2d(st + R::kStageBytes / 2, s1.map, chunk * kRowWords, y1, &bars[in]);
    }
    in = in + 1 == R::kDepth ? 0 : in + 1;
    ++flying;
  }
  // Waits for the oldest chunk; its stage, or 0 if the wait ran out.
  __device__ __forceinline__ uint32_t wait(bool copied, uint32_t limit, unsigned *err) {
    if ((BITS == 4 || BITS == 8 || !copied) && !__all_sync(0xFFFFFFFFu, mbar_try_wait(&bars[out], parity))) {
      uint32_t polls = 0;
      do {
        if (++polls >= limit) {
          if (lane == 0) atomicOr(err, kErrTimeoutBit);
          return 0;
        }
      } while (!__all_sync(0xFFFFFFFFu, mbar_try_wait(&bars[out], parity)));
    }
    __syncwarp();
    return base + out * R::kStageBytes;
  }
  // The stage may be filled again.
  __device__ __forceinline__ void done() {
    __syncwarp();
    out = out + 1 == R::kDepth ? 0 : out + 1;
    if (out == 0) parity ^= 1;
    --flying;
  }
  // No copy may land after the block has left (flying: a wait has run out).  Not with the
  // caller's limit, which may be one poll.
  __device__ __forceinline__ void drain(bool copied, unsigned *err) {
    while (flying > 0) {
      wait(copied, kDefaultWaitLimit, err);
      done();
    }
  }
};

// The bf16 planes of v: the nearest bf16 number, then that of what is left of it, exactly (two
// hold v to 2^-18 of itself, three all of its 24 bits).  What is not finite stays in the first;
// what would round to infinity is cut there instead.
__device__ __forceinline__ void store_planes(uint16_t *p, int64_t plane, int planes, float v) {
  for (int i = 0; i < planes; ++i) {
    uint32_t near = static_cast<uint32_t>(f32_to_bf16_bits(v)) << 16;
    if ((near & 0x7F800000u) == 0x7F800000u && fabsf(v) < INFINITY) near = __float_as_uint(v) & 0xFFFF0000u;
    p[i * plane] = static_cast<uint16_t>(near >> 16);
    v = (near & 0x7F800000u) != 0x7F800000u ? v - __uint_as_float(near) : 0.0f;
  }
}

// -------------------------------------------------------- gate and up ----

struct alignas(1024) GateUpShared {  // the ring follows (swizzled boxes want 1024), then the plan
  alignas(16) float heads[kMoeWarps][32 * kMoePass];  // sums of a warp's first task where it began in an earlier one
  int task[2][kMoeWarps];  // the task that goes on in the next warp, the head's; -1: none
  alignas(16) uint64_t bars[kMoeWarps * 4];
  uint32_t unread[32];
};
struct MoeMaps {
  CUtensorMap gate, up, down;
};

// gate / (1 + exp(-gate)) * up, by exp(-|gate|) so that the divisor is in [1, 2]: exp(-gate)
// itself leaves fp32, and __fdividef's range, below -87, where the product with up need not
// have vanished.
__device__ __forceinline__ float silu_times(float gate, float up) {
  const float e = expf(-fabsf(gate));
  return __fdividef(gate >= 0.0f ? gate : gate * e, 1.0f + e) * up;
}

// h = silu(gate x) * (up x).  A task is a unit and 16 rows of gate and of up.  A block has
// a run of tasks, whose chunks, in order, are cut evenly over its warps; a task within one
// warp is finished there (gate and up of a row are in the same lane), one that is cut is
// joined through shared memory at the end.
template <int BITS, int G>
struct GateUp {
  using R = Run<BITS, G>;
  const MoeArgs &a;
  GateUpShared &sh;
  MoeEntry *plan;
  int units;
  Ring<BITS, G> ring;
  Source gate, up;
  const char *scales, *biases;
  bool copied;
  int lane, warp, tiles, groups, chunks;
  int task, chunk, unit, tile, left;  // what is multiplied next, chunks left to this warp
  int l_chunk, l_unit, l_tile, l_left, l_row;  // what is loaded next
  bool l_fresh;                       // its unit's x is not in L1 yet
  int s_chunk, s_unit, s_tile;        // whose scales are loaded next, and where they are
  const char *s_at, *b_at;
  int sb_bytes;
  bool whole;
  Scales<R::kSteps> next;
  Factors<BITS> factors{a.code_scale};

  __device__ __forceinline__ void advance_load() {
    if (l_left <= 0) return;
    ring.issue(gate, up, l_row, l_row, l_chunk);
    if (l_fresh)
      touch_x<R::kChunk, true>(smem_u32(sh.unread), a.x, a.x_plane, a.x_planes, &plan[plan[l_unit].unit_first],
                               plan[l_unit].unit_count, a.w.hidden, l_chunk, lane);
    --l_left;
    if (++l_chunk == chunks) {
      l_chunk = 0;
      l_fresh = false;
      l_row += 16;
      if (++l_tile == tiles) {
        l_tile = 0, ++l_unit, l_fresh = true;
        if (l_left > 0) l_row = plan[l_unit].unit_expert * a.w.inner;
      }
    }
  }
  // The next chunk's scales, of the row that this lane stands for.
  __device__ __forceinline__ void load_scales() {
    next.load(s_at, b_at, a.w.sb_type, whole, groups - s_chunk * R::kSteps);
    s_at += R::kSteps * sb_bytes, b_at += R::kSteps * sb_bytes;
    if (++s_chunk == chunks) {
      if (++s_tile == tiles) s_tile = 0, ++s_unit;
      s_chunk = 0;
      if (s_unit < units) point_scales();
    }
  }
  __device__ __forceinline__ void point_scales() {
    const int64_t row = static_cast<int64_t>(plan[s_unit].unit_expert) * a.w.inner + s_tile * 16 + lane / 4 + 8 * (lane % 2);
    const int64_t at = (row * groups + s_chunk * R::kSteps) * sb_bytes;
    s_at = scales + at, b_at = biases + at;
  }
  __device__ __forceinline__ float *starts(int w) const {
    static_assert(R::kDepth * R::kStageBytes >= 32 * kMoePass * 4, "a warp's sums fit its ring");
    return reinterpret_cast<float *>(reinterpret_cast<unsigned char *>(&sh) + sizeof(GateUpShared) + w * R::kWarpBytes);
  }
  __device__ __forceinline__ void run_task() {
    const int g = lane / 4, t = lane % 4, count = plan[unit].unit_count;
    const MoeEntry *listed = &plan[plan[unit].unit_first];
    Columns c;
    c.planes = a.x_planes;
    c.plane = a.x_plane;
    const int token = listed[g < count ? g : 0].token;
    c.x = a.x + static_cast<int64_t>(token) * a.w.hidden + t * R::kCodes;
    const uint32_t spread = ring.base + R::kDepth * R::kStageBytes, own_scales = spread + (lane % 4) * 64 + lane / 4 * 8;
    float acc[8] = {};
    const int c0 = chunk, c1 = min(chunks, chunk + left);
    for (; chunk < c1; ++chunk) {
      // (the chunk before is read: done() has met the warp)
      next.spread(own_scales, a.w.sb_type);
      if (--left > 0) load_scales();
      const uint32_t stage = ring.wait(copied, a.wait_limit, a.err);
      if (!stage) {
        left = l_left = 0;
        return;
      }
      consume<BITS, G>(stage, lane, c, chunk * R::kChunk, groups - chunk * R::kSteps, spread, factors, acc);
      ring.done();
      advance_load();
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] *= kUnscale;
    if (c0 == 0 && c1 == chunks) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int place = 2 * t + i;
        if (place < count) {
          const int slot = listed[place].listed;
          uint16_t *to = a.h + static_cast<int64_t>(slot) * a.w.inner + tile * 16 + g;
          const float h0 = silu_times(acc[i], acc[4 + i]), h1 = silu_times(acc[2 + i], acc[6 + i]);
          store_planes(to, a.h_plane, a.h_planes, h0);
          store_planes(to + 8, a.h_plane, a.h_planes, h1);
        }
      }
    } else {
      const int kind = c0 == 0 ? 0 : 1;
      if (lane == 0) sh.task[kind][warp] = task;
      // a task that goes on is the warp's last: its ring is free
      float *to = kind ? sh.heads[warp] : starts(warp);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<float2 *>(to + ((q / 2) * 16 + (q % 2) * 8 + g) * kMoePass + 2 * t) = make_float2(acc[2 * q], acc[2 * q + 1]);
    }
    chunk = 0;
    ++task;
    if (++tile == tiles) tile = 0, ++unit;
  }
};

template <int BITS, int G>
__global__ void __launch_bounds__(kMoeThreads, 2)
gate_up_kernel(const __grid_constant__ MoeArgs a, const __grid_constant__ MoeMaps maps) {
  using R = Run<BITS, G>;
  extern __shared__ __align__(1024) unsigned char raw[];
  GateUp<BITS, G> s{a, *reinterpret_cast<GateUpShared *>(raw),
                    reinterpret_cast<MoeEntry *>(raw + sizeof(GateUpShared) + kMoeWarps * R::kWarpBytes + 16)};
  s.warp = threadIdx.x / 32, s.lane = threadIdx.x % 32;
  s.ring.init(raw + sizeof(GateUpShared), s.sh.bars, s.warp, s.lane);
  if (threadIdx.x < 2 * kMoeWarps) s.sh.task[threadIdx.x / kMoeWarps][threadIdx.x % kMoeWarps] = -1;
  // The plan and x's planes are complete.  Kernels launched from here on may read the plan
  // too, before this one is done.
  griddep_wait();
  griddep_launch_dependents();
  s.units = read_plan(a.plan, s.plan, a.tokens * a.route.top_k);
  s.tiles = a.w.inner / 16, s.groups = a.w.hidden / G, s.chunks = (a.w.hidden + R::kChunk - 1) / R::kChunk;
  // Tasks t0 .. t1 of the block, an even share; steps from .. of the warp.
  const int tasks = s.units * s.tiles, grid = gridDim.x, block = blockIdx.x;
  const int share = tasks / grid, rest = tasks - share * grid;
  const int t0 = share * block + min(block, rest), t1 = t0 + share + (block < rest);
  const int steps = (t1 - t0) * s.chunks;
  auto cut = [&](int w) { return steps / kMoeWarps * w + steps % kMoeWarps * w / kMoeWarps; };
  const int from = cut(s.warp);
  s.left = s.l_left = cut(s.warp + 1) - from;
  s.task = t0 + from / s.chunks;
  s.chunk = s.l_chunk = from % s.chunks;
  s.unit = s.l_unit = s.task / s.tiles;
  s.tile = s.l_tile = s.task % s.tiles;
  s.l_fresh = true;
  s.l_row = s.left > 0 ? s.plan[s.unit].unit_expert * a.w.inner + s.tile * 16 : 0;
  s.copied = static_cast<int64_t>(a.w.hidden) * BITS % 128 != 0;
  s.gate = Source{&maps.gate, s.copied ? a.w.w[0] : nullptr, a.w.hidden / 32 * BITS};
  s.up = Source{&maps.up, s.copied ? a.w.w[1] : nullptr, a.w.hidden / 32 * BITS};
  s.scales = static_cast<const char *>(s.lane % 4 < 2 ? a.w.scales[0] : a.w.scales[1]);
  s.biases = static_cast<const char *>(s.lane % 4 < 2 ? a.w.biases[0] : a.w.biases[1]);
  for (int i = 0; i < R::kDepth; ++i) s.advance_load();
  s.sb_bytes = a.w.sb_type == kTypeF32 ? 4 : 2;
  s.whole = a.w.sb_type != kTypeF32 && s.groups % R::kSteps == 0;
  s.s_chunk = s.chunk, s.s_unit = s.unit, s.s_tile = s.tile;
  if (s.left > 0) s.point_scales(), s.load_scales();
  while (s.left > 0) {
    s.run_task();
  }
  s.ring.drain(s.copied, a.err);
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  const int r = threadIdx.x % 16, place = threadIdx.x / 16;
  for (int w = 0; w < kMoeWarps; ++w) {
    const int task = s.sh.task[0][w];
    if (task < 0) continue;
    const int unit = task / s.tiles, tile = task % s.tiles;
    if (place >= s.plan[unit].unit_count) continue;
    const int at = r * kMoePass + place, two = 16 * kMoePass;
    float gate = s.starts(w)[at], up = s.starts(w)[at + two];
    for (int v = w + 1; v < kMoeWarps; ++v)
      if (s.sh.task[1][v] == task) gate += s.sh.heads[v][at], up += s.sh.heads[v][at + two];
    const int slot = s.plan[s.plan[unit].unit_first + place].listed;
    const float h = silu_times(gate, up);
    store_planes(a.h + static_cast<int64_t>(slot) * a.w.inner + tile * 16 + r, a.h_plane, a.h_planes, h);
  }
}

// ---------------------------------------------------------------- down ----

struct alignas(1024) DownShared {  // then the ring, the plan, z: float [slots][32]
  alignas(16) float heads[kMoeWarps][kMoePass][32];
  alignas(16) uint64_t bars[kMoeWarps * 4];
  uint32_t unread[32];
  unsigned char unit_from[kMoeMaxSlots], unit_to[kMoeMaxSlots];
};

// y = sum over a token's slots of weight * (down h).  A cluster takes 32 rows of every
// unit: the steps (unit, chunk), in order, are cut evenly over the cluster's warps, so a
// warp's first unit may have begun in another warp.  Sums from a unit's first chunk on go
// to z, those of a unit that began earlier to the warp's head; after the cluster's barrier
// its blocks add them up, token by token, in a fixed order.
template <int BITS, int G>
__global__ void __launch_bounds__(kMoeThreads, 2)
down_kernel(const __grid_constant__ MoeArgs a, const __grid_constant__ MoeMaps maps, int cluster) {
  using R = Run<BITS, G>;
  extern __shared__ __align__(1024) unsigned char raw[];
  DownShared &sh = *reinterpret_cast<DownShared *>(raw);
  const int slots = a.tokens * a.route.top_k;
  MoeEntry *plan = reinterpret_cast<MoeEntry *>(raw + sizeof(DownShared) + kMoeWarps * R::kWarpBytes);
  float *z = reinterpret_cast<float *>(plan + slots);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  Ring<BITS, G> ring;
  ring.init(raw + sizeof(DownShared), sh.bars, warp, lane);
  const int units = read_plan(a.plan, plan, slots);
  const int rank = blockIdx.x % cluster, row0 = blockIdx.x / cluster * 32;
  const int groups = a.w.inner / G, chunks = (a.w.inner + R::kChunk - 1) / R::kChunk;
  const int total = units * chunks;  // at most 2^22: sizes are at most 2^20
  // Warps that share the steps, none without any; warp w begins at step total * w / warps.
  const int warps = min(cluster * kMoeWarps, total), self = rank * kMoeWarps + warp;
  const int step0 = self < warps ? total * self / warps : total;
  const int step1 = self < warps ? total * (self + 1) / warps : total;
  // The warps that have a unit's first and last step: step s is in warp w where
  // total * w / warps <= s < total * (w + 1) / warps, so w = ((s + 1) * warps - 1) / total.
  for (int u = threadIdx.x; u < units; u += kMoeThreads) {
    sh.unit_from[u] = static_cast<unsigned char>(((u * chunks + 1) * warps - 1) / total);
    sh.unit_to[u] = static_cast<unsigned char>(((u + 1) * chunks * warps - 1) / total);
  }
  const char *const scales = static_cast<const char *>(a.w.scales[2]);
  const char *const biases = static_cast<const char *>(a.w.biases[2]);
  // this lane's row for scales: row g + 8 (t % 2) of tile t / 2
  const int sb_bytes = a.w.sb_type == kTypeF32 ? 4 : 2;
  const bool whole = a.w.sb_type != kTypeF32 && groups % R::kSteps == 0;
  Scales<R::kSteps> next;
  const char *s_at = nullptr, *b_at = nullptr;
  auto point_scales = [&](int unit, int chunk) {
    const int64_t row = static_cast<int64_t>(plan[unit].unit_expert) * a.w.hidden + row0 + g + 8 * t;
    const int64_t at = (row * groups + chunk * R::kSteps) * sb_bytes;
    s_at = scales + at, b_at = biases + at;
  };
  auto load_scales = [&](int chunk) {
    next.load(s_at, b_at, a.w.sb_type, whole, groups - chunk * R::kSteps);
    s_at += R::kSteps * sb_bytes, b_at += R::kSteps * sb_bytes;
  };
  const bool copied = static_cast<int64_t>(a.w.inner) * BITS % 128 != 0;
  const Source down{&maps.down, copied ? a.w.w[2] : nullptr, a.w.inner / 32 * BITS};
  const int first_unit = step0 / chunks, first_chunk = step0 - first_unit * chunks;
  int load_step = step0, load_unit = first_unit, load_chunk = first_chunk;
  auto touch_h = [&](int unit, int chunk) {
    touch_x<R::kChunk, false>(smem_u32(sh.unread), a.h, a.h_plane, a.h_planes, &plan[plan[unit].unit_first],
                              plan[unit].unit_count, a.w.inner, chunk, lane);
  };
  int load_row = step0 < step1 ? plan[load_unit].unit_expert * a.w.hidden + row0 : 0;
  auto load_next = [&](bool touch) {
    if (load_step >= step1) return;
    ring.issue(down, down, load_row, load_row + 16, load_chunk);
    if (touch) touch_h(load_unit, load_chunk);
    ++load_step;
    if (++load_chunk == chunks) {
      load_chunk = 0, ++load_unit;
      if (load_step < step1) load_row = plan[load_unit].unit_expert * a.w.hidden + row0;
    }
  };
  for (int i = 0; i < R::kDepth; ++i) load_next(false);
  if (step0 < step1) point_scales(first_unit, first_chunk), load_scales(first_chunk);
  griddep_wait();  // h is complete; the weights above do not depend on it
  for (int i = step0, u = first_unit, k = first_chunk; i < load_step; ++i) {
    touch_h(u, k);
    if (++k == chunks) k = 0, ++u;
  }

  const uint32_t spread = ring.base + R::kDepth * R::kStageBytes, own_scales = spread + t * 64 + g * 8;
  const Factors<BITS> factors(a.code_scale);
  int step = step0;
  auto run_unit = [&](int unit, int j0) {
    const int j1 = min(chunks, j0 + (step1 - step));
    const int count = plan[unit].unit_count;
    const MoeEntry *listed = &plan[plan[unit].unit_first];
    Columns c;
    c.planes = a.h_planes;
    c.plane = a.h_plane;
    const int own_slot = listed[g < count ? g : 0].listed;
    c.x = a.h + static_cast<int64_t>(own_slot) * a.w.inner + t * R::kCodes;
    float acc[8] = {};
    for (int j = j0; j < j1; ++j) {
      next.spread(own_scales, a.w.sb_type);
      ++step;
      if (step < step1) {
        const bool same = j + 1 < chunks;
        if (!same) point_scales(unit + 1, 0);
        load_scales(same ? j + 1 : 0);
      }
      const uint32_t stage = ring.wait(copied, a.wait_limit, a.err);
      if (!stage) {
        step = load_step = step1;
        return;
      }
      consume<BITS, G>(stage, lane, c, j * R::kChunk, groups - j * R::kSteps, spread, factors, acc);
      ring.done();
      load_next(true);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int place = 2 * t + i;
      if (place < count) {
        float *to = j0 == 0 ? z + listed[place].listed * 32 : sh.heads[warp][place];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          to[(q / 2) * 16 + (q % 2) * 8 + g] = acc[2 * q + i] * kUnscale;
      }
    }
  };
  for (int unit = first_unit; step < step1; ++unit) {
    const int j0 = unit == first_unit ? first_chunk : 0;
    run_unit(unit, j0);
  }
  ring.drain(copied, a.err);
  asm volatile("cp.async.wait_all;" ::: "memory");
  cluster_barrier();

  // The block's tokens are rank, rank + cluster, ...: their slots' sums, weighted, go to the
  // block's own z (nobody else reads a slot of its tokens), then the tokens'.
  const uint32_t z_at = smem_u32(z) + lane * 4, heads_at = smem_u32(sh.heads) + lane * 4;
  const int top = a.route.top_k, own = a.tokens > rank ? (a.tokens - rank + cluster - 1) / cluster : 0;
  for (int i = warp; i < own * top; i += kMoeWarps) {
    const int slot = (i / top * cluster + rank) * top + i % top;
    const int at = plan[slot].slot_unit, unit = at >> 3, place = at & 7;
    float v = 0.0f;
    if (unit >= 0) {
      const int from = sh.unit_from[unit], to = sh.unit_to[unit];
      v = remote_f32(z_at + slot * 128, from / kMoeWarps);
#pragma unroll 4
      for (int w = from + 1; w <= to; ++w)
        v += remote_f32(heads_at + ((w % kMoeWarps) * kMoePass + place) * 128, w / kMoeWarps);
      v *= plan[slot].slot_weight;
    }
    z[slot * 32 + lane] = v;
  }
  __syncthreads();
  for (int i = warp; i < own; i += kMoeWarps) {
    const int token = i * cluster + rank;
    float sum = 0.0f;
    for (int k = 0; k < top; ++k) sum += z[(token * top + k) * 32 + lane];
    const int64_t at = static_cast<int64_t>(token) * a.w.hidden + row0 + lane;
    if (a.y_type == kTypeF32) static_cast<float *>(a.y)[at] = sum;
    else static_cast<uint16_t *>(a.y)[at] = a.y_type == kTypeBF16 ? ElemBF16::from_f32(sum) : ElemF16::from_f32(sum);
  }
  cluster_barrier();  // no block leaves while another reads its sums
}

// -------------------------------------------------------------- launch ----

// Boxes of 16 rows of a chunk, over all experts' rows (none where the kernels copy).
template <int BITS, int G>
cudaError_t weight_map(CUtensorMap *map, const uint32_t *w, int64_t rows, int cols) {
  using R = Run<BITS, G>;
  const uint64_t words = static_cast<uint64_t>(cols) * BITS / 32;
  if (words % 4 != 0) return cudaSuccess;
  return encode_map_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, w, words, rows, words * 4, R::kRowBytes / 4, 16, R::kSwizzle);
}

template <int BITS, int G>
cudaError_t launch_moe(const MoeArgs &a, cudaStream_t stream) {
  using R = Run<BITS, G>;
  const size_t ring = kMoeWarps * R::kWarpBytes;
  const int slots = a.tokens * a.route.top_k;
  MoeMaps maps = {};
  const int64_t inner_rows = static_cast<int64_t>(a.w.experts) * a.w.inner;
  const int64_t hidden_rows = static_cast<int64_t>(a.w.experts) * a.w.hidden;
  cudaError_t e = weight_map<BITS, G>(&maps.gate, a.w.w[0], inner_rows, a.w.hidden);
  if (e == cudaSuccess) e = weight_map<BITS, G>(&maps.up, a.w.w[1], inner_rows, a.w.hidden);
  if (e == cudaSuccess) e = weight_map<BITS, G>(&maps.down, a.w.w[2], hidden_rows, a.w.inner);
  if (e != cudaSuccess) return e;
  {
    constexpr auto kernel = gate_up_kernel<BITS, G>;
    // (16 more: a run's last word may lie past its row)
    const size_t bytes = sizeof(GateUpShared) + ring + 16 + static_cast<size_t>(slots) * sizeof(MoeEntry);
    e = ensure_smem_limit<kernel>(bytes);
    if (e != cudaSuccess) return e;
    const int64_t tasks = static_cast<int64_t>(slots) * (a.w.inner / 16), most = 2 * sm_count();
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tasks < most ? tasks : most));
    cfg.blockDim = dim3(kMoeThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, a, maps);
    if (e != cudaSuccess) return e;
  }
  constexpr auto kernel = down_kernel<BITS, G>;
  const size_t bytes = sizeof(DownShared) + static_cast<size_t>(slots) * (128 + sizeof(MoeEntry)) + ring;
  e = ensure_smem_limit<kernel>(bytes);
  if (e != cudaSuccess) return e;
  const int tiles = a.w.hidden / 32;
  int cluster = 1;
  while (cluster < kMoeMaxCluster && tiles * cluster < sm_count()) cluster *= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles * cluster);
  cfg.blockDim = dim3(kMoeThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a, maps, cluster);
}

template <int BITS>
cudaError_t launch_moe_bits(const MoeArgs &a, cudaStream_t stream) {
  switch (a.w.group) {
    case 32: return launch_moe<BITS, 32>(a, stream);
    case 64: return launch_moe<BITS, 64>(a, stream);
    default: return launch_moe<BITS, 128>(a, stream);
  }
}

// moe_bits_*.cu
cudaError_t launch_moe_bits_1_2(const MoeArgs &a, cudaStream_t stream);
cudaError_t launch_moe_bits_3(const MoeArgs &a, cudaStream_t stream);
cudaError_t launch_moe_bits_4(const MoeArgs &a, cudaStream_t stream);
cudaError_t launch_moe_bits_5_6(const MoeArgs &a, cudaStream_t stream);
cudaError_t launch_moe_bits_8(const MoeArgs &a, cudaStream_t stream);

}  // namespace qmm
