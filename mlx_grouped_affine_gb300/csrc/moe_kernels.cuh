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
// sectors) stays in L1 or L2.  Bound by memory, then by the instructions that spread codes
// (9 per 8 codes of 4 bits).  A warp works on its own: 32 weight rows (two 16-row tiles of
// the MMA, sharing the x operand) and a range of groups, whose codes each lane copies to
// its own places in shared memory (cp.async, kDepth groups ahead), so that loads in flight
// cost no registers and need no block barrier.  8 tokens fill the MMA's columns; 16 slots
// of an expert are taken per pass over its weights.
#pragma once
#include "moe_route.cuh"

namespace qmm {

constexpr int kMoeThreads = 256, kMoeWarps = kMoeThreads / 32;
constexpr int kMoePass = 16;      // slots of an expert per pass over its weights
constexpr int kMoeMaxCluster = 8;

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
  unsigned *err;
};

// ------------------------------------------------------------- the plan ----
// Which slots (token * top_k + place) go to which expert.  Every block works it out for
// itself: that is cheaper than waiting for another kernel's answer.  A unit is an expert
// with up to kMoePass of its slots; units are in order of experts, slots within them in
// order of slots, so that all blocks agree.
struct alignas(16) MoePlan {
  int units;
  int table[kMoeMaxExperts];        // slots of an expert; then first slot | first unit << 16
  short unit_expert[kMoeMaxSlots];
  short unit_first[kMoeMaxSlots];   // in list
  short unit_count[kMoeMaxSlots];
  short list[kMoeMaxSlots];         // slots by expert
  short slot_expert[kMoeMaxSlots];  // -1: no part in y
  short slot_place[kMoeMaxSlots];   // among its expert's slots
  float slot_weight[kMoeMaxSlots];
};

template <int NV>
__device__ __noinline__ void route_token(const Routing &r, int experts, int t, int lane, int &id, float &weight) {
  route_row<NV>(r, experts, t, lane, id, weight);
}

static __device__ __noinline__ void make_plan(const MoeArgs &a, MoePlan &p) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, top = a.route.top_k;
  for (int e = threadIdx.x; e < a.w.experts; e += kMoeThreads) p.table[e] = 0;
  for (int t = warp; t < a.tokens; t += kMoeWarps) {
    int id = -1;
    float weight = 0.0f;
    if (!a.route.logits) {
      if (lane < top) id = a.route.ids[t * top + lane], weight = a.route.weights[t * top + lane];
    } else if (a.w.experts <= 128) {
      route_token<4>(a.route, a.w.experts, t, lane, id, weight);
    } else if (a.w.experts <= 256) {
      route_token<8>(a.route, a.w.experts, t, lane, id, weight);
    } else {
      route_token<32>(a.route, a.w.experts, t, lane, id, weight);
    }
    if (lane < top) {
      if (id < 0 || id >= a.w.experts) {
        if (blockIdx.x == 0) atomicOr(a.err, kErrIndexBit);
        id = -1;
      }
      if (weight == 0.0f) id = -1;
      p.slot_expert[t * top + lane] = static_cast<short>(id);
      p.slot_weight[t * top + lane] = weight;
    }
  }
  __syncthreads();
  const int slots = a.tokens * top;
  if (warp == 0) {
    for (int s0 = 0; s0 < slots; s0 += 32) {  // places: slots of the same expert before
      const int s = s0 + lane, e = s < slots ? p.slot_expert[s] : -1;
      const unsigned same = __match_any_sync(0xFFFFFFFFu, e);
      const int place = __popc(same & ((1u << lane) - 1u)) + (e < 0 ? 0 : p.table[e]);
      __syncwarp();
      if (e >= 0) {
        p.slot_place[s] = static_cast<short>(place);
        if (same >> lane == 1u) p.table[e] = place + 1;  // the last of them
      }
      __syncwarp();
    }
    int before = 0;  // slots | units << 16 of the experts before
    for (int e0 = 0; e0 < a.w.experts; e0 += 32) {
      const int e = e0 + lane, n = e < a.w.experts ? p.table[e] : 0;
      const int units = (n + kMoePass - 1) / kMoePass, own = n | units << 16;
      int sum = own;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
        if (lane >= d) sum += o;
      }
      const int at = before + sum - own, first = at & 0xFFFF, unit = at >> 16;
      if (n > 0) p.table[e] = at;
      for (int i = 0; i < units; ++i) {
        p.unit_expert[unit + i] = static_cast<short>(e);
        p.unit_first[unit + i] = static_cast<short>(first + i * kMoePass);
        p.unit_count[unit + i] = static_cast<short>(min(kMoePass, n - i * kMoePass));
      }
      before += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    if (lane == 0) p.units = before >> 16;
  }
  __syncthreads();
  for (int s = threadIdx.x; s < slots; s += kMoeThreads) {
    const int e = p.slot_expert[s];
    if (e >= 0) p.list[(p.table[e] & 0xFFFF) + p.slot_place[s]] = static_cast<short>(s);
  }
  __syncthreads();
}

// ------------------------------------------------------------ the codes ----

// A lane's part of a group: the G / 4 codes [t G / 4, (t + 1) G / 4) for lane 4 g + t, so
// that the four lanes of an MMA row are in one group.
template <int BITS, int G>
struct Run {
  static constexpr int kCodes = G / 4;
  static constexpr int kBits = kCodes * BITS;
  static constexpr bool kWhole = kBits % 32 == 0;  // whole words, else shifted into place
  static constexpr int kGroupWords = G * BITS / 32;
  static constexpr int words() {
    int n = 0;
    for (int t = 0; t < 4; ++t) {
      const int w = (t * kBits % 32 + kBits + 31) / 32;
      n = w > n ? w : n;
    }
    return n;
  }
  static constexpr int kWords = words();
  // A copy's words: as many as the run's alignment (its own size) allows.
  static constexpr int kPiece = !kWhole ? 1 : kWords % 4 == 0 ? 4 : kWords % 2 == 0 ? 2 : 1;
  static constexpr int kPieces = kWords / kPiece;
  // Codes j and j + half of a word share a register (one mask for both) where a word holds
  // whole codes; otherwise neighbours do.
  static constexpr bool kSplit = kWhole && (BITS == 2 || BITS == 4 || BITS == 8);
  static constexpr int kSub = kCodes < 16 ? kCodes : 16;  // codes spread at a time
  static constexpr int kDepth = kWords <= 2 ? 6 : kWords <= 4 ? 4 : kWords <= 6 ? 3 : 2;
  static constexpr int kStageBytes = 32 * (16 * kWords + 8);  // a warp's group: codes, then scales
};

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Codes as bf16 pairs, each code * 2^-6.  A bf16 pattern P <= 0xFF is worth P * 2^-133, so
// a code at bit o of a half reads as c * 2^(o - 133), and times 2^(127 - o) it is exact and
// normal.  (kCodeScale undoes the 2^-6.)
constexpr float kCodeScale = 64.0f;
template <int BITS, int G>
__device__ __forceinline__ void spread_codes(const uint32_t *v, int sub, uint32_t (&p)[Run<BITS, G>::kSub / 2]) {
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
        p[i * kHalf + j] = bf16x2_mul((w >> sh) & (kMask << o), ((254u - o) << 7) * 0x00010001u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < R::kSub / 2; ++i)
      p[i] = bf16x2_mul(pair_at<BITS>(v, sub * R::kSub + 2 * i), (254u << 7) * 0x00010001u);
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

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ------------------------------------------------------------- the ring ----

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, uint32_t bytes = BYTES) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(bytes)
                 : "memory");
}

// Where a lane's codes, scale and bias of a unit's rows are: tile 0 and 1 at rows g (and 8
// rows on, g + 8), of two matrices or of one.
struct RowPtrs {
  const char *w[2];
  const char *s, *b;  // of the row whose scale this lane copies: tile t / 2, half t % 2
};

template <int BITS, int G>
struct Ring {
  using R = Run<BITS, G>;
  uint32_t base;        // this warp's stages
  int64_t half_bytes;   // 8 rows of codes
  int sb_bytes;
  int lane;

  // The copies of group j of the rows, as one commit group (empty if !live).
  __device__ __forceinline__ void issue(int stage, const RowPtrs &p, int j, bool live) const {
    if (live) {
      const uint32_t st = base + stage * R::kStageBytes;
      const int t = lane % 4;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const char *src = p.w[q / 2] + (q % 2) * half_bytes + static_cast<int64_t>(j) * (R::kGroupWords * 4);
        if constexpr (R::kWhole) {
          src += t * (R::kWords * 4);
#pragma unroll
          for (int i = 0; i < R::kPieces; ++i)
            copy_async<4 * R::kPiece>(st + ((q * R::kPieces + i) * 32 + lane) * (4 * R::kPiece), src + 4 * R::kPiece * i);
        } else {
          const int first = t * R::kBits / 32;
#pragma unroll
          for (int i = 0; i < R::kWords; ++i) {
            const bool in = first + i < R::kGroupWords;
            copy_async<4>(st + ((q * R::kWords + i) * 32 + lane) * 4, src + 4 * (in ? first + i : 0), in ? 4u : 0u);
          }
        }
      }
      // scale and bias: the aligned word that holds them
      const uint32_t sb = st + 32 * 16 * R::kWords + ((t * 8 + lane / 4) * 8);
      const int64_t off = static_cast<int64_t>(j) * sb_bytes;
      copy_async<4>(sb, reinterpret_cast<const char *>(reinterpret_cast<uintptr_t>(p.s + off) & ~uintptr_t(3)));
      copy_async<4>(sb + 4, reinterpret_cast<const char *>(reinterpret_cast<uintptr_t>(p.b + off) & ~uintptr_t(3)));
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
};

__device__ __forceinline__ uint2 lds2(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
template <int N>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t *v) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(a));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(a));
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[0]) : "r"(a));
}

// The MMA's columns: rows of x (or h) of up to 16 slots, lane 4 g + t reading column g.
struct Columns {
  const uint16_t *x[2];  // this lane's column of each half of the pass, at its run
  bool live[2];
  int halves;            // halves of the pass in use: 1 or 2
  int planes;
  int64_t plane;
};

// One group of 32 rows: acc[half][4 tile + 2 row half + column] += s sum(c x) + b sum(x).
template <int BITS, int G>
__device__ __forceinline__ void consume(const Ring<BITS, G> &ring, int stage, const Columns &c, int j, int sb_type,
                                        uint32_t odd, float (&acc)[2][8]) {
  using R = Run<BITS, G>;
  const uint32_t st = ring.base + stage * R::kStageBytes;
  const int lane = ring.lane, t = lane % 4;
  float part[2][2][4] = {}, ones[2][4] = {};
  uint32_t v[4][R::kWords + 1];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
#pragma unroll
    for (int i = 0; i < R::kPieces; ++i)
      lds_words<R::kPiece>(st + ((q * R::kPieces + i) * 32 + lane) * (4 * R::kPiece), &v[q][R::kPiece * i]);
    v[q][R::kWords] = 0;
    if constexpr (!R::kWhole) {
      const uint32_t sh = t * R::kBits % 32;
#pragma unroll
      for (int i = 0; i < R::kWords; ++i) v[q][i] = __funnelshift_r(v[q][i], v[q][i + 1], sh);
    }
  }
#pragma unroll
  for (int sub = 0; sub < R::kCodes / R::kSub; ++sub) {
    uint32_t code[4][R::kSub / 2];
#pragma unroll
    for (int q = 0; q < 4; ++q) spread_codes<BITS, G>(v[q], sub, code[q]);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (half < c.halves) {
        for (int plane = c.planes - 1; plane >= 0; --plane) {  // the smallest parts first
          uint32_t x[R::kSub / 2];
          if (c.live[half]) {
            pair_x<BITS, G>(c.x[half] + plane * c.plane + static_cast<int64_t>(j) * G + sub * R::kSub, x);
          } else {
#pragma unroll
            for (int i = 0; i < R::kSub / 2; ++i) x[i] = 0;
          }
#pragma unroll
          for (int m = 0; m < R::kSub / 4; ++m) {
#pragma unroll
            for (int tile = 0; tile < 2; ++tile)
              mma_bf16(part[half][tile], code[2 * tile][2 * m], code[2 * tile + 1][2 * m], code[2 * tile][2 * m + 1],
                       code[2 * tile + 1][2 * m + 1], x[2 * m], x[2 * m + 1]);
            constexpr uint32_t kOne = 0x3F803F80u;
            mma_bf16(ones[half], kOne, kOne, kOne, kOne, x[2 * m], x[2 * m + 1]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint2 sb = lds2(st + 32 * 16 * R::kWords + (q * 8 + lane / 4) * 8);
    float s, b;
    if (sb_type == kTypeBF16) {
      s = __uint_as_float(odd ? sb.x & 0xFFFF0000u : sb.x << 16);
      b = __uint_as_float(odd ? sb.y & 0xFFFF0000u : sb.y << 16);
    } else if (sb_type == kTypeF16) {
      s = ElemF16::to_f32(odd ? sb.x >> 16 : sb.x & 0xFFFFu);
      b = ElemF16::to_f32(odd ? sb.y >> 16 : sb.y & 0xFFFFu);
    } else {
      s = __uint_as_float(sb.x);
      b = __uint_as_float(sb.y);
    }
    s *= kCodeScale;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (half < c.halves) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float &y = acc[half][2 * q + i];
          y = fmaf(s, part[half][q / 2][2 * (q % 2) + i], fmaf(b, ones[half][i], y));
        }
      }
    }
  }
}

// The bf16 planes of v: its leading bits cut off 8 at a time (three hold all 24).  What is
// not finite stays in the first.
__device__ __forceinline__ void store_planes(uint16_t *p, int64_t plane, int planes, float v) {
  for (int i = 0; i < planes; ++i) {
    const uint32_t cut = __float_as_uint(v) & 0xFFFF0000u;
    p[i * plane] = static_cast<uint16_t>(cut >> 16);
    const bool more = (cut & 0x7F800000u) != 0x7F800000u;
    v = more ? v - __uint_as_float(cut) : 0.0f;
  }
}

// -------------------------------------------------------- gate and up ----

struct alignas(16) GateUpShared {
  MoePlan plan;
  alignas(16) float sums[kMoeWarps][32][kMoePass];
};
static_assert(sizeof(GateUpShared) % 16 == 0, "the ring's copies are 16 bytes wide");

// h = silu(gate x) * (up x).  An item is a unit and 16 rows of gate and of up, its groups
// split over the block's warps and joined through shared memory.
template <int BITS, int G>
__global__ void __launch_bounds__(kMoeThreads, 2) gate_up_kernel(const __grid_constant__ MoeArgs a) {
  using R = Run<BITS, G>;
  extern __shared__ __align__(128) unsigned char raw[];
  GateUpShared &sh = *reinterpret_cast<GateUpShared *>(raw);
  griddep_launch_dependents();
  make_plan(a, sh.plan);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int tiles = a.w.inner / 16, groups = a.w.hidden / G;
  const int items = sh.plan.units * tiles;
  const int j0 = groups * warp / kMoeWarps, j1 = groups * (warp + 1) / kMoeWarps;
  const int64_t row_bytes = static_cast<int64_t>(groups) * (R::kGroupWords * 4);
  Ring<BITS, G> ring;
  ring.base = smem_u32(raw) + sizeof(GateUpShared) + warp * (R::kDepth * R::kStageBytes);
  ring.half_bytes = 8 * row_bytes;
  ring.sb_bytes = a.w.sb_type == kTypeF32 ? 4 : 2;
  ring.lane = lane;

  RowPtrs p;
  int load_item = blockIdx.x, load_j = j0;
  auto point = [&](int item) {
    const int unit = item / tiles, row0 = (item - unit * tiles) * 16;
    const int64_t row = static_cast<int64_t>(sh.plan.unit_expert[unit]) * a.w.inner + row0 + g;
    p.w[0] = reinterpret_cast<const char *>(a.w.w[0]) + row * row_bytes;
    p.w[1] = reinterpret_cast<const char *>(a.w.w[1]) + row * row_bytes;
    const int64_t at = (row + 8 * (t % 2)) * groups * ring.sb_bytes;
    p.s = static_cast<const char *>(a.w.scales[t / 2]) + at;
    p.b = static_cast<const char *>(a.w.biases[t / 2]) + at;
  };
  int stage_in = 0, stage_out = 0;
  auto load_next = [&]() {
    const bool live = j0 < j1 && load_item < items;
    if (live && load_j == j0) point(load_item);
    ring.issue(stage_in, p, load_j, live);
    stage_in = stage_in + 1 == R::kDepth ? 0 : stage_in + 1;
    if (live && ++load_j == j1) load_j = j0, load_item += gridDim.x;
  };
  for (int i = 0; i < R::kDepth - 1; ++i) load_next();

  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int unit = item / tiles, row0 = (item - unit * tiles) * 16;
    const int count = sh.plan.unit_count[unit], first = sh.plan.unit_first[unit];
    const int64_t row = static_cast<int64_t>(sh.plan.unit_expert[unit]) * a.w.inner + row0 + g;
    const uint32_t row_odd = static_cast<uint32_t>(row * groups);
    Columns c;
    c.halves = count > 8 ? 2 : 1;
    c.planes = a.x_planes;
    c.plane = a.x_plane;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      c.live[half] = 8 * half + g < count;
      const int token = c.live[half] ? sh.plan.list[first + 8 * half + g] / a.route.top_k : 0;
      c.x[half] = a.x + static_cast<int64_t>(token) * a.w.hidden + t * R::kCodes;
    }
    float acc[2][8] = {};
    for (int j = j0; j < j1; ++j) {
      load_next();
      asm volatile("cp.async.wait_group %0;" ::"n"(R::kDepth - 1) : "memory");
      __syncwarp();
      consume<BITS, G>(ring, stage_out, c, j, a.w.sb_type, (row_odd + j) & 1u, acc);
      stage_out = stage_out + 1 == R::kDepth ? 0 : stage_out + 1;
      __syncwarp();  // (scales are read across lanes: before the stage is filled again)
    }
#pragma unroll
    for (int half = 0; half < 2; ++half)
      if (half < c.halves)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<float2 *>(&sh.sums[warp][(q / 2) * 16 + (q % 2) * 8 + g][half * 8 + 2 * t]) =
              make_float2(acc[half][2 * q], acc[half][2 * q + 1]);
    __syncthreads();
    const int r = threadIdx.x % 16;
    for (int k = threadIdx.x / 16; k < count; k += kMoeThreads / 16) {
      float gate = 0.0f, up = 0.0f;
#pragma unroll
      for (int i = 0; i < kMoeWarps; ++i) gate += sh.sums[i][r][k], up += sh.sums[i][16 + r][k];
      const float h = gate / (1.0f + expf(-gate)) * up;
      store_planes(a.h + static_cast<int64_t>(sh.plan.list[first + k]) * a.w.inner + row0 + r, a.h_plane, a.h_planes, h);
    }
    __syncthreads();  // before the next item's sums
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---------------------------------------------------------------- down ----

struct alignas(16) DownShared {
  MoePlan plan;
  alignas(16) float heads[kMoeWarps][kMoePass][32];
  // then z: float [slots][32], then the ring
};
static_assert(sizeof(DownShared) % 16 == 0, "the ring's copies are 16 bytes wide");

__device__ __forceinline__ float remote_f32(uint32_t addr, uint32_t rank) {
  uint32_t far;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(far) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(far) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// y = sum over a token's slots of weight * (down h).  A cluster takes 32 rows of every
// unit: the steps (unit, group), in order, are cut evenly over the cluster's warps, so a
// warp's first unit may have begun in another warp.  Sums from a unit's first group on go
// to z, those of a unit that began earlier to the warp's head; after the cluster's barrier
// its blocks add them up, token by token, in a fixed order.
template <int BITS, int G>
__global__ void __launch_bounds__(kMoeThreads, 2) down_kernel(const __grid_constant__ MoeArgs a, int cluster) {
  using R = Run<BITS, G>;
  extern __shared__ __align__(128) unsigned char raw[];
  DownShared &sh = *reinterpret_cast<DownShared *>(raw);
  float *z = reinterpret_cast<float *>(raw + sizeof(DownShared));
  const int slots = a.tokens * a.route.top_k;
  make_plan(a, sh.plan);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int rank = blockIdx.x % cluster, row0 = blockIdx.x / cluster * 32;
  const int groups = a.w.inner / G, warps = cluster * kMoeWarps;
  const int total = sh.plan.units * groups;  // at most 2^24: sizes are at most 2^20
  auto begin_of = [&](int w) { return total * w / warps; };
  const int step0 = begin_of(rank * kMoeWarps + warp), step1 = begin_of(rank * kMoeWarps + warp + 1);
  const int64_t row_bytes = static_cast<int64_t>(groups) * (R::kGroupWords * 4);
  Ring<BITS, G> ring;
  ring.base = smem_u32(z + slots * 32) + warp * (R::kDepth * R::kStageBytes);
  ring.half_bytes = 8 * row_bytes;
  ring.sb_bytes = a.w.sb_type == kTypeF32 ? 4 : 2;
  ring.lane = lane;

  RowPtrs p;
  int load_step = step0, load_unit = step0 / groups, load_j = step0 - load_unit * groups;
  const int first_unit = load_unit, first_j = load_j;
  auto point = [&](int unit) {
    const int64_t row = static_cast<int64_t>(sh.plan.unit_expert[unit]) * a.w.hidden + row0 + g;
    p.w[0] = reinterpret_cast<const char *>(a.w.w[2]) + row * row_bytes;
    p.w[1] = p.w[0] + 16 * row_bytes;
    const int64_t at = (row + 8 * t) * groups * ring.sb_bytes;  // row half t % 2 of tile t / 2
    p.s = static_cast<const char *>(a.w.scales[2]) + at;
    p.b = static_cast<const char *>(a.w.biases[2]) + at;
  };
  int stage_in = 0, stage_out = 0;
  if (step0 < step1) point(load_unit);
  auto load_next = [&]() {
    const bool live = load_step < step1;
    if (live && load_j == groups) point(++load_unit), load_j = 0;
    ring.issue(stage_in, p, load_j, live);
    stage_in = stage_in + 1 == R::kDepth ? 0 : stage_in + 1;
    ++load_step, ++load_j;
  };
  for (int i = 0; i < R::kDepth - 1; ++i) load_next();
  griddep_wait();  // h is complete; the weights above do not depend on it

  int step = step0;
  for (int unit = first_unit; step < step1; ++unit) {
    const int j0 = unit == first_unit ? first_j : 0;
    const int j1 = min(groups, j0 + (step1 - step));
    const int count = sh.plan.unit_count[unit], first = sh.plan.unit_first[unit];
    const int64_t row = static_cast<int64_t>(sh.plan.unit_expert[unit]) * a.w.hidden + row0 + g;
    const uint32_t row_odd = static_cast<uint32_t>(row * groups);
    Columns c;
    c.halves = count > 8 ? 2 : 1;
    c.planes = a.h_planes;
    c.plane = a.h_plane;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      c.live[half] = 8 * half + g < count;
      const int slot = c.live[half] ? sh.plan.list[first + 8 * half + g] : 0;
      c.x[half] = a.h + static_cast<int64_t>(slot) * a.w.inner + t * R::kCodes;
    }
    float acc[2][8] = {};
    for (int j = j0; j < j1; ++j) {
      load_next();
      asm volatile("cp.async.wait_group %0;" ::"n"(R::kDepth - 1) : "memory");
      __syncwarp();
      consume<BITS, G>(ring, stage_out, c, j, a.w.sb_type, (row_odd + j) & 1u, acc);
      stage_out = stage_out + 1 == R::kDepth ? 0 : stage_out + 1;
      __syncwarp();
    }
    step += j1 - j0;
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = half * 8 + 2 * t + i;
        if (k < count) {
          float *to = j0 == 0 ? z + sh.plan.list[first + k] * 32 : sh.heads[warp][k];
#pragma unroll
          for (int q = 0; q < 4; ++q) to[(q / 2) * 16 + (q % 2) * 8 + g] = acc[half][2 * q + i];
        }
      }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  cluster_barrier();

  const uint32_t z_at = smem_u32(z) + lane * 4, heads_at = smem_u32(sh.heads) + lane * 4;
  for (int token = warp * cluster + rank; token < a.tokens; token += warps) {
    float sum = 0.0f;
#pragma unroll 4
    for (int k = 0; k < a.route.top_k; ++k) {
      const int slot = token * a.route.top_k + k, e = sh.plan.slot_expert[slot];
      if (e < 0) continue;
      const int place = sh.plan.slot_place[slot], unit = (sh.plan.table[e] >> 16) + place / kMoePass;
      const int begin = unit * groups, end = begin + groups;
      // the warp that has the unit's first step, and those that carry on
      int w = (begin * warps + warps - 1) / total;
      while (w > 0 && begin_of(w) > begin) --w;
      while (begin_of(w + 1) <= begin) ++w;
      float v = remote_f32(z_at + slot * 128, w / kMoeWarps);
      for (++w; w < warps && begin_of(w) < end; ++w)
        if (begin_of(w) < begin_of(w + 1))
          v += remote_f32(heads_at + ((w % kMoeWarps) * kMoePass + place % kMoePass) * 128, w / kMoeWarps);
      sum = fmaf(sh.plan.slot_weight[slot], v, sum);
    }
    const int64_t at = static_cast<int64_t>(token) * a.w.hidden + row0 + lane;
    if (a.y_type == kTypeF32) static_cast<float *>(a.y)[at] = sum;
    else static_cast<uint16_t *>(a.y)[at] = a.y_type == kTypeBF16 ? ElemBF16::from_f32(sum) : ElemF16::from_f32(sum);
  }
  cluster_barrier();  // no block leaves while another reads its sums
}

// -------------------------------------------------------------- launch ----

template <int BITS, int G>
cudaError_t launch_moe(const MoeArgs &a, cudaStream_t stream) {
  using R = Run<BITS, G>;
  const size_t ring = kMoeWarps * R::kDepth * R::kStageBytes;
  const int slots = a.tokens * a.route.top_k;
  const int units = slots < a.w.experts ? slots : a.w.experts;  // near enough for the grid
  {
    constexpr auto kernel = gate_up_kernel<BITS, G>;
    const size_t bytes = sizeof(GateUpShared) + ring;
    cudaError_t e = ensure_smem_limit<kernel>(bytes);
    if (e != cudaSuccess) return e;
    const int64_t items = static_cast<int64_t>(units + slots / kMoePass) * (a.w.inner / 16);
    const int64_t most = 2 * sm_count();
    kernel<<<static_cast<unsigned>(items < most ? items : most), kMoeThreads, bytes, stream>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  constexpr auto kernel = down_kernel<BITS, G>;
  const size_t bytes = sizeof(DownShared) + static_cast<size_t>(slots) * 128 + ring;
  const cudaError_t e = ensure_smem_limit<kernel>(bytes);
  if (e != cudaSuccess) return e;
  const int tiles = a.w.hidden / 32;
  int cluster = 1;
  while (cluster < kMoeMaxCluster && tiles * cluster < 2 * sm_count()) cluster *= 2;
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
  return cudaLaunchKernelEx(&cfg, kernel, a, cluster);
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
