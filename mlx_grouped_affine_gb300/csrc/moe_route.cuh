// Routing of a token by one warp: its top experts and their weights, from its logits.
// Shared by qmm_moe_route and by the plan of qmm_moe_layer.
#pragma once
#include "common.cuh"

namespace qmm {

// Logits in the order of unsigned integers: larger logits first, NaN as -infinity, the two
// zeros equal.  0 is below all of them (an expert that is taken, a place past the last).
__device__ __forceinline__ uint32_t logit_key(float l) {
  const uint32_t b = __float_as_uint(l != l ? -INFINITY : l + 0.0f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ float load_logit(const void *p, int type, int64_t at) {
  if (type == kTypeF32) return static_cast<const float *>(p)[at];
  const uint32_t h = static_cast<const uint16_t *>(p)[at];
  return type == kTypeBF16 ? bf16_bits_to_f32(h) : ElemF16::to_f32(h);
}

// 16-bit logits leave room for the expert in the same word, below the ordered pattern and
// counted down: one comparison then settles equal logits too.
__device__ __forceinline__ uint32_t packed_key(const void *p, int type, int64_t at, int expert) {
  const uint32_t h = static_cast<const uint16_t *>(p)[at], infinity = type == kTypeBF16 ? 0x7F80u : 0x7C00u;
  const uint32_t v = (h & 0x7FFFu) > infinity ? infinity | 0x8000u : h == 0x8000u ? 0u : h;  // NaN; -0
  return (v ^ (v & 0x8000u ? 0xFFFFu : 0x8000u)) << 16 | (0xFFFFu - static_cast<uint32_t>(expert));
}
template <bool PACKED>
__device__ __forceinline__ float logit_of(uint32_t key, int type) {
  if constexpr (!PACKED) return key_logit(key);
  const uint32_t o = key >> 16, h = o & 0x8000u ? o ^ 0x8000u : ~o & 0xFFFFu;
  return type == kTypeBF16 ? bf16_bits_to_f32(h) : ElemF16::to_f32(h);
}

// Sum over the warp, in an order that does not depend on anything.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

// The whole warp routes row `row`: lane j < top_k gets its j-th expert and that one's weight.
// NV = ceil(experts / 32), or more: expert 32 i + lane is entry i of a lane.
template <int NV, bool PACKED = false>
__device__ __forceinline__ void route_row(const Routing &r, int experts, int64_t row, int lane, int &id, float &weight) {
  uint32_t key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = 32 * i + lane;
    const int64_t at = row * experts + e;
    key[i] = e >= experts ? 0u : PACKED ? packed_key(r.logits, r.type, at, e) : logit_key(load_logit(r.logits, r.type, at));
  }
  float total = 1.0f, largest = 0.0f;
  uint32_t chosen = 0;
  id = 0;
  if (!r.sigmoid) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) m = max(m, key[i]);
    largest = logit_of<PACKED>(__reduce_max_sync(0xFFFFFFFFu, m), r.type);
    if (!r.normalize) {  // (the sum over all cancels where the chosen are divided by theirs)
      float part = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float l = logit_of<PACKED>(key[i], r.type);
        if (key[i] != 0u && l != -INFINITY) part += l == largest ? 1.0f : expf(l - largest);
      }
      total = warp_sum(part);
    }
  }
#pragma unroll 1
  for (int j = 0; j < r.top_k; ++j) {
    // the lane's first largest entry, the warp's largest, its lowest expert
    uint32_t best = 0, top, e;
    if constexpr (PACKED) {
#pragma unroll
      for (int i = 0; i < NV; ++i) best = max(best, key[i]);
      top = __reduce_max_sync(0xFFFFFFFFu, best);
      e = 0xFFFFu - (top & 0xFFFFu);
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] = key[i] == top ? 0u : key[i];
    } else {
      int at = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (key[i] > best) best = key[i], at = i;
      top = __reduce_max_sync(0xFFFFFFFFu, best);
      e = __reduce_min_sync(0xFFFFFFFFu, best == top ? 32u * at + lane : 0xFFFFu);
      if ((e & 31u) == static_cast<uint32_t>(lane)) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (i == static_cast<int>(e >> 5)) key[i] = 0;
      }
    }
    if (lane == j) id = static_cast<int>(e), chosen = top;
  }
  // softmax: exp(l - largest).  sigmoid: exp(min(l, 0)) / (1 + exp(-|l|)), and where they are
  // divided by their sum, exp(min(l, 0) - min(largest, 0)) in its place: those of logits below
  // -88 do not fit fp32, but their ratios do.  (With __expf, off by 2^-24 of its argument,
  // weights of logits spread by 10 are three times as far off, for 0.5 us of 8192 tokens over
  // 256 experts.)
  const float l = lane < r.top_k ? logit_of<PACKED>(chosen, r.type) : -INFINITY;
  if (r.sigmoid) {
    const float first = __shfl_sync(0xFFFFFFFFu, l, 0);
    largest = r.normalize ? fminf(first, 0.0f) : 0.0f;
  }
  float score = 0.0f;
  if (lane < r.top_k && l != -INFINITY) {
    const float x = r.sigmoid ? fminf(l, 0.0f) : l;
    score = x == largest ? 1.0f : expf(x - largest);
    if (r.sigmoid) score /= 1.0f + expf(-fabsf(l));
  }
  if (r.normalize) total = warp_sum(score);
  weight = total > 0.0f ? score / total * r.scale : 0.0f;
}

}  // namespace qmm
