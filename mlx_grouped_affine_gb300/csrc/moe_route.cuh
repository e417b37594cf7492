// Routing of a token by one warp: its top experts and their weights, from its logits.
// Shared by qmm_moe_route and by the expert kernels, which route for themselves.
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

// Sum over the warp, in an order that does not depend on anything.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

// The whole warp routes row `row`.  Lane j < top_k returns the row's j-th expert and its
// weight.  NV = ceil(experts / 32), or more: expert 32 i + lane is entry i of a lane.
template <int NV>
__device__ __forceinline__ void route_row(const Routing &r, int experts, int64_t row, int lane,
                                          int &id, float &weight) {
  uint32_t key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = 32 * i + lane;
    key[i] = e < experts ? logit_key(load_logit(r.logits, r.type, row * experts + e)) : 0u;
  }
  float total = 1.0f, largest = 0.0f;
  if (!r.sigmoid) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) m = max(m, key[i]);
    largest = key_logit(__reduce_max_sync(0xFFFFFFFFu, m));
    if (!r.normalize) {  // (the sum over all cancels where the chosen are divided by theirs)
      float part = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float l = key_logit(key[i]);
        if (key[i] != 0u && l != -INFINITY) part += l == largest ? 1.0f : __expf(l - largest);
      }
      total = warp_sum(part);
    }
  }
  uint32_t chosen = 0;
  id = 0;
  for (int j = 0; j < r.top_k; ++j) {
    // the lane's first largest entry, the warp's largest, its lowest expert
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (key[i] > best) best = key[i], at = i;
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
    const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, best == top ? 32u * at + lane : 0xFFFFu);
    if ((e & 31u) == static_cast<uint32_t>(lane)) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i == static_cast<int>(e >> 5)) key[i] = 0;
    }
    if (lane == j) id = static_cast<int>(e), chosen = top;
  }
  const float l = key_logit(chosen);
  float score = 0.0f;
  // Sigmoids that are divided by their sum are taken relative to the largest of them, as
  // exponentials of log sigmoid(l) = min(l, 0) - log(1 + exp(-|l|)): those of logits below
  // -88 do not fit fp32, but their ratios do.
  const bool relative = r.sigmoid && r.normalize;
  // (Few instructions: an expert kernel runs them once a block, each line of them a miss of
  // the instruction cache.  __expf is off by 2^-21 and 2^-24 of its argument.)
  float x = l;
  if (relative) {
    x = fminf(l, 0.0f) - log1pf(__expf(-fabsf(l)));
    largest = __shfl_sync(0xFFFFFFFFu, x, 0);
  }
  if (lane < r.top_k && l != -INFINITY) {
    const bool alone = r.sigmoid && !relative;
    score = alone || x != largest ? __expf(alone ? -l : x - largest) : 1.0f;
    if (alone) score = __fdividef(1.0f, 1.0f + score);
  }
  if (r.normalize) total = warp_sum(score);
  weight = total > 0.0f ? __fdividef(score, total) * r.scale : 0.0f;
}

}  // namespace qmm
