// qmm_moe_experts and qmm_moe_layer: gated feed-forward of each token's experts.  The plan
// (routing, which slots go to which expert) and x's bf16 planes in one small kernel, then
// gate and up with silu, then down with the sum over a token's experts (moe_kernels.cuh).
//
// The plan is one block's work of a few microseconds, nearly all of it latency: misses of
// the instruction cache, one trip to memory for the logits, two warp reductions a choice.
// When every block of the expert kernels made its own plan instead, that was 24 000 cycles
// at the start of each of them (16 tokens of 8 experts); reading it takes 1 500.
#include "moe_kernels.cuh"
#include "moe_route.cuh"
#include "workspace.h"

namespace qmm {
namespace {

constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;

struct PlanShared {
  alignas(16) short expert[kMoeMaxSlots];  // of a slot; -1: no part in y
  short place[kMoeMaxSlots];               // among its expert's slots
  float weight[kMoeMaxSlots];
  int table[kMoeMaxExperts];               // of experts that have slots: the first in `list` | first unit << 16
  int part[kMoeMaxSlots / 32];
};

template <int NV>
__device__ __noinline__ void route_tokens(const Routing r, int tokens, int experts, PlanShared &p) {
  const int lane = threadIdx.x % 32;
  for (int t = threadIdx.x / 32; t < tokens; t += kPlanWarps) {
    int id;
    float weight;
    route_row<NV>(r, experts, t, lane, id, weight);
    if (lane < r.top_k) {
      p.expert[t * r.top_k + lane] = static_cast<short>(weight == 0.0f ? -1 : id);
      p.weight[t * r.top_k + lane] = weight;
    }
  }
}

__device__ void make_plan(const Routing r, const int tokens, const int experts, unsigned *err, PlanShared &p,
                          MoePlan *out) {
  const int slots = tokens * r.top_k, s = threadIdx.x, lane = s % 32;
  if (!r.logits) {
    if (s < slots) {
      int id = r.ids[s];
      const float weight = r.weights[s];
      if (id < 0 || id >= experts) {
        atomicOr(err, kErrIndexBit);
        id = -1;
      }
      p.expert[s] = static_cast<short>(weight == 0.0f ? -1 : id);
      p.weight[s] = weight;
    }
  } else if (experts <= 128) {
    route_tokens<4>(r, tokens, experts, p);
  } else if (experts <= 256) {
    route_tokens<8>(r, tokens, experts, p);
  } else {
    route_tokens<32>(r, tokens, experts, p);
  }
  if (s >= slots && s < (slots + 7) / 8 * 8) p.expert[s] = -1;
  __syncthreads();
  // Slots of the same expert, before this one and in all: every pair of slots is compared.
  // Then the scan over slots of (slots, units) that begin with each expert's first slot.
  int mine = 0, sum = 0;
  if (s / 32 * 32 < slots) {  // (whole warps)
    const int e = s < slots ? p.expert[s] : -1;
    int before = 0, all = 0;
    for (int o = 0; o < slots; o += 8) {
      const uint4 u = *reinterpret_cast<const uint4 *>(&p.expert[o]);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const bool same = static_cast<short>(w[k / 2] >> (16 * (k % 2))) == e;
        all += same;
        before += same && o + k < s;
      }
    }
    if (e >= 0) p.place[s] = static_cast<short>(before);
    if (e >= 0 && before == 0) mine = all | (all + kMoePass - 1) / kMoePass << 16;
    sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= d) sum += o;
    }
    if (lane == 31) p.part[s / 32] = sum;
  }
  __syncthreads();
  if (s / 32 * 32 < slots) {
    int at = sum - mine;
    for (int k = 0; k < s / 32; ++k) at += p.part[k];
    if (mine) {
      const int e = p.expert[s], n = mine & 0xFFFF, units = mine >> 16, unit = at >> 16;
      p.table[e] = at;
      for (int k = 0; k < units; ++k) {
        MoeEntry &u = out->entries[unit + k];
        u.unit_expert = static_cast<short>(e);
        u.unit_first = static_cast<short>((at & 0xFFFF) + k * kMoePass);
        u.unit_count = static_cast<short>(min(kMoePass, n - k * kMoePass));
      }
    }
    if (s / 32 == (slots - 1) / 32 && lane == 31) out->units = (at + mine) >> 16;
  }
  __syncthreads();
  if (s < slots) {
    const int e = p.expert[s], at = e < 0 ? 0 : p.table[e], place = e < 0 ? 0 : p.place[s];
    if (e >= 0) {
      out->entries[(at & 0xFFFF) + place].listed = static_cast<short>(s);
      out->entries[(at & 0xFFFF) + place].token = static_cast<short>(s / r.top_k);
    }
    // (unit and place side by side: the unit's first place is a multiple of kMoePass)
    out->entries[s].slot_unit = static_cast<short>(e < 0 ? -1 : (at >> 16) * kMoePass + place);
    out->entries[s].slot_weight = p.weight[s];
  }
}

// Block 0: the plan.  Block 1 + t (where x is not bf16): token t's row of x, cut into planes.
__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(const __grid_constant__ Routing r, int tokens, int experts, unsigned *err, MoePlan *plan,
            const void *__restrict__ x, int x_type, int hidden, uint16_t *__restrict__ planes, int64_t plane, int count) {
  __shared__ PlanShared shared;
  griddep_launch_dependents();
  if (blockIdx.x == 0) {
    make_plan(r, tokens, experts, err, shared, plan);
    return;
  }
  const int64_t row = static_cast<int64_t>(blockIdx.x - 1) * hidden;
  for (int i = threadIdx.x; i < hidden; i += kPlanThreads)
    store_planes(planes + row + i, plane, count, load_logit(x, x_type, row + i));
}

int64_t round128(int64_t n) { return (n + 127) / 128 * 128; }

}  // namespace

size_t moe_workspace_bytes(int64_t tokens, int64_t top_k, int64_t hidden, int64_t inner) {
  return static_cast<size_t>(kWorkspaceAlign + round128(sizeof(MoePlan)) + 2 * 3 * round128(tokens * hidden) +
                             2 * 3 * round128(tokens * top_k * inner));
}

cudaError_t launch_moe_experts(const void *x, int x_type, int tokens, const Routing &r, const ExpertWeights &w,
                               void *y, int y_type, void *workspace, size_t workspace_bytes,
                               cudaStream_t stream) {
  MoeArgs a;
  a.err = device_error_word();
  if (!a.err) return cudaErrorInvalidSymbol;
  const Workspace ws = aligned_workspace(workspace, workspace_bytes);
  MoePlan *plan = reinterpret_cast<MoePlan *>(ws.base);
  uint16_t *planes = reinterpret_cast<uint16_t *>(ws.base + round128(sizeof(MoePlan)));
  const int64_t n = static_cast<int64_t>(tokens) * w.hidden;
  a.route = r;
  a.w = w;
  a.tokens = tokens;
  a.y = y;
  a.y_type = y_type;
  a.plan = plan;
  a.wait_limit = wait_limit();
  a.code_scale = kCodeScale;
  a.x_plane = round128(n);
  a.x_planes = x_type == kTypeBF16 ? 1 : x_type == kTypeF16 ? 2 : 3;
  a.x = x_type == kTypeBF16 ? static_cast<const uint16_t *>(x) : planes;
  a.h = planes + 3 * a.x_plane;
  a.h_plane = round128(static_cast<int64_t>(tokens) * r.top_k * w.inner);
  // Two planes hold silu(gate) * up to 2^-18, well below y's own rounding where it has 16 bits
  // (2^-9 and 2^-12); the third costs down half as many products again.
  a.h_planes = y_type == kTypeF32 ? 3 : 2;
  plan_kernel<<<a.x == planes ? 1 + tokens : 1, kPlanThreads, 0, stream>>>(r, tokens, w.experts, a.err, plan, x, x_type, w.hidden,
                                                                           planes, a.x_plane, a.x_planes);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  switch (w.bits) {
    case 1:
    case 2: return launch_moe_bits_1_2(a, stream);
    case 3: return launch_moe_bits_3(a, stream);
    case 4: return launch_moe_bits_4(a, stream);
    case 5:
    case 6: return launch_moe_bits_5_6(a, stream);
    case 8: return launch_moe_bits_8(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace qmm
