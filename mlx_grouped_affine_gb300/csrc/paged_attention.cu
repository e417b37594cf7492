// qmm_paged_attention: which kernel serves a call.
#include "paged.cuh"
#include "workspace.h"

namespace qmm {

namespace paged {

cudaError_t key_map(const AttnArgs &a, int type, int rows, CUtensorMap *k) {
  const uint64_t dims[4] = {static_cast<uint64_t>(a.D), static_cast<uint64_t>(a.page),
                            static_cast<uint64_t>(a.Hkv), static_cast<uint64_t>(a.num_pages)};
  const uint64_t strides[3] = {static_cast<uint64_t>(a.token_stride) * 2, static_cast<uint64_t>(a.head_stride) * 2,
                               static_cast<uint64_t>(a.page_stride) * 2};
  const uint32_t box[4] = {64, static_cast<uint32_t>(rows), 1, 1};
  return encode_map_4d(k, type == kTypeF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                       a.k, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

cudaError_t query_map(const AttnArgs &a, int type, CUtensorMap *q) {
  const uint64_t dims[4] = {static_cast<uint64_t>(a.D), static_cast<uint64_t>(a.Hq), static_cast<uint64_t>(a.T), 1};
  const uint64_t token = static_cast<uint64_t>(a.q_stride) * 2;
  const uint64_t strides[3] = {static_cast<uint64_t>(a.D) * 2, token, token};
  const uint32_t box[4] = {64, static_cast<uint32_t>(a.Gs), static_cast<uint32_t>(a.TH), 1};
  return encode_map_4d(q, type == kTypeF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                       a.q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace paged

namespace {
constexpr size_t kDescBytes = 16 << 10;  // 32 bytes for each of up to 512 blocks
constexpr size_t kFewBytes = 12 << 20;   // region of the kernel of few rows
// Rows a kv head that it takes.  Measured, few / many kernel in us: 16 requests
// over 4000 keys 58 / 80 at 16 rows, 82 / 81 at 32, 173 / 83 at 64; one over 32000
// keys 35 / 50, 40 / 50, 64 / 50; 4 over 300 keys 14 / 23, 15 / 23, 18 / 25.
constexpr int kFewRows = 32;
}  // namespace

cudaError_t launch_paged_attention(const void *q, int64_t q_stride, int tokens, int q_heads,
                                   const PagedPool &pool, const int *table, int64_t table_stride,
                                   const int *starts, const int *seq, int requests, int64_t max_new,
                                   float scale, bool causal, int window, void *out,
                                   int64_t out_stride, float *lse, void *workspace,
                                   size_t workspace_bytes, cudaStream_t stream) {
  paged::AttnArgs a{};
  a.q = q;
  a.q_stride = q_stride;
  a.k = pool.k;
  a.v = pool.v;
  a.page_stride = pool.page_stride;
  a.head_stride = pool.head_stride;
  a.token_stride = pool.token_stride;
  a.table = table;
  a.table_stride = table_stride;
  a.starts = starts;
  a.seq = seq;
  a.out = out;
  a.out_stride = out_stride;
  a.lse = lse;
  a.err = device_error_word();
  if (!a.err) return cudaErrorInvalidSymbol;
  a.spin_limit = wait_limit();
  a.page = pool.page_size;
  a.num_pages = static_cast<int>(pool.num_pages);
  a.T = tokens;
  a.B = requests;
  a.Hq = q_heads;
  a.Hkv = pool.heads;
  a.G = q_heads / pool.heads;
  a.D = pool.head_dim;
  const int64_t keys = table_stride < 0x7FFFFFFF / pool.page_size ? table_stride * pool.page_size : 0x7FFFFFFF;
  a.max_keys = static_cast<int>(keys);
  a.causal = causal;
  a.window = window;
  a.scale_log2 = scale * paged::kLog2e;
  a.min_rows = 0;
  a.max_rows = 0x7FFFFFFF;
  // The workspace: block descriptors and pieces of cut items, a region for
  // each of the two kernels that a call may launch.  Its base here and the offsets of
  // regions, pieces and rows are multiples of 32 bytes, the prompt kernel's widest
  // store.
  static_assert(kDescBytes % kWorkspaceAlign == 0 && kFewBytes % kWorkspaceAlign == 0, "regions are aligned");
  const Workspace room = aligned_workspace(workspace, workspace_bytes);
  char *ws = room.base;
  auto region = [&](paged::AttnArgs &x, size_t at) {
    x.desc = reinterpret_cast<int *>(ws + at);
    x.ws = reinterpret_cast<float *>(ws + at + kDescBytes);
  };
  region(a, 0);
  if (pool.type == kTypeF32 || a.D > 128)
    return launch_attention_tiles(a, pool.type, room.bytes - kDescBytes, stream);
  // Few rows a kv head: the kernel of 16-row items, whose cost is the bytes of K
  // and V; many: the one of 256-row items, whose cost is the tensor pipe's.  The
  // second takes scores times a positive scale only.
  const int64_t most_rows = max_new * a.G;
  if (most_rows <= kFewRows || !(scale > 0.f))
    return launch_attention_decode(a, pool.type, kFewBytes - kDescBytes, stream);
  // Requests of both kinds: one kernel after the other, each leaving the other's
  // requests alone (63 single tokens over 100 to 8000 keys and 512 tokens over 8000: 266
  // us; each alone 170 and 83).  Not when no request can be of the first kind: a group
  // has more heads than that kernel takes rows, or there are more tokens than the other
  // requests can have.
  const bool few = requests > 1 && a.G <= kFewRows && tokens <= (requests - 1) * max_new + kFewRows / a.G;
  paged::AttnArgs many = a;
  region(many, kFewBytes);
  if (few) {
    a.max_rows = kFewRows;
    many.min_rows = kFewRows + 1;
    const cudaError_t e = launch_attention_decode(a, pool.type, kFewBytes - kDescBytes, stream);
    if (e != cudaSuccess) return e;
  }
  return launch_attention_prefill(many, pool.type, room.bytes - kFewBytes - kDescBytes, stream);
}

}  // namespace qmm
