// Block table, slot map and positions of a step, from request lengths.
//
// With pages(n) = ceil(n / P), request b needs pages(past + new) - pages(past)
// fresh pages; two prefix sums over the requests (new tokens, fresh pages)
// place its tokens in the step and its pages in the free list.  A token's
// position is past + i, its slot page * P + position % P, where the page is
// the table's (the request's open page) or comes from the free list directly:
// no token waits for a table entry that this call writes.
//
// One launch, no communication between blocks: every block computes the
// prefix sums of all requests (a few hundred bytes to some KB from L2) and
// then fills its own stretch of tokens and pages.  (Lengths updated in place: the
// blocks read past lengths all through the launch, so where there are several a
// second, small launch writes the new ones.)  The bytes are few; what it
// costs is the chain launch - lengths - scan - table or free entry - store:
// 4 us for 256 requests of a token each, 9 for 1000 requests with 256k tokens.
#include "paged.cuh"

namespace qmm {
namespace {

// Measured, 256 requests of one token / 1000 requests of 256k tokens: 256 threads
// 3.6 / 13.2 us, 512 4.2 / 9.3, 1024 6.1 / 8.4.
constexpr int NT = 512;

struct PlanArgs {
  const int *past, *fresh_tokens, *free_pages, *next_in;
  int *table, *starts, *seq, *positions, *slots, *next_out;
  int64_t table_stride;
  int requests, free_count, page, width, tokens;
  unsigned *err;
};

// Inclusive scans of two values a thread over the block, and their totals.
struct Pair {
  long long x, y;
};
__device__ __forceinline__ Pair scan_pair(Pair v, Pair *sums, Pair *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, v.x, d), y = __shfl_up_sync(0xffffffffu, v.y, d);
    if (lane >= d) {
      v.x += x;
      v.y += y;
    }
  }
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  Pair before{0, 0}, all{0, 0};
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const Pair s = sums[w];
    if (w < warp) {
      before.x += s.x;
      before.y += s.y;
    }
    all.x += s.x;
    all.y += s.y;
  }
  *total = all;
  return Pair{before.x + v.x, before.y + v.y};
}

// The last of the n ascending values that is <= key (the first is).
__device__ __forceinline__ int last_at_most(const long long *v, int n, long long key) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] <= key) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Request b's lengths before and after the step; nothing past what positions can
// count or the table's rows can hold.  (Plain loads: `past` may be `seq`, which the
// same thread writes afterwards.)
struct Lengths {
  int past, len;
  bool bad;
};
__device__ __forceinline__ Lengths lengths_of(const PlanArgs &a, int b) {
  const int p = a.past[b], n = a.fresh_tokens[b];
  const long long most = min(static_cast<long long>(a.width) * a.page, 0x7FFFFFFFll);
  const long long past = max(p, 0), len = past + max(n, 0);
  return Lengths{static_cast<int>(min(past, most)), static_cast<int>(min(len, most)), p < 0 || n < 0 || len > most};
}

__global__ void __launch_bounds__(NT) page_plan_kernel(PlanArgs a) {
  __shared__ Pair sums[NT / 32];
  __shared__ long long first_token[NT], first_page[NT];
  __shared__ int past_of[NT];
  const int tid = threadIdx.x;
  const unsigned P = a.page;
  const int raw_next = a.next_in ? __ldg(a.next_in) : 0;
  const long long next = max(raw_next, 0);
  bool bad = raw_next < 0;
  long long tokens_before = 0, pages_before = 0;

  for (int base = 0; base < a.requests; base += NT) {
    const int b = base + tid;
    Pair mine{0, 0};
    int past = 0;
    if (b < a.requests) {
      const Lengths x = lengths_of(a, b);
      bad |= x.bad;
      past = x.past;
      mine.x = x.len - x.past;
      mine.y = (x.len + static_cast<long long>(P) - 1) / P - (x.past + static_cast<long long>(P) - 1) / P;
      if (blockIdx.x == 0 && a.seq) a.seq[b] = x.len;
    }
    Pair total;
    const Pair incl = scan_pair(mine, sums, &total);
    first_token[tid] = tokens_before + incl.x - mine.x;
    first_page[tid] = pages_before + incl.y - mine.y;
    past_of[tid] = past;
    if (blockIdx.x == 0 && b < a.requests) {
      // Requests past the step's room keep their place at its end.
      a.starts[b] = static_cast<int>(min(first_token[tid], static_cast<long long>(a.tokens)));
      if (b == a.requests - 1) {
        const long long all = tokens_before + incl.x;
        a.starts[a.requests] = static_cast<int>(min(all, static_cast<long long>(a.tokens)));
        bad |= all > a.tokens;
      }
    }
    __syncthreads();
    const int here = min(NT, a.requests - base);
    // Fresh pages of these requests, in this block's share.
    for (long long j = blockIdx.x * static_cast<long long>(NT) + tid; j < total.y;
         j += static_cast<long long>(gridDim.x) * NT) {
      const long long g = pages_before + j;
      const int e = last_at_most(first_page, here, g);
      const long long held = (past_of[e] + static_cast<long long>(P) - 1) / P;
      const long long at = next + g;
      bad |= at >= a.free_count;
      a.table[(base + e) * a.table_stride + held + (g - first_page[e])] =
          at < a.free_count ? __ldg(a.free_pages + at) : -1;
    }
    // Tokens of these requests, in this block's share.
    const long long t1 = min(tokens_before + total.x, static_cast<long long>(a.tokens));
    for (long long t = tokens_before + blockIdx.x * static_cast<long long>(NT) + tid; t < t1;
         t += static_cast<long long>(gridDim.x) * NT) {
      const int e = last_at_most(first_token, here, t);
      const unsigned pos = past_of[e] + static_cast<unsigned>(t - first_token[e]);
      const unsigned pg = pos / P;
      const unsigned held = (static_cast<unsigned>(past_of[e]) + P - 1) / P;
      int id;
      if (pg < held) {
        id = __ldg(a.table + (base + e) * a.table_stride + pg);
      } else {
        const long long at = next + first_page[e] + (pg - held);
        id = at < a.free_count ? __ldg(a.free_pages + at) : -1;
      }
      const long long slot = static_cast<long long>(id) * P + (pos - pg * P);
      const bool fits = id >= 0 && slot <= 0x7FFFFFFFll;
      bad |= !fits;
      a.positions[t] = static_cast<int>(pos);
      a.slots[t] = fits ? static_cast<int>(slot) : -1;
    }
    tokens_before += total.x;
    pages_before += total.y;
    __syncthreads();
  }
  // Room past the last token: no position, no slot.
  for (long long t = tokens_before + blockIdx.x * static_cast<long long>(NT) + tid; t < a.tokens;
       t += static_cast<long long>(gridDim.x) * NT) {
    a.positions[t] = 0;
    a.slots[t] = -1;
  }
  if (blockIdx.x == 0 && tid == 0) {
    if (a.requests == 0) a.starts[0] = 0;
    *a.next_out = static_cast<int>(max(next, min(next + pages_before, static_cast<long long>(a.free_count))));
  }
  if (bad) atomicOr(a.err, kErrIndexBit);
}

__global__ void __launch_bounds__(NT) lengths_in_place_kernel(PlanArgs a) {
  const long long b = blockIdx.x * static_cast<long long>(NT) + threadIdx.x;
  if (b < a.requests) a.seq[b] = lengths_of(a, static_cast<int>(b)).len;
}

}  // namespace

cudaError_t launch_page_plan(const int *past, const int *fresh, int requests, const int *free_pages,
                             int free_count, const int *next_in, int page, int *table,
                             int64_t table_stride, int tokens, int *starts, int *seq, int *positions,
                             int *slots, int *next_out, cudaStream_t stream) {
  PlanArgs a{past, fresh, free_pages, next_in, table, starts, seq, positions, slots, next_out,
             table_stride, requests, free_count, page,
             static_cast<int>(table_stride < 0x7FFFFFFF ? table_stride : 0x7FFFFFFF), tokens,
             device_error_word()};
  if (!a.err) return cudaErrorInvalidSymbol;
  int64_t blocks = (static_cast<int64_t>(tokens) + NT - 1) / NT;
  if (blocks > sm_count()) blocks = sm_count();
  if (blocks < 1) blocks = 1;
  // In place, a single block's thread reads a length before it writes it.
  const bool later = seq == past && blocks > 1;
  if (later) a.seq = nullptr;
  page_plan_kernel<<<static_cast<unsigned>(blocks), NT, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (!later || e != cudaSuccess) return e;
  a.seq = seq;
  lengths_in_place_kernel<<<static_cast<unsigned>((static_cast<int64_t>(requests) + NT - 1) / NT), NT, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace qmm
