// Page tables and slot maps of a serving step, built on the device from the
// requests' lengths: request b holds cached[b] tokens in its pages and gets
// new[b] more. With need(n) = ceil(n / page),
//   cu[b]    = sum of new[] before b                  (token offsets)
//   first[b] = sum of need(cached + new) - need(cached) before b
//   entry l of request b, need(cached) <= l < need(cached + new), becomes
//            free[first[b] + l - need(cached)]
//   token t of request b: position cached[b] + t - cu[b], slot page * size +
//            position % size.
//
// Bound by latency: two dependent global loads (lengths, then a table or
// free-list entry) around a scan. Every block scans all B lengths itself into
// shared memory (8 bytes per request), so blocks need nothing from one
// another, one launch does it all, and the rest is two binary searches in
// shared memory (GPU time: 64 requests with a token each 5 us, 500 prompts in 65536
// places 8). The entries a block reads (below need(cached)) and the
// entries any block writes (from there on) are disjoint.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "host_util.h"
#include "launch.h"

#define MATTN_API extern "C" __attribute__((visibility("default")))

namespace mattn {
namespace {

constexpr int kPlanThreads = 256;
// Tokens that a block more is worth: it scans the lengths once more. 65536 places for 4000
// requests: 512: 13.0 us, 1024: 14.2, 256: 19.4; 16000 with a token each: 16.3, 19.1, 14.9.
constexpr int kPlanTokens = 512;
constexpr int kPlanMaxB = 16384;   // 8 (B + 1) bytes of shared memory

struct PlanArgs {
  const int* cached;
  const int* fresh;
  int B;
  int* table;
  int per;
  const int* free_pages;
  int n_free;
  int shift;  // log2(page size)
  int* seq_lens;
  int* cu;
  long long* slots;
  int* positions;
  int* seq_ids;
  int cap;
  int* info;
};

__device__ __forceinline__ long long plan_pages(long long tokens, int shift, int per) {
  return min((tokens + (1ll << shift) - 1) >> shift, (long long)per);
}

__device__ __forceinline__ int clamp_int(long long x) {
  return x > INT_MAX ? INT_MAX : (int)x;
}

// The last i in [0, n) with a[i] <= x (a ascending, a[0] <= x).
__device__ __forceinline__ int last_at_most(const int* a, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PlanArgs p) {
  extern __shared__ int sh[];
  int* cu = sh;                // [B + 1]
  int* first = sh + p.B + 1;   // [B + 1]
  __shared__ long long warp_tok[kPlanThreads / 32], warp_pg[kPlanThreads / 32];
  __shared__ int over;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) over = 0;
  early_start();

  // exclusive scan: a thread sums its run of requests, warps scan the sums
  const int run = (p.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(tid * run, p.B), b1 = min(b0 + run, p.B);
  long long tok = 0, pg = 0;
  int n_over = 0;
  for (int b = b0; b < b1; ++b) {
    const long long c = max(p.cached[b], 0), n = max(p.fresh[b], 0);
    cu[b] = clamp_int(tok);
    first[b] = clamp_int(pg);
    tok += n;
    pg += plan_pages(c + n, p.shift, p.per) - plan_pages(c, p.shift, p.per);
    n_over += c + n > ((long long)p.per << p.shift);
  }
  long long tok_in = tok, pg_in = pg;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, tok_in, d);
    const long long b = __shfl_up_sync(0xffffffffu, pg_in, d);
    if (lane >= d) {
      tok_in += a;
      pg_in += b;
    }
  }
  if (lane == 31) {
    warp_tok[warp] = tok_in;
    warp_pg[warp] = pg_in;
  }
  __syncthreads();
  if (n_over) atomicAdd(&over, n_over);  // a count: no order matters
  long long tok_at = tok_in - tok, pg_at = pg_in - pg, tok_all = 0, pg_all = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) {
      tok_at += warp_tok[w];
      pg_at += warp_pg[w];
    }
    tok_all += warp_tok[w];
    pg_all += warp_pg[w];
  }
  for (int b = b0; b < b1; ++b) {
    cu[b] = clamp_int(cu[b] + tok_at);
    first[b] = clamp_int(first[b] + pg_at);
  }
  const int total = clamp_int(tok_all), pages = clamp_int(pg_all);
  if (tid == 0) {
    cu[p.B] = total;
    first[p.B] = pages;
  }
  __syncthreads();

  const int gtid = blockIdx.x * kPlanThreads + tid, gsize = gridDim.x * kPlanThreads;
  // tokens: owner, position, slot; past the last one all are -1
  for (long long t64 = gtid; t64 < p.cap; t64 += gsize) {
    const int t = (int)t64;
    long long slot = -1;
    int pos_out = -1, id = -1;
    if (t < total) {
      id = last_at_most(cu, p.B, t);
      const long long c = max(p.cached[id], 0);
      const long long pos = c + t - cu[id];
      pos_out = clamp_int(pos);
      const long long lp = pos >> p.shift;
      if (lp < p.per) {
        const long long have = plan_pages(c, p.shift, p.per);
        int page = -1;
        if (lp < have) {
          page = p.table[(size_t)id * p.per + lp];
        } else {
          const long long at = first[id] + (lp - have);
          if (at < p.n_free && MATTN_IN_BOUNDS(kSitePlan, at, p.n_free)) page = p.free_pages[at];
        }
        if (page >= 0) slot = ((long long)page << p.shift) + (pos & ((1ll << p.shift) - 1));
      }
    }
    p.slots[t] = slot;
    p.positions[t] = pos_out;
    p.seq_ids[t] = id;
  }
  // new page-table entries
  for (long long i64 = gtid; i64 < pages; i64 += gsize) {
    const int i = (int)i64;
    const int b = last_at_most(first, p.B, i);
    const long long lp = plan_pages(max(p.cached[b], 0), p.shift, p.per) + (i - first[b]);
    if (MATTN_IN_BOUNDS(kSitePlan, lp, p.per))
      p.table[(size_t)b * p.per + lp] = i < p.n_free ? p.free_pages[i] : -1;
  }
  for (int b = gtid; b <= p.B; b += gsize) {
    p.cu[b] = cu[b];
    if (b < p.B) p.seq_lens[b] = clamp_int((long long)max(p.cached[b], 0) + max(p.fresh[b], 0));
  }
  if (gtid == 0) {
    const int taken = min(pages, p.n_free);
    p.info[0] = total;
    p.info[1] = taken;
    p.info[2] = pages - taken;
    p.info[3] = over;
  }
}

}  // namespace
}  // namespace mattn

MATTN_API attn_status attn_page_plan(const int* cached_lens, const int* new_lens, int B,
                                     int* page_table, int pages_per_seq, int page_size,
                                     const int* free_pages, int num_free, int* seq_lens,
                                     int* cu_new, long long* slots, int* positions, int* seq_ids,
                                     int max_tokens, int* info, struct CUstream_st* stream) {
  using namespace mattn;
  if (B < 1 || pages_per_seq < 1 || num_free < 0 || max_tokens < 0) return ATTN_ERR_INVALID_ARG;
  int shift = 4;
  while (shift < 7 && (1 << shift) != page_size) ++shift;
  if ((1 << shift) != page_size || B > kPlanMaxB) return ATTN_ERR_UNSUPPORTED;
  if (!cached_lens || !new_lens || !page_table || !seq_lens || !cu_new || !info ||
      (num_free > 0 && !free_pages) || (max_tokens > 0 && (!slots || !positions || !seq_ids)))
    return ATTN_ERR_INVALID_ARG;
  const void* ints[] = {cached_lens, new_lens, page_table, free_pages, seq_lens,
                        cu_new, positions, seq_ids, info};
  for (const void* x : ints)
    if (reinterpret_cast<uintptr_t>(x) & 3) return ATTN_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(slots) & 7) return ATTN_ERR_MISALIGNED;
  // Every block reads the lengths, the free list and the table while others write:
  // what is written overlaps nothing.
  struct Range {
    const void* at;
    long long bytes;
  };
  const long long tokens = max_tokens, entries = (long long)B * pages_per_seq;
  const Range ranges[] = {{seq_lens, 4LL * B}, {cu_new, 4LL * B + 4}, {slots, 8 * tokens},
                          {positions, 4 * tokens}, {seq_ids, 4 * tokens}, {info, 16},
                          {page_table, 4 * entries}, {cached_lens, 4LL * B}, {new_lens, 4LL * B},
                          {free_pages, 4LL * num_free}};
  constexpr int kWritten = 7, kRanges = sizeof(ranges) / sizeof(ranges[0]);
  for (int i = 0; i < kWritten; ++i)
    for (int j = i + 1; j < kRanges; ++j) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(ranges[i].at);
      const uintptr_t b = reinterpret_cast<uintptr_t>(ranges[j].at);
      if (ranges[i].bytes && ranges[j].bytes && a < b + ranges[j].bytes && b < a + ranges[i].bytes)
        return ATTN_ERR_INVALID_ARG;
    }
  static DeviceOnce ready;
  const cudaError_t err = ready.allow_smem(page_plan_kernel, 2 * (kPlanMaxB + 1) * (int)sizeof(int));
  if (err != cudaSuccess) return cuda_status(err);
  const PlanArgs args{cached_lens, new_lens, B, page_table, pages_per_seq, free_pages, num_free,
                   shift, seq_lens, cu_new, slots, positions, seq_ids, max_tokens, info};
  const int blocks =
      std::max(1, std::min(2 * sm_count(), max_tokens / kPlanTokens + (max_tokens % kPlanTokens != 0)));
  return cuda_status(launch_early(page_plan_kernel, blocks, kPlanThreads, 2 * (B + 1) * sizeof(int),
                                  reinterpret_cast<cudaStream_t>(stream), args));
}

namespace mattn {
MATTN_DEBUG_RECORD_ACCESSORS(page_plan)
}  // namespace mattn
