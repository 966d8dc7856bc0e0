// Eviction from the bf16 paged cache by accumulated attention weight: of every (sequence,
// key/value head)'s keys the first `first`, the last `recent` and the heaviest of those between
// stay, keep in all beside the first; their rows move together, in order.
//
// Two kernels. The first finds, per pair, the kept keys: the key of rank keep - recent in the
// order (weight descending, index ascending) by a radix selection on the weights' bits (ordered
// as unsigned numbers; 11, 11 and 10 bits, so that three histograms of the weights, staged in
// shared memory, give it exactly), then an ascending list of those above it. Bound by latency: a
// pair's candidates are dealt out to a cluster of up to eight blocks, each of which adds up the
// histograms of all by 16-byte reads of their shared memory.
//
// The second moves the rows. HBM is the bound: every kept row is read and written once. In
// place, kept key m's row goes from kept[m] to first + m <= kept[m], so in ascending batches
// no write reaches a later batch's source; inside a batch all rows are read before one is
// written (a barrier). A block therefore owns some channels of one pair's K or V rows from the
// first batch to the last, alone or with the others of its cluster, behind the cluster's barrier.
// The next batch's rows are read while the last one's are written, and the places of the one
// after it are looked up meanwhile, one row per thread. Into other pages no order is needed and
// batches are dealt out too; there this kernel's first blocks list the pages that go, which takes
// the tables' entries.
//
// 8 sequences of 32768 keys, 8 heads of 128 channels, 8192 kept: 125 us, 4.4 TB/s of the 545 MB
// that must move; into other pages 116. 32 of 8000, 4000 kept: 200 us, 5.3 TB/s. Rows in flight are the bound: with half
// of them per block (2 pieces per thread, or 128 threads) 158 and 250 us.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "common.cuh"
#include "host_util.h"
#include "launch.h"

#define MATTN_API extern "C" __attribute__((visibility("default")))

namespace mattn {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelStaged = 48 * 1024;  // weights of a block that are staged (4 bytes each)
constexpr int kSelBins = 2048;
constexpr int kSelOwnBins = kSelBins / kSelThreads;
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;  // 16-byte pieces of a thread in flight
constexpr int kMoveBlocks = 4;  // blocks per SM
constexpr int kMaxCluster = 8;  // blocks of a cluster, on any device

struct EvictArgs {
  const float* weights;
  float* weights_out;
  const int* seq_lens;
  const int* starts;  // or nullptr: sink
  int sink, keep, recent;
  char* k;
  char* v;
  const int* table;
  const int* new_table;  // or nullptr: in place
  int per, new_per;
  int B, Hkv, max_len, shift, num_pages, stride;
  int row_bytes;
  int* kept;  // [B][Hkv][keep]
  int* new_lens;
  int* freed;
  int max_freed;
  int* info;
  int select_cluster;  // blocks of a pair in the selection
  int move_cluster;    // blocks that share the batches of a move in place
  int splits, piece;   // the move: parts of a row of `piece` bytes
  int chunks;          // the move into other pages: runs of positions
  int lists, list_run; // blocks that list the freed pages first, sequences of each
};

struct EvictSeq {
  int len, first, held;  // keys, those that stay in front, those of the others that stay
  bool cut;
  __device__ __forceinline__ int new_len() const { return first + held; }
};

__device__ __forceinline__ EvictSeq evict_seq(const EvictArgs& a, int b) {
  EvictSeq s;
  s.len = max(0, min(a.seq_lens[b], a.max_len));
  s.first = max(0, min(a.starts ? a.starts[b] : a.sink, s.len));
  s.cut = s.len - s.first > a.keep;
  s.held = min(s.len - s.first, a.keep);
  return s;
}

// Pages of a sequence that it no longer uses: entries [stay, have) of its table row, but for those
// that a new table keeps (evict_list).
__device__ __forceinline__ int2 evict_pages(const EvictArgs& a, const EvictSeq& s) {
  const int up = (1 << a.shift) - 1;
  const int have = (s.len + up) >> a.shift;
  const int stay = a.new_table ? s.first >> a.shift : (s.new_len() + up) >> a.shift;
  return make_int2(stay, have);
}

// A weight's bits as a number that grows with it: NaN above all, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(uint32_t u) {
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  if (u == 0x80000000u) u = 0;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// All threads of the cluster: what they read and wrote before lies before what any does after.
__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::
          : "memory");
}

// The same for the blocks that share a pair's batches, or the threads of the one that has them.
__device__ __forceinline__ void ranks_sync(int ranks) {
  if (ranks > 1)
    cluster_sync();
  else
    __syncthreads();
}

// The int at the same place in the shared memory of the cluster's block `rank`, and four of them.
__device__ __forceinline__ int cluster_read(const int* p, int rank) {
  uint32_t at;
  int x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
  return x;
}

__device__ __forceinline__ int4 cluster_read4(const int* p, int rank) {
  uint32_t at;
  int4 x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "r"(at)
               : "memory");
  return x;
}

// Sum over the block of `mine`, and of those of the threads before: by a scan of warp sums.
template <int WARPS = kSelWarps>
__device__ __forceinline__ int block_before(int mine, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += o;
  }
  __syncthreads();  // warp_sums of an earlier call have been read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int w = lane < WARPS ? warp_sums[lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += o;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  return x - mine + (warp ? before : 0);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  extern __shared__ uint32_t staged[];
  __shared__ alignas(16) int hist[3][kSelBins];
  __shared__ int sums[kSelWarps], equals[kSelWarps];
  __shared__ int found_bin, found_above, count[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ranks = a.select_cluster, pair = blockIdx.x / ranks, rank = blockIdx.x % ranks;
  const int b = pair / a.Hkv, h = pair % a.Hkv;
  early_start();
  const EvictSeq s = evict_seq(a, b);
  if (h == 0 && rank == 0) {  // the sequence's length and, in place, its pages that go
    if (tid == 0) a.new_lens[b] = s.new_len();
  }
  if (h == 0 && rank == 0 && !a.new_table) {
    int gone = 0, cuts = 0, total, all_cuts;
    const int upto = b == a.B - 1 ? a.B : b;
    for (int i = tid; i < upto; i += kSelThreads) {
      const EvictSeq o = evict_seq(a, i);
      const int2 pages = evict_pages(a, o);
      if (i < b) gone += max(0, pages.y - pages.x);
      cuts += o.cut;
    }
    block_before(gone, sums, total);
    block_before(cuts, sums, all_cuts);
    const int2 pages = evict_pages(a, s);
    const int n = max(0, pages.y - pages.x);
    for (int i = tid; i < n; i += kSelThreads)
      if (total + i < a.max_freed && MATTN_IN_BOUNDS(kSiteEvict, pages.x + i, a.per))
        a.freed[total + i] = a.table[(size_t)b * a.per + pages.x + i];
    if (tid == 0 && b == a.B - 1) {
      a.info[0] = total + n;
      a.info[1] = all_cuts;
    }
  }
  int* kept = a.kept + (size_t)pair * a.keep;
  const int each = rank * kSelThreads + tid, all = ranks * kSelThreads;
  if (!s.cut) {
    for (int m = each; m < a.keep; m += all) kept[m] = m < s.held ? s.first + m : -1;
    return;
  }
  const int cands = s.len - s.first - a.recent, k = a.keep - a.recent;  // k of them stay
  for (int m = each; m < a.recent; m += all) kept[k + m] = s.len - a.recent + m;
  if (k == 0) return;
  // this block's candidates
  const int begin = (int)((long long)cands * rank / ranks);
  const int c = (int)((long long)cands * (rank + 1) / ranks) - begin;
  const uint32_t* w =
      reinterpret_cast<const uint32_t*>(a.weights + (size_t)pair * a.stride + s.first + begin);
  const bool stage = c <= kSelStaged;
  if (stage)
    for (int i = tid; i < c; i += kSelThreads) staged[i] = weight_key(w[i]);
  auto key_at = [&](int i) { return stage ? staged[i] : weight_key(w[i]); };
  for (int i = tid; i < 3 * kSelBins; i += kSelThreads) (&hist[0][0])[i] = 0;
  __syncthreads();

  // The threshold: the largest key that at least k candidates reach, digit by digit.
  uint32_t prefix = 0, mask = 0;
  int left = k;  // candidates to take among those that share the prefix
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digits = pass == 2 ? 1023u : 2047u;
    for (int i0 = warp * 32; i0 < c; i0 += kSelThreads) {
      const int i = i0 + lane;
      int bin = -1;
      if (i < c) {
        const uint32_t key = key_at(i);
        if ((key & mask) == prefix) bin = (int)((key >> shift) & digits);
      }
      // equal weights are common (keys that no row looked at): one add for a whole warp
      int same;
      __match_all_sync(0xffffffffu, bin, &same);
      if (same) {
        if (lane == 0 && bin >= 0) atomicAdd(&hist[pass][bin], 32);
      } else if (bin >= 0) {
        atomicAdd(&hist[pass][bin], 1);
      }
    }
    cluster_sync();
    // from the largest digit down: thread t holds the four bins down from hi
    static_assert(kSelOwnBins == 4, "one 16-byte word of bins per thread");
    const int hi = kSelBins - 1 - kSelOwnBins * tid;
    int n[kSelOwnBins] = {};
#pragma unroll 4
    for (int r = 0; r < ranks; ++r) {
      // (every block begins with its own bins, so that they do not all ask the same one)
      const int4 x = cluster_read4(&hist[pass][hi - 3], (rank + r) & (ranks - 1));
      n[0] += x.w;
      n[1] += x.z;
      n[2] += x.y;
      n[3] += x.x;
    }
    int total;
    int above = block_before(n[0] + n[1] + n[2] + n[3], sums, total);
#pragma unroll
    for (int e = 0; e < kSelOwnBins; ++e) {
      if (above < left && left <= above + n[e]) {
        found_bin = hi - e;
        found_above = above;
      }
      above += n[e];
    }
    __syncthreads();
    left -= found_above;
    prefix |= (uint32_t)found_bin << shift;
    mask |= digits << shift;
  }

  // The list, ascending: every warp counts a run of candidates, then writes its part.
  const int lo = (int)((long long)c * warp / kSelWarps);
  const int hi = (int)((long long)c * (warp + 1) / kSelWarps);
  int above = 0, equal = 0;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t key = i < hi ? key_at(i) : 0u;
    above += __popc(__ballot_sync(0xffffffffu, i < hi && key > prefix));
    equal += __popc(__ballot_sync(0xffffffffu, i < hi && key == prefix));
  }
  __syncthreads();
  if (lane == 0) {
    sums[warp] = above;
    equals[warp] = equal;
  }
  __syncthreads();
  above = equal = 0;
  for (int i = 0; i < warp; ++i) {
    above += sums[i];
    equal += equals[i];
  }
  if (tid == kSelThreads - 1) {  // the block's, for those of the blocks behind it
    count[0] = above + sums[warp];
    count[1] = equal + equals[warp];
  }
  cluster_sync();
  for (int r = 0; r < rank; ++r) {
    above += cluster_read(&count[0], r);
    equal += cluster_read(&count[1], r);
  }
  const uint32_t below = (1u << lane) - 1u;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t key = i < hi ? key_at(i) : 0u;
    const uint32_t gt = __ballot_sync(0xffffffffu, i < hi && key > prefix);
    const uint32_t eq = __ballot_sync(0xffffffffu, i < hi && key == prefix);
    const int g = above + __popc(gt & below), e = equal + __popc(eq & below);
    const bool take = (gt >> lane & 1) || ((eq >> lane & 1) && e < left);
    const int m = g + min(e, left);
    if (take && MATTN_IN_BOUNDS(kSiteEvict, m, a.keep)) kept[m] = s.first + begin + i;
    above += __popc(gt);
    equal += __popc(eq);
  }
  cluster_sync();  // no block ends while others read its shared memory
}

constexpr uint32_t kNoRow = 0xffffffffu;

// Row of the pool (counted over all pages and heads) that a head's key at a position of sequence
// b has, or kNoRow outside the pool.
__device__ __forceinline__ uint32_t evict_row(const EvictArgs& a, const int* table, int per, int b,
                                              int h, int pos) {
  const int lp = pos >> a.shift;
  if (lp >= per || !MATTN_IN_BOUNDS(kSiteEvict, lp, per)) return kNoRow;
  const int page = table[(size_t)b * per + lp];
  if (page < 0 || page >= a.num_pages) return kNoRow;
  return (((uint32_t)page * a.Hkv + h) << a.shift) + (pos & ((1 << a.shift) - 1));
}

// Where a key's row comes from and goes to; equal: it stays.
__device__ __forceinline__ uint2 evict_way(const EvictArgs& a, const EvictSeq& s, const int* kept,
                                           int b, int h, int n, int to) {
  if (n >= to) return make_uint2(kNoRow, kNoRow);
  const int src = n < s.first || !s.cut ? n : kept[n - s.first];
  if (!a.new_table && src == n) return make_uint2(kNoRow, kNoRow);
  const uint32_t dst = evict_row(a, a.new_table ? a.new_table : a.table,
                                 a.new_table ? a.new_per : a.per, b, h, n);
  return make_uint2(evict_row(a, a.table, a.per, b, h, src), dst);
}

// With a new table: the pages that go, of list_run sequences from b on. An entry that the new table
// has in the same place, among those that it still uses, stays; so those of the sequences before
// are counted entry by entry.
__device__ __noinline__ void evict_list(const EvictArgs& a, int b) {
  constexpr int kWarps = kMoveThreads / 32;
  __shared__ int sums[kWarps];
  const int tid = threadIdx.x;
  auto named = [&](const EvictSeq& s) {
    return min(a.new_per, (s.new_len() + (1 << a.shift) - 1) >> a.shift);
  };
  auto same = [&](int i, int page) {
    return MATTN_IN_BOUNDS(kSiteEvict, page, a.per) &&
           a.new_table[(size_t)i * a.new_per + page] == a.table[(size_t)i * a.per + page];
  };
  const int end = min(b + a.list_run, a.B), upto = end == a.B ? a.B : b;
  int team = 1;  // threads of a sequence: as many as there are, up to a warp
  while (team < 32 && 2 * team * upto <= kMoveThreads) team *= 2;
  int gone = 0, cuts = 0, at, all_cuts;
  for (int i = tid / team; i < upto; i += kMoveThreads / team) {
    const EvictSeq s = evict_seq(a, i);
    const int2 pages = evict_pages(a, s);
    if (tid % team == 0) cuts += s.cut;
    if (i >= b) continue;
    if (tid % team == 0) gone += pages.y - pages.x;
    const int to = named(s);
#pragma unroll 4
    for (int p = pages.x + tid % team; p < to; p += team) gone -= same(i, p);
  }
  block_before<kWarps>(gone, sums, at);
  block_before<kWarps>(cuts, sums, all_cuts);
  for (int i = b; i < end; ++i) {
    const EvictSeq s = evict_seq(a, i);
    const int2 pages = evict_pages(a, s);
    const int to = named(s);
    for (int p0 = pages.x; p0 < pages.y; p0 += kMoveThreads) {
      const int p = p0 + tid;
      const bool goes = p < pages.y && !(p < to && same(i, p));
      int n;
      const int place = at + block_before<kWarps>(goes, sums, n);
      if (goes && place < a.max_freed && MATTN_IN_BOUNDS(kSiteEvict, p, a.per))
        a.freed[place] = a.table[(size_t)i * a.per + p];
      at += n;
    }
  }
  if (tid == 0 && end == a.B) {
    a.info[0] = at;
    a.info[1] = all_cuts;
  }
}

__global__ void __launch_bounds__(kMoveThreads, kMoveBlocks) evict_move_kernel(const EvictArgs a) {
  __shared__ uint2 ways[2][kMoveThreads];  // of a batch's rows: at most kMoveThreads
  early_start();
  if ((int)blockIdx.x < a.lists) return evict_list(a, blockIdx.x * a.list_run);
  const int ranks = a.move_cluster, block = blockIdx.x - a.lists;
  const int rank = block % ranks, unit = block / ranks;
  const int parts = 2 * a.splits * a.chunks + 1;
  const int pair = unit / parts, part = unit % parts;
  const int b = pair / a.Hkv, h = pair % a.Hkv;
  const EvictSeq s = evict_seq(a, b);
  const int* kept = a.kept + (size_t)pair * a.keep;
  const int end = s.new_len();
  const int tid = threadIdx.x;
  if (part == parts - 1) {  // the weights; where they went from is 0
    const float* in = a.weights + (size_t)pair * a.stride;
    float* out = a.weights_out + (size_t)pair * a.stride;
    const int each = rank * kMoveThreads + tid, all = ranks * kMoveThreads;
    for (int n0 = 0; n0 < end; n0 += all * kMoveUnroll) {
      float x[kMoveUnroll];
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        const int n = n0 + u * all + each;
        x[u] = n < end ? in[n < s.first || !s.cut ? n : kept[n - s.first]] : 0.0f;
      }
      ranks_sync(ranks);
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        const int n = n0 + u * all + each;
        if (n < end) out[n] = x[u];
      }
    }
    for (int n = end + each; n < s.len; n += all) out[n] = 0.0f;
    return;
  }
  const bool in_place = a.new_table == nullptr;
  if (in_place && !s.cut) return;
  char* pool = part & 1 ? a.v : a.k;
  const int split = (part >> 1) % a.splits, chunk = (part >> 1) / a.splits;
  const int lanes = a.piece / 16;  // threads of a row
  const int row = tid / lanes, rows = kMoveThreads / lanes, own = rows * kMoveUnroll;
  const int col = split * a.piece + tid % lanes * 16;
  const int batch = own * ranks;
  int from = s.first, to = end;
  if (!in_place) {  // all pages from the first that holds a key that may go, in runs
    from = s.first >> a.shift << a.shift;
    const int batches = (end - from + batch - 1) / batch;
    const int lo = from + (int)((long long)batches * chunk / a.chunks) * batch;
    to = min(end, from + (int)((long long)batches * (chunk + 1) / a.chunks) * batch);
    from = lo;
  }
  [[maybe_unused]] const long long bytes = ((long long)a.num_pages * a.Hkv << a.shift) * a.row_bytes;
  const int mine = from + rank * own + tid;  // thread t < own looks up row t of the block's
  auto way = [&](int n0) {
    return tid < own ? evict_way(a, s, kept, b, h, n0 + mine - from, to) : make_uint2(kNoRow, kNoRow);
  };
  uint4 x[kMoveUnroll];
  uint32_t dst[kMoveUnroll];
  auto load = [&](const uint2* ways, uint4 (&x)[kMoveUnroll], uint32_t (&dst)[kMoveUnroll]) {
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const uint2 way = ways[u * rows + row];
      x[u] = make_uint4(0, 0, 0, 0);
      dst[u] = way.x == way.y ? kNoRow : way.y;
      if (dst[u] != kNoRow && way.x != kNoRow) {
        const size_t at = (size_t)way.x * a.row_bytes + col;
        if (MATTN_IN_BOUNDS(kSiteEvictRow, at + 15, bytes))
          x[u] = *reinterpret_cast<const uint4*>(pool + at);
      }
    }
  };
  ways[0][tid] = way(from);
  ways[1][tid] = way(from + batch);
  __syncthreads();
  load(ways[0], x, dst);
  int turn = 0;
  for (int n0 = from; n0 < to; n0 += batch, turn ^= 1) {
    const uint2 later = way(n0 + 2 * batch);
    ranks_sync(ranks);  // every row of the batch is read before one is written
    uint4 next[kMoveUnroll];
    uint32_t next_dst[kMoveUnroll];
    load(ways[turn ^ 1], next, next_dst);
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const size_t at = (size_t)dst[u] * a.row_bytes + col;
      if (dst[u] != kNoRow && MATTN_IN_BOUNDS(kSiteEvictRow, at + 15, bytes))
        *reinterpret_cast<uint4*>(pool + at) = x[u];
      x[u] = next[u];
      dst[u] = next_dst[u];
    }
    ways[turn][tid] = later;
  }
}

bool overlap(const void* p, size_t n, const void* q, size_t m) {
  const char *a = static_cast<const char*>(p), *b = static_cast<const char*>(q);
  return p && q && n && m && a < b + m && b < a + n;
}

}  // namespace
}  // namespace mattn

MATTN_API attn_status attn_cache_evict(const float* weights, float* weights_out, int weights_stride,
                                       const int* seq_lens, const int* starts, int sink, int keep,
                                       int recent, void* k, void* v, int num_pages, int page_size,
                                       const int* page_table, int pages_per_seq,
                                       const int* new_table, int new_pages_per_seq, int B, int Hkv,
                                       int max_len, int D, int* kept, int* new_lens, int* freed,
                                       int max_freed, int* info, struct CUstream_st* stream) {
  using namespace mattn;
  if (B < 0 || Hkv < 1 || max_len < 0 || sink < 0 || keep < 1 || recent < 0 || recent > keep ||
      max_freed < 0 || weights_stride < max_len || num_pages < 1 || pages_per_seq < 1)
    return ATTN_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
    return ATTN_ERR_UNSUPPORTED;
  if ((long long)pages_per_seq * page_size < (long long)max_len) return ATTN_ERR_INVALID_ARG;
  if (new_table && new_pages_per_seq < 1) return ATTN_ERR_INVALID_ARG;
  const long long pairs = (long long)B * Hkv;
  if (pairs > 65535 || B > 16384 || max_len > INT_MAX - 65536 ||
      (long long)sink + keep > INT_MAX - 65536)
    return ATTN_ERR_UNSUPPORTED;
  // the freed pages are counted in an int
  if ((long long)B * pages_per_seq > INT_MAX) return ATTN_ERR_UNSUPPORTED;
  // rows of a pool are counted in 32 bits, the largest number meaning none
  if ((long long)num_pages * Hkv * page_size > 0xffffffffLL) return ATTN_ERR_UNSUPPORTED;
  if (B == 0) return ATTN_OK;
  if (!weights || !weights_out || !seq_lens || !k || !v || !page_table || !kept || !new_lens ||
      !info || (max_freed > 0 && !freed))
    return ATTN_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15u)
    return ATTN_ERR_MISALIGNED;
  const void* words[] = {weights,    weights_out, seq_lens, starts, page_table,
                         new_table, kept,        new_lens, freed,  info};
  for (const void* x : words)
    if (reinterpret_cast<uintptr_t>(x) & 3u) return ATTN_ERR_MISALIGNED;
  // What is written may overlap nothing else, but for the weights in place.
  const size_t w_bytes = (size_t)pairs * weights_stride * 4;
  const size_t pool_bytes = (size_t)num_pages * Hkv * page_size * D * 2;
  struct Range {
    const void* p;
    size_t n;
  };
  const Range written[] = {{weights_out, w_bytes},
                           {k, pool_bytes},
                           {v, pool_bytes},
                           {kept, (size_t)pairs * keep * 4},
                           {new_lens, (size_t)B * 4},
                           {freed, (size_t)max_freed * 4},
                           {info, 8}};
  const Range read[] = {{seq_lens, (size_t)B * 4},
                        {starts, (size_t)B * 4},
                        {page_table, (size_t)B * pages_per_seq * 4},
                        {new_table, (size_t)B * (size_t)std::max(0, new_pages_per_seq) * 4},
                        {weights == weights_out ? nullptr : weights, w_bytes}};
  for (const Range& x : written) {
    for (const Range& y : read)
      if (overlap(x.p, x.n, y.p, y.n)) return ATTN_ERR_INVALID_ARG;
    for (const Range& y : written)
      if (&x < &y && overlap(x.p, x.n, y.p, y.n)) return ATTN_ERR_INVALID_ARG;
  }

  EvictArgs a{};
  a.weights = weights;
  a.weights_out = weights_out;
  a.seq_lens = seq_lens;
  a.starts = starts;
  a.sink = sink;
  a.keep = keep;
  a.recent = recent;
  a.k = static_cast<char*>(k);
  a.v = static_cast<char*>(v);
  a.table = page_table;
  a.new_table = new_table;
  a.per = pages_per_seq;
  a.new_per = new_pages_per_seq;
  a.B = B;
  a.Hkv = Hkv;
  a.max_len = max_len;
  a.shift = 4;
  while ((1 << a.shift) != page_size) ++a.shift;
  a.num_pages = num_pages;
  a.stride = weights_stride;
  a.row_bytes = 2 * D;
  a.kept = kept;
  a.new_lens = new_lens;
  a.freed = freed;
  a.max_freed = max_freed;
  a.info = info;
  const long long sms = sm_count();
  // Blocks of a pair in the selection: as long as each has 2048 keys or more and all run at once,
  // two per SM. (8 x 32768 keys of 8 heads: 1, 2, 4, 8 blocks 146, 129, 125, 140 us for the call;
  // 60000 keys of 8 heads 223, 82, 65, 59 us.)
  a.select_cluster = 1;
  while (a.select_cluster < kMaxCluster && max_len >= 2 * 2048LL * a.select_cluster &&
         2 * pairs * a.select_cluster <= 2 * sms)
    a.select_cluster *= 2;
  // The move: three blocks or more per SM. Into other pages by runs of whole rows. In place first
  // by the channels, down to 64 bytes, then by clusters. (8 x 32768 keys of 8 heads, 8192 kept:
  // four parts of a row 126 us, two parts and clusters of two 148 us: their barrier costs more
  // than a block's. 60000 keys of 8 heads, 16000 kept, four parts: clusters of four 70 us, of
  // eight 60 us.)
  const long long want = 3 * sms;
  a.move_cluster = a.splits = a.chunks = 1;
  // Every block that lists freed pages counts those of all sequences before its own, so up to 128
  // of them. (1024 sequences of 500 keys, one head, pages of 16: 64, 128, 256 blocks 58, 54, 58 us;
  // 8192 of 200 keys 313, 271, 277 us.)
  a.list_run = (B + 127) / 128;
  a.lists = new_table ? (B + a.list_run - 1) / a.list_run : 0;
  const int batch = kMoveThreads * 16 / a.row_bytes * kMoveUnroll;
  const long long most = ((long long)std::min(max_len, keep) + page_size + batch - 1) / batch;
  if (new_table) {
    a.chunks = (int)std::max(1LL, std::min(most, (want + 2 * pairs - 1) / (2 * pairs)));
  } else {
    while (2 * pairs * a.splits < want && a.row_bytes / a.splits > 64) a.splits *= 2;
    while (a.move_cluster < kMaxCluster && 2 * pairs * a.splits * a.move_cluster < want &&
           a.move_cluster < most)
      a.move_cluster *= 2;
  }
  a.piece = a.row_bytes / a.splits;

  static DeviceOnce ready;
  attn_status st = cuda_status(ready.allow_smem(evict_select_kernel, kSelStaged * 4));
  if (st != ATTN_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int slice = max_len / a.select_cluster + 1;
  const size_t smem = (size_t)std::min(slice, kSelStaged) * 4;
  st = cuda_status(launch_early_clusters(evict_select_kernel, (unsigned)(pairs * a.select_cluster),
                                         a.select_cluster, kSelThreads, smem, s, a));
  if (st != ATTN_OK) return st;
  const unsigned blocks =
      (unsigned)(a.lists + pairs * (2 * a.splits * a.chunks + 1) * a.move_cluster);
  return cuda_status(launch_early_clusters(evict_move_kernel, blocks, a.move_cluster, kMoveThreads, 0,
                                           s, a));
}

namespace mattn {
MATTN_DEBUG_RECORD_ACCESSORS(evict)
}  // namespace mattn
