// Eviction from the bf16 paged cache by accumulated attention weight: of every (sequence,
// key/value head)'s keys the first `first`, the last `recent` and the heaviest of those between
// stay, keep in all beside the first; their rows move together, in order.
//
// Two kernels. The first finds, per pair, the kept keys: the key of rank keep - recent in the
// order (weight descending, index ascending) by a radix selection on the weights' bits (ordered
// as unsigned numbers; 11, 11 and 10 bits, so that three histograms of the block's weights,
// staged in shared memory, give it exactly), then an ascending list of those above it. Bound by
// latency: one block per pair, six passes over weights in shared memory.
//
// The second moves the rows. HBM is the bound: every kept row is read and written once. In
// place, kept key m's row goes from kept[m] to first + m <= kept[m], so in ascending batches
// no write reaches a later batch's source; inside a batch all rows are read before one is
// written (a barrier). A block therefore owns some channels of one pair's K or V rows from the
// first batch to the last, and pairs x channels give the parallelism. Into other pages no order
// is needed and batches are dealt out too.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "host_util.h"
#include "launch.h"

#define MATTN_API extern "C" __attribute__((visibility("default")))

namespace mattn {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelStaged = 48 * 1024;  // weights of a pair that are staged (4 bytes each)
constexpr int kSelBins = 2048;
constexpr int kMoveThreads = 512;
constexpr int kMoveUnroll = 4;  // 16-byte pieces of a thread in flight

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
  int splits, piece;  // the move: parts of a row of `piece` bytes
  int chunks;         // the move into other pages: runs of positions
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

// Pages of a sequence that it no longer uses: entries [stay, have) of its table row.
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

// Sum over the block of `mine`, and of those of the threads before: by a scan of warp sums.
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
  int w = lane < kSelWarps ? warp_sums[lane] : 0;
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
  __shared__ int hist[kSelBins];
  __shared__ int sums[kSelWarps], equals[kSelWarps];
  __shared__ int found_bin, found_above;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv;
  early_start();
  const EvictSeq s = evict_seq(a, b);
  if (h == 0) {  // the sequence's length and its pages that go
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
    if (tid == 0) {
      a.new_lens[b] = s.new_len();
      if (b == a.B - 1) {
        a.info[0] = total + n;
        a.info[1] = all_cuts;
      }
    }
  }
  int* kept = a.kept + (size_t)blockIdx.x * a.keep;
  if (!s.cut) {
    for (int m = tid; m < a.keep; m += kSelThreads) kept[m] = m < s.held ? s.first + m : -1;
    return;
  }
  const int c = s.len - s.first - a.recent, k = a.keep - a.recent;  // k of c candidates stay
  for (int m = tid; m < a.recent; m += kSelThreads) kept[k + m] = s.len - a.recent + m;
  if (k == 0) return;
  const uint32_t* w =
      reinterpret_cast<const uint32_t*>(a.weights + (size_t)blockIdx.x * a.stride + s.first);
  const bool stage = c <= kSelStaged;
  if (stage)
    for (int i = tid; i < c; i += kSelThreads) staged[i] = weight_key(w[i]);
  auto key_at = [&](int i) { return stage ? staged[i] : weight_key(w[i]); };

  // The threshold: the largest key that at least k candidates reach, digit by digit.
  uint32_t prefix = 0, mask = 0;
  int left = k;  // candidates to take among those that share the prefix
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digits = pass == 2 ? 1023u : 2047u;
    for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
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
        if (lane == 0 && bin >= 0) atomicAdd(&hist[bin], 32);
      } else if (bin >= 0) {
        atomicAdd(&hist[bin], 1);
      }
    }
    __syncthreads();
    // from the largest digit down: thread t holds the bins 2047 - 2t and 2046 - 2t
    const int hi = kSelBins - 1 - 2 * tid;
    const int n0 = hist[hi], n1 = hist[hi - 1];
    int total;
    const int above = block_before(n0 + n1, sums, total);
    if (above < left && left <= above + n0 + n1) {
      const bool second = left > above + n0;
      found_bin = second ? hi - 1 : hi;
      found_above = second ? above + n0 : above;
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
  const uint32_t below = (1u << lane) - 1u;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t key = i < hi ? key_at(i) : 0u;
    const uint32_t gt = __ballot_sync(0xffffffffu, i < hi && key > prefix);
    const uint32_t eq = __ballot_sync(0xffffffffu, i < hi && key == prefix);
    const int g = above + __popc(gt & below), e = equal + __popc(eq & below);
    const bool take = (gt >> lane & 1) || ((eq >> lane & 1) && e < left);
    const int m = g + min(e, left);
    if (take && MATTN_IN_BOUNDS(kSiteEvict, m, a.keep)) kept[m] = s.first + i;
    above += __popc(gt);
    equal += __popc(eq);
  }
}

// Byte offset of a head's row at a position of sequence b, or -1 outside the pool.
__device__ __forceinline__ long long evict_row(const EvictArgs& a, const int* table, int per,
                                               int b, int h, int pos) {
  const int lp = pos >> a.shift;
  if (lp >= per || !MATTN_IN_BOUNDS(kSiteEvict, lp, per)) return -1;
  const int page = table[(size_t)b * per + lp];
  if (page < 0 || page >= a.num_pages) return -1;
  return ((((long long)page * a.Hkv + h) << a.shift) + (pos & ((1 << a.shift) - 1))) * a.row_bytes;
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
  early_start();
  const int parts = 2 * a.splits * a.chunks + 1;
  const int pair = blockIdx.x / parts, part = blockIdx.x % parts;
  const int b = pair / a.Hkv, h = pair % a.Hkv;
  const EvictSeq s = evict_seq(a, b);
  const int* kept = a.kept + (size_t)pair * a.keep;
  auto source = [&](int n) { return n < s.first || !s.cut ? n : kept[n - s.first]; };
  const int end = s.new_len();
  if (part == parts - 1) {  // the weights; where they went from is 0
    const float* in = a.weights + (size_t)pair * a.stride;
    float* out = a.weights_out + (size_t)pair * a.stride;
    for (int n0 = 0; n0 < end; n0 += kMoveThreads * kMoveUnroll) {
      float x[kMoveUnroll];
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        const int n = n0 + u * kMoveThreads + threadIdx.x;
        x[u] = n < end ? in[source(n)] : 0.0f;
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        const int n = n0 + u * kMoveThreads + threadIdx.x;
        if (n < end) out[n] = x[u];
      }
    }
    __syncthreads();
    for (int n = end + threadIdx.x; n < s.len; n += kMoveThreads) out[n] = 0.0f;
    return;
  }
  const bool in_place = a.new_table == nullptr;
  if (in_place && !s.cut) return;
  char* pool = part & 1 ? a.v : a.k;
  const int split = (part >> 1) % a.splits, chunk = (part >> 1) / a.splits;
  const int lanes = a.piece / 16;  // threads of a row
  const int row = threadIdx.x / lanes, rows = kMoveThreads / lanes;
  const int col = split * a.piece + threadIdx.x % lanes * 16;
  int from = s.first, to = end;
  if (!in_place) {  // all pages from the first that holds a key that may go, in runs
    from = s.first >> a.shift << a.shift;
    const int batch = rows * kMoveUnroll;
    const int batches = (end - from + batch - 1) / batch;
    const int lo = from + (int)((long long)batches * chunk / a.chunks) * batch;
    to = min(end, from + (int)((long long)batches * (chunk + 1) / a.chunks) * batch);
    from = lo;
  }
  [[maybe_unused]] const long long bytes = ((long long)a.num_pages * a.Hkv << a.shift) * a.row_bytes;
  for (int n0 = from; n0 < to; n0 += rows * kMoveUnroll) {
    uint4 x[kMoveUnroll];
    long long dst[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int n = n0 + u * rows + row;
      dst[u] = -1;
      x[u] = make_uint4(0, 0, 0, 0);
      if (n < to) {
        const int src = source(n);
        if (!in_place || src != n) {
          dst[u] = evict_row(a, in_place ? a.table : a.new_table, in_place ? a.per : a.new_per, b,
                             h, n);
          const long long at = evict_row(a, a.table, a.per, b, h, src);
          if (at >= 0 && MATTN_IN_BOUNDS(kSiteEvictRow, at + col + 15, bytes))
            x[u] = *reinterpret_cast<const uint4*>(pool + at + col);
          if (at == dst[u]) dst[u] = -1;
        }
      }
    }
    if (in_place) __syncthreads();  // every row of the batch is read before one is written
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u)
      if (dst[u] >= 0 && MATTN_IN_BOUNDS(kSiteEvictRow, dst[u] + col + 15, bytes))
        *reinterpret_cast<uint4*>(pool + dst[u] + col) = x[u];
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
  // Blocks of the move: about eight per SM. In place by splitting the rows, down to 64 bytes;
  // into other pages by runs of whole rows.
  const long long want = 8LL * sm_count();
  a.splits = a.chunks = 1;
  if (new_table) {
    const int batch = kMoveThreads * 16 / a.row_bytes * kMoveUnroll;
    const long long most = ((long long)std::min(max_len, keep) + page_size + batch - 1) / batch;
    a.chunks = (int)std::max(1LL, std::min(most, (want + 2 * pairs - 1) / (2 * pairs)));
  } else {
    while (2 * pairs * a.splits < want && a.row_bytes / a.splits > 64) a.splits *= 2;
  }
  a.piece = a.row_bytes / a.splits;

  static DeviceOnce ready;
  attn_status st = cuda_status(ready.allow_smem(evict_select_kernel, kSelStaged * 4));
  if (st != ATTN_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const size_t smem = (size_t)std::min(max_len, kSelStaged) * 4;
  st = cuda_status(launch_early(evict_select_kernel, (unsigned)pairs, kSelThreads, smem, s, a));
  if (st != ATTN_OK) return st;
  const unsigned blocks = (unsigned)(pairs * (2 * a.splits * a.chunks + 1));
  return cuda_status(launch_early(evict_move_kernel, blocks, kMoveThreads, 0, s, a));
}

namespace mattn {
MATTN_DEBUG_RECORD_ACCESSORS(evict)
}  // namespace mattn
