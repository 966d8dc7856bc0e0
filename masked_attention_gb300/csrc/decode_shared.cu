// Decode attention over a bf16 paged cache for sequences of their own lengths, groups of which
// share their first keys (a long prompt behind many requests):
//
//   O = softmax(mask(mod(scale q K^T))) V  over the shared keys and the sequence's own, merged:
//   with parts (O_p, LSE_p) over disjoint keys, LSE = ln sum e^LSE_p, O = sum e^(LSE_p - LSE) O_p.
//
// A shared key row is read once for all query rows of the group's sequences (as long as they
// are no more than 128 of a key/value head, else once per 128), so HBM's part is
// (shared + sum of own keys) * 4 D bytes per key/value head, against sequences * shared without.
// With 128 rows a tile of 128 keys is 64 KB and 2 x 2 * 128^3 operations, so the tensor cores,
// the exponentials and HBM all matter, and the product runs on tcgen05 with 128-row tiles.
//
// Work. A piece is a run of 64-key tiles of one key/value head for one 128-row block: of a
// group's shared keys with up to 128 / R of its sequences (R query rows each: the heads of the
// key/value head times Sq), or of one sequence's own keys with its R rows (the tile's other rows
// idle: HBM bounds these). All pieces' tiles, one after the other, each with a constant for its
// start and end, are dealt out evenly to two CTAs per SM (one's softmax runs under the other's
// products). Shared keys with several row blocks are cut into chunks of one CTA's share first,
// all blocks of a chunk side by side, so that CTAs that read the same keys do so at the same time
// and the second reads them from the L2. A small first kernel lays the pieces out from the
// lengths on the device, CTAs leave fp32 partial results in the workspace, a third kernel joins
// them.
//
// Within a CTA: warps 0 to 3 softmax, a thread per query row (TMEM lane); warp 4 finds the pieces,
// tells the others through shared memory and copies (TMA); warp 5 issues S = Q K^T, of the next
// tile as soon as the softmax has this one's scores in registers; warp 6 O += P V (P: bf16 in
// tensor memory, in two places of its own, rounded to 8 bits as in the other bf16 calls; its sum
// is of the unrounded values) and, while it waits for P, zeroes the values of keys that no row
// sees. (One warp for both products was what a tile waited for: 1900
// cycles, of which 900 its waits.) Tiles of 64 keys, not 128: five K or V tiles then fit beside Q
// twice per SM instead of two, so that the next ones arrive while this one is worked on.
//
// 32 heads on 8 of 128 channels, bf16. 16 sequences of 32768 own keys: 313 us, 6.8 TB/s, the rate
// of a copy. 64 of 4000: 168 us, 6.3 TB/s. 64 sequences behind 32768 shared keys, 700 own keys
// each: 80 us, 4.0 TB/s and 440 TFLOP/s, for 47 us of bytes. What it takes beyond them: three
// dependent kernels, 14 us in a captured graph for one sequence of one key (the plan is one block,
// the join reads every part back: with half of these keys 8 and 14 us, cold); a second reading of
// each shared tile, out of the L2, by the second block of 128 rows (one own key each: 32 sequences
// 49 us, 64 60); and the pieces' starts and ends. A soft-cap adds 6 us to the 80 of 61 ragged sequences of
// fixed lengths: 16 packed operations per pair of scores, in the warps that hold rows. With a
// window the tiles between the sequences' windows are read and multiplied, too.
#include <algorithm>
#include <climits>
#include <cmath>

#include "host_util.h"
#include "launch.h"
#include "soft_cap.cuh"

#define MATTN_API extern "C" __attribute__((visibility("default")))

namespace mattn {
namespace {

constexpr int kShThreads = 256;
constexpr int kShProducer = 4, kShQK = 5, kShPV = 6;  // warps; 0 to 3: softmax
constexpr int kShRegsSoftmax = 176, kShRegsOther = 80;  // 128 x 176 + 128 x 80 = 256 x 128
constexpr int kShPerSm = 2;
constexpr int kShMaxB = 4096;  // the plan holds 48 bytes of each in shared memory
constexpr int kShMaxRows = 16;
constexpr int kShKeys = 64;       // keys of a tile
// What counts in the dealing out: a tile of a sequence's own keys, of shared ones (whose rows keep
// all warps busy), and a piece's start and end. (64 sequences behind 32768 keys, 1 key each, with
// kShCost 12, 16, 24, 32: 70, 68, 61, 61 us; kShShared 7 to 9 makes no difference, 13 costs 15 %.
// Six ragged batches with a soft-cap, 100 to 130 us: kShCost 16 takes 2 % less, 48 3 % more,
// kShShared 12 5 % more.)
constexpr int kShOwn = 8, kShShared = 8, kShCost = 24;
constexpr int kShPlanThreads = 256;
constexpr int kShPlanWarps = kShPlanThreads / 32;
// Shared keys below this are read by each sequence itself: all but the first find them in the L2,
// and a shared run is one more part to join. (64 sequences with 700 own keys behind 128, 256 and
// 512 shared ones, in groups of 2: shared 52.8, 55.0, 59.0 us, by each itself 50.9, 54.3, 59.8 us;
// in one group 48.0, 47.5, 47.8 and 46.1, 46.7, 48.5 us.) The bound knows nothing of the group's
// size: with 50 own keys each large groups lose by it (64, 256 and 1024 sequences behind 448 keys
// 33, 83, 258 us, with a bound of 64 24.6, 50, 163; behind 128 keys 25, 55, 168 and 23, 46, 152).
constexpr int kShMinShared = 512;

struct ShDesc {  // pieces of the same keys: one per key/value head and, of shared keys, row block
  long long start;  // of the first one in the dealing out, of length sh_length() each
  int tiles;
  int key0;      // first key of the first tile, a multiple of the page size
  int klo, khi;  // keys of the piece
  int seq, nseq;  // sequences of its rows, in blocks; the first one's table row is read
  int blocks;     // row blocks of shared keys (a head's pieces side by side); 0: own keys
  int base;       // number of its first piece among those of its kind
};

struct ShSeq {  // how to find a sequence's parts
  int pdesc, chunks;  // pieces of its group's shared keys: from pdesc on
  int block, row0;    // its block there, its first row in it
  int sdesc;          // pieces of its own keys, or -1
};

struct ShHead {
  long long total, share;  // positions dealt out, and per CTA
  int n_prefix;            // descriptions of shared keys come first
  int n_desc;
};

// A piece's tile t begins at kShCost + t * w behind the piece's start, w by its kind, and is the
// CTA's that has that position.
__host__ __device__ __forceinline__ int sh_weight(int shared) { return shared ? kShShared : kShOwn; }
__device__ __forceinline__ long long sh_length(int shared, int tiles) {
  return kShCost + (long long)tiles * sh_weight(shared);
}

// Quotient of positions: 64-bit divisions take several hundred cycles, and positions past 32
// bits need tens of millions of keys.
__device__ __forceinline__ long long sh_div(long long a, long long b) {
  return (a | b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

struct ShProblem {
  const int* seq_lens;
  const int* starts;  // [G + 1]
  const int* shared_lens;
  const int* table;
  const float* slopes;
  void* o;
  float* lse;
  int B, Hq, Hkv, Sq, R, G, max_len;
  int seqs_per_block;  // 128 / R
  int shift, pages_per_seq, num_pages;
  unsigned variant;
  int window;
  float scale2, softcap2, softcap_e;
  int ctas, max_desc, max_prefix, max_parts;
  ShHead* head;
  ShDesc* desc;   // [max_desc]
  ShSeq* seqs;    // [B]
  float *p_lse, *p_o, *s_lse, *s_o;  // partial results: shared [slots][128], own [slots][R]
  long long p_slots, s_slots;
  int* status;
  uint64_t timeout_ns;
  unsigned fault_inject;
};

// ------------------------------------------------------------------------- the plan
struct ShGroup {
  int blocks, tiles;        // row blocks, tiles of its shared keys
  int key0, low, shared;    // first key of the first tile, first one that is seen, their end
  int chunks, desc, base;   // runs of tiles, first description, first piece's number
  long long start;          // and that one's position
};

__device__ __forceinline__ int sh_len(const ShProblem& p, int b) {
  return max(0, min(p.seq_lens[b], p.max_len));
}
// First key that some row of a sequence sees.
__device__ __forceinline__ int sh_low(const ShProblem& p, int len) {
  return p.variant & ATTN_MASK_WINDOW ? (int)max(0ll, (long long)len - p.Sq - p.window + 1) : 0;
}
// A tile begins with a page, or in the middle of one of 128 keys.
__device__ __forceinline__ int sh_down(const ShProblem& p, int key) {
  const int s = min(p.shift, 6);
  return key >> s << s;
}
__device__ __forceinline__ int sh_tiles(int keys) { return (keys + kShKeys - 1) / kShKeys; }

// Block-wide scan: sum (or maximum) of the threads before, and of all.
template <bool kMax, typename T>
__device__ __forceinline__ T plan_scan(T mine, T* warps, T& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto join = [](T a, T b) { return kMax ? (a > b ? a : b) : a + b; };
  T x = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T o = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x = join(x, o);
  }
  __syncthreads();
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  T before = __shfl_up_sync(0xffffffffu, x, 1);
  if (lane == 0) before = 0;  // neutral: values are not negative
  all = 0;
#pragma unroll
  for (int i = 0; i < kShPlanWarps; ++i) {
    if (i < warp) before = join(before, warps[i]);
    all = join(all, warps[i]);
  }
  return before;
}

// Sum over the block.
__device__ __forceinline__ long long plan_sum(long long mine, long long* warps) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = mine;
  __syncthreads();
  long long all = 0;
#pragma unroll
  for (int i = 0; i < kShPlanWarps; ++i) all += warps[i];
  return all;
}

__global__ void __launch_bounds__(kShPlanThreads) shared_plan_kernel(const ShProblem p) {
  extern __shared__ __align__(16) int plan_smem[];
  int* group_of = plan_smem;                     // [B]: its group, or -1
  int* begin = group_of + ((p.B + 3) & ~3);      // [G + 1]
  ShGroup* groups = reinterpret_cast<ShGroup*>(begin + ((p.G + 4) & ~3));  // [G]
  __shared__ long long warps[kShPlanWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  early_start();
  for (int b = tid; b < p.B; b += kShPlanThreads) group_of[b] = -1;
  // the groups' first sequences, ascending whatever they hold
  long long carry = 0, all;
  for (int g0 = 0; p.G > 0 && g0 <= p.G; g0 += kShPlanThreads) {
    const int g = g0 + tid;
    const long long x = g <= p.G ? max(0, min(p.starts[g], p.B)) : 0;
    const long long before = plan_scan<true>(x, warps, all);
    if (g <= p.G) begin[g] = (int)max(carry, max(before, x));
    carry = max(carry, all);
  }
  __syncthreads();
  // shared keys of the groups that have two sequences or more, a warp each
  long long work = 0;
  for (int g = warp; g < p.G; g += kShPlanWarps) {
    const int b0 = begin[g], n = begin[g + 1] - b0;
    ShGroup gr{};
    if (n > 1) {
      int longest = 0, low = INT_MAX;
      for (int b = b0 + lane; b < b0 + n; b += 32) {
        const int len = sh_len(p, b);
        longest = max(longest, len);
        if (len > 0) low = min(low, sh_low(p, len));
      }
      longest = __reduce_max_sync(0xffffffffu, longest);
      low = __reduce_min_sync(0xffffffffu, low);
      const int end = min(p.shared_lens[g], longest);
      if (end >= kShMinShared) {
        gr.shared = end;
        gr.blocks = (n + p.seqs_per_block - 1) / p.seqs_per_block;
        gr.low = min(low, end);
        gr.key0 = sh_down(p, gr.low);
        gr.tiles = low < end ? sh_tiles(end - gr.key0) : 0;
        for (int b = b0 + lane; b < b0 + n; b += 32) group_of[b] = g;
      }
    }
    if (lane == 0) {
      groups[g] = gr;
      work += (long long)gr.tiles * gr.blocks;
    }
  }
  __syncthreads();
  // a sequence's own keys
  struct Own {
    int klo, len, key0, tiles;
  };
  auto own_of = [&](int b) {
    Own w;
    w.len = sh_len(p, b);
    const int g = group_of[b];
    w.klo = max(g >= 0 ? groups[g].shared : 0, sh_low(p, w.len));
    w.key0 = sh_down(p, w.klo);
    w.tiles = w.len > w.klo ? sh_tiles(w.len - w.key0) : 0;
    return w;
  };
  // Keys of several row blocks are cut into chunks, each a CTA's share: what all tiles and the
  // pieces of whole groups take, then with that many chunks' starts and ends once more.
  long long length = work * kShShared;
  for (int b = tid; b < p.B; b += kShPlanThreads) {
    const int n = own_of(b).tiles;
    work += n;
    length += n ? sh_length(0, n) : 0;
  }
  const long long least = sh_div(plan_sum(work, warps) * p.Hkv + p.ctas - 1, p.ctas);  // tiles
  const long long plain = plan_sum(length, warps);
  auto share_of = [&](long long n) { return sh_div(n * p.Hkv + p.ctas - 1, p.ctas); };
  long long chunk = 1, pieces = 0;
  for (int pass = 0; pass < 2; ++pass) {
    const long long cut = pass ? plan_sum(pieces, warps) * kShCost : 0;
    chunk = max(max(1ll, (least + 1) / 2), sh_div(max(0ll, share_of(plain + cut) - kShCost), kShShared));
    pieces = 0;
    for (int g = tid; g < p.G; g += kShPlanThreads) {
      ShGroup& gr = groups[g];
      if (!gr.tiles) continue;
      gr.chunks = gr.blocks > 1 ? (int)sh_div(gr.tiles + chunk - 1, chunk) : 1;
      pieces += (long long)gr.chunks * gr.blocks;
    }
  }
  const long long total = (plain + plan_sum(pieces, warps) * kShCost) * p.Hkv;
  // no less than a tile, so that every CTA within a piece has one of it
  const long long share = max((long long)max(kShOwn, kShShared), sh_div(total + p.ctas - 1, p.ctas));
  // positions: of the shared keys, group by group, then of the sequences' own keys
  long long at = 0, base = 0;
  int n_prefix = 0;
  for (int g0 = 0; g0 < p.G; g0 += kShPlanThreads) {
    const int g = g0 + tid;
    long long n = 0, count = 0, len = 0, all_n, all_count, all_len;
    if (g < p.G && groups[g].tiles) {
      n = groups[g].chunks;
      count = n * groups[g].blocks * p.Hkv;
      len = (long long)p.Hkv * groups[g].blocks *
            ((long long)groups[g].tiles * kShShared + groups[g].chunks * kShCost);
    }
    const long long n0 = n_prefix + plan_scan<false>(n, warps, all_n);
    const long long b0 = base + plan_scan<false>(count, warps, all_count);
    const long long a0 = at + plan_scan<false>(len, warps, all_len);
    if (n) {
      groups[g].desc = (int)n0;
      groups[g].base = (int)b0;
      groups[g].start = a0;
    }
    n_prefix += (int)all_n;
    base += all_count;
    at += all_len;
  }
  if (tid == 0) *p.head = ShHead{total, share, n_prefix, n_prefix + p.B};
  __syncthreads();
  for (int g = warp; g < p.G; g += kShPlanWarps) {  // a lane per chunk
    const ShGroup gr = groups[g];
    for (int c = lane; gr.tiles && c < gr.chunks; c += 32) {
      // the first `more` ones are a tile longer
      const int len = gr.tiles / gr.chunks, more = gr.tiles - len * gr.chunks;
      const int t0 = c * len + min(c, more), t1 = t0 + len + (c < more);
      ShDesc x;
      x.tiles = t1 - t0;
      x.start = gr.start + (long long)p.Hkv * gr.blocks * ((long long)t0 * kShShared + c * kShCost);
      x.key0 = gr.key0 + t0 * kShKeys;
      x.klo = max(x.key0, gr.low);
      x.khi = min(gr.shared, gr.key0 + t1 * kShKeys);
      x.seq = begin[g];
      x.nseq = begin[g + 1] - begin[g];
      x.blocks = gr.blocks;
      x.base = gr.base + c * gr.blocks * p.Hkv;
      if (MATTN_IN_BOUNDS(kSiteShPlan, gr.desc + c, p.max_prefix)) p.desc[gr.desc + c] = x;
    }
  }
  for (int b0 = 0; b0 < p.B; b0 += kShPlanThreads) {
    const int b = b0 + tid;
    Own w{0, 0, 0, 0};
    if (b < p.B) w = own_of(b);
    const long long len = w.tiles ? p.Hkv * sh_length(0, w.tiles) : 0;
    long long all_len;
    const long long a0 = at + plan_scan<false>(len, warps, all_len);
    at += all_len;
    if (b >= p.B) continue;
    ShDesc x;
    x.start = a0;
    x.tiles = w.tiles;  // 0: a piece that is passed over
    x.key0 = w.key0;
    x.klo = w.klo;
    x.khi = w.len;
    x.seq = b;
    x.nseq = 1;
    x.blocks = 0;
    x.base = b * p.Hkv;
    if (MATTN_IN_BOUNDS(kSiteShPlan, n_prefix + b, p.max_desc)) p.desc[n_prefix + b] = x;
    ShSeq q{0, 0, 0, 0, w.tiles ? n_prefix + b : -1};
    const int g = group_of[b];
    if (g >= 0 && groups[g].tiles) {
      q.pdesc = groups[g].desc;
      q.chunks = groups[g].chunks;
      q.block = (b - begin[g]) / p.seqs_per_block;
      q.row0 = (b - begin[g] - q.block * p.seqs_per_block) * p.R;
    }
    p.seqs[b] = q;
  }
}

// ------------------------------------------------------------------------- the pieces
template <int D>
struct ShCfg {
  static constexpr int kBoxes = D / 64;
  static constexpr int kQBox = kTile * 128;        // 128 query rows x 64 channels
  static constexpr int kQBytes = kBoxes * kQBox;
  static constexpr int kBox = kShKeys * 128;       // 64 keys x 64 channels
  static constexpr int kTileBytes = kBoxes * kBox;
  // Places of K and of V tiles. Rings of their own: each has one warp that sees every pass of it
  // (a warp that waited for every other pass of a shared place would take one for the next).
  // Values stay longer, from before their scores to the end of their product.
  static constexpr int kKSlots = D == 128 ? 2 : 5, kVSlots = D == 128 ? 3 : 5;
  static constexpr int kSlots = kKSlots + kVSlots;
  static constexpr int kSmem = kQBytes + kSlots * kTileBytes;
  // Tensor memory: S (64 columns), P twice (32 each), O.
  static constexpr uint32_t kColP = kShKeys, kColO = 2 * kShKeys;
  // A sequence's rows alone (at most 16) stand in one half of the Q tile or the other, row 0 or
  // row 64 of it, so that the next piece's are there early.
  static constexpr int kHalf = 64 * 128;
  static_assert(kSmem + 1024 <= 113 * 1024 + 512, "two CTAs per SM");
};

constexpr int kShMsgs = 4;
struct ShMsg {  // a run of tiles, as the producer tells it
  int tiles;    // 0: no more
  int key0, klo, khi, seq, nseq, shared, h;
  long long slot;  // of its partial result
};

// Of 32 keys those from `from` to `to` - 1, a bit each.
__device__ __forceinline__ unsigned sh_span(int from, int to) {
  from = max(from, 0);
  to = min(to, 32);
  return from < to ? (~0u >> (32 - (to - from))) << from : 0u;
}

// Of the 32 keys from j0 on those that some row of a block of sequences sees. (A sequence's rows
// see one run of keys, all of them together.)
__device__ __forceinline__ unsigned sh_seen(const ShProblem& p, int seq, int nseq, int j0) {
  unsigned mine = 0;
  for (int i = threadIdx.x & 31; i < nseq; i += 32) {
    const int len = sh_len(p, seq + i);
    mine |= sh_span(sh_low(p, len) - j0, len - j0);
  }
  return __reduce_or_sync(0xffffffffu, mine);
}

// Whether a block's sequences may leave some of the keys [from, to) to nobody: they end apart, so
// with a window their runs of keys may lie apart, too. (Runs that all meet at one place do not.
// Asked once per piece: with sh_seen() for every tile 64 sequences behind 8192 keys, window 4096,
// took 34 to 37 us instead of 32.)
__device__ __forceinline__ bool sh_apart(const ShProblem& p, int seq, int nseq, int from, int to) {
  int low = INT_MAX, high = 0, near = INT_MAX, far = 0;  // least and largest start and end
  for (int i = threadIdx.x & 31; i < nseq; i += 32) {
    const int len = sh_len(p, seq + i), at = sh_low(p, len);
    if (len == 0) continue;
    low = min(low, at);
    high = max(high, at);
    near = min(near, len);
    far = max(far, len);
  }
  constexpr unsigned all = 0xffffffffu;
  return __reduce_max_sync(all, high) > __reduce_min_sync(all, near) ||
         __reduce_min_sync(all, low) > from || __reduce_max_sync(all, far) < to;
}

__device__ __forceinline__ bool sh_wait(uint64_t* bar, uint32_t parity, const Watchdog& wd) {
  const uint32_t hint = wd.timeout_ns < 1000000ull ? (uint32_t)wd.timeout_ns : 1000000u;
  const bool done = mbar_try_wait(bar, parity) || mbar_try_wait_sleep(bar, parity, hint) ||
                    wait_bounded(bar, parity, wd);
  return __all_sync(0xffffffffu, done);
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

struct ShRing {
  uint32_t slot = 0, pass = 0;
  __device__ __forceinline__ void next(uint32_t n) {
    if (++slot == n) {
      slot = 0;
      pass ^= 1;
    }
  }
};

// The producer's walk over the CTA's share of the pieces: runs of tiles [t0, t1).
struct ShWalk {
  ShDesc d, ahead;   // this piece and, read early, the one behind it
  int at, n_desc;     // the piece's description
  int h, block;       // its head and row block
  int t0, t1;
  long long lo, hi;  // positions still to go
  __device__ __forceinline__ void enter(const ShProblem& p) {
    ahead = p.desc[min(at + 1, n_desc - 1)];
  }
  // From position lo: the run that begins there (false: none left).
  __device__ __forceinline__ bool find(const ShProblem& p) {
    while (lo < hi) {
      const long long len = sh_length(d.blocks, d.tiles);
      const long long start = d.start + piece() * len;
      const long long end = min(hi, start + len);
      const int w = sh_weight(d.blocks);
      t0 = (int)sh_div(max(0ll, lo - start - kShCost) + w - 1, w);
      t1 = min(d.tiles, (int)sh_div(max(0ll, end - start - kShCost) + w - 1, w));
      if (t0 < t1) return true;
      lo = end;
      if (lo < start + len || lo >= hi) return false;  // the share ends inside the piece
      step(p);
    }
    return false;
  }
  __device__ __forceinline__ int piece() const { return h * max(1, d.blocks) + block; }
  __device__ __forceinline__ void step(const ShProblem& p) {
    if (++block < d.blocks) return;
    block = 0;
    if (++h < p.Hkv) return;
    h = 0;
    ++at;
    d = ahead;
    while (d.tiles == 0 && at + 1 < n_desc) d = p.desc[++at];
    enter(p);
  }
  __device__ __forceinline__ bool next(const ShProblem& p) {
    const long long len = sh_length(d.blocks, d.tiles);
    lo = d.start + (piece() + 1) * len;
    if (lo >= hi) return false;
    step(p);
    return find(p);
  }
};

// The steps of a tile's softmax, on the thread's 64 scores in registers. They are kept apart,
// each once in the code: a piece's first and last tiles run all of them, and with masked copies
// of each step their instructions did not stay in the cache (a piece of one tile took 10000
// cycles).

// The soft-cap's series alone, for two scores below a quarter of the cap (soft_cap_near).
__device__ __forceinline__ float2 cap_near2(float2 s, float inv) {
  constexpr float kX2 = 0.25f * 0.69314718f * 0.69314718f;
  auto two = [](float x) { return make_float2(x, x); };
  const float2 y = fmul2(s, two(inv)), y2 = fmul2(y, y);
  float2 q = ffma2(y2, two(62.0f / 2835.0f * kX2 * kX2 * kX2 * kX2), two(-17.0f / 315.0f * kX2 * kX2 * kX2));
  q = ffma2(y2, q, two(2.0f / 15.0f * kX2 * kX2));
  q = ffma2(y2, q, two(-1.0f / 3.0f * kX2));
  return ffma2(fmul2(s, y2), q, s);
}

// Score modifications: x becomes the modified score in log2 units (SCORE 0: stays the product).
// pos: the row's position less the tile's first key. mine: the thread has a row; the others hold
// products with what earlier rows or kernels left in the Q tile, and have no say in the branch.
template <int SCORE>
__device__ __forceinline__ void sh_modify(const ShProblem& p, float slope2, int pos, bool mine,
                                          float (&x)[64]) {
  if constexpr (SCORE == 0) return;
  const float2 sl = make_float2(p.scale2, p.scale2);
  float size = 0.0f;
#pragma unroll
  for (int c = 0; c < 64; c += 2) {
    float2 y = fmul2(make_float2(x[c], x[c + 1]), sl);
    if constexpr (SCORE & 1) {
      y.x -= slope2 * float(pos - c);
      y.y -= slope2 * float(pos - c - 1);
    }
    x[c] = y.x;
    x[c + 1] = y.y;
    if constexpr (SCORE & 2) size = fmax3(size, fabsf(y.x), fabsf(y.y));
  }
  if constexpr (SCORE & 2) {
    // (a NaN leaves `size` as it is and passes through the series too)
    if (__all_sync(0xffffffffu, !mine || size * p.softcap_e < kCapNear)) {
#pragma unroll
      for (int c = 0; c < 64; c += 2) {
        const float2 y = cap_near2(make_float2(x[c], x[c + 1]), p.softcap_e);
        x[c] = y.x;
        x[c + 1] = y.y;
      }
    } else {
#pragma unroll
      for (int c = 0; c < 64; ++c) x[c] = soft_cap(x[c], p.softcap2, p.softcap_e);
    }
  }
}

// P of 32 scores as packed bf16, and their sum. scale: what is left to multiply them with.
__device__ __forceinline__ float sh_exp32(const float* x, float scale, float m, uint32_t* pk) {
  float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
  const float2 sl = make_float2(scale, scale), mm = make_float2(-m, -m);
#pragma unroll
  for (int c = 0; c < 32; c += 2) {
    const float2 y = ffma2(make_float2(x[c], x[c + 1]), sl, mm);
    const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
    sum[(c / 2) & 1] = fadd2(sum[(c / 2) & 1], e);
    pk[c / 2] = pack_bf16x2(e.x, e.y);
  }
  const float2 t = fadd2(sum[0], sum[1]);
  return t.x + t.y;
}

template <int D, int SCORE>
__global__ void __launch_bounds__(kShThreads, kShPerSm)
    decode_shared_kernel(const __grid_constant__ CUtensorMap tm_qs,
                         const __grid_constant__ CUtensorMap tm_q1,
                         const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const ShProblem p) {
  using C = ShCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;
  uint8_t* sK = smem + C::kQBytes;
  uint8_t* sV = sK + C::kKSlots * C::kTileBytes;
  __shared__ uint64_t bars[10 + 2 * kShMsgs + 2 * C::kSlots];
  __shared__ ShMsg msgs[kShMsgs];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_word;
  uint64_t *q_full = bars, *q_empty = bars + 2, *s_full = bars + 4, *s_free = bars + 5,
           *p_full = bars + 6, *pv_done = bars + 7, *o_free = bars + 8, *drain = bars + 9,
           *msg_full = bars + 10,
           *msg_empty = msg_full + kShMsgs, *k_full = msg_empty + kShMsgs,
           *k_empty = k_full + C::kKSlots, *v_full = k_empty + C::kKSlots,
           *v_empty = v_full + C::kVSlots;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &abort_word;
  const Watchdog wd{abort_flag, p.status, p.timeout_ns};
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(q_empty + i, 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_free, 4);
    mbar_init(p_full, 4);
    mbar_init(pv_done, 1);
    mbar_init(o_free, 4);
    mbar_init(drain, 2);
    for (int i = 0; i < kShMsgs; ++i) {
      mbar_init(msg_full + i, 1);
      mbar_init(msg_empty + i, 6);  // the products' two warps and four of the softmax
    }
    for (int i = 0; i < 2 * C::kSlots; ++i) mbar_init(k_full + i, 1);
    abort_word = 0;
    fence_barrier_init();
  }
  if (warp == kShQK) {
    tmem_alloc(&tmem_base, 256);
    tmem_relinquish();
  }
  if (warp == kShProducer && lane == 0) {
    prefetch_tmap(&tm_qs);
    prefetch_tmap(&tm_q1);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  early_start();
  // The next message, or false (and ok = false where the wait ran out).
  ShRing mr;
  auto next_msg = [&](ShMsg& m, bool& ok) {
    ok = sh_wait(msg_full + mr.slot, mr.pass, wd);
    if (!ok) return false;
    m = msgs[mr.slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(msg_empty + mr.slot);
    mr.next(kShMsgs);
    return m.tiles > 0;
  };

  if (warp >= kShProducer) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kShRegsOther));
  if (warp == kShProducer) {
    const bool issue = !(p.fault_inject & ATTN_FAULT_NO_LOADS);
    ShRing kr, vr;
    uint32_t q_pass[2] = {0, 0}, half = 0;  // parity of the halves' release, half in turn
    uint32_t q_armed = 0, q_seen = 0;       // halves with a copy, parity of their latest
    const int per_tile = max(1, kShKeys >> p.shift), page_rows = min(kShKeys, 1 << p.shift);
    ShWalk walk;
    const ShHead head = *p.head;
    walk.lo = min(head.total, blockIdx.x * head.share);
    walk.hi = min(head.total, walk.lo + head.share);
    bool ok = true, more = walk.lo < walk.hi;
    if (more) {
      walk.n_desc = head.n_desc;
      // The last piece that starts at or before lo, 32 probes at a time (pieces without tiles
      // start where the next one does).
      int from = 0, to = head.n_desc;
      while (to - from > 1) {
        const int step = (to - from + 31) / 32, at = from + lane * step;
        const bool below = at < to && p.desc[at].start <= walk.lo;
        const int hit = 31 - __clz(__ballot_sync(0xffffffffu, below));  // lane 0's always is
        to = min(to, from + (hit + 1) * step);
        from += hit * step;
      }
      walk.at = from;
      walk.d = p.desc[walk.at];
      walk.enter(p);
      const int n = max(1, walk.d.blocks);
      walk.block = (int)sh_div(walk.lo - walk.d.start, sh_length(walk.d.blocks, walk.d.tiles));
      walk.h = walk.block / n;
      walk.block -= walk.h * n;
      more = walk.find(p);
    }
    while (ok) {
      ok = sh_wait(msg_empty + mr.slot, mr.pass ^ 1, wd);
      if (!ok) break;
      if (lane == 0) {
        ShMsg m{};
        if (more) {
          const ShDesc& d = walk.d;
          m.tiles = walk.t1 - walk.t0;
          m.key0 = d.key0 + walk.t0 * kShKeys;
          m.klo = d.klo;
          m.khi = d.khi;
          m.seq = d.seq + walk.block * p.seqs_per_block;
          m.nseq = min(d.nseq - walk.block * p.seqs_per_block, p.seqs_per_block);
          m.shared = d.blocks;
          m.h = walk.h;
          m.slot = (long long)blockIdx.x + d.base + walk.piece();
        }
        msgs[mr.slot] = m;
        mbar_arrive(msg_full + mr.slot);
      }
      __syncwarp();
      mr.next(kShMsgs);
      if (!more) break;
      // A lane per page of a tile, its entry read one tile ahead. Pages past the last one with
      // keys repeat it; one outside the pool reads as zeros (past the map's end).
      const int last = (walk.d.khi - 1) >> p.shift;
      const int* row = p.table + (size_t)walk.d.seq * p.pages_per_seq;
      auto page_of = [&](int t) {
        if (lane >= per_tile) return 0;
        const int lp = min(((walk.d.key0 + t * kShKeys) >> p.shift) + lane, last);
        return MATTN_IN_BOUNDS(kSiteShTable, lp, p.pages_per_seq) ? row[lp] : -1;
      };
      int page = page_of(walk.t0);
      // the rows: both halves for a block of sequences, one for a sequence alone
      const bool block = walk.d.blocks;
      if (block) half = 0;
      for (int i = 0; i < 2 && ok; ++i)
        if (block || i == (int)half) {
          ok = sh_wait(q_empty + i, (i ? q_pass[1] : q_pass[0]) ^ 1, wd);
          if (i) q_pass[1] ^= 1;
          else q_pass[0] ^= 1;
        }
      if (!ok) break;
      if (issue) {
        q_armed |= 1u << half;
        q_seen ^= 1u << half;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full + half, (block ? p.seqs_per_block * p.R : p.R) * D * 2);
#pragma unroll
          for (int bx = 0; bx < C::kBoxes; ++bx)
            tma_load_4d(sQ + bx * C::kQBox + half * C::kHalf, block ? &tm_qs : &tm_q1, q_full + half,
                        bx * 64, 0, walk.h, walk.d.seq + walk.block * p.seqs_per_block);
        }
      }
      __syncwarp();
      half = block ? 0 : half ^ 1;
      for (int t = walk.t0; t < walk.t1 && ok; ++t) {
        const int z = (page < 0 || page >= p.num_pages ? p.num_pages : page) * p.Hkv + walk.h;
        const int y = (walk.d.key0 + t * kShKeys) & ((1 << p.shift) - 1);  // pages of 128: 0 or 64
        if (t + 1 < walk.t1) page = page_of(t + 1);
        auto load = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* full, uint64_t* empty,
                        uint32_t pass) {
          if (!sh_wait(empty, pass ^ 1, wd)) return false;
          if (lane == 0 && issue) mbar_arrive_expect_tx(full, C::kTileBytes);
          __syncwarp();
          if (issue && lane < per_tile) {
#pragma unroll
            for (int bx = 0; bx < C::kBoxes; ++bx)
              tma_load_3d(dst + bx * C::kBox + lane * page_rows * 128, map, full, bx * 64, y, z);
          }
          __syncwarp();
          return true;
        };
        ok = load(sK + kr.slot * C::kTileBytes, &tm_k, k_full + kr.slot, k_empty + kr.slot, kr.pass);
        if (!ok) break;
        kr.next(C::kKSlots);
        ok = load(sV + vr.slot * C::kTileBytes, &tm_v, v_full + vr.slot, v_empty + vr.slot, vr.pass);
        if (!ok) break;
        vr.next(C::kVSlots);
      }
      more = ok && walk.next(p);
    }
    // On the way out of a failed wait copies in flight land first (an unused slot's wait ends
    // at once).
    if (!ok && issue) {
      for (int i = 0; i < C::kKSlots; ++i, kr.next(C::kKSlots)) wait_drain(k_full + kr.slot, kr.pass ^ 1);
      for (int i = 0; i < C::kVSlots; ++i, vr.next(C::kVSlots)) wait_drain(v_full + vr.slot, vr.pass ^ 1);
      for (int i = 0; i < 2; ++i)
        if (q_armed >> i & 1) wait_drain(q_full + i, (q_seen >> i & 1) ^ 1);
    }
  } else if (warp == kShQK) {
    constexpr uint32_t kIdesc = idesc_bf16(128, kShKeys, false);
    const uint64_t dQ = sdesc_sw128(smem_u32(sQ), 16, 1024);
    const uint64_t dK = sdesc_sw128(smem_u32(sK), 16, 1024);
    ShRing kr;
    uint32_t q_pass = 0, half = 0, s_pass = 0;  // q_pass: a bit per half of the rows
    bool ok = true;
    ShMsg m;
    while (ok && next_msg(m, ok)) {
      if (m.shared) half = 0;
      ok = sh_wait(q_full + half, q_pass >> half & 1, wd);
      q_pass ^= 1u << half;
      for (int t = 0; t < m.tiles && ok; ++t) {
        // once the tile is there and the scores before it have been read
        ok = sh_wait(k_full + kr.slot, kr.pass, wd) && sh_wait(s_free, s_pass ^ 1, wd);
        if (!ok) break;
        s_pass ^= 1;
        tc_fence_after();
        const uint64_t q0 = dQ + (uint64_t)((half * C::kHalf) >> 4);
        const uint64_t k0 = dK + (uint64_t)((kr.slot * C::kTileBytes) >> 4);
        uint64_t a[D / 16], b[D / 16];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          a[kk] = q0 + (uint64_t)(((kk / 4) * C::kQBox + (kk % 4) * 32) >> 4);
          b[kk] = k0 + (uint64_t)(((kk / 4) * C::kBox + (kk % 4) * 32) >> 4);
        }
        mma_ss_warp<D / 16>(tmem, a, b, kIdesc, 0u);
        mma_commit_warp(s_full);
        mma_commit_warp(k_empty + kr.slot);
        kr.next(C::kKSlots);
      }
      if (!ok) break;
      mma_commit_warp(q_empty + half);
      if (m.shared) mma_commit_warp(q_empty + 1);
      half = m.shared ? 0 : half ^ 1;
    }
    mma_commit_warp(drain);
    __syncwarp();
    wait_drain(drain, 0);
  } else if (warp == kShPV) {
    constexpr uint32_t kIdesc = idesc_bf16(128, D, true);
    const uint64_t dV = sdesc_sw128(smem_u32(sV), C::kBox, 1024);
    ShRing vr;
    uint32_t p_pass = 0, o_pass = 0, place = 0;  // place: of the next P
    bool ok = true;
    ShMsg m;
    while (ok && next_msg(m, ok)) {
      const bool apart = m.shared && (p.variant & ATTN_MASK_WINDOW) &&
                         sh_apart(p, m.seq, m.nseq, max(m.klo, m.key0),
                                  min(m.khi, m.key0 + m.tiles * kShKeys));
      for (int t = 0; t < m.tiles && ok; ++t) {
        ok = sh_wait(v_full + vr.slot, vr.pass, wd);
        // Values of keys that no row of the block sees are zeroed before their product (P is 0
        // there, and they may be anything).
        const int j0 = m.key0 + t * kShKeys;
        if (ok && (apart || j0 < m.klo || j0 + kShKeys > m.khi)) {
#pragma unroll 1
          for (int at = 0; at < kShKeys; at += 32) {
            unsigned seen = sh_span(m.klo - j0 - at, m.khi - j0 - at);
            if (apart) seen &= sh_seen(p, m.seq, m.nseq, j0 + at);
            if (seen == ~0u) continue;
            uint8_t* rows = sV + vr.slot * C::kTileBytes + at * 128 + lane * 16;
#pragma unroll
            for (int r = 0; r < 32; r += 4)  // four rows of 128 bytes
              if (!(seen >> (r + lane / 8) & 1))
#pragma unroll
                for (int bx = 0; bx < C::kBoxes; ++bx)
                  *reinterpret_cast<uint4*>(rows + bx * C::kBox + r * 128) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (ok && t == 0) {  // O of the piece before has been read
          ok = sh_wait(o_free, o_pass ^ 1, wd);
          o_pass ^= 1;
        }
        ok = ok && sh_wait(p_full, p_pass, wd);
        if (!ok) break;
        p_pass ^= 1;
        tc_fence_after();
        const uint64_t v0 = dV + (uint64_t)((vr.slot * C::kTileBytes) >> 4);
        uint32_t a[kShKeys / 16];
        uint64_t b[kShKeys / 16];
#pragma unroll
        for (int kk = 0; kk < kShKeys / 16; ++kk) {
          a[kk] = tmem + C::kColP + kShKeys / 2 * place + kk * 8;
          b[kk] = v0 + (uint64_t)((kk * 16 * 128) >> 4);
        }
        mma_ts_warp<kShKeys / 16>(tmem + C::kColO, a, b, kIdesc, t > 0 ? 1u : 0u);
        mma_commit_warp(pv_done);
        mma_commit_warp(v_empty + vr.slot);
        place ^= 1;
        vr.next(C::kVSlots);
      }
    }
    mma_commit_warp(drain);
    __syncwarp();
    wait_drain(drain, 0);
  } else if (warp < kShProducer) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kShRegsSoftmax));
    const int t = threadIdx.x;  // row of the block, TMEM lane
    const uint32_t lanes = uint32_t(warp * 32) << 16;
    const uint32_t colO = tmem + lanes + C::kColO;
    const bool causal = p.variant & ATTN_MASK_CAUSAL, windowed = p.variant & ATTN_MASK_WINDOW;
    // the row's sequence of the block, its head of the group and its token
    const int rq = t / p.R, rr = t - rq * p.R, rg = rr / p.Sq, rs = rr - rg * p.Sq;
    uint32_t s_pass = 0, pv_count = 0;  // pv_count: tiles before this one
    bool ok = true;
    ShMsg msg;
    int known = -1;  // first sequence of the rows that `len` was read for
    int len = 0;
    while (ok && next_msg(msg, ok)) {
      const int rows = msg.nseq * p.R;
      const bool mine = t < rows, active = warp * 32 < rows;  // a warp without rows keeps step
      if (!msg.shared) {
        len = msg.khi;
        known = -1;
      } else if (known != msg.seq) {
        known = msg.seq;
        len = mine ? sh_len(p, msg.seq + rq) : 0;
      }
      const int pos = len - p.Sq + rs;
      int lo = 0, hi = 0;  // keys that the row sees
      if (mine && pos >= 0) {
        hi = min(msg.khi, causal ? pos + 1 : len);
        lo = max(msg.klo, windowed ? pos - p.window + 1 : 0);
      }
      float slope2 = 0.0f;
      if constexpr (SCORE & 1) {
        const int hq = msg.h * (p.Hq / p.Hkv) + (mine ? rg : 0);
        slope2 = (p.slopes ? p.slopes[hq] : exp2f(-8.0f * float(hq + 1) / float(p.Hq))) * kLog2e;
      }
      float m = -INFINITY, l = 0.0f;
      for (int i = 0; i < msg.tiles; ++i) {
        const int j0 = msg.key0 + i * kShKeys;
        const int from = lo - j0, to = hi - j0;  // columns that the row sees
        const bool whole = __all_sync(0xffffffffu, !mine || (from <= 0 && to >= kShKeys));
        ok = sh_wait(s_full, s_pass, wd);
        if (!ok) break;
        s_pass ^= 1;
        tc_fence_after();
        float x[64];
        uint32_t(&v0)[32] = *reinterpret_cast<uint32_t(*)[32]>(x);
        uint32_t(&v1)[32] = *reinterpret_cast<uint32_t(*)[32]>(x + 32);
        tmem_ld32(tmem + lanes, v0);
        tmem_ld32(tmem + lanes + 32, v1);
        tmem_ld_wait_regs(v0);
        tmem_ld_wait_regs(v1);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_free);
        if (active) {
          sh_modify<SCORE>(p, slope2, pos - j0, mine, x);
          if (!whole) {
#pragma unroll
            for (int c = 0; c < 64; ++c) x[c] = c >= from && c < to ? x[c] : -INFINITY;
          }
          const float scale = SCORE == 0 ? p.scale2 : 1.0f;
          const float mt = row_max<64>(x) * scale;
          // The reference moves when a row's scores pass it by 2^8, or when it has none.
          const bool move = mine && mt > m + 8.0f;
          if (__any_sync(0xffffffffu, move)) {
            const float m_new = move ? mt : m;
            const float fix = move ? ex2_approx(m - m_new) : 1.0f;  // from -inf: 0
            if (i > 0) {  // O as the tile before left it
              ok = sh_wait(pv_done, (pv_count & 1) ^ 1, wd);
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32(colO + c, o);
                tmem_ld_wait_regs(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fix);
                tmem_st32(colO + c, o);
              }
            }
            l *= fix;
            m = m_new;
          }
          const float ref = m == -INFINITY ? 0.0f : m;
          uint32_t pk[32];
          l += sh_exp32(x, scale, ref, pk);
          l += sh_exp32(x + 32, scale, ref, pk + 16);
          // (the place of the tile two before, whose product was waited for below)
          tmem_st32(tmem + lanes + C::kColP + kShKeys / 2 * (pv_count & 1), pk);
          tmem_st_wait();
        }
        // Every phase of pv_done is seen in turn: two that end unseen would look like none. (The
        // scores of a tile may come before the product of the one before.)
        if (i > 0) {
          ok = sh_wait(pv_done, (pv_count & 1) ^ 1, wd);
          if (!ok) break;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
        ++pv_count;
      }
      ok = ok && sh_wait(pv_done, (pv_count & 1) ^ 1, wd);
      if (!ok) break;
      tc_fence_after();
      if (active) {
        // the part's O / l and LSE (log2); rows of a column chunk side by side
        const int stride = msg.shared ? kTile : p.R;
        const bool there =
            mine && MATTN_IN_BOUNDS(kSiteShPart, msg.slot, msg.shared ? p.p_slots : p.s_slots);
        float* po = (msg.shared ? p.p_o : p.s_o) + msg.slot * stride * D;
        const bool none = l == 0.0f;  // no key: O = 0, LSE = -inf. NaN passes through
        const float inv = none ? 0.0f : 1.0f / l;
        if (there)
          ((msg.shared ? p.p_lse : p.s_lse) + msg.slot * stride)[t] = none ? -INFINITY : m + __log2f(l);
        float4* out = reinterpret_cast<float4*>(po) + t;
#pragma unroll 1
        for (int c = 0; c < D; c += 64) {
          uint32_t o[2][32];
          tmem_ld32(colO + c, o[0]);
          tmem_ld32(colO + c + 32, o[1]);
          tmem_ld_wait_regs(o[0]);
          tmem_ld_wait_regs(o[1]);
          if (there) {
#pragma unroll
            for (int e = 0; e < 64; e += 4, out += stride) {
              const uint32_t* v = o[e / 32] + e % 32;
              *out = none ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                          : make_float4(__uint_as_float(v[0]) * inv, __uint_as_float(v[1]) * inv,
                                        __uint_as_float(v[2]) * inv, __uint_as_float(v[3]) * inv);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kShQK) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// ------------------------------------------------------------------------- the join
// A block joins the rows of one sequence and key/value head. A warp lists their parts; then a
// thread takes 4 channels of a row, and where rows are few the parts are spread over groups of
// threads, whose results meet in shared memory. Bound by latency: the sequence, its pieces, then
// the parts, four loads of them at a time. Everything in a fixed order.
constexpr int kShJoinThreads = 256;

struct ShAcc {
  float m, l;
  float4 o;
  __device__ __forceinline__ void add(float e, float w, const float4& x) {  // w: weight of part e
    const float to = fmaxf(m, e), ref = to == -INFINITY ? 0.0f : to;
    const float fix = ex2_approx(m - ref), k = w * ex2_approx(e - ref);  // -inf -> 0
    l = l * fix + k;
    o = make_float4(o.x * fix + k * x.x, o.y * fix + k * x.y, o.z * fix + k * x.z, o.w * fix + k * x.w);
    m = to;
  }
};

template <int D>
__global__ void __launch_bounds__(kShJoinThreads) shared_join_kernel(const ShProblem p) {
  extern __shared__ int parts[];  // slots of the partial results, ~slot for the own keys'
  __shared__ float4 other_o[kShJoinThreads];
  __shared__ float other_m[kShJoinThreads], other_l[kShJoinThreads];
  __shared__ int n_parts;
  const int tid = threadIdx.x, lane = tid & 31;
  const int b = blockIdx.x / p.Hkv, h = blockIdx.x % p.Hkv;
  early_start();
  const ShSeq s = p.seqs[b];
  if (tid < 32) {
    const ShHead head = *p.head;
    const int pieces = s.chunks + (s.sdesc >= 0);
    int n = 0;
    for (int i0 = 0; i0 < pieces; i0 += 32) {
      const int i = i0 + lane;
      int first = 0, count = 0;
      if (i < pieces) {
        const bool own = i == s.chunks;
        const ShDesc d = p.desc[own ? s.sdesc : s.pdesc + i];
        const int piece = own ? h : h * d.blocks + s.block;
        const long long start = d.start + piece * sh_length(d.blocks, d.tiles) + kShCost;
        const int c0 = (int)sh_div(start, head.share);
        const long long last = start + (long long)(d.tiles - 1) * sh_weight(d.blocks);
        count = (int)sh_div(last, head.share) - c0 + 1;
        first = d.base + piece + c0;
        if (own) first = ~first;
      }
      int before = count;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, before, d);
        if (lane >= d) before += o;
      }
      const int total = __shfl_sync(0xffffffffu, before, 31);
      before += n - count;
      for (int k = 0; k < count; ++k)
        if (MATTN_IN_BOUNDS(kSiteShPart, before + k, p.max_parts))
          parts[before + k] = first < 0 ? first - k : first + k;
      n += total;
    }
    if (lane == 0) n_parts = n;
  }
  __syncthreads();
  const int n = n_parts, per = p.R * (D / 4);
  const bool wide = per >= kShJoinThreads;  // several items per thread; else one, and groups
  const int groups = wide ? 1 : kShJoinThreads / per, group = wide ? 0 : tid / per;
  for (int item = wide ? tid : tid - group * per; item < per; item += wide ? kShJoinThreads : per) {
    const int r = item % p.R, c4 = item / p.R;
    ShAcc a{-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
    if (group < groups) {
      for (int k0 = group; k0 < n; k0 += 4 * groups) {
        float e[4];
        float4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = k0 + i * groups;
          e[i] = -INFINITY;
          x[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (k < n) {
            const int part = parts[k];
            const bool own = part < 0;
            const long long slot = own ? ~part : part;
            const int stride = own ? p.R : kTile, row = own ? r : s.row0 + r;
            if (MATTN_IN_BOUNDS(kSiteShPart, slot, own ? p.s_slots : p.p_slots)) {
              e[i] = (own ? p.s_lse : p.p_lse)[slot * stride + row];
              x[i] = reinterpret_cast<const float4*>((own ? p.s_o : p.p_o) +
                                                     slot * stride * D)[c4 * stride + row];
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) a.add(e[i], 1.0f, x[i]);
      }
    }
    if (groups > 1) {
      other_m[tid] = a.m;
      other_l[tid] = a.l;
      other_o[tid] = a.o;
      __syncthreads();
      if (group > 0) return;
      for (int g = 1; g < groups; ++g) {
        const int at = g * per + item;
        const float l = other_l[at], inv = l != 0.0f ? 1.0f / l : 0.0f;
        const float4 x = other_o[at];
        a.add(other_m[at], l, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
      }
    } else if (group > 0) {
      return;  // a thread left over
    }
    const long long row = ((long long)b * p.Hq + (long long)h * (p.Hq / p.Hkv)) * p.Sq + r;
    if (!MATTN_IN_BOUNDS(kSiteShOut, row, (long long)p.B * p.Hq * p.Sq)) continue;
    const bool any = !(a.l == 0.0f);
    const float inv = any ? 1.0f / a.l : 0.0f;
    const uint2 out = any ? make_uint2(pack_bf16x2(a.o.x * inv, a.o.y * inv),
                                       pack_bf16x2(a.o.z * inv, a.o.w * inv))
                          : make_uint2(0u, 0u);
    reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + row * D)[c4] = out;
    if (c4 == 0) p.lse[row] = any ? (a.m + __log2f(a.l)) * kLn2 : -INFINITY;
  }
}

// ------------------------------------------------------------------------- host side
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

struct ShLayout {
  int ctas, max_desc, max_prefix;
  long long p_slots, s_slots;
  size_t desc, seqs, p_lse, p_o, s_lse, s_o, total;
};

ShLayout sh_layout(int B, int Hq, int Hkv, int Sq, int G, int max_len, int D) {
  ShLayout w;
  const long long R = (long long)Hq / Hkv * Sq, per_block = std::max(1LL, kTile / R);
  // two CTAs per SM, or one per tile where there are fewer (a sequence's own keys may begin
  // inside a tile)
  const long long tiles = (long long)B * Hkv * (((long long)max_len + kShKeys - 1) / kShKeys + 1);
  w.ctas = (int)std::max(1LL, std::min<long long>(kShPerSm * sm_count(), tiles));
  // Chunks of shared keys: each holds half of a CTA's share of the tiles or more, but for one of
  // each group; so chunks * blocks of all groups are at most 2 ctas / Hkv and the blocks
  // themselves, the chunks no more than that.
  const long long shared = std::min(G, B / 2);
  w.max_prefix = shared ? (int)(2 * w.ctas / Hkv + B / per_block + shared + 1) : 0;
  w.max_desc = w.max_prefix + B;
  w.p_slots = shared ? w.ctas + (long long)w.max_prefix * Hkv : 0;
  w.s_slots = w.ctas + (long long)B * Hkv;
  size_t at = up256(sizeof(ShHead));
  auto take = [&](size_t n) {
    const size_t x = at;
    at += up256(n);
    return x;
  };
  w.desc = take(sizeof(ShDesc) * w.max_desc);
  w.seqs = take(sizeof(ShSeq) * B);
  w.p_lse = take(sizeof(float) * w.p_slots * kTile);
  w.s_lse = take(sizeof(float) * w.s_slots * R);
  w.p_o = take(sizeof(float) * w.p_slots * kTile * D);
  w.s_o = take(sizeof(float) * w.s_slots * R * D);
  w.total = at;
  return w;
}

// 4-D view [B][Hkv][R][D] of the queries; box: `seqs` sequences' rows of one key/value head.
bool make_map_rows(CUtensorMap* map, const void* q, int B, int Hkv, int R, int D, int seqs) {
  EncodeTiledFn fn = get_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)R, (cuuint64_t)Hkv, (cuuint64_t)B};
  cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)R * D * 2, (cuuint64_t)Hkv * R * D * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)R, 1, (cuuint32_t)seqs};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct ShMaps {
  CUtensorMap qs, q1, k, v;
};

template <int D, int SCORE>
cudaError_t launch_main(const ShMaps& m, const ShProblem& p, cudaStream_t s) {
  using C = ShCfg<D>;
  static DeviceOnce ready;
  cudaError_t e = ready.allow_smem(decode_shared_kernel<D, SCORE>, C::kSmem);
  if (e != cudaSuccess) return e;
  // setmaxnreg.inc draws on the registers that the block holds: refuse where they do not cover
  // the split (the increase would wait for ever)
  static KernelRegs known;
  int regs = 0;
  if ((e = known.get(decode_shared_kernel<D, SCORE>, regs)) != cudaSuccess) return e;
  if (128 * (kShRegsSoftmax + kShRegsOther) > regs * kShThreads) return cudaErrorInvalidConfiguration;
  return launch_early(decode_shared_kernel<D, SCORE>, (unsigned)p.ctas, kShThreads, C::kSmem, s,
                      m.qs, m.q1, m.k, m.v, p);
}

template <int D>
cudaError_t launch_shared(const void* q, const void* k, const void* v, ShProblem& p,
                          cudaStream_t s) {
  ShMaps m;
  const long long slices = (long long)p.num_pages * p.Hkv;
  if (!make_map_rows(&m.qs, q, p.B, p.Hkv, p.R, D, p.seqs_per_block) ||
      !make_map_rows(&m.q1, q, p.B, p.Hkv, p.R, D, 1) ||
      !make_map_bf16_3d(&m.k, k, slices, 1 << p.shift, D, std::min(kShKeys, 1 << p.shift)) ||
      !make_map_bf16_3d(&m.v, v, slices, 1 << p.shift, D, std::min(kShKeys, 1 << p.shift)))
    return cudaErrorInvalidValue;
  const size_t plan_smem = sizeof(int) * (((p.B + 3) & ~3) + ((p.G + 4) & ~3)) + sizeof(ShGroup) * p.G;
  static DeviceOnce ready;
  cudaError_t e = ready.allow_smem(shared_plan_kernel, 226 * 1024 - 1024);
  if (e != cudaSuccess) return e;
  e = launch_early(shared_plan_kernel, 1u, kShPlanThreads, plan_smem, s, p);
  if (e != cudaSuccess) return e;
  switch (((p.variant & ATTN_SCORE_ALIBI) ? 1 : 0) | ((p.variant & ATTN_SCORE_SOFTCAP) ? 2 : 0)) {
    case 0: e = launch_main<D, 0>(m, p, s); break;
    case 1: e = launch_main<D, 1>(m, p, s); break;
    case 2: e = launch_main<D, 2>(m, p, s); break;
    default: e = launch_main<D, 3>(m, p, s);
  }
  if (e != cudaSuccess) return e;
  return launch_early(shared_join_kernel<D>, (unsigned)(p.B * p.Hkv), kShJoinThreads,
                      sizeof(int) * p.max_parts, s, p);
}

}  // namespace
}  // namespace mattn

MATTN_API size_t attn_decode_shared_workspace_bytes(int B, int Hq, int Hkv, int Sq, int G,
                                                    int max_len, int D) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Sq < 1 || G < 0 || max_len < 0 || (D != 64 && D != 128) ||
      Hq % Hkv || (long long)Hq / Hkv * Sq > mattn::kShMaxRows)
    return 0;
  return mattn::sh_layout(B, Hq, Hkv, Sq, G, max_len, D).total;
}

MATTN_API attn_status attn_decode_shared(const void* q, const void* k, const void* v, void* o,
                                         float* lse, int B, int Hq, int Hkv, int Sq, int max_len,
                                         int D, unsigned variant, const attn_params* p,
                                         const int* seq_lens, const int* group_starts,
                                         const int* shared_lens, int G, void* workspace,
                                         size_t workspace_bytes, struct CUstream_st* stream) {
  using namespace mattn;
  if (!p || B < 0 || Hq < 1 || Hkv < 1 || Sq < 0 || max_len < 0 || G < 0 || Hq % Hkv)
    return ATTN_ERR_INVALID_ARG;
  if (!p->page_table) return ATTN_ERR_INVALID_ARG;
  attn_status st = paged_args(variant, p, D);
  if (st != ATTN_OK) return st;
  if ((long long)(Hq / Hkv) * Sq > kShMaxRows || (long long)B * Hkv > 65535 || B > kShMaxB ||
      G > kShMaxB || max_len > INT_MAX - 65536 ||
      (long long)p->num_pages * Hkv + Hkv > INT_MAX)
    return ATTN_ERR_UNSUPPORTED;
  if (B == 0 || Sq == 0) return ATTN_OK;
  if ((long long)p->pages_per_seq * p->page_size < (long long)max_len) return ATTN_ERR_INVALID_ARG;
  if (!q || !k || !v || !o || !lse || !seq_lens || !workspace ||
      (G > 0 && (!group_starts || !shared_lens)))
    return ATTN_ERR_INVALID_ARG;
  const void* vecs[] = {q, k, v, o};
  for (const void* x : vecs)
    if (reinterpret_cast<uintptr_t>(x) & 15u) return ATTN_ERR_MISALIGNED;
  const void* words[] = {lse, seq_lens, group_starts, shared_lens, p->page_table, p->alibi_slopes};
  for (const void* x : words)
    if (reinterpret_cast<uintptr_t>(x) & 3u) return ATTN_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return ATTN_ERR_MISALIGNED;
  const ShLayout w = sh_layout(B, Hq, Hkv, Sq, G, max_len, D);
  if (workspace_bytes < w.total) return ATTN_ERR_WORKSPACE_TOO_SMALL;

  ShProblem f{};
  f.seq_lens = seq_lens;
  f.starts = group_starts;
  f.shared_lens = shared_lens;
  f.table = p->page_table;
  f.slopes = p->alibi_slopes;
  f.o = o;
  f.lse = lse;
  f.B = B;
  f.Hq = Hq;
  f.Hkv = Hkv;
  f.Sq = Sq;
  f.R = Hq / Hkv * Sq;
  f.G = G;
  f.max_len = max_len;
  f.seqs_per_block = kTile / f.R;
  f.shift = 4;
  while ((1 << f.shift) != p->page_size) ++f.shift;
  f.pages_per_seq = p->pages_per_seq;
  f.num_pages = p->num_pages;
  f.variant = variant;
  f.window = p->window;
  f.scale2 = (p->scale != 0.0f ? p->scale : 1.0f / std::sqrt((float)D)) * kLog2e;
  f.softcap2 = p->softcap * kLog2e;
  f.softcap_e = 2.0f / p->softcap;
  f.ctas = w.ctas;
  f.max_desc = w.max_desc;
  f.max_prefix = w.max_prefix;
  // a part per CTA and piece that meet, and a sequence's pieces lie one behind the other
  f.max_parts = w.ctas + w.max_prefix + 1;
  char* ws = static_cast<char*>(workspace);
  f.head = reinterpret_cast<ShHead*>(ws);
  f.desc = reinterpret_cast<ShDesc*>(ws + w.desc);
  f.seqs = reinterpret_cast<ShSeq*>(ws + w.seqs);
  f.p_lse = reinterpret_cast<float*>(ws + w.p_lse);
  f.p_o = reinterpret_cast<float*>(ws + w.p_o);
  f.s_lse = reinterpret_cast<float*>(ws + w.s_lse);
  f.s_o = reinterpret_cast<float*>(ws + w.s_o);
  f.p_slots = w.p_slots;
  f.s_slots = w.s_slots;
  f.status = p->status ? p->status : library_status();
  if (!f.status) return ATTN_ERR_CUDA;
  f.timeout_ns = p->timeout_ns ? p->timeout_ns : 4000000000ull;
  f.fault_inject = p->fault_inject;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return cuda_status(D == 64 ? launch_shared<64>(q, k, v, f, s) : launch_shared<128>(q, k, v, f, s));
}

namespace mattn {
MATTN_DEBUG_RECORD_ACCESSORS(decode_shared)
}  // namespace mattn
