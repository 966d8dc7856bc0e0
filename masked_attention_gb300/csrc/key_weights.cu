// The attention weight that each cached key received:
//
//   w[b][hk][j] = decay * previous[b][hk][j]
//                 + sum over the query rows (h, r) of key/value head hk that see key j of
//                   exp(score_mod(scale <q[b,h,r], k[b,hk,j]>) - LSE[b,h,r])
//
// from the queries and the LSE of an attention call that has run (one decode step, or the last
// tokens of a prompt); the sum over a head's keys of its new part is its number of rows.
//
// Every key row is read once for all query rows of its head: 2 D bytes against 2 D products a
// row, so HBM is the bound up to about 290 rows (group * Sq) and the tensor cores behind that; the
// special-function units, one exponential a score, would take 390 rows in a key's time.
//
// Scores are computed transposed, S^T = K Q^T, on tcgen05: 128 keys are the M of a product (TMEM
// lanes), up to 256 query rows its N. A key is then one thread's: its weight is a sum over that
// thread's own columns, in a fixed order, without a shuffle or an atomic, and bitwise
// reproducible whatever CTA has the tile.
//
// The tiles of 128 keys of all (sequence, key/value head) pairs, one after the other, are dealt
// out evenly to one CTA per SM. Warp 8 streams them by TMA (and the query rows, per pair or,
// with more than 256 of them, block by block for two tiles at a time), warp 9 issues the
// products, and two warpgroups take turns with the tiles, so that one's exponentials run under
// the other's product.
//
// 16 x 32768 keys of 8 heads of 128 channels, 4 rows each: 174 us, 6.4 TB/s of keys and weights,
// 0.93 of a copy's rate. 8 x 40960 keys, 256 rows: 158 us, 1.1 PFLOP/s, for 102 us of bytes; 512
// rows 323 us. There latency is the bound: tensor cores and special-function units are busy for a
// third of the time each and HBM little longer (2 x 40960 keys, 59 us), while the two warps of a
// scheduler that add the columns up wait, most of all on loads. Tiles in the masked form take
// about three times as long (240 rows, every tile masked: 459 us).
#include <algorithm>
#include <climits>
#include <cmath>

#include "host_util.h"
#include "launch.h"
#include "soft_cap.cuh"

#define MATTN_API extern "C" __attribute__((visibility("default")))

namespace mattn {
namespace {

constexpr int kKwThreads = 320;
constexpr int kKwProducer = 8, kKwMma = 9;  // warps; 0 to 7: two warpgroups
constexpr int kKwMaxN = 256;                // query rows of one product
constexpr int kKwMaxSlots = 8;  // tiles of keys
constexpr int kKwQSlots = 2;    // blocks of query rows

struct KwProblem {
  const float* lse;
  const float* previous;  // or nullptr
  float* weights;
  const int* seq_lens;  // or nullptr: max_len each
  const int* table;     // or nullptr: contiguous keys
  const float* slopes;
  int B, Hq, Hkv, Sq, D, max_len, stride;  // stride: row length of the weights
  int shift, pages_per_seq, num_pages;
  unsigned variant;
  int window;
  float decay, scale2, softcap2, softcap_e;  // scale and cap in log2 units
  int n_cols, blocks;                        // query rows per product, products per tile
  int k_slots;
  int* status;
  uint64_t timeout_ns;
  unsigned fault_inject;
};

struct KwRange {
  int len, first, tiles;  // keys, first visible tile, tiles from there on
};

__device__ __forceinline__ KwRange kw_range(const KwProblem& p, int b) {
  KwRange r;
  r.len = p.max_len;
  if (p.seq_lens) r.len = max(0, min(p.seq_lens[b], p.max_len));
  r.first = 0;
  if (p.variant & ATTN_MASK_WINDOW)
    r.first = (int)(max(0ll, (long long)r.len - p.Sq - p.window + 1) / kTile);
  r.tiles = max(0, (r.len + kTile - 1) / kTile - r.first);
  return r;
}

// A CTA's walk over its tiles, the CTA's share of one pair after the other; every role walks
// alike. (Tile by tile a walk's bookkeeping cost the MMA warp 900 cycles each.)
struct KwWalk {
  int b, hk, tile;  // tile counts from the sequence's first visible one
  long long left;   // tiles still to go
  KwRange r;
  __device__ __forceinline__ int run() const {  // tiles of this pair
    return (int)min(left, (long long)(r.tiles - tile));
  }
  __device__ __forceinline__ void next_pair(const KwProblem& p) {
    left -= run();
    tile = 0;
    if (left <= 0 || ++hk < p.Hkv) return;
    hk = 0;
    do r = kw_range(p, ++b);
    while (r.tiles == 0 && b + 1 < p.B);  // left > 0: a later sequence has tiles
  }
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// The wait, naming the registers so that no use moves above it.
__device__ __forceinline__ void tmem_ld16_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// One column, read and waited for.
__device__ __forceinline__ float tmem_column(uint32_t taddr) {
  uint32_t x;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(x) : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(x) : : "memory");
  return __uint_as_float(x);
}

__device__ __forceinline__ bool kw_wait(uint64_t* bar, uint32_t parity, const Watchdog& wd) {
  // a sleeping try first: the timer that bounds the wait takes long to read
  const uint32_t hint = wd.timeout_ns < 1000000ull ? (uint32_t)wd.timeout_ns : 1000000u;
  const bool done = mbar_try_wait(bar, parity) || mbar_try_wait_sleep(bar, parity, hint) ||
                    wait_bounded(bar, parity, wd);
  return __all_sync(0xffffffffu, done);
}

// A place in a ring of `n` buffers and the parity of its pass. (Counted, not divided out: a
// division by the ring's length takes a lone warp some 150 cycles, and four of them a tile
// were what bounded one decode step.)
struct KwRing {
  uint32_t slot = 0, pass = 0;
  __device__ __forceinline__ void next(uint32_t n) {
    if (++slot == n) {
      slot = 0;
      pass ^= 1;
    }
  }
};

// What a warpgroup keeps of a block's query rows (columns of the product), in shared memory.
struct KwColumns {
  float nlse[kKwMaxN];   // -LSE in log2 units; -inf: the column adds nothing
  float slope[kKwMaxN];  // ALiBi slope in log2 units
  int pos[kKwMaxN];      // the row's position; -1: none
  int skip[4];           // per warp: a row without an LSE is among its columns
};

// Sum over COLS columns of exp2(score - lse) for the thread's key j.
template <int SCORE, bool kMask, int COLS>
__device__ __forceinline__ void kw_add(const KwProblem& p, const KwColumns& col, int c0, int j,
                                       int len, const uint32_t* v, float2 (&sum)[4]) {
  const bool causal = p.variant & ATTN_MASK_CAUSAL, windowed = p.variant & ATTN_MASK_WINDOW;
  const float2 sl = make_float2(p.scale2, p.scale2);
#pragma unroll
  for (int c = 0; c < COLS; c += 4) {
    // keeps the reads of later columns' constants behind (they would fill the registers)
    if (c % 16 == 0) asm volatile("" ::: "memory");
    const float4 nl = *reinterpret_cast<const float4*>(col.nlse + c0 + c);
    int4 pos;
    float4 slope;
    if constexpr (kMask || (SCORE & 1)) pos = *reinterpret_cast<const int4*>(col.pos + c0 + c);
    if constexpr (SCORE & 1) slope = *reinterpret_cast<const float4*>(col.slope + c0 + c);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 s = make_float2(__uint_as_float(v[c + 2 * h]), __uint_as_float(v[c + 2 * h + 1]));
      const float2 n = h ? make_float2(nl.z, nl.w) : make_float2(nl.x, nl.y);
      float2 x;
      if constexpr (SCORE == 0) {
        x = ffma2(s, sl, n);
      } else {
        x = fmul2(s, sl);
        if constexpr (SCORE & 1) {
          const float2 m = h ? make_float2(slope.z, slope.w) : make_float2(slope.x, slope.y);
          x.x -= m.x * float((h ? pos.z : pos.x) - j);
          x.y -= m.y * float((h ? pos.w : pos.y) - j);
        }
        if constexpr (SCORE & 2) {
          x.x = soft_cap(x.x, p.softcap2, p.softcap_e);
          x.y = soft_cap(x.y, p.softcap2, p.softcap_e);
        }
        x = fadd2(x, n);
      }
      float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
      if constexpr (kMask) {
        auto keep = [&](int i) {
          return i >= 0 && (causal ? j <= i : j < len) && (!windowed || i - j < p.window);
        };
        e.x = keep(h ? pos.z : pos.x) ? e.x : 0.0f;
        e.y = keep(h ? pos.w : pos.y) ? e.y : 0.0f;
      }
      const int a = (c / 2 + h) & 3;
      sum[a] = fadd2(sum[a], e);
    }
  }
}

template <int D, int SCORE>
__global__ void __launch_bounds__(kKwThreads, 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k, const KwProblem p) {
  constexpr int kBoxes = D / 64;
  constexpr int kBoxBytes = kTile * 128;
  constexpr int kTileBytes = kBoxes * kBoxBytes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int q_box = p.n_cols * 128, q_bytes = kBoxes * q_box;  // n_cols % 16 == 0: 2048 | q_box
  uint8_t* sQ = smem;
  uint8_t* sK = smem + kKwQSlots * q_bytes;
  __shared__ __align__(16) KwColumns columns[2];
  __shared__ uint64_t bars[11 + 2 * kKwMaxSlots];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_word;
  __shared__ long long run_sum[kKwThreads];
  __shared__ long long first_tile, total_tiles;
  __shared__ int first_b;
  uint64_t *q_full = bars, *q_empty = bars + 2, *s_full = bars + 4, *s_free = bars + 6,
           *drain = bars + 8, *wg_bar = bars + 9, *k_full = bars + 11,
           *k_empty = k_full + kKwMaxSlots;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &abort_word;
  const Watchdog wd{abort_flag, p.status, p.timeout_ns};

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(q_empty + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(s_free + i, 4);
      mbar_init(wg_bar + i, 4);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < p.k_slots; ++i) {
      mbar_init(k_full + i, 1);
      mbar_init(k_empty + i, 1);
    }
    abort_word = 0;
    first_tile = 0;
    first_b = p.B;
    fence_barrier_init();
  }
  if (warp == kKwMma) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == kKwProducer && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
  }
  early_start();

  // This CTA's tiles [lo, hi) of all: a thread adds up a run of sequences.
  const int run = (p.B + kKwThreads - 1) / kKwThreads;
  const int r0 = min((int)threadIdx.x * run, p.B), r1 = min(r0 + run, p.B);
  long long own = 0;
  for (int b = r0; b < r1; ++b) own += (long long)kw_range(p, b).tiles * p.Hkv;
  run_sum[threadIdx.x] = own;
  __syncthreads();
  if (warp == 0) {  // exclusive sums of the runs, 10 threads' at a time
    constexpr int per = kKwThreads / 32;
    long long s = 0;
#pragma unroll
    for (int i = 0; i < per; ++i) s += run_sum[lane * per + i];
    long long before = s;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, before, d);
      if (lane >= d) before += o;
    }
    if (lane == 31) total_tiles = before;
    before -= s;
#pragma unroll
    for (int i = 0; i < per; ++i) {
      const long long mine = run_sum[lane * per + i];
      run_sum[lane * per + i] = before;
      before += mine;
    }
  }
  __syncthreads();
  const long long total = total_tiles;
  const long long share = (total + gridDim.x - 1) / gridDim.x;
  const long long lo = min(total, blockIdx.x * share), hi = min(total, lo + share);
  {
    long long at = run_sum[threadIdx.x];
    for (int b = r0; b < r1 && at <= lo; ++b) {
      const long long n = (long long)kw_range(p, b).tiles * p.Hkv;
      if (lo < at + n) {
        first_b = b;
        first_tile = lo - at;
      }
      at += n;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  KwWalk walk{};
  walk.left = hi - lo;
  if (walk.left > 0) {
    walk.b = first_b;
    walk.r = kw_range(p, walk.b);
    walk.hk = (int)(first_tile / walk.r.tiles);
    walk.tile = (int)(first_tile % walk.r.tiles);
  }
  const int R = p.Hq / p.Hkv * p.Sq;

  if (warp == kKwProducer) {
    const bool issue = !(p.fault_inject & ATTN_FAULT_NO_LOADS);
    KwRing kr, qr;
    bool ok = true;
    // A lane per page of a tile, its table entry read one tile ahead. Pages past the last one
    // with keys repeat it (their keys are masked); one outside the pool reads as zeros (past
    // the map's end).
    auto page_of = [&](const KwWalk& w, int i) {
      if (!p.table || lane >= (kTile >> p.shift)) return 0;
      const int lp = min(((w.r.first + w.tile + i) * kTile >> p.shift) + lane,
                         (w.r.len - 1) >> p.shift);
      int phys = -1;
      if (MATTN_IN_BOUNDS(kSiteKwTable, lp, p.pages_per_seq))
        phys = p.table[(size_t)w.b * p.pages_per_seq + lp];
      return phys;
    };
    auto load_rows = [&](int nb, int pair) {
      if (!kw_wait(q_empty + qr.slot, qr.pass ^ 1, wd)) return false;
      if (lane == 0 && issue) {
        mbar_arrive_expect_tx(q_full + qr.slot, q_bytes);
#pragma unroll
        for (int bx = 0; bx < kBoxes; ++bx)
          tma_load_3d(sQ + qr.slot * q_bytes + bx * q_box, &tm_q, q_full + qr.slot, bx * 64,
                      nb * p.n_cols, pair);
      }
      __syncwarp();
      qr.next(kKwQSlots);
      return true;
    };
    while (walk.left > 0 && ok) {
      const int run = walk.run(), pair = walk.b * p.Hkv + walk.hk;
      int page = page_of(walk, 0);
      for (int i = 0; i < run && ok; ++i) {
        // blocks of rows go before every group of tiles, their first one before the tiles
        if (p.blocks > 1 ? (i & 1) == 0 : i == 0) ok = load_rows(0, pair);
        ok = ok && kw_wait(k_empty + kr.slot, kr.pass ^ 1, wd);
        if (!ok) break;
        uint64_t* full = k_full + kr.slot;
        uint8_t* dst = sK + kr.slot * kTileBytes;
        if (lane == 0 && issue) mbar_arrive_expect_tx(full, kTileBytes);
        __syncwarp();
        if (!p.table) {
          if (lane == 0 && issue)
#pragma unroll
            for (int bx = 0; bx < kBoxes; ++bx)
              tma_load_3d(dst + bx * kBoxBytes, &tm_k, full, bx * 64,
                          (walk.r.first + walk.tile + i) * kTile, pair);
        } else if (issue && lane < (kTile >> p.shift)) {
          const int phys = page < 0 || page >= p.num_pages ? p.num_pages : page;
#pragma unroll
          for (int bx = 0; bx < kBoxes; ++bx)
            tma_load_3d(dst + bx * kBoxBytes + (lane << p.shift) * 128, &tm_k, full, bx * 64, 0,
                        phys * p.Hkv + walk.hk);
        }
        if (i + 1 < run) page = page_of(walk, i + 1);
        __syncwarp();
        kr.next(p.k_slots);
        if (p.blocks > 1 && ((i & 1) || i + 1 == run))
          for (int nb = 1; nb < p.blocks && ok; ++nb) ok = load_rows(nb, pair);
      }
      walk.next_pair(p);
    }
    // On the way out of a failed wait copies in flight land first. The next pass of a slot not
    // begun, its latest copy is that of the pass before: parity pass ^ 1, which a slot that
    // was never used has too.
    if (!ok && issue) {
      for (int i = 0; i < p.k_slots; ++i, kr.next(p.k_slots))
        wait_drain(k_full + kr.slot, kr.pass ^ 1);
      for (int i = 0; i < kKwQSlots; ++i, qr.next(kKwQSlots))
        wait_drain(q_full + qr.slot, qr.pass ^ 1);
    }
  } else if (warp == kKwMma) {
    const uint32_t idesc = idesc_bf16(128, p.n_cols, false);
    const uint64_t a0 = sdesc_sw128(smem_u32(sK), 16, 1024);
    const uint64_t b0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
    KwRing kr, qr;
    uint32_t x = 0, s_pass = 0;  // s_pass: bit x is the parity of that warpgroup's buffer
    bool ok = true;
    // S^T of the tile in K slot `slot` and the query rows in use, for warpgroup x
    auto product = [&](uint32_t slot) {
      if (!kw_wait(s_free + x, ((s_pass >> x) & 1) ^ 1, wd)) return false;
      s_pass ^= 1u << x;
      tc_fence_after();
      const uint64_t ak = a0 + (uint64_t)((slot * kTileBytes) >> 4);
      const uint64_t bq = b0 + (uint64_t)((qr.slot * q_bytes) >> 4);
      uint64_t a[D / 16], b[D / 16];
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        a[kk] = ak + (uint64_t)(((kk / 4) * kBoxBytes + (kk % 4) * 32) >> 4);
        b[kk] = bq + (uint64_t)(((kk / 4) * q_box + (kk % 4) * 32) >> 4);
      }
      mma_ss_warp<D / 16>(tmem + kKwMaxN * x, a, b, idesc, 0u);
      mma_commit_warp(s_full + x);
      x ^= 1;
      return true;
    };
    while (walk.left > 0 && ok) {
      const int run = walk.run();
      if (p.blocks == 1) {
        ok = kw_wait(q_full + qr.slot, qr.pass, wd);
        for (int i = 0; i < run && ok; ++i) {
          ok = kw_wait(k_full + kr.slot, kr.pass, wd) && product(kr.slot);
          if (ok) mma_commit_warp(k_empty + kr.slot);
          kr.next(p.k_slots);
        }
        if (ok) mma_commit_warp(q_empty + qr.slot);
        qr.next(kKwQSlots);
      } else {
        for (int i = 0; i < run && ok; i += 2) {
          const int g = min(2, run - i);
          KwRing kn = kr;
          for (int nb = 0; nb < p.blocks && ok; ++nb) {
            ok = kw_wait(q_full + qr.slot, qr.pass, wd);
            kn = kr;
            x = 0;
            for (int m = 0; m < g && ok; ++m) {
              ok = (nb > 0 || kw_wait(k_full + kn.slot, kn.pass, wd)) && product(kn.slot);
              if (ok && nb == p.blocks - 1) mma_commit_warp(k_empty + kn.slot);
              kn.next(p.k_slots);
            }
            if (ok) mma_commit_warp(q_empty + qr.slot);
            qr.next(kKwQSlots);
          }
          kr = kn;
        }
      }
      walk.next_pair(p);
    }
    mma_commit_warp(drain);
    __syncwarp();
    wait_drain(drain, 0);
  } else if (warp < kKwProducer) {
    const uint32_t x = warp >> 2;     // warpgroup
    const int t = threadIdx.x & 127;  // key of the tile, TMEM lane
    const uint32_t cols = tmem + (uint32_t((warp & 3) * 32) << 16) + kKwMaxN * x;
    KwColumns& col = columns[x];
    // Keys before the first visible tile only decay.
    if (p.variant & ATTN_MASK_WINDOW) {
      for (long long pr = blockIdx.x; pr < (long long)p.B * p.Hkv; pr += gridDim.x) {
        const KwRange r = kw_range(p, (int)(pr / p.Hkv));
        const int n = min(r.first * kTile, r.len);
        for (int j = threadIdx.x; j < n; j += 256) {
          const size_t at = (size_t)pr * p.stride + j;
          if (MATTN_IN_BOUNDS(kSiteKwOut, at, (size_t)p.B * p.Hkv * p.stride))
            p.weights[at] = p.previous ? p.decay * p.previous[at] : 0.0f;
        }
      }
    }
    uint32_t turn = 0, s_it = 0, wg_it = 0;  // turn: the warpgroup of the pair's first tile
    bool ok = true;
    // The warpgroup meets (a bounded wait, so that no warp is left behind in one).
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(wg_bar + x);
      return kw_wait(wg_bar + x, wg_it++ & 1, wd);
    };
    // The columns of a (pair, block) are read one use ahead, two by each thread.
    float ahead[2];
    auto read_lse = [&](const KwWalk& w, int nb) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = t + 128 * i, row = nb * p.n_cols + c;
        ahead[i] = INFINITY;  // adds nothing
        if (c < p.n_cols && row < R) {
          const size_t at = ((size_t)w.b * p.Hq + (size_t)w.hk * (p.Hq / p.Hkv)) * p.Sq + row;
          if (MATTN_IN_BOUNDS(kSiteKwLse, at, (size_t)p.B * p.Hq * p.Sq)) ahead[i] = p.lse[at];
        }
      }
    };
    // A row whose LSE is -inf adds nothing, whatever its query holds: it has no position, and
    // the masked form of the sum, which leaves NaN out too, is taken for its block.
    bool skip = false;
    auto set_columns = [&](const KwWalk& w, int nb) {
      if (!meet()) return false;  // the block before has been used by all
      bool none = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = t + 128 * i, row = nb * p.n_cols + c;
        if (c < p.n_cols) {
          const bool empty = ahead[i] == -INFINITY, there = row < R;
          none |= empty;
          col.nlse[c] = empty ? -INFINITY : -ahead[i] * kLog2e;
          col.pos[c] = there && !empty ? w.r.len - p.Sq + row % p.Sq : -1;
          if constexpr (SCORE & 1) {
            const int h = w.hk * (p.Hq / p.Hkv) + (there ? row / p.Sq : 0);
            const float slope = p.slopes ? p.slopes[h] : exp2f(-8.0f * float(h + 1) / float(p.Hq));
            col.slope[c] = slope * kLog2e;
          }
        }
      }
      none = __any_sync(0xffffffffu, none);
      if (lane == 0) col.skip[warp & 3] = none;
      if (!meet()) return false;
      const int4 all = *reinterpret_cast<const int4*>(col.skip);
      skip = all.x | all.y | all.z | all.w;
      return true;
    };
    const bool causal = p.variant & ATTN_MASK_CAUSAL, windowed = p.variant & ATTN_MASK_WINDOW;
    if (walk.left > 0) read_lse(walk, 0);
    while (walk.left > 0 && ok) {
      const int run = walk.run(), len = walk.r.len;
      const size_t row0 = (size_t)(walk.b * p.Hkv + walk.hk) * p.stride;
      KwWalk next = walk;
      next.next_pair(p);
      if (p.blocks == 1) {
        ok = set_columns(walk, 0);
        if (!ok) break;
        if (next.left > 0) read_lse(next, 0);
      }
      for (int i0 = 0; i0 < run && ok; i0 += 2) {
        const int i = i0 + (int)(p.blocks > 1 ? x : x ^ turn);  // this warpgroup's tile
        const bool mine = i < run;
        const int j0 = (walk.r.first + walk.tile + i) * kTile, j = j0 + t;
        const bool whole = j0 + kTile <= len && len >= p.Sq &&
                           (!causal || j0 + kTile - 1 <= len - p.Sq) &&
                           (!windowed || len - 1 - j0 < p.window);
        const size_t at = row0 + j;
        const bool store = mine && j < len &&
                           MATTN_IN_BOUNDS(kSiteKwOut, at, (size_t)p.B * p.Hkv * p.stride);
        float old = 0.0f;
        if (store && p.previous) {
          old = p.previous[at];
          // a line per warp, to be in the L2 when its tile comes
          constexpr int kAhead = 8 * kTile;
          if (lane == 0 && j < len - kAhead)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.previous + at + kAhead));
        }
        float2 sum[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[k] = make_float2(0.0f, 0.0f);
        for (int nb = 0; nb < p.blocks && ok; ++nb) {
          if (p.blocks > 1) {
            ok = set_columns(walk, nb);
            if (!ok) break;
            if (nb + 1 < p.blocks) read_lse(walk, nb + 1);
            else if (i0 + 2 < run) read_lse(walk, 0);
            else if (next.left > 0) read_lse(next, 0);
          }
          if (!mine) continue;
          ok = kw_wait(s_full + x, s_it & 1, wd);
          if (!ok) break;
          ++s_it;
          tc_fence_after();
          auto columns_sum = [&](auto mask) {
            constexpr bool kMask = decltype(mask)::value;
            if (p.n_cols == 16) {
              uint32_t v[16];
              tmem_ld16(cols, v);
              tmem_ld16_wait(v);
              kw_add<SCORE, kMask, 16>(p, col, 0, j, len, v, sum);
              return;
            }
            // The next 32 columns are on their way while 32 are worked on (16 at a time, the
            // loads' latency bounded it: 3600 cycles for 256 columns). The last load of an even
            // number repeats the last columns: a load under a condition would cost registers.
            uint32_t v0[32], v1[32];
            tmem_ld32(cols, v0);
            int c = 0;
            for (; c + 64 <= p.n_cols; c += 64) {
              tmem_ld_wait_regs(v0);
              tmem_ld32(cols + c + 32, v1);
              kw_add<SCORE, kMask, 32>(p, col, c, j, len, v0, sum);
              tmem_ld_wait_regs(v1);
              tmem_ld32(cols + min(c + 64, p.n_cols - 32), v0);
              kw_add<SCORE, kMask, 32>(p, col, c + 32, j, len, v1, sum);
            }
            tmem_ld_wait_regs(v0);
            if (c < p.n_cols) kw_add<SCORE, kMask, 32>(p, col, c, j, len, v0, sum);
          };
          bool plain = whole && !skip;
          // Columns behind the head's rows hold zeros times the key: NaN where it has an infinity,
          // which the masked form leaves out (they have no position). The last one tells.
          if (plain && (nb + 1) * p.n_cols > R)
            plain = !__any_sync(0xffffffffu, isnan(tmem_column(cols + p.n_cols - 1)));
          if (plain) columns_sum(std::false_type{});
          else columns_sum(std::true_type{});
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_free + x);
        }
        if (store && ok) {
          const float2 s = fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3]));
          p.weights[at] = p.previous ? fmaf(p.decay, old, s.x + s.y) : s.x + s.y;
        }
      }
      turn = (turn + run) & 1;
      walk = next;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kKwMma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

constexpr int kKwSmem = 232448 - 12 * 1024;  // per CTA, less the static part

template <int D, int SCORE>
cudaError_t launch_typed(const CUtensorMap& mq, const CUtensorMap& mk, const KwProblem& p,
                         unsigned grid, size_t smem, cudaStream_t s) {
  static DeviceOnce ready;
  const cudaError_t e = ready.allow_smem(key_weights_kernel<D, SCORE>, kKwSmem);
  if (e != cudaSuccess) return e;
  return launch_early(key_weights_kernel<D, SCORE>, grid, kKwThreads, smem, s, mq, mk, p);
}

template <int D>
cudaError_t launch_key_weights(const void* q, const void* k, KwProblem& p, cudaStream_t s) {
  const int R = p.Hq / p.Hkv * p.Sq;
  // Query rows of a product: all, up to 256; more of them in blocks of like size.
  p.blocks = (R + kKwMaxN - 1) / kKwMaxN;
  p.n_cols = (R + p.blocks - 1) / p.blocks;
  p.n_cols = p.n_cols <= 16 ? 16 : (p.n_cols + 31) / 32 * 32;
  const int q_bytes = p.n_cols * D * 2, k_bytes = kTile * D * 2;
  // Two places for query rows leave two tiles of keys or more. (One place and four tiles for 256
  // rows of 128 channels: 8 x 40960 keys 160 us for 156, 64 x 704 keys 56 for 54; one place for
  // all: 64 x 704 keys and 4 rows 19.6 for 18.0.)
  p.k_slots = std::min(kKwMaxSlots, (kKwSmem - 1024 - kKwQSlots * q_bytes) / k_bytes);
  CUtensorMap mq, mk;
  const bool paged = p.table != nullptr;
  if (!make_map_bf16_3d(&mq, q, (long long)p.B * p.Hkv, R, D, p.n_cols) ||
      !make_map_bf16_3d(&mk, k, paged ? (long long)p.num_pages * p.Hkv : (long long)p.B * p.Hkv,
                        paged ? 1 << p.shift : p.max_len, D, paged ? 1 << p.shift : kTile))
    return cudaErrorInvalidValue;
  const size_t smem = 1024 + kKwQSlots * q_bytes + p.k_slots * k_bytes;
  const long long tiles = (long long)p.B * p.Hkv * ((p.max_len + kTile - 1) / kTile);
  const unsigned grid = (unsigned)std::min<long long>(sm_count(), tiles);
  switch (((p.variant & ATTN_SCORE_ALIBI) ? 1 : 0) | ((p.variant & ATTN_SCORE_SOFTCAP) ? 2 : 0)) {
    case 0: return launch_typed<D, 0>(mq, mk, p, grid, smem, s);
    case 1: return launch_typed<D, 1>(mq, mk, p, grid, smem, s);
    case 2: return launch_typed<D, 2>(mq, mk, p, grid, smem, s);
    default: return launch_typed<D, 3>(mq, mk, p, grid, smem, s);
  }
}

}  // namespace
}  // namespace mattn

MATTN_API attn_status attn_key_weights(const void* q, const void* k, const float* lse,
                                       const float* previous, float decay, float* weights, int B,
                                       int Hq, int Hkv, int Sq, int max_len, int D,
                                       int weights_stride, unsigned variant, const attn_params* p,
                                       const int* seq_lens, struct CUstream_st* stream) {
  using namespace mattn;
  if (!p || B < 0 || Hq < 1 || Hkv < 1 || Sq < 1 || max_len < 0 || Hq % Hkv ||
      weights_stride < max_len || !std::isfinite(decay))
    return ATTN_ERR_INVALID_ARG;
  attn_status st = paged_args(variant, p, D);
  if (st != ATTN_OK) return st;
  if ((long long)B * Hkv > 65535 || max_len > INT_MAX - 255 ||
      (long long)Hq / Hkv * Sq > INT_MAX / 256)
    return ATTN_ERR_UNSUPPORTED;
  if (B == 0 || max_len == 0) return ATTN_OK;
  if (p->page_table && (long long)p->pages_per_seq * p->page_size < (long long)max_len)
    return ATTN_ERR_INVALID_ARG;
  if (p->page_table && (long long)p->num_pages * Hkv + Hkv > INT_MAX) return ATTN_ERR_UNSUPPORTED;
  if (!k || !weights || !q || !lse) return ATTN_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k)) & 15u)
    return ATTN_ERR_MISALIGNED;
  const void* words[] = {lse, previous, weights, seq_lens, p->page_table, p->alibi_slopes};
  for (const void* x : words)
    if (reinterpret_cast<uintptr_t>(x) & 3u) return ATTN_ERR_MISALIGNED;
  // the previous weights are read where they are written, or apart
  const size_t bytes = (size_t)B * Hkv * weights_stride * sizeof(float);
  const char *a = reinterpret_cast<const char*>(previous), *w = reinterpret_cast<char*>(weights);
  if (a && a != w && a < w + bytes && w < a + bytes) return ATTN_ERR_INVALID_ARG;

  KwProblem f{};
  f.lse = lse;
  f.previous = decay != 0.0f ? previous : nullptr;
  f.weights = weights;
  f.seq_lens = seq_lens;
  f.table = p->page_table;
  f.slopes = p->alibi_slopes;
  f.B = B;
  f.Hq = Hq;
  f.Hkv = Hkv;
  f.Sq = Sq;
  f.D = D;
  f.max_len = max_len;
  f.stride = weights_stride;
  f.shift = 7;
  if (p->page_table)
    while ((1 << f.shift) != p->page_size) --f.shift;
  f.pages_per_seq = p->pages_per_seq;
  f.num_pages = p->num_pages;
  f.variant = variant;
  f.window = p->window;
  f.decay = decay;
  f.scale2 = (p->scale != 0.0f ? p->scale : 1.0f / std::sqrt((float)D)) * kLog2e;
  f.softcap2 = p->softcap * kLog2e;
  f.softcap_e = 2.0f / p->softcap;
  f.status = p->status ? p->status : library_status();
  if (!f.status) return ATTN_ERR_CUDA;
  f.timeout_ns = p->timeout_ns ? p->timeout_ns : 4000000000ull;
  f.fault_inject = p->fault_inject;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return cuda_status(D == 64 ? launch_key_weights<64>(q, k, f, s)
                             : launch_key_weights<128>(q, k, f, s));
}

namespace mattn {
MATTN_DEBUG_RECORD_ACCESSORS(key_weights)
}  // namespace mattn
