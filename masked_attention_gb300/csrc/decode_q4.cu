// Decode attention over the 4-bit paged cache (record layout: cache_q4.cuh):
// a few new query rows per sequence against sequences of their own lengths.
//
//   O = softmax(mask(mod(scale q K^T))) V,   K[j][c] = (n - 8) sK[j][c / 32],
//   V likewise. With group g's channels summed apart,
//   q . K[j] = sum_g sK[j][g] (q . (n - 8))_g,
// so the products run on the codes themselves, which bf16 and fp16 hold
// exactly, and the scales multiply fp32 sums (K) and the probabilities (V):
// no dequantised value is ever rounded.
//
// HBM is the floor: every visible record row is read once for all query rows
// of its key/value head (4.5 bits an element: 144 bytes a token at D = 128),
// 3.6 times less than the bf16 cache; so the instructions that unpack the
// codes are the near bound, and the layout of the products is chosen for them:
//  - scores are computed transposed, S^T = K q^T (mma m16n8k16: 16 keys, 8
//    query rows), and so is O^T = V^T P^T. The codes are then the A operand
//    (the 16-wide one), and up to 8 query rows cost one product, 9 to 16 two
//    that share the unpacked codes.
//  - ldmatrix on the packed bytes puts a key's 8 channels of one 32-channel
//    group into a lane (K), and with .trans four channels of two neighbouring
//    keys (V): both are what the A fragments need up to the order of the
//    channels, which q's fragments and O's rows follow. q's fragments stay in
//    shared memory: the registers go to more warps.
//  - a code n becomes the exact fp16 value n - 8 by one AND/OR into the mantissa
//    of 1024 or 64 and one packed subtraction, two codes at a time. (The bits
//    alone, as fp16 subnormals, need no subtraction, but the products then keep
//    about 14 bits below the largest: their sums are aligned to the exponents of
//    the operands as encoded. O was up to 2 % off.)
//  - P^T comes out of S^T's accumulators by movmatrix.
// P is rounded to fp16 after the V scale multiplied it: with y = score +
// log2(scale of the key's largest V group), the running reference m keeps
// 2^(y - m) <= 2^15 and at 2^8 for the largest key when m last moved, so fp16's
// 11 bits hold over 22 binades below the largest weighted scale of all groups, and
// 14 below that of each group while no key's V scales lie 2^8 or more apart. From the first
// tile on where a visible key's do (or are zero in a group that has values in other keys,
// or below 2^-98), a warp rounds P to two bf16 parts instead, which have 16 bits and
// fp32's range for every group by itself (16 sequences x 32768 keys: 164 us against 117;
// the test, a window of 8 binades that scales stay in, costs 1 % there, 3 % with a soft-cap
// and 6 % for short sequences: 80 x 16 heads x 1300 keys 64 -> 68). Groups that are zero in
// every key stay with fp16.
// m moves (and O and l are rescaled) only when a key passes its bound, which one vote per
// 32 keys decides. Sums are fp32.
//
// The tiles of 32 keys of all (sequence, key/value head) pairs, one after the
// other, are dealt out evenly: CTA c of C takes tiles [c N / C, (c + 1) N / C), so
// ragged lengths and few sequences load the SMs alike and the grid is one
// resident wave (16 sequences x 8 heads in equal splits of 8 CTAs per SM ran 2.1
// waves: 135 us against 125 of the kernel as it then was). A pair that lies within one CTA is written at once; one that
// is cut leaves fp32 partial results in the workspace, which a second, small
// kernel joins by the online-softmax merge (its start is programmatic: it is set
// up while the first one ends). Within a CTA four warps stream every
// fourth tile through buffers of their own (cp.async, 16-byte chunks swizzled for
// ldmatrix) and their states meet in shared memory.
// With a window the tiles are those of the first `sink` keys, then those of the
// window.
//
// 16 sequences of 32768 keys, 32 query and 8 key/value heads of 128: 117.4 us for the
// call, 604 MB at 0.76 of a plain copy's rate. What bounds it is issue: 635 instructions
// per warp and tile, of which the tensor products hold the issue port about 8 slots each
// (with the products cut out the same loads take 99.6 us, and the whole takes no less out
// of the L2). Q K^T on tcgen05 instead (K's values unpacked into tensor memory as the
// 128-row operand, q as the 16-wide one) took 139 us: the unpacking stays, and a block
// barrier and a round trip through tensor memory per tile come on top.
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include "cache_q4.cuh"
#include "host_util.h"
#include "launch.h"
#include "soft_cap.cuh"

#define MATTN_API extern "C" __attribute__((visibility("default")))

namespace mattn {
namespace {

constexpr int kQ4Threads = 128;
constexpr int kQ4Warps = 4;
constexpr int kQ4Tile = 32;    // keys per warp step
constexpr int kQ4Stages = 2;   // per-warp tile buffers
constexpr int kQ4MaxRows = 16;
// What a segment's start and end cost beside its tiles (61 ragged sequences of up to 15001
// keys and a soft-cap: 10: 124.6 us, 12: 124.9, 16: 125.3, 24: 127.7; 7 of 40000, 8 heads of
// 64, 16 rows: 64.8, 64.8, 64.1, 63.5; 0, before other steps, 27 more on the former)
constexpr int kQ4SegmentCost = 16;
constexpr float kQ4Head = 15.0f;   // log2 bound of a scaled weight
constexpr float kQ4Start = 8.0f;   // log2 of the largest one when the reference moves
constexpr uint32_t kQ4Tiny = 0x12801280u;  // bf16 2^-90, twice: smaller V scales count as this,
                                           // so that unscaled weights stay within fp32
constexpr uint32_t kQ4Spread = 8u << 7;    // a key's V scales may lie this far apart, as bf16
                                           // bits (2^8), for weights in fp16
constexpr uint32_t kQ4Outside = 0xfc00fc00u;  // bits of a distance of kQ4Spread or more, twice
// Lower ends of such windows that hold, of scales >= 0 (NaN aside), 0 alone (and
// 2^-133, where the lower half borrows) and none.
constexpr uint32_t kQ4NoValues = 0xfc01u, kQ4Apart = 0xfc00fc00u;

struct Q4Problem {
  const void* q;
  const uint8_t* pool;
  void* o;
  float* lse;
  const int* seq_lens;
  const int* table;
  const float* slopes;
  int B, Hq, Hkv, Sq, max_len;
  int pages_per_seq, num_pages, shift;
  unsigned variant;
  int window, sink;
  float scale2;       // scale * log2 e
  float softcap2;     // softcap * log2 e
  float softcap_e;    // 2 / softcap: e^(2 s / softcap) from s in log2 units
  // Workspace, or nullptr: then one CTA per pair. Partial results by slot: CTA +
  // pair (both ascend along the tiles, so each cut has its own).
  int2* ws_meta;   // [pairs]: first and last CTA of a cut pair; first = -1: done
  float* ws_lse;   // [slots][R], log2
  float* ws_o;     // [slots][R][D]
  long long slots;
};

// A sequence's tiles: those of the sinks, then those from win_tile on.
struct Q4Range {
  int len, win_tile, sink_tiles, tiles;
  // What a pair counts for in the dealing out: its tiles, and the start and
  // end of a segment as so many more.
  __device__ __forceinline__ int cost() const { return tiles ? tiles + kQ4SegmentCost : 0; }
};

__device__ __forceinline__ Q4Range q4_range(const Q4Problem& p, int b) {
  Q4Range r;
  const long long held = (long long)p.pages_per_seq << p.shift;
  r.len = max(0, min(p.seq_lens[b], (int)min((long long)p.max_len, held)));
  r.win_tile = r.sink_tiles = 0;
  if (p.variant & ATTN_MASK_WINDOW) {
    const int w0 = (int)max(0ll, (long long)r.len - p.Sq - p.window + 1);
    r.win_tile = w0 / kQ4Tile;
    r.sink_tiles = min(r.win_tile, (min(p.sink, r.len) + kQ4Tile - 1) / kQ4Tile);
  }
  r.tiles = r.sink_tiles + max(0, (r.len + kQ4Tile - 1) / kQ4Tile - r.win_tile);
  return r;
}

template <int D, int NT>
struct Q4Cfg {
  static constexpr int G = D / kQ4Group;                  // scales per row
  static constexpr int kRow = D / 2;                      // bytes of a row of codes
  static constexpr int kCodes = kQ4Tile * kRow;
  static constexpr int kScales = kQ4Tile * G * 2;
  static constexpr int kStage = 2 * kCodes + 2 * kScales;  // K, V codes, K, V scales
  static constexpr int kWarp = kQ4Stages * kStage;
  static constexpr int kState = 8 * NT * (2 + D) * 4;      // a warp's m, l, O at the end
  static constexpr int kQ = NT * G * 512;                  // q fragments, 16 bytes per lane
  static constexpr int kOff = NT * G * 64;                 // the scores' offsets, 16 bytes per t
  static constexpr int kSmem = kQ4Warps * (kWarp + kState) + kQ + kOff + NT * 8 * 4;
  // Rows of codes are D / 2 bytes; chunk c (16 bytes) of row r stands at place
  // c ^ swz(r), so that the 8 rows of an ldmatrix matrix hit distinct banks.
  static __device__ __forceinline__ int swz(int row) {
    return D == 128 ? (row >> 1) & 3 : (row >> 2) & 1;
  }
};

// CTAs per SM that the registers are cut to. What is measured is issue, not
// latency: one more CTA at fewer registers spills and is slower (16 x 32768 keys, 8
// key/value heads of 128: 118 us, with two 126, with four 127; with 16 query rows each
// 176, with three 180; 32 x 32768 keys, heads of 64: 145, with three the same, with five 160).
template <int D, int NT>
constexpr int q4_per_sm() {
  return D == 128 ? (NT == 1 ? 3 : 2) : (NT == 1 ? 4 : 3);
}

__device__ __forceinline__ void cp_async16z(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// c += A (16x16) B (16x8), fp32 accumulators
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (x & mask) | bits in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "r"(mask), "r"(bits));
  return y;
}

// Nibbles 0 to 3 of both halves of w as exact fp16 pairs (n - 8, n' - 8): the
// nibble's bits in the mantissa of 1024 or, one nibble up, of 64. kOdd false:
// nibbles 1 and 3 keep the offset, 64 + n.
template <bool kOdd>
__device__ __forceinline__ void nibble_pairs(uint32_t w, uint32_t (&f)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t x = j & 2 ? w >> 8 : w;
    const uint32_t raw = j & 1 ? and_or(x, 0x00f000f0u, 0x54005400u)    // 64 + n
                               : and_or(x, 0x000f000fu, 0x64006400u);   // 1024 + n
    if ((j & 1) && !kOdd) {
      f[j] = raw;
      continue;
    }
    const uint32_t off = j & 1 ? 0x54805480u : 0x64086408u;         // 72, 1032
    const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&raw),
                              *reinterpret_cast<const __half2*>(&off));
    f[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Nibbles 0 to 3 of both halves of w as exact bf16 pairs (n - 8, n' - 8): the
// nibble's bits in the mantissa of 128, less 136.
__device__ __forceinline__ void nibble_pairs_bf16(uint32_t w, uint32_t (&f)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t raw = and_or(w >> (4 * j), 0x000f000fu, 0x43004300u), off = 0x43084308u;
    const __nv_bfloat162 h = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&raw),
                                     *reinterpret_cast<const __nv_bfloat162*>(&off));
    f[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The G bf16 scales of one row, two to a word.
template <int G>
__device__ __forceinline__ void load_scales(const uint8_t* p, uint32_t (&w)[G / 2]) {
  if constexpr (G == 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x;
    w[1] = u.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

__device__ __forceinline__ float scale_of(uint32_t w, int i) {  // i = 0 or 1
  return __uint_as_float(i ? w & 0xffff0000u : w << 16);
}

// A run of tiles of one pair: the CTA's share of it.
struct Q4Segment {
  int b, hkv;
  int len, win_tile, sink_tiles;
  int v_last, n_tiles;   // this warp's last tile and its count (every kQ4Warps-th)
  long long slot;        // partial result, or -1: all of the pair's tiles
};

template <int D, int NT, int SCORE>
__global__ void __launch_bounds__(kQ4Threads, q4_per_sm<D, NT>())
    decode_q4_kernel(const Q4Problem p) {
  using C = Q4Cfg<D, NT>;
  constexpr int G = C::G;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;  // fragment coordinates
  const int group = p.Hq / p.Hkv;
  const int R = group * p.Sq;
  [[maybe_unused]] const size_t total_rows = (size_t)p.B * p.Hq * p.Sq;
  const bool causal = p.variant & ATTN_MASK_CAUSAL, windowed = p.variant & ATTN_MASK_WINDOW;
  early_start();

  // this CTA's first pair and tiles [lo, hi) of all
  int b = blockIdx.x / p.Hkv, hkv = blockIdx.x % p.Hkv;
  long long lo = 0, hi = LLONG_MAX, seq_start = 0;
  bool last_cta = false;
  if (p.ws_meta) {
    // A thread adds up a run of sequences; a scan over the block places the runs.
    __shared__ long long sums[kQ4Warps];
    __shared__ long long found_start;
    __shared__ int found;
    const int run = (p.B + kQ4Threads - 1) / kQ4Threads;
    const int r0 = min((int)threadIdx.x * run, p.B), r1 = min(r0 + run, p.B);
    long long mine = 0;
    int last_cost = 0;
    for (int i = r0; i < r1; ++i) mine += last_cost = q4_range(p, i).cost();
    long long upto = mine;  // inclusive
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += v;
    }
    if (lane == 31) sums[warp] = upto;
    if (threadIdx.x == 0) found = p.B;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kQ4Warps; ++w) {
      if (w < warp) upto += sums[w];
      total += sums[w];
    }
    total *= p.Hkv;
    // CTAs that take part: each has a tile for every warp, on the average
    const int ctas = (int)max(1ll, min((long long)gridDim.x, (total + kQ4Warps - 1) / kQ4Warps));
    if (blockIdx.x >= ctas) return;
    last_cta = blockIdx.x == ctas - 1;
    lo = total * blockIdx.x / ctas;
    hi = total * (blockIdx.x + 1) / ctas;
    // the first sequence that ends past lo, or starts there without tiles
    if (r0 < r1 && (upto * p.Hkv > lo || (upto - last_cost) * p.Hkv >= lo)) atomicMin(&found, r0);
    __syncthreads();
    if (r0 < r1 && found == r0) {
      long long at = upto - mine;
      int i = r0;
      for (; i < r1 - 1; ++i) {
        const int c = q4_range(p, i).cost();
        if ((at + c) * p.Hkv > lo || at * p.Hkv >= lo) break;
        at += c;
      }
      found_start = at * p.Hkv;
      sums[0] = i;
    }
    __syncthreads();
    b = found < p.B ? (int)sums[0] : p.B;
    seq_start = found_start;
    hkv = 0;
  }

  // The CTA's next segment, false at the end. Sequences without tiles on the
  // way get their empty rows.
  Q4Range rg;
  int rg_of = -1;
  auto next_segment = [&](Q4Segment& sg) -> bool {
    for (; b < p.B; ++b, hkv = 0) {
      if (rg_of != b) {
        rg = q4_range(p, b);
        rg_of = b;
        const int cost = rg.cost();
        if (p.ws_meta && cost > 0) hkv = max(0, (int)((lo - seq_start) / cost));
      }
      const int cost = rg.cost();
      if (p.ws_meta && seq_start >= hi && !(last_cta && cost == 0)) return false;
      if (p.ws_meta && cost == 0) {
        const size_t row0 = (size_t)b * p.Hq * p.Sq;
        for (int i = threadIdx.x; i < p.Hq * p.Sq * (D / 2); i += kQ4Threads)
          if (MATTN_IN_BOUNDS(kSiteQ4Out, row0 + i / (D / 2), total_rows))
            static_cast<uint32_t*>(p.o)[row0 * (D / 2) + i] = 0u;
        for (int i = threadIdx.x; i < p.Hq * p.Sq; i += kQ4Threads) p.lse[row0 + i] = -INFINITY;
        for (int i = threadIdx.x; i < p.Hkv; i += kQ4Threads)
          p.ws_meta[(size_t)b * p.Hkv + i].x = -1;
        continue;
      }
      for (; hkv < p.Hkv; ++hkv) {
        int v_begin = 0, v_end = rg.tiles;
        if (p.ws_meta) {
          // the pair's tiles follow its own cost
          const long long start = seq_start + (long long)hkv * cost + kQ4SegmentCost;
          if (start >= hi) return false;
          v_begin = (int)max(0ll, lo - start);
          v_end = (int)min((long long)rg.tiles, hi - start);
          if (v_begin >= rg.tiles) continue;
        }
        const bool cut = v_begin > 0 || v_end < rg.tiles;
        const int pair = b * p.Hkv + hkv;
        if (p.ws_meta && threadIdx.x == 0) {
          if (v_begin == 0) p.ws_meta[pair].x = cut ? (int)blockIdx.x : -1;
          if (v_end == rg.tiles) p.ws_meta[pair].y = (int)blockIdx.x;
        }
        sg.b = b;
        sg.hkv = hkv;
        sg.len = rg.len;
        sg.win_tile = rg.win_tile;
        sg.sink_tiles = rg.sink_tiles;
        const int v_first = v_begin + warp;
        sg.n_tiles = v_first < v_end ? (v_end - v_first + kQ4Warps - 1) / kQ4Warps : 0;
        sg.v_last = v_first + (sg.n_tiles - 1) * kQ4Warps;
        sg.slot = cut ? (long long)blockIdx.x + pair : -1;
        ++hkv;
        if (!p.ws_meta) b = p.B;  // one pair per CTA
        return true;
      }
      seq_start += (long long)cost * p.Hkv;
    }
    return false;
  };

  // A segment's tiles through the warp's buffers. Their pages are looked up 16
  // tiles at a time, lane 2i + h the page of tile i's 16-key half h (or -1), one
  // batch ahead.
  const Q4Layout L{D, 1 << p.shift};
  const uint32_t area = smem_u32(smem) + warp * C::kWarp;
  const uint8_t* area_ptr = smem + warp * C::kWarp;
  float* states = reinterpret_cast<float*>(smem + kQ4Warps * C::kWarp);
  uint4* qs = reinterpret_cast<uint4*>(smem + kQ4Warps * (C::kWarp + C::kState));  // [NT][G][32 lanes]
  float4* offs = reinterpret_cast<float4*>(qs + C::kQ / 16);                        // [NT][G][4]
  float* units = reinterpret_cast<float*>(offs + C::kOff / 16);                     // [NT * 8]
  // First key of the warp's tile i: the last keys come first, where scores that fall
  // with the distance are largest, so that the reference stays (64 sequences x 8000 keys
  // with ALiBi: 122 us, ascending 155; without: 118 and 119).
  auto key_of = [&](const Q4Segment& sg, int i) {
    const int v = sg.v_last - i * kQ4Warps;
    return (v < sg.sink_tiles ? v : v - sg.sink_tiles + sg.win_tile) * kQ4Tile;
  };
  auto look_up = [&](const Q4Segment& sg, int i0) -> int {
    const int i = i0 + (lane >> 1);
    if (i >= sg.n_tiles) return -1;
    const int lp = (key_of(sg, i) + 16 * (lane & 1)) >> p.shift;
    if (lp >= p.pages_per_seq) return -1;
    const long long at = (long long)sg.b * p.pages_per_seq + lp;
    if (!MATTN_IN_BOUNDS(kSiteQ4Table, at, (long long)p.B * p.pages_per_seq)) return -1;
    const int pg = p.table[at];
    return pg >= 0 && pg < p.num_pages ? pg : -1;
  };
  int pages = -1, pages_next = -1;
  const uint32_t page_stride = (uint32_t)p.Hkv * L.bytes();
  [[maybe_unused]] const long long pool_bytes = (long long)p.num_pages * page_stride;
  // Whether the 16 bytes at x lie in the pool (true in the release build).
  [[maybe_unused]] auto in_pool = [&](const uint8_t* x) {
    return MATTN_IN_BOUNDS(kSiteQ4Pool, x - p.pool, pool_bytes) &&
           MATTN_IN_BOUNDS(kSiteQ4Pool, x + 15 - p.pool, pool_bytes);
  };
  constexpr int kScaleChunks = C::kScales / 32;  // 16-byte chunks of K (or V) scales per half
  // lane's chunk of the scales: half, K or V, place
  const bool sc_half = lane / kScaleChunks & 1;
  const int sc_src = (lane / (2 * kScaleChunks) ? L.v_scales() : L.k_scales()) +
                     (lane % kScaleChunks) * 16 - lane * 16;
  const uint32_t sc_dst = 2 * C::kCodes + (lane / kScaleChunks) % 2 * (C::kScales / 2) +
                          lane / (2 * kScaleChunks) * C::kScales + lane % kScaleChunks * 16;
  auto load_tile = [&](const Q4Segment& sg, int i) {  // into buffer i % kQ4Stages; i = 0, 1, 2, ...
    if ((i & 15) == 0) {
      pages = pages_next;
      pages_next = look_up(sg, i + 16);
    }
    const uint32_t dst = area + (i & (kQ4Stages - 1)) * C::kStage;
    const int key0 = key_of(sg, i);
    const uint8_t* head_pool = p.pool + (size_t)sg.hkv * L.bytes() + lane * 16;
    const uint32_t lane_dst = dst + lane / G * C::kRow + (lane % G ^ C::swz(lane / G)) * 16;
    auto half_codes = [&](int h, const uint8_t* k, uint32_t bytes) {  // 16 keys, K and V
      const uint8_t* v = k + L.v_codes();
      if (bytes && !(in_pool(k) && in_pool(v + (D / 64 - 1) * 512))) bytes = 0;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const uint32_t d = lane_dst + (16 * h + c * (32 / G)) * C::kRow;
        cp_async16z(d, k + c * 512, bytes);
        cp_async16z(d + C::kCodes, v + c * 512, bytes);
      }
    };
    const int pg0 = __shfl_sync(0xffffffffu, pages, 2 * (i & 15));
    const uint8_t* rec0 = head_pool + (size_t)(uint32_t)max(pg0, 0) * page_stride;
    const int in0 = key0 & (L.page - 1);
    const uint32_t bytes0 = pg0 >= 0 ? 16u : 0u;
    const uint8_t* k0 = rec0 + in0 * L.code_row();
    half_codes(0, k0, bytes0);
    const uint8_t* sc = rec0 + in0 * L.scale_row() + sc_src;
    uint32_t sc_bytes = bytes0;
    if (L.page >= kQ4Tile) {  // the whole tile lies in one page
      half_codes(1, k0 + 16 * L.code_row(), bytes0);
      if (sc_half) sc += 16 * L.scale_row();
    } else {
      const int pg1 = __shfl_sync(0xffffffffu, pages, 2 * (i & 15) + 1);
      const uint8_t* rec1 = head_pool + (size_t)(uint32_t)max(pg1, 0) * page_stride;
      half_codes(1, rec1, pg1 >= 0 ? 16u : 0u);
      if (sc_half) {
        sc = rec1 + sc_src;
        sc_bytes = pg1 >= 0 ? 16u : 0u;
      }
    }
    if (lane < 4 * kScaleChunks) {
      if (sc_bytes && !in_pool(sc)) sc_bytes = 0;
      cp_async16z(dst + sc_dst, sc, sc_bytes);
    }
    cp_async_commit();
  };
  auto start_loads = [&](const Q4Segment& sg) {
    pages_next = look_up(sg, 0);
    if (sg.n_tiles > 0) load_tile(sg, 0);
    if (sg.n_tiles > 1) load_tile(sg, 1);
  };

  Q4Segment cur;
  if (!next_segment(cur)) return;
  start_loads(cur);
  for (;;) {
    const int len = cur.len, first_pos = len - p.Sq;  // absolute position of query row 0
    const size_t row0 = (size_t)(cur.b * p.Hq + cur.hkv * group) * p.Sq;

    // Meanwhile q^T's fragments (B operand) are prepared in shared memory, in fp16,
    // each warp a fourth of them: a row is scaled by a power of two that brings its
    // largest channel to [2^14, 2^15), so bf16's 8 bits are exact (channels 2^28 times
    // smaller lose bits below 2^-39 of the largest). Channel order of a lane's 8 per
    // group: pairs (0, 4), (1, 5) | (2, 6), (3, 7). Rows past R are 0.
    {
      const __nv_bfloat16* Q = static_cast<const __nv_bfloat16*>(p.q) + row0 * D;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = nt * 8 + g;
        uint4 x[G];
        uint32_t m2 = 0;  // largest |q| as bits, two at a time: ordered like the values, NaN last
#pragma unroll
        for (int a = 0; a < G; ++a) {
          x[a] = make_uint4(0, 0, 0, 0);
          if (r < R && MATTN_IN_BOUNDS(kSiteQ4Q, row0 + r, total_rows))
            x[a] = *reinterpret_cast<const uint4*>(Q + (size_t)r * D + 32 * a + 8 * t);
          const uint32_t u[4] = {x[a].x, x[a].y, x[a].z, x[a].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) m2 = __vmaxu2(m2, u[i] & 0x7fff7fffu);
        }
        m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, 1));
        m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, 2));
        const uint32_t big = max(m2 & 0xffff0000u, m2 << 16);
        const bool fine = big < 0x7f800000u;
        const int ex = max((int)(big >> 23) - 127, -100);  // floor(log2)
        const float up = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
        // scores per product, log2; a row with an infinity or NaN scores NaN
        if (warp == 0 && t == 0) units[r] = fine ? exp2f((float)(ex - 14)) * p.scale2 : NAN;
#pragma unroll
        for (int a = 0; a < G; ++a) {
          if ((nt * G + a) % kQ4Warps != warp) continue;
          const uint32_t u[4] = {x[a].x, x[a].y, x[a].z, x[a].w};
          float c[8], sum = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) c[i] = fine ? scale_of(u[i / 2], i & 1) * up : 0.0f;
          qs[(nt * G + a) * 32 + lane] = make_uint4(pack_f16x2(c[0], c[4]), pack_f16x2(c[1], c[5]),
                                                    pack_f16x2(c[2], c[6]), pack_f16x2(c[3], c[7]));
          // -72 sum(q) over the nibbles that keep their offset: per lane channels
          // 1, 3, 5, 7; of row g, stored for the lane t that holds columns 2t, 2t + 1
          sum = c[1] + c[3] + c[5] + c[7];
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          if (t < 2) reinterpret_cast<float*>(offs + (nt * G + a) * 4 + g / 2)[g % 2 + 2 * t] = -72.0f * sum;
        }
      }
    }
    __syncthreads();

    // the lane's query rows (columns 2t, 2t + 1 of each 8)
    float unit[NT][2], slope2[NT][2];
    int pos[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = nt * 8 + 2 * t + e;
        unit[nt][e] = units[r];
        const int hg = r < R ? r / p.Sq : 0;
        pos[nt][e] = first_pos + (r < R ? r % p.Sq : 0);
        const int h = cur.hkv * group + hg;
        slope2[nt][e] =
            (SCORE & 1) ? (p.slopes ? p.slopes[h] : exp2f(-8.0f * float(h + 1) / float(p.Hq))) * kLog2e
                        : 0.0f;
      }

    float o[G][2][NT][4];  // [group][channel pair] x (channel, row) of each 8 rows
#pragma unroll
    for (int a = 0; a < G; ++a)
#pragma unroll
      for (int jp = 0; jp < 2; ++jp)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          o[a][jp][nt][0] = o[a][jp][nt][1] = o[a][jp][nt][2] = o[a][jp][nt][3] = 0.0f;
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.0f;
    }
    // The 8 binades that the V scales of the warp's keys lie in: the bf16 bits of their lower
    // end (kQ4NoValues: the group is zero), of two groups to a word, and log2 of their upper
    // end. Where a tile's do not, they are looked at key by key. 0: no key yet; kQ4Apart: a
    // key's scales lay too far apart for weights in fp16.
    uint32_t low[G / 2] = {};
    float lsm = 0.0f;

    // One tile of 32 keys. kMask: some (key, row) pair of it is masked.
    auto process = [&](const uint32_t stage_off, const int key0, auto mask_tag) {
      constexpr bool kMask = decltype(mask_tag)::value;
      // an ldmatrix row is a key: the lane's, with the place of chunk 0
      const uint32_t rows = area + stage_off + lane * C::kRow + C::swz(lane) * 16;
      const uint8_t* scales = area_ptr + stage_off + 2 * C::kCodes;
      float x[2][NT][4];
      uint32_t sk[4][G / 2];
#pragma unroll
      for (int i = 0; i < 4; ++i) load_scales<G>(scales + (8 * i + g) * 2 * G, sk[i]);
#pragma unroll
      for (int a = 0; a < G; ++a) {
        uint32_t w[4];  // the lane's 8 channels of group a, for keys g, g + 8, g + 16, g + 24
        ldsm4(rows ^ (a * 16), w);
        uint4 qf[NT];
        float4 off[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          qf[nt] = qs[(nt * G + a) * 32 + lane];
          off[nt] = offs[(nt * G + a) * 4 + t];
        }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          uint32_t f[2][4];
          nibble_pairs<false>(w[2 * mt], f[0]);
          nibble_pairs<false>(w[2 * mt + 1], f[1]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float d[4] = {off[nt].x, off[nt].y, off[nt].z, off[nt].w};
            mma_f16(d, f[0][0], f[1][0], f[0][1], f[1][1], qf[nt].x, qf[nt].y);
            mma_f16(d, f[0][2], f[1][2], f[0][3], f[1][3], qf[nt].z, qf[nt].w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float s = scale_of(sk[2 * mt + (e >> 1)][a / 2], a & 1);
              x[mt][nt][e] = a == 0 ? s * d[e] : fmaf(s, d[e], x[mt][nt][e]);
            }
          }
        }
      }
      uint32_t sv[2][2][G / 2];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        load_scales<G>(scales + C::kScales + (8 * i + g) * 2 * G, sv[i >> 1][i & 1]);
      // score modification and mask. Without a modification the scores stay in
      // the products' units and `unit` enters with the exponent.
      auto each_score = [&](auto f) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) f(x[mt][nt][e], nt, e, 16 * mt + 8 * (e >> 1));
      };
      if constexpr (SCORE != 0)
        each_score([&](float& s, int nt, int e, int) { s *= unit[nt][e & 1]; });
      if constexpr ((SCORE & 1) != 0) {
        float dist[NT][2];  // to the lane's first key; conversions are slow, so one per row
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) dist[nt][e] = float(pos[nt][e] - key0 - g);
        each_score([&](float& s, int nt, int e, int key) {
          s = fmaf(-slope2[nt][e & 1], dist[nt][e & 1] - float(key), s);
        });
      }
      if constexpr ((SCORE & 2) != 0) {
        float big = 0.0f;
        each_score([&](float& s, int, int, int) { big = fmaxf(big, fabsf(s)); });
        // scores are mostly well below their cap
        if (__all_sync(0xffffffffu, big * p.softcap_e < kCapNear))
          each_score([&](float& s, int, int, int) { s = soft_cap_near(s, p.softcap_e); });
        else
          each_score([&](float& s, int, int, int) { s = soft_cap(s, p.softcap2, p.softcap_e); });
      }
      if constexpr (kMask)
        each_score([&](float& s, int nt, int e, int key) {
          const int j = key0 + key + g, i = pos[nt][e & 1];
          bool keep = j < len && i >= 0;
          if (causal) keep = keep && j <= i;
          if (windowed) keep = keep && (i - j < p.window || j < p.sink);
          s = keep ? s : -INFINITY;
        });
      auto log2_of = [&](float s, int nt, int e) { return SCORE ? s : s * unit[nt][e]; };
      // The reference follows keys that pass its bound. First a quick bound: the
      // lane's largest score with the upper end of the window that V scales lie in. Whether
      // the tile's do, each lane tests for one key.
      uint32_t out = 0, mine[G / 2];
      load_scales<G>(scales + C::kScales + lane * 2 * G, mine);
#pragma unroll
      for (int i = 0; i < G / 2; ++i) out |= mine[i] - low[i];
      bool over = (out & kQ4Outside) != 0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float y = fmaxf(fmaxf(x[0][nt][e], x[0][nt][e + 2]), fmaxf(x[1][nt][e], x[1][nt][e + 2]));
          over = over || log2_of(y, nt, e) + lsm > m[nt][e] + kQ4Head;
        }
      auto weights = [&]() {  // a masked key's is -0, one too small for fp32 +0
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float ref = m[nt][e] == -INFINITY ? 0.0f : m[nt][e];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float& s = x[k >> 1][nt][e + 2 * (k & 1)];
              const bool masked = kMask && s == -INFINITY;  // in any row, one of NaN too
              s = masked ? -0.0f : ex2_approx(SCORE ? s - ref : fmaf(s, unit[nt][e], -ref));
              l[nt][e] += s;
            }
          }
      };
      if (__any_sync(0xffffffffu, over)) {
        if (low[0] != kQ4Apart) {
          uint32_t hi = kQ4Tiny >> 16, lo = 0xffffu, held = 0;  // of the lane's key
#pragma unroll
          for (int a = 0; a < G; ++a) {
            const uint32_t s = mine[a / 2] >> (a & 1 ? 16 : 0) & 0x7fffu;
            hi = max(hi, s);
            lo = min(lo, s - 1);  // a zero is the largest here
            held |= s ? 1u << a : 0u;
          }
          bool seen = true;  // by some row
          if constexpr (kMask) {
            const int j = key0 + lane, i = max(max(first_pos, 0), causal ? j : 0);
            seen = j < len && (!windowed || i - j < p.window || j < p.sink);
          }
          const bool far = seen && (!held || hi - lo > kQ4Spread);
          const uint32_t top = __reduce_max_sync(0xffffffffu, seen ? hi : 0u) >> 7;  // 0: no key
          const uint32_t some = __reduce_or_sync(0xffffffffu, seen ? held : 0u);
          const uint32_t every = __reduce_and_sync(0xffffffffu, seen ? held : ~0u);
          uint32_t before = some;  // the groups that had values, if a key was there
          if (low[0]) {
            before = 0;
#pragma unroll
            for (int a = 0; a < G; ++a)
              before |= (low[a / 2] >> (a & 1 ? 16 : 0) & 0xffffu) != kQ4NoValues ? 1u << a : 0u;
          }
          if (__any_sync(0xffffffffu, far) || (top && (some != every || some != before))) {
            low[0] = kQ4Apart;
          } else if (top) {
            lsm = (float)(int)top - 126.0f;
#pragma unroll
            for (int i = 0; i < G / 2; ++i)
              low[i] = (some >> (2 * i) & 1 ? (top - 7) << 7 : kQ4NoValues) |
                       (some >> (2 * i + 1) & 1 ? (top - 7) << 7 : kQ4NoValues) << 16;
          }
        }
        float lsv[2][2];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float big = __uint_as_float(kQ4Tiny & 0xffff0000u);
#pragma unroll
            for (int a = 0; a < G; ++a) big = fmaxf(big, fabsf(scale_of(sv[mt][e][a / 2], a & 1)));
            lsv[mt][e] = __log2f(big);
          }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float y = -INFINITY;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              y = fmaxf(y, log2_of(x[k >> 1][nt][e + 2 * (k & 1)], nt, e) + lsv[k >> 1][k & 1]);
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
            // each row by itself: its result does not depend on the others'
            const float m_new = y > m[nt][e] + kQ4Head ? y - kQ4Start : m[nt][e];
            const float c = m_new == -INFINITY ? 1.0f : ex2_approx(m[nt][e] - m_new);  // -inf -> 0
            m[nt][e] = m_new;
            l[nt][e] *= c;
#pragma unroll
            for (int a = 0; a < G; ++a)
#pragma unroll
              for (int jp = 0; jp < 2; ++jp) {
                o[a][jp][nt][e] *= c;
                o[a][jp][nt][e + 2] *= c;
              }
          }
        if (low[0] == kQ4Apart) {  // O^T += V^T P^T, P as the sum of two bf16 halves
          weights();
#pragma unroll
          for (int a = 0; a < G; ++a) {
            uint32_t w[4];
            ldsm4_t((rows ^ (a * 16)) + C::kCodes, w);
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              uint32_t f[2][4];
              nibble_pairs_bf16(w[2 * mt], f[0]);
              nibble_pairs_bf16(w[2 * mt + 1], f[1]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                uint32_t b[2][2];  // [keys' half][the larger part, what it leaves]
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const float s = scale_of(sv[mt][e][a / 2], a & 1);
                  float p0 = x[mt][nt][2 * e] * s, p1 = x[mt][nt][2 * e + 1] * s;
                  if constexpr (kMask) {
                    p0 = signbit(x[mt][nt][2 * e]) ? 0.0f : p0;
                    p1 = signbit(x[mt][nt][2 * e + 1]) ? 0.0f : p1;
                  }
                  const uint32_t big = pack_bf16x2(p0, p1);
                  b[e][0] = transpose8(big);
                  b[e][1] = transpose8(pack_bf16x2(p0 - scale_of(big, 0), p1 - scale_of(big, 1)));
                }
#pragma unroll
                for (int jp = 0; jp < 2; ++jp)
#pragma unroll
                  for (int part = 0; part < 2; ++part)
                    mma_bf16(o[a][jp][nt], f[0][2 * jp], f[0][2 * jp + 1], f[1][2 * jp],
                             f[1][2 * jp + 1], b[0][part], b[1][part]);
              }
            }
          }
          return;
        }
      }
      weights();
      // O^T += V^T P^T
#pragma unroll
      for (int a = 0; a < G; ++a) {
        uint32_t w[4];  // 4 channels of group a for key pairs 2t, 2t + 1 of each 8 keys
        ldsm4_t((rows ^ (a * 16)) + C::kCodes, w);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          uint32_t f[2][4];
          nibble_pairs<true>(w[2 * mt], f[0]);
          nibble_pairs<true>(w[2 * mt + 1], f[1]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float pv[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              pv[e] = x[mt][nt][e] * scale_of(sv[mt][e >> 1][a / 2], a & 1);
              // a masked key adds nothing, whatever its scale holds
              if constexpr (kMask) pv[e] = signbit(x[mt][nt][e]) ? 0.0f : pv[e];
            }
            const uint32_t b0 = transpose8(pack_f16x2(pv[0], pv[1]));
            const uint32_t b1 = transpose8(pack_f16x2(pv[2], pv[3]));
#pragma unroll
            for (int jp = 0; jp < 2; ++jp)
              mma_f16(o[a][jp][nt], f[0][2 * jp], f[0][2 * jp + 1], f[1][2 * jp], f[1][2 * jp + 1],
                      b0, b1);
          }
        }
      }
    };

    for (int i = 0; i < cur.n_tiles; ++i) {
      if (i + 1 < cur.n_tiles) cp_async_wait<1>();
      else cp_async_wait<0>();
      __syncwarp();
      const int key0 = key_of(cur, i), key_end = key0 + kQ4Tile;
      const bool whole = key_end <= len && first_pos >= 0 && (!causal || key_end - 1 <= first_pos) &&
                         (!windowed || len - 1 - key0 < p.window || key_end <= p.sink);
      const uint32_t stage_off = (i & (kQ4Stages - 1)) * C::kStage;
      if (whole) process(stage_off, key0, std::false_type{});
      else process(stage_off, key0, std::true_type{});
      __syncwarp();
      if (i + 2 < cur.n_tiles) load_tile(cur, i + 2);
    }
    // the next segment's first tiles are on their way during this one's end
    Q4Segment nxt;
    const bool more = next_segment(nxt);
    if (more) start_loads(nxt);

    // the warps' states meet in shared memory: m, l (8 NT each), O [8 NT][D]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 4);
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 8);
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 16);
      }
    constexpr int kR = 8 * NT;
    float* wm = states + warp * (C::kState / 4);
    float* wl = wm + kR;
    float* wo = wl + kR;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (g == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          wm[nt * 8 + 2 * t + e] = m[nt][e];
          wl[nt * 8 + 2 * t + e] = l[nt][e];
        }
      }
#pragma unroll
      for (int a = 0; a < G; ++a)
#pragma unroll
        for (int jp = 0; jp < 2; ++jp)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float2*>(wo + (nt * 8 + 2 * t + e) * D + 32 * a + 4 * g + 2 * jp) =
                make_float2(o[a][jp][nt][e], o[a][jp][nt][e + 2]);
    }
    __syncthreads();
    for (int idx = threadIdx.x; idx < R * (D / 4); idx += kQ4Threads) {
      const int r = idx / (D / 4), c = idx % (D / 4) * 4;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kQ4Warps; ++w)
        M = fmaxf(M, states[w * (C::kState / 4) + r]);
      float Ls = 0.0f;
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kQ4Warps; ++w) {
        const float* st = states + w * (C::kState / 4);
        const float wt = M != -INFINITY ? ex2_approx(st[r] - M) : 1.0f;  // -inf -> 0
        const float4 x = *reinterpret_cast<const float4*>(st + 2 * kR + r * D + c);
        Ls += wt * st[kR + r];
        acc = make_float4(acc.x + wt * x.x, acc.y + wt * x.y, acc.z + wt * x.z, acc.w + wt * x.w);
      }
      // a row without a key: O = 0, LSE = -inf. NaN sums pass through.
      const bool none = Ls == 0.0f;
      const float lse2 = none ? -INFINITY : M + __log2f(Ls);
      acc = none ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                 : make_float4(acc.x / Ls, acc.y / Ls, acc.z / Ls, acc.w / Ls);
      if (!MATTN_IN_BOUNDS(kSiteQ4Out, row0 + r, total_rows)) continue;
      if (cur.slot >= 0) {
        if (!MATTN_IN_BOUNDS(kSiteQ4Out, cur.slot, p.slots)) continue;
        *reinterpret_cast<float4*>(p.ws_o + ((size_t)cur.slot * R + r) * D + c) = acc;
        if (c == 0) p.ws_lse[(size_t)cur.slot * R + r] = lse2;
      } else {
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + (row0 + r) * D + c) =
            make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
        if (c == 0) p.lse[row0 + r] = lse2 * kLn2;
      }
    }
    if (!more) break;
    cur = nxt;
  }
}

constexpr int merge_warps(int W) { return W > kQ4Warps ? W : kQ4Warps; }  // of a block

// Joins the partial results of the pairs that several CTAs share: W warps per
// row of o take its parts in turn (a fixed order), each lane D / 32 channels.
// Bound by latency: two dependent loads, then the parts' rows from the L2.
template <int D, int W>
__global__ void __launch_bounds__(32 * merge_warps(W)) q4_merge_kernel(const Q4Problem p) {
  constexpr int V = D / 32;
  constexpr int kWarps = merge_warps(W);
  __shared__ float sh[kWarps][D + 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long rows = (long long)p.B * p.Hq * p.Sq;
  const long long row = (long long)blockIdx.x * (kWarps / W) + warp / W;
  early_start();
  float M = -INFINITY, L = 0.0f, acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
  bool mine = false;
  if (row < rows) {
    const int group = p.Hq / p.Hkv, R = group * p.Sq;
    const long long bh = row / p.Sq;
    const int h = (int)(bh % p.Hq);
    const long long pair = bh / p.Hq * p.Hkv + h / group;
    const int r = h % group * p.Sq + (int)(row % p.Sq);
    const int2 ctas = p.ws_meta[pair];
    mine = ctas.x >= 0;
    if (mine) {
      for (int c0 = ctas.x + warp % W; c0 <= ctas.y; c0 += 32 * W) {  // 32 parts at a time
        const int c = c0 + lane * W;
        float lse = -INFINITY;
        if (c <= ctas.y && MATTN_IN_BOUNDS(kSiteQ4Out, c + pair, p.slots))
          lse = p.ws_lse[(c + pair) * R + r];
        float m = lse;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float m_new = fmaxf(M, m);
        const float ref = m_new == -INFINITY ? 0.0f : m_new;
        const float w = ex2_approx(lse - ref), fix = ex2_approx(M - ref);  // -inf -> 0
        L *= fix;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] *= fix;
        M = m_new;
        const int n = min(32, (ctas.y - c0) / W + 1);
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
          const float wk = __shfl_sync(0xffffffffu, w, k);
          const long long slot = c0 + (long long)k * W + pair;
          if (!MATTN_IN_BOUNDS(kSiteQ4Out, slot, p.slots)) continue;
          const float* part = p.ws_o + (slot * R + r) * D + lane * V;
          float x[V];
          if constexpr (V == 4) {
            const float4 f = *reinterpret_cast<const float4*>(part);
            x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
          } else {
            const float2 f = *reinterpret_cast<const float2*>(part);
            x[0] = f.x, x[1] = f.y;
          }
          L += wk;
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] += wk * x[i];
        }
      }
    }
  }
  if constexpr (W > 1) {  // W = the block's warps: one row
    sh[warp][D] = M;
    sh[warp][D + 1] = L;
#pragma unroll
    for (int i = 0; i < V; ++i) sh[warp][lane * V + i] = acc[i];
    __syncthreads();
    if (warp) return;
#pragma unroll
    for (int k = 1; k < W; ++k) M = fmaxf(M, sh[k][D]);
    L = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const float w = M == -INFINITY ? 1.0f : ex2_approx(sh[k][D] - M);
      L += w * sh[k][D + 1];
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += w * sh[k][lane * V + i];
    }
  }
  if (!mine || !MATTN_IN_BOUNDS(kSiteQ4Out, row, rows)) return;
  const bool any = !(L == 0.0f);  // else no key in any part
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.o) + row * D + lane * V;
#pragma unroll
  for (int i = 0; i < V; i += 2)
    *reinterpret_cast<uint32_t*>(out + i) =
        any ? pack_bf16x2(acc[i] / L, acc[i + 1] / L) : 0u;
  if (lane == 0) p.lse[row] = any ? (M + __log2f(L)) * kLn2 : -INFINITY;
}

template <int D>
cudaError_t launch_merge(const Q4Problem& p, int ctas, cudaStream_t stream) {
  const long long rows = (long long)p.B * p.Hq * p.Sq;
  // One warp per row where a pair is cut into few parts, a block of 4 or 16 warps
  // where the CTAs are at least 8 or 32 times the pairs: parts in turn are what a
  // row waits for (1 sequence x 1 head, 60000 keys, 456 parts: 18 us with 16 warps,
  // 24 with 8, 29 with 4), but 16 warps for 8 parts cost more than they save (7
  // sequences x 8 heads of 64, 16 rows: 68 us against 65).
  const long long pairs = (long long)p.B * p.Hkv;
  if (ctas >= 32 * pairs)
    return launch_early(q4_merge_kernel<D, 16>, (unsigned)rows, 32 * merge_warps(16), 0, stream, p);
  if (ctas >= 8 * pairs)
    return launch_early(q4_merge_kernel<D, 4>, (unsigned)rows, 32 * merge_warps(4), 0, stream, p);
  return launch_early(q4_merge_kernel<D, 1>, (unsigned)((rows + kQ4Warps - 1) / kQ4Warps),
                      32 * merge_warps(1), 0, stream, p);
}

// Up to this many tiles a pair is one CTA's, whatever the workspace: sharing it out
// costs the merge, a launch (1 sequence x 8 heads, 1100 keys, 35 tiles: 11 us alone
// and 12 shared; 2000 keys, 63 tiles: 17 and 12).
constexpr int kQ4DirectTiles = 40;
constexpr int kQ4CtasPerSm = 4;  // most resident CTAs that a call uses

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// CTAs that share `tiles` tiles: a resident wave, or one per four tiles (a
// warp each) where there are fewer.
int q4_ctas(long long tiles, int resident) {
  return (int)std::max(1LL, std::min<long long>(resident, (tiles + kQ4Warps - 1) / kQ4Warps));
}

struct Q4Workspace {
  size_t lse, o, total;  // meta at 0
};

Q4Workspace q4_workspace(long long pairs, int ctas, int R, int D) {
  const size_t slots = (size_t)(pairs + ctas);
  Q4Workspace w;
  w.lse = align256(pairs * sizeof(int2));
  w.o = w.lse + align256(slots * R * sizeof(float));
  w.total = w.o + align256(slots * R * D * sizeof(float));
  return w;
}

template <int D, int NT, int SCORE>
cudaError_t launch_typed(Q4Problem& p, long long tiles, void* ws, size_t ws_bytes,
                         cudaStream_t stream) {
  using C = Q4Cfg<D, NT>;
  static DeviceOnce ready;
  const cudaError_t err = ready.allow_smem(decode_q4_kernel<D, NT, SCORE>, C::kSmem);
  if (err != cudaSuccess) return err;
  static const int per_sm = [] {
    int n = 1;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, decode_q4_kernel<D, NT, SCORE>, kQ4Threads,
                                                  C::kSmem);
    return std::max(1, std::min(n, kQ4CtasPerSm));
  }();
  const long long pairs = (long long)p.B * p.Hkv;
  const int R = p.Hq / p.Hkv * p.Sq;
  // As many CTAs as the workspace has slots for; one per pair, writing o and
  // lse at once, where that is no fewer or pairs are short.
  int ctas = q4_ctas(tiles * pairs, per_sm * sm_count());
  const int want = ctas;
  while (ctas > 1 && q4_workspace(pairs, ctas, R, D).total > ws_bytes) ctas /= 2;
  const bool split = ws && tiles > kQ4DirectTiles && ctas > 1 && (ctas == want || ctas > pairs);
  if (!split) {
    return launch_early(decode_q4_kernel<D, NT, SCORE>, (unsigned)pairs, kQ4Threads, C::kSmem, stream, p);
  }
  const Q4Workspace w = q4_workspace(pairs, ctas, R, D);
  p.slots = pairs + ctas;
  p.ws_meta = static_cast<int2*>(ws);
  p.ws_lse = reinterpret_cast<float*>(static_cast<char*>(ws) + w.lse);
  p.ws_o = reinterpret_cast<float*>(static_cast<char*>(ws) + w.o);
  const cudaError_t e = launch_early(decode_q4_kernel<D, NT, SCORE>, ctas, kQ4Threads, C::kSmem, stream, p);
  return e != cudaSuccess ? e : launch_merge<D>(p, ctas, stream);
}

template <int D, int NT>
cudaError_t launch_score(Q4Problem& p, long long tiles, void* ws, size_t n, cudaStream_t s) {
  switch (((p.variant & ATTN_SCORE_ALIBI) ? 1 : 0) | ((p.variant & ATTN_SCORE_SOFTCAP) ? 2 : 0)) {
    case 0: return launch_typed<D, NT, 0>(p, tiles, ws, n, s);
    case 1: return launch_typed<D, NT, 1>(p, tiles, ws, n, s);
    case 2: return launch_typed<D, NT, 2>(p, tiles, ws, n, s);
    default: return launch_typed<D, NT, 3>(p, tiles, ws, n, s);
  }
}

}  // namespace
}  // namespace mattn

MATTN_API size_t attn_decode_q4_workspace_bytes(int B, int Hq, int Hkv, int Sq, int max_len, int D) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Sq < 1 || max_len < 1 || (D != 64 && D != 128)) return 0;
  using namespace mattn;
  const long long pairs = (long long)B * Hkv;
  const long long tiles = ((long long)max_len + kQ4Tile - 1) / kQ4Tile;
  if (tiles <= kQ4DirectTiles || Hq % Hkv) return 0;
  return q4_workspace(pairs, q4_ctas(tiles * pairs, kQ4CtasPerSm * sm_count()),
                      Hq / Hkv * Sq, D).total;
}

MATTN_API attn_status attn_decode_q4(const void* q, const void* pool, void* o, float* lse, int B,
                                     int Hq, int Hkv, int Sq, int max_len, int D, unsigned variant,
                                     const attn_params* p, const int* seq_lens, int sink,
                                     void* workspace, size_t workspace_bytes,
                                     struct CUstream_st* stream) {
  using namespace mattn;
  if (!p || B < 0 || Hq < 1 || Hkv < 1 || Sq < 0 || max_len < 0 || sink < 0 || Hq % Hkv)
    return ATTN_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || p->dtype != ATTN_BF16) return ATTN_ERR_UNSUPPORTED;
  if (variant & ~(ATTN_MASK_BITS | ATTN_SCORE_BITS)) return ATTN_ERR_INVALID_ARG;
  if (variant & ~(unsigned)(ATTN_MASK_CAUSAL | ATTN_MASK_WINDOW | ATTN_SCORE_ALIBI | ATTN_SCORE_SOFTCAP))
    return ATTN_ERR_UNSUPPORTED;
  if ((variant & ATTN_MASK_WINDOW) && p->window < 1) return ATTN_ERR_INVALID_ARG;
  if ((variant & ATTN_SCORE_SOFTCAP) &&
      !(p->softcap > 0.0f && std::isfinite(p->softcap) && std::isfinite(2.0f / p->softcap)))
    return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(p->scale) || p->scale < 0.0f) return ATTN_ERR_INVALID_ARG;
  if (p->q_offset || p->kv_offset) return ATTN_ERR_UNSUPPORTED;
  if ((long long)(Hq / Hkv) * Sq > kQ4MaxRows || (long long)B * Hkv > 65535)
    return ATTN_ERR_UNSUPPORTED;
  if (!q4_page_ok(p->page_size)) return ATTN_ERR_UNSUPPORTED;
  if (max_len > INT_MAX - 255) return ATTN_ERR_UNSUPPORTED;  // tile ends are int
  if (B == 0 || Sq == 0) return ATTN_OK;
  if (p->num_pages < 1 || p->pages_per_seq < 1 ||
      (long long)p->pages_per_seq * p->page_size < (long long)max_len)
    return ATTN_ERR_INVALID_ARG;
  if (!q || !pool || !o || !lse || !seq_lens || !p->page_table) return ATTN_ERR_INVALID_ARG;
  const void* vecs[] = {q, pool, o};
  for (const void* x : vecs)
    if (reinterpret_cast<uintptr_t>(x) & 15u) return ATTN_ERR_MISALIGNED;
  const void* words[] = {lse, seq_lens, p->page_table, p->alibi_slopes};
  for (const void* x : words)
    if (reinterpret_cast<uintptr_t>(x) & 3u) return ATTN_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return ATTN_ERR_MISALIGNED;

  Q4Problem f{};
  f.q = q;
  f.pool = static_cast<const uint8_t*>(pool);
  f.o = o;
  f.lse = lse;
  f.seq_lens = seq_lens;
  f.table = p->page_table;
  f.slopes = p->alibi_slopes;
  f.B = B;
  f.Hq = Hq;
  f.Hkv = Hkv;
  f.Sq = Sq;
  f.max_len = max_len;
  f.pages_per_seq = p->pages_per_seq;
  f.num_pages = p->num_pages;
  f.shift = 4;
  while ((1 << f.shift) != p->page_size) ++f.shift;
  f.variant = variant;
  f.window = p->window;
  f.sink = sink;
  f.scale2 = (p->scale != 0.0f ? p->scale : 1.0f / std::sqrt((float)D)) * kLog2e;
  f.softcap2 = p->softcap * kLog2e;
  f.softcap_e = 2.0f / p->softcap;

  // most tiles that a sequence can have: its whole length, or sinks and window
  long long tiles = ((long long)max_len + kQ4Tile - 1) / kQ4Tile;
  if (variant & ATTN_MASK_WINDOW)
    tiles = std::min(tiles, ((long long)sink + kQ4Tile - 1) / kQ4Tile +
                                ((long long)p->window + Sq - 1 + 2 * kQ4Tile - 2) / kQ4Tile);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool two = (Hq / Hkv) * Sq > 8;
  if (D == 64)
    return cuda_status(two ? launch_score<64, 2>(f, tiles, workspace, workspace_bytes, s)
                           : launch_score<64, 1>(f, tiles, workspace, workspace_bytes, s));
  return cuda_status(two ? launch_score<128, 2>(f, tiles, workspace, workspace_bytes, s)
                         : launch_score<128, 1>(f, tiles, workspace, workspace_bytes, s));
}

namespace mattn {
MATTN_DEBUG_RECORD_ACCESSORS(decode_q4)
}  // namespace mattn
