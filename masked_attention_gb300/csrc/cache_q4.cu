// The 4-bit paged cache: new key and value rows are quantised into the page
// records at their slots, and rows are read back as bf16. Record layout:
// cache_q4.cuh. Per 32 channels of a row
//
//   s = bf16(max|x| / 7),  code = clamp(rint(x / s), -8, 7) + 8
//
// rint rounds ties to even; s = 0 stores code 8 throughout; a group that holds
// an infinity or NaN gets s = NaN, so it reads back as NaN. The quotient is
// x times an approximate reciprocal, corrected once by its exact remainder:
// q = q0 + (x - q0 s) / s. A tie, an exact k + 1/2, comes out exactly (the error
// of q0, 2^-22, is squared), and since x and s have 8 significant bits every other
// quotient is at least 2^-9 away from a tie; so the codes are those of exact
// division.
//
// Bound by HBM (a bf16 element is 2 bytes, a stored one 0.5625), with the
// quantiser's instructions close behind. A lane holds 16 channels of a row (32 bytes
// of bf16, 8 of codes), half of a scale's, so the largest magnitude takes one
// shuffle. A warp takes a batch of a token's K and V rows, with the slot (read:
// and the codes) of its next batch on the way; where a token's rows do not fill
// batches, the rows of all tokens in a line are cut into batches. 16384 tokens x 8 heads
// of 128 channels written and read: 33.6 us, 0.75 of a plain copy's rate.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "cache_q4.cuh"
#include "host_util.h"
#include "launch.h"

#define MATTN_API extern "C" __attribute__((visibility("default")))

namespace mattn {
namespace {

constexpr int kCacheThreads = 256;
constexpr int kCacheWarps = kCacheThreads / 32;
constexpr int kCacheRows = 4;   // rows in flight per lane group
constexpr int kCachePerSm = 3;  // blocks per SM. 16384 tokens x 8 heads of 128 channels, write and
                                // read: 33.7 us; 4 blocks 36.2; 2 rows at 4 blocks 35.5, 1 row
                                // at 6 blocks 42.9

struct CacheArgs {
  char* x[2];            // K and V rows (store: read, load: written)
  long long sb[2], sh[2], ss[2], span[2];  // bytes
  uint8_t* pool;
  const long long* slots;  // [B][S]
  int B, Hkv, S, num_pages, shift;
  int period;              // batches of rows per token; packed: rows per token
  uint32_t per_row, per_s;  // packed: ceil(2^32 / rows per token), ceil(2^32 / S)
  bool wide;               // rows are 32-byte aligned
};

// The eight codes of a word, exactly: the definition itself.
__device__ __noinline__ uint32_t encode_exact(uint4 v, float s) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
    int c = 0;
    if (s > 0.0f) c = (int)fminf(fmaxf(rintf(__fdiv_rn(x, s)), -8.0f), 7.0f);
    word |= (uint32_t)(c + 8) << (4 * i);
  }
  return word;
}

// Quantises a lane's 16 channels (two neighbouring lanes share a scale): the
// code words and the scale's bf16 bits.
__device__ __forceinline__ void encode(const uint4 (&v)[2], uint32_t (&word)[2], uint32_t& scale) {
  const uint32_t u[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
  uint32_t m2 = 0;  // largest |x| as bits, two at a time: ordered like the values, NaN last
#pragma unroll
  for (int i = 0; i < 8; ++i) m2 = __vmaxu2(m2, u[i] & 0x7fff7fffu);
  m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, 1));
  const uint32_t m = max(m2 & 0xffff0000u, m2 << 16);
  float s = 0.0f;
  if (m >= 0x7f800000u) {
    scale = 0x7fffu;
  } else {
    const __nv_bfloat16 b = __float2bfloat16_rn(__fdiv_rn(__uint_as_float(m), 7.0f));
    scale = *reinterpret_cast<const unsigned short*>(&b);
    s = __bfloat162float(b);
  }
  // kMagic + q is a float whose low mantissa bits hold rint(q)
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
  const float inv = __fdividef(1.0f, s);
  const float2 inv2 = make_float2(inv, inv), s2 = make_float2(-s, -s);
  const float2 up = make_float2(kMagic, kMagic);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      const uint32_t p = u[4 * k + i];
      const float2 x = make_float2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u));
      const float2 q = fmul2(x, inv2);
      const float2 t = fadd2(ffma2(ffma2(q, s2, x), inv2, q), up);
      w = w * 16u + __float_as_uint(t.y);
      w = w * 16u + __float_as_uint(t.x);
    }
    word[k] = w - (0x4b400000u - 8u) * 0x11111111u;  // the magic's bits, off all eight
  }
  // zero, NaN and tiny scales, where the remainder or the reciprocal leaves
  // fp32's normal range
  if (!(s > 1e-30f)) {
    word[0] = encode_exact(v[0], s);
    word[1] = encode_exact(v[1], s);
  }
}

// The eight values of a word, (n - 8) * scale rounded once to bf16: 128 + n has
// n's bits in its mantissa, n - 8 is exact, and the packed product rounds.
__device__ __forceinline__ uint4 decode(uint32_t w, uint32_t scale) {
  const uint32_t s2 = scale | scale << 16, off = 0x43084308u;  // 136
  uint32_t p[4];  // pairs (i, i + 4)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t raw = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 n = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&raw),
                                     *reinterpret_cast<const __nv_bfloat162*>(&off));
    const __nv_bfloat162 x = __hmul2(n, *reinterpret_cast<const __nv_bfloat162*>(&s2));
    p[i] = *reinterpret_cast<const uint32_t*>(&x);
  }
  return make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410),
                    __byte_perm(p[0], p[1], 0x7632), __byte_perm(p[2], p[3], 0x7632));
}

// 32 bytes of a row: one access where its rows are aligned to that (`wide`),
// else two, which then leave every 32-byte sector to two instructions.
__device__ __forceinline__ void load32(const uint4* p, bool wide, uint4 (&v)[2]) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x),
                   "=r"(v[1].y), "=r"(v[1].z), "=r"(v[1].w)
                 : "l"(p));
  } else {
    v[0] = p[0];
    v[1] = p[1];
  }
}

__device__ __forceinline__ void store32(uint4* p, bool wide, const uint4& a, const uint4& b) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a.x), "r"(a.y),
                 "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    p[0] = a;
    p[1] = b;
  }
}

// Units of a batch of rows (kCacheRows per lane group); a warp takes every
// stride-th. A unit is a batch of one token's K and V rows, the batch first, or
// (packed) the next rows of all tokens' in a line. Where a unit begins, kept without
// divisions: batch is the batch or (packed) the row of its token.
struct Cursor {
  long long u, token;
  int batch, b, s;
};

template <int D, bool kLoad, bool kPacked>
__global__ void __launch_bounds__(kCacheThreads, kCachePerSm)
    cache_q4_kernel(const CacheArgs a) {
  constexpr int R = kCacheRows;
  constexpr int LANES = D / 16;     // lanes per row
  constexpr int SUBS = 32 / LANES;  // rows side by side in a warp
  const int lane = threadIdx.x & 31, part = lane % LANES, sub = lane / LANES;
  const Q4Layout L{D, 1 << a.shift};
  const int rows = 2 * a.Hkv;  // K rows of all heads, then V rows
  const long long tokens = (long long)a.B * a.S;
  const long long units = kPacked ? (tokens * rows + SUBS * R - 1) / (SUBS * R) : tokens * a.period;
  const long long stride = (long long)gridDim.x * kCacheWarps;
  Cursor c;
  c.u = (long long)blockIdx.x * kCacheWarps + (threadIdx.x >> 5);
  early_start();
  if (c.u >= units) return;
  constexpr int kStep = kPacked ? SUBS * R : 1;
  c.token = c.u * kStep / a.period;
  c.batch = (int)(c.u * kStep % a.period);
  c.b = (int)(c.token / a.S);
  c.s = (int)(c.token % a.S);
  const long long dt = stride * kStep / a.period;
  const int dbatch = (int)(stride * kStep % a.period), db = (int)(dt / a.S), ds = (int)(dt % a.S);
  const long long page_bytes = (long long)a.Hkv * L.bytes();
  auto advance = [&](Cursor& k) {
    k.u += stride;
    k.batch += dbatch;
    const int carry = k.batch >= a.period;
    k.batch -= carry ? a.period : 0;
    k.token += dt + carry;
    k.s += ds + carry;
    k.b += db;
    if (k.s >= a.S) {
      k.s -= a.S;
      ++k.b;
    }
  };
  // Row r of a unit for this lane group: its token (`ahead` of the unit's first; -1: no
  // row) and its row there.
  auto place = [&](const Cursor& k, int r, int& row) -> int {
    row = (kPacked ? k.batch : k.batch * SUBS * R) + r * SUBS + sub;
    if constexpr (!kPacked) return row < rows ? 0 : -1;
    const int ahead = (int)__umulhi(row, a.per_row);
    row -= ahead * rows;
    return k.token + ahead < tokens ? ahead : -1;
  };
  constexpr int kSlots = kPacked ? R : 1;  // slots of a unit: one token's, or each row's
  auto slots_of = [&](const Cursor& k, long long (&slot)[kSlots]) {
#pragma unroll
    for (int r = 0; r < kSlots; ++r) {
      int row, ahead = 0;
      if constexpr (kPacked) ahead = place(k, r, row);
      slot[r] = k.u < units && ahead >= 0 ? a.slots[k.token + ahead] : -1;
    }
  };
  // its bf16 row; nullptr: none
  auto bf16_row = [&](const Cursor& k, int r) -> uint4* {
    int row;
    const int ahead = place(k, r, row);
    int b = k.b, s = k.s;
    if constexpr (kPacked) {  // over the sequence's end; a unit has at most 16 tokens
      s += ahead;
      const int over = a.S > 16 ? s >= a.S : (int)__umulhi(s, a.per_s);
      b += over;
      s -= over * a.S;
    }
    const int v = row >= a.Hkv ? 1 : 0, h = row - v * a.Hkv;
    const long long at = v ? b * a.sb[1] + s * a.ss[1] + h * a.sh[1]
                           : b * a.sb[0] + s * a.ss[0] + h * a.sh[0];
    if (ahead < 0 || !MATTN_IN_BOUNDS(kSiteCacheRow, at + part * 32, a.span[v] - 31)) return nullptr;
    return reinterpret_cast<uint4*>((v ? a.x[1] : a.x[0]) + at + part * 32);
  };
  // its codes and scale in the record, for a slot of the pool; nullptr: none
  auto code_row = [&](const Cursor& k, int r, const long long (&slots)[kSlots],
                      uint8_t*& scale) -> uint8_t* {
    int row;
    const int ahead = place(k, r, row);
    const long long slot = slots[kPacked ? r : 0];
    const long long page = slot >> a.shift;
    if (ahead < 0 || slot < 0 || page >= a.num_pages) return nullptr;
    const int v = row >= a.Hkv ? 1 : 0, h = row - v * a.Hkv;
    uint8_t* rec = a.pool + page * page_bytes + (long long)h * L.bytes();
    const int in_page = (int)(slot & (L.page - 1));
    scale = rec + (v ? L.v_scales() : L.k_scales()) + in_page * L.scale_row() + part / 2 * 2;
    uint8_t* code = rec + (v ? L.v_codes() : 0) + in_page * L.code_row() + part * 8;
    [[maybe_unused]] const long long pool_bytes = a.num_pages * page_bytes;
    if (!MATTN_IN_BOUNDS(kSiteCacheRec, code + 7 - a.pool, pool_bytes) ||
        !MATTN_IN_BOUNDS(kSiteCacheRec, scale + 1 - a.pool, pool_bytes))
      return nullptr;
    return code;
  };

  if constexpr (!kLoad) {
    long long slot[kSlots];
    slots_of(c, slot);
    while (c.u < units) {
      uint4 raw[R][2];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint4* x = bf16_row(c, r);
        raw[r][0] = raw[r][1] = make_uint4(0, 0, 0, 0);
        if (x) load32(x, a.wide, raw[r]);
      }
      const Cursor now = c;
      advance(c);
      long long slot_next[kSlots];
      slots_of(c, slot_next);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        uint32_t word[2], sc;
        encode(raw[r], word, sc);
        uint8_t* scale;
        uint8_t* code = code_row(now, r, slot, scale);
        if (!code) continue;
        *reinterpret_cast<uint2*>(code) = make_uint2(word[0], word[1]);
        if (part % 2 == 0) *reinterpret_cast<unsigned short*>(scale) = (unsigned short)sc;
      }
#pragma unroll
      for (int r = 0; r < kSlots; ++r) slot[r] = slot_next[r];
    }
  } else {
    // the codes of the next unit, and the slots of the one after it, are on
    // their way while a unit is written
    auto fetch = [&](const Cursor& k, const long long (&slot)[kSlots], uint2 (&word)[R],
                     uint32_t (&sc)[R]) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        uint8_t* scale;
        const uint8_t* code = code_row(k, r, slot, scale);
        word[r] = code ? *reinterpret_cast<const uint2*>(code) : make_uint2(0x88888888u, 0x88888888u);
        sc[r] = code ? *reinterpret_cast<const unsigned short*>(scale) : 0u;
      }
    };
    uint2 word[R];
    uint32_t sc[R];
    long long slot[kSlots];
    slots_of(c, slot);
    fetch(c, slot, word, sc);
    Cursor ahead = c;
    advance(ahead);
    slots_of(ahead, slot);
    while (c.u < units) {
      uint2 word_next[R];
      uint32_t sc_next[R];
      const Cursor next = ahead;
      if (next.u < units) fetch(next, slot, word_next, sc_next);
      advance(ahead);
      slots_of(ahead, slot);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        uint4* x = bf16_row(c, r);
        if (!x) continue;
        store32(x, a.wide, decode(word[r].x, sc[r]), decode(word[r].y, sc[r]));
      }
      c = next;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        word[r] = word_next[r];
        sc[r] = sc_next[r];
      }
    }
  }
}

template <int D, bool kLoad>
cudaError_t launch_cache(CacheArgs& a, cudaStream_t stream) {
  constexpr int kBatch = 32 / (D / 16) * kCacheRows;
  const long long rows = 2LL * a.Hkv, tokens = (long long)a.B * a.S;
  const long long batches = (rows + kBatch - 1) / kBatch;
  // Packed where a token's rows leave more than a quarter of its batches empty: its
  // rows cost more to find, but no lane waits. Write and read, in place of batches of
  // one token's: 91993 tokens x 1 head of 64: 23 us against 185; 16384 x 4 of 128: 24
  // against 33, x 6 (12 of 16 rows): 35 against 33, x 8: 43 against 34.
  const bool packed = 4 * rows < 3 * batches * kBatch;
  const long long units = packed ? (tokens * rows + kBatch - 1) / kBatch : tokens * batches;
  a.period = (int)(packed ? rows : batches);
  a.per_row = (uint32_t)((0xffffffffull + rows) / rows);
  a.per_s = a.S > 1 ? (uint32_t)((0xffffffffull + a.S) / a.S) : 0;
  const int blocks = (int)std::min<long long>(kCachePerSm * sm_count(),
                                              (units + kCacheWarps - 1) / kCacheWarps);
  return packed ? launch_early(cache_q4_kernel<D, kLoad, true>, blocks, kCacheThreads, 0, stream, a)
                : launch_early(cache_q4_kernel<D, kLoad, false>, blocks, kCacheThreads, 0, stream, a);
}

attn_status run_cache(bool load, const attn_view* k, const attn_view* v, const long long* slots,
                      void* pool, int num_pages, int page_size, int B, int Hkv, int S, int D,
                      cudaStream_t stream) {
  if (B < 0 || Hkv < 1 || S < 0 || num_pages < 1) return ATTN_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || !q4_page_ok(page_size)) return ATTN_ERR_UNSUPPORTED;
  if (B == 0 || S == 0) return ATTN_OK;
  if (!k || !v || !k->data || !v->data || !slots || !pool) return ATTN_ERR_INVALID_ARG;
  CacheArgs a{};
  const attn_view* x[] = {k, v};
  for (int t = 0; t < 2; ++t) {
    const attn_view& w = *x[t];
    if (w.stride_b < 0 || w.stride_h < 0 || w.stride_s < 0) return ATTN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(w.data) & 15u) || (B > 1 && w.stride_b % 8) ||
        (Hkv > 1 && w.stride_h % 8) || (S > 1 && w.stride_s % 8))
      return ATTN_ERR_MISALIGNED;
    // rows that are written have to be distinct places
    if (load && ((B > 1 && !w.stride_b) || (Hkv > 1 && !w.stride_h) || (S > 1 && !w.stride_s)))
      return ATTN_ERR_INVALID_ARG;
    a.x[t] = static_cast<char*>(w.data);
    a.sb[t] = B > 1 ? w.stride_b * 2 : 0;
    a.sh[t] = Hkv > 1 ? w.stride_h * 2 : 0;
    a.ss[t] = S > 1 ? w.stride_s * 2 : 0;
    a.span[t] = (B - 1) * a.sb[t] + (Hkv - 1) * a.sh[t] + (S - 1) * a.ss[t] + 2LL * D;
  }
  if ((reinterpret_cast<uintptr_t>(pool) & 15u) || (reinterpret_cast<uintptr_t>(slots) & 7u))
    return ATTN_ERR_MISALIGNED;
  a.wide = true;
  for (int t = 0; t < 2; ++t)
    a.wide = a.wide && !((reinterpret_cast<uintptr_t>(a.x[t]) | a.sb[t] | a.sh[t] | a.ss[t]) & 31);
  a.pool = static_cast<uint8_t*>(pool);
  a.slots = slots;
  a.Hkv = Hkv;
  a.S = S;
  a.B = B;
  if (S == 1) {  // the batch is the sequence
    for (int t = 0; t < 2; ++t) a.ss[t] = a.sb[t];
    a.S = B;
    a.B = 1;
  }
  a.num_pages = num_pages;
  a.shift = 4;
  while ((1 << a.shift) != page_size) ++a.shift;
  if (load) return cuda_status(D == 64 ? launch_cache<64, true>(a, stream) : launch_cache<128, true>(a, stream));
  return cuda_status(D == 64 ? launch_cache<64, false>(a, stream) : launch_cache<128, false>(a, stream));
}

}  // namespace
}  // namespace mattn

MATTN_API size_t attn_cache_q4_bytes(int num_pages, int Hkv, int page_size, int D) {
  if (num_pages < 1 || Hkv < 1 || (D != 64 && D != 128) || !mattn::q4_page_ok(page_size)) return 0;
  return (size_t)num_pages * Hkv * mattn::Q4Layout{D, page_size}.bytes();
}

MATTN_API attn_status attn_cache_store_q4(const attn_view* k, const attn_view* v,
                                          const long long* slots, void* pool, int num_pages,
                                          int page_size, int B, int Hkv, int S, int D,
                                          struct CUstream_st* stream) {
  return mattn::run_cache(false, k, v, slots, pool, num_pages, page_size, B, Hkv, S, D,
                          reinterpret_cast<cudaStream_t>(stream));
}

MATTN_API attn_status attn_cache_load_q4(const void* pool, int num_pages, int page_size,
                                         const long long* slots, const attn_view* k,
                                         const attn_view* v, int B, int Hkv, int S, int D,
                                         struct CUstream_st* stream) {
  return mattn::run_cache(true, k, v, slots, const_cast<void*>(pool), num_pages, page_size, B, Hkv,
                          S, D, reinterpret_cast<cudaStream_t>(stream));
}

namespace mattn {
MATTN_DEBUG_RECORD_ACCESSORS(cache_q4)
}  // namespace mattn
