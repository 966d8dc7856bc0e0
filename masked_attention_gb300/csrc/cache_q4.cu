// The 4-bit paged cache: new key and value rows are quantised into the page
// records at their slots, and rows are read back as bf16. Record layout:
// cache_q4.cuh. Per 32 channels of a row
//
//   s = bf16(max|x| / 7),  code = clamp(rint(x / s), -8, 7) + 8
//
// rint rounds ties to even; s = 0 stores code 8 throughout; a group that holds
// an infinity or NaN gets s = NaN, so it reads back as NaN. x / s and the tie
// are decided exactly, so the codes do not depend on how the quotient is
// computed: c = rint(x / s) from an approximate reciprocal, then the
// remainder x - c s (exact in fp32: x and s have 8 significant bits, c three)
// tells whether the exact quotient could have rounded elsewhere, and only
// then the group's lane divides.
//
// Bound by HBM (a bf16 element is 2 bytes, a stored one 0.5625). A lane
// holds 8 channels of a row: 16 bytes of bf16, one 4-byte word of codes; a
// scale's 32 channels are four neighbouring lanes. K and V rows of a token and
// head are handled together, several rows per lane in flight.
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
constexpr int kCacheRows = 2;  // (K, V) row pairs in flight per lane group

struct CacheArgs {
  char* x[2];            // K and V rows (store: read, load: written)
  long long sb[2], sh[2], ss[2], span[2];  // bytes
  uint8_t* pool;
  const long long* slots;  // [B][S]
  int Hkv, S, num_pages, shift;
  long long units;  // row pairs: tokens * heads
};

// The eight codes of a lane, exactly: the definition itself.
__device__ __noinline__ uint32_t encode_exact(const float* x, float s) {
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    int c = 0;
    if (s > 0.0f) c = (int)fminf(fmaxf(rintf(__fdiv_rn(x[i], s)), -8.0f), 7.0f);
    word |= (uint32_t)(c + 8) << (4 * i);
  }
  return word;
}

// Quantises a lane's 8 channels (four lanes share a scale): the code word and
// the scale's bf16 bits.
__device__ __forceinline__ void encode(const uint4& v, uint32_t& word, uint32_t& scale) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  float x[8];
  uint32_t m = 0;  // largest |x| as bits: orders like the values, NaN last
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    m = max(m, max((u[i] << 16) & 0x7fff0000u, u[i] & 0x7fff0000u));
  }
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  float s = 0.0f;
  if (m >= 0x7f800000u) {
    scale = 0x7fffu;
  } else {
    const __nv_bfloat16 b = __float2bfloat16_rn(__fdiv_rn(__uint_as_float(m), 7.0f));
    scale = *reinterpret_cast<const unsigned short*>(&b);
    s = __bfloat162float(b);
  }
  // fast form: kMagic + c is a float whose low mantissa bits hold c
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
  const float inv = __fdividef(1.0f, s);
  float worst = s > 1e-30f ? 0.0f : INFINITY;  // tiny, zero, NaN scales: the exact form
  word = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    const float t = fmaf(x[i], inv, kMagic);
    const float c = t - kMagic;
    worst = fmaxf(worst, fabsf(fmaf(-c, s, x[i])));
    word = word * 16u + (__float_as_uint(t) - 0x4b400000u + 8u);
  }
  // |remainder| below s/2 by more than the reciprocal's error: c is right
  if (!(worst < s * (0.5f - 1e-5f))) word = encode_exact(x, s);
}

template <int D, bool kLoad>
__global__ void __launch_bounds__(kCacheThreads) cache_q4_kernel(const CacheArgs a) {
  constexpr int LANES = D / 8;      // lanes per row
  constexpr int SUBS = 32 / LANES;  // rows side by side in a warp
  const int lane = threadIdx.x & 31, chunk = lane % LANES, sub = lane / LANES;
  const Q4Layout L{D, 1 << a.shift};
  const long long warp = (long long)blockIdx.x * (kCacheThreads / 32) + (threadIdx.x >> 5);
  const long long step = (long long)gridDim.x * (kCacheThreads / 32) * SUBS * kCacheRows;
  for (long long u0 = warp * SUBS * kCacheRows; u0 < a.units; u0 += step) {
    long long at[kCacheRows][2];       // byte offset of the row's chunk in K and V
    uint8_t* rec[kCacheRows];          // the row's page record, nullptr: no slot
    int row[kCacheRows];               // its row in the page
    bool have[kCacheRows];
    uint4 raw[kCacheRows][2];
    uint32_t code[kCacheRows][2], sc[kCacheRows][2];
#pragma unroll
    for (int r = 0; r < kCacheRows; ++r) {
      const long long u = u0 + r * SUBS + sub;
      have[r] = u < a.units;
      rec[r] = nullptr;
      row[r] = 0;
      at[r][0] = at[r][1] = 0;
      if (!have[r]) continue;
      const long long token = u / a.Hkv;
      const int h = (int)(u - token * a.Hkv);
      const long long b = token / a.S, s = token - b * a.S;
      const long long slot = a.slots[token];
      const long long page = slot >> a.shift;
      if (slot >= 0 && page < a.num_pages) {
        rec[r] = a.pool + ((size_t)page * a.Hkv + h) * L.bytes();
        row[r] = (int)(slot & (L.page - 1));
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        at[r][t] = b * a.sb[t] + h * a.sh[t] + s * a.ss[t] + chunk * 16;
        if (!MATTN_IN_BOUNDS(kSiteCacheRow, at[r][t], a.span[t] - 15)) have[r] = false;
      }
    }
    if constexpr (!kLoad) {
#pragma unroll
      for (int r = 0; r < kCacheRows; ++r)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          raw[r][t] = have[r] && rec[r] ? *reinterpret_cast<const uint4*>(a.x[t] + at[r][t])
                                        : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < kCacheRows; ++r)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          encode(raw[r][t], code[r][t], sc[r][t]);
          if (!have[r] || !rec[r]) continue;
          *reinterpret_cast<uint32_t*>(rec[r] + (t ? L.v_codes() : 0) + row[r] * L.code_row() +
                                       chunk * 4) = code[r][t];
          if (chunk % 4 == 0)
            *reinterpret_cast<unsigned short*>(rec[r] + (t ? L.v_scales() : L.k_scales()) +
                                               row[r] * L.scale_row() + chunk / 4 * 2) =
                (unsigned short)sc[r][t];
        }
    } else {
#pragma unroll
      for (int r = 0; r < kCacheRows; ++r)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          code[r][t] = 0;
          sc[r][t] = 0;  // no slot: (0 - 8) * 0, stored as zeros below
          if (!have[r] || !rec[r]) continue;
          code[r][t] = *reinterpret_cast<const uint32_t*>(
              rec[r] + (t ? L.v_codes() : 0) + row[r] * L.code_row() + chunk * 4);
          sc[r][t] = *reinterpret_cast<const unsigned short*>(
              rec[r] + (t ? L.v_scales() : L.k_scales()) + row[r] * L.scale_row() + chunk / 4 * 2);
        }
#pragma unroll
      for (int r = 0; r < kCacheRows; ++r)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!have[r]) continue;
          const float s = __uint_as_float(sc[r][t] << 16);
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float lo = (float)(int)((code[r][t] >> (8 * i)) & 15u) - 8.0f;
            const float hi = (float)(int)((code[r][t] >> (8 * i + 4)) & 15u) - 8.0f;
            o[i] = rec[r] ? pack_bf16x2(lo * s, hi * s) : 0u;
          }
          *reinterpret_cast<uint4*>(a.x[t] + at[r][t]) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
  }
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
    a.x[t] = static_cast<char*>(w.data);
    a.sb[t] = B > 1 ? w.stride_b * 2 : 0;
    a.sh[t] = Hkv > 1 ? w.stride_h * 2 : 0;
    a.ss[t] = S > 1 ? w.stride_s * 2 : 0;
    a.span[t] = (B - 1) * a.sb[t] + (Hkv - 1) * a.sh[t] + (S - 1) * a.ss[t] + 2LL * D;
  }
  if ((reinterpret_cast<uintptr_t>(pool) & 15u) || (reinterpret_cast<uintptr_t>(slots) & 7u))
    return ATTN_ERR_MISALIGNED;
  a.pool = static_cast<uint8_t*>(pool);
  a.slots = slots;
  a.Hkv = Hkv;
  a.S = S;
  a.num_pages = num_pages;
  a.shift = 4;
  while ((1 << a.shift) != page_size) ++a.shift;
  a.units = (long long)B * S * Hkv;
  const long long per_block = (long long)(kCacheThreads / 32) * (32 / (D / 8)) * kCacheRows;
  const int blocks = (int)std::min<long long>(8LL * sm_count(), (a.units + per_block - 1) / per_block);
  if (load) {
    if (D == 64) cache_q4_kernel<64, true><<<blocks, kCacheThreads, 0, stream>>>(a);
    else cache_q4_kernel<128, true><<<blocks, kCacheThreads, 0, stream>>>(a);
  } else {
    if (D == 64) cache_q4_kernel<64, false><<<blocks, kCacheThreads, 0, stream>>>(a);
    else cache_q4_kernel<128, false><<<blocks, kCacheThreads, 0, stream>>>(a);
  }
  return cuda_status(cudaGetLastError());
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
