// Kernels and argument checks of the norm and rotation, shared by the calls with one position
// per token (norm_rope.cu) and with one per axis (norm_rope_axes.cu).
//
// Per-head RMS norm of queries and keys with the position rotation, in one
// pass from the projection's layout to the attention's (any strides), and its
// gradient. A row is one head of one token, D channels:
//
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r,  y = n w,  z = R(pos) y
//   z[c] = y[c] cos - y[c'] sin,  z[c'] = y[c'] cos + y[c] sin
// for the channel pairs (c, c') of the rotation; channels past rot_dim pass. With several
// axes (kAxes) pos is the position on the axis of the pair (c, c').
//
// Gradient, from the row's x (r and n are computed again) and dz:
//   dy = R(pos)^T dz,  dw = sum over rows of dy n,  dn = dy w,
//   dx = r (dn - n mean(dn n))
//
// Bound by HBM: a row is read and written once (forward), or read twice and
// written once (gradient); what competes are the instructions per row. A lane
// holds 32 bytes of a row, two 16-byte chunks that are each other's rotation
// partners (or, past rot_dim and interleaved, any two), so a rotation needs no
// exchange between lanes, a row takes 4 to 16 lanes, and its sums two to four
// shuffles; the arithmetic is on packed fp32 pairs. (With one chunk per lane and the
// partner's by shuffle: 128 instead of 95 instructions per two rows of
// 128 bf16 channels, and 245 instead of 185 in the gradient.) A block's 8 warps take
// 8 consecutive tokens (fewer tokens: the heads of one). An item is kRows rows per lane
// group; the next item's rows arrive in shared memory (asynchronous copies, each
// thread its own) while one is computed, and a token's cos and sin stay in
// registers from one item to the next. Queries and keys are two passes over the
// tokens, so that one set of weights is held at a time. All arithmetic is fp32;
// each output is rounded once. 16384 tokens x 40 heads of 128 bf16 channels: 60 us, 0.84
// of a plain copy's rate; the gradient of 32768 x 32 heads: 144 us, 0.83.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "host_util.h"
#include "launch.h"

namespace mattn {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRopePerSm = 2;  // blocks per SM: 3, with 80 registers, spilled (66 against 60 us
                               // on 16384 tokens x 40 heads of 128 bf16 channels)
// Row steps (a row of each lane group) per item. The gradient needs more rows in
// flight at its 128 registers: 3 against 1 is 144 against 153 us on the training
// shape (B 8, 16 + 16 heads, S 4096, D 128); the forward: 2: 60 us, 1: 67, 3: 62.
template <bool kBwd>
constexpr int rope_rows() { return kBwd ? 3 : 2; }
constexpr int kRopeMaxBlocks = 608;  // most blocks: the gradient's workspace holds one partial
                                     // weight gradient of each

struct View {
  char* p;
  long long sb, sh, ss;  // bytes
  long long bytes;       // extent, for the debug build's checks
};

struct RopeArgs {
  View x[2], z[2], dx[2];  // queries, keys: input, output (gradient: dz), gradient out
  const float* w[2];       // norm weights or nullptr (no norm)
  const float* table;      // [max_pos][rot]: cos then sin, or nullptr (no rotation)
  const int* pos;          // [B][S] or nullptr (position s)
  float* part;             // gradient: [blocks][2][D]
  float eps;
  int S, H[2], rot, max_pos;
  int together;         // warps of a block with tokens of their own: 8 or 1
  int per_item;         // heads per item
  int items[2];         // items per token
  long long groups;     // ceil(tokens / together)
  int B;
  // several axes: pos is [axes][B][S], pos_axis = B * S; the axis of pair i in bits
  // 2 (i % 32) and up of pair_axis[i / 32]
  int axes;
  long long pos_axis;
  unsigned long long pair_axis[2];
};
constexpr int kRopeMaxAxes = 4;

template <bool kBf16>
struct Chunk {  // 16 bytes of a row
  static constexpr int N = kBf16 ? 8 : 4;
};

// Channel pairs, for the packed fp32 instructions (two lanes each).
template <bool kBf16, int P>
__device__ __forceinline__ void unpack(const uint4& v, float2 (&f)[P]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if constexpr (kBf16)
      f[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
    else
      f[i] = make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
  }
}

template <bool kBf16, int P>
__device__ __forceinline__ uint4 pack(const float2 (&f)[P]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if constexpr (kBf16) {
      u[i] = pack_bf16x2(f[i].x, f[i].y);
    } else {
      u[2 * i] = __float_as_uint(f[i].x);
      u[2 * i + 1] = __float_as_uint(f[i].y);
    }
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// The two chunks of a row that a lane holds: partners of the rotation where
// they lie below rot_dim, else one in each half of what is left. Neighbouring lanes'
// chunks are neighbours, so an access covers whole sectors (two neighbouring chunks
// per lane: 165 against 124 us, interleaved, 15795 tokens x 88 heads of 64 fp32 channels).
template <int N, int LANES>
__device__ __forceinline__ void lane_chunks(const RopeArgs& a, bool inter, int part, int (&ch)[2]) {
  const int pairs = a.table && !inter ? a.rot / (2 * N) : 0;  // lanes with partners
  if (part < pairs) {
    ch[0] = part * N;
    ch[1] = part * N + a.rot / 2;
  } else {
    ch[0] = (part + pairs) * N;
    ch[1] = (part + LANES) * N;
  }
}

// A token's rotation as the lane's channels see it:
//   z0 = c0 y0 + e0 y0',  z1 = c1 y1 + e1 y1'
// with y' the other chunk or, interleaved, the neighbouring channel. The transpose
// is the same with e negated. A chunk past rot_dim does not turn: its y' is left out, which
// may be an infinity (0 times it is NaN).
template <int N, bool kInter>
struct Rotation {
  float2 c[2][N / 2], e[2][N / 2];

  // Worked out where it is used: kept for the rows, it cost the gradient 2 us of 146.
  static __device__ __forceinline__ bool turns(const RopeArgs& a, const int (&ch)[2], int k) {
    return a.table && ch[kInter ? k : 0] < a.rot;
  }

  __device__ __forceinline__ void load(const RopeArgs& a, int pos, const int (&ch)[2]) {
    const float* row = a.table + (size_t)pos * a.rot;
    const int half = a.rot / 2;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!turns(a, ch, k)) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          c[k][i] = both(1.0f);
          e[k][i] = both(0.0f);
        }
      } else if constexpr (kInter) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          const float cs = row[ch[k] / 2 + i], sn = row[half + ch[k] / 2 + i];
          c[k][i] = both(cs);
          e[k][i] = make_float2(-sn, sn);
        }
      } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          const float4 cv = *reinterpret_cast<const float4*>(row + ch[0] + i);
          const float4 sv = *reinterpret_cast<const float4*>(row + half + ch[0] + i);
          c[k][i / 2] = make_float2(cv.x, cv.y);
          c[k][i / 2 + 1] = make_float2(cv.z, cv.w);
          const float2 sign = both(k ? 1.0f : -1.0f);
          e[k][i / 2] = fmul2(sign, make_float2(sv.x, sv.y));
          e[k][i / 2 + 1] = fmul2(sign, make_float2(sv.z, sv.w));
        }
      }
    }
  }

  // The same with a position per axis. Four neighbouring pairs of one axis (axes that take
  // runs of pairs) are two 16-byte loads, others eight of 4 bytes.
  __device__ __forceinline__ void load_axes(const RopeArgs& a, const int (&pos)[kRopeMaxAxes],
                                            const int (&ch)[2]) {
    const int half = a.rot / 2;
    auto row = [&](unsigned axis) {
      const int lo = axis & 1 ? pos[1] : pos[0], hi = axis & 1 ? pos[3] : pos[2];
      return a.table + (size_t)(axis & 2 ? hi : lo) * a.rot;
    };
    constexpr int Q = kInter ? N / 2 : N;  // pairs of a chunk: one chunk's, or both chunks' same
    constexpr int G = Q < 4 ? Q : 4;
#pragma unroll
    for (int k = 0; k < (kInter ? 2 : 1); ++k) {
      const int first = kInter ? ch[k] / 2 : ch[0];
      if (!turns(a, ch, k)) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          c[k][i] = both(1.0f);
          e[k][i] = both(0.0f);
          if constexpr (!kInter) {
            c[1][i] = both(1.0f);
            e[1][i] = both(0.0f);
          }
        }
        continue;
      }
#pragma unroll
      for (int g = 0; g < Q; g += G) {
        const int at = first + g;  // a multiple of G: one word holds the group's axes
        const unsigned bits =
            (unsigned)(a.pair_axis[at >> 5] >> (2 * (at & 31))) & ((1u << (2 * G)) - 1u);
        float cs[G], sn[G];
        if (G == 4 && bits == (bits & 3u) * 0x55u) {
          const float* r = row(bits & 3u) + at;
          const float4 cv = *reinterpret_cast<const float4*>(r);
          const float4 sv = *reinterpret_cast<const float4*>(r + half);
          cs[0] = cv.x, cs[1] = cv.y, cs[G - 2] = cv.z, cs[G - 1] = cv.w;
          sn[0] = sv.x, sn[1] = sv.y, sn[G - 2] = sv.z, sn[G - 1] = sv.w;
        } else {
#pragma unroll
          for (int i = 0; i < G; ++i) {
            const float* r = row((bits >> (2 * i)) & 3u) + at + i;
            cs[i] = r[0];
            sn[i] = r[half];
          }
        }
#pragma unroll
        for (int i = 0; i < G; ++i) {
          if constexpr (kInter) {
            c[k][g + i] = both(cs[i]);
            e[k][g + i] = make_float2(-sn[i], sn[i]);
          } else {
            float2 &c0 = c[0][(g + i) / 2], &c1 = c[1][(g + i) / 2];
            float2 &e0 = e[0][(g + i) / 2], &e1 = e[1][(g + i) / 2];
            if (i & 1) {
              c0.y = c1.y = cs[i];
              e0.y = -sn[i], e1.y = sn[i];
            } else {
              c0.x = c1.x = cs[i];
              e0.x = -sn[i], e1.x = sn[i];
            }
          }
        }
      }
    }
  }

  // c y + e y'
  __device__ __forceinline__ float2 turn(const RopeArgs& a, const int (&ch)[2],
                                         const float2 (&y)[2][N / 2], int k, int i) const {
    const float2 other = kInter ? make_float2(y[k][i].y, y[k][i].x) : y[1 - k][i];
    return ffma2(y[k][i], c[k][i], turns(a, ch, k) ? fmul2(other, e[k][i]) : both(0.0f));
  }
};

// Sum over the LANES lanes of a row.
template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int d = 1; d < LANES; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

// 16-byte asynchronous copy into the thread's own place of shared memory.
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src))
               : "memory");
}

template <int D, bool kBf16, bool kInter, bool kBwd, bool kAxes>
__global__ void __launch_bounds__(kRopeThreads, kRopePerSm)
    norm_rope_kernel(const RopeArgs a) {
  constexpr int N = Chunk<kBf16>::N, P = N / 2;
  constexpr int LANES = D / (2 * N);  // lanes per row
  constexpr int SUBS = 32 / LANES;    // rows side by side in a warp
  constexpr int kRows = rope_rows<kBwd>();
  constexpr int kSlots = kBwd ? 4 : 2;  // two chunks of x, and of the gradient's dz
  extern __shared__ uint4 ring[];       // [2][kRows][kSlots][threads]: a thread's own chunks
  auto place = [&](int buf, int r, int slot) -> uint4& {
    return ring[((buf * kRows + r) * kSlots + slot) * kRopeThreads + threadIdx.x];
  };
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / LANES;
  early_start();
  const int apart = warp / a.together;       // head item within the group
  const int spread = kRopeWarps / a.together;
  int ch[2];
  lane_chunks<N, LANES>(a, kInter, lane % LANES, ch);
  const int c0 = ch[0] * (16 / N), c1 = ch[1] * (16 / N);  // bytes, c0 < c1

  for (int t = 0; t < 2; ++t) {
    if (a.H[t] == 0) {  // no rows: their share of a weight gradient is 0
      if constexpr (kBwd)
        for (int c = threadIdx.x; c < D; c += kRopeThreads)
          a.part[(size_t)blockIdx.x * 2 * D + t * D + c] = 0.0f;
      continue;
    }
    const bool norm = a.w[t] != nullptr;
    auto weight = [&](int k, int i) {
      return norm ? make_float2(a.w[t][ch[k] + 2 * i], a.w[t][ch[k] + 2 * i + 1]) : both(1.0f);
    };
    float2 w[2][P], dw[2][P];  // the gradient's weights and sums
    if constexpr (kBwd) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < P; ++i) {
          w[k][i] = weight(k, i);
          dw[k][i] = both(0.0f);
        }
    }
    // the block's run of items, the head items of a token group one after the other
    const int per_group = (a.items[t] + spread - 1) / spread;
    const long long n = a.groups * per_group;
    const long long u0 = n * blockIdx.x / gridDim.x;
    const int count = (int)(n * (blockIdx.x + 1) / gridDim.x - u0);
    // the next item's token (b, s) and head item
    const long long token0 = u0 / per_group * a.together + warp % a.together;
    int b = (int)(token0 / a.S), s = (int)(token0 - (long long)b * a.S);
    int it = (int)(u0 % per_group);
    constexpr int kPos = kAxes ? kRopeMaxAxes : 1;
    int pos_next[kPos];
    pos_next[0] = -1;
    const View &xv = a.x[t], &zv = a.z[t], &ov = kBwd ? a.dx[t] : a.z[t];
    const char *x_at = nullptr, *z_at = nullptr;  // its first row of this lane, head 0
    char *o_at = nullptr, *o_next = nullptr;
    auto enter_token = [&]() {
      if (b >= a.B) return;
      x_at = xv.p + b * xv.sb + s * xv.ss + sub * xv.sh;
      if constexpr (kBwd) z_at = zv.p + b * zv.sb + s * zv.ss + sub * zv.sh;
      o_next = ov.p + b * ov.sb + s * ov.ss + sub * ov.sh;
      if constexpr (kAxes) {
#pragma unroll
        for (int x = 0; x < kPos; ++x)
          pos_next[x] = x < a.axes ? a.pos[x * a.pos_axis + (size_t)b * a.S + s] : 0;
      } else {
        pos_next[0] = !a.table ? 0 : a.pos ? a.pos[(size_t)b * a.S + s] : s;
      }
    };
    auto head_of = [&](int item) { return (item * spread + apart) * a.per_item; };
    // heads of an item (the same for the whole warp)
    auto heads_of = [&](int item) { return min(a.H[t] - head_of(item), a.per_item); };
    const long long x_step = SUBS * xv.sh, z_step = SUBS * zv.sh, o_step = SUBS * ov.sh;
    auto fetch = [&](int buf) {
      if (b < a.B) {
        const int heads = heads_of(it) - sub;
        const char* x = x_at + head_of(it) * xv.sh;
        const char* z = kBwd ? z_at + head_of(it) * zv.sh : nullptr;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          if (r * SUBS < heads) {
            if ((!kBwd || norm) && MATTN_IN_BOUNDS(kSiteRope, x + c1 + 15 - xv.p, xv.bytes)) {
              cp_async16(&place(buf, r, 0), x + c0);
              cp_async16(&place(buf, r, 1), x + c1);
            }
            if (kBwd && MATTN_IN_BOUNDS(kSiteRope, z + c1 + 15 - zv.p, zv.bytes)) {
              cp_async16(&place(buf, r, 2), z + c0);
              cp_async16(&place(buf, r, 3), z + c1);
            }
          }
          x += x_step;
          if constexpr (kBwd) z += z_step;
        }
      }
      cp_async_commit();
    };

    Rotation<N, kInter> rot;
    bool live = false;
    enter_token();
    if (count > 0) fetch(0);
    for (int i = 0; i < count; ++i) {
      const int item = it;
      int pos[kPos];
#pragma unroll
      for (int x = 0; x < kPos; ++x) pos[x] = pos_next[x];
      const bool there = b < a.B;
      o_at = o_next;
      if (++it == per_group) {
        it = 0;
        for (s += a.together; s >= a.S; s -= a.S) ++b;
        enter_token();
      }
      if (i + 1 < count) fetch((i + 1) & 1);
      if (item == 0 || i == 0) {  // another token
        live = there && (!a.table || (pos[0] >= 0 && pos[0] < a.max_pos));
#pragma unroll
        for (int x = 1; x < kPos; ++x) live = live && pos[x] >= 0 && pos[x] < a.max_pos;
        if (live) {
          if constexpr (kAxes) rot.load_axes(a, pos, ch);
          else rot.load(a, pos[0], ch);
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < P; ++j) {
              if constexpr (kBwd) {  // the transpose
                rot.e[k][j] = fmul2(rot.e[k][j], both(-1.0f));
              } else if (norm) {  // z = r (x (w c) + x' (w' e))
                const float2 own = weight(k, j);
                rot.c[k][j] = fmul2(rot.c[k][j], own);
                rot.e[k][j] = fmul2(rot.e[k][j], kInter ? make_float2(own.y, own.x) : weight(1 - k, j));
              }
            }
        }
      }
      if (i + 1 < count) cp_async_wait<1>();
      else cp_async_wait<0>();
      const int heads = live ? heads_of(item) : 0;
      char* out = o_at + head_of(item) * ov.sh;
#pragma unroll
      for (int r = 0; r < kRows; ++r, out += o_step) {
        if (r * SUBS >= heads) break;
        const bool here = r * SUBS + sub < heads;
        float2 x[2][P], y[2][P];
        float ri = 1.0f;
        if (!kBwd || norm) {
          unpack<kBf16>(place(i & 1, r, 0), x[0]);
          unpack<kBf16>(place(i & 1, r, 1), x[1]);
          if (norm) {
            float2 q = fmul2(x[0][0], x[0][0]), q1 = fmul2(x[1][0], x[1][0]);
#pragma unroll
            for (int j = 1; j < P; ++j) {
              q = ffma2(x[0][j], x[0][j], q);
              q1 = ffma2(x[1][j], x[1][j], q1);
            }
            q = fadd2(q, q1);
            ri = rsqrtf(row_sum<LANES>(q.x + q.y) * (1.0f / D) + a.eps);
          }
        }
        if constexpr (!kBwd) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < P; ++j) y[k][j] = fmul2(both(ri), rot.turn(a, ch, x, k, j));
        } else {
          float2 g[2][P];
          unpack<kBf16>(place(i & 1, r, 2), g[0]);
          unpack<kBf16>(place(i & 1, r, 3), g[1]);
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < P; ++j) y[k][j] = rot.turn(a, ch, g, k, j);  // dy
          if (norm) {
            float2 q = both(0.0f);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int j = 0; j < P; ++j) {
                x[k][j] = fmul2(x[k][j], both(ri));  // n
                const float2 yn = fmul2(y[k][j], x[k][j]);
                if (here) dw[k][j] = fadd2(dw[k][j], yn);
                q = ffma2(yn, w[k][j], q);
              }
            const float2 m = both(row_sum<LANES>(q.x + q.y) * (-1.0f / D));
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int j = 0; j < P; ++j)
                y[k][j] = fmul2(both(ri), ffma2(x[k][j], m, fmul2(y[k][j], w[k][j])));
          }
        }
        if (here && MATTN_IN_BOUNDS(kSiteRope, out + c1 + 15 - ov.p, ov.bytes)) {
          *reinterpret_cast<uint4*>(out + c0) = pack<kBf16>(y[0]);
          *reinterpret_cast<uint4*>(out + c1) = pack<kBf16>(y[1]);
        }
      }
    }

    if constexpr (kBwd) {  // the block's weight gradient, always in the same order
      float* sh = reinterpret_cast<float*>(ring);  // [warps][D]
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float v = i & 1 ? dw[k][i / 2].y : dw[k][i / 2].x;
#pragma unroll
          for (int d = LANES; d < 32; d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
          if (sub == 0) sh[warp * D + ch[k] + i] = v;
        }
      __syncthreads();
      for (int c = threadIdx.x; c < D; c += kRopeThreads) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < kRopeWarps; ++k) v += sh[k * D + c];
        a.part[(size_t)blockIdx.x * 2 * D + t * D + c] = v;
      }
      __syncthreads();
    }
  }
}

// Sum of the blocks' partial weight gradients, in a fixed order: one block per
// 32 columns, 32 rows of threads each taking every 32nd partial.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* part, int n, int D, float* dwq,
                                                       float* dwk) {
  early_start();
  __shared__ float sh[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;  // of 2 D
  float v = 0.0f;
  for (int i = threadIdx.y; i < n; i += 32) v += part[(size_t)i * 2 * D + col];
  sh[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = row_sum<32>(sh[threadIdx.x][threadIdx.y]);
  if (threadIdx.x == 0) {
    const int c = blockIdx.x * 32 + threadIdx.y;
    float* out = c < D ? dwq : dwk;
    if (out) out[c % D] = v;
  }
}

template <int D, bool kBf16, bool kBwd, bool kAxes>
cudaError_t launch_typed(RopeArgs& a, bool inter, int B, float* const* dw, cudaStream_t stream) {
  constexpr int kSubs = 32 / (D / (2 * Chunk<kBf16>::N));
  a.B = B;
  const long long tokens = (long long)B * a.S;
  const int resident = kRopePerSm * sm_count();
  // 8 tokens per block, each warp through all heads of its own, so that a token's
  // rotation is loaded once; with fewer tokens than resident blocks (a decode step)
  // one per block, and one row per lane group and item, so that the heads spread over
  // the warps. 2000 tokens x 40 heads of 128 bf16 channels: 12 us against 24; the
  // gradient of 2400 tokens x 5 heads of 64: 17 against 28; 300 tokens: the same;
  // 32 tokens x 72 heads of 128: 25 against 24.
  const bool many = tokens >= resident;
  a.together = many ? kRopeWarps : 1;
  a.per_item = many ? kSubs * rope_rows<kBwd>() : kSubs;
  a.groups = (tokens + a.together - 1) / a.together;
  long long items = 0;
  for (int t = 0; t < 2; ++t) {
    a.items[t] = (a.H[t] + a.per_item - 1) / a.per_item;
    items += a.items[t];
  }
  const long long all = many ? a.groups * items : a.groups * ((items + kRopeWarps - 1) / kRopeWarps);
  const int blocks = (int)std::min<long long>(std::min(resident, kRopeMaxBlocks), all);
  constexpr int kSmem = 2 * rope_rows<kBwd>() * (kBwd ? 4 : 2) * kRopeThreads * (int)sizeof(uint4);
  static DeviceOnce ready[2];
  cudaError_t e = inter ? ready[1].allow_smem(norm_rope_kernel<D, kBf16, true, kBwd, kAxes>, kSmem)
                        : ready[0].allow_smem(norm_rope_kernel<D, kBf16, false, kBwd, kAxes>, kSmem);
  if (e != cudaSuccess) return e;
  e = inter ? launch_early(norm_rope_kernel<D, kBf16, true, kBwd, kAxes>, blocks, kRopeThreads, kSmem, stream, a)
            : launch_early(norm_rope_kernel<D, kBf16, false, kBwd, kAxes>, blocks, kRopeThreads, kSmem, stream, a);
  if (e != cudaSuccess || !kBwd || (!dw[0] && !dw[1])) return e;
  return launch_early(rope_dw_kernel, 2 * D / 32, dim3(32, 32), 0, stream, a.part, blocks, D, dw[0], dw[1]);
}

template <bool kBwd, bool kAxes = false>
cudaError_t launch_rope(RopeArgs& a, const attn_rope_params* p, int B, int D, float* const* dw,
                        cudaStream_t s) {
  const bool inter = p->interleaved != 0;
  if (p->dtype == ATTN_BF16)
    return D == 64 ? launch_typed<64, true, kBwd, kAxes>(a, inter, B, dw, s)
                   : launch_typed<128, true, kBwd, kAxes>(a, inter, B, dw, s);
  return D == 64 ? launch_typed<64, false, kBwd, kAxes>(a, inter, B, dw, s)
                 : launch_typed<128, false, kBwd, kAxes>(a, inter, B, dw, s);
}

// Checks one tensor and turns its strides into bytes. An output's rows have to be
// distinct places (no stride of 0); `from` is the input that it may be itself.
attn_status take_view(View& v, const attn_view* t, int B, int H, int S, int D, int elem,
                      bool output = false, const View* from = nullptr) {
  if (!t || !t->data) return ATTN_ERR_INVALID_ARG;
  if (t->stride_b < 0 || t->stride_h < 0 || t->stride_s < 0) return ATTN_ERR_INVALID_ARG;
  const long long unit = 16 / elem;
  if ((reinterpret_cast<uintptr_t>(t->data) & 15u) || (B > 1 && t->stride_b % unit) ||
      (H > 1 && t->stride_h % unit) || (S > 1 && t->stride_s % unit))
    return ATTN_ERR_MISALIGNED;
  v.p = static_cast<char*>(t->data);
  v.sb = B > 1 ? t->stride_b * elem : 0;
  v.sh = H > 1 ? t->stride_h * elem : 0;
  v.ss = S > 1 ? t->stride_s * elem : 0;
  v.bytes = (B - 1) * v.sb + (H - 1) * v.sh + (S - 1) * v.ss + (long long)D * elem;
  if (output && ((B > 1 && !v.sb) || (H > 1 && !v.sh) || (S > 1 && !v.ss))) return ATTN_ERR_INVALID_ARG;
  if (from && from->p == v.p && (from->sb != v.sb || from->sh != v.sh || from->ss != v.ss))
    return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

// Every check that the forward and its gradient share; fills `a`.
attn_status rope_args(RopeArgs& a, const attn_rope_params* p, int B, int Hq, int Hkv, int S, int D) {
  if (!p || B < 0 || Hq < 0 || Hkv < 0 || S < 0) return ATTN_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
  if (p->dtype != ATTN_BF16 && p->dtype != ATTN_F32) return ATTN_ERR_UNSUPPORTED;
  if (!std::isfinite(p->eps) || p->eps < 0.0f) return ATTN_ERR_INVALID_ARG;
  if (p->cos_sin) {
    if (p->rot_dim < 16 || p->rot_dim > D || p->rot_dim % 16) return ATTN_ERR_UNSUPPORTED;
    if (p->max_pos < 1 || (!p->positions && S > p->max_pos)) return ATTN_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(p->cos_sin) & 15u) return ATTN_ERR_MISALIGNED;
  }
  const void* words[] = {p->q_weight, p->k_weight, p->positions};
  for (const void* x : words)
    if (reinterpret_cast<uintptr_t>(x) & 3u) return ATTN_ERR_MISALIGNED;
  a.w[0] = p->q_weight;
  a.w[1] = p->k_weight;
  a.table = p->cos_sin;
  a.pos = p->positions;
  a.eps = p->eps;
  a.S = S;
  a.H[0] = Hq;
  a.H[1] = Hkv;
  a.rot = p->rot_dim;
  a.max_pos = p->max_pos;
  return ATTN_OK;
}

inline size_t rope_workspace(int D) { return sizeof(float) * 2 * D * kRopeMaxBlocks; }

// The axis of each channel pair, packed for the kernel.
inline attn_status take_axes(RopeArgs& a, const attn_rope_params* p, int axes,
                             const unsigned char* pair_axis, int B, int S) {
  if (axes < 1 || axes > kRopeMaxAxes || !pair_axis || !p->cos_sin || !p->positions)
    return ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < p->rot_dim / 2; ++i) {
    if (pair_axis[i] >= axes) return ATTN_ERR_INVALID_ARG;
    a.pair_axis[i >> 5] |= (unsigned long long)pair_axis[i] << (2 * (i & 31));
  }
  a.axes = axes;
  a.pos_axis = (long long)B * S;
  return ATTN_OK;
}

// The calls' bodies (axes and pair_axis: with kAxes only).
template <bool kAxes>
attn_status rope_forward(const attn_view* const (&in)[2], const attn_view* const (&out)[2], int B,
                         int Hq, int Hkv, int S, int D, const attn_rope_params* p, int axes,
                         const unsigned char* pair_axis, struct CUstream_st* stream) {
  RopeArgs a{};
  attn_status st = rope_args(a, p, B, Hq, Hkv, S, D);
  if (kAxes && st == ATTN_OK) st = take_axes(a, p, axes, pair_axis, B, S);
  if (st != ATTN_OK || B == 0 || S == 0 || Hq + Hkv == 0) return st;
  const int elem = p->dtype == ATTN_F32 ? 4 : 2;
  for (int t = 0; t < 2; ++t) {
    if (a.H[t] == 0) continue;
    if ((st = take_view(a.x[t], in[t], B, a.H[t], S, D, elem)) != ATTN_OK) return st;
    if ((st = take_view(a.z[t], out[t], B, a.H[t], S, D, elem, true, &a.x[t])) != ATTN_OK) return st;
  }
  return cuda_status(launch_rope<false, kAxes>(a, p, B, D, nullptr,
                                               reinterpret_cast<cudaStream_t>(stream)));
}

template <bool kAxes>
attn_status rope_backward(const attn_view* const (&in)[2], const attn_view* const (&dz)[2],
                          const attn_view* const (&dx)[2], float* dq_weight, float* dk_weight,
                          void* workspace, size_t workspace_bytes, int B, int Hq, int Hkv, int S,
                          int D, const attn_rope_params* p, int axes,
                          const unsigned char* pair_axis, struct CUstream_st* stream) {
  RopeArgs a{};
  attn_status st = rope_args(a, p, B, Hq, Hkv, S, D);
  if (kAxes && st == ATTN_OK) st = take_axes(a, p, axes, pair_axis, B, S);
  if (st != ATTN_OK) return st;
  if ((dq_weight && !p->q_weight) || (dk_weight && !p->k_weight)) return ATTN_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(dq_weight) & 3u) || (reinterpret_cast<uintptr_t>(dk_weight) & 3u))
    return ATTN_ERR_MISALIGNED;
  const int elem = p->dtype == ATTN_F32 ? 4 : 2;
  if (B > 0 && S > 0) {
    for (int t = 0; t < 2; ++t) {
      if (a.H[t] == 0) continue;
      if (a.w[t] && (st = take_view(a.x[t], in[t], B, a.H[t], S, D, elem)) != ATTN_OK) return st;
      if ((st = take_view(a.z[t], dz[t], B, a.H[t], S, D, elem)) != ATTN_OK) return st;
      if ((st = take_view(a.dx[t], dx[t], B, a.H[t], S, D, elem, true, &a.z[t])) != ATTN_OK) return st;
    }
  }
  if (!workspace) return ATTN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return ATTN_ERR_MISALIGNED;
  if (workspace_bytes < rope_workspace(D)) return ATTN_ERR_WORKSPACE_TOO_SMALL;
  a.part = static_cast<float*>(workspace);
  float* dw[] = {dq_weight, dk_weight};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (B == 0 || S == 0 || Hq + Hkv == 0) {  // no rows: the weights' gradients are 0
    for (float* g : dw)
      if (g && (st = cuda_status(cudaMemsetAsync(g, 0, sizeof(float) * D, s))) != ATTN_OK) return st;
    return ATTN_OK;
  }
  return cuda_status(launch_rope<true, kAxes>(a, p, B, D, dw, s));
}

}  // namespace
}  // namespace mattn
