// Per-head RMS norm of queries and keys with the position rotation, in one
// pass from the projection's layout to the attention's (any strides), and its
// gradient. A row is one head of one token, D channels:
//
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r,  y = n w,  z = R(pos) y
//   z[c] = y[c] cos - y[c'] sin,  z[c'] = y[c'] cos + y[c] sin
// for the channel pairs (c, c') of the rotation; channels past rot_dim pass.
//
// Gradient, from the row's x (r and n are computed again) and dz:
//   dy = R(pos)^T dz,  dw = sum over rows of dy n,  dn = dy w,
//   dx = r (dn - n mean(dn n))
//
// Bound by HBM: a row is read and written once (forward), or read twice and
// written once (gradient). A lane holds 16 bytes of a row, so a row takes 8
// to 32 lanes and the row sums are a few shuffles; the rotation's partner
// channels are in a lane rot_dim/2 away (shuffle) or, interleaved, in the same
// lane. A warp takes a unit of up to kRows rows per lane group from one token,
// with all their loads in flight at once, and keeps the token's cos and sin in
// registers from unit to unit. All arithmetic is fp32; each output is rounded
// once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "host_util.h"
#include "launch.h"

#define MATTN_API extern "C" __attribute__((visibility("default")))

namespace mattn {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRows = 4;           // rows in flight per lane group
constexpr int kRopeBwdBlocks = 608;  // most blocks of the gradient (4 per SM of 152): the
                                     // workspace holds one partial weight gradient each

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
  int blocks_q, blocks_all;  // head blocks of q, and of q and k together, per token
  int per_block;             // heads per block
  long long units;           // tokens * blocks_all
};

template <bool kBf16>
struct Chunk {  // 16 bytes of a row
  static constexpr int N = kBf16 ? 8 : 4;
};

template <bool kBf16>
__device__ __forceinline__ void unpack(const uint4& v, float* f) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kBf16) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    } else {
      f[i] = __uint_as_float(u[i]);
    }
  }
}

template <bool kBf16>
__device__ __forceinline__ uint4 pack(const float* f) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kBf16) u[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    else u[i] = __float_as_uint(f[i]);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// A token's rotation as the lane's channels see it: z = c y + e y', y' the
// partner channel (e = -sin for the first of a pair, +sin for the second).
// The transpose is the same with e negated. Interleaved: c and e of pair i.
template <int N, bool kInter>
struct Rotation {
  static constexpr int M = kInter ? N / 2 : N;
  float c[M], e[M];
  int mate;  // partner lane

  __device__ __forceinline__ void load(const RopeArgs& a, int pos, int chunk, int lane) {
    const int ch = chunk * N, half = a.rot / 2;
    mate = lane;
    if (!a.table || ch >= a.rot) {
#pragma unroll
      for (int i = 0; i < M; ++i) {
        c[i] = 1.0f;
        e[i] = 0.0f;
      }
      return;
    }
    const float* row = a.table + (size_t)pos * a.rot;
    if constexpr (kInter) {
#pragma unroll
      for (int i = 0; i < M; ++i) {
        c[i] = row[ch / 2 + i];
        e[i] = row[half + ch / 2 + i];
      }
    } else {
      const bool second = ch >= half;
      const int at = second ? ch - half : ch;
      mate = second ? lane - half / N : lane + half / N;
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const float4 cv = *reinterpret_cast<const float4*>(row + at + i);
        const float4 sv = *reinterpret_cast<const float4*>(row + half + at + i);
        const float cs[4] = {cv.x, cv.y, cv.z, cv.w}, sn[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          c[i + j] = cs[j];
          e[i + j] = second ? sn[j] : -sn[j];
        }
      }
    }
  }

  // sign 1: rotate, -1: the transpose
  __device__ __forceinline__ void apply(float* y, float sign) const {
    if constexpr (kInter) {
#pragma unroll
      for (int i = 0; i < M; ++i) {
        const float s = sign * e[i], a = y[2 * i], b = y[2 * i + 1];
        y[2 * i] = a * c[i] - b * s;
        y[2 * i + 1] = b * c[i] + a * s;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float o = __shfl_sync(0xffffffffu, y[i], mate);
        y[i] = y[i] * c[i] + (sign * e[i]) * o;
      }
    }
  }
};

template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int d = 1; d < LANES; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

template <int D, bool kBf16, bool kInter, bool kBwd>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const RopeArgs a) {
  constexpr int N = Chunk<kBf16>::N;
  constexpr int LANES = D / N;        // lanes per row
  constexpr int SUBS = 32 / LANES;    // rows side by side in a warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunk = lane % LANES, sub = lane / LANES;

  float w[2][N], dw[2][N];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      w[t][i] = a.w[t] ? a.w[t][chunk * N + i] : 1.0f;
      dw[t][i] = 0.0f;
    }

  // a warp's run of consecutive units: the same token again and again
  const long long nw = (long long)gridDim.x * kRopeWarps;
  const long long wid = (long long)blockIdx.x * kRopeWarps + warp;
  long long u = a.units * wid / nw;
  const long long u_end = a.units * (wid + 1) / nw;
  long long token = u / a.blocks_all;
  int blk = (int)(u - token * a.blocks_all);
  int b = (int)(token / a.S), s = (int)(token - (long long)b * a.S);
  Rotation<N, kInter> rot;
  bool live = false, fresh = true;

  for (; u < u_end; ++u) {
    if (fresh) {
      const int pos = !a.table ? 0 : a.pos ? a.pos[(size_t)b * a.S + s] : s;
      live = !a.table || (pos >= 0 && pos < a.max_pos);
      if (live) rot.load(a, pos, chunk, lane);
      fresh = false;
    }
    if (live) {
      auto rows = [&](const int t, float (&wt)[N], float (&dwt)[N], int h_begin) {
        const View& xv = a.x[t];
        const View& zv = a.z[t];
        const bool norm = a.w[t] != nullptr;
        const int h_end = min(a.H[t], h_begin + a.per_block);
        const char* xp = xv.p + b * xv.sb + s * xv.ss + chunk * 16;
        char* zp = zv.p + b * zv.sb + s * zv.ss + chunk * 16;
        char* dp = kBwd ? a.dx[t].p + b * a.dx[t].sb + s * a.dx[t].ss + chunk * 16 : nullptr;
        for (int h0 = h_begin; h0 < h_end; h0 += SUBS * kRows) {
          uint4 xr[kRows], gr[kRows];
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            const int h = h0 + r * SUBS + sub;
            xr[r] = gr[r] = make_uint4(0, 0, 0, 0);
            if (h < h_end) {
              const long long at = h * xv.sh;
              if ((!kBwd || norm) && MATTN_IN_BOUNDS(kSiteRope, xp + at - xv.p, xv.bytes))
                xr[r] = *reinterpret_cast<const uint4*>(xp + at);
              if (kBwd && MATTN_IN_BOUNDS(kSiteRope, zp + h * zv.sh - zv.p, zv.bytes))
                gr[r] = *reinterpret_cast<const uint4*>(zp + h * zv.sh);
            }
          }
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            if (h0 + r * SUBS >= h_end) break;  // the whole warp is past the last head
            const int h = h0 + r * SUBS + sub;
            float x[N], y[N];
            unpack<kBf16>(xr[r], x);
            float ri = 1.0f;
            if (norm) {
              float ss = 0.0f;
#pragma unroll
              for (int i = 0; i < N; ++i) ss += x[i] * x[i];
              ri = rsqrtf(row_sum<LANES>(ss) * (1.0f / D) + a.eps);
              if (h >= h_end) ri = 0.0f;  // no row: adds nothing, eps = 0 included
            }
            if constexpr (!kBwd) {
#pragma unroll
              for (int i = 0; i < N; ++i) y[i] = x[i] * ri * wt[i];
              rot.apply(y, 1.0f);
              if (h < h_end && MATTN_IN_BOUNDS(kSiteRope, zp + h * zv.sh - zv.p, zv.bytes))
                *reinterpret_cast<uint4*>(zp + h * zv.sh) = pack<kBf16>(y);
            } else {
              unpack<kBf16>(gr[r], y);
              rot.apply(y, -1.0f);  // dy
              if (norm) {
                float dot = 0.0f;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                  x[i] *= ri;                    // n
                  dwt[i] += y[i] * x[i];
                  y[i] *= wt[i];                 // dn
                  dot += y[i] * x[i];
                }
                dot = row_sum<LANES>(dot) * (1.0f / D);
#pragma unroll
                for (int i = 0; i < N; ++i) y[i] = ri * (y[i] - x[i] * dot);
              }
              if (h < h_end &&
                  MATTN_IN_BOUNDS(kSiteRope, dp + h * a.dx[t].sh - a.dx[t].p, a.dx[t].bytes))
                *reinterpret_cast<uint4*>(dp + h * a.dx[t].sh) = pack<kBf16>(y);
            }
          }
        }
      };
      if (blk < a.blocks_q) rows(0, w[0], dw[0], blk * a.per_block);
      else rows(1, w[1], dw[1], (blk - a.blocks_q) * a.per_block);
    }
    if (++blk == a.blocks_all) {
      blk = 0;
      fresh = true;
      if (++s == a.S) {
        s = 0;
        ++b;
      }
    }
  }

  if constexpr (kBwd) {  // the block's weight gradients, always in the same order
    __shared__ float sh[kRopeWarps][2][D];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float v = dw[t][i];
#pragma unroll
        for (int d = LANES; d < 32; d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        if (sub == 0) sh[warp][t][chunk * N + i] = v;
      }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * D; c += kRopeThreads) {
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < kRopeWarps; ++k) v += sh[k][c / D][c % D];
      a.part[(size_t)blockIdx.x * 2 * D + c] = v;
    }
  }
}

// Sum of the blocks' partial weight gradients, in a fixed order: one block per
// 32 columns, 32 rows of threads each taking every 32nd partial.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* part, int n, int D, float* dwq,
                                                       float* dwk) {
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

template <int D, bool kBf16, bool kBwd>
cudaError_t launch_typed(RopeArgs& a, bool inter, int B, float* const* dw, cudaStream_t stream) {
  constexpr int kSubs = 32 / (D / Chunk<kBf16>::N);
  const long long tokens = (long long)B * a.S;
  const int blocks_max = kBwd ? std::min(kRopeBwdBlocks, 4 * sm_count()) : 4 * sm_count();
  // Heads per unit: as many as a warp has in flight, but fewer where the
  // tokens alone do not give every warp of the grid one unit (a decode step's
  // few tokens: one row per lane group and unit, so the rows spread over the SMs).
  a.per_block = kSubs * kRows;
  auto count = [&](int per) {
    a.per_block = per;
    a.blocks_q = (a.H[0] + per - 1) / per;
    a.blocks_all = a.blocks_q + (a.H[1] + per - 1) / per;
    a.units = tokens * a.blocks_all;
  };
  for (int per = kSubs * kRows; per >= kSubs; per >>= 1) {
    count(per);
    if (a.units >= (long long)blocks_max * kRopeWarps) break;
  }
  const int blocks = (int)std::min<long long>(blocks_max, (a.units + kRopeWarps - 1) / kRopeWarps);
  if (inter) norm_rope_kernel<D, kBf16, true, kBwd><<<blocks, kRopeThreads, 0, stream>>>(a);
  else norm_rope_kernel<D, kBf16, false, kBwd><<<blocks, kRopeThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !kBwd || (!dw[0] && !dw[1])) return e;
  rope_dw_kernel<<<2 * D / 32, dim3(32, 32), 0, stream>>>(a.part, blocks, D, dw[0], dw[1]);
  return cudaGetLastError();
}

template <bool kBwd>
cudaError_t launch_rope(RopeArgs& a, const attn_rope_params* p, int B, int D, float* const* dw,
                        cudaStream_t s) {
  const bool inter = p->interleaved != 0;
  if (p->dtype == ATTN_BF16)
    return D == 64 ? launch_typed<64, true, kBwd>(a, inter, B, dw, s)
                   : launch_typed<128, true, kBwd>(a, inter, B, dw, s);
  return D == 64 ? launch_typed<64, false, kBwd>(a, inter, B, dw, s)
                 : launch_typed<128, false, kBwd>(a, inter, B, dw, s);
}

// Checks one tensor and turns its strides into bytes.
attn_status take_view(View& v, const attn_view* t, int B, int H, int S, int D, int elem) {
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

}  // namespace
}  // namespace mattn

MATTN_API attn_status attn_qk_norm_rope(const attn_view* q, const attn_view* k,
                                        const attn_view* q_out, const attn_view* k_out, int B,
                                        int Hq, int Hkv, int S, int D, const attn_rope_params* p,
                                        struct CUstream_st* stream) {
  using namespace mattn;
  RopeArgs a{};
  attn_status st = rope_args(a, p, B, Hq, Hkv, S, D);
  if (st != ATTN_OK || B == 0 || S == 0 || Hq + Hkv == 0) return st;
  const int elem = p->dtype == ATTN_F32 ? 4 : 2;
  const attn_view* in[] = {q, k};
  const attn_view* out[] = {q_out, k_out};
  for (int t = 0; t < 2; ++t) {
    if (a.H[t] == 0) continue;
    if ((st = take_view(a.x[t], in[t], B, a.H[t], S, D, elem)) != ATTN_OK) return st;
    if ((st = take_view(a.z[t], out[t], B, a.H[t], S, D, elem)) != ATTN_OK) return st;
  }
  return cuda_status(launch_rope<false>(a, p, B, D, nullptr, reinterpret_cast<cudaStream_t>(stream)));
}

MATTN_API size_t attn_qk_norm_rope_bwd_workspace_bytes(int D) {
  return D == 64 || D == 128 ? sizeof(float) * 2 * D * mattn::kRopeBwdBlocks : 0;
}

MATTN_API attn_status attn_qk_norm_rope_bwd(const attn_view* q, const attn_view* k,
                                            const attn_view* dq_out, const attn_view* dk_out,
                                            const attn_view* dq, const attn_view* dk,
                                            float* dq_weight, float* dk_weight, void* workspace,
                                            size_t workspace_bytes, int B, int Hq, int Hkv, int S,
                                            int D, const attn_rope_params* p,
                                            struct CUstream_st* stream) {
  using namespace mattn;
  RopeArgs a{};
  attn_status st = rope_args(a, p, B, Hq, Hkv, S, D);
  if (st != ATTN_OK) return st;
  if ((dq_weight && !p->q_weight) || (dk_weight && !p->k_weight)) return ATTN_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(dq_weight) & 3u) || (reinterpret_cast<uintptr_t>(dk_weight) & 3u))
    return ATTN_ERR_MISALIGNED;
  const int elem = p->dtype == ATTN_F32 ? 4 : 2;
  const attn_view* in[] = {q, k};
  const attn_view* dz[] = {dq_out, dk_out};
  const attn_view* dx[] = {dq, dk};
  if (B > 0 && S > 0) {
    for (int t = 0; t < 2; ++t) {
      if (a.H[t] == 0) continue;
      if (a.w[t] && (st = take_view(a.x[t], in[t], B, a.H[t], S, D, elem)) != ATTN_OK) return st;
      if ((st = take_view(a.z[t], dz[t], B, a.H[t], S, D, elem)) != ATTN_OK) return st;
      if ((st = take_view(a.dx[t], dx[t], B, a.H[t], S, D, elem)) != ATTN_OK) return st;
    }
  }
  if (!workspace) return ATTN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return ATTN_ERR_MISALIGNED;
  if (workspace_bytes < attn_qk_norm_rope_bwd_workspace_bytes(D)) return ATTN_ERR_WORKSPACE_TOO_SMALL;
  a.part = static_cast<float*>(workspace);
  float* dw[] = {dq_weight, dk_weight};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (B == 0 || S == 0 || Hq + Hkv == 0) {  // no rows: the weights' gradients are 0
    for (float* g : dw)
      if (g && (st = cuda_status(cudaMemsetAsync(g, 0, sizeof(float) * D, s))) != ATTN_OK) return st;
    return ATTN_OK;
  }
  return cuda_status(launch_rope<true>(a, p, B, D, dw, s));
}

namespace mattn {
MATTN_DEBUG_RECORD_ACCESSORS(norm_rope)
}  // namespace mattn
