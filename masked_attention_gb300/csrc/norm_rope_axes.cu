// Norm and rotation of queries and keys with positions on several axes (time, height and width
// of images and video): channel pair i turns by the angle of its axis' position (kernels:
// norm_rope_kernel.cuh).
//
// Bound by HBM like the one-axis calls: a token's positions and its cosines and sines are read
// once for all of its heads, so picking them pair by pair costs little. 16384 tokens x 40 heads
// of 128 bf16 channels, three axes: 60.4 us, 0.84 of a plain copy's rate (one axis: 60); the
// gradient of 32768 x 32 heads, pairs dealt to three axes one by one: 142 us, 0.84.
#include "norm_rope_kernel.cuh"

#define MATTN_API extern "C" __attribute__((visibility("default")))

MATTN_API attn_status attn_qk_norm_rope_axes(const attn_view* q, const attn_view* k,
                                             const attn_view* q_out, const attn_view* k_out, int B,
                                             int Hq, int Hkv, int S, int D,
                                             const attn_rope_params* p, int axes,
                                             const unsigned char* pair_axis,
                                             struct CUstream_st* stream) {
  return mattn::rope_forward<true>({q, k}, {q_out, k_out}, B, Hq, Hkv, S, D, p, axes, pair_axis,
                                   stream);
}

MATTN_API attn_status attn_qk_norm_rope_axes_bwd(
    const attn_view* q, const attn_view* k, const attn_view* dq_out, const attn_view* dk_out,
    const attn_view* dq, const attn_view* dk, float* dq_weight, float* dk_weight, void* workspace,
    size_t workspace_bytes, int B, int Hq, int Hkv, int S, int D, const attn_rope_params* p,
    int axes, const unsigned char* pair_axis, struct CUstream_st* stream) {
  return mattn::rope_backward<true>({q, k}, {dq_out, dk_out}, {dq, dk}, dq_weight, dk_weight,
                                    workspace, workspace_bytes, B, Hq, Hkv, S, D, p, axes,
                                    pair_axis, stream);
}

namespace mattn {
MATTN_DEBUG_RECORD_ACCESSORS(norm_rope_axes)
}  // namespace mattn
