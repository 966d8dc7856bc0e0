// Norm and rotation of queries and keys with one position per token (kernels:
// norm_rope_kernel.cuh).
#include "norm_rope_kernel.cuh"

#define MATTN_API extern "C" __attribute__((visibility("default")))

MATTN_API attn_status attn_qk_norm_rope(const attn_view* q, const attn_view* k,
                                        const attn_view* q_out, const attn_view* k_out, int B,
                                        int Hq, int Hkv, int S, int D, const attn_rope_params* p,
                                        struct CUstream_st* stream) {
  return mattn::rope_forward<false>({q, k}, {q_out, k_out}, B, Hq, Hkv, S, D, p, 0, nullptr,
                                    stream);
}

MATTN_API size_t attn_qk_norm_rope_bwd_workspace_bytes(int D) {
  return D == 64 || D == 128 ? mattn::rope_workspace(D) : 0;
}

MATTN_API attn_status attn_qk_norm_rope_bwd(const attn_view* q, const attn_view* k,
                                            const attn_view* dq_out, const attn_view* dk_out,
                                            const attn_view* dq, const attn_view* dk,
                                            float* dq_weight, float* dk_weight, void* workspace,
                                            size_t workspace_bytes, int B, int Hq, int Hkv, int S,
                                            int D, const attn_rope_params* p,
                                            struct CUstream_st* stream) {
  return mattn::rope_backward<false>({q, k}, {dq_out, dk_out}, {dq, dk}, dq_weight, dk_weight,
                                     workspace, workspace_bytes, B, Hq, Hkv, S, D, p, 0, nullptr,
                                     stream);
}

namespace mattn {
MATTN_DEBUG_RECORD_ACCESSORS(norm_rope)
}  // namespace mattn
