// The 4-bit cache's page record, shared by the kernels that write and read it.
//
// A (page, key/value head) owns one contiguous record:
//   K codes  [page][D/2]   bytes; byte b of a row holds channel 2b in its low
//                          nibble and 2b + 1 in its high one
//   V codes  [page][D/2]
//   K scales [page][D/32]  bf16, one per 32 consecutive channels
//   V scales [page][D/32]  bf16
// A code n stands for (n - 8) * scale. Every piece starts on a 16-byte
// boundary (page >= 16), and a token's 32 channels of one scale are 16 bytes.
#pragma once

#include <cstddef>
#include <cstdint>

namespace mattn {

constexpr int kQ4Group = 32;  // channels per scale

struct Q4Layout {
  int D, page;
  __host__ __device__ constexpr int code_row() const { return D / 2; }
  __host__ __device__ constexpr int scale_row() const { return D / kQ4Group * 2; }
  __host__ __device__ constexpr int v_codes() const { return page * code_row(); }
  __host__ __device__ constexpr int k_scales() const { return 2 * page * code_row(); }
  __host__ __device__ constexpr int v_scales() const { return k_scales() + page * scale_row(); }
  __host__ __device__ constexpr int bytes() const { return v_scales() + page * scale_row(); }
};

inline bool q4_page_ok(int page) {
  return page == 16 || page == 32 || page == 64 || page == 128;
}

}  // namespace mattn
