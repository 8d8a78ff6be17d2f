// feed_forward.cuh -- what the kernels of the feed-forward products share: the epilogue's arguments, and how operands
// are mapped.
#pragma once

#include "common.cuh"
#include "kernels.h"
#include "linear.cuh"

namespace molora {

// What the epilogue reads and writes.
struct FEpi {
  const float* sx;   // [N x K blocks]
  const float* sw;   // [blocks of W's rows x K blocks]
  const float* bias;
  const void* res;   // slopes: dh
  void* y;           // slopes: dproj
  int64_t N;
  int32_t d_out;     // outputs; gated: d_ff
  int32_t up;        // gated: Wu's first block of rows in sw
  molora_activation act;
  bool y_bf16;
  bool tma_y;        // rows of y on 16-byte boundaries
  bool tma_res;      // the residual comes through the staging boxes (slopes: dh does)
};

inline FEpi ff_epilogue_of(const FeedForwardArgs& a) {
  FEpi e = {a.x_scale, a.w_scale, a.bias, a.residual, a.y, a.N, a.d_out, (a.d_out + 127) / 128, a.act, a.y_bf16, false, false};
  e.tma_y = a.d_out % (a.y_bf16 ? 8 : 4) == 0 && aligned(a.y, 16) && aligned(a.residual, 16);
  return e;
}

inline int64_t ff_rows_of_w(const FeedForwardArgs& a) { return (int64_t)a.d_out * (a.gated ? 2 : 1); }

// K blocks of 128 bytes.
inline int ff_k_blocks(const FeedForwardArgs& a) {
  return (int)(((int64_t)a.d_in * (a.dtype == MOLORA_E4M3 ? 1 : 2) + kRowBytes - 1) / kRowBytes);
}

inline bool ff_operand_map(CUtensorMap* m, const FeedForwardArgs& a, const void* base, int64_t rows, uint32_t box_rows) {
  const bool fp8 = a.dtype == MOLORA_E4M3;
  return linear_map(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, fp8 ? 1 : 2, base,
                    (uint64_t)rows, (uint64_t)a.d_in, fp8 ? 128 : 64, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

// blocks_tc.cu: e4m3, many tokens, in tiles of BN rows of W (256, 192 or 128).
cudaError_t launch_blocks_tc(const FeedForwardArgs& a, int BN, cudaStream_t stream);

}  // namespace molora
