// The costs by which molora_linear_blocks and molora_gated_linear choose their kernel and its tiles, for given sizes on
// GB300's 152 SMs: no GPU is asked.
#include "feed_forward.cu"

namespace {

const molora::Resident kResident = {{0, 152, 76, 50, 36, 28, 23, 19, 15}};

molora::FeedForwardArgs args_of(int gated, int fp8, int64_t N, int32_t d_in, int32_t d_out) {
  molora::FeedForwardArgs a = {};
  a.gated = gated, a.dtype = fp8 ? MOLORA_E4M3 : MOLORA_BF16, a.N = N, a.d_in = d_in, a.d_out = d_out, a.y_bf16 = true;
  return a;
}

}  // namespace

// In tiles of `tile` rows of W (the pairs' kernels), or of `tile` tokens (few tokens' kernel).
extern "C" MOLORA_API int64_t pairs_cost(int gated, int fp8, int64_t N, int32_t d_in, int32_t d_out, int tile) {
  return molora::tc_cycles(args_of(gated, fp8, N, d_in, d_out), kResident, tile);
}
extern "C" MOLORA_API int64_t few_cost(int gated, int fp8, int64_t N, int32_t d_in, int32_t d_out, int tile) {
  const molora::FeedForwardArgs a = args_of(gated, fp8, N, d_in, d_out);
  return molora::skinny_cycles(kResident, molora::ff_rows_of_w(a), N, molora::ff_k_blocks(a), fp8 != 0, tile);
}
