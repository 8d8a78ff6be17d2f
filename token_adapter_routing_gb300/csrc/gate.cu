// gate.cu -- expert-style gate over given logits: softmax or sigmoid scores, a bias that only
// moves the choice, groups of which the best are kept, the k best experts, renormalised weights.
//
// A token belongs to TL lanes of a warp; lane l of them holds experts l, l + TL, l + 2 TL, ...: every
// load is of consecutive logits, whatever K and the rows' alignment.
//
// Everything the choice depends on is reproducible: e = expf(l - max) and 1 / (1 + expf(-l)) are
// single fp32 operations, and the softmax's denominator is summed in two fp32 terms (error about
// 2^-46) and rounded once, so it does not depend on the order of the sum.
#include "common.cuh"
#include "kernels.h"

namespace molora {

namespace {

constexpr int kGateWarps = 8;
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kFloatMax = 3.4028234663852886e38f;

struct GateArgs {
  int64_t N;
  int32_t K;
  const float* bias;
  int32_t G, keep, group_top;
  uint32_t per_inverse;  // ceil(2^20 / (K / G)): a * per_inverse >> 20 is expert a's group
  int32_t k;
  bool sigmoid, renorm;
  float scale;
  int32_t* ids;
  float* w;
  int32_t* err_word;
};

// hi + lo += v, without losing v's low bits.  The _rn forms are never fused with the operation
// that made an operand, so every rounding here is the one written.
__device__ __forceinline__ void two_sum(float& hi, float& lo, float v) {
  const float s = __fadd_rn(hi, v), b = __fsub_rn(s, hi);
  lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(v, b)));
  hi = s;
}

// Order-preserving map of a float (not NaN) to an unsigned integer.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);  // -0 and +0 are equal
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// The scores s and choices c of this lane's experts, from their logits l (-inf past K) and biases.
template <int TL, int V>
__device__ __forceinline__ void gate_scores(const GateArgs& a, float (&l)[V], const float (&b)[V], float (&s)[V],
                                            float (&c)[V]) {
  const float inf = __int_as_float(0x7f800000);
  const bool by_logit = !a.bias && (a.G == 1 || a.group_top == 1);
  bool bad = false;
  float m = -inf;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    bad |= l[i] != l[i] || b[i] != b[i];
    l[i] = l[i] != l[i] ? -inf : fminf(l[i], kFloatMax);
    m = fmaxf(m, l[i]);
  }
  if (bad) report(a.err_word, MOLORA_DEV_BAD_LOGIT);
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = __frcp_rn(__fadd_rn(1.f, expf(-l[i])));
  } else {
#pragma unroll
    for (int off = TL / 2; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
    float hi = 0.f, lo = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[i] = l[i] == -inf ? 0.f : expf(l[i] - m);
      two_sum(hi, lo, s[i]);
    }
#pragma unroll
    for (int off = TL / 2; off; off >>= 1) {
      const float oh = __shfl_xor_sync(kFull, hi, off), ol = __shfl_xor_sync(kFull, lo, off);
      two_sum(hi, lo, oh);
      lo = __fadd_rn(lo, ol);
    }
    // the lanes may have added in different orders: the first one's sum, rounded once, is the token's
    const float total = __shfl_sync(kFull, __fadd_rn(hi, lo), 0, TL);
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = total > 0.f ? __fdiv_rn(s[i], total) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    c[i] = l[i] == -inf ? -inf : by_logit ? l[i] : __fadd_rn(s[i], b[i]);
    c[i] = c[i] > -inf ? fminf(c[i], kFloatMax) : -inf;
  }
}

// The k largest choices by k rounds of a maximum over the token's lanes, ties to the lower index;
// stores the token's ids and weights if `live`.
template <int TL, int V>
__device__ __forceinline__ void gate_rounds(const GateArgs& a, float (&c)[V], const float (&s)[V], int64_t t, bool live) {
  const float inf = __int_as_float(0x7f800000);
  const int sub = threadIdx.x & (TL - 1);
  int place[V];  // the round that took expert sub + TL * i
#pragma unroll
  for (int i = 0; i < V; ++i) place[i] = -1;
  int found = 0;
  float sum = 0.f;
  for (int j = 0; j < a.k; ++j) {
    float best = c[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = fmaxf(best, c[i]);
#pragma unroll
    for (int off = TL / 2; off; off >>= 1) best = fmaxf(best, __shfl_xor_sync(kFull, best, off));
    int at = INT32_MAX;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
      if (c[i] == best) at = sub + TL * i;
#pragma unroll
    for (int off = TL / 2; off; off >>= 1) at = min(at, __shfl_xor_sync(kFull, at, off));
    if (best > -inf) {
      ++found;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (at == sub + TL * i) c[i] = -inf, place[i] = j, sum += s[i];
    }
  }
#pragma unroll
  for (int off = TL / 2; off; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
  if (!live) return;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (place[i] >= 0) {
      const float w = !a.renorm ? s[i] : sum > 0.f ? s[i] / sum : 0.f;
      a.ids[t * a.k + place[i]] = sub + TL * i;
      a.w[t * a.k + place[i]] = w * a.scale;
    }
  for (int j = found + sub; j < a.k; j += TL) a.ids[t * a.k + j] = -1, a.w[t * a.k + j] = 0.f;
}

}  // namespace

// Up to 64 experts in one group: TL lanes a token, so that a warp's every instruction works for
// 32 / TL tokens and a maximum over the lanes takes log2(TL) steps.
template <typename T, int TL, int V>
__global__ void __launch_bounds__(kGateWarps * 32) gate_small_kernel(const T* __restrict__ logits, const GateArgs a) {
  constexpr int kTokens = 32 / TL;  // of a warp
  const int lane = threadIdx.x & 31, sub = lane & (TL - 1), warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_launch_dependents();
  float b[V];
#pragma unroll
  for (int i = 0; i < V; ++i) b[i] = a.bias && sub + TL * i < a.K ? a.bias[sub + TL * i] : 0.f;
  for (int64_t t0 = ((int64_t)blockIdx.x * kGateWarps + warp) * kTokens; t0 < a.N;
       t0 += (int64_t)gridDim.x * kGateWarps * kTokens) {
    const int64_t t = t0 + lane / TL;
    const bool live = t < a.N;
    float l[V], s[V], c[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
      l[i] = live && sub + TL * i < a.K ? to_float(logits[t * a.K + sub + TL * i]) : __int_as_float(0xff800000);
    gate_scores<TL, V>(a, l, b, s, c);
    gate_rounds<TL, V>(a, c, s, t, live);
  }
}

// More experts, or groups: a warp a token.  The k-th largest of the 32 lanes' own maxima is a bound
// that the k largest choices reach and few others do; those that do (k and a few) are ranked by
// counting, in shared memory, instead of k rounds over all of them.
template <typename T, int V>
__global__ void __launch_bounds__(kGateWarps * 32) gate_topk_kernel(const T* __restrict__ logits, const GateArgs a) {
  extern __shared__ float choices[];  // [warps][K], with groups
  __shared__ float2 cand[kGateWarps][32];  // (choice, expert) of those that reach the bound
  __shared__ float cand_s[kGateWarps][32];
  const float inf = __int_as_float(0x7f800000);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t below = (1u << lane) - 1u;
  pdl_wait();
  pdl_launch_dependents();
  float b[V];
#pragma unroll
  for (int i = 0; i < V; ++i) b[i] = a.bias && lane + 32 * i < a.K ? a.bias[lane + 32 * i] : 0.f;
  for (int64_t t = (int64_t)blockIdx.x * kGateWarps + warp; t < a.N; t += (int64_t)gridDim.x * kGateWarps) {
    float l[V], s[V], c[V];
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = lane + 32 * i < a.K ? to_float(logits[t * a.K + lane + 32 * i]) : -inf;
    gate_scores<32, V>(a, l, b, s, c);
    if (a.G > 1) {
      // each group's best, or best two, by 32 / G lanes rounded down to a power of two
      float* mine = choices + (size_t)warp * a.K;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane + 32 * i < a.K) mine[lane + 32 * i] = c[i];
      __syncwarp();
      const int per = a.K / a.G;
      int lanes = 1;
      while (lanes * 2 * a.G <= 32) lanes *= 2;
      const int g = lane / lanes;
      float c1 = -inf, c2 = -inf;
      if (g < a.G) {
        for (int i = lane & (lanes - 1); i < per; i += lanes) {
          const float v = mine[g * per + i];
          c2 = fmaxf(c2, fminf(c1, v));
          c1 = fmaxf(c1, v);
        }
      }
      for (int off = 1; off < lanes; off <<= 1) {
        const float o1 = __shfl_xor_sync(kFull, c1, off), o2 = __shfl_xor_sync(kFull, c2, off);
        c2 = fmaxf(fminf(c1, o1), fmaxf(c2, o2));
        c1 = fmaxf(c1, o1);
      }
      const float rank = a.group_top == 1 ? c1 : __fadd_rn(c1, c2);
      uint32_t kept = 0;  // bit g: group g stays
      uint32_t key = g < a.G && (lane & (lanes - 1)) == 0 ? ordered(rank) : 0u;
      for (int j = 0; j < a.keep; ++j) {
        const uint32_t best = __reduce_max_sync(kFull, key);
        const int win = __ffs(__ballot_sync(kFull, key == best)) - 1;
        kept |= 1u << (win / lanes);
        if (lane == win) key = 0u;
      }
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (!((kept >> (((lane + 32 * i) * a.per_inverse) >> 20 & 31u)) & 1u)) c[i] = -inf;
      __syncwarp();
    }
    float most = c[0];
#pragma unroll
    for (int i = 1; i < V; ++i) most = fmaxf(most, c[i]);
    uint32_t key = ordered(most), bound = 0;
    for (int j = 0; j < a.k; ++j) {
      bound = __reduce_max_sync(kFull, key);
      const uint32_t same = __ballot_sync(kFull, key == bound);
      if (lane == __ffs(same) - 1) key = 0u;
    }
    int n = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool in = c[i] > -inf && ordered(c[i]) >= bound;
      const uint32_t who = __ballot_sync(kFull, in);
      const int at = n + __popc(who & below);
      if (in && at < 32) {
        cand[warp][at] = make_float2(c[i], __int_as_float(lane + 32 * i));
        cand_s[warp][at] = s[i];
      }
      n += __popc(who);
    }
    if (n > 32) {  // many equal choices
      gate_rounds<32, V>(a, c, s, t, true);
      continue;
    }
    __syncwarp();
    const float2 mine = cand[warp][lane < n ? lane : 0];
    const float score = cand_s[warp][lane < n ? lane : 0];
    int rank = 0;
    for (int i = 0; i < n; ++i) {
      const float2 o = cand[warp][i];
      rank += o.x > mine.x || (o.x == mine.x && __float_as_int(o.y) < __float_as_int(mine.y));
    }
    const bool chosen = lane < n && rank < a.k;
    float sum = chosen ? score : 0.f;
#pragma unroll
    for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
    if (chosen) {
      const float w = !a.renorm ? score : sum > 0.f ? score / sum : 0.f;
      a.ids[t * a.k + rank] = __float_as_int(mine.y);
      a.w[t * a.k + rank] = w * a.scale;
    }
    if (lane >= n && lane < a.k) a.ids[t * a.k + lane] = -1, a.w[t * a.k + lane] = 0.f;
    __syncwarp();
  }
}

namespace {

template <typename T>
cudaError_t launch_gate_typed(const T* logits, const GateArgs& a, cudaStream_t stream) {
  const dim3 block(kGateWarps * 32);
  auto grid = [&](int tokens) {
    const int64_t blocks = (a.N + (int64_t)kGateWarps * tokens - 1) / (kGateWarps * tokens), most = (int64_t)num_sms() * 8;
    return dim3((unsigned)(blocks < most ? blocks : most));
  };
  if (a.G == 1 && a.K <= 64) {
    if (a.K <= 16) return launch_kernel(gate_small_kernel<T, 8, 2>, grid(4), block, 0, stream, 0, logits, a);
    if (a.K <= 32) return launch_kernel(gate_small_kernel<T, 8, 4>, grid(4), block, 0, stream, 0, logits, a);
    return launch_kernel(gate_small_kernel<T, 8, 8>, grid(4), block, 0, stream, 0, logits, a);
  }
  const size_t smem = a.G > 1 ? sizeof(float) * kGateWarps * a.K : 0;
  if (a.K <= 64) return launch_kernel(gate_topk_kernel<T, 2>, grid(1), block, smem, stream, 0, logits, a);
  if (a.K <= 128) return launch_kernel(gate_topk_kernel<T, 4>, grid(1), block, smem, stream, 0, logits, a);
  if (a.K <= 256) return launch_kernel(gate_topk_kernel<T, 8>, grid(1), block, smem, stream, 0, logits, a);
  return launch_kernel(gate_topk_kernel<T, 16>, grid(1), block, smem, stream, 0, logits, a);
}

}  // namespace

cudaError_t launch_gate_topk(const void* logits, molora_dtype dtype, int64_t N, int32_t K, bool sigmoid,
                             const float* bias, int32_t groups, int32_t keep, int32_t group_top, int32_t k, bool renorm,
                             float scale, int32_t* ids, float* w, int32_t* err_word, cudaStream_t stream) {
  const uint32_t per = (uint32_t)(K / groups);
  // exact for a < 512 and per <= 512: the excess a * (per_inverse - 2^20 / per) / 2^20 < 2^-11 < 1 / per
  const GateArgs a = {N, K, bias, groups, keep, group_top, ((1u << 20) + per - 1) / per, k, sigmoid, renorm, scale,
                      ids, w, err_word};
  if (dtype == MOLORA_BF16) return launch_gate_typed(static_cast<const __nv_bfloat16*>(logits), a, stream);
  return launch_gate_typed(static_cast<const float*>(logits), a, stream);
}

}  // namespace molora
