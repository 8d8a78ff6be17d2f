// gate.cu -- expert-style gate over given logits: softmax or sigmoid scores, a bias that only
// moves the choice, groups of which the best are kept, the k best experts, renormalised weights.
//
// A token belongs to TL lanes of a warp; lane l of them holds experts l, l + TL, l + 2 TL, ...: every
// load is of consecutive logits, whatever K and the rows' alignment.
//
// Bound by instructions, not bytes: 16384 x 256 fp32 in 8 groups takes 18.1 us (its 17.8 MB would take 2.6),
// about 1000 warp instructions a token: the sigmoids 2.5 us of it, the bound 1.0, the candidates 2.3, their
// ranks 2.0.  Fetching the next token's logits ahead, or other grids, gained nothing.  40961 x 60 bf16 with a
// bias takes 16.4 us, 32 x 64 1.6 us, a launch.
//
// Everything the choice depends on is reproducible: e = expf(l - max) and 1 / (1 + expf(-l)) are
// single fp32 operations, and the softmax's denominator is a sum of integers (each e in units of 2^-44 of the
// largest) that is rounded once, so it does not depend on the order of the sum.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace molora {

namespace {

constexpr int kGateWarps = 8;
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kFloatMax = 3.4028234663852886e38f;
constexpr float kLowest = -__builtin_huge_valf();

struct GateArgs {
  int64_t N;
  int32_t K;
  const float* bias;
  int32_t G, keep, group_top;
  int32_t group_lanes;   // lanes that look for a group's best: 32 / G rounded down to a power of two
  uint32_t per_inverse;  // ceil(2^20 / (K / G)): a * per_inverse >> 20 is expert a's group
  int32_t k;
  bool sigmoid, renorm;
  float scale;
  int32_t* ids;
  float* w;
  int32_t* err_word;
};

// Order-preserving map of a float (not NaN) to an unsigned integer.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);  // -0 and +0 are equal
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float from_ordered(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// What a token's scores come from: its largest logit and, where needed, the softmax's denominator.
struct Norms {
  float most, total;
};

__device__ __forceinline__ float score_of(const GateArgs& a, float l, const Norms& n) {
  if (a.sigmoid) return __frcp_rn(__fadd_rn(1.f, expf(-l)));
  const float e = l == kLowest ? 0.f : expf(l - n.most);
  return n.total > 0.f ? __fdiv_rn(e, n.total) : 0.f;
}

// The biases of this lane's experts first, first + step, ..., made finite or -inf.
template <int V>
__device__ __forceinline__ void gate_bias(const GateArgs& a, int first, int step, float (&b)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    b[i] = a.bias && first + step * i < a.K ? a.bias[first + step * i] : 0.f;
    if (b[i] != b[i]) {
      report(a.err_word, MOLORA_DEV_BAD_LOGIT);
      b[i] = kLowest;
    }
    b[i] = fminf(b[i], kFloatMax);
  }
}

// The choices c of this lane's experts from their logits l (-inf past K, NaN made -inf and +inf finite
// here) and biases.  Returns what score_of needs; the softmax's denominator is left at 1 where the
// choice does not need it and the weights are renormalised anyway.
template <int TL, int V>
__device__ __forceinline__ Norms gate_choices(const GateArgs& a, float (&l)[V], const float (&b)[V], float (&c)[V]) {
  const bool by_logit = !a.bias && (a.G == 1 || a.group_top == 1);
  bool odd = false;
#pragma unroll
  for (int i = 0; i < V; ++i) odd |= !(l[i] <= kFloatMax);
  if (__any_sync(kFull, odd)) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (l[i] != l[i]) report(a.err_word, MOLORA_DEV_BAD_LOGIT);
      l[i] = l[i] != l[i] ? kLowest : fminf(l[i], kFloatMax);
    }
  }
  Norms n = {0.f, 1.f};
  if (!a.sigmoid) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
#pragma unroll
    for (int off = TL / 2; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
    n.most = m;
    if (!by_logit || !a.renorm) {
      // e in units of 2^-22 and 2^-44, summed as integers: exact whatever the order (what an e below 2^-21
      // has under 2^-44 is cut: 512 experts lose less than 2^-35), 512 experts fit 32 bits
      uint32_t hi = 0, lo = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        c[i] = l[i] == kLowest ? 0.f : expf(l[i] - m);
        const float u = c[i] * 4194304.f;
        const uint32_t h = __float2uint_rz(u);
        hi += h;
        lo += __float2uint_rz((u - (float)h) * 4194304.f);
      }
      if constexpr (TL == 32) {
        hi = __reduce_add_sync(kFull, hi);
        lo = __reduce_add_sync(kFull, lo);
      } else {
#pragma unroll
        for (int off = TL / 2; off; off >>= 1) {
          hi += __shfl_xor_sync(kFull, hi, off);
          lo += __shfl_xor_sync(kFull, lo, off);
        }
      }
      n.total = __ull2float_rn(((unsigned long long)hi << 22) + lo) * 5.6843418860808015e-14f;  // 2^-44
    }
  }
  if (by_logit) {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = l[i];
  } else if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      c[i] = l[i] == kLowest ? kLowest : __fadd_rn(__frcp_rn(__fadd_rn(1.f, expf(-l[i]))), b[i]);
  } else {
    const bool some = n.total > 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = l[i] == kLowest || !some ? kLowest : __fadd_rn(__fdiv_rn(c[i], n.total), b[i]);
  }
  return n;
}

// The k largest choices by k rounds of a maximum over the token's lanes, ties to the lower index;
// stores the token's ids and weights if `live`.
template <int TL, int V>
__device__ __forceinline__ void gate_rounds(const GateArgs& a, float (&c)[V], const float (&l)[V], const Norms& n,
                                            int64_t t, bool live) {
  const int sub = threadIdx.x & (TL - 1);
  int place[V];  // the round that took expert sub + TL * i
#pragma unroll
  for (int i = 0; i < V; ++i) place[i] = -1;
  int found = 0;
  for (int j = 0; j < a.k; ++j) {
    float top = c[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = fmaxf(top, c[i]);
#pragma unroll
    for (int off = TL / 2; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
    int at = INT32_MAX;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
      if (c[i] == top) at = sub + TL * i;
#pragma unroll
    for (int off = TL / 2; off; off >>= 1) at = min(at, __shfl_xor_sync(kFull, at, off));
    if (top > kLowest) {
      ++found;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (at == sub + TL * i) c[i] = kLowest, place[i] = j;
    }
  }
  float s[V], sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    s[i] = 0.f;
    if (place[i] >= 0) s[i] = score_of(a, l[i], n), sum += s[i];
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

// Stores the ids and weights of a token whose found experts, best first, stand with their scores in the warp's
// first lanes: the sum of the scores depends on their order alone.
__device__ __forceinline__ void gate_store(const GateArgs& a, float score, int id, int found, int64_t t) {
  const int lane = threadIdx.x & 31;
  if (lane >= found) score = 0.f, id = -1;
  float sum = score;
  if (a.renorm) {
#pragma unroll
    for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
  }
  if (lane < a.k) {
    const float w = !a.renorm ? score : sum > 0.f ? score / sum : 0.f;
    a.ids[t * a.k + lane] = id;
    a.w[t * a.k + lane] = w * a.scale;
  }
}

// The same for a warp a token, with the choices as ordered integers: a maximum, and the lowest index that
// has it, is one instruction over the warp.
template <int V, bool kBlocked>
__device__ __forceinline__ void gate_rounds_warp(const GateArgs& a, const float (&c)[V], const float (&l)[V],
                                                 const Norms& n, int64_t t) {
  const int lane = threadIdx.x & 31;
  auto expert = [&](int i) { return (uint32_t)(kBlocked ? V * lane + i : lane + 32 * i); };
  const uint32_t none = ordered(kLowest);
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = ordered(c[i]);
  uint32_t mine = 0;  // lane j: the expert of round j
  int found = 0;
  for (; found < a.k; ++found) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = max(best, key[i]);
    const uint32_t top = __reduce_max_sync(kFull, best);
    if (top <= none) break;
    uint32_t at = 0xffffffffu;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
      if (key[i] == top) at = expert(i);
    at = __reduce_min_sync(kFull, at);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (at == expert(i)) key[i] = 0u;
    if (lane == found) mine = at;
  }
  float logit = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float from = __shfl_sync(kFull, l[i], kBlocked ? mine / V : mine & 31);
    if ((int)(kBlocked ? mine % V : mine >> 5) == i) logit = from;
  }
  gate_store(a, lane < found ? score_of(a, logit, n) : 0.f, (int)mine, found, t);
}

}  // namespace

// Up to 16 experts in one group: TL lanes a token, so that a warp's every instruction works for
// 32 / TL tokens and a maximum over the lanes takes log2(TL) steps.  (With 64 experts, 8 a lane, this
// took 18 us where a warp a token takes 16, and twice as long for a few tokens.)
template <typename T, int TL, int V>
__global__ void __launch_bounds__(kGateWarps * 32, 4) gate_small_kernel(const T* __restrict__ logits, const GateArgs a) {
  constexpr int kTokens = 32 / TL;  // of a warp
  const int lane = threadIdx.x & 31, sub = lane & (TL - 1), warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_launch_dependents();
  float b[V];
  gate_bias<V>(a, sub, TL, b);
  for (int64_t t0 = ((int64_t)blockIdx.x * kGateWarps + warp) * kTokens; t0 < a.N;
       t0 += (int64_t)gridDim.x * kGateWarps * kTokens) {
    const int64_t t = t0 + lane / TL;
    const bool live = t < a.N;
    float l[V], c[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
      l[i] = live && sub + TL * i < a.K ? to_float(logits[t * a.K + sub + TL * i]) : kLowest;
    const Norms n = gate_choices<TL, V>(a, l, b, c);
    gate_rounds<TL, V>(a, c, l, n, t, live);
  }
}

// More experts, or groups: a warp a token, 32 V experts at most.  With up to four a lane the choice is made
// in rounds; with more, the k-th largest of the 32 lanes' own maxima is a bound that the k largest choices
// reach and few others do, and those that do (k and a few) are ranked by counting, in shared memory
// (16384 x 256, top 8 by logits: 10.5 us, 14.0 in rounds; 512 experts 31.4 against 37.7).
//
// kBlocked: groups of 32 / G whole lanes, which hold V consecutive experts each (32 V experts in a power of
// two of groups): a group's best two come from registers and a few shuffles, and a lane stays or goes as one
// (16384 x 256 in 8 groups 18.1 us; 19.3 through shared memory, which other sizes take).
template <typename T, int V, bool kBlocked>
__global__ void __launch_bounds__(kGateWarps * 32, V <= 8 ? 4 : 2) gate_topk_kernel(const T* __restrict__ logits, const GateArgs a) {
  extern __shared__ float choices[];  // [warps][K], with groups that do not follow the lanes
  __shared__ float2 cand[kGateWarps][32];  // (choice, expert) of those that reach the bound
  __shared__ float cand_l[kGateWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t below = (1u << lane) - 1u;
  auto expert = [&](int i) { return kBlocked ? V * lane + i : lane + 32 * i; };
  pdl_wait();
  pdl_launch_dependents();
  float b[V];
  gate_bias<V>(a, expert(0), kBlocked ? 1 : 32, b);
  for (int64_t t = (int64_t)blockIdx.x * kGateWarps + warp; t < a.N; t += (int64_t)gridDim.x * kGateWarps) {
    float l[V], c[V];
    const T* row = logits + t * a.K;
    if constexpr (kBlocked) {
      constexpr int kBytes = V * sizeof(T) < 16 ? V * sizeof(T) : 16, kEach = kBytes / sizeof(T);
      struct alignas(kBytes) Run {
        T v[kEach];
      };
#pragma unroll
      for (int i = 0; i < V; i += kEach) {
        const Run run = *reinterpret_cast<const Run*>(row + expert(i));
#pragma unroll
        for (int j = 0; j < kEach; ++j) l[i + j] = to_float(run.v[j]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) l[i] = expert(i) < a.K ? to_float(row[expert(i)]) : kLowest;
    }
    const Norms n = gate_choices<32, V>(a, l, b, c);
    if (kBlocked || a.G > 1) {
      // each group's best, or best two
      float* mine = choices + (size_t)warp * a.K;
      const int lanes = a.group_lanes, g = lane / lanes;
      float c1 = kLowest, c2 = kLowest;
      if constexpr (kBlocked) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          c2 = fmaxf(c2, fminf(c1, c[i]));
          c1 = fmaxf(c1, c[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (expert(i) < a.K) mine[expert(i)] = c[i];
        __syncwarp();
        const int per = a.K / a.G;
        if (g < a.G) {
          for (int i = lane & (lanes - 1); i < per; i += lanes) {
            const float v = mine[g * per + i];
            c2 = fmaxf(c2, fminf(c1, v));
            c1 = fmaxf(c1, v);
          }
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
      if constexpr (kBlocked) {
        if (!((kept >> g) & 1u))
#pragma unroll
          for (int i = 0; i < V; ++i) c[i] = kLowest;
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (!((kept >> ((expert(i) * a.per_inverse) >> 20 & 31u)) & 1u)) c[i] = kLowest;
        __syncwarp();
      }
    }
    if constexpr (V <= 4) {
      gate_rounds_warp<V, kBlocked>(a, c, l, n, t);
      continue;
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
    const float least = fmaxf(from_ordered(bound), -kFloatMax);  // experts that are out are below
    int count = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool in = c[i] >= least;
      const uint32_t who = __ballot_sync(kFull, in);
      const int at = count + __popc(who & below);
      if (in && at < 32) {
        cand[warp][at] = make_float2(c[i], __int_as_float(expert(i)));
        cand_l[warp][at] = l[i];
      }
      count += __popc(who);
    }
    if (count > 32) {  // many equal choices
      gate_rounds_warp<V, kBlocked>(a, c, l, n, t);
      continue;
    }
    __syncwarp();
    const bool has = lane < count;
    const float2 mine = cand[warp][has ? lane : 0];
    int rank = 0;
#pragma unroll 4
    for (int i = 0; i < count; ++i) {
      const float2 o = cand[warp][i];
      rank += o.x > mine.x || (o.x == mine.x && __float_as_int(o.y) < __float_as_int(mine.y));
    }
    const bool chosen = has && rank < a.k;
    const float score = chosen ? score_of(a, cand_l[warp][lane], n) : 0.f;
    __syncwarp();
    if (chosen) cand[warp][rank] = make_float2(score, mine.y);
    __syncwarp();
    gate_store(a, cand[warp][lane].x, __float_as_int(cand[warp][lane].y), min(count, a.k), t);
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
  if (a.G == 1 && a.K <= 16) {
    if (a.K <= 8) return launch_kernel(gate_small_kernel<T, 8, 1>, grid(4), block, 0, stream, 0, logits, a);
    return launch_kernel(gate_small_kernel<T, 8, 2>, grid(4), block, 0, stream, 0, logits, a);
  }
  auto go = [&](auto blocked) {
    constexpr bool kB = decltype(blocked)::value;
    const size_t smem = a.G > 1 && !kB ? sizeof(float) * kGateWarps * a.K : 0;
    if (a.K <= 32) return launch_kernel(gate_topk_kernel<T, 1, kB>, grid(1), block, smem, stream, 0, logits, a);
    if (a.K <= 64) return launch_kernel(gate_topk_kernel<T, 2, kB>, grid(1), block, smem, stream, 0, logits, a);
    if (a.K <= 128) return launch_kernel(gate_topk_kernel<T, 4, kB>, grid(1), block, smem, stream, 0, logits, a);
    if (a.K <= 256) return launch_kernel(gate_topk_kernel<T, 8, kB>, grid(1), block, smem, stream, 0, logits, a);
    return launch_kernel(gate_topk_kernel<T, 16, kB>, grid(1), block, smem, stream, 0, logits, a);
  };
  const bool powers = a.K >= 32 && (a.K & (a.K - 1)) == 0 && a.G > 1 && (a.G & (a.G - 1)) == 0;
  if (powers && (reinterpret_cast<uintptr_t>(logits) & 15) == 0) return go(std::true_type());
  return go(std::false_type());
}

}  // namespace

cudaError_t launch_gate_topk(const void* logits, molora_dtype dtype, int64_t N, int32_t K, bool sigmoid,
                             const float* bias, int32_t groups, int32_t keep, int32_t group_top, int32_t k, bool renorm,
                             float scale, int32_t* ids, float* w, int32_t* err_word, cudaStream_t stream) {
  const uint32_t per = (uint32_t)(K / groups);
  // exact for a < 512 and per <= 512: the excess a * (per_inverse - 2^20 / per) / 2^20 < 2^-11 < 1 / per
  int32_t lanes = 1;
  while (lanes * 2 * groups <= 32) lanes *= 2;
  const GateArgs a = {N, K, bias, groups, keep, group_top, lanes, ((1u << 20) + per - 1) / per, k, sigmoid, renorm, scale,
                      ids, w, err_word};
  if (dtype == MOLORA_BF16) return launch_gate_typed(static_cast<const __nv_bfloat16*>(logits), a, stream);
  return launch_gate_typed(static_cast<const float*>(logits), a, stream);
}

}  // namespace molora
