// lora_update.cu -- the shrink for a product that takes the adapters' update along as further K blocks
// (linear_tc_kernel):
//
//   G[t, a*r + j] = scale * c[t,a] * (h[t,:] A_a)[j],   c[t,a] = sum_j [ids[t,j] == a] w[t,j]
//
// written as two bf16 planes G_hi + G_lo [N x K*r] (relative error 2^-17).
//
// Bound by reading h once from L2, where the norm has just left it.  A tile of 128 tokens x up to 256
// of the K*r columns belongs to a cluster of C CTAs that split d_in, so each reads its own columns of h
// and rows of A and nothing twice; their partial sums meet through distributed shared memory in rank
// order.  (Splitting the columns instead, as stacked_shrink_kernel does to exchange a router's hidden
// units, reads h C times: the whole projection of 4096 x 2048 -> 6144 with 4 adapters of rank 16 took 96 us
// with it and takes 87 with this.)  What is left is the way through: 8 K blocks a CTA, then the join.
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "linear.cuh"

namespace molora {

namespace {

constexpr int kKBlock = 64;
constexpr int kEpiWarps = 8, kThreads = 32 * (kEpiWarps + 2);
constexpr int kStages = 6;
constexpr size_t kSlack = 1024, kSmemLimit = 227 * 1024;

struct __align__(8) UCtrl {
  uint64_t full[kStages];
  uint64_t empty[kStages];
  uint64_t done;
  uint32_t tmem_base;
  int32_t abort;
};

struct UpdatePlan {
  int C;          // CTAs of a cluster: d_in split C ways
  int KC, NA;     // adapters, and columns, of a tile
  int groups;     // column tiles
  int nkb;
  int S;          // stages
  uint32_t stage_bytes, tmem_cols, off_ctrl, smem;
};

}  // namespace

__global__ void __launch_bounds__(kThreads, 1)
    lora_update_kernel(int64_t N, int32_t d_in, int32_t K, int32_t r, int32_t k, const int32_t* __restrict__ ids,
                       const float* __restrict__ w, float scale, __nv_bfloat16* __restrict__ g_hi,
                       __nv_bfloat16* __restrict__ g_lo, int32_t* err_word, const UpdatePlan P,
                       const __grid_constant__ CUtensorMap map_h, const __grid_constant__ CUtensorMap map_a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  UCtrl* ctrl = reinterpret_cast<UCtrl*>(sm + P.off_ctrl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = P.C, NA = P.NA, S = P.S;
  const int rank = (int)cluster_ctarank();
  const unsigned tile = blockIdx.x / (unsigned)C;
  const int a0 = (int)(tile % (unsigned)P.groups) * P.KC;
  const int64_t t0 = (int64_t)(tile / (unsigned)P.groups) * kRows;
  const int kb0 = P.nkb * rank / C, kb1 = P.nkb * (rank + 1) / C;
  volatile int32_t* abort = &ctrl->abort;

  if (warp == 9) {
    tmem_alloc(&ctrl->tmem_base, P.tmem_cols);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&ctrl->full[s], 1);
      mbar_init(&ctrl->empty[s], 1);
    }
    mbar_init(&ctrl->done, 1);
    ctrl->abort = 0;
    mbar_fence_init();
    tma_prefetch_desc(&map_h);
    tma_prefetch_desc(&map_a);
  }
  pdl_wait();
  __syncthreads();
  pdl_launch_dependents();  // with this CTA's TMEM held
  tc_fence_after();
  const uint32_t tmem = ctrl->tmem_base;

  // of the join below: 8 columns of a token a thread (one adapter's, since r >= 16), the CTA's share of the rows
  const int per_row = NA / 8, first = kRows * rank / C, rows = kRows * (rank + 1) / C - first;
  auto coefficient = [&](int q) {
    const int64_t t = t0 + first + q / per_row;
    const int c0 = (q % per_row) * 8, a = a0 + c0 / r;
    float coef = 0.f;
    if (q >= rows * per_row || t >= N || a >= K) return coef;
    for (int j = 0; j < k; ++j) {
      const int32_t id = ids[t * k + j];
      if (id == a) coef += w ? w[t * k + j] : 1.f;
      if ((id < 0 || id >= K) && a == 0 && c0 == 0) report(err_word, MOLORA_DEV_BAD_ADAPTER_ID);
    }
    return coef * scale;
  };
  float coef = warp < kEpiWarps ? coefficient(tid) : 0.f;  // on its way under the MMAs

  if (warp == 8) {
    if (elect_one()) {
      int issued = 0, s = 0;
      uint32_t phase = 1;  // the first use of a stage finds it empty
      for (int kb = kb0; kb < kb1; ++kb, ++issued) {
        if (issued >= S && !mbar_wait_spin(&ctrl->empty[s], phase, abort)) break;
        uint8_t* st = sm + (size_t)s * P.stage_bytes;
        mbar_arrive_expect_tx(&ctrl->full[s], P.stage_bytes);
        tma_load_2d(smem_u32(st), &map_h, kb * kKBlock, (int32_t)t0, &ctrl->full[s]);
        // 64 rows of each adapter of the tile; past the last adapter there is nothing (zeros)
        for (int j = 0; j < P.KC; ++j)
          tma_load_2d(smem_u32(st + kRows * 128 + (size_t)j * kKBlock * r * 2), &map_a, 0, (a0 + j) * d_in + kb * kKBlock,
                      &ctrl->full[s]);
        if (++s == S) s = 0, phase ^= 1;
      }
      for (int q = 0; q < S && q < issued; ++q) mbar_wait(&ctrl->full[q], (uint32_t)((issued - 1 - q) / S) & 1u);
    }
    __syncwarp();
  } else if (warp == 9) {
    if (elect_one()) {
      const uint32_t idesc = idesc_bf16_f32(kRows, (uint32_t)NA, false, true);
      const SmemLayout swa = r == 16 ? kSwizzle32B : r == 32 ? kSwizzle64B : kSwizzle128B;
      const uint64_t dh = smem_desc(smem_u32(sm), 16, 1024, kSwizzle128B);
      const uint64_t da = smem_desc(smem_u32(sm + kRows * 128), (uint32_t)kKBlock * r * 2, 8u * r * 2, swa);
      bool ok = true;
      int s = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait_spin(&ctrl->full[s], phase, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t at = (uint32_t)s * (P.stage_bytes >> 4);
        umma_stage<false, false>(tmem, (uint32_t)dh + at, (uint32_t)da + at, (uint32_t)(dh >> 32), (uint32_t)(da >> 32),
                                 idesc, kb != kb0, (uint32_t)(16 * r * 2) >> 4);
        umma_commit(&ctrl->empty[s]);
        if (++s == S) s = 0, phase ^= 1;
      }
      if (!ok) report(err_word, MOLORA_DEV_WAIT_TIMEOUT);
      umma_commit(&ctrl->done);
    }
    __syncwarp();
  }
  __syncthreads();  // every load has landed

  // partial sums [token][NA + 4] in the ring (the padding spreads the rows over the banks)
  float* part = reinterpret_cast<float*>(sm);
  const int stride = NA + 4;
  // a thread whose wait ran out has NaN for its sums, and so has all that is made of them, the tokens' y at last
  const bool have = mbar_wait(&ctrl->done, 0) && !*abort;
  if (!have) report(err_word, MOLORA_DEV_WAIT_TIMEOUT);
  tc_fence_after();
  if (warp < kEpiWarps) {
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t base = tmem + ((uint32_t)(quarter * 32) << 16);
    for (int c = (warp >> 2) * 16; c < NA; c += 32) {
      float v[16];
      if (__all_sync(0xffffffffu, have))
        tmem_ld16(base + (uint32_t)c, v);
      else
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(0x7fffffffu);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(part + row * stride + c + 4 * i) =
            make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (C > 1) cluster_sync();
  for (int q = tid; warp < kEpiWarps && q < rows * per_row; q += kEpiWarps * 32) {
    const int row = first + q / per_row, c0 = (q % per_row) * 8;
    const int64_t t = t0 + row;
    const int a = a0 + c0 / r;
    if (t >= N || a >= K) continue;
    float v[8] = {};
    const uint32_t at = smem_u32(part + row * stride + c0);
    for (int c = 0; c < C; ++c) {
      const uint32_t from = C > 1 ? dsmem_addr(at, (uint32_t)c) : dsmem_addr(at, 0);
      const float4 p0 = dsmem_ld_f4(from), p1 = dsmem_ld_f4(from + 16);
      v[0] += p0.x, v[1] += p0.y, v[2] += p0.z, v[3] += p0.w;
      v[4] += p1.x, v[5] += p1.y, v[6] += p1.z, v[7] += p1.w;
    }
    if (q != tid) coef = coefficient(q);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float g0 = coef * v[2 * i], g1 = coef * v[2 * i + 1];
      const __nv_bfloat16 h0 = __float2bfloat16_rn(g0), h1 = __float2bfloat16_rn(g1);
      const __nv_bfloat16 l0 = __float2bfloat16_rn(g0 - __bfloat162float(h0));
      const __nv_bfloat16 l1 = __float2bfloat16_rn(g1 - __bfloat162float(h1));
      hi[i] = (uint32_t)__bfloat16_as_ushort(h0) | ((uint32_t)__bfloat16_as_ushort(h1) << 16);
      lo[i] = (uint32_t)__bfloat16_as_ushort(l0) | ((uint32_t)__bfloat16_as_ushort(l1) << 16);
    }
    const int64_t out = t * ((int64_t)K * r) + (int64_t)a0 * r + c0;
    *reinterpret_cast<uint4*>(g_hi + out) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(g_lo + out) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  __syncthreads();
  if (C > 1) cluster_sync();  // no CTA leaves while another may still read its partial sums
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, P.tmem_cols);
  }
}

namespace {

PFN_cuTensorMapEncodeTiled_v12000 update_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    else
      cudaGetLastError();
  });
  return fn;
}

bool update_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_cols, uint32_t box_rows,
                CUtensorMapSwizzle swz) {
  auto enc = update_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * 2};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t lora_update_bytes(int64_t N, int32_t KR) { return ((size_t)N * (size_t)KR * 2 + 255) / 256 * 256; }

bool lora_update_supported(molora_dtype dtype, int64_t N, int32_t d_in, int32_t K, int32_t r) {
  // the adapters' rows are seen as one array of K * d_in of them, with 32-bit coordinates
  return dtype == MOLORA_BF16 && N > 0 && d_in % kKBlock == 0 && (r == 16 || r == 32 || r == 64) &&
         (int64_t)(K + 256 / r) * d_in <= INT32_MAX && update_encoder() != nullptr;
}

cudaError_t launch_lora_update(const void* h, int64_t N, int32_t d_in, const void* A, int32_t K, int32_t r,
                               const int32_t* ids, const float* w, int32_t k, float scale, void* g_hi, void* g_lo,
                               int32_t* err_word, cudaStream_t stream) {
  UpdatePlan p = {};
  p.groups = (K * r + 255) / 256;
  p.KC = (K + p.groups - 1) / p.groups;
  p.groups = (K + p.KC - 1) / p.KC;
  p.NA = p.KC * r;
  p.nkb = d_in / kKBlock;
  const int64_t tiles = (N + kRows - 1) / kRows * p.groups;
  p.C = 1;
  while (p.C < 8 && tiles * p.C * 2 <= num_sms() && p.nkb >= p.C * 4) p.C *= 2;
  p.stage_bytes = (uint32_t)(kRows * 128 + ((p.NA * kKBlock * 2 + 1023) / 1024) * 1024);
  p.tmem_cols = 32;
  while (p.tmem_cols < (uint32_t)p.NA) p.tmem_cols *= 2;
  p.S = (int)((kSmemLimit - sizeof(UCtrl) - kSlack) / p.stage_bytes);
  if (p.S > kStages) p.S = kStages;
  size_t ring = (size_t)p.S * p.stage_bytes;
  const size_t partial = (size_t)kRows * (p.NA + 4) * sizeof(float);
  if (ring < partial) ring = partial;
  p.off_ctrl = (uint32_t)ring;
  p.smem = (uint32_t)(ring + sizeof(UCtrl) + kSlack);
  // 116 KB at least: neither this CTA nor one that takes all of TMEM (those take as much) can then hold
  // columns that the other waits for while it is itself waited for, by its cluster or by the next kernel
  if (p.smem < 116 * 1024) p.smem = 116 * 1024;
  CUtensorMap map_h, map_a;
  const CUtensorMapSwizzle swz = r == 16   ? CU_TENSOR_MAP_SWIZZLE_32B
                                 : r == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                           : CU_TENSOR_MAP_SWIZZLE_128B;
  if (!update_map(&map_h, h, (uint64_t)N, (uint64_t)d_in, kKBlock, kRows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !update_map(&map_a, A, (uint64_t)K * d_in, (uint64_t)r, (uint32_t)r, kKBlock, swz))
    return cudaErrorNotSupported;
  static std::atomic<uint64_t> allowed;
  const cudaError_t set = allow_smem(lora_update_kernel, allowed, kSmemLimit);
  if (set != cudaSuccess) return set;
  return launch_kernel(lora_update_kernel, dim3((unsigned)(tiles * p.C)), dim3(kThreads), p.smem, stream, p.C, N, d_in, K,
                       r, k, ids, w, scale, static_cast<__nv_bfloat16*>(g_hi), static_cast<__nv_bfloat16*>(g_lo),
                       err_word, p, map_h, map_a);
}

}  // namespace molora
