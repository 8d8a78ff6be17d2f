// linear.cu -- the base product with its epilogue on the 5th-generation tensor cores, bf16 or
// e4m3 operands with fp32 accumulators in TMEM:
//
//   y[t,o] = act(sx[t] * sw[o] * sum_i x[t,i] W[o,i] + bias[o]) + residual[t,o]
//
// x and W are both rows along d_in (K-major), so a stage of either is a 128-byte-swizzled box of
// rows x 128 bytes, 64 bf16 or 128 e4m3 elements of K, and the two types differ in the MMA's kind and
// in nothing else.  Elements past the arrays' ends are loaded as zeros and never stored.
//
// linear_tc_kernel (many tokens): a persistent kernel over tiles of 256 tokens x BN outputs, each made
//   by a pair of CTAs with cta_group::2 MMAs.  Each CTA loads its 128 token rows and half of the
//   tile's W rows: a pair reads every operand byte once from shared memory per MMA, which
//   one CTA alone cannot feed at full rate.  A TMA warp and an MMA warp run ahead of 12 (or 8, see
//   tc_sides) epilogue warps by two TMEM accumulators.  Bound by the tensor cores: 8192 x 4096 x 4096 bf16
//   143 us (1920 TFLOP/s; tensor pipe active in 89% of the cycles), 151 with bias, SiLU and residual (165 and 174 in
//   a long loop, at the power limit); e4m3 76 us (3600).  4096 x 2048 x 6144 e4m3 with scales, bias and GELU's tanh form 40 us, 36 without: there
//   the epilogue of 224 columns is nearly as long as a tile's 16 K blocks.
// linear_skinny_kernel (few tokens): W's rows are the MMA's M (128 outputs a CTA), the tokens its N
//   (16 .. 256), so that no MMA row is spent on tokens that are not there; d_in is split over a
//   cluster of CTAs whose partial sums meet through distributed shared memory in rank order.  Bound by
//   reading W, and the way through the kernel: one token, 4096 x 4096 bf16, 7.4 us (W's bytes: 5.0).
// linear_any_kernel (fp32, and rows that start anywhere): the same split, with the operands fetched and
//   laid out by the CTA's threads.
// linear_few_kernel (a token of little W or of rows that start anywhere, a few of fp32): the CUDA cores.
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>
#ifdef MOLORA_TUNING_ENV
#include <cstdlib>
#endif

#include "common.cuh"
#include "kernels.h"
#include "linear.cuh"

namespace molora {

namespace {

constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpiWarps + 2);  // + TMA warp (8) + MMA warp (9)
constexpr int kAnyThreads = 512;    // linear_any_kernel: 15 warps that lay out operands + MMA warp (15)
constexpr int kCutters = kAnyThreads - 32;
constexpr int kSpan = 8;            // K blocks summed in TMEM before fp32 registers take over

struct __align__(8) LCtrl {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t done;
  uint64_t res_full[12];
  uint32_t tmem_base;
  int32_t abort;
};

// What the epilogue reads and writes.
struct Epi {
  const float* sx;
  const float* sw;
  const float* bias;
  const void* res;
  void* y;
  int64_t N;
  int32_t d_out;
  molora_activation act;
  bool y_bf16;
  bool tma_y;    // rows of y and residual on 16-byte boundaries: linear_tc_kernel moves them by TMA
};

struct TcPlan {
  int BN;                // outputs per tile
  int S;                 // stages
  int nkb;               // K blocks of 128 bytes
  int nkg;               // K blocks of 64 of the adapters' update (0: none)
  int group;             // token tiles per group of tiles (they share W's rows in L2)
  int64_t m_tiles, tiles;
  int32_t n_tiles;
  uint32_t stage_bytes, off_b, off_stage, off_ctrl, tmem_cols, smem;
};

// The sums of a tile of 128 outputs x tokens that its 8 epilogue warps keep: warp w's lanes have outputs
// 32 (w % 4) .. + 31, columns 16 (w / 4) + 32 j .. + 15.  TMEM's own are added every kSpan K blocks,
// in two buffers of BN columns in turn (see linear_tc_kernel).
template <int J>
struct TileSums {
  float v[J][16];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 16; ++i) v[j][i] = 0.f;
  }
  __device__ __forceinline__ void add(uint32_t tmem, int tokens) {
    const int warp = threadIdx.x >> 5;
    const uint32_t base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = (warp >> 2) * 16 + 32 * j;
      if (c >= tokens) continue;
      float p[16];
      tmem_ld16(base + (uint32_t)c, p);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[j][i] += p[i];
    }
  }
  // Span number `c`: waits for its MMAs, takes its sums and frees its buffer.
  __device__ __forceinline__ bool take(LCtrl* ctrl, int c, uint32_t tmem, int BN, int tokens) {
    if (!__all_sync(0xffffffffu, mbar_wait_spin(&ctrl->tfull[c & 1], (uint32_t)(c >> 1) & 1u, &ctrl->abort))) return false;
    tc_fence_after();
    add(tmem + (uint32_t)((c & 1) * BN), tokens);
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&ctrl->tempty[c & 1]);
    return true;
  }
};

// Ends such a tile, whose d_in was split over a cluster's C CTAs: each CTA's sums go to shared memory,
// [token][output] in the stage ring (free: every load has landed and every MMA is done); each CTA then adds
// its share of the elements in rank order, reading the others' through distributed shared memory, and
// writes it.  Four outputs at a time and U such quads in flight a thread: element by element, one
// remote access after another, this was 12 of 20 us at 257 x 1031 x 517.  kAgain: a sum that is NaN is made anew by
// `again(t, o)`.  Called by all threads; `have` is false
// where a wait ran out: such a thread's sums are NaN, and so is what any CTA of the cluster makes of them.  (Leaving
// their outputs unwritten takes a flag of the cluster: 0.1 to 0.4 us a call, however it is passed on.)
template <int U, bool kAgain, int J, typename F>
__device__ __forceinline__ void split_epilogue(const Epi& E, const TileSums<J>& sums, bool have, uint8_t* sm, int C, int rank,
                                               int32_t o0, int64_t t0, int tokens, int32_t* err_word, F again) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float* part = reinterpret_cast<float*>(sm);
  if (!have) report(err_word, MOLORA_DEV_WAIT_TIMEOUT);
  if (warp < kEpiWarps) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = (warp >> 2) * 16 + 32 * j;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (c + i < tokens) part[(c + i) * kRows + (warp & 3) * 32 + lane] = have ? sums.v[j][i] : __uint_as_float(0x7fffffffu);
    }
  }
  __syncthreads();
  if (C > 1) cluster_sync();
  if (warp < kEpiWarps) {
    const bool vec = E.tma_y;  // (d_out a multiple of 4 and y, residual aligned)
    const bool bias_vec = vec && (reinterpret_cast<uintptr_t>(E.bias) & 15u) == 0;
    const bool sw_vec = vec && (reinterpret_cast<uintptr_t>(E.sw) & 15u) == 0;
    const int quads = tokens * (kRows / 4), step = C * 256;
    for (int q0 = rank * 256 + tid; q0 < quads; q0 += U * step) {
      Quad v[U], res[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int q = q0 + u * step, o = o0 + (q % (kRows / 4)) * 4;
        if (q >= quads || o >= E.d_out) continue;
        const int64_t row = (t0 + q / (kRows / 4)) * E.d_out;
        if (E.res) {
          if (E.y_bf16)
            res[u].load(static_cast<const __nv_bfloat16*>(E.res) + row, o, E.d_out, vec);
          else
            res[u].load(static_cast<const float*>(E.res) + row, o, E.d_out, vec);
        }
        float4 p[8];
        const uint32_t at = smem_u32(part + 4 * q);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (c < C) p[c] = C > 1 ? dsmem_ld_f4(dsmem_addr(at, (uint32_t)c)) : *reinterpret_cast<const float4*>(part + 4 * q);
        v[u].v[0] = p[0].x, v[u].v[1] = p[0].y, v[u].v[2] = p[0].z, v[u].v[3] = p[0].w;
#pragma unroll
        for (int c = 1; c < 8; ++c)
          if (c < C) v[u].v[0] += p[c].x, v[u].v[1] += p[c].y, v[u].v[2] += p[c].z, v[u].v[3] += p[c].w;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int q = q0 + u * step, o = o0 + (q % (kRows / 4)) * 4;
        if (q >= quads || o >= E.d_out) continue;
        const int64_t t = t0 + q / (kRows / 4), row = t * E.d_out;
        if constexpr (kAgain) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (o + i < E.d_out && v[u].v[i] != v[u].v[i]) v[u].v[i] = again(t, o + i);
        }
        if (E.sx) {
          Quad w;
          w.load(E.sw, o, E.d_out, sw_vec);
          const float sx = E.sx[t];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[u].v[i] *= sx * w.v[i];
        }
        if (E.bias) {
          Quad w;
          w.load(E.bias, o, E.d_out, bias_vec);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[u].v[i] += w.v[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u].v[i] = activate(v[u].v[i], E.act);
        if (E.res)
#pragma unroll
          for (int i = 0; i < 4; ++i) v[u].v[i] += res[u].v[i];
        if (E.y_bf16)
          v[u].store(static_cast<__nv_bfloat16*>(E.y) + row, o, E.d_out, vec);
        else
          v[u].store(static_cast<float*>(E.y) + row, o, E.d_out, vec);
      }
    }
  }
  __syncthreads();
  if (C > 1) cluster_sync();  // no CTA leaves while another may still read its partial sums
}

}  // namespace

// linear_tc_kernel's epilogue: groups of 4 warps that share a tile's chunks, and the CTA's threads.  Three groups
// where a chunk's registers allow it: 8192 x 1024 -> 4096 e4m3 with two 43 us, with three 39, and with GELU 56
// and 52; 4096 x 1024 -> 4096 bf16 with GELU's tanh form 34 and 31.  Where K is long the tensor cores bound both
// (8192 x 4096 x 4096 bf16 141 and 142).
constexpr int tc_sides(bool promote) { return promote ? 2 : 3; }
constexpr int tc_threads(bool promote) { return 32 * (4 * tc_sides(promote) + 2); }

// kPromote: a tensor core cuts what its sums lose in an addition, always towards zero, so a long chain of
// MMAs drifts: 256 of them (d_in = 4096) leave an fp32 result 4e-6 short, 40 times what rounding
// would.  For fp32 y the epilogue warps take the sums of every 8 K blocks (32 MMAs) into registers
// and add there.  With e4m3 operands it takes the adapters' update along: the product's sums are
// scaled in registers before the update's, which have no scales, are added.
template <bool kFp8, bool kPromote, bool kY16>
__global__ void __launch_bounds__(tc_threads(kPromote), 1)
    linear_tc_kernel(const Epi E, const TcPlan P, int32_t* err_word, const __grid_constant__ CUtensorMap map_x,
                     const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_y,
                     const __grid_constant__ CUtensorMap map_ghi, const __grid_constant__ CUtensorMap map_glo,
                     const __grid_constant__ CUtensorMap map_b, const __grid_constant__ CUtensorMap map_r) {
  constexpr int kParts = kY16 ? 1 : 2;  // boxes of a chunk of 32 columns of y
  constexpr uint32_t kSet = kParts * kBox;
  constexpr int kSides = tc_sides(kPromote), kWarps = 4 * kSides, kMine = (8 + kSides - 1) / kSides;  // chunks a warp
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  LCtrl* ctrl = reinterpret_cast<LCtrl*>(sm + P.off_ctrl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int BN = P.BN, S = P.S, nkb = P.nkb;
  // the adapters' update is more K blocks: (G_hi, B), (G_lo, B) in turn
  const int all = nkb + 2 * P.nkg;
  // the end of the K blocks from `first` on that are summed in TMEM together
  auto span_end = [&](int first) {
    if (!kPromote) return all;
    if (kFp8) return first < nkb ? nkb : all;
    return min(first + kSpan, all);
  };
  const uint32_t rank = cluster_ctarank();
  const uint16_t both = 0x3;
  const int64_t pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  volatile int32_t* abort = &ctrl->abort;
  // tiles in groups of P.group token tiles: within a group, the token tile runs fastest
  auto tile_at = [&](int64_t pt, int32_t& m0, int32_t& n0) {
    const int64_t span = (int64_t)P.group * P.n_tiles, grp = pt / span;
    const int64_t first = grp * P.group, left = P.m_tiles - first, rows = left < P.group ? left : P.group;
    const int64_t in = pt - grp * span;
    m0 = (int32_t)((first + in % rows) * 2 * kRows + rank * kRows);
    n0 = (int32_t)(in / rows) * BN;
  };

  if (warp == kWarps + 1) {
    tmem_alloc_pair(&ctrl->tmem_base, P.tmem_cols);
    tmem_relinquish_pair();
  }
  if (warp == kWarps && lane == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&ctrl->full[s], 1);
      mbar_init(&ctrl->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctrl->tfull[b], 1);
      mbar_init(&ctrl->tempty[b], 2 * kWarps);
    }
    mbar_init(&ctrl->done, 1);
    for (int b = 0; b < kWarps; ++b) mbar_init(&ctrl->res_full[b], 1);
    ctrl->abort = 0;
    mbar_fence_init();
    tma_prefetch_desc(&map_x);
    tma_prefetch_desc(&map_w);
    if (P.nkg) {
      tma_prefetch_desc(&map_ghi);
      tma_prefetch_desc(&map_glo);
      tma_prefetch_desc(&map_b);
    }
    if (E.tma_y) tma_prefetch_desc(&map_y);
    if (E.tma_y && E.res) tma_prefetch_desc(&map_r);
  }
  pdl_wait();
  __syncthreads();
  // only now, with this CTA's TMEM held, may the next kernel's CTAs come and ask for theirs
  pdl_launch_dependents();
  tc_fence_after();
  const uint32_t tmem = ctrl->tmem_base;
  cluster_sync();  // every CTA's barriers are initialised before another signals them

  if (warp == kWarps) {
    if (elect_one()) {
      const int elems = kFp8 ? 128 : 64;  // K elements per stage
      int s = 0, issued = 0;
      uint32_t phase = 1;  // the first use of a stage finds it empty
      bool ok = true;
      for (int64_t pt = pair; pt < P.tiles && ok; pt += pairs) {
        int32_t m0, n0;
        tile_at(pt, m0, n0);
        for (int kb = 0; kb < all; ++kb) {
          if (issued >= S && !mbar_wait_spin(&ctrl->empty[s], phase, abort)) {
            ok = false;
            break;
          }
          // the leader's barrier counts both CTAs' bytes
          const uint32_t bar = dsmem_addr(smem_u32(&ctrl->full[s]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&ctrl->full[s], 2 * P.stage_bytes);
          uint8_t* st = sm + (size_t)s * P.stage_bytes;
          const int32_t n = n0 + (int32_t)rank * (BN / 2);
          if (kb < nkb) {
            tma_load_2d_pair(smem_u32(st), &map_x, kb * elems, m0, bar);
            tma_load_2d_pair(smem_u32(st + P.off_b), &map_w, kb * elems, n, bar);
          } else {
            const int g = (kb - nkb) >> 1;
            tma_load_2d_pair(smem_u32(st), (kb - nkb) & 1 ? &map_glo : &map_ghi, g * 64, m0, bar);
            // B's columns in boxes of 64 rows x 16 columns, as many bytes as W's box
            for (int q = 0; q < BN / 32; ++q)
              tma_load_2d_pair(smem_u32(st + P.off_b + q * 2048), &map_b, n + q * 16, g * 64, bar);
          }
          if (issued < S) ++issued;
          if (++s == S) s = 0, phase ^= 1;
        }
      }
      // the last fill of every stage has been consumed before the CTA leaves
      for (int i = 0; i < issued; ++i) {
        if (issued < S) {
          mbar_wait(&ctrl->empty[i], 0);
        } else {
          mbar_wait(&ctrl->empty[s], phase);
          if (++s == S) s = 0, phase ^= 1;
        }
      }
    }
    __syncwarp();
  } else if (warp == kWarps + 1) {
    if (rank == 0 && elect_one()) {
      const uint32_t idesc = kFp8 ? idesc_e4m3_f32(2 * kRows, (uint32_t)BN) : idesc_bf16_f32(2 * kRows, (uint32_t)BN, false, false);
      // descriptors of stage 0: K-major operands of 128-byte rows, and the update's B (see the TMA warp)
      const uint64_t da = smem_desc(smem_u32(sm), 16, 1024, kSwizzle128B);
      const uint64_t db = smem_desc(smem_u32(sm + P.off_b), 16, 1024, kSwizzle128B);
      const uint64_t dg = smem_desc(smem_u32(sm + P.off_b), 2048, 256, kSwizzle32B);
      const uint32_t a_lo = (uint32_t)da, b_lo = (uint32_t)db, desc_hi = (uint32_t)(da >> 32);
      const uint32_t g_lo = (uint32_t)dg, g_hi = (uint32_t)(dg >> 32);
      int s = 0, tc = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int64_t pt = pair; pt < P.tiles && ok; pt += pairs) {
        for (int first = 0, last; first < all && ok; first = last, ++tc) {
          const int buf = tc & 1;
          last = span_end(first);
          if (tc >= 2 && !mbar_wait_spin(&ctrl->tempty[buf], (uint32_t)((tc >> 1) - 1) & 1u, abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + (uint32_t)(buf * (P.tmem_cols / 2));
          for (int kb = first; kb < last; ++kb) {
            if (!mbar_wait_spin(&ctrl->full[s], phase, abort)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t at = (uint32_t)s * (P.stage_bytes >> 4);
            if (kb >= nkb)  // B's columns are MN-major
              umma_stage<true, false>(d, a_lo + at, g_lo + at, desc_hi, g_hi, idesc_bf16_f32(2 * kRows, (uint32_t)BN, false, true),
                                      kb != first, 32);
            else
              umma_stage<true, kFp8>(d, a_lo + at, b_lo + at, desc_hi, desc_hi, idesc, kb != first);
            umma_commit_pair(&ctrl->empty[s], both);
            if (++s == S) s = 0, phase ^= 1;
          }
          if (ok) umma_commit_pair(&ctrl->tfull[buf], both);
        }
      }
      if (!ok) report(err_word, MOLORA_DEV_WAIT_TIMEOUT);
      umma_commit_pair(&ctrl->done, both);  // arrives in both CTAs once every MMA has completed
    }
    __syncwarp();
  } else {
    // epilogue: warps w, w + 4, ... share 32 rows and take chunks of 32 columns in turn
    const int quarter = warp & 3, side = warp >> 2;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    // y leaves through boxes of 32 rows x 64 bytes: one of bf16, two of fp32.  The residual's chunk is fetched
    // into them while the chunk's sums are awaited and worked on, is read from there and makes room for
    // y's.  (Loaded into registers, a row a lane, it took fp32 y from 230 to 310 us at 8192 x 4096 x 4096,
    // now to 250.)  One set of boxes a warp: the store before has long read it, and a second would take
    // a stage from the ring (140 -> 145 us).
    uint8_t* set = sm + P.off_stage + (size_t)warp * kSet;
    const bool add = E.tma_y && E.res;
    int tc = 0, chunk = 0, asked = 0;  // chunks done, and residual chunks on their way or taken
    auto ask = [&](int32_t col, int32_t m0) {
      if (lane == 0) {
        bulk_wait_read<0>();  // the last store has read the boxes
        mbar_arrive_expect_tx(&ctrl->res_full[warp], kSet);
        for (int q = 0; q < kParts; ++q)  // (past d_out there is nothing: zeros)
          tma_load_2d(smem_u32(set + q * kBox), &map_r, col + q * 16, m0, &ctrl->res_full[warp]);
      }
      ++asked;
    };
    bool ok = true;
    for (int64_t pt = pair; pt < P.tiles && ok; pt += pairs) {
      int32_t m0, n0;
      tile_at(pt, m0, n0);
      m0 += quarter * 32;
      const int64_t t = (int64_t)m0 + lane;
      const float sx = E.sx && t < E.N ? E.sx[t] : 1.f;
      const int chunks = m0 < E.N ? min(BN / 32, (E.d_out - n0 + 31) / 32) : 0;
      // while the tile's MMAs run: this lane's column of each of its chunks' scales and biases, which a
      // chunk's rows get by shuffles, and the residual's rows on their way to L2
      float cs[kMine], cb[kMine];
#pragma unroll
      for (int q = 0; q < kMine; ++q) {
        const int o = n0 + (side + kSides * q) * 32 + lane;
        const bool in = side + kSides * q < chunks && o < E.d_out;
        cs[q] = in && E.sw ? E.sw[o] : 1.f;
        cb[q] = in && E.bias ? E.bias[o] : 0.f;
      }
      if (add && side == 0 && chunks > 0 && t < E.N) {
        const uint32_t esize = kY16 ? 2 : 4;
        prefetch_l2_bulk(static_cast<const uint8_t*>(E.res) + (t * E.d_out + n0) * esize,
                         (uint32_t)min(BN, E.d_out - n0) * esize);
      }
      // a chunk of 32 columns from its sums to y
      auto finish = [&](int c, float (&v)[32]) {
        const int col = n0 + c * 32;
        if (add && asked == chunk) ask(col, m0);
        if (E.sx && !kPromote) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            v[i] = fmaf(v[i], sx * __shfl_sync(0xffffffffu, cs[0], i), __shfl_sync(0xffffffffu, cb[0], i));
        } else if (E.bias) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] += __shfl_sync(0xffffffffu, cb[0], i);
        }
#pragma unroll
        for (int q = 0; q < kMine - 1; ++q) cs[q] = cs[q + 1], cb[q] = cb[q + 1];
        apply_act(v, E.act);
        if (E.tma_y) {
          auto piece = [&](int i) { return set + (i >> 2) * kBox + swz_offset((uint32_t)lane, (uint32_t)i & 3u, 64); };
          if (add) {
            if (!__all_sync(0xffffffffu, mbar_wait(&ctrl->res_full[warp], (uint32_t)chunk & 1u))) {
              ok = false;
              return;
            }
            uint4 q[4 * kParts];
#pragma unroll
            for (int i = 0; i < 4 * kParts; ++i) q[i] = *reinterpret_cast<const uint4*>(piece(i));
#pragma unroll
            for (int i = 0; i < 4 * kParts; ++i) {
              const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if constexpr (kY16) {
                  v[8 * i + 2 * j] += __uint_as_float(w[j] << 16);
                  v[8 * i + 2 * j + 1] += __uint_as_float(w[j] & 0xffff0000u);
                } else {
                  v[4 * i + j] += __uint_as_float(w[j]);
                }
              }
            }
          } else {
            if (lane == 0) bulk_wait_read<0>();  // the last store has read the boxes
            __syncwarp();
          }
#pragma unroll
          for (int i = 0; i < 4 * kParts; ++i) {
            uint4 q;
            if constexpr (kY16)
              q = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                             pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
            else
              q = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                             __float_as_uint(v[4 * i + 3]));
            *reinterpret_cast<uint4*>(piece(i)) = q;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            for (int q = 0; q < kParts && col + q * 16 < E.d_out; ++q)
              tma_store_2d(&map_y, smem_u32(set + q * kBox), col + q * 16, m0);
            bulk_commit();
          }
          ++chunk;
        } else {
          // rows that are not 16-byte aligned: turned in shared memory, written a row at a time
          float* turned = reinterpret_cast<float*>(sm + P.off_stage + (size_t)warp * kTurn);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 32; ++i) turned[lane * 32 + (i ^ lane)] = v[i];
          __syncwarp();
          for (int q = 0; q < 32 && m0 + q < E.N; ++q) {
            if (col + lane >= E.d_out) continue;
            const int64_t at = ((int64_t)m0 + q) * E.d_out + col + lane;
            float o = turned[q * 32 + (lane ^ q)];
            if constexpr (kY16) {
              if (E.res) o += to_float(static_cast<const __nv_bfloat16*>(E.res)[at]);
              static_cast<__nv_bfloat16*>(E.y)[at] = __float2bfloat16_rn(o);
            } else {
              if (E.res) o += static_cast<const float*>(E.res)[at];
              static_cast<float*>(E.y)[at] = o;
            }
          }
        }
      };
      auto wait_sums = [&]() {  // the next buffer of sums
        ok = __all_sync(0xffffffffu, mbar_wait_spin(&ctrl->tfull[tc & 1], (uint32_t)(tc >> 1) & 1u, abort));
        tc_fence_after();
        return tmem + lanes + (uint32_t)((tc & 1) * (P.tmem_cols / 2));
      };
      auto free_sums = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(dsmem_addr(smem_u32(&ctrl->tempty[tc & 1]), 0));
        ++tc;
      };
      if (add && side < chunks) ask(n0 + side * 32, m0);
      if constexpr (kPromote) {
        float acc[3][32];
        for (int first = 0; first < all; first = span_end(first)) {
          const uint32_t base = wait_sums();
          if (!ok) break;
#pragma unroll
          for (int q = 0; q < 3; ++q) {
            if (side + kSides * q >= chunks) continue;
            uint32_t r[32];
            tmem_ld32_start(base + (uint32_t)((side + kSides * q) * 32), r);
            tmem_ld_wait(r);
            if (first) {
#pragma unroll
              for (int i = 0; i < 32; ++i) acc[q][i] += __uint_as_float(r[i]);
            } else if (kFp8) {  // the scales belong to the product, not to the update
#pragma unroll
              for (int i = 0; i < 32; ++i) acc[q][i] = __uint_as_float(r[i]) * (sx * __shfl_sync(0xffffffffu, cs[q], i));
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) acc[q][i] = __uint_as_float(r[i]);
            }
          }
          free_sums();
        }
        if (!ok) break;
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          if (side + kSides * q >= chunks) continue;
          if (ok) finish(side + kSides * q, acc[q]);
        }
      } else {
        const uint32_t base = wait_sums();
        if (!ok) break;
        uint32_t r[32];
        if (side < chunks) tmem_ld32_start(base + (uint32_t)(side * 32), r);
        for (int c = side; c < chunks && ok; c += kSides) {
          float v[32];
          tmem_ld_wait(r);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
          if (c + kSides < chunks) tmem_ld32_start(base + (uint32_t)((c + kSides) * 32), r);
          finish(c, v);
        }
        free_sums();
      }
    }
    if (!ok) {
      if (asked > chunk) mbar_wait(&ctrl->res_full[warp], (uint32_t)chunk & 1u);
      *abort = 1;
      if (lane == 0) report(err_word, MOLORA_DEV_WAIT_TIMEOUT);
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  if (warp == kWarps + 1 && lane == 0) mbar_wait(&ctrl->done, 0);
  __syncthreads();
  cluster_sync();  // neither CTA leaves, nor frees its TMEM, while the other may still signal or use it
  if (warp == kWarps + 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, P.tmem_cols);
  }
}

// ---------------------------------------------------------------------------------------------
struct SkinnyPlan {
  int BN;                // tokens per tile (MMA N)
  int C;                 // CTAs of a cluster: d_in split C ways
  int S;
  int nkb;
  int32_t o_tiles, t_tiles;
  uint32_t stage_bytes, off_b, off_ctrl, tmem_cols, smem;
};

// J: columns of sums a thread keeps, 32 J tokens a tile (few: small code, which a launch fetches cold).
template <bool kFp8, int J>
__global__ void __launch_bounds__(kThreads, 1)
    linear_skinny_kernel(const Epi E, const SkinnyPlan P, int32_t* err_word, const __grid_constant__ CUtensorMap map_x,
                         const __grid_constant__ CUtensorMap map_w) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  LCtrl* ctrl = reinterpret_cast<LCtrl*>(sm + P.off_ctrl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int BN = P.BN, S = P.S, C = P.C;
  const int rank = (int)cluster_ctarank();
  const unsigned tile = blockIdx.x / (unsigned)C;
  const int32_t o0 = (int32_t)(tile % (unsigned)P.o_tiles) * kRows, t0 = (int32_t)(tile / (unsigned)P.o_tiles) * BN;
  const int kb0 = (int)((int64_t)P.nkb * rank / C), kb1 = (int)((int64_t)P.nkb * (rank + 1) / C);
  const int tokens = (int)min((int64_t)BN, E.N - t0);
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
    for (int c = 0; c < 2; ++c) {
      mbar_init(&ctrl->tfull[c], 1);
      mbar_init(&ctrl->tempty[c], kEpiWarps);
    }
    mbar_init(&ctrl->done, 1);
    ctrl->abort = 0;
    mbar_fence_init();
    tma_prefetch_desc(&map_x);
    tma_prefetch_desc(&map_w);
  }
  pdl_wait();
  __syncthreads();
  // only now, with this CTA's TMEM held, may the next kernel's CTAs come and ask for theirs
  pdl_launch_dependents();
  tc_fence_after();
  const uint32_t tmem = ctrl->tmem_base;
  const int spans = kFp8 ? 1 : (kb1 - kb0 + kSpan - 1) / kSpan;
  TileSums<J> sums;
  sums.zero();
  bool have = true;

  if (warp == 8) {
    if (elect_one()) {
      const int elems = kFp8 ? 128 : 64;
      int issued = 0, s = 0;
      uint32_t phase = 1;  // the first use of a stage finds it empty
      for (int kb = kb0; kb < kb1; ++kb, ++issued) {
        if (issued >= S && !mbar_wait_spin(&ctrl->empty[s], phase, abort)) break;
        uint8_t* st = sm + (size_t)s * P.stage_bytes;
        mbar_arrive_expect_tx(&ctrl->full[s], P.stage_bytes);
        tma_load_2d(smem_u32(st), &map_w, kb * elems, o0, &ctrl->full[s]);
        tma_load_2d(smem_u32(st + P.off_b), &map_x, kb * elems, t0, &ctrl->full[s]);
        if (++s == S) s = 0, phase ^= 1;
      }
      for (int q = 0; q < S && q < issued; ++q) mbar_wait(&ctrl->full[q], (uint32_t)((issued - 1 - q) / S) & 1u);
    }
    __syncwarp();
  } else if (warp == 9) {
    if (elect_one()) {
      const uint32_t idesc = kFp8 ? idesc_e4m3_f32(kRows, (uint32_t)BN) : idesc_bf16_f32(kRows, (uint32_t)BN, false, false);
      const uint64_t da = smem_desc(smem_u32(sm), 16, 1024, kSwizzle128B);
      const uint64_t db = smem_desc(smem_u32(sm + P.off_b), 16, 1024, kSwizzle128B);
      const uint32_t a_lo = (uint32_t)da, b_lo = (uint32_t)db, desc_hi = (uint32_t)(da >> 32);
      bool ok = true;
      int s = 0;
      uint32_t phase = 0;
      for (int c = 0; c < spans && ok; ++c) {
        const int first = kb0 + (kFp8 ? 0 : c * kSpan), last = kFp8 ? kb1 : min(first + kSpan, kb1);
        if (c >= 2 && !mbar_wait_spin(&ctrl->tempty[c & 1], (uint32_t)((c >> 1) - 1) & 1u, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)((c & 1) * BN);
        for (int kb = first; kb < last; ++kb) {
          if (!mbar_wait_spin(&ctrl->full[s], phase, abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t at = (uint32_t)s * (P.stage_bytes >> 4);
          umma_stage<false, kFp8>(d, a_lo + at, b_lo + at, desc_hi, desc_hi, idesc, kb != first);
          umma_commit(&ctrl->empty[s]);
          if (++s == S) s = 0, phase ^= 1;
        }
        if (ok) umma_commit(&ctrl->tfull[c & 1]);
      }
      if (!ok) report(err_word, MOLORA_DEV_WAIT_TIMEOUT);
      umma_commit(&ctrl->done);
    }
    __syncwarp();
  } else {
    for (int c = 0; c < spans && have; ++c) have = sums.take(ctrl, c, tmem, BN, tokens);
  }
  // every MMA is done; the TMA warp has seen every load land
  have = mbar_wait(&ctrl->done, 0) && have && !*abort;
  __syncthreads();
  split_epilogue<J >= 2 ? 4 : 2, false>(E, sums, have, sm, C, rank, o0, t0, tokens, err_word,
                                        [](int64_t, int32_t) { return 0.f; });
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, P.tmem_cols);
  }
}

// ---------------------------------------------------------------------------------------------
struct AnyPlan {
  int BN;                // tokens per tile (MMA N)
  int C;                 // CTAs of a cluster: d_in split C ways
  int S;
  int nkb;               // K blocks of 64 elements
  int32_t o_tiles;
  bool grid;             // both arrays start on 16-byte boundaries
  uint32_t plane, stage_bytes, off_ctrl, tmem_cols, smem;
};

namespace {

// 8 consecutive elements of a row, fetched before they are needed and then cut into bf16 planes (16 bytes
// each) whose sum they are: one plane for bf16 and e4m3, whose values bf16 holds, three for fp32, by
// cutting its 24 bits into 8 + 8 + 8.  `at` is the first element's place in the array, `left` how many
// there are in the row (the others are 0).  kVec: rows start on 16-byte boundaries.  Else, with `grid`
// (the array starts on one), the elements are read in whole pieces of that grid, the array's last ones
// excepted (`total` elements).  load_inside reads from the grid's boundary `sh` elements before the first
// one; two pieces' worth from there, and four elements, have to be the array's.
template <typename T, bool kVec>
struct Piece;

template <bool kVec>
struct Piece<float, kVec> {
  static constexpr int kPlanes = 3;
  static constexpr int kGrid = 4;  // elements of a 16-byte piece
  uint4 w[kVec ? 2 : 3];
  int shift;
  __device__ __forceinline__ void load_inside(const float* p, int sh) {
    shift = sh;
    const uint4* q = reinterpret_cast<const uint4*>(p);
    w[0] = q[0], w[1] = q[1];
    if (!kVec) w[kVec ? 0 : 2] = q[2];
  }
  __device__ __forceinline__ void load(const float* p, int64_t at, int left, int64_t total, bool grid) {
    shift = 0;
    const int64_t base = at & ~int64_t(3);
    if (kVec && left >= 8) {
      const uint4* q = reinterpret_cast<const uint4*>(p + at);
      w[0] = q[0], w[1] = q[1];
    } else if (!kVec && grid && base + 12 <= total && left > 0) {
      shift = (int)(at - base);
      const uint4* q = reinterpret_cast<const uint4*>(p + base);
      w[0] = q[0], w[1] = q[1];
      if (shift) w[kVec ? 0 : 2] = q[2];
    } else {
      uint32_t u[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = j < left ? __float_as_uint(p[at + j]) : 0u;
      w[0] = make_uint4(u[0], u[1], u[2], u[3]), w[1] = make_uint4(u[4], u[5], u[6], u[7]);
    }
  }
  __device__ __forceinline__ void cut(int left, uint4 (&out)[3]) const {
    const uint4 last = w[kVec ? 1 : 2];
    uint32_t e[12] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w, last.x, last.y, last.z, last.w};
    if (!kVec) {
      if (shift & 2)
#pragma unroll
        for (int j = 0; j < 10; ++j) e[j] = e[j + 2];
      if (shift & 1)
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = e[j + 1];
      if (left < 8)
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = j < left ? e[j] : 0u;
    }
    uint32_t pl[3][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t part[3][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t f = e[2 * j + h];
        part[0][h] = f & 0xffff0000u;
        const float r = __uint_as_float(f) - __uint_as_float(part[0][h]);
        part[1][h] = __float_as_uint(r) & 0xffff0000u;
        part[2][h] = __float_as_uint(r - __uint_as_float(part[1][h]));
      }
#pragma unroll
      for (int k = 0; k < 3; ++k) pl[k][j] = __byte_perm(part[k][0], part[k][1], 0x7632);
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) out[k] = make_uint4(pl[k][0], pl[k][1], pl[k][2], pl[k][3]);
  }
};

template <bool kVec>
struct Piece<__nv_bfloat16, kVec> {
  static constexpr int kPlanes = 1;
  static constexpr int kGrid = 8;
  uint4 w[2];
  int shift;
  __device__ __forceinline__ void load_inside(const __nv_bfloat16* p, int sh) {
    shift = sh;
    const uint4* q = reinterpret_cast<const uint4*>(p);
    w[0] = q[0], w[1] = q[1];
  }
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int64_t at, int left, int64_t total, bool grid) {
    shift = 0;
    const int64_t base = at & ~int64_t(7);
    if (grid && base + 16 <= total && left > 0) {
      shift = (int)(at - base);
      const uint4* q = reinterpret_cast<const uint4*>(p + base);
      w[0] = q[0];
      if (shift) w[1] = q[1];
    } else {
      uint32_t u[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = j < left ? (uint32_t)__bfloat16_as_ushort(p[at + j]) : 0u;
      w[0] = make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
    }
  }
  __device__ __forceinline__ void cut(int left, uint4 (&out)[1]) const {
    uint32_t e[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
    if (shift & 4)
#pragma unroll
      for (int j = 0; j < 4; ++j) e[j] = e[j + 2];
    if (shift & 4) e[4] = e[6], e[5] = e[7];
    if (shift & 2)
#pragma unroll
      for (int j = 0; j < 5; ++j) e[j] = e[j + 1];
    if (shift & 1)
#pragma unroll
      for (int j = 0; j < 4; ++j) e[j] = __funnelshift_r(e[j], e[j + 1], 16);
    if (left < 8) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (2 * j >= left) e[j] = 0u;
        if (2 * j + 1 >= left) e[j] &= 0xffffu;
      }
    }
    out[0] = make_uint4(e[0], e[1], e[2], e[3]);
  }
};

template <bool kVec>
struct Piece<__nv_fp8_e4m3, kVec> {
  static constexpr int kPlanes = 1;
  static constexpr int kGrid = 4;  // (4-byte pieces)
  uint32_t w[3];
  int shift;
  __device__ __forceinline__ void load_inside(const __nv_fp8_e4m3* p, int sh) {
    shift = sh * 8;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
    w[0] = q[0], w[1] = q[1], w[2] = q[2];
  }
  __device__ __forceinline__ void load(const __nv_fp8_e4m3* p, int64_t at, int left, int64_t total, bool grid) {
    shift = 0;
    const int64_t base = at & ~int64_t(3);
    const uint8_t* bytes = reinterpret_cast<const uint8_t*>(p);
    if (grid && base + 12 <= total && left > 0) {
      shift = (int)(at - base) * 8;
      const uint32_t* q = reinterpret_cast<const uint32_t*>(bytes + base);
      w[0] = q[0], w[1] = q[1], w[2] = q[2];
    } else {
      w[0] = w[1] = w[2] = 0u;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < left) w[j >> 2] |= (uint32_t)bytes[at + j] << (8 * (j & 3));
    }
  }
  __device__ __forceinline__ void cut(int left, uint4 (&out)[1]) const {
    const uint32_t e[2] = {__funnelshift_r(w[0], w[1], shift), __funnelshift_r(w[1], w[2], shift)};
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        __nv_fp8_e4m3 v;
        v.__x = (__nv_fp8_storage_t)((e[j >> 1] >> (16 * (j & 1) + 8 * h)) & 0xffu);
        f[h] = 2 * j + h < left ? static_cast<float>(v) : 0.f;
      }
      b[j] = pack_bf16(f[0], f[1]);
    }
    out[0] = make_uint4(b[0], b[1], b[2], b[3]);
  }
};

}  // namespace

// Operands that TMA cannot fetch or the tensor cores do not multiply: rows that start anywhere, and fp32.
// The orientation and the split of linear_skinny_kernel; 15 warps fetch both operands and lay them out
// as bf16 planes in the swizzled stages.  fp32 is three planes, x = x1 + x2 + x3 exactly, and
//   x w = x1 w1 + x1 w2 + x2 w1 + x2 w2 + x1 w3 + x3 w1 + (terms below 2^-21 of |x w|, 2^-24 of it on average)
// which is six bf16 products with fp32 sums: an fp32 product at a sixth of the bf16 rate, four times the CUDA
// cores'.  All but the first are 2^-7 of it and less, and sum apart: their long chain's drift is theirs.  The second
// plane of an infinity is NaN (inf - inf), as a NaN's is: every output that reads one comes out NaN, and outputs that
// are NaN, no others, are summed again on the CUDA cores, so that no token's bits or time depend on its neighbours'.
//
// Bound by the threads that cut the operands: 15 warps, with their next pieces on the way while a stage is
// written and handed over.  1024 x 4096 x 4096 fp32 324 us (106 TFLOP/s, 577 us for the library's fp32 product);
// of 5100 cycles a K block, the MMAs are 1500 and the operands' way from L2 1000.
template <typename T, bool kVec, int J>
__global__ void __launch_bounds__(kAnyThreads, 1)
    linear_any_kernel(const Epi E, const AnyPlan P, const T* __restrict__ x, const T* __restrict__ W, int32_t d_in,
                      int32_t* err_word) {
  constexpr int kPlanes = Piece<T, kVec>::kPlanes;
  constexpr int kPieces = ((kRows + 32 * J) * 8 + kCutters - 1) / kCutters;  // of a stage, a thread
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  LCtrl* ctrl = reinterpret_cast<LCtrl*>(sm + P.off_ctrl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int BN = P.BN, S = P.S, C = P.C;
  const int rank = (int)cluster_ctarank();
  const unsigned tile = blockIdx.x / (unsigned)C;
  const int32_t o0 = (int32_t)(tile % (unsigned)P.o_tiles) * kRows;
  const int64_t t0 = (int64_t)(tile / (unsigned)P.o_tiles) * BN;
  const int kb0 = (int)((int64_t)P.nkb * rank / C), kb1 = (int)((int64_t)P.nkb * (rank + 1) / C);
  const int tokens = (int)min((int64_t)BN, E.N - t0);
  volatile int32_t* abort = &ctrl->abort;

  if (warp == 15) {
    tmem_alloc(&ctrl->tmem_base, P.tmem_cols);
    tmem_relinquish();
  }
  if (warp == 14 && lane == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&ctrl->full[s], kCutters / 32);
      mbar_init(&ctrl->empty[s], 1);
    }
    for (int c = 0; c < 2; ++c) {
      mbar_init(&ctrl->tfull[c], 1);
      mbar_init(&ctrl->tempty[c], kEpiWarps);
    }
    mbar_init(&ctrl->done, 1);
    ctrl->abort = 0;
    mbar_fence_init();
  }
  pdl_wait();
  __syncthreads();
  pdl_launch_dependents();  // with this CTA's TMEM held (see linear_tc_kernel)
  tc_fence_after();
  const uint32_t tmem = ctrl->tmem_base;
  const int spans = (kb1 - kb0 + kSpan - 1) / kSpan;
  TileSums<J> sums;
  sums.zero();
  bool have = true;

  if (warp < 15) {
    int taken = 0;
    Piece<T, kVec> piece[kPieces];  // of the rows of W, then x, 8 pieces each
    // rows past the last one are read as the last one: what comes of them is not stored
    const T* src[kPieces];  // its boundary in the grid
    uint32_t shifts = 0;    // 4 bits a piece: the elements between the boundary and the piece's first one
    auto row_of = [&](int j) { return (tid + j * kCutters) >> 3; };
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int row = row_of(j);
      const int64_t at = (row < kRows ? (int64_t)min(o0 + row, E.d_out - 1) : t0 + min(row - kRows, tokens - 1)) * d_in +
                         ((tid + j * kCutters) & 7) * 8;
      const uint32_t sh = kVec ? 0u : (uint32_t)(at & (Piece<T, kVec>::kGrid - 1));
      shifts |= sh << (4 * j);
      src[j] = (row < kRows ? W : x) + (at - sh);
    }
    // a block of which every piece can be read from its boundary without leaving the row
    auto inside = [&](int kb) { return (kVec || P.grid) && (int64_t)kb * 64 + 56 + (kVec ? 8 : 16) <= d_in; };
    auto left_of = [&](int j, int kb) { return d_in - kb * 64 - ((tid + j * kCutters) & 7) * 8; };
    auto fetch = [&](int kb) {
      if (inside(kb)) {
#pragma unroll
        for (int j = 0; j < kPieces; ++j)
          if (row_of(j) < kRows + BN) piece[j].load_inside(src[j] + (int64_t)kb * 64, (int)(shifts >> (4 * j)) & 15);
      } else {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
          const bool is_w = row_of(j) < kRows;
          if (row_of(j) < kRows + BN)
            piece[j].load(is_w ? W : x, (src[j] - (is_w ? W : x)) + ((shifts >> (4 * j)) & 15) + (int64_t)kb * 64,
                          left_of(j, kb), is_w ? (int64_t)E.d_out * d_in : E.N * d_in, P.grid);
        }
      }
    };
    fetch(kb0);
    for (int kb = kb0; kb < kb1; ++kb) {
      const int i = kb - kb0, s = i % S, use = i / S;
      if (use > 0 && !__all_sync(0xffffffffu, mbar_wait_spin(&ctrl->empty[s], (uint32_t)(use - 1) & 1u, abort))) break;
      uint8_t* st = sm + (size_t)s * P.stage_bytes;
      auto write = [&](bool whole) {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
          if (row_of(j) >= kRows + BN) continue;
          uint4 p[kPlanes];
          piece[j].cut(whole ? 8 : left_of(j, kb), p);
          const uint32_t at = sw128_offset((uint32_t)row_of(j), (uint32_t)(tid + j * kCutters) & 7u);
#pragma unroll
          for (int k = 0; k < kPlanes; ++k) *reinterpret_cast<uint4*>(st + k * P.plane + at) = p[k];
        }
      };
      if (inside(kb))
        write(true);
      else
        write(false);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctrl->full[s]);
      if (kb + 1 < kb1) fetch(kb + 1);
      // the last span's sums, with this one's first stages already filled
      if (warp < kEpiWarps && i >= kSpan && i % kSpan == 2 && have) have = sums.take(ctrl, taken++, tmem, BN, tokens);
    }
    while (warp < kEpiWarps && taken < spans && have) have = sums.take(ctrl, taken++, tmem, BN, tokens);
  } else {
    if (elect_one()) {
      const uint32_t idesc = idesc_bf16_f32(kRows, (uint32_t)BN, false, false);
      const uint32_t first = smem_u32(sm);
      const uint64_t da = smem_desc(first, 16, 1024, kSwizzle128B);
      const uint32_t a_lo = (uint32_t)da, b_lo = a_lo + ((uint32_t)kRows * kRowBytes >> 4), desc_hi = (uint32_t)(da >> 32);
      bool ok = true;
      const uint32_t step = P.plane >> 4, cross = tmem + 2u * (uint32_t)BN;
      int s = 0;
      uint32_t phase = 0;
      for (int c = 0; c < spans && ok; ++c) {
        const int from = kb0 + c * kSpan, last = min(from + kSpan, kb1);
        if (c >= 2 && !mbar_wait_spin(&ctrl->tempty[c & 1], (uint32_t)((c >> 1) - 1) & 1u, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)((c & 1) * BN);
        for (int kb = from; kb < last; ++kb) {
          if (!mbar_wait_spin(&ctrl->full[s], phase, abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a1 = a_lo + (uint32_t)s * (P.stage_bytes >> 4), b1 = a1 + (b_lo - a_lo);
          umma_stage<false, false>(d, a1, b1, desc_hi, desc_hi, idesc, kb != from);
          if (kPlanes == 3) {
            const uint32_t a2 = a1 + step, a3 = a2 + step, b2 = b1 + step, b3 = b2 + step;
            umma_stage<false, false>(cross, a1, b2, desc_hi, desc_hi, idesc, kb != kb0);
            umma_stage<false, false>(cross, a2, b1, desc_hi, desc_hi, idesc, 1);
            umma_stage<false, false>(cross, a2, b2, desc_hi, desc_hi, idesc, 1);
            umma_stage<false, false>(cross, a1, b3, desc_hi, desc_hi, idesc, 1);
            umma_stage<false, false>(cross, a3, b1, desc_hi, desc_hi, idesc, 1);
          }
          umma_commit(&ctrl->empty[s]);
          if (++s == S) s = 0, phase ^= 1;
        }
        if (ok) umma_commit(&ctrl->tfull[c & 1]);
      }
      if (!ok) report(err_word, MOLORA_DEV_WAIT_TIMEOUT);
      umma_commit(&ctrl->done);
    }
    __syncwarp();
  }
  have = mbar_wait(&ctrl->done, 0) && have && !*abort;
  if (kPlanes == 3 && warp < kEpiWarps && __all_sync(0xffffffffu, have)) {
    tc_fence_after();
    sums.add(tmem + 2u * (uint32_t)BN, tokens);
    tc_fence_before();
  }
  __syncthreads();
  split_epilogue<2, kPlanes == 3>(E, sums, have, sm, C, rank, o0, t0, tokens, err_word, [&](int64_t t, int32_t o) {
    float v = 0.f;
    for (int i = 0; i < d_in; ++i) v = fmaf(to_float(x[t * d_in + i]), to_float(W[(int64_t)o * d_in + i]), v);
    return v;
  });
  if (warp == 15) {
    tc_fence_after();
    tmem_dealloc(tmem, P.tmem_cols);
  }
}

// ---------------------------------------------------------------------------------------------
constexpr int kFewWarps = 4;

// A token or a few: R outputs a warp on the CUDA cores, W's rows straight into registers, U loads of 16 bytes
// (kVec: rows on 16-byte boundaries) or of an element of each row in flight a lane; x comes from L1.  Bound by
// those loads (one token, 4096 x 4096 fp32 from HBM 12.0 us, 5600 GB/s) and, with each further token, by the
// instructions that multiply.
template <typename T, bool kVec, int NT, int R>
__global__ void __launch_bounds__(kFewWarps * 32)
    linear_few_kernel(const Epi E, const T* __restrict__ x, const T* __restrict__ W, int32_t d_in) {
  constexpr uint32_t n = kVec ? 16 / sizeof(T) : 1;
  constexpr int U = kVec ? 4 : 8;
  struct alignas(kVec ? 16 : sizeof(T)) Run {
    T v[n];
  };
  const int lane = threadIdx.x & 31;
  const int64_t o0 = ((int64_t)blockIdx.x * kFewWarps + (threadIdx.x >> 5)) * R;
  pdl_wait();
  pdl_launch_dependents();
  if (o0 >= E.d_out) return;
  const T* rows[R];
#pragma unroll
  for (int q = 0; q < R; ++q) rows[q] = W + min(o0 + q, (int64_t)E.d_out - 1) * d_in;
  // past the last token the last one again: a test in the loop would keep its loads from running ahead
  const T* tokens[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) tokens[t] = x + (NT > 2 ? min((int64_t)t, E.N - 1) : (int64_t)t) * d_in;
  float sum[R][NT] = {};
  for (uint32_t i = lane * n; i < (uint32_t)d_in; i += 32 * n * U) {
    Run w[U][R];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int q = 0; q < R; ++q)
        if (i + 32 * n * u < (uint32_t)d_in) w[u][q] = *reinterpret_cast<const Run*>(rows[q] + i + 32 * n * u);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + 32 * n * u >= (uint32_t)d_in) continue;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const Run a = *reinterpret_cast<const Run*>(tokens[t] + i + 32 * n * u);
#pragma unroll
        for (int j = 0; j < (int)n; ++j) {
          const float v = to_float(a.v[j]);
#pragma unroll
          for (int q = 0; q < R; ++q) sum[q][t] = fmaf(v, to_float(w[u][q].v[j]), sum[q][t]);
        }
      }
    }
  }
  float v = 0.f;  // of lane q * NT + t
#pragma unroll
  for (int q = 0; q < R; ++q)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int off = 16; off; off >>= 1) sum[q][t] += __shfl_xor_sync(0xffffffffu, sum[q][t], off);
      if (lane == q * NT + t) v = sum[q][t];
    }
  const int64_t o = o0 + lane / NT, t = lane % NT, at = t * E.d_out + o;
  if (lane >= R * NT || o >= E.d_out || t >= E.N) return;
  if (E.sx) v *= E.sx[t] * E.sw[o];
  if (E.bias) v += E.bias[o];
  v = activate(v, E.act);
  if (E.y_bf16) {
    if (E.res) v += to_float(static_cast<const __nv_bfloat16*>(E.res)[at]);
    static_cast<__nv_bfloat16*>(E.y)[at] = __float2bfloat16_rn(v);
  } else {
    if (E.res) v += static_cast<const float*>(E.res)[at];
    static_cast<float*>(E.y)[at] = v;
  }
}

// ---------------------------------------------------------------------------------------------
namespace {

PFN_cuTensorMapEncodeTiled_v12000 linear_encoder() {
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

}  // namespace

bool linear_map(CUtensorMap* m, CUtensorMapDataType type, uint32_t esize, const void* base, uint64_t rows, uint64_t cols,
                uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swz) {
  auto enc = linear_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * esize};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t es[2] = {1, 1};
  return enc(m, type, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool linear_map_3d(CUtensorMap* m, CUtensorMapDataType type, const void* base, const uint64_t (&size)[3],
                   const uint64_t (&step)[2], const uint32_t (&box)[3], CUtensorMapSwizzle swz) {
  auto enc = linear_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {size[0], size[1], size[2]};
  cuuint64_t strides[2] = {step[0], step[1]};
  cuuint32_t boxes[3] = {box[0], box[1], box[2]};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, type, 3, const_cast<void*>(base), dims, strides, boxes, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

bool operand_map(CUtensorMap* m, const LinearArgs& a, const void* base, int64_t rows, uint32_t box_rows) {
  const bool fp8 = a.dtype == MOLORA_E4M3;
  return linear_map(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, fp8 ? 1 : 2, base,
                    (uint64_t)rows, (uint64_t)a.d_in, fp8 ? 128 : 64, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

int ask_resident(int C) {
  static std::atomic<uint64_t> allowed;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(C * num_sms()));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kMaxSmem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)C;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (allow_smem(linear_skinny_kernel<false, 1>, allowed, kMaxSmem) == cudaSuccess &&
      cudaOccupancyMaxActiveClusters(&n, linear_skinny_kernel<false, 1>, &cfg) == cudaSuccess && n > 0)
    return n;
  cudaGetLastError();
  return num_sms() / C * 3 / 4;
}

}  // namespace

Resident resident_clusters() {
  static std::atomic<int> known[64][9];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) dev = -1;
  Resident r = {};
  r.of[1] = num_sms();
  for (int C = 2; C <= 8; ++C) {
    r.of[C] = dev >= 0 ? known[dev][C].load(std::memory_order_relaxed) : 0;
    if (r.of[C]) continue;
    r.of[C] = ask_resident(C);
    if (dev >= 0) known[dev][C].store(r.of[C], std::memory_order_relaxed);
  }
  return r;
}

namespace {

Epi epilogue_of(const LinearArgs& a) {
  Epi e = {a.x_scale, a.w_scale, a.bias, a.residual, a.y, a.N, a.d_out, a.act, a.y_bf16, false};
  e.tma_y = a.d_out % (a.y_bf16 ? 8 : 4) == 0 && aligned(a.y, 16) && aligned(a.residual, 16);
  return e;
}

int k_blocks(const LinearArgs& a) {
  return (int)(((int64_t)a.d_in * (a.dtype == MOLORA_E4M3 ? 1 : 2) + kRowBytes - 1) / kRowBytes);
}

cudaError_t launch_tc(const LinearArgs& a, int BN, bool promote, const LinearUpdate* u, cudaStream_t stream) {
  const bool fp8 = a.dtype == MOLORA_E4M3;
  Epi e = epilogue_of(a);
  TcPlan p = {};
  p.BN = BN;
  p.nkb = k_blocks(a);
  p.nkg = u ? (u->KR + 63) / 64 : 0;
  p.m_tiles = (a.N + 2 * kRows - 1) / (2 * kRows);
  p.n_tiles = (a.d_out + BN - 1) / BN;
  p.tiles = p.m_tiles * p.n_tiles;
  p.group = 8;
  p.off_b = kRows * kRowBytes;
  p.stage_bytes = p.off_b + (uint32_t)(BN / 2) * kRowBytes;
  p.tmem_cols = tmem_columns(2 * (uint32_t)(BN <= 64 ? 64 : BN <= 128 ? 128 : 256));
  CUtensorMap mx, mw, my = {}, mr = {};
  auto rows_map = [&](CUtensorMap* m, const void* base) {
    return linear_map(m, a.y_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.y_bf16 ? 2 : 4, base,
                      (uint64_t)a.N, (uint64_t)a.d_out, a.y_bf16 ? 32 : 16, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  };
  if (e.tma_y && (!rows_map(&my, a.y) || (a.residual && !rows_map(&mr, a.residual)))) e.tma_y = false;
  const uint32_t boxes = 4 * tc_sides(promote) * (e.tma_y && a.y_bf16 ? kBox : kTurn);
  const size_t fixed = boxes + sizeof(LCtrl) + kSmemSlack;
  p.S = (int)((kMaxSmem - fixed) / p.stage_bytes);
  if (p.S > kMaxStages) p.S = kMaxStages;
  p.off_stage = (uint32_t)p.S * p.stage_bytes;
  p.off_ctrl = p.off_stage + boxes;
  // one CTA an SM, alone: an allocation of TMEM never waits for another CTA's, which could in turn
  // be waiting for a partner that this kernel's other CTAs keep out
  p.smem = kMaxSmem;
  if (!operand_map(&mx, a, a.x, a.N, kRows) || !operand_map(&mw, a, a.W, a.d_out, (uint32_t)(BN / 2)))
    return cudaErrorNotSupported;
  const auto BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap ghi = {}, glo = {}, mb = {};
  if (u && (!linear_map(&ghi, BF, 2, u->g_hi, (uint64_t)a.N, (uint64_t)u->KR, 64, kRows, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !linear_map(&glo, BF, 2, u->g_lo, (uint64_t)a.N, (uint64_t)u->KR, 64, kRows, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !linear_map(&mb, BF, 2, u->B, (uint64_t)u->KR, (uint64_t)a.d_out, 16, 64, CU_TENSOR_MAP_SWIZZLE_32B)))
    return cudaErrorNotSupported;
  const bool y16 = a.y_bf16;
  auto kernel = fp8 ? promote ? y16 ? linear_tc_kernel<true, true, true> : linear_tc_kernel<true, true, false>
                              : y16 ? linear_tc_kernel<true, false, true> : linear_tc_kernel<true, false, false>
                : promote ? linear_tc_kernel<false, true, false>  // (for fp32 y only)
                          : y16 ? linear_tc_kernel<false, false, true> : linear_tc_kernel<false, false, false>;
  static std::atomic<uint64_t> allowed[8];
  const cudaError_t set = allow_smem(kernel, allowed[4 * fp8 + 2 * promote + y16], kMaxSmem);
  if (set != cudaSuccess) return set;
  const int64_t most = num_sms() / 2;
  const dim3 grid((unsigned)(2 * (p.tiles < most ? p.tiles : most)));
  return launch_kernel(kernel, grid, dim3(tc_threads(promote)), p.smem, stream, 2, e, p, a.err_word, mx, mw, my, ghi, glo, mb,
                       mr);
}

// Cycles that linear_skinny_kernel takes in tiles of BN tokens, and linear_tc_kernel in tiles of BN outputs, as
// measured on GB300 with 64 to 6144 outputs, d_in 1024 to 4096 and 1 to 4096 tokens (within 20%): what
// a K block takes, a join or a last epilogue that grows with the tile, and the way through.  The split
// product is 7.7 us for 16 tokens of 4096 x 4096, 16.4 for 256 and 23.4 for 512, the pairs' 16.6, 17.1 and 17.5.
int64_t skinny_cycles(const LinearArgs& a, const Resident& r, int BN) {
  const int64_t tiles = (((int64_t)a.d_out + kRows - 1) / kRows) * ((a.N + BN - 1) / BN);
  const int nkb = k_blocks(a), C = split_of(r, tiles, nkb);
  const int64_t waves = (tiles + r.of[C] - 1) / r.of[C];
  return 6500 + waves * ((nkb + C - 1) / C * (420 + BN * 3 / 2) + 48 * BN);
}

int64_t tc_cycles(const LinearArgs& a, const Resident& r, int BN, int blocks) {
  const int64_t m_tiles = (a.N + 2 * kRows - 1) / (2 * kRows);
  const int64_t tiles = m_tiles * ((a.d_out + BN - 1) / BN), waves = (tiles + r.of[2] - 1) / r.of[2];
  return 8000 + waves * blocks * (2 * BN + 90 > 420 ? 2 * BN + 90 : 420);
}

cudaError_t launch_skinny(const LinearArgs& a, const Resident& r, int BN, cudaStream_t stream) {
  const bool fp8 = a.dtype == MOLORA_E4M3;
  const Epi e = epilogue_of(a);
  SkinnyPlan p = {};
  p.BN = BN;
  p.nkb = k_blocks(a);
  p.o_tiles = (a.d_out + kRows - 1) / kRows;
  p.t_tiles = (int32_t)((a.N + p.BN - 1) / p.BN);
  const int64_t tiles = (int64_t)p.o_tiles * p.t_tiles;
  p.C = split_of(r, tiles, p.nkb);
  p.off_b = kRows * kRowBytes;
  p.stage_bytes = p.off_b + (uint32_t)p.BN * kRowBytes;
  p.tmem_cols = tmem_columns(2 * (uint32_t)p.BN);
  const size_t fixed = sizeof(LCtrl) + kSmemSlack;
  const size_t partial = (size_t)p.BN * kRows * sizeof(float);
  const int need = (p.nkb + p.C - 1) / p.C;
  p.S = (int)((kMaxSmem - fixed) / p.stage_bytes);
  if (p.S > kMaxStages) p.S = kMaxStages;
  if (p.S > need) p.S = need;
  size_t ring = (size_t)p.S * p.stage_bytes;
  if (ring < partial) ring = partial;
  p.off_ctrl = (uint32_t)ring;
  p.smem = (uint32_t)(ring + sizeof(LCtrl) + kSmemSlack);
  // 116 KB at least: neither this CTA nor one that takes all of TMEM (those take as much) can then hold
  // columns that the other waits for while it is itself waited for, by its cluster or by the next kernel
  if (p.smem < 116 * 1024) p.smem = 116 * 1024;
  CUtensorMap mx, mw;
  if (!operand_map(&mx, a, a.x, a.N, (uint32_t)p.BN) || !operand_map(&mw, a, a.W, a.d_out, kRows))
    return cudaErrorNotSupported;
  auto go = [&](auto kernel, std::atomic<uint64_t>& allowed) {
    const cudaError_t set = allow_smem(kernel, allowed, kMaxSmem);
    if (set != cudaSuccess) return set;
    return launch_kernel(kernel, dim3((unsigned)(tiles * p.C)), dim3(kThreads), p.smem, stream, p.C, e, p, a.err_word, mx,
                         mw);
  };
  static std::atomic<uint64_t> allowed[8];
  switch (p.BN) {
    case 16:
    case 32:
      return fp8 ? go(linear_skinny_kernel<true, 1>, allowed[0]) : go(linear_skinny_kernel<false, 1>, allowed[1]);
    case 64:
      return fp8 ? go(linear_skinny_kernel<true, 2>, allowed[2]) : go(linear_skinny_kernel<false, 2>, allowed[3]);
    case 128:
      return fp8 ? go(linear_skinny_kernel<true, 4>, allowed[4]) : go(linear_skinny_kernel<false, 4>, allowed[5]);
    default:
      return fp8 ? go(linear_skinny_kernel<true, 8>, allowed[6]) : go(linear_skinny_kernel<false, 8>, allowed[7]);
  }
}

template <typename T, bool kVec>
cudaError_t launch_any(const LinearArgs& a, cudaStream_t stream) {
  const Epi e = epilogue_of(a);
  AnyPlan p = {};
  const int planes = sizeof(T) == 4 ? 3 : 1;
  p.nkb = (int)(((int64_t)a.d_in + 63) / 64);
  p.o_tiles = (int32_t)(((int64_t)a.d_out + kRows - 1) / kRows);
  auto tiles_at = [&](int BN) { return p.o_tiles * ((a.N + BN - 1) / BN); };
  const bool wide = (kVec || planes == 1) && a.N > 64 && tiles_at(128) >= num_sms();  // (unaligned fp32: too many registers)
  p.BN = a.N <= 16 ? 16 : a.N <= 32 ? 32 : wide ? 128 : 64;
  const int64_t tiles = tiles_at(p.BN);
  p.C = split_of(resident_clusters(), tiles, p.nkb);
  p.grid = aligned(a.x, 16) && aligned(a.W, 16);
  p.plane = (uint32_t)(kRows + p.BN) * kRowBytes;
  p.stage_bytes = planes * p.plane;
  p.tmem_cols = tmem_columns((planes == 3 ? 3u : 2u) * (uint32_t)p.BN);
  const size_t fixed = sizeof(LCtrl) + kSmemSlack, partial = (size_t)p.BN * kRows * sizeof(float);
  p.S = (int)((kMaxSmem - fixed) / p.stage_bytes);
  if (p.S > 4) p.S = 4;
  size_t ring = (size_t)p.S * p.stage_bytes;
  if (ring < partial) ring = partial;
  p.off_ctrl = (uint32_t)ring;
  p.smem = (uint32_t)(ring + fixed);
  if (p.smem < 116 * 1024) p.smem = 116 * 1024;  // see launch_skinny
  auto go = [&](auto kernel, std::atomic<uint64_t>& allowed) {
    const cudaError_t set = allow_smem(kernel, allowed, kMaxSmem);
    if (set != cudaSuccess) return set;
    return launch_kernel(kernel, dim3((unsigned)(tiles * p.C)), dim3(kAnyThreads), p.smem, stream, p.C, e, p,
                         static_cast<const T*>(a.x), static_cast<const T*>(a.W), a.d_in, a.err_word);
  };
  static std::atomic<uint64_t> allowed[3];
  if (p.BN <= 32) return go(linear_any_kernel<T, kVec, 1>, allowed[0]);
  if constexpr (kVec || sizeof(T) != 4) {
    if (p.BN == 128) return go(linear_any_kernel<T, kVec, 4>, allowed[2]);
  }
  return go(linear_any_kernel<T, kVec, 2>, allowed[1]);
}

}  // namespace

namespace {

template <typename T, bool kVec, int NT, int R>
cudaError_t launch_few(const LinearArgs& a, cudaStream_t stream) {
  const dim3 grid((unsigned)(((int64_t)a.d_out + kFewWarps * R - 1) / (kFewWarps * R)));
  return launch_kernel(linear_few_kernel<T, kVec, NT, R>, grid, dim3(kFewWarps * 32), 0, stream, 0, epilogue_of(a),
                       static_cast<const T*>(a.x), static_cast<const T*>(a.W), a.d_in);
}

// Whether linear_few_kernel is the faster one, and in which form (us here, on the tensor cores):
//   fp32, up to 4 tokens:  4096 x 4096, 1, 2 and 4 tokens 6.6, 10 and 12, 21; 1024 x 1024 2.3, 2.5 and 3.0, 7.1.
//     For one or two tokens, outputs enough to fill the GPU share x, two a warp (one token of 4096 x 4096 6.6, with
//     one output a warp 8.3; of 1024 x 1024 2.4 and 2.3)
//   rows that start anywhere, two tokens, four of fp32:  4095 x 4096 fp32 8.2, 10 and 17, 26; bf16 8.7 and 12.5, 14;
//     e4m3 8.7 and 12.6, 16; but four tokens of bf16 17, 14
//   bf16 and e4m3, up to four tokens that are 8 KB together, up to 2 MB of W:  1024 x 1024 bf16 2.5, 2.5 and 2.7,
//     4.2; e4m3 2.4 to 2.8, 3.8; one token of 4096 -> 512 bf16 5.4, 5.7; of 4096 -> 4096 e4m3 7.6, 6.5, bf16 7.2, 7.4
//     with W in L2 and 12.3, 9.3 from HBM
// Returns cudaErrorNotSupported where it is not.
cudaError_t try_few(const LinearArgs& a, cudaStream_t stream) {
  using F = float;
  using B = __nv_bfloat16;
  using Q = __nv_fp8_e4m3;
  if (a.N > 4) return cudaErrorNotSupported;
  const int64_t row_bytes = (int64_t)a.d_in * (a.dtype == MOLORA_F32 ? 4 : a.dtype == MOLORA_BF16 ? 2 : 1);
  const bool vec = row_bytes % 16 == 0 && aligned(a.x, 16) && aligned(a.W, 16), wide = a.d_out >= 2048;
  if (a.dtype == MOLORA_F32) {
    if (vec && a.N == 1) return wide ? launch_few<F, true, 1, 2>(a, stream) : launch_few<F, true, 1, 1>(a, stream);
    if (vec && a.N == 2) return wide ? launch_few<F, true, 2, 2>(a, stream) : launch_few<F, true, 2, 1>(a, stream);
    if (vec) return launch_few<F, true, 4, 1>(a, stream);
    if (a.N == 1) return launch_few<F, false, 1, 1>(a, stream);
    return a.N == 2 ? launch_few<F, false, 2, 2>(a, stream) : launch_few<F, false, 4, 2>(a, stream);
  }
  const bool bf16 = a.dtype == MOLORA_BF16;
  if (!vec) {
    if (a.N == 1) return bf16 ? launch_few<B, false, 1, 1>(a, stream) : launch_few<Q, false, 1, 1>(a, stream);
    if (a.N == 2) return bf16 ? launch_few<B, false, 2, 2>(a, stream) : launch_few<Q, false, 2, 2>(a, stream);
    return cudaErrorNotSupported;
  }
  if (row_bytes * a.N > 8192 || row_bytes * a.d_out > 2 << 20) return cudaErrorNotSupported;
  if (a.N == 1) return bf16 ? launch_few<B, true, 1, 1>(a, stream) : launch_few<Q, true, 1, 1>(a, stream);
  if (a.N == 2) return bf16 ? launch_few<B, true, 2, 2>(a, stream) : launch_few<Q, true, 2, 1>(a, stream);
  return bf16 ? launch_few<B, true, 4, 2>(a, stream) : launch_few<Q, true, 4, 1>(a, stream);
}

}  // namespace

// Whether TMA can fetch the operands: bf16 or e4m3 rows that start on 16-byte boundaries.
static bool tma_rows(const LinearArgs& a) {
  if (a.dtype != MOLORA_BF16 && a.dtype != MOLORA_E4M3) return false;
  return a.d_in % (a.dtype == MOLORA_E4M3 ? 16 : 8) == 0 && aligned(a.x, 16) && aligned(a.W, 16) &&
         linear_encoder() != nullptr;
}

bool linear_takes_update(const LinearArgs& a, const void* B, int32_t KR) {
  return tma_rows(a) && a.N > 256 && a.d_out % 8 == 0 && KR % 8 == 0 && aligned(B, 16);
}

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t stream, const LinearUpdate* update) {
  if (!update) {
    const cudaError_t few = try_few(a, stream);
    if (few != cudaErrorNotSupported) return few;
  }
  if (!tma_rows(a)) {
    if (a.dtype == MOLORA_BF16) return launch_any<__nv_bfloat16, false>(a, stream);
    if (a.dtype == MOLORA_E4M3) return launch_any<__nv_fp8_e4m3, false>(a, stream);
    return a.d_in % 4 == 0 && aligned(a.x, 16) && aligned(a.W, 16) ? launch_any<float, true>(a, stream)
                                                                    : launch_any<float, false>(a, stream);
  }
  // K blocks of fp32 results that sum in registers (see linear_tc_kernel), which hold 96 columns a thread;
  // e4m3 sums are half as many and drift a tenth as far (2e-7 at d_in = 4096)
  const int blocks = k_blocks(a) + (update ? (update->KR + 63) / 64 * 2 : 0);
  const bool promote = a.dtype == MOLORA_E4M3 ? update != nullptr : !a.y_bf16 && blocks > kSpan;
  const Resident r = resident_clusters();
  int best = 128, split = 0;
  int64_t cost = INT64_MAX;
  for (int BN : {16, 32, 64, 128, 256}) {
    if (update || (BN > 16 && BN / 2 >= a.N)) break;
    const int64_t c = skinny_cycles(a, r, BN);
    if (c < cost) cost = c, split = BN;
  }
  // up to 32 tokens the pairs' 256 rows were never faster, and the call is the host's
  for (int BN : {256, 224, 192, 160, 128, 96, 64}) {
    if ((split && a.N <= 32) || (promote && BN > 192)) continue;
    const int64_t c = tc_cycles(a, r, BN, blocks);
    if (c < cost) cost = c, best = BN, split = 0;
  }
#ifdef MOLORA_TUNING_ENV
  if (const char* g = getenv("MOLORA_LIN_BN")) best = atoi(g);
  if (const char* g = getenv("MOLORA_LIN_SKINNY")) split = atoi(g);
#endif
  return split ? launch_skinny(a, r, split, stream) : launch_tc(a, best, promote, update, stream);
}

}  // namespace molora
