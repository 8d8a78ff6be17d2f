// feed_forward.cu -- the products of a layer's feed-forward half on the 5th-generation tensor cores:
//
//   blocks:  y[t,o] = act(sum_b sx[t,b] sw[o/128,b] sum_{i in b} x[t,i] W[o,i] + bias[o]) + residual[t,o]
//            e4m3 operands with one fp32 scale for each 128 columns of a row of x, and each 128 x 128 of W
//   gated:   h[t,f] = act(g[t,f]) u[t,f],  [g | u] = x [Wg; Wu]^T, in bf16, or in e4m3 with such scales
//   slopes:  dproj = [dh u act'(g) | dh act(g)], the first step of the gated block's backward pass (gated_grad.cu)
//
// Both projections of the gated block are one product: a tile's columns are as many rows of Wg as of Wu, so that the
// sums of g[t,f] and u[t,f] meet in the registers of one thread and neither goes to memory.  The backward pass makes
// them again, for the memory, not the time: at 4096 x 2048 -> 6144 they are 200 MB in fp32 that every layer would hold from
// one pass to the other; writing and reading them back would take 60 us, part of it under the forward's MMAs, the product takes 107.
//
// ff_tc_kernel (bf16, many tokens): linear_tc_kernel's pipeline (linear.cu): persistent pairs of CTAs with tiles of 256 tokens x
//   BN rows of W, a TMA warp and an MMA warp ahead of 8 epilogue warps by two TMEM accumulators.
// blocks_tc_kernel (e4m3, many tokens): blocks_tc.cu.
// ff_skinny_kernel (few tokens): W's rows are the MMA's M, the tokens its N, d_in split over a cluster; bound by reading W.
//   The gated block's dx = [dg | du] [Wg; Wu] is such a product too: W's columns are M, read as they lie (MN-major), and
//   2 d_ff is what is split.
#include <cudaTypedefs.h>

#include <atomic>
#ifdef MOLORA_TUNING_ENV
#include <cstdlib>
#endif

#include "feed_forward.cuh"

namespace molora {

namespace {

constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpiWarps + 2);  // + TMA warp (8) + MMA warp (9)
enum Mode { kLinear, kGated, kSlopes, kInput };  // (kInput: dx of the gated block)
constexpr int kSpan = 8;     // bf16, few tokens: K blocks summed in TMEM before fp32 registers take over

struct __align__(8) FCtrl {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t done;
  uint64_t res_full[kEpiWarps * 2];
  uint32_t tmem_base;
  int32_t abort;
};

struct FPlan {
  int BN;                // rows of W a tile
  int S;                 // stages
  int nkb;               // K blocks of 128 bytes
  int group;             // token tiles per group of tiles (they share W's rows in L2)
  // (32 bits: 2^27 tiles would be an output of 10^13 bytes)
  int32_t m_tiles, n_tiles, tiles;
  uint32_t stage_bytes, off_b, off_stage, off_ctrl, tmem_cols, smem;
};

}  // namespace

// kLong: d_in is more than kChain K blocks, whose chains registers add.
template <Mode kMode, bool kLong>
__global__ void __launch_bounds__(kThreads, 1)
    ff_tc_kernel(const FEpi E, const FPlan P, int32_t* err_word, const __grid_constant__ CUtensorMap map_x,
                 const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_y,
                 const __grid_constant__ CUtensorMap map_r) {
  constexpr int kWarps = kEpiWarps;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  FCtrl* ctrl = reinterpret_cast<FCtrl*>(sm + P.off_ctrl);
  // (the warp's number, and the like, from lane 0: in uniform registers)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int BN = P.BN, S = P.S, nkb = P.nkb, width = BN / 2;  // outputs a tile
  const uint32_t rank = cluster_ctarank();
  const uint16_t both = 0x3;
  const int32_t pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  volatile int32_t* abort = &ctrl->abort;
  // tiles in groups of P.group token tiles: within a group, the token tile runs fastest
  auto tile_at = [&](int32_t pt, int32_t& m0, int32_t& n0) {
    const int32_t span = P.group * P.n_tiles, grp = pt / span;
    const int32_t first = grp * P.group, left = P.m_tiles - first, rows = left < P.group ? left : P.group;
    const int32_t in = pt - grp * span;
    m0 = (first + in % rows) * 2 * kRows + (int32_t)rank * kRows;
    n0 = in / rows * width;
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
    for (int b = 0; b < kWarps * 2; ++b) mbar_init(&ctrl->res_full[b], 1);
    ctrl->abort = 0;
    mbar_fence_init();
    tma_prefetch_desc(&map_x);
    tma_prefetch_desc(&map_w);
    if (E.tma_y) tma_prefetch_desc(&map_y);
    if (E.tma_res) tma_prefetch_desc(&map_r);
  }
  pdl_wait();
  __syncthreads();
  // only now, with this CTA's TMEM held, may the next kernel's CTAs come and ask for theirs
  pdl_launch_dependents();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctrl->tmem_base, 0);
  cluster_sync();  // every CTA's barriers are initialised before another signals them

  if (warp == kWarps) {
    if (elect_one()) {
      int s = 0, issued = 0;
      uint32_t phase = 1;  // the first use of a stage finds it empty
      bool ok = true;
      for (int32_t pt = pair; pt < P.tiles && ok; pt += pairs) {
        int32_t m0, n0;
        tile_at(pt, m0, n0);
        const int32_t n = n0 + (int32_t)rank * E.d_out;  // one CTA brings rows of Wg and the other of Wu
        for (int kb = 0; kb < nkb; ++kb) {
          if (issued >= S && !mbar_wait_spin(&ctrl->empty[s], phase, abort)) {
            ok = false;
            break;
          }
          // the leader's barrier counts both CTAs' bytes
          const uint32_t bar = dsmem_addr(smem_u32(&ctrl->full[s]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&ctrl->full[s], 2 * P.stage_bytes);
          uint8_t* st = sm + (size_t)s * P.stage_bytes;
          tma_load_2d_pair(smem_u32(st), &map_x, kb * 64, m0, bar);
          tma_load_2d_pair(smem_u32(st + P.off_b), &map_w, kb * 64, n, bar);
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
      const uint32_t idesc = idesc_bf16_f32(2 * kRows, (uint32_t)BN, false, false);
      const uint64_t da = smem_desc(smem_u32(sm), 16, 1024, kSwizzle128B);
      const uint64_t db = smem_desc(smem_u32(sm + P.off_b), 16, 1024, kSwizzle128B);
      const uint32_t a_lo = (uint32_t)da, b_lo = (uint32_t)db, desc_hi = (uint32_t)(da >> 32);
      int s = 0, tc = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int32_t pt = pair; pt < P.tiles && ok; pt += pairs) {
        for (int from = 0; ok && from < nkb; ++tc) {
          const int to = kLong ? min(from + kChain, nkb) : nkb;
          const int buf = tc & 1;
          if (tc >= 2 && !mbar_wait_spin(&ctrl->tempty[buf], (uint32_t)((tc >> 1) - 1) & 1u, abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + (uint32_t)(buf * (P.tmem_cols / 2));
          for (int kb = from; kb < to; ++kb) {
            if (!mbar_wait_spin(&ctrl->full[s], phase, abort)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t at = (uint32_t)s * (P.stage_bytes >> 4);
            umma_stage<true, false>(d, a_lo + at, b_lo + at, desc_hi, desc_hi, idesc, kb != from);
            umma_commit_pair(&ctrl->empty[s], both);
            if (++s == S) s = 0, phase ^= 1;
          }
          if (ok) umma_commit_pair(&ctrl->tfull[buf], both);
          from = to;
        }
      }
      if (!ok) report(err_word, MOLORA_DEV_WAIT_TIMEOUT);
      umma_commit_pair(&ctrl->done, both);  // arrives in both CTAs once every MMA has completed
    }
    __syncwarp();
  } else {
    // epilogue: warps w and w + 4 share 32 rows and take chunks of 32 outputs in turn
    const int quarter = warp & 3, side = warp >> 2;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    // Outputs leave through a ring of two staging boxes; dh's chunks come through two of their own.
    constexpr int kOwn = kMode == kSlopes ? 2 : 0;
    uint8_t* in_ring = sm + P.off_stage + (size_t)warp * (2 + kOwn) * kBox;
    uint8_t* ring = in_ring + kOwn * kBox;
    int tc = 0, used = 0, asked = 0, taken = 0;  // accumulators done with, boxes written; dh's chunks on their way or taken, and taken
    auto in_box = [&](int n) { return in_ring + (size_t)(n & 1) * kBox; };
    auto ask = [&](int32_t col, int32_t m0) {  // (the box's last chunk has been read by every lane, see below)
      if (lane == 0) {
        uint64_t* bar = &ctrl->res_full[warp * 2 + (asked & 1)];
        mbar_arrive_expect_tx(bar, kBox);
        tma_load_2d(smem_u32(in_box(asked)), &map_r, col, m0, bar);
      }
      ++asked;
    };
    // the next chunk that was asked for; false where the wait ran out
    auto await = [&]() {
      return __all_sync(0xffffffffu, mbar_wait(&ctrl->res_full[warp * 2 + (taken & 1)], (uint32_t)(taken / 2) & 1u));
    };
    auto piece = [&](uint8_t* box, int i) { return box + swz_offset((uint32_t)lane, (uint32_t)i, 64); };
    // 32 columns of this warp's rows into a box, ready to be stored by lane 0
    auto stage = [&](const float (&v)[32]) {
      uint8_t* box = ring + (size_t)(used & 1) * kBox;
      if (lane == 0) bulk_wait_read<1>();  // the store that last left the box has read it
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(piece(box, i)) =
            make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                       pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
      fence_proxy_async_smem();
      __syncwarp();
      ++used;
      return box;
    };
    // rows of dh that start anywhere: a lane a column, into the same box
    auto fetch = [&](int32_t col, int32_t row) {
      __syncwarp();
      uint8_t* box = in_box(asked);
      const __nv_bfloat16* dh = static_cast<const __nv_bfloat16*>(E.res) + (int64_t)row * E.d_out + col + lane;
      const bool in = col + lane < E.d_out;
#pragma unroll
      for (int r0 = 0; r0 < 32; r0 += 16) {  // (loads before stores: these could be to the same memory)
        __nv_bfloat16 v[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = in && row + r0 + r < E.N ? dh[(int64_t)(r0 + r) * E.d_out] : __float2bfloat16_rn(0.f);
#pragma unroll
        for (int r = 0; r < 16; ++r)
          *reinterpret_cast<__nv_bfloat16*>(box + swz_offset((uint32_t)(r0 + r), (uint32_t)lane >> 3, 64) + (lane & 7) * 2) = v[r];
      }
      ++asked;
    };
    const uint32_t tempty = dsmem_addr(smem_u32(&ctrl->tempty[0]), 0);
    bool ok = true;
    int32_t pt = pair;
    for (; pt < P.tiles && ok; pt += ok ? pairs : 0) {
      int32_t m0, n0;
      tile_at(pt, m0, n0);
      m0 += quarter * 32;
      const int chunks = m0 < E.N ? min(width / 32, (E.d_out - n0 + 31) / 32) : 0;
      // h's chunk from its finished values
      auto put = [&](float (&v)[32], int32_t col) {
        if (E.tma_y) {
          const uint8_t* box = stage(v);
          if (lane == 0) {
            tma_store_2d(&map_y, smem_u32(box), col, m0);
            bulk_commit();
          }
        } else {
          // rows that are not 16-byte aligned: turned in shared memory, written a row at a time
          float* turned = reinterpret_cast<float*>(ring);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 32; ++i) turned[lane * 32 + (i ^ lane)] = v[i];
          __syncwarp();
          __nv_bfloat16* y = static_cast<__nv_bfloat16*>(E.y) + (int64_t)m0 * E.d_out + col + lane;
          if (col + lane < E.d_out) {
            if (m0 + 32 <= E.N) {
#pragma unroll 8
              for (int q = 0; q < 32; ++q) y[(int64_t)q * E.d_out] = __float2bfloat16_rn(turned[q * 32 + (lane ^ q)]);
            } else {
              for (int q = 0; m0 + q < E.N; ++q) y[(int64_t)q * E.d_out] = __float2bfloat16_rn(turned[q * 32 + (lane ^ q)]);
            }
          }
        }
      };
      if (E.tma_res) {
        for (int c = side; c < chunks; c += 2) ask(n0 + c * 32, m0);
      } else if (kMode == kSlopes) {
        for (int c = side; c < chunks; c += 2) fetch(n0 + c * 32, m0);
      }
      auto sums_ready = [&]() {
        ok = __all_sync(0xffffffffu, mbar_wait_spin(&ctrl->tfull[tc & 1], (uint32_t)(tc >> 1) & 1u, abort));
        if (ok) tc_fence_after();
        return ok;
      };
      auto free_sums = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_read(tempty + (tc & 1) * 8);
      };
      float sums[kLong ? 2 : 1][64];  // kLong: of this warp's chunks, the gate's 32 columns and the up projection's
      if constexpr (kLong) {
#pragma unroll
        for (int k = 0; k < 64; ++k) sums[0][k] = sums[1][k] = 0.f;
        for (int left = nkb; left > 0 && sums_ready(); left -= kChain) {
          const uint32_t base = tmem + lanes + (uint32_t)((tc & 1) * (P.tmem_cols / 2));
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            if (side + 2 * n >= chunks) continue;
#pragma unroll
            for (int h = 0; h < 64; h += 16) {
              float r[16];
              tmem_ld16(base + (uint32_t)((h < 32 ? 0 : width - 32) + (side + 2 * n) * 32 + h), r);
#pragma unroll
              for (int k = 0; k < 16; ++k) sums[n][h + k] += r[k];
            }
          }
          free_sums();
          ++tc;
        }
        if (!ok) break;
      } else {
        if (!sums_ready()) break;
        if (side >= chunks) free_sums();
      }
      const uint32_t base = tmem + lanes + (uint32_t)((tc & 1) * (P.tmem_cols / 2));
#pragma unroll(kLong ? 2 : 1)
      for (int n = 0; n < 2; ++n) {  // (tiles of 256 rows of W at most: two chunks a warp)
        const int c = side + 2 * n;
        if (c >= chunks) break;
        float g[32], u[32];
        if constexpr (kLong) {
#pragma unroll
          for (int i = 0; i < 32; ++i) g[i] = sums[n][i], u[i] = sums[n][32 + i];
        } else {
          uint32_t rg[32], ru[32];
          tmem_ld32_start(base + (uint32_t)(c * 32), rg);
          tmem_ld32_start(base + (uint32_t)(width + c * 32), ru);
          tmem_ld_wait(rg);
          tmem_ld_bind(ru);
          if (c + 2 >= chunks) free_sums();
#pragma unroll
          for (int i = 0; i < 32; ++i) g[i] = __uint_as_float(rg[i]), u[i] = __uint_as_float(ru[i]);
        }
        const int32_t col = n0 + c * 32;
        if constexpr (kMode == kGated) {
          apply_act(g, E.act);
#pragma unroll
          for (int i = 0; i < 32; ++i) g[i] *= u[i];
          put(g, col);
        } else {
          uint8_t* box = in_box(taken);
          if (E.tma_res) {
            if (!(ok = await())) break;
          } else {
            __syncwarp();
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 d = *reinterpret_cast<const uint4*>(piece(box, i));
            const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float dh = __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
              float a, s;
              act_and_slope(g[8 * i + j], E.act, a, s);
              g[8 * i + j] = dh * u[8 * i + j] * s;
              u[8 * i + j] = dh * a;
            }
          }
          ++taken;
          const uint8_t* from = stage(g);  // (after its __syncwarp every lane has read dh's box)
          if (lane == 0) {
            tma_store_3d(&map_y, smem_u32(from), col, 0, m0);
            bulk_commit();
          }
          from = stage(u);
          if (lane == 0) {
            tma_store_3d(&map_y, smem_u32(from), col, 1, m0);
            bulk_commit();
          }
        }
      }
      if (!kLong) ++tc;
    }
    if (!ok) {
      for (; E.tma_res && taken < asked; ++taken) await();  // no copy is left in flight
      *abort = 1;
      if (lane == 0) report(err_word, MOLORA_DEV_WAIT_TIMEOUT);
      if constexpr (kMode == kSlopes) {
        // what is lost of dproj is NaN, and so is what the products after this kernel make of it
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
#pragma unroll 1
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(piece(ring, i)) = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
        fence_proxy_async_smem();
        __syncwarp();
#pragma unroll 1
        for (; pt < P.tiles && lane == 0; pt += pairs) {
          int32_t m0, n0;
          tile_at(pt, m0, n0);
          m0 += quarter * 32;
#pragma unroll 1
          for (int c = side; m0 < E.N && c < width / 32 && n0 + c * 32 < E.d_out; c += 2) {
            tma_store_3d(&map_y, smem_u32(ring), n0 + c * 32, 0, m0);
            tma_store_3d(&map_y, smem_u32(ring), n0 + c * 32, 1, m0);
            bulk_commit();
          }
        }
      }
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
namespace {

struct FSkinnyPlan {
  int BN;                // tokens per tile (MMA N)
  int C;                 // CTAs of a cluster: d_in split C ways
  int S;
  int nkb;
  int32_t o_tiles, t_tiles;
  uint32_t stage_bytes, off_b, off_ctrl, tmem_cols, smem;
};

// Ends a tile whose d_in was split over a cluster's C CTAs (as linear.cu's split_epilogue does): each CTA's sums
// [token][row of W] go to shared memory, each CTA adds its share of the outputs in rank order, reading the others'
// through distributed shared memory, and writes it.  Where `have` is false a wait ran out: such a thread's sums are
// NaN, and so is what any CTA of the cluster makes of them.
template <Mode kMode, int U, int J>
__device__ __forceinline__ void ff_join(const FEpi& E, const float (&sums)[J][16], bool have, uint8_t* sm, int C, int rank,
                                        int32_t o0, int64_t t0, int tokens, int32_t* err_word) {
  constexpr int kParts = kMode == kGated ? 2 : 1, kQuads = kRows / 4 / kParts;  // quads of outputs a token
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float* part = reinterpret_cast<float*>(sm);
  if (!have) report(err_word, MOLORA_DEV_WAIT_TIMEOUT);
  if (warp < kEpiWarps) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = (warp >> 2) * 16 + 32 * j;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (c + i < tokens) part[(c + i) * kRows + (warp & 3) * 32 + lane] = have ? sums[j][i] : __uint_as_float(0x7fffffffu);
    }
  }
  __syncthreads();
  if (C > 1) cluster_sync();
  if (warp < kEpiWarps) {
    const bool vec = E.tma_y;  // (d_out a multiple of 4 and y, residual aligned)
    const bool bias_vec = vec && (reinterpret_cast<uintptr_t>(E.bias) & 15u) == 0;
    const int quads = tokens * kQuads, step = C * 256;
    for (int q0 = rank * 256 + tid; q0 < quads; q0 += U * step) {
      Quad v[U][kParts], res[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int q = q0 + u * step, o = o0 + (q % kQuads) * 4;
        if (q >= quads || o >= E.d_out) continue;
        const int64_t row = (t0 + q / kQuads) * E.d_out;
        if (kMode == kLinear && E.res) {
          if (E.y_bf16)
            res[u].load(static_cast<const __nv_bfloat16*>(E.res) + row, o, E.d_out, vec);
          else
            res[u].load(static_cast<const float*>(E.res) + row, o, E.d_out, vec);
        }
#pragma unroll
        for (int h = 0; h < kParts; ++h) {
          float4 p[8];
          const float* mine = part + (q / kQuads) * kRows + h * (kRows / 2) + (q % kQuads) * 4;
          const uint32_t at = smem_u32(mine);
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c < C) p[c] = C > 1 ? dsmem_ld_f4(dsmem_addr(at, (uint32_t)c)) : *reinterpret_cast<const float4*>(mine);
          float(&s)[4] = v[u][h].v;
          s[0] = p[0].x, s[1] = p[0].y, s[2] = p[0].z, s[3] = p[0].w;
#pragma unroll
          for (int c = 1; c < 8; ++c)
            if (c < C) s[0] += p[c].x, s[1] += p[c].y, s[2] += p[c].z, s[3] += p[c].w;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int q = q0 + u * step, o = o0 + (q % kQuads) * 4;
        if (q >= quads || o >= E.d_out) continue;
        const int64_t t = t0 + q / kQuads, row = t * E.d_out;
        Quad& y = v[u][0];
        if constexpr (kMode == kGated) {
#pragma unroll
          for (int i = 0; i < 4; ++i) y.v[i] = activate(y.v[i], E.act) * v[u][kParts - 1].v[i];
        } else {
          if (E.bias) {
            Quad b;
            b.load(E.bias, o, E.d_out, bias_vec);
#pragma unroll
            for (int i = 0; i < 4; ++i) y.v[i] += b.v[i];
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) y.v[i] = activate(y.v[i], E.act);
          if (E.res)
#pragma unroll
            for (int i = 0; i < 4; ++i) y.v[i] += res[u].v[i];
        }
        if (E.y_bf16)
          y.store(static_cast<__nv_bfloat16*>(E.y) + row, o, E.d_out, vec);
        else
          y.store(static_cast<float*>(E.y) + row, o, E.d_out, vec);
      }
    }
  }
  __syncthreads();
  if (C > 1) cluster_sync();  // no CTA leaves while another may still read its partial sums
}

}  // namespace

// J: columns of sums a thread keeps, 32 J tokens a tile.  Warp w's lanes have rows 32 (w % 4) .. + 31 of the tile's 128
// of W, columns 16 (w / 4) + 32 j .. + 15 of its tokens.
template <bool kFp8, Mode kMode, int J>
__global__ void __launch_bounds__(kThreads, 1)
    ff_skinny_kernel(const FEpi E, const FSkinnyPlan P, int32_t* err_word, const __grid_constant__ CUtensorMap map_x,
                     const __grid_constant__ CUtensorMap map_w) {
  constexpr int kWidth = kMode == kGated ? kRows / 2 : kRows;  // outputs a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  FCtrl* ctrl = reinterpret_cast<FCtrl*>(sm + P.off_ctrl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int BN = P.BN, S = P.S, C = P.C;
  const int rank = (int)cluster_ctarank();
  const unsigned tile = blockIdx.x / (unsigned)C;
  const int32_t o0 = (int32_t)(tile % (unsigned)P.o_tiles) * kWidth, t0 = (int32_t)(tile / (unsigned)P.o_tiles) * BN;
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
  constexpr int kEach = kFp8 ? 1 : kSpan;  // K blocks an accumulator holds
  const int spans = (kb1 - kb0 + kEach - 1) / kEach;
  float sums[J][16];
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i) sums[j][i] = 0.f;
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
        if constexpr (kMode == kInput) {  // K runs over the gate's columns of dproj, then the up's
          const int32_t plane = kb >= P.nkb / 2, k = (kb - (plane ? P.nkb / 2 : 0)) * 64;
          tma_load_3d(smem_u32(st), &map_w, o0, k, plane, &ctrl->full[s]);
          tma_load_3d(smem_u32(st + kAtom), &map_w, o0 + 64, k, plane, &ctrl->full[s]);
          tma_load_3d(smem_u32(st + P.off_b), &map_x, k, plane, t0, &ctrl->full[s]);
          if (++s == S) s = 0, phase ^= 1;
          continue;
        }
        tma_load_2d(smem_u32(st), &map_w, kb * elems, o0, &ctrl->full[s]);
        if (kMode == kGated) tma_load_2d(smem_u32(st + kWidth * kRowBytes), &map_w, kb * elems, E.d_out + o0, &ctrl->full[s]);
        tma_load_2d(smem_u32(st + P.off_b), &map_x, kb * elems, t0, &ctrl->full[s]);
        if (++s == S) s = 0, phase ^= 1;
      }
      for (int q = 0; q < S && q < issued; ++q) mbar_wait(&ctrl->full[q], (uint32_t)((issued - 1 - q) / S) & 1u);
    }
    __syncwarp();
  } else if (warp == 9) {
    if (elect_one()) {
      const uint32_t idesc = kFp8 ? idesc_e4m3_f32(kRows, (uint32_t)BN) : idesc_bf16_f32(kRows, (uint32_t)BN, kMode == kInput, false);
      const uint64_t da = smem_desc(smem_u32(sm), kMode == kInput ? kAtom : 16, 1024, kSwizzle128B);
      const uint64_t db = smem_desc(smem_u32(sm + P.off_b), 16, 1024, kSwizzle128B);
      const uint32_t a_lo = (uint32_t)da, b_lo = (uint32_t)db, desc_hi = (uint32_t)(da >> 32);
      bool ok = true;
      int s = 0;
      uint32_t phase = 0;
      for (int c = 0; c < spans && ok; ++c) {
        const int first = kb0 + c * kEach, last = min(first + kEach, kb1);
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
          if constexpr (kMode == kInput)
            umma_stage_steps<false>(d, a_lo + at, b_lo + at, desc_hi, desc_hi, idesc, kb != first, 16 * kRowBytes / 16, 2);
          else
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
    const uint32_t base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int c0 = (warp >> 2) * 16;
    // e4m3: the K block's scales, of this warp's rows of W, and lane i of the i-th token of each 16
    const float* pw = nullptr;
    const float* px[J];
    float row = 0.f, col[J];
    if constexpr (kFp8) {
      const int32_t block = o0 / 128 + (kMode == kGated && (warp & 2) ? E.up : 0);
      pw = E.sw + (int64_t)block * P.nkb;
      row = pw[kb0];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int64_t t = t0 + c0 + 32 * j + (lane & 15);
        px[j] = E.sx + (t < E.N ? t : 0) * P.nkb;
        col[j] = px[j][kb0];
      }
    }
    for (int c = 0; c < spans && have; ++c) {
      float sc[J];
      if constexpr (kFp8) {
#pragma unroll
        for (int j = 0; j < J; ++j) sc[j] = row * col[j];
        if (c + 1 < spans) {
          row = pw[kb0 + c + 1];
#pragma unroll
          for (int j = 0; j < J; ++j) col[j] = px[j][kb0 + c + 1];
        }
      }
      have = __all_sync(0xffffffffu, mbar_wait_spin(&ctrl->tfull[c & 1], (uint32_t)(c >> 1) & 1u, abort));
      if (!have) break;
      tc_fence_after();
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (c0 + 32 * j >= tokens) continue;
        float p[16];
        tmem_ld16(base + (uint32_t)((c & 1) * BN + c0 + 32 * j), p);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if constexpr (kFp8)
            sums[j][i] = fmaf(p[i], __shfl_sync(0xffffffffu, sc[j], i), sums[j][i]);
          else
            sums[j][i] += p[i];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctrl->tempty[c & 1]);
    }
  }
  // every MMA is done; the TMA warp has seen every load land
  have = mbar_wait(&ctrl->done, 0) && have && !*abort;
  __syncthreads();
  ff_join<kMode == kInput ? kLinear : kMode, J >= 2 && kMode != kGated ? 4 : 2>(E, sums, have, sm, C, rank, o0, t0, tokens, err_word);
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, P.tmem_cols);
  }
}

// ---------------------------------------------------------------------------------------------
namespace {

cudaError_t launch_tc(const FeedForwardArgs& a, Mode mode, int BN, cudaStream_t stream) {
  FEpi e = ff_epilogue_of(a);
  FPlan p = {};
  const int width = BN / 2;
  const int64_t m_tiles = (a.N + 2 * kRows - 1) / (2 * kRows), n_tiles = ((int64_t)a.d_out + width - 1) / width;
  if (m_tiles * n_tiles > INT32_MAX / 16) return cudaErrorNotSupported;
  p.BN = BN;
  p.nkb = ff_k_blocks(a);
  p.m_tiles = (int32_t)m_tiles;
  p.n_tiles = (int32_t)n_tiles;
  p.tiles = p.m_tiles * p.n_tiles;
  p.group = 8;
  p.off_b = kRows * kRowBytes;
  p.stage_bytes = p.off_b + (uint32_t)(BN / 2) * kRowBytes;
  p.tmem_cols = tmem_columns(2 * (uint32_t)(BN <= 64 ? 64 : BN <= 128 ? 128 : 256));
  CUtensorMap mx, mw, my = {}, mr = {};
  const auto BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  auto rows_map = [&](CUtensorMap* m, const void* base) {
    return linear_map(m, BF, 2, base, (uint64_t)a.N, (uint64_t)a.d_out, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  };
  if (mode == kSlopes) {
    const uint64_t half = ((uint64_t)a.d_out + 7) & ~uint64_t(7);
    if (!linear_map_3d(&my, BF, a.y, {half, 2, (uint64_t)a.N}, {2 * half, 4 * half}, {32, 1, 32}, CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorNotSupported;
    e.tma_res = a.d_out % 8 == 0 && aligned(a.residual, 16) && rows_map(&mr, a.residual);
  } else if (e.tma_y && !rows_map(&my, a.y)) {
    e.tma_y = false;
  }
  const uint32_t boxes = kEpiWarps * (mode == kSlopes ? 4 : 2) * kBox;
  static_assert(2 * kBox >= kTurn, "a warp's boxes hold a turned chunk");
  const size_t fixed = boxes + sizeof(FCtrl) + kSmemSlack;
  p.S = (int)((kMaxSmem - fixed) / p.stage_bytes);
  if (p.S > kMaxStages) p.S = kMaxStages;
  p.off_stage = (uint32_t)p.S * p.stage_bytes;
  p.off_ctrl = p.off_stage + boxes;
  // one CTA an SM, alone: an allocation of TMEM never waits for another CTA's (see linear.cu)
  p.smem = kMaxSmem;
  if (!ff_operand_map(&mx, a, a.x, a.N, kRows) || !ff_operand_map(&mw, a, a.W, ff_rows_of_w(a), (uint32_t)(BN / 2)))
    return cudaErrorNotSupported;
  auto go = [&](auto kernel, std::atomic<uint64_t>& allowed) {
    const cudaError_t set = allow_smem(kernel, allowed, kMaxSmem);
    if (set != cudaSuccess) return set;
    const int32_t most = num_sms() / 2;
    const dim3 grid((unsigned)(2 * (p.tiles < most ? p.tiles : most)));
    return launch_kernel(kernel, grid, dim3(kThreads), p.smem, stream, 2, e, p, a.err_word, mx, mw, my, mr);
  };
  static std::atomic<uint64_t> allowed[4];
  if (p.nkb > kChain)
    return mode == kSlopes ? go(ff_tc_kernel<kSlopes, true>, allowed[0]) : go(ff_tc_kernel<kGated, true>, allowed[1]);
  return mode == kSlopes ? go(ff_tc_kernel<kSlopes, false>, allowed[2]) : go(ff_tc_kernel<kGated, false>, allowed[3]);
}

// The plan of a product of o_tiles x 128 rows of W with N tokens, in tiles of BN tokens.
FSkinnyPlan skinny_plan(const Resident& r, int64_t o_tiles, int64_t N, int nkb, int BN) {
  FSkinnyPlan p = {};
  p.BN = BN;
  p.nkb = nkb;
  p.o_tiles = (int32_t)o_tiles;
  p.t_tiles = (int32_t)((N + BN - 1) / BN);
  p.C = split_of(r, o_tiles * p.t_tiles, nkb);
  p.off_b = kRows * kRowBytes;
  p.stage_bytes = p.off_b + (uint32_t)BN * kRowBytes;
  p.tmem_cols = tmem_columns(2 * (uint32_t)BN);
  const size_t fixed = sizeof(FCtrl) + kSmemSlack;
  const size_t partial = (size_t)BN * kRows * sizeof(float);
  const int need = (nkb + p.C - 1) / p.C;
  p.S = (int)((kMaxSmem - fixed) / p.stage_bytes);
  if (p.S > kMaxStages) p.S = kMaxStages;
  if (p.S > need) p.S = need;
  size_t ring = (size_t)p.S * p.stage_bytes;
  if (ring < partial) ring = partial;
  p.off_ctrl = (uint32_t)ring;
  p.smem = (uint32_t)(ring + fixed);
  if (p.smem < 116 * 1024) p.smem = 116 * 1024;  // no two CTAs that could wait for each other's TMEM share an SM (see linear.cu)
  return p;
}

template <bool kFp8, Mode kMode>
cudaError_t launch_skinny_kernel(const FEpi& e, const FSkinnyPlan& p, int32_t* err_word, cudaStream_t stream, const CUtensorMap& mx,
                                 const CUtensorMap& mw) {
  static std::atomic<uint64_t> allowed[4];
  auto go = [&](auto kernel, int n) {
    const cudaError_t set = allow_smem(kernel, allowed[n], kMaxSmem);
    if (set != cudaSuccess) return set;
    const int64_t ctas = (int64_t)p.o_tiles * p.t_tiles * p.C;
    if (ctas > INT32_MAX) return cudaErrorNotSupported;
    return launch_kernel(kernel, dim3((unsigned)ctas), dim3(kThreads), p.smem, stream, p.C, e, p, err_word, mx, mw);
  };
  switch (p.BN) {
    case 16:
    case 32:
      return go(ff_skinny_kernel<kFp8, kMode, 1>, 0);
    case 64:
      return go(ff_skinny_kernel<kFp8, kMode, 2>, 1);
    case 128:
      return go(ff_skinny_kernel<kFp8, kMode, 4>, 2);
    default:
      return go(ff_skinny_kernel<kFp8, kMode, 8>, 3);
  }
}

cudaError_t launch_skinny(const FeedForwardArgs& a, const Resident& r, int BN, cudaStream_t stream) {
  const FEpi e = ff_epilogue_of(a);
  const int width = a.gated ? kRows / 2 : kRows;
  const FSkinnyPlan p = skinny_plan(r, ((int64_t)a.d_out + width - 1) / width, a.N, ff_k_blocks(a), BN);
  CUtensorMap mx, mw;
  if (!ff_operand_map(&mx, a, a.x, a.N, (uint32_t)p.BN) || !ff_operand_map(&mw, a, a.W, ff_rows_of_w(a), (uint32_t)width))
    return cudaErrorNotSupported;
  if (a.dtype != MOLORA_E4M3) return launch_skinny_kernel<false, kGated>(e, p, a.err_word, stream, mx, mw);
  return a.gated ? launch_skinny_kernel<true, kGated>(e, p, a.err_word, stream, mx, mw)
                 : launch_skinny_kernel<true, kLinear>(e, p, a.err_word, stream, mx, mw);
}

// Cycles that ff_skinny_kernel takes in tiles of BN tokens, and the pairs' kernels in tiles of BN rows of W: what a K block takes,
// what ends a tile, and the way through.  Fitted to 130 sizes on GB300 (1 to 2048 tokens, d_in 1024 to 4096, 1024 to 12288
// rows of W): the choice is 0.8% off the fastest on average, 15% at most; with e4m3 to 121 more (128 to 8192 tokens, each kind
// of y, bias and residual): 0.7%, 11%.  With e4m3 a K block of many tokens takes long, as its sums are scaled: 200 tokens of
// 1024 -> 1024 gated 6.1 us in tiles of 32, 7.7 in tiles of 128.
int64_t skinny_cycles(const Resident& r, int64_t rows_of_w, int64_t N, int nkb, bool fp8, int BN) {
  const int64_t tiles = ((rows_of_w + kRows - 1) / kRows) * ((N + BN - 1) / BN);
  const int C = split_of(r, tiles, nkb);
  const int64_t waves = (tiles + r.of[C] - 1) / r.of[C], blocks = (nkb + C - 1) / C;
  if (fp8) return 4000 + waves * (blocks * (450 + 5 * BN) + 60 * BN);
  return 6600 + waves * (blocks * (730 + BN * 3 / 5) + 38 * BN);
}

// The tile of the least cost.
int best_skinny(const Resident& r, int64_t rows_of_w, int64_t N, int nkb, bool fp8, int64_t& cost) {
  int best = 0;
  cost = INT64_MAX;
  for (int BN : {16, 32, 64, 128, 256}) {
    if (BN > 16 && BN / 2 >= N) break;
    const int64_t c = skinny_cycles(r, rows_of_w, N, nkb, fp8, BN);
    if (c < cost) cost = c, best = BN;
  }
  return best;
}

int64_t tc_cycles(const FeedForwardArgs& a, const Resident& r, int BN) {
  const int width = a.gated ? BN / 2 : BN;
  const int64_t m_tiles = (a.N + 2 * kRows - 1) / (2 * kRows), blocks = ff_k_blocks(a);
  const int64_t tiles = m_tiles * (((int64_t)a.d_out + width - 1) / width), waves = (tiles + r.of[2] - 1) / r.of[2];
  if (a.dtype == MOLORA_E4M3) {
    // (rows of y that TMA cannot write: by the byte)
    const int64_t by_lanes = ff_epilogue_of(a).tma_y ? 0 : 15 * width * (a.y_bf16 ? 2 : 4);
    return 8000 + waves * (blocks * (150 + BN * 7 / 5) + 1000 + by_lanes);
  }
  return 6300 + waves * (blocks * (160 + BN * 8 / 5) + 450);
}

// The pairs' tile of the least cost, if that is below `cost`, else 0.
int best_tc(const FeedForwardArgs& a, const Resident& r, int64_t cost) {
  int best = 0;
  for (int BN : {256, 192, 128, 64}) {
    if (BN == 64 && a.dtype == MOLORA_E4M3) continue;
    const int64_t c = tc_cycles(a, r, BN);
    if (c < cost) cost = c, best = BN;
  }
#ifdef MOLORA_TUNING_ENV
  if (const char* g = getenv("MOLORA_FF_BN")) best = atoi(g);
#endif
  return best;
}

}  // namespace

cudaError_t launch_feed_forward(const FeedForwardArgs& a, cudaStream_t stream) {
  const Resident r = resident_clusters();
  int64_t cost;
  int split = best_skinny(r, ff_rows_of_w(a), a.N, ff_k_blocks(a), a.dtype == MOLORA_E4M3, cost);
#ifdef MOLORA_TUNING_ENV
  if (const char* g = getenv("MOLORA_FF_SKINNY")) split = atoi(g), cost = split ? 0 : INT64_MAX;
#endif
  // Up to 32 tokens are bound by reading W, of which the costs, cycles of the tensor cores' side, say nothing: there clusters that
  // split d_in read faster than the pairs, whatever their tiles.  Of 90 sizes (each of the three products; 1, 16 and 32 tokens;
  // d_in 128 to 16384, 4096 to 65536 outputs) few tokens' kernel took 0.48 to 1.00 of the pairs' time at 73, 1.01 to 1.16 at 8 (wide
  // W, short rows) and 1.04 to 1.59 at 128 -> 65536 (e4m3 blocks, 32 tokens, us: 4096 -> 4096 8.0 and 13.3, 1024 -> 28672 14.9
  // and 12.9).
  const int pairs = a.N <= 32 && cost < INT64_MAX ? 0 : best_tc(a, r, cost);
  if (!pairs) return launch_skinny(a, r, split, stream);
  return a.dtype == MOLORA_E4M3 ? launch_blocks_tc(a, pairs, stream) : launch_tc(a, kGated, pairs, stream);
}

cudaError_t launch_gated_slope(const GatedGradArgs& g, cudaStream_t stream) {
  const FeedForwardArgs a = {true, g.x, MOLORA_BF16, nullptr, g.N, g.d_in, g.W, nullptr, g.d_ff, nullptr, g.act, g.dh, g.dproj, true,
                             g.err_word};
  return launch_tc(a, kSlopes, best_tc(a, resident_clusters(), INT64_MAX), stream);
}

int64_t gated_input_cycles(const GatedGradArgs& a) {
  int64_t cost;
  best_skinny(resident_clusters(), a.d_in, a.N, 2 * (int)(((int64_t)a.d_ff + 63) / 64), false, cost);
  return cost;
}

cudaError_t launch_gated_input(const GatedGradArgs& a, cudaStream_t stream) {
  const Resident r = resident_clusters();
  const uint64_t N = (uint64_t)a.N, F = (uint64_t)a.d_ff, D = (uint64_t)a.d_in, half = (F + 7) & ~uint64_t(7);
  const int nkb = 2 * (int)((F + 63) / 64);
  int64_t cost;
  const int BN = best_skinny(r, a.d_in, a.N, nkb, false, cost);
  FEpi e = {};
  e.N = a.N;
  e.d_out = a.d_in;
  e.act = MOLORA_ACT_NONE;
  e.y = a.dx;
  e.y_bf16 = e.tma_y = true;
  const auto BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto S128 = CU_TENSOR_MAP_SWIZZLE_128B;
  CUtensorMap mx, mw;
  if (!linear_map_3d(&mx, BF, a.dproj, {F, 2, N}, {2 * half, 4 * half}, {64, 1, (uint32_t)BN}, S128) ||
      !linear_map_3d(&mw, BF, a.W, {D, F, 2}, {2 * D, 2 * F * D}, {64, 64, 1}, S128))
    return cudaErrorNotSupported;
  return launch_skinny_kernel<false, kInput>(e, skinny_plan(r, ((int64_t)a.d_in + kRows - 1) / kRows, a.N, nkb, BN), a.err_word, stream, mx, mw);
}

}  // namespace molora
