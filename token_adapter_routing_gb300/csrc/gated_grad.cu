// gated_grad.cu -- the gradients of the gated feed-forward block h = act(g) u, [g | u] = x [Wg; Wu]^T, from those of its
// projections, dproj = [dg | du] (feed_forward.cu):
//
//   dx = dg Wg + du Wu            2 d_ff terms an element
//   dWg = dg^T x,  dWu = du^T x   N terms an element
//
// Both products are tiles of one persistent kernel of CTA pairs (linear.cu's pipeline: a TMA warp and an MMA warp ahead of
// the epilogue by two TMEM accumulators), so that the second's tiles fill the pairs that the first leaves idle.
// No operand is transposed in memory: what is not K-major (W in dx, both operands in dW) is read by the tensor
// cores as it lies, MN-major, in boxes of 64 columns x 64 rows of K.  Bound by the tensor cores: 4096 x 2048 -> 6144, both
// products, 250 us (1.65 PFLOP/s).
// Sums of more than kChain K blocks (2 d_ff or N past 8192) are chains that registers add.
// Few tokens leave most pairs without a tile of dx, and the others with sums of 2 d_ff terms: there ff_skinny_kernel
// (feed_forward.cu) makes dx, d_ff split over clusters.
#include <cudaTypedefs.h>

#include <atomic>
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
constexpr int kSets = 2;                        // staging boxes an epilogue warp: all that it stores of a tile of 256 columns
constexpr uint32_t kOutBox = 32 * kRowBytes;    // 32 rows of 64 columns
constexpr uint32_t kStageA = kRows * kRowBytes;

struct __align__(8) GCtrl {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t done;
  uint32_t tmem_base;
  int32_t abort;
};

// dx's tiles (the longer sums, where N < 2 d_ff) go round the pairs, then dW's: as many of them to each pair that is a tile
// of dx short as take no longer than one, the rest round the pairs again, these first.
struct GPlan {
  int BN;                    // columns a tile
  int S;
  int64_t tiles_x, tiles_w;  // dx's, dW's (gate and up rows)
  int32_t n_tiles;           // tiles across d_in
  int64_t m_tiles_x, m_tiles_w;  // down N, down d_ff
  int32_t kb_half, kb_x, kb_w;   // K blocks of 64: of one projection, of a tile of dx, of one of dW
  int32_t group;
  int32_t pairs;             // of CTAs
  int32_t full, ahead;       // pairs with one tile of dx more than the others, and dW's tiles that the others get first
  int64_t N;
  int32_t d_in, d_ff;
  uint32_t stage_bytes, off_stage, off_ctrl, tmem_cols;
};

struct GTile {
  bool x;          // of dx
  int32_t plane;   // of dW: 0 gate, 1 up
  int32_t m0, n0;  // this CTA's first row, the tile's first column
  int32_t kbs;
};

// The j-th tile of a pair; false if it has no more.
__device__ __forceinline__ bool tile_at(const GPlan& P, int32_t pair, int64_t j, uint32_t rank, GTile& t) {
  const bool full = pair < P.full;
  const int64_t mine = P.tiles_x / P.pairs + full;
  t.x = j < mine;
  int64_t i;
  if (t.x) {
    i = pair + j * P.pairs;
  } else {
    j -= mine;
    if (!full && j < P.ahead) {
      i = (int64_t)(pair - P.full) * P.ahead + j;
    } else {
      if (!full) j -= P.ahead;
      i = (int64_t)(P.pairs - P.full) * P.ahead + (full ? pair + P.pairs : pair) - P.full + j * P.pairs;
    }
    if (i >= P.tiles_w) return false;
  }
  const int64_t m_tiles = t.x ? P.m_tiles_x : 2 * P.m_tiles_w;
  // groups of row tiles that share the other operand's columns in L2: within one the row tile runs fastest
  const int64_t span = (int64_t)P.group * P.n_tiles, grp = i / span;
  const int64_t first = grp * P.group, left = m_tiles - first, rows = left < P.group ? left : P.group;
  const int64_t in = i - grp * span;
  int64_t m = first + in % rows;
  t.plane = !t.x && m >= P.m_tiles_w;
  if (t.plane) m -= P.m_tiles_w;
  t.m0 = (int32_t)(m * 2 * kRows + rank * kRows);
  t.n0 = (int32_t)(in / rows) * P.BN;
  t.kbs = t.x ? P.kb_x : P.kb_w;
  return true;
}

}  // namespace

// map_pk, map_pm: dproj [N x 2 x d_ff] in boxes of 128 tokens x 64 columns (K-major rows of dx's product), and of 64
// tokens x 64 (MN-major rows of dW's).  map_b[0], map_b[1]: W [2 x d_ff x d_in] and x [1 x N x d_in] in boxes of 64 x 64.
// map_dx, map_dw: the outputs, [1 x N x d_in] and [2 x d_ff x d_in].
// kLong: some tile has more than kChain K blocks, whose chains registers add.
template <bool kLong>
__global__ void __launch_bounds__(kThreads, 1)
    grad_tc_kernel(const GPlan P, int32_t* err_word, const __grid_constant__ CUtensorMap map_pk,
                   const __grid_constant__ CUtensorMap map_pm, const __grid_constant__ CUtensorMap map_w,
                   const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_dx,
                   const __grid_constant__ CUtensorMap map_dw) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  GCtrl* ctrl = reinterpret_cast<GCtrl*>(sm + P.off_ctrl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int BN = P.BN, S = P.S;
  const uint32_t rank = cluster_ctarank();
  const uint16_t both = 0x3;
  const int32_t pair = blockIdx.x / 2;
  volatile int32_t* abort = &ctrl->abort;

  if (warp == kEpiWarps + 1) {
    tmem_alloc_pair(&ctrl->tmem_base, P.tmem_cols);
    tmem_relinquish_pair();
  }
  if (warp == kEpiWarps && lane == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&ctrl->full[s], 1);
      mbar_init(&ctrl->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctrl->tfull[b], 1);
      mbar_init(&ctrl->tempty[b], 2 * kEpiWarps);
    }
    mbar_init(&ctrl->done, 1);
    ctrl->abort = 0;
    mbar_fence_init();
    if (P.tiles_x) {
      tma_prefetch_desc(&map_pk);
      tma_prefetch_desc(&map_w);
      tma_prefetch_desc(&map_dx);
    }
    if (P.tiles_w) {
      tma_prefetch_desc(&map_pm);
      tma_prefetch_desc(&map_x);
      tma_prefetch_desc(&map_dw);
    }
  }
  pdl_wait();
  __syncthreads();
  // only now, with this CTA's TMEM held, may the next kernel's CTAs come and ask for theirs
  pdl_launch_dependents();
  tc_fence_after();
  const uint32_t tmem = ctrl->tmem_base;
  cluster_sync();  // every CTA's barriers are initialised before another signals them

  if (warp == kEpiWarps) {
    if (elect_one()) {
      int s = 0, issued = 0;
      uint32_t phase = 1;  // the first use of a stage finds it empty
      bool ok = true;
      GTile t;
      for (int64_t i = 0; ok && tile_at(P, pair, i, rank, t); ++i) {
        const CUtensorMap* map_b = t.x ? &map_w : &map_x;
        const int32_t n = t.n0 + (int32_t)rank * (BN / 2);
        for (int kb = 0; kb < t.kbs; ++kb) {
          if (issued >= S && !mbar_wait_spin(&ctrl->empty[s], phase, abort)) {
            ok = false;
            break;
          }
          // the leader's barrier counts both CTAs' bytes
          const uint32_t bar = dsmem_addr(smem_u32(&ctrl->full[s]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&ctrl->full[s], 2 * P.stage_bytes);
          const uint32_t st = smem_u32(sm + (size_t)s * P.stage_bytes);
          int32_t k, plane = 0;
          if (t.x) {  // K runs over the gate's columns of dproj, then the up's
            plane = kb >= P.kb_half;
            k = (kb - (plane ? P.kb_half : 0)) * 64;
            tma_load_3d_pair(st, &map_pk, k, plane, t.m0, bar);
          } else {  // K runs over tokens
            k = kb * 64;
            tma_load_3d_pair(st, &map_pm, t.m0, t.plane, k, bar);
            tma_load_3d_pair(st + kAtom, &map_pm, t.m0 + 64, t.plane, k, bar);
          }
          for (int q = 0; q < BN / 128; ++q) tma_load_3d_pair(st + kStageA + q * kAtom, map_b, n + q * 64, k, plane, bar);
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
  } else if (warp == kEpiWarps + 1) {
    if (rank == 0 && elect_one()) {
      // K-major rows of 128 bytes; MN-major boxes of 64 columns, kAtom bytes apart, groups of 8 rows of K 1024
      const uint64_t dk = smem_desc(smem_u32(sm), 16, 1024, kSwizzle128B), dm = smem_desc(smem_u32(sm), kAtom, 1024, kSwizzle128B);
      const uint32_t k_lo = (uint32_t)dk, m_lo = (uint32_t)dm, hi = (uint32_t)(dk >> 32);
      int s = 0, tc = 0;
      uint32_t phase = 0;
      bool ok = true;
      GTile t;
      for (int64_t i = 0; ok && tile_at(P, pair, i, rank, t); ++i) {
        const uint32_t idesc = idesc_bf16_f32(2 * kRows, (uint32_t)BN, !t.x, true);
        const uint32_t a_lo = t.x ? k_lo : m_lo, a_step = t.x ? 2 : 16 * kRowBytes / 16;
        for (int from = 0; ok && from < t.kbs; ++tc) {
          const int to = kLong ? min(from + kChain, t.kbs) : t.kbs;
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
            umma_stage_steps<true>(d, a_lo + at, m_lo + (kStageA >> 4) + at, hi, hi, idesc, kb != from, a_step, 16 * kRowBytes / 16);
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
    // epilogue: warps w and w + 4 share 32 rows and take chunks of 64 columns in turn
    const int quarter = warp & 3, side = warp >> 2;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    uint8_t* ring = sm + P.off_stage + (size_t)warp * kSets * kOutBox;
    int tc = 0, used = 0;
    bool ok = true;
    GTile t;
    for (int64_t i = 0; ok && tile_at(P, pair, i, rank, t); ++i) {
      const int32_t row = t.m0 + quarter * 32;
      const int64_t rows = t.x ? P.N : P.d_ff;
      const int chunks = row < rows ? min(BN / 64, (P.d_in - t.n0 + 63) / 64) : 0;
      auto sums_ready = [&]() {
        ok = __all_sync(0xffffffffu, mbar_wait_spin(&ctrl->tfull[tc & 1], (uint32_t)(tc >> 1) & 1u, abort));
        if (ok) tc_fence_after();
        return ok;
      };
      auto sums_taken = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_read(dsmem_addr(smem_u32(&ctrl->tempty[tc & 1]), 0));
        ++tc;
      };
      // 64 columns of this warp's rows, sum(k) each, to the outputs
      auto put = [&](int c, auto sum) {
        uint8_t* box = ring + (size_t)(used & (kSets - 1)) * kOutBox;
        if (lane == 0) bulk_wait_read<kSets - 1>();  // the store that last left the box has read it
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          auto two = [&](int k) { return pack_bf16(sum(8 * q + k), sum(8 * q + k + 1)); };
          *reinterpret_cast<uint4*>(box + swz_offset((uint32_t)lane, (uint32_t)q, 128)) = make_uint4(two(0), two(2), two(4), two(6));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(t.x ? &map_dx : &map_dw, smem_u32(box), t.n0 + c * 64, row, t.plane);
          bulk_commit();
        }
        ++used;
      };
      if (kLong && t.kbs > kChain) {
        float sums[2][64];  // of this warp's chunks
#pragma unroll
        for (int k = 0; k < 64; ++k) sums[0][k] = sums[1][k] = 0.f;
        for (int left = t.kbs; left > 0 && sums_ready(); left -= kChain) {
          const uint32_t base = tmem + lanes + (uint32_t)((tc & 1) * (P.tmem_cols / 2));
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            if (side + 2 * n >= chunks) continue;
#pragma unroll
            for (int h = 0; h < 64; h += 16) {
              float r[16];
              tmem_ld16(base + (uint32_t)((side + 2 * n) * 64 + h), r);
#pragma unroll
              for (int k = 0; k < 16; ++k) sums[n][h + k] += r[k];
            }
          }
          sums_taken();
        }
        if (!ok) break;
#pragma unroll
        for (int n = 0; n < 2; ++n)
          if (side + 2 * n < chunks) put(side + 2 * n, [&](int k) { return sums[n][k]; });
      } else {
        if (!sums_ready()) break;
        const uint32_t base = tmem + lanes + (uint32_t)((tc & 1) * (P.tmem_cols / 2));
        for (int c = side; c < chunks; c += 2) {
          uint32_t r[2][32];
          tmem_ld32_start(base + (uint32_t)(c * 64), r[0]);
          tmem_ld32_start(base + (uint32_t)(c * 64 + 32), r[1]);
          tmem_ld_wait(r[0]);
          tmem_ld_bind(r[1]);
          put(c, [&](int k) { return __uint_as_float(r[k / 32][k % 32]); });
        }
        sums_taken();
      }
    }
    if (!ok) {
      *abort = 1;
      if (lane == 0) report(err_word, MOLORA_DEV_WAIT_TIMEOUT);
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  if (warp == kEpiWarps + 1 && lane == 0) mbar_wait(&ctrl->done, 0);
  __syncthreads();
  cluster_sync();  // neither CTA leaves, nor frees its TMEM, while the other may still signal or use it
  if (warp == kEpiWarps + 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, P.tmem_cols);
  }
}

// ---------------------------------------------------------------------------------------------
cudaError_t launch_gated_grad(const GatedGradArgs& a, cudaStream_t stream) {
  const cudaError_t slope = launch_gated_slope(a, stream);
  if (slope != cudaSuccess || (!a.dx && !a.dW)) return slope;
  const uint64_t N = (uint64_t)a.N, F = (uint64_t)a.d_ff, D = (uint64_t)a.d_in, half = (F + 7) & ~uint64_t(7);
  GPlan p = {};
  p.N = a.N;
  p.d_in = a.d_in;
  p.d_ff = a.d_ff;
  p.m_tiles_x = (a.N + 2 * kRows - 1) / (2 * kRows);
  p.m_tiles_w = ((int64_t)a.d_ff + 2 * kRows - 1) / (2 * kRows);
  p.kb_half = (int32_t)((F + 63) / 64);
  p.kb_x = 2 * p.kb_half;
  p.kb_w = (int32_t)((N + 63) / 64);
  p.group = 8;
  const int64_t most = num_sms() / 2;
  // A K block of a tile takes 600 cycles at 256 columns, 420 at 128.  Returns those of the longest pair.
  auto plan = [&](int BN, bool with_x, bool with_w) {
    p.BN = BN;
    p.n_tiles = (int32_t)(((int64_t)a.d_in + BN - 1) / BN);
    p.tiles_x = with_x ? p.m_tiles_x * p.n_tiles : 0;
    p.tiles_w = with_w ? 2 * p.m_tiles_w * p.n_tiles : 0;
    const int64_t tiles = p.tiles_x + p.tiles_w;
    p.pairs = (int32_t)(tiles < most ? tiles : most);
    p.full = (int32_t)(p.tiles_x % p.pairs);
    const int64_t others = p.pairs - p.full, long_as = p.kb_x / p.kb_w, share = p.tiles_w / others;
    p.ahead = p.full ? (int32_t)(long_as < share ? long_as : share) : 0;
    const int64_t rest = p.tiles_w - others * p.ahead, extra = rest % p.pairs;
    const int64_t all = p.tiles_x / p.pairs * p.kb_x + rest / p.pairs * p.kb_w;
    const int64_t of_full = p.full ? all + p.kb_x + (extra > others ? p.kb_w : 0) : 0;
    const int64_t of_others = all + (int64_t)p.ahead * p.kb_w + (extra ? p.kb_w : 0);
    return (of_full > of_others ? of_full : of_others) * (BN == 256 ? 600 : 420);
  };
  // The wider tiles where they are over first.
  auto best = [&](bool with_x, bool with_w) {
    const int64_t narrow = plan(128, with_x, with_w), wide = plan(256, with_x, with_w);
    return wide > narrow ? plan(128, with_x, with_w) : wide;
  };
  // Few tokens' dx is a few tiles of long sums: its 2 d_ff split over clusters, in a launch of its own, where that is over
  // before the tiles are (256 tokens, 1024 -> 4096: 21 us with dproj, 45 in tiles; dW too, 31 and 48).  Both uses, with dW
  // and without, are counted whichever it is, so that dx has the same bits in either.
  bool with_x = a.dx && 2 * gated_input_cycles(a) + best(false, true) >= best(true, false) + best(true, true);
#ifdef MOLORA_TUNING_ENV
  if (const char* g = getenv("MOLORA_FF_DX")) with_x = a.dx && atoi(g) != 0;
#endif
  if (a.dx && !with_x) {
    const cudaError_t input = launch_gated_input(a, stream);
    if (input != cudaSuccess || !a.dW) return input;
  }
  best(with_x, a.dW != nullptr);
  p.stage_bytes = kStageA + (uint32_t)(p.BN / 128) * kAtom;
  const uint32_t boxes = kEpiWarps * kSets * kOutBox;
  p.S = (int)((kMaxSmem - boxes - sizeof(GCtrl) - kSmemSlack) / p.stage_bytes);
  if (p.S > kMaxStages) p.S = kMaxStages;
  p.off_stage = (uint32_t)p.S * p.stage_bytes;
  p.off_ctrl = p.off_stage + boxes;
  p.tmem_cols = 2 * (uint32_t)p.BN;
  const auto BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto S128 = CU_TENSOR_MAP_SWIZZLE_128B;
  CUtensorMap pk = {}, pm = {}, w = {}, x = {}, dx = {}, dw = {};
  if (with_x && (!linear_map_3d(&pk, BF, a.dproj, {F, 2, N}, {2 * half, 4 * half}, {64, 1, 128}, S128) ||
               !linear_map_3d(&w, BF, a.W, {D, F, 2}, {2 * D, 2 * F * D}, {64, 64, 1}, S128) ||
               !linear_map_3d(&dx, BF, a.dx, {D, N, 1}, {2 * D, 2 * N * D}, {64, 32, 1}, S128)))
    return cudaErrorNotSupported;
  if (a.dW && (!linear_map_3d(&pm, BF, a.dproj, {F, 2, N}, {2 * half, 4 * half}, {64, 1, 64}, S128) ||
               !linear_map_3d(&x, BF, a.x, {D, N, 1}, {2 * D, 2 * N * D}, {64, 64, 1}, S128) ||
               !linear_map_3d(&dw, BF, a.dW, {D, F, 2}, {2 * D, 2 * F * D}, {64, 32, 1}, S128)))
    return cudaErrorNotSupported;
  auto go = [&](auto kernel, std::atomic<uint64_t>& allowed) {
    const cudaError_t set = allow_smem(kernel, allowed, kMaxSmem);
    if (set != cudaSuccess) return set;
    const dim3 grid((unsigned)(2 * p.pairs));
    // one CTA an SM, alone: an allocation of TMEM never waits for another CTA's (see linear.cu)
    return launch_kernel(kernel, grid, dim3(kThreads), kMaxSmem, stream, 2, p, a.err_word, pk, pm, w, x, dx, dw);
  };
  static std::atomic<uint64_t> allowed[2];
  const bool longer = (p.tiles_x && p.kb_x > kChain) || (p.tiles_w && p.kb_w > kChain);
  return longer ? go(grad_tc_kernel<true>, allowed[0]) : go(grad_tc_kernel<false>, allowed[1]);
}

}  // namespace molora
