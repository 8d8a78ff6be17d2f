// blocks_tc.cu -- many tokens times weights in e4m3, with scales for each block of 128: molora_linear_blocks, and
// molora_gated_linear's e4m3 form (see feed_forward.cu).
//
// A persistent kernel of CTA pairs as linear_tc_kernel (linear.cu) is.  Scales change with every K block of 128, so an
// accumulator in TMEM holds one K block, and the epilogue warps add it, scaled, to sums in fp32 registers while the next
// one's MMAs run.  That is one fma an element and K block, 280 cycles an SM, and as much again to read TMEM, against the
// 512 cycles of the MMAs: it fits beside them only if little else is done, and what is done one after the other (a wait,
// a load, the sums, a hand-back: 800 to 900 cycles now) is what bounds the kernel.  What it came down to, in us at
// 8192 x 4096 -> 4096 bf16 y:
//   * accumulators given back without a release, which waits for every load in flight: 331 -> 218
//   * x's scales gathered ahead into shared memory by two warps of their own (they lie token by token, 32 lines of L1 a
//     warp and K block), registers enough for the warp that issues the MMAs: 218 -> 129
//   * few instructions in the loop (addresses that flip by xor, one vote a wait, fmas in pairs), loads of 32 columns
//     with the next under way, a box for every piece a tile's outputs leave by: 129 -> 121
//   * no register spilled (a piece's columns by a constant offset, not a table): 121 -> 112 (103 without a residual)
//   * the bias by way of shared memory, no work on pieces that are not there, kernels of their own for rows that TMA cannot
//     write (nothing spilled): 113.8 -> 110.8; such rows 16 at a time without a branch for each: fp32 5000 x 2064 -> 4097
//     145 -> 107, those of the last tokens too: 1237 x 2064 -> 1541 19.4 -> 15.9; the first scales gathered by the eight
//     warps that wait for them: 1024 x 4096 -> 1024 14.5 -> 13.8
// A product without scales takes 76: the finishing of a tile (1 to 2 us, under which the next tile's first two K
// blocks run, then the tensor cores wait) and the chain above are the difference.
// Tried and left: four warps a scheduler with half the sums each (126); accumulators in halves of 128 columns, which the
// tensor cores make less quickly (141); four accumulators with tiles of 128 columns (1024 x 4096 -> 1024 13.3 -> 13.9: it is
// not the way to and fro); loads of 64 columns (118); the next K block's scales, or the look whether it is there, before the
// last sums (123, 131: more registers than there are); the residual asked for in mid-tile (115).
#include <cudaTypedefs.h>

#include <atomic>

#include "feed_forward.cuh"

namespace molora {

namespace {

constexpr int kSides = 2, kWarps = 4 * kSides;   // epilogue warps: groups of four share 32 rows each
constexpr int kThreadsB = 32 * (kWarps + 4);     // + TMA warp, MMA warp, two that gather scales
// 128 sums a thread, 64 more on their way from TMEM and what the epilogue works with take more than the 168 registers that
// 384 threads are launched with, so the last warpgroup gives up its own: 256 x 232 + 128 x 40 = 384 x 168.
constexpr int kEpiRegisters = 232, kOtherRegisters = 40;

// The scales of kScaleSpan K blocks of a tile: for each K block the 4 pieces' of each side, and the CTA's 128 tokens'; and
// what is added to the tile's columns.
constexpr int kScaleSpan = 16, kScaleStride = kRows + 1;
struct __align__(16) Scales {
  float w[kScaleSpan][8];
  float bias[256];     // (a tile's last span's)
  float x[kScaleSpan * kScaleStride];
};

struct __align__(16) BCtrl {
  uint64_t tfull[2];   // (one's address and the other's differ in one bit)
  uint64_t tempty[2];
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t sfull[2];
  uint64_t sempty[2];
  uint64_t done;
  uint64_t res_full[kWarps];
  uint32_t tmem_base;
  int32_t abort;
};

struct BPlan {
  int BN;                // rows of W a tile
  int S;                 // stages
  int nkb;               // K blocks of 128
  int group;             // token tiles per group of tiles (they share W's rows in L2)
  // (32 bits: 2^27 tiles would be an output of 10^13 bytes)
  int32_t m_tiles, n_tiles, tiles;
  uint32_t box;          // bytes of staging a warp
  uint32_t stage_bytes, off_b, off_stage, off_scales, off_ctrl, tmem_cols, smem;
};

// The h-th piece of 32 columns of a side's warps: its columns of TMEM from the side's first (side * 32), and of the outputs
// from the tile's first.  Gated, pieces come in pairs, of the gate's rows of W and the up projection's.
template <bool kGated>
__device__ __forceinline__ uint32_t piece_column(const BPlan& P, int h) {
  return kGated ? (h & 1) * ((uint32_t)P.BN / 2) + (h >> 1) * kSides * 32 : h * kSides * 32;
}
template <bool kGated>
__device__ __forceinline__ int piece_output(int side, int h) {
  return (side + kSides * (kGated ? h >> 1 : h)) * 32;
}

// max(a, b, c), NaN if any is
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// SiLU, and the tanh form of GELU, of 32 values v / (1 + 2^z) (see activate) with one reciprocal for two: 1 / a = b / (a b).
// A tile's activations are not under any MMA here, and their powers and reciprocals are what bounds them (gated 4096 x
// 2048 -> 6144 96.0 -> 93.9 us).  A pair whose product passes 2^125 (SiLU: v that sum to less than -86) or is NaN has a
// reciprocal each, in a branch of its own, which costs less than limits on every z (8192 x 1024 -> 1541 bf16, tanh, 54.8 -> 52.6
// us; gated 8192 x 1024 -> 1024 24.4 -> 24.6).  A value's last bits depend on its pair, and on nothing else.
__device__ __forceinline__ void activate_pairs(float (&v)[32], bool silu) {
  constexpr float kMost = 0x1p125f;  // (its reciprocal is a normal number)
  float d[32], p[16];
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const float x = v[i], z = silu ? -1.4426950408889634f * x : x * fmaf(-0.10294324f * x, x, -2.3022082f);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d[i]) : "f"(z));
    d[i] += 1.f;
    if (i & 1) p[i / 2] = d[i - 1] * d[i];
  }
  auto over = [](float a) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
    return r;
  };
  float most[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) most[i] = max_nan(p[3 * i], p[3 * i + 1], p[3 * i + 2]);
  most[0] = max_nan(most[0], most[1], most[2]);
  most[0] = max_nan(most[0], max_nan(most[3], most[4], p[15]), most[0]);
  if (most[0] < kMost) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float r = over(p[i]);
      v[2 * i] *= r * d[2 * i + 1];
      v[2 * i + 1] *= r * d[2 * i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const bool one = p[i] < kMost;
      const float r0 = over(one ? p[i] : d[2 * i]), r1 = over(one ? p[i] : d[2 * i + 1]);
      v[2 * i] *= one ? r0 * d[2 * i + 1] : r0;
      v[2 * i + 1] *= one ? r1 * d[2 * i] : r1;
    }
  }
}

}  // namespace

// kTma: y (and the residual) move by TMA.
template <bool kGated, bool kY16, bool kTma>
__global__ void __launch_bounds__(kThreadsB, 1)
    blocks_tc_kernel(const FEpi E, const BPlan P, int32_t* err_word, const __grid_constant__ CUtensorMap map_x,
                     const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_y,
                     const __grid_constant__ CUtensorMap map_r) {
  constexpr int kOut = kGated ? 2 : 4;               // output pieces of 32 columns a warp
  constexpr int kParts = kY16 ? 1 : 2;               // one's boxes: 32 rows of 64 bytes
  constexpr uint32_t kPiece = kParts * kBox;
  constexpr int kRound = kY16 ? kOut : 2;            // pieces that leave together
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  BCtrl* ctrl = reinterpret_cast<BCtrl*>(sm + P.off_ctrl);
  // (the warp's number, and the like, from lane 0: in uniform registers)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int BN = P.BN, S = P.S, nkb = P.nkb, width = kGated ? BN / 2 : BN;  // outputs a tile
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
      mbar_init(&ctrl->sfull[b], 64);
      mbar_init(&ctrl->sempty[b], kWarps);
    }
    mbar_init(&ctrl->done, 1);
    for (int b = 0; b < kWarps; ++b) mbar_init(&ctrl->res_full[b], 1);
    ctrl->abort = 0;
    mbar_fence_init();
    tma_prefetch_desc(&map_x);
    tma_prefetch_desc(&map_w);
    if (kTma) tma_prefetch_desc(&map_y);
    if (E.tma_res) tma_prefetch_desc(&map_r);
  }
  pdl_wait();
  if (warp < kWarps) {  // the first span of scales, by all the warps that would wait for it
    int32_t m0, n0;
    tile_at(pair, m0, n0);
    Scales* to = reinterpret_cast<Scales*>(sm + P.off_scales);
    const int k = tid & 15, c = tid >> 4, col = n0 + piece_output<kGated>(c >> 2, c & 3);
    if (k < nkb) {
      for (int r = c; r < kRows && m0 + r < E.N; r += 2 * kWarps)
        cp_async_4(smem_u32(to->x + k * kScaleStride + r), E.sx + (int64_t)(m0 + r) * nkb + k);
      if (c < 8 && col < E.d_out)
        cp_async_4(smem_u32(&to->w[k][c]), E.sw + (int64_t)(col / 128 + (kGated && (c & 1) ? E.up : 0)) * nkb + k);
    }
    if (!kGated && E.bias && nkb <= kScaleSpan && tid < width) {
      const bool in = n0 + tid < E.d_out;  // (the others are 0, as activations go by pairs)
      cp_async_4(smem_u32(&to->bias[tid]), E.bias + (in ? n0 + tid : 0), in ? 4 : 0);
    }
  }
  __syncthreads();
  // only now, with this CTA's TMEM held, may the next kernel's CTAs come and ask for theirs
  pdl_launch_dependents();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctrl->tmem_base, 0);
  cluster_sync();  // every CTA's barriers are initialised before another signals them

  if (warp >= kWarps) {
    registers_down<kOtherRegisters>();
    if (warp == kWarps && elect_one()) {
      int s = 0, issued = 0;
      uint32_t phase = 1;  // the first use of a stage finds it empty
      bool ok = true;
      for (int32_t pt = pair; pt < P.tiles && ok; pt += pairs) {
        int32_t m0, n0;
        tile_at(pt, m0, n0);
        // the pair's halves of the MMA's columns: gated, one CTA brings rows of Wg and the other of Wu
        const int32_t n = kGated ? n0 + (int32_t)rank * E.d_out : n0 + (int32_t)rank * (BN / 2);
        for (int kb = 0; kb < nkb; ++kb) {
          if (issued >= S && !mbar_wait_spin(&ctrl->empty[s], phase, abort)) {
            ok = false;
            break;
          }
          // the leader's barrier counts both CTAs' bytes
          const uint32_t bar = dsmem_addr(smem_u32(&ctrl->full[s]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&ctrl->full[s], 2 * P.stage_bytes);
          uint8_t* st = sm + (size_t)s * P.stage_bytes;
          tma_load_2d_pair(smem_u32(st), &map_x, kb * 128, m0, bar);
          tma_load_2d_pair(smem_u32(st + P.off_b), &map_w, kb * 128, n, bar);
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
    if (warp == kWarps + 1 && rank == 0 && elect_one()) {
      const uint32_t idesc = idesc_e4m3_f32(2 * kRows, (uint32_t)BN);
      const uint64_t da = smem_desc(smem_u32(sm), 16, 1024, kSwizzle128B);
      const uint64_t db = smem_desc(smem_u32(sm + P.off_b), 16, 1024, kSwizzle128B);
      const uint32_t a_lo = (uint32_t)da, b_lo = (uint32_t)db, desc_hi = (uint32_t)(da >> 32);
      int s = 0, tc = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int32_t pt = pair; pt < P.tiles && ok; pt += pairs) {
        for (int kb = 0; kb < nkb && ok; ++kb, ++tc) {
          const int buf = tc & 1;
          if (tc >= 2 && !(ok = mbar_wait_spin(&ctrl->tempty[buf], (uint32_t)((tc >> 1) - 1) & 1u, abort))) break;
          if (!(ok = mbar_wait_spin(&ctrl->full[s], phase, abort))) break;
          tc_fence_after();
          const uint32_t at = (uint32_t)s * (P.stage_bytes >> 4);
          umma_stage<true, true>(tmem + (uint32_t)buf * (P.tmem_cols / 2), a_lo + at, b_lo + at, desc_hi, desc_hi, idesc, 0);
          umma_commit_pair(&ctrl->tfull[buf], both);
          umma_commit_pair(&ctrl->empty[s], both);
          if (++s == S) s = 0, phase ^= 1;
        }
      }
      if (!ok) report(err_word, MOLORA_DEV_WAIT_TIMEOUT);
      umma_commit_pair(&ctrl->done, both);  // arrives in both CTAs once every MMA has completed
    }
    if (warp >= kWarps + 2) {  // the scales: 16 lanes a token, a K block each
      const int l = (warp - kWarps - 2) * 32 + lane, k = l & 15;
      int n = 0;
      bool ok = true;
      for (int32_t pt = pair; pt < P.tiles && ok; pt += pairs) {
        int32_t m0, n0;
        tile_at(pt, m0, n0);
        for (int kb = 0; kb < nkb; kb += kScaleSpan, ++n) {
          if (n >= 2 && !mbar_wait_spin(&ctrl->sempty[n & 1], (uint32_t)((n >> 1) - 1) & 1u, abort)) {
            ok = false;
            break;
          }
          Scales* to = reinterpret_cast<Scales*>(sm + P.off_scales) + (n & 1);
          if (n > 0 && kb + k < nkb) {  // (the first span: above)
            for (int r = l >> 4; r < kRows && m0 + r < E.N; r += 4)
              cp_async_4(smem_u32(to->x + k * kScaleStride + r), E.sx + (int64_t)(m0 + r) * nkb + kb + k);
            for (int c = l >> 4; c < 8; c += 4) {  // piece c & 3 of side c / 4
              const int32_t col = n0 + piece_output<kGated>(c >> 2, c & 3);
              if (col < E.d_out)
                cp_async_4(smem_u32(&to->w[k][c]), E.sw + (int64_t)(col / 128 + (kGated && (c & 1) ? E.up : 0)) * nkb + kb + k);
            }
          }
          if (!kGated && E.bias && n > 0 && kb + kScaleSpan >= nkb)
            for (int c = l; c < width; c += 64) {
              const bool in = n0 + c < E.d_out;
              cp_async_4(smem_u32(&to->bias[c]), E.bias + (in ? n0 + c : 0), in ? 4 : 0);
            }
          cp_async_mbar_arrive(&ctrl->sfull[n & 1]);
        }
      }
      cp_async_wait_all();
    }
    __syncwarp();
  } else {
    registers_up<kEpiRegisters>();
    cp_async_wait_all();
    named_barrier(1, 32 * kWarps);
    const int quarter = warp & 3, side = warp >> 2;
    uint8_t* box = sm + P.off_stage + (size_t)warp * P.box;
    const uint32_t tempty = dsmem_addr(smem_u32(&ctrl->tempty[0]), 0), tfull = smem_u32(&ctrl->tfull[0]);
    const uint32_t first = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)side * 32;  // this warp's columns of an accumulator
    int tc = 0, spans = 0;     // accumulators, and spans of scales, done with
    int asked = 0, taken = 0;  // rounds of the residual on their way or taken, and taken
    bool ok = true;
    for (int32_t pt = pair; pt < P.tiles && ok; pt += pairs) {
      int32_t m0, n0;
      tile_at(pt, m0, n0);
      m0 += quarter * 32;
      // output piece o's first column; it is the outputs' where that is below d_out, in the tile and for rows that are there
      auto column = [&](int o) { return n0 + piece_output<kGated>(side, kGated ? 2 * o : o); };
      auto there = [&](int o) { return column(o) < n0 + width && column(o) < E.d_out && m0 < E.N; };
      // the residual's pieces of a round come into the boxes that the outputs' leave from
      auto ask = [&](int round) {
        if (lane == 0) {
          bulk_wait_read<0>();  // the last stores have read the boxes
          uint32_t bytes = 0;
#pragma unroll
          for (int o = 0; o < kRound; ++o) bytes += there(round * kRound + o) ? kPiece : 0u;
          mbar_arrive_expect_tx(&ctrl->res_full[warp], bytes);
#pragma unroll
          for (int o = 0; o < kRound; ++o)
            if (there(round * kRound + o))
              for (int q = 0; q < kParts; ++q)
                tma_load_2d(smem_u32(box + o * kPiece + q * kBox), &map_r, column(round * kRound + o) + q * 16, m0, &ctrl->res_full[warp]);
        }
        ++asked;
      };
      if (!kGated && kTma && E.tma_res) ask(0);
      float acc[4][32];
#pragma unroll
      for (int h = 0; h < 4; ++h)
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[h][i] = 0.f;
      // K blocks of a span of scales, with as few instructions as they come down to
      auto add_span = [&](auto count, int blocks, uint32_t sx, uint32_t sw) {
        constexpr int kPieces = decltype(count)::value;
        uint32_t buf = (uint32_t)tc & 1u, parity = (uint32_t)(tc >> 1) & 1u;
        const uint32_t flip = P.tmem_cols / 2;
        uint32_t from = first + buf * flip, full_at = tfull + buf * 8, free_at = tempty + buf * 8;
        tc += blocks;
        for (; blocks > 0; --blocks, sx += kScaleStride * 4, sw += 32) {
          const float row = lds_f32(sx);
          const float4 w = lds_f32x4(sw);
          if (!mbar_try_wait_all(full_at, parity)) {
            ok = __all_sync(0xffffffffu, mbar_wait_spin(&ctrl->tfull[buf], parity, abort));
            if (!ok) return;
          }
          tc_fence_after();
          // a piece is on its way from TMEM while the one before it is added
          uint32_t r[2][32];
          tmem_ld32_start(from + piece_column<kGated>(P, 0), r[0]);
#pragma unroll
          for (int h = 0; h < kPieces; ++h) {
            tmem_ld_wait(r[h & 1]);
            if (h + 1 < kPieces) {
              tmem_ld32_start(from + piece_column<kGated>(P, h + 1), r[(h + 1) & 1]);
            } else {
              tc_fence_before();
              if (lane == 0) mbar_arrive_cluster_read(free_at);
            }
            const float scale = row * (h == 0 ? w.x : h == 1 ? w.y : h == 2 ? w.z : w.w);
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              fma_pair(acc[h][i], acc[h][i + 1], __uint_as_float(r[h & 1][i]), __uint_as_float(r[h & 1][i + 1]), scale);
          }
          parity ^= buf, buf ^= 1;
          from = first + (buf ? flip : 0u), full_at ^= 8, free_at ^= 8;
        }
      };
      for (int kb = 0; kb < nkb && ok; kb += kScaleSpan, ++spans) {
        ok = __all_sync(0xffffffffu, mbar_wait_spin(&ctrl->sfull[spans & 1], (uint32_t)(spans >> 1) & 1u, abort));
        if (!ok) break;
        const uint32_t sw = smem_u32(sm + P.off_scales) + (spans & 1) * (uint32_t)sizeof(Scales) + side * 16;
        const uint32_t sx = sw - side * 16 + (uint32_t)offsetof(Scales, x) + (quarter * 32 + lane) * 4;
        const int blocks = min(nkb - kb, kScaleSpan);
        if (BN == 256 || (kGated && BN == 192 && side == 0))
          add_span(std::integral_constant<int, 4>{}, blocks, sx, sw);
        else if (!kGated && BN == 192)
          add_span(std::integral_constant<int, 3>{}, blocks, sx, sw);
        else
          add_span(std::integral_constant<int, 2>{}, blocks, sx, sw);
        __syncwarp();
        if (lane == 0 && (kGated || kb + kScaleSpan < nkb)) mbar_arrive(&ctrl->sempty[spans & 1]);
      }
      if (!ok) break;
      if constexpr (kGated) {
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          if (E.act == MOLORA_ACT_SILU)
            activate_pairs(acc[2 * o], true);
          else if (E.act == MOLORA_ACT_GELU_TANH)
            activate_pairs(acc[2 * o], false);
          else
            apply_act(acc[2 * o], E.act);
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[o][i] = acc[2 * o][i] * acc[2 * o + 1][i];
        }
      } else {
        const uint32_t bias = smem_u32(&(reinterpret_cast<Scales*>(sm + P.off_scales) + ((spans - 1) & 1))->bias[side * 32]);
        if (E.bias || E.act != MOLORA_ACT_NONE) {
#pragma unroll
          for (int o = 0; o < 4; ++o) {
            if (!there(o)) continue;
            if (E.bias) {
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 b = lds_f32x4(bias + (o * kSides * 32 + i) * 4);
                acc[o][i] += b.x, acc[o][i + 1] += b.y, acc[o][i + 2] += b.z, acc[o][i + 3] += b.w;
              }
            }
            if (E.act == MOLORA_ACT_SILU || E.act == MOLORA_ACT_GELU_TANH)
              activate_pairs(acc[o], E.act == MOLORA_ACT_SILU);
            else
              apply_act(acc[o], E.act);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->sempty[(spans - 1) & 1]);
      }
      if constexpr (kTma) {
        auto chunk = [&](int o, int i) { return box + o * kPiece + (i >> 2) * kBox + swz_offset((uint32_t)lane, (uint32_t)i & 3u, 64); };
#pragma unroll
        for (int round = 0; round < kOut / kRound; ++round) {
          if (!kGated && kTma && E.tma_res) {
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&ctrl->res_full[warp], (uint32_t)taken & 1u)))) break;
            ++taken;
#pragma unroll
            for (int o = 0; o < kRound; ++o) {
              float(&v)[32] = acc[round * kRound + o];
              if (!there(round * kRound + o)) continue;
#pragma unroll
              for (int i = 0; i < 4 * kParts; ++i) {
                const uint4 q = *reinterpret_cast<const uint4*>(chunk(o, i));
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
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
            }
          } else {
            if (lane == 0) bulk_wait_read<0>();  // the last stores have read the boxes
            __syncwarp();
          }
#pragma unroll
          for (int o = 0; o < kRound; ++o) {
            const float(&v)[32] = acc[round * kRound + o];
#pragma unroll
            for (int i = 0; i < 4 * kParts; ++i) {
              uint4 q;
              if constexpr (kY16)
                q = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                               pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
              else
                q = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                               __float_as_uint(v[4 * i + 3]));
              *reinterpret_cast<uint4*>(chunk(o, i)) = q;
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
#pragma unroll
            for (int o = 0; o < kRound; ++o)
              if (there(round * kRound + o))
                for (int q = 0; q < kParts && column(round * kRound + o) + q * 16 < E.d_out; ++q)
                  tma_store_2d(&map_y, smem_u32(box + o * kPiece + q * kBox), column(round * kRound + o) + q * 16, m0);
            bulk_commit();
          }
          if (!kGated && kTma && E.tma_res && round + 1 < kOut / kRound) ask(round + 1);
        }
      } else {
        // rows that are not 16-byte aligned: turned in shared memory, written a row at a time, 16 rows' residuals on their way
        // together
        float* turned = reinterpret_cast<float*>(box);
        const int rows = E.N - m0 < 32 ? (int)(E.N - m0) : 32;
        auto residual = [&](int64_t at) {
          if constexpr (kGated)
            return 0.f;
          else if constexpr (kY16)
            return to_float(static_cast<const __nv_bfloat16*>(E.res)[at]);
          else
            return static_cast<const float*>(E.res)[at];
        };
        auto put = [&](int64_t at, float v) {
          if constexpr (kY16)
            static_cast<__nv_bfloat16*>(E.y)[at] = __float2bfloat16_rn(v);
          else
            static_cast<float*>(E.y)[at] = v;
        };
        const bool res = !kGated && E.res;
        auto write = [&](auto all, int64_t to) {
#pragma unroll 1
          for (int q0 = 0; q0 < rows; q0 += 16, to += 16 * (int64_t)E.d_out) {
            auto in = [&](int q) { return decltype(all)::value || q0 + q < rows; };
            float v[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) v[q] = res && in(q) ? residual(to + q * (int64_t)E.d_out) : 0.f;
#pragma unroll
            for (int q = 0; q < 16; ++q) v[q] += turned[(q0 + q) * 32 + (lane ^ (q0 + q))];
#pragma unroll
            for (int q = 0; q < 16; ++q)
              if (in(q)) put(to + q * (int64_t)E.d_out, v[q]);
          }
        };
#pragma unroll
        for (int o = 0; o < kOut; ++o) {
          if (!there(o)) continue;
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 32; ++i) turned[lane * 32 + (i ^ lane)] = acc[o][i];
          __syncwarp();
          if (column(o) + lane >= E.d_out) continue;
          const int64_t to = (int64_t)m0 * E.d_out + column(o) + lane;
          if (rows == 32)
            write(std::true_type{}, to);
          else if (res)
            write(std::false_type{}, to);
          else
            for (int q = 0; q < rows; ++q) put(to + q * (int64_t)E.d_out, turned[q * 32 + (lane ^ q)]);
        }
      }
    }
    if (!ok) {
      // no copy is left in flight
      if (taken < asked) mbar_wait(&ctrl->res_full[warp], (uint32_t)taken & 1u);
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

cudaError_t launch_blocks_tc(const FeedForwardArgs& a, int BN, cudaStream_t stream) {
  FEpi e = ff_epilogue_of(a);
  BPlan p = {};
  const int width = a.gated ? BN / 2 : BN;
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
  p.tmem_cols = tmem_columns(2 * (uint32_t)(BN <= 128 ? 128 : 256));
  CUtensorMap mx, mw, my = {}, mr = {};
  auto rows_map = [&](CUtensorMap* m, const void* base) {
    return linear_map(m, a.y_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.y_bf16 ? 2 : 4, base,
                      (uint64_t)a.N, (uint64_t)a.d_out, a.y_bf16 ? 32 : 16, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  };
  if (e.tma_y && (!rows_map(&my, a.y) || (a.residual && !rows_map(&mr, a.residual)))) e.tma_y = false;
  e.tma_res = e.tma_y && a.residual;
  p.box = (a.gated ? 2 : 4) * kBox;  // all of a tile's pieces of bf16, half of them of fp32
  static_assert(kTurn <= 2 * kBox, "a warp's boxes hold a turned piece");
  const size_t boxes = (size_t)kWarps * p.box, fixed = boxes + 2 * sizeof(Scales) + sizeof(BCtrl) + kSmemSlack;
  p.S = (int)((kMaxSmem - fixed) / p.stage_bytes);
  if (p.S > kMaxStages) p.S = kMaxStages;
  p.off_stage = (uint32_t)p.S * p.stage_bytes;
  p.off_scales = p.off_stage + (uint32_t)boxes;
  p.off_ctrl = p.off_scales + 2 * (uint32_t)sizeof(Scales);
  // one CTA an SM, alone: an allocation of TMEM never waits for another CTA's (see linear.cu)
  p.smem = kMaxSmem;
  if (!ff_operand_map(&mx, a, a.x, a.N, kRows) || !ff_operand_map(&mw, a, a.W, ff_rows_of_w(a), (uint32_t)(BN / 2)))
    return cudaErrorNotSupported;
  auto go = [&](auto kernel, std::atomic<uint64_t>& allowed) {
    const cudaError_t set = allow_smem(kernel, allowed, kMaxSmem);
    if (set != cudaSuccess) return set;
    const int32_t most = num_sms() / 2;
    const dim3 grid((unsigned)(2 * (p.tiles < most ? p.tiles : most)));
    return launch_kernel(kernel, grid, dim3(kThreadsB), p.smem, stream, 2, e, p, a.err_word, mx, mw, my, mr);
  };
  static std::atomic<uint64_t> allowed[6];
  if (a.gated) return e.tma_y ? go(blocks_tc_kernel<true, true, true>, allowed[0]) : go(blocks_tc_kernel<true, true, false>, allowed[1]);
  if (a.y_bf16) return e.tma_y ? go(blocks_tc_kernel<false, true, true>, allowed[2]) : go(blocks_tc_kernel<false, true, false>, allowed[3]);
  return e.tma_y ? go(blocks_tc_kernel<false, false, true>, allowed[4]) : go(blocks_tc_kernel<false, false, false>, allowed[5]);
}

}  // namespace molora
