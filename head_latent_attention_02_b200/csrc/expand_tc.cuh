// expand_tc.cuh -- keys and values of the attended rows, per head, on sm_100a
// tensor cores: K_h[t] = W_UK[h] c_t and V_h[t] = W_UV[h] c_t for the latents
// c_t (512 channels) of a page list (Day 27 tutorial "The Direct Form
// Explains the Meaning").
//
// A cluster of two CTAs computes 256 rows (four pages) x 256 columns (a head's
// 128 keys and 128 values) at a time (cta_group::2): each CTA holds its 128
// rows' latents, all 512 channels of them, in shared memory for as many heads
// as its run covers, and streams the weights: the first CTA W_UK[h], the second
// W_UV[h], each of which the pair's MMA reads for both.  A tile so loads 128 KB
// a CTA where the general tile of gemm_tc.cuh, which streams both operands,
// loads 256 KB; at 512 channels a tile lasts 4096 clocks, and 64 bytes a clock
// and SM is more than L2 delivers (8192 + 2048 rows, 128 heads: 400 us streaming
// both, 260 us this way, 1.32 PFLOP/s).  Two accumulators let the epilogue
// overlap the next tile.
//
// Roles per CTA (192 threads): warp 0 loads, warp 1 of the first CTA issues,
// warps 2-5 take 32 rows each from tensor memory through a swizzled staging
// tile to the scratch by TMA stores.
//
// Every wait is bounded and records MLA_ERR_TIMEOUT when it gives up.
#pragma once
#include <cuda.h>

#include "common.cuh"
#include "ptx.cuh"

namespace mla {
namespace ex {

constexpr int kWidth = 512, kHead = 128;
constexpr int kPanels = kWidth / 64;
constexpr int kPanelBytes = 128 * 128;        // 128 rows x 64 channels
constexpr int kStages = 5;                    // weight panels in flight
constexpr int kStageWarp = 32 * 128;          // staging: 32 rows x 64 columns a warp
constexpr int kOffW = kPanels * kPanelBytes;
constexpr int kOffStage = kOffW + kStages * kPanelBytes;
constexpr int kOffBar = kOffStage + 4 * kStageWarp;
constexpr int kSmemBytes = kOffBar + 512 + 1024;
constexpr int kThreads = 192;
constexpr int kTmemCols = 512;
// the largest finite bf16: what rounds past it is not finite either
constexpr float kMostBf16 = 3.38953139e38f;
static_assert(kSmemBytes <= 232448, "shared memory budget");

struct Params {
  const PageEntry* pages;  // four entries a row tile
  const ChunkPlan* plan;
  int n_heads;                 // heads of this launch
  long long rows_cap;          // rows per head of the scratch
  const int* norm_c;           // [sequences], see value_exponent
  const int* norm_w;           // [heads of this launch]
  uint8_t* as_half;            // [heads of this launch][rows_cap / 128]: the values' type
};

// Tensor maps (64 columns, 128-byte swizzle):
//   c       (channel, cache row), box {64, 64}
//   uk, uv  (channel, weight row) over [heads x 128, 512], box {64, 128}
//   k, v    (column, row, panel) over the scratch [heads x rows_cap, 128], box {64, 32, 1}
struct Maps {
  CUtensorMap c, uk, uv, k, v;
};

struct Bars {
  uint64_t c_full[kPanels], c_empty[kPanels];
  uint64_t w_full[kStages], w_empty[kStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t agreed;       // the epilogue warps have looked at a tile's values
  uint32_t fits[2];      // even and odd tiles: a byte a warp, 1: its values fit halves
  uint32_t tmem_base;
};
static_assert(sizeof(Bars) <= 512, "barrier block too large");

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
expand_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps mp) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bar = reinterpret_cast<Bars*>(smem + kOffBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kPanels; ++i) {
      mbar_init(&bar->c_full[i], 1);
      mbar_init(&bar->c_empty[i], 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar->w_full[i], 1);
      mbar_init(&bar->w_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->acc_full[i], 1);
      mbar_init(&bar->acc_empty[i], 8);    // four epilogue warps of each CTA
    }
    mbar_init(&bar->agreed, 4);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(&bar->tmem_base, kTmemCols);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  // the page list is complete, and the scratch no longer read, after this wait
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the pair's run of (row tile, head) tiles, heads innermost
  const int tiles = p.plan->n_row_tiles * p.n_heads;
  const int run = (tiles + pairs - 1) / pairs;
  const int u0 = min(tiles, pair * run), u1 = min(tiles, u0 + run);

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    if (lane == 0) {
      prefetch_tmap(&mp.c);
      prefetch_tmap(rank ? &mp.uv : &mp.uk);
      bool ok = true;
      auto wait = [&](uint64_t* b, int use) {
        if (!mbar_wait(b, (use & 1) ^ 1)) {
          set_status(MLA_ERR_TIMEOUT);
          ok = false;
        }
        return ok;
      };
      // the pair's bytes are counted on the first CTA's barriers
      auto expect = [&](uint64_t* b) {
        if (rank == 0) mbar_arrive_expect_tx(b, 2 * kPanelBytes);
        return mapa(smem_u32(b), 0);
      };
      int held = -1, fills = 0, n = 0;
      for (int u = u0; ok && u < u1; ++u) {
        const int mt = u / p.n_heads, h = u % p.n_heads;
        const bool fresh = mt != held;
        int y0 = 0, y1 = 0;
        if (fresh) {
          y0 = p.pages[4 * mt + 2 * rank].row;
          y1 = p.pages[4 * mt + 2 * rank + 1].row;
        }
        for (int k = 0; k < kPanels; ++k, ++n) {
          if (fresh) {
            if (!wait(&bar->c_empty[k], fills)) break;
            const uint32_t b = expect(&bar->c_full[k]);
            tma_load_2d_pair(smem + k * kPanelBytes, &mp.c, b, k * 64, y0);
            tma_load_2d_pair(smem + k * kPanelBytes + kPanelBytes / 2, &mp.c, b, k * 64, y1);
          }
          const int s = n % kStages;
          if (!wait(&bar->w_empty[s], n / kStages)) break;
          tma_load_2d_pair(smem + kOffW + s * kPanelBytes, rank ? &mp.uv : &mp.uk,
                           expect(&bar->w_full[s]), k * 64, h * kHead);
        }
        if (fresh) {
          held = mt;
          ++fills;
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    if (rank == 0) {          // the whole warp, converged
      constexpr uint32_t idesc = idesc_bf16_f32(256, 256, false, false);
      const uint64_t cd = smem_desc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t wd = smem_desc_sw128(smem_u32(smem + kOffW), 16, 1024);
      bool ok = true;
      auto wait = [&](uint64_t* b, uint32_t parity) {
        if (ok && !__all_sync(0xffffffffu, mbar_wait(b, parity))) {
          if (lane == 0) set_status(MLA_ERR_TIMEOUT);
          ok = false;
        }
      };
      int held = -1, fills = 0, n = 0;
      for (int u = u0; ok && u < u1; ++u) {
        const int mt = u / p.n_heads, ab = (u - u0) & 1;
        const bool fresh = mt != held;
        const bool leaves = u + 1 == u1 || (u + 1) / p.n_heads != mt;
        wait(&bar->acc_empty[ab], (((u - u0) >> 1) & 1) ^ 1);
        for (int k = 0; ok && k < kPanels; ++k, ++n) {
          const int s = n % kStages;
          if (fresh) wait(&bar->c_full[k], fills & 1);
          wait(&bar->w_full[s], (n / kStages) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t a = cd + k * (kPanelBytes >> 4), b = wd + s * (kPanelBytes >> 4);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_pair_bf16_ss_elect(tmem + ab * 256, a + 2 * ks, b + 2 * ks, idesc,
                                   (k | ks) ? 1u : 0u);
          mma_pair_commit_both_elect(&bar->w_empty[s]);
          if (leaves) mma_pair_commit_both_elect(&bar->c_empty[k]);
        }
        if (ok) mma_pair_commit_both_elect(&bar->acc_full[ab]);
        if (fresh) {
          held = mt;
          ++fills;
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // Rows without data are zeros (a weight of zero times NaN is NaN).  A value
    // that is not finite is stored as zero and marks the row's key as NaN
    // instead: queries that see the row get NaN, queries whose mask hides it
    // are not touched by it.  So the values are looked at first; they are written
    // last, when the CTA's four warps, whose 128 rows are one tile of the
    // attention, have agreed on their type.
    const int quad = warp & 3;
    const int row = rank * 128 + quad * 32 + lane;      // row of the pair's tile
    uint4* stage = reinterpret_cast<uint4*>(smem + kOffStage + quad * kStageWarp);
    if (lane == 0) {
      prefetch_tmap(&mp.k);
      prefetch_tmap(&mp.v);
    }
    int held = -1, norm_c = 0;
    bool live = false;
    int norm_w = u0 < u1 ? p.norm_w[u0 % p.n_heads] : 0;      // read a tile ahead
    for (int u = u0; u < u1; ++u) {
      const int mt = u / p.n_heads, h = u % p.n_heads, ab = (u - u0) & 1;
      if (mt != held) {
        const PageEntry page = p.pages[4 * mt + row / 64];
        live = row % 64 < page.n;
        norm_c = p.norm_c[page.seq];
        held = mt;
      }
      const float size = power_of_two(value_exponent(norm_c, norm_w));
      if (u + 1 < u1) norm_w = p.norm_w[h + 1 < p.n_heads ? h + 1 : 0];
      if (!__all_sync(0xffffffffu, mbar_wait(&bar->acc_full[ab], ((u - u0) >> 1) & 1))) {
        if (lane == 0) set_status(MLA_ERR_TIMEOUT);
        break;
      }
      tc_fence_after();
      const uint32_t acc = tmem + ab * 256 + ((uint32_t)(quad * 32) << 16);
      const int y = (int)(h * p.rows_cap) + mt * 256 + rank * 128 + quad * 32;
      // The row's values, scaled, and the largest and least magnitude of those that
      // are not zero.  Zeros and what is not finite are rare: they are looked for
      // only where the first pass over all values shows one.
      float val[4][32];
      tmem_ld128_sync(acc + 128, val);
      const uint64_t size2 = pack_f32x2(size, size);
      float most = 0.f, least = INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          unpack_f32x2(mul_f32x2(pack_f32x2(val[c][i], val[c][i + 1]), size2), val[c][i],
                       val[c][i + 1]);
          most = max_abs_nan(most, val[c][i], val[c][i + 1]);
          least = min_abs(least, val[c][i], val[c][i + 1]);
        }
      bool fine = true;
      if (__any_sync(0xffffffffu, live && (!(most <= kMostBf16) || least == 0.f))) {
        most = 0.f;
        least = INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float a = fabsf(val[c][i]);
            if (!(a <= kMostBf16)) {
              fine = false;
              val[c][i] = 0.f;
            } else {
              most = fmaxf(most, a);
              least = a > 0.f ? fminf(least, a) : least;
            }
          }
      }
      const bool fits =
          __all_sync(0xffffffffu, !live || (most <= kMostHalf && least >= kLeastHalf));
      if (lane == 0) {
        reinterpret_cast<volatile uint8_t*>(&bar->fits[ab])[quad] = fits;
        mbar_arrive(&bar->agreed);
      }
      // 64 columns of the warp's rows: 16-bit pairs -> staging -> scratch, 32 columns
      // (a lane's pieces 4 k to 4 k + 3) at a time
      auto begin = [&] {
        if (lane == 0) bulk_wait_read<0>();         // the last store has left the staging tile
        __syncwarp();
      };
      auto put = [&](int k, uint32_t (&w)[16]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          stage[lane * 8 + ((4 * k + i) ^ (lane & 7))] =
              live ? make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3])
                   : make_uint4(0u, 0u, 0u, 0u);
      };
      auto end = [&](const CUtensorMap* map, int c) {
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(map, stage, 0, y, c);
          bulk_commit();
        }
      };
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        begin();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float v[32];
          uint32_t w[16];
          tmem_ld32_sync(acc + 64 * c + 32 * k, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = pack2(v[2 * i], v[2 * i + 1]);
          if (c == 0 && k == 0 && !fine) w[0] = 0x7fff7fffu;        // NaN
          put(k, w);
        }
        end(&mp.k, c);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_pair(mapa(smem_u32(&bar->acc_empty[ab]), 0));
      if (!__all_sync(0xffffffffu, mbar_wait(&bar->agreed, (u - u0) & 1))) {
        if (lane == 0) set_status(MLA_ERR_TIMEOUT);
        break;
      }
      // the next such record is the other one; this one is written again only
      // when all four warps have passed that
      const bool half = *reinterpret_cast<volatile uint32_t*>(&bar->fits[ab]) == 0x01010101u;
      if (quad == 0 && lane == 0) p.as_half[(long long)h * p.rows_cap / 128 + 2 * mt + rank] = half;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        begin();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float(&v)[32] = val[2 * c + k];
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            w[i] = half ? pack2_half(v[2 * i], v[2 * i + 1]) : pack2(v[2 * i], v[2 * i + 1]);
          put(k, w);
        }
        end(&mp.v, c);
      }
    }
    if (lane == 0) bulk_wait_all();       // complete before the attention reads them
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();     // no CTA leaves while the pair's MMAs may read its shared memory
  asm volatile("griddepcontrol.launch_dependents;");
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

}  // namespace ex
}  // namespace mla
