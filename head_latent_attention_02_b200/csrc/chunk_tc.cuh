// chunk_tc.cuh -- attention of a ragged chunk of new tokens over expanded
// keys and values, on sm_100a tensor cores.
//
// The direct form (Day 27 tutorial "The Direct Form Explains the Meaning"): per
// head h, with K_h = W_UK[h] c and V_h = W_UV[h] c expanded once per call,
//     S[q, t] = scale * (q_nope . K_h[t] + q_rope . k_rope[t]),
//     v[q, h] = softmax_t(S masked by key_pos(t) <= q_pos(q)) V_h
// costs 2 (192 + 128) flops per query, row and head against 2 (576 + 512) in
// the absorbed form, so it is the cheaper one as soon as the expansion
// (2 * 512 * 256 flops per row and head) is shared by enough queries.
//
// Decomposition.  A CTA takes 256 consecutive tokens of one sequence and one
// head, as two query tiles of 128 rows, and walks the sequence's rows in tiles
// of 128 (two pages of the list).  S and O of both query tiles fill the 512
// tensor-memory columns; P (bf16) overwrites its S.  The tensor core works on
// one query tile while the other one's softmax runs:
//     ... P0 V | S0 | P1 V | S1 | P0 V | S0 ...
// At 192 + 128 columns a tile costs the tensor core 1280 clocks and its
// exponentials the special-function units 1024, so the products bound the
// loop as long as a tile's softmax finishes within the other tile's products.
//
// Roles (320 threads): warp 0 loads by TMA, warp 1 issues the MMAs, warps 2-5
// and 6-9 run the softmax of query tiles 0 and 1 (a thread per query row, so
// that row statistics need no exchange between threads).  The running maximum
// is only raised when it grew by more than 2^8 (the weights then stay below
// 2^8, harmless in fp32 sums and in bf16, whose precision is relative); O is
// rescaled by the softmax threads in that rare case.  S of step j is issued
// after P V of step j - 1 and its barrier covers both, so O is at rest while
// a softmax thread holds S.
//
// Every wait is bounded and records MLA_ERR_TIMEOUT when it gives up.
#pragma once
#include <cuda.h>

#include "common.cuh"
#include "ptx.cuh"
#include "gemm_tc.cuh"

namespace mla {
namespace ck {

constexpr int kDn = 128, kDr = 64, kDv = 128, kDc = 512;
constexpr int kQTile = 128, kKTile = 128;
constexpr int kItemTokens = 2 * kQTile;
constexpr int kPanel = 128 * 128;            // 128 rows x 64 bf16: 16 KB
constexpr int kQBytes = 3 * kPanel;          // a query tile: two nope panels, one rope panel
constexpr int kRing = 8;                     // panels in flight: a tile's keys take 3, its values 2
constexpr int kOffRing = 2 * kQBytes;
constexpr int kOffBar = kOffRing + kRing * kPanel;
constexpr int kSmemBytes = kOffBar + 512 + 1024;
constexpr int kThreads = 320;
constexpr int kTmemCols = 512;
constexpr int kColS = 0, kColO = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMargin = 8.0f;              // log2 units: lazy rescale margin
static_assert(kSmemBytes <= 232448, "shared memory budget");

struct Item {
  int b;         // sequence; its rows start at page entry `entry`
  int tok0, n;   // tokens [tok0, tok0 + n), n <= 256
  int entry;     // first page entry of the sequence (even)
  int tiles;     // 128-row tiles of the sequence; -1: the sequence is invalid
};

// What the planner leaves on the device.
struct Plan {
  int n_items;
  int n_row_tiles;    // 256-row tiles of the page list (the expansion's row tiles)
};

struct Params {
  const Plan* plan;
  const Item* items;
  const gm::PageEntry* pages;
  const int32_t* q_pos;
  int H, h0, n_heads;          // heads of the call; first head and heads of this launch
  long long rows_cap;          // rows per head of the key and value scratch
  float scale_log2, scale;
  __nv_bfloat16* v;            // [n_tok, H, 128]
  float* lse;                  // [n_tok, H] or null
};

// Tensor maps (64 columns, 128-byte swizzle):
//   q   (column, token, panel) over q [n_tok, H x 192], box {64, 128, 3}
//   k,v (column, row, panel) over the scratch [heads x rows_cap, 128], box {64, 128, 2}
//   kr  (column, row) over the rotary scratch [rows_cap, 64], box {64, 128}
struct Maps {
  CUtensorMap q, k, v, kr;
};

struct Bars {
  uint64_t q_full[2];
  uint64_t full[kRing], empty[kRing];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint32_t tmem_base;
  int n_tiles[2];
  int q_max[2];
};
static_assert(sizeof(Bars) <= 512, "barrier block too large");

__device__ __forceinline__ float exp2_fast(float x) { return ex2_approx(x); }

// Visible rows of one page: those with data whose position is not past qp.
__device__ __forceinline__ int visible(const gm::PageEntry& e, int qp) {
  if (e.kpos > qp) return 0;
  const long long d = (long long)qp - e.kpos + 1;
  return d < e.n ? (int)d : e.n;
}

__global__ void __launch_bounds__(kThreads, 1)
chunk_attn_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps mp) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bar = reinterpret_cast<Bars*>(smem + kOffBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // the item list and the expanded rows are complete after this wait
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if ((int)blockIdx.x >= p.plan->n_items) return;
  const Item it = p.items[blockIdx.x];
  const int hl = blockIdx.y, h = p.h0 + hl;

  if (it.tiles < 0) {      // invalid sequence: NaN
    for (int i = threadIdx.x; i < it.n * kDv; i += kThreads)
      p.v[((long long)(it.tok0 + i / kDv) * p.H + h) * kDv + i % kDv] =
          __float2bfloat16_rn(__int_as_float(0x7fc00000));
    if (p.lse)
      for (int i = threadIdx.x; i < it.n; i += kThreads)
        p.lse[(long long)(it.tok0 + i) * p.H + h] = __int_as_float(0x7fc00000);
    return;
  }

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bar->q_full[t], 1);
      mbar_init(&bar->s_full[t], 1);
      mbar_init(&bar->p_full[t], 4);
      mbar_init(&bar->o_full[t], 1);
      bar->n_tiles[t] = 0;
      bar->q_max[t] = INT32_MIN;
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&bar->full[i], 1);
      mbar_init(&bar->empty[i], 1);
    }
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&bar->tmem_base, kTmemCols);
  __syncthreads();
  // the last tile that each query tile sees: no query's position lies before it
  if (threadIdx.x < it.n) atomicMax(&bar->q_max[threadIdx.x >> 7], p.q_pos[it.tok0 + threadIdx.x]);
  __syncthreads();
  for (int j = threadIdx.x; j < it.tiles; j += kThreads) {
    const gm::PageEntry e0 = p.pages[it.entry + 2 * j], e1 = p.pages[it.entry + 2 * j + 1];
#pragma unroll
    for (int t = 0; t < 2; ++t)
      if (t * kQTile < it.n && (visible(e0, bar->q_max[t]) > 0 || visible(e1, bar->q_max[t]) > 0))
        atomicMax(&bar->n_tiles[t], j + 1);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  const int nt0 = bar->n_tiles[0], nt1 = bar->n_tiles[1];
  const int nt = max(nt0, nt1);

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    if (lane == 0 && nt > 0) {
      prefetch_tmap(&mp.q);
      prefetch_tmap(&mp.k);
      prefetch_tmap(&mp.v);
      prefetch_tmap(&mp.kr);
      const int krow = (int)(hl * p.rows_cap) + it.entry * kPage;
      auto load_q = [&](int t) {
        mbar_arrive_expect_tx(&bar->q_full[t], kQBytes);
        tma_load_3d(smem + t * kQBytes, &mp.q, &bar->q_full[t], 0, it.tok0 + t * kQTile, 3 * h);
      };
      int n = 0;
      bool ok = true;
      // panel i of tile j: i 0, 1 the keys' panels, 2 the rotary keys, 3, 4 the values'
      auto load = [&](int j, int i) {
        const int slot = n % kRing;
        if (!mbar_wait(&bar->empty[slot], ((n / kRing) & 1) ^ 1)) {
          set_status(MLA_ERR_TIMEOUT);
          return false;
        }
        uint8_t* dst = smem + kOffRing + slot * kPanel;
        mbar_arrive_expect_tx(&bar->full[slot], kPanel);
        if (i < 2) tma_load_3d(dst, &mp.k, &bar->full[slot], 0, krow + j * kKTile, i);
        else if (i == 2) tma_load_2d(dst, &mp.kr, &bar->full[slot], 0, it.entry * kPage + j * kKTile);
        else tma_load_3d(dst, &mp.v, &bar->full[slot], 0, krow + j * kKTile, i - 3);
        ++n;
        return true;
      };
      if (nt0 > 0) load_q(0);
      for (int j = 0; ok && j < nt; ++j) {
        for (int i = 0; ok && i < 5; ++i) {
          ok = load(j, i);
          if (j == 0 && i == 2 && nt1 > 0) load_q(1);
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    if (lane == 0 && nt > 0) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(kQTile, kKTile, false, false);
      constexpr uint32_t idesc_o = idesc_bf16_f32(kQTile, kDv, false, true);
      const uint32_t ring = smem_u32(smem + kOffRing);
      bool ok = true;
      auto wait = [&](uint64_t* b, uint32_t parity) {
        if (ok && !mbar_wait(b, parity)) {
          set_status(MLA_ERR_TIMEOUT);
          ok = false;
        }
      };
      // panel n of the stream of panels: tile j's keys are 5 j .. 5 j + 2, its
      // values 5 j + 3 and 5 j + 4
      auto wait_panels = [&](int n, int count) {
        for (int i = n; i < n + count; ++i) wait(&bar->full[i % kRing], (i / kRing) & 1);
        tc_fence_after();
      };
      auto free_panels = [&](int n, int count) {
        for (int i = n; i < n + count; ++i) mma_commit(&bar->empty[i % kRing]);
      };
      for (int j = 0; ok && j <= nt; ++j) {
        if (j > 0) wait_panels(5 * (j - 1) + 3, 2);
        if (j < nt) wait_panels(5 * j, 3);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int mine = t ? nt1 : nt0;
          const uint32_t s_col = tmem + kColS + t * kKTile, o_col = tmem + kColO + t * kDv;
          if (j > 0 && j - 1 < mine) {
            wait(&bar->p_full[t], (j - 1) & 1);
            tc_fence_after();
            if (!ok) break;
            // 16 rows of both 64-column value panels per step, rows outermost
            const int n0 = 5 * (j - 1) + 3;
            const uint32_t v0 = ring + (n0 % kRing) * kPanel, v1 = ring + ((n0 + 1) % kRing) * kPanel;
            // the panels' distance; the ring may put the second one first
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              if (v1 > v0) {
                mma_bf16_ts(o_col, s_col + 8 * ks, smem_desc_sw128(v0 + ks * 2048, v1 - v0, 1024),
                            idesc_o, (j > 1 || ks > 0) ? 1u : 0u);
              } else {
                constexpr uint32_t idesc_h = idesc_bf16_f32(kQTile, 64, false, true);
                mma_bf16_ts(o_col, s_col + 8 * ks, smem_desc_sw128(v0 + ks * 2048, kPanel, 1024),
                            idesc_h, (j > 1 || ks > 0) ? 1u : 0u);
                mma_bf16_ts(o_col + 64, s_col + 8 * ks,
                            smem_desc_sw128(v1 + ks * 2048, kPanel, 1024), idesc_h,
                            (j > 1 || ks > 0) ? 1u : 0u);
              }
            }
            if (j == mine) mma_commit(&bar->o_full[t]);
          }
          if (j < mine) {
            wait(&bar->q_full[t], 0);
            if (!ok) break;
            const uint32_t q0 = smem_u32(smem + t * kQBytes);
#pragma unroll
            for (int pn = 0; pn < 3; ++pn) {
              const uint32_t kb = ring + ((5 * j + pn) % kRing) * kPanel;
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                mma_bf16_ss(s_col, smem_desc_sw128(q0 + pn * kPanel + ks * 32, 16, 1024),
                            smem_desc_sw128(kb + ks * 32, 16, 1024), idesc_s,
                            (pn | ks) ? 1u : 0u);
            }
            mma_commit(&bar->s_full[t]);
          }
        }
        if (j > 0) free_panels(5 * (j - 1) + 3, 2);
        if (j < nt) free_panels(5 * j, 3);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int t = warp >= 6 ? 1 : 0;
    const int quad = warp & 3;
    const int row = quad * 32 + lane;                 // row of the query tile
    const int tok = t * kQTile + row;                 // token of the item
    const int mine = t ? nt1 : nt0;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t s_col = tmem + kColS + t * kKTile + lanes;
    const uint32_t o_col = tmem + kColO + t * kDv + lanes;
    const int qp = tok < it.n ? p.q_pos[it.tok0 + tok] : INT32_MIN;
    float m = kNegInf, l = 0.f;       // running maximum (unscaled scores), sum of weights
    bool ok = true;
    if (mine > 0) {
      const gm::PageEntry* pe = p.pages + it.entry;
      gm::PageEntry e0 = pe[0], e1 = pe[1];
      for (int j = 0; j < mine; ++j) {
        const int v0 = visible(e0, qp), v1 = visible(e1, qp);
        if (j + 1 < mine) {
          e0 = pe[2 * j + 2];
          e1 = pe[2 * j + 3];
        }
        const bool all = __all_sync(0xffffffffu, v0 == kPage && v1 == kPage);
        if (!__all_sync(0xffffffffu, mbar_wait(&bar->s_full[t], j & 1))) {
          if (lane == 0) set_status(MLA_ERR_TIMEOUT);
          ok = false;
          break;
        }
        tc_fence_after();
        float s[4][32];
        tmem_ld128_sync(s_col, s);
        if (!all) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              s[c][i] = (c & 1) * 32 + i < (c < 2 ? v0 : v1) ? s[c][i] : kNegInf;
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mx[c] = fmaxf(s[c][0], s[c][1]);
#pragma unroll
          for (int i = 2; i < 32; i += 2) mx[c] = fmaxf(mx[c], fmaxf(s[c][i], s[c][i + 1]));
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const bool raise = top * p.scale_log2 > m * p.scale_log2 + kMargin;
        if (__any_sync(0xffffffffu, raise)) {
          const float m_new = raise ? top : m;
          // nothing seen so far (m = -inf): sums and O are zero whatever the factor
          const float f = m_new == m ? 1.f : exp2_fast((m - m_new) * p.scale_log2);
          l *= f;
          m = m_new;
          if (j > 0) {
#pragma unroll 1
            for (int c = 0; c < kDv; c += 32) {
              float o[32];
              tmem_ld32_sync(o_col + c, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= f;
              tmem_st32(o_col + c, o);
            }
          }
        }
        const float off = m == kNegInf ? 0.f : -m * p.scale_log2;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float w[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int c0 = 2 * c + i / 16, i0 = 2 * (i % 16);
            const float a = exp2_fast(fmaf(s[c0][i0], p.scale_log2, off));
            const float b = exp2_fast(fmaf(s[c0][i0 + 1], p.scale_log2, off));
            sum[i & 3] += a + b;
            w[i] = __uint_as_float(gm::pack2(a, b));
          }
          tmem_st32(s_col + 32 * c, w);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->p_full[t]);
      }
      if (ok && !__all_sync(0xffffffffu, mbar_wait(&bar->o_full[t], 0))) {
        if (lane == 0) set_status(MLA_ERR_TIMEOUT);
        ok = false;
      }
      tc_fence_after();
    }
    // a query that sees no row: zero, and a log sum of -infinity
    const bool none = l == 0.f;
    const float inv = none ? 0.f : 1.f / l;
    __nv_bfloat16* o = p.v + ((long long)(it.tok0 + tok) * p.H + h) * kDv;
#pragma unroll 1
    for (int c = 0; c < kDv; c += 32) {
      float a[32];
      if (mine > 0 && ok) {
        tmem_ld32_sync(o_col + c, a);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) a[i] = 0.f;
      }
      if (tok < it.n) {
        uint4* d = reinterpret_cast<uint4*>(o + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = none ? 0u : gm::pack2(a[8 * i + 2 * k] * inv, a[8 * i + 2 * k + 1] * inv);
          d[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    if (p.lse && tok < it.n)
      p.lse[(long long)(it.tok0 + tok) * p.H + h] = none ? kNegInf : m * p.scale + logf(l);
    tc_fence_before();
  }

  __syncwarp();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace ck
}  // namespace mla
