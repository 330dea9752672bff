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
constexpr int kSlot = 2 * kPanel;            // a tile's keys (without the rotary part) or its values
constexpr int kSlots = 3, kRotSlots = 2;
constexpr int kOffRing = 2 * kQBytes;
constexpr int kOffRot = kOffRing + kSlots * kSlot;
constexpr int kOffBar = kOffRot + kRotSlots * kPanel;
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
//   k,v (column, row, panel) over the scratch [heads x rows_cap, 128], box
//       {64, 128, 2}: two 64-column panels of 16 KB
//   kr  (column, row) over the rotary scratch [rows_cap, 64], box {64, 128}
struct Maps {
  CUtensorMap q, k, v, kr;
};

struct Bars {
  uint64_t q_full[2];
  uint64_t full[kSlots], empty[kSlots];        // keys of tile 0, values of tile 0, keys of tile 1, ...
  uint64_t rot_full[kRotSlots], rot_empty[kRotSlots];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint32_t tmem_base;
  int n_tiles[2];
  int q_max[2], q_min[2];
  int n_full[2];               // leading tiles that every query of the tile sees whole
};
static_assert(sizeof(Bars) <= 512, "barrier block too large");

// max that keeps NaN (fmaxf drops it): a NaN score makes the row's maximum, and
// with it the whole row, NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

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
      bar->q_min[t] = INT32_MAX;
      bar->n_full[t] = INT32_MAX;
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&bar->full[i], 1);
      mbar_init(&bar->empty[i], 1);
    }
    for (int i = 0; i < kRotSlots; ++i) {
      mbar_init(&bar->rot_full[i], 1);
      mbar_init(&bar->rot_empty[i], 1);
    }
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&bar->tmem_base, kTmemCols);
  __syncthreads();
  // the tiles that each query tile needs (up to the last one that any of its
  // queries sees) and the leading ones that need no mask
  if (threadIdx.x < it.n) {
    const int qp = p.q_pos[it.tok0 + threadIdx.x];
    atomicMax(&bar->q_max[threadIdx.x >> 7], qp);
    atomicMin(&bar->q_min[threadIdx.x >> 7], qp);
  }
  __syncthreads();
  for (int j = threadIdx.x; j < it.tiles; j += kThreads) {
    const gm::PageEntry e0 = p.pages[it.entry + 2 * j], e1 = p.pages[it.entry + 2 * j + 1];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (t * kQTile >= it.n) continue;
      if (visible(e0, bar->q_max[t]) > 0 || visible(e1, bar->q_max[t]) > 0)
        atomicMax(&bar->n_tiles[t], j + 1);
      if (visible(e0, bar->q_min[t]) < kPage || visible(e1, bar->q_min[t]) < kPage)
        atomicMin(&bar->n_full[t], j);
    }
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
      bool ok = true;
      auto wait = [&](uint64_t* b, int use) {      // the slot's use-th filling may start
        if (!mbar_wait(b, (use & 1) ^ 1)) {
          set_status(MLA_ERR_TIMEOUT);
          ok = false;
        }
        return ok;
      };
      auto load = [&](const CUtensorMap* map, int n, int row) {
        const int slot = n % kSlots;
        if (!wait(&bar->empty[slot], n / kSlots)) return;
        mbar_arrive_expect_tx(&bar->full[slot], kSlot);
        tma_load_3d(smem + kOffRing + slot * kSlot, map, &bar->full[slot], 0, row, 0);
      };
      if (nt0 > 0) load_q(0);
      for (int j = 0; ok && j < nt; ++j) {
        load(&mp.k, 2 * j, krow + j * kKTile);
        const int rs = j % kRotSlots;
        if (!ok || !wait(&bar->rot_empty[rs], j / kRotSlots)) break;
        mbar_arrive_expect_tx(&bar->rot_full[rs], kPanel);
        tma_load_2d(smem + kOffRot + rs * kPanel, &mp.kr, &bar->rot_full[rs], 0,
                    it.entry * kPage + j * kKTile);
        if (j == 0 && nt1 > 0) load_q(1);
        load(&mp.v, 2 * j + 1, krow + j * kKTile);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    if (lane == 0 && nt > 0) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(kQTile, kKTile, false, false);
      constexpr uint32_t idesc_o = idesc_bf16_f32(kQTile, kDv, false, true);
      // Descriptors of the first panels; a panel, a slot or a K step further is
      // an addition (16-byte units) that never leaves the address field.  The
      // issuing thread shares its scheduler with softmax warps: building each
      // descriptor anew cost it 1400 clocks for the eight MMAs of a P V.
      const uint64_t dq = smem_desc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t dk = smem_desc_sw128(smem_u32(smem + kOffRing), 16, 1024);
      const uint64_t dr = smem_desc_sw128(smem_u32(smem + kOffRot), 16, 1024);
      // values: 16 rows of both 64-column panels per step, rows outermost
      const uint64_t dv = smem_desc_sw128(smem_u32(smem + kOffRing), kPanel, 1024);
      bool ok = true;
      auto wait = [&](uint64_t* b, uint32_t parity) {
        if (ok && !mbar_wait(b, parity)) {
          set_status(MLA_ERR_TIMEOUT);
          ok = false;
        }
      };
      for (int j = 0; ok && j <= nt; ++j) {
        const int kn = 2 * j, vn = 2 * j - 1;      // their places in the stream of slots
        const int ks_n = kn % kSlots, vs_n = vn < 0 ? 0 : vn % kSlots;   // and their slots
        if (j > 0) wait(&bar->full[vs_n], (vn / kSlots) & 1);
        if (!ok) break;
        const uint64_t kd = dk + ks_n * (kSlot >> 4), vd = dv + vs_n * (kSlot >> 4);
        const uint64_t rd = dr + (j % kRotSlots) * (kPanel >> 4);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int mine = t ? nt1 : nt0;
          const uint32_t s_col = tmem + kColS + t * kKTile, o_col = tmem + kColO + t * kDv;
          if (j > 0 && j - 1 < mine) {
            wait(&bar->p_full[t], (j - 1) & 1);
            tc_fence_after();
            if (!ok) break;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              mma_bf16_ts(o_col, s_col + 8 * ks, vd + ks * (2048 >> 4), idesc_o,
                          (j > 1 || ks > 0) ? 1u : 0u);
            if (j == mine) mma_commit(&bar->o_full[t]);
          }
          // both query tiles are done with the values: their slot takes the
          // keys of the next step, whose load needs all the time it can get
          if (t == 1 && j > 0) mma_commit(&bar->empty[vs_n]);
          if (j < mine) {
            if (t == 0 || nt0 <= j) {      // the first query tile of the step
              wait(&bar->full[ks_n], (kn / kSlots) & 1);
              wait(&bar->rot_full[j % kRotSlots], (j / kRotSlots) & 1);
            }
            if (j == 0) wait(&bar->q_full[t], 0);
            tc_fence_after();
            if (!ok) break;
            const uint64_t qd = dq + t * (kQBytes >> 4);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              const uint32_t at = (ks >> 2) * (kPanel >> 4) + (ks & 3) * 2;
              mma_bf16_ss(s_col, qd + at, kd + at, idesc_s, ks ? 1u : 0u);
            }
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_bf16_ss(s_col, qd + 2 * (kPanel >> 4) + ks * 2, rd + ks * 2, idesc_s, 1u);
            mma_commit(&bar->s_full[t]);
          }
        }
        if (j < nt) {
          mma_commit(&bar->empty[ks_n]);
          mma_commit(&bar->rot_empty[j % kRotSlots]);
        }
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
      const int n_full = bar->n_full[t];
      for (int j = 0; j < mine; ++j) {
        int v0 = kPage, v1 = kPage;
        if (j >= n_full) {
          v0 = visible(pe[2 * j], qp);
          v1 = visible(pe[2 * j + 1], qp);
        }
        const bool all = j < n_full || __all_sync(0xffffffffu, v0 == kPage && v1 == kPage);
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
          mx[c] = max_nan(s[c][0], s[c][1]);
#pragma unroll
          for (int i = 2; i < 32; i += 2) mx[c] = max_nan(mx[c], max_nan(s[c][i], s[c][i + 1]));
        }
        const float top = max_nan(max_nan(mx[0], mx[1]), max_nan(mx[2], mx[3]));
        const bool raise = !(top * p.scale_log2 <= m * p.scale_log2 + kMargin);   // or NaN
        if (__any_sync(0xffffffffu, raise)) {
          const float m_new = raise ? top : m;
          // nothing seen so far (m = -inf): sums and O are zero whatever the factor
          const float f = m_new == m ? 1.f : ex2_approx((m - m_new) * p.scale_log2);
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
            const float x = fmaf(s[c0][i0], p.scale_log2, off);
            const float y = fmaf(s[c0][i0 + 1], p.scale_log2, off);
            const float a = ex2_approx(x), b = ex2_approx(y);
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
