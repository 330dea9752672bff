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
// Decomposition.  A cluster of two CTAs takes 512 consecutive tokens of one
// sequence and one head, as two query tiles of 256 rows (128 in each CTA), and
// walks the sequence's rows in tiles of 128 (two pages of the list).  The MMAs
// act on the pair (cta_group::2): each CTA holds half of a tile's keys (64
// rows) and half of its values (64 columns) in shared memory and the tensor
// cores read both halves, so a CTA loads 40 KB a tile instead of 80 KB.  With one
// CTA per 256 tokens the ring held a tile and a half and its loads, 1.5 us
// from issue to landing, stalled the products.  S and O of both query tiles
// fill the 512 tensor-memory columns; P (16 bits, half or bf16 as the tile's
// values are) overwrites its S.  The
// tensor core works on one query tile while the other one's softmax runs:
//     ... P0 V | S0 | P1 V | S1 | P0 V | S0 ...
// At 192 + 128 columns a tile costs the tensor core 1280 clocks and its
// exponentials the special-function units 1024.  What bounds it is the way from
// scores to weights, about 1500 clocks, against 1280 of the other query tile's
// products: 2048 tokens over 10 240 rows, 128 heads take 1175 us (1.32 PFLOP/s).
//
// Roles (384 threads a CTA): warp 0 loads by TMA, warp 1 of the first CTA
// issues the MMAs, warps 4-7 and 8-11 run the softmax of query tiles 0 and 1 (a
// thread per query row, so that row statistics need no exchange between
// threads).  The running maximum is only raised when it grew by more than
// 2^4, which keeps the weights in range; O is rescaled by the softmax threads
// in that rare case.  S of step j is issued after P V of step j - 1 and its barrier
// covers both, so O is at rest while a softmax thread holds S.
//
// Every wait is bounded and records MLA_ERR_TIMEOUT when it gives up.
#pragma once
#include <cuda.h>

#include <type_traits>

#include "common.cuh"
#include "ptx.cuh"

namespace mla {
namespace ck {

constexpr int kDn = 128, kDr = 64, kDv = 128, kDc = 512;
constexpr int kQTile = 128, kKTile = 128;
constexpr int kPairTile = 2 * kQTile;        // rows of a query tile, both CTAs
constexpr int kItemTokens = 2 * kPairTile;
constexpr int kPanel = 128 * 128;            // 128 rows x 64 bf16: 16 KB
constexpr int kQBytes = 3 * kPanel;          // a query tile: two nope panels, one rope panel
// a CTA's half of a tile's keys and of its values
constexpr int kKeySlot = kPanel + kPanel / 2;   // 64 rows x two panels and the rotary panel
constexpr int kValSlot = kPanel;                // 128 rows x one panel
constexpr int kKeySlots = 3, kValSlots = 3;     // 120 KB: three tiles
constexpr int kOffKeys = 2 * kQBytes;
constexpr int kOffVals = kOffKeys + kKeySlots * kKeySlot;
constexpr int kOffBar = kOffVals + kValSlots * kValSlot;
constexpr int kSmemBytes = kOffBar + 512 + 1024;
constexpr int kThreads = 384;
// registers a thread: launched with 168, redistributed between the warpgroup
// that loads and issues and the two that hold a row of scores each
constexpr int kRegsIssue = 88, kRegsSoftmax = 208;
static_assert(kRegsIssue + 2 * kRegsSoftmax == 3 * 168, "register split");
constexpr int kTmemCols = 512;
constexpr int kColS = 0, kColO = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMargin = 4.0f;              // log2 units: lazy rescale margin
// weights are kept times 2^11: at most 2^15, the top of half's range, so that
// the small ones of a long row reach 2^-35 before they vanish
constexpr float kShift = 11.0f;
static_assert(kSmemBytes <= 232448, "shared memory budget");

struct Item {
  int b;         // sequence; its rows start at page entry `entry`
  int tok0, n;   // tokens [tok0, tok0 + n), n <= 512
  int entry;     // first page entry of the sequence (even)
  int tiles;     // 128-row tiles of the sequence; -1: the sequence is invalid
  // of each query tile: the tiles up to the last one that any of its queries
  // sees, and the leading ones that every query sees whole
  int need[2], full[2];
};

struct Params {
  const ChunkPlan* plan;
  const Item* items;
  const PageEntry* pages;
  const int32_t* q_pos;
  int H, h0, n_heads;          // heads of the call; first head and heads of this launch
  long long rows_cap;          // rows per head of the key and value scratch
  const int* norm_c;           // [sequences], see value_exponent
  const int* norm_w;           // [heads of this launch]
  const uint8_t* as_half;      // [heads of this launch][rows_cap / 128]: the values' type
  float scale_log2, scale;
  __nv_bfloat16* v;            // [n_tok, H, 128]
  float* lse;                  // [n_tok, H] or null
};

// Tensor maps (64 columns, 128-byte swizzle):
//   q   (column, token, panel) over q [n_tok, H x 192], box {64, 128, 3}
//   k,v (column, row, panel) over the scratch [heads x rows_cap, 128], boxes
//       {64, 64, 2} and {64, 128, 1}
//   kr  (column, row) over the rotary scratch [rows_cap, 64], box {64, 64}
struct Maps {
  CUtensorMap q, k, v, kr;
};

struct Bars {
  uint64_t q_full[2];
  uint64_t k_full[kKeySlots], k_empty[kKeySlots], v_full[kValSlots], v_empty[kValSlots];
  uint64_t s_full[2], o_full[2];
  uint64_t p_full[2][2];                       // query tile, half of the weights' columns
  uint32_t tmem_base;
};
static_assert(sizeof(Bars) <= 512, "barrier block too large");

// Visible rows of one page: those with data whose position is not past qp.
__device__ __forceinline__ int visible(const PageEntry& e, int qp) {
  if (e.kpos > qp) return 0;
  const long long d = (long long)qp - e.kpos + 1;
  return d < e.n ? (int)d : e.n;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
chunk_attn_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps mp) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bar = reinterpret_cast<Bars*>(smem + kOffBar);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  // the item list and the expanded rows are complete after this wait
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int item = blockIdx.x >> 1;
  const int rank = (int)cluster_ctarank();
  if (item >= p.plan->n_items) return;       // both CTAs of the pair
  const Item it = p.items[item];
  const int hl = blockIdx.y, h = p.h0 + hl;

  if (it.tiles < 0) {      // invalid sequence: NaN
    for (int i = rank * kThreads + threadIdx.x; i < it.n * kDv; i += 2 * kThreads)
      p.v[((long long)(it.tok0 + i / kDv) * p.H + h) * kDv + i % kDv] =
          __float2bfloat16_rn(__int_as_float(0x7fc00000));
    if (p.lse)
      for (int i = rank * kThreads + threadIdx.x; i < it.n; i += 2 * kThreads)
        p.lse[(long long)(it.tok0 + i) * p.H + h] = __int_as_float(0x7fc00000);
    return;
  }

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bar->q_full[t], 1);
      mbar_init(&bar->s_full[t], 1);
      mbar_init(&bar->p_full[t][0], 8);    // four softmax warps of each CTA
      mbar_init(&bar->p_full[t][1], 8);
      mbar_init(&bar->o_full[t], 1);
    }
    for (int i = 0; i < kKeySlots; ++i) {
      mbar_init(&bar->k_full[i], 1);
      mbar_init(&bar->k_empty[i], 1);
    }
    for (int i = 0; i < kValSlots; ++i) {
      mbar_init(&bar->v_full[i], 1);
      mbar_init(&bar->v_empty[i], 1);
    }
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(&bar->tmem_base, kTmemCols);
  tc_fence_before();
  __syncthreads();
  cluster_sync();       // the peer's barriers are ready
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  const int nt0 = uniform(it.need[0]), nt1 = uniform(it.need[1]);
  const int nt = max(nt0, nt1);
  // the sequence's first tile of as_half
  const int type0 = uniform((int)((hl * p.rows_cap + (long long)it.entry * kPage) / kKTile));

  if (warp < 4) {
    setmaxnreg_dec<kRegsIssue>();
    if (warp == 0) {
      // ------------------------------------------------------------ loads
      if (lane == 0 && nt > 0) {
        prefetch_tmap(&mp.q);
        prefetch_tmap(&mp.k);
        prefetch_tmap(&mp.v);
        prefetch_tmap(&mp.kr);
        const int krow = (int)(hl * p.rows_cap) + it.entry * kPage;
        // the pair's bytes are counted on the first CTA's barriers
        auto expect = [&](uint64_t* b, int bytes) {
          if (rank == 0) mbar_arrive_expect_tx(b, 2 * bytes);
          return mapa(smem_u32(b), 0);
        };
        auto load_q = [&](int t) {
          const uint32_t b = expect(&bar->q_full[t], kQBytes);
          tma_load_3d_pair(smem + t * kQBytes, &mp.q, b, 0, it.tok0 + t * kPairTile + rank * kQTile, 3 * h);
        };
        bool ok = true;
        auto wait = [&](uint64_t* b, int use) {      // the slot's use-th filling may start
          if (!mbar_wait(b, (use & 1) ^ 1)) {
            set_status(MLA_ERR_TIMEOUT);
            ok = false;
          }
          return ok;
        };
        if (nt0 > 0) load_q(0);
        for (int j = 0; ok && j < nt; ++j) {
          const int ks = j % kKeySlots, vs = j % kValSlots;
          if (!wait(&bar->k_empty[ks], j / kKeySlots)) break;
          uint8_t* key = smem + kOffKeys + ks * kKeySlot;
          uint32_t b = expect(&bar->k_full[ks], kKeySlot);
          tma_load_3d_pair(key, &mp.k, b, 0, krow + j * kKTile + rank * 64, 0);
          tma_load_2d_pair(key + kPanel, &mp.kr, b, 0, it.entry * kPage + j * kKTile + rank * 64);
          if (j == 0 && nt1 > 0) load_q(1);
          if (!wait(&bar->v_empty[vs], j / kValSlots)) break;
          b = expect(&bar->v_full[vs], kValSlot);
          tma_load_3d_pair(smem + kOffVals + vs * kValSlot, &mp.v, b, 0, krow + j * kKTile, rank);
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA
      if (rank == 0 && nt > 0) {        // the whole warp, converged
        constexpr uint32_t idesc_s = idesc_bf16_f32(kPairTile, kKTile, false, false);
        constexpr uint32_t idesc_pv = idesc_bf16_f32(kPairTile, kDv, false, true);
        // Descriptors of the first panels; a panel, a slot or a K step further is
        // an addition (16-byte units) that never leaves the address field.  The
        // issuing warp shares its scheduler with softmax warps: building each
        // descriptor anew cost it 1400 clocks for the eight MMAs of a P V.
        const uint64_t dq = smem_desc_sw128(smem_u32(smem), 16, 1024);
        const uint64_t dk = smem_desc_sw128(smem_u32(smem + kOffKeys), 16, 1024);
        // values: 16 rows of the CTA's 64-column panel per step, rows outermost
        const uint64_t dv = smem_desc_sw128(smem_u32(smem + kOffVals), kPanel, 1024);
        bool ok = true;
        auto wait = [&](uint64_t* b, uint32_t parity) {
          if (ok && !__all_sync(0xffffffffu, mbar_wait(b, parity))) {
            if (lane == 0) set_status(MLA_ERR_TIMEOUT);
            ok = false;
          }
        };
        int half = 0;
        for (int j = 0; ok && j <= nt; ++j) {
          // P V of step j - 1, then S of step j, for each query tile; what was
          // loaded is waited for first, off the chain from weights to scores
          const uint32_t idesc_o = uniform(half) ? idesc_half_f32(idesc_pv) : idesc_pv;
          if (j < nt) half = p.as_half[type0 + j];
          const int ks_n = j % kKeySlots, vs_n = (j + kValSlots - 1) % kValSlots;
          if (j < nt) wait(&bar->k_full[ks_n], (j / kKeySlots) & 1);
          if (j > 0) wait(&bar->v_full[vs_n], ((j - 1) / kValSlots) & 1);
          if (!ok) break;
          const uint64_t kd = dk + ks_n * (kKeySlot >> 4), vd = dv + vs_n * (kValSlot >> 4);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int mine = t ? nt1 : nt0;
            const uint32_t s_col = tmem + kColS + t * kKTile, o_col = tmem + kColO + t * kDv;
            if (j > 0 && j - 1 < mine) {
#pragma unroll
              for (int part = 0; part < 2; ++part) {
                wait(&bar->p_full[t][part], (j - 1) & 1);
                tc_fence_after();
                if (!ok) break;
#pragma unroll
                for (int ks = 4 * part; ks < 4 * part + 4; ++ks)
                  mma_pair_bf16_ts_elect(o_col, s_col + 8 * ks, vd + ks * (2048 >> 4), idesc_o,
                                         (j > 1 || ks > 0) ? 1u : 0u);
              }
              if (!ok) break;
              if (j == mine) mma_pair_commit_both_elect(&bar->o_full[t]);
            }
            if (j < mine) {
              if (j == 0) {
                wait(&bar->q_full[t], 0);
                if (!ok) break;
              }
              tc_fence_after();
              const uint64_t qd = dq + t * (kQBytes >> 4);
              // query panels are 128 rows high, a CTA's key panels 64
#pragma unroll
              for (int ks = 0; ks < 12; ++ks)
                mma_pair_bf16_ss_elect(s_col, qd + (ks >> 2) * (kPanel >> 4) + (ks & 3) * 2,
                                       kd + (ks >> 2) * (kPanel >> 5) + (ks & 3) * 2, idesc_s,
                                       ks ? 1u : 0u);
              mma_pair_commit_both_elect(&bar->s_full[t]);
            }
          }
          if (j > 0) mma_pair_commit_both_elect(&bar->v_empty[vs_n]);
          if (j < nt) mma_pair_commit_both_elect(&bar->k_empty[ks_n]);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<kRegsSoftmax>();
    const int t = warp >= 8 ? 1 : 0;
    const int quad = warp & 3;
    const int row = quad * 32 + lane;                 // row of the query tile
    const int tok = t * kPairTile + rank * kQTile + row;   // token of the item
    const int mine = t ? nt1 : nt0;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t s_col = tmem + kColS + t * kKTile + lanes;
    const uint32_t o_col = tmem + kColO + t * kDv + lanes;
    const int qp = tok < it.n ? p.q_pos[it.tok0 + tok] : INT32_MIN;
    float m = kNegInf, l = 0.f;       // running maximum (unscaled scores), sum of weights
    float unscale = 1.f;              // of the values (value_exponent)
    bool ok = true;
    if (mine > 0) {
      const PageEntry* pe = p.pages + it.entry;
      const int n_full = it.full[t];
      for (int j = 0; j < mine; ++j) {
        const bool half = p.as_half[type0 + j];     // under way during the wait for the scores
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
          mx[c] = fmaxf(s[c][0], s[c][1]);
#pragma unroll
          for (int i = 2; i < 32; i += 2) mx[c] = fmaxf(mx[c], fmaxf(s[c][i], s[c][i + 1]));
        }
        // NaN scores are left out of the maximum; their weights are NaN, and so
        // are the row's sum and its output
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const bool raise = !(top * p.scale_log2 <= m * p.scale_log2 + kMargin);
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
        const float off = m == kNegInf ? 0.f : kShift - m * p.scale_log2;
        const uint64_t off2 = pack_f32x2(off, off), mul2 = pack_f32x2(p.scale_log2, p.scale_log2);
        uint64_t sum[2] = {0ull, 0ull};
        // the weights of 64 columns at a time, so that P V may start on the first
        // half while the second one is computed
        auto weights = [&](auto as_half) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int c0 = 2 * c + i / 16, i0 = 2 * (i % 16);
              float x, y;
              unpack_f32x2(fma_f32x2(pack_f32x2(s[c0][i0], s[c0][i0 + 1]), mul2, off2), x, y);
              x = ex2_approx(x);
              y = ex2_approx(y);
              sum[i & 1] = add_f32x2(sum[i & 1], pack_f32x2(x, y));
              w[i] = __uint_as_float(decltype(as_half)::value ? pack2_half(x, y) : pack2(x, y));
            }
            tmem_st32(s_col + 32 * c, w);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_pair(mapa(smem_u32(&bar->p_full[t][c]), 0));
          }
        };
        if (half) weights(std::true_type());
        else weights(std::false_type());
        float a0, a1;
        unpack_f32x2(add_f32x2(sum[0], sum[1]), a0, a1);
        l += a0 + a1;
      }
      unscale = power_of_two(-value_exponent(p.norm_c[p.items[item].b], p.norm_w[blockIdx.y]));
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
            w[k] = none ? 0u
                        : pack2(a[8 * i + 2 * k] * inv * unscale, a[8 * i + 2 * k + 1] * inv * unscale);
          d[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    if (p.lse && tok < it.n)
      p.lse[(long long)(it.tok0 + tok) * p.H + h] = none ? kNegInf : m * p.scale + (logf(l) - kShift / kLog2e);
    tc_fence_before();
  }

  __syncwarp();
  __syncthreads();
  cluster_sync();       // no CTA leaves while the pair's MMAs may read its shared memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

}  // namespace ck
}  // namespace mla
