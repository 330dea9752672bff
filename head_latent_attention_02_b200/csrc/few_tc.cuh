// few_tc.cuh -- attention of few new tokens over the paged latent cache in the
// absorbed form, on sm_100a tensor cores (the small-chunk route of
// mla_chunk_attn).
//
// What it computes (Day 27 tutorial "Move the Key Projection Into the Query",
// "Move the Value Expansion After the Weighted Sum"): with q_abs = [W_UK^T
// q_nope | q_rope],
//     S[r, t] = scale * (q_abs[r] . [c_t | k_rope_t]),   o[r] = sum_t P[r, t] c_t
// for rows r = (token, head) of one sequence and its cached rows t.
//
// Decomposition.  A stream is 128 consecutive (token, head) rows of one
// sequence, a tile one page (64 rows) of it, and the units (stream, tile) are
// shared out in contiguous runs of equal length over pairs of CTAs.  The two
// CTAs of a pair are independent: each computes all scores and half of o's 512
// columns, because o for 128 rows in fp32 would take the whole tensor memory of
// an SM.  That computes S twice, but no weight, maximum or barrier crosses from
// one SM to another, and what both read of the cache comes from memory once.
//   tensor memory   o 256 columns | S 2 x 64 | four query panels 128
//   shared memory   five query panels 80 KB | the tile's panels: a ring of the
//                   four that are this CTA's value columns (3 tiles, 96 KB), and
//                   two groups, three panels and two, of the other four and the
//                   rotary one (40 KB, each refilled once its scores are taken: a
//                   wait costs the issuing warp 150 clocks of a tile's 2500, so
//                   panels do not wait one by one)
// A weight is kept as the sum of two bfloat16 (its rounding and what that left
// over), both in its score's tensor-memory columns, and o takes both products:
// 512 clocks more of 2500 a tile, and an error of the weights of 2^-16.
//
// Those 2500 are tensor clocks: 36 score steps of 32 (queries in tensor memory)
// or 48 clocks (in shared memory, whose reads bound products of 64 columns), and
// eight value steps of 128.  A tile takes about 2900: 16 tokens of 128 heads over
// 4081 rows each 41 us.
//
// A tile that some row does not see whole may hold anything where it is not
// seen: scores there are replaced, and its value panels are cleared of
// infinities and NaN before the product (a weight of zero times NaN is NaN);
// a cached row with one gives NaN scores to the queries that do see it.
//
// Roles (256 threads): warp 0 loads, warp 1 issues the MMAs (converged), warps
// 4-7 run the softmax, a thread per row, and write o's partial sums.
//
// Every wait is bounded and records MLA_ERR_TIMEOUT when it gives up.
#pragma once
#include <cuda.h>

#include "common.cuh"
#include "ptx.cuh"

namespace mla {
namespace fw {

constexpr int kRows = 128;                   // rows of a stream
constexpr int kDc = 512, kDr = 64, kWidth = kDc + kDr;
constexpr int kHalf = kDc / 2;               // value columns of a CTA
constexpr int kQPanel = kRows * 128;         // 16 KB
constexpr int kPanel = kPage * 128;          // 8 KB: 64 rows x 64 columns
constexpr int kVSlot = 4 * kPanel;
constexpr int kVSlots = 3;
constexpr int kQSmem = 5;                    // panels that are not value columns; their queries too
constexpr int kXFirst = 3;                   // panels of their first group
constexpr int kOffV = kQSmem * kQPanel;
constexpr int kOffX = kOffV + kVSlots * kVSlot;
constexpr int kOffBar = kOffX + kQSmem * kPanel;
constexpr int kSmemBytes = kOffBar + 512 + 1024;
constexpr int kThreads = 256;
constexpr int kTmemCols = 512;
constexpr int kColO = 0, kColS = 256, kColQ = 384;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMargin = 8.0f;              // log2 units: lazy rescale margin
static_assert(kSmemBytes <= 232448, "shared memory budget");

struct Stream {
  int q_row;        // first row of q_abs: token * H + head
  int rows;         // rows that exist (1 .. 128)
  int entry;        // first page entry of the sequence
  int tiles;        // pages up to the last one that any row sees
  int off;          // units before this stream
  int q_min, q_max; // least and largest query position of its rows
};

// What the planner leaves on the device.
struct Plan {
  int n_streams;
  int units, chunk;   // all units; units of a pair's run
};

struct Params {
  const Plan* plan;
  const Stream* streams;
  const PageEntry* pages;
  const int32_t* q_pos;
  int H;
  int rotary_moved;    // rotary keys come from the scratch (relocated rows)
  float scale_log2, scale;
  // o over a run's share of a stream, normalised: [slots][128 column groups][128
  // rows][4] (a thread holds a row, so a store of four columns is 512 contiguous
  // bytes a warp) and its log sum, [slots][128].
  // The slot of pair g's share of stream i is g + i: from one share to the next
  // the pair or the stream advances, so no two have the same.
  float* partial;
  float* partial_lse;
};

// Tensor maps (128-byte swizzle): q (column, row of q_abs), box {64, 128}; c
// (column, cache row), box {64, 64}; c4 (64-column offset, cache row, panel),
// box {64, 64, 4}; kr (column, row) over moved rotary keys, box {64, 64}
struct Maps {
  CUtensorMap q, c, c4, kr;
};

struct Bars {
  uint64_t q_full, q_empty;
  uint64_t v_full[kVSlots], v_empty[kVSlots];
  uint64_t x_full[2], x_empty[2];
  uint64_t s_full[2], p_full[2];
  uint64_t o_done[2];   // P c of one more even, odd tile complete
  uint64_t o_free;      // o of one more stream read
  uint64_t broken_set;  // the softmax warps have agreed on the broken rows of a tile
  uint32_t broken[2][2];  // those rows, a bit each: of this tile and, cleared, of the next
  uint32_t tmem_base;
};
static_assert(sizeof(Bars) <= 512, "barrier block too large");

// Last stream whose offset is <= u (streams without tiles share their
// successor's offset), by a whole warp: 32 offsets a load, where a binary
// search chains a load per step.
__device__ __forceinline__ int stream_of(const Stream* s, int n, int u) {
  const int lane = threadIdx.x & 31;
  int before = 0, of_these = 32;
  for (int i = 0; i < n && of_these == 32; i += 32) {
    of_these = __popc(__ballot_sync(0xffffffffu, i + lane < n && s[min(i + lane, n - 1)].off <= u));
    before += of_these;
  }
  return max(before - 1, 0);
}

// Visible rows of one page: those with data whose position is not past qp.
__device__ __forceinline__ int visible(const PageEntry& e, int qp) {
  if (e.kpos > qp) return 0;
  const long long d = (long long)qp - e.kpos + 1;
  return d < e.n ? (int)d : e.n;
}

// Infinities and NaN among eight bf16 become zeros; true if there are any.
__device__ __forceinline__ bool clear_broken(uint4& u) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool lo = (w[i] & 0x7f80u) == 0x7f80u, hi = (w[i] & 0x7f800000u) == 0x7f800000u;
    if (lo) w[i] &= 0xffff0000u;
    if (hi) w[i] &= 0x0000ffffu;
    any = any || lo || hi;
  }
  return any;
}

__global__ void __launch_bounds__(kThreads, 1)
few_attn_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps mp) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bar = reinterpret_cast<Bars*>(smem + kOffBar);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int pair = blockIdx.x >> 1, half = blockIdx.x & 1;

  if (threadIdx.x == 0) {
    mbar_init(&bar->q_full, 1);
    mbar_init(&bar->q_empty, 1);
    for (int i = 0; i < kVSlots; ++i) {
      mbar_init(&bar->v_full[i], 1);
      mbar_init(&bar->v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->x_full[i], 1);
      mbar_init(&bar->x_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->s_full[i], 1);
      mbar_init(&bar->p_full[i], 4);
      mbar_init(&bar->o_done[i], 1);
    }
    mbar_init(&bar->o_free, 4);
    mbar_init(&bar->broken_set, 4);
    for (int i = 0; i < 4; ++i) bar->broken[i >> 1][i & 1] = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&bar->tmem_base, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  // queries and plan are complete after this wait
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n_streams = p.plan->n_streams;
  const long long first = (long long)pair * p.plan->chunk;
  const int u0 = (int)min((long long)p.plan->units, first);
  const int u1 = (int)min((long long)p.plan->units, first + p.plan->chunk);
  const int s0 = u0 < u1 ? stream_of(p.streams, n_streams, u0) : 0;

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    if (lane == 0 && u0 < u1) {
      prefetch_tmap(&mp.q);
      prefetch_tmap(&mp.c);
      prefetch_tmap(&mp.c4);
      bool ok = true;
      auto wait = [&](uint64_t* b, int use) {      // the slot's use-th filling may start
        if (!mbar_wait(b, (use & 1) ^ 1)) {
          set_status(MLA_ERR_TIMEOUT);
          ok = false;
        }
        return ok;
      };
      int nv = 0, nq = 0;
      for (int u = u0, si = s0; ok && u < u1; ++si) {
        const Stream s = p.streams[si];
        const int end = min(u1, s.off + s.tiles);
        if (u >= end) continue;
        // Queries: the five panels that meet no value columns stay in shared memory; the
        // four of this CTA's value columns go through two slots of the value
        // ring into tensor memory.
        for (int i = 0; ok && i < 2; ++i, ++nv) {
          const int slot = nv % kVSlots;
          if (!wait(&bar->v_empty[slot], nv / kVSlots)) break;
          mbar_arrive_expect_tx(&bar->v_full[slot], 2 * kQPanel);
          for (int k = 0; k < 2; ++k)
            tma_load_2d(smem + kOffV + slot * kVSlot + k * kQPanel, &mp.q, &bar->v_full[slot],
                        half * kHalf + (2 * i + k) * 64, s.q_row);
        }
        if (!ok || !wait(&bar->q_empty, nq)) break;
        mbar_arrive_expect_tx(&bar->q_full, kQSmem * kQPanel);
        for (int i = 0; i < kQSmem; ++i)
          tma_load_2d(smem + i * kQPanel, &mp.q, &bar->q_full,
                      i < 4 ? (1 - half) * kHalf + i * 64 : kDc, s.q_row);
        ++nq;
        int row = p.pages[s.entry + (u - s.off)].row;
        for (; ok && u < end; ++u, ++nv) {
          const int j = u - s.off, y = row;
          if (u + 1 < end) row = p.pages[s.entry + j + 1].row;
          const int vs = nv % kVSlots;
          if (!wait(&bar->v_empty[vs], nv / kVSlots)) break;
          mbar_arrive_expect_tx(&bar->v_full[vs], kVSlot);
          tma_load_3d(smem + kOffV + vs * kVSlot, &mp.c4, &bar->v_full[vs], 0, y, 4 * half);
          for (int g = 0; g < 2; ++g) {
            if (!wait(&bar->x_empty[g], u - u0)) break;
            mbar_arrive_expect_tx(&bar->x_full[g], (g ? kQSmem - kXFirst : kXFirst) * kPanel);
            for (int i = g ? kXFirst : 0; i < (g ? kQSmem : kXFirst); ++i) {
              uint8_t* dst = smem + kOffX + i * kPanel;
              if (i == 4 && p.rotary_moved)
                tma_load_2d(dst, &mp.kr, &bar->x_full[g], 0, (s.entry + j) * kPage);
              else
                tma_load_2d(dst, &mp.c, &bar->x_full[g], i < 4 ? (1 - half) * kHalf + i * 64 : kDc,
                            y);
            }
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    if (u0 < u1) {            // the whole warp, converged
      constexpr uint32_t idesc_s = idesc_bf16_f32(kRows, kPage, false, false);
      constexpr uint32_t idesc_o = idesc_bf16_f32(kRows, kHalf, false, true);
      const uint64_t dq = smem_desc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t dv = smem_desc_sw128(smem_u32(smem + kOffV), 16, 1024);
      const uint64_t dx = smem_desc_sw128(smem_u32(smem + kOffX), 16, 1024);
      // values: 16 rows of four 64-column panels per step, rows outermost
      const uint64_t dc = smem_desc_sw128(smem_u32(smem + kOffV), kPanel, 1024);
      bool ok = true;
      auto wait = [&](uint64_t* b, uint32_t parity) {
        if (ok && !__all_sync(0xffffffffu, mbar_wait(b, parity))) {
          if (lane == 0) set_status(MLA_ERR_TIMEOUT);
          ok = false;
        }
        return ok;
      };
      // P c of every tile before the n-th complete.  A parity tells a phase from
      // its two neighbours: tile n - 3 is over (the scores of tile n - 1, whose
      // weights were waited for, followed its product) and tile n + 1 is not begun.
      auto wait_done = [&](int n) {
        return n == 0 || wait(&bar->o_done[(n - 1) & 1], ((n - 1) >> 1) & 1);
      };
      int nv = 0, nq = 0, n = 0;     // value slots taken; streams; tiles
      for (int u = u0, si = s0; ok && u < u1; ++si) {
        const Stream s = p.streams[si];
        const int end = min(u1, s.off + s.tiles);
        if (u >= end) continue;
        // the earlier stream's products no longer read its queries
        if (!wait_done(n)) break;
        for (int i = 0; i < 2; ++i, ++nv) {
          const int slot = nv % kVSlots;
          if (!wait(&bar->v_full[slot], (nv / kVSlots) & 1)) break;
          tc_fence_after();
          const uint64_t d = dv + slot * (kVSlot >> 4);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tmem_cp_128x256b_elect(tmem + kColQ + 32 * (2 * i + (k >> 2)) + 8 * (k & 3),
                                   d + (k >> 2) * (kQPanel >> 4) + (k & 3) * 2);
          mma_commit_elect(&bar->v_empty[slot]);
        }
        if (!ok || !wait(&bar->q_full, nq & 1)) break;
        const int tiles = end - u;
        u = end;
        // scores of one tile, into S buffer n & 1
        int vq = nv;
        auto scores = [&](int at) {
          const int vs = vq % kVSlots;
          const uint32_t col = tmem + kColS + 64 * (at & 1);
          if (!wait(&bar->v_full[vs], (vq / kVSlots) & 1)) return;
          ++vq;
          tc_fence_after();
          const uint64_t d = dv + vs * (kVSlot >> 4);
#pragma unroll
          for (int k = 0; k < 16; ++k)
            mma_bf16_ts_elect(col, tmem + kColQ + 8 * k, d + (k >> 2) * (kPanel >> 4) + (k & 3) * 2,
                              idesc_s, k ? 1u : 0u);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (!wait(&bar->x_full[g], at & 1)) return;
            tc_fence_after();
#pragma unroll
            for (int k = g ? 4 * kXFirst : 0; k < 4 * (g ? kQSmem : kXFirst); ++k)
              mma_bf16_ss_elect(col, dq + (k >> 2) * (kQPanel >> 4) + (k & 3) * 2,
                                dx + (k >> 2) * (kPanel >> 4) + (k & 3) * 2, idesc_s, 1u);
            mma_commit_elect(&bar->x_empty[g]);
          }
          mma_commit_elect(&bar->s_full[at & 1]);
        };
        scores(n);
        for (int i = 0; ok && i < tiles; ++i, ++n, ++nv) {
          if (i + 1 < tiles) scores(n + 1);
          else mma_commit_elect(&bar->q_empty);
          // the earlier stream's o has been read
          if (ok && i == 0 && nq > 0) wait(&bar->o_free, (nq - 1) & 1);
          if (!ok || !wait(&bar->p_full[n & 1], (n >> 1) & 1)) break;
          tc_fence_after();
          const int vs = nv % kVSlots;
          const uint32_t pc = tmem + kColS + 64 * (n & 1);
          const uint64_t d = dc + vs * (kVSlot >> 4);
#pragma unroll
          for (int k = 0; k < 8; ++k)          // the weights' roundings, then what they left over
            mma_bf16_ts_elect(tmem + kColO, pc + 8 * k, d + (k & 3) * (2048 >> 4), idesc_o,
                              (i | k) ? 1u : 0u);
          mma_commit_elect(&bar->v_empty[vs]);
          mma_commit_elect(&bar->o_done[n & 1]);
        }
        ++nq;
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax
    const int quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    bool ok = true;
    auto wait = [&](uint64_t* b, uint32_t parity) {
      if (ok && !__all_sync(0xffffffffu, mbar_wait(b, parity))) {
        if (lane == 0) set_status(MLA_ERR_TIMEOUT);
        ok = false;
      }
      return ok;
    };
    int n = 0, nv = 0, agreed = 0;
    for (int u = u0, si = s0; ok && u < u1; ++si) {
      const Stream s = p.streams[si];
      const int end = min(u1, s.off + s.tiles);
      if (u >= end) continue;
      nv += 2;                                  // the queries' slots
      const int qp = row < s.rows ? p.q_pos[(s.q_row + row) / p.H] : s.q_min;
      float m = kNegInf, l = 0.f;
      const int begin = u;
      for (; u < end; ++u, ++n, ++nv) {
        const PageEntry e = p.pages[s.entry + (u - s.off)];
        const bool mixed = visible(e, s.q_min) < kPage;
        const int seen = mixed ? visible(e, qp) : kPage;
        const uint32_t col = tmem + kColS + 64 * (n & 1) + lanes;
        if (!wait(&bar->s_full[n & 1], (n >> 1) & 1)) break;
        tc_fence_after();
        float x[2][32];
        tmem_ld64_sync(col, x);
        if (mixed) {
          // value panels: 2048 pieces of 16 bytes, 16 a thread; piece i lies in
          // row i / 8 mod 64 (the swizzle moves it within its row only).  The
          // four warps agree on the broken rows before any of them goes on; the
          // record of the next such tile is cleared before any can reach it.
          if (!wait(&bar->v_full[nv % kVSlots], (nv / kVSlots) & 1)) break;
          uint4* v = reinterpret_cast<uint4*>(smem + kOffV + nv % kVSlots * kVSlot);
#pragma unroll 4
          for (int i = row; i < kVSlot / 16; i += 128) {
            uint4 w = v[i];
            if (clear_broken(w)) {
              v[i] = w;
              const int k = i / 8 % 64;
              atomicOr(&bar->broken[(agreed >> 1) & 1][k >> 5], 1u << (k & 31));
            }
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar->broken_set);
          if (!wait(&bar->broken_set, 0)) break;
          const volatile uint32_t* rec = bar->broken[(agreed >> 1) & 1];
          const uint32_t b0 = rec[0], b1 = rec[1];
          if (row < 2) bar->broken[((agreed >> 1) & 1) ^ 1][row] = 0;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar->broken_set);
          if (!wait(&bar->broken_set, 1)) break;
          agreed += 2;
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (((c ? b1 : b0) >> i) & 1u) x[c][i] = __int_as_float(0x7fc00000);
              x[c][i] = 32 * c + i < seen ? x[c][i] : kNegInf;
            }
        }
        float mx[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          mx[c] = fmaxf(x[c][0], x[c][1]);
#pragma unroll
          for (int i = 2; i < 32; i += 2) mx[c] = fmaxf(mx[c], fmaxf(x[c][i], x[c][i + 1]));
        }
        // NaN scores are left out of the maximum; their weights are NaN, and so
        // are the row's sum and its output
        const float top = fmaxf(mx[0], mx[1]);
        const bool raise = !(top * p.scale_log2 <= m * p.scale_log2 + kMargin);
        if (__any_sync(0xffffffffu, raise)) {
          const float m_new = raise ? top : m;
          const float f = m_new == m ? 1.f : ex2_approx((m - m_new) * p.scale_log2);
          l *= f;
          m = m_new;
          if (u > begin) {
            // o is at rest once P c of tile n - 1 is done (of tile n - 3 it is: the
            // scores at hand followed it; that of tile n waits for these weights)
            if (!wait(&bar->o_done[(n - 1) & 1], ((n - 1) >> 1) & 1)) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kHalf; c += 32) {
              float o[32];
              tmem_ld32_sync(tmem + kColO + lanes + c, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= f;
              tmem_st32(tmem + kColO + lanes + c, o);
            }
          }
        }
        const float off = m == kNegInf ? 0.f : -m * p.scale_log2;
        float sum[2] = {0.f, 0.f};
        float hi[32], lo[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float a = ex2_approx(fmaf(x[i >> 4][2 * (i & 15)], p.scale_log2, off));
          const float b = ex2_approx(fmaf(x[i >> 4][2 * (i & 15) + 1], p.scale_log2, off));
          sum[0] += a;
          sum[1] += b;
          const uint32_t w = pack2(a, b);
          hi[i] = __uint_as_float(w);
          lo[i] = __uint_as_float(pack2(a - lo_f(w), b - hi_f(w)));
        }
        tmem_st32(col, hi);
        tmem_st32(col + 32, lo);
        l += sum[0] + sum[1];
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->p_full[n & 1]);
      }
      if (!ok) break;
      // o of this run's share of the stream, normalised, with its log sum
      if (!wait(&bar->o_done[(n - 1) & 1], ((n - 1) >> 1) & 1)) break;
      tc_fence_after();
      const int slot = pair + si;
      const bool none = l == 0.f;
      const float inv = none ? 0.f : 1.f / l;
      float4* o = reinterpret_cast<float4*>(p.partial) +
                  ((long long)slot * (kDc / 4) + half * (kHalf / 4)) * kRows + row;
#pragma unroll 1
      for (int c = 0; c < kHalf; c += 32) {
        float a[32];
        tmem_ld32_sync(tmem + kColO + lanes + c, a);
        if (row < s.rows) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            o[(c / 4 + i) * kRows] =
                none ? make_float4(0.f, 0.f, 0.f, 0.f)
                     : make_float4(a[4 * i] * inv, a[4 * i + 1] * inv, a[4 * i + 2] * inv,
                                   a[4 * i + 3] * inv);
        }
      }
      if (half == 0 && row < s.rows)
        p.partial_lse[slot * kRows + row] = none ? kNegInf : m * p.scale + logf(l);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->o_free);
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;");
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace fw
}  // namespace mla
