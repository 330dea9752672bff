// gemm_tc.cuh -- bf16 matrix products with fused epilogues on sm_100a tensor
// cores: D[m, n] = sum_k A[m, k] B[n, k], both operands K-major, fp32
// accumulation in tensor memory; out = act(x W^T + bias) + residual
// (mla_linear).
//
// Tile.  A cluster of two CTAs computes 256 x (NB x BN) (cta_group::2, BN <= 256,
// NB 1 or 2): each CTA holds 128 rows of A and half of each of B's NB column
// blocks in shared memory, and the pair's MMA reads both halves.  What such
// tiles run into first is the way from L2: at BN = 256 a CTA loads 64 bytes a
// clock of MMA time with NB = 1, 48 with NB = 2.  NB = 1 has two accumulators
// (2 x 256 tensor-memory columns), so that the epilogue of one tile overlaps
// the next one's products; with NB = 2 both belong to one tile, and the next
// tile's products start on a block as soon as it is drained.
//
// Roles per CTA (192 threads): warp 0 loads its CTA's operand halves by TMA
// into a ring of stages; warp 1 of the first CTA issues the MMAs of the pair;
// warps 2-5 read the accumulator (32 lanes each) and apply the epilogue.
//
// Work.  Pairs take whole tiles for as many full rounds as there are; the
// tiles that are left (fewer than pairs) are split along K into contiguous
// runs of (tile, k-step) units of equal length, so that few tiles with a long K
// still fill every SM.  A split tile's partial sums go to the workspace, a
// slot of the pair that made them, and a second launch (mla_linear.cu) adds them in the
// order of the pairs: the result does not depend on timing.
//
// A step's bookkeeping is on the critical path: both rings are walked by a
// single thread or warp, and what it computes between a wait and the next one
// adds to every step.  So slots and parities are counted, not divided out,
// descriptors are added up, and the next stage's barrier is looked at while
// this one's MMAs are issued (850 clocks a step before, 640 after, where the
// step's MMAs take 128 for 64 columns: 256 x 2048 x 2048 18.7 to 14.8 us).
//
// Measured: 4096 x 7168 x 16384 with residual 606 us alone (1.59 PFLOP/s); 16 x
// 7168 x 16384 42 us (5.6 TB/s of weights) and 6 us for the second launch.
//
// Every wait is bounded and records MLA_ERR_TIMEOUT when it gives up.
#pragma once
#include <cuda.h>

#include "common.cuh"
#include "ptx.cuh"

namespace mla {
namespace gm {

constexpr int kRows = 128;               // A rows of a CTA
constexpr int kPairRows = 256;
constexpr int kKStep = 64;               // K of a stage: 128 bytes of bf16
constexpr int kABytes = kRows * 128;     // 16 KB
constexpr int kMaxBN = 256;
constexpr int kMaxStages = 12;
constexpr int kThreads = 192;
constexpr int kSmemMax = 232448;
constexpr int kBarBytes = 512;
constexpr int kTmemCols = 512;
constexpr int kGroupM = 8;               // row tiles that share a pass over the column tiles

enum Act : int { kNone = 0, kSilu = 1, kGelu = 2 };

struct Params {
  int k_steps, n_mt, n_nt, BN, NB, stages;
  int P;                     // 64-K panels of a stage; > 1: three-axis maps over whole panels
  int rounds;                // whole tiles of each pair
  int chunk;                 // units of a pair's run over the tiles that are left; 0: whole tiles
  // the M x N result; swapped: A holds W's rows and B x's
  int swapped, M, N, act;
  long long res_stride, out_stride;
  const float* bias;
  const __nv_bfloat16* residual;
  __nv_bfloat16* out;
  float* partial;            // split: [2 x pairs][NB x BN][256]
  int vec;                   // out and residual rows take 16-byte accesses
};

struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint32_t tmem_base;
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier block too large");

struct Seg {
  int tile, k0, k1;
};

// The i-th segment of a pair's work; false when there is none.
__device__ __forceinline__ bool segment(const Params& p, int tiles, int pair, int pairs, int i, Seg* s) {
  if (i < p.rounds || !p.chunk) {
    const long long t = pair + (long long)i * pairs;
    if (t >= tiles) return false;
    s->tile = (int)t;
    s->k0 = 0;
    s->k1 = p.k_steps;
    return true;
  }
  i -= p.rounds;
  const int base = p.rounds * pairs;
  const long long U = (long long)(tiles - base) * p.k_steps;
  const long long u0 = (long long)pair * p.chunk;
  const long long u1 = u0 + p.chunk < U ? u0 + p.chunk : U;
  const long long at = i == 0 ? u0 : (u0 / p.k_steps + i) * p.k_steps;
  if (at >= u1) return false;
  s->tile = base + (int)(at / p.k_steps);
  s->k0 = (int)(at % p.k_steps);
  s->k1 = (int)(u1 - at < p.k_steps - s->k0 ? s->k0 + (u1 - at) : p.k_steps);
  return true;
}

// Row and column tile of tile t: kGroupM row tiles wide, so that the tiles in
// flight at one time share rows of both operands in L2.
__device__ __forceinline__ void tile_at(const Params& p, int t, int* mt, int* nt) {
  const int g = t / (kGroupM * p.n_nt);
  const int first = g * kGroupM;
  const int wide = min(kGroupM, p.n_mt - first);
  const int in = t - g * kGroupM * p.n_nt;
  *mt = first + in % wide;
  *nt = in / wide;
}

// GELU(v) = max(v, 0) - |v| Q(|v|) with the normal distribution's upper tail Q:
// with 1 + erf nothing is left of the result below v = -5.  Q(a) exp(a^2 / 2) is t
// times a polynomial of degree 8 in t = 1 / (1 + 0.35 a), fitted here by least
// squares (reweighted towards equal relative errors, 3.2e-8 up to a = 13.5);
// with erfcf the kernel spilled and every product took 10 to 35 % longer.
__device__ __forceinline__ float gelu(float v) {
  const float a = fabsf(v), t = __fdividef(1.f, fmaf(0.35f, a, 1.f));
  float q = -0.0291259643f;
  q = fmaf(q, t, 0.143872693f);
  q = fmaf(q, t, -0.255505472f);
  q = fmaf(q, t, 0.158930287f);
  q = fmaf(q, t, -0.0229377802f);
  q = fmaf(q, t, 0.105433188f);
  q = fmaf(q, t, 0.119852379f);
  q = fmaf(q, t, 0.139859095f);
  q = fmaf(q, t, 0.139621571f);
  q *= t * ex2_approx(a * a * -0.72134752f);
  return v > 14.f ? v : fmaxf(v, 0.f) - a * q;
}

// v = act(v).  The choice stands outside of the loops: a branch per value keeps
// one value's divide from overlapping the next one's (64 columns of SiLU took
// 3.5 us of a 16 us call that way).
template <int n>
__device__ __forceinline__ void activate_all(float (&v)[n], int act) {
  if (act == kSilu) {
#pragma unroll
    for (int j = 0; j < n; ++j) {
      // below zero v e^v / (1 + e^v): e^-v leaves the range (and __fdividef's) near -88
      const float t = __expf(-fabsf(v[j]));
      v[j] = __fdividef(v[j] < 0.f ? v[j] * t : v[j], 1.f + t);
    }
  } else if (act == kGelu) {
#pragma unroll
    for (int j = 0; j < n; ++j) v[j] = gelu(v[j]);
  }
}

// What the epilogue adds to 32 consecutive columns of one row: the bias and the
// residual (bf16 pairs), all loaded before the accumulator they meet is ready
// and before any store, which may be to the residual's own place: loads that
// wait for one another cost a trip to memory each.
struct Addend {
  float bias[32];
  uint32_t res[16];
};

__device__ __forceinline__ void load_addend(const Params& p, int m, int n, Addend& d) {
  if (p.bias) {
#pragma unroll
    for (int j = 0; j < 32; ++j) d.bias[j] = n + j < p.N ? __ldg(p.bias + n + j) : 0.f;
  }
  if (p.residual && m < p.M) {
    const __nv_bfloat16* r = p.residual + (long long)m * p.res_stride + n;
    if (p.vec && n + 32 <= p.N) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 u = reinterpret_cast<const uint4*>(r)[j];
        d.res[4 * j] = u.x;
        d.res[4 * j + 1] = u.y;
        d.res[4 * j + 2] = u.z;
        d.res[4 * j + 3] = u.w;
      }
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(r);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        d.res[j] = (n + 2 * j < p.N ? (uint32_t)h[2 * j] : 0u) |
                   (n + 2 * j + 1 < p.N ? (uint32_t)h[2 * j + 1] << 16 : 0u);
    }
  }
}

// 32 consecutive results of one row: out[m][n .. n + 32) = act(v + bias) +
// residual.  Columns past N and rows that take no 16-byte access go one by one.
__device__ __forceinline__ void finish32(const Params& p, int m, int n, float (&v)[32], const Addend& d) {
  if (p.bias) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] += d.bias[j];
  }
  activate_all(v, p.act);
  if (m >= p.M) return;
  if (p.residual) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      v[2 * j] += lo_f(d.res[j]);
      v[2 * j + 1] += hi_f(d.res[j]);
    }
  }
  __nv_bfloat16* o = p.out + (long long)m * p.out_stride + n;
  if (p.vec && n + 32 <= p.N) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float* y = v + 8 * j;
      reinterpret_cast<uint4*>(o)[j] =
          make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (n + j < p.N) o[j] = __float2bfloat16_rn(v[j]);
  }
}

// ta over A, box {64, 128}; tb over B, box {64, BN / 2}; with P > 1 both as
// (64-column offset, row, panel), P panels deep, so that a box row is 128 P
// contiguous bytes.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
gemm_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap ta,
            const __grid_constant__ CUtensorMap tb) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int S = p.stages;
  const int P = p.P;
  const int b_panel = p.BN / 2 * 128;
  const int a_bytes = P * kABytes;
  const int NB = p.NB, b_bytes = P * b_panel;      // one column block of B
  const int stage = a_bytes + NB * b_bytes;
  Bars* bar = reinterpret_cast<Bars*>(smem + S * stage);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&bar->full[i], 1);
      mbar_init(&bar->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->acc_full[i], 1);
      mbar_init(&bar->acc_empty[i], 8);    // four epilogue warps of each CTA
    }
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(&bar->tmem_base, kTmemCols);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  // operands and workspace may come from the launch before this one
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tiles = p.n_mt * p.n_nt;

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    if (lane == 0) {
      prefetch_tmap(&ta);
      prefetch_tmap(&tb);
      // the pair's bytes are counted on the first CTA's barriers
      const uint32_t fb0 = mapa(smem_u32(&bar->full[0]), 0);
      bool ok = true;
      Seg s;
      int slot = 0;
      uint32_t empty = 1;      // parity of the slot's last emptying; any at first
      for (int i = 0; ok && segment(p, tiles, pair, pairs, i, &s); ++i) {
        int mt, nt;
        tile_at(p, s.tile, &mt, &nt);
        const int ra = mt * kPairRows + (int)rank * kRows, rb = nt * NB * p.BN + (int)rank * (p.BN / 2);
        for (int k = s.k0; k < s.k1; ++k) {
          if (!mbar_wait(&bar->empty[slot], empty)) {
            set_status(MLA_ERR_TIMEOUT);
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&bar->full[slot], 2 * stage);
          const uint32_t fb = fb0 + slot * 8;
          uint8_t* dst = smem + slot * stage;
          if (P == 1) {
            tma_load_2d_pair(dst, &ta, fb, k * kKStep, ra);
            for (int nb = 0; nb < NB; ++nb)
              tma_load_2d_pair(dst + a_bytes + nb * b_bytes, &tb, fb, k * kKStep, rb + nb * p.BN);
          } else {
            tma_load_3d_pair(dst, &ta, fb, 0, ra, k * P);
            for (int nb = 0; nb < NB; ++nb)
              tma_load_3d_pair(dst + a_bytes + nb * b_bytes, &tb, fb, 0, rb + nb * p.BN, k * P);
          }
          if (++slot == S) {
            slot = 0;
            empty ^= 1;
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    if (rank == 0) {        // the whole warp, converged
      const uint32_t idesc = idesc_bf16_f32(kPairRows, p.BN, false, false);
      // Descriptors of the first stage; a stage, panel or K step further is an
      // addition (16-byte units) that never leaves the address field.
      const uint64_t a0 = smem_desc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t b0 = smem_desc_sw128(smem_u32(smem + a_bytes), 16, 1024);
      const uint32_t stage16 = stage >> 4, block16 = b_bytes >> 4, panel16 = b_panel >> 4;
      bool ok = true;
      Seg s;
      int slot = 0;
      uint32_t full = 0;       // parity of the slot's filling
      bool ready = false;      // a look ahead found the slot filled
      for (int i = 0; ok && segment(p, tiles, pair, pairs, i, &s); ++i) {
        for (int k = s.k0; ok && k < s.k1; ++k) {
          if (!__all_sync(0xffffffffu, ready || mbar_wait(&bar->full[slot], full))) {
            if (lane == 0) set_status(MLA_ERR_TIMEOUT);
            ok = false;
            break;
          }
          tc_fence_after();
          const int at = slot;
          if (++slot == S) {
            slot = 0;
            full ^= 1;
          }
          ready = mbar_test(&bar->full[slot], full);     // under way while the MMAs are issued
          for (int nb = 0; nb < NB; ++nb) {
            const int ab = NB == 2 ? nb : i & 1;
            if (k == s.k0) {
              if (!__all_sync(0xffffffffu, mbar_wait(&bar->acc_empty[ab],
                                                     ((NB == 2 ? i : i >> 1) & 1) ^ 1))) {
                if (lane == 0) set_status(MLA_ERR_TIMEOUT);
                ok = false;
                break;
              }
              tc_fence_after();
            }
            uint64_t ad = a0 + at * stage16, bd = b0 + at * stage16 + nb * block16;
            for (int pn = 0; pn < P; ++pn) {
              mma_pair_bf16_ss_elect4(tmem + ab * kMaxBN, ad, bd, idesc, (k - s.k0) | pn);
              ad += kABytes >> 4;
              bd += panel16;
            }
          }
          mma_pair_commit_both_elect(&bar->empty[at]);
        }
        if (ok) mma_pair_commit_both_elect(&bar->acc_full[NB == 2 ? 0 : i & 1]);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3;
    const int row = (int)rank * kRows + quad * 32 + lane;      // row of the pair's tile
    Seg s;
    for (int i = 0; segment(p, tiles, pair, pairs, i, &s); ++i) {
      int mt, nt;
      tile_at(p, s.tile, &mt, &nt);
      const bool part = s.k1 - s.k0 < p.k_steps;
      const int m = mt * kPairRows + row;          // row of A
      const int n0 = nt * NB * p.BN;               // first row of B
      Addend add;
      if (!part && !p.swapped) load_addend(p, m, n0, add);
      const int full = NB == 2 ? 0 : i & 1;
      if (!__all_sync(0xffffffffu,
                      mbar_wait(&bar->acc_full[full], (NB == 2 ? i : i >> 1) & 1))) {
        if (lane == 0) set_status(MLA_ERR_TIMEOUT);
        break;
      }
      tc_fence_after();
      for (int nb = 0; nb < NB; ++nb) {
        const int ab = NB == 2 ? nb : full;
        const uint32_t acc = tmem + ab * kMaxBN + ((uint32_t)(quad * 32) << 16);
        const int c0 = nb * p.BN;                  // column of the tile
        if (part) {
          // the pair's first slot holds a segment that starts its run, the
          // second one that ends it
          const bool first = (long long)(s.tile - p.rounds * pairs) * p.k_steps + s.k0 ==
                             (long long)pair * p.chunk;
          float* o = p.partial +
                     ((long long)(2 * pair + (first ? 0 : 1)) * NB * p.BN + c0) * kPairRows + row;
#pragma unroll 1
          for (int c = 0; c < p.BN; c += 32) {
            float v[32];
            tmem_ld32_sync(acc + c, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[(long long)(c + j) * kPairRows] = v[j];
          }
        } else if (p.swapped) {
          const float bias = p.bias && m < p.N ? __ldg(p.bias + m) : 0.f;   // feature of this lane
#pragma unroll 1
          for (int c = 0; c < p.BN; c += 32) {
            const int t0 = n0 + c0 + c;
            if (t0 >= p.M) break;
            float v[32], r[32];
            tmem_ld32_sync(acc + c, v);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              r[j] = p.residual && m < p.N && t0 + j < p.M
                         ? __bfloat162float(p.residual[(long long)(t0 + j) * p.res_stride + m])
                         : 0.f;
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] += bias;
            activate_all(v, p.act);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (m < p.N && t0 + j < p.M)
                p.out[(long long)(t0 + j) * p.out_stride + m] = __float2bfloat16_rn(v[j] + r[j]);
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < p.BN; c += 32) {
            const int n = n0 + c0 + c;
            if (n >= p.N) break;
            float v[32];
            tmem_ld32_sync(acc + c, v);
            finish32(p, m, n, v, add);
            // the next 32 columns'; past this block they lie in the next one
            if (n + 32 < p.N && c0 + c + 32 < NB * p.BN) load_addend(p, m, n + 32, add);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_pair(mapa(smem_u32(&bar->acc_empty[ab]), 0));
      }
    }
  }

  // the launch after this one may be scheduled; it waits for this one's end
  // before it reads its results
  asm volatile("griddepcontrol.launch_dependents;");
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();     // no CTA leaves while the pair's MMAs may read its shared memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

}  // namespace gm
}  // namespace mla
