// mla_linear.cu -- out = act(x W^T + bias) + residual (mla_linear).
//
// The output projection of a prompt chunk (Day 27 tutorial "Move the Value
// Expansion After the Weighted Sum": each head's value joins the shared W_O)
// with the residual added where the product leaves the accumulator, and the
// layer's other products.  bf16 operands whose rows take TMA (16-byte pitch
// and base) run on the tensor cores (gemm_tc.cuh); fp32 and everything else
// on the CUDA cores below.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "mla.h"
#include "common.cuh"
#include "ptx.cuh"
#include "host_tma.cuh"
#include "gemm_tc.cuh"

namespace mla {
namespace {

// ------------------------------------------------------------ CUDA cores
constexpr int kTK = 16;
constexpr int kTN = 64;

struct SimtArgs {
  int M, N, K, act;
  long long x_stride, w_stride, res_stride, out_stride;
  const void* x;
  const void* w;
  const float* bias;
  const void* residual;
  void* out;
};

// A TM x 64 tile of the result per block of 256 threads, TM / 16 x 4 values a
// thread; K in steps of 16 through shared memory, the next step's elements on
// their way while this one's products run.  fp32 accumulation.
template <typename T, int TM>
__global__ void __launch_bounds__(256) linear_simt_kernel(const __grid_constant__ SimtArgs a) {
  constexpr int R = TM / 16;
  __shared__ float xs[kTK][TM + 4];
  __shared__ float ws[kTK][kTN + 4];
  const int m0 = blockIdx.y * TM, n0 = blockIdx.x * kTN;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const T* x = static_cast<const T*>(a.x);
  const T* w = static_cast<const T*>(a.w);
  constexpr int XE = TM * kTK / 256, WE = kTN * kTK / 256;
  float xr[XE], wr[WE];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int i = 0; i < XE; ++i) {
      const int e = i * 256 + threadIdx.x, r = e / kTK, k = k0 + e % kTK;
      xr[i] = m0 + r < a.M && k < a.K ? to_f(x[(long long)(m0 + r) * a.x_stride + k]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < WE; ++i) {
      const int e = i * 256 + threadIdx.x, r = e / kTK, k = k0 + e % kTK;
      wr[i] = n0 + r < a.N && k < a.K ? to_f(w[(long long)(n0 + r) * a.w_stride + k]) : 0.f;
    }
  };
  float acc[R][4] = {};
  fetch(0);
  for (int k0 = 0; k0 < a.K; k0 += kTK) {
#pragma unroll
    for (int i = 0; i < XE; ++i) {
      const int e = i * 256 + threadIdx.x;
      xs[e % kTK][e / kTK] = xr[i];
    }
#pragma unroll
    for (int i = 0; i < WE; ++i) {
      const int e = i * 256 + threadIdx.x;
      ws[e % kTK][e / kTK] = wr[i];
    }
    __syncthreads();
    if (k0 + kTK < a.K) fetch(k0 + kTK);
#pragma unroll
    for (int k = 0; k < kTK; ++k) {
      float xv[R], wv[4];
#pragma unroll
      for (int u = 0; u < R; ++u) xv[u] = xs[k][ty * R + u];
#pragma unroll
      for (int v = 0; v < 4; ++v) wv[v] = ws[k][tx * 4 + v];
#pragma unroll
      for (int u = 0; u < R; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[u][v] = fmaf(xv[u], wv[v], acc[u][v]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int u = 0; u < R; ++u)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int m = m0 + ty * R + u, n = n0 + tx * 4 + v;
      if (m >= a.M || n >= a.N) continue;
      float y = acc[u][v] + (a.bias ? a.bias[n] : 0.f);
      if (a.act == gm::kSilu) {
        const float t = expf(-fabsf(y));      // see activate_all
        y = (y < 0.f ? y * t : y) / (1.f + t);
      }
      if (a.act == gm::kGelu) y = 0.5f * y * erfcf(y * -0.70710678118654752f);
      if (a.residual) y += to_f(static_cast<const T*>(a.residual)[(long long)m * a.res_stride + n]);
      static_cast<T*>(a.out)[(long long)m * a.out_stride + n] = from_f<T>(y);
    }
}

template <typename T>
void launch_simt(const SimtArgs& a, cudaStream_t st) {
  const unsigned nb = (unsigned)((a.N + kTN - 1) / kTN);
  // few rows: tiles of 16 rows, so that a short product has blocks for more SMs.
  // Tiles of 16 and of 64 rows, fp32 (us): 16 x 1024 x 1001 45, 68; 256 x 1024 x 1001 68, 69;
  // 512 x 256 x 1001 46, 69; 512 x 1024 x 1001 111, 70; 1024 x 256 x 1001 68, 69;
  // 1024 x 1024 x 1001 200, 97.  They cross near 256 tiles of 16 rows; 512 rows is late
  // for wide results and early for narrow ones.
  if (a.M <= 512)
    linear_simt_kernel<T, 16><<<dim3(nb, (unsigned)((a.M + 15) / 16)), 256, 0, st>>>(a);
  else
    linear_simt_kernel<T, 64><<<dim3(nb, (unsigned)((a.M + 63) / 64)), 256, 0, st>>>(a);
}

// ------------------------------------------------------------ tensor cores
// Sum of a split tile's partials in the order of the pairs, and the epilogue.
// grid (tiles that were split, columns / 8); 256 threads, one row of the tile
// each, eight columns.
__global__ void __launch_bounds__(256) linear_finish_kernel(const __grid_constant__ gm::Params p,
                                                            int base) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int t = blockIdx.x, c0 = blockIdx.y * 8, row = threadIdx.x, wide = p.NB * p.BN;
  const long long u0 = (long long)t * p.k_steps;
  const int g0 = (int)(u0 / p.chunk), g1 = (int)((u0 + p.k_steps - 1) / p.chunk);
  if (g0 == g1) return;                    // one pair made the whole tile
  int mt, nt;
  gm::tile_at(p, base + t, &mt, &nt);
  const int a = mt * gm::kPairRows + row, b = nt * wide + c0;    // operand rows
  if (p.swapped ? (a >= p.N || b >= p.M) : (a >= p.M || b >= p.N)) return;
  // the residual first: the stores may be to its own place
  float v[8] = {}, r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int m = p.swapped ? b + j : a, n = p.swapped ? a : b + j;
    r[j] = p.residual && m < p.M && n < p.N
               ? __bfloat162float(p.residual[(long long)m * p.res_stride + n])
               : 0.f;
  }
#pragma unroll 4
  for (int g = g0; g <= g1; ++g) {
    const int second = (long long)g * p.chunk < u0 ? 1 : 0;   // the tile starts inside the run
    const float* s = p.partial + ((long long)(2 * g + second) * wide + c0) * gm::kPairRows + row;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += s[(long long)j * gm::kPairRows];
  }
  const bool vec = !p.swapped && p.vec && b + 8 <= p.N;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int n = p.swapped ? a : b + j;
    if (p.bias && n < p.N) v[j] += __ldg(p.bias + n);
  }
  gm::activate_all(v, p.act);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] += r[j];
  if (vec) {
    *reinterpret_cast<uint4*>(p.out + (long long)a * p.out_stride + b) =
        make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int m = p.swapped ? b + j : a, n = p.swapped ? a : b + j;
    if (m < p.M && n < p.N) p.out[(long long)m * p.out_stride + n] = __float2bfloat16_rn(v[j]);
  }
}

struct TilePlan {
  int swapped, BN, NB, n_mt, n_nt, P, k_steps, stages, rounds, chunk, grid;
  size_t ws;
};

// Which operand takes the tile's 256 rows, how wide the tile is, and how much
// of the work is split along K.  Few rows of x: W takes the rows (its stream is
// what the call costs) and the tile is as wide as x is high.  Otherwise the
// shape with the least estimated time: a pair's step costs the larger of its
// MMAs (2 NB BN clocks), its operand loads at about 50 bytes a clock and SM, and
// the issuing warp's bookkeeping (300 clocks a step and 350 a panel); a split
// costs a second launch and the partial sums' trip through memory; two column
// blocks cost an epilogue that little overlaps.  Split and not: 700 x 2048 x
// 7168 29.0 and 42.9 us, 1024 x 512 x 16384 27.2 and 32.1.
TilePlan plan_tiles(int M, int N, int K, int sms) {
  TilePlan t = {};
  const int pairs = sms / 2 > 0 ? sms / 2 : 1;
  t.swapped = M <= 128;
  // panels of a stage: long box rows where W is streamed once.  Four, two and one
  // panel (us): 16 x 7168 x 16384 45.5, 47.2, 48.2; 32 rows 45.6, 47.1, 48.4; 48 rows
  // 48.1, 47.1, 48.8; 128 rows 51.3, 49.9, 50.8; 16 x 7168 x 2048 10.5, 12.2, 14.0; 64 rows
  // 13.7, 14.8, 14.7 (four would be the better choice there: a short K).
  t.P = K % 64 == 0 && t.swapped ? (M <= 32 ? 4 : 2) : 1;
  const int step_k = gm::kKStep * t.P;
  t.k_steps = (K + step_k - 1) / step_k;
  double best = 0;
  const int rows = t.swapped ? N : M, cols = t.swapped ? M : N;
  t.n_mt = (rows + gm::kPairRows - 1) / gm::kPairRows;
  for (int nb = 1; nb <= (t.swapped ? 1 : 2); ++nb)
    for (int bn = 32; bn <= gm::kMaxBN; bn += 32) {
      if (t.swapped ? (bn != (cols + 31) / 32 * 32) : (bn < 64 && cols > bn)) continue;
      if (nb == 2 && bn < 192) continue;
      const long long n_nt = (cols + nb * bn - 1) / (nb * bn), tiles = (long long)t.n_mt * n_nt;
      const double load = (gm::kRows + nb * bn / 2) * 128 / 50.0, mma = 2.0 * nb * bn;
      const double step = std::max(t.P * std::max(mma, load), 300.0 + 350.0 * t.P);
      const double tile = t.k_steps * step;
      const long long rounds = tiles / pairs, left = tiles - rounds * pairs;
      // a run of at least eight steps of 64, so that a partial sum is worth its trip
      long long run = (left * t.k_steps + pairs - 1) / pairs;
      const long long least = (8 + t.P - 1) / t.P < t.k_steps ? (8 + t.P - 1) / t.P : t.k_steps;
      if (run < least) run = least;
      // one or two partial sums a pair, written and read at about 1600 bytes a
      // clock, and the second launch
      const long long used = left > 0 ? (left * t.k_steps + run - 1) / run : 0;
      const double trip = 4500 + 2.6 * used * nb * bn * gm::kPairRows * sizeof(float) / 1600.0;
      const bool split = left > 0 && run * step + trip < tile;
      const double drain = nb == 2 ? 8.0 * nb * bn * (rounds + 1) : 4.0 * bn;
      const double cost = rounds * tile + (left ? (split ? run * step + trip : tile) : 0) + drain;
      if (best == 0 || cost < best) {
        best = cost;
        t.BN = bn;
        t.NB = nb;
        t.n_nt = (int)n_nt;
        t.rounds = (int)rounds;
        t.chunk = split ? (int)run : 0;
        t.grid = 2 * (int)(rounds ? pairs : split ? used : left);
        t.ws = split ? (size_t)(2 * used) * nb * bn * gm::kPairRows * sizeof(float) : 0;
      }
    }
  const int stage = t.P * (gm::kABytes + t.NB * t.BN / 2 * 128);
  t.stages = (gm::kSmemMax - gm::kBarBytes - 1024) / stage;
  if (t.stages > gm::kMaxStages) t.stages = gm::kMaxStages;
  return t;
}

bool tc_shape(int dtype, int M, int N, int K) {
  return dtype == MLA_BF16 && M > 0 && N > 0 && K > 0;
}

}  // namespace

int linear_take_status() { return take_module_status(); }

}  // namespace mla

using namespace mla;

extern "C" size_t mla_linear_workspace_size(int32_t dtype, int32_t M, int32_t N, int32_t K) {
  if (!tc_shape(dtype, M, N, K)) return 0;
  const int sms = current_sms();
  return sms ? plan_tiles(M, N, K, sms).ws : 0;
}

extern "C" mla_status_t mla_linear(int32_t dtype, int32_t M, int32_t N, int32_t K, const void* x,
                                   int64_t x_stride, const void* w, int64_t w_stride,
                                   const float* bias, int32_t act, const void* residual,
                                   int64_t res_stride, void* out, int64_t out_stride,
                                   void* workspace, size_t ws_bytes, mla_stream_t stream) {
  if ((dtype != MLA_F32 && dtype != MLA_BF16) || M < 0 || N < 0 || K < 1 || act < gm::kNone ||
      act > gm::kGelu || x_stride < K || w_stride < K || out_stride < N ||
      (residual && res_stride < N))
    return MLA_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return MLA_OK;
  const size_t es = dtype == MLA_BF16 ? 2 : 4;
  if (!x || !w || !out || !ptr_aligned(x, es) || !ptr_aligned(w, es) || !ptr_aligned(out, es) ||
      !ptr_aligned(residual, es) || !ptr_aligned(bias, 4))
    return MLA_ERR_INVALID_ARG;
  // in place: the same rows, or one thread's results are another one's residual
  if (residual == out && M > 1 && res_stride != out_stride) return MLA_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool tma = dtype == MLA_BF16 && ptr_aligned(x, 16) && ptr_aligned(w, 16) &&
                   x_stride % 8 == 0 && w_stride % 8 == 0 && x_stride < (1ll << 38) &&
                   w_stride < (1ll << 38);
  if (!tma) {
    if (((long long)M + 63) / 64 > 65535) return MLA_ERR_UNSUPPORTED;   // grid limit
    SimtArgs a;
    a.M = M;
    a.N = N;
    a.K = K;
    a.act = act;
    a.x_stride = x_stride;
    a.w_stride = w_stride;
    a.res_stride = res_stride;
    a.out_stride = out_stride;
    a.x = x;
    a.w = w;
    a.bias = bias;
    a.residual = residual;
    a.out = out;
    if (dtype == MLA_BF16) launch_simt<__nv_bfloat16>(a, st);
    else launch_simt<float>(a, st);
    return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
  }
  const int sms = current_sms();
  if (!sms) return MLA_ERR_CUDA;
  const TilePlan t = plan_tiles(M, N, K, sms);
  if ((long long)t.n_mt * t.n_nt > INT32_MAX) return MLA_ERR_UNSUPPORTED;
  if (t.ws && (!workspace || ws_bytes < t.ws)) return MLA_ERR_WORKSPACE;
  if (t.ws && !ptr_aligned(workspace, 256)) return MLA_ERR_INVALID_ARG;
  gm::Params p = {};
  p.k_steps = t.k_steps;
  p.n_mt = t.n_mt;
  p.n_nt = t.n_nt;
  p.BN = t.BN;
  p.NB = t.NB;
  p.rounds = t.rounds;
  p.stages = t.stages;
  p.P = t.P;
  p.chunk = t.chunk;
  p.swapped = t.swapped;
  p.M = M;
  p.N = N;
  p.act = act;
  p.res_stride = res_stride;
  p.out_stride = out_stride;
  p.bias = bias;
  p.residual = static_cast<const __nv_bfloat16*>(residual);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.partial = static_cast<float*>(workspace);
  p.vec = ptr_aligned(out, 16) && out_stride % 8 == 0 &&
          (!residual || (ptr_aligned(residual, 16) && res_stride % 8 == 0));
  CUtensorMap ta, tb;
  const void* a = t.swapped ? w : x;
  const void* b = t.swapped ? x : w;
  const uint64_t ar = t.swapped ? N : M, br = t.swapped ? M : N;
  const uint64_t as = t.swapped ? w_stride : x_stride, bs = t.swapped ? x_stride : w_stride;
  const bool mapped = t.P == 1 ? map_rows(&ta, a, K, ar, as, gm::kRows) &&
                                     map_rows(&tb, b, K, br, bs, t.BN / 2)
                               : map_panels(&ta, a, K, ar, as, gm::kRows, t.P) &&
                                     map_panels(&tb, b, K, br, bs, t.BN / 2, t.P);
  if (!mapped) return MLA_ERR_CUDA;
  const int smem = t.stages * t.P * (gm::kABytes + t.NB * t.BN / 2 * 128) + gm::kBarBytes + 1024;
  if (cudaFuncSetAttribute(gm::gemm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           gm::kSmemMax) != cudaSuccess)
    return MLA_ERR_CUDA;
  if (launch_dependent(gm::gemm_kernel, dim3(t.grid), dim3(gm::kThreads), smem, st,
                       true, p, ta, tb) != cudaSuccess)
    return MLA_ERR_CUDA;
  const int base = t.rounds * (t.grid / 2);
  if (t.chunk &&
      launch_dependent(linear_finish_kernel, dim3(t.n_mt * t.n_nt - base, t.NB * t.BN / 8),
                       dim3(256), 0, st, true, p, base) != cudaSuccess)
    return MLA_ERR_CUDA;
  return MLA_OK;
}
