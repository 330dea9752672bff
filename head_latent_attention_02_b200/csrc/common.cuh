// common.cuh -- shared definitions of libmla's kernels.  Each translation unit
// that includes it is a module with a status word of its own.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "mla.h"

namespace mla {

// Device status word: the first error a kernel meets while it runs.
__device__ int g_status;

__device__ __forceinline__ void set_status(int code) { atomicCAS(&g_status, 0, code); }

// Reads and clears the status word of the module (translation unit) that
// calls it; mla_get_status asks every module after synchronising the stream.
static inline int take_module_status() {
  int v = 0;
  const int zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_status, sizeof(int)) != cudaSuccess ||
      cudaMemcpyToSymbol(g_status, &zero, sizeof(int)) != cudaSuccess)
    return MLA_ERR_CUDA;
  return v;
}

template <typename T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// Round a float to the nearest bfloat16 and back (the precision an operand
// has inside a bf16 tensor-core product).
__device__ __forceinline__ float round_bf16(float x) {
  return __bfloat162float(__float2bfloat16_rn(x));
}

// Two floats as a pair of bfloat16 (the first one in the low half), and back.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

constexpr int kPage = 64;
constexpr int kMaxVersions = 8;
constexpr float kNegInf = -__builtin_huge_valf();

// Two floats as a pair of halves.
__device__ __forceinline__ uint32_t pack2_half(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 64 rows of the paged cache that a chunk call attends (mla_chunk.cu).
struct PageEntry {
  int row;      // physical cache row of the page's first row; past the cache: no rows
  int kpos;     // request position of that row
  short n;      // rows that hold data (0 .. 64)
  short ver;    // relocation version
  int seq;      // sequence it belongs to
};

// What the planner of a chunk call leaves on the device.
struct ChunkPlan {
  int n_items;
  int n_row_tiles;      // 256-row tiles of the page list (the expansion's row tiles)
};

// Expanded values are kept times 2^k, k for each sequence and head, which the
// attention takes back from its result: |V| <= |c| |w| then bounds them by 2^15,
// whatever the size of latents and weights.  A tile of 128 rows whose values are
// zero or lie between 2^-16 and half's largest number is held in halves (with the
// weights that meet it, which have to be of the same type): down to 2^-16 a
// half's rounding, a step of 2^-24 there, is no larger than a bfloat16's, and
// above 2^-14 it is eight times smaller.  Other tiles (rows or channels 2^-31 below
// the bound) are held in bfloat16.  The error of the result is 2.0e-3 with halves
// and 3.0e-3 without (1.66e-3 of it is the result's own rounding).
//
// The norms come as the largest exponents of the squares, E with |x|^2 < 2^(E + 1).
constexpr int kNoNorm = -10000;      // no vector, or zeros alone
__device__ __forceinline__ int value_exponent(int norm_c, int norm_w) {
  // |c| |w| < 2^((norm_c + norm_w + 2) / 2); values past 2^128 are infinite
  return min(max(15 - ((norm_c + norm_w + 3) >> 1), -113), 100);
}
__device__ __forceinline__ float power_of_two(int k) { return __int_as_float((k + 127) << 23); }
constexpr float kLeastHalf = 1.52587890625e-5f, kMostHalf = 65504.f;   // see above

// Description of one mla_decode call as the kernels see it.
struct DecodeArgs {
  int B, s_q, n_q, H, n_h, d_c, d_r, n_ver;
  int qH;                       // heads per query row of the q_abs the kernels read
  const int32_t* head_ids;      // [n_h] output head of each decoded head, or null = 0..n_h-1
  const float* key_inv;         // QK-normed decode: [n_pages * 64] inverse key RMS per cache row
  int max_pages, max_segs, max_gather;
  long long n_pages;
  float scale;
  const void* q_abs;
  const void* cache;
  const int32_t* block_table;
  const mla_seg_t* segs;
  const int32_t* gather_rows;   // may be null
  const int32_t* n_gather;      // null when gather_rows is null
  const int32_t* q_pos;
  float* o_lat;
  float* lse;
};

// Output head of the k-th decoded head: head_ids[k], or k when the call gives
// no list.  An id outside [0, H) records MLA_ERR_BAD_INDEX and yields -1 (the
// head's results are not written).
__device__ __forceinline__ int head_of(const DecodeArgs& a, int k) {
  if (!a.head_ids) return k;
  const int h = __ldg(a.head_ids + k);
  if (h < 0 || h >= a.H) {
    set_status(MLA_ERR_BAD_INDEX);
    return -1;
  }
  return h;
}

// Cache row of attended index `i` of sequence b (page mode: i-th row of the
// concatenated segments; gather mode: gather_rows[b][i]).  Returns false when
// the row cannot be located (bad gather row or page id), after recording
// MLA_ERR_BAD_INDEX.  On success fills the physical row (page*64+slot), the
// row's request position and its query version.
__device__ __forceinline__ bool locate_row(const DecodeArgs& a, int b, int i, long long* phys,
                                           int* kpos, int* ver) {
  const mla_seg_t* sg = a.segs + (size_t)b * a.max_segs;
  int row = -1, s_hit = -1;
  if (a.gather_rows) {
    row = a.gather_rows[(size_t)b * a.max_gather + i];
    for (int s = 0; s < a.max_segs; ++s) {
      if (row >= sg[s].row_begin && row < sg[s].row_end) { s_hit = s; break; }
    }
  } else {
    int rem = i;
    for (int s = 0; s < a.max_segs; ++s) {
      const int len = sg[s].row_end - sg[s].row_begin;
      if (len <= 0) continue;
      if (rem < len) { s_hit = s; row = sg[s].row_begin + rem; break; }
      rem -= len;
    }
  }
  if (s_hit < 0 || row < 0 || row / kPage >= a.max_pages) {
    set_status(MLA_ERR_BAD_INDEX);
    return false;
  }
  const int page = a.block_table[(size_t)b * a.max_pages + row / kPage];
  const int v = sg[s_hit].q_version;
  if (page < 0 || page >= a.n_pages || v < 0 || v >= a.n_ver) {
    set_status(MLA_ERR_BAD_INDEX);
    return false;
  }
  *phys = (long long)page * kPage + (row % kPage);
  *kpos = sg[s_hit].key_pos_base + (row - sg[s_hit].row_begin);
  *ver = v;
  return true;
}

// Number of attended rows of sequence b.
__device__ __forceinline__ int attended_rows(const DecodeArgs& a, int b) {
  if (a.gather_rows) return a.n_gather[b];
  const mla_seg_t* sg = a.segs + (size_t)b * a.max_segs;
  int n = 0;
  for (int s = 0; s < a.max_segs; ++s) n += max(0, sg[s].row_end - sg[s].row_begin);
  return n;
}

}  // namespace mla
