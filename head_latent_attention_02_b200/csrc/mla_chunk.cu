// mla_chunk.cu -- attention of a ragged chunk of new tokens over the paged
// latent cache (mla_chunk_attn): host side, planner and the small kernels.
//
// Three routes compute the same result, chosen by a rule on sizes (chunk_route):
//   expanded   bf16 rows of 512 + 64, 128-wide heads: keys and values are
//              expanded once per call into the workspace (expand_tc.cuh), the
//              rotary keys moved to their request positions, and the direct
//              form attends over them (chunk_tc.cuh).  For chunks.
//   absorbed   few tokens over those rows (few_tc.cuh), between the
//              absorption of the queries and a value expansion that joins the
//              shares of split sequences.
//   generic    fp32 and other widths: one kernel on the CUDA cores.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "mla.h"
#include "common.cuh"
#include "ptx.cuh"
#include "host_tma.cuh"
#include "expand_tc.cuh"
#include "chunk_tc.cuh"
#include "few_tc.cuh"

namespace mla {
namespace {

constexpr int kPlanThreads = 1024;
constexpr float kNaN = __builtin_nanf("");

struct ChunkArgs {
  int B, n_tok, H, d_n, d_r, d_v, n_ver, max_pages, max_segs;
  long long n_pages;
  double rope_base;
  int delta[kMaxVersions];
  const void* q;
  const int32_t* tok_start;
  const int32_t* q_pos;
  const void* cache;
  const int32_t* block_table;
  const mla_seg_t* segs;
};

// Pages of sequence b's segments; -1 when its token range or its segment table
// is invalid (the rules of mla_decode; positions that do not fit in 32 bits).
__device__ int sequence_pages(const ChunkArgs& a, int b) {
  const int t0 = a.tok_start[b], t1 = a.tok_start[b + 1];
  if (t0 < 0 || t1 < t0 || t1 > a.n_tok) return -1;
  const mla_seg_t* sg = a.segs + (size_t)b * a.max_segs;
  int prev_end = 0, pages = 0;
  for (int s = 0; s < a.max_segs; ++s) {
    const int rb = sg[s].row_begin, re = sg[s].row_end;
    if (re == rb) continue;
    if (rb < prev_end || re < rb || rb % kPage != 0 ||
        (long long)re > (long long)a.max_pages * kPage ||
        sg[s].q_version < 0 || sg[s].q_version >= a.n_ver ||
        (long long)sg[s].key_pos_base + (re - rb) > (long long)INT32_MAX + 1)
      return -1;
    prev_end = re;
    pages += (re - rb + kPage - 1) / kPage;
  }
  return pages;
}

// The i-th page of sequence b's segments (i below sequence_pages): false when
// its id is out of range.
__device__ bool page_at(const ChunkArgs& a, int b, int i, PageEntry* e) {
  const mla_seg_t* sg = a.segs + (size_t)b * a.max_segs;
  for (int s = 0; s < a.max_segs; ++s) {
    const int len = sg[s].row_end - sg[s].row_begin;
    if (len <= 0) continue;
    const int np = (len + kPage - 1) / kPage;
    if (i >= np) {
      i -= np;
      continue;
    }
    const int row = sg[s].row_begin + i * kPage;
    const int page = a.block_table[(size_t)b * a.max_pages + row / kPage];
    if (page < 0 || page >= a.n_pages) return false;
    e->row = page * kPage;
    e->kpos = sg[s].key_pos_base + i * kPage;
    e->n = min(kPage, sg[s].row_end - row);
    e->ver = sg[s].q_version;
    e->seq = b;
    return true;
  }
  return false;
}

// Exclusive sums of x over the block's threads on top of *carry, which ends as
// the running total; scratch holds an element a warp.  Page counts are summed in 64
// bits: tables may list any number of pages, whatever max_rows allows of them.
template <typename T>
__device__ T block_scan(T x, T* scratch, T* carry) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int warps = blockDim.x >> 5;
  T y = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T z = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) y += z;
  }
  if (lane == 31) scratch[wid] = y;
  __syncthreads();
  if (wid == 0) {
    T t = lane < warps ? scratch[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const T z = __shfl_up_sync(0xffffffffu, t, d);
      if (lane >= d) t += z;
    }
    if (lane < warps) scratch[lane] = t;
  }
  __syncthreads();
  const T out = *carry + (wid ? scratch[wid - 1] : 0) + y - x;
  const T total = scratch[warps - 1];
  __syncthreads();
  if (threadIdx.x == 0) *carry += total;
  __syncthreads();
  return out;
}

// Largest x over the block's threads up to this one and over *carry, which ends
// as the largest of all.
__device__ int block_scan_max(int x, int* scratch, int* carry) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int warps = blockDim.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x = max(x, z);
  }
  if (lane == 31) scratch[wid] = x;
  __syncthreads();
  if (wid == 0) {
    int t = lane < warps ? scratch[lane] : INT32_MIN;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, t, d);
      if (lane >= d) t = max(t, z);
    }
    if (lane < warps) scratch[lane] = t;
  }
  __syncthreads();
  const int out = max(max(*carry, x), wid ? scratch[wid - 1] : INT32_MIN);
  const int total = scratch[warps - 1];
  __syncthreads();
  if (threadIdx.x == 0) *carry = max(*carry, total);
  __syncthreads();
  return out;
}

// last index i in [0, n) with off[i] <= x (off ascending, off[0] <= x)
__device__ __forceinline__ int last_at_most(const int* off, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (off[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// A sequence's tokens and table.  A token range is only taken if it starts at or
// behind every start before it: ranges are then disjoint.
struct SeqRange {
  bool ranged, wrong;     // its token range holds; the range or the segment table does not
  int tokens, pages;      // of a range that holds; pages (0 if `wrong`)
};

// Sequence b by its thread, for all threads of a block at once (b >= B: none);
// *latest: the last start so far.
__device__ SeqRange read_sequence(const ChunkArgs& a, int b, int* scratch, int* latest) {
  SeqRange r = {false, false, 0, 0};
  const int from = b < a.B ? a.tok_start[b] : INT32_MIN;
  const bool behind = from == block_scan_max(from, scratch, latest);
  if (b < a.B) {
    const int to = a.tok_start[b + 1], k = sequence_pages(a, b);
    r.wrong = k < 0 || !behind;
    r.ranged = behind && from >= 0 && to >= from && to <= a.n_tok;
    if (r.ranged) r.tokens = to - from;
    if (r.tokens > 0 && !r.wrong) r.pages = k;
  }
  return r;
}

// Flags of a sequence: its tokens get NaN; its token range is invalid (no tokens).
constexpr int kInvalid = 1, kNoRange = 2;

enum TokState : int { kNone = 0, kLive = 1, kBad = 2 };

// One CTA, after the page list: the streams of the tokens [slab0, slab0 +
// slab_n) with their tile counts (pages up to the last one that any row sees),
// each token's state, and the run length.  A run that no stream boundary falls
// into saves a pair its second set of partial sums: with equal streams, a
// divisor or multiple of their length is taken if it costs at most a quarter
// more tiles a pair.
struct FewToken {
  int state;              // TokState
  int stream, row;        // first stream of its sequence, and that stream's first row
};

struct FewPlan {
  int slab0, slab_n, pairs;
  fw::Plan* plan;
  fw::Stream* streams;
  FewToken* tokens;
};

__device__ void plan_few(const ChunkArgs& a, const FewPlan& f, const int* seq,
                         const PageEntry* pages) {
  const int slab0 = f.slab0, slab_n = f.slab_n, pairs = f.pairs;
  fw::Plan* plan = f.plan;
  fw::Stream* streams = f.streams;
  FewToken* tokens = f.tokens;
  __shared__ int scratch[33], n_st, units, longest, shortest;
  const int* pg = seq;
  const int* bad = seq + 2 * (a.B + 1);
  if (threadIdx.x == 0) {
    n_st = units = longest = 0;
    shortest = INT32_MAX;
  }
  for (int t = threadIdx.x; t < slab_n; t += kPlanThreads) tokens[t].state = kNone;
  __syncthreads();
  // streams, in the order of the sequences
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    int ns = 0, t0 = 0, t1 = 0;
    if (b < a.B && bad[b] != kNoRange) {
      t0 = max(a.tok_start[b] - slab0, 0);           // tokens of the slab
      t1 = min(a.tok_start[b + 1] - slab0, slab_n);
      if (!bad[b] && t1 > t0) ns = ((t1 - t0) * a.H + fw::kRows - 1) / fw::kRows;
    }
    const int at = block_scan(ns, scratch, &n_st);
    for (int t = t0; t < t1; ++t) tokens[t] = {bad[b] ? kBad : kLive, at, t0 * a.H};
    for (int k = 0; k < ns; ++k) {
      fw::Stream s;
      s.q_row = t0 * a.H + k * fw::kRows;
      s.rows = min(fw::kRows, t1 * a.H - s.q_row);
      s.entry = pg[b];
      s.q_min = INT32_MAX;
      s.q_max = INT32_MIN;
      for (int t = s.q_row / a.H; t <= (s.q_row + s.rows - 1) / a.H; ++t) {
        s.q_min = min(s.q_min, a.q_pos[slab0 + t]);
        s.q_max = max(s.q_max, a.q_pos[slab0 + t]);
      }
      s.tiles = pg[b + 1] - pg[b];
      while (s.tiles > 0 && fw::visible(pages[s.entry + s.tiles - 1], s.q_max) == 0) --s.tiles;
      s.off = 0;
      streams[at + k] = s;
      if (s.tiles > 0) {
        atomicMax(&longest, s.tiles);
        atomicMin(&shortest, s.tiles);
      }
    }
  }
  __syncthreads();
  const int n = n_st;
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    const int off = block_scan(i < n ? streams[i].tiles : 0, scratch, &units);
    if (i < n) streams[i].off = off;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int run = max(1, (units + pairs - 1) / pairs);
    if (units > 0 && longest == shortest) {
      const int live = units / longest;          // streams with tiles
      int even = 0;
      if (live > pairs) {
        even = longest * ((live + pairs - 1) / pairs);
      } else {
        for (int parts = min(longest, pairs / live); parts >= 1 && !even; --parts)
          if (longest % parts == 0) even = longest / parts;
      }
      if (even > 0 && 4ll * even <= 5ll * run) run = even;
    }
    plan->n_streams = n;
    plan->units = units;
    plan->chunk = run;
  }
}

// The streams of a later slab.
__global__ void __launch_bounds__(kPlanThreads) few_plan_kernel(
    const __grid_constant__ ChunkArgs a, const __grid_constant__ FewPlan f, const int* seq,
    const PageEntry* pages) {
  asm volatile("griddepcontrol.launch_dependents;");
  plan_few(a, f, seq, pages);
}

// One CTA: validates the sequences, lists their pages (an even number each, so
// that a 128-row tile belongs to one sequence; a multiple of four in all) and
// their 512-token items.  seq: page offset [B + 1], item offset [B + 1], flag
// [B].  norms: cleared, for the n_norms that the next launch finds.
// A sequence that does not fit `cap` pages is invalid.  The item and stream lists
// rely on disjoint token ranges.
// kFew: the absorbed route's streams follow, in place of the items.  That kernel
// is launched as a dependent of the absorption, whose results it does not read:
// it works beside it and only waits for it before it ends, so that what follows
// finds both complete.
template <bool kFew>
__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(
    const __grid_constant__ ChunkArgs a, const __grid_constant__ FewPlan f, int cap, ChunkPlan* plan,
    int* seq, ck::Item* items, PageEntry* pages, int* norms, int n_norms) {
  asm volatile("griddepcontrol.launch_dependents;");
  __shared__ int scratch[33], n_it, used, latest;
  __shared__ long long page_scratch[33], n_pg;
  for (int i = threadIdx.x; i < n_norms; i += kPlanThreads) norms[i] = kNoNorm;
  int* pg = seq;
  int* itm = seq + a.B + 1;
  int* bad = seq + 2 * (a.B + 1);
  if (threadIdx.x == 0) {
    n_pg = n_it = used = 0;
    latest = INT32_MIN;
  }
  __syncthreads();
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    const SeqRange r = read_sequence(a, b, scratch, &latest);
    const long long np = (r.pages + 1) / 2 * 2, po = block_scan(np, page_scratch, &n_pg);
    const int io = block_scan(r.tokens > 0 ? (r.tokens - 1) / ck::kItemTokens + 1 : 0, scratch, &n_it);
    if (b < a.B) {
      const bool wrong = r.wrong || po + np > cap;
      pg[b] = (int)min(po, (long long)cap);
      itm[b] = io;
      bad[b] = !r.ranged ? kNoRange : wrong ? kInvalid : 0;
      if (wrong) set_status(MLA_ERR_BAD_INDEX);
      else atomicMax(&used, (int)(po + np));
    }
  }
  __syncthreads();
  const int in_use = used, whole = (in_use + 3) / 4 * 4;      // cap is a multiple of four
  if (threadIdx.x == 0) {
    pg[a.B] = (int)min(n_pg, (long long)cap);
    itm[a.B] = n_it;
    plan->n_items = n_it;
    plan->n_row_tiles = whole / 4;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < whole; e += kPlanThreads) {
    PageEntry pe = {INT32_MAX - 2 * kPage, INT32_MAX, 0, 0, 0};   // no rows
    if (e < in_use) {
      const int b = last_at_most(pg, a.B, e);
      if (!bad[b] && e - pg[b] < sequence_pages(a, b) && !page_at(a, b, e - pg[b], &pe)) {
        set_status(MLA_ERR_BAD_INDEX);
        atomicExch(&bad[b], kInvalid);
      }
    }
    pages[e] = pe;
  }
  __syncthreads();
  if constexpr (kFew) {
    plan_few(a, f, seq, pages);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int total = itm[a.B];
  for (int i = threadIdx.x; i < total; i += kPlanThreads) {
    const int b = last_at_most(itm, a.B, i);
    // the last tokens, which see the most rows, first
    const int k = itm[b + 1] - 1 - i;
    ck::Item it;
    it.b = b;
    it.tok0 = a.tok_start[b] + k * ck::kItemTokens;
    it.n = min(ck::kItemTokens, a.tok_start[b + 1] - it.tok0);
    it.entry = pg[b];
    it.tiles = atomicAdd(&bad[b], 0) ? -1 : (pg[b + 1] - pg[b]) / 2;
    items[i] = it;
  }
}

// Squared norm of 512 channels, four threads a row; every thread of
// the four gets it.  Half of the row's additions are independent of the other half.
__device__ __forceinline__ float row_norm_sq(const __nv_bfloat16* row, int part) {
  const uint4* src = reinterpret_cast<const uint4*>(row) + part;
  float a = 0.f, b = 0.f;
#pragma unroll 8
  for (int i = 0; i < ck::kDc / 32; ++i) {
    const uint4 u = src[4 * i];
    a = fmaf(lo_f(u.x), lo_f(u.x), a); b = fmaf(hi_f(u.x), hi_f(u.x), b);
    a = fmaf(lo_f(u.y), lo_f(u.y), a); b = fmaf(hi_f(u.y), hi_f(u.y), b);
    a = fmaf(lo_f(u.z), lo_f(u.z), a); b = fmaf(hi_f(u.z), hi_f(u.z), b);
    a = fmaf(lo_f(u.w), lo_f(u.w), a); b = fmaf(hi_f(u.w), hi_f(u.w), b);
  }
  a += b;
  a += __shfl_xor_sync(0xffffffffu, a, 1);
  return a + __shfl_xor_sync(0xffffffffu, a, 2);
}

// The same of the channels times `size`, a power of two.
__device__ __noinline__ float row_norm_sq_scaled(const __nv_bfloat16* row, int part, float size) {
  float a = 0.f;
  for (int i = part; i < ck::kDc; i += 4) {
    const float x = __bfloat162float(row[i]) * size;
    a = fmaf(x, x, a);
  }
  a += __shfl_xor_sync(0xffffffffu, a, 1);
  return a + __shfl_xor_sync(0xffffffffu, a, 2);
}

// Raises *m to the largest exponent of a squared norm of a warp's eight rows.  A
// row that is not finite has values of zero and NaN keys: no part in the bound.
// Squares that leave 32 bits are taken again of scaled channels (2^70: squares of
// 2^128 / 2^70 and of 2^-133 2^70 stay inside).
__device__ __forceinline__ void note_norm(const __nv_bfloat16* row, int part, int* m) {
  float sq = row_norm_sq(row, part);
  int up = 0;
  if (__any_sync(0xffffffffu, !(sq >= 0x1p-100f && sq < INFINITY))) {
    const float large = row_norm_sq_scaled(row, part, 0x1p-70f);
    const float small = row_norm_sq_scaled(row, part, 0x1p70f);
    if (sq < 0x1p-100f) {
      sq = small;
      up = -140;
    } else if (!(sq < INFINITY)) {      // NaN stays NaN
      sq = large;
      up = 140;
    }
  }
  const int e = sq > 0.f && sq < INFINITY ? ilogbf(sq) + up : kNoNorm;
  const int top = __reduce_max_sync(0xffffffffu, e);
  if ((threadIdx.x & 31) == 0) atomicMax(m, top);
}

// need and full of query tile t of an item, by 256 threads.
__device__ void item_tiles(const ChunkArgs& a, ck::Item& item, int t, const PageEntry* pages) {
  __shared__ int q_max, q_min, need, full;
  if (threadIdx.x == 0) {
    q_max = INT32_MIN;
    q_min = INT32_MAX;
    need = 0;
    full = INT32_MAX;
  }
  __syncthreads();
  const int first = t * ck::kPairTile, n = min(item.n - first, ck::kPairTile);
  for (int i = threadIdx.x; i < n; i += 256) {
    const int qp = a.q_pos[item.tok0 + first + i];
    atomicMax(&q_max, qp);
    atomicMin(&q_min, qp);
  }
  __syncthreads();
  if (n > 0)
    for (int j = threadIdx.x; j < item.tiles; j += 256) {
      const PageEntry e0 = pages[item.entry + 2 * j], e1 = pages[item.entry + 2 * j + 1];
      if (ck::visible(e0, q_max) > 0 || ck::visible(e1, q_max) > 0) atomicMax(&need, j + 1);
      if (ck::visible(e0, q_min) < kPage || ck::visible(e1, q_min) < kPage) atomicMin(&full, j);
    }
  __syncthreads();
  if (threadIdx.x == 0) {
    item.need[t] = need;
    item.full[t] = full;
  }
}

// Blocks [0, cap): rotary keys of the listed pages at their request positions,
// kr[64 e + r] = R(delta[version]) k_rope of page entry e's row r (a plain copy
// where delta is zero; rows without data are zeros), and the largest norm of
// each sequence's latents.  The blocks after them: the largest norm of 64 rows of
// W_UV each, into their head's.  The latents and weights read here are read again by the expansion,
// from L2.  256 threads, four a row.  The last blocks: what each query tile of an
// item sees (ck::Item::need and full), once for all heads: as a part of the
// attention's own prologue it took 2 us of every 30 us item of a short context.
// (Without kNorms, the rotary keys alone.)
template <bool kNorms>
__global__ void __launch_bounds__(256) chunk_rotary_kernel(const __grid_constant__ ChunkArgs a,
                                                           int cap, const ChunkPlan* plan,
                                                           const PageEntry* pages,
                                                           const __nv_bfloat16* w_uv,
                                                           __nv_bfloat16* kr, ck::Item* items,
                                                           int* norm_c, int* norm_w) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ double2 cs[ck::kDr / 2];
  const int r = threadIdx.x >> 2, part = threadIdx.x & 3;
  if (kNorms && (int)blockIdx.x >= cap + a.H * ck::kDv / 64) {
    const int k = blockIdx.x - cap - a.H * ck::kDv / 64;
    if (k / 2 < plan->n_items) item_tiles(a, items[k / 2], k & 1, pages);
    return;
  }
  if ((int)blockIdx.x >= cap) {
    const int k = blockIdx.x - cap;
    note_norm(w_uv + ((size_t)k * 64 + r) * ck::kDc, part, &norm_w[k / (ck::kDv / 64)]);
    return;
  }
  if ((int)blockIdx.x >= 4 * plan->n_row_tiles) return;
  const PageEntry e = pages[blockIdx.x];
  const int delta = e.n > 0 ? a.delta[e.ver] : 0;
  if (delta != 0) {
    for (int i = threadIdx.x; i < ck::kDr / 2; i += 256)
      sincos((double)delta * pow(a.rope_base, -2.0 * i / ck::kDr), &cs[i].y, &cs[i].x);
    __syncthreads();
  }
  const __nv_bfloat16* row = static_cast<const __nv_bfloat16*>(a.cache) +
                             ((long long)e.row + r) * (ck::kDc + ck::kDr);
  uint4 u[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  if (r < e.n) {
    const uint4* src = reinterpret_cast<const uint4*>(row + ck::kDc + part * 16);
    u[0] = src[0];
    u[1] = src[1];
    if (delta != 0) {
      uint32_t* w = reinterpret_cast<uint32_t*>(u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double2 t = cs[part * 8 + i];
        const double x0 = lo_f(w[i]), x1 = hi_f(w[i]);
        w[i] = pack2((float)(x0 * t.x - x1 * t.y), (float)(x0 * t.y + x1 * t.x));
      }
    }
  }
  uint4* dst =
      reinterpret_cast<uint4*>(kr + ((long long)blockIdx.x * kPage + r) * ck::kDr + part * 16);
  dst[0] = u[0];
  dst[1] = u[1];
  // rows 8 w .. 8 w + 7 of warp w; beyond the page's data the last row again
  if (kNorms && e.n > 0)
    note_norm(row - (r < e.n ? 0 : (r - e.n + 1) * (ck::kDc + ck::kDr)), part, &norm_c[e.seq]);
}

// ------------------------------------------------------------ absorbed route
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four 8 x 8 tiles of 16-bit elements, a row address per lane (tile lane / 8).
template <bool kTurned>
__device__ __forceinline__ void load_tiles(const __nv_bfloat16* p, uint32_t (&x)[4]) {
  if constexpr (kTurned)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(smem_u32(p)) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(smem_u32(p)) : "memory");
}

// Absorbed queries q_abs[t, h] = [W_UK[h]^T q_nope | q_rope] (Day 27 tutorial "Move
// the Key Projection Into the Query"; the rotary part is rotated already).  Block
// (64 latent channels, head, 64 tokens), four warps of 16 channels each; W_UK[h]'s
// rows are channels, so its tiles are turned on their way from shared memory
// (mma.sync: for few tokens the weights' stream is what the product costs).  All
// loads of a block are under way at once, and the small blocks of 16 tokens
// and 128 heads fill every SM several times.  The decode's absorption takes its
// queries in two arrays, which a launch before it had to split, and 128 tokens a
// launch: with it a call over 1000 rows took 286 us for 512 tokens of 64 heads, 48
// for 256 of 8 and 32 for one of 128 heads, this way 260, 37 and 34.  16 tokens of
// 128 heads: 8.6 us (17 MB of weights, 2 TB/s).
constexpr int kFaThreads = 128, kFaTokens = 64, kFaCols = 64, kFaK = 128;
constexpr int kFaPitchW = kFaCols + 8, kFaPitchQ = kFaK + 8;

__global__ void __launch_bounds__(kFaThreads) few_absorb_kernel(int n, int H, int d_n,
                                                                const __nv_bfloat16* q,
                                                                const __nv_bfloat16* w_uk,
                                                                __nv_bfloat16* q_abs) {
  asm volatile("griddepcontrol.launch_dependents;");
  __shared__ __align__(16) __nv_bfloat16 sw[kFaK * kFaPitchW], sq[kFaTokens * kFaPitchQ];
  const int part = blockIdx.x, h = blockIdx.y, t0 = blockIdx.z * kFaTokens;
  const int nt = min(kFaTokens, n - t0), mt = (nt + 15) / 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int width = d_n + fw::kDr;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  float d[kFaTokens / 16][2][4] = {};
  for (int k0 = 0; k0 < d_n; k0 += kFaK) {
    const int kc = min(kFaK, d_n - k0), ks = (kc + 15) / 16;
    // every load before the first store, which the compiler may not pass
    constexpr int kW = kFaK * (kFaCols / 8) / kFaThreads, kQ = kFaTokens * (kFaK / 8) / kFaThreads;
    uint4 xw[kW], xq[kQ];
#pragma unroll
    for (int u = 0; u < kW; ++u) {
      const int i = threadIdx.x + u * kFaThreads, k = i / (kFaCols / 8), c = i % (kFaCols / 8) * 8;
      xw[u] = k < kc ? *reinterpret_cast<const uint4*>(w_uk + ((size_t)h * d_n + k0 + k) * fw::kDc +
                                                       part * kFaCols + c)
                     : zero;
    }
#pragma unroll
    for (int u = 0; u < kQ; ++u) {
      const int i = threadIdx.x + u * kFaThreads, t = i / (kFaK / 8), k = i % (kFaK / 8) * 8;
      xq[u] = t < nt && k < kc ? *reinterpret_cast<const uint4*>(
                                     q + ((size_t)(t0 + t) * H + h) * width + k0 + k)
                               : zero;
    }
    if (k0) __syncthreads();
#pragma unroll
    for (int u = 0; u < kW; ++u) {
      const int i = threadIdx.x + u * kFaThreads, k = i / (kFaCols / 8), c = i % (kFaCols / 8) * 8;
      *reinterpret_cast<uint4*>(sw + k * kFaPitchW + c) = xw[u];
    }
#pragma unroll
    for (int u = 0; u < kQ; ++u) {
      const int i = threadIdx.x + u * kFaThreads, t = i / (kFaK / 8), k = i % (kFaK / 8) * 8;
      *reinterpret_cast<uint4*>(sq + t * kFaPitchQ + k) = xq[u];
    }
    __syncthreads();
    const int in = lane & 7, lo = lane >> 3 & 1, hi = lane >> 4;
#pragma unroll
    for (int s = 0; s < kFaK / 16; ++s) {
      if (s >= ks) break;
      uint32_t b[4];
      load_tiles<true>(sw + (16 * s + 8 * lo + in) * kFaPitchW + 16 * warp + 8 * hi, b);
#pragma unroll
      for (int m = 0; m < kFaTokens / 16; ++m) {
        if (m >= mt) break;
        uint32_t a[4];
        load_tiles<false>(sq + (16 * m + 8 * lo + in) * kFaPitchQ + 16 * s + 8 * hi, a);
        mma_16x8x16(d[m][0], a[0], a[1], a[2], a[3], b[0], b[1]);
        mma_16x8x16(d[m][1], a[0], a[1], a[2], a[3], b[2], b[3]);
      }
    }
  }
  // through shared memory, so that a row's 128 bytes are written together
  __syncthreads();
#pragma unroll
  for (int m = 0; m < kFaTokens / 16; ++m)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t* o = reinterpret_cast<uint32_t*>(
          sw + (16 * m + 8 * half + (lane >> 2)) * kFaPitchW + 16 * warp + 2 * (lane & 3));
      o[0] = pack2(d[m][0][2 * half], d[m][0][2 * half + 1]);
      o[4] = pack2(d[m][1][2 * half], d[m][1][2 * half + 1]);
    }
  __syncthreads();
#pragma unroll
  for (int i = threadIdx.x; i < kFaTokens * (kFaCols / 8); i += kFaThreads) {
    const int t = i / (kFaCols / 8), c = i % (kFaCols / 8) * 8;
    if (t < nt)
      *reinterpret_cast<uint4*>(q_abs + ((size_t)(t0 + t) * H + h) * fw::kWidth + part * kFaCols + c) =
          *reinterpret_cast<const uint4*>(sw + t * kFaPitchW + c);
  }
  if (part == 0)
    for (int i = threadIdx.x; i < nt * (fw::kDr / 8); i += kFaThreads) {
      const size_t at = (size_t)(t0 + i / (fw::kDr / 8)) * H + h;
      const int c = i % (fw::kDr / 8) * 8;
      *reinterpret_cast<uint4*>(q_abs + at * fw::kWidth + fw::kDc + c) =
          *reinterpret_cast<const uint4*>(q + at * width + d_n + c);
    }
}

// The shares of a row merged by log-sum-exp and the value expansion, in one
// launch: block (head, 16 tokens), 512 threads.
//   Join, a warp per token: a lane per share for the weights, then a lane per four
//   columns of 128.  o is kept as two bf16 (its rounding and what that leaves).
//   v = W_UV[h] o: 16 x 8 products of 16 (mma.sync: with 16 rows the weights'
//   stream is what they cost), a warp for two groups of eight value channels and
//   half of the latent's.  The order of the 32 channels of a step does not matter as
//   long as both operands have the same: a lane takes eight consecutive ones of its
//   row of either, so that a load is 16 bytes and feeds two products; a pitch of 16
//   words modulo 32 keeps the rows of a load of shared memory apart.
// Tokens of no sequence keep what their rows held.  A join, the value product of
// mla_out_proj and a store as three launches took 424 us for 512 tokens of 64 heads
// over 1000 rows each, the whole call, where this took 286, and 43 for 16 tokens
// where it took 38.  16 tokens of 128 heads: 17 us from memory (34 MB, 2 TB/s).
constexpr int kFvTokens = 16, kFvThreads = 512, kFvPitch = fw::kDc + 32;

// o in two parts; weights of the shares, later the sums of eight warps
size_t few_value_smem(int pairs) {
  return sizeof(__nv_bfloat16) * 2 * kFvTokens * kFvPitch +
         std::max(sizeof(float) * kFvTokens * (size_t)pairs, sizeof(float4) * 16 * 32);
}

__global__ void __launch_bounds__(kFvThreads) few_value_kernel(
    int n, int H, int d_v, int pairs, const fw::Plan* plan, const fw::Stream* streams,
    const FewToken* tokens, const float* partial, const float* partial_lse, const __nv_bfloat16* w_uv,
    __nv_bfloat16* out, float* lse) {
  extern __shared__ __align__(16) uint8_t sm_fv[];
  __nv_bfloat16* o_hi = reinterpret_cast<__nv_bfloat16*>(sm_fv);       // [16][pitch]
  __nv_bfloat16* o_lo = o_hi + kFvTokens * kFvPitch;
  float* weight = reinterpret_cast<float*>(o_lo + kFvTokens * kFvPitch);   // [16][pairs]
  const int h = blockIdx.x, t0 = blockIdx.y * kFvTokens;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int run = plan->chunk;
  {
    const int i = warp, t = t0 + i;
    float4 acc[4] = {};
    const FewToken tok = t < n ? tokens[t] : FewToken{kNone, 0, 0};
    if (tok.state == kLive) {
      const int r = t * H + h;
      const int si = tok.stream + (r - tok.row) / fw::kRows;
      const fw::Stream s = streams[si];
      const int in = r - s.q_row;
      const int g0 = s.tiles > 0 ? s.off / run : 0;
      const int ng = s.tiles > 0 ? (s.off + s.tiles - 1) / run - g0 + 1 : 0;
      const float* ls = partial_lse + (size_t)(g0 + si) * fw::kRows + in;
      float top = kNegInf;
      bool nan = false;
      for (int g = lane; g < ng; g += 32) {
        const float x = ls[(size_t)g * fw::kRows];
        nan = nan || x != x;
        top = fmaxf(top, x);
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      if (__any_sync(0xffffffffu, nan)) top = kNaN;
      float tot = 0.f;
      if (top != kNegInf)
        for (int g = lane; g < ng; g += 32) {
          const float w = __expf(ls[(size_t)g * fw::kRows] - top);
          weight[i * pairs + g] = w;
          tot += w;
        }
#pragma unroll
      for (int d = 16; d; d >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, d);
      __syncwarp();
      if (lse && lane == 0) lse[r] = tot == 0.f ? kNegInf : top + logf(tot);
      if (tot != 0.f) {
        const float4* src = reinterpret_cast<const float4*>(partial) +
                            ((size_t)(g0 + si) * (fw::kDc / 4) + lane) * fw::kRows + in;
#pragma unroll 4
        for (int g = 0; g < ng; ++g) {
          const float w = weight[i * pairs + g];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float4 x = src[((size_t)g * (fw::kDc / 4) + 32 * c) * fw::kRows];
            acc[c].x = fmaf(w, x.x, acc[c].x);
            acc[c].y = fmaf(w, x.y, acc[c].y);
            acc[c].z = fmaf(w, x.z, acc[c].z);
            acc[c].w = fmaf(w, x.w, acc[c].w);
          }
        }
        const float inv = 1.f / tot;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          acc[c].x *= inv;
          acc[c].y *= inv;
          acc[c].z *= inv;
          acc[c].w *= inv;
        }
      }
    } else if (tok.state == kBad && lse && lane == 0) {
      lse[(size_t)t * H + h] = kNaN;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float4 x = acc[c];
      const uint32_t w0 = pack2(x.x, x.y), w1 = pack2(x.z, x.w);
      const int at = i * kFvPitch + 128 * c + 4 * lane;
      *reinterpret_cast<uint2*>(o_hi + at) = make_uint2(w0, w1);
      *reinterpret_cast<uint2*>(o_lo + at) =
          make_uint2(pack2(x.x - lo_f(w0), x.y - hi_f(w0)), pack2(x.z - lo_f(w1), x.w - hi_f(w1)));
    }
  }
  __syncthreads();

  const int row = lane >> 2, part = lane & 3;
  const __nv_bfloat16* a_hi = o_hi + row * kFvPitch + 8 * part;
  const __nv_bfloat16* a_lo = o_lo + row * kFvPitch + 8 * part;
  auto words = [](const __nv_bfloat16* p) { return *reinterpret_cast<const uint4*>(p); };
  const int first = warp >> 3 ? fw::kDc / 2 : 0;      // latent channels of this warp
  float4* other = reinterpret_cast<float4*>(weight);  // the upper half's sums
  for (int j0 = 0; j0 < (d_v + 7) / 8; j0 += 16) {
    const int c0 = 8 * (j0 + (warp & 7));             // value channels c0 .. + 7, c0 + 64 .. + 7
    const __nv_bfloat16* w[2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
      w[u] = w_uv + ((size_t)h * d_v + min(c0 + 64 * u + row, d_v - 1)) * fw::kDc + 8 * part;
    float d[2][4] = {};
    if (c0 < d_v) {
#pragma unroll 4
      for (int k = first; k < first + fw::kDc / 2; k += 32) {
        const uint4 b[2] = {words(w[0] + k), words(w[1] + k)};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const __nv_bfloat16* a = (half ? a_lo : a_hi) + k;
          const uint4 x = words(a), y = words(a + 8 * kFvPitch);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            mma_16x8x16(d[u], x.x, y.x, x.y, y.y, b[u].x, b[u].y);
            mma_16x8x16(d[u], x.z, y.z, x.w, y.w, b[u].z, b[u].w);
          }
        }
      }
    }
    __syncthreads();
    if (warp >= 8) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
        other[(2 * (warp & 7) + u) * 32 + lane] = make_float4(d[u][0], d[u][1], d[u][2], d[u][3]);
    }
    __syncthreads();
    if (warp >= 8) continue;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float4 x = other[(2 * warp + u) * 32 + lane];
      const float y[4] = {d[u][0] + x.x, d[u][1] + x.y, d[u][2] + x.z, d[u][3] + x.w};
      const int c = c0 + 64 * u + 2 * part;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int t = t0 + row + 8 * half;
        const int st = t < n ? tokens[t].state : kNone;
        if (st == kNone) continue;
        __nv_bfloat16* o = out + ((size_t)t * H + h) * d_v + c;
        const float y0 = st == kBad ? kNaN : y[2 * half], y1 = st == kBad ? kNaN : y[2 * half + 1];
        if (c + 1 < d_v && d_v % 2 == 0) *reinterpret_cast<uint32_t*>(o) = pack2(y0, y1);
        else if (c < d_v) {
          o[0] = __float2bfloat16_rn(y0);
          if (c + 1 < d_v) o[1] = __float2bfloat16_rn(y1);
        }
      }
    }
  }
}

// ------------------------------------------------------------ generic widths
// One block per (token, head), any widths, fp32 arithmetic: the head's absorbed
// query W_UK[h]^T q_nope and its rotary part turned by -delta[version] (in
// shared memory, not rounded), an online softmax over chunks of 128 rows, and
// the value expansion.  Scores: four threads a row, so that a load of a warp
// touches eight rows and a thread's loads are all under way at once (a thread a
// row waited 11 000 clocks a chunk of 48-wide rows for its line-by-line loads).
// Weighted sum: (row group, channels), so that narrow latents keep all threads
// at work.  kVec: four elements a load, for widths that are multiples of four.
// A masked row is not read.  Bound by the latency of its chain: 8 heads, 75
// tokens over up to 331 rows of 48 take 18.5 us (33 with a thread a row).
constexpr int kGenThreads = 128;

int generic_groups(int d_c, bool vec) {
  const int units = vec ? d_c / 4 : d_c;
  int wide = 1;
  while (wide < units && wide < kGenThreads) wide *= 2;
  return kGenThreads / wide;
}

bool generic_vec(const mla_dims_t* d) { return d->d_c % 4 == 0 && d->d_r % 4 == 0; }

size_t generic_smem(const mla_dims_t* d, int n_ver) {
  const size_t row = (size_t)d->d_c + d->d_r, query = n_ver * row + d->d_n + d->d_r;
  return sizeof(float) * ((query + 3) / 4 * 4 +
                          (size_t)generic_groups(d->d_c, generic_vec(d)) * d->d_c +
                          2 * kGenThreads + 8) +
         sizeof(int) * kGenThreads;
}

// n consecutive elements, n = 4 (aligned to them) or 1
template <int n, typename T>
__device__ __forceinline__ void load_some(const T* src, float (&x)[n]) {
  if constexpr (n == 1) {
    x[0] = to_f(src[0]);
  } else if constexpr (sizeof(T) == 4) {
    const float4 u = *reinterpret_cast<const float4*>(src);
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(src);
    x[0] = lo_f(u.x); x[1] = hi_f(u.x); x[2] = lo_f(u.y); x[3] = hi_f(u.y);
  }
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kGenThreads) chunk_generic_kernel(
    const __grid_constant__ ChunkArgs a, int cap, int d_c, int groups, float scale, const T* w_uk,
    const T* w_uv, T* v, float* lse) {
  constexpr int V = kVec ? 4 : 1;
  extern __shared__ __align__(16) float sm_gen[];
  const int t = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = d_c + a.d_r;
  float* qa = sm_gen;                        // [n_ver][row]
  float* qn = qa + a.n_ver * row;            // [d_n + d_r]
  float* acc = sm_gen + (a.n_ver * row + a.d_n + a.d_r + 3) / 4 * 4;   // [groups][d_c]
  float* pw = acc + groups * d_c;            // [128] weights of the chunk
  float* score = pw + kGenThreads;           // [128]
  float* red = score + kGenThreads;          // [8]
  int* prow = reinterpret_cast<int*>(red + 8);   // [128] cache rows, -1: none
  __shared__ long long page_scratch[kGenThreads / 32], n_pg;
  __shared__ int s_b, s_np, s_bad, latest, scratch[kGenThreads / 32];
  __shared__ PageEntry s_page[2][2];         // the pages of this chunk and of the next one
  if (tid == 0) {
    s_b = -1;
    s_bad = 0;
    latest = INT32_MIN;
    n_pg = 0;
  }
  const T* q = static_cast<const T*>(a.q) + ((size_t)t * a.H + h) * (a.d_n + a.d_r);
  for (int k = tid; k < a.d_n + a.d_r; k += kGenThreads) qn[k] = to_f(q[k]);
  for (int k = tid; k < groups * d_c; k += kGenThreads) acc[k] = 0.f;
  __syncthreads();
  // ranges that hold are disjoint: at most one thread finds the token in its own
  for (int b0 = 0; b0 < a.B; b0 += kGenThreads) {
    const int b = b0 + tid;
    SeqRange r = read_sequence(a, b, scratch, &latest);
    const long long np = (r.pages + 1) / 2 * 2;      // as chunk_plan_kernel counts them
    const long long po = block_scan(np, page_scratch, &n_pg);
    if (b < a.B && po + np > cap) r.wrong = true;
    if (r.wrong) set_status(MLA_ERR_BAD_INDEX);
    if (r.tokens > 0 && t >= a.tok_start[b] && t - a.tok_start[b] < r.tokens) {
      s_b = b;
      s_np = r.wrong ? 0 : r.pages;
      s_bad = r.wrong;
    }
  }
  for (int c = tid; c < d_c; c += kGenThreads) {
    const T* w = w_uk + (size_t)h * a.d_n * d_c + c;
    float s = 0.f;
#pragma unroll 8
    for (int k = 0; k < a.d_n; ++k) s = fmaf(to_f(w[(size_t)k * d_c]), qn[k], s);
    for (int u = 0; u < a.n_ver; ++u) qa[u * row + c] = s;
  }
  for (int i = tid; i < a.n_ver * (a.d_r / 2); i += kGenThreads) {
    const int u = i / (a.d_r / 2), k = i % (a.d_r / 2);
    const float x0 = qn[a.d_n + 2 * k], x1 = qn[a.d_n + 2 * k + 1];
    double sn = 0.0, cs = 1.0;
    if (a.delta[u] != 0) sincos(-(double)a.delta[u] * pow(a.rope_base, -2.0 * k / a.d_r), &sn, &cs);
    qa[u * row + d_c + 2 * k] = (float)(x0 * cs - x1 * sn);
    qa[u * row + d_c + 2 * k + 1] = (float)(x0 * sn + x1 * cs);
  }
  __syncthreads();
  const int b = s_b;
  if (b < 0) return;
  const int np = s_np;
  PageEntry e;
  for (int k = tid; k < np; k += kGenThreads)
    if (!page_at(a, b, k, &e)) s_bad = 1;
  __syncthreads();
  const size_t at = (size_t)t * a.H + h;
  if (s_bad) {
    if (tid == 0) set_status(MLA_ERR_BAD_INDEX);
    for (int d = tid; d < a.d_v; d += kGenThreads) v[at * a.d_v + d] = from_f<T>(kNaN);
    if (lse && tid == 0) lse[at] = kNaN;
    return;
  }
  const T* cache = static_cast<const T*>(a.cache);
  const int qp = a.q_pos[t];
  const int wide = kGenThreads / groups;
  auto list_pages = [&](int i) {             // the pages of the i-th chunk
    if (tid >= 2) return;
    PageEntry x = {0, 0, 0, 0};
    if (2 * i + tid < np) page_at(a, b, 2 * i + tid, &x);
    s_page[i & 1][tid] = x;
  };
  // row r of the chunk: its cache row, -1 where there is none that the token sees
  auto row_of = [&](const PageEntry* pages, int r) {
    const PageEntry& x = pages[r / kPage];
    return r % kPage < x.n && (long long)x.kpos + r % kPage <= qp ? x.row + r % kPage : -1;
  };
  float m = kNegInf, l = 0.f;
  list_pages(0);
  __syncthreads();
  for (int base = 0; base < np * kPage; base += kGenThreads) {
    const PageEntry* pages = s_page[(base / kGenThreads) & 1];
    list_pages(base / kGenThreads + 1);
    const int part = tid & 3;
#pragma unroll
    for (int i = 0; i < kGenThreads / 32; ++i) {
      const int at = i * 32 + tid / 4, phys = row_of(pages, at);
      float d[V] = {};
      if (phys >= 0) {
        const T* r = cache + (size_t)phys * row;
        const float* x = qa + pages[at / kPage].ver * row;
#pragma unroll 4
        for (int k = part * V; k < row; k += 4 * V) {
          float y[V], z[V];
          load_some<V>(r + k, y);
          load_some<V>(x + k, z);
#pragma unroll
          for (int u = 0; u < V; ++u) d[u] = fmaf(z[u], y[u], d[u]);
        }
      }
      float s = kVec ? (d[0] + d[V / 2]) + (d[V / 4] + d[V - 1]) : d[0];
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      if (part == 0) score[at] = s * scale;
    }
    __syncthreads();
    const int phys = row_of(pages, tid);
    const float s = phys < 0 ? kNegInf : score[tid];
    // the chunk's maximum and sum; a NaN score makes the sum NaN
    float mx = s;
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane == 0) red[warp] = mx;
    __syncthreads();
    const float m_new = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float p = phys < 0 ? 0.f : expf(s - (m_new == kNegInf ? 0.f : m_new));
    pw[tid] = p;
    prow[tid] = phys;
    float sum = p;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) red[4 + warp] = sum;
    __syncthreads();
    const float f = m == kNegInf ? 0.f : expf(m - m_new);
    l = l * f + ((red[4] + red[5]) + (red[6] + red[7]));
    m = m_new;
    for (int c = tid % wide * V; c < d_c; c += wide * V) {
      float* o = acc + (tid / wide) * d_c + c;
      float sum_c[V];
#pragma unroll
      for (int u = 0; u < V; ++u) sum_c[u] = o[u] * f;
#pragma unroll 8
      for (int k = tid / wide; k < kGenThreads; k += groups) {
        float y[V] = {};
        if (prow[k] >= 0) load_some<V>(cache + (size_t)prow[k] * row + c, y);
#pragma unroll
        for (int u = 0; u < V; ++u) sum_c[u] = fmaf(pw[k], y[u], sum_c[u]);
      }
#pragma unroll
      for (int u = 0; u < V; ++u) o[u] = sum_c[u];
    }
    __syncthreads();
  }
  const bool none = l == 0.f;
  for (int c = tid; c < d_c; c += kGenThreads) {
    float o = 0.f;
    for (int g = 0; g < groups; ++g) o += acc[g * d_c + c];
    acc[c] = none ? 0.f : o / l;
  }
  __syncthreads();
  for (int d = warp; d < a.d_v; d += kGenThreads / 32) {
    const T* w = w_uv + ((size_t)h * a.d_v + d) * d_c;
    float s = 0.f;
    for (int c = lane; c < d_c; c += 32) s = fmaf(to_f(w[c]), acc[c], s);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) v[at * a.d_v + d] = from_f<T>(s);
  }
  if (lse && tid == 0) lse[at] = none ? kNegInf : m + logf(l);
}

// ------------------------------------------------------------ host
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

bool expandable(const mla_dims_t* d) {
  return d->dtype == MLA_BF16 && d->d_c == ck::kDc && d->d_r == ck::kDr && d->d_n == ck::kDn &&
         d->d_v == ck::kDv;
}

// rows of the absorbed route; query parts in 16-byte words
bool decodable(const mla_dims_t* d) {
  return d->dtype == MLA_BF16 && d->d_c == ck::kDc && d->d_r == ck::kDr && d->d_n % 8 == 0;
}

struct Layout {
  bool expanded, generic;
  int cap;                     // page entries
  // expanded
  int heads, groups;           // heads per launch; launches
  long long rows_cap;
  size_t k, v, norms, as_half;
  // both
  size_t plan, seq, items, pages, kr;
  // absorbed
  int slab, max_streams;       // tokens of a pass; streams of a pass at most
  size_t few_plan, streams, tokens, q_abs, partial, partial_lse;
  size_t total;
};

// Expanded when its estimated time (microseconds) is the lower one.  The host knows
// the tokens and the rows of all sequences only, and one route serves the whole
// call: the estimates take every sequence to be of the average size, and both
// sides were measured on equal ones.  A chunk beside many single tokens counts as
// rows x average tokens, below what the absorbed route then computes.
//   Expanded: a row's expansion costs 2 * 512 * 256 flops a head at 1.15 PFLOP/s;
//   a query, row and head 2 * 320 at 0.7, in query tiles of 256, but no less than
//   one item's way through a sequence, 1.9 us per 128 rows.
//   Absorbed: a query, row and head 2 * 1088 at 0.76 PFLOP/s, 5.5 ns a query and
//   head for absorption, partial sums and value expansion.
// Tokens a sequence at which the two take the same time, measured and by this
// estimate, and that time (sequences x cached rows):
//                1 x 4096        4 x 2048        16 x 1024       1 x 16384
//   16 heads     172, 235; 93    82, 69; 88      69, 53; 165     310, 347; 302
//   64 heads     82, 100; 137    79, 82; 264     61, 57; 545     127, 141; 458
//   128 heads    90, 106; 268    75, 84; 500     61, 58; 1150    135, 143; 970
bool chunk_route(const mla_dims_t* d, int B, int n_tok, long long max_rows) {
  if (!expandable(d)) return false;
  const double rows = (double)max_rows, heads = d->H, per = std::ceil((double)n_tok / B);
  const double e = 25 + rows * heads * 262144.0 / 1.15e9 +
                   std::max(rows * heads * std::ceil(per / 256) * 256 * 640.0 / 0.7e9,
                            rows / B / 128 * 1.9);
  const double s = 38 + rows * per * heads * 2176.0 / 0.76e9 + n_tok * heads * 0.0055;
  return e < s;
}

bool make_layout(const mla_dims_t* d, int B, int n_tok, int n_ver, int max_pages, int max_segs,
                 long long max_rows, Layout* l) {
  *l = Layout{};
  if (d->H > 65535) return false;       // grid limit
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = up256(at + bytes);
    return here;
  };
  // page entries, an even number a sequence
  const long long cap = ((max_rows + kPage - 1) / kPage + B + 3) / 4 * 4;
  l->cap = (int)std::min<long long>(cap, INT32_MAX);
  l->expanded = chunk_route(d, B, n_tok, max_rows);
  l->generic = !decodable(d);
  if (l->generic) {        // 48 KB of shared memory, a little of it static
    if (generic_smem(d, n_ver) > 48 * 1024 - 256) return false;
    take(256);        // it needs none; an empty workspace is not told from an error
    l->total = at;
    return true;
  }
  l->plan = take(sizeof(ChunkPlan));
  l->seq = take(sizeof(int) * (3 * (size_t)B + 2));
  l->items = take(sizeof(ck::Item) * ((size_t)n_tok / ck::kItemTokens + B));
  l->pages = take(sizeof(PageEntry) * (size_t)cap);
  l->kr = take((size_t)cap * kPage * ck::kDr * 2);
  if (l->expanded) {
    l->rows_cap = cap * kPage;
    const size_t head = (size_t)l->rows_cap * (ck::kDn + ck::kDv) * 2;
    int hg = (int)std::min<size_t>(d->H, std::max<size_t>(1, ((size_t)1 << 30) / head));
    l->groups = (d->H + hg - 1) / hg;
    l->heads = (d->H + l->groups - 1) / l->groups;
    if (l->rows_cap * l->heads + 4 * kPage > INT32_MAX) return false;
    l->k = take((size_t)l->rows_cap * l->heads * ck::kDn * 2);
    l->v = take((size_t)l->rows_cap * l->heads * ck::kDv * 2);
    l->norms = take(sizeof(int) * ((size_t)B + d->H));
    l->as_half = take((size_t)l->rows_cap / ck::kKTile * l->heads);
  } else {
    // tokens per pass: 32768 (token, head) rows, which bounds the workspace
    l->slab = std::min(n_tok, std::max(1, 32768 / d->H));
    const size_t n = l->slab, rows = n * d->H;
    const int pairs = current_sms() / 2;
    if (pairs == 0) return false;
    l->max_streams = (int)(rows / fw::kRows) + std::min(B, l->slab);   // with a token in it
    // (stream, page) units and rows of the page list are counted in 32 bits
    if (cap * kPage > INT32_MAX ||
        (long long)(rows / fw::kRows) * std::min<long long>(cap, max_pages) + cap > INT32_MAX)
      return false;
    l->few_plan = take(sizeof(fw::Plan));
    l->streams = take(sizeof(fw::Stream) * (size_t)l->max_streams);
    l->tokens = take(n * sizeof(FewToken));
    l->q_abs = take(rows * fw::kWidth * 2);
    const size_t slots = (size_t)pairs + l->max_streams;
    l->partial = take(slots * fw::kRows * fw::kDc * 4);
    l->partial_lse = take(slots * fw::kRows * 4);
  }
  l->total = at;
  return true;
}

bool chunk_dims_ok(const mla_dims_t* d) {
  return d && d->H > 0 && d->d_c > 0 && d->d_r > 0 && d->d_r % 2 == 0 && d->d_n > 0 &&
         d->d_v > 0 && (d->dtype == MLA_F32 || d->dtype == MLA_BF16) && std::isfinite(d->scale) &&
         d->scale > 0.f && d->rope_base > 0.0;
}

mla_status_t run_expanded(const mla_dims_t* d, const ChunkArgs& a, const Layout& l, uint8_t* ws,
                          const void* w_uk, const void* w_uv, void* v, float* lse, cudaStream_t st) {
  const int sms = current_sms();
  if (!sms) return MLA_ERR_CUDA;
  ChunkPlan* plan = reinterpret_cast<ChunkPlan*>(ws + l.plan);
  ck::Item* items = reinterpret_cast<ck::Item*>(ws + l.items);
  PageEntry* pages = reinterpret_cast<PageEntry*>(ws + l.pages);
  __nv_bfloat16* kr = reinterpret_cast<__nv_bfloat16*>(ws + l.kr);
  int* norm_c = reinterpret_cast<int*>(ws + l.norms);
  int* norm_w = norm_c + a.B;
  const uint64_t cache_rows = (uint64_t)a.n_pages * kPage;

  ex::Maps xm;
  ck::Maps mp;
  const uint64_t q_ext[3] = {64, (uint64_t)a.n_tok, 3ull * d->H};
  const uint64_t q_str[2] = {(uint64_t)d->H * (ck::kDn + ck::kDr) * 2, 128};
  const uint32_t q_box[3] = {64, ck::kQTile, 3};
  const uint64_t s_ext[3] = {64, (uint64_t)l.rows_cap * l.heads, 2};
  const uint64_t s_str[2] = {(uint64_t)ck::kDn * 2, 128};
  const uint32_t k_box[3] = {64, ck::kKTile / 2, 2}, v_box[3] = {64, ck::kKTile, 1};
  const uint32_t o_box[3] = {64, 32, 1};
  if (!map_rows(&xm.c, a.cache, ck::kDc, cache_rows, ck::kDc + ck::kDr, kPage) ||
      !map_bf16(&mp.q, a.q, 3, q_ext, q_str, q_box) ||
      !map_bf16(&mp.k, ws + l.k, 3, s_ext, s_str, k_box) ||
      !map_bf16(&mp.v, ws + l.v, 3, s_ext, s_str, v_box) ||
      !map_bf16(&xm.k, ws + l.k, 3, s_ext, s_str, o_box) ||
      !map_bf16(&xm.v, ws + l.v, 3, s_ext, s_str, o_box) ||
      !map_rows(&mp.kr, kr, ck::kDr, (uint64_t)l.rows_cap, ck::kDr, ck::kKTile / 2))
    return MLA_ERR_CUDA;
  if (cudaFuncSetAttribute(ex::expand_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           ex::kSmemBytes) != cudaSuccess ||
      cudaFuncSetAttribute(ck::chunk_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           ck::kSmemBytes) != cudaSuccess)
    return MLA_ERR_CUDA;

  chunk_plan_kernel<false><<<1, kPlanThreads, 0, st>>>(
      a, FewPlan{}, l.cap, plan, reinterpret_cast<int*>(ws + l.seq), items, pages, norm_c,
      a.B + d->H);
  if (cudaGetLastError() != cudaSuccess) return MLA_ERR_CUDA;
  const int max_items = a.n_tok / ck::kItemTokens + a.B;
  if (launch_dependent(chunk_rotary_kernel<true>,
                       dim3(l.cap + d->H * ck::kDv / 64 + 2 * max_items), dim3(256), 0, st, true, a,
                       l.cap, plan, static_cast<const PageEntry*>(pages),
                       static_cast<const __nv_bfloat16*>(w_uv), kr, items, norm_c,
                       norm_w) != cudaSuccess)
    return MLA_ERR_CUDA;

  ex::Params g;
  g.pages = pages;
  g.plan = plan;
  g.rows_cap = l.rows_cap;
  g.norm_c = norm_c;
  g.as_half = ws + l.as_half;
  ck::Params p;
  p.plan = plan;
  p.items = items;
  p.pages = pages;
  p.q_pos = a.q_pos;
  p.H = d->H;
  p.rows_cap = l.rows_cap;
  p.norm_c = norm_c;
  p.as_half = ws + l.as_half;
  p.scale = d->scale;
  p.scale_log2 = d->scale * ck::kLog2e;
  p.v = static_cast<__nv_bfloat16*>(v);
  p.lse = lse;
  for (int h0 = 0; h0 < d->H; h0 += l.heads) {
    const int nh = std::min(l.heads, d->H - h0);
    const uint64_t w_rows = (uint64_t)nh * ck::kDn;
    if (!map_rows(&xm.uk, static_cast<const __nv_bfloat16*>(w_uk) + (size_t)h0 * ck::kDn * ck::kDc,
                  ck::kDc, w_rows, ck::kDc, 128) ||
        !map_rows(&xm.uv, static_cast<const __nv_bfloat16*>(w_uv) + (size_t)h0 * ck::kDv * ck::kDc,
                  ck::kDc, w_rows, ck::kDc, 128))
      return MLA_ERR_CUDA;
    g.n_heads = nh;
    g.norm_w = p.norm_w = norm_w + h0;
    const long long tiles = (long long)l.cap / 4 * nh;
    const int grid = 2 * (int)std::min<long long>(tiles, sms / 2 > 0 ? sms / 2 : 1);
    if (launch_dependent(ex::expand_kernel, dim3(grid), dim3(ex::kThreads), ex::kSmemBytes, st, true,
                         g, xm) != cudaSuccess)
      return MLA_ERR_CUDA;
    p.h0 = h0;
    p.n_heads = nh;
    if (launch_dependent(ck::chunk_attn_kernel, dim3(2 * max_items, nh), dim3(ck::kThreads),
                         ck::kSmemBytes, st, true, p, mp) != cudaSuccess)
      return MLA_ERR_CUDA;
  }
  return MLA_OK;
}

template <typename T>
mla_status_t run_generic(const mla_dims_t* d, const ChunkArgs& a, int cap, const void* w_uk,
                         const void* w_uv, void* v, float* lse, cudaStream_t st) {
  const bool vec = generic_vec(d);
  auto kernel = vec ? chunk_generic_kernel<T, true> : chunk_generic_kernel<T, false>;
  kernel<<<dim3(a.n_tok, d->H), kGenThreads, generic_smem(d, a.n_ver), st>>>(
      a, cap, d->d_c, generic_groups(d->d_c, vec), d->scale, static_cast<const T*>(w_uk),
      static_cast<const T*>(w_uv), static_cast<T*>(v), lse);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

mla_status_t run_absorbed(const mla_dims_t* d, const ChunkArgs& a, const Layout& l, uint8_t* ws,
                          const void* w_uk, const void* w_uv, void* v, float* lse,
                          cudaStream_t st) {
  const int pairs = current_sms() / 2;
  if (!pairs) return MLA_ERR_CUDA;
  ChunkPlan* cplan = reinterpret_cast<ChunkPlan*>(ws + l.plan);
  int* seq = reinterpret_cast<int*>(ws + l.seq);
  PageEntry* pages = reinterpret_cast<PageEntry*>(ws + l.pages);
  __nv_bfloat16* kr = reinterpret_cast<__nv_bfloat16*>(ws + l.kr);
  fw::Plan* plan = reinterpret_cast<fw::Plan*>(ws + l.few_plan);
  fw::Stream* streams = reinterpret_cast<fw::Stream*>(ws + l.streams);
  FewToken* tokens = reinterpret_cast<FewToken*>(ws + l.tokens);

  fw::Params p;
  p.plan = plan;
  p.streams = streams;
  p.pages = pages;
  p.H = d->H;
  p.rotary_moved = 0;
  for (int i = 0; i < a.n_ver; ++i) p.rotary_moved |= a.delta[i] != 0;
  p.scale = d->scale;
  p.scale_log2 = d->scale * fw::kLog2e;
  p.partial = reinterpret_cast<float*>(ws + l.partial);
  p.partial_lse = reinterpret_cast<float*>(ws + l.partial_lse);
  fw::Maps mp;
  const uint64_t cache_rows = (uint64_t)a.n_pages * kPage;
  const uint64_t c_ext[3] = {64, cache_rows, fw::kWidth / 64};
  const uint64_t c_str[2] = {(uint64_t)fw::kWidth * 2, 128};
  const uint32_t c_box[3] = {64, kPage, 4};
  if (!map_rows(&mp.c, a.cache, fw::kWidth, cache_rows, fw::kWidth, kPage) ||
      !map_bf16(&mp.c4, a.cache, 3, c_ext, c_str, c_box) ||
      !map_rows(&mp.kr, kr, fw::kDr, (uint64_t)l.cap * kPage, fw::kDr, kPage))
    return MLA_ERR_CUDA;
  if (cudaFuncSetAttribute(fw::few_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           fw::kSmemBytes) != cudaSuccess)
    return MLA_ERR_CUDA;
  const __nv_bfloat16* wv = static_cast<const __nv_bfloat16*>(w_uv);
  for (int t0 = 0; t0 < a.n_tok; t0 += l.slab) {
    const int n = std::min(l.slab, a.n_tok - t0), rows = n * d->H;
    const __nv_bfloat16* q =
        static_cast<const __nv_bfloat16*>(a.q) + (size_t)t0 * d->H * (d->d_n + d->d_r);
    few_absorb_kernel<<<dim3(fw::kDc / kFaCols, d->H, (n + kFaTokens - 1) / kFaTokens), kFaThreads,
                        0, st>>>(n, d->H, d->d_n, q, static_cast<const __nv_bfloat16*>(w_uk),
                                 reinterpret_cast<__nv_bfloat16*>(ws + l.q_abs));
    if (cudaGetLastError() != cudaSuccess) return MLA_ERR_CUDA;
    const FewPlan few = {t0, n, pairs, plan, streams, tokens};
    if (t0 == 0) {
      if (launch_dependent(chunk_plan_kernel<true>, dim3(1), dim3(kPlanThreads), 0, st, true, a, few,
                           l.cap, cplan, seq, reinterpret_cast<ck::Item*>(ws + l.items), pages,
                           static_cast<int*>(nullptr), 0) != cudaSuccess)
        return MLA_ERR_CUDA;
      if (p.rotary_moved &&
          launch_dependent(chunk_rotary_kernel<false>, dim3(l.cap), dim3(256), 0, st, true, a, l.cap,
                           cplan, static_cast<const PageEntry*>(pages), wv, kr,
                           static_cast<ck::Item*>(nullptr), static_cast<int*>(nullptr),
                           static_cast<int*>(nullptr)) != cudaSuccess)
        return MLA_ERR_CUDA;
    } else {
      few_plan_kernel<<<1, kPlanThreads, 0, st>>>(a, few, seq, pages);
      if (cudaGetLastError() != cudaSuccess) return MLA_ERR_CUDA;
    }
    p.q_pos = a.q_pos + t0;
    if (!map_rows(&mp.q, ws + l.q_abs, fw::kWidth, rows, fw::kWidth, fw::kRows))
      return MLA_ERR_CUDA;
    if (launch_dependent(fw::few_attn_kernel, dim3(2 * pairs), dim3(fw::kThreads), fw::kSmemBytes,
                         st, true, p, mp) != cudaSuccess)
      return MLA_ERR_CUDA;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(v) + (size_t)t0 * d->H * d->d_v;
    float* lse_out = lse ? lse + (size_t)t0 * d->H : nullptr;
    if (launch_dependent(few_value_kernel, dim3(d->H, (n + kFvTokens - 1) / kFvTokens),
                         dim3(kFvThreads), (int)few_value_smem(pairs), st, true, n, d->H, d->d_v, pairs,
                         static_cast<const fw::Plan*>(plan), static_cast<const fw::Stream*>(streams),
                         static_cast<const FewToken*>(tokens), static_cast<const float*>(p.partial),
                         static_cast<const float*>(p.partial_lse), wv, out, lse_out) != cudaSuccess)
      return MLA_ERR_CUDA;
  }
  return MLA_OK;
}

}  // namespace

int chunk_take_status() { return take_module_status(); }

}  // namespace mla

using namespace mla;

extern "C" size_t mla_chunk_workspace_size(const mla_dims_t* dims, int32_t B, int32_t n_tok,
                                           int32_t n_ver, int32_t max_pages, int32_t max_segs,
                                           int64_t max_rows) {
  if (!chunk_dims_ok(dims) || B < 1 || n_tok < 1 || n_ver < 1 || n_ver > kMaxVersions ||
      max_pages < 1 || max_segs < 1 || max_rows < 0 || max_rows > INT32_MAX)
    return 0;
  Layout l;
  return make_layout(dims, B, n_tok, n_ver, max_pages, max_segs, max_rows, &l) ? l.total : 0;
}

extern "C" mla_status_t mla_chunk_attn(const mla_dims_t* dims, int32_t B, int32_t n_tok,
                                       const void* q, const int32_t* tok_start,
                                       const int32_t* q_pos, const void* w_uk, const void* w_uv,
                                       const void* cache, int64_t n_pages,
                                       const int32_t* block_table, int32_t max_pages,
                                       const mla_seg_t* segs, int32_t max_segs,
                                       const int32_t* delta, int32_t n_ver, int64_t max_rows,
                                       void* v, float* lse, void* workspace, size_t ws_bytes,
                                       mla_stream_t stream) {
  if (!chunk_dims_ok(dims) || B < 0 || n_tok < 0 || n_ver < 1 || !delta || n_pages < 1 ||
      max_pages < 1 || max_segs < 1 || max_rows < 0)
    return MLA_ERR_INVALID_ARG;
  if (dims->page_size != kPage || n_ver > kMaxVersions || n_pages > INT32_MAX / kPage - 2 ||
      (long long)max_pages * kPage > INT32_MAX || max_rows > INT32_MAX)
    return MLA_ERR_UNSUPPORTED;
  if (B == 0 || n_tok == 0) return MLA_OK;
  if (!q || !tok_start || !q_pos || !w_uk || !w_uv || !cache || !block_table || !segs || !v ||
      !ptr_aligned(cache, 256) || !ptr_aligned(q, 16) || !ptr_aligned(w_uk, 16) ||
      !ptr_aligned(w_uv, 16) || !ptr_aligned(v, 16) || !ptr_aligned(lse, 4) ||
      !ptr_aligned(tok_start, 4) || !ptr_aligned(q_pos, 4) || !ptr_aligned(block_table, 4) ||
      !ptr_aligned(segs, 4))
    return MLA_ERR_INVALID_ARG;
  Layout l;
  if (!make_layout(dims, B, n_tok, n_ver, max_pages, max_segs, max_rows, &l))
    return MLA_ERR_UNSUPPORTED;
  if (!workspace || ws_bytes < l.total) return MLA_ERR_WORKSPACE;
  if (!ptr_aligned(workspace, 256)) return MLA_ERR_INVALID_ARG;
  ChunkArgs a;
  a.B = B;
  a.n_tok = n_tok;
  a.H = dims->H;
  a.d_n = dims->d_n;
  a.d_r = dims->d_r;
  a.d_v = dims->d_v;
  a.n_ver = n_ver;
  a.max_pages = max_pages;
  a.max_segs = max_segs;
  a.n_pages = n_pages;
  a.rope_base = dims->rope_base;
  for (int i = 0; i < kMaxVersions; ++i) a.delta[i] = i < n_ver ? delta[i] : 0;
  a.q = q;
  a.tok_start = tok_start;
  a.q_pos = q_pos;
  a.cache = cache;
  a.block_table = block_table;
  a.segs = segs;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (l.expanded) return run_expanded(dims, a, l, ws, w_uk, w_uv, v, lse, st);
  if (!l.generic) return run_absorbed(dims, a, l, ws, w_uk, w_uv, v, lse, st);
  if (dims->dtype == MLA_BF16) return run_generic<__nv_bfloat16>(dims, a, l.cap, w_uk, w_uv, v, lse, st);
  return run_generic<float>(dims, a, l.cap, w_uk, w_uv, v, lse, st);
}
