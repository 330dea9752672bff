// mla_tokens.cu -- the token side of a prompt chunk: rotary positions with
// several axes (mla_rope_axes) and the append of a ragged chunk to the paged
// latent cache (mla_append_tokens).
//
// Rotation (Day 27 tutorial "Multi-Head Latent Attention", section "Position
// Rotations Complicate the Absorption", with one position per axis): the
// d_r / 2 pairs of a vector are cut into n_axes runs of sections[a] pairs; pair
// i of run a turns by pos[a][token] * base^(-2i / d_r), i counted over the
// whole vector, so that equal positions on every axis are the one-axis
// rotation.  Angles are computed in double (a float angle at position 10^6 is
// off by 0.03 rad).
//
// Append: token i of sequence b becomes the cache row of logical row
// row0[b] + i: [c * w / sqrt(mean(c^2) + eps) | R(pos) k] from the raw row
// [c | k] of the down-projection, rounded to the storage type; a low-bit
// pool gets the codes of that rounded row.
//
// Both are bound by memory for long chunks and by the latency of one chain of
// loads for a few tokens.  Rotation of 4099 tokens x 64 heads, as slices of
// 192-wide queries: 14.6 us (67 MB, 4.6 TB/s); of 16 x 128: 2.6 us.  Append with
// RMSNorm of 8192 tokens: 8.1 us (19 MB, 2.3 TB/s); of 64: 4.0 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "mla.h"
#include "common.cuh"

namespace mla {
namespace {

constexpr int kMaxPairs = 64;       // d_r <= 128
constexpr int kMaxAxes = 4;
constexpr int kRopeThreads = 256;
constexpr int kRopeUnroll = 8;      // 16-byte loads a thread has on their way
constexpr int kRopeTokens = 8;      // tokens of a block at most
constexpr int kTokThreads = 256;    // append: a warp per token

// Frequencies of the pairs, and the first pair of each axis' run.
struct Axes {
  int n, half;
  int first[kMaxAxes + 1];
  double theta[kMaxPairs];
  __device__ int axis_of(int pair) const {
    int x = 0;
#pragma unroll
    for (int i = 1; i < kMaxAxes; ++i) x += (i < n && pair >= first[i]) ? 1 : 0;
    return x;
  }
};

bool make_axes(const mla_dims_t* d, int n_axes, const int32_t* sections, Axes* ax) {
  ax->n = n_axes;
  ax->half = d->d_r / 2;
  int sum = 0;
  for (int i = 0; i < n_axes; ++i) {
    ax->first[i] = sum;
    if (sections[i] < 0 || sections[i] > ax->half - sum) return false;
    sum += sections[i];
  }
  for (int i = n_axes; i <= kMaxAxes; ++i) ax->first[i] = sum;
  // base^(-2i / d_r) as powers of one ratio: 128 products in 80-bit arithmetic
  // stay far below half a unit of the double they are rounded to, and cost the
  // host 0.1 us where as many calls of pow take 2 us of a 4 us launch
  const long double ratio = powl((long double)d->rope_base, -2.0L / d->d_r);
  long double th = 1.0L;
  for (int i = 0; i < ax->half; ++i, th *= ratio) ax->theta[i] = (double)th;
  return sum == ax->half;
}

// Eight consecutive elements, in 16-byte pieces, and as floats.
struct alignas(16) Raw8f {
  float4 lo, hi;
};
template <typename T> struct RawGroup;
template <> struct RawGroup<__nv_bfloat16> { using type = uint4; };
template <> struct RawGroup<float> { using type = Raw8f; };
__device__ __forceinline__ void open_group(const uint4& u, float (&v)[8]) {
  v[0] = lo_f(u.x); v[1] = hi_f(u.x); v[2] = lo_f(u.y); v[3] = hi_f(u.y);
  v[4] = lo_f(u.z); v[5] = hi_f(u.z); v[6] = lo_f(u.w); v[7] = hi_f(u.w);
}
__device__ __forceinline__ void open_group(const Raw8f& u, float (&v)[8]) {
  v[0] = u.lo.x; v[1] = u.lo.y; v[2] = u.lo.z; v[3] = u.lo.w;
  v[4] = u.hi.x; v[5] = u.hi.y; v[6] = u.hi.z; v[7] = u.hi.w;
}
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  open_group(*reinterpret_cast<const typename RawGroup<T>::type*>(p), v);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// Cosine and sine of pos * theta.  kExact: in double throughout.  Otherwise the
// angle is reduced to a fraction of a turn in double and the functions are
// float, off by at most 2^-22 each: far below a rounding to bf16, and a short
// chain where the double functions take 1 to 2 us, most of a small call.
template <bool kExact>
__device__ __forceinline__ void trig(double angle, double& c, double& s) {
  sincos(angle, &s, &c);
}
template <>
__device__ __forceinline__ void trig<false>(double angle, double& c, double& s) {
  const double turns = angle * 0.15915494309189535;      // 1 / (2 pi)
  float fs, fc;
  sincospif((float)(2.0 * (turns - rint(turns))), &fs, &fc);
  c = fc;
  s = fs;
}

// The turned pair, in double (fp32 rows, rounded once) or in float.
template <typename T> struct Trig;
template <> struct Trig<float> { using type = double2; };
template <> struct Trig<__nv_bfloat16> { using type = float2; };
__device__ __forceinline__ void turn(double2 cs, float x0, float x1, float& y0, float& y1) {
  y0 = (float)((double)x0 * cs.x - (double)x1 * cs.y);
  y1 = (float)((double)x0 * cs.y + (double)x1 * cs.x);
}
__device__ __forceinline__ void turn(float2 cs, float x0, float x1, float& y0, float& y1) {
  y0 = x0 * cs.x - x1 * cs.y;
  y1 = x0 * cs.y + x1 * cs.x;
}

// ---------------------------------------------------------------------------
struct RopeArgs {
  int n_tok, n_heads, heads_per_block, tok_per_block;
  int inverse;
  long long x_tok, x_head, o_tok, o_head;   // strides in elements
  const int32_t* pos;                       // [n_axes, n_tok]
  const void* x;
  void* out;
};

// grid (token blocks, head blocks).  A block computes the sines and cosines of
// its tokens once, in shared memory, while the vectors they turn are on their
// way: a thread issues its loads before it waits for the table.  kVec:
// 16-byte accesses (d_r, strides and pointers are multiples of eight elements).
template <typename T, bool kVec>
__global__ void __launch_bounds__(kRopeThreads) rope_axes_kernel(const __grid_constant__ RopeArgs a,
                                                                 const __grid_constant__ Axes ax) {
  using CS = typename Trig<T>::type;
  __shared__ CS cs[kRopeTokens * kMaxPairs];
  const int t0 = blockIdx.x * a.tok_per_block, nt = min(a.tok_per_block, a.n_tok - t0);
  const int h0 = blockIdx.y * a.heads_per_block, nh = min(a.heads_per_block, a.n_heads - h0);
  const T* x = static_cast<const T*>(a.x) + (long long)t0 * a.x_tok + (long long)h0 * a.x_head;
  T* out = static_cast<T*>(a.out) + (long long)t0 * a.o_tok + (long long)h0 * a.o_head;
  const int per = kVec ? ax.half / 4 : ax.half;      // work items of a head
  const int n = nt * nh * per;
  auto table = [&] {
    for (int i = threadIdx.x; i < nt * ax.half; i += kRopeThreads) {
      const int t = i / ax.half, p = i % ax.half;
      double sn, c;
      trig<sizeof(T) == 4>((double)a.pos[(size_t)ax.axis_of(p) * a.n_tok + t0 + t] * ax.theta[p], c, sn);
      if (a.inverse) sn = -sn;
      cs[i].x = c;
      cs[i].y = sn;
    }
    __syncthreads();
  };
  // A thread's items are `step` apart; their token, head and pair advance by
  // constant amounts with a carry, so that the divisions happen once.
  int p = threadIdx.x % per, h = threadIdx.x / per % nh, t = threadIdx.x / per / nh;
  const int dp = kRopeThreads % per, dh = kRopeThreads / per % nh, dt = kRopeThreads / per / nh;
  auto advance = [&] {
    p += dp;
    h += dh;
    t += dt;
    if (p >= per) {
      p -= per;
      ++h;
    }
    if (h >= nh) {
      h -= nh;
      ++t;
    }
  };
  if constexpr (kVec) {
    using Raw = typename RawGroup<T>::type;
    for (int base = threadIdx.x; base < n || base == threadIdx.x; base += kRopeThreads * kRopeUnroll) {
      Raw raw[kRopeUnroll];
      const int p0 = p, h0_ = h, t0_ = t;
#pragma unroll
      for (int u = 0; u < kRopeUnroll; ++u) {
        if (base + u * kRopeThreads < n)
          raw[u] = *reinterpret_cast<const Raw*>(x + t * a.x_tok + h * a.x_head + p * 8);
        advance();
      }
      if (base == threadIdx.x) table();
      p = p0;
      h = h0_;
      t = t0_;
#pragma unroll
      for (int u = 0; u < kRopeUnroll; ++u) {
        if (base + u * kRopeThreads < n) {
          const CS* c = cs + t * ax.half + p * 4;
          float v[8], y[8];
          open_group(raw[u], v);
#pragma unroll
          for (int j = 0; j < 4; ++j) turn(c[j], v[2 * j], v[2 * j + 1], y[2 * j], y[2 * j + 1]);
          store8(out + t * a.o_tok + h * a.o_head + p * 8, y);
        }
        advance();
      }
    }
  } else {
    table();
    for (int i = threadIdx.x; i < n; i += kRopeThreads, advance()) {
      const T* src = x + t * a.x_tok + h * a.x_head + 2 * p;
      T* d = out + t * a.o_tok + h * a.o_head + 2 * p;
      float y0, y1;
      turn(cs[t * ax.half + p], to_f(src[0]), to_f(src[1]), y0, y1);
      d[0] = from_f<T>(y0);
      d[1] = from_f<T>(y1);
    }
  }
}

// ---------------------------------------------------------------------------
struct AppendTokArgs {
  int B, n_tok, d_c, d_r, max_pages, bits_c;   // bits_c 0: rows of the storage type
  long long n_pages, kv_stride;
  const void* kv;
  const int32_t* tok_start;   // [B + 1]
  const int32_t* row0;        // [B]
  const int32_t* pos;         // [n_axes, n_tok]
  const float* norm_w;        // [d_c] or null
  float eps;
  const float* scale_c;
  const float* scale_r;
  void* cache;
  const int32_t* block_table;
};

// The sequence that token t belongs to, by the whole warp: the number of
// starts at or before t, less one (the loads of a batch of 32 sequences are
// independent of one another, where a binary search chains them).  -1: the
// token lies behind the last sequence; -2: it is left out because starts are not in
// order.  A range that does not hold (0 <= start <= end <= n_tok) or starts before an
// earlier start owns nothing, as in mla_chunk_attn.
__device__ __noinline__ int owner_out_of_order(const int32_t* tok_start, int B, int n_tok, int t,
                                               int lane) {
  int latest = INT32_MIN;
  bool behind = true;
  for (int j = 0; j < B; j += 32) {
    const int b = min(j + lane, B - 1), from = tok_start[b], to = tok_start[b + 1];
    const unsigned in = __ballot_sync(0xffffffffu, j + lane < B && from >= 0 && from <= t && t < to &&
                                                       to <= n_tok);
    behind = behind && from <= t;
    // the first range with t in it: a later one would start inside of it
    const int k = in ? __ffs(in) - 1 : 32;
    latest = max(latest, __reduce_max_sync(0xffffffffu, lane < k ? from : INT32_MIN));
    if (in) return __shfl_sync(0xffffffffu, from, k) >= latest ? j + k : -2;
  }
  return __all_sync(0xffffffffu, behind && tok_start[B] <= t) ? -1 : -2;
}

__device__ __forceinline__ int owner_of(const int32_t* tok_start, int B, int n_tok, int t, int lane) {
  int n = 0, last = INT32_MIN;
  bool ordered = true;
  for (int j = 0; j <= B; j += 32) {
    const int from = tok_start[min(j + lane, B)];
    const unsigned in = __ballot_sync(0xffffffffu, j + lane <= B && from <= t);
    // the starts at or before t come first
    ordered = ordered && (in & (in + 1u)) == 0u && (in == 0u || n == j);
    n += __popc(in);
    if (from <= t) last = max(last, from);
  }
  if (n == 0 && ordered) return -2;
  if (ordered && __reduce_max_sync(0xffffffffu, last) == tok_start[n - 1]) {
    if (n == B + 1) return -1;
    if (tok_start[n - 1] >= 0 && tok_start[n] <= n_tok) return n - 1;
  }
  return owner_out_of_order(tok_start, B, n_tok, t, lane);
}

template <typename T>
__device__ __forceinline__ void load_group(const T* p, bool vec, int n, float (&v)[8]) {
  if (vec) {
    load8(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? to_f(p[j]) : 0.f;
  }
}

__device__ __forceinline__ uint32_t code_of(float x, float scale, int bits) {
  const int lo = -(1 << (bits - 1)), hi = (1 << (bits - 1)) - 1;
  return (uint32_t)min(hi, max(lo, (int)rintf(x / scale))) & ((1u << bits) - 1u);
}

// A warp per token; lane l holds the latent groups of eight channels l, l + 32,
// ... (kHeld of them in registers, which covers 512 channels; wider rows are
// read again) and the rotary pairs l, l + 32, ...  The token's row, its norm
// weights and its first rotary pair are on their way before the owner search,
// whose loads (starts, then row0 and the page id) form a chain of their own.
// kLow: a packed pool.  What decides a code is computed in double, since one
// rounding of a value next to the border of two codes moves it by a whole step;
// rows of the storage type use float.
constexpr int kHeld = 2;

template <typename T, bool kLow>
__global__ void __launch_bounds__(kTokThreads) append_tokens_kernel(
    const __grid_constant__ AppendTokArgs a, const __grid_constant__ Axes ax) {
  using A = typename std::conditional<kLow, double, float>::type;
  constexpr bool kExact = kLow || sizeof(T) == 4;
  const long long gw = (long long)blockIdx.x * (kTokThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (gw >= a.n_tok) return;
  const int t = (int)gw;
  const T* src = static_cast<const T*>(a.kv) + (long long)t * a.kv_stride;
  const int groups = (a.d_c + 7) / 8;
  const bool vec_in = a.d_c % 8 == 0 && (reinterpret_cast<uintptr_t>(src) & 15) == 0;
  const bool vec_w = a.norm_w && a.d_c % 8 == 0 && (reinterpret_cast<uintptr_t>(a.norm_w) & 15) == 0;
  float v[kHeld][8], w[kHeld][8];
#pragma unroll
  for (int u = 0; u < kHeld; ++u) {
    const int g = lane + 32 * u;
    if (g >= groups) break;
    load_group(src + 8 * g, vec_in, a.d_c - 8 * g, v[u]);
    if (a.norm_w) load_group(a.norm_w + 8 * g, vec_w, a.d_c - 8 * g, w[u]);
  }
  const T* key = src + a.d_c;
  const bool has_pair = lane < ax.half;
  const float k0 = has_pair ? to_f(key[2 * lane]) : 0.f, k1 = has_pair ? to_f(key[2 * lane + 1]) : 0.f;
  double2 cs = make_double2(1.0, 0.0);
  if (has_pair)
    trig<kExact>((double)a.pos[(size_t)ax.axis_of(lane) * a.n_tok + t] * ax.theta[lane], cs.x, cs.y);

  const int b = owner_of(a.tok_start, a.B, a.n_tok, t, lane);
  if (t == 0)        // for all tokens: a range that does not hold
    for (int j = lane; j < a.B; j += 32) {
      const int from = a.tok_start[j], to = a.tok_start[j + 1];
      if (from < 0 || to < from || to > a.n_tok) set_status(MLA_ERR_BAD_INDEX);
    }
  if (b == -1) return;
  int page = -1, slot = 0;
  if (b >= 0) {
    const long long r = (long long)a.row0[b] + (t - a.tok_start[b]);
    if (r >= 0 && r / kPage < a.max_pages) {
      page = a.block_table[(size_t)b * a.max_pages + r / kPage];
      slot = (int)(r % kPage);
    }
  }
  if (page < 0 || page >= a.n_pages) {
    if (lane == 0) set_status(MLA_ERR_BAD_INDEX);
    return;
  }

  A inv = (A)1;
  if (a.norm_w) {
    A ss = (A)0;
#pragma unroll
    for (int u = 0; u < kHeld; ++u)
      if (lane + 32 * u < groups) {
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += (A)v[u][j] * (A)v[u][j];
      }
    for (int g = lane + 32 * kHeld; g < groups; g += 32) {
      float x[8];
      load_group(src + 8 * g, vec_in, a.d_c - 8 * g, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += (A)x[j] * (A)x[j];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    inv = (A)1 / sqrt(ss / (A)a.d_c + (A)a.eps);
  }
  const size_t row = (size_t)page * kPage + slot;
  const size_t row_bytes = kLow ? (size_t)(a.d_c * a.bits_c + a.d_r * 4) / 8
                                : ((size_t)a.d_c + a.d_r) * sizeof(T);
  uint8_t* dst = static_cast<uint8_t*>(a.cache) + row * row_bytes;
  T* dst_t = reinterpret_cast<T*>(dst);
  const bool vec_out = a.d_c % 8 == 0 && (reinterpret_cast<uintptr_t>(dst) & 15) == 0;
  auto store_group = [&](int g, float (&x)[8], const float (&wt)[8]) {
    const int n = min(8, a.d_c - 8 * g);
    if (a.norm_w) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = (float)((A)x[j] * inv * (A)wt[j]);
    }
    if constexpr (!kLow) {
      if (vec_out) {
        store8(dst_t + 8 * g, x);
      } else {
        for (int j = 0; j < n; ++j) dst_t[8 * g + j] = from_f<T>(x[j]);
      }
    } else {
      uint32_t word = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        word |= code_of(to_f(from_f<T>(x[j])), a.scale_c[8 * g + j], a.bits_c) << (a.bits_c * j);
      if (a.bits_c == 4) reinterpret_cast<uint32_t*>(dst)[g] = word;
      else reinterpret_cast<uint16_t*>(dst)[g] = (uint16_t)word;
    }
  };
#pragma unroll
  for (int u = 0; u < kHeld; ++u)
    if (lane + 32 * u < groups) store_group(lane + 32 * u, v[u], w[u]);
  for (int g = lane + 32 * kHeld; g < groups; g += 32) {
    float x[8], wt[8] = {};
    load_group(src + 8 * g, vec_in, a.d_c - 8 * g, x);
    if (a.norm_w) load_group(a.norm_w + 8 * g, vec_w, a.d_c - 8 * g, wt);
    store_group(g, x, wt);
  }
  for (int i = lane; i < ax.half; i += 32) {
    float x0 = k0, x1 = k1, y0, y1;
    if (i != lane) {
      x0 = to_f(key[2 * i]);
      x1 = to_f(key[2 * i + 1]);
      trig<kExact>((double)a.pos[(size_t)ax.axis_of(i) * a.n_tok + t] * ax.theta[i], cs.x, cs.y);
    }
    turn(cs, x0, x1, y0, y1);
    if constexpr (!kLow) {
      dst_t[a.d_c + 2 * i] = from_f<T>(y0);
      dst_t[a.d_c + 2 * i + 1] = from_f<T>(y1);
    } else {
      dst[a.d_c * a.bits_c / 8 + i] =
          (uint8_t)(code_of(to_f(from_f<T>(y0)), a.scale_r[2 * i], 4) |
                    code_of(to_f(from_f<T>(y1)), a.scale_r[2 * i + 1], 4) << 4);
    }
  }
}

bool aligned_to(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

bool rotary_dims_ok(const mla_dims_t* d) {
  return d && d->d_r > 0 && d->d_r % 2 == 0 && d->rope_base > 0.0 &&
         (d->dtype == MLA_F32 || d->dtype == MLA_BF16);
}

}  // namespace

// Reads and clears this module's status word (mla_get_status calls it after
// synchronising the stream).
int tokens_take_status() { return take_module_status(); }

}  // namespace mla

using namespace mla;

extern "C" mla_status_t mla_rope_axes(const mla_dims_t* dims, int32_t n_tok, int32_t n_heads,
                                      const void* x, int64_t x_tok_stride, int64_t x_head_stride,
                                      const int32_t* pos, int32_t n_axes, const int32_t* sections,
                                      int32_t inverse, void* out, int64_t out_tok_stride,
                                      int64_t out_head_stride, mla_stream_t stream) {
  if (!rotary_dims_ok(dims) || n_tok < 0 || n_heads < 1 || n_axes < 1 || !sections ||
      (inverse != 0 && inverse != 1))
    return MLA_ERR_INVALID_ARG;
  if (n_axes > kMaxAxes || dims->d_r > 2 * kMaxPairs) return MLA_ERR_UNSUPPORTED;
  Axes ax;
  if (!make_axes(dims, n_axes, sections, &ax)) return MLA_ERR_INVALID_ARG;
  if (n_tok == 0) return MLA_OK;
  const size_t es = dims->dtype == MLA_BF16 ? 2 : 4;
  if (!x || !pos || !out || !aligned_to(x, es) || !aligned_to(out, es) || !aligned_to(pos, 4))
    return MLA_ERR_INVALID_ARG;
  // vectors of one tensor must not overlap: a head's d_r elements lie within
  // its stride, or a token's heads are the outer axis
  const int64_t d_r = dims->d_r;
  auto apart = [&](int64_t tok, int64_t head) {
    return (head >= d_r && (n_tok == 1 || tok >= head * (n_heads - 1) + d_r)) ||
           (tok >= d_r && (n_heads == 1 || head >= tok * (n_tok - 1) + d_r));
  };
  if (x_tok_stride < 0 || x_head_stride < 0 ||
      (!apart(out_tok_stride, out_head_stride) && (n_tok > 1 || n_heads > 1)))
    return MLA_ERR_INVALID_ARG;
  // in place: the same vectors, or one thread's results are another one's input
  if (x == out && ((n_tok > 1 && x_tok_stride != out_tok_stride) ||
                   (n_heads > 1 && x_head_stride != out_head_stride)))
    return MLA_ERR_INVALID_ARG;
  RopeArgs a;
  a.n_tok = n_tok;
  a.n_heads = n_heads;
  a.inverse = inverse;
  a.x_tok = x_tok_stride;
  a.x_head = x_head_stride;
  a.o_tok = out_tok_stride;
  a.o_head = out_head_stride;
  a.pos = pos;
  a.x = x;
  a.out = out;
  const bool vec = dims->d_r % 8 == 0 && aligned_to(x, 16) && aligned_to(out, 16) &&
                   x_tok_stride % 8 == 0 && x_head_stride % 8 == 0 && out_tok_stride % 8 == 0 &&
                   out_head_stride % 8 == 0;
  const int per = vec ? ax.half / 4 : ax.half;
  // One batch of loads a thread: as many tokens as fill it, heads split when
  // one token holds more.  Few tokens: one load a thread, so that the heads
  // of a token spread over several SMs.  Slices of 192-wide queries, few and many
  // loads a thread (us): 8 heads 64 tokens 2.6, 3.0; 256 3.1, 3.1; 512 5.0, 3.1;
  // 64 heads 64 2.9, 3.6; 128 3.4, 3.6; 256 5.3, 3.7; 512 8.9, 3.7; 128 heads 64 3.3, 3.7;
  // 128 5.3, 3.7; 512 14.9, 4.8.  So the sides cross at about 8192 (token, head) pairs,
  // and 512 tokens is late for many heads.
  const int items = kRopeThreads * (n_tok >= 512 ? kRopeUnroll : 1);
  int hpb = items / per > 0 ? items / per : 1, tpb = 1;
  if (hpb > n_heads) hpb = n_heads;
  if ((n_heads + hpb - 1) / hpb > 65535) hpb = (n_heads + 65534) / 65535;
  if (hpb == n_heads && n_tok >= 512) {
    tpb = items / (per * n_heads);
    if (tpb < 1) tpb = 1;
    if (tpb > kRopeTokens) tpb = kRopeTokens;
  }
  a.heads_per_block = hpb;
  a.tok_per_block = tpb;
  const dim3 grid((n_tok + tpb - 1) / tpb, (n_heads + hpb - 1) / hpb);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dims->dtype == MLA_BF16) {
    if (vec) rope_axes_kernel<__nv_bfloat16, true><<<grid, kRopeThreads, 0, st>>>(a, ax);
    else rope_axes_kernel<__nv_bfloat16, false><<<grid, kRopeThreads, 0, st>>>(a, ax);
  } else {
    if (vec) rope_axes_kernel<float, true><<<grid, kRopeThreads, 0, st>>>(a, ax);
    else rope_axes_kernel<float, false><<<grid, kRopeThreads, 0, st>>>(a, ax);
  }
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

extern "C" mla_status_t mla_append_tokens(const mla_dims_t* dims, int32_t B, int32_t n_tok,
                                          const void* kv, int64_t kv_stride,
                                          const int32_t* tok_start, const int32_t* row0,
                                          const int32_t* pos, int32_t n_axes,
                                          const int32_t* sections, const float* norm_weight,
                                          float norm_eps, int32_t bits_c, int32_t bits_r,
                                          const float* scale_c, const float* scale_r, void* cache,
                                          int64_t n_pages, const int32_t* block_table,
                                          int32_t max_pages, mla_stream_t stream) {
  if (!rotary_dims_ok(dims) || dims->d_c < 1 || B < 0 || n_tok < 0 || n_axes < 1 || !sections ||
      n_pages < 1 || max_pages < 1 || kv_stride < (int64_t)dims->d_c + dims->d_r)
    return MLA_ERR_INVALID_ARG;
  if (norm_weight && !(norm_eps >= 0.f)) return MLA_ERR_INVALID_ARG;
  if (dims->page_size != kPage || n_axes > kMaxAxes || dims->d_r > 2 * kMaxPairs)
    return MLA_ERR_UNSUPPORTED;
  const bool low = bits_c != 0 || bits_r != 0;
  if (low && (!((bits_c == 4 || bits_c == 2) && bits_r == 4) || dims->d_c % (32 / bits_c) != 0 ||
              dims->d_r % 8 != 0 || dims->d_c > INT32_MAX / 8))
    return MLA_ERR_UNSUPPORTED;
  if (low != (scale_c != nullptr) || low != (scale_r != nullptr)) return MLA_ERR_INVALID_ARG;
  Axes ax;
  if (!make_axes(dims, n_axes, sections, &ax)) return MLA_ERR_INVALID_ARG;
  if (n_tok == 0 || B == 0) return MLA_OK;
  const size_t es = dims->dtype == MLA_BF16 ? 2 : 4;
  if (!kv || !tok_start || !row0 || !pos || !cache || !block_table || !aligned_to(kv, es) ||
      !aligned_to(cache, low ? 4 : es) || !aligned_to(tok_start, 4) || !aligned_to(row0, 4) ||
      !aligned_to(pos, 4) || !aligned_to(block_table, 4) || !aligned_to(norm_weight, 4) ||
      !aligned_to(scale_c, 4) || !aligned_to(scale_r, 4))
    return MLA_ERR_INVALID_ARG;
  AppendTokArgs a;
  a.B = B;
  a.n_tok = n_tok;
  a.d_c = dims->d_c;
  a.d_r = dims->d_r;
  a.max_pages = max_pages;
  a.bits_c = bits_c;
  a.n_pages = n_pages;
  a.kv_stride = kv_stride;
  a.kv = kv;
  a.tok_start = tok_start;
  a.row0 = row0;
  a.pos = pos;
  a.norm_w = norm_weight;
  a.eps = norm_eps;
  a.scale_c = scale_c;
  a.scale_r = scale_r;
  a.cache = cache;
  a.block_table = block_table;
  const unsigned blocks = (unsigned)(((long long)n_tok * 32 + kTokThreads - 1) / kTokThreads);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dims->dtype == MLA_BF16) {
    if (low) append_tokens_kernel<__nv_bfloat16, true><<<blocks, kTokThreads, 0, st>>>(a, ax);
    else append_tokens_kernel<__nv_bfloat16, false><<<blocks, kTokThreads, 0, st>>>(a, ax);
  } else {
    if (low) append_tokens_kernel<float, true><<<blocks, kTokThreads, 0, st>>>(a, ax);
    else append_tokens_kernel<float, false><<<blocks, kTokThreads, 0, st>>>(a, ax);
  }
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
