// host_tma.cuh -- host helpers shared by the ABI's translation units: the
// tensor-map encoder and the per-device properties a launch needs.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

namespace mla {

static inline bool ptr_aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// cuTensorMapEncodeTiled, fetched from the driver at run time so that the
// library loads on machines without a driver.
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static inline EncodeTiledFn encode_tiled() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// bf16 tensor map with 128-byte swizzle; strides in bytes for axes 1 ..
// rank - 1.  Elements outside the extents read as zeros.
static inline bool map_bf16(CUtensorMap* m, const void* base, int rank, const uint64_t* extent,
                            const uint64_t* stride, const uint32_t* box) {
  EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  cuuint64_t d[4], s[3];
  cuuint32_t b[4], e[4] = {1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = extent[i];
    b[i] = box[i];
    if (i) s[i - 1] = stride[i - 1];
  }
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), d, s, b,
            e, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A row-major [rows, cols] bf16 matrix, `pitch` elements between rows, in
// boxes of 64 columns x box_rows.
static inline bool map_rows(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows,
                            uint64_t pitch, uint32_t box_rows) {
  const uint64_t extent[2] = {cols, rows}, stride[1] = {pitch * 2};
  const uint32_t box[2] = {64, box_rows};
  return map_bf16(m, base, 2, extent, stride, box);
}

// The same matrix as (64-column offset, row, 64-column panel) in boxes of 64 x
// box_rows x panels: a box row is 128 * panels contiguous bytes, which the
// memory serves better than single 128-byte pieces.  cols is a multiple of 64.
static inline bool map_panels(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows,
                              uint64_t pitch, uint32_t box_rows, uint32_t panels) {
  const uint64_t extent[3] = {64, rows, cols / 64}, stride[2] = {pitch * 2, 128};
  const uint32_t box[3] = {64, box_rows, panels};
  return map_bf16(m, base, 3, extent, stride, box);
}

// SMs of the current device; 0 when it cannot be queried.
static inline int current_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return sms;
}

// A launch that may start while the launch before it still runs; its kernel
// waits on the device (griddepcontrol.wait) before it reads that one's results.
template <typename... P, typename... A>
static inline cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, int smem,
                                           cudaStream_t st, bool dependent, A&&... args) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = pdl;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace mla
