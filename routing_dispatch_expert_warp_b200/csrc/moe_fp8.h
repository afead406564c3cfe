// What the 8-bit floating point kernels (moe_fp8_quant.cu, moe_fp8_gemm.cu, moe_fp8_few.cu) and
// their calls (moe_api.cu) share.  It stands apart from moe_internal.h and moe_device.cuh: the
// benchmark's record of the bf16 grouped GEMM's traffic holds for those files' code.
#pragma once

#include "moe_internal.h"

namespace moe {

// A bucket of a product reaches outside its rows (a DevError, see moe_device.cuh).
constexpr unsigned int DEV_BAD_BUCKET = 4;
static_assert(DEV_BAD_BUCKET > DEV_RECV_OVERFLOW, "the status codes are distinct");

// Launchers: see include/moe.h.
cudaError_t launch_fp8_quantize_rows(int dtype, const void* x, int64_t rows_in, int64_t cols,
                                     const int32_t* assign_row, int k, int64_t rows_out,
                                     void* q, float* scale, cudaStream_t st);
cudaError_t launch_fp8_quantize_weights(int dtype, const void* w, int64_t E, int64_t n,
                                        int64_t cols, void* q, float* scale, cudaStream_t st);
// One grouped product: out (w1 == nullptr), or h and h_scale of the gate (w0) and up (w1)
// weights.  Sizes checked by the caller.
struct Fp8Gemm {
  int E;
  int64_t rows, N, K;
  const void* a;            // [rows, K]
  const float* a_scale;     // [rows, ceil(K / 128)]
  const int32_t* seg_start; // [E]
  const int32_t* seg_count; // [E]
  const void* w0;           // [E, N, K]
  const float* w_scale0;    // [E, ceil(N / 128), ceil(K / 128)]
  const void* w1;
  const float* w_scale1;
  void* out;                // [rows, N] bf16
  void* h;                  // [rows, N] e4m3
  float* h_scale;           // [rows, ceil(N / 128)]
  bool follows;             // the launch before in the stream is the product that made a: only
                            // a and a_scale depend on it
};
// Most rows of a product: rounded up to whole tiles of 128 they still fit in an int.
constexpr int64_t kFp8MaxRows = 2147483647LL - 127;
// Most tiles of a product: so does a block's step past the last one.
constexpr int64_t kFp8MaxTiles = 2147483647LL - 65535;
// Workspace of the fp8 products: the status record, then arrival counters (zero between
// calls), then partial sums.
constexpr size_t kFp8CountersOffset = 256;
constexpr size_t kFp8PartialsOffset = 4096;
size_t fp8_workspace_bytes();
cudaError_t launch_fp8_gemm(const Fp8Gemm& g, void* ws, uint64_t wait_ns, cudaStream_t st,
                            const char** why);

// cuTensorMapEncodeTiled of the driver (nullptr: not available).
using TensorMapEncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                       const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                       const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                       CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
TensorMapEncodeFn tensor_map_encoder();

// Programmatic dependent launch: the blocks of a kernel launched by launch_overlapping may start
// while the launch before is ending; here they wait until it has completed and its writes are
// visible (at once when there is nothing to wait for).  It saves 2 us a launch.  Loads of what
// that launch wrote are plain ones: a read-only load (__ldg, or one through a const __restrict__
// pointer) promises that nothing writes there while the kernel runs, and may go ahead of the wait.
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A launch whose blocks may start while the launch before in the stream is ending: each begins
// with wait_for_previous().
template <typename... Params, typename... Args>
cudaError_t launch_overlapping(void (*kernel)(Params...), int64_t blocks, int threads, int smem,
                               cudaStream_t st, const Args&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (err == cudaSuccess) note_launch();
  return err;
}

}  // namespace moe
