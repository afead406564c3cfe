// What the kernels of the 8-bit floating point products share: the parameters of a launch, the
// table of buckets, wrappers of single instructions, and the tensor maps.  Included by those
// kernels' files only.
#pragma once

#include <cuda_fp8.h>

#include "moe_fp8.h"

namespace moe {

struct Fp8Params {
  const int32_t* seg_start;  // [E] first row of each bucket
  const int32_t* seg_count;  // [E] rows of each bucket
  int E;
  int64_t rows;        // rows of a, a_scale and the outputs (at most kFp8MaxRows)
  int K;               // reduction length (a multiple of 16)
  int N;               // output columns (LINEAR a multiple of 8, GATED of 16)
  int n_blocks;        // tiles along the output columns
  int kb;              // ceil(K / 128)
  int nsb;             // rows of a weight's scales: ceil(N / 128)
  const float* a_scale;   // [rows, kb]
  const float* w_scale0;  // [E, nsb, kb] of the weight (LINEAR) or of W_gate
  const float* w_scale1;  // [E, nsb, kb] of W_up
  __nv_bfloat16* out;     // LINEAR: [rows, N]
  uint8_t* h;             // GATED: [rows, N] e4m3
  float* h_scale;         // GATED: [rows, nsb]
  unsigned int* arrivals; // pieces of a cut tile that are done (0 between launches)
  float* partials;        // 2 slots a CTA, see the kernels
  DevStatus* status;
  uint64_t wait_ns;
  bool follows;  // see Fp8Gemm
};

// The kernel for buckets of few rows (moe_fp8_few.cu).
cudaError_t launch_fp8_few_rows(const Fp8Gemm& g, const Fp8Params& p, cudaStream_t st,
                                const char** why);

namespace {

constexpr int BK = 128;      // bytes = e4m3 values of a stage's rows: one block of the scales
constexpr int BN = 256;      // weight rows of a tile
constexpr int HALF_N = BN / 2;
constexpr int STAGES = 4;
constexpr int B_BYTES = BN * BK;
// Limit of the waits for a block's own copies and MMAs before it exits, whatever the limit of
// the others is: these end by themselves within microseconds.
constexpr uint64_t kDrainNs = 1000000000ull;

enum Mode { FP8_LINEAR = 0, FP8_GATED = 1 };

constexpr int SLOT_FLOATS = 64 * BN;  // partial sums of a piece

// Programmatic dependent launch: let the next launch's blocks start as this one's leave their
// SMs.
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// 32 lanes x 16 columns of tensor memory, on their way until tmem_ld_wait().
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// One arrival by the threads whose `who` is not 0, without a branch.
__device__ __forceinline__ void arrive_if(uint64_t* bar, uint32_t who) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_addr(bar)),
      "r"(who)
      : "memory");
}

// 4 scales from block kb on (0 past the last of n).
__device__ __forceinline__ float4 scales4(const float* s, int kb, int n) {
  if ((n & 3) == 0)
    return kb < n ? *reinterpret_cast<const float4*>(s + kb) : make_float4(0.f, 0.f, 0.f, 0.f);
  return make_float4(kb < n ? s[kb] : 0.f, kb + 1 < n ? s[kb + 1] : 0.f,
                     kb + 2 < n ? s[kb + 2] : 0.f, kb + 3 < n ? s[kb + 3] : 0.f);
}
__device__ __forceinline__ float pick(const float4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void tc_mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::f8f6f4 with e4m3 A/B, fp32 D, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4)                                // D format: f32 (A and B format 0: e4m3)
         | (static_cast<uint32_t>(N >> 3) << 17)  // N / 8
         | (static_cast<uint32_t>(M >> 4) << 24); // M / 16
}

// silu(g) u.  (The fast division gives 0 for a divisor above 2^126, which a gate below -87.3 has:
// |silu| is below 2^-119 there.)
__device__ __forceinline__ float silu_mul(float g, float u) {
  return __fdividef(g, 1.0f + __expf(-g)) * u;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// How a block of h is quantised, from its largest magnitude's bits: h times fp32(448 / m), rounded
// to fp32 and then to e4m3.  (h is off by more than these roundings are: of 512 x 2048 entries they
// alone moved one code, the sums of h seven.)
struct RowQuant {
  float m, r;
  bool bad;  // an infinity or a NaN in the block: NaN in all of it
  __device__ __forceinline__ explicit RowQuant(uint32_t bits) {
    bad = bits >= 0x7F800000u;
    m = fmaxf(__uint_as_float(bits), 7.8886090522101181e-31f);  // 2^-100
    r = __fdiv_rn(448.0f, m);
  }
  __device__ __forceinline__ uint32_t pack(float a, float b, float c, float d) const {
    return bad ? 0x7F7F7F7Fu : e4m3x4(a * r, b * r, c * r, d * r);
  }
  __device__ __forceinline__ float scale() const {
    return bad ? __uint_as_float(0x7FFFFFFFu) : __fdiv_rn(m, 448.0f);
  }
};

// The bucket table of a launch in shared memory.
struct Buckets {
  int start[MOE_MAX_EXPERTS];
  int count[MOE_MAX_EXPERTS];
  int tile_base[MOE_MAX_EXPERTS + 1];  // first tile of each bucket
};

// By one whole warp: every bucket cut to the rows there are, and the tiles before each.
template <int ROWS>  // of a tile
__device__ void build_buckets(Buckets& t, const Fp8Params& p, int lane) {
  int64_t carry = 0;
  for (int e0 = 0; e0 < p.E; e0 += 32) {
    const int e = e0 + lane;
    int mb = 0;
    if (e < p.E) {
      const int s = p.seg_start[e];
      int c = p.seg_count[e];
      if (c < 0 || (c > 0 && (s < 0 || static_cast<int64_t>(s) + c > p.rows))) {
        if (blockIdx.x == 0)
          record_error(p.status, DEV_BAD_BUCKET, 40, static_cast<unsigned long long>(e));
        c = 0;
      }
      t.start[e] = s;
      t.count[e] = c;  // (at most kFp8MaxRows: the next sum fits)
      mb = (c + ROWS - 1) / ROWS;
    }
    int v = mb;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, v, off);
      if (lane >= off) v += o;
    }
    if (e < p.E) t.tile_base[e] = static_cast<int>(carry + v - mb) * p.n_blocks;
    carry += __shfl_sync(0xffffffffu, v, 31);
  }
  // (only buckets that overlap can have more tiles than an int counts: then none is taken)
  const bool fits = carry * p.n_blocks <= kFp8MaxTiles;
  if (!fits && blockIdx.x == 0)
    record_error(p.status, DEV_BAD_BUCKET, 40, static_cast<unsigned long long>(p.E - 1));
  if (lane == 0) t.tile_base[p.E] = fits ? static_cast<int>(carry) * p.n_blocks : 0;
}

struct Tile {
  int e, nb, row0, valid;  // expert, column block, first row, rows from there in the bucket
};

template <int ROWS>
__device__ __forceinline__ Tile decode(const Buckets& t, const Fp8Params& p, int tile) {
  int lo = 0, hi = p.E - 1;  // largest e with tile_base[e] <= tile
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.tile_base[mid] <= tile) lo = mid;
    else hi = mid - 1;
  }
  const int mbs = (t.count[lo] + ROWS - 1) / ROWS;
  const int local = tile - t.tile_base[lo];
  Tile r;
  r.e = lo;
  r.nb = local / mbs;
  const int mb = local - r.nb * mbs;
  r.row0 = t.start[lo] + mb * ROWS;
  r.valid = t.count[lo] - mb * ROWS;
  return r;
}

// ------------------------------------------------------------------ tensor maps
inline bool encode(CUtensorMap* m, int rank, const void* base, const cuuint64_t* dims,
                   const cuuint64_t* strides, const cuuint32_t* box) {
  const cuuint32_t estr[3] = {1, 1, 1};
  return tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, static_cast<cuuint32_t>(rank),
                              const_cast<void*>(base), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [rows, K] bytes, boxes of box_rows x 128
inline bool map_rows(CUtensorMap* m, const void* base, int64_t rows, int64_t K, uint32_t box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
  const cuuint32_t box[2] = {BK, box_rows};
  return encode(m, 2, base, dims, strides, box);
}

// [E, N, K] bytes, boxes of 1 x box_n x 128
inline bool map_weights(CUtensorMap* m, const void* base, int64_t E, int64_t N, int64_t K,
                        uint32_t box_n) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(N),
                              static_cast<cuuint64_t>(E)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(N * K)};
  const cuuint32_t box[3] = {BK, box_n, 1};
  return encode(m, 3, base, dims, strides, box);
}

// One launch of at most one block per SM and `most` blocks.
template <typename... Params, typename... Args>
cudaError_t launch_product(void (*kernel)(Params...), int64_t most, int threads, int smem,
                           cudaStream_t st, const Args&... args) {
  cudaError_t err = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  return launch_overlapping(kernel, most < sm_count() ? most : sm_count(), threads, smem, st,
                            args...);
}

}  // namespace
}  // namespace moe
