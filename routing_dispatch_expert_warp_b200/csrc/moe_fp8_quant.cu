// Quantisation to 8-bit floating point (e4m3) with one fp32 scale for each block of 128:
// rows of activations (a block is 128 columns of a row) and expert weights (a block is
// 128 x 128 entries of a weight).
//
// For a block with largest magnitude m, taken as at least 2^-100 (so that 448 / m is finite):
//   scale = fp32(m / 448),   q = the e4m3 number nearest to 448 x / m, ties to even,
// the quotient taken exactly: the largest entry maps to +-448, the largest e4m3 number.  A
// block that holds an infinity or a NaN gets scale NaN and NaN in every entry.
//
// The exact quotient without a division per entry:
//   bf16 x.  With p = fp32(x fp32(448 / m)), |p / Q - 1| < 2^-22 for the quotient Q = 448 x / m.
//   x and m have 8 significant bits, so Q = 7 X / M times a power of two with integers X, M <
//   256, and a border between two e4m3 numbers is an odd o <= 31 times a power of two.  When Q
//   is not on the border it is at least 1 / (31 x 255) > 2^-13 away from it (7 X 2^i and o M are
//   different integers); so p rounded to 16 fractional bits (an integer add and mask) lies on
//   Q's side of every border, and exactly on the border when Q does, and the conversion then
//   rounds as it would round Q.  (Such borders are common: X / M is often a short fraction.)
//   fp32 x.  With r = fp32(448 / m), x r (1 - 2^-21) and x r (1 + 2^-21), each rounded twice by at
//   most 2^-24, lie on either side of Q.  When both convert to the same number it is Q's.  That
//   holds but for one entry in some 10^5 (more when x has few significant bits and Q hits
//   borders), whose quotient is then taken exactly: c = 448 x by a power of two that brings m to
//   [4, 8), kept as hi + lo; one division step with its remainder gives the fp32 quotient q1 and
//   the sign of Q - q1; when the sign is not 0, q1's last bit is made odd towards it ("round to
//   odd"), so that the conversion sees which side of a border Q is on.  (The exact quotient for
//   every entry: 231 us instead of 190 for 4 x 14336 x 4096 weights.)
//
// These kernels are bound by reading x and writing q: 6.6 TB/s for bf16 weights (4 x 14336 x 4096
// in 106 us), 6.2 for fp32 ones; rows of bf16 5.3 to 5.6 (16384 x 7168 in 66 us, 65536 x 4096 in
// 144), of fp32 6.3 to 6.6 (93 and 202 us).
#include <cuda_fp8.h>

#include "moe_fp8.h"

namespace moe {
namespace {

constexpr uint32_t kAmaxFloorBits = 27u << 23;  // 2^-100
constexpr uint32_t kInfBits = 0x7F800000u;

__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// 16 consecutive entries of a row in registers, as loaded (bf16 pairs or fp32).
template <bool BF16>
struct Piece {
  uint4 v[BF16 ? 2 : 4];
  __device__ __forceinline__ void load(const void* base, int64_t elem) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) +
                                                    elem * (BF16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < (BF16 ? 2 : 4); ++i) v[i] = p[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (BF16 ? 2 : 4); ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ uint32_t word(int i) const {
    const uint4& u = v[i >> 2];
    return (i & 3) == 0 ? u.x : (i & 3) == 1 ? u.y : (i & 3) == 2 ? u.z : u.w;
  }
  __device__ __forceinline__ float value(int i) const {
    if (BF16) {
      const uint32_t w = word(i >> 1);
      return (i & 1) ? bf16_hi(w) : bf16_lo(w);
    }
    return __uint_as_float(word(i));
  }
  // largest magnitude as bits: NaN > infinity > every number
  __device__ __forceinline__ uint32_t amax_bits() const {
    uint32_t m = 0;
    if (BF16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) m = __vmaxu2(m, word(i) & 0x7FFF7FFFu);
      m = max(m & 0xFFFFu, m >> 16) << 16;
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) m = max(m, word(i) & 0x7FFFFFFFu);
    }
    return m;
  }
};

// What the entries of a block are multiplied by, from its largest magnitude.
template <bool BF16>
struct Quant {
  bool bad;
  float scale;  // fp32(m / 448), NaN for a bad block
  float m;
  float r;      // fp32(448 / m)

  __device__ __forceinline__ explicit Quant(uint32_t bits) {
    bad = bits >= kInfBits;
    m = __uint_as_float(bits < kAmaxFloorBits ? kAmaxFloorBits : bits);
    scale = bad ? __uint_as_float(0x7FFFFFFFu) : __fdiv_rn(m, 448.0f);
    r = __fdiv_rn(448.0f, m);
  }
  __device__ __forceinline__ float quotient(float x) const {
    if (BF16) return __uint_as_float((__float_as_uint(x * r) + 0x40u) & 0xFFFFFF80u);
    const float p2 = __uint_as_float((256u - (__float_as_uint(m) >> 23)) << 23);
    const float c = 448.0f * p2, ms = m * p2, rinv = __frcp_rn(ms);
    const float hi = x * c;
    const float lo = fmaf(x, c, -hi);
    const float q0 = hi * rinv;
    const float q1 = fmaf(fmaf(-q0, ms, hi) + lo, rinv, q0);
    const float rem = fmaf(-q1, ms, hi) + lo;
    uint32_t b = __float_as_uint(q1);
    if (rem != 0.0f)  // away from 0 when Q is beyond q1, towards 0 when it is short of it
      b = ((__float_as_uint(rem) ^ b) >> 31 ? b - 1u : b) | 1u;
    // (a quotient that underflowed to 0 may have lost its sign)
    return __uint_as_float((b & 0x7FFFFFFFu) | (__float_as_uint(x) & 0x80000000u));
  }
  __device__ __forceinline__ uint4 convert(const Piece<BF16>& p) const {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = p.value(4 * i), b = p.value(4 * i + 1), c = p.value(4 * i + 2),
                  d = p.value(4 * i + 3);
      bool settled = false;
      if (!BF16) {
        const float r0 = r * (1.0f - 0x1p-21f), r1 = r * (1.0f + 0x1p-21f);
        w[i] = pack_e4m3x4(a * r0, b * r0, c * r0, d * r0);
        settled = w[i] == pack_e4m3x4(a * r1, b * r1, c * r1, d * r1);
      }
      if (!settled) w[i] = pack_e4m3x4(quotient(a), quotient(b), quotient(c), quotient(d));
      if (bad) w[i] = 0x7F7F7F7Fu;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// A warp takes 512 columns of a row, 8 lanes for each of their 4 blocks, 16 entries a lane; of
// rows of one block it takes 4, of rows of two it takes 2 (FOLD = 2, 1; 100000 rows of 16 in bf16:
// 10 us instead of 31).  The registers are held down for the sake of loads in flight: fp32 rows
// of 7168 take 93 us with 5 blocks an SM, 98 with 4.
// With a table of rows (`assign_row`, [rows_in, k]) the row is written to each of its k rows
// inside [0, rows_out); without one to the row of its own index.
template <bool BF16, int FOLD>
__global__ void __launch_bounds__(256, BF16 ? 8 : 5) quantize_rows_kernel(
    const void* x, int64_t rows_in, int cols, int chunks, const int32_t* assign_row, int k,
    int64_t rows_out, uint8_t* q, float* scale) {
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const int64_t items = ((rows_in + (1 << FOLD) - 1) >> FOLD) * chunks;
  const int sub = lane >> 3;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  const int nblocks = (cols + 127) >> 7;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
       item < items; item += warps) {
    const int64_t first = item / chunks;
    const int64_t row = (first << FOLD) + (FOLD == 0 ? 0 : sub >> (2 - FOLD));
    const int col = static_cast<int>(item - first * chunks) * 512 +
                    (sub & ((4 >> FOLD) - 1)) * 128 + (lane & 7) * 16;
    const bool in = (FOLD == 0 || row < rows_in) && col < cols;
    static_assert(MOE_MAX_TOPK <= 8, "a block's 8 lanes hold the row's entries of assign_row");
    int32_t mine = -1;
    if (assign_row != nullptr && (FOLD == 0 || row < rows_in) && (lane & 7) < k)
      mine = assign_row[row * k + (lane & 7)];
    Piece<BF16> p;
    if (in) p.load(x, row * cols + col);
    else p.zero();
    uint32_t m = p.amax_bits();
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
    const Quant<BF16> qt(m);
    const uint4 w = qt.convert(p);
    const int n_out = assign_row != nullptr ? k : 1;
    for (int j = 0; j < n_out; ++j) {
      const int64_t to =
          assign_row != nullptr ? __shfl_sync(0xffffffffu, mine, j, 8) : row;
      if (to < 0 || to >= rows_out || !in) continue;
      *reinterpret_cast<uint4*>(q + to * cols + col) = w;
      if ((lane & 7) == 0) scale[to * nblocks + (col >> 7)] = qt.scale;
    }
  }
}

// One CTA per 128 x 128 block: 8 threads a row, 32 rows at a time, the block kept in
// registers between the two passes over it.
template <bool BF16>
__global__ void __launch_bounds__(256) quantize_weights_kernel(
    const void* w, int64_t n, int64_t cols, int nb, int kb, int64_t blocks, uint8_t* q,
    float* scale) {
  wait_for_previous();
  __shared__ uint32_t part[2][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int parity = 0;
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x, parity ^= 1) {
    const int64_t en = b / kb;  // e * nb + block of rows
    const int ki = static_cast<int>(b - en * kb);
    const int64_t e = en / nb;
    const int64_t r0 = (en - e * nb) * 128 + (threadIdx.x >> 3);
    const int64_t col = static_cast<int64_t>(ki) * 128 + (threadIdx.x & 7) * 16;
    Piece<BF16> p[4];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (r0 + 32 * i < n && col < cols) p[i].load(w, (e * n + r0 + 32 * i) * cols + col);
      else p[i].zero();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, p[i].amax_bits());
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) part[parity][warp] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, part[parity][i]);
    const Quant<BF16> qt(m);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r0 + 32 * i < n && col < cols)
        *reinterpret_cast<uint4*>(q + (e * n + r0 + 32 * i) * cols + col) = qt.convert(p[i]);
    if (threadIdx.x == 0) scale[b] = qt.scale;
  }
}

}  // namespace

cudaError_t launch_fp8_quantize_rows(int dtype, const void* x, int64_t rows_in, int64_t cols,
                                     const int32_t* assign_row, int k, int64_t rows_out,
                                     void* q, float* scale, cudaStream_t st) {
  if (rows_in == 0) return cudaSuccess;
  const int chunks = static_cast<int>((cols + 511) / 512);
  const int fold = cols <= 128 ? 2 : cols <= 256 ? 1 : 0;
  const int64_t blocks = (((rows_in + (1 << fold) - 1) >> fold) * chunks + 7) / 8;
  const int64_t most = static_cast<int64_t>(sm_count()) * 64;
  const int64_t grid = blocks < most ? blocks : most;
  uint8_t* out = static_cast<uint8_t*>(q);
  const bool bf16 = dtype == MOE_BF16;
  auto kernel = bf16 ? quantize_rows_kernel<true, 0> : quantize_rows_kernel<false, 0>;
  if (fold == 1) kernel = bf16 ? quantize_rows_kernel<true, 1> : quantize_rows_kernel<false, 1>;
  if (fold == 2) kernel = bf16 ? quantize_rows_kernel<true, 2> : quantize_rows_kernel<false, 2>;
  return launch_overlapping(kernel, grid, 256, 0, st, x, rows_in, static_cast<int>(cols), chunks,
                            assign_row, k, rows_out, out, scale);
}

cudaError_t launch_fp8_quantize_weights(int dtype, const void* w, int64_t E, int64_t n,
                                        int64_t cols, void* q, float* scale, cudaStream_t st) {
  const int nb = static_cast<int>((n + 127) / 128), kb = static_cast<int>((cols + 127) / 128);
  const int64_t blocks = E * nb * kb;
  const int64_t most = static_cast<int64_t>(sm_count()) * 64;
  const int64_t grid = blocks < most ? blocks : most;
  uint8_t* out = static_cast<uint8_t*>(q);
  return launch_overlapping(
      dtype == MOE_BF16 ? quantize_weights_kernel<true> : quantize_weights_kernel<false>, grid,
      256, 0, st, w, n, cols, nb, kb, blocks, out, scale);
}

}  // namespace moe
