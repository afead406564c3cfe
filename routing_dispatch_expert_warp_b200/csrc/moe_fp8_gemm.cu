// Products of ragged expert buckets with their expert's weight in 8-bit floating point (e4m3),
// one fp32 scale for each block of 128 along the reduction, and the SwiGLU expert FFN on them:
//   out[r, n] = sum over blocks b of  a_scale[r, b] w_scale[e, n / 128, b]
//                                     sum over c in block b of  a[r, c] w[e, n, c]
// for the rows r of bucket e.  The inner sums run on the 5th-generation tensor cores
// (tcgen05, e4m3 operands, fp32 accumulators in tensor memory), 128 columns at a time; the
// outer sum, whose factors change every 128 columns, runs in fp32 registers of the epilogue
// warps, which take the tensor cores' partial tile out of tensor memory after each block while
// the next block's MMAs fill the other half of it.
//
// Tile: 128 bucket rows x 256 weight rows.  FP8_LINEAR: 256 output columns.  FP8_GATED: 128
// columns of h, the weight rows being 128 of W_gate over the same 128 of W_up, so gate and up
// of an entry meet in one thread and a tile's 128 columns are one block of h's quantisation:
// the epilogue writes h = silu(gate) * up as e4m3 with its scale, and no h in higher precision
// exists.
//
// Block = 10 warps, one block per SM, persistent over tiles (numbered expert by expert,
// column block by column block, row blocks innermost, so that blocks running at the same time
// share weight tiles through L2; the table of tiles is built on the device):
//   warp 0 (one lane)  TMA producer: 128 x 128 bytes of rows, 256 x 128 of weights, 128-byte
//                      swizzle, 4 stages.  Of a bucket's last rows only as many groups of 32
//                      as hold rows are loaded.
//   warp 1 (one lane)  4 MMAs (K = 32 each) a stage into one of two accumulators (256 columns).
//   warps 2-9          epilogue: warp w has lane quarter w % 4 of tensor memory and half
//                      (w - 2) / 4 of the accumulator's columns: each thread sums 128 entries
//                      of one row.  A warp without bucket rows only keeps step.
// Every wait is bounded as in the bf16 expert GEMM.
#include <cuda_fp8.h>

#include "moe_internal.h"

namespace moe {
namespace {

constexpr int BM = 128;
constexpr int BK = 128;  // bytes = e4m3 values of a stage's rows: one block of the scales
constexpr int BN = 256;
constexpr int STAGES = 4;
constexpr int A_BYTES = BM * BK;
constexpr int B_BYTES = BN * BK;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr int ACC_COLS = 256;
constexpr int TMEM_COLS = 512;
constexpr int DYN_SMEM = STAGES * STAGE_BYTES + 1024;

enum Mode { FP8_LINEAR = 0, FP8_GATED = 1 };

struct Fp8Params {
  const int32_t* seg_start;  // [E] first row of each bucket
  const int32_t* seg_count;  // [E] rows of each bucket
  int E;
  int64_t rows;        // rows of a, a_scale and the outputs
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
  DevStatus* status;
  uint64_t wait_ns;
};

// acc += v * s for 16 columns of a thread's accumulator row, as packed pairs of fp32 FMAs.
__device__ __forceinline__ void fma_chunk(uint64_t (&acc)[64], int at, const uint32_t (&v)[16],
                                          uint64_t ss) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint64_t vv;
    asm("mov.b64 %0, {%1, %2};" : "=l"(vv) : "r"(v[2 * i]), "r"(v[2 * i + 1]));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc[at + i]) : "l"(vv), "l"(ss));
  }
}

__device__ __forceinline__ uint64_t both(float s) {
  uint64_t ss;
  asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "r"(__float_as_uint(s)));
  return ss;
}

// 32 lanes x 16 columns of tensor memory; the wait makes the loaded values usable.
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

__device__ __forceinline__ float2 unpack2(uint64_t v) {
  uint32_t lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
  return make_float2(__uint_as_float(lo), __uint_as_float(hi));
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

__device__ __forceinline__ float silu_mul(float g, float u) {
  return g / (1.0f + __expf(-g)) * u;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// The bucket table of a launch in shared memory.
struct Buckets {
  int start[MOE_MAX_EXPERTS];
  int count[MOE_MAX_EXPERTS];
  int tile_base[MOE_MAX_EXPERTS + 1];  // first tile of each bucket
};

// By one whole warp: every bucket cut to the rows there are, and the tiles before each.
__device__ void build_buckets(Buckets& t, const Fp8Params& p, int lane) {
  int carry = 0;
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
      t.count[e] = c;
      mb = (c + BM - 1) / BM;
    }
    int v = mb;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, v, off);
      if (lane >= off) v += o;
    }
    if (e < p.E) t.tile_base[e] = (carry + v - mb) * p.n_blocks;
    carry += __shfl_sync(0xffffffffu, v, 31);
  }
  if (lane == 0) t.tile_base[p.E] = carry * p.n_blocks;
}

struct Tile {
  int e, nb, row0, valid;  // expert, column block, first row, rows from there in the bucket
};

__device__ __forceinline__ Tile decode(const Buckets& t, const Fp8Params& p, int tile) {
  int lo = 0, hi = p.E - 1;  // largest e with tile_base[e] <= tile
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.tile_base[mid] <= tile) lo = mid;
    else hi = mid - 1;
  }
  const int mbs = (t.count[lo] + BM - 1) / BM;
  const int local = tile - t.tile_base[lo];
  Tile r;
  r.e = lo;
  r.nb = local / mbs;
  const int mb = local - r.nb * mbs;
  r.row0 = t.start[lo] + mb * BM;
  r.valid = t.count[lo] - mb * BM;
  return r;
}

// tm_a: rows in boxes of 128, tm_a32: the same rows in boxes of 32; tm_b0, tm_b1: the weights.
template <int MODE>
__global__ void __launch_bounds__(THREADS, 1) fp8_grouped_gemm_kernel(
    const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_a32,
    const __grid_constant__ CUtensorMap tm_b0, const __grid_constant__ CUtensorMap tm_b1,
    const Fp8Params p) {
  constexpr bool GATED = MODE == FP8_GATED;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[STAGES];
  __shared__ __align__(8) uint64_t empty_bar[STAGES];
  __shared__ __align__(8) uint64_t tfull_bar[2];
  __shared__ __align__(8) uint64_t tempty_bar[2];
  __shared__ __align__(8) uint64_t amax_bar;
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ uint32_t tmem_base_s;
  __shared__ volatile int abort_s;
  __shared__ Buckets bk;
  __shared__ uint32_t amax_s[2][2][BM];  // GATED: [tile parity][column half][row]

  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (warp == 0) {
    build_buckets(bk, p, lane);
    if (lane == 0) {
      prefetch_tensormap(&tm_a);
      prefetch_tensormap(&tm_a32);
      prefetch_tensormap(&tm_b0);
      if (GATED) prefetch_tensormap(&tm_b1);
    }
  } else if (warp == 1) {
    tmem_alloc(&tmem_base_s, TMEM_COLS);
    tmem_relinquish();
  } else if (threadIdx.x == 64) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull_bar[a], 1);
      mbar_init(&tempty_bar[a], EPI_WARPS);
    }
    mbar_init(&amax_bar, EPI_WARPS);
    mbar_init(&drain_bar, 1);
    abort_s = 0;
    fence_barrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem_base = tmem_base_s;
  const int total = bk.tile_base[p.E];

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      uint32_t armed = 0, armed_parity = 0;
      bool ok = true;
      for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
        const Tile t = decode(bk, p, tile);
        const int groups = t.valid > 96 ? 4 : (t.valid + 31) >> 5;  // of 32 rows
        for (int kb = 0; kb < p.kb; ++kb) {
          if (!mbar_wait(&empty_bar[s], ph ^ 1u, p.wait_ns, &abort_s)) {
            if (!abort_s)
              record_error(p.status, DEV_TIMEOUT, 41, static_cast<unsigned long long>(tile));
            abort_s = 1;
            ok = false;
            break;
          }
          uint8_t* sa = smem + s * STAGE_BYTES;
          uint8_t* sb = sa + A_BYTES;
          mbar_arrive_expect_tx(&full_bar[s], B_BYTES + groups * 32 * BK);
          armed |= 1u << s;
          armed_parity = (armed_parity & ~(1u << s)) | (ph << s);
          if (groups == 4) {
            tma_load_2d(sa, &tm_a, &full_bar[s], kb * BK, t.row0);
          } else {
            for (int g = 0; g < groups; ++g)
              tma_load_2d(sa + g * 32 * BK, &tm_a32, &full_bar[s], kb * BK, t.row0 + g * 32);
          }
          if (GATED) {
            tma_load_3d(sb, &tm_b0, &full_bar[s], kb * BK, t.nb * 128, t.e);
            tma_load_3d(sb + B_BYTES / 2, &tm_b1, &full_bar[s], kb * BK, t.nb * 128, t.e);
          } else {
            tma_load_3d(sb, &tm_b0, &full_bar[s], kb * BK, t.nb * BN, t.e);
          }
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // every fill this thread armed must land before the block can exit
      for (int q = 0; q < STAGES; ++q)
        if ((armed >> q) & 1u)
          mbar_wait(&full_bar[q], (armed_parity >> q) & 1u, p.wait_ns, nullptr);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(BM, BN);
      int s = 0;
      uint32_t ph = 0;
      int acc = 0;
      uint32_t aph = 0;
      bool ok = true, issued = false;
      for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
        for (int kb = 0; kb < p.kb; ++kb) {
          if (!mbar_wait(&tempty_bar[acc], aph ^ 1u, p.wait_ns, &abort_s) ||
              !mbar_wait(&full_bar[s], ph, p.wait_ns, &abort_s)) {
            if (!abort_s)
              record_error(p.status, DEV_TIMEOUT, 42, static_cast<unsigned long long>(tile));
            abort_s = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_addr = smem_addr(smem + s * STAGE_BYTES);
          const uint32_t b_addr = a_addr + A_BYTES;
          const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * ACC_COLS);
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            tc_mma_e4m3(d_tmem, sw128_kmajor_desc(a_addr + kk * 32),
                        sw128_kmajor_desc(b_addr + kk * 32), idesc, kk != 0 ? 1u : 0u);
          issued = true;
          tc_commit(&empty_bar[s]);
          tc_commit(&tfull_bar[acc]);
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
          acc ^= 1;
          if (acc == 0) aph ^= 1u;
        }
      }
      if (!ok && issued) {  // MMAs still reading smem / writing TMEM must finish first
        tc_commit(&drain_bar);
        mbar_wait(&drain_bar, 0, p.wait_ns, nullptr);
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3;           // TMEM lane quarter this warp may access
    const int half = (warp - 2) >> 2; // its half of the accumulator's columns
    const int r = q * 32 + lane;      // accumulator row of this thread
    // GATED: gate columns [64 half, +64) and the up columns 128 further; else [128 half, +128)
    const uint32_t col0 = static_cast<uint32_t>(GATED ? 64 * half : 128 * half);
    int acc_i = 0;
    uint32_t aph = 0;
    uint32_t xph = 0;
    bool ok = true;
    for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
      const Tile t = decode(bk, p, tile);
      const bool live = 32 * q < t.valid;  // the warp has bucket rows
      const bool row_ok = r < t.valid;
      const int64_t row = static_cast<int64_t>(t.row0) + (row_ok ? r : 0);
      const float* sa = p.a_scale + row * p.kb;
      // the weight's block of columns; one past the last is summed but never stored
      const int sb = GATED ? t.nb : min(2 * t.nb + half, p.nsb - 1);
      const int64_t sw = (static_cast<int64_t>(t.e) * p.nsb + sb) * p.kb;
      const float* s0 = p.w_scale0 + sw;
      const float* s1 = GATED ? p.w_scale1 + sw : nullptr;
      uint64_t acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0ull;
      float na = 0.f, n0 = 0.f, n1 = 0.f;  // the next block's scales
      if (live) {
        na = __ldg(sa);
        n0 = __ldg(s0);
        if (GATED) n1 = __ldg(s1);
      }
      for (int kb = 0; kb < p.kb; ++kb) {
        const float f0 = na * n0, f1 = GATED ? na * n1 : 0.f;
        if (live && kb + 1 < p.kb) {
          na = __ldg(sa + kb + 1);
          n0 = __ldg(s0 + kb + 1);
          if (GATED) n1 = __ldg(s1 + kb + 1);
        }
        const bool got = mbar_wait(&tfull_bar[acc_i], aph, p.wait_ns, &abort_s);
        if (!__all_sync(0xffffffffu, got)) {
          if (lane == 0 && !abort_s)
            record_error(p.status, DEV_TIMEOUT, 43, static_cast<unsigned long long>(tile));
          abort_s = 1;
          ok = false;
          break;
        }
        if (live) {
          // 16 columns at a time, the next ones on their way while these are summed
          tc_fence_after();
          const uint32_t ta = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                              static_cast<uint32_t>(acc_i * ACC_COLS) + col0;
          const uint64_t ss0 = both(f0), ss1 = both(f1);
          uint32_t v[2][16];
          tmem_ld16(ta, v[0]);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            tmem_wait16(v[c & 1]);
            if (c < 7) {
              const int n = c + 1;
              tmem_ld16(ta + (GATED ? (n & 3) * 16 + (n >> 2) * 128 : n * 16), v[n & 1]);
            }
            fma_chunk(acc, c * 8, v[c & 1], GATED && c >= 4 ? ss1 : ss0);
          }
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty_bar[acc_i]);
        acc_i ^= 1;
        if (acc_i == 0) aph ^= 1u;
      }
      if (!ok) break;
      if (GATED) {
        // h of this thread's 64 columns over its gate half of the accumulators, the row's
        // largest magnitude over both halves, then e4m3 and the scale
        uint32_t m = 0;
        if (live) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 g = unpack2(acc[i]), u = unpack2(acc[32 + i]);
            const uint32_t h0 = __float_as_uint(silu_mul(g.x, u.x));
            const uint32_t h1 = __float_as_uint(silu_mul(g.y, u.y));
            m = max(m, max(h0 & 0x7FFFFFFFu, h1 & 0x7FFFFFFFu));
            asm("mov.b64 %0, {%1, %2};" : "=l"(acc[i]) : "r"(h0), "r"(h1));
          }
        }
        amax_s[xph][half][r] = m;
        __syncwarp();
        if (lane == 0) mbar_arrive(&amax_bar);
        const bool got = mbar_wait(&amax_bar, xph, p.wait_ns, &abort_s);
        if (!__all_sync(0xffffffffu, got)) {
          if (lane == 0 && !abort_s)
            record_error(p.status, DEV_TIMEOUT, 44, static_cast<unsigned long long>(tile));
          abort_s = 1;
          break;
        }
        m = max(m, amax_s[xph][half ^ 1][r]);
        xph ^= 1u;
        if (row_ok) {
          const bool bad = m >= 0x7F800000u;
          const float mf = fmaxf(__uint_as_float(m), 7.8886090522101181e-31f);  // 2^-100
          const float rs = __fdiv_rn(448.0f, mf);
          const int col = t.nb * 128 + 64 * half;
          uint8_t* to = p.h + row * p.N + col;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 a = unpack2(acc[8 * i + 2 * j]), b = unpack2(acc[8 * i + 2 * j + 1]);
              w[j] = bad ? 0x7F7F7F7Fu : e4m3x4(a.x * rs, a.y * rs, b.x * rs, b.y * rs);
            }
            if (col + 16 * i < p.N)
              *reinterpret_cast<uint4*>(to + 16 * i) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          if (half == 0)
            p.h_scale[row * p.nsb + t.nb] =
                bad ? __uint_as_float(0x7FFFFFFFu) : __fdiv_rn(mf, 448.0f);
        }
      } else if (row_ok) {
        const int col = t.nb * BN + 128 * half;
        __nv_bfloat16* to = p.out + row * p.N + col;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 v = unpack2(acc[4 * i + j]);
            w[j] = pack_bf16x2(v.x, v.y);
          }
          if (col + 8 * i < p.N)
            *reinterpret_cast<uint4*>(to + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// ------------------------------------------------------------------ tensor maps
bool encode(CUtensorMap* m, int rank, const void* base, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  const cuuint32_t estr[3] = {1, 1, 1};
  return tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, static_cast<cuuint32_t>(rank),
                              const_cast<void*>(base), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [rows, K] bytes, boxes of box_rows x 128
bool map_rows(CUtensorMap* m, const void* base, int64_t rows, int64_t K, uint32_t box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
  const cuuint32_t box[2] = {BK, box_rows};
  return encode(m, 2, base, dims, strides, box);
}

// [E, N, K] bytes, boxes of 1 x box_n x 128
bool map_weights(CUtensorMap* m, const void* base, int64_t E, int64_t N, int64_t K,
                 uint32_t box_n) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(N),
                              static_cast<cuuint64_t>(E)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(N * K)};
  const cuuint32_t box[3] = {BK, box_n, 1};
  return encode(m, 3, base, dims, strides, box);
}

template <int MODE>
cudaError_t launch(const CUtensorMap& a, const CUtensorMap& a32, const CUtensorMap& b0,
                   const CUtensorMap& b1, const Fp8Params& p, cudaStream_t st) {
  cudaError_t err = cudaFuncSetAttribute(fp8_grouped_gemm_kernel<MODE>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, DYN_SMEM);
  if (err != cudaSuccess) return err;
  // at most one row block per bucket for its ragged end, and the rest full
  int64_t tiles = (p.rows / BM + (p.rows < p.E ? p.rows : p.E)) * p.n_blocks;
  if (tiles > sm_count()) tiles = sm_count();
  if (tiles < 1) tiles = 1;
  fp8_grouped_gemm_kernel<MODE><<<static_cast<unsigned>(tiles), THREADS, DYN_SMEM, st>>>(
      a, a32, b0, b1, p);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

size_t fp8_workspace_bytes() { return kFp8PartialsOffset; }

cudaError_t launch_fp8_gemm(const Fp8Gemm& g, void* ws, uint64_t wait_ns, cudaStream_t st,
                            const char** why) {
  if (g.rows == 0) return cudaSuccess;
  if (tensor_map_encoder() == nullptr) {
    *why = "cuTensorMapEncodeTiled is not available from the driver";
    return cudaErrorNotSupported;
  }
  const bool gated = g.w1 != nullptr;
  CUtensorMap a, a32, b0, b1;
  if (!map_rows(&a, g.a, g.rows, g.K, BM) || !map_rows(&a32, g.a, g.rows, g.K, 32) ||
      !map_weights(&b0, g.w0, g.E, g.N, g.K, gated ? 128 : BN) ||
      (gated && !map_weights(&b1, g.w1, g.E, g.N, g.K, 128))) {
    *why = "tensor map encoding failed (pointer alignment or sizes)";
    return cudaErrorInvalidValue;
  }
  if (!gated) b1 = b0;
  Fp8Params p{};
  p.seg_start = g.seg_start;
  p.seg_count = g.seg_count;
  p.E = g.E;
  p.rows = g.rows;
  p.K = static_cast<int>(g.K);
  p.N = static_cast<int>(g.N);
  p.n_blocks = static_cast<int>(gated ? (g.N + 127) / 128 : (g.N + BN - 1) / BN);
  p.kb = static_cast<int>((g.K + BK - 1) / BK);
  p.nsb = static_cast<int>((g.N + 127) / 128);
  p.a_scale = g.a_scale;
  p.w_scale0 = g.w_scale0;
  p.w_scale1 = g.w_scale1;
  p.out = static_cast<__nv_bfloat16*>(g.out);
  p.h = static_cast<uint8_t*>(g.h);
  p.h_scale = g.h_scale;
  p.status = static_cast<DevStatus*>(ws);
  p.wait_ns = wait_ns;
  return gated ? launch<FP8_GATED>(a, a32, b0, b1, p, st) : launch<FP8_LINEAR>(a, a32, b0, b1, p, st);
}

}  // namespace moe
