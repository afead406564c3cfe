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
// Tile: 128 bucket rows x 256 weight rows, as two halves of 128 weight rows that share the rows'
// tile in shared memory and have accumulators, barriers and epilogue warps of their own.
// FP8_LINEAR: half h is output columns [128 h, +128) of the tile's 256.  FP8_GATED: the tile is
// 128 columns of h, half h 64 of them: 64 rows of W_gate over the same 64 of W_up, so gate and
// up of an entry meet in one thread, and the tile's 128 columns are one block of h's
// quantisation: the epilogue writes h = silu(gate) * up as e4m3 with its scale, and no h in
// higher precision exists.
//
// Block = 12 warps, one block per SM, persistent over tiles (numbered expert by expert,
// column block by column block, row blocks innermost, so that blocks running at the same time
// share weight tiles through L2; the table of tiles is built on the device).  Every tile starts
// at stage 0 of the ring of 4 and at accumulator 0; each barrier's parity is a bit of a mask.
//   warp 0             TMA producer: 128 x 128 bytes of rows, 256 x 128 of weights, 128-byte
//                      swizzle.  Of a bucket's last rows only as many groups of 32 as hold rows
//                      are loaded.
//   warps 1, 2         MMA issuers, one for each half: 4 MMAs (128 x 128 x 32) a block into one
//                      of the half's two accumulators; one commit tells the producer that the
//                      half has left the stage and the epilogue that its sums are there.
//   warp 3             scales: the products a_scale * w_scale of 4 blocks at a time, a turn
//                      ahead, from global to shared memory.
//   warps 4-11         epilogue: warp w has lane quarter w % 4 of tensor memory in half
//                      (w - 4) / 4: each thread sums 128 entries of one row.  A warp without
//                      bucket rows only keeps step.
// A hand-over between an MMA issuer and an epilogue takes some 200 cycles each way.  With the
// halves apart, four accumulators of 128 columns are on their way round instead of two of 256,
// and one half's epilogue computes while the other's waits.  (One issuer with MMAs of 256
// columns for both halves, at that step and in bursts: 115 us for 4096 x 4096 x 7168 and 1.44 ms
// for the Mixtral-8x7B shaped prefill, against 116.5 and 1.45 here; but 8.1 ms for the
// DeepSeek-shaped prefill of 16384 tokens against 7.6, and 16.4 us for 13 ragged buckets against
// 15.6.)
// What it measured: 4096 x 4096 x 7168 in 117 us in a burst after a pause, 2.05 PFLOP/s; back to
// back for a second 133 to 137, 1.75 to 1.81, as the card's power limit lowers the clock to some
// 1.58 GHz.  The Mixtral-8x7B shaped prefill of 4096 tokens 1.49 and 1.70 to 1.72 ms (1.42 GHz),
// the DeepSeek-shaped one of 16384 tokens 7.0 to 7.2 and 8.0 to 8.4 ms (1.30 GHz).
// What bounds it, beside the power: no unit is full.  In that first case the tensor pipe is busy
// 61% of the time, the FMA pipe 18%, the issue slots 42%; operands come from L2 at 10 TB/s.  The
// rest is waiting: for the hand-overs, and in the epilogue for tensor memory, 16 columns at a
// time with one load in flight.  Without the epilogue's sums the copies and MMAs run at some 2.5
// PFLOP/s, without the MMAs the sums do as well.  Each instruction of the epilogue's loop
// counts: its own loads of scales cost a fifth, a warp number that is not known to be uniform 5
// to 9%, and four copies of the loop instead of two missed the instruction cache.
// Tiles are not cut along the reduction, so a product of few tiles leaves SMs idle: 128 and 256
// rows x 4096 x 14336, 16 and 32 tiles, take 51 us, where reading the weight takes 9.  Cutting
// was tried with a join that stored each lane's sums 512 bytes apart, between fences (256 x 4096
// x 14336 60 us whole, 55 cut; 384 x 7168 x 2048 17 whole, 41 cut), not with the join of
// moe_fp8_few.cu.
// Every wait is bounded as in the bf16 expert GEMM.
#include <mutex>

#include "moe_fp8_gemm.cuh"

namespace moe {
namespace {

constexpr int BM = 128;
// Rows an expert of the buffers (the host does not know the buckets) up to which moe_fp8_few.cu
// takes a product.  That kernel against this one, us, equal buckets that fill the buffers: the
// FFN of 8 experts of 4096 x 14336, 32 rows a bucket 237 and 258, 64 rows 271 and 272, 96 rows
// 478 and 279; that of 256 experts of 7168 x 2048, 32 rows 1731 and 1971, 64 rows 1987 and 1986,
// 96 rows 3734 and 2153; one product of 1 x 4096 x 14336, 32 rows 22 and 49, 64 rows 28 and 50,
// 256 rows 63 and 51.  So 33 to 64 rows an expert could as well go there, and few tiles should.
// 256 experts of 2048 x 7168 with 8192 rows, uneven: the longest bucket 267 rows 645 and 661,
// 1337 rows 702 and 694, 3293 rows 694 and 641.
constexpr int kFewRows = 32;
constexpr int A_BYTES = BM * BK;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int CTRL_WARPS = 4;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 32 * (CTRL_WARPS + EPI_WARPS);
// The launch's 168 registers a thread are split anew: 128 x 72 + 256 x 216 = 384 x 168.  All warps
// of a warpgroup have to execute the same setmaxnreg: the four control warps do before they part.
constexpr int LAUNCH_REGS = 168, CTRL_REGS = 72, EPI_REGS = 216;
static_assert(32 * (CTRL_WARPS * CTRL_REGS + EPI_WARPS * EPI_REGS) <= THREADS * LAUNCH_REGS,
              "setmaxnreg.inc would wait for registers that the block does not have");
constexpr int TMEM_COLS = 512;  // 2 halves x 2 accumulators x 128
// per epilogue warp: 32 rows x 64 bytes of output on their way to whole-row stores
constexpr int OUT_STAGE = 32 * 64;
constexpr int DYN_SMEM = STAGES * STAGE_BYTES + EPI_WARPS * OUT_STAGE + 1024;  // + alignment

// acc += v * s for 16 columns of a thread's accumulator row, as packed pairs of fp32 FMAs.
__device__ __forceinline__ void fma16(float2 (&acc)[64], int at, const uint32_t (&v)[16],
                                      float s) {
  const float2 ss = make_float2(s, s);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    acc[at / 2 + i] = __ffma2_rn(
        make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), ss,
        acc[at / 2 + i]);
}
template <int REGS>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}

// 64 bytes of each of a warp's 32 rows, a row's 16 words in its lane: through `buf` (16-byte
// piece c of row r at r * 64 + ((c ^ ((r >> 1) & 3)) * 16)), so that 4 lanes store a row's 64
// bytes at once, 8 rows an instruction.  Only rows before `rows` and the first `bytes` of the 64
// (a multiple of 16) are stored; to: the first row's 64 bytes, rows `stride` bytes apart.
__device__ __forceinline__ void store_rows64(uint8_t* buf, const uint32_t (&w)[16], uint8_t* to,
                                             int64_t stride, int rows, int bytes, int lane) {
  const int sw = (lane >> 1) & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint4*>(buf + lane * 64 + ((i ^ sw) << 4)) =
        make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  __syncwarp();
  const int seg = lane & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2);
    if (r < rows && seg * 16 < bytes)
      *reinterpret_cast<uint4*>(to + r * stride + seg * 16) =
          *reinterpret_cast<const uint4*>(buf + r * 64 + ((seg ^ ((r >> 1) & 3)) << 4));
  }
  __syncwarp();
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
  __shared__ __align__(8) uint64_t done_bar[2][STAGES];  // a half's MMAs on the stage are done
  __shared__ __align__(8) uint64_t tempty_bar[2][2];     // [half][accumulator]
  __shared__ __align__(8) uint64_t sfull_bar[2];         // 4 blocks' scales are there
  __shared__ __align__(8) uint64_t sfree_bar[2];         // ... and have been read
  __shared__ __align__(8) uint64_t amax_bar;
  __shared__ __align__(8) uint64_t drain_bar[2];
  __shared__ uint32_t tmem_base_s;
  __shared__ volatile int abort_s;
  __shared__ Buckets bk;
  __shared__ float scale_s[2][4][2][BM];  // [turn][block][LINEAR: half, GATED: gate, up][row]
  __shared__ uint32_t amax_s[2][2][BM];   // GATED: [tile parity][column half][row]

  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // uniform
  const int lane = threadIdx.x & 31;

  if (warp == 0) {
    if (lane == 0) {
      prefetch_tensormap(&tm_a);
      prefetch_tensormap(&tm_a32);
      prefetch_tensormap(&tm_b0);
      if (GATED) prefetch_tensormap(&tm_b1);
    }
    if (!p.follows) wait_for_previous();
    build_buckets<BM>(bk, p, lane);
  } else if (warp == 1) {
    tmem_alloc(&tmem_base_s, TMEM_COLS);
    tmem_relinquish();
  } else if (threadIdx.x == 64) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&done_bar[0][s], 1);
      mbar_init(&done_bar[1][s], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&tempty_bar[i >> 1][i & 1], EPI_WARPS / 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull_bar[i], 1);
      mbar_init(&sfree_bar[i], EPI_WARPS);
      mbar_init(&drain_bar[i], 1);
    }
    mbar_init(&amax_bar, EPI_WARPS);
    abort_s = 0;
    fence_barrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  if (GATED) let_next_start();  // the down product's blocks: they wait before they read h
  const uint32_t tmem_base = tmem_base_s;
  const int total = bk.tile_base[p.E];
  const int KB = p.kb;

  // The whole warp waits for a barrier.  Once a wait has run out, here or elsewhere in the
  // block, every role's next wait fails and the roles unwind.
  auto await = [&](uint64_t* bar, uint32_t parity, unsigned site, int tile) {
    uint64_t since = 0;
    while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
      const uint64_t now = global_ns();
      if (since == 0) since = now;
      if (__any_sync(0xffffffffu, abort_s != 0 || now - since > p.wait_ns)) {
        if (lane == 0) {
          if (!abort_s)
            record_error(p.status, DEV_TIMEOUT, site, static_cast<unsigned long long>(tile));
          abort_s = 1;
        }
        return false;
      }
    }
    return true;
  };

  if (warp < CTRL_WARPS) {
    regs_dec<CTRL_REGS>();
    if (warp == 0) {
      // ---------------------------------------------------------------- TMA producer
      uint32_t fills = 0;  // bit s: parity of stage s's next fill
      uint32_t armed = 0, armed_parity = 0;
      bool ok = true, waited = false;
      int early = 0;  // blocks of the first tile whose weights were loaded ahead
      for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
        const Tile t = decode<BM>(bk, p, tile);
        const int groups = t.valid > BM - 32 ? BM / 32 : (t.valid + 31) >> 5;  // of 32 rows
        auto load_weights = [&](int kb) {
          const int s = kb & (STAGES - 1);
          uint8_t* sb = smem + s * STAGE_BYTES + A_BYTES;
          mbar_arrive_expect_tx(&full_bar[s], B_BYTES + groups * 32 * BK);
          if (GATED) {
  #pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint8_t* to = sb + h * HALF_N * BK;
              tma_load_3d(to, &tm_b0, &full_bar[s], kb * BK, t.nb * 128 + h * 64, t.e);
              tma_load_3d(to + 64 * BK, &tm_b1, &full_bar[s], kb * BK, t.nb * 128 + h * 64, t.e);
            }
          } else {
            tma_load_3d(sb, &tm_b0, &full_bar[s], kb * BK, t.nb * BN, t.e);
          }
        };
        if (!waited) {  // when it follows, the first blocks' weights do not depend on the other
          early = min(STAGES, KB);
          if (elect_one())
            for (int kb = 0; kb < early; ++kb) load_weights(kb);
          __syncwarp();
          wait_for_previous();
          waited = true;
        }
  #pragma unroll 1
        for (int kb = 0; kb < KB; ++kb) {
          const int s = kb & (STAGES - 1);
          const uint32_t par = (fills >> s) & 1u;
          const bool ahead = early > 0;
          if (!ahead && (!await(&done_bar[0][s], par ^ 1u, 41, tile) ||
                         !await(&done_bar[1][s], par ^ 1u, 41, tile))) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + s * STAGE_BYTES;
          if (elect_one()) {
            if (!ahead) load_weights(kb);
            if (groups == 4) {
              tma_load_2d(sa, &tm_a, &full_bar[s], kb * BK, t.row0);
            } else {
              for (int g = 0; g < groups; ++g)
                tma_load_2d(sa + g * 32 * BK, &tm_a32, &full_bar[s], kb * BK, t.row0 + g * 32);
            }
          }
          __syncwarp();
          if (ahead) --early;
          armed |= 1u << s;
          armed_parity = (armed_parity & ~(1u << s)) | (par << s);
          fills ^= 1u << s;
        }
      }
      if (!waited) wait_for_previous();
      // every fill must land before the block can exit
      for (int s = 0; s < STAGES; ++s)
        if ((armed >> s) & 1u)
          mbar_wait(&full_bar[s], (armed_parity >> s) & 1u, kDrainNs, nullptr);
      __syncwarp();
    } else if (warp < 3) {
      // ---------------------------------------------------------------- MMA issuers
      wait_for_previous();
      constexpr uint32_t idesc = idesc_e4m3_f32(BM, HALF_N);
      const int h = warp - 1;
      const uint64_t a_desc = sw128_kmajor_desc(smem_addr(smem));
      const uint64_t b_desc = sw128_kmajor_desc(smem_addr(smem) + A_BYTES + h * HALF_N * BK);
      uint32_t fills = 0, uses = 0;  // parities: stage s's next fill, accumulator j's next use
      bool ok = true, issued = false;
      for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
  #pragma unroll 4
        for (int kb = 0; kb < KB; ++kb) {
          const int s = kb & (STAGES - 1), j = kb & 1;
          if (!await(&full_bar[s], (fills >> s) & 1u, 42, tile) ||
              !await(&tempty_bar[h][j], ((uses >> j) & 1u) ^ 1u, 42, tile)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t d_tmem = tmem_base + static_cast<uint32_t>((2 * h + j) * HALF_N);
  #pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk)  // descriptors count 16-byte units
              tc_mma_e4m3(d_tmem, a_desc + (s * STAGE_BYTES + kk * 32) / 16,
                          b_desc + (s * STAGE_BYTES + kk * 32) / 16, idesc, kk != 0 ? 1u : 0u);
            tc_commit(&done_bar[h][s]);
          }
          __syncwarp();
          issued = true;
          fills ^= 1u << s;
          uses ^= 1u << j;
        }
      }
      if (!ok && issued) {  // MMAs still reading smem / writing TMEM must finish first
        if (elect_one()) tc_commit(&drain_bar[h]);
        mbar_wait(&drain_bar[h], 0, kDrainNs, nullptr);
        __syncwarp();
      }
    } else if (warp == 3) {
      // ---------------------------------------------------------------- scales
      wait_for_previous();
      // A lane has rows lane + 32 i of the tile.  (The epilogue's threads loading their own rows'
      // scales took a fifth of its time: 32 rows' lanes are 32 passes of the L1.)
      uint32_t turns = 0;  // of 4 blocks, over all tiles
      bool ok = true;
      for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
        const Tile t = decode<BM>(bk, p, tile);
        const float* sa = p.a_scale + (static_cast<int64_t>(t.row0) + lane) * KB;
        const int64_t w_row = static_cast<int64_t>(t.e) * p.nsb;
        // LINEAR: the two halves' blocks of columns (one past the last is never stored)
        const float* s0 = p.w_scale0 + (w_row + (GATED ? t.nb : 2 * t.nb)) * KB;
        const float* s1 = GATED ? p.w_scale1 + (w_row + t.nb) * KB
                                : p.w_scale0 + (w_row + min(2 * t.nb + 1, p.nsb - 1)) * KB;
        for (int k0 = 0; k0 < KB; k0 += 4) {
          float4 a[4];
  #pragma unroll
          for (int m = 0; m < 4; ++m)
            a[m] = lane + 32 * m < t.valid
                       ? scales4(sa + static_cast<int64_t>(32 * m) * KB, k0, KB)
                       : make_float4(0.f, 0.f, 0.f, 0.f);
          const float4 w0 = scales4(s0, k0, KB), w1 = scales4(s1, k0, KB);
          const uint32_t b = turns & 1u;
          if (!await(&sfree_bar[b], ((turns >> 1) & 1u) ^ 1u, 45, tile)) {
            ok = false;
            break;
          }
  #pragma unroll
          for (int k = 0; k < 4; ++k)
  #pragma unroll
            for (int m = 0; m < 4; ++m) {
              scale_s[b][k][0][lane + 32 * m] = pick(a[m], k) * pick(w0, k);
              scale_s[b][k][1][lane + 32 * m] = pick(a[m], k) * pick(w1, k);
            }
          __syncwarp();
          arrive_if(&sfull_bar[b], lane == 0);
          ++turns;
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    regs_inc<EPI_REGS>();
    wait_for_previous();
    const int q = warp & 3;                     // TMEM lane quarter this warp may access
    const int half = (warp - CTRL_WARPS) >> 2;  // which half's accumulators
    const int r = q * 32 + lane;                // accumulator row of this thread
    const uint32_t first = lane == 0;
    const uint32_t ta = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                        static_cast<uint32_t>(2 * half * HALF_N);
    uint8_t* stage_out = smem + STAGES * STAGE_BYTES + (warp - CTRL_WARPS) * OUT_STAGE;
    uint32_t fills = 0;  // bit s: parity of stage s's next fill
    uint32_t turns = 0, xph = 0;
    bool ok = true;
    for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
      const Tile t = decode<BM>(bk, p, tile);
      const bool live = 32 * q < t.valid;  // the warp has bucket rows
      float2 acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.f, 0.f);
#pragma unroll 2
      for (int kb = 0; kb < KB; ++kb) {
        const int s = kb & (STAGES - 1), j = kb & 1;
        const uint32_t b = turns & 1u;
        if (s == 0 && !await(&sfull_bar[b], (turns >> 1) & 1u, 46, tile)) {
          ok = false;
          break;
        }
        const float f = scale_s[b][s][GATED ? 0 : half][r];
        const float g = GATED ? scale_s[b][s][1][r] : f;
        if (!await(&done_bar[half][s], (fills >> s) & 1u, 43, tile)) {
          ok = false;
          break;
        }
        fills ^= 1u << s;
        if (live) {
          tc_fence_after();
          const uint32_t from = ta + static_cast<uint32_t>(j * HALF_N);
          uint32_t v[2][16];
          // 16 columns at a time, the next ones on their way while these are summed
          tmem_ld16(from, v[0]);
#pragma unroll
          for (int c = 0; c < 7; ++c) {
            tmem_wait16(v[c & 1]);
            tmem_ld16(from + (c + 1) * 16, v[(c + 1) & 1]);
            fma16(acc, 16 * c, v[c & 1], c >= 4 ? g : f);
          }
          tmem_wait16(v[1]);
          tc_fence_before();
          arrive_if(&tempty_bar[half][j], first);
          fma16(acc, 16 * 7, v[1], g);
        } else {
          arrive_if(&tempty_bar[half][j], first);
        }
        if (s == STAGES - 1 || kb == KB - 1) {  // every lane has read the 4 blocks' scales
          __syncwarp();
          arrive_if(&sfree_bar[b], first);
          ++turns;
        }
      }
      if (!ok) break;
      const int left = t.valid - 32 * q;  // rows of this warp, from its first
      if (GATED) {
        // h of this thread's 64 columns over its gate half of the accumulators, the row's
        // largest magnitude over both halves, then e4m3 and the scale
        uint32_t m = 0;
        if (live) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            acc[i].x = silu_mul(acc[i].x, acc[32 + i].x);
            acc[i].y = silu_mul(acc[i].y, acc[32 + i].y);
            m = max(m, max(__float_as_uint(acc[i].x) & 0x7FFFFFFFu,
                           __float_as_uint(acc[i].y) & 0x7FFFFFFFu));
            if (i % 4 == 3) asm volatile("" ::: "memory");  // (not all quotients at once)
          }
        }
        amax_s[xph][half][r] = m;
        __syncwarp();
        arrive_if(&amax_bar, first);
        if (!await(&amax_bar, xph, 44, tile)) break;
        m = max(m, amax_s[xph][half ^ 1][r]);
        xph ^= 1u;
        if (live) {
          const RowQuant rq(m);
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            w[i] = rq.pack(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x, acc[2 * i + 1].y);
          const int col = t.nb * 128 + 64 * half;
          store_rows64(stage_out, w, p.h + (static_cast<int64_t>(t.row0) + 32 * q) * p.N + col,
                       p.N, left, p.N - col, lane);
          if (half == 0 && lane < left)
            p.h_scale[(static_cast<int64_t>(t.row0) + r) * p.nsb + t.nb] = rq.scale();
        }
      } else if (live) {
        const int col = t.nb * BN + HALF_N * half;
        uint8_t* to = reinterpret_cast<uint8_t*>(
            p.out + (static_cast<int64_t>(t.row0) + 32 * q) * p.N + col);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            w[i] = pack_bf16x2(acc[16 * c + i].x, acc[16 * c + i].y);
          store_rows64(stage_out, w, to + 64 * c, static_cast<int64_t>(p.N) * 2, left,
                       2 * (p.N - col - 32 * c), lane);
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

template <int MODE>
cudaError_t launch(const CUtensorMap& a, const CUtensorMap& a32, const CUtensorMap& b0,
                   const CUtensorMap& b1, const Fp8Params& p, cudaStream_t st) {
  // at most one ragged row block per bucket, the rest full
  const int64_t tiles = (p.rows / BM + (p.rows < p.E ? p.rows : p.E)) * p.n_blocks;
  return launch_product(fp8_grouped_gemm_kernel<MODE>, tiles, THREADS, DYN_SMEM, st, a, a32, b0,
                        b1, p);
}

}  // namespace

TensorMapEncodeFn tensor_map_encoder() {
  static TensorMapEncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* at = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &at, 12000, cudaEnableDefault,
                                         &found) == cudaSuccess &&
        found == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<TensorMapEncodeFn>(at);
  });
  return fn;
}

size_t fp8_workspace_bytes() {
  return kFp8PartialsOffset + sizeof(float) * SLOT_FLOATS * 2 * static_cast<size_t>(sm_count());
}

cudaError_t launch_fp8_gemm(const Fp8Gemm& g, void* ws, uint64_t wait_ns, cudaStream_t st,
                            const char** why) {
  if (g.rows == 0) return cudaSuccess;
  if (tensor_map_encoder() == nullptr) {
    *why = "cuTensorMapEncodeTiled is not available from the driver";
    return cudaErrorNotSupported;
  }
  const bool gated = g.w1 != nullptr;
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
  p.arrivals = reinterpret_cast<unsigned int*>(static_cast<uint8_t*>(ws) + kFp8CountersOffset);
  p.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kFp8PartialsOffset);
  p.status = static_cast<DevStatus*>(ws);
  p.wait_ns = wait_ns;
  p.follows = g.follows;
  if (g.rows <= kFewRows * static_cast<int64_t>(g.E)) return launch_fp8_few_rows(g, p, st, why);
  CUtensorMap a, a32, b0, b1;
  if (!map_rows(&a, g.a, g.rows, g.K, BM) || !map_rows(&a32, g.a, g.rows, g.K, 32) ||
      !map_weights(&b0, g.w0, g.E, g.N, g.K, gated ? 64 : BN) ||
      (gated && !map_weights(&b1, g.w1, g.E, g.N, g.K, 64))) {
    *why = "tensor map encoding failed (pointer alignment or sizes)";
    return cudaErrorInvalidValue;
  }
  if (!gated) b1 = b0;
  return gated ? launch<FP8_GATED>(a, a32, b0, b1, p, st)
               : launch<FP8_LINEAR>(a, a32, b0, b1, p, st);
}

}  // namespace moe
