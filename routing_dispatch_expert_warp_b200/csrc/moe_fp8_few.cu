// The products of moe_fp8_gemm.cu for buckets of few rows (decode steps): the operands change
// places.  A tile is 256 weight rows x up to 64 bucket rows; the weight rows are the MMA's 128
// rows twice over (two halves), the bucket rows its N = 16 .. 64 columns, taken in steps of 16.
// What bounds such a product is reading each expert's weight once.  With the rows in the MMA's
// 128 places, 4 rows cost the tensor cores and the epilogue as much as 128 (and power, which the
// clocks pay for): a DeepSeek-shaped decode step of 4 rows an expert takes 2.08 ms there and 1.60
// to 1.68 here, where a block of 128 costs the epilogue 16 sums a thread; that is 6.6 to 6.9
// TB/s.  32 experts of 7168 x 2048 with 128 rows take 77 to 81 us, 5.8 to 6.1 TB/s; one token
// through the Mixtral-8x7B shaped experts 67 to 69, of which reading the weights is 54.
//
// FP8_LINEAR: the halves are 128 output columns each.  FP8_GATED: 128 rows of W_gate and the
// same 128 of W_up; a thread has one column of h, and a tile's 128 columns are one block of h's
// quantisation.
//
// Block = 12 warps, one block per SM, persistent over tiles or pieces of tiles (Schedule):
//   warp 0      TMA producer: 256 x 128 bytes of weights and 16 .. 64 x 128 of rows a stage.
//   warp 1      MMA issuer: 2 x 4 MMAs (128 x n x 32) a stage into the stage's own accumulators
//               (64 columns for each half), one commit.
//   warp 2      scales: a_scale * w_scale of 4 blocks at a time, a turn ahead.
//   warps 4-11  epilogue: lane quarter w % 4 in half (w - 4) / 4: a thread sums one weight row's
//               entries of up to 64 bucket rows, each with that row's scale (a broadcast read
//               of shared memory).  At the end the sums go through shared memory, 16 bucket
//               rows at a time, to warps that take whole rows; those of a piece go to the
//               workspace instead, and the CTA whose piece arrives last adds the pieces up.
#include "moe_fp8_gemm.cuh"

namespace moe {
namespace {

constexpr int TM = 64;                 // bucket rows of a tile
constexpr int ROWS_BYTES = TM * BK;
constexpr int STAGE_BYTES = B_BYTES + ROWS_BYTES;
constexpr int CTRL_WARPS = 4;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 32 * (CTRL_WARPS + EPI_WARPS);
constexpr int TMEM_COLS = 512;         // 4 stages x 2 halves x 64
constexpr int OUT_ROWS = 16;           // bucket rows on their way through shared memory
constexpr int OUT_BYTES = OUT_ROWS * BN * 4;
constexpr int DYN_SMEM = STAGES * STAGE_BYTES + 2 * OUT_BYTES + 1024;  // + alignment
static_assert(SLOT_FLOATS == TM * BN, "partial sums of a piece: [64 bucket rows][256 weight rows]");

// The work of one CTA: tiles, or pieces of tiles along the reduction.
struct Piece {
  int tile;
  int kb0, kb1;  // its blocks of the reduction
  int slot;      // -1: the whole tile; else where its partial sums go, 2 slots a CTA
};

struct Schedule {
  int rounds;      // whole tiles this CTA takes: blockIdx.x + i * gridDim.x
  int ctas;        // that share the blocks of all tiles, when tiles are cut (else 0)
  int64_t units;   // those blocks: total * KB

  __device__ Schedule(int total, int KB) {
    const int G = static_cast<int>(gridDim.x);
    const int full = total / G, rest = total - full * G;
    // Whole tiles: the last round's `rest` tiles share the memory's rate, but an SM alone still
    // needs 2/5 of the time for a block that it needs when all SMs load.  Cut tiles keep all SMs
    // loading to the end and cost a join, as long as 4 blocks.  (Two experts' rows, K = 4096, 148
    // SMs: N = 20480, 12 left over, 42.0 us whole, 35.6 cut; N = 4096, 32 left over, 18.8 and
    // 16.6; N = 8192, 64 left over, 20.9 and 21.5; N = 28672, 76 left over, 44.1 and 45.1.)  Over
    // many rounds it gains little, and runs of neighbouring tiles lose that again.  Whole and
    // cut, us, after `full` whole rounds of 14336 x 4096: 6 rounds 150.7 and 145.8, 9 216.5 and
    // 213.8, 12 282.0 and 282.4, 15 349.4 and 351.1, 20 461.2 and 459.2, 26 595.3 and 597.5; of
    // 7168 x 2048: 6 81.5 and 79.4, 9 117.1 and 113.7, 12 150.3 and 150.2, 15 187.4 and 183.6, 20
    // 242.4 and 239.7, 26 314.1 and 309.1; 27 of the DeepSeek-shaped decode step 1588 and 1603.
    const bool cut = full < 10 && rest != 0 &&
                     static_cast<int64_t>(2 * G - 5 * rest) * KB > 20 * G;
    rounds = cut ? 0 : full + (static_cast<int>(blockIdx.x) < rest ? 1 : 0);
    units = cut ? static_cast<int64_t>(total) * KB : 0;
    ctas = units < 4 * G ? static_cast<int>((units + 3) >> 2) : G;
  }
  // first block of CTA c, and the CTA that has block u
  __device__ int64_t begin(int c) const { return units * c / ctas; }
  __device__ int owner(int64_t u) const { return static_cast<int>(((u + 1) * ctas - 1) / units); }
  // The i-th piece of this CTA (i counts up from 0); false past the last.
  __device__ bool get(int i, int KB, Piece& w) const {
    if (i < rounds) {
      w.tile = static_cast<int>(blockIdx.x + static_cast<unsigned>(i) * gridDim.x);
      w.kb0 = 0;
      w.kb1 = KB;
      w.slot = -1;
      return true;
    }
    const int c = static_cast<int>(blockIdx.x);
    if (c >= ctas) return false;
    const int64_t u0 = begin(c), u1 = begin(c + 1);
    const int first = static_cast<int>(u0 / KB);
    const int t = first + i - rounds;
    const int64_t t0 = static_cast<int64_t>(t) * KB;
    if (t0 >= u1) return false;
    w.tile = t;
    w.kb0 = t0 < u0 ? static_cast<int>(u0 - t0) : 0;
    w.kb1 = u1 - t0 < KB ? static_cast<int>(u1 - t0) : KB;
    w.slot = w.kb0 == 0 && w.kb1 == KB ? -1 : 2 * c + (t == first ? 0 : 1);
    return true;
  }
};

__device__ __forceinline__ unsigned add_acq_rel(unsigned* at, unsigned v) {
  unsigned before;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;"
               : "=r"(before)
               : "l"(at), "r"(v)
               : "memory");
  return before;
}

// One bucket row of a tile: the lane's sums of weight rows 4 lane .. + 3 of either half.
template <int MODE>
__device__ __forceinline__ void finish_row(const Fp8Params& p, int64_t row, int nb, float4 a,
                                           float4 b, int lane) {
  if (MODE == FP8_GATED) {
    const float h0 = silu_mul(a.x, b.x), h1 = silu_mul(a.y, b.y), h2 = silu_mul(a.z, b.z),
                h3 = silu_mul(a.w, b.w);
    uint32_t most = max(max(__float_as_uint(h0) & 0x7FFFFFFFu, __float_as_uint(h1) & 0x7FFFFFFFu),
                        max(__float_as_uint(h2) & 0x7FFFFFFFu, __float_as_uint(h3) & 0x7FFFFFFFu));
    most = __reduce_max_sync(0xffffffffu, most);
    const RowQuant rq(most);
    const int col = nb * HALF_N + 4 * lane;
    if (col < p.N)
      *reinterpret_cast<uint32_t*>(p.h + row * p.N + col) = rq.pack(h0, h1, h2, h3);
    if (lane == 0) p.h_scale[row * p.nsb + nb] = rq.scale();
  } else {
    const int col = nb * BN + 4 * lane;
    if (col < p.N)
      *reinterpret_cast<uint2*>(p.out + row * p.N + col) =
          make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
    if (col + HALF_N < p.N)
      *reinterpret_cast<uint2*>(p.out + row * p.N + col + HALF_N) =
          make_uint2(pack_bf16x2(b.x, b.y), pack_bf16x2(b.z, b.w));
  }
}

// tm_a: the bucket rows in boxes of 16; tm_b0, tm_b1: the weights in boxes of 256 (LINEAR) or
// 128 (GATED) rows.
template <int MODE>
__global__ void __launch_bounds__(THREADS, 1) fp8_few_rows_kernel(
    const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b0,
    const __grid_constant__ CUtensorMap tm_b1, const Fp8Params p) {
  constexpr bool GATED = MODE == FP8_GATED;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[STAGES];
  __shared__ __align__(8) uint64_t done_bar[STAGES];
  __shared__ __align__(8) uint64_t tempty_bar[STAGES];
  __shared__ __align__(8) uint64_t sfull_bar[2];  // 4 blocks' scales are there
  __shared__ __align__(8) uint64_t sfree_bar[2];  // ... and have been read
  __shared__ __align__(8) uint64_t out_bar;       // 16 rows' sums are in shared memory
  __shared__ __align__(8) uint64_t join_bar[2];   // partial sums written; who was last
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ uint32_t tmem_base_s;
  __shared__ volatile int abort_s;
  __shared__ int last_s;
  __shared__ Buckets bk;
  __shared__ __align__(16) float scale_s[2][4][2][TM];  // [turn][block][half][bucket row]

  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // uniform
  const int lane = threadIdx.x & 31;

  if (warp == 0) {
    if (lane == 0) {
      prefetch_tensormap(&tm_a);
      prefetch_tensormap(&tm_b0);
      if (GATED) prefetch_tensormap(&tm_b1);
    }
    if (!p.follows) wait_for_previous();
    build_buckets<TM>(bk, p, lane);
  } else if (warp == 1) {
    tmem_alloc(&tmem_base_s, TMEM_COLS);
    tmem_relinquish();
  } else if (threadIdx.x == 64) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&done_bar[s], 1);
      mbar_init(&tempty_bar[s], EPI_WARPS);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull_bar[i], 1);
      mbar_init(&sfree_bar[i], EPI_WARPS);
    }
    mbar_init(&out_bar, EPI_WARPS);
    mbar_init(&join_bar[0], EPI_WARPS);
    mbar_init(&join_bar[1], 1);
    mbar_init(&drain_bar, 1);
    abort_s = 0;
    fence_barrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  if (GATED) let_next_start();  // the down product's blocks: they wait before they read h
  const uint32_t tmem_base = tmem_base_s;
  const int KB = p.kb;
  const Schedule sched(bk.tile_base[p.E], KB);

  // The whole warp waits for a barrier.  Once a wait has run out, here or elsewhere in the
  // block, every role's next wait fails and the roles unwind.
  auto await = [&](uint64_t* bar, uint32_t parity, unsigned site, int tile) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const bool got = mbar_wait(bar, parity, p.wait_ns, &abort_s);
    if (__all_sync(0xffffffffu, got)) return true;
    if (lane == 0) {
      if (!abort_s)
        record_error(p.status, DEV_TIMEOUT, site, static_cast<unsigned long long>(tile));
      abort_s = 1;
    }
    return false;
  };
  // bucket rows of a tile in steps of 16
  auto steps_of = [](const Tile& t) { return t.valid > TM - 16 ? TM / 16 : (t.valid + 15) >> 4; };

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    uint32_t fills = 0;  // bit s: parity of stage s's next fill
    uint32_t armed = 0, armed_parity = 0;
    bool ok = true, waited = false;
    int early = 0;  // blocks of the first piece whose weights were loaded ahead
    int s = 0;      // the next block's stage
    Piece w;
    for (int i = 0; ok && sched.get(i, KB, w); ++i) {
      const Tile t = decode<TM>(bk, p, w.tile);
      const int steps = steps_of(t);
      auto load_weights = [&](int kb, int s) {
        uint8_t* to = smem + s * STAGE_BYTES;
        mbar_arrive_expect_tx(&full_bar[s], B_BYTES + steps * 16 * BK);
        if (GATED) {
          tma_load_3d(to, &tm_b0, &full_bar[s], kb * BK, t.nb * HALF_N, t.e);
          tma_load_3d(to + HALF_N * BK, &tm_b1, &full_bar[s], kb * BK, t.nb * HALF_N, t.e);
        } else {
          tma_load_3d(to, &tm_b0, &full_bar[s], kb * BK, t.nb * BN, t.e);
        }
      };
      if (!waited) {  // when it follows, the first blocks' weights do not depend on the other
        early = min(STAGES, w.kb1 - w.kb0);
        if (elect_one())
          for (int j = 0; j < early; ++j) load_weights(w.kb0 + j, j);
        __syncwarp();
        wait_for_previous();
        waited = true;
      }
#pragma unroll 1
      for (int kb = w.kb0; kb < w.kb1; ++kb, s = (s + 1) & (STAGES - 1)) {
        const uint32_t par = (fills >> s) & 1u;
        const bool ahead = early > 0;
        if (!ahead && !await(&done_bar[s], par ^ 1u, 51, w.tile)) {
          ok = false;
          break;
        }
        uint8_t* rows = smem + s * STAGE_BYTES + B_BYTES;
        if (elect_one()) {
          if (!ahead) load_weights(kb, s);
          for (int g = 0; g < steps; ++g)
            tma_load_2d(rows + g * 16 * BK, &tm_a, &full_bar[s], kb * BK, t.row0 + g * 16);
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
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    wait_for_previous();
    const uint64_t w_desc = sw128_kmajor_desc(smem_addr(smem));
    const uint64_t r_desc = sw128_kmajor_desc(smem_addr(smem) + B_BYTES);
    uint32_t fills = 0;  // stage s's next fill, and its accumulators' next use
    bool ok = true, issued = false;
    int s = 0;  // the next block's stage
    Piece w;
    for (int i = 0; ok && sched.get(i, KB, w); ++i) {
      const uint32_t idesc = idesc_e4m3_f32(128, 16 * steps_of(decode<TM>(bk, p, w.tile)));
#pragma unroll 1
      for (int kb = w.kb0; kb < w.kb1; ++kb, s = (s + 1) & (STAGES - 1)) {
        const uint32_t par = (fills >> s) & 1u;
        if (!await(&full_bar[s], par, 52, w.tile) || !await(&tempty_bar[s], par ^ 1u, 52, w.tile)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk)  // descriptors count 16-byte units
              tc_mma_e4m3(tmem_base + static_cast<uint32_t>((2 * s + h) * TM),
                          w_desc + (s * STAGE_BYTES + h * HALF_N * BK + kk * 32) / 16,
                          r_desc + (s * STAGE_BYTES + kk * 32) / 16, idesc, kk != 0 ? 1u : 0u);
          tc_commit(&done_bar[s]);
        }
        __syncwarp();
        issued = true;
        fills ^= 1u << s;
      }
    }
    if (!ok && issued) {  // MMAs still reading smem / writing TMEM must finish first
      if (elect_one()) tc_commit(&drain_bar);
      mbar_wait(&drain_bar, 0, kDrainNs, nullptr);
      __syncwarp();
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------------- scales
    wait_for_previous();
    uint32_t turns = 0;  // of 4 blocks, over all pieces
    bool ok = true;
    Piece w;
    for (int i = 0; ok && sched.get(i, KB, w); ++i) {
      const Tile t = decode<TM>(bk, p, w.tile);
      const float* sa = p.a_scale + (static_cast<int64_t>(t.row0) + lane) * KB;
      const int64_t w_row = static_cast<int64_t>(t.e) * p.nsb;
      // LINEAR: the two halves' blocks of columns (one past the last is never stored)
      const float* s0 = p.w_scale0 + (w_row + (GATED ? t.nb : 2 * t.nb)) * KB;
      const float* s1 = GATED ? p.w_scale1 + (w_row + t.nb) * KB
                              : p.w_scale0 + (w_row + min(2 * t.nb + 1, p.nsb - 1)) * KB;
      for (int k0 = w.kb0 & ~3; k0 < w.kb1; k0 += 4) {
        float4 a[2];
#pragma unroll
        for (int m = 0; m < 2; ++m)
          a[m] = lane + 32 * m < t.valid
                     ? scales4(sa + static_cast<int64_t>(32 * m) * KB, k0, KB)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 w0 = scales4(s0, k0, KB), w1 = scales4(s1, k0, KB);
        const uint32_t b = turns & 1u;
        if (!await(&sfree_bar[b], ((turns >> 1) & 1u) ^ 1u, 53, w.tile)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            scale_s[b][k][0][lane + 32 * m] = pick(a[m], k) * pick(w0, k);
            scale_s[b][k][1][lane + 32 * m] = pick(a[m], k) * pick(w1, k);
          }
        __syncwarp();
        arrive_if(&sfull_bar[b], lane == 0);
        ++turns;
      }
    }
  } else if (warp >= CTRL_WARPS) {
    // ---------------------------------------------------------------- epilogue
    wait_for_previous();
    const int ew = warp - CTRL_WARPS;
    const int q = warp & 3;          // TMEM lane quarter this warp may access
    const int half = ew >> 2;
    const int r = half * HALF_N + q * 32 + lane;  // weight row of this thread in the tile
    const uint32_t first = lane == 0;
    const uint32_t ta = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                        static_cast<uint32_t>(half * TM);
    float* stage_out = reinterpret_cast<float*>(smem + STAGES * STAGE_BYTES);
    uint32_t fills = 0;  // bit s: parity of stage s's next fill
    uint32_t turns = 0, oph = 0, jph = 0;
    int s = 0;  // the next block's stage
    bool ok = true;
    Piece w;
    for (int i = 0; ok && sched.get(i, KB, w); ++i) {
      const int tile = w.tile;
      const Tile t = decode<TM>(bk, p, tile);
      const int steps = steps_of(t);
      const int valid = min(t.valid, TM);
      float acc[TM];
#pragma unroll
      for (int c = 0; c < TM; ++c) acc[c] = 0.f;
#pragma unroll 1
      for (int kb = w.kb0; kb < w.kb1; ++kb, s = (s + 1) & (STAGES - 1)) {
        const uint32_t b = turns & 1u;
        const bool turn = (kb & 3) == 0 || kb == w.kb0;  // the first of the 4 blocks' scales
        if ((turn && !await(&sfull_bar[b], (turns >> 1) & 1u, 54, tile)) ||
            !await(&done_bar[s], (fills >> s) & 1u, 55, tile)) {
          ok = false;
          break;
        }
        fills ^= 1u << s;
        tc_fence_after();
        const float4* f = reinterpret_cast<const float4*>(scale_s[b][kb & 3][half]);
        const uint32_t from = ta + static_cast<uint32_t>(2 * s * TM);
#pragma unroll
        for (int g = 0; g < TM / 16; ++g)
          if (g < steps) {
            uint32_t v[16];
            tmem_ld16(from + 16 * g, v);
            const float4 f0 = f[4 * g], f1 = f[4 * g + 1], f2 = f[4 * g + 2], f3 = f[4 * g + 3];
            tmem_wait16(v);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float4 fc = c == 0 ? f0 : c == 1 ? f1 : c == 2 ? f2 : f3;
              float* a = acc + 16 * g + 4 * c;
              a[0] = fmaf(__uint_as_float(v[4 * c]), fc.x, a[0]);
              a[1] = fmaf(__uint_as_float(v[4 * c + 1]), fc.y, a[1]);
              a[2] = fmaf(__uint_as_float(v[4 * c + 2]), fc.z, a[2]);
              a[3] = fmaf(__uint_as_float(v[4 * c + 3]), fc.w, a[3]);
            }
          }
        tc_fence_before();
        arrive_if(&tempty_bar[s], first);
        if ((kb & 3) == 3 || kb == w.kb1 - 1) {  // every lane has read the 4 blocks' scales
          __syncwarp();
          arrive_if(&sfree_bar[b], first);
          ++turns;
        }
      }
      if (!ok) break;
      if (w.slot >= 0) {
        // a piece: its sums go to the workspace; the CTA whose piece of the tile is the last to
        // arrive there adds all of them up, first piece first
        float* to = p.partials + static_cast<int64_t>(w.slot) * SLOT_FLOATS + r;
#pragma unroll
        for (int c = 0; c < TM; ++c)
          if (c < valid) __stcg(to + c * BN, acc[c]);
        const int64_t tile0 = static_cast<int64_t>(tile) * KB;
        // its pieces' CTAs; each has the tile as its run's first, but for the first of them when
        // that one's run starts in a tile before
        const int c0 = sched.owner(tile0), c1 = sched.owner(tile0 + KB - 1);
        const bool starts = sched.begin(c0) == tile0;
        __syncwarp();
        arrive_if(&join_bar[0], first);
        if (warp == CTRL_WARPS) {
          if (!await(&join_bar[0], jph, 57, tile)) break;
          if (lane == 0) {
            // release: the sums of all the block's warps, which the barrier has brought here;
            // acquire: the other blocks' sums, for the warps that the next barrier lets go
            // (c0 tells cut tiles apart: only the last tile of a run goes on in the next one)
            const unsigned before = add_acq_rel(p.arrivals + c0, 1u);
            const int is_last = before == static_cast<unsigned>(c1 - c0);
            if (is_last) p.arrivals[c0] = 0u;  // as the next launch wants it
            last_s = is_last;
          }
          __syncwarp();
          arrive_if(&join_bar[1], first);
        }
        if (!await(&join_bar[1], jph, 58, tile)) break;
        jph ^= 1u;
        if (last_s != 0) {
#pragma unroll 1
          for (int m = ew; m < valid; m += EPI_WARPS) {
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
#pragma unroll 8
            for (int c = c0; c <= c1; ++c) {
              const int slot = 2 * c + (c == c0 && !starts ? 1 : 0);
              const float4* from = reinterpret_cast<const float4*>(
                                       p.partials + static_cast<int64_t>(slot) * SLOT_FLOATS +
                                       m * BN) + lane;
              const float4 x = __ldcg(from), y = __ldcg(from + HALF_N / 4);
              a.x += x.x;
              a.y += x.y;
              a.z += x.z;
              a.w += x.w;
              b.x += y.x;
              b.y += y.y;
              b.z += y.z;
              b.w += y.w;
            }
            finish_row<MODE>(p, static_cast<int64_t>(t.row0) + m, t.nb, a, b, lane);
          }
        }
        continue;
      }
      // whole tiles: 16 bucket rows at a time through shared memory, two buffers in turn (a warp
      // writes a buffer again only after all have been through the other one's barrier)
#pragma unroll
      for (int g = 0; g < TM / 16; ++g)
        if (ok && g < steps) {
          float* buf = stage_out + (oph & 1u) * (OUT_ROWS * BN);
#pragma unroll
          for (int c = 0; c < 16; ++c) buf[c * BN + r] = acc[16 * g + c];
          __syncwarp();
          arrive_if(&out_bar, first);
          ok = await(&out_bar, oph & 1u, 56, tile);
          oph ^= 1u;
          if (ok)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const int c = ew + m * EPI_WARPS;
              if (16 * g + c < valid) {
                const float4* row = reinterpret_cast<const float4*>(buf + c * BN) + lane;
                finish_row<MODE>(p, static_cast<int64_t>(t.row0) + 16 * g + c, t.nb, row[0],
                                 row[HALF_N / 4], lane);
              }
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
cudaError_t launch(const CUtensorMap& a, const CUtensorMap& b0, const CUtensorMap& b1,
                   const Fp8Params& p, cudaStream_t st) {
  // at most one ragged row block per bucket, the rest full; each can be cut into pieces
  const int64_t tiles = (p.rows / TM + (p.rows < p.E ? p.rows : p.E)) * p.n_blocks;
  return launch_product(fp8_few_rows_kernel<MODE>, tiles * ((p.kb + 3) / 4), THREADS, DYN_SMEM,
                        st, a, b0, b1, p);
}

}  // namespace

cudaError_t launch_fp8_few_rows(const Fp8Gemm& g, const Fp8Params& p, cudaStream_t st,
                                const char** why) {
  const bool gated = g.w1 != nullptr;
  CUtensorMap a, b0, b1;
  if (!map_rows(&a, g.a, g.rows, g.K, 16) ||
      !map_weights(&b0, g.w0, g.E, g.N, g.K, gated ? HALF_N : BN) ||
      (gated && !map_weights(&b1, g.w1, g.E, g.N, g.K, HALF_N))) {
    *why = "tensor map encoding failed (pointer alignment or sizes)";
    return cudaErrorInvalidValue;
  }
  if (!gated) b1 = b0;
  return gated ? launch<FP8_GATED>(a, b0, b1, p, st) : launch<FP8_LINEAR>(a, b0, b1, p, st);
}

}  // namespace moe
