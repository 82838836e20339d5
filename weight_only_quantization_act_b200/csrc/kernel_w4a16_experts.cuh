// kernel_w4a16_experts.cuh - products of many rows with their experts' packed 4-bit weights: Y[r] = X'[r] deq(W_e)^T
// for the sorted rows of each expert, optionally with the SiLU gate of a stacked gate and up projection in the
// epilogue. An expert with up to 8 rows is left to kernel_w4a16_few.cuh.
//
// Mathematics: Y[m, o] = sum_g step[o, g] sum_{k in g} (q[o, k] - z[o, g]) x'[m, k]. The tensor cores sum a group's
// q - z, exact in bf16, into a fresh fp32 accumulator; the epilogue warps scale each group by its fp32 step and add
// it to fp32 sums in registers. So the weight enters with its exact value (a zero point beyond +-240, which
// takes a group of nearly equal weights, leaves q - z rounded to bf16: the rounding that a restored bf16 weight
// has everywhere), and a code costs less than its dequantization: two masks per word split it into even and odd
// nibbles, a byte permute puts a byte of each under a zero byte (the byte's copied sign), which is the bf16
// subnormal q 2^-133 or 16 q 2^-133, and one paired bf16 FMA gives (q - z) 2^-6 for two in-features in their natural
// order. The 2^6 goes into the step.
//
// The weights stand on the MMA's M side, read from tensor memory, and the expert's tokens on its N side, whose
// width is set per tile: a tile is 256 weight rows (128 per CTA of a pair; gated: 128 outputs, their gate and up rows
// in turns of 16) times up to 192 tokens of one expert, N the tokens rounded up to 16, so a ragged expert wastes less
// than 16 columns of tensor work. Experts of more than 192 rows are cut into tiles of nearly equal width. A row of
// the accumulator is a weight row, so its lanes store consecutive outputs of one token and no store goes past an
// expert's last row.
//
// Bounds: at N = 192 a group takes the tensor cores 768 cycles, the unpacking about 200 and the scaling about 140
// issue cycles of every SM quarter. Below N = 100 the codes arrive no faster than that from HBM (9 KB per SM and
// group, 400 cycles at the 6.6 TB/s of a copy). 192 and not 256 tokens: two accumulators of N columns and two operand
// buffers of 64 fill tensor memory. Where every tile of the call is narrower, three groups (up to 96 tokens) or four (up to
// 64) are in flight instead of two: the way from a group's end through the unpackers and scaling warps to the next group's
// MMAs takes about 2000 cycles.
//
// Persistent, clusters of 2 CTAs, one CTA per SM; every CTA makes the table of tiles from the row offsets for
// itself and takes each n-th tile, so nothing is exchanged between pairs. Warps of a CTA:
//   0      TMA of this CTA's half of the tile's token rows, a group at a time (two boxes of 64 in-features, 128-byte
//          swizzle, the box's height 32, 64 or 96 rows), into a ring of 4
//   1      tensor memory; the even CTA issues the pair MMAs (cta_group::2, M = 256, N, K = 16, A from tensor memory)
//          into two to four accumulators in turn, one group each
//   2      TMA of the code words, 128 rows x 256 in-features at a time (128 bytes of a row), into a ring of its own
//   3      steps and zero points of those rows and groups by cp.async, counted on the same barrier
//   4-11   scaling and epilogue: two warps per quarter of the rows, alternate blocks of 32 tokens
//   12-19  unpackers: two sets of four warps that take groups in turn, a weight row per lane, into as many operand buffers
// The thread that issues the MMAs waits once per group: one barrier counts the token rows, the unpacked operand and the
// reading of the accumulator that the group will overwrite, and one commit per group tells all three that it is done
// (with a wait and a commit for each, and per 64 in-features, that thread took 1700 cycles per group). Every wait
// is bounded, and one that gives up ends its role.
//
// Measured (B200, calls back to back on a router's counts): 16384 rows to 32 experts of 4096 -> 2 x 2048, gated, 650 us, 0.85
// PFLOP/s (the kernel by itself 638; 512 rows to each expert 589); 600 rows to 8 of 14336 -> 4096 150 to 161 us; 12 rows to
// each of 8 of 4096 -> 2 x 14336, gated, 232 us, and the same for 9 to 64 rows each. Two things bound it. A group's work is
// short against what surrounds it: the barriers alone, with neither unpacking, scaling, loads nor more than one MMA, take 700
// cycles per group, and what counted most was every instruction in the loops of the unpackers and scaling warps (for the
// 16384 rows, where the kernel stood at 553 us in a probe: a test per block, the remote barrier's address made anew for each
// arrival, an unlikely branch before the stores and a poll with a suspend time together 742 against 581; unpackers that share
// each group instead of taking them in turn 581 against 553). And at 192 tokens the accumulators that fit are two, so the
// scaling of a group has one group's MMAs to hide behind.
#pragma once
#include <cstdint>
#include <type_traits>
#include <cuda.h>
#include <cuda_bf16.h>

#include "dequant_w4.cuh"
#include "kernel_w4a16.cuh"
#include "kernel_w4a16_few.cuh"
#include "ptx.cuh"

namespace awq {
namespace grp {

constexpr int HALF = 128;                         // weight rows per CTA
constexpr int BN = 192;                           // tokens per tile at most
constexpr int BK = 64;
constexpr int UK = 16;
constexpr int STAGES = 4;                         // token ring, and ring of group barriers
constexpr int X_BOX = 32;                         // token rows per TMA box: this, twice or three times it
constexpr int X_HALF_BYTES = BN / 2 * BK * 2;     // 12 KB  this CTA's token rows, 64 in-features
constexpr int X_BYTES = 2 * X_HALF_BYTES;
constexpr int A_COLS = BK;                        // operand buffer: two in-features per 32-bit column, 128 of them
constexpr int CSTAGES = 4;                        // code ring: two groups per slot, 32 words = 128 bytes of each row
constexpr int C_BYTES = HALF * 128;               // 16 KB  code words
constexpr int P_BYTES = HALF * 2 * 4;             // 1 KB   steps (zero points) of two groups
constexpr int CSTAGE_BYTES = C_BYTES + 2 * P_BYTES;
constexpr int FIRST_EPI = 4, EPI_WARPS = 8;
constexpr int FIRST_DQ = 12, DQ_SETS = 2, DQ_WARPS = 4 * DQ_SETS;
constexpr int THREADS = 32 * (FIRST_DQ + DQ_WARPS);
// 640 threads x 96 registers at launch; the scaling warps hold 96 sums each
constexpr int LAUNCH_REGS = 96, EPI_REGS = 152, DQ_REGS = 64, ROLE_REGS = 48;
static_assert(32 * (FIRST_EPI * ROLE_REGS + EPI_WARPS * EPI_REGS + DQ_WARPS * DQ_REGS) <= THREADS * LAUNCH_REGS,
              "the shares fit what the block was launched with");
constexpr int BLOCK = 32;                         // tokens per load of a scaling warp
constexpr int CHUNKS = BN / BLOCK / 2;            // blocks per scaling warp
constexpr int MAX_EXPERTS = 1024;
constexpr int TABLE_BYTES = 2 * (MAX_EXPERTS + 1) * 4;
constexpr int SMEM_BYTES = STAGES * X_BYTES + CSTAGES * CSTAGE_BYTES + TABLE_BYTES + 1024;
constexpr uint32_t TMEM_COLS = 512;
static_assert(2 * (BN + A_COLS) <= TMEM_COLS && 3 * (96 + A_COLS) <= TMEM_COLS && 4 * (64 + A_COLS) <= TMEM_COLS &&
                  STAGES >= 4,
              "accumulators and operand buffers fit tensor memory");
static_assert(SMEM_BYTES <= 232448, "fits the 227 KB of dynamic shared memory");
static_assert(X_HALF_BYTES % 1024 == 0 && CSTAGE_BYTES % 1024 == 0 && BN / 2 == 3 * X_BOX,
              "tiles stay 1024-byte aligned and the largest box fits");

struct Params {
  const int* offsets;      // [E + 1]
  const float* steps;      // [E][O][G]
  const float* zeros;
  uint16_t* Y;             // [R][ldy]
  int64_t R, O, G, ldy;
  int E;
  int n_bands;             // tiles along the weight rows
  int pair_params;         // steps and zero points of two groups can be copied as 8 bytes
  int stall_tile;          // test hook: at this tile the MMAs wait for what nobody signals (-1: nowhere)
  DeviceStatus* status;
  uint64_t limit_ns;
};

struct Tile {
  int e, band, row0, tokens;  // first sorted row and number of rows
  __device__ __forceinline__ uint32_t n() const { return static_cast<uint32_t>((tokens + 15) & ~15); }
};

__device__ __forceinline__ int token_tiles(int rows) { return (rows + BN - 1) / BN; }
// Rows per token tile: nearly equal tiles, full ones where there are so many that rounding up to 16 could
// leave the last one empty.
__device__ __forceinline__ int tile_rows(int rows, int tiles) {
  return tiles >= BN / 16 ? BN : ((rows + tiles - 1) / tiles + 15) & ~15;
}

__device__ __forceinline__ Tile tile_of(int t, const int* first_tile, const int* first_row, int E) {
  int lo = 0, hi = E - 1;  // the last e with first_tile[e] <= t; an expert without tiles never is
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first_tile[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  const int rows = first_row[lo + 1] - first_row[lo];
  const int tiles = token_tiles(rows), per = tile_rows(rows, tiles);
  const int local = t - first_tile[lo];
  Tile r;
  r.e = lo;
  r.band = local / tiles;
  const int start = (local - r.band * tiles) * per;
  r.row0 = first_row[lo] + start;
  r.tokens = min(per, rows - start);
  return r;
}

__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Pair MMA with A from tensor memory (each CTA's 128 rows in its own), B half from each CTA's shared memory.
__device__ __forceinline__ void umma_bf16_pair_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                  uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on a barrier of either CTA of the pair after tensor-memory accesses alone, which the tcgen05 fences around
// it order: no release of this thread's other writes to the cluster (a fence that takes longer than the unpacking of a
// k-block).
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// y += s * v on both fp32 lanes, v given as two registers.
__device__ __forceinline__ void fma_f32x2(uint64_t& y, uint64_t s, uint32_t lo, uint32_t hi) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(y) : "l"(f32x2_pack(lo, hi)), "l"(s));
}

// (q - z) 2^-6 of the word's eight codes, two per register in the order of the in-features. `zb`: -z 2^-6 in both
// halves; exact for |z| <= 240.
__device__ __forceinline__ void unpack_word(uint32_t w, uint32_t zb, uint32_t* o) {
  const uint32_t even = w & 0x0F0F0F0Fu, odd = w & 0xF0F0F0F0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // bytes: even_j, its sign (0), odd_j, the sign of even_j (0)
    const uint32_t sel = (8u | j) << 12 | (4u | j) << 8 | (8u | j) << 4 | j;
    uint32_t t;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(t) : "r"(even), "r"(odd), "r"(sel));
    // low half q 2^-133 * 2^127, high half 16 q 2^-133 * 2^123
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(o[j]) : "r"(t), "r"(0x7D007F00u), "r"(zb));
  }
}
// The same for any zero point: q - z rounded to bf16 (both scalings are exact).
__device__ __forceinline__ uint32_t unpack_pair_any(uint32_t byte, float z) {
  const float lo = __fsub_rn(static_cast<float>(byte & 0xFu), z) * 0.015625f;
  const float hi = __fsub_rn(static_cast<float>(byte >> 4), z) * 0.015625f;
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Bounded waits. One that gives up, after the limit or because another has, says so, and from there on its role arrives on no
// barrier and issues no copy, MMA or store that only a completed wait allows: nothing downstream takes an unfinished group
// for a finished one, and no more than the rings hold is in flight. The status and the clock are looked at after 64
// polls, so a wait that is met costs its poll and one branch; a time that the hardware may suspend the thread for, given
// with the poll, cost 2 to 4 % by waking it late.
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, DeviceStatus* st, uint64_t limit, unsigned where) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if (status_code(st) != 0u) return false;
    if (global_timer_ns() - t0 > limit) {
      raise_timeout(st, where);
      return false;
    }
  }
  return true;
}
// For one thread. Where all lanes of a warp poll, lane 0 arrives for them if it has not given up itself: the phase is then
// complete, also for a lane that has, whose own reading may have come too early and which discards the tile.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const Params& p, unsigned where) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, p.status, p.limit_ns, where);
}
// For a whole warp, which gets one answer: lane 0 decides to give up. (The scaling warps vote once per tile, since nothing but
// their arrivals counts until then: with a vote per wait 600 rows to 8 experts of 14336 -> 4096 took 169 us, not 156.)
__device__ __forceinline__ bool wait_warp_slow(uint32_t bar, uint32_t parity, DeviceStatus* st, uint64_t limit, unsigned where) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t i = 0;; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (i < 64) continue;
    bool give_up = false;
    if ((threadIdx.x & 31) == 0) {
      const uint64_t now = global_timer_ns();
      if (i == 64) t0 = now;
      give_up = status_code(st) != 0u;
      if (!give_up && now - t0 > limit) {
        raise_timeout(st, where);
        give_up = true;
      }
    }
    if (__any_sync(0xffffffffu, give_up)) return false;
  }
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const Params& p, unsigned where) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || wait_warp_slow(bar, parity, p.status, p.limit_ns, where);
}
// The status as lane 0 finds it, for the whole warp.
__device__ __forceinline__ bool warp_ok(const DeviceStatus* st) { return __shfl_sync(0xffffffffu, status_code(st), 0) == 0u; }

template <bool GATED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    w4a16_experts_kernel(const __grid_constant__ CUtensorMap tmX1, const __grid_constant__ CUtensorMap tmX2,
                         const __grid_constant__ CUtensorMap tmX3, const __grid_constant__ CUtensorMap tmC, Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t bars[2 * STAGES + 2 * CSTAGES + 2];
  __shared__ uint32_t tmem_slot;
  __shared__ int widest;  // tokens of the call's widest tile
  int* first_row = reinterpret_cast<int*>(smem + STAGES * X_BYTES + CSTAGES * CSTAGE_BYTES);  // [E + 1]
  int* first_tile = first_row + MAX_EXPERTS + 1;                                              // [E + 1]

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const uint32_t bar0 = smem_u32(&bars[0]);
  // group i of this pair's tiles, numbered through them: stage i % 4, phase i / 4; accumulator and operand i % depth
  auto full_bar = [&](uint32_t i) { return bar0 + 8u * (i % STAGES); };             // even CTA: group can be issued
  auto done_bar = [&](uint32_t i) { return bar0 + 8u * (STAGES + i % STAGES); };    // group accumulated
  auto parity = [](uint32_t i) { return (i / STAGES) & 1u; };
  auto cfull_bar = [&](int c) { return bar0 + 8u * (2 * STAGES + c); };             // codes and parameters landed
  auto cempty_bar = [&](int c) { return bar0 + 8u * (2 * STAGES + CSTAGES + c); };  // and read
  const uint32_t full0 = map_to_rank(bar0, 0);  // the even CTA's full_bar(0)
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 2 * CSTAGES), never_bar = drain_bar + 8u;
  const uint32_t smem_base = smem_u32(smem);
  auto x_tile = [&](uint32_t i) { return smem_base + (i % STAGES) * X_BYTES; };
  auto c_tile = [&](int c) { return smem_base + static_cast<uint32_t>(STAGES * X_BYTES + c * CSTAGE_BYTES); };

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1 + 2 * 4 + 2 * EPI_WARPS);  // TMA arm; both CTAs' unpackers of the group and scaling warps
      mbar_init(done_bar(s), 1);
    }
    for (int c = 0; c < CSTAGES; ++c) {
      mbar_init(cfull_bar(c), 1 + 32);      // TMA arm, and the copies of each lane of warp 3
      mbar_init(cempty_bar(c), DQ_WARPS + EPI_WARPS);
    }
    mbar_init(drain_bar, 1);
    mbar_init(never_bar, 1);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(&tmem_slot), TMEM_COLS);
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmX1);
    tma_prefetch_desc(&tmX2);
    tma_prefetch_desc(&tmX3);
    tma_prefetch_desc(&tmC);
  }
  // the table of tiles, with the rows clamped and rising, so that whatever stands in offsets no access leaves X and Y and
  // the tiles are as few as the host has counted
  for (int e = static_cast<int>(threadIdx.x); e <= p.E; e += THREADS)
    first_row[e] = min(max(p.offsets[e], 0), static_cast<int>(p.R));
  __syncthreads();
  if (warp == 2) {
    int carry = 0, most = 0;
    for (int e0 = 0; e0 <= p.E; e0 += 32) {  // running maximum
      const int e = e0 + lane;
      int row = e <= p.E ? first_row[e] : 0;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, row, d);
        if (lane >= d) row = max(row, o);
      }
      row = max(row, carry);
      if (e <= p.E) first_row[e] = row;
      carry = __shfl_sync(0xffffffffu, row, 31);
    }
    __syncwarp();
    carry = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      const int rows = e < p.E ? first_row[e + 1] - first_row[e] : 0;
      const int tiles = rows > few::TOKENS ? token_tiles(rows) * p.n_bands : 0;
      if (tiles > 0) most = max(most, min(rows, tile_rows(rows, token_tiles(rows))));
      int inc = tiles;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
      }
      if (e < p.E) first_tile[e] = carry + inc - tiles;
      carry += __shfl_sync(0xffffffffu, inc, 31);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
      first_tile[p.E] = carry;
      widest = most;
    }
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  DeviceStatus* st = p.status;
  const int pair = static_cast<int>(blockIdx.x >> 1);
  const int n_pairs = static_cast<int>(gridDim.x >> 1);
  const int num_tiles = first_tile[p.E];
  const int num_groups = static_cast<int>(p.G);
  const int num_slots = (num_groups + 1) / 2;
  // groups in flight, and the columns of each: an accumulator, then an operand buffer
  const uint32_t depth = widest > 96 ? 2u : widest > 64 ? 3u : 4u;
  const uint32_t acc_cols = widest > 96 ? BN : widest > 64 ? 96u : 64u, buf_cols = acc_cols + A_COLS;
  auto tile_at = [&](int t) { return tile_of(t, first_tile, first_row, p.E); };

  if (warp < FIRST_EPI) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(ROLE_REGS));
    if (warp == 0 && elect_one()) {
      // ------------------------------------------------------------------------------ TMA (token rows)
      uint32_t i = 0;
      const uint64_t pol = policy_evict_normal();
      bool ok = true;
      for (int t = pair; ok && t < num_tiles && status_code(st) == 0u; t += n_pairs) {
        const Tile tile = tile_at(t);
        const int half = static_cast<int>(tile.n() / 2);
        const int boxes = (half + X_BOX - 1) / X_BOX;
        const CUtensorMap* map = boxes == 1 ? &tmX1 : boxes == 2 ? &tmX2 : &tmX3;
        const uint32_t bytes = static_cast<uint32_t>(boxes * X_BOX * BK * 2 * 2 * 2);  // both halves, both CTAs
        const int32_t row = tile.row0 + static_cast<int32_t>(rank) * half;
        for (int g = 0; g < num_groups; ++g, ++i) {
          ok = i < STAGES || wait(done_bar(i), parity(i - STAGES), p, kSiteTmaEmpty);
          if (!ok) break;
          const uint32_t fb = full0 + 8u * (i % STAGES);
          if (rank == 0) mbar_arrive_expect_tx(full_bar(i), bytes);
          tma_load_2d_pair_hint(x_tile(i), map, g * 2 * BK, row, fb, pol);
          tma_load_2d_pair_hint(x_tile(i) + X_HALF_BYTES, map, g * 2 * BK + BK, row, fb, pol);
        }
      }
    } else if (warp == 1 && rank == 0 && elect_one()) {
      // ------------------------------------------------------------------------------ MMA (even CTA)
      uint32_t i = 0, buf = 0;
      const uint64_t desc0 = smem_desc_sw128(x_tile(0));
      bool ok = true;
      for (int t = pair; ok && t < num_tiles && status_code(st) == 0u; t += n_pairs) {
        const uint32_t idesc = idesc_bf16_f32(2 * HALF, tile_at(t).n());
        if (t == p.stall_tile) ok = wait(never_bar, 0u, p, kSiteMmaInjected);
        for (int g = 0; ok && g < num_groups; ++g, ++i) {
          ok = wait(full_bar(i), parity(i), p, kSiteMmaFull);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem_base + buf * buf_cols, a = d + acc_cols;
          if (++buf == depth) buf = 0;
          const uint64_t b = desc0 + (i % STAGES) * (X_BYTES >> 4);
#pragma unroll
          for (int kk = 0; kk < 2 * BK / UK; ++kk)  // 16 in-features: 8 columns of A, 32 bytes of B's rows
            umma_bf16_pair_ts(d, a + static_cast<uint32_t>(kk * UK / 2),
                              b + static_cast<uint64_t>(((kk >> 2) * X_HALF_BYTES + (kk & 3) * UK * 2) >> 4), idesc,
                              kk != 0 ? 1u : 0u);
          umma_commit_pair(done_bar(i), 0x3);
        }
      }
      umma_commit_pair(drain_bar, 0x1);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(drain_bar, 0u))
        if (global_timer_ns() - t0 > p.limit_ns) {
          raise_timeout(st, kSiteDrainMma);
          break;
        }
    } else if (warp == 2 && elect_one()) {
      // ------------------------------------------------------------------------------ TMA (codes)
      int slot = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = pair; ok && t < num_tiles && status_code(st) == 0u; t += n_pairs) {
        const Tile tile = tile_at(t);
        const int32_t w0 = tile.e * static_cast<int32_t>(p.O);
        for (int j = 0; j < num_slots; ++j) {
          ok = wait(cempty_bar(slot), phase ^ 1u, p, kSiteTmaProduced);
          if (!ok) break;
          mbar_arrive_expect_tx(cfull_bar(slot), C_BYTES);
          if (GATED) {
            const int32_t out0 = tile.band * HALF + static_cast<int32_t>(rank) * (HALF / 2);
            const int32_t up = static_cast<int32_t>(p.O / 2);
#pragma unroll
            for (int b = 0; b < 8; ++b)  // gate and up rows of 16 outputs in turn
              tma_load_2d(c_tile(slot) + static_cast<uint32_t>(b * 2048), &tmC, j * 32,
                          w0 + out0 + (b >> 1) * 16 + (b & 1) * up, cfull_bar(slot));
          } else {
            tma_load_2d(c_tile(slot), &tmC, j * 32, w0 + tile.band * 2 * HALF + static_cast<int32_t>(rank) * HALF,
                        cfull_bar(slot));
          }
          if (++slot == CSTAGES) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
    } else if (warp == 3) {
      // ------------------------------------------------------------------------------ steps and zero points
      int slot = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = pair; ok && t < num_tiles && warp_ok(st); t += n_pairs) {
        const Tile tile = tile_at(t);
        int64_t row[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = lane + 32 * i;
          int64_t o;  // rows past the end read the last row: what comes of them is not stored
          if (GATED)
            o = min(static_cast<int64_t>(tile.band) * HALF + rank * (HALF / 2) + i * 16 + (r & 15), p.O / 2 - 1) +
                ((r >> 4) & 1) * (p.O / 2);
          else
            o = min(static_cast<int64_t>(tile.band) * 2 * HALF + rank * HALF + r, p.O - 1);
          row[i] = (static_cast<int64_t>(tile.e) * p.O + o) * p.G;
        }
        for (int j = 0; j < num_slots; ++j) {
          ok = wait_warp(cempty_bar(slot), phase ^ 1u, p, kSiteTmaProduced);
          if (!ok) break;
          const int g = 2 * j;
          const uint32_t dst = c_tile(slot) + C_BYTES + static_cast<uint32_t>(lane * 8);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t d = dst + static_cast<uint32_t>(i * 256);
            if (p.pair_params) {
              few::cp_async8(d, p.steps + row[i] + g);
              few::cp_async8(d + P_BYTES, p.zeros + row[i] + g);
            } else {
              few::cp_async4(d, p.steps + row[i] + g);
              few::cp_async4(d + P_BYTES, p.zeros + row[i] + g);
              if (g + 1 < num_groups) {
                few::cp_async4(d + 4, p.steps + row[i] + g + 1);
                few::cp_async4(d + P_BYTES + 4, p.zeros + row[i] + g + 1);
              }
            }
          }
          cp_async_arrive(cfull_bar(slot));
          if (++slot == CSTAGES) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      few::cp_async_wait_all();
    }
    __syncwarp();
  } else if (warp >= FIRST_DQ) {
    // ------------------------------------------------------------------------------ unpackers
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(DQ_REGS));
    const int set = (warp - FIRST_DQ) / 4;  // takes the groups with g % 2 == set, a slot's first or second
    const int quarter = warp & 3;
    const int r = lane + 32 * quarter;      // the lane's row of the CTA's 128
    const uint32_t sw = static_cast<uint32_t>(r & 7);
    const uint32_t ta = tmem_base + acc_cols + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t first = c_tile(0) + static_cast<uint32_t>(r * 128);
    const uint32_t at0 = (static_cast<uint32_t>(4 * set) ^ sw) << 4, at1 = (static_cast<uint32_t>(4 * set + 1) ^ sw) << 4;
    const uint32_t at2 = (static_cast<uint32_t>(4 * set + 2) ^ sw) << 4, at3 = (static_cast<uint32_t>(4 * set + 3) ^ sw) << 4;
    const uint32_t zp = static_cast<uint32_t>(C_BYTES + P_BYTES + set * 4) - static_cast<uint32_t>(r * 120);  // from `line`
    int slot = 0;
    uint32_t phase = 0, i = 0;
    bool ok = true;
    for (int t = pair; ok && t < num_tiles && warp_ok(st); t += n_pairs) {
      uint32_t buf = (i + static_cast<uint32_t>(set)) % depth;
      uint32_t n = i + static_cast<uint32_t>(set);
      i += static_cast<uint32_t>(num_groups);
#pragma unroll 1
      for (int j = 0; j < num_slots; ++j) {
        ok = wait_warp(cfull_bar(slot), phase, p, kSiteTmaEmpty);
        if (!ok) break;
        if (n != i) {  // the last slot may hold one group
          const uint32_t line = first + static_cast<uint32_t>(slot * CSTAGE_BYTES);
          float z;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(z) : "r"(line + zp) : "memory");
          const bool far = __any_sync(0xffffffffu, !(fabsf(z) <= 240.0f));
          const __nv_bfloat162 zz = __float2bfloat162_rn(z * -0.015625f);
          const uint32_t zb = *reinterpret_cast<const uint32_t*>(&zz);
          const uint32_t to = ta + buf * buf_cols;
          buf += 2;
          if (buf >= depth) buf -= depth;
          uint32_t o[32];
          {
            const uint4 w0 = few::lds128(line + at0), w1 = few::lds128(line + at1);
            const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int c = 0; c < 8; ++c) unpack_word(w[c], zb, o + 4 * c);
          }
          const uint4 w0 = few::lds128(line + at2), w1 = few::lds128(line + at3);
          ok = n < depth || wait_warp(done_bar(n - depth), parity(n - depth), p, kSiteTmaProduced);
          if (!ok) break;
          tc_fence_after();  // the MMAs that read the buffer come before the stores below
          tmem_st32(to, o);
          {
            const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int c = 0; c < 8; ++c) unpack_word(w[c], zb, o + 4 * c);
          }
          tmem_st32(to + 32u, o);
          if (far) {  // the words again, eight columns at a time
            tmem_wait_st();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              const uint32_t at =
                  line + ((static_cast<uint32_t>(4 * set + (c >> 1)) ^ sw) << 4) + static_cast<uint32_t>((c & 1) * 8);
              uint32_t v[2], f[8];
              asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(at) : "memory");
#pragma unroll
              for (int k = 0; k < 8; ++k) f[k] = unpack_pair_any((v[k / 4] >> (8 * (k & 3))) & 0xFFu, z);
              tmem_st8(to + static_cast<uint32_t>(c * 8), f);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_pair(full0 + 8u * (n % STAGES));
          n += 2;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(cempty_bar(slot));
        if (++slot == CSTAGES) {
          slot = 0;
          phase ^= 1u;
        }
      }
    }
  } else {
    // ------------------------------------------------------------------------------ scaling and epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
    const int quarter = warp & 3, half = (warp - FIRST_EPI) / 4;
    const int r = lane + 32 * quarter;
    int slot = 0;
    const uint32_t c_first = c_tile(0) + C_BYTES + static_cast<uint32_t>(r * 8);
    const uint32_t ta0 = tmem_base + static_cast<uint32_t>(half * BLOCK) + (static_cast<uint32_t>(quarter * 32) << 16);
    uint32_t phase = 0, i = 0, buf = 0, ct = c_first, ta = ta0;
    int who = lane;  // the lane with 0 here arrives for the warp; -1 in a lane that has given up
    if (lane == 0)  // every accumulator is free
      for (uint32_t d = 0; d < depth; ++d) mbar_arrive_pair(map_to_rank(full_bar(d), 0));
    for (int t = pair; t < num_tiles && warp_ok(st); t += n_pairs) {
      const Tile tile = tile_at(t);
      const int blocks = (tile.tokens + BLOCK - 1) / BLOCK;
      const int mine = (blocks - half + 1) / 2;  // this warp's blocks: half, half + 2, ...
      uint64_t y[CHUNKS][BLOCK / 2];
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
        for (int k = 0; k < BLOCK / 2; ++k) y[c][k] = 0ull;
      // the tile's groups, for a warp with N blocks (one without any reads a block of no token): a test per block in the loop,
      // which also kept the accumulator's loads from being moved, cost a tile of 192 tokens a tenth of its time
      auto scale_groups = [&](auto blocks_c) {
        constexpr int N = decltype(blocks_c)::value;
        float2 steps = make_float2(0.0f, 0.0f);
#pragma unroll (N > 1 ? 1 : 2)
        for (int g = 0; g < num_groups; ++g, ++i) {
          if ((g & 1) == 0) {
            if (!wait(cfull_bar(slot), phase, p, kSiteTmaEmpty)) who = -1;
            steps = few::lds64f(ct);
            __syncwarp();
            if (who == 0) mbar_arrive(cempty_bar(slot));
            ct += CSTAGE_BYTES;
            if (++slot == CSTAGES) {
              slot = 0;
              ct = c_first;
              phase ^= 1u;
            }
          }
          const uint32_t s64 = __float_as_uint(((g & 1) ? steps.y : steps.x) * 64.0f);
          const uint64_t ss = f32x2_pack(s64, s64);
          if (!wait(done_bar(i), parity(i), p, kSiteEpiAccFull)) who = -1;
          __syncwarp();
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < N; ++c) {
            float v[BLOCK];  // columns past the tile's are of no token
            tmem_ld32(ta + static_cast<uint32_t>(c * 2 * BLOCK), v);
#pragma unroll
            for (int k = 0; k < BLOCK / 2; ++k) fma_f32x2(y[c][k], ss, __float_as_uint(v[2 * k]), __float_as_uint(v[2 * k + 1]));
          }
          tc_fence_before();
          __syncwarp();
          if (who == 0) mbar_arrive_pair(full0 + 8u * ((i + depth) % STAGES));  // the group that overwrites it
          ta += buf_cols;
          if (++buf == depth) {
            buf = 0;
            ta = ta0;
          }
        }
      };
      if (mine >= 3) scale_groups(std::integral_constant<int, 3>{});
      else if (mine == 2) scale_groups(std::integral_constant<int, 2>{});
      else scale_groups(std::integral_constant<int, 1>{});
      if (__any_sync(0xffffffffu, who < 0)) break;  // nothing of an unfinished tile is stored

      int64_t o, n_out;
      if (GATED) {
        n_out = p.O / 2;
        o = static_cast<int64_t>(tile.band) * HALF + rank * (HALF / 2) + quarter * 16 + (lane & 15);
      } else {
        n_out = p.O;
        o = static_cast<int64_t>(tile.band) * 2 * HALF + rank * HALF + quarter * 32 + lane;
      }
      const bool real = o < n_out;
      uint16_t* dst = p.Y + static_cast<int64_t>(tile.row0) * p.ldy + o;
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) {
        if (c >= mine) break;
        const int tok0 = (2 * c + half) * BLOCK;
#pragma unroll
        for (int k = 0; k < BLOCK / 2; ++k) {
          uint32_t lo, hi;
          asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(y[c][k]));
          if (GATED) {
            // lanes 0-15 hold the gate of both tokens of a pair, lanes 16-31 the up value: each half gets what it
            // lacks for one of the two tokens
            const bool low = lane < 16;
            const float other = __uint_as_float(__shfl_xor_sync(0xffffffffu, low ? hi : lo, 16));
            const float own = __uint_as_float(low ? lo : hi);
            const float out = few::silu(low ? own : other) * (low ? other : own);
            const int tok = tok0 + 2 * k + (low ? 0 : 1);
            const __nv_bfloat16 b = __float2bfloat16_rn(out);
            if (real && tok < tile.tokens) dst[tok * p.ldy] = *reinterpret_cast<const uint16_t*>(&b);
          } else {
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
            const uint32_t u = *reinterpret_cast<const uint32_t*>(&b);
            const int tok = tok0 + 2 * k;
            if (real && tok < tile.tokens) dst[tok * p.ldy] = static_cast<uint16_t>(u);
            if (real && tok + 1 < tile.tokens) dst[(tok + 1) * p.ldy] = static_cast<uint16_t>(u >> 16);
          }
        }
      }
    }
    __syncwarp();
  }

  // After a timeout: time for the copies in flight to land. A role that gave up has seen the status set, so it waits here, and
  // the pair ends together.
  if (!warp_ok(st)) {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 50000ull) __nanosleep(1000);
    __syncwarp();
  }
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
  // Launched while the few-token kernel's last CTAs run: what follows this kernel on the stream has to wait for both.
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace grp
}  // namespace awq
