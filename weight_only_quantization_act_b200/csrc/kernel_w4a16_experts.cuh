// kernel_w4a16_experts.cuh - products of many rows with their experts' packed 4-bit weights: Y[r] = X'[r] deq(W_e)^T
// for the sorted rows of each expert, optionally with the SiLU gate of a stacked gate and up projection in the
// epilogue. deq(W)[o, k] = bf16(RN32(RN32(q - z) * step)), as in the many-token kernel of w4a16_gemm; an expert with few
// rows is left to kernel_w4a16_few.cuh.
//
// The weights stand on the MMA's M side and the expert's tokens on its N side, whose width is set per tile: a tile
// is 256 weight rows (128 per CTA of a pair; gated: 128 outputs, their gate and up rows in turns of 16) times up to
// 256 tokens of one expert, N the tokens rounded up to 16, so a ragged expert wastes less than 16 columns of tensor
// work. Experts of more than 256 rows are cut into tiles of nearly equal width. A row of the accumulator is a weight
// row, so its lanes store consecutive outputs of one token and no store goes past an expert's last row.
//
// Bounds: at N = 256 a k-block of 64 in-features takes the tensor cores 512 cycles and the dequantization about
// 205 issue cycles of every SM quarter; below N = 100 the dequantization is the longer one, and it then consumes packed weights
// at about the rate that HBM delivers them (4 KB per SM in 205 cycles).
//
// Persistent, clusters of 2 CTAs, one CTA per SM; every CTA makes the table of tiles from the row offsets for
// itself and takes each n-th tile, so nothing is exchanged between pairs. Warps of a CTA:
//   0      TMA of this CTA's half of the tile's token rows (boxes of 32 rows x 64 in-features, 128-byte swizzle),
//          counted on the even CTA's barrier
//   1      tensor memory; the even CTA issues the pair MMAs (cta_group::2, M = 256, N, K = 16) into two
//          256-column accumulators in turn, so the epilogue of a tile overlaps the next one
//   2-5    epilogue
//   6      TMA of the code words, 128 rows x 256 in-features at a time (128 bytes of a row), into a ring of its own
//   7      steps and zero points of those rows and groups by cp.async, counted on the same barrier
//   8-23   dequantizers: warps 8 + 4 s .. 11 + 4 s fill operand stage s, a weight row per lane, and hold the result
//          in registers until the stage is free
// Every wait is bounded.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "dequant_w4.cuh"
#include "kernel_w4a16.cuh"
#include "kernel_w4a16_few.cuh"
#include "ptx.cuh"

namespace awq {
namespace grp {

constexpr int HALF = 128;                         // weight rows per CTA, and token rows per CTA at most
constexpr int BN = 256;                           // tokens per tile at most
constexpr int BK = 64;
constexpr int UK = 16;
constexpr int STAGES = 4;
constexpr int A_BYTES = HALF * BK * 2;            // 16 KB  dequantized weight rows
constexpr int X_BYTES = HALF * BK * 2;            // 16 KB  token rows
constexpr int STAGE_BYTES = A_BYTES + X_BYTES;
constexpr int X_BOX = 32;                         // token rows per TMA box
constexpr int X_BOX_BYTES = X_BOX * BK * 2;
constexpr int CSTAGES = 4;                        // code ring
constexpr int SLOT_KB = 4;                        // k-blocks per code slot: 32 words = 128 bytes of each row
constexpr int C_BYTES = HALF * 128;               // 16 KB  code words
constexpr int P_BYTES = HALF * 2 * 4;             // 1 KB   steps (zero points) of two groups
constexpr int CSTAGE_BYTES = C_BYTES + 2 * P_BYTES;
constexpr int DQ_WARPS = 4 * STAGES;
constexpr int FIRST_DQ = 8;
constexpr int THREADS = 32 * (FIRST_DQ + DQ_WARPS);
constexpr int MAX_EXPERTS = 1024;
constexpr int TABLE_BYTES = 2 * (MAX_EXPERTS + 1) * 4;
constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + CSTAGES * CSTAGE_BYTES + TABLE_BYTES + 1024;
constexpr uint32_t TMEM_COLS = 512;
static_assert(SMEM_BYTES <= 232448, "fits the 227 KB of dynamic shared memory");
static_assert(STAGE_BYTES % 1024 == 0 && CSTAGE_BYTES % 1024 == 0, "tiles stay 1024-byte aligned");
static_assert(SLOT_KB == STAGES, "each set of dequantizers has at most one k-block of a code slot");

struct Params {
  const int* offsets;      // [E + 1]
  const float* steps;      // [E][O][G]
  const float* zeros;
  uint16_t* Y;             // [R][ldy]
  int64_t R, O, G, ldy;
  int E;
  int min_rows;            // experts with fewer rows are left to another kernel
  int n_bands;             // tiles along the weight rows
  int num_kb;              // K / 64
  int pair_params;         // steps and zero points of two groups can be copied as 8 bytes
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
  return tiles >= 16 ? BN : ((rows + tiles - 1) / tiles + 15) & ~15;
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

template <bool GATED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    w4a16_experts_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmC, Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t bars[2 * STAGES + 2 * CSTAGES + 5];
  __shared__ uint32_t tmem_slot;
  int* first_row = reinterpret_cast<int*>(smem + STAGES * STAGE_BYTES + CSTAGES * CSTAGE_BYTES);  // [E + 1]
  int* first_tile = first_row + MAX_EXPERTS + 1;                                                   // [E + 1]

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const uint32_t bar0 = smem_u32(&bars[0]);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };                             // even CTA: operands ready
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };                 // MMAs done with stage
  auto cfull_bar = [&](int c) { return bar0 + 8u * (2 * STAGES + c); };             // codes and parameters landed
  auto cempty_bar = [&](int c) { return bar0 + 8u * (2 * STAGES + CSTAGES + c); };  // and read
  auto accf_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 * CSTAGES + a); };      // tile accumulated
  auto acce_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 * CSTAGES + 2 + a); };  // accumulator read
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 2 * CSTAGES + 4);
  const uint32_t smem_base = smem_u32(smem);
  auto a_tile = [&](int s) { return smem_base + static_cast<uint32_t>(s * STAGE_BYTES); };
  auto x_tile = [&](int s) { return a_tile(s) + A_BYTES; };
  auto c_tile = [&](int c) { return smem_base + static_cast<uint32_t>(STAGES * STAGE_BYTES + c * CSTAGE_BYTES); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1 + 2 * 4);    // TMA arm, and the stage's four dequantizer warps of both CTAs
      mbar_init(empty_bar(s), 1);
    }
    for (int c = 0; c < CSTAGES; ++c) {
      mbar_init(cfull_bar(c), 1 + 32);      // TMA arm, and the copies of each lane of warp 7
      mbar_init(cempty_bar(c), DQ_WARPS);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(accf_bar(a), 1);
      mbar_init(acce_bar(a), 8);            // 4 epilogue warps x 2 CTAs
    }
    mbar_init(drain_bar, 1);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(&tmem_slot), TMEM_COLS);
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmC);
  }
  // the table of tiles, with the rows clamped so that whatever stands in offsets no access leaves X and Y
  for (int e = static_cast<int>(threadIdx.x); e <= p.E; e += THREADS)
    first_row[e] = min(max(p.offsets[e], 0), static_cast<int>(p.R));
  __syncthreads();
  if (warp == 2) {
    int carry = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      const int rows = e < p.E ? max(first_row[e + 1] - first_row[e], 0) : 0;
      const int tiles = rows >= p.min_rows ? token_tiles(rows) * p.n_bands : 0;
      int inc = tiles;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
      }
      if (e < p.E) first_tile[e] = carry + inc - tiles;
      carry += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) first_tile[p.E] = carry;
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  DeviceStatus* st = p.status;
  const int pair = static_cast<int>(blockIdx.x >> 1);
  const int n_pairs = static_cast<int>(gridDim.x >> 1);
  const int num_tiles = first_tile[p.E];
  const int num_slots = (p.num_kb + SLOT_KB - 1) / SLOT_KB;
  auto tile_at = [&](int t) { return tile_of(t, first_tile, first_row, p.E); };

  if (warp == 0) {
    // ------------------------------------------------------------------------------ TMA (token rows)
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = pair; ok && t < num_tiles; t += n_pairs) {
        const Tile tile = tile_at(t);
        const int half = static_cast<int>(tile.n() / 2);
        const int boxes = (half + X_BOX - 1) / X_BOX;
        const int32_t row = tile.row0 + static_cast<int32_t>(rank) * half;
        for (int kb = 0; kb < p.num_kb; ++kb) {
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, st, p.limit_ns, kSiteTmaEmpty)) {
            ok = false;
            break;
          }
          const uint32_t fb = map_to_rank(full_bar(stage), 0);
          if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), static_cast<uint32_t>(2 * boxes * X_BOX_BYTES));
          const uint64_t pol = policy_evict_normal();
          for (int b = 0; b < boxes; ++b)
            tma_load_2d_pair_hint(x_tile(stage) + static_cast<uint32_t>(b * X_BOX_BYTES), &tmX, kb * BK, row + b * X_BOX,
                                  fb, pol);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------------------ MMA (even CTA)
    if (rank == 0 && elect_one()) {
      int stage = 0, i = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = pair; ok && t < num_tiles; t += n_pairs, ++i) {
        const uint32_t idesc = idesc_bf16_f32(2 * HALF, tile_at(t).n());
        const int acc = i & 1;
        if (i >= 2 && !mbar_wait(acce_bar(acc), static_cast<uint32_t>(i / 2 - 1) & 1u, st, p.limit_ns, kSiteMmaAccEmpty)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int kb = 0; kb < p.num_kb; ++kb) {
          if (!mbar_wait(full_bar(stage), phase, st, p.limit_ns, kSiteMmaFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < BK / UK; ++kk)
            umma_bf16_pair(tmem_base + static_cast<uint32_t>(acc * BN), smem_desc_sw128(a_tile(stage) + kk * UK * 2),
                           smem_desc_sw128(x_tile(stage) + kk * UK * 2), idesc, (kb | kk) != 0 ? 1u : 0u);
          umma_commit_pair(empty_bar(stage), 0x3);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit_pair(accf_bar(acc), 0x3);
      }
      umma_commit_pair(drain_bar, 0x1);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(drain_bar, 0u))
        if (global_timer_ns() - t0 > p.limit_ns) {
          raise_timeout(st, kSiteDrainMma);
          break;
        }
    }
    __syncwarp();
  } else if (warp == 6) {
    // ------------------------------------------------------------------------------ TMA (codes)
    if (elect_one()) {
      bool ok = true;
      int slot = 0;
      uint32_t phase = 0;
      for (int t = pair; ok && t < num_tiles; t += n_pairs) {
        const Tile tile = tile_at(t);
        const int32_t w0 = tile.e * static_cast<int32_t>(p.O);
        for (int j = 0; j < num_slots; ++j) {
          if (!mbar_wait(cempty_bar(slot), phase ^ 1u, st, p.limit_ns, kSiteTmaProduced)) {
            ok = false;
            break;
          }
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
    }
    __syncwarp();
  } else if (warp == 7) {
    // ------------------------------------------------------------------------------ steps and zero points
    bool ok = true;
    int slot = 0;
    uint32_t phase = 0;
    const int num_groups = p.num_kb / 2;
    for (int t = pair; ok && t < num_tiles; t += n_pairs) {
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
        if (!dq::warp_wait_any(cempty_bar(slot), phase ^ 1u, st, p.limit_ns, kSiteTmaProduced, false)) {
          ok = false;
          break;
        }
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
  } else if (warp >= FIRST_DQ) {
    // ------------------------------------------------------------------------------ dequantizers
    const int s_own = (warp - FIRST_DQ) / 4;
    const int r = lane + 32 * ((warp - FIRST_DQ) & 3);  // the lane's row of the CTA's 128
    bool ok = true;
    int slot = 0, use = 0, first = s_own;  // first: this set's k-block of the tile's first slot
    uint32_t phase = 0;
    for (int t = pair; ok && t < num_tiles; t += n_pairs) {
      for (int j = 0; j < num_slots; ++j) {
        if (!dq::warp_wait_any(cfull_bar(slot), phase, st, p.limit_ns, kSiteTmaEmpty, false)) {
          ok = false;
          break;
        }
        const bool mine = j * SLOT_KB + first < p.num_kb;
        uint32_t v[32];
        if (mine) {
          const uint32_t line = c_tile(slot) + static_cast<uint32_t>(r * 128);
          const uint32_t sw = static_cast<uint32_t>(r & 7);
          const uint4 w0 = few::lds128(line + (((2u * first) ^ sw) << 4));
          const uint4 w1 = few::lds128(line + (((2u * first + 1u) ^ sw) << 4));
          const uint32_t pa = c_tile(slot) + C_BYTES + static_cast<uint32_t>(r * 8 + (first >> 1) * 4);
          float stp, z;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(stp) : "r"(pa) : "memory");
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(z) : "r"(pa + P_BYTES) : "memory");
          const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
          dequant_words<8>(w, z, stp, v);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(cempty_bar(slot));
        if (++slot == CSTAGES) {
          slot = 0;
          phase ^= 1u;
        }
        if (!mine) continue;
        if (use > 0 && !dq::warp_wait_any(empty_bar(s_own), static_cast<uint32_t>(use - 1) & 1u, st, p.limit_ns,
                                          kSiteMmaFull, true)) {
          ok = false;
          break;
        }
        ++use;
        store_words_sw128<8>(v, a_tile(s_own) + static_cast<uint32_t>(r) * 128u, r, 0);
        fence_proxy_async_smem();  // the tensor cores read these bytes through the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(map_to_rank(full_bar(s_own), 0));
      }
      // k-blocks are numbered through the pair's tiles: stage = number % STAGES, so a tile whose k-blocks are
      // no multiple of STAGES moves the sets
      first = (first + SLOT_KB - p.num_kb % SLOT_KB) % SLOT_KB;
    }
  } else {
    // ------------------------------------------------------------------------------ epilogue
    const int quarter = warp & 3;
    int i = 0;
    for (int t = pair; t < num_tiles; t += n_pairs, ++i) {
      const Tile tile = tile_at(t);
      const int acc = i & 1;
      if (!dq::warp_wait_any(accf_bar(acc), static_cast<uint32_t>(i / 2) & 1u, st, p.limit_ns, kSiteEpiAccFull, false)) break;
      tc_fence_after();
      const uint32_t ta = tmem_base + static_cast<uint32_t>(acc * BN) + (static_cast<uint32_t>(quarter * 32) << 16);
      const int chunks = static_cast<int>(tile.n() / 16);
      int64_t o, n_out;
      if (GATED) {
        n_out = p.O / 2;
        o = static_cast<int64_t>(tile.band) * HALF + rank * (HALF / 2) + quarter * 16 + (lane & 15);
      } else {
        n_out = p.O;
        o = static_cast<int64_t>(tile.band) * 2 * HALF + rank * HALF + quarter * 32 + lane;
      }
      const bool real = o < n_out;
      uint16_t* y = p.Y + static_cast<int64_t>(tile.row0) * p.ldy + o;
      auto emit = [&](const uint32_t (&v)[16], int c) {
        if (GATED) {
          // lanes 0-15 hold the gate of both tokens of a pair, lanes 16-31 the up value: each half gets what it
          // lacks for one of the two tokens
          const bool low = lane < 16;
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            const float other = __uint_as_float(__shfl_xor_sync(0xffffffffu, low ? v[k + 1] : v[k], 16));
            const float own = __uint_as_float(low ? v[k] : v[k + 1]);
            const float out = few::silu(low ? own : other) * (low ? other : own);
            const int tok = c * 16 + k + (low ? 0 : 1);
            const __nv_bfloat16 b = __float2bfloat16_rn(out);
            if (real && tok < tile.tokens) y[tok * p.ldy] = *reinterpret_cast<const uint16_t*>(&b);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const __nv_bfloat16 b = __float2bfloat16_rn(__uint_as_float(v[k]));
            if (real && c * 16 + k < tile.tokens) y[(c * 16 + k) * p.ldy] = *reinterpret_cast<const uint16_t*>(&b);
          }
        }
      };
      uint32_t va[16], vb[16];
      dq::tmem_ld16_issue(ta, va);
      for (int c = 0; c < chunks; c += 2) {
        dq::tmem_wait_ld16(va);
        if (c + 1 < chunks) dq::tmem_ld16_issue(ta + static_cast<uint32_t>((c + 1) * 16), vb);
        emit(va, c);
        if (c + 1 < chunks) {
          dq::tmem_wait_ld16(vb);
          if (c + 2 < chunks) dq::tmem_ld16_issue(ta + static_cast<uint32_t>((c + 2) * 16), va);
          emit(vb, c + 1);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(map_to_rank(acce_bar(acc), 0));
    }
    __syncwarp();
  }

  if (status_code(st) != 0u) {  // after a timeout: give the copies in flight time to land
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 50000ull) __nanosleep(1000);
  }
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

}  // namespace grp
}  // namespace awq
