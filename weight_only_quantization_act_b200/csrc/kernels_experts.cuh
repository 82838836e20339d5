// kernels_experts.cuh - tokens sorted by expert and back: the counting sort of a router's picks, the gather
// of token rows into expert order (optionally divided by each expert's scales), the weighted sum back per
// token, and the gradients of both.
//
// A slot s = t * top_k + j is the j-th pick of token t. order[r] is the slot of sorted row r, pos[s] the row of
// slot s, -1 where a pick names no expert. Every kernel checks the index that it loads against the array
// that it indexes, so whatever stands in order, pos or offsets no access leaves the arguments.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

#include "dequant_w4.cuh"
#include "ptx.cuh"

namespace awq {
namespace ex {

constexpr int SORT_THREADS = 256;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_ITERS = 16;                                   // slots per lane and tile at most
constexpr int SORT_ALONE = SORT_THREADS * SORT_ITERS;            // 4096 slots: one CTA sorts these alone
constexpr int MAX_EXPERTS = 1024;
constexpr int SORT_MAX_BLOCKS = 256;

template <typename ID>
__device__ __forceinline__ int expert_of(const ID* ids, int64_t s, int64_t n, int E) {
  if (s >= n) return -1;
  const ID v = ids[s];
  return v >= 0 && v < static_cast<ID>(E) ? static_cast<int>(v) : -1;
}

// counts[b][e]: picks of expert e among block b's slots.
template <typename ID>
__global__ void __launch_bounds__(SORT_THREADS) expert_count_kernel(const ID* __restrict__ ids, int64_t n, int E,
                                                                    int64_t per_block, int* __restrict__ counts) {
  __shared__ int hist[MAX_EXPERTS];
  for (int e = threadIdx.x; e < E; e += SORT_THREADS) hist[e] = 0;
  __syncthreads();
  const int64_t begin = blockIdx.x * per_block, end = min(begin + per_block, n);
  for (int64_t s = begin + threadIdx.x; s < end; s += SORT_THREADS) {
    const int e = expert_of(ids, s, n, E);
    if (e >= 0) atomicAdd(&hist[e], 1);  // a count: the order of the additions does not show
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += SORT_THREADS) counts[static_cast<int64_t>(blockIdx.x) * E + e] = hist[e];
}

// Exclusive prefix sum of v[0..E-1] in place by the whole block (E <= 4 * SORT_THREADS); returns the total.
__device__ __forceinline__ int block_scan(int* v, int E, int* warp_sums) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int x[4], mine = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = threadIdx.x * 4 + i;
    x[i] = e < E ? v[e] : 0;
    mine += x[i];
  }
  int inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  int before = inc - mine, all = 0;
  for (int w = 0; w < SORT_WARPS; ++w) {
    if (w < warp) before += warp_sums[w];
    all += warp_sums[w];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = threadIdx.x * 4 + i;
    if (e < E) v[e] = before;
    before += x[i];
  }
  __syncthreads();
  return all;
}

// Stable counting sort. Block b places its slots; with counts == nullptr there is one block, which counts
// for itself. Inside a block the slots are taken in tiles of up to 4096; each warp takes an eighth of the tile, consecutive
// slots, 32 at a time, and a lane's rank among equal picks is the popcount of the match mask below it
// plus the warp's running count, so equal picks keep the order of their slots.
template <typename ID>
__global__ void __launch_bounds__(SORT_THREADS) expert_place_kernel(const ID* __restrict__ ids, int64_t n, int E,
                                                                    int64_t per_block, const int* __restrict__ counts,
                                                                    int* __restrict__ offsets, int* __restrict__ order,
                                                                    int* __restrict__ pos) {
  extern __shared__ int sort_smem[];
  int* base = sort_smem;               // [E] next row of each expert for this block
  int* whist = sort_smem + E;          // [SORT_WARPS][E]
  __shared__ int warp_sums[SORT_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t begin = blockIdx.x * per_block, end = min(begin + per_block, n);

  // all[e] over the blocks, into base, and before[e] over those before this one, into whist's first row: a warp takes every
  // eighth block's counts, 32 experts at a time
  if (counts != nullptr) {
    for (int e = threadIdx.x; e < E; e += SORT_THREADS) base[e] = whist[e] = 0;
    __syncthreads();
    for (int e = lane; e < E; e += 32) {
      int all = 0, before = 0;
#pragma unroll 8
      for (unsigned b = warp; b < gridDim.x; b += SORT_WARPS) {
        const int c = counts[static_cast<int64_t>(b) * E + e];
        all += c;
        before += b < blockIdx.x ? c : 0;
      }
      if (all != 0) atomicAdd(&base[e], all);  // counts: the order of the additions does not show
      if (before != 0) atomicAdd(&whist[e], before);
    }
  } else {
    for (int e = threadIdx.x; e < E; e += SORT_THREADS) base[e] = 0;
    __syncthreads();
    for (int64_t s = begin + threadIdx.x; s < end; s += SORT_THREADS) {
      const int e = expert_of(ids, s, n, E);
      if (e >= 0) atomicAdd(&base[e], 1);
    }
  }
  __syncthreads();
  const int routed = block_scan(base, E, warp_sums);
  if (blockIdx.x == 0) {
    for (int e = threadIdx.x; e < E; e += SORT_THREADS) offsets[e] = base[e];
    if (threadIdx.x == 0) offsets[E] = routed;
    __syncthreads();
  }
  if (counts != nullptr) {
    for (int e = threadIdx.x; e < E; e += SORT_THREADS) base[e] += whist[e];
    __syncthreads();
  }

  const int iters = static_cast<int>(min((per_block + SORT_THREADS - 1) / SORT_THREADS, static_cast<int64_t>(SORT_ITERS)));
  for (int64_t tile = begin; tile < end; tile += iters * SORT_THREADS) {
    for (int i = threadIdx.x; i < SORT_WARPS * E; i += SORT_THREADS) whist[i] = 0;
    __syncthreads();
    int* mine = whist + warp * E;
    int ranks[SORT_ITERS], picks[SORT_ITERS];
    const int64_t s0 = tile + warp * 32 * iters + lane;
#pragma unroll
    for (int i = 0; i < SORT_ITERS; ++i) {
      if (i >= iters) break;
      const int64_t s = s0 + i * 32;
      const int e = expert_of(ids, s, end, E);
      const unsigned same = __match_any_sync(0xffffffffu, e);
      const int below = __popc(same & ((1u << lane) - 1u));
      picks[i] = e;
      ranks[i] = e >= 0 ? mine[e] + below : 0;
      __syncwarp();
      if (e >= 0 && below == 0) mine[e] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    // each warp's first row of each expert; the next tile starts behind this one
    for (int e = threadIdx.x; e < E; e += SORT_THREADS) {
      int at = base[e];
#pragma unroll
      for (int w = 0; w < SORT_WARPS; ++w) {
        const int c = whist[w * E + e];
        whist[w * E + e] = at;
        at += c;
      }
      base[e] = at;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < SORT_ITERS; ++i) {
      const int64_t s = s0 + i * 32;
      if (i < iters && s < end) {
        const int row = picks[i] >= 0 ? mine[picks[i]] + ranks[i] : -1;
        pos[s] = row;
        if (row >= 0) order[row] = static_cast<int>(s);
        if (s >= routed) order[s] = -1;  // rows behind the last: no slot writes them
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------------------------------------ rows
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  f[0] = __uint_as_float(v.x << 16); f[1] = __uint_as_float(v.x & 0xFFFF0000u);
  f[2] = __uint_as_float(v.y << 16); f[3] = __uint_as_float(v.y & 0xFFFF0000u);
  f[4] = __uint_as_float(v.z << 16); f[5] = __uint_as_float(v.z & 0xFFFF0000u);
  f[6] = __uint_as_float(v.w << 16); f[7] = __uint_as_float(v.w & 0xFFFF0000u);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    r[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// The expert whose rows hold `row`: the last e with first[e] <= row; `first` in shared memory, where a step of the search
// takes a tenth of its time in L2.
__device__ __forceinline__ int expert_of_row(const int* first, int E, int row) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= row) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The row kernels are bound by HBM: a thread keeps several 16-byte loads in flight, the threads of a block neighbours.
constexpr int ROW_THREADS = 128;
constexpr int AT_ONCE = 4;                                       // 16-byte pieces of a row per thread and turn
constexpr int ROW_PIECES = ROW_THREADS * AT_ONCE;                // 4096 columns a turn

__device__ __forceinline__ uint4 ld_row(const uint16_t* row, int64_t piece) {
  return __ldg(reinterpret_cast<const uint4*>(row) + piece);
}

// Xs[r] = X[order[r] / top_k]: a row per block.
__global__ void __launch_bounds__(ROW_THREADS) expert_gather_kernel(const uint16_t* __restrict__ X, int64_t ldx, int64_t T,
                                                                    int64_t K, const int* __restrict__ order, int top_k,
                                                                    uint16_t* __restrict__ Xs, int64_t ldxs) {
  const int64_t r = blockIdx.x;
  const int slot = order[r];
  if (slot < 0 || slot >= T * top_k) return;
  const uint16_t* src = X + static_cast<int64_t>(slot / top_k) * ldx;
  uint4* dst = reinterpret_cast<uint4*>(Xs + r * ldxs);
  const int64_t pieces = K / 8;
  for (int64_t c = threadIdx.x; c < pieces; c += ROW_PIECES) {
    uint4 v[AT_ONCE];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i)
      if (c + i * ROW_THREADS < pieces) v[i] = ld_row(src, c + i * ROW_THREADS);
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i)
      if (c + i * ROW_THREADS < pieces) dst[c + i * ROW_THREADS] = v[i];
  }
}

__device__ __forceinline__ uint64_t f32x2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Xs[r] = bf16(RN32(X[order[r] / top_k] / s)), s the scale of r's expert: a block takes a run of sorted rows, most of them of
// one expert, and 1024 columns, so a thread reads its 8 scales once per expert and not once per row (the scales of a row
// are twice its bytes).
// Division-free but for 1 of 4000 elements: with r = RN32(1 / s) a normal number, r- = RN32(r (1 - 2^-22)) and r+ =
// RN32(r (1 + 2^-22)) enclose 1 / s, so RN32(x r-) and RN32(x r+) enclose RN32(x / s) (rounding keeps order), and where both
// round to the same bf16 that is the result. Where they do not, the division decides. (8 divisions per 16 bytes, or a test of
// every quotient's low bits, took twice the time that the rows take from HBM.)
// Measured (B200): 65536 rows of 4096 columns for 128 experts with the sort in 128 us, 4.4 TB/s; this kernel 113, with 57 % of
// DRAM's rate and 2.1 of 4 instructions per cycle, so bound by neither: its warps (40 % of what an SM holds) wait for their
// loads. With a row's address and expert made by every thread 161, with 8 rows in flight (96 registers) 181, runs of 64
// rows the same.
constexpr int RUN = 32;
__global__ void __launch_bounds__(ROW_THREADS) expert_gather_scaled_kernel(
    const uint16_t* __restrict__ X, int64_t ldx, int64_t T, int64_t K, const int* __restrict__ offsets, int E,
    const int* __restrict__ order, int top_k, const float* __restrict__ scales, uint16_t* __restrict__ Xs, int64_t ldxs,
    int64_t n_rows) {
  __shared__ const uint16_t* rows[RUN];  // of X; null where no slot stands
  __shared__ __align__(16) int experts[RUN];
  __shared__ int first[MAX_EXPERTS];
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * RUN;
  for (int e = threadIdx.x; e < E; e += ROW_THREADS) first[e] = __ldg(offsets + e);
  int my_slot = -1;
  if (threadIdx.x < RUN && r0 + threadIdx.x < n_rows) my_slot = __ldg(order + r0 + threadIdx.x);
  __syncthreads();
  if (threadIdx.x < RUN) {
    const bool real = my_slot >= 0 && my_slot < T * top_k;
    rows[threadIdx.x] = real ? X + static_cast<int64_t>(my_slot / top_k) * ldx : nullptr;
    experts[threadIdx.x] = real ? expert_of_row(first, E, static_cast<int>(r0 + threadIdx.x)) : -1;
  }
  __syncthreads();
  const int64_t c = static_cast<int64_t>(blockIdx.y) * ROW_THREADS + threadIdx.x;
  if (c >= K / 8) return;
  uint64_t below[4], above[4];  // r- and r+ of two columns each
  const float* sc = nullptr;    // the expert's scales
  bool divide = false;          // a scale whose reciprocal is no normal number
  int have = -1;
  uint16_t* dst = Xs + r0 * ldxs + c * 8;
#pragma unroll 1
  for (int i0 = 0; i0 < RUN; i0 += AT_ONCE) {
    const int4 es = *reinterpret_cast<const int4*>(experts + i0);
    uint4 v[AT_ONCE];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i)
      if (rows[i0 + i] != nullptr) v[i] = ld_row(rows[i0 + i], c);
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i, dst += ldxs) {
      const int e = i == 0 ? es.x : i == 1 ? es.y : i == 2 ? es.z : es.w;
      if (e < 0) continue;
      if (e != have) {
        have = e;
        divide = false;
        sc = scales + e * K + c * 8;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 two = __ldg(reinterpret_cast<const float2*>(sc) + k);
          const float ra = __fdiv_rn(1.0f, two.x), rb = __fdiv_rn(1.0f, two.y);
          divide |= !(fabsf(ra) >= 2.0e-38f && fabsf(ra) <= 3.0e38f && fabsf(rb) >= 2.0e-38f && fabsf(rb) <= 3.0e38f);
          below[k] = f32x2_pack(__float_as_uint(ra * (1.0f - 0x1p-22f)), __float_as_uint(rb * (1.0f - 0x1p-22f)));
          above[k] = f32x2_pack(__float_as_uint(ra * (1.0f + 0x1p-22f)), __float_as_uint(rb * (1.0f + 0x1p-22f)));
        }
      }
      const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint32_t q[4], differ = divide ? 1u : 0u;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint64_t two = f32x2_pack(x[k] << 16, x[k] & 0xFFFF0000u);
        q[k] = f32x2_to_bf16x2(f32x2_mul(two, below[k]));
        differ |= q[k] ^ f32x2_to_bf16x2(f32x2_mul(two, above[k]));
      }
      if (differ != 0u) {
        float f[8];
        unpack8(v[i], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = __fdiv_rn(f[k], __ldg(sc + k));
        const uint4 exact = pack8(f);
        q[0] = exact.x;
        q[1] = exact.y;
        q[2] = exact.z;
        q[3] = exact.w;
      }
      *reinterpret_cast<uint4*>(dst) = make_uint4(q[0], q[1], q[2], q[3]);
    }
  }
}

// Y[t] = sum over token t's routed slots, in slot order, of weight * Ys[pos], in fp32: a token per block, the rows of four
// slots on their way at once.
__global__ void __launch_bounds__(ROW_THREADS) expert_combine_kernel(const uint16_t* __restrict__ Ys, int64_t ldys, int64_t K,
                                                                     const int* __restrict__ pos, int top_k, int64_t n_rows,
                                                                     const float* __restrict__ weights,
                                                                     uint16_t* __restrict__ Y, int64_t ldy) {
  constexpr int SLOTS = 4, PIECES = 2;
  const int64_t t = blockIdx.x, pieces = K / 8;
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * (ROW_THREADS * PIECES) + threadIdx.x;
  float acc[PIECES][8];
#pragma unroll
  for (int i = 0; i < PIECES; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[i][k] = 0.0f;
  for (int j0 = 0; j0 < top_k; j0 += SLOTS) {
    int row[SLOTS];
    float w[SLOTS];
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
      const int64_t s = t * top_k + j0 + j;
      row[j] = j0 + j < top_k ? __ldg(pos + s) : -1;
      if (row[j] >= n_rows) row[j] = -1;
      w[j] = weights != nullptr && j0 + j < top_k ? __ldg(weights + s) : 1.0f;
    }
    uint4 v[SLOTS][PIECES];
#pragma unroll
    for (int j = 0; j < SLOTS; ++j)
#pragma unroll
      for (int i = 0; i < PIECES; ++i)
        if (row[j] >= 0 && c0 + i * ROW_THREADS < pieces) v[j][i] = ld_row(Ys + row[j] * ldys, c0 + i * ROW_THREADS);
#pragma unroll
    for (int j = 0; j < SLOTS; ++j)
#pragma unroll
      for (int i = 0; i < PIECES; ++i)
        if (row[j] >= 0 && c0 + i * ROW_THREADS < pieces) {
          float f[8];
          unpack8(v[j][i], f);
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[i][k] = fmaf(w[j], f[k], acc[i][k]);
        }
  }
#pragma unroll
  for (int i = 0; i < PIECES; ++i)
    if (c0 + i * ROW_THREADS < pieces)
      reinterpret_cast<uint4*>(Y + t * ldy)[c0 + i * ROW_THREADS] = pack8(acc[i]);
}

// The same with Ys[pos] / scales[expert] for weight * Ys[pos]: the gradient of the scaled gather.
__global__ void __launch_bounds__(ROW_THREADS) expert_combine_scaled_kernel(
    const uint16_t* __restrict__ Ys, int64_t ldys, int64_t K, const int* __restrict__ pos, int top_k, int64_t n_rows,
    const int* __restrict__ offsets, int E, const float* __restrict__ scales, uint16_t* __restrict__ Y, int64_t ldy) {
  __shared__ int rows[ROW_THREADS], experts[ROW_THREADS], first[MAX_EXPERTS];
  const int64_t t = blockIdx.x;
  for (int e = threadIdx.x; e < E; e += ROW_THREADS) first[e] = __ldg(offsets + e);
  const int64_t c = static_cast<int64_t>(blockIdx.y) * ROW_THREADS + threadIdx.x;
  float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  for (int j0 = 0; j0 < top_k; j0 += ROW_THREADS) {
    const int n = min(top_k - j0, ROW_THREADS);
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < n) {
      const int row = pos[t * top_k + j0 + threadIdx.x];
      const bool real = row >= 0 && row < n_rows;
      rows[threadIdx.x] = real ? row : -1;
      experts[threadIdx.x] = real ? expert_of_row(first, E, row) : -1;
    }
    __syncthreads();
    if (c >= K / 8) continue;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      if (rows[j] < 0) continue;
      float f[8];
      unpack8(ld_row(Ys + rows[j] * ldys, c), f);
      const float4* sc = reinterpret_cast<const float4*>(scales + experts[j] * K + c * 8);
      const float4 lo = __ldg(sc), hi = __ldg(sc + 1);
      acc[0] += __fdiv_rn(f[0], lo.x); acc[1] += __fdiv_rn(f[1], lo.y);
      acc[2] += __fdiv_rn(f[2], lo.z); acc[3] += __fdiv_rn(f[3], lo.w);
      acc[4] += __fdiv_rn(f[4], hi.x); acc[5] += __fdiv_rn(f[5], hi.y);
      acc[6] += __fdiv_rn(f[6], hi.z); acc[7] += __fdiv_rn(f[7], hi.w);
    }
  }
  if (c < K / 8) reinterpret_cast<uint4*>(Y + t * ldy)[c] = pack8(acc);
}

// dYs[pos] = weight * dY[t], dweights = <dY[t], Ys[pos]> in fp32 (fixed order: a thread's columns in order, then
// the warp's butterfly, then the warps in order), 0 for slots without a row. One block per slot.
__global__ void __launch_bounds__(ROW_THREADS) expert_combine_backward_kernel(
    const uint16_t* __restrict__ dY, int64_t lddy, const uint16_t* __restrict__ Ys, int64_t ldys, int64_t K,
    const int* __restrict__ pos, int top_k, int64_t n_rows, const float* __restrict__ weights, uint16_t* __restrict__ dYs,
    int64_t lddys, float* __restrict__ dweights) {
  __shared__ float sums[ROW_THREADS / 32];
  const int64_t s = blockIdx.x, t = s / top_k, pieces = K / 8;
  const int row = pos[s];
  if (row < 0 || row >= n_rows) {
    if (threadIdx.x == 0) dweights[s] = 0.0f;
    return;
  }
  const float w = weights[s];
  const uint16_t* g_row = dY + t * lddy;
  const uint16_t* y_row = Ys + row * ldys;
  uint4* dst = reinterpret_cast<uint4*>(dYs + row * lddys);
  float dot = 0.0f;
  for (int64_t c = threadIdx.x; c < pieces; c += ROW_PIECES) {
    uint4 vg[AT_ONCE], vy[AT_ONCE];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i)
      if (c + i * ROW_THREADS < pieces) {
        vy[i] = ld_row(y_row, c + i * ROW_THREADS);
        vg[i] = ld_row(g_row, c + i * ROW_THREADS);
      }
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i)
      if (c + i * ROW_THREADS < pieces) {
        float g[8], y[8];
        unpack8(vg[i], g);
        unpack8(vy[i], y);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          dot = fmaf(g[k], y[k], dot);
          g[k] *= w;
        }
        dst[c + i * ROW_THREADS] = pack8(g);
      }
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) dot += __shfl_xor_sync(0xffffffffu, dot, d);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = dot;
  __syncthreads();
  if (threadIdx.x == 0) {
    float v = 0.0f;
    for (int i = 0; i < ROW_THREADS / 32; ++i) v += sums[i];
    dweights[s] = v;
  }
}

}  // namespace ex
}  // namespace awq
