// kernel_w4a16_few.cuh - products of a few tokens with packed 4-bit weights, for one layer or for the rows
// of each expert: Y = X' deq(W)^T, optionally with a bias or with the SiLU gate of a stacked gate and up
// projection in the epilogue.
//
// Mathematics: per group g of 128 in-features and token m, with a power of two c[m, g] that brings the group's largest
// |x'| to 2^14..2^15 and xs = c x',
//   Y[m, o] = sum_g step[o, g] / c[m, g] (sum_{k in g} q[o, k] xs[m, k] - z[o, g] sum_{k in g} xs[m, k]).
// A nibble in place under the exponent bits of 1024 is the fp16 number 1024 + q (bits 0-3) or 1024 + 16 q (bits
// 4-7), so one AND-OR per two codes and one shift per eight make the operand. In-features of the second kind
// enter as xs / 16, which makes that operand 64 + q, and what the constants add, 1024 or 64 times sums of xs, is
// subtracted per group and token. xs is exact in fp16 down to 2^-27 of the group's largest value and below
// that off by 2^-39 of it, so the weights enter with their exact value; the tensor cores sum in fp32, the
// step and zero point are applied once per group and output in fp32. (bf16 patterns 128 + q need a shift for
// every pair of codes: the ALU pipe, at half rate, then took longer than the loads.)
//
// The bound is HBM: a weight is read once and used for at most 8 tokens (0.5 byte per 16 operations), so
// what matters is bytes in flight and few instructions per weight. A one-token product cannot fill the
// tcgen05 tile (N >= 16 with operands staged in tensor or shared memory and a barrier per group), whose
// hand-offs bound the few-token kernel of w4a16_gemm; a warp-level MMA takes its A operand from the registers
// that unpacked it.
//
// A CTA of 8 warps owns 128 weight rows (gated: 64 gate rows and the 64 up rows of the same outputs) and a
// slice of the groups; each warp owns 16 rows. A lane copies the 16-byte pieces that it will itself unpack
// (row l / 4 and row l / 4 + 8, 32 codes of a group each) into its own ring in shared memory with cp.async, so
// the codes need no barrier at all. Both MMA operands name the in-features of a group in the order that the
// unpacking gives, so X is permuted once, on its way into shared memory. The slices of a row block are the
// CTAs of one cluster (at most 8), which add their fp32 partial sums through distributed shared memory in
// slice order: one launch, no workspace, the same result every time.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace awq {
namespace few {

constexpr int WARPS = 8;
constexpr int THREADS = 32 * WARPS;
constexpr int ROWS = 16 * WARPS;                       // weight rows per CTA
constexpr int TOKENS = 8;                              // tokens per pass over the weights
constexpr int UNIT = 2;                                // groups per ring stage
constexpr int DEPTH = 4;                               // ring stages
constexpr int CODE_BYTES = 16 * UNIT * 64;             // a warp's codes of one stage: 16 rows x 2 groups
constexpr int STAGE_BYTES = CODE_BYTES + 16 * UNIT * 8;  // and their steps and zero points
constexpr int RING_BYTES = WARPS * DEPTH * STAGE_BYTES;
constexpr int PART_LD = ROWS + 4;                      // partial sums [TOKENS][PART_LD]
constexpr int PART_BYTES = TOKENS * PART_LD * 4;
constexpr int X_MAX_BYTES = 57344;                     // X of one chunk of groups: 28 groups of 8 tokens
constexpr int MAX_SLICES = 8;                          // portable cluster size

// Shared memory for chunks of `xg` groups of `mp` tokens (mp = 1, 2, 4 or 8).
__host__ __device__ constexpr int smem_bytes(int xg, int mp) {
  return RING_BYTES + PART_BYTES + xg * 256 * mp + xg * TOKENS * 16;
}
constexpr int SMEM_MAX = smem_bytes(X_MAX_BYTES / 256, 1);
static_assert(SMEM_MAX >= smem_bytes(X_MAX_BYTES / 2048, 8), "one token's groups take the most sums");

struct Params {
  const uint16_t* X;        // [R][ldx] bf16
  const uint32_t* codes;    // [E][O][K / 8]
  const float* steps;       // [E][O][G]
  const float* zeros;       // [E][O][G]
  const uint16_t* bias;     // [O] bf16 or null
  const int* offsets;       // [E + 1] first row of each expert, or null: one layer, rows 0..R-1
  uint16_t* Y;              // [R][ldy] bf16
  int64_t R, ldx, ldy, O, K, G;
  int max_rows;             // experts with more rows are left to another kernel
  int g_per;                // groups per slice, even
  int xg;                   // groups per X chunk, even
  int mp_log2;              // log2 of the tokens that the X chunk has room for
  int pair_params;          // steps and zero points of two groups can be copied as 8 bytes
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float2 lds64f(uint32_t a) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t cluster_addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
  return v;
}
// c (16 x 8 fp32) += a (16 x 16 fp16) b (16 x 8 fp16)
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// Codes 0 and 4 of a word as fp16 (1024 + q); codes 1 and 5 as 1024 + 16 q. The other four: the same of w >> 8.
__device__ __forceinline__ uint32_t code_even(uint32_t w) { return (w & 0x000F000Fu) | 0x64006400u; }
__device__ __forceinline__ uint32_t code_odd(uint32_t w) { return (w & 0x00F000F0u) | 0x64006400u; }
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
// a / (1 + exp(-a)) for a result that is rounded to bf16: the fast exponential is off by (2 + |a|) units of 2^-23 and the fast
// quotient by 2 of its own, a bf16 step is 2^-8.
__device__ __forceinline__ float silu(float a) { return __fdividef(a, 1.0f + __expf(-a)); }

template <bool GATED>
__global__ void __launch_bounds__(THREADS) w4a16_few_kernel(const Params p) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g8 = lane >> 2, t4 = lane & 3;
  const int slice = static_cast<int>(blockIdx.x), slices = static_cast<int>(gridDim.x);
  const int64_t e = blockIdx.z;

  int64_t row0 = 0, rows = p.R;
  if (p.offsets != nullptr) {  // clamped, so that whatever stands there no access leaves X and Y
    row0 = min(max(static_cast<int64_t>(p.offsets[e]), int64_t(0)), p.R);
    rows = min(max(static_cast<int64_t>(p.offsets[e + 1]), row0), p.R) - row0;
  }
  if (rows == 0 || rows > p.max_rows) return;  // the same for every CTA of the cluster

  const int64_t n_out = GATED ? p.O / 2 : p.O;
  constexpr int OUT_ROWS = GATED ? ROWS / 2 : ROWS;
  const int64_t out0 = static_cast<int64_t>(blockIdx.y) * OUT_ROWS;
  // weight row of this warp's tile row r (0..15); rows past the end read the last row and are not stored
  auto weight_row = [&](int r) -> int64_t {
    if (GATED) return min(out0 + warp * 8 + (r & 7), n_out - 1) + (r >> 3) * n_out;
    return min(out0 + warp * 16 + r, n_out - 1);
  };

  const int g_begin = slice * p.g_per;
  const int g_end = min(g_begin + p.g_per, static_cast<int>(p.G));
  const int n_groups = max(g_end - g_begin, 0);
  const int n_units = (n_groups + UNIT - 1) / UNIT;

  const uint8_t* ring_ptr = smem + warp * DEPTH * STAGE_BYTES;
  const uint32_t ring = smem_u32(ring_ptr);
  float* part = reinterpret_cast<float*>(smem + RING_BYTES);
  uint8_t* xs = smem + RING_BYTES + PART_BYTES;                      // [group][word][token][t4] 16 bytes
  // [group][TOKENS]: what the constants add, the sum of xs, 1 / c
  float4* sx = reinterpret_cast<float4*>(xs + (p.xg * 256 << p.mp_log2));
  const int mp = 1 << p.mp_log2;

  const int64_t words = p.K / 8;
  const uint32_t* code_lo = p.codes + (e * p.O + weight_row(g8)) * words + t4 * 4 + g_begin * 16;
  const uint32_t* code_hi = p.codes + (e * p.O + weight_row(g8 + 8)) * words + t4 * 4 + g_begin * 16;
  const float* param = (lane < 16 ? p.steps : p.zeros) + (e * p.O + weight_row(lane & 15)) * p.G + g_begin;

  // copies of unit u into the slot at byte `at` of the ring
  auto issue = [&](int u, uint32_t at) {
    if (u < n_units) {
      const uint32_t dst = ring + at + static_cast<uint32_t>(lane * 16);
      const uint32_t* lo = code_lo + u * (UNIT * 16);
      const uint32_t* hi = code_hi + u * (UNIT * 16);
      const float* src = param + u * UNIT;
      const uint32_t pd = ring + at + CODE_BYTES + static_cast<uint32_t>(lane * 8);
      cp_async16(dst, lo);
      cp_async16(dst + 512u, hi);
      if (UNIT * u + 1 < n_groups) {
        cp_async16(dst + 1024u, lo + 16);
        cp_async16(dst + 1536u, hi + 16);
        if (p.pair_params) {
          cp_async8(pd, src);
        } else {
          cp_async4(pd, src);
          cp_async4(pd + 4u, src + 1);
        }
      } else {
        cp_async4(pd, src);
      }
    }
    cp_async_commit();
  };

  // X of tokens m0..m0+mt-1 and groups gc..gc+ng-1 as fp16, scaled and permuted so that one 16-byte piece (in-features
  // 8w..8w+7) holds the pairs (0, 4), (1, 5) / 16, (2, 6), (3, 7) / 16, and the sums of each token's groups. The 16 threads
  // of a token's group are neighbours.
  auto stage_x = [&](int64_t m0, int mt, int gc, int ng) {
    const int per_token = ng * 16;
    const int total = per_token * mt;
    for (int base = 0; base < total; base += THREADS) {
      const int i = base + static_cast<int>(threadIdx.x);
      const bool real = i < total;
      const int m = i / per_token, c = i - m * per_token;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (real) v = *reinterpret_cast<const uint4*>(p.X + (row0 + m0 + m) * p.ldx + static_cast<int64_t>(gc) * 128 + c * 8);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t most = 0u;  // exponent bits of the group's largest value
#pragma unroll
      for (int k = 0; k < 4; ++k) most = max(most, max(w[k] & 0x7F80u, (w[k] >> 16) & 0x7F80u));
#pragma unroll
      for (int d = 1; d < 16; d *= 2) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
      // c = 2^(14 - exponent), kept below 2^127 so that 1 / c is a normal number
      const uint32_t field = min(268u - (most >> 7), 253u);
      const float scale = __uint_as_float(field << 23), back = __uint_as_float((254u - field) << 23);
      __half2 h[4];  // pairs (0, 4), (1, 5) / 16, (2, 6), (3, 7) / 16
      const float s16 = scale * 0.0625f;
      h[0] = __floats2half2_rn(bf16_lo(v.x) * scale, bf16_lo(v.z) * scale);
      h[1] = __floats2half2_rn(bf16_hi(v.x) * s16, bf16_hi(v.z) * s16);
      h[2] = __floats2half2_rn(bf16_lo(v.y) * scale, bf16_lo(v.w) * scale);
      h[3] = __floats2half2_rn(bf16_hi(v.y) * s16, bf16_hi(v.w) * s16);
      const float2 f0 = __half22float2(h[0]), f1 = __half22float2(h[1]), f2 = __half22float2(h[2]), f3 = __half22float2(h[3]);
      float even = (f0.x + f0.y) + (f2.x + f2.y), odd = 16.0f * ((f1.x + f1.y) + (f3.x + f3.y));
#pragma unroll
      for (int d = 1; d < 16; d *= 2) {
        even += __shfl_xor_sync(0xffffffffu, even, d);
        odd += __shfl_xor_sync(0xffffffffu, odd, d);
      }
      if (real) {
        const int grp = c >> 4, t = (c >> 2) & 3, word = c & 3;
        *reinterpret_cast<uint4*>(xs + (((grp * 4 + word) * mp + m) * 4 + t) * 16) = *reinterpret_cast<const uint4*>(h);
        if ((c & 15) == 0) sx[grp * TOKENS + m] = make_float4(fmaf(1024.0f, even, 64.0f * odd), even + odd, back, 0.0f);
      }
    }
  };

  for (int64_t m0 = 0; m0 < rows; m0 += TOKENS) {
    const int mt = static_cast<int>(min(rows - m0, static_cast<int64_t>(TOKENS)));
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < DEPTH - 1; ++u) issue(u, static_cast<uint32_t>(u * STAGE_BYTES));
    uint32_t at = 0u, ahead = (DEPTH - 1) * STAGE_BYTES;  // slots of unit u and of unit u + DEPTH - 1
    // lanes of tokens past mp read another token's piece: their columns are never stored
    const uint8_t* x_lane = xs + ((((g8 & (mp - 1)) * 4) + t4) * 16);
    int chunk_end = 0, chunk0 = 0;
    for (int u = 0; u < n_units; ++u) {
      if (UNIT * u >= chunk_end) {
        chunk0 = UNIT * u;
        chunk_end = min(chunk0 + p.xg, n_groups);
        __syncthreads();  // the previous chunk has been read
        stage_x(m0, mt, g_begin + chunk0, chunk_end - chunk0);
        __syncthreads();
      }
      cp_async_wait<DEPTH - 2>();
      __syncwarp();  // the stage's steps and zero points, copied by other lanes, and the slot of unit u - 1 read
      issue(u + DEPTH - 1, ahead);
      const uint8_t* slot = ring_ptr + at;
      at = at == (DEPTH - 1) * STAGE_BYTES ? 0u : at + STAGE_BYTES;
      ahead = ahead == (DEPTH - 1) * STAGE_BYTES ? 0u : ahead + STAGE_BYTES;
      const float2* pa = reinterpret_cast<const float2*>(slot + CODE_BYTES) + g8;
      const float2 st_lo = pa[0], st_hi = pa[8], z_lo = pa[16], z_hi = pa[24];
      // The groups of a unit side by side, in two chains of MMAs each, so that loads, unpacking and MMAs of one hide the
      // others' latency. A last unit of one group multiplies whatever stands in the slot and drops it.
      const bool both = UNIT * u + 1 < n_groups;
      const uint8_t* xu = x_lane + (UNIT * u - chunk0) * (mp * 256);
      const float4* su = sx + (UNIT * u - chunk0) * TOKENS + 2 * t4;
      float s[UNIT][2][4];
#pragma unroll
      for (int i = 0; i < UNIT; ++i) {
        const uint4 lo = *reinterpret_cast<const uint4*>(slot + i * 1024 + lane * 16);
        const uint4 hi = *reinterpret_cast<const uint4*>(slot + i * 1024 + 512 + lane * 16);
        const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint4 x = *reinterpret_cast<const uint4*>(xu + (i * 4 + w) * mp * 64);
          const uint32_t l8 = wl[w] >> 8, h8 = wh[w] >> 8;
          if (w == 0) {
            mma16816_first(s[i][0], code_even(wl[w]), code_even(wh[w]), code_odd(wl[w]), code_odd(wh[w]), x.x, x.y);
            mma16816_first(s[i][1], code_even(l8), code_even(h8), code_odd(l8), code_odd(h8), x.z, x.w);
          } else {
            mma16816(s[i][0], code_even(wl[w]), code_even(wh[w]), code_odd(wl[w]), code_odd(wh[w]), x.x, x.y);
            mma16816(s[i][1], code_even(l8), code_even(h8), code_odd(l8), code_odd(h8), x.z, x.w);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < UNIT; ++i) {
        if (i == 1 && !both) break;
        const float4 m0s = su[i * TOKENS], m1s = su[i * TOKENS + 1];
        const float zl = i == 0 ? z_lo.x : z_lo.y, zh = i == 0 ? z_hi.x : z_hi.y;
        const float sl = i == 0 ? st_lo.x : st_lo.y, sh = i == 0 ? st_hi.x : st_hi.y;
        acc[0] = fmaf(sl * m0s.z, fmaf(-zl, m0s.y, (s[i][0][0] - m0s.x) + s[i][1][0]), acc[0]);
        acc[1] = fmaf(sl * m1s.z, fmaf(-zl, m1s.y, (s[i][0][1] - m1s.x) + s[i][1][1]), acc[1]);
        acc[2] = fmaf(sh * m0s.z, fmaf(-zh, m0s.y, (s[i][0][2] - m0s.x) + s[i][1][2]), acc[2]);
        acc[3] = fmaf(sh * m1s.z, fmaf(-zh, m1s.y, (s[i][0][3] - m1s.x) + s[i][1][3]), acc[3]);
      }
    }
    cp_async_wait<0>();

    // partial sums of this slice; CTA r of the cluster adds and stores the r-th share of the outputs
    float* mine = part + warp * 16 + g8;
    mine[(2 * t4) * PART_LD] = acc[0];
    mine[(2 * t4 + 1) * PART_LD] = acc[1];
    mine[(2 * t4) * PART_LD + 8] = acc[2];
    mine[(2 * t4 + 1) * PART_LD + 8] = acc[3];
    cluster_sync();
    const uint32_t part_a = smem_u32(part);
    auto total = [&](int idx) {
      float v = 0.0f;
      for (int r = 0; r < slices; ++r) v += ld_cluster_f32(map_to_rank(part_a + static_cast<uint32_t>(idx * 4), r));
      return v;
    };
    const int share = (OUT_ROWS + slices - 1) / slices;
    const int first = slice * share;
    const int n_rows = max(0, min(share, OUT_ROWS - first));
    for (int i = static_cast<int>(threadIdx.x); i < n_rows * mt; i += THREADS) {
      const int m = i / n_rows, r = first + i - m * n_rows;
      const int64_t o = out0 + r;
      if (o >= n_out) continue;
      float v;
      if (GATED) {
        const int idx = m * PART_LD + (r >> 3) * 16 + (r & 7);
        const float a = total(idx), b = total(idx + 8);
        v = silu(a) * b;
      } else {
        v = total(m * PART_LD + r);
        if (p.bias != nullptr) v += bf16_lo(p.bias[o]);
      }
      const __nv_bfloat16 y = __float2bfloat16_rn(v);
      p.Y[(row0 + m0 + m) * p.ldy + o] = *reinterpret_cast<const uint16_t*>(&y);
    }
    cluster_sync();  // every CTA has read this one's partial sums
  }
}

}  // namespace few
}  // namespace awq
