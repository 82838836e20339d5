// kernel_w4a16_few.cuh - products of a few tokens with packed 4-bit weights, for one layer or for the rows
// of each expert: Y = X' deq(W)^T, optionally with a bias or with the SiLU gate of a stacked gate and up
// projection in the epilogue.
//
// Mathematics: per group g of 128 in-features and token m, with a power of two c[m, g] that brings the group's largest
// |x'| to 2^14..2^15 and xs = c x',
//   Y[m, o] = sum_g step[o, g] / c[m, g] (sum_{k in g} q[o, k] xs[m, k] - z[o, g] sum_{k in g} xs[m, k]).
// A nibble in bits 4-7 of a half-word is the fp16 subnormal q 2^-20, so an AND and at most one shift per two codes make the
// operand, and the 2^20 goes into 1 / c. A bf16 x is exact in fp16 down to 2^-31 of its group's largest and below that
// off by 2^-39 of it, so the weights enter with their exact value; the tensor cores sum 15 |xs| at most in fp32, the step
// and zero point are applied once per group and output in fp32.
// The tensor cores line products up by the exponents of the operands as they are stored, 2^-14 for every subnormal, and cut
// what is below fp32's last place there, so a nibble has to stand high. Measured error ahead of the output's rounding, of its
// norm, 28672 in-features: 3e-6 at most for activations around zero, with outliers, of one sign and squared (2.4e-6 is
// what the measurement resolves), as for the plain fp32 form. With nibbles in bits 0-3 and 4-7, one shift per eight codes,
// 4e-4 for squared ones (and 34.8 us, not 36.9, for 28672 -> 8192), in bits 2-5 and 6-9 5e-5 (34.9), all in bits 6-9 5e-6 (37.0).
// Nibbles under the exponent of 1024 or 64, 1024 + q, whose constants' sums have to be taken off again, 1.2e-3 (36.5).
// (bf16 patterns 128 + q need a shift for every pair of codes.)
//
// The bound is HBM: a weight is read once and used for at most 8 tokens (0.5 byte per 16 operations), so
// what matters is bytes in flight and few instructions per weight. A one-token product cannot fill the
// tcgen05 tile (N >= 16 with operands staged in tensor or shared memory and a barrier per group), whose
// hand-offs bound the few-token kernel of w4a16_gemm; a warp-level MMA takes its A operand from the registers
// that unpacked it.
//
// A CTA of 4 warps owns 128 weight rows (gated: 64 gate rows and the 64 up rows of the same outputs) and a
// slice of the groups; a warp owns 32 rows, two MMA tiles, so a piece of X read from shared memory serves both. A
// lane loads the 16-byte pieces that it will itself unpack (rows l / 4 + 0, 8, 16, 24, 32 codes of a group each)
// straight into registers, three groups ahead, the L2 fetching a row's next three groups along. X as fp16, its sums
// (MMAs too, with a constant operand), the steps and the zero points of a chunk of groups stand in shared
// memory. Both MMA operands name the in-features of a group in the order that the unpacking gives,
// so X is permuted once, on its way there. The slices of a row block are the CTAs of one cluster (at most 8), which
// add their fp32 partial sums through distributed shared memory in slice order: one launch, no workspace, the same
// result every time.
//
// Measured (B200, weights that no cache holds): 28672 -> 8192 for one token in 35.4 us in a graph and 37.6 as calls, for 8
// tokens 49 and 51 (w4a16_gemm 50.4 and 52.3, 51 and 53); 4096 -> 4096 8.0 and 10.9 (10.6 and 17.2); 5 tokens 4224 -> 2 x
// 10756, gated, 23.9 and 25.7; 8 experts of 4096 -> 2 x 14336, gated, with 1, 2, 4 and 8 rows each 118, 126, 139 and 168 us
// back to back. That is 3.7 and, with 2 rows, 4.2 TB/s of packed weights. Without the loads of the codes the rest takes
// 29.6 us of the 35.4 and 105 of the 126, so it is bound twice: by the instructions of a group, and by how many loads the SM
// keeps in flight and how they fall on DRAM pages.
// Layouts, measured before the nibbles moved to bits 4-7, on the same weights again and again, 32 us for 28672 -> 8192 in a
// graph and 135 for 2 rows to each of 8 experts: one group ahead and 4 CTAs per SM 36 and 201 us, three ahead and 4 CTAs
// (which spills, and opens more rows at once) 36 and 235, seven ahead and 2 CTAs 35 and 163, four ahead 32 and 143; a bulk
// prefetch of each row into L2 instead 36 and 201; a predicate per load of X and addresses made per group 33 and 142.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace awq {
namespace few {

constexpr int WARPS = 4;
constexpr int THREADS = 32 * WARPS;
constexpr int ROWS = 32 * WARPS;                       // weight rows per CTA
constexpr int TOKENS = 8;                              // tokens at most, of the layer or of an expert
constexpr int DEPTH = 4;                               // groups in registers: one in use, three on their way
constexpr int CTAS_PER_SM = 3;
constexpr int PART_LD = ROWS + 4;                      // partial sums [TOKENS][PART_LD]
constexpr int PART_BYTES = TOKENS * PART_LD * 4;
constexpr int PARAM_LD = ROWS + 1;                     // steps and zero points [group][PARAM_LD], written down a column
constexpr int CHUNK_BYTES = 54 * 1024;                 // shared memory of a CTA, nearly all for a chunk of groups
constexpr int MAX_SLICES = 8;                          // portable cluster size

// Shared memory for chunks of `xg` groups of `mp` tokens (mp = 1, 2, 4 or 8).
__host__ __device__ constexpr int smem_bytes(int xg, int mp) {
  return PART_BYTES + xg * 256 * mp + (xg * PARAM_LD + 1) / 2 * 16 + xg * TOKENS * 8;
}
// The most groups that fit: what precedes a chunk's first group (its X, steps and zero points on their way, the sums of X)
// leaves the loads of the codes with the three groups ahead, so few and long chunks, as equal as DEPTH lets them be. With 67 KB
// per CTA the L1 that remains holds too few loads: 28672 -> 8192 for 8 tokens 49 to 58 us, 5 gated tokens 4224 -> 2 x 10756
// 24 to 33.
__host__ __device__ constexpr int chunk_groups(int mp) {
  return (CHUNK_BYTES - PART_BYTES) / (256 * mp + 8 * PARAM_LD + TOKENS * 8) / DEPTH * DEPTH;
}
constexpr int SMEM_MAX = CHUNK_BYTES;
static_assert(smem_bytes(chunk_groups(1), 1) <= SMEM_MAX && smem_bytes(chunk_groups(2), 2) <= SMEM_MAX &&
                  smem_bytes(chunk_groups(4), 4) <= SMEM_MAX && smem_bytes(chunk_groups(8), 8) <= SMEM_MAX &&
                  (SMEM_MAX + 1024) * CTAS_PER_SM <= 228 * 1024,
              "the largest chunk");

struct Params {
  const uint16_t* X;        // [R][ldx] bf16
  const uint32_t* codes;    // [E][O][K / 8]
  const float* steps;       // [E][O][G]
  const float* zeros;       // [E][O][G]
  const uint16_t* bias;     // [O] bf16 or null
  const int* offsets;       // [E + 1] first row of each expert, or null: one layer, rows 0..R-1
  uint16_t* Y;              // [R][ldy] bf16
  int64_t R, ldx, ldy, O, K, G;
  int g_per;                // groups per slice
  int xg;                   // groups per X chunk
  int mp_log2;              // log2 of the tokens that the X chunk has room for
};

__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
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
// 16 bytes of codes; the L2 fetches the 256 bytes around them, four groups of the row.
__device__ __forceinline__ uint4 ldg_codes(const uint32_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
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
// c = a b
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// Two codes of a word, n and n + 4, as fp16 numbers q 2^-20.
template <int N>
__device__ __forceinline__ uint32_t codes_of(uint32_t w) {
  return (N == 0 ? w << 4 : w >> (4 * N - 4)) & 0x00F000F0u;
}
constexpr uint32_t MINUS_ONE = 0x80108010u;  // in the same units
__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
// The larger exponent (bits 7-14) of two bf16 numbers.
__device__ __forceinline__ uint32_t exponent_max(uint32_t v) { return max(v & 0x7F80u, (v >> 16) & 0x7F80u); }
// a / (1 + exp(-a)) as a exp(-|a|) / (1 + exp(-|a|)) below zero, where exp(-a) would pass the largest float while the
// quotient is still a normal number (from -88.7 down). The quotient by a number from 1 to 2 is off by 2 units of 2^-23 as the
// fast one, where a bf16 step is 2^-8; rounded to nearest it cost the experts' gated products of 16384 rows 6 % (638 to 673 us).
__device__ __forceinline__ float silu(float a) {
  const float t = expf(-fabsf(a));
  return __fdividef(a < 0.0f ? a * t : a, 1.0f + t);
}

template <bool GATED>
__global__ void __launch_bounds__(THREADS, CTAS_PER_SM) w4a16_few_kernel(const Params p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint4 zero;      // X of tokens past mp
  __shared__ unsigned apart;  // bit m: token m is summed term by term in this slice
  if (threadIdx.x == 0) {
    zero = make_uint4(0u, 0u, 0u, 0u);
    apart = 0u;
  }
  // The experts' grouped kernel reads nothing that this one writes: it may start once every CTA of this one has.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g8 = lane >> 2, t4 = lane & 3;
  const int slice = static_cast<int>(blockIdx.x), slices = static_cast<int>(gridDim.x);
  const int64_t e = blockIdx.z;

  int64_t row0 = 0, rows = p.R;
  if (p.offsets != nullptr) {  // clamped, so that whatever stands there no access leaves X and Y
    row0 = min(max(static_cast<int64_t>(p.offsets[e]), int64_t(0)), p.R);
    rows = min(max(static_cast<int64_t>(p.offsets[e + 1]), row0), p.R) - row0;
  }
  // the same for every CTA of the cluster; experts with more rows are left to another kernel
  if (rows == 0 || rows > TOKENS) return;
  const int mt = static_cast<int>(rows);

  const int64_t n_out = GATED ? p.O / 2 : p.O;
  constexpr int OUT_ROWS = GATED ? ROWS / 2 : ROWS;
  const int64_t out0 = static_cast<int64_t>(blockIdx.y) * OUT_ROWS;
  // Weight row of this warp's row r (0..31); rows past the end read the last row and are not stored. Gated: rows 0-7 of
  // each MMA tile are gate rows, rows 8-15 the up rows of the same outputs, so one lane holds both.
  auto weight_row = [&](int r) -> int64_t {
    if (GATED) return min(out0 + warp * 16 + (r >> 4) * 8 + (r & 7), n_out - 1) + ((r >> 3) & 1) * n_out;
    return min(out0 + warp * 32 + r, n_out - 1);
  };

  const int g_begin = slice * p.g_per;
  const int n_groups = max(min(p.g_per, static_cast<int>(p.G) - g_begin), 0);
  const int mp = 1 << p.mp_log2;

  float* part = reinterpret_cast<float*>(smem);
  uint8_t* xs = smem + PART_BYTES;                                         // [group][word][token][t4] 16 bytes
  float2* param = reinterpret_cast<float2*>(xs + (p.xg * 256 << p.mp_log2));  // [group][PARAM_LD]: step, zero point
  float2* sx = param + (p.xg * PARAM_LD + 1) / 2 * 2;  // [group][TOKENS]: -(sum of xs) 2^-20, 2^20 / c

  const uint32_t* codes = p.codes + e * p.O * (p.K / 8) + g_begin * 16;
  const uint32_t* code[4];  // the lane's pieces of its rows g8, g8 + 8, g8 + 16, g8 + 24
#pragma unroll
  for (int j = 0; j < 4; ++j) code[j] = codes + weight_row(g8 + 8 * j) * (p.K / 8) + t4 * 4;
  uint4 w[DEPTH][4];
  int left = n_groups;  // from the groups that `code` stands at
  auto load = [&](int d, int ahead) {
    if (ahead < left) {
#pragma unroll
      for (int j = 0; j < 4; ++j) w[d][j] = ldg_codes(code[j] + ahead * 16);
    }
  };

  // X of the tokens and of groups gc..gc+ng-1 as fp16, scaled and permuted so that one 16-byte piece (in-features
  // 8w..8w+7) holds the pairs (0, 4), (1, 5), (2, 6), (3, 7). The 16 threads of a token's group are neighbours.
  auto stage_x = [&](int gc, int ng) {
    const int per_token = ng * 16;
    constexpr int AT_ONCE = 4;  // loads in flight per thread
    const uint16_t* src = p.X + row0 * p.ldx + static_cast<int64_t>(gc) * 128;
    int m = 0, c = static_cast<int>(threadIdx.x);  // the thread's next token and 16-byte piece
    while (c >= per_token) c -= per_token, ++m;
    // all threads of a warp take the same number of turns: its pieces are of neighbouring groups, 16 threads each
    for (int left = per_token * mt - static_cast<int>(threadIdx.x & ~31u); left > 0; left -= AT_ONCE * THREADS) {
      uint4 v[AT_ONCE];
      int to[AT_ONCE];
#pragma unroll
      for (int k = 0; k < AT_ONCE; ++k) {
        v[k] = make_uint4(0u, 0u, 0u, 0u);
        to[k] = m < mt ? m << 16 | c : -1;
        if (m < mt) v[k] = *reinterpret_cast<const uint4*>(src + m * p.ldx + c * 8);
        c += THREADS;
        while (c >= per_token) c -= per_token, ++m;
      }
#pragma unroll
      for (int k = 0; k < AT_ONCE; ++k) {
        if (k * THREADS >= left) break;
        // exponent of the group's largest value
        uint32_t most = max(max(exponent_max(v[k].x), exponent_max(v[k].y)), max(exponent_max(v[k].z), exponent_max(v[k].w)));
#pragma unroll
        for (int d = 1; d < 16; d *= 2) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
        // c = 2^(14 - exponent), below 2^127; 2^20 / c is a normal number up to an exponent of 121
        const uint32_t field = min(268u - (most >> 7), 253u);
        const float scale = __uint_as_float(field << 23);
        __half2 h[4];
        h[0] = __floats2half2_rn(bf16_lo(v[k].x) * scale, bf16_lo(v[k].z) * scale);
        h[1] = __floats2half2_rn(bf16_hi(v[k].x) * scale, bf16_hi(v[k].z) * scale);
        h[2] = __floats2half2_rn(bf16_lo(v[k].y) * scale, bf16_lo(v[k].w) * scale);
        h[3] = __floats2half2_rn(bf16_hi(v[k].y) * scale, bf16_hi(v[k].w) * scale);
        if (to[k] >= 0) {
          const int mk = to[k] >> 16, ck = to[k] & 0xFFFF;
          const int grp = ck >> 4, t = (ck >> 2) & 3, word = ck & 3;
          *reinterpret_cast<uint4*>(xs + (((grp * 4 + word) * mp + mk) * 4 + t) * 16) = *reinterpret_cast<const uint4*>(h);
          if ((ck & 15) == 0) {
            sx[grp * TOKENS + mk].y = __uint_as_float(min(274u - field, 254u) << 23);
            if (field < 20u) atomicOr(&apart, 1u << mk);  // 2^122 and more, infinities, NaN
          }
        }
      }
    }
  };
  // The B operand of in-features 8 w.. of a group: lanes of tokens past mp read a zero that stays where it is.
  const bool x_real = g8 < mp;
  const uint32_t x_lane = x_real ? smem_u32(xs) + static_cast<uint32_t>(((g8 * 4) + t4) * 16) : smem_u32(&zero);
  const uint32_t x_word = x_real ? static_cast<uint32_t>(mp * 64) : 0u, x_group = 4 * x_word;
  uint4 x[4];
  auto load_x = [&](uint32_t at) {
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = lds128(at + k * x_word);
  };
  // Minus the sum of xs per group and token.
  auto sum_x = [&](int ng) {
    for (int gx = warp; gx < ng; gx += WARPS) {
      load_x(x_lane + gx * x_group);
      float s[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k == 0) mma16816_first(s, MINUS_ONE, MINUS_ONE, MINUS_ONE, MINUS_ONE, x[k].x, x[k].y);
        else mma16816(s, MINUS_ONE, MINUS_ONE, MINUS_ONE, MINUS_ONE, x[k].x, x[k].y);
        mma16816(s, MINUS_ONE, MINUS_ONE, MINUS_ONE, MINUS_ONE, x[k].z, x[k].w);
      }
      if (g8 == 0) {  // the rows of the result are all the same
        sx[gx * TOKENS + 2 * t4].x = s[0];
        sx[gx * TOKENS + 2 * t4 + 1].x = s[1];
      }
    }
  };

  float acc[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
  for (int d = 0; d < DEPTH - 1; ++d) load(d, d);
  for (int chunk0 = 0; chunk0 < n_groups; chunk0 += p.xg) {
    const int chunk = min(p.xg, n_groups - chunk0);
    __syncthreads();  // the previous chunk has been read
    // steps and zero points, a row of this warp's at a time: a row's groups are neighbours
    for (int gl = lane; gl < chunk; gl += 32) {
      const int64_t first = (e * p.O + weight_row(0)) * p.G + g_begin + chunk0 + gl;
      const float* ps = p.steps + first;
      const float* pz = p.zeros + first;
      const int64_t up = n_out * p.G;                            // gated: from a gate row to its up row
      int rows_left = static_cast<int>(min(n_out - 1 - weight_row(0), int64_t(32)));  // rows past the end: the last one's
      uint32_t dst = smem_u32(param + gl * PARAM_LD + warp * 32);
#pragma unroll 4
      for (int r = 0; r < (GATED ? 16 : 32); ++r) {
        // gated: gate row r is row r % 8 of MMA tile r / 8, its up row 8 behind it
        const uint32_t to = dst + static_cast<uint32_t>((GATED ? (r >> 3) * 16 + (r & 7) : r) * 8);
        cp_async4(to, ps);
        cp_async4(to + 4u, pz);
        if (GATED) {
          cp_async4(to + 64u, ps + up);
          cp_async4(to + 68u, pz + up);
        }
        if (--rows_left >= 0) {
          ps += p.G;
          pz += p.G;
        }
      }
    }
    stage_x(g_begin + chunk0, chunk);
    __syncthreads();
    sum_x(chunk);
    cp_async_wait_all();
    __syncthreads();
    const float2* pa = param + warp * 32 + g8;
    const float2* sa = sx + 2 * t4;
    uint32_t xa = x_lane;
    for (int g0 = 0; g0 < chunk; g0 += DEPTH) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        if (g0 + d >= chunk) break;
        load((d + DEPTH - 1) % DEPTH, d + DEPTH - 1);
        load_x(xa);
        const float4 sums = *reinterpret_cast<const float4*>(sa);  // two tokens
        float s[2][4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t lo = word_of(w[d][2 * i], k), hi = word_of(w[d][2 * i + 1], k);
            if (k == 0)
              mma16816_first(s[i], codes_of<0>(lo), codes_of<0>(hi), codes_of<1>(lo), codes_of<1>(hi), x[k].x, x[k].y);
            else
              mma16816(s[i], codes_of<0>(lo), codes_of<0>(hi), codes_of<1>(lo), codes_of<1>(hi), x[k].x, x[k].y);
            mma16816(s[i], codes_of<2>(lo), codes_of<2>(hi), codes_of<3>(lo), codes_of<3>(hi), x[k].z, x[k].w);
          }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 lo = pa[16 * i], hi = pa[16 * i + 8];
          acc[i][0] = fmaf(lo.x, fmaf(lo.y, sums.x, s[i][0]) * sums.y, acc[i][0]);
          acc[i][1] = fmaf(lo.x, fmaf(lo.y, sums.z, s[i][1]) * sums.w, acc[i][1]);
          acc[i][2] = fmaf(hi.x, fmaf(hi.y, sums.x, s[i][2]) * sums.y, acc[i][2]);
          acc[i][3] = fmaf(hi.x, fmaf(hi.y, sums.z, s[i][3]) * sums.w, acc[i][3]);
        }
        pa += PARAM_LD;
        sa += TOKENS;
        xa += x_group;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) code[j] += DEPTH * 16;
      left -= DEPTH;
    }
  }

  // partial sums of this slice; CTA r of the cluster adds and stores the r-th share of the outputs
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float* mine = part + warp * 32 + i * 16 + g8;
    mine[(2 * t4) * PART_LD] = acc[i][0];
    mine[(2 * t4 + 1) * PART_LD] = acc[i][1];
    mine[(2 * t4) * PART_LD + 8] = acc[i][2];
    mine[(2 * t4 + 1) * PART_LD + 8] = acc[i][3];
  }
  // What the group sums cannot give, since they take z sum x off sum q x: tokens with an infinity or a NaN again (or with a
  // value of 2^122 and more, whose 2^20 / c is no number), term by term from the weights as fp32 numbers, so that each
  // output is the infinity or the NaN of the definition (as in the experts' grouped kernel). A column of the MMA is a token,
  // so the others have not been touched.
  const unsigned tokens_apart = apart;
  if (tokens_apart != 0u) {
    __syncwarp();
#pragma unroll 1
    for (unsigned rest = tokens_apart; rest != 0u; rest &= rest - 1u) {
      const int m = __ffs(rest) - 1;
      const uint16_t* xr = p.X + (row0 + m) * p.ldx + static_cast<int64_t>(g_begin) * 128 + lane * 4;
#pragma unroll 1
      for (int r = 0; r < 32; ++r) {
        const int64_t wr = weight_row(r), first = (e * p.O + wr) * p.G + g_begin;
        const uint32_t* c = codes + wr * (p.K / 8) + (lane >> 1);
        float v = 0.0f;
#pragma unroll 1
        for (int g = 0; g < n_groups; ++g) {
          const uint2 x4 = *reinterpret_cast<const uint2*>(xr + g * 128);
          const uint32_t q = c[g * 16] >> ((lane & 1) * 16);
          const float step = p.steps[first + g], z = p.zeros[first + g];
          v = fmaf((static_cast<float>(q & 15u) - z) * step, bf16_lo(x4.x), v);
          v = fmaf((static_cast<float>((q >> 4) & 15u) - z) * step, bf16_hi(x4.x), v);
          v = fmaf((static_cast<float>((q >> 8) & 15u) - z) * step, bf16_lo(x4.y), v);
          v = fmaf((static_cast<float>((q >> 12) & 15u) - z) * step, bf16_hi(x4.y), v);
        }
#pragma unroll
        for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
        if (lane == 0) part[m * PART_LD + warp * 32 + r] = v;
      }
    }
  }
  if (slices > 1) cluster_sync();
  else __syncthreads();
  const uint32_t part_a = smem_u32(part);
  auto total = [&](int idx) {
    if (slices == 1) return part[idx];
    float from[MAX_SLICES];  // all of them on their way before the first is added
#pragma unroll
    for (int r = 0; r < MAX_SLICES; ++r)
      from[r] = r < slices ? ld_cluster_f32(map_to_rank(part_a + static_cast<uint32_t>(idx * 4), r)) : 0.0f;
    float v = 0.0f;
#pragma unroll
    for (int r = 0; r < MAX_SLICES; ++r) v += from[r];
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
    p.Y[(row0 + m) * p.ldy + o] = *reinterpret_cast<const uint16_t*>(&y);
  }
  if (slices > 1) cluster_sync();  // every CTA has read this one's partial sums
}

}  // namespace few
}  // namespace awq
