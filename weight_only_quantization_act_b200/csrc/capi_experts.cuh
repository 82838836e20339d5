// capi_experts.cuh - host side of the one-token products, the expert sort with its gathers and sums, and the
// experts' products: argument validation and launches (included by awq_capi.cu, whose helpers it uses).
#pragma once

namespace {

// A bf16 output that is stored element by element: any row stride of at least `cols`.
awq_status check_output(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld) {
  if (p == nullptr) return fail(AWQ_ERR_INVALID_ARG, "%s is null", name);
  if ((reinterpret_cast<uintptr_t>(p) & 1u) != 0) return fail(AWQ_ERR_INVALID_ARG, "%s is not 2-byte aligned", name);
  if (rows > 1 && ld < cols)
    return fail(AWQ_ERR_INVALID_ARG, "%s row stride %lld must be >= %lld", name, static_cast<long long>(ld),
                static_cast<long long>(cols));
  return AWQ_OK;
}

awq_status check_packed(const void* codes, const float* steps, const float* zeros, int64_t O, int64_t K, int gated) {
  if (K % 128 != 0) return fail(AWQ_ERR_INVALID_ARG, "K (%lld) must be a multiple of 128", static_cast<long long>(K));
  if (O < 1 || O >= (1ll << 31)) return fail(AWQ_ERR_INVALID_ARG, "O (%lld) out of range", static_cast<long long>(O));
  if (gated != 0 && gated != 1) return fail(AWQ_ERR_INVALID_ARG, "gated must be 0 or 1, not %d", gated);
  if (gated && O % 2 != 0)
    return fail(AWQ_ERR_INVALID_ARG, "gated needs an even O (gate rows, then up rows), not %lld", static_cast<long long>(O));
  if (codes == nullptr || steps == nullptr || zeros == nullptr || !aligned16(codes))
    return fail(AWQ_ERR_INVALID_ARG, "codes (16-byte aligned), steps and zeros must be given");
  if ((reinterpret_cast<uintptr_t>(steps) | reinterpret_cast<uintptr_t>(zeros)) & 3u)
    return fail(AWQ_ERR_INVALID_ARG, "steps and zeros must be 4-byte aligned");
  return AWQ_OK;
}

// An array of int32 or float.
awq_status check_words(const char* name, const void* p) {
  if (p == nullptr) return fail(AWQ_ERR_INVALID_ARG, "%s must be given", name);
  if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0) return fail(AWQ_ERR_INVALID_ARG, "%s is not 4-byte aligned", name);
  return AWQ_OK;
}

awq_status check_experts(int64_t E) {
  if (E < 1 || E > AWQ_MAX_EXPERTS)
    return fail(AWQ_ERR_INVALID_ARG, "%lld experts: 1 to %d are supported", static_cast<long long>(E), AWQ_MAX_EXPERTS);
  return AWQ_OK;
}

int64_t few_row_blocks(int64_t O, bool gated) {
  const int64_t out_rows = gated ? awq::few::ROWS / 2 : awq::few::ROWS;
  return ((gated ? O / 2 : O) + out_rows - 1) / out_rows;
}

awq_status check_few_rows(int64_t O, bool gated) {
  if (few_row_blocks(O, gated) > 65535)  // the grid's y extent
    return fail(AWQ_ERR_INVALID_ARG, "O (%lld) is too large", static_cast<long long>(O));
  return AWQ_OK;
}

// Rows of every expert, or of the one layer (E = 1, offsets null), through the few-token kernel. `active` experts
// can have rows, each up to `tokens` of them.
awq_status launch_few(awq::few::Params& p, int64_t E, int64_t active, int64_t tokens, bool gated, int sms,
                      cudaStream_t st) {
  const int64_t n_rb = few_row_blocks(p.O, gated);
  // The number of slices that takes the fewest steps: waves of CTAs times a CTA's groups, and what a CTA does before
  // and after them, which takes about as long as 10 groups.
  int64_t slices = 1, best = 0;
  for (int64_t n = 1; n <= awq::few::MAX_SLICES && 2 * n <= std::max<int64_t>(p.G, 2); ++n) {
    const int64_t slots = static_cast<int64_t>(awq::few::CTAS_PER_SM) * sms / n * n;
    const int64_t steps = (n_rb * active * n + slots - 1) / slots * ((p.G + n - 1) / n + 10);
    if (n == 1 || steps < best) {
      best = steps;
      slices = n;
    }
  }
  p.g_per = static_cast<int>((p.G + slices - 1) / slices);
  slices = (p.G + p.g_per - 1) / p.g_per;
  p.mp_log2 = tokens <= 1 ? 0 : tokens <= 2 ? 1 : tokens <= 4 ? 2 : 3;
  const int most = awq::few::chunk_groups(1 << p.mp_log2), chunks = (p.g_per + most - 1) / most;
  p.xg = ((p.g_per + chunks - 1) / chunks + awq::few::DEPTH - 1) / awq::few::DEPTH * awq::few::DEPTH;  // equal chunks
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(slices), static_cast<unsigned>(n_rb), static_cast<unsigned>(E));
  cfg.blockDim = dim3(awq::few::THREADS);
  cfg.dynamicSmemBytes = static_cast<size_t>(awq::few::smem_bytes(p.xg, 1 << p.mp_log2));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(slices);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (gated)
    AWQ_CUDA(cudaLaunchKernelEx(&cfg, awq::few::w4a16_few_kernel<true>, p));
  else
    AWQ_CUDA(cudaLaunchKernelEx(&cfg, awq::few::w4a16_few_kernel<false>, p));
  return check_launch("w4a16_few_kernel");
}

}  // namespace

extern "C" awq_status awq_w4a16_gemv(const void* X, int64_t M, int64_t K, int64_t ldx, const uint32_t* codes,
                                     const float* steps, const float* zeros, int64_t O, const void* bias, int gated,
                                     void* Y, int64_t ldy, awq_stream_t stream) {
  AWQ_TRY(check_matrix("X", X, M, K, ldx));
  AWQ_TRY(check_packed(codes, steps, zeros, O, K, gated));
  if (M > AWQ_GEMV_MAX_TOKENS)
    return fail(AWQ_ERR_INVALID_ARG, "%lld tokens: awq_w4a16_gemv takes 1 to %d, awq_w4a16_gemm any number",
                static_cast<long long>(M), AWQ_GEMV_MAX_TOKENS);
  AWQ_TRY(check_output("Y", Y, M, gated ? O / 2 : O, ldy));
  if (bias != nullptr && gated) return fail(AWQ_ERR_INVALID_ARG, "bias and gated cannot be combined");
  if ((reinterpret_cast<uintptr_t>(bias) & 1u) != 0) return fail(AWQ_ERR_INVALID_ARG, "bias is not 2-byte aligned");
  AWQ_TRY(check_few_rows(O, gated != 0));
  DeviceInfo* d = nullptr;
  AWQ_TRY(device_info(&d));
  awq::few::Params p = {};
  p.X = static_cast<const uint16_t*>(X);
  p.codes = codes;
  p.steps = steps;
  p.zeros = zeros;
  p.bias = static_cast<const uint16_t*>(bias);
  p.Y = static_cast<uint16_t*>(Y);
  p.R = M;
  p.ldx = ldx;
  p.ldy = ldy;
  p.O = O;
  p.K = K;
  p.G = K / 128;
  AWQ_TRY(launch_few(p, 1, 1, M, gated != 0, d->sms, reinterpret_cast<cudaStream_t>(stream)));
  return ok();
}

// ------------------------------------------------------------------------------------------- expert sort
namespace {
int64_t sort_blocks(int64_t n) {
  if (n <= awq::ex::SORT_ALONE) return 1;  // one block counts and places
  return std::min<int64_t>((n + 1023) / 1024, awq::ex::SORT_MAX_BLOCKS);
}

awq_status check_rows_args(int64_t T, int64_t top_k, int64_t K) {
  if (top_k < 1) return fail(AWQ_ERR_INVALID_ARG, "top_k (%lld) must be at least 1", static_cast<long long>(top_k));
  if (T >= (1ll << 31) || top_k >= (1ll << 31) || T * top_k >= (1ll << 31))
    return fail(AWQ_ERR_INVALID_ARG, "too many slots");
  if (K % 8 != 0) return fail(AWQ_ERR_INVALID_ARG, "K (%lld) must be a multiple of 8", static_cast<long long>(K));
  if (K > 65535ll * 8 * awq::ex::ROW_THREADS)  // the grid's y extent
    return fail(AWQ_ERR_INVALID_ARG, "K (%lld) is too large", static_cast<long long>(K));
  return AWQ_OK;
}

// Blocks along the columns where a thread takes `pieces` of 8 columns.
unsigned column_blocks(int64_t K, int pieces) {
  const int64_t per_block = 8ll * awq::ex::ROW_THREADS * pieces;
  return static_cast<unsigned>((K + per_block - 1) / per_block);
}

template <typename ID>
awq_status launch_sort(const ID* ids, int64_t n, int E, int* counts, int* offsets, int* order, int* pos, cudaStream_t st) {
  const int64_t blocks = sort_blocks(n);
  const int64_t per_block = (n + blocks - 1) / blocks;
  const size_t smem = static_cast<size_t>(1 + awq::ex::SORT_WARPS) * E * sizeof(int);
  if (blocks > 1) {
    awq::ex::expert_count_kernel<ID><<<static_cast<unsigned>(blocks), awq::ex::SORT_THREADS, 0, st>>>(ids, n, E, per_block,
                                                                                                  counts);
    AWQ_TRY(check_launch("expert_count_kernel"));
  }
  awq::ex::expert_place_kernel<ID><<<static_cast<unsigned>(blocks), awq::ex::SORT_THREADS, smem, st>>>(
      ids, n, E, per_block, blocks > 1 ? counts : nullptr, offsets, order, pos);
  return check_launch("expert_place_kernel");
}
}  // namespace

extern "C" size_t awq_expert_sort_workspace_size(int64_t n_slots, int64_t E) {
  if (n_slots < 1 || E < 1 || E > AWQ_MAX_EXPERTS) return 0;
  const int64_t blocks = sort_blocks(n_slots);
  return blocks == 1 ? 0 : static_cast<size_t>(blocks) * static_cast<size_t>(E) * sizeof(int);
}

extern "C" awq_status awq_expert_sort(const void* ids, int id_bytes, int64_t n_slots, int64_t E, void* workspace,
                                      size_t ws_bytes, int32_t* offsets, int32_t* order, int32_t* pos,
                                      awq_stream_t stream) {
  if (id_bytes != 4 && id_bytes != 8) return fail(AWQ_ERR_INVALID_ARG, "id_bytes must be 4 or 8, not %d", id_bytes);
  if (n_slots < 1 || n_slots >= (1ll << 31))
    return fail(AWQ_ERR_INVALID_ARG, "n_slots (%lld) out of range", static_cast<long long>(n_slots));
  AWQ_TRY(check_experts(E));
  if (ids == nullptr || offsets == nullptr || order == nullptr || pos == nullptr)
    return fail(AWQ_ERR_INVALID_ARG, "ids, offsets, order and pos must be given");
  if ((reinterpret_cast<uintptr_t>(ids) & static_cast<uintptr_t>(id_bytes - 1)) != 0)
    return fail(AWQ_ERR_INVALID_ARG, "ids is not %d-byte aligned", id_bytes);
  if ((reinterpret_cast<uintptr_t>(offsets) | reinterpret_cast<uintptr_t>(order) | reinterpret_cast<uintptr_t>(pos)) & 3u)
    return fail(AWQ_ERR_INVALID_ARG, "offsets, order and pos must be 4-byte aligned");
  const size_t need = awq_expert_sort_workspace_size(n_slots, E);
  if (need > 0 && (workspace == nullptr || ws_bytes < need))
    return fail(AWQ_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, workspace ? ws_bytes : 0);
  if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) & 3u) != 0)
    return fail(AWQ_ERR_INVALID_ARG, "workspace is not 4-byte aligned");
  DeviceInfo* d = nullptr;
  AWQ_TRY(device_info(&d));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int* counts = static_cast<int*>(workspace);
  if (id_bytes == 4)
    AWQ_TRY(launch_sort(static_cast<const int32_t*>(ids), n_slots, static_cast<int>(E), counts, offsets, order, pos, st));
  else
    AWQ_TRY(launch_sort(static_cast<const int64_t*>(ids), n_slots, static_cast<int>(E), counts, offsets, order, pos, st));
  return ok();
}

extern "C" awq_status awq_expert_gather(const void* X, int64_t T, int64_t K, int64_t ldx, int64_t top_k,
                                        const int32_t* offsets, int64_t E, const int32_t* order, const float* scales,
                                        void* Xs, int64_t ldxs, awq_stream_t stream) {
  AWQ_TRY(check_matrix("X", X, T, K, ldx));
  AWQ_TRY(check_rows_args(T, top_k, K));
  AWQ_TRY(check_matrix("Xs", Xs, T * top_k, K, ldxs));
  AWQ_TRY(check_experts(E));
  AWQ_TRY(check_words("offsets", offsets));
  AWQ_TRY(check_words("order", order));
  if (!aligned16(scales)) return fail(AWQ_ERR_INVALID_ARG, "scales is not 16-byte aligned");
  DeviceInfo* d = nullptr;
  AWQ_TRY(device_info(&d));
  const int64_t n = T * top_k;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (scales == nullptr) {
    awq::ex::expert_gather_kernel<<<static_cast<unsigned>(n), awq::ex::ROW_THREADS, 0, st>>>(
        static_cast<const uint16_t*>(X), ldx, T, K, order, static_cast<int>(top_k), static_cast<uint16_t*>(Xs), ldxs);
  } else {
    const dim3 grid(static_cast<unsigned>((n + awq::ex::RUN - 1) / awq::ex::RUN), column_blocks(K, 1));
    awq::ex::expert_gather_scaled_kernel<<<grid, awq::ex::ROW_THREADS, 0, st>>>(
        static_cast<const uint16_t*>(X), ldx, T, K, offsets, static_cast<int>(E), order, static_cast<int>(top_k), scales,
        static_cast<uint16_t*>(Xs), ldxs, n);
  }
  AWQ_TRY(check_launch("expert_gather_kernel"));
  return ok();
}

namespace {
awq_status combine(const void* Ys, int64_t T, int64_t K, int64_t ldys, int64_t top_k, const int32_t* pos,
                   const float* weights, const int32_t* offsets, int64_t E, const float* scales, void* Y, int64_t ldy,
                   awq_stream_t stream) {
  DeviceInfo* d = nullptr;
  AWQ_TRY(device_info(&d));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (scales == nullptr) {
    const dim3 grid(static_cast<unsigned>(T), column_blocks(K, 2));
    awq::ex::expert_combine_kernel<<<grid, awq::ex::ROW_THREADS, 0, st>>>(
        static_cast<const uint16_t*>(Ys), ldys, K, pos, static_cast<int>(top_k), T * top_k, weights,
        static_cast<uint16_t*>(Y), ldy);
  } else {
    const dim3 grid(static_cast<unsigned>(T), column_blocks(K, 1));
    awq::ex::expert_combine_scaled_kernel<<<grid, awq::ex::ROW_THREADS, 0, st>>>(
        static_cast<const uint16_t*>(Ys), ldys, K, pos, static_cast<int>(top_k), T * top_k, offsets, static_cast<int>(E),
        scales, static_cast<uint16_t*>(Y), ldy);
  }
  AWQ_TRY(check_launch("expert_combine_kernel"));
  return ok();
}
}  // namespace

extern "C" awq_status awq_expert_gather_backward(const void* dXs, int64_t T, int64_t K, int64_t lddxs, int64_t top_k,
                                                 const int32_t* offsets, int64_t E, const int32_t* pos,
                                                 const float* scales, void* dX, int64_t lddx, awq_stream_t stream) {
  AWQ_TRY(check_matrix("dX", dX, T, K, lddx));
  AWQ_TRY(check_rows_args(T, top_k, K));
  AWQ_TRY(check_matrix("dXs", dXs, T * top_k, K, lddxs));
  AWQ_TRY(check_experts(E));
  AWQ_TRY(check_words("offsets", offsets));
  AWQ_TRY(check_words("pos", pos));
  if (!aligned16(scales)) return fail(AWQ_ERR_INVALID_ARG, "scales is not 16-byte aligned");
  return combine(dXs, T, K, lddxs, top_k, pos, nullptr, offsets, E, scales, dX, lddx, stream);
}

extern "C" awq_status awq_expert_combine(const void* Ys, int64_t T, int64_t O, int64_t ldys, int64_t top_k,
                                         const int32_t* pos, const float* weights, void* Y, int64_t ldy,
                                         awq_stream_t stream) {
  AWQ_TRY(check_matrix("Y", Y, T, O, ldy));
  AWQ_TRY(check_rows_args(T, top_k, O));
  AWQ_TRY(check_matrix("Ys", Ys, T * top_k, O, ldys));
  AWQ_TRY(check_words("pos", pos));
  if (weights != nullptr) AWQ_TRY(check_words("weights", weights));
  return combine(Ys, T, O, ldys, top_k, pos, weights, nullptr, 0, nullptr, Y, ldy, stream);
}

extern "C" awq_status awq_expert_combine_backward(const void* dY, int64_t T, int64_t O, int64_t lddy, const void* Ys,
                                                  int64_t ldys, int64_t top_k, const int32_t* pos, const float* weights,
                                                  void* dYs, int64_t lddys, float* dweights, awq_stream_t stream) {
  AWQ_TRY(check_matrix("dY", dY, T, O, lddy));
  AWQ_TRY(check_rows_args(T, top_k, O));
  AWQ_TRY(check_matrix("Ys", Ys, T * top_k, O, ldys));
  AWQ_TRY(check_matrix("dYs", dYs, T * top_k, O, lddys));
  AWQ_TRY(check_words("pos", pos));
  AWQ_TRY(check_words("weights", weights));
  AWQ_TRY(check_words("dweights", dweights));
  DeviceInfo* d = nullptr;
  AWQ_TRY(device_info(&d));
  awq::ex::expert_combine_backward_kernel<<<static_cast<unsigned>(T * top_k), awq::ex::ROW_THREADS, 0,
                                            reinterpret_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint16_t*>(dY), lddy, static_cast<const uint16_t*>(Ys), ldys, O, pos, static_cast<int>(top_k),
      T * top_k, weights, static_cast<uint16_t*>(dYs), lddys, dweights);
  AWQ_TRY(check_launch("expert_combine_backward_kernel"));
  return ok();
}

// --------------------------------------------------------------------------------------- experts' products
extern "C" size_t awq_w4a16_experts_workspace_size(int64_t R, int64_t E, int64_t K, int64_t O) {
  if (R < 1 || E < 1 || E > AWQ_MAX_EXPERTS || K < 128 || O < 1) return 0;
  return 512;  // status word
}

extern "C" awq_status awq_w4a16_experts(const void* Xs, int64_t R, int64_t K, int64_t ldx, const int32_t* offsets, int64_t E,
                                        const uint32_t* codes, const float* steps, const float* zeros, int64_t O, int gated,
                                        void* Y, int64_t ldy, void* workspace, size_t ws_bytes, awq_stream_t stream) {
  AWQ_TRY(check_matrix("Xs", Xs, R, K, ldx));
  AWQ_TRY(check_packed(codes, steps, zeros, O, K, gated));
  AWQ_TRY(check_experts(E));
  AWQ_TRY(check_words("offsets", offsets));
  AWQ_TRY(check_output("Y", Y, R, gated ? O / 2 : O, ldy));
  const size_t need = awq_w4a16_experts_workspace_size(R, E, K, O);
  if (workspace == nullptr || ws_bytes < need)
    return fail(AWQ_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, workspace ? ws_bytes : 0);
  if (!aligned16(workspace)) return fail(AWQ_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
  // Experts of up to 8 rows run the few-token kernel, the others the grouped one. Everything that can be refused is
  // looked at before the first of the two is launched.
  const bool grouped = R > awq::few::TOKENS;
  const int64_t tile_out = gated ? awq::grp::HALF : 2 * awq::grp::HALF;
  const int64_t n_bands = ((gated ? O / 2 : O) + tile_out - 1) / tile_out;
  AWQ_TRY(check_few_rows(O, gated));
  if (grouped && (E * O >= (1ll << 31) || (R / awq::grp::BN + E) * n_bands >= (1ll << 31)))
    return fail(AWQ_ERR_INVALID_ARG, "too many weight rows or tiles");
  DeviceInfo* d = nullptr;
  AWQ_TRY(device_info(&d));
  CUtensorMap tmX[3], tmC;  // boxes of 32, 64 and 96 rows
  if (grouped) {
    for (int i = 0; i < 3; ++i) AWQ_TRY(make_tmap(&tmX[i], Xs, R, K, ldx, (i + 1) * awq::grp::X_BOX));
    AWQ_TRY(make_tmap_codes_sw128(&tmC, codes, E * O, K / 8, gated ? 16 : awq::grp::HALF));
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  awq::few::Params p = {};
  p.X = static_cast<const uint16_t*>(Xs);
  p.codes = codes;
  p.steps = steps;
  p.zeros = zeros;
  p.offsets = offsets;
  p.Y = static_cast<uint16_t*>(Y);
  p.R = R;
  p.ldx = ldx;
  p.ldy = ldy;
  p.O = O;
  p.K = K;
  p.G = K / 128;
  AWQ_TRY(launch_few(p, E, std::min(E, R), R, gated != 0, d->sms, st));
  if (!grouped) return ok();
  awq::grp::Params q = {};
  q.offsets = offsets;
  q.steps = steps;
  q.zeros = zeros;
  q.Y = static_cast<uint16_t*>(Y);
  q.R = R;
  q.O = O;
  q.G = K / 128;
  q.ldy = ldy;
  q.E = static_cast<int>(E);
  q.n_bands = static_cast<int>(n_bands);
  q.pair_params = q.G % 2 == 0 && ((reinterpret_cast<uintptr_t>(steps) | reinterpret_cast<uintptr_t>(zeros)) & 7u) == 0;
  q.status = static_cast<awq::DeviceStatus*>(workspace);
  q.limit_ns = g_wait_limit_ns.load();
  q.stall_tile = g_experts_stall.load();
  // The two kernels write different rows, so the second starts as the first one's SMs fall free (an empty grouped kernel
  // costs 8 us by itself).
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * d->expert_clusters));
  cfg.blockDim = dim3(awq::grp::THREADS);
  cfg.dynamicSmemBytes = awq::grp::SMEM_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (gated)
    AWQ_CUDA(cudaLaunchKernelEx(&cfg, awq::grp::w4a16_experts_kernel<true>, tmX[0], tmX[1], tmX[2], tmC, q));
  else
    AWQ_CUDA(cudaLaunchKernelEx(&cfg, awq::grp::w4a16_experts_kernel<false>, tmX[0], tmX[1], tmX[2], tmC, q));
  AWQ_TRY(check_launch("w4a16_experts_kernel"));
  return ok();
}
