// Kernels of pa_cross and of the shared part of pa_decode_shared: attention of
// packed query rows over whole paged key ranges (rows_kernel), the merge of
// pa_cross's partitions, and their launchers.

#include <algorithm>
#include <type_traits>

#include "pa_launch.h"
#include "pa_rows.cuh"

namespace pa {
namespace host {
namespace {

template <typename T, int D, bool KSPLIT>
pa_status launch(RowsParams prm, const void* q, cudaStream_t stream) {
  using Tl = RowsTiling<D, KSPLIT>;
  auto kern = rows_kernel<T, D, KSPLIT>;
  static bool configured[kMaxDevices] = {};
  if constexpr (Tl::PASS_REGS) {
    // the softmax warps would wait for good for registers the launch did not bring
    // (the package's build refuses such a kernel, build.py; other builds end here)
    static const int regs = [&] {
      cudaFuncAttributes at = {};
      return cudaFuncGetAttributes(&at, kern) == cudaSuccess ? at.numRegs : 0;
    }();
    if (regs < Tl::LAUNCH_REGS) return PA_ERR_CUDA;
  }
  if (!opt_in_smem(kern, Tl::SMEM, configured)) return PA_ERR_CUDA;
  const pa_dtype dt = std::is_same<T, __half>::value ? PA_F16 : PA_BF16;
  const int64_t rows = static_cast<int64_t>(prm.NB) * prm.Hkv * prm.S;
  CUtensorMap tmq, tmk, tmv;
  if (!query_rows_map(&tmq, q, prm.T, prm.H, D, prm.H / prm.Hkv, prm.qpt, dt) ||
      !row_map_now(&tmk, prm.k_cache, rows, D, std::min(prm.S, Tl::BN), dt) ||
      !row_cols_map(&tmv, prm.v_cache, rows, D, std::min(prm.S, Tl::BN), dt))
    return PA_ERR_CUDA;
  const int64_t groups = ceil_div(prm.max_rows, Tl::NQ * prm.qpt);
  const dim3 grid(static_cast<unsigned>(groups * prm.Hkv), prm.parts, prm.items);
  prm.longest_first = !prm.shared_lens && prm.items > 1 && prm.items <= 32 &&
                      static_cast<int64_t>(grid.x) * grid.y * grid.z > Tl::CTAS * sm_count();
  kern<<<grid, Tl::THREADS, Tl::SMEM, stream>>>(prm, tmq, tmk, tmv);
  return cuda_status();
}

template <typename T>
pa_status by_size(const RowsParams& prm, const void* q, int D, bool split_keys, cudaStream_t st) {
  if (D == 64 && split_keys) return launch<T, 64, true>(prm, q, st);
  if (D == 128)
    return split_keys ? launch<T, 128, true>(prm, q, st) : launch<T, 128, false>(prm, q, st);
  if (D == 256 && !split_keys) return launch<T, 256, false>(prm, q, st);
  return PA_ERR_INVALID;
}

template <int D>
pa_status merge(const RowsParams& prm, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(static_cast<int64_t>(prm.max_rows) * prm.H, 4)),
                     prm.items);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cross_merge_kernel<D>, prm) == cudaSuccess ? cuda_status()
                                                                            : PA_ERR_CUDA;
}

}  // namespace

pa_status launch_rows(const RowsParams& prm, const void* q, pa_dtype dt, int D, bool split_keys,
                      cudaStream_t stream) {
  return dt == PA_BF16 ? by_size<__nv_bfloat16>(prm, q, D, split_keys, stream)
                       : by_size<__half>(prm, q, D, split_keys, stream);
}

pa_status launch_cross_merge(const RowsParams& prm, int D, cudaStream_t stream) {
  if (prm.parts <= 1) return PA_OK;
  if (D == 64) return merge<64>(prm, stream);
  if (D == 128) return merge<128>(prm, stream);
  return merge<256>(prm, stream);
}

bool take_error_rows(unsigned int* bits) { return take_error_word(bits); }

}  // namespace host
}  // namespace pa
