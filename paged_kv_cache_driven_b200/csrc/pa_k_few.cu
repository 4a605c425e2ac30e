// The grouped-query kernel on few packed query rows over whole key ranges
// (pa_cross with few rows, and the shared part of small groups in
// pa_decode_shared), and its launcher.

#include <type_traits>

#include "pa_gqa.cuh"
#include "pa_launch.h"

namespace pa {
namespace host {
namespace {

// One CTA per (partition, KV head, item).
template <typename T, typename TO, int D, int S, int NHT>
pa_status launch(const DecodeParamsFew& prm, cudaStream_t stream) {
  using Tg = GqaTiling<D, 2>;
  auto kern = paged_decode_gqa_kernel<T, TO, D, S, false, NHT, T, DecodeParamsFew>;
  static bool configured[kMaxDevices] = {};
  if (!opt_in_smem(kern, Tg::SMEM, configured)) return PA_ERR_CUDA;
  const int64_t rows = static_cast<int64_t>(prm.NB) * prm.Hkv * S;
  const pa_dtype dt = std::is_same<T, __half>::value ? PA_F16 : PA_BF16;
  CUtensorMap tmk, tmv;
  if (!row_map_now(&tmk, prm.k_cache, rows, D, S < 16 ? S : 16, dt) ||
      !row_map_now(&tmv, prm.v_cache, rows, D, S < 16 ? S : 16, dt))
    return PA_ERR_CUDA;
  const dim3 grid(prm.parts, prm.Hkv, prm.items);
  kern<<<grid, (Tg::NC + 1) * 32, Tg::SMEM, stream>>>(prm, tmk, tmv);
  return cuda_status();
}

template <typename T, typename TO>
pa_status by_shape(const DecodeParamsFew& prm, int D, int S, cudaStream_t st) {
  const bool wide = prm.max_rows * (prm.H / prm.Hkv) > 8;  // two 8-row column tiles per CTA
#define PA_CASE(DD, SS) \
  if (D == DD && S == SS) \
    return wide ? launch<T, TO, DD, SS, 2>(prm, st) : launch<T, TO, DD, SS, 1>(prm, st);
  PA_CASE(64, 8) PA_CASE(64, 16) PA_CASE(64, 32) PA_CASE(64, 64) PA_CASE(64, 128)
  PA_CASE(128, 8) PA_CASE(128, 16) PA_CASE(128, 32) PA_CASE(128, 64) PA_CASE(128, 128)
  PA_CASE(256, 8) PA_CASE(256, 16) PA_CASE(256, 32) PA_CASE(256, 64) PA_CASE(256, 128)
#undef PA_CASE
  return PA_ERR_INVALID;
}

template <typename T>
pa_status by_out(const DecodeParamsFew& prm, pa_dtype out_dt, int D, int S, cudaStream_t st) {
  switch (out_dt) {
    case PA_F32: return by_shape<T, float>(prm, D, S, st);
    case PA_F16: return by_shape<T, __half>(prm, D, S, st);
    case PA_BF16: return by_shape<T, __nv_bfloat16>(prm, D, S, st);
  }
  return PA_ERR_INVALID;
}

}  // namespace

pa_status launch_few(const DecodeParamsFew& prm, pa_dtype dt, pa_dtype out_dt, int D, int S,
                     cudaStream_t stream) {
  // (the plan sends no more here: a CTA's columns are all the rows of its KV head)
  if (static_cast<int64_t>(prm.max_rows) * (prm.H / prm.Hkv) > 16) return PA_ERR_INVALID;
  return dt == PA_BF16 ? by_out<__nv_bfloat16>(prm, out_dt, D, S, stream)
                       : by_out<__half>(prm, out_dt, D, S, stream);
}

bool take_error_few(unsigned int* bits) { return take_error_word(bits); }

}  // namespace host
}  // namespace pa
