// Kernels of pa_rope, pa_rope_append and pa_rope_append_fp8, for both 16-bit
// types, both pair layouts and every head size, and their launcher.

#include <algorithm>

#include "pa_launch.h"
#include "pa_rope.cuh"

namespace pa {
namespace host {
namespace {

template <typename T, int LAYOUT, int MODE, int EPT, int LPR>
pa_status launch(RopeParams prm, cudaStream_t stream) {
  // Tokens that fill the GPU go kRopeTokens (as many as leave four CTAs per SM,
  // about 1,000 threads' rows each) to a CTA. Fewer tokens than two CTAs per
  // SM have their rows spread over CTAs, down to one row per thread.
  constexpr int RPP = 256 / LPR;
  const int64_t sms = sm_count();
  const int64_t most = ceil_div(prm.rows, RPP);
  int64_t chunks = std::max<int64_t>(1, std::min(most, ceil_div(2 * sms, prm.T)));
  prm.chunk_rows = static_cast<int>(ceil_div(ceil_div(prm.rows, chunks), RPP) * RPP);
  chunks = ceil_div(prm.rows, prm.chunk_rows);
  prm.chunks = static_cast<int>(chunks);
  if (chunks == 1) prm.chunk_rows = prm.rows;
  prm.toks = 1;
  if (chunks == 1)
    while (prm.toks < kRopeTokens && prm.toks * prm.rows < 16 * RPP &&
           static_cast<int64_t>(prm.T) >= 2 * prm.toks * 4 * sms)
      prm.toks *= 2;
  const int64_t groups = ceil_div(prm.T, prm.toks);
  rope_kernel<T, LAYOUT, MODE, EPT, LPR>
      <<<static_cast<unsigned>(groups * chunks), 256, 0, stream>>>(prm);
  return cuda_status();
}

template <typename T, int LAYOUT, int MODE, int EPT>
pa_status by_size(const RopeParams& prm, cudaStream_t st) {
  if (prm.D <= 64) return launch<T, LAYOUT, MODE, EPT, 64 / EPT>(prm, st);
  if (prm.D <= 128) return launch<T, LAYOUT, MODE, EPT, 128 / EPT>(prm, st);
  return launch<T, LAYOUT, MODE, EPT, 256 / EPT>(prm, st);
}

// 16 elements per thread where head and rotation are multiples of 16 (in the
// half layout each piece is then 8 aligned elements on one side of the
// rotation's end), else 8, in the half layout one by one.
template <typename T, int MODE>
pa_status by_layout(const RopeParams& prm, int interleaved, cudaStream_t st) {
  if (interleaved)
    return prm.D % 16 == 0 ? by_size<T, kPairs, MODE, 16>(prm, st)
                           : by_size<T, kPairs, MODE, 8>(prm, st);
  return prm.D % 16 == 0 && prm.rot % 16 == 0 ? by_size<T, kHalf, MODE, 16>(prm, st)
                                              : by_size<T, kHalfAny, MODE, 8>(prm, st);
}

template <typename T>
pa_status by_mode(const RopeParams& prm, int interleaved, int mode, cudaStream_t st) {
  switch (mode) {
    case kNoCache: return by_layout<T, kNoCache>(prm, interleaved, st);
    case kCache16: return by_layout<T, kCache16>(prm, interleaved, st);
    case kCache8: return by_layout<T, kCache8>(prm, interleaved, st);
  }
  return PA_ERR_INVALID;
}

}  // namespace

pa_status launch_rope(const RopeParams& prm, pa_dtype dt, int interleaved, int mode,
                      cudaStream_t stream) {
  return dt == PA_BF16 ? by_mode<__nv_bfloat16>(prm, interleaved, mode, stream)
                       : by_mode<__half>(prm, interleaved, mode, stream);
}

bool take_error_rope(unsigned int* bits) { return take_error_word(bits); }

}  // namespace host
}  // namespace pa
