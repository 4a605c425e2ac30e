// The tails of pa_decode_shared (the decode kernels' partition pass over the
// tokens behind each request's shared part) and the merge that joins each
// request's shared and tail results, with their launchers.

#include <climits>

#include "pa_gqa.cuh"
#include "pa_launch.h"
#include "pa_rows.cuh"

namespace pa {

// One warp per (request, head): slots 0 .. of the shared part's partitions of
// P_shared keys, then slots part0 .. of the tail's.
template <int D>
__global__ void __launch_bounds__(128)
    shared_merge_kernel(const DecodeParamsTail p, int P_shared, pa_dtype out_dt, int S) {
  const int lane = threadIdx.x & 31;
  const int64_t ih = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const bool live = ih < static_cast<int64_t>(p.B) * p.H;
  int L = 0, sh = 0;
  if (live) {  // inputs of the passes before, not their results
    L = min(__ldg(p.seq_lens + ih / p.H), p.MB * S);
    sh = shared_part(__ldg(p.shared_lens + ih / p.H), L, p.shared_cap, S);
  }
  grid_dependency_wait();
  if (!live) return;
  const int tail = max(0, min(L - sh, p.L_cap));
  merge_row<D>(p.ws_m, p.ws_l, p.ws_acc, ih, p.NP, 0, (sh + P_shared - 1) / P_shared, p.part0,
               (tail + p.P - 1) / p.P, p.out, out_dt, lane);
}

namespace host {
namespace {

// The tails' launch. Right behind the shared part's pass it is a programmatic
// dependent of it, which lets its CTAs take the SMs that the last wave of that
// pass leaves idle: both only read the inputs and write slots of their own. The
// merge, the next dependent, needs both passes; so the grid has a plane more,
// one CTA of which waits for the shared part's pass to be done (blockIdx.z == B).
template <typename Kern, typename... Args>
pa_status launch_tail_pass(Kern kern, dim3 grid, int threads, int smem, bool overlap,
                           cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = overlap ? dim3(grid.x, grid.y, grid.z + 1) : grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = overlap ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? cuda_status() : PA_ERR_CUDA;
}

// One KV head per query head: one CTA per (partition, head, request).
template <typename T, int D, int S, bool WIDE>
pa_status tails_single(const DecodeParamsTail& prm, cudaStream_t stream) {
  using Tl = DecodeTiling<D, S, 2, WIDE>;
  auto kern = paged_decode_partition_kernel<T, float, D, S, false, T, false, DecodeParamsTail, WIDE>;
  static bool configured[kMaxDevices] = {};
  if (!opt_in_smem(kern, Tl::SMEM, configured)) return PA_ERR_CUDA;
  return launch_tail_pass(kern, dim3(prm.tail_parts, prm.H, prm.B), Tl::NW * 32, Tl::SMEM,
                          prm.part0 > 0, stream, prm);
}

// (wide CTAs for up to four of them per SM, as pa_decode's)
template <typename T, int D, int S>
pa_status tails_single(const DecodeParamsTail& prm, cudaStream_t stream) {
  constexpr bool two = DecodeTiling<D, S, 2, false>::NW != DecodeTiling<D, S, 2, true>::NW;
  const int64_t ctas = static_cast<int64_t>(prm.tail_parts) * prm.H * prm.B;
  if (two && ctas <= 4 * static_cast<int64_t>(sm_count()))
    return tails_single<T, D, S, two>(prm, stream);
  return tails_single<T, D, S, false>(prm, stream);
}

// Grouped heads: one CTA per (partition, KV head and chunk of 16 heads, request).
template <typename T, int D, int S, int NHT>
pa_status tails_grouped(const DecodeParamsTail& prm, cudaStream_t stream) {
  using Tg = GqaTiling<D, 2>;
  auto kern = paged_decode_gqa_kernel<T, float, D, S, false, NHT, T, DecodeParamsTail>;
  static bool configured[kMaxDevices] = {};
  if (!opt_in_smem(kern, Tg::SMEM, configured)) return PA_ERR_CUDA;
  const int64_t rows = static_cast<int64_t>(prm.NB) * prm.Hkv * S;
  const pa_dtype dt = std::is_same<T, __half>::value ? PA_F16 : PA_BF16;
  CUtensorMap tmk, tmv;
  if (!row_map_now(&tmk, prm.k_cache, rows, D, S < 16 ? S : 16, dt) ||
      !row_map_now(&tmv, prm.v_cache, rows, D, S < 16 ? S : 16, dt))
    return PA_ERR_CUDA;
  const int G = prm.H / prm.Hkv;
  const dim3 grid(prm.tail_parts, prm.Hkv * ((G + 15) / 16), prm.B);
  return launch_tail_pass(kern, grid, (Tg::NC + 1) * 32, Tg::SMEM, prm.part0 > 0, stream, prm, tmk,
                          tmv);
}

template <typename T>
pa_status tails(const DecodeParamsTail& prm, int D, int S, cudaStream_t st) {
  const int G = prm.H / prm.Hkv;
#define PA_CASE(DD, SS)                                    \
  if (D == DD && S == SS)                                  \
    return G == 1  ? tails_single<T, DD, SS>(prm, st)      \
           : G > 8 ? tails_grouped<T, DD, SS, 2>(prm, st)  \
                   : tails_grouped<T, DD, SS, 1>(prm, st);
  PA_CASE(64, 8) PA_CASE(64, 16) PA_CASE(64, 32)
  PA_CASE(128, 8) PA_CASE(128, 16) PA_CASE(128, 32)
  PA_CASE(256, 8) PA_CASE(256, 16) PA_CASE(256, 32)
#undef PA_CASE
  return PA_ERR_INVALID;
}

template <int D>
pa_status merge(const DecodeParamsTail& prm, int P_shared, pa_dtype out_dt, int S,
                cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  const int64_t pairs = static_cast<int64_t>(prm.B) * prm.H;
  cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(pairs, 4)));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  // (nothing was launched before it where no request can have a key: what runs
  // before is then not ours, and it reads the lengths only after that)
  cfg.numAttrs = prm.NP > 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, shared_merge_kernel<D>, prm, P_shared, out_dt, S) == cudaSuccess
             ? cuda_status()
             : PA_ERR_CUDA;
}

}  // namespace

pa_status launch_tails(const DecodeParamsTail& prm, pa_dtype dt, int D, int S,
                       cudaStream_t stream) {
  return dt == PA_F16 ? tails<__half>(prm, D, S, stream) : tails<__nv_bfloat16>(prm, D, S, stream);
}

pa_status launch_shared_merge(const DecodeParamsTail& prm, int P_shared, pa_dtype out_dt, int D,
                              int S, cudaStream_t stream) {
  if (D == 64) return merge<64>(prm, P_shared, out_dt, S, stream);
  if (D == 128) return merge<128>(prm, P_shared, out_dt, S, stream);
  return merge<256>(prm, P_shared, out_dt, S, stream);
}

bool take_error_shared(unsigned int* bits) { return take_error_word(bits); }

}  // namespace host
}  // namespace pa
