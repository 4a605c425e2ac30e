// The tails of pa_decode_shared (the decode kernels' partition pass over the
// tokens behind each request's shared part) and the merge that joins each
// request's shared and tail results, with their launchers.

#include <climits>

#include "pa_gqa.cuh"
#include "pa_launch.h"
#include "pa_rows.cuh"

namespace pa {

// Whether this warp's DL values per lane of `na` rows of partial results hold an
// infinity or a NaN.
template <int D>
__device__ __forceinline__ bool any_unbounded(const float* acc, int na, int lane) {
  bool bad = false;
  for (int q = 0; q < na; ++q)
    for (int d = lane; d < D; d += 32)
      bad |= !(fabsf(acc[static_cast<int64_t>(q) * D + d]) < INFINITY);
  return __any_sync(kFullMask, bad);
}

// One (request, head)'s result over its first `n` tokens, by one warp with plain
// loads, into slot 0 of its partial results: m and l in base 2, lane's D / 32
// columns of O. About a microsecond per token; see where it is called.
template <int D>
__device__ __noinline__ void own_part(const DecodeParamsTail& p, int64_t ih, int n, pa_dtype dt,
                                      int S, int lane) {
  constexpr int DL = D / 32;
  const bool bf = dt == PA_BF16;
  auto widen = [&](const uint16_t* src, float (&f)[DL]) {
#pragma unroll
    for (int e = 0; e < DL; ++e)
      f[e] = bf ? Elem<__nv_bfloat16>::one(src[e]) : Elem<__half>::one(src[e]);
  };
  const int i = static_cast<int>(ih / p.H);
  const int hk = static_cast<int>(ih - static_cast<int64_t>(i) * p.H) / (p.H / p.Hkv);
  const int32_t* table = p.block_tables + static_cast<int64_t>(i) * p.MB;
  float q[DL], o[DL], x[DL];
  widen(static_cast<const uint16_t*>(p.q) + ih * D + lane * DL, q);
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < DL; ++e) o[e] = 0.f;
  for (int tok = 0; tok < n; ++tok) {
    const int id = table[tok / S];
    if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.NB)) {
      raise_error(PA_DEVERR_BLOCK_ID);
      continue;
    }
    const int64_t at =
        ((static_cast<int64_t>(id) * p.Hkv + hk) * S + tok % S) * D + lane * DL;
    widen(static_cast<const uint16_t*>(p.k_cache) + at, x);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < DL; ++e) s = fmaf(q[e], x[e], s);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(kFullMask, s, off);
    s *= p.q_scale;
    const float mn = fmaxf(m, s);
    const float mr = mn == -INFINITY ? 0.f : mn;
    const float alpha = exp2f(m - mr), w = exp2f(s - mr);
    l = fmaf(l, alpha, w);
    widen(static_cast<const uint16_t*>(p.v_cache) + at, x);
#pragma unroll
    for (int e = 0; e < DL; ++e) o[e] = fmaf(o[e], alpha, w * x[e]);
    m = mn;
  }
  float* acc = p.ws_acc + ih * p.NP * D + lane * DL;
#pragma unroll
  for (int e = 0; e < DL; ++e) acc[e] = o[e];
  if (lane == 0) {
    p.ws_m[ih * p.NP] = m;
    p.ws_l[ih * p.NP] = l;
  }
  __syncwarp();
}

// One warp per (request, head): slots 0 .. of the shared part's partitions of
// P_shared keys, then slots part0 .. of the tail's.
//
// The group's product runs over the longest request's tokens; a request that ends
// before has zero weights there, and 0 times an infinity or a NaN in V is NaN. So
// where such a request's partial results are not all finite, the warp works its
// part out anew over the tokens that it sees. (Nothing else looks for it: a
// request that names all shared tokens pays one comparison.)
template <int D>
__global__ void __launch_bounds__(128)
    shared_merge_kernel(const __grid_constant__ DecodeParamsTail p, int P_shared, pa_dtype dt,
                        pa_dtype out_dt, int S) {
  const int lane = threadIdx.x & 31;
  const int64_t ih = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const bool live = ih < static_cast<int64_t>(p.B) * p.H;
  int L = 0, sh = 0;
  bool cut = false;
  if (live) {  // inputs of the passes before, not their results
    const int shared = __ldg(p.shared_lens + ih / p.H), len = __ldg(p.seq_lens + ih / p.H);
    L = min(len, p.MB * S);
    sh = shared_part(shared, L, p.shared_cap, S);
    // (the passes check the same, but a bound of zero leaves its pass out)
    if (lane == 0 && (len < 0 || len > p.MB * S || L - sh > p.L_cap || shared < 0 ||
                      shared > p.shared_cap))
      raise_error(PA_DEVERR_SEQ_LEN);
    if (ih == 0 && lane == 0 && p.part0 > 0 &&
        (__ldg(p.group_start) != 0 || __ldg(p.group_start + p.NG) != p.B))
      raise_error(PA_DEVERR_SEQ_LEN);  // requests outside every group
    cut = sh < shared_part(shared, p.shared_cap, p.shared_cap, S);
  }
  grid_dependency_wait();
  if (!live) return;
  const int tail = max(0, min(L - sh, p.L_cap));
  int na = (sh + P_shared - 1) / P_shared;
  if (cut && any_unbounded<D>(p.ws_acc + ih * p.NP * D, na, lane)) {
    own_part<D>(p, ih, sh, dt, S, lane);
    na = 1;
  }
  merge_row<D>(p.ws_m, p.ws_l, p.ws_acc, ih, p.NP, 0, na, p.part0, (tail + p.P - 1) / p.P, p.out,
               out_dt, lane);
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
pa_status merge(const DecodeParamsTail& prm, int P_shared, pa_dtype dt, pa_dtype out_dt, int S,
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
  return cudaLaunchKernelEx(&cfg, shared_merge_kernel<D>, prm, P_shared, dt, out_dt, S) ==
                 cudaSuccess
             ? cuda_status()
             : PA_ERR_CUDA;
}

}  // namespace

pa_status launch_tails(const DecodeParamsTail& prm, pa_dtype dt, int D, int S,
                       cudaStream_t stream) {
  return dt == PA_F16 ? tails<__half>(prm, D, S, stream) : tails<__nv_bfloat16>(prm, D, S, stream);
}

pa_status launch_shared_merge(const DecodeParamsTail& prm, int P_shared, pa_dtype dt,
                              pa_dtype out_dt, int D, int S, cudaStream_t stream) {
  if (D == 64) return merge<64>(prm, P_shared, dt, out_dt, S, stream);
  if (D == 128) return merge<128>(prm, P_shared, dt, out_dt, S, stream);
  return merge<256>(prm, P_shared, dt, out_dt, S, stream);
}

bool take_error_shared(unsigned int* bits) { return take_error_word(bits); }

}  // namespace host
}  // namespace pa
