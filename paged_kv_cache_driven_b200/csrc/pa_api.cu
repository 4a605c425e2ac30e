// The C-ABI layer (pagedattn.h): argument validation, launch planning, the
// split-KV workspace layout, tensor-map encoding and dispatch to the launchers
// of the translation units that hold the kernels (pa_k_*.cu), the device
// error words, and pa_decode_noalloc's static scratch. Every check runs on the
// host before anything is launched.

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "pa_launch.h"
#include "pagedattn.h"

using pa::host::ceil_div;
using pa::host::kMaxDevices;

namespace {

constexpr int kDefaultPartition = 512;  // tokens per split-KV partition when splitting

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool cache_dtype_ok(pa_dtype dt) { return dt == PA_F16 || dt == PA_BF16; }

bool out_dtype_ok(pa_dtype dt) { return dt == PA_F16 || dt == PA_BF16 || dt == PA_F32; }

bool decode_shape_ok(int D, int S) {
  return (D == 64 || D == 128 || D == 256) && (S == 8 || S == 16 || S == 32);
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

using pa::host::sm_count;

// Chooses the partition length. Returns false on an invalid `partition`.
//   -1      never split: one partition covering any length up to MB * S
//   > 0     that many tokens (a multiple of S)
//   0       automatic: 512-token partitions, halved (down to 64 tokens, staying a
//           multiple of S) while the grid would hold fewer CTAs than the device
//           has SMs, so that small batches still spread over every SM; no split
//           if one partition covers every request. (Measured at batch 1, 32
//           heads, 1.3K tokens: 256-token partitions, 192 CTAs, are fastest for
//           head sizes 64 to 256; 64-token ones, 672 CTAs, are 40 % slower,
//           each CTA's fixed start and end costing more than its short stream.)
//           Contexts of 32K tokens and more take partitions of up to 2048
//           tokens while the grid keeps 8 CTAs per SM.
//           A small grid then has a partition count of 3, 5, 6 or 7 rounded
//           to a power of two (the next, else the previous; partitions re-cut
//           evenly in whole blocks) when the grid stays within two CTAs per SM,
//           so that its split can merge inside a cluster (cluster_merge).
bool plan(int B, int H, int S, int max_seq_len, int partition, int* P_out, int* NP_out) {
  if (max_seq_len < 0 || S <= 0) return false;
  int P;
  if (partition < 0) {
    if (partition != -1) return false;
    *P_out = 0;
    *NP_out = 1;
    return true;
  } else if (partition > 0) {
    if (partition % S != 0) return false;
    P = partition;
  } else {
    P = kDefaultPartition;
    const int64_t target = sm_count();
    const int64_t pairs = static_cast<int64_t>(B > 0 ? B : 1) * (H > 0 ? H : 1);
    while (P > 64 && (P / 2) % S == 0 && pairs * ceil_div(max_seq_len, P) < target) P /= 2;
    // long contexts (32K tokens and more) take partitions of up to 2048 tokens
    // while the grid keeps at least 8 CTAs per SM: fewer partials and per-CTA
    // starts (8 x U[32K, 131K] tokens on 32 heads: 1.627 ms against 1.658 ms
    // at 512; shorter requests run best at 512)
    if (max_seq_len >= 32768)
      while (P < 2048 && pairs * ceil_div(max_seq_len, 2 * P) >= 8 * target) P *= 2;
    const int64_t n = ceil_div(max_seq_len, P);
    if (n > 2 && n < 8 && (n & (n - 1)) != 0) {
      const int64_t up = n < 4 ? 4 : 8;
      for (const int64_t c : {up, up / 2}) {
        if (pairs * c > 2 * target) continue;
        // c partitions of a whole number of blocks; where blocks do not divide
        // evenly the last one or two hold no token (they only join the merge)
        *P_out = static_cast<int>(ceil_div(ceil_div(max_seq_len, c), S) * S);
        *NP_out = static_cast<int>(c);
        return true;
      }
    }
  }
  const int64_t np = ceil_div(max_seq_len, P);
  if (np <= 1) {
    *P_out = 0;
    *NP_out = 1;
    return true;
  }
  if (np * P > INT_MAX) return false;
  *P_out = P;
  *NP_out = static_cast<int>(np);
  return true;
}

// The automatic plan for grouped-query heads (Hkv < H): the partition pass then
// has B * Hkv * ceil(G / 16) CTAs per partition (G = H / Hkv), up to 16 query
// heads per CTA. Where that grid at 512-token partitions holds at most two
// CTAs per SM, the partitions are halved (down to 128 tokens, multiples of S)
// while the grid stays within that bound: a small grid is resident at once,
// so shorter partitions shorten every CTA's stream (64 query heads on 8 KV
// heads, head_dim 128: one request of 1,332 tokens 19.5 -> 15.4 us, four of
// 2,048 23.6 -> 19.5 us). Larger grids, explicit partitions and one KV head per
// query head take plan().
bool plan_grouped(int B, int H, int Hkv, int S, int max_seq_len, int partition, int* P_out,
                  int* NP_out) {
  if (Hkv <= 0 || Hkv >= H || H % Hkv != 0 || partition != 0 || max_seq_len < 0 || S <= 0)
    return plan(B, H, S, max_seq_len, partition, P_out, NP_out);
  const int64_t ctas = static_cast<int64_t>(B > 0 ? B : 1) * Hkv * ceil_div(H / Hkv, 16);
  const int64_t cap = 2 * static_cast<int64_t>(sm_count());
  int P = kDefaultPartition;
  if (ctas * ceil_div(max_seq_len, P) > cap) return plan(B, H, S, max_seq_len, 0, P_out, NP_out);
  while (P > 128 && (P / 2) % S == 0 && ctas * ceil_div(max_seq_len, P / 2) <= cap) P /= 2;
  const int64_t np = ceil_div(max_seq_len, P);
  *P_out = np <= 1 ? 0 : P;
  *NP_out = np <= 1 ? 1 : static_cast<int>(np);
  return true;
}

// Whether a partition pass of B x H x NP CTAs holds at most two CTAs per SM
// (a small grid: resident at once, so its split can merge inside clusters).
bool small_grid(int B, int H, int NP) {
  return static_cast<int64_t>(B) * H * NP <= 2 * static_cast<int64_t>(sm_count());
}

// Whether the partition pass takes its wide CTA shapes (DecodeTiling, WIDE):
// grids of at most four CTAs per SM, the small grids among them (head_dim 64,
// block 8, 512 CTAs: 21.5 us wide against 23.6 narrow).
bool wide_grid(int B, int H, int NP) {
  return static_cast<int64_t>(B) * H * NP <= 4 * static_cast<int64_t>(sm_count());
}

// Whether an automatic split of NP partitions over B x H (request, head) pairs
// merges inside clusters instead of through the workspace and the merge
// kernel: NP is a portable cluster size (2, 4 or 8; the cluster spans the
// grid's x dimension, the partitions of one pair), and the grid fits within two
// CTAs per SM, so that it is resident at once and the CTAs that wait at their
// cluster's barrier hold no SM another CTA is queued for. Large grids keep the
// merge kernel, which overlaps their last wave.
bool cluster_merge(int B, int H, int NP) {
  if (NP != 2 && NP != 4 && NP != 8) return false;
  return small_grid(B, H, NP);
}

// Split-KV workspace: m and l [B, H, NP], then (256-byte aligned) acc [B, H, NP, D].
size_t acc_offset(size_t n) { return align256(n * 2 * sizeof(float)); }

size_t workspace_for(int B, int H, int D, int NP) {
  if (NP <= 1) return 0;
  const size_t n = static_cast<size_t>(B) * H * NP;
  return acc_offset(n) + n * D * sizeof(float);
}

// Points the kernel parameters at the workspace parts for NP > 1 partitions.
void set_split(pa::DecodeParams& prm, void* workspace, int B, int H, int P, int NP,
               int64_t L_max) {
  const size_t n = static_cast<size_t>(B) * H * NP;
  uint8_t* base = static_cast<uint8_t*>(workspace);
  prm.ws_m = reinterpret_cast<float*>(base);
  prm.ws_l = prm.ws_m + n;
  prm.ws_acc = reinterpret_cast<float*>(base + acc_offset(n));
  prm.P = P;
  prm.NP = NP;
  prm.L_cap = static_cast<int>(std::min<int64_t>(L_max, static_cast<int64_t>(NP) * P));
}

// ---- tensor maps of the caches, for the tiled TMA loads ---------------------
// Each cache [NB, Hkv, S, D] is viewed as a 2-D array of NB * Hkv * S rows of D
// elements; a box is 64 elements x min(S, 16) rows with the 128-byte swizzle.
// Encoding goes through the driver's cuTensorMapEncodeTiled (looked up once);
// the last few maps are kept, keyed by everything they encode, since a cache is
// decoded over and over.

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

struct RowMapKey {
  const void* base;
  int64_t rows;
  int D, box_rows, dt;
  bool operator==(const RowMapKey& o) const {
    return base == o.base && rows == o.rows && D == o.D && box_rows == o.box_rows && dt == o.dt;
  }
};

}  // namespace

namespace pa {
namespace host {

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    cudaGetLastError();  // clear the error state of the failed query
    return 148;
  }
  return n;
}

// kind: 0 = f16, 1 = bf16: boxes of 64 elements, so every box row is 128 bytes,
// the 128-byte swizzle's width; 2 = one-byte E4M3 codes: a box spans the whole
// D-byte row, unswizzled (the consumer converts it to 16-bit tiles itself).
static bool encode_row_map(CUtensorMap* out, const void* base, int64_t rows, int D, int box_rows,
                           int kind) {
  auto fn = encode_fn();
  if (!fn) return false;
  const bool codes = kind == 2;
  const cuuint64_t esize = codes ? 1 : 2;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(D) * esize};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(codes ? D : 128 / esize),
                             static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  const CUtensorMapDataType type =
      codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8
            : (kind == 1 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16);
  return fn(out, type, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            codes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static bool row_map_kind(CUtensorMap* out, const void* base, int64_t rows, int D, int box_rows,
                         int kind) {
  static std::mutex mu;
  static RowMapKey keys[16];
  static CUtensorMap maps[16];
  static int used = 0, next = 0;
  const RowMapKey key{base, rows, D, box_rows, kind};
  std::lock_guard<std::mutex> lock(mu);
  for (int k = 0; k < used; ++k)
    if (keys[k] == key) {
      *out = maps[k];
      return true;
    }
  CUtensorMap map;
  if (!encode_row_map(&map, base, rows, D, box_rows, kind)) return false;
  const int slot = used < 16 ? used++ : next;
  next = (slot + 1) % 16;
  keys[slot] = key;
  maps[slot] = map;
  *out = map;
  return true;
}

bool row_map(CUtensorMap* out, const void* base, int64_t rows, int D, int box_rows, pa_dtype dt) {
  return row_map_kind(out, base, rows, D, box_rows, dt == PA_BF16 ? 1 : 0);
}

bool query_rows_map(CUtensorMap* out, const void* q, int64_t T, int H, int D, int heads, int rows,
                    pa_dtype dt) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H),
                              static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2,
                                 static_cast<cuuint64_t>(H) * D * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(rows)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(out, dt == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
            3, const_cast<void*>(q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool row_cols_map(CUtensorMap* out, const void* base, int64_t rows, int D, int box_rows,
                  pa_dtype dt) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t cols = static_cast<cuuint32_t>(D / 64);
  const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(rows), cols};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, 128};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), cols};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(out, dt == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
            3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool row_map_now(CUtensorMap* out, const void* base, int64_t rows, int D, int box_rows,
                 pa_dtype dt) {
  return encode_row_map(out, base, rows, D, box_rows, dt == PA_BF16 ? 1 : 0);
}

bool row_map_codes(CUtensorMap* out, const void* base, int64_t rows, int D, int box_rows) {
  return row_map_kind(out, base, rows, D, box_rows, 2);
}

// ---- paged prefill -------------------------------------------------------------
// The packed queries [T, H, D] as a 3-D tensor map (D, H, T) whose box is one
// 64-element column block of one head for 128 consecutive query rows; rows
// past T read as zeros.
bool query_map(CUtensorMap* out, const void* q, int64_t T, int H, int D, pa_dtype dt) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H),
                              static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2,
                                 static_cast<cuuint64_t>(H) * D * 2};
  const cuuint32_t box[3] = {64, 1, 128};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(out, dt == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
            3, const_cast<void*>(q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace host
}  // namespace pa

extern "C" {

const char* pa_status_string(pa_status s) {
  switch (s) {
    case PA_OK: return "PA_OK";
    case PA_ERR_INVALID: return "PA_ERR_INVALID";
    case PA_ERR_OOM: return "PA_ERR_OOM";
    case PA_ERR_OUT_OF_RANGE: return "PA_ERR_OUT_OF_RANGE";
    case PA_ERR_CUDA: return "PA_ERR_CUDA";
  }
  return "PA_ERR_UNKNOWN";
}

int pa_version(void) { return 100; }

pa_status pa_kv_append(const void* k, const void* v, const int64_t* slot_mapping, void* k_cache,
                       void* v_cache, int T, int H, int D, int S, int NB, pa_dtype dt,
                       void* stream) {
  if (T < 0 || H <= 0 || D <= 0 || S <= 0 || NB < 0 || !cache_dtype_ok(dt)) return PA_ERR_INVALID;
  if (D % 8 != 0) return PA_ERR_INVALID;  // rows move as 16-byte vectors
  if (T == 0) return PA_OK;
  if (!k || !v || !slot_mapping || !k_cache || !v_cache) return PA_ERR_INVALID;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache))
    return PA_ERR_INVALID;
  return pa::host::launch_kv_append(k, v, slot_mapping, k_cache, v_cache, T, H, D, S, NB,
                                    static_cast<cudaStream_t>(stream));
}

pa_status pa_copy_blocks(void* k_cache, void* v_cache, const int32_t* src_dst, int n, int H,
                         int S, int D, int NB, pa_dtype dt, void* stream) {
  if (n < 0 || H <= 0 || S <= 0 || D <= 0 || NB < 0 || !cache_dtype_ok(dt) || D % 8 != 0)
    return PA_ERR_INVALID;
  if (n == 0) return PA_OK;
  if (!k_cache || !v_cache || !src_dst || !aligned16(k_cache) || !aligned16(v_cache))
    return PA_ERR_INVALID;
  return pa::host::launch_copy_blocks(k_cache, v_cache, src_dst, n, H, S, D, NB,
                                      static_cast<cudaStream_t>(stream));
}

pa_status pa_decode_plan(int B, int H, int D, int S, int max_seq_len, int partition,
                         int* partition_tokens, int* num_partitions) {
  (void)B;
  (void)H;
  (void)D;
  if (!partition_tokens || !num_partitions) return PA_ERR_INVALID;
  int P, NP;
  if (!plan(B, H, S, max_seq_len, partition, &P, &NP)) return PA_ERR_INVALID;
  *partition_tokens = P;
  *num_partitions = NP;
  return PA_OK;
}

size_t pa_decode_workspace_bytes(int B, int H, int D, int S, int max_seq_len, int partition) {
  int P, NP;
  if (B < 0 || H <= 0 || D <= 0 || !plan(B, H, S, max_seq_len, partition, &P, &NP)) return 0;
  // grouped-query heads may split finer (plan_grouped); one KV head has the
  // fewest CTAs per partition and so the most partitions
  int Pg, NPg;
  if (H > 1 && plan_grouped(B, H, 1, S, max_seq_len, partition, &Pg, &NPg)) NP = std::max(NP, NPg);
  return workspace_for(B, H, D, NP);
}

pa_status pa_decode_plan_grouped(int B, int H, int Hkv, int D, int S, int max_seq_len,
                                 int partition, int* partition_tokens, int* num_partitions) {
  (void)D;
  if (!partition_tokens || !num_partitions || Hkv <= 0 || H <= 0 || H % Hkv != 0)
    return PA_ERR_INVALID;
  int P, NP;
  if (!plan_grouped(B, H, Hkv, S, max_seq_len, partition, &P, &NP)) return PA_ERR_INVALID;
  *partition_tokens = P;
  *num_partitions = NP;
  return PA_OK;
}

}  // extern "C"

namespace {

// The host checks of pa_decode's arguments, workspace aside (shared by its
// variants). On PA_OK, *P / *NP hold the plan and *noop is set for B == 0.
pa_status decode_check(const void* out, pa_dtype out_dt, const void* q, const void* k_cache,
                       const void* v_cache, const int32_t* block_tables, int MB,
                       const int32_t* seq_lens, float scale, int B, int H, int Hkv, int D, int S,
                       int NB, pa_dtype dt, int partition, int max_seq_len, int* P, int* NP,
                       bool* noop) {
  *noop = false;
  if (B < 0 || H <= 0 || NB < 0 || MB < 0) return PA_ERR_INVALID;
  if (Hkv <= 0 || H % Hkv != 0) return PA_ERR_INVALID;
  if (!cache_dtype_ok(dt) || !out_dtype_ok(out_dt) || !decode_shape_ok(D, S)) return PA_ERR_INVALID;
  if (!std::isfinite(scale)) return PA_ERR_INVALID;
  if (B > 65535 || H > 65535) return PA_ERR_INVALID;  // grid y / z limits
  const int64_t L_max = static_cast<int64_t>(MB) * S;
  if (L_max > INT_MAX || max_seq_len < 0 || max_seq_len > L_max) return PA_ERR_INVALID;
  if (!plan_grouped(B, H, Hkv, S, max_seq_len, partition, P, NP)) return PA_ERR_INVALID;
  if (B == 0) {
    *noop = true;
    return PA_OK;
  }
  if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens || MB == 0)
    return PA_ERR_INVALID;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
    return PA_ERR_INVALID;
  return PA_OK;
}

// pa_decode and pa_decode_append: k_new / v_new null = plain decode.
pa_status decode_impl(void* out, pa_dtype out_dt, const void* q, const void* k_new,
                      const void* v_new, const void* k_cache, const void* v_cache,
                      const int32_t* block_tables, int MB, const int32_t* seq_lens, float scale,
                      int B, int H, int Hkv, int D, int S, int NB, pa_dtype dt, int partition,
                      int max_seq_len, void* workspace, size_t ws_bytes, void* stream) {
  int P, NP;
  bool noop;
  const pa_status chk = decode_check(out, out_dt, q, k_cache, v_cache, block_tables, MB, seq_lens,
                                     scale, B, H, Hkv, D, S, NB, dt, partition, max_seq_len, &P,
                                     &NP, &noop);
  if (chk != PA_OK || noop) return chk;
  const int64_t L_max = static_cast<int64_t>(MB) * S;
  const size_t need = workspace_for(B, H, D, NP);
  if (need > 0 && (!workspace || ws_bytes < need || !aligned16(workspace))) return PA_ERR_INVALID;

  pa::DecodeParams prm{};
  prm.out = out;
  prm.q = q;
  prm.k_cache = k_cache;
  prm.v_cache = v_cache;
  prm.block_tables = block_tables;
  prm.seq_lens = seq_lens;
  prm.q_scale = scale * 1.4426950408889634f;  // log2(e)
  prm.v_scale = 1.f;
  prm.MB = MB;
  prm.B = B;
  prm.H = H;
  prm.Hkv = Hkv;
  prm.NB = NB;
  if (NP > 1) {
    set_split(prm, workspace, B, H, P, NP, L_max);
  } else {
    prm.P = static_cast<int>(L_max > 0 ? L_max : S);  // one partition covers every block
    prm.NP = 1;
    prm.L_cap = static_cast<int>(L_max);
  }
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  prm.k_new = k_new;
  prm.v_new = v_new;
  if (H != Hkv)  // (the grouped-query kernel always merges through the workspace)
    return pa::host::launch_grouped(prm, dt, out_dt, D, S, k_new != nullptr, st);
  const bool cluster = partition == 0 && cluster_merge(B, H, prm.NP);
  return pa::host::launch_decode16(prm, dt, out_dt, D, S, k_new != nullptr, cluster,
                                   wide_grid(B, H, prm.NP), st);
}

}  // namespace

extern "C" {

pa_status pa_decode(void* out, pa_dtype out_dt, const void* q, const void* k_cache,
                    const void* v_cache, const int32_t* block_tables, int MB,
                    const int32_t* seq_lens, float scale, int B, int H, int D, int S, int NB,
                    pa_dtype dt, int partition, int max_seq_len, void* workspace,
                    size_t ws_bytes, void* stream) {
  return decode_impl(out, out_dt, q, nullptr, nullptr, k_cache, v_cache, block_tables, MB,
                     seq_lens, scale, B, H, H, D, S, NB, dt, partition, max_seq_len, workspace,
                     ws_bytes, stream);
}

pa_status pa_decode_append(void* out, pa_dtype out_dt, const void* q, const void* k_new,
                           const void* v_new, void* k_cache, void* v_cache,
                           const int32_t* block_tables, int MB, const int32_t* seq_lens,
                           float scale, int B, int H, int D, int S, int NB, pa_dtype dt,
                           int partition, int max_seq_len, void* workspace, size_t ws_bytes,
                           void* stream) {
  if (B > 0 && (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new)))
    return PA_ERR_INVALID;
  return decode_impl(out, out_dt, q, B > 0 ? k_new : nullptr, v_new, k_cache, v_cache,
                     block_tables, MB, seq_lens, scale, B, H, H, D, S, NB, dt, partition,
                     max_seq_len, workspace, ws_bytes, stream);
}

pa_status pa_decode_gqa(void* out, pa_dtype out_dt, const void* q, const void* k_new,
                        const void* v_new, void* k_cache, void* v_cache,
                        const int32_t* block_tables, int MB, const int32_t* seq_lens, float scale,
                        int B, int H, int Hkv, int D, int S, int NB, pa_dtype dt, int partition,
                        int max_seq_len, void* workspace, size_t ws_bytes, void* stream) {
  if ((k_new == nullptr) != (v_new == nullptr)) return PA_ERR_INVALID;
  if (k_new && B > 0 && (!aligned16(k_new) || !aligned16(v_new))) return PA_ERR_INVALID;
  return decode_impl(out, out_dt, q, B > 0 ? k_new : nullptr, v_new, k_cache, v_cache,
                     block_tables, MB, seq_lens, scale, B, H, Hkv, D, S, NB, dt, partition,
                     max_seq_len, workspace, ws_bytes, stream);
}

pa_status pa_prefill(void* out, pa_dtype out_dt, const void* q, const void* k_cache,
                     const void* v_cache, const int32_t* block_tables, int MB,
                     const int32_t* seq_lens, const int32_t* q_start, float scale, int B, int H,
                     int Hkv, int D, int S, int NB, pa_dtype dt, int T, int max_q_len,
                     void* stream) {
  if (B < 0 || H <= 0 || Hkv <= 0 || H % Hkv != 0 || T < 0 || max_q_len < 0 || MB < 0 || NB < 0)
    return PA_ERR_INVALID;
  if (!cache_dtype_ok(dt) || !out_dtype_ok(out_dt)) return PA_ERR_INVALID;
  if (!(D == 64 || D == 128 || D == 256) || !(S == 8 || S == 16 || S == 32 || S == 64 || S == 128))
    return PA_ERR_INVALID;
  if (!std::isfinite(scale) || !(scale > 0.f)) return PA_ERR_INVALID;
  if (B == 0 || T == 0 || max_q_len == 0) return PA_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens || !q_start)
    return PA_ERR_INVALID;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
    return PA_ERR_INVALID;
  if (NB == 0 || static_cast<int64_t>(NB) * Hkv * S > INT_MAX) return PA_ERR_INVALID;
  // grid (H, row blocks of up to 256 rows, B): the y and z extents are 16-bit
  if (ceil_div(max_q_len, 128) > 65535 || B > 65535) return PA_ERR_INVALID;
  pa::PrefillParams prm;
  prm.out = out;
  prm.k_cache = k_cache;
  prm.v_cache = v_cache;
  prm.block_tables = block_tables;
  prm.seq_lens = seq_lens;
  prm.q_start = q_start;
  prm.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  prm.MB = MB;
  prm.B = B;
  prm.H = H;
  prm.Hkv = Hkv;
  prm.NB = NB;
  prm.T = T;
  prm.max_q_len = max_q_len;
  return pa::host::launch_prefill(prm, q, dt, out_dt, D, S, static_cast<cudaStream_t>(stream));
}

pa_status pa_kv_append_fp8(const void* k, const void* v, pa_dtype in_dt,
                           const int64_t* slot_mapping, void* k_cache, void* v_cache,
                           float k_scale, float v_scale, int T, int H, int D, int S, int NB,
                           void* stream) {
  if (T < 0 || H <= 0 || D <= 0 || S <= 0 || NB < 0 || !cache_dtype_ok(in_dt)) return PA_ERR_INVALID;
  if (D % 16 != 0) return PA_ERR_INVALID;  // 8-byte code vectors, 16-byte cache rows
  if (!(std::isfinite(k_scale) && k_scale > 0.f && std::isfinite(v_scale) && v_scale > 0.f))
    return PA_ERR_INVALID;
  if (T == 0) return PA_OK;
  if (!k || !v || !slot_mapping || !k_cache || !v_cache) return PA_ERR_INVALID;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache))
    return PA_ERR_INVALID;
  return pa::host::launch_kv_append_fp8(k, v, in_dt, slot_mapping, k_cache, v_cache, k_scale,
                                        v_scale, T, H, D, S, NB, static_cast<cudaStream_t>(stream));
}

// pa_decode_fp8 and pa_decode_append_fp8: k_new / v_new null = plain decode.
// pa_decode_gqa_fp8: Hkv < H (grouped-query heads; no fused append).
static pa_status decode_fp8_impl(void* out, pa_dtype out_dt, const void* q, pa_dtype q_dt,
                                 const void* k_new, const void* v_new, const void* k_cache,
                                 const void* v_cache, float k_scale, float v_scale,
                                 const int32_t* block_tables, int MB, const int32_t* seq_lens,
                                 float scale, int B, int H, int Hkv, int D, int S, int NB,
                                 int partition, int max_seq_len, void* workspace,
                                 size_t ws_bytes, void* stream) {
  if (B < 0 || H <= 0 || NB < 0 || MB < 0) return PA_ERR_INVALID;
  if (Hkv <= 0 || H % Hkv != 0 || (k_new && Hkv != H)) return PA_ERR_INVALID;
  if (!cache_dtype_ok(q_dt) || !out_dtype_ok(out_dt) || !decode_shape_ok(D, S)) return PA_ERR_INVALID;
  if (!std::isfinite(scale)) return PA_ERR_INVALID;
  if (!(std::isfinite(k_scale) && k_scale > 0.f && std::isfinite(v_scale) && v_scale > 0.f))
    return PA_ERR_INVALID;
  if (B > 65535 || H > 65535) return PA_ERR_INVALID;
  const int64_t L_max = static_cast<int64_t>(MB) * S;
  if (L_max > INT_MAX || max_seq_len < 0 || max_seq_len > L_max) return PA_ERR_INVALID;
  int P, NP;
  if (!plan_grouped(B, H, Hkv, S, max_seq_len, partition, &P, &NP)) return PA_ERR_INVALID;
  if (B == 0) return PA_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens || MB == 0)
    return PA_ERR_INVALID;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
    return PA_ERR_INVALID;
  const size_t need = workspace_for(B, H, D, NP);
  if (need > 0 && (!workspace || ws_bytes < need || !aligned16(workspace))) return PA_ERR_INVALID;
  pa::DecodeParams prm{};
  prm.out = out;
  prm.q = q;
  prm.k_cache = k_cache;
  prm.v_cache = v_cache;
  prm.block_tables = block_tables;
  prm.seq_lens = seq_lens;
  prm.q_scale = scale * k_scale * 1.4426950408889634f;  // K's scale folded into q, log2(e)
  prm.v_scale = v_scale;
  prm.MB = MB;
  prm.B = B;
  prm.H = H;
  prm.Hkv = Hkv;
  prm.NB = NB;
  if (NP > 1) {
    set_split(prm, workspace, B, H, P, NP, L_max);
  } else {
    prm.P = static_cast<int>(L_max > 0 ? L_max : S);
    prm.NP = 1;
    prm.L_cap = static_cast<int>(L_max);
  }
  if (Hkv != H)  // grouped-query heads: the tensor-core kernel
    return pa::host::launch_grouped_fp8(prm, q_dt, out_dt, D, S,
                                        static_cast<cudaStream_t>(stream));
  const bool append = k_new != nullptr;
  if (append && (!v_new || !aligned16(k_new) || !aligned16(v_new))) return PA_ERR_INVALID;
  prm.k_new = k_new;
  prm.v_new = v_new;
  const bool cluster = partition == 0 && cluster_merge(B, H, prm.NP);
  return pa::host::launch_decode_fp8(prm, q_dt, out_dt, D, S, cluster, wide_grid(B, H, prm.NP),
                                     append, k_scale, static_cast<cudaStream_t>(stream));
}

pa_status pa_decode_fp8(void* out, pa_dtype out_dt, const void* q, pa_dtype q_dt,
                        const void* k_cache, const void* v_cache, float k_scale, float v_scale,
                        const int32_t* block_tables, int MB, const int32_t* seq_lens, float scale,
                        int B, int H, int D, int S, int NB, int partition, int max_seq_len,
                        void* workspace, size_t ws_bytes, void* stream) {
  return decode_fp8_impl(out, out_dt, q, q_dt, nullptr, nullptr, k_cache, v_cache, k_scale,
                         v_scale, block_tables, MB, seq_lens, scale, B, H, H, D, S, NB,
                         partition, max_seq_len, workspace, ws_bytes, stream);
}

pa_status pa_decode_gqa_fp8(void* out, pa_dtype out_dt, const void* q, pa_dtype q_dt,
                            const void* k_cache, const void* v_cache, float k_scale,
                            float v_scale, const int32_t* block_tables, int MB,
                            const int32_t* seq_lens, float scale, int B, int H, int Hkv, int D,
                            int S, int NB, int partition, int max_seq_len, void* workspace,
                            size_t ws_bytes, void* stream) {
  return decode_fp8_impl(out, out_dt, q, q_dt, nullptr, nullptr, k_cache, v_cache, k_scale,
                         v_scale, block_tables, MB, seq_lens, scale, B, H, Hkv, D, S, NB,
                         partition, max_seq_len, workspace, ws_bytes, stream);
}

pa_status pa_decode_append_fp8(void* out, pa_dtype out_dt, const void* q, pa_dtype q_dt,
                               const void* k_new, const void* v_new, void* k_cache,
                               void* v_cache, float k_scale, float v_scale,
                               const int32_t* block_tables, int MB, const int32_t* seq_lens,
                               float scale, int B, int H, int D, int S, int NB, int partition,
                               int max_seq_len, void* workspace, size_t ws_bytes, void* stream) {
  if (B > 0 && (!k_new || !v_new)) return PA_ERR_INVALID;
  return decode_fp8_impl(out, out_dt, q, q_dt, B > 0 ? k_new : nullptr, v_new, k_cache, v_cache,
                         k_scale, v_scale, block_tables, MB, seq_lens, scale, B, H, H, D, S, NB,
                         partition, max_seq_len, workspace, ws_bytes, stream);
}

pa_status pa_get_device_error(void* stream, uint32_t* flags) {
  if (!flags) return PA_ERR_INVALID;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return PA_ERR_CUDA;
  unsigned int v = 0;
  using namespace pa::host;
  if (!take_error_append(&v) || !take_error_decode16(&v) || !take_error_grouped(&v) ||
      !take_error_fp8(&v) || !take_error_prefill(&v) || !take_error_rope(&v) ||
      !take_error_rows(&v) || !take_error_shared(&v) || !take_error_few(&v))
    return PA_ERR_CUDA;
  *flags = v;
  return PA_OK;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// pa_decode_noalloc: decode whose split-KV partials live in a static device
// array instead of a caller-provided workspace, for callers that cannot
// allocate device memory (see pagedattn.h). It reuses pa_decode unchanged.
// ---------------------------------------------------------------------------

namespace {

static __device__ __align__(256) unsigned char g_noalloc_scratch[PA_NOALLOC_SCRATCH_BYTES];

// Device address of g_noalloc_scratch per device, looked up with the device
// current and keyed by the context it was looked up in: a context that is torn
// down and created again (cudaDeviceReset, for one) loads the module again, and
// the array can move. The host-side name of the array is only a stand-in for
// the symbol, never a usable device address.
struct ScratchAddr {
  unsigned long long ctx_id = 0;  // cuCtxGetId of the context the address belongs to
  void* addr = nullptr;
};
std::mutex g_noalloc_mu;
ScratchAddr g_noalloc_addr[kMaxDevices];

using CtxGetCurrentFn = CUresult (*)(CUcontext*);
using CtxGetIdFn = CUresult (*)(CUcontext, unsigned long long*);

// The unique id of the current context (0 if the driver does not give one).
unsigned long long current_context_id() {
  static CtxGetCurrentFn get_current = nullptr;
  static CtxGetIdFn get_id = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuCtxGetCurrent", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_current = reinterpret_cast<CtxGetCurrentFn>(f);
    f = nullptr;
    if (cudaGetDriverEntryPoint("cuCtxGetId", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_id = reinterpret_cast<CtxGetIdFn>(f);
  });
  CUcontext ctx = nullptr;
  unsigned long long id = 0;
  if (!get_current || !get_id || get_current(&ctx) != CUDA_SUCCESS || !ctx ||
      get_id(ctx, &id) != CUDA_SUCCESS)
    return 0;
  return id;
}

}  // namespace

extern "C" size_t pa_noalloc_scratch_bytes(void) { return PA_NOALLOC_SCRATCH_BYTES; }

extern "C" pa_status pa_decode_noalloc(void* out, pa_dtype out_dt, const void* q,
                                       const void* k_cache, const void* v_cache,
                                       const int32_t* block_tables, int MB,
                                       const int32_t* seq_lens, float scale, int B, int H, int D,
                                       int S, int NB, pa_dtype dt, int partition, int max_seq_len,
                                       void* stream) {
  // pa_decode's own checks first, so a bad argument is PA_ERR_INVALID, never PA_ERR_OOM
  int P, NP;
  bool noop;
  const pa_status st = decode_check(out, out_dt, q, k_cache, v_cache, block_tables, MB, seq_lens,
                                    scale, B, H, H, D, S, NB, dt, partition, max_seq_len, &P, &NP,
                                    &noop);
  if (st != PA_OK || noop) return st;
  const size_t need = workspace_for(B, H, D, NP);
  if (need > PA_NOALLOC_SCRATCH_BYTES) return PA_ERR_OOM;  // larger than the static array
  void* scratch = nullptr;
  if (need > 0) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return PA_ERR_CUDA;
    const unsigned long long ctx = current_context_id();
    std::lock_guard<std::mutex> lock(g_noalloc_mu);
    ScratchAddr& a = g_noalloc_addr[dev];
    if (!a.addr || a.ctx_id != ctx || ctx == 0) {
      void* p = nullptr;
      if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || !p) return PA_ERR_CUDA;
      a.addr = p;
      a.ctx_id = ctx;
    }
    scratch = a.addr;
  }
  return pa_decode(out, out_dt, q, k_cache, v_cache, block_tables, MB, seq_lens, scale, B, H, D, S,
                   NB, dt, partition, max_seq_len, scratch, PA_NOALLOC_SCRATCH_BYTES, stream);
}

// ---------------------------------------------------------------------------
// pa_rope, pa_rope_append, pa_rope_append_fp8
// ---------------------------------------------------------------------------

namespace {

// The checks that the three share (Hkv rows of k; v and the caches apart).
bool rope_args_ok(const pa::RopeParams& prm, pa_dtype dt) {
  if (prm.T < 0 || prm.H < 0 || prm.Hkv < 0 || !cache_dtype_ok(dt)) return false;
  if (prm.D <= 0 || prm.D % 8 != 0 || prm.D > 256) return false;
  if (prm.rot < 2 || prm.rot % 2 != 0 || prm.rot > prm.D) return false;
  if (!std::isfinite(prm.amplitude) || !(std::isfinite(prm.eps) && prm.eps >= 0.f)) return false;
  const int64_t q_row = static_cast<int64_t>(prm.H) * prm.D;
  const int64_t k_row = static_cast<int64_t>(prm.Hkv) * prm.D;
  return q_row <= INT_MAX / 2 && k_row <= INT_MAX / 4;
}

bool rows_ok(const void* p, int64_t stride, int heads, int D) {
  return p && aligned16(p) && stride % 8 == 0 && stride >= static_cast<int64_t>(heads) * D;
}

bool rope_pointers_ok(const pa::RopeParams& prm) {
  if (!prm.positions || !prm.table || (reinterpret_cast<uintptr_t>(prm.table) & 7u)) return false;
  if (prm.H > 0 && (!rows_ok(prm.q, prm.q_stride, prm.H, prm.D) ||
                    !rows_ok(prm.q_out, prm.q_out_stride, prm.H, prm.D)))
    return false;
  if (prm.Hkv > 0 && !rows_ok(prm.k, prm.k_stride, prm.Hkv, prm.D)) return false;
  return (!prm.q_weight || aligned16(prm.q_weight)) && (!prm.k_weight || aligned16(prm.k_weight));
}

pa::RopeParams rope_params(void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride,
                           const void* k, int64_t k_stride, const int32_t* positions,
                           const double* table, int rot_dim, float amplitude,
                           const void* q_weight, const void* k_weight, float eps, int T, int H,
                           int Hkv, int D) {
  pa::RopeParams prm{};
  prm.q_out = q_out;
  prm.q_out_stride = q_out_stride;
  prm.q = q;
  prm.q_stride = q_stride;
  prm.k = k;
  prm.k_stride = k_stride;
  prm.positions = positions;
  prm.table = table;
  prm.rot = rot_dim;
  prm.amplitude = amplitude;
  prm.q_weight = H > 0 ? q_weight : nullptr;
  prm.k_weight = Hkv > 0 ? k_weight : nullptr;
  prm.eps = eps;
  prm.T = T;
  prm.H = H;
  prm.Hkv = Hkv;
  prm.D = D;
  prm.rows = H + Hkv;
  return prm;
}

// The append forms' part, and the launch.
pa_status rope_append(pa::RopeParams& prm, const void* v, int64_t v_stride,
                      const int64_t* slot_mapping, void* k_cache, void* v_cache, int S, int NB,
                      pa_dtype dt, int interleaved, int mode, void* stream) {
  if (!rope_args_ok(prm, dt) || prm.Hkv <= 0 || S <= 0 || NB < 0) return PA_ERR_INVALID;
  if (prm.T == 0) return PA_OK;
  if (!rope_pointers_ok(prm) || !rows_ok(v, v_stride, prm.Hkv, prm.D)) return PA_ERR_INVALID;
  if (!slot_mapping || !k_cache || !v_cache || !aligned16(k_cache) || !aligned16(v_cache))
    return PA_ERR_INVALID;
  prm.v = v;
  prm.v_stride = v_stride;
  prm.slots = slot_mapping;
  prm.k_cache = k_cache;
  prm.v_cache = v_cache;
  prm.S = S;
  prm.n_slots = static_cast<int64_t>(NB) * S;
  prm.rows = prm.H + 2 * prm.Hkv;
  return pa::host::launch_rope(prm, dt, interleaved, mode, static_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

pa_status pa_rope_table(double* table, int rot_dim, double base, pa_rope_scaling scaling,
                        double factor, double low, double high, double original_len,
                        float* amplitude) {
  constexpr double kTwoPi = 6.283185307179586476925;
  if (!table || !amplitude || rot_dim < 2 || rot_dim % 2 != 0) return PA_ERR_INVALID;
  if (!(std::isfinite(base) && base > 1.0)) return PA_ERR_INVALID;
  if (scaling < PA_ROPE_PLAIN || scaling > PA_ROPE_BANDS) return PA_ERR_INVALID;
  if (scaling != PA_ROPE_PLAIN && !(std::isfinite(factor) && factor >= 1.0)) return PA_ERR_INVALID;
  if (scaling == PA_ROPE_NTK && rot_dim == 2) return PA_ERR_INVALID;
  const bool ranged = scaling == PA_ROPE_YARN || scaling == PA_ROPE_BANDS;
  if (ranged && !(std::isfinite(high) && std::isfinite(original_len) && low > 0.0 && high > low &&
                  original_len > 0.0))
    return PA_ERR_INVALID;
  if (scaling == PA_ROPE_NTK)
    base *= std::pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2));
  // YaRN: the pair index that makes r turns over original_len positions
  auto pair_of = [&](double r) {
    return rot_dim * std::log(original_len / (r * kTwoPi)) / (2.0 * std::log(base));
  };
  double first = 0.0, last = 0.0;  // pairs up to `first` keep f_j, from `last` on f_j / factor
  if (scaling == PA_ROPE_YARN) {
    first = std::max(std::floor(pair_of(high)), 0.0);
    last = std::min(std::ceil(pair_of(low)), rot_dim - 1.0);
    if (last <= first) last = first + 1e-3;
  }
  for (int j = 0; j < rot_dim / 2; ++j) {
    double f = std::pow(base, -2.0 * j / rot_dim);
    if (scaling == PA_ROPE_LINEAR) {
      f /= factor;
    } else if (scaling == PA_ROPE_YARN) {
      const double ramp = std::min(std::max((j - first) / (last - first), 0.0), 1.0);
      f = f / factor * ramp + f * (1.0 - ramp);
    } else if (scaling == PA_ROPE_BANDS) {
      const double turns = original_len * f / kTwoPi;  // original_len / wavelength
      const double keep = std::min(std::max((turns - low) / (high - low), 0.0), 1.0);
      f = f / factor * (1.0 - keep) + f * keep;
    }
    table[j] = f / kTwoPi;
  }
  *amplitude = scaling == PA_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return PA_OK;
}

pa_status pa_rope(void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                  const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                  const int32_t* positions, const double* table, int rot_dim, int interleaved,
                  float amplitude, const void* q_weight, const void* k_weight, float eps, int T,
                  int H, int Hkv, int D, pa_dtype dt, void* stream) {
  pa::RopeParams prm = rope_params(q_out, q_out_stride, q, q_stride, k, k_stride, positions, table,
                                   rot_dim, amplitude, q_weight, k_weight, eps, T, H, Hkv, D);
  if (!rope_args_ok(prm, dt)) return PA_ERR_INVALID;
  if (T == 0 || H + Hkv == 0) return PA_OK;
  if (!rope_pointers_ok(prm) || (Hkv > 0 && !rows_ok(k_out, k_out_stride, Hkv, D)))
    return PA_ERR_INVALID;
  prm.k_out = k_out;
  prm.k_out_stride = k_out_stride;
  return pa::host::launch_rope(prm, dt, interleaved, 0, static_cast<cudaStream_t>(stream));
}

pa_status pa_rope_append(void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride,
                         const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                         const int32_t* positions, const int64_t* slot_mapping, void* k_cache,
                         void* v_cache, const double* table, int rot_dim, int interleaved,
                         float amplitude, const void* q_weight, const void* k_weight, float eps,
                         int T, int H, int Hkv, int D, int S, int NB, pa_dtype dt, void* stream) {
  pa::RopeParams prm = rope_params(q_out, q_out_stride, q, q_stride, k, k_stride, positions, table,
                                   rot_dim, amplitude, q_weight, k_weight, eps, T, H, Hkv, D);
  return rope_append(prm, v, v_stride, slot_mapping, k_cache, v_cache, S, NB, dt, interleaved, 1,
                     stream);
}

pa_status pa_rope_append_fp8(void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride,
                             const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                             const int32_t* positions, const int64_t* slot_mapping, void* k_cache,
                             void* v_cache, float k_scale, float v_scale, const double* table,
                             int rot_dim, int interleaved, float amplitude, const void* q_weight,
                             const void* k_weight, float eps, int T, int H, int Hkv, int D, int S,
                             int NB, pa_dtype dt, void* stream) {
  if (D % 16 != 0) return PA_ERR_INVALID;  // as pa_kv_append_fp8: 16-byte cache rows
  auto scale_ok = [](float s) { return s >= 0x1p-60f && s <= 0x1p60f; };
  if (!scale_ok(k_scale) || !scale_ok(v_scale)) return PA_ERR_INVALID;
  pa::RopeParams prm = rope_params(q_out, q_out_stride, q, q_stride, k, k_stride, positions, table,
                                   rot_dim, amplitude, q_weight, k_weight, eps, T, H, Hkv, D);
  prm.k_scale = k_scale;
  prm.v_scale = v_scale;
  return rope_append(prm, v, v_stride, slot_mapping, k_cache, v_cache, S, NB, dt, interleaved, 2,
                     stream);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// pa_cross and pa_decode_shared
// ---------------------------------------------------------------------------

namespace {

constexpr int kKeyTile = 128;  // keys per tile of the rows kernel

struct RowsPlan {
  bool few;         // the grouped-query kernel (launch_few), else the rows kernel
  bool split_keys;  // rows kernel: the CTA's two streams on one row tile
  int P, parts;     // keys per partition (a multiple of kKeyTile), partitions
};

// The grouped-query kernel's layout for up to 16 rows per item and KV head: as
// plan_grouped, 512-key partitions, halved (down to 128) while the grid stays
// within two CTAs per SM, doubled (up to 2048) for 32K keys and more while it
// keeps 8 CTAs per SM. At head size 64 an SM holds some seven of its CTAs: up to
// 8 partitions may fill that (8 single tokens on 20 heads over 1,536 keys: 17.6 us
// at 256 keys, 20.6 at 512; but 4 x 8 KV heads over 5,120 keys 27.1 us at 256, 20
// partitions, against 22.9 at 512).
RowsPlan plan_few(int items, int Hkv, int D, int max_len, int partition) {
  const int64_t sms = sm_count();
  const int64_t ctas = static_cast<int64_t>(std::max(items, 1)) * Hkv;
  int64_t P = kDefaultPartition;
  if (partition > 0) {
    P = partition;
  } else if (partition < 0) {
    P = std::max<int64_t>(1, ceil_div(max_len, kKeyTile)) * kKeyTile;
  } else {
    auto fits = [&](int64_t parts) {
      return ctas * parts <= 2 * sms || (D == 64 && parts <= 8 && ctas * parts <= 7 * sms);
    };
    while (P > kKeyTile && fits(ceil_div(max_len, P / 2))) P /= 2;
    if (max_len >= 32768)
      while (P < 2048 && ctas * ceil_div(max_len, 2 * P) >= 8 * sms) P *= 2;
  }
  RowsPlan pl{};
  pl.few = true;
  pl.parts = static_cast<int>(std::max<int64_t>(1, ceil_div(max_len, P)));
  pl.P = static_cast<int>(P);
  return pl;
}

// How the attention over whole key ranges is laid out. Up to 16 rows per item
// and KV head go to the grouped-query kernel (plan_few), whose small CTAs share
// an SM: 8 single tokens on 20 heads over up to 1,500 keys took 30.9 us on the
// rows kernel. The rest goes to the rows kernel: `items` with up to max_rows query
// tokens each, G heads per KV head, keys up to max_len.
//
// The choice minimises an estimate of the time, in units of 1.2 us: waves of CTAs
// x (key tiles per CTA x a tile's time + 4 for a CTA's start and end), plus,
// where the keys are split, the merge. `behind` is the time of the work that may
// run beside it (the tails of pa_decode_shared; 0 for pa_cross): it proceeds on the
// SMs that one wave leaves free, at up to 1.3 times their share (what bounds it is
// HBM), and what then remains of it follows. Leaving SMs free pays: 64 requests
// behind 2,048 tokens on 40 heads 69.3 us with 120 CTAs for the shared part, 65.0
// with 40; 24 behind 4,000 on 32/8 heads 32.3 us with 128 CTAs, 22.4 with 64.
RowsPlan plan_rows(int items, int max_rows, int G, int Hkv, int D, int max_len, int partition,
                   double behind) {
  if (static_cast<int64_t>(max_rows) * G <= 16)
    return plan_few(items, Hkv, D, max_len, partition);
  const int64_t tiles = std::max<int64_t>(1, ceil_div(max_len, kKeyTile));
  const int qpt = kKeyTile / G;
  const int64_t sms = sm_count();
  RowsPlan best{};
  double best_cost = 0.0;
  bool any = false;
  // head size 64 has two CTAs of one row tile per SM, 256 one
  const int64_t slots = D == 64 ? 2 * sms : sms;
  for (int split = D == 128 ? 1 : 0; split >= 0; --split) {
    const int row_tiles = (split || D != 128) ? 1 : 2;
    if (row_tiles == 2 && max_rows <= qpt) continue;  // nothing for the second half
    const double tile_cost = split ? 1.0 : (D == 256 ? 3.0 : (D == 64 ? 1.6 : 2.0));
    const int64_t ctas = static_cast<int64_t>(std::max(items, 1)) * Hkv *
                         std::max<int64_t>(1, ceil_div(max_rows, row_tiles * qpt));
    const int64_t most =
        partition == 0 ? std::min(tiles, std::max<int64_t>(8, 2 * slots / ctas + 1)) : 1;
    for (int64_t c = 1; c <= most; ++c) {
      int64_t per = ceil_div(tiles, c);
      if (partition > 0) per = partition / kKeyTile;
      const int64_t parts = ceil_div(tiles, per);
      const int64_t waves = ceil_div(ctas * parts, slots);
      double cost = static_cast<double>(waves) * (per * tile_cost + 4.0);
      if (behind > 0.0) {
        const double free = std::max(0.0, 1.0 - static_cast<double>(ctas * parts) / slots);
        cost += std::max(0.0, behind - std::min(1.0, 1.3 * free) * cost);
      }
      if (parts > 1)  // the merge: its launch (or a part more), its reads and writes
        cost += (behind > 0.0 ? 0.1 * parts : 1.5) +
                static_cast<double>(items) * max_rows * Hkv * G * parts * D * 8.0 / 9.0e6;
      if (!any || cost < best_cost) {
        any = true;
        best_cost = cost;
        best.split_keys = split != 0 || D == 64;
        best.parts = static_cast<int>(parts);
        best.P = static_cast<int>(per * kKeyTile);
      }
    }
  }
  return best;
}

// The time of the tails' pass in the same units: their bytes (half of the bound on
// average) at HBM's rate, at least one CTA's time (2.9) for each wave of CTAs.
double tail_time(int B, int H, int Hkv, int D, int S, int max_tail_len, int parts) {
  if (parts <= 0 || B <= 0) return 0.0;
  const int G = H / Hkv;
  const double bytes = static_cast<double>(B) * (0.5 * max_tail_len + 0.5 * S) * Hkv * D * 4.0;
  const int64_t per_sm = G == 1 ? (D == 64 ? 6 : 3) : (D == 64 ? 7 : (D == 128 ? 4 : 2));
  const int64_t ctas = static_cast<int64_t>(B) * parts * (G == 1 ? H : Hkv * ((G + 15) / 16));
  return std::max(bytes / 7.8e6, 2.9 * ceil_div(ctas, per_sm * sm_count()));
}

// (P is then at most INT_MAX)
bool rows_len_ok(int max_len) { return max_len >= 0 && max_len <= INT_MAX - (kKeyTile - 1); }

bool rows_shape_ok(int H, int Hkv, int D) {
  return H > 0 && Hkv > 0 && H % Hkv == 0 && H / Hkv <= 128 && H <= 65535 &&
         (D == 64 || D == 128 || D == 256);
}

// Launches the attention over whole key ranges that `pl` chose.
pa_status launch_key_ranges(const RowsPlan& pl, const pa::RowsParams& r, const void* q,
                            float scale, pa_dtype dt, int D, cudaStream_t st) {
  if (!pl.few) return pa::host::launch_rows(r, q, dt, D, pl.split_keys, st);
  pa::DecodeParamsFew f{};
  f.out = r.out;
  f.q = q;
  f.k_cache = r.k_cache;
  f.v_cache = r.v_cache;
  f.block_tables = r.block_tables;
  f.seq_lens = r.lens;
  f.shared_lens = r.shared_lens;
  f.start = r.start;
  f.ws_m = r.ws_m;
  f.ws_l = r.ws_l;
  f.ws_acc = r.ws_acc;
  f.q_scale = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  f.v_scale = 1.f;
  f.MB = r.MB;
  f.B = r.items;
  f.H = r.H;
  f.Hkv = r.Hkv;
  f.NB = r.NB;
  f.P = r.P;
  f.NP = r.NP;
  f.L_cap = r.L_cap;
  f.T = r.T;
  f.max_rows = r.max_rows;
  f.items = r.items;
  f.parts = r.parts;
  return pa::host::launch_few(f, dt, r.out_dt, D, r.S, st);
}

struct SharedPlan {
  RowsPlan rows;
  int shared_parts, tail_P, tail_parts;
};

SharedPlan plan_shared(int B, int NG, int H, int Hkv, int D, int S, int max_group,
                       int max_shared_len, int max_tail_len) {
  SharedPlan s{};
  int P = 0, NP = 1;
  plan_grouped(B, H, Hkv, S, max_tail_len, 0, &P, &NP);
  s.tail_parts = max_tail_len > 0 ? NP : 0;
  s.rows = plan_rows(NG, max_group, H / Hkv, Hkv, D, max_shared_len, 0,
                     tail_time(B, H, Hkv, D, S, max_tail_len, s.tail_parts));
  s.shared_parts = max_shared_len > 0 ? s.rows.parts : 0;
  s.tail_P = P > 0 ? P : static_cast<int>(ceil_div(std::max(max_tail_len, 1), S) * S);
  return s;
}

bool shared_bounds_ok(int B, int NG, int H, int Hkv, int D, int S, int max_group,
                      int max_shared_len, int max_tail_len) {
  // (the tails' grid has a plane more than requests)
  return B >= 0 && NG >= 0 && B <= 65534 && NG <= 65534 && rows_shape_ok(H, Hkv, D) &&
         decode_shape_ok(D, S) && max_group >= 0 && rows_len_ok(max_shared_len) &&
         max_tail_len >= 0 && max_tail_len <= INT_MAX - 4096;
}

}  // namespace

extern "C" {

size_t pa_cross_workspace_bytes(int B, int T, int H, int Hkv, int D, int max_q_len, int max_kv_len,
                                int partition) {
  if (B <= 0 || T <= 0 || max_q_len <= 0 || !rows_len_ok(max_kv_len) || !rows_shape_ok(H, Hkv, D))
    return 0;
  if (partition < -1 || (partition > 0 && partition % kKeyTile != 0)) return 0;
  const RowsPlan pl = plan_rows(B, std::min(max_q_len, T), H / Hkv, Hkv, D, max_kv_len, partition,
                                0.0);
  return workspace_for(T, H, D, pl.parts);
}

pa_status pa_cross(void* out, pa_dtype out_dt, const void* q, const void* k_cache,
                   const void* v_cache, const int32_t* block_tables, int MB,
                   const int32_t* kv_lens, const int32_t* q_start, float scale, int B, int H,
                   int Hkv, int D, int S, int NB, pa_dtype dt, int T, int max_q_len,
                   int max_kv_len, int partition, void* workspace, size_t ws_bytes, void* stream) {
  if (B < 0 || T < 0 || max_q_len < 0 || MB < 0 || NB < 0 || !rows_shape_ok(H, Hkv, D))
    return PA_ERR_INVALID;
  if (!cache_dtype_ok(dt) || !out_dtype_ok(out_dt)) return PA_ERR_INVALID;
  if (!(S == 8 || S == 16 || S == 32 || S == 64 || S == 128)) return PA_ERR_INVALID;
  if (!std::isfinite(scale) || !(scale > 0.f)) return PA_ERR_INVALID;
  if (partition < -1 || (partition > 0 && partition % kKeyTile != 0)) return PA_ERR_INVALID;
  const int64_t L_max = static_cast<int64_t>(MB) * S;
  if (L_max > INT_MAX || !rows_len_ok(max_kv_len) || max_kv_len > L_max) return PA_ERR_INVALID;
  if (B == 0 || T == 0 || max_q_len == 0) return PA_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !kv_lens || !q_start || MB == 0)
    return PA_ERR_INVALID;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
    return PA_ERR_INVALID;
  if (B > 65535 || NB == 0 || static_cast<int64_t>(NB) * Hkv * S > INT_MAX) return PA_ERR_INVALID;
  const int G = H / Hkv;
  const int max_rows = std::min(max_q_len, T);
  const RowsPlan pl = plan_rows(B, max_rows, G, Hkv, D, max_kv_len, partition, 0.0);
  // grid: x row tiles and KV heads (merge: row and head pairs), y partitions
  if (static_cast<int64_t>(max_rows) * H > INT_MAX || pl.parts > 65535) return PA_ERR_INVALID;
  const size_t need = workspace_for(T, H, D, pl.parts);
  if (need > 0 && (!workspace || ws_bytes < need || !aligned16(workspace))) return PA_ERR_INVALID;
  pa::RowsParams prm{};
  prm.out = out;
  prm.out_dt = out_dt;
  prm.k_cache = k_cache;
  prm.v_cache = v_cache;
  prm.block_tables = block_tables;
  prm.lens = kv_lens;
  prm.start = q_start;
  prm.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  prm.MB = MB;
  prm.items = B;
  prm.H = H;
  prm.Hkv = Hkv;
  prm.NB = NB;
  prm.T = T;
  prm.S = S;
  prm.max_rows = max_rows;
  prm.L_cap = max_kv_len;
  prm.P = pl.P;
  prm.parts = prm.NP = pl.parts;
  prm.qpt = kKeyTile / G;
  if (need > 0) {
    const size_t n = static_cast<size_t>(T) * H * pl.parts;
    uint8_t* base = static_cast<uint8_t*>(workspace);
    prm.ws_m = reinterpret_cast<float*>(base);
    prm.ws_l = prm.ws_m + n;
    prm.ws_acc = reinterpret_cast<float*>(base + acc_offset(n));
  }
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const pa_status rc = launch_key_ranges(pl, prm, q, scale, dt, D, st);
  return rc != PA_OK ? rc : pa::host::launch_cross_merge(prm, D, st);
}

size_t pa_decode_shared_workspace_bytes(int B, int NG, int H, int Hkv, int D, int S, int max_group,
                                        int max_shared_len, int max_tail_len) {
  if (!shared_bounds_ok(B, NG, H, Hkv, D, S, max_group, max_shared_len, max_tail_len) || B == 0)
    return 0;
  const SharedPlan pl = plan_shared(B, NG, H, Hkv, D, S, std::min(max_group, B), max_shared_len,
                                    max_tail_len);
  const size_t n = static_cast<size_t>(B) * H * (pl.shared_parts + pl.tail_parts);
  return n == 0 ? 0 : acc_offset(n) + n * D * sizeof(float);
}

pa_status pa_decode_shared(void* out, pa_dtype out_dt, const void* q, const void* k_cache,
                           const void* v_cache, const int32_t* block_tables, int MB,
                           const int32_t* seq_lens, const int32_t* shared_lens,
                           const int32_t* group_start, int NG, float scale, int B, int H, int Hkv,
                           int D, int S, int NB, pa_dtype dt, int max_group, int max_shared_len,
                           int max_tail_len, void* workspace, size_t ws_bytes, void* stream) {
  if (!shared_bounds_ok(B, NG, H, Hkv, D, S, max_group, max_shared_len, max_tail_len))
    return PA_ERR_INVALID;
  if (!cache_dtype_ok(dt) || !out_dtype_ok(out_dt) || MB < 0 || NB < 0) return PA_ERR_INVALID;
  if (!std::isfinite(scale) || !(scale > 0.f)) return PA_ERR_INVALID;
  const int64_t L_max = static_cast<int64_t>(MB) * S;
  if (L_max > INT_MAX || max_shared_len > L_max || max_tail_len > L_max) return PA_ERR_INVALID;
  if (B == 0) return PA_OK;
  // every request belongs to a group
  if (NG == 0 || max_group == 0) return PA_ERR_INVALID;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens || !shared_lens ||
      !group_start || MB == 0)
    return PA_ERR_INVALID;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
    return PA_ERR_INVALID;
  if (NB == 0 || static_cast<int64_t>(NB) * Hkv * S > INT_MAX) return PA_ERR_INVALID;
  const int G = H / Hkv;
  max_group = std::min(max_group, B);
  const SharedPlan pl = plan_shared(B, NG, H, Hkv, D, S, max_group, max_shared_len, max_tail_len);
  const int NP = pl.shared_parts + pl.tail_parts;
  const size_t n = static_cast<size_t>(B) * H * NP;
  const size_t need = n == 0 ? 0 : acc_offset(n) + n * D * sizeof(float);
  if (need > 0 && (!workspace || ws_bytes < need || !aligned16(workspace))) return PA_ERR_INVALID;
  uint8_t* base = static_cast<uint8_t*>(workspace);
  float* ws_m = reinterpret_cast<float*>(base);
  float* ws_l = need > 0 ? ws_m + n : nullptr;
  float* ws_acc = need > 0 ? reinterpret_cast<float*>(base + acc_offset(n)) : nullptr;
  const double scale_log2 = static_cast<double>(scale) * 1.4426950408889634;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);

  if (pl.shared_parts > 0) {
    pa::RowsParams prm{};
    prm.k_cache = k_cache;
    prm.v_cache = v_cache;
    prm.block_tables = block_tables;
    prm.lens = seq_lens;
    prm.shared_lens = shared_lens;
    prm.start = group_start;
    prm.ws_m = ws_m;
    prm.ws_l = ws_l;
    prm.ws_acc = ws_acc;
    prm.scale_log2 = static_cast<float>(scale_log2);
    prm.MB = MB;
    prm.items = NG;
    prm.H = H;
    prm.Hkv = Hkv;
    prm.NB = NB;
    prm.T = B;
    prm.S = S;
    prm.max_rows = max_group;
    prm.L_cap = max_shared_len;
    prm.P = pl.rows.P;
    prm.parts = pl.rows.parts;
    prm.NP = NP;
    prm.qpt = kKeyTile / G;
    const pa_status rc = launch_key_ranges(pl.rows, prm, q, scale, dt, D, st);
    if (rc != PA_OK) return rc;
  }
  pa::DecodeParamsTail t{};
  t.out = out;
  t.q = q;
  t.k_cache = k_cache;
  t.v_cache = v_cache;
  t.block_tables = block_tables;
  t.seq_lens = seq_lens;
  t.shared_lens = shared_lens;
  t.group_start = group_start;
  t.NG = NG;
  t.ws_m = ws_m;
  t.ws_l = ws_l;
  t.ws_acc = ws_acc;
  t.q_scale = static_cast<float>(scale_log2);
  t.v_scale = 1.f;
  t.MB = MB;
  t.B = B;
  t.H = H;
  t.Hkv = Hkv;
  t.NB = NB;
  t.P = pl.tail_P;
  t.NP = NP;
  t.L_cap = max_tail_len;
  t.part0 = pl.shared_parts;
  t.shared_cap = max_shared_len;
  t.tail_parts = pl.tail_parts;
  if (pl.tail_parts > 0) {
    const pa_status rc = pa::host::launch_tails(t, dt, D, S, st);
    if (rc != PA_OK) return rc;
  }
  return pa::host::launch_shared_merge(t, pl.rows.P, dt, out_dt, D, S, st);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// The same calls on argument blocks.
// ---------------------------------------------------------------------------

extern "C" {

pa_status pa_rope_call(const pa_rope_args* a) {
  if (!a) return PA_ERR_INVALID;
  return pa_rope(a->q_out, a->q_out_stride, a->k_out, a->k_out_stride, a->q, a->q_stride, a->k,
                 a->k_stride, a->positions, a->table, a->rot_dim, a->interleaved, a->amplitude,
                 a->q_weight, a->k_weight, a->eps, a->T, a->H, a->Hkv, a->D,
                 static_cast<pa_dtype>(a->dt), a->stream);
}

pa_status pa_rope_append_call(const pa_rope_args* a) {
  if (!a) return PA_ERR_INVALID;
  return pa_rope_append(a->q_out, a->q_out_stride, a->q, a->q_stride, a->k, a->k_stride, a->v,
                        a->v_stride, a->positions, a->slot_mapping, a->k_cache, a->v_cache,
                        a->table, a->rot_dim, a->interleaved, a->amplitude, a->q_weight,
                        a->k_weight, a->eps, a->T, a->H, a->Hkv, a->D, a->S, a->NB,
                        static_cast<pa_dtype>(a->dt), a->stream);
}

pa_status pa_rope_append_fp8_call(const pa_rope_args* a) {
  if (!a) return PA_ERR_INVALID;
  return pa_rope_append_fp8(a->q_out, a->q_out_stride, a->q, a->q_stride, a->k, a->k_stride, a->v,
                            a->v_stride, a->positions, a->slot_mapping, a->k_cache, a->v_cache,
                            a->k_scale, a->v_scale, a->table, a->rot_dim, a->interleaved,
                            a->amplitude, a->q_weight, a->k_weight, a->eps, a->T, a->H, a->Hkv,
                            a->D, a->S, a->NB, static_cast<pa_dtype>(a->dt), a->stream);
}

pa_status pa_cross_call(const pa_ranges_args* a) {
  if (!a) return PA_ERR_INVALID;
  return pa_cross(a->out, static_cast<pa_dtype>(a->out_dt), a->q, a->k_cache, a->v_cache,
                  a->block_tables, a->MB, a->lens, a->start, a->scale, a->B, a->H, a->Hkv, a->D,
                  a->S, a->NB, static_cast<pa_dtype>(a->dt), a->T, a->max_q_len, a->max_kv_len,
                  a->partition, a->workspace, a->ws_bytes, a->stream);
}

pa_status pa_decode_shared_call(const pa_ranges_args* a) {
  if (!a) return PA_ERR_INVALID;
  return pa_decode_shared(a->out, static_cast<pa_dtype>(a->out_dt), a->q, a->k_cache, a->v_cache,
                          a->block_tables, a->MB, a->lens, a->shared_lens, a->start, a->NG,
                          a->scale, a->B, a->H, a->Hkv, a->D, a->S, a->NB,
                          static_cast<pa_dtype>(a->dt), a->max_group, a->max_shared_len,
                          a->max_tail_len, a->workspace, a->ws_bytes, a->stream);
}

}  // extern "C"
