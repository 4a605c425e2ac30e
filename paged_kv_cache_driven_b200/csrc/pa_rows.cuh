// Attention of packed query rows over whole paged key ranges, on the
// fifth-generation tensor cores: pa_cross, and the shared part of
// pa_decode_shared.
//
// What it computes: item i (a request's queries, or the queries of a group of
// requests) has the query tokens start[i] .. start[i+1] - 1, and every one of
// them sees the same keys, tokens 0 .. L - 1 of one block table:
//   out[r, h] = softmax_t(scale * q[r, h] . K_t) V_t,   no causal mask.
// The G = H / Hkv query heads of a KV head read the same keys too, so the rows
// of one contraction are (token, head of the group) pairs: a 128-row tile is
// qpt = 128 / G tokens x G heads, loaded by one TMA box per 64-element column
// block (box 64 x G heads x qpt tokens), row r = token r / G, head r % G. K and V
// are thus read once for all of a tile's tokens and heads.
//
// One CTA per (row tiles, KV head, partition of the keys, item), up to 640 threads
// in the roles of the causal prefill kernel: two softmax warpgroups per stream (one
// at head size 64), producer warps (one lane per cache block and TMA box), an MMA
// issuer warp that also owns tensor memory. Two streams ping-pong, so that the
// tensor cores work for one while the other's softmax runs:
//   KSPLIT = false  stream t takes row tile t: both read every key tile;
//   KSPLIT = true   one row tile (few rows): stream t takes the key tiles
//                   t, t + 2, ..., and the CTA joins the two results at its end
//                   through the K ring's memory. A key tile then costs half the
//                   time, which brings few rows over long keys close to the
//                   rate at which HBM delivers the keys.
// Few CTAs are multiplied by partitions of the keys, whose results (m, l, O) a
// merge kernel joins. Scores, softmax statistics and output accumulate in fp32;
// the weights enter the second product as two 16-bit terms, value and rounding
// residue: 2^-16 of a weight for bf16, 2^-22 for f16 (see kWeightShift for small
// weights). One f16 term would leave 2^-11 of a weight, as much as an fp16 output's
// own rounding.
//
// Every wait is bounded (about a second); a timeout sets PA_DEVERR_TIMEOUT, stops
// all roles, waits for the copies and MMAs in flight and frees tensor memory.
#pragma once

#include <cuda.h>

#include "pa_decode.cuh"
#include "pa_prefill.cuh"

namespace pa {

template <int D, bool KSPLIT>
struct RowsTiling {
  static constexpr int BM = 128;              // query rows per tile (MMA M)
  static constexpr int BN = D == 64 ? 64 : 128;  // keys per tile
  // Streams: two, or one at head size 256, which fills tensor and shared memory.
  // At head size 64 two CTAs share an SM (256 tensor-memory columns and 81 KB
  // each) and cover each other's start and end, and a stream is one warpgroup with
  // tiles of 64 keys, whose threads hold whole rows: four chains of product,
  // softmax, product are then under way on an SM, and none waits for another's
  // row maximum. 128 rows x 128 keys take 0.95 us of an SM in bf16, where two chains
  // of two warpgroups each took 1.16 (16 ragged prompts on 32 heads, in a captured
  // graph, 117.4 -> 98.7 us; a CTA's end, which joins the streams, 1.5 us more).
  static constexpr int NST = D == 256 ? 1 : 2;
  static constexpr int HALVES = D == 64 ? 1 : 2;  // warpgroups that share a stream's keys
  static constexpr int SWARPS = 4 * HALVES;       // softmax warps per stream
  static constexpr int CTAS = D == 64 ? 2 : 1;  // per SM
  static constexpr int NQ = KSPLIT ? 1 : NST;  // query tiles held
  static constexpr int KST = D == 256 ? 1 : (D == 64 ? 4 : 2);  // K stages
  static constexpr int VST = KST;                                // V stages
  // Producer warps: a warp gets a TMA box out about every 90 cycles (one lane
  // each; 180 from a single lane), so one warp with all 32 boxes of a K and a V
  // tile in blocks of 16 held the pipeline at 3,300 cycles per key tile. K has
  // NKP warps that share a tile's column blocks; V has one, whose boxes span all
  // column blocks (V's tile may lie block by block: see dV; K's has to be whole
  // columns of 128 rows).
  // (At head size 64, one warp for both operands' boxes held a pair of 64-key steps
  // at 1.65 us in blocks of 16, 2.2 in blocks of 8; two warps 1.3.)
  static constexpr int NKP = D == 64 ? 1 : 2, NPROD = NKP + 1;
  static constexpr int COLB = D / 64;
  static constexpr int CB_BYTES = 128 * 128;  // one column block of 128 rows (D = 64 has one)
  static constexpr int Q_BYTES = BM * D * 2;
  static constexpr int KV_BYTES = BN * D * 2;
  static constexpr int OFF_K = NQ * Q_BYTES;
  static constexpr int OFF_V = OFF_K + KST * KV_BYTES;
  static constexpr int OFF_XCH = OFF_V + VST * KV_BYTES;
  // [stream][phase parity][half][row]
  static constexpr int XCH_BYTES = HALVES == 2 ? NST * 2 * 2 * BM * 4 : 0;
  static constexpr int OFF_BAR = OFF_XCH + XCH_BYTES;
  static constexpr int SMEM = 1024 + OFF_BAR + 256;
  static constexpr int STHREADS = NST * SWARPS * 32;  // softmax threads
  // Two CTAs of 11 warps would leave 88 registers per thread, and the softmax warps
  // spilled some of their rows: at head size 64 the CTA is launched with an idle
  // twelfth warp, and its third warpgroup passes registers to the first two.
  static constexpr bool PASS_REGS = D == 64;
  static constexpr int THREADS = STHREADS + NPROD * 32 + (PASS_REGS ? 64 : 32);
  static constexpr int LAUNCH_REGS = 80, SOFTMAX_REGS = 96, OTHER_REGS = 48;  // (PASS_REGS)
  static_assert(!PASS_REGS || (STHREADS * SOFTMAX_REGS + (THREADS - STHREADS) * OTHER_REGS <=
                                   THREADS * LAUNCH_REGS &&
                               THREADS - STHREADS == 128 &&
                               CTAS * THREADS * LAUNCH_REGS <= 65536),
                "registers");
  static constexpr uint32_t TMEM_COLS = 512 / CTAS;
  // a stream's tensor memory: scores, then weights, in the first BN columns, output
  // in the next D
  static constexpr uint32_t TST = TMEM_COLS / NST;
  // an SM holds CTAS of these, no more: their tensor memory is what there is
  static_assert((CTAS + 1) * SMEM > 232448, "CTAs per SM");
  static_assert(CTAS * SMEM <= 232448 && BN + D <= TST, "CTAs per SM");
  static_assert(!KSPLIT || NST == 2, "two streams share the keys");
  static_assert(!KSPLIT || (D * 128 * 4 <= KST * KV_BYTES && SWARPS * 4096 <= Q_BYTES &&
                            SWARPS * 4096 <= VST * KV_BYTES / 2 &&
                            4 * 128 * 4 <= VST * KV_BYTES / 2),
                "the join's exchange fits the rings");
  static_assert(SMEM <= 232448, "shared memory per CTA");
};

// ---- MMA issue by a whole warp ----------------------------------------------------
// The issuing warp runs these with all its lanes, one elected lane's instruction
// taking effect (`on`), and with descriptors that are a uniform base plus a
// constant: the operands then stay in uniform registers. Issued from inside an
// `if (lane == 0)`, with each descriptor put together from its fields, an MMA took
// the issuing lane some 87 cycles, more than the tensor core needs for it.

// One lane of the (converged) warp.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t on;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(on));
  return on;
}

__device__ __forceinline__ void mma_ss_on(uint32_t on, uint32_t d_tmem, uint64_t a_desc,
                                          uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}

__device__ __forceinline__ void mma_ts_on(uint32_t on, uint32_t d_tmem, uint32_t a_tmem,
                                          uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}

__device__ __forceinline__ void commit_on(uint32_t on, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar)),
      "r"(on)
      : "memory");
}

__device__ __forceinline__ void prefetch_map(const void* tmap) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tmap)) : "memory");
}

// One arrival for a whole warp (its lanes' earlier writes are ordered before it).
__device__ __forceinline__ void arrive_warp(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// Stores 4 W bytes of each of a warp's 32 rows (lane r holds row r's W words; the
// rows' destinations differ, rows from `rows` on are not stored) through 32 x W
// words of shared memory, so that every store instruction writes whole
// segments of 4 W bytes: stored from the row's own lane, each instruction would
// touch 32 lines. 16-byte pieces are placed so that neither side conflicts.
template <int W>
__device__ __forceinline__ void store_rows(uint8_t* buf, const uint32_t (&w)[W], uint8_t* dst,
                                           int rows, int lane) {
  static_assert(W == 32 || W == 16, "32 columns in 32 or 16 bits");
  constexpr int NP = W / 4;  // 16-byte pieces per row
  auto place = [](int row, int piece) {
    const int x = W == 32 ? row & 7 : (row >> 1) & 3;
    return row * W * 4 + ((piece ^ x) << 4);
  };
  __syncwarp();  // the warp's previous use of buf is over
#pragma unroll
  for (int k = 0; k < NP; ++k)
    *reinterpret_cast<uint4*>(buf + place(lane, k)) =
        make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
  __syncwarp();
  const int piece = lane % NP;
#pragma unroll
  for (int base = 0; base < 32; base += 32 / NP) {
    const int row = base + lane / NP;
    const uint64_t at = __shfl_sync(kFullMask, reinterpret_cast<uint64_t>(dst), row);
    const uint4 x = *reinterpret_cast<const uint4*>(buf + place(row, piece));
    if (row < rows) reinterpret_cast<uint4*>(at)[piece] = x;
  }
}

// 32 consecutive output elements of each of a warp's rows, in the output's type.
__device__ __forceinline__ void store_out(uint8_t* buf, const float (&v)[32], void* out,
                                          pa_dtype dt, int64_t at, int rows, int lane) {
  constexpr int C = 32;
  if (dt == PA_F32) {
    uint32_t w[C];
#pragma unroll
    for (int c = 0; c < C; ++c) w[c] = __float_as_uint(v[c]);
    store_rows<C>(buf, w, reinterpret_cast<uint8_t*>(static_cast<float*>(out) + at), rows, lane);
  } else {
    uint32_t w[C / 2];
#pragma unroll
    for (int c = 0; c < C / 2; ++c)
      w[c] = dt == PA_BF16 ? pack_pair<__nv_bfloat16>(v[2 * c], v[2 * c + 1])
                           : pack_pair<__half>(v[2 * c], v[2 * c + 1]);
    store_rows<C / 2>(buf, w, reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(out) + at), rows,
                      lane);
  }
}

// f16 weights are held as 2^7 times what they are (the sum l alike): f16 ends at
// 2^-24, and a weight is at most 2^8 (the reference maximum may lag by that much),
// so the steps of the smallest weights lie at 2^-31 of the largest instead of 2^-24.
constexpr float kWeightShift = 7.f;

template <typename T, int D, bool KSPLIT>
__global__ void __launch_bounds__(RowsTiling<D, KSPLIT>::THREADS, RowsTiling<D, KSPLIT>::CTAS)
    rows_kernel(const RowsParams p, const __grid_constant__ CUtensorMap tmq,
                const __grid_constant__ CUtensorMap tmk,
                const __grid_constant__ CUtensorMap tmv) {
  constexpr bool F16 = std::is_same<T, __half>::value;
  using Tl = RowsTiling<D, KSPLIT>;
  constexpr int NST = Tl::NST, BN = Tl::BN, HALVES = Tl::HALVES;
  constexpr uint32_t TST = Tl::TST;

  grid_dependents_launch();  // what follows on the stream may be scheduled early
  const int G = p.H / p.Hkv;
  const int qpt = p.qpt;
  const int tok_cta = Tl::NQ * qpt;  // query tokens per CTA
  const int ngroups = (p.max_rows + tok_cta - 1) / tok_cta;
  const int hk = blockIdx.x / ngroups;
  const int tok0 = (blockIdx.x - hk * ngroups) * tok_cta;
  const int part = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.S;

  if (threadIdx.x == 0) {  // the tensor maps' first use then finds them cached
    prefetch_map(&tmq);
    prefetch_map(&tmk);
    prefetch_map(&tmv);
  }
  // The item, its queries and (pa_cross) its number of keys. Where there is more than
  // a wave of CTAs, those of long items start first, so that the last to end are
  // short ones: the item is then the blockIdx.z-th in descending order of length,
  // found by each warp from the lengths, one per lane, so of at most 32 (in a captured
  // graph: 16 ragged prompts 98.7 -> 92.9 us on 32 heads of 64, 8 prompts 80.5 -> 62
  // on 16/4 heads of 256).
  int i = blockIdx.z, q0, q1, L = 0;
  if (p.longest_first) {
    const int k = min(lane, p.items - 1);
    const int from = p.start[k], to = p.start[k + 1], len = p.lens[k];
    if (!__all_sync(kFullMask, len == __shfl_sync(kFullMask, len, 0))) {
      int rank = 0;
      for (int o = 0; o < p.items; ++o) {
        const int other = __shfl_sync(kFullMask, len, o);
        rank += other > len || (other == len && o < lane);
      }
      i = __ffs(__ballot_sync(kFullMask, rank == i && lane < p.items)) - 1;
    }
    q0 = __shfl_sync(kFullMask, from, i);
    q1 = __shfl_sync(kFullMask, to, i);
    L = __shfl_sync(kFullMask, len, i);
  } else {
    q0 = p.start[i];
    q1 = p.start[i + 1];
    if (!p.shared_lens) L = p.lens[i];
  }
  const int n = q1 - q0;
  const bool first_cta = blockIdx.x == 0 && part == 0;
  if (n < 0 || q0 < 0 || q1 > p.T || n > p.max_rows) {
    if (threadIdx.x == 0 && first_cta) raise_error(PA_DEVERR_SEQ_LEN);
    return;
  }
  if (tok0 >= n) return;
  const int ntok = min(n - tok0, tok_cta);
  // the keys, and the row of the block table that names them
  int trow = i;
  if (p.shared_lens) {
    // the longest shared part of the CTA's requests, through that request's table
    int best = 0, who = q0 + tok0;
    for (int r = lane; r < ntok; r += 32) {
      const int b = q0 + tok0 + r;
      const int sh = p.shared_lens[b], len = p.lens[b];
      if (warp == 0 && hk == 0 && part == 0 && (sh < 0 || sh > p.L_cap || len < 0))
        raise_error(PA_DEVERR_SEQ_LEN);
      const int e = shared_part(sh, len, p.L_cap, S);
      if (e > best) best = e, who = b;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      const int e = __shfl_xor_sync(kFullMask, best, o), b = __shfl_xor_sync(kFullMask, who, o);
      if (e > best || (e == best && b < who)) best = e, who = b;
    }
    L = best;
    trow = who;
  } else {
    if (L < 0 || L > p.L_cap) {
      if (threadIdx.x == 0 && first_cta) raise_error(PA_DEVERR_SEQ_LEN);
      L = L < 0 ? 0 : p.L_cap;
    }
  }
  const int64_t t_beg64 = static_cast<int64_t>(part) * p.P;
  const bool direct = !p.shared_lens && L <= p.P;  // the only partition: final output
  if (t_beg64 >= L) {
    if (direct && part == 0)  // no keys at all: zero rows
      for (int64_t e = threadIdx.x; e < static_cast<int64_t>(ntok) * G * D; e += blockDim.x) {
        const int64_t row = e / (G * D);
        const int64_t at = (static_cast<int64_t>(q0 + tok0 + row) * p.H + hk * G) * D +
                           (e - row * (G * D));
        if (p.out_dt == PA_F32)
          static_cast<float*>(p.out)[at] = 0.f;
        else
          static_cast<uint16_t*>(p.out)[at] = 0;
      }
    return;
  }
  const int t_beg = static_cast<int>(t_beg64);
  const int t_end = static_cast<int>(min(t_beg64 + p.P, static_cast<int64_t>(L)));
  const int NK = (t_end - t_beg + BN - 1) / BN;  // key tiles of the CTA
  // key tiles each stream takes, and its query tokens' rows
  auto rows_of = [&](int t) {
    return (KSPLIT ? ntok : max(0, min(qpt, ntok - t * qpt))) * G;
  };
  auto tiles_of = [&](int t) { return KSPLIT ? (NK + 1 - t) >> 1 : (rows_of(t) > 0 ? NK : 0); };
  const int nq = KSPLIT ? 1 : (rows_of(NST - 1) > 0 ? NST : 1);  // query tiles holding rows

  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = sm;
  uint8_t* sK = sm + Tl::OFF_K;
  uint8_t* sV = sm + Tl::OFF_V;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Tl::OFF_BAR);
  uint64_t* q_full = bars;
  uint64_t* k_full = bars + 1;             // [KST]
  uint64_t* k_empty = k_full + Tl::KST;    // [KST]
  uint64_t* v_full = k_empty + Tl::KST;    // [VST]
  uint64_t* v_empty = v_full + Tl::VST;    // [VST]
  uint64_t* s_full = v_empty + Tl::VST;    // [NST]
  uint64_t* p_full = s_full + NST;         // [NST]
  uint64_t* o_done = p_full + NST;         // [NST]
  uint64_t* xch_bar = o_done + NST;        // [NST]: the stream's two halves have posted
  uint64_t* mma_done = xch_bar + NST;
  float* xch = reinterpret_cast<float*>(sm + Tl::OFF_XCH);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((1 + 2 * Tl::KST + 2 * Tl::VST + 4 * NST + 1) * 8 + 8 <= 256, "barriers");

  constexpr int NKP = Tl::NKP, kProducer = Tl::SWARPS * NST, kIssuer = kProducer + Tl::NPROD;
  const bool producer = warp >= kProducer && warp < kIssuer;
  // A TMA box takes a cache block, or half of one of 128 tokens where a key tile has 64.
  const int SB = min(S, BN), bpt = BN / SB;  // rows per box, boxes per key tile
  static_assert(BN >= 64, "two boxes per block at most");
  const int halved = BN < 128 && S > BN ? 1 : 0;
  const int box0 = t_beg / SB, nblk = (t_end + S - 1) / S;
  const int32_t* table = p.block_tables + static_cast<int64_t>(trow) * p.MB;
  // the block id of this lane's box in key tile j (-1: none or invalid)
  auto block_id = [&](int j) {
    const int lb = (box0 + j * bpt + lane) >> halved;
    int id = -1;
    if (lane < bpt && lb < nblk) {
      id = table[lb];
      if (id < 0 || id >= p.NB) {
        raise_error(PA_DEVERR_BLOCK_ID);
        id = -1;
      }
    }
    return id;
  };
  // part of one K or V tile: every lane issues the boxes of its block (K: of the
  // warp's column blocks; V: one of all column blocks)
  const int col0 = (warp - kProducer) % NKP;
  auto load_tile = [&](bool v, int j, int id) {
    const int st = j % (v ? Tl::VST : Tl::KST);
    uint8_t* dst = (v ? sV : sK) + st * Tl::KV_BYTES;
    uint64_t* full = &(v ? v_full : k_full)[st];
    const int nvalid = __popc(__ballot_sync(kFullMask, id >= 0));
    if (lane == 0)
      mbar_arrive_expect_tx(full, static_cast<uint32_t>(nvalid) * SB * 128 *
                                      (v ? Tl::COLB : Tl::COLB / NKP));
    __syncwarp();
    if (id >= 0) {
      const int y = (id * p.Hkv + hk) * S + (BN < 128 ? (box0 + j) & halved : 0) * SB;
      if (v) {
        tc::tma_load_3d(dst + lane * SB * 128 * Tl::COLB, &tmv, 0, y, 0, full);
      } else {
#pragma unroll
        for (int c = 0; c < Tl::COLB / NKP; ++c) {
          const int col = col0 + c * NKP;
          tma_load_2d_nohint(dst + col * Tl::CB_BYTES + lane * SB * 128, &tmk, col * 64, y, full);
        }
      }
    }
  };
  // whether tile j's stage is free
  auto stage_free = [&](bool v, int j) {
    const int ns = v ? Tl::VST : Tl::KST;
    return j < ns ||
           wait_warp(&(v ? v_empty : k_empty)[j % ns], ((j / ns) - 1) & 1, abort_flag);
  };
  // The producers issue Q and the first tiles before the CTA-wide sync, under the
  // tensor-memory allocation.
  static_assert(Tl::KST == Tl::VST, "the first tiles");
  const bool is_v = warp == kProducer + NKP;
  const int ahead = min(NK, Tl::KST);
  int next_id = -1;
  if (producer) {
    if (warp == kProducer && lane == 0) {
      mbar_init(q_full, 1);
      for (int s = 0; s < Tl::KST; ++s) {
        mbar_init(&k_full[s], NKP);
        mbar_init(&k_empty[s], 1);
        mbar_init(&v_full[s], 1);
        mbar_init(&v_empty[s], 1);
      }
      for (int t = 0; t < NST; ++t) {
        mbar_init(&s_full[t], 1);
        mbar_init(&p_full[t], Tl::SWARPS);  // one arrival per softmax warp
        mbar_init(&o_done[t], 1);
        mbar_init(&xch_bar[t], Tl::SWARPS);
      }
      mbar_init(mma_done, 1);
      *abort_flag = 0;
      fence_mbar_init();
    }
    next_id = block_id(0);
    asm volatile("bar.sync 2, %0;" ::"n"(Tl::NPROD * 32) : "memory");  // the barriers are there
    if (warp == kProducer && lane == 0) {
      mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(nq) * Tl::COLB * G * qpt * 128);
      for (int t = 0; t < nq; ++t)
#pragma unroll
        for (int c = 0; c < Tl::COLB; ++c)
          tc::tma_load_3d(sQ + t * Tl::Q_BYTES + c * Tl::CB_BYTES, &tmq, c * 64, hk * G,
                          q0 + tok0 + t * qpt, q_full);
    }
    __syncwarp();
    for (int j = 0; j < ahead; ++j) {
      load_tile(is_v, j, next_id);
      if (j + 1 < NK) next_id = block_id(j + 1);
    }
  }
  if (warp == kIssuer) {
    __syncwarp();
    tc::tmem_alloc(tmem_slot, Tl::TMEM_COLS);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  auto give_regs = [] {
    if constexpr (Tl::PASS_REGS)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Tl::OTHER_REGS));
  };
  if (producer) {
    give_regs();
    // ---------------- producers: the rest of their operand's tiles ----------------
    int issued = ahead;
    for (int j = ahead; j < NK; ++j) {
      if (!stage_free(is_v, j)) break;
      load_tile(is_v, j, next_id);
      issued = j + 1;
      if (j + 1 < NK) next_id = block_id(j + 1);
    }
    // copies in flight land before the CTA can exit
    if (lane == 0) {
      mbar_wait_bounded(q_full, 0);
      for (int j = max(issued - Tl::KST, 0); j < issued; ++j)
        mbar_wait_bounded(&(is_v ? v_full : k_full)[j % Tl::KST], (j / Tl::KST) & 1);
    }
    __syncwarp();
  } else if (warp == kIssuer) {
    give_regs();
    // ---------------- MMA issuer (one elected lane), V tail zeroing (whole warp) ----------------
    constexpr int fmt = F16 ? 0 : 1;
    constexpr uint32_t idesc_s = tc::instr_desc_f16(fmt, 0, 0, Tl::BM, BN);
    constexpr uint32_t idesc_o = tc::instr_desc_f16(fmt, 0, 1, Tl::BM, D);
    const uint32_t on = elect_one();
    // (addresses are counted in 16 bytes in a descriptor's low 14 bits: a tile's
    // step adds to them without a carry)
    const uint64_t dQ = tc::smem_desc_sw128(smem_u32(sQ), 16, 1024);
    const uint64_t dK = tc::smem_desc_sw128(smem_u32(sK), 16, 1024);
    // V's tile: for each box its COLB column blocks of SB rows one after
    // the other. As an MN-major operand 64 columns lie SB rows apart, and 8 keys
    // 8 rows (one cache block, for S = 8); 16 keys are a whole cache block, or a
    // part of one.
    const uint64_t dV = tc::smem_desc_sw128(smem_u32(sV), SB * 128, S == 8 ? 1024 * Tl::COLB : 1024);
    const int lg = SB <= 16 ? 0 : 31 - __clz(SB >> 4);  // log2 of a block's 16-key steps
    auto issue_s = [&](int t, int j) {  // S_t = Q K_j^T
      const uint64_t qd = dQ + (KSPLIT ? 0 : t) * (Tl::Q_BYTES >> 4);
      const uint64_t kd = dK + (j % Tl::KST) * (Tl::KV_BYTES >> 4);
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        const uint32_t off = ((s >> 2) * Tl::CB_BYTES + (s & 3) * 32) >> 4;
        mma_ss_on(on, tmem + t * TST, qd + off, kd + off, idesc_s, s > 0);
      }
      commit_on(on, &s_full[t]);
    };
    auto issue_pv = [&](int t, int st, uint32_t accumulate) {  // O_t += P_t V
      const uint64_t vd = dV + st * (Tl::KV_BYTES >> 4);
      const uint32_t tS = tmem + t * TST, tO = tS + BN;
#pragma unroll
      for (int s = 0; s < BN / 16; ++s) {
        const uint64_t bdesc =
            vd + static_cast<uint32_t>((((s >> lg) * Tl::COLB << lg) + (s & ((1 << lg) - 1))) * 128);
        const uint32_t pa = tS + 32 * (s >> 1) + 8 * (s & 1);  // keys 16s .. 16s + 15
        mma_ts_on(on, tO, pa, bdesc, idesc_o, s > 0 ? 1u : accumulate);
        mma_ts_on(on, tO, pa + 16, bdesc, idesc_o, 1u);
      }
    };
    auto k_ready = [&](int j) {
      const bool r = wait_warp(&k_full[j % Tl::KST], (j / Tl::KST) & 1, abort_flag);
      tc::fence_after_sync();
      return r;
    };
    bool ok = wait_warp(q_full, 0, abort_flag) && k_ready(0);
    if (ok) {
      for (int t = 0; t < nq; ++t) issue_s(t, 0);
      commit_on(on, &k_empty[0]);
      if (KSPLIT && NK > 1) {
        ok = k_ready(1);
        if (ok) {
          issue_s(1, 1);
          commit_on(on, &k_empty[1 % Tl::KST]);
        }
      }
    }
    for (int j = 0; ok && j < NK; ++j) {
      const int st = j % Tl::VST;
      ok = wait_warp(&v_full[st], (j / Tl::VST) & 1, abort_flag);
      if (!ok) break;
      const int kb = t_beg + j * BN;
      if (kb + BN > t_end) {
        // keys past the end: P is 0 there, and 0 * NaN would not be
        uint8_t* vs = sV + st * Tl::KV_BYTES;
        for (int r = t_end - kb + lane; r < BN; r += 32) {
          uint8_t* row = vs + (r / SB * Tl::COLB * SB + r % SB) * 128;
#pragma unroll
          for (int c = 0; c < Tl::COLB; ++c)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              reinterpret_cast<uint4*>(row + c * SB * 128)[k] = make_uint4(0, 0, 0, 0);
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
      }
      if constexpr (KSPLIT) {
        const int t = j & 1;
        ok = wait_warp(&p_full[t], (j >> 1) & 1, abort_flag);
        if (!ok) break;
        tc::fence_after_sync();
        issue_pv(t, st, j > 1);
        if (j + 2 >= NK) commit_on(on, &o_done[t]);
        commit_on(on, &v_empty[st]);
        if (j + 2 < NK) {
          ok = k_ready(j + 2);
          if (!ok) break;
          issue_s(t, j + 2);
          commit_on(on, &k_empty[(j + 2) % Tl::KST]);
        }
      } else {
        for (int t = 0; ok && t < nq; ++t) {
          ok = wait_warp(&p_full[t], j & 1, abort_flag);
          if (!ok) break;
          tc::fence_after_sync();
          issue_pv(t, st, j > 0);
          if (j == NK - 1) commit_on(on, &o_done[t]);
          if (j + 1 < NK) {
            ok = k_ready(j + 1);
            if (!ok) break;
            issue_s(t, j + 1);
          }
        }
        if (ok) {
          commit_on(on, &v_empty[st]);
          if (j + 1 < NK) commit_on(on, &k_empty[(j + 1) % Tl::KST]);
        }
      }
    }
    // every MMA issued has completed before tensor memory is released
    __syncwarp();
    commit_on(on, mma_done);
    mbar_wait_bounded(mma_done, 0);
    __syncwarp();
  } else if (warp < kProducer) {
    if constexpr (Tl::PASS_REGS)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Tl::SOFTMAX_REGS));
    // ---------------- softmax: SWARPS warps serve a stream; where they are two
    // warpgroups, half hw of them takes keys 64 hw .. 64 hw + 63 of each key tile and
    // output columns hw D / 2 .. of each row; thread r of a warpgroup owns row r ----------------
    constexpr int HK = BN / HALVES;  // keys per half
    constexpr int HD = D / HALVES;   // output columns per half
    static_assert(HK == 64, "scores per thread");
    const int t = warp / Tl::SWARPS;
    const int hw = (warp >> 2) & (HALVES - 1);
    const int r = threadIdx.x & 127;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tT = tmem + t * TST + lane_base;
    const uint32_t tS = tT + hw * HK, tO = tT + BN + hw * HD;
    const int nrow = rows_of(t);
    const bool row_on = r < nrow;
    const bool warp_on = (warp & 3) * 32 < nrow;  // a warp without rows only keeps step
    const int rtok = r / G;
    const int tok = q0 + tok0 + (KSPLIT ? 0 : t * qpt) + rtok;  // this row's query token
    const int head = hk * G + (r - rtok * G);
    int lim = t_end;  // this row sees the keys below
    if (p.shared_lens && row_on)
      lim = min(lim, shared_part(p.shared_lens[tok], p.lens[tok], p.L_cap, S));
    float m = -INFINITY, l = 0.f;  // l: this half's share of the running sum
    const int nkt = tiles_of(t);
    bool ok = nkt > 0;
    auto slot = [&](int j, int half) { return xch + ((t * 2 + (j & 1)) * 2 + half) * Tl::BM; };
    for (int j = 0; ok && j < nkt; ++j) {
      ok = wait_warp(&s_full[t], j & 1, abort_flag);
      if (!ok) break;
      if (!warp_on) {  // (one arrival per phase: it waits for the phase it arrived at)
        if constexpr (HALVES == 2) {
          arrive_warp(&xch_bar[t], lane);
          ok = wait_warp(&xch_bar[t], j & 1, abort_flag);
          if (!ok) break;
        }
        arrive_warp(&p_full[t], lane);
        continue;
      }
      tc::fence_after_sync();
      const int kb = t_beg + (KSPLIT ? 2 * j + t : j) * BN + hw * HK;
      float x[HK];
      {
        uint32_t u[HK];
#pragma unroll
        for (int c4 = 0; c4 < HK / 32; ++c4)
          tc::tmem_ld32(tS + c4 * 32, *reinterpret_cast<uint32_t(*)[32]>(&u[c4 * 32]));
        tc::tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < HK; ++c) x[c] = __uint_as_float(u[c]);
        if (kb + HK > lim) {  // only tiles that reach past the row's last key pay for the mask
#pragma unroll
          for (int c = 0; c < HK; ++c) x[c] = kb + c >= lim ? -INFINITY : x[c];
        }
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < HK; c += 2) mx[(c >> 1) & 3] = fmax3(mx[(c >> 1) & 3], x[c], x[c + 1]);
      const float hmax = fmax3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
      float rmax = hmax;
      if constexpr (HALVES == 2) {
        // the row's max over both halves (slots alternate with the key tile, so a
        // half never overwrites a value the other has not read yet)
        slot(j, hw)[r] = hmax;
        arrive_warp(&xch_bar[t], lane);
        ok = wait_warp(&xch_bar[t], j & 1, abort_flag);
        if (!ok) break;
        rmax = fmaxf(hmax, slot(j, hw ^ 1)[r]);
      }
      // The reference max only moves when the tile max exceeds it by more than
      // 2^8 in weight; the weights stay <= 256 (2^15 with f16's shift), exact in the
      // final ratio. For bf16 it is scale x the score, a score's distance from it
      // one fused operation, and the weight of a score whose 32-bit steps exceed 1
      // (2^24 and more) off by up to half a step, which bf16 has the range for and
      // the ratio cancels. f16 has not, so there m is a score and the distance is
      // taken before it is scaled.
      const float top = F16 ? rmax : rmax * p.scale_log2;
      const bool grow = F16 ? (top - m) * p.scale_log2 > 8.f : top > m + 8.f;  // (from m = -inf too)
      const float m_use = grow ? top : m;
      const float alpha = grow ? fast_exp2(F16 ? (m - m_use) * p.scale_log2 : m - m_use) : 1.f;
      m = m_use;
      // a row without keys so far keeps m = -inf; its weights are 2^-inf = 0
      const float m_ref = m_use == -INFINITY ? 0.f : m_use;
      // P over this half's scores, 8 keys at a time: keys 2k, 2k+1 of a 32-key
      // chunk q as one 16-bit pair in column 32q + k, and the pair's rounding
      // residues, themselves rounded, in column 32q + 16 + k
      const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
      const float2 nm2 = make_float2(-m_ref, -m_ref);
      const float2 shift2 = make_float2(kWeightShift, kWeightShift);
      float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int g = 0; g < HK / 8; ++g) {
        float* v = &x[8 * g];
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 vv = make_float2(v[2 * e], v[2 * e + 1]);
          const float2 tt = F16 ? ffma2(fadd2(vv, nm2), sc2, shift2) : ffma2(vv, sc2, nm2);
          const float2 pe = make_float2(fast_exp2(tt.x), fast_exp2(tt.y));
          acc[e & 1] = fadd2(acc[e & 1], pe);
          hi[e] = pack_pair<T>(pe.x, pe.y);
          const float2 hh = Elem<T>::pair(hi[e]);
          lo[e] = pack_pair<T>(pe.x - hh.x, pe.y - hh.y);
        }
        const uint32_t col = 32 * (g >> 2) + 4 * (g & 3);  // within this half's 64 columns
        tc::tmem_st4(tS + col, hi);
        tc::tmem_st4(tS + col + 16, lo);
      }
      // The stream's previous product has completed (the commit that released
      // these scores covers it): rescale the rows whose max moved.
      if (j > 0 && __any_sync(kFullMask, grow)) {
#pragma unroll 1
        for (int c4 = 0; c4 < HD / 32; ++c4) {
          uint32_t u[32];
          tc::tmem_ld32(tO + c4 * 32, u);
          tc::tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c) u[c] = __float_as_uint(__uint_as_float(u[c]) * alpha);
          tc::tmem_st32(tO + c4 * 32, u);
        }
      }
      l = l * alpha + ((acc[0].x + acc[0].y) + (acc[1].x + acc[1].y));
      tc::tmem_wait_st();
      tc::fence_before_sync();
      arrive_warp(&p_full[t], lane);
    }
    if constexpr (HALVES == 2) {  // the row's sum over both halves
      if (ok) {
        slot(nkt, hw)[r] = l;
        arrive_warp(&xch_bar[t], lane);
        ok = wait_warp(&xch_bar[t], nkt & 1, abort_flag);
      }
      if (ok) l += slot(nkt, hw ^ 1)[r];
    }
    if constexpr (F16) m *= p.scale_log2;
    if (ok) ok = wait_warp(&o_done[t], 0, abort_flag);
    // The output columns this warp finishes, and its weights: of this stream's
    // result and (KSPLIT) of the other's. Joining, stream t finishes the t-th half
    // of each half's columns, and leaves the others to the other stream.
    constexpr int FC = KSPLIT ? HD / 2 : HD;   // columns to finish
    constexpr int CH = 32;                     // columns at a time
    static_assert(FC % CH == 0, "whole loads of columns");
    const int col0 = hw * HD + (KSPLIT ? t * FC : 0);
    float w0 = 1.f, w1 = 0.f;
    // 4 KB for its output on the way out: of the stream's query tile, or, of a
    // single stream, of the K ring
    const int sw = warp & (Tl::SWARPS - 1);  // of the stream's warps
    uint8_t* buf = (NST == 1 ? sK : sQ + (KSPLIT ? 0 : t) * Tl::Q_BYTES) + sw * 4096;
    static_assert(NST == 1 ? Tl::KST * Tl::KV_BYTES >= 32768 : Tl::Q_BYTES >= Tl::SWARPS * 4096,
                  "the warps' buffers");
    float* jO = reinterpret_cast<float*>(sK);   // [D][128] the columns left, by column
    float* jml = reinterpret_cast<float*>(sV);  // [stream][2][128] m and l
    bool join = false;
    if constexpr (KSPLIT) {
      if (t == 1) buf = sV + Tl::VST * Tl::KV_BYTES / 2 + sw * 4096;
      join = NK > 1;
      // The rings' memory is free once both streams' MMAs are done with it.
      if (join && ok) ok = wait_warp(&o_done[t ^ 1], 0, abort_flag);
      if (join && ok && warp_on) {
        tc::fence_after_sync();
        const int left = hw * HD + (t ^ 1) * FC;  // columns for the other stream
#pragma unroll 1
        for (int c0 = 0; c0 < FC; c0 += CH) {
          uint32_t u[CH];
          tc::tmem_ld32(tT + BN + left + c0, u);
          tc::tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < CH; ++c) jO[(left + c0 + c) * 128 + r] = __uint_as_float(u[c]);
        }
        if (hw == 0) {
          jml[t * 256 + r] = m;
          jml[t * 256 + 128 + r] = l;
        }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(Tl::STHREADS) : "memory");  // every softmax thread, aborted or not
      if (join && ok) {
        const float mo = jml[(t ^ 1) * 256 + r], lo = jml[(t ^ 1) * 256 + 128 + r];
        const float M = fmaxf(m, mo);
        w0 = m == -INFINITY ? 0.f : fast_exp2(m - M);
        w1 = mo == -INFINITY ? 0.f : fast_exp2(mo - M);
        l = w0 * l + w1 * lo;
        m = M;
      }
      // one key tile: stream 0 alone has a result, and finishes all its columns
    }
    if (ok && warp_on) {
      tc::fence_after_sync();
      const int64_t ih = static_cast<int64_t>(tok) * p.H + head;
      constexpr float kUnshift = F16 ? 0x1p-7f : 1.f;  // (of partial results)
      const float inv = direct ? (l != 0.f ? 1.f / l : 0.f) : kUnshift;
      const float f0 = w0 * inv, f1 = w1 * inv;
      const int rows = nrow - (warp & 3) * 32;  // this warp's
      const int n_cols = KSPLIT && !join ? HD : FC;
      void* dst = direct ? p.out : static_cast<void*>(p.ws_acc);
      const pa_dtype dst_dt = direct ? p.out_dt : PA_F32;
      const int64_t row_at = (direct ? ih : ih * p.NP + part) * D;
#pragma unroll 1
      for (int c0 = 0; c0 < n_cols; c0 += CH) {
        uint32_t u[CH];
        tc::tmem_ld32(tT + BN + col0 + c0, u);
        tc::tmem_wait_ld();
        float v[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) v[c] = __uint_as_float(u[c]) * f0;
        if (join) {
#pragma unroll
          for (int c = 0; c < CH; ++c) v[c] = fmaf(jO[(col0 + c0 + c) * 128 + r], f1, v[c]);
        }
        store_out(buf, v, dst, dst_dt, row_at + col0 + c0, rows, lane);
      }
      if (!direct && hw == 0 && row_on && (!join || t == 0)) {
        p.ws_m[ih * p.NP + part] = m;
        p.ws_l[ih * p.NP + part] = l * kUnshift;
      }
    }
  } else {
    give_regs();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kIssuer) {
    __syncwarp();
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, Tl::TMEM_COLS);
  }
}

// ---- merges ---------------------------------------------------------------------

// The log-sum-exp join of one (row, head)'s results, by one warp: slots
// a0 .. a0 + na - 1 and b0 .. b0 + nb - 1 (in that order) of its NP,
//   M = max m;  out = sum 2^(m - M) acc / sum 2^(m - M) l;  all zero without any.
template <int D>
__device__ __forceinline__ void merge_row(const float* ws_m, const float* ws_l,
                                          const float* ws_acc, int64_t ih, int NP, int a0, int na,
                                          int b0, int nb, void* out, pa_dtype out_dt, int lane) {
  constexpr int DL = D / 32;
  const float* m = ws_m + ih * NP;
  const float* l = ws_l + ih * NP;
  const float* acc = ws_acc + ih * NP * D + lane * DL;
  const int n = na + nb;
  auto slot_of = [&](int q) { return q < na ? a0 + q : b0 + (q - na); };
  // the first results' rows and everyone's m and l are asked for together
  constexpr int FIRST = D == 256 ? 4 : 8;
  float2 v0[FIRST][DL / 2];
#pragma unroll
  for (int r = 0; r < FIRST; ++r)
    if (r < n) {
#pragma unroll
      for (int e = 0; e < DL / 2; ++e)
        v0[r][e] = reinterpret_cast<const float2*>(
            acc + static_cast<int64_t>(slot_of(r)) * D)[e];
    }
  const float m0 = lane < n ? m[slot_of(lane)] : -INFINITY;
  const float l0 = lane < n ? l[slot_of(lane)] : 0.f;
  float M = m0;
  for (int q = lane + 32; q < n; q += 32) M = fmaxf(M, m[slot_of(q)]);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, o));
  float lsum = 0.f, a[DL];
#pragma unroll
  for (int e = 0; e < DL; ++e) a[e] = 0.f;
  for (int c = 0; c < n; c += 32) {
    const int q = c + lane;
    float wq = 0.f;
    if (q < n) {
      const float mq = c == 0 ? m0 : m[slot_of(q)];
      wq = mq == -INFINITY ? 0.f : exp2f(mq - M);
      lsum = fmaf(wq, c == 0 ? l0 : l[slot_of(q)], lsum);
    }
    const int lim = min(32, n - c);
    if (c == 0) {
#pragma unroll
      for (int r = 0; r < FIRST; ++r) {
        const float w = __shfl_sync(kFullMask, wq, r);
        if (r < n) {
#pragma unroll
          for (int e = 0; e < DL / 2; ++e) {
            a[2 * e] = fmaf(w, v0[r][e].x, a[2 * e]);
            a[2 * e + 1] = fmaf(w, v0[r][e].y, a[2 * e + 1]);
          }
        }
      }
    }
#pragma unroll 4
    for (int r = c == 0 ? FIRST : 0; r < lim; ++r) {
      const float w = __shfl_sync(kFullMask, wq, r);
      const float* row = acc + static_cast<int64_t>(slot_of(c + r)) * D;
#pragma unroll
      for (int e = 0; e < DL; e += 2) {
        const float2 v = *reinterpret_cast<const float2*>(row + e);
        a[e] = fmaf(w, v.x, a[e]);
        a[e + 1] = fmaf(w, v.y, a[e + 1]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) lsum += __shfl_xor_sync(kFullMask, lsum, o);
  // (a sum that is NaN, of a NaN in q or in a key, stays NaN)
  const float inv = lsum != 0.f ? 1.f / lsum : 0.f;
  const int64_t at = ih * D + lane * DL;
#pragma unroll
  for (int e = 0; e < DL; ++e) {
    const float o = a[e] * inv;
    if (out_dt == PA_F32)
      static_cast<float*>(out)[at + e] = o;
    else if (out_dt == PA_BF16)
      static_cast<__nv_bfloat16*>(out)[at + e] = __float2bfloat16_rn(o);
    else
      static_cast<__half*>(out)[at + e] = __float2half_rn(o);
  }
}

// pa_cross: joins the partitions of the requests that have more than one. Grid:
// (warps of (row, head) pairs, request).
template <int D>
__global__ void __launch_bounds__(128) cross_merge_kernel(const RowsParams p) {
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.y;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int q0 = p.start[i], q1 = p.start[i + 1];
  int L = p.lens[i];
  grid_dependency_wait();
  const int n = q1 - q0;
  if (n < 0 || q0 < 0 || q1 > p.T || n > p.max_rows) return;
  L = max(0, min(L, p.L_cap));
  const int parts = static_cast<int>((static_cast<int64_t>(L) + p.P - 1) / p.P);
  if (parts <= 1 || w >= static_cast<int64_t>(n) * p.H) return;
  merge_row<D>(p.ws_m, p.ws_l, p.ws_acc, static_cast<int64_t>(q0) * p.H + w, p.NP, 0, parts, 0, 0,
               p.out, p.out_dt, lane);
}

}  // namespace pa
