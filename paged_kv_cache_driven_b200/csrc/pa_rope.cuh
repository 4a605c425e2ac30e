// Rotary positions with per-head norms, alone and with the append to the paged
// cache on the way (pa_rope, pa_rope_append, pa_rope_append_fp8).
//
// A row is one head's D elements of one token. With x its fp32 values:
//   x <- x * (1 / sqrt(mean(x^2) + eps)) * weight        (where a weight is given)
//   (a, b) <- (a c - b s, b c + a s)                      for each rotated pair,
// c, s = amplitude * cos, sin of 2 pi frac(position * table[pair]), elements
// past rot_dim unchanged; then one rounding to the output type (or to E4M3
// after the division by the cache's scale). The turns position * table[pair]
// are taken in 64 bits and reduced before they become an angle: in fp32 a
// position of 10^6 would leave an angle with an error of some 0.06.
//
// A stream bound by HBM, close to being bound by instructions: each value is read
// once and written once, and a value's share of a thread's work is some eight
// instructions. One CTA takes up to 8 tokens (kRopeTokens) with all their rows,
// or, of few tokens, a run of one token's rows. Their sines and cosines are
// computed once, into shared memory, under the first rows' loads. A thread owns
// EPT elements of a row (16; 8 where the sizes do not divide), LPR threads a
// row, 256 / LPR rows at a time, and loads a row ahead of the one that it works
// on: 16 elements halve what a row costs in addresses, shuffles and shared
// memory against 8. What a thread owns are pairs, not consecutive elements: in
// the half layout it loads two 16-byte pieces rot_dim / 2 apart, which keeps both
// components of a pair in one thread (no exchange between lanes). Its pairs go two
// by two through the packed fp32 instructions.
#pragma once

#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {

// How a row's elements are paired and moved.
enum : int {
  kPairs = 0,     // interleaved: elements 2j, 2j + 1; a thread's are consecutive
  kHalf = 1,      // elements j, j + rot / 2: two pieces of EPT / 2 elements, aligned
  kHalfAny = 2    // the same for any even rot: single elements (16,384 tokens of 32 + 32
                  // heads of 96: 174 us with 24 rotated, 86 with all by kHalf)
};
enum : int { kNoCache = 0, kCache16 = 1, kCache8 = 2 };
constexpr int kRopeTokens = 8;  // most tokens of a CTA

// A thread's elements of a row, as they lie in memory: EPT / 2 pairs.
template <int EPT>
struct PairFrag {
  uint32_t w[EPT / 2];
};

// The elements a, b of pair j in the half layouts: rotated pairs lie rot / 2
// apart, the others (which pass through) (D - rot) / 2 apart.
__device__ __forceinline__ void half_pair(int j, int rot, int D, int& a, int& b) {
  const int r2 = rot >> 1;
  if (j < r2) {
    a = j;
    b = j + r2;
  } else {
    a = rot + (j - r2);
    b = a + ((D - rot) >> 1);
  }
}

// Where a thread's elements lie in a row: its first pair, and the elements of
// its two pieces (kPairs: a its first element).
struct Place {
  int pair, a, b;
};

// kPairs: word e = pair e; the half layouts: the first EPT / 4 words components a
// of pairs 0, 1, ..., the others components b.
template <int LAYOUT, int EPT>
__device__ __forceinline__ PairFrag<EPT> load_pairs(const uint16_t* row, const Place& pc, int rot,
                                                    int D) {
  PairFrag<EPT> f;
  if constexpr (LAYOUT == kHalfAny) {
#pragma unroll
    for (int e = 0; e < EPT / 4; ++e) {
      uint32_t u[2], v[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        int a, b;
        half_pair(pc.pair + 2 * e + k, rot, D, a, b);
        u[k] = row[a];
        v[k] = row[b];
      }
      f.w[e] = u[0] | (u[1] << 16);
      f.w[EPT / 4 + e] = v[0] | (v[1] << 16);
    }
  } else {
#pragma unroll
    for (int k = 0; k < EPT / 8; ++k) {
      const uint16_t* src = LAYOUT == kPairs ? row + pc.a + 8 * k : row + (k == 0 ? pc.a : pc.b);
      const uint4 x = __ldcs(reinterpret_cast<const uint4*>(src));
      f.w[4 * k] = x.x, f.w[4 * k + 1] = x.y, f.w[4 * k + 2] = x.z, f.w[4 * k + 3] = x.w;
    }
  }
  return f;
}

template <int LAYOUT, int EPT>
__device__ __forceinline__ void store_pairs(uint16_t* row, const Place& pc, int rot, int D,
                                            const PairFrag<EPT>& f) {
  if constexpr (LAYOUT == kHalfAny) {
#pragma unroll
    for (int e = 0; e < EPT / 2; ++e) {
      int a, b;
      half_pair(pc.pair + e, rot, D, a, b);
      row[a] = static_cast<uint16_t>(f.w[e >> 1] >> (16 * (e & 1)));
      row[b] = static_cast<uint16_t>(f.w[EPT / 4 + (e >> 1)] >> (16 * (e & 1)));
    }
  } else {
#pragma unroll
    for (int k = 0; k < EPT / 8; ++k) {
      uint16_t* dst = LAYOUT == kPairs ? row + pc.a + 8 * k : row + (k == 0 ? pc.a : pc.b);
      *reinterpret_cast<uint4*>(dst) =
          make_uint4(f.w[4 * k], f.w[4 * k + 1], f.w[4 * k + 2], f.w[4 * k + 3]);
    }
  }
}

// Components a and b of the pairs in fp32, two pairs to a vector, and back (one
// rounding).
template <typename T, int LAYOUT, int EPT>
__device__ __forceinline__ void unpack_pairs(const PairFrag<EPT>& f, float2 (&a)[EPT / 4],
                                             float2 (&b)[EPT / 4]) {
#pragma unroll
  for (int e = 0; e < EPT / 4; ++e) {
    if constexpr (LAYOUT == kPairs) {
      const float2 u = Elem<T>::pair(f.w[2 * e]), v = Elem<T>::pair(f.w[2 * e + 1]);
      a[e] = make_float2(u.x, v.x);
      b[e] = make_float2(u.y, v.y);
    } else {
      a[e] = Elem<T>::pair(f.w[e]);
      b[e] = Elem<T>::pair(f.w[EPT / 4 + e]);
    }
  }
}

template <typename T>
__device__ __forceinline__ uint32_t pack16(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack16<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack16<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <typename T, int LAYOUT, int EPT>
__device__ __forceinline__ PairFrag<EPT> pack_pairs(const float2 (&a)[EPT / 4],
                                                    const float2 (&b)[EPT / 4]) {
  PairFrag<EPT> f;
#pragma unroll
  for (int e = 0; e < EPT / 4; ++e) {
    if constexpr (LAYOUT == kPairs) {
      f.w[2 * e] = pack16<T>(a[e].x, b[e].x);
      f.w[2 * e + 1] = pack16<T>(a[e].y, b[e].y);
    } else {
      f.w[e] = pack16<T>(a[e].x, a[e].y);
      f.w[EPT / 4 + e] = pack16<T>(b[e].x, b[e].y);
    }
  }
  return f;
}

__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)));
  return as_f2(d);
}

// The divisor of an E4M3 cache: fp32 quotients x / scale, correctly rounded (the
// rule of kv_append_fp8_kernel), for two values at a time. With y = RN(1 / scale),
// q = x y is off by less than two units in the last place, one correction
// q + (x - scale q) y makes it a faithful quotient, and a second one, by Markstein's
// theorem ("Computation of elementary functions on the IBM RISC System/6000
// processor", 1990), the correctly rounded one; the remainders are exact as long
// as nothing leaves the normal range. So x is first cut to +-512 scale, whose
// codes are those of the limit 448 all the same (NaN stays NaN), and scales lie in
// [2^-60, 2^60]. (Quotients so small that a remainder is not exact are far below
// 2^-10, code 0.) 12,289 tokens of 32 heads: 105 us a call; a branch to the
// division for other scales took 7 us more.
struct Quotient {
  float scale, inv, lim;
  __device__ __forceinline__ explicit Quotient(float s)
      : scale(s), inv(1.f / s), lim(512.f * s) {}
  __device__ __forceinline__ float cut(float x) const {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(lim));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(y), "f"(-lim));
    return y;
  }
  // (on -x, and with the remainder's sign turned: a correction by it then leaves
  // the sign of a zero quotient as it is)
  __device__ __forceinline__ float2 of(float2 x) const {
    const float2 n = make_float2(cut(-x.x), cut(-x.y));
    const float2 ny = make_float2(-inv, -inv), s = make_float2(scale, scale);
    float2 q = fmul2(n, ny);
    q = ffma2(ffma2(s, q, n), ny, q);
    return ffma2(ffma2(s, q, n), ny, q);
  }
};

// The pairs as E4M3 codes of fp32(value / scale) (round to nearest even,
// saturated), stored to a row of codes.
template <int LAYOUT, int EPT>
__device__ __forceinline__ void store_codes(uint8_t* row, const Place& pc, int rot, int D,
                                            const float2 (&a)[EPT / 4], const float2 (&b)[EPT / 4],
                                            const Quotient& div) {
  uint32_t ca[EPT / 8], cb[EPT / 8];  // kPairs: codes 0-7, 8-15 in order; else a's, b's
#pragma unroll
  for (int e = 0; e < EPT / 8; ++e) {
    const float2 x0 = div.of(a[2 * e]), x1 = div.of(a[2 * e + 1]);
    const float2 y0 = div.of(b[2 * e]), y1 = div.of(b[2 * e + 1]);
    if constexpr (LAYOUT == kPairs) {
      ca[e] = float2_to_e4m3x2(x0.x, y0.x) |
              (static_cast<uint32_t>(float2_to_e4m3x2(x0.y, y0.y)) << 16);
      cb[e] = float2_to_e4m3x2(x1.x, y1.x) |
              (static_cast<uint32_t>(float2_to_e4m3x2(x1.y, y1.y)) << 16);
    } else {
      ca[e] = float2_to_e4m3x2(x0.x, x0.y) |
              (static_cast<uint32_t>(float2_to_e4m3x2(x1.x, x1.y)) << 16);
      cb[e] = float2_to_e4m3x2(y0.x, y0.y) |
              (static_cast<uint32_t>(float2_to_e4m3x2(y1.x, y1.y)) << 16);
    }
  }
  if constexpr (LAYOUT == kPairs) {
    if constexpr (EPT == 16)
      *reinterpret_cast<uint4*>(row + pc.a) = make_uint4(ca[0], cb[0], ca[1], cb[1]);
    else
      *reinterpret_cast<uint2*>(row + pc.a) = make_uint2(ca[0], cb[0]);
  } else if constexpr (LAYOUT == kHalf) {
    static_assert(EPT == 16, "the half layout's pieces are 8 elements");
    *reinterpret_cast<uint2*>(row + pc.a) = make_uint2(ca[0], ca[1]);
    *reinterpret_cast<uint2*>(row + pc.b) = make_uint2(cb[0], cb[1]);
  } else {
#pragma unroll
    for (int e = 0; e < EPT / 2; ++e) {
      int ia, ib;
      half_pair(pc.pair + e, rot, D, ia, ib);
      row[ia] = static_cast<uint8_t>(ca[e >> 2] >> (8 * (e & 3)));
      row[ib] = static_cast<uint8_t>(cb[e >> 2] >> (8 * (e & 3)));
    }
  }
}

// One operand's rows of a CTA: `nr` heads of each of ntok tokens from `row` (the
// first token's first head), numbered token after token; a thread walks numbers
// sub, sub + RPP, ... by steps, without a division.
struct Rows {
  const uint16_t* ptr;  // the thread's next row
  int64_t jump;         // elements from a token's last row to the next one's first
  int nr, tok, row;     // tok, row of that next row
  __device__ __forceinline__ void normalise() {
    while (row >= nr) {
      row -= nr;
      ++tok;
      ptr += jump;
    }
  }
};

// The rows of a token: H of q, Hkv of k, and with a cache Hkv of v. LPR:
// threads per row, a power of two >= D / EPT. A CTA takes the rows row0 .. row1 - 1
// of `toks` tokens from token t0, operand after operand: v (a copy), k, q.
template <typename T, int LAYOUT, int MODE, int EPT, int LPR>
__global__ void __launch_bounds__(256, 4) rope_kernel(const RopeParams p) {
  constexpr int RPP = 256 / LPR;      // rows the CTA takes at a time
  constexpr int PT = EPT / 2;         // pairs of a thread
  constexpr int NV = EPT / 4;         // vectors of two pairs
  constexpr int NP = LPR * PT;        // pairs of a row, rounded up
  using Frag = PairFrag<EPT>;
  // by pair, a thread's groups of four LPR groups apart (16-byte loads of
  // neighbouring threads are then neighbours)
  __shared__ __align__(16) float s_cos[kRopeTokens][NP], s_sin[kRopeTokens][NP];
  __shared__ __align__(16) float s_neg[kRopeTokens][NP];    // -sin
  __shared__ __align__(16) float s_wa[2][NP], s_wb[2][NP];  // norm weights, q and k
  __shared__ int64_t s_dst[kRopeTokens];  // cache element of (head 0, this token), or -1
  auto at_pair = [](int j) { return ((j % PT / 4) * LPR + j / PT) * 4 + j % 4; };
  const int D = p.D, rot = p.rot, half = p.rot >> 1;
  const int grp = blockIdx.x / p.chunks;
  const int row0 = (blockIdx.x - grp * p.chunks) * p.chunk_rows;
  const int row1 = min(row0 + p.chunk_rows, p.rows);
  const int t0 = grp * p.toks;
  const int ntok = min(p.toks, p.T - t0);
  const int sub = threadIdx.x / LPR, pl = threadIdx.x % LPR;
  const bool lane_on = pl * EPT < D;
  Place pc{pl * PT, pl * EPT, 0};
  if constexpr (LAYOUT != kPairs) half_pair(pc.pair, rot, D, pc.a, pc.b);
  // this CTA's heads of q, k and v
  const int qh = min(row0, p.H), qn = min(row1, p.H) - qh;
  const int kh = min(max(row0 - p.H, 0), p.Hkv), kn = min(max(row1 - p.H, 0), p.Hkv) - kh;
  const int vs = p.H + p.Hkv;
  const int vh = max(row0 - vs, 0), vn = MODE == kNoCache ? 0 : max(row1 - vs, 0) - vh;

  auto rows_of = [&](const void* base, int64_t stride, int h0, int nr) {
    Rows r;
    r.ptr = static_cast<const uint16_t*>(base) + t0 * stride + static_cast<int64_t>(h0 + sub) * D;
    r.jump = stride - static_cast<int64_t>(nr) * D;
    r.nr = nr;
    r.tok = 0;
    r.row = sub;
    return r;
  };
  // loads the next row (nothing past the last token), and steps on
  auto load_next = [&](Rows& r) {
    Frag f{};
    r.normalise();
    if (r.tok < ntok && lane_on) f = load_pairs<LAYOUT, EPT>(r.ptr, pc, rot, D);
    r.row += RPP;
    r.ptr += RPP * D;
    return f;
  };
  Rows rq = rows_of(p.q, p.q_stride, qh, qn), rk = rows_of(p.k, p.k_stride, kh, kn), rv{};
  Frag fq{}, fk{}, fv{};
  if (qn > 0) fq = load_next(rq);
  if (kn > 0) fk = load_next(rk);
  if constexpr (MODE != kNoCache) {
    rv = rows_of(p.v, p.v_stride, vh, vn);
    if (vn > 0) fv = load_next(rv);
  }

  // the tokens' sines and cosines, their places in the cache, the norm weights
  for (int x = threadIdx.x; x < ntok * half; x += 256) {
    const int tok = x / half, j = x - tok * half;
    const double turns = __ldg(p.table + j);
    const double pos = static_cast<double>(__ldg(p.positions + t0 + tok));
    const double r = fma(pos, turns, -rint(pos * turns));  // [-1/2, 1/2]
    float sn, cs;
    sincospif(2.f * static_cast<float>(r), &sn, &cs);
    s_cos[tok][at_pair(j)] = cs * p.amplitude;
    s_sin[tok][at_pair(j)] = sn * p.amplitude;
    s_neg[tok][at_pair(j)] = -(sn * p.amplitude);
  }
  if (MODE != kNoCache && threadIdx.x < ntok) {
    const int64_t slot = __ldg(p.slots + t0 + threadIdx.x);
    int64_t dst = -1;
    if (slot >= p.n_slots) {
      if (row0 == 0) raise_error(PA_DEVERR_SLOT);
    } else if (slot >= 0) {
      const int64_t blk = slot / p.S;
      dst = (blk * p.Hkv * p.S + (slot - blk * p.S)) * D;
    }
    s_dst[threadIdx.x] = dst;
  }
  if (threadIdx.x < LPR && lane_on) {
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const void* wt = part == 0 ? p.q_weight : p.k_weight;
      if (!wt) continue;
      float2 a[NV], b[NV];
      unpack_pairs<T, LAYOUT, EPT>(
          load_pairs<LAYOUT, EPT>(static_cast<const uint16_t*>(wt), pc, rot, D), a, b);
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        *reinterpret_cast<float2*>(&s_wa[part][at_pair(pc.pair + 2 * e)]) = a[e];
        *reinterpret_cast<float2*>(&s_wb[part][at_pair(pc.pair + 2 * e)]) = b[e];
      }
    }
  }
  __syncthreads();
  const float inv_d = 1.f / static_cast<float>(D);
  const int64_t head_step = static_cast<int64_t>(p.S) * D;

  // this thread's NV vectors of a table by pair
  auto by_pair = [&](const float* tab, float2 (&v)[NV]) {
#pragma unroll
    for (int e = 0; e < NV; e += 2) {
      const float4 x = *reinterpret_cast<const float4*>(tab + (e / 2 * LPR + pl) * 4);
      v[e] = make_float2(x.x, x.y);
      v[e + 1] = make_float2(x.z, x.w);
    }
  };
  // All rows of an operand: `work(fragment, token, head)` on the loaded row while
  // the next one is on its way. Every thread of the CTA takes every turn (the
  // norm's shuffles need whole warps); turns past the last row have on = false.
  auto run = [&](Rows& r, Frag cur, int h0, auto&& work) {
    if (r.nr <= 0) return;
    const int total = ntok * r.nr;
    int tok = 0, row = sub;  // the row being worked on
#pragma unroll 1
    for (int base = 0; base < total; base += RPP) {
      const Frag nxt = load_next(r);
      while (row >= r.nr) {
        row -= r.nr;
        ++tok;
      }
      work(cur, tok, h0 + row, tok < ntok && lane_on);
      row += RPP;
      cur = nxt;
    }
  };
  // norm and rotation of a row; what: 0 q, 1 k
  auto turn = [&](const Frag& f, int what, bool norm, int tok, bool on, float2 (&a)[NV],
                  float2 (&b)[NV]) {
    unpack_pairs<T, LAYOUT, EPT>(f, a, b);
    if (norm) {
      float2 s2 = fmul2(a[0], a[0]), z2 = fmul2(b[0], b[0]);
#pragma unroll
      for (int e = 1; e < NV; ++e) {
        s2 = ffma2(a[e], a[e], s2);
        z2 = ffma2(b[e], b[e], z2);
      }
      s2 = fadd2(s2, z2);
      float ss = s2.x + s2.y;
#pragma unroll
      for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(kFullMask, ss, o);
      const float inv = rsqrtf(fmaf(ss, inv_d, p.eps));
      const float2 i2 = make_float2(inv, inv);
      float2 wa[NV], wb[NV];
      by_pair(s_wa[what], wa);
      by_pair(s_wb[what], wb);
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        a[e] = fmul2(fmul2(a[e], i2), wa[e]);
        b[e] = fmul2(fmul2(b[e], i2), wb[e]);
      }
    }
    if (!on || pc.pair >= half) return;  // past the rotation pairs pass through
    float2 c[NV], s[NV], n[NV];
    by_pair(s_cos[tok], c);
    by_pair(s_sin[tok], s);
    by_pair(s_neg[tok], n);
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      const float2 x = a[e], y = b[e];
      const float2 u = ffma2(y, n[e], fmul2(x, c[e])), v = ffma2(x, s[e], fmul2(y, c[e]));
      // (an infinity times a zero sine would be no zero: pairs past the rotation
      // are chosen, not multiplied; in the aligned half layout a thread's are all
      // on one side)
      if (LAYOUT == kHalf || pc.pair + 2 * e < half) {
        a[e].x = u.x;
        b[e].x = v.x;
      }
      if (LAYOUT == kHalf || pc.pair + 2 * e + 1 < half) {
        a[e].y = u.y;
        b[e].y = v.y;
      }
    }
  };

  if constexpr (MODE != kNoCache) {
    const Quotient div(p.v_scale);
    run(rv, fv, vh, [&](const Frag& f, int tok, int head, bool on) {
      const int64_t at = on ? s_dst[tok] : -1;
      if (at < 0) return;  // padding, or a slot past the cache
      const int64_t dst = at + head * head_step;
      if constexpr (MODE == kCache16) {  // bit for bit
        store_pairs<LAYOUT, EPT>(static_cast<uint16_t*>(p.v_cache) + dst, pc, rot, D, f);
      } else {
        float2 a[NV], b[NV];
        unpack_pairs<T, LAYOUT, EPT>(f, a, b);
        store_codes<LAYOUT, EPT>(static_cast<uint8_t*>(p.v_cache) + dst, pc, rot, D, a, b, div);
      }
    });
  }
  const bool q_norm = p.q_weight != nullptr, k_norm = p.k_weight != nullptr;
  {
    const Quotient div(p.k_scale);
    run(rk, fk, kh, [&](const Frag& f, int tok, int head, bool on) {
      float2 a[NV], b[NV];
      turn(f, 1, k_norm, tok, on, a, b);
      if (!on) return;
      if constexpr (MODE == kNoCache) {
        store_pairs<LAYOUT, EPT>(static_cast<uint16_t*>(p.k_out) + (t0 + tok) * p.k_out_stride +
                                     static_cast<int64_t>(head) * D,
                                 pc, rot, D, pack_pairs<T, LAYOUT, EPT>(a, b));
      } else {
        const int64_t at = s_dst[tok];
        if (at < 0) return;
        const int64_t dst = at + head * head_step;
        if constexpr (MODE == kCache16)
          store_pairs<LAYOUT, EPT>(static_cast<uint16_t*>(p.k_cache) + dst, pc, rot, D,
                                   pack_pairs<T, LAYOUT, EPT>(a, b));
        else
          store_codes<LAYOUT, EPT>(static_cast<uint8_t*>(p.k_cache) + dst, pc, rot, D, a, b, div);
      }
    });
  }
  run(rq, fq, qh, [&](const Frag& f, int tok, int head, bool on) {
    float2 a[NV], b[NV];
    turn(f, 0, q_norm, tok, on, a, b);
    if (on)
      store_pairs<LAYOUT, EPT>(static_cast<uint16_t*>(p.q_out) + (t0 + tok) * p.q_out_stride +
                                   static_cast<int64_t>(head) * D,
                               pc, rot, D, pack_pairs<T, LAYOUT, EPT>(a, b));
  });
}

}  // namespace pa
