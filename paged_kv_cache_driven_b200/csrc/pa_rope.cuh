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
// A stream bound by HBM: each value is read once and written once, and a value's
// work is a dozen instructions. One CTA takes up to 8 tokens (kRopeTokens) with
// all their rows, or, of few tokens, a run of one token's rows. Their sines and
// cosines are computed once, into shared memory, under the first rows' loads. A
// thread owns four pairs of a row, LPR threads a row, 256 / LPR rows at a time,
// and loads U rows ahead of the U rows that it works on. Pairs, not
// consecutive elements, are what a thread owns: in the half layout it loads two
// 8-byte pieces rot_dim / 2 apart, which keeps both components of a pair in
// one thread (no exchange between lanes); warps still read whole lines.
#pragma once

#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {

// How a row's elements are paired and moved.
enum : int {
  kPairs = 0,     // interleaved: elements 2j, 2j + 1; a thread's 8 are consecutive (16 bytes)
  kHalf = 1,      // elements j, j + rot / 2, rot a multiple of 8: two 8-byte pieces
  kHalfAny = 2    // the same for any even rot: single elements
};
enum : int { kNoCache = 0, kCache16 = 1, kCache8 = 2 };

constexpr int kRopeTokens = 8;  // most tokens of a CTA

// A thread's 8 elements of a row, as they lie in memory: 4 pairs.
struct PairFrag {
  uint32_t w[4];
};

// The first elements a, b of a thread's pieces (kHalf; pair 4 * pl): rotated
// pairs lie rot / 2 apart, the others (which pass through) (D - rot) / 2 apart.
__device__ __forceinline__ void half_pieces(int j, int rot, int D, int& a, int& b) {
  const int r2 = rot >> 1;
  if (j < r2) {
    a = j;
    b = j + r2;
  } else {
    a = rot + (j - r2);
    b = a + ((D - rot) >> 1);
  }
}

// Loads 4 pairs into fragment words: kPairs word e = pair e; kHalf words 0, 1 =
// components a of pairs 0..3, words 2, 3 = components b.
template <int LAYOUT>
__device__ __forceinline__ PairFrag load_pairs(const uint16_t* row, int pl, int rot, int D) {
  PairFrag f;
  if constexpr (LAYOUT == kPairs) {
    const uint4 x = __ldcs(reinterpret_cast<const uint4*>(row) + pl);
    f.w[0] = x.x, f.w[1] = x.y, f.w[2] = x.z, f.w[3] = x.w;
  } else if constexpr (LAYOUT == kHalf) {
    int a, b;
    half_pieces(4 * pl, rot, D, a, b);
    const uint2 x = __ldcs(reinterpret_cast<const uint2*>(row + a));
    const uint2 y = __ldcs(reinterpret_cast<const uint2*>(row + b));
    f.w[0] = x.x, f.w[1] = x.y, f.w[2] = y.x, f.w[3] = y.y;
  } else {
    uint16_t u[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      int a, b;
      half_pieces(4 * pl + e, rot, D, a, b);
      u[e] = __ldcs(reinterpret_cast<const unsigned short*>(row + a));
      u[4 + e] = __ldcs(reinterpret_cast<const unsigned short*>(row + b));
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      f.w[e] = static_cast<uint32_t>(u[2 * e]) | (static_cast<uint32_t>(u[2 * e + 1]) << 16);
  }
  return f;
}

template <int LAYOUT>
__device__ __forceinline__ void store_pairs(uint16_t* row, int pl, int rot, int D,
                                            const PairFrag& f) {
  if constexpr (LAYOUT == kPairs) {
    reinterpret_cast<uint4*>(row)[pl] = make_uint4(f.w[0], f.w[1], f.w[2], f.w[3]);
  } else if constexpr (LAYOUT == kHalf) {
    int a, b;
    half_pieces(4 * pl, rot, D, a, b);
    *reinterpret_cast<uint2*>(row + a) = make_uint2(f.w[0], f.w[1]);
    *reinterpret_cast<uint2*>(row + b) = make_uint2(f.w[2], f.w[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      int a, b;
      half_pieces(4 * pl + e, rot, D, a, b);
      row[a] = static_cast<uint16_t>(f.w[e >> 1] >> (16 * (e & 1)));
      row[b] = static_cast<uint16_t>(f.w[2 + (e >> 1)] >> (16 * (e & 1)));
    }
  }
}

// Components (a, b) of the 4 pairs in fp32, and back (one rounding).
template <typename T, int LAYOUT>
__device__ __forceinline__ void unpack_pairs(const PairFrag& f, float (&a)[4], float (&b)[4]) {
  if constexpr (LAYOUT == kPairs) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 v = Elem<T>::pair(f.w[e]);
      a[e] = v.x;
      b[e] = v.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float2 u = Elem<T>::pair(f.w[e]), v = Elem<T>::pair(f.w[2 + e]);
      a[2 * e] = u.x, a[2 * e + 1] = u.y;
      b[2 * e] = v.x, b[2 * e + 1] = v.y;
    }
  }
}

template <typename T>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  const T a = to_out<T>(lo), b = to_out<T>(hi);
  return static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(&a)) |
         (static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(&b)) << 16);
}

template <typename T, int LAYOUT>
__device__ __forceinline__ PairFrag pack_pairs(const float (&a)[4], const float (&b)[4]) {
  PairFrag f;
  if constexpr (LAYOUT == kPairs) {
#pragma unroll
    for (int e = 0; e < 4; ++e) f.w[e] = pack16<T>(a[e], b[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      f.w[e] = pack16<T>(a[2 * e], a[2 * e + 1]);
      f.w[2 + e] = pack16<T>(b[2 * e], b[2 * e + 1]);
    }
  }
  return f;
}

// The 4 pairs as E4M3 codes of fp32(value / scale) (one correctly rounded
// division, round to nearest even, saturated), stored to a row of codes.
template <int LAYOUT>
__device__ __forceinline__ void store_codes(uint8_t* row, int pl, int rot, int D,
                                            const float (&a)[4], const float (&b)[4],
                                            float scale) {
  if constexpr (LAYOUT == kPairs) {
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c[e] = float2_to_e4m3x2(__fdiv_rn(a[e], scale), __fdiv_rn(b[e], scale));
    reinterpret_cast<uint2*>(row)[pl] = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
  } else {
    uint32_t c[4];  // a01, a23, b01, b23
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      c[e] = float2_to_e4m3x2(__fdiv_rn(a[2 * e], scale), __fdiv_rn(a[2 * e + 1], scale));
      c[2 + e] = float2_to_e4m3x2(__fdiv_rn(b[2 * e], scale), __fdiv_rn(b[2 * e + 1], scale));
    }
    if constexpr (LAYOUT == kHalf) {
      int ia, ib;
      half_pieces(4 * pl, rot, D, ia, ib);
      *reinterpret_cast<uint32_t*>(row + ia) = c[0] | (c[1] << 16);
      *reinterpret_cast<uint32_t*>(row + ib) = c[2] | (c[3] << 16);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        int ia, ib;
        half_pieces(4 * pl + e, rot, D, ia, ib);
        row[ia] = static_cast<uint8_t>(c[e >> 1] >> (8 * (e & 1)));
        row[ib] = static_cast<uint8_t>(c[2 + (e >> 1)] >> (8 * (e & 1)));
      }
    }
  }
}

// The rows of a token: H of q, Hkv of k, and with a cache Hkv of v. LPR:
// threads per row, a power of two >= D / 8. A CTA's work is the rows row0 ..
// row1 - 1 of `toks` tokens from token t0, numbered token after token; thread
// group `sub` takes numbers sub, sub + RPP, ...
template <typename T, int LAYOUT, int MODE, int LPR>
__global__ void __launch_bounds__(256, 4) rope_kernel(const RopeParams p) {
  constexpr int RPP = 256 / LPR;  // rows the CTA takes at a time
  constexpr int U = 2;            // passes a thread has in flight
  constexpr int NP = LPR * 4;     // pairs of a row, rounded up
  __shared__ __align__(16) float s_cos[kRopeTokens][NP], s_sin[kRopeTokens][NP];
  __shared__ __align__(16) float s_wa[2][NP], s_wb[2][NP];  // norm weights by pair, q and k
  __shared__ int64_t s_dst[kRopeTokens];      // cache element of (head 0, this token), or -1
  const int D = p.D, rot = p.rot, half = p.rot >> 1;
  const int grp = blockIdx.x / p.chunks;
  const int row0 = (blockIdx.x - grp * p.chunks) * p.chunk_rows;
  const int nrow = min(p.chunk_rows, p.rows - row0);
  const int t0 = grp * p.toks;
  const int ntok = min(p.toks, p.T - t0);
  const int total = ntok * nrow;
  const int sub = threadIdx.x / LPR, pl = threadIdx.x % LPR;
  const bool lane_on = pl * 8 < D;
  const uint16_t* q = static_cast<const uint16_t*>(p.q);
  const uint16_t* k = static_cast<const uint16_t*>(p.k);
  const uint16_t* v = static_cast<const uint16_t*>(p.v);

  // number -> token of the CTA and row (one token: no division)
  auto split = [&](int n, int& tok, int& row) {
    tok = p.toks > 1 ? static_cast<int>((static_cast<uint64_t>(n) * p.row_magic) >> 32) : 0;
    row = row0 + n - tok * nrow;
  };
  auto load = [&](int n, PairFrag& f) {
    if (n >= total || !lane_on) return;
    int tok, row;
    split(n, tok, row);
    const int64_t t = t0 + tok;
    const uint16_t* src = q + t * p.q_stride + static_cast<int64_t>(row) * D;
    if (row >= p.H) src = k + t * p.k_stride + static_cast<int64_t>(row - p.H) * D;
    if (MODE != kNoCache && row >= p.H + p.Hkv)
      src = v + t * p.v_stride + static_cast<int64_t>(row - p.H - p.Hkv) * D;
    f = load_pairs<LAYOUT>(src, pl, rot, D);
  };

  PairFrag cur[U] = {};
#pragma unroll
  for (int u = 0; u < U; ++u) load(u * RPP + sub, cur[u]);

  // the tokens' sines and cosines, their places in the cache, the norm weights
  for (int x = threadIdx.x; x < ntok * half; x += 256) {
    const int tok = x / half, j = x - tok * half;
    const double turns = __ldg(p.table + j);
    const double pos = static_cast<double>(__ldg(p.positions + t0 + tok));
    const double r = fma(pos, turns, -rint(pos * turns));  // [-1/2, 1/2]
    float sv, cv;
    sincospif(2.f * static_cast<float>(r), &sv, &cv);
    s_cos[tok][j] = cv * p.amplitude;
    s_sin[tok][j] = sv * p.amplitude;
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
  const bool q_norm = p.q_weight != nullptr, k_norm = p.k_weight != nullptr;
  if (threadIdx.x < LPR && lane_on) {
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const void* wt = part == 0 ? p.q_weight : p.k_weight;
      if (!wt) continue;
      float a[4], b[4];
      unpack_pairs<T, LAYOUT>(load_pairs<LAYOUT>(static_cast<const uint16_t*>(wt), pl, rot, D), a,
                              b);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s_wa[part][4 * pl + e] = a[e];
        s_wb[part][4 * pl + e] = b[e];
      }
    }
  }
  __syncthreads();
  const float inv_d = 1.f / static_cast<float>(D);
  const int64_t head_step = static_cast<int64_t>(p.S) * D;

#pragma unroll 1
  for (int base = sub; base - sub < total; base += U * RPP) {
    PairFrag nxt[U] = {};
#pragma unroll
    for (int u = 0; u < U; ++u) load(base + (U + u) * RPP, nxt[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int n = base + u * RPP;
      if (n - sub >= total) break;  // (the whole CTA's)
      int tok, row;
      split(n, tok, row);
      const bool on = n < total && lane_on;
      const bool is_q = row < p.H;
      const bool is_v = MODE != kNoCache && row >= p.H + p.Hkv;
      float a[4], b[4];
      unpack_pairs<T, LAYOUT>(cur[u], a, b);
      if (q_norm || k_norm) {  // the sum over the row's threads: every lane takes the shuffles
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
#pragma unroll
        for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(kFullMask, ss, o);
        if (is_q ? q_norm : (k_norm && !is_v)) {
          const float inv = rsqrtf(fmaf(ss, inv_d, p.eps));
          const float4 wa = *reinterpret_cast<const float4*>(&s_wa[is_q ? 0 : 1][4 * pl]);
          const float4 wb = *reinterpret_cast<const float4*>(&s_wb[is_q ? 0 : 1][4 * pl]);
          a[0] *= inv * wa.x, a[1] *= inv * wa.y, a[2] *= inv * wa.z, a[3] *= inv * wa.w;
          b[0] *= inv * wb.x, b[1] *= inv * wb.y, b[2] *= inv * wb.z, b[3] *= inv * wb.w;
        }
      }
      if (!on) continue;
      if (!is_v && 4 * pl < half) {
        const float4 c4 = *reinterpret_cast<const float4*>(&s_cos[tok][4 * pl]);
        const float4 s4 = *reinterpret_cast<const float4*>(&s_sin[tok][4 * pl]);
        const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // past the rotation pairs pass through (an infinity times a zero sine is no zero);
          // in the vector half layout a thread's pairs are all on one side
          if (LAYOUT == kHalf || 4 * pl + e < half) {
            const float x = a[e], y = b[e];
            a[e] = x * c[e] - y * s[e];
            b[e] = y * c[e] + x * s[e];
          }
        }
      }
      if (MODE == kNoCache || is_q) {
        const int64_t t = t0 + tok;
        uint16_t* dst = static_cast<uint16_t*>(p.q_out) + t * p.q_out_stride +
                        static_cast<int64_t>(row) * D;
        if (!is_q)
          dst = static_cast<uint16_t*>(p.k_out) + t * p.k_out_stride +
                static_cast<int64_t>(row - p.H) * D;
        store_pairs<LAYOUT>(dst, pl, rot, D, pack_pairs<T, LAYOUT>(a, b));
      } else if constexpr (MODE != kNoCache) {
        const int64_t at = s_dst[tok];
        if (at < 0) continue;  // padding, or a slot past the cache
        const int64_t dst = at + (row - p.H - (is_v ? p.Hkv : 0)) * head_step;
        void* cache = is_v ? p.v_cache : p.k_cache;
        if constexpr (MODE == kCache16)  // values pass bit for bit
          store_pairs<LAYOUT>(static_cast<uint16_t*>(cache) + dst, pl, rot, D,
                              is_v ? cur[u] : pack_pairs<T, LAYOUT>(a, b));
        else
          store_codes<LAYOUT>(static_cast<uint8_t*>(cache) + dst, pl, rot, D, a, b,
                              is_v ? p.v_scale : p.k_scale);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) cur[u] = nxt[u];
  }
}

}  // namespace pa
