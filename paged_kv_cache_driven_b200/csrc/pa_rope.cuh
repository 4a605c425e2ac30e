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
// work is a dozen instructions. One CTA takes the rows (or a run of them) of one
// token, so the D / 2 sines and cosines are computed once per CTA and kept in
// registers over its rows: a thread owns four pairs of a row, D / 8 threads a
// row, 256 / LPR rows at a time. Pairs, not consecutive elements, are what a
// thread owns: in the half layout it loads two 8-byte pieces rot_dim / 2
// apart, which keeps both components of a pair in one thread (no exchange
// between lanes); warps still read whole 128-byte lines.
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

// One CTA per (token, run of chunk_rows rows). Rows of a token: H of q, Hkv of
// k, and with a cache Hkv of v. LPR: threads per row, a power of two >= D / 8.
template <typename T, int LAYOUT, int MODE, int LPR>
__global__ void __launch_bounds__(256) rope_kernel(const RopeParams p) {
  constexpr int RPP = 256 / LPR;  // rows the CTA takes at a time
  constexpr int U = 4;            // rows a thread has in flight
  __shared__ float2 cs[128];
  const int t = blockIdx.x / p.chunks;
  const int row0 = (blockIdx.x - t * p.chunks) * p.chunk_rows;
  const int row1 = min(row0 + p.chunk_rows, p.rows);
  const int sub = threadIdx.x / LPR, pl = threadIdx.x % LPR;
  const bool lane_on = pl * 8 < p.D;
  const int D = p.D, rot = p.rot;

  int64_t slot = 0;
  if constexpr (MODE != kNoCache) {
    slot = __ldg(p.slots + t);
    if (slot >= p.n_slots) {
      if (threadIdx.x == 0 && row0 == 0) raise_error(PA_DEVERR_SLOT);
      slot = -1;
    }
  }
  const int64_t blk = slot < 0 ? 0 : slot / p.S;
  const int64_t off = slot < 0 ? 0 : slot - blk * p.S;
  const uint16_t* q = static_cast<const uint16_t*>(p.q) + t * p.q_stride;
  const uint16_t* k = static_cast<const uint16_t*>(p.k) + t * p.k_stride;
  const uint16_t* v = static_cast<const uint16_t*>(p.v) + t * p.v_stride;
  // kind of a row: 0 q, 1 k, 2 v; -1: nothing to do (past the end, or skipped)
  auto kind_of = [&](int row) {
    if (row >= row1 || !lane_on) return -1;
    if (row < p.H) return 0;
    if (MODE != kNoCache && slot < 0) return -1;
    return row < p.H + p.Hkv ? 1 : 2;
  };

  float c[4], s[4];
  float wa[2][4], wb[2][4];  // norm weights of this thread's pairs, q and k
#pragma unroll 1
  for (int base = row0; base < row1; base += U * RPP) {
    PairFrag f[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = base + u * RPP + sub;
      const int kind = kind_of(row);
      f[u].w[0] = f[u].w[1] = f[u].w[2] = f[u].w[3] = 0;
      if (kind < 0) continue;
      const uint16_t* src = kind == 0   ? q + row * D
                            : kind == 1 ? k + (row - p.H) * D
                                        : v + (row - p.H - p.Hkv) * D;
      f[u] = load_pairs<LAYOUT>(src, pl, rot, D);
    }
    if (base == row0) {  // the token's sines and cosines, under the first loads
      if (threadIdx.x < rot >> 1) {
        const double turns = __ldg(p.table + threadIdx.x);
        const double pos = static_cast<double>(__ldg(p.positions + t));
        const double r = fma(pos, turns, -rint(pos * turns));  // [-1/2, 1/2]
        float sv, cv;
        sincospif(2.f * static_cast<float>(r), &sv, &cv);
        cs[threadIdx.x] = make_float2(cv * p.amplitude, sv * p.amplitude);
      }
      if (lane_on) {
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const void* wt = part == 0 ? p.q_weight : p.k_weight;
          if (!wt) continue;
          const PairFrag wf = load_pairs<LAYOUT>(static_cast<const uint16_t*>(wt), pl, rot, D);
          unpack_pairs<T, LAYOUT>(wf, wa[part], wb[part]);
        }
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = 4 * pl + e;
        const float2 v2 = j < rot >> 1 ? cs[j] : make_float2(1.f, 0.f);
        c[e] = v2.x;
        s[e] = v2.y;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = base + u * RPP + sub;
      const int kind = kind_of(row);
      float a[4], b[4];
      unpack_pairs<T, LAYOUT>(f[u], a, b);
      // the norm's sum over the row's threads (every lane takes the shuffles)
      if (p.q_weight || p.k_weight) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
#pragma unroll
        for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(kFullMask, ss, o);
        const bool norm = kind == 0 ? p.q_weight != nullptr : kind == 1 && p.k_weight != nullptr;
        if (norm) {
          const float inv = 1.f / sqrtf(ss / static_cast<float>(D) + p.eps);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[e] *= inv * (kind == 0 ? wa[0][e] : wa[1][e]);
            b[e] *= inv * (kind == 0 ? wb[0][e] : wb[1][e]);
          }
        }
      }
      if (kind < 0) continue;
      if (kind == 2) {  // values pass as they are
        if constexpr (MODE != kNoCache) {
          const int64_t dst = ((blk * p.Hkv + (row - p.H - p.Hkv)) * p.S + off) * D;
          if constexpr (MODE == kCache16)
            store_pairs<LAYOUT>(static_cast<uint16_t*>(p.v_cache) + dst, pl, rot, D, f[u]);
          else
            store_codes<LAYOUT>(static_cast<uint8_t*>(p.v_cache) + dst, pl, rot, D, a, b,
                                p.v_scale);
        }
        continue;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (4 * pl + e < rot >> 1) {  // others pass through (an infinity times 0 is no 0)
          const float x = a[e], y = b[e];
          a[e] = x * c[e] - y * s[e];
          b[e] = y * c[e] + x * s[e];
        }
      }
      if (kind == 0 || MODE == kNoCache) {
        uint16_t* dst = kind == 0
                            ? static_cast<uint16_t*>(p.q_out) + t * p.q_out_stride + row * D
                            : static_cast<uint16_t*>(p.k_out) + t * p.k_out_stride +
                                  (row - p.H) * D;
        store_pairs<LAYOUT>(dst, pl, rot, D, pack_pairs<T, LAYOUT>(a, b));
      } else {
        const int64_t dst = ((blk * p.Hkv + (row - p.H)) * p.S + off) * D;
        if constexpr (MODE == kCache16)
          store_pairs<LAYOUT>(static_cast<uint16_t*>(p.k_cache) + dst, pl, rot, D,
                              pack_pairs<T, LAYOUT>(a, b));
        else if constexpr (MODE == kCache8)
          store_codes<LAYOUT>(static_cast<uint8_t*>(p.k_cache) + dst, pl, rot, D, a, b,
                              p.k_scale);
      }
    }
  }
}

}  // namespace pa
