// Rotary positions with several axes (mkv_rope).
//
// Frequency i < R/2 of a head rotates the channel pair (a, b) = (x[i], x[i + R/2]) or, with
// neighbouring pairs, (x[2i], x[2i + 1]) by the angle pos[axis(i)][row] * inv_freq[i]:
//   a' = a cos - b sin,  b' = b cos + a sin;  channels from R on are passed through.
//
// The angle is formed in fp64, as turns: position times frequency, times 1 / (2 pi), three roundings in
// all (two products and the constant), so it is off by at most 3 2^-53 of itself: 7e-7 rad at position
// 2^31 and frequency 1, where one fp32 rounding of the angle would be off by up to 64 rad.  It is reduced to a
// fraction of a turn and only then rounded to fp32 for the sine and cosine.  The rotation itself is
// fp32, rounded once to bf16.
//
// Bound by memory: q and k are read and written once.  A CTA takes a few rows: its threads first
// load their vectors, then compute the rows' sines and cosines into shared memory (each angle once
// for all heads) while the loads are in flight, then rotate and store.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "device_util.cuh"
#include "mkv_internal.h"

namespace mkv {
namespace {

constexpr int kThreads = 256;
constexpr int kSms = 148;

__device__ __forceinline__ void sincos_turns(int32_t pos, float inv_freq, float* s, float* c) {
  constexpr double kInvTwoPi = 0.15915494309189533577;
  const double turns = static_cast<double>(pos) * static_cast<double>(inv_freq) * kInvTwoPi;
  sincospif(2.0f * static_cast<float>(turns - rint(turns)), s, c);
}

// The sines and cosines of `rows` rows from row0 on, [row][frequency].
__device__ __forceinline__ void fill_table(const RopeParams& p, int64_t row0, int rows, float* sn, float* cs) {
  for (int i = threadIdx.x; i < rows * p.half; i += kThreads) {
    const int f = i % p.half;
    const int32_t pos = p.positions[p.axis[f] * p.rows + row0 + i / p.half];
    sincos_turns(pos, p.inv_freq[f], &sn[i], &cs[i]);
  }
}

__device__ __forceinline__ void rotate(uint32_t& a, uint32_t& b, const float* s, const float* c) {
  const float a0 = bf16_lo(a), a1 = bf16_hi(a), b0 = bf16_lo(b), b1 = bf16_hi(b);
  a = pack_bf16x2(fmaf(a0, c[0], -b0 * s[0]), fmaf(a1, c[1], -b1 * s[1]));
  b = pack_bf16x2(fmaf(b0, c[0], a0 * s[0]), fmaf(b1, c[1], a1 * s[1]));
}
// A word that holds a whole pair.
__device__ __forceinline__ void rotate_word(uint32_t& w, float s, float c) {
  const float a = bf16_lo(w), b = bf16_hi(w);
  w = pack_bf16x2(fmaf(a, c, -b * s), fmaf(b, c, a * s));
}

// 16-byte vectors.  A unit is 16 channels: the vectors of 8 pairs (x[8u..], x[R/2 + 8u..]), two
// neighbouring vectors with neighbouring pairs, or two neighbouring vectors that pass through.  A CTA
// takes as many rows as give each thread kUnits units, all of which it loads at once (128 bytes).
constexpr int kUnits = 4;

template <int D, bool NEXT>
__global__ void __launch_bounds__(kThreads) rope_vec_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kPer = D / 16;  // units of a head
  extern __shared__ __align__(16) float table[];
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.cta_rows;
  const int rows = static_cast<int>(min(static_cast<int64_t>(p.cta_rows), p.rows - row0));
  float* sn = table;
  float* cs = table + p.cta_rows * p.half;
  const int heads = p.Hq + p.Hkv, rot = p.half / 8;  // (rot units of a head are rotated)
  const int units = rows * heads * kPer;
  bool have_table = false;
  for (int u0 = threadIdx.x; u0 < units || !have_table; u0 += kUnits * kThreads) {
    uint4 a[kUnits], b[kUnits];
    uint4* to[kUnits];
    int at[kUnits];  // first table entry of the unit's pairs, -1: passes through
#pragma unroll
    for (int e = 0; e < kUnits; ++e) {
      const int u = u0 + e * kThreads;
      if (u >= units) continue;
      const int c = u % kPer, i = u / kPer;
      const int r = static_cast<int>(__umulhi(i, p.heads_magic)), h = i - r * heads;
      const bool is_q = h < p.Hq;
      const uint16_t* in = is_q ? p.q_in + (row0 + r) * p.q_in_stride + h * D
                                : p.k_in + (row0 + r) * p.k_in_stride + (h - p.Hq) * D;
      uint16_t* out = is_q ? p.q_out + (row0 + r) * p.q_out_stride + h * D
                           : p.k_out + (row0 + r) * p.k_out_stride + (h - p.Hq) * D;
      const bool pair = NEXT || c >= rot;  // the unit's two vectors are neighbours
      const int first = pair ? 2 * c : c, second = pair ? 2 * c + 1 : c + rot;
      a[e] = reinterpret_cast<const uint4*>(in)[first];
      b[e] = reinterpret_cast<const uint4*>(in)[second];
      to[e] = reinterpret_cast<uint4*>(out) + first;
      at[e] = c < rot ? r * p.half + 8 * c : -1;
    }
    if (!have_table) {  // (computed while the vectors are on their way)
      fill_table(p, row0, rows, sn, cs);
      __syncthreads();
      have_table = true;
    }
#pragma unroll
    for (int e = 0; e < kUnits; ++e) {
      if (u0 + e * kThreads >= units) continue;
      if (at[e] >= 0) {
        float s[8], k[8];
        const float4* s4 = reinterpret_cast<const float4*>(sn + at[e]);
        const float4* c4 = reinterpret_cast<const float4*>(cs + at[e]);
        *reinterpret_cast<float4*>(s) = s4[0];
        *reinterpret_cast<float4*>(s + 4) = s4[1];
        *reinterpret_cast<float4*>(k) = c4[0];
        *reinterpret_cast<float4*>(k + 4) = c4[1];
        if (NEXT) {
          rotate_word(a[e].x, s[0], k[0]);
          rotate_word(a[e].y, s[1], k[1]);
          rotate_word(a[e].z, s[2], k[2]);
          rotate_word(a[e].w, s[3], k[3]);
          rotate_word(b[e].x, s[4], k[4]);
          rotate_word(b[e].y, s[5], k[5]);
          rotate_word(b[e].z, s[6], k[6]);
          rotate_word(b[e].w, s[7], k[7]);
        } else {
          rotate(a[e].x, b[e].x, s, k);
          rotate(a[e].y, b[e].y, s + 2, k + 2);
          rotate(a[e].z, b[e].z, s + 4, k + 4);
          rotate(a[e].w, b[e].w, s + 6, k + 6);
        }
      }
      to[e][0] = a[e];
      to[e][NEXT || at[e] < 0 ? 1 : rot] = b[e];
    }
  }
}

// Any even R, alignment and stride: one pair (or two channels that pass through) at a time.
__global__ void __launch_bounds__(kThreads) rope_any_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ __align__(16) float table[];
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.cta_rows;
  const int rows = static_cast<int>(min(static_cast<int64_t>(p.cta_rows), p.rows - row0));
  float* sn = table;
  float* cs = table + p.cta_rows * p.half;
  fill_table(p, row0, rows, sn, cs);
  __syncthreads();
  const int heads = p.Hq + p.Hkv, per = p.D / 2;
  for (int u = threadIdx.x; u < rows * heads * per; u += kThreads) {
    const int c = u % per, h = u / per % heads, lr = u / per / heads;
    const int64_t r = row0 + lr;
    const bool is_q = h < p.Hq;
    const int hh = is_q ? h : h - p.Hq;
    const uint16_t* in = (is_q ? p.q_in + r * p.q_in_stride : p.k_in + r * p.k_in_stride) + hh * p.D;
    uint16_t* out = (is_q ? p.q_out + r * p.q_out_stride : p.k_out + r * p.k_out_stride) + hh * p.D;
    const int i0 = c >= p.half || p.next ? 2 * c : c, i1 = c >= p.half || p.next ? 2 * c + 1 : c + p.half;
    uint32_t w = in[i0] | static_cast<uint32_t>(in[i1]) << 16;
    if (c < p.half) rotate_word(w, sn[lr * p.half + c], cs[lr * p.half + c]);
    out[i0] = static_cast<uint16_t>(w);
    out[i1] = static_cast<uint16_t>(w >> 16);
  }
}

}  // namespace

cudaError_t launch_rope(RopeParams& p, cudaStream_t s) {
  if (p.rows <= 0) return cudaSuccess;
  const int64_t heads = p.Hq + p.Hkv, per_row = heads * (p.vec ? p.D / 16 : p.D / 2);
  // Rows of a CTA: kUnits units a thread, but no fewer CTAs than two for each of the 148 SMs where there
  // are as many rows: the few rows of a decode step wait for one CTA's chain of loads, angles and stores.
  // Device time in us without that limit, with one, two and four CTAs per SM: 64 rows of 32/8 heads, D 128:
  // 2.9, 2.3, 2.3, 2.3; 900 rows of 16/4, D 64: 3.4, 2.9, 2.7, 4.6; 600 rows of 32/8, D 128: 4.0, 4.0, 3.8,
  // 4.8; 444 rows of 24/4, D 256: 4.0, 4.0, 3.5, 3.4; from 4000 rows on within 2% of one another.
  int64_t r = std::max<int64_t>(1, kUnits * kThreads / per_row);
  r = std::min<int64_t>({r, 64, std::max<int64_t>(1, p.rows / (2 * kSms))});
  p.cta_rows = static_cast<int32_t>(r);
  // i / heads for the units of a CTA (i < 2^32 / heads; at least two heads, one of q and one of k)
  p.heads_magic = static_cast<uint32_t>((1ull << 32) / heads + 1);
  const unsigned grid = static_cast<unsigned>((p.rows + r - 1) / r);
  const size_t smem = sizeof(float) * 2 * r * p.half;
#define MKV_ROPE(D)                                                   \
  (p.next ? rope_vec_kernel<D, true><<<grid, kThreads, smem, s>>>(p)  \
          : rope_vec_kernel<D, false><<<grid, kThreads, smem, s>>>(p))
  if (!p.vec) rope_any_kernel<<<grid, kThreads, smem, s>>>(p);
  else if (p.D == 64) MKV_ROPE(64);
  else if (p.D == 128) MKV_ROPE(128);
  else MKV_ROPE(256);
#undef MKV_ROPE
  return cudaGetLastError();
}

}  // namespace mkv
