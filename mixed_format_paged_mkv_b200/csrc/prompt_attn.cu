// Causal attention over whole packed prompts (mkv_prompt_attention).
//
// For query token i and head h of a prompt (KV head h / g):
//   out[i][h] = sum_{j <= i} p_j V_j / sum_{j <= i} p_j,  p_j = 2^(c (q.k_j - m)),  c = scale log2 e
// with a reference m per row that follows the running maximum of q.k_j.  One pass over the keys:
// neither the scores nor the probabilities leave the SM.
//
// Rows.  A tile holds 128 query rows of one KV head: floor(128 / g) tokens times the g heads that
// share the KV head, token-major, so K and V are read once for all of them and only the keys up to
// the tile's last token are visited.  A CTA works on items of NT tiles (D 64 and 128: two tiles,
// whose softmax and tensor work alternate; D 256: one tile with two score buffers).
//
// Roles (one CTA per SM):
//   softmax warps  4 per tile, one row per thread: scores from tensor memory, probabilities back
//                  into it as bf16, running sum and reference in registers, output at the end
//   producer       one thread: tensor-map loads of Q and of K/V chunks into a ring
//   MMA            one thread: S = Q K^T and O += P V (P read from tensor memory)
//   guard (2 warps) on chunks that the causal line or the prompt's end crosses: zeroes V rows past
//                  the end and replaces non-finite V elements by zero, because 0 x inf would reach
//                  rows that do not see them; the rows that do see them get them back at the end
//
// Tensor memory (512 columns): score buffers in columns 0-255 (128 fp32 columns each; the bf16
// probabilities overwrite the scores they come from), outputs from column 256 on.
//
// Precision: products of bf16 with fp32 sums; the softmax's maximum, sum and output are fp32.  The
// probabilities are rounded to bf16 (relative 2^-9 each) because they are a tensor-core operand.
// The reference m moves only when a row's maximum exceeds it by more than 8 in log2 units, so
// p <= 2^8 and the sums stay far inside fp32; each move rescales the fp32 output.
#include <cuda_runtime.h>
#include <stdint.h>

#include "mkv_internal.h"
#include "tc_util.cuh"

namespace mkv {
namespace {

template <int D_>
struct Cfg {
  static constexpr int D = D_;
  static constexpr int NT = D == 256 ? 1 : 2;     // query tiles of an item
  static constexpr int SB = D == 256 ? 2 : 1;     // score buffers per tile
  static constexpr int CK = D == 256 ? 64 : 128;  // keys of a K or V chunk
  static constexpr int HALVES = 128 / CK;         // chunks of a 128-key tile
  static constexpr int BLK = D / 64;              // 64-channel blocks (128 bytes: the swizzle span)
  static constexpr int STAGES = D == 64 ? 8 : 5;
  static constexpr int Q_BLOCK = 128 * 128;
  static constexpr int Q_TILE = BLK * Q_BLOCK;
  static constexpr int KV_BLOCK = CK * 128;
  static constexpr int CHUNK = BLK * KV_BLOCK;
  static constexpr int SMEM_Q = NT * Q_TILE;
  static constexpr int SMEM = SMEM_Q + STAGES * CHUNK + 1024 /* alignment */ + 512 /* barriers */;
  static constexpr int SOFT_WARPS = 4 * NT;
  static constexpr int THREADS = 32 * (SOFT_WARPS + 4);
  static constexpr uint32_t IDESC_S = tc_idesc_bf16(128, CK, false);
  static constexpr uint32_t IDESC_PV = tc_idesc_bf16(128, D, true);
  static_assert(SMEM <= 232448, "shared memory of a CTA");
};

constexpr uint32_t kOutCol = 256;       // first output column in tensor memory
constexpr float kRescaleAbove = 8.0f;   // log2 units a row's maximum may exceed its reference by
constexpr int kFlagSlots = 8;           // items the guard may run ahead of the softmax warps

template <class C>
struct Bars {
  uint64_t q_full, q_empty;
  uint64_t kv_full[C::STAGES], kv_empty[C::STAGES], v_ready[C::STAGES];
  uint64_t s_full[C::NT * C::SB], p_full[C::NT * C::SB];
  uint64_t o_done[C::NT], o_free[C::NT];
  uint32_t tmem;
  int32_t abort;
  int32_t bad[kFlagSlots];  // item number whose V had a non-finite element on a guarded chunk
};

// One item: NT tiles of consecutive tokens of a prompt, for one KV head.
struct Item {
  int row0, len, t0, h;  // first packed row and length of the prompt, first token, KV head
};

__device__ __forceinline__ bool get_item(const PromptParams& p, int NT, int64_t index, Item& it) {
  if (index >= static_cast<int64_t>(p.n_units) * p.Hkv) return false;
  const int u = static_cast<int>(index / p.Hkv);
  it.h = static_cast<int>(index % p.Hkv);
  int lo = 0, hi = p.n_seqs - 1;  // the prompt whose units include u
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (u < p.seq[mid].unit_end) hi = mid;
    else lo = mid + 1;
  }
  it.row0 = p.seq[lo].row0;
  it.len = p.seq[lo].len;
  it.t0 = (p.seq[lo].unit_end - 1 - u) * NT * p.tile_tokens;  // last tokens (most keys) first
  return true;
}

// 128-key tiles that query tile t of an item visits (0: the tile has no tokens).
__device__ __forceinline__ int key_tiles(const Item& it, int t, int TT) {
  const int t0 = it.t0 + t * TT;
  return t0 < it.len ? (min(it.len, t0 + TT) + 127) >> 7 : 0;
}

// A chunk that starts at key c0 needs the guard: some row of the item does not see all its keys.
template <class C>
__device__ __forceinline__ bool guarded(const Item& it, int c0) {
  return c0 + C::CK > it.t0 + 1;
}

// Bounded wait that also ends when another warp gave up; false: leave the role's loops.
template <class B>
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, B* b, int32_t* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t start = global_timer_ns();
  for (;;) {
    if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
    if (*reinterpret_cast<volatile int32_t*>(&b->abort)) return false;
    if (global_timer_ns() - start > 2000000000ull) {
      *reinterpret_cast<volatile int32_t*>(&b->abort) = 1;
      flag_status(status, kStatusTimeout);
      return false;
    }
  }
}

// 8 bf16 values: whether one is infinite or NaN.
__device__ __forceinline__ bool nonfinite8(const uint4& v) {
  auto bad = [](uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
  };
  return bad(v.x) || bad(v.y) || bad(v.z) || bad(v.w);
}
__device__ __forceinline__ uint32_t zero_nonfinite(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
  return w;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    prompt_kernel(const __grid_constant__ PromptParams p, const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  constexpr int NT = C::NT, SB = C::SB, CK = C::CK, HALVES = C::HALVES, BLK = C::BLK, D = C::D;
  constexpr int ST = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sq = smem;
  uint8_t* skv = smem + C::SMEM_Q;
  Bars<C>* b = reinterpret_cast<Bars<C>*>(skv + ST * C::CHUNK);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int TT = p.tile_tokens;

  if (tid == 0) {
    mbar_init(&b->q_full, 1);
    mbar_init(&b->q_empty, 1);
    for (int i = 0; i < ST; ++i) {
      mbar_init(&b->kv_full[i], 1);
      mbar_init(&b->kv_empty[i], 3);  // the MMA commit and the two guard warps
      mbar_init(&b->v_ready[i], 64);
    }
    for (int i = 0; i < NT * SB; ++i) {
      mbar_init(&b->s_full[i], 1);
      mbar_init(&b->p_full[i], 128);
    }
    for (int i = 0; i < NT; ++i) {
      mbar_init(&b->o_done[i], 1);
      mbar_init(&b->o_free[i], 128);
    }
    b->abort = 0;
    for (int i = 0; i < kFlagSlots; ++i) b->bad[i] = -1;
    mbar_fence_init();
  }
  if (warp == C::SOFT_WARPS) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(&b->tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = b->tmem;
  const int64_t first = blockIdx.x, step = gridDim.x;

  if (warp == C::SOFT_WARPS) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      uint32_t ring = 0;  // chunks loaded so far
      int n_item = 0;
      bool go = true;
      Item it;
      for (int64_t idx = first; go && get_item(p, NT, idx, it); idx += step, ++n_item) {
        int n = 0, tiles = 0;
        for (int t = 0; t < NT; ++t) {
          const int nt = key_tiles(it, t, TT);
          n = max(n, nt);
          tiles += nt > 0;
        }
        if (n_item > 0 && !wait_bar(&b->q_empty, (n_item - 1) & 1, b, p.status)) break;
        mbar_arrive_expect_tx(&b->q_full, tiles * BLK * TT * p.g * 128);
        for (int t = 0; t < tiles; ++t)
          for (int k = 0; k < BLK; ++k)
            tma_load_4d(sq + t * C::Q_TILE + k * C::Q_BLOCK, &qmap, 64 * k, 0, it.h,
                        it.row0 + it.t0 + t * TT, &b->q_full);
        auto load = [&](const CUtensorMap* map, int key) {
          const int s = ring % ST;
          if (ring >= ST && !wait_bar(&b->kv_empty[s], (ring / ST - 1) & 1, b, p.status)) return false;
          mbar_arrive_expect_tx(&b->kv_full[s], C::CHUNK);
          for (int k = 0; k < BLK; ++k)
            tma_load_3d(skv + s * C::CHUNK + k * C::KV_BLOCK, map, 64 * k, it.h, it.row0 + key,
                        &b->kv_full[s]);
          ++ring;
          return true;
        };
        for (int j = -SB; go && j < n; ++j) {  // V of tile j, then K of tile j + SB
          for (int f = 0; go && f < HALVES && j >= 0; ++f) go = load(&vmap, 128 * j + CK * f);
          for (int f = 0; go && f < HALVES && j + SB < n; ++f) go = load(&kmap, 128 * (j + SB) + CK * f);
        }
      }
      // every copy has landed and every chunk was consumed before the CTA ends
      const uint64_t limit = *reinterpret_cast<volatile int32_t*>(&b->abort) ? 100000000ull : 2000000000ull;
      for (uint32_t r = ring > ST ? ring - ST : 0; r < ring; ++r) {
        mbar_wait(&b->kv_full[r % ST], (r / ST) & 1, limit);
        mbar_wait(&b->kv_empty[r % ST], (r / ST) & 1, limit);
      }
      if (n_item > 0) mbar_wait(&b->q_empty, (n_item - 1) & 1, limit);
    }
    __syncwarp();
  } else if (warp == C::SOFT_WARPS + 1) {
    // ---------------------------------------------------------------- MMA
    if (lane == 0) {
      uint32_t ring = 0, v_phase = 0;         // chunks consumed; phases of v_ready, a bit a stage
      uint32_t n_p[NT * SB] = {};             // probability tiles consumed per buffer
      uint32_t n_out[NT] = {};                // items that had tile t so far
      int n_item = 0;
      bool go = true;
      Item it;
      for (int64_t idx = first; go && get_item(p, NT, idx, it); idx += step, ++n_item) {
        int n[NT], nmax = 0;
        for (int t = 0; t < NT; ++t) nmax = max(nmax, n[t] = key_tiles(it, t, TT));
        auto wait_k = [&](uint32_t r) {
          return wait_bar(&b->kv_full[r % ST], (r / ST) & 1, b, p.status);
        };
        auto wait_v = [&](uint32_t r, int key) {
          const uint32_t s = r % ST;
          if (!guarded<C>(it, key)) return wait_k(r);
          const bool ok = wait_bar(&b->v_ready[s], (v_phase >> s) & 1, b, p.status);
          v_phase ^= 1u << s;
          return ok;
        };
        // S[t] (buffer sb) = Q[t] K^T for the CK keys of ring chunk r, columns CK * f on
        auto scores = [&](int t, int sb, int f, uint32_t r) {
          const uint32_t qa = smem_addr(sq + t * C::Q_TILE);
          const uint32_t ka = smem_addr(skv + (r % ST) * C::CHUNK);
          const uint32_t d = tmem + (t * SB + sb) * 128 + CK * f;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc_mma_ss(d, tc_smem_desc(qa + (k / 4) * C::Q_BLOCK + (k % 4) * 32, 16, 1024),
                      tc_smem_desc(ka + (k / 4) * C::KV_BLOCK + (k % 4) * 32, 16, 1024), C::IDESC_S, k > 0);
        };
        // O[t] (+)= P[t] V for the CK keys of ring chunk r
        auto values = [&](int t, int sb, int f, uint32_t r, bool acc) {
          const uint32_t va = smem_addr(skv + (r % ST) * C::CHUNK);
          const uint32_t pa = tmem + (t * SB + sb) * 128 + (CK / 2) * f;
#pragma unroll
          for (int k = 0; k < CK / 16; ++k)
            tc_mma_ts(tmem + kOutCol + t * D, pa + 8 * k, tc_smem_desc(va + 2048 * k, C::KV_BLOCK, 1024),
                      C::IDESC_PV, acc || k > 0);
        };
        go = wait_bar(&b->q_full, n_item & 1, b, p.status);
        for (int j = 0; go && j < SB && j < nmax; ++j) {  // the first score tiles
          for (int f = 0; go && f < HALVES; ++f) {
            if (!(go = wait_k(ring))) break;
            for (int t = 0; t < NT; ++t)
              if (j < n[t]) {
                scores(t, j, f, ring);
                if (f + 1 == HALVES) tc_commit(&b->s_full[t * SB + j]);
              }
            tc_commit(&b->kv_empty[ring % ST]);
            ++ring;
          }
        }
        if (go && nmax <= SB) tc_commit(&b->q_empty);
        for (int j = 0; go && j < nmax; ++j) {
          const int sb = j % SB;
          const uint32_t rv = ring, rk = ring + HALVES;  // chunks of V tile j and K tile j + SB
          const bool more = j + SB < nmax;
          bool have_v = false, have_k = false;
          for (int t = 0; go && t < NT; ++t) {
            if (j >= n[t]) continue;
            const int buf = t * SB + sb;
            if (j == 0 && n_out[t]++ > 0 && !(go = wait_bar(&b->o_free[t], n_out[t] & 1, b, p.status))) break;
            if (!(go = wait_bar(&b->p_full[buf], n_p[buf]++ & 1, b, p.status))) break;
            tc_fence_after();
            for (int f = 0; f < HALVES; ++f) {
              if (!have_v && !(go = wait_v(rv + f, 128 * j + CK * f))) break;
              tc_fence_after();
              values(t, sb, f, rv + f, j > 0 || f > 0);
            }
            if (!go) break;
            have_v = true;
            tc_commit(&b->o_done[t]);
            if (t == NT - 1 || j >= n[NT - 1])
              for (int f = 0; f < HALVES; ++f) tc_commit(&b->kv_empty[(rv + f) % ST]);
            if (j + SB < n[t]) {
              for (int f = 0; f < HALVES; ++f) {
                if (!have_k && !(go = wait_k(rk + f))) break;
                scores(t, sb, f, rk + f);
              }
              if (!go) break;
              have_k = true;
              tc_commit(&b->s_full[buf]);
            }
            if (more && (t == NT - 1 || j >= n[NT - 1]))
              for (int f = 0; f < HALVES; ++f) tc_commit(&b->kv_empty[(rk + f) % ST]);
          }
          if (go && j + SB + 1 == nmax) tc_commit(&b->q_empty);  // the item's last scores are issued
          ring += HALVES + (more ? HALVES : 0);
        }
      }
    }
    __syncwarp();
  } else if (warp >= C::SOFT_WARPS + 2) {
    // ---------------------------------------------------------------- guard
    // (follows every chunk, so that the parity it waits for is never more than a phase away)
    const int gtid = tid - 32 * (C::SOFT_WARPS + 2);
    uint32_t ring = 0;
    int n_item = 0;
    bool go = true;
    Item it;
    for (int64_t idx = first; go && get_item(p, NT, idx, it); idx += step, ++n_item) {
      int n = 0;
      for (int t = 0; t < NT; ++t) n = max(n, key_tiles(it, t, TT));
      // one chunk: K, or V with first key c0
      auto chunk = [&](bool value, int c0) {
        const int s = ring % ST;
        if (!__all_sync(0xffffffffu, wait_bar(&b->kv_full[s], (ring / ST) & 1, b, p.status))) return false;
        if (value && guarded<C>(it, c0)) {
          uint4* v = reinterpret_cast<uint4*>(skv + s * C::CHUNK);
          bool found = false;
          for (int i = gtid; i < C::CHUNK / 16; i += 64) {  // 16 bytes of one key's row
            const int key = c0 + (i / 8) % CK;
            if (key >= it.len) {
              v[i] = make_uint4(0, 0, 0, 0);
            } else {
              const uint4 x = v[i];
              if (nonfinite8(x)) {
                v[i] = make_uint4(zero_nonfinite(x.x), zero_nonfinite(x.y), zero_nonfinite(x.z), zero_nonfinite(x.w));
                found = true;
              }
            }
          }
          if (found) *reinterpret_cast<volatile int32_t*>(&b->bad[n_item % kFlagSlots]) = n_item;
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // these stores -> tensor core
          mbar_arrive(&b->v_ready[s]);
        }
        if (lane == 0) mbar_arrive(&b->kv_empty[s]);
        ++ring;
        return true;
      };
      for (int j = -SB; go && j < n; ++j) {
        for (int f = 0; go && f < HALVES && j >= 0; ++f) go = chunk(true, 128 * j + CK * f);
        for (int f = 0; go && f < HALVES && j + SB < n; ++f) go = chunk(false, 0);
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax and output
    const int t = warp / 4, r = tid & 127;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t o_addr = tmem + lane_base + kOutCol + t * D;
    const int tok = min(r / p.g, TT - 1), gi = r - (r / p.g) * p.g;
    const float c = p.c;
    const uint64_t c2 = f32x2(c, c);
    uint32_t n_s[SB] = {}, n_o = 0;  // score tiles per buffer, P V products of this tile so far
    int n_item = 0;
    bool go = true;
    Item it;
    for (int64_t idx = first; go && get_item(p, NT, idx, it); idx += step, ++n_item) {
      const int n = key_tiles(it, t, TT);
      const int pos = it.t0 + t * TT + tok;
      const bool mine = r < TT * p.g && pos < it.len;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        const int sb = SB == 1 ? 0 : j & 1;
        const int buf = t * SB + sb;
        if (!(go = __all_sync(0xffffffffu, wait_bar(&b->s_full[buf], n_s[sb]++ & 1, b, p.status)))) break;
        tc_fence_after();
        const uint32_t s_addr = tmem + lane_base + buf * 128;
        const int vis = pos + 1 - 128 * j;  // visible columns of this row (>= 128: all)
        const bool masked = __any_sync(0xffffffffu, vis < 128);
        uint32_t x[32], y[32];
        float mx = -INFINITY;
        tmem_ld32(x, s_addr);
        tmem_wait_ld(x);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t(&cur)[32] = k & 1 ? y : x;
          uint32_t(&nxt)[32] = k & 1 ? x : y;
          if (k < 3) tmem_ld32(nxt, s_addr + 32 * (k + 1));
          if (masked) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              mx = fmaxf(mx, 32 * k + i < vis ? __uint_as_float(cur[i]) : -INFINITY);
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              mx = fmaxf(mx, fmaxf(__uint_as_float(cur[i]), __uint_as_float(cur[i + 1])));
          }
          if (k < 3) tmem_wait_ld(nxt);
        }
        const bool up = (mx - m) * c > kRescaleAbove;
        if (j == 0) {
          m = mx;
        } else if (__any_sync(0xffffffffu, up)) {
          const float mn = up ? mx : m;
          const float a = up ? fast_exp2((m - mn) * c) : 1.f;
          m = mn;
          l *= a;
          if (!(go = __all_sync(0xffffffffu, wait_bar(&b->o_done[t], (n_o - 1) & 1, b, p.status)))) break;
          tc_fence_after();
#pragma unroll 1
          for (int k = 0; k < D / 32; ++k) {
            tmem_ld32(x, o_addr + 32 * k);
            tmem_wait_ld(x);
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * a);
            tmem_st32(o_addr + 32 * k, x);
          }
        }
        const float mc = m == -INFINITY ? 0.f : m * c;
        const uint64_t mc2 = f32x2(-mc, -mc);
        uint64_t l2 = 0;
        tmem_ld32(x, s_addr);
        tmem_wait_ld(x);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t(&cur)[32] = k & 1 ? y : x;
          uint32_t(&nxt)[32] = k & 1 ? x : y;
          if (k < 3) tmem_ld32(nxt, s_addr + 32 * (k + 1));
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint64_t z = fma2(f32x2(__uint_as_float(cur[2 * i]), __uint_as_float(cur[2 * i + 1])), c2, mc2);
            float p0 = fast_exp2(f32x2_lo(z)), p1 = fast_exp2(f32x2_hi(z));
            if (masked) {
              if (32 * k + 2 * i >= vis) p0 = 0.f;
              if (32 * k + 2 * i + 1 >= vis) p1 = 0.f;
            }
            l2 = add2(l2, f32x2(p0, p1));
            pk[i] = pack_bf16x2(p0, p1);
          }
          if (k < 3) tmem_wait_ld(nxt);
          tmem_st16(s_addr + 16 * k, pk);  // columns whose scores were read already
        }
        l += f32x2_lo(l2) + f32x2_hi(l2);
        // With two score buffers this tile may be done before the last tile's product; the next
        // scores follow that product, so waiting for it here costs nothing and keeps the parity
        // that the waits on o_done use no more than a phase away.
        if (SB > 1 && j > 0 &&
            !(go = __all_sync(0xffffffffu, wait_bar(&b->o_done[t], (n_o - 1) & 1, b, p.status))))
          break;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&b->p_full[buf]);
        ++n_o;
      }
      if (!go) break;
      if (n == 0) continue;  // (o_free[t] counts the items that have this tile)
      // ---- output
      if (!(go = __all_sync(0xffffffffu, wait_bar(&b->o_done[t], (n_o - 1) & 1, b, p.status)))) break;
      tc_fence_after();
      const float inv = 1.f / l;
      const bool bad = *reinterpret_cast<volatile int32_t*>(&b->bad[n_item % kFlagSlots]) == n_item;
      uint16_t* out = p.out + (static_cast<int64_t>(it.row0 + pos) * p.Hq + it.h * p.g + gi) * D;
#pragma unroll 1
      for (int k = 0; k < D / 32; ++k) {
        uint32_t x[32];
        tmem_ld32(x, o_addr + 32 * k);
        tmem_wait_ld(x);
        if (mine && bad) {  // non-finite V elements that this row sees, on the chunks the guard cleaned
          const int e0 = (it.t0 + 1) / CK * CK;
#pragma unroll 1
          for (int key = e0; key <= pos; ++key) {
            const uint16_t* v = p.v + static_cast<int64_t>(it.row0 + key) * p.v_stride + it.h * D + 32 * k;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if ((v[i] & 0x7f80u) == 0x7f80u)
                x[i] = __float_as_uint(__uint_as_float(x[i]) + bf16_bits_to_float(v[i]));
          }
        }
        if (mine) {
          uint4* o4 = reinterpret_cast<uint4*>(out + 32 * k);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_bf16x2(__uint_as_float(x[8 * i + 2 * e]) * inv, __uint_as_float(x[8 * i + 2 * e + 1]) * inv);
            o4[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      mbar_arrive(&b->o_free[t]);
    }
  }
  __syncthreads();
  if (*reinterpret_cast<volatile int32_t*>(&b->abort)) {
    // a wait gave up: give MMAs in flight a bounded time to end before their memory is released
    const uint64_t start = global_timer_ns();
    while (global_timer_ns() - start < 1000000ull) {
    }
    __syncthreads();
  }
  if (warp == C::SOFT_WARPS) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                 CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                 CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

// bf16 tensor map with 128-byte swizzle and zero fill: dims and box innermost first.
bool make_map(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
              const cuuint32_t* box) {
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  const EncodeTiled fn = encode_tiled();
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch(const PromptParams& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                   cudaStream_t s) {
  using C = Cfg<D>;
  auto* fn = &prompt_kernel<C>;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  fn<<<static_cast<unsigned>(p.n_units * p.Hkv), C::THREADS, C::SMEM, s>>>(p, q, k, v);
  return cudaGetLastError();
}

}  // namespace

int prompt_tiles_per_unit(int D) { return D == 256 ? Cfg<256>::NT : Cfg<128>::NT; }

cudaError_t launch_prompt(const PromptParams& p, const PromptInputs& in, cudaStream_t s) {
  if (p.n_units <= 0) return cudaSuccess;
  const cuuint64_t D = p.D, g = p.g, Hkv = p.Hkv, rows = in.rows;
  CUtensorMap q, k, v;
  const cuuint64_t qd[4] = {D, g, Hkv, rows}, qs[3] = {2 * D, 2 * g * D, 2ull * in.q_stride};
  const cuuint32_t qb[4] = {64, static_cast<cuuint32_t>(p.g), 1, static_cast<cuuint32_t>(p.tile_tokens)};
  const cuuint64_t kd[3] = {D, Hkv, rows}, ks[2] = {2 * D, 2ull * in.k_stride}, vs[2] = {2 * D, 2ull * in.v_stride};
  const cuuint32_t kb[3] = {64, 1, static_cast<cuuint32_t>(p.D == 256 ? Cfg<256>::CK : Cfg<128>::CK)};
  if (!make_map(&q, in.q, 4, qd, qs, qb) || !make_map(&k, in.k, 3, kd, ks, kb) || !make_map(&v, in.v, 3, kd, vs, kb))
    return cudaErrorInvalidValue;
  return p.D == 64 ? launch<64>(p, q, k, v, s) : p.D == 128 ? launch<128>(p, q, k, v, s) : launch<256>(p, q, k, v, s);
}

}  // namespace mkv
