// Causal attention over whole packed prompts (mkv_prompt_attention).
//
// For query token i and head h of a prompt (KV head h / g):
//   out[i][h] = sum_{j <= i} p_j V_j / sum_{j <= i} p_j,  p_j = 2^(c (q.k_j - m)),  c = scale log2 e
// with a reference m per row that follows the running maximum of q.k_j.  One pass over the keys:
// neither the scores nor the probabilities leave the SM.
//
// Rows.  A tile holds 128 query rows of one KV head: floor(128 / g) tokens times the g heads that
// share the KV head, token-major, so K and V are read once for all of them and only the keys up to
// the tile's last token are visited.  An item is NT tiles of consecutive tokens (D 64 and 128: two,
// which share K and V; D 256: one, whose output takes half of tensor memory).  A CTA (one per SM)
// works on items until none is left; it gets the next one by cluster launch control.  Items go out
// prompt by prompt, the longest first, and within a prompt those with most keys first.  A CTA claims an
// item when it starts the one before, so that the loads of the next are never waited for; the claim
// therefore does not know how long the present item takes, which shows where an SM gets few items: one
// prompt of 2048 tokens, 32/8 heads, D 128 (1.7 items per SM) takes 50 us where free SMs taking the
// items would need 37.
//
// Roles:
//   softmax warps  4 per tile, one row per thread: scores from tensor memory, probabilities back
//                  into it as bf16, running sum and reference in registers, output at the end
//   producer       tensor-map loads of Q and of K/V chunks into a ring
//   MMA            a warp per tile, one lane of which issues S = Q K^T and O += P V (P is read from
//                  tensor memory)
//   guard          on V chunks that the causal line or the prompt's end crosses: zeroes V rows past
//                  the end and replaces non-finite V elements by zero, because 0 x inf would reach
//                  rows that do not see them; the rows that do see them get them back at the end,
//                  added as they are: a weight that underflowed gives an infinity here, and NaN in
//                  a chunk that went to the tensor core as it was (0 x inf), so the contract says no
//                  more than that such a channel is non-finite
//
// Tensor memory (512 columns): NT x SB score buffers of KT fp32 columns, whose first half the bf16
// probabilities overwrite, then NT outputs of D columns.
//
// Precision: products of bf16 with fp32 sums; the softmax's maximum, sum and output are fp32.  The
// probabilities are rounded to bf16 (relative 2^-8 each) because they are a tensor-core operand.
// The reference m moves only when a row's maximum exceeds it by more than 8 in log2 units, so
// p <= 2^8 and the sums stay far inside fp32; each move rescales the fp32 output.
//
// Measured (one B200, one prompt of 8192 tokens, causal FLOPs; from a cool card to one at its power
// limit): 32/8 heads, D 128: 440-460 us, 1250-1200 TFLOP/s; 24/4 heads, D 256: 655-772 us, 1260-1070
// TFLOP/s; 16/16 heads, D 64: 199 us, 690 TFLOP/s.  Device time at D 128, 32/8 heads over prompts of 64 to
// 4096 tokens: 3.6 us + 0.9 us a step + 4.1 us an item (of each SM's share), and the claim's imbalance.
//   D 128: scores of 64 keys take 48 cycles per MMA instead of 32, since each reads 6 KB of operands
//          from shared memory; with the products and the softmax's share of tensor memory the tensor
//          path needs about 1600 of the 1740 cycles of a step.  Steps of 128 keys read less but leave
//          room for one score buffer only, and then each tile's softmax and MMAs take turns: 493 us.
//   D 256: one tile's chain: MMAs for 2050 of the 3250 cycles of a step, then what one step's scores,
//          probabilities and products wait for one another; K and V come from L2 once per 128 rows
//          (128 KB a step, 10 TB/s over all SMs, of 11.6 that loads alone reach), which adds 300.
//   D 64:  the exponentials (16 a cycle and SM) are 1024 of the 1500 cycles of a step; two score
//          buffers instead of three: 204 us.  Part of the exponentials as a polynomial on the FMA
//          pipe: 218 us, the issue slots it takes cost more than the ex2 it saves.
//   All:   one MMA warp for both tiles instead of one each: 614 us for 483 (D 128, at that step); the
//          reference moved with every new maximum: 565 us for 438; (s - m) c in two operations instead
//          of s c - m c in one: 490 us, so scores whose scaled size passes 2^30 (where the rounding of
//          m c alone passes 2^6) may make their row NaN; the next step's scores loaded while this one's
//          exponentials run: 626 us for 454 (the probabilities reach the tensor core later).
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "mkv_internal.h"
#include "tc_util.cuh"

namespace mkv {
namespace {

template <int D_>
struct Cfg {
  static constexpr int D = D_;
  static constexpr int NT = D == 256 ? 1 : 2;     // query tiles of an item
  static constexpr int SB = D == 64 ? 3 : 2;      // score buffers per tile
  static constexpr int KT = D == 256 ? 128 : 64;  // keys of a step (of a score buffer)
  static constexpr uint32_t OUT = NT * SB * KT;   // first output column in tensor memory
  static_assert(OUT + NT * D <= 512, "tensor memory");
  static constexpr int PH = KT / 64;              // the probabilities of a step are handed on by 64 keys
  static constexpr int BLK = D / 64;              // 64-channel blocks (128 bytes: the swizzle span)
  // ring chunks: K of a step in KC chunks of all its keys and KB blocks each, V in VC chunks of VK
  // keys and all channels
  static constexpr int KC = D == 256 ? 2 : 1, KB = BLK / KC;
  static constexpr int VC = D == 256 ? 2 : 1, VK = KT / VC;
  static constexpr int K_BLOCK = KT * 128, V_BLOCK = VK * 128;
  static constexpr int CHUNK = KB * K_BLOCK;
  static_assert(CHUNK == BLK * V_BLOCK, "K and V chunks share the ring");
  static constexpr int STAGES = D == 64 ? 16 : D == 128 ? 10 : 5;
  static constexpr int Q_BLOCK = 128 * 128;
  static constexpr int Q_TILE = BLK * Q_BLOCK;
  static constexpr int SMEM_Q = NT * Q_TILE;
  static constexpr int SMEM = SMEM_Q + STAGES * CHUNK + 1024 /* alignment */ + 1024 /* barriers */;
  // warps: softmax (4 a tile), producer, guard, MMA (1 a tile)
  static constexpr int PRODUCER = 4 * NT, GUARD = PRODUCER + 1, MMA = GUARD + 1;
  static constexpr int WARPS = MMA + NT, THREADS = 32 * WARPS;
  static constexpr uint32_t IDESC_S = tc_idesc_bf16(128, KT, false);
  static constexpr uint32_t IDESC_PV = tc_idesc_bf16(128, D, true);
  static_assert(SMEM <= 232448, "shared memory of a CTA");
};

// Descriptors without their start address: K-major rows, and V's rows that run along the channels.
constexpr uint64_t kDescK = tc_smem_desc(0, 16, 1024);
template <class C>
constexpr uint64_t kDescV = tc_smem_desc(0, C::V_BLOCK, 1024);
constexpr float kRescaleAbove = 8.0f;   // log2 units a row's maximum may exceed its reference by
constexpr int kFlagSlots = 8;           // items the guard may run ahead of the softmax warps

// Position in the ring of chunks: the stage, and how often the ring went round.
template <int STAGES>
struct Ring {
  uint32_t stage = 0, round = 0;
  __device__ __forceinline__ void step() {
    if (++stage == STAGES) {
      stage = 0;
      ++round;
    }
  }
  __device__ __forceinline__ Ring plus(int n) const {
    Ring r = *this;
    for (int i = 0; i < n; ++i) r.step();
    return r;
  }
};

template <class C>
struct Bars {
  uint64_t q_full, q_empty;
  uint64_t kv_full[C::STAGES], kv_empty[C::STAGES], v_guard[C::STAGES], v_ready[C::STAGES];
  uint64_t s_full[C::NT * C::SB], p_full[C::NT * C::SB][C::PH], o_done[C::NT * C::SB];
  uint64_t o_free[C::NT];
  uint64_t next_full[2], next_empty[2];
  uint4 next[2];            // answers that name the next items
  uint32_t tmem;
  int32_t abort;
  int32_t bad[kFlagSlots];  // item number whose V had a non-finite element on a guarded chunk
};

// One item: NT tiles of consecutive tokens of a prompt, for one KV head.
struct Item {
  int row0, len, t0, h;  // first packed row and length of the prompt, first token, KV head
};

__device__ __forceinline__ Item get_item(const PromptParams& p, int NT, int64_t index) {
  Item it;
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
  return it;
}

// Steps of KT keys that query tile t of an item visits (0: the tile has no tokens).
template <class C>
__device__ __forceinline__ int key_steps(const Item& it, int t, int TT) {
  const int t0 = it.t0 + t * TT;
  return t0 < it.len ? (min(it.len, t0 + TT) + C::KT - 1) / C::KT : 0;
}

// A V chunk that starts at key c0 needs the guard: some row of the item does not see all its keys.
template <class C>
__device__ __forceinline__ bool guarded(const Item& it, int c0) {
  return c0 + C::VK > it.t0 + 1;
}

// Bounded wait of one thread that also ends when another warp gave up; false: leave the role's
// loops.  An attempt suspends the thread for up to 50 us, so that waiting warps leave the issue slots
// and the shared-memory pipe to the others.  Reading the timer takes longer than most waits, so the
// first attempts do without.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, int32_t* abort, int32_t* status) {
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait_sleep(bar, parity, 50000u)) return true;
  const uint64_t start = global_timer_ns();
  for (;;) {
    if (mbar_try_wait_sleep(bar, parity, 50000u)) return true;
    if (*reinterpret_cast<volatile int32_t*>(abort)) return false;
    if (global_timer_ns() - start > 2000000000ull) {
      *reinterpret_cast<volatile int32_t*>(abort) = 1;
      flag_status(status, kStatusTimeout);
      return false;
    }
  }
}
template <class B>
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, B* b, int32_t* status) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, &b->abort, status);
}
// The same for a whole warp: where the first attempt fails, one lane waits and the others follow it.
template <class B>
__device__ __forceinline__ bool wait_bar_warp(uint64_t* bar, uint32_t parity, B* b, int32_t* status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = wait_slow(bar, parity, &b->abort, status);
  return __shfl_sync(0xffffffffu, static_cast<int>(ok), 0) != 0;
}
// For the warp that feeds the tensor core: it spins for a while, since waking up costs more.
template <class B>
__device__ __forceinline__ bool wait_spin(uint64_t* bar, uint32_t parity, B* b, int32_t* status) {
#pragma unroll 1
  for (int i = 0; i < 1000; ++i)
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return wait_bar_warp(bar, parity, b, status);
}

// Index of the CTA's n-th item, -1: none (or a wait gave up).  Called by a whole warp or by one
// thread of it; either counts once on next_empty.
template <bool ONE, class B>
__device__ __forceinline__ int64_t next_item(int n, B* b, int32_t* status) {
  if (n == 0) return blockIdx.x;
  const int s = (n - 1) & 1;
  uint64_t* bar = &b->next_full[s];
  const uint32_t parity = ((n - 1) >> 1) & 1;
  if (!(ONE ? wait_bar(bar, parity, b, status) : wait_bar_warp(bar, parity, b, status))) return -1;
  const int64_t index = clc_answer(&b->next[s]);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // this read, then the next answer
  if (!ONE) __syncwarp();
  if (ONE || (threadIdx.x & 31) == 0) mbar_arrive(&b->next_empty[s]);
  return index;
}

// Two bf16 values: bits 15 and 31 say which are infinite or NaN (the sum carries into them from an
// exponent of ones only); the other bits mean nothing.
__device__ __forceinline__ uint32_t nonfinite_bits(uint32_t w) { return (w & 0x7f807f80u) + 0x00800080u; }
__device__ __forceinline__ uint32_t zero_nonfinite(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
  return w;
}

// 32 bytes to global memory, at once where the address allows: a row's lanes write to different rows,
// and whole sectors halve the requests.
__device__ __forceinline__ void store32(uint16_t* to, const uint32_t (&w)[8], int aligned32) {
  if (aligned32) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    prompt_kernel(const __grid_constant__ PromptParams p, const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  constexpr int NT = C::NT, SB = C::SB, KT = C::KT, KC = C::KC, VC = C::VC, VK = C::VK, BLK = C::BLK, D = C::D;
  constexpr int ST = C::STAGES, PH = C::PH;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sq = smem;
  uint8_t* skv = smem + C::SMEM_Q;
  Bars<C>* b = reinterpret_cast<Bars<C>*>(skv + ST * C::CHUNK);
  static_assert(sizeof(Bars<C>) <= 1024, "barriers");
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (known to be the same for the whole warp)
  const int TT = p.tile_tokens;

  if (warp == C::GUARD && lane < 3) tensor_map_prefetch(lane == 0 ? &qmap : lane == 1 ? &kmap : &vmap);
  if (tid == 0) {
    mbar_init(&b->q_full, 1);
    mbar_init(&b->q_empty, NT);
    for (int i = 0; i < ST; ++i) {
      mbar_init(&b->kv_full[i], 1);
      mbar_init(&b->kv_empty[i], NT);
      mbar_init(&b->v_guard[i], 1);
      mbar_init(&b->v_ready[i], 1);
    }
    for (int i = 0; i < NT * SB; ++i) {
      mbar_init(&b->s_full[i], 1);
      for (int h = 0; h < C::PH; ++h) mbar_init(&b->p_full[i][h], 4);
      mbar_init(&b->o_done[i], 1);
    }
    for (int i = 0; i < NT; ++i) mbar_init(&b->o_free[i], 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b->next_full[i], 1);
      mbar_init(&b->next_empty[i], C::WARPS);
    }
    b->abort = 0;
    for (int i = 0; i < kFlagSlots; ++i) b->bad[i] = -1;
    mbar_fence_init();
  }
  if (warp == C::PRODUCER) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(&b->tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // (all 512 columns of tensor memory are this CTA's: they start at column 0)

  if (warp == C::PRODUCER) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      Ring<ST> ring;  // the next chunk to load
      int n_item = 0, asked = 0;
      bool go = true;
      // the item after next is asked for when every role has taken the one before it
      auto ask = [&] {
        const int s = asked & 1;
        if (asked >= 2 && !wait_bar(&b->next_empty[s], ((asked >> 1) - 1) & 1, b, p.status)) return false;
        mbar_arrive_expect_tx(&b->next_full[s], 16);
        clc_request(&b->next[s], &b->next_full[s]);
        ++asked;
        return true;
      };
      // the stage of the ring's next chunk, once it is free
      auto stage = [&] {
        go = go && (ring.round == 0 || wait_bar(&b->kv_empty[ring.stage], (ring.round - 1) & 1, b, p.status));
        if (go) mbar_arrive_expect_tx(&b->kv_full[ring.stage], C::CHUNK);
        return ring.stage;
      };
      ask();
      while (go) {
        const int64_t idx = next_item<true>(n_item, b, p.status);
        if (idx < 0) break;
        if (n_item > 0 && !ask()) break;
        const Item it = get_item(p, NT, idx);
        int n = 0, tiles = 0;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int nt = key_steps<C>(it, t, TT);
          n = max(n, nt);
          tiles += nt > 0;
        }
        if (n_item > 0 && !wait_bar(&b->q_empty, (n_item - 1) & 1, b, p.status)) break;
        ++n_item;
        mbar_arrive_expect_tx(&b->q_full, tiles * BLK * TT * p.g * 128);
        for (int t = 0; t < tiles; ++t)
          for (int k = 0; k < BLK; ++k)
            tma_load_4d(sq + t * C::Q_TILE + k * C::Q_BLOCK, &qmap, 64 * k, 0, it.h, it.row0 + it.t0 + t * TT,
                        &b->q_full);
        for (int j = -SB; go && j < n; ++j) {  // V of step j, then K of step j + SB
          for (int f = 0; go && f < VC && j >= 0; ++f) {
            const int s = stage(), key = KT * j + VK * f;
            if (!go) break;
            for (int k = 0; k < BLK; ++k)
              tma_load_3d(skv + s * C::CHUNK + k * C::V_BLOCK, &vmap, 64 * k, it.h, it.row0 + key, &b->kv_full[s]);
            if (guarded<C>(it, key)) mbar_arrive(&b->v_guard[s]);
            ring.step();
          }
          for (int f = 0; go && f < KC && j + SB < n; ++f) {
            const int s = stage();
            if (!go) break;
            for (int k = 0; k < C::KB; ++k)
              tma_load_3d(skv + s * C::CHUNK + k * C::K_BLOCK, &kmap, 64 * (C::KB * f + k), it.h,
                          it.row0 + KT * (j + SB), &b->kv_full[s]);
            ring.step();
          }
        }
      }
      // every copy and answer has landed and every chunk was consumed before the CTA ends
      const uint64_t limit = *reinterpret_cast<volatile int32_t*>(&b->abort) ? 100000000ull : 2000000000ull;
      for (uint32_t s = 0; s < ST; ++s) {  // each stage's last round
        const uint32_t rounds = ring.round + (s < ring.stage ? 1 : 0);
        if (rounds == 0) continue;
        mbar_wait(&b->kv_full[s], (rounds - 1) & 1, limit);
        mbar_wait(&b->kv_empty[s], (rounds - 1) & 1, limit);
      }
      if (n_item > 0) mbar_wait(&b->q_empty, (n_item - 1) & 1, limit);
      mbar_wait(&b->next_full[(asked - 1) & 1], ((asked - 1) >> 1) & 1, limit);
    }
    __syncwarp();
  } else if (warp >= C::MMA) {
    // ---------------------------------------------------------------- MMA, one warp per tile
    // Per step: O (+)= P V of step j, then S = Q K^T of step j + SB.  The tensor core's queue holds a
    // few MMAs only, so what a warp spends on looking at barriers between them would be lost; with a
    // warp per tile it passes while the other tile's MMAs run.  (A warp runs as a whole and one lane
    // issues: control flow and operands are then known to be uniform, as the MMAs' operands have to
    // be.  It walks over every chunk of the item, also those that only the other tile needs.)
    const int t = warp - C::MMA;
    Ring<ST> ring;                          // the next chunk
    uint32_t v_phase = 0;                   // phases of v_ready, a bit a stage
    uint32_t p_phase = 0;                   // phases of p_full, a bit a buffer of the tile
    uint32_t n_out = 0;                     // items that had this tile so far
    const uint32_t lead = elect_lane() ? 1u : 0u;
    // start addresses of the operands' descriptors, in units of 16 bytes
    const uint32_t q16 = (smem_addr(sq) + t * C::Q_TILE) >> 4, kv16 = smem_addr(skv) >> 4;
    const uint32_t o = C::OUT + t * D;
    bool go = true;
    for (int n_item = 0; go; ++n_item) {
      const int64_t idx = next_item<false>(n_item, b, p.status);
      if (idx < 0) break;
      const Item it = get_item(p, NT, idx);
      const int n = key_steps<C>(it, t, TT);
      const int nmax = NT == 1 ? n : max(n, key_steps<C>(it, 1 - t, TT));
      if (!(go = wait_spin(&b->q_full, n_item & 1, b, p.status))) break;
#pragma unroll 1
      for (int j = -SB, sb = 0; go && j < nmax; ++j, sb = sb + 1 == SB ? 0 : sb + 1) {
        const int buf = t * SB + sb;
        const bool do_v = j >= 0, do_k = j + SB < nmax;
        const bool pv = do_v && j < n, qk = do_k && j + SB < n;
        const Ring<ST> rv = ring, rk = do_v ? ring.plus(VC) : ring;  // V chunks of step j, K of j + SB
        const uint32_t p_par = (p_phase >> sb) & 1;
        // barriers of the chunks: V through the guard where the causal line or the prompt's end cross
        uint64_t *v_bar[VC], *k_bar[KC];
        uint32_t v_par[VC], k_par[KC];
#pragma unroll
        for (int f = 0; f < VC; ++f) {
          const Ring<ST> r = rv.plus(f);
          const bool guard = do_v && guarded<C>(it, KT * j + VK * f);
          v_bar[f] = guard ? &b->v_ready[r.stage] : &b->kv_full[r.stage];
          v_par[f] = guard ? (v_phase >> r.stage) & 1 : r.round & 1;
          if (guard) v_phase ^= 1u << r.stage;
        }
#pragma unroll
        for (int f = 0; f < KC; ++f) {
          const Ring<ST> r = rk.plus(f);
          k_bar[f] = &b->kv_full[r.stage];
          k_par[f] = r.round & 1;
        }
        // One look at all barriers of a step together costs a third of looking at one after the other
        // (about 130 cycles each); only what is not there yet is waited for below.
        bool ready = false;
        if (pv && qk) {
          bool all = true;
#pragma unroll
          for (int h = 0; h < PH; ++h) all &= mbar_try_wait(&b->p_full[buf][h], p_par);
#pragma unroll
          for (int f = 0; f < VC; ++f) all &= mbar_try_wait(v_bar[f], v_par[f]);
#pragma unroll
          for (int f = 0; f < KC; ++f) all &= mbar_try_wait(k_bar[f], k_par[f]);
          ready = __all_sync(0xffffffffu, all);
        }
        if (pv) {
          // (the last item's output has been read before the first product overwrites it)
          if (j == 0 && n_out++ > 0 && !(go = wait_spin(&b->o_free[t], n_out & 1, b, p.status))) break;
#pragma unroll
          for (int h = 0; h < PH; ++h) {  // 64 keys at a time, as the probabilities come
            constexpr int kPerChunk = C::VK / 64;
            const Ring<ST> r = rv.plus(h / kPerChunk);
            if (!ready) {
              if (h % kPerChunk == 0) go = go && wait_spin(v_bar[h / kPerChunk], v_par[h / kPerChunk], b, p.status);
              go = go && wait_spin(&b->p_full[buf][h], p_par, b, p.status);
              if (!go) break;
            }
            tc_fence_after();
            const uint32_t vd = kv16 + r.stage * (C::CHUNK / 16) + (h % kPerChunk) * (64 * 128 / 16);
            const uint32_t pa = buf * KT + 32 * h;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc_mma_ts(lead, o, pa + 8 * k, vd + (2048 / 16) * k, kDescV<C>, C::IDESC_PV, h > 0 || k > 0 || j > 0);
            if ((h + 1) % kPerChunk == 0) tc_commit(lead, &b->kv_empty[r.stage]);
          }
          if (!go) break;
          tc_commit(lead, &b->o_done[buf]);
          p_phase ^= 1u << sb;
        } else if (do_v) {  // chunks that only the other tile uses
#pragma unroll
          for (int f = 0; f < VC; ++f) {
            if (!(go = go && wait_spin(v_bar[f], v_par[f], b, p.status))) break;
            if (lead) mbar_arrive(&b->kv_empty[rv.plus(f).stage]);
          }
        }
        if (qk) {
#pragma unroll
          for (int f = 0; f < KC; ++f) {
            const Ring<ST> r = rk.plus(f);
            if (!ready && !(go = wait_spin(k_bar[f], k_par[f], b, p.status))) break;
            tc_fence_after();
            const uint32_t qd = q16 + f * C::KB * C::Q_BLOCK / 16;
            const uint32_t kd = kv16 + r.stage * (C::CHUNK / 16);
#pragma unroll
            for (int k = 0; k < 4 * C::KB; ++k)
              tc_mma_ss(lead, buf * KT, qd + ((k / 4) * C::Q_BLOCK + (k % 4) * 32) / 16,
                        kd + ((k / 4) * C::K_BLOCK + (k % 4) * 32) / 16, kDescK, C::IDESC_S, f > 0 || k > 0);
            if (f + 1 == KC) tc_commit(lead, &b->s_full[buf]);
            tc_commit(lead, &b->kv_empty[r.stage]);
          }
          if (j + SB + 1 == n) tc_commit(lead, &b->q_empty);  // this tile's last scores are issued
        } else if (do_k) {
#pragma unroll
          for (int f = 0; f < KC; ++f) {
            if (!(go = go && wait_spin(k_bar[f], k_par[f], b, p.status))) break;
            if (lead) mbar_arrive(&b->kv_empty[rk.plus(f).stage]);
          }
        }
        ring = do_k ? rk.plus(KC) : rk;
      }
      if (go && n == 0 && lead) mbar_arrive(&b->q_empty);
    }
    __syncwarp();
  } else if (warp == C::GUARD) {
    // ---------------------------------------------------------------- guard
    // (The producer tells it of a chunk's load, per stage, so that the parities it waits for are
    // never more than a phase away.)
    Ring<ST> ring;
    uint32_t g_phase = 0;  // phases of v_guard, a bit a stage
    bool go = true;
    for (int n_item = 0; go; ++n_item) {
      const int64_t idx = next_item<false>(n_item, b, p.status);
      if (idx < 0) break;
      const Item it = get_item(p, NT, idx);
      int n = 0;
#pragma unroll
      for (int t = 0; t < NT; ++t) n = max(n, key_steps<C>(it, t, TT));
      auto scan = [&](int c0) {  // the chunk at the ring's position, with first key c0
        const int s = ring.stage;
        if (!wait_bar_warp(&b->v_guard[s], (g_phase >> s) & 1, b, p.status)) return false;
        g_phase ^= 1u << s;
        if (!wait_bar_warp(&b->kv_full[s], ring.round & 1, b, p.status)) return false;
        // (Half of what a guarded chunk costs is on the way to the prompt's output, so the scan is three
        // instructions a word: with a test per value it took 5000 to 23000 cycles an item.)
        uint4* v = reinterpret_cast<uint4*>(skv + s * C::CHUNK);
        uint32_t found = 0;
#pragma unroll 8
        for (int i = lane; i < C::CHUNK / 16; i += 32) {
          const uint4 x = v[i];
          found |= nonfinite_bits(x.x) | nonfinite_bits(x.y) | nonfinite_bits(x.z) | nonfinite_bits(x.w);
        }
        const bool past = c0 + VK > it.len;
        const bool dirty = __any_sync(0xffffffffu, found & 0x80008000u);
        if (past || dirty) {
#pragma unroll 1
          for (int i = lane; i < C::CHUNK / 16; i += 32) {  // 16 bytes of one key's row
            const int key = c0 + (i / 8) % VK;
            const uint4 x = v[i];
            v[i] = key >= it.len ? make_uint4(0, 0, 0, 0)
                                 : make_uint4(zero_nonfinite(x.x), zero_nonfinite(x.y), zero_nonfinite(x.z), zero_nonfinite(x.w));
          }
        }
        if (dirty && lane == 0) *reinterpret_cast<volatile int32_t*>(&b->bad[n_item % kFlagSlots]) = n_item;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // these stores -> tensor core
        __syncwarp();
        if (lane == 0) mbar_arrive(&b->v_ready[s]);
        return true;
      };
#pragma unroll 1
      for (int j = -SB; go && j < n; ++j) {
        for (int f = 0; go && f < VC && j >= 0; ++f, ring.step())
          if (guarded<C>(it, KT * j + VK * f)) go = scan(KT * j + VK * f);
        for (int f = 0; f < KC && j + SB < n; ++f) ring.step();
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax and output
    const int t = warp / 4, r = tid & 127;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t o_addr = lane_base + C::OUT + t * D;
    const int tok = min(r / p.g, TT - 1), gi = r - (r / p.g) * p.g;
    const float c = p.c;
    const uint64_t c2 = f32x2(c, c);
    uint32_t phase = 0;   // phases of this tile's score buffers, a bit a buffer
    bool go = true;
    for (int n_item = 0; go; ++n_item) {
      const int64_t idx = next_item<false>(n_item, b, p.status);
      if (idx < 0) break;
      const Item it = get_item(p, NT, idx);
      const int n = key_steps<C>(it, t, TT);
      if (n == 0) continue;
      const int pos = it.t0 + t * TT + tok;
      const bool mine = r < TT * p.g && pos < it.len;
      float m = -INFINITY;
      uint64_t l2 = 0;
      // Waits for the last product of buffer sb.  (A step's scores follow the product of SB steps
      // before, so by the step after the one meant that buffer's barrier is at most a phase away.)
      auto wait_product = [&](int sb) {
        const bool ok = wait_bar_warp(&b->o_done[t * SB + sb], (~phase >> sb) & 1, b, p.status);
        tc_fence_after();
        return ok;
      };
      int last = 0;  // the last step's buffer
      for (int j = 0, sb = 0; j < n; ++j, last = sb, sb = sb + 1 == SB ? 0 : sb + 1) {
        const int buf = t * SB + sb;
        if (!(go = wait_bar_warp(&b->s_full[buf], (phase >> sb) & 1, b, p.status))) break;
        tc_fence_after();
        const uint32_t s_addr = lane_base + buf * KT;
        uint32_t x[KT / 32][32];
#pragma unroll
        for (int k = 0; k < KT / 32; ++k) tmem_ld32(x[k], s_addr + 32 * k);
#pragma unroll
        for (int k = 0; k < KT / 32; ++k) tmem_wait_ld(x[k]);
        const int vis = pos + 1 - KT * j;  // visible columns of this row (>= KT: all)
        if (__any_sync(0xffffffffu, vis < KT)) {
#pragma unroll
          for (int i = 0; i < KT; ++i)
            if (i >= vis) x[i / 32][i % 32] = 0xff800000u;  // -inf
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < KT / 2; ++i)
          mx[i % 4] = max3(mx[i % 4], __uint_as_float(x[i / 16][2 * (i % 16)]),
                               __uint_as_float(x[i / 16][2 * (i % 16) + 1]));
        // (NaN is no maximum here; a visible score that is NaN or +inf makes its exponent, and with it
        // the row's sum and output, NaN, as in the formula)
        const float top = max3(max3(mx[0], mx[1], mx[2]), mx[3], mx[3]);
        const bool up = (top - m) * c > kRescaleAbove;
        if (j == 0) {
          m = top;
        } else if (__any_sync(0xffffffffu, up)) {
          const float mn = up ? top : m;
          // (from the references as they are subtracted from scores, with their rounding)
          const float a = up ? fast_exp2(__fsub_rn(__fmul_rn(m, c), __fmul_rn(mn, c))) : 1.f;
          m = mn;
          l2 = mul2(l2, f32x2(a, a));
          if (!(go = wait_product(last))) break;
#pragma unroll 1
          for (int k = 0; k < D / 16; ++k) {
            uint32_t o[16];
            tmem_ld16(o, o_addr + 16 * k);
            tmem_wait_ld(o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
            tmem_st16(o_addr + 16 * k, o);
          }
        }
        const float mc = m == -INFINITY ? 0.f : __fmul_rn(m, c);
        const uint64_t mc2 = f32x2(-mc, -mc);
        uint64_t la = 0, lb = 0;
#pragma unroll
        for (int h = 0; h < PH; ++h) {
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const uint32_t(&xs)[32] = x[2 * h + i / 16];
            const uint64_t z =
                fma2(f32x2(__uint_as_float(xs[2 * (i % 16)]), __uint_as_float(xs[2 * (i % 16) + 1])), c2, mc2);
            const float p0 = fast_exp2(f32x2_lo(z)), p1 = fast_exp2(f32x2_hi(z));
            uint64_t& l = i % 2 ? lb : la;
            l = add2(l, f32x2(p0, p1));
            pk[i] = pack_bf16x2(p0, p1);
          }
          tmem_st32(s_addr + 32 * h, pk);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&b->p_full[buf][h]);
        }
        l2 = add2(l2, add2(la, lb));
        phase ^= 1u << sb;
      }
      if (!go) break;
      // ---- output
      if (!(go = wait_product(last))) break;
      // (a row whose scores are all -inf has no weights: NaN, as in the formula)
      const float inv = m == -INFINITY ? __uint_as_float(0x7fc00000u) : 1.f / (f32x2_lo(l2) + f32x2_hi(l2));
      const bool bad = *reinterpret_cast<volatile int32_t*>(&b->bad[n_item % kFlagSlots]) == n_item;
      uint16_t* out = p.out + (static_cast<int64_t>(it.row0 + pos) * p.Hq + it.h * p.g + gi) * D;
#pragma unroll 1
      for (int k = 0; k < D / 64; ++k) {  // 64 channels: 128 bytes of the row
        uint32_t x[2][32];
        tmem_ld32(x[0], o_addr + 64 * k);
        tmem_ld32(x[1], o_addr + 64 * k + 32);
        tmem_wait_ld(x[0]);
        tmem_wait_ld(x[1]);
        if (k + 1 == D / 64) {  // the tile's columns are free for the next item
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&b->o_free[t]);
        }
        if (mine) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint64_t o = mul2(f32x2(__uint_as_float(x[i / 2][16 * (i % 2) + 2 * e]),
                                            __uint_as_float(x[i / 2][16 * (i % 2) + 2 * e + 1])),
                                      f32x2(inv, inv));
              w[e] = pack_bf16x2(f32x2_lo(o), f32x2_hi(o));
            }
            store32(out + 64 * k + 16 * i, w, p.out32);
          }
        }
        __syncwarp();
      }
      if (mine && bad) {  // non-finite V elements that this row sees, of the chunks that the guard cleaned
#pragma unroll 1
        for (int key = (it.t0 + 1) / VK * VK; key <= pos; ++key) {
          const uint16_t* v = p.v + static_cast<int64_t>(it.row0 + key) * p.v_stride + it.h * D;
#pragma unroll 1
          for (int i = 0; i < D; ++i)
            if ((v[i] & 0x7f80u) == 0x7f80u)
              out[i] = static_cast<uint16_t>(pack_bf16x2(bf16_bits_to_float(out[i]) + bf16_bits_to_float(v[i]), 0.f));
        }
      }
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
  if (warp == C::PRODUCER) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(b->tmem) : "memory");
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
  static std::atomic<uint64_t> prepared{0};  // devices whose limit is raised already, a bit a device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(prepared.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) prepared.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
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
  const cuuint32_t kb[3] = {64, 1, static_cast<cuuint32_t>(p.D == 256 ? Cfg<256>::KT : Cfg<128>::KT)};
  const cuuint32_t vb[3] = {64, 1, 64};
  if (!make_map(&q, in.q, 4, qd, qs, qb) || !make_map(&k, in.k, 3, kd, ks, kb) || !make_map(&v, in.v, 3, kd, vs, vb))
    return cudaErrorInvalidValue;
  return p.D == 64 ? launch<64>(p, q, k, v, s) : p.D == 128 ? launch<128>(p, q, k, v, s) : launch<256>(p, q, k, v, s);
}

}  // namespace mkv
