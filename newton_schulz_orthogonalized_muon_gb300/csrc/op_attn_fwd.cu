// Attention, forward: o_i = sum_j p_ij v_j, p_ij = exp(scale q_i . k_j -
// lse_i), in one pass over the keys with a running maximum and sum.
//
// An item is two tiles of 128 queries of one head, which walk the key tiles
// that they see.  Warp 0 loads by TMA, warp 1 issues every tcgen05.mma, and
// each tile has a warpgroup of its own (warps 4 - 7, 8 - 11) with one thread a
// query: while one tile's scores go through the exponential, the tensor pipe
// works for the other.  The scores (fp32) and o stay in TMEM; the
// probabilities are rounded to the operands' 16-bit type and written over the
// scores, from where the second product takes them as its A operand.  The row
// sum is taken from the probabilities before they are rounded.
//
// o of a walk over very many keys is handed over in parts to fp32 sums in
// memory (see op_attn.cuh), which follow the same maximum.
//
// A CTA that is done with its item takes over one that has not started yet
// (a cluster launch control request), and loads it and forms its first scores
// while the last item's outputs are written.
//
// The maximum that a row's exponents are taken against is raised only when a
// new score passes it by more than 2^8 (in exp2 units): o and the sum are
// then scaled down in TMEM.  Below that the probabilities stay under 256,
// exact in the same relative precision, and o is left alone.  (fp16: 2^4
// instead of 2^8, and all of them and their sum lifted by 2^11, so that small
// ones keep their bits; see op_attn.cuh.)
//
// Bound by the products together with what feeds them: two 128 x 128 tile
// pairs with dim 128 take 2048 cycles of the tensor pipe, and as many of
// shared memory, from which the score products take 128 bytes a cycle beside
// the loads of K and V; 32768 exponentials run next to them.  Measured: 8192
// causal tokens of 32 heads (8 of keys), dim 128, bf16, in 362 us, 1520
// TFLOP/s of the visible pairs' products, about 3180 cycles a step (377 to 380
// us where calls follow one another under the power limit).  dim 64, 8 x 1024
// causal tokens of 12 heads: 33 us, 390 TFLOP/s, 23% of the tensor pipe, one
// CTA an SM.  (Two warps a row's half each, 16 for the softmax, took 439 us
// with dim 128: a meeting a step and registers that spill cost more than the
// shorter way saves.)
#include <cstddef>

#include "common.cuh"
#include "internal.h"
#include "op_attn.cuh"

namespace muon {
namespace {

using namespace attn;

constexpr int CTRL_WARPS = 4;
constexpr int THREADS = 32 * (CTRL_WARPS + 8);
constexpr int ROWS = 2 * TILE;
template <typename T>
constexpr int SUM_TILES = SUM_ROWS<T> / TILE;        // key tiles between handovers of o (PARTS)

template <int DP>
struct Smem {
  static constexpr int T = tile_bytes<DP>();
  static constexpr int RK = 3;
  static constexpr int RV = DP == 128 ? 2 : 3;
  static constexpr int K_OFF = 2 * T;
  static constexpr int V_OFF = K_OFF + RK * T;
  static constexpr int BAR_OFF = V_OFF + RV * T;
  static constexpr int BYTES = BAR_OFF + 512;
  static_assert(BYTES <= 232448, "shared memory");
};

struct Item {
  int more;                  // 0: there is none, the CTA is done
  int beg, end;              // key tiles of both query tiles
  Range r[2];                // and of each
  int i0, rows;              // the first query, and queries from there to the sequence's end
  int nk, off;               // keys of the sequence; the position of query 0 among them
  void* out;                 // the first query's row of o
  float* lse;
};

// Phases are counted by the warps that wait, on through the items of a CTA.
struct Bars {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[3], k_empty[3], v_full[3], v_empty[3];
  uint64_t s_full[2], p_full[2], o_done[2], o_free[2];
  uint64_t edge, asked;
  uint64_t item_full[2], item_empty[2];
  alignas(16) uint4 answer;           // to a request for another item
  Item item[2];                       // announced by the loading warp
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Bars) <= 512, "barrier block");
// shared-memory address of a barrier; `bb` is the block's
#define BAR(f) (bb + static_cast<uint32_t>(offsetof(Bars, f)))

// Asks for a CTA of this grid that has not started; the answer is 16 bytes.
__device__ __forceinline__ void ask_next(uint32_t answer, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   answer),
               "r"(bar)
               : "memory");
}
// Its number, or -1 when all have started.
__device__ __forceinline__ int answered(uint32_t answer) {
  int id;
  asm volatile(
      "{\n"
      " .reg .b128 a;\n"
      " .reg .pred p;\n"
      " .reg .b32 x;\n"
      " ld.shared.b128 a, [%1];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n"
      " mov.b32 %0, -1;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 x, a;\n"
      " @p mov.b32 %0, x;\n"
      "}\n"
      : "=r"(id)
      : "r"(answer)
      : "memory");
  return id;
}

// ----------------------------------------------------------------- loads
template <typename T, int DP, bool PARTS>
__device__ __forceinline__ void load_role(const AttnParams& p, const CUtensorMap* mq, const CUtensorMap* mk,
                                          const CUtensorMap* mv, int tiles, int total, uint32_t sb, uint32_t bb, Bars* bar) {
  using S = Smem<DP>;
  volatile int* abort = &bar->abort;
  const int lane = threadIdx.x & 31, group = p.heads / p.kv_heads;
  Ring<S::RK> rk;
  Ring<S::RV> rv;
  Ring<2> items;
  uint32_t q_ph[2] = {1u, 1u}, ask_ph = 0, edges = 0;
  unsigned taken = 0;
  bool ok = true;
  PackedIndex index;
  if (p.cu_q != nullptr) index.fill(p, ROWS);
  for (int id = static_cast<int>(blockIdx.x); ok;) {
    __syncwarp();
    if (lane == 0 && id >= 0) {
      if constexpr (PARTS) {
        taken = atomicAdd(p.counter, 1u);
      } else {
        fence_proxy_async_smem();                  // every lane has read the last answer
        mbar_expect_at(BAR(asked), 16);
        ask_next(BAR(answer), BAR(asked));
      }
    }
    Item t;
    Work w{};
    t.more = id >= 0;
    if (id >= 0) {
      w = find_work(p, true, ROWS, p.heads, tiles, static_cast<uint32_t>(id), &index);
      t.i0 = w.tile * ROWS;
      t.rows = w.nq - t.i0;
      t.nk = w.nk;
      t.off = w.nk - w.nq;
      t.beg = t.end = 0;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        t.r[k] = Range{0, 0};
        if (w.ok && k * TILE < t.rows) t.r[k] = key_tiles(p, w, t.i0 + k * TILE, min(t.i0 + (k + 1) * TILE, w.nq) - 1);
      }
      if (t.r[0].count > 0 || t.r[1].count > 0) {
        t.beg = t.r[0].count == 0 ? t.r[1].first : t.r[1].count == 0 ? t.r[0].first : min(t.r[0].first, t.r[1].first);
        t.end = max(t.r[0].first + t.r[0].count, t.r[1].first + t.r[1].count);
      }
      const long long q0 = w.q0 + t.i0;
      t.out = static_cast<T*>(p.out) + w.b * p.ob + q0 * p.os + w.h * p.oh;
      t.lse = p.lse + w.b * p.lse_b + w.h * p.lse_h + q0;
    }
    if (w.ok || id < 0) {
      ok = wait_warp(BAR(item_empty) + 8 * items.s, items.ph ^ 1u, abort, p);
      if (!ok) break;
      if (lane == 0) {
        bar->item[items.s] = t;
        mbar_arrive_at(BAR(item_full) + 8 * items.s);
      }
      items.next();
    }
    if (id < 0) break;
    if (t.end > t.beg) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (ok && t.r[k].count > 0) {
          ok = wait_warp(BAR(q_empty) + 8 * k, q_ph[k], abort, p);
          q_ph[k] ^= 1u;
          if (ok && lane == 0) {
            mbar_expect_at(BAR(q_full) + 8 * k, S::T);
            load_tile<DP>(sb + k * S::T, mq, BAR(q_full) + 8 * k, w.h, w.q0 + t.i0 + k * TILE, w.b);
          }
        }
      }
      const int hk = w.h / group;
      for (int tile = t.beg; ok && tile < t.end; ++tile) {
        const int row = w.k0 + tile * TILE, valid = w.nk - tile * TILE;
        ok = wait_warp(BAR(k_empty) + 8 * rk.s, rk.ph ^ 1u, abort, p);
        if (!ok) break;
        if (lane == 0) {
          // rows past the sequence give scores that are masked, whatever they hold
          mbar_expect_at(BAR(k_full) + 8 * rk.s, S::T);
          load_tile<DP>(sb + S::K_OFF + rk.s * S::T, mk, BAR(k_full) + 8 * rk.s, hk, row, w.b);
        }
        rk.next();
        ok = wait_warp(BAR(v_empty) + 8 * rv.s, rv.ph ^ 1u, abort, p);
        if (!ok) break;
        const bool edge = p.cu_q != nullptr && valid < TILE;
        const uint32_t vt = sb + S::V_OFF + rv.s * S::T, fv = BAR(v_full) + 8 * rv.s;
        if (lane == 0) {
          mbar_expect_at(edge ? BAR(edge) : fv, S::T);
          load_tile<DP>(vt, mv, edge ? BAR(edge) : fv, hk, row, w.b);
        }
        if (edge) {
          ok = finish_edge_tile<DP>(vt, BAR(edge), edges, valid, abort, p);
          if (!ok) break;
          if (lane == 0) mbar_arrive_at(fv);
        }
        rv.next();
      }
    }
    if constexpr (PARTS) {                         // as many CTAs as there is scratch for, which take from a counter
      const unsigned next = gridDim.x + __shfl_sync(0xffffffffu, taken, 0);
      id = next < static_cast<unsigned>(total) ? static_cast<int>(next) : -1;
    } else {
      ok = ok && wait_warp(BAR(asked), ask_ph, abort, p);
      if (!ok) break;
      ask_ph ^= 1u;
      id = answered(BAR(answer));
    }
  }
  // after a wait ran out: a millisecond for copies in flight to land
  if (*abort != 0 && lane == 0) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {
    }
  }
  __syncwarp();
}

// -------------------------------------------------------------- products
template <typename T, int DP, bool PARTS>
__device__ __forceinline__ void product_role(const AttnParams& p, uint32_t sb, uint32_t bb, uint32_t tmem, Bars* bar) {
  using S = Smem<DP>;
  volatile int* abort = &bar->abort;
  Ring<S::RK> rk;                                // the K tile of the scores to come
  Ring<S::RV> rv;
  Ring<2> items;
  uint32_t q_ph[2] = {0u, 0u}, p_ph[2] = {0u, 0u}, free_ph[2] = {1u, 1u};
  bool ok = true;
  while (ok && wait_warp(BAR(item_full) + 8 * items.s, items.ph, abort, p)) {
    const Item& t = bar->item[items.s];
    const bool more = t.more != 0;
    const int beg = t.beg, end = t.end, first[2] = {t.r[0].first, t.r[1].first},
              last[2] = {t.r[0].first + t.r[0].count - 1, t.r[1].first + t.r[1].count - 1};
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive_at(BAR(item_empty) + 8 * items.s);
    items.next();
    if (!more) break;
    if (end <= beg) continue;
    auto sees = [&](int k, int tile) { return tile >= first[k] && tile <= last[k]; };
    auto scores = [&](int k, int tile) {
      mma_over_dim<T, DP>(tmem + k * TILE, desc_dim(sb + k * S::T), desc_dim(sb + S::K_OFF + rk.s * S::T));
      commit_warp(BAR(s_full) + 8 * k);
      if (tile == last[k]) commit_warp(BAR(q_empty) + 8 * k);
    };
    uint32_t acc[2] = {0u, 0u};
    ok = wait_warp(BAR(k_full) + 8 * rk.s, rk.ph, abort, p);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (ok && last[k] >= first[k]) {
        ok = wait_warp(BAR(q_full) + 8 * k, q_ph[k], abort, p);
        q_ph[k] ^= 1u;
      }
      if (ok && sees(k, beg)) {
        tc_fence_after();
        scores(k, beg);
      }
    }
    if (ok) commit_warp(BAR(k_empty) + 8 * rk.s);
    rk.next();
    for (int tile = beg; ok && tile < end; ++tile) {
      const bool next = tile + 1 < end;
      // this step's tiles before the probabilities, so that no wait stands between products
      ok = wait_warp(BAR(v_full) + 8 * rv.s, rv.ph, abort, p) &&
           (!next || wait_warp(BAR(k_full) + 8 * rk.s, rk.ph, abort, p));
      if (!ok) break;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (ok && sees(k, tile)) {
          ok = wait_warp(BAR(p_full) + 8 * k, p_ph[k], abort, p);
          p_ph[k] ^= 1u;
          if (ok && acc[k] == 0u) {              // over the last item's o
            ok = wait_warp(BAR(o_free) + 8 * k, free_ph[k], abort, p);
            free_ph[k] ^= 1u;
          }
          if (ok) {
            tc_fence_after();
            // a new part: the softmax warps have taken o before they wrote these probabilities
            if constexpr (PARTS) {
              if ((tile - first[k]) % SUM_TILES<T> == 0) acc[k] = 0u;
            }
            mma_over_tokens<T, DP, TILE>(tmem + 256 + k * TILE, tmem + k * TILE,
                                         desc_tokens(sb + S::V_OFF + rv.s * S::T), acc[k]);
            commit_warp(BAR(o_done) + 8 * k);
            acc[k] = 1u;
          }
        }
        // over the probabilities just used: the tensor pipe runs in order
        if (ok && next && sees(k, tile + 1)) scores(k, tile + 1);
      }
      if (!ok) break;
      commit_warp(BAR(v_empty) + 8 * rv.s);
      rv.next();
      if (next) {
        commit_warp(BAR(k_empty) + 8 * rk.s);
        rk.next();
      }
    }
  }
  // after a wait ran out: the products in flight end by themselves, a millisecond for them
  if (*abort != 0 && (threadIdx.x & 31) == 0) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {
    }
  }
  __syncwarp();
}

// ------------------------------------------------------- softmax, output
// A row's sums of o from its walk's parts, column k at [32 k] ...
template <int DP>
__device__ __forceinline__ float* part_sums(const AttnParams& p, int t, int quad, int lane) {
  return p.part + ((static_cast<long long>(blockIdx.x) * 2 + t) * 4 + quad) * (32 * DP) + lane;
}
// ... and the factor that brings them from reference `base` to `top`.
__device__ __forceinline__ float rescale(float base, float top, float c) {
  return base == top ? 1.f : exp2_fast((base - top) * c);
}

template <typename T, int DP, bool PARTS>
__device__ __forceinline__ void softmax_role(const AttnParams& p, uint32_t bb, uint32_t tmem, Bars* bar) {
  volatile int* abort = &bar->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = (warp - CTRL_WARPS) >> 2, quad = warp & 3;
  const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
  const uint32_t s_at = tmem + lanes + t * TILE, o_at = tmem + lanes + 256 + t * TILE;
  const float c = p.scale * LOG2E;
  const F2 cc = f2_make(c, c);
  Ring<2> items;
  uint32_t steps = 0;                              // of this tile so far: the phases of its barriers
  while (wait_warp(BAR(item_full) + 8 * items.s, items.ph, abort, p)) {
    const Item& it = bar->item[items.s];
    if (it.more == 0) break;
    const int cnt = it.r[t].count, i0 = it.i0, nk = it.nk, off = it.off, first = it.r[t].first;
    const int q0 = i0 + t * TILE, q = q0 + quad * 32 + lane;
    float top = -INFINITY;                         // the scores' reference, before scaling
    F2 sum2 = f2_make(0.f, 0.f);
    [[maybe_unused]] float base = top;             // PARTS: the reference of the handed over sums
    bool ok = true;
    for (int i = 0; i < cnt; ++i, ++steps) {
      const int j0 = (first + i) * TILE;
      if constexpr (PARTS) {
        if (i > 0 && i % SUM_TILES<T> == 0) {
          ok = wait_warp(BAR(o_done) + 8 * t, (steps - 1) & 1u, abort, p);
          if (!ok) break;
          tc_fence_after();
          float* sums = part_sums<DP>(p, t, quad, lane);
          const float f = rescale(base, top, c);
#pragma unroll 1
          for (int k = 0; k < DP; k += 32) {
            float o[32];
            tmem_ld32(o_at + k, o);
            tmem_ld_wait();
            float* at = sums + 32 * k;
#pragma unroll
            for (int e = 0; e < 32; ++e) at[32 * e] = i == SUM_TILES<T> ? o[e] : fmaf(at[32 * e], f, o[e]);
          }
          base = top;
        }
      }
      float v[TILE];
      ok = wait_warp(BAR(s_full) + 8 * t, steps & 1u, abort, p);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < TILE; k += 32) tmem_ld32(s_at + k, v + k);
      tmem_ld_wait();
      if (j0 + TILE > nk ||
          (p.causal && (j0 + TILE - 1 > q0 + off || (p.window > 0 && q0 + TILE - 1 + off - j0 >= p.window)))) {
        int lo = 0, hi = nk - j0;
        if (p.causal) {
          hi = min(hi, q + off + 1 - j0);
          if (p.window > 0) lo = q + off - p.window + 1 - j0;
        }
#pragma unroll
        for (int k = 0; k < TILE; k += 32) {
          const uint32_t m = bits32(lo - k, hi - k);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!(m & (1u << e))) v[k + e] = -INFINITY;
        }
      }
      float m[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
      for (int k = 4; k < TILE; k += 8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) m[e] = k + 4 + e < TILE ? fmaxf(fmaxf(m[e], v[k + e]), v[k + 4 + e]) : fmaxf(m[e], v[k + e]);
      }
      const float mt = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
      if (i == 0) {
        top = mt;
      } else {
        const bool up = mt > top && (top == -INFINITY || (mt - top) * c > raise<T>());
        if (__any_sync(0xffffffffu, up)) {
          ok = wait_warp(BAR(o_done) + 8 * t, (steps - 1) & 1u, abort, p);
          if (!ok) break;
          tc_fence_after();
          const float f = !up ? 1.f : top == -INFINITY ? 0.f : exp2_fast((top - mt) * c);
          if (up) top = mt;
          sum2 = f2_mul(sum2, f2_make(f, f));
#pragma unroll 1
          for (int k = 0; k < DP; k += 32) {
            float o[32];
            tmem_ld32(o_at + k, o);
            tmem_ld_wait();
            uint32_t* u = reinterpret_cast<uint32_t*>(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= f;
            tmem_st32(o_at + k, u);
          }
          tmem_st_wait();
        }
      }
      const float ref = top == -INFINITY ? 0.f : fmaf(-top, c, static_cast<float>(lift_forward<T>()));
      const F2 rr = f2_make(ref, ref);
      F2 here = f2_make(0.f, 0.f);                 // this tile's sum: small values meet each other first
#pragma unroll
      for (int k = 0; k < TILE; k += 64) {
#pragma unroll
        for (int e = k; e < k + 64; e += 2) {
          const float2 a = f2_split(f2_fma(f2_make(v[e], v[e + 1]), cc, rr));
          v[e] = exp2_fast(a.x);
          v[e + 1] = exp2_fast(a.y);
          here = f2_add(here, f2_make(v[e], v[e + 1]));
        }
        store_rounded<T, 32>(s_at + k / 2, v + k);
      }
      sum2 = f2_add(sum2, here);
      warp_arrive(BAR(p_full) + 8 * t);
    }
    if (ok && cnt > 0) ok = wait_warp(BAR(o_done) + 8 * t, (steps - 1) & 1u, abort, p);
    if (!ok) break;
    tc_fence_after();
    if constexpr (PARTS) {
      if (cnt > SUM_TILES<T>) {                    // the last part's o joins the others
        const float* sums = part_sums<DP>(p, t, quad, lane);
        const float f = rescale(base, top, c);
#pragma unroll 1
        for (int k = 0; k < DP; k += 32) {
          float o[32];
          tmem_ld32(o_at + k, o);
          tmem_ld_wait();
          const float* at = sums + 32 * k;
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = fmaf(at[32 * e], f, o[e]);
          tmem_st32(o_at + k, reinterpret_cast<const uint32_t*>(o));
        }
        tmem_st_wait();
      }
    }
    const float2 s2 = f2_split(sum2);
    const float sum = s2.x + s2.y, inv = sum == 0.f ? 0.f : 1.f / sum;
    const int row = t * TILE + quad * 32, rows = it.rows - row;      // the warp's first query, and queries from it on
    T* out = static_cast<T*>(it.out) + row * p.os;
    if (lane < rows) it.lse[row + lane] = sum == 0.f ? -INFINITY : fmaf(top, p.scale, logf(sum * lowered(lift_forward<T>())));
    if (cnt > 0) {
      float mul[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) mul[k] = __shfl_sync(0xffffffffu, inv, (lane >> 2) + 8 * k);
#pragma unroll 1
      for (int k = 0; k < DP; k += 32) store_rows<T>(o_at + k, out + k, p.os, rows, p.dim - k, mul);
      warp_arrive(BAR(o_free) + 8 * t);
    } else if (lane < rows) {
      for (int k = 0; k < p.dim; k += 8) *reinterpret_cast<uint4*>(out + lane * p.os + k) = make_uint4(0u, 0u, 0u, 0u);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive_at(BAR(item_empty) + 8 * items.s);
    items.next();
  }
}

template <typename T, int DP, bool PARTS>
__global__ void __launch_bounds__(THREADS, 1)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv, const AttnParams p, int tiles, int total) {
  using S = Smem<DP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* bar = reinterpret_cast<Bars*>(smem + S::BAR_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sb = smem_u32(smem), bb = sb + S::BAR_OFF;
  if (!swizzle_aligned(sb, p)) return;
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->q_full[i], 1);
      mbar_init(&bar->q_empty[i], 1);
      mbar_init(&bar->s_full[i], 1);
      mbar_init(&bar->p_full[i], 4);
      mbar_init(&bar->o_done[i], 1);
      mbar_init(&bar->o_free[i], 4);
      mbar_init(&bar->item_full[i], 1);
      mbar_init(&bar->item_empty[i], 1 + 8);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&bar->k_full[i], 1);
      mbar_init(&bar->k_empty[i], 1);
      mbar_init(&bar->v_full[i], 1);
      mbar_init(&bar->v_empty[i], 1);
    }
    mbar_init(&bar->edge, 1);
    mbar_init(&bar->asked, 1);
    bar->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&bar->tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem;
  // a softmax thread holds a row of 128 scores: registers move from the
  // control warps (4 x 32 x 88 + 8 x 32 x 200 of the 384 x 168 at launch)
  if (warp < CTRL_WARPS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0) load_role<T, DP, PARTS>(p, &mq, &mk, &mv, tiles, total, sb, bb, bar);
    if (warp == 1) product_role<T, DP, PARTS>(p, sb, bb, tmem, bar);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    softmax_role<T, DP, PARTS>(p, bb, tmem, bar);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <typename T, int DP, bool PARTS>
cudaError_t launch_items(const AttnParams& p, const CUtensorMap* m, long long grid, long long tiles, long long items,
                         cudaStream_t s) {
  auto kern = attn_fwd_kernel<T, DP, PARTS>;
  static std::atomic<unsigned long long> done;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), Smem<DP>::BYTES, done);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(grid), THREADS, Smem<DP>::BYTES, s>>>(m[0], m[1], m[2], p, static_cast<int>(tiles),
                                                                     static_cast<int>(items));
  return cudaGetLastError();
}

template <typename T, int DP>
cudaError_t launch_dims(const AttnParams& p, const CUtensorMap* m, int sms, cudaStream_t s) {
  const bool packed = p.cu_q != nullptr;
  const long long tiles = tile_bound(p.sq, ROWS, p.batch, packed);
  const long long items = tiles * p.heads * (packed ? 1 : p.batch);
  if (items > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  if (p.part == nullptr) return launch_items<T, DP, false>(p, m, items, tiles, items, s);
  const cudaError_t e = cudaMemsetAsync(p.counter, 0, sizeof(unsigned), s);
  if (e != cudaSuccess) return e;
  const long long ctas = attn_part_ctas(p.dim, false, sms);
  return launch_items<T, DP, true>(p, m, items < ctas ? items : ctas, tiles, items, s);
}

template <typename T>
cudaError_t launch_type(const AttnParams& p, const CUtensorMap* m, int sms, cudaStream_t s) {
  return p.dim <= 64 ? launch_dims<T, 64>(p, m, sms, s) : launch_dims<T, 128>(p, m, sms, s);
}

}  // namespace

int attn_qtiles(int sq, int batch, bool packed) { return static_cast<int>(tile_bound(sq, TILE, batch, packed)); }

cudaError_t launch_attn_fwd(const AttnParams& p, const CUtensorMap* m, int sms, cudaStream_t s) {
  return p.dtype == DT_BF16 ? launch_type<__nv_bfloat16>(p, m, sms, s) : launch_type<__half>(p, m, sms, s);
}

}  // namespace muon
