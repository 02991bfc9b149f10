// The backward pass of attention, recomputing the probabilities.
//
//   p_ij = exp(scale q_i . k_j - lse_i),  delta_i = do_i . o_i
//   dv_j = sum_i p_ij do_i,   ds_ij = p_ij (do_i . v_j - delta_i)
//   dq_i = scale sum_j ds_ij k_j,   dk_j = scale sum_i ds_ij q_i
//
// attn_prep_kernel writes -lse_i log2(e) and -delta_i, tile by tile (HBM-bound:
// it reads o and do).  attn_bwd_kernel has two kinds of items.  One owns a
// tile of 128 keys, walks the query tiles that see them (of every query head
// that shares the key head) and keeps dk and dv in TMEM; the other owns a
// tile of 128 queries, walks its key tiles and keeps dq in TMEM.  No value is
// added by atomics, so results do not change from call to call; the price is
// that scores and dP are formed twice, seven products a tile pair, not five.
//
// Warp-specialised: warp 0 loads tiles by TMA, warp 1 issues every
// tcgen05.mma, the other warps turn scores into p and ds.  p and ds never
// leave the SM: each warp writes its 16-bit values over the fp32 scores (or
// dP) that it read, and the next product takes them from TMEM as its A
// operand.  For dk and dv the scores are transposed (rows are keys), so that
// p and ds are that operand as they stand.
//
// With dim 128 the products bind: 2048 (dk, dv) and 1536 (dq) cycles of the
// tensor pipe for 128 x 128 pairs, measured 2600 to 2900 and 2030, as shared
// memory, from which N = 128 products take 128 bytes a cycle, is as busy.
// 8192 causal tokens of 32 heads (8 of keys), bf16: 1.09 ms, 1270 TFLOP/s of
// the five products that the gradient needs, 1770 of the seven.  With short
// sequences and dim 64 the way of a tile through the element-wise warps
// binds: 8 x 1024 causal tokens of 12 heads take 74 us, 440 TFLOP/s of five,
// with 46% of the issue slots and 30% of the tensor pipe used.  (p and ds of
// a tile in one go, with half the barriers, took 82 us: no product then runs
// beside them.)
#include <cstddef>

#include "common.cuh"
#include "internal.h"
#include "op_attn.cuh"

namespace muon {
namespace {

using namespace attn;

constexpr int CTRL_WARPS = 2;
constexpr int COLS = 32;                          // scores of a row that a warp has

// The tile that stays has 128 rows; the walked ones 128 with dim up to 128
// and 64 with dim up to 64, where 256 of the SM's 512 TMEM columns and under
// half of its shared memory are enough, so that two CTAs share an SM and each
// fills the other's waits.
template <int DP>
struct Shape {
  static constexpr int WT = DP;                             // rows of a walked tile
  static constexpr int PARTS = WT / COLS;                   // warps of a TMEM lane quadrant
  static constexpr int CALC = 4 * PARTS;
  static constexpr int THREADS = 32 * (CTRL_WARPS + CALC);
  static constexpr int CTAS = DP == 64 ? 2 : 1;             // of an SM
  static constexpr uint32_t TMEM = DP == 64 ? 256 : 512;    // columns
};

// ------------------------------------------------------------ statistics
// -lse log2(e) and -delta of one tile of queries, 128 values each (the sign
// that two-wide additions want), padded: rows past the sequence and rows that
// see no key get -inf, so that their p is 0.
template <typename T, int DP>
__global__ void __launch_bounds__(256) attn_prep_kernel(const AttnParams p, int tiles) {
  constexpr int LPR = DP / 8;                     // lanes of a row, 16 bytes each
  constexpr int N = TILE * LPR / 256;             // rows of a thread
  __shared__ Work sw;
  pdl_launch_dependents();
  if (threadIdx.x < 32) {
    const Work w = find_work(p, true, TILE, p.heads, tiles, blockIdx.x);
    if (threadIdx.x == 0) sw = w;
  }
  __syncthreads();
  const Work w = sw;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.counter = 0u;      // of the gradient kernel's items
  if (!w.ok) return;
  const int l = threadIdx.x % LPR, r0 = w.tile * TILE + threadIdx.x / LPR;
  const T* o = static_cast<const T*>(p.o) + w.b * p.ob + static_cast<long long>(w.q0) * p.os + w.h * p.oh + 8 * l;
  const T* g = static_cast<const T*>(p.dout) + w.b * p.dob + static_cast<long long>(w.q0) * p.dos + w.h * p.doh + 8 * l;
  const float* lse = p.lse + w.b * p.lse_b + w.h * p.lse_h + w.q0;
  const long long at = ((static_cast<long long>(w.b) * p.heads + w.h) * tiles + w.qtile) * TILE;
  uint4 a[N], b[N];
  float e[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int i = r0 + k * (256 / LPR);
    a[k] = b[k] = make_uint4(0u, 0u, 0u, 0u);
    e[k] = -INFINITY;
    if (i < w.nq) {
      if (8 * l < p.dim) {
        a[k] = ld_stream16(o + static_cast<long long>(i) * p.os);
        b[k] = ld_stream16(g + static_cast<long long>(i) * p.dos);
      }
      if (l == 0) e[k] = lse[i];
    }
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    float x[8], y[8], s = 0.f;
    unpack16<T>(a[k], x);
    unpack16<T>(b[k], y);
#pragma unroll
    for (int c = 0; c < 8; ++c) s = fmaf(x[c], y[c], s);
#pragma unroll
    for (int c = LPR / 2; c > 0; c >>= 1) s += __shfl_xor_sync(0xffffffffu, s, c);
    if (l == 0) {
      const int i = r0 + k * (256 / LPR);
      p.stat_lse[at + i] = e[k] == -INFINITY ? -INFINITY : -e[k] * LOG2E;
      p.stat_delta[at + i] = -s;
    }
  }
}

// --------------------------------------------------------- shared memory
// Two tiles stay (K and V, or Q and dO); the rings hold the tiles that are
// walked: three of the operand that two products a step read, two of the other.
template <int DP>
struct Smem {
  static constexpr int WT = Shape<DP>::WT;
  static constexpr int OWN = tile_bytes<DP>();    // a tile that stays
  static constexpr int T = OWN / TILE * WT;       // a walked one
  static constexpr int RA = 3;
  static constexpr int RB = DP == 128 ? 2 : 3;
  static constexpr int STAT = 2 * WT * 4;         // lse and delta of one walked query tile
  static constexpr int A_OFF = 2 * OWN;
  static constexpr int B_OFF = A_OFF + RA * T;
  static constexpr int STAT_OFF = B_OFF + RB * T;
  static constexpr int BAR_OFF = STAT_OFF + RB * STAT;
  static constexpr int BYTES = BAR_OFF + 320;
  static_assert(BYTES * Shape<DP>::CTAS <= 232448 - 1024 * (Shape<DP>::CTAS - 1), "shared memory");
};

// Every barrier's phases are counted by the warps that wait on it, on through
// the items of a CTA.
struct Bars {
  uint64_t own[2], own_empty[2];      // the two tiles that stay: loaded, and read by their last product
  uint64_t a_full[3], a_empty[3];     // walked tiles
  uint64_t b_full[3], b_empty[3];
  uint64_t s_full, s_free;            // scores: formed; read into registers (dq)
  uint64_t p_full;                    // dk, dv: probabilities written
  uint64_t dpk_full, dsk_full;        //   dP formed, ds written
  uint64_t dp_full[2], ds_full[2];    // dq: the same, twice
  uint64_t done, acc_free;            // an item's sums formed; read
  uint64_t edge[2];
  uint64_t id_full[2], id_empty[2];   // the items that the loading warp announces
  uint32_t id[2];
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Bars) <= 320, "barrier block");
// shared-memory address of a barrier; `bb` is the block's
#define BAR(f) (bb + static_cast<uint32_t>(offsetof(Bars, f)))

__device__ __forceinline__ void init_bars(Bars* s, int calc_warps) {
  for (int i = 0; i < 2; ++i) {
    mbar_init(&s->own[i], 1);
    mbar_init(&s->own_empty[i], 1);
    mbar_init(&s->dp_full[i], 1);
    mbar_init(&s->ds_full[i], calc_warps);
    mbar_init(&s->edge[i], 1);
    mbar_init(&s->id_full[i], 1);
    mbar_init(&s->id_empty[i], 1 + calc_warps);
  }
  for (int i = 0; i < 3; ++i) {
    mbar_init(&s->a_full[i], 1);
    mbar_init(&s->a_empty[i], 1);
    mbar_init(&s->b_full[i], 1);
    mbar_init(&s->b_empty[i], 1);
  }
  mbar_init(&s->s_full, 1);
  mbar_init(&s->s_free, calc_warps);
  mbar_init(&s->p_full, calc_warps);
  mbar_init(&s->dpk_full, 1);
  mbar_init(&s->dsk_full, calc_warps);
  mbar_init(&s->done, 1);
  mbar_init(&s->acc_free, calc_warps);
  s->abort = 0;
  fence_mbar_init();
}

// What every warp knows of the launch.
struct Grid {
  const CUtensorMap *mq, *mk, *mv, *mdo;
  uint32_t nk, total;        // items of dk and dv, and all
  int ktiles, qtiles;
};

// The items that the loading warp announced, for another warp of the CTA.
struct Items {
  Ring<2> at;
  __device__ __forceinline__ bool next(uint32_t bb, const Bars* bar, const Grid& g, volatile int* abort,
                                       const AttnParams& p, uint32_t* id) {
    if (!wait_warp(BAR(id_full) + 8 * at.s, at.ph, abort, p)) return false;
    *id = *const_cast<const volatile uint32_t*>(&bar->id[at.s]);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive_at(BAR(id_empty) + 8 * at.s);
    at.next();
    return *id < g.total;
  }
};

// One item: what it owns and what it walks.
struct Item {
  bool dkv;
  Work w;
  int own;                   // first row of the tile that stays, in its sequence
  Range r;                   // walked tiles (of every head of the group: dk, dv)
  int n;                     // steps
};

template <int WT>
__device__ __forceinline__ Item find_item(const AttnParams& p, const Grid& g, uint32_t id) {
  Item t;
  t.dkv = id < g.nk;
  t.w = t.dkv ? find_work(p, false, TILE, p.kv_heads, g.ktiles, id)
              : find_work(p, true, TILE, p.heads, g.qtiles, id - g.nk);
  t.own = t.w.tile * TILE;
  t.r = Range{0, 0};
  if (t.w.ok)
    t.r = t.dkv ? query_tiles<WT>(p, t.w, t.own, min(t.own + TILE, t.w.nk) - 1)
                : key_tiles<WT>(p, t.w, t.own, min(t.own + TILE, t.w.nq) - 1);
  t.n = t.r.count * (t.dkv ? p.heads / p.kv_heads : 1);
  return t;
}

// ----------------------------------------------------------------- loads
template <typename T, int DP>
__device__ __forceinline__ void load_role(const AttnParams& p, const Grid& g, uint32_t sb, uint32_t bb, Bars* bar) {
  volatile int* abort = &bar->abort;
  using S = Smem<DP>;
  constexpr int WT = S::WT, BOX = DP == 64 ? 64 : TILE;      // rows of a walked tile, of a map's box
  const int lane = threadIdx.x & 31;
  Ring<S::RA> ra;
  Ring<S::RB> rb;
  uint32_t edges[2] = {0u, 0u}, own_ph = 1u;                 // the first item finds its places free
  // The CTA's first item is its own number; the next ones are taken from a
  // counter (which the statistics kernel sets to 0) while an item is under
  // way, so that long and short items even out.  Which CTA computes an item
  // changes nothing in its result.
  Ring<2> ids;
  uint32_t id = blockIdx.x, next_id = 0;
  auto take = [&]() {
    if (lane == 0) next_id = p.counter != nullptr ? gridDim.x + atomicAdd(p.counter, 1u) : id + gridDim.x;
  };
  bool ok = true, waited = false;
  for (;; id = __shfl_sync(0xffffffffu, next_id, 0)) {
    ok = ok && wait_warp(BAR(id_empty) + 8 * ids.s, ids.ph ^ 1u, abort, p);
    if (!ok) break;
    if (lane == 0) {
      *const_cast<volatile uint32_t*>(&bar->id[ids.s]) = id;
      mbar_arrive_at(BAR(id_full) + 8 * ids.s);
    }
    ids.next();
    if (id >= g.total) break;
    const Item t = find_item<WT>(p, g, id);
    if (t.n == 0) {
      if (!waited) pdl_wait();
      waited = true;
      take();
      continue;
    }
    const Work& w = t.w;
    // dk, dv: K and V stay, Q and dO are walked; dq: Q and dO stay, K and V are walked
    const CUtensorMap* own0 = t.dkv ? g.mk : g.mq;
    const CUtensorMap* own1 = t.dkv ? g.mv : g.mdo;
    const CUtensorMap* walk_a = t.dkv ? g.mq : g.mk;
    const CUtensorMap* walk_b = t.dkv ? g.mdo : g.mv;
    const int own_row = (t.dkv ? w.k0 : w.q0) + t.own, group = p.heads / p.kv_heads;
    const int first = t.dkv ? w.q0 : w.k0, len = t.dkv ? w.nq : w.nk;
    const int h0 = t.dkv ? w.h * group : w.h / group, h1 = t.dkv ? h0 + group : h0 + 1;
    ok = wait_warp(BAR(own_empty), own_ph, abort, p);
    if (!ok) break;
    if (lane == 0) {
      mbar_expect_at(BAR(own), S::OWN);
      load_tile<DP, TILE, BOX>(sb, own0, BAR(own), w.h, own_row, w.b);
    }
    bool second = true;                                      // the other own tile is still to come
    for (int h = h0; ok && h < h1; ++h) {
      const long long stat = ((static_cast<long long>(w.b) * p.heads + h) * g.qtiles + w.qtile) * TILE;
      for (int i0 = t.r.first * WT; i0 < (t.r.first + t.r.count) * WT; i0 += WT) {
        const int row = first + i0, valid = len - i0;
        const bool edge = p.cu_q != nullptr && valid < WT;
        const uint32_t at = sb + S::A_OFF + ra.s * S::T, bt = sb + S::B_OFF + rb.s * S::T;
        const uint32_t fa = BAR(a_full) + 8 * ra.s, fb = BAR(b_full) + 8 * rb.s;
        ok = wait_warp(BAR(a_empty) + 8 * ra.s, ra.ph ^ 1u, abort, p);
        if (!ok) break;
        if (lane == 0) {
          if (!edge) mbar_expect_at(fa, S::T);
          else mbar_expect_at(BAR(edge), S::T);
          load_tile<DP, WT, BOX>(at, walk_a, edge ? BAR(edge) : fa, h, row, w.b);
        }
        if (second) {                                        // after what the first scores want
          second = false;
          ok = wait_warp(BAR(own_empty) + 8, own_ph, abort, p);
          if (!ok) break;
          if (lane == 0) {
            mbar_expect_at(BAR(own) + 8, S::OWN);
            load_tile<DP, TILE, BOX>(sb + S::OWN, own1, BAR(own) + 8, w.h, own_row, w.b);
          }
          if (!waited) pdl_wait();                           // statistics and counter are the previous kernel's
          waited = true;
          take();
        }
        ok = wait_warp(BAR(b_empty) + 8 * rb.s, rb.ph ^ 1u, abort, p);
        if (!ok) break;
        if (lane == 0) {
          if (!edge) mbar_expect_at(fb, S::T + (t.dkv ? S::STAT : 0));
          else mbar_expect_at(BAR(edge) + 8, S::T + (t.dkv ? S::STAT : 0));
          const uint32_t to = edge ? BAR(edge) + 8 : fb;
          load_tile<DP, WT, BOX>(bt, walk_b, to, h, row, w.b);
          if (t.dkv) {
            const uint32_t st = sb + S::STAT_OFF + rb.s * S::STAT;
            bulk_load(st, p.stat_lse + stat + i0, WT * 4, to);
            bulk_load(st + WT * 4, p.stat_delta + stat + i0, WT * 4, to);
          }
        }
        if (edge) {
          // a packed sequence ends inside the tile: the next one's rows become zeros, so that a NaN
          // or an infinity there has no part in a product with a zero probability
          ok = finish_edge_tile<DP, WT>(at, BAR(edge), edges[0], valid, abort, p);
          if (ok && lane == 0) mbar_arrive_at(fa);
          ok = ok && finish_edge_tile<DP, WT>(bt, BAR(edge) + 8, edges[1], valid, abort, p);
          if (ok && lane == 0) mbar_arrive_at(fb);
          if (!ok) break;
        }
        ra.next();
        rb.next();
      }
    }
    own_ph ^= 1u;
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
template <typename T, int DP>
__device__ __forceinline__ void product_role(const AttnParams& p, const Grid& g, uint32_t sb, uint32_t bb,
                                             uint32_t tmem, Bars* bar) {
  using S = Smem<DP>;
  constexpr int WT = S::WT;
  constexpr uint32_t S_COL = 0, DP_COL = WT;
  constexpr uint32_t DV_COL = 2 * WT, DK_COL = 2 * WT + DP;          // dk, dv
  constexpr uint32_t DQ_COL = 3 * WT;                                // dq: dP twice
  volatile int* abort = &bar->abort;
  const uint64_t own0 = desc_dim(sb), own1 = desc_dim(sb + S::OWN);
  Ring<S::RA> ra, na;                        // this step's walked tile, and the next one's
  Ring<S::RB> rb, nb;
  Ring<2> buf, next;                         // the two places of dP (dq)
  uint32_t own_ph = 0, k_ph = 0, s_ph = 0, acc_ph = 1;
  auto wait_a = [&]() { return wait_warp(BAR(a_full) + 8 * na.s, na.ph, abort, p); };
  auto wait_b = [&]() { return wait_warp(BAR(b_full) + 8 * nb.s, nb.ph, abort, p); };
  auto scores = [&](bool last) {
    mma_over_dim<T, DP, WT>(tmem + S_COL, own0, desc_dim(sb + S::A_OFF + na.s * S::T));
    commit_warp(BAR(s_full));
    if (last) commit_warp(BAR(own_empty));
    na.next();
  };
  auto dprobs = [&](uint32_t col, uint32_t full, bool last) {
    mma_over_dim<T, DP, WT>(tmem + col, own1, desc_dim(sb + S::B_OFF + nb.s * S::T));
    commit_warp(full);
    if (last) commit_warp(BAR(own_empty) + 8);
  };
  bool ok = true, was_dkv = false;
  Items items;
  for (uint32_t id; ok && items.next(bb, bar, g, abort, p, &id);) {
    const Item t = find_item<WT>(p, g, id);
    if (t.n == 0) continue;
    // an item's first products go ahead of the previous item's outputs; its
    // sums wait for them.  From dk, dv to dq the places differ: wait at once.
    bool sums_free = false;
    if (!t.dkv && was_dkv) {
      ok = wait_warp(BAR(acc_free), acc_ph, abort, p);
      sums_free = true;
    }
    was_dkv = t.dkv;
    ok = ok && wait_warp(BAR(own), own_ph, abort, p) && wait_a();
    if (!ok) break;
    tc_fence_after();
    scores(t.n == 1);
    ok = wait_warp(BAR(own) + 8, own_ph, abort, p) && wait_b();
    if (!ok) break;
    own_ph ^= 1u;
    tc_fence_after();
    uint32_t acc = 0;
    if (t.dkv) {
      dprobs(DP_COL, BAR(dpk_full), t.n == 1);
      nb.next();
      for (int left = t.n - 1; left >= 0; --left, k_ph ^= 1u, acc = 1) {
        // a step's tiles are waited for before the probabilities, so that
        // products follow one another without a wait in between
        ok = (left == 0 || wait_a()) && wait_warp(BAR(p_full), k_ph, abort, p) &&
             (acc != 0 || wait_warp(BAR(acc_free), acc_ph, abort, p));
        if (!ok) break;
        tc_fence_after();
        mma_over_tokens<T, DP, COLS, WT>(tmem + DV_COL, tmem + S_COL, desc_tokens<WT>(sb + S::B_OFF + rb.s * S::T), acc);
        commit_warp(BAR(b_empty) + 8 * rb.s);      // dP, issued earlier, has read this dO tile too
        rb.next();
        // the next scores overwrite the probabilities: the tensor pipe runs in order
        if (left > 0) scores(left == 1);
        ok = (left == 0 || wait_b()) && wait_warp(BAR(dsk_full), k_ph, abort, p);
        if (!ok) break;
        tc_fence_after();
        mma_over_tokens<T, DP, COLS, WT>(tmem + DK_COL, tmem + DP_COL, desc_tokens<WT>(sb + S::A_OFF + ra.s * S::T), acc);
        commit_warp(BAR(a_empty) + 8 * ra.s);
        ra.next();
        if (left > 0) {
          dprobs(DP_COL, BAR(dpk_full), left == 1);
          nb.next();
        }
      }
    } else {
      auto ahead = [&](bool last) {
        dprobs(DP_COL + next.s * WT, BAR(dp_full) + 8 * next.s, last);
        commit_warp(BAR(b_empty) + 8 * nb.s);
        nb.next();
        rb.next();
        next.next();
      };
      ahead(t.n == 1);
      for (int left = t.n - 1; left >= 0; --left, s_ph ^= 1u, acc = 1) {
        // the next tile's scores and dP (over the ds before last, which dq has read: the tensor pipe runs in order)
        if (left > 0) {
          ok = wait_a() && wait_b() && wait_warp(BAR(s_free), s_ph, abort, p);
          if (!ok) break;
          tc_fence_after();
          scores(left == 1);
          ahead(left == 1);
        }
        ok = wait_warp(BAR(ds_full) + 8 * buf.s, buf.ph, abort, p) &&
             (acc != 0 || sums_free || wait_warp(BAR(acc_free), acc_ph, abort, p));
        if (!ok) break;
        tc_fence_after();
        mma_over_tokens<T, DP, COLS, WT>(tmem + DQ_COL, tmem + DP_COL + buf.s * WT,
                                         desc_tokens<WT>(sb + S::A_OFF + ra.s * S::T), acc);
        commit_warp(BAR(a_empty) + 8 * ra.s);
        ra.next();
        buf.next();
      }
    }
    if (!ok) break;
    commit_warp(BAR(done));
    acc_ph ^= 1u;
  }
  if (*abort != 0) {
    // the products in flight end by themselves: a millisecond for them
    if ((threadIdx.x & 31) == 0) {
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 1000000ull) {
      }
    }
  }
  __syncwarp();
}

// --------------------------------------------- probabilities and outputs
template <typename T, int DP>
struct Calc {
  using S = Smem<DP>;
  static constexpr int WT = S::WT;
  const AttnParams& p;
  uint8_t* smem;
  uint32_t bb, tmem, lanes;
  volatile int* abort;
  int quad, part, c0, lane;
  Ring<S::RB> rb;
  Ring<2> buf;
  uint32_t s_ph = 0, k_ph = 0, done_ph = 0;

  // dk and dv.  A warp has 32 keys (TMEM rows) by 32 queries; thread t of it
  // the keys t / 4 + 8 k, k = 0 .. 3, and the queries 8 j + 2 (t % 4) + {0,
  // 1}, j = 0 .. 3.  Value (k, j, e) is v[16 (k / 2) + 4 j + 2 (k % 2) + e].
  // The queries' statistics are columns here: with one row a thread every
  // thread read all of them, and shared memory's bandwidth, which the
  // products need, bound the step.
  __device__ __forceinline__ bool dkv_steps(const Item& t) {
    constexpr uint32_t ROWS16 = 16u << 16;         // the warp's second 16 TMEM rows
    const int j = t.own + quad * 32 + (lane >> 2); // the first of this thread's keys
    const int c1 = c0 + 2 * (lane & 3);            // and queries of a tile
    const float c = p.scale * LOG2E;
    const F2 cc = f2_make(c, c);
    const int off = t.w.nk - t.w.nq;
    const uint32_t s_at = tmem + lanes + c0, dp_at = tmem + lanes + WT + c0;
    int q0 = t.r.first * WT;
    const int q_end = (t.r.first + t.r.count) * WT;
    for (int i = 0; i < t.n; ++i) {
      const float* st = reinterpret_cast<const float*>(smem + S::STAT_OFF + rb.s * S::STAT) + c1;
      // queries q0 .. q0 + WT - 1 against keys own .. own + 127: does everyone see everything?
      const bool mask =
          p.causal && (t.own + TILE - 1 > q0 + off || (p.window > 0 && q0 + WT - 1 + off - t.own >= p.window));
      float v[COLS], d[COLS];
      uint32_t r16[COLS / 2];
      if (!wait_warp(BAR(b_full) + 8 * rb.s, rb.ph, abort, p) || !wait_warp(BAR(s_full), s_ph, abort, p)) return false;
      s_ph ^= 1u;
      tc_fence_after();
      tmem_ld_16x32(s_at, v);
      tmem_ld_16x32(s_at + ROWS16, v + 16);
      float2 e[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) e[q] = *reinterpret_cast<const float2*>(st + 8 * q);
      tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float* u = v + 16 * (k >> 1) + 4 * q + 2 * (k & 1);
          const float2 x = f2_split(f2_fma(f2_make(u[0], u[1]), cc, f2_make(e[q].x, e[q].y)));
          u[0] = exp2_fast(x.x);
          u[1] = exp2_fast(x.y);
        }
      }
      if (mask) {
        // the queries (columns) that see key j + 8 k: [lo, hi)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int lo = j + 8 * k - off - q0 - c1, hi = p.window > 0 ? lo + p.window : WT;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float* u = v + 16 * (k >> 1) + 4 * q + 2 * (k & 1);
            if (8 * q < lo || 8 * q >= hi) u[0] = 0.f;
            if (8 * q + 1 < lo || 8 * q + 1 >= hi) u[1] = 0.f;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < COLS / 2; ++k) r16[k] = pack2<T>(v[2 * k], v[2 * k + 1]);
      tmem_st_16x16(s_at, r16);
      tmem_st_16x16(s_at + ROWS16, r16 + 8);
      tmem_st_wait();
      warp_arrive(BAR(p_full));
      if (!wait_warp(BAR(dpk_full), k_ph, abort, p)) return false;
      k_ph ^= 1u;
      tc_fence_after();
      tmem_ld_16x32(dp_at, d);
      tmem_ld_16x32(dp_at + ROWS16, d + 16);
#pragma unroll
      for (int q = 0; q < 4; ++q) e[q] = *reinterpret_cast<const float2*>(st + WT + 8 * q);
      tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < COLS; k += 2) {
        const int q = (k >> 2) & 3;
        const float2 x =
            f2_split(f2_mul(f2_make(v[k], v[k + 1]), f2_add(f2_make(d[k], d[k + 1]), f2_make(e[q].x, e[q].y))));
        r16[k >> 1] = pack2<T>(x.x, x.y);
      }
      tmem_st_16x16(dp_at, r16);
      tmem_st_16x16(dp_at + ROWS16, r16 + 8);
      tmem_st_wait();
      warp_arrive(BAR(dsk_full));
      rb.next();
      q0 += WT;
      if (q0 == q_end) q0 = t.r.first * WT;        // the group's next head
    }
    return true;
  }

  // dq: one query a thread, 32 keys of it
  __device__ __forceinline__ bool dq_steps(const Item& t, int qtiles) {
    const int q = t.own + quad * 32 + lane;
    const float c = p.scale * LOG2E;
    const int off = t.w.nk - t.w.nq;
    const long long at =
        ((static_cast<long long>(t.w.b) * p.heads + t.w.h) * qtiles + t.w.qtile + t.w.tile) * TILE + quad * 32 + lane;
    pdl_wait();                                    // the statistics are the previous kernel's
    const float lse = p.stat_lse[at], delta = p.stat_delta[at];
    const F2 cc = f2_make(c, c), ll = f2_make(lse, lse), dd = f2_make(delta, delta);
    for (int j0 = t.r.first * WT; j0 < (t.r.first + t.r.count) * WT; j0 += WT) {
      const bool mask =
          j0 + WT > t.w.nk ||
          (p.causal && (j0 + WT - 1 > t.own + off || (p.window > 0 && t.own + TILE - 1 + off - j0 >= p.window)));
      float v[COLS], d[COLS];
      if (!wait_warp(BAR(s_full), s_ph, abort, p)) return false;
      s_ph ^= 1u;
      tc_fence_after();
      tmem_ld32(tmem + lanes + c0, v);
      tmem_ld_wait();
      warp_arrive(BAR(s_free));
#pragma unroll
      for (int k = 0; k < COLS; k += 2) {
        const float2 a = f2_split(f2_fma(f2_make(v[k], v[k + 1]), cc, ll));
        v[k] = exp2_fast(a.x);
        v[k + 1] = exp2_fast(a.y);
      }
      if (mask) {
        // keys (columns) [lo, hi) are seen by query q
        int lo = 0, hi = t.w.nk - j0 - c0;
        if (p.causal) {
          hi = min(hi, q + off + 1 - j0 - c0);
          if (p.window > 0) lo = q + off - p.window + 1 - j0 - c0;
        }
#pragma unroll
        for (int k = 0; k < COLS; ++k)
          if (k < lo || k >= hi) v[k] = 0.f;
      }
      if (!wait_warp(BAR(dp_full) + 8 * buf.s, buf.ph, abort, p)) return false;
      tc_fence_after();
      const uint32_t dp = tmem + lanes + WT + buf.s * WT + c0;
      tmem_ld32(dp, d);
      tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < COLS; k += 2) {
        const float2 x = f2_split(f2_mul(f2_make(v[k], v[k + 1]), f2_add(f2_make(d[k], d[k + 1]), dd)));
        v[k] = x.x;
        v[k + 1] = x.y;
      }
      store_rounded<T, COLS / 2>(dp, v);
      warp_arrive(BAR(ds_full) + 8 * buf.s);
      buf.next();
    }
    return true;
  }

  // The sums of an item, 64 columns a warp (dk, dv) or 32 (dq), to memory.
  __device__ __forceinline__ bool outputs(const Item& t) {
    const Work& w = t.w;
    const int first = t.own + quad * 32;
    T* out;
    long long stride;
    int col, rows;
    uint32_t at;
    float mul = p.scale;
    if (t.dkv) {
      // dv by the first half of the warps, dk by the others
      const bool is_dv = part < Shape<DP>::PARTS / 2;
      col = part % (Shape<DP>::PARTS / 2) * 64;
      stride = is_dv ? p.dvs : p.dks;
      out = is_dv ? static_cast<T*>(p.dv) + w.b * p.dvb + w.h * p.dvh : static_cast<T*>(p.dk) + w.b * p.dkb + w.h * p.dkh;
      out += (w.k0 + first) * stride + col;
      rows = w.nk - first;
      at = tmem + lanes + 2 * WT + (is_dv ? 0 : DP) + col;
      if (is_dv) mul = 1.f;
    } else {
      col = c0;
      stride = p.dqs;
      out = static_cast<T*>(p.dq) + w.b * p.dqb + w.h * p.dqh + (w.q0 + first) * stride + col;
      rows = w.nq - first;
      at = tmem + lanes + 3 * WT + col;
    }
    if (t.n == 0) {
      const int width = t.dkv ? 64 : COLS;
      if (lane < rows)
        for (int k = 0; k < width && col + k < p.dim; k += 8)
          *reinterpret_cast<uint4*>(out + lane * stride + k) = make_uint4(0u, 0u, 0u, 0u);
      return true;
    }
    if (!wait_warp(BAR(done), done_ph, abort, p)) return false;
    done_ph ^= 1u;
    tc_fence_after();
    store_rows<T>(at, out, stride, rows, p.dim - col, mul);
    if (t.dkv) store_rows<T>(at + 32, out + 32, stride, rows, p.dim - col - 32, mul);
    warp_arrive(BAR(acc_free));
    return true;
  }
};

// Items [0, nk) are key tiles (dk, dv), the rest query tiles (dq), each kind
// from its longest to its shortest.  CTAs stay on their SMs and take item after
// item: an item's tiles are loaded, and its first products formed, while the
// previous one ends.  (A CTA an item spent 5 us on start, first loads and
// outputs, beside about 1.2 us a step.)
template <typename T, int DP>
__global__ void __launch_bounds__(Shape<DP>::THREADS, Shape<DP>::CTAS)
    attn_bwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo,
                    const AttnParams p, uint32_t nk, uint32_t total, int ktiles, int qtiles) {
  using S = Smem<DP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* bar = reinterpret_cast<Bars*>(smem + S::BAR_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sb = smem_u32(smem), bb = sb + S::BAR_OFF;
  if (!swizzle_aligned(sb, p)) return;
  const Grid g{&mq, &mk, &mv, &mdo, nk, total, ktiles, qtiles};
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&mq);
    tma_prefetch_map(&mk);
    tma_prefetch_map(&mv);
    tma_prefetch_map(&mdo);
    init_bars(bar, Shape<DP>::CALC);
  }
  if (warp == 1) tmem_alloc(&bar->tmem, Shape<DP>::TMEM);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem;
  if (warp == 0) {
    load_role<T, DP>(p, g, sb, bb, bar);
  } else if (warp == 1) {
    product_role<T, DP>(p, g, sb, bb, tmem, bar);
  } else {
    const int quad = warp & 3, part = (warp - CTRL_WARPS) >> 2;
    Calc<T, DP> calc{p, smem, bb, tmem, static_cast<uint32_t>(quad * 32) << 16, &bar->abort, quad, part, COLS * part, lane};
    Items items;
    for (uint32_t id; items.next(bb, bar, g, &bar->abort, p, &id);) {
      const Item t = find_item<S::WT>(p, g, id);
      if (!t.w.ok) continue;
      const bool ok = t.n == 0 || (t.dkv ? calc.dkv_steps(t) : calc.dq_steps(t, qtiles));
      if (!ok || !calc.outputs(t)) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, Shape<DP>::TMEM);
}

template <typename T, int DP>
cudaError_t launch_dims(const AttnParams& p, const CUtensorMap* m, bool prep, int sms, cudaStream_t s) {
  const bool packed = p.cu_q != nullptr;
  const long long seqs = packed ? 1 : p.batch;
  const long long qt = p.qtiles, kt = tile_bound(p.sk, TILE, p.batch, packed);
  const long long nq = p.sq > 0 ? qt * p.heads * seqs : 0, nk = p.sk > 0 ? kt * p.kv_heads * seqs : 0;
  if (nq + nk > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  if (prep) {
    attn_prep_kernel<T, DP><<<static_cast<unsigned>(nq), 256, 0, s>>>(p, static_cast<int>(qt));
    return cudaGetLastError();
  }
  auto kern = attn_bwd_kernel<T, DP>;
  static std::atomic<unsigned long long> done;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), Smem<DP>::BYTES, done);
  if (e != cudaSuccess) return e;
  const long long slots = static_cast<long long>(sms) * Shape<DP>::CTAS;
  const unsigned grid = static_cast<unsigned>(nq + nk < slots ? nq + nk : slots);
  // its prologue overlaps the statistics kernel (the wait for them is in the roles); without that one, no overlap
  e = launch_k(p.sq > 0, kern, dim3(grid), dim3(Shape<DP>::THREADS), Smem<DP>::BYTES, s, m[0], m[1], m[2], m[3], p,
               static_cast<uint32_t>(nk), static_cast<uint32_t>(nq + nk), static_cast<int>(kt), static_cast<int>(qt));
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const AttnParams& p, const CUtensorMap* m, bool prep, int sms, cudaStream_t s) {
  return p.dim <= 64 ? launch_dims<T, 64>(p, m, prep, sms, s) : launch_dims<T, 128>(p, m, prep, sms, s);
}

}  // namespace

cudaError_t launch_attn_bwd(const AttnParams& p, const CUtensorMap* m, bool prep, int sms, cudaStream_t s) {
  return p.dtype == DT_BF16 ? launch_type<__nv_bfloat16>(p, m, prep, sms, s)
                            : launch_type<__half>(p, m, prep, sms, s);
}

}  // namespace muon
