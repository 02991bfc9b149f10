// The backward pass of attention, recomputing the probabilities.
//
//   p_ij = exp(scale q_i . k_j - lse_i),  delta_i = do_i . o_i
//   dv_j = sum_i p_ij do_i,   ds_ij = p_ij (do_i . v_j - delta_i)
//   dq_i = scale sum_j ds_ij k_j,   dk_j = scale sum_i ds_ij q_i
//
// attn_prep_kernel writes -lse_i log2(e) and -delta_i, tile by tile (HBM-bound:
// it reads o and do).  fp16: the first 14 above, the second 2^-14 as large, so
// that p comes out lifted by 2^14 and ds as it is (see op_attn.cuh).  attn_bwd_kernel has two kinds of items.  One owns a
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
// 8192 causal tokens of 32 heads (8 of keys), bf16: 1.08 ms, 1270 TFLOP/s of
// the five products that the gradient needs, 1780 of the seven (this kernel
// alone; a call takes 1.11 ms, and 1.20 to 1.24 where calls follow one another
// under the power limit).  With short sequences and dim 64 the way of a tile
// through the element-wise warps binds: 8 x 1024 causal tokens of 12 heads take
// 66 us (a call 75), 490 TFLOP/s of five, with 51% of the issue slots and 36%
// of the tensor pipe used.  (p and ds of
// a tile in one go, with half the barriers, took 11% longer: no product then
// runs beside them.)
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
// that two-wide additions want; lifted and lowered), padded: rows past the sequence and rows that
// see no key get -inf, so that their p is 0.  8192 tokens of 32 heads of 128:
// 31 us, 4.3 TB/s.
constexpr int PREP = 512;                         // threads
template <typename T, int DP>
__global__ void __launch_bounds__(PREP) attn_prep_kernel(const AttnParams p, int tiles) {
  constexpr int LPR = DP / 8;                     // lanes of a row, 16 bytes each
  constexpr int N = TILE * LPR / PREP;            // rows of a thread
  pdl_launch_dependents();
  const Work w = find_work(p, true, TILE, p.heads, tiles, blockIdx.x);
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
    const int i = r0 + k * (PREP / LPR);
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
      const int i = r0 + k * (PREP / LPR);
      p.stat_lse[at + i] = e[k] == -INFINITY ? -INFINITY : fmaf(-e[k], LOG2E, static_cast<float>(lift_backward<T>()));
      p.stat_delta[at + i] = -s * lowered(lift_backward<T>());
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
  static constexpr int STAT = 2 * TILE * 4;       // lse and delta of a walked query tile, or of the one that stays
  static constexpr int A_OFF = 2 * OWN;
  static constexpr int B_OFF = A_OFF + RA * T;
  static constexpr int STAT_OFF = B_OFF + RB * T;
  static constexpr int BAR_OFF = STAT_OFF + RB * STAT;
  static constexpr int BYTES = BAR_OFF + 448;
  static_assert(BYTES * Shape<DP>::CTAS <= 232448 - 1024 * (Shape<DP>::CTAS - 1), "shared memory");
};

// One item.  The loading warp finds it and announces it: where it lies costs
// several divisions and, with packed sequences, a walk through their offsets,
// 1200 cycles that no other warp spends.
enum Kind : int { DQ = 0, DKV = 1, NO_MORE = 2 };
struct Item {
  int kind;
  int n;                     // steps
  int start;                 // walked row of the first of them
  int parts;                 // a walk in parts, each an item: SUM_ADD: not the first, SUM_KEEP: not the last
  int own;                   // first row of the tile that stays, in its sequence
  int rows;                  // rows from there to the sequence's end
  int first, last;           // walked rows: whole tiles, those of a head
  int nk, off;               // keys of the sequence; the position of query 0 among them
  void* out[2];              // that first row of dq, or of dv and dk
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
  uint64_t dv_done, done, acc_free;   // an item's dv formed; all its sums; read
  uint64_t edge[2];
  uint64_t stat[2];                   // dq: statistics of an item's queries, by turns
  uint64_t item_full[2], item_empty[2];
  Item item[2];                       // announced by the loading warp
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Bars) <= 448, "barrier block");
// shared-memory address of a barrier; `bb` is the block's
#define BAR(f) (bb + static_cast<uint32_t>(offsetof(Bars, f)))

__device__ __forceinline__ void init_bars(Bars* s, int calc_warps) {
  for (int i = 0; i < 2; ++i) {
    mbar_init(&s->own[i], 1);
    mbar_init(&s->own_empty[i], 1);
    mbar_init(&s->dp_full[i], 1);
    mbar_init(&s->ds_full[i], calc_warps);
    mbar_init(&s->edge[i], 1);
    mbar_init(&s->stat[i], 1);
    mbar_init(&s->item_full[i], 1);
    mbar_init(&s->item_empty[i], 1 + calc_warps);
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
  mbar_init(&s->dv_done, 1);
  mbar_init(&s->done, 1);
  mbar_init(&s->acc_free, calc_warps);
  s->abort = 0;
  fence_mbar_init();
}

// The loading warp's view of the launch.
struct Grid {
  const CUtensorMap *mq, *mk, *mv, *mdo;
  uint32_t nk, total;        // items of dk and dv, and all
  int ktiles, qtiles;
};

// The announced items, for another warp of the CTA: next() waits for one,
// free() gives its place back.
struct Items {
  uint32_t bb;
  const Bars* bar;
  Ring<2> at;
  __device__ __forceinline__ const Item* next(volatile int* abort, const AttnParams& p) {
    if (!wait_warp(BAR(item_full) + 8 * at.s, at.ph, abort, p)) return nullptr;
    const Item* t = &bar->item[at.s];
    return t->kind == NO_MORE ? nullptr : t;
  }
  __device__ __forceinline__ void free() {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive_at(BAR(item_empty) + 8 * at.s);
    at.next();
  }
};

// ----------------------------------------------------------------- loads
template <typename T, int DP, bool PARTS>
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
  Ring<2> items, stats;
  uint32_t id = blockIdx.x, next_id = 0;
  bool ok = true, waited = false;
  auto wait_stats = [&]() {                                  // statistics and counter are the previous kernel's
    if (!waited) pdl_wait();
    waited = true;
  };
  auto take = [&]() {
    wait_stats();
    if (lane == 0) next_id = p.counter != nullptr ? gridDim.x + atomicAdd(p.counter, 1u) : id + gridDim.x;
  };
  const int group = p.heads / p.kv_heads;
  PackedIndex index;
  if (p.cu_q != nullptr) index.fill(p, TILE);
  for (;; id = __shfl_sync(0xffffffffu, next_id, 0)) {
    Item t;
    Work w{};
    int steps = 0;
    const bool end = id >= g.total, dkv = id < g.nk;
    t.kind = end ? NO_MORE : dkv ? DKV : DQ;
    if (!end) {
      w = find_work(p, !dkv, TILE, dkv ? p.kv_heads : p.heads, dkv ? g.ktiles : g.qtiles, dkv ? id : id - g.nk,
                    &index);
      if (!w.ok) {
        take();
        continue;
      }
      t.own = w.tile * TILE;
      t.rows = (dkv ? w.nk : w.nq) - t.own;
      const Range r = dkv ? query_tiles<WT>(p, w, t.own, min(t.own + TILE, w.nk) - 1)
                          : key_tiles<WT>(p, w, t.own, min(t.own + TILE, w.nq) - 1);
      steps = r.count * (dkv ? group : 1);
      t.first = r.first * WT;
      t.last = (r.first + r.count) * WT;
      t.nk = w.nk;
      t.off = w.nk - w.nq;
      const long long k0 = w.k0 + t.own, q0 = w.q0 + t.own;
      t.out[0] = dkv ? static_cast<T*>(p.dv) + w.b * p.dvb + w.h * p.dvh + k0 * p.dvs
                     : static_cast<T*>(p.dq) + w.b * p.dqb + w.h * p.dqh + q0 * p.dqs;
      t.out[1] = static_cast<T*>(p.dk) + w.b * p.dkb + w.h * p.dkh + k0 * p.dks;
    }
    // dk, dv: K and V stay, Q and dO are walked; dq: Q and dO stay, K and V are walked
    const CUtensorMap* own0 = dkv ? g.mk : g.mq;
    const CUtensorMap* own1 = dkv ? g.mv : g.mdo;
    const CUtensorMap* walk_a = dkv ? g.mq : g.mk;
    const CUtensorMap* walk_b = dkv ? g.mdo : g.mv;
    const int own_row = (dkv ? w.k0 : w.q0) + t.own;
    const int first = dkv ? w.q0 : w.k0, len = dkv ? w.nq : w.nk;
    int h = dkv ? w.h * group : w.h / group, i0 = t.first;
    for (int done = 0; ok;) {                                // the walk's parts, mostly one
      t.n = PARTS ? min(steps - done, SUM_ROWS<T> / WT) : steps;
      t.start = i0;
      t.parts = (done > 0 ? SUM_ADD : 0) | (done + t.n < steps ? SUM_KEEP : 0);
      ok = wait_warp(BAR(item_empty) + 8 * items.s, items.ph ^ 1u, abort, p);
      if (!ok) break;
      if (lane == 0) {
        bar->item[items.s] = t;
        mbar_arrive_at(BAR(item_full) + 8 * items.s);
      }
      items.next();
      if (end) break;
      if (steps == 0) {
        take();
        break;
      }
      ok = wait_warp(BAR(own_empty), own_ph, abort, p);
      if (!ok) break;
      if (lane == 0) {
        mbar_expect_at(BAR(own), S::OWN);
        load_tile<DP, TILE, BOX>(sb, own0, BAR(own), w.h, own_row, w.b);
      }
      for (int k = 0; k < t.n; ++k) {
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
        if (k == 0) {                                        // the other own tile, after what the first scores want
          ok = wait_warp(BAR(own_empty) + 8, own_ph, abort, p);
          if (!ok) break;
          if (lane == 0) {
            mbar_expect_at(BAR(own) + 8, S::OWN);
            load_tile<DP, TILE, BOX>(sb + S::OWN, own1, BAR(own) + 8, w.h, own_row, w.b);
          }
          if (done == 0) take();
        }
        ok = wait_warp(BAR(b_empty) + 8 * rb.s, rb.ph ^ 1u, abort, p);
        if (!ok) break;
        if (lane == 0) {
          const uint32_t to = edge ? BAR(edge) + 8 : fb;
          const uint32_t st = sb + S::STAT_OFF + rb.s * S::STAT;
          // statistics: of each walked tile, or of the one that stays, with the first walked tile
          const long long stat = ((static_cast<long long>(w.b) * p.heads + (dkv ? h : w.h)) * g.qtiles + w.qtile) * TILE;
          mbar_expect_at(to, S::T + (dkv ? 2 * WT * 4 : 0));
          load_tile<DP, WT, BOX>(bt, walk_b, to, h, row, w.b);
          if (dkv) {
            bulk_load(st, p.stat_lse + stat + i0, WT * 4, to);
            bulk_load(st + TILE * 4, p.stat_delta + stat + i0, WT * 4, to);
          } else if (k == 0) {
            // a barrier of their own: the walked tiles get further ahead of the warps that read these
            const uint32_t bs = BAR(stat) + 8 * stats.s;
            mbar_expect_at(bs, 2 * TILE * 4);
            bulk_load(st, p.stat_lse + stat + t.own, TILE * 4, bs);
            bulk_load(st + TILE * 4, p.stat_delta + stat + t.own, TILE * 4, bs);
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
        i0 += WT;
        if (i0 == t.last) {                                  // on to the group's next head
          i0 = t.first;
          ++h;
        }
      }
      own_ph ^= 1u;
      if (!dkv) stats.next();
      done += t.n;
      if (!PARTS || done == steps) break;
    }
    if (!ok || end) break;
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
__device__ __forceinline__ void product_role(const AttnParams& p, uint32_t sb, uint32_t bb, uint32_t tmem, Bars* bar) {
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
  Items items{bb, bar, {}};
  while (ok) {
    const Item* t = items.next(abort, p);
    if (t == nullptr) break;
    const int n = t->n;
    const bool dkv = t->kind == DKV;
    items.free();
    if (n == 0) continue;
    // an item's first products go ahead of the previous item's outputs; its
    // sums wait for them.  From dk, dv to dq the places differ: wait at once.
    bool sums_free = false;
    if (!dkv && was_dkv) {
      ok = wait_warp(BAR(acc_free), acc_ph, abort, p);
      sums_free = true;
    }
    was_dkv = dkv;
    ok = ok && wait_warp(BAR(own), own_ph, abort, p) && wait_a();
    if (!ok) break;
    tc_fence_after();
    scores(n == 1);
    ok = wait_warp(BAR(own) + 8, own_ph, abort, p) && wait_b();
    if (!ok) break;
    own_ph ^= 1u;
    tc_fence_after();
    uint32_t acc = 0;
    if (dkv) {
      dprobs(DP_COL, BAR(dpk_full), n == 1);
      nb.next();
      for (int left = n - 1; left >= 0; --left, k_ph ^= 1u, acc = 1) {
        // a step's tiles are waited for before the probabilities, so that
        // products follow one another without a wait in between
        ok = (left == 0 || wait_a()) && wait_warp(BAR(p_full), k_ph, abort, p) &&
             (acc != 0 || wait_warp(BAR(acc_free), acc_ph, abort, p));
        if (!ok) break;
        tc_fence_after();
        mma_over_tokens<T, DP, COLS, WT>(tmem + DV_COL, tmem + S_COL, desc_tokens<WT>(sb + S::B_OFF + rb.s * S::T), acc);
        commit_warp(BAR(b_empty) + 8 * rb.s);      // dP, issued earlier, has read this dO tile too
        if (left == 0) commit_warp(BAR(dv_done));
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
      ahead(n == 1);
      for (int left = n - 1; left >= 0; --left, s_ph ^= 1u, acc = 1) {
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
template <typename T, int DP, bool PARTS>
struct Calc {
  using S = Smem<DP>;
  static constexpr int WT = S::WT;
  const AttnParams& p;
  uint8_t* smem;
  uint32_t bb, tmem, lanes;
  volatile int* abort;
  int quad, part, c0, lane;
  Ring<S::RB> rb;
  Ring<2> buf, stats;
  uint32_t s_ph = 0, k_ph = 0, dv_ph = 0, done_ph = 0;

  // dP - delta (of two), lowered as far as p is lifted
  static __device__ __forceinline__ F2 dp_less_delta(float a, float b, F2 delta) {
    if constexpr (lift_backward<T>() == 0) return f2_add(f2_make(a, b), delta);
    constexpr float k = lowered(lift_backward<T>());
    return f2_fma(f2_make(a, b), f2_make(k, k), delta);
  }

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
    const int n = t.n, own = t.own, off = t.off, first = t.first, last = t.last;
    const uint32_t s_at = tmem + lanes + c0, dp_at = tmem + lanes + WT + c0;
    int q0 = t.start;
    for (int i = 0; i < n; ++i) {
      const float* st = reinterpret_cast<const float*>(smem + S::STAT_OFF + rb.s * S::STAT) + c1;
      // queries q0 .. q0 + WT - 1 against keys own .. own + 127: does everyone see everything?
      const bool mask = p.causal && (own + TILE - 1 > q0 + off || (p.window > 0 && q0 + WT - 1 + off - own >= p.window));
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
          const int lo = j + 8 * k - off - q0 - c1;
          const uint32_t m = bits32(lo, p.window > 0 ? lo + p.window : COLS);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float* u = v + 16 * (k >> 1) + 4 * q + 2 * (k & 1);
            if (!(m & (1u << (8 * q)))) u[0] = 0.f;
            if (!(m & (2u << (8 * q)))) u[1] = 0.f;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < COLS / 2; ++k) r16[k] = pack2<T>(v[2 * k], v[2 * k + 1]);
      tmem_st_16x16(s_at, r16);
      tmem_st_16x16(s_at + ROWS16, r16 + 8);
      // delta now: once dv has read its tiles, the place of the statistics is filled again
#pragma unroll
      for (int q = 0; q < 4; ++q) e[q] = *reinterpret_cast<const float2*>(st + TILE + 8 * q);
      tmem_st_wait();
      warp_arrive(BAR(p_full));
      if (!wait_warp(BAR(dpk_full), k_ph, abort, p)) return false;
      k_ph ^= 1u;
      tc_fence_after();
      tmem_ld_16x32(dp_at, d);
      tmem_ld_16x32(dp_at + ROWS16, d + 16);
      tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < COLS; k += 2) {
        const int q = (k >> 2) & 3;
        const float2 x = f2_split(f2_mul(f2_make(v[k], v[k + 1]), dp_less_delta(d[k], d[k + 1], f2_make(e[q].x, e[q].y))));
        r16[k >> 1] = pack2<T>(x.x, x.y);
      }
      tmem_st_16x16(dp_at, r16);
      tmem_st_16x16(dp_at + ROWS16, r16 + 8);
      tmem_st_wait();
      warp_arrive(BAR(dsk_full));
      rb.next();
      q0 += WT;
      if (q0 == last) q0 = first;                  // the group's next head
    }
    return true;
  }

  // dq: one query a thread, 32 keys of it
  __device__ __forceinline__ bool dq_steps(const Item& t) {
    const float c = p.scale * LOG2E;
    const int own = t.own, off = t.off, nk = t.nk, first = t.start, last = t.start + t.n * WT;
    const int q = own + quad * 32 + lane;
    // the statistics came with the first walked tile; nothing is loaded over
    // them before every warp has let its first scores go
    if (!wait_warp(BAR(stat) + 8 * stats.s, stats.ph, abort, p)) return false;
    stats.next();
    const float* st = reinterpret_cast<const float*>(smem + S::STAT_OFF + rb.s * S::STAT) + quad * 32 + lane;
    const float lse = st[0], delta = st[TILE];
    const F2 cc = f2_make(c, c), ll = f2_make(lse, lse), dd = f2_make(delta, delta);
    for (int j0 = first; j0 < last; j0 += WT) {
      const bool mask = j0 + WT > nk || (p.causal && (j0 + WT - 1 > own + off ||
                                                      (p.window > 0 && own + TILE - 1 + off - j0 >= p.window)));
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
        int lo = 0, hi = nk - j0 - c0;
        if (p.causal) {
          hi = min(hi, q + off + 1 - j0 - c0);
          if (p.window > 0) lo = q + off - p.window + 1 - j0 - c0;
        }
        const uint32_t m = bits32(lo, hi);
#pragma unroll
        for (int k = 0; k < COLS; ++k)
          if (!(m & (1u << k))) v[k] = 0.f;
      }
      if (!wait_warp(BAR(dp_full) + 8 * buf.s, buf.ph, abort, p)) return false;
      tc_fence_after();
      const uint32_t dp = tmem + lanes + WT + buf.s * WT + c0;
      tmem_ld32(dp, d);
      tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < COLS; k += 2) {
        const float2 x = f2_split(f2_mul(f2_make(v[k], v[k + 1]), dp_less_delta(d[k], d[k + 1], dd)));
        v[k] = x.x;
        v[k + 1] = x.y;
      }
      store_rounded<T, COLS / 2>(dp, v);
      warp_arrive(BAR(ds_full) + 8 * buf.s);
      buf.next();
      rb.next();
    }
    return true;
  }

  // The sums of an item, 64 columns a warp (dk, dv) or 32 (dq), to memory; of a
  // part of a walk, added up in the CTA's scratch.
  // dv goes while dk's last product runs.
  __device__ __forceinline__ bool outputs(const Item& t) {
    constexpr int HALF = Shape<DP>::PARTS / 2;     // dv by the first half of the warps, dk by the others
    const bool dkv = t.kind == DKV, is_dk = part >= HALF, is_dv = dkv && !is_dk;
    const int width = dkv ? 64 : COLS, col = dkv ? part % HALF * 64 : c0, rows = t.rows - quad * 32;
    const long long stride = dkv ? (is_dk ? p.dks : p.dvs) : p.dqs;
    T* out = static_cast<T*>(t.out[dkv && is_dk]) + quad * 32 * stride + col;
    if (t.n == 0) {
      if (lane < rows)
        for (int k = 0; k < width && col + k < p.dim; k += 8)
          *reinterpret_cast<uint4*>(out + lane * stride + k) = make_uint4(0u, 0u, 0u, 0u);
      return true;
    }
    if (!wait_warp(is_dv ? BAR(dv_done) : BAR(done), is_dv ? dv_ph : done_ph, abort, p)) return false;
    done_ph ^= 1u;
    if (dkv) dv_ph ^= 1u;
    tc_fence_after();
    const uint32_t at = tmem + lanes + (dkv ? 2 * WT + (is_dk ? DP : 0) : 3 * WT) + col;
    float* sums = p.part + static_cast<long long>(blockIdx.x) * (2 * TILE * DP) + ((part * 4 + quad) * 64) * 32;
    const float m = is_dv ? lowered(lift_backward<T>()) : p.scale, mul[4] = {m, m, m, m};
#pragma unroll 1
    for (int k = 0; k < width; k += 32)
      store_rows<T, PARTS>(at + k, out + k, stride, rows, p.dim - col - k, mul, t.parts, sums + 32 * k);
    warp_arrive(BAR(acc_free));
    return true;
  }
};

// Items [0, nk) are key tiles (dk, dv), the rest query tiles (dq), each kind
// from its longest to its shortest.  CTAs stay on their SMs and take item after
// item: an item's tiles are loaded, and its first products formed, while the
// previous one ends.  (A CTA an item spent 5 us on start, first loads and
// outputs, beside about 1.2 us a step.)
template <typename T, int DP, bool PARTS>
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
    load_role<T, DP, PARTS>(p, g, sb, bb, bar);
  } else if (warp == 1) {
    product_role<T, DP>(p, sb, bb, tmem, bar);
  } else {
    const int quad = warp & 3, part = (warp - CTRL_WARPS) >> 2;
    Calc<T, DP, PARTS> calc{p, smem, bb, tmem, static_cast<uint32_t>(quad * 32) << 16, &bar->abort, quad, part, COLS * part, lane};
    Items items{bb, bar, {}};
    while (const Item* t = items.next(&bar->abort, p)) {
      const bool ok = t->n == 0 || (t->kind == DKV ? calc.dkv_steps(*t) : calc.dq_steps(*t));
      if (!ok || !calc.outputs(*t)) break;
      items.free();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, Shape<DP>::TMEM);
}

template <typename T, int DP, bool PARTS>
cudaError_t launch_items(const AttnParams& p, const CUtensorMap* m, unsigned grid, long long nk, long long total,
                         long long ktiles, long long qtiles, cudaStream_t s) {
  auto kern = attn_bwd_kernel<T, DP, PARTS>;
  static std::atomic<unsigned long long> done;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), Smem<DP>::BYTES, done);
  if (e != cudaSuccess) return e;
  // its prologue overlaps the statistics kernel (the wait for them is in the roles); without that one, no overlap
  e = launch_k(p.sq > 0 && pdl_level() >= 1, kern, dim3(grid), dim3(Shape<DP>::THREADS), Smem<DP>::BYTES, s, m[0], m[1], m[2], m[3], p,
               static_cast<uint32_t>(nk), static_cast<uint32_t>(total), static_cast<int>(ktiles), static_cast<int>(qtiles));
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int DP>
cudaError_t launch_dims(const AttnParams& p, const CUtensorMap* m, bool prep, int sms, cudaStream_t s) {
  const bool packed = p.cu_q != nullptr;
  const long long seqs = packed ? 1 : p.batch;
  const long long qt = p.qtiles, kt = tile_bound(p.sk, TILE, p.batch, packed);
  const long long nq = p.sq > 0 ? qt * p.heads * seqs : 0, nk = p.sk > 0 ? kt * p.kv_heads * seqs : 0;
  if (nq + nk > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  if (prep) {
    attn_prep_kernel<T, DP><<<static_cast<unsigned>(nq), PREP, 0, s>>>(p, static_cast<int>(qt));
    return cudaGetLastError();
  }
  const long long slots = static_cast<long long>(sms) * Shape<DP>::CTAS;
  const unsigned grid = static_cast<unsigned>(nq + nk < slots ? nq + nk : slots);
  return p.part != nullptr ? launch_items<T, DP, true>(p, m, grid, nk, nq + nk, kt, qt, s)
                           : launch_items<T, DP, false>(p, m, grid, nk, nq + nk, kt, qt, s);
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
