// The backward pass of attention, recomputing the probabilities.
//
//   p_ij = exp(scale q_i . k_j - lse_i),  delta_i = do_i . o_i
//   dv_j = sum_i p_ij do_i,   ds_ij = p_ij (do_i . v_j - delta_i)
//   dq_i = scale sum_j ds_ij k_j,   dk_j = scale sum_i ds_ij q_i
//
// attn_prep_kernel writes lse_i log2(e) and delta_i, tile by tile (HBM-bound:
// it reads o and do).  attn_bwd_kernel has two kinds of items.  One owns a
// tile of 128 keys, walks the query tiles that see them (of every query head
// that shares the key head) and keeps dk and dv in TMEM; the other owns a
// tile of 128 queries, walks its key tiles and keeps dq in TMEM.  No value is added
// by atomics, so results do not change from call to call; the price is that
// scores and dP are formed twice, seven products a tile pair instead of five.
//
// Both are bound by the tensor cores and the exponentials: per tile pair of
// 128 x 128 with dim 128 the products take 1024 (768) cycles of the tensor
// pipe at its full rate.  Warp-specialised: warp 0 loads tiles by TMA,
// warp 1 issues every tcgen05.mma, the other warps turn
// scores into p and ds.  p and ds never leave the SM: each warp writes its 16
// bit values over the fp32 scores (or dP) that it read, and the next product
// takes them from TMEM as its A operand.  Scores are transposed in the dkv
// kernel (rows are keys), so that p and ds are that operand as they stand.
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
  static constexpr int BYTES = BAR_OFF + 256;
  static_assert(BYTES * Shape<DP>::CTAS <= 232448 - 1024 * (Shape<DP>::CTAS - 1), "shared memory");
};

struct Bars {
  uint64_t own[2];          // the two tiles that stay
  uint64_t a_full[3], a_empty[3];
  uint64_t b_full[3], b_empty[3];
  uint64_t s_full, s_free;  // scores: written, and read into registers
  uint64_t p_full;
  uint64_t dp_full[2], ds_full[2];
  uint64_t done, edge;
  uint32_t tmem;
  int abort;
  Work work;
};
static_assert(sizeof(Bars) <= 256, "barrier block");
// shared-memory address of a barrier; `bb` is the block's
#define BAR(f) (bb + static_cast<uint32_t>(offsetof(Bars, f)))

__device__ __forceinline__ void init_bars(Bars* s, int calc_warps) {
  for (int i = 0; i < 2; ++i) {
    mbar_init(&s->own[i], 1);
    mbar_init(&s->dp_full[i], 1);
    mbar_init(&s->ds_full[i], calc_warps);
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
  mbar_init(&s->done, 1);
  mbar_init(&s->edge, 1);
  s->abort = 0;
  fence_mbar_init();
}

// ------------------------------------------------------------- dk and dv
// A warp has 32 keys (TMEM rows) by 32 queries; thread t of it the keys t / 4
// + 8 k, k = 0 .. 3, and the queries 8 j + 2 (t % 4) + {0, 1}, j = 0 .. 3.
// Value (k, j, e) is v[16 (k / 2) + 4 j + 2 (k % 2) + e].  The queries'
// statistics are columns here: with one row a thread every thread read all of
// them, and shared memory's bandwidth, which the products need, bound the
// step (2970 cycles with dim 128 against 2048 of products).
template <typename T, int DP>
__device__ __forceinline__ void dkv_item(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                                         const CUtensorMap& mdo, const AttnParams& p, int tiles, int qtiles,
                                         uint32_t item) {
  using S = Smem<DP>;
  constexpr int WT = S::WT, BOX = DP == 64 ? 64 : TILE;      // rows of a walked tile, of a map's box
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* bar = reinterpret_cast<Bars*>(smem + S::BAR_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sb = smem_u32(smem), bb = sb + S::BAR_OFF;
  if (!swizzle_aligned(sb, p)) return;
  if (warp == 0) {
    const Work w = find_work(p, false, TILE, p.kv_heads, tiles, item);
    if (lane == 0) {
      bar->work = w;
      init_bars(bar, Shape<DP>::CALC);
    }
  }
  if (warp == 1) tmem_alloc(&bar->tmem, Shape<DP>::TMEM);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Work w = bar->work;
  volatile int* abort = &bar->abort;
  const uint32_t tmem = bar->tmem;
  constexpr uint32_t S_COL = 0, DP_COL = WT, DV_COL = 2 * WT, DK_COL = 2 * WT + DP;
  const int group = p.heads / p.kv_heads;
  const int j0 = w.tile * TILE;
  Range r{0, 0};
  if (w.ok) r = query_tiles<WT>(p, w, j0, min(j0 + TILE, w.nk) - 1);
  const int n = r.count * group;                   // steps: the group's heads one after another

  if (warp == 0 && n > 0) {
    // ---------------------------------------------------------- loads
    if (lane == 0) {
      mbar_expect_at(BAR(own), S::OWN);
      load_tile<DP, TILE, BOX>(sb, &mk, BAR(own), w.h, w.k0 + j0, w.b);
    }
    bool first = true;
    uint32_t edges = 0;
    int ia = 0, ib = 0;
    Ring<S::RA> ra;
    Ring<S::RB> rb;
    bool ok = true;
    for (int hq = w.h * group; ok && hq < (w.h + 1) * group; ++hq) {
      const long long stat = ((static_cast<long long>(w.b) * p.heads + hq) * qtiles + w.qtile) * TILE;
      for (int i0 = r.first * WT; i0 < (r.first + r.count) * WT; i0 += WT) {
        const int row = w.q0 + i0, valid = w.nq - i0;
        const bool edge = p.cu_q != nullptr && valid < WT;
        const uint32_t at = sb + S::A_OFF + ra.s * S::T, bt = sb + S::B_OFF + rb.s * S::T;
        const uint32_t fa = BAR(a_full) + 8 * ra.s, fb = BAR(b_full) + 8 * rb.s;
        ok = wait_warp(BAR(a_empty) + 8 * ra.s, ra.ph ^ 1u, abort, p);
        if (!ok) break;
        if (edge) {
          ok = load_edge_tile<DP, WT, BOX>(at, &mq, BAR(edge), edges, hq, row, valid, abort, p);
          if (!ok) break;
          if (lane == 0) mbar_arrive_at(fa);
        } else if (lane == 0) {
          mbar_expect_at(fa, S::T);
          load_tile<DP, WT, BOX>(at, &mq, fa, hq, row, w.b);
        }
        ++ia;
        ra.next();
        if (first) {                               // after what the first scores want
          first = false;
          if (lane == 0) {
            mbar_expect_at(BAR(own) + 8, S::OWN);
            load_tile<DP, TILE, BOX>(sb + S::OWN, &mv, BAR(own) + 8, w.h, w.k0 + j0, w.b);
          }
          pdl_wait();                              // the statistics are the previous kernel's
        }
        ok = wait_warp(BAR(b_empty) + 8 * rb.s, rb.ph ^ 1u, abort, p);
        if (!ok) break;
        if (edge) {
          ok = load_edge_tile<DP, WT, BOX>(bt, &mdo, BAR(edge), edges, hq, row, valid, abort, p);
          if (!ok) break;
        }
        if (lane == 0) {
          const uint32_t st = sb + S::STAT_OFF + rb.s * S::STAT;
          mbar_expect_at(fb, S::STAT + (edge ? 0 : S::T));
          bulk_load(st, p.stat_lse + stat + i0, WT * 4, fb);
          bulk_load(st + WT * 4, p.stat_delta + stat + i0, WT * 4, fb);
          if (!edge) load_tile<DP, WT, BOX>(bt, &mdo, fb, hq, row, w.b);
        }
        ++ib;
        rb.next();
      }
    }
    if (*abort != 0 && lane == 0) {
      mbar_wait_bounded(&bar->own[0], 0, nullptr, DRAIN_NS);
      if (!first) mbar_wait_bounded(&bar->own[1], 0, nullptr, DRAIN_NS);
      drain_ring<S::RA>(bar->a_full, ia);
      drain_ring<S::RB>(bar->b_full, ib);
    }
    __syncwarp();
  } else if (warp == 1 && n > 0) {
    // -------------------------------------------------------- products
    const uint64_t k_d = desc_dim(sb), v_d = desc_dim(sb + S::OWN);
    Ring<S::RA> ra, na;                            // this step's Q tile, and the next one's
    Ring<S::RB> rb, nb;
    auto scores = [&]() {
      mma_over_dim<T, DP, WT>(tmem + S_COL, k_d, desc_dim(sb + S::A_OFF + na.s * S::T));
      commit_warp(BAR(s_full));
      na.next();
    };
    auto dprobs = [&]() {
      mma_over_dim<T, DP, WT>(tmem + DP_COL, v_d, desc_dim(sb + S::B_OFF + nb.s * S::T));
      commit_warp(BAR(dp_full));
      nb.next();
    };
    // a step's tiles are waited for before the probabilities, so that
    // products follow one another without a wait in between
    auto wait_a = [&]() { return wait_warp(BAR(a_full) + 8 * na.s, na.ph, abort, p); };
    auto wait_b = [&]() { return wait_warp(BAR(b_full) + 8 * nb.s, nb.ph, abort, p); };
    bool ok = wait_warp(BAR(own), 0, abort, p) && wait_a();
    if (ok) {
      tc_fence_after();
      scores();
      ok = wait_warp(BAR(own) + 8, 0, abort, p) && wait_b();
    }
    if (ok) {
      tc_fence_after();
      dprobs();
    }
    uint32_t ph = 0, acc = 0;
    for (int left = n - 1; ok && left >= 0; --left, ph ^= 1u, acc = 1) {
      ok = (left == 0 || wait_a()) && wait_warp(BAR(p_full), ph, abort, p);
      if (!ok) break;
      tc_fence_after();
      mma_over_tokens<T, DP, COLS, WT>(tmem + DV_COL, tmem + S_COL, desc_tokens<WT>(sb + S::B_OFF + rb.s * S::T), acc);
      commit_warp(BAR(b_empty) + 8 * rb.s);        // dP, issued earlier, has read this dO tile too
      rb.next();
      // the next scores overwrite the probabilities: the tensor pipe runs in order
      if (left > 0) scores();
      ok = (left == 0 || wait_b()) && wait_warp(BAR(ds_full), ph, abort, p);
      if (!ok) break;
      tc_fence_after();
      mma_over_tokens<T, DP, COLS, WT>(tmem + DK_COL, tmem + DP_COL, desc_tokens<WT>(sb + S::A_OFF + ra.s * S::T), acc);
      commit_warp(BAR(a_empty) + 8 * ra.s);
      ra.next();
      if (left > 0) dprobs();
    }
    commit_warp(BAR(done));
    if (!ok && lane == 0) mbar_wait_bounded(&bar->done, 0, nullptr, DRAIN_NS);
    __syncwarp();
  } else if (warp >= CTRL_WARPS && w.ok) {
    // --------------------------------------- probabilities, then outputs
    const int quad = warp & 3, part = (warp - CTRL_WARPS) >> 2, c0 = COLS * part;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const int j = j0 + quad * 32 + (lane >> 2);    // the first of this thread's keys
    const int c1 = c0 + 2 * (lane & 3);            // and queries of a tile
    const float c = p.scale * LOG2E;
    const F2 cc = f2_make(c, c);
    const int off = w.nk - w.nq;
    const uint32_t s_at = tmem + lanes + S_COL + c0, dp_at = tmem + lanes + DP_COL + c0;
    constexpr uint32_t ROWS16 = 16u << 16;         // the warp's second 16 TMEM rows
    Ring<S::RB> rb;
    uint32_t ph = 0;
    bool ok = true;
    int q0 = r.first * WT;
    const int q_end = (r.first + r.count) * WT;
    for (int i = 0; i < n; ++i) {
      const float* st = reinterpret_cast<const float*>(smem + S::STAT_OFF + rb.s * S::STAT) + c1;
      // queries q0 .. q0 + WT - 1 against keys j0 .. j0 + 127: does everyone see everything?
      const bool mask = p.causal && (j0 + TILE - 1 > q0 + off || (p.window > 0 && q0 + WT - 1 + off - j0 >= p.window));
      float v[COLS], d[COLS];
      uint32_t r16[COLS / 2];
      ok = wait_warp(BAR(b_full) + 8 * rb.s, rb.ph, abort, p) && wait_warp(BAR(s_full), ph, abort, p);
      if (!ok) break;
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
      ok = wait_warp(BAR(dp_full), ph, abort, p);
      if (!ok) break;
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
      warp_arrive(BAR(ds_full));
      rb.next();
      ph ^= 1u;
      q0 += WT;
      if (q0 == q_end) q0 = r.first * WT;          // the group's next head
    }
    if (ok && n > 0) {
      ok = wait_warp(BAR(done), 0, abort, p);
      tc_fence_after();
    }
    if (ok) {
      // dv by the first half of the warps, dk by the others, 64 columns a warp,
      // through K's and V's places in shared memory
      const bool is_dv = part < Shape<DP>::PARTS / 2;
      const int x = part % (Shape<DP>::PARTS / 2), first = j0 + quad * 32;
      const long long stride = is_dv ? p.dvs : p.dks, t = w.k0 + first;
      T* out = (is_dv ? static_cast<T*>(p.dv) + w.b * p.dvb + w.h * p.dvh : static_cast<T*>(p.dk) + w.b * p.dkb + w.h * p.dkh) +
               t * stride + 64 * x;
      if (n > 0) {
        store_block<T, 64>(tmem + lanes + (is_dv ? DV_COL : DK_COL) + 64 * x,
                           sb + (is_dv ? S::OWN : 0) + x * BOX_BYTES, quad * 32, 0, out, stride, w.nk - first,
                           p.dim - 64 * x, is_dv ? 1.f : p.scale);
      } else if (first + lane < w.nk) {
        for (int k = 0; k < 64 && 64 * x + k < p.dim; k += 8)
          *reinterpret_cast<uint4*>(out + lane * stride + k) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, Shape<DP>::TMEM);
}

// -------------------------------------------------------------------- dq
template <typename T, int DP>
__device__ __forceinline__ void dq_item(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                                        const CUtensorMap& mdo, const AttnParams& p, int tiles, uint32_t item) {
  using S = Smem<DP>;
  constexpr int WT = S::WT, BOX = DP == 64 ? 64 : TILE;      // rows of a walked tile, of a map's box
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* bar = reinterpret_cast<Bars*>(smem + S::BAR_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sb = smem_u32(smem), bb = sb + S::BAR_OFF;
  if (!swizzle_aligned(sb, p)) return;
  if (warp == 0) {
    const Work w = find_work(p, true, TILE, p.heads, tiles, item);
    if (lane == 0) {
      bar->work = w;
      init_bars(bar, Shape<DP>::CALC);
    }
  }
  if (warp == 1) tmem_alloc(&bar->tmem, Shape<DP>::TMEM);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Work w = bar->work;
  volatile int* abort = &bar->abort;
  const uint32_t tmem = bar->tmem;
  // dP is kept twice, so that the next tile's products need not wait for this tile's ds
  constexpr uint32_t S_COL = 0, DP_COL = WT, DQ_COL = 3 * WT;
  const int hk = w.h / (p.heads / p.kv_heads);
  const int i0 = w.tile * TILE;
  Range r{0, 0};
  if (w.ok) r = key_tiles<WT>(p, w, i0, min(i0 + TILE, w.nq) - 1);
  const int n = r.count;

  if (warp == 0 && n > 0) {
    // ---------------------------------------------------------- loads
    if (lane == 0) {
      mbar_expect_at(BAR(own), S::OWN);
      load_tile<DP, TILE, BOX>(sb, &mq, BAR(own), w.h, w.q0 + i0, w.b);
    }
    bool first = true;
    uint32_t edges = 0;
    int ia = 0, ib = 0;
    Ring<S::RA> ra;
    Ring<S::RB> rb;
    for (int j = r.first * WT; j < (r.first + r.count) * WT; j += WT) {
      const int row = w.k0 + j, valid = w.nk - j;
      const bool edge = p.cu_q != nullptr && valid < WT;
      const uint32_t at = sb + S::A_OFF + ra.s * S::T, bt = sb + S::B_OFF + rb.s * S::T;
      const uint32_t fa = BAR(a_full) + 8 * ra.s, fb = BAR(b_full) + 8 * rb.s;
      if (!wait_warp(BAR(a_empty) + 8 * ra.s, ra.ph ^ 1u, abort, p)) break;
      if (edge) {
        if (!load_edge_tile<DP, WT, BOX>(at, &mk, BAR(edge), edges, hk, row, valid, abort, p)) break;
        if (lane == 0) mbar_arrive_at(fa);
      } else if (lane == 0) {
        mbar_expect_at(fa, S::T);
        load_tile<DP, WT, BOX>(at, &mk, fa, hk, row, w.b);
      }
      ++ia;
      ra.next();
      if (first) {                                 // after what the first scores want
        first = false;
        if (lane == 0) {
          mbar_expect_at(BAR(own) + 8, S::OWN);
          load_tile<DP, TILE, BOX>(sb + S::OWN, &mdo, BAR(own) + 8, w.h, w.q0 + i0, w.b);
        }
      }
      if (!wait_warp(BAR(b_empty) + 8 * rb.s, rb.ph ^ 1u, abort, p)) break;
      if (edge) {
        if (!load_edge_tile<DP, WT, BOX>(bt, &mv, BAR(edge), edges, hk, row, valid, abort, p)) break;
        if (lane == 0) mbar_arrive_at(fb);
      } else if (lane == 0) {
        mbar_expect_at(fb, S::T);
        load_tile<DP, WT, BOX>(bt, &mv, fb, hk, row, w.b);
      }
      ++ib;
      rb.next();
    }
    if (*abort != 0 && lane == 0) {
      mbar_wait_bounded(&bar->own[0], 0, nullptr, DRAIN_NS);
      if (!first) mbar_wait_bounded(&bar->own[1], 0, nullptr, DRAIN_NS);
      drain_ring<S::RA>(bar->a_full, ia);
      drain_ring<S::RB>(bar->b_full, ib);
    }
    __syncwarp();
  } else if (warp == 1 && n > 0) {
    // -------------------------------------------------------- products
    const uint64_t q_d = desc_dim(sb), do_d = desc_dim(sb + S::OWN);
    Ring<S::RA> ra, na;                            // this step's K tile, and the next one's
    Ring<S::RB> nb;
    Ring<2> buf, next;                             // the two places of dP
    auto scores = [&]() {
      mma_over_dim<T, DP, WT>(tmem + S_COL, q_d, desc_dim(sb + S::A_OFF + na.s * S::T));
      commit_warp(BAR(s_full));
      na.next();
    };
    auto dprobs = [&]() {
      mma_over_dim<T, DP, WT>(tmem + DP_COL + next.s * WT, do_d, desc_dim(sb + S::B_OFF + nb.s * S::T));
      commit_warp(BAR(dp_full) + 8 * next.s);
      commit_warp(BAR(b_empty) + 8 * nb.s);
      nb.next();
      next.next();
    };
    auto wait_a = [&]() { return wait_warp(BAR(a_full) + 8 * na.s, na.ph, abort, p); };
    auto wait_b = [&]() { return wait_warp(BAR(b_full) + 8 * nb.s, nb.ph, abort, p); };
    bool ok = wait_warp(BAR(own), 0, abort, p) && wait_a();
    if (ok) {
      tc_fence_after();
      scores();
      ok = wait_warp(BAR(own) + 8, 0, abort, p) && wait_b();
    }
    if (ok) {
      tc_fence_after();
      dprobs();
    }
    uint32_t ph = 0, acc = 0;
    for (int left = n - 1; ok && left >= 0; --left, ph ^= 1u, acc = 1) {
      // the next tile's scores and dP (over the ds before last, which dq has read: the tensor pipe runs in order)
      if (left > 0) {
        ok = wait_a() && wait_b() && wait_warp(BAR(s_free), ph, abort, p);
        if (!ok) break;
        tc_fence_after();
        scores();
        dprobs();
      }
      ok = wait_warp(BAR(ds_full) + 8 * buf.s, buf.ph, abort, p);
      if (!ok) break;
      tc_fence_after();
      mma_over_tokens<T, DP, COLS, WT>(tmem + DQ_COL, tmem + DP_COL + buf.s * WT,
                                       desc_tokens<WT>(sb + S::A_OFF + ra.s * S::T), acc);
      commit_warp(BAR(a_empty) + 8 * ra.s);
      ra.next();
      buf.next();
    }
    commit_warp(BAR(done));
    if (!ok && lane == 0) mbar_wait_bounded(&bar->done, 0, nullptr, DRAIN_NS);
    __syncwarp();
  } else if (warp >= CTRL_WARPS && w.ok) {
    // --------------------------------------- probabilities, then outputs
    const int quad = warp & 3, part = (warp - CTRL_WARPS) >> 2, c0 = COLS * part;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const int q = i0 + quad * 32 + lane;           // this thread's query
    const float c = p.scale * LOG2E;
    const int off = w.nk - w.nq;
    const long long at = ((static_cast<long long>(w.b) * p.heads + w.h) * tiles + w.qtile + w.tile) * TILE + quad * 32 + lane;
    pdl_wait();                                    // the statistics are the previous kernel's
    const float lse = n > 0 ? p.stat_lse[at] : 0.f, delta = n > 0 ? p.stat_delta[at] : 0.f;
    const F2 cc = f2_make(c, c), ll = f2_make(lse, lse), dd = f2_make(delta, delta);
    Ring<2> buf;
    uint32_t ph = 0;
    bool ok = true;
    for (int j0 = r.first * WT; j0 < (r.first + r.count) * WT; j0 += WT) {
      const bool mask = j0 + WT > w.nk ||
                        (p.causal && (j0 + WT - 1 > i0 + off || (p.window > 0 && i0 + TILE - 1 + off - j0 >= p.window)));
      float v[COLS];
      ok = wait_warp(BAR(s_full), ph, abort, p);
      if (!ok) break;
      tc_fence_after();
      tmem_ld32(tmem + lanes + S_COL + c0, v);
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
        int lo = 0, hi = w.nk - j0 - c0;
        if (p.causal) {
          hi = min(hi, q + off + 1 - j0 - c0);
          if (p.window > 0) lo = q + off - p.window + 1 - j0 - c0;
        }
#pragma unroll
        for (int k = 0; k < COLS; ++k)
          if (k < lo || k >= hi) v[k] = 0.f;
      }
      ok = wait_warp(BAR(dp_full) + 8 * buf.s, buf.ph, abort, p);
      if (!ok) break;
      tc_fence_after();
      const uint32_t dp = tmem + lanes + DP_COL + buf.s * WT + c0;
      float d[COLS];
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
      ph ^= 1u;
    }
    if (ok && n > 0) {
      ok = wait_warp(BAR(done), 0, abort, p);
      tc_fence_after();
    }
    if (ok) {
      // 32 columns a warp, through Q's place in shared memory
      const int first = i0 + quad * 32;
      T* out = static_cast<T*>(p.dq) + w.b * p.dqb + static_cast<long long>(w.q0 + first) * p.dqs + w.h * p.dqh + c0;
      if (n > 0) {
        store_block<T, COLS>(tmem + lanes + DQ_COL + c0, sb + c0 / 64 * BOX_BYTES, quad * 32, c0 % 64 / 8, out, p.dqs,
                             w.nq - first, p.dim - c0, p.scale);
      } else if (q < w.nq) {
        for (int k = 0; k < COLS && c0 + k < p.dim; k += 8)
          *reinterpret_cast<uint4*>(out + lane * p.dqs + k) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, Shape<DP>::TMEM);
}

// Items [0, nk) are key tiles (dk, dv), the rest query tiles (dq): one launch,
// so that the short items of one kind fill the SMs beside the last long ones
// of the other.
template <typename T, int DP>
__global__ void __launch_bounds__(Shape<DP>::THREADS, Shape<DP>::CTAS)
    attn_bwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo,
                    const AttnParams p, uint32_t nk, int ktiles, int qtiles) {
  if (threadIdx.x < 32) {
    if ((threadIdx.x & 31) == 0) {
      tma_prefetch_map(&mq);
      tma_prefetch_map(&mk);
      tma_prefetch_map(&mv);
      tma_prefetch_map(&mdo);
    }
    __syncwarp();
  }
  if (blockIdx.x < nk)
    dkv_item<T, DP>(mq, mk, mv, mdo, p, ktiles, qtiles, blockIdx.x);
  else
    dq_item<T, DP>(mq, mk, mv, mdo, p, qtiles, blockIdx.x - nk);
}

template <typename T, int DP>
cudaError_t launch_dims(const AttnParams& p, const CUtensorMap* m, bool prep, cudaStream_t s) {
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
  // its prologue overlaps the statistics kernel (the wait for them is in the items); without that one, no overlap
  e = launch_k(p.sq > 0, kern, dim3(static_cast<unsigned>(nq + nk)), dim3(Shape<DP>::THREADS), Smem<DP>::BYTES, s, m[0],
               m[1], m[2], m[3], p, static_cast<uint32_t>(nk), static_cast<int>(kt), static_cast<int>(qt));
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const AttnParams& p, const CUtensorMap* m, bool prep, cudaStream_t s) {
  return p.dim <= 64 ? launch_dims<T, 64>(p, m, prep, s) : launch_dims<T, 128>(p, m, prep, s);
}

}  // namespace

cudaError_t launch_attn_bwd(const AttnParams& p, const CUtensorMap* m, bool prep, cudaStream_t s) {
  return p.dtype == DT_BF16 ? launch_type<__nv_bfloat16>(p, m, prep, s) : launch_type<__half>(p, m, prep, s);
}

}  // namespace muon
