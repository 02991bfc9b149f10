// Products of the linear layers of a mixture-of-experts model, whose tokens
// are grouped by expert, and products of 8-bit operands:
//   forward   y_t = W_e x_t            for the tokens t of expert e,
//   input     dx_t = W_e^T dy_t,
//   weight    dW_e = sum over e's tokens of dy_t x_t^T  (+ add),
//   8 bits    y_t = W x_t, codes times powers of two.
//
// All are one product on the tensor cores, D[m][n] = sum_k A[m][k] B[n][k],
// whose result is stored as rows n of consecutive m:
//              m (A)                n (B)              k
//   forward    outputs (W)          tokens (x)         columns
//   input      columns (W)          tokens (dy)        outputs
//   weight     columns (x)          outputs (dy)       tokens
//   8 bits     outputs (W's codes)  tokens (x's codes) columns
// A CTA pair forms 256 m (128 a CTA) by up to 256 n, 224 with 8 bits, whose scales
// need TMEM too (tcgen05.mma.cta_group::2), in one of two accumulators that tiles
// take in turn: one is read out while the other's products run.  (The parts of a
// tile's sum over more than 2048 tokens all go to one, so the products wait for each
// read-out: 8 experts of 6144 tokens 2048 x 1408 209 - 216 us.)  The ragged
// dimension, tokens, is n: the tensor core takes n in steps of 32, so an expert's
// last tile costs what it has, where rows of m would be padded to 256 (17% of the
// work at 768 tokens an expert).  (Tiles of twice the n in both accumulators, with a
// quarter less to shared memory, are finished half by half in turn: 64 experts of
// 768 rows, 1408 -> 2048 in 217 us against 205, 16384 x 4096 x 14336 in 8 bits in 644
// against 635.)
//
// Operands come by TMA with 128-byte swizzle, K-major or MN-major as they lie in
// memory, through a ring of 16 KB slots for each.  Eight epilogue warps
// turn 32 x 32 blocks around through shared memory (a lane holds one m), so that
// rows leave in whole sectors.
//
// The groups' offsets are device data: every CTA clamps them (to the token
// axis and the largest before them) and counts the tiles for itself.
//
// Measured, calls that follow one another: 49152 rows through 64 experts 2048 ->
// 1408 forward 213 - 222 us, input's gradient 200 - 207, weights' 217 - 225 (1.3 PFLOP/s,
// the pipe 81, 81 and 66% busy), all under the power cap at 1.3 to 1.6 GHz; 48 rows
// 37 - 38 us (214 MB at 5.7 TB/s); 16384 x 4096 -> 14336 in 8 bits 632 - 652 us by the
// box (3.0 PFLOP/s, the pipe 84% busy), 16 rows 13.3 (58.7 MB at 4.4 TB/s).  Within a tile a step's operands come
// from L2 at 52 to 60 bytes a cycle and SM, which bounds the weights' gradients.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "op_common.cuh"
#include "op_pair.cuh"

namespace muon {
namespace {

constexpr int MT = 256;                  // m of a pair's tile
constexpr int BOX = 64 * 128;            // 64 rows of 128 bytes
constexpr int STAGE = 2 * BOX;           // a step's part of an operand: 128 rows of 128 bytes, or 64 of 256
constexpr int SLOTS = 6;                 // steps of both operands in flight
constexpr int EPI_WARPS = 8, SLOT = 2048;
constexpr int STEPS_SUM = 32;            // weight: steps of 64 tokens an accumulator takes
constexpr int PART_WARP = 4 * 1024;      // floats of scratch of an epilogue warp
constexpr int B_OFF = SLOTS * STAGE;
constexpr int EPI_OFF = 2 * B_OFF;
constexpr int GROUP_OFF = EPI_OFF + EPI_WARPS * SLOT;
// 8 bits: the tokens' scales on their way, those of a tile for each of four blocks
constexpr int SB_SLOTS = 3, SB_ROW = 224, SB_SLOT = 4 * SB_ROW;
constexpr int SB_OFF = GROUP_OFF + 2 * 4 * (kMaxExperts + 4);
constexpr int BAR_OFF = SB_OFF + SB_SLOTS * SB_SLOT;
constexpr int SMEM = BAR_OFF + 512;
constexpr unsigned long long DRAIN_NS = 1000000000ull;
static_assert(SMEM <= 232448, "shared memory");

template <int KIND>
struct Traits {
  static constexpr bool kTokens = KIND != PRODUCT_WEIGHT;                   // n are tokens
  static constexpr bool kRagged = KIND == PRODUCT_FORWARD || KIND == PRODUCT_INPUT;   // of several experts
  static constexpr bool kAmn = KIND == PRODUCT_INPUT || KIND == PRODUCT_WEIGHT;   // A is read MN-major
  static constexpr bool kBmn = KIND == PRODUCT_WEIGHT;
  static constexpr bool k8 = KIND == PRODUCT_ACT8;
  static constexpr int BK = k8 ? 128 : 64;                                  // 128 bytes
  static constexpr int EPI_WARP0 = k8 ? 8 : 4;
  static constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
  // most n of an accumulator: two and, for 8 bits, the scales share 512 columns of TMEM
  static constexpr int NT = k8 ? 224 : 256;
};
// The scales in TMEM, by groups of four 128-column blocks: a 32-bit word a row
// of A (4 columns of 32 lanes) and of B (8), a byte for each block.
constexpr int SF_SLOTS = 3, SF_COLS = 12;
static_assert(2 * Traits<PRODUCT_ACT8>::NT + SF_SLOTS * SF_COLS <= 512, "TMEM");

struct alignas(16) Bars {
  uint64_t full[SLOTS];                  // the leader's, for both CTAs
  uint64_t empty[SLOTS];                 // each CTA's own
  uint64_t own[SLOTS];                   // weight: this CTA's part of an expert's last step
  uint64_t tfull[2], tempty[2];
  uint64_t sf_full[SF_SLOTS];            // 8 bits: the leader's, scales written by both CTAs
  uint64_t sf_empty[SF_SLOTS];
  uint64_t sb_full[SB_SLOTS], sb_empty[SB_SLOTS];   // 8 bits: each CTA's own, scales as they are in memory
  uint64_t drain;
  uint4 token[2];                        // sent, received (see send_token)
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Bars) <= 512 && SB_OFF % 16 == 0, "barrier block");

// n of the tiles that a row of `len` is cut into, at most `most`: as few tiles as
// there can be, of about one size (all but the last `most`, where that one is
// not small and they need not be even).
__host__ __device__ __forceinline__ int tile_n(int len, int most, bool even) {
  const int tiles = (len + most - 1) / most, rest = len % most;
  if (tiles <= 1) return most;
  if (!even && (rest == 0 || rest >= most / 2)) return most;
  return ((len + tiles - 1) / tiles + 31) / 32 * 32;
}

struct Tile {
  int e, m0, n0;       // group, first m, first n (of the token axis, or of the outputs)
  int n;               // that exist
  int t0, len;         // weight: first token and tokens of the group, or of its split
  int split;
  int steps;

  __device__ __forceinline__ int padded() const { return (n + 31) / 32 * 32; }       // the n that the product takes
};

// The tiles in order of their groups; a thread asks for rising numbers.  What does
// not hang on the offsets the host has worked out: a division takes 150 cycles, and
// a short call waits for the first tile's.
template <int KIND>
struct Tiles {
  const ProductParams& p;
  const int* at;       // [groups + 1] offsets
  const int* pre;      // [groups + 1] tiles before a group (ragged)
  int total, size, nt; // size, nt: n of a tile and such tiles, of group `of` where they are ragged
  int e = 0, of = -1;

  __device__ __forceinline__ Tiles(const ProductParams& q, const int* a)
      : p(q), at(a), pre(a + kMaxExperts + 4), total(Traits<KIND>::kRagged ? pre[q.groups] : q.total), size(q.size), nt(q.nt) {}
  // A group's tiles go eight m at a time: the pairs that run together share
  // panels of A and of B in L2.
  __device__ __forceinline__ void place(uint32_t in, Tile& t) const {
    const uint32_t band = in < 8u * nt ? 0u : in / (8u * nt), r = in - band * 8u * nt;
    const uint32_t rows = min(8u, static_cast<uint32_t>(p.mt) - band * 8u), j = rows == 8u ? r >> 3 : r / rows;
    t.m0 = static_cast<int>(band * 8u + r - j * rows) * MT;
    t.n0 = static_cast<int>(j) * size;
  }
  // (by way of shuffles: one tile for the warp)
  __device__ __forceinline__ Tile get(int i) {
    Tile t;
    if constexpr (KIND == PRODUCT_ACT8) {
      t.e = t.t0 = t.len = t.split = 0;
      place(i, t);
      t.n = min(size, p.tokens - t.n0);
      t.steps = (p.k + Traits<KIND>::BK - 1) / Traits<KIND>::BK;
    } else if constexpr (Traits<KIND>::kRagged) {
      while (pre[e + 1] <= i) ++e;
      if (e != of) {
        of = e;
        const int len = at[e + 1] - at[e];
        size = tile_n(len, p.most, true);
        nt = len <= size ? 1 : (len + size - 1) / size;
      }
      t.e = e;
      place(i - pre[e], t);
      t.n0 += at[e];
      t.n = min(size, at[e + 1] - t.n0);
      t.steps = (p.k + Traits<KIND>::BK - 1) / Traits<KIND>::BK;
      t.t0 = t.len = t.split = 0;
    } else {
      uint32_t u = static_cast<uint32_t>(i);
      t.split = 0;
      if (p.splits > 1) {                // splits of a tile are neighbours
        const uint32_t n = static_cast<uint32_t>(p.splits), v = u / n;
        t.split = static_cast<int>(u - v * n);
        u = v;
      }
      const uint32_t per = static_cast<uint32_t>(p.mt) * nt, g = p.groups == 1 ? 0u : u / per;
      t.e = static_cast<int>(g);
      place(u - g * per, t);
      t.n = min(size, p.n - t.n0);
      t.t0 = at[t.e];
      t.len = at[t.e + 1] - t.t0;
      t.steps = (t.len + Traits<KIND>::BK - 1) / Traits<KIND>::BK;
      if (p.splits > 1) {                // below 2^32: 2^24 steps, fewer splits than SMs
        const uint32_t steps = t.steps, k0 = steps * t.split / p.splits, k1 = steps * (t.split + 1) / p.splits;
        t.t0 += static_cast<int>(k0 * Traits<KIND>::BK);
        t.len = min(t.len, static_cast<int>(k1 * Traits<KIND>::BK)) - static_cast<int>(k0 * Traits<KIND>::BK);
        t.steps = static_cast<int>(k1 - k0);
      }
    }
    t.n = __shfl_sync(0xffffffffu, t.n, 0);
    t.m0 = __shfl_sync(0xffffffffu, t.m0, 0);
    t.n0 = __shfl_sync(0xffffffffu, t.n0, 0);
    t.e = __shfl_sync(0xffffffffu, t.e, 0);
    t.t0 = __shfl_sync(0xffffffffu, t.t0, 0);
    t.len = __shfl_sync(0xffffffffu, t.len, 0);
    t.split = __shfl_sync(0xffffffffu, t.split, 0);
    t.steps = __shfl_sync(0xffffffffu, t.steps, 0);
    return t;
  }
};

// Offsets and tile counts into shared memory; one warp.
template <int KIND>
__device__ __forceinline__ void count_tiles(const ProductParams& p, int* at) {
  int* pre = at + kMaxExperts + 4;
  const int lane = threadIdx.x & 31;
  int last = 0, tiles = 0;               // offset and tiles of the groups so far
  int ahead[4];                          // four at a time: one after the other they took 600 cycles each
  for (int d0 = 0; d0 <= p.groups; d0 += 32) {
    const int d = d0 + lane, turn = (d0 >> 5) & 3;
    if (turn == 0) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        ahead[q] = d + 32 * q <= p.groups ? p.offsets[d + 32 * q] : p.tokens;
    }
    int v = min(max(turn == 0 ? ahead[0] : turn == 1 ? ahead[1] : turn == 2 ? ahead[2] : ahead[3], 0), p.tokens);
    v = max(v, last);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = max(v, u);
    }
    int before = __shfl_up_sync(0xffffffffu, v, 1);
    if (lane == 0) before = d0 == 0 ? v : last;
    int c = 0;                           // tiles of group d - 1
    if constexpr (Traits<KIND>::kRagged) {
      const int len = v - before;
      if (len > 0) {
        const int size = tile_n(len, p.most, true);
        c = (len + size - 1) / size * p.mt;
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += u;
      }
    }
    if (d <= p.groups) {
      at[d] = v;
      pre[d] = tiles + c;
    }
    last = __shfl_sync(0xffffffffu, v, 31);
    tiles += __shfl_sync(0xffffffffu, c, 31);
  }
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// An arrival on a barrier of the pair that orders no memory, for what is done in
// TMEM and waited for there, a fence of the tensor core's before it.  (With a
// release it waited 950 cycles for the stores of the results before.  That of the
// scales waited for the weight's bytes that were asked for ahead: 16 x 4096 x
// 14336 18.3 us, 13.9 without.)
__device__ __forceinline__ void arrive_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Scales of a group of blocks to the 32 TMEM lanes of a warp.
__device__ __forceinline__ void tmem_st4(uint32_t taddr, uint32_t w) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %1, %1, %1};" ::"r"(taddr), "r"(w) : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* w) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The two halves of cluster_sync_all.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// What a whole warp issues, by one of its lanes: the lanes stay together, so that
// addresses and coordinates are kept in uniform registers, which these
// instructions take.  (Loops of a single lane took 550 cycles a step and more.)
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  asm volatile(
      "{\n"
      " .reg .pred q;\n"
      " elect.sync _|q, 0xffffffff;\n"
      " @q mbarrier.arrive.shared::cta.b64 _, [%0];\n"
      "}\n" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void warp_expect(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n"
      " .reg .pred q;\n"
      " elect.sync _|q, 0xffffffff;\n"
      " @q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n"
      "}\n" ::"r"(bar),
      "r"(bytes)
      : "memory");
}
// PAIR: `bar` is the leader's (a shared::cluster address), else this CTA's
template <bool PAIR>
__device__ __forceinline__ void warp_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  if constexpr (PAIR)
    asm volatile(
        "{\n"
        " .reg .pred q;\n"
        " elect.sync _|q, 0xffffffff;\n"
        " @q cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
        "%4}], [%5];\n"
        "}\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "{\n"
        " .reg .pred q;\n"
        " elect.sync _|q, 0xffffffff;\n"
        " @q cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n"
        "}\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
// Commits the products so far to a barrier of both CTAs.
__device__ __forceinline__ void warp_commit(uint32_t bar) {
  asm volatile(
      "{\n"
      " .reg .pred q;\n"
      " .reg .b16 m;\n"
      " elect.sync _|q, 0xffffffff;\n"
      " mov.b16 m, 3;\n"
      " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n"
      "}\n" ::"r"(bar)
      : "memory");
}

// A step's products of a pair, up to four of 32 bytes of k.  Descriptors by their
// low words (the high ones do not change); ADV: from one product's operands to
// the next, in their units of 16 bytes.
template <int ADV_A, int ADV_B, bool RAGGED>
__device__ __forceinline__ void mma_step(uint32_t d, uint32_t a, uint32_t ahi, uint32_t b, uint32_t bhi, uint32_t id,
                                         uint32_t acc, int count) {
  if constexpr (RAGGED) {
    asm volatile(
        "{\n"
        " .reg .pred p, q, t, q1, q2, q3;\n"
        " .reg .b64 a, b;\n"
        " elect.sync _|q, 0xffffffff;\n"
        " setp.ne.b32 p, %6, 0;\n"
        " setp.eq.b32 t, 0, 0;\n"
        " setp.gt.and.s32 q1, %7, 1, q;\n"
        " setp.gt.and.s32 q2, %7, 2, q;\n"
        " setp.gt.and.s32 q3, %7, 3, q;\n"
        " mov.b64 a, {%1, %2};\n"
        " mov.b64 b, {%3, %4};\n"
        " @q tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n"
        " add.s64 a, a, %8;\n"
        " add.s64 b, b, %9;\n"
        " @q1 tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, t;\n"
        " add.s64 a, a, %8;\n"
        " add.s64 b, b, %9;\n"
        " @q2 tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, t;\n"
        " add.s64 a, a, %8;\n"
        " add.s64 b, b, %9;\n"
        " @q3 tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, t;\n"
        "}\n" ::"r"(d),
        "r"(a), "r"(ahi), "r"(b), "r"(bhi), "r"(id), "r"(acc), "r"(count), "n"(ADV_A), "n"(ADV_B)
        : "memory");
  } else {
    asm volatile(
        "{\n"
        " .reg .pred p, q, t;\n"
        " .reg .b64 a, b;\n"
        " elect.sync _|q, 0xffffffff;\n"
        " setp.ne.b32 p, %6, 0;\n"
        " setp.eq.b32 t, 0, 0;\n"
        " mov.b64 a, {%1, %2};\n"
        " mov.b64 b, {%3, %4};\n"
        " @q tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n"
        " add.s64 a, a, %7;\n"
        " add.s64 b, b, %8;\n"
        " @q tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, t;\n"
        " add.s64 a, a, %7;\n"
        " add.s64 b, b, %8;\n"
        " @q tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, t;\n"
        " add.s64 a, a, %7;\n"
        " add.s64 b, b, %8;\n"
        " @q tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, t;\n"
        "}\n" ::"r"(d),
        "r"(a), "r"(ahi), "r"(b), "r"(bhi), "r"(id), "r"(acc), "n"(ADV_A), "n"(ADV_B)
        : "memory");
  }
}
// The same of e4m3 codes, with the scales in TMEM columns sa and sb, a power of
// two a row and 32 k.
__device__ __forceinline__ void mma_step_scaled(uint32_t d, uint32_t a, uint32_t ahi, uint32_t b, uint32_t bhi, uint32_t id,
                                                uint32_t sa, uint32_t sb, uint32_t acc) {
  asm volatile(
      "{\n"
      " .reg .pred p, q, t;\n"
      " .reg .b64 a, b;\n"
      " elect.sync _|q, 0xffffffff;\n"
      " setp.ne.b32 p, %8, 0;\n"
      " setp.eq.b32 t, 0, 0;\n"
      " mov.b64 a, {%1, %2};\n"
      " mov.b64 b, {%3, %4};\n"
      " @q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], a, b, %5, [%6], [%7], p;\n"
      " add.s64 a, a, 2;\n"
      " add.s64 b, b, 2;\n"
      " @q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], a, b, %5, [%6], [%7], t;\n"
      " add.s64 a, a, 2;\n"
      " add.s64 b, b, 2;\n"
      " @q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], a, b, %5, [%6], [%7], t;\n"
      " add.s64 a, a, 2;\n"
      " add.s64 b, b, 2;\n"
      " @q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], a, b, %5, [%6], [%7], t;\n"
      "}\n" ::"r"(d),
      "r"(a), "r"(ahi), "r"(b), "r"(bhi), "r"(id), "r"(sa), "r"(sb), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void store_any(void* base, long long i, int dtype, float v) {
  if (dtype == DT_F16)
    static_cast<__half*>(base)[i] = __float2half_rn(v);
  else
    store_from_f32(base, i, dtype, v);
}
__device__ __forceinline__ void load4(const void* base, long long i, int dtype, float* f) {
  if (dtype == DT_F32) {
    const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
  } else {
    const uint2 raw = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i);
    float2 a, b;
    if (dtype == DT_BF16) {
      a = unpack2(*reinterpret_cast<const __nv_bfloat162*>(&raw.x)), b = unpack2(*reinterpret_cast<const __nv_bfloat162*>(&raw.y));
    } else {
      a = unpack2(*reinterpret_cast<const __half2*>(&raw.x)), b = unpack2(*reinterpret_cast<const __half2*>(&raw.y));
    }
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
  }
}

// 32 m (TMEM lanes) x 32 n (columns) of results, spread over the warp in 8 x 8
// tiles as the matrix instructions' accumulators are, rounded to T, two n in a
// register: w[8 a + 2 j + b] of thread t is m = 16 a + 8 b + t / 4, n = 8 j + 2
// (t % 4) and the next.
template <typename T>
__device__ __forceinline__ void tmem_block(uint32_t taddr, uint32_t* w) {
  float v[2][16];
#pragma unroll
  for (int a = 0; a < 2; ++a)
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(v[a][0]), "=f"(v[a][1]), "=f"(v[a][2]), "=f"(v[a][3]), "=f"(v[a][4]), "=f"(v[a][5]), "=f"(v[a][6]),
          "=f"(v[a][7]), "=f"(v[a][8]), "=f"(v[a][9]), "=f"(v[a][10]), "=f"(v[a][11]), "=f"(v[a][12]), "=f"(v[a][13]),
          "=f"(v[a][14]), "=f"(v[a][15])
        : "r"(taddr + (static_cast<uint32_t>(16 * a) << 16)));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int j = 0; j < 8; ++j) w[8 * a + j] = pack2<T>(v[a][2 * j], v[a][2 * j + 1]);
}

// Such a block to `rows` rows (n) of 32 m at `to`: tiles are stored to shared
// memory transposed, rows of 64 bytes with their 16-byte parts swizzled.
__device__ __forceinline__ void store_packed(uint32_t slot, const uint32_t* w, uint16_t* to, long long ld, int rows, int lane) {
  __syncwarp();
  // w[8 a + 2 j + b]: the tile of m 16 a + 8 b .., n 8 j ..; a lane gives row
  // lane % 8 (n) of tile lane / 8 of the four that an instruction stores
  const int b = (lane >> 3) & 1, j = lane >> 4;
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = 16 * h + 8 * j + (lane & 7), part = 2 * a + b;
      asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                       slot + n * 64 + ((part ^ ((n >> 1) & 3)) << 4)),
                   "r"(w[8 * a + 4 * h]), "r"(w[8 * a + 4 * h + 1]), "r"(w[8 * a + 4 * h + 2]), "r"(w[8 * a + 4 * h + 3])
                   : "memory");
    }
  __syncwarp();
  const int r = lane >> 2, q = lane & 3;
  uint4 x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = lds16(slot + (r + 8 * i) * 64 + ((q ^ ((r >> 1) & 3)) << 4));
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (r + 8 * i < rows) *reinterpret_cast<uint4*>(to + (r + 8 * i) * ld + q * 8) = x[i];
}

// What is added to a block of 32 m by 32 n, from `add`: a lane has 4 m of every
// fourth row.
__device__ __forceinline__ void load_added(const ProductParams& p, long long add, int rows, int lane, float (*f)[4]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if ((lane >> 3) + 4 * i < rows) load4(p.add, add + ((lane >> 3) + 4 * i) * p.ldadd + (lane & 7) * 4, p.odtype, f[i]);
}

// The block in fp32, v[j] row j, to rows of 32 m from (out, add), of any type and
// place.  Rows past `rows` and m past `ms` are not there.  f: what is added, where
// rows are wide.
template <bool ADD>
__device__ __forceinline__ void store_block(const ProductParams& p, uint8_t* slot, const float* v, float (*f)[4], long long out,
                                            long long add, int rows, int ms, int lane) {
  if (!p.vec || ms < 32) {
    // a lane has one m: rows leave as they are, in 7200 cycles for 80 rows a warp
    // (13000 by way of shared memory, an element at a time)
    if (lane >= ms) return;
    auto rows_of_type = [&](auto type) {
      using O = decltype(type);
      O* to = static_cast<O*>(p.out) + out + lane;
      const O* more = static_cast<const O*>(p.add) + add + lane;
#pragma unroll
      for (int h = 0; h < 32; h += 8) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[j] = v[h + j];
          if (ADD && p.add != nullptr && h + j < rows) x[j] += to_f32(more[(h + j) * p.ldadd]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (h + j < rows) to[(h + j) * p.ldo] = from_f32<O>(x[j]);
      }
    };
    if (p.odtype == DT_F32)
      rows_of_type(0.f);
    else if (p.odtype == DT_BF16)
      rows_of_type(__nv_bfloat16{});
    else
      rows_of_type(__half{});
    return;
  }
  const uint32_t s = smem_u32(slot);
  __syncwarp();
  const int wr = lane >> 3, wq = lane & 7;
#pragma unroll
  for (int h = 0; h < 32; h += 16) {       // 16 rows at a time
    if (h > 0) __syncwarp();
#pragma unroll
    for (int j = 0; j < 16; ++j) asm volatile("st.shared.f32 [%0], %1;" ::"r"(s + j * 128 + lane * 4), "f"(v[h + j]) : "memory");
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = h + wr + 4 * i;
      if (r >= rows) break;
      const uint4 raw = lds16(s + (wr + 4 * i) * 128 + wq * 16);
      float4 x = make_float4(__uint_as_float(raw.x), __uint_as_float(raw.y), __uint_as_float(raw.z), __uint_as_float(raw.w));
      if (ADD && p.add != nullptr) x.x += f[h / 4 + i][0], x.y += f[h / 4 + i][1], x.z += f[h / 4 + i][2], x.w += f[h / 4 + i][3];
      const long long to = out + r * p.ldo + wq * 4;
      if (p.odtype == DT_F32)
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + to) = x;
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + to) =
            p.odtype == DT_BF16 ? make_uint2(pack2<__nv_bfloat16>(x.x, x.y), pack2<__nv_bfloat16>(x.z, x.w))
                                : make_uint2(pack2<__half>(x.x, x.y), pack2<__half>(x.z, x.w));
    }
  }
}

// Rows [from, to) of the result set to zero by warp `w` of `warps`.
__device__ __forceinline__ void zero_rows(const ProductParams& p, int from, int to, int w, int warps, int lane) {
  for (int r = from + w; r < to; r += warps) {
    uint16_t* row = static_cast<uint16_t*>(p.out) + r * p.ldo;
    if (p.vec) {
      for (int c = lane * 8; c < p.m; c += 256) *reinterpret_cast<uint4*>(row + c) = make_uint4(0u, 0u, 0u, 0u);
    } else {
      for (int c = lane; c < p.m; c += 32) row[c] = 0;
    }
  }
}

// An expert's last tokens, where the products take some that are not its own.
template <int KIND>
__device__ __forceinline__ bool mended(const Tile& t, int k) {
  return KIND == PRODUCT_WEIGHT && k == t.steps - 1 && (t.len & 15) != 0;
}
template <int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Traits<KIND>::THREADS, 1)
    product_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                   const __grid_constant__ CUtensorMap mb32, const ProductParams p) {
  using T = Traits<KIND>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* bar = reinterpret_cast<Bars*>(smem + BAR_OFF);
  int* at = reinterpret_cast<int*>(smem + GROUP_OFF);
  // (by way of a shuffle: known to be one for the warp, so that what follows from
  // it is kept in uniform registers)
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = static_cast<int>(cluster_id_x()), npairs = static_cast<int>(num_clusters_x());
  const uint32_t sb = smem_u32(smem);
  if (threadIdx.x == 0) {
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(&bar->full[s], KIND == PRODUCT_WEIGHT ? 2 : 1);
      mbar_init(&bar->empty[s], 1);
      mbar_init(&bar->own[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&bar->tfull[a], 1);
      mbar_init(&bar->tempty[a], 2 * EPI_WARPS);
    }
    for (int s = 0; s < SF_SLOTS; ++s) {
      mbar_init(&bar->sf_full[s], 8);
      mbar_init(&bar->sf_empty[s], 1);
    }
    for (int s = 0; s < SB_SLOTS; ++s) {
      mbar_init(&bar->sb_full[s], 1);
      mbar_init(&bar->sb_empty[s], 4);
    }
    mbar_init(&bar->drain, 1);
    bar->token[0] = make_uint4(0u, 0u, 0u, 0u);
    bar->abort = (sb & 1023u) != 0u ? 1 : 0;       // the swizzled boxes need 1 KB boundaries
    if (bar->abort) atomicOr(p.err, ERRBIT_TIMEOUT);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(&bar->tmem, 512);
  if (warp == 3 && lane == 0 && p.tokens > 0) {
    tma_prefetch_map(&ma);
    tma_prefetch_map(&mb);
    if (!T::kBmn) tma_prefetch_map(&mb32);
  }
  // the cluster's barrier passes while the kernel before is waited for (after it, it
  // held the first loads up by 1000 cycles)
  tc_fence_before();
  cluster_arrive();
  if (warp == 2) {
    // (what follows the CTA's barrier comes after this wait too)
    pdl_wait();
    if constexpr (KIND != PRODUCT_ACT8) count_tiles<KIND>(p, at);
  }
  pdl_launch_dependents();
  cluster_wait();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bar->tmem, 0);
  volatile int* abort = &bar->abort;
  Tiles<KIND> tiles(p, at);

  if (warp == 0 || warp == 3) {
    // -------------------------------------------------------------- loads
    // Warp 0 loads A and says what a step brings, warp 3 loads B, in few large
    // boxes.
    const uint32_t lead = mapa_shared(smem_u32(&bar->full[0]), 0), here = smem_u32(&bar->full[0]),
                   owns = smem_u32(&bar->own[0]);
    Ring<SLOTS> r;
    bool ok = true;
    for (int i = pair; ok && i < tiles.total; i += npairs) {
      const Tile t = tiles.get(i);
      // of B, this CTA's half, in boxes of 128 or 32 tokens, or of 64 outputs
      const int part = t.padded() / 2, n0 = t.n0 + static_cast<int>(rank) * part, m0 = t.m0 + static_cast<int>(rank) * 128;
      const uint32_t bytes = STAGE + static_cast<uint32_t>(T::kBmn     ? (part + 63) / 64 * BOX
                                                           : part > 64 ? 2 * BOX
                                                                       : (part + 31) / 32 * (BOX / 2));       // of a step
      auto load_b = [&](auto own, int k, uint32_t to, uint32_t fb) {
        constexpr bool PAIR = !decltype(own)::value;
        if constexpr (T::kBmn) {
          for (int c = 0; c < part; c += 64) warp_load<PAIR>(to + c * 128, &mb, fb, n0 + c, t.t0 + k * 64, 0);
        } else if (part > 64) {
          warp_load<PAIR>(to, &mb, fb, k * T::BK, n0, 0);
        } else {
          for (int c = 0; c < part; c += 32) warp_load<PAIR>(to + c * 128, &mb32, fb, k * T::BK, n0 + c, 0);
        }
      };
      auto load_a = [&](auto own, int k, uint32_t to, uint32_t fb) {
        constexpr bool PAIR = !decltype(own)::value;
        if constexpr (T::kAmn) {
          const int row = KIND == PRODUCT_WEIGHT ? t.t0 + k * 64 : k * 64, e = KIND == PRODUCT_WEIGHT ? 0 : t.e;
          warp_load<PAIR>(to, &ma, fb, m0, row, e);
          warp_load<PAIR>(to + BOX, &ma, fb, m0 + 64, row, e);
        } else {
          warp_load<PAIR>(to, &ma, fb, k * T::BK, m0, t.e);
        }
      };
      using Own = std::integral_constant<bool, true>;
      using Pair = std::integral_constant<bool, false>;
#pragma unroll 1
      for (int k = 0; k < t.steps; ++k) {
        // an expert's last tokens go to this CTA's own warp, which clears what
        // follows them (see below)
        const bool own = mended<KIND>(t, k);
        ok = wait_warp(&bar->empty[r.s], r.ph ^ 1u, abort, p);
        if (!ok) break;
        const uint32_t fb = lead + r.s * 8, ob = owns + r.s * 8, to = sb + r.s * STAGE;
        if (warp == 0) {
          if (own) warp_expect(ob, bytes);
          if (rank == 0) {
            // (the weight's barriers count two arrivals, one of them the clearing warp's)
            if (KIND == PRODUCT_WEIGHT && !own) warp_arrive(here + r.s * 8);
            warp_expect(here + r.s * 8, own ? static_cast<uint32_t>(sizeof(uint4)) : 2 * bytes);
          }
          if (own)
            load_a(Own{}, k, to, ob);
          else
            load_a(Pair{}, k, to, fb);
        } else {
          if (own)
            load_b(Own{}, k, to + B_OFF, ob);
          else
            load_b(Pair{}, k, to + B_OFF, fb);
        }
        r.next();
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // --------------------------------------------------------- products
      // 16 bits: fp32 results, operands bf16 or fp16.  8 bits: e4m3, scales 2^(byte - 127), the byte of a word at 4 (B)
      // and 29 (A)
      const uint32_t type = T::k8 ? 1u << 23 : (1u << 4) | (p.f16 ? 0u : (1u << 7) | (1u << 10));
      const uint32_t id0 = type | (T::kAmn ? 1u << 15 : 0u) | (T::kBmn ? 1u << 16 : 0u) | ((MT >> 4) << 24);
      Ring<SF_SLOTS> rs;
      Ring<SLOTS> r;
      const uint64_t a0 = T::kAmn ? sdesc_sw128(sb, BOX, 1024) : sdesc_sw128(sb, 16, 1024);
      const uint64_t b0 = T::kBmn ? sdesc_sw128(sb + B_OFF, BOX, 1024) : sdesc_sw128(sb + B_OFF, 16, 1024);
      const uint32_t alo = static_cast<uint32_t>(a0), ahi = static_cast<uint32_t>(a0 >> 32), blo = static_cast<uint32_t>(b0),
                     bhi = static_cast<uint32_t>(b0 >> 32), empty0 = smem_u32(&bar->empty[0]);
      int acc = 0;
      uint32_t ph = 0u;                  // the accumulators' phases, a bit each
      bool ok = true;
      for (int i = pair; ok && i < tiles.total; i += npairs) {
        const Tile t = tiles.get(i);
        const uint32_t id = id0 | (static_cast<uint32_t>(t.padded() >> 3) << 17), d = tmem + acc * T::NT;
        // Steps in runs that are alike: the part of a sum that an accumulator takes
        // (weight), a group of four blocks' scales (8 bits).
        constexpr int RUN = KIND == PRODUCT_WEIGHT ? STEPS_SUM : T::k8 ? 4 : 1 << 30;
        for (int k = 0; ok && k < t.steps;) {
          if (k == 0 || KIND == PRODUCT_WEIGHT) {
            ok = wait_warp<0, true>(&bar->tempty[acc], ((ph >> acc) & 1u) ^ 1u, abort, p);
            if (!ok) break;
            tc_fence_after();
          }
          if constexpr (T::k8) {
            ok = wait_warp<0, true>(&bar->sf_full[rs.s], rs.ph, abort, p);
            if (!ok) break;
            tc_fence_after();
          }
          const int end = min(t.steps, k + RUN);
#pragma unroll 1
          for (const int k0 = k; k < end; ++k) {
            ok = wait_warp<0, KIND == PRODUCT_WEIGHT>(&bar->full[r.s], r.ph, abort, p);
            if (!ok) break;
            const uint32_t a = alo + r.s * (STAGE >> 4), b = blo + r.s * (STAGE >> 4);
            // of 16 k: two rows of 8 in an MN-major operand, 32 bytes of a K-major one
            if constexpr (T::k8) {
              const uint32_t sf = tmem + 2 * T::NT + rs.s * SF_COLS;
              mma_step_scaled(d, a, ahi, b, bhi, id | ((k & 3u) << 4) | ((k & 3u) << 29), sf, sf + 4, k);
            } else {
              mma_step<T::kAmn ? 2048 >> 4 : 2, T::kBmn ? 2048 >> 4 : 2, KIND == PRODUCT_WEIGHT>(
                  d, a, ahi, b, bhi, id, k - k0, (min(t.len - k * 64, 64) + 15) / 16);
            }
            warp_commit(empty0 + r.s * 8);
            r.next();
          }
          if (!ok) break;
          if constexpr (T::k8) {         // the scales of a group of blocks are used
            warp_commit(smem_u32(&bar->sf_empty[rs.s]));
            rs.next();
          }
          if (KIND == PRODUCT_WEIGHT || k == t.steps) {
            warp_commit(smem_u32(&bar->tfull[acc]));
            ph ^= 1u << acc;
          }
        }
        if (t.steps > 0) acc ^= 1;
      }
      commit_pair(&bar->drain, 0x1);
      if (lane == 0) mbar_wait_bounded(&bar->drain, 0, nullptr, DRAIN_NS);
    }
    __syncwarp();
  } else if (warp == 2 && T::k8) {
    if constexpr (T::k8) {
      // The tokens' scales, SB_ROW bytes for each of four blocks.  (Loaded by the
      // warps that use them, one group ahead, they were waited for 2700 cycles a
      // group, whose products take 1800.)
      Ring<SB_SLOTS> rb;
      bool ok = true;
      for (int i = pair; ok && i < tiles.total; i += npairs) {
        const Tile t = tiles.get(i);
        const uint32_t bytes = static_cast<uint32_t>(min(SB_ROW, (p.tokens - t.n0 + 15) / 16 * 16));
        for (int k0 = 0; k0 < t.steps; k0 += 4) {
          ok = wait_warp(&bar->sb_empty[rb.s], rb.ph ^ 1u, abort, p);
          if (!ok) break;
          const int live = min(4, t.steps - k0);
          if (lane == 0) mbar_arrive_expect_tx(&bar->sb_full[rb.s], bytes * live);
          __syncwarp();
          if (lane < live)
            bulk_load(sb + SB_OFF + rb.s * SB_SLOT + lane * SB_ROW, p.scales + (k0 + lane) * p.lds + t.n0, bytes,
                      smem_u32(&bar->sb_full[rb.s]));
          rb.next();
        }
      }
      __syncwarp();
    }
  } else if (warp == 2) {
    if constexpr (KIND == PRODUCT_WEIGHT) {
      // Tokens behind an expert's last one are another's.  Products take 16 at
      // a time, so where the last 16 are not all its own the others' rows are
      // cleared, in both operands: what they hold may be infinite or NaN.
      const uint32_t full = mapa_shared(smem_u32(&bar->full[0]), 0), to = mapa_shared(smem_u32(&bar->token[1]), 0);
      uint32_t phases = 0;               // of own[], a bit each
      int first = 0;                     // the tile's first slot
      bool ok = true;
      auto clear = [&](uint32_t base, int boxes, int rest) {
        const int rows = 16 - (rest & 15);
        const uint32_t zero[4] = {0u, 0u, 0u, 0u};
        for (int c = lane; c < rows * boxes * 8; c += 32) {
          const int box = c / (rows * 8), in = c - box * rows * 8;
          sts16(base + box * BOX + rest * 128 + in * 16, zero);
        }
      };
      for (int i = pair; ok && i < tiles.total; i += npairs) {
        const Tile t = tiles.get(i);
        if (t.steps == 0) continue;
        if (mended<KIND>(t, t.steps - 1)) {
          const int s = (first + t.steps - 1) % SLOTS, rest = t.len & 63;
          ok = wait_warp(&bar->own[s], (phases >> s) & 1u, abort, p);
          if (!ok) break;
          phases ^= 1u << s;
          clear(sb + s * STAGE, 2, rest);
          clear(sb + B_OFF + s * STAGE, (t.padded() / 2 + 63) / 64, rest);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (rank == 0)
              mbar_arrive(&bar->full[s]);
            else
              send_token(to, smem_u32(&bar->token[0]), full + s * 8);
          }
          __syncwarp();
        }
        first = (first + t.steps) % SLOTS;
      }
    }
  } else if (T::k8 && warp >= 4 && warp < T::EPI_WARP0) {
    if constexpr (T::k8) {
      // Scales, four blocks at a time, to this warp's lanes: each row of 32
      // lanes of TMEM holds all of them.  The product reads its CTA's own copy,
      // of all n.  (What is behind the last token or block is of no meaning: no
      // result of such n is stored, no product takes such a byte.)
      const uint32_t lead = mapa_shared(smem_u32(&bar->sf_full[0]), 0);
      const uint32_t at0 = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 2 * T::NT;
      Ring<SF_SLOTS> rs;
      Ring<SB_SLOTS> rb;
      // The weight's bytes, one a lane for 32 blocks, loaded 32 blocks ahead.
      Tile t;
      int i = pair;                      // of the blocks that are loaded next
      int k = 0;
      uint32_t next = 0u, now = 0u;
      auto load = [&]() {
        if (i >= tiles.total) return;
        if (k == 0) t = tiles.get(i);
        const int m0 = t.m0 + static_cast<int>(rank) * 128;
        next = k + lane < t.steps && m0 < p.m ? p.wscales[(k + lane) * p.ws_col + (m0 >> 7) * p.ws_row] : 127u;
        k += 32;
        if (k >= t.steps) {
          k = 0;
          i += npairs;
        }
      };
      load();
      bool ok = true;
      for (int j = pair; ok && j < tiles.total; j += npairs) {
        const int steps = tiles.get(j).steps;
        for (int k0 = 0; k0 < steps; k0 += 4) {
          if ((k0 & 31) == 0) {
            now = next;
            load();
          }
          ok = wait_warp(&bar->sb_full[rb.s], rb.ph, abort, p);
          if (!ok) break;
          uint32_t word[8];
          const uint8_t* f = smem + SB_OFF + rb.s * SB_SLOT + lane;
#pragma unroll
          for (int c = 0; c < 7; ++c)
            word[c] = f[c * 32] | f[SB_ROW + c * 32] << 8 | f[2 * SB_ROW + c * 32] << 16 |
                      static_cast<uint32_t>(f[3 * SB_ROW + c * 32]) << 24;
          word[7] = 0u;
          uint32_t wword = 0u;
#pragma unroll
          for (int q = 0; q < 4; ++q) wword |= __shfl_sync(0xffffffffu, now, (k0 & 31) + q) << (8 * q);
          __syncwarp();                  // every lane's reads are behind the arrival
          if (lane == 0) mbar_arrive(&bar->sb_empty[rb.s]);
          rb.next();
          ok = wait_warp(&bar->sf_empty[rs.s], rs.ph ^ 1u, abort, p);
          if (!ok) break;
          tc_fence_after();
          tmem_st4(at0 + rs.s * SF_COLS, wword);
          tmem_st8(at0 + rs.s * SF_COLS + 4, word);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_relaxed(lead + rs.s * 8);
          rs.next();
        }
      }
    }
  } else if (warp >= T::EPI_WARP0) {
    // ----------------------------------------------------------- epilogue
    // Two warps for each quarter of an accumulator's m, every other 32 n each.
    const int ew = warp - T::EPI_WARP0, quad = warp & 3, half = ew >> 2;
    uint8_t* slot = smem + EPI_OFF + ew * SLOT;
    const uint32_t te[2] = {mapa_shared(smem_u32(&bar->tempty[0]), 0), mapa_shared(smem_u32(&bar->tempty[1]), 0)};
    const bool packed = p.vec && p.odtype != DT_F32 && p.add == nullptr;
    int acc = 0;
    uint32_t ph = 0u;                    // the accumulators' phases, a bit each
    bool ok = true;
    for (int i = pair; ok && i < tiles.total; i += npairs) {
      const Tile t = tiles.get(i);
      const int m0 = t.m0 + static_cast<int>(rank) * 128 + quad * 32, ms = p.m - m0;
      const bool some = T::kTokens || t.steps > 0;
      // weight: tokens past an accumulator's part are added in fp32, in scratch
      // that each thread reads back what it wrote to
      const int parts = T::kTokens ? 1 : max(1, (t.steps + STEPS_SUM - 1) / STEPS_SUM);
      if constexpr (!T::kTokens) {
        // what is added, to L2 while the products run: a row a lane, 32 m
        if (p.add != nullptr && ms > 0) {
          const int es = p.odtype == DT_F32 ? 4 : 2;
          for (int c = half * 32 + lane; c < t.n; c += 64) {
            const char* row = static_cast<const char*>(p.add) + (t.e * p.add_group + (t.n0 + c) * p.ldadd + m0) * es;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(row));
          }
        }
      }
      for (int j = 0; j < parts; ++j) {
        const int n = t.n, n0 = t.n0;
        const long long out = (T::kTokens ? 0 : t.e * p.out_group + t.split * p.out_split) + n0 * p.ldo + m0;
        const long long add = (T::kTokens ? 0 : t.e * p.add_group) + n0 * p.ldadd + m0;
        // what is added to this warp's first block is asked for before the wait,
        // each other block's when the one before is stored (8 experts of 125 rows,
        // 768 x 2304 in fp32: 30.3 us; asked for when it is due 32.8, with a second
        // set of registers 31.2)
        float f[8][4];
        const bool adds = !T::kTokens && p.add != nullptr && p.vec && ms >= 32 && j == parts - 1;
        if constexpr (!T::kTokens) {
          if (adds) load_added(p, add + half * 32 * p.ldadd, n - half * 32, lane, f);
        }
        if (some) {
          ok = wait_warp<32>(&bar->tfull[acc], (ph >> acc) & 1u, abort, p);
          if (!ok) break;
          ph ^= 1u << acc;
          tc_fence_after();
        }
        const uint32_t from = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * T::NT;
        auto read = [&]() {              // the accumulator may be written again
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_relaxed(te[acc]);
        };
        if (packed && some && ms >= 32 && parts == 1) {
          // all of this warp's blocks to registers first, rounded: the next
          // products wait for this
          uint32_t w[4][16];
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int c = half * 32 + b * 64;
            if (c < n) {
              if (p.odtype == DT_BF16)
                tmem_block<__nv_bfloat16>(from + c, w[b]);
              else
                tmem_block<__half>(from + c, w[b]);
            }
          }
          read();
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int c = half * 32 + b * 64;
            if (c < n) store_packed(smem_u32(slot), w[b], static_cast<uint16_t*>(p.out) + out + c * p.ldo, p.ldo, n - c, lane);
          }
          continue;
        }
#pragma unroll 1
        for (int c = half * 32; c < n; c += 64) {
          float v[32];
          if (some) {
            tmem_ld32(from + c, v);
          } else {
#pragma unroll
            for (int q = 0; q < 32; ++q) v[q] = 0.f;
          }
          if (some && c + 64 >= n) read();
          if constexpr (!T::kTokens) {
            if (parts > 1) {
              float* own = p.part + (static_cast<long long>(pair * 2 + static_cast<int>(rank)) * EPI_WARPS + ew) * PART_WARP +
                           (c >> 6) * 1024 + lane;
              if (j > 0) {
#pragma unroll
                for (int q = 0; q < 32; ++q) v[q] += own[q * 32];
              }
              if (j < parts - 1) {
#pragma unroll
                for (int q = 0; q < 32; ++q) own[q * 32] = v[q];
                continue;
              }
            }
          }
          if (ms > 0) store_block<!T::kTokens>(p, slot, v, f, out + c * p.ldo, add + c * p.ldadd, n - c, ms, lane);
          if constexpr (!T::kTokens) {
            if (adds && c + 64 < n) load_added(p, add + (c + 64) * p.ldadd, n - c - 64, lane, f);
          }
        }
        if (some && half * 32 >= n) read();
      }
      if (some && t.steps > 0) acc ^= 1;
    }
    if constexpr (T::kRagged) {
      const int w = (pair * 2 + static_cast<int>(rank)) * EPI_WARPS + ew, warps = npairs * 2 * EPI_WARPS;
      zero_rows(p, 0, at[0], w, warps, lane);
      zero_rows(p, at[p.groups], p.tokens, w, warps, lane);
    }
  }
  tc_fence_before();
  __syncthreads();
  // after a wait ran out: copies in flight get a millisecond to land before
  // the pair's memory is given up; none is issued any more
  if (threadIdx.x == 0 && *abort != 0) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {
    }
  }
  __syncwarp();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

template <int KIND>
cudaError_t launch_kind(ProductParams p, const CUtensorMap* maps, int pairs, cudaStream_t s) {
  p.mt = (p.m + MT - 1) / MT;
  long long total;
  if constexpr (Traits<KIND>::kRagged) {
    // at most: the tokens' experts are on the device
    total = static_cast<long long>(p.mt) * (p.tokens / p.most + (p.tokens < p.groups ? p.tokens : p.groups));
  } else {
    const int len = Traits<KIND>::kTokens ? p.tokens : p.n;
    p.size = tile_n(len, p.most, Traits<KIND>::kTokens);
    p.nt = len <= p.size ? 1 : (len + p.size - 1) / p.size;
    total = static_cast<long long>(p.mt) * p.nt * p.groups * p.splits;
  }
  if (total > 0x3FFFFFFFll) return cudaErrorInvalidValue;
  p.total = static_cast<int>(total);
  static std::atomic<unsigned long long> done;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(product_kernel<KIND>), SMEM, done);
  if (e != cudaSuccess) return e;
  const long long some = total < 1 ? 1 : total < pairs ? total : pairs;
  const cudaError_t l = launch_k(pdl_level() >= 1, product_kernel<KIND>, dim3(2 * static_cast<unsigned>(some)),
                                 dim3(Traits<KIND>::THREADS), SMEM, s, maps[0], maps[1], maps[2], p);
  return l != cudaSuccess ? l : cudaGetLastError();
}

// dw = add + the splits' partial results, in their order.
__global__ void __launch_bounds__(256) product_join_kernel(const ProductParams p, const float* part) {
  const long long each = static_cast<long long>(p.n) * p.m, count = p.groups * each;
  pdl_wait();                            // launched while the partial results are still being formed
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < count; i += gridDim.x * 256ll) {
    const long long e = i / each, in = i - e * each;
    const int n = static_cast<int>(in / p.m), m = static_cast<int>(in - static_cast<long long>(n) * p.m);
    float v = 0.f;
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) v += part[s * count + i];
    if (p.add != nullptr) v += load_f32(p.add, e * p.add_group + n * p.ldadd + m, p.odtype);
    store_any(p.out, e * p.out_group + n * p.ldo + m, p.odtype, v);
  }
}

// How a problem is cut: the most n of a tile and, for the weight's gradient, the
// parts that an expert's tokens are split into (a second kernel adds their
// results).  Wide tiles bring less to shared memory for each product; narrow ones
// and splits give every pair of SMs something to do, down to a step's 330 cycles
// of issue, which 160 n take: 1001 x 2042 x 1411 in 8 bits takes 15.7 us with the
// widest tiles and 10.5 with what this gives; the gradient of one weight 192 x 2088
// over 46894 rows 212 us without splits and 62 with them.
struct Plan {
  int most, splits;
};
Plan plan_of(int kind, long long tokens, int groups, int m, int n, int k, int pairs) {
  const bool k8 = kind == PRODUCT_ACT8, weight = kind == PRODUCT_WEIGHT;
  const long long mt = (m + MT - 1) / MT, each = (tokens + groups - 1) / groups;
  const long long len = weight ? n : each, steps = weight ? (each + 63) / 64 : (k + (k8 ? 127 : 63)) / (k8 ? 128 : 64);
  Plan best{};
  long long least = 0;
  for (int most = 32; most <= (k8 ? 224 : 256); most += 32) {
    const long long size = tile_n(static_cast<int>(len < 1 ? 1 : len), most, !weight), rows = size < len ? size : len;
    const long long tiles = groups * mt * ((len + size - 1) / size), step = std::max<long long>(330, 2 * ((rows + 31) / 32 * 32));
    for (int splits = 1; splits == 1 || (weight && tiles * splits <= pairs && steps / splits >= 8); ++splits) {
      // cycles: a turn of tiles, and for splits a launch and what they write and read
      const long long turns = (tiles * splits + pairs - 1) / pairs, join = splits > 1 ? 6000 + groups * (1ll * n * m) * splits / 400 : 0;
      const long long cost = turns * ((steps + splits - 1) / splits * step + 2500) + join;
      if (best.most == 0 || cost <= least) {
        best = Plan{most, splits};
        least = cost;
      }
    }
  }
  return best;
}

}  // namespace

namespace {
// Scratch of the weight's gradient: the CTAs' sums over more tokens than an
// accumulator takes, then the splits' results.
uint64_t sums_bytes(int64_t tokens, int sms) {
  return tokens > STEPS_SUM * 64 ? static_cast<uint64_t>(sms) * EPI_WARPS * PART_WARP * 4 : 0;
}
}  // namespace

uint64_t product_part_bytes(int64_t tokens, int cols, int out, int groups, int sms) {
  const Plan plan = plan_of(PRODUCT_WEIGHT, tokens, groups, cols, out, 0, sms / 2);
  const uint64_t split = plan.splits > 1 ? static_cast<uint64_t>(plan.splits) * groups * out * cols * 4 : 0;
  return sums_bytes(tokens, sms) + split;
}

cudaError_t launch_product(const ProductParams& q, const CUtensorMap* maps, int sms, cudaStream_t s, int* launches) {
  ProductParams p = q;
  const Plan plan = plan_of(p.kind, p.tokens, p.groups, p.m, p.n, p.k, sms / 2);
  p.most = plan.most;
  p.splits = plan.splits;
  *launches = 1;
  float* split = nullptr;
  if (p.splits > 1) {
    split = p.part + sums_bytes(p.tokens, sms) / 4;
    p.out = split;
    p.add = nullptr;
    p.odtype = DT_F32;
    p.ldo = p.m;
    p.out_group = static_cast<long long>(p.n) * p.m;
    p.out_split = p.groups * p.out_group;
  }
  const int es = p.odtype == DT_F32 ? 4 : 2;
  auto fits = [es](const void* at, long long ld, long long group) {
    return reinterpret_cast<uintptr_t>(at) % 16 == 0 && ld * es % 16 == 0 && group * es % 16 == 0;
  };
  p.vec = fits(p.out, p.ldo, p.out_group) && (p.add == nullptr || fits(p.add, p.ldadd, p.add_group)) && p.m % 8 == 0;
  cudaError_t e;
  switch (p.kind) {
    case PRODUCT_FORWARD: e = launch_kind<PRODUCT_FORWARD>(p, maps, sms / 2, s); break;
    case PRODUCT_ACT8: e = launch_kind<PRODUCT_ACT8>(p, maps, sms / 2, s); break;
    case PRODUCT_INPUT: e = launch_kind<PRODUCT_INPUT>(p, maps, sms / 2, s); break;
    default: e = launch_kind<PRODUCT_WEIGHT>(p, maps, sms / 2, s);
  }
  if (e != cudaSuccess || p.splits == 1) return e;
  *launches = 2;
  ProductParams j = q;
  j.splits = p.splits;
  const long long want = (p.out_split + 255) / 256;
  e = launch_k(pdl_level() >= 1, product_join_kernel, dim3(static_cast<unsigned>(want < sms * 8ll ? want : sms * 8ll)), dim3(256), 0,
               s, j, static_cast<const float*>(split));
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace muon
