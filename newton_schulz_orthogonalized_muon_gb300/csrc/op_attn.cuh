// What the attention kernels share: how a work item finds its sequence, the
// operand tiles in shared memory, and the tensor-core and TMEM access.
//
// A tile is 64 or 128 rows (tokens of one head) by DP = 64 or 128 columns of
// 16-bit elements, in boxes of 64 columns (128-byte rows, 128-byte swizzle),
// as TMA writes them from a 4-D map {dim, head, token, batch}.  Columns past
// `dim` and, in the batched form, rows past the sequence are filled with
// zeros.  One such tile serves both as a K-major operand (the product runs
// over dim) and as an MN-major one (over tokens).
#pragma once

#include "common.cuh"
#include "internal.h"
#include "op_common.cuh"

namespace muon {
namespace attn {

constexpr int TILE = 128;                    // rows of a tile
constexpr int BOX_BYTES = 128 * 128;         // 128 rows x 64 16-bit columns
constexpr float LOG2E = 1.4426950408889634f;

// The tensor core adds each product of 16 rows to its fp32 accumulator with
// truncation, so a sum of one sign comes out too small, the more the longer
// (walks of 8192, 65536 and 524288 rows: by 5e-5, 4e-4 and 3e-3 of itself).
// Results are rounded by up to 2^-12 (fp16) or 2^-9 (bf16), five times what
// 8192 or 65536 rows lose.  Walks over more rows are handed over in parts of
// as many, which are added up in fp32 with rounding, in scratch memory of the
// CTA (p.part): each value is read back by the thread that wrote it.  (Kernels
// of their own: the hot loops took 3 to 4% longer with the code for parts
// beside them.)
template <typename T>
constexpr int SUM_ROWS = attn_sum_rows(std::is_same<T, __nv_bfloat16>::value);

template <int DP>
__host__ __device__ constexpr int tile_bytes() {
  return DP / 64 * BOX_BYTES;
}

// ------------------------------------------------------------- work items
// One tile of rows of one sequence, and the sequence on both token axes.
struct Work {
  int q0, nq;        // first query token and queries
  int k0, nk;        // first key token and keys
  int tile;          // the item's tile within the sequence
  int qtile;         // the sequence's first query tile in the padded numbering
  int b, h;          // batch index (0 when packed), head of the item's axis
  int ok;            // 0: the grid's bound is above the real number of tiles
};

// Packed sequences: finds the sequence that tile `tile` (of `rows` rows) of
// the query (by_q) or key axis belongs to.  Every sequence has ceil(length /
// rows) tiles; the tokens before the first offset and after the last form
// sequences of their own that see nothing.  Offsets are device data and not
// trusted: they are clamped to the axis and to the largest before them.  All
// 32 lanes call it.
__device__ __forceinline__ Work find_packed(const AttnParams& p, bool by_q, int rows, int tile) {
  const int lane = threadIdx.x & 31;
  const int n = p.batch;
  int pq = 0, pk = 0, tiles = 0, qtiles = 0;
  Work w{};
  for (int d0 = 0; d0 <= n + 1; d0 += 32) {
    const int d = d0 + lane;                     // segment d ends at offset d (the last: at the axis' end)
    int eq = d <= n ? min(max(p.cu_q[d], 0), p.sq) : p.sq;
    int ek = d <= n ? min(max(p.cu_k[d], 0), p.sk) : p.sk;
    eq = max(eq, pq);
    ek = max(ek, pk);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, eq, o), c = __shfl_up_sync(0xffffffffu, ek, o);
      if (lane >= o) {
        eq = max(eq, a);
        ek = max(ek, c);
      }
    }
    int bq = __shfl_up_sync(0xffffffffu, eq, 1), bk = __shfl_up_sync(0xffffffffu, ek, 1);
    if (lane == 0) {
      bq = pq;
      bk = pk;
    }
    int nq = eq - bq, nk = ek - bk;
    const int tq = (nq + TILE - 1) / TILE;
    const int t = ((by_q ? nq : nk) + rows - 1) / rows;
    int st = t, sq = tq;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, st, o), c = __shfl_up_sync(0xffffffffu, sq, o);
      if (lane >= o) {
        st += a;
        sq += c;
      }
    }
    const int first = tiles + st - t;
    const unsigned hit = __ballot_sync(0xffffffffu, tile >= first && tile < first + t);
    if (hit != 0) {
      const int src = __ffs(hit) - 1;
      if (d < 1 || d > n) {                      // not a sequence: nothing on the other axis
        if (by_q)
          nk = 0;
        else
          nq = 0;
      }
      w.q0 = __shfl_sync(0xffffffffu, bq, src);
      w.nq = __shfl_sync(0xffffffffu, nq, src);
      w.k0 = __shfl_sync(0xffffffffu, bk, src);
      w.nk = __shfl_sync(0xffffffffu, nk, src);
      w.tile = tile - __shfl_sync(0xffffffffu, first, src);
      w.qtile = __shfl_sync(0xffffffffu, qtiles + sq - tq, src);
      w.ok = 1;
      return w;
    }
    tiles += __shfl_sync(0xffffffffu, st, 31);
    qtiles += __shfl_sync(0xffffffffu, sq, 31);
    pq = __shfl_sync(0xffffffffu, eq, 31);
    pk = __shfl_sync(0xffffffffu, ek, 31);
  }
  return w;
}

// The first 32 segments of packed sequences as find_packed meets them, one a
// lane, for a warp that looks for many tiles: a search that starts from the
// offsets each time took 0.3 us an item and more.
struct PackedIndex {
  int q0 = 0, nq = 0, k0 = 0, nk = 0;      // the lane's segment
  int qt = 0, ft[2] = {0, 0}, nt[2] = {0, 0};      // its first padded query tile; first tile and tiles by keys, queries
  __device__ __forceinline__ void fill(const AttnParams& p, int rows) {
    const int d = threadIdx.x & 31, n = p.batch;
    int eq = d <= n ? min(max(p.cu_q[d], 0), p.sq) : p.sq, ek = d <= n ? min(max(p.cu_k[d], 0), p.sk) : p.sk;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, eq, o), c = __shfl_up_sync(0xffffffffu, ek, o);
      if (d >= o) {
        eq = max(eq, a);
        ek = max(ek, c);
      }
    }
    q0 = __shfl_up_sync(0xffffffffu, eq, 1);
    k0 = __shfl_up_sync(0xffffffffu, ek, 1);
    if (d == 0) q0 = k0 = 0;
    nq = eq - q0;
    nk = ek - k0;
    nt[0] = (nk + rows - 1) / rows;
    nt[1] = (nq + rows - 1) / rows;
    const int padded = (nq + TILE - 1) / TILE;
    int s[3] = {nt[0], nt[1], padded};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const int a = __shfl_up_sync(0xffffffffu, s[i], o);
        if (d >= o) s[i] += a;
      }
    ft[0] = s[0] - nt[0];
    ft[1] = s[1] - nt[1];
    qt = s[2] - padded;
    if (d < 1 || d > n) nt[0] = -nt[0], nt[1] = -nt[1];      // not a sequence
  }
  // false: the tile is none of theirs
  __device__ __forceinline__ bool find(bool by_q, int tile, Work* w) const {
    const int f = by_q ? ft[1] : ft[0], n = by_q ? nt[1] : nt[0];
    const unsigned hit = __ballot_sync(0xffffffffu, tile >= f && tile < f + abs(n));
    if (hit == 0) return false;
    const int src = __ffs(hit) - 1;
    const bool seq = __shfl_sync(0xffffffffu, n, src) > 0;
    const int sq = __shfl_sync(0xffffffffu, nq, src), sk = __shfl_sync(0xffffffffu, nk, src);
    *w = Work{__shfl_sync(0xffffffffu, q0, src), seq || by_q ? sq : 0, __shfl_sync(0xffffffffu, k0, src),
              seq || !by_q ? sk : 0, tile - __shfl_sync(0xffffffffu, f, src), __shfl_sync(0xffffffffu, qt, src), 0, 0, 1};
    return true;
  }
};

// Work item `item` of a grid of tiles of `rows` rows x (heads x batch), heads
// fastest.  The longest items of a causal grid come first: the key tiles in
// their order, the query tiles (`tiles` of them at most) from the last.
// index: of the packed sequences, with these rows; nullptr: none.
__device__ __forceinline__ Work find_work(const AttnParams& p, bool by_q, int rows, int heads, int tiles,
                                          uint32_t item, const PackedIndex* index = nullptr) {
  const uint32_t hb = static_cast<uint32_t>(heads) * (p.cu_q != nullptr ? 1u : static_cast<uint32_t>(p.batch));
  int tile = static_cast<int>(item / hb);
  const uint32_t r = item % hb;
  if (by_q) tile = tiles - 1 - tile;
  Work w;
  if (p.cu_q != nullptr) {
    if (index == nullptr || !index->find(by_q, tile, &w)) w = find_packed(p, by_q, rows, tile);
    w.b = 0;
  } else {
    w = Work{0, p.sq, 0, p.sk, tile, 0, static_cast<int>(r / heads), 0, 1};
  }
  w.h = static_cast<int>(r % heads);
  return w;
}

// Tiles of an axis: exact in the batched form, a bound when packed (every
// sequence, and what lies outside them, can end in a part of a tile).
inline long long tile_bound(int len, int rows, int batch, bool packed) {
  return packed ? len / rows + static_cast<long long>(batch) + 2 : (len + rows - 1) / rows;
}

struct Range {
  int first, count;
};

// Key tiles of ROWS rows that the queries [i0, i1] of a sequence see (count 0:
// none).
template <int ROWS = TILE>
__device__ __forceinline__ Range key_tiles(const AttnParams& p, const Work& w, int i0, int i1) {
  int beg = 0, end = w.nk;
  if (p.causal) {
    const int off = w.nk - w.nq;
    end = min(end, i1 + off + 1);
    if (p.window > 0) beg = max(0, i0 + off - p.window + 1);
  }
  if (end <= beg) return Range{0, 0};
  return Range{beg / ROWS, (end + ROWS - 1) / ROWS - beg / ROWS};
}

// Query tiles that see any of the keys [j0, j1].
template <int ROWS>
__device__ __forceinline__ Range query_tiles(const AttnParams& p, const Work& w, int j0, int j1) {
  int beg = 0, end = w.nq;
  if (p.causal) {
    const int off = w.nk - w.nq;
    beg = max(0, j0 - off);
    if (p.window > 0) end = static_cast<int>(min(static_cast<long long>(end), static_cast<long long>(j1) - off + p.window));
  }
  if (end <= beg) return Range{0, 0};
  return Range{beg / ROWS, (end + ROWS - 1) / ROWS - beg / ROWS};
}

// ------------------------------------------------------------------- waits
// Every lane polls; the warp leaves together.  Gives up (and says so in the
// error word) after the time limit, or when another warp gave up.
__device__ __forceinline__ bool wait_warp(uint32_t a, uint32_t parity, volatile int* abort, const AttnParams& p) {
  if (__all_sync(0xffffffffu, mbar_try_wait(a, parity))) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (__all_sync(0xffffffffu, mbar_try_wait(a, parity))) return true;
    if ((it & 31u) == 0u) {
      const bool late = globaltimer_ns() - t0 > p.timeout_ns;
      if (__any_sync(0xffffffffu, late || *abort != 0)) {
        if ((threadIdx.x & 31) == 0) {
          if (late) atomicOr(p.err, ERRBIT_TIMEOUT);
          *abort = 1;
        }
        return false;
      }
    }
  }
}

// The swizzled tiles need shared memory that starts on a 1 KB boundary, which
// a kernel without static shared memory gets.
__device__ __forceinline__ bool swizzle_aligned(uint32_t base, const AttnParams& p) {
  if ((base & 1023u) == 0u) return true;
  if (threadIdx.x == 0) atomicOr(p.err, ERRBIT_TIMEOUT);
  return false;
}

// -------------------------------------------------------------------- TMA
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z,
                                            int u) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(u), "r"(bar)
      : "memory");
}
// Loads a tile of ROWS rows that starts at token `row`, by one lane, signalled
// on `bar` (which the caller has armed with the tile's bytes); the map's boxes
// have BOX rows.
template <int DP, int ROWS = TILE, int BOX = TILE>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar, int h, int row, int b) {
#pragma unroll
  for (int x = 0; x < DP / 64; ++x)
#pragma unroll
    for (int y = 0; y < ROWS; y += BOX) tma_load_4d(dst + (x * ROWS + y) * 128, map, bar, 64 * x, h, row + y, b);
}

// The same tile, of a packed sequence that ends inside it, once it is loaded
// (signalled on `edge`, a barrier of the loading warp): the next sequence's
// rows, which were loaded with it, are overwritten with zeros, so that a NaN
// or an infinity there has no part in a product with a zero probability.  By
// the whole warp; on return the tile is complete for the async proxy.
template <int DP, int ROWS = TILE>
__device__ __forceinline__ bool finish_edge_tile(uint32_t dst, uint32_t edge, uint32_t& phase, int valid,
                                                 volatile int* abort, const AttnParams& p) {
  const int lane = threadIdx.x & 31;
  if (!wait_warp(edge, phase & 1u, abort, p)) return false;
  ++phase;
#pragma unroll
  for (int x = 0; x < DP / 64; ++x)
    for (int i = valid * 8 + lane; i < ROWS * 8; i += 32)
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst + x * ROWS * 128 + i * 16), "r"(0u) : "memory");
  fence_proxy_async_smem();
  __syncwarp();
  return true;
}

// ---------------------------------------------------------------- tcgen05
// kind::f16 with 16-bit operands of T and fp32 accumulation, M = 128.
template <typename T>
__device__ __forceinline__ constexpr uint32_t idesc(int n, int b_mn_major) {
  const uint32_t fmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  return (1u << 4) | (fmt << 7) | (fmt << 10) | (static_cast<uint32_t>(b_mn_major) << 16) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(TILE >> 4) << 24);
}
// The products are issued by one warp whose lanes stay together: every value
// is warp-uniform and the instructions themselves pick one lane, once for
// four products.  (Issued from a branch that one lane takes, with descriptors
// rebuilt each time, a product of 64 cycles took about 100 to issue.)
//
// Four products of 16 along the summed index; SS: A from shared memory, its
// descriptor 32 bytes further each time, and so B's (K-major).
__device__ __forceinline__ void umma_ss4(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n"
      " .reg .pred p, q, t;\n"
      " .reg .b64 a1, a2, a3, b1, b2, b3;\n"
      " elect.sync _|q, 0xffffffff;\n"
      " setp.ne.b32 p, %4, 0;\n"
      " setp.eq.b32 t, 0, 0;\n"
      " add.s64 a1, %1, 2;\n"
      " add.s64 b1, %2, 2;\n"
      " add.s64 a2, %1, 4;\n"
      " add.s64 b2, %2, 4;\n"
      " add.s64 a3, %1, 6;\n"
      " add.s64 b3, %2, 6;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n"
      "}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
// A from TMEM: 16 tokens are eight columns; after two products `skip` more
// columns to the next 32 tokens.  B MN-major: 16 rows, 2 KB, further each time.
template <int SKIP>
__device__ __forceinline__ void umma_ts4(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n"
      " .reg .pred p, q, t;\n"
      " .reg .b32 a1, a2, a3;\n"
      " .reg .b64 b1, b2, b3;\n"
      " elect.sync _|q, 0xffffffff;\n"
      " setp.ne.b32 p, %4, 0;\n"
      " setp.eq.b32 t, 0, 0;\n"
      " add.s32 a1, %1, 8;\n"
      " add.s64 b1, %2, 128;\n"
      " add.s32 a2, %1, %5;\n"
      " add.s64 b2, %2, 256;\n"
      " add.s32 a3, %1, %6;\n"
      " add.s64 b3, %2, 384;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n"
      "}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc), "n"(16 + SKIP), "n"(24 + SKIP)
      : "memory");
}
// arrives on `bar` when every product issued so far by this warp is done
__device__ __forceinline__ void commit_warp(uint32_t bar) {
  asm volatile(
      "{\n"
      " .reg .pred q;\n"
      " elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n"
      "}\n" ::"r"(bar)
      : "memory");
}
// Descriptors of a tile of ROWS rows: K-major (over dim) and MN-major (over
// tokens).  A step along either adds its byte offset / 16.
__device__ __forceinline__ uint64_t desc_dim(uint32_t tile) { return sdesc_sw128(tile, 16, 1024); }
template <int ROWS = TILE>
__device__ __forceinline__ uint64_t desc_tokens(uint32_t tile) { return sdesc_sw128(tile, ROWS * 128, 1024); }

// D[128 x N] = A B^T over dim: both tiles K-major, B of N rows.
template <typename T, int DP, int N = TILE>
__device__ __forceinline__ void mma_over_dim(uint32_t d, uint64_t a, uint64_t b) {
  constexpr uint32_t id = idesc<T>(N, 0);
#pragma unroll
  for (int x = 0; x < DP / 64; ++x) umma_ss4(d, a + x * (TILE * 128 >> 4), b + x * (N * 128 >> 4), id, x != 0 ? 1u : 0u);
}
// D[128 x DP] (+)= A B over N tokens: A 16-bit in TMEM, CHUNK tokens (two a
// column) at a time with CHUNK columns from one chunk to the next; B a tile
// of N rows read MN-major.
template <typename T, int DP, int CHUNK, int N = TILE>
__device__ __forceinline__ void mma_over_tokens(uint32_t d, uint32_t a, uint64_t b, uint32_t acc) {
  static_assert(CHUNK == 32 || CHUNK == N, "chunks of a warp's columns, or of a row");
  constexpr uint32_t id = idesc<T>(DP, 1);
  constexpr int kSkip = CHUNK == 32 ? 16 : 0;
#pragma unroll
  for (int k = 0; k < N / 64; ++k)
    umma_ts4<kSkip>(d, a + k * (32 + 2 * kSkip), b + k * (4 * 2048 >> 4), id, k != 0 ? 1u : acc);
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// 16 rows x 32 columns, spread over the warp as the matrix instructions'
// accumulators are: v[4 j ..] of thread t are columns 8 j + 2 (t % 4) + {0, 1}
// of row t / 4, then of row t / 4 + 8.  (A value that belongs to a column is
// then wanted by a quarter of the threads, not by all.)
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// The same values in 16 bits, two a column: r[2 j] is column 4 j + t % 4 of
// row t / 4, r[2 j + 1] of row t / 4 + 8.
__device__ __forceinline__ void tmem_st_16x16(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// bits [lo, hi) of 32
__device__ __forceinline__ uint32_t bits32(int lo, int hi) {
  return __funnelshift_lc(0u, ~0u, max(lo, 0)) & ~__funnelshift_lc(0u, ~0u, max(hi, 0));
}

// Probabilities are rounded to T times 2^N, taken back from what they are
// summed to: fp16 has few bits left below 2^-14 and none below 2^-25, and
// over many keys such probabilities add up.  (bf16 has fp32's range: N = 0.)
// Forward they reach 2^raise, backward about 1.
template <typename T>
__host__ __device__ constexpr int lift_forward() {
  return std::is_same<T, __half>::value ? 11 : 0;
}
template <typename T>
__host__ __device__ constexpr float raise() {
  return std::is_same<T, __half>::value ? 4.f : 8.f;
}
template <typename T>
__host__ __device__ constexpr int lift_backward() {
  return std::is_same<T, __half>::value ? 14 : 0;
}
// 2^-n
__host__ __device__ constexpr float lowered(int n) { return 1.f / static_cast<float>(1 << n); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 32 x 32 fp32 TMEM values of this warp's rows, rounded to T, out to `dst` (row
// 0, column 0; `rows` rows and `cols` columns of it exist), the rows lane / 4 +
// 8 k of a lane times mul[k].
// Read in the accumulators' layout, and four lanes trade their words, so that
// they write 64 bytes of a row: a row a lane, 16 bytes at a time, took twice
// as long.
// parts: SUM_ADD, the values in `sums` (32 x 32 of this warp's) are added
// first; SUM_KEEP, the result goes there instead, as it is.
enum : int { SUM_ADD = 1, SUM_KEEP = 2 };
template <typename T, bool PARTS = false>
__device__ __forceinline__ void store_rows(uint32_t taddr, T* dst, long long stride, int rows, int cols, const float* mul,
                                           int parts = 0, float* sums = nullptr) {
  if (cols <= 0) return;
  const int lane = threadIdx.x & 31, c = lane & 3;
  float v[32];
  tmem_ld_16x32(taddr, v);
  tmem_ld_16x32(taddr + (16u << 16), v + 16);
  tmem_ld_wait();
  if constexpr (PARTS) {
    if (parts & SUM_ADD) {
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] += sums[e * 32 + lane];
    }
    if (parts & SUM_KEEP) {
#pragma unroll
      for (int e = 0; e < 32; ++e) sums[e * 32 + lane] = v[e];
      return;
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {              // row lane / 4 + 8 k
    uint32_t w[4];                           // word q: columns 8 q + 2 c, + 1
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float* u = v + 16 * (k >> 1) + 4 * q + 2 * (k & 1);
      w[q] = pack2<T>(u[0] * mul[k], u[1] * mul[k]);
    }
    // transposed over the four lanes: lane c gets columns 8 c .. 8 c + 7
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
      const bool up = (c & o) != 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if ((q & o) == 0) {
          const uint32_t send = up ? w[q] : w[q | o];
          const uint32_t got = __shfl_xor_sync(0xffffffffu, send, o);
          if (up)
            w[q] = got;
          else
            w[q | o] = got;
        }
      }
    }
    const int r = (lane >> 2) + 8 * k;
    if (r < rows && 8 * c < cols) *reinterpret_cast<uint4*>(dst + r * stride + 8 * c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// one arrival of a warp whose lanes' TMEM accesses are complete
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive_at(bar);
}

// 2 N values of a row, rounded to T, into N = 16 or 32 TMEM columns.
template <typename T, int N>
__device__ __forceinline__ void store_rounded(uint32_t taddr, const float* v) {
  uint32_t r[N];
#pragma unroll
  for (int k = 0; k < N; ++k) r[k] = pack2<T>(v[2 * k], v[2 * k + 1]);
  if constexpr (N == 32)
    tmem_st32(taddr, r);
  else
    tmem_st16(taddr, r);
  tmem_st_wait();
}

}  // namespace attn
}  // namespace muon
