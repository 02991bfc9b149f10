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
// A CTA pair forms 256 m (128 a CTA) by up to 256 n (tcgen05.mma.cta_group::2).
// The ragged dimension, tokens, is n: the tensor core takes n in steps of 32,
// so an expert's last tile costs what it has, where rows of m would be padded
// to 256 (17% of the work at 768 tokens an expert).  Operands come by TMA with
// 128-byte swizzle, K-major or MN-major as they lie in memory, through a ring
// of five stages; two accumulators in TMEM, so that a tile's results leave
// while the next is formed.  Eight epilogue warps turn 32 x 32 blocks around
// through shared memory (a lane holds one m), so that rows leave in whole
// sectors.
//
// The groups' offsets are device data: every CTA clamps them (to the token
// axis and the largest before them) and counts the tiles for itself.
#include "common.cuh"
#include "internal.h"
#include "op_common.cuh"
#include "op_pair.cuh"

namespace muon {
namespace {

constexpr int MT = 256;                  // m of a pair's tile
constexpr int BOX = 64 * 128;            // 64 rows of 128 bytes
constexpr int STAGES = 5, STAGE = 4 * BOX;
constexpr int EPI_WARPS = 8, SLOT = 4096;
constexpr int STEPS_SUM = 32;            // weight: steps of 64 tokens an accumulator takes
constexpr int PART_WARP = 4 * 1024;      // floats of scratch of an epilogue warp
constexpr int EPI_OFF = STAGES * STAGE;
constexpr int GROUP_OFF = EPI_OFF + EPI_WARPS * SLOT;
// 8 bits: the tokens' scales on their way, 256 of each of four blocks
constexpr int SB_SLOTS = 4, SB_SLOT = 4 * 256;
constexpr int SB_OFF = GROUP_OFF + 2 * 4 * (kMaxExperts + 4);
constexpr int BAR_OFF = SB_OFF + SB_SLOTS * SB_SLOT;
constexpr int SMEM = BAR_OFF + 512;
constexpr unsigned long long DRAIN_NS = 1000000000ull;
static_assert(SMEM <= 232448, "shared memory");

template <int KIND>
struct Traits {
  static constexpr bool kTokens = KIND != PRODUCT_WEIGHT;                   // n are tokens
  static constexpr bool kAmn = KIND == PRODUCT_INPUT || KIND == PRODUCT_WEIGHT;   // A is read MN-major
  static constexpr bool kBmn = KIND == PRODUCT_WEIGHT;
  static constexpr bool k8 = KIND == PRODUCT_ACT8;
  static constexpr int BK = k8 ? 128 : 64;                                  // 128 bytes
  static constexpr int EPI_WARP0 = k8 ? 8 : 4;
  static constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
  // most n of a tile: two accumulators and, for 8 bits, the scales share 512 columns of TMEM
  static constexpr int NT = k8 ? 224 : 256;
};
// The scales in TMEM, by groups of four 128-column blocks: a 32-bit word a row
// of A (4 columns of 32 lanes) and of B (8), a byte for each block.
constexpr int SF_SLOTS = 5, SF_COLS = 12;
static_assert(2 * Traits<PRODUCT_ACT8>::NT + SF_SLOTS * SF_COLS <= 512, "TMEM");

struct alignas(16) Bars {
  uint64_t full[STAGES];                 // the leader's, for both CTAs
  uint64_t empty[STAGES];                // each CTA's own
  uint64_t own[STAGES];                  // weight: this CTA's part of an expert's last step
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

// n of the tiles that a row of `len` is cut into: as few tiles as there can be,
// of about one size where the last would be small.
template <int NT>
__host__ __device__ __forceinline__ int tile_n(int len, bool even) {
  const int tiles = (len + NT - 1) / NT, rest = len % NT;
  if (tiles <= 1) return NT;
  if (!even && (rest == 0 || rest >= NT / 2)) return NT;
  return ((len + tiles - 1) / tiles + 31) / 32 * 32;
}

struct Tile {
  int e, m0, n0;       // group, first m, first n (of the token axis, or of the outputs)
  int n;               // that exist
  int t0, len;         // weight: the group's first token and tokens
  int steps;
};

// The tiles in order of their groups; a thread asks for rising numbers.
template <int KIND>
struct Tiles {
  const ProductParams& p;
  const int* at;       // [groups + 1] offsets
  const int* pre;      // [groups + 1] tiles before a group (tokens)
  int mt, total, e = 0;

  __device__ __forceinline__ Tiles(const ProductParams& q, const int* a) : p(q), at(a), pre(a + kMaxExperts + 4) {
    mt = (p.m + MT - 1) / MT;
    total = Traits<KIND>::kTokens ? pre[p.groups] : p.groups * mt * ((p.n + nsize() - 1) / nsize());
  }
  __device__ __forceinline__ int nsize() const { return tile_n<Traits<KIND>::NT>(p.n, false); }
  // A group's tiles go eight m at a time: the pairs that run together share
  // panels of A and of B in L2.
  __device__ __forceinline__ void place(int in, int nt, int& m0, int& n0, int size) const {
    const int band = in / (8 * nt), r = in - band * 8 * nt, rows = min(8, mt - band * 8), j = r / rows;
    m0 = (band * 8 + r - j * rows) * MT;
    n0 = j * size;
  }
  __device__ __forceinline__ Tile get(int i) {
    Tile t;
    if constexpr (Traits<KIND>::kTokens) {
      while (pre[e + 1] <= i) ++e;
      const int len = at[e + 1] - at[e], size = tile_n<Traits<KIND>::NT>(len, true);
      t.e = e;
      place(i - pre[e], (len + size - 1) / size, t.m0, t.n0, size);
      t.n0 += at[e];
      t.n = min(size, at[e + 1] - t.n0);
      t.steps = (p.k + Traits<KIND>::BK - 1) / Traits<KIND>::BK;
      t.t0 = t.len = 0;
    } else {
      const int size = nsize(), per = mt * ((p.n + size - 1) / size);
      t.e = i / per;
      place(i - t.e * per, per / mt, t.m0, t.n0, size);
      t.n = min(size, p.n - t.n0);
      t.t0 = at[t.e];
      t.len = at[t.e + 1] - t.t0;
      t.steps = (t.len + Traits<KIND>::BK - 1) / Traits<KIND>::BK;
    }
    return t;
  }
};

// Offsets and tile counts into shared memory; one warp.
template <int KIND>
__device__ __forceinline__ void count_tiles(const ProductParams& p, int* at) {
  int* pre = at + kMaxExperts + 4;
  const int lane = threadIdx.x & 31, mt = (p.m + MT - 1) / MT;
  int last = 0, tiles = 0;               // offset and tiles of the groups so far
  for (int d0 = 0; d0 <= p.groups; d0 += 32) {
    const int d = d0 + lane;
    int v = d <= p.groups ? min(max(p.offsets != nullptr ? p.offsets[d] : d == 0 ? 0 : p.tokens, 0), p.tokens) : p.tokens;
    v = max(v, last);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = max(v, u);
    }
    int before = __shfl_up_sync(0xffffffffu, v, 1);
    if (lane == 0) before = d0 == 0 ? v : last;
    int c = 0;                           // tiles of group d - 1
    if constexpr (Traits<KIND>::kTokens) {
      const int len = v - before;
      if (len > 0) {
        const int size = tile_n<Traits<KIND>::NT>(len, true);
        c = (len + size - 1) / size * mt;
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

// Pair product of e4m3 codes; the scales' columns, a power of two a row and 32 k.
__device__ __forceinline__ void mma_pair_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sa, uint32_t sb,
                                                uint32_t acc) {
  asm volatile(
      "{\n"
      " .reg .pred p, q;\n"
      " elect.sync _|q, 0xffffffff;\n"
      " setp.ne.b32 p, %6, 0;\n"
      " @q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n"
      "}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(sa), "r"(sb), "r"(acc)
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

// A 32 x 32 block of results to rows `rows` of 32 m from (out, add): lane l
// holds m = l, v[j] is row j.  Rows past `rows` and m past `ms` are not there.
// 16-bit results without `add` go through shared memory as pairs: lanes 2i and
// 2i + 1 exchange, so that each has two consecutive m of one row.
__device__ __forceinline__ void store_block(const ProductParams& p, uint8_t* slot, const float* v, long long out,
                                            long long add, int rows, int ms, int lane) {
  const uint32_t s = smem_u32(slot);
  __syncwarp();
  if (p.vec && ms >= 32 && p.odtype != DT_F32 && p.add == nullptr) {
    const uint32_t to = s + (lane & 1) * 64 + (lane >> 1) * 4, sel = lane & 1 ? 0x3276u : 0x5410u;
    const bool bf = p.odtype == DT_BF16;
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const uint32_t w = bf ? pack2<__nv_bfloat16>(v[j], v[j + 1]) : pack2<__half>(v[j], v[j + 1]);
      const uint32_t o = __shfl_xor_sync(0xffffffffu, w, 1);
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + j * 64), "r"(__byte_perm(w, o, sel)) : "memory");
    }
    __syncwarp();
    const int r = lane >> 2, q = lane & 3;
#pragma unroll
    for (int i = 0; i < 32; i += 8)
      if (r + i < rows)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + out + (r + i) * p.ldo + q * 8) = lds16(s + (r + i) * 64 + q * 16);
    return;
  }
#pragma unroll
  for (int j = 0; j < 32; ++j) asm volatile("st.shared.f32 [%0], %1;" ::"r"(s + j * 128 + lane * 4), "f"(v[j]) : "memory");
  __syncwarp();
  if (p.vec && ms >= 32) {
    const int r = lane >> 3, q = lane & 7;
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
      float f[4][4];
      if (p.add != nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (r + h + 4 * i < rows) load4(p.add, add + (r + h + 4 * i) * p.ldadd + q * 4, p.odtype, f[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (r + h + 4 * i >= rows) break;
        const uint4 raw = lds16(s + (r + h + 4 * i) * 128 + q * 16);
        float4 x = make_float4(__uint_as_float(raw.x), __uint_as_float(raw.y), __uint_as_float(raw.z), __uint_as_float(raw.w));
        if (p.add != nullptr) x.x += f[i][0], x.y += f[i][1], x.z += f[i][2], x.w += f[i][3];
        const long long to = out + (r + h + 4 * i) * p.ldo + q * 4;
        if (p.odtype == DT_F32)
          *reinterpret_cast<float4*>(static_cast<float*>(p.out) + to) = x;
        else
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + to) =
              p.odtype == DT_BF16 ? make_uint2(pack2<__nv_bfloat16>(x.x, x.y), pack2<__nv_bfloat16>(x.z, x.w))
                                  : make_uint2(pack2<__half>(x.x, x.y), pack2<__half>(x.z, x.w));
      }
    }
    return;
  }
  if (lane < ms) {
#pragma unroll 1
    for (int j = 0; j < 32 && j < rows; ++j) {
      float x;
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(s + j * 128 + lane * 4));
      if (p.add != nullptr) x += load_f32(p.add, add + j * p.ldadd + lane, p.odtype);
      store_any(p.out, out + j * p.ldo + lane, p.odtype, x);
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

template <int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Traits<KIND>::THREADS, 1)
    product_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                   const __grid_constant__ CUtensorMap mb32, const ProductParams p) {
  using T = Traits<KIND>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* bar = reinterpret_cast<Bars*>(smem + BAR_OFF);
  int* at = reinterpret_cast<int*>(smem + GROUP_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = static_cast<int>(cluster_id_x()), npairs = static_cast<int>(num_clusters_x());
  const uint32_t sb = smem_u32(smem);
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
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
  if (warp == 2) count_tiles<KIND>(p, at);
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = bar->tmem;
  volatile int* abort = &bar->abort;
  Tiles<KIND> tiles(p, at);

  if (warp == 0 || warp == 3) {
    if (lane == 0) {
      // ------------------------------------------------------------ loads
      // Warp 0 loads A and says what is to come, warp 3 loads B, in few large
      // boxes: a thread issues a load in some 200 cycles, a step's products
      // take 512.
      const bool is_a = warp == 0;
      const uint32_t lead = mapa_shared(smem_u32(&bar->full[0]), 0);
      Ring<STAGES> r;
      bool ok = true;
      for (int i = pair; ok && i < tiles.total; i += npairs) {
        const Tile t = tiles.get(i);
        const int m0 = t.m0 + static_cast<int>(rank) * 128;
        // of B, this CTA's half: boxes of 128 or 32 tokens, or of 64 outputs
        const int half = (t.n + 31) / 32 * 16, n0 = t.n0 + static_cast<int>(rank) * half;
        const bool one = !T::kBmn && half > 64;
        const int boxes = one ? 1 : T::kBmn ? (half + 63) / 64 : (half + 31) / 32;
        const uint32_t bytes = 2 * BOX + boxes * (one ? 2 * BOX : T::kBmn ? BOX : BOX / 2);
        for (int k = 0; k < t.steps; ++k) {
          ok = wait_one(&bar->empty[r.s], r.ph ^ 1u, abort, p);
          if (!ok) break;
          const uint32_t a = sb + r.s * STAGE, b = a + 2 * BOX, fb = lead + r.s * 8;
          if constexpr (KIND == PRODUCT_WEIGHT) {
            const int row = t.t0 + k * 64;
            if (k == t.steps - 1 && (t.len & 15) != 0) {
              // an expert's last tokens: to this CTA's own warp, which clears
              // what follows them (see below)
              uint64_t* own = &bar->own[r.s];
              if (is_a) {
                mbar_arrive_expect_tx(own, bytes);
                if (rank == 0) mbar_arrive_expect_tx(&bar->full[r.s], sizeof(uint4));
                tma_load_3d(a, &ma, own, m0, row, 0);
                tma_load_3d(a + BOX, &ma, own, m0 + 64, row, 0);
              } else {
                for (int c = 0; c < boxes; ++c) tma_load_3d(b + c * BOX, &mb, own, n0 + c * 64, row, 0);
              }
            } else if (is_a) {
              if (rank == 0) {
                mbar_arrive(&bar->full[r.s]);
                mbar_arrive_expect_tx(&bar->full[r.s], 2 * bytes);
              }
              tma_load_3d_pair(a, &ma, fb, m0, row, 0);
              tma_load_3d_pair(a + BOX, &ma, fb, m0 + 64, row, 0);
            } else {
              for (int c = 0; c < boxes; ++c) tma_load_3d_pair(b + c * BOX, &mb, fb, n0 + c * 64, row, 0);
            }
          } else if (is_a) {
            if (rank == 0) mbar_arrive_expect_tx(&bar->full[r.s], 2 * bytes);
            if constexpr (T::kAmn) {
              tma_load_3d_pair(a, &ma, fb, m0, k * T::BK, t.e);
              tma_load_3d_pair(a + BOX, &ma, fb, m0 + 64, k * T::BK, t.e);
            } else {
              tma_load_3d_pair(a, &ma, fb, k * T::BK, m0, t.e);
            }
          } else if (one) {
            tma_load_3d_pair(b, &mb, fb, k * T::BK, n0, 0);
          } else {
            for (int c = 0; c < boxes; ++c) tma_load_3d_pair(b + c * (BOX / 2), &mb32, fb, k * T::BK, n0 + c * 32, 0);
          }
          r.next();
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      // --------------------------------------------------------- products
      // 16 bits: fp32 results, operands bf16 or fp16.  8 bits: e4m3, scales 2^(byte - 127), the byte of a word at 4 (B)
      // and 29 (A)
      const uint32_t type = T::k8 ? 1u << 23 : (1u << 4) | (p.f16 ? 0u : (1u << 7) | (1u << 10));
      const uint32_t id0 = type | (T::kAmn ? 1u << 15 : 0u) | (T::kBmn ? 1u << 16 : 0u) | ((MT >> 4) << 24);
      Ring<SF_SLOTS> rs;
      Ring<STAGES> r;
      int acc = 0;
      uint32_t acc_ph = 0;
      bool ok = true;
      for (int i = pair; ok && i < tiles.total; i += npairs) {
        const Tile t = tiles.get(i);
        const uint32_t id = id0 | (static_cast<uint32_t>((t.n + 31) / 32 * 4) << 17);
        const int part = KIND == PRODUCT_WEIGHT ? STEPS_SUM : t.steps;
        for (int k0 = 0; ok && k0 < t.steps; k0 += part) {
          ok = wait_warp<0, true>(&bar->tempty[acc], acc_ph ^ 1u, abort, p);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + acc * T::NT;
          const int k1 = min(k0 + part, t.steps);
          for (int k = k0; k < k1; ++k) {
            ok = wait_warp<0, KIND == PRODUCT_WEIGHT>(&bar->full[r.s], r.ph, abort, p);
            if (!ok) break;
            if constexpr (T::k8) {
              if ((k & 3) == 0) ok = wait_warp<0, true>(&bar->sf_full[rs.s], rs.ph, abort, p);
              if (!ok) break;
            }
            tc_fence_after();
            const uint32_t sa = sb + r.s * STAGE;
            const uint64_t a = T::kAmn ? sdesc_sw128(sa, BOX, 1024) : sdesc_sw128(sa, 16, 1024);
            const uint64_t b = T::kBmn ? sdesc_sw128(sa + 2 * BOX, BOX, 1024) : sdesc_sw128(sa + 2 * BOX, 16, 1024);
            // steps of 16 k: two rows of 8 in an MN-major operand, 32 bytes of a K-major one
            const int kks = KIND == PRODUCT_WEIGHT ? (min(t.len - k * 64, 64) + 15) / 16 : 4;
            if constexpr (T::k8) {
              const uint32_t sf = tmem + 2 * T::NT + rs.s * SF_COLS, ids = id | ((k & 3u) << 4) | ((k & 3u) << 29);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_pair_scaled(d, a + kk * 2, b + kk * 2, ids, sf, sf + 4, kk != 0 || k != k0 ? 1u : 0u);
              if ((k & 3) == 3 || k == k1 - 1) {
                commit_pair(&bar->sf_empty[rs.s], 0x3);
                rs.next();
              }
            } else {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                if (kk < kks)
                  mma_pair(d, a + kk * (T::kAmn ? 2048 >> 4 : 2), b + kk * (T::kBmn ? 2048 >> 4 : 2), id,
                           kk != 0 || k != k0 ? 1u : 0u);
            }
            commit_pair(&bar->empty[r.s], 0x3);
            r.next();
          }
          if (!ok) break;
          commit_pair(&bar->tfull[acc], 0x3);
          acc ^= 1;
          if (acc == 0) acc_ph ^= 1u;
        }
      }
      commit_pair(&bar->drain, 0x1);
      if (lane == 0) mbar_wait_bounded(&bar->drain, 0, nullptr, DRAIN_NS);
    }
    __syncwarp();
  } else if (warp == 2 && T::k8) {
    if constexpr (T::k8) {
      // The tokens' scales, 256 bytes for each of four blocks.  (Loaded by the
      // warps that use them, one group ahead, they were waited for 2700 cycles a
      // group, whose products take 1800.)
      Ring<SB_SLOTS> rb;
      bool ok = true;
      for (int i = pair; ok && i < tiles.total; i += npairs) {
        const Tile t = tiles.get(i);
        const uint32_t bytes = static_cast<uint32_t>(min(256, (p.tokens - t.n0 + 15) / 16 * 16));
        for (int k0 = 0; k0 < t.steps; k0 += 4) {
          ok = wait_warp(&bar->sb_empty[rb.s], rb.ph ^ 1u, abort, p);
          if (!ok) break;
          const int live = min(4, t.steps - k0);
          if (lane == 0) mbar_arrive_expect_tx(&bar->sb_full[rb.s], bytes * live);
          __syncwarp();
          if (lane < live)
            bulk_load(sb + SB_OFF + rb.s * SB_SLOT + lane * 256, p.scales + (k0 + lane) * p.lds + t.n0, bytes,
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
      int s = 0;                         // the tile's first stage
      bool ok = true;
      for (int i = pair; ok && i < tiles.total; i += npairs) {
        const Tile t = tiles.get(i);
        if (t.steps == 0) continue;
        s = (s + t.steps - 1) % STAGES;
        const int rest = t.len & 63, first = rest;
        if ((rest & 15) != 0) {
          ok = wait_warp(&bar->own[s], (phases >> s) & 1u, abort, p);
          if (!ok) break;
          phases ^= 1u << s;
          const int rows = 16 - (rest & 15), boxes = 2 + ((t.n + 31) / 32 * 16 + 63) / 64;
          const uint32_t zero[4] = {0u, 0u, 0u, 0u};
          for (int c = lane; c < rows * boxes * 8; c += 32) {
            const int box = c / (rows * 8), in = c - box * rows * 8;
            sts16(sb + s * STAGE + box * BOX + first * 128 + in * 16, zero);
          }
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
        s = (s + 1) % STAGES;
      }
    }
  } else if (T::k8 && warp >= 4 && warp < T::EPI_WARP0) {
    if constexpr (T::k8) {
      // Scales, four blocks at a time, to this warp's lanes: each row of 32
      // lanes of TMEM holds all of them.  The product reads its CTA's own copy,
      // of all n.  (What is behind the last token or block is of no meaning: no
      // result of such n is stored, no product takes such a byte.)
      const int ksteps = (p.k + T::BK - 1) / T::BK;
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
        for (int k0 = 0; k0 < ksteps; k0 += 4) {
          if ((k0 & 31) == 0) {
            now = next;
            load();
          }
          ok = wait_warp(&bar->sb_full[rb.s], rb.ph, abort, p);
          if (!ok) break;
          uint32_t word[8];
          const uint8_t* from = smem + SB_OFF + rb.s * SB_SLOT + lane;
#pragma unroll
          for (int c = 0; c < 7; ++c)
            word[c] = from[c * 32] | from[256 + c * 32] << 8 | from[512 + c * 32] << 16 | static_cast<uint32_t>(from[768 + c * 32]) << 24;
          word[7] = 0u;
          uint32_t wword = 0u;
#pragma unroll
          for (int q = 0; q < 4; ++q) wword |= __shfl_sync(0xffffffffu, now, (k0 & 31) + q) << (8 * q);
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
          if (lane == 0) mbar_arrive_cluster(lead + rs.s * 8);
          rs.next();
        }
      }
    }
  } else if (warp >= T::EPI_WARP0) {
    // ----------------------------------------------------------- epilogue
    const int ew = warp - T::EPI_WARP0, quad = warp & 3, half = ew >> 2;
    uint8_t* slot = smem + EPI_OFF + ew * SLOT;
    const uint32_t te[2] = {mapa_shared(smem_u32(&bar->tempty[0]), 0), mapa_shared(smem_u32(&bar->tempty[1]), 0)};
    int acc = 0;
    uint32_t acc_ph = 0;
    bool ok = true;
    for (int i = pair; ok && i < tiles.total; i += npairs) {
      const Tile t = tiles.get(i);
      const int m0 = t.m0 + static_cast<int>(rank) * 128 + quad * 32, ms = p.m - m0;
      const long long out = (T::kTokens ? 0 : t.e * p.out_group) + t.n0 * p.ldo + m0;
      const long long add = (T::kTokens ? 0 : t.e * p.add_group) + t.n0 * p.ldadd + m0;
      if constexpr (T::kTokens) {
        ok = wait_warp<100>(&bar->tfull[acc], acc_ph, abort, p);
        if (!ok) break;
        tc_fence_after();
        const uint32_t from = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * T::NT;
        for (int c = half * 32; c < t.n; c += 64) {
          float v[32];
          tmem_ld32(from + c, v);
          if (c + 64 >= t.n) {           // this warp's last block: the accumulator is read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(te[acc]);
          }
          if (ms > 0) store_block(p, slot, v, out + c * p.ldo, add, t.n - c, ms, lane);
        }
        if (half * 32 >= t.n) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(te[acc]);
        }
        acc ^= 1;
        if (acc == 0) acc_ph ^= 1u;
      } else {
        // Tokens past an accumulator's part are added in fp32, in scratch that
        // each thread reads back what it wrote to.
        float* part = p.part + (static_cast<long long>(pair * 2 + rank) * EPI_WARPS + ew) * PART_WARP + lane;
        for (int k0 = 0; k0 < t.steps || k0 == 0; k0 += STEPS_SUM) {
          const bool last = k0 + STEPS_SUM >= t.steps;
          if (t.steps > 0) {
            ok = wait_warp<100>(&bar->tfull[acc], acc_ph, abort, p);
            if (!ok) break;
            tc_fence_after();
          }
          const uint32_t from = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * T::NT;
#pragma unroll 1
          for (int c = half * 32; c < t.n; c += 64) {
            float v[32];
            if (t.steps > 0) {
              tmem_ld32(from + c, v);
            } else {
#pragma unroll
              for (int q = 0; q < 32; ++q) v[q] = 0.f;
            }
            float* own = part + (c >> 6) * 1024;
            if (k0 > 0) {
#pragma unroll
              for (int q = 0; q < 32; ++q) v[q] += own[q * 32];
            }
            if (!last) {
#pragma unroll
              for (int q = 0; q < 32; ++q) own[q * 32] = v[q];
            } else if (ms > 0) {
              store_block(p, slot, v, out + c * p.ldo, add + c * p.ldadd, t.n - c, ms, lane);
            }
          }
          if (t.steps > 0) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(te[acc]);
            acc ^= 1;
            if (acc == 0) acc_ph ^= 1u;
          }
        }
      }
    }
    if constexpr (T::kTokens) {
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
cudaError_t launch_kind(const ProductParams& p, const CUtensorMap* maps, int pairs, cudaStream_t s) {
  const long long mt = (p.m + MT - 1) / MT;
  // tiles, at most: the tokens' experts are on the device
  const long long nt = Traits<KIND>::kTokens
                           ? p.tokens / Traits<KIND>::NT + (p.tokens < p.groups ? p.tokens : p.groups)
                           : static_cast<long long>(p.groups) * ((p.n + 31) / 32);
  if (mt * nt > 0x3FFFFFFFll) return cudaErrorInvalidValue;
  static std::atomic<unsigned long long> done;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(product_kernel<KIND>), SMEM, done);
  if (e != cudaSuccess) return e;
  const long long some = mt * nt < 1 ? 1 : mt * nt < pairs ? mt * nt : pairs;
  product_kernel<KIND><<<dim3(2 * static_cast<unsigned>(some)), Traits<KIND>::THREADS, SMEM, s>>>(maps[0], maps[1],
                                                                                                    maps[2], p);
  return cudaGetLastError();
}

}  // namespace

uint64_t product_part_bytes(int64_t tokens, int sms) {
  return tokens > STEPS_SUM * 64 ? static_cast<uint64_t>(sms) * EPI_WARPS * PART_WARP * 4 : 0;
}

cudaError_t launch_product(const ProductParams& q, const CUtensorMap* maps, int pairs, cudaStream_t s) {
  ProductParams p = q;
  const int es = p.odtype == DT_F32 ? 4 : 2;
  auto fits = [es](const void* at, long long ld, long long group) {
    return reinterpret_cast<uintptr_t>(at) % 16 == 0 && ld * es % 16 == 0 && group * es % 16 == 0;
  };
  p.vec = fits(p.out, p.ldo, p.out_group) && (p.add == nullptr || fits(p.add, p.ldadd, p.add_group)) && p.m % 8 == 0;
  switch (p.kind) {
    case PRODUCT_FORWARD: return launch_kind<PRODUCT_FORWARD>(p, maps, pairs, s);
    case PRODUCT_ACT8: return launch_kind<PRODUCT_ACT8>(p, maps, pairs, s);
    case PRODUCT_INPUT: return launch_kind<PRODUCT_INPUT>(p, maps, pairs, s);
    default: return launch_kind<PRODUCT_WEIGHT>(p, maps, pairs, s);
  }
}

}  // namespace muon
