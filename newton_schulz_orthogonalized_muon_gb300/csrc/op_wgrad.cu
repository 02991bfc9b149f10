// The weight's gradient of a linear layer from its input kept in 8 bits:
//   dw[o][n] = sum over tokens t of dy[t][o] x[t][n]  (+ add[o][n]),
//   x[t][n] = code[t][n] 2^(scale[n / 128][t] - 127), exact in bf16.
//
// A product on the tensor cores, 256 x 256 outputs a CTA pair
// (tcgen05.mma.cta_group::2), 64 tokens a step.  dy and the codes come by
// TMA; eight warps a CTA turn its 128 columns of codes into bf16 and write
// them back to shared memory in the layout that TMA would have given a bf16
// operand.  (Loading the codes straight into registers saves a pass through
// shared memory, but the fence that hands the written operand to the tensor
// core also waits for a thread's loads in flight: 4.0 ms at 16384 x 4096 x
// 14336.)  Both operands have tokens, the summed index, as rows: they are
// read MN-major.
//
// The tensor core adds each 16-token product to its fp32 accumulator with
// truncation, an error that grows with the number of additions.  So after
// every 2048 tokens the accumulator is handed to the epilogue warps, which
// add it to a running sum in registers (128 values a thread) with rounding,
// while the other of two accumulators takes the next tokens.
//
// Few tiles and many tokens: the tokens are split over several pairs, whose
// fp32 partial results a second kernel adds in a fixed order.
//
// 16384 tokens, 4096 columns, 14336 outputs in 1.19 ms, 1620 TFLOP/s, bound by
// the products (and, in calls that follow one another, by the power limit: 1.26
// to 1.28 ms); 1001 x 2048 x 1408 with `add` in 21 us with cold caches (18 in
// calls that follow one another), of which 14 are a CTA's start, first loads
// and epilogue.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"
#include "op_common.cuh"
#include "op_pair.cuh"

namespace muon {
namespace {

constexpr int BK = 64;                   // tokens a step
constexpr int STEPS_SUM = 32;            // steps an accumulator takes: 2048 tokens
constexpr int PT = 256;                  // a pair's tile: 256 x 256
constexpr int CODE_WARPS = 8, EPI_WARPS = 8;
constexpr int THREADS = 32 * (4 + CODE_WARPS + EPI_WARPS);
constexpr int BOX = 64 * 128;            // 64 tokens x 64 16-bit (128 8-bit) columns
// rings, of this CTA's 128 columns of a step: dy and codes, which come from
// global memory, deep; the converted x shallow
constexpr int DY_STAGES = 5, CODE_STAGES = 6, X_STAGES = 4;
// The code warps work in groups on alternate steps: a step's way through one
// warp (barrier, shared memory, conversion, fence) takes about 1000 cycles,
// twice what its products take.
constexpr int GROUPS = 2, GROUP_WARPS = CODE_WARPS / GROUPS;
constexpr int TOK = 8 / GROUP_WARPS;     // sets of eight tokens a warp takes of a step
static_assert(CODE_STAGES % GROUPS == 0 && X_STAGES % GROUPS == 0, "a group keeps to its stages");
constexpr int CODE_OFF = DY_STAGES * 2 * BOX;
constexpr int X_OFF = CODE_OFF + CODE_STAGES * BOX;
constexpr int SLOT = 4096;               // 32 x 32 fp32 of an epilogue warp
constexpr int EPI_OFF = X_OFF + X_STAGES * 2 * BOX;
constexpr int SCALE_OFF = EPI_OFF + EPI_WARPS * SLOT;
constexpr int BAR_OFF = SCALE_OFF + CODE_STAGES * BK;
constexpr int SMEM = BAR_OFF + 512;
constexpr unsigned long long DRAIN_NS = 1000000000ull;
static_assert(SMEM <= 232448, "shared memory");

struct alignas(16) Bars {
  uint64_t dy_full[DY_STAGES], dy_empty[DY_STAGES];         // full: the leader's, for both CTAs
  uint64_t code_full[CODE_STAGES], code_empty[CODE_STAGES]; // each CTA's own
  uint64_t x_full[X_STAGES], x_empty[X_STAGES];             // full: the leader's, for both CTAs
  uint64_t x_here[X_STAGES];                                // the other CTA's: its half of x is written
  uint4 token[2];                                           // sent, received (see send_token)
  uint64_t tfull[2], tempty[2];
  uint64_t drain;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Bars) <= 512, "barrier block");

// 16 codes to 16 bf16, times `unit`, a power of two (exact; infinity for a
// block that held a NaN or an infinity, whose codes are 0).  By way of fp16
// and fp32: six instructions a pair, two of them on the ALU pipe that bounds
// the conversion (placing the bits of two codes in bf16 takes four there).
__device__ __forceinline__ void convert16(const uint4& c, float unit, uint32_t* r) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const __half2 h = __half2(
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[k >> 1] >> (16 * (k & 1))), __NV_E4M3));
    const float2 f = __half22float2(h);
    r[k] = pack_bf16x2(f.x * unit, f.y * unit);
  }
}

// A 32 x 32 block of fp32 values in a warp's slot of shared memory, its
// 16-byte chunks swizzled: lanes read and write either a row each or, eight
// lanes a row, parts of rows that are next to each other in memory.
__device__ __forceinline__ uint32_t slot_at(int row, int chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }

// The block of `add` from (o, n) into the slot, zeros outside it.
__device__ __forceinline__ void load_block(const WgradParams& p, uint8_t* slot, int o, int n, int lane) {
  const int r = lane >> 3, q = lane & 7;
  const long long at = static_cast<long long>(o + r) * p.ldadd + n + 4 * q;
  const bool inside = p.vec_add && o + 32 <= p.out && n + 32 <= p.cols;
  if (inside && p.odtype == DT_F32) {
    float4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.add) + at + 4 * i * p.ldadd);
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<float4*>(slot + slot_at(r + 4 * i, q)) = x[i];
    return;
  }
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    float* to = reinterpret_cast<float*>(slot + slot_at(r + 4 * i, q));
#pragma unroll 1
    for (int e = 0; e < 4; ++e)
      to[e] = o + r + 4 * i < p.out && n + 4 * q + e < p.cols ? load_f32(p.add, at + 4 * i * p.ldadd + e, p.odtype) : 0.f;
  }
}

// The slot out to the block of dw (or of a split's partial results) from (o, n).
__device__ __forceinline__ void store_block(const WgradParams& p, float* part, const uint8_t* slot, int o, int n, int lane) {
  const int r = lane >> 3, q = lane & 7;
  const int dtype = part != nullptr ? DT_F32 : p.odtype;
  const long long ld = part != nullptr ? p.cols : p.ldw;
  void* out = part != nullptr ? part : p.dw;
  const long long at = static_cast<long long>(o + r) * ld + n + 4 * q;
  const bool vec = part != nullptr ? (p.cols & 3) == 0 : p.vec != 0;
  if (vec && n + 32 <= p.cols && dtype == DT_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (o + r + 4 * i < p.out)
        *reinterpret_cast<float4*>(static_cast<float*>(out) + at + 4 * i * ld) =
            *reinterpret_cast<const float4*>(slot + slot_at(r + 4 * i, q));
    return;
  }
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    if (o + r + 4 * i >= p.out) break;
    const float4 v = *reinterpret_cast<const float4*>(slot + slot_at(r + 4 * i, q));
    if (vec && n + 32 <= p.cols) {
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at + 4 * i * ld) =
          make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    } else {
      const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + 4 * q + e < p.cols) store_from_f32(out, at + 4 * i * ld + e, dtype, f[e]);
    }
  }
}

struct Item {
  int o, n;              // tile indices
  int k0, k1;            // steps [k0, k1)
  int split;
};

// Tiles go eight output blocks at a time, the pairs that run together share
// dy and x panels in L2; splits of one tile are neighbours.  (In 32 bits, and
// without divisions by splits that there are not: every warp starts with this,
// and 64-bit divisions held the first load for 3000 cycles.)
__device__ __forceinline__ Item item_of(const WgradParams& p, uint32_t i) {
  Item t{0, 0, 0, static_cast<int>((p.rows + BK - 1) / BK), 0};
  if (p.splits > 1) {
    // steps * splits stays below 2^32: at most 2^24 steps, and fewer splits than SMs
    const uint32_t n = static_cast<uint32_t>(p.splits), steps = static_cast<uint32_t>(t.k1), split = i % n;
    i /= n;
    t.split = static_cast<int>(split);
    t.k0 = static_cast<int>(steps * split / n);
    t.k1 = static_cast<int>(steps * (split + 1) / n);
  }
  const uint32_t per = 8u * static_cast<uint32_t>(p.tiles_n), band = i / per, in = i - band * per;
  const uint32_t rows = min(8u, static_cast<uint32_t>(p.tiles_o) - band * 8u);
  const uint32_t n = rows == 8u ? in >> 3 : in / rows;
  t.n = static_cast<int>(n);
  t.o = static_cast<int>(band * 8u + in - n * rows);
  return t;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    act8_wgrad_kernel(const __grid_constant__ CUtensorMap mdy, const __grid_constant__ CUtensorMap mcode,
                      const WgradParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* bar = reinterpret_cast<Bars*>(smem + BAR_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = static_cast<int>(cluster_id_x()), npairs = static_cast<int>(num_clusters_x());
  const uint32_t sb = smem_u32(smem);
  if (threadIdx.x == 0) {
    for (int s = 0; s < DY_STAGES; ++s) {
      mbar_init(&bar->dy_full[s], 1);
      mbar_init(&bar->dy_empty[s], 1);
    }
    for (int s = 0; s < CODE_STAGES; ++s) {
      mbar_init(&bar->code_full[s], 2);            // codes, scales
      mbar_init(&bar->code_empty[s], GROUP_WARPS);
    }
    for (int s = 0; s < X_STAGES; ++s) {
      mbar_init(&bar->x_full[s], GROUP_WARPS);     // and the other CTA's token
      mbar_init(&bar->x_here[s], GROUP_WARPS);
      mbar_init(&bar->x_empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&bar->tfull[a], 1);
      mbar_init(&bar->tempty[a], 2 * EPI_WARPS);
    }
    mbar_init(&bar->drain, 1);
    bar->token[0] = make_uint4(0u, 0u, 0u, 0u);
    bar->abort = (sb & 1023u) != 0u ? 1 : 0;       // the swizzled boxes need 1 KB boundaries
    if (bar->abort) atomicOr(p.err, ERRBIT_TIMEOUT);
    fence_mbar_init();
  }
  pdl_launch_dependents();
  if (warp == 0) tmem_alloc_pair(&bar->tmem, 512);
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = bar->tmem;
  volatile int* abort = &bar->abort;
  const int items = p.tiles_o * p.tiles_n * p.splits;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
    if (warp != 1) {
      if (lane == 0) {
        // Loads: warp 0 dy, warp 2 codes, warp 3 scales.  (One thread for
        // all three took 1000 cycles a step, twice what the products take.)
        Ring<DY_STAGES> rd;
        Ring<CODE_STAGES> rc;
        bool ok = true;
        if (warp == 0) pdl_wait();                 // dy may come from the padding kernel
        const uint32_t lead = mapa_shared(smem_u32(&bar->dy_full[0]), 0);
        for (int i = pair; ok && i < items; i += npairs) {
          const Item t = item_of(p, i);
          const int blk = 2 * t.n + static_cast<int>(rank);
          if (warp == 0) {
            const int o0 = t.o * PT + static_cast<int>(rank) * 128;
            for (int k = t.k0; k < t.k1; ++k) {
              ok = wait_one(&bar->dy_empty[rd.s], rd.ph ^ 1u, abort, p);
              if (!ok) break;
              const uint32_t fb = lead + rd.s * 8;
              if (rank == 0) mbar_arrive_expect_tx(&bar->dy_full[rd.s], 4 * BOX);
              tma_load_3d_pair(sb + rd.s * 2 * BOX, &mdy, fb, o0, k * BK, 0);
              tma_load_3d_pair(sb + rd.s * 2 * BOX + BOX, &mdy, fb, o0 + 64, k * BK, 0);
              rd.next();
            }
          } else {
            const uint8_t* from = p.scales + blk * p.lds;
            const bool live = blk * 128 < p.cols;
            for (int k = t.k0; k < t.k1; ++k) {
              ok = wait_one(&bar->code_empty[rc.s], rc.ph ^ 1u, abort, p);
              if (!ok) break;
              uint64_t* cf = &bar->code_full[rc.s];
              if (warp == 2) {
                mbar_arrive_expect_tx(cf, BOX);
                tma_load_3d(sb + CODE_OFF + rc.s * BOX, &mcode, cf, blk * 128, k * BK, 0);
              } else if (live) {
                // the step's scale bytes, whole 16-byte groups (lds is a multiple of them)
                const long long t0 = static_cast<long long>(k) * BK;
                const uint32_t bytes = p.rows - t0 >= BK ? BK : static_cast<uint32_t>((p.rows - t0 + 15) / 16 * 16);
                mbar_arrive_expect_tx(cf, bytes);
                bulk_load(sb + SCALE_OFF + rc.s * BK, from + t0, bytes, smem_u32(cf));
              } else {
                mbar_arrive(cf);
              }
              rc.next();
            }
          }
        }
      }
    } else if (rank != 0) {
      // ------------------------------- this CTA's halves of x, reported
      const uint32_t full = mapa_shared(smem_u32(&bar->x_full[0]), 0), to = mapa_shared(smem_u32(&bar->token[1]), 0);
      Ring<X_STAGES> rx;
      bool ok = true;
      for (int i = pair; ok && i < items; i += npairs) {
        const Item t = item_of(p, i);
        for (int k = t.k0; k < t.k1; ++k) {
          ok = wait_warp(&bar->x_here[rx.s], rx.ph, abort, p);
          if (!ok) break;
          if (lane == 0) send_token(to, smem_u32(&bar->token[0]), full + rx.s * 8);
          __syncwarp();
          rx.next();
        }
      }
    } else {
      // ----------------------------------------------------- products
      // both operands MN-major; M = 256 over the pair, N = 256
      const uint32_t id = idesc_bf16_f32(PT, PT, 1) | (1u << 15);
      Ring<DY_STAGES> rd;
      Ring<X_STAGES> rx;
      int acc = 0;
      uint32_t acc_ph = 0;
      bool ok = true;
      for (int i = pair; ok && i < items; i += npairs) {
        const Item t = item_of(p, i);
        for (int k0 = t.k0; ok && k0 < t.k1; k0 += STEPS_SUM) {
          ok = wait_warp<0, true>(&bar->tempty[acc], acc_ph ^ 1u, abort, p);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + acc * PT;
          const int k1 = min(k0 + STEPS_SUM, t.k1);
          for (int k = k0; k < k1; ++k) {
            ok = wait_warp(&bar->dy_full[rd.s], rd.ph, abort, p) && wait_warp<0, true>(&bar->x_full[rx.s], rx.ph, abort, p);
            if (!ok) break;
            tc_fence_after();
            const uint64_t a = sdesc_sw128(sb + rd.s * 2 * BOX, BOX, 1024);
            const uint64_t b = sdesc_sw128(sb + X_OFF + rx.s * 2 * BOX, BOX, 1024);
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              mma_pair(d, a + kk * (2048 >> 4), b + kk * (2048 >> 4), id, kk != 0 || k != k0 ? 1u : 0u);
            commit_pair(&bar->x_empty[rx.s], 0x3);
            commit_pair(&bar->dy_empty[rd.s], 0x3);
            rd.next();
            rx.next();
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
  } else if (warp < 4 + CODE_WARPS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    // ------------------------------------------------ codes to bf16
    // A chunk is 16 columns of a token.  Eight lanes hold eight tokens of one
    // chunk column, so that their swizzled 16-byte accesses fall on different
    // banks; a thread has chunk columns j and j + 4 of TOK tokens.
    const int cw = warp - 4, group = cw / GROUP_WARPS;
    const int r0 = (cw % GROUP_WARPS) * 8 * TOK + (lane & 7), j = lane >> 3;
    // byte offsets of token r0 in a stage: chunk columns j and j + 4 of the
    // codes; the 16-byte chunks 2 j and 2 j + 1 of its rows in both boxes of x
    const uint32_t row = r0 * 128, sw = lane & 7;
    const uint32_t from0 = CODE_OFF + row + ((j ^ sw) << 4), from1 = CODE_OFF + row + (((j + 4) ^ sw) << 4);
    const uint32_t to0 = X_OFF + row + (((2 * j) ^ sw) << 4), to1 = X_OFF + row + (((2 * j + 1) ^ sw) << 4);
    Ring<CODE_STAGES> rc;
    Ring<X_STAGES> rx;
    rc.s = rx.s = group;
    int turn = 0;
    bool ok = true;
    for (int i = pair; ok && i < items; i += npairs) {
      const Item t = item_of(p, i);
      const bool live = (2 * t.n + static_cast<int>(rank)) * 128 < p.cols;
      for (int k = t.k0; k < t.k1; ++k) {
        const bool mine = turn == group;
        if (++turn == GROUPS) turn = 0;
        if (!mine) continue;
        ok = wait_warp(&bar->code_full[rc.s], rc.ph, abort, p);
        if (!ok) break;
        ok = wait_warp(&bar->x_empty[rx.s], rx.ph ^ 1u, abort, p);
        if (!ok) break;
        const uint32_t src = sb + rc.s * BOX, dst = sb + rx.s * 2 * BOX;
        // tokens of this step that exist, from r0 on; none in a block past the last: no scale is there
        const long long left = live ? p.rows - static_cast<long long>(k) * BK - r0 : 0;
        const uint8_t* sc = smem + SCALE_OFF + rc.s * BK + r0;
        // kept a short loop: twenty warps of three kinds share the instruction cache
#pragma unroll 1
        for (int q = 0; q < 8 * TOK; q += 8) {
          const uint4 ca = lds16(src + from0 + q * 128), cb = lds16(src + from1 + q * 128);
          const float unit = __int_as_float(q < left ? sc[q] << 23 : 0);
          uint32_t r[16];
          convert16(ca, unit, r);
          convert16(cb, unit, r + 8);
          sts16(dst + to0 + q * 128, r);
          sts16(dst + to1 + q * 128, r + 4);
          sts16(dst + to0 + q * 128 + BOX, r + 8);
          sts16(dst + to1 + q * 128 + BOX, r + 12);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (rank != 0)
            mbar_arrive(&bar->x_here[rx.s]);
          else if (cw % GROUP_WARPS == 0)
            mbar_arrive_expect_tx(&bar->x_full[rx.s], sizeof(uint4));
          else
            mbar_arrive(&bar->x_full[rx.s]);
          mbar_arrive(&bar->code_empty[rc.s]);
        }
        rc.next(GROUPS);
        rx.next(GROUPS);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    // ------------------------------------------------------- epilogue
    const int ew = warp - 4 - CODE_WARPS, quad = warp & 3, half = ew >> 2;
    uint8_t* slot = smem + EPI_OFF + ew * SLOT;
    const uint32_t te[2] = {mapa_shared(smem_u32(&bar->tempty[0]), 0), mapa_shared(smem_u32(&bar->tempty[1]), 0)};
    int acc = 0;
    uint32_t acc_ph = 0;
    bool ok = true;
    for (int i = pair; ok && i < items; i += npairs) {
      const Item t = item_of(p, i);
      const int o0 = t.o * PT + static_cast<int>(rank) * 128 + quad * 32;
      const int n0 = t.n * PT + half * 128;
      // a running sum starts from `add`, read while the first products run
      float v[128];
      const bool add = p.add != nullptr && p.splits == 1;
#pragma unroll
      for (int c = 0; c < 128; c += 32) {
        if (add) {
          __syncwarp();
          load_block(p, slot, o0, n0 + c, lane);
          __syncwarp();
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float4 x = add ? *reinterpret_cast<const float4*>(slot + slot_at(lane, q)) : make_float4(0.f, 0.f, 0.f, 0.f);
          v[c + 4 * q] = x.x;
          v[c + 4 * q + 1] = x.y;
          v[c + 4 * q + 2] = x.z;
          v[c + 4 * q + 3] = x.w;
        }
      }
      for (int k0 = t.k0; k0 < t.k1; k0 += STEPS_SUM) {
        ok = wait_warp<500>(&bar->tfull[acc], acc_ph, abort, p);
        if (!ok) break;
        tc_fence_after();
        const uint32_t at = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * PT + half * 128;
#pragma unroll
        for (int c = 0; c < 128; c += 16) {
          float w[16];
          tmem_ld16(at + c, w);
#pragma unroll
          for (int e = 0; e < 16; ++e) v[c + e] += w[e];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(te[acc]);
        acc ^= 1;
        if (acc == 0) acc_ph ^= 1u;
      }
      if (!ok) break;
      // out through shared memory, 32 x 32 at a time
      float* part = p.splits > 1 ? p.part + static_cast<long long>(t.split) * p.out * p.cols : nullptr;
#pragma unroll
      for (int c = 0; c < 128; c += 32) {
        if (n0 + c >= p.cols || o0 >= p.out) continue;
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q)
          *reinterpret_cast<float4*>(slot + slot_at(lane, q)) =
              make_float4(v[c + 4 * q], v[c + 4 * q + 1], v[c + 4 * q + 2], v[c + 4 * q + 3]);
        __syncwarp();
        store_block(p, part, slot, o0, n0 + c, lane);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // after a wait ran out, whichever warp's it was: copies in flight (their
  // barriers may never complete, the peer's part missing) get a millisecond
  // to land before the pair's memory is given up; none is issued any more
  if (threadIdx.x == 0 && *abort != 0) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {
    }
  }
  __syncwarp();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 0) tmem_dealloc_pair(tmem, 512);
}

// dw = add + the splits' partial results, in their order.  (Splits are for few
// tiles: outputs fit 32 bits.)
__global__ void __launch_bounds__(256) act8_wgrad_join_kernel(const WgradParams p) {
  const uint32_t cols = static_cast<uint32_t>(p.cols), count = static_cast<uint32_t>(p.out) * cols;
  pdl_wait();                            // launched while the partial results are still being formed
  for (uint32_t i = blockIdx.x * 256u + threadIdx.x; i < count; i += gridDim.x * 256u) {
    const uint32_t o = i / cols, n = i - o * cols;
    float v = 0.f;
#pragma unroll 8
    for (int s = 0; s < p.splits; ++s) v += p.part[static_cast<long long>(s) * count + i];
    if (p.add != nullptr) v += load_f32(p.add, o * p.ldadd + n, p.odtype);
    store_from_f32(p.dw, o * p.ldw + n, p.odtype, v);
  }
}

// dy with rows on 16-byte boundaries, for TMA: a warp a row, eight elements a lane.
__global__ void __launch_bounds__(256) pad_rows_kernel(const __nv_bfloat16* src, long long lds, __nv_bfloat16* dst,
                                                       long long ldd, long long rows, int cols) {
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  for (long long r = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); r < rows;
       r += static_cast<long long>(gridDim.x) * 8) {
    const __nv_bfloat16* from = src + r * lds;
    for (int c = lane * 8; c < cols; c += 256) {
      float f[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = c + k < cols ? to_f32(from[c + k]) : 0.f;
      *reinterpret_cast<uint4*>(dst + r * ldd + c) = pack16<__nv_bfloat16>(f);
    }
  }
}

}  // namespace

int wgrad_splits(long long rows, int cols, int out, int pairs) {
  const long long tiles = static_cast<long long>((out + PT - 1) / PT) * ((cols + PT - 1) / PT);
  const long long steps = (rows + BK - 1) / BK;
  // as many splits as there are pairs for each tile, of at least eight steps
  long long s = pairs / tiles;
  if (s > steps / 8) s = steps / 8;
  return s < 1 ? 1 : static_cast<int>(s);
}

cudaError_t launch_pad_rows(const __nv_bfloat16* src, long long lds, __nv_bfloat16* dst, long long ldd, long long rows,
                            int cols, int sms, cudaStream_t s) {
  const long long want = (rows + 7) / 8;
  pad_rows_kernel<<<static_cast<unsigned>(want < sms * 8LL ? want : sms * 8LL), 256, 0, s>>>(src, lds, dst, ldd, rows,
                                                                                             cols);
  return cudaGetLastError();
}

cudaError_t launch_act8_wgrad(const WgradParams& q, const CUtensorMap* maps, bool padded, int pairs, cudaStream_t s) {
  WgradParams p = q;
  p.tiles_o = (p.out + PT - 1) / PT;
  p.tiles_n = (p.cols + PT - 1) / PT;
  const long long items = static_cast<long long>(p.tiles_o) * p.tiles_n * p.splits;
  if (items > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const long long es = p.odtype == DT_F32 ? 4 : 2;
  p.vec = reinterpret_cast<uintptr_t>(p.dw) % (4 * es) == 0 && p.ldw % 4 == 0;
  p.vec_add = reinterpret_cast<uintptr_t>(p.add) % 16 == 0 && p.ldadd * es % 16 == 0;
  static std::atomic<unsigned long long> done;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(act8_wgrad_kernel), SMEM, done);
  if (e != cudaSuccess) return e;
  const cudaError_t l = launch_k(padded && pdl_level() >= 1, act8_wgrad_kernel, dim3(2 * static_cast<unsigned>(items < pairs ? items : pairs)),
                                 dim3(THREADS), SMEM, s, maps[0], maps[1], p);
  return l != cudaSuccess ? l : cudaGetLastError();
}

cudaError_t launch_act8_wgrad_join(const WgradParams& p, int sms, cudaStream_t s) {
  const long long want = (static_cast<long long>(p.out) * p.cols + 255) / 256;
  const cudaError_t e = launch_k(pdl_level() >= 1, act8_wgrad_join_kernel, dim3(static_cast<unsigned>(want < sms * 8LL ? want : sms * 8LL)),
                                 dim3(256), 0, s, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace muon
