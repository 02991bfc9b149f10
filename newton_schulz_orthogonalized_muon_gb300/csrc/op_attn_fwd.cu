// Attention, forward: o_i = sum_j p_ij v_j, p_ij = exp(scale q_i . k_j -
// lse_i), in one pass over the keys with a running maximum and sum.
//
// A CTA owns two tiles of 128 queries of one head and walks the key tiles
// that they see.  Warp 0 loads by TMA, warp 1 issues every tcgen05.mma, and
// each tile has a warpgroup of its own (warps 4 - 7, 8 - 11) with one thread a
// query: while one tile's scores go through the exponential, the tensor pipe
// works for the other.  The scores (fp32) and o
// stay in TMEM; the probabilities are rounded to the operands' 16-bit type
// and written over the scores, from where the second product takes them as
// its A operand.  The row sum is taken from the probabilities before they
// are rounded.
//
// The maximum that a row's exponents are taken against is raised only when a
// new score passes it by more than 2^8 (in exp2 units): o and the sum are
// then scaled down in TMEM.  Below that the probabilities stay under 256,
// exact in the same relative precision, and o is left alone.
//
// Bound by the tensor cores and the exponentials alike: a 128 x 128 tile
// pair with dim 128 takes 1024 cycles of products and 16384 exponentials.
// Measured: 8192 causal tokens of 32 heads (8 of keys), dim 128, bf16, in
// 371 us, 1480 TFLOP/s of the visible pairs' products.
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
constexpr float RAISE = 8.f;

template <int DP>
struct Smem {
  static constexpr int T = tile_bytes<DP>();
  static constexpr int RK = 3;
  static constexpr int RV = DP == 128 ? 2 : 3;
  static constexpr int K_OFF = 2 * T;
  static constexpr int V_OFF = K_OFF + RK * T;
  static constexpr int BAR_OFF = V_OFF + RV * T;
  static constexpr int BYTES = BAR_OFF + 256;
  static_assert(BYTES <= 232448, "shared memory");
};

struct Bars {
  uint64_t q_full[2];
  uint64_t k_full[3], k_empty[3], v_full[3], v_empty[3];
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t drain, edge;
  uint32_t tmem;
  int abort;
  Work work;
};
static_assert(sizeof(Bars) <= 256, "barrier block");
// shared-memory address of a barrier; `bb` is the block's
#define BAR(f) (bb + static_cast<uint32_t>(offsetof(Bars, f)))

template <typename T, int DP>
__global__ void __launch_bounds__(THREADS, 1)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv, const AttnParams p, int tiles) {
  using S = Smem<DP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* bar = reinterpret_cast<Bars*>(smem + S::BAR_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sb = smem_u32(smem), bb = sb + S::BAR_OFF;
  if (!swizzle_aligned(sb, p)) return;
  if (warp == 0) {
    const Work w = find_work(p, true, ROWS, p.heads, tiles, blockIdx.x);
    if (lane == 0) {
      bar->work = w;
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bar->q_full[i], 1);
        mbar_init(&bar->s_full[i], 1);
        mbar_init(&bar->p_full[i], 4);
        mbar_init(&bar->o_done[i], 1);
      }
      for (int i = 0; i < 3; ++i) {
        mbar_init(&bar->k_full[i], 1);
        mbar_init(&bar->k_empty[i], 1);
        mbar_init(&bar->v_full[i], 1);
        mbar_init(&bar->v_empty[i], 1);
      }
      mbar_init(&bar->drain, 1);
      mbar_init(&bar->edge, 1);
      bar->abort = 0;
      fence_mbar_init();
    }
  }
  if (warp == 1) tmem_alloc(&bar->tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Work w = bar->work;
  volatile int* abort = &bar->abort;
  const uint32_t tmem = bar->tmem;
  const int hk = w.h / (p.heads / p.kv_heads);
  const int i0 = w.tile * ROWS;
  // key tiles of each query tile, and of both
  Range r[2] = {{0, 0}, {0, 0}};
  if (w.ok) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
      if (i0 + t * TILE < w.nq) r[t] = key_tiles(p, w, i0 + t * TILE, min(i0 + (t + 1) * TILE, w.nq) - 1);
  }
  int beg = 0, end = 0;
  if (r[0].count > 0 || r[1].count > 0) {
    beg = r[0].count == 0 ? r[1].first : r[1].count == 0 ? r[0].first : min(r[0].first, r[1].first);
    end = max(r[0].first + r[0].count, r[1].first + r[1].count);
  }
  const int n = end - beg;
  auto sees = [&](int t, int tile) { return tile >= r[t].first && tile < r[t].first + r[t].count; };

  // a softmax thread holds a row of 128 scores: registers move from the
  // control warps (4 x 32 x 88 + 8 x 32 x 200 of the 384 x 168 at launch)
  if (warp < CTRL_WARPS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0 && n > 0) {
      // ---------------------------------------------------------- loads
      if (lane == 0) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (r[t].count > 0) {
            mbar_expect_at(BAR(q_full) + 8 * t, S::T);
            load_tile<DP>(sb + t * S::T, &mq, BAR(q_full) + 8 * t, w.h, w.q0 + i0 + t * TILE, w.b);
          }
        }
      }
      uint32_t edges = 0;
      int ik = 0, iv = 0;
      for (int i = 0; i < n; ++i) {
        const int j = (beg + i) * TILE, row = w.k0 + j, valid = w.nk - j;
        const int sk = i % S::RK, sv = i % S::RV;
        if (i >= S::RK && !wait_warp(BAR(k_empty) + 8 * sk, (i / S::RK - 1) & 1, abort, p)) break;
        if (lane == 0) {
          // rows past the sequence give scores that are masked, whatever they hold
          mbar_expect_at(BAR(k_full) + 8 * sk, S::T);
          load_tile<DP>(sb + S::K_OFF + sk * S::T, &mk, BAR(k_full) + 8 * sk, hk, row, w.b);
        }
        ++ik;
        if (i >= S::RV && !wait_warp(BAR(v_empty) + 8 * sv, (i / S::RV - 1) & 1, abort, p)) break;
        const bool edge = p.cu_q != nullptr && valid < TILE;
        const uint32_t vt = sb + S::V_OFF + sv * S::T, fv = BAR(v_full) + 8 * sv;
        if (lane == 0) {
          mbar_expect_at(edge ? BAR(edge) : fv, S::T);
          load_tile<DP>(vt, &mv, edge ? BAR(edge) : fv, hk, row, w.b);
        }
        if (edge) {
          if (!finish_edge_tile<DP>(vt, BAR(edge), edges, valid, abort, p)) break;
          if (lane == 0) mbar_arrive_at(fv);
        }
        ++iv;
      }
      if (*abort != 0 && lane == 0) {
        for (int t = 0; t < 2; ++t)
          if (r[t].count > 0) mbar_wait_bounded(&bar->q_full[t], 0, nullptr, DRAIN_NS);
        drain_ring<S::RK>(bar->k_full, ik);
        drain_ring<S::RV>(bar->v_full, iv);
      }
      __syncwarp();
    } else if (warp == 1 && n > 0) {
      // -------------------------------------------------------- products
      Ring<S::RK> rk;                              // the K tile of the scores to come
      Ring<S::RV> rv;
      uint32_t ph[2] = {0u, 0u}, acc[2] = {0u, 0u};
      auto scores = [&](int t) {
        mma_over_dim<T, DP>(tmem + t * TILE, desc_dim(sb + t * S::T), desc_dim(sb + S::K_OFF + rk.s * S::T));
        commit_warp(BAR(s_full) + 8 * t);
      };
      bool ok = wait_warp(BAR(k_full), 0, abort, p);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (ok && r[t].count > 0) ok = wait_warp(BAR(q_full) + 8 * t, 0, abort, p);
        if (ok && sees(t, beg)) {
          tc_fence_after();
          scores(t);
        }
      }
      if (ok) commit_warp(BAR(k_empty));
      rk.next();
      for (int tile = beg; ok && tile < end; ++tile) {
        const bool more = tile + 1 < end;
        // this step's tiles before the probabilities, so that no wait stands between products
        ok = wait_warp(BAR(v_full) + 8 * rv.s, rv.ph, abort, p) &&
             (!more || wait_warp(BAR(k_full) + 8 * rk.s, rk.ph, abort, p));
        if (!ok) break;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (ok && sees(t, tile)) {
            ok = wait_warp(BAR(p_full) + 8 * t, ph[t], abort, p);
            if (ok) {
              tc_fence_after();
              mma_over_tokens<T, DP, TILE>(tmem + 256 + t * TILE, tmem + t * TILE,
                                           desc_tokens(sb + S::V_OFF + rv.s * S::T), acc[t]);
              commit_warp(BAR(o_done) + 8 * t);
              ph[t] ^= 1u;
              acc[t] = 1u;
            }
          }
          // over the probabilities just used: the tensor pipe runs in order
          if (ok && more && sees(t, tile + 1)) scores(t);
        }
        if (!ok) break;
        commit_warp(BAR(v_empty) + 8 * rv.s);
        rv.next();
        if (more) {
          commit_warp(BAR(k_empty) + 8 * rk.s);
          rk.next();
        }
      }
      if (!ok) {
        commit_warp(BAR(drain));
        if (lane == 0) mbar_wait_bounded(&bar->drain, 0, nullptr, DRAIN_NS);
        __syncwarp();
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    if (w.ok) {
      // ------------------------------------------------ softmax, output
      const int t = (warp - CTRL_WARPS) >> 2, quad = warp & 3;
      const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
      const uint32_t s_at = tmem + lanes + t * TILE, o_at = tmem + lanes + 256 + t * TILE;
      const int q0 = i0 + t * TILE, q = q0 + quad * 32 + lane;
      const int off = w.nk - w.nq;
      const float c = p.scale * LOG2E;
      float top = -INFINITY;                         // the scores' reference, before scaling
      F2 sum2 = f2_make(0.f, 0.f);
      bool ok = true;
      const int cnt = r[t].count;
      for (int i = 0; i < cnt; ++i) {
        const int j0 = (r[t].first + i) * TILE;
        float v[TILE];
        ok = wait_warp(BAR(s_full) + 8 * t, i & 1, abort, p);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < TILE; k += 32) tmem_ld32(s_at + k, v + k);
        tmem_ld_wait();
        if (j0 + TILE > w.nk ||
            (p.causal && (j0 + TILE - 1 > q0 + off || (p.window > 0 && q0 + TILE - 1 + off - j0 >= p.window)))) {
          int lo = 0, hi = w.nk - j0;
          if (p.causal) {
            hi = min(hi, q + off + 1 - j0);
            if (p.window > 0) lo = q + off - p.window + 1 - j0;
          }
#pragma unroll
          for (int k = 0; k < TILE; ++k)
            if (k < lo || k >= hi) v[k] = -INFINITY;
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
          const bool up = mt > top && (top == -INFINITY || (mt - top) * c > RAISE);
          if (__any_sync(0xffffffffu, up)) {
            ok = wait_warp(BAR(o_done) + 8 * t, (i - 1) & 1, abort, p);
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
        const float ref = top == -INFINITY ? 0.f : -top * c;
        const F2 cc = f2_make(c, c), rr = f2_make(ref, ref);
#pragma unroll
        for (int k = 0; k < TILE; k += 64) {
#pragma unroll
          for (int e = k; e < k + 64; e += 2) {
            const float2 a = f2_split(f2_fma(f2_make(v[e], v[e + 1]), cc, rr));
            v[e] = exp2_fast(a.x);
            v[e + 1] = exp2_fast(a.y);
            sum2 = f2_add(sum2, f2_make(v[e], v[e + 1]));
          }
          store_rounded<T, 32>(s_at + k / 2, v + k);
        }
        warp_arrive(BAR(p_full) + 8 * t);
      }
      if (ok && cnt > 0) {
        ok = wait_warp(BAR(o_done) + 8 * t, (cnt - 1) & 1, abort, p);
        tc_fence_after();
      }
      if (ok) {
        const float2 s2 = f2_split(sum2);
        const float sum = s2.x + s2.y;
        const int first = q0 + quad * 32;          // of the warp's queries
        T* out = static_cast<T*>(p.out) + w.b * p.ob + static_cast<long long>(w.q0 + first) * p.os + w.h * p.oh;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        if (cnt > 0) {
          // through this tile's Q, which every product has read
#pragma unroll
          for (int x = 0; x < DP / 64; ++x)
            store_block<T>(o_at + 64 * x, sb + t * S::T + x * BOX_BYTES, quad * 32, out + 64 * x, p.os, w.nq - first,
                           p.dim - 64 * x, inv);
        } else if (q < w.nq) {
          for (int k = 0; k < p.dim; k += 8)
            *reinterpret_cast<uint4*>(out + lane * p.os + k) = make_uint4(0u, 0u, 0u, 0u);
        }
        if (q < w.nq)
          p.lse[w.b * p.lse_b + w.h * p.lse_h + w.q0 + q] =
              sum == 0.f ? -INFINITY : fmaf(top, p.scale, logf(sum));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <typename T, int DP>
cudaError_t launch_dims(const AttnParams& p, const CUtensorMap* m, cudaStream_t s) {
  const bool packed = p.cu_q != nullptr;
  const long long tiles = tile_bound(p.sq, ROWS, p.batch, packed);
  const long long items = tiles * p.heads * (packed ? 1 : p.batch);
  if (items > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  auto kern = attn_fwd_kernel<T, DP>;
  static std::atomic<unsigned long long> done;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), Smem<DP>::BYTES, done);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(items), THREADS, Smem<DP>::BYTES, s>>>(m[0], m[1], m[2], p, static_cast<int>(tiles));
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const AttnParams& p, const CUtensorMap* m, cudaStream_t s) {
  return p.dim <= 64 ? launch_dims<T, 64>(p, m, s) : launch_dims<T, 128>(p, m, s);
}

}  // namespace

int attn_qtiles(int sq, int batch, bool packed) { return static_cast<int>(tile_bound(sq, TILE, batch, packed)); }

cudaError_t launch_attn_fwd(const AttnParams& p, const CUtensorMap* m, cudaStream_t s) {
  return p.dtype == DT_BF16 ? launch_type<__nv_bfloat16>(p, m, s) : launch_type<__half>(p, m, s);
}

}  // namespace muon
