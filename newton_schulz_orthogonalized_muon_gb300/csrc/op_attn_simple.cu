// Attention, forward and backward, one warp a query (or key) row.
//
//   s_ij = scale q_i . k_j for the keys that query i sees, lse_i = log sum_j
//   exp(s_ij), o_i = sum_j exp(s_ij - lse_i) v_j
//   delta_i = do_i . o_i,  p_ij = exp(s_ij - lse_i),
//   dv_j = sum_i p_ij do_i,  ds_ij = p_ij (do_i . v_j - delta_i) scale,
//   dq_i = sum_j ds_ij k_j,  dk_j = sum_i ds_ij q_i
// Query i of a sequence with sq queries and sk keys stands at place
// i + sk - sq; causal: it sees the keys up to its place, with a window only
// the last `window` of them.  A query that sees no key has o = 0, lse = -inf
// and no part in any gradient.
#include "common.cuh"
#include "internal.h"
#include "op_attn.cuh"
#include "op_common.cuh"

namespace muon {
namespace {

constexpr int MAXE = 4;           // 128 / 32 elements of a row a lane

template <typename T>
__device__ __forceinline__ void load_row(const void* base, long long off, int dim, float* f) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int e = 0; e < MAXE; ++e) f[e] = lane + 32 * e < dim ? to_f32(static_cast<const T*>(base)[off + lane + 32 * e]) : 0.f;
}
template <typename T>
__device__ __forceinline__ void store_row(void* base, long long off, int dim, const float* f) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int e = 0; e < MAXE; ++e)
    if (lane + 32 * e < dim) static_cast<T*>(base)[off + lane + 32 * e] = from_f32<T>(f[e]);
}
__device__ __forceinline__ float dot(const float* a, const float* b) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < MAXE; ++e) s = fmaf(a[e], b[e], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// The sequence that token t of the packed axis belongs to, or of the batch.
struct Seq {
  int b;                // batch index (0 when packed)
  int q0, k0, nq, nk;   // first token and length, on each axis
};

__device__ Seq seq_of(const AttnParams& p, int index, bool of_query, int token) {
  if (p.cu_q == nullptr) return Seq{index, 0, 0, p.sq, p.sk};
  for (int i = 0; i < p.batch; ++i) {
    const Span a = span_of(p.cu_q, i, p.sq), b = span_of(p.cu_k, i, p.sk);
    const Span& m = of_query ? a : b;
    if (token >= m.start && token < m.start + m.len) return Seq{0, a.start, b.start, a.len, b.len};
  }
  return Seq{0, 0, 0, 0, 0};
}

// mode 0: forward; 1: dq and delta; 2: dk and dv
template <typename T, int MODE>
__global__ void __launch_bounds__(128) attn_row_kernel(const AttnParams p) {
  const int token = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int h = blockIdx.y, b = blockIdx.z;
  if (token >= (MODE == 2 ? p.sk : p.sq)) return;
  const Seq s = seq_of(p, b, MODE != 2, token);
  const int d = p.dim, group = p.heads / p.kv_heads;
  if constexpr (MODE != 2) {
    const int hk = h / group, i = token - s.q0;
    const long long qo = s.b * p.qb + token * p.qs + h * p.qh;
    float q[MAXE], acc[MAXE] = {0.f, 0.f, 0.f, 0.f};
    load_row<T>(p.q, qo, d, q);
    const Keys see = keys_of(p, i, s.nq, s.nk);
    if (MODE == 0) {
      float m = -INFINITY, l = 0.f;
      for (int j = see.first; j < see.end; ++j) {
        float k[MAXE], v[MAXE];
        load_row<T>(p.k, s.b * p.kb + (s.k0 + j) * p.ks + hk * p.kh, d, k);
        load_row<T>(p.v, s.b * p.vb + (s.k0 + j) * p.vs + hk * p.vh, d, v);
        const float x = dot(q, k) * p.scale;
        const float mn = fmaxf(m, x);
        const float c = expf(m - mn), e = expf(x - mn);
        l = l * c + e;
        for (int a = 0; a < MAXE; ++a) acc[a] = acc[a] * c + e * v[a];
        m = mn;
      }
      for (int a = 0; a < MAXE; ++a) acc[a] = l > 0.f || l != l ? acc[a] / l : 0.f;
      store_row<T>(p.out, s.b * p.ob + token * p.os + h * p.oh, d, acc);
      if (lane == 0) p.lse[b * p.lse_b + h * p.lse_h + token] = see.end > see.first ? m + logf(l) : -INFINITY;
    } else {
      float g[MAXE], o[MAXE];
      load_row<T>(p.dout, s.b * p.dob + token * p.dos + h * p.doh, d, g);
      load_row<T>(p.o, s.b * p.ob + token * p.os + h * p.oh, d, o);
      const float delta = dot(g, o), lse = p.lse[b * p.lse_b + h * p.lse_h + token];
      if (lane == 0) p.delta[b * p.lse_b + h * p.lse_h + token] = delta;
      for (int j = see.first; j < see.end; ++j) {
        float k[MAXE], v[MAXE];
        load_row<T>(p.k, s.b * p.kb + (s.k0 + j) * p.ks + hk * p.kh, d, k);
        load_row<T>(p.v, s.b * p.vb + (s.k0 + j) * p.vs + hk * p.vh, d, v);
        const float pr = expf(dot(q, k) * p.scale - lse);
        const float ds = pr * (dot(g, v) - delta) * p.scale;
        for (int a = 0; a < MAXE; ++a) acc[a] = fmaf(ds, k[a], acc[a]);
      }
      store_row<T>(p.dq, s.b * p.dqb + token * p.dqs + h * p.dqh, d, acc);
    }
  } else {
    const int j = token - s.k0;
    float k[MAXE], v[MAXE], dk[MAXE] = {0.f, 0.f, 0.f, 0.f}, dv[MAXE] = {0.f, 0.f, 0.f, 0.f};
    load_row<T>(p.k, s.b * p.kb + token * p.ks + h * p.kh, d, k);
    load_row<T>(p.v, s.b * p.vb + token * p.vs + h * p.vh, d, v);
    for (int hq = h * group; hq < (h + 1) * group; ++hq) {
      for (int i = 0; i < s.nq; ++i) {
        const Keys see = keys_of(p, i, s.nq, s.nk);
        if (j < see.first || j >= see.end) continue;
        const int tq = s.q0 + i;
        float q[MAXE], g[MAXE];
        load_row<T>(p.q, s.b * p.qb + tq * p.qs + hq * p.qh, d, q);
        load_row<T>(p.dout, s.b * p.dob + tq * p.dos + hq * p.doh, d, g);
        const float pr = expf(dot(q, k) * p.scale - p.lse[b * p.lse_b + hq * p.lse_h + tq]);
        const float ds = pr * (dot(g, v) - p.delta[b * p.lse_b + hq * p.lse_h + tq]) * p.scale;
        for (int a = 0; a < MAXE; ++a) {
          dk[a] = fmaf(ds, q[a], dk[a]);
          dv[a] = fmaf(pr, g[a], dv[a]);
        }
      }
    }
    store_row<T>(p.dk, s.b * p.dkb + token * p.dks + h * p.dkh, d, dk);
    store_row<T>(p.dv, s.b * p.dvb + token * p.dvs + h * p.dvh, d, dv);
  }
}

template <int MODE>
cudaError_t launch_mode(const AttnParams& p, cudaStream_t s) {
  const int n = MODE == 2 ? p.sk : p.sq;
  if (n == 0) return cudaSuccess;
  const dim3 grid((n + 3) / 4, MODE == 2 ? p.kv_heads : p.heads, p.cu_q != nullptr ? 1 : p.batch);
  if (p.dtype == DT_BF16)
    attn_row_kernel<__nv_bfloat16, MODE><<<grid, 128, 0, s>>>(p);
  else
    attn_row_kernel<__half, MODE><<<grid, 128, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_fwd(const AttnParams& p, cudaStream_t s) { return launch_mode<0>(p, s); }
cudaError_t launch_attn_bwd(const AttnParams& p, cudaStream_t s) {
  const cudaError_t e = launch_mode<1>(p, s);
  return e != cudaSuccess ? e : launch_mode<2>(p, s);
}

}  // namespace muon
