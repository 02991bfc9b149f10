// Layer norm, forward and backward, with the reduction of the weight's and
// the bias's gradient.
//
//   mu = mean(x), r = (mean((x - mu)^2) + eps)^(-1/2), xh = (x - mu) r
//   y = xh w + b
//   g = dy w,  dx = r (g - mean(g) - xh mean(g xh))
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Both directions are bound by HBM: the forward pass reads x and writes y, the
// backward pass reads x and dy and writes dx, and each element is touched
// once.  A row lives in the registers of TPR threads (EPT elements each);
// the mean is taken first and the squares about it second, with what the
// mean's rounding left over taken out, so that a large mean does not cancel.  CTAs are persistent: the weight stays in registers,
// the next row's loads are issued before the current row's reduction, and the
// backward pass keeps its share of dw and db in registers over all its rows.
// Each CTA writes one partial row of dw and db, and a second kernel adds the
// partial rows in a fixed order, so results do not change from call to call.
#include "common.cuh"
#include "internal.h"
#include "op_common.cuh"

namespace muon {
namespace {

// The TPR threads of one row add up two values; every thread gets both sums.
// TPR = 32: one warp, no barrier.  Otherwise the row's threads are the CTA,
// and `slot` alternates between calls so that one barrier is enough.
template <int TPR>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2* smem, int slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if constexpr (TPR == 32) {
    return make_float2(a, b);
  } else {
    constexpr int W = TPR / 32;
    float2* s = smem + slot * 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) s[warp] = make_float2(a, b);
    __syncthreads();
    float2 v = lane < W ? s[lane] : make_float2(0.f, 0.f);
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    return make_float2(__shfl_sync(0xffffffffu, v.x, 0), __shfl_sync(0xffffffffu, v.y, 0));
  }
}

// The elements of a row that one thread holds.  VEC = 1: element e is column
// e TPR + t; otherwise 16-byte vectors, vector v starts at column
// (v TPR + t) VEC.
template <typename T, int VEC, int TPR, int EPT>
struct RowPart {
  static constexpr int NV = EPT / VEC;
  static_assert(VEC * NV == EPT, "whole vectors");
  using Raw = typename std::conditional<VEC == 1, T, uint4>::type;
  Raw raw[NV];

  static __device__ __forceinline__ int col(int e, int t) {
    return VEC == 1 ? e * TPR + t : ((e / VEC) * TPR + t) * VEC + e % VEC;
  }
  __device__ __forceinline__ void load(const T* row, int t, int cols) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TPR + t) * VEC;
      if constexpr (VEC == 1) {
        raw[v] = c < cols ? row[c] : from_f32<T>(0.f);
      } else {
        raw[v] = c < cols ? ld_stream16(row + c) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if constexpr (VEC == 1)
        f[v] = to_f32(raw[v]);
      else
        unpack16<T>(raw[v], f + v * VEC);
    }
  }
  static __device__ __forceinline__ void store(T* row, int t, int cols, const float* f) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TPR + t) * VEC;
      if (c < cols) {
        if constexpr (VEC == 1)
          row[c] = from_f32<T>(f[v]);
        else
          *reinterpret_cast<uint4*>(row + c) = pack16<T>(f + v * VEC);
      }
    }
  }
};

// The weight's (or bias's) values at a thread's columns; `none` where there
// is no such tensor.  p.wvec: its storage is 16-byte aligned, so the VEC
// values of a vector are read by 16-byte loads.
template <int VEC, int TPR, int EPT, typename T>
__device__ __forceinline__ void load_affine(const NormParams& p, const void* base, float none, int t, float* w) {
  using Part = RowPart<T, VEC, TPR, EPT>;
#pragma unroll
  for (int v = 0; v < Part::NV; ++v) {
    const int c = Part::col(v * VEC, t);
    if (base == nullptr || c >= p.cols) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) w[v * VEC + i] = none;
    } else if (VEC > 1 && p.wvec) {
      if (p.wdtype == DT_F32) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4)
          unpack16<float>(*reinterpret_cast<const uint4*>(static_cast<const float*>(base) + c + i), w + v * VEC + i);
      } else if constexpr (VEC == 8) {
        unpack16<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(base) + c), w + v * VEC);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) w[v * VEC + i] = load_f32(base, c + i, p.wdtype);
    }
  }
}

// TPR threads a row; CTAs of TPR threads, or of 128 with four rows at once
// when one warp is enough for a row.
template <int TPR>
struct NormCfg {
  static constexpr int THREADS = TPR == 32 ? 128 : TPR;
  static constexpr int GROUPS = THREADS / TPR;
};

template <typename T, int VEC, int TPR, int EPT>
__global__ void __launch_bounds__(NormCfg<TPR>::THREADS) norm_fwd_kernel(const NormParams p) {
  using Part = RowPart<T, VEC, TPR, EPT>;
  constexpr int G = NormCfg<TPR>::GROUPS;
  __shared__ float2 red[64];
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const int cols = p.cols;
  constexpr bool kReg = EPT <= 8;      // weight and bias stay in registers
  float w[EPT], b[EPT];
  if constexpr (kReg) {
    load_affine<VEC, TPR, EPT, T>(p, p.weight, 1.f, t, w);
    load_affine<VEC, TPR, EPT, T>(p, p.bias, 0.f, t, b);
  }
  const float inv = 1.f / static_cast<float>(cols);
  const long long step = static_cast<long long>(gridDim.x) * G;
  long long row = static_cast<long long>(blockIdx.x) * G + grp;
  Part next;
  if (row < p.rows) next.load(static_cast<const T*>(p.x) + row * p.ldx, t, cols);
  for (; row < p.rows; row += step) {
    float x[EPT];
    next.get(x);
    if (row + step < p.rows) next.load(static_cast<const T*>(p.x) + (row + step) * p.ldx, t, cols);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < EPT; ++e) s += x[e];
    const float mu = row_sum2<TPR>(s, 0.f, red, 0).x * inv;
    float q = 0.f, left = 0.f;
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      x[e] -= mu;
      const float d = Part::col(e, t) < cols ? x[e] : 0.f;
      left += d;
      q = fmaf(d, d, q);
    }
    // the sum's rounding left mu off by off = mean(x - mu): taken out of the
    // differences, the variance and the mean itself
    const float2 two = row_sum2<TPR>(q, left, red, 1);
    const float off = two.y * inv;
    const float r = rsqrtf(fmaxf(fmaf(-off, off, two.x * inv), 0.f) + p.eps);
    if constexpr (!kReg) {
      load_affine<VEC, TPR, EPT, T>(p, p.weight, 1.f, t, w);
      load_affine<VEC, TPR, EPT, T>(p, p.bias, 0.f, t, b);
    }
#pragma unroll
    for (int e = 0; e < EPT; ++e) x[e] = fmaf((x[e] - off) * r, w[e], b[e]);
    Part::store(static_cast<T*>(p.y) + row * p.ldy, t, cols, x);
    if (t == 0) {
      p.mean[row] = mu + off;
      p.rstd[row] = r;
    }
  }
}

// dw and db of a CTA's rows: ACC_REG keeps them in registers, otherwise in
// shared memory (each thread its own columns, no barrier), for rows so wide
// that the registers would spill.
template <typename T, int VEC, int TPR, int EPT, bool ACC_REG>
__global__ void __launch_bounds__(NormCfg<TPR>::THREADS) norm_bwd_kernel(const NormParams p) {
  using Part = RowPart<T, VEC, TPR, EPT>;
  constexpr int G = NormCfg<TPR>::GROUPS;
  extern __shared__ float acc[];       // [2][TPR * EPT], element e of thread t at e TPR + t
  __shared__ float2 red[64];
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const int cols = p.cols;
  float w[EPT], dw[ACC_REG ? EPT : 1], db[ACC_REG ? EPT : 1];
  if constexpr (ACC_REG) load_affine<VEC, TPR, EPT, T>(p, p.weight, 1.f, t, w);
#pragma unroll
  for (int e = 0; e < EPT; ++e) {
    if constexpr (ACC_REG) {
      dw[e] = db[e] = 0.f;
    } else {
      acc[e * TPR + t] = 0.f;
      acc[(EPT + e) * TPR + t] = 0.f;
    }
  }
  const float inv = 1.f / static_cast<float>(cols);
  const long long step = static_cast<long long>(gridDim.x) * G;
  long long row = static_cast<long long>(blockIdx.x) * G + grp;
  Part nx, ny;
  float nmu = 0.f, nr = 0.f;
  auto fetch = [&](long long k) {
    nx.load(static_cast<const T*>(p.x) + k * p.ldx, t, cols);
    ny.load(static_cast<const T*>(p.dy) + k * p.lddy, t, cols);
    nmu = p.mean[k];
    nr = p.rstd[k];
  };
  if (row < p.rows) fetch(row);
  int slot = 0;
  for (; row < p.rows; row += step) {
    float xh[EPT], g[EPT];
    nx.get(xh);
    ny.get(g);
    const float mu = nmu, r = nr;
    if (row + step < p.rows) fetch(row + step);
    if constexpr (!ACC_REG) load_affine<VEC, TPR, EPT, T>(p, p.weight, 1.f, t, w);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      xh[e] = (xh[e] - mu) * r;
      const float d = g[e];            // zero past the last column
      if constexpr (ACC_REG) {
        dw[e] = fmaf(d, xh[e], dw[e]);
        db[e] += d;
      } else {
        acc[e * TPR + t] = fmaf(d, xh[e], acc[e * TPR + t]);
        acc[(EPT + e) * TPR + t] += d;
      }
      g[e] = d * w[e];
      s1 += g[e];
      s2 = fmaf(g[e], xh[e], s2);
    }
    const float2 s = row_sum2<TPR>(s1, s2, red, slot);
    slot ^= 1;
    const float c1 = s.x * inv, c2 = s.y * inv;
#pragma unroll
    for (int e = 0; e < EPT; ++e) g[e] = r * (g[e] - fmaf(xh[e], c2, c1));
    Part::store(static_cast<T*>(p.y) + row * p.ldy, t, cols, g);
  }
  // this CTA's partial row: the groups' sums added in their order
  float* pw = p.part + static_cast<long long>(blockIdx.x) * 2 * cols;
  if constexpr (G > 1) {
    for (int k = 0; k < G; ++k) {
      if (grp == k) {
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
          const int i = e * TPR + t;
          acc[i] = (k == 0 ? 0.f : acc[i]) + dw[e];
          acc[i + EPT * TPR] = (k == 0 ? 0.f : acc[i + EPT * TPR]) + db[e];
        }
      }
      __syncthreads();
    }
    if (grp != 0) return;
  }
#pragma unroll
  for (int e = 0; e < EPT; ++e) {
    const int c = Part::col(e, t);
    if (c < cols) {
      if constexpr (G > 1 || !ACC_REG) {
        pw[c] = acc[e * TPR + t];
        pw[cols + c] = acc[(EPT + e) * TPR + t];
      } else {
        pw[c] = dw[e];
        pw[cols + c] = db[e];
      }
    }
  }
}

// out[c] = sum over k of part[k][c]: 32 columns a CTA, eight threads a column
// over the partial rows, joined in a fixed order.
__global__ void __launch_bounds__(256) norm_join_kernel(const float* part, int parts, int cols2, float* dw, float* db) {
  __shared__ float s[8][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), k0 = threadIdx.x >> 5;
  float v = 0.f;
  if (c < cols2) {
#pragma unroll 8
    for (int k = k0; k < parts; k += 8) v += part[static_cast<long long>(k) * cols2 + c];
  }
  s[k0][threadIdx.x & 31] = v;
  __syncthreads();
  if (k0 == 0 && c < cols2) {
    float a = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) a += s[k][threadIdx.x & 31];
    const int cols = cols2 >> 1;
    if (c < cols)
      dw[c] = a;
    else
      db[c - cols] = a;
  }
}

template <typename T, int VEC, int TPR, int EPT, bool BWD>
cudaError_t launch_cfg(const NormParams& p, int parts, cudaStream_t s) {
  if constexpr (BWD) {
    // registers hold dw and db up to eight elements a thread
    constexpr bool kReg = EPT <= 8;
    constexpr int smem = (NormCfg<TPR>::GROUPS > 1 || !kReg) ? 2 * TPR * EPT * 4 : 0;
    auto kern = norm_bwd_kernel<T, VEC, TPR, EPT, kReg>;
    if (smem > 48 * 1024) {
      static std::atomic<unsigned long long> done;
      const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem, done);
      if (e != cudaSuccess) return e;
    }
    kern<<<parts, NormCfg<TPR>::THREADS, smem, s>>>(p);
  } else {
    norm_fwd_kernel<T, VEC, TPR, EPT><<<parts, NormCfg<TPR>::THREADS, 0, s>>>(p);
  }
  return cudaGetLastError();
}

// Threads a row: the fewest that hold it at eight elements each.
template <typename T, int VEC, bool BWD>
cudaError_t launch_width(const NormParams& p, int parts, cudaStream_t s) {
  switch (norm_threads(p.cols)) {
    case 32: return launch_cfg<T, VEC, 32, 8, BWD>(p, parts, s);
    case 128: return launch_cfg<T, VEC, 128, 8, BWD>(p, parts, s);
    case 256: return launch_cfg<T, VEC, 256, 8, BWD>(p, parts, s);
    case 512: return launch_cfg<T, VEC, 512, 8, BWD>(p, parts, s);
    default:
      return p.cols <= 8192 ? launch_cfg<T, VEC, 1024, 8, BWD>(p, parts, s)
                            : launch_cfg<T, VEC, 1024, 16, BWD>(p, parts, s);
  }
}

template <typename T, bool BWD>
cudaError_t launch_type(const NormParams& p, int parts, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  auto whole = [](const void* q, long long ld) {
    return reinterpret_cast<uintptr_t>(q) % 16 == 0 && (ld * static_cast<long long>(sizeof(T))) % 16 == 0;
  };
  const bool vec = p.cols % V == 0 && whole(p.x, p.ldx) && whole(p.y, p.ldy) && (!BWD || whole(p.dy, p.lddy));
  NormParams q = p;
  q.wvec = whole(p.weight, 0) && whole(p.bias, 0);
  return vec ? launch_width<T, V, BWD>(q, parts, s) : launch_width<T, 1, BWD>(q, parts, s);
}

template <bool BWD>
cudaError_t launch_any(const NormParams& p, int parts, cudaStream_t s) {
  switch (p.dtype) {
    case DT_F32: return launch_type<float, BWD>(p, parts, s);
    case DT_BF16: return launch_type<__nv_bfloat16, BWD>(p, parts, s);
    default: return launch_type<__half, BWD>(p, parts, s);
  }
}

}  // namespace

int norm_threads(int cols) {
  return cols <= 256 ? 32 : cols <= 1024 ? 128 : cols <= 2048 ? 256 : cols <= 4096 ? 512 : 1024;
}

// CTAs of a pass: as many as the rows need, at most what fills the SMs with
// 1024 threads each (the kernels' registers allow about that).
int norm_parts(long long rows, int cols, int sms) {
  const int tpr = norm_threads(cols);
  const int groups = tpr == 32 ? 4 : 1;
  const long long want = (rows + groups - 1) / groups;
  const long long most = static_cast<long long>(sms) * (tpr >= 1024 ? 1 : 1024 / (tpr == 32 ? 128 : tpr));
  return static_cast<int>(want < most ? want : most);
}

cudaError_t launch_norm_fwd(const NormParams& p, int parts, cudaStream_t s) { return launch_any<false>(p, parts, s); }
cudaError_t launch_norm_bwd(const NormParams& p, int parts, cudaStream_t s) { return launch_any<true>(p, parts, s); }

cudaError_t launch_norm_join(const NormParams& p, int parts, float* dw, float* db, cudaStream_t s) {
  norm_join_kernel<<<(2 * p.cols + 31) / 32, 256, 0, s>>>(p.part, parts, 2 * p.cols, dw, db);
  return cudaGetLastError();
}

}  // namespace muon
