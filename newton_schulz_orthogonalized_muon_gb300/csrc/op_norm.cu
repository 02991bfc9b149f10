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
// once.  The mean is taken first and the squares about it second, with what
// the mean's rounding left over taken out, so that a large mean does not
// cancel.
//
// Two kinds of kernel.  Rows on 16-byte boundaries of up to 8192 columns
// (batch kernels): a persistent CTA an SM takes batches of G R rows, TPR
// threads a row, R rows a thread at once; a warp of its own copies the
// batches into a ring in shared memory, some 100 KB ahead, and the R rows
// share each reduction and its barrier.  One row at a time, 512 threads a row
// and loads one row ahead, took 160 us for 32768 x 4096 bf16 backward against
// a floor of 119: a row's reduction is a chain of about 1500 cycles.  Other
// rows (row kernels) are loaded into registers one row ahead.
//
// 32768 x 4096 bf16: 98 us forward (5.5 TB/s), 135 us backward (6.0) and 8 us
// for the join, half of it beside the main kernel; 32768 x 4096 fp32 5.9 and
// 6.2 TB/s.  Row kernels: 32768 x 4095 bf16 2.2 and 3.6 TB/s (an element at a
// time), 8192 x 16384 bf16 3.6 and 2.8 (sums in shared memory).
//
// The backward pass keeps its share of dw and db in registers over all its
// rows (in shared memory above 8192 columns).  Each CTA writes one partial
// row of dw and db, and a second kernel adds the partial rows in a fixed
// order, so results do not change from call to call.
#include "common.cuh"
#include "internal.h"
#include "op_common.cuh"

namespace muon {
namespace {

// TPR threads of a row form a group, which meets at a named barrier (one
// warp: none), so that a CTA's rows do not wait on each other.
template <int TPR>
__device__ __forceinline__ void group_sync(int grp) {
  if constexpr (TPR == 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(grp + 1), "n"(TPR) : "memory");
}

// A group adds up N values a thread; every thread gets all N sums.  Within a
// warp the lanes halve the values between them at each step (N = 8: nine
// shuffles, not forty); the warps' sums meet in `smem` (N * TPR / 32 floats
// of this group, another place at every other call, so that one barrier is
// enough).
template <int TPR, int N>
__device__ __forceinline__ void group_sum(float* v, float* smem, int grp) {
  constexpr int W = TPR / 32;
  const int lane = threadIdx.x & 31;
  float u[N];
#pragma unroll
  for (int i = 0; i < N; ++i) u[i] = v[i];
  int n = N;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = (lane & o) != 0;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        if (i < n) {
          const float send = up ? u[i] : u[i + n], keep = up ? u[i + n] : u[i];
          u[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
      }
    } else {
      u[0] += __shfl_xor_sync(0xffffffffu, u[0], o);
    }
  }
  // lanes [i L, (i + 1) L) hold this warp's sum of value i
  constexpr int L = 32 / N;
  if constexpr (W == 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, u[0], i * L);
  } else {
    constexpr int PER = N * W >= 32 ? N * W / 32 : 1;     // sums a lane reads
    constexpr int S = W / PER;                            // lanes of a value
    const int warp = (threadIdx.x % TPR) >> 5;
    if (lane % L == 0) smem[lane / L * W + warp] = u[0];
    group_sync<TPR>(grp);
    float a = 0.f;
    if (lane * PER < N * W) {
#pragma unroll
      for (int i = 0; i < PER; ++i) a += smem[lane * PER + i];
    }
#pragma unroll
    for (int o = S / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, a, i * S);
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
  // from shared memory; zeros where `in` is false
  __device__ __forceinline__ void load_shared(uint32_t row, int t, int cols, bool in) {
    if constexpr (VEC > 1) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * TPR + t) * VEC;
        raw[v] = in && c < cols ? lds16(row + c * static_cast<int>(sizeof(T))) : make_uint4(0u, 0u, 0u, 0u);
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
  // the elements as pairs, for two-wide arithmetic
  __device__ __forceinline__ void get2(F2* f) const {
    float v[EPT];
    get(v);
#pragma unroll
    for (int i = 0; i < EPT / 2; ++i) f[i] = f2_make(v[2 * i], v[2 * i + 1]);
  }
  static __device__ __forceinline__ void store2(T* row, int t, int cols, const F2* f) {
    float v[EPT];
#pragma unroll
    for (int i = 0; i < EPT / 2; ++i) {
      const float2 u = f2_split(f[i]);
      v[2 * i] = u.x;
      v[2 * i + 1] = u.y;
    }
    store(row, t, cols, v);
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

template <int VEC, int TPR, int EPT, typename T>
__device__ __forceinline__ void load_affine2(const NormParams& p, const void* base, float none, int t, F2* w) {
  float v[EPT];
  load_affine<VEC, TPR, EPT, T>(p, base, none, t, v);
#pragma unroll
  for (int i = 0; i < EPT / 2; ++i) w[i] = f2_make(v[2 * i], v[2 * i + 1]);
}

// A CTA's partial row of dw and db from shared memory.
template <typename T, int VEC, int TPR, int EPT>
__device__ __forceinline__ void store_sums(const NormParams& p, const float* acc, int t) {
  using Part = RowPart<T, VEC, TPR, EPT>;
  float* pw = p.part + static_cast<long long>(blockIdx.x) * 2 * p.cols;
#pragma unroll
  for (int e = 0; e < EPT; ++e) {
    const int c = Part::col(e, t);
    if (c < p.cols) {
      pw[c] = acc[e * TPR + t];
      pw[p.cols + c] = acc[(EPT + e) * TPR + t];
    }
  }
}
// The same from the registers of G groups (others: grp >= G), added in their
// order.  Every thread of the CTA calls it.
template <typename T, int VEC, int TPR, int EPT, int G>
__device__ __forceinline__ void store_partial(const NormParams& p, const float* dw, const float* db, float* acc, int t,
                                              int grp) {
  for (int k = 0; k < G; ++k) {
    if (grp == k) {
#pragma unroll
      for (int e = 0; e < EPT; ++e) {
        const int i = e * TPR + t;
        acc[i] = (k == 0 ? 0.f : acc[i]) + dw[e];
        acc[i + EPT * TPR] = (k == 0 ? 0.f : acc[i + EPT * TPR]) + db[e];
      }
    }
    if (G > 1) __syncthreads();
  }
  if (grp == 0) store_sums<T, VEC, TPR, EPT>(p, acc, t);
}

// mean(d^2) about a mean that is `off` too small: not below 0, NaN stays.
__device__ __forceinline__ float variance(float sq, float off) {
  const float v = fmaf(-off, off, sq);
  return v < 0.f ? 0.f : v;
}

// ---------------------------------------------------------- row kernels
// One row at a time and group of TPR threads, for rows that the batch kernels
// do not take.  Backward a CTA of several groups has one partial row of dw and
// db: 4099 x 1023 fp32 with 128 threads a CTA took 16.4 us, with 512 14.5 (a
// group of one warp: 4 and 16 groups the same or worse).
template <int TPR, bool BWD>
struct RowCfg {
  static constexpr int THREADS = TPR == 32 ? 128 : BWD && TPR < 512 ? 512 : TPR;
  static constexpr int GROUPS = THREADS / TPR;
};

template <typename T, int VEC, int TPR, int EPT>
__global__ void __launch_bounds__(RowCfg<TPR, false>::THREADS) norm_row_fwd_kernel(const NormParams p) {
  using Part = RowPart<T, VEC, TPR, EPT>;
  constexpr int G = RowCfg<TPR, false>::GROUPS;
  __shared__ float red[G][2][2 * TPR / 32];
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const int cols = p.cols;
  const float inv = 1.f / static_cast<float>(cols);
  const long long step = static_cast<long long>(gridDim.x) * G;
  long long row = static_cast<long long>(blockIdx.x) * G + grp;
  Part next;
  if (row < p.rows) next.load(static_cast<const T*>(p.x) + row * p.ldx, t, cols);
  for (; row < p.rows; row += step) {
    float x[EPT];
    next.get(x);
    if (row + step < p.rows) next.load(static_cast<const T*>(p.x) + (row + step) * p.ldx, t, cols);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < EPT; ++e) s[0] += x[e];
    group_sum<TPR, 1>(s, red[grp][0], grp);
    const float mu = s[0] * inv;
    s[0] = s[1] = 0.f;
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      x[e] -= mu;
      const float d = Part::col(e, t) < cols ? x[e] : 0.f;
      s[0] = fmaf(d, d, s[0]);
      s[1] += d;
    }
    // the sum's rounding left mu off by off = mean(x - mu): taken out of the
    // differences, the variance and the mean itself
    group_sum<TPR, 2>(s, red[grp][1], grp);
    const float off = s[1] * inv;
    const float r = rsqrtf(variance(s[0] * inv, off) + p.eps);
    float w[EPT];
    load_affine<VEC, TPR, EPT, T>(p, p.weight, 1.f, t, w);
#pragma unroll
    for (int e = 0; e < EPT; ++e) x[e] = (x[e] - off) * r * w[e];
    load_affine<VEC, TPR, EPT, T>(p, p.bias, 0.f, t, w);
#pragma unroll
    for (int e = 0; e < EPT; ++e) x[e] += w[e];
    Part::store(static_cast<T*>(p.y) + row * p.ldy, t, cols, x);
    if (t == 0) {
      p.mean[row] = mu + off;
      p.rstd[row] = r;
    }
  }
}

// ACC_REG keeps dw and db in registers, otherwise in shared memory (each
// thread its own columns, no barrier), for rows so wide that the registers
// would spill.
template <typename T, int VEC, int TPR, int EPT, bool ACC_REG>
__global__ void __launch_bounds__(RowCfg<TPR, true>::THREADS) norm_row_bwd_kernel(const NormParams p) {
  using Part = RowPart<T, VEC, TPR, EPT>;
  constexpr int G = RowCfg<TPR, true>::GROUPS;
  extern __shared__ __align__(128) float acc[];        // [2][TPR * EPT], element e of thread t at e TPR + t
  __shared__ float red[G][2][2 * TPR / 32];
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const int cols = p.cols;
  pdl_launch_dependents();
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
  int turn = 0;
  for (; row < p.rows; row += step, turn ^= 1) {
    float xh[EPT], g[EPT];
    nx.get(xh);
    ny.get(g);
    const float mu = nmu, r = nr;
    if (row + step < p.rows) fetch(row + step);
    if constexpr (!ACC_REG) load_affine<VEC, TPR, EPT, T>(p, p.weight, 1.f, t, w);
    float s[2] = {0.f, 0.f};
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
      s[0] += g[e];
      s[1] = fmaf(g[e], xh[e], s[1]);
    }
    group_sum<TPR, 2>(s, red[grp][turn], grp);
    const float c1 = s[0] * inv, c2 = s[1] * inv;
#pragma unroll
    for (int e = 0; e < EPT; ++e) g[e] = r * (g[e] - fmaf(xh[e], c2, c1));
    Part::store(static_cast<T*>(p.y) + row * p.ldy, t, cols, g);
  }
  if constexpr (ACC_REG)
    store_partial<T, VEC, TPR, EPT, G>(p, dw, db, acc, t, grp);
  else
    store_sums<T, VEC, TPR, EPT>(p, acc, t);
}

// -------------------------------------------------------- batch kernels
constexpr int CALC = 512;                  // threads that calculate; one more warp copies
constexpr int RING_BYTES = 196608;
constexpr int RING_MAX = 8;

template <int TPR, int R, int EPT>
struct BatchCfg {
  static constexpr int G = CALC / TPR;     // rows side by side
  // dw and db in shared memory instead of registers (backward, sixteen
  // elements a thread: 17 warps leave 96 registers)
  static constexpr bool SHARED_SUMS = EPT > 8;
  static constexpr int SUMS = SHARED_SUMS ? 2 * TPR * EPT * 4 : 0;
  static constexpr int B = G * R;          // rows of a batch: row r G + g of group g
  static constexpr int RED = G * 2 * 2 * R * (TPR / 32) * 4;
  static constexpr int OFF_LATE = 2 * RING_MAX * 8;      // a wait ran out
  static constexpr int OFF_RED = OFF_LATE + 16;
  static constexpr int OFF_SUMS = (OFF_RED + RED + 127) / 128 * 128;
  static constexpr int OFF_RING = OFF_SUMS + SUMS;
  static constexpr int RING = RING_BYTES - SUMS;
  static constexpr int SMEM = OFF_RING + RING;
};

// The copying warp: batch after batch into the ring, `arrays` rows' sets a
// slot (x, then dy).  Rows without a gap go in one copy.
template <typename T, int B, bool BWD>
__device__ __forceinline__ void copy_batches(const NormParams& p, uint32_t ring, uint64_t* full, uint64_t* empty,
                                             volatile int* late, int depth, int row_bytes) {
  const int lane = threadIdx.x & 31;
  const long long batches = (p.rows + B - 1) / B;
  int slot = 0;
  uint32_t parity = 1;                     // the first round finds every slot free
  for (long long i = blockIdx.x; i < batches; i += gridDim.x) {
    // the lanes leave together: they meet again below
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(&empty[slot], parity, late, p.timeout_ns))) {
      if (lane == 0) {
        if (*late == 0) atomicOr(p.err, ERRBIT_TIMEOUT);
        *late = 1;
      }
      return;
    }
    const long long row = i * B;
    const int n = static_cast<int>(min(static_cast<long long>(B), p.rows - row));
    const uint32_t dst = ring + slot * (BWD ? 2 : 1) * B * row_bytes;
    if (lane == 0) mbar_arrive_expect_tx(&full[slot], (BWD ? 2 : 1) * n * row_bytes);
    __syncwarp();
#pragma unroll
    for (int a = 0; a < (BWD ? 2 : 1); ++a) {
      const T* src = static_cast<const T*>(a == 0 ? p.x : p.dy);
      const long long ld = a == 0 ? p.ldx : p.lddy;
      if (ld == p.cols) {
        if (lane == a) bulk_load(dst + a * B * row_bytes, src + row * ld, n * row_bytes, smem_u32(&full[slot]));
      } else {
        for (int k = lane; k < n; k += 32)
          bulk_load(dst + (a * B + k) * row_bytes, src + (row + k) * ld, row_bytes, smem_u32(&full[slot]));
      }
    }
    if (++slot == depth) {
      slot = 0;
      parity ^= 1u;
    }
  }
}

template <typename T, int TPR, int EPT, int R, bool BWD>
__global__ void __launch_bounds__(CALC + 32, 1) norm_batch_kernel(const NormParams p) {
  constexpr int VEC = 16 / sizeof(T);
  using Part = RowPart<T, VEC, TPR, EPT>;
  using C = BatchCfg<TPR, R, EPT>;
  constexpr int G = C::G, B = C::B;
  extern __shared__ __align__(128) uint8_t dyn[];
  uint64_t* full = reinterpret_cast<uint64_t*>(dyn);
  uint64_t* empty = full + RING_MAX;
  volatile int* late = reinterpret_cast<int*>(dyn + C::OFF_LATE);
  const uint32_t ring = smem_u32(dyn + C::OFF_RING);
  const int cols = p.cols, row_bytes = cols * static_cast<int>(sizeof(T));
  const int slot_bytes = (BWD ? 2 : 1) * B * row_bytes;
  const int depth = min(C::RING / slot_bytes, RING_MAX);
  if (threadIdx.x == 0) {
    for (int i = 0; i < depth; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], CALC / 32);
    }
    *late = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (BWD) pdl_launch_dependents();
  constexpr int H = EPT / 2;               // elements in pairs: two-wide fp32 arithmetic
  constexpr bool kRegSums = BWD && !C::SHARED_SUMS;
  F2 dw[kRegSums ? H : 1], db[kRegSums ? H : 1];
  // in shared memory, pair e of thread t at (e TPR + t), dw then db: each thread its own, no barrier
  F2* sums = reinterpret_cast<F2*>(dyn + C::OFF_SUMS);
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  if (threadIdx.x >= CALC) {
    copy_batches<T, B, BWD>(p, ring, full, empty, late, depth, row_bytes);
  } else {
    float* red = reinterpret_cast<float*>(dyn + C::OFF_RED) + grp * (2 * 2 * R * (TPR / 32));
    const int lane = threadIdx.x & 31;
    F2 w[H], b[BWD ? 1 : H];
    load_affine2<VEC, TPR, EPT, T>(p, p.weight, 1.f, t, w);
    if constexpr (!BWD) load_affine2<VEC, TPR, EPT, T>(p, p.bias, 0.f, t, b);
    if constexpr (BWD) {
#pragma unroll
      for (int e = 0; e < H; ++e) {
        if constexpr (kRegSums)
          dw[e] = db[e] = f2_make(0.f, 0.f);
        else
          sums[e * TPR + t] = sums[(H + e) * TPR + t] = f2_make(0.f, 0.f);
      }
    }
    const float inv = 1.f / static_cast<float>(cols);
    const long long batches = (p.rows + B - 1) / B;
    float nmu[R], nr[R];                   // the next batch's statistics (backward)
    auto stats = [&](long long i) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const long long row = i * B + r * G + grp;
        nmu[r] = row < p.rows ? p.mean[row] : 0.f;
        nr[r] = row < p.rows ? p.rstd[row] : 0.f;
      }
    };
    if (BWD && blockIdx.x < batches) stats(blockIdx.x);
    int slot = 0, turn = 0;
    uint32_t parity = 0;
    // A wait ran out: no further waits, the error word tells.  No thread leaves: its group meets at barriers.
    bool gave_up = false;
    for (long long i = blockIdx.x; i < batches; i += gridDim.x, turn ^= 1) {
      if (!gave_up && !mbar_wait_bounded(&full[slot], parity, late, p.timeout_ns)) {
        if (*late == 0) atomicOr(p.err, ERRBIT_TIMEOUT);
        *late = 1;
        gave_up = true;
      }
      const uint32_t at = ring + slot * slot_bytes;
      Part x[R], dy[BWD ? R : 1];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bool in = i * B + r * G + grp < p.rows;
        x[r].load_shared(at + (r * G + grp) * row_bytes, t, cols, in);
        if constexpr (BWD) dy[r].load_shared(at + (B + r * G + grp) * row_bytes, t, cols, in);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);
      if (++slot == depth) {
        slot = 0;
        parity ^= 1u;
      }
      if constexpr (BWD) {
        // xh and g of every row stay in registers over the reduction
        F2 xh[R][H], g[R][H];
        float rs[R], s[2 * R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const F2 nm = f2_make(-nmu[r], -nmu[r]), rr = f2_make(nr[r], nr[r]);
          rs[r] = nr[r];
          F2 d[H], s1 = f2_make(0.f, 0.f), s2 = s1;
          x[r].get2(xh[r]);
          dy[r].get2(d);
#pragma unroll
          for (int e = 0; e < H; ++e) {    // d is zero past the last column and the last row
            xh[r][e] = f2_mul(f2_add(xh[r][e], nm), rr);
            if constexpr (kRegSums) {
              dw[e] = f2_fma(d[e], xh[r][e], dw[e]);
              db[e] = f2_add(db[e], d[e]);
            } else {
              F2* at = sums + e * TPR + t;
              at[0] = f2_fma(d[e], xh[r][e], at[0]);
              at[H * TPR] = f2_add(at[H * TPR], d[e]);
            }
            g[r][e] = f2_mul(d[e], w[e]);
            s1 = f2_add(s1, g[r][e]);
            s2 = f2_fma(g[r][e], xh[r][e], s2);
          }
          const float2 a1 = f2_split(s1), a2 = f2_split(s2);
          s[2 * r] = a1.x + a1.y;
          s[2 * r + 1] = a2.x + a2.y;
        }
        if (i + gridDim.x < batches) stats(i + gridDim.x);
        group_sum<TPR, 2 * R>(s, red + turn * (2 * R * (TPR / 32)), grp);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const long long row = i * B + r * G + grp;
          if (row >= p.rows) break;
          const float c1 = -s[2 * r] * inv, c2 = -s[2 * r + 1] * inv;
          const F2 k1 = f2_make(c1, c1), k2 = f2_make(c2, c2), rr = f2_make(rs[r], rs[r]);
#pragma unroll
          for (int e = 0; e < H; ++e) g[r][e] = f2_mul(f2_add(g[r][e], f2_fma(xh[r][e], k2, k1)), rr);
          Part::store2(static_cast<T*>(p.y) + row * p.ldy, t, cols, g[r]);
        }
      } else {
        F2 v[R][H];
        float mu[R], s[2 * R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          x[r].get2(v[r]);
          F2 a = v[r][0];
#pragma unroll
          for (int e = 1; e < H; ++e) a = f2_add(a, v[r][e]);
          const float2 u = f2_split(a);
          mu[r] = u.x + u.y;
        }
        group_sum<TPR, R>(mu, red, grp);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          mu[r] *= inv;
          const F2 nm = f2_make(-mu[r], -mu[r]);
          s[2 * r] = s[2 * r + 1] = 0.f;
#pragma unroll
          for (int k = 0; k < EPT / VEC; ++k) {
            F2 q = f2_make(0.f, 0.f), left = q;
#pragma unroll
            for (int e = k * VEC / 2; e < (k + 1) * VEC / 2; ++e) {
              v[r][e] = f2_add(v[r][e], nm);
              q = f2_fma(v[r][e], v[r][e], q);
              left = f2_add(left, v[r][e]);
            }
            if (Part::col(k * VEC, t) < cols) {      // a vector is inside the row or past it
              const float2 a = f2_split(q), c = f2_split(left);
              s[2 * r] += a.x + a.y;
              s[2 * r + 1] += c.x + c.y;
            }
          }
        }
        group_sum<TPR, 2 * R>(s, red + 2 * R * (TPR / 32), grp);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const long long row = i * B + r * G + grp;
          if (row >= p.rows) break;
          // what the sum's rounding left in mu, as in the row kernel
          const float off = s[2 * r + 1] * inv;
          const float rs = rsqrtf(variance(s[2 * r] * inv, off) + p.eps);
          const F2 no = f2_make(-off, -off), rr = f2_make(rs, rs);
#pragma unroll
          for (int e = 0; e < H; ++e) v[r][e] = f2_fma(f2_mul(f2_add(v[r][e], no), rr), w[e], b[e]);
          Part::store2(static_cast<T*>(p.y) + row * p.ldy, t, cols, v[r]);
          if (t == 0) {
            p.mean[row] = mu[r] + off;
            p.rstd[row] = rs;
          }
        }
      }
    }
  }
  __syncthreads();                         // every batch is read
  // after a wait ran out, copies may still be in flight, and none is issued
  // any more: a millisecond for them to land, in which the CTA's memory is kept
  if (threadIdx.x == CALC && *late != 0) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {
    }
  }
  if constexpr (BWD) {                     // the ring's place takes the sums
    if (kRegSums || grp < G) {             // the copying warp has no sums of its own in shared memory
      float dwf[EPT], dbf[EPT];
#pragma unroll
      for (int e = 0; e < H; ++e) {
        const float2 a = f2_split(kRegSums ? dw[kRegSums ? e : 0] : sums[e * TPR + t]);
        const float2 c = f2_split(kRegSums ? db[kRegSums ? e : 0] : sums[(H + e) * TPR + t]);
        dwf[2 * e] = a.x;
        dwf[2 * e + 1] = a.y;
        dbf[2 * e] = c.x;
        dbf[2 * e + 1] = c.y;
      }
      store_partial<T, VEC, TPR, EPT, G>(p, dwf, dbf, reinterpret_cast<float*>(dyn + C::OFF_RING), t, grp);
    }
  }
}

// out[c] = sum over k of part[k][c]: 32 columns a CTA, 32 threads a column
// over the partial rows, joined in a fixed order.
constexpr int JOIN = 32;

__global__ void __launch_bounds__(32 * JOIN) norm_join_kernel(const float* part, int parts, int cols2, float* dw,
                                                              float* db) {
  __shared__ float s[JOIN][33];
  const int l = threadIdx.x & 31, k0 = threadIdx.x >> 5, c = blockIdx.x * 32 + l;
  pdl_wait();                          // launched while the partial rows are still being formed
  float v = 0.f;
  if (c < cols2) {
#pragma unroll 8
    for (int k = k0; k < parts; k += JOIN) v += part[static_cast<long long>(k) * cols2 + c];
  }
  s[k0][l] = v;
  __syncthreads();
  // warp k0 joins column k0 of this CTA: lane l has its l-th sum
  v = s[l][k0];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int out = blockIdx.x * 32 + k0, cols = cols2 >> 1;
  if (l == 0 && out < cols2) (out < cols ? dw[out] : db[out - cols]) = v;
}

template <typename T, int VEC, int TPR, int EPT, bool BWD>
cudaError_t launch_rows(const NormParams& p, int parts, cudaStream_t s) {
  constexpr int kThreads = RowCfg<TPR, BWD>::THREADS;
  if constexpr (BWD) {
    constexpr bool kReg = EPT <= 8;
    constexpr int kSmem = 2 * TPR * EPT * 4;
    static std::atomic<unsigned long long> done;
    auto kern = norm_row_bwd_kernel<T, VEC, TPR, EPT, kReg>;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), kSmem, done);
    if (e != cudaSuccess) return e;
    kern<<<parts, kThreads, kSmem, s>>>(p);
  } else {
    norm_row_fwd_kernel<T, VEC, TPR, EPT><<<parts, kThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

template <typename T, int TPR, int EPT, int R, bool BWD>
cudaError_t launch_batch(const NormParams& p, int parts, cudaStream_t s) {
  using C = BatchCfg<TPR, R, EPT>;
  static std::atomic<unsigned long long> done;
  auto kern = norm_batch_kernel<T, TPR, EPT, R, BWD>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), C::SMEM, done);
  if (e != cudaSuccess) return e;
  kern<<<parts, CALC + 32, C::SMEM, s>>>(p);
  return cudaGetLastError();
}

bool whole16(const void* q, long long bytes) { return reinterpret_cast<uintptr_t>(q) % 16 == 0 && bytes % 16 == 0; }

// Rows on 16-byte boundaries, at most 8192 columns: the batch kernels.
bool takes_batches(const NormParams& p, bool bwd) {
  const long long es = p.dtype == DT_F32 ? 4 : 2;
  return p.cols <= 8192 && p.cols * es % 16 == 0 && whole16(p.x, p.ldx * es) && whole16(p.y, p.ldy * es) &&
         (!bwd || whole16(p.dy, p.lddy * es));
}

// Rows a thread has at once: four of 16-bit elements forward, two otherwise
// (what registers hold; a batch of 32-bit rows backward is 64 KB).
constexpr int norm_rows_at_once(int size, bool bwd) { return size == 2 && !bwd ? 4 : 2; }

// Threads a row: the fewest that hold it at eight elements each (sixteen
// above 4096 columns).
template <typename T, bool BWD>
cudaError_t launch_type(const NormParams& q, int parts, cudaStream_t s) {
  NormParams p = q;
  p.wvec = whole16(p.weight, 0) && whole16(p.bias, 0);
  if (takes_batches(p, BWD)) {
    constexpr int R = norm_rows_at_once(sizeof(T), BWD);
    if (p.cols <= 256) return launch_batch<T, 32, 8, R, BWD>(p, parts, s);
    if (p.cols <= 1024) return launch_batch<T, 128, 8, R, BWD>(p, parts, s);
    if (p.cols <= 2048) return launch_batch<T, 256, 8, R, BWD>(p, parts, s);
    if (p.cols <= 4096) return launch_batch<T, 512, 8, R, BWD>(p, parts, s);
    return launch_batch<T, 512, 16, 1, BWD>(p, parts, s);
  }
  if (p.cols <= 256) return launch_rows<T, 1, 32, 8, BWD>(p, parts, s);
  if (p.cols <= 1024) return launch_rows<T, 1, 128, 8, BWD>(p, parts, s);
  if (p.cols <= 2048) return launch_rows<T, 1, 256, 8, BWD>(p, parts, s);
  if (p.cols <= 4096) return launch_rows<T, 1, 512, 8, BWD>(p, parts, s);
  if (p.cols <= 8192) return launch_rows<T, 1, 1024, 8, BWD>(p, parts, s);
  constexpr int V = 16 / sizeof(T);
  const long long es = sizeof(T);
  if (p.cols % V == 0 && whole16(p.x, p.ldx * es) && whole16(p.y, p.ldy * es) && (!BWD || whole16(p.dy, p.lddy * es)))
    return launch_rows<T, V, 1024, 16, BWD>(p, parts, s);
  return launch_rows<T, 1, 1024, 16, BWD>(p, parts, s);
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

// CTAs of a pass, the partial rows of dw and db among them at most.  Batch
// kernels: one an SM.  Row kernels: what fills an SM with 1024 threads.
int norm_parts(const NormParams& p, bool bwd, int sms) {
  long long want, most = sms;
  if (takes_batches(p, bwd)) {
    const int rows = p.cols <= 256 ? 16 : p.cols <= 1024 ? 4 : p.cols <= 2048 ? 2 : 1;
    const int b = rows * (p.cols > 4096 ? 1 : norm_rows_at_once(p.dtype == DT_F32 ? 4 : 2, bwd));
    want = (p.rows + b - 1) / b;
  } else {
    const int tpr = p.cols <= 256 ? 32 : p.cols <= 1024 ? 128 : p.cols <= 2048 ? 256 : p.cols <= 4096 ? 512 : 1024;
    const int threads = tpr == 32 ? 128 : bwd && tpr < 512 ? 512 : tpr, b = threads / tpr;
    want = (p.rows + b - 1) / b;
    most = static_cast<long long>(sms) * (1024 / threads);
  }
  return static_cast<int>(want < most ? want : most);
}

// Partial rows that a pass over this many rows can have, whatever its types and alignment.
int norm_max_parts(long long rows, int cols, int sms) {
  const long long most = static_cast<long long>(sms) * (cols <= 256 ? 8 : cols <= 4096 ? 2 : 1);
  return static_cast<int>(rows < most ? rows : most);
}

cudaError_t launch_norm_fwd(const NormParams& p, int parts, cudaStream_t s) { return launch_any<false>(p, parts, s); }
cudaError_t launch_norm_bwd(const NormParams& p, int parts, cudaStream_t s) { return launch_any<true>(p, parts, s); }

cudaError_t launch_norm_join(const NormParams& p, int parts, float* dw, float* db, cudaStream_t s) {
  // overlaps its launch with the pass that forms the partial rows
  const cudaError_t e = launch_k(pdl_level() >= 1, norm_join_kernel, dim3((2 * p.cols + 31) / 32), dim3(32 * JOIN), 0, s,
                                 static_cast<const float*>(p.part), parts, 2 * p.cols, dw, db);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace muon
