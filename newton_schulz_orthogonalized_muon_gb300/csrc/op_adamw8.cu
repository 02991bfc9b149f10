// AdamW over many tensors whose states are kept in 8 bits.
//
// A tensor is cut into blocks of 128 elements.  The average m of the gradients
// is kept as e4m3 codes of m 2^-e, e the smallest integer >= -111 with which
// the block's largest magnitude is 448 or less; e + 127 in a byte.  Of the
// average v of their squares the root r is kept, which has half of v's range
// in powers of two, as codes without a sign: code c > 0 stands for
//   (1 + (c & 15) / 16) 2^((c >> 4) - 8),  up to 248,  times 2^e,
// 0 for 0: 16 binades in steps of 1/16 (v itself: 32 binades).  A root that is
// not 0 gets code 1 at least, since the step divides by it.
//
// Rounding.  An average moves by (1 - beta) of the difference, often less than
// half a step of its codes: rounded to nearest it would never move.  So a
// value is rounded up where its part past a code plus a number in [0, 1) is 1
// or more, which keeps it right on average.  The number of element i is
// (b + u) / 256, b the byte i % 4 of a 32-bit hash of i / 4 and the seed (the
// finalizer that C. Wellons published as lowbias32): the same call gives the
// same result.  Both states of an element use one number: errors of one sign
// in m and r cancel in part in m / r.
//
// u is one for a call.  At 1/2 a move below 1/512 of a step is never taken: a
// step being 1/8 (m) or 1/16 (r) of a value at most, an average then stays
// where it is within 2^-12 / (1 - beta) of its value (v, twice r's part and half
// the move: the same).  That is 2^-7 at 31/32.  Past it a seed's u is its
// multiple of the golden ratio, of which any run of seeds fills [0, 1) evenly,
// in steps of 2^-11: an element's number is then uniform in steps of 2^-19 over
// the calls, as fine as fp32 has r past a code, and no move is too small.
// Kept / true v after 6 / (1 - beta2) steps of the rule at beta2 = 0.9999: 1.003,
// 1.000 and 1.02 (gradients that fall to a half, rise, are normal), where u = 1/2
// gives 3.97, 0.31 and 2.2; with normal gradients 1.005 both ways at 0.95.
//
// The step is as adamw_kernel's, on the states' values in fp32:
//   m <- m + (1 - beta1)(g - m);  v <- r^2 + (1 - beta2)(g^2 - r^2);  r = v^(1/2)
//   p <- p decay - size m / (eps + r)
// and only then are m and r rounded to codes.  g is cut to 2^63 in magnitude, so
// that squares are finite.  The root and the quotient are the hardware's
// approximations, off by up to 2^-22 of themselves.  Of 6.7e7 codes 25 (m) and 75 (r)
// are other than the rule's on 64 bits with bf16 gradients, 116 and 46 with fp32
// ones; in fp32 operation by operation, with a rounded root and quotient, 25 and 78,
// 84 and 65.
//
// Bound by HBM: 10 bytes an element with bf16 parameters and gradients (fp32
// states: 22).  A thread has 16 elements, 8 lanes a block.  1.05e9 bf16
// parameters: 1.62 ms, 6.5 TB/s; their states' values in bf16 0.90 ms, 6.7 TB/s.
// 5.4e8 fp32 parameters with fp32 gradients 1.39 ms, 6.2 TB/s, with bf16 ones 1.20;
// bf16 parameters with fp32 gradients 0.94.  Four CTAs an SM leave a thread 64
// registers, 116 to 160 bytes of which are spilled.  Tensors that no vector access
// fits go an element at a time, 4.4 to 4.9 ms.
#include "common.cuh"
#include "internal.h"
#include "op_code8.cuh"
#include "op_common.cuh"

namespace muon {
namespace {

constexpr int A8_THREADS = 256, A8_EACH = 16, A8_CHUNK = A8_THREADS * A8_EACH;

__device__ __forceinline__ uint32_t hash32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7FEB352Du;
  x ^= x >> 15;
  x *= 0x846CA68Bu;
  return x ^ (x >> 16);
}

// The scale byte of roots whose largest has these fp32 bits.
__device__ __forceinline__ int root_scale_byte(int bits) {
  const int k = (bits >> 23) - 127;
  const int e = (bits & 0x7FFFFF) <= 0x780000 ? k - 7 : k - 6;   // 248 = 1.9375 * 2^7
  return max(e + 127, 16);
}

// The value of a root's code, before its scale.
__device__ __forceinline__ float root_value(uint32_t c) { return c == 0u ? 0.f : __uint_as_float((c << 19) + (119u << 23)); }

// 32 bytes, read or written once.
__device__ __forceinline__ void load32(const void* p, uint4* v) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x), "=r"(v[1].y), "=r"(v[1].z), "=r"(v[1].w)
               : "l"(p));
}
__device__ __forceinline__ void store32(void* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
               "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// 16 elements of type T from `i`; of the tensor's n elements where not VEC.
template <typename T, bool VEC>
__device__ __forceinline__ void load16(const void* base, long long i, long long n, float* f) {
  const T* from = static_cast<const T*>(base) + i;
  if constexpr (VEC) {
    constexpr int kStep = 16 / static_cast<int>(sizeof(T));
#pragma unroll
    for (int k = 0; k < 16; k += 2 * kStep) {
      uint4 v[2];
      load32(from + k, v);
      unpack16<T>(v[0], f + k);
      unpack16<T>(v[1], f + k + kStep);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k) f[k] = i + k < n ? to_f32(from[k]) : 0.f;
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store16(void* base, long long i, long long n, const float* f) {
  T* to = static_cast<T*>(base) + i;
  if constexpr (VEC) {
    constexpr int kStep = 16 / static_cast<int>(sizeof(T));
#pragma unroll
    for (int k = 0; k < 16; k += 2 * kStep) store32(to + k, pack16<T>(f + k), pack16<T>(f + k + kStep));
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (i + k < n) to[k] = from_f32<T>(f[k]);
  }
}
template <bool VEC>
__device__ __forceinline__ void load_codes(const uint8_t* base, long long i, long long n, uint32_t* w) {
  if constexpr (VEC) {
    const uint4 v = ld_stream16(base + i);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const uint32_t b = i + k < n ? base[i + k] : 0u;
      w[k >> 2] = (k & 3) == 0 ? b : w[k >> 2] | (b << (8 * (k & 3)));
    }
  }
}
template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* base, long long i, long long n, const uint32_t* w) {
  if constexpr (VEC) {
    *reinterpret_cast<uint4*>(base + i) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (i + k < n) base[i + k] = static_cast<uint8_t>(w[k >> 2] >> (8 * (k & 3)));
  }
}

// Largest (NaN if one is) and smallest magnitude of three.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// The largest of a block's magnitudes, as bits (they compare as integers, NaN
// above infinity).
__device__ __forceinline__ int block_max(float x) {
  int v = __float_as_int(x) & 0x7FFFFFFF;
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__device__ __forceinline__ float sqrt_ftz(float v) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_ftz(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// The values of four roots' codes before their scale, none of them 0.
__device__ __forceinline__ void roots4(uint32_t w, float* f) {
#pragma unroll
  for (int q = 0; q < 4; ++q) f[q] = __uint_as_float(__byte_perm(w, 0u, 0x4044u | (q << 8)) * 8u + (119u << 23));
}
// some byte of a word is 0
__device__ __forceinline__ bool zero_byte(uint32_t w) { return ((w - 0x01010101u) & ~w & 0x80808080u) != 0u; }

// Bits 16 + S .. 23 + S of four words as four bytes.
template <int S>
__device__ __forceinline__ uint32_t gather4(const uint32_t* t) {
  const uint32_t a = __byte_perm(t[0], t[1], 0x7632) >> S, b = __byte_perm(t[2], t[3], 0x7632) >> S;
  return __byte_perm(a, b, 0x6420);
}

// The step of 16 elements, and their states' new codes.  Measured by what it
// executes: at the copy rate the SMs have 57 instructions for an element, 28 on
// the ALU pipe; the plain way took 70 (45 of those), this one 48.  Arithmetic goes
// two elements at a time; codes are cut out of the fp32 pattern, scaled so that
// they lie in it as they are kept; and what only small values need (codes below
// the normal range, least codes, zeros) is done where a thread has one.
template <typename TP, typename TG, bool VEC>
__device__ __forceinline__ void step16(const Adamw8Params& p, const Adamw8Tensor& t, long long i) {
  const long long n = t.numel, blk = i >> 7;
  // lanes past the end stay for the block's maxima
  const bool in = VEC || i < n;
  const long long at = in ? i : 0, end = in ? n : 0;
  float g[16], w[16], m[16], r[16];
  uint32_t mc[4], rc[4];
  load16<TG, VEC>(t.g, at, end, g);
  load16<TP, VEC>(t.p, at, end, w);
  load_codes<VEC>(t.m, at, end, mc);
  load_codes<VEC>(t.r, at, end, rc);
  const float mu = __int_as_float(in ? t.ms[blk] << 23 : 0), ru = __int_as_float(in ? t.rs[blk] << 23 : 0);
  const F2 mu2 = f2_make(mu, mu), ru2 = f2_make(ru, ru), b1 = f2_make(p.omb1, p.omb1), b2 = f2_make(p.omb2, p.omb2),
           eps = f2_make(p.eps, p.eps), decay = f2_make(p.decay, p.decay), size = f2_make(-p.size, -p.size),
           minus = f2_make(-1.f, -1.f);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    e4m3x4_values(mc[k], 1.f, m + 4 * k);
    roots4(rc[k], r + 4 * k);
    if (zero_byte(rc[k])) {
#pragma unroll
      for (int q = 0; q < 4; ++q) r[4 * k + q] = root_value((rc[k] >> (8 * q)) & 255u);
    }
  }
  // a finite gradient is 2^63 at most: an infinite square would make its block's
  // states NaN, and the parameters of all 128 elements with the next step
  float gtop = 0.f;
#pragma unroll
  for (int k = 0; k < 16; k += 2) gtop = max3(gtop, g[k], g[k + 1]);
  if (!(gtop < 0x1p63f)) {
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (fabsf(g[k]) < INFINITY) g[k] = fminf(fmaxf(g[k], -0x1p63f), 0x1p63f);
  }
  float mtop = 0.f, rtop = 0.f, mlow = INFINITY, rlow = INFINITY;
#pragma unroll
  for (int k = 0; k < 16; k += 2) {
    const F2 gg = f2_make(g[k], g[k + 1]), m0 = f2_mul(f2_make(m[k], m[k + 1]), mu2), r0 = f2_mul(f2_make(r[k], r[k + 1]), ru2);
    const F2 mm = f2_fma(b1, f2_fma(m0, minus, gg), m0);
    const F2 sq = f2_mul(r0, r0);
    const float2 v = f2_split(f2_fma(b2, f2_fma(gg, gg, f2_mul(sq, minus)), sq));
    r[k] = sqrt_ftz(v.x);
    r[k + 1] = sqrt_ftz(v.y);
    const float2 d = f2_split(f2_add(f2_make(r[k], r[k + 1]), eps));
    const F2 u = f2_mul(f2_mul(mm, size), f2_make(rcp_ftz(d.x), rcp_ftz(d.y)));
    const float2 x = f2_split(f2_fma(f2_make(w[k], w[k + 1]), decay, u)), y = f2_split(mm);
    w[k] = x.x;
    w[k + 1] = x.y;
    m[k] = y.x;
    m[k + 1] = y.y;
    mtop = max3(mtop, y.x, y.y);
    rtop = max3(rtop, r[k], r[k + 1]);
    mlow = min3(mlow, y.x, y.y);
    rlow = min3(rlow, r[k], r[k + 1]);
  }
  store16<TP, VEC>(t.p, at, end, w);
  const int mb = block_max(mtop), rb = block_max(rtop);
  const bool mfine = mb < 0x7F800000, rfine = rb < 0x7F800000;
  const int me = mfine ? e4m3_scale_byte(mb) : 255, re = rfine ? root_scale_byte(rb) : 255;
  const float mi = __int_as_float((254 - me) << 23), ri = __int_as_float((254 - re) << 23);
  // Exponents such that a code lies in bits 20 .. 26 (m) and 19 .. 26 (r): e4m3's
  // 2^e has e + 7 there, a root's 2^e has e + 8.
  const F2 mi2 = f2_make(mi * 256.f, mi * 256.f), ri2 = f2_make(ri * 512.f, ri * 512.f);
  const bool plain = mlow * mi >= 0.015625f && rlow * ri >= 0.0078125f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t h = hash32(static_cast<uint32_t>(i >> 2) + k + p.salt);
    if (plain) {
      uint32_t tm[4], tr[4];
#pragma unroll
      for (int q = 0; q < 4; q += 2) {
        const float2 y = f2_split(f2_mul(f2_make(m[4 * k + q], m[4 * k + q + 1]), mi2));
        const float2 z = f2_split(f2_mul(f2_make(r[4 * k + q], r[4 * k + q + 1]), ri2));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // the element's byte at bit 11, and the call's part of its unit
          const uint32_t noise = __byte_perm(h, 0u, 0x4404u | ((q + e) << 4)) * 8u + p.part;
          tm[q + e] = noise * 2u + __float_as_uint(e == 0 ? y.x : y.y);
          tr[q + e] = noise + __float_as_uint(e == 0 ? z.x : z.y);
        }
      }
      const uint32_t sign = __byte_perm(__byte_perm(tm[0], tm[1], 0x0073), __byte_perm(tm[2], tm[3], 0x0073), 0x5410);
      mc[k] = gather4<4>(tm) | (sign & 0x80808080u);
      rc[k] = gather4<3>(tr);
    } else {
      uint32_t mw = 0u, rw = 0u;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int j = 4 * k + q;
        const uint32_t byte = (h >> (8 * q)) & 255u;
        float y = fabsf(m[j]) * mi;
        const bool low = y < 0.015625f;            // 2^-6: steps of 2^-9 below
        y = low ? y + 0.015625f : y;
        const uint32_t c = (__float_as_uint(y) + (byte << 12) + 2u * p.part) >> 20;
        mw |= (min(c - (low ? 968u : 960u), 0x7Eu) | (__float_as_uint(m[j]) >> 31 << 7)) << (8 * q);
        const float z = r[j] * ri;
        const int d = static_cast<int>((__float_as_uint(z) + (byte << 11) + p.part) >> 19) - 1904;
        rw |= (z > 0.f ? static_cast<uint32_t>(min(max(d, 1), 255)) : 0u) << (8 * q);
      }
      mc[k] = mfine ? mw : 0u;
      rc[k] = rfine ? rw : 0u;
    }
  }
  store_codes<VEC>(t.m, at, end, mc);
  store_codes<VEC>(t.r, at, end, rc);
  if ((threadIdx.x & 7) == 0 && in) {
    t.ms[blk] = static_cast<uint8_t>(me);
    t.rs[blk] = static_cast<uint8_t>(re);
  }
}

// The tensor that the CTA's chunk belongs to.
__device__ __forceinline__ int tensor_of(const Adamw8Params& p, uint32_t chunk) {
  int lo = 0, hi = p.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.t[mid].chunk0 <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

template <typename TP, typename TG>
__global__ void __launch_bounds__(A8_THREADS, 4) adamw8_kernel(const __grid_constant__ Adamw8Params p) {
  const Adamw8Tensor& t = p.t[tensor_of(p, blockIdx.x)];
  const long long i0 = static_cast<long long>(blockIdx.x - t.chunk0) * A8_CHUNK, i = i0 + threadIdx.x * A8_EACH;
  if (t.vec && i0 + A8_CHUNK <= t.numel)
    step16<TP, TG, true>(p, t, i);
  else
    step16<TP, TG, false>(p, t, i);
}

template <typename T>
__global__ void __launch_bounds__(A8_THREADS) adamw8_restore_kernel(const __grid_constant__ Adamw8Params p) {
  const Adamw8Tensor& t = p.t[tensor_of(p, blockIdx.x)];
  const long long n = t.numel, i = static_cast<long long>(blockIdx.x - t.chunk0) * A8_CHUNK + threadIdx.x * A8_EACH;
  if (i >= n) return;
  const float mu = __int_as_float(t.ms[i >> 7] << 23), ru = __int_as_float(t.rs[i >> 7] << 23);
  const bool vec = t.vec && i + A8_EACH <= n;
  uint32_t mc[4], rc[4];
  float f[16];
  if (vec) {
    load_codes<true>(t.m, i, n, mc);
    load_codes<true>(t.r, i, n, rc);
  } else {
    load_codes<false>(t.m, i, n, mc);
    load_codes<false>(t.r, i, n, rc);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) e4m3x4_values(mc[k], mu, f + 4 * k);
  if (vec)
    store16<T, true>(t.p, i, n, f);
  else
    store16<T, false>(t.p, i, n, f);
#pragma unroll
  for (int k = 0; k < 16; ++k) f[k] = root_value((rc[k >> 2] >> (8 * (k & 3))) & 255u) * ru;
  if (vec)
    store16<T, true>(const_cast<void*>(t.g), i, n, f);
  else
    store16<T, false>(const_cast<void*>(t.g), i, n, f);
}

}  // namespace

// Numbers the chunks of q.t[0 .. n - 1]; the number of all.
static long long number_chunks(Adamw8Params& q) {
  long long chunks = 0;
  for (int i = 0; i < q.n; ++i) {
    q.t[i].chunk0 = static_cast<uint32_t>(chunks);
    chunks += (q.t[i].numel + A8_CHUNK - 1) / A8_CHUNK;
  }
  return chunks;
}

cudaError_t launch_adamw8(Adamw8Params& q, cudaStream_t s) {
  const long long chunks = number_chunks(q);
  if (chunks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(chunks));
  const bool pb = q.pdtype == DT_BF16, gb = q.gdtype == DT_BF16;
  if (pb && gb)
    adamw8_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, A8_THREADS, 0, s>>>(q);
  else if (pb)
    adamw8_kernel<__nv_bfloat16, float><<<grid, A8_THREADS, 0, s>>>(q);
  else if (gb)
    adamw8_kernel<float, __nv_bfloat16><<<grid, A8_THREADS, 0, s>>>(q);
  else
    adamw8_kernel<float, float><<<grid, A8_THREADS, 0, s>>>(q);
  return cudaGetLastError();
}

cudaError_t launch_adamw8_restore(Adamw8Params& q, cudaStream_t s) {
  const long long chunks = number_chunks(q);
  if (chunks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(chunks));
  if (q.pdtype == DT_BF16)
    adamw8_restore_kernel<__nv_bfloat16><<<grid, A8_THREADS, 0, s>>>(q);
  else
    adamw8_restore_kernel<float><<<grid, A8_THREADS, 0, s>>>(q);
  return cudaGetLastError();
}

}  // namespace muon
