// Activations kept in 8 bits between the forward and the backward pass.
//
// Each token's row is cut into blocks of 128 columns.  A block with largest
// magnitude a is stored as e4m3 codes of x 2^-e, rounded to nearest even,
// with the smallest e (at least -111) for which a 2^-e <= 448, the largest
// e4m3 value.  The scale 2^e is a power of two: scaling is exact, the codes
// are the only rounding, and code times scale is exact in bf16 (4
// significant bits; e >= -111 keeps the smallest code's value 2^(e-9) a
// normal bf16 number).  e + 127 is kept in one byte.  A block with a NaN or
// an infinity gets the byte 255 and codes 0, which restore to NaN: a wrong
// activation stays visible in every gradient that it reaches.
//
// Both directions are bound by HBM.  A group of 16 lanes handles a block, 8
// columns a lane, so a 16-bit input is one 16-byte load a lane; a warp
// handles its 16 rows of one block column two at a time, and 16 lanes write
// the rows' scale bytes at once (scales lie block column by block column,
// one byte a row, as the weight-gradient kernel reads them).  Measured at
// 16384 x 14336 bf16: stored in 119 us (5.9 TB/s), restored in 106 us (6.6).
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"
#include "op_common.cuh"

namespace muon {
namespace {

constexpr int ABLK = 128;       // columns of a block
constexpr int AROWS = 16;       // rows of a warp's work item
constexpr int AWARPS = 8;

// The scale byte of a block with largest magnitude a (finite, >= 0).
__device__ __forceinline__ int scale_byte(float a) {
  // a = m 2^k, 1 <= m < 2 (a below the normal range: k <= -127, clamped)
  const int bits = __float_as_int(a);
  const int k = (bits >> 23) - 127;
  const int e = (bits & 0x7FFFFF) <= 0x600000 ? k - 8 : k - 7;   // 448 = 1.75 * 2^8
  return max(e + 127, 16);
}

// Eight consecutive values of a row from column c, as loaded: zeros past the
// last column and past the last row.
template <typename T, bool VEC>
struct Eight {
  static constexpr int NV = VEC ? 8 * static_cast<int>(sizeof(T)) / 16 : 1;
  using Raw = typename std::conditional<VEC, uint4, T>::type;
  Raw raw[VEC ? NV : 8];

  __device__ __forceinline__ void load(const T* row, int c, int cols, bool in) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        raw[i] = in && c < cols ? ld_stream16(row + c + i * (16 / sizeof(T))) : make_uint4(0u, 0u, 0u, 0u);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) raw[i] = in && c + i < cols ? row[c + i] : from_f32<T>(0.f);
    }
  }
  __device__ __forceinline__ void get(float* f) const {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < NV; ++i) unpack16<T>(raw[i], f + i * (16 / sizeof(T)));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = to_f32(raw[i]);
    }
  }
  // Bits of the block's largest magnitude in fp32, over the 16 lanes that hold
  // it.  Magnitudes compare as their bit patterns, NaN above infinity; 16-bit
  // ones two at a time.
  __device__ __forceinline__ int block_top() const {
    if constexpr (VEC && sizeof(T) == 2) {
      constexpr uint32_t kMag = 0x7FFF7FFFu;
      uint32_t m = __vmaxu2(__vmaxu2(raw[0].x & kMag, raw[0].y & kMag), __vmaxu2(raw[0].z & kMag, raw[0].w & kMag));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
      const uint16_t top = static_cast<uint16_t>(max(m >> 16, m & 0xFFFFu));
      return __float_as_int(to_f32(*reinterpret_cast<const T*>(&top))) & 0x7FFFFFFF;
    } else {
      float f[8];
      get(f);
      int top = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) top = max(top, __float_as_int(f[k]) & 0x7FFFFFFF);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      return top;
    }
  }
};

__device__ __forceinline__ uint32_t e4m3x4(const float* f) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[0], f[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[2], f[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// The four values of a word of codes, each times `unit`.
__device__ __forceinline__ void e4m3x4_values(uint32_t w, float unit, float* f) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * k)), __NV_E4M3));
    const float2 v = __half22float2(h);
    f[2 * k] = v.x * unit;
    f[2 * k + 1] = v.y * unit;
  }
}

// A warp takes AROWS rows of one block column, two rows at a time, with the
// loads of AHEAD row pairs in flight: 2 pairs took 132 us, 4 119 us, 8 (with
// fewer warps on an SM) 126 us at 16384 x 14336.  The instructions count as
// well: with the maximum taken one value at a time 4 pairs took 130 us.
template <typename T, bool VEC>
__global__ void __launch_bounds__(AWARPS * 32, VEC && sizeof(T) == 2 ? 6 : 4) act8_store_kernel(const Act8Params p, int blocks) {
  constexpr int AHEAD = 4;
  const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
  const long long groups = (p.rows + AROWS - 1) / AROWS;
  const long long item = static_cast<long long>(blockIdx.x) * AWARPS + (threadIdx.x >> 5);
  if (item >= groups * blocks) return;
  const int blk = static_cast<int>(item % blocks);
  const long long r0 = item / blocks * AROWS;
  const int c = blk * ABLK + l * 8;
  const long long rows = c < p.cols ? p.rows : 0;      // that this lane has codes of
  int mine = 0;                       // an even lane's: scale byte of row r0 + l + half
#pragma unroll
  for (int i0 = 0; i0 < AROWS; i0 += 2 * AHEAD) {
    Eight<T, VEC> in[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const long long r = r0 + i0 + 2 * j + half;
      in[j].load(static_cast<const T*>(p.x) + r * p.ldx, c, p.cols, r < p.rows);
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int i = i0 + 2 * j;
      const long long r = r0 + i + half;
      const int top = in[j].block_top();
      const bool fine = top < 0x7F800000;
      const int e = fine ? scale_byte(__int_as_float(top)) : 255;
      const float unit = __int_as_float((254 - e) << 23);       // 2^-(e - 127)
      float f[8];
      in[j].get(f);
      const F2 uu = f2_make(unit, unit);
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float2 v = f2_split(f2_mul(f2_make(f[k], f[k + 1]), uu));
        f[k] = v.x;
        f[k + 1] = v.y;
      }
      const uint32_t lo = e4m3x4(f), hi = e4m3x4(f + 4);
      const uint2 code = fine ? make_uint2(lo, hi) : make_uint2(0u, 0u);
      if (r < rows) {
        uint8_t* to = p.codes + r * p.ldc + c;
        if (VEC || c + 8 <= p.cols) {
          *reinterpret_cast<uint2*>(to) = code;
        } else {
          for (int k = 0; c + k < p.cols; ++k) to[k] = static_cast<uint8_t>((k < 4 ? code.x : code.y) >> (8 * (k & 3)));
        }
      }
      if (l == i) mine = e;
    }
  }
  const long long r = r0 + l + half;
  if (l % 2 == 0 && r < p.rows) p.scales[blk * p.lds + r] = static_cast<uint8_t>(mine);
}

// Rows that 16-byte stores do not fit go by way of shared memory, so that a
// warp's lanes write elements next to each other: 16384 x 14330 bf16 took 644
// us with eight elements a lane.
template <typename T, bool VEC>
__global__ void __launch_bounds__(AWARPS * 32) act8_restore_kernel(const Act8Params p, int blocks) {
  __shared__ __align__(16) T rows[VEC ? 1 : AWARPS][2][VEC ? 8 : ABLK];
  const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
  const long long groups = (p.rows + AROWS - 1) / AROWS;
  const long long item = static_cast<long long>(blockIdx.x) * AWARPS + (threadIdx.x >> 5);
  if (item >= groups * blocks) return;
  const int blk = static_cast<int>(item % blocks);
  const long long r0 = item / blocks * AROWS;
  const int c = blk * ABLK + l * 8;
  const bool live = c < p.cols;
  uint2 w[AROWS / 2];
  int e[AROWS / 2];
#pragma unroll
  for (int j = 0; j < AROWS / 2; ++j) {
    const long long r = r0 + 2 * j + half;
    const bool in = live && r < p.rows;
    w[j] = in ? *reinterpret_cast<const uint2*>(p.codes + r * p.ldc + c) : make_uint2(0u, 0u);
    e[j] = in ? p.scales[blk * p.lds + r] : 0;
  }
  T* out = static_cast<T*>(p.out);
#pragma unroll
  for (int j = 0; j < AROWS / 2; ++j) {
    const long long r = r0 + 2 * j;
    if (r >= p.rows) break;
    float f[8];
    const float unit = __int_as_float(e[j] << 23);              // 255: infinity, times code 0: NaN
    e4m3x4_values(w[j].x, unit, f);
    e4m3x4_values(w[j].y, unit, f + 4);
    constexpr int kStep = 16 / static_cast<int>(sizeof(T));
    if constexpr (VEC) {
      if (live && r + half < p.rows) {
#pragma unroll
        for (int i = 0; i < 8; i += kStep) *reinterpret_cast<uint4*>(out + (r + half) * p.ldx + c + i) = pack16<T>(f + i);
      }
    } else {
      T(*to)[ABLK] = rows[threadIdx.x >> 5];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; i += kStep) *reinterpret_cast<uint4*>(&to[half][l * 8 + i]) = pack16<T>(f + i);
      __syncwarp();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (r + h >= p.rows) break;
        T* row = out + (r + h) * p.ldx + blk * ABLK;
#pragma unroll
        for (int i = lane; i < ABLK; i += 32)
          if (blk * ABLK + i < p.cols) row[i] = to[h][i];
      }
    }
  }
}

// 16-byte loads (stores) need rows of whole 8-column groups on 16-byte
// boundaries; anything else goes element by element.
template <typename T>
cudaError_t launch_type(const Act8Params& p, bool store, cudaStream_t s) {
  const int blocks = (p.cols + ABLK - 1) / ABLK;
  const long long items = (p.rows + AROWS - 1) / AROWS * blocks;
  const long long ctas = (items + AWARPS - 1) / AWARPS;
  if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(ctas));
  const void* base = store ? p.x : p.out;
  const bool vec = p.cols % 8 == 0 && reinterpret_cast<uintptr_t>(base) % 16 == 0 &&
                   p.ldx * static_cast<long long>(sizeof(T)) % 16 == 0;
  if (store) {
    if (vec)
      act8_store_kernel<T, true><<<grid, AWARPS * 32, 0, s>>>(p, blocks);
    else
      act8_store_kernel<T, false><<<grid, AWARPS * 32, 0, s>>>(p, blocks);
  } else {
    if (vec)
      act8_restore_kernel<T, true><<<grid, AWARPS * 32, 0, s>>>(p, blocks);
    else
      act8_restore_kernel<T, false><<<grid, AWARPS * 32, 0, s>>>(p, blocks);
  }
  return cudaGetLastError();
}

cudaError_t launch_any(const Act8Params& p, bool store, cudaStream_t s) {
  switch (p.dtype) {
    case DT_F32: return launch_type<float>(p, store, s);
    case DT_BF16: return launch_type<__nv_bfloat16>(p, store, s);
    default: return launch_type<__half>(p, store, s);
  }
}

}  // namespace

cudaError_t launch_act8_store(const Act8Params& p, cudaStream_t s) { return launch_any(p, true, s); }
cudaError_t launch_act8_restore(const Act8Params& p, cudaStream_t s) { return launch_any(p, false, s); }

}  // namespace muon
