// A weight in 8 bits: e4m3 codes with one power of two for each block of 128 x
// 128, the smallest 2^e, e >= -111, with which the block's largest magnitude
// is 448 or less (the activations' rule, op_act8.cu); e + 127 is kept in a
// byte.  As the scale is one for a square, the codes of the transpose are the
// codes transposed: the gradient of a layer's input takes those, with the
// scales read the other way round.  A block with a NaN or an infinity gets the
// byte 255 and codes 0, which stand for NaN.
//
// Bound by HBM.  A CTA takes a block: it is read once into registers (a half
// warp a row, 8 columns a thread), its codes leave as they are and, turned
// around in shared memory, as the transpose's.  A block's loads and its stores
// do not overlap, so the more blocks an SM holds the better, and 512 threads
// with 3 CTAs an SM keep more bytes in flight than 256 with 4 (14336 x 4096
// bf16: codes 34 us against 41, with the transpose's 44 against 50; with 4 CTAs of
// 512, 47 and 58: with 3 the 16-bit kernels spill 16 to 32 bytes a thread, with 4
// more).  That is 176 MB one way at 5.2 TB/s, 235 MB with the
// transpose's at 5.4; the way back, which needs no maximum first, takes 30 us.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"
#include "op_code8.cuh"
#include "op_common.cuh"

namespace muon {
namespace {

constexpr int BLK = 128;
constexpr int WTHREADS = 512;
constexpr int ROWS = WTHREADS / 16;                // rows of a pass, 16 threads each
constexpr int PASSES = BLK / ROWS;
constexpr int LINES = WTHREADS / BLK;              // rows of a pass of single elements

// The transpose's codes from the tile of codes, 16 rows (band) by 4 columns a
// thread, turned around as 4 x 4 bytes.
__device__ __forceinline__ void store_transposed(const Weight8Params& p, const uint32_t (*tile)[BLK / 4], long long o0, int c0) {
  if (threadIdx.x >= 256) return;
  const int band = threadIdx.x & 7, word = threadIdx.x >> 3;
  uint32_t t[4][4];                                  // column, four rows a word
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t a[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) a[k] = tile[band * 16 + i * 4 + k][word ^ (4 * band)];
    const uint32_t x = __byte_perm(a[0], a[1], 0x5140), y = __byte_perm(a[2], a[3], 0x5140);
    const uint32_t z = __byte_perm(a[0], a[1], 0x7362), u = __byte_perm(a[2], a[3], 0x7362);
    t[0][i] = __byte_perm(x, y, 0x5410);
    t[1][i] = __byte_perm(x, y, 0x7632);
    t[2][i] = __byte_perm(z, u, 0x5410);
    t[3][i] = __byte_perm(z, u, 0x7632);
  }
  const long long o = o0 + band * 16;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int cc = c0 + word * 4 + k;
    if (cc >= p.cols || o >= p.out) continue;
    uint8_t* to = p.codes_t + cc * p.ldt + o;
    if (o + 16 <= p.out)
      *reinterpret_cast<uint4*>(to) = make_uint4(t[k][0], t[k][1], t[k][2], t[k][3]);
    else
#pragma unroll
      for (int q = 0; q < 16; ++q)
        if (o + q < p.out) to[q] = static_cast<uint8_t>(t[k][q >> 2] >> (8 * (q & 3)));
  }
}

// Eight codes of row o from column c.
__device__ __forceinline__ void store_eight(const Weight8Params& p, long long o, int c, uint2 code) {
  if (o >= p.out || c >= p.cols) return;
  uint8_t* to = p.codes + o * p.ldc + c;
  if (c + 8 <= p.cols)
    *reinterpret_cast<uint2*>(to) = code;
  else
    for (int k = 0; c + k < p.cols; ++k) to[k] = static_cast<uint8_t>((k < 4 ? code.x : code.y) >> (8 * (k & 3)));
}

// The block's scale byte from each thread's largest magnitude, as bits.
__device__ __forceinline__ int block_scale(int top, int* tops) {
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < WTHREADS / 32; ++i) top = max(top, tops[i]);
  return top < 0x7F800000 ? e4m3_scale_byte(top) : 255;
}

// The tile of codes in shared memory: word w of row r at w ^ 4 ((r >> 4) & 7).
// The transposing reads, 8 bands of 16 rows by 4 neighbouring words, then fall on
// 32 different banks.
template <typename T, bool VEC>
__global__ void __launch_bounds__(WTHREADS, sizeof(T) == 2 ? 3 : 2) weight8_store_kernel(const Weight8Params p, int blocks_c) {
  __shared__ __align__(16) uint32_t tile[BLK][BLK / 4];
  __shared__ int tops[WTHREADS / 32];
  const int kb = blockIdx.x % blocks_c, ob = blockIdx.x / blocks_c;
  const long long o0 = static_cast<long long>(ob) * BLK;
  const T* w = static_cast<const T*>(p.w);
  int top = 0, e;
  if constexpr (VEC) {
    constexpr int kStep = 16 / static_cast<int>(sizeof(T)), NV = 8 / kStep;
    const int l = threadIdx.x & 15, r0 = threadIdx.x >> 4, c = kb * BLK + l * 8;
    uint4 raw[PASSES][NV];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const long long o = o0 + r0 + ROWS * i;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        raw[i][v] = o < p.out && c < p.cols ? ld_stream16(w + o * p.ldw + c + v * kStep) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float f[kStep];
        unpack16<T>(raw[i][v], f);
#pragma unroll
        for (int k = 0; k < kStep; ++k) top = max(top, __float_as_int(f[k]) & 0x7FFFFFFF);
      }
    e = block_scale(top, tops);
    const float unit = __int_as_float((254 - e) << 23);
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = r0 + ROWS * i;
      float f[8];
#pragma unroll
      for (int v = 0; v < NV; ++v) unpack16<T>(raw[i][v], f + v * kStep);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= unit;
      const uint2 code = e != 255 ? make_uint2(e4m3x4(f), e4m3x4(f + 4)) : make_uint2(0u, 0u);
      store_eight(p, o0 + r, c, code);
      if (p.codes_t != nullptr) *reinterpret_cast<uint2*>(&tile[r][(2 * l) ^ (4 * ((r >> 4) & 7))]) = code;
    }
  } else {
    // rows without common alignment: a warp's lanes read elements next to each
    // other, every fourth row a thread, and the codes leave by way of the tile
    // (2612 x 6570 bf16, both ways round and back: 68 us; 154 with eight elements
    // a lane)
    const int lc = threadIdx.x & 127, r0 = threadIdx.x >> 7, c = kb * BLK + lc;
    T raw[BLK / LINES];
#pragma unroll
    for (int i = 0; i < BLK / LINES; ++i) {
      const long long o = o0 + r0 + LINES * i;
      raw[i] = o < p.out && c < p.cols ? w[o * p.ldw + c] : from_f32<T>(0.f);
    }
#pragma unroll
    for (int i = 0; i < BLK / LINES; ++i) top = max(top, __float_as_int(to_f32(raw[i])) & 0x7FFFFFFF);
    e = block_scale(top, tops);
    const float unit = __int_as_float((254 - e) << 23);
    uint8_t* bytes = reinterpret_cast<uint8_t*>(tile);
#pragma unroll
    for (int i = 0; i < BLK / LINES; i += 4) {
      float f[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = to_f32(raw[i + k]) * unit;
      const uint32_t code = e != 255 ? e4m3x4(f) : 0u;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = r0 + LINES * (i + k);
        bytes[r * BLK + (((lc >> 2) ^ (4 * ((r >> 4) & 7))) << 2) + (lc & 3)] = static_cast<uint8_t>(code >> (8 * k));
      }
    }
    __syncthreads();
    const int l = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = (threadIdx.x >> 4) + ROWS * i;
      store_eight(p, o0 + r, kb * BLK + l * 8, *reinterpret_cast<const uint2*>(&tile[r][(2 * l) ^ (4 * ((r >> 4) & 7))]));
    }
  }
  if (threadIdx.x == 0) p.scales[kb * p.lds + ob] = static_cast<uint8_t>(e);
  if (p.codes_t == nullptr) return;
  __syncthreads();
  store_transposed(p, tile, o0, kb * BLK);
}

// A half warp takes 128 columns of a row, 8 a lane; rows a block apart share a scale.
template <typename T, bool VEC>
__global__ void __launch_bounds__(WTHREADS) weight8_restore_kernel(const Weight8Params p, int blocks_c) {
  const int kb = blockIdx.x % blocks_c, ob = blockIdx.x / blocks_c;
  const int l = threadIdx.x & 15, r0 = threadIdx.x >> 4, c = kb * BLK + l * 8;
  const long long o0 = static_cast<long long>(ob) * BLK;
  const float unit = __int_as_float(p.scales[kb * p.lds + ob * p.lds_row] << 23);      // 255: infinity, times 0: NaN
  T* w = static_cast<T*>(const_cast<void*>(p.w));
  __shared__ T rows[VEC ? 1 : ROWS][VEC ? 1 : BLK + 2];
  if (VEC && c >= p.cols) return;
  uint2 code[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const long long o = o0 + r0 + ROWS * i;
    code[i] = make_uint2(0u, 0u);
    if (o < p.out && c < p.cols) {
      const uint8_t* from = p.codes + o * p.ldc + c;
      if (c + 8 <= p.cols) {
        code[i] = *reinterpret_cast<const uint2*>(from);
      } else {
        for (int k = 0; c + k < p.cols; ++k) (k < 4 ? code[i].x : code[i].y) |= static_cast<uint32_t>(from[k]) << (8 * (k & 3));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const long long o = o0 + r0 + ROWS * i;
    if (VEC && o >= p.out) break;
    float f[8];
    e4m3x4_values(code[i].x, unit, f);
    e4m3x4_values(code[i].y, unit, f + 4);
    if constexpr (VEC) {
      constexpr int kStep = 16 / static_cast<int>(sizeof(T));
      T* to = w + o * p.ldw + c;
#pragma unroll
      for (int k = 0; k < 8; k += kStep) *reinterpret_cast<uint4*>(to + k) = pack16<T>(f + k);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) rows[r0][l * 8 + k] = from_f32<T>(f[k]);
      __syncthreads();
      // a warp's lanes write elements next to each other
      const int cc = kb * BLK + (threadIdx.x & 127);
      for (int r = threadIdx.x >> 7; r < ROWS; r += LINES)
        if (cc < p.cols && o0 + ROWS * i + r < p.out) w[(o0 + ROWS * i + r) * p.ldw + cc] = rows[r][threadIdx.x & 127];
      __syncthreads();
    }
  }
}

template <typename T>
cudaError_t launch_type(const Weight8Params& p, bool store, cudaStream_t s) {
  const int blocks_c = static_cast<int>((p.cols + BLK - 1) / BLK);
  const long long ctas = (p.out + BLK - 1) / BLK * blocks_c;
  if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(ctas));
  // 16-byte accesses need rows of whole 8-column groups on 16-byte boundaries
  const bool vec = p.cols % 8 == 0 && reinterpret_cast<uintptr_t>(p.w) % 16 == 0 &&
                   p.ldw * static_cast<long long>(sizeof(T)) % 16 == 0;
  if (store) {
    if (vec)
      weight8_store_kernel<T, true><<<grid, WTHREADS, 0, s>>>(p, blocks_c);
    else
      weight8_store_kernel<T, false><<<grid, WTHREADS, 0, s>>>(p, blocks_c);
  } else {
    if (vec)
      weight8_restore_kernel<T, true><<<grid, WTHREADS, 0, s>>>(p, blocks_c);
    else
      weight8_restore_kernel<T, false><<<grid, WTHREADS, 0, s>>>(p, blocks_c);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_weight8(const Weight8Params& p, bool store, cudaStream_t s) {
  switch (p.dtype) {
    case DT_F32: return launch_type<float>(p, store, s);
    case DT_BF16: return launch_type<__nv_bfloat16>(p, store, s);
    default: return launch_type<__half>(p, store, s);
  }
}

}  // namespace muon
