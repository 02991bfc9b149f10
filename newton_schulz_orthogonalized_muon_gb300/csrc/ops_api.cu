// C ABI of the training operators (see include/muon.h): checks of the
// arguments, workspace layout and launches.  No exception leaves an entry.
#include <algorithm>
#include <cmath>
#include <string>

#include "common.cuh"
#include "handle.h"
#include "internal.h"
#include "muon.h"

using namespace muon;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 30;     // token and row counts fit an int with room to spare

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
uint64_t round256(uint64_t v) { return (v + 255) / 256 * 256; }
bool op_dtype(int32_t t) { return t == MUON_F32 || t == MUON_BF16 || t == MUON_F16; }

template <typename F>
muon_status_t guarded(muon_handle_t h, F&& f) noexcept {
  HandleLock lock(h);
  try {
    return f();
  } catch (...) {
    return MUON_ERR_WORKSPACE;       // host memory ran out
  }
}

const char* const kBadOperand =
    "operands need 16-byte aligned pointers and positive strides that are multiples of 8 elements";

#define MUON_CHECK(cond, msg) \
  do {                        \
    if (!(cond)) return fail(h, MUON_ERR_INVALID_ARG, msg); \
  } while (0)

muon_status_t check_norm(muon_handle_t h, int64_t rows, int64_t cols, int32_t dtype, int32_t wdtype) {
  MUON_CHECK(rows >= 0 && rows <= kMaxTokens, "rows must be in [0, 2^30]");
  MUON_CHECK(cols >= 1 && cols <= kNormMaxCols, "cols must be in [1, 16384]");
  MUON_CHECK(op_dtype(dtype), "dtype must be MUON_F32, MUON_BF16 or MUON_F16");
  MUON_CHECK(wdtype == MUON_F32 || wdtype == dtype, "wdtype must be MUON_F32 or dtype");
  return MUON_OK;
}

muon_status_t check_act8(muon_handle_t h, const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds,
                         int64_t rows, int64_t cols) {
  MUON_CHECK(rows >= 0 && rows <= kMaxTokens && cols >= 0 && cols <= kMaxTokens, "negative or oversized shape");
  if (rows == 0 || cols == 0) return MUON_OK;
  MUON_CHECK(codes != nullptr && scales != nullptr, "codes or scales is NULL");
  MUON_CHECK(ldc % 128 == 0 && ldc >= cols && aligned(codes, 16),
             "codes need a row stride that is a multiple of 128 and a 16-byte aligned start");
  MUON_CHECK(lds % 16 == 0 && lds >= rows && aligned(scales, 16),
             "scales need a block stride that is a multiple of 16 and a 16-byte aligned start");
  return MUON_OK;
}

// Scratch of the CTAs whose walks are over more rows than one accumulator
// takes (a bound when packed: the sequences' lengths are on the device).
uint64_t attn_part_bytes(muon_handle_t h, const muon_attention_t& a, bool bwd) {
  if (a.sq == 0 || a.sk == 0) return 0;
  const int64_t reach = a.window > 0 ? int64_t(a.window) + 128 : kMaxTokens;       // of the rows that a tile sees
  const int64_t keys = std::min<int64_t>(a.sk, reach), queries = std::min<int64_t>(a.sq, reach) * (a.heads / a.kv_heads);
  if (std::max<int64_t>(keys, bwd ? queries : 0) <= attn_sum_rows(a.dtype == MUON_BF16)) return 0;
  return static_cast<uint64_t>(attn_part_ctas(a.dim, bwd, h->num_sms)) * attn_part_floats(a.dim) * 4;
}

// Two statistics of every query, by tiles of 128, then a counter.
uint64_t attn_stat_bytes(const muon_attention_t& a) {
  const bool packed = a.cu_seqlens_q != nullptr;
  const uint64_t b = packed ? 1 : static_cast<uint64_t>(a.batch);
  return 2 * 512 * b * static_cast<uint64_t>(a.heads) * static_cast<uint64_t>(attn_qtiles(a.sq, a.batch, packed));
}

uint64_t attn_workspace(muon_handle_t h, const muon_attention_t& a) {
  return a.sq > 0 ? attn_stat_bytes(a) + 256 + attn_part_bytes(h, a, true) : 0;
}

muon_status_t check_attention(muon_handle_t h, const muon_attention_t* a) {
  MUON_CHECK(a != nullptr, "a is NULL");
  MUON_CHECK(a->batch >= 0 && a->sq >= 0 && a->sk >= 0 && a->sq <= kMaxTokens && a->sk <= kMaxTokens,
             "negative or oversized shape");
  MUON_CHECK(a->batch <= 65535, "batch must be at most 65535");
  MUON_CHECK(a->heads >= 1 && a->heads <= 65535 && a->kv_heads >= 1 && a->heads % a->kv_heads == 0,
             "heads must be in [1, 65535] and a multiple of kv_heads");
  MUON_CHECK(a->dim >= 8 && a->dim <= 128 && a->dim % 8 == 0, "dim must be a multiple of 8 in [8, 128]");
  MUON_CHECK(a->dtype == MUON_BF16 || a->dtype == MUON_F16, "dtype must be MUON_BF16 or MUON_F16");
  MUON_CHECK(a->window >= 0 && (a->window == 0 || a->causal), "a window needs causal = 1 and a length >= 0");
  MUON_CHECK(std::isfinite(a->scale) && a->scale > 0.f, "scale must be finite and above 0");
  MUON_CHECK((a->cu_seqlens_q == nullptr) == (a->cu_seqlens_k == nullptr),
             "cu_seqlens_q and cu_seqlens_k go together");
  return MUON_OK;
}

// The stride of a dimension of one element is never used.
bool bad_operand(const void* p, const int64_t* st, const int64_t* size) {
  bool bad = p == nullptr || !aligned(p, 16);
  for (int i = 0; i < 3; ++i) bad = bad || (size[i] > 1 && (st[i] % 8 || st[i] < 8 || st[i] > (int64_t(1) << 38)));
  return bad;
}

// Map of an operand [batch][token][head][dim] with boxes of one head, `tokens`
// tokens and 64 columns (a whole 128-byte swizzle row).
bool attn_map(muon_handle_t h, CUtensorMap* map, const void* base, const int64_t* st, const int64_t* size, int dim,
              int dtype, uint32_t tokens) {
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(size[2]),
                        static_cast<cuuint64_t>(size[1]), static_cast<cuuint64_t>(size[0])};
  cuuint64_t strides[3];
  for (int i = 0; i < 3; ++i)
    strides[i] = size[2 - i] > 1 ? static_cast<cuuint64_t>(st[2 - i]) * 2 : static_cast<cuuint64_t>(dim) * 2;
  cuuint32_t box[4] = {64, 1, tokens, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return h->encode(map, dtype == MUON_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                   const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

AttnParams attn_params(muon_handle_t h, const muon_attention_t& a) {
  AttnParams p{};
  p.err = h->err;
  p.timeout_ns = h->timeout_ns;
  p.qtiles = attn_qtiles(a.sq, a.batch, a.cu_seqlens_q != nullptr);
  const bool packed = a.cu_seqlens_q != nullptr;
  auto set = [packed](const int64_t* st, long long* b, long long* s, long long* hh) {
    *b = packed ? 0 : st[0];
    *s = st[1];
    *hh = st[2];
  };
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.lse = a.lse;
  set(a.q_stride, &p.qb, &p.qs, &p.qh);
  set(a.k_stride, &p.kb, &p.ks, &p.kh);
  set(a.v_stride, &p.vb, &p.vs, &p.vh);
  set(a.o_stride, &p.ob, &p.os, &p.oh);
  set(a.dout_stride, &p.dob, &p.dos, &p.doh);
  set(a.dq_stride, &p.dqb, &p.dqs, &p.dqh);
  set(a.dk_stride, &p.dkb, &p.dks, &p.dkh);
  set(a.dv_stride, &p.dvb, &p.dvs, &p.dvh);
  p.lse_h = a.sq;
  p.lse_b = static_cast<long long>(a.heads) * a.sq;
  p.cu_q = a.cu_seqlens_q;
  p.cu_k = a.cu_seqlens_k;
  p.batch = a.batch;
  p.sq = a.sq;
  p.sk = a.sk;
  p.heads = a.heads;
  p.kv_heads = a.kv_heads;
  p.dim = a.dim;
  p.causal = a.causal ? 1 : 0;
  p.window = a.window < kMaxTokens ? a.window : static_cast<int>(kMaxTokens);   // nothing is further away
  p.dtype = a.dtype;
  p.scale = a.scale;
  return p;
}

// Map of [rows][cols], row stride ld elements of `size` bytes (bf16 or
// bytes), in boxes of 64 rows and one 128-byte swizzle row of columns.
bool rows_map(muon_handle_t h, CUtensorMap* map, const void* base, int64_t cols, int64_t rows, int64_t ld, int size,
              uint32_t box_cols) {
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), 1};
  const cuuint64_t pitch = static_cast<cuuint64_t>(ld) * static_cast<cuuint64_t>(size);
  cuuint64_t strides[2] = {pitch, pitch * static_cast<cuuint64_t>(rows)};
  cuuint32_t box[3] = {box_cols, 64, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return h->encode(map, size == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3,
                   const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scratch of a weight gradient: the splits' partial results, then dy with
// padded rows where TMA cannot read it in place.
struct WgradPlan {
  int splits;
  uint64_t part_bytes, pad_bytes;
  uint64_t bytes() const { return part_bytes + pad_bytes; }
};

WgradPlan wgrad_plan(muon_handle_t h, const void* dy, int64_t lddy, int64_t rows, int64_t cols, int64_t out) {
  WgradPlan w{};
  w.splits = wgrad_splits(rows, static_cast<int>(cols), static_cast<int>(out), h->num_sms / 2);
  if (w.splits > 1) w.part_bytes = round256(static_cast<uint64_t>(w.splits) * out * cols * 4);
  if (rows > 0 && ((rows > 1 && lddy % 8 != 0) || !aligned(dy, 16)))
    w.pad_bytes = round256(static_cast<uint64_t>(rows) * ((out + 7) / 8 * 8) * 2);
  return w;
}

}  // namespace

extern "C" {

muon_status_t muon_layer_norm_forward(muon_handle_t h, const void* x, int64_t ldx, const void* weight,
                                      const void* bias, void* y, int64_t ldy, float* mean, float* rstd, int64_t rows,
                                      int64_t cols, int32_t dtype, int32_t wdtype, float eps, void* stream_arg) {
  if (h == nullptr) return MUON_ERR_INVALID_ARG;
  return guarded(h, [&]() -> muon_status_t {
    const muon_status_t st = check_norm(h, rows, cols, dtype, wdtype);
    if (st != MUON_OK) return st;
    MUON_CHECK(std::isfinite(eps) && eps >= 0.f, "eps must be finite and not negative");
    if (rows == 0) return MUON_OK;
    MUON_CHECK(x != nullptr && y != nullptr && mean != nullptr && rstd != nullptr, "NULL tensor pointer");
    MUON_CHECK((ldx >= cols && ldy >= cols) || rows == 1, "row strides must be at least cols");
    DeviceGuard guard(h->device);
    cudaStream_t stream = static_cast<cudaStream_t>(stream_arg);
    NormParams p{};
    p.x = x;
    p.y = y;
    p.weight = weight;
    p.bias = bias;
    p.mean = mean;
    p.rstd = rstd;
    p.rows = rows;
    p.ldx = ldx;
    p.ldy = ldy;
    p.cols = static_cast<int>(cols);
    p.dtype = dtype;
    p.wdtype = wdtype;
    p.eps = eps;
    p.err = h->err;
    p.timeout_ns = h->timeout_ns;
    h->prof_tag = -1;
    MUON_LAUNCH(MUON_K_LAYER_NORM, launch_norm_fwd(p, norm_parts(p, false, h->num_sms), stream),
                "layer norm launch");
    return MUON_OK;
  });
}

muon_status_t muon_layer_norm_workspace(muon_handle_t h, int64_t rows, int64_t cols, uint64_t* bytes) {
  if (h == nullptr || bytes == nullptr) return MUON_ERR_INVALID_ARG;
  return guarded(h, [&]() -> muon_status_t {
    const muon_status_t st = check_norm(h, rows, cols, MUON_F32, MUON_F32);
    if (st != MUON_OK) return st;
    *bytes = round256(static_cast<uint64_t>(norm_max_parts(rows, static_cast<int>(cols), h->num_sms)) * 2 * cols * 4);
    return MUON_OK;
  });
}

muon_status_t muon_layer_norm_backward(muon_handle_t h, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                       const float* mean, const float* rstd, const void* weight, void* dx,
                                       int64_t lddx, float* dweight, float* dbias, int64_t rows, int64_t cols,
                                       int32_t dtype, int32_t wdtype, void* workspace, size_t workspace_bytes,
                                       void* stream_arg) {
  if (h == nullptr) return MUON_ERR_INVALID_ARG;
  return guarded(h, [&]() -> muon_status_t {
    uint64_t need = 0;
    muon_status_t st = check_norm(h, rows, cols, dtype, wdtype);
    if (st == MUON_OK) st = muon_layer_norm_workspace(h, rows, cols, &need);
    if (st != MUON_OK) return st;
    MUON_CHECK(dweight != nullptr && dbias != nullptr, "dweight or dbias is NULL");
    NormParams p{};
    p.cols = static_cast<int>(cols);
    cudaStream_t stream = static_cast<cudaStream_t>(stream_arg);
    if (rows > 0) {
      MUON_CHECK(dy != nullptr && x != nullptr && dx != nullptr && mean != nullptr && rstd != nullptr,
                 "NULL tensor pointer");
      MUON_CHECK((ldx >= cols && lddx >= cols && lddy >= cols) || rows == 1, "row strides must be at least cols");
      MUON_CHECK(workspace != nullptr && workspace_bytes >= need && aligned(workspace, 256),
                 "the workspace is too small or not 256-byte aligned");
    }
    DeviceGuard guard(h->device);
    p.x = x;
    p.dy = dy;
    p.y = dx;
    p.weight = weight;
    p.mean = const_cast<float*>(mean);
    p.rstd = const_cast<float*>(rstd);
    p.part = static_cast<float*>(workspace);
    p.err = h->err;
    p.timeout_ns = h->timeout_ns;
    p.rows = rows;
    p.ldx = ldx;
    p.ldy = lddx;
    p.lddy = lddy;
    p.dtype = dtype;
    p.wdtype = wdtype;
    h->prof_tag = -1;
    const int parts = norm_parts(p, true, h->num_sms);
    if (rows > 0) MUON_LAUNCH(MUON_K_LAYER_NORM, launch_norm_bwd(p, parts, stream), "layer norm backward launch");
    MUON_LAUNCH(MUON_K_LAYER_NORM, launch_norm_join(p, parts, dweight, dbias, stream), "layer norm join launch");
    return MUON_OK;
  });
}

muon_status_t muon_attention_forward(muon_handle_t h, const muon_attention_t* a, void* stream_arg) {
  return muon_attention_forward_ex(h, a, nullptr, 0, stream_arg);
}

muon_status_t muon_attention_forward_workspace(muon_handle_t h, const muon_attention_t* a, uint64_t* bytes) {
  if (h == nullptr || bytes == nullptr) return MUON_ERR_INVALID_ARG;
  return guarded(h, [&]() -> muon_status_t {
    const muon_status_t st = check_attention(h, a);
    if (st != MUON_OK) return st;
    const uint64_t part = attn_part_bytes(h, *a, false);
    *bytes = part > 0 ? part + 256 : 0;            // and a counter
    return MUON_OK;
  });
}

muon_status_t muon_attention_forward_ex(muon_handle_t h, const muon_attention_t* a, void* workspace,
                                        size_t workspace_bytes, void* stream_arg) {
  if (h == nullptr) return MUON_ERR_INVALID_ARG;
  return guarded(h, [&]() -> muon_status_t {
    const muon_status_t st = check_attention(h, a);
    if (st != MUON_OK) return st;
    const uint64_t part = attn_part_bytes(h, *a, false);
    MUON_CHECK(workspace == nullptr || part == 0 || (workspace_bytes >= part + 256 && aligned(workspace, 256)),
               "the workspace is too small or not 256-byte aligned");
    const bool packed = a->cu_seqlens_q != nullptr;
    if (a->sq == 0 || (a->batch == 0 && !packed)) return MUON_OK;
    const int64_t nb = packed ? 1 : a->batch;
    const int64_t qn[3] = {nb, a->sq, a->heads}, kn[3] = {nb, a->sk, a->kv_heads};
    MUON_CHECK(!bad_operand(a->q, a->q_stride, qn) && !bad_operand(a->o, a->o_stride, qn) &&
                   (a->sk == 0 || (!bad_operand(a->k, a->k_stride, kn) && !bad_operand(a->v, a->v_stride, kn))),
               kBadOperand);
    MUON_CHECK(a->lse != nullptr, "lse is NULL");
    DeviceGuard guard(h->device);
    cudaStream_t stream = static_cast<cudaStream_t>(stream_arg);
    AttnParams p = attn_params(h, *a);
    p.out = a->o;
    if (part > 0 && workspace != nullptr) {
      p.part = static_cast<float*>(workspace);
      p.counter = reinterpret_cast<unsigned*>(static_cast<uint8_t*>(workspace) + part);
    }
    CUtensorMap m[3] = {};
    bool ok = attn_map(h, &m[0], a->q, a->q_stride, qn, a->dim, a->dtype, 128);
    if (a->sk > 0)
      ok = ok && attn_map(h, &m[1], a->k, a->k_stride, kn, a->dim, a->dtype, 128) &&
           attn_map(h, &m[2], a->v, a->v_stride, kn, a->dim, a->dtype, 128);
    if (!ok) return fail(h, MUON_ERR_CUDA, "tensor map encoding failed");
    h->prof_tag = -1;
    MUON_LAUNCH(MUON_K_ATTENTION, launch_attn_fwd(p, m, h->num_sms, stream), "attention launch");
    return MUON_OK;
  });
}

muon_status_t muon_attention_workspace(muon_handle_t h, const muon_attention_t* a, uint64_t* bytes) {
  if (h == nullptr || bytes == nullptr) return MUON_ERR_INVALID_ARG;
  return guarded(h, [&]() -> muon_status_t {
    const muon_status_t st = check_attention(h, a);
    if (st != MUON_OK) return st;
    *bytes = attn_workspace(h, *a);
    return MUON_OK;
  });
}

muon_status_t muon_attention_backward(muon_handle_t h, const muon_attention_t* a, void* workspace,
                                      size_t workspace_bytes, void* stream_arg) {
  if (h == nullptr) return MUON_ERR_INVALID_ARG;
  return guarded(h, [&]() -> muon_status_t {
    const muon_status_t st = check_attention(h, a);
    if (st != MUON_OK) return st;
    const bool packed = a->cu_seqlens_q != nullptr;
    if ((a->sq == 0 && a->sk == 0) || (a->batch == 0 && !packed)) return MUON_OK;
    const int64_t nb = packed ? 1 : a->batch;
    const int64_t qn[3] = {nb, a->sq, a->heads}, kn[3] = {nb, a->sk, a->kv_heads};
    MUON_CHECK((a->sq == 0 ||
                !(bad_operand(a->q, a->q_stride, qn) || bad_operand(a->o, a->o_stride, qn) ||
                  bad_operand(a->dout, a->dout_stride, qn) || bad_operand(a->dq, a->dq_stride, qn))) &&
                   (a->sk == 0 ||
                    !(bad_operand(a->k, a->k_stride, kn) || bad_operand(a->v, a->v_stride, kn) ||
                      bad_operand(a->dk, a->dk_stride, kn) || bad_operand(a->dv, a->dv_stride, kn))),
               kBadOperand);
    if (a->sq > 0) {
      MUON_CHECK(a->lse != nullptr, "lse is NULL");
      MUON_CHECK(workspace != nullptr && workspace_bytes >= attn_workspace(h, *a) && aligned(workspace, 256),
                 "the workspace is too small or not 256-byte aligned");
    }
    DeviceGuard guard(h->device);
    cudaStream_t stream = static_cast<cudaStream_t>(stream_arg);
    AttnParams p = attn_params(h, *a);
    p.o = a->o;
    p.dout = a->dout;
    p.dq = a->dq;
    p.dk = a->dk;
    p.dv = a->dv;
    p.stat_lse = static_cast<float*>(workspace);
    p.stat_delta = p.stat_lse + attn_stat_bytes(*a) / 8;
    p.counter = a->sq > 0 ? reinterpret_cast<unsigned*>(static_cast<uint8_t*>(workspace) + attn_stat_bytes(*a)) : nullptr;
    if (attn_part_bytes(h, *a, true) > 0)
      p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + attn_stat_bytes(*a) + 256);
    CUtensorMap m[4] = {};
    const uint32_t tokens = a->dim <= 64 ? 64 : 128;
    bool ok = true;
    if (a->sq > 0)
      ok = attn_map(h, &m[0], a->q, a->q_stride, qn, a->dim, a->dtype, tokens) &&
           attn_map(h, &m[3], a->dout, a->dout_stride, qn, a->dim, a->dtype, tokens);
    if (a->sk > 0)
      ok = ok && attn_map(h, &m[1], a->k, a->k_stride, kn, a->dim, a->dtype, tokens) &&
           attn_map(h, &m[2], a->v, a->v_stride, kn, a->dim, a->dtype, tokens);
    if (!ok) return fail(h, MUON_ERR_CUDA, "tensor map encoding failed");
    h->prof_tag = -1;
    if (a->sq > 0) MUON_LAUNCH(MUON_K_ATTENTION, launch_attn_bwd(p, m, true, h->num_sms, stream), "attention statistics launch");
    MUON_LAUNCH(MUON_K_ATTENTION, launch_attn_bwd(p, m, false, h->num_sms, stream), "attention backward launch");
    return MUON_OK;
  });
}

muon_status_t muon_act8_store(muon_handle_t h, const void* x, int64_t ldx, uint8_t* codes, int64_t ldc,
                              uint8_t* scales, int64_t lds, int64_t rows, int64_t cols, int32_t dtype,
                              void* stream_arg) {
  if (h == nullptr) return MUON_ERR_INVALID_ARG;
  return guarded(h, [&]() -> muon_status_t {
    MUON_CHECK(op_dtype(dtype), "dtype must be MUON_F32, MUON_BF16 or MUON_F16");
    const muon_status_t st = check_act8(h, codes, ldc, scales, lds, rows, cols);
    if (st != MUON_OK) return st;
    if (rows == 0 || cols == 0) return MUON_OK;
    MUON_CHECK(x != nullptr && (ldx >= cols || rows == 1), "x is NULL or its row stride is below cols");
    DeviceGuard guard(h->device);
    cudaStream_t stream = static_cast<cudaStream_t>(stream_arg);
    const Act8Params p{x, nullptr, codes, scales, rows, ldx, ldc, lds, static_cast<int>(cols), dtype};
    h->prof_tag = -1;
    MUON_LAUNCH(MUON_K_ACT8, launch_act8_store(p, stream), "act8 store launch");
    return MUON_OK;
  });
}

muon_status_t muon_act8_restore(muon_handle_t h, const uint8_t* codes, int64_t ldc, const uint8_t* scales,
                                int64_t lds, void* out, int64_t ldo, int64_t rows, int64_t cols, int32_t dtype,
                                void* stream_arg) {
  if (h == nullptr) return MUON_ERR_INVALID_ARG;
  return guarded(h, [&]() -> muon_status_t {
    MUON_CHECK(op_dtype(dtype), "dtype must be MUON_F32, MUON_BF16 or MUON_F16");
    const muon_status_t st = check_act8(h, codes, ldc, scales, lds, rows, cols);
    if (st != MUON_OK) return st;
    if (rows == 0 || cols == 0) return MUON_OK;
    MUON_CHECK(out != nullptr && (ldo >= cols || rows == 1), "out is NULL or its row stride is below cols");
    DeviceGuard guard(h->device);
    cudaStream_t stream = static_cast<cudaStream_t>(stream_arg);
    const Act8Params p{nullptr, out,  const_cast<uint8_t*>(codes), const_cast<uint8_t*>(scales), rows, ldo, ldc,
                       lds,     static_cast<int>(cols), dtype};
    h->prof_tag = -1;
    MUON_LAUNCH(MUON_K_ACT8, launch_act8_restore(p, stream), "act8 restore launch");
    return MUON_OK;
  });
}

muon_status_t muon_act8_weight_grad_workspace(muon_handle_t h, const void* dy, int64_t lddy, int64_t rows,
                                              int64_t cols, int64_t out, uint64_t* bytes) {
  if (h == nullptr || bytes == nullptr) return MUON_ERR_INVALID_ARG;
  return guarded(h, [&]() -> muon_status_t {
    MUON_CHECK(rows >= 0 && rows <= kMaxTokens && cols >= 0 && cols <= kMaxTokens && out >= 0 && out <= kMaxTokens,
               "negative or oversized shape");
    *bytes = cols == 0 || out == 0 ? 0 : wgrad_plan(h, dy, lddy, rows, cols, out).bytes();
    return MUON_OK;
  });
}

muon_status_t muon_act8_weight_grad(muon_handle_t h, const void* dy, int64_t lddy, const uint8_t* codes, int64_t ldc,
                                    const uint8_t* scales, int64_t lds, const void* add, int64_t ldadd, void* dw,
                                    int64_t lddw, int64_t rows, int64_t cols, int64_t out, int32_t odtype,
                                    void* workspace, size_t workspace_bytes, void* stream_arg) {
  if (h == nullptr) return MUON_ERR_INVALID_ARG;
  return guarded(h, [&]() -> muon_status_t {
    const muon_status_t st = check_act8(h, codes, ldc, scales, lds, rows, cols);
    if (st != MUON_OK) return st;
    MUON_CHECK(out >= 0 && out <= kMaxTokens, "negative or oversized shape");
    MUON_CHECK(odtype == MUON_F32 || odtype == MUON_BF16, "odtype must be MUON_F32 or MUON_BF16");
    if (cols == 0 || out == 0) return MUON_OK;
    MUON_CHECK(dw != nullptr && (lddw >= cols || out == 1), "dw is NULL or its row stride is below cols");
    MUON_CHECK(add == nullptr || ldadd >= cols || out == 1, "add's row stride is below cols");
    MUON_CHECK(rows == 0 || (dy != nullptr && (lddy >= out || rows == 1)), "dy is NULL or its row stride is below out");
    const WgradPlan plan = wgrad_plan(h, dy, lddy, rows, cols, out);
    MUON_CHECK(plan.bytes() == 0 ||
                   (workspace != nullptr && workspace_bytes >= plan.bytes() && aligned(workspace, 256)),
               "the workspace is too small or not 256-byte aligned");
    DeviceGuard guard(h->device);
    cudaStream_t stream = static_cast<cudaStream_t>(stream_arg);
    WgradParams p{};
    p.codes = codes;
    p.scales = scales;
    p.add = add;
    p.dw = dw;
    p.part = static_cast<float*>(workspace);
    p.rows = rows;
    p.ldc = ldc;
    p.lds = lds;
    p.ldadd = ldadd;
    p.ldw = lddw;
    p.cols = static_cast<int>(cols);
    p.out = static_cast<int>(out);
    p.odtype = odtype;
    p.splits = plan.splits;
    p.err = h->err;
    p.timeout_ns = h->timeout_ns;
    h->prof_tag = -1;
    CUtensorMap maps[2] = {};
    if (rows > 0) {
      const void* base = dy;
      int64_t ld = lddy;
      if (plan.pad_bytes > 0) {
        __nv_bfloat16* pad = reinterpret_cast<__nv_bfloat16*>(static_cast<uint8_t*>(workspace) + plan.part_bytes);
        ld = (out + 7) / 8 * 8;
        MUON_LAUNCH(MUON_K_WGRAD, launch_pad_rows(static_cast<const __nv_bfloat16*>(dy), lddy, pad, ld, rows, p.out,
                                                  h->num_sms, stream),
                    "row padding launch");
        base = pad;
      }
      if (rows == 1) ld = (out + 7) / 8 * 8;
      if (!rows_map(h, &maps[0], base, out, rows, ld, 2, 64) ||
          !rows_map(h, &maps[1], codes, cols, rows, ldc, 1, 128))
        return fail(h, MUON_ERR_CUDA, "tensor map encoding failed");
    }
    MUON_LAUNCH(MUON_K_WGRAD, launch_act8_wgrad(p, maps, rows > 0 && plan.pad_bytes > 0, h->num_sms / 2, stream), "weight gradient launch");
    if (p.splits > 1)
      MUON_LAUNCH(MUON_K_WGRAD, launch_act8_wgrad_join(p, h->num_sms, stream), "weight gradient join launch");
    return MUON_OK;
  });
}

}  // extern "C"
