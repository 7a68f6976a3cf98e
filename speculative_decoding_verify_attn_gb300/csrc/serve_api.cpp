// C ABI of the serving operators (include/spec_serve.h): argument validation, workspace sizing and
// kernel launches.  As in api.cpp nothing here allocates memory or keeps state between calls.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "serve_internal.h"
#include "spec_serve.h"
#include "tensor_map.h"

namespace {

using specv::LogprobParams;
using specv::ServeAttnParams;

constexpr int64_t kMaxTokens = 1 << 22;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int elem_bytes(int dtype) { return dtype == SPEC_BF16 ? 2 : 4; }

struct Shape {
  int B, Hq, Hkv, D, T, max_q, window, q_dtype, kv_dtype, o_dtype;
};

int check_shape(const Shape& s) {
  if (s.B < 1 || s.B > 4096 || s.Hq < 1 || s.Hq > 4096 || s.Hkv < 1 || s.Hq % s.Hkv != 0) return SPEC_ERR_INVALID_ARG;
  if (s.T < 0 || s.window < 0) return SPEC_ERR_INVALID_ARG;
  if (s.max_q < 1) return SPEC_ERR_INVALID_ARG;
  if (s.kv_dtype != SPEC_F32 && s.kv_dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (s.o_dtype != SPEC_F32 && s.o_dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (s.q_dtype != SPEC_F32 && s.q_dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (s.q_dtype != s.kv_dtype) return SPEC_ERR_UNSUPPORTED;
  if (s.D != 64 && s.D != 128) return SPEC_ERR_UNSUPPORTED;
  if (s.Hq / s.Hkv > 32 || s.T > kMaxTokens) return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

// a 16-byte aligned base whose strides are multiples of 16 bytes
bool vector_layout(const void* p, int dtype, int64_t s0, int64_t s1, int64_t s2 = 0) {
  const int64_t per = 16 / elem_bytes(dtype);
  return p && aligned(p, 16) && s0 >= 0 && s1 >= 0 && s2 >= 0 && s0 % per == 0 && s1 % per == 0 && s2 % per == 0;
}
bool o_layout(const void* o, int dtype, int64_t st, int64_t sh) {
  return o && st >= 0 && sh >= 0 && aligned(o, elem_bytes(dtype));
}
bool int_layout(const int32_t* p) { return p && aligned(p, 4); }

int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return SPEC_ERR_INVALID_ARG;
  return !ws || have < need || !aligned(ws, 256) ? SPEC_ERR_WORKSPACE : SPEC_OK;
}

int serve_grid() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
  return sms < specv::kServeMaxGrid ? sms : specv::kServeMaxGrid;
}

// Few query rows per kv head: the mma.sync kernel; more rows need the tcgen05 kernel's tiles.  Measured at
// 8 sequences of 16K-32K, 32/8 heads, mma.sync against tcgen05: 4 rows 115 and 150 us, 16 rows 122 and
// 151 us, 24 rows 142 and 164 us, 32 rows 157 and 165 us; one sequence of 2000 tokens, where launches
// count (1 against 3 at least): 27-29 and 31-36 us.
bool use_mma(int kv_dtype, int max_q, int G) {
  return kv_dtype == SPEC_BF16 && (int64_t)max_q * G <= specv::kMmaMaxRows;
}
int chunk_row_tile(int kv_dtype) { return kv_dtype == SPEC_BF16 ? specv::kTcRows : specv::kF32Rows; }

constexpr float kLog2e = 1.4426950408889634f;
// what multiplies the scores, scale * log2(e), has to be finite as well
bool good_scale(float scale) { return scale >= 0.f && isfinite(scale * kLog2e); }

ServeAttnParams base_params(const Shape& s, float scale) {
  ServeAttnParams p;
  memset(&p, 0, sizeof(p));
  p.B = s.B; p.Hq = s.Hq; p.Hkv = s.Hkv; p.G = s.Hq / s.Hkv; p.D = s.D; p.T = s.T; p.max_q = s.max_q;
  p.window = s.window;
  p.o_bf16 = s.o_dtype == SPEC_BF16;
  p.scale_log2 = (scale != 0.f ? scale : 1.0f / sqrtf((float)s.D)) * kLog2e;
  return p;
}

// K or V as (column in half, token, half of D, kv head, page): one box is a page's rows, or a tile's
// 128 where pages are larger; packed rows are one page.  False where the layout does not suit a map.
bool encode_kv(CUtensorMap* m, const void* base, const ServeAttnParams& p) {
  specv::EncodeTiledFn fn = specv::encode_fn();
  if (!fn) return false;
  const int64_t tokens = p.paged ? p.page_size : p.T, pages = p.paged ? p.num_pages : 1;
  const int64_t sp = p.paged ? p.kv_sp : p.kv_st * p.T;
  cuuint64_t dims[5] = {64, (cuuint64_t)tokens, (cuuint64_t)p.D / 64, (cuuint64_t)p.Hkv, (cuuint64_t)pages};
  cuuint64_t strides[4] = {(cuuint64_t)p.kv_st * 2, 128, (cuuint64_t)p.kv_sh * 2, (cuuint64_t)sp * 2};
  for (cuuint64_t s : strides)
    if (s == 0 || s >= ((cuuint64_t)1 << 40)) return false;
  const bool whole = p.tma_page_keys == specv::kTcKeys;
  cuuint32_t box[5] = {64, (cuuint32_t)p.tma_page_keys, whole ? (cuuint32_t)p.D / 64 : 1u, 1, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// `keys`: more keys than this no row sees.
int launch_chunk(ServeAttnParams& p, int kv_dtype, int64_t keys, void* ws, cudaStream_t stream) {
  const bool bf16 = kv_dtype == SPEC_BF16;
  p.row_tile = chunk_row_tile(kv_dtype);
  p.unit_keys = bf16 ? specv::kTcKeys : specv::kF32Keys;
  p.min_units = 2;
  // measured 7000 cycles a piece on the tcgen05 kernel, whose units take 2700; the fp32 kernel's units take
  // as long and its pieces start and end faster
  p.piece_cost = bf16 ? 3.f : 1.f;
  p.cut_cost = bf16 ? 7.f : 3.f;
  specv::chunk_workspace_carve(ws, &p);
  CUtensorMap tm[2];
  if (bf16) {
    memset(tm, 0, sizeof(tm));
    // whole tiles per copy, or pages of at least kTmaMinPage tokens that divide a tile
    if (!p.paged || p.page_size % specv::kTcKeys == 0) p.tma_page_keys = specv::kTcKeys;
    else if (specv::kTcKeys % p.page_size == 0 && p.page_size >= specv::kTmaMinPage) p.tma_page_keys = p.page_size;
    // a copy of a packed tile is never issued where T < kTcKeys
    p.use_tma = p.tma_page_keys > 0 && encode_kv(&tm[0], p.k, p) && encode_kv(&tm[1], p.v, p);
  }
  // a tile's rows see at most `keys` keys and those that its tokens lie apart
  const int64_t span = keys + (p.row_tile + p.G - 1) / p.G;
  p.light = p.B <= specv::kLightMaxB && span / p.unit_keys + 2 <= specv::kLightUnits;
  p.first = p.light && !p.k_new;
  if (!p.first && specv::launch_chunk_prepare(p, elem_bytes(kv_dtype), stream) != cudaSuccess) return SPEC_ERR_CUDA;
  const cudaError_t e = bf16 ? specv::launch_chunk_tc(p, &tm[0], &tm[1], stream) : specv::launch_chunk_f32(p, stream);
  if (e != cudaSuccess) return SPEC_ERR_CUDA;
  return p.light || specv::launch_chunk_merge(p, stream) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t spec_serve_struct_size(int which) {
  switch (which) {
    case 0: return sizeof(spec_paged_args);
    case 1: return sizeof(spec_prefill_args);
    case 2: return sizeof(spec_logprob_args);
    default: return 0;
  }
}

// ------------------------------------------------------------------ spec_paged_attn
static Shape paged_shape(const spec_paged_args* a) {
  // no chunk is longer than all rows together
  const int max_q = a->max_q > a->T && a->T > 0 ? a->T : a->max_q;
  return Shape{a->B, a->Hq, a->Hkv, a->D, a->T, max_q, a->window, a->q_dtype, a->kv_dtype, a->o_dtype};
}

size_t spec_paged_attn_workspace(const spec_paged_args* a) {
  if (!a || check_shape(paged_shape(a)) != SPEC_OK) return 0;
  const int G = a->Hq / a->Hkv;
  return use_mma(a->kv_dtype, paged_shape(a).max_q, G)
             ? specv::mma_workspace_bytes(a->D)
             : specv::chunk_workspace_bytes(a->T, G, a->B, a->D, chunk_row_tile(a->kv_dtype));
}

int spec_paged_attn(const spec_paged_args* a, spec_stream_t stream) {
  if (!a) return SPEC_ERR_INVALID_ARG;
  const Shape s = paged_shape(a);
  int st = check_shape(s);
  if (st != SPEC_OK) return st;
  if (a->page_size < 1 || a->page_size > 65536 || a->num_pages < 1 || a->table_cols < 1 || a->table_stride < 0 ||
      (int64_t)a->table_cols * a->page_size > (1 << 30))
    return SPEC_ERR_INVALID_ARG;
  if (!good_scale(a->scale)) return SPEC_ERR_INVALID_ARG;
  if ((a->k_new == nullptr) != (a->v_new == nullptr)) return SPEC_ERR_INVALID_ARG;
  if (a->T == 0) return SPEC_OK;
  if (!vector_layout(a->q, a->q_dtype, a->q_stride_t, a->q_stride_h) ||
      !vector_layout(a->k_pages, a->kv_dtype, a->kv_stride_p, a->kv_stride_h, a->kv_stride_t) ||
      !vector_layout(a->v_pages, a->kv_dtype, 0, 0) || !o_layout(a->o, a->o_dtype, a->o_stride_t, a->o_stride_h))
    return SPEC_ERR_INVALID_ARG;
  if (a->k_new && (!vector_layout(a->k_new, a->kv_dtype, a->new_stride_t, a->new_stride_h) ||
                   !vector_layout(a->v_new, a->kv_dtype, 0, 0)))
    return SPEC_ERR_INVALID_ARG;
  if (!int_layout(a->page_table) || !int_layout(a->q_start) || !int_layout(a->kv_len)) return SPEC_ERR_INVALID_ARG;
  if ((st = check_workspace(a->workspace, a->workspace_bytes, spec_paged_attn_workspace(a))) != SPEC_OK) return st;

  ServeAttnParams p = base_params(s, a->scale);
  p.paged = 1;
  p.page_size = a->page_size; p.num_pages = a->num_pages; p.table_cols = a->table_cols;
  p.page_shift = -1;
  for (int i = 0; i <= 16; ++i)
    if (a->page_size == 1 << i) p.page_shift = i;
  p.table = a->page_table; p.table_stride = a->table_stride;
  p.q_start = a->q_start; p.kv_len = a->kv_len;
  p.q = a->q; p.q_st = a->q_stride_t; p.q_sh = a->q_stride_h;
  p.k = a->k_pages; p.v = a->v_pages;
  p.kv_sp = a->kv_stride_p; p.kv_sh = a->kv_stride_h; p.kv_st = a->kv_stride_t;
  p.k_new = a->k_new; p.v_new = a->v_new; p.new_st = a->new_stride_t; p.new_sh = a->new_stride_h;
  p.o = a->o; p.o_st = a->o_stride_t; p.o_sh = a->o_stride_h;
  if ((p.grid = serve_grid()) < 1) return SPEC_ERR_CUDA;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  int64_t keys = (int64_t)a->table_cols * a->page_size;
  if (!use_mma(a->kv_dtype, s.max_q, p.G))
    return launch_chunk(p, a->kv_dtype, a->window > 0 && a->window < keys ? a->window : keys, a->workspace, cs);
  // the longest segment a sequence can have: the table's capacity, or its window
  if (a->window > 0 && keys > (int64_t)a->window + s.max_q + 15) keys = (int64_t)a->window + s.max_q + 15;
  p.direct = keys <= specv::kMmaDirectKeys;
  specv::mma_workspace_carve(a->workspace, &p);
  return specv::launch_paged_mma(p, cs) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

// ------------------------------------------------------------------ spec_prefill_attn
static Shape prefill_shape(const spec_prefill_args* a) {
  return Shape{a->B, a->Hq, a->Hkv, a->D, a->T, a->T > 1 ? a->T : 1, a->window, a->q_dtype, a->kv_dtype, a->o_dtype};
}

size_t spec_prefill_attn_workspace(const spec_prefill_args* a) {
  if (!a || check_shape(prefill_shape(a)) != SPEC_OK) return 0;
  return specv::chunk_workspace_bytes(a->T, a->Hq / a->Hkv, a->B, a->D, chunk_row_tile(a->kv_dtype));
}

int spec_prefill_attn(const spec_prefill_args* a, spec_stream_t stream) {
  if (!a) return SPEC_ERR_INVALID_ARG;
  const Shape s = prefill_shape(a);
  int st = check_shape(s);
  if (st != SPEC_OK) return st;
  if (!good_scale(a->scale)) return SPEC_ERR_INVALID_ARG;
  if (a->T == 0) return SPEC_OK;
  if (!vector_layout(a->q, a->q_dtype, a->q_stride_t, a->q_stride_h) ||
      !vector_layout(a->k, a->kv_dtype, a->kv_stride_t, a->kv_stride_h) || !vector_layout(a->v, a->kv_dtype, 0, 0) ||
      !o_layout(a->o, a->o_dtype, a->o_stride_t, a->o_stride_h) || !int_layout(a->seq_start))
    return SPEC_ERR_INVALID_ARG;
  if ((st = check_workspace(a->workspace, a->workspace_bytes, spec_prefill_attn_workspace(a))) != SPEC_OK) return st;

  ServeAttnParams p = base_params(s, a->scale);
  p.q_start = a->seq_start;
  p.q = a->q; p.q_st = a->q_stride_t; p.q_sh = a->q_stride_h;
  p.k = const_cast<void*>(a->k); p.v = const_cast<void*>(a->v);
  p.kv_st = a->kv_stride_t; p.kv_sh = a->kv_stride_h;
  p.o = a->o; p.o_st = a->o_stride_t; p.o_sh = a->o_stride_h;
  if ((p.grid = serve_grid()) < 1) return SPEC_ERR_CUDA;
  return launch_chunk(p, a->kv_dtype, a->window > 0 && a->window < a->T ? a->window : a->T, a->workspace,
                      reinterpret_cast<cudaStream_t>(stream));
}

// ------------------------------------------------------------------ spec_token_logprobs
static int check_logprobs(const spec_logprob_args* a) {
  if (a->N < 0 || a->N > (1 << 24) || a->V < 1 || a->V > (1 << 24)) return SPEC_ERR_INVALID_ARG;
  if (a->K < 0 || a->K > a->V) return SPEC_ERR_INVALID_ARG;
  if (a->K > 32) return SPEC_ERR_UNSUPPORTED;
  if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}

size_t spec_token_logprobs_workspace(const spec_logprob_args* a) {
  if (!a || check_logprobs(a) != SPEC_OK) return 0;
  return specv::logprob_workspace_bytes(a->N, a->V, a->K);
}

int spec_token_logprobs(const spec_logprob_args* a, spec_stream_t stream) {
  if (!a) return SPEC_ERR_INVALID_ARG;
  int st = check_logprobs(a);
  if (st != SPEC_OK) return st;
  if (a->N == 0) return SPEC_OK;
  if (!a->logits || !aligned(a->logits, elem_bytes(a->dtype)) || a->logits_stride < a->V) return SPEC_ERR_INVALID_ARG;
  if ((a->tokens == nullptr) != (a->logprobs == nullptr)) return SPEC_ERR_INVALID_ARG;
  if ((a->top_ids == nullptr) != (a->K == 0) || (a->top_logprobs == nullptr) != (a->K == 0)) return SPEC_ERR_INVALID_ARG;
  if (!a->logprobs && !a->entropy && a->K == 0) return SPEC_ERR_INVALID_ARG;
  const void* words[5] = {a->tokens, a->logprobs, a->entropy, a->top_ids, a->top_logprobs};
  for (const void* w : words)
    if (!aligned(w, 4)) return SPEC_ERR_INVALID_ARG;
  if ((st = check_workspace(a->workspace, a->workspace_bytes, spec_token_logprobs_workspace(a))) != SPEC_OK) return st;
  LogprobParams p;
  memset(&p, 0, sizeof(p));
  p.N = a->N; p.V = a->V; p.K = a->K;
  p.bf16 = a->dtype == SPEC_BF16;
  p.slices = specv::logprob_slices(a->N, a->V);
  p.logits = a->logits; p.stride = a->logits_stride;
  p.tokens = a->tokens; p.logprobs = a->logprobs; p.entropy = a->entropy;
  p.top_ids = a->top_ids; p.top_lp = a->top_logprobs;
  specv::logprob_workspace_carve(a->workspace, &p);
  return specv::launch_token_logprobs(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? SPEC_OK
                                                                                               : SPEC_ERR_CUDA;
}

}  // extern "C"
