// C ABI of the cache operators (include/spec_cache.h): argument validation, workspace sizing and kernel
// launches.  As in serve_api.cpp nothing here allocates memory or keeps state between calls.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "cache_internal.h"
#include "spec_cache.h"

namespace {

using specv::Kv8Params;
using specv::PageArrays;
using specv::PageParams;
using specv::RotaryParams;

constexpr int64_t kMaxTokens = 1 << 22;
constexpr size_t kStatusBytes = 256;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
// a 16-byte aligned base whose strides are multiples of 16 bytes
bool vector_layout(const void* p, int elem, int64_t s0, int64_t s1, int64_t s2 = 0) {
  const int64_t per = 16 / elem;
  return p && aligned(p, 16) && s0 >= 0 && s1 >= 0 && s2 >= 0 && s0 % per == 0 && s1 % per == 0 && s2 % per == 0;
}
bool int_layout(const int32_t* p) { return p && aligned(p, 4); }
int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return SPEC_ERR_INVALID_ARG;
  return !ws || have < need || !aligned(ws, 256) ? SPEC_ERR_WORKSPACE : SPEC_OK;
}
int sm_grid() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
  return sms < specv::kServeMaxGrid ? sms : specv::kServeMaxGrid;
}
int log2_of(int n) {
  for (int i = 0; i <= 16; ++i)
    if (n == 1 << i) return i;
  return -1;
}
constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------ rotary
int check_rotary(const spec_rotary_args* a) {
  if (a->T < 0 || a->Hq < 0 || a->Hkv < 0 || a->Hq > 4096 || a->Hkv > 4096 || a->Hq + a->Hkv < 1) return SPEC_ERR_INVALID_ARG;
  if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (a->layout != SPEC_ROTARY_HALF && a->layout != SPEC_ROTARY_PAIRS) return SPEC_ERR_INVALID_ARG;
  if (a->inverse != 0 && a->inverse != 1) return SPEC_ERR_INVALID_ARG;
  if (a->D < 1 || a->rot < 2 || a->rot % 2 != 0 || a->rot > a->D) return SPEC_ERR_INVALID_ARG;
  const int64_t row = (int64_t)a->D * (a->dtype == SPEC_F32 ? 4 : 2);
  if (row % 16 != 0 || row > 2048 || a->T > kMaxTokens) return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

// ------------------------------------------------------------------ the cache in 8 bits
struct Cache8 {
  int B, Hkv, D, T, max_q, page_size, num_pages, table_cols, block;
};
int check_cache8(const Cache8& s) {
  if (s.B < 1 || s.B > 4096 || s.Hkv < 1 || s.Hkv > 4096 || s.T < 0 || s.max_q < 1) return SPEC_ERR_INVALID_ARG;
  if (s.D != 64 && s.D != 128) return SPEC_ERR_UNSUPPORTED;
  return s.T > kMaxTokens ? SPEC_ERR_UNSUPPORTED : SPEC_OK;
}
int check_pages8(const Cache8& s, int64_t table_stride) {
  if (s.page_size < 1 || s.page_size > 65536 || s.num_pages < 1 || s.table_cols < 1 || table_stride < 0 ||
      (int64_t)s.table_cols * s.page_size > (1 << 30))
    return SPEC_ERR_INVALID_ARG;
  return s.block < 1 || s.page_size % s.block != 0 ? SPEC_ERR_INVALID_ARG : SPEC_OK;
}
// the parts that the append and the attention share
template <typename Args>
bool cache8_layout(const Args* a) {
  return vector_layout(a->k_pages, 1, a->kv_stride_p, a->kv_stride_h, a->kv_stride_t) && vector_layout(a->v_pages, 1, 0, 0) &&
         a->k_exp && a->v_exp && a->exp_stride_p >= 0 && a->exp_stride_h >= 0 && int_layout(a->page_table) &&
         int_layout(a->q_start) && int_layout(a->kv_len);
}
// what the append writes does not overlap, as far as single strides say
template <typename Args>
bool cache8_writable(const Args* a) {
  auto apart = [](int n, int64_t stride, int row) { return n == 1 || stride >= row; };
  const int blocks = a->page_size / a->block;
  return a->k_pages != a->v_pages && a->k_exp != a->v_exp && apart(a->num_pages, a->kv_stride_p, a->D) &&
         apart(a->Hkv, a->kv_stride_h, a->D) && apart(a->page_size, a->kv_stride_t, a->D) &&
         apart(a->num_pages, a->exp_stride_p, blocks) && apart(a->Hkv, a->exp_stride_h, blocks);
}
template <typename Args>
Kv8Params cache8_params(const Args* a, int max_q) {
  Kv8Params p;
  memset(&p, 0, sizeof(p));
  p.B = a->B; p.Hkv = a->Hkv; p.D = a->D; p.T = a->T; p.max_q = max_q;
  p.paged = 1;
  p.page_size = a->page_size; p.num_pages = a->num_pages; p.table_cols = a->table_cols;
  p.page_shift = log2_of(a->page_size);
  p.table = a->page_table; p.table_stride = a->table_stride;
  p.q_start = a->q_start; p.kv_len = a->kv_len;
  p.k = a->k_pages; p.v = a->v_pages;
  p.kv_sp = a->kv_stride_p; p.kv_sh = a->kv_stride_h; p.kv_st = a->kv_stride_t;
  p.k_exp = a->k_exp; p.v_exp = a->v_exp; p.exp_sp = a->exp_stride_p; p.exp_sh = a->exp_stride_h;
  p.block = a->block; p.block_shift = log2_of(a->block);
  p.k_new = a->k_new; p.v_new = a->v_new; p.new_st = a->new_stride_t; p.new_sh = a->new_stride_h;
  p.status = reinterpret_cast<uint32_t*>(a->workspace);
  return p;
}

Cache8 paged8_shape(const spec_paged8_args* a) {
  const int max_q = a->max_q > a->T && a->T > 0 ? a->T : a->max_q;  // no chunk is longer than all rows together
  return Cache8{a->B, a->Hkv, a->D, a->T, max_q, a->page_size, a->num_pages, a->table_cols, a->block};
}
int check_paged8(const spec_paged8_args* a) {
  const int st = check_cache8(paged8_shape(a));
  if (st != SPEC_OK) return st;
  if (a->Hq < 1 || a->Hq > 4096 || a->Hq % a->Hkv != 0 || a->window < 0) return SPEC_ERR_INVALID_ARG;
  if (a->o_dtype != SPEC_F32 && a->o_dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (a->q_dtype != SPEC_F32 && a->q_dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  return a->q_dtype != SPEC_BF16 || a->Hq / a->Hkv > 32 ? SPEC_ERR_UNSUPPORTED : SPEC_OK;
}
bool few_rows(const spec_paged8_args* a) {
  return (int64_t)paged8_shape(a).max_q * (a->Hq / a->Hkv) <= specv::kMmaMaxRows;
}

// ------------------------------------------------------------------ pages
template <typename Args>
int check_tables(const Args* a) {
  if (a->B < 1 || a->B > 4096 || a->table_cols < 1 || (int64_t)a->B * a->table_cols > (1 << 26)) return SPEC_ERR_INVALID_ARG;
  if (a->num_pages < 1 || a->num_pages > (1 << 24) || a->num_arrays < 0 || a->num_arrays > 4096) return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}
// an output is its input, or (as far as its first element says) another tensor
template <typename Args>
bool table_layout(const Args* a) {
  if (!int_layout(a->page_table) || !int_layout(a->table_out) || a->table_stride < 0 || a->table_out_stride < 0) return false;
  if (a->B > 1 && a->table_out_stride < a->table_cols) return false;  // rows of an output do not overlap
  return a->page_table != a->table_out || a->B == 1 || a->table_stride == a->table_out_stride;
}
int check_arrays(const spec_page_array* arrays, int n) {
  if (n > 0 && !arrays) return SPEC_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    const spec_page_array& x = arrays[i];
    if (!x.base || x.page_bytes < 1 || x.page_bytes > ((int64_t)1 << 32) || x.stride_bytes < x.page_bytes) return SPEC_ERR_INVALID_ARG;
  }
  return SPEC_OK;
}
// copies in launches of as many arrays as fit one's parameters
int copy_pages(const PageParams& p, const spec_page_array* arrays, int n, int max_pairs, cudaStream_t stream) {
  for (int at = 0; at < n && max_pairs > 0;) {
    PageArrays a;
    memset(&a, 0, sizeof(a));
    for (; at < n && a.n < PageArrays::kMax; ++at) {
      const spec_page_array& x = arrays[at];
      const int64_t pieces = (x.page_bytes + specv::kPagePiece - 1) / specv::kPagePiece;
      a.base[a.n] = reinterpret_cast<char*>(x.base);
      a.stride[a.n] = x.stride_bytes;
      a.bytes[a.n] = x.page_bytes;
      a.pieces[a.n + 1] = a.pieces[a.n] + (int32_t)pieces;  // at most 48 * 2^18
      ++a.n;
    }
    if (specv::launch_page_copy(p, a, max_pairs, stream) != cudaSuccess) return SPEC_ERR_CUDA;
  }
  return SPEC_OK;
}

}  // namespace

extern "C" {

size_t spec_cache_struct_size(int which) {
  switch (which) {
    case 0: return sizeof(spec_rotary_args);
    case 1: return sizeof(spec_kv8_append_args);
    case 2: return sizeof(spec_paged8_args);
    case 3: return sizeof(spec_page_fork_args);
    case 4: return sizeof(spec_page_compact_args);
    case 5: return sizeof(spec_page_array);
    default: return 0;
  }
}

// ------------------------------------------------------------------ spec_rotary
size_t spec_rotary_workspace(const spec_rotary_args* a) { return a && check_rotary(a) == SPEC_OK ? kStatusBytes : 0; }

int spec_rotary(const spec_rotary_args* a, spec_stream_t stream) {
  if (!a) return SPEC_ERR_INVALID_ARG;
  int st = check_rotary(a);
  if (st != SPEC_OK) return st;
  if (!(a->amplitude >= 0.f) || !isfinite(a->amplitude)) return SPEC_ERR_INVALID_ARG;
  if (!a->positions && (a->B < 1 || a->B > 4096)) return SPEC_ERR_INVALID_ARG;
  if (a->T == 0) return SPEC_OK;
  const int elem = a->dtype == SPEC_F32 ? 4 : 2;
  if (a->Hq > 0 && (!vector_layout(a->q, elem, a->q_stride_t, a->q_stride_h) ||
                    !vector_layout(a->q_out, elem, a->qo_stride_t, a->qo_stride_h)))
    return SPEC_ERR_INVALID_ARG;
  if (a->Hkv > 0 && (!vector_layout(a->k, elem, a->k_stride_t, a->k_stride_h) ||
                     !vector_layout(a->k_out, elem, a->ko_stride_t, a->ko_stride_h)))
    return SPEC_ERR_INVALID_ARG;
  const bool q_in = a->q == a->q_out, k_in = a->k == a->k_out;
  // in place the strides have to be the same where they are stepped over
  if (a->Hq > 0 && q_in && ((a->T > 1 && a->q_stride_t != a->qo_stride_t) || (a->Hq > 1 && a->q_stride_h != a->qo_stride_h)))
    return SPEC_ERR_INVALID_ARG;
  if (a->Hkv > 0 && k_in && ((a->T > 1 && a->k_stride_t != a->ko_stride_t) || (a->Hkv > 1 && a->k_stride_h != a->ko_stride_h)))
    return SPEC_ERR_INVALID_ARG;
  // rows of an output do not overlap, as far as single strides say, and q and k have an output each
  if ((a->T > 1 && ((a->Hq > 0 && a->qo_stride_t < a->D) || (a->Hkv > 0 && a->ko_stride_t < a->D))) ||
      (a->Hq > 1 && a->qo_stride_h < a->D) || (a->Hkv > 1 && a->ko_stride_h < a->D))
    return SPEC_ERR_INVALID_ARG;
  if (a->Hq > 0 && a->Hkv > 0 && (a->q_out == a->k_out || a->q_out == a->k || a->k_out == a->q)) return SPEC_ERR_INVALID_ARG;
  if (!a->steps || !aligned(a->steps, 8)) return SPEC_ERR_INVALID_ARG;
  if (a->positions ? !aligned(a->positions, 4) : !int_layout(a->q_start) || !int_layout(a->kv_len)) return SPEC_ERR_INVALID_ARG;
  if ((st = check_workspace(a->workspace, a->workspace_bytes, kStatusBytes)) != SPEC_OK) return st;
  RotaryParams p;
  memset(&p, 0, sizeof(p));
  p.T = a->T; p.Hq = a->Hq; p.Hkv = a->Hkv; p.D = a->D; p.rot = a->rot; p.B = a->B;
  p.pairs = a->layout == SPEC_ROTARY_PAIRS;
  p.f32 = a->dtype == SPEC_F32;
  p.negate = a->inverse;
  p.amplitude = a->amplitude != 0.f ? a->amplitude : 1.f;
  p.q = a->q; p.q_st = a->q_stride_t; p.q_sh = a->q_stride_h;
  p.k = a->k; p.k_st = a->k_stride_t; p.k_sh = a->k_stride_h;
  p.qo = a->q_out; p.qo_st = a->qo_stride_t; p.qo_sh = a->qo_stride_h;
  p.ko = a->k_out; p.ko_st = a->ko_stride_t; p.ko_sh = a->ko_stride_h;
  p.copy_q = !q_in && a->rot < a->D;
  p.copy_k = !k_in && a->rot < a->D;
  p.steps = reinterpret_cast<const unsigned long long*>(a->steps);
  p.positions = a->positions;
  p.q_start = a->q_start; p.kv_len = a->kv_len;
  p.status = reinterpret_cast<uint32_t*>(a->workspace);
  const int sms = sm_grid();
  if (sms < 1) return SPEC_ERR_CUDA;
  // a token per CTA as long as that does not make waves
  for (p.tile = 1; p.tile < specv::kRotaryMaxTile && a->T > (int64_t)p.tile * sms * 4;) p.tile *= 2;
  return specv::launch_rotary(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

int spec_rotary_steps(int32_t rot, int32_t kind, double base, double factor, double length, double low, double high,
                      int64_t* steps, float* amplitude) {
  const double pi = 3.14159265358979323846;
  if (!steps || rot < 2 || rot % 2 != 0 || rot > 1024 || kind < SPEC_ROTARY_PLAIN || kind > SPEC_ROTARY_YARN) return SPEC_ERR_INVALID_ARG;
  if (!(base > 1) || !isfinite(base)) return SPEC_ERR_INVALID_ARG;
  if (kind != SPEC_ROTARY_PLAIN && (!(factor >= 1) || !isfinite(factor))) return SPEC_ERR_INVALID_ARG;
  const bool bands = kind == SPEC_ROTARY_BANDS || kind == SPEC_ROTARY_YARN;
  if (bands && (!(length > 0) || !isfinite(length) || !(low > 0) || !(low < high) || !isfinite(high))) return SPEC_ERR_INVALID_ARG;
  if (kind == SPEC_ROTARY_NTK) {
    if (rot == 2) return SPEC_ERR_INVALID_ARG;
    base *= pow(factor, rot / (rot - 2.0));
    if (!isfinite(base)) return SPEC_ERR_INVALID_ARG;
  }
  // pairs that make `turns` turns over `length` positions
  auto pair_of = [&](double turns) { return rot * log(length / (2 * pi * turns)) / (2 * log(base)); };
  double from = 0, to = 0;
  if (kind == SPEC_ROTARY_YARN) {
    from = fmax(floor(pair_of(high)), 0);
    to = fmin(ceil(pair_of(low)), rot - 1.0);
    if (!(to - from >= 0.001)) to = from + 0.001;
  }
  for (int i = 0; i < rot / 2; ++i) {
    double f = pow(base, -2.0 * i / rot);
    if (kind == SPEC_ROTARY_LINEAR) {
      f /= factor;
    } else if (kind == SPEC_ROTARY_BANDS) {
      const double waves = length * f / (2 * pi);  // length / wavelength
      const double share = fmin(fmax((waves - low) / (high - low), 0), 1);
      f = share * f + (1 - share) * f / factor;
    } else if (kind == SPEC_ROTARY_YARN) {
      const double ramp = fmin(fmax((i - from) / (to - from), 0), 1);
      f = (1 - ramp) * f + ramp * f / factor;
    }
    steps[i] = (int64_t)(f / (2 * pi) * 18446744073709551616.0);  // f <= 1: below 2^62
  }
  if (amplitude) *amplitude = kind == SPEC_ROTARY_YARN ? (float)(1 + 0.1 * log(factor)) : 1.f;
  return SPEC_OK;
}

// ------------------------------------------------------------------ spec_kv8_append
static Cache8 append_shape(const spec_kv8_append_args* a) {
  return Cache8{a->B, a->Hkv, a->D, a->T, a->T > 1 ? a->T : 1, a->page_size, a->num_pages, a->table_cols, a->block};
}
static int check_append(const spec_kv8_append_args* a) {
  const int st = check_cache8(append_shape(a));
  if (st != SPEC_OK) return st;
  return a->src_dtype != SPEC_F32 && a->src_dtype != SPEC_BF16 ? SPEC_ERR_INVALID_ARG : SPEC_OK;
}

size_t spec_kv8_append_workspace(const spec_kv8_append_args* a) { return a && check_append(a) == SPEC_OK ? kStatusBytes : 0; }

int spec_kv8_append(const spec_kv8_append_args* a, spec_stream_t stream) {
  if (!a) return SPEC_ERR_INVALID_ARG;
  int st = check_append(a);
  if (st != SPEC_OK || (st = check_pages8(append_shape(a), a->table_stride)) != SPEC_OK) return st;
  if (a->T == 0) return SPEC_OK;
  const int elem = a->src_dtype == SPEC_F32 ? 4 : 2;
  if (!cache8_layout(a) || !cache8_writable(a) || !vector_layout(a->k_new, elem, a->new_stride_t, a->new_stride_h) ||
      !vector_layout(a->v_new, elem, 0, 0))
    return SPEC_ERR_INVALID_ARG;
  if ((st = check_workspace(a->workspace, a->workspace_bytes, kStatusBytes)) != SPEC_OK) return st;
  Kv8Params p = cache8_params(a, append_shape(a).max_q);
  p.src_f32 = a->src_dtype == SPEC_F32;
  if ((p.grid = sm_grid()) < 1) return SPEC_ERR_CUDA;
  return specv::launch_kv8_append(p, true, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

// ------------------------------------------------------------------ spec_paged_attn8
size_t spec_paged_attn8_workspace(const spec_paged8_args* a) {
  if (!a || check_paged8(a) != SPEC_OK) return 0;
  return few_rows(a) ? specv::mma_workspace_bytes(a->D)
                     : specv::chunk_workspace_bytes(a->T, a->Hq / a->Hkv, a->B, a->D, specv::kTcRows);
}

int spec_paged_attn8(const spec_paged8_args* a, spec_stream_t stream) {
  if (!a) return SPEC_ERR_INVALID_ARG;
  int st = check_paged8(a);
  if (st != SPEC_OK || (st = check_pages8(paged8_shape(a), a->table_stride)) != SPEC_OK) return st;
  if (!(a->scale >= 0.f) || !isfinite(a->scale * kLog2e)) return SPEC_ERR_INVALID_ARG;
  if ((a->k_new == nullptr) != (a->v_new == nullptr)) return SPEC_ERR_INVALID_ARG;
  if (a->T == 0) return SPEC_OK;
  if (!cache8_layout(a) || !vector_layout(a->q, 2, a->q_stride_t, a->q_stride_h) || !a->o || a->o_stride_t < 0 ||
      a->o_stride_h < 0 || !aligned(a->o, a->o_dtype == SPEC_F32 ? 4 : 2))
    return SPEC_ERR_INVALID_ARG;
  // rows of o do not overlap, as far as single strides say
  if ((a->T > 1 && a->o_stride_t < a->D) || (a->Hq > 1 && a->o_stride_h < a->D)) return SPEC_ERR_INVALID_ARG;
  if (a->k_new && (!cache8_writable(a) || !vector_layout(a->k_new, 2, a->new_stride_t, a->new_stride_h) || !vector_layout(a->v_new, 2, 0, 0)))
    return SPEC_ERR_INVALID_ARG;
  if ((st = check_workspace(a->workspace, a->workspace_bytes, spec_paged_attn8_workspace(a))) != SPEC_OK) return st;

  Kv8Params p = cache8_params(a, paged8_shape(a).max_q);
  p.Hq = a->Hq; p.G = a->Hq / a->Hkv; p.window = a->window;
  p.q = a->q; p.q_st = a->q_stride_t; p.q_sh = a->q_stride_h;
  p.o = a->o; p.o_st = a->o_stride_t; p.o_sh = a->o_stride_h; p.o_bf16 = a->o_dtype == SPEC_BF16;
  p.scale_log2 = (a->scale != 0.f ? a->scale : 1.0f / sqrtf((float)a->D)) * kLog2e;
  if ((p.grid = sm_grid()) < 1) return SPEC_ERR_CUDA;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  int64_t keys = (int64_t)a->table_cols * a->page_size;
  if (few_rows(a)) {
    // the longest segment a sequence can have: the table's capacity, or its window
    if (a->window > 0 && keys > (int64_t)a->window + p.max_q + 15) keys = (int64_t)a->window + p.max_q + 15;
    p.direct = keys <= specv::kMmaDirectKeys;
    p.first = !a->k_new;
    specv::mma_workspace_carve(a->workspace, &p);
    if (a->k_new && specv::launch_kv8_append(p, true, cs) != cudaSuccess) return SPEC_ERR_CUDA;
    return specv::launch_paged8_mma(p, cs) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
  }
  p.row_tile = specv::kTcRows;
  p.unit_keys = specv::kTcKeys;
  p.min_units = 2;
  p.piece_cost = 3.f;
  p.cut_cost = 7.f;  // 3, 7 and 12: 24 mixed sequences, rows of 64, 125 us each; 16 of up to 700 tokens, rows of 128, 574, 574 and 560
  p.share_piece = 3;
  specv::chunk_workspace_carve(a->workspace, &p);
  if (a->window > 0 && a->window < keys) keys = a->window;
  // a tile's rows see at most `keys` keys and those that its tokens lie apart
  const int64_t span = keys + (p.row_tile + p.G - 1) / p.G;
  p.light = p.B <= specv::kLightMaxB && span / p.unit_keys + 2 <= specv::kLightUnits;
  p.first = p.light && !a->k_new;
  if (!p.light) {
    // the plan clears the status; the append runs behind it
    Kv8Params plan = p;
    plan.k_new = plan.v_new = nullptr;
    if (specv::launch_chunk_prepare(plan, 2, cs) != cudaSuccess) return SPEC_ERR_CUDA;
  }
  if (a->k_new && specv::launch_kv8_append(p, p.light, cs) != cudaSuccess) return SPEC_ERR_CUDA;
  if (specv::launch_chunk8_tc(p, cs) != cudaSuccess) return SPEC_ERR_CUDA;
  return p.light || specv::launch_chunk_merge(p, cs) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

// ------------------------------------------------------------------ spec_page_fork
static int check_fork(const spec_page_fork_args* a) {
  const int st = check_tables(a);
  if (st != SPEC_OK) return st;
  return a->page_size < 1 || a->page_size > 65536 || (int64_t)a->table_cols * a->page_size > (1 << 30) ? SPEC_ERR_INVALID_ARG
                                                                                                        : SPEC_OK;
}

size_t spec_page_fork_workspace(const spec_page_fork_args* a) {
  return a && check_fork(a) == SPEC_OK ? specv::page_workspace_bytes(a->B, a->table_cols, a->num_pages, false) : 0;
}

int spec_page_fork(const spec_page_fork_args* a, spec_stream_t stream) {
  if (!a) return SPEC_ERR_INVALID_ARG;
  int st = check_fork(a);
  if (st != SPEC_OK || (st = check_arrays(a->arrays, a->num_arrays)) != SPEC_OK) return st;
  if (!table_layout(a) || !int_layout(a->held) || !int_layout(a->kv_len) || !int_layout(a->refs) || !int_layout(a->parent) ||
      !int_layout(a->held_out) || !int_layout(a->kv_len_out) || !int_layout(a->refs_out) || !aligned(a->grow, 4))
    return SPEC_ERR_INVALID_ARG;
  if ((st = check_workspace(a->workspace, a->workspace_bytes, spec_page_fork_workspace(a))) != SPEC_OK) return st;
  PageParams p;
  memset(&p, 0, sizeof(p));
  p.B = a->B; p.cols = a->table_cols; p.page_size = a->page_size; p.num_pages = a->num_pages;
  p.table = a->page_table; p.table_st = a->table_stride;
  p.held = a->held; p.kv_len = a->kv_len; p.refs = a->refs; p.parent = a->parent; p.grow = a->grow;
  p.table_out = a->table_out; p.table_out_st = a->table_out_stride;
  p.held_out = a->held_out; p.kv_len_out = a->kv_len_out; p.refs_out = a->refs_out;
  specv::page_workspace_carve(a->workspace, &p);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (specv::launch_page_fork(p, cs) != cudaSuccess) return SPEC_ERR_CUDA;
  // without grow no page is written to, so none is copied
  return a->grow ? copy_pages(p, a->arrays, a->num_arrays, a->B, cs) : SPEC_OK;
}

// ------------------------------------------------------------------ spec_page_compact
size_t spec_page_compact_workspace(const spec_page_compact_args* a) {
  return a && check_tables(a) == SPEC_OK ? specv::page_workspace_bytes(a->B, a->table_cols, a->num_pages, true) : 0;
}

int spec_page_compact(const spec_page_compact_args* a, spec_stream_t stream) {
  if (!a) return SPEC_ERR_INVALID_ARG;
  int st = check_tables(a);
  if (st != SPEC_OK || (st = check_arrays(a->arrays, a->num_arrays)) != SPEC_OK) return st;
  if (!table_layout(a) || !int_layout(a->held) || !int_layout(a->refs) || !int_layout(a->refs_out) || !aligned(a->moved, 4) ||
      !aligned(a->num_live, 4))
    return SPEC_ERR_INVALID_ARG;
  if ((st = check_workspace(a->workspace, a->workspace_bytes, spec_page_compact_workspace(a))) != SPEC_OK) return st;
  PageParams p;
  memset(&p, 0, sizeof(p));
  p.B = a->B; p.cols = a->table_cols; p.num_pages = a->num_pages; p.compact = 1;
  p.table = a->page_table; p.table_st = a->table_stride;
  p.held = a->held; p.refs = a->refs;
  p.table_out = a->table_out; p.table_out_st = a->table_out_stride;
  p.refs_out = a->refs_out; p.moved_out = a->moved; p.num_live = a->num_live;
  specv::page_workspace_carve(a->workspace, &p);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (specv::launch_page_compact(p, cs) != cudaSuccess) return SPEC_ERR_CUDA;
  return copy_pages(p, a->arrays, a->num_arrays, a->num_pages / 2, cs);
}

}  // extern "C"
