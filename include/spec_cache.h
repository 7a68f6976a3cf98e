/*
 * spec_cache.h -- C ABI of libspecverify, part three: what a serving loop does to its paged KV cache
 * around the attention of spec_serve.h, on the same GPU and with the same conventions.
 *
 *   spec_rotary          Rotary positions of the new tokens' queries and keys.
 *   spec_kv8_append      The new tokens' K/V written into a paged cache held in 8 bits (e4m3) with a
 *                        power-of-two scale for each block of tokens and kv head.
 *   spec_paged_attn8     spec_paged_attn over such a cache.
 *   spec_page_fork       Sequences forked, freed and grown: page tables and holders of pages, with
 *                        copies of shared pages that are about to be written.
 *   spec_page_compact    The pages in use moved to the lowest ids.
 *
 * Conventions are those of spec_serve.h: device pointers owned by the caller, strides in ELEMENTS with
 * the innermost dimension contiguous, asynchronous calls on the given stream of the calling thread's
 * current device, no allocation, no global mutable state, host validation before any launch, negative
 * return codes, a caller workspace (256-byte aligned; calls that share one must not overlap, and that
 * includes replays of captured graphs) whose first 32-bit word is the call's device status, cleared by the
 * call.  A call can be captured into a CUDA graph; everything it reads from device memory is read anew
 * by each replay.  All five give the same result every time.
 *
 * The cache in 8 bits: k_pages, v_pages [num_pages, Hkv, page_size, D] of e4m3 (sign, 4 exponent bits, 3
 * mantissa bits, 448 the largest value) and k_exp, v_exp [num_pages, Hkv, page_size / block] of bytes.
 * Slot i of a page stands for e4m3 value * 2^(byte[i / block] - 127).  Bytes below 63 or above 191 count
 * as 63 and 191.  A power of two costs nothing in a format with an exponent of its own, multiplies
 * exactly, and a block whose scale grows keeps its old values exactly (but for those that become
 * subnormal).
 */
#ifndef SPEC_CACHE_H_
#define SPEC_CACHE_H_

#include "spec_serve.h"

#ifdef __cplusplus
extern "C" {
#endif

/* further flag of the device status word */
enum {
  SPEC_STATUS_NO_PAGE = 64 /* spec_page_fork: fewer free pages than needed */
};

/* ------------------------------------------------------------------------------------------
 * spec_rotary
 *
 * Row t at position p turns pair i of the first `rot` values of each head by p * f_i:
 *     (a, b) -> amplitude * (a cos - b sin, b cos + a sin),  angle = 2 pi * frac(p * steps[i] / 2^64)
 * (inverse: by -p * f_i, which with amplitude 1 undoes it, and is the gradient's way back).  Pair i is
 * values (i, i + rot / 2) (SPEC_ROTARY_HALF) or (2 i, 2 i + 1) (SPEC_ROTARY_PAIRS); values rot .. D - 1
 * pass through.  steps [rot / 2] are turns per position in units of 2^-64, so that p * steps[i] modulo
 * 2^64 is the phase without any rounding, however far p; spec_rotary_steps makes them.
 *   positions [T] int32, any value; or NULL: row q_start[b] + j of sequence b is at position
 *   kv_len[b] - n_b + j, as in spec_paged_attn; rows of no sequence are then left as they were, and so
 *   are those of sequences with bad data (SPEC_STATUS_BAD_RANGE, SPEC_STATUS_BAD_KV_LEN); a row that lies in
 *   several sequences belongs to the first of them.
 * Layout: q, q_out [T, Hq, D]; k, k_out [T, Hkv, D]; either may be missing (NULL with 0 heads).  An output
 *   that is its input (same pointer, same strides) is turned in place; otherwise none overlaps an input.
 *   Rows of an output do not overlap each other, so broadcast rows are not turned in place.
 * Types: dtype SPEC_BF16 or SPEC_F32 for all of them.  Strides are multiples of 16 bytes, pointers
 *   16-byte aligned (steps: 8).  The arithmetic is fp32, rounded once.
 * Limits: rows of 16 to 2048 bytes, a multiple of 16; rot even, 2 <= rot <= D; Hq, Hkv <= 4096;
 *   0 <= T <= 2^22 (0: nothing is launched); 1 <= B <= 4096 where positions is NULL; amplitude >= 0 and
 *   finite (0: 1).
 * ---------------------------------------------------------------------------------------- */
enum { SPEC_ROTARY_HALF = 0, SPEC_ROTARY_PAIRS = 1 };

typedef struct spec_rotary_args {
  int32_t T, Hq, Hkv, D, rot;
  int32_t layout, dtype, inverse;
  int32_t B;
  float amplitude;
  const void* q;
  int64_t q_stride_t, q_stride_h;
  const void* k;
  int64_t k_stride_t, k_stride_h;
  void* q_out;
  int64_t qo_stride_t, qo_stride_h;
  void* k_out;
  int64_t ko_stride_t, ko_stride_h;
  const int64_t* steps;
  const int32_t* positions;
  const int32_t* q_start;
  const int32_t* kv_len;
  void* workspace;
  size_t workspace_bytes;
} spec_rotary_args;

size_t spec_rotary_workspace(const spec_rotary_args* args);
int spec_rotary(const spec_rotary_args* args, spec_stream_t stream);

/* Turns per position in units of 2^-64 for i = 0 .. rot / 2 - 1, on the host.  With f_i = base^(-2 i / rot):
 *   SPEC_ROTARY_PLAIN   f_i
 *   SPEC_ROTARY_LINEAR  f_i / factor
 *   SPEC_ROTARY_NTK     f_i of the base  base * factor^(rot / (rot - 2))  (rot > 2)
 *   SPEC_ROTARY_BANDS   f_i where the wavelength 2 pi / f_i is below length / high, f_i / factor where it is
 *                       above length / low, between them mixed in proportion to length / wavelength
 *   SPEC_ROTARY_YARN    f_i (1 - r_i) + f_i / factor r_i, r_i the ramp from 0 to 1 between the pairs that make
 *                       `high` turns (rounded down) and `low` turns (rounded up) over `length` positions;
 *                       *amplitude = 1 + 0.1 ln factor (else 1)
 * length is the context that the model was trained with.  base > 1, factor >= 1, 0 < low < high and length > 0
 * where they are used, all finite. */
enum {
  SPEC_ROTARY_PLAIN = 0,
  SPEC_ROTARY_LINEAR = 1,
  SPEC_ROTARY_NTK = 2,
  SPEC_ROTARY_BANDS = 3,
  SPEC_ROTARY_YARN = 4
};
int spec_rotary_steps(int32_t rot, int32_t kind, double base, double factor, double length, double low, double high,
                      int64_t* steps, float* amplitude);

/* ------------------------------------------------------------------------------------------
 * spec_kv8_append
 *
 * Writes the K/V rows of the new tokens (sequence b: rows q_start[b] .. q_start[b + 1] - 1, the last n_b of
 * its kv_len[b] tokens) into their slots.  For each block of tokens that gets new ones, and each head:
 *     e  = the least integer in [-64, 64] with  max |x| <= 448 * 2^e  over the block's new finite values, and
 *          no less than the block's present exponent if the block holds earlier tokens of the sequence
 *     x -> e4m3(x / 2^e), to nearest even, +-448 beyond it (infinities too), NaN for NaN
 * Earlier tokens of the block are brought to e the same way (nothing happens to them if e has not grown).
 * After a rollback (spec_commit) a block keeps the exponent that it had.
 * Slots at or past kv_len[b] are left as they were, other blocks' exponents too.
 * A block that is written to must belong to its sequence alone (spec_page_fork sees to that).
 *
 * Layout: k_new, v_new [T, Hkv, D] (equal strides), src_dtype SPEC_BF16 or SPEC_F32; k_pages, v_pages with any
 *   strides for page, head and token, equal for both (kv_stride_*; multiples of 16, pointers 16-byte
 *   aligned); k_exp, v_exp with any strides for page and head, equal for both, a head's blocks contiguous.  K and V, pages, heads and tokens
 *   do not overlap each other.
 * Limits as spec_paged_attn; block >= 1 divides page_size.
 * Data errors as spec_paged_attn: bad sequences (SPEC_STATUS_BAD_RANGE, SPEC_STATUS_BAD_KV_LEN) and
 *   blocks of a page id out of range (SPEC_STATUS_BAD_PAGE) are not written.
 * ---------------------------------------------------------------------------------------- */
typedef struct spec_kv8_append_args {
  int32_t B, Hkv, D, T;
  int32_t src_dtype;
  int32_t page_size, num_pages, table_cols;
  int32_t block, reserved0;
  const void* k_new;
  const void* v_new;
  int64_t new_stride_t, new_stride_h;
  void* k_pages;
  void* v_pages;
  int64_t kv_stride_p, kv_stride_h, kv_stride_t;
  uint8_t* k_exp;
  uint8_t* v_exp;
  int64_t exp_stride_p, exp_stride_h;
  const int32_t* page_table;
  int64_t table_stride;
  const int32_t* q_start;
  const int32_t* kv_len;
  void* workspace;
  size_t workspace_bytes;
} spec_kv8_append_args;

size_t spec_kv8_append_workspace(const spec_kv8_append_args* args);
int spec_kv8_append(const spec_kv8_append_args* args, spec_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * spec_paged_attn8
 *
 * spec_paged_attn over a cache in 8 bits: the same rows, positions, window, limits and data errors, with
 * k and v the values that the cache stands for.
 *   k_new / v_new set (both or neither): the call first does what spec_kv8_append does, and the attention
 *   sees the new tokens as the cache holds them.
 * Types: q and k_new / v_new SPEC_BF16; o_dtype SPEC_F32 or SPEC_BF16.
 * Layout of the cache as spec_kv8_append; rows of o do not overlap each other.
 * Finiteness as there; besides, a row's largest |q| times scale is below 2^70 (else that row's o is unspecified).
 * Accumulation is fp32.  K, V and the queries enter the products in fp16, which holds e4m3 values and bf16
 *   queries without rounding: queries are scaled by a power of two, one for the rows of a sequence and kv head in
 *   chunks of up to 32 query rows (tokens x heads of the group), one for each row in larger ones, and only parts
 *   below 2^-29 of the largest lose bits.  Probabilities are rounded to fp16 as weights of V's scales, p 2^ev: those
 *   below 2^-32 of a row's largest lose bits.  Larger chunks bring V and K of 32 neighbouring keys to the largest of their
 *   blocks' scales where these lie within 2^15 of each other, which is exact (the largest then counts in p 2^ev); keys
 *   farther apart keep their own scales, which takes longer.
 * ---------------------------------------------------------------------------------------- */
typedef struct spec_paged8_args {
  int32_t B, Hq, Hkv, D, T, max_q;
  int32_t q_dtype, o_dtype;
  int32_t page_size, num_pages, table_cols;
  int32_t window, block;
  float scale;                /* 0: 1/sqrt(D) */
  const void* q;
  int64_t q_stride_t, q_stride_h;
  void* k_pages;              /* written only with k_new / v_new */
  void* v_pages;
  int64_t kv_stride_p, kv_stride_h, kv_stride_t;
  uint8_t* k_exp;             /* written only with k_new / v_new */
  uint8_t* v_exp;
  int64_t exp_stride_p, exp_stride_h;
  const int32_t* page_table;
  int64_t table_stride;
  const int32_t* q_start;
  const int32_t* kv_len;
  const void* k_new;
  const void* v_new;
  int64_t new_stride_t, new_stride_h;
  void* o;
  int64_t o_stride_t, o_stride_h;
  void* workspace;
  size_t workspace_bytes;
} spec_paged8_args;

size_t spec_paged_attn8_workspace(const spec_paged8_args* args);
int spec_paged_attn8(const spec_paged8_args* args, spec_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * spec_page_fork
 *
 * One step of a batch of sequences whose pages may be shared.  Row b holds the pages page_table[b, 0 ..
 * held[b] - 1]; refs[p] counts the holders of page p (every row that holds it, and whatever else the caller counts
 * there; a count above 0 that leaves out rows is not noticed); a page with refs[p] <= 0 is free.  After the
 * call row b goes on from what row parent[b] was:
 *     parent[b] == -1: the row is empty (no tokens, no pages); grow[b] does not matter
 *     else: it has the kv_len[parent[b]] tokens of that row and room for grow[b] more, kv_len_out[b] =
 *     kv_len[parent[b]] + grow[b] (what spec_paged_attn takes for a chunk of grow[b] new tokens), and holds
 *     exactly the pages that they need.
 * Pages of the earlier tokens are shared with the parent; one that the new tokens start in the middle of and
 * that anyone else holds is replaced by a copy, in all `arrays` (if every holder is a row that writes to it,
 * the lowest of them keeps it).  Pages no longer held lose a holder.  New pages are the lowest free ids, given
 * to the rows in order, a row's copy first, then its further pages.  Pages that lose their last holder in
 * this call are free in it.
 * All or nothing: with any data error (SPEC_STATUS_BAD_RANGE: a parent outside [-1, B);
 * SPEC_STATUS_BAD_KV_LEN: a length or held count below 0, more tokens than held pages, grow < 0, or more than
 * table_cols pages; SPEC_STATUS_BAD_PAGE: a held entry that is no page, or a page that refs says is free;
 * SPEC_STATUS_NO_PAGE: too few free pages) nothing is changed.
 *
 * Layout: page_table, table_out [B, table_cols] int32 with row strides; held, kv_len, parent, grow (NULL: 0)
 *   [B], refs [num_pages] int32; table_out, held_out, kv_len_out, refs_out: outputs, each the input itself or
 *   apart from all inputs.  Entries of table_out past held_out[b] are left as they were.
 *   arrays (host memory, read during the call): page p of an array is the page_bytes bytes at
 *   base + p * stride_bytes; pages of an array do not overlap.  Any alignment; copies are fastest where all
 *   three are multiples of 16.
 * Limits: 1 <= B <= 4096; 1 <= table_cols; B * table_cols <= 2^26; 1 <= num_pages <= 2^24;
 *   1 <= page_size <= 65536; table_cols * page_size <= 2^30; 0 <= num_arrays <= 4096.
 * ---------------------------------------------------------------------------------------- */
typedef struct spec_page_array {
  void* base;
  int64_t stride_bytes, page_bytes;
} spec_page_array;

typedef struct spec_page_fork_args {
  int32_t B, table_cols, page_size, num_pages, num_arrays, reserved0;
  const int32_t* page_table;
  int64_t table_stride;
  const int32_t* held;
  const int32_t* kv_len;
  const int32_t* refs;
  const int32_t* parent;
  const int32_t* grow;
  int32_t* table_out;
  int64_t table_out_stride;
  int32_t* held_out;
  int32_t* kv_len_out;
  int32_t* refs_out;
  const spec_page_array* arrays;
  void* workspace;
  size_t workspace_bytes;
} spec_page_fork_args;

size_t spec_page_fork_workspace(const spec_page_fork_args* args);
int spec_page_fork(const spec_page_fork_args* args, spec_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * spec_page_compact
 *
 * With L pages in use (refs[p] > 0), those at or past L move, in ascending order, into the free ones below
 * L, in ascending order, in all `arrays`; the tables' held entries and refs follow.  moved[p] (optional): the
 * new id of page p, -1 for a free page; num_live (optional): L.
 * Pages at or past L then hold what they held, and may be given back.
 * All or nothing: a held count outside [0, table_cols] (SPEC_STATUS_BAD_KV_LEN) or a held entry that is no page
 * in use (SPEC_STATUS_BAD_PAGE) changes nothing.
 * Layout and limits as spec_page_fork.
 * ---------------------------------------------------------------------------------------- */
typedef struct spec_page_compact_args {
  int32_t B, table_cols, num_pages, num_arrays;
  const int32_t* page_table;
  int64_t table_stride;
  const int32_t* held;
  const int32_t* refs;
  int32_t* table_out;
  int64_t table_out_stride;
  int32_t* refs_out;
  int32_t* moved;
  int32_t* num_live;
  const spec_page_array* arrays;
  void* workspace;
  size_t workspace_bytes;
} spec_page_compact_args;

size_t spec_page_compact_workspace(const spec_page_compact_args* args);
int spec_page_compact(const spec_page_compact_args* args, spec_stream_t stream);

/* sizeof() of this header's structs as compiled: which = 0 spec_rotary_args, 1 spec_kv8_append_args,
 * 2 spec_paged8_args, 3 spec_page_fork_args, 4 spec_page_compact_args, 5 spec_page_array; else 0. */
size_t spec_cache_struct_size(int which);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_CACHE_H_ */
