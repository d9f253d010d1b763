// Internal launchers of the attention side (norm and rotation, append, paged attention), called by
// the C ABI layer after host validation.  Each returns the hipError_t of its launch(es).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ql {

// Unsigned division of dividends below 2^31 by a fixed divisor, by multiplication (Granlund and
// Montgomery 1994): n / d = (mulhi(n, mul) + n) >> sh with
// sh = ceil(log2 d) and mul = floor(2^32 (2^sh - d) / d) + 1.
struct FastDiv {
  uint32_t mul, sh;
#ifdef __HIPCC__
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, mul) + n) >> sh; }
#endif
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f{0, 0};
  while (f.sh < 31 && (1u << f.sh) < d) ++f.sh;
  f.mul = (uint32_t)(((((uint64_t)1 << f.sh) - d) << 32) / d + 1);
  return f;
}

// Per-head norm and rotation of q and k rows, and the append to a paged cache (norm_rope.hip).
// Strides in bytes; a NULL source is absent (0 heads).
struct NormRopeArgs {
  const uint8_t *q, *k, *v;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;
  uint8_t *q_out, *k_out, *v_out;  // k_out and v_out: tensors, or the cache's pages
  int64_t qo_ts, qo_hs, ko_ts, ko_hs, vo_ts, vo_hs;
  int64_t page_stride;     // append: pages of k_out and v_out
  const int64_t* slots;    // append: cache slot of each token, or NULL
  int64_t n_slots;
  int page_size;
  FastDiv page_div;
  int hq, hk, hv;  // heads of q, k and v
  int64_t t;
  int d, rot, interleaved;
  const void *q_weight, *k_weight;  // [d] or NULL
  int wdt;
  float eps;
  const int64_t* positions;
  const float* cos_sin;  // [max_pos, rot]: cosines, then sines
  int64_t max_pos;
};
hipError_t launch_norm_rope(const NormRopeArgs& a, int dt, hipStream_t s);
// The append to a cache in 4 bits: k_out and v_out are the codes, with the strides of k_out.  hk and hv are 0 (what
// the norm and rotation of q goes by); the rows of k and v are cache_heads each.
struct Append4Args : NormRopeArgs {
  int cache_heads;
  uint32_t *k_groups, *v_groups;
  int64_t group_ps, group_ts, group_hs;  // words
  int group;
  double inv_d;  // 1 / d
};
hipError_t launch_append4(const Append4Args& a, int dt, hipStream_t s);
// The values of its rows.
struct Read4Args {
  const uint8_t *k, *v;
  int64_t page_stride, token_stride, head_stride;  // bytes
  const uint32_t *kg, *vg;
  int64_t group_ps, group_ts, group_hs;  // words
  uint8_t *k_out, *v_out;
  int64_t ko_ts, ko_hs, vo_ts, vo_hs;  // bytes
  const int64_t* slots;
  int64_t n_slots;
  int page_size;
  FastDiv page_div;
  int hk, d, group;
  int64_t t;
};
hipError_t launch_read4(const Read4Args& a, int dt, hipStream_t s);

// The tables of a batch (kv_extend.hip).
struct ExtendArgs {
  const int32_t *counts, *lens;
  int n_seqs;
  int32_t* table;
  int64_t table_stride, max_pages;
  int page_size;
  FastDiv page_div;
  int32_t* free_pages;  // NULL: no list
  int64_t free_cap;
  const int32_t* free_count;
  int32_t *lens_out, *free_count_out, *cu_q;
  int64_t *positions, *slots;
  int64_t rows;
  int32_t* info;
};
hipError_t launch_kv_extend(const ExtendArgs& a, hipStream_t s);

// Paged attention (attn_few.hip: sequences of few rows; attn_tile.hip: the others and the joining of
// split items).  Strides in bytes.
constexpr int kAttnTileKeys = 64;  // keys of the tile kernel's unit of work
// Waves of its workgroups, 32 query rows each (256 values a head fill a SIMD's registers).
constexpr int attn_tile_waves(int d) { return d == 256 ? 4 : 8; }
constexpr int kAttnFewKeys = 128;   // keys of the few-row kernel's unit
constexpr int kAttnFewKeys4 = 256;  // the same over a cache in 4 bits
struct AttnRecord;
struct AttnArgs {
  const uint8_t* q;
  int64_t q_ts, q_hs;
  const uint8_t *k, *v;
  int64_t page_stride, token_stride, head_stride;
  int n_pages, page_size;
  int page16;  // pages are multiples of 16 slots, and 16 rows of one lie within 2^31 bytes
  FastDiv page_div;
  const int32_t* table;
  int64_t table_stride;  // entries
  int max_kv;            // tokens of a block-table row
  const int32_t *cu_q, *kv_lens;
  int n_seqs;
  int64_t t;
  int max_q;
  int hk, g;  // kv heads, query heads of each
  FastDiv g_div;
  float sl;  // scale * log2(e)
  int window;
  const float* sinks;
  uint8_t* out;
  int64_t out_ts, out_hs;
  // the plan
  int few_rows;  // sequences of at most this many rows go to the few-row kernel
  int nw_few, cap_few, part_floats, join_few;
  int nw_tile, items_tile, plan_tiles, join_tile;
  int few_by_item, tile_by_item;  // records by item, else by workgroup
  AttnRecord* rec;
  float *part, *part_tile;
};
// The same over a cache in 4 bits: k and v are the codes (strides of AttnArgs), kp and vp a word of scale
// and bias (fp16) per group.
struct AttnArgs4 : AttnArgs {
  const uint8_t *kp, *vp;
  int64_t p_page_stride, p_token_stride, p_head_stride;  // bytes
  int group_log2;
  int io;  // dtype of q and out
};
// How a call is run, from what the host knows (the lengths are device values).
struct AttnPlan {
  bool ok;        // the work is within the kernels' 32-bit unit counts
  int nc;         // 16-row column tiles of the few-row kernel, 0: not launched
  bool tile;      // whether the tile kernel is launched
  int few_rows, nw_few, cap_few, part_floats, join_few;
  int nw_tile, items_tile, plan_tiles, join_tile;
  size_t part_off, part_tile_off, bytes;  // workspace: records, pieces of either kernel
};
AttnPlan attn_plan(int64_t t, int64_t n_seqs, int64_t hq, int64_t hk, int d, int64_t max_q, int64_t max_kv,
                   int64_t window, int few_keys);
// Sets the kind of records.
void attn_record_kind(AttnArgs& a);
hipError_t launch_attn_few(const AttnArgs& a, int dt, int d, int nc, hipStream_t s);
hipError_t launch_attn_tile(const AttnArgs& a, int dt, int d, hipStream_t s);
hipError_t launch_attn_few4(const AttnArgs4& a, int d, int nc, hipStream_t s);
hipError_t launch_attn_tile4(const AttnArgs4& a, int d, hipStream_t s);
hipError_t launch_attn_join(const AttnArgs& a, int dt, int d, hipStream_t s);

}  // namespace ql
