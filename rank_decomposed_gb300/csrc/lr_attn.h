// Shared by the attention kernels: device parameters and the layout of the
// partial results.
#pragma once

#include "lr_internal.h"

namespace lr {

struct AttnParams {
  const uint16_t* q;
  int64_t ldq;
  const uint16_t* k;
  const uint16_t* v;
  int64_t ld;                 // row stride of both pools, elements
  int64_t pool_blocks;
  int32_t block_rows;
  int32_t block_shift;        // log2(block_rows), or -1
  int32_t n_heads, n_kv, group;
  float scale_log2;           // scale * log2(e): scores are kept in powers of two
  const int32_t* prefix_blocks;
  const int32_t* prefix_len;
  int32_t cap_prefix;         // rows
  int32_t M, n_seq, max_q;
  const int32_t* q_start;
  const int32_t* block_table;
  int32_t blocks_per_seq;
  const int32_t* lengths;
  int32_t cap_own;            // rows
  // Partial results.  Slot i of row r = m * n_heads + head: numerators
  // po[(i * M * n_heads + r) * head_dim ..], and pml[i * M * n_heads + r] =
  // (running maximum, sum), sum = 0 where the slot saw no key, -0 where the keys
  // that the row sees all scored minus infinity.  The prefix's slots come first.
  float* po;
  float2* pml;
  int32_t prefix_slots, own_slots;
  void* out;
  int64_t ldo;
  int32_t out_f32;
  int32_t* status;
};

// What a tensor-core launch takes, prefix and own tokens: each sequence's rows
// by themselves (whole) or the rows of the batch packed into tiles; cut along
// the keys into `slots` ranges.
struct AttnPart {
  bool whole;
  int32_t slots;
  bool two;  // each range has two slots of results
};

// Query rows of a tensor-core tile: their heads of one key head fill its 128
// rows as far as whole rows do.
inline int attn_tile_rows(int group) { return 128 / group; }

lr_status launch_attn_rows(const AttnParams& p, int head_dim, cudaStream_t s);
lr_status launch_attn_tiles(const AttnParams& p, int head_dim, const AttnPart& part, cudaStream_t s);
lr_status configure_attn_tiles();
// Tensor map over query rows [M][ld]: element (c, h, m) is column h * head_dim
// + c of row m; a box takes 64 columns of box_heads heads of box_rows rows.
lr_status encode_map_heads(CUtensorMap* map, const void* base, uint64_t head_dim, uint64_t heads, uint64_t rows,
                           uint64_t ld, uint32_t box_heads, uint32_t box_rows);
lr_status launch_attn_join(const AttnParams& p, int head_dim, cudaStream_t s);
lr_status configure_attn();
// The host-side argument checks of the entry points.
lr_status check_kv_cache(const char* who, const lr_kv_cache* c);
lr_status check_append(const void* k, int64_t ldk, const void* v, int64_t ldv, const void* q, int64_t ldq,
                       int32_t n_heads, lr_dtype in_dtype, int64_t M, const int32_t* pos, const int32_t* rows,
                       const lr_head_map* hm, const lr_kv_cache* cache, const void* q_out, int64_t ldqo);
lr_status check_attention(const void* q, int64_t ldq, const void* out, int64_t ldo, lr_dtype out_dtype, int64_t M,
                          const lr_attn_desc* d, const void* workspace, size_t ws_bytes);

#ifdef __CUDACC__
// A sequence's query rows and own length, clamped to what the capacities allow.
// Row j sees the own tokens up to len - n + j: of n rows that are more than
// max_q, the first nq = max_q still see what they would.
struct SeqView {
  int32_t q0, nq, n, len;
};
__device__ __forceinline__ SeqView seq_view(const AttnParams& p, int b, bool tell) {
  SeqView s;
  bool bad = false;
  if (p.q_start != nullptr) {
    const int a = p.q_start[b], e = p.q_start[b + 1];
    s.q0 = a < 0 ? 0 : (a > p.M ? p.M : a);
    const int end = e < 0 ? 0 : (e > p.M ? p.M : e);
    s.nq = end > s.q0 ? end - s.q0 : 0;
    bad = a < 0 || e > p.M || e < a || s.nq > p.max_q;
    s.n = s.nq;
    if (s.nq > p.max_q) s.nq = p.max_q;
  } else {
    s.q0 = b;
    s.n = s.nq = b < p.M ? 1 : 0;
  }
  const int len = p.lengths[b];
  s.len = len < 0 ? 0 : (len > p.cap_own ? p.cap_own : len);
  if (tell && (bad || (s.len != len && s.nq > 0))) {  // a place without rows may hold any length
    int32_t* st = p.status;
    if (st != nullptr) atomicCAS(st, 0, LR_ERR_INDEX_RANGE);
  }
  return s;
}
__device__ __forceinline__ int prefix_rows(const AttnParams& p, int len, bool tell) {
  const int n = len < 0 ? 0 : (len > p.cap_prefix ? p.cap_prefix : len);
  if (tell && n != len && p.status != nullptr) atomicCAS(p.status, 0, LR_ERR_INDEX_RANGE);
  return n;
}
__device__ __forceinline__ int prefix_view(const AttnParams& p, bool tell) {
  return p.cap_prefix > 0 ? prefix_rows(p, *p.prefix_len, tell) : 0;
}
#endif

}  // namespace lr
