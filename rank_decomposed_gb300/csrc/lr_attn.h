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
  // A cache in 8 bits: k and v point to codes, ld counts them.
  const float* k_scale;
  const float* v_scale;
  int32_t window, sinks;      // window 0: none
  int32_t direct;             // by rows: one range and one part, results go straight to out
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

// A launch by rows over a cache in 8 bits.
struct Rows8Launch {
  int32_t tile;      // rows of a CTA: 8, 16 or 32
  int32_t least;     // chunks of 16 keys of a range, at least
  int32_t tiles[2];  // row tiles of the prefix part; row tiles per sequence of the other (set by the launch)
  int32_t ctas0;     // CTAs of the prefix part (set by the launch)
};
lr_status launch_attn_rows8(const AttnParams& p, int head_dim, Rows8Launch rl, cudaStream_t s);
lr_status configure_attn8();
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
                       const lr_head_map* hm, const lr_kv_cache* cache, const void* q_out, int64_t ldqo,
                       const char* who = "kv_append");
// Of a cache in 8 bits, beyond check_kv_cache.
lr_status check_scales(const char* who, const lr_kv_cache* c, const float* k_scale, const float* v_scale);
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
// (a length that is given without pages has the capacity 0)
__device__ __forceinline__ int prefix_view(const AttnParams& p, bool tell) {
  if (p.cap_prefix > 0) return prefix_rows(p, *p.prefix_len, tell);
  if (tell && p.prefix_len != nullptr) prefix_rows(p, *p.prefix_len, true);
  return 0;
}

// Rows of no sequence come out zero: CTA `item` of `items` takes every items-th row of q.
__device__ __forceinline__ void zero_rows(const AttnParams& p, int item, int items, int head_dim, int threads) {
  const int from = p.q_start ? p.q_start[0] : 0, to = p.q_start ? p.q_start[p.n_seq] : p.n_seq;
  const int size = p.out_f32 ? 4 : 2, vecs = p.n_heads * head_dim * size / 16;
  for (int64_t m = item; m < p.M; m += items)
    if (m < from || m >= to) {
      uint4* row = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + m * p.ldo * size);
      for (int i = threadIdx.x; i < vecs; i += threads) row[i] = make_uint4(0, 0, 0, 0);
    }
}

// The chunks of 16 keys that the rows of a CTA walk with a window: the prefix's, then
// the own ones, less those between the sinks and the first row's window.
struct WindowList {
  int32_t np;             // chunks of the prefix
  int32_t skip, skipped;  // from chunk `skip` on so many are left out
  int32_t chunks;         // that are left
  int32_t lo_min;         // lowest position in the window of the first row
  // Chunk c of the list: its number in its part.
  __device__ __forceinline__ int place(int c, bool& shared) const {
    if (c >= skip) c += skipped;
    shared = c < np;
    return shared ? c : c - np;
  }
};
// first: the first row's own place, kmax: the own tokens that the last row sees.
__device__ __forceinline__ WindowList window_list(int P, int first, int kmax, int window, int sinks) {
  WindowList w;
  w.np = (P + 15) / 16;
  w.chunks = w.np + (kmax + 15) / 16;
  w.lo_min = P + first - window + 1;
  auto chunk_of = [&](int t) { return t < P ? t / 16 : w.np + (t - P) / 16; };
  w.skip = sinks <= 0 ? 0 : (sinks - 1 < P + kmax ? chunk_of(sinks - 1) + 1 : w.chunks);
  if (w.skip > w.chunks) w.skip = w.chunks;
  const int to = w.lo_min > 0 ? chunk_of(w.lo_min) : 0;
  w.skipped = to > w.skip ? to - w.skip : 0;
  if (w.skipped > w.chunks - w.skip) w.skipped = w.chunks - w.skip;
  w.chunks -= w.skipped;
  return w;
}
#endif

}  // namespace lr
