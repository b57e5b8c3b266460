// Attention of a batch that shares a prefix: entry point, the choice of kernel
// and of key ranges, the kernel for few query rows, and the join of partial
// results.
//
// For a query row with visible keys t in parts i (the shared prefix and the
// sequence's own tokens, each cut along the keys):
//   m_i = max_t s_t,  l_i = sum_t 2^(s_t - m_i),  o_i = sum_t 2^(s_t - m_i) v_t,
//   out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,   M = max_i m_i,
// with s_t = scale log2(e) q . k_t.  The prefix is read for all rows of the
// batch at once, whichever sequences they belong to: M * group rows a key head
// share each key, where a sequence's own keys serve only its own rows.
#include <cuda_bf16.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "lr_attn.h"
#include "lr_ptx.cuh"

namespace lr {
namespace {

// ------------------------------------------------------- rows kernel
// Few query rows against many keys: bound by the bytes of K and V.  A CTA takes
// 16 rows (query rows times the heads of one key head) and a range of keys;
// each of its four warps walks chunks of 16 keys (they never cross a page) on
// its own: a ring of chunks filled by 16-byte asynchronous copies, S = Q K^T
// and O += P V by m16n8k16 products with Q and O in registers, and its own
// running maximum and sum, so no warp waits for another until the end, where
// the four join through shared memory.  With 16 rows a tile the products are far
// from any bound (16 rows use 1/8 of a tcgen05 tile's lanes, hence mma.sync from
// registers, which needs no TMEM and no second pipeline to start).
// Measured with the join, caches cold: one row of 64 heads over 8 behind 16000,
// 60000, 128000 tokens 26, 52, 95 us (2.5, 4.7, 5.5 TB/s); of 32 over 32 behind 60000
// 160 us (6.1 TB/s); three short sequences 12 us, 10 with warm caches, all of it latency.
constexpr int kRowsWarps = 4;
constexpr int kRowsTile = 16;
constexpr int kRowsChunk = 16;
constexpr int kRowsStages = 3;

template <int HD>
constexpr int rows_smem() {
  return kRowsWarps * kRowsStages * kRowsChunk * HD * 2 * 2;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
  const int n = live ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return static_cast<uint32_t>(f32_to_bf16_rn(lo)) | (static_cast<uint32_t>(f32_to_bf16_rn(hi)) << 16);
}

// Byte offset of 16-byte column c of row r in a [16][HD] tile: columns are
// permuted by the row, so that the eight rows of a matrix load lie in
// different banks.
template <int HD>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return static_cast<uint32_t>(r * HD * 2 + ((c ^ (r & 7)) << 4));
}

// One launch takes both parts: the prefix for all rows and the own tokens.
struct RowsLaunch {
  int32_t tiles[2];   // row tiles of the prefix part; row tiles per sequence of the other
  int32_t ctas0;      // CTAs of the prefix part
};

template <int HD>
__device__ __forceinline__ void attn_rows_cta(const AttnParams& p, const RowsLaunch& rl) {
  constexpr int kC16 = HD / 8;  // 16-byte columns of a row
  extern __shared__ __align__(128) uint8_t sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.group;
  // CTA -> part, row tile, key head, key range
  const int which = static_cast<int>(blockIdx.x) < rl.ctas0 ? 0 : 1;
  const bool prefix = which == 0;
  const int slots = prefix ? p.prefix_slots : p.own_slots;
  int idx = static_cast<int>(blockIdx.x) - (which ? rl.ctas0 : 0);
  const int split = idx % slots;
  idx /= slots;
  const int kvh = idx % p.n_kv;
  const int tile = idx / p.n_kv;
  const int tiles = which ? rl.tiles[1] : rl.tiles[0];

  // This CTA's rows: r = (query row - q0) * G + head in the group.
  int q0, n_rows, row0, len, nq, n;
  const int32_t* pages;
  const bool tell = kvh == 0 && threadIdx.x == 0 && split == 0;
  if (prefix) {
    q0 = 0;
    n = nq = p.M;
    len = prefix_view(p, tell);
    pages = p.prefix_blocks;
    row0 = tile * kRowsTile;
  } else {
    const int b = tile / tiles;
    const SeqView v = seq_view(p, b, tell);
    q0 = v.q0;
    nq = v.nq;
    n = v.n;
    len = v.len;
    pages = p.block_table + static_cast<int64_t>(b) * p.blocks_per_seq;
    row0 = (tile % tiles) * kRowsTile;
  }
  n_rows = nq * G - row0;
  if (n_rows <= 0) return;
  if (n_rows > kRowsTile) n_rows = kRowsTile;

  // Visible keys: all of the prefix; own tokens up to a row's own.
  const int r_lo = lane >> 2;  // this lane's two rows in the tile: r_lo, r_lo + 8
  int vis[2];
  int kmax = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = row0 + r_lo + 8 * i;
    vis[i] = prefix ? len : len - n + r / G + 1;
  }
  kmax = prefix ? len : len - n + (row0 + n_rows - 1) / G + 1;
  if (kmax < 0) kmax = 0;
  const int all_chunks = (kmax + kRowsChunk - 1) / kRowsChunk;
  const int per = (all_chunks + slots - 1) / slots;
  const int c_lo = split * per;
  const int c_hi = c_lo + per < all_chunks ? c_lo + per : all_chunks;

  // Q in the A layout of m16n8k16.
  uint32_t qa[HD / 16][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int rr = r_lo + 8 * i;
    const int r = row0 + rr;
    const bool live = rr < n_rows;
    const uint16_t* src = p.q + static_cast<int64_t>(q0 + r / G) * p.ldq + static_cast<int64_t>(kvh * G + r % G) * HD;
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk) {
      const int col = kk * 16 + (lane & 3) * 2;
      qa[kk][i] = live ? *reinterpret_cast<const uint32_t*>(src + col) : 0u;
      qa[kk][i + 2] = live ? *reinterpret_cast<const uint32_t*>(src + col + 8) : 0u;
    }
  }

  float o[HD / 8][4];
#pragma unroll
  for (int n = 0; n < HD / 8; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[n][j] = 0.f;
  float mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};

  // Ring of this warp: stage s holds K [16][HD] then V [16][HD].
  constexpr uint32_t kTile = kRowsChunk * HD * 2;
  const uint32_t ring = smem_u32(sm) + warp * kRowsStages * 2 * kTile;
  const int mine = c_hi - c_lo > warp ? (c_hi - c_lo - warp + kRowsWarps - 1) / kRowsWarps : 0;
  int ids = 0;  // lane i: page of this warp's chunk i of the current 32
  auto page_of = [&](int i) {
    if ((i & 31) == 0) {
      const int c = c_lo + warp + (i + lane) * kRowsWarps;
      const int t = c * kRowsChunk;
      ids = i + lane < mine ? pages[p.block_shift >= 0 ? t >> p.block_shift : t / p.block_rows] : -1;
      if (i + lane < mine && (ids < 0 || ids >= p.pool_blocks)) {
        report_status(p.status, LR_ERR_REMAP_RANGE);
        ids = -1;
      }
    }
    return __shfl_sync(0xffffffffu, ids, i & 31);
  };
  // an instruction copies kRows rows
  constexpr int kRows = 32 / kC16;
  const int r_in = lane / kC16, col = lane % kC16;
  const int64_t head_off = static_cast<int64_t>(kvh) * HD + col * 8;
  const int64_t step = kRows * p.ld;
  auto issue = [&](int i) {
    if (i < mine) {
      const int page = page_of(i);
      const int t0 = (c_lo + warp + i * kRowsWarps) * kRowsChunk;
      const int in_page = t0 - (p.block_shift >= 0 ? t0 >> p.block_shift << p.block_shift : t0 / p.block_rows * p.block_rows);
      const int live = page < 0 ? 0 : kmax - t0;  // rows of the chunk that hold visible tokens
      const int64_t off = page < 0 ? 0 : (static_cast<int64_t>(page) * p.block_rows + in_page + r_in) * p.ld + head_off;
      const uint16_t* kp = p.k + off;
      const uint16_t* vp = p.v + off;
      const uint32_t st = ring + (i % kRowsStages) * 2 * kTile;
#pragma unroll
      for (int j = 0; j < kRowsChunk / kRows; ++j, kp += step, vp += step) {
        const int r = j * kRows + r_in;
        const bool in = r < live;
        cp16(st + swz<HD>(r, col), in ? kp : p.k, in);
        cp16(st + kTile + swz<HD>(r, col), in ? vp : p.v, in);
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kRowsStages - 1; ++i) issue(i);

  for (int i = 0; i < mine; ++i) {
    issue(i + kRowsStages - 1);
    cp_wait<kRowsStages - 1>();
    __syncwarp();
    const uint32_t st = ring + (i % kRowsStages) * 2 * kTile;
    const int t0 = (c_lo + warp + i * kRowsWarps) * kRowsChunk;
    float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    {
      const int r = (lane & 7) + ((lane & 16) >> 1), cc = (lane >> 3) & 1;
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk) {
        uint32_t b0, b1, b2, b3;  // keys 0-7: k 0-7, 8-15; keys 8-15: the same
        ldsm4(st + swz<HD>(r, kk * 2 + cc), b0, b1, b2, b3);
        mma16816(s[0], qa[kk], b0, b1);
        mma16816(s[1], qa[kk], b2, b3);
      }
    }
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = t0 + n * 8 + (lane & 3) * 2 + (j & 1);
        s[n][j] = t < vis[j >> 1] ? s[n][j] * p.scale_log2 : -INFINITY;
        top[j >> 1] = fmaxf(top[j >> 1], s[n][j]);
      }
    float ref[2], fac[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], 1));
      top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], 2));
      const float now = fmaxf(mx[k], top[k]);
      ref[k] = now == -INFINITY ? 0.f : now;  // nothing visible yet: every power is 2^-inf = 0
      fac[k] = exp2f(mx[k] - ref[k]);
      mx[k] = now;
    }
    if (__any_sync(0xffffffffu, fac[0] != 1.f || fac[1] != 1.f)) {
#pragma unroll
      for (int n = 0; n < HD / 8; ++n) {
        o[n][0] *= fac[0], o[n][1] *= fac[0];
        o[n][2] *= fac[1], o[n][3] *= fac[1];
      }
      sum[0] *= fac[0], sum[1] *= fac[1];
    }
    uint32_t pa[4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[n][j] = exp2f(s[n][j] - ref[j >> 1]);
        sum[j >> 1] += s[n][j];
      }
      // the accumulators' layout is that of the next product's A operand; the
      // product takes bf16, so the probabilities round here (the sum does not)
      pa[n * 2] = pack_bf16(s[n][0], s[n][1]);
      pa[n * 2 + 1] = pack_bf16(s[n][2], s[n][3]);
    }
    {
      const int r = lane & 15, cc = lane >> 4;
#pragma unroll
      for (int n = 0; n < HD / 16; ++n) {
        uint32_t b0, b1, b2, b3;  // columns 0-7: keys 0-7, 8-15; columns 8-15: the same
        ldsm4t(st + kTile + swz<HD>(r, n * 2 + cc), b0, b1, b2, b3);
        mma16816(o[2 * n], pa, b0, b1);
        mma16816(o[2 * n + 1], pa, b2, b3);
      }
    }
    __syncwarp();
  }
  cp_wait<0>();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 1);
    sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 2);
  }

  // Join the four warps: numerators in the ring's space, [warp][16][HD].
  __shared__ float2 ml[kRowsWarps][kRowsTile];
  __syncthreads();
  float* jo = reinterpret_cast<float*>(sm) + warp * kRowsTile * HD;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r_lo + 8 * i;
    if ((lane & 3) == 0) ml[warp][r] = make_float2(mx[i], sum[i]);
#pragma unroll
    for (int n = 0; n < HD / 8; ++n)
      *reinterpret_cast<float2*>(jo + r * HD + n * 8 + (lane & 3) * 2) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
  }
  __syncthreads();
  const int64_t slot_rows = static_cast<int64_t>(p.M) * p.n_heads;
  const int64_t base = ((prefix ? 0 : p.prefix_slots) + split) * slot_rows;
  for (int idx = threadIdx.x; idx < n_rows * (HD / 4); idx += kRowsWarps * 32) {
    const int rr = idx / (HD / 4), c = idx % (HD / 4);
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kRowsWarps; ++w) m = fmaxf(m, ml[w][rr].x);
    const float ref = m == -INFINITY ? 0.f : m;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll
    for (int w = 0; w < kRowsWarps; ++w) {
      const float f = exp2f(ml[w][rr].x - ref);
      const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(sm) + (w * kRowsTile + rr) * HD + c * 4);
      l += f * ml[w][rr].y;
      acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
    }
    const int r = row0 + rr;
    const int64_t at = base + static_cast<int64_t>(q0 + r / G) * p.n_heads + kvh * G + r % G;
    *reinterpret_cast<float4*>(p.po + at * HD + c * 4) = acc;
    if (c == 0) {
      const int sees = prefix ? len : len - n + r / G + 1;
      p.pml[at] = make_float2(m, l == 0.f && sees > c_lo * kRowsChunk ? -0.f : l);
    }
  }
}

template <int HD>
__global__ void __launch_bounds__(kRowsWarps * 32)
    attn_rows_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ RowsLaunch rl) {
  pdl_launch_dependents();
  pdl_wait();
  attn_rows_cta<HD>(p, rl);
}

// --------------------------------------------------------------- join
// W warps per (row, head), each with every W-th slot's numerators and all
// slots' weights.  Bound by the way to the partial results, which were written
// just before and lie in L2.  One warp has the loads of four slots in flight
// together, which is enough for few slots; from 16 slots on four warps share them.
// Whole calls with one warp and with four: 5 sequences behind 131000 tokens (38
// slots) 107, 97 us; 4 behind 16000 (38 slots) 44, 33; 200 behind 1000 (2 slots)
// 59, 68; 100 of 56 heads behind 300 (2 slots) 40, 44.
constexpr int kMaxSlots = 64;  // of each part

template <int HD, int W>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kE = HD / 32;  // elements per lane
  constexpr int kRows = 8 / W;
  __shared__ float parts[W > 1 ? 8 : 1][HD];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t rows = static_cast<int64_t>(p.M) * p.n_heads;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kRows + warp / W;
  const int m = static_cast<int>(r / p.n_heads), h = static_cast<int>(r - static_cast<int64_t>(m) * p.n_heads);
  int from = 0, to = p.n_seq;
  if (p.q_start != nullptr) {
    from = p.q_start[0];
    to = p.n_seq > 0 ? p.q_start[p.n_seq] : from;
  }
  // A part without pages has no CTA of the rows kernel: what it holds is looked at here.
  if (blockIdx.x == 0 && (p.cap_own == 0 || p.cap_prefix == 0)) {
    for (int b = threadIdx.x; p.cap_own == 0 && b < p.n_seq; b += 256) seq_view(p, b, true);
    if (p.cap_prefix == 0 && p.prefix_len != nullptr && threadIdx.x == 0) prefix_rows(p, *p.prefix_len, true);
  }
  float acc[kE], inv = 0.f;
#pragma unroll
  for (int j = 0; j < kE; ++j) acc[j] = 0.f;
  if (r < rows && m >= from && m < to) {
    const int slots = p.prefix_slots + p.own_slots;
    float top = -INFINITY;
    for (int i = lane; i < slots; i += 32) top = fmaxf(top, p.pml[i * rows + r].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float ref = top == -INFINITY ? 0.f : top;
    float l = 0.f;
    for (int i0 = 0; i0 < slots; i0 += 32) {
      // lane i holds the weight of slot i0 + i
      const float2 ml = i0 + lane < slots ? p.pml[(i0 + lane) * rows + r] : make_float2(-INFINITY, 0.f);
      const float w = ml.y == 0.f ? 0.f : exp2f(ml.x - ref);  // 0: nothing was stored
      l += w * ml.y;
      const int here = slots - i0 < 32 ? slots - i0 : 32;
#pragma unroll 4
      for (int i = warp % W; i < here; i += W) {
        // no branch on the weight, so that several slots' loads are in flight
        const float f = __shfl_sync(0xffffffffu, w, i);
        const float* src = p.po + ((i0 + i) * rows + r) * HD + lane * kE;
        if (kE == 4) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          if (f != 0.f) x = *reinterpret_cast<const float4*>(src);
          acc[0] += f * x.x, acc[1] += f * x.y, acc[kE - 2] += f * x.z, acc[kE - 1] += f * x.w;
        } else {
          float2 x = make_float2(0.f, 0.f);
          if (f != 0.f) x = *reinterpret_cast<const float2*>(src);
          acc[0] += f * x.x, acc[1] += f * x.y;
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (l != 0.f) {
      inv = 1.f / l;
    } else {  // no visible key: zeros; only keys of score minus infinity: 0 / 0
      bool none = false;
      for (int i = lane; i < slots; i += 32) none |= signbit(p.pml[i * rows + r].y);
      inv = __any_sync(0xffffffffu, none) ? NAN : 0.f;
    }
  }
  if (W > 1) {
#pragma unroll
    for (int j = 0; j < kE; ++j) parts[warp][lane * kE + j] = acc[j];
    __syncthreads();
    if (warp % W) return;
#pragma unroll
    for (int j = 0; j < kE; ++j)
#pragma unroll
      for (int k = 1; k < W; ++k) acc[j] += parts[warp + k][lane * kE + j];
  }
  if (r >= rows) return;
#pragma unroll
  for (int j = 0; j < kE; ++j) acc[j] *= inv;
  const int64_t off = static_cast<int64_t>(m) * p.ldo + static_cast<int64_t>(h) * HD + lane * kE;
  if (p.out_f32) {
    float* dst = static_cast<float*>(p.out) + off;
#pragma unroll
    for (int j = 0; j < kE; j += 2) *reinterpret_cast<float2*>(dst + j) = make_float2(acc[j], acc[j + 1]);
  } else {
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + off);
#pragma unroll
    for (int j = 0; j < kE; j += 2) dst[j / 2] = pack_bf16(acc[j], acc[j + 1]);
  }
}

template <typename... KArgs, typename... Args>
lr_status launch(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, const char* what,
                 Args... args) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  if (pdl_enabled()) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e != cudaSuccess) return cuda_fail(e, what);
  return LR_OK;
}

lr_status bad(lr_status st, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  set_error("%s", msg);
  return st;
}

int cdiv(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }
int64_t larger(int64_t a, int64_t b) { return a > b ? a : b; }
int64_t smaller(int64_t a, int64_t b) { return a < b ? a : b; }

// No sequence has more rows than the call.
int64_t most_q(int64_t M, const lr_attn_desc* d) { return d->max_q < M ? d->max_q : (M < 1 ? 1 : M); }

// Key ranges for `ctas` row tiles: as many as fill `want` CTAs, none shorter
// than min_keys.
int slots_for(int64_t ctas, int64_t keys, int64_t want, int64_t min_keys) {
  if (keys <= 0) return 0;
  int64_t n = ctas >= want || ctas < 1 ? 1 : want / ctas;
  const int64_t most = cdiv(keys, min_keys);
  if (n > most) n = most;
  if (n > kMaxSlots) n = kMaxSlots;
  return static_cast<int>(n);
}

// How a call is cut, from its capacities alone (lengths are on the device).
struct AttnPlan {
  bool tiles;         // on the tensor-core tiles; else by rows
  bool whole;         // tiles: each sequence's rows by themselves
  int32_t tile_slots;
  bool two;
  int32_t prefix_slots, own_slots;  // slots of partial results (0, 0: none, results go straight to out)
  size_t ml_off, bytes;
};

// Key ranges of the tensor-core tiles are no shorter than this.  256 sequences
// with heads of 64 behind 1500 tokens: 27, 26, 25, 29, 38 us with 1, 2, 4, 8, 16;
// long contexts fill the GPU with longer ranges and do not depend on it.
constexpr int kMinSteps = 4;
constexpr int kMostHeads = 64;  // query heads a key head: a tile has two query rows at least

// Rows or tiles.  A call on the tiles starts 8 to 10 us later (its CTAs take a
// whole SM each, set up TMEM and a pipeline of five roles, and end through
// TMEM), and after that it is the faster one wherever a tile's 128 rows are used.
// The rows kernel takes 3.7 us for each wave of CTAs (two an SM with heads of 128,
// four with 64) and reads the keys once for every 16 rows, 512 bytes for a key of
// 128 elements, from L2 at 8 TB/s (16e3 keys a us).  It is taken when that comes
// to 12 us at most, and always when all rows fit one tile of it.  Measured on the
// device, caches cold (rows, tiles), of 64 heads over 8: 4 rows behind 200 tokens 13,
// 22 us; 8 behind 2000 24, 26; 15 behind 1300 24, 26; 8 behind 16000 40, 33; 94 behind
// 119 32, 29; 1 behind 128000 95, 95.  Of 8 heads over 2 of 64, on both sides of the
// choice: 256 rows behind 1500 23, 25, 320 rows 28, 27; 256 behind 2000 26, 26, 320
// rows 32, 28; 192 behind 3000 26, 26, 256 rows 31, 27.  Calls of other shapes agree
// within 2 us but for a few that go on tiles and would be quicker by rows: 96 rows in 3
// sequences of 32 heads 30 for 26, 400 rows of 8 heads of 64 behind 500 28 for 22.
bool by_rows(int64_t M, int64_t mq, int G, const lr_attn_desc* d, int64_t cap_prefix, int64_t cap_own) {
  const int forced = test_attention_kernel();
  if (forced != 0) return forced == 1;
  if (M * G <= kRowsTile) return true;
  const double kv = d->cache.n_kv_heads;
  const double shared = kv * static_cast<double>(cdiv(M * G, kRowsTile));
  const double own = kv * static_cast<double>(cdiv(mq * G, kRowsTile)) * static_cast<double>(d->n_seq);
  const double wide = d->cache.head_dim / 128.0;
  const double keys = (shared * static_cast<double>(cap_prefix) + own * static_cast<double>(cap_own)) * wide;
  return 3.7 * wide * (shared + own) / (2.0 * num_sms()) + keys / 16e3 <= 12.0;
}

// CTAs of a planned call, by rows or on tiles (key ranges of tiles are another
// dimension of their grid).
int64_t plan_ctas(int64_t M, const lr_attn_desc* d, const AttnPlan& a) {
  const int64_t G = d->n_heads / d->cache.n_kv_heads, mq = most_q(M, d), pair = 2 * attn_tile_rows(static_cast<int>(G));
  if (a.tiles) return (a.whole ? d->n_seq * static_cast<int64_t>(cdiv(mq, pair)) : cdiv(M, pair)) * d->cache.n_kv_heads;
  return (static_cast<int64_t>(cdiv(M * G, kRowsTile)) * a.prefix_slots +
          d->n_seq * static_cast<int64_t>(cdiv(mq * G, kRowsTile)) * a.own_slots) * d->cache.n_kv_heads;
}

size_t result_bytes(int64_t rows, int64_t each) { return static_cast<size_t>(rows * each + 255) / 256 * 256; }

AttnPlan attn_plan(int64_t M, const lr_attn_desc* d) {
  AttnPlan a;
  memset(&a, 0, sizeof(a));
  const int G = d->n_heads / d->cache.n_kv_heads;
  const int64_t kv = d->cache.n_kv_heads, mq = most_q(M, d);
  const int64_t cap_prefix = static_cast<int64_t>(d->cap_prefix_blocks) * d->cache.block_rows;
  const int64_t cap_own = static_cast<int64_t>(d->blocks_per_seq) * d->cache.block_rows;
  const int64_t pair = 2 * attn_tile_rows(G);
  a.tiles = !by_rows(M, mq, G, d, cap_prefix, cap_own);
  // (the packed lists hold a sequence's number in 16 bits)
  a.whole = a.tiles && d->n_seq > 0 && (mq * G > 64 || (d->q_start != nullptr && d->n_seq > 32767));
  if (a.tiles) {
    // Steps of a row tile pair when all is full; packed tiles have the own tokens
    // of every sequence in them.
    const int64_t ctas = (a.whole ? larger(d->n_seq * cdiv(mq, pair), cdiv(M, pair)) : cdiv(M, pair)) * kv;
    const int64_t seqs = a.whole ? 1 : (d->n_seq < pair / 2 ? d->n_seq : pair / 2);
    const int64_t steps = cdiv(cap_prefix, 128) + cdiv(seqs * cap_own, 128);
    a.tile_slots = slots_for(ctas, steps, num_sms(), kMinSteps);
    if (a.tile_slots > kMaxSlots / 2) a.tile_slots = kMaxSlots / 2;
    if (a.tile_slots < 1) a.tile_slots = 1;
    // a row tile alone in its CTA gives two results a range (whole turns have
    // such tiles whatever their lengths)
    a.two = a.tile_slots > 1 && (a.whole || cdiv(M, attn_tile_rows(G)) % 2 == 1);
    a.prefix_slots = a.tile_slots > 1 ? a.tile_slots * (a.two ? 2 : 1) : 0;
  } else {
    // One wave: a row of 64 heads over 8 behind 16000 tokens takes 24, 26, 32 us
    // with 1, 2, 4 CTAs an SM, one of 32 over 32 behind 60000 167, 156, 155.
    const int64_t want = num_sms() * 2;
    a.prefix_slots = slots_for(static_cast<int64_t>(cdiv(M * G, kRowsTile)) * kv, cap_prefix, want, 128);
    // (rows of no sequence count as if they had one: the workspace's bound goes by rows)
    const int64_t own_tiles = larger(d->n_seq * cdiv(mq * G, kRowsTile), cdiv(M * G, kRowsTile));
    a.own_slots = d->n_seq == 0 ? 0 : slots_for(own_tiles * kv, cap_own, want, 128);
  }
  const int64_t rows = M * d->n_heads * (a.prefix_slots + a.own_slots);
  a.ml_off = result_bytes(rows, d->cache.head_dim * 4);
  a.bytes = a.ml_off + result_bytes(rows, 8);
  return a;
}

// Workspace for every call of up to M rows with up to d's sequences and pages.
// What a call itself needs goes up and down with its sizes, as the kernels and
// key ranges change (64 heads over 8 behind 8192 tokens: 18 MB for 64 rows, 16 for
// 256, none for 512), and a program that allocates once for its largest batch must
// serve the smaller ones.  R = M * n_heads rows have R times the most key ranges of
// results; and no call has more than
//   on tiles    ranges * row tile pairs <= SMs, 256 rows a pair, two results a range:
//               512 SMs;
//   by rows     of each part, either ranges * CTAs <= 2 SMs, with 16 rows a CTA, or one
//               range, R <= 104 SMs * 128 / head_dim by the limit of by_rows: 416 SMs at
//               most; or no more than one row tile a key head: 2 * 16 n_kv.
size_t attn_workspace(int64_t M, const lr_attn_desc* d) {
  // (zero for sizes that the call refuses, those that would overflow below among them)
  const int64_t cap_prefix = static_cast<int64_t>(d->cap_prefix_blocks) * d->cache.block_rows;
  const int64_t cap_own = d->n_seq > 0 ? static_cast<int64_t>(d->blocks_per_seq) * d->cache.block_rows : 0;
  if (M * d->n_heads > 0x7FFFFFFF || cap_prefix > 0x7FFFFFFF || cap_own > 0x7FFFFFFF) return 0;
  const int64_t R = M * d->n_heads;
  const int64_t pair = 2 * attn_tile_rows(d->n_heads / d->cache.n_kv_heads);
  const int64_t by_rows = smaller((cap_prefix + 127) / 128, kMaxSlots) + smaller((cap_own + 127) / 128, kMaxSlots);
  const int64_t steps = (cap_prefix + 127) / 128 + (smaller(d->n_seq, pair / 2) * cap_own + 127) / 128;
  const int64_t on_tiles = smaller((steps + kMinSteps - 1) / kMinSteps, kMaxSlots / 2);
  const int64_t one_tile = smaller(R, static_cast<int64_t>(kRowsTile) * d->cache.n_kv_heads);
  int64_t most = larger(512 * static_cast<int64_t>(num_sms()), 2 * one_tile);
  if (test_attention_kernel() == 1) most = larger(most, 2 * R);
  const int64_t rows = smaller(R * larger(by_rows, on_tiles > 1 ? 2 * on_tiles : 0), most);
  return result_bytes(rows, d->cache.head_dim * 4) + result_bytes(rows, 8);
}

lr_status check_desc(const char* who, int64_t M, const lr_attn_desc* d) {
  if (d == nullptr) return bad(LR_ERR_INVALID_ARG, "%s: null descriptor", who);
  lr_status st = check_kv_cache(who, &d->cache);
  if (st != LR_OK) return st;
  const lr_kv_cache& c = d->cache;
  if (M < 0 || M > 0x7FFFFFFF) return bad(LR_ERR_INVALID_ARG, "%s: bad M", who);
  if (d->n_heads <= 0 || d->n_heads % c.n_kv_heads)
    return bad(LR_ERR_INVALID_ARG, "%s: n_heads must be a positive multiple of n_kv_heads", who);
  if (c.head_dim != 64 && c.head_dim != 128)
    return bad(LR_ERR_UNSUPPORTED, "%s: head_dim %d is neither 64 nor 128", who, c.head_dim);
  if (c.block_rows % 16) return bad(LR_ERR_UNSUPPORTED, "%s: block_rows %d is not a multiple of 16", who, c.block_rows);
  if (d->n_heads / c.n_kv_heads > kMostHeads)
    return bad(LR_ERR_UNSUPPORTED, "%s: more than 64 query heads a key head", who);
  if (c.n_kv_heads > 65535) return bad(LR_ERR_UNSUPPORTED, "%s: more than 65535 key heads", who);
  if (!(d->scale > 0.f) || std::isinf(d->scale)) return bad(LR_ERR_INVALID_ARG, "%s: scale must be positive and finite", who);
  if (d->cap_prefix_blocks < 0 || d->blocks_per_seq < 0 || d->n_seq < 0)
    return bad(LR_ERR_INVALID_ARG, "%s: negative size", who);
  if (static_cast<int64_t>(d->cap_prefix_blocks) * c.block_rows > 0x7FFFFF00 ||
      static_cast<int64_t>(d->blocks_per_seq) * c.block_rows > 0x7FFFFF00)
    return bad(LR_ERR_INVALID_ARG, "%s: a context's rows overflow int32", who);
  if (d->cap_prefix_blocks > 0 && (!d->prefix_blocks || !d->prefix_len))
    return bad(LR_ERR_INVALID_ARG, "%s: null prefix", who);
  if (d->n_seq > 0 && (!d->lengths || (d->blocks_per_seq > 0 && !d->block_table)))
    return bad(LR_ERR_INVALID_ARG, "%s: null lengths or block table", who);
  if (d->q_start == nullptr ? (d->max_q != 1 || M < d->n_seq) : (d->max_q < 1))
    return bad(LR_ERR_INVALID_ARG, "%s: max_q must be at least 1, and 1 with a row for each sequence without q_start", who);
  // the own tokens of 128 sequences are counted in 32 bits
  if (static_cast<int64_t>(d->blocks_per_seq) * c.block_rows > 0x7FFFFFFF / 128)
    return bad(LR_ERR_UNSUPPORTED, "%s: an own context of more than 16 million rows", who);
  if (M * d->n_heads > 0x7FFFFFFF ||
      cdiv(most_q(M, d) * (d->n_heads / c.n_kv_heads), kRowsTile) * static_cast<int64_t>(d->n_seq) > 0x7FFFFFFF)
    return bad(LR_ERR_UNSUPPORTED, "%s: too many rows for one launch", who);
  return LR_OK;
}

}  // namespace

lr_status launch_attn_rows(const AttnParams& p, int head_dim, cudaStream_t s) {
  RowsLaunch rl;
  rl.tiles[0] = cdiv(static_cast<int64_t>(p.M) * p.group, kRowsTile);
  rl.tiles[1] = cdiv(static_cast<int64_t>(p.max_q) * p.group, kRowsTile);
  const int64_t ctas0 = static_cast<int64_t>(rl.tiles[0]) * p.n_kv * p.prefix_slots;
  const int64_t ctas = ctas0 + static_cast<int64_t>(rl.tiles[1]) * p.n_seq * p.n_kv * p.own_slots;
  if (ctas == 0) return LR_OK;
  rl.ctas0 = static_cast<int32_t>(ctas0);
  const dim3 grid(static_cast<unsigned>(ctas));
  if (head_dim == 64)
    return launch(attn_rows_kernel<64>, grid, dim3(kRowsWarps * 32), rows_smem<64>(), s, "attn_rows", p, rl);
  return launch(attn_rows_kernel<128>, grid, dim3(kRowsWarps * 32), rows_smem<128>(), s, "attn_rows", p, rl);
}

template <int HD>
static lr_status join(const AttnParams& p, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(p.M) * p.n_heads;
  if (p.prefix_slots + p.own_slots >= 16)
    return launch(attn_join_kernel<HD, 4>, dim3(cdiv(rows, 2)), dim3(256), 0, s, "attn_join", p);
  return launch(attn_join_kernel<HD, 1>, dim3(cdiv(rows, 8)), dim3(256), 0, s, "attn_join", p);
}

lr_status launch_attn_join(const AttnParams& p, int head_dim, cudaStream_t s) {
  return head_dim == 64 ? join<64>(p, s) : join<128>(p, s);
}

lr_status configure_attn() {
  cudaError_t e = cudaFuncSetAttribute(attn_rows_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, rows_smem<64>());
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attn_rows_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, rows_smem<128>());
  if (e != cudaSuccess) return cuda_fail(e, "attention: set smem");
  return LR_OK;
}

lr_status check_attention(const void* q, int64_t ldq, const void* out, int64_t ldo, lr_dtype out_dtype, int64_t M,
                          const lr_attn_desc* d, const void* workspace, size_t ws_bytes) {
  const char* who = "prefix_attention";
  lr_status st = check_desc(who, M, d);
  if (st != LR_OK) return st;
  if (out_dtype != LR_BF16 && out_dtype != LR_F32) return bad(LR_ERR_INVALID_ARG, "%s: bad output dtype", who);
  if (M == 0) return LR_OK;
  const lr_kv_cache& c = d->cache;
  const int64_t width = static_cast<int64_t>(d->n_heads) * c.head_dim;
  auto aligned = [](const void* x, uintptr_t a) { return (reinterpret_cast<uintptr_t>(x) & (a - 1)) == 0; };
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || ldq % 8 || ldo % 8 || ldq < width || ldo < width)
    return bad(LR_ERR_INVALID_ARG, "%s: q and out must be 16-byte aligned with leading dimensions >= %lld, multiples of 8", who,
               static_cast<long long>(width));
  const AttnPlan plan = attn_plan(M, d);
  if (plan_ctas(M, d, plan) > 0x7FFFFFFF) return bad(LR_ERR_UNSUPPORTED, "%s: too many rows for one launch", who);
  if (plan.bytes > 0 && (workspace == nullptr || !aligned(workspace, 256)))
    return bad(LR_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  if (ws_bytes < plan.bytes)
    return bad(LR_ERR_INVALID_ARG, "%s: workspace %zu < %zu bytes", who, ws_bytes, plan.bytes);
  return LR_OK;
}

}  // namespace lr

using namespace lr;

extern "C" {

size_t lr_prefix_attention_workspace_bytes(int64_t M, const lr_attn_desc* d) {
  if (d == nullptr || M <= 0 || M > 0x7FFFFFFF || d->cache.n_kv_heads <= 0 || d->n_heads < d->cache.n_kv_heads || d->max_q < 1 ||
      d->n_heads / d->cache.n_kv_heads > kMostHeads || d->cap_prefix_blocks < 0 || d->blocks_per_seq < 0 || d->n_seq < 0 ||
      d->cache.block_rows <= 0 || d->cache.head_dim <= 0 || d->cache.head_dim > 128)
    return 0;
  return attn_workspace(M, d);
}

lr_status lr_prefix_attention(const void* q, int64_t ldq, void* out, int64_t ldo, lr_dtype out_dtype, int64_t M,
                              const lr_attn_desc* d, void* workspace, size_t ws_bytes, int32_t* dev_status,
                              lr_stream s) {
  lr_status st = check_attention(q, ldq, out, ldo, out_dtype, M, d, workspace, ws_bytes);
  if (st != LR_OK || M == 0) return st;
  const lr_kv_cache& c = d->cache;
  const AttnPlan plan = attn_plan(M, d);
  st = ensure_configured();
  if (st != LR_OK) return st;

  AttnParams p;
  memset(&p, 0, sizeof(p));
  p.q = static_cast<const uint16_t*>(q);
  p.ldq = ldq;
  p.k = static_cast<const uint16_t*>(c.k);
  p.v = static_cast<const uint16_t*>(c.v);
  p.ld = c.ld;
  p.pool_blocks = c.pool_blocks;
  p.block_rows = c.block_rows;
  p.block_shift = -1;
  for (int i = 4; i < 31; ++i)
    if (c.block_rows == 1 << i) p.block_shift = i;
  p.n_heads = d->n_heads;
  p.n_kv = c.n_kv_heads;
  p.group = d->n_heads / c.n_kv_heads;
  p.scale_log2 = d->scale * 1.4426950408889634f;
  p.prefix_blocks = d->prefix_blocks;
  p.prefix_len = d->prefix_len;
  p.cap_prefix = d->cap_prefix_blocks * c.block_rows;
  p.M = static_cast<int32_t>(M);
  p.n_seq = d->n_seq;
  p.max_q = static_cast<int32_t>(most_q(M, d));
  p.q_start = d->q_start;
  p.block_table = d->block_table;
  p.blocks_per_seq = d->blocks_per_seq;
  p.lengths = d->lengths;
  p.cap_own = d->blocks_per_seq * c.block_rows;
  p.po = static_cast<float*>(workspace);
  p.pml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + plan.ml_off);
  p.prefix_slots = plan.prefix_slots;
  p.own_slots = plan.own_slots;
  p.out = out;
  p.ldo = ldo;
  p.out_f32 = out_dtype == LR_F32;
  p.status = dev_status;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(s);
  if (plan.tiles) {
    st = launch_attn_tiles(p, c.head_dim, AttnPart{plan.whole, plan.tile_slots, plan.two}, cs);
    if (plan.tile_slots == 1) return st;
  } else {
    st = launch_attn_rows(p, c.head_dim, cs);
  }
  if (st != LR_OK) return st;
  return launch_attn_join(p, c.head_dim, cs);
}

}  // extern "C"
