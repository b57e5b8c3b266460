// Attention over a cache held in 8 bits, for few query rows a sequence: a stream
// over the codes.
//
// A code is exact in 16-bit floats, and one instruction turns two codes into two
// of them, where bf16 would take five; so the products run on f16.
//   S = Q K^T:  a row of Q times the power of two that brings its largest element
//     to 2^14: exact but for elements under 2^-28 of it.  Back with the page's
//     scale: s = scale log2(e) 2^x ks (code . q).
//   O = P V:  the page's scale of V, 2^ev, goes into the powers, which keep a
//     reference of their own, m + dv, 7 below the largest s + ev: P' = 2^((s - m) + (ev - dv))
//     <= 2^15 for the product, O = sum P' code, and P = 2^(s - m) for the sum l = sum P.
//     out = 2^dv O / l.  (With the scale left in V, a page of large values that no row
//     attends to would push the others' powers under what f16 holds; with the largest power
//     at 1, the tail of a long context beside a few keys that take the most.  Scores enter by
//     their differences alone: a reference s + ev loses the scale beside scores of 2^24.)
//
// Bound by the bytes of K and V.  A CTA takes 8 NT rows (query rows times the heads
// of one key head) and a range of keys; each of its four warps walks chunks of 16
// keys on its own: a ring of chunks filled by 16-byte asynchronous copies, both
// products by m16n8k16 with the codes as the operand of 16 rows (keys, or elements
// of the head), so that the eight rows of a group of eight query heads fill the other
// operand, and its own maxima and sums, until the four join through shared memory.
// A lane reads 16 neighbouring codes of a key for S (the order of the head's
// elements in the reduction is free, Q has the same), and 16 neighbouring codes of
// four keys for O.
// Roundings: Q to f16 (above), powers to f16, whose error of 2^-11 is an eighth of
// bf16's (below 2^-21 of the largest, 2^-32 of that); scores, maxima, sums and O are fp32.
//
// Measured with the join, heads of 128, 64 over 8: one sequence of 131000 tokens 59 us
// (268 MB: 4.5 TB/s, 0.68 of the copy rate), 64 of 300 to 6000 86 us (415 MB, 4.8 TB/s,
// 0.72), 256 of 100 to 1500 78 us.  A copy of the kernel that only loads takes 126 of 144 us
// for 64 sequences of 6000: ranges start with three trips to memory one after another
// (lengths, pages, keys), and four CTAs an SM hide part of them.  Two stages a warp
// and five CTAs, four stages and three: even.  Products by m16n8k32 on the codes as they
// are, with Q as two e4m3 parts: even (what the conversions save, the second part costs).
// Several rows a key head in the other operand's eight columns: 16 and 32 rows a CTA cost
// two and four times the products, and are chosen where that many rows share the keys (32
// rows of heads of 128 take 255 registers and spill 180 to 330 bytes).  One width serves both
// parts of a launch: behind a short prefix that many sequences share, the own tokens' CTAs
// have the prefix's width, too.
#include <cuda_fp16.h>

#include <cmath>
#include <cstring>

#include "lr_attn.h"
#include "lr_ptx.cuh"

namespace lr {
namespace {

constexpr int kWarps = 4;
constexpr int kChunk = 16;
constexpr int kStages = 3;
constexpr float kSlack = 8.f;  // how far powers may pass their reference before it moves
constexpr float kLift = 7.f;   // powers for the product are 2^kLift times as large: 2^15 at most

template <int HD, int NT>
constexpr int smem8() {
  const int ring = kWarps * kStages * kChunk * HD * 2, join = kWarps * 8 * NT * (HD + 4) * 4;
  return ring > join ? ring : join;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void* src, bool live) {
  const int n = live ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
// The two codes in the low and in the high half of w, as f16.
__device__ __forceinline__ uint32_t f16_lo(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(w));
  return h;
}
__device__ __forceinline__ uint32_t f16_hi(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(h) : "r"(w));
  return h;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
  return h;
}
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Byte offsets of 16-byte unit u of key t in a chunk's tile of K and of V: units are
// permuted so that the lanes of a load lie in different banks (K: neighbouring keys,
// all units of a half row; V: every second key, one or two units).
template <int HD>
__device__ __forceinline__ uint32_t k_at(int t, int u) {
  return HD == 128 ? t * 128 + ((u ^ ((t & 1) << 2)) << 4) : t * 64 + (u << 4);
}
template <int HD>
__device__ __forceinline__ uint32_t v_at(int t, int u) {
  if (HD == 128) return t * 128 + ((u ^ ((t >> 1 & 3) << 1)) << 4);
  return (t >> 1) * 128 + ((((t & 1) << 2 | u) ^ ((t >> 1 & 3) << 1)) << 4);
}

template <int HD, int NT, bool WIN>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 4 : (NT == 2 ? 3 : 2))
    attn_rows8_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ Rows8Launch rl) {
  constexpr int kTile = 8 * NT;            // rows of the CTA
  constexpr int kPieces = HD / 64;         // 16-byte pieces of a key in a lane
  constexpr int kSteps = HD / 16;          // of the reduction over the head; tiles of 16 of its elements
  constexpr uint32_t kBytes = kChunk * HD; // of a chunk's K or V
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ float4 stats[kWarps][kTile];           // m, l, dv, whether a key was seen
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int G = p.group;
  // CTA -> part, row tile, key range, key head
  const int which = static_cast<int>(blockIdx.x) < rl.ctas0 ? 0 : 1;
  const bool prefix = !WIN && which == 0;
  const int slots = prefix ? p.prefix_slots : p.own_slots;
  int idx = static_cast<int>(blockIdx.x) - (which ? rl.ctas0 : 0);
  const int kvh = idx % p.n_kv;
  idx /= p.n_kv;
  const int split = idx % slots;
  const int tile = idx / slots;
  const bool tell = kvh == 0 && threadIdx.x == 0 && split == 0;

  // This CTA's rows, r = (query row - q0) * G + head in the group, and its list of
  // chunks: the prefix's, or the own tokens', or, with a window, the prefix's and then
  // the own ones less those, from skip on, that no row sees.
  int q0, n_rows, row0, P = 0, len, n, nq;
  const int32_t* own_pages = p.block_table;
  if (prefix) {
    q0 = 0;
    n = nq = p.M;
    len = prefix_view(p, tell);
    row0 = tile * kTile;
  } else {
    const int b = tile / rl.tiles[1];
    const SeqView v = seq_view(p, b, tell);
    q0 = v.q0, nq = v.nq, n = v.n, len = v.len;
    own_pages += static_cast<int64_t>(b) * p.blocks_per_seq;
    row0 = (tile - b * rl.tiles[1]) * kTile;
    if (WIN)
      P = prefix_view(p, tell);
    else if (p.direct)
      prefix_view(p, tell);  // (no pages of it; no join looks at a length that is given all the same)
  }
  if (p.direct && kvh == 0 && split == 0) zero_rows(p, tile, p.n_seq * rl.tiles[1], HD, kWarps * 32);
  n_rows = nq * G - row0;
  if (n_rows <= 0) return;
  if (n_rows > kTile) n_rows = kTile;
  // own tokens that the last row sees, or all of the prefix
  int kmax = prefix ? len : len - n + (row0 + n_rows - 1) / G + 1;
  if (kmax < 0) kmax = 0;
  WindowList w;
  if (WIN) w = window_list(P, len - n + row0 / G, kmax, p.window, p.sinks);
  const int chunks = WIN ? w.chunks : (kmax + kChunk - 1) / kChunk;
  int per = (chunks + slots - 1) / slots;
  if (per < rl.least) per = rl.least;
  const int64_t from64 = static_cast<int64_t>(split) * per;
  const int c_lo = from64 < chunks ? static_cast<int>(from64) : chunks;
  const int c_hi = c_lo + per < chunks ? c_lo + per : chunks;
  const int64_t slot_rows = static_cast<int64_t>(p.M) * p.n_heads;
  const int64_t slot0 = ((prefix ? 0 : p.prefix_slots) + split) * slot_rows;
  if (c_lo >= c_hi && !p.direct) {
    for (int rr = threadIdx.x; rr < n_rows; rr += kWarps * 32) {
      const int r = row0 + rr;
      p.pml[slot0 + static_cast<int64_t>(q0 + r / G) * p.n_heads + kvh * G + r % G] = make_float2(-INFINITY, 0.f);
    }
    return;
  }

  // Q as the operand of eight columns: lane (g, c) holds row g's elements 64 j + 16 c + 4 s ..
  uint32_t qb[NT][kSteps][2];
  float back[NT][2];          // what a product of rows 2c, 2c + 1 counts
  int hi[NT][2], lo[NT][2];   // visible positions: below hi, and from lo on
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int rr = t * 8 + g, r = row0 + rr;
    const uint16_t* src = p.q + static_cast<int64_t>(q0 + r / G) * p.ldq + static_cast<int64_t>(kvh * G + r % G) * HD;
    float x[kPieces][16];
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < kPieces; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (rr < n_rows) w = *reinterpret_cast<const uint4*>(src + j * 64 + c * 16 + h * 8);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[j][h * 8 + 2 * k] = __uint_as_float(u[k] << 16);
          x[j][h * 8 + 2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float m = fabsf(x[j][h * 8 + k]);
          if (m < INFINITY) top = fmaxf(top, m);
        }
      }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    int e = top > 0.f ? 14 + 127 - static_cast<int>(__float_as_uint(top) >> 23) : 0;
    e = e > 126 ? 126 : e;  // (bf16 is a multiple of 2^-133, so that nothing rounds where this holds)
    const float f = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
#pragma unroll
    for (int j = 0; j < kPieces; ++j)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        qb[t][j * 4 + s][0] = pack_f16(x[j][4 * s] * f, x[j][4 * s + 1] * f);
        qb[t][j * 4 + s][1] = pack_f16(x[j][4 * s + 2] * f, x[j][4 * s + 3] * f);
      }
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23) * p.scale_log2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      back[t][i] = __shfl_sync(0xffffffffu, inv, (2 * c + i) * 4);
      const int own = len - n + (row0 + t * 8 + 2 * c + i) / G;  // a row's own place
      hi[t][i] = prefix ? len : P + (own + 1 > 0 ? own + 1 : 0);
      lo[t][i] = WIN ? P + own - p.window + 1 : 0;
    }
  }

  // All rows see the positions below all_hi, and from all_lo on.
  int all_hi, all_lo = 0;
  {
    const int own = len - n + row0 / G, last = len - n + (row0 + n_rows - 1) / G;
    all_hi = prefix ? len : P + (own + 1 > 0 ? own + 1 : 0);
    if (WIN) all_lo = P + last - p.window + 1;
  }

  float o[NT][kSteps][4];  // elements 16 g + 2 i, + 1 (in steps of two) of rows 2c, 2c + 1
  float m[NT][2], dv[NT][2], l[NT][2];
  uint32_t saw = 0;  // bit 2 t + i: a key of that row
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
    m[t][0] = m[t][1] = dv[t][0] = dv[t][1] = -INFINITY;  // (no key yet)
    l[t][0] = l[t][1] = 0.f;
  }

  // Ring of this warp: a stage holds K then V of a chunk.
  const uint32_t ring = smem_u32(sm) + warp * kStages * 2 * kBytes;
  const int mine = c_hi - c_lo > warp ? (c_hi - c_lo - warp + kWarps - 1) / kWarps : 0;
  // Chunk i of this warp: its number in the list, its first token in its part.
  auto place = [&](int i, bool& shared) {
    int k = c_lo + warp + i * kWarps;
    shared = prefix;
    if (WIN) k = w.place(k, shared);
    return k * kChunk;
  };
  auto index_of = [&](int t) { return p.block_shift >= 0 ? t >> p.block_shift : t / p.block_rows; };
  // Lane i: page and scales (ks, and the bits of V's) of chunk i of the 32 that are being
  // asked for; the next 32 are looked up half way through.  The scales, a trip behind their
  // page, hold up no copy: they are kept for the 32 that are being worked on.
  int ids = -1, next_ids = -1;
  float2 asked = make_float2(0.f, 1.f), next_sc = asked, sc = asked;
  auto look = [&](int i, int& id, float2& s) {
    id = -1;
    s = make_float2(0.f, 1.f);
    if (i >= mine) return;
    bool shared;
    const int t = place(i, shared);
    const int page = (shared ? p.prefix_blocks : own_pages)[index_of(t)];
    if (page < 0 || page >= p.pool_blocks) {
      report_status(p.status, LR_ERR_REMAP_RANGE);
      s.y = 7.52316385e-37f;  // 2^-120, as of a page of zeros
      return;
    }
    id = page;
    const int64_t at = static_cast<int64_t>(page) * p.n_kv + kvh;
    s.x = p.k_scale[at];
    s.y = p.v_scale[at];
  };
  constexpr int kCols = HD / 16, kRows = 32 / kCols;  // an instruction copies kRows rows
  const int r_in = lane / kCols, col = lane % kCols;
  const uint8_t* k8 = reinterpret_cast<const uint8_t*>(p.k);
  const uint8_t* v8 = reinterpret_cast<const uint8_t*>(p.v);
  const int64_t head_off = static_cast<int64_t>(kvh) * HD + col * 16;
  auto issue = [&](int i) {
    if (i < mine) {
      if ((i & 31) == 0) ids = next_ids, asked = next_sc;
      if ((i & 31) == 16) look((i & ~31) + 32 + lane, next_ids, next_sc);
      const int page = __shfl_sync(0xffffffffu, ids, i & 31);
      const int stage = i % kStages;
      bool shared;
      const int t0 = place(i, shared);
      const int in_page = t0 - index_of(t0) * p.block_rows;
      const int pos0 = WIN && !shared ? P + t0 : t0;
      // tokens of the chunk that some row sees
      const int live = page < 0 ? 0 : (WIN && shared ? P - t0 : kmax - t0);
      const int64_t off = page < 0 ? 0 : (static_cast<int64_t>(page) * p.block_rows + in_page + r_in) * p.ld + head_off;
      const uint32_t st = ring + stage * 2 * kBytes;
      const int64_t step = kRows * p.ld;
      const uint8_t *kp = k8 + off, *vp = v8 + off;
      // (nearly all chunks are whole)
      if (live >= kChunk && (!WIN || pos0 >= w.lo_min || pos0 + kChunk <= p.sinks)) {
#pragma unroll
        for (int j = 0; j < kChunk / kRows; ++j, kp += step, vp += step) {
          const int r = j * kRows + r_in;
          cp16(st + k_at<HD>(r, col), kp);
          cp16(st + kBytes + v_at<HD>(r, col), vp);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kChunk / kRows; ++j, kp += step, vp += step) {
          const int r = j * kRows + r_in;
          const bool in = r < live && (!WIN || pos0 + r >= w.lo_min || pos0 + r < p.sinks);
          cp16_or_zero(st + k_at<HD>(r, col), in ? kp : k8, in);
          cp16_or_zero(st + kBytes + v_at<HD>(r, col), in ? vp : v8, in);
        }
      }
    }
    cp_commit();
  };
  look(lane, next_ids, next_sc);
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);

  for (int i = 0; i < mine; ++i) {
    issue(i + kStages - 1);
    cp_wait<kStages - 1>();
    __syncwarp();
    const int stage = i % kStages;
    const uint32_t st = ring + stage * 2 * kBytes;
    if ((i & 31) == 0) sc = asked;
    const float ks = __shfl_sync(0xffffffffu, sc.x, i & 31);
    // a power of two: its exponent
    const float ev = static_cast<float>(static_cast<int>(__float_as_uint(__shfl_sync(0xffffffffu, sc.y, i & 31)) >> 23 & 0xFFu) - 127);
    bool shared;
    const int t0 = place(i, shared);
    const int pos0 = WIN && !shared ? P + t0 : t0;
    const int end = WIN && shared ? P : 0x7FFFFFFF;

    float s[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const uint4 a = lds16(st + k_at<HD>(g, j * 4 + c)), b = lds16(st + k_at<HD>(g + 8, j * 4 + c));
      const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t a0 = f16_lo(aw[k]), a1 = f16_lo(bw[k]), a2 = f16_hi(aw[k]), a3 = f16_hi(bw[k]);
#pragma unroll
        for (int t = 0; t < NT; ++t) mma(s[t], a0, a1, a2, a3, qb[t][j * 4 + k][0], qb[t][j * 4 + k][1]);
      }
    }
    // s[0], s[1]: key g of rows 2c, 2c + 1; s[2], s[3]: key g + 8
    bool move = false;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float unit = ks * back[t][r];
        s[t][r] = s[t][r] * unit, s[t][r + 2] *= unit;
      }
    const int last = pos0 + kChunk;
    if (last <= all_hi && last <= end && (!WIN || pos0 >= all_lo || last <= p.sinks)) {  // all rows see the chunk
      saw = ~0u;
    } else {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int at = pos0 + g + (j >> 1) * 8, r = j & 1;
          const bool sees = at < (hi[t][r] < end ? hi[t][r] : end) && (!WIN || at >= lo[t][r] || at < p.sinks);
          if (!sees) s[t][j] = -INFINITY;
          if (sees) saw |= 1u << (2 * t + r);
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float base = m[t][r] == -INFINITY ? 0.f : m[t][r];
        const float limit = kSlack + fminf(0.f, dv[t][r] + (kLift - ev));
        move |= s[t][r] - base > limit || s[t][r + 2] - base > limit;
      }
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float top = fmaxf(s[t][r], s[t][r + 2]);
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
          const float now = fmaxf(m[t][r], top);
          const bool none = now == -INFINITY;
          const float less = none ? 0.f : m[t][r] - now, as_was = dv[t][r] + less;
          const float next = none ? -INFINITY : fmaxf(as_was, top - now + (ev - kLift));
          const float f = ex2(less), fo = none ? 1.f : ex2(as_was - next);
          m[t][r] = now, dv[t][r] = next;
          l[t][r] *= f;
#pragma unroll
          for (int i2 = 0; i2 < kSteps; ++i2) o[t][i2][r] *= fo, o[t][i2][r + 2] *= fo;
        }
    }
    uint32_t pb[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = j & 1;
        // (no key yet: every power is 2^-inf = 0)
        const bool none = m[t][r] == -INFINITY;
        const float u = s[t][j] - (none ? 0.f : m[t][r]);
        l[t][r] += ex2(u);
        x[j] = ex2(u + (none ? 0.f : ev - dv[t][r]));
      }
      // the product takes f16: its powers round here, those of the sum do not
      pb[t][0] = transposed(pack_f16(x[0], x[1]));
      pb[t][1] = transposed(pack_f16(x[2], x[3]));
    }
    {
      const uint32_t vt = st + kBytes;
      constexpr int kWords = HD / 32;  // of four codes, of each key
      uint32_t w[4][kWords];           // keys 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int t = 2 * c + (k & 1) + (k >> 1) * 8;
        if (HD == 128) {
          const uint4 x = lds16(vt + v_at<HD>(t, g));
          w[k][0] = x.x, w[k][1] = x.y, w[k][kWords - 2] = x.z, w[k][kWords - 1] = x.w;
        } else {
          const uint2 x = lds8(vt + v_at<HD>(t, g >> 1) + (g & 1) * 8);
          w[k][0] = x.x, w[k][1] = x.y;
        }
      }
#pragma unroll
      for (int d = 0; d < kWords; ++d) {
        // elements 4 d .. 4 d + 3 of the lane: pairs of keys side by side
        const uint32_t x0 = __byte_perm(w[0][d], w[1][d], 0x5140), x1 = __byte_perm(w[0][d], w[1][d], 0x7362);
        const uint32_t y0 = __byte_perm(w[2][d], w[3][d], 0x5140), y1 = __byte_perm(w[2][d], w[3][d], 0x7362);
        const uint32_t a[4] = {f16_lo(x0), f16_hi(x0), f16_lo(y0), f16_hi(y0)};
        const uint32_t b[4] = {f16_lo(x1), f16_hi(x1), f16_lo(y1), f16_hi(y1)};
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          mma(o[t][2 * d], a[0], a[1], a[2], a[3], pb[t][0], pb[t][1]);
          mma(o[t][2 * d + 1], b[0], b[1], b[2], b[3], pb[t][0], pb[t][1]);
        }
      }
    }
    __syncwarp();
  }
  cp_wait<0>();

  // Join the four warps: numerators in the ring's space, [warp][row][HD + 4].
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[t][r] += __shfl_xor_sync(0xffffffffu, l[t][r], x);
#pragma unroll
  for (int x = 4; x < 32; x <<= 1) saw |= __shfl_xor_sync(0xffffffffu, saw, x);
  __syncthreads();
  float* jo = reinterpret_cast<float*>(sm) + warp * kTile * (HD + 4);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int rr = t * 8 + 2 * c + r;
      if (g == 0) stats[warp][rr] = make_float4(m[t][r], l[t][r], dv[t][r], saw >> (2 * t + r) & 1u ? 1.f : 0.f);
      float* dst = jo + rr * (HD + 4) + g * (HD / 8);
#pragma unroll
      for (int i = 0; i < kSteps; i += 2)
        *reinterpret_cast<float4*>(dst + 2 * i) = make_float4(o[t][i][r], o[t][i][r + 2], o[t][i + 1][r], o[t][i + 1][r + 2]);
    }
  __syncthreads();
  for (int x = threadIdx.x; x < n_rows * (HD / 4); x += kWarps * 32) {
    const int rr = x / (HD / 4), d = x % (HD / 4);
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stats[w][rr].x);
    const float ref = top == -INFINITY ? 0.f : top;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    bool any = false;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 st = stats[w][rr];
      sum += ex2(st.x - ref) * st.y;
      any |= st.w != 0.f;
      if (st.z == -INFINITY) continue;  // nothing was summed
      // (the lift apart: with it 2^dv of the smallest scale would be subnormal)
      const float f = exp2f(st.x - ref + (st.z + kLift));
      float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(sm) + (w * kTile + rr) * (HD + 4) + d * 4);
      constexpr float kLower = 1.f / (1 << static_cast<int>(kLift));
      v.x *= kLower, v.y *= kLower, v.z *= kLower, v.w *= kLower;
      acc.x += f * v.x, acc.y += f * v.y, acc.z += f * v.z, acc.w += f * v.w;
    }
    const int r = row0 + rr;
    const int64_t row = q0 + r / G, head = kvh * G + r % G;
    if (p.direct) {  // the only range of keys
      const float inv = sum != 0.f ? 1.f / sum : (any ? NAN : 0.f);
      acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
      const int64_t at = row * p.ldo + head * HD + d * 4;
      if (p.out_f32) {
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = acc;
      } else {
        uint2 w;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(acc.y), "f"(acc.x));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(acc.w), "f"(acc.z));
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = w;
      }
      continue;
    }
    const int64_t at = slot0 + row * p.n_heads + head;
    if (sum != 0.f) *reinterpret_cast<float4*>(p.po + at * HD + d * 4) = acc;
    if (d == 0) p.pml[at] = make_float2(top, sum == 0.f && any ? -0.f : sum);
  }
}

template <int HD, int NT, bool WIN>
lr_status launch_as(const AttnParams& p, const Rows8Launch& rl, unsigned ctas, cudaStream_t s) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem8<HD, NT>();
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  if (pdl_enabled()) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_rows8_kernel<HD, NT, WIN>, p, rl);
  return e == cudaSuccess ? LR_OK : cuda_fail(e, "attn_rows8");
}

template <int HD, bool WIN>
lr_status launch_hd(const AttnParams& p, const Rows8Launch& rl, unsigned ctas, cudaStream_t s) {
  if (rl.tile == 8) return launch_as<HD, 1, WIN>(p, rl, ctas, s);
  if (rl.tile == 16) return launch_as<HD, 2, WIN>(p, rl, ctas, s);
  return launch_as<HD, 4, WIN>(p, rl, ctas, s);
}

template <int HD, bool WIN>
cudaError_t configure_hd() {
  cudaError_t e = cudaFuncSetAttribute(attn_rows8_kernel<HD, 1, WIN>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem8<HD, 1>());
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attn_rows8_kernel<HD, 2, WIN>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem8<HD, 2>());
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attn_rows8_kernel<HD, 4, WIN>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem8<HD, 4>());
  return e;
}

}  // namespace

lr_status launch_attn_rows8(const AttnParams& p, int head_dim, Rows8Launch rl, cudaStream_t s) {
  rl.tiles[0] = static_cast<int32_t>((static_cast<int64_t>(p.M) * p.group + rl.tile - 1) / rl.tile);
  rl.tiles[1] = static_cast<int32_t>((static_cast<int64_t>(p.max_q) * p.group + rl.tile - 1) / rl.tile);
  const int64_t ctas0 = static_cast<int64_t>(rl.tiles[0]) * p.n_kv * p.prefix_slots;
  const int64_t ctas = ctas0 + static_cast<int64_t>(rl.tiles[1]) * p.n_seq * p.n_kv * p.own_slots;
  if (ctas == 0) return LR_OK;
  rl.ctas0 = static_cast<int32_t>(ctas0);
  const unsigned n = static_cast<unsigned>(ctas);
  if (head_dim == 64) return p.window > 0 ? launch_hd<64, true>(p, rl, n, s) : launch_hd<64, false>(p, rl, n, s);
  return p.window > 0 ? launch_hd<128, true>(p, rl, n, s) : launch_hd<128, false>(p, rl, n, s);
}

lr_status configure_attn8() {
  cudaError_t e = configure_hd<64, false>();
  if (e == cudaSuccess) e = configure_hd<64, true>();
  if (e == cudaSuccess) e = configure_hd<128, false>();
  if (e == cudaSuccess) e = configure_hd<128, true>();
  return e == cudaSuccess ? LR_OK : cuda_fail(e, "attention in 8 bits: set smem");
}

}  // namespace lr
