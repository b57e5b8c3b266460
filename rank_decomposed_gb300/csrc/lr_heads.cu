// Norms of query and key heads with the position rotation in the same pass,
// and the append of keys and values to a paged cache, of bf16 or of 8 bits, with
// both on the way.
//
// For a head x at position p:  y = x * gain / sqrt(mean(x^2) + eps), then the
// pairs (a, b) of its first rot_dim elements become (a c - b s, b c + a s).
// Everything is fp32 in registers; the one rounding is the store to bf16 (the
// type of the cache and of the attention's operands).
//
// Bound by memory (a head is read and written once; about ten operations per
// element) or, for a few rows, by the launch.  A head belongs to a group of
// 8, 16 or 32 lanes with 8 neighbouring elements each: one 16-byte load and
// store per lane for bf16, the sum of squares by butterflies in the group, and
// the partner elements of the half style by shuffles.  A warp keeps the angles
// and the gains of its lanes in registers and walks several heads of one row
// with them: read per head, the angles (64 bytes a lane) would be four times
// the head's own bytes.
// Measured: 8191 rows of 64 + 8 heads of 128 in 63 us (302 MB and the angles: 4.9
// TB/s; a plain copy of the same bytes between two fresh buffers takes 50), an
// append of 4099 rows of 32 + 32 heads 24 us (134 MB, 5.6 TB/s), 64 rows of a
// decode step 6 us, one token 5 us, of which 3 are the launch and two trips to
// memory (positions, then angles) the rest.  Streaming hints on loads and stores
// changed nothing, the next heads asked for before the present ones are worked on
// took 64 us for the first and 25 to 31 for the second.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <type_traits>

#include "lr_attn.h"
#include "lr_ptx.cuh"

namespace lr {
namespace {

struct HeadParams {
  const void* src[3];   // q, k, v
  int64_t ld[3];
  void* dst[3];         // q_out, k_out or the K pool, the V pool
  int64_t ldo[3];
  int32_t heads[3];
  int32_t head_dim, lanes;
  float eps;
  const uint16_t* gain[2];
  int32_t rot_dim;
  const float* cos_sin;
  int64_t max_pos;
  const int32_t* pos;
  const int32_t* rows;  // append: the pool rows of k and v
  int64_t pool_rows;
  const int32_t* n_active;
  int32_t M;
  int32_t chunk;          // heads per warp
  int32_t warp_end[2];    // a row's warps: those of q, then of k, then of v
  int32_t row_warps;
  int32_t* status;
};

template <bool F32>
struct Raw;
template <>
struct Raw<false> {
  uint4 a;
};
template <>
struct Raw<true> {
  float4 a, b;
};

__device__ __forceinline__ void load_raw(Raw<false>& r, const void* base, int64_t off) {
  r.a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + off);
}
__device__ __forceinline__ void load_raw(Raw<true>& r, const void* base, int64_t off) {
  const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + off);
  r.a = p[0];
  r.b = p[1];
}
__device__ __forceinline__ void widen8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = __uint_as_float(w[j] << 16);
    x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack(const Raw<false>& r, float (&x)[8]) { widen8(r.a, x); }
__device__ __forceinline__ void unpack(const Raw<true>& r, float (&x)[8]) {
  x[0] = r.a.x, x[1] = r.a.y, x[2] = r.a.z, x[3] = r.a.w;
  x[4] = r.b.x, x[5] = r.b.y, x[6] = r.b.z, x[7] = r.b.w;
}

// The lane's partner elements: `from` holds them in the same order.
__device__ __forceinline__ void partners(const Raw<false>& r, float (&y)[8], int from) {
  uint4 v;
  v.x = __shfl_sync(0xffffffffu, r.a.x, from);
  v.y = __shfl_sync(0xffffffffu, r.a.y, from);
  v.z = __shfl_sync(0xffffffffu, r.a.z, from);
  v.w = __shfl_sync(0xffffffffu, r.a.w, from);
  widen8(v, y);
}
__device__ __forceinline__ void partners(const Raw<true>& r, float (&y)[8], int from) {
  float x[8];
  unpack(r, x);
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = __shfl_sync(0xffffffffu, x[j], from);
}

// Heads in flight per group: their loads are issued together.
constexpr int kFlight = 4;
// Small CTAs: a warp of few heads that is done makes room at once.
constexpr int kHeadWarps = 2, kHeadCtas = 12;
// Rounds of kFlight heads for one warp, at most.  1, 2, 4, 8: 8191 rows 71, 67, 68,
// 90 us cold, the append of 4099 rows 28, 25, 24, 24, 2000 rows 24, 23, 26, 30.
constexpr int kMostRounds = 2;

enum { ROT_NONE = 0, ROT_OF_HALVES = 1, ROT_OF_PAIRS = 2 };

// A head's result is inv * (x u + x' w) with x' the partner elements, u = gain
// cos and w = -+ gain' sin (gain' the partner's gain): u and w are the lane's
// for the whole row, so that a head costs two multiplications and an addition
// per element beside its norm.  Lanes past rot_dim have u = gain and no x'.
//
// A warp's heads are all of one kind.  Its first heads are asked for before the
// position, whose angles take two more trips to memory.
template <bool F32, bool NORM, int ROT>
__device__ __forceinline__ void heads_warp(const HeadParams& p, int64_t warp) {
  const int lane = threadIdx.x & 31;
  const int64_t m64 = warp / p.row_warps;
  int n = p.M;
  if (p.n_active != nullptr) {
    const int a = *p.n_active;
    n = a < 0 ? 0 : (a < n ? a : n);
  }
  if (m64 >= n) return;  // whole warps
  const int m = static_cast<int>(m64);
  const int part = static_cast<int>(warp - m64 * p.row_warps);
  const int kind = part < p.warp_end[0] ? 0 : (part < p.warp_end[1] ? 1 : 2);
  const int first = (part - (kind ? p.warp_end[kind - 1] : 0)) * p.chunk;
  const int sub = lane & (p.lanes - 1);      // lane in its group
  const int grp = lane / p.lanes, groups = 32 / p.lanes;
  const int e = sub * 8;                     // first element of this lane
  const bool lives = e < p.head_dim;         // a head of 192 leaves 8 lanes idle
  const int last = first + p.chunk < p.heads[kind] ? first + p.chunk : p.heads[kind];
  const int64_t src0 = m * p.ld[kind] + e;

  Raw<F32> raw[kFlight];
  auto ask = [&](int h0) {
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int h = h0 + f * groups + grp;
      if (h < last && lives)
        load_raw(raw[f], p.src[kind], src0 + h * p.head_dim);
      else
        memset(&raw[f], 0, sizeof(raw[f]));
    }
  };
  ask(first);

  // What a row's position and pool row allow: values need both, too.
  bool pos_ok = true;
  int64_t at = 0;
  if (ROT != ROT_NONE) {
    at = p.pos[m];
    pos_ok = at >= 0 && at < p.max_pos;
    if (!pos_ok && lane == 0 && part == 0) report_status(p.status, LR_ERR_INDEX_RANGE);
  }
  int64_t row = m;
  bool store = true;
  if (kind > 0 && p.rows != nullptr) {
    row = p.rows[m];
    const bool row_ok = row >= 0 && row < p.pool_rows;
    if (!row_ok && lane == 0) report_status(p.status, LR_ERR_REMAP_RANGE);
    store = row_ok && pos_ok;
  }
  const bool maps = kind < 2;  // values pass through
  const bool turns = ROT != ROT_NONE && maps && pos_ok && e < p.rot_dim;
  int partner = lane;
  float u[8], w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] = 1.f, w[j] = 0.f;
  if (NORM && maps && lives && p.gain[kind] != nullptr) widen8(*reinterpret_cast<const uint4*>(p.gain[kind] + e), u);
  if (turns) {
    const float* ang = p.cos_sin + at * p.rot_dim;
    const int half = p.rot_dim >> 1;
    float c[8], s[8];
    if (ROT == ROT_OF_HALVES) {
      const bool a = e < half;  // this lane holds the pairs' a, else their b
      const int i = a ? e : e - half;
      partner = a ? lane + (half >> 3) : lane - (half >> 3);
      if (NORM && p.gain[kind] != nullptr)
        widen8(*reinterpret_cast<const uint4*>(p.gain[kind] + (a ? e + half : e - half)), w);
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        const float4 cv = *reinterpret_cast<const float4*>(ang + i + j);
        const float4 sv = *reinterpret_cast<const float4*>(ang + half + i + j);
        c[j] = cv.x, c[j + 1] = cv.y, c[j + 2] = cv.z, c[j + 3] = cv.w;
        s[j] = sv.x, s[j + 1] = sv.y, s[j + 2] = sv.z, s[j + 3] = sv.w;
      }
      const bool unit = !NORM || p.gain[kind] == nullptr;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[j] *= c[j];
        w[j] = (a ? -s[j] : s[j]) * (unit ? 1.f : w[j]);
      }
    } else {
      const float4 cv = *reinterpret_cast<const float4*>(ang + (e >> 1));
      const float4 sv = *reinterpret_cast<const float4*>(ang + half + (e >> 1));
      c[0] = c[1] = cv.x, c[2] = c[3] = cv.y, c[4] = c[5] = cv.z, c[6] = c[7] = cv.w;
      s[0] = s[1] = sv.x, s[2] = s[3] = sv.y, s[4] = s[5] = sv.z, s[6] = s[7] = sv.w;
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float g0 = u[j], g1 = u[j + 1];
        w[j] = -g1 * s[j], w[j + 1] = g0 * s[j + 1];
        u[j] = g0 * c[j], u[j + 1] = g1 * c[j + 1];
      }
    }
  }

  const float inv_d = 1.f / static_cast<float>(p.head_dim);
  uint16_t* dst = static_cast<uint16_t*>(p.dst[kind]) + row * p.ldo[kind] + e;
  for (int h0 = first;;) {
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      if (h0 + f * groups >= last) break;  // the whole warp is past its heads
      const int h = h0 + f * groups + grp;
      float x[8], y[8];
      unpack(raw[f], x);
      // all of a warp takes part in the shuffles, heads or not
      float inv = 1.f;
      if (NORM) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
        for (int o = p.lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (maps) inv = rsqrtf(fmaf(ss, inv_d, p.eps));
      }
      if (ROT == ROT_OF_HALVES) partners(raw[f], y, partner);
      if (turns) {
        if (ROT == ROT_OF_PAIRS) {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = x[j ^ 1];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = fmaf(x[j], u[j], y[j] * w[j]) * inv;
      } else if (NORM && maps) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= u[j] * inv;
      }
      if (h < last && lives && store) {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
          memcpy(&o[j], &b, 4);
          if (ROT != ROT_NONE && !pos_ok) o[j] = 0u;
        }
        *reinterpret_cast<uint4*>(dst + h * p.head_dim) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    h0 += kFlight * groups;
    if (h0 >= last) break;
    ask(h0);
  }
}

template <bool F32, bool NORM, int ROT>
__global__ void __launch_bounds__(kHeadWarps * 32, kHeadCtas) heads_kernel(const __grid_constant__ HeadParams p) {
  pdl_launch_dependents();
  pdl_wait();
  heads_warp<F32, NORM, ROT>(p, static_cast<int64_t>(blockIdx.x) * kHeadWarps + (threadIdx.x >> 5));
}

// ------------------------------------------------- append in 8 bits
//   y = norm and rotation of x, fp32;  e = least integer >= -120 with max |y| <= 448 2^e
//   over the new rows of a page and head (no less than the page's, if tokens precede
//   them there);  scale = 2^e,  code = rn_e4m3(y 2^-e).
// The one rounding is the code's, and of codes made anew that become subnormal: the
// type of the cache.  Scales are powers of two, so that nothing else rounds.
//
// The keys and values that go to one page share a scale a head, so the unit of
// work is a run, the new rows of one page, of one head.  A warp takes the runs of one
// head that start among `window` tokens, as many rows at a time as its registers hold
// (eight rounds of one to four): it norms and rotates their elements, finds the largest
// magnitude of each run, fixes the exponents and stores the codes.  Where pages are longer
// a CTA looks at up to 62 tokens: of a run that is too long for a warp each of its four
// warps holds a part, and they tell each other their largest magnitudes; the other runs
// they share out.  Pages beyond that (over 64 rows for heads of 128) are walked piece by
// piece, twice.  A lane's eight elements of a row are two times four, for the half style
// of rotation the a and the b of four pairs: the pairs' cosines and sines are loaded once
// and no element is exchanged.  Runs follow from the rows alone: one starts where a row
// does not follow the row before it or opens a page.  A warp looks at one token for a
// decode step, whose rows are all of different pages, and at up to 16 where 16 warps an SM
// remain.
//
// Bound by memory in bytes (4099 rows of 32 + 32 heads: 101 MB and the angles, 15 us), but a
// head takes 1200 instructions a warp of 16 rows, behind several trips to memory one after
// another (rows, positions, elements and angles, the page's scale), and 128 registers leave
// room for 16 warps an SM: 37.5 us, 2.7 TB/s, 36 % of the issue slots (with one head a warp
// 41); with norms 45.  64 rows of a decode step with their queries 5 us.  In pages of 64 rows
// the 4099 take 52 us (walked twice, 93), with norms 59, in pages of 256, which are walked, 128
// and 175; 777 fp32 rows of 2 heads of 64 in pages of 64 8 (walked, 19), 300 of 8 + 8 heads
// 8.5 (38), the decode step 5 (5).  These are calls in turn over pages whose scales have grown
// before; where every page's scale grows, so that the codes before the new rows are made anew,
// and caches are flushed the 4099 take 48 us (43 without), the decode step 14 (10).  With norms
// the rotated variants spill (a warp's runs 8 to 124 bytes, teams 110 to 220, walked pages 670 to
// 1360), without them the walked ones (270 to 640) alone.
// Others measured for the 4099 rows in pages of 16: a warp a run
// without windows 56; eight warps a page with a barrier a head 84; the elements in shared
// memory and two walks 48 to 57; elements held as they were loaded and mapped twice 42 to 48.
struct AppendParams {
  HeadParams h;           // sources, maps, positions and rows as for the bf16 cache; dst[1], dst[2] hold codes
  float* scale[2];        // of the keys, of the values: [page][head]
  int32_t block_rows;
  int32_t window;
  int32_t block_shift;    // log2(block_rows), or -1
  int32_t hold;           // rows that a warp holds, 32 at most
  int32_t q_blocks;       // CTAs of the queries' heads, before the others
};

constexpr int kLeast8 = -120;  // exponent of the scale of a page of zeros
constexpr int kAppendWarps = 4, kRounds = 8;  // rounds of rows that a warp holds

// The least e with x <= 448 * 2^e for a finite x >= 0: 448 = 1.75 * 2^8, so the
// mantissa's part above 1.75 carries into the exponent.
__device__ __forceinline__ int exponent8(float x) {
  const int e = static_cast<int>((__float_as_uint(x) + 0x1FFFFFu) >> 23) - 127 - 8;
  return e < kLeast8 ? kLeast8 : e;
}
__device__ __forceinline__ float power_of(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Two codes; the first argument's is the low byte.
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
  return c;
}
// Codes of four elements, scaled by 2^d (d <= 0).
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w >> (16 * i))));
    __half2 x;
    memcpy(&x, &h, 4);
    const float2 y = __half22float2(x);
    out |= codes2(y.x * f, y.y * f) << (16 * i);
  }
  return out;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// How a page's rows are held: all of them by a warp; by the warps of a CTA, each a part of
// a run, who tell each other their largest magnitudes; or not, and walked twice.
enum { kByWarp, kByTeam, kWalked, kByWarpTwo };  // (the last: for two heads)
template <bool F32, bool NORM, int ROT, int HOW>
__global__ void __launch_bounds__(kAppendWarps * 32, 4) append8_kernel(const __grid_constant__ AppendParams a) {
  pdl_launch_dependents();
  pdl_wait();
  const HeadParams& p = a.h;
  if (static_cast<int>(blockIdx.x) < a.q_blocks) {
    heads_warp<F32, NORM, ROT>(p, static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5));
    return;
  }
  constexpr bool LONG = HOW == kWalked, TEAM = HOW == kByTeam;
  constexpr int kEach = HOW == kByWarpTwo ? 2 : 1;
  __shared__ float tops[TEAM ? 2 : 1][kAppendWarps];
  const int lane = threadIdx.x & 31, part = TEAM ? threadIdx.x >> 5 : 0;  // of a run
  const uint32_t warp = TEAM ? blockIdx.x - a.q_blocks : (blockIdx.x - a.q_blocks) * kAppendWarps + (threadIdx.x >> 5);  // (below 2^31)
  const int heads = p.heads[1], br = a.block_rows;
  // head fastest: the warps of a CTA share the angles of their tokens
  const uint32_t groups_of = (heads + kEach - 1) / kEach, rest = warp / groups_of;
  const int head0 = static_cast<int>(warp - rest * groups_of) * kEach;
  const int kind = 1 + static_cast<int>(rest & 1);
  const int64_t first_m = static_cast<int64_t>(rest >> 1) * a.window;
  int n = p.M;
  if (p.n_active != nullptr) {
    const int x = *p.n_active;
    n = x < 0 ? 0 : (x < n ? x : n);
  }
  if (first_m >= n) return;  // whole warps
  const int base = static_cast<int>(first_m);
  const int log_groups = p.lanes == 8 ? 2 : (p.lanes == 16 ? 1 : 0), groups = 1 << log_groups;
  const int sub = lane & (p.lanes - 1), grp = lane >> (5 - log_groups);
  const bool lives = sub * 8 < p.head_dim;
  const bool maps = kind == 1;
  const bool turns = ROT != ROT_NONE && maps && sub * 8 < p.rot_dim;
  const int half = p.rot_dim >> 1;
  // the lane's elements: four from o1 on and four from o2 on
  const bool halves = ROT == ROT_OF_HALVES && turns;
  const int o1 = halves ? sub * 4 : sub * 8, o2 = halves ? half + sub * 4 : sub * 8 + 4;
  const float inv_d = 1.f / static_cast<float>(p.head_dim);
  constexpr int kSize = F32 ? 4 : 2;
  float gain[NORM ? 8 : 1];
  if (NORM) {
#pragma unroll
    for (int j = 0; j < 8; ++j) gain[j] = 1.f;
    if (maps && lives && p.gain[1] != nullptr) {
      const uint2 x = *reinterpret_cast<const uint2*>(p.gain[1] + o1), y = *reinterpret_cast<const uint2*>(p.gain[1] + o2);
      widen8(make_uint4(x.x, x.y, y.x, y.y), *reinterpret_cast<float(*)[8]>(gain));
    }
  }

  // Lane i holds the row of token base - 1 + i; a row that continues the one before
  // it in its page belongs to that one's run.
  auto row_of = [&](int m) { return m >= 0 && m < n ? p.rows[m] : -1; };
  auto page_of = [&](int row) { return a.block_shift >= 0 ? row >> a.block_shift : row / br; };
  auto continues = [&](int before, int row) {
    return row > 0 && row < p.pool_rows && row == before + 1 && row != page_of(row) * br;
  };
  // A team looks at twice as many tokens.
  using Mask = std::conditional_t<TEAM, uint64_t, uint32_t>;
  constexpr int kSeen = TEAM ? 63 : 31;
  auto first_of = [](Mask m) { return (TEAM ? __ffsll(static_cast<long long>(m)) : __ffs(static_cast<int>(m))) - 1; };
  // (the positions of the same tokens on the way with the rows)
  const int near = ROT != ROT_NONE && !LONG && base + lane < n ? p.pos[base + lane] : -1;
  const int seen = row_of(base - 1 + lane);
  const int before = __shfl_up_sync(0xffffffffu, seen, 1);
  Mask follows = __ballot_sync(0xffffffffu, lane > 0 && continues(before, seen)) >> 1;  // bit i: token base + i
  int seen2 = -1;
  if (TEAM) {
    seen2 = row_of(base + 31 + lane);
    const int last = __shfl_sync(0xffffffffu, seen, 31), up = __shfl_up_sync(0xffffffffu, seen2, 1);
    follows |= static_cast<Mask>(static_cast<uint64_t>(__ballot_sync(0xffffffffu, continues(lane > 0 ? up : last, seen2))) << (TEAM ? 31 : 0));
  }
  const int here = n - base < a.window ? n - base : a.window;  // (at most kSeen - 1)
  Mask starts = ~follows & ((static_cast<Mask>(1) << here) - 1);
  // A team's runs that one warp does not hold are taken by all of it, first; of the others
  // every warp has a quarter.
  Mask together = 0;
  if (TEAM && (follows & ((static_cast<Mask>(2) << here) - 1)) == 0) {  // single rows
    const int share = (here + kAppendWarps - 1) / kAppendWarps;
    starts &= ((static_cast<Mask>(1) << share) - 1) << (part * share);
  } else if (TEAM) {
    for (Mask left = starts; left != 0; left &= left - 1) {
      const int i = first_of(left), run = 1 + first_of(~(follows >> i >> 1));
      if (run > a.hold || i + run == kSeen) together |= left & (~left + 1);
    }
    starts &= ~together;
    const int share = (__popcll(starts) + kAppendWarps - 1) / kAppendWarps;
    Mask mine = 0;
    for (int k = 0; starts != 0 && k < (part + 1) * share; ++k, starts &= starts - 1)
      if (k >= part * share) mine |= starts & (~starts + 1);
    starts = mine;
  }
  int turn = 0;
  // The largest of the team's.
  auto of_team = [&](float m) {
    if (lane == 0) tops[turn][part] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAppendWarps; ++w) m = fmaxf(m, tops[turn][w]);
    turn ^= 1;
    return m;
  };

  while (together != 0 || starts != 0) {
    const bool joint = TEAM && together != 0;
    Mask left = joint ? together : starts;
    // The next runs that fit, or one: tokens m0 .. m0 + total, bit k of `opens` where one starts.
    const int i0 = first_of(left);
    int m0 = base + i0, total = 0, run_row = -1, run_rows = 0;
    uint32_t opens = 0;
    while (left != 0) {
      const int i = first_of(left);
      const Mask tail = ~(follows >> i >> 1);
      int run = 1 + first_of(tail);  // (the highest bit of follows is clear: there is a zero)
      if (joint) run_row = i + 1 < 32 ? __shfl_sync(0xffffffffu, seen, i + 1) : __shfl_sync(0xffffffffu, seen2, i + 1 - 32);
      if (i + run == kSeen) {         // it goes on behind what the lanes hold
        const int row0 = joint ? run_row : __shfl_sync(0xffffffffu, seen, i + 1);
        for (;;) {
          const int r = row_of(base + i + run + lane);
          const uint32_t more = __ballot_sync(0xffffffffu, r == row0 + run + lane && r < p.pool_rows && page_of(r) == page_of(row0));
          const int k = more == ~0u ? 32 : __ffs(~more) - 1;
          run += k;
          if (k < 32) break;
        }
      }
      if (total > 0 && (total + run > a.hold || i != i0 + total)) break;
      opens |= 1u << (i - i0);
      total += run;
      left &= left - 1;
      if (joint) {
        run_rows = run;
        break;
      }
    }
    if (joint)
      together = left;
    else
      starts = left;
    const int skip = joint ? part * a.hold : 0;  // this warp's part of the run
    if (joint) {
      total = total - skip < 0 ? 0 : (total - skip < a.hold ? total - skip : a.hold);
      m0 += skip;
    }

    // Lane k: token m0 + k, its row and the scale of its page.
    const bool one = joint || (opens & (opens - 1)) == 0;
    int row = lane < total ? p.rows[m0 + lane] : -1;
    int joint_at = 0;  // position of the run's first row
    if (joint && ROT != ROT_NONE) joint_at = i0 < 32 ? __shfl_sync(0xffffffffu, near, i0) : p.pos[base + i0];
    const bool row_ok = row >= 0 && row < p.pool_rows;
    if (lane < total && !row_ok) report_status(p.status, LR_ERR_REMAP_RANGE);
    if (!row_ok) row = -1;
    const int opener = joint ? 0 : 31 - __clz(opens & (0xffffffffu >> (31 - lane)));  // lane of the run's first token
    const int row0 = joint ? (run_row >= 0 && run_row < p.pool_rows ? run_row : -1) : __shfl_sync(0xffffffffu, row, opener);
    const int page = row0 < 0 ? 0 : page_of(row0);
    float* scale = a.scale[kind - 1] + static_cast<int64_t>(page) * heads + head0;
    float old = 0.f;

    const uint8_t* src = static_cast<const uint8_t*>(p.src[kind]) + (static_cast<int64_t>(m0) * p.ld[kind] + static_cast<int64_t>(head0) * p.head_dim) * kSize;
    const int64_t step = p.ld[kind] * kSize;
    // Position of lane k's token, -1 where it is none or out of range: such a row counts
    // for nothing.
    auto position = [&](int t, bool tell) {
      if (t >= total) return -1;
      if (ROT == ROT_NONE) return 0;
      const int at = p.pos[m0 + t];
      if (at >= 0 && at < p.max_pos) return at;
      if (tell) report_status(p.status, LR_ERR_INDEX_RANGE);
      return -1;
    };
    // The lane's elements of row t of the batch, as they come.
    auto load = [&](const uint8_t* from, bool in, float (&x)[8]) {
      const int between = (o2 - o1) * kSize;
      if (F32) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f), w = v;
        if (in) v = *reinterpret_cast<const float4*>(from), w = *reinterpret_cast<const float4*>(from + between);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w, x[4] = w.x, x[5] = w.y, x[6] = w.z, x[7] = w.w;
      } else {  // (two elements a register until they are used)
        uint2 v = make_uint2(0, 0), w = v;
        if (in) v = *reinterpret_cast<const uint2*>(from), w = *reinterpret_cast<const uint2*>(from + between);
        x[0] = __uint_as_float(v.x), x[2] = __uint_as_float(v.y), x[4] = __uint_as_float(w.x), x[6] = __uint_as_float(w.y);
      }
    };
    auto turn_by = [&](int at, float4& c, float4& s) {
      if (ROT == ROT_NONE || !turns) return;  // (of a row that counts for nothing, any)
      const float* ang = p.cos_sin + static_cast<uint64_t>(static_cast<uint32_t>(at < 0 ? 0 : at)) * static_cast<uint32_t>(p.rot_dim) + sub * 4;
      c = *reinterpret_cast<const float4*>(ang), s = *reinterpret_cast<const float4*>(ang + half);
    };
    // Normed and rotated.  The row's factor goes to the elements before their scale does: a head of zeros
    // has the factor eps^-1/2 and the scale 2^-120, whose quotient may be infinite.
    auto map = [&](float (&x)[8], const float4& c, const float4& s) {
      if (!F32) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const uint32_t w = __float_as_uint(x[j]);
          x[j] = __uint_as_float(w << 16), x[j + 1] = __uint_as_float(w & 0xFFFF0000u);
        }
      }
      float inv = 1.f;
      if (NORM && maps) {  // (all of the warp)
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
        for (int o = p.lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        inv = rsqrtf(fmaf(ss, inv_d, p.eps));
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= gain[NORM ? j : 0];
      }
      if (ROT != ROT_NONE && turns) {
        const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = ROT == ROT_OF_HALVES ? k : 2 * k, j = ROT == ROT_OF_HALVES ? k + 4 : 2 * k + 1;
          const float u = x[i], w = x[j];
          x[i] = u * cv[k] - w * sv[k];
          x[j] = w * cv[k] + u * sv[k];
        }
      }
      if (NORM && maps) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= inv;
      }
    };
    auto largest = [&](const float (&x)[8]) {
      float m = 0.f;  // (passes a NaN over: of NaN alone, zero)
#pragma unroll
      for (int j = 0; j < 8; j += 2) m = max3(m, fabsf(x[j]), fabsf(x[j + 1]));
      return m;
    };
    uint8_t* codes = static_cast<uint8_t*>(p.dst[kind]) + static_cast<int64_t>(head0) * p.head_dim;
    auto keep = [&](uint8_t* d, const float (&x)[8], float unit) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = codes2(x[2 * j] * unit, x[2 * j + 1] * unit);
      *reinterpret_cast<uint32_t*>(d + o1) = w[0] | w[1] << 16;
      *reinterpret_cast<uint32_t*>(d + o2) = w[2] | w[3] << 16;
    };
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);

    // The batch in registers, unless it is one long run.
    int at = -1;
    if (LONG || ROT == ROT_NONE || m0 - base + total > 32) {
      at = position(lane, true);
    } else {
      at = __shfl_sync(0xffffffffu, near, (m0 - base + lane) & 31);
      if (lane >= total) {
        at = -1;
      } else if (at < 0 || at >= p.max_pos) {
        report_status(p.status, LR_ERR_INDEX_RANGE);
        at = -1;
      }
    }
    // Row of the run's first token that counts, -1 if none does: rows before it are the page's
    // earlier ones, and a run that counts for nothing leaves its page alone.
    int first_row = row0;
    if (ROT != ROT_NONE) {
      auto lead_of = [&](int from, int n) {  // of n tokens of one run: how many are before the first that counts
        for (int t = 0; t < n; t += 32) {
          const int x = t + lane < n ? p.pos[from + t + lane] : -1;
          const uint32_t counts = __ballot_sync(0xffffffffu, x >= 0 && x < p.max_pos);
          if (counts != 0) return t + __ffs(counts) - 1;
        }
        return -1;
      };
      const uint32_t counts = __ballot_sync(0xffffffffu, at >= 0 && row >= 0);
      int lead = 0;
      if (joint) {
        if (joint_at < 0 || joint_at >= p.max_pos) lead = lead_of(base + i0, run_rows);
      } else if (LONG && total > 32) {
        if ((counts & 1u) == 0) lead = lead_of(m0, total);
      } else if (counts != __ballot_sync(0xffffffffu, row >= 0)) {
        const uint32_t later = opens & ~((2u << opener) - 1);  // (of lane 31 none)
        const int end = later != 0 ? __ffs(later) - 1 : total;
        const uint32_t mine = counts >> opener << opener & (end < 32 ? (1u << end) - 1 : ~0u);
        lead = mine != 0 ? __ffs(mine) - 1 - opener : -1;
      }
      if (lead != 0) first_row = lead < 0 || row0 < 0 ? -1 : row0 + lead;
    }
    const int held_rows = first_row < 0 ? 0 : first_row - page * br;
    // (what the lanes know of the rows serves several heads)
#pragma unroll 1
    for (int head = 0; head < kEach && (kEach == 1 || head0 + head < heads); ++head, ++scale, src += p.head_dim * kSize, codes += p.head_dim) {
      old = held_rows > 0 ? *scale : 0.f;
      float top = 0.f, all = 0.f;
      float x[kRounds][8];
      const bool held = !LONG || total <= a.hold;
      if (held) {
        const uint8_t* from = src + grp * step + o1 * kSize;
#pragma unroll
        for (int f = 0; f < kRounds; ++f, from += step << log_groups) {
          if (f << log_groups >= total) break;
          load(from, (f << log_groups) + grp < total && lives, x[f]);
        }
        float4 next_c = none, next_s = none;  // asked for a round ahead
        int next_at = __shfl_sync(0xffffffffu, at, grp);
        turn_by(next_at, next_c, next_s);
#pragma unroll
        for (int f = 0; f < kRounds; ++f) {
          if (f << log_groups >= total) break;
          const int where = next_at;
          const float4 c = next_c, s = next_s;
          if (f + 1 < kRounds) {
            next_at = __shfl_sync(0xffffffffu, at, ((f + 1 << log_groups) + grp) & 31);
            turn_by(next_at, next_c, next_s);
          }
          map(x[f], c, s);
          float m = largest(x[f]);
          if (where < 0) m = 0.f;
          if (one) {
            all = fmaxf(all, m);
          } else {  // of each row, in its lane
            for (int o = p.lanes >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            m = __shfl_sync(0xffffffffu, m, (lane & (groups - 1)) << (5 - log_groups));
            if (lane >> log_groups == f) top = m;
          }
        }
      }
      // The exponent of lane k's run, its scale, and the codes of the rows before it.
      auto settle = [&](float top) {
        int e = exponent8(top);
        bool grows = false;
        if (held_rows > 0) {
          const int had = static_cast<int>(__float_as_uint(old) >> 23 & 0xFFu) - 127;
          grows = e > had;
          if (!grows) e = had;
        }
        e = e < kLeast8 ? kLeast8 : (e > 120 ? 120 : e);  // (a scale that was none)
        // the codes of the rows before a run, anew
        const bool opens_run = first_row >= 0 && (joint ? lane == 0 : lane == opener && lane < total);
        for (uint32_t left = __ballot_sync(0xffffffffu, grows && opens_run); left != 0; left &= left - 1) {
          const int who = __ffs(left) - 1;
          const int first = joint ? first_row : __shfl_sync(0xffffffffu, first_row, who), rows = first - page_of(first) * br;
          const int less = (static_cast<int>(__float_as_uint(__shfl_sync(0xffffffffu, old, who)) >> 23 & 0xFFu) - 127) - __shfl_sync(0xffffffffu, e, who);
          const float f = power_of(less < -126 ? -126 : less);
          for (int t = grp + (joint ? part << log_groups : 0); t < rows && lives; t += joint ? kAppendWarps << log_groups : groups) {
            uint2* y = reinterpret_cast<uint2*>(codes + static_cast<int64_t>(first - rows + t) * p.ldo[kind] + sub * 8);
            uint2 w = *y;
            w.x = rescale4(w.x, f), w.y = rescale4(w.y, f);
            *y = w;
          }
        }
        if (opens_run && !(joint && part > 0)) *scale = power_of(e);
        return e;
      };
      // A run by itself: the largest finite magnitude of one that is long or has
      // infinities (they end as NaN), or its codes.
      auto by_itself = [&](int t0, int end, bool storing, float unit, int first_row) {
        float m = 0.f;
        constexpr int kTogether = LONG ? 4 : 1;  // rounds whose loads are on their way together
        int next[kTogether];  // positions are asked for a turn ahead, as the angles wait for them
        auto ask = [&](int t) {
#pragma unroll
          for (int k = 0; k < kTogether; ++k) {
            const int r = t + (k << log_groups) + grp;
            next[k] = r < end ? position(r, !storing && !held) : -1;
          }
        };
        ask(t0);
#pragma unroll 1
        for (int t = t0; t < end; t += kTogether << log_groups) {
          float y[kTogether][8];
          float4 c[kTogether], s[kTogether];
          int where[kTogether];
#pragma unroll
          for (int k = 0; k < kTogether; ++k) {
            const int r = t + (k << log_groups) + grp;
            c[k] = s[k] = none;
            where[k] = next[k];
            load(src + r * step + o1 * kSize, r < end && lives, y[k]);
          }
#pragma unroll
          for (int k = 0; k < kTogether; ++k) turn_by(where[k], c[k], s[k]);
          ask(t + (kTogether << log_groups));
#pragma unroll
          for (int k = 0; k < kTogether; ++k) {
            map(y[k], c[k], s[k]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (fabsf(y[k][j]) == INFINITY) y[k][j] = NAN;
            if (where[k] >= 0) m = fmaxf(m, largest(y[k]));
            if (storing && where[k] >= 0 && lives)
              keep(codes + static_cast<int64_t>(first_row + t - t0 + (k << log_groups) + grp) * p.ldo[kind], y[k], unit);
          }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        return m;
      };
      if (held && one) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
        top = joint ? of_team(all) : all;
      } else if (held) {
        for (int o = 1; o < 32; o <<= 1) {
          const float y = __shfl_down_sync(0xffffffffu, top, o);
          const int whose = __shfl_down_sync(0xffffffffu, opener, o);
          if (lane + o < 32 && whose == opener) top = fmaxf(top, y);
        }
        top = __shfl_sync(0xffffffffu, top, opener);
      }
      const bool alone = !held || __any_sync(0xffffffffu, top == INFINITY);
      if (joint && alone) {
        const int e = settle(of_team(by_itself(0, total, false, 0.f, 0)));
        if (row0 >= 0) by_itself(0, total, true, power_of(-e), row0 + skip);
        continue;
      }
      if (alone) {  // each of the batch's runs
#pragma unroll 1
        for (int storing = 0; storing < 2; ++storing) {
          const int e = storing ? settle(top) : 0;
          for (uint32_t left = opens; left != 0; left &= left - 1) {
            const int who = __ffs(left) - 1, after = left & (left - 1) ? __ffs(left & (left - 1)) - 1 : total;
            const int first = __shfl_sync(0xffffffffu, row, who);
            if (first < 0) continue;
            const float m = by_itself(who, after, storing, power_of(-__shfl_sync(0xffffffffu, e, who)), first);
            if (opener == who && !storing) top = m;
          }
        }
        continue;
      }
      const int e = settle(top);
      if (one) {
        const uint32_t counts = __ballot_sync(0xffffffffu, at >= 0);
        const float unit = power_of(-e);
        uint8_t* d = codes + static_cast<int64_t>(row0 + skip + grp) * p.ldo[kind];
#pragma unroll
        for (int f = 0; f < kRounds; ++f, d += p.ldo[kind] << log_groups) {
          if (f << log_groups >= total) break;
          if (row0 >= 0 && (counts >> ((f << log_groups) + grp) & 1u) && lives) keep(d, x[f], unit);
        }
      } else {
        const int live_row = at < 0 ? -1 : row;
#pragma unroll
        for (int f = 0; f < kRounds; ++f) {
          if (f << log_groups >= total) break;
          const int t = (f << log_groups) + grp;
          const int to = __shfl_sync(0xffffffffu, live_row, t & 31);
          const float unit = power_of(-__shfl_sync(0xffffffffu, e, t & 31));
          if (t < total && to >= 0 && lives) keep(codes + static_cast<int64_t>(to) * p.ldo[kind], x[f], unit);
        }
      }
    }
  }
}

template <bool F32, bool NORM, int HOW>
auto append8_of(int rot) {
  return rot == ROT_NONE ? append8_kernel<F32, NORM, ROT_NONE, HOW>
                         : (rot == ROT_OF_HALVES ? append8_kernel<F32, NORM, ROT_OF_HALVES, HOW> : append8_kernel<F32, NORM, ROT_OF_PAIRS, HOW>);
}
template <bool F32, bool NORM>
auto append8_of(int rot, int how) {
  if constexpr (!NORM)
    if (how == kByWarpTwo) return append8_of<F32, false, kByWarpTwo>(rot);
  return how == kByWarp ? append8_of<F32, NORM, kByWarp>(rot)
                        : (how == kByTeam ? append8_of<F32, NORM, kByTeam>(rot) : append8_of<F32, NORM, kWalked>(rot));
}

template <bool F32, bool NORM>
auto kernel_of(int rot) {
  return rot == ROT_NONE ? heads_kernel<F32, NORM, ROT_NONE>
                         : (rot == ROT_OF_HALVES ? heads_kernel<F32, NORM, ROT_OF_HALVES> : heads_kernel<F32, NORM, ROT_OF_PAIRS>);
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

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

lr_status check_map(const char* who, const lr_head_map* hm) {
  if (hm == nullptr) return bad(LR_ERR_INVALID_ARG, "%s: null head map", who);
  if (hm->head_dim <= 0 || hm->rot_dim < 0) return bad(LR_ERR_INVALID_ARG, "%s: non-positive head_dim or negative rot_dim", who);
  if (hm->head_dim % 64 || hm->head_dim > 256)
    return bad(LR_ERR_UNSUPPORTED, "%s: head_dim %d is not a multiple of 64 up to 256", who, hm->head_dim);
  if (hm->rot_dim % 16 || hm->rot_dim > hm->head_dim)
    return bad(LR_ERR_UNSUPPORTED, "%s: rot_dim %d is not a multiple of 16 up to head_dim", who, hm->rot_dim);
  if (hm->norm && !(hm->eps >= 0.f)) return bad(LR_ERR_INVALID_ARG, "%s: eps must be >= 0", who);
  if (!aligned16(hm->q_gain) || !aligned16(hm->k_gain))
    return bad(LR_ERR_INVALID_ARG, "%s: gains must be 16-byte aligned", who);
  if (hm->rot_dim > 0) {
    if (hm->rot_style != LR_ROT_HALF && hm->rot_style != LR_ROT_PAIR)
      return bad(LR_ERR_INVALID_ARG, "%s: bad rot_style", who);
    if (hm->cos_sin == nullptr || !aligned16(hm->cos_sin) || hm->max_pos <= 0)
      return bad(LR_ERR_INVALID_ARG, "%s: cos_sin must be a 16-byte aligned table of max_pos > 0 positions", who);
  }
  return LR_OK;
}

// One of the tensors whose heads are read or written.
lr_status check_rows(const char* who, const char* name, const void* p, int64_t ld, int64_t width) {
  if (p == nullptr) return bad(LR_ERR_INVALID_ARG, "%s: null %s", who, name);
  if (!aligned16(p) || ld % 8 || ld < width)
    return bad(LR_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned with a leading dimension >= %lld that is a multiple of 8",
               who, name, static_cast<long long>(width));
  return LR_OK;
}

void set_map(HeadParams& p, const lr_head_map* hm) {
  p.head_dim = hm->head_dim;
  p.lanes = hm->head_dim <= 64 ? 8 : (hm->head_dim <= 128 ? 16 : 32);
  p.eps = hm->eps;
  p.gain[0] = static_cast<const uint16_t*>(hm->q_gain);
  p.gain[1] = static_cast<const uint16_t*>(hm->k_gain);
  p.rot_dim = hm->rot_dim;
  p.cos_sin = hm->cos_sin;
  p.max_pos = hm->max_pos;
}

int rot_of(const lr_head_map* hm) {
  return hm->rot_dim == 0 ? ROT_NONE : (hm->rot_style == LR_ROT_HALF ? ROT_OF_HALVES : ROT_OF_PAIRS);
}

// Cuts the rows' heads over warps; the CTAs that they take.
int64_t cut_heads(HeadParams& p, int cta_warps = kHeadWarps) {
  // Heads per warp: one a group while the rows do not fill the GPU (16 warps an
  // SM), then more, so that the angles are read once for them.  (4, 16 or 64 warps:
  // 256 fp32 rows of 64 heads 11, 10, 14 us, 500 rows 13, 12, 13.)
  const int groups = 32 / p.lanes;
  const int64_t want = static_cast<int64_t>(num_sms()) * 16;
  auto warps_of = [&](int kind) { return (p.heads[kind] + p.chunk - 1) / p.chunk; };
  for (p.chunk = groups;; p.chunk += groups) {
    p.warp_end[0] = warps_of(0);
    p.warp_end[1] = p.warp_end[0] + warps_of(1);
    p.row_warps = p.warp_end[1] + warps_of(2);
    if (p.chunk >= kFlight * groups * kMostRounds || static_cast<int64_t>(p.M) * p.row_warps <= want) break;
  }
  return (static_cast<int64_t>(p.M) * p.row_warps + cta_warps - 1) / cta_warps;
}

template <typename Params>
lr_status launch_warps(void (*kern)(Params), int64_t blocks, const Params& p, cudaStream_t s, int cta_warps = kHeadWarps) {
  if (blocks > 0x7FFFFFFF) return bad(LR_ERR_UNSUPPORTED, "heads: too many rows and heads for one launch");
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(cta_warps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  if (pdl_enabled()) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e != cudaSuccess) return cuda_fail(e, "heads");
  return LR_OK;
}

lr_status launch_heads(HeadParams& p, const lr_head_map* hm, lr_dtype in_dtype, cudaStream_t s) {
  set_map(p, hm);
  const int rot = rot_of(hm);
  auto kern = in_dtype == LR_F32 ? (hm->norm ? kernel_of<true, true>(rot) : kernel_of<true, false>(rot))
                                 : (hm->norm ? kernel_of<false, true>(rot) : kernel_of<false, false>(rot));
  return launch_warps(kern, cut_heads(p), p, s);
}

lr_status launch_append8(AppendParams& a, const lr_head_map* hm, lr_dtype in_dtype, cudaStream_t s) {
  HeadParams& p = a.h;
  set_map(p, hm);
  const int32_t kv = p.heads[1];
  int64_t q_blocks = 0;
  if (p.heads[0] > 0) {  // the queries are cut as by themselves
    p.heads[1] = p.heads[2] = 0;
    q_blocks = cut_heads(p, kAppendWarps);
    p.heads[1] = p.heads[2] = kv;
  }
  // Tokens that a warp looks at for runs: more only while enough warps remain.
  a.hold = kRounds * (32 / p.lanes);
  int how = a.block_rows <= a.hold ? kByWarp : (a.block_rows <= kAppendWarps * a.hold ? kByTeam : kWalked);
  const int64_t each = how == kByTeam ? 1 : kAppendWarps;  // windows of a CTA
  const int64_t want = static_cast<int64_t>(num_sms()) * 4 * each;
  const int most = how == kByTeam ? 62 : 16;
  for (a.window = how == kByTeam ? kAppendWarps : 1; a.window < most && (static_cast<int64_t>(p.M) / (2 * a.window)) * 2 * kv >= want;) a.window *= 2;
  a.window = a.window < most ? a.window : most;
  const int64_t windows = (static_cast<int64_t>(p.M) + a.window - 1) / a.window;
  // Two heads a warp share what it finds out about its rows, where enough warps remain: 4099 rows
  // of 32 + 32 heads 41 us, so 37.5.  Not with norms, whose gains and sums take the registers
  // (16000 rows of 32 + 32 heads 171, so 174).
  if (how == kByWarp && !hm->norm && windows * 2 * ((kv + 1) / 2) >= want) how = kByWarpTwo;
  const int64_t blocks = (windows * 2 * (how == kByWarpTwo ? (kv + 1) / 2 : kv) + each - 1) / each;
  if (q_blocks + blocks > 0x7FFFFFFF / kAppendWarps) return bad(LR_ERR_UNSUPPORTED, "heads: too many rows and heads for one launch");
  a.q_blocks = static_cast<int32_t>(q_blocks);
  const int rot = rot_of(hm);
  auto kern = in_dtype == LR_F32 ? (hm->norm ? append8_of<true, true>(rot, how) : append8_of<true, false>(rot, how))
                                 : (hm->norm ? append8_of<false, true>(rot, how) : append8_of<false, false>(rot, how));
  return launch_warps(kern, q_blocks + blocks, a, s, kAppendWarps);
}

lr_status check_common(const char* who, lr_dtype in_dtype, int64_t M, const int32_t* pos, const lr_head_map* hm,
                       int32_t n_heads, int32_t n_kv_heads) {
  lr_status st = check_map(who, hm);
  if (st != LR_OK) return st;
  if (in_dtype != LR_BF16 && in_dtype != LR_F32) return bad(LR_ERR_INVALID_ARG, "%s: bad input dtype", who);
  if (n_heads < 0 || n_kv_heads < 0) return bad(LR_ERR_INVALID_ARG, "%s: negative head count", who);
  if (n_heads > 65536 || n_kv_heads > 65536) return bad(LR_ERR_UNSUPPORTED, "%s: more than 65536 heads", who);
  if (M < 0 || M > 0x7FFFFFFF) return bad(LR_ERR_INVALID_ARG, "%s: bad M", who);
  if (M > 0 && hm->rot_dim > 0 && pos == nullptr) return bad(LR_ERR_INVALID_ARG, "%s: null positions", who);
  return LR_OK;
}

}  // namespace

lr_status check_kv_cache(const char* who, const lr_kv_cache* c) {
  if (c == nullptr) return bad(LR_ERR_INVALID_ARG, "%s: null cache", who);
  if (c->n_kv_heads <= 0 || c->head_dim <= 0 || c->block_rows <= 0 || c->pool_blocks < 0)
    return bad(LR_ERR_INVALID_ARG, "%s: bad cache sizes", who);
  if (c->pool_blocks > 0x7FFFFFFF / c->block_rows)
    return bad(LR_ERR_INVALID_ARG, "%s: the cache's rows overflow int32", who);
  const int64_t width = static_cast<int64_t>(c->n_kv_heads) * c->head_dim;
  lr_status st = check_rows(who, "K pool", c->k, c->ld, width);
  if (st != LR_OK) return st;
  return check_rows(who, "V pool", c->v, c->ld, width);
}

lr_status check_scales(const char* who, const lr_kv_cache* c, const float* k_scale, const float* v_scale) {
  if (c->ld % 16) return bad(LR_ERR_INVALID_ARG, "%s: the 8-bit pools' leading dimension must be a multiple of 16", who);
  auto bad_scale = [](const float* p) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & 3u) != 0; };
  if (bad_scale(k_scale) || bad_scale(v_scale))
    return bad(LR_ERR_INVALID_ARG, "%s: the scales of an 8-bit cache must be 4-byte aligned device arrays", who);
  return LR_OK;
}

lr_status check_append(const void* k, int64_t ldk, const void* v, int64_t ldv, const void* q, int64_t ldq,
                       int32_t n_heads, lr_dtype in_dtype, int64_t M, const int32_t* pos, const int32_t* rows,
                       const lr_head_map* hm, const lr_kv_cache* cache, const void* q_out, int64_t ldqo, const char* who) {
  lr_status st = check_kv_cache(who, cache);
  if (st != LR_OK) return st;
  st = check_common(who, in_dtype, M, pos, hm, n_heads, cache->n_kv_heads);
  if (st != LR_OK) return st;
  if (hm->head_dim != cache->head_dim) return bad(LR_ERR_INVALID_ARG, "%s: the head map's head_dim is not the cache's", who);
  if (M == 0) return LR_OK;
  if (rows == nullptr) return bad(LR_ERR_INVALID_ARG, "%s: null rows", who);
  const int64_t wk = static_cast<int64_t>(cache->n_kv_heads) * hm->head_dim;
  if ((st = check_rows(who, "k", k, ldk, wk)) != LR_OK) return st;
  if ((st = check_rows(who, "v", v, ldv, wk)) != LR_OK) return st;
  if (n_heads > 0) {
    const int64_t wq = static_cast<int64_t>(n_heads) * hm->head_dim;
    if ((st = check_rows(who, "q", q, ldq, wq)) != LR_OK) return st;
    if ((st = check_rows(who, "q_out", q_out, ldqo, wq)) != LR_OK) return st;
    if (q == q_out && (in_dtype != LR_BF16 || ldq != ldqo))
      return bad(LR_ERR_INVALID_ARG, "%s: in place needs bf16 and one leading dimension", who);
  }
  return LR_OK;
}

}  // namespace lr

using namespace lr;

extern "C" {

lr_status lr_rope_table(int64_t max_pos, int32_t rot_dim, double theta, float* out) {
  if (max_pos < 0 || rot_dim <= 0 || rot_dim % 2 || !(theta > 0) || std::isinf(theta))
    return bad(LR_ERR_INVALID_ARG, "rope_table: max_pos >= 0, an even rot_dim > 0 and a finite theta > 0 are wanted");
  if (max_pos > 0 && out == nullptr) return bad(LR_ERR_INVALID_ARG, "rope_table: null output");
  const int half = rot_dim / 2;
  for (int i = 0; i < half; ++i) {
    const double f = std::pow(theta, -2.0 * i / rot_dim);
    for (int64_t p = 0; p < max_pos; ++p) {
      out[p * rot_dim + i] = static_cast<float>(std::cos(static_cast<double>(p) * f));
      out[p * rot_dim + half + i] = static_cast<float>(std::sin(static_cast<double>(p) * f));
    }
  }
  return LR_OK;
}

lr_status lr_qk_norm_rope(const void* q, int64_t ldq, int32_t n_heads, const void* k, int64_t ldk,
                          int32_t n_kv_heads, lr_dtype in_dtype, int64_t M, const int32_t* pos,
                          const int32_t* n_active, const lr_head_map* hm, void* q_out, int64_t ldqo,
                          void* k_out, int64_t ldko, int32_t* dev_status, lr_stream s) {
  const char* who = "qk_norm_rope";
  lr_status st = check_common(who, in_dtype, M, pos, hm, n_heads, n_kv_heads);
  if (st != LR_OK) return st;
  if (M == 0 || n_heads + n_kv_heads == 0) return LR_OK;
  const int64_t wq = static_cast<int64_t>(n_heads) * hm->head_dim, wk = static_cast<int64_t>(n_kv_heads) * hm->head_dim;
  if (n_heads > 0) {
    if ((st = check_rows(who, "q", q, ldq, wq)) != LR_OK) return st;
    if ((st = check_rows(who, "q_out", q_out, ldqo, wq)) != LR_OK) return st;
    if (q == q_out && (in_dtype != LR_BF16 || ldq != ldqo))
      return bad(LR_ERR_INVALID_ARG, "%s: in place needs bf16 and one leading dimension", who);
  }
  if (n_kv_heads > 0) {
    if ((st = check_rows(who, "k", k, ldk, wk)) != LR_OK) return st;
    if ((st = check_rows(who, "k_out", k_out, ldko, wk)) != LR_OK) return st;
    if (k == k_out && (in_dtype != LR_BF16 || ldk != ldko))
      return bad(LR_ERR_INVALID_ARG, "%s: in place needs bf16 and one leading dimension", who);
  }
  HeadParams p;
  memset(&p, 0, sizeof(p));
  p.src[0] = q, p.src[1] = k;
  p.ld[0] = ldq, p.ld[1] = ldk;
  p.dst[0] = q_out, p.dst[1] = k_out;
  p.ldo[0] = ldqo, p.ldo[1] = ldko;
  p.heads[0] = n_heads, p.heads[1] = n_kv_heads;
  p.pos = pos;
  p.n_active = n_active;
  p.M = static_cast<int32_t>(M);
  p.status = dev_status;
  return launch_heads(p, hm, in_dtype, reinterpret_cast<cudaStream_t>(s));
}

lr_status lr_kv_append(const void* k, int64_t ldk, const void* v, int64_t ldv, const void* q, int64_t ldq,
                       int32_t n_heads, lr_dtype in_dtype, int64_t M, const int32_t* pos,
                       const int32_t* rows, const int32_t* n_active, const lr_head_map* hm,
                       const lr_kv_cache* cache, void* q_out, int64_t ldqo, int32_t* dev_status, lr_stream s) {
  lr_status st = check_append(k, ldk, v, ldv, q, ldq, n_heads, in_dtype, M, pos, rows, hm, cache, q_out, ldqo);
  if (st != LR_OK || M == 0) return st;
  HeadParams p;
  memset(&p, 0, sizeof(p));
  p.src[0] = q, p.src[1] = k, p.src[2] = v;
  p.ld[0] = ldq, p.ld[1] = ldk, p.ld[2] = ldv;
  p.dst[0] = q_out, p.dst[1] = cache->k, p.dst[2] = cache->v;
  p.ldo[0] = ldqo, p.ldo[1] = p.ldo[2] = cache->ld;
  p.heads[0] = n_heads, p.heads[1] = p.heads[2] = cache->n_kv_heads;
  p.pos = pos;
  p.rows = rows;
  p.pool_rows = cache->pool_blocks * cache->block_rows;
  p.n_active = n_active;
  p.M = static_cast<int32_t>(M);
  p.status = dev_status;
  return launch_heads(p, hm, in_dtype, reinterpret_cast<cudaStream_t>(s));
}

lr_status lr_kv_append8(const void* k, int64_t ldk, const void* v, int64_t ldv, const void* q, int64_t ldq,
                        int32_t n_heads, lr_dtype in_dtype, int64_t M, const int32_t* pos,
                        const int32_t* rows, const int32_t* n_active, const lr_head_map* hm,
                        const lr_kv_cache8* cache, void* q_out, int64_t ldqo, int32_t* dev_status, lr_stream s) {
  const char* who = "kv_append8";
  if (cache == nullptr) return bad(LR_ERR_INVALID_ARG, "%s: null cache", who);
  const lr_kv_cache& c = cache->pages;
  lr_status st = check_append(k, ldk, v, ldv, q, ldq, n_heads, in_dtype, M, pos, rows, hm, &c, q_out, ldqo, who);
  if (st == LR_OK) st = check_scales(who, &c, cache->k_scale, cache->v_scale);
  if (st != LR_OK || M == 0) return st;
  AppendParams a;
  memset(&a, 0, sizeof(a));
  HeadParams& p = a.h;
  p.src[0] = q, p.src[1] = k, p.src[2] = v;
  p.ld[0] = ldq, p.ld[1] = ldk, p.ld[2] = ldv;
  p.dst[0] = q_out, p.dst[1] = c.k, p.dst[2] = c.v;
  p.ldo[0] = ldqo, p.ldo[1] = p.ldo[2] = c.ld;
  p.heads[0] = n_heads, p.heads[1] = p.heads[2] = c.n_kv_heads;
  p.pos = pos;
  p.rows = rows;
  p.pool_rows = c.pool_blocks * c.block_rows;
  p.n_active = n_active;
  p.M = static_cast<int32_t>(M);
  p.status = dev_status;
  a.scale[0] = cache->k_scale, a.scale[1] = cache->v_scale;
  a.block_rows = c.block_rows;
  a.block_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (c.block_rows == 1 << i) a.block_shift = i;
  return launch_append8(a, hm, in_dtype, reinterpret_cast<cudaStream_t>(s));
}

}  // extern "C"
