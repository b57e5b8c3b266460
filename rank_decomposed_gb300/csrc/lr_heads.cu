// Norms of query and key heads with the position rotation in the same pass,
// and the append of keys and values to a paged cache with both on the way.
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

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

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
__global__ void __launch_bounds__(kHeadWarps * 32, kHeadCtas) heads_kernel(const __grid_constant__ HeadParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * kHeadWarps + (threadIdx.x >> 5);
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

lr_status launch_heads(HeadParams& p, const lr_head_map* hm, lr_dtype in_dtype, cudaStream_t s) {
  p.head_dim = hm->head_dim;
  p.lanes = hm->head_dim <= 64 ? 8 : (hm->head_dim <= 128 ? 16 : 32);
  p.eps = hm->eps;
  p.gain[0] = static_cast<const uint16_t*>(hm->q_gain);
  p.gain[1] = static_cast<const uint16_t*>(hm->k_gain);
  p.rot_dim = hm->rot_dim;
  p.cos_sin = hm->cos_sin;
  p.max_pos = hm->max_pos;
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
  const int64_t blocks = (static_cast<int64_t>(p.M) * p.row_warps + kHeadWarps - 1) / kHeadWarps;
  if (blocks > 0x7FFFFFFF) return bad(LR_ERR_UNSUPPORTED, "heads: too many rows and heads for one launch");
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kHeadWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  if (pdl_enabled()) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  const int rot = hm->rot_dim == 0 ? ROT_NONE : (hm->rot_style == LR_ROT_HALF ? ROT_OF_HALVES : ROT_OF_PAIRS);
  auto kern = in_dtype == LR_F32 ? (hm->norm ? kernel_of<true, true>(rot) : kernel_of<true, false>(rot))
                                 : (hm->norm ? kernel_of<false, true>(rot) : kernel_of<false, false>(rot));
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e != cudaSuccess) return cuda_fail(e, "heads");
  return LR_OK;
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

lr_status check_append(const void* k, int64_t ldk, const void* v, int64_t ldv, const void* q, int64_t ldq,
                       int32_t n_heads, lr_dtype in_dtype, int64_t M, const int32_t* pos, const int32_t* rows,
                       const lr_head_map* hm, const lr_kv_cache* cache, const void* q_out, int64_t ldqo) {
  const char* who = "kv_append";
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

}  // extern "C"
