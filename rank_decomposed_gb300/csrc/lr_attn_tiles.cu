// Attention of many query rows on the 5th-generation tensor cores: the shared
// prefix against all rows of the batch, and whole ragged turns (prefix and own
// tokens in one pass).
//
//   S = Q K^T;  P = 2^(scale log2(e) S - m);  O = sum P V;  l = sum P;  out = O / l
// in one walk over the keys, with the running maximum m of each row.
//
// Rows are query rows times the G query heads of one key head: a tile is
// floor(128 / G) query rows, so its G heads share every key that is loaded.
// A CTA holds two row tiles, or, when there are rows for one tile only, one row
// tile against alternate keys twice; either way two independent softmax rings
// keep the tensor pipe busy while the other one's powers are computed.  It walks
// steps, one key tile of 128 keys a ring; the steps of a row tile pair are cut
// into `slots` ranges, one a CTA, and a second kernel joins their results.
//   whole turns: the tiles are of one sequence's query rows; its prefix and own
//     key tiles serve both rings.
//   packed rows: the tiles are of any query rows of the batch, 16 or more
//     sequences of one row each as a rule.  A prefix tile serves both rings; the
//     own tokens of the sequences follow in tiles of the ring that holds their
//     rows, each sequence's in groups of 16 keys one after another, so that a
//     tile holds up to eight sequences.  The product of a group's 16 keys has the
//     output lanes of all other sequences' rows disabled: no sequence's values,
//     NaN or infinite as they may be, reach another's.  (A tile for each
//     sequence's last tokens instead: 100 sequences of 56 heads with up to 50 own
//     tokens 110 us, so 41.  The own tokens in a second kernel beside this one:
//     64 sequences behind 8192 tokens 62 us, then, in one pass, 48.)
// A sequence is taken whole when its rows times G may pass 64: 40 turns of 4, 8,
// 16, 32 rows and G = 8 behind 2000 tokens take 75, 75, 77, 111 us whole and 40,
// 50, 87, 128 us packed; 20 of 16, 40, 64, 100 rows and G = 1 120, 121, 122, 127
// whole and 52, 63, 103, 116 packed.
//   warps 0-3, 4-7  softmax of ring 0 and 1, one row per thread;
//   warps 8-11      load K and V tiles of 128 keys (three warps: 250 us for
//                   ragged turns of 33 to 300 rows behind 4096 tokens, four 237);
//   warp 14         looks the tiles' pages up, four tiles in one trip to memory
//                   and some tiles ahead of the loads: a loading warp that waited
//                   for a page's number would load nothing;
//   warp 13         hands landed tiles on: the copies write shared memory by the
//                   generic proxy and the products read it by the async one, and
//                   the fence between the two takes some 400 cycles, which the
//                   issuing warp has not;
//   warp 12         tcgen05.mma issue: S = Q K^T (Q, K in shared memory) and
//                   O += P V (P in TMEM, where the softmax warps put it over
//                   S; V in shared memory as it lies in the cache, keys along
//                   the reduction, which is the operand's MN-major form).  A
//                   second issuing warp, one a ring, took 320 us for the ragged
//                   turns instead of 243, and 275 instead of 251 with the turns
//                   handed from one to the other.
// The tiles come by 16-byte asynchronous copies into the layout of the 128-byte
// swizzle.  A page may be 16 rows long and a TMA box cannot cross one: sixteen
// boxes a tile took 1340 cycles from L2, where one 128-row box takes 630, and
// the products of two rings take 2048 for two tiles.  The copies also fill with
// zeros where no token lies, so that whatever a last page holds behind its
// tokens stays out (0 * NaN would be NaN).
// P is handed on in halves of its keys (in one piece: ragged turns 267 us, 253),
// and the products themselves release the tiles (the softmax warps instead, once
// they see the next scores: 259).
// The order of the products is  S0 S1 | PV0 S0' PV1 S1' | ...: S0' needs
// softmax 0 to be through with S0 (its P has been consumed by PV0, issued just
// before), and runs while softmax 1 works.
//
// The running maximum moves only when it would grow by more than 2^8 in the
// powers: until then powers up to 256 are summed against the older maximum
// (exact in fp32 and in bf16's range), and O in TMEM needs no rescaling.
//
// Bound: a step's four products of 128 x 128 x 128 are 2048 cycles of the tensor
// pipe (heads of 128), and a step takes some 2950, by latency: a ring's scores are
// seen 250 cycles after their last product, loaded 200 later, their maximum known
// after 400 more and the first half of P after another 400 (512 cycles of each
// softmax are the exponentials, and two warps share a scheduler), and every wait
// of the issuing warp queues behind the products that it issued.  No resource is
// full by itself: the ragged turns take 250 us, and in copies made for timing 248
// with an eighth of the loads, 242 without the exponentials, 234 with half of the
// products of S.  A CTA's first score comes some 5
// us after its start (lengths, pages, keys: three trips to memory one after
// another) and its results take 4 us more after its last product.  Measured, with
// heads of 128 and 64 over 8: 12 ragged turns 247 us (tensor floor 143), 64
// sequences behind 8192 tokens 46 us with the join (bytes 15), 5 behind 131000 92
// us (bytes 80: 87 % of the copy rate).
#include <cuda_bf16.h>

#include <cmath>
#include <cstring>

#include "lr_attn.h"
#include "lr_ptx.cuh"

namespace lr {
namespace {

constexpr int kThreads = 512;        // 8 softmax warps, 4 producers, an MMA issuer, a relay, the pages, one idle
constexpr int kMmaWarp = 12, kRelayWarp = 13, kPageWarp = 14;
constexpr int kLooked = 6;           // tiles whose pages are known, from their K load to their V product
// Registers: the launch gives 128 a thread; the softmax warps hold a row of 128
// scores and take what the others leave (256 * 208 + 128 * 40 + 128 * 56 = 512 * 128).
constexpr int kRegsSoftmax = 208, kRegsLoad = 40, kRegsIssue = 56;
constexpr int kKeys = 128;           // keys per tile
constexpr int kPage = 16;            // rows of a page, at least
constexpr uint32_t kTmemCols = 512;  // S0, S1 (128 each), O0, O1 (head_dim each)
constexpr float kSlack = 8.f;

template <int HD>
struct Shape {
  static constexpr int kChunks = HD / 64;              // 128-byte swizzled columns of a tile
  static constexpr int kChunkBytes = 128 * 128;        // 128 rows of 64 bf16
  static constexpr int kTileBytes = kChunks * kChunkBytes;
  static constexpr int kSlots = HD == 128 ? 5 : 10;    // ring of K and V tiles
  static constexpr int kTail = 3 * 1024;                  // barriers and the lists of own tokens
  static constexpr int kSmem = (2 + kSlots) * kTileBytes + kTail;
};

struct TileParams {
  AttnParams p;
  int32_t mt;         // query rows per tile
  int32_t pairs;      // tile pairs per sequence (whole), or in all
  int32_t slots;
  int32_t direct;     // one key range: results go straight to out
  int32_t two;        // two slots a key range (somewhere a row tile is alone in its CTA)
  int32_t stall;      // fault-injection hook: the producer issues nothing
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Sixteen bytes, or sixteen zeros (src is not read then).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool live) {
  const int n = live ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// Arrives on `bar` (which counts this thread) once its copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

#define LR_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define LR_I8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])

// 32 lanes x 32 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
      "%29,%30,%31}, [%32];"
      : LR_R8(r, 0), LR_R8(r, 8), LR_R8(r, 16), LR_R8(r, 24)
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
      "%29,%30,%31};" ::LR_I8(r, 0),
      LR_I8(r, 8), LR_I8(r, 16), LR_I8(r, 24), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::LR_I8(r, 0),
      LR_I8(r, 8), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The products of one tile pair, each issued as one block: eight or four
// instructions whose operands differ by constants.  The issuing warp shares its
// scheduler with softmax warps, and every instruction between two products
// delays the tensor pipe: with one lane of a divergent warp computing 64-bit
// descriptors, a pair of 128 x 128 x 128 products took 1630 cycles beside
// warps that issue all the time; so, from a converged warp, it takes 1130 (1030
// alone; the pipe needs 1024).
//
// Descriptor words: a shared-memory tile with the 128-byte swizzle has the low
// word address / 16 | (leading offset / 16) << 16 and this high word (stride
// between groups of eight rows 1024 bytes, version 1, 128-byte swizzle).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lead_bytes) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lead_bytes >> 4) << 16);
}

// S = Q K^T over one chunk of 64 columns of the head, both K-major: four
// products of 16 columns (32 bytes) each.  acc: add to D from the first on.
__device__ __forceinline__ void mma_qk_chunk(uint32_t d, uint32_t q_lo, uint32_t k_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, t;\n\t.reg .b64 x, y;\n\t.reg .b32 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "mov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t"
      "add.u32 a, %1, 2;\n\tadd.u32 b, %2, 2;\n\tmov.b64 x, {a, %3};\n\tmov.b64 y, {b, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, t;\n\t"
      "add.u32 a, %1, 4;\n\tadd.u32 b, %2, 4;\n\tmov.b64 x, {a, %3};\n\tmov.b64 y, {b, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, t;\n\t"
      "add.u32 a, %1, 6;\n\tadd.u32 b, %2, 6;\n\tmov.b64 x, {a, %3};\n\tmov.b64 y, {b, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, t;\n\t}" ::"r"(d),
      "r"(q_lo), "r"(k_lo), "r"(kDescHi), "r"(idesc), "r"(acc)
      : "memory");
}

// O += P V over 64 keys: P in TMEM (two keys a column), V with the keys along
// the reduction, in steps of 16 keys (2048 bytes; element (key, column) of
// chunks [128 keys][64 columns], columns contiguous: MN-major; groups of eight
// keys 1024 bytes apart, chunks of columns the leading offset).
__device__ __forceinline__ void mma_pv_half(uint32_t d, uint32_t p_at, uint32_t v_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, t;\n\t.reg .b64 y;\n\t.reg .b32 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "mov.b64 y, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t"
      "add.u32 a, %1, 8;\n\tadd.u32 b, %2, 128;\n\tmov.b64 y, {b, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %4, t;\n\t"
      "add.u32 a, %1, 16;\n\tadd.u32 b, %2, 256;\n\tmov.b64 y, {b, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %4, t;\n\t"
      "add.u32 a, %1, 24;\n\tadd.u32 b, %2, 384;\n\tmov.b64 y, {b, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %4, t;\n\t}" ::"r"(d),
      "r"(p_at), "r"(v_lo), "r"(kDescHi), "r"(idesc), "r"(acc)
      : "memory");
}

// The same, always added to O, with the output lanes of others[k]'s set bits left
// alone in the product of the k-th 16 keys.
__device__ __forceinline__ void mma_pv_half_some(uint32_t d, uint32_t p_at, uint32_t v_lo, uint32_t idesc,
                                                 const uint4* others) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint4 off = others[k];
    asm volatile(
        "{\n\t.reg .pred t;\n\t.reg .b64 y;\n\t"
        "setp.eq.b32 t, 0, 0;\n\t"
        "mov.b64 y, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, {%5, %6, %7, %8}, t;\n\t}" ::"r"(d),
        "r"(p_at + k * 8), "r"(v_lo + k * 128), "r"(kDescHi), "r"(idesc), "r"(off.x), "r"(off.y), "r"(off.z), "r"(off.w)
        : "memory");
  }
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_lane() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// 3-D tiled load, as tma_load_2d.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y,
                                            int32_t z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}

template <int N>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_fewer() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Two fp32 values as one operand of the packed instructions.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// What lies behind the tiles in shared memory.
struct __align__(16) Tail {
  uint64_t q_full;
  uint64_t landed[10], full[10], empty[10];
  uint64_t s_full[2], p_ready[2][2], o_done[2];  // P is handed on in two halves of its keys
  uint64_t drain;
  // Tiles in the order of their K loads: of each group of 16 keys the first pool
  // row (-1: none, zeros), the keys that hold tokens, and for own tokens of packed
  // rows the output lanes of other sequences (row r: bit r mod 32 of word r / 32).
  uint64_t looked_up[kLooked], done_with[kLooked];
  uint4 others[kLooked][8];
  int rows[kLooked][8];
  uint8_t live[kLooked][8];
  uint32_t tmem_base;
  int abort;
  int warp_sum[8];
  // Packed rows, per query row of each tile: its sequence (-1: none; counted from
  // the CTA's first row without q_start), and the groups of 16 own keys of the
  // sequences up to it, each sequence's counted at its last row in the tile.
  int16_t seq[2][128];
  int groups[2][128];
};
static_assert(sizeof(Tail) <= Shape<64>::kTail, "the tail of shared memory");

template <int HD, bool WHOLE>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tiles_kernel(const __grid_constant__ TileParams a, const __grid_constant__ CUtensorMap map_q) {
  using S = Shape<HD>;
  constexpr int kSlots = S::kSlots;
  extern __shared__ __align__(1024) uint8_t smem[];
  const AttnParams& p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* q_sm = smem;                            // two row tiles
  uint8_t* ring = smem + 2 * S::kTileBytes;
  Tail& bars = *reinterpret_cast<Tail*>(ring + kSlots * S::kTileBytes);
  int& abort_sh = bars.abort;
  if (smem_u32(smem) & 1023u) {  // the swizzle's pattern needs it; there is no room to round up
    if (threadIdx.x == 0) report_status(p.status, LR_ERR_UNSUPPORTED);
    return;
  }

  if (threadIdx.x == 0) {
    mbar_init(&bars.q_full, 1);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&bars.landed[s], 128);  // every producer thread's copies
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars.s_full[t], 1);
      mbar_init(&bars.p_ready[t][0], 4);
      mbar_init(&bars.p_ready[t][1], 4);
      mbar_init(&bars.o_done[t], 1);
    }
    mbar_init(&bars.drain, 1);
    for (int e = 0; e < kLooked; ++e) {
      mbar_init(&bars.looked_up[e], 1);
      mbar_init(&bars.done_with[e], WHOLE ? 4 : 5);  // the producer warps, and the issuer for the lanes
    }
    abort_sh = 0;
    fence_mbar_init();
  }
  pdl_launch_dependents();
  pdl_wait();

  // ---- this CTA's rows and keys
  // CTAs in the order of their work, the most first: the last rows of turns see the
  // most keys (a prompt of 4000 rows with 64 heads over 8 271 us, 302 with the first
  // rows first), key heads side by side.
  const int kvh = blockIdx.x % p.n_kv, split = blockIdx.z, G = p.group;
  const int item = blockIdx.x / p.n_kv;
  const int seq_of = WHOLE ? item % p.n_seq : 0;
  const int pair = WHOLE ? a.pairs - 1 - item / p.n_seq : item;
  const bool tell = threadIdx.x == 0 && kvh == 0 && split == 0;
  const int prefix_len = p.prefix_len != nullptr ? *p.prefix_len : 0;  // on its way while the lists are made
  int q0 = 0, nq = p.M, n_seen = 0, own = 0, mrel;
  const int32_t* own_pages = nullptr;
  if (WHOLE) {
    const int b = seq_of;
    const SeqView v = seq_view(p, b, tell && pair == 0);
    q0 = v.q0, nq = v.nq, n_seen = v.n, own = v.len;
    own_pages = p.block_table + static_cast<int64_t>(b) * p.blocks_per_seq;
  }
  mrel = pair * 2 * a.mt;
  if (WHOLE && a.direct && kvh == 0 && threadIdx.x < 32 * 8) {  // rows of no sequence: zeros
    const int from = p.q_start ? p.q_start[0] : 0, to = p.q_start ? p.q_start[p.n_seq] : p.n_seq;
    const int esz = p.out_f32 ? 4 : 2;
    const int vecs = p.n_heads * HD * esz / 16;
    for (int m = item; m < p.M; m += gridDim.x / p.n_kv)
      if (m < from || m >= to) {
        uint4* row = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + m * p.ldo * esz);
        for (int i = threadIdx.x; i < vecs; i += 32 * 8) row[i] = make_uint4(0, 0, 0, 0);
      }
  }
  if (tell && item == 0) prefix_rows(p, prefix_len, true);
  if (nq - mrel <= 0) return;
  // query rows of each tile
  const int rows0 = nq - mrel < a.mt ? nq - mrel : a.mt;
  const int left = nq - mrel - a.mt;
  const int rows1 = left < 0 ? 0 : (left < a.mt ? left : a.mt);
  const bool dual = rows1 == 0;  // one row tile, both rings
  // own tokens that a tile's last row sees
  auto seen = [&](int m) {
    const int v = own - n_seen + m + 1;
    return v < 0 ? 0 : v;
  };
  // own key tiles of each ring's rows: 128 tokens of the sequence, or eight
  // groups of 16 of the packed sequences, one after another
  const int first_seq = p.q_start == nullptr ? mrel : 0;
  int own0, own1, see = 0;
  if (WHOLE) {
    const int see0 = seen(mrel + rows0 - 1), see1 = dual ? 0 : seen(mrel + a.mt + rows1 - 1);
    see = see0 > see1 ? see0 : see1;
    own0 = (see0 + kKeys - 1) / kKeys, own1 = (see1 + kKeys - 1) / kKeys;
  } else {
    if (threadIdx.x < 256) (&bars.seq[0][0])[threadIdx.x] = -1;
    __syncthreads();
    const int m_end = mrel + rows0 + rows1;
    if (p.q_start == nullptr) {
      const int m = mrel + static_cast<int>(threadIdx.x);
      if (m < m_end && m < p.n_seq) bars.seq[m - mrel >= a.mt][(m - mrel) % a.mt] = static_cast<int16_t>(m - mrel);
    } else {
      for (int b = threadIdx.x; b < p.n_seq; b += kThreads) {
        const int from = p.q_start[b], to = p.q_start[b + 1];
        if ((from < 0 || to > p.M || to < from || to - from > p.max_q) && kvh == 0 && split == 0)
          report_status(p.status, LR_ERR_INDEX_RANGE);
        for (int m = from > mrel ? from : mrel; m < to && m < m_end; ++m)
          bars.seq[m - mrel >= a.mt][(m - mrel) % a.mt] = static_cast<int16_t>(b);
      }
    }
    __syncthreads();
    int sum = 0;
    if (threadIdx.x < 256) {
      const int t = threadIdx.x >> 7, j = threadIdx.x & 127, rows = t ? rows1 : rows0;
      const int b = bars.seq[t][j];
      if (j < rows && b >= 0 && (j == rows - 1 || bars.seq[t][j + 1] != b)) {
        const SeqView v = seq_view(p, first_seq + b, kvh == 0 && split == 0);
        int vis = v.len - v.n + (mrel + t * a.mt + j - v.q0) + 1;
        vis = vis > v.len ? v.len : vis;
        if (vis > 0) sum = (vis + kPage - 1) / kPage;
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
      }
      if (lane == 31) bars.warp_sum[warp] = sum;
    }
    __syncthreads();
    if (threadIdx.x < 256) {
      for (int w = warp & ~3; w < warp; ++w) sum += bars.warp_sum[w];
      (&bars.groups[0][0])[threadIdx.x] = sum;
    }
    __syncthreads();
    own0 = (bars.groups[0][127] + 7) / 8, own1 = (bars.groups[1][127] + 7) / 8;
  }
  const int P = prefix_rows(p, prefix_len, false);
  const int np = (P + kKeys - 1) / kKeys;
  // Steps: step s is key tile s of both rings' lists (prefix tiles, then own
  // ones), or, with one row tile, tiles 2 s and 2 s + 1 of its list.
  const int list0 = np + own0, list1 = dual ? list0 : np + own1;
  const int e0 = dual ? (list0 + 1) >> 1 : list0, e1 = dual ? list0 >> 1 : list1;  // steps that ring 0, 1 take
  const int64_t steps = e0 > e1 ? e0 : e1;
  // The ranges are equal in time: a step of packed own tokens loads a tile for
  // each ring and takes 5/4 of the time of a prefix step (64 sequences of up to 512
  // own tokens behind 8192 shared: 57, 52, 48, 48, 50 us with 3, 4, 5, 6, 8 quarters;
  // 200 of 300 behind 1000: 63, 59, 59, 56, 61; MHA of 1000 behind 4099: 73, 71, 71, 73, 77).
  const int64_t shared_steps = dual ? (np + 1) >> 1 : np;
  auto cut = [&](int i) {
    if (WHOLE) return static_cast<int>(steps * i / a.slots);
    const int at = static_cast<int>((4 * shared_steps + 5 * (steps - shared_steps)) * i / a.slots);  // quarters of a prefix step
    const int more = at - 4 * static_cast<int>(shared_steps);
    return more <= 0 ? at / 4 : static_cast<int>(shared_steps) + more / 5;
  };
  const int s_lo = cut(split), s_hi = cut(split + 1);
  auto of_range = [&](int e) {
    const int c = (e < s_hi ? e : s_hi) - s_lo;
    return c < 0 ? 0 : c;
  };
  const int n = s_hi - s_lo, n0 = of_range(e0), n1 = of_range(e1);  // n is the larger of the two
  // the first n_both of them have one key tile for both rings
  const int n_both = dual ? 0 : (WHOLE ? n : of_range(np));
  if (warp == kMmaWarp) {
    tmem_alloc(&bars.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;

  // softmax state of this thread's row
  const int ringi = warp >> 2;                     // 0, 1: softmax warps
  const int trow = threadIdx.x & 127;
  const int tile = dual ? 0 : (ringi & 1);
  const int live_rows = (tile ? rows1 : rows0) * G;
  const int my_n = (ringi & 1) ? n1 : n0;
  const int my_seq = WHOLE || trow / G >= a.mt ? -1 : bars.seq[tile][trow / G];
  // One row tile: its two rings' results are joined here, or have a slot each.
  const bool joins = dual && a.direct;
  float mref = -INFINITY, sum = 0.f;
  bool sees = false;  // a token at all
  float2* hand_ml = reinterpret_cast<float2*>(ring + 128 * (HD + 4) * 4);  // behind ring 1's numerators

  if (warp >= 8) {
    if (warp < kMmaWarp) {
      regs_fewer<kRegsLoad>();
      // ---------------------------------------------------- producers
      if (!a.stall && n > 0) {
        if (warp == 8 && lane == 0) {
          const uint32_t bytes = static_cast<uint32_t>(a.mt * G * 128 * S::kChunks) * (dual ? 1u : 2u);
          const uint64_t pol = l2_policy_evict_last();
          mbar_arrive_expect_tx(&bars.q_full, bytes);
          for (int t = 0; t < (dual ? 1 : 2); ++t)
            for (int c = 0; c < S::kChunks; ++c)
              tma_load_3d(q_sm + t * S::kTileBytes + c * S::kChunkBytes, &map_q, &bars.q_full, c * 64, kvh * G,
                          q0 + mrel + t * a.mt, pol);
        }
        // Each warp takes two groups of 16 keys of a tile; an instruction
        // copies kRows whole rows, and the swizzle repeats after kTurn of them.
        constexpr int kCols = HD / 8, kRows = 32 / kCols, kTurn = 8 / kRows;
        const int g0 = (warp - 8) * 2;
        const int r_in = lane / kCols, col = lane % kCols;
        const int64_t head_off = static_cast<int64_t>(kvh) * HD + col * 8;
        const int64_t step = static_cast<int64_t>(kRows) * p.ld;
        uint32_t dst0[kTurn];
#pragma unroll
        for (int j = 0; j < kTurn; ++j) {
          const int r = j * kRows + r_in;
          dst0[j] = smem_u32(ring) + (col >> 3) * S::kChunkBytes + (g0 * kPage + r) * 128 + (((col & 7) ^ r) << 4);
        }
        const uint32_t dst_row = smem_u32(ring) + (col >> 3) * S::kChunkBytes + (g0 * kPage + r_in) * 128;
        // In the order in which the products take the tiles: V of step i and K of
        // the next, ring by ring, or once for both.  One copy of the loading code
        // serves all (the loops stay loops): every warp role runs code of its own
        // and all of it has to stay in the instruction caches.
        int slot = 0, tile_no = 0;
        int at0 = 0, at1 = 0;  // the number of each ring's tile
        uint32_t phase = 1;
        bool ok = true;
#pragma unroll 1
        for (int i = -1; i < n && ok; ++i) {
#pragma unroll 1
          for (int x = 0; x < 4; ++x) {
            const int t = x >> 1, is_k = x & 1;
            const int j = i + is_k;  // the step that the tile is of
            if (j < 0 || !(j < n_both ? t == 0 : j < (t ? n1 : n0))) continue;
            int e = t ? at1 : at0;
            if (is_k) {
              e = tile_no++;
              if (t)
                at1 = e;
              else
                at0 = e;
              ok = mbar_wait(&bars.looked_up[e % kLooked], (e / kLooked) & 1, &abort_sh);
            }
            e %= kLooked;
            ok = __all_sync(0xffffffffu, ok && mbar_wait(&bars.empty[slot], phase, &abort_sh));
            if (!ok) break;
            const uint16_t* pool = is_k ? p.k : p.v;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int row = bars.rows[e][g0 + h];
              const int live = bars.live[e][g0 + h];
              const uint16_t* src = pool + static_cast<int64_t>((row < 0 ? 0 : row) + r_in) * p.ld + head_off;
              const uint32_t at = slot * S::kTileBytes + h * kPage * 128;
              if (live >= kPage) {
#pragma unroll
                for (int c = 0; c < kPage / kRows; ++c, src += step)
                  cp_async16(dst0[c % kTurn] + at + c / kTurn * 1024, src);
              } else {
#pragma unroll 1
                for (int c = 0; c < kPage / kRows; ++c, src += step)
                  cp_async16_or_zero(dst_row + at + c * kRows * 128 + (((c * kRows + r_in) ^ col) & 7) * 16, src,
                                     c * kRows + r_in < live);
              }
            }
            cp_async_arrive(&bars.landed[slot]);
            if (++slot == kSlots) slot = 0, phase ^= 1;
            if (!is_k) {
              __syncwarp();
              if (lane == 0) mbar_arrive(&bars.done_with[e]);
            }
          }
        }
        cp_async_wait_all();
        if (!ok && lane == 0) {
          abort_sh = 1;
          report_status(p.status, LR_ERR_TIMEOUT);
          if (warp == 8) mbar_wait(&bars.q_full, 0, nullptr);  // the copy in flight lands before the CTA ends
        }
      }
    } else {
      regs_fewer<kRegsIssue>();
      // K and V tiles of this CTA
      const int loads = 2 * (n_both + (n0 > n_both ? n0 - n_both : 0) + (n1 > n_both ? n1 - n_both : 0));
      if (warp == kPageWarp) {
        // ------------------------------------------------------- pages
        // Four tiles at a time, a lane for each group: a page's number takes a trip
        // to memory, and one for four tiles is soon enough.
        bool ok = true;
        int e = 0;
        uint32_t phase = 0;  // of the entries
        const int pairs = (n0 < n1 ? n0 : n1) - n_both;
        auto index_of = [&](int t) { return p.block_shift >= 0 ? t >> p.block_shift : t / p.block_rows; };
#pragma unroll 1
        for (int k0 = 0; k0 < (a.stall ? 0 : loads / 2) && ok; k0 += 4) {
          // the tiles in the order of their loads: those for both rings, then each
          // ring's in turn, then what one ring has more than the other
          const int k = k0 + (lane >> 3), g = lane & 7;
          int j = k, t = 0;
          if (k >= n_both) {
            const int x = k - n_both;
            j = n_both + (x < 2 * pairs ? x >> 1 : x - pairs);
            t = x < 2 * pairs ? x & 1 : n1 > n0;
          }
          const int c = dual ? 2 * (s_lo + j) + t : s_lo + j;
          const int32_t* pages = p.prefix_blocks;
          int t0 = c * kKeys + g * kPage, limit = k < loads / 2 ? P : 0;
          int row = -1, live = 0;
          uint4 others = make_uint4(0, 0, 0, 0);
          if (WHOLE && c >= np && k < loads / 2) {
            pages = own_pages;
            t0 -= np * kKeys, limit = see;
          }
          if (!WHOLE && c >= np) {
            const int list = dual ? 0 : t;
            const int* groups = bars.groups[list];
            const int16_t* seq = bars.seq[list];
            const int group = (c - np) * 8 + g;
            limit = 0;
            others = make_uint4(~0u, ~0u, ~0u, ~0u);
            if (group < groups[127]) {
              int r = 0;  // the first row with more than `group` groups
#pragma unroll 1
              for (int half = 64; half > 0; half >>= 1)
                if (groups[r + half - 1] <= group) r += half;
              const int b = first_seq + seq[r];
              pages = p.block_table + static_cast<int64_t>(b) * p.blocks_per_seq;
              limit = p.lengths[b];
              t0 = (group - (r > 0 ? groups[r - 1] : 0)) * kPage;
              int from = r;
              while (from > 0 && seq[from - 1] == seq[r]) --from;
              uint32_t off[4];
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const int lo = from * G - 32 * w, hi = (r + 1) * G - 32 * w;
                const uint32_t below = lo <= 0 ? 0u : (lo >= 32 ? ~0u : (1u << lo) - 1u);
                const uint32_t under = hi <= 0 ? 0u : (hi >= 32 ? ~0u : (1u << hi) - 1u);
                off[w] = ~(under & ~below);
              }
              others = make_uint4(off[0], off[1], off[2], off[3]);
            }
          }
          // A group in a list of packed rows holds a token: its page is asked for
          // beside the sequence's length.
          if (!WHOLE && c >= np ? others.x != ~0u || others.y != ~0u || others.z != ~0u || others.w != ~0u : t0 < limit) {
            const int x = index_of(t0);
            const int page = pages[x];
            live = limit < p.cap_own || c < np ? limit - t0 : p.cap_own - t0;
            live = live > kPage ? kPage : live;
            if (page < 0 || page >= p.pool_blocks) {  // reads as zeros
              report_status(p.status, LR_ERR_REMAP_RANGE);
              live = 0;
            } else {
              row = page * p.block_rows + (t0 - x * p.block_rows);
            }
          }
#pragma unroll 1
          for (int q = 0; q < 4 && k0 + q < loads / 2; ++q) {
            ok = __all_sync(0xffffffffu, mbar_wait(&bars.done_with[e], phase ^ 1u, &abort_sh));
            if (!ok) break;
            if (lane >> 3 == q) {
              bars.rows[e][g] = row;
              bars.live[e][g] = static_cast<uint8_t>(live);
              if (!WHOLE) bars.others[e][g] = others;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.looked_up[e]);
            if (++e == kLooked) e = 0, phase ^= 1u;
          }
        }
        if (!ok && lane == 0) {
          abort_sh = 1;
          report_status(p.status, LR_ERR_TIMEOUT);
        }
      } else if (warp == kRelayWarp) {
        bool ok = true;
#pragma unroll 1
        for (int l = 0; l < loads && ok; ++l) {
          ok = __all_sync(0xffffffffu, mbar_wait(&bars.landed[l % kSlots], (l / kSlots) & 1, &abort_sh));
          fence_proxy_async_smem();
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(&bars.full[l % kSlots]);
        }
        if (!ok && lane == 0) {
          abort_sh = 1;
          report_status(p.status, LR_ERR_TIMEOUT);
        }
      } else if (warp == kMmaWarp) {
        // ----------------------------------------------------------- MMA
        if (n > 0 && elect_lane()) {
          constexpr uint32_t kIdS = idesc_bf16_f32(128, kKeys);
          constexpr uint32_t kIdO = idesc_bf16_f32(128, HD) | (1u << 16);  // B is MN-major
          const uint32_t q_lo = desc_lo(smem_u32(q_sm), 16), r_k = desc_lo(smem_u32(ring), 16);
          const uint32_t r_v = desc_lo(smem_u32(ring), S::kChunkBytes);
          const uint32_t q_step = dual ? 0 : S::kTileBytes >> 4;
          bool ok = mbar_wait(&bars.q_full, 0, &abort_sh);
          // The ring's slots in the order of the loads: wait for the next one.
          int slot = -1;
          uint32_t phase = 0;
          auto next_slot = [&]() {
            if (++slot == kSlots) slot = 0, phase ^= 1;
            if (ok) ok = mbar_wait(&bars.full[slot], phase, &abort_sh);
            tc_fence_after();
            return slot;
          };
          auto qk = [&](int t, int at) {
            if (!ok) return;
            const uint32_t k_at = r_k + at * (S::kTileBytes >> 4), q_at = q_lo + t * q_step;
#pragma unroll
            for (int c = 0; c < S::kChunks; ++c)
              mma_qk_chunk(tmem + t * kKeys, q_at + c * (S::kChunkBytes >> 4), k_at + c * (S::kChunkBytes >> 4), kIdS, c);
            tc_commit(&bars.s_full[t]);
          };
          // round r of ring t; its last one completes the ring's O
          auto pv = [&](int t, int at, int r, int e, bool last) {
            const uint32_t v_at = r_v + at * (S::kTileBytes >> 4), p_at = tmem + t * kKeys, d = tmem + 256 + t * HD;
            const bool some = !WHOLE && (dual ? 2 * (s_lo + r) + t : s_lo + r) >= np;
            if (some && ok) ok = mbar_wait(&bars.looked_up[e & 15], e >> 4, &abort_sh);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if (ok) ok = mbar_wait(&bars.p_ready[t][half], r & 1, &abort_sh);
              if (!ok) return;
              tc_fence_after();
              // packed rows start from a cleared O
              if (some)
                mma_pv_half_some(d, p_at + half * 32, v_at + half * (64 * 128 >> 4), kIdO, &bars.others[e & 15][half * 4]);
              else
                mma_pv_half(d, p_at + half * 32, v_at + half * (64 * 128 >> 4), kIdO, WHOLE ? r | half : 1);
            }
            if (last) tc_commit(&bars.o_done[t]);
          };
          auto release = [&](int at) {
            if (ok) tc_commit(&bars.empty[at]);
          };
          // Step i's second products, then the next step's first ones (step -1: the
          // first ones alone).  A tile for both rings is released after the second
          // ring's product.
          int looked = 0, e0 = 0, e1 = 0, n0_e = 0, next_e = 0;  // the entries of the rings' tiles: number, and turn in bit 4
#pragma unroll 1
          for (int i = -1; i < n && ok; ++i) {
            const bool both = i < n_both, both1 = i + 1 < n_both;
            int at_v = -1, at_k = -1;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int mine = t ? n1 : n0;
              if (i >= 0 && i < mine) {
                if (!both || at_v < 0) at_v = next_slot();
                const int e = both ? e0 : (t ? e1 : e0);
                pv(t, at_v, i, e, i + 1 == mine);
                if (!both) release(at_v);
                if (!WHOLE && ok && (!both || t == 1)) mbar_arrive(&bars.done_with[e & 15]);
              }
              if (i + 1 < mine) {
                if (!both1 || at_k < 0) {
                  at_k = next_slot();
                  next_e = looked;
                  if ((++looked & 15) == kLooked) looked = (looked >> 4 ^ 1) << 4;
                }
                qk(t, at_k);
                if (!both1) release(at_k);
                if (t)
                  e1 = next_e;
                else
                  n0_e = next_e;
              }
            }
            e0 = n0_e;
            if (both && at_v >= 0) release(at_v);
            if (both1 && at_k >= 0) release(at_k);
          }
          if (!ok) {
            abort_sh = 1;
            report_status(p.status, LR_ERR_TIMEOUT);
          }
          // every MMA issued by this thread completes before TMEM is released
          tc_commit(&bars.drain);
          mbar_wait(&bars.drain, 0, nullptr);
        }
        __syncwarp();
      }
    }
  } else {
    regs_more<kRegsSoftmax>();
    if (n > 0) {
      // ------------------------------------------------------- softmax
      const int t = ringi;
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t s_at = tmem + t * kKeys + lanes, o_at = tmem + 256 + t * HD + lanes;
      // own tokens that this row sees (rows past the tile's are never stored), and
      // where its sequence's lie in the list of packed tiles
      int vis = 0, list_lo = 0, list_hi = 0;
      if (WHOLE) {
        vis = seen(mrel + tile * a.mt + trow / G);
      } else if (my_seq >= 0) {
        const SeqView v = seq_view(p, first_seq + my_seq, false);
        vis = v.len - v.n + (mrel + tile * a.mt + trow / G - v.q0) + 1;
        vis = vis > v.len ? v.len : (vis < 0 ? 0 : vis);
        int r = trow / G;
        while (r < (tile ? rows1 : rows0) - 1 && bars.seq[tile][r + 1] == my_seq) ++r;
        list_lo = r > 0 ? bars.groups[tile][r - 1] * kPage : 0;
        list_hi = bars.groups[tile][r] * kPage;
      }
      sees = P > 0 || vis > 0;
      if (!WHOLE) {  // the rows of a tile do not all take part in its first product
        uint32_t z[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) z[j] = 0;
#pragma unroll 1
        for (int c = 0; c < HD / 16; ++c) tmem_st16(o_at + c * 16, z);
        tmem_st_wait();
      }
      const bool busy = (warp & 3) * 32 < live_rows;  // a warp without rows only keeps the rings moving
      bool ok = true;
      // a ring without keys waits for nothing else: its Q tile, where the rows are turned
      // below, may still be on its way here
      if (my_n == 0) ok = mbar_wait(&bars.q_full, 0, &abort_sh);
      for (int i = 0; i < my_n && ok; ++i) {
        ok = mbar_wait(&bars.s_full[t], i & 1, &abort_sh);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        // Of the tile's eight groups of 16 keys the row takes those in `use`, and of
        // these the keys below hi.  The others are keys of other sequences: the
        // row's output lane is off in their products, so that they only have to
        // stay out of its maximum and sum, and that goes by whole groups.
        const int c = dual ? 2 * (s_lo + i) + t : s_lo + i;
        int hi = P - c * kKeys, end = kKeys;
        uint32_t use = 0xFFu;
        if (c >= np) {
          const int first = (c - np) * kKeys;
          hi = vis - first;
          if (!WHOLE) {
            const int from = list_lo - first > 0 ? list_lo - first : 0;
            end = list_hi - first < kKeys ? list_hi - first : kKeys;
            use = end > from ? (0xFFu >> (8 - end / kPage)) & (0xFFu << (from / kPage)) : 0u;
            hi = use ? list_lo - first + vis : kKeys;
          }
        }
        const bool mine = use != 0;
        if (WHOLE && busy && !__any_sync(0xffffffffu, hi > 0)) {  // none of the warp's rows: P = 0
          uint32_t z[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) z[j] = 0;
#pragma unroll 1
          for (int k = 0; k < kKeys / 32; ++k) tmem_st16(s_at + k * 16, z);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.p_ready[t][0]);
        } else if (busy && (WHOLE || __any_sync(0xffffffffu, mine))) {
          uint32_t s[kKeys];
#pragma unroll
          for (int c = 0; c < kKeys / 32; ++c) tmem_ld32(s_at + c * 32, s + c * 32);
          tmem_ld_wait();
          // groups that some row of the warp sees a part of
          const uint32_t beyond = hi >= end ? 0u : (hi <= 0 ? use : use & (0xFFu << (hi / kPage)));
          const uint32_t cut = __reduce_or_sync(0xffffffffu, beyond);
          if (cut != 0) {
#pragma unroll
            for (int g = 0; g < 8; ++g)
              if (cut >> g & 1u) {
                const int left = use >> g & 1u ? hi - g * kPage : kPage;
#pragma unroll
                for (int j = 0; j < kPage; ++j)
                  if (j >= left) s[g * kPage + j] = 0xFF800000u;  // -inf
              }
          }
          const bool full = WHOLE || __all_sync(0xffffffffu, use == 0xFFu);
          float tops[8];
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            const uint32_t* x = s + g * kPage;
            float m = max3(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]));
#pragma unroll
            for (int j = 3; j < 15; j += 2) m = max3(m, __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
            tops[g] = fmaxf(m, __uint_as_float(x[15]));
          }
          if (!full) {
#pragma unroll
            for (int g = 0; g < 8; ++g)
              if ((use >> g & 1u) == 0) tops[g] = -INFINITY;
          }
          const float top = fmaxf(max3(max3(tops[0], tops[1], tops[2]), tops[3], tops[4]), max3(tops[5], tops[6], tops[7]));
          const float now = mine ? fmaxf(mref, top * p.scale_log2) : mref;
          const bool move = now > mref + kSlack;  // -inf + 8 is -inf: the first key moves it
          if (__any_sync(0xffffffffu, move)) {
            const float next = move ? now : mref;
            const float f = next == -INFINITY ? 1.f : ex2(mref - next);
            sum *= f;
            mref = next;
            if (i > 0) {
#pragma unroll 1
              for (int c = 0; c < HD / 16; ++c) {
                uint32_t o[16];
                tmem_ld16(o_at + c * 16, o);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                tmem_st16(o_at + c * 16, o);
              }
            }
          }
          const float neg = mref == -INFINITY ? 0.f : -mref;
          const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2), neg2 = pack2(neg, neg);
          uint64_t part[8];  // of each group
#pragma unroll
          for (int c = 0; c < kKeys / 64; ++c) {
            uint32_t w[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const int at = c * 64 + 2 * j, g = at / kPage;
              float x, y;
              unpack2(fma2(pack2(__uint_as_float(s[at]), __uint_as_float(s[at + 1])), scale2, neg2), x, y);
              x = ex2(x);
              y = ex2(y);
              part[g] = at % kPage == 0 ? pack2(x, y) : add2(part[g], pack2(x, y));
              // the product takes bf16: the powers round here, their sum does not
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(y), "f"(x));
            }
            tmem_st32(s_at + c * 32, w);
            if (c == 0) {
              tmem_st_wait();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bars.p_ready[t][0]);
            }
          }
          if (!full) {
#pragma unroll
            for (int g = 0; g < 8; ++g)
              if ((use >> g & 1u) == 0) part[g] = 0;
          }
          float pa, pb;
          unpack2(add2(add2(add2(part[0], part[1]), add2(part[2], part[3])),
                       add2(add2(part[4], part[5]), add2(part[6], part[7]))), pa, pb);
          if (mine) sum += pa + pb;
          tmem_st_wait();
        } else if (lane == 0) {
          mbar_arrive(&bars.p_ready[t][0]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_ready[t][1]);
      }
      if (ok && my_n > 0) {
        ok = mbar_wait(&bars.o_done[t], 0, &abort_sh);
        // the ring is the other one's too: its products end before it is written below
        if (ok && joins && t == 1) ok = mbar_wait(&bars.o_done[0], 0, &abort_sh);
        tc_fence_after();
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok && lane == 0) {
        abort_sh = 1;
        report_status(p.status, LR_ERR_TIMEOUT);
      }
      if (ok && joins && t == 1 && n1 > 0 && busy) {  // ring 1 hands its part to ring 0
        hand_ml[trow] = make_float2(mref, sum);
        float* dst = reinterpret_cast<float*>(ring) + trow * (HD + 4);
#pragma unroll 1
        for (int c = 0; c < HD / 16; ++c) {
          uint32_t o[16];
          tmem_ld16(o_at + c * 16, o);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; j += 4)
            *reinterpret_cast<uint4*>(dst + c * 16 + j) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
        }
      }
    }
    tc_fence_before();
    if (joins) named_bar_sync(1, 256);  // the softmax warps
    tc_fence_after();
    // (one answer for the warp: another warp may give up just now, and a part of a
    // warp must not go where its lanes wait for each other)
    const bool gave_up = __any_sync(0xffffffffu, *static_cast<volatile int*>(&abort_sh) != 0);
    if (!(joins && ringi == 1) && !gave_up) {
      // ------------------------------------------------- rows to memory
      const int t = ringi;
      const bool busy = (warp & 3) * 32 < live_rows;
      const bool live = trow < live_rows;
      if (busy) {
        const uint32_t o_at = tmem + 256 + t * HD + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const bool both = joins && n1 > 0;
        float f0 = 1.f, f1 = 0.f, m = mref, l = sum;
        if (both) {
          const float2 o = hand_ml[trow];
          m = fmaxf(mref, o.x);
          const float ref = m == -INFINITY ? 0.f : m;
          f0 = ex2(mref - ref);
          f1 = ex2(o.x - ref);
          l = f0 * sum + f1 * o.y;
        }
        if (my_n == 0) f0 = 0.f;  // nothing was summed: TMEM holds no result
        const int64_t qrow = q0 + mrel + tile * a.mt + trow / G;
        const int head = kvh * G + trow % G;
        const int slot = a.two ? 2 * split + (dual ? t : 0) : split;
        const int64_t slot_rows = static_cast<int64_t>(p.M) * p.n_heads;
        const int64_t at = slot * slot_rows + qrow * p.n_heads + head;
        if (a.direct) {
          // a packed row of no sequence comes out zero, and so does one that sees no key;
          // one that sees keys of score minus infinity alone is 0 / 0
          const float inv = !WHOLE && my_seq < 0 ? 0.f : (l != 0.f ? 1.f / l : (sees ? NAN : 0.f));
          f0 *= inv;
          f1 *= inv;
        } else if (live) {
          p.pml[at] = make_float2(m, l == 0.f && sees ? -0.f : l);
          if (a.two && !dual) p.pml[at + slot_rows] = make_float2(-INFINITY, 0.f);
        }
        const float* other = reinterpret_cast<const float*>(ring) + trow * (HD + 4);
        // A thread holds a row; memory wants rows side by side (16 bytes a lane
        // of 32 rows each touch 32 lines).  The warp turns half a row at a time
        // in its part of this ring's Q tile, which no product reads any more;
        // 16-byte columns are permuted by the row against bank conflicts.
        constexpr int kHalf = HD / 2, kVec = kHalf / 4, kPer = 32 / kVec;
        float4* stage = reinterpret_cast<float4*>(q_sm + t * S::kTileBytes + (warp & 3) * (S::kTileBytes / 4));
        const int64_t row_off = a.direct ? qrow * p.ldo + static_cast<int64_t>(head) * HD : at * HD;
        const int left = live_rows - (warp & 3) * 32;  // rows of this warp
        // (Code that runs once is short: it costs what its fetching costs.)
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
#pragma unroll 1
          for (int c = 0; c < kHalf / 32; ++c) {
            uint32_t r[32];
            tmem_ld32(o_at + half * kHalf + c * 32, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
              if (f0 != 0.f)
                x = make_float4(__uint_as_float(r[j]) * f0, __uint_as_float(r[j + 1]) * f0,
                                __uint_as_float(r[j + 2]) * f0, __uint_as_float(r[j + 3]) * f0);
              if (both) {
                const float4 y = *reinterpret_cast<const float4*>(other + half * kHalf + c * 32 + j);
                x.x = fmaf(y.x, f1, x.x), x.y = fmaf(y.y, f1, x.y);
                x.z = fmaf(y.z, f1, x.z), x.w = fmaf(y.w, f1, x.w);
              }
              stage[lane * kVec + ((c * 8 + j / 4) ^ (lane & 7))] = x;
            }
          }
          __syncwarp();
          // eight stores at a time, so that their reads overlap
#pragma unroll 1
          for (int i0 = 0; i0 < 32 / kPer; i0 += 8) {
            float4 x[8];
            int64_t off[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = (i0 + i) * kPer + lane / kVec, c = lane % kVec;
              x[i] = stage[r * kVec + (c ^ (r & 7))];
              off[i] = __shfl_sync(0xffffffffu, row_off, r) + half * kHalf + c * 4;
            }
            const int live_here = left - i0 * kPer - lane / kVec;
            if (a.direct && !p.out_f32) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                uint2 w;
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(x[i].y), "f"(x[i].x));
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(x[i].w), "f"(x[i].z));
                if (i * kPer < live_here) *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + off[i]) = w;
              }
            } else {
              float* dst = a.direct ? static_cast<float*>(p.out) : p.po;
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (i * kPer < live_here) *reinterpret_cast<float4*>(dst + off[i]) = x[i];
            }
          }
          __syncwarp();
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int HD, bool WHOLE>
lr_status launch_tiles(const TileParams& a, dim3 grid, cudaStream_t s) {
  using Sh = Shape<HD>;
  CUtensorMap mq;
  lr_status st = encode_map_heads(&mq, a.p.q, HD, a.p.n_heads, a.p.M, a.p.ldq, a.p.group, a.mt);
  if (st != LR_OK) return st;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Sh::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  if (pdl_enabled()) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  cudaError_t e = cudaLaunchKernelEx(&cfg, attn_tiles_kernel<HD, WHOLE>, a, mq);
  if (e != cudaSuccess) return cuda_fail(e, "attn_tiles");
  return LR_OK;
}

}  // namespace

lr_status launch_attn_tiles(const AttnParams& p, int head_dim, const AttnPart& part, cudaStream_t s) {
  TileParams a;
  memset(&a, 0, sizeof(a));
  a.p = p;
  a.mt = attn_tile_rows(p.group);
  const int per_pair = 2 * a.mt;
  a.pairs = ((part.whole ? p.max_q : p.M) + per_pair - 1) / per_pair;
  a.slots = part.slots;
  a.direct = part.slots == 1;
  a.two = part.two;
  a.stall = test_stall_producer();
  const int64_t ctas = static_cast<int64_t>(a.pairs) * (part.whole ? p.n_seq : 1) * p.n_kv;
  const dim3 grid(static_cast<unsigned>(ctas), 1, part.slots);
  if (head_dim == 64) return part.whole ? launch_tiles<64, true>(a, grid, s) : launch_tiles<64, false>(a, grid, s);
  return part.whole ? launch_tiles<128, true>(a, grid, s) : launch_tiles<128, false>(a, grid, s);
}

lr_status configure_attn_tiles() {
  auto set = [](auto kern, int smem) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  };
  cudaError_t e = set(attn_tiles_kernel<64, true>, Shape<64>::kSmem);
  if (e == cudaSuccess) e = set(attn_tiles_kernel<64, false>, Shape<64>::kSmem);
  if (e == cudaSuccess) e = set(attn_tiles_kernel<128, true>, Shape<128>::kSmem);
  if (e == cudaSuccess) e = set(attn_tiles_kernel<128, false>, Shape<128>::kSmem);
  if (e != cudaSuccess) return cuda_fail(e, "attention tiles: set smem");
  return LR_OK;
}

}  // namespace lr
