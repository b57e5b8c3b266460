/*
 * lr.h -- C ABI of liblr, the GB300 (sm_103a) factorized-linear inference path.
 *
 * What it computes comes from DeInfer: Efficient Parallel Inferencing for
 * Decomposed Large Language Models (Huang, Huang, Liao, Wen), as summarised on
 * gist.science/paper/2604.17709 (English page) and gist.science/es/paper/
 * 2604.17709 (Spanish page).  Every weight W[d_in][d_out] of a transformer
 * block is approximated by two low-rank factors, W ~ A_r B_r (Spanish page,
 * "Resumen Tecnico" section 1; English page section 1), and a layer is
 * evaluated as a down projection followed by an up projection (English page
 * section 2.A).  For decoding under a static CUDA graph, rows scattered over
 * paged memory are first listed in a remap table and copied into a fixed
 * buffer; the graph then runs fixed-size GEMMs on that buffer (English page
 * section 2.C).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Pointers marked "device" are CUDA device pointers owned by the caller; the
 *   library never allocates, frees or keeps them past the call (the graph
 *   object keeps them, see lr_graph_capture).  Pointers marked "host" are
 *   ordinary host memory.
 * - bf16 means IEEE bfloat16 bit patterns (uint16_t).  All matrices are
 *   row-major with the leading dimension given in elements.
 * - Factors are stored out-major, the layout of a linear layer's weight:
 *   the down factor A_r[d_in][r] is stored transposed as At[r][d_in] and the
 *   up factor B_r[r][d_out] as Bt[d_out][r].  Every tensor-core operand is
 *   then contiguous along the reduction dimension.
 * - Work is enqueued on the given stream (0 = the legacy default stream) and
 *   runs asynchronously.  Argument errors are detected on the host before
 *   anything is enqueued and returned as LR_ERR_INVALID_ARG or
 *   LR_ERR_UNSUPPORTED; nothing is launched in that case.
 * - Device-side problems never trap: a kernel that meets one stores the first
 *   error code into the caller's int32 device word `dev_status` (compare-and-
 *   swap from 0) and finishes safely.  The caller reads it after synchronising
 *   and resets it to 0.
 * - Every wait inside a kernel is bounded (about two seconds); a wait that
 *   runs out reports LR_ERR_TIMEOUT through dev_status and the kernel returns.
 * - No exception crosses this interface.  lr_last_error() gives a one-line
 *   description of the last host-side error of the calling thread.
 */
#ifndef LR_H_
#define LR_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* lr_stream; /* a cudaStream_t */

typedef enum {
  LR_OK = 0,
  LR_ERR_INVALID_ARG = 1,  /* null pointer, bad size, misalignment, small buffer */
  LR_ERR_UNSUPPORTED = 2,  /* a dimension outside what the kernels handle */
  LR_ERR_CUDA = 3,         /* a CUDA runtime/driver call failed */
  LR_ERR_TIMEOUT = 4,      /* device: a bounded wait ran out */
  LR_ERR_REMAP_RANGE = 5,  /* device: a remap entry outside the pool */
  LR_ERR_STATE = 6,        /* wrong object state (e.g. replaying a destroyed graph) */
  LR_ERR_INDEX_RANGE = 7   /* device: a position, length or row offset outside its range */
} lr_status;

typedef enum { LR_BF16 = 0, LR_F32 = 1 } lr_dtype;

/* One factor pair (A_r, B_r) of a decomposed projection, W ~ A_r B_r.
 * At: device bf16 [r][d_in]  (A_r transposed), row stride d_in.
 * Bt: device bf16 [d_out][r] (B_r transposed), row stride r.
 * d_in, d_out and r must be positive multiples of 64 (LR_ERR_UNSUPPORTED
 * otherwise); both pointers must be 16-byte aligned. */
typedef struct {
  const void* At;
  const void* Bt;
  int32_t d_in;
  int32_t d_out;
  int32_t r;
} lr_factor;

/* lr_factor_pack: the factors in the pages' orientation, W ~ A_r B_r
 * (Spanish page, "Resumen Tecnico" section 1), to the layout above.
 *   A: device bf16 [d_in][r] row-major (A_r);  B: device bf16 [r][d_out]
 *   row-major (B_r).  At: device bf16 [r][d_in], Bt: device bf16 [d_out][r],
 *   written as the exact transposes (bit-for-bit copies of every element).
 *   d_in, d_out, r positive multiples of 64 (LR_ERR_UNSUPPORTED otherwise);
 *   every pointer 16-byte aligned; the four buffers must not overlap
 *   (LR_ERR_INVALID_ARG).  Enqueued on s; a one-time step when a model's
 *   factors are loaded, not part of a decode step. */
lr_status lr_factor_pack(const void* A, const void* B, int32_t d_in, int32_t d_out, int32_t r, void* At,
                         void* Bt, lr_stream s);

/* Projections of a block, in this order (English page section 2.D: attention
 * and MLP projections are all decomposed). */
enum { LR_Q = 0, LR_K = 1, LR_V = 2, LR_O = 3, LR_GATE = 4, LR_UP = 5, LR_DOWN = 6 };

/* A decomposed LLaMA-style block whose attention core is attention over a
 * one-token context (each query head returns the value vector of its kv head).
 * q: d_model -> n_heads*head_dim, k/v: d_model -> n_kv_heads*head_dim,
 * o: n_heads*head_dim -> d_model, gate/up: d_model -> d_ff, down: d_ff -> d_model.
 * n_heads must be a multiple of n_kv_heads (MHA, GQA, MQA); head_dim a multiple
 * of 64; d_model at most 8192; RMSNorm has unit gain and the given eps.
 * The MLP is SiLU-GLU or, with mlp = LR_MLP_RELU, a non-GLU ReLU MLP. */
/* MLP variants (English page section 2.D: GLU and non-GLU MLPs). */
enum { LR_MLP_SWIGLU = 0, /* h += down(silu(gate(n2)) * up(n2)) (LLaMA) */
       LR_MLP_RELU = 1    /* h += down(relu(up(n2))), gate unused (OPT) */ };

typedef struct {
  int32_t d_model;
  int32_t d_ff;
  int32_t n_heads;
  int32_t n_kv_heads;
  int32_t head_dim;
  float eps;
  lr_factor f[7];
  int32_t mlp;  /* LR_MLP_SWIGLU or LR_MLP_RELU; with LR_MLP_RELU f[LR_GATE] is not read */
} lr_block_desc;

/* ---------------------------------------------------------------------------
 * lr_linear_forward: y = (x A_r) B_r for M rows.
 * English page section 2.A (down projection, then up projection); Spanish
 * page "Resumen Tecnico" section 1 (W ~ A B).
 *   x  device bf16 [M][ldx], ldx >= d_in, ldx multiple of 8, x 16-byte aligned.
 *   y  device [M][ldy] of y_dtype (LR_BF16 or LR_F32), ldy >= d_out.
 *   The intermediate t = x A_r is rounded to bf16 (round to nearest even) and
 *   kept in `workspace`; the sums accumulate in fp32.  A bf16 y is the
 *   round-to-nearest-even image of the fp32 y.
 *   workspace: device, at least lr_linear_workspace_bytes(M, f) bytes, 256-byte
 *   aligned; it holds t (M x r bf16) and, for M > 256, one int32 completion
 *   counter per 256-row band of the one-launch prefill form.  Its contents on
 *   entry do not matter (every element that is read was written, or
 *   cleared, by the same call).  Calls that share a workspace must be
 *   ordered on one stream.
 *   M = 0 is a no-op.  M <= 256 runs the decode kernels, larger M the prefill
 *   kernels (on SM pairs; a linear under 1.5e12 flops runs its down and up
 *   projections in one launch).  The result is deterministic (no
 *   floating-point atomics) and the same whichever form runs. */
size_t lr_linear_workspace_bytes(int64_t M, const lr_factor* f);
lr_status lr_linear_forward(const void* x, int64_t ldx, void* y, int64_t ldy, lr_dtype y_dtype,
                            int64_t M, const lr_factor* f, void* workspace, size_t ws_bytes,
                            int32_t* dev_status, lr_stream s);

/* ---------------------------------------------------------------------------
 * lr_linear_forward_noalloc: the same computation as lr_linear_forward for
 * callers that cannot allocate device memory.  The paper has no counterpart;
 * this is an interface convenience.
 *   Some callers cannot hand the library a workspace: code that runs where
 *   cudaMalloc is forbidden or unwanted (an allocator-free embedded runtime, a
 *   plugin that receives only raw pointers and a stream, a serving loop whose
 *   device memory is fixed at start-up), or code that must not risk the
 *   implicit device synchronisation an allocation can cause.  This entry point
 *   keeps the intermediate t = x A_r in a static device array of
 *   LR_NOALLOC_SCRATCH_BYTES (4 MiB) inside the library instead.  Every GPU
 *   that loads the library holds that array until the process exits.  The
 *   call itself allocates nothing (no cudaMalloc/cudaFree, no allocating
 *   library routine).
 *   Arguments, layouts, checks and results are those of lr_linear_forward
 *   without the workspace.  lr_linear_workspace_bytes(M, f) (about M * r * 2)
 *   must not exceed LR_NOALLOC_SCRATCH_BYTES; larger problems are rejected
 *   with LR_ERR_UNSUPPORTED and a message in lr_last_error().
 *   The first call on each device looks up the array's device address
 *   (cudaGetSymbolAddress); make that first call before any stream capture.
 *   All calls share the one array and it keeps the last call's contents.
 *   Nothing in it needs to start at zero (each call writes every element it
 *   reads).  Calls that overlap on the GPU (on different streams, say) race on
 *   it: order them on one stream. */
#define LR_NOALLOC_SCRATCH_BYTES (4u << 20)
lr_status lr_linear_forward_noalloc(const void* x, int64_t ldx, void* y, int64_t ldy,
                                    lr_dtype y_dtype, int64_t M, const lr_factor* f,
                                    int32_t* dev_status, lr_stream s);

/* ---------------------------------------------------------------------------
 * lr_block_forward: one decomposed block applied in place to the fp32 residual
 * stream h (device fp32 [M][d_model], 16-byte aligned):
 *   n1 = RMSNorm(h); q,k,v = LR(n1); h += LR_o(attn(v));
 *   n2 = RMSNorm(h); h += LR_down(silu(LR_gate(n2)) * LR_up(n2))
 *   (non-GLU: h += LR_down(relu(LR_up(n2)))).
 * Spanish page section 1 (attention and MLP projections decomposed) and
 * section 2 "Generalizacion"; English page section 2.D (MHA/GQA/MQA, GLU MLP).
 * Linear inputs are rounded to bf16.  scratch: device, at least
 * lr_block_scratch_bytes(M, b) bytes, 256-byte aligned; its contents on entry
 * do not matter.  M = 0 is a no-op.  Each linear runs as lr_linear_forward
 * would at the same M (decode kernels up to 256 rows, the SM-pair prefill
 * GEMM above, one launch per linear below 1.5e12 flops); the result does not
 * depend on which form runs. */
size_t lr_block_scratch_bytes(int64_t M, const lr_block_desc* b);
lr_status lr_block_forward(float* h, int64_t M, const lr_block_desc* b, void* scratch,
                           size_t scratch_bytes, int32_t* dev_status, lr_stream s);

/* ---------------------------------------------------------------------------
 * remap_compact: the copy of the preparation stage (English page section 2.C):
 *   buf[i][:] = pool[remap[i]][:] for 0 <= i < min(*n_active, cap), zero rows
 *   for i >= *n_active.  Bit-exact byte copy of row_bytes per row.
 *   pool: device [pool_rows][row_bytes]; buf: device [cap][row_bytes];
 *   remap: device int32 [cap]; n_active: device int32 (read on the device, so
 *   the launch parameters never change with the batch).  row_bytes must be a
 *   positive multiple of 16 and every pointer 16-byte aligned.  An entry
 *   outside [0, pool_rows) gives a zero row and LR_ERR_REMAP_RANGE in
 *   dev_status. */
lr_status remap_compact(const void* pool, int64_t pool_rows, int64_t row_bytes,
                        const int32_t* remap, const int32_t* n_active, void* buf, int64_t cap,
                        int32_t* dev_status, lr_stream s);

/* remap_scatter: the inverse copy, pool[remap[i]][:] = buf[i][:] for
 * 0 <= i < min(*n_active, cap).  Same arguments and checks as remap_compact;
 * an out-of-range entry is skipped and reported.  Targets must be distinct
 * (remap_build makes them so); with duplicates the surviving row is
 * unspecified. */
lr_status remap_scatter(const void* buf, const int32_t* remap, const int32_t* n_active,
                        void* pool, int64_t pool_rows, int64_t row_bytes, int64_t cap,
                        int32_t* dev_status, lr_stream s);

/* remap_build (host only): the scan of the preparation stage (English page
 * section 2.C, "remapping index list (a new block table)").
 *   lengths: host int32 [n_seq]; block_table: host int32 [n_seq][blocks_per_seq],
 *   entry (s, b) = physical block of logical block b of sequence s.
 *   For each sequence in order, its last tail_rows positions (all positions if
 *   tail_rows <= 0) are mapped to physical rows
 *   block_table[s][p / block_rows] * block_rows + p % block_rows.
 *   Outputs (host): remap_out[cap] (unused entries -1), *n_active_out, and
 *   *n_runs_out = number of maximal runs of consecutive physical rows.
 *   LR_ERR_INVALID_ARG if the rows exceed cap, a needed table entry is
 *   negative, a length is negative or exceeds the table, or two rows coincide. */
lr_status remap_build(const int32_t* lengths, int64_t n_seq, const int32_t* block_table,
                      int32_t blocks_per_seq, int32_t block_rows, int32_t tail_rows, int64_t cap,
                      int32_t* remap_out, int32_t* n_active_out, int32_t* n_runs_out);

/* ---------------------------------------------------------------------------
 * lr_kv_reconstruct: the reconstruction of a low-rank KV cache under a static
 * graph (English page section 2.C: scattered latent rows are listed by a
 * remap table, copied into a contiguous buffer, and "the contiguous buffer is
 * multiplied by the upward projection matrices to reconstruct the KV cache"
 * in one large fixed-size GEMM; the latent KV grows with the context, English
 * page section 1).
 *   latent_buf[i][:] = latent_pool[remap[i]][:] for i < *n_active, zero rows
 *   otherwise (as remap_compact), then out = latent_buf Bt^T, i.e.
 *   out[i][n] = sum_j latent_buf[i][j] * B_r[j][n].
 *   latent_pool: device bf16 [pool_rows][r]; latent_buf: device bf16 [cap][r];
 *   Bt: device bf16 [d_kv][r] (the up factor transposed); out: device bf16
 *   [cap][d_kv].  r and d_kv positive multiples of 64, pointers 16-byte
 *   aligned.  Rows past *n_active come out zero.  cap and every pointer are
 *   fixed, so the two launches can be captured once and replayed per step.
 *   Out-of-range remap entries give zero rows and LR_ERR_REMAP_RANGE. */
lr_status lr_kv_reconstruct(const void* latent_pool, int64_t pool_rows, int32_t r,
                            const int32_t* remap, const int32_t* n_active, int64_t cap,
                            void* latent_buf, const void* Bt, int32_t d_kv, void* out,
                            int32_t* dev_status, lr_stream s);

/* ---------------------------------------------------------------------------
 * The block-granular form of the same reconstruction: the remap lists whole
 * paged blocks (the pages' "new block table", English page section 2.C), and
 * the up-projection GEMM reads each listed block straight from the latent
 * pool -- no compacted copy is written or read back.
 *
 * remap_build_blocks (host only): for each sequence in order, the physical
 * blocks that hold its positions 0 .. L-1 (the first ceil(L / block_rows)
 * entries of its block-table row).
 *   lengths: host int32 [n_seq]; block_table: host int32 [n_seq][blocks_per_seq].
 *   Outputs (host): blocks_out[cap_blocks] (unused entries -1), *n_blocks_out,
 *   *n_runs_out = maximal runs of consecutive block ids.
 *   LR_ERR_INVALID_ARG if the blocks exceed cap_blocks, a needed entry is
 *   negative, a length does not fit its table row, or a block is listed twice.
 *   Position p of sequence s sits at row block_rows * i + p % block_rows of
 *   the reconstruction, i being the list index of its block. */
lr_status remap_build_blocks(const int32_t* lengths, int64_t n_seq, const int32_t* block_table,
                             int32_t blocks_per_seq, int32_t block_rows, int64_t cap_blocks,
                             int32_t* blocks_out, int32_t* n_blocks_out, int32_t* n_runs_out);

/* lr_kv_latent_write: the producer side of the low-rank KV cache (English
 * page section 1: the latent KV grows with the context; section 2.C: it is
 * kept in paged memory).  The down projection of k or v for M new tokens is
 * written straight into their rows of the paged latent pool:
 *   latent_pool[rows[m]][:] = bf16(x[m] A_r)   for m < M,
 * summed in fp32 and rounded to nearest even, with A_r given transposed as
 * At [r][d_in].  x: device bf16 [M][ldx]; rows: device int32 [M] (for one new
 * token per sequence, remap_build with tail_rows = 1 on the grown lengths);
 * latent_pool: device bf16 [pool_rows][r].  d_in, r positive multiples of 64;
 * pointers 16-byte aligned, ldx >= d_in and a multiple of 8.  Entries of rows
 * outside [0, pool_rows) are skipped and reported as LR_ERR_REMAP_RANGE;
 * rows must be distinct.  Other pool rows are not touched.  The values are
 * those the down launch of lr_linear_forward writes for t.  M = 0 is a
 * no-op. */
lr_status lr_kv_latent_write(const void* x, int64_t ldx, int64_t M, const void* At, int32_t d_in, int32_t r,
                             const int32_t* rows, void* latent_pool, int64_t pool_rows, int32_t* dev_status,
                             lr_stream s);

/* lr_kv_reconstruct_paged: with 16-row blocks,
 *   out[16 i + j][n] = sum_c latent_pool[16 blocks[i] + j][c] * B_r[c][n]
 * for i < *n_blocks and j < 16; rows of blocks i >= *n_blocks are zero.
 *   latent_pool: device bf16 [pool_blocks * 16][r]; blocks: device int32
 *   [cap_blocks]; n_blocks: device int32 (read on the device, so a captured
 *   graph serves every batch); Bt: device bf16 [d_kv][r]; out: device bf16
 *   [cap_blocks * 16][d_kv].  r and d_kv positive multiples of 64; pointers
 *   16-byte aligned.  A listed block outside [0, pool_blocks) reads as zeros
 *   and reports LR_ERR_REMAP_RANGE.  The rows past a sequence's length in its
 *   last block are reconstructed from whatever the pool holds there; the
 *   caller ignores them.  One launch. */
lr_status lr_kv_reconstruct_paged(const void* latent_pool, int64_t pool_blocks, int32_t r, const int32_t* blocks,
                                  const int32_t* n_blocks, int64_t cap_blocks, const void* Bt, int32_t d_kv,
                                  void* out, int32_t* dev_status, lr_stream s);

/* ---------------------------------------------------------------------------
 * Rank-space sharding of one factorized linear, simulated on this GPU (English
 * page section 2.A, "Highly Efficient Low-Rank Communication": the down
 * projection is split by columns and its output all-gathered in the low-rank
 * space; the up projection runs in shard mode, with no reduce-sum).
 *
 * The rank columns are split over G simulated processes in blocks of 64: process g
 * owns rank columns R_g = [64*floor(g*nr/G), 64*floor((g+1)*nr/G)) with
 * nr = r/64, and output columns O_g likewise over d_out/64 blocks.  Then
 *   1. down, per process:  t_g = x A_r[:, R_g]   into process g's own buffer
 *      (bf16 [M][|R_g|], the rows R_g of At);
 *   2. all-gather in rank space, emulated by device-to-device copies of every
 *      t_g into the columns R_g of one gathered t (bf16 [M][r]);
 *   3. up, shard mode, per process:  y[:, O_g] = t B_r[:, O_g]  (the rows O_g
 *      of Bt), written straight into the caller's y.
 * Every launch is issued on `s`, one process after another.  y equals
 * lr_linear_forward's result up to the fp32 summation order of the split GEMMs.
 * Arguments and checks as lr_linear_forward, plus 1 <= n_shards <= r/64 and
 * n_shards <= d_out/64 (else LR_ERR_INVALID_ARG); the workspace (device,
 * 256-byte aligned, caller-owned) holds the G process buffers and the
 * gathered t: lr_rank_sharded_workspace_bytes bytes.  M == 0 is a no-op. */
size_t lr_rank_sharded_workspace_bytes(int64_t M, const lr_factor* f, int32_t n_shards);
lr_status lr_linear_forward_rank_sharded(const void* x, int64_t ldx, void* y, int64_t ldy,
                                         lr_dtype y_dtype, int64_t M, const lr_factor* f,
                                         int32_t n_shards, void* workspace, size_t ws_bytes,
                                         int32_t* dev_status, lr_stream s);

/* lr_rank_shard_comm_bytes (host only): collective bytes that the busiest of
 * the G processes receives for one factorized linear, with the column split
 * above and elements of elem_bytes bytes:
 *   *rank_space = (r - min_g |R_g|) * M * elem_bytes    (ring all-gather of t,
 *                 the low-rank scheme);
 *   *full_space = 2 (d_out - min_g |O_g|) * M * elem_bytes  (ring all-reduce of
 *                 y, i.e. reduce-scatter then all-gather: the reduce-sum in the
 *                 full dimension that a naive split of the two factors needs).
 * LR_ERR_INVALID_ARG on a negative M, non-positive sizes, r or d_out not a
 * multiple of 64, or n_shards outside [1, min(r, d_out)/64]. */
lr_status lr_rank_shard_comm_bytes(int64_t M, int32_t d_out, int32_t r, int32_t n_shards,
                                   int32_t elem_bytes, int64_t* rank_space, int64_t* full_space);

/* ---------------------------------------------------------------------------
 * Attention over a context, for decoding with a full (reconstructed or
 * ordinary) KV cache: the pages' block with a real attention core instead of
 * the one-token context of lr_block_forward.  The cache is paged as the latent
 * pool is: page b holds rows b * block_rows .. b * block_rows + block_rows - 1
 * of the K and of the V pool, and a row holds one token's n_kv_heads heads of
 * head_dim elements.  lr_kv_reconstruct_paged's output, with one page a list
 * entry, is such a pool.
 *   k, v: device bf16 [pool_blocks * block_rows][ld], 16-byte aligned, ld a
 *   multiple of 8 and >= n_kv_heads * head_dim (both may point into one pool
 *   of [K | V] rows).  pool_blocks * block_rows is at most 2^31 - 1; element
 *   offsets are 64-bit. */
typedef struct {
  void* k;
  void* v;
  int64_t ld;
  int64_t pool_blocks;
  int32_t block_rows;
  int32_t n_kv_heads;
  int32_t head_dim;
} lr_kv_cache;

/* How the heads of queries and keys are prepared, for a head x of head_dim
 * elements at position p:
 *   norm != 0:  x <- x * gain / sqrt(mean(x^2) + eps);  gain: device bf16
 *               [head_dim], NULL for unit gain; q and k have their own.
 *   rot_dim > 0: the pairs (a, b) of the first rot_dim elements turn by the
 *               angles of p, (a, b) <- (a c - b s, b c + a s); pair i is
 *               (x[i], x[i + rot_dim/2]) for LR_ROT_HALF and
 *               (x[2i], x[2i+1]) for LR_ROT_PAIR; the other elements pass.
 *   cos_sin: device fp32 [max_pos][rot_dim], 16-byte aligned: the rot_dim/2
 *   cosines of a position, then the sines (lr_rope_table).
 * The arithmetic is fp32; a result is rounded once, to bf16.
 * head_dim: a multiple of 64, at most 256; rot_dim: a multiple of 16, at most
 * head_dim (LR_ERR_UNSUPPORTED otherwise). */
enum { LR_ROT_HALF = 0, LR_ROT_PAIR = 1 };
typedef struct {
  int32_t head_dim;
  int32_t norm;
  float eps;
  const void* q_gain;
  const void* k_gain;
  int32_t rot_dim;
  int32_t rot_style;
  const float* cos_sin;
  int64_t max_pos;
} lr_head_map;

/* lr_rope_table (host only): out[p][i] = cos(p f_i), out[p][rot_dim/2 + i] =
 * sin(p f_i) with f_i = theta^(-2i/rot_dim), for p < max_pos; the angle and
 * its functions are computed in 64 bits and rounded once to fp32.  out: host
 * fp32 [max_pos][rot_dim].  rot_dim positive and even, theta > 0. */
lr_status lr_rope_table(int64_t max_pos, int32_t rot_dim, double theta, float* out);

/* lr_qk_norm_rope: norm and rotation of the heads of M rows of queries and
 * keys in one pass (one launch).
 *   q: device [M][ldq] of in_dtype (LR_BF16 or LR_F32), head h in columns
 *   h * head_dim ..; k likewise with n_kv_heads heads; n_heads or n_kv_heads
 *   may be 0 (its pointers are not read).  q_out, k_out: device bf16 [M][ldqo]
 *   and [M][ldko].  A bf16 q_out may be q itself, with the same leading
 *   dimension (k_out and k likewise); any other overlap is not allowed.
 *   pos: device int32 [M], the rows' positions (not read when rot_dim is 0).
 *   n_active: device int32 or NULL; rows m >= *n_active are neither read nor
 *   written, so a captured call serves every batch up to M.
 *   Pointers 16-byte aligned, leading dimensions multiples of 8 and at least
 *   heads * head_dim.  A position outside [0, max_pos) gives a zero row and
 *   LR_ERR_INDEX_RANGE in dev_status.  M = 0 is a no-op. */
lr_status lr_qk_norm_rope(const void* q, int64_t ldq, int32_t n_heads, const void* k, int64_t ldk,
                          int32_t n_kv_heads, lr_dtype in_dtype, int64_t M, const int32_t* pos,
                          const int32_t* n_active, const lr_head_map* hm, void* q_out, int64_t ldqo,
                          void* k_out, int64_t ldko, int32_t* dev_status, lr_stream s);

/* lr_kv_append: the new tokens' keys, normed and rotated as above, and their
 * values, written to their rows of the paged cache:
 *   cache.k[rows[m]] = heads(k[m]), cache.v[rows[m]] = bf16(v[m])  for m < M.
 * With n_heads > 0 the tokens' queries are prepared in the same launch
 * (q -> q_out, as lr_qk_norm_rope).  rows: device int32 [M] (remap_build with
 * tail_rows = the new tokens of a sequence gives them); rows must be distinct.
 * A row outside the pool is skipped and reported as LR_ERR_REMAP_RANGE; a
 * position outside [0, max_pos) writes neither key nor value, gives a zero
 * query row and reports LR_ERR_INDEX_RANGE.  Other pool rows are not touched.
 * hm->head_dim must equal cache->head_dim; the other arguments and checks are
 * those of lr_qk_norm_rope. */
lr_status lr_kv_append(const void* k, int64_t ldk, const void* v, int64_t ldv, const void* q, int64_t ldq,
                       int32_t n_heads, lr_dtype in_dtype, int64_t M, const int32_t* pos,
                       const int32_t* rows, const int32_t* n_active, const lr_head_map* hm,
                       const lr_kv_cache* cache, void* q_out, int64_t ldqo, int32_t* dev_status, lr_stream s);

/* A paged cache held in 8 bits.  A pool holds codes of e4m3 (four exponent and
 * three mantissa bits, largest value 448, one NaN, no infinity), and every page
 * has a scale for each of its key heads: an element stands for
 *   code * scale[page][head],  page = row / block_rows.
 * pages: k and v point to the codes, device e4m3 [pool_blocks * block_rows][ld],
 *   16-byte aligned, ld (elements, one byte each) a multiple of 16; the other
 *   fields as for a bf16 cache.
 * k_scale, v_scale: device fp32 [pool_blocks][n_kv_heads], powers of two from
 *   2^-120 to 2^120 (lr_kv_append8 writes them so).  A scale that is none is
 *   not looked for; results over its page are then unspecified. */
typedef struct {
  lr_kv_cache pages;
  float* k_scale;
  float* v_scale;
} lr_kv_cache8;

/* lr_kv_append8: lr_kv_append to a cache held in 8 bits.  For each key head, the
 * keys (normed and rotated, fp32) and the values that go to one page:
 *   e = the least integer, -120 at least, with |x| <= 448 * 2^e for every finite
 *       element x of them;
 *   where the page's rows before the first new one hold tokens (all of them, if
 *   that one is not the page's row 0), e is no less than the page's present
 *   scale, and if it is greater the codes of those rows are made anew,
 *   code <- rn(code * old scale / 2^e);
 *   scale = 2^e, code = rn(x / scale) to the nearest e4m3, ties to even.
 * A scale only grows while a page fills, by powers of two, so that making codes
 * anew rounds nothing but what becomes e4m3-subnormal.  A NaN or infinite
 * element becomes NaN.  Other rows of the page, and other pages, are not touched.
 * The new rows of one page stand one after another in the call, in ascending
 * order without gaps, as remap_build lists them; rows that do not (one page met
 * twice, a row twice) leave that page's codes and scales unspecified.
 * A row outside the pool or a position outside [0, max_pos) is skipped and
 * reported as in lr_kv_append, and is none of the new rows above: a page without
 * another one keeps its codes and scales.  The arguments and checks are otherwise
 * lr_kv_append's. */
lr_status lr_kv_append8(const void* k, int64_t ldk, const void* v, int64_t ldv, const void* q, int64_t ldq,
                        int32_t n_heads, lr_dtype in_dtype, int64_t M, const int32_t* pos,
                        const int32_t* rows, const int32_t* n_active, const lr_head_map* hm,
                        const lr_kv_cache8* cache, void* q_out, int64_t ldqo, int32_t* dev_status, lr_stream s);

/* lr_kv_copy_pages: whole pages of caches, for forks (a sequence's last, partly
 * filled page is copied before either copy grows; full pages can be shared) and
 * for compaction:
 *   page dst[i] <- page src[i] of every cache, keys, values and scales,
 *   for 0 <= i < min(*n_pages, cap).
 *   caches: host array of n_caches (the layers of a model, as a rule); all have
 *   the same sizes and leading dimension and all are of one kind: scales NULL for
 *   bf16 (ld a multiple of 8), both given for 8 bits.  n_kv_heads * head_dim is a
 *   multiple of 16; columns past it are not copied.
 *   src, dst: device int32 [cap]; n_pages: device int32, or NULL for cap.  An
 *   entry whose source or target lies outside the pool is skipped and reported
 *   as LR_ERR_REMAP_RANGE.  All copies run at once: targets are distinct, and no
 *   target is the source of another entry (a page that two entries write, or one
 *   writes and another reads, is left unspecified).  An entry with src = dst
 *   changes nothing.  One launch for every 128 caches.  cap = 0 or n_caches = 0
 *   is a no-op. */
lr_status lr_kv_copy_pages(const lr_kv_cache8* caches, int32_t n_caches, const int32_t* src, const int32_t* dst,
                           const int32_t* n_pages, int64_t cap, int32_t* dev_status, lr_stream s);

/* lr_prefix_attention: attention of a batch whose sequences share a prefix.
 * Sequence b has the shared tokens 0 .. *prefix_len - 1, kept once in the
 * pages prefix_blocks, and lengths[b] own tokens after them in the pages of
 * row b of block_table (own token t in entry t / block_rows).  Its query rows
 * are rows q_start[b] .. q_start[b+1] - 1 of q: its last own tokens.  Row j of
 * n sees the whole prefix and the own tokens t <= lengths[b] - n + j, and
 *   out = sum_t softmax_t(scale q . k_t) v_t
 * for each of n_heads heads (query head h reads kv head h / (n_heads /
 * n_kv_heads)).  A row that sees no token comes out zero, and so does a row of
 * q that belongs to no sequence; one whose tokens all have the score minus
 * infinity is NaN, as the formula is.  Pool rows that hold no token of the batch
 * (the ends of last pages among them) do not reach the result, whatever they
 * hold, nor does a sequence's own token reach another sequence's rows.  Within
 * a sequence of several query rows a token that a row does not see has the
 * weight 0 there, which leaves a NaN or infinity among its values a NaN.
 *   q: device bf16 [M][ldq]; out: device [M][ldo] of out_dtype (LR_BF16 or
 *   LR_F32); M < 2^31; 16-byte aligned, ldq and ldo multiples of 8 and >=
 *   n_heads * head_dim.
 *   prefix_blocks: device int32 [cap_prefix_blocks]; prefix_len: device int32
 *   (both may be NULL when cap_prefix_blocks is 0: no shared part; a prefix_len
 *   that is given then has the capacity 0).
 *   q_start: device int32 [n_seq + 1], not decreasing, within [0, M]; NULL
 *   when every sequence has one row (M = n_seq then; M > n_seq leaves zero
 *   rows).  max_q: the most rows that a sequence may have (1 for NULL).
 *   block_table: device int32 [n_seq][blocks_per_seq]; lengths: device int32
 *   [n_seq].
 *   Lengths, pages and row offsets are read on the device: a captured call
 *   serves every batch within the capacities.  A length outside its capacity
 *   (block_rows times the pages it may use) is clamped and reported as
 *   LR_ERR_INDEX_RANGE (an own length only where its sequence has query rows),
 *   as is a q_start outside [0, M], one that decreases, or more than max_q rows
 *   (such a sequence's rows past max_q are unspecified).
 *   A listed page outside [0, pool_blocks) reads as zeros and reports
 *   LR_ERR_REMAP_RANGE.
 *   head_dim 64 or 128; block_rows a multiple of 16; blocks_per_seq * block_rows
 *   below 2^24; n_heads a multiple of n_kv_heads with at most 64 query heads a
 *   kv head (LR_ERR_UNSUPPORTED otherwise, LR_ERR_INVALID_ARG for a remainder); scale > 0 and finite.
 *   workspace: device, 256-byte aligned, of
 *   lr_prefix_attention_workspace_bytes(M, d) bytes (a call that needs less
 *   takes less); contents on entry do not matter; calls that share it must be
 *   ordered on one stream.  That size does not fall as M, n_seq or the numbers
 *   of pages grow, and max_q and q_start do not enter it: a workspace for a
 *   program's largest sizes serves all its calls with the same heads and page
 *   rows.  It is 512 rows of results an SM (40 MB for heads of 128) at most,
 *   unless n_kv_heads alone gives more.
 *   Scores, softmax statistics and sums are fp32; probabilities are rounded to
 *   bf16 for the second product.  The result is deterministic.  M = 0 or
 *   n_seq = 0 with M = 0 is a no-op. */
typedef struct {
  lr_kv_cache cache;
  int32_t n_heads;
  float scale;
  const int32_t* prefix_blocks;
  int32_t cap_prefix_blocks;
  const int32_t* prefix_len;
  int32_t n_seq;
  const int32_t* q_start;
  int32_t max_q;
  const int32_t* block_table;
  int32_t blocks_per_seq;
  const int32_t* lengths;
} lr_attn_desc;

size_t lr_prefix_attention_workspace_bytes(int64_t M, const lr_attn_desc* d);
lr_status lr_prefix_attention(const void* q, int64_t ldq, void* out, int64_t ldo, lr_dtype out_dtype, int64_t M,
                              const lr_attn_desc* d, void* workspace, size_t ws_bytes, int32_t* dev_status,
                              lr_stream s);

/* lr_cache_attention: lr_prefix_attention over a cache of either kind, with or
 * without a sliding window.
 *   base: as there.  With k_scale and v_scale (both or neither) the cache is held
 *   in 8 bits: base.cache is lr_kv_cache8's pages and these are its scales; else
 *   it is bf16.
 *   window: 0 for none.  With window > 0, row j of a sequence's n, at position
 *   p = *prefix_len + lengths[b] - n + j, sees of the tokens that it would see
 *   without one (the prefix's and its own, at positions 0, 1, ...) those at
 *   positions t > p - window and the first `sinks`, t < sinks (sinks >= 0, and 0
 *   without a window).  Pages that no row of the batch sees are not read; their
 *   table entries may be anything.
 *   workspace: lr_cache_attention_workspace_bytes(M, d) bytes.  As there, the rule
 *   does not fall as sizes grow, bounds every call of up to M rows, and knows neither
 *   max_q and q_start nor the window and the kind of cache; it is no less than
 *   lr_prefix_attention_workspace_bytes.
 *   What is not said here is as there, but for the arithmetic over 8 bits.  An
 *   element of a query counts to 2^-39 of its row's largest (those above 2^-28 of
 *   it, exactly); probabilities round to f16, whose small ones, under 2^-21 of the
 *   largest product of a probability and a page's scale of V, keep a multiple of
 *   2^-31 of it; values of a page whose scale of V is under 2^-60 keep a multiple of
 *   2^-84.  The V scales of one head are to lie within 2^100 of each other, any under
 *   2^-60 counting as that (keys of a smaller one may be lost from the sum).  Scores,
 *   scale q . k, are to lie under 2^22, and a row's largest finite query element times
 *   a scale of K times `scale` under 2^128 (beyond, weights may be wrong or NaN).
 *   Without a window and scales it is lr_prefix_attention. */
typedef struct {
  lr_attn_desc base;
  const float* k_scale;
  const float* v_scale;
  int32_t window;
  int32_t sinks;
} lr_cache_attn_desc;

size_t lr_cache_attention_workspace_bytes(int64_t M, const lr_cache_attn_desc* d);
lr_status lr_cache_attention(const void* q, int64_t ldq, void* out, int64_t ldo, lr_dtype out_dtype, int64_t M,
                             const lr_cache_attn_desc* d, void* workspace, size_t ws_bytes, int32_t* dev_status,
                             lr_stream s);

/* lr_block_forward_cached: the block of lr_block_forward with attention over a
 * context: n1 = RMSNorm(h); q, k, v = LR(n1); the new tokens' keys and values
 * are appended to the layer's cache (q and k normed and rotated as ctx->heads
 * says); h += LR_o(attention of q over the context); the MLP follows.
 *   h: device fp32 [M][d_model], row m the token at position pos[m] whose cache
 *   row is rows[m]; ctx->attn describes the same M rows (q_start, or one row a
 *   sequence) and its lengths count the new tokens.  The cache is this layer's;
 *   n_heads, n_kv_heads and head_dim of ctx and block must agree, and head_dim
 *   and block_rows are those that lr_prefix_attention takes.
 *   Rows m >= *n_active (NULL: none) append nothing; their h is unspecified.
 *   scratch: device, lr_block_cached_scratch_bytes(M, b, ctx) bytes, which
 *   grows with M and the context's capacities as its parts do, 256-byte
 *   aligned.  Checks, reports and capture as for the parts.  M = 0 is
 *   a no-op. */
typedef struct {
  lr_attn_desc attn;
  lr_head_map heads;
  const int32_t* pos;
  const int32_t* rows;
  const int32_t* n_active;
} lr_context;

size_t lr_block_cached_scratch_bytes(int64_t M, const lr_block_desc* b, const lr_context* ctx);
lr_status lr_block_forward_cached(float* h, int64_t M, const lr_block_desc* b, const lr_context* ctx,
                                  void* scratch, size_t scratch_bytes, int32_t* dev_status, lr_stream s);

/* ---------------------------------------------------------------------------
 * A decode step of a layer stack over fixed buffers (English page section 2.C:
 * addresses and launch parameters stay fixed while the logical batch changes):
 *   xbuf = remap_compact(pool_in); h = widen(xbuf); for each layer:
 *   lr_block_forward(h, cap rows); ybuf = bf16(h); remap_scatter(ybuf -> pool_out).
 * pool_in/pool_out: device bf16 [pool_rows][d_model] (may be the same buffer);
 * xbuf/ybuf: device bf16 [cap][d_model]; h: device fp32 [cap][d_model];
 * scratch: max over layers of lr_block_scratch_bytes(cap, layer).
 * All layers must share d_model.  Rows i >= *n_active run through the layers
 * as zero rows and are not scattered. */
enum { LR_STACK_AUTO = 0, LR_STACK_LAYERED = 1 };
typedef struct {
  int32_t n_layers;
  const lr_block_desc* layers; /* host array [n_layers]; copied by the calls */
  const void* pool_in;
  void* pool_out;
  int64_t pool_rows;
  const int32_t* remap;
  const int32_t* n_active;
  int64_t cap;
  void* xbuf;
  float* h;
  void* ybuf;
  void* scratch;
  size_t scratch_bytes;
  int32_t* dev_status;
  /* LR_STACK_AUTO (= LR_STACK_LAYERED): one launch per kernel, chained by
   * programmatic dependent launch.  Other values are rejected
   * (LR_ERR_INVALID_ARG). */
  int32_t mode;
} lr_stack_desc;

/* Scratch the step needs: the block buffers of the largest layer (layers run
 * one after another and reuse them).  Uses only n_layers, layers and cap of
 * the descriptor.  A captured graph keeps using its scratch until
 * lr_graph_destroy. */
size_t lr_stack_scratch_bytes(const lr_stack_desc* st);

/* Enqueue one step eagerly on stream s. */
lr_status lr_stack_forward(const lr_stack_desc* st, lr_stream s);

/* Capture one step into a CUDA graph owned by the library (captured on a
 * private stream; the caller's streams are not touched).  The graph keeps the
 * descriptor's device pointers: they must stay valid until lr_graph_destroy.
 * Per step only the contents of remap, *n_active and the pool change. */
typedef struct lr_graph lr_graph;
lr_status lr_graph_capture(const lr_stack_desc* st, lr_graph** out);
lr_status lr_graph_replay(lr_graph* g, lr_stream s);
lr_status lr_graph_destroy(lr_graph* g);

/* Number of kernel launches one step enqueues (eager or in the graph). */
int64_t lr_stack_launch_count(const lr_stack_desc* st);

const char* lr_status_string(lr_status st);
const char* lr_last_error(void);

/* ---------------------------------------------------------------------------
 * Testing hook (no counterpart on the pages).  lr_test_stall_producer(1) makes
 * the producers of every decode-size GEMM, every SM-pair prefill GEMM and every
 * attention launch on tensor-core tiles afterwards issue no copy, so the bounded wait of the thread that
 * consumes the copies runs out:
 * the launch reports LR_ERR_TIMEOUT through dev_status (after about two
 * seconds), releases its resources and returns, and the context stays usable.
 * lr_test_stall_producer(0) restores normal launches.  It exists for the
 * failure-detection tests only; nothing else sets it, and no environment
 * variable does. */
void lr_test_stall_producer(int32_t on);

/* Testing hook (no counterpart on the pages).  Prefill-size GEMMs (M > 256)
 * take their 256-row bands in groups, all of a group's bands for one weight
 * tile before the next; a prefill-size linear runs its down and up
 * projections in one launch, the up-projection tiles of each group placed a
 * number of groups (the lag) after that group's down-projection tiles and
 * waiting for them.  lr_test_prefill_schedule(lag, group) fixes the lag (at
 * most the number of groups) and the bands per group of later launches;
 * 0 restores the automatic choice of either, and a negative lag runs the two
 * projections as two launches.  It exists so tests can make
 * the up projection wait and vary the order of the tiles; results do not
 * depend on it.  Nothing else sets it, and no environment variable does. */
void lr_test_prefill_schedule(int32_t lag, int32_t group);

/* Testing hook (no counterpart on the pages).  lr_prefix_attention and
 * lr_cache_attention have a kernel for few query rows and one on tensor-core
 * tiles and choose by the call's sizes.  lr_test_attention_kernel(1) makes every later call take the first,
 * 2 the second, 0 restores the choice; the workspace rule follows.  It exists
 * so that tests can run both on one problem.  Nothing else sets it, and no
 * environment variable does. */
void lr_test_attention_kernel(int32_t which);


#ifdef __cplusplus
}
#endif
#endif /* LR_H_ */
