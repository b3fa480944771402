/*
 * tq.h -- C ABI of the int4 KV-cache decode path for NVIDIA GB300 (sm_103a).
 *
 * Two operations, as the pages describe the method:
 *
 *   quantize-on-store   fp16 K/V rows -> packed int4 codes + fp16 scale/bias,
 *                       written in place into a preallocated cache
 *                       ("turboquant-llama3.170B" README, decode-step listing:
 *                        RoPE, then quantize K,V to int4, then fused sdpa_int4;
 *                        "Fused int4 Attention for Gemma 4 31B", Background:
 *                        MLX-style int4 with a per-group scale and bias).
 *   fused decode attention (sdpa_int4)
 *                       one query token per sequence attends over the int4
 *                       cache; dequantisation happens in registers, softmax is
 *                       online, the sequence is split into chunks (512 tokens by
 *                       default) whose partial softmax states are merged by a
 *                       log-sum-exp reduce ("turboquant-llama3.170B" README,
 *                       kernel paragraph and split-K paragraph; Gemma page,
 *                       "What I Built Instead": sdpa_int4(Q, K_int4, V_int4)).
 *
 * Conventions shared by every entry point
 *   - All array pointers are DEVICE pointers owned by the caller.  The library
 *     allocates no device memory and keeps no per-call state between calls.
 *   - fp16 values are passed as uint16_t holding IEEE binary16 bits.
 *   - Calls are asynchronous on `stream` (a cudaStream_t passed as void*;
 *     NULL = the legacy default stream) and never synchronise the host.
 *   - Host-side argument checks run before any launch and return a status;
 *     nothing is launched when a check fails.  TQ_ERR_CUDA means a launch was
 *     attempted and CUDA reported an error; tq_last_cuda_error() returns it.
 *   - Kernels never trap.  Device-detected problems (a write position past the
 *     cache capacity, a length outside [0, max_seq_len], a pipeline wait that
 *     timed out) skip the offending work and OR a TQ_DEV_* bit into the
 *     optional `status` word (device int32, may be NULL).  The caller zeroes it
 *     when it wants to start afresh.
 *   - Inputs containing NaN or Inf give unspecified (but finite-time) results.
 *
 * Cache layout (one cache = one attention layer), all row-major:
 *   k_codes, v_codes  uint8  [batch][num_kv_heads][capacity][head_dim / 2]
 *                     element 2i of a row is the low nibble of byte i
 *                     (the Gemma page reads codes with masks 0xF, 0xF0, ...,
 *                      low nibble first)
 *   k_scale, k_bias,  fp16   [batch][num_kv_heads][capacity][head_dim / 64]
 *   v_scale, v_bias          one (scale, bias) per group of 64 consecutive
 *                            head_dim elements; value ~ scale * code + bias
 * Requirements: head_dim in {64, 128, 256}; group_size == 64; capacity a
 * positive multiple of 16; every array 16-byte aligned (256 recommended).
 */
#ifndef TQ_H
#define TQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define TQ_ABI_VERSION 2
#define TQ_GROUP_SIZE 64
#define TQ_DEFAULT_CHUNK 512

typedef enum tq_status {
    TQ_OK = 0,
    TQ_ERR_NULL = 1,        /* a required pointer is NULL */
    TQ_ERR_SHAPE = 2,       /* inconsistent or out-of-range sizes */
    TQ_ERR_CAPACITY = 3,    /* max_seq_len (or n_new) larger than the cache capacity */
    TQ_ERR_WORKSPACE = 4,   /* workspace NULL or smaller than required */
    TQ_ERR_CUDA = 5,        /* CUDA reported an error (see tq_last_cuda_error) */
    TQ_ERR_UNSUPPORTED = 6, /* head_dim / group / GQA ratio / impl not implemented */
    TQ_ERR_ALIGN = 7        /* an array is not 16-byte (workspace: 256-byte) aligned */
} tq_status;

/* Bits ORed into the optional device status word. */
#define TQ_DEV_WRITE_POS 0x1 /* append: write_pos[b] < 0 or write_pos[b] + n_new > capacity; rows skipped */
#define TQ_DEV_SEQ_LEN 0x2   /* decode: seq_lens[b] < 0 or > max_seq_len; clamped into range */
#define TQ_DEV_TIMEOUT 0x4   /* a pipeline wait exceeded its time limit; the CTA gave up, what the call wrote (also accumulated weights) is undefined */
#define TQ_DEV_PAGE 0x8      /* paged cache: a block-table entry outside [0, num_pages); page 0 used instead */
#define TQ_DEV_BLOCK 0x10    /* tq_sdpa_blocks_decode: a listed block starts at or past seq_lens[b]; left out */
#define TQ_DEV_NO_PAGE 0x20  /* tq_pages_reserve: fewer free pages than wanted; nothing was changed */
#define TQ_DEV_SOURCE 0x40   /* tq_pages_fork: sources[b] outside [-1, batch); the sequence keeps its own pages */

/* Rotation flags ("Running and Evaluating TurboQuant optimized Gemma 4",
 * TurboQuant section: vectors are rotated by the normalised Sylvester Hadamard
 * matrix H = H_n / sqrt(n) before quantisation, which spreads outliers over
 * all coordinates; H is its own inverse).  In this library H is applied by an
 * fp32 fast transform (stages h = 1, 2, ..., n/2) and rounded to fp16.
 *   TQ_ROTATE_K  keys are stored as quantize(H k); decode then uses H q, and
 *                (H q).(H k) = q.k leaves the scores unchanged.
 *   TQ_ROTATE_V  values are stored as quantize(H v); decode returns H o of the
 *                attention output o over them, which is the output over v. */
#define TQ_ROTATE_K 0x1u
#define TQ_ROTATE_V 0x2u

/* tq_decode_step_ex / tq_paged_decode_step: after the step, add n_new to
 * write_pos[b] and to seq_lens[b] on the device (both arrays are written;
 * they must not overlap).  A step captured once in a CUDA graph can then be
 * replayed token after token with no host work; the graph keeps the
 * max_seq_len it was captured with, which must stay an upper bound of the
 * advancing lengths. */
#define TQ_STEP_ADVANCE 0x100u

/* Decode implementations (tq_sdpa_int4_decode_impl and friends). */
typedef enum tq_impl {
    TQ_IMPL_AUTO = 0, /* the tensor-core path */
    TQ_IMPL_MMA = 1,  /* mma.sync tensor-core tiles fed by TMA */
    TQ_IMPL_SIMT = 2  /* CUDA-core fp32 path (comparison baseline) */
} tq_impl;

typedef struct tq_kv_cache {
    uint8_t* k_codes;  /* [B][Hkv][cap][D * bits / 8] */
    uint8_t* v_codes;  /* [B][Hkv][cap][D * bits / 8] */
    uint16_t* k_scale; /* [B][Hkv][cap][D/64] fp16 */
    uint16_t* k_bias;
    uint16_t* v_scale;
    uint16_t* v_bias;
    int32_t batch;
    int32_t num_kv_heads;
    int32_t head_dim;
    int32_t group_size; /* must be 64 */
    int32_t capacity;   /* tokens per (sequence, kv head) */
    int32_t bits;       /* code width: 4 (two codes per byte, element 2i in the low
                           nibble of byte i) or 8 (one code per byte; the
                           TurboQuant Gemma 4 page's --kv-bits 8), every
                           head_dim */
} tq_kv_cache;

/* Paged cache: a pool of pages, each holding page_tokens consecutive tokens of
 * one sequence for every kv head, and a block table mapping each sequence's
 * logical pages to pool pages (for ragged batches: the "turboquant-llama3.170B"
 * README's 18% concatenation gap is what a cache that grows by reallocation
 * costs).  Row t of (sequence b, kv head h) is row
 * t % page_tokens of head h in page block_table[b * max_pages_per_seq +
 * t / page_tokens].  The caller owns the pool and the table and allocates
 * pages before appending into them; a table entry outside [0, num_pages) sets
 * TQ_DEV_PAGE and page 0 is used instead (no fault). */
typedef struct tq_paged_kv_cache {
    uint8_t* k_codes;  /* [num_pages][Hkv][page_tokens][D * bits / 8] */
    uint8_t* v_codes;
    uint16_t* k_scale; /* [num_pages][Hkv][page_tokens][D/64] fp16 */
    uint16_t* k_bias;
    uint16_t* v_scale;
    uint16_t* v_bias;
    const int32_t* block_table; /* device [batch][max_pages_per_seq] */
    int32_t batch;
    int32_t num_kv_heads;
    int32_t head_dim;
    int32_t group_size;  /* must be 64 */
    int32_t page_tokens; /* a multiple of 128 */
    int32_t num_pages;
    int32_t max_pages_per_seq; /* logical capacity = max_pages_per_seq * page_tokens */
    int32_t bits;              /* code width, as in tq_kv_cache */
} tq_paged_kv_cache;

/* ABI version of the loaded library (TQ_ABI_VERSION it was built with). */
int32_t tq_abi_version(void);

/* Human-readable name of a status code (static string, never NULL). */
const char* tq_status_string(tq_status s);

/* The cudaError_t of the most recent TQ_ERR_CUDA on the calling host thread. */
int32_t tq_last_cuda_error(void);

/* Diagnostic of the device-side failure path (no counterpart on the pages):
 * the decode kernels wait on their pipeline stages with a time limit and,
 * when a wait runs out, OR TQ_DEV_TIMEOUT into the status word and leave.
 * This call runs that wait on one CTA: it copies 1,024 bytes from `src`
 * (device, 16-byte aligned) into shared memory and waits for the copy, then
 * waits on a barrier that nothing arrives at, giving up after `limit_us`
 * microseconds (1..100000).  It then ORs TQ_DEV_TIMEOUT into *status and
 * writes to *copied the sum (mod 2^32) of the 256 32-bit words it copied
 * (0xFFFFFFFF if even the copy had not landed).  Nothing is in flight when
 * the kernel ends.  Null pointers: TQ_ERR_NULL; misaligned src:
 * TQ_ERR_ALIGN; limit out of range: TQ_ERR_SHAPE. */
tq_status tq_wait_timeout_selftest(const void* src, int32_t* status, uint32_t limit_us,
                                   uint32_t* copied, void* stream);

/* Bytes of the six cache arrays together, each rounded up to 256 bytes, as
 * laid out by tq_kv_cache_carve.  0 for invalid sizes.  Host-only. */
size_t tq_kv_cache_bytes(int32_t batch, int32_t num_kv_heads, int32_t head_dim,
                         int32_t group_size, int32_t capacity);

/* Point the six arrays of *cache into one caller-owned allocation `base` of
 * at least tq_kv_cache_bytes(...) bytes (256-byte aligned), and fill in the
 * sizes.  Order: k_codes, v_codes, k_scale, k_bias, v_scale, v_bias.
 * Host-only (no device access). */
tq_status tq_kv_cache_carve(tq_kv_cache* cache, void* base, int32_t batch,
                            int32_t num_kv_heads, int32_t head_dim,
                            int32_t group_size, int32_t capacity);

/* The same for a code width of `bits` (4 or 8); the two functions above are
 * bits = 4 (and tq_kv_cache_carve sets cache->bits = 4). */
size_t tq_kv_cache_bytes_ex(int32_t batch, int32_t num_kv_heads, int32_t head_dim,
                            int32_t group_size, int32_t bits, int32_t capacity);
tq_status tq_kv_cache_carve_ex(tq_kv_cache* cache, void* base, int32_t batch,
                               int32_t num_kv_heads, int32_t head_dim,
                               int32_t group_size, int32_t bits, int32_t capacity);

/* Quantize-on-store.
 * k_new, v_new: fp16 [batch][num_kv_heads][n_new][head_dim], contiguous.
 * write_pos:    device int32 [batch]; token i of sequence b goes to cache row
 *               write_pos[b] + i.  The caller advances its lengths afterwards.
 * Per group of 64 elements x_0..x_63 (fp32 arithmetic, round-to-nearest-even):
 *   mn, mx = min, max;  scale = fp16(fp32(mx - mn) / 15);  bias = fp16(mn)
 *   code_i = clamp(rint(fp32(x_i - bias) / float(scale)), 0, 15), or 0 when
 *   float(scale) == 0;  a zero minimum is stored as +0, and mx is the first
 *   element holding the largest value (so a group of zeros opening with -0
 *   stores scale -0).
 * Bit-identical to the CPU oracle.  Rows with an out-of-range write position
 * are skipped and TQ_DEV_WRITE_POS is set. */
tq_status tq_quantize_kv_append(const tq_kv_cache* cache, const uint16_t* k_new,
                                const uint16_t* v_new, int32_t n_new,
                                const int32_t* write_pos, int32_t* status,
                                void* stream);

/* tq_quantize_kv_append with rotation: flags TQ_ROTATE_K / TQ_ROTATE_V rotate
 * each new K / V row by H (see the rotation flags above) before it is
 * quantized; the rotation is fused into the same kernel (no extra pass over
 * the rows).  Rotated rows are fp16_rne(fp32 transform), then quantized by the
 * rule above.  Other flag bits: TQ_ERR_UNSUPPORTED. */
tq_status tq_quantize_kv_append_ex(const tq_kv_cache* cache, const uint16_t* k_new,
                                   const uint16_t* v_new, int32_t n_new,
                                   const int32_t* write_pos, uint32_t flags,
                                   int32_t* status, void* stream);

/* out[r] = fp16_rne(H x[r]) for `rows` rows of `dim` fp16 values (dim 64, 128
 * or 256; device pointers, 16-byte aligned; out may equal x).  H as for the
 * rotation flags.  rows = 0 launches nothing. */
tq_status tq_hadamard_rotate(const uint16_t* x, int64_t rows, int32_t dim,
                             uint16_t* out, void* stream);

/* ------------------------------------------------------------ paged cache --
 * Bytes of a page pool for these sizes (the six arrays, each 256-aligned),
 * 0 for invalid sizes.  Host-only. */
size_t tq_paged_kv_cache_bytes(int32_t num_pages, int32_t num_kv_heads, int32_t head_dim,
                               int32_t group_size, int32_t bits, int32_t page_tokens);

/* Fill *cache with the arrays carved from `base` (device, 256-byte aligned,
 * tq_paged_kv_cache_bytes long) and the given block table.  Host-only. */
tq_status tq_paged_kv_cache_carve(tq_paged_kv_cache* cache, void* base, const int32_t* block_table,
                                  int32_t batch, int32_t num_kv_heads, int32_t head_dim,
                                  int32_t group_size, int32_t bits, int32_t page_tokens,
                                  int32_t num_pages, int32_t max_pages_per_seq);

/* tq_quantize_kv_append_ex into a paged cache (rows through the block table). */
tq_status tq_paged_quantize_kv_append(const tq_paged_kv_cache* cache, const uint16_t* k_new,
                                      const uint16_t* v_new, int32_t n_new,
                                      const int32_t* write_pos, uint32_t flags,
                                      int32_t* status, void* stream);

/* tq_sdpa_int4_decode_ex / tq_decode_step_ex over a paged cache: the same
 * arithmetic and, for chunk >= 128, the same split plan as the contiguous
 * cache (runs start on page-aligned tile boundaries; smaller chunks are
 * raised to the tile), so the results are identical to a contiguous cache
 * holding the same rows.  Tensor-core path only. */
tq_status tq_paged_sdpa_int4_decode(const tq_paged_kv_cache* cache, const uint16_t* q,
                                    int32_t num_q_heads, const int32_t* seq_lens,
                                    int32_t max_seq_len, float attn_scale, int32_t chunk,
                                    uint32_t flags, void* workspace, size_t workspace_bytes,
                                    uint16_t* out, int32_t* status, void* stream);
tq_status tq_paged_decode_step(const tq_paged_kv_cache* cache, const uint16_t* k_new,
                               const uint16_t* v_new, int32_t n_new, const int32_t* write_pos,
                               const uint16_t* q, int32_t num_q_heads, const int32_t* seq_lens,
                               int32_t max_seq_len, float attn_scale, int32_t chunk, uint32_t flags,
                               void* workspace, size_t workspace_bytes, uint16_t* out,
                               int32_t* status, void* stream);

/* ------------------------------------------------------------ host buffers --
 * tq_decode_step_ex with the step's inputs and output in host memory: copies
 * q [batch][num_q_heads][head_dim] and k_new / v_new [batch][Hkv][n_new][D]
 * (fp16, host; page-locked for the copies to be asynchronous) into `staging`
 * (device, 256-byte aligned, tq_host_staging_bytes long), runs the step, and
 * copies the fp16 output back to h_out (host).  Everything is queued on
 * `stream` in one call (no host synchronisation): h_out holds the result once
 * the stream has reached it.  write_pos, seq_lens, workspace and status stay
 * device-side, as for tq_decode_step_ex.  The call a serving loop makes once
 * per step when its activations live on the host.  When all four host buffers
 * are page-locked and mapped (cudaHostAlloc, torch pin_memory) the kernels
 * read and write them in place (GPU-addressable host memory, NVLink-C2C on
 * Grace-Blackwell) and `staging` is not touched. */
size_t tq_host_staging_bytes(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                             int32_t head_dim, int32_t n_new);
tq_status tq_decode_step_host(const tq_kv_cache* cache, const uint16_t* h_k_new,
                              const uint16_t* h_v_new, int32_t n_new, const int32_t* write_pos,
                              const uint16_t* h_q, int32_t num_q_heads, const int32_t* seq_lens,
                              int32_t max_seq_len, float attn_scale, int32_t chunk, uint32_t flags,
                              void* workspace, size_t workspace_bytes, void* staging,
                              size_t staging_bytes, uint16_t* h_out, int32_t* status, void* stream);

/* Workspace bytes tq_sdpa_int4_decode needs for these sizes (an upper bound
 * that does not depend on the device).  Host-only. */
size_t tq_sdpa_workspace_bytes(int32_t batch, int32_t num_q_heads,
                               int32_t num_kv_heads, int32_t head_dim,
                               int32_t max_seq_len, int32_t chunk);

/* Fused int4 decode attention (Sq = 1, GQA).
 * q:        fp16 [batch][num_q_heads][head_dim]; query head h reads KV head
 *           h / (num_q_heads / num_kv_heads)  (num_q_heads / num_kv_heads <= 8)
 * seq_lens: device int32 [batch]; sequence b attends to cache rows
 *           [0, seq_lens[b]); 0 gives an all-zero output row
 * max_seq_len: host bound on seq_lens (1 <= max_seq_len <= capacity); sizes the grid
 * attn_scale: multiplies q.k (1/sqrt(head_dim) for Llama, 1.0 for Gemma)
 * chunk:    split-K chunk in tokens (multiple of 16; TQ_DEFAULT_CHUNK = 512).
 *           The sequence is split into balanced runs, one per CTA, of whole
 *           units of min(chunk, pipeline tile) tokens (the tile is 384 tokens
 *           for contiguous int4 caches at head_dim 128, else 128 tokens when a
 *           token's codes take under 128 bytes, 64 otherwise); each run
 *           keeps one running softmax
 *           state and the runs' states are merged by a log-sum-exp reduce
 *           (tq_sdpa_int4_reduce; with at most 8 runs in a grid of one wave the
 *           runs of each (sequence, kv head) form one thread-block cluster and
 *           merge in phase 1 with the reduce's operations, bit for bit the same
 *           output).  The result is the same as merging one state per chunk
 *           (see tq_sdpa_int4_partial with chunks_per_split = 1).
 * workspace: device scratch (256-byte aligned) of at least
 *           tq_sdpa_workspace_bytes(...) bytes holding the fp32 partial states,
 *           room for a rotated query and, for batches whose grid spans several
 *           waves, the device-computed dispatch order of the runs (longest
 *           first); contents on entry are ignored.
 * out:      fp16 [batch][num_q_heads][head_dim], round-to-nearest-even.
 * Accumulation is fp32; result within 2e-3 abs / 1e-3 rel-L2 of fp64 attention
 * over the dequantised cache. */
tq_status tq_sdpa_int4_decode(const tq_kv_cache* cache, const uint16_t* q,
                              int32_t num_q_heads, const int32_t* seq_lens,
                              int32_t max_seq_len, float attn_scale,
                              int32_t chunk, void* workspace,
                              size_t workspace_bytes, uint16_t* out,
                              int32_t* status, void* stream);

/* Same as tq_sdpa_int4_decode with an explicit implementation choice. */
tq_status tq_sdpa_int4_decode_impl(const tq_kv_cache* cache, const uint16_t* q,
                                   int32_t num_q_heads, const int32_t* seq_lens,
                                   int32_t max_seq_len, float attn_scale,
                                   int32_t chunk, void* workspace,
                                   size_t workspace_bytes, uint16_t* out,
                                   int32_t* status, tq_impl impl, void* stream);

/* One decode step: quantize-on-store of the new tokens, then fused int4 decode
 * attention over the cache that now holds them ("turboquant-llama3.170B"
 * README, decode-step listing: quantize K,V to int4, then fused sdpa_int4).
 * Arguments as tq_quantize_kv_append and tq_sdpa_int4_decode (tensor-core
 * path); results identical to calling the two in order on `stream`.  The
 * decode launch may start while the append still runs and waits for it only
 * in the CTAs whose runs read an appended row.  seq_lens must already count
 * the new tokens (typically write_pos[b] + n_new). */
tq_status tq_decode_step(const tq_kv_cache* cache, const uint16_t* k_new,
                         const uint16_t* v_new, int32_t n_new,
                         const int32_t* write_pos, const uint16_t* q,
                         int32_t num_q_heads, const int32_t* seq_lens,
                         int32_t max_seq_len, float attn_scale, int32_t chunk,
                         void* workspace, size_t workspace_bytes,
                         uint16_t* out, int32_t* status, void* stream);

/* Decode over a cache written with rotation flags (the same flags as its
 * appends): TQ_ROTATE_K rotates the query (into the workspace) before phase
 * 1; TQ_ROTATE_V applies H to the merged output before its fp16 rounding.
 * Otherwise as tq_sdpa_int4_decode / tq_decode_step (a rotated step appends
 * its rows inside the decode kernel like an unrotated one, rotating each row
 * across the lanes that hold it). */
tq_status tq_sdpa_int4_decode_ex(const tq_kv_cache* cache, const uint16_t* q,
                                 int32_t num_q_heads, const int32_t* seq_lens,
                                 int32_t max_seq_len, float attn_scale, int32_t chunk,
                                 uint32_t flags, void* workspace, size_t workspace_bytes,
                                 uint16_t* out, int32_t* status, void* stream);
tq_status tq_decode_step_ex(const tq_kv_cache* cache, const uint16_t* k_new,
                            const uint16_t* v_new, int32_t n_new,
                            const int32_t* write_pos, const uint16_t* q,
                            int32_t num_q_heads, const int32_t* seq_lens,
                            int32_t max_seq_len, float attn_scale, int32_t chunk,
                            uint32_t flags, void* workspace, size_t workspace_bytes,
                            uint16_t* out, int32_t* status, void* stream);

/* The split plan tq_sdpa_int4_decode uses on the current device: *n_splits
 * runs per (sequence, kv head), the longest *max_run_tokens tokens long.
 * Host-side query (reads device attributes). */
tq_status tq_sdpa_plan(const tq_kv_cache* cache, int32_t num_q_heads,
                       int32_t max_seq_len, int32_t chunk, tq_impl impl,
                       int32_t* n_splits, int32_t* max_run_tokens);

/* The split plan rule itself, without a device: the runs per (sequence, kv
 * head) for `batch` sequences of up to `max_seq_len` tokens, `num_kv_heads`
 * kv heads, runs made of whole units of min(chunk, tile_tokens) tokens, on a
 * device that holds `resident_ctas` phase-1 CTAs at once (tq_sdpa_plan passes
 * the SM count x the CTAs per SM and the kernel's tile: 384 tokens for a
 * contiguous int4 cache at head_dim 128, one CTA per SM; else 128 tokens when a
 * token's codes take under 128 bytes, 64 otherwise).  Picks the run count
 * n <= min(units, 2048 / (batch * num_kv_heads)) that minimises, with
 * W = ceil(batch * num_kv_heads * n / resident_ctas) waves,
 *   W * (ceil(units / n) * unit + 2 * tile_tokens) + R,
 * R = tile_tokens for the reduce, or 0 when `merge` is nonzero and the
 * decode merges the runs itself (n = 1, or n <= 8 with W = 1: one
 * thread-block cluster per sequence and kv head); the fewest runs on a tie.
 * tq_sdpa_plan passes merge = 1 (0 for the CUDA-core implementation); steps
 * with TQ_ROTATE_V or TQ_STEP_ADVANCE, whose reduce has other work, plan with
 * merge = 0.  Chunk and tile_tokens must be positive multiples of 16 and every
 * count positive (TQ_ERR_SHAPE), the outputs non-null (TQ_ERR_NULL).  Pure
 * host arithmetic. */
tq_status tq_split_plan(int32_t batch, int32_t num_kv_heads, int32_t max_seq_len,
                        int32_t chunk, int32_t tile_tokens, int32_t resident_ctas,
                        int32_t merge, int32_t* n_splits, int32_t* max_run_tokens);

/* Split-K phase 1 alone ("turboquant-llama3.170B" README, split-K paragraph:
 * Phase 1 = partial attention over 512-token chunks processed in parallel).
 * Each part covers `chunks_per_split` consecutive chunks (1 = one state per
 * chunk, the pages' form), np = ceil(ceil(max_seq_len / chunk) /
 * chunks_per_split); or, with chunks_per_split = 0, the runs
 * tq_sdpa_int4_decode uses (np = n_splits of tq_sdpa_plan).  fp32 outputs:
 *   part_m   [batch][num_q_heads][np]  max over the part of the scaled score
 *            (natural-log units; -inf for an empty part)
 *   part_l   [batch][num_q_heads][np]  sum of exp(score - m)  (0 if empty)
 *   part_acc [batch][num_q_heads][np][head_dim]  sum of exp(score - m) * v
 * Parts past seq_lens[b] are empty.  Arrays must hold np entries per (b, h). */
tq_status tq_sdpa_int4_partial(const tq_kv_cache* cache, const uint16_t* q,
                               int32_t num_q_heads, const int32_t* seq_lens,
                               int32_t max_seq_len, float attn_scale,
                               int32_t chunk, int32_t chunks_per_split,
                               float* part_m, float* part_l, float* part_acc,
                               int32_t* status, tq_impl impl, void* stream);

/* Expand rows [0, n_rows) of every (sequence, KV head) of the cache into fp16
 * K and V, k_out / v_out [batch][num_kv_heads][n_rows][head_dim] (device,
 * caller-owned, 16-byte aligned):
 *   value = fp16_rne(fp32(scale * code + bias))
 * (one fp32 rounding -- the product is exact -- then RNE to binary16).  This
 * is the float cache of the dequantize-then-attend decode that the fused
 * kernel replaces ("Fused int4 Attention for Gemma 4 31B on Apple Silicon",
 * What I Built Instead); it is here as that comparison point, not as a step of
 * the fused path.  Errors: TQ_ERR_NULL, TQ_ERR_SHAPE (n_rows < 0),
 * TQ_ERR_CAPACITY (n_rows > capacity), TQ_ERR_ALIGN, plus the cache checks.
 * n_rows = 0 launches nothing. */
tq_status tq_dequantize_kv(const tq_kv_cache* cache, int32_t n_rows,
                           uint16_t* k_out, uint16_t* v_out, void* stream);

/* Split-K phase 2 alone ("Phase 2 (reduce)" of the same paragraph): per (b, h),
 *   M = max over parts with l > 0 of m,  w_c = exp(m_c - M),
 *   out = sum_c w_c acc_c / sum_c w_c l_c   (fp16, RNE; all-empty rows -> 0).
 * Inputs laid out as tq_sdpa_int4_partial writes them, n_parts per (b, h),
 * 1 <= n_parts <= 8192. */
tq_status tq_sdpa_int4_reduce(const float* part_m, const float* part_l,
                              const float* part_acc, int32_t batch,
                              int32_t num_q_heads, int32_t head_dim,
                              int32_t n_parts, uint16_t* out, void* stream);

/* Size of the library-owned device array tq_sdpa_int4_decode_noalloc keeps its
 * partial states in (per GPU that loads the library, held until exit). */
#define TQ_NOALLOC_SCRATCH_BYTES (4u << 20)

/* Fused int4 decode attention for callers that cannot allocate device memory.
 * The pages have no counterpart of this entry point.  It is
 * tq_sdpa_int4_decode (tensor-core path) without the workspace argument: the
 * split-K partial states go to a fixed TQ_NOALLOC_SCRATCH_BYTES device array
 * inside the library, so the call allocates nothing.  Meant for callers that
 * have no allocator at hand or may not use one: code in host callbacks or
 * other paths where cudaMalloc is forbidden, plugins of frameworks that own
 * all device memory, plain C programs that link only this library.
 *   - Same arguments, layouts and results as tq_sdpa_int4_decode, bit for
 *     bit (the same plan and kernels).  One difference in speed: batches
 *     whose grid spans several waves run in grid order, without the
 *     longest-run-first dispatch pass of the workspace decode.
 *   - Requests whose partial states do not fit the array return
 *     TQ_ERR_WORKSPACE before any launch.  They need, with P = batch *
 *     num_q_heads * n_splits (n_splits as tq_sdpa_plan reports) and A(n) = n
 *     rounded up to a multiple of 256,  2 * A(4 P) + 4 P * head_dim  bytes
 *     (m and l, each 256-byte aligned, then acc).
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress, with that device current); make that first call
 *     before any stream capture.  The address is kept per device and looked
 *     up again when the device has a new context (after cudaDeviceReset);
 *     make that next call before any capture too.
 *   - All calls on a device share the array and it keeps the last call's
 *     contents; nothing in it needs clearing (each call writes every element
 *     it reads), but calls that overlap on the GPU (other streams, other host
 *     threads) race on it and may return wrong results: serialise them. */
tq_status tq_sdpa_int4_decode_noalloc(const tq_kv_cache* cache, const uint16_t* q,
                                      int32_t num_q_heads, const int32_t* seq_lens,
                                      int32_t max_seq_len, float attn_scale,
                                      int32_t chunk, uint16_t* out,
                                      int32_t* status, void* stream);

/* ------------------------------------------------------- rotary positions --
 * Turns query and key rows by rotary positions with up to four axes (time,
 * height, width, ... of text, images and video), from the projections' layout
 * into the append's ("turboquant-llama3.170B" README, decode-step listing:
 * RoPE comes before the quantize-on-store).
 * Pair i (0 <= i < rotary_dim / 2) of a row at position t of sequence b turns by
 *   angle = positions[axis(i)][b][t] * inv_freq[i],
 * where the first sections[0] pairs follow axis 0, the next sections[1] axis 1,
 * and so on.  A pair is (x_i, x_{i + rotary_dim/2}), or with TQ_ROPE_PAIRS
 * (x_{2i}, x_{2i+1}); it becomes (x1 cos - x2 sin, x2 cos + x1 sin), computed
 * in fp32 from an angle reduced in fp64 and rounded once.  Elements from
 * rotary_dim on are copied.  TQ_ROPE_INVERSE turns by -angle: the transpose,
 * hence also the gradient of the rows.
 *   q, k       tq_rope_rows each (k may be NULL): x[b * stride_b + t * stride_t
 *              + h * stride_h + d] in, out [batch][num_heads][n][head_dim]
 *              contiguous; strides in elements, multiples of 8, not negative
 *   positions  device int32 [n_axes][batch][n] (any value, also negative)
 *   inv_freq   device fp32 [rotary_dim / 2]
 *   sections   HOST int32 [n_axes], sum rotary_dim / 2 (zeros allowed)
 * head_dim 64, 128 or 256; rotary_dim a multiple of 16 up to head_dim; batch
 * and heads up to 65,535; n = 0 launches nothing.  An out that overlaps an x or the other
 * out: TQ_ERR_SHAPE. */
#define TQ_ROPE_PAIRS 0x1u
#define TQ_ROPE_INVERSE 0x2u
#define TQ_ROPE_MAX_AXES 4
typedef struct tq_rope_rows {
    const uint16_t* x;
    uint16_t* out;
    int64_t stride_b, stride_t, stride_h;
    int32_t num_heads;
} tq_rope_rows;
tq_status tq_rope_axes(const tq_rope_rows* q, const tq_rope_rows* k, const int32_t* positions,
                       const float* inv_freq, int32_t n_axes, const int32_t* sections, int32_t batch,
                       int32_t n, int32_t head_dim, int32_t rotary_dim, uint32_t flags, void* stream);

/* ----------------------------------------------------------- sparse decode --
 * Decode attention over the blocks of cached tokens that a cheap score selects
 * for the query, instead of all of them.  Blocks are block_tokens = 32, 64 or
 * 128 consecutive tokens of a sequence; block j holds rows
 * [j * block_tokens, (j + 1) * block_tokens).  Works on every cache the decode
 * works on (int4 and int8, contiguous and paged, rotated with the flags it was
 * written with).
 *
 * Bounds: for every block and kv head the least and the greatest cached key of
 * each channel, fp16 [batch][num_kv_heads][ceil(capacity / block_tokens)][2]
 * [head_dim] (0: least, 1: greatest), of the keys scale * code + bias rounded to
 * the nearest fp16 (the decode does not round them); of the rotated keys where
 * keys are stored rotated.  Keys that are no numbers (an infinite scale times
 * code 0, say) are left out of them.  tq_block_bounds_bytes: their size (0 for
 * invalid sizes).
 * tq_kv_block_bounds recomputes the bounds of every block that rows
 * [start[b], start[b] + n_rows) of sequence b touch, from the block's rows
 * below start[b] + n_rows: call it after each append (the prompt's too) with
 * where it wrote and n_new.  (A step with TQ_STEP_ADVANCE has moved write_pos on:
 * where it wrote is the value before.)  Caches of up to 2^30 tokens (all the entry points from here on).
 * Other blocks are left as they were.  A range outside the cache sets
 * TQ_DEV_WRITE_POS and leaves that sequence out. */
size_t tq_block_bounds_bytes(int32_t batch, int32_t num_kv_heads, int32_t head_dim, int32_t capacity,
                             int32_t block_tokens);
tq_status tq_kv_block_bounds(const tq_kv_cache* cache, int32_t block_tokens, const int32_t* start,
                             int32_t n_rows, uint16_t* bounds, int32_t* status, void* stream);
tq_status tq_paged_kv_block_bounds(const tq_paged_kv_cache* cache, int32_t block_tokens,
                                   const int32_t* start, int32_t n_rows, uint16_t* bounds,
                                   int32_t* status, void* stream);

/* Selection: blocks [batch][num_kv_heads][n_select], ascending, -1 behind the
 * last where a sequence has fewer.  With nb = ceil(seq_lens[b] / block_tokens):
 * all of them if nb <= n_select; else the first n_first, the last n_last and,
 * of the others, the n_select - n_first - n_last of greatest score
 *   max over the kv head's query heads of  sum_d max(q_d least_d, q_d greatest_d),
 * which no q.k of the block exceeds by more than its keys' rounding, 2^-11
 * sum_d |q_d k_d| (2^-25 |q_d| where fp16 is subnormal).  Equal scores: the
 * lowest index first.  The order is that of the exact scores of these bounds
 * (blocks whose fp32 scores are too close to the border are scored again to 48
 * bits, in the workspace).  With a query or bounds that are no numbers the list
 * holds blocks of the sequence or -1, but which is not said.
 * n_first + n_last <= n_select; at most 22,528 blocks (TQ_ERR_UNSUPPORTED).
 * What the bounds of always listed blocks hold does not matter.  Where a copy
 * gave up (TQ_DEV_TIMEOUT), the places of the scored blocks are -1.
 * The bounds are those of a cache of `capacity` tokens.  flags: TQ_ROTATE_K
 * where its keys are stored rotated (TQ_ROTATE_V is ignored).
 * workspace: tq_sparse_workspace_bytes(...) bytes, 256-byte aligned, one per
 * call in flight. */
size_t tq_sparse_workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                 int32_t head_dim, int32_t max_seq_len, int32_t n_select,
                                 int32_t block_tokens);
tq_status tq_select_blocks(const uint16_t* bounds, const uint16_t* q, int32_t batch, int32_t num_q_heads,
                           int32_t num_kv_heads, int32_t head_dim, int32_t capacity,
                           const int32_t* seq_lens, int32_t max_seq_len, int32_t block_tokens,
                           int32_t n_select, int32_t n_first, int32_t n_last, uint32_t flags,
                           void* workspace, size_t workspace_bytes, int32_t* blocks, int32_t* status,
                           void* stream);

/* The decode (tq_sdpa_int4_decode_ex) over the rows below seq_lens[b] of the
 * listed blocks: blocks [batch][num_kv_heads][n_select], entries below 0 are
 * empty, an entry that starts at or past seq_lens[b] sets TQ_DEV_BLOCK and is
 * left out.  Any order; a block listed twice counts twice.  A kv head whose
 * list is empty gives zero output rows.  Precision as the decode's, and as
 * there rows whose scale or bias is not finite leave their heads' outputs
 * undefined. */
tq_status tq_sdpa_blocks_decode(const tq_kv_cache* cache, const uint16_t* q, int32_t num_q_heads,
                                const int32_t* seq_lens, int32_t max_seq_len, float attn_scale,
                                const int32_t* blocks, int32_t n_select, int32_t block_tokens,
                                uint32_t flags, void* workspace, size_t workspace_bytes, uint16_t* out,
                                int32_t* status, void* stream);
tq_status tq_paged_sdpa_blocks_decode(const tq_paged_kv_cache* cache, const uint16_t* q,
                                      int32_t num_q_heads, const int32_t* seq_lens, int32_t max_seq_len,
                                      float attn_scale, const int32_t* blocks, int32_t n_select,
                                      int32_t block_tokens, uint32_t flags, void* workspace,
                                      size_t workspace_bytes, uint16_t* out, int32_t* status,
                                      void* stream);

/* Both in one call: the selection into `blocks`, then the decode over it. */
tq_status tq_sparse_decode(const tq_kv_cache* cache, const uint16_t* bounds, const uint16_t* q,
                           int32_t num_q_heads, const int32_t* seq_lens, int32_t max_seq_len,
                           float attn_scale, int32_t block_tokens, int32_t n_select, int32_t n_first,
                           int32_t n_last, uint32_t flags, void* workspace, size_t workspace_bytes,
                           int32_t* blocks, uint16_t* out, int32_t* status, void* stream);
tq_status tq_paged_sparse_decode(const tq_paged_kv_cache* cache, const uint16_t* bounds, const uint16_t* q,
                                 int32_t num_q_heads, const int32_t* seq_lens, int32_t max_seq_len,
                                 float attn_scale, int32_t block_tokens, int32_t n_select,
                                 int32_t n_first, int32_t n_last, uint32_t flags, void* workspace,
                                 size_t workspace_bytes, int32_t* blocks, uint16_t* out, int32_t* status,
                                 void* stream);

/* --------------------------------------------------------------- eviction --
 * The decode (tq_sdpa_int4_decode_ex) that also keeps account of what was
 * attended to: for every row t < seq_lens[b] of kv head h
 *   weights[b][h][t] = decay * weights[b][h][t] + sum over the kv head's query
 *                      heads of softmax(attn_scale q.K)_t
 * (decay = 0: the old value is not read).  weights: fp32 [batch][num_kv_heads]
 * [capacity]; rows from seq_lens[b] on are neither read nor written, so the
 * caller zeroes a row's weight no later than its append (an array that starts
 * as zeros, or that tq_kv_evict wrote, is ready).  A query head whose every
 * score is -inf adds nothing; where scores are no numbers, outputs and weights
 * of their kv head are undefined.  A weight is as exact as the
 * scores in fp32 leave it.  With S the largest |attn_scale| sum_d |q_d| (scale
 * code_d + |bias_d|) of a row (q as it meets the keys: rotated and rounded where
 * they are), a head's weights are within 1e-5 relative (L2) of fp64 over the same
 * cache where S is at most 64.  Above, the error grows with S: 1e-7 S over a
 * head's rows, 2.5e-7 S for a single one are the most that was measured, 2e-5 S
 * what the sums allow.
 * workspace: tq_weights_workspace_bytes(...) bytes (the scores, 4 bytes per
 * query head and token of max_seq_len, and the decode's), 256-byte aligned, one
 * per call in flight. */
size_t tq_weights_workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                  int32_t head_dim, int32_t max_seq_len);
tq_status tq_sdpa_decode_weights(const tq_kv_cache* cache, const uint16_t* q, int32_t num_q_heads,
                                 const int32_t* seq_lens, int32_t max_seq_len, float attn_scale,
                                 float decay, float* weights, uint32_t flags, void* workspace,
                                 size_t workspace_bytes, uint16_t* out, int32_t* status, void* stream);
tq_status tq_paged_sdpa_decode_weights(const tq_paged_kv_cache* cache, const uint16_t* q,
                                       int32_t num_q_heads, const int32_t* seq_lens, int32_t max_seq_len,
                                       float attn_scale, float decay, float* weights, uint32_t flags,
                                       void* workspace, size_t workspace_bytes, uint16_t* out,
                                       int32_t* status, void* stream);

/* Eviction by weight: of every (sequence, kv head) of src with more than `keep`
 * rows, the last `recent` rows and, of the rows before them, the keep - recent
 * of greatest weight (equal weights, and -0 and 0, the lowest row first) move,
 * in their order, to rows [0, keep) of dst; one with at most `keep` rows moves
 * whole.  Codes, scales and biases are copied as they are.
 *   weights      fp32 [batch][num_kv_heads][src capacity], 16-byte aligned
 *   dst_weights  fp32 [batch][num_kv_heads][dst capacity]: the kept rows'
 *                weights, zeros behind them
 *   dst_lens     int32 [batch]: min(seq_lens[b], keep)
 *   kept         int32 [batch][num_kv_heads][keep]: the src row of each dst
 *                row, -1 behind the last
 * Rows of dst behind the kept ones are left as they were; dst's block bounds are
 * the caller's to recompute.  Weights that are no numbers may rank anywhere.
 * Both caches have the same batch, heads, head_dim and bits; 0 <= recent <= keep
 * <= dst capacity; batch * num_kv_heads <= 65,535.  What is written (dst's
 * arrays, dst_weights, dst_lens, kept) must not overlap what is read (src's
 * arrays, the tables, weights, seq_lens) or one another (TQ_ERR_SHAPE); paged
 * caches may share a pool (the same six arrays and page size; not the table),
 * but a page in both tables (or twice in dst's) gives undefined rows. */
tq_status tq_kv_evict(const tq_kv_cache* src, const tq_kv_cache* dst, const float* weights,
                      const int32_t* seq_lens, int32_t max_seq_len, int32_t keep, int32_t recent,
                      float* dst_weights, int32_t* dst_lens, int32_t* kept, int32_t* status, void* stream);
tq_status tq_paged_kv_evict(const tq_paged_kv_cache* src, const tq_paged_kv_cache* dst,
                            const float* weights, const int32_t* seq_lens, int32_t max_seq_len,
                            int32_t keep, int32_t recent, float* dst_weights, int32_t* dst_lens,
                            int32_t* kept, int32_t* status, void* stream);

/* ------------------------------------------------------ several query rows --
 * Attention of a chunk of new tokens over the cache that already holds them (a
 * prompt, a piece of one, drafted tokens to be checked), and cross attention
 * over an encoder's states held in a cache.
 *   q         tq_query_rows: x[b * stride_b + h * stride_h + t * stride_t + d],
 *             n rows of num_heads heads per sequence; strides in elements,
 *             multiples of 8, not negative.  (tq_rope_axes writes rows so:
 *             [batch][num_heads][n][head_dim].)
 *   q_lens    device int32 [batch]: how many of the n rows are sequence b's; NULL:
 *             all.  Rows behind them are not read, and out is left as it was there.
 *   seq_lens  device int32 [batch]: the rows of the cache, the chunk's included
 * Row i < q_lens[b] stands at position p = seq_lens[b] - q_lens[b] + i and attends
 * to the cached rows t <= p, of them the last `window` ones where window > 0.
 * TQ_CHUNK_FULL: every row attends to all of [0, seq_lens[b]) (window must be 0).
 * A row with nothing to attend to (p < 0, an empty sequence) is a row of zeros.
 *   out       fp16 [batch][n][num_heads][head_dim], contiguous: the rows that an
 *             output projection takes
 * out, the workspace and the status word must not overlap one another, the span from
 * q's first row to its last, the lengths or the cache (TQ_ERR_SHAPE).
 * Head grouping, lengths and max_seq_len, attn_scale and the rotation flags as in
 * tq_sdpa_int4_decode_ex; lengths outside [0, n] and [0, max_seq_len] are clamped
 * and set TQ_DEV_SEQ_LEN.
 * Cached values enter as scale * code + bias rounded to fp16 (above 65,504: that),
 * softmax weights as fp16, queries turned for TQ_ROTATE_K as fp16 again; sums and
 * softmax states are fp32.  So against fp64 attention over the dequantised cache a score
 * is off by 2^-11 attn_scale sum_d |q_d K_d| at most (with TQ_ROTATE_K by twice that),
 * and an output by what such scores make of it, 2^-10 sum_t p_t |V_t| and its own
 * rounding (all rows together: 4e-4 rel-L2 for normally distributed rows, up to 1.5e-3
 * with a key channel twenty times as large).  Weights below 2^-21 of a row's largest,
 * p_max, have fewer bits: the tokens t that hold them add up to 2^-32 p_max sum_t |V_t|.
 * The tensor cores' sums are cut off, not rounded: at most 2^-11 sum_t p_t |V_t| of an
 * output (5e-5 of it where all values have one sign), whatever the length.  Scores from
 * some 10^6 on in magnitude leave fp32 too few bits for a softmax: rows that have such
 * are undefined.  Cached rows whose scale or bias is not finite leave the outputs of the
 * rows that attend to them undefined, and no others; so do query rows that are not
 * finite for themselves.
 * One contiguous row per sequence (n = 1, no q_lens, no window) is that decode itself,
 * which rounds no key: closer than the same row passed in another way.
 * workspace: tq_chunk_workspace_bytes(...) bytes, 256-byte aligned, one per call in
 * flight (not looked at where n = 0; past 8,192 tokens it holds the output's rows in
 * fp32); it also serves fewer rows, sequences and tokens of the same heads.  n = 0
 * launches nothing.  batch and kv heads up to 65,535, n * num_heads up to 2^28, tiles of
 * 128 rows over all sequences and kv heads below 2^30, caches up to 2^30 tokens. */
#define TQ_CHUNK_FULL 0x200u
typedef struct tq_query_rows {
    const uint16_t* x;
    int64_t stride_b, stride_h, stride_t;
    int32_t num_heads;
    int32_t n;
} tq_query_rows;
size_t tq_chunk_workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                int32_t head_dim, int32_t n, int32_t max_seq_len);
tq_status tq_sdpa_chunk(const tq_kv_cache* cache, const tq_query_rows* q, const int32_t* q_lens,
                        const int32_t* seq_lens, int32_t max_seq_len, float attn_scale, int32_t window,
                        uint32_t flags, void* workspace, size_t workspace_bytes, uint16_t* out,
                        int32_t* status, void* stream);
tq_status tq_paged_sdpa_chunk(const tq_paged_kv_cache* cache, const tq_query_rows* q, const int32_t* q_lens,
                              const int32_t* seq_lens, int32_t max_seq_len, float attn_scale,
                              int32_t window, uint32_t flags, void* workspace, size_t workspace_bytes,
                              uint16_t* out, int32_t* status, void* stream);

/* Diagnostic of the failure path inside the kernel of tq_sdpa_chunk: the same call
 * (causal, no q_lens, no window, every n in tiles) whose CTAs bring `copies` tiles of
 * keys and values each (0 and up) and then no more.  What waits for the next ones gives up
 * after limit_us microseconds (1..100000; tq_sdpa_chunk itself: 2 s) and sets
 * TQ_DEV_TIMEOUT in *status (not NULL); nothing is in flight when the kernel ends, and
 * what it wrote to out is undefined.  With no fewer copies than there are (two for each
 * 128 tokens, or 64 at head_dim 256) it is that call's result. */
tq_status tq_chunk_timeout_selftest(const tq_kv_cache* cache, const tq_query_rows* q, const int32_t* seq_lens,
                                    int32_t max_seq_len, float attn_scale, uint32_t limit_us, int32_t copies,
                                    void* workspace, size_t workspace_bytes, uint16_t* out, int32_t* status,
                                    void* stream);

/* --------------------------------------------------------- pages of a pool --
 * Keeps account of a paged cache's pages on the device.  The caller owns
 *   refs   int32 [num_pages]: how many table entries name each page (0: free); a
 *          caller that keeps a page in a list of its own adds to it
 *   held   int32 [batch]: sequence b's pages are the first held[b] entries of its
 *          row of cache->block_table, which these calls write
 * all zeros for a pool without sequences.  A pool that several caches share (tables
 * of their own over the same arrays) takes one refs.  Entries outside the pool and
 * held[b] outside [0, max_pages_per_seq] set TQ_DEV_PAGE and count for nothing (held[b]
 * as the nearest bound).  A page's codes are below 2^31 bytes, tables and pools of up to
 * 2^30 entries (TQ_ERR_SHAPE).
 * The arrays, the workspace, the tables and the cache's arrays must not overlap
 * (TQ_ERR_SHAPE; but see tq_pages_compact).
 * workspace: tq_pages_workspace_bytes(...) bytes, 256-byte aligned, one per call in
 * flight. */
size_t tq_pages_workspace_bytes(int32_t batch, int32_t num_pages, int32_t max_pages_per_seq);

/* Every sequence b takes over the pages that sequence sources[b] held before the
 * call (sources[b] = b: its own; -1: none), and lets go of the others: table rows,
 * held, lens (int32 [batch], may be NULL) and refs follow; entries behind the held
 * ones become -1, lens of a sequence without a source 0.  No row is copied: pages
 * that several sequences name are shared until one of them writes there
 * (tq_pages_reserve).  Beam search reorders its beams so, a prompt is forked into
 * several answers, a sequence that ended is freed. */
tq_status tq_pages_fork(const tq_paged_kv_cache* cache, int32_t* refs, int32_t* held, int32_t* lens,
                        const int32_t* sources, void* workspace, size_t workspace_bytes,
                        int32_t* status, void* stream);

/* Makes rows [start[b], start[b] + n_rows) of every sequence writable: call it
 * before each append with its write_pos and n_new.
 *   - Entries from held[b] up to the last of these rows' get free pages.
 *   - A held page with refs > 1 that these rows fall into is replaced by a free one,
 *     into which its rows below start[b] are copied (the rest of the new page is left
 *     as it was).  Where all that name a page write to it in this call, the last
 *     sequence keeps it.
 * Sequence by sequence and entry by entry the free page of the lowest number is
 * taken.  Where there are not enough nothing changes and TQ_DEV_NO_PAGE is set.  A
 * sequence whose rows are not in [0, capacity] sets TQ_DEV_WRITE_POS and is left
 * out (start[b] = -1 for a slot without a sequence: the append leaves it out, too). */
tq_status tq_pages_reserve(const tq_paged_kv_cache* cache, int32_t* refs, int32_t* held,
                           const int32_t* start, int32_t n_rows, void* workspace,
                           size_t workspace_bytes, int32_t* status, void* stream);

/* Moves the pages in use (refs > 0) to the lowest numbers: with n_live of them, the
 * i-th used page at or behind n_live moves, rows and all, to the i-th free page
 * before it; the others stay.
 *   table_out  int32 [batch][max_pages_per_seq], may be cache->block_table: the held
 *              entries by their new numbers, the others as they are
 *   refs_out   int32 [num_pages], may be refs
 *   n_live     int32 [1]
 *   moved      int32 [num_pages], may be NULL: each used page's new number (its own
 *              where it stayed), -1 for free ones; for page lists of the caller's
 * Rows of the pages that were moved from are left as they were. */
tq_status tq_pages_compact(const tq_paged_kv_cache* cache, const int32_t* refs, const int32_t* held,
                           int32_t* table_out, int32_t* refs_out, int32_t* n_live, int32_t* moved,
                           void* workspace, size_t workspace_bytes, int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* TQ_H */
