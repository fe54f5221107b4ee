/*
 * rpa.h -- C ABI of the GB300 (sm_103a) ragged paged attention library.
 *
 * The operations, each one asynchronous call on a caller-supplied CUDA stream:
 *
 *   rpa_forward          ragged paged attention over a packed prefill+decode batch
 *                        (tpu-inference "ragged_paged_attention/v2/kernel.py",
 *                        ref_ragged_paged_attention and ragged_paged_attention).
 *   rpa_update_kv_cache  scatter of the batch's new K/V tokens into their pages
 *                        (no counterpart on the pages beyond the v2 wrapper's TODO for a
 *                        cache-write kernel; defined like the MLA update_kv_cache).
 *                        rpa_forward_update does both in one call.
 *   mla_rpa_forward      MLA latent attention with its cache update
 *                        (tpu-inference "mla/v1/kernel.py", update_kv_cache and
 *                        mla_ragged_paged_attention / ref_mla_ragged_paged_attention).
 *   sparse_mla_forward   DSA sparse MLA over selected units of a paged latent cache
 *                        (sglang-jax "dsa/sparse_mla_prefill.py", sparse_mla_attention and
 *                        _sparse_mla_kernel_chunked_hminor).
 *   rpa_cross_forward    attention to all the keys of a sequence, whatever their number.
 *   rope_apply           rotary positions on packed queries and keys.
 *   rpa_g4_forward       rpa_forward over a cache of 4-bit values with a scale and a minimum a group,
 *                        which rpa_g4_update_kv_cache writes and rpa_g4_read_kv_cache reads back.
 *   rpa_key_weights      the attention that each cached key gets, added up over calls, and
 *   rpa_evict_kv_cache   the keys with the most of it kept at the front of their pages.
 *   rpa_rope_update_kv_cache
 *                        rpa_update_kv_cache with the rotation, and the rounding to the
 *                        cache's type, on the way; rpa_rope_forward_update attends in the
 *                        same call.
 *
 * Conventions shared by every entry point
 *   - Every tensor argument is a DEVICE pointer owned by the caller; the library
 *     never frees or retains it.  Row-major, densely packed, 16-byte aligned.
 *   - The library allocates no memory.  Scratch (work lists, split-KV partials,
 *     the device error word) lives in a caller-provided workspace whose size the
 *     matching *_workspace_size() call returns; the workspace must be 256-byte
 *     aligned, must be zero-filled once after it is allocated (the library keeps it
 *     consistent from then on), and must not be shared by two calls in flight at once.
 *   - Calls are asynchronous on `stream` and never synchronise with the host, so
 *     they can be captured in a CUDA graph.  A call may stand right behind kernels of the
 *     caller's that write its tensors, lengths and page tables, also ones that let the next
 *     launch of the stream start early.  Sizes read from device memory
 *     (num_seqs, cu_q_lens, kv_lens, page tables, indices) are validated on the
 *     device: a bad value sets a bit in the workspace's error word, the offending
 *     sequence/query is skipped (its output rows are left untouched), and no
 *     out-of-range address is ever formed.  rpa_check_device_status() reads the word.
 *   - Host-side arguments (shapes, dtypes, options) are validated before any launch;
 *     a bad one returns a negative status and launches nothing.
 *   - Optional values use a "none" encoding: sliding_window = 0, soft_cap = 0,
 *     k_scale = v_scale = 0, mask_value = NaN (meaning -0.7 * FLT_MAX, the pages'
 *     DEFAULT_MASK_VALUE).
 *   - Masking follows the pages: RPA adds mask_value to a masked logit, MLA
 *     substitutes it.  With a mask value at or below -1e30 a masked key's weight
 *     underflows to exactly zero in float32 (the key at the query's own position is
 *     always visible), so the kernels skip masked keys outright.  Any larger finite
 *     mask_value leaves masked keys real weight: then every key below kv_len takes
 *     part (future keys of a prefill chunk and keys outside the window alike) with
 *     mask_value added or substituted.  +inf is rejected with RPA_ERR_VALUE.
 */
#ifndef RPA_GB300_RPA_H_
#define RPA_GB300_RPA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define RPA_ABI_VERSION 1

/* Every entry point below is exported from the shared library. */
#if defined(__GNUC__)
#define RPA_API __attribute__((visibility("default")))
#else
#define RPA_API
#endif

/* Status codes returned by every call. */
typedef enum {
    RPA_OK = 0,
    RPA_ERR_NULL = -1,          /* a required pointer is NULL */
    RPA_ERR_SHAPE = -2,         /* inconsistent sizes (Hq % Hkv, odd combined heads, ...) */
    RPA_ERR_DTYPE = -3,         /* unsupported dtype combination */
    RPA_ERR_VALUE = -4,         /* bad option value (sliding_window < 0, soft_cap < 0, ...) */
    RPA_ERR_UNSUPPORTED = -5,   /* valid on the pages but not implemented here */
    RPA_ERR_CUDA = -6,          /* a CUDA runtime call failed (see rpa_last_error) */
    RPA_ERR_DEVICE_CHECK = -7,  /* rpa_check_device_status found a device-side error */
    RPA_ERR_WORKSPACE = -8      /* workspace NULL, misaligned or too small */
} rpa_status;

/* Element types. */
typedef enum {
    RPA_DTYPE_BF16 = 1,
    RPA_DTYPE_FP8_E4M3 = 2,
    RPA_DTYPE_F32 = 3,
    RPA_DTYPE_INT8 = 4,          /* two's-complement bytes (RPA K/V only) */
    RPA_DTYPE_G4 = 6,            /* rows of 4-bit values with a scale and a minimum for each group of them (the
                                  * rpa_g4_* calls, rpa_key_weights and rpa_evict_kv_cache only; their layout is
                                  * described there) */
    RPA_DTYPE_INT4 = 5           /* two's-complement 4-bit values, two to a byte along the head
                                  * dimension: element 2i of a row in the low nibble (bits 0-3) of
                                  * the row's byte i, element 2i+1 in the high nibble (RPA K/V only;
                                  * a head row is head_dim / 2 bytes) */
} rpa_dtype;

/* Bits of the device error word (OR-ed together). */
#define RPA_DEV_ERR_NUM_SEQS   0x01u  /* num_seqs / distribution outside [0, max_num_seqs] */
#define RPA_DEV_ERR_Q_LEN      0x02u  /* q_len < 0 or q_len > kv_len for some sequence */
#define RPA_DEV_ERR_KV_LEN     0x04u  /* cdiv(kv_len, page_size) > pages_per_seq */
#define RPA_DEV_ERR_PAGE       0x08u  /* a used page index outside [0, total_num_pages) */
#define RPA_DEV_ERR_TOKENS     0x10u  /* cu_q_lens[num_seqs] > max_num_tokens or not monotone */
#define RPA_DEV_ERR_POSITION   0x20u  /* sparse: query position outside [0, seq_len) */
#define RPA_DEV_ERR_TIMEOUT    0x40u  /* a pipeline wait gave up after its time limit (2 s) */
#define RPA_DEV_ERR_BATCH_KIND 0x80u  /* a sequence of the class rpa_params.batch_kind excludes */
#define RPA_DEV_ERR_BUDGET     0x100u /* eviction: a budget outside [0, max_keys] */

/* rpa_params.batch_kind: what the caller knows of the batch's mix (the MLA v1 page keys its
 * decode-only, prefill-only and mixed kernels on its `distribution`).  A sequence is decode-class
 * when q_len * (num_q_heads / num_kv_heads) <= 16, prefill-class otherwise. */
#define RPA_BATCH_MIXED        0      /* unknown or mixed: every kernel is launched */
#define RPA_BATCH_DECODE_ONLY  1      /* no prefill-class sequence: the prefill launches are skipped */
#define RPA_BATCH_PREFILL_ONLY 2      /* no decode-class sequence: the decode launch is skipped */

/* CUDA stream handle (ABI-compatible with cudaStream_t). */
typedef struct CUstream_st* rpa_stream_t;

/* ---------------------------------------------------------------------- */
/* Standard ragged paged attention                                         */
/* ---------------------------------------------------------------------- */

/* Problem description shared by rpa_forward / rpa_update_kv_cache.
 * Layouts (tpu-inference RPA v2, ref_ragged_paged_attention):
 *   q          [max_num_tokens, num_q_heads, head_dim]               q_dtype (bf16)
 *   kv_pages   [total_num_pages, page_size, num_combined_kv_heads, head_dim]  kv_dtype;
 *              combined head 2j holds K and 2j+1 holds V of KV head j
 *   kv_lens    int32 [max_num_seqs]   keys of each sequence, including its new tokens
 *   page_indices int32 [max_num_seqs, pages_per_seq]   logical -> physical page
 *   cu_q_lens  int32 [max_num_seqs + 1]   sequence i owns tokens [cu_q_lens[i], cu_q_lens[i+1])
 *   num_seqs   int32 [1] (device)   only the first num_seqs sequences are processed
 *   out        [max_num_tokens, num_q_heads, head_dim]   q_dtype; rows of tokens
 *              >= cu_q_lens[num_seqs] are not written
 * Query j of sequence i sits at position kv_len - q_len + j; key k is visible when
 * k <= q_pos and (sliding_window == 0 or k > q_pos - sliding_window).  Q head h reads
 * KV head h / (num_q_heads / num_kv_heads).  Logits: sm_scale * q.k, then
 * soft_cap * tanh(x / soft_cap) when soft_cap != 0.  When k_scale (v_scale) != 0 the
 * keys (values) are dequantised as bf16(float(k) * k_scale) before the dot products.
 * kv_dtype int8 and int4 (the v2 kernel's packed integer KV): two's-complement integers, read
 * as their exact value without a scale and dequantised like any other dtype with one; int4
 * packs two values a byte (RPA_DTYPE_INT4), so kv_pages (and new_k / new_v) rows are
 * head_dim / 2 bytes. */
typedef struct {
    uint32_t struct_size;        /* sizeof(rpa_params) */
    uint32_t version;            /* RPA_ABI_VERSION */
    int32_t max_num_tokens;
    int32_t num_q_heads;
    int32_t num_combined_kv_heads;
    int32_t head_dim;            /* 64, 128 or 256; 96 or 192 for attention over a bf16 cache without
                                    scales, with a power-of-two page_size >= 8 and a mask_value at or
                                    below -1e30 (the cache write takes any of the five) */
    int32_t total_num_pages;
    int32_t page_size;
    int32_t max_num_seqs;
    int32_t pages_per_seq;
    int32_t q_dtype;             /* RPA_DTYPE_BF16 */
    int32_t kv_dtype;            /* RPA_DTYPE_BF16, RPA_DTYPE_FP8_E4M3, RPA_DTYPE_INT8 or RPA_DTYPE_INT4 */
    float sm_scale;
    int32_t sliding_window;      /* 0 = none */
    float soft_cap;              /* 0 = none */
    float mask_value;            /* NaN = default */
    float k_scale;               /* 0 = none */
    float v_scale;               /* 0 = none */
    /* RPA_BATCH_*; a sequence the hint excludes is skipped (its rows are not written) and sets
     * RPA_DEV_ERR_BATCH_KIND.  Optional: a struct_size that ends before this field means
     * RPA_BATCH_MIXED. */
    int32_t batch_kind;
} rpa_params;

/* Bytes of workspace rpa_forward needs for these maxima. */
RPA_API int rpa_workspace_size(const rpa_params* p, size_t* bytes);

/* Ragged paged attention over the whole batch (every sequence, prefill and decode,
 * in one call).  `out` must not alias `q` or `kv_pages`. */
RPA_API int rpa_forward(const rpa_params* p, const void* q, const void* kv_pages, const int32_t* kv_lens,
                const int32_t* page_indices, const int32_t* cu_q_lens, const int32_t* num_seqs,
                void* out, void* workspace, size_t workspace_bytes, rpa_stream_t stream);

/* rpa_forward without a workspace argument, for callers that cannot allocate device
 * memory (for example a plugin inside an application whose memory manager owns the
 * whole GPU, or a serving loop that must not call cudaMalloc, which can synchronise
 * the device, once it is running).  The pages have no counterpart: it is a packaging
 * of rpa_forward, with the same arguments minus the workspace and the same results.
 *   - Scratch is a fixed array of RPA_NOALLOC_SCRATCH_BYTES inside the library; every
 *     GPU that loads the library holds it until the process exits.  Problems whose
 *     rpa_workspace_size() exceeds it are rejected with RPA_ERR_WORKSPACE before any
 *     launch.  The call allocates nothing itself.
 *   - Every call looks up the array's device address in the context current on the
 *     calling thread, so a host application's own (non-primary) context and a device
 *     reset between calls are both handled.  The first call in a context also loads
 *     the library's device code there; make that first call before any stream capture.
 *   - All calls share the one array and it keeps the previous call's contents; the
 *     kernels reset what they need.  Calls that overlap on the GPU (two streams, or
 *     two threads) race on it: serialise them.
 *   - Device-side metadata errors skip the offending sequence as in rpa_forward, but
 *     the error word is not reported (there is no workspace to pass to
 *     rpa_check_device_status). */
#define RPA_NOALLOC_SCRATCH_BYTES (64u << 20)
RPA_API int rpa_forward_noalloc(const rpa_params* p, const void* q, const void* kv_pages, const int32_t* kv_lens,
                                const int32_t* page_indices, const int32_t* cu_q_lens, const int32_t* num_seqs,
                                void* out, rpa_stream_t stream);

/* Write token j of sequence i (position kv_len - q_len + j) into slot
 * page_indices[i, pos / page_size], pos % page_size of kv_pages, in place:
 * new_k[t, g, :] to combined head 2g and new_v[t, g, :] to 2g+1.
 *   new_k, new_v  [max_num_tokens, num_combined_kv_heads / 2, head_dim]  kv_dtype
 * Bytes are copied unchanged; every other byte of kv_pages is left as it was.
 * `workspace` is optional (may be NULL): when given, device-side metadata errors are
 * recorded in its error word (it needs at least 256 bytes). */
RPA_API int rpa_update_kv_cache(const rpa_params* p, const void* new_k, const void* new_v, void* kv_pages,
                        const int32_t* kv_lens, const int32_t* page_indices, const int32_t* cu_q_lens,
                        const int32_t* num_seqs, void* workspace, size_t workspace_bytes,
                        rpa_stream_t stream);

/* rpa_update_kv_cache followed by rpa_forward, in one call with one launch fewer: the cache
 * write of the batch's new K/V rows (exactly as rpa_update_kv_cache: bit-exact, in place)
 * runs in the same launch as the work-list plan, and the attention launches read the cache
 * only after both have ended, so the new tokens attend to themselves. The tpu-inference RPA
 * v2 wrapper leaves this write inside the attention call as a TODO; this is that fused form.
 * Arguments as in the two calls; `workspace` is rpa_forward's (its error word also records the
 * cache write's metadata errors). `out` must not alias q, kv_pages, new_k or new_v. */
RPA_API int rpa_forward_update(const rpa_params* p, const void* q, const void* new_k, const void* new_v,
                               void* kv_pages, const int32_t* kv_lens, const int32_t* page_indices,
                               const int32_t* cu_q_lens, const int32_t* num_seqs, void* out, void* workspace,
                               size_t workspace_bytes, rpa_stream_t stream);

/* ---------------------------------------------------------------------- */
/* Rotary positions                                                         */
/* ---------------------------------------------------------------------- */

/* Pair i of a head's first rotary_dim elements turns by the angle position * f_i:
 *   (x, y) -> amplitude * (x cos - y sin, y cos + x sin),
 * where f_i = base^(-2i / rotary_dim), changed by `scaling`; elements past rotary_dim stay as
 * they are.  pairing names the pair's two elements. */
#define RPA_ROPE_HALF        0   /* i and i + rotary_dim / 2 */
#define RPA_ROPE_INTERLEAVED 1   /* 2i and 2i + 1 */

#define RPA_ROPE_SCALE_NONE   0
#define RPA_ROPE_SCALE_LINEAR 1  /* f_i / factor */
#define RPA_ROPE_SCALE_NTK    2  /* base * factor^(rotary_dim / (rotary_dim - 2)) for base (rotary_dim > 2) */
/* With n_i = original_max_position * f_i / (2 pi), the turns of pair i over the original context:
 * f_i where n_i >= high_freq_factor, f_i / factor where n_i <= low_freq_factor, between them
 * linear in n_i. */
#define RPA_ROPE_SCALE_LLAMA3 3
/* f_i for the pairs below `low`, f_i / factor from `high` on, between them linear in i, with
 * low = max(floor(c(beta_fast)), 0), high = min(ceil(c(beta_slow)), rotary_dim - 1) and
 * c(n) = rotary_dim * ln(original_max_position / (2 pi n)) / (2 ln base). */
#define RPA_ROPE_SCALE_YARN   4

#define RPA_ROPE_MAX_DIM 256

typedef struct {
    uint32_t struct_size;        /* sizeof(rope_params) */
    uint32_t version;            /* RPA_ABI_VERSION */
    int32_t rotary_dim;          /* even, 0 to RPA_ROPE_MAX_DIM; 0 turns nothing */
    int32_t pairing;             /* RPA_ROPE_HALF or RPA_ROPE_INTERLEAVED */
    int32_t scaling;             /* RPA_ROPE_SCALE_* */
    int32_t original_max_position;  /* LLAMA3 and YARN */
    double base;                 /* > 1 */
    double factor;               /* >= 1; every scaling but NONE */
    double low_freq_factor;      /* LLAMA3: 0 < low_freq_factor < high_freq_factor */
    double high_freq_factor;
    double beta_fast;            /* YARN: beta_fast > beta_slow > 0 */
    double beta_slow;
    double attention_factor;     /* the amplitude; 0 = 1, for YARN 0.1 ln(factor) + 1 */
} rope_params;

/* What the calls below take: a plain host value that rope_table_init fills once and the caller
 * keeps.  step[i] is f_i / (2 pi), pair i's turn per position, as a fraction of 2^64: the kernels
 * multiply it by the position modulo 2^64, which leaves the fraction of a turn exactly, however
 * far the position, and take the sine and cosine of that in float32.  A caller with frequencies
 * of its own fills the table itself. */
typedef struct {
    uint32_t struct_size;        /* sizeof(rope_table) */
    uint32_t version;            /* RPA_ABI_VERSION */
    int32_t rotary_dim;
    int32_t pairing;
    float amplitude;             /* finite */
    uint32_t reserved;           /* 0 */
    uint64_t step[RPA_ROPE_MAX_DIM / 2];  /* rotary_dim / 2 are used */
} rope_table;

/* Fills *t from *p on the host (no GPU is needed). */
RPA_API int rope_table_init(const rope_params* p, rope_table* t);

/* Strides count elements; 0 stands for the dense layout [num_tokens, heads, head_dim]'s.  Each is
 * a multiple of 8, 0 to 2^30; a row's head_dim elements are adjacent.  Rows of an output
 * must not overlap: tokens outside heads (token stride >= (heads - 1) * head stride + head_dim) or
 * heads outside tokens. */
typedef struct {
    uint32_t struct_size;        /* sizeof(rope_apply_params) */
    uint32_t version;            /* RPA_ABI_VERSION */
    int32_t num_tokens;          /* >= 0 */
    int32_t num_q_heads;
    int32_t num_k_heads;         /* 0 with k and k_out NULL */
    int32_t head_dim;            /* multiple of 16, up to 512, >= the table's rotary_dim */
    int32_t inverse;             /* 1: the transposed map, by the opposite angle (with amplitude 1 the
                                    inverse; it takes an output's gradient to the input's) */
    int32_t reserved;            /* 0 */
    int64_t q_token_stride, q_head_stride, k_token_stride, k_head_stride;
    int64_t q_out_token_stride, q_out_head_stride, k_out_token_stride, k_out_head_stride;
} rope_apply_params;

/* q [num_tokens, num_q_heads, head_dim] and k [num_tokens, num_k_heads, head_dim], bf16, turned by
 * positions int32 [num_tokens] (any value, negative ones too) into q_out and k_out, bf16: computed
 * in float32, rounded once.  q_out may be q and k_out may be k (with the same strides); otherwise
 * outputs overlap neither inputs nor each other.  Operands that share no element may lie between one
 * another where their token strides are equal, and their head strides are or each stays inside a part
 * of the token; other interleaved layouts are refused. */
RPA_API int rope_apply(const rope_apply_params* p, const rope_table* t, const void* q, const void* k,
                       const int32_t* positions, void* q_out, void* k_out, rpa_stream_t stream);

/* Token and head strides of q, new_k and new_v, as in rope_apply_params (slices of one projection's
 * output, say); NULL in place of the struct, or 0 in a field, stands for the dense layout. */
typedef struct {
    uint32_t struct_size;        /* sizeof(rope_strides) */
    uint32_t version;            /* RPA_ABI_VERSION */
    int64_t q_token, q_head, k_token, k_head, v_token, v_head;
} rope_strides;

/* rpa_update_kv_cache with what precedes it: new_k turned to its position, both rounded to the
 * cache's type, and the queries turned beside them.
 *   q             [max_num_tokens, num_q_heads, head_dim] bf16, or NULL with q_out NULL: no queries
 *   new_k, new_v  [max_num_tokens, num_combined_kv_heads / 2, head_dim] bf16, whatever kv_dtype is
 *   positions     int32 [max_num_tokens], or NULL: the position of the token's slot,
 *                 kv_len - q_len + j (the slot is that one either way)
 *   q_out         [max_num_tokens, num_q_heads, head_dim] bf16, dense; may be q if q is dense
 * The cache gets x / k_scale (x / v_scale; no division with scale 0), x in float32 after the turn and
 * the quotient as its product with the scale's float32 reciprocal (exact for powers of two, else within
 * 2^-23 of itself for scales up to 2^126), rounded to nearest even: to bf16; to e4m3, +-448 at most,
 * NaN kept; to int8 or int4, within [-128, 127] or [-8, 7], NaN as 0.  rpa_forward with the same
 * scales reads it back.
 * head_dim and kv_dtype as rpa_update_kv_cache; int4 takes rotary_dim a multiple of 4.
 * A scale's reciprocal must be finite.  Only the slots of the batch's tokens are written, and the
 * q_out rows of those tokens: a token whose metadata is bad is skipped whole, as are the tokens
 * from cu_q_lens[num_seqs] on.  Two tokens of a batch that name one slot leave it undefined.
 * `workspace` is optional, as for rpa_update_kv_cache. */
RPA_API int rpa_rope_update_kv_cache(const rpa_params* p, const rope_table* t, const rope_strides* strides,
                                     const void* q, const void* new_k, const void* new_v, void* kv_pages,
                                     const int32_t* kv_lens, const int32_t* page_indices, const int32_t* cu_q_lens,
                                     const int32_t* num_seqs, const int32_t* positions, void* q_out, void* workspace,
                                     size_t workspace_bytes, rpa_stream_t stream);

/* rpa_rope_update_kv_cache, then rpa_forward of the turned queries over the updated cache, in one
 * call (`out` equals the two calls' up to rounding: the keys of a decode may be split elsewhere).
 * `q_rot` is rpa_rope_update_kv_cache's q_out (not NULL; the caller's, holding the turned queries
 * afterwards), `out` and `workspace` are rpa_forward's; the workspace's error word also records the
 * cache write's metadata errors.  `out` must not alias q, q_rot, kv_pages, new_k or new_v. */
RPA_API int rpa_rope_forward_update(const rpa_params* p, const rope_table* t, const rope_strides* strides, const void* q,
                                    const void* new_k, const void* new_v, void* kv_pages, const int32_t* kv_lens,
                                    const int32_t* page_indices, const int32_t* cu_q_lens, const int32_t* num_seqs,
                                    const int32_t* positions, void* q_rot, void* out, void* workspace,
                                    size_t workspace_bytes, rpa_stream_t stream);

/* ---------------------------------------------------------------------- */
/* Cross attention                                                          */
/* ---------------------------------------------------------------------- */

/* Attention of a packed batch's queries to all the cached keys of their sequence: a decoder's
 * tokens to its encoder's states, whose number has nothing to do with the queries', or a
 * sequence's own tokens in both directions.  Arguments and layouts are rpa_forward's, with these
 * differences: kv_lens[i] is any number of keys from 0 on, fewer than the queries or more; every
 * query sees keys [0, kv_lens[i]); a sequence without keys gets rows of zeros; sliding_window is 0
 * and mask_value NaN.  The keys and values are written by rpa_update_kv_cache or
 * rpa_rope_update_kv_cache (with cu_q_lens and kv_lens of the encoder's side).  `workspace`:
 * rpa_cross_workspace_size bytes, as rpa_forward's. */
RPA_API int rpa_cross_workspace_size(const rpa_params* p, size_t* bytes);
RPA_API int rpa_cross_forward(const rpa_params* p, const void* q, const void* kv_pages, const int32_t* kv_lens,
                              const int32_t* page_indices, const int32_t* cu_q_lens, const int32_t* num_seqs, void* out,
                              void* workspace, size_t workspace_bytes, rpa_stream_t stream);

/* ---------------------------------------------------------------------- */
/* 4-bit caches with a scale and a minimum a group                          */
/* ---------------------------------------------------------------------- */

/* A cache of RPA_DTYPE_G4 is uint8 [total_num_pages, page_size, num_kv_heads, RPA_G4_ROW_BYTES(head_dim)]
 * (num_kv_heads = num_combined_kv_heads / 2).  A row holds a token's K and V of one KV head:
 *   bytes [0, head_dim / 2)         K's numbers, element 2i in the low half of byte i, 2i + 1 in the high half
 *   bytes [head_dim / 2, head_dim)  V's
 *   then                            (s, m), two bf16, of each group of K and then of each group of V
 * A group is RPA_G4_GROUP(head_dim) elements; an element is s n + m with its number n in 0..15.  head_dim is 64,
 * 128 or 256; kv_dtype RPA_DTYPE_G4, k_scale and v_scale 0, mask_value NaN. */
#define RPA_G4_GROUP(head_dim) ((head_dim) == 64 ? 32 : 64)
#define RPA_G4_ROW_BYTES(head_dim) ((head_dim) + 8 * ((head_dim) / RPA_G4_GROUP(head_dim)))

/* rpa_rope_update_kv_cache into such a cache: the same arguments, the same rows and slots.  K (after its turn) and V
 * are rounded to bf16, as a bf16 cache would hold them; a NaN then counts as 0 and what lies beyond +-2^48 as
 * that.  Of a group, m is the least, s the bf16 nearest to (greatest - least) / 15, and n is (x - m) / s
 * rounded to nearest even, 15 at most (0 where s is 0).  rotary_dim is a multiple of 16. */
RPA_API int rpa_g4_update_kv_cache(const rpa_params* p, const rope_table* t, const rope_strides* strides, const void* q,
                                   const void* new_k, const void* new_v, void* kv_pages, const int32_t* kv_lens,
                                   const int32_t* page_indices, const int32_t* cu_q_lens, const int32_t* num_seqs,
                                   const int32_t* positions, void* q_out, void* workspace, size_t workspace_bytes,
                                   rpa_stream_t stream);

/* The K and V rows of the batch's tokens as bf16 (s n + m rounded once): token j of sequence i from position
 * kv_len - q_len + j, where the update put it; with q_len = kv_len a whole sequence.
 *   k_out, v_out  [max_num_tokens, num_kv_heads, head_dim] bf16, dense; rows of tokens that are skipped (bad
 *                 metadata, or past cu_q_lens[num_seqs]) are not written
 * `workspace` is optional, as for the update.  num_q_heads is num_kv_heads or any multiple. */
RPA_API int rpa_g4_read_kv_cache(const rpa_params* p, const void* kv_pages, const int32_t* kv_lens,
                                 const int32_t* page_indices, const int32_t* cu_q_lens, const int32_t* num_seqs, void* k_out,
                                 void* v_out, void* workspace, size_t workspace_bytes, rpa_stream_t stream);

/* rpa_forward over such a cache: the same arguments, masks and options (sliding_window, soft_cap, batch_kind).
 * `workspace`: rpa_g4_workspace_size bytes.  Sequences of more than 16 query rows a KV head see K rounded to bf16 and V
 * to f16, or to bf16 where a group of V that a tile of queries sees has s >= 4, |m| >= 2^20, or both s < 2^-9 and |m| < 2^-6
 * (the weights are rounded to the same type; prompts over such caches take up to twice as long).  V in f16 is within 2^-10 of
 * itself from 2^-4 on and within 2^-14 in all below; in bf16 within 2^-8 of itself. */
RPA_API int rpa_g4_workspace_size(const rpa_params* p, size_t* bytes);
RPA_API int rpa_g4_forward(const rpa_params* p, const void* q, const void* kv_pages, const int32_t* kv_lens,
                           const int32_t* page_indices, const int32_t* cu_q_lens, const int32_t* num_seqs, void* out,
                           void* workspace, size_t workspace_bytes, rpa_stream_t stream);

/* ---------------------------------------------------------------------- */
/* Key weights and eviction                                                 */
/* ---------------------------------------------------------------------- */

/* The attention that each cached key gets from the batch's queries, added to what it had:
 *   weights_out[page, h, slot] = keep * weights[page, h, slot] + the sum, over the sequence's query tokens in the
 *   batch and the q heads of KV head h's group, of the key's softmax probability (scores, soft cap, causal mask and
 *   window as rpa_forward's)
 *   weights, weights_out  float32 [total_num_pages, num_kv_heads, page_size]; weights_out may be weights; weights may
 *                         be NULL with keep 0, and is not read then
 * for every key of the batch's sequences (0 new weight where no query sees it); other entries are left as they are, as
 * are those of sequences without queries.  Sequences of a batch may share pages only where weights_out is not weights (or keep
 * is 0): a shared slot then gets one sequence's result.  In place one would read what another has written, and add to
 * that, in some runs and not in others; nothing records it.  kv_dtype is
 * RPA_DTYPE_BF16 or RPA_DTYPE_G4, head_dim 64, 128 or 256, k_scale and v_scale 0, mask_value NaN; batch_kind is not
 * looked at.  Queries: a decode step's, to add up over steps, or a prompt's last ones.  `workspace`: rpa_key_weights_workspace_size bytes,
 * up to half a GB of it for the scores of sequences of up to 16 query rows a KV head; those past it are computed twice. */
RPA_API int rpa_key_weights_workspace_size(const rpa_params* p, size_t* bytes);
RPA_API int rpa_key_weights(const rpa_params* p, const void* q, const void* kv_pages, const int32_t* kv_lens,
                            const int32_t* page_indices, const int32_t* cu_q_lens, const int32_t* num_seqs, const float* weights,
                            float* weights_out, float keep, void* workspace, size_t workspace_bytes, rpa_stream_t stream);

typedef struct {
    uint32_t struct_size;        /* sizeof(rpa_evict_params) */
    uint32_t version;            /* RPA_ABI_VERSION */
    int32_t num_kv_heads;
    int32_t row_bytes;           /* bytes of a token's K and V of one KV head, adjacent in the cache: 4 head_dim (bf16),
                                    2 head_dim (fp8, int8), head_dim (int4), RPA_G4_ROW_BYTES; a multiple of 16 */
    int32_t total_num_pages;
    int32_t page_size;
    int32_t max_num_seqs;
    int32_t pages_per_seq;
    int32_t max_keys;            /* > 0, >= sinks + recent: places of slots_out a head */
    int32_t sinks;               /* >= 0: a sequence's first keys, which always stay */
    int32_t recent;              /* >= 0: and its last ones: those in the last slots, or with positions those that came last */
    int32_t reserved;            /* 0 */
    int32_t* positions;          /* when each key came (below), or NULL; a struct_size that ends before it counts as NULL */
} rpa_evict_params;

/* Leaves each sequence and KV head its budgets[i] keys of the largest weights, in the first slots of its pages.
 *   kv_pages    the cache, written in place: [total_num_pages, page_size, num_kv_heads, row_bytes]
 *   kv_lens     int32 [max_num_seqs]   keys now; page_indices, num_seqs as everywhere
 *   weights     float32 [total_num_pages, num_kv_heads, page_size], as rpa_key_weights leaves them
 *   budgets     int32 [max_num_seqs]   0 to max_keys
 *   kv_lens_out int32 [max_num_seqs]   keys afterwards: min(kv_len, max(budget, sinks + recent)); may be kv_lens, or NULL
 *   slots_out   int32 [max_num_seqs, num_kv_heads, max_keys]   the slot that the key in slot j had; places from the new
 *               length on are not written
 *   weights_out float32, as weights: the kept keys' weights in their new slots; may be weights, or NULL
 * The first `sinks` and the last `recent` keys come before all others, then larger weights (NaN last), then lower slots.
 * Kept keys in the first slots stay where they are; the others move, in their order, to the slots of the keys that
 * go, in theirs.  (A key's own position is in its rotation: attention over what is left is by rpa_forward without a
 * window, new tokens with `positions` of their own.)  Slots behind the new length keep what they hold.  No page may belong to two
 * sequences, be the other in the batch or not (its keys would move under it), nor twice to one.  A sequence whose metadata is bad is left alone.  `workspace`: rpa_evict_workspace_size
 * bytes.
 *
 * rpa_evict_params.positions: int32, as weights, written in place.  After one call the order of the slots is no longer the
 * order in which the keys came, so a cache that is cut again and again gives positions: without them `recent` means the last
 * slots, which hold the newest keys only until a call has moved some.  An entry below 0 (memset it all to -1 at first, and the
 * entries of a page that another sequence gets, whose weights are 0 then, too) is a new key's: new keys get the numbers behind the greatest entry of
 * their head, in the order of their slots, and keep them from then on; `recent` keys are those whose numbers are among the
 * head's last `recent`.  The entries of the slots from the new length to the old one become -1 again and their weights_out 0, so
 * that tokens written there are new and start without weight (without positions those weights stay as they are, and
 * rpa_key_weights would add to them).  Entries of the caller's own (at most 2^30, different within a sequence's head) do as well. */
RPA_API int rpa_evict_workspace_size(const rpa_evict_params* p, size_t* bytes);
RPA_API int rpa_evict_kv_cache(const rpa_evict_params* p, void* kv_pages, const int32_t* kv_lens, const int32_t* page_indices,
                               const int32_t* num_seqs, const float* weights, const int32_t* budgets, int32_t* kv_lens_out,
                               int32_t* slots_out, float* weights_out, void* workspace, size_t workspace_bytes,
                               rpa_stream_t stream);

/* ---------------------------------------------------------------------- */
/* MLA latent ragged paged attention                                       */
/* ---------------------------------------------------------------------- */

/* Layouts (tpu-inference MLA v1, mla_ragged_paged_attention):
 *   ql_nope    [max_num_tokens, num_q_heads, lkv_dim]        bf16, or fp8 e4m3 (q_dtype)
 *   q_pe       [max_num_tokens, num_q_heads, r_dim]          same dtype as ql_nope
 *   new_kv_c   [max_num_tokens, lkv_dim]                     bf16
 *   new_k_pe   [max_num_tokens, r_dim]                       bf16
 *   cache_kv_c [total_num_pages, page_size / kv_packing, kv_packing, lkv_dim_pad] bf16
 *   cache_k_pe [total_num_pages, page_size / kv_packing, kv_packing, r_dim_pad]   bf16
 *              (token t of a page is row t of the page: same bytes as [P, page_size, D])
 *   kv_lens    int32 [max_num_seqs]; page_indices int32 [max_num_seqs * pages_per_seq]
 *   cu_q_lens  int32 [max_num_seqs + 1]; distribution int32 [3] (device):
 *              (decode_end, prefill_end, num_seqs); only distribution[2] bounds the work
 *   out        [max_num_tokens, num_q_heads, lkv_dim]        bf16
 * Key = [kv_c | k_pe], value = kv_c, one latent head shared by all q heads; masked
 * logits are replaced by mask_value (see the header note on masking).  fp8 queries are
 * widened exactly to bf16 before the products; the output stays bf16 (the MLA v1 page
 * writes it in the query dtype, which for fp8 would throw away most of its precision). */
typedef struct {
    uint32_t struct_size;        /* sizeof(mla_params) */
    uint32_t version;            /* RPA_ABI_VERSION */
    int32_t max_num_tokens;
    int32_t num_q_heads;         /* multiple of 128 (one two-CTA tile) */
    int32_t lkv_dim;             /* 512 */
    int32_t r_dim;               /* 64 */
    int32_t lkv_dim_pad;         /* align(lkv_dim, 128) */
    int32_t r_dim_pad;           /* align(r_dim, 128) */
    int32_t total_num_pages;
    int32_t page_size;
    int32_t kv_packing;          /* 2 for bf16 */
    int32_t max_num_seqs;
    int32_t pages_per_seq;
    float sm_scale;
    int32_t sliding_window;      /* 0 = none */
    float soft_cap;              /* 0 = none */
    float mask_value;            /* NaN = default */
    /* Optional (read only when struct_size covers them, else bf16 queries): */
    int32_t q_dtype;             /* RPA_DTYPE_BF16 (0 is taken as bf16) or RPA_DTYPE_FP8_E4M3 for
                                    ql_nope and q_pe */
    float q_scale;               /* fp8 queries: every score is multiplied by it after sm_scale
                                    (0 = 1); must be 0 for bf16 queries */
} mla_params;

RPA_API int mla_workspace_size(const mla_params* p, size_t* bytes);

/* Scatter the batch's new latent rows into the caches, in place (update_kv_cache):
 * token j of sequence i < distribution[2] goes to position kv_len - q_len + j; its
 * kv_c row is copied to cache_kv_c and its k_pe row to cache_k_pe with columns
 * [r_dim, r_dim_pad) written as zero.  `workspace` is optional, as for
 * rpa_update_kv_cache. */
RPA_API int mla_update_kv_cache(const mla_params* p, const void* new_kv_c, const void* new_k_pe, void* cache_kv_c,
                        void* cache_k_pe, const int32_t* kv_lens, const int32_t* page_indices,
                        const int32_t* cu_q_lens, const int32_t* distribution, void* workspace,
                        size_t workspace_bytes, rpa_stream_t stream);

/* mla_update_kv_cache followed by attention of every query token over the updated
 * caches (the caches are modified in place).  The cache write runs in the same launch as
 * the work-list plan (the MLA v1 page leaves fusing it as a TODO); attention starts once
 * both have ended. */
RPA_API int mla_rpa_forward(const mla_params* p, const void* ql_nope, const void* q_pe, const void* new_kv_c,
                    const void* new_k_pe, void* cache_kv_c, void* cache_k_pe, const int32_t* kv_lens,
                    const int32_t* page_indices, const int32_t* cu_q_lens, const int32_t* distribution,
                    void* out, void* workspace, size_t workspace_bytes, rpa_stream_t stream);

/* ---------------------------------------------------------------------- */
/* DSA sparse MLA                                                           */
/* ---------------------------------------------------------------------- */

/* Layouts (sglang-jax sparse_mla_attention, paged per-request mode):
 *   q          [batch, num_queries, num_heads, dk]    bf16 (dk = 576 = 512 + 64)
 *   cache      [total_num_pages * page_size, row_stride]  bf16 (row_stride >= dk; the
 *              [P, page_size / packing, packing, row_stride] cache has these bytes)
 *   indices    int32 [batch, num_queries, topk]   unit ids, -1 = empty slot
 *   positions  int32 [batch, num_queries]         query positions (causal bound)
 *   page_table int32 [batch, max_pages]           logical -> physical page
 *   out        [batch, num_queries, num_heads, dv]  float32 (dv = 512)
 * A unit u covers tokens [u * read_block, (u + 1) * read_block).  Token kp of slot i
 * is a key when u >= 0, kp <= position and kp < seq_len; it is read from row
 * page_table[b, kp / page_size] * page_size + kp % page_size.  Keys form a multiset
 * (a unit named twice counts twice); a query with no key outputs zeros.
 * read_block must divide page_size. */
typedef struct {
    uint32_t struct_size;        /* sizeof(sparse_params) */
    uint32_t version;            /* RPA_ABI_VERSION */
    int32_t batch;
    int32_t num_queries;
    int32_t num_heads;           /* multiple of 128 (one two-CTA tile) */
    int32_t dk;                  /* 576 */
    int32_t dv;                  /* 512 */
    int32_t row_stride;          /* elements per cache row (640) */
    int32_t topk;
    int32_t read_block;
    int32_t page_size;
    int32_t max_pages;
    int32_t total_num_pages;
    int32_t seq_len;
    float sm_scale;              /* required, > 0 */
} sparse_params;

RPA_API int sparse_mla_workspace_size(const sparse_params* p, size_t* bytes);

RPA_API int sparse_mla_forward(const sparse_params* p, const void* q, const void* cache, const int32_t* indices,
                       const int32_t* positions, const int32_t* page_table, float* out, void* workspace,
                       size_t workspace_bytes, rpa_stream_t stream);

/* Packed-ragged mode with the self-write (sglang-jax "dsa/sparse_mla_prefill.py",
 * prefill_write_and_attend_ragged and the ragged branch of sparse_mla_attention): several
 * requests' tokens packed along one axis.
 *   ql         [num_tokens, num_heads, dv]      bf16 absorbed latent query (dv = 512)
 *   qpe        [num_tokens, num_heads, rope]    bf16 rope query (rope = 64); the query is
 *              their concatenation (dk = dv + rope = 576)
 *   kvc, kpe   [num_tokens, dv], [num_tokens, rope]  bf16 new latent rows (both NULL: no write)
 *   cache      [total_num_pages * page_size, row_stride]  bf16, written in place
 *   topk       int32 [num_tokens, topk]   request-local unit ids, -1 = empty slot
 *   positions  int32 [num_tokens]         absolute query positions
 *   loc        int32 [num_tokens]         flat cache row of each token's new row (-1 = none;
 *              NULL with kvc/kpe NULL)
 *   seq_lens   int32 [num_seqs]           each request's key length (causal bound)
 *   cu_q_lens  int32 [num_seqs + 1]       request r owns tokens [cu_q_lens[r], cu_q_lens[r+1])
 *   cu_kv_lens int32 [num_seqs + 1]       page-aligned key offsets into page_indices' runs
 *   page_indices int32 [num_page_ids]     packed physical page ids
 *   out        [num_tokens, num_heads, dv]  float32
 * First every token's row [kvc | kpe | zeros] is written to cache row loc[t] (rows outside
 * the cache are dropped; two tokens naming one row leave either's). Then token t attends as
 * in sparse_mla_forward, where its request r is the number of cu_q_lens[1..num_seqs]
 * entries <= t (clipped to num_seqs - 1), the causal bound is seq_lens[r], and key kp sits
 * in page page_indices[min(cu_kv_lens[r] / page_size + kp / page_size, num_page_ids - 1)].
 * read_block must divide page_size. */
typedef struct {
    uint32_t struct_size;        /* sizeof(sparse_ragged_params) */
    uint32_t version;            /* RPA_ABI_VERSION */
    int32_t num_tokens;
    int32_t num_seqs;
    int32_t num_heads;           /* multiple of 128 */
    int32_t dv;                  /* 512 */
    int32_t rope;                /* 64 */
    int32_t row_stride;          /* elements per cache row (>= dv + rope, multiple of 8) */
    int32_t topk;
    int32_t read_block;
    int32_t page_size;
    int32_t num_page_ids;
    int32_t total_num_pages;
    float sm_scale;              /* required, > 0 */
} sparse_ragged_params;

RPA_API int sparse_mla_ragged_workspace_size(const sparse_ragged_params* p, size_t* bytes);

RPA_API int sparse_mla_write_and_attend_ragged(const sparse_ragged_params* p, const void* ql, const void* qpe,
                                               const void* kvc, const void* kpe, void* cache, const int32_t* topk,
                                               const int32_t* positions, const int32_t* loc,
                                               const int32_t* seq_lens, const int32_t* cu_q_lens,
                                               const int32_t* cu_kv_lens, const int32_t* page_indices, float* out,
                                               void* workspace, size_t workspace_bytes, rpa_stream_t stream);

/* ---------------------------------------------------------------------- */
/* Status and diagnostics                                                   */
/* ---------------------------------------------------------------------- */

/* Synchronises `stream`, reads the workspace's device error word into *bits (may be
 * NULL) and clears it.  Returns RPA_ERR_DEVICE_CHECK when any bit was set. */
RPA_API int rpa_check_device_status(void* workspace, uint32_t* bits, rpa_stream_t stream);

/* Failure-path check (diagnostics): launches one thread that waits, through the same bounded
 * wait every pipeline of the library uses, on a barrier nothing arrives on.  The wait gives up
 * after its limit (2 s), sets RPA_DEV_ERR_TIMEOUT in the workspace's error word and the kernel
 * returns: rpa_check_device_status then reports it, and the context stays usable.
 * `workspace` needs at least 256 bytes. */
RPA_API int rpa_selftest_bounded_wait(void* workspace, size_t workspace_bytes, rpa_stream_t stream);

/* Per-kernel timing (diagnostics).  While enabled, every kernel the library launches
 * is bracketed by two CUDA events on its launch stream (a GPU-side timestamp pair; no
 * host synchronisation).  rpa_profile_read synchronises on the recorded events and
 * reports, per kernel name, the number of launches and their summed duration since
 * the last rpa_profile_reset.  Entries are written to out[0 .. max_entries) in name
 * order; *n_entries receives the total number of kernel names. */
typedef struct {
    char name[48];
    int64_t launches;
    double total_ms;
} rpa_kernel_time;

RPA_API int rpa_profile_enable(int on);
RPA_API int rpa_profile_reset(void);
RPA_API int rpa_profile_read(rpa_kernel_time* out, int max_entries, int* n_entries);

/* Number of kernels the library has launched since it was loaded, counted whether or not
 * timing is enabled (a host-side counter; no synchronisation). */
RPA_API int64_t rpa_launch_count(void);

/* Thread-local description of the last failed call ("" if none). */
RPA_API const char* rpa_last_error(void);

/* RPA_ABI_VERSION of the loaded library. */
RPA_API int rpa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* RPA_GB300_RPA_H_ */
