/*
 * kvpool.h -- C ABI of the GB300 (sm_103a) KV-cache codec for multi-agent
 * KV sharing.
 *
 * Three containers, all position-independent byte blobs in device memory:
 *
 *  SharedKVPool -- "PolyKV: A Shared Asymmetrically-Compressed KV Cache Pool
 *    for Multi-Agent LLM Inference", 2.A (write once, read many; one object
 *    whose size does not depend on the number of agents) and 2.B (keys int8
 *    with one symmetric scale per layer tensor; values rotated by a fast
 *    Walsh-Hadamard transform, normalised, mapped to the 8-level Lloyd-Max
 *    codebook for N(0,1) and packed at 3 bits).
 *
 *  CacheCard -- "QKVShare: Quantized KV-Cache Handoff for Multi-Agent
 *    On-Device LLMs", Methodology 1-3 (per-token bitwidth from {2,4,8,16},
 *    quantized KV groups plus metadata seq_len / model_id / position offset;
 *    the receiver rebuilds 16-bit past_key_values from it).
 *
 *  Pages -- an agent's own growing cache beside the pool it shares: pages of
 *    tokens, written a token or a prompt at a time, attended over and joined
 *    with attention over the pool ("PolyKV" 2.A gives each agent a cache of
 *    its own on top of the shared one; the papers leave its form open).
 *
 * Conventions shared by every entry point
 * ----------------------------------------
 *  - KV tensors are bf16, one tensor per layer, layout [H][T][d] contiguous
 *    (the Hugging Face past_key_values layout at batch 1).  head_dim d must
 *    be 64 or 128.
 *  - Arrays of per-layer tensor pointers (k_layers, k_dst, ...) are HOST
 *    arrays of DEVICE pointers; the library reads them during the call only
 *    (they are copied into the kernel launch), so the caller may reuse them
 *    as soon as the call returns.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream).  Every compute call only enqueues work on that stream and
 *    returns; it never allocates, frees or synchronises device memory.  The
 *    only synchronising calls are kvpool_status, cachecard_status,
 *    cachecard_read_header and kvpages_status, which say so.
 *  - The caller owns every buffer.  Device pointers to KV tensors must be
 *    16-byte aligned; pool, card and page buffers 256-byte aligned; workspaces
 *    16-byte aligned.
 *  - Errors: 0 is success, negative values are KVP_ERR_*.  Everything the
 *    host can check (null pointers, shapes, alignment, buffer sizes) is
 *    checked before any work is enqueued, and nothing is enqueued on error.
 *    Conditions only the device can see (non-finite input, a value whose
 *    fp16 scale overflows, an invalid bitwidth in device memory) are
 *    recorded in an error word inside the pool / card header and returned
 *    by the *_status calls.  No kernel traps or asserts.  Two kinds of
 *    device-side wait exist, both bounded: the pool encoder's key-quantize
 *    work waits for its layer's scale, released by another block of the same
 *    kernel; pool attention, CacheCard unpack and attention over pages wait
 *    on mbarriers for their own bulk copies into shared memory.  A wait that
 *    runs out is recorded in the container's error word and reported as
 *    KVP_ERR_TIMEOUT by kvpool_status / cachecard_status / kvpages_status; the
 *    CUDA context stays usable.
 */
#ifndef KVPOOL_H
#define KVPOOL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
#define KVP_OK 0
#define KVP_ERR_ARG (-1)            /* null pointer, bad count or range      */
#define KVP_ERR_UNSUPPORTED_D (-2)  /* head_dim other than 64 or 128         */
#define KVP_ERR_ALIGN (-3)          /* pointer not aligned as required       */
#define KVP_ERR_SIZE (-4)           /* buffer too small / shape too large    */
#define KVP_ERR_CUDA (-5)           /* a CUDA call or kernel launch failed   */
#define KVP_ERR_NONFINITE (-6)      /* input held Inf or NaN                 */
#define KVP_ERR_RANGE (-7)          /* a scale or zero point overflowed fp16 */
#define KVP_ERR_BITS (-8)           /* CacheCard bitwidth not in {2,4,8,16}  */
#define KVP_ERR_HEADER (-9)         /* not a pool / card, or shape mismatch  */
#define KVP_ERR_TIMEOUT (-10)       /* a bounded device-side wait ran out    */
#define KVP_ERR_PAGE (-11)          /* slot, page id or length out of range  */

/* Largest layer count one call accepts. */
#define KVP_MAX_LAYERS 512

/* Key formats of a pool (the pool header records which one it holds). */
#define KVP_K_PER_TENSOR 0  /* one fp32 scale per layer's key tensor ("PolyKV" 2.B.1 text) */
#define KVP_K_Q8_0 1        /* q8_0 blocks: 32 keys along d share an fp16 scale (the label
                               "q8_0" that "PolyKV" 2.B.1 gives the same step)            */

/* Formats of a page container's keys and values. */
#define KVP_PAGES_BF16 0  /* both bf16                                               */
#define KVP_PAGES_K8V8 1  /* both q8_0: 32 along d share an fp16 scale, 8-bit codes  */
#define KVP_PAGES_K8V4 2  /* keys q8_0; values 4-bit, asymmetric groups of 32 along d
                             with an fp16 scale and zero point                      */

/* Shape of one KV cache: n_layers tensors of [n_kv_heads][n_tokens][head_dim]. */
typedef struct kvp_shape {
    int32_t n_layers;
    int32_t n_kv_heads;
    int32_t head_dim;
    int32_t n_tokens;
} kvp_shape;

/* CacheCard header, byte-for-byte the first 128 bytes of a card. */
typedef struct kvp_card_header {
    uint32_t magic;         /* 0x4343564B, bytes "KVCC"                        */
    uint32_t version;       /* 1                                              */
    int32_t seq_len;        /* T                                              */
    int32_t n_layers;       /* L                                              */
    int32_t n_kv_heads;     /* H                                              */
    int32_t head_dim;       /* d                                              */
    int32_t group_size;     /* 32                                             */
    int32_t dtype;          /* 1 = bf16                                       */
    uint64_t model_id;      /* opaque id of the model that produced the cache */
    int64_t pos_offset;     /* position of token 0 in the sender's sequence   */
    uint64_t off_bits;      /* byte offset of uint8 bits[T]                    */
    uint64_t off_offsets;   /* byte offset of uint32 off[T] (record offsets)   */
    uint64_t off_layers;    /* byte offset of layer 0's records                */
    uint64_t layer_stride;  /* bytes per layer                                 */
    uint64_t total_bytes;   /* bytes of the whole card                         */
    uint32_t error;         /* device-detected error bits                      */
    uint32_t reserved[9];
} kvp_card_header;

/* ---------------------------------------------------------------------- */
/* SharedKVPool                                                            */
/* ---------------------------------------------------------------------- */

/* Exact byte size of the pool for this shape, or 0 for an invalid shape.
 * Independent of how many agents will read it ("PolyKV" 2.A).
 * Pool layout (every section 256-byte aligned): 256-byte header (magic
 * "KVPL", version 1, L, H, d, T, error word, section offsets), fp32 K scale
 * per layer, then per layer: int8 K codes [H][T][d], 3-bit V codes
 * [H][T][3d/8] (8 codes c_0..c_7 = the 24-bit little-endian word
 * sum c_j << 3j), fp16 sigma [H][T]. */
size_t kvpool_pool_bytes(const kvp_shape *shape);

/* Bytes of device workspace kvpool_encode needs for this shape (0 for an
 * invalid shape).  The workspace holds the encoder's work-queue control
 * block (queue head, per-layer key maxima and ready flags) and per-layer
 * quantization parameters; its contents need no initialisation and are
 * dead after the encode's kernels finish. */
size_t kvpool_workspace_bytes(const kvp_shape *shape);

/* Encode a whole KV cache into a pool ("PolyKV" 2.B).
 *  k_layers, v_layers: host arrays of n_layers device pointers, each a bf16
 *    [H][T][d] tensor (16-byte aligned).
 *  Keys: per layer, s = max|k| / 127 rounded once to fp32; code = the
 *    integer nearest to the exact k/s (ties to even), in [-127,127]; s = 0
 *    gives all-zero codes.
 *  Values: per (token, head) vector v, y = H_d v (Sylvester-order
 *    Walsh-Hadamard), sigma = ||v||/sqrt(d) stored as fp16, u = y/||v||, and
 *    code = number of Lloyd-Max thresholds (midpoints of
 *    +-0.2451/0.7560/1.3440/2.1520) not above u; a zero vector codes as 4.
 *  pool: pool_bytes >= kvpool_pool_bytes(shape), 256-byte aligned; fully
 *    overwritten.  ws: ws_bytes >= kvpool_workspace_bytes(shape).
 * Non-finite input or a sigma above the fp16 range is reported by
 * kvpool_status (the affected codes are then unspecified). */
int kvpool_encode(const kvp_shape *shape, const void *const *k_layers,
                  const void *const *v_layers, void *pool, size_t pool_bytes,
                  void *ws, size_t ws_bytes, void *stream);

/* Pool bytes for key format k_mode (KVP_K_PER_TENSOR: as kvpool_pool_bytes;
 * KVP_K_Q8_0: that plus the block scales, 2 * n_layers * H * T * d/32 bytes
 * rounded up to 256).  0 for an invalid shape or format. */
size_t kvpool_pool_bytes_ex(const kvp_shape *shape, int k_mode);

/* kvpool_encode with the key format chosen by k_mode.  KVP_K_PER_TENSOR is
 * kvpool_encode.  KVP_K_Q8_0 ("PolyKV" 2.B.1 labels the key step "q8_0"):
 * every 32 consecutive keys of a vector share the scale
 * s_b = fp16(max|k| / 127) (round to nearest even); code = the integer
 * nearest to the exact k / s_b (ties to even) clamped to [-127, 127] (the
 * clamp only acts when s_b is an fp16 subnormal); s_b = 0 gives codes 0.  No
 * layer-wide maximum is needed, so keys and values are encoded in one pass.
 * Values as kvpool_encode.  pool_bytes >= kvpool_pool_bytes_ex(shape,
 * k_mode); ws as kvpool_encode.  A block whose scale overflows fp16 is
 * reported as KVP_ERR_RANGE by kvpool_status, non-finite keys as
 * KVP_ERR_NONFINITE (they code as 0).  Returns KVP_ERR_ARG for an unknown
 * k_mode. */
int kvpool_encode_ex(const kvp_shape *shape, int k_mode, const void *const *k_layers,
                     const void *const *v_layers, void *pool, size_t pool_bytes,
                     void *ws, size_t ws_bytes, void *stream);

/* Fan-out decode ("PolyKV" 2.A PooledAgent, 2.B.2 dequantization): read
 * layers [layer_begin, layer_end) of the pool once and write the decoded
 * bf16 K and V into each of n_agents caches.
 *  K: bf16(q * s_l), or bf16(q * s_b) with the key's block scale in a
 *    q8_0 pool (the format is read from the pool header on the device).
 *    V: bf16(sigma_h * (H_d c) / sqrt(d)) with c the centroids of the codes
 *    (the orthonormal transform is its own inverse).
 *  shape must equal the shape the pool was encoded with.
 *  k_dst, v_dst: host arrays of n_agents * n_layers device pointers,
 *    agent-major (entry a * n_layers + l is agent a's layer l, a bf16
 *    [H][T][d] tensor, 16-byte aligned).  Only entries of layers in the
 *    range are read; the others may be NULL.
 * The pool is only read, so decodes of one pool may run concurrently on
 * several streams.  A pool whose header does not match `shape` is left
 * undecoded and kvpool_status reports KVP_ERR_HEADER. */
int kvpool_decode_into(const void *pool, const kvp_shape *shape, int layer_begin,
                       int layer_end, int n_agents, void *const *k_dst,
                       void *const *v_dst, void *stream);

/* Synchronises `stream`, then returns KVP_OK or the first device-detected
 * error recorded in the pool's header (KVP_ERR_HEADER if `pool` does not
 * hold a version-1 pool). */
int kvpool_status(const void *pool, void *stream);

/* Size of the library's own device scratch array used by
 * kvpool_encode_noalloc (256 KiB on every GPU that loads the library, held
 * until the process exits). */
#define KVP_NOALLOC_SCRATCH_BYTES 262144

/* kvpool_encode without a caller workspace.  This entry point has no
 * counterpart in the papers; it exists for callers that cannot allocate
 * device memory -- e.g. a plug-in inside another program's process that must
 * not allocate behind its host's memory manager, or a latency-critical caller
 * for which a cudaMalloc could synchronise the device.  It allocates nothing
 * (no cudaMalloc, cudaFree or allocating library call): the workspace is a
 * fixed array of KVP_NOALLOC_SCRATCH_BYTES in the library's device memory.
 *  Arguments and results are those of kvpool_encode minus ws / ws_bytes.
 *  The encoder's workspace is a control block of about 6 KB plus 16 bytes
 *    per layer, so every shape kvpool_encode accepts fits in the array.  A
 *    shape it refuses is refused here with the same code, before anything
 *    is enqueued.
 *  The first call in each CUDA context looks up the array's device address
 *    (with that context current) and caches it under the driver's context
 *    id; make that first call before any stream capture.  A context created
 *    later (after cudaDeviceReset, say) gets a fresh lookup on its first
 *    call, so the library may outlive a context.
 *  Every call on a device shares the one array.  The encoder overwrites
 *    everything it reads from it, so nothing needs clearing between calls,
 *    but calls that overlap on the GPU (other streams, no ordering between
 *    them) race on the array: order them on one stream or with events. */
int kvpool_encode_noalloc(const kvp_shape *shape, const void *const *k_layers,
                          const void *const *v_layers, void *pool, size_t pool_bytes,
                          void *stream);

/* ---------------------------------------------------------------------- */
/* Attention over the pool                                                 */
/* ---------------------------------------------------------------------- */

/* Bytes of device workspace kvpool_attend needs (0 for an invalid shape or
 * head count).  Holds per-split partial results; no initialisation. */
size_t kvpool_attend_workspace_bytes(const kvp_shape *shape, int n_agents, int n_q_heads);

/* One decode step of attention of n_agents agents' queries over layer
 * `layer` of the pool, computed from the compressed bytes without writing any
 * bf16 cache: the fused attention over the quantized cache that "QKVShare"
 * (Significance) leaves as future work, on "PolyKV" 2.A's shared pool.
 *  q: device bf16 [n_agents][n_q_heads][head_dim], 16-byte aligned; query head
 *    j reads KV head j / (n_q_heads / n_kv_heads) (n_q_heads a multiple of
 *    n_kv_heads: grouped-query attention).
 *  For each (agent, head): s_t = scale * (q . k_t) over the T pooled tokens
 *    with k_t = code_t * s_layer (q8_0 pools: code * s_b per 32-key block;
 *    the format is read from the pool header); out = sum_t softmax(s)_t v_t with v_t the
 *    decoded value (sigma_t * H_d c_t / sqrt(d), accumulated in the rotated
 *    domain and transformed once); lse = log sum_t exp(s_t) (natural log), so a
 *    caller can merge with attention over its own further tokens.
 *  out: device fp32 [n_agents][n_q_heads][head_dim] (16-byte aligned); lse:
 *    device fp32 [n_agents][n_q_heads].  ws: kvpool_attend_workspace_bytes.
 *  Precision: scores are exact products accumulated in fp32 (q8_0: exact
 *  per-block partial sums, each scaled by its block scale in fp32);
 *  probabilities times sigma enter the value product as fp16, centroids as
 *  fp16.  A pool whose header does not match `shape` is not read and
 *  kvpool_status reports KVP_ERR_HEADER.  The kernel streams the pool's bytes
 *  into shared memory with bulk copies and waits on them for at most about
 *  half a second; should a wait run out, out / lse are unspecified and
 *  kvpool_status reports KVP_ERR_TIMEOUT.  Errors are recorded in the pool's
 *  error word (the only bytes of the pool a call may write). */
int kvpool_attend(const void *pool, const kvp_shape *shape, int layer, int n_agents, int n_q_heads,
                  const void *q, float scale, float *out, float *lse, void *ws, size_t ws_bytes,
                  void *stream);

/* Bytes of device workspace kvpool_attend_lora needs (0 for an invalid shape,
 * head count or rank). */
size_t kvpool_attend_lora_workspace_bytes(const kvp_shape *shape, int n_agents, int n_q_heads, int rank);

/* Pool attention for agents that differ by a LoRA adapter on the value
 * projection, with one shared low-rank cache ("LRAgent": BaseLRShared shares
 * the base cache and the low-rank cache X A between agents, each agent keeping
 * its own up-projection B; Flash-LoRA-Attention computes
 * P (V_base + V_lr B) as P V_base + (P V_lr) B, so the up-projection is
 * applied once per query instead of expanding the cache).  Agent a's value of
 * token t at KV head h is
 *   v = (the pool's decoded value) + sum_k v_lr[t][k] * lora_b[a][k][h*d + i];
 * otherwise as kvpool_attend (same out, lse, GQA map and key formats).
 *  rank: 16 or 32 (KVP_ERR_ARG otherwise).
 *  v_lr: device bf16 [n_tokens][rank], the layer's shared low-rank cache
 *    (16-byte aligned).  It enters the product as fp16: exact for values in
 *    fp16's normal range, |x| in [2^-14, 65504].
 *  lora_b: device bf16 [n_agents][rank][n_kv_heads * head_dim], each agent's
 *    up-projection with rank-major rows (the transpose of a PyTorch LoRA
 *    B weight), 16-byte aligned.
 *  ws: kvpool_attend_lora_workspace_bytes. */
int kvpool_attend_lora(const void *pool, const kvp_shape *shape, int layer, int n_agents, int n_q_heads,
                       const void *q, float scale, int rank, const void *v_lr, const void *lora_b, float *out,
                       float *lse, void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------- */
/* CacheCard                                                               */
/* ---------------------------------------------------------------------- */

/* Exact byte size of a card for these per-token bitwidths (host array of
 * n_tokens values), or 0 if the shape or any bitwidth is invalid.
 * Card layout: 128-byte header (kvp_card_header), uint8 bits[T], uint32
 * off[T] (16-byte aligned; exclusive prefix sum of record sizes), then
 * n_layers layers of layer_stride bytes (256-byte aligned).  A token's
 * record in one layer, b in {2,4,8}: K codes [H][d] then V codes [H][d] at b
 * bits (each group of 32 coordinates a little-endian bit string, code j at
 * bits j*b..j*b+b-1), then K (fp16 scale, fp16 zero) [H][d/32], then V
 * (scale, zero) [H][d/32]; b = 16: K then V verbatim.  Records are padded to
 * 16 bytes. */
size_t cachecard_bytes(const kvp_shape *shape, const uint8_t *bits_host);

/* Pack a CacheCard ("QKVShare" Methodology 1-2).
 *  bits_dev: device array of n_tokens bitwidths in {2,4,8,16}.
 *  For b < 16, per group of 32 coordinates of one (layer, token, K|V, head):
 *    s_h = fp16((max-min)/(2^b-1)), z_h = fp16(min), code =
 *    clamp(nearest integer to (x - z_h)/s_h, 0, 2^b-1) (0 when s_h = 0).
 *    b = 16 copies the bf16 values.
 *  card: card_bytes bytes, 256-byte aligned; must hold cachecard_bytes()
 *    for these bits, otherwise nothing but the header is written and
 *    cachecard_status reports KVP_ERR_SIZE (KVP_ERR_BITS for an invalid
 *    bitwidth). */
int cachecard_pack(const kvp_shape *shape, uint64_t model_id, int64_t pos_offset,
                   const uint8_t *bits_dev, const void *const *k_layers,
                   const void *const *v_layers, void *card, size_t card_bytes,
                   void *stream);

/* Copy the card's 128-byte header to *out (synchronises `stream`).  Returns
 * KVP_ERR_HEADER if the magic or version is wrong. */
int cachecard_read_header(const void *card, kvp_card_header *out, void *stream);

/* Receiver injection ("QKVShare" Methodology 3): rebuild every layer's bf16
 * K and V ([H][T][d]) from the card: x = bf16(q * s_h + z_h), 16-bit tokens
 * verbatim.  hdr is the header read by cachecard_read_header.  k_dst, v_dst:
 * host arrays of n_layers device pointers (16-byte aligned).  The header's
 * fields are checked on the host (KVP_ERR_HEADER); a token whose bitwidth is
 * invalid or whose record offset is not 16-byte aligned or does not fit the
 * layer stride is left unwritten, and cachecard_status then reports
 * KVP_ERR_HEADER.  Where the shape allows it (see kvp_test_limit_next_unpack)
 * records are staged through shared memory by bulk copies. */
int cachecard_unpack(const void *card, const kvp_card_header *hdr,
                     void *const *k_dst, void *const *v_dst, void *stream);

/* Receiver injection at other positions: as cachecard_unpack, but every key
 * is moved from its position in the sender's sequence (hdr->pos_offset + t)
 * to pos_dst + t.  The card's metadata carries the position offset
 * ("QKVShare" Methodology 2), and a reused segment's key positions are
 * re-aligned to the target agent's ("KVCMAS", How it is used).  Under rotary
 * position embedding -- dims i and i + d/2 turned through p * w_i at
 * position p, the Hugging Face Llama pairing -- that is one further turn of
 * every pair through (pos_dst - hdr->pos_offset) * w_i.
 *   inv_freq: HOST array of head_dim/2 fp32 frequencies w_i (radians per
 *     position; the model's rotary inverse frequencies, any scaling already
 *     applied).  Copied into the launch, so it may be freed on return.
 *   The angle is formed and its sine and cosine taken in fp64; each key is
 *   dequantized and turned in fp32 and rounded to bf16 once.  Values are
 *   unpacked exactly as by cachecard_unpack.  pos_dst == hdr->pos_offset
 *   gives cachecard_unpack's output bit for bit.
 * Returns KVP_ERR_ARG for a null inv_freq, a non-finite frequency or a shift
 * that overflows int64; otherwise as cachecard_unpack. */
int cachecard_unpack_at(const void *card, const kvp_card_header *hdr, int64_t pos_dst,
                        const float *inv_freq, void *const *k_dst, void *const *v_dst,
                        void *stream);

/* Synchronises `stream`, then returns KVP_OK or the first device-detected
 * error recorded in the card's header. */
int cachecard_status(const void *card, void *stream);

/* ---------------------------------------------------------------------- */
/* Pages: an agent's own cache                                             */
/* ---------------------------------------------------------------------- */

/* Most sequences of one kvpages_attend call. */
#define KVP_PAGES_MAX_SEQS 4096

/* A page container: n_pages pages in each of n_layers layers; a page holds
 * page_tokens tokens (a power of two, 16 to 1024) of all KV heads.  Which
 * pages hold which sequence is the caller's: a table row of page ids per
 * sequence; sequences may share pages. */
typedef struct kvp_pages_config {
    int32_t n_layers;
    int32_t n_kv_heads; /* at most 4096 */
    int32_t head_dim;
    int32_t page_tokens;
    int32_t n_pages;
    int32_t format;     /* KVP_PAGES_* */
} kvp_pages_config;

/* A bf16 tensor [tokens][heads][head_dim] with strides in elements (multiples
 * of 8; the innermost dimension contiguous): the slices of a fused projection's
 * output, or of a [heads][tokens][head_dim] tensor, as they lie. */
typedef struct kvp_rows {
    const void *ptr;
    int64_t token_stride;
    int64_t head_stride;
} kvp_rows;

/* Exact byte size of a container, or 0 for an invalid configuration.
 * Layout: 256-byte header (magic "KVPG", version 1, L, H, d, page_tokens,
 * error word, format, n_pages, layer stride, total bytes), then per layer
 * (256-byte aligned) n_pages x H tiles of page_tokens / 16 blocks; a block is
 * 16 tokens of one head: keys, values, key scales, value scales. */
size_t kvpages_bytes(const kvp_pages_config *cfg);

/* Writes the header (and clears the error word).  The pages need no
 * initialisation: what was never written is never read. */
int kvpages_init(const kvp_pages_config *cfg, void *pages, size_t pages_bytes, void *stream);

/* Write new tokens of one layer: the norm of every query and key head, the
 * position rotation, and the quantised write, in one pass.
 *  q, k, v: [n_tokens][n_q_heads or n_kv_heads][head_dim] rows.  q and q_out
 *    may be NULL when n_q_heads is 0.
 *  slots: device int64[n_tokens], the place of each token: page id *
 *    page_tokens + index in the page.  Negative: the token is not cached (its
 *    outputs are still written).  Two tokens of a call may not share a slot.
 *  q_norm, k_norm: device bf16[head_dim] or NULL: y = x / sqrt(mean(x^2) +
 *    eps) * w per head, in fp32; NULL leaves the heads as they are.
 *  rot_dim: 0, 64, or 128 at head_dim 128: dims i and i + rot_dim/2
 *    (i < rot_dim/2) turned by positions[t] * inv_freq[i]; the rest pass.
 *    positions: device int64[n_tokens]; inv_freq: HOST array of rot_dim/2
 *    fp32 frequencies (below 2^60 in magnitude), read during the call only.  The
 *    angle is reduced to a turn with an error below |position| * 2^-64 turns, its
 *    sine and cosine taken in fp32.
 *  q_out: device bf16 [n_tokens][n_q_heads][head_dim] contiguous.
 *  k_out, v_out: device bf16 [n_tokens][n_kv_heads][head_dim] contiguous, or
 *    NULL: the keys and values as the cache now holds them, for a prompt's own
 *    attention.  No output may overlap an input, except that q_out may be q's
 *    own contiguous tensor.
 * Codes: 8-bit s = fp16(max|x| * fl(1/127)), code = RNE(x / s) in [-127, 127],
 * of the rotated key in fp32 (never rounded to bf16 first); 4-bit
 * s = fp16(fl(max - min) * fl(1/15)), z = fp16(min), code = RNE((x - z) / s) in
 * [0, 15]; s = 0 gives codes 0.  Non-finite elements are kept in BF16 pages;
 * elsewhere they count and code as zeros and kvpages_status reports
 * KVP_ERR_NONFINITE; a scale or zero point beyond fp16 is held at its largest
 * value and reported as KVP_ERR_RANGE; a slot past the container is not
 * written and reported as KVP_ERR_PAGE. */
int kvpages_append(void *pages, const kvp_pages_config *cfg, int layer, int n_tokens, int n_q_heads,
                   const kvp_rows *q, const kvp_rows *k, const kvp_rows *v, const int64_t *slots,
                   const int64_t *positions, const void *q_norm, const void *k_norm, float eps, int rot_dim,
                   const float *inv_freq, void *q_out, void *k_out, void *v_out, void *stream);

/* Read sequences back as bf16 past_key_values of one layer.
 *  table: device int32 [n_seqs][max_pages] page ids; lens: device
 *    int32[n_seqs] tokens of each sequence (table entries past a sequence's
 *    length are not read).
 *  k_dst, v_dst: device bf16 [n_seqs][n_kv_heads][max_tokens][head_dim];
 *    sequence b's first min(lens[b], max_tokens) tokens, zeros after them.
 * A page id outside the container, or a length beyond its table row, reads as
 * zeros and is reported by kvpages_status as KVP_ERR_PAGE. */
int kvpages_read(const void *pages, const kvp_pages_config *cfg, int layer, int n_seqs, const int32_t *table,
                 int max_pages, const int32_t *lens, int max_tokens, void *k_dst, void *v_dst, void *stream);

/* Bytes of device workspace kvpages_attend needs (0 for invalid counts).  No
 * initialisation. */
size_t kvpages_attend_workspace_bytes(const kvp_pages_config *cfg, int n_seqs, int n_q_tokens, int n_q_heads);

/* Attention of each sequence's newest n_q_tokens tokens (1 to 64; already
 * written to the pages) over the sequence's pages, causal among themselves:
 * query token i of sequence b sees the first lens[b] - (n_q_tokens - 1 - i)
 * tokens.
 *  q: device bf16 [n_seqs][n_q_tokens][n_q_heads][head_dim]; query head j reads
 *    KV head j / (n_q_heads / n_kv_heads).
 *  table, max_pages, lens: as kvpages_read; n_seqs at most KVP_PAGES_MAX_SEQS,
 *    and n_seqs * max_pages * page_tokens below 2^35.
 *  base_out, base_lse: device fp32 [n_seqs][n_q_tokens][n_q_heads]([head_dim]),
 *    both or neither (NULL): attention of the same queries over other tokens,
 *    as kvpool_attend leaves it.  The result is then attention over both.
 *  out: device bf16 [n_seqs][n_q_tokens][n_q_heads][head_dim].  lse: device
 *    fp32 [n_seqs][n_q_tokens][n_q_heads] or NULL (natural log).  No output may
 *    overlap an input or another output, except that lse may be base_lse.
 * An Inf or NaN value of a BF16 page is one in its dim for the queries that see
 * its token (weights are positive, however small), and touches no others.  Finite
 * values give finite results up to bf16's largest.  Weights below 2^-118 of the
 * largest count as zero; where a sequence holds values of 2^64 or more, so do its
 * values below 2^-86.
 * A query that sees no token gets the base's output and lse, or zeros and -inf
 * without one.  Scores are products of the stored codes accumulated in fp32 (over
 * 8-bit keys a query row enters as fp16 times a power of two, exactly but for
 * elements below 2^-28 of its largest); softmax statistics are fp32, exponentials
 * the hardware's in base 2 (2^-22); the weights (times the values' scales) enter
 * the value product as a sum of two bf16 (2^-17).  The kernel waits for its bulk
 * copies of the pages at most about half a second; should a wait run out, the
 * outputs are unspecified and kvpages_status reports KVP_ERR_TIMEOUT.  A page id
 * outside the container or a length beyond its table row is skipped and reported
 * by kvpages_status as KVP_ERR_PAGE.
 * Speed: the lengths are known on the device only, so it is max_pages that chooses
 * how the work is split.  Where no row can hold more than some thousand tokens, a
 * team of warps takes each row tile, in one launch; otherwise equal runs of all
 * tokens are joined by a second one.  A table trimmed to the longest sequence is
 * therefore faster for short ones: 15 of 200 tokens take 6.3 us, 10.1 with rows for
 * 32768 tokens (64 of them 11.5 and 18.9; from some 2000 tokens on no difference). */
int kvpages_attend(const void *pages, const kvp_pages_config *cfg, int layer, int n_seqs, int n_q_tokens,
                   int n_q_heads, const void *q, float scale, const int32_t *table, int max_pages,
                   const int32_t *lens, const float *base_out, const float *base_lse, void *out, float *lse, void *ws,
                   size_t ws_bytes, void *stream);

/* Synchronises `stream`, then returns KVP_OK or the first device-detected
 * error recorded in the container's header (KVP_ERR_HEADER if `pages` does not
 * hold a version-1 container, or a call described another one). */
int kvpages_status(const void *pages, void *stream);

/* ---------------------------------------------------------------------- */
/* Diagnostics                                                             */
/* ---------------------------------------------------------------------- */

/* Static, human-readable text for a status code. */
const char *kvp_strerror(int status);

/* Number of kernels this library has launched in this process. */
uint64_t kvp_launch_count(void);

/* Bandwidth probes (the papers have no counterpart: measurement support).
 * They give the HBM ceiling of the access pattern each codec kernel uses, so
 * a benchmark can report a kernel against its own pattern's ceiling.
 *  KVP_PROBE_STORE: write `bytes` to dst with 16-byte streaming stores, one
 *    resident grid walking the buffer (the one-agent decode's and the card
 *    unpack's store pattern).  bytes a multiple of 16.
 *  KVP_PROBE_BULK_STORE: write `bytes` to dst as 4 KB bulk copies from
 *    shared memory, one per warp (the fan-out decode's store pattern).
 *    bytes a multiple of 4096.
 *  KVP_PROBE_COPY: copy `bytes` from src to dst with 16-byte loads and
 *    stores (read + write).  bytes a multiple of 16; src 256-byte aligned.
 * dst: device buffer of at least `bytes`, 256-byte aligned; its contents are
 * overwritten with an arbitrary pattern.  Enqueues one kernel on `stream`.
 * Returns KVP_ERR_ARG (unknown mode, null pointer, zero bytes),
 * KVP_ERR_ALIGN or KVP_ERR_SIZE before launching anything. */
#define KVP_PROBE_STORE 0
#define KVP_PROBE_BULK_STORE 1
#define KVP_PROBE_COPY 2
int kvp_bandwidth_probe(int mode, void *dst, const void *src, size_t bytes, void *stream);

/* Failure-path testing.  The pool encoder's key-quantization work waits, with
 * an iteration limit, for a per-layer "scale ready" flag set by other blocks
 * of the same kernel; a wait that runs out is reported by kvpool_status as
 * KVP_ERR_TIMEOUT and leaves the CUDA context usable.  Calling this with
 * layer >= 0 makes the NEXT kvpool_encode on this thread leave that layer's
 * flag unset and wait at most spin_iters iterations (about 100 ns each), so
 * a test can exercise that path; layer < 0 restores normal operation.
 * Returns KVP_OK. */
int kvp_test_fail_next_encode(int layer, uint32_t spin_iters);

/* Failure-path testing of pool attention.  Its split kernel waits, with a
 * bounded number of polls, for the bulk copies of each sub-chunk; a wait that
 * runs out is reported by kvpool_status as KVP_ERR_TIMEOUT (the block first
 * lets its copies in flight land, with the normal limit) and leaves the CUDA
 * context usable.  Makes the NEXT kvpool_attend / kvpool_attend_lora on this
 * thread poll each sub-chunk's copies at most `polls` times (0: not at all, so
 * every block gives up on its first sub-chunk).  Returns KVP_OK. */
int kvp_test_limit_next_attend(uint32_t polls);

/* Failure-path testing of CacheCard unpack.  Where the shape lets it stage
 * records in shared memory (d = 128 or an even n_kv_heads, and 32 n_kv_heads
 * head_dim bytes of buffers per block within 96 KB), unpack waits, with a
 * bounded number of polls, for the bulk copies of each record; a wait that
 * runs out is reported by cachecard_status as KVP_ERR_TIMEOUT (the warp
 * first lets its copies in flight land, with the normal limit, and leaves
 * that layer's outputs incomplete) and leaves the CUDA context usable.
 * Makes the NEXT cachecard_unpack / cachecard_unpack_at on this thread poll
 * each record's copies at most `polls` times (0: not at all, so every warp
 * gives up on its first record); other shapes ignore it.  Returns KVP_OK. */
int kvp_test_limit_next_unpack(uint32_t polls);

/* Failure-path testing of attention over pages: makes the NEXT kvpages_attend
 * on this thread poll each block's copy at most `polls` times (0: not at all,
 * so every warp gives up on its first block, lets its copies in flight land
 * with the normal limit, and leaves its rows unwritten); kvpages_status then
 * reports KVP_ERR_TIMEOUT and the CUDA context stays usable.  Returns KVP_OK. */
int kvp_test_limit_next_pages_attend(uint32_t polls);

/* The same for the lanes of every warp whose bits are set in `lanes`; the other
 * lanes wait with the normal limit.  A warp gives up if any of its lanes does:
 * with one bit set the outcome is that of kvp_test_limit_next_pages_attend. */
int kvp_test_limit_next_pages_attend_lanes(uint32_t polls, uint32_t lanes);

#ifdef __cplusplus
}
#endif

#endif /* KVPOOL_H */
