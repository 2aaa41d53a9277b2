/*
 * tk.h -- C ABI of libtk: byte-level BPE encoding on one GB300 (sm_103a).
 *
 * The library encodes typed text segments into token ids with a tiktoken-style
 * encoding: a bytes->rank table whose rank is the id, the cl100k split pattern,
 * and a dict of special tokens ("tiktoken Deep Dive", "An encoding is three
 * objects, not a model").  One call encodes a whole prompt of ordered
 * (text, allow_special) segments ("Making Kimi K3 Tokenization 18x Faster For
 * Million Token Agentic Workloads", "One native call for the whole serving
 * path"); every step of the encode runs in CUDA kernels, ordered on the
 * caller's stream.
 *
 * Conventions
 *   - "d_" pointers are device pointers, "h_" pointers are host pointers.
 *   - The caller owns every input and output buffer.  tk_load copies its
 *     tables into library-owned device memory; a workspace owns the scratch
 *     of one encode in flight (one workspace per concurrent stream).
 *   - Every function returns TK_OK (0) or a negative TK_E_* code, and leaves
 *     outputs unspecified on error.  tk_last_error() gives a one-line message
 *     for the calling thread's last failure.
 *   - Ids are int32; token byte offsets are int64.  Texts are limited to
 *     2^31 - 1024 bytes per call.
 */
#ifndef TK_H
#define TK_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct tk_tokenizer tk_tokenizer;
typedef struct tk_workspace tk_workspace;

enum {
  TK_OK = 0,
  TK_E_ARG = -1,      /* bad argument (null pointer, negative size, unknown pattern) */
  TK_E_TABLE = -2,    /* rank/special table rejected by tk_load */
  TK_E_UTF8 = -3,     /* input text is not valid UTF-8 (position in tk_last_error) */
  TK_E_CAPACITY = -4, /* output buffer too small; the required size is still returned */
  TK_E_CUDA = -5,     /* a CUDA runtime call failed */
  TK_E_NOMEM = -6,    /* host or device allocation failed */
  TK_E_TIMEOUT = -7,  /* a bounded device-side wait gave up (never expected) */
  TK_E_BADID = -8,    /* tk_decode met an id that is neither a rank nor a special */
  TK_E_LIMIT = -9     /* input exceeds the workspace's max_bytes / max_segments */
};

enum { TK_PATTERN_CL100K = 1, TK_PATTERN_R50K_DIGITS = 2 };

/*
 * tk_load -- build a tokenizer from host arrays (copied; the caller may free
 * them on return).
 *
 *   rank_bytes, rank_off[n+1], rank_ids[n]: mergeable token i is
 *       rank_bytes[rank_off[i] .. rank_off[i+1]) with rank (= id) rank_ids[i]
 *       ("tiktoken Deep Dive", "An encoding is three objects": one map
 *       bytes -> rank where the rank is the token id).  rank_off[0] must be 0.
 *   spec_bytes, spec_off[n_spec+1], spec_ids[n_spec]: special tokens, matched
 *       by exact string outside the merge loop ("Special tokens and the
 *       injection nobody plans for").  May be empty (n_spec = 0).
 *   pattern_id: TK_PATTERN_CL100K, the pattern printed in "tiktoken Deep
 *       Dive", "The split pattern"; or TK_PATTERN_R50K_DIGITS, the same
 *       alternation with r50k's digit clause " ?\p{N}++" (an unbounded digit
 *       run with an optional leading space; "r50k, cl100k, o200k") in place
 *       of cl100k's \p{N}{1,3}+.
 *
 * Rejected with TK_E_TABLE: a missing single byte ("The byte floor": all 256
 * bytes must be tokens), duplicate token bytes, duplicate ids, ids >= 2^20 - 1,
 * empty tokens, specials longer than 64 bytes or not valid UTF-8, special ids
 * that collide with ranks, and specials that can overlap one another in text
 * (a suffix of one equal to a prefix of another, or one inside another).
 * The handle is immutable after load and may be shared across threads.
 */
int tk_load(const uint8_t* rank_bytes, const int64_t* rank_off, const uint32_t* rank_ids,
            int64_t n, const uint8_t* spec_bytes, const int64_t* spec_off,
            const int32_t* spec_ids, int64_t n_spec, int pattern_id, tk_tokenizer** out);

void tk_free(tk_tokenizer* tok);

/*
 * tk_workspace_create -- allocate the device scratch for encodes of up to
 * max_bytes bytes in up to max_segments segments ("tokenizers v1: encode,
 * decode and scaling, measured", "Key Technical Improvements": the merge
 * working set lives in a caller-owned scratch buffer, so an encode never
 * touches an allocator).  About 44 bytes of device memory per byte of
 * max_bytes (11.9 GB for max_bytes = 256 MiB: seven 4-byte arrays indexed
 * by byte position for the long-piece merges, the per-tile staging of the
 * ids, the host-call staging, the mid-piece lists and the bitmaps).  A
 * workspace serves one encode at a time.
 */
int tk_workspace_create(const tk_tokenizer* tok, int64_t max_bytes, int64_t max_segments,
                        tk_workspace** out);

void tk_workspace_free(tk_workspace* ws);

/*
 * tk_encode_segments -- encode S ordered segments in one call.
 *
 *   d_text[n_bytes]: the segments' UTF-8 bytes, concatenated.
 *   d_seg_off[S+1]: segment s is d_text[d_seg_off[s] .. d_seg_off[s+1]);
 *       d_seg_off[0] = 0, non-decreasing, d_seg_off[S] = n_bytes.
 *   d_allow_special[S]: 1 = special strings in this segment become their
 *       special ids; 0 = they are ordinary text ("Making Kimi K3
 *       Tokenization ...", "Why Kimi K3 tokenization is non-trivial": user and
 *       tool text keeps literal control strings as text).
 *   tiktoken_safe: 1 = first cut each segment into windows of at most 400,000
 *       characters, then cut runs of white-space or non-white-space
 *       characters at 25,000 characters ("One native call for the whole
 *       serving path"); each piece is encoded on its own.
 *   d_out_ids[out_capacity]: receives the ids in input order.
 *       out_capacity >= n_bytes always suffices (every token covers >= 1 byte).
 *   d_out_offsets[S+1]: segment s's ids are d_out_ids[d_out_offsets[s] ..
 *       d_out_offsets[s+1]); d_out_offsets[S] is the total.
 *   h_n_ids: receives the total number of ids (also when it exceeds
 *       out_capacity, in which case TK_E_CAPACITY is returned).
 *   cuda_stream: a cudaStream_t (NULL = legacy default stream).  The encode
 *       is ordered on this stream: the kernels of the pre-tokens of 5 bytes
 *       or more run on the workspace's side streams, forked from and joined
 *       back into cuda_stream by events, so work queued on cuda_stream before
 *       the call is seen and work queued after it waits for the whole encode.
 *       The one device->host status read goes on cuda_stream (on the graph's
 *       stream for a replayed call, below); the call returns after that read
 *       completes.
 *
 * Repeated calls: when a workspace sees the same arguments (tokenizer,
 * buffer addresses, sizes, tiktoken_safe, attached cache) a second time in a
 * row, for a call under 16 MiB, it captures the call's launches into a CUDA
 * graph and replays it from then on (on a stream of its own, joined with cuda_stream by events, with
 * the same ordering as above).  The buffers' contents may change between
 * calls; the graph reads them when it runs.  Calls with per-kernel profiling
 * on, and every call after a capture that failed, launch directly.
 *
 * Errors: TK_E_ARG, TK_E_LIMIT (n_bytes or S above the workspace's limits),
 * TK_E_UTF8 (invalid UTF-8; tk_last_error gives the first bad byte offset),
 * TK_E_CAPACITY, TK_E_CUDA, TK_E_TIMEOUT.
 */
int tk_encode_segments(const tk_tokenizer* tok, tk_workspace* ws, const uint8_t* d_text,
                       int64_t n_bytes, const int64_t* d_seg_off,
                       const uint8_t* d_allow_special, int64_t S, int tiktoken_safe,
                       int32_t* d_out_ids, int64_t out_capacity, int64_t* d_out_offsets,
                       int64_t* h_n_ids, void* cuda_stream);

/*
 * tk_encode_segments_host -- the same encode for callers whose data lives in
 * host memory: h_text, h_seg_off, h_allow_special are copied to the
 * workspace's device staging buffers, the encode runs on cuda_stream, and the
 * ids and offsets are copied back into h_out_ids[out_capacity] and
 * h_out_offsets[S+1].  Pinned host buffers make the copies asynchronous.
 * Same arguments and errors as tk_encode_segments.
 */
int tk_encode_segments_host(const tk_tokenizer* tok, tk_workspace* ws, const uint8_t* h_text,
                            int64_t n_bytes, const int64_t* h_seg_off,
                            const uint8_t* h_allow_special, int64_t S, int tiktoken_safe,
                            int32_t* h_out_ids, int64_t out_capacity, int64_t* h_out_offsets,
                            int64_t* h_n_ids, void* cuda_stream);

/*
 * tk_decode -- ids -> bytes on the device ("tiktoken Deep Dive", "The byte
 * floor": a round trip reproduces the input byte for byte; "Pitfalls that
 * bite in production": the output is the concatenated bytes of all ids, since
 * one character's bytes may be spread over several ids).
 *
 *   d_ids[n]: ids (ranks or specials).  d_out[cap]: receives the bytes of each
 *   id in turn.  h_len: the total byte length (also when it exceeds cap, then
 *   TK_E_CAPACITY).  An id that is neither a rank nor a special (for example
 *   one in the reserved gap below the specials) gives TK_E_BADID.
 *   Uses the workspace for scratch (n <= max_bytes).
 */
int tk_decode(const tk_tokenizer* tok, tk_workspace* ws, const int32_t* d_ids, int64_t n,
              uint8_t* d_out, int64_t cap, int64_t* h_len, void* cuda_stream);

/*
 * tk_decode_segments -- tk_decode of S sequences at once (the ids of an
 * encode_segments call, say): d_ids[n] with d_id_off[S+1] (0 = d_id_off[0] <=
 * ... <= d_id_off[S] = n, else TK_E_ARG) -> their bytes one after the other in
 * d_out[cap] and d_byte_off[S+1], the byte offset of each sequence's first
 * byte (d_byte_off[S] = *h_len, the total).  Errors as for tk_decode.
 */
int tk_decode_segments(const tk_tokenizer* tok, tk_workspace* ws, const int32_t* d_ids, int64_t n,
                       const int64_t* d_id_off, int64_t S, uint8_t* d_out, int64_t cap,
                       int64_t* d_byte_off, int64_t* h_len, void* cuda_stream);

/*
 * tk_decode_stream -- incremental decode of ids that arrive in pieces
 * ("tiktoken Deep Dive", "Pitfalls that bite in production": tokens are not
 * characters, so a token can end inside a character; accumulate the bytes and
 * hold back any trailing partial sequence).
 *
 *   state: caller-owned, zeroed before the first call of a stream; holds the
 *       0..3 bytes held back by the previous call.
 *   d_ids[n]: the next ids.  final: nonzero on the last call of the stream
 *       (nothing is held back then; n may be 0 to flush).
 *   d_out[cap]: receives the held-back bytes of the previous call, then the
 *       bytes of d_ids; *h_len = the bytes it may emit now: all of them except
 *       a trailing proper prefix of a well-formed UTF-8 character (a lead byte
 *       C2..F4 with fewer continuation bytes than it announces, the second in
 *       its allowed range), which is kept in state for the next call.  A
 *       surrogate prefix (ED A0..BF) is not held: no character completes it.
 *   cap must hold state->n_pending + the bytes of d_ids; on TK_E_CAPACITY,
 *   *h_len is that total and state is unchanged (the call may be repeated),
 *   as for TK_E_BADID.  Uses the workspace for scratch (n <= max_bytes).
 */
typedef struct tk_decode_state {
  uint8_t pending[4]; /* held-back bytes (n_pending of them) */
  int32_t n_pending;  /* 0..3 */
} tk_decode_state;

int tk_decode_stream(const tk_tokenizer* tok, tk_workspace* ws, tk_decode_state* state,
                     const int32_t* d_ids, int64_t n, int final, uint8_t* d_out, int64_t cap,
                     int64_t* h_len, void* cuda_stream);

/*
 * tk_decode_noalloc -- tk_decode for callers that cannot allocate device
 * memory (a server whose memory pool already holds the device's memory, or a
 * latency-critical path that must not enter the allocator or the device
 * synchronisation cudaFree may imply).  The pages have no counterpart: this
 * is an engineering entry point of this library.
 *
 *   Same arguments and results as tk_decode, without a workspace: d_ids[n]
 *   (n <= 1,048,576, else TK_E_LIMIT), d_out[cap], *h_len = total bytes
 *   (TK_E_CAPACITY when it exceeds cap), TK_E_BADID for an unknown id.
 *   Allocates nothing: its scratch (about 4 KiB of look-back descriptors and
 *   a status block) is a fixed array compiled into the library, held by every
 *   GPU that loads it until the process exits.
 *
 *   The first call on a device looks up that array's device address (with
 *   that device current) and keeps it for the life of the process; make that
 *   first call before any stream capture.  The kept address belongs to the
 *   device's current context: after cudaDeviceReset on that device, do not
 *   call this entry point again in the same process.
 *   All calls on a device share the array: calls that overlap on the GPU race,
 *   so serialise them (for example on one stream).  Each call clears the part
 *   of the array it uses before its kernel runs, then copies its 64-byte
 *   status back into host memory and waits for cuda_stream to finish (every
 *   call synchronises cuda_stream).
 */
int tk_decode_noalloc(const tk_tokenizer* tok, const int32_t* d_ids, int64_t n, uint8_t* d_out,
                      int64_t cap, int64_t* h_len, void* cuda_stream);

/*
 * Cross-call word cache ("Making Kimi K3 Tokenization 18x Faster ...", "Where
 * the speed comes from": repeated words are merged once; "tokenizers v1",
 * "Key Technical Improvements": a word cache).  Within one call every
 * pre-token over 16 bytes is merged once per distinct byte string; a cache
 * keeps those merges between calls, for agent loops that resend most of
 * their prompt.  A hit returns the ids merged earlier for the same bytes and
 * the same tokenizer, so results never change.
 *
 *   tk_cache_create: device memory for max_bytes bytes of cached pieces (and
 *       as many ids, plus an index); nothing is evicted: once full, new
 *       pieces are merged but not added.  The cache belongs to tok.
 *   tk_workspace_set_cache: encodes on ws look pieces up in cache (before
 *       merging) and add the ones they merged (after); NULL detaches.  Encodes
 *       that share a cache must not overlap in time.
 *   tk_cache_clear: empties it (on cuda_stream).  tk_cache_stats: entries,
 *       bytes and ids held (synchronises the device).
 *   tk_last_cache_stats: pieces the workspace's last encode found in the
 *       cache and added to it.
 */
typedef struct tk_cache tk_cache;
int tk_cache_create(const tk_tokenizer* tok, int64_t max_bytes, tk_cache** out);
void tk_cache_free(tk_cache* cache);
int tk_cache_clear(tk_cache* cache, void* cuda_stream);
int tk_cache_stats(const tk_cache* cache, int64_t* n_entries, int64_t* bytes_used, int64_t* ids_used);
int tk_workspace_set_cache(tk_workspace* ws, tk_cache* cache);
int tk_last_cache_stats(const tk_workspace* ws, int64_t* hits, int64_t* inserts);

/*
 * From device ids to a paged key/value cache.  The encode leaves a batch's
 * ids and their offsets on the device; the three calls below take those
 * offsets on (as they are where a request is one segment; of requests of several,
 * gathered on the device at each one's first): tk_kv_plan places every
 * request's new tokens in the cache's blocks, tk_kv_append stores their keys and
 * values there, tk_kv_attend reads them back for the new tokens, which may be
 * drafted trees.  The pages have no counterpart: these are engineering entry points of this library.
 *
 * All buffers, handles and the stream belong to the current device (a handle is refused
 * where another one is current; of plain pointers the caller has to see to it).
 * The calls only queue work on cuda_stream: none waits for the device, allocates
 * or copies to the host, and all may be captured into a CUDA graph.  What is
 * wrong with the arguments comes back as TK_E_ARG / TK_E_LIMIT; what is wrong
 * with the data is found on the device, never reads or writes outside the
 * buffers, and is reported where each call says.
 */
enum { TK_BF16 = 1, TK_F16 = 2 };

/*
 * tk_kv_plan -- block tables and slot maps from request lengths.
 *
 *   d_off[R+1]: request r's new tokens are d_off[r] .. d_off[r+1) (the encode's
 *       d_out_offsets at the requests' first segments); non-decreasing.  Tokens
 *       before d_off[0] and past d_off[R] are padding: position 0, slot -1, request -1, mask 0.
 *   d_ctx[R]: tokens of r already in the cache.  d_table[R][table_stride]: its
 *       blocks in order, the first ceil(ctx/block_size) of them filled in.
 *   d_free[n_free]: ids of free blocks; d_cursor: the first unused entry (one
 *       int64, e.g. an earlier call's d_info; NULL = 0).
 *   d_parent[T]: NULL, or the tokens are drafted trees: the parent of a token
 *       as an index among its request's new tokens (before the token itself;
 *       any other value = the token continues the context).  At most 64 new
 *       tokens a request then.
 *   block_size: a power of two, 16 to 128.
 *
 * In the order of the requests each takes the free blocks that its new tokens
 * need.  A request is placed if d_ctx[r] >= 0, d_off[r+1] <= T, its blocks fit table_width, a
 * tree holds at most 64 tokens, and the free list reaches; the others get
 * no slots and no blocks (slots -1, their table rows as they were).  d_info tells of them:
 * tk_kv_attend cannot, it takes the last tokens of such a request's context for its new
 * ones, so its rows mean nothing.  R, T < 2^31.
 * Offsets that start below 0 or decrease place nothing: every token counts as
 * padding, d_info[3] is the first such request, with TK_E_LIMIT.
 *
 *   d_table: the new blocks are written behind the filled ones.
 *   d_slot[T]: block * block_size + place in the block of every new token, or
 *       -1.  Token i of a request is stored at ctx + i, drafted or not.
 *   d_pos[T]: ctx + i, for trees ctx + depth (the token's position in its text).
 *   d_req[T]: the token's request.
 *   d_len[R]: tokens in the cache afterwards: ctx + new, or ctx if not placed.
 *   d_mask[T]: with d_parent only: bit j = new token j is the token itself or
 *       above it.
 *   d_info[4]: cursor after the call, free blocks asked for by all requests,
 *       status of the first request not placed (TK_E_LIMIT, TK_E_CAPACITY; 0
 *       if all were), that request (-1).
 *
 * No output overlaps an input (d_len is not d_ctx, d_info not where d_cursor is): TK_E_ARG.
 */
int tk_kv_plan(const int64_t* d_off, const int32_t* d_ctx, int64_t R, int64_t T, int block_size,
               int32_t* d_table, int64_t table_stride, int64_t table_width, const int32_t* d_free,
               int64_t n_free, const int64_t* d_cursor, const int32_t* d_parent, int32_t* d_pos,
               int64_t* d_slot, int32_t* d_req, int32_t* d_len, int64_t* d_mask, int64_t* d_info,
               void* cuda_stream);

/*
 * A paged cache: the caller's memory for n_blocks blocks of block_size tokens,
 * n_heads heads and head_dim elements, keys and values each.
 *
 *   d_k, d_v: element (block b, head h, token s, x) is at b * stride[0] +
 *       h * stride[1] + s * stride[2] + x, in elements (stride NULL = the
 *       packed [n_blocks][n_heads][block_size][head_dim]).  16-byte aligned,
 *       strides multiples of 8 elements.
 *   block_size: a power of two, 16 to 128.  head_dim: a multiple of 16, at
 *       most 256 (tk_kv_attend: 64 or 128).  type: TK_BF16 or TK_F16.
 *
 * At most 1,024 heads.  The handle holds the geometry only and belongs to the
 * current device; one per layer, over one set of block tables.
 */
typedef struct tk_kv_cache tk_kv_cache;
int tk_kv_cache_create(void* d_k, void* d_v, int type, int64_t n_blocks, int n_heads, int block_size,
                       int head_dim, const int64_t* stride, tk_kv_cache** out);
void tk_kv_cache_free(tk_kv_cache* cache);

/*
 * tk_kv_append -- norm of queries and keys for each head, rotation by
 * position, and the store into the cache, in one pass over the projection.
 *
 *   d_qkv[T][row_stride]: a token's n_q_heads query heads, then the cache's
 *       n_heads key heads, then as many value heads (cache type).
 *   d_q_gain, d_k_gain [head_dim] fp32: y = x / sqrt(mean(x^2) + eps) * gain
 *       for each head (NULL = that side has no norm).  Means, norms and
 *       rotations are computed in fp32 and rounded once.  n_q_heads <= 1,024, T <= 2^26.
 *   d_rope[rope_len][rot_dim/2][2] fp32: (cos, sin) of every position, for the
 *       first rot_dim elements of a head (a multiple of 16; NULL with rot_dim
 *       0 = none).  neighbours = 0 turns the pairs (i, i + rot_dim/2), 1 the
 *       pairs (2i, 2i + 1).
 *   d_pos[T] (with d_rope), d_slot[T]: as tk_kv_plan writes them.  A slot that
 *       is negative or past the cache stores nothing.  A position outside
 *       [0, rope_len) gives NaN in the rotated elements.
 *   d_q[T][n_q_heads][head_dim]: the queries, packed.
 */
int tk_kv_append(const tk_kv_cache* cache, const void* d_qkv, int64_t row_stride, int64_t T,
                 int n_q_heads, const float* d_q_gain, const float* d_k_gain, float eps,
                 const float* d_rope, int64_t rope_len, int rot_dim, int neighbours,
                 const int32_t* d_pos, const int64_t* d_slot, void* d_q, void* cuda_stream);

/* Scratch of one tk_kv_attend in flight (about 40 MB, whatever the sizes). */
typedef struct tk_kv_workspace tk_kv_workspace;
int tk_kv_workspace_create(tk_kv_workspace** out);
void tk_kv_workspace_free(tk_kv_workspace* ws);

/*
 * tk_kv_attend -- attention of each request's new tokens over its cache, for
 * drafted trees, single tokens and chunks of a prompt.
 *
 *   d_q[T]: head h of token t is at t * q_stride + h * head_dim (the cache's type,
 *       16-byte aligned, q_stride a multiple of 8); n_q_heads is a multiple of
 *       the cache's n_heads, and query head h reads the cache's head
 *       h / (n_q_heads / n_heads).
 *   d_off[R+1], d_len[R], d_table: as tk_kv_plan has them; d_len counts the
 *       new tokens, which are stored already.
 *   max_new: no request has more new tokens than this (T always holds, but the rows of a
 *       request and key head choose the kernel: one token of 64 requests over 1k, 4 query heads a
 *       key head, takes 56 us with max_new = 1 and 73 with T).
 *   d_mask[T]: NULL = new token i sees the context and the new tokens up to
 *       itself.  Else it sees the context and those new tokens j whose bit j
 *       is set, itself included only if its own bit is (requests of at most
 *       64 new tokens).
 *   scale: the factor on q.k before the softmax, above 0 and below 1e38.
 *   d_out[T][n_q_heads][head_dim] (the cache's type), d_lse[T][n_q_heads]
 *       (fp32, NULL = not wanted): the natural log of the row's sum of
 *       exponentials.  A row that sees nothing gives 0 and -infinity.
 *       Scores, softmax and sums are fp32; the weights are rounded to the
 *       cache's type for the product with the values (fp16: a weight below
 *       about 2^-32 of the row's largest counts as 0).  Tokens that the mask
 *       hides, and cache places past d_len, have no influence, whatever they hold.
 *
 * R <= 2^20, T <= 2^26, T * n_q_heads < 2^31.  The launch is cooperative (one CTA
 * for each SM); a call uses the workspace until it ends, so calls in flight at
 * the same time need one each.
 *
 * Found on the device: a request with more than max_new new tokens, with more
 * than 64 under a mask, with d_len below its new tokens, or past table_width
 * blocks, or with offsets outside [0, T].  Its rows are 0 (lse -infinity), and
 * tk_kv_status tells of it.  A block id outside the cache reads as zeros.  Tokens of no
 * request (before d_off[0], from d_off[R] on) give 0 and -infinity.
 * A call whose offsets decrease gives them for every token, and so may one of too much
 * work: 2^30 tiles of keys or more, over all key heads and tiles of query rows, three
 * tiles more for each of these (64 keys and 32 or 128 rows a tile; 128 and 256 from
 * 129 rows a key head on; from 2^31 on it always does).
 * tk_kv_status waits for cuda_stream and gives what the workspace's calls
 * since the last tk_kv_status met first (a timeout before others): TK_OK,
 * TK_E_LIMIT (h_request: the request; -1 if nothing was done) or TK_E_TIMEOUT (a wait
 * on the device gave up, never expected; the outputs are unspecified).
 */
int tk_kv_attend(const tk_kv_cache* cache, tk_kv_workspace* ws, const void* d_q, int64_t q_stride,
                 int n_q_heads, const int64_t* d_off, int64_t R, int64_t T, int64_t max_new,
                 const int32_t* d_len, const int32_t* d_table, int64_t table_stride,
                 int64_t table_width, const int64_t* d_mask, float scale, void* d_out, float* d_lse,
                 void* cuda_stream);
int tk_kv_status(tk_kv_workspace* ws, int64_t* h_request, void* cuda_stream);

/*
 * Per-kernel timing of encodes on a workspace, for benchmarks.  With
 * profiling on, every kernel launch of tk_encode_segments /
 * tk_encode_segments_host / tk_decode is bracketed by CUDA events recorded on
 * the call's own stream; after each call the elapsed times are added to
 * per-kernel totals.  tk_profile_enable(ws, 1) turns it on and clears the
 * totals; 0 turns it off.  tk_profile_read copies up to max entries (kernel
 * name, total milliseconds, number of launches) and returns how many kernels
 * have entries.  Names are static strings owned by the library.
 */
int tk_profile_enable(tk_workspace* ws, int on);
int tk_profile_read(const tk_workspace* ws, int max, const char** names, double* total_ms,
                    int64_t* launches);

/*
 * Counts of the last completed tk_encode_segments(_host) call on a workspace
 * (host copies, no device access): pre-tokens found by the split, ids
 * produced, and pre-tokens that took the long-piece merge.  Any pointer may be
 * NULL.
 */
int tk_last_stats(const tk_workspace* ws, int64_t* n_pretokens, int64_t* n_ids, int64_t* n_long);

/* Number of mergeable ranks, specials, and the largest id of a tokenizer. */
int64_t tk_n_ranks(const tk_tokenizer* tok);
int64_t tk_n_specials(const tk_tokenizer* tok);
int64_t tk_max_id(const tk_tokenizer* tok);

/* Static description of a status code, and the calling thread's last error. */
const char* tk_status_string(int code);
const char* tk_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* TK_H */
