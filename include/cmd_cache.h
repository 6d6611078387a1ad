/*
 * cmd_cache.h - a paged key-value cache and the operators of a serving step
 * on it, on one GPU (GB300, sm_103a): C ABI, in the same library as cmd.h.
 *
 * A Command runs elementwise ops over views whose addresses are sums of
 * index * stride. Next to it, a program that generates text needs addresses
 * that go through a table, sums over a sequence, and angles of positions:
 *
 *   cmd_rope              rotary positions of queries and keys, and their
 *                         gradient (training);
 *   cmd_cache_append      new tokens' keys (rotated) and values into the cache;
 *   cmd_attention_decode  attention of one new token per sequence;
 *   cmd_cache_select      which sequences go on: fork, free, grow, in one step;
 *   cmd_cache_compact     the pages in use moved to the front of the pool;
 *
 * where it drafts several tokens ahead and has them checked in one pass:
 *
 *   cmd_attention_drafts  attention of a tree of drafted tokens per sequence,
 *                         and the weight that each cached token gets;
 *   cmd_draft_path        the branch that agrees with the model's choices;
 *   cmd_cache_accept      that branch's tokens moved together, the rest dropped;
 *
 * and where the cache has a budget:
 *
 *   cmd_cache_evict       the tokens of the least weight dropped, those kept
 *                         moved together.
 *
 * The cache. Two pools of pages, keys and values, each a tensor of logical
 * sizes [pages, page_size, kv_heads, dim] and any strides with a unit stride
 * along dim (slots outermost in a page, heads outermost, or interleaved with
 * another tensor). A sequence is a row of a page table, i32 [rows, columns]:
 * entry j is the page that holds its tokens j * page_size and on. Entries
 * past the sequence's length are never read. A length is 0 to columns *
 * page_size: one outside is reported and held to that range. A page that
 * several rows list is shared; refs, i32 [pages], counts how many hold it, and
 * a count of zero makes a page free. Tables, lengths and counts live on the
 * device and every operator works on them there, so a whole generation step can
 * be captured in a CUDA graph.
 *
 * Tensors are given as cmd_operand (a pointer the GPU can address, sizes and
 * element strides >= 0). Outputs must address distinct elements and must not
 * overlap an input, except where "in place" is allowed. Element types are
 * CMD_F32, CMD_F16 and CMD_BF16 for numbers (one type within a call; all
 * arithmetic is in 32 bits, rounded once to the output's type, but for the
 * softmax weights of 16-bit caches, see the attention) and CMD_I32 for tables,
 * lengths, positions and counts.
 *
 * Every launch is asynchronous on cuda_stream (NULL = the legacy default
 * stream), on the current device, allocates nothing, may be captured, and
 * returns a cmd_status (cmd_last_error() explains it) for what the host can
 * see. What only the device can see (a page number outside the pool, a table
 * that is full, a pool with no free page) the kernels check themselves: they
 * access nothing out of bounds, and set bits in the i32 word that `status`
 * points to (NULL: not reported), read with cmd_cache_status.
 */
#ifndef CMD_CACHE_H
#define CMD_CACHE_H

#include "cmd.h"

#ifdef __cplusplus
extern "C" {
#endif

#define CMD_CACHE_MAX_DIM 256  /* head dim of the attention and the rotation */
#define CMD_CACHE_MAX_POOLS 64 /* pools of one select, compact or accept call */
#define CMD_CACHE_MAX_LAYERS 32 /* layers of one evict call */
#define CMD_CACHE_MAX_DRAFTS 256 /* drafted tokens of a sequence */

/* Bits of the device status word. */
#define CMD_CACHE_BAD_PAGE 1  /* a table entry names no page of the pool; its tokens were skipped */
#define CMD_CACHE_BAD_INDEX 2 /* a row, parent or position outside its range, skipped; a length, held to its range */
#define CMD_CACHE_FULL_TABLE 4 /* a row would need more columns than its table has; dropped */
#define CMD_CACHE_NO_PAGES 8  /* the pool had no free page left for a row; dropped */
#define CMD_CACHE_SHARED_PAGE 16 /* tokens would move into a page that others hold too; left as they are */
#define CMD_CACHE_TIMEOUT 32 /* a kernel's wait took too long (never expected): its outputs are not valid, and NaN where it gave up */

typedef struct cmd_operand {
  void* ptr; /* NULL: absent, where an operand is optional */
  int32_t dtype; /* cmd_dtype */
  int32_t rank;
  int64_t sizes[CMD_MAX_RANK];
  int64_t strides[CMD_MAX_RANK]; /* in elements */
} cmd_operand;

/* ---- rotary positions ---------------------------------------------------- */

typedef enum cmd_rope_layout {
  CMD_ROPE_HALF = 0,        /* pair i of a head is elements (i, i + n_pairs) */
  CMD_ROPE_INTERLEAVED = 1  /* ... elements (2 i, 2 i + 1) */
} cmd_rope_layout;

/* The rotation of a head: pair i of its first 2 * n_pairs elements, (a, b),
 * becomes scale * (a cos t - b sin t, b cos t + a sin t), with the angle t of
 * position p being p * turns[i] / 2^64 of a full turn. The product is taken
 * modulo 2^64, which drops whole turns exactly, so that an angle is as good
 * at position 10^6 as at position 1. Elements past the first 2 * n_pairs are
 * copied. turns: n_pairs 64-bit words in device memory, 8-byte aligned. */
typedef struct cmd_rope_spec {
  const uint64_t* turns;
  int32_t n_pairs;  /* 0: no rotation, a copy (cmd_cache_append: without q) */
  int32_t layout;   /* cmd_rope_layout */
  float scale;
  int32_t backward; /* 1: turn by -t, the gradient of the same call with 0 */
} cmd_rope_spec;

typedef enum cmd_rope_scaling {
  CMD_ROPE_SCALING_NONE = 0,
  CMD_ROPE_SCALING_LINEAR = 1, /* every frequency divided by factor */
  CMD_ROPE_SCALING_BASE = 2,   /* base * factor^(d / (d - 2)), d = 2 n_pairs: the slowest frequency is divided by factor,
                                  the fastest kept */
  CMD_ROPE_SCALING_PARTS = 3   /* pairs that make at least beta_fast turns over original_length kept, those that make
                                  at most beta_slow divided by factor, a linear ramp over the pair's index between: from
                                  the index that makes beta_fast, rounded down and at least 0, to that which makes
                                  beta_slow, rounded up and at most 2 n_pairs - 1 (the last pair's is n_pairs - 1) */
} cmd_rope_scaling;

/* turns[i] = 2^64 * base^(-i / n_pairs) / (2 pi), scaled as `scaling` says, rounded to an integer, for i < n_pairs;
 * turns is host memory. factor >= 1; original_length, beta_fast > beta_slow > 0 are read by CMD_ROPE_SCALING_PARTS
 * only. base > 1 (>= 1 for n_pairs = 1, but by parts). Host only. */
cmd_status cmd_rope_turns(int32_t n_pairs, double base, int32_t scaling, double factor, double original_length,
                          double beta_fast, double beta_slow, uint64_t* turns);

/* Rotate q and k (either may be absent: NULL operands) into q_out and k_out.
 * Operands have rank 3 [tokens, heads, dim] or 4 [batch, tokens, heads, dim],
 * unit stride along dim, dim <= CMD_CACHE_MAX_DIM; q and k agree in dtype, rank, batch,
 * tokens and dim and may differ in heads. Inputs may be broadcast (stride 0).
 * An output may be the identical view of its input (in place). positions: i32
 * [tokens] or [batch, tokens] (rank one or two less than q's... its leading
 * dims), any strides, any sign. */
cmd_status cmd_rope(const cmd_operand* q, const cmd_operand* q_out, const cmd_operand* k, const cmd_operand* k_out,
                    const cmd_operand* positions, const cmd_rope_spec* rope, void* cuda_stream);

/* ---- append ----------------------------------------------------------------- */

/* Store each token's key (rotated by its position) and value at slot
 * position % page_size of page tables[row][position / page_size]. A token with
 * a negative position is padding: it is not stored. No two tokens of a call
 * may name the same slot of the same page. */
typedef struct cmd_append_args {
  cmd_operand k, v;             /* [tokens, kv_heads, dim] */
  cmd_operand k_cache, v_cache; /* [pages, page_size, kv_heads, dim]; written */
  cmd_operand tables;           /* i32 [rows, columns] */
  cmd_operand positions;        /* i32 [tokens] */
  cmd_operand rows;             /* i32 [tokens]: each token's table row; absent: token t has row t */
  cmd_operand q, q_out;         /* optional: [tokens, q_heads, dim], rotated by the same positions (in place allowed) */
  cmd_rope_spec rope;           /* n_pairs 0: keys stored as they are (q must be absent) */
  int32_t* status;
} cmd_append_args;

cmd_status cmd_cache_append(const cmd_append_args* args, void* cuda_stream);

/* ---- attention of one new token per sequence ---------------------------------- */

/* For row r and query head h (which reads kv head h / (q_heads / kv_heads)),
 * over the tokens t of the row with max(0, n - window) <= t < n, n = lengths[r]
 * (window 0: all of them), s_t = scale * dot(q, k_t), or softcap * tanh(that /
 * softcap) where softcap > 0:
 *   out = sum_t exp(s_t - lse) v_t,   lse = log sum_t exp(s_t).
 * A row with no token, or whose scores are all -infinity, gives out = 0 and
 * lse = -infinity. Nothing outside those tokens enters, whatever the pages
 * hold there (infinities and NaN included).
 *
 * The work is split over the sequences' lengths in equal parts and joined
 * through workspace: cmd_attention_workspace bytes of device memory, 16-byte
 * aligned, of any contents, apart from all else of the call, used by one call at
 * a time (streams that overlap need one each). Results do not depend on the
 * timing of the parts. columns * page_size * kv_heads stays below 2^35.
 *
 * The weights of 16-bit caches are multiplied with the values as the sum of two
 * 16-bit numbers each: to 2^-16 of itself in bf16 and 2^-22 in f16 (there no
 * finer than 2^-40 of the largest weight); their sum, lse and everything else
 * are in 32 bits. A 16-bit value of infinity inside a row makes its element of
 * out NaN or infinite. */
typedef struct cmd_attention_args {
  cmd_operand q, out;           /* [rows, q_heads, dim], dim <= CMD_CACHE_MAX_DIM */
  cmd_operand lse;              /* optional: f32 [rows, q_heads] */
  cmd_operand k_cache, v_cache; /* [pages, page_size, kv_heads, dim]; kv_heads divides q_heads */
  cmd_operand tables;           /* i32 [rows, columns] */
  cmd_operand lengths;          /* i32 [rows] */
  float scale;                  /* > 0 */
  float softcap;                /* 0: none */
  int32_t window;               /* 0: none */
  int32_t reserved;             /* 0 */
  void* workspace;
  int64_t workspace_bytes;
  int32_t* status;
} cmd_attention_args;

/* Workspace bytes for any call with at most q_heads / kv_heads query heads to a kv head and at most this dim (whatever
 * the number of heads, rows and lengths). */
cmd_status cmd_attention_workspace(int32_t q_heads, int32_t kv_heads, int32_t dim, int64_t* bytes);
cmd_status cmd_attention_decode(const cmd_attention_args* args, void* cuda_stream);

/* ---- attention of drafted tokens -------------------------------------------------- */

/* The last `drafts` tokens of row r's lengths[r] are guesses, stored in the
 * cache behind the others in any order that puts a guess behind the one that it
 * goes on from. parents[r][i] is the draft that draft i goes on from, below i;
 * -1: the tokens before the drafts; less: draft i is padding. (So is one whose
 * parent is; a parent of i or above is reported, and its draft padding.) Draft i
 * sees the lengths[r] - drafts tokens before the drafts, its ancestors and
 * itself, and with a window those at most window - 1 positions back, where a
 * draft's position is lengths[r] - drafts + its number of ancestors. Over them,
 * scores, out and lse are as in cmd_attention_decode, which this is for one
 * draft. Nothing that a draft does not see enters its output. Padding, and rows
 * of length 0, give out = 0 and lse = -infinity; so do rows whose length is
 * negative or below `drafts` (reported).
 *
 * weights, where given, gets the attention that each token of each row received:
 *   weights[r][h][t] += sum over the drafts and the query heads that read kv
 *                       head h of exp(s_t - lse),
 * for the tokens t < lengths[r] that are seen, in 32 bits, in an order that does
 * not depend on timing. It reaches at least columns * page_size tokens.
 *
 * The softmax weights of 16-bit caches are held as there, in f16 no finer than
 * 2^-36 of the largest. workspace as there, of cmd_drafts_workspace bytes. Limits:
 * drafts <= CMD_CACHE_MAX_DRAFTS, drafts * q_heads <= 2^20. */
typedef struct cmd_drafts_args {
  cmd_operand q, out;           /* [rows, drafts, q_heads, dim], dim <= CMD_CACHE_MAX_DIM */
  cmd_operand lse;              /* optional: f32 [rows, drafts, q_heads] */
  cmd_operand k_cache, v_cache; /* [pages, page_size, kv_heads, dim]; kv_heads divides q_heads */
  cmd_operand tables;           /* i32 [rows, columns] */
  cmd_operand lengths;          /* i32 [rows], drafts included */
  cmd_operand parents;          /* i32 [rows, drafts]; absent: each goes on from the one before */
  cmd_operand weights;          /* optional: f32 [rows, kv_heads, tokens], unit stride along tokens; added to */
  float scale;                  /* > 0 */
  float softcap;                /* 0: none */
  int32_t window;               /* 0: none */
  int32_t reserved;             /* 0 */
  void* workspace;
  int64_t workspace_bytes;
  int32_t* status;
} cmd_drafts_args;

/* Workspace bytes for a call of as many drafts with at most these rows and query heads, q_heads / kv_heads of them to a
 * kv head, this dim and these tokens: columns * page_size where weights are given, else 0. (For one draft with weights
 * that is up to a GiB, which its scores are kept in: 4 bytes for each query head, token and row.) */
cmd_status cmd_drafts_workspace(int64_t rows, int32_t drafts, int32_t q_heads, int32_t kv_heads, int32_t dim, int64_t tokens,
                                int64_t* bytes);
/* ... for this very call, whose arguments are checked but for the workspace: no more than the above, and without room for
 * scores where none are kept (32-bit caches, rows that are no whole 16-byte vectors, scores of more than a GiB). Host only. */
cmd_status cmd_attention_drafts_workspace(const cmd_drafts_args* args, int64_t* bytes);
cmd_status cmd_attention_drafts(const cmd_drafts_args* args, void* cuda_stream);

/* ---- the accepted branch -------------------------------------------------------- */

/* Walks each row's tree (parents as above) along the model's choices: from draft
 * 0 (the model's own last choice, say, which needs no check) to the first draft
 * that goes on from it and whose token is choices[r][0], what the model chooses
 * after draft 0, and so on. path[r] lists the drafts passed, ascending, then -1;
 * counts[r] says how many they are, and last[r] what the model chooses after the
 * last of them. Where draft 0 is no root (parents[r][0] is not -1) nothing is
 * passed: counts 0, last -1. All i32. */
typedef struct cmd_path_args {
  cmd_operand tokens, choices; /* [rows, drafts] */
  cmd_operand parents;         /* [rows, drafts]; absent: each goes on from the one before */
  cmd_operand path;            /* [rows, drafts] */
  cmd_operand counts, last;    /* [rows] */
  int32_t* status;
} cmd_path_args;

cmd_status cmd_draft_path(const cmd_path_args* args, void* cuda_stream);

/* Of row r's last `drafts` tokens, keeps those listed in the first counts[r]
 * entries of path[r] (ascending, each below `drafts`): in every pool the j-th one
 * moves from its slot to slot lengths[r] - drafts + j, and lengths_out[r] =
 * lengths[r] - drafts + counts[r]. Pages past that are released (refs_out). Rows
 * of length 0 stay as they are. (Of a length beyond the table, which is held to it
 * and reported, the drafts are the table's last tokens.) A row whose list is not
 * as above, or whose moves would meet pages that do not exist or write to one
 * that others hold too (refs above 1), keeps none of its drafts (reported); one
 * shorter than `drafts` stays as it is (reported). Pools as tensors, since parts
 * of a page move; the same sizes and element type in all of them; a model with
 * more makes a call for each CMD_CACHE_MAX_POOLS, with the same inputs. */
typedef struct cmd_accept_args {
  cmd_operand tables;       /* i32 [rows, columns], each row dense */
  cmd_operand lengths;      /* i32 [rows], drafts included; dense (as all vectors here) */
  cmd_operand refs;         /* i32 [pages] */
  cmd_operand path;         /* i32 [rows, drafts], each row dense */
  cmd_operand counts;       /* i32 [rows] */
  cmd_operand lengths_out;  /* i32 [rows] */
  cmd_operand refs_out;     /* i32 [pages] */
  const cmd_operand* pools; /* n_pools of [pages, page_size, kv_heads, dim] (host array, read during the call) */
  int32_t n_pools;          /* at least 1 */
  int32_t reserved;         /* 0 */
  int32_t* status;
} cmd_accept_args;

cmd_status cmd_cache_accept(const cmd_accept_args* args, void* cuda_stream);

/* ---- eviction --------------------------------------------------------------------- */

/* Holds rows to a budget: of a row of n > budget tokens, each kv head of each
 * layer keeps the last `recent` tokens and, of those before, the budget - recent
 * of the largest weights (of equal ones the earliest; NaN counts as less than any
 * number). They move to the row's first `budget` slots in their order, keys,
 * values and weights; the weights past them, up to n, become 0. lengths_out[r] =
 * budget, and pages past it are released (refs_out). Rows of at most budget
 * tokens stay as they are; so does a row whose length is beyond its table, where
 * a page does not exist, or one of those that it goes on with is held by others
 * too (refs above 1) (reported; lengths_out is then the length, held to the table).
 * Positions are no longer slots then: keys keep the rotation they were stored
 * with. All layers have the same sizes and element type; a model with more than
 * CMD_CACHE_MAX_LAYERS makes a call for each so many, with the same inputs.
 * workspace: cmd_evict_workspace bytes, 16-byte aligned, of any contents. */
typedef struct cmd_evict_args {
  cmd_operand tables;                    /* i32 [rows, columns], each row dense */
  cmd_operand lengths;                   /* i32 [rows], dense (as all vectors here) */
  cmd_operand refs;                      /* i32 [pages] */
  cmd_operand lengths_out;               /* i32 [rows] */
  cmd_operand refs_out;                  /* i32 [pages] */
  const cmd_operand *k_caches, *v_caches; /* n_layers of [pages, page_size, kv_heads, dim] (host arrays, as the next) */
  const cmd_operand* weights;            /* n_layers of f32 [rows, kv_heads, tokens], unit stride along tokens; tokens >=
                                            columns * page_size */
  int32_t n_layers;                      /* at least 1 */
  int32_t budget;                        /* >= recent */
  int32_t recent;                        /* >= 0 */
  int32_t reserved;                      /* 0 */
  void* workspace;
  int64_t workspace_bytes;
  int32_t* status;
} cmd_evict_args;

/* For a call with at most these rows, layers, heads and budget (or columns * page_size, where that is less). */
cmd_status cmd_evict_workspace(int64_t rows, int32_t layers, int32_t kv_heads, int32_t budget, int64_t* bytes);
cmd_status cmd_cache_evict(const cmd_evict_args* args, void* cuda_stream);

/* ---- pages ---------------------------------------------------------------------- */

/* Rows and pages of a select or compact call number at most 2^30 each.
 *
 * The pools of a call: each as many pages of page_bytes bytes, page_stride bytes
 * apart (>= page_bytes), the bytes of a page dense. A model with more than
 * CMD_CACHE_MAX_POOLS of them makes a call for each so many, all with the same
 * inputs: every call writes the same tables, lengths and counts. */
typedef struct cmd_pool {
  void* ptr;
  int64_t page_bytes;
  int64_t page_stride;
} cmd_pool;

/* New row i goes on from old row parents[i], with room for grow[i] more
 * tokens; parents[i] = -1 starts an empty row. An old row that no new row
 * names is freed; one that several name is forked. In the order of i:
 *   - whole pages of the parent are shared by all of its children;
 *   - the page in progress (length % page_size != 0) stays with the first
 *     child whose table has room, and every other child gets a copy in a page
 *     of its own;
 *   - pages for the tokens to come are added up to length + grow[i].
 * New pages are the free ones in ascending order, dealt out in the order of i,
 * where a page is free when nothing holds it once the old rows are gone and the
 * new ones (those that will get none too) hold what they share. Then lengths_out[i] = length + grow[i]; table
 * entries past it are -1. A row whose table is too short for it is dropped:
 * length 0, no pages (status bit FULL_TABLE). So is a row whose new pages would
 * lie past the last free one (NO_PAGES). It keeps its place in the order: rows
 * after it get the pages after those that it asked for, so that every later row
 * that needs a new page is dropped too, and those that need none go on. (The old
 * tables, lengths and counts are as they were: a caller may free rows and select
 * anew from them.) Counts may include holders outside the tables.
 * workspace: cmd_select_workspace bytes, 16-byte aligned, of any contents. */
typedef struct cmd_select_args {
  cmd_operand tables;      /* i32 [old_rows, columns], each row dense */
  cmd_operand lengths;     /* i32 [old_rows], dense (as all vectors here) */
  cmd_operand refs;        /* i32 [pages] */
  cmd_operand parents;     /* i32 [new_rows] */
  cmd_operand grow;        /* optional: i32 [new_rows], >= 0 */
  cmd_operand tables_out;  /* i32 [new_rows, columns] */
  cmd_operand lengths_out; /* i32 [new_rows] */
  cmd_operand refs_out;    /* i32 [pages] */
  const cmd_pool* pools;   /* n_pools pools of `pages` pages each (host array, read during the call) */
  int32_t n_pools;
  int32_t page_size;
  void* workspace;
  int64_t workspace_bytes;
  int32_t* status;
} cmd_select_args;

cmd_status cmd_select_workspace(int64_t old_rows, int64_t new_rows, int64_t pages, int64_t* bytes);
cmd_status cmd_cache_select(const cmd_select_args* args, void* cuda_stream);

/* Move the pages in use to the front: with n pages in use, the k-th used page
 * at or past index n moves to the k-th free page before it. page_map_out[p] is
 * page p's new number (-1: free); tables and counts are rewritten to it,
 * table entries past a row's length to -1. Afterwards pages n and on are free.
 * workspace: cmd_compact_workspace bytes, 16-byte aligned, of any contents. */
typedef struct cmd_compact_args {
  cmd_operand tables;       /* i32 [rows, columns], each row dense */
  cmd_operand lengths;      /* i32 [rows] */
  cmd_operand refs;         /* i32 [pages] */
  cmd_operand tables_out;   /* i32 [rows, columns] */
  cmd_operand refs_out;     /* i32 [pages] */
  cmd_operand page_map_out; /* i32 [pages] */
  const cmd_pool* pools;
  int32_t n_pools;
  int32_t page_size;
  void* workspace;
  int64_t workspace_bytes;
  int32_t* status;
} cmd_compact_args;

cmd_status cmd_compact_workspace(int64_t pages, int64_t* bytes);
cmd_status cmd_cache_compact(const cmd_compact_args* args, void* cuda_stream);

/* Wait for cuda_stream, read the status word and clear the bits that it held:
 * CMD_OK for 0, else CMD_ERR_DEVICE_TIMEOUT for TIMEOUT, CMD_ERR_ARG for BAD_PAGE or BAD_INDEX, CMD_ERR_LIMIT for
 * FULL_TABLE or NO_PAGES and CMD_ERR_ALIAS for SHARED_PAGE (the first that holds), with the bits in *bits (when non-NULL) and a message. A word may
 * serve several streams: bits that work on another one sets meanwhile stay for
 * the next call. */
cmd_status cmd_cache_status(int32_t* status, int32_t* bits, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* CMD_CACHE_H */
