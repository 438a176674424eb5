/*
 * spec_verify_target.h -- C ABI of the operators around one verification call.
 *
 * A round of the target model runs its new tokens (the draft, or a chunk of a
 * prompt) over the sequences' cached keys and values, and its logits are adjusted
 * before spec_verify reads them:
 *   spec_verify_rotate_append    rotary positions on q and k; k and v go to their pages
 *   spec_verify_attention        the new tokens' attention over the paged cache
 *   spec_verify_process_logits   penalties for repeated tokens, biases, grammar masks
 *   spec_verify_history_add      keeps the tokens that the penalties count
 *
 * Conventions are those of spec_verify.h: device pointers, asynchronous on
 * `stream`, nothing allocated and nothing kept, argument errors returned before
 * anything is enqueued.  Arguments come in structures of 8-byte fields; set
 * struct_size = sizeof(structure).  Strides count elements; the innermost
 * dimension is contiguous.  row_status [B] may be NULL; the calls OR their bits
 * into it (they never clear it), so that one array can collect a round's problems.
 * A sequence with a bit set gets NaN outputs instead of results (see each call); it
 * never makes a call read or write out of range.
 */
#ifndef SPEC_VERIFY_TARGET_H
#define SPEC_VERIFY_TARGET_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* a third element type, for q, k, v and the cache (16-bit only there) */
#define SV_F16 2

#define SV_ROW_BAD_PENALTY 0x100u /* repetition not finite or <= 0; frequency or presence not finite */
#define SV_ROW_BAD_SLOT 0x200u    /* history slot outside [0, slots) */
#define SV_ROW_BAD_LENGTH 0x400u  /* num_new outside [0, N], cache_lens < 0, or past the page or rotary table */
#define SV_ROW_BAD_PAGE 0x800u    /* a page id in use is outside [0, pages) */

#define SV_MAX_POSITIONS (SV_MAX_GAMMA + 1) /* logit rows per sequence */
#define SV_MAX_HEAD_DIM 256                 /* spec_verify_rotate_append */
#define SV_MAX_GROUP 64                     /* query heads per cache head */

/*
 * Token history.  Per slot (a sequence's place in the server): seen [slots, words], a
 * bit plane, token t at bit t & 31 of word t >> 5, words >= ceil(V / 32) (bits from V on
 * are ignored); counts [slots, V].  A token of the prompt or the output sets its bit; one of the output
 * adds 1 to its count.
 *
 * tokens [B, L] (row stride tokens_stride); of row b the first prompt_lens[b]
 * (NULL: none) belong to the prompt, those from there to total_lens[b] (NULL: L)
 * to the output; lengths are clamped to [0, L].  Ids outside [0, V) are skipped,
 * so spec_verify's out_tokens (padded with -1) can be added as they are.
 * slot_of [B] (NULL: row b is slot b); rows whose slot is outside [0, slots) are
 * skipped.  clear != 0 empties the rows' slots first.
 */
typedef struct {
    uint64_t struct_size;
    uint32_t* seen;
    int32_t* counts;
    int64_t slots, words, V;
    const int32_t* slot_of;
    const int32_t* tokens;
    int64_t B, L, tokens_stride;
    const int32_t* prompt_lens;
    const int32_t* total_lens;
    int64_t clear;
} sv_history_args;

int spec_verify_history_add(const sv_history_args* args, void* stream);

/*
 * Adjusts logits [B, N, V] (SV_F32 or SV_BF16) before they are verified.  Row i of
 * sequence b follows the sequence's history and the draft tokens x_1..x_i:
 *   n(t)  = count of t in the output, plus its occurrences in x_1..x_i
 *   seen  = t in the prompt, or n(t) > 0
 *   z     = seen ? (z > 0 ? z / repetition_b : z * repetition_b) : z
 *   z     = z - frequency_b * n(t) - presence_b * [n(t) > 0]
 *   z     = z + sum of the sequence's biases for t
 *   z     = -inf where the mask's bit of t is 0
 * in 32 bits, rounded once to the logits' type.  The same call serves the target's
 * gamma+1 rows and the drafter's rows (N = 1: the plain decoding step).
 *
 * logits, out      may be the same memory (an element is read and written by one block
 *                  alone, with a barrier between its copy and a second look);
 *                  otherwise they must not overlap
 * seen .. slot_of  the history, as above; seen = NULL: no history
 * draft_tokens     [B, draft_len] or NULL; ids outside [0, V) are skipped
 * repetition, frequency, presence  [B] float or NULL (1, 0, 0)
 * bias_*           ids [bias_total], values [bias_total], offsets [B+1] into them
 *                  (clamped to [0, bias_total]), or NULL; repeated ids add up in
 *                  order; ids outside [0, V) are skipped
 * mask             bit planes as in the history, 1 = allowed, or NULL;
 *                  mask_stride_n = 0: one mask per sequence.  Rows of at least
 *                  ceil(V / 32) words; masked logits are not read
 * A sequence with a bad penalty or slot gets NaN rows.
 */
typedef struct {
    uint64_t struct_size;
    const void* logits;
    void* out;
    int64_t dtype, B, N, V;
    int64_t logits_stride_b, logits_stride_n, out_stride_b, out_stride_n;
    const uint32_t* seen;
    const int32_t* counts;
    int64_t slots, words;
    const int32_t* slot_of;
    const int32_t* draft_tokens;
    int64_t draft_stride, draft_len;
    const float* repetition;
    const float* frequency;
    const float* presence;
    const int32_t* bias_ids;
    const float* bias_values;
    const int32_t* bias_offsets;
    int64_t bias_total;
    const uint32_t* mask;
    int64_t mask_stride_b, mask_stride_n;
    uint32_t* row_status;
} sv_logits_args;

int spec_verify_process_logits(const sv_logits_args* args, void* stream);

/*
 * The paged cache of the two calls below.  Key of position j of sequence b, head h:
 *   k_pages + page * stride_page + h * stride_head + (j % page_size) * stride_slot,
 *   page = page_table[b * page_table_stride + j / page_size],
 * `dim` contiguous elements, and the same for v.  page_size is a multiple of 16;
 * all strides and base addresses are multiples of 16 bytes.  cache_lens[b] tokens
 * are in the cache before the call; new token i of sequence b has position
 * cache_lens[b] + i, for i < num_new[b] (NULL: N).
 */
typedef struct {
    void* k_pages;
    void* v_pages;
    int64_t pages, page_size;
    int64_t k_stride_page, k_stride_head, k_stride_slot;
    int64_t v_stride_page, v_stride_head, v_stride_slot;
    const int32_t* page_table;
    int64_t page_table_stride, pages_per_seq;
    const int32_t* cache_lens;
    const int32_t* num_new;
} sv_paged_cache;

/*
 * Rotates q and k by their positions and writes k and v to the cache.
 * q [B, N, q_heads, dim], k, v [B, N, kv_heads, dim] (SV_BF16 or SV_F16; dim a
 * multiple of 16, at most SV_MAX_HEAD_DIM).  The first rot_dim elements of a head
 * (a multiple of 16) are rotated in pairs: (j, j + rot_dim/2), or with interleaved
 * != 0 (2j, 2j + 1); pair j of position p by the angle whose cosine and sine are
 * table[p][0][j] and table[p][1][j] (float, [table_len, 2, rot_dim/2], 16-byte
 * aligned; any scaling of the positions is in the table):
 *   (a, b) -> (a cos - b sin, b cos + a sin)
 * q_out may be q.  Rows past num_new[b] of q_out are zeros; a sequence with bad
 * lengths gets NaN rows and writes nothing to the cache; a token whose page id is bad
 * is not written to the cache.
 */
typedef struct {
    uint64_t struct_size;
    const void* q;
    void* q_out;
    const void* k;
    const void* v;
    int64_t dtype, B, N, q_heads, kv_heads, dim;
    int64_t q_stride_b, q_stride_n, q_stride_h;
    int64_t o_stride_b, o_stride_n, o_stride_h;
    int64_t k_stride_b, k_stride_n, k_stride_h;
    int64_t v_stride_b, v_stride_n, v_stride_h;
    const float* table;
    int64_t table_len, rot_dim, interleaved;
    sv_paged_cache cache;
    uint32_t* row_status;
} sv_rotate_args;

int spec_verify_rotate_append(const sv_rotate_args* args, void* stream);

/*
 * Attention of the new tokens over the cache that holds them too:
 *   out[b, i, h] = sum_j softmax_j(scale * q[b, i, h] . k_j) v_j,
 * j over the positions of cache head h / (q_heads / kv_heads) with
 * j <= cache_lens[b] + i and, for window > 0, j > cache_lens[b] + i - window.
 * q, out [B, N, q_heads, dim], SV_BF16 or SV_F16 as the cache; dim 64 or 128.
 * scale is positive and finite.  Scores, the softmax and the sums are held in 32 bits;
 * its weights enter the product with v in the cache's 16-bit type (fp16: those below
 * 2^-21 of the row's largest with a fixed step of 2^-31 of it).  Rows past num_new[b]
 * are zeros.  What the cache holds at positions that no new token sees may be anything
 * (NaN among it).  A NaN or infinity among the keys reaches the tokens that see its
 * position; among the values, where some of the new tokens see its position, it may
 * reach the others of the sequence as well, as 0 times it.
 * max_context: an upper bound of cache_lens + num_new known to the host, or 0 (the
 * page table's width); it only sizes the launch.
 * workspace: spec_verify_attention_workspace_size() bytes, 256-byte aligned, needs
 * no initialisation; calls on one workspace must not overlap.  A call enqueues two
 * kernels that hand over through it: threads that share a workspace (and a stream) must
 * not be in this function at the same time.
 * wait_limit_ns: limit of a device-side wait (0: 2 s); a call in which one runs
 * out sets SV_ROW_INTERNAL and gives NaN for the rows concerned.
 * A sequence with bad lengths gets NaN rows; so do the rows of a tile that meets a bad
 * page id (the sequence's status has SV_ROW_BAD_PAGE, and none of its rows is to be used).
 */
typedef struct {
    uint64_t struct_size;
    const void* q;
    void* out;
    int64_t dtype, B, N, q_heads, kv_heads, dim;
    int64_t q_stride_b, q_stride_n, q_stride_h;
    int64_t o_stride_b, o_stride_n, o_stride_h;
    double scale;
    int64_t window, max_context;
    sv_paged_cache cache;
    void* workspace;
    int64_t workspace_bytes;
    uint32_t* row_status;
    uint64_t wait_limit_ns;
} sv_attention_args;

size_t spec_verify_attention_workspace_size(int64_t B, int64_t N, int64_t q_heads, int64_t kv_heads, int64_t dim);
int spec_verify_attention(const sv_attention_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_VERIFY_TARGET_H */
