/*
 * kvcache.h -- C ABI of the paged 8-bit KV cache (sm_103a): appending keys and
 * values, attention over them, and the bookkeeping of the pages.
 *
 * The noflash-attention forum post's LLM benchmark (ai-navigate-news, table
 * "PyTorch LLM Inference") decodes against a KV cache; attn_fwd_splitkv does
 * that for one dense 16-bit cache per sequence.  Here the cache is cut into
 * pages that sequences hold through a table, and its values are e4m3 with one
 * power-of-two scale per (page, KV head), which halves the bytes a decode step
 * reads.
 *
 * Conventions (as in attn.h): device pointers owned by the caller, 16-byte
 * aligned (scales and int32 arrays: 4 bytes), dense row-major; work enqueued on `stream`; no allocation, no
 * synchronisation.  Lengths, tables and counts live on the device, so a
 * decoding loop needs no host round trip and may be captured in a graph.
 *
 *   k_pages, v_pages : [n_pages, Hkv, page, D]  e4m3 (sign, 4 exponent bits
 *                      with bias 7, 3 mantissa bits; no infinities)
 *   k_scale, v_scale : [n_pages, Hkv]           fp32, 2^e with -126 <= e <= 120
 *   table            : [B, max_pages]           int32 page ids, -1: none
 *   lens             : [B]                      int32 positions held
 *   refs             : [n_pages]                int32 sequences holding a page
 * Token t of sequence b is row t % page of page table[b][t / page]; its key is
 * the e4m3 value times the page's scale for that head.  page is 16, 32, 64 or
 * 128; D is 64 or 128.  The 16-bit dtype is ATTN_F16 or ATTN_BF16.
 *
 * What the device finds wrong (a page id outside the pool where a token is
 * needed, a length past the table, a bad parent) is skipped, never read or
 * written, and recorded in the status word: attn_sync_status() then returns
 * ATTN_ERR_PAGE, or ATTN_ERR_POOL when a pool had too few free pages (one after
 * the other when both happened).
 */
#ifndef TME_KVCACHE_H
#define TME_KVCACHE_H

#include <stddef.h>

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Quantises new keys and values into the cache.  k, v: 16-bit, element (b, h, t,
 * d) at b*stride_b + h*stride_h + t*stride_t + d elements (strides multiples of
 * 8, for both).  Sequence b takes its first n = n_new[b] (NULL: T) tokens, 0 <= n
 * <= T; they become positions lens[b] - n .. lens[b] - 1, so lens holds the
 * lengths after the call and is not changed by it (every layer appends with the
 * same lens).  The pages must already be in the table, and pages that take
 * tokens belong to one sequence only (kvp_reserve and kvp_reassign see to both).
 *
 * The scale of a (page, head) is the smallest power of two that brings every
 * finite magnitude the page holds to at most 448.  When new tokens raise it, the
 * page's earlier tokens are rounded to it again: a power of two moves e4m3
 * values exactly except those that become subnormal.  Values round to nearest
 * even; infinities are stored as the largest magnitude, NaN as NaN.  Rows past
 * the last token are left as they were.
 *
 * lens has to hold the tokens: after a kvp_reserve that found no room it does
 * not, and the same n_new would be written over the newest ones.  Look at its
 * info[0] first, or use kv8_append_step.
 */
int kv8_append(const void* k, const void* v, void* k_pages, void* v_pages, float* k_scale,
               float* v_scale, const int* table, const int* lens, const int* n_new, int B,
               int Hkv, int T, int D, int page, int n_pages, int max_pages, long long stride_b,
               long long stride_h, long long stride_t, int dtype, void* stream);

/*
 * kv8_append for a step that no host looks at: granted (one int32 on the device,
 * written by kvp_reserve_step; NULL: 1) is 0 when the step was given no room,
 * and nothing is read or written then.
 */
int kv8_append_step(const void* k, const void* v, void* k_pages, void* v_pages, float* k_scale,
                    float* v_scale, const int* table, const int* lens, const int* n_new,
                    const int* granted, int B, int Hkv, int T, int D, int page, int n_pages,
                    int max_pages, long long stride_b, long long stride_h, long long stride_t,
                    int dtype, void* stream);

/*
 * Attention of the newest Nq positions of every sequence over its cache:
 * q, out [B, Hq, Nq, D] (dtype), lse [B, Hq, Nq] fp32.  Query i of sequence b
 * stands at position p = lens[b] - Nq + i and sees keys j <= p; with window > 0
 * only those with j > p - window or j < sinks (0: no window).  A query before
 * the sequence's first position, and so every query of an empty one, gets out = 0
 * and lse = -inf.  Query head h reads KV head h / (Hq / Hkv).
 *
 * Built for few query rows (a decoding step or a draft: all G * Nq rows of a KV
 * head share one pass over its keys up to 32 rows, longer blocks take more
 * passes).  Every CTA takes an equal share of all sequences' visible keys, found
 * on the device from lens, so mixed lengths are balanced without the host.
 * The keys' part of the arithmetic is exact in fp16 (e4m3 fits), scores, softmax
 * statistics and sums are fp32, the softmax terms of the value product fp16.
 * B <= 1024, and all sequences' table capacity times KV heads and passes under
 * 2^31 tiles of 32 tokens (ATTN_ERR_UNSUPPORTED otherwise).  Rows past a
 * sequence's end and keys that no query of the call sees may hold anything; a NaN
 * or infinity in a value that one of several queries (Nq > 1) sees reaches the
 * queries of the call that do not see it, too.
 * With a window kvp_reserve has given back what the tokens it made room for do not
 * see: where a sequence took fewer than Nq of them, the first of the Nq queries may
 * want such a page, which is recorded as a bad one (kv8_attn_step takes the counts).
 * workspace: kv8_attn_workspace_size() bytes.
 */
int kv8_attn(const void* q, const void* k_pages, const void* v_pages, const float* k_scale,
             const float* v_scale, const int* table, const int* lens, void* out, float* lse,
             void* workspace, size_t workspace_bytes, int B, int Hq, int Hkv, int Nq, int D,
             int page, int n_pages, int max_pages, float scale, int window, int sinks, int dtype,
             void* stream);

/*
 * kv8_attn for the tokens of one step.  n_new [B] on the device (NULL: Nq each):
 * the first n = n_new[b] queries are the sequence's n newest positions, as
 * kv8_append takes the first n tokens: query i < n stands at lens[b] - n + i, the
 * others see nothing (out = 0, lse = -inf).  A count outside [0, Nq] or past lens[b]
 * is recorded like a bad length, and none of the sequence's queries sees anything.
 * granted (one int32 on the device, written by kvp_reserve_step; NULL: 1): where it
 * is 0 no query of the call sees anything.  Other arguments are kv8_attn's.
 */
int kv8_attn_step(const void* q, const void* k_pages, const void* v_pages, const float* k_scale,
                  const float* v_scale, const int* table, const int* lens, const int* n_new,
                  const int* granted, void* out, float* lse, void* workspace,
                  size_t workspace_bytes, int B, int Hq, int Hkv, int Nq, int D, int page,
                  int n_pages, int max_pages, float scale, int window, int sinks, int dtype,
                  void* stream);

/* Workspace bytes kv8_attn needs on the current device (partial results of the
 * shares that end inside a sequence); 0 for invalid sizes.  Host-only apart from
 * the SM count. */
size_t kv8_attn_workspace_size(int B, int Hq, int Hkv, int Nq, int D);

/*
 * Which sequences begin with the same pages, as kvp_reassign leaves them: fills plan
 * (kvp_plan_words(n_seqs) int32 on the device) for kv8_attn_shared.  Sequences whose
 * first pages are the same, in whole runs of 128 positions, form a group; where some of
 * them share more than the others, each joins the group that leaves it the least to
 * read.  A group is kept when reading its prefix once saves min_saved positions or more
 * (members less one, times the prefix), and the attention follows all that are kept.  min_saved -1
 * keeps those that save 8192, and leaves the rest to the attention: it follows the plan where its groups save
 * 128 MB of keys and values in all, and of these the ones with enough members for the call's rows (D = 64: 8, 6 with
 * 9 to 16 query rows of a KV head; D = 128: 3; any with more rows); other sequences read for
 * themselves.  table [n_seqs, max_pages] and lens are not changed.  n_seqs <= 1024.
 *
 * The plan stays right while every sequence keeps the pages it begins with: appends, kvp_reserve
 * without a window and kvp_compact keep them; after kvp_reassign it is made anew.  (Work
 * grows with n_seqs^2 times the prefix's runs: it is for a fork, not for every step.)
 */
int kvp_find_shared(const int* table, const int* lens, int n_seqs, int max_pages, int page,
                    int min_saved, int* plan, void* stream);

/* int32 words of a plan; 0 for invalid counts.  Host-only. */
size_t kvp_plan_words(int n_seqs);

/*
 * kv8_attn_step, without a window, for sequences that share prefixes: the prefix of a
 * group is read once for all rows of its sequences (which then meet it as one matrix on
 * the tensor cores), the rest as there, and the two parts are merged by their LSEs in
 * fp32.  plan is kvp_find_shared's for the same table; something else than a plan for B
 * sequences is recorded like a bad page, and every sequence then reads for itself.
 * n_new and granted as in kv8_attn_step, other arguments and limits as in kv8_attn; up to 2^20
 * rows (G Nq) of a KV head.
 *
 * Within a group's prefix the values of 128 positions meet the product at one power of two, the
 * largest of their pages' scales and of those before: where scales differ by more than 2^15 the
 * smaller ones' values lose bits that stand 2^-33 below the larger's magnitude.  A
 * NaN or infinity in a value of the prefix reaches all rows of the group's
 * sequences, those before its position too.
 * workspace: kv8_attn_shared_workspace_size() bytes: all rows in fp32 twice (8 bytes per value of q), whether they
 * share or not, and up to 40 MB of parts.
 */
int kv8_attn_shared(const void* q, const void* k_pages, const void* v_pages, const float* k_scale,
                    const float* v_scale, const int* table, const int* lens, const int* n_new,
                    const int* granted, const int* plan, void* out, float* lse, void* workspace,
                    size_t workspace_bytes, int B, int Hq, int Hkv, int Nq, int D, int page,
                    int n_pages, int max_pages, float scale, int dtype, void* stream);

/* Workspace bytes of kv8_attn_shared on the current device; 0 for invalid sizes. */
size_t kv8_attn_shared_workspace_size(int B, int Hq, int Hkv, int Nq, int D);

/*
 * Copies pages src[i] to dst[i], keys, values and scales, for i < min(*count,
 * max_count), in each of n_layers pools that follow one another ([n_layers,
 * n_pages, ...]).  src, dst and count are device arrays; no dst may be a src or
 * repeat.  An id outside the pool is skipped and recorded.
 */
int kv8_copy_pages(void* k_pages, void* v_pages, float* k_scale, float* v_scale, const int* src,
                   const int* dst, const int* count, int max_count, int n_layers, int Hkv,
                   int page, int D, int n_pages, void* stream);

/*
 * Makes room for n_new[b] tokens of each of n_seqs sequences (0: it rests):
 * adds them to lens and fills the table with free pages (refs 0), lowest id
 * first, sequences in order.  With window > 0 a sequence that takes tokens first
 * gives back the pages that no query from its first new position on can see
 * (all their positions >= sinks and <= lens - window, lens before the call; the
 * search goes back to the columns an earlier call has emptied, so a cache keeps
 * one window and one number of sinks).
 * When pages or table columns run out nothing changes and ATTN_ERR_POOL is
 * recorded.  info[4] (device): 1 done / 0 not, pages taken, pages given back,
 * pages still free.  workspace: kvp_workspace_size() bytes.
 */
int kvp_reserve(int* table, int* lens, int* refs, const int* n_new, int n_seqs, int max_pages,
                int n_pages, int page, int window, int sinks, int* info, void* workspace,
                size_t workspace_bytes, void* stream);

/*
 * kvp_reserve that also writes info[0] to granted (one int32 on the device, or
 * NULL), which no other call writes: the step's appends and attention read it.
 */
int kvp_reserve_step(int* table, int* lens, int* refs, const int* n_new, int n_seqs, int max_pages,
                     int n_pages, int page, int window, int sinks, int* info, int* granted,
                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gives every sequence the content of another, all at once: sequence c becomes
 * what parents[c] was before the call; parents[c] = c keeps it, -1 frees it.
 * This frees finished sequences, forks one for n-best sampling and reorders
 * beams.  Full pages are shared (refs counts their holders).  A partly filled
 * last page stays with the parent itself if it keeps its content, else with
 * its first child; every other child gets a free page (lowest id first, children
 * in order) and the pair is listed in copy_src / copy_dst [n_seqs], to be given
 * to kv8_copy_pages before the next append.  A bad parent keeps its sequence and
 * is recorded; too few free pages change nothing and record ATTN_ERR_POOL.
 * info[4] (device): 1 done / 0 not, pairs to copy, pages given back, pages free.
 */
int kvp_reassign(int* table, int* lens, int* refs, const int* parents, int n_seqs, int max_pages,
                 int n_pages, int page, int* copy_src, int* copy_dst, int* info, void* workspace,
                 size_t workspace_bytes, void* stream);

/*
 * Renumbers the held pages so that they are [0, n_held): the i-th free id below
 * n_held takes the page of the i-th held id from n_held on.  The moves are
 * listed in move_src / move_dst [n_pages / 2], for kv8_copy_pages.  table_out and
 * refs_out may be table and refs.  info[4] (device): 1, moves, pages held, pages
 * free.  (A pool may then be cut to its first info[2] pages.)
 */
int kvp_compact(const int* table, const int* refs, int* table_out, int* refs_out, int n_seqs,
                int max_pages, int n_pages, int* move_src, int* move_dst, int* info,
                void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of the kvp_ calls; 0 for invalid sizes.  Host-only. */
size_t kvp_workspace_size(int n_seqs, int max_pages, int n_pages);

#ifdef __cplusplus
}
#endif

#endif /* TME_KVCACHE_H */
