/*
 * rope.h -- C ABI of rotary positions (sm_103a): queries and keys turned pair by
 * pair by an angle that grows with their position, ahead of the attention calls
 * of attn.h; and the cache's append that does it on the way (kvcache.h).
 *
 * Conventions as in attn.h: device pointers owned by the caller, work enqueued on
 * `stream`; no allocation, no synchronisation.
 *
 * The first `rot` dimensions of a head's row (rot even, 2 <= rot <= D) are rot / 2
 * pairs: (x[i], x[i + rot / 2]), or (x[2 i], x[2 i + 1]) when interleaved.  Pair i of
 * a row at position p becomes
 *     a' = A (a cos t - b sin t),  b' = A (b cos t + a sin t),  t = p f_i;
 * dimensions from rot on stay.  turns[i] holds the frequency f_i (radians per
 * position) as a fraction of a turn in 64 bits, round(f_i / (2 pi) * 2^64) mod 2^64, on the
 * device: angles of far positions lose nothing then.  Scaling for long contexts
 * is a choice of the f_i and of A.  The arithmetic is fp32, each result rounded once.
 */
#ifndef TME_ROPE_H
#define TME_ROPE_H

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Turns the rows of q [B, Hq, N, D] and k [B, Hk, N, D] (16 bits, ATTN_F16 or
 * ATTN_BF16; k and k_out NULL with Hk = 0: q alone) into q_out and k_out.  D is 64 or
 * 128.  Row n of sequence b stands at positions[b * ps_b + n * ps_n] (int32, any
 * sign), or where positions is NULL at start + n.  transposed = 1 turns back
 * (by -t, times A): the gradient of the call with 0, given the gradient of its
 * results.
 *
 * strides (host): 14 element counts, the batch, head and row strides of q, k, q_out and
 * k_out, then ps_b and ps_n; those of the 16-bit tensors are multiples of 8 and their pointers
 * 16-byte aligned.  Rows are dense.  A result may be its input (the same pointer and
 * strides); any other overlap is the caller's mistake.  Up to 2^27 tokens (B N) and 65535 heads (Hq + Hk);
 * positions counted from start end below 2^31.
 */
int rope_apply(const void* q, const void* k, void* q_out, void* k_out,
               const unsigned long long* turns, const int* positions, int start, int B, int Hq,
               int Hk, int N, int D, int rot, int interleaved, float amplitude, int transposed,
               const long long* strides, int dtype, void* stream);

/*
 * kv8_append_step with rotated keys: token t of sequence b is turned to the
 * position it takes in the cache, lens[b] - n + t, and quantised from fp32 (no
 * rounding to 16 bits between); values and everything else as there.  A key's infinities and
 * NaN go through the rotation's arithmetic first.
 *
 * q (NULL: none) [B, Hq, T, D] are the step's queries, turned to the same positions
 * into q_out (which may be q); rows from n_new[b] on, and all rows of a sequence whose
 * count does not fit or of a step without room, become 0.
 *
 * strides (host): batch, head and row strides of k and v (both), of q and of q_out.  T and the
 * positions of a table row together stay below 2^31; with q, up to 2^27 tokens (B T) and 65535 query heads.
 */
int kv8_append_rope(const void* k, const void* v, void* k_pages, void* v_pages, float* k_scale,
                    float* v_scale, const int* table, const int* lens, const int* n_new,
                    const int* granted, const void* q, void* q_out,
                    const unsigned long long* turns, int rot, int interleaved, float amplitude,
                    int B, int Hq, int Hkv, int T, int D, int page, int n_pages, int max_pages,
                    const long long* strides, int dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TME_ROPE_H */
