/*
 * pagedkv.h — C ABI of the GB300 (sm_103a) paged KV-cache library.
 *
 * The paged KV-cache hot path of an LLM decode server: slot filling, cache
 * writes (BF16, FP8-E4M3 K with BF16 V, FP8 K and V, fused RMSNorm/RoPE K, V
 * only), paged decode and chunked-prefill attention over those caches, an FP8
 * cache with block scales, windows with sinks, and page moves. The calls that
 * the source pages have, and their argument order, follow the Rust launchers on
 * the pages
 *   "spark_model/layers/ops/kv_cache.rs"              (written [kv_cache.rs]) and
 *   "metrale_model_layers/layers/ops/kv_cache_fp8k.rs" (written [kv_cache_fp8k.rs]),
 * with the launcher's GPU/kernel handles dropped and the stream last.
 *
 * Conventions for every call
 *   - Pointers marked "device" are CUDA device (or managed) memory owned by
 *     the caller; the library never allocates, frees or keeps them, and never
 *     synchronises. Every call is asynchronous on `stream` and returns once
 *     the work is queued. The stream is a cudaStream_t passed as void* (NULL
 *     means the legacy default stream), so that this header and its callers
 *     (C code, ctypes) need no CUDA header; the scope table's listing writes
 *     it as cudaStream_t.
 *   - BF16 data are passed as their 16-bit patterns (kv_bf16_t), FP8 data as
 *     E4M3 ("FN": no infinities, max 448, NaN 0x7F/0xFF) codes (kv_e4m3_t).
 *   - Cache pools are [num_blocks, block_size, num_kv_heads, head_dim], row
 *     major ("NHD" within a block). A flat slot s is row s % block_size of
 *     block s / block_size, so its num_kv_heads * head_dim elements start at
 *     element s * num_kv_heads * head_dim of the pool base pointer.
 *   - A negative slot in slot_mapping marks a padding token: nothing is
 *     written for it.
 *   - Return value: KV_OK, or an error code below. Argument errors are found
 *     on the host before anything is queued. Errors in device-resident data
 *     (a slot or block id outside the pool, a table shorter than a sequence)
 *     cannot be seen on the host; keeping them in range is the caller's
 *     contract, as with the pages' kernels. Calls with no work
 *     (count == 0, num_tokens == 0, num_seqs == 0) return KV_OK and launch
 *     nothing, as [kv_cache.rs] `fill_slots_from_block_table` does for
 *     count == 0.
 */
#ifndef PAGEDKV_H
#define PAGEDKV_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define PAGEDKV_API __attribute__((visibility("default")))
#else
#define PAGEDKV_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t kv_bf16_t; /* BF16 bit pattern */
typedef uint8_t kv_e4m3_t;  /* FP8 E4M3 code */

enum kv_status {
    KV_OK = 0,
    KV_ERR_INVALID_ARG = 1,  /* null pointer with work to do, bad shape or stride */
    KV_ERR_UNSUPPORTED = 2,  /* legal but outside what the kernels implement */
    KV_ERR_CUDA = 3,         /* a CUDA runtime or driver call failed */
    KV_ERR_DEVICE = 4        /* kv_get_device_error only: a kernel reported a fault in device
                                data or a wait timeout since the last read */
};

/* Human-readable text of a status code (static storage). */
PAGEDKV_API const char *kv_status_string(int status);

/* ------------------------------------------------------------------------
 * Slot filling.  [kv_cache.rs] `fill_slots_from_block_table`.
 *
 * slots[i] = block_table[p / block_size] * block_size + p % block_size for
 * p = start_pos + i, i < count.
 *   slots        device int64[count], written.
 *   block_table  device int32[ceil((start_pos + count) / block_size)], the
 *                sequence's physical block ids in logical order. A negative
 *                id gives a negative (skipped) slot.
 *   block_size   > 0.
 * ---------------------------------------------------------------------- */
PAGEDKV_API int kv_fill_slots(int64_t *slots, const int32_t *block_table, uint32_t start_pos, uint32_t count,
                  uint32_t block_size, void *stream);

/* ------------------------------------------------------------------------
 * BF16 cache write.  [kv_cache.rs] `reshape_and_cache` ("BF16 reshape and
 * cache — no quantization, direct BF16 copy"; its kernel-name line is a
 * garbled FP8 name and is not followed).
 *
 * For token t < num_tokens with slot = slot_mapping[t] >= 0 and head h:
 *   k_cache[slot][h][:] = key[t * key_stride + h * head_dim + :]
 *   v_cache[slot][h][:] = value[t * value_stride + h * head_dim + :]
 * bit for bit.
 *   key, value        device bf16, row t at element t * key_stride (resp.
 *                     value_stride); strides >= num_kv_heads * head_dim.
 *   k_cache, v_cache  device bf16 pools.
 *   slot_mapping      device int64[num_tokens].
 * Distinct tokens must not share a slot (their order is then unspecified).
 * ---------------------------------------------------------------------- */
PAGEDKV_API int kv_write_bf16(const kv_bf16_t *key, const kv_bf16_t *value, kv_bf16_t *k_cache,
                  kv_bf16_t *v_cache, const int64_t *slot_mapping, uint32_t num_tokens,
                  uint32_t num_kv_heads, uint32_t head_dim, uint32_t block_size,
                  uint32_t key_stride, uint32_t value_stride, void *stream);

/* ------------------------------------------------------------------------
 * FP8-K / BF16-V cache write.  [kv_cache_fp8k.rs] module invariants: K is
 * stored as k / k_scale in E4M3 in the NHD layout; argument order of
 * `reshape_and_cache_fp8k_turbo3v` without its TurboQuant-V arguments. V is a
 * BF16 copy as in kv_write_bf16.
 *
 * code = E4M3(round-to-nearest-even, saturating to +-448)(fp32(k) / k_scale),
 * where the quotient is the IEEE binary32 division rounded to nearest; NaN
 * inputs give 0x7F. Bit-exact.
 *   k_cache_fp8  device uint8 pool; v_cache device bf16 pool.
 *   k_scale      per-tensor scale, finite and > 0.
 * ---------------------------------------------------------------------- */
PAGEDKV_API int kv_write_fp8k(const kv_bf16_t *key, const kv_bf16_t *value, kv_e4m3_t *k_cache_fp8,
                  kv_bf16_t *v_cache, const int64_t *slot_mapping, uint32_t num_tokens,
                  uint32_t num_kv_heads, uint32_t head_dim, uint32_t block_size,
                  uint32_t key_stride, uint32_t value_stride, float k_scale, void *stream);

/* ------------------------------------------------------------------------
 * FP8 K and V cache write.  [kv_cache.rs] `reshape_and_cache_fp8`: K stored
 * as k / k_scale and V as v / v_scale, both E4M3 with the rule of
 * kv_write_fp8k, into two uint8 pools of the NHD layout. Argument order of
 * that launcher (scales before strides); its cache_stride is implied by the
 * layout and dropped. Bit-exact.
 *   k_scale, v_scale  per-tensor scales, finite and > 0.
 * ---------------------------------------------------------------------- */
PAGEDKV_API int kv_write_fp8(const kv_bf16_t *key, const kv_bf16_t *value, kv_e4m3_t *k_cache_fp8,
                             kv_e4m3_t *v_cache_fp8, const int64_t *slot_mapping, uint32_t num_tokens,
                             uint32_t num_kv_heads, uint32_t head_dim, uint32_t block_size, float k_scale,
                             float v_scale, uint32_t key_stride, uint32_t value_stride, void *stream);

/* ------------------------------------------------------------------------
 * Fused K path.  [kv_cache.rs] `fused_k_norm_rope_cache_write_bf16`: RMSNorm,
 * then RoPE, then the BF16 paged write in one kernel, K kept above BF16
 * precision throughout and rounded once at the write.
 *
 * For token t with slot >= 0 and head h, x = k_in[t][h][:] (contiguous
 * [num_tokens, num_kv_heads, head_dim], no stride argument on the page):
 *   y_d = x_d / sqrt(mean(x^2) + rms_eps) * k_norm_weight[d]
 *   for i < rotary_dim/2, angle = positions[t] * theta^(-2i/rotary_dim):
 *     o_i = y_i cos - y_{i+R/2} sin,  o_{i+R/2} = y_{i+R/2} cos + y_i sin
 *   o_d = y_d for d >= rotary_dim
 *   k_cache[slot][h][d] = BF16_RNE(o_d)
 * The result is within 1 BF16 ulp of the exactly rounded value.
 *   k_norm_weight  device bf16[head_dim], shared by all heads.
 *   positions      device int32[num_tokens], >= 0.
 *   rotary_dim     even, 8 <= rotary_dim <= head_dim, multiple of 8.
 * The V half goes through kv_write_v_only.
 * ---------------------------------------------------------------------- */
PAGEDKV_API int kv_write_fused_k_norm_rope_bf16(const kv_bf16_t *k_in, const kv_bf16_t *k_norm_weight,
                                    const int32_t *positions, kv_bf16_t *k_cache,
                                    const int64_t *slot_mapping, uint32_t num_tokens,
                                    uint32_t num_kv_heads, uint32_t head_dim, uint32_t rotary_dim,
                                    uint32_t block_size, float rms_eps, float theta, void *stream);

/* ------------------------------------------------------------------------
 * MRoPE-interleaved fused K path. [kv_cache.rs]
 * `fused_k_norm_rope_cache_write_bf16_mrope`: as
 * kv_write_fused_k_norm_rope_bf16, but rotation pair i of token t turns by
 * pos * theta^(-2i/rotary_dim) with pos = (pos_t, pos_h, pos_w)[i % 3][t].
 * With pos_t == pos_h == pos_w the result is bit-identical to
 * kv_write_fused_k_norm_rope_bf16.
 *   pos_t, pos_h, pos_w  device int32[num_tokens] each.
 * ---------------------------------------------------------------------- */
PAGEDKV_API int kv_write_fused_k_norm_rope_bf16_mrope(
    const kv_bf16_t *k_in, const kv_bf16_t *k_norm_weight, const int32_t *pos_t, const int32_t *pos_h,
    const int32_t *pos_w, kv_bf16_t *k_cache, const int64_t *slot_mapping, uint32_t num_tokens,
    uint32_t num_kv_heads, uint32_t head_dim, uint32_t rotary_dim, uint32_t block_size, float rms_eps,
    float theta, void *stream);

/* ------------------------------------------------------------------------
 * FP8-output fused K path. [kv_cache.rs] `fused_k_norm_rope_cache_write_fp8`:
 * the same RMSNorm and RoPE with no BF16 rounding; the result times
 * inv_scale (finite, > 0; inv_scale = 1 / k_scale of the FP8-K decode) is
 * cast once to E4M3, round to nearest even, saturating to +-448. The code
 * equals the correctly rounded one except where the exact scaled value lies
 * within ~2^-19 (relative) of the midpoint between two codes; there either
 * neighbour may be stored.
 *   k_cache_fp8  device uint8 pool [num_blocks, block_size, num_kv_heads, head_dim].
 * ---------------------------------------------------------------------- */
PAGEDKV_API int kv_write_fused_k_norm_rope_fp8(const kv_bf16_t *k_in, const kv_bf16_t *k_norm_weight,
                                               const int32_t *positions, kv_e4m3_t *k_cache_fp8,
                                               const int64_t *slot_mapping, uint32_t num_tokens,
                                               uint32_t num_kv_heads, uint32_t head_dim, uint32_t rotary_dim,
                                               uint32_t block_size, float rms_eps, float theta, float inv_scale,
                                               void *stream);

/* ------------------------------------------------------------------------
 * Rotary positions (not on the pages, whose rotation comes with an RMSNorm, in
 * one layout and for K alone). Pair i < rotary_dim / 2 of a head is its elements
 * i and i + rotary_dim / 2, or (interleaved nonzero) 2i and 2i + 1; a row at
 * position P has
 *   o_x = a_i (x cos(P f_i) - y sin(P f_i)),  o_y = a_i (y cos(P f_i) + x sin(P f_i))
 * for each pair (x, y) and its elements from rotary_dim on unchanged. f_i and a_i
 * come from a table, built once:
 *
 * kv_rope_frequencies (host) writes rotary_dim / 2 frequencies, radians per
 * position: theta^(-2i/rotary_dim), for contexts longer than the trained_len
 * positions that a model was trained on scaled by `factor` s
 *   KV_ROPE_LINEAR    f / s (positions interpolated)
 *   KV_ROPE_BASE      theta s^(R/(R-2)) in place of theta: the slowest pair slowed
 *                     by s, the fastest kept
 *   KV_ROPE_BY_TURNS  f (k + (1 - k) / s), k from 0 for pairs that make `low` turns
 *                     over trained_len positions (or fewer) to 1 for those that
 *                     make `high`, linear in the turns
 *   KV_ROPE_BY_INDEX  the same, k linear in i between the pairs at which
 *                     theta^(-2i/R) trained_len / 2 pi is `high` and `low` (rounded
 *                     down and up to a whole index)
 * The arguments that a scaling does not name are not looked at.
 *
 * kv_rope_table (host) makes the table of rotary_dim / 2 frequencies in [0,
 * 2^60] and one amplitude a (1, or what a model's scaling asks for, such as 0.1 ln
 * s + 1): uint32[rotary_dim / 2][4], in host memory, which the caller copies to the
 * device (16-byte aligned) for the calls below.
 * ---------------------------------------------------------------------- */
enum kv_rope_scaling {
    KV_ROPE_PLAIN = 0,
    KV_ROPE_LINEAR = 1,
    KV_ROPE_BASE = 2,
    KV_ROPE_BY_TURNS = 3,
    KV_ROPE_BY_INDEX = 4
};

PAGEDKV_API int kv_rope_frequencies(double *freqs, uint32_t rotary_dim, double theta, int scaling, double factor,
                                    double trained_len, double low, double high);
PAGEDKV_API int kv_rope_table(uint32_t *table, const double *freqs, uint32_t rotary_dim, float amplitude);

/* Rotates num_heads heads of each row of x (bf16, row t at element t * x_stride)
 * into out (row t at t * out_stride); the angles are exact for any int32 position
 * and each result is within 1 BF16 ulp of the exactly rounded one, or within 2^-38 of
 * |a| (|x| + |y|) where the two products cancel beyond that (for x and y below 2^127;
 * larger ones may overflow on the way). A pair that holds an infinity or a NaN gives what
 * the formula gives, and no other pair is touched by it. `inverse`
 * nonzero turns back by the same angles (with the same amplitude): the gradient of
 * the rotation, or (with positions that are differences) rows moved to others.
 *   out        may be x itself, with the same stride; no other overlap.
 *   positions  device int32[num_tokens], any sign.
 * Supported: head_dim 64, 128 or 256; rotary_dim a multiple of 8 up to head_dim;
 * any alignment and strides of x and out (16-byte ones are faster). */
PAGEDKV_API int kv_rope(const kv_bf16_t *x, kv_bf16_t *out, const uint32_t *rope_table, const int32_t *positions,
                        uint32_t num_tokens, uint32_t num_heads, uint32_t head_dim, uint32_t rotary_dim,
                        uint32_t x_stride, uint32_t out_stride, int interleaved, int inverse, void *stream);

/* A step's queries, keys and values in one call: for each token t with slot =
 * slot_mapping[t] >= 0, its num_q_heads heads of q are rotated into q_out, its keys
 * rotated into row `slot` of the K pool, and its values copied into the V pool
 * (bf16), or keys and values stored as E4M3(x / scale), as kv_write_fp8k and
 * kv_write_fp8 do, the rotated key in 32 bits (its code is the correctly rounded one
 * except where the rotated key is within 2^-21 of itself, or within 2^-38 of its pair's
 * |a| (|x| + |y|), of a midpoint between two codes). A negative slot:
 * nothing is written for the token, its row of q_out included.
 *   q, key, value  device bf16 rows at element strides, such as parts of a fused
 *                  projection's rows; any alignment and strides.
 *   q_out          may be q itself, with the same stride; no other overlap.
 *                  With num_q_heads 0, q and q_out are not looked at.
 * Supported: as kv_rope; pools 16-byte aligned. */
PAGEDKV_API int kv_append_rope_bf16(const kv_bf16_t *q, const kv_bf16_t *key, const kv_bf16_t *value,
                                    kv_bf16_t *q_out, kv_bf16_t *k_cache, kv_bf16_t *v_cache,
                                    const uint32_t *rope_table, const int32_t *positions,
                                    const int64_t *slot_mapping, uint32_t num_tokens, uint32_t num_q_heads,
                                    uint32_t num_kv_heads, uint32_t head_dim, uint32_t rotary_dim,
                                    uint32_t block_size, uint32_t q_stride, uint32_t key_stride,
                                    uint32_t value_stride, uint32_t q_out_stride, int interleaved, void *stream);

PAGEDKV_API int kv_append_rope_fp8k(const kv_bf16_t *q, const kv_bf16_t *key, const kv_bf16_t *value,
                                    kv_bf16_t *q_out, kv_e4m3_t *k_cache_fp8, kv_bf16_t *v_cache,
                                    const uint32_t *rope_table, const int32_t *positions,
                                    const int64_t *slot_mapping, uint32_t num_tokens, uint32_t num_q_heads,
                                    uint32_t num_kv_heads, uint32_t head_dim, uint32_t rotary_dim,
                                    uint32_t block_size, uint32_t q_stride, uint32_t key_stride,
                                    uint32_t value_stride, uint32_t q_out_stride, int interleaved, float k_scale,
                                    void *stream);

PAGEDKV_API int kv_append_rope_fp8(const kv_bf16_t *q, const kv_bf16_t *key, const kv_bf16_t *value,
                                   kv_bf16_t *q_out, kv_e4m3_t *k_cache_fp8, kv_e4m3_t *v_cache_fp8,
                                   const uint32_t *rope_table, const int32_t *positions,
                                   const int64_t *slot_mapping, uint32_t num_tokens, uint32_t num_q_heads,
                                   uint32_t num_kv_heads, uint32_t head_dim, uint32_t rotary_dim,
                                   uint32_t block_size, uint32_t q_stride, uint32_t key_stride,
                                   uint32_t value_stride, uint32_t q_out_stride, int interleaved, float k_scale,
                                   float v_scale, void *stream);

/* ------------------------------------------------------------------------
 * V-only write.  [kv_cache.rs] `reshape_and_cache_flash_v_only`: the V half
 * of kv_write_bf16, so that the fused K kernel stays the only writer of K.
 * ---------------------------------------------------------------------- */
PAGEDKV_API int kv_write_v_only(const kv_bf16_t *value, kv_bf16_t *v_cache, const int64_t *slot_mapping,
                    uint32_t num_tokens, uint32_t num_kv_heads, uint32_t head_dim,
                    uint32_t block_size, uint32_t value_stride, void *stream);

/* ------------------------------------------------------------------------
 * Paged decode attention.  [kv_cache.rs] `paged_decode_attn_fp8` doc (one
 * query per (query head, sequence); block_tables int32[num_seqs *
 * max_blocks_per_seq]; seq_lens int32[num_seqs]) and the argument list of
 * `paged_decode_attn_bf16k_turbo3v` without its TurboQuant-V arguments
 * (q_stride, sliding_window). [kv_cache_fp8k.rs]: the FP8 variant multiplies
 * the stored K by k_scale, which follows inv_sqrt_d in the argument list.
 *
 * For sequence s and query head h, with g = num_q_heads / num_kv_heads and
 * KV head h / g, L = seq_lens[s] (cached tokens, the current token included)
 * and start = (sliding_window > 0 ? max(0, L - sliding_window) : 0):
 *   position p in [start, L) lives at row p % block_size of block
 *   block_tables[s * max_blocks_per_seq + p / block_size];
 *   score_p = inv_sqrt_d * (q[s * q_stride + h * head_dim + :] . k_p)
 *   output[s][h][:] = sum_p softmax(score)_p * v_p     (zeros if L == 0)
 *   q       device bf16; q_stride (elements between sequences) >= num_q_heads * head_dim.
 *   output  device float32[num_seqs, num_q_heads, head_dim], written.
 *   seq_lens[s] <= max_blocks_per_seq * block_size.
 * Supported: head_dim in {64, 128, 256}; block_size a power
 * of two in [16, 256]; g <= 16; q, caches and q_stride 16-byte aligned;
 * output 8-byte aligned. Anything else returns KV_ERR_UNSUPPORTED.
 * With a workspace registered by kv_set_decode_workspace, the positions of
 * all sequences are shared out equally among the CTAs and a sequence split
 * between CTAs is merged afterwards (flash-decoding); without one every
 * (sequence, KV head group) runs in one CTA (same result, less parallelism).
 * ---------------------------------------------------------------------- */
PAGEDKV_API int paged_decode_attn_bf16(const kv_bf16_t *q, const kv_bf16_t *k_cache, const kv_bf16_t *v_cache,
                           float *output, const int32_t *block_tables, const int32_t *seq_lens,
                           uint32_t max_blocks_per_seq, uint32_t num_seqs, uint32_t num_q_heads,
                           uint32_t num_kv_heads, uint32_t head_dim, uint32_t block_size,
                           float inv_sqrt_d, uint32_t q_stride, uint32_t sliding_window,
                           void *stream);

PAGEDKV_API int paged_decode_attn_fp8k(const kv_bf16_t *q, const kv_e4m3_t *k_cache_fp8,
                           const kv_bf16_t *v_cache, float *output, const int32_t *block_tables,
                           const int32_t *seq_lens, uint32_t max_blocks_per_seq,
                           uint32_t num_seqs, uint32_t num_q_heads, uint32_t num_kv_heads,
                           uint32_t head_dim, uint32_t block_size, float inv_sqrt_d,
                           float k_scale, uint32_t q_stride, uint32_t sliding_window,
                           void *stream);

/* ------------------------------------------------------------------------
 * FP8 K and V paged decode.  [kv_cache.rs] `paged_decode_attn_fp8` (its
 * argument order, with num_seqs, q_stride and sliding_window as in the
 * calls above and cache_stride dropped): as paged_decode_attn_fp8k, with
 * v_p = E4M3 code * v_scale (v_scale finite and > 0) read from a uint8 V
 * pool.
 * ---------------------------------------------------------------------- */
PAGEDKV_API int paged_decode_attn_fp8(const kv_bf16_t *q, const kv_e4m3_t *k_cache_fp8,
                                      const kv_e4m3_t *v_cache_fp8, float *output, const int32_t *block_tables,
                                      const int32_t *seq_lens, uint32_t max_blocks_per_seq, uint32_t num_seqs,
                                      uint32_t num_q_heads, uint32_t num_kv_heads, uint32_t head_dim,
                                      uint32_t block_size, float inv_sqrt_d, float k_scale, float v_scale,
                                      uint32_t q_stride, uint32_t sliding_window, void *stream);

/* ------------------------------------------------------------------------
 * Multi-token (chunked-prefill) paged attention.  [kv_cache.rs] "Batched
 * prefill variants (N tokens)" gives only the heading; the reading here:
 * sequence s brings n_s = query_start_loc[s+1] - query_start_loc[s] query
 * tokens, the last n_s of its seq_lens[s] cached positions (their K/V
 * already written). Query j of s (row query_start_loc[s] + j of q, at
 * position P = seq_lens[s] - n_s + j) attends causally, over positions
 * [start, P] with start = (sliding_window > 0 ? max(0, P + 1 -
 * sliding_window) : 0): exactly what the paged decode attends for that
 * sequence cut to length P + 1. A query with P < 0 gives zeros. GQA,
 * inv_sqrt_d (here >= 0), the block tables and (FP8) k_scale are as in the
 * decode calls.
 *   q                bf16 rows [num_q_tokens], row stride q_stride elements,
 *                    head h at +h * head_dim.
 *   query_start_loc  device int32[num_seqs + 1], non-decreasing, from 0 to
 *                    num_q_tokens (a violation sets bit 2 of the device
 *                    fault word and that sequence's rows are skipped).
 *   output           device float32[num_q_tokens, num_q_heads, head_dim].
 * Precision: scores and sums in fp32; the PV product takes the softmax
 * weights as f16 (one rounding, relative error at most 2^-11) against V as
 * f16: E4M3 codes exactly, BF16 values as v * 2^-8 rounded to f16, exact for
 * 2^-6 <= |v| < 2^24 and within 2^-17 below. BF16 V values of magnitude
 * 2^24 or more are outside the supported range: the outputs of every query
 * whose keys share a 128-key tile with one are not finite.
 * Supported: head_dim 64 or 128; block_size a power of two in
 * [16, 256]; q, caches, q_stride and output 16-byte aligned. No workspace
 * is used.
 * ---------------------------------------------------------------------- */
PAGEDKV_API int paged_prefill_attn_bf16(const kv_bf16_t *q, const kv_bf16_t *k_cache, const kv_bf16_t *v_cache,
                                        float *output, const int32_t *block_tables, const int32_t *seq_lens,
                                        const int32_t *query_start_loc, uint32_t max_blocks_per_seq,
                                        uint32_t num_seqs, uint32_t num_q_tokens, uint32_t num_q_heads,
                                        uint32_t num_kv_heads, uint32_t head_dim, uint32_t block_size,
                                        float inv_sqrt_d, uint32_t q_stride, uint32_t sliding_window,
                                        void *stream);

PAGEDKV_API int paged_prefill_attn_fp8k(const kv_bf16_t *q, const kv_e4m3_t *k_cache_fp8,
                                        const kv_bf16_t *v_cache, float *output, const int32_t *block_tables,
                                        const int32_t *seq_lens, const int32_t *query_start_loc,
                                        uint32_t max_blocks_per_seq, uint32_t num_seqs, uint32_t num_q_tokens,
                                        uint32_t num_q_heads, uint32_t num_kv_heads, uint32_t head_dim,
                                        uint32_t block_size, float inv_sqrt_d, float k_scale, uint32_t q_stride,
                                        uint32_t sliding_window, void *stream);

/* Multi-token paged attention over an FP8 K and V cache (the cache that
 * kv_write_fp8 fills and paged_decode_attn_fp8 reads): as
 * paged_prefill_attn_fp8k, with v_p = E4M3 code * v_scale (v_scale finite and
 * > 0) read from a uint8 V pool. head_dim 64 or 128. */
PAGEDKV_API int paged_prefill_attn_fp8(const kv_bf16_t *q, const kv_e4m3_t *k_cache_fp8,
                                       const kv_e4m3_t *v_cache_fp8, float *output, const int32_t *block_tables,
                                       const int32_t *seq_lens, const int32_t *query_start_loc,
                                       uint32_t max_blocks_per_seq, uint32_t num_seqs, uint32_t num_q_tokens,
                                       uint32_t num_q_heads, uint32_t num_kv_heads, uint32_t head_dim,
                                       uint32_t block_size, float inv_sqrt_d, float k_scale, float v_scale,
                                       uint32_t q_stride, uint32_t sliding_window, void *stream);

/* ------------------------------------------------------------------------
 * FP8-K paged decode without any caller-provided memory. The source pages
 * have no counterpart of this call; it exists for callers that cannot give
 * the library a device allocation: applications whose device memory belongs
 * to another allocator (a framework memory pool, a serving engine that
 * reserves all of HBM for its KV cache) cannot set a raw buffer aside for a
 * library, and a cudaMalloc of their own would fail or break that
 * allocator's accounting. Like every call here it uses the CUDA API, so it
 * must not be made from a host function enqueued with cudaLaunchHostFunc.
 *
 * Same arguments, results and limits as paged_decode_attn_fp8k; the
 * split-KV scratch comes from a fixed 64 MiB array in the library's own
 * device memory, which every GPU that loads the library keeps until the
 * process exits. The call allocates and frees nothing. It returns
 * KV_ERR_UNSUPPORTED when the shape's worst-case scratch
 * (kv_decode_workspace_bytes of the same arguments) exceeds 64 MiB.
 * The first call on a device, with that device current, looks up the
 * array's device address (cudaGetSymbolAddress) and caches it: make that
 * first call before any stream capture, and do not call it on a device
 * after a cudaDeviceReset in the same process (the cached address belonged
 * to the reset context). All calls share the one array; no call reads what
 * an earlier one left there (but for partial sums where a wait gave up: bit 0
 * of the fault word, and that output is unspecified). Calls whose work may
 * overlap on the GPU (different streams, other devices' calls aside) race on
 * the array: order them.
 * ---------------------------------------------------------------------- */
PAGEDKV_API int paged_decode_attn_fp8k_static_scratch(
    const kv_bf16_t *q, const kv_e4m3_t *k_cache_fp8, const kv_bf16_t *v_cache, float *output,
    const int32_t *block_tables, const int32_t *seq_lens, uint32_t max_blocks_per_seq, uint32_t num_seqs,
    uint32_t num_q_heads, uint32_t num_kv_heads, uint32_t head_dim, uint32_t block_size, float inv_sqrt_d,
    float k_scale, uint32_t q_stride, uint32_t sliding_window, void *stream);

/* ------------------------------------------------------------------------
 * Sliding window with sinks (the source pages have the window only; dropping
 * a sequence's first tokens costs a model that rests attention on them far
 * more than any others). As the calls without `_sinks`, but a query at position
 * P attends every position p <= P with
 *   sliding_window == 0  or  p > P - sliding_window  or  p < num_sinks.
 * num_sinks 0 is the plain window; with sliding_window 0 it changes nothing.
 * Blocks that hold no attended position are not read: their table entries may
 * hold anything (kv_free_window_blocks makes them -1).
 * ---------------------------------------------------------------------- */
PAGEDKV_API int paged_decode_attn_bf16_sinks(const kv_bf16_t *q, const kv_bf16_t *k_cache,
                                             const kv_bf16_t *v_cache, float *output, const int32_t *block_tables,
                                             const int32_t *seq_lens, uint32_t max_blocks_per_seq,
                                             uint32_t num_seqs, uint32_t num_q_heads, uint32_t num_kv_heads,
                                             uint32_t head_dim, uint32_t block_size, float inv_sqrt_d,
                                             uint32_t q_stride, uint32_t sliding_window, uint32_t num_sinks,
                                             void *stream);

PAGEDKV_API int paged_decode_attn_fp8k_sinks(const kv_bf16_t *q, const kv_e4m3_t *k_cache_fp8,
                                             const kv_bf16_t *v_cache, float *output, const int32_t *block_tables,
                                             const int32_t *seq_lens, uint32_t max_blocks_per_seq,
                                             uint32_t num_seqs, uint32_t num_q_heads, uint32_t num_kv_heads,
                                             uint32_t head_dim, uint32_t block_size, float inv_sqrt_d,
                                             float k_scale, uint32_t q_stride, uint32_t sliding_window,
                                             uint32_t num_sinks, void *stream);

PAGEDKV_API int paged_decode_attn_fp8_sinks(const kv_bf16_t *q, const kv_e4m3_t *k_cache_fp8,
                                            const kv_e4m3_t *v_cache_fp8, float *output,
                                            const int32_t *block_tables, const int32_t *seq_lens,
                                            uint32_t max_blocks_per_seq, uint32_t num_seqs, uint32_t num_q_heads,
                                            uint32_t num_kv_heads, uint32_t head_dim, uint32_t block_size,
                                            float inv_sqrt_d, float k_scale, float v_scale, uint32_t q_stride,
                                            uint32_t sliding_window, uint32_t num_sinks, void *stream);

/* Multi-token forms: as paged_prefill_attn_* with the mask above, inv_sqrt_d >
 * 0, and the output rows in BF16, bf16[num_q_tokens, num_q_heads, head_dim],
 * 16-byte aligned: the softmax weights enter the products rounded to 11 bits,
 * so a 32-bit row would hold nothing that BF16's 8 bits drop but rounding, at
 * twice the bytes. A V value that is not finite makes the rows of every query
 * whose keys share a 128-key tile with it non-finite. */
PAGEDKV_API int paged_prefill_attn_bf16_sinks(const kv_bf16_t *q, const kv_bf16_t *k_cache,
                                              const kv_bf16_t *v_cache, kv_bf16_t *output,
                                              const int32_t *block_tables, const int32_t *seq_lens,
                                              const int32_t *query_start_loc, uint32_t max_blocks_per_seq,
                                              uint32_t num_seqs, uint32_t num_q_tokens, uint32_t num_q_heads,
                                              uint32_t num_kv_heads, uint32_t head_dim, uint32_t block_size,
                                              float inv_sqrt_d, uint32_t q_stride, uint32_t sliding_window,
                                              uint32_t num_sinks, void *stream);

PAGEDKV_API int paged_prefill_attn_fp8k_sinks(const kv_bf16_t *q, const kv_e4m3_t *k_cache_fp8,
                                              const kv_bf16_t *v_cache, kv_bf16_t *output,
                                              const int32_t *block_tables, const int32_t *seq_lens,
                                              const int32_t *query_start_loc, uint32_t max_blocks_per_seq,
                                              uint32_t num_seqs, uint32_t num_q_tokens, uint32_t num_q_heads,
                                              uint32_t num_kv_heads, uint32_t head_dim, uint32_t block_size,
                                              float inv_sqrt_d, float k_scale, uint32_t q_stride,
                                              uint32_t sliding_window, uint32_t num_sinks, void *stream);

PAGEDKV_API int paged_prefill_attn_fp8_sinks(const kv_bf16_t *q, const kv_e4m3_t *k_cache_fp8,
                                             const kv_e4m3_t *v_cache_fp8, kv_bf16_t *output,
                                             const int32_t *block_tables, const int32_t *seq_lens,
                                             const int32_t *query_start_loc, uint32_t max_blocks_per_seq,
                                             uint32_t num_seqs, uint32_t num_q_tokens, uint32_t num_q_heads,
                                             uint32_t num_kv_heads, uint32_t head_dim, uint32_t block_size,
                                             float inv_sqrt_d, float k_scale, float v_scale, uint32_t q_stride,
                                             uint32_t sliding_window, uint32_t num_sinks, void *stream);

/* ------------------------------------------------------------------------
 * Paged decode over shared prefixes (not on the pages). Sequences that hold the same
 * blocks - forks of one prompt, a batch under one system prompt - attend the same
 * rows of the cache; the calls above read them once for each sequence, these once for
 * each group of sequences, as one matrix product for all members.
 *
 * kv_prefix_plan finds what the members of each group share and cuts it into pieces,
 * on the device, into `plan`; the attention calls of every layer of a step, or of
 * several steps, then take that plan. Group g is sequences group_start[g] to
 * group_start[g+1] - 1. Shared are the leading whole blocks for which every member
 * that is longer than the block and attends it has the same table entry; groups that
 * share nothing, or too little to be worth it, are attended member by member. So the
 * groups are a hint: the result is that of the `_sinks` call (the block-scaled one)
 * over the same tables, lengths and window, in BF16, whatever they are - but for the
 * roundings and for values that are not finite, both below.
 * What is worth it is decided for BF16 caches (a plan knows no type): over 8-bit caches
 * pairs, and groups of four and eight over few positions, are slower shared than alone;
 * leave such groups out of group_start.
 *   plan         device memory of kv_prefix_plan_bytes(...), 16-byte aligned, written.
 *   group_start  device int32[num_groups + 1], non-decreasing, in [0, num_seqs] (otherwise
 *                bit 2 of the fault word is set and nothing is shared).
 *   head_dim     (and the other shapes, the window and num_sinks) as the attention
 *                call's.
 * A plan stays good while the shared blocks stay where they are and no length drops
 * below what it shares: lengths may grow from step to step. A sequence that is
 * replaced, or a block that moves or is freed (kv_compact_blocks, kv_free_blocks, and
 * under a window kv_free_window_blocks), needs a new plan. A plan made for other
 * arguments (shapes, num_groups, window, sinks) sets bit 6 of the fault word and is not
 * used: each sequence is attended by itself.
 * Supported: head_dim 64 or 128, block_size a power of two in [16, 256], num_groups up
 * to 4,096. Tables of at most 128 positions need no plan: none is written, and the
 * attention calls do not look at the buffer (which they take all the same).
 * ---------------------------------------------------------------------- */
PAGEDKV_API size_t kv_prefix_plan_bytes(uint32_t num_seqs, uint32_t num_groups, uint32_t num_q_heads,
                                        uint32_t num_kv_heads);

PAGEDKV_API int kv_prefix_plan(void *plan, const int32_t *block_tables, const int32_t *seq_lens,
                               const int32_t *group_start, uint32_t max_blocks_per_seq, uint32_t num_seqs,
                               uint32_t num_groups, uint32_t num_q_heads, uint32_t num_kv_heads, uint32_t head_dim,
                               uint32_t block_size, uint32_t sliding_window, uint32_t num_sinks, void *stream);

/* Decode with a plan: arguments as the `_sinks` calls (the block-scaled one), with
 * inv_sqrt_d > 0, the plan after the lengths and num_groups after num_seqs. The rows
 * are BF16, bf16[num_seqs, num_q_heads, head_dim], 8-byte aligned: the shared
 * positions' softmax weights enter the products rounded to 11 bits, as the prefill's.
 * The shared positions' BF16 V values are held as f16 of v 2^-8: exactly for 2^-9 <= |v| <
 * 2^24, within 2^-17 below, where the `_sinks` calls hold any value exactly (values of
 * order 10^-3 are off by up to 0.8%); own positions and E4M3 values exactly. A shared V
 * value that is not finite, or a BF16 one of 2^24 or more, makes the rows that attend it
 * non-finite, and may make those of any member of its group so (a weight of zero times
 * it is a NaN); one among a sequence's own positions makes that sequence's rows alone.
 * A workspace of at least kv_prefix_workspace_bytes(...) has to be registered by
 * kv_set_decode_workspace, else KV_ERR_UNSUPPORTED (tables of at most 128 positions
 * need none and are attended without the plan).
 * Supported: head_dim 64 or 128, the rest as the decodes. */
PAGEDKV_API int paged_decode_attn_bf16_prefix(const kv_bf16_t *q, const kv_bf16_t *k_cache,
                                              const kv_bf16_t *v_cache, kv_bf16_t *output,
                                              const int32_t *block_tables, const int32_t *seq_lens,
                                              const void *plan, uint32_t max_blocks_per_seq, uint32_t num_seqs,
                                              uint32_t num_groups, uint32_t num_q_heads, uint32_t num_kv_heads,
                                              uint32_t head_dim, uint32_t block_size, float inv_sqrt_d,
                                              uint32_t q_stride, uint32_t sliding_window, uint32_t num_sinks,
                                              void *stream);

PAGEDKV_API int paged_decode_attn_fp8k_prefix(const kv_bf16_t *q, const kv_e4m3_t *k_cache_fp8,
                                              const kv_bf16_t *v_cache, kv_bf16_t *output,
                                              const int32_t *block_tables, const int32_t *seq_lens,
                                              const void *plan, uint32_t max_blocks_per_seq, uint32_t num_seqs,
                                              uint32_t num_groups, uint32_t num_q_heads, uint32_t num_kv_heads,
                                              uint32_t head_dim, uint32_t block_size, float inv_sqrt_d,
                                              float k_scale, uint32_t q_stride, uint32_t sliding_window,
                                              uint32_t num_sinks, void *stream);

PAGEDKV_API int paged_decode_attn_fp8_prefix(const kv_bf16_t *q, const kv_e4m3_t *k_cache_fp8,
                                             const kv_e4m3_t *v_cache_fp8, kv_bf16_t *output,
                                             const int32_t *block_tables, const int32_t *seq_lens,
                                             const void *plan, uint32_t max_blocks_per_seq, uint32_t num_seqs,
                                             uint32_t num_groups, uint32_t num_q_heads, uint32_t num_kv_heads,
                                             uint32_t head_dim, uint32_t block_size, float inv_sqrt_d,
                                             float k_scale, float v_scale, uint32_t q_stride,
                                             uint32_t sliding_window, uint32_t num_sinks, void *stream);

PAGEDKV_API int paged_decode_attn_fp8_block_prefix(const kv_bf16_t *q, const kv_e4m3_t *k_cache_fp8,
                                                   const kv_e4m3_t *v_cache_fp8, const float *k_scales,
                                                   const float *v_scales, kv_bf16_t *output,
                                                   const int32_t *block_tables, const int32_t *seq_lens,
                                                   const void *plan, uint32_t max_blocks_per_seq,
                                                   uint32_t num_seqs, uint32_t num_groups, uint32_t num_q_heads,
                                                   uint32_t num_kv_heads, uint32_t head_dim,
                                                   uint32_t block_size, float inv_sqrt_d, uint32_t q_stride,
                                                   uint32_t sliding_window, uint32_t num_sinks, void *stream);

PAGEDKV_API size_t kv_prefix_workspace_bytes(uint32_t max_blocks_per_seq, uint32_t num_seqs,
                                             uint32_t num_groups, uint32_t num_q_heads, uint32_t num_kv_heads,
                                             uint32_t head_dim, uint32_t block_size);

/* ------------------------------------------------------------------------
 * FP8 cache with one scale for each block and KV head (not on the pages, whose
 * FP8 caches have one scale for a whole tensor: one outlier then sets the grid of
 * every token). The codes are in uint8 pools of the usual layout, the scales in
 * k_scales and v_scales, float32[num_blocks, num_kv_heads]; an element is its
 * E4M3 code times the scale of its block and head.
 *
 * kv_write_fp8_block writes the tokens that a prefill with the same
 * query_start_loc attends from: sequence s's last n_s = query_start_loc[s+1] -
 * query_start_loc[s] positions (a decode step: query_start_loc = 0, 1, 2, ...).
 * Query j of s is row query_start_loc[s] + j of key and value, at position
 * seq_lens[s] - n_s + j, in block block_tables[s][position / block_size]. For
 * each block that this touches, each head, and K and V each:
 *   s' = the least power of two with |x| <= 448 s' for the finite new values x
 *        of the block and head, at least 2^-60, and at least the block's
 *        present scale where the block holds earlier positions of s
 *   code = E4M3(x / s'), round to nearest even; NaN gives 0x7F, an infinity
 *        +-448
 *   where s' exceeds the present scale, the earlier positions' codes c become
 *        E4M3(c * scale / s'): exact unless that is below 2^-6
 * Present scales are powers of two, as this call writes them. A block that
 * holds no earlier position takes its scale from the new values alone, whatever
 * its entry held. Rows of the block past seq_lens[s] stay as
 * they are. A block may not be written for two sequences in one call (copy a
 * shared one first: kv_fork_blocks, kv_copy_blocks). A negative table entry
 * skips its positions, and positions below 0 or past the table are skipped. A
 * bad query_start_loc sets bit 2 of the fault word, a sequence longer than its
 * table bit 1; with bit 2 set, other sequences of the call may be skipped too.
 *   key, value   device bf16 rows at element strides key_stride, value_stride
 *                >= num_kv_heads * head_dim.
 * Supported: head_dim 64, 128 or 256; block_size a power of two in [16, 256];
 * code pools 16-byte aligned.
 * ---------------------------------------------------------------------- */
PAGEDKV_API int kv_write_fp8_block(const kv_bf16_t *key, const kv_bf16_t *value, kv_e4m3_t *k_cache_fp8,
                                   kv_e4m3_t *v_cache_fp8, float *k_scales, float *v_scales,
                                   const int32_t *block_tables, const int32_t *seq_lens,
                                   const int32_t *query_start_loc, uint32_t max_blocks_per_seq,
                                   uint32_t num_seqs, uint32_t num_tokens, uint32_t num_kv_heads,
                                   uint32_t head_dim, uint32_t block_size, uint32_t key_stride,
                                   uint32_t value_stride, void *stream);

/* Paged decode over that cache: as paged_decode_attn_fp8_sinks with each
 * position's K and V scaled by its block's scales, any finite scales in [2^-60,
 * 2^120]. head_dim 64, 128 or 256. */
PAGEDKV_API int paged_decode_attn_fp8_block(const kv_bf16_t *q, const kv_e4m3_t *k_cache_fp8,
                                            const kv_e4m3_t *v_cache_fp8, const float *k_scales,
                                            const float *v_scales, float *output, const int32_t *block_tables,
                                            const int32_t *seq_lens, uint32_t max_blocks_per_seq,
                                            uint32_t num_seqs, uint32_t num_q_heads, uint32_t num_kv_heads,
                                            uint32_t head_dim, uint32_t block_size, float inv_sqrt_d,
                                            uint32_t q_stride, uint32_t sliding_window, uint32_t num_sinks,
                                            void *stream);

/* Multi-token form over that cache: as paged_prefill_attn_fp8_sinks (BF16
 * rows out), with the block scales, of the same range. head_dim 64 or 128. */
PAGEDKV_API int paged_prefill_attn_fp8_block(const kv_bf16_t *q, const kv_e4m3_t *k_cache_fp8,
                                             const kv_e4m3_t *v_cache_fp8, const float *k_scales,
                                             const float *v_scales, kv_bf16_t *output, const int32_t *block_tables,
                                             const int32_t *seq_lens, const int32_t *query_start_loc,
                                             uint32_t max_blocks_per_seq, uint32_t num_seqs, uint32_t num_q_tokens,
                                             uint32_t num_q_heads, uint32_t num_kv_heads, uint32_t head_dim,
                                             uint32_t block_size, float inv_sqrt_d, uint32_t q_stride,
                                             uint32_t sliding_window, uint32_t num_sinks, void *stream);

/* ------------------------------------------------------------------------
 * Pages of a cache (not on the pages): copying, sharing on a fork, freeing and
 * compacting, all on device-resident block tables, with no host round trip.
 * ref_counts int32[num_blocks] holds the number of table entries that name
 * each block; a block whose count is 0 (or less) is free. Allocation takes the
 * free blocks with the lowest ids, so every result is a function of the inputs
 * alone. Ids
 * and rows are checked against num_blocks and num_seqs on the device: one out of
 * range is skipped and sets bit 4 of the fault word. The calls on one set of
 * tables and counts belong on one stream, or in an order of the caller's.
 *
 * kv_copy_blocks: for every pool p and pair i, block dst_blocks[i] of pool p
 * becomes a copy of block src_blocks[i]. A pair with a negative id is padding
 * (beside a negative source the destination is not looked at; a source out of
 * range sets bit 4 beside any destination).
 * No block may be the destination of two pairs, or of one and the source of
 * another.
 *   pools, block_bytes   HOST arrays of num_pools device base pointers and of
 *                        the bytes of one block in each (e.g. every layer's K
 *                        and V codes and their scales); read before the call
 *                        returns.
 *   src_blocks, dst_blocks   device int32[num_pairs].
 * ---------------------------------------------------------------------- */
PAGEDKV_API int kv_copy_blocks(void *const *pools, const size_t *block_bytes, uint32_t num_pools,
                               const int32_t *src_blocks, const int32_t *dst_blocks, uint32_t num_pairs,
                               uint32_t num_blocks, void *stream);

/* Entries [first_block[s], end_block[s]) of each row s become -1 and their
 * blocks' counts drop by one (rows with first >= end stay; the range is cut to
 * the table). An entry whose block's count is 0 already sets bit 4.
 *   block_tables int32[num_seqs, max_blocks_per_seq] and ref_counts, updated;
 *   first_block, end_block  device int32[num_seqs]. */
PAGEDKV_API int kv_free_blocks(int32_t *block_tables, int32_t *ref_counts, const int32_t *first_block,
                               const int32_t *end_block, uint32_t max_blocks_per_seq, uint32_t num_seqs,
                               uint32_t num_blocks, void *stream);

/* The same for the blocks that a window has left behind: those that hold
 * neither a sink nor a position at or past seq_lens[s] - sliding_window, which
 * no decode at this length or a later one, and no prefill of later tokens,
 * attends. sliding_window 0 frees nothing. A length past the table is cut to it,
 * as those calls cut it, and sets bit 1. */
PAGEDKV_API int kv_free_window_blocks(int32_t *block_tables, int32_t *ref_counts, const int32_t *seq_lens,
                                      uint32_t max_blocks_per_seq, uint32_t num_seqs, uint32_t num_blocks,
                                      uint32_t block_size, uint32_t sliding_window, uint32_t num_sinks,
                                      void *stream);

/* Row dst_seqs[i] becomes a fork of row src_seqs[i], for every i < num_forks:
 * the same length, the same full blocks (each counted once more; -1 entries
 * stay -1), and for a partly filled last block a free block of its own, with
 * the pair (copy_src[i], copy_dst[i]) to hand to kv_copy_blocks; (-1, -1)
 * where there is none. The free blocks go to the forks in order of i. The
 * destination rows must be free (released by kv_free_blocks): what they held
 * is overwritten, not released. Forks that write the same row are invalid, and so
 * is a fork that reads a row which a fork of this call names as its destination
 * (the one that names it is made all the same): an invalid fork (also: a row out
 * of range, a length past the table) sets bit 4, one that finds no free block
 * sets bit 5; either leaves its row as it was and gets the pair (-2, -2).
 *   block_tables, seq_lens int32[num_seqs], ref_counts (16-byte aligned)
 *   updated; src_seqs, dst_seqs device int32[num_forks]; copy_src, copy_dst
 *   device int32[num_forks], written.
 * Supported: num_seqs / 16 + num_forks up to 51,200 (shared memory of one CTA). */
PAGEDKV_API int kv_fork_blocks(int32_t *block_tables, int32_t *seq_lens, int32_t *ref_counts,
                               const int32_t *src_seqs, const int32_t *dst_seqs, int32_t *copy_src,
                               int32_t *copy_dst, uint32_t num_forks, uint32_t max_blocks_per_seq,
                               uint32_t num_seqs, uint32_t num_blocks, uint32_t block_size, void *stream);

/* With U blocks in use, the i-th lowest used block with an id >= U moves to the
 * i-th lowest free id below U, so that the blocks in use become 0 .. U-1. The
 * call writes the new tables and counts and the list of moves; kv_copy_blocks
 * moves the data (no source is a destination).
 *   new_tables, new_ref_counts  the tables and counts after the moves; each may
 *                be the input itself. An entry of block_tables that names a free
 *                block becomes -1 and sets bit 4.
 *   new_ids      device int32[num_blocks]: each block's new id (its own where
 *                it stays), -1 for a free one.
 *   copy_src, copy_dst  device int32[num_blocks / 2]: the moves in order, then
 *                (-1, -1).
 *   num_used     device int32[1]: U. */
PAGEDKV_API int kv_compact_blocks(const int32_t *block_tables, const int32_t *ref_counts, int32_t *new_tables,
                                  int32_t *new_ref_counts, int32_t *new_ids, int32_t *copy_src,
                                  int32_t *copy_dst, int32_t *num_used, uint32_t max_blocks_per_seq,
                                  uint32_t num_seqs, uint32_t num_blocks, void *stream);

/* ------------------------------------------------------------------------
 * Split-KV workspace (not on the pages: flash-decoding partials and the
 * combine step need scratch). The caller allocates device memory of at
 * least kv_decode_workspace_bytes(...) for the largest decode it will run
 * and registers it for the current device; NULL (or 0 bytes) unregisters.
 *
 * kv_decode_workspace_bytes takes the decode's table geometry
 * (max_blocks_per_seq, num_seqs, num_q_heads, num_kv_heads, head_dim,
 * block_size: the same values the decode call gets) rather than a split
 * count: the kernel cuts the tiles of all sequences (16 positions each),
 * taken in sequence order, into equal chunks, about one per SM, sized on
 * the device from the actual sequence lengths, and a sequence is split
 * where a chunk boundary falls inside it; a caller cannot know those splits
 * in advance. The size covers the worst case, a sequence as long as its
 * table allows (T = ceil(max_blocks_per_seq * block_size / 16) tiles) cut
 * by chunks of 16 tiles into P = (T <= 1 ? T : (T - 2) / 16 + 2) pieces
 * (integer division): 256 bytes of header, then num_seqs * num_kv_heads
 * 4-byte piece counts rounded up to a multiple of 256 bytes, then
 * num_seqs * P * num_q_heads * (head_dim + 2) * 4 bytes of partials. A
 * smaller registered workspace is still used, with longer chunks (or none
 * where it holds fewer than two pieces per sequence), and gives the same
 * results.
 * Decode calls on that device use it in stream order, so decode calls that
 * may run concurrently on different streams need separate devices or must be
 * ordered by the caller. The library never frees it.
 * ---------------------------------------------------------------------- */
PAGEDKV_API size_t kv_decode_workspace_bytes(uint32_t max_blocks_per_seq, uint32_t num_seqs,
                                 uint32_t num_q_heads, uint32_t num_kv_heads, uint32_t head_dim,
                                 uint32_t block_size);
PAGEDKV_API int kv_set_decode_workspace(void *device_ptr, size_t bytes);

/* ------------------------------------------------------------------------
 * Device-side fault word. Kernels that meet bad device data (a slot mapping
 * or table value they refuse to use, a pipeline wait that ran out of time)
 * skip the work, set a bit here and return instead of faulting or hanging.
 * kv_get_device_error synchronises the current device, returns the bits seen
 * since the last clear (0 = none) in *bits and clears them. Its status is
 * KV_ERR_DEVICE when any bit was set, KV_OK when none was, KV_ERR_CUDA when
 * the synchronisation or a read failed (*bits then unspecified) and
 * KV_ERR_INVALID_ARG for a null bits pointer. The other calls never
 * synchronise, so they cannot see these faults and never return
 * KV_ERR_DEVICE.
 *   bit 0: a decode pipeline wait timed out (that call's output is unspecified)
 *   bit 1: seq_lens[s] exceeded max_blocks_per_seq * block_size (clamped)
 *   bit 2: a prefill query_start_loc was decreasing, negative or past
 *          num_q_tokens (that sequence skipped)
 *   bit 3: (bounds-checking build only) a slot or block id outside the pool
 *          set by kv_debug_set_pool
 *   bit 4: a page call (kv_copy_blocks to kv_compact_blocks) met an id, a row
 *          or a count out of range (skipped)
 *   bit 5: kv_fork_blocks found no free block for a fork (not made)
 *   bit 6: a prefix plan that was made for other arguments (not used)
 *   (bits 1 and 2 also cover kv_write_fp8_block, bit 1 kv_free_window_blocks, bit 2
 *   kv_prefix_plan's group_start;
 *   bit 0 also covers the prefill pipeline and the waits of the fused K write and
 *   of the calls that rotate for their shared-memory copy of the sin/cos table)
 * ---------------------------------------------------------------------- */
PAGEDKV_API int kv_get_device_error(uint32_t *bits);

/* ------------------------------------------------------------------------
 * Bounds checking (a separate build of this library, compiled with
 * PAGEDKV_DEBUG_BOUNDS: libpagedkv_debug.so). Device data that index the
 * pools (slot mappings, block tables) are the caller's contract and go
 * unchecked in the product build. In the bounds-checking build every kernel
 * checks each slot against num_blocks * block_size and each block id
 * against num_blocks, as set here for the current device (num_blocks 0:
 * unchecked, the initial state). A write skips a row whose slot is out of
 * the pool; an attention call reads block 0 in place of a block id out of
 * the pool; either sets bit 3 of the fault word. Nothing traps. The call
 * synchronises. The product build returns KV_ERR_UNSUPPORTED.
 * ---------------------------------------------------------------------- */
PAGEDKV_API int kv_debug_set_pool(uint32_t num_blocks, uint32_t block_size);

/* Bounds-checking build only: how long each pipeline wait of the paged
 * decode kernels (a consumer waiting for a loaded tile, the loader waiting
 * for a free stage) may take on the current device before the kernel gives
 * up, sets bit 0 of the fault word and returns; 0 restores the default of
 * 2 s, which the product build always uses. Whatever the limit, a decode CTA
 * that gave up first waits (with the 2 s limit) until every copy it issued
 * into its shared memory has landed, so that nothing is left in flight.
 * The call synchronises. The product build returns KV_ERR_UNSUPPORTED. */
PAGEDKV_API int kv_debug_set_wait_limit(uint64_t nanoseconds);

/* Number of decode CTAs per SM and SM count the library launches with on the
 * current device, for benchmarks (optional outputs may be NULL). */
PAGEDKV_API int kv_device_info(int *num_sms, int *decode_ctas);

#ifdef __cplusplus
}
#endif
#endif /* PAGEDKV_H */
