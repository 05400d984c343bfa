/*
 * gbattn_rotary.h -- C ABI of rotary positions (sm_103a), beside gbattn.h.
 *
 * Pair i < rot_dim / 2 of a head's first rot_dim values, of a token at
 * position t, is turned by the angle a = t * f_i:
 *     (x, y) -> gain * (x cos a - y sin a, x sin a + y cos a)
 * with (x, y) at i and i + rot_dim / 2 (half layout) or at 2 i and 2 i + 1
 * (interleaved).  The rest of the head stays as it is.
 *
 * The frequencies are held as `steps`: f_i / 2 pi modulo 1 in units of 2^-64
 * turns, made once on the host (attn_rotary_frequencies, attn_rotary_steps)
 * and copied to the device by the caller.  The angle of any 32-bit position,
 * negative ones included, is then reduced exactly; it is off by what f_i / 2 pi
 * was rounded by (2^-52 of it) times t.
 *
 * Conventions are those of gbattn.h (ownership, streams, errors, dev_status,
 * head sizes), and:
 *  - q, k, v are bf16 [num_tokens, heads, D]; a token's [heads, D] is
 *    contiguous, token t at t * stride elements (parts of a fused projection).
 *    Strides are multiples of 8 and at least heads * D.
 *  - an output may be its input (the same pointer and stride); else outputs
 *    must not overlap the inputs or each other (GBATTN_ERR_INVALID_ARG).  Parts
 *    of one buffer that lie between one another have the same token stride.
 *  - products and cosines are fp32, rounded once to bf16.
 */
#ifndef GBATTN_ROTARY_H
#define GBATTN_ROTARY_H

#include "gbattn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * How frequencies change for contexts longer than the trained length L, by a
 * factor s >= 1 (f_i = base^(-2 i / rot_dim) before).
 */
typedef enum {
    GBATTN_ROTARY_PLAIN = 0,
    GBATTN_ROTARY_LINEAR = 1,   /* f / s */
    GBATTN_ROTARY_NTK = 2,      /* base * s^(rot_dim / (rot_dim - 2)) in base's place */
    GBATTN_ROTARY_BY_PARTS = 3, /* g f + (1 - g) f / s, g = clamp((L f / 2 pi - low) / (high - low), 0, 1):
                                   by the turns that a pair makes over L */
    GBATTN_ROTARY_YARN = 4      /* the same with g falling from 1 to 0 in equal steps of i from floor(i(high)) to
                                   ceil(i(low)), i(r) = rot_dim ln(L / 2 pi r) / (2 ln base) being the pair that
                                   makes r turns over L (the ends kept within [0, rot_dim - 1] and 0.001 apart at
                                   least); gain = 0.1 ln s + 1 (YaRN, Peng et al. 2023) */
} gbattn_rotary_scaling;

/*
 * attn_rotary_frequencies -- host function: f_i of a head, rot_dim / 2
 * doubles, and the gain (1 but for YARN).
 *   base    > 1
 *   factor  s >= 1 (unused by PLAIN); low, high, length: turns 0 < low < high
 *           and L > 0 (BY_PARTS and YARN only)
 * Errors: GBATTN_ERR_INVALID_ARG (null output, rot_dim odd or below 2, NTK with
 * rot_dim 2, numbers out of range or not finite), GBATTN_ERR_UNSUPPORTED
 * (unknown scaling).
 */
gbattn_status attn_rotary_frequencies(int rot_dim, double base, gbattn_rotary_scaling scaling, double factor, double low,
                                      double high, double length, double* inv_freq, double* gain);

/*
 * attn_rotary_steps -- host function: steps[i] = frac(inv_freq[i] / 2 pi) * 2^64
 * rounded, for n frequencies (finite; a negative one turns the other way).
 * Errors: GBATTN_ERR_INVALID_ARG.
 */
gbattn_status attn_rotary_steps(const double* inv_freq, int n, uint64_t* steps);

/*
 * attn_rotary -- turn queries and keys.
 *   q, k        device bf16 [num_tokens, Hq (Hkv), D] with token strides; k and
 *               k_out may be NULL with Hkv = 0
 *   positions   device int32 [num_tokens]
 *   steps       device uint64 [rot_dim / 2], 8-byte aligned
 *   rot_dim     even, 2 <= rot_dim <= D
 *   interleaved, transpose: 0 or 1.  transpose turns by -a: of gradients,
 *               dx = gain * R(-a) dy for y = gain * R(a) x
 *   gain        finite
 * num_tokens = 0 does nothing; the pointers may then be NULL.
 * Errors: GBATTN_ERR_INVALID_ARG, GBATTN_ERR_UNSUPPORTED (head size, rot_dim,
 * num_tokens >= 2^30, (Hq + 2 Hkv) * D >= 2^30), GBATTN_ERR_ALIGNMENT (a
 * tensor or a stride off 16 bytes), GBATTN_ERR_DEVICE / GBATTN_ERR_CUDA.
 */
gbattn_status attn_rotary(const void* q, long long q_stride, const void* k, long long k_stride, const int32_t* positions,
                          int num_tokens, const uint64_t* steps, int rot_dim, int interleaved, int transpose, float gain,
                          int Hq, int Hkv, int D, void* q_out, long long q_out_stride, void* k_out,
                          long long k_out_stride, void* stream);

/*
 * attn_rotary_kv_cache_write -- attn_rotary of the queries, and
 * attn_kv_cache_write of the turned keys and of the values, in one pass: what
 * a serving step does between its projection and attn_fwd_paged or
 * attn_fwd_paged_prefill.
 *   q, key, value, positions, steps, rot_dim, interleaved, gain, q_out
 *               as for attn_rotary (Hkv >= 1)
 *   slot_mapping, kv_cache, num_blocks, block_size
 *               as for attn_kv_cache_write; a token with a negative slot is
 *               not stored (its queries are turned), a slot past the cache
 *               is skipped and sets GBATTN_DEV_BAD_INDEX.  Slots are to be
 *               distinct: of one given twice, parts of different tokens may
 *               be stored.
 * Errors as for attn_rotary, and those of attn_kv_cache_write's cache.
 */
gbattn_status attn_rotary_kv_cache_write(const void* q, long long q_stride, const void* key, long long key_stride,
                                         const void* value, long long value_stride, const int32_t* positions,
                                         const int32_t* slot_mapping, int num_tokens, const uint64_t* steps, int rot_dim,
                                         int interleaved, float gain, void* q_out, long long q_out_stride,
                                         void* kv_cache, int num_blocks, int block_size, int Hq, int Hkv, int D,
                                         uint32_t* dev_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GBATTN_ROTARY_H */
