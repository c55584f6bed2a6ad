/*
 * kda_linear.h - C ABI of linear attention with a decay per head, on the slot
 * cache of kda.h.
 *
 * The operation. The recurrent state of kda.h without the delta rule, and with
 * one decay for a head's whole state: per head, with S a dk x dv matrix, one
 * token applies
 *     S <- a S + k v^T ;   o = S^T q
 * with a a scalar. a is either fixed per head or given per token and head.
 *
 * Layouts. As in kda.h: the cache is float, slot s at cache + s * slot_stride,
 * laid out [H][dv][dk], so kda_state_pack and kda_state_unpack move these
 * states too, and a slot id < 0 marks a padding row. The token inputs come with
 * a stride between tokens, so they can be slices of one projection's output:
 *   q, k    bf16   token t's heads at q + t * q_stride, laid out [Hk][dk]
 *   v       bf16   token t's heads at v + t * v_stride, laid out [H][dv]
 *   alpha   float  token t's decays at alpha + t * alpha_stride, laid out [H];
 *                  alpha_stride = 0: the same decays for every token
 *   out     float  [rows][H][dv], contiguous, 16-byte aligned (with KDA_OUT_BF16
 *                  bf16, 8-byte aligned): stricter than kda.h's, KDA_ERR_ALIGN
 * Hk divides H: heads h of H / Hk consecutive ones share key head h / (H / Hk).
 * q is used as given: any 1/sqrt(dk) scale is the caller's.
 *
 * Decays are meant to lie in [0, 1]; a = 0 forgets the state. They are only
 * ever multiplied (no logarithm, no division), so any finite value gives what
 * the formula gives as long as its products stay in fp32 range. A NaN or an
 * infinity among a row's inputs or in its state reaches outputs and states of
 * that row and head only (in kda_lin_prefill also outputs of up to 63 earlier
 * tokens of the row, and an infinity can become a NaN there).
 *
 * Supported shapes: dk, dv in {64, 128}; any H, Hk >= 1 with Hk dividing H. A
 * call whose grid would pass 2^31 workgroups or 2^32 threads is refused
 * (KDA_ERR_UNSUPPORTED); one of fewer than 2^20 (row, head) pairs fits.
 *
 * Ownership, ordering, errors and device errors are those of kda.h: the library
 * allocates nothing, never synchronizes, and enqueues on `stream`, which must
 * belong to the current device. Options: tile_w as stated per call; flags
 * KDA_OUT_BF16 and KDA_CHECK_SLOTS; KDA_RAW_INPUTS is KDA_ERR_UNSUPPORTED;
 * verify_form must be 0 (KDA_ERR_INVALID).
 */
#ifndef KDA_LINEAR_H
#define KDA_LINEAR_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Token inputs. Host struct; pointers are device memory. q, k and v are 16-byte
 * aligned with strides that are multiples of 8 (KDA_ERR_ALIGN), alpha is 4-byte
 * aligned. q_stride and k_stride are at least Hk * dk, v_stride at least H * dv,
 * alpha_stride 0 or at least H (KDA_ERR_INVALID); none of them, nor H * dv, is
 * above 2^24 (KDA_ERR_UNSUPPORTED). */
typedef struct kda_lin_tokens {
    const uint16_t *q, *k, *v;
    const float *alpha;
    int64_t q_stride, k_stride, v_stride, alpha_stride;
    int32_t Hk;
} kda_lin_tokens;

/*
 * Single-token step for B rows: row b reads token b, updates the state of slot
 * slot_ids[b] in place (all H heads) and writes out[b]. With epi the output
 * gate of kda.h is applied (gate bf16 [B][H][dv], contiguous, 8-byte aligned). Slot ids must be
 * distinct. tile_w: 0 or one of 4, 8, 16, 32, 64, 128 with tile_w <= dv (and
 * tile_w == dv with the gate); results are bit-identical for every width.
 */
int kda_lin_decode_step(float *cache, int64_t num_slots, int64_t slot_stride, const int32_t *slot_ids,
                        int32_t B, int32_t H, int32_t dk, int32_t dv, const kda_lin_tokens *x, void *out,
                        const kda_epilogue *epi, int32_t *dev_err, const kda_options *opts, void *stream);

/*
 * Packed prompts: row b runs tokens [cu_seqlens[b], cu_seqlens[b+1]) of n_tok
 * (any length, 0 included) from the state in its slot; out gets every token's
 * read-out and the slot the final state. Slot ids must be distinct. Tokens of out outside every row keep
 * their contents. ckpt_pos, ckpt: as for kda_prefill (the state after the first
 * ckpt_pos[b] tokens to ckpt[b], 0 = before the prompt, < 0 = none; past the
 * row is KDA_DEVERR_CKPT). Outputs and states agree with successive
 * kda_lin_decode_step calls to fp32 rounding (states, decayed scores and decayed
 * tokens enter products to 2^-133, which cuts bits off those below 2^-109); with
 * KDA_OUT_BF16 each output is the fp32 one rounded to nearest even. tile_w must be 0.
 * workspace: device memory of at least kda_lin_prefill_workspace() bytes,
 * 16-byte aligned (NULL where that is 0), not shared by calls that may overlap;
 * its contents need no initialization and are dead when the stream has passed
 * the call. Smaller is KDA_ERR_INVALID.
 */
int kda_lin_prefill(float *cache, int64_t num_slots, int64_t slot_stride, const int32_t *slot_ids,
                    const int32_t *cu_seqlens, int32_t B, int32_t n_tok, int32_t H, int32_t dk, int32_t dv,
                    const kda_lin_tokens *x, void *out, const int32_t *ckpt_pos, float *ckpt,
                    void *workspace, size_t workspace_bytes, int32_t *dev_err, const kda_options *opts,
                    void *stream);

/* Host only. Workspace bytes kda_lin_prefill needs for these sizes (to *bytes): never less for a larger B or
 * n_tok, so that a buffer for the largest call serves the smaller ones, and at most 1024 states of dk x dv with a
 * decay each (64 MiB and 4 KiB at 128 x 128). */
int kda_lin_prefill_workspace(int32_t B, int32_t n_tok, int32_t H, int32_t dk, int32_t dv, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* KDA_LINEAR_H */
