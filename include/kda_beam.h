/*
 * kda_beam.h -- C ABI of the steps that several continuations of one prompt
 * need beside the KDA token step (kda.h) and paged softmax attention
 * (kda_attn.h): beam search, and samples that take over one another's state.
 *
 *   kda_beam_select   the best continuations of every group of beams
 *   kda_beam_reorder  S and conv windows of the sequences that were chosen
 *
 * The pages of the key/value cache follow with kda_attn_fork.  The rows that
 * kda_beam_select returns are what kda_beam_reorder and kda_attn_fork take.
 *
 * Conventions are those of kda.h: device pointers, work on the caller's stream,
 * no allocation and no synchronisation per call, arguments checked on the host
 * before any launch, KDA_FAULT_INJECT (names "beam_select", "beam_reorder";
 * "all" includes them).
 */
#ifndef KDA_BEAM_H
#define KDA_BEAM_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most beams of a group, and most continuations returned for one. */
#define KDA_BEAM_MAX_BEAMS 64
#define KDA_BEAM_MAX_NUM 64

/* Bytes of device workspace of kda_beam_select; 0 for sizes that it refuses. */
KDA_API size_t kda_beam_select_workspace_bytes(const kda_ctx *ctx, int groups, int beams, int vocab, int num);

/*
 * Of each group of beams, the num best continuations.  Beam k of group g, row
 * r = g * beams + k of the logits, goes on with token v at the score
 *     scores[g][k] + logits[r][v] - ln(sum over v' of exp(logits[r][v'])),
 * and the num highest of a group's beams * vocab scores are returned, highest
 * first, of equal ones those of the lower beam, then of the lower token, first.
 * A score that is NaN (a row with a NaN or +infinite logit, or whose logits are
 * all -infinity) counts as -infinity.  Scores of different beams are compared in
 * 64 bits, those of one beam as its logits are: the larger logit has the higher score
 * also where 64 bits hold the two for equal (beyond scores[g][k] of 1e9 or so).  The sums
 * of a row's num largest terms are taken in 64 bits too, those of its other terms
 * in fp32.
 *   logits    [groups * beams][vocab] fp32, or bf16 if logits_bf16 is nonzero,
 *             rows row_stride elements apart (>= vocab); aligned to their type
 *   scores    [groups][beams] fp32: what the beams have gathered so far.  At the
 *             first step of a search, whose beams are alike, 0 for one of them and
 *             -infinity for the others
 *   done      [groups][beams] bytes or NULL: nonzero where a beam has come to its
 *             end.  It goes on with end_token alone, at the score that it has; its
 *             logits are not read
 *   num       1 to 64, at most beams * vocab
 *   keep_places  nonzero (with num == beams): the beams that go on keep their
 *             places, so that no state moves that need not.  A beam's best chosen
 *             continuation comes to place k, its own; the others, highest first, to
 *             the places that are left, lowest first.  rows[rows[b]] == rows[b] then
 *             holds, which in-place reordering wants
 *   out_scores [groups][num] fp32, out_tokens [groups][num] int32,
 *   out_rows   [groups][num] int32: r of the beam that goes on
 *   workspace kda_beam_select_workspace_bytes bytes, 16-byte aligned
 * fp32 and int32 arrays are 4-byte aligned; no output may overlap an input.  groups == 0
 * is a no-op.  beams from 1
 * to 64 (more, or a larger num: KDA_ERR_UNSUPPORTED), beams * vocab below 2^31,
 * groups * beams up to 2^30.  The result does not depend on the order in which
 * parts of the work end.
 */
KDA_API kda_status kda_beam_select(kda_ctx *ctx, int groups, int beams, int vocab, const void *logits,
                                   int logits_bf16, long long row_stride, const float *scores,
                                   const uint8_t *done, int end_token, int num, int keep_places,
                                   float *out_scores, int32_t *out_tokens, int32_t *out_rows,
                                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * Sequence b goes on from sequence rows[b]: S_out[b] = S[rows[b]] and
 * conv_out[b] = conv_state[rows[b]], for b = 0 .. B - 1.
 *   rows       [B] int32, 4-byte aligned: 0 .. B - 1, or -1: that sequence is left
 *              as it is.  Any other value is an error: the sequence is left as it
 *              is, and kda_sync_status reports KDA_ERR_INVALID_ARG.
 *   S, S_out   [B][H][d][d] fp32, or bf16 if s_bf16 is nonzero
 *   conv_state, conv_out  [B][3][3*H*d] fp32
 * Either S_out == S and conv_out == conv_state (in place: a sequence that another
 * one goes on from has to stay, rows[rows[b]] == rows[b], as keep_places arranges
 * it; one that goes on from a sequence that does not is an error as above, and only
 * sequences with rows[b] != b move), or neither overlaps its input.  Rows are copied
 * bit by bit.  B == 0 is a no-op.
 */
KDA_API kda_status kda_beam_reorder(kda_ctx *ctx, int B, const int32_t *rows, const void *S,
                                    const float *conv_state, void *S_out, float *conv_out, int s_bf16,
                                    void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_BEAM_H */
