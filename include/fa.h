/*
 * fa.h -- C ABI of the GB300 (sm_103a) tiled exact attention library.
 *
 * The operation is exact softmax attention for training, computed the way the
 * FlashAttention method does it:
 *
 *   forward  ("What Ordinary Autograd Saves: Tiling the Forward Pass Is Only
 *            Half the Algorithm", section "The implementation under test"):
 *            an online-softmax pass over key/value tiles that never forms the
 *            Tq x Tk score matrix and returns O and the per-row logsumexp L.
 *   backward ("What Ordinary Autograd Saves", section "Why this is
 *            FlashAttention's second idea"; "Backward Pass Implementation",
 *            section "The Recomputation Strategy"): keeps only O and L from the
 *            forward and rebuilds every score/probability tile on chip from Q,
 *            K and L, with D = rowsum(dO * O), dS = P * (dP - D),
 *            dV += P^T dO, dK += dS^T Q * scale, dQ += dS K * scale.
 *
 * Tensors (all row-major, contiguous, device memory, 16-byte aligned):
 *   Q, dQ   bf16 [B, Hq,  Tq, d]
 *   K, dK   bf16 [B, Hkv, Tk, d]
 *   V, dV   bf16 [B, Hkv, Tk, dv]
 *   O, dO   bf16 [B, Hq,  Tq, dv]
 *   L       fp32 [B, Hq,  Tq]   natural-log logsumexp of the scaled scores
 * Query head h reads key/value head h / (Hq / Hkv) (grouped-query attention in
 * the repeat_interleave order of "The Autograd Memory Trap", section "The GQA
 * Expansion Question"); Hq must be a multiple of Hkv.
 *
 * Masking: key j is visible to query i iff j < Tk and, when causal, also
 * j <= i + (Tk - Tq) (bottom-right alignment, the same as top-left when
 * Tq == Tk).  A causal sliding window of W >= 1 keys (the local-attention
 * layers of "The Autograd Memory Trap", section "Assumptions and
 * Uncertainties", item 3, which attend to a bounded number of keys) further
 * requires j > i + (Tk - Tq) - W: each row sees at most its last W keys.
 * A query row that sees no key gets O = 0, L = -inf, dQ = 0 and contributes
 * nothing to dK, dV.  A row with a NaN among the scores it sees gets O = L = NaN.
 *
 * Supported: d and dv each in {64, 128} (dv may differ from d).  Any B, Hq, Hkv, Tq, Tk >= 0 (ragged tails
 * are handled; a zero-sized problem is a no-op; Tk == 0 yields O = 0 and
 * L = -inf), up to size limits: Tq <= 65535 * 256, B * Hkv * ceil(Tk / 128)
 * < 2^31, B * Hq < 2^31 (beyond them FA_ERR_UNSUPPORTED).
 *
 * Ownership and execution: the caller allocates and frees every buffer,
 * including the backward workspace.  The library never allocates or frees
 * device memory and never synchronises the stream (fa_last_device_status
 * excepted); all work is enqueued on `stream` (a cudaStream_t, NULL for the
 * legacy default stream).  Inputs are read-only; outputs are fully overwritten.
 *
 * Errors: a bad argument returns FA_ERR_INVALID_ARG and an unsupported shape
 * FA_ERR_UNSUPPORTED, before anything is enqueued.  A CUDA launch or
 * tensor-map error returns FA_ERR_CUDA.  Every on-chip wait of the kernels is
 * bounded in time; if one gives up, the kernel stops, leaves its outputs
 * undefined and records FA_ERR_TIMEOUT in a device status word that
 * fa_last_device_status reports.
 */
#ifndef FA_GB300_H
#define FA_GB300_H

#include <stddef.h>

#if defined(__GNUC__)
#define FA_API __attribute__((visibility("default")))
#else
#define FA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1,
  FA_ERR_UNSUPPORTED = 2,
  FA_ERR_CUDA = 3,
  FA_ERR_TIMEOUT = 4,
  FA_ERR_SCRATCH_TOO_SMALL = 5
} fa_status;

typedef struct {
  int B, Hq, Hkv, Tq, Tk, d, dv;
  int causal; /* 0 or 1 */
  float scale; /* multiplies Q K^T; <= 0 selects 1/sqrt(d) */
  int window;  /* causal sliding window in keys; 0 = none; > 0 needs causal == 1 */
} fa_dims;

/* Forward pass: O = softmax(scale * Q K^T + mask) V, L = logsumexp rows.
 * Only O and L need to be kept for the backward pass. */
FA_API fa_status fa_forward(const fa_dims* dims, const void* Q, const void* K, const void* V, void* O, float* L,
                     void* stream);

/* Size in bytes of the scratch buffer for fa_backward's fastest schedule:
 * an fp32 dQ accumulator [B, Hq, ceil(Tq/128)*128, d] plus two fp32 row
 * vectors (D and log2-scaled L) of B*Hq*ceil(Tq/128)*128 entries, plus
 * alignment; without a causal mask also room for the partial dK / dV of up
 * to min(B*Hkv*ceil(Tk/128), 128) key tiles whose work may be split in two
 * (fp32, 2 x 128 x (d + dv) each) and a 4-byte counter per such tile.
 * Returns 0 for invalid dims. */
FA_API size_t fa_backward_workspace_bytes(const fa_dims* dims);

/* The least workspace fa_backward accepts: the dQ accumulator and the two
 * row vectors alone.  With less than fa_backward_workspace_bytes(dims) the
 * backward runs every key tile as one work item (same results, a slower
 * last round without a causal mask).  Equal to fa_backward_workspace_bytes
 * with a causal mask.  Returns 0 for invalid dims. */
FA_API size_t fa_backward_workspace_min_bytes(const fa_dims* dims);

/* Backward pass from O, L of fa_forward (same dims) and the upstream gradient
 * dO.  Writes dQ, dK, dV.  `workspace` must hold at least
 * fa_backward_workspace_min_bytes(dims) bytes (fa_backward_workspace_bytes
 * for the fastest schedule), 256-byte aligned; its contents on entry are
 * ignored. */
FA_API fa_status fa_backward(const fa_dims* dims, const void* Q, const void* K, const void* V, const void* O,
                      const void* dO, const float* L, void* dQ, void* dK, void* dV, void* workspace,
                      size_t workspace_bytes, void* stream);

/* The backward in separately launchable stages, for callers that interleave
 * other work or time the stages: bit 0 = preprocess (D = rowsum(dO * O), L in
 * log2 units, zero the dQ accumulator and the split-tile counters in
 * `workspace`), bit 1 = the main
 * recompute kernel (dK, dV, dQ accumulation), bit 2 = dQ cast.  Stages must run
 * in order on the same workspace; fa_backward is fa_backward_stages(..., 7). */
enum { FA_BWD_PRE = 1, FA_BWD_MAIN = 2, FA_BWD_CAST = 4, FA_BWD_ALL = 7 };
FA_API fa_status fa_backward_stages(const fa_dims* dims, const void* Q, const void* K, const void* V, const void* O,
                                    const void* dO, const float* L, void* dQ, void* dK, void* dV, void* workspace,
                                    size_t workspace_bytes, int stages, void* stream);

/* Backward pass for callers that cannot allocate device memory, such as code
 * running inside a host framework that passes it only its inputs and outputs
 * and owns every other byte of device memory, or a latency-critical loop that
 * must not call cudaMalloc.  Same arguments and results as fa_backward, but
 * no workspace: the scratch comes from a fixed array of
 * FA_NOALLOC_SCRATCH_BYTES that the library keeps in device memory on every
 * GPU that loads it, for the life of the process.  This entry point has no
 * counterpart on the pages; it is an interface convenience.
 *  - A problem whose fa_backward_workspace_min_bytes exceeds
 *    FA_NOALLOC_SCRATCH_BYTES is rejected with FA_ERR_SCRATCH_TOO_SMALL
 *    before anything is enqueued (use fa_backward for it); one that fits
 *    the minimum but not fa_backward_workspace_bytes runs unsplit.
 *  - Nothing is allocated or freed.  The first call on each device looks up
 *    the array's device address with that device current and keeps it for
 *    the life of the process; make that first call before any stream capture
 *    on the device.  Resetting the device (cudaDeviceReset) after that first
 *    call is not supported: the kept address would point into the destroyed
 *    context.  (The device status word behind fa_last_device_status is kept
 *    the same way.)
 *  - All calls on a device share the array.  Calls that may overlap on the
 *    GPU race on it; the caller must order them (e.g. one stream).  Stale
 *    contents from an earlier call are harmless: every part of the scratch the
 *    backward reads is rewritten (the dQ accumulator is zeroed) first. */
#define FA_NOALLOC_SCRATCH_BYTES (32u << 20)
FA_API fa_status fa_backward_noalloc(const fa_dims* dims, const void* Q, const void* K, const void* V,
                                     const void* O, const void* dO, const float* L, void* dQ, void* dK, void* dV,
                                     void* stream);

/* ---------------------------------------------------------------------------
 * Attention with modified scores.  Between the scaled product and the softmax
 *   x_ij = scale * q_i . k_j
 *   x_ij = softcap * tanh(x_ij / softcap)            softcap > 0
 *   x_ij = x_ij - slopes[h] * |i + (Tk - Tq) - j|    slopes given (fp32 [Hq])
 * in this order; L is the logsumexp of the modified scores.  The masks are those
 * above (causal, window, ragged ends), or those of a mask plan.  The gradients
 * go through the cap; the slopes are constants and have none.
 *
 * softcap is 0 (none) or between 2^-10 and 2^10; a capped score is off by at
 * most 2^-20 of the cap (fp32 arithmetic with one reciprocal for four scores),
 * which at 2^10 is half a step of a bf16 weight.  Slopes may have any sign; biases
 * are off by a few of fp32's roundings of their size, and L with them.  With
 * slopes, Tq and Tk are at most 2^24 (distances stay exact in fp32).  Everything
 * else is as for fa_forward / fa_backward: layouts, head sizes, empty rows,
 * workspace, errors.  Values at masked places have to be finite too (a masked
 * pair has weight 0, and 0 * NaN is NaN), and with a cap those of V are taken to be
 * below 2^20 in magnitude (the weights of a capped row, up to 2^90, are summed before
 * they are normalised).  fa_backward_noalloc has no form with modified scores. */
typedef struct {
  float softcap;
  const float* slopes; /* device, [Hq], or NULL */
  const void* plan;    /* device, written by fa_mask_plan for the same B, Tq, Tk, causal and window; or NULL */
} fa_scores;

/* A mask plan holds, for one batch of sequences, which keys each row sees, in
 * the form the kernels walk (per-row key intervals and per-tile ranges).  It
 * serves every layer, head and direction that has the same B, Tq, Tk, causal
 * and window; other fields of dims do not matter to it.
 *   doc_q int32 [B, Tq], doc_k int32 [B, Tk] (both or neither): row i sees key j
 *     only if doc_q[i] == doc_k[j]; negative ids (and 2^31 - 1) are padding, which
 *     sees nothing and is not seen.  Any order is served; key documents in
 *     ascending order (packed rows, padding last) are the fast case.
 *   prefix int32 [B], or [B, Tq] with prefix_per_row = 1; needs causal and no window: row i
 *     also sees the keys j < prefix, those after it among them.
 * With both, a key has to be in the row's document and causal or in the prefix.
 * The plan buffer has fa_mask_plan_bytes(dims) bytes, 16-byte aligned. */
FA_API size_t fa_mask_plan_bytes(const fa_dims* dims);
FA_API fa_status fa_mask_plan(const fa_dims* dims, const int* doc_q, const int* doc_k, const int* prefix,
                              int prefix_per_row, void* plan, size_t plan_bytes, void* stream);

/* fa_forward and fa_backward_stages with modified scores (scores NULL or all
 * zero: the same as those calls).
 * A forward of few query rows over many keys splits the keys over the SMs where it
 * is given a workspace (256-byte aligned, contents ignored) of at least
 * fa_forward_scored_workspace_bytes (0 where nothing is split; it asks the current
 * device for its SMs); with less, or NULL, it runs unsplit: same results up to
 * rounding, slower. */
FA_API size_t fa_forward_scored_workspace_bytes(const fa_dims* dims, const fa_scores* scores);
FA_API fa_status fa_forward_scored(const fa_dims* dims, const fa_scores* scores, const void* Q, const void* K,
                                   const void* V, void* O, float* L, void* workspace, size_t workspace_bytes,
                                   void* stream);
/* Workspace for fa_backward_scored's fastest schedule on the current device (room
 * for the partial sums of split work items); the least that it accepts is
 * fa_backward_workspace_min_bytes(dims).  0 for invalid arguments. */
FA_API size_t fa_backward_scored_workspace_bytes(const fa_dims* dims, const fa_scores* scores);
FA_API fa_status fa_backward_scored(const fa_dims* dims, const fa_scores* scores, const void* Q, const void* K,
                                    const void* V, const void* O, const void* dO, const float* L, void* dQ, void* dK,
                                    void* dV, void* workspace, size_t workspace_bytes, int stages, void* stream);

/* Rotary positions of Q and K, the step before the attention, with one to four
 * position axes (one for text; time, height and width for images and video).
 *   bf16 Q, Qo [B, Hq, T, d] and K, Ko [B, Hk, T, d] with the given strides (in
 *   elements; batch, head, token; channels contiguous).  The inputs may be
 *   views of a packed projection.  Qo / Ko may be Q / K themselves (same
 *   strides), and otherwise must not overlap them.
 *   positions: int32 or int64 (pos_bytes 4 or 8), entry (a, b, t) at
 *   a * pos_axis_stride + b * pos_batch_stride + t; any value, also negative.
 *   inv_freq: fp32 [rot / 2], radians per position step, |inv_freq| <= 1 for
 *   full accuracy (each further factor of two costs one bit of the angle's 64).
 * Frequency f belongs to the axis whose section holds it (section[0] frequencies
 * of axis 0, then section[1] of axis 1, ...; the sections add up to rot / 2)
 * and turns its channel pair by positions[axis][b][t] * inv_freq[f]:
 *   (x, y) -> (x cos - y sin, y cos + x sin).
 * Pair f is channels (f, f + rot / 2), or (2 f, 2 f + 1) with interleaved = 1;
 * channels rot .. d-1 are copied.  inverse = 1 turns back, which is the gradient:
 * it takes dQo, dKo to dQ, dK.  d is 64 or 128, rot a multiple of 16 up to d.
 * Pointers are 16-byte aligned and strides multiples of 8 elements.  Hk = 0 (or
 * Hq = 0) leaves K (or Q) out. */
typedef struct {
  int B, Hq, Hk, T, d, rot, axes, interleaved, pos_bytes;
  int section[4];
  long long q_stride[3], k_stride[3], qo_stride[3], ko_stride[3];
  long long pos_axis_stride, pos_batch_stride;
} fa_rotary_dims;
FA_API fa_status fa_rotary(const fa_rotary_dims* dims, const void* Q, const void* K, const void* positions,
                           const float* inv_freq, void* Qo, void* Ko, int inverse, void* stream);

/* Static description of a status code. */
FA_API const char* fa_status_string(fa_status s);

/* Synchronises `stream`, then reports (and clears) the device status word:
 * FA_ERR_TIMEOUT if a kernel gave up waiting since the last call, FA_ERR_CUDA
 * if the stream holds an asynchronous CUDA error, FA_OK otherwise. */
FA_API fa_status fa_last_device_status(void* stream);

/* Number of kernel launches the last call of fa_forward, fa_backward (any form of
 * them) or fa_mask_plan on this host thread enqueued (for launch accounting). */
FA_API int fa_last_launch_count(void);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_H */
