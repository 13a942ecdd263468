/*
 * sa.h -- C ABI of libsa.so, a B200 (sm_100a) SageAttention-style low-bit attention
 * forward with optional SLA-style block sparsity.
 *
 * The method (sources, by page and section):
 *   - "AIGC weekend special 5.10: full-stack optimisation of visual-generation
 *     inference", section 1 (TurboDiffusion), 1.2 Method, item (1): SageAttention2++
 *     quantises Q and K to low bit and runs Q.K^T on tensor cores; item (2): SLA
 *     sparse attention is orthogonal to it and runs on top of it.
 *   - "Video-Generation-101: inference systems", kernel paragraph and reference [3]:
 *     format / thread-granularity / accumulation co-design with outlier smoothing.
 *   - "Video-Generation-101 research log", section 5.5 table: INT4/INT8 Q.K^T with
 *     FP8/FP16 P.V.
 *   - NetEase article on the TurboDiffusion release, "attention acceleration" section
 *     and the SLA figure caption: only the critical blocks of the attention weights
 *     get exact (sparse) attention.
 * Numerical definition implemented (the pages give the outline; each detail they leave
 * open is stated here):
 *   per (b,h): mean_k[c] = fp32( sum_t K[t,c] (fp64) / N );
 *   Q: per 128-token block, scale_q = max|q| / 127, q_i8 = rint_even(q / scale_q);
 *   K: ks = K - mean_k (fp32), per 64-token block scale_k = max|ks| / 127,
 *      k_i8 = rint_even(ks / scale_k); codes clamp to [-127, 127]; zero block -> scale 0;
 *   V: per channel scale_v = max_t |v| / 448, v_fp8 = e4m3_rn_satfinite(v / scale_v);
 *   S = q_i8 . k_i8^T exact in int32; s = S * (scale_q * scale_k * sm_scale);
 *   online softmax in fp32 over the kept 64-key blocks, two blocks per step;
 *   p8 = e4m3(448 * exp(s - m)); l = sum of p8; acc = sum p8 * v_fp8 (fp32);
 *   O = acc * scale_v / l (bf16), 0 for a row with no kept key.
 *
 * Conventions for every entry point:
 *   - Tensors are contiguous row-major.  q, k, v, o: bf16 [B,H,N,d].  d must be 128, except
 *     that sa_attn_fwd and sa_attn_fwd_causal also take d = 64: they zero-pad q, k, v to 128
 *     channels in the workspace and copy out o's first 64, which gives exactly the d = 64
 *     definition (zero channels add nothing to S and leave every scale and code unchanged).
 *     Npad = 128 * ceil(N/128); nq = ceil(N/128); nk = ceil(N/64).  B * H <= 65535 (the
     heads are a grid dimension of the prologue kernels), else SA_ERR_UNSUPPORTED.
 *   - Device pointers are owned by the caller; the library never frees them.  All
 *     pointers must be 16-byte aligned.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).  Every
 *     call only enqueues work on that stream and returns without synchronising, except
 *     sa_get_device_status, which synchronises the device.
 *   - Argument errors are detected on the host before any launch; outputs are then
 *     untouched.  Launch failures return SA_ERR_CUDA.  Device-side bounded waits that
 *     expire set a device status word read by sa_get_device_status, and so do
 *     page numbers, lengths and offsets in device memory that are out of range (see the
 *     cache calls, which skip what they would have reached).
 *   - Block mask: uint8 [B,H,nq,nk], nonzero keeps the (128-query x 64-key) block; NULL
 *     keeps every block.  Masked blocks are neither loaded nor computed.  With a mask,
 *     nk <= 16384 (N <= 1,048,576), else SA_ERR_UNSUPPORTED.
 *   - Library workspace.  The entry points marked "uses the library workspace" keep their
 *     intermediates (quantised Q/K/V, scales, partial sums, masks, SLA states) in ONE
 *     buffer per device, owned by the library and grown on demand.  Growing it
 *     synchronises the device and frees the old buffer; the library holds a lock from a
 *     call's workspace request until that call's launches are enqueued, so calls from
 *     several host threads cannot free memory another call is about to use.  The buffer
 *     is NOT per stream: two such calls in flight at once on different streams of one
 *     device overwrite each other's intermediates and give wrong results without any
 *     error.  Order such calls on one stream (or with events).  sa_attn_fwd_quantized,
 *     sa_debug_qk_s32 and sa_w8a8_gemm use no workspace; sa_quantize_qk_noalloc uses its
 *     own fixed array (see there).
 *   - The library caches per-device state (the workspace, tensor-map encoder, kernel
 *     attributes and the scratch array's address) for the life of the process: do not use
 *     it across cudaDeviceReset.
 */
#ifndef SA_H
#define SA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SA_OK = 0,
    SA_ERR_INVALID_ARG = 1,    /* null pointer, non-positive size, size overflow */
    SA_ERR_UNSUPPORTED = 2,    /* d != 128, B * H > 65535, or no sm_100 device */
    SA_ERR_MISALIGNED = 3,     /* a pointer is not 16-byte aligned */
    SA_ERR_CUDA = 4,           /* a CUDA runtime/driver call or launch failed */
    SA_ERR_OOM = 5,            /* the library workspace could not be allocated */
    SA_ERR_DEVICE_TIMEOUT = 6, /* a device-side bounded wait expired */
    SA_ERR_SCRATCH_LIMIT = 7,  /* the problem needs more than a fixed scratch array holds */
    SA_ERR_BAD_INDEX = 8       /* a page, length or offset read on the device is out of range */
} sa_status;

/* Quantise Q and smooth + quantise K (the Q/K half of the prologue).
 * Sources: TurboDiffusion digest 1.2(1) (Q/K to INT8 on tensor cores);
 * Video-Generation-101 reference [3] (outlier smoothing).
 * Outputs (device, caller-owned):
 *   q_i8 int8 [B,H,Npad,d] (rows >= N zero), q_scale fp32 [B,H,nq],
 *   k_i8 int8 [B,H,Npad,d] (rows >= N zero), k_scale fp32 [B,H,nk],
 *   k_mean fp32 [B,H,d].
 * Results are bit-identical to the definition above (the K mean whenever the fp64 sum
 * of the column is exact, which holds for bf16 inputs of ordinary range).
 * Uses the library workspace for per-block fp64 partial sums of K. */
sa_status sa_quantize_qk(const void *q, const void *k, int B, int H, int N, int d,
                         int8_t *q_i8, float *q_scale, int8_t *k_i8, float *k_scale,
                         float *k_mean, void *stream);

/* sa_quantize_qk without any device allocation.  The method's pages have no counterpart
 * for this; it exists for callers that cannot call cudaMalloc: code whose device memory is
 * owned by a host framework or memory pool that has already reserved the device (so a
 * library allocation would fail or fragment it), and latency-critical loops that cannot
 * afford cudaMalloc's implicit synchronisation.  The library workspace that sa_quantize_qk
 * grows on first use is replaced by a fixed 4 MiB device array compiled into the library
 * (each GPU that loads the library holds it until the process exits).
 * Arguments, outputs and results are exactly those of sa_quantize_qk.
 * Limit: B * H * ceil(N / 1024) <= 4096 (e.g. 40 heads of up to 104,448 tokens); larger
 * problems return SA_ERR_SCRATCH_LIMIT before any launch.
 * The first call on each device looks up the array's device address (a synchronous
 * runtime call), so make that first call before any stream capture.  All calls share the
 * array: calls whose kernels overlap on the same device (e.g. on two streams) race on it
 * and must be ordered by the caller.  No state carries over between calls. */
sa_status sa_quantize_qk_noalloc(const void *q, const void *k, int B, int H, int N, int d,
                                 int8_t *q_i8, float *q_scale, int8_t *k_i8, float *k_scale,
                                 float *k_mean, void *stream);

/* Quantise V to FP8 e4m3 per channel, stored transposed (the V half of the prologue).
 * Source: Video-Generation-101 research log 5.5 (FP8 P.V).
 * Outputs: v_fp8_t uint8 e4m3 [B,H,d,Npad] (keys contiguous, keys >= N zero),
 *          v_scale fp32 [B,H,d].  Bit-identical to the definition above.
 * Uses the library workspace for per-channel maxima. */
sa_status sa_quantize_v(const void *v, int B, int H, int N, int d, uint8_t *v_fp8_t,
                        float *v_scale, void *stream);

/* Full forward: prologue into the library workspace, then the fused attention kernel.
 * Sources: all of the above; FlashAttention tiling (digest timeline, 2022.06) for the
 * online softmax.  o: bf16 [B,H,N,d] (device, caller-owned).  sm_scale: the logit scale,
 * normally 1/sqrt(d).  block_mask: see conventions, or NULL.
 * The workspace is library-owned, per device, grow-only (cudaMalloc on first use or
 * growth, so the first call at a new size must not be inside a stream capture). */
sa_status sa_attn_fwd(const void *q, const void *k, const void *v, void *o, int B, int H,
                      int N, int d, float sm_scale, const uint8_t *block_mask, void *stream);

/* Causal forward: as sa_attn_fwd, where query row r attends to the keys t <= r only.
 * Source: "AIGC weekend special 5.10", sections 4 (HiAR: causal generation over all blocks
 * at each denoising step) and 6 (SDVG: autoregressive video diffusion).  Reading: the
 * quantisation is unchanged (scales over all N tokens); a tile of 128 queries visits its
 * kept blocks j <= 2i + 1 in pairs, as without causality, and keys after the row are left
 * out of the max and the sums.  block_mask (or NULL) is intersected with the causal
 * block pattern.  Uses the library workspace (plus nq * nk bytes per head for the mask). */
sa_status sa_attn_fwd_causal(const void *q, const void *k, const void *v, void *o, int B, int H, int N,
                             int d, float sm_scale, const uint8_t *block_mask, void *stream);

/* Variable-length batch: nseq independent sequences of lengths seqlens[i] (host array,
 * each >= 1), packed back to back: sequence i is a [1, H, N_i, d] bf16 block of q, k, v
 * and o starting H * (N_0 + ... + N_{i-1}) * d elements in.  Each sequence is computed as
 * sa_attn_fwd (causal = 0) or sa_attn_fwd_causal without a mask (causal != 0) would compute
 * it alone, with the same results.  Every block must start 16-byte aligned (H * N_i * d is a
 * multiple of 8 elements, which d = 128 guarantees).  All sizes are checked before the first
 * launch.  The sequences are taken longest first in groups: a group takes the next sequence
 * while its heads padded to its longest stay within twice their own padded size, or below
 * 2^20 padded token-heads; each group is one prologue and one attention launch (the kernels
 * read every head's own length from a table), so a batch of short sequences is a single
 * launch of each kernel.  The workspace is sized for the largest group, plus the table,
 * which is uploaded through a library-owned page-locked host buffer. */
sa_status sa_attn_fwd_varlen(const void *q, const void *k, const void *v, void *o, int nseq, const int *seqlens,
                             int H, int d, float sm_scale, int causal, void *stream);

/* Debug (host only, no CUDA call): the groups sa_attn_fwd_varlen forms for these lengths.
 * group_of[i] (host array of nseq) receives the group of sequence i; groups are numbered
 * in launch order (longest sequences first).  Returns the number of groups, or -1 on bad
 * arguments (nseq < 1, H < 1, a null pointer or a length < 1). */
int sa_debug_varlen_groups(int nseq, const int *seqlens, int H, int *group_of);

/* Full forward on HOST buffers: q, k, v, o bf16 [B,H,N,d] and block_mask (or NULL) in host
 * memory, page-locked for the copies to overlap (pageable memory works but serialises).
 * The B*H heads are independent, so they are processed in chunks of consecutive heads
 * (one head first, then growing by one head per chunk up to about 64 MB of q, so that the
 * first upload, which nothing overlaps, is short): the upload of chunk c+1 and the
 * download of chunk c-1 run on two library-owned streams while chunk c runs sa_attn_fwd's
 * prologue and kernel on `stream`.  The call returns after enqueueing; the work is
 * complete when `stream` reaches the point after the call (o is then filled), and q, k,
 * v, o and block_mask must stay valid until then.  Device staging (two chunks) is
 * library-owned, per device and grow-only, like the workspace.  Calls for the same device
 * from several host threads are serialised.  Results are identical to sa_attn_fwd on the
 * same inputs. */
sa_status sa_attn_fwd_host(const void *q, const void *k, const void *v, void *o, int B, int H,
                           int N, int d, float sm_scale, const uint8_t *block_mask, void *stream);

/* The fused attention kernel alone, on already-quantised inputs (the layouts written by
 * sa_quantize_qk and sa_quantize_v).  For callers that reuse quantised K/V across
 * queries, and for timing the kernel without the prologue.  Allocates nothing. */
sa_status sa_attn_fwd_quantized(const int8_t *q_i8, const float *q_scale, const int8_t *k_i8,
                                const float *k_scale, const uint8_t *v_fp8_t,
                                const float *v_scale, void *o, int B, int H, int N, int d,
                                float sm_scale, const uint8_t *block_mask, void *stream);

/* Block-mask producer: the keep mask block_mask uint8 [B,H,ceil(N/128),ceil(N/64)] (device,
 * caller-owned, fully written) for q, k bf16 [B,H,N,d] (device).
 * Sources: NetEase article on the TurboDiffusion release, attention-acceleration section,
 * SLA figure caption (selection from predicted, compressed attention weights);
 * "Video-Generation-101 research log" section 5.5, SpargeAttention row (a block selector
 * ahead of the sparse low-bit kernel).  Reading: Q is mean-pooled per 128-token block and
 * K per 64-token block (fp64 sums in token order, rounded to fp32); each pair is scored by
 * the fp64 dot product of the two means (channel order); row i keeps its keep_per_row
 * highest-scoring key blocks (ties: lower block index), plus blocks 2i and 2i+1 when
 * keep_diagonal is non-zero.  keep_per_row >= 1 (values >= ceil(N/64) keep every block).
 * Needs ceil(N/64) <= 4096 (else SA_ERR_UNSUPPORTED).  Uses the library workspace for the
 * block means and the scores.  The result is a deterministic function of q and k. */
sa_status sa_block_mask(const void *q, const void *k, int B, int H, int N, int d, int keep_per_row,
                        int keep_diagonal, uint8_t *block_mask, void *stream);

/* Debug: the block means of sa_block_mask, qbar fp32 [B,H,ceil(N/128),d] and kbar fp32
 * [B,H,ceil(N/64),d] (device, caller-owned).  Allocates nothing. */
sa_status sa_debug_pool(const void *q, const void *k, int B, int H, int N, int d, float *qbar,
                        float *kbar, void *stream);

/* ---- W8A8 linear layer: y = x . w^T with x [M,K] and w [N,K] both quantised to INT8 with
 * one scale per 128 x 128 block, products on the INT8 tensor cores.
 * Sources: NetEase article on the TurboDiffusion release, W8A8 linear-layer section
 * (weights and activations of the linear layers to 8 bits, 128 x 128 blocks, INT8 tensor
 * cores); "AIGC weekend special 5.10" section 1.2 Method, item (4).
 * Definition (readings where the pages are silent): a block's scale is max|x| / 127 over
 * the block (fp32), codes rint_even(x / scale) clamped to [-127, 127], a zero block has
 * scale 0 and codes 0; K is padded with zero codes to kpad = 128 * ceil(K/128);
 * y[m,n] = bf16_rn( acc ), acc = 0, then for each k-block b = 0, 1, ... in order:
 *   acc = fmaf( (float) S_b, sx[m/128][b] * sw[n/128][b], acc )   (fp32, one rounding),
 * S_b the exact int32 dot product of the 128 codes of block b. */

/* Block quantisation of x bf16 [rows, cols] (device): codes int8 [rows, 128*ceil(cols/128)]
 * (padding columns written as zero), scales fp32 [ceil(rows/128), ceil(cols/128)] (both
 * device, caller-owned).  cols % 8 == 0 and ceil(rows/128) <= 65535, else SA_ERR_UNSUPPORTED.
 * Bit-identical to the definition above.  Allocates nothing.  Used for the weights once and
 * for the activations on every call. */
sa_status sa_w8a8_quantize(const void *x, int rows, int cols, int8_t *codes, float *scales, void *stream);

/* y bf16 [M, N] (device, caller-owned) from quantised x (codes [M, kpad], scales
 * [ceil(M/128), kpad/128]) and w (codes [N, kpad], scales [ceil(N/128), kpad/128]), as laid
 * out by sa_w8a8_quantize.  N % 8 == 0, else SA_ERR_UNSUPPORTED.
 * Bit-identical to the definition above.  Allocates nothing. */
sa_status sa_w8a8_gemm(const int8_t *x_codes, const float *x_scales, const int8_t *w_codes,
                       const float *w_scales, int M, int N, int K, void *y, void *stream);

/* The linear layer: quantises x bf16 [M, K] into the library workspace, then sa_w8a8_gemm
 * with the pre-quantised weight.  K % 8 == 0 and N % 8 == 0, else SA_ERR_UNSUPPORTED.
 * Workspace rules as for sa_attn_fwd. */
sa_status sa_w8a8_linear(const void *x, const int8_t *w_codes, const float *w_scales, int M, int N,
                         int K, void *y, void *stream);

/* ---- SLA: sparse quantised attention on the critical blocks plus linear attention on the
 * marginal blocks.
 * Sources: NetEase article on the TurboDiffusion release, attention-acceleration section
 * (SLA combines sparse and linear attention; its figure caption splits the attention
 * weights into three classes handled at different costs); "AIGC weekend special 5.10"
 * section 1.2 Method item (2) (SLA runs on top of SageAttention).  The pages give no
 * formula for the linear part.  Reading: block classes come per (128-query block,
 * 64-key block) in classes uint8 [B,H,nq,nk] (device): 0 = negligible (skipped), 1 =
 * marginal (linear attention), >= 2 = critical (sparse quantised attention).  The linear
 * part is kernelised linear attention over the keys of the row's marginal blocks,
 *     O_lin[r] = sum_t w_t v_t / sum_t w_t,  w_t = phi(q_r) . phi(k_t)   (0 if no such key),
 * with phi = SA_PHI_SOFTMAX (softmax over the d features of a row) or SA_PHI_ELU1
 * (elu(x) + 1), projected by W: out[r][c] = sum_e W[c][e] O_lin[r][e], W fp32 [d][d]
 * (device; NULL = identity; in SLA a trained layer).  Evaluated in fp32 in the factorised
 * form phi(q)^T (sum_t phi(k_t) v_t^T) / (phi(q) . sum_t phi(k_t)): per 64-key block
 * the state sum_t phi(k_t) [v_t, 1]^T (128 x 129), then per 128-query block the sum of
 * its marginal blocks' states on the tensor cores (TF32 products of the 0/1 class matrix
 * with the states split into two TF32 terms, about 22 significant bits each, fp32
 * accumulation), then the division and projection.
 * Needs ceil(N/64) <= 4096 (else SA_ERR_UNSUPPORTED).  Uses the library workspace for
 * the states of one group of heads at a time: 69,632 bytes per 64-key block and per
 * 128-query block of a head, at most about 1 GiB (one head at least). */
enum { SA_PHI_SOFTMAX = 0, SA_PHI_ELU1 = 1 };

/* The linear branch alone: out fp32 [B,H,N,d] (device, caller-owned) = W O_lin. */
sa_status sa_sla_linear(const void *q, const void *k, const void *v, const uint8_t *classes, int B, int H,
                        int N, int d, int phi, const float *proj, float *out, void *stream);

/* The SLA forward: o bf16 [B,H,N,d] = the quantised attention of sa_attn_fwd restricted to
 * the critical blocks (a row without one gives 0), plus the projected linear branch,
 * added in fp32 and rounded once to bf16.  The linear branch runs first, into the library
 * workspace in fp32 (a further 4 * d bytes per query token), and the sparse part's
 * epilogue adds it to O before O's only rounding. */
sa_status sa_sla_fwd(const void *q, const void *k, const void *v, void *o, int B, int H, int N, int d,
                     float sm_scale, const uint8_t *classes, int phi, const float *proj, void *stream);

/* ---- Generation over a cache: rotary positions, a paged INT8 key/value cache, attention over it.
 * Sources: "AIGC weekend special 5.10", sections 4 (HiAR) and 6 (SDVG): causal and
 * autoregressive video generation, where each new latent frame attends to the frames before
 * it, whose keys and values are kept; section 1.2 Method item (1): low-bit keys.  The pages
 * give no cache format and no position code; what is computed is stated here in full.
 *
 * Conventions of these calls, beyond those above:
 *   - dtype is SA_BF16, SA_FP16 or (sa_rope, sa_cache_read) SA_FP32, the type of q, k, v, o.
 *   - Tokens are packed: T tokens, those of sequence b being tok_start[b] .. tok_start[b + 1] - 1
 *     (int32 [B + 1], device).  kv_lens[b] (int32 [B], device) counts the cached tokens of
 *     sequence b INCLUDING these n = tok_start[b + 1] - tok_start[b], which stand at the
 *     positions kv_lens[b] - n .. kv_lens[b] - 1.  A token whose position is negative is
 *     padding (kv_lens[b] = 0 for an idle row of a fixed batch): it is not stored, reads as
 *     zero and attends to nothing.  Tokens before tok_start[0] or from tok_start[B] on belong to no
 *     sequence: they are not read, and their rows of the outputs are left as they were.
 *   - page_table int32 [B, max_pages] (device): token t of sequence b is row t % 64 of page
 *     page_table[b][t / 64].  Entries past a sequence's last page are not read.
 *   - The cache, device memory of the caller: codes int8 [num_pages, H, 64, d] and scales fp32
 *     [num_pages, H] (>= 0), for keys and for values; a value is scale * code.  d = 64 or 128.
 *   - Lengths, offsets and pages are read on the device, so a captured graph follows their
 *     changes.  One that is out of range (page outside [0, num_pages), length above
 *     64 * max_pages, offsets that decrease or pass T) sets SA_ERR_BAD_INDEX in the device
 *     status word: nothing is stored through it, a bad page reads as NaN, and a sequence whose
 *     length or offsets are bad is left out, its output rows as they were (appending and
 *     reading may leave out others beside offsets that decrease).  Attention of few rows (16 of a
 *     sequence and head or fewer on average) leaves out, in the same way, a call of more than 2^39
 *     blocks, counted for each head and each 8 rows.
 *   - T = 0 (N = 0) is a valid call that does nothing.
 *   - The codes, k, v, q, o, x, y and the workspace are 16-byte aligned; freqs 8-byte; the int32
 *     and the other fp32 arrays 4-byte.  Token strides are in elements, multiples of 16 bytes, and at
 *     least a token's heads * d; a token's heads follow each other without a gap.  B <= 2^20,
 *     T <= 2^30, H <= 65535, 64 * max_pages <= 2^30, num_pages * H * d / 2 <= 2^31 - 1 and
 *     (T / 64 + 2 B) * H <= 2^31 - 1, else SA_ERR_UNSUPPORTED.
 *   - No call uses the library workspace or allocates anything. */
enum { SA_BF16 = 0, SA_FP16 = 1, SA_FP32 = 2 };
enum { SA_ROPE_PLAIN = 0, SA_ROPE_LINEAR = 1, SA_ROPE_BASE = 2, SA_ROPE_RAMP = 3 };
enum { SA_CACHE_PAGE = 64 };

/* Host only: the rotation frequencies (radians per position) freqs double [rot / 2] and the
 * amplitude of a rotary code of `rot` channels (a multiple of 16):
 *   SA_ROPE_PLAIN   base^(-2i/rot);
 *   SA_ROPE_LINEAR  the same divided by factor (positions squeezed);
 *   SA_ROPE_BASE    with base * factor^(rot/(rot-2)) for base: the fastest pair as it was, the
 *                   slowest divided by factor;
 *   SA_ROPE_RAMP    pairs that turn more than beta_fast times within original_len positions as
 *                   they were, those that turn less than beta_slow times divided by factor, the
 *                   ones between mixed linearly in the pair's index, from the (real) index that
 *                   turns beta_fast times, rounded down, to the one that turns beta_slow times,
 *                   rounded up, both of which may lie outside the pairs; amplitude
 *                   0.1 ln(factor) + 1 (Peng et al., "YaRN", 2023).
 * base > 1, factor >= 1; original_len >= 1 and beta_fast > beta_slow > 0 for SA_ROPE_RAMP. */
sa_status sa_rope_frequencies(int rot, double base, int scaling, double factor, int original_len,
                              double beta_fast, double beta_slow, double *freqs, float *amplitude);

/* One tensor of a rotation: x -> y, [B, heads, N, d] by element strides of batch, head and
 * token (channels contiguous).  y == x with equal strides rotates in place; x and y must not
 * overlap in any other way, nor y's elements each other (a stride of 0 over more than one is
 * refused, and so is y == x with other strides).  Of two tensors, neither's y is the other's x or y. */
typedef struct {
    const void *x;
    void *y;
    int64_t x_batch, x_head, x_tok, y_batch, y_head, y_tok;
    int heads;
} sa_rope_tensor;

/* Rotary positions of one or two tensors (q, and k if count = 2) that share their tokens, in
 * one launch.  Pair i of the first `rot` channels of a head -- channels (i, i + rot/2), or
 * (2i, 2i + 1) if interleaved -- turns by the angle pos * freqs[i] (fp64, freqs device [rot/2])
 * and is multiplied by amplitude; inverse != 0 turns the other way, which is the transposed
 * map.  The other channels are copied.  Computed in fp32, rounded once.
 * pos int32 (device): token n of batch b on axis a is pos[a * pos_axis + b * pos_batch + n];
 * pair i belongs to axis a where sections[0] + .. + sections[a - 1] <= i; sections (host,
 * axes <= 4 counts that sum to rot / 2) may be NULL with axes = 1.  pos_batch = 0 shares the
 * positions among the batches.  d a multiple of 16 up to 256, rot a multiple of 16 up to d. */
sa_status sa_rope(const sa_rope_tensor *tensors, int count, int dtype, int B, int N, int d, int rot,
                  int interleaved, const int32_t *pos, int64_t pos_axis, int64_t pos_batch, int axes,
                  const int *sections, const double *freqs, float amplitude, int inverse, void *stream);

/* Writes the new tokens k, v [T, H, d] (SA_BF16 or SA_FP16, token strides k_tok, v_tok) into
 * the cache.  For each block of 64 tokens and each head, keys and values apart: s_new =
 * fl(max|x| / 127) over the block's new tokens; the scale becomes s = s_new for a block without
 * older tokens, else max(s_old, s_new), the older codes c becoming rint(fl(c * fl(s_old / s)));
 * the new codes are rint(fl(x / s)) within +-127 (fl: one rounding to fp32; rint: ties to
 * even; codes 0 where s = 0).  A code that was written at once is off by at most s/2; each
 * later growth of the block's scale adds at most s/2 of the new scale.  Non-finite values make the block read as NaN.
 * Sequences must not share a page that this call writes. */
sa_status sa_cache_append(const void *k, const void *v, int dtype, int64_t T, int64_t k_tok, int64_t v_tok,
                          const int32_t *tok_start, const int32_t *kv_lens, const int32_t *page_table, int B,
                          int max_pages, int8_t *k_codes, float *k_scale, int8_t *v_codes, float *v_scale,
                          int num_pages, int H, int d, void *stream);

/* Reads the values of the tokens at tok_start / kv_lens out of the cache: k, v contiguous
 * [T, H, d] of dtype (either may be NULL), scale * code rounded once. */
sa_status sa_cache_read(void *k, void *v, int dtype, int64_t T, const int32_t *tok_start,
                        const int32_t *kv_lens, const int32_t *page_table, int B, int max_pages,
                        const int8_t *k_codes, const float *k_scale, const int8_t *v_codes,
                        const float *v_scale, int num_pages, int H, int d, void *stream);

/* Attention of the T query tokens q [T, H * group, d] (SA_BF16 or SA_FP16, token stride q_tok)
 * over the cache, whose tokens include the queries' own (append first).  Query head h reads
 * key/value head h / group (H * group <= 65535, T * group <= 2^30 and T * H * group <= 2^34, else
 * SA_ERR_UNSUPPORTED).  The query at position p sees the tokens t < kv_lens[b] with
 * t <= p (causal != 0) and t > p - window (window > 0; 0: no window).
 *   o [T, H * group, d] (contiguous, dtype, apart from q in memory) = sum_t softmax_t(q . k_t * sm_scale) v_t, and lse
 *   fp32 [T, H * group] (or NULL) = log sum_t exp(q . k_t * sm_scale); a query that sees
 *   nothing has o = 0 and lse = -inf.  sm_scale is positive and finite.
 * Products of fp16 operands (the codes and, up to a power of two for each row, q are exact; a softmax
 * weight times its block's value scale is rounded to fp16: off by at most 2^-11 of itself or 2^-31 of the
 * largest such product that the row sees), sums and statistics in fp32.  The result does not depend on
 * timing, and a row's not on blocks that it does not see.  One kernel takes the whole call, by its
 * rows (T * group) to a sequence on average: long pieces among many single tokens are faster as a
 * call of their own.  workspace: device memory of at least
 * sa_cache_attn_workspace_bytes(T, B, H, group, d) bytes, which the call may overwrite and which no other
 * call may use meanwhile; it need not be set before or kept after. */
sa_status sa_cache_attn(const void *q, void *o, float *lse, int dtype, int64_t T, int64_t q_tok,
                        const int32_t *tok_start, const int32_t *kv_lens, const int32_t *page_table, int B,
                        int max_pages, const int8_t *k_codes, const float *k_scale, const int8_t *v_codes,
                        const float *v_scale, int num_pages, int H, int group, int d, int causal, int window,
                        float sm_scale, void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace that sa_cache_attn needs for these sizes on the current device (0: sizes
 * that it refuses, or no device). */
size_t sa_cache_attn_workspace_bytes(int64_t T, int B, int H, int group, int d);

/* Debug (host only): in later sa_cache_attn calls of the process this worker (a block of the
 * kernel of many rows, a warp of the other) gives up after its first work as if a wait had expired,
 * for tests of failure detection; -1: none.  Such a call sets SA_ERR_DEVICE_TIMEOUT; of the rows
 * that the worker has part in, those that it begins are left as they were or NaN, those that it goes
 * on with are NaN. */
void sa_debug_cache_attn_quit(int worker);

/* Debug (host only): the steps of 256 rows by 128 keys that sa_cache_attn's tensor-core kernel
 * takes for each key/value head of a sequence of n queries over len cached tokens (-1: refused). */
int64_t sa_debug_cache_steps(int n, int len, int group, int causal, int window);

/* Debug: the int32 S = q_i8 . k_i8^T tiles computed by the same tcgen05 INT8 path the
 * attention kernel uses, stored to s_out int32 [B,H,Npad,Npad] (padded rows/keys
 * included).  For bit-exact checks on small problems only.  Allocates nothing. */
sa_status sa_debug_qk_s32(const int8_t *q_i8, const int8_t *k_i8, int B, int H, int N, int d,
                          int32_t *s_out, void *stream);

/* Debug: launches a one-CTA kernel whose mbarrier wait can never complete, bounded by
 * timeout_us microseconds; the kernel then records SA_ERR_DEVICE_TIMEOUT in the device
 * status word and returns.  Exercises the failure path without faulting the GPU. */
sa_status sa_debug_wait_timeout(int timeout_us, void *stream);


/* Synchronises the current device, returns and clears its device status word
 * (SA_OK, SA_ERR_DEVICE_TIMEOUT or SA_ERR_BAD_INDEX), or SA_ERR_CUDA if synchronisation
 * failed. */
sa_status sa_get_device_status(void);

/* Human-readable name of a status code (static string). */
const char *sa_status_string(sa_status s);

/* Bytes of library workspace sa_attn_fwd needs for this problem size, d = 128 or 64 (0 on
 * bad sizes).  Causal calls with a keep mask add B * H * ceil(N/128) * ceil(N/64) bytes. */
size_t sa_workspace_bytes(int B, int H, int N, int d);

/* Measurement aid (no counterpart on the pages): the device's own 8-bit tensor-core rate,
 * the denominator of the attention kernel's roofline.  Launches one CTA per SM; each
 * issues `reps` chains of four tcgen05 MMAs of M = 128, N = 256, K = 32 (one K = 128
 * contraction, the way the attention kernel issues them) from shared memory into tensor
 * memory: kind 0 = kind::i8 (int8 x int8 -> int32), kind 1 = kind::f8f6f4 with e4m3
 * operands (-> fp32).  The caller times the launch (e.g. with CUDA events on `stream`);
 * it performs SMs * reps * 4 * 2*128*256*32 operations.  reps in [1, 2^20]; the final
 * bounded wait reports through sa_get_device_status. */
sa_status sa_debug_mma_peak(int kind, int reps, void *stream);

/* Frees the current device's workspace (synchronises the device first). */
sa_status sa_release_workspace(void);

/* Padded token count Npad = 128 * ceil(N/128) (0 for N < 1). */
int64_t sa_padded_len(int N);

#ifdef __cplusplus
}
#endif

#endif /* SA_H */
