/*
 * clover.h - C ABI of the GB300 (sm_103a) block-diffusion MoE denoising step.
 *
 * The operations follow "Clover-35B-A3B: how a diffusion model gets to 680
 * tokens a second, read from its files" (cited below as "Files"):
 *   - "What Clover is": per layer 256 routed experts, top-8 routing, one
 *     always-on shared expert; hidden 2,048; expert = gate and up 2,048 x 512,
 *     down 512 x 2,048; untied output head 248,320 x 2,048 read in full each
 *     step; block_size 32, mask_token_id 151669, low-confidence threshold 0.95.
 *   - "The expert selection": per-token top-8 routing probabilities.
 *   - "How it writes", steps 1-4: the block denoising loop and its unmask rule.
 *
 * Conventions shared by every entry point:
 *   - All tensor pointers are DEVICE pointers on the current CUDA device,
 *     owned by the caller. The library allocates no device memory; every
 *     scratch buffer lives in a caller-provided workspace whose size the
 *     matching *_workspace_bytes() call returns. A workspace must be
 *     zero-filled before its first use; afterwards the library keeps its
 *     control words consistent between calls. One workspace must not be used
 *     by two calls that may run at the same time.
 *   - bf16 tensors are passed as `const uint16_t*` (their bit patterns),
 *     row-major, densely packed, 16-byte aligned.
 *   - Every call is asynchronous on `stream` unless stated otherwise, and
 *     returns CLOVER_OK or a negative status. Argument errors are detected on
 *     the host before anything is enqueued. clover_last_error() returns the
 *     message of the last failing call on the calling thread.
 *   - Kernels never trap. A wait inside a kernel that exceeds its time limit
 *     records a flag in the workspace and the kernel returns;
 *     clover_workspace_status() reports it as CLOVER_ERR_DEVICE_TIMEOUT.
 *   - Shapes: hidden % 128 == 0, d_ff % 64 == 0, 1 <= top_k <= 32,
 *     top_k <= n_experts <= 256, hidden <= 8192, 1 <= tokens <= 1024,
 *     vocab >= 2, 0 <= mask_id < vocab. Other shapes return
 *     CLOVER_ERR_UNSUPPORTED_SHAPE; there is no fallback path. Above 32
 *     tokens an expert's tokens are processed in tiles of at most 128: an
 *     expert that more tokens select is streamed once per tile of its tokens
 *     (the tiles run side by side, so the repeat reads mostly come from L2);
 *     above 256 positions the head streams once per 256 positions.
 */
#ifndef CLOVER_H_
#define CLOVER_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define CLOVER_OK 0
#define CLOVER_ERR_INVALID_ARG (-1)
#define CLOVER_ERR_WORKSPACE_TOO_SMALL (-2)
#define CLOVER_ERR_CUDA (-3)
#define CLOVER_ERR_NOT_CONVERGED (-4)
#define CLOVER_ERR_UNSUPPORTED_SHAPE (-5)
#define CLOVER_ERR_DEVICE_TIMEOUT (-6)

/* cudaStream_t and cudaEvent_t are pointers to these opaque structs. */
typedef struct CUstream_st* clover_stream_t;
typedef struct CUevent_st* clover_event_t;

/* Model dimensions. Files, "What Clover is": hidden 2048, n_experts 256,
 * top_k 8, d_ff 512, vocab 248320, mask_id 151669; moe_block_coreset_enabled
 * with top_p 0.9. rms_eps is the epsilon of the unit-weight RMSNorm placed
 * before each MoE sublayer and before the head (a reading; the pages give no
 * norm).
 * coreset_top_p: 0 disables the block coreset; a value in (0, 1] enables it
 * (Files, "The expert selection"): per block, each expert's mass is the sum of
 * the softmax probabilities of the slots that select it; the kept set is the
 * shortest prefix of experts by mass (descending, lower id first) whose
 * cumulative mass reaches coreset_top_p x total and that holds at least
 * top_k experts; every token then takes its top_k within the kept set. The
 * coreset is available for calls of at most 32 positions forming one block. */
typedef struct {
    int32_t hidden;    /* H */
    int32_t n_experts; /* E, routed experts per layer */
    int32_t top_k;     /* K */
    int32_t d_ff;      /* F, expert intermediate width */
    int32_t vocab;     /* V */
    int32_t mask_id;   /* mask token id; never predicted */
    float rms_eps;
    float coreset_top_p; /* 0 = off */
} clover_dims;

/* One MoE layer's weights (device pointers). Files, "What Clover is". */
typedef struct {
    const uint16_t* router_w;   /* bf16 [E][H]                                   */
    const float* router_bias;   /* fp32 [E] added to the router logits, or NULL  */
    const uint16_t* gate_up;    /* bf16 [E][2F][H]: rows 0..F-1 gate, F..2F-1 up */
    const uint16_t* down;       /* bf16 [E][H][F]                                */
    const uint16_t* sh_gate_up; /* bf16 [2F][H], shared expert                   */
    const uint16_t* sh_down;    /* bf16 [H][F],  shared expert                   */
    /* Low-bit expert weights (format of clover_quantize_q4). When gate_up_q is
     * non-NULL all eight fields below must be set and the four bf16 expert
     * pointers above are ignored (may be NULL); the router stays bf16. */
    const uint8_t* gate_up_q;    /* codes [E][2F][H/2]   */
    const uint16_t* gate_up_s;   /* scales [E][H/64][2F] */
    const uint8_t* down_q;       /* codes [E][H][F/2]    */
    const uint16_t* down_s;      /* scales [E][F/64][H]  */
    const uint8_t* sh_gate_up_q; /* codes [2F][H/2]      */
    const uint16_t* sh_gate_up_s;/* scales [H/64][2F]    */
    const uint8_t* sh_down_q;    /* codes [H][F/2]       */
    const uint16_t* sh_down_s;   /* scales [F/64][H]     */
} clover_moe_layer;

/* Bytes of workspace clover_moe_block_step needs for up to max_tokens tokens.
 * Returns 0 for an unsupported shape. Host-only. */
size_t clover_moe_workspace_bytes(const clover_dims* dims, int32_t max_tokens);

/* One pre-norm MoE sublayer on M tokens (Files, "What Clover is" and "The
 * expert selection"):
 *   xn  = bf16(RMSNorm(x_in))
 *   p   = softmax(xn W_r^T + b), top-k by p (ties to the lower expert id),
 *         w = p_sel / sum(p_sel)
 *   y_t = sum_k w_tk * E_{i_tk}(xn_t) + S(xn_t),  E(x) = bf16(silu(x W_g^T) *
 *         (x W_u^T)) W_d^T, S the shared expert with weight 1
 *   x_out = x_in + y
 * x_in, x_out: fp32 [M][H]; x_out may equal x_in (in place), other overlap is
 * not allowed. topk_idx (int32 [M][K]) and topk_w (fp32 [M][K]) receive the
 * selection in descending probability order; either may be NULL.
 * Each selected expert's weights are read from HBM once per call (up to 32
 * tokens; above, once per tile of 128 of its tokens, the repeats of one
 * expert's tiles requested together so that L2 serves them). */
int clover_moe_block_step(const clover_dims* dims, const clover_moe_layer* layer,
                          const float* x_in, float* x_out,
                          int32_t* topk_idx, float* topk_w, int32_t M,
                          void* workspace, size_t workspace_bytes, clover_stream_t stream);

/* Low-bit expert weights. The pages name INT4 for one deployment (Files,
 * "What 680 tokens a second has to be") but give no format; this format is
 * the library's own. Quantizes n_mats bf16 matrices w [n_mats][rows][cols]
 * (cols % 64 == 0) into 4-bit codes q [n_mats][rows][cols/2] and bf16 scales
 * s [n_mats][cols/64][rows]: per row and group of 64 columns,
 *   s = bf16(float32(max |w|) / 7)          (IEEE fp32 division, nearest even)
 *   u = clamp(rint(float32(w) / s), -8, 7) + 8   (u = 8 where s = 0)
 * and the weight a product then uses is bf16((u - 8) s). Codes are packed
 * eight to a little-endian 32-bit word, nibble i (bits 4i..4i+3) holding
 * element (0, 2, 4, 6, 1, 3, 5, 7)[i] of the eight. All pointers are device
 * pointers, 16-byte aligned; asynchronous on `stream`. */
int clover_quantize_q4(const uint16_t* w, int32_t n_mats, int32_t rows, int32_t cols, uint8_t* q,
                       uint16_t* s, clover_stream_t stream);

/* Bytes of workspace clover_lmhead_unmask needs. Host-only. */
size_t clover_head_workspace_bytes(const clover_dims* dims, int32_t max_tokens);

/* Output head, statistics and the low-confidence unmask rule on M positions
 * (Files, "What Clover is": untied head read in full; "How it writes", steps
 * 2-3).
 *   z_p,v = alpha_p * (bf16(RMSNorm(x_p)) . W_h[v]),  z_p,mask_id = -inf
 *   argmax_p = lowest v with the largest z, max_logit_p = max z,
 *   lse_p = log sum_v exp(z_p,v), max_prob_p = exp(max_logit_p - lse_p)
 * The full logits are never written. Then, for each group of `block`
 * consecutive positions: every position with masked_p != 0 and
 * max_prob_p > threshold is committed; if none is, the masked position with
 * the largest max_prob (lowest index on ties) is committed. Committing sets
 * tokens_p = argmax_p and masked_p = 0.
 * head_w: bf16 [V][H]. x: fp32 [M][H] (pre-norm). logit_scale: fp32 [M] or
 * NULL (= 1). tokens int32 [M], masked uint8 [M]: in/out. argmax int32 [M],
 * max_logit, lse, max_prob fp32 [M]: out. n_committed: device int32 scalar,
 * out (number committed by this call). M % block == 0 is not required; the
 * last group may be shorter. Above 256 positions, block must be at most 256
 * (the head then runs on whole blocks, at most 256 positions at a time). A committed slot (masked_p == 0) whose token id
 * lies outside [0, V) is left as it is and reported through the workspace
 * status word (clover_workspace_status). */
int clover_lmhead_unmask(const clover_dims* dims, const uint16_t* head_w, const float* x,
                         const float* logit_scale, float threshold, int32_t block,
                         int32_t* tokens, uint8_t* masked,
                         int32_t* argmax, float* max_logit, float* lse, float* max_prob,
                         int32_t* n_committed, int32_t M,
                         void* workspace, size_t workspace_bytes, clover_stream_t stream);

/* Accept rules of clover_lmhead_accept. */
#define CLOVER_ACCEPT_EXACT 0
#define CLOVER_ACCEPT_THRESHOLD 1

/* Bytes of workspace clover_lmhead_accept needs for up to max_rows rows.
 * Host-only. */
size_t clover_accept_workspace_bytes(const clover_dims* dims, int32_t max_rows);

/* Output head of a verify pass fused with the self-speculative accept test
 * (Files, "Two ways to run it": a round keeps the longest prefix of drafts
 * the causal pass accepts, plus one token at the boundary; the exact rule
 * keeps a draft only if it is the causal pass's argmax, the threshold rule
 * if its probability is at least min(ratio, delta e^-H), H the entropy of the
 * causal distribution, defaults ratio 0.9 and delta 0.6).
 * The M rows form M / block blocks; in each, row j < block - 1 is the
 * distribution draft[j] is tested against and the last row gives the token
 * after the final draft. Per row, as clover_lmhead_unmask (mask token at
 * -inf): argmax, max_logit, lse, max_prob, plus
 *   entropy_p = -sum_v p_v ln p_v  (p = softmax of z_p),
 *   p_draft_p = p at draft[p]      (0 for the mask token or an id outside
 *                                   [0, V); the last row of a block: ignored)
 * Per block b: accept_len[b] = r, the number of leading rows whose draft is
 * accepted (exact: draft == argmax; threshold: p_draft >= min(ratio,
 * delta e^-entropy), fp32), and out_tokens[b*block + j] = draft for j < r,
 * argmax of row r at j = r, -1 after (r + 1 tokens).
 * head_w: bf16 [V][H]. x: fp32 [M][H] (pre-norm). logit_scale: fp32 [M] or
 * NULL. draft: int32 [M], in. rule: CLOVER_ACCEPT_EXACT or
 * CLOVER_ACCEPT_THRESHOLD (then 0 < ratio <= 1 and a finite delta > 0).
 * argmax, max_logit, lse, max_prob, entropy, p_draft: [M] out, each may be
 * NULL. accept_len int32 [M / block], out_tokens int32 [M]: out. Requires
 * block >= 2 and M % block == 0. */
int clover_lmhead_accept(const clover_dims* dims, const uint16_t* head_w, const float* x,
                         const float* logit_scale, const int32_t* draft, int32_t rule, float ratio,
                         float delta, int32_t block,
                         int32_t* argmax, float* max_logit, float* lse, float* max_prob,
                         float* entropy, float* p_draft, int32_t* accept_len, int32_t* out_tokens,
                         int32_t M, void* workspace, size_t workspace_bytes, clover_stream_t stream);

/* Bytes of workspace the denoise entry points need. Host-only. */
size_t clover_denoise_workspace_bytes(const clover_dims* dims, int32_t max_tokens);

/* Byte offset, within a denoise workspace sized for max_tokens, of the
 * residual stream that the last clover_denoise_step left there: fp32 [M][H],
 * the output of the last MoE sublayer (the input of the final RMSNorm and
 * the head). Host-only. Returns 0 for invalid dims or max_tokens (the offset
 * itself is never 0). */
size_t clover_denoise_hidden_offset(const clover_dims* dims, int32_t max_tokens);

/* One block-diffusion denoising step over M positions (Files, "How it
 * writes", steps 1-3): x_p = E[tokens_p] + ctx_p (the mask token's embedding
 * while masked), n_layers MoE sublayers as in clover_moe_block_step, a final
 * RMSNorm, then clover_lmhead_unmask's statistics and unmask rule.
 * layers: HOST array of n_layers structs (the pointers inside are device
 * pointers). embed: bf16 [V][H]. ctx: fp32 [M][H], fixed per block.
 * head_w: bf16 [V][H]. logit_scale: fp32 [M] or NULL. tokens, masked: in/out.
 * The positions form M / block independent blocks (M % block == 0). */
int clover_denoise_step(const clover_dims* dims, const clover_moe_layer* layers, int32_t n_layers,
                        const uint16_t* embed, const float* ctx, const uint16_t* head_w,
                        const float* logit_scale, float threshold, int32_t block,
                        int32_t* tokens, uint8_t* masked, int32_t M,
                        void* workspace, size_t workspace_bytes, clover_stream_t stream);

/* Repeats clover_denoise_step until no position is masked or max_steps steps
 * ran (Files, "How it writes", step 4). Synchronises `stream` once per step to
 * read the number of masked positions left. *steps_taken (host) receives the
 * number of steps. Returns CLOVER_ERR_NOT_CONVERGED if positions are still
 * masked after max_steps steps. */
int clover_denoise_block(const clover_dims* dims, const clover_moe_layer* layers, int32_t n_layers,
                         const uint16_t* embed, const float* ctx, const uint16_t* head_w,
                         const float* logit_scale, float threshold, int32_t block,
                         int32_t* tokens, uint8_t* masked, int32_t M, int32_t max_steps,
                         int32_t* steps_taken,
                         void* workspace, size_t workspace_bytes, clover_stream_t stream);

/* Synchronises `stream`, then reads and clears the device status word of a
 * workspace used by any call above. Returns CLOVER_OK, or
 * CLOVER_ERR_DEVICE_TIMEOUT if a kernel gave up on a wait (the message names
 * which), or CLOVER_ERR_CUDA. */
int clover_workspace_status(void* workspace, size_t workspace_bytes, clover_stream_t stream);

/* Timing hook: when `begin`/`end` are non-NULL, every later launch of the
 * expert kernel (one per MoE sublayer) records begin[i % capacity] before and
 * end[i % capacity] after launch i on the launching stream; i restarts at 0
 * at each call of this function. Pass NULL to stop. Process-wide, not
 * thread-safe. Returns the number of launches recorded since the last call. */
int32_t clover_profile_expert_events(clover_event_t* begin, clover_event_t* end, int32_t capacity);

/* Copies the last error message of the calling thread into buf (at most n
 * bytes, NUL-terminated). Returns its full length. */
int32_t clover_last_error(char* buf, size_t n);

/* Same operation and arguments as clover_lmhead_unmask, without the
 * workspace. (The pages have no counterpart: this is a library convenience.)
 * For callers that cannot allocate device memory -- a plug-in inside an
 * application that owns all GPU memory and hands out no allocator, or a
 * latency-critical loop that must not synchronise on an allocation. The
 * scratch lives in a 1 MiB array inside the library that
 * every GPU loading the library keeps until the process exits; it fits up to
 * 102 positions at hidden 2048 (the rule: clover_head_workspace_bytes(dims, M)
 * <= 1 MiB). Larger sizes return CLOVER_ERR_WORKSPACE_TOO_SMALL and nothing
 * runs. Every call looks up the array's device address in the current
 * context; the first call on a device also loads the library's kernels
 * there, so make that first call before any stream capture. The call
 * allocates nothing. It checks every argument before it enqueues anything,
 * then clears the array's control words on the stream, so the status of a
 * call must be read (clover_lmhead_unmask_static_status) before the next
 * call. All calls share the one array: calls that may overlap on the GPU
 * (other streams, other threads) race and must be serialised by the caller. */
int clover_lmhead_unmask_static(const clover_dims* dims, const uint16_t* head_w, const float* x,
                                const float* logit_scale, float threshold, int32_t block,
                                int32_t* tokens, uint8_t* masked,
                                int32_t* argmax, float* max_logit, float* lse, float* max_prob,
                                int32_t* n_committed, int32_t M, clover_stream_t stream);

/* The device status of the last clover_lmhead_unmask_static call, which has
 * no workspace to pass to clover_workspace_status: synchronises `stream`,
 * reads the status word of the library's static scratch array, and if it is
 * set clears the array's control words and returns
 * CLOVER_ERR_DEVICE_TIMEOUT (a wait that gave up, or a committed slot whose
 * token id lies outside [0, V); the message names which); else CLOVER_OK.
 * (The pages have no counterpart.) */
int clover_lmhead_unmask_static_status(clover_stream_t stream);

/* ---- Routed experts as separate operations ------------------------------
 * The steps of a routed-expert sublayer for callers whose layer differs from
 * clover_moe_block_step's (another score function, expert groups, longer
 * inputs, hardware 4-bit experts): route -> quantize (gathering the rows into
 * expert order) -> product with SwiGLU -> quantize -> product -> combine.
 * The conventions at the top of this file hold, with these differences: the
 * limits on shapes are the ones stated per call, a call with no rows
 * (M == 0 or n_rows == 0) is valid and needs no data pointers, and none of
 * the calls changes its inputs. Rows, and a token's K slots, count up to 2^29
 * in any one call. */

/* Score functions of clover_route. */
#define CLOVER_SCORE_SOFTMAX 0
#define CLOVER_SCORE_SIGMOID 1

/* Types of an input that may come in more than one. */
#define CLOVER_TYPE_F32 0
#define CLOVER_TYPE_BF16 1

/* Selection rule of clover_route. 1 <= n_experts <= 512; 1 <= top_k <=
 * min(32, n_experts); 1 <= n_groups <= 32, dividing n_experts; 1 <= top_groups
 * <= n_groups; group_rank 1 or 2; scale finite. */
typedef struct {
    int32_t n_experts;   /* E */
    int32_t top_k;       /* K */
    int32_t score;       /* CLOVER_SCORE_*                                     */
    int32_t n_groups;    /* experts form n_groups runs of E / n_groups ids     */
    int32_t top_groups;  /* groups that stay selectable (n_groups = all)       */
    int32_t group_rank;  /* a group ranks by the sum of its 1 or 2 best experts */
    int32_t renormalise; /* nonzero: a token's weights are divided by their sum */
    float scale;         /* factor of every weight                             */
} clover_routing;

/* Bytes of workspace clover_route needs for up to max_tokens tokens. Returns
 * 0 for an unsupported rule or max_tokens < 0. Host-only. */
size_t clover_route_workspace_bytes(const clover_routing* routing, int32_t max_tokens);

/* Expert selection from given router logits, M tokens x E experts.
 *   s = softmax(the token's logits) or 1 / (1 + e^-logit)
 *   key = logit without a bias (s grows with it), s + bias with one
 * A NaN logit counts as -inf, one above the largest finite fp32 as that
 * value. An expert is live for a token unless its logit is -inf or its bias
 * is NaN or -inf. With n_groups >
 * 1 the top_groups groups of the largest rank stay (rank 1: the group's
 * largest key; rank 2: the sum of its up to two largest s + bias; a group
 * without a live expert is last; ties to the lower group). The top_k live
 * experts of the largest keys in the groups that stay are selected, in
 * descending order (ties to the lower id); their weights are s, divided by
 * their sum if renormalise is set, times scale. A token with fewer than
 * top_k such experts (a padding row has none) gets index -1 and weight 0 in
 * the places left over. Keys and ranks closer than fp32 can tell apart are
 * compared in fp64 (ranks that are equal but for fp64's rounding, such as the
 * same two scores and two biases paired otherwise, may order either way).
 * logits: logits_type [M] rows of E, row t at element t * ld (ld >= E),
 * aligned to its element size. bias: fp32 [E] or NULL; it takes part in the
 * selection only. topk_idx int32 [M][K], topk_w fp32 [M][K]: out.
 * Grouping (offsets, rows and pos all set, or all NULL): offsets int32
 * [E + 1], rows int32 [M * K], pos int32 [M][K]. The selected slots t * K + k
 * are listed in rows by expert, then token; expert e's are rows[offsets[e]]
 * .. rows[offsets[e + 1] - 1]. pos[t][k] is the place of slot (t, k) in rows,
 * or -1. Places of rows from offsets[E] on are left as they were.
 * M * top_k <= 2^29. Every result is independent of the launch shape. */
int clover_route(const clover_routing* routing, const void* logits, int32_t logits_type, int64_t ld,
                 const float* bias, int32_t M, int32_t* topk_idx, float* topk_w, int32_t* offsets,
                 int32_t* rows, int32_t* pos, void* workspace, size_t workspace_bytes,
                 clover_stream_t stream);

/* Microscaled 4-bit formats (the tensor cores' own): e2m1 values 0, 0.5, 1,
 * 1.5, 2, 3, 4, 6 and a sign bit, with one scale per block of consecutive
 * columns: */
#define CLOVER_FP4_NV 0 /* blocks of 16, scale e4m3                    */
#define CLOVER_FP4_MX 1 /* blocks of 32, scale e8m0 (a power of two)   */

/* Bytes of the scales of n_mats matrices [rows][cols], each in tiles of 128
 * rows x 4 blocks (512 bytes): tile (mat, rows / 128, blocks / 4) in row-major
 * order, the scale of row r, block b of a tile at byte (r % 32) * 16 +
 * (r / 32) * 4 + b. Rows and blocks are padded to whole tiles. Returns 0 for
 * arguments that clover_quantize_fp4 refuses or a size past 2^62. Host-only. */
size_t clover_fp4_scale_bytes(int32_t format, int32_t n_mats, int32_t rows, int32_t cols);

/* The same for n_rows rows in n_groups consecutive groups: group g (rows
 * offsets[g] .. offsets[g + 1] - 1) begins at row tile offsets[g] / 128 + g,
 * so n_rows / 128 + n_groups row tiles are enough for any offsets. */
size_t clover_fp4_grouped_scale_bytes(int32_t format, int32_t n_rows, int32_t n_groups, int32_t cols);

/* Quantises n_mats matrices x [rows][cols] (x_type fp32 or bf16; row i of the
 * n_mats * rows rows at element i * ldx, ldx >= cols; rows 16-byte aligned;
 * cols % 64 == 0, 64 <= cols <= 2^20) to codes [n_mats][rows][cols / 2] (the
 * even column in the low nibble) and scales. With y = x 2^-scale_exp (fp32,
 * |scale_exp| <= 64) and amax the largest |y| of a block, the block's scale is
 *   NV: s = e4m3(amax / 6), round to nearest even, at most 448
 *   MX: s = 2^(floor(log2 amax) - 2), exponent at least -127 (amax = 0: -127)
 * and each code is the e2m1 value nearest to y / s (ties to the even code, at
 * most 6; 0 where s = 0); it stands for code * s * 2^scale_exp. A block whose
 * y hold a NaN or an infinity gets the scale NaN and codes 0. Scale bytes of
 * padding are not written. codes and scales 16-byte aligned. */
int clover_quantize_fp4(int32_t format, const void* x, int32_t x_type, int64_t ldx, int32_t n_mats,
                        int32_t rows, int32_t cols, int32_t scale_exp, uint8_t* codes, uint8_t* scales,
                        clover_stream_t stream);

/* The same for n_rows rows in groups (offsets int32 [n_groups + 1] on the
 * device, ascending from 0; 1 <= n_groups <= 512), such as the rows of
 * clover_route: row i is quantised from x row src_rows[i] / src_div (NULL: i),
 * 0 <= that < n_src. Rows from offsets[n_groups] on are left as they were.
 * Offsets outside [0, n_rows] count as the nearer end; a row whose source
 * lies outside [0, n_src) gets codes and scales of zeros. */
int clover_quantize_fp4_rows(int32_t format, const void* x, int32_t x_type, int64_t ldx, int32_t n_src,
                             int32_t cols, int32_t scale_exp, const int32_t* src_rows, int32_t src_div,
                             int32_t n_rows, const int32_t* offsets, int32_t n_groups, uint8_t* codes,
                             uint8_t* scales, clover_stream_t stream);

/* What the codes stand for, code * s * 2^scale_exp rounded to bf16 (exact
 * unless it leaves bf16's range): out bf16 [n_mats][rows][cols]; with offsets
 * (NULL: matrices) rows in n_groups groups, n_mats = 1, rows from
 * offsets[n_groups] on left as they were. */
int clover_dequantize_fp4(int32_t format, const uint8_t* codes, const uint8_t* scales, int32_t n_mats,
                          int32_t rows, int32_t cols, int32_t scale_exp, const int32_t* offsets,
                          int32_t n_groups, uint16_t* out, clover_stream_t stream);

/* Epilogues of clover_fp4_product. */
#define CLOVER_FP4_PLAIN 0
#define CLOVER_FP4_SWIGLU 1

/* Bytes of workspace clover_fp4_product needs (its status word; calls that
 * may run at the same time may share it). Host-only. */
size_t clover_fp4_product_workspace_bytes(void);

/* *workspace receives the device address, on the current device, of a
 * workspace for clover_fp4_product that lives in the library: 256 bytes, zeroed
 * when the library is loaded, that calls on any streams may share. For callers
 * who keep none: clover_workspace_status reads and clears it, and so reports a
 * wait that ran out in any of them. Enqueues nothing. */
int clover_fp4_product_shared_workspace(void** workspace);

/* Products of rows with the matrix of their group, both in a microscaled
 * 4-bit format, on the tensor cores (fp32 accumulation):
 *   z_i = alpha * group_alpha[g] * (A_i . B_g^T) for row i of group g (alpha finite)
 *   CLOVER_FP4_PLAIN:  y_i = bf16(z_i)                         [N]
 *   CLOVER_FP4_SWIGLU: y_i = bf16(silu(z_i[0..N/2)) * z_i[N/2..N))  [N / 2]
 * a_codes [n_rows][K / 2] with a_scales as clover_quantize_fp4_rows writes
 * them for offsets (int32 [n_groups + 1], device). offsets NULL: all rows
 * form one group, the layout clover_quantize_fp4 gives one matrix too.
 * b_codes [n_groups][N][K / 2]; b_scales as clover_quantize_fp4 writes them
 * for n_groups matrices of N rows, or, with SwiGLU, for 2 n_groups matrices
 * of N / 2 rows (each group's gate rows, then its up rows: the codes lie the
 * same way). group_alpha: fp32 [n_groups] or NULL. y: bf16, 16-byte aligned;
 * rows outside every group are left as they were. K % 64 == 0, 64 <= K <=
 * 2^20; 1 <= N <= 2^24 (even with SwiGLU); offsets outside [0, n_rows] count
 * as the nearer end. A NaN scale makes its row's (or its column's) results
 * NaN. Results do not depend on the other rows of the call. */
int clover_fp4_product(int32_t format, const uint8_t* a_codes, const uint8_t* a_scales, int32_t n_rows,
                       const uint8_t* b_codes, const uint8_t* b_scales, const int32_t* offsets,
                       int32_t n_groups, int32_t N, int32_t K, float alpha, const float* group_alpha,
                       int32_t epilogue, uint16_t* y, void* workspace, size_t workspace_bytes,
                       clover_stream_t stream);

/* Weighted sum of expert rows, and what a sublayer adds to it:
 *   x_out[t] = x[t] + sum_k w[t][k] * y[pos[t][k]] + shared[t]
 * y: bf16 [n_rows][H]; pos int32 and w fp32 [M][K] as clover_route gives
 * them: a slot whose place lies outside [0, n_rows) adds nothing, whatever its
 * weight. shared: bf16 [M][H] or NULL. x: fp32 [M][H] or NULL (zeros); x_out
 * fp32 [M][H] may equal x, other overlap is not allowed. H % 8 == 0,
 * 1 <= K <= 32. The sum is in fp32: x, then the slots in order, then shared. */
int clover_moe_combine(const uint16_t* y, int32_t n_rows, const int32_t* pos, const float* w,
                       const uint16_t* shared, const float* x, float* x_out, int32_t M, int32_t K, int32_t H,
                       clover_stream_t stream);

/* ---- Attention ------------------------------------------------------------
 * Softmax attention with grouped heads (query head h reads key/value head
 * h / (q_heads / kv_heads)), over a paged 4-bit cache or over a packed prompt.
 * The conventions at the top of this file hold, with the limits stated here:
 * head_dim 64 or 128; 1 <= kv_heads <= 256, 1 to 64 query heads to each; 1 to
 * 1,024 sequences; up to 2^24 rows and positions in any one call. A call with
 * no rows is valid and needs no data pointers. None of the calls changes its
 * inputs.
 *
 * Sequences. Rows offsets[s] .. offsets[s + 1] - 1 of a call (offsets int32
 * [n_seqs + 1] on the device, ascending from 0) belong to sequence s, whose
 * length is len: they are its LAST positions, row offsets[s] + i position
 * p = len - n + i of n rows. Offsets outside [0, rows] count as the nearer end.
 * Rows from offsets[n_seqs] on belong to no sequence: nothing of theirs is
 * written, and what they hold changes no result. (It may be read, so all rows
 * of q, k and v must be memory that a kernel can read, as must rows at negative
 * positions and keys past k_offsets[n_seqs].)
 *
 * Visibility. The query at position p sees positions below
 *   block 0:      len                    (all of them)
 *   block n >= 1: min(len, (p / n + 1) n)  (its own block of n and what lies
 *                 before; 1: causal; 32: block-causal), none if p < 0
 * With z_j = scale * q . k_j over the positions it sees (scale finite, > 0):
 *   out = bf16(sum_j softmax(z)_j v_j),  lse = ln sum_j e^z_j
 * A query that sees nothing, or whose z are all -inf, gets out 0 and lse -inf.
 * Scores, softmax statistics and sums are fp32; the softmax's numerators are
 * rounded to the products' 16-bit type. What a query does not see does not
 * change its results, whatever it holds. Outputs must not overlap inputs, nor
 * each other. The results of a call do not change from run to run.
 *
 * One workspace may serve calls of both attention operations, of different
 * shapes, one after the other, if it is large enough for each. */

/* Strided rows of heads (bf16 unless a call says otherwise): row i, head h at
 * element i * row_stride + h * head_stride, head_dim contiguous elements. data
 * and the strides in bytes are multiples of 16; a stride is at least head_dim
 * where there is more than one row (head), at most 2^36 elements. */
typedef struct {
    const void* data;
    int64_t row_stride;
    int64_t head_stride;
} clover_rows;

/* A paged cache of keys and values in the CLOVER_FP4_NV format (e2m1 codes, an
 * e4m3 scale for 16 elements). pages: uint8
 * [n_pages][kv_heads][page_tokens / 16][18 head_dim], 16-byte aligned: the
 * tokens of a page in sixteens, each 16 rows of key codes (head_dim / 2 bytes,
 * the even element in the low nibble), 16 rows of key scales (head_dim / 16
 * bytes), and the same of the values. Keys stand for code * scale * 2^k_exp,
 * values for code * scale * 2^v_exp. page_tokens: a multiple of 16, 16 to
 * 65,536; 1 <= n_pages; |k_exp|, |v_exp| <= 64. */
typedef struct {
    uint8_t* pages;
    int32_t n_pages;
    int32_t page_tokens;
    int32_t kv_heads;
    int32_t head_dim;
    int32_t k_exp;
    int32_t v_exp;
} clover_kv_cache;

/* Sequences of a cache: offsets as above, lens int32 [n_seqs] their lengths
 * INCLUDING the call's rows (below 0 counts as 0, past the table's
 * max_pages * page_tokens, which may not exceed 2^24, as that), table int32
 * [n_seqs][max_pages] the page of positions j * page_tokens and on. All on the
 * device. A page id outside [0, n_pages) stands for no page: nothing is
 * written to it, its positions read as zeros and no query sees them. */
typedef struct {
    const int32_t* offsets;
    const int32_t* lens;
    const int32_t* table;
    int32_t n_seqs;
    int32_t max_pages;
} clover_kv_seqs;

/* Bytes of one page. Returns 0 for an unsupported shape. Host-only. */
size_t clover_kv_page_bytes(int32_t page_tokens, int32_t kv_heads, int32_t head_dim);

/* Quantises rows of keys and values (type fp32 or bf16) into the cache, at the
 * positions the rows have. Codes and scales as clover_quantize_fp4 (NV) gives
 * them with scale_exp k_exp or v_exp; a block of 16 with a NaN or an infinity
 * becomes NaN. Rows at negative positions are left out. Two rows of a call must
 * not have the same place (a page listed twice). */
int clover_kv_write(const clover_kv_cache* cache, const clover_kv_seqs* seqs, const clover_rows* k, const clover_rows* v,
                    int32_t type, int32_t n_rows, clover_stream_t stream);

/* The other way: k_out, v_out bf16 [n_rows][kv_heads][head_dim] receive what
 * the positions of the rows stand for (exact unless it leaves bf16's range),
 * zeros at negative positions. With n = len, a whole sequence. */
int clover_kv_read(const clover_kv_cache* cache, const clover_kv_seqs* seqs, uint16_t* k_out, uint16_t* v_out,
                   int32_t n_rows, clover_stream_t stream);

/* Bytes of workspace clover_kv_attention needs for up to n_rows rows of n_seqs
 * sequences with a table of max_pages (no data pointer is looked at). Returns 0
 * for an unsupported shape. Host-only. */
size_t clover_kv_attention_workspace_bytes(const clover_kv_cache* cache, int32_t n_rows, int32_t q_heads,
                                           int32_t n_seqs, int32_t max_pages);

/* Attention of n_rows query rows over the cache (the rows' own keys and values
 * among it: write them first). q: bf16. out: bf16
 * [n_rows][q_heads][head_dim], 16-byte aligned. lse: fp32 [n_rows][q_heads] or
 * NULL. */
int clover_kv_attention(const clover_kv_cache* cache, const clover_kv_seqs* seqs, const clover_rows* q, int32_t n_rows,
                        int32_t q_heads, float scale, int32_t block, uint16_t* out, float* lse, void* workspace,
                        size_t workspace_bytes, clover_stream_t stream);

/* *status receives the device address, on the current device, of 256 bytes in
 * the library, zeroed when it is loaded, in which calls of both attention
 * operations record a wait that ran out beside their workspace's status word.
 * For callers whose workspaces do not outlive the call: clover_workspace_status
 * (with 256 bytes) reads and clears it. Enqueues nothing. */
int clover_attention_shared_status(void** status);

/* Packed prompts: query rows by offsets, keys and values by k_offsets (int32
 * [n_seqs + 1]; a sequence's len is its number of keys; the same array as
 * offsets where every position has a query). */
typedef struct {
    const int32_t* offsets;
    const int32_t* k_offsets;
    int32_t n_seqs;
} clover_prompt_seqs;

/* Bytes of workspace clover_prompt_attention needs for up to n_rows rows and
 * n_keys keys of n_seqs sequences. Returns 0 for an unsupported shape.
 * Host-only. */
size_t clover_prompt_attention_workspace_bytes(int32_t n_rows, int32_t n_keys, int32_t n_seqs, int32_t q_heads,
                                               int32_t kv_heads, int32_t head_dim);

/* Attention of n_rows query rows over n_keys key/value rows, bf16. out and lse
 * as in clover_kv_attention. */
int clover_prompt_attention(const clover_prompt_seqs* seqs, const clover_rows* q, const clover_rows* k,
                            const clover_rows* v, int32_t n_rows, int32_t n_keys, int32_t q_heads, int32_t kv_heads,
                            int32_t head_dim, float scale, int32_t block, uint16_t* out, float* lse, void* workspace,
                            size_t workspace_bytes, clover_stream_t stream);

/* Library version as major*10000 + minor*100 + patch. */
int32_t clover_version(void);

#ifdef __cplusplus
}
#endif

#endif /* CLOVER_H_ */
