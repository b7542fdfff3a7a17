/*
 * moegg.h -- C ABI of libmoegg: the contiguous grouped block-scaled GEMM used
 * by MoE expert layers, with its fused epilogue, for AMD Instinct MI355X
 * (gfx950).
 *
 * What one call computes (cuDNN frontend pages "Grouped GEMM + Quant (SM100)",
 * "Grouped GEMM + SwiGLU (SM100)", "Grouped GEMM + sReLU (SM100)" and
 * "Grouped GEMM + dGLU (SM100)", §Equations of each):
 *
 *   rows m of A in [padded_offsets[g-1], padded_offsets[g]) belong to expert g
 *   acc[m,n] = sum_k dequant(A[m,k], SFA) * dequant(B[g,n,k], SFB)
 *   C = alpha_g * acc                       (forward activations)
 *   R = alpha_g^2 * acc                     (backward activations)
 *   then the activation / gating epilogue selected by `act`, and the output
 *   formatting selected by `d_dtype`:
 *     BF16  D (round to nearest even) + per-group amax = max |D| (fp32, before
 *           rounding) over the group's rows and all output columns;
 *     E4M3  D and D_col, the same logical output quantised over 32-column row
 *           blocks (SFD_row) and 32-row column blocks (SFD_col):
 *           SFD = smallest power of two >= norm_const * amax_blk / 448 (E8M0
 *           byte, 0 for an all-zero block), D_q = E4M3_rne(D * norm_const / SFD).
 *
 * Layouts ("logical" layouts defined by this library; every tensor is dense,
 * row-major, with no padding between rows):
 *   A       (valid_m, K)   E4M3 or E5M2 codes, or (valid_m, K/2) packed E2M1 pairs
 *                          (the even K element in the low nibble), or BF16
 *   B       (L, N, K)      same encoding as A, K contiguous ("K-major")
 *   SFA     (valid_m, K/32) E8M0 bytes, row-major: byte kb of row r (the
 *           scale of A[r, 32 kb .. 32 kb + 31]) at r * K/32 + kb (MX formats
 *           only; "Grouped GEMM + Quant (SM100)", §Shapes, SFA)
 *   SFB     (L, N, K/32) E8M0 bytes, row-major: expert g's row n at
 *           (g * N + n) * K/32 ("Grouped GEMM + Quant (SM100)", §Shapes, SFB)
 *   With sf_layout = MOEGG_SF_KPLANES the same bytes come instead as K-block
 *   planes of 32-bit words, (K/128, rows, 4): byte kb of row r at
 *   4 * ((kb / 4) * rows + r) + kb % 4 (rows = valid_m for SFA, L * N for a
 *   dense SFB, N for one expert's discrete SFB).  A plane holds the scales of
 *   128 consecutive K elements of every row, so those of a row tile for one
 *   K-step are contiguous and the kernel fetches them in whole cache lines
 *   (the pages' own kernels likewise take scale factors in a tiled layout of
 *   their own, §Shapes and Divisibility).  moegg_sf_to_kplanes converts.
 *   Discrete weights (the pages' b_ptrs / sfb_ptrs mode, "Grouped GEMM +
 *   sReLU (SM100)", §Discrete-weight wrapper): instead of B and SFB the
 *   caller passes device arrays of L device pointers; b_ptrs[g] points to
 *   expert g's (N, K) weights in B's encoding and sfb_ptrs[g] (MX only) to
 *   its (N, K/32) row-major scales (or (K/128, N, 4) planes with
 *   MOEGG_SF_KPLANES).  Each pointer must be 16-byte aligned
 *   (the kernel ignores its low 4 bits); entries of experts with no rows are
 *   never read.
 *   padded_offsets (L) int32, cumulative group ends; padded_offsets[L-1] <=
 *                          valid_m (the pages: equal to it; where it is less,
 *                          the rows behind it are neither read nor written);
 *                          every entry a multiple of m_aligned and
 *                          nondecreasing (empty groups repeat the previous end)
 *   alpha, beta (L) fp32; prob (valid_m) fp32; norm_const (1) fp32
 *   C       (valid_m, N) BF16                      [optional forward output]
 *   D, D_col (valid_m, N_out) BF16 or E4M3 codes   N_out = N/2 for SwiGLU and
 *                                                  GeGLU, 2N for dSwiGLU and
 *                                                  dGeGLU, else N
 *                                                  (dC for the backward
 *                                                  activations)
 *   SFD_row (valid_m, N_out/32) E8M0; SFD_col (N_out, valid_m/32) E8M0
 *   amax    (L) fp32, written by the call (zero-filled first); for dSwiGLU /
 *           dGeGLU with MX operands and a BF16 dC, (L, 2): the max |dC| of
 *           the first and of the second blocks of the pairs over the group's
 *           rows (the block-scaled dGLU contract's amax of shape (L, 2, 1);
 *           which quantity each entry holds is this library's reading)
 *   C_in    saved forward pre-activation, BF16: (valid_m, 2N) [dSwiGLU, dGeGLU]
 *           or (valid_m, N) [dsReLU]
 *   dprob   (valid_m) fp32, caller-zeroed, accumulated with atomics [dSwiGLU, dsReLU,
 *           dGeGLU]
 *
 * Ownership: every pointer is a caller-owned device pointer (except the
 * problem/args structs, which are host memory read during the call only).
 * The library keeps no pointer after a call returns and allocates no device
 * memory.  Buffers must stay alive and unchanged until the stream has run
 * the work.  Calls are asynchronous on `stream` (a hipStream_t; NULL = the
 * null stream).
 *
 * Errors: every shape, dtype, alignment and presence rule is checked on the
 * host before any HIP call; a failing call returns a status and enqueues
 * nothing.  padded_offsets values are device data and are not read on the
 * host (moegg_check_offsets is the opt-in, synchronising validator).
 * moegg_last_error() returns a thread-local text describing the last failure.
 */
#ifndef MOEGG_H_
#define MOEGG_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOEGG_ABI_VERSION 5 /* counts changes of the structs and of what a function takes, not new functions */

typedef enum moegg_status {
  MOEGG_OK = 0,
  MOEGG_ERROR_INVALID_VALUE = 1, /* bad shape, dtype combination, NULL where required */
  MOEGG_ERROR_MISALIGNED = 2,    /* pointer not 16-byte aligned */
  MOEGG_ERROR_NOT_SUPPORTED = 3, /* valid per the pages, not supported by this library (e.g. K % 128 != 0) */
  MOEGG_ERROR_LAUNCH = 4         /* a HIP runtime call failed */
} moegg_status;

typedef enum moegg_dtype {
  MOEGG_DT_NONE = 0,
  MOEGG_DT_E4M3 = 1,   /* OCP E4M3FN: A/B operands (MXFP8) or D/D_col outputs */
  MOEGG_DT_E2M1X2 = 2, /* packed OCP E2M1 pairs: A/B operands (MXFP4) */
  MOEGG_DT_BF16 = 3,   /* A/B operands (dense BF16 backend) or C / D outputs */
  MOEGG_DT_E5M2 = 4,   /* OCP E5M2: A/B operands (MXFP8, "Grouped GEMM + Quant", §Data Types) */
  MOEGG_DT_F32 = 5     /* fp32: layer operators only (router logits, linear's y and dw, the norm's stream) */
} moegg_dtype;

typedef enum moegg_sf_layout {
  MOEGG_SF_ROW_MAJOR = 0, /* SFA (valid_m, K/32), SFB (L, N, K/32): the default */
  MOEGG_SF_KPLANES = 1    /* SFA (K/128, valid_m, 4), SFB (K/128, L*N, 4) 32-bit word planes */
} moegg_sf_layout;

typedef enum moegg_act {
  MOEGG_ACT_NONE = 0,    /* D = prob * C            ("Grouped GEMM + Quant", Step 2)        */
  MOEGG_ACT_SWIGLU = 1,  /* D = prob * X_b * swish(G_b), pairs [X_b|G_b] of 32 columns
                            ("Grouped GEMM + SwiGLU", Step 2)                               */
  MOEGG_ACT_SRELU = 2,   /* D = prob * relu(C)^2, optional tanh soft clamp s
                            ("Grouped GEMM + sReLU", §Equations / §Tanh soft clamp)          */
  MOEGG_ACT_DSWIGLU = 3, /* dC = [d_input|d_gate] from R and beta*C_in, dprob += row sums
                            ("Grouped GEMM + dGLU", BF16 contract and block-scaled contract,
                            dSwiGLU): BF16 operands -> BF16 dC; MX operands -> BF16 dC + amax
                            (L, 2), or E4M3 dC as D/D_col with SFD_row/SFD_col             */
  MOEGG_ACT_DSRELU = 4,  /* sReLU backward: R = alpha_g^2 acc, C_in the saved forward C
                            (N wide, no beta), dC = R prob f'(C), dprob += sum R f(C),
                            f(C) = (s tanh(relu(C)/s))^2 or relu(C)^2 for s = 0 (derived
                            from "Grouped GEMM + sReLU", §Equations / §Tanh soft clamp; its
                            backward page is not among the sources).  Output formats as
                            dSwiGLU, amax (L) for a BF16 dC with MX operands              */
  MOEGG_ACT_GEGLU = 5,   /* D = gamma prob (U_b + offset) G_b sigmoid(a G_b), pairs [G_b|U_b]
                            of 32 columns, gate first, both clamped to [clamp_min, clamp_max]
                            ("Grouped GEMM + GLU + Hadamard", §Equations, GeGLU; the page's
                            constants are a = 1.702, offset = 1)                          */
  MOEGG_ACT_DGEGLU = 6,  /* dGeGLU backward: C_in pairs [gate_b|up_b], dC = [dgate_b|dup_b],
                            gate clamped above at clamp_max, up to [clamp_min, clamp_max],
                            dprob += row sums ("Grouped GEMM + dGLU", dGeGLU equations; the
                            page's defaults a = 1.702, offset = 1, clamps -7 / 7).  Output
                            formats as dSwiGLU (amax (L, 2) = [dgate, dup] blocks)        */
  MOEGG_ACT_GELU = 7     /* y = z / 2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))): moegg_linear only */
} moegg_act;

/* Problem description (host struct). */
typedef struct moegg_problem {
  int32_t num_groups;   /* L, 1..1024 ("Shapes and Divisibility": expert count <= 1024) */
  int32_t m_aligned;    /* group row alignment; multiple of 128 here                     */
  int64_t valid_m;      /* rows of A and of every row tensor: padded_offsets[L-1], or more (rows
                           behind the last group are left as they were); multiple of
                           m_aligned, < 2^31 here                                         */
  int32_t n;            /* GEMM N (rows of each expert's B); multiple of 32, <= 2^20 here
                           (64 for SwiGLU / GeGLU)                                        */
  int32_t k;            /* reduction length K; multiple of 128 bytes per row here (128
                           E4M3 / E5M2, 256 E2M1, 64 BF16 elements), <= 2^20             */
  int32_t ab_dtype;     /* moegg_dtype of A and B: E4M3 | E5M2 | E2M1X2 | BF16            */
  int32_t c_dtype;      /* NONE (C not written) | BF16                                    */
  int32_t d_dtype;      /* BF16 (needs amax) | E4M3 (needs SFD_row, SFD_col, norm_const)  */
  int32_t act;          /* moegg_act                                                      */
  float srelu_tanh_s;   /* sReLU soft clamp s; 0 = plain relu^2                           */
  /* GeGLU / dGeGLU constants (read for those activations only; no implicit
   * defaults: the pages' values are gamma 1, geglu_alpha 1.702, linear_offset 1,
   * dGeGLU clamps -7 / 7; +-INFINITY disables a clamp) */
  float glu_gamma;      /* GeGLU output scale                                             */
  float geglu_alpha;    /* sigmoid input scale                                            */
  float linear_offset;  /* offset added to the (clamped) up branch                       */
  float glu_clamp_min;  /* lower clamp (GeGLU: both halves; dGeGLU: up)                   */
  float glu_clamp_max;  /* upper clamp (both halves, both directions)                     */
  int32_t sf_layout;    /* moegg_sf_layout of SFA / SFB (MX operands; 0 = row-major)       */
} moegg_problem;

/* Tensor pointers (device memory, caller-owned).  NULL where not used. */
typedef struct moegg_args {
  const void* a;
  const void* b;
  const uint8_t* sfa;            /* MX operands only; (valid_m, K/32) E8M0 (or planes, sf_layout) */
  const uint8_t* sfb;            /* MX operands only; (L, N, K/32) E8M0 (or planes, sf_layout) */
  const int32_t* padded_offsets;
  const float* alpha;
  const float* prob;             /* required ("prob ... Required", Quant page) */
  const float* beta;             /* dSwiGLU only (L) */
  const float* norm_const;       /* required iff d_dtype == E4M3 */
  const void* c_in;              /* backward: saved forward C, BF16 (valid_m, 2N) or (valid_m, N) dsReLU */
  void* c;                       /* optional C output (c_dtype BF16) */
  void* d;                       /* D (or dC for the backward activations) */
  void* d_col;                   /* E4M3 only */
  uint8_t* sfd_row;              /* E4M3 only */
  uint8_t* sfd_col;              /* E4M3 only */
  float* amax;                   /* BF16 D: (L), or (L, 2) for dSwiGLU / dGeGLU with MX operands */
  float* dprob;                  /* backward activations, caller-zeroed */
  const void* const* b_ptrs;     /* discrete weights instead of b: (L) device array, 8-byte aligned */
  const uint8_t* const* sfb_ptrs;/* discrete weights, MX only, instead of sfb: (L) device array */
} moegg_args;

/* Validate problem + pointers on the host.  No HIP call.  MOEGG_OK if
 * moegg_run would launch (or, for valid_m == 0, only zero-fill amax).
 * The rules are the pages' ("Grouped GEMM + Quant (SM100)", §Support Surface
 * and Constraints: §Layouts and Strides (16-byte alignment), §Data Types and
 * §Additional Type Constraints (A and B of one dtype, the SFD trio together),
 * §Scale Factor Output Requirements (amax with a BF16 D), §Shapes and
 * Divisibility (L <= 1024, groups aligned to m_aligned; that valid_m covers
 * padded_offsets[L-1] is device data and not checked here); "Grouped GEMM +
 * dGLU (SM100)", §Support Surface and Constraints for the backward tensors), plus this library's own limits,
 * reported as MOEGG_ERROR_NOT_SUPPORTED (K a multiple of 128 bytes per row,
 * N a multiple of 32, m_aligned a multiple of 128). */
moegg_status moegg_check(const moegg_problem* problem, const moegg_args* args);

/* Validate (as moegg_check), then enqueue the whole path on `stream`
 * (hipStream_t): the amax zero-fill (when amax is used) and the grouped GEMM
 * with its epilogue ("Grouped GEMM + Quant (SM100)", §Equations, Steps 1-3, and
 * the other pages' §Equations).  valid_m == 0: returns MOEGG_OK after
 * enqueuing only the amax zero-fill. */
moegg_status moegg_run(const moegg_problem* problem, const moegg_args* args, void* stream);

/* Opt-in validator of device padded_offsets (synchronises `stream`) against
 * the pages' offset rules ("Grouped GEMM + Quant (SM100)", §Shapes: the
 * cumulative sum of aligned group sizes with valid_m its last entry; §Shapes
 * and Divisibility: every group aligned to m_aligned): entries nondecreasing,
 * multiples of m_aligned, last == valid_m.  MOEGG_OK or
 * MOEGG_ERROR_INVALID_VALUE (MOEGG_ERROR_LAUNCH if the copy fails).  Where
 * valid_m is a capacity (moegg_sort_rows) and not the rows in use, which only
 * the device knows, this is stricter than moegg_run: a plan of moegg_sort is
 * checked with its last offset as valid_m. */
moegg_status moegg_check_offsets(const moegg_problem* problem, const int32_t* padded_offsets,
                                 void* stream);

/* Lay out E8M0 scale bytes given row-major as (rows, K/32) (SFA with rows =
 * valid_m, a dense SFB with rows = L * N, one expert's SFB with rows = N)
 * as the K-block word planes (K/128, rows, 4) that MOEGG_SF_KPLANES reads:
 * dst[4 * ((kb / 4) * rows + r) + kb % 4] = src[r * K/32 + kb].  The layout is
 * this library's; the scale values follow "Grouped GEMM + Quant (SM100)",
 * §Shapes (SFA, SFB: one E8M0 byte per 32 K elements).  Enqueued on `stream`
 * with no allocation and no synchronisation (capturable).  k must be a
 * positive multiple of 128, rows >= 0 (0: nothing enqueued); src and dst are
 * caller-owned device buffers of rows * K/32 bytes, 16-byte aligned, not
 * overlapping.  Returns MOEGG_OK, MOEGG_ERROR_INVALID_VALUE,
 * MOEGG_ERROR_MISALIGNED or MOEGG_ERROR_LAUNCH. */
moegg_status moegg_sf_to_kplanes(const uint8_t* src, uint8_t* dst, int64_t rows, int32_t k, void* stream);

/* ==========================================================================
 * Layer operators: what stands around the grouped product in an MoE layer.
 * The norm before it, the router's choice, tokens sorted by expert and back,
 * and the matrix product with bias, activation and residual, each with its
 * gradient; and activations kept in 8 bits for those gradients.
 *
 * They follow the conventions above: caller-owned dense row-major device
 * tensors (16-byte aligned; vectors 4-byte aligned), no device allocation,
 * asynchronous on `stream`, capturable (kernels only), every argument checked
 * on the host before any HIP call.  Values in index tensors are device data:
 * an index out of range is never followed (each function says what it counts
 * as).  An output shares no memory with an input, a workspace or another
 * output, but where a function says so.  A workspace belongs to one call at a
 * time: calls that may run at the same time (other streams, graphs replayed
 * side by side) need their own.  A problem that would need more than 2^32
 * threads in a launch is refused.
 * Results do not depend on the order in which workgroups run.
 * ========================================================================== */

typedef enum moegg_score {
  MOEGG_SCORE_SOFTMAX = 0, /* p = softmax over the experts */
  MOEGG_SCORE_SIGMOID = 1  /* p_e = 1 / (1 + exp(-logit_e)) */
} moegg_score;

typedef struct moegg_route_problem {
  int64_t num_tokens;   /* T >= 0                                              */
  int32_t num_experts;  /* E, 1..1024                                          */
  int32_t top_k;        /* 1..min(E, 32)                                       */
  int32_t dtype;        /* logits (and dlogits): BF16 | F32                    */
  int32_t score;        /* moegg_score                                         */
  int32_t renormalise;  /* weights divided by the sum of the chosen scores     */
  float scale;          /* factor of the weights; finite                       */
} moegg_route_problem;

/* Router: the top_k experts of every token and their weights.
 *   key_e   = logit_e, or p_e + bias_e (evaluated in 64 bits) where bias is given: the bias
 *             (E, fp32) steers the choice and not the weights
 *   ids     (T, top_k) int32: experts of the largest keys, largest first, ties to the lowest index
 *   weights (T, top_k) fp32: scale p_j, or scale p_j / sum_i p_i over the chosen with renormalise
 * Experts with a logit of -infinity or NaN (or a key of NaN or -infinity) are
 * never chosen; where fewer than top_k remain, the ids that are left are -1
 * with weight 0.  +infinity counts as the largest finite number.  A NaN logit
 * makes the token's weights NaN where they come from a softmax over all
 * experts (no renormalise), and has no other effect. */
moegg_status moegg_route(const moegg_route_problem* problem, const void* logits, const float* bias, int32_t* ids,
                         float* weights, void* stream);

/* Gradient of moegg_route's weights: dlogits (T, E, dtype of the logits) from
 * dweights (T, top_k) and the ids that moegg_route returned for these logits
 * (ids outside 0..E-1 have no gradient; an id that appears twice in a token
 * counts twice).  The choice itself, and so the bias, has no gradient. */
moegg_status moegg_route_backward(const moegg_route_problem* problem, const void* logits, const int32_t* ids,
                                  const float* dweights, void* dlogits, void* stream);

/* Router that chooses groups of experts first: moegg_route among the experts of
 * the top_groups groups with the largest scores (ties to the lowest group).
 * Experts [i, i + 1) E / num_groups are group i.  A group's score is the sum
 * of its `best` largest p_e + bias_e (p_e without a bias), or with best = 1 and
 * no bias its largest logit, among the experts that can be chosen (where fewer
 * than `best` can, of those; a group of none comes last).  Scores are decided
 * in 64 bits.  p, weights and what cannot be chosen are as in moegg_route (p
 * over all experts, of all groups); the gradient is moegg_route_backward with
 * these ids. */
typedef struct moegg_route_groups {
  int32_t num_groups;   /* 1..64, a divisor of E                               */
  int32_t top_groups;   /* 1..num_groups                                       */
  int32_t best;         /* 1 or 2                                              */
} moegg_route_groups;

moegg_status moegg_route_grouped(const moegg_route_problem* problem, const moegg_route_groups* groups, const void* logits,
                                 const float* bias, int32_t* ids, float* weights, void* stream);

typedef struct moegg_sort_problem {
  int64_t num_tokens;   /* T >= 0                                              */
  int32_t top_k;        /* slots per token, 1..32; slot t * top_k + j          */
  int32_t num_experts;  /* L, 1..1024                                          */
  int32_t m_aligned;    /* rows of an expert are padded to a multiple of this: 1..65536
                           (128 or a multiple for moegg_run, 1 for moegg_linear) */
  int64_t rows;         /* rows of the sorted tensors, >= moegg_sort_rows()    */
} moegg_sort_problem;

/* Rows that any routing of the problem's slots fits into (a multiple of
 * m_aligned): rows is a host number, where the rows in use,
 * padded_offsets[L-1], are known to the device alone.  -1 for an invalid
 * problem or one with 2^31 rows or more.  moegg_run takes this number as
 * valid_m: it works through the rows that padded_offsets names and leaves
 * those behind the last expert as they were. */
int64_t moegg_sort_rows(const moegg_sort_problem* problem);
/* Bytes of workspace of moegg_sort (may be 0); -1 for an invalid problem. */
int64_t moegg_sort_workspace(const moegg_sort_problem* problem);

/* Slots sorted by expert, stable (an expert's rows in the order of their slots).
 *   ids (T, top_k) int32; any value outside 0..L-1 drops the slot
 *   padded_offsets (L) int32: end of every expert's padded rows (moegg_run's layout)
 *   row_of (T, top_k) int32: the slot's row, -1 if dropped
 *   slot_of (rows) int32: the row's slot, -1 for padding and for rows behind the last expert
 *   weights (T, top_k) fp32 and prob (rows) fp32, both or neither: prob[row] = weights[slot], 0
 *   where there is no slot (moegg_run's prob) */
moegg_status moegg_sort(const moegg_sort_problem* problem, const int32_t* ids, const float* weights,
                        int32_t* padded_offsets, int32_t* row_of, int32_t* slot_of, float* prob, void* workspace,
                        int64_t workspace_bytes, void* stream);

typedef struct moegg_exchange_problem {
  int64_t num_tokens;   /* T >= 0                                              */
  int64_t rows;         /* as sorted                                           */
  int32_t top_k;
  int32_t num_experts;  /* L                                                   */
  int32_t width;        /* H: multiple of 8; of 128 for MX rows (256 for E2M1X2), <= 2^20 */
  int32_t dtype;        /* of the rows written: BF16 | E4M3 | E5M2 | E2M1X2    */
  int32_t sf_layout;    /* moegg_sf_layout of the scales of MX rows            */
} moegg_exchange_problem;

/* rows[row_of[t, j]] = x[t]: x (T, H) BF16; out (rows, H) in `dtype`, with E8M0
 * scales in sf for the MX types: (rows, H/32), or (H/128, rows, 4) planes.
 * These are moegg_run's A and SFA.  A block of 32 is scaled by the smallest
 * power of two >= amax / q_max (448, 57344 or 6) and rounded to nearest even;
 * a block of zeros has scale byte 0, a block with a NaN or an infinity has
 * zero codes and scale byte 255 (NaN).  Padding rows inside the experts'
 * rows become zero (scale byte 0); rows behind the last expert are left as
 * they were. */
moegg_status moegg_dispatch(const moegg_exchange_problem* problem, const void* x, const int32_t* row_of,
                            const int32_t* slot_of, const int32_t* padded_offsets, void* out, uint8_t* sf,
                            void* stream);

/* y[t] = residual[t] + sum_j weights[t, j] rows_in[row_of[t, j]], summed in fp32
 * in the order residual last, rounded once: rows_in (rows, H) BF16, weights
 * (T, top_k) fp32 or NULL (ones), residual (T, H) BF16 or NULL, y (T, H) BF16
 * (may be residual itself).  Dropped slots add nothing.  `dtype` must be BF16.
 * Without weights this is also the gradient of moegg_dispatch. */
moegg_status moegg_combine(const moegg_exchange_problem* problem, const void* rows_in, const int32_t* row_of,
                           const float* weights, const void* residual, void* y, void* stream);

/* Gradient of moegg_combine: out[row_of[t, j]] = weights[t, j] dy[t] in `dtype`
 * (padding and rows behind the last expert as in moegg_dispatch), and, where
 * dweights (T, top_k) is given, dweights[t, j] = sum_h dy[t, h] rows_in[row_of[t, j], h]
 * (0 for a dropped slot); rows_in is needed for it and otherwise NULL.  out
 * may not overlap rows_in.  The residual's gradient is dy itself. */
moegg_status moegg_combine_backward(const moegg_exchange_problem* problem, const void* dy, const int32_t* row_of,
                                    const int32_t* slot_of, const int32_t* padded_offsets, const void* rows_in,
                                    const float* weights, void* out, uint8_t* sf, float* dweights, void* stream);

/* values[slot] = rows_values[row_of[slot]] (0 for a dropped slot): fp32 numbers
 * of the rows back in the order of the slots (moegg_run's dprob -> the gradient
 * of the weights). */
moegg_status moegg_unsort(const float* rows_values, const int32_t* row_of, float* values, int64_t num_slots,
                          int64_t rows, void* stream);

/* Matrix product with bias, activation and residual, dense or grouped.
 *   z = x w_g^T + bias_g;  c = bf16(z);  y = act(z) + residual
 * for the rows [offsets[g-1], offsets[g]) of group g (any nondecreasing ends,
 * no alignment; of ends that decrease or leave the rows none is followed outside
 * them, but what the rows then hold is not defined; y may be residual itself,
 * both BF16), or for all m rows where offsets is NULL (num_groups 1).
 * act: NONE, SRELU (relu(z)^2), GELU, or SWIGLU on [X | G] pairs of 32 columns
 * as in moegg_run (N_out = n / 2, else N_out = n).  Sums are fp32.  A NaN in z
 * is a NaN in y, whatever the activation. */
typedef struct moegg_linear_problem {
  int64_t m;            /* rows, 0..2^31-1024                                  */
  int32_t n;            /* multiple of 8 (64 for SWIGLU), <= 2^20              */
  int32_t k;            /* multiple of 8, <= 2^20                              */
  int32_t num_groups;   /* 1..1024                                             */
  int32_t act;          /* moegg_act                                           */
  int32_t dtype;        /* y (forward) or dw (backward): BF16 | F32            */
} moegg_linear_problem;

typedef struct moegg_linear_args {
  const void* x;          /* (m, k) BF16                                       */
  const void* w;          /* (L, n, k) BF16                                    */
  const float* bias;      /* (L, n) fp32 or NULL                  [forward]    */
  const void* residual;   /* (m, N_out) BF16 or NULL              [forward]    */
  const int32_t* offsets; /* (L) int32 group ends, or NULL                     */
  void* y;                /* (m, N_out)                           [forward]    */
  void* c;                /* (m, n) BF16: forward: written if not NULL; backward: read, unless act is NONE */
  const void* dy;         /* (m, N_out) BF16                      [backward]   */
  void* dx;               /* (m, k) BF16 or NULL                  [backward]   */
  void* dw;               /* (L, n, k) or NULL                    [backward]   */
  float* db;              /* (L, n) fp32 or NULL                  [backward]   */
  void* workspace;        /* 16-byte aligned, moegg_linear*_workspace() bytes (NULL for 0) */
  int64_t workspace_bytes;
} moegg_linear_args;

/* Workspace bytes of a forward / backward call; -1 for an invalid problem.
 * The backward's depends on which of dx, dw and db are asked for (flags 1, 2, 4). */
int64_t moegg_linear_workspace(const moegg_linear_problem* problem);
int64_t moegg_linear_backward_workspace(const moegg_linear_problem* problem, int32_t want);

/* Forward.  Rows behind the last group are left as they were.  m == 0:
 * nothing is enqueued. */
moegg_status moegg_linear(const moegg_linear_problem* problem, const moegg_linear_args* args, void* stream);

/* Gradients: dz = dy act'(c), rounded to BF16 as the operand of both products;
 * dx = dz w_g (rows behind the last group left as they were); dw_g = dz^T x
 * and db_g = column sums of the unrounded dz over the group's rows (zero for
 * an empty group; rows behind the last group are not read).  Whatever is NULL
 * of dx, dw and db is not computed (all three may be NULL where m is 0, else
 * one is required).  The residual's gradient is dy itself.  A
 * NaN in c is a NaN in dz. */
moegg_status moegg_linear_backward(const moegg_linear_problem* problem, const moegg_linear_args* args, void* stream);

/* moegg_linear with c kept in 8 bits, and moegg_linear_backward from an input
 * or a pre-activation kept in 8 bits.  8-bit tensors are MX rows: E4M3 or E5M2
 * codes with an E8M0 byte for every 32 columns, as moegg_dispatch,
 * moegg_rms_norm and moegg_quantise write them (and as moegg_run takes its A).
 * c is formed from the unrounded z, a block with a NaN or an infinity as in
 * moegg_dispatch; it is read back as the values that its codes stand for.  x
 * is read as those values in BF16 (exact but below 2^-126), the operand of dw. */
typedef struct moegg_linear_saved {
  int32_t x_dtype;        /* of args.x: BF16, or in the backward E4M3 | E5M2: codes (m, k), k a multiple of 32 */
  int32_t x_sf_layout;    /* moegg_sf_layout of x_sf (K-block planes: k a multiple of 128) */
  int32_t c_dtype;        /* of args.c: BF16, or E4M3 | E5M2: codes (m, n), n a multiple of 32 */
  int32_t reserved;       /* 0                                                 */
  const uint8_t* x_sf;    /* (m, k/32) or (k/128, m, 4); NULL for a BF16 x      */
  uint8_t* c_sf;          /* (m, n/32): written by the forward, read by the backward; NULL for a BF16 c */
} moegg_linear_saved;

/* Workspace bytes; -1 for an invalid problem. */
int64_t moegg_linear_saving_workspace(const moegg_linear_problem* problem, const moegg_linear_saved* saved);
int64_t moegg_linear_saved_backward_workspace(const moegg_linear_problem* problem, const moegg_linear_saved* saved,
                                              int32_t want);
/* As moegg_linear; args.c is required where c_dtype is one of 8 bits. */
moegg_status moegg_linear_saving(const moegg_linear_problem* problem, const moegg_linear_args* args,
                                 const moegg_linear_saved* saved, void* stream);
/* As moegg_linear_backward. */
moegg_status moegg_linear_saved_backward(const moegg_linear_problem* problem, const moegg_linear_args* args,
                                         const moegg_linear_saved* saved, void* stream);

/* Rows to 8 bits and back: x (rows, width) BF16 or F32 (`x_dtype`) to codes of
 * `dtype` (E4M3 | E5M2) and E8M0 scales sf, (rows, width/32) or with
 * MOEGG_SF_KPLANES (width/128, rows, 4), scaled and rounded as in
 * moegg_dispatch; and codes and scales to x, rounded once to nearest even (a
 * scale byte of 255 stands for NaN).  width: a multiple of 32 (planes: 128),
 * <= 2^20; rows: 0..2^31-1.  The operand that is not written is read only. */
moegg_status moegg_quantise(const void* x, int32_t x_dtype, int64_t rows, int32_t width, int32_t dtype, int32_t sf_layout,
                            uint8_t* codes, uint8_t* sf, void* stream);
moegg_status moegg_dequantise(const uint8_t* codes, const uint8_t* sf, int64_t rows, int32_t width, int32_t dtype,
                              int32_t sf_layout, void* x, int32_t x_dtype, void* stream);

/* Root-mean-square norm with the residual's addition:
 *   h = x + residual, rounded once to the stream's type (without a residual h is x)
 *   y = h / sqrt(mean(h^2) + eps) * weight
 * over each row of `width` columns, the norm of the h that is stored.  y comes
 * as BF16, as MX rows (codes with scales, scaled and rounded from the unrounded
 * y as in moegg_dispatch: moegg_run's A and SFA) or as both.  Sums are held in
 * 64 bits: no finite h overflows or vanishes in them.  The factors of one value, (h /
 * sqrt(...)) weight and in the gradient dy weight, are multiplied in fp32: a product
 * beyond its range is infinite (and its row's dx NaN), one below it 0.  A NaN or an
 * infinity in a row is one of that row alone. */
typedef struct moegg_norm_problem {
  int64_t rows;         /* 0..2^31-1                                           */
  int32_t width;        /* multiple of 8 (128 for MX rows, 256 for E2M1X2), <= 32768 */
  int32_t x_dtype;      /* x: BF16 | F32 (the stream's without a residual)     [forward] */
  int32_t stream_dtype; /* residual, h, dh and dx: BF16 | F32 (F32 where x is) */
  int32_t mx_dtype;     /* codes: NONE | E4M3 | E5M2 | E2M1X2                  [forward] */
  int32_t sf_layout;    /* moegg_sf_layout of sf                               [forward] */
  float eps;            /* > 0, finite                                         */
} moegg_norm_problem;

typedef struct moegg_norm_args {
  const void* x;          /* (rows, width)                                     [forward] */
  const void* residual;   /* (rows, width) or NULL                             [forward] */
  const float* weight;    /* (width) fp32                                      */
  void* h;                /* (rows, width): forward: written, with a residual (may be the residual itself),
                             NULL without one; backward: read (x where there was no residual) */
  void* y;                /* (rows, width) BF16; NULL: MX rows alone           [forward] */
  uint8_t* codes;         /* (rows, width) (E2M1X2: width / 2), with mx_dtype  [forward] */
  uint8_t* sf;            /* (rows, width/32) or (width/128, rows, 4)          [forward] */
  const void* dy;         /* (rows, width) BF16                                [backward] */
  const void* dh;         /* (rows, width) or NULL: what reaches h from elsewhere (the residual stream) [backward] */
  void* dx;               /* (rows, width) or NULL; may be dh itself           [backward] */
  float* dweight;         /* (width) fp32 or NULL                              [backward] */
  void* workspace;        /* 16-byte aligned (with dweight)                    [backward] */
  int64_t workspace_bytes;
} moegg_norm_args;

moegg_status moegg_rms_norm(const moegg_norm_problem* problem, const moegg_norm_args* args, void* stream);

/* Gradients: dx of x and of the residual alike (both are h's), dh included;
 * dweight = sum over the rows (zero without rows).  Whatever is NULL of dx and
 * dweight is not computed (both may be NULL where rows is 0, else one is
 * required).  The workspace is needed with dweight alone. */
int64_t moegg_rms_norm_backward_workspace(const moegg_norm_problem* problem);
moegg_status moegg_rms_norm_backward(const moegg_norm_problem* problem, const moegg_norm_args* args, void* stream);

/* Output width N_out for a problem (N/2 SwiGLU / GeGLU, 2N dSwiGLU / dGeGLU, else N);
 * -1 if invalid act. */
int64_t moegg_n_out(const moegg_problem* problem);

const char* moegg_status_string(moegg_status status);
const char* moegg_last_error(void);   /* thread-local detail of the last failure */
int moegg_abi_version(void);

/* Testing hook; no passage defines it and it changes no result.  Caps the
 * persistent workgroups that later moegg_run calls launch, from any thread
 * (0 or a negative value: no cap, the default of one workgroup per compute
 * unit).  With a small cap every workgroup walks many output tiles, so that a
 * problem small enough for a CPU reference still passes through every
 * tile-to-tile hand-off of the kernel.  Returns the previous cap. */
int moegg_set_grid_limit(int max_workgroups);

#ifdef __cplusplus
}
#endif

#endif /* MOEGG_H_ */
