/*
 * moe.h -- C ABI of the single-GPU forward pass of one routed
 * Mixture-of-Experts layer (GB300, sm_103a).
 *
 * The forward pass is five calls, made in this order on one stream:
 *
 *   moe_route_topk          softmax top-K routing of the router logits
 *   moe_permute             counts, offsets, row maps; dispatch of the
 *                           activations into the expert-grouped buffer
 *   moe_grouped_swiglu_gemm per-expert gate/up GEMM with SiLU(gate) * up
 *   moe_grouped_down_gemm   per-expert down GEMM
 *   moe_combine             weighted sum of each token's expert outputs
 *
 * Sources, by page title and section:
 *   "MoE inference and expert parallelism" (blog.vllbc.top): the routing
 *     section and Table 3-1 (softmax top-K with renormalisation, SwiGLU experts
 *     with W1/W3 = gate/up and W2 = down, moe_sum, DeepSeek-V3 shared expert,
 *     Eq. 12) and the forward-pass section (fused_topk -> moe_align_block_size
 *     -> W1/W3 GEMM -> activation -> W2 GEMM -> moe_sum).
 *   "Inference INFRA methodology (5): MoE inference -- Batch, DeepEP, DeepGEMM
 *     and load balancing" (yfxerp.com): section "DeepGEMM" (static
 *     [E_loc, M_max, K] buffer with a device-resident masked_m read at run
 *     time, no MMA for tiles that hold only padding, FP8 with the 128-wide K
 *     promotion to FP32, contiguous layout for prefill).
 *   "vLLM EPLB" (pnsm.cn): section 1.2 (physical_to_logical_map,
 *     logical_to_physical_map, logical_replica_count).
 *   "MoonEP: dynamic redundant experts" (wineandchord.com): sections "Why
 *     dynamic routing is hard" (counts sum to the routed records) and
 *     "Zero-copy and static buffer" (offsets / cu_seqlens, padding described
 *     by the plan).
 *
 * Conventions shared by every call
 *   - All data pointers are DEVICE pointers unless a comment says otherwise.
 *     The caller allocates and owns every buffer, including the workspace.
 *     The library never allocates, frees or synchronises; every call only
 *     enqueues kernels (and memsets) on `stream`, so a sequence of calls can be
 *     captured in a CUDA graph once the first call on the device has been made
 *     outside of capture (it caches device attributes).
 *   - Return status: checked on the host from the arguments and from the
 *     launch; nothing is enqueued when a call returns MOE_ERR_INVALID or
 *     MOE_ERR_UNSUPPORTED.  Data-dependent problems found on the device set
 *     bits of the caller's int32 `err_flag` (MOE_FLAG_*); tokens are never
 *     dropped silently.
 *   - Layouts are row-major.  Counts: T tokens, H hidden, I expert
 *     intermediate, E logical routed experts, K experts per token, P physical
 *     slots (P == E without a replica map), S = has_shared (0/1).  The shared
 *     expert, when present, is slot P.
 *   - Dtypes: bf16 is IEEE binary32's upper half, e4m3 is OCP FP8 E4M3,
 *     e2m1 is OCP FP4 E2M1 (weights only; the FP4 experts of "Inference INFRA
 *     methodology (5)", shape-evolution table, DS-V4-Pro row).
 *     mxfp4 is OCP Microscaling FP4: E2M1 codes in blocks of 32 along the
 *     reduced dimension that share one UE8M0 scale byte (see "MXFP4" below).
 *     Supported combinations (act / wt / out): F32/F32/F32, BF16/BF16/BF16,
 *     BF16/E4M3/BF16, BF16/E2M1/BF16, BF16/MXFP4/BF16.  `wt` is the type of
 *     the expert weights; the grouped activations Xg and Hg are of type wt,
 *     except that they are E4M3 when wt is E2M1.  Yg is F32 when wt is F32,
 *     else BF16.
 *   - e4m3 and e2m1 scales are fp32: weights one per 128x128 block
 *     ([slots][N/128][K/128]), grouped activations one per 1x128 group
 *     ([rows][cols/128]).  Quantised value = code * scale.
 *   - MXFP4: rows of K codes, packed as e2m1 weights are (K/2 bytes), and
 *     K/32 scale bytes per row, row-major ([rows][K/32]).  Scale byte s stands
 *     for 2^(s - 127); s = 255 stands for NaN.  Value = code * 2^(s - 127).
 *     Both operands of a product have this form: weights W13 / W2 with scales
 *     [P+S][2I][H/32] / [P+S][H][I/32], grouped activations Xg / Hg with scales
 *     [rows][H/32] / [rows][I/32].  The calls below take these byte arrays
 *     through their `float*` scale arguments.  Codes must be 16-byte aligned
 *     and scales 4-byte aligned.
 *   - e2m1 weights are packed two codes per byte along the reduced
 *     dimension: byte j of a row holds column 2j in bits 0-3 and column 2j+1
 *     in bits 4-7 (a row of K codes is K/2 bytes).  Their base address must
 *     be 32-byte aligned.
 *   - Weights are stored transposed with the reduced dimension contiguous:
 *     W13 [P+S][2I][H] (rows 0..I-1 = gate W1^T, rows I..2I-1 = up W3^T),
 *     W2 [P+S][H][I].  Slot s holds the weights of the logical expert
 *     physical_to_logical[s] (a replica is a copy).
 *   - Grouped buffers have `rows` rows: (P+S)*M_max (masked layout, row of
 *     slot s rank r = s*M_max + r) or T*K + S*T (contiguous layout, row =
 *     offsets[s] + r).  Rows of a slot hold its tokens in ascending token
 *     order.  Rows at or past masked_m[s] are padding: no call writes them.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum moe_status {
  MOE_OK = 0,
  MOE_ERR_INVALID = -1,     /* a null pointer, a size out of range, an inconsistent problem */
  MOE_ERR_UNSUPPORTED = -2, /* a valid problem this build does not run (dtype combination, alignment) */
  MOE_ERR_CUDA = -3,        /* a CUDA runtime error at launch */
  MOE_ERR_WORKSPACE = -4    /* workspace smaller than moe_workspace_bytes() */
} moe_status;

typedef enum moe_dtype { MOE_F32 = 0, MOE_BF16 = 1, MOE_E4M3 = 2, MOE_E2M1 = 3, MOE_MXFP4 = 4 } moe_dtype;

typedef enum moe_layout { MOE_LAYOUT_MASKED = 0, MOE_LAYOUT_CONTIG = 1 } moe_layout;

/* Bits of the device error flag. */
#define MOE_FLAG_OVERFLOW 1   /* a slot received more than M_max rows (masked layout); extra rows not written, their row_of is -1 */
/* an expert id outside [0,E), or one token naming an expert twice (the record
 * with the larger k is the one not placed) */
#define MOE_FLAG_BAD_EXPERT 2
/* a physical_to_logical entry outside [0,E), or a routed expert held by no
 * slot or by more than P-E+1 slots (its records are not placed) */
#define MOE_FLAG_BAD_MAP 4
#define MOE_FLAG_TIMEOUT 8    /* a pipeline wait inside a GEMM kernel gave up; its outputs are incomplete */

/* CUDA stream, ABI-compatible with cudaStream_t. */
typedef struct CUstream_st* moe_stream_t;

typedef struct moe_problem {
  int32_t T;          /* tokens, >= 0 */
  int32_t H;          /* hidden size */
  int32_t I;          /* expert intermediate size */
  int32_t E;          /* logical routed experts, 1..1024 */
  int32_t K;          /* experts per token, 1..min(E, 32) */
  int32_t P;          /* physical slots, >= E (== E without a replica map) */
  int32_t M_max;      /* rows per slot of the masked layout; >= T when has_shared; unused for contiguous */
  int32_t has_shared; /* 1 = one always-on shared expert in slot P, weight 1 */
  int32_t act;        /* moe_dtype of x */
  int32_t wt;         /* moe_dtype of the expert weights, Xg and Hg */
  int32_t out;        /* moe_dtype of the layer output */
  int32_t layout;     /* moe_layout of the grouped buffers */
} moe_problem;

/* Library version, (major << 16) | minor. */
int32_t moe_version(void);

/* A static string naming a status code. */
const char* moe_status_string(int32_t status);

/* Rows of the grouped buffers for this problem (see the conventions above). */
int64_t moe_grouped_rows(const moe_problem* p);

/* Workspace bytes one call sequence needs (the maximum over all calls).
 * One workspace may serve every call of a layer as long as the calls are
 * ordered on one stream.  The bytes depend on the current device's SM count:
 * ask with the device current that runs the calls (a call that is given less
 * than it needs there answers MOE_ERR_WORKSPACE).  A workspace is 16-byte
 * aligned.  Returns 0 for an invalid problem. */
size_t moe_workspace_bytes(const moe_problem* p);

/* Issue counters ("Inference INFRA methodology (5)", section "DeepGEMM": a tile
 * whose first row is at or past masked_m issues no MMA).  After a tensor-core
 * moe_grouped_swiglu_gemm, moe_grouped_down_gemm or moe_grouped_ffn call, the
 * first MOE_STATS_BYTES of the workspace hold int32 counters
 * [2 phases][MOE_STATS_CTAS][2]: for each CTA, the units it issued (token
 * chunk x weight-tile pair x K split) and the token tiles among them (one per
 * slot and chunk of at most BM rows, BM = moe_gemm_tile_rows; a GEMM that runs
 * on SM pairs counts each pair's units once, in its first CTA).  Summed over
 * CTAs, the token tiles of a GEMM equal the sum over slots of
 * ceil(masked_m[s] / BM).  Phase 1 is the down GEMM of moe_grouped_ffn and
 * zero otherwise (MXFP4: two launches, and phase 0 is the down GEMM's).  The
 * counters stay valid until the next call that uses the workspace. */
#define MOE_STATS_CTAS 256
#define MOE_STATS_BYTES (2 * MOE_STATS_CTAS * 2 * 4)

/* Token rows BM of one tile of the tensor-core GEMM of step 3 (step = 3) or
 * step 4 (step = 4) for this problem ("Inference INFRA methodology (5)",
 * section "DeepGEMM": the tile height BM of the padding-waste ratio
 * ceil(M_e / BM) * BM / M_e).  For bf16 experts 128.  For FP8 / FP4 experts
 * 256 with at least 128 rows per slot on average (and, for step 4, H a multiple
 * of 256): those GEMMs run on pairs of SMs (thread-block clusters of two), each
 * SM holding 128 of the tile's token rows and one of its two 128-row weight
 * tiles, with one cta_group::2 MMA over both; else 64: one CTA per SM with
 * M = 64 MMAs.  moe_grouped_ffn runs on single CTAs: 64-row tiles for FP8 /
 * FP4 experts, 128 for bf16.  For MXFP4 experts 256 with at least 128 rows per
 * slot on average (step 4: and H a multiple of 256), on SM pairs as above; else
 * 128.
 * 0 for an invalid problem or one whose GEMMs run on the CUDA cores (F32).
 * Host only; touches no GPU. */
int32_t moe_gemm_tile_rows(const moe_problem* p, int32_t step);

/* Check a problem without touching the GPU: MOE_OK, MOE_ERR_INVALID or
 * MOE_ERR_UNSUPPORTED. */
moe_status moe_check_problem(const moe_problem* p);

/* Step 1 (routing; "MoE inference and expert parallelism", routing section,
 * Table 3-1).  For each token t: the K largest of the E logits, in descending
 * order, ties to the lower expert index; weights
 * w[t,k] = exp(l_k - l_max) / sum_j exp(l_j - l_max) over the chosen K
 * (= softmax over all E renormalised over the K; fp32).
 *   logits [T][E] fp32 (device, read), ids [T][K] int32 and w [T][K] fp32
 *   (device, written).  One warp per token. */
moe_status moe_route_topk(const moe_problem* p, const float* logits, int32_t* ids, float* w, moe_stream_t stream);

/* Step 1, DeepSeek-V3 variant ("MoE inference and expert parallelism", routing
 * section, Table 3-1: sigmoid scoring with e_score_correction_bias, grouped
 * top-k; the bias decides which experts are chosen, the weights use the
 * unbiased scores).  Per token: s_e = sigmoid(l_e), key_e = s_e + bias_e;
 * the E experts form n_group contiguous groups of E/n_group, a group scored by
 * its largest key; the topk_group best groups are kept, then the K largest
 * keys among their experts (all ties to the lower index; keys compared in
 * fp64).  w[t,k] = s_{e_k} (divided by the sum over the K when renormalize),
 * times scale.
 *   logits [T][E] fp32, bias [E] fp32 or NULL (device, read); ids [T][K] int32,
 *   w [T][K] fp32 (device, written).  Requires 1 <= n_group <= 32, E % n_group
 *   == 0, 1 <= topk_group <= n_group, K <= topk_group * E / n_group. */
moe_status moe_route_grouped_topk(const moe_problem* p, const float* logits, const float* bias, int32_t n_group,
                                  int32_t topk_group, int32_t renormalize, float scale, int32_t* ids, float* w,
                                  moe_stream_t stream);

/* Step 2 (dispatch; "Inference INFRA methodology (5)", section "DeepGEMM";
 * "vLLM EPLB", section 1.2; "MoonEP", sections "Why dynamic routing is hard"
 * and "Zero-copy and static buffer").
 *   ids [T][K] int32: logical expert ids (from moe_route_topk).
 *   x [T][H]: activations, dtype p->act.
 *   phys_to_log [P] int32 or NULL: physical_to_logical_map.  With a map, a
 *     record (t, k) of logical expert e goes to the (t mod c)-th slot holding
 *     e, slots taken in ascending index, c = logical_replica_count[e]
 *     (round-robin by token index).  Without one, slot = e and P must be E.
 * Writes:
 *   masked_m [P+S] int32: rows per slot (the shared slot holds T).
 *   offsets [P+S+1] int32: exclusive prefix sum of masked_m.
 *   row_of [T][K+S] int32: grouped row of record (t,k); column K is the
 *     shared expert's row.  -1 for a record that was not placed (see err_flag).
 *     The calls that read row_of take any entry outside [0, rows) for -1.
 *   src_of [rows] int32: token of each written row (padding rows untouched).
 *   xg [rows][H], dtype p->wt (e4m3 for E2M1 weights): x[t] copied to its
 *     rows; for e4m3 each row is
 *     quantised per 1x128 group: s = amax/448 (fp32 IEEE division, s = 1 for an
 *     all-zero group), code = e4m3(x / s) nearest-even, saturating; for
 *     MXFP4 each row is quantised as moe_mx_quantize does.
 *   xg_scales [rows][H/128] fp32: the group scales (e4m3); [rows][H/32] scale
 *     bytes (MXFP4); else NULL.
 *   err_flag: device int32, MOE_FLAG_* bits are OR-ed in (never cleared).
 *   workspace: device scratch of moe_workspace_bytes(p) bytes. */
moe_status moe_permute(const moe_problem* p, const int32_t* ids, const void* x, const int32_t* phys_to_log,
                       int32_t* masked_m, int32_t* offsets, int32_t* row_of, int32_t* src_of, void* xg,
                       float* xg_scales, int32_t* err_flag, void* workspace, size_t workspace_bytes,
                       moe_stream_t stream);

/* moe_permute for callers that cannot allocate device memory.  The pages
 * describe no such variant; it is an addition of this library.
 * Some callers cannot call cudaMalloc where they run the layer: an inference
 * engine plugin whose enqueue step must not allocate, code running while its
 * stream is being captured into a CUDA graph, a framework whose device memory
 * all belongs to its own pool.  This call takes the same arguments and writes
 * the same outputs as moe_permute, but needs no workspace: its scratch is a
 * fixed 4 MiB array inside the library, which every GPU that loads the library
 * keeps until the process exits.
 *   - A problem whose scratch exceeds 4 MiB is rejected with MOE_ERR_WORKSPACE
 *     before anything is enqueued (the scratch is (4*P*ceil(T/32) + 4) +
 *     4*P*ceil(T/32) + 4*T*K + 4*P + 4*E + 4*E bytes, each term rounded up
 *     to 256; the prefill workload T=8192, E=P=512, K=10 needs about 1.3 MiB).
 *   - The first call on a device looks up the array's device address (with
 *     that device current) and keeps it; make that first call outside of any
 *     stream capture.  The kept address is valid for the life of the device's
 *     primary context: do not call this entry point again after
 *     cudaDeviceReset on that device.
 *   - All calls share the one array, which keeps the previous call's contents
 *     (the call clears what must start at zero itself).  Calls that overlap on
 *     the GPU -- on different streams, or from different threads, without
 *     ordering between them -- race on it and give wrong results. */
moe_status moe_permute_no_workspace(const moe_problem* p, const int32_t* ids, const void* x,
                                    const int32_t* phys_to_log, int32_t* masked_m, int32_t* offsets,
                                    int32_t* row_of, int32_t* src_of, void* xg, float* xg_scales, int32_t* err_flag,
                                    moe_stream_t stream);

/* Step 3 (expert gate/up; "MoE inference and expert parallelism", routing
 * section: SwiGLU with W1 = gate, W3 = up; "Inference INFRA methodology (5)",
 * section "DeepGEMM": masked_m read on the device, no MMA for padding tiles,
 * FP8 accumulated in FP32 once per 128-wide K block).
 * For every slot s and row r < masked_m[s] (row index per the layout):
 *   g = W1[s] . xg[row], u = W3[s] . xg[row], h = SiLU(g) * u
 *   hg[row][0..I) = h, stored as p->wt (e4m3 for E2M1 weights; e4m3: 1x128
 *   groups as in moe_permute, scales in hg_scales [rows][I/128]; bf16:
 *   nearest-even; f32: as is).
 *   MXFP4: hg is the MXFP4 form of h (one block per 32 columns of I).
 *   xg_scales / w13_scales / hg_scales: e4m3 / e2m1 / MXFP4 weights only, else
 *   NULL.
 *   masked_m [P+S], offsets [P+S+1]: as written by moe_permute (device).
 * bf16 / e4m3 / e2m1 / MXFP4 run on the tcgen05 tensor cores and need H, I
 * multiples of 128 (e2m1: e4m3 x e2m1 products, kind::f8f6f4; MXFP4:
 * block-scaled e2m1 x e2m1 products, kind::mxf4, the scales applied by the
 * tensor core). */
moe_status moe_grouped_swiglu_gemm(const moe_problem* p, const void* xg, const float* xg_scales, const void* w13,
                                   const float* w13_scales, const int32_t* masked_m, const int32_t* offsets,
                                   void* hg, float* hg_scales, int32_t* err_flag, void* workspace,
                                   size_t workspace_bytes, moe_stream_t stream);

/* Step 4 (expert down): yg[row][0..H) = W2[s] . hg[row] for every valid row,
 * stored as fp32 (wt = F32) or bf16.  Same skipping and promotion as step 3. */
moe_status moe_grouped_down_gemm(const moe_problem* p, const void* hg, const float* hg_scales, const void* w2,
                                 const float* w2_scales, const int32_t* masked_m, const int32_t* offsets,
                                 void* yg, int32_t* err_flag, void* workspace, size_t workspace_bytes,
                                 moe_stream_t stream);

/* Steps 3 and 4 in one call (the fused path of "MoE inference and expert
 * parallelism", routing section: "fused MoE" runs the grouped gate/up, the
 * activation and the grouped down GEMM as one unit of work).  Same arguments,
 * outputs and numerics as moe_grouped_swiglu_gemm followed by
 * moe_grouped_down_gemm (hg/hg_scales are still written; yg is bit-identical
 * to the two separate calls).  For bf16, e4m3 and e2m1 weights it is one persistent
 * cooperative launch in which a CTA moves on to down tiles as soon as every
 * gate/up tile of that slot has released its rows of h, so the down GEMM's
 * weight streaming overlaps the end of gate/up (plus the split-K reduction
 * kernel when the down GEMM is split).  All CTAs of it must be resident at once:
 * the launch fails (MOE_ERR_CUDA) if the device cannot co-schedule them.  MXFP4
 * problems run the two GEMMs as two launches (and the reduction when the down
 * GEMM is split), the second of which starts on its weights while the first
 * ends; fp32 problems run the two CUDA-core GEMMs one after the other.
 * workspace: moe_workspace_bytes(p) bytes (for the cooperative launch it holds
 * the per-slot ready counters, cleared by this call). */
moe_status moe_grouped_ffn(const moe_problem* p, const void* xg, const float* xg_scales, const void* w13,
                           const float* w13_scales, const void* w2, const float* w2_scales, const int32_t* masked_m,
                           const int32_t* offsets, void* hg, float* hg_scales, void* yg, int32_t* err_flag,
                           void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* Step 5 (combine; "MoE inference and expert parallelism", routing section:
 * moe_sum / TopKWeightAndReduce, DeepSeek-V3 Eq. 12 for the shared expert):
 *   out[t] = sum_{k<K} w[t,k] * yg[row_of[t,k]]  (+ yg[row_of[t,K]] if S),
 * summed in fp32 in k order, then rounded once to p->out.  Records with
 * row_of = -1 are skipped.  yg [rows][H] (F32 or BF16 per p->wt), row_of
 * [T][K+S], w [T][K] fp32, out [T][H] (p->out). */
moe_status moe_combine(const moe_problem* p, const void* yg, const int32_t* row_of, const float* w, void* out,
                       moe_stream_t stream);

/* Steps 1 and 2 in one call ("MoE inference and expert parallelism", routing
 * section and forward-pass section: fused_topk followed by the dispatch).
 * Same arguments, outputs and numerics as moe_route_topk followed by
 * moe_permute (ids and w are written and bit-identical to moe_route_topk's).
 * Batches of at most 256 records (T*K <= 256) without a replica map and with
 * E <= 256 run as one launch: every CTA chooses the experts of all tokens
 * (one warp per token, the router's own per-token code) and derives the layout
 * from them in shared memory; other batches run the two calls' kernels back
 * to back.  workspace: moe_workspace_bytes(p) bytes. */
moe_status moe_route_permute(const moe_problem* p, const float* logits, const void* x, const int32_t* phys_to_log,
                             int32_t* ids, float* w, int32_t* masked_m, int32_t* offsets, int32_t* row_of,
                             int32_t* src_of, void* xg, float* xg_scales, int32_t* err_flag, void* workspace,
                             size_t workspace_bytes, moe_stream_t stream);

/* Steps 3, 4 and 5 in one call ("MoE inference and expert parallelism",
 * routing section: fused MoE runs the grouped GEMMs, the activation and
 * moe_sum as one unit of work).  Same arguments and numerics as
 * moe_grouped_swiglu_gemm, moe_grouped_down_gemm and moe_combine in that order
 * (row_of and w as written by moe_permute and the router; hg, hg_scales and
 * yg are written as by those calls; out is bit-identical to moe_combine's).
 * bf16 experts run both GEMMs in one launch (as moe_grouped_ffn); FP8, FP4 and
 * MXFP4 experts in two.  When the down GEMM is split along K (decode-sized slots),
 * the combine runs inside the split-K reduction: each record's row is
 * reduced over the splits and enters its token's k-order sum in the same
 * kernel; otherwise the combine kernel follows the down GEMM.
 * workspace: moe_workspace_bytes(p) bytes. */
moe_status moe_ffn_combine(const moe_problem* p, const void* xg, const float* xg_scales, const void* w13,
                           const float* w13_scales, const void* w2, const float* w2_scales, const int32_t* masked_m,
                           const int32_t* offsets, const int32_t* row_of, const float* w, void* hg, float* hg_scales,
                           void* yg, void* out, int32_t* err_flag, void* workspace, size_t workspace_bytes,
                           moe_stream_t stream);

/* EPLB load statistics ("vLLM EPLB", section 1.2: expert_load_pass and
 * expert_load_window).  Copies this pass's per-slot row counts masked_m[0..P)
 * (as written by moe_permute; the shared slot is not recorded) into row
 * (pass mod window) of load_window [window][P] int32 (device). */
moe_status moe_eplb_record(const moe_problem* p, const int32_t* masked_m, int64_t pass, int32_t window,
                           int32_t* load_window, moe_stream_t stream);

/* Rebalance from a load window ("vLLM EPLB", section 1.2: the window's physical
 * loads are summed per logical expert through physical_to_logical_map, then
 * replicas are re-assigned).  logical_load [E] int64 = sum over the window and
 * over the slots holding each expert; new_phys_to_log [P]: slots 0..E-1 hold
 * experts 0..E-1, slots E..P-1 hold the P-E experts with the largest load in
 * descending order (ties to the lower index) -- the single-GPU policy of this
 * library (the page's node / GPU packing is a multi-node control plane).
 * phys_to_log [P] is the map the window was recorded with (NULL when P == E).
 * Requires P - E <= E.  A map entry outside [0,E) sets MOE_FLAG_BAD_MAP.  One
 * CTA; all pointers device. */
moe_status moe_eplb_rebalance(const moe_problem* p, const int32_t* load_window, int32_t window,
                              const int32_t* phys_to_log, int64_t* logical_load, int32_t* new_phys_to_log,
                              int32_t* err_flag, moe_stream_t stream);

/* ---------------------------------------------------------------------------
 * MXFP4 (the pages describe none; OCP Microscaling Formats v1.0, with the
 * conversion rule of its section 6.3).  Additions of this library.
 *
 * A row of `cols` values (cols a multiple of 32) becomes cols/2 code bytes and
 * cols/32 scale bytes.  Per block of 32: e = floor(log2(largest magnitude)) - 2
 * clamped to [-127, 125] (e = 0 for an all-zero block), scale byte = e + 127,
 * code = E2M1(x * 2^-e), nearest with ties to the even code, saturating at 6;
 * the sign of a zero is kept.  A block that holds a NaN or an infinity gets the
 * scale byte 255 and codes 0.
 * ------------------------------------------------------------------------- */

/* x [rows][cols] (dtype F32 or BF16) -> codes [rows][cols/2], scales
 * [rows][cols/32].  x 16-byte aligned, codes 4-byte aligned. */
moe_status moe_mx_quantize(int32_t dtype, int64_t rows, int64_t cols, const void* x, uint8_t* codes, uint8_t* scales,
                           moe_stream_t stream);

/* codes, scales -> out [rows][cols] (dtype F32 or BF16): code * 2^(s - 127),
 * exact in both types (infinite where that passes their largest value, which
 * scale bytes 253 and 254 can); NaN where s = 255.  out 16-byte aligned, codes 4-byte
 * aligned. */
moe_status moe_mx_dequantize(int32_t dtype, int64_t rows, int64_t cols, const uint8_t* codes, const uint8_t* scales,
                             void* out, moe_stream_t stream);

/* ---------------------------------------------------------------------------
 * Load-balance loss of the router ("MoE inference and expert parallelism" names
 * the bias-based alternative only; the loss of Switch Transformers, and
 * DeepSeek-V3's sequence-wise form).  Additions of this library.
 *
 * The T tokens fall into nseq segments: token t belongs to segment b when
 * seq_offsets[b] <= t < seq_offsets[b+1] (ascending; device; NULL with nseq = 1:
 * one segment of all tokens).  Tokens outside every segment, and tokens with
 * valid[t] = 0 (valid [T] bytes, device, NULL: all valid), take no part, whatever
 * their logits and ids are, and their gradient is 0.  For the n tokens that are
 * left in a segment:
 *   p_t = softmax(l_t), or sigmoid(l_t) / sum_e sigmoid(l_te)    (score)
 *   counts[b][e] = ids equal to e among them,  prob_sum[b][e] = sum_t p_te
 *   tokens[b] = n,  loss[b] = coef * E / (K n^2) * sum_e counts * prob_sum
 * A logit of -inf gives p = 0; a token whose logits are all -inf gives a row of
 * zeros.  Finite logits may have any size; a score that is below 2^-46 of its
 * row's sum may count as 0.  An empty segment has zeros everywhere.  Sums are fp32 in a fixed order: the
 * same inputs give the same bits.
 * ------------------------------------------------------------------------- */
typedef enum moe_score { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score;

/* Workspace bytes of moe_balance_loss; 0 for an invalid problem or nseq < 1. */
size_t moe_balance_workspace_bytes(const moe_problem* p, int32_t nseq);

/* logits [T][E] fp32, ids [T][K] int32 (as written by a router); loss [nseq],
 * counts [nseq][E] int32, prob_sum [nseq][E], tokens [nseq] int32 (device,
 * written).  An id outside [0,E) is not counted and sets MOE_FLAG_BAD_EXPERT. */
moe_status moe_balance_loss(const moe_problem* p, const float* logits, const int32_t* ids, const uint8_t* valid,
                            const int32_t* seq_offsets, int32_t nseq, int32_t score, float coef, float* loss,
                            int32_t* counts, float* prob_sum, int32_t* tokens, int32_t* err_flag, void* workspace,
                            size_t workspace_bytes, moe_stream_t stream);

/* Gradient: dlogits [T][E] = sum_b dloss[b] * d loss[b] / d logits, the counts
 * held constant (they come from a choice, not from a product).  counts and
 * tokens as written by moe_balance_loss, dloss [nseq] fp32 (device).  Every
 * element of dlogits is written. */
moe_status moe_balance_loss_backward(const moe_problem* p, const float* logits, const uint8_t* valid,
                                     const int32_t* seq_offsets, int32_t nseq, int32_t score, float coef,
                                     const int32_t* counts, const int32_t* tokens, const float* dloss,
                                     float* dlogits, moe_stream_t stream);

/* ---------------------------------------------------------------------------
 * The norms around the layer (DeepSeek-V3 Eq. 12 adds the layer's output to its
 * input u_t, which the pages take normed).  Additions of this library.  Per
 * token, with rms(v) = v / sqrt(mean(v^2) + eps):
 *   y  = x + res_scale * gate * rms(block) * w_post     (the norm after)
 *   xn = rms(y) * w_pre                                 (the norm before the next)
 * computed in fp32 (xn from the unrounded y) and rounded once.  block = NULL:
 * y = x (nothing of the norm after is read; y may be NULL).  w_pre and xn =
 * NULL together: only y.  x, block, y, xn [T][H] and w_post, w_pre [H] are of
 * `dtype` (F32 or BF16), and so is the gate: none, one value a channel [H], or one a token [T].
 * 1 <= H <= 16384, T <= 2^30; any alignment of the type's own size.  Outputs overlap no
 * input and no other output, except that y may be x.
 * ------------------------------------------------------------------------- */
typedef enum moe_gate { MOE_GATE_NONE = 0, MOE_GATE_CHANNEL = 1, MOE_GATE_TOKEN = 2 } moe_gate;

moe_status moe_block_norm(int32_t dtype, int32_t T, int32_t H, const void* x, const void* block, int32_t gate_kind,
                          const void* gate, const void* w_post, const void* w_pre, float res_scale, float eps,
                          void* y, void* xn, moe_stream_t stream);

/* Workspace bytes of moe_block_norm_backward; 0 for sizes out of range. */
size_t moe_block_norm_workspace_bytes(int32_t T, int32_t H);

/* Gradient of moe_block_norm, from its inputs.  dy [T][H]: gradient of y (NULL:
 * zero).  dxn [T][H]: gradient of xn (NULL with w_pre: zero).  At least one of
 * them.  Written: dx [T][H] and, with block, dblock [T][H] (`dtype`); fp32
 * dw_post [H] (with block), dgate [H] or [T] (with block and a gate), dw_pre [H] (with w_pre).
 * dw_post, dgate and dw_pre may be NULL.  Sums over tokens are fp32 in a fixed
 * order.  Outputs overlap no input and no other output, except that dx may be dy. */
moe_status moe_block_norm_backward(int32_t dtype, int32_t T, int32_t H, const void* x, const void* block,
                                   int32_t gate_kind, const void* gate, const void* w_post, const void* w_pre,
                                   float res_scale, float eps, const void* dy, const void* dxn, void* dx,
                                   void* dblock, float* dgate, float* dw_post, float* dw_pre, void* workspace,
                                   size_t workspace_bytes, moe_stream_t stream);

/* ---------------------------------------------------------------------------
 * Activation checkpoints in 8 bits.  Additions of this library.
 *
 * A row of `cols` values becomes cols E4M3 codes and ceil(cols / 128) fp32
 * scales, one per group of 128 values (a row's last group may be shorter): s =
 * largest magnitude * fp32(1/448) (rounded to fp32; 1 where it is 0), code =
 * E4M3(x / s), the nearest to the exact quotient with ties to the even code,
 * saturating at 448; the sign of a zero is kept.  A group that holds a NaN or an infinity gets a NaN scale and
 * codes 0.  Value = code * s, rounded once to the output's type; before that it
 * is within 2^-4 of x, relative, where |x| >= 2^-6 s, and within 2^-10 s below
 * that.  A scale below 2^-126 (a group of magnitudes below 448 * 2^-126) has
 * few bits, and codes may saturate: up to 7 * 2^-144 is added to both, which
 * only fp32 values of a like size notice.  Outputs overlap no input.
 * ------------------------------------------------------------------------- */

/* x [rows][cols] (dtype F32 or BF16, any alignment of the type's own size) ->
 * codes [rows][cols], scales [rows][ceil(cols / 128)].  rows, cols <= 2^33,
 * rows * cols <= 2^40, fewer than 2^32 groups. */
moe_status moe_fp8_quantize(int32_t dtype, int64_t rows, int64_t cols, const void* x, uint8_t* codes, float* scales,
                            moe_stream_t stream);

/* codes, scales -> out [rows][cols] (dtype F32 or BF16). */
moe_status moe_fp8_dequantize(int32_t dtype, int64_t rows, int64_t cols, const uint8_t* codes, const float* scales,
                              void* out, moe_stream_t stream);

/* ---------------------------------------------------------------------------
 * Training the experts (the pages treat inference alone).  Additions of this
 * library, for bf16 experts (BF16/BF16/BF16; others answer
 * MOE_ERR_UNSUPPORTED).  A training pass is the forward pass with step 3 in the
 * form that keeps its results:
 *
 *   moe_route_topk, moe_permute, moe_grouped_swiglu_gemm_save,
 *   moe_grouped_down_gemm, moe_combine
 *
 * and its gradient, in this order on one stream:
 *
 *   moe_combine_backward      dout -> dyg, wg, dw
 *   moe_grouped_ffn_backward  dyg -> dxg and the weights' gradients
 *   moe_permute_backward      dxg -> dx
 *   moe_route_backward        dw -> dlogits
 *
 * What the gradient reads of the forward pass: ids, w, row_of, masked_m,
 * offsets, xg, yg and the checkpoint gu.  Rows at or past masked_m[s] are
 * neither read into a result nor written, whatever they hold; a record that was
 * not placed (row_of = -1) contributes nothing and has dw = 0.  Weights'
 * gradients are per slot: replicas of one expert each have their own.  Sums are
 * fp32 in a fixed order: the same inputs give the same bits.  No workspace.
 * Counts and offsets that lead outside the grouped buffers are cut to them.
 * ------------------------------------------------------------------------- */

/* Step 3 that also keeps g and u for the gradient: with (g, u) the products of
 * a row with W13's gate and up rows,
 *   hg [rows][I] bf16: SiLU(g) * u,
 *   gu [rows][2I]: the codes of the row (g, u) as moe_fp8_quantize has them (of
 *     the fp32 sums; a code whose quotient lies within the sums' rounding of the
 *     middle of two may be either), gu_scales [rows][2I/128] the scales.
 * xg, w13, hg and gu 16-byte aligned. */
moe_status moe_grouped_swiglu_gemm_save(const moe_problem* p, const void* xg, const void* w13, const int32_t* masked_m,
                                        const int32_t* offsets, void* hg, uint8_t* gu, float* gu_scales,
                                        int32_t* err_flag, moe_stream_t stream);

/* Gradient of moe_combine: for every placed record (t, k) with grouped row r,
 *   the gradient of yg[r] is wg[r] * dyg[r] with dyg[r] = dout[t] and wg[r] =
 *     w[t,k] (the shared expert's: 1), kept apart so that the product is not
 *     rounded to bf16,
 *   dw[t,k] = sum_h dout[t,h] * yg[r,h]  (fp32; the shared expert has none).
 * dout [T][H], yg and dyg [rows][H] bf16, wg [rows] fp32; dyg may be yg.  dw
 * [T][K], or NULL: it is not computed and yg is not read (and may be NULL). */
moe_status moe_combine_backward(const moe_problem* p, const void* dout, const void* yg, const int32_t* row_of,
                                const float* w, void* dyg, float* wg, float* dw, moe_stream_t stream);

/* Gradient of steps 3 and 4.  With g, u the values of the checkpoint and s =
 * sigmoid(g), for every valid row:
 *   dh = wg[row] * W2[s]^T . dyg[row],  hg[row] = wg[row] * g s u,
 *   dgu[row] = (dh u s (1 + g (1 - s)), dh g s),
 *   dxg[row] = W13[s]^T . dgu[row]
 * and for every slot, summed over its valid rows,
 *   dw13[s] = dgu^T xg [2I][H],  dw2[s] = dyg^T hg [H][I].
 * dgu [rows][2I] and hg [rows][I] are bf16 (written; products take them in that
 * form), dxg [rows][H] is fp32 (a token's rows of it are still to be added).  wg NULL: every row has weight 1.  dw13, dw2: dw_dtype BF16 or F32; `accumulate` (F32
 * alone, else MOE_ERR_UNSUPPORTED) adds to what they hold, otherwise every
 * element is written, zeros for a slot without rows.  dxg, dw13 and dw2 may each
 * be NULL where they are not wanted (then w13, xg are not read).  All but wg and
 * gu_scales 16-byte aligned; outputs overlap no input and no other output. */
moe_status moe_grouped_ffn_backward(const moe_problem* p, const void* dyg, const float* wg, const void* xg,
                                    const void* w13, const void* w2, const uint8_t* gu, const float* gu_scales,
                                    const int32_t* masked_m, const int32_t* offsets, void* dgu, void* hg, float* dxg, void* dw13, void* dw2,
                                    int32_t dw_dtype, int32_t accumulate, int32_t* err_flag, moe_stream_t stream);

/* Gradient of the dispatch: dx[t] = sum over the token's placed records of
 * dxg[row], in fp32 in k order (the shared expert's last), rounded once.  dxg
 * [rows][H] fp32, dx [T][H] bf16, 16-byte aligned. */
moe_status moe_permute_backward(const moe_problem* p, const float* dxg, const int32_t* row_of, void* dx,
                                moe_stream_t stream);

/* Gradient of the router's weights with the choice held constant; any problem
 * type.  dlogits [T][E] = add (or zeros), plus at expert ids[t,k]:
 *   SOFTMAX (moe_route_topk):  w_k (dw_k - sum_j w_j dw_j); w as that call wrote
 *     it, logits are not read;
 *   SIGMOID (moe_route_grouped_topk): s_k (1 - s_k) ds_k with s = sigmoid(logits),
 *     ds_k = scale (dw_k - sum_j s_j dw_j / S) / S with S = sum_j s_j when
 *     `renormalize`, else scale dw_k; w is not read.  A token whose S is 0 has 0.
 * renormalize and scale: as in that call (SOFTMAX ignores them).  add [T][E]
 * fp32 or NULL, for instance the gradient of moe_balance_loss; dlogits may be
 * add.  Ids outside [0,E) are skipped. */
moe_status moe_route_backward(const moe_problem* p, int32_t score, const float* logits, const int32_t* ids,
                              const float* w, const float* dw, int32_t renormalize, float scale, const float* add,
                              float* dlogits, moe_stream_t stream);

/* The four calls of the gradient in one, four launches: moe_combine_backward and
 * moe_route_backward in one, the two of moe_grouped_ffn_backward,
 * moe_permute_backward; the same arguments and the same results.  dyg, wg, dgu, hg and dxg are buffers between the steps, written as by
 * those calls; dw [T][K] is written too.  dw13 and dw2 may each be NULL. */
moe_status moe_layer_backward(const moe_problem* p, const void* dout, const void* yg, const int32_t* row_of,
                              const int32_t* ids, const float* w, const void* xg, const void* w13, const void* w2,
                              const uint8_t* gu, const float* gu_scales, const int32_t* masked_m,
                              const int32_t* offsets, int32_t score, const float* logits, int32_t renormalize,
                              float scale, const float* add, void* dyg, float* wg, void* dgu, void* hg, float* dxg,
                              float* dw, void* dx, float* dlogits, void* dw13, void* dw2, int32_t dw_dtype,
                              int32_t accumulate, int32_t* err_flag, moe_stream_t stream);

/* Diagnostic, an addition of this library (the pages describe none): runs the
 * bounded wait that every kernel here uses on an mbarrier that nothing
 * completes, with a limit of `cycles` SM cycles (1 .. 4e9), so that the expiry
 * path can be checked without a fault: the kernel ORs MOE_FLAG_TIMEOUT into
 * *err_flag (device int32) and returns; the context stays usable. */
moe_status moe_selftest_bounded_wait(int64_t cycles, int32_t* err_flag, moe_stream_t stream);

/* Host helper ("vLLM EPLB", section 1.2): invert a physical_to_logical map.
 * All pointers are HOST pointers.  p2l [P] in, l2p [E][R] out (slots of each
 * logical expert in ascending order, padded with -1), rc [E] out.  Returns
 * the largest replica count, or MOE_ERR_INVALID for an entry outside [0,E) or
 * an expert with more than R replicas. */
int32_t moe_eplb_invert(int32_t P, int32_t E, const int32_t* p2l, int32_t R, int32_t* l2p, int32_t* rc);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */
