/*
 * libdgfp8 -- FP8 GEMM with fine-grained block scaling for MI355X (gfx950).
 *
 * C ABI.  Plain pointers and sizes only.  Every pointer marked "device" is a
 * device address on the current HIP device; "stream" is a hipStream_t passed
 * as void* (NULL selects the default stream).  All work is enqueued on that
 * stream and the call returns without synchronising.  The caller owns every
 * buffer, including the optional split-K workspace of dg_fp8_gemm_nt_ws; the
 * library allocates no device memory and keeps no device state besides the
 * compute-unit count used for the persistent grid.
 *
 * Errors: every entry point validates its arguments on the host and returns a
 * dg_status.  Nothing aborts and no exception crosses the ABI.  A problem
 * with a zero-sized dimension returns DG_SUCCESS without launching anything.
 * Device-side preconditions that are not checked are stated per function.
 *
 * Method (pages on DeepGEMM): D(bf16) = A . B^T in the NT layout (both
 * operands K-major), with E4M3 A carrying one fp32 scale per row per 128-wide
 * K block and E4M3 B one fp32 scale per 128x128 block; every K block's partial
 * product is scaled and promoted into an fp32 accumulator.  Sources: page
 * "GitHub 推荐：DeepSeek 开源周最大黑马 DeepGEMM…" (问题判断: 128x128 block
 * scaling; 创新之处: per-block scaling through promotion; 解法哲学: the
 * fp8_gemm_nt call with a caller-provided output d); page juejin.cn post on
 * DeepGEMM (section 3: two-level accumulation and M-only grouping; section
 * 4(3): dense, contiguous and masked GEMM types; section 5: API names).
 *
 * Scale-factor contract (all GEMM entry points):
 *   SFA is fp32, logically [rows, K/128]; element (i, kb) lives at
 *       sfa[i * sfa_sm + kb * sfa_sk]  (row-major: sfa_sm = K/128, sfa_sk = 1;
 *       MN-major / "transposed": sfa_sm = 1, sfa_sk = rows).
 *   SFB is fp32, logically [ceil(N/128), K/128]; element (nb, kb) at
 *       sfb[nb * sfb_sn + kb * sfb_sk]; output column j uses nb = j / 128.
 *   E4M3 is the OCP "FN" flavour (largest finite 448, no infinities).
 *   Strides are in elements and must be >= 0.
 *   Scale values (fp32 entry points): finite fp32, negative ones flipping the
 *   sign of their block's contribution.  A zero scale makes its block
 *   contribute nothing, as the definition says.  Subnormal scales are applied
 *   exactly as long as the product sfa * sfb of a row's block is at least
 *   2^-189; smaller products contribute nothing.  A product of 2^65 or more,
 *   or an infinite or NaN scale, gives NaN in every output it weights.  (The
 *   casts produce scales between fp32(1e-4)/448 and 2^121.)
 *
 * Alignment contract: K % 128 == 0; lda, ldb and the A/B base addresses are
 * multiples of 16 bytes; N % 8 == 0, ldd % 8 == 0 and D is 16-byte aligned.
 * Violations return DG_ERROR_NOT_SUPPORTED.
 *
 * Accuracy (measured on gfx950 and pinned by tests): within one 128-wide K
 * block the matrix unit keeps each product only within a 14-bit window below
 * the block's largest product, cutting each toward zero.  Every block's
 * partial is then promoted into an fp32 accumulator.  The promotion rounds the
 * partial's excess bits to nearest even, and truncates toward minus infinity
 * the accumulator bits that a larger partial pushes below the fp32 grid.  The
 * bf16 output is rounded to nearest even once.  Results are deterministic and
 * do not depend on the persistent grid width.  A K split changes only the
 * last bits: its partial tiles are added in split order.
 *
 * Size contract: one group's A rows and B rows are addressed with 32-bit byte
 * offsets (rows x leading dimension < 2^32), and no size, leading dimension,
 * scale stride or group stride may exceed 2^40; larger values return
 * DG_ERROR_NOT_SUPPORTED before anything is launched (the casts and the
 * scale packing apply the 2^40 bound too).
 */
#ifndef DGFP8_H_
#define DGFP8_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum dg_status {
  DG_SUCCESS = 0,
  DG_ERROR_INVALID_VALUE = 1,     /* null pointer, negative size, bad stride, bad group count */
  DG_ERROR_NOT_SUPPORTED = 2,     /* K % 128 != 0, misaligned pointer / leading dimension, N % 8 != 0 */
  DG_ERROR_MISALIGNED_LAYOUT = 3, /* contiguous layout: m_total % 128 != 0 */
  DG_ERROR_LAUNCH = 4,            /* HIP reported an error at launch */
  DG_ERROR_SCRATCH_LIMIT = 5      /* dg_fp8_gemm_nt_noalloc: the problem needs more split-K scratch than its static maximum */
} dg_status;

/* Human-readable name of a status; never NULL.  Errors are returned rather
 * than raised, so the caller decides how to report them (page "GitHub 推荐：
 * DeepSeek 开源周最大黑马 DeepGEMM…", 解法哲学 and 可复用的模式与技巧: host-side
 * assertions on every layout field give the caller a clear error). */
const char* dg_status_string(dg_status status);

/*
 * Dense GEMM: D[m, n] = sum_kb sfa[m, kb] * sfb[n/128, kb] * sum_{k in kb} A[m, k] * B[n, k],
 * rounded to bf16 (round to nearest even).
 *   a   device, E4M3 [m, k], row stride lda (bytes = elements)
 *   sfa device, fp32, see the scale-factor contract (rows = m)
 *   b   device, E4M3 [n, k], row stride ldb
 *   sfb device, fp32 [ceil(n/128), k/128] with strides sfb_sn, sfb_sk
 *   d   device, bf16 [m, n], row stride ldd (elements); fully overwritten
 * Never splits the K range (see dg_fp8_gemm_nt_ws); equivalent to
 * dg_fp8_gemm_nt_ws with no workspace.
 * Page "GitHub 推荐…DeepGEMM…", 解法哲学 (fp8_gemm_nt with output d);
 * page juejin.cn, section 4(3) (dense GEMM type).
 */
dg_status dg_fp8_gemm_nt(const void* a, int64_t lda,
                         const float* sfa, int64_t sfa_sm, int64_t sfa_sk,
                         const void* b, int64_t ldb,
                         const float* sfb, int64_t sfb_sn, int64_t sfb_sk,
                         void* d, int64_t ldd,
                         int64_t m, int64_t n, int64_t k,
                         void* stream);

/*
 * Dense GEMM as dg_fp8_gemm_nt, with a caller-provided workspace that lets a
 * small-m problem (too few output tiles to occupy the device) split its K
 * blocks over several workgroups per output tile.  Each split unit sums its
 * K blocks in order into an fp32 partial tile; the last unit to finish adds
 * the partials in split order and writes D.  Results are deterministic and
 * independent of dg_set_num_cus, but may differ from the unsplit sum in the
 * last fp32 bits (both within the method's tolerance).
 *   ws        device, 16-byte aligned, ws_bytes long, or NULL (no split).
 *             Its first 256 KiB hold arrival counters: they must be zero
 *             before the workspace is first used, and every completed call
 *             leaves them zero, so a workspace can be reused by any later call
 *             on the same stream.  Calls that may run concurrently need
 *             distinct workspaces.  The rest holds fp32 partial tiles.
 *   ws_bytes  at least dg_fp8_gemm_nt_workspace_size(m, n, k) to enable the
 *             split; a smaller (or NULL) workspace runs the unsplit kernel.
 * Split-K is this library's answer to small m on a 256-CU device; the pages
 * only note that thin shapes (small M, large N and K) run at low efficiency
 * (page discosf.com news post on DeepGEMM, sections 4.3 and 5.4).
 */
dg_status dg_fp8_gemm_nt_ws(const void* a, int64_t lda,
                            const float* sfa, int64_t sfa_sm, int64_t sfa_sk,
                            const void* b, int64_t ldb,
                            const float* sfb, int64_t sfb_sn, int64_t sfb_sk,
                            void* d, int64_t ldd,
                            int64_t m, int64_t n, int64_t k,
                            void* ws, size_t ws_bytes,
                            void* stream);

/*
 * Accumulating dense GEMM: D = RNE_bf16(C + A . B^T), C an fp32 addend of D's
 * shape added to the fp32 result before the single rounding to bf16.  The
 * optional c argument of fp8_gemm_nt (page "GitHub 推荐…DeepGEMM…", 解法哲学);
 * the pages say no more about it, and this reading is the plainest one.
 * Same arguments, workspace rules and results as dg_fp8_gemm_nt_ws, plus
 *   c    device, fp32 [m, n], row stride ldc (elements); read only, must not
 *        overlap d
 * Errors (for m, n > 0): null c or ldc < n -> DG_ERROR_INVALID_VALUE;
 * c not 16-byte aligned or ldc % 4 != 0 -> DG_ERROR_NOT_SUPPORTED.
 */
dg_status dg_fp8_gemm_nt_acc(const void* a, int64_t lda,
                             const float* sfa, int64_t sfa_sm, int64_t sfa_sk,
                             const void* b, int64_t ldb,
                             const float* sfb, int64_t sfb_sn, int64_t sfb_sk,
                             const float* c, int64_t ldc,
                             void* d, int64_t ldd,
                             int64_t m, int64_t n, int64_t k,
                             void* ws, size_t ws_bytes,
                             void* stream);

/*
 * Dense GEMM for callers that cannot allocate device memory (code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc).
 * Same arguments (without ws, ws_bytes) and results as dg_fp8_gemm_nt_ws given
 * a workspace of dg_fp8_gemm_nt_workspace_size(m, n, k) bytes: the split-K
 * partial tiles and arrival counters live in a static device array of the
 * library instead, 16 MiB of partials plus the 256 KiB counter block
 * (16.25 MiB per device, held from the device's first such call until the
 * process ends).  Nothing is allocated and nothing is freed.
 *   A problem whose split plan needs more than that returns
 *   DG_ERROR_SCRATCH_LIMIT before anything is launched (call
 *   dg_fp8_gemm_nt_ws with a workspace of your own instead).
 *   Every call on one device shares that device's array: calls that may
 *   overlap on one device (other streams, other host threads) race and give
 *   wrong results; calls in order on one stream are safe.  The counters are
 *   zero when the array is first used and every completed call leaves them
 *   zero.
 */
dg_status dg_fp8_gemm_nt_noalloc(const void* a, int64_t lda,
                                 const float* sfa, int64_t sfa_sm, int64_t sfa_sk,
                                 const void* b, int64_t ldb,
                                 const float* sfb, int64_t sfb_sn, int64_t sfb_sk,
                                 void* d, int64_t ldd,
                                 int64_t m, int64_t n, int64_t k,
                                 void* stream);

/* Workspace bytes dg_fp8_gemm_nt_ws needs to split this problem; 0 when the
 * problem runs unsplit (or the sizes are invalid).  Depends only on m, n, k
 * and the device's compute-unit count. */
size_t dg_fp8_gemm_nt_workspace_size(int64_t m, int64_t n, int64_t k);

/* The output tile (block_m x block_n) and K split count dg_fp8_gemm_nt_ws
 * would use for this problem with a workspace of ws_bytes (0: none).  The
 * choice is a pure function of the shape and the device's compute-unit count,
 * made by a cost model rather than by timing candidates (page "GitHub 推荐：
 * DeepSeek 开源周最大黑马 DeepGEMM…", 创新之处 on the analytical heuristics
 * that rank a small, constrained set of block shapes; page "企业官网建设流程
 * 全解析", section 2.1 on per-shape configurations).  For profiling and logs; the
 * choice never changes results beyond the split-K note above.  Errors: null
 * outputs or non-positive sizes -> DG_ERROR_INVALID_VALUE, k % 128 != 0 ->
 * DG_ERROR_NOT_SUPPORTED. */
dg_status dg_fp8_gemm_nt_tile_config(int64_t m, int64_t n, int64_t k, size_t ws_bytes,
                                     int* block_m, int* block_n, int* splits);

/*
 * M-grouped GEMM, contiguous layout (MoE prefill / training forward).
 * The rows of all groups are concatenated along M; each group's segment is
 * padded to a multiple of 128 rows (dg_get_mk_alignment_for_contiguous_layout).
 *   a         device, E4M3 [m_total, k], row stride lda
 *   sfa       device, fp32, rows = m_total (scale-factor contract)
 *   b         device, E4M3 [num_groups, n, k]; group g starts at b + g * b_group_stride,
 *             rows of a group have stride ldb
 *   sfb       device, fp32 [num_groups, ceil(n/128), k/128]; group g at sfb + g * sfb_group_stride
 *   d         device, bf16 [m_total, n], row stride ldd
 *   m_indices device, int32 [m_total]: group of each row, -1 on padding rows
 * Row i with m_indices[i] = g >= 0 gets row i of A times B[g]^T.  Rows with
 * m_indices[i] == -1 are NOT written (their contents are left untouched).
 * Preconditions (not checked on the device): in each aligned 128-row block
 * every row with m_indices >= 0 has the same value, which lies in
 * [0, num_groups).  The group of a block is read from its first row; a block
 * whose first row is -1 is skipped entirely.
 * The work is one or two kernel launches on the same stream, planned from the
 * sizes alone (the host never reads m_indices, so the call can be captured in
 * a graph): when groups average two or more 128-row blocks, pairs of
 * consecutive blocks of one group run as 256-row tiles and the blocks left
 * over as 128-row tiles in a second launch, both tile lists built on the
 * device; otherwise one tile per block, split into two launches when the tiles
 * end in a thinly filled last round.  Every row is computed with the same
 * operations in all of these plans, so the results do not depend on the plan
 * or on dg_set_num_cus.  No K is split (see the _ws variant).
 * Errors: m_total % 128 != 0 -> DG_ERROR_MISALIGNED_LAYOUT.
 * Page juejin.cn, sections 3 and 4(3) (M-only grouping, contiguous layout
 * aligned to the M block); page "GitHub 推荐…", 风险与不足 (128-row padding).
 */
dg_status dg_m_grouped_fp8_gemm_nt_contiguous(const void* a, int64_t lda,
                                              const float* sfa, int64_t sfa_sm, int64_t sfa_sk,
                                              const void* b, int64_t ldb, int64_t b_group_stride,
                                              const float* sfb, int64_t sfb_sn, int64_t sfb_sk,
                                              int64_t sfb_group_stride,
                                              void* d, int64_t ldd,
                                              const int32_t* m_indices, int64_t m_total,
                                              int64_t n, int64_t k, int num_groups,
                                              void* stream);

/*
 * M-grouped GEMM, masked layout (MoE decode; usable under HIP graph capture).
 *   a        device, E4M3 [num_groups, max_m, k]; group g at a + g * a_group_stride, rows lda
 *   sfa      device, fp32 [num_groups, max_m, k/128]; group g at sfa + g * sfa_group_stride,
 *            then the scale-factor contract with rows = max_m
 *   b, sfb   as in the contiguous variant
 *   d        device, bf16 [num_groups, max_m, n]; group g at d + g * d_group_stride, rows ldd
 *   masked_m device, int32 [num_groups]: valid rows of each group, read on the
 *            device at run time (never by the host), clamped to [0, max_m]
 *   expected_m  hint of the typical masked_m (it picks the tile height: at most
 *            64 selects 64-row tiles, made for decode); never changes results
 * For group g, rows i < masked_m[g] get A[g, i] times B[g]^T; rows at or beyond
 * masked_m[g] are left untouched.
 * Page juejin.cn, section 4(3) (masked grouped GEMM for decode with graphs).
 */
dg_status dg_m_grouped_fp8_gemm_nt_masked(const void* a, int64_t lda, int64_t a_group_stride,
                                          const float* sfa, int64_t sfa_sm, int64_t sfa_sk,
                                          int64_t sfa_group_stride,
                                          const void* b, int64_t ldb, int64_t b_group_stride,
                                          const float* sfb, int64_t sfb_sn, int64_t sfb_sk,
                                          int64_t sfb_group_stride,
                                          void* d, int64_t ldd, int64_t d_group_stride,
                                          const int32_t* masked_m, int num_groups,
                                          int64_t max_m, int64_t n, int64_t k,
                                          int64_t expected_m,
                                          void* stream);

/*
 * Per-token FP8 cast (the library's GEMMs take E4M3 inputs; the caller does the
 * cast: page ssnai.com DeepGEMM analysis, the warning that casting is the
 * caller's job).  For each row i and 128-wide block kb of a bf16 [m, k] input:
 *   amax = max |x|;  s = fl32(max(amax, 1e-4) / 448)  (IEEE fp32 division);
 *   if ue8m0 != 0: s = smallest power of two >= s;
 *   q = E4M3 round-to-nearest-even of clamp(fl32(x / s), -448, 448), sign kept.
 *   x   device, bf16 [m, k], row stride ldx (elements), 16-byte aligned rows
 *   q   device, E4M3 [m, k], row stride ldq (bytes), 16-byte aligned rows
 *   sf  device, fp32 [m, k/128]: element (i, kb) at sf[i * sf_sm + kb * sf_sk]
 * Results are bit-exact with the definition above.
 */
dg_status dg_per_token_cast_fp8(const void* x, int64_t ldx,
                                void* q, int64_t ldq,
                                float* sf, int64_t sf_sm, int64_t sf_sk,
                                int64_t m, int64_t k, int ue8m0,
                                void* stream);

/* Same as dg_per_token_cast_fp8 for an fp32 [m, k] input. */
dg_status dg_per_token_cast_fp8_f32(const void* x, int64_t ldx,
                                    void* q, int64_t ldq,
                                    float* sf, int64_t sf_sm, int64_t sf_sk,
                                    int64_t m, int64_t k, int ue8m0,
                                    void* stream);

/*
 * Weight-side cast: fp32 [n, k] -> E4M3 [n, k] with one scale per 128x128 block
 * (rows beyond n in the last block do not exist and do not enter its amax).
 * The weights' block granularity is the method's (page "GitHub 推荐：DeepSeek
 * 开源周最大黑马 DeepGEMM…", 问题判断); the pages tell users to prepare
 * weights and scales with the library's weight conversion tools (page
 * ssnai.com DeepGEMM analysis, the FP8/FP4 pitfall notes and Mega MoE steps).
 * Same scale and code rules as dg_per_token_cast_fp8, amax taken over the block.
 *   sf  device, fp32 [ceil(n/128), k/128]: element (nb, kb) at sf[nb * sf_sn + kb * sf_sk]
 */
dg_status dg_per_block_cast_fp8(const void* x, int64_t ldx,
                                void* q, int64_t ldq,
                                float* sf, int64_t sf_sn, int64_t sf_sk,
                                int64_t n, int64_t k, int ue8m0,
                                void* stream);

/*
 * Packed UE8M0 scales (the exponent-only scale format; page "GitHub 推荐：DeepSeek
 * 开源周最大黑马 DeepGEMM…", 可复用的模式与技巧 "UE8M0 int32 packing" and
 * the SF dual path next to it; page ssnai.com DeepGEMM analysis, on the scale
 * formats of the two GPU generations).
 *
 * Packed contract: a scale word is an int32 holding the 8-bit biased
 * exponents e (value 2^(e-127)) of 4 consecutive K blocks, little-endian:
 * byte j (bits 8j..8j+7) of word w belongs to K block 4w + j.  Bytes past the
 * last K block are ignored.  e = 255 is not a scale (outside the contract).
 *   SFA words: logically [rows, ceil(K/512)]; word (i, w) at sfa[i * sfa_sm + w * sfa_sk]
 *   SFB words: logically [ceil(N/128), ceil(K/512)]; word (nb, w) at sfb[nb * sfb_sn + w * sfb_sk]
 * Strides are in int32 elements.  With such scales each K block's product
 * 2^(ea + eb - 254) * P is exact in the accumulator's exponent range, so these
 * entry points run kernels without any per-block rescaling; with power-of-two
 * fp32 scales the fp32 entry points give bit-identical results.
 */

/* Dense GEMM as dg_fp8_gemm_nt_ws (same workspace rules) with packed UE8M0 scales. */
dg_status dg_fp8_gemm_nt_ue8m0(const void* a, int64_t lda,
                               const int32_t* sfa, int64_t sfa_sm, int64_t sfa_sk,
                               const void* b, int64_t ldb,
                               const int32_t* sfb, int64_t sfb_sn, int64_t sfb_sk,
                               void* d, int64_t ldd,
                               int64_t m, int64_t n, int64_t k,
                               void* ws, size_t ws_bytes,
                               void* stream);

/* Contiguous grouped GEMM as dg_m_grouped_fp8_gemm_nt_contiguous with packed
 * UE8M0 scales (sfb_group_stride in int32 elements). */
dg_status dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0(const void* a, int64_t lda,
                                                    const int32_t* sfa, int64_t sfa_sm, int64_t sfa_sk,
                                                    const void* b, int64_t ldb, int64_t b_group_stride,
                                                    const int32_t* sfb, int64_t sfb_sn, int64_t sfb_sk,
                                                    int64_t sfb_group_stride,
                                                    void* d, int64_t ldd,
                                                    const int32_t* m_indices, int64_t m_total,
                                                    int64_t n, int64_t k, int num_groups,
                                                    void* stream);

/*
 * Contiguous grouped GEMM as dg_m_grouped_fp8_gemm_nt_contiguous, with a
 * split-K workspace (caller-owned, 16-byte aligned, same contract as the dense
 * one: the first 256 KiB are arrival counters, zero before first use and left
 * zero by every completed call; calls that may overlap need distinct
 * workspaces).  When the paired plan runs and ws_bytes is at least
 * dg_m_grouped_fp8_gemm_nt_contiguous_workspace_size(...), the second launch
 * (the blocks no pair covers, typically one per group) splits K over the CUs
 * its few tiles would leave idle: the kernel picks the split from the number
 * of leftover blocks it finds, so the call stays graph-capturable.  Each split
 * sums its K range in order and the last to arrive adds the fp32 partial tiles
 * in split order, so results are deterministic and independent of
 * dg_set_num_cus; rows of leftover blocks may differ from the unsplit call in
 * the last bits, rows of paired blocks do not.  With ws null or too small the
 * call behaves as dg_m_grouped_fp8_gemm_nt_contiguous.
 * Errors: as dg_m_grouped_fp8_gemm_nt_contiguous; ws not 16-byte aligned ->
 * DG_ERROR_NOT_SUPPORTED.
 * Splitting K over workgroups is this library's addition for a 256-CU device
 * (the pages only note low efficiency for thin shapes: page "企业官网建设流程全解析",
 * sections 4.3 and 5.4).
 */
dg_status dg_m_grouped_fp8_gemm_nt_contiguous_ws(const void* a, int64_t lda,
                                                 const float* sfa, int64_t sfa_sm, int64_t sfa_sk,
                                                 const void* b, int64_t ldb, int64_t b_group_stride,
                                                 const float* sfb, int64_t sfb_sn, int64_t sfb_sk,
                                                 int64_t sfb_group_stride,
                                                 void* d, int64_t ldd,
                                                 const int32_t* m_indices, int64_t m_total,
                                                 int64_t n, int64_t k, int num_groups,
                                                 void* ws, size_t ws_bytes, void* stream);

/* As dg_m_grouped_fp8_gemm_nt_contiguous_ws with packed UE8M0 scales. */
dg_status dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0_ws(const void* a, int64_t lda,
                                                       const int32_t* sfa, int64_t sfa_sm, int64_t sfa_sk,
                                                       const void* b, int64_t ldb, int64_t b_group_stride,
                                                       const int32_t* sfb, int64_t sfb_sn, int64_t sfb_sk,
                                                       int64_t sfb_group_stride,
                                                       void* d, int64_t ldd,
                                                       const int32_t* m_indices, int64_t m_total,
                                                       int64_t n, int64_t k, int num_groups,
                                                       void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes the _ws contiguous calls can use for this problem (0: the
 * plan never splits K).  Non-positive sizes, k % 128 != 0, m_total % 128 != 0 or
 * num_groups < 1 give 0. */
size_t dg_m_grouped_fp8_gemm_nt_contiguous_workspace_size(int64_t m_total, int64_t n, int64_t k,
                                                          int num_groups);

/* Masked grouped GEMM as dg_m_grouped_fp8_gemm_nt_masked with packed UE8M0
 * scales (group strides in int32 elements). */
dg_status dg_m_grouped_fp8_gemm_nt_masked_ue8m0(const void* a, int64_t lda, int64_t a_group_stride,
                                                const int32_t* sfa, int64_t sfa_sm, int64_t sfa_sk,
                                                int64_t sfa_group_stride,
                                                const void* b, int64_t ldb, int64_t b_group_stride,
                                                const int32_t* sfb, int64_t sfb_sn, int64_t sfb_sk,
                                                int64_t sfb_group_stride,
                                                void* d, int64_t ldd, int64_t d_group_stride,
                                                const int32_t* masked_m, int num_groups,
                                                int64_t max_m, int64_t n, int64_t k,
                                                int64_t expected_m,
                                                void* stream);

/*
 * Scale transform fp32 -> packed UE8M0: for every row i and K block kb,
 * e = biased exponent of sf(i, kb), plus 1 when any mantissa bit is set (the
 * smallest power of two >= the scale, as the casts' ue8m0 mode), stored in
 * byte kb % 4 of word (i, kb / 4); bytes past the last K block are 0.  Exact for
 * power-of-two scales, which is what the casts produce with ue8m0 != 0.  Inputs
 * must be positive normal fp32 no larger than 2^127 (other values are outside
 * the contract).
 *   sf   device, fp32 [rows, kblocks]: element (i, kb) at sf[i * sf_s0 + kb * sf_s1]
 *   out  device, int32 [rows, ceil(kblocks/4)]: word (i, w) at out[i * out_s0 + w * out_s1]
 * Errors: negative sizes/strides or null pointers -> DG_ERROR_INVALID_VALUE;
 * pointers not 4-byte aligned -> DG_ERROR_NOT_SUPPORTED.
 */
dg_status dg_pack_ue8m0(const float* sf, int64_t sf_s0, int64_t sf_s1,
                        int32_t* out, int64_t out_s0, int64_t out_s1,
                        int64_t rows, int64_t kblocks,
                        void* stream);

/*
 * Plan of the contiguous grouped GEMM: 0 (default) picks by the cost model;
 * 1 forces the paired plan (256-row tiles on pairs of consecutive 128-row
 * blocks of one group, found on the device from m_indices, and 128-row tiles on
 * the blocks no pair covers: two launches); 2 forces one tile per 128-row
 * block.  Layouts of more than 2048 blocks always take plan 2.  Every plan
 * computes each output row with the same operations, so the choice never
 * changes a bit of the result; it is a tuning and testing knob, process-wide.
 * Errors: plan outside 0..2 -> DG_ERROR_INVALID_VALUE.
 */
dg_status dg_set_contiguous_plan(int plan);

/*
 * Plan of the dense GEMM (dg_fp8_gemm_nt and its variants): instance < 0
 * (default) picks the kernel instance and K split by the cost model; otherwise
 * every following dense call in the process uses this instance, with `splits`
 * K splits when the call has a workspace that holds them (else 1).  The
 * workspace-size and tile-config queries report the forced plan.  Instances:
 *   0 128x256, 1 128x128, 2 256x256, 3 128x64, 4 64x64  (LDS stages shared by
 *     the workgroup's waves)
 *   6 192x256
 * A tuning and testing knob (the split changes the fp32 summation order, so
 * results may differ in the last bits between plans).
 * Errors: instance > 6 or splits < 1 -> DG_ERROR_INVALID_VALUE; instance 5
 * (masked groups only), or splits > 1 with instance 2 or 6 (no split-K
 * variant), or splits > 65536 -> DG_ERROR_NOT_SUPPORTED.
 */
dg_status dg_set_dense_plan(int instance, int splits);

/* Row alignment of each group's segment in the contiguous layout: 128.
 * (Page ssnai.com DeepGEMM analysis: the alignment query for contiguous MoE.) */
int dg_get_mk_alignment_for_contiguous_layout(void);

/* Element types of the calls below. */
typedef enum dg_dtype { DG_F32 = 0, DG_BF16 = 1, DG_F16 = 2 } dg_dtype;

/*
 * ---------------------------------------------------------------------------
 * int8 GEMM with a scale per token and per channel
 *
 *   D[m, n] = sfa[m] * sfb[n] * sum_k A[m, k] * B[n, k]
 * A and B int8, K-major.  The sums are exact in int32; the result is
 * fp32(sum) * sfa * sfb, each step rounded to fp32, then rounded once to D's type.  So it
 * does not depend on tiles, splits or the grid width, and rows past a group's
 * end, or padding, change nothing.  Scales: sfa[i * sfa_s] for row i, sfb[j * sfb_s]
 * for channel j; any fp32 (a NaN or infinite scale shows in its row or column).
 *   d     device, out_dtype (DG_BF16, DG_F16 or DG_F32), row stride ldd (elements);
 *         16-byte stores where its rows lie on such boundaries, single elements
 *         elsewhere, so any n and ldd >= n will do
 * Alignment: K % 16 == 0 and K <= 131071; lda, ldb and the A/B base addresses are
 * multiples of 16 bytes.  A K that is no multiple of 128 costs one more step a
 * tile.  Violations return DG_ERROR_NOT_SUPPORTED.  The size contract above holds.
 *
 * The three forms take the tiles, plans, workspace and control calls of their
 * FP8 counterparts (dg_set_dense_plan, dg_set_contiguous_plan, dg_set_num_cus).
 */

/* Dense.  ws as in dg_fp8_gemm_nt_ws (the workspaces are interchangeable); NULL:
 * no K split. */
dg_status dg_int8_gemm_nt(const void* a, int64_t lda, const float* sfa, int64_t sfa_s,
                          const void* b, int64_t ldb, const float* sfb, int64_t sfb_s,
                          void* d, int out_dtype, int64_t ldd,
                          int64_t m, int64_t n, int64_t k,
                          void* ws, size_t ws_bytes, void* stream);
size_t dg_int8_gemm_nt_workspace_size(int64_t m, int64_t n, int64_t k);

/* M-grouped, contiguous layout: groups, m_indices, ws and preconditions as in
 * dg_m_grouped_fp8_gemm_nt_contiguous_ws.  b int8 [num_groups, n, k], sfb fp32
 * [num_groups, n] with group stride sfb_group_stride. */
dg_status dg_m_grouped_int8_gemm_nt_contiguous(const void* a, int64_t lda, const float* sfa, int64_t sfa_s,
                                               const void* b, int64_t ldb, int64_t b_group_stride,
                                               const float* sfb, int64_t sfb_s, int64_t sfb_group_stride,
                                               void* d, int out_dtype, int64_t ldd,
                                               const int32_t* m_indices, int64_t m_total,
                                               int64_t n, int64_t k, int num_groups,
                                               void* ws, size_t ws_bytes, void* stream);
size_t dg_m_grouped_int8_gemm_nt_contiguous_workspace_size(int64_t m_total, int64_t n, int64_t k,
                                                           int num_groups);

/* M-grouped, masked layout: masked_m and expected_m as in
 * dg_m_grouped_fp8_gemm_nt_masked.  sfa fp32 [num_groups, max_m], sfb fp32
 * [num_groups, n]. */
dg_status dg_m_grouped_int8_gemm_nt_masked(const void* a, int64_t lda, int64_t a_group_stride,
                                           const float* sfa, int64_t sfa_s, int64_t sfa_group_stride,
                                           const void* b, int64_t ldb, int64_t b_group_stride,
                                           const float* sfb, int64_t sfb_s, int64_t sfb_group_stride,
                                           void* d, int out_dtype, int64_t ldd, int64_t d_group_stride,
                                           const int32_t* masked_m, int num_groups,
                                           int64_t max_m, int64_t n, int64_t k,
                                           int64_t expected_m, void* stream);

/*
 * int8 cast of rows (a token's activations, or a channel's weights):
 *   amax = max |x| over the row;  s = fl32(max(amax, 1e-4) / 127);
 *   q = fl32(x / s) rounded to the nearest whole number, ties to even: -127..127.
 * Bit-exact with this definition.  A row with an infinity or a NaN gets an
 * infinite or NaN scale and unspecified codes: the product's row shows it.  The floor of 1e-4
 * is the FP8 cast's; a row whose maximum lies below it uses fewer than 127 steps.
 *   x   device, dtype (DG_F32 or DG_BF16) [m, k], row stride ldx, rows at 16-byte
 *       boundaries
 *   q   device, int8 [m, k], row stride ldq, rows at 16-byte boundaries
 *   sf  device, fp32 [m], stride sf_s
 * Limits: k % 16 == 0, m <= 2^23.
 */
dg_status dg_per_token_cast_int8(const void* x, int dtype, int64_t ldx, void* q, int64_t ldq,
                                 float* sf, int64_t sf_s, int64_t m, int64_t k, void* stream);

/*
 * ---------------------------------------------------------------------------
 * Mixture of experts: routing, expert layout, dispatch, combination
 *
 * What stands between a router's logits and the grouped GEMMs above, and
 * between their outputs and the tokens.  All calls read their sizes from the
 * host and everything else on the device, so a whole layer can be captured in
 * a graph.  Element types are named by dg_dtype; 16-bit rows move in 16-byte
 * pieces (see each call's alignment).  Statistics and sums are fp32.
 */
typedef enum dg_route_score { DG_ROUTE_SOFTMAX = 0, DG_ROUTE_SIGMOID = 1 } dg_route_score;

/*
 * Routing: the topk experts of each token and their weights.
 *   logits  device, dtype [tokens, experts], row stride ld; element-aligned (rows
 *           at 16-byte boundaries load faster)
 *   bias    device, fp32 [experts] or NULL: added to the scores for the choice,
 *           never for the weights (balancing of the experts' load)
 *   indices device, int32 [tokens, topk], row stride ldi
 *   weights device, fp32 [tokens, topk], row stride ldw
 * Scores s: softmax over the token's logits, or the sigmoid of each.  Experts are
 * ranked by s + bias, or without a bias by the logit itself (the same order,
 * without the merging of close scores by rounding).  groups > 1 splits the experts into
 * equal consecutive groups, of which only the best topk_groups take part: by
 * their largest key (group_top2 == 0), or by the sum of the two largest s + bias
 * (group_top2 != 0; a single available expert counts alone).  Of equal keys, and
 * of equal groups, the lower number comes first.  Slot j of a token is its j-th
 * largest key:
 *   w_j = scale * s_j,  or  scale * s_j / (sum of the chosen s)  if renormalize != 0
 * (0 if that sum is 0: every chosen sigmoid underflowed).
 *   Scores are fp32, within a few units of their last place, and a row's softmax is summed in an
 * order that depends on tokens, experts and groups.  With a bias or group sums, keys that close
 * may be ranked differently in calls of different sizes; the same call always gives the same bits.
 *   Unavailable experts: a logit or a bias of -inf takes an expert out.  Where
 * fewer than topk are left, the last slots get index -1 and weight 0 (a row
 * masked whole gets only those).  A NaN logit or bias (and, under softmax, a
 * logit of +inf) also takes its expert out, and makes the token's weights NaN.
 * Limits: 1 <= experts <= 1024, 1 <= topk <= min(64, experts), 1 <= topk_groups <=
 * groups <= 64, experts % groups == 0, tokens <= 2^23.
 * Errors: null pointers, sizes or enumerators outside these, ld < experts, ldi or
 * ldw < topk -> DG_ERROR_INVALID_VALUE; experts, topk, groups or tokens above
 * their maximum, strides over 2^40, misaligned pointers -> DG_ERROR_NOT_SUPPORTED.
 */
dg_status dg_route_topk(const void* logits, int dtype, int64_t ld, const float* bias,
                        int32_t* indices, int64_t ldi, float* weights, int64_t ldw,
                        int64_t tokens, int experts, int topk, int groups, int topk_groups,
                        int group_top2, int score, int renormalize, float scale, void* stream);

/*
 * Gradient of dg_route_topk's weights with respect to the logits, the choice
 * held fixed: dlogits[t, e] = sum_j dweights[t, j] * d w[t, j] / d logits[t, e].
 * Every element of dlogits is written.
 *   indices   as dg_route_topk wrote them: the experts of a token are distinct;
 *             an index outside [0, experts) marks an unused slot
 *   dweights  device, fp32 [tokens, topk], row stride ldw
 *   dlogits   device, dtype [tokens, experts], row stride ldd; must not overlap logits
 * Under plain softmax every score depends on every logit: a token with a NaN (or +inf) logit
 * gets a row of NaN.  In the other forms only the chosen experts' logits enter, so such a logit
 * of an expert that is not chosen leaves the row finite, though the token's weights are NaN.
 * Limits and errors as dg_route_topk (ldd < experts -> DG_ERROR_INVALID_VALUE).
 */
dg_status dg_route_topk_grad(const void* logits, int dtype, int64_t ld, const int32_t* indices, int64_t ldi,
                             const float* dweights, int64_t ldw, void* dlogits, int64_t ldd,
                             int64_t tokens, int experts, int topk, int score, int renormalize,
                             float scale, void* stream);

/*
 * Expert layout for dg_m_grouped_*_gemm_nt_contiguous: a row for each slot (t, j)
 * whose index is in [0, experts).  Experts follow one another in order, each
 * from a multiple of 128 rows; within an expert the rows are in order of token and slot,
 * so the layout is a function of the indices alone.
 *   indices   device, int32 [tokens, topk], row stride ldi; others than 0..experts-1
 *             have no row (dropped assignments)
 *   rows      rows of the layout, a multiple of 128.
 *             dg_expert_layout_rows() rows hold every routing; where fewer are
 *             given, slots beyond them are dropped
 *   m_indices device, int32 [rows]: expert of the row, -1 where it holds no slot
 *   row_slot  device, int32 [rows]: t * topk + j of the row's slot, or -1
 *   slot_row  device, int32 [tokens, topk], dense: row of the slot, or -1
 *   counts    device, int32 [experts]: slots of each expert
 *   ws        device, 16-byte aligned, dg_expert_layout_workspace_size() bytes
 *             (contents do not matter); not used, and may be NULL, up to 3072 slots
 * Limits: experts <= 1024, topk <= 64, tokens * topk <= 2^30, rows < 2^31.
 * Errors: rows % 128 != 0 -> DG_ERROR_MISALIGNED_LAYOUT; null pointers, negative
 * sizes, ldi < topk, ws too small -> DG_ERROR_INVALID_VALUE; beyond the limits, or
 * misaligned -> DG_ERROR_NOT_SUPPORTED.  tokens == 0 clears the layout.
 */
dg_status dg_expert_layout_contiguous(const int32_t* indices, int64_t ldi, int64_t tokens, int topk, int experts,
                                      int64_t rows, int32_t* m_indices, int32_t* row_slot, int32_t* slot_row,
                                      int32_t* counts, void* ws, size_t ws_bytes, void* stream);

/* Rows that hold every routing of these sizes in the contiguous layout (a
 * multiple of 128); 0 for sizes outside the limits. */
int64_t dg_expert_layout_rows(int64_t tokens, int topk, int experts);

/* Workspace bytes that serve the two layout calls: 0 up to 1024 slots. */
size_t dg_expert_layout_workspace_size(int64_t tokens, int topk, int experts);

/*
 * Expert layout for dg_m_grouped_*_gemm_nt_masked: the slots of expert e get the
 * rows e * max_m, e * max_m + 1, ... in order of token and slot; those past max_m
 * are dropped.  masked_m receives min(slots of e, max_m).  Other arguments,
 * limits (experts * max_m < 2^31) and errors as the contiguous call's.
 *   row_slot  device, int32 [experts * max_m]
 */
dg_status dg_expert_layout_masked(const int32_t* indices, int64_t ldi, int64_t tokens, int topk, int experts,
                                  int64_t max_m, int32_t* masked_m, int32_t* row_slot, int32_t* slot_row,
                                  void* ws, size_t ws_bytes, void* stream);

/*
 * Dispatch: quantizes each token's row once, as dg_per_token_cast_fp8 (the same
 * codes and scales, bit for bit), and writes it to the row of each of its slots.
 * Rows no slot has are left untouched.
 *   x         device, dtype (DG_F32 or DG_BF16) [tokens, k], row stride ldx, rows at
 *             16-byte boundaries
 *   slot_row  device, int32 [tokens, topk], row stride lds; values outside
 *             [0, rows) are skipped.  No row may be named twice.
 *   q         device, E4M3 [rows, k], row stride ldq (bytes), rows at 16-byte boundaries
 *   sf        device, fp32 [rows, k/128]: element (r, kb) at sf[r * sf_sm + kb * sf_sk]
 * Limits: k % 128 == 0, topk <= 64, tokens <= 2^23.  Errors as the casts'.
 */
dg_status dg_dispatch_cast_fp8(const void* x, int dtype, int64_t ldx, const int32_t* slot_row, int64_t lds,
                               void* q, int64_t ldq, float* sf, int64_t sf_sm, int64_t sf_sk,
                               int64_t tokens, int topk, int64_t rows, int64_t k, int ue8m0, void* stream);

/* Dispatch with the int8 cast of dg_per_token_cast_int8: q int8 [rows, k], sf
 * fp32 [rows] with stride sf_s.  k % 16 == 0. */
dg_status dg_dispatch_cast_int8(const void* x, int dtype, int64_t ldx, const int32_t* slot_row, int64_t lds,
                                void* q, int64_t ldq, float* sf, int64_t sf_s,
                                int64_t tokens, int topk, int64_t rows, int64_t k, void* stream);

/*
 * Combination: out[t] = sum_j weights[t, j] * y[slot_row[t, j]] over the slots that
 * have a row, summed in slot order in fp32 and rounded once to out's type.  A
 * token without any row gets zeros; rows no slot names are not read.
 *   y         device, bf16 [rows, h], row stride ldy: the grouped GEMM's output
 *   slot_row  device, int32 [tokens, topk], row stride lds; values outside [0, rows)
 *             are skipped
 *   weights   device, fp32 [tokens, topk], row stride ldw, or NULL: all ones (the
 *             gradient of dispatching tokens to rows)
 *   out       device, out_dtype (DG_BF16 or DG_F32) [tokens, h], row stride ldo
 * Limits: h % 8 == 0, topk <= 64, tokens <= 2^23; rows of y and out at 16-byte
 * boundaries.
 */
dg_status dg_combine(const void* y, int64_t ldy, const int32_t* slot_row, int64_t lds,
                     const float* weights, int64_t ldw, void* out, int out_dtype, int64_t ldo,
                     int64_t tokens, int topk, int64_t rows, int64_t h, void* stream);

/*
 * Gradient of dg_combine:
 *   dy[r] = weights[t, j] * dout[t] where slot (t, j) has row r, zero elsewhere (bf16);
 *   dweights[t, j] = <dout[t], y[slot_row[t, j]]> in fp32, 0 without a row.
 *   dout      device, bf16 [tokens, h], row stride ldo
 *   row_slot  device, int32 [rows], as the layout call wrote it beside slot_row: it
 *             says which rows of dy to clear
 *   dy        device, bf16 [rows, h], row stride lddy, must not overlap y or dout
 *   dweights  device, fp32 [tokens, topk], row stride lddw
 * Other arguments and limits as dg_combine.
 */
dg_status dg_combine_grad(const void* dout, int64_t ldo, const void* y, int64_t ldy,
                          const int32_t* slot_row, int64_t lds, const int32_t* row_slot,
                          const float* weights, int64_t ldw, void* dy, int64_t lddy,
                          float* dweights, int64_t lddw,
                          int64_t tokens, int topk, int64_t rows, int64_t h, void* stream);

/*
 * ---------------------------------------------------------------------------
 * Around the products of a layer: norm, gated activation, weights' gradients
 *
 * What a layer needs besides routing: the norm before it (with the residual's
 * addition and the cast), the gated activation between its two products (with the
 * cast, and an 8-bit checkpoint of its input), their gradients, and the gradients of the
 * weights over each expert's rows, from the 8-bit activations that the forward pass
 * kept.  Conventions as above: sizes on the host, everything else on the device;
 * statistics and sums in fp32; rows at 16-byte boundaries; strides in elements.
 * Codes and scales follow dg_per_token_cast_fp8 and dg_per_token_cast_int8 for
 * the fp32 values that are cast, except that a NaN shows: a block (int8: a row) that
 * holds one gets a NaN scale.
 */

/*
 * Root-mean-square norm of rows, with the residual's addition:
 *   h = x + residual, rounded to x's type;
 *   rstd = (sum h^2 / k + eps)^-1/2;   y = h * rstd * weight, rounded to x's type.
 * The norm is that of the rounded h, so that h and rstd are all its gradient needs.
 * y's fp32 value is (h * weight) * rstd: a product of 16-bit h and weight is exact, so that one
 * rounding stands before the store or the cast (h * weight past fp32's range shows).
 *   x         device, dtype [rows, k], row stride ldx
 *   residual  device, dtype [rows, k], row stride ldr, or NULL: h = x
 *   weight    device, [k] of weight_dtype (dtype or DG_F32), 16-byte aligned, or NULL: ones
 *   eps       >= 0, finite.  A row of zeros with eps == 0 gives NaN
 *   h         device, dtype [rows, k], row stride ldh, or NULL: not written
 *   y         device, dtype [rows, k], row stride ldy
 *   rstd      device, fp32 [rows], or NULL: not written
 * h and y may be x or residual (same address and stride), not each other.  An element past
 * 1.8e19 overflows its square: rstd is 0 then.  A NaN or an infinity makes its row NaN
 * (where it is finite, 0).
 * Limits: k % 8 == 0, k <= 16384, rows <= 2^23 (2^21 where k > 8192) -> otherwise
 * DG_ERROR_NOT_SUPPORTED, as for misaligned rows.  k == 0: nothing is written, rstd and int8 scales
 * neither.
 */
dg_status dg_rms_norm(const void* x, int dtype, int64_t ldx, const void* residual, int64_t ldr,
                      const void* weight, int weight_dtype, float eps, void* h, int64_t ldh,
                      void* y, int64_t ldy, float* rstd, int64_t rows, int64_t k, void* stream);

/* The same with the FP8 cast of y's fp32 values: q E4M3 [rows, k], row stride ldq; sf fp32
 * [rows, k/128] with strides sf_sm, sf_sk; ue8m0 as in the casts.  k % 128 == 0.
 * y may be NULL: not written. */
dg_status dg_rms_norm_cast_fp8(const void* x, int dtype, int64_t ldx, const void* residual, int64_t ldr,
                               const void* weight, int weight_dtype, float eps, void* h, int64_t ldh,
                               void* y, int64_t ldy, float* rstd, void* q, int64_t ldq,
                               float* sf, int64_t sf_sm, int64_t sf_sk,
                               int64_t rows, int64_t k, int ue8m0, void* stream);

/* The same with the int8 cast: q int8 [rows, k], sf fp32 [rows] with stride sf_s.
 * k % 16 == 0. */
dg_status dg_rms_norm_cast_int8(const void* x, int dtype, int64_t ldx, const void* residual, int64_t ldr,
                                const void* weight, int weight_dtype, float eps, void* h, int64_t ldh,
                                void* y, int64_t ldy, float* rstd, void* q, int64_t ldq,
                                float* sf, int64_t sf_s, int64_t rows, int64_t k, void* stream);

/*
 * Gradient of the norm, with n = h * rstd:
 *   dx = dh + rstd * (weight * dy - n * mean(weight * dy * n)),  rounded to dtype;
 *   dweight = sum over the rows of dy * n,  fp32.
 * dx is the gradient of x and of the residual alike.
 *   dy, h     device, dtype [rows, k]: the gradient of y, and h as the norm wrote it
 *   rstd      device, fp32 [rows], as the norm wrote it
 *   dh        device, dtype [rows, k], row stride lddh: the gradient that reaches h by another
 *             way (the residual stream), or NULL: none
 *   dx        device, dtype [rows, k], row stride lddx; may be dy, h or dh (same stride)
 *   dweight   device, fp32 [k], or NULL: not computed.  Overwritten; without rows, zeros
 *   ws        device, 16-byte aligned, dg_rms_norm_grad_workspace_size() bytes (contents do
 *             not matter); may be NULL without dweight
 * Sums are taken in an order that rows and k alone give.  Limits as dg_rms_norm.
 */
dg_status dg_rms_norm_grad(const void* dy, int dtype, int64_t lddy, const void* h, int64_t ldh,
                           const void* weight, int weight_dtype, const float* rstd,
                           const void* dh, int64_t lddh, void* dx, int64_t lddx, float* dweight,
                           int64_t rows, int64_t k, void* ws, size_t ws_bytes, void* stream);
size_t dg_rms_norm_grad_workspace_size(int64_t rows, int64_t k);

/*
 * Gated activation with the FP8 cast:  a = silu(h[:, :inner]) * h[:, inner:], silu(g) =
 * g / (1 + e^-g), in fp32 from the stored h, then cast in blocks of 128.
 *   h         device, dtype [rows, 2 * inner], row stride ldh: gate and up side by side
 *   m_indices device, int32 [rows], or NULL: rows whose entry is negative are left untouched
 *             (the contiguous layout's padding)
 *   masked_m  device, int32 [num_groups], or NULL: rows is num_groups * max_m, and only the first
 *             masked_m[g] rows of each group's are done (clamped to 0..max_m).  Not both
 *   q, sf     device, E4M3 [rows, inner], fp32 [rows, inner/128] with strides sf_sm, sf_sk
 *   hq, hsf   device, E4M3 [rows, 2 * inner], fp32 [rows, 2 * inner / 128]: the FP8 cast of h
 *             itself, for dg_swiglu_grad; or hq NULL: none
 * Limits: inner % 128 == 0, inner <= 2^24, rows <= 2^23, num_groups <= 1024.
 */
dg_status dg_swiglu_cast_fp8(const void* h, int dtype, int64_t ldh, const int32_t* m_indices,
                             const int32_t* masked_m, int num_groups, void* q, int64_t ldq,
                             float* sf, int64_t sf_sm, int64_t sf_sk, void* hq, int64_t ldhq,
                             float* hsf, int64_t hsf_sm, int64_t hsf_sk,
                             int64_t rows, int64_t inner, int ue8m0, void* stream);

/* The same with the int8 cast: q int8 [rows, inner], sf fp32 [rows] with stride sf_s.
 * inner % 16 == 0, inner <= 16384.  inner == 0: the scales of rows of zeros. */
dg_status dg_swiglu_cast_int8(const void* h, int dtype, int64_t ldh, const int32_t* m_indices,
                              const int32_t* masked_m, int num_groups, void* q, int64_t ldq,
                              float* sf, int64_t sf_s, int64_t rows, int64_t inner, void* stream);

/*
 * Gradient of the gated activation, with g, u the halves of h and s = 1 / (1 + e^-g):
 *   dh[:, :inner] = da * u * s * (1 + g * (1 - s)),   dh[:, inner:] = da * g * s.
 *   da        device, dtype [rows, inner], row stride ldda
 *   h         device, dtype [rows, 2 * inner]; or NULL and
 *   hq, hsf   the checkpoint that dg_swiglu_cast_fp8 wrote: the gradient at the values that it
 *             stands for
 *   m_indices, masked_m as in dg_swiglu_cast_fp8
 *   dh        device, dtype [rows, 2 * inner], row stride lddh; may be h (same stride)
 *   q, sf     device, E4M3 [rows, 2 * inner], fp32 [rows, 2 * inner / 128]: the FP8 cast of dh's fp32
 *             values, for the product that follows; or q NULL: none
 * inner % 128 == 0 with codes on either side, otherwise inner % 8 == 0; limits as above.
 */
dg_status dg_swiglu_grad(const void* da, int dtype, int64_t ldda, const void* h, int64_t ldh,
                         const void* hq, int64_t ldhq, const float* hsf, int64_t hsf_sm, int64_t hsf_sk,
                         const int32_t* m_indices, const int32_t* masked_m, int num_groups,
                         void* dh, int64_t lddh, void* q, int64_t ldq,
                         float* sf, int64_t sf_sm, int64_t sf_sk,
                         int64_t rows, int64_t inner, int ue8m0, void* stream);

/*
 * Gradient of a weight [n, k] of a product y = x . W^T:  dw[n, k] = sum over the rows r of
 * dy[r, n] * x[r, k].
 *   dy        device, bf16 [rows, n], row stride lddy
 *   x         device, [rows, k], row stride ldx: bf16 where sf is NULL; otherwise E4M3 codes with
 *             scales sf, fp32 [rows, k/128] with strides sf_sm, sf_sk (the operand that the forward
 *             product read).  A code times its scale enters the product rounded to bf16: exact where
 *             the scale is a power of two.
 *   dw        device, out_dtype (DG_F32 or DG_BF16) [n, k], row stride lddw
 *   accumulate  nonzero: the sum is added to dw (DG_F32 only)
 *   ws        device, 16-byte aligned, dg_weight_grad_workspace_size() bytes (contents do not
 *             matter): lets several workgroups share a tile's rows where there are few tiles; NULL
 *             or smaller: they do not.  Calls that may overlap need distinct ones
 * Sums are fp32, in an order that the sizes, num_groups and whether ws is there alone give.
 * Limits: n % 8 == 0, k % 8 == 0 (codes: k % 128 == 0), n, k, lddy, ldx, sf_sm < 2^24, rows < 2^31, at
 * most 2^22 tiles of 128 x 128 in dw (of all groups), rows of dy, x and dw at 16-byte boundaries ->
 * otherwise DG_ERROR_NOT_SUPPORTED.  rows == 0 gives zeros.
 */
dg_status dg_weight_grad(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                         const float* sf, int64_t sf_sm, int64_t sf_sk,
                         void* dw, int out_dtype, int64_t lddw, int accumulate,
                         int64_t rows, int64_t n, int64_t k, void* ws, size_t ws_bytes, void* stream);
size_t dg_weight_grad_workspace_size(int64_t rows, int64_t n, int64_t k, int num_groups);

/*
 * The same for each group (expert) of rows: dw [num_groups, n, k] with group stride
 * dw_group_stride, at least k: no element of dw may belong to two groups.  Groups follow one
 * another, each from a multiple of `alignment` rows (128: dg_expert_layout_contiguous; 1: no
 * padding), counts[g] rows of which count; what lies between them may hold anything.  A group
 * without rows gets zeros (accumulate: nothing).
 *   counts    device, int32 [num_groups]; negative ones count as 0, and rows past `rows` are
 *             left out
 * num_groups <= 1024.
 */
dg_status dg_m_grouped_weight_grad_contiguous(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                              const float* sf, int64_t sf_sm, int64_t sf_sk,
                                              void* dw, int out_dtype, int64_t lddw, int64_t dw_group_stride,
                                              const int32_t* counts, int num_groups, int64_t alignment,
                                              int accumulate, int64_t rows, int64_t n, int64_t k,
                                              void* ws, size_t ws_bytes, void* stream);

/* The same in the masked layout: group g's rows are g * max_m .. g * max_m + masked_m[g] - 1
 * (masked_m clamped to 0..max_m) of [num_groups * max_m, ...] operands. */
dg_status dg_m_grouped_weight_grad_masked(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                          const float* sf, int64_t sf_sm, int64_t sf_sk,
                                          void* dw, int out_dtype, int64_t lddw, int64_t dw_group_stride,
                                          const int32_t* masked_m, int num_groups, int64_t max_m,
                                          int accumulate, int64_t n, int64_t k,
                                          void* ws, size_t ws_bytes, void* stream);

/*
 * Width of the persistent GEMM grid in compute units (default: all CUs of the
 * current device).  Results never depend on it.  num_cus <= 0 restores the
 * default.  (Analog of set_num_sms: page ssnai.com DeepGEMM analysis.)
 */
dg_status dg_set_num_cus(int num_cus);
int dg_get_num_cus(void);

#ifdef __cplusplus
}
#endif

#endif /* DGFP8_H_ */
