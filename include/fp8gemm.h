/*
 * fp8gemm.h -- C ABI of libfp8gemm.so: fine-grained block-scaled E4M3 GEMM
 * (Y = X * W^T, BF16 out) and its quantizers, hand-written for AMD gfx950
 * (MI355X, CDNA4).
 *
 * Sources (page title, section):
 *   [DG]  "DeepGEMM 完全拆解：300 行 FP8 GEMM 内核，如何逼近 Hopper 的算力峰值"
 *   [TC]  "GPU GEMM 优化完全拆解(四): tcgen05 与 Blackwell", section 六 (6.1)
 *   [MLC] "Blackwell Tensor Core: tcgen05.mma", section "Block-Scaled MMA"
 *
 * Common conventions
 *   - Every pointer argument is a DEVICE pointer owned by the caller.  The
 *     library never allocates, frees, retains or synchronizes; each call only
 *     enqueues kernels on `stream` (a hipStream_t, NULL = the null stream) and
 *     returns.  Outputs must not alias inputs.
 *   - E4M3 is OCP E4M3FN (bias 7, largest finite 448, NaN = S.1111.111).
 *     BF16 outputs are stored as raw uint16_t bit patterns, rounded to
 *     nearest-even.
 *   - Layouts are row-major.  The activation scale table is "MN-major":
 *     sa[kb][m] at sa + kb*M + m, kb = k/128  ([DG] "为什么只做 NT 布局": the
 *     (M, K/128) activation scales are handed over transposed as (K/128, M)).
 *     The weight scale table is sb[nb][kb] at sb + nb*(K/128) + kb, nb = n/128.
 *   - K must be a multiple of 128 (the scale granularity along K; [DG]
 *     "线程组织": the K block is fixed at 128 because scaling is per 128
 *     channels).
 *   - Errors are detected on the host before anything is enqueued:
 *       FP8_ERR_INVALID_ARG  null pointer, negative or oversized dimension,
 *                            unknown flag bit
 *       FP8_ERR_SHAPE        K % 128 != 0; N % 128 != 0 for grouped calls
 *       FP8_ERR_ALIGNMENT    a pointer not 16-byte aligned
 *       FP8_ERR_NO_DEVICE    no HIP device is usable
 *       FP8_ERR_LAUNCH       the kernel launch reported an error
 *       FP8_ERR_SCRATCH      the workspace is smaller than the call needs
 *                            (fp8_gemm_nt_noalloc: the problem needs more
 *                            split-K scratch than its fixed array holds)
 *     A call with an empty problem (M == 0, E == 0, N == 0 ...) returns FP8_OK
 *     and enqueues nothing.  Device-side data (expert indices, valid counts)
 *     is never reported as an error: its handling is defined per call.
 *   - NaN or infinite inputs give unspecified (but in-bounds) results.
 *   - Thread safety: all calls are reentrant; the only global state is a
 *     per-device cache of the compute-unit count, filled once.
 */
#ifndef FP8GEMM_H
#define FP8GEMM_H
#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FP8_OK = 0,
    FP8_ERR_INVALID_ARG = 1,
    FP8_ERR_SHAPE = 2,
    FP8_ERR_ALIGNMENT = 3,
    FP8_ERR_UNSUPPORTED = 4,
    FP8_ERR_NO_DEVICE = 5,
    FP8_ERR_LAUNCH = 6,
    FP8_ERR_SCRATCH = 7
} fp8_status;

/* Quantizers: round each group's scale up to a power of two (UE8M0, [DG]
 * "离群值如何摧毁 per-tensor 量化": Blackwell MXFP8 takes power-of-two UE8M0
 * scales).  GEMMs: the scales are powers of two; only the biased exponent of
 * each FP32 scale is used (value 2^(e-127)) and the block scaling runs inside
 * the matrix instruction. */
#define FP8_FLAG_UE8M0 1u

/* GEMMs only: form each 128-K block partial with the FP8 matrix instruction
 * (twice the FP16 matrix rate) instead of exactly.
 *
 * Default (flag clear): the E4M3 operands are widened to FP16, which is exact,
 * and multiplied by FP16 matrix instructions: every product is exact and
 * every sum FP32-accurate, so Y is the exact block-scaled sum up to FP32
 * accumulation and BF16 rounding, i.e. within |y - ref| <= 8e-3*|ref| +
 * 1e-3*rms(ref) of the exact value ref barring cancellation below FP32
 * precision ([DG] "细粒度缩放在 GEMM 层面引爆的两个问题": the promotion exists
 * so that the sum is accumulated at full precision).
 *
 * FP8_FLAG_FAST_ACCUM: the FP8 instruction of gfx950 truncates, within each
 * group of 8 consecutive K, every product toward zero to a multiple of
 * 2^(E-13), 2^E being the group's largest product magnitude (measured; the
 * analog of the limited FP8 accumulation precision the DeepGEMM page reports
 * for H800 tensor cores).  Per output element the error therefore stays below
 *   2^-10 * sum over 8-groups g of sa*sb * max_{k in g} |x[m][k]| * max_{k in g} |w[n][k]|
 * (decoded E4M3 values, the scales of g's block) plus FP32/BF16 rounding,
 * which can exceed the tolerance above where the sum cancels.  With
 * FP8_FLAG_UE8M0 the block scaling then runs inside the scaled FP8
 * instruction and the K sum stays in its FP32 accumulator. */
#define FP8_FLAG_FAST_ACCUM 2u

/*
 * Activation quantizer, 1x128 groups ([DG] "离群值如何摧毁 per-tensor 量化":
 * activations are grouped per token and per 128 channels; the scale is the
 * group's absolute maximum over 448, computed online).
 *   x   fp32 (M, K)           input
 *   xq  u8   (M, K)           output codes, q = E4M3(fl32(x / s))
 *   sa  fp32 [K/128][M]       output scales, s = fl32(max(amax, 1e-4) / 448)
 *                             (rounded up to 2^k with FP8_FLAG_UE8M0)
 */
fp8_status fp8_quant_1x128(const float* x, int64_t M, int64_t K, uint8_t* xq,
                           float* sa, uint32_t flags, void* stream);

/*
 * Weight quantizer, 128x128 blocks ([DG] same section: weights are grouped 128
 * input by 128 output channels).  The last block row is ragged when
 * N % 128 != 0.
 *   w   fp32 (N, K)                 input
 *   wq  u8   (N, K)                 output codes
 *   sb  fp32 [ceil(N/128)][K/128]   output block scales (as for sa)
 */
fp8_status fp8_quant_128x128(const float* w, int64_t N, int64_t K, uint8_t* wq,
                             float* sb, uint32_t flags, void* stream);

/*
 * Dense NT GEMM ([DG] "为什么只做 NT 布局": Y = X W^T with X (M,K) row-major and
 * W stored (N,K) K-contiguous; [TC] 6.1 block-scaled GEMM definition;
 * [DG] "主循环骨架": FP32 partial sums of each 128-K block are multiplied by
 * sA*sB and added to a full-precision accumulator).
 *   Y[m][n] = sum_kb sa[kb][m] * sb[n/128][kb] * sum_{k in kb} xq[m][k]*wq[n][k]
 *   xq u8 (M,K), sa fp32 [K/128][M], wq u8 (N,K), sb fp32 [ceil(N/128)][K/128],
 *   y  bf16 bits (M,N).
 * flags: FP8_FLAG_UE8M0, FP8_FLAG_FAST_ACCUM.  Uses the caller's buffers only
 * (equivalent to fp8_gemm_nt_ws with no workspace).
 * Scales are finite and non-negative; a zero scale is taken to come with
 * all-zero codes in its group (the quantizers never write one: their scales
 * are at least 1e-4/448).  The default path keeps its accumulator in units
 * of the current block's scale product and skips a zero factor, so nonzero
 * codes under a zero scale are outside its contract.
 */
fp8_status fp8_gemm_nt(const uint8_t* xq, const float* sa, const uint8_t* wq,
                       const float* sb, uint16_t* y, int64_t M, int64_t N,
                       int64_t K, uint32_t flags, void* stream);

/*
 * fp8_gemm_nt with a caller-owned device workspace.  For decode-sized M (the
 * default path: M <= 64; FP8_FLAG_FAST_ACCUM: M <= 32) and fewer 96-column
 * tiles than compute units, the decode kernel splits K over up to 8
 * workgroups per tile when `workspace` holds their FP32 partial sums, and a
 * second kernel adds them in split order (the same result for the same
 * split).  fp8_gemm_workspace_size() gives the bytes that enable
 * the split for a shape on the current device (0: no split).  With a smaller
 * or no workspace the GEMM runs unsplit.  The workspace is only read and
 * written by this call's kernels, in stream order; calls that overlap on one
 * workspace race.  workspace_bytes > 0 needs a non-NULL, 16-byte aligned
 * workspace.
 */
fp8_status fp8_gemm_nt_ws(const uint8_t* xq, const float* sa, const uint8_t* wq,
                          const float* sb, uint16_t* y, int64_t M, int64_t N,
                          int64_t K, uint32_t flags, void* workspace,
                          size_t workspace_bytes, void* stream);

/*
 * fp8_gemm_nt for callers that cannot allocate (code under graph capture,
 * tight serving loops, harnesses that forbid hipMalloc): fp8_gemm_nt_ws with
 * the split-K workspace taken from a fixed 8 MiB device array inside the
 * library (one per GPU, loaded with the library, held until the process
 * ends) instead of the caller's memory.  Calls no hipMalloc, hipFree or
 * other allocating routine; the first call on a device looks up that
 * device's array.  The result equals fp8_gemm_nt_ws with a workspace of
 * fp8_gemm_workspace_size() bytes.  A shape whose split needs more than the
 * array (none on a device of up to 341 compute units) returns
 * FP8_ERR_SCRATCH before any launch.  Every call on one GPU shares the
 * array: calls that overlap on one GPU (several streams, or several host
 * threads) race on it and must be ordered by the caller.  Each split writes
 * every partial sum it covers before the reduction reads it, so nothing
 * needs clearing between calls.
 */
fp8_status fp8_gemm_nt_noalloc(const uint8_t* xq, const float* sa, const uint8_t* wq,
                               const float* sb, uint16_t* y, int64_t M, int64_t N,
                               int64_t K, uint32_t flags, void* stream);

/* Workspace bytes with which fp8_gemm_nt_ws splits K for this shape and these
 * flags on the current device (0 when it does not split, or on bad
 * arguments). */
size_t fp8_gemm_workspace_size(int64_t M, int64_t N, int64_t K, uint32_t flags);

/*
 * Dense NT GEMM whose output is quantized for the next GEMM in the epilogue
 * ([DG] "为什么只做 NT 布局": DeepGEMM leaves the activation quantization to
 * the caller, to be fused into the kernel that produces the activations).
 * Y is computed as by fp8_gemm_nt and, instead of BF16, written as the 1x128
 * activation quantizer would write it, from the FP32 accumulator:
 *   yq  u8   (M,N)         E4M3 codes, E4M3(acc / s)
 *   sy  fp32 [N/128][M]    s = fl32(max(amax, 1e-4)/448) over the 128
 *                          columns of the group (rounded up to 2^k with
 *                          FP8_FLAG_UE8M0, which also marks the input scales)
 * so (yq, sy) is the (xq, sa) of a following fp8_gemm_nt with K = N.
 * N % 128 == 0; flags as for fp8_gemm_nt.
 */
fp8_status fp8_gemm_nt_qout(const uint8_t* xq, const float* sa, const uint8_t* wq,
                            const float* sb, uint8_t* yq, float* sy, int64_t M,
                            int64_t N, int64_t K, uint32_t flags, void* stream);

/*
 * Grouped GEMM, contiguous layout ([DG] "分组 GEMM 的两种布局": the tokens of
 * each expert form one segment along M, N and K are shared by all experts,
 * each segment is aligned to the M block reported by
 * fp8_get_mk_alignment_for_contiguous_layout()).
 *   xq u8 (M,K), sa fp32 [K/128][M], m_indices int32 (M) on the device,
 *   wq u8 (E,N,K), sb fp32 (E, N/128, K/128), y bf16 bits (M,N).  N % 128 == 0.
 *   Row r uses expert m_indices[r].  Each aligned 128-row block is computed
 *   with the expert of its first row whose index lies in [0,E); a row is
 *   written only if its index equals that expert, every other row (padding
 *   rows with -1, out-of-range indices, rows of another expert in the same
 *   block) is left untouched.
 */
fp8_status fp8_grouped_gemm_contiguous(const uint8_t* xq, const float* sa,
                                       const uint8_t* wq, const float* sb,
                                       const int32_t* m_indices, uint16_t* y,
                                       int64_t M, int64_t N, int64_t K,
                                       int32_t E, uint32_t flags, void* stream);

/*
 * Grouped GEMM, masked layout ([DG] "分组 GEMM 的两种布局": decode with counts
 * unknown to the host, only the valid positions are computed; [DG]
 * "统一块调度器与 rasterization": the scheduler skips experts without work and
 * covers only valid rows).
 *   xq u8 (E,max_m,K), sa fp32 [K/128][E*max_m], masked_m int32 (E) on the
 *   device, wq u8 (E,N,K), sb fp32 (E,N/128,K/128), y bf16 bits (E,max_m,N).
 *   N % 128 == 0.  Row m of expert e is written iff m < clamp(masked_m[e], 0,
 *   max_m); every other row of y is left untouched and rows of xq past the
 *   count need not hold finite values.
 */
fp8_status fp8_grouped_gemm_masked(const uint8_t* xq, const float* sa,
                                   const uint8_t* wq, const float* sb,
                                   const int32_t* masked_m, uint16_t* y,
                                   int32_t E, int64_t max_m, int64_t N,
                                   int64_t K, uint32_t flags, void* stream);

/*
 * MXFP8 quantizer, for activations and weights alike ([TC] sections 6.1 and
 * 6.3: the MX formats share one E8M0 scale, a pure power of two, over 32
 * consecutive elements along K; [TC] 5.4 names MXFP8 among the inputs of
 * DeepGEMM's Blackwell path).  The scale of a group is the power of two at or
 * above max(amax, 1e-4) / 448 (the pages give no rule; this is the UE8M0 rule
 * of the 1x128 groups), so no code saturates.  The scale bytes are packed and
 * transposed ([TC] 5.4: DeepGEMM's Blackwell path takes packed UE8M0 scales
 * in a transposed layout): the 4 bytes of the groups of one 128-K block of a
 * row form one dword, and the dwords are laid out [K/128][R].
 *   x  fp32 (R, K)          input, K % 128 == 0
 *   q  u8   (R, K)          output codes, q = E4M3(x / s)
 *   e  u32  [K/128][R]      output scales: byte t of e[kb*R + r] is the scale
 *                           byte b of group 4*kb + t of row r, s = 2^(b - 127)
 */
fp8_status fp8_quant_mx(const float* x, int64_t R, int64_t K, uint8_t* q,
                        uint32_t* e, void* stream);

/*
 * Dense NT GEMM on MXFP8 operands ([TC] 6.1 with scale vector length 32:
 *   Y[m][n] = sum_g 2^(ea(m,g)-127) * 2^(eb(n,g)-127)
 *                   * sum_{k in group g} xq[m][k] * wq[n][k]).
 *   xq u8 (M,K), ea u32 [K/128][M], wq u8 (N,K), eb u32 [K/128][N] (packed as
 *   fp8_quant_mx writes them; ea[kb][m] byte t is the exponent byte of group
 *   4*kb + t), y bf16 bits (M,N); K % 128 == 0.  Every lane of the scaled
 *   matrix instruction holds one 32-group of its row and takes that group's
 *   byte as its scale, so the whole K sum stays in the instruction's FP32
 *   accumulator.  Accuracy: that of the FP8 instruction (the bound stated at
 *   FP8_FLAG_FAST_ACCUM, with each 32-group's scales).  flags must be 0.
 */
fp8_status fp8_gemm_nt_mx(const uint8_t* xq, const uint32_t* ea,
                          const uint8_t* wq, const uint32_t* eb, uint16_t* y,
                          int64_t M, int64_t N, int64_t K, uint32_t flags,
                          void* stream);

/*
 * MXFP4 weight quantizer ([TC] 6.3: MXFP4 = E2M1 elements with one E8M0 scale
 * per 32; [TC] notes on operand majors: two 4-bit values are packed per byte
 * along K).  The scale of a group is the power of two at or above
 * max(amax, 1e-4) / 6, 6 being the largest E2M1 magnitude (a reading, as for
 * MXFP8), so no element saturates; elements round to nearest, ties to even.
 *   x  fp32 (R, K)          input, K % 128 == 0
 *   q  u8   (R, K/2)        output: element k of a row in byte k/2, the even
 *                           one in the low nibble (E2M1: sign bit 3,
 *                           exponent bits 2..1, mantissa bit 0)
 *   e  u32  [K/128][R]      output scales, packed as by fp8_quant_mx
 */
fp8_status fp8_quant_mxfp4(const float* x, int64_t R, int64_t K, uint8_t* q,
                           uint32_t* e, void* stream);

/*
 * Dense NT GEMM with MXFP8 activations and MXFP4 weights (weight-only 4-bit
 * decode: half the weight bytes of MXFP8):
 *   Y[m][n] = sum_g 2^(ea(m,g)-127) * 2^(eb(n,g)-127)
 *                   * sum_{k in group g} xq[m][k] * E2M1(wq, n, k)
 *   xq u8 (M,K), ea u32 [K/128][M] (fp8_quant_mx), wq u8 (N, K/2),
 *   eb u32 [K/128][N] (fp8_quant_mxfp4), y bf16 bits (M,N); K % 128 == 0.
 *   The scaled matrix instruction takes W as an E2M1 operand and each lane's
 *   group scale; the K sum stays in its FP32 accumulator.  Accuracy: that of
 *   the FP8 instruction, as for fp8_gemm_nt_mx.  flags must be 0.
 */
fp8_status fp8_gemm_nt_mx_w4(const uint8_t* xq, const uint32_t* ea,
                             const uint8_t* wq, const uint32_t* eb, uint16_t* y,
                             int64_t M, int64_t N, int64_t K, uint32_t flags,
                             void* stream);

/*
 * The kernel instances a GEMM call would launch, computed on the host from
 * the shape and a compute-unit count (no device needed): the persistent tile
 * schedule of [DG] "统一块调度器与 rasterization" and the tile choice of
 * [DG] "非对齐块大小" (pick the tile whose count fills the machine's waves
 * best).
 *   layout   0 dense (fp8_gemm_nt), 1 contiguous, 2 masked (max_m as M)
 *   flags    FP8_FLAG_* of the call, plus FP8_PLAN_MX (fp8_gemm_nt_mx /
 *            fp8_gemm_nt_mx_w4) or FP8_PLAN_QOUT (fp8_gemm_nt_qout), dense only
 *   workspace_bytes  what an fp8_gemm_nt_ws call would pass
 * Masked plans count every expert's max_m rows (the kernel counts the valid
 * ones on the device), per expert.  A masked launch has one workgroup per
 * possible tile (grid = tiles per expert, times E at the call); every other
 * tile-kernel launch is persistent (grid = min(tiles, CUs)).
 */
#define FP8_PLAN_MX 0x100u
#define FP8_PLAN_QOUT 0x200u
typedef struct {
    int32_t exact;          /* 1: exact partials (FP16 instruction); 0: FP8 instruction */
    int32_t kernel;         /* 0: tile kernel; 1: decode kernel (M <= 32); 2: X-resident decode kernel;
                               3: exact decode kernel (M <= 64, X in chunks); 4: exact decode kernel
                               with X resident (M <= 64, short K ranges) */
    int32_t tile_m, tile_n; /* workgroup tile of the main launch (decode kernels: all M rows x tile_n columns) */
    int32_t waves;          /* waves per workgroup */
    int32_t grid;           /* workgroups of the main launch */
    int64_t tiles;          /* tiles of the main launch (decode kernels: workgroups) */
    int64_t main_rows;      /* rows [0, main_rows) in the main launch (contiguous); else M */
    int32_t tail_tile_m, tail_tile_n; /* tile of a second launch, or 0: contiguous, over rows
                               [main_rows, M); dense, over columns [main_cols, N) */
    int64_t tail_tiles;
    int32_t k_splits;       /* decode kernel: workgroups along K per tile */
    size_t workspace_bytes; /* workspace the split uses */
    int64_t main_cols;      /* columns [0, main_cols) in the main launch (dense); else N */
    int32_t paired;         /* contiguous, 1: three launches share the 128-row blocks, split on
                               the device from m_indices: the main launch takes 256-row tiles
                               over pairs of consecutive blocks of one expert, the middle launch
                               (mid_tile_m x mid_tile_n) and the tail launch the blocks left,
                               each in whole rounds of its tiles where a last partial round
                               would leave over half of the compute units idle; tiles,
                               mid_tiles and tail_tiles are then upper bounds, and main_rows M */
    int32_t mid_tile_m, mid_tile_n;
    int64_t mid_tiles;
} fp8_gemm_plan_t;
fp8_status fp8_gemm_plan(int32_t layout, int64_t M, int64_t N, int64_t K,
                         uint32_t flags, int32_t compute_units,
                         size_t workspace_bytes, fp8_gemm_plan_t* plan);

/* ---------------------------------------------------------------------------
 * Gated feed-forward block: both projections, the activation and the product.
 *   g = X Wg^T,  u = X Wu^T,  h = act(g) * u
 * ------------------------------------------------------------------------- */

/* Activations.  SILU: act(g) = g / (1 + e^-g).  GELU (the tanh form):
 * act(g) = g / (1 + e^-t), t = 2 sqrt(2/pi) (g + 0.044715 g^3). */
#define FP8_ACT_SILU 0
#define FP8_ACT_GELU 1

/*
 * Forward on block-scaled E4M3 operands.
 *   xq u8 (M,K), sa fp32 [K/128][M], wgq and wuq u8 (N,K), sbg and sbu fp32
 *   [ceil(N/128)][K/128] as for fp8_gemm_nt; any M and N, K % 128 == 0.
 *   h bf16 bits (M,N); g and u bf16 bits (M,N), both or neither: the
 *   projections, which the gradient needs.
 * g and u are formed with exact block partials as on fp8_gemm_nt's default
 * path; the activation and the product are FP32, and each output is rounded
 * once.  flags: FP8_FLAG_UE8M0 (the scales are powers of two).
 * workspace: where the output has too few tiles to fill the device, or has
 * few tokens and is quantized, fp8_gated_workspace_size() bytes (0: none is
 * used) hold FP32 sums for a second kernel; without them, or with fewer, one
 * kernel does all, slower.  outputs (of the size query): 0 h, 1 h with g and
 * u, 2 quantized.
 */
fp8_status fp8_gated_nt(const uint8_t* xq, const float* sa, const uint8_t* wgq,
                        const float* sbg, const uint8_t* wuq, const float* sbu,
                        uint16_t* h, uint16_t* g, uint16_t* u, int64_t M,
                        int64_t N, int64_t K, int32_t act, uint32_t flags,
                        void* workspace, size_t workspace_bytes, void* stream);
size_t fp8_gated_workspace_size(int64_t M, int64_t N, int64_t K, int32_t outputs);

/*
 * The kernels a fp8_gated_nt (outputs 0, 1) or fp8_gated_nt_qout (2) call
 * launches, computed on the host from the shape, a compute-unit count and the
 * workspace the call passes (no device needed).
 */
typedef struct {
    int32_t few_tokens;     /* 1: the kernel built around the weights' stream; 0: the tile kernel */
    int32_t tile_m, tile_n; /* rows and output columns of a workgroup (few tokens: M in whole 16s) */
    int32_t k_splits;       /* workgroups along K per tile */
    int32_t joined;         /* 1: a second kernel forms the outputs from FP32 sums */
    int64_t tiles;
    size_t workspace_bytes; /* of FP32 sums */
} fp8_gated_plan_t;
fp8_status fp8_gated_plan(int64_t M, int64_t N, int64_t K, int32_t outputs,
                          int32_t compute_units, size_t workspace_bytes,
                          fp8_gated_plan_t* plan);

/*
 * fp8_gated_nt with h quantized for the next GEMM (the down projection), from
 * the FP32 values, as fp8_gemm_nt_qout does:
 *   hq u8 (M,N) E4M3 codes, sh fp32 [N/128][M] 1x128 scales; N % 128 == 0.
 * The scale follows the group's FP32 maximum.  A power-of-two scale is a step
 * function of it: where max|h| / 448 in unlimited precision lies within the
 * FP32 error of a power of two, the scale is that power or its double, and the
 * codes go with it; either pair stands for h to within an E4M3 rounding.
 */
fp8_status fp8_gated_nt_qout(const uint8_t* xq, const float* sa, const uint8_t* wgq,
                             const float* sbg, const uint8_t* wuq, const float* sbu,
                             uint8_t* hq, float* sh, int64_t M, int64_t N,
                             int64_t K, int32_t act, uint32_t flags,
                             void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradient of the gated block, BF16 operands (the activations and weights
 * before quantization; quantization is taken as the identity):
 *   dg = dh * u * act'(g),  du = dh * act(g)
 *   dX = dg Wg + du Wu,  dWg = dg^T X,  dWu = du^T X
 *   dh, g, u (M,N), x (M,K), wg, wu (N,K), dx (M,K), dwg, dwu (N,K): bf16
 *   bits; any M and N, K % 128 == 0.  dx may be NULL, and dwg and dwu may
 *   both be NULL (not computed).  With M == 0 dwg and dwu are zeros, with
 *   N == 0 dx is.
 * dg and du are formed in FP32 and rounded to BF16, the matrix instruction's
 * type; sums are FP32, and each result is rounded once.  The workspace (dg
 * and du, and FP32 sums and counts where a contraction is split) is required:
 * fp8_gated_grad_workspace_size() bytes, else FP8_ERR_SCRATCH.  It needs no
 * clearing; calls that overlap in time need one each.
 */
fp8_status fp8_gated_nt_grad(const uint16_t* dh, const uint16_t* g, const uint16_t* u,
                             const uint16_t* x, const uint16_t* wg, const uint16_t* wu,
                             uint16_t* dx, uint16_t* dwg, uint16_t* dwu, int64_t M,
                             int64_t N, int64_t K, int32_t act, void* workspace,
                             size_t workspace_bytes, void* stream);
size_t fp8_gated_grad_workspace_size(int64_t M, int64_t N, int64_t K);

/*
 * The products a fp8_gated_nt_grad call launches, computed on the host from
 * the shape, which results are wanted (dx, dw: 0 or 1) and a compute-unit
 * count (no device needed).
 */
typedef struct {
    int32_t dx_tile_n, dw_tile_n;   /* columns of a tile of 128 rows: 128 or 256 */
    int32_t dx_splits, dw_splits;   /* workgroups along the contraction per tile */
    int32_t dw_first;               /* 1: dW's tiles are started first */
    int64_t dx_tiles, dw_tiles;     /* 0 where not wanted */
    size_t workspace_bytes;
} fp8_gated_grad_plan_t;
fp8_status fp8_gated_grad_plan(int64_t M, int64_t N, int64_t K, int32_t dx,
                               int32_t dw, int32_t compute_units,
                               fp8_gated_grad_plan_t* plan);

/* ---------------------------------------------------------------------------
 * Matrix-vector products with 4-bit weights and group scales, for up to 16
 * tokens (M <= 16, else FP8_ERR_SHAPE).
 * ------------------------------------------------------------------------- */

/* Value of `group` for MXFP4 weights (E2M1 with one E8M0 scale per 32). */
#define FP8_W4_MXFP4 0

/*
 * y[m][n] = sum_k x[m][k] w[n][k]
 *   x bf16 bits (M,K), y bf16 bits (M,N); any N, K % 128 == 0.
 *   w u8 (N,K/2): two codes per byte, the even element in the low nibble.
 *   group == FP8_W4_MXFP4: w = E2M1 * 2^(e-127), s = u32 [K/128][N] packed
 *     scale bytes, both as fp8_quant_mxfp4 writes them; z NULL.
 *   group 32, 64 or 128: w = s * (q - z), q = 0..15; s bf16 bits [K/group][N];
 *     z u8 [K/group][N] (values 0..15: the low four bits count), or NULL for 8
 *     everywhere.
 * Every product x (q - z), or x w for MXFP4, is exact; the sums are FP32, y is
 * rounded once, and an infinite or NaN x gives what the definition gives.
 * MXFP4 weights of 2^128 and more (e >= 253) are infinite, and e = 255 is NaN.
 */
fp8_status fp8_gemv_w4(const uint16_t* x, const uint8_t* w, const void* s,
                       const uint8_t* z, uint16_t* y, int64_t M, int64_t N,
                       int64_t K, int32_t group, void* stream);

/* The gated block on such weights: y = act(x Wg^T) * (x Wu^T), one kernel.
 * zg and zu: both or neither. */
fp8_status fp8_gated_gemv_w4(const uint16_t* x, const uint8_t* wg, const void* sg,
                             const uint8_t* zg, const uint8_t* wu, const void* su,
                             const uint8_t* zu, uint16_t* y, int64_t M, int64_t N,
                             int64_t K, int32_t group, int32_t act, void* stream);

/*
 * 4-bit integer weight quantizer, one scale per `group` (32, 64, 128) along K:
 *   z given:  lo = min(w, 0), hi = max(w, 0) over the group, s =
 *             bf16((hi - lo) / 15), z = clamp(round(-lo / s), 0, 15)
 *   z NULL:   s = bf16(max|w| / 7), z = 8
 *   q = clamp(round(w / s) + z, 0, 15);  s is at least bf16(1e-8)
 * Roundings to nearest, ties to even; quotients correctly rounded FP32.
 *   w fp32 (N,K) -> q u8 (N,K/2), s bf16 bits [K/group][N], z u8 [K/group][N]
 */
fp8_status fp8_quant_int4(const float* w, int64_t N, int64_t K, int32_t group,
                          uint8_t* q, uint16_t* s, uint8_t* z, void* stream);

/* ---------------------------------------------------------------------------
 * Global gradient norm over many tensors, and clipping.
 *   norm = sqrt(sum over all tensors and elements of g^2)
 *   out  = g * min(1, max_norm / (norm + 1e-6))
 * ------------------------------------------------------------------------- */
#define FP8_TYPE_F32 0
#define FP8_TYPE_BF16 1
#define FP8_TYPE_F16 2

/*
 * grads, outs, sizes, types: HOST arrays of `count` device pointers, element
 * counts and FP8_TYPE_*, read during the call only.  Tensors need no more
 * alignment than their elements; outs[i] may be grads[i] (in place), and
 * overlaps nothing else.  norm: one FP32 on the device.  Squares are summed
 * in FP64 in a fixed order.  A NaN among the gradients makes the norm and all
 * outputs NaN; an infinity makes the factor 0.  The workspace is required:
 * fp8_clip_workspace_size() bytes, 8-byte aligned, else FP8_ERR_SCRATCH (the
 * size is 0 for bad sizes, and where 120 tensors in turn hold more than 2^43
 * elements, which is FP8_ERR_UNSUPPORTED).
 */
fp8_status fp8_clip_grad_norm(const void* const* grads, void* const* outs,
                              const int64_t* sizes, const int32_t* types,
                              int32_t count, float max_norm, float* norm,
                              void* workspace, size_t workspace_bytes, void* stream);
size_t fp8_clip_workspace_size(const int64_t* sizes, int32_t count);

/* ---------------------------------------------------------------------------
 * Around the experts' products: the router's choice, tokens sorted by expert
 * and back.  Unlike the calls above these take pointers of any alignment that
 * their elements have, except where a call says otherwise.  A call whose launch
 * would have 2^32 threads or more is FP8_ERR_UNSUPPORTED: the router's of more
 * than 2^26 - 4 rows, the combine's gradient of more than 2^24 - 1 tokens and 32s
 * of rows to clear, the moving of rows of more than 2^26 - 4 runs of 4 KB of a
 * token (the combine's of 2 KB) and 8s of rows to clear, the quantizing
 * dispatch's of more than 2^26 - 32 runs of 1024 elements.
 * ------------------------------------------------------------------------- */

/*
 * The k experts of each row with the largest logits, and their weights.
 *   logits  type FP8_TYPE_F32 or FP8_TYPE_BF16 (T,E); 1 <= k <= E <= 1024, k <= 64
 *   ids     int32 (T,k): experts by falling logit, equal logits by rising
 *           index.  An expert whose logit is -infinity is never chosen: where
 *           too few are left, the last ids are -1 and their weights 0.
 *   weights fp32 (T,k): scale * p[id], p = softmax(logits[t]); with
 *           renormalize divided by the chosen p's sum.
 * A NaN ranks above all numbers; a row with a NaN or +infinity among its
 * chosen logits (without renormalize: among all) has NaN weights.
 */
fp8_status fp8_route_topk(const void* logits, int64_t T, int32_t E, int32_t k, int32_t type,
                          int32_t renormalize, float scale, float* weights,
                          int32_t* ids, void* stream);

/*
 * Its gradient, the choice held fixed: dlogits (T,E) in the logits' type from
 * dweights fp32 (T,k), the same logits, ids, k, renormalize and scale:
 *   G = sum_j p_j dw_j over the chosen (p renormalized if the weights were)
 *   dlogits[e] = scale * (sum over j with ids_j = e of p_j dw_j - p_e G),
 * p_e being 0 for experts not chosen with renormalize.  ids outside [0,E) add
 * nothing (their dweights are not read into any sum).
 */
fp8_status fp8_route_topk_grad(const float* dweights, const void* logits, const int32_t* ids,
                               int64_t T, int32_t E, int32_t k, int32_t type,
                               int32_t renormalize, float scale, void* dlogits,
                               void* stream);

/*
 * Rows of the experts' buffers for `pairs` (token, choice) pairs, pair
 * t * k + j being token t's j-th expert: a stable sort by expert.
 *   ids     int32 (id_bytes 4) or int64 (8), (pairs); one outside [0,E) has no
 *           expert.  E <= 1024.
 *   pos     int32 (pairs): the pair's row, or -1; may be NULL
 *   src     int32 (rows): the row's pair, or -1
 * Contiguous layout (fp8_grouped_gemm_contiguous): the experts' segments
 * follow each other, each in whole `align` rows (a power of two up to 1024;
 * 128 for the grouped GEMM, 16 for fp8_add_adapters).
 *   m_indices int32 (rows): the row's expert, -1 on rows without a pair
 *   counts  int32 (E): each expert's pairs; may be NULL
 *   rows    fp8_expert_rows() always suffices; with fewer, pairs whose row
 *           would lie behind have none (pos -1)
 *   keep    nonzero: pairs without an expert get rows too, in a segment behind
 *           the experts' whose m_indices are -1 (then one expert more counts
 *           in fp8_expert_rows)
 * Masked layout (fp8_grouped_gemm_masked): expert e's rows begin at e * max_m;
 * its pairs from the max_m-th on have none.
 *   src     int32 (E*max_m);  masked_m int32 (E): min(pairs, max_m) of each
 * Every output is written whole.  workspace: fp8_expert_sort_workspace_size()
 * bytes, 16-byte aligned, else FP8_ERR_SCRATCH (0 for few pairs); no clearing;
 * calls that overlap in time need one each.
 */
int64_t fp8_expert_rows(int64_t pairs, int32_t E, int32_t align);
size_t fp8_expert_sort_workspace_size(int64_t pairs, int32_t E);
fp8_status fp8_expert_sort_contiguous(const void* ids, int32_t id_bytes, int64_t pairs,
                                      int32_t E, int32_t align, int64_t rows, int32_t keep,
                                      int32_t* pos, int32_t* src, int32_t* m_indices,
                                      int32_t* counts, void* workspace,
                                      size_t workspace_bytes, void* stream);
fp8_status fp8_expert_sort_masked(const void* ids, int32_t id_bytes, int64_t pairs,
                                  int32_t E, int64_t max_m, int32_t* pos, int32_t* src,
                                  int32_t* masked_m, void* workspace,
                                  size_t workspace_bytes, void* stream);

/*
 * Tokens to their experts' rows: xs[pos[t][j]] = x[t].
 *   x (T,K) and xs (rows,K) of one type (FP8_TYPE_F32 or FP8_TYPE_BF16), pos
 *   int32 (T,k), each row named at most once; a place outside [0,rows) is none.
 *   src int32 (rows) or NULL: with it, rows whose src is negative become
 *   zeros; without it they stay as they are.
 * The gradient is fp8_expert_combine of dxs without weights.
 */
fp8_status fp8_expert_dispatch(const void* x, const int32_t* pos, const int32_t* src,
                               void* xs, int64_t T, int32_t k, int64_t rows, int64_t K,
                               int32_t type, void* stream);

/*
 * The same with the rows quantized as fp8_quant_1x128 does (from FP32 values):
 *   xq u8 (rows,K), sa fp32 [K/128][rows]; K % 128 == 0.  Rows without a token
 *   stay as they are (the grouped GEMMs do not use them).  x, xq and sa
 *   16-byte aligned.  flags: FP8_FLAG_UE8M0.
 */
fp8_status fp8_expert_dispatch_quant(const void* x, const int32_t* pos, uint8_t* xq,
                                     float* sa, int64_t T, int32_t k, int64_t rows,
                                     int64_t K, int32_t type, uint32_t flags,
                                     void* stream);

/*
 * Experts' rows back to their tokens: out[t] = sum_j weights[t][j] * y[pos[t][j]]
 * over the pairs that have a row, in FP32 in the order of j, rounded once.
 *   y (rows,N), out (T,N) of one type, weights fp32 (T,k) or NULL (1).
 */
fp8_status fp8_expert_combine(const void* y, const int32_t* pos, const float* weights,
                              void* out, int64_t T, int32_t k, int64_t rows, int64_t N,
                              int32_t type, void* stream);

/*
 * Its gradient: dy[pos[t][j]] = weights[t][j] * dout[t], and dweights[t][j] =
 * <dout[t], y[pos[t][j]]> in FP32 (0 for a pair without a row).  Each row is named
 * at most once, as the sorts do: of a row named twice dy holds one pair's part.
 *   dout (T,N), y and dy (rows,N) of one type; dy or dweights may be NULL (not
 *   computed; y is read for dweights only).  src as for fp8_expert_dispatch.
 */
fp8_status fp8_expert_combine_grad(const void* dout, const void* y, const int32_t* pos,
                                   const float* weights, const int32_t* src, void* dy,
                                   float* dweights, int64_t T, int32_t k, int64_t rows,
                                   int64_t N, int32_t type, void* stream);

/* ---------------------------------------------------------------------------
 * Low-rank adapters of many requests beside one projection:
 *   out[t] = y[t] + scale[a] * (x[t] A_a^T) B_a^T,  a the adapter of token t
 * ------------------------------------------------------------------------- */
/*
 *   x bf16 bits (T,K), a bf16 bits (L,R,K), b bf16 bits (L,N,R), scale fp32 (L),
 *   y and out bf16 bits (T,N), out may be y; any N, K % 128 == 0, R a multiple
 *   of 8 up to 128 (smaller adapters: zeros in the rest of a or b).
 *   src, index int32 (rows): src and m_indices of fp8_expert_sort_contiguous
 *   over the tokens' adapters with align 16.  Rows whose src is outside [0,T)
 *   have no token.  Tokens whose index is outside [0,L) take y as it is, and
 *   tokens in no row are not written: sort with `keep` where out is not y.  A
 *   row whose index differs from that of its tile of 16 (the first of its rows
 *   that has a token) is not computed.  Each token stands in at most one row.
 * The products' sums are FP32, x A^T enters the second one as an FP32 value, and
 * out is rounded once.  Infinities and NaN give what the formula, with scale applied to
 * x A^T, makes of them.  x, a, b and workspace 16-byte aligned; workspace:
 * fp8_adapters_workspace_size() bytes, else FP8_ERR_SCRATCH; no clearing;
 * calls that overlap in time need one each.
 */
fp8_status fp8_add_adapters(const uint16_t* x, const uint16_t* a, const uint16_t* b,
                            const float* scale, const int32_t* src, const int32_t* index,
                            const uint16_t* y, uint16_t* out, int64_t T, int64_t N,
                            int64_t K, int32_t L, int32_t R, int64_t rows,
                            void* workspace, size_t workspace_bytes, void* stream);
size_t fp8_adapters_workspace_size(int64_t T, int32_t L, int64_t rows, int64_t N,
                                   int64_t K, int32_t R);

/* The kernels a fp8_add_adapters call launches (host arithmetic, no device needed). */
typedef struct {
    int64_t tiles;          /* of 16 rows */
    int64_t k_splits;       /* workgroups along K of the first kernel */
    int64_t k_range, n_range;   /* of a workgroup of the first and the second kernel */
    size_t workspace_bytes;
    int32_t group;          /* tiles per workgroup of the two: 1 or 4 */
    int32_t whole;          /* not 0: one kernel instead of the two, with as many workgroups
                             * per tile and no workspace */
} fp8_adapters_plan_t;
fp8_status fp8_adapters_plan(int64_t T, int32_t L, int64_t rows, int64_t N, int64_t K,
                             int32_t R, int32_t compute_units, fp8_adapters_plan_t* plan);

/* M alignment every expert segment of the contiguous layout must have
 * ([DG] "分组 GEMM 的两种布局": the alignment query).  Returns 128. */
int32_t fp8_get_mk_alignment_for_contiguous_layout(void);

/* Static description of a status code (never NULL). */
const char* fp8_status_string(fp8_status status);

#ifdef __cplusplus
}
#endif
#endif
