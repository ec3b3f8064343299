/*
 * w4a8.h -- C ABI of libw4a8.so: W4A8 (LiquidQuant) and W4FP8 (INT4 x FP8)
 * GEMM for AMD Instinct MI355X (gfx950).
 *
 * Sources, cited by page title and part of the page:
 *   [LG] "LiquidGEMM: Hardware-Efficient W4A8 GEMM Kernel for High-
 *        Performance LLM Serving", Pith review of arXiv 2509.01229 --
 *        "What carries the argument" (dequantisation identity, offset a),
 *        referee summary (two-level quantisation: per-channel INT8 then
 *        per-group UINT4; INT8 MMA on dequantised weights), major comment 3
 *        (integer scale s_u8, paper Sec. 4 Eq. 7), minor comment 2 (rounding
 *        to nearest, Eq. 10), circularity audit (Eq. 11/12, range [-119,119]),
 *        parameter ledger (group size 64).
 *   [FQ] "FireQ: Fast INT4-FP8 Kernel and RoPE-aware Quantization for LLM
 *        Inference Acceleration", arXiv 2505.20839, abstract (INT4 weights,
 *        FP8 activations, channel-wise scaling, all linear layers).
 *
 * Conventions for every entry point:
 *   - All array arguments are DEVICE pointers, owned by the caller.  The
 *     library never allocates or frees device memory and keeps no state
 *     besides a per-device cache of the device architecture check and, for
 *     w4a8_gemm_noalloc, one static device array per GPU (below).
 *   - Work is enqueued on `stream` (NULL = the default stream) and the call
 *     returns without synchronising.  Faults inside kernels surface at the
 *     caller's next synchronisation, as usual in HIP.
 *   - Arguments are validated on the host BEFORE any HIP call; on a
 *     validation error nothing is enqueued and no output is touched.
 *   - Matrices are row-major.  Y[M][N] = X[M][K] . W[N][K]^T: W holds one row
 *     per output channel, K contiguous.
 *   - M = 0 or N = 0 is a valid empty problem: once the sizes and modes are
 *     valid the call returns W4A8_OK without checking pointers (nothing is
 *     read or written) and launches nothing.
 *   - Shape constraints: K a positive multiple of 128, N a multiple of 64,
 *     group in {64, 128}.  For every GEMM: M*K < 2^31 and N*K < 2^32 (the
 *     kernels address operands with 32-bit buffer ranges); larger problems
 *     return W4A8_ERR_SHAPE (split M across calls).
 *   - An int32 sum of INT8 products is exact whatever the codes for K up to
 *     W4A8_EXACT_MAX_K (127 * 128 * 131072 < 2^31).  The GEMMs also take
 *     longer rows, whose sums are exact while they lie within int32;
 *     w4a8_moe and w4a8_gemm_lora do not.
 *   - Alignment (W4A8_ERR_ALIGNMENT otherwise): the byte and element
 *     arrays -- W, X, Xq, wq, wq8, s_u8, a_u8, Y and any workspace -- start
 *     on a 16-byte boundary (the kernels move them in 16-byte pieces); the
 *     float32 / int32 vectors -- sx, sw, offsets, fsc, tscale -- on a 4-byte
 *     boundary.
 *
 * Packed 4-bit weight layout (W4A8_LAYOUT_VERSION 1), wq = N*K/2 bytes:
 *   the [N][K] matrix of 4-bit codes is cut into tiles of 16 rows x 128 K.
 *   Tile (nt, kt) = rows 16nt..16nt+15, columns 128kt..128kt+127 occupies
 *   bytes [1024*(nt*(K/128) + kt), +1024).  Inside a tile, "lane"
 *   L = 16*G + r (r = row within the tile, G = 0..3) owns the 16 bytes at
 *   offset 16*L; they cover tile columns 32G .. 32G+31.  Dword d (0..3) of
 *   those 16 bytes covers columns 32G+8d .. 32G+8d+7; its byte b (0..3)
 *   holds column 32G+8d+b in the low nibble and column 32G+8d+4+b in the
 *   high nibble.  One 16-byte load by one lane thus carries 32 weights of one
 *   output channel: two K-steps of the INT8 matrix core, one of the FP8 one.
 * Per-group parameters (LiquidQuant mode), s_u8 and a_u8, N*K/group bytes
 * each, in "panel" order: output channels are taken in panels of 64
 * (p = n/64); the parameters of panel p and group j (columns
 * j*group .. j*group+group-1) are the 64 bytes at offset 64*(p*(K/group) + j),
 * and channel n sits at byte 4*(n%16) + (n%64)/16 of them.  A lane that
 * handles row r of the four 16-row tiles of a panel thus reads the
 * parameters of all four with one 4-byte load.  Scales: sw[N], sx[M] float32.
 */
#ifndef W4A8_H
#define W4A8_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h> /* hipStream_t */

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    W4A8_OK = 0,
    W4A8_ERR_NULL_PTR = 1,    /* a required pointer is NULL                     */
    W4A8_ERR_SHAPE = 2,       /* negative size, K % 128, N % 64, group, qmax     */
    W4A8_ERR_ALIGNMENT = 3,   /* a pointer breaks the alignment rule above       */
    W4A8_ERR_WORKSPACE = 4,   /* workspace smaller than the call's size function */
    W4A8_ERR_UNSUPPORTED = 5, /* device is not gfx950, or a bad mode/flag value  */
    W4A8_ERR_HIP = 6          /* a HIP call failed; see w4a8_last_hip_error()    */
} w4a8_status_t;

#define W4A8_LAYOUT_VERSION 1
#define W4A8_EXACT_MAX_K 131072

enum { W4A8_PACK_LQQ = 0, W4A8_PACK_INT4_SYM = 1 };
enum { W4A8_OUT_F16 = 0, W4A8_OUT_I32 = 1 };
enum { W4FP8_OUT_BF16 = 0, W4FP8_OUT_F32 = 1 };

/*
 * Offline weight quantisation and packing, on the device.
 *
 * mode W4A8_PACK_LQQ ([LG] referee summary, "What carries the argument",
 * major comment 3, minor comment 2, circularity audit):
 *   1. per output channel n: sw[n] = max_k |W[n][k]| / qmax_i8 (float32),
 *      Q = clamp(round_half_even(W / sw[n]), -qmax_i8, qmax_i8) (float32
 *      arithmetic; a row with no positive scale gets sw = 1 and Q = 0);
 *   2. per group j of `group` columns: m = min Q, R = max Q - m,
 *      s_u8 = max(1, ceil(R/15)), a_u8 = 128 + m,
 *      q = min(floor((2(Q - m) + s)/(2s)), floor((127 - m)/s))  -- nearest
 *      with ties upward, saturated so that the decoded INT8 never exceeds
 *      127 (the saturation never acts when qmax_i8 = 119, the pages'
 *      protective range);
 *   3. the decode used by w4a8_gemm is (q*s_u8 + a_u8) XOR 0x80 on a byte.
 *   qmax_i8 in [1, 127]; 127 is the symmetric full range, 119 the pages'.
 * mode W4A8_PACK_INT4_SYM ([FQ] abstract): sw[n] = max|W[n]|/7,
 *   q = clamp(round_half_even(W/sw), -7, 7), stored as sign-magnitude
 *   nibbles (bit 3 = sign, bits 0..2 = |q|).  group, qmax_i8, s_u8, a_u8
 *   are ignored and may be 0 / NULL.
 * W: float32 [N][K].  Outputs: wq [N*K/2] (layout above), s_u8 and a_u8
 * [N*K/group] (panel order above), sw [N].
 */
w4a8_status_t w4a8_pack(const float* W, int N, int K, int group, int qmax_i8,
                        int mode, uint8_t* wq, uint8_t* s_u8, uint8_t* a_u8,
                        float* sw, hipStream_t stream);

/*
 * Per-token symmetric INT8 activation quantisation (the input side of the
 * W4A8 contraction, [LG] referee summary: 8-bit activations):
 *   sx[m] = max_k |X[m][k]| / 127 (float32), Xq = clamp(rne(X/sx), -127, 127).
 * X: float32 [M][K]; Xq: int8 [M][K]; sx: float32 [M].  K % 16 == 0.
 */
w4a8_status_t w4a8_quant_act(const float* X, int M, int K, int8_t* Xq,
                             float* sx, hipStream_t stream);

/*
 * Per-token FP8 activation quantisation ([FQ] abstract: activations in
 * FP8): sx[m] = max|X[m]| / 448 (float32); Xq = OCP e4m3 ("fn": no
 * infinities, largest 448) of the float32 quotient X/sx, nearest with ties
 * to even, saturating at +-448, sign kept for zeros.  K % 16 == 0.
 */
w4a8_status_t w4fp8_quant_act(const float* X, int M, int K, uint8_t* Xq,
                              float* sx, hipStream_t stream);

/* Element types of the activations handed to the _ex quantisers. */
enum { W4A8_IN_F32 = 0, W4A8_IN_F16 = 1, W4A8_IN_BF16 = 2 };

/*
 * The two quantisers above for activations held as float32, IEEE fp16 or
 * bfloat16 (in_type), the forms a model's linear layers receive.  Each
 * element is widened to float32 -- exact for all three types -- and then
 * quantised exactly as w4a8_quant_act / w4fp8_quant_act do.  X: [M][K]
 * elements of in_type, 16-byte aligned; Xq, sx as above; K % 16 == 0.
 * Unknown in_type: W4A8_ERR_UNSUPPORTED.
 */
w4a8_status_t w4a8_quant_act_ex(const void* X, int in_type, int M, int K,
                                int8_t* Xq, float* sx, hipStream_t stream);
w4a8_status_t w4fp8_quant_act_ex(const void* X, int in_type, int M, int K,
                                 uint8_t* Xq, float* sx, hipStream_t stream);

/*
 * Bytes of device workspace w4a8_gemm and w4fp8_gemm need for this problem:
 * when the matrix-core kernel has too few output tiles to fill the GPU it
 * splits K across workgroups, writes partial tiles (splits x M x N x 4
 * bytes: int32 for w4a8_gemm, float32 for w4fp8_gemm) and sums them in split
 * order in a second kernel (deterministic; exact for int32).  w4a8_gemm and
 * w8a8_gemm may instead split K between the wave pairs of a workgroup and
 * need half of it, or none; the size returned covers every entry point.
 * Returns 0 when no split is used and when splitk != 0 (streamed kernel,
 * which reduces on chip).  The size does not depend on the group size
 * (partials are per output element), so the call takes the split factor in
 * its place: an explicit split selects the streamed kernel, which needs no
 * workspace.  The workspace is scratch: its contents on entry are ignored
 * and undefined on return; calls that share a workspace must be ordered on
 * one stream.
 */
size_t w4a8_workspace_size(int M, int N, int K, int splitk);

/*
 * W4A8 GEMM ([LG] referee summary and "What carries the argument"):
 *   acc[m][n] = sum_k X[m][k] * Qhat[n][k]   (exact int32)
 *   Qhat[n][k] = (q[n][k] * s_u8[n][k/group] + a_u8[n][k/group]) XOR 0x80
 *   out_type W4A8_OUT_F16: Y[m][n] = fp16_rne((float(acc) * sx[m]) * sw[n])
 *   out_type W4A8_OUT_I32: Y[m][n] = acc[m][n] (sx, sw may be NULL)
 * X: int8 [M][K] per-token quantised; wq, s_u8, a_u8, sw from w4a8_pack
 * (LQQ mode, same N, K, group); Y: fp16 or int32 [M][N].
 * Kernel choice is a function of the shape: M >= 64 with N % 256 == 0 runs
 * a matrix-core tile kernel (256-row workgroup tiles on 16 x 16 x 64
 * instructions; 128-row tiles on 16 x 16 x 64 at two workgroups per CU when
 * a workgroup covers at most 64 K-steps of a grid under four waves, else
 * on 32 x 32 x 32; with too few tiles to fill the GPU, K is split across
 * workgroups, or between the two wave pairs of 128-channel workgroups);
 * otherwise the streamed-tile kernel runs (one, two or
 * four 16-row blocks of X per workgroup sharing each decoded weight), with
 * `splitk` K-slices per output tile.
 * splitk: 0 = automatic; 1, 2, 4, 8 or 16 (at most K/128) forces the
 * streamed-tile kernel with that split.  The int32 result depends on
 * neither choice.
 */
w4a8_status_t w4a8_gemm(const int8_t* X, const float* sx, const uint8_t* wq,
                        const uint8_t* s_u8, const uint8_t* a_u8,
                        const float* sw, void* Y, int out_type, int M, int N,
                        int K, int group, int splitk, void* workspace,
                        size_t workspace_bytes, hipStream_t stream);

/*
 * The kernel plan w4a8_gemm takes for a shape (a pure function of M, N, K
 * and splitk, computed on the host; group does not enter it), for callers
 * that size launches or check a configuration.  Outputs:
 *   *kernel         0 = streamed-tile kernel, 1 = tile kernel on
 *                   16 x 16 x 64 instructions, 2 = tile kernel on
 *                   32 x 32 x 32 instructions;
 *   *tile_rows      rows of X per workgroup (16, 32 or 64 streamed; 128 or
 *                   256 for the tile kernels);
 *   *tile_channels  output channels per workgroup;
 *   *splits         workgroups sharing one output tile's K range (int32
 *                   partials in the workspace when > 1);
 *   *k_parts        groups of waves of one workgroup splitting its K range
 *                   (streamed: K-splitting waves; tile kernels: 1 or 2).
 * An empty problem (M or N = 0), for which w4a8_gemm launches nothing,
 * reports the streamed kernel's plan.  W4A8_ERR_NULL_PTR if an output
 * pointer is NULL; W4A8_ERR_SHAPE for a shape or splitk that w4a8_gemm
 * rejects.
 */
w4a8_status_t w4a8_gemm_plan(int M, int N, int K, int splitk, int* kernel,
                             int* tile_rows, int* tile_channels, int* splits,
                             int* k_parts);

/*
 * w4a8_gemm for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * Arguments, results and errors are those of w4a8_gemm (same kernels, same
 * bits), without the workspace: the split-K partials go to a static device
 * array of this library, W4A8_NOALLOC_SCRATCH_BYTES long, one per GPU,
 * held until the process ends.  Every problem size w4a8_gemm accepts needs
 * at most 32 MiB of partials (at most 256 workgroups of 128 x 256 int32
 * each); a problem whose w4a8_workspace_size(M, N, K, splitk) exceeded the
 * array would return W4A8_ERR_WORKSPACE.  No call allocates or frees
 * memory.  All calls on one GPU share its array: calls that may overlap in
 * time on one GPU (different streams, no ordering between them) race and
 * must not be issued.  Calls ordered on one stream are safe, and so are
 * calls on different GPUs.
 */
#define W4A8_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
w4a8_status_t w4a8_gemm_noalloc(const int8_t* X, const float* sx,
                                const uint8_t* wq, const uint8_t* s_u8,
                                const uint8_t* a_u8, const float* sw, void* Y,
                                int out_type, int M, int N, int K, int group,
                                int splitk, hipStream_t stream);

/*
 * Grouped W4A8 GEMM for mixture-of-experts layers (the pages evaluate
 * Mixtral-8x7B; [LG] review, "What would settle it"): E experts, each a
 * w4a8_gemm of its own rows against its own packed weights, in one launch.
 *   X, Y: [M][K] int8 / [M][N] fp16 or int32, rows grouped by expert:
 *     rows offsets[e] .. offsets[e+1]-1 belong to expert e.
 *   offsets: device int32 [E+1], non-decreasing, offsets[0] = 0,
 *     offsets[E] <= M (read on the device; values are clamped to [0, M], so
 *     inconsistent offsets leave rows unwritten but never access outside X,
 *     Y or sx).
 *   wq, s_u8, a_u8, sw: the E experts' w4a8_pack outputs (same N, K, group)
 *     laid end to end: expert e at wq + e*N*K/2, s_u8/a_u8 + e*N*K/group,
 *     sw + e*N.
 *   max_rows: host-side bound on any expert's row count (sizes the grid;
 *     rows beyond it are not computed).
 * Results per expert are exactly those of w4a8_gemm on that expert's rows.
 * Kernel: streamed tiles when max_rows < 64, else matrix-core tiles (N % 256
 * == 0); no K split, no workspace.  M * K < 2^31.
 */
w4a8_status_t w4a8_gemm_grouped(const int8_t* X, const float* sx,
                                const int32_t* offsets, int E,
                                const uint8_t* wq, const uint8_t* s_u8,
                                const uint8_t* a_u8, const float* sw, void* Y,
                                int out_type, int M, int N, int K, int group,
                                int max_rows, hipStream_t stream);

/*
 * Ablation variants of w4a8_gemm's matrix-core kernel, for measuring what
 * the method's two ideas buy on this hardware ([LG] referee summary: the
 * ablation separating LiquidQuant from the pipeline; "What carries the
 * argument").  All three run on the 32 x 32 x 32 tile kernel (the one
 * w4a8_gemm uses for long-K 128-row tiles; its other plans use a
 * 16 x 16 x 64 kernel with the same decode), so they differ only in the
 * decode:
 *   W4A8_ABL_LQQ          LiquidQuant decode interleaved with the matrix
 *                         cores (the method);
 *   W4A8_ABL_AFFINE16     same stored codes and parameters, decoded as the
 *                         conventional signed value s*q + min (min =
 *                         a_u8 - 128) one code per 16-bit lane, the
 *                         overflow-safe form without the UINT8 shift;
 *   W4A8_ABL_LQQ_COARSE   LiquidQuant decode, but each K-step's weights are
 *                         decoded in one block after that step's matrix-core
 *                         instructions instead of interleaved with them.
 * All three return the same results bit for bit (the decode identity).
 * Arguments as w4a8_gemm without splitk / workspace; only shapes that the
 * unsplit matrix-core kernel serves (M >= 64, N % 256 == 0, no K split in
 * w4a8_workspace_size) are accepted, others return W4A8_ERR_UNSUPPORTED.
 */
enum { W4A8_ABL_LQQ = 0, W4A8_ABL_AFFINE16 = 1, W4A8_ABL_LQQ_COARSE = 2 };
w4a8_status_t w4a8_gemm_ablation(int variant, const int8_t* X, const float* sx,
                                 const uint8_t* wq, const uint8_t* s_u8,
                                 const uint8_t* a_u8, const float* sw, void* Y,
                                 int out_type, int M, int N, int K, int group,
                                 hipStream_t stream);

/*
 * W4FP8 GEMM ([FQ] abstract: INT4 weights x FP8 activations):
 *   acc[m][n] = sum_k e4m3(X[m][k]) * q[n][k]  (float32 accumulation; q is
 *   converted exactly to e4m3, |q| <= 7)
 *   out_type W4FP8_OUT_BF16: Y = bf16_rne((acc * sx[m]) * sw[n])
 *   out_type W4FP8_OUT_F32:  Y = (acc * sx[m]) * sw[n] as float32
 * X: e4m3 bytes [M][K]; wq, sw from w4a8_pack in INT4_SYM mode.
 * Kernel choice as for w4a8_gemm (matrix-core tiles for M >= 64 with
 * N % 256 == 0, else streamed tiles; splitk != 0 forces the streamed kernel);
 * workspace: at least w4a8_workspace_size(M, N, K, splitk) bytes, 16-byte
 * aligned, NULL allowed when that is 0.  The float32 sum order depends on
 * the kernel choice (results within the FP8 path's error bound either way).
 */
w4a8_status_t w4fp8_gemm(const uint8_t* X_e4m3, const float* sx,
                         const uint8_t* wq, const float* sw, void* Y,
                         int out_type, int M, int N, int K, int splitk,
                         void* workspace, size_t workspace_bytes,
                         hipStream_t stream);

/*
 * Packing for the folded per-group FP8 format ([FQ] abstract: a per-tensor
 * scale keeps the FP8 weights from underflowing once the INT4 scaling
 * factors are folded into them; the formulas are this library's reading):
 *   t         = max|W| / 448                      (1 for an all-zero W)
 *   s_g[n][j] = max_{k in group j} |W[n][k]| / 7  (1 for an all-zero group)
 *   f[n][j]   = s_g[n][j] / t                     (float32 divisions, RNE)
 *   q[n][k]   = clamp(rne(W[n][k] / s_g[n][k/group]), -7, 7)
 * W: float32 [N][K]; wq: N*K/2 bytes, sign-magnitude codes in the packed
 * layout above (as INT4_SYM mode); fsc: float32 [K/group][N], fsc[j][n] =
 * f[n][j] (group-major, so one K-step's factors of adjacent channels are
 * adjacent); tscale: one float32, t.  Four kernels on `stream`; fsc is
 * scratch between them.  N * (K/group) < 2^29.
 */
w4a8_status_t w4fp8g_pack(const float* W, int N, int K, int group, uint8_t* wq,
                          float* fsc, float* tscale, hipStream_t stream);

/*
 * GEMM on the folded per-group FP8 weights of w4fp8g_pack:
 *   w8[n][k]  = sign(q) * e4m3_rne(float32(|q[n][k]| * f[n][k/group]))
 *   acc[m][n] = sum_k e4m3(X[m][k]) * w8[n][k]   (float32 accumulation)
 *   out_type W4FP8_OUT_BF16: Y = bf16_rne((acc * sx[m]) * t)
 *   out_type W4FP8_OUT_F32:  Y = (acc * sx[m]) * t as float32
 * w8 is formed in registers per (channel, group) from a table of the eight
 * magnitudes; it is never stored.  X, sx: w4fp8_quant_act outputs; fsc,
 * tscale, wq from w4fp8g_pack with the same N, K, group.  Kernel choice,
 * splitk and workspace as for w4fp8_gemm.
 */
w4a8_status_t w4fp8g_gemm(const uint8_t* X_e4m3, const float* sx,
                          const uint8_t* wq, const float* fsc,
                          const float* tscale, void* Y, int out_type, int M,
                          int N, int K, int group, int splitk, void* workspace,
                          size_t workspace_bytes, hipStream_t stream);

/*
 * W8A8 comparison path ([LG] "If this is right": W4A8's lower memory
 * traffic should beat W8A8 in small-batch, memory-bound runs and match or
 * beat it in large-batch, compute-bound ones).  The weights are the first
 * LiquidQuant level alone: per output channel, sw[n] = max|W[n]|/127 and
 * Q[n][k] = clamp(rne(W[n][k]/sw[n]), -127, 127) (float32, as w4a8_pack's
 * first level), stored as int8 in the 8-bit tile layout:
 *   tile (nt, kt) of 16 rows x 128 K occupies bytes [2048*(nt*(K/128)+kt),
 *   +2048); inside it, byte 1024*u + 16*(16*G + r) + j holds row 16nt + r,
 *   column 128kt + 32G + 16u + j (G 0..3, u 0..1, j 0..15).
 * w8a8_pack: W float32 [N][K] -> wq8 (N*K bytes), sw (N floats).
 * w8a8_gemm: acc[m][n] = sum_k X[m][k] * Q[n][k] (exact int32), then the
 *   w4a8_gemm epilogue (out_type W4A8_OUT_F16 or W4A8_OUT_I32).  The same
 *   kernels as w4a8_gemm with the decode step removed; kernel choice,
 *   splitk and workspace as for w4a8_gemm.  N * K < 2^31.
 */
w4a8_status_t w8a8_pack(const float* W, int N, int K, int8_t* wq8, float* sw,
                        hipStream_t stream);
w4a8_status_t w8a8_gemm(const int8_t* X, const float* sx, const int8_t* wq8,
                        const float* sw, void* Y, int out_type, int M, int N,
                        int K, int splitk, void* workspace,
                        size_t workspace_bytes, hipStream_t stream);

/*
 * Layers whose rows choose their own weights: a router picks the experts of
 * every token (w4a8_route), a few tokens pass through a whole
 * mixture-of-experts layer (w4a8_moe), and the rows of a shared projection
 * each add the low-rank adapter of their request (w4a8_gemm_lora).  The
 * conventions above hold; outputs and workspace overlap no other argument,
 * and calls that share a workspace must be ordered on one stream.  A call
 * whose arguments are device arrays of choices (ids, adapter) reads them on
 * the device, so a captured graph follows their contents.
 */
#define W4A8_MAX_EXPERTS 512
#define W4A8_MAX_TOPK 16
#define W4A8_MOE_MAX_TOKENS 256
#define W4A8_LORA_MAX_RANK 128

/*
 * Top-k gating of router logits and the grouping of the chosen slots.
 *   logits: [T][E] elements of in_type (W4A8_IN_*), aligned to an element,
 *     widened to float32 (exact).  An expert whose logit is -inf or NaN is not
 *     available to that token.
 *   ids[t][j]     int32 [T][k]: the expert with the j-th largest logit (ties
 *     go to the lowest index), -1 where fewer than j+1 are available;
 *   weights[t][j] float32 [T][k]: e_j / sum of e over the token's available
 *     experts (renormalize 0) or over its chosen ones (renormalize 1), with
 *     e_i = exp(x_i - max x), 1 where x_i equals the maximum (so +inf logits
 *     share the weight); 0 where ids is -1;
 *   offsets       int32 [E+1]: experts' ranges of `rows`, as
 *     w4a8_gemm_grouped takes them; offsets[E] = slots with an expert;
 *   rows          int32 [T*k]: the slots t*k + j in order of expert, then
 *     slot (row p of a grouped problem is token rows[p] / k); -1 from
 *     offsets[E] on.
 * 1 <= E <= W4A8_MAX_EXPERTS, 1 <= k <= min(E, W4A8_MAX_TOPK), T * E < 2^31.
 * T = 0 writes offsets (zeros) only; the other pointers may be NULL then.
 * ids, weights, offsets, rows: 4-byte aligned.  workspace: at least
 * w4a8_route_workspace_size bytes (0 for a few tokens: NULL allowed),
 * 16-byte aligned.  No atomics order anything: results are reproducible.
 */
size_t w4a8_route_workspace_size(int T, int E, int k);
w4a8_status_t w4a8_route(const void* logits, int in_type, int T, int E, int k,
                         int renormalize, int32_t* ids, float* weights,
                         int32_t* offsets, int32_t* rows, void* workspace,
                         size_t workspace_bytes, hipStream_t stream);

/*
 * A whole mixture-of-experts layer for at most W4A8_MOE_MAX_TOKENS tokens
 * (longer batches: w4a8_gemm_grouped on w4a8_route's grouping).
 *   X: [T][H] elements of in_type; ids int32 [T][k], weights float32 [T][k]
 *     (w4a8_route's, or any: an id outside [0, E) is no expert, a token may
 *     name an expert twice);
 *   wq13, s13, a13, sw13: the experts' w4a8_pack outputs (LQQ) of
 *     W13[e] = float32 [2F][H], gate rows 0..F-1, up rows F..2F-1, laid end
 *     to end as for w4a8_gemm_grouped; wq2, s2, a2, sw2: those of
 *     W2[e] = [H][F]; one group size for both.
 * Per slot (t, j) with expert e, all in float32 unless said:
 *   Xq, sx = INT8 of token t as w4a8_quant_act;
 *   g, u = ((exact int32 product) * sx) * sw13[e], h = g / (1 + exp(-g)) * u;
 *   hq, sh = INT8 of h as w4a8_quant_act; y = ((int32 product) * sh) * sw2[e];
 *   Y[t] = sum over j (ascending) of weights[t][j] * y, rounded once to
 *   out_type (W4A8_IN_*).  A slot of weight 0 adds nothing, a token without
 *   an expert gives zeros.  A token with an element that is not finite, or
 *   whose h overflows float32, gives NaN (other tokens are unaffected).
 * H % 128 = 0, F % 128 = 0, both <= W4A8_EXACT_MAX_K, 2 F H < 2^32; 1 <= E <=
 * W4A8_MAX_EXPERTS, 1 <= k <= W4A8_MAX_TOPK.  X, Y and the byte arrays
 * 16-byte aligned, the others 4-byte.  workspace: w4a8_moe_workspace_size
 * bytes, 16-byte aligned, contents ignored and undefined afterwards.
 */
size_t w4a8_moe_workspace_size(int T, int E, int k, int H, int F);
w4a8_status_t w4a8_moe(const void* X, int in_type, const int32_t* ids,
                       const float* weights, int T, int E, int k,
                       const uint8_t* wq13, const uint8_t* s13,
                       const uint8_t* a13, const float* sw13,
                       const uint8_t* wq2, const uint8_t* s2,
                       const uint8_t* a2, const float* sw2, void* Y,
                       int out_type, int H, int F, int group, void* workspace,
                       size_t workspace_bytes, hipStream_t stream);

/*
 * A shared W4A8 projection with the low-rank adapter each row selects:
 *   Y[m] = fp16_rne( (acc[m] * sx[m]) * sw
 *                    + scale[a] * (X[m] . A[a]^T) . B[a]^T ),  a = adapter[m]
 * acc as w4a8_gemm on the INT8 rows (Xq, sx) that w4a8_quant_act_ex gives
 * for X; the adapter's products are float32 sums over the stored values, the
 * inner one held in float32 (the outer one meets it as it is for bfloat16,
 * for fp16 within 2^-23, one unit in its last place, or 2^-50 of the largest
 * of 32 ranks), and Y is rounded once.
 *   X: [M][K], A: [n_adapters][R][K], B: [n_adapters][N][R], all fp16 or all
 *     bfloat16 (in_type); scale: float32 [n_adapters]; adapter: int32 [M],
 *     values outside [0, n_adapters) select none, in any order.  Adapters of
 *     smaller rank are padded with zero rows of A (or columns of B).
 *   wq, s_u8, a_u8, sw: w4a8_pack (LQQ) of the shared weights.
 * R a multiple of 8, 8 <= R <= W4A8_LORA_MAX_RANK; n_adapters = 0 is
 * w4a8_gemm (A, B, scale unread).  Sizes as w4a8_gemm, K at most
 * W4A8_EXACT_MAX_K.  X, A, B, Y and the byte arrays 16-byte aligned, the
 * others 4-byte.  workspace: w4a8_gemm_lora_workspace_size bytes, 16-byte
 * aligned.
 */
size_t w4a8_gemm_lora_workspace_size(int M, int N, int K, int R);
w4a8_status_t w4a8_gemm_lora(const void* X, int in_type, const uint8_t* wq,
                             const uint8_t* s_u8, const uint8_t* a_u8,
                             const float* sw, const void* A, const void* B,
                             const float* scale, int n_adapters, int R,
                             const int32_t* adapter, void* Y, int M, int N,
                             int K, int group, void* workspace,
                             size_t workspace_bytes, hipStream_t stream);

/* Static English text for a status code (never NULL). */
const char* w4a8_status_str(w4a8_status_t status);

/* hipError_t of this thread's last W4A8_ERR_HIP, 0 if none. */
int w4a8_last_hip_error(void);

/* W4A8_LAYOUT_VERSION of the compiled library. */
int w4a8_layout_version(void);

#ifdef __cplusplus
}
#endif

#endif /* W4A8_H */
