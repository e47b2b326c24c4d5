/*
 * gfg.h — grouped FP8 (E4M3) block-scaled GEMM for MI355X (gfx950).
 *
 * C ABI of libgfg.so.  The operations are those of the first reference page,
 * "Grouped and Batched GEMM kernels with blockscaling matching DeepGEMM API"
 * (sections "Summary" and "DeepGEMM conformance details"):
 *
 *   D[rows of expert g] = A[rows] . B[g]^T          (contiguous layout)
 *   D[g, m, :]          = A[g, m, :] . B[g]^T       (masked layout, m < masked_m[g])
 *
 * with FP8 E4M3FN operands, one E8M0 scale per (1,128) block of A (per token,
 * per 128 channels, stored transposed as [ceil(K/128), M]) and one per
 * (128,128) block of B.  An E8M0 byte b means the scale 2^(b-127); b = 255
 * is NaN.  The product is exactly the product of the dequantized operands up
 * to fp32 summation order; D is rounded once to bf16 or f16 (nearest even).
 *
 * Conventions for every entry point:
 *  - Tensors are dense, row-major, contiguous, with the last named axis
 *    fastest.  "K-contiguous" ("nt"): A rows and B rows both run along K.
 *  - GEMM tensor pointers are DEVICE pointers owned by the caller.  The
 *    library never allocates, frees or synchronizes inside a GEMM call; the
 *    call is asynchronous on `stream` (a hipStream_t, NULL = null stream).
 *    It runs on the calling thread's current device, to which the pointers and
 *    the stream must belong.  (The torch-facing calls make the tensors' device
 *    current and refuse a stream of another one.)
 *  - Quantizer pointers are HOST pointers owned by the caller; the quantizers
 *    are synchronous CPU functions.
 *  - Return value: GFG_OK (0) or an error code; no exceptions cross the ABI.
 *    grouped_fp8_last_error() returns a thread-local message for the last failure on
 *    the calling thread (valid until that thread's next call).
 *  - Argument checks (null pointers, sizes, enum values) happen on the host
 *    before anything is launched.  Device-resident metadata cannot be
 *    checked without a sync, so the kernels treat a grouped_layout entry
 *    outside [0, G) as padding and clamp masked_m[g] into [0, M_max].
 */
#ifndef GFG_H
#define GFG_H

#include <stdint.h>

#if defined(__GNUC__)
#define GFG_API __attribute__((visibility("default")))
#else
#define GFG_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

enum gfg_status {
    GFG_OK = 0,
    GFG_EINVAL = 1,       /* bad pointer, size or enum value                      */
    GFG_EUNSUPPORTED = 2, /* valid for the method, outside what the kernels tile  */
    GFG_EHIP = 3,         /* a HIP runtime call or kernel launch failed           */
    GFG_ERANGE = 4        /* quantizer: a block scale falls outside E8M0's range  */
};

enum gfg_out_dtype { GFG_OUT_BF16 = 0, GFG_OUT_F16 = 1, GFG_OUT_F32 = 2 /* where a call says so */ };
enum gfg_in_dtype { GFG_IN_F32 = 0, GFG_IN_BF16 = 1, GFG_IN_F16 = 2 };

/*
 * Contiguous grouped GEMM (the DeepGEMM-style m_grouped ... contiguous op).
 *
 *   a              [M][K]               e4m3 bytes
 *   a_scale        [ceil(K/128)][M]     E8M0 bytes, per token per 128-K block (transposed)
 *   b              [G][N][K]            e4m3 bytes
 *   b_scale        [G][ceil(N/128)][ceil(K/128)]  E8M0 bytes, K-block fastest
 *   grouped_layout [M]                  int32 expert id per row, -1 = padding
 *   d              [M][N]               bf16 or f16, written for rows whose
 *                                       grouped_layout is in [0, G); padding rows
 *                                       are left untouched
 *
 * Layout precondition: each expert's rows form runs that start on a multiple
 * of 128, padded with -1 up to the next multiple of 128, so every aligned
 * 128-row tile belongs to one expert (the expert of its first row; a tile
 * whose first row is padding is skipped).  A row whose entry differs from its
 * tile's expert is left untouched.
 *
 * Sizes: M >= 0 (M = 0 is a no-op), N > 0 and K > 0 multiples of 128 with
 * N <= 2^30 and K <= 2^23 (else GFG_EUNSUPPORTED), 1 <= G <= 65535, ceil(M/128) <= 4096 (else
 * GFG_EUNSUPPORTED).  The kernels address one expert's B and the A-scale
 * tensor with 32-bit byte offsets: N*K (bytes of one expert's B) and the
 * scale tensor's bytes (here ceil(K/128)*M; for the MX GEMMs below, one
 * byte per 32 K elements of every row) must stay below 2^32, else
 * GFG_EUNSUPPORTED.  These bounds hold for every entry point below.
 */
GFG_API int grouped_fp8_gemm_contiguous(const void* a, const uint8_t* a_scale,
                                const void* b, const uint8_t* b_scale,
                                const int32_t* grouped_layout, void* d,
                                int64_t M, int64_t N, int64_t K, int32_t G,
                                int32_t out_dtype, void* stream);

/*
 * Masked grouped GEMM (the DeepGEMM-style m_grouped ... masked op).
 *
 *   a         [G][M_max][K]               e4m3 bytes
 *   a_scale   [G][ceil(K/128)][M_max]     E8M0 bytes (the transposed layout, per group)
 *   b         [G][N][K]                   e4m3 bytes
 *   b_scale   [G][ceil(N/128)][ceil(K/128)]
 *   masked_m  [G]                         int32, DEVICE memory: rows computed per group
 *   d         [G][M_max][N]               rows m < masked_m[g] written, others untouched
 *
 * Sizes: M_max >= 0, N and K positive multiples of 128 (N <= 2^30, K <= 2^23),
 * 1 <= G <= 65535,
 * G * ceil(M_max/128) <= 4096 (else GFG_EUNSUPPORTED).
 */
GFG_API int grouped_fp8_gemm_masked(const void* a, const uint8_t* a_scale,
                            const void* b, const uint8_t* b_scale,
                            const int32_t* masked_m, void* d,
                            int32_t G, int64_t M_max, int64_t N, int64_t K,
                            int32_t out_dtype, void* stream);

/*
 * gemm1 of the expert MLP with its silu_mul epilogue (third reference page,
 * the pull request "flydsl mxfp4 a4w4 MoE: bring gemm1/gemm2 to parity with
 * the HIP backend", section "Changes", item gemm1), on the FP8 block-scaled
 * operands above.  Each expert's B holds 2*I rows: rows [0, I) are the gate
 * projection, rows [I, 2*I) the up projection.  For every computed row m:
 *
 *   h = A[m] . B[g]^T  (length 2*I, fp32),   out[m, j] = silu(h[j]) * h[I + j]
 *
 * with silu(x) = x / (1 + e^-x), e^-x taken by the hardware base-2
 * exponential and the division by the hardware reciprocal, then one rounding
 * to bf16 or f16.  Rows are chosen exactly as in the GEMMs above.
 *
 *   b        [G][2*I][K]                     e4m3 bytes (gate rows, then up rows)
 *   b_scale  [G][2*I/128][ceil(K/128)]       E8M0 bytes
 *   d        contiguous [M][I], masked [G][M_max][I]   bf16 or f16
 *   (a, a_scale, grouped_layout, masked_m as in the GEMMs)
 *
 * Sizes: as the GEMM with N = 2*I, and I a positive multiple of 128
 * (else GFG_EUNSUPPORTED; I <= 0 is GFG_EINVAL).  These entry points also
 * need M (M_max) a multiple of 4 and a_scale 4-byte aligned
 * (else GFG_EUNSUPPORTED).
 */
GFG_API int grouped_fp8_gemm_silu_mul_contiguous(const void* a, const uint8_t* a_scale,
                                         const void* b, const uint8_t* b_scale,
                                         const int32_t* grouped_layout, void* d,
                                         int64_t M, int64_t I, int64_t K, int32_t G,
                                         int32_t out_dtype, void* stream);
GFG_API int grouped_fp8_gemm_silu_mul_masked(const void* a, const uint8_t* a_scale,
                                     const void* b, const uint8_t* b_scale,
                                     const int32_t* masked_m, void* d,
                                     int32_t G, int64_t M_max, int64_t I, int64_t K,
                                     int32_t out_dtype, void* stream);

/*
 * MXFP8 grouped GEMM: the same two layouts on MX operands (third reference
 * page, "flydsl mxfp4 a4w4 MoE: bring gemm1/gemm2 to parity with the HIP
 * backend", section "Notes": MX kernels with E8M0 scales; here with E4M3
 * elements).  Every row of A and of B carries one E8M0 scale per 32
 * consecutive K elements; the hardware applies each one to its 32 products
 * inside the scaled MFMA.
 *
 *   a, b, grouped_layout / masked_m, d   as in the GEMMs above
 *   a_scale   contiguous [K/32][M], masked [G][K/32][M_max]   (transposed, per 32-wide K block)
 *   b_scale   [G][K/32][N]
 *
 * Sizes: as the GEMMs above, and N a multiple of 256, M (M_max) a multiple
 * of 4, a_scale and b_scale 4-byte aligned (else GFG_EUNSUPPORTED).
 */
GFG_API int grouped_mxfp8_gemm_contiguous(const void* a, const uint8_t* a_scale,
                                  const void* b, const uint8_t* b_scale,
                                  const int32_t* grouped_layout, void* d,
                                  int64_t M, int64_t N, int64_t K, int32_t G,
                                  int32_t out_dtype, void* stream);
GFG_API int grouped_mxfp8_gemm_masked(const void* a, const uint8_t* a_scale,
                              const void* b, const uint8_t* b_scale,
                              const int32_t* masked_m, void* d,
                              int32_t G, int64_t M_max, int64_t N, int64_t K,
                              int32_t out_dtype, void* stream);

/*
 * MX quantizer (CPU, synchronous) for the MXFP8 GEMM's operands:
 *   x [G][R][K] float -> q [G][R][K] e4m3, scale_t [G][K/32][R] E8M0
 * (A: G = 1, R = M; masked A: G groups of R = M_max; B: G experts of R = N).
 * Per row and 32-wide K block, the "Even" scale rounding of the third
 * reference page ("flydsl mxfp4 a4w4 MoE: bring gemm1/gemm2 to parity with
 * the HIP backend", section "Notes"): amax = max|x| is rounded to 3 fraction
 * bits (nearest, ties to even), t = floor(log2(rounded amax)) - 8 (t = 0 for
 * an all-zero block), scale byte t + 127, q = E4M3(clamp(x / 2^t, -448, 448))
 * nearest-even.  K must be a multiple of 32 (else GFG_EUNSUPPORTED);
 * GFG_ERANGE if t falls outside [-127, 127] or a value is not finite.
 */
GFG_API int fp8_quantize_mx_1x32(const float* x, int32_t G, int64_t R, int64_t K,
                         uint8_t* q, uint8_t* scale_t);

/*
 * MXFP4 grouped GEMM: the two layouts on E2M1 operands (the "mxfp4 (a4w4)"
 * element type of the third reference page, "flydsl mxfp4 a4w4 MoE: bring
 * gemm1/gemm2 to parity with the HIP backend", section "Summary"), one E8M0
 * scale per 32 K elements of every row, as in the MXFP8 GEMM.  K counts E2M1
 * elements; each row of a and b is K/2 bytes, two elements per byte with
 * the lower K index in the low nibble (as fp4_quantize_mx_1x32 writes).
 *
 *   a         contiguous [M][K/2], masked [G][M_max][K/2]      E2M1, two per byte
 *   b         [G][N][K/2]
 *   a_scale   contiguous [K/32][M], masked [G][K/32][M_max]
 *   b_scale   [G][K/32][N]
 *
 * Sizes: as the MXFP8 GEMM, with K a multiple of 256 (else GFG_EUNSUPPORTED).
 */
GFG_API int grouped_mxfp4_gemm_contiguous(const void* a, const uint8_t* a_scale,
                                  const void* b, const uint8_t* b_scale,
                                  const int32_t* grouped_layout, void* d,
                                  int64_t M, int64_t N, int64_t K, int32_t G,
                                  int32_t out_dtype, void* stream);
GFG_API int grouped_mxfp4_gemm_masked(const void* a, const uint8_t* a_scale,
                              const void* b, const uint8_t* b_scale,
                              const int32_t* masked_m, void* d,
                              int32_t G, int64_t M_max, int64_t N, int64_t K,
                              int32_t out_dtype, void* stream);

/*
 * a4w4 gemm1 with silu_mul: the gemm1 of the third reference page as the
 * page runs it ("mxfp4 (a4w4)" operands, section "Summary"; the silu_mul
 * epilogue, section "Changes", item gemm1).  The operands are those of the
 * MXFP4 GEMM above; the epilogue is that of grouped_fp8_gemm_silu_mul_*:
 * each expert's B holds 2*I rows, gate rows [0, I) then up rows [I, 2*I),
 * and for every computed row m
 *
 *   h = A[m] . B[g]^T  (length 2*I, fp32),   out[m, j] = silu(h[j]) * h[I + j]
 *
 *   a         contiguous [M][K/2], masked [G][M_max][K/2]      E2M1, two per byte
 *   b         [G][2*I][K/2]                                    (gate rows, then up rows)
 *   a_scale   contiguous [K/32][M], masked [G][K/32][M_max]    E8M0 bytes
 *   b_scale   [G][K/32][2*I]
 *   d         contiguous [M][I], masked [G][M_max][I]          bf16 or f16
 *   (grouped_layout, masked_m, out_dtype, stream as in the GEMMs)
 *
 * Sizes: K (E2M1 elements) a multiple of 256, I a positive multiple of 128,
 * M (M_max) a multiple of 4, both scale tensors 4-byte aligned (else
 * GFG_EUNSUPPORTED; I <= 0 or K <= 0 is GFG_EINVAL).  Rows are chosen as in
 * the GEMMs; other rows of d are left untouched.
 */
GFG_API int grouped_mxfp4_gemm_silu_mul_contiguous(const void* a, const uint8_t* a_scale,
                                           const void* b, const uint8_t* b_scale,
                                           const int32_t* grouped_layout, void* d,
                                           int64_t M, int64_t I, int64_t K, int32_t G,
                                           int32_t out_dtype, void* stream);
GFG_API int grouped_mxfp4_gemm_silu_mul_masked(const void* a, const uint8_t* a_scale,
                                       const void* b, const uint8_t* b_scale,
                                       const int32_t* masked_m, void* d,
                                       int32_t G, int64_t M_max, int64_t I, int64_t K,
                                       int32_t out_dtype, void* stream);

/*
 * MXFP4 quantizer (CPU, synchronous):
 *   x [G][R][K] float -> q [G][R][K/2] (two E2M1 codes per byte), scale_t [G][K/32][R] E8M0.
 * Per row and 32-wide K block, the "Even" scale rounding at E2M1's precision:
 * amax = max|x| rounded to 1 fraction bit (nearest, ties to even),
 * t = floor(log2(rounded amax)) - 2 (t = 0 for an all-zero block), scale
 * byte t + 127, code = E2M1(clamp(x / 2^t, -6, 6))
 * nearest-even (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6; bit 3 the sign).
 * Byte i of a row holds elements 2i (low nibble) and 2i + 1.  K must be a
 * multiple of 128 (else GFG_EUNSUPPORTED); GFG_ERANGE as fp8_quantize_mx_1x32.
 */
GFG_API int fp4_quantize_mx_1x32(const float* x, int32_t G, int64_t R, int64_t K,
                         uint8_t* q, uint8_t* scale_t);

/*
 * Host quantizers (CPU, synchronous), ceil-E8M0 scales and nearest-even E4M3:
 * for each block, t = the smallest integer with 448 * 2^t >= amax (t = 0 for
 * an all-zero block), scale byte = t + 127, q = E4M3(x / 2^t).  The rounding
 * up of the scale is what keeps |x / scale| <= 448 (first reference page,
 * section "DeepGEMM conformance details").  Ragged K (and N) are allowed:
 * a partial block uses only its elements.  Returns GFG_ERANGE if a block
 * needs t outside [-127, 127] or holds a non-finite value.
 *
 * fp8_quantize_act_1x128:    x [M][K] float -> q [M][K] e4m3, scale_t [ceil(K/128)][M]
 * fp8_quantize_weight_128x128: w [G][N][K] float -> q [G][N][K], scale [G][ceil(N/128)][ceil(K/128)]
 */
GFG_API int fp8_quantize_act_1x128(const float* x, int64_t M, int64_t K,
                           uint8_t* q, uint8_t* scale_t);
GFG_API int fp8_quantize_weight_128x128(const float* w, int32_t G, int64_t N, int64_t K,
                                uint8_t* q, uint8_t* scale);

/*
 * Device quantizer (GPU, asynchronous on `stream`): the activation quantizer
 * above, run on the device, producing the A operand of either GEMM layout.
 *
 *   x        [G][M][K]            float32 (in_dtype GFG_IN_F32) or bfloat16
 *                                 (GFG_IN_BF16), DEVICE memory, 16-byte aligned
 *   q        [G][M][K]            e4m3 bytes, DEVICE memory, 16-byte aligned
 *   scale_t  [G][K/128][M]        E8M0 bytes, DEVICE memory (the transposed
 *                                 per-token layout, per group)
 *
 * G = 1 gives the contiguous layout's a / a_scale; G groups of M = M_max rows
 * give the masked layout's.  Per (1,128) block: t = the smallest integer with
 * 448 * 2^t >= max|x| (t = 0 for an all-zero block), scale byte t + 127,
 * q = E4M3(x / 2^t) nearest-even, as in the host quantizer (first reference
 * page, sections "Summary" and "DeepGEMM conformance details").  Where the
 * host quantizer returns GFG_ERANGE the device one cannot stop; instead a
 * block with a NaN or infinity gets scale byte 255 (E8M0 NaN) and q = 0x7F
 * (E4M3 NaN) for all its elements, and a block so small that t < -127 gets
 * t = -127 (which still keeps |x / 2^t| <= 448).
 *
 * Sizes: G in [1, 65535]; M, K >= 0 (either 0 is a no-op); K a multiple of
 * 128, M <= 2^30, K <= 2^24 and G * ceil(M/32) * K/128 < 2^31 - 64 (else
 * GFG_EUNSUPPORTED).  The library allocates and synchronizes nothing.
 */
GFG_API int fp8_quantize_act_1x128_device(const void* x, int32_t in_dtype, int32_t G, int64_t M, int64_t K,
                                          uint8_t* q, uint8_t* scale_t, void* stream);

/*
 * Token quantizer for the 8-bit integer products below (GPU, asynchronous on
 * `stream`): one scale per row.  With amax = max(max_k |x[m, k]|, 2^-100),
 *
 *   scale[m] = amax / 127,   q[m, k] = rint(x[m, k] * (127 / amax))
 *
 * every operation a single fp32 rounding to nearest, rint to even, so codes
 * lie in [-127, 127].  A row of zeros has codes 0.  A row with a NaN or an
 * infinity gets scale NaN and codes 0, which makes its products NaN.  Weights
 * [G][N][K] are G * N rows: the same call makes their per-channel scales.
 *
 *   x [M][K] GFG_IN_F32, _BF16 or _F16 ; q [M][K] int8 ; scale [M] float
 *   (x and q 16-byte aligned, scale 4-byte aligned, else GFG_EINVAL)
 *
 * Sizes: M >= 0 (0 is a no-op) and below 2^31, K a multiple of 16 up to
 * 2^17 - 16 (else GFG_EUNSUPPORTED).
 */
GFG_API int int8_quantize_token_device(const void* x, int32_t in_dtype, int64_t M, int64_t K, int8_t* q,
                                       float* scale, void* stream);

/*
 * 8-bit integer matrix product with one scale per token and per channel:
 *
 *   d[m, n] = (sum_k a[m, k] b[n, k]) * a_scale[m] * b_scale[n] + bias[n]
 *
 * The sum is an exact 32-bit integer; the scales and the bias are applied in
 * fp32, first a_scale, then b_scale, and d is rounded once.  So sum * a_scale has
 * to lie in fp32's range itself, also where b_scale would bring it back (it always
 * does for an a_scale below 2^97).
 *
 *   a [M][K] int8 ; a_scale [M] float ; b [N][K] int8 ; b_scale [N] float
 *   bias [N] float or NULL ; d [M][N] bf16 or f16
 *   (a and b 16-byte aligned, d 8-byte aligned, the rest 4-byte aligned, else
 *   GFG_EINVAL)
 *
 * Sizes: M >= 0 (0 is a no-op), M <= 128 * 65535, any N in [1, 2^28], K a
 * multiple of 16 up to 2^17 - 16, and few enough output tiles for one launch
 * (M * N below 2^36 always has; else GFG_EUNSUPPORTED).
 *
 * int8_linear is the token quantizer and this product in one call, from
 * x [M][K] in 32 or 16 bits: a 16-byte aligned device workspace of at least
 * int8_linear_workspace_bytes(M, K) bytes holds the codes and scales between
 * them (it needs no initialization; a call leaves nothing in it for the next).
 * Up to 4 rows (with at most 32 KB of codes) are quantized inside the product's
 * kernel, in one launch, with the same results.
 */
GFG_API int int8_gemm(const int8_t* a, const float* a_scale, const int8_t* b, const float* b_scale,
                      const float* bias, void* d, int64_t M, int64_t N, int64_t K, int32_t out_dtype, void* stream);
GFG_API int64_t int8_linear_workspace_bytes(int64_t M, int64_t K);
GFG_API int int8_linear(const void* x, int32_t in_dtype, const int8_t* b, const float* b_scale, const float* bias,
                        void* d, int64_t M, int64_t N, int64_t K, int32_t out_dtype, void* workspace,
                        int64_t workspace_bytes, void* stream);

/*
 * The 8-bit integer product in the two grouped layouts of the FP8 GEMM, with
 * the same rules for grouped_layout and masked_m: rows that belong to no
 * expert are left untouched.
 *
 *   contiguous: a [M][K], a_scale [M], grouped_layout [M], d [M][N]
 *   masked:     a [G][M_max][K], a_scale [G][M_max], masked_m [G], d [G][M_max][N]
 *   both:       b [G][N][K], b_scale [G][N]
 *
 * Sizes: N and K as in int8_gemm, 1 <= G <= 65535 (else GFG_EINVAL), at most
 * 4096 tiles of 128 rows (ceil(M / 128), or G * ceil(M_max / 128); else
 * GFG_EUNSUPPORTED).
 */
GFG_API int grouped_int8_gemm_contiguous(const int8_t* a, const float* a_scale, const int8_t* b,
                                         const float* b_scale, const int32_t* grouped_layout, void* d, int64_t M,
                                         int64_t N, int64_t K, int32_t G, int32_t out_dtype, void* stream);
GFG_API int grouped_int8_gemm_masked(const int8_t* a, const float* a_scale, const int8_t* b, const float* b_scale,
                                     const int32_t* masked_m, void* d, int32_t G, int64_t M_max, int64_t N,
                                     int64_t K, int32_t out_dtype, void* stream);

/*
 * Top-k router of a mixture-of-experts layer: for every token the k experts
 * of the largest logits, in falling order, ties to the lowest index.
 *
 *   score     softmax over all E experts, or sigmoid of each logit
 *   chosen by the logit, or, with a bias, by score + bias[e] (which selects
 *             only; the weight stays the score)
 *   weights   score * scale, or, renormalized, score / (sum of the chosen
 *             scores) * scale (0 where that sum is 0)
 *
 * An expert whose logit (or, with a bias, whose score + bias[e]) is -infinity or
 * NaN is never chosen; where fewer than k are left, the remaining ids are -1 with
 * weight 0 (the layers below skip them).
 *
 *   logits [T][E] GFG_IN_F32, _BF16 or _F16 ; bias [E] float or NULL
 *   ids [T][k] int32 ; weights [T][k] float
 *
 * Sizes: T >= 0 (0 is a no-op) and below 2^31, 1 <= k <= E (else GFG_EINVAL),
 * E <= 1024 and k <= 64 (else GFG_EUNSUPPORTED).
 */
enum gfg_moe_score { GFG_SCORE_SOFTMAX = 0, GFG_SCORE_SIGMOID = 1 };
GFG_API int moe_topk(const void* logits, int32_t in_dtype, const float* bias, int32_t* ids, float* weights, int64_t T,
                     int64_t E, int64_t k, int32_t score, int32_t renormalize, float scale, void* stream);

/*
 * A whole mixture-of-experts layer for a few tokens (two or three launches):
 *
 *   g | u = W1[e] x[t],  h = silu(g) * u,
 *   out[t] = sum over j of topk_weights[t, j] * (W2[e] h),  e = topk_ids[t, j]
 *
 * Ids outside [0, E) (another rank's experts, or none) contribute nothing; a
 * token with no expert here gets zeros.  A token may name an expert twice.
 * The tokens stay in 16 bits, the hidden rows keep 16 significant bits (of any
 * finite fp32 value), all sums are fp32 and out is rounded once.  Scales multiply
 * sums of the raw codes (of a 128-block in FP8, of a row in int8), so those sums
 * have to lie in fp32's range themselves; tokens and hidden values below 2^105
 * always keep them there.  Two calls with the same operands give the same bytes.
 * For more than 1024 pairs use the grouped products on the same weights.
 *
 *   x, out [T][H] bf16 or f16 (dtype GFG_OUT_*) ; topk_ids [T][k] int32 ;
 *   topk_weights [T][k] float
 *   moe_fp8_layer:  w1 [E][2*I][H] e4m3 (gate rows, then up rows), w1_scale
 *                   [E][2*I/128][H/128] E8M0 ; w2 [E][H][I], w2_scale
 *                   [E][H/128][I/128]: the B operands of the FP8 GEMMs
 *   moe_int8_layer: w1 [E][2*I][H] int8, w1_scale [E][2*I] float ; w2
 *                   [E][H][I], w2_scale [E][H]: those of the int8 products
 *   workspace       16-byte aligned device memory, at least
 *                   moe_layer_workspace_bytes(T, k, H, I) bytes, uninitialized
 *
 * Sizes: T >= 0 (0 is a no-op), T * k <= 1024, E <= 1024, H and I multiples of
 * 128 up to 32256 (else GFG_EUNSUPPORTED).
 */
GFG_API int64_t moe_layer_workspace_bytes(int64_t T, int64_t k, int64_t H, int64_t I);
GFG_API int moe_fp8_layer(const void* x, int32_t dtype, const int32_t* topk_ids, const float* topk_weights,
                          const void* w1, const uint8_t* w1_scale, const void* w2, const uint8_t* w2_scale, void* out,
                          int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, void* workspace,
                          int64_t workspace_bytes, void* stream);
GFG_API int moe_int8_layer(const void* x, int32_t dtype, const int32_t* topk_ids, const float* topk_weights,
                           const int8_t* w1, const float* w1_scale, const int8_t* w2, const float* w2_scale, void* out,
                           int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, void* workspace,
                           int64_t workspace_bytes, void* stream);

/*
 * FP8 linear layer (GPU, asynchronous on `stream`): the dense product on the
 * grouped GEMMs' operands, from one token on, with its quantizers and its
 * gradients.  Per block, t = the smallest integer with 448 * 2^t >= max|v| (t = 0
 * for zeros, at least -127), scale byte t + 127, code E4M3(v / 2^t) to nearest even;
 * a block with a NaN or an infinity gets byte 255 (NaN) and the codes of NaN, so
 * whatever it enters is NaN.  A last block of fewer elements has a scale of its own.
 *
 * fp8_gemm: d[m, n] = sum_k a[m, k] b[n, k] + bias[n]
 *   a [M][K] e4m3 ; a_scale [ceil(K/128)][a_scale_ld] E8M0, row m in byte m,
 *   a_scale_ld >= M (the grouped GEMMs' layout has a_scale_ld = M)
 *   b [N][K] e4m3 ; b_scale [ceil(N/128)][ceil(K/128)] E8M0
 *   bias [N] float or NULL ; d [M][N] bf16 or f16
 * fp8_linear: the same from x [M][K] (GFG_IN_F32, _BF16 or _F16), which it
 *   quantizes in blocks of 1 x 128 into the workspace (at least
 *   fp8_linear_workspace_bytes(M, K) bytes of device memory, 16-byte aligned,
 *   uninitialized; a call leaves nothing in it for the next).  Few or short rows
 *   are quantized inside the product's launch, others in one before it.
 *
 * The sums are fp32 sums of the matrix instruction's products of 128 k, inside
 * which a product 2^14 times smaller than another of its group of 16 may be
 * dropped: an error of about 1.5e-5 of the result's norm where a group's operands are
 * drawn alike.  dw's groups are 16 tokens: of sizes from 2^-4 to 2^4 about 5e-5, from
 * 2^-8 to 2^8 6e-5.  d is rounded once.
 *
 * fp8_linear_backward, for y = x W^T + bias and the gradient dy of y:
 *   dx = Q(dy) W          dy in blocks of 1 x 128 along N
 *   dW = Q(dy^T) Q(x^T)^T both in blocks of 128 tokens
 *   dbias = the sum of dy over the tokens, in fp32
 *   dy [M][N], x [M][K] (the same in_dtype) ; b_t [K][N] e4m3, b_t_scale
 *   [ceil(K/128)][ceil(N/128)]: the transposed weight (fp8_quantize_weight_device)
 *   dx [M][K] bf16 or f16 ; dw [N][K] bf16, f16 or GFG_OUT_F32 ; dbias [N] float
 *   Each of dx, dw and dbias may be NULL (not all), and is then not computed; x
 *   is read for dw, b_t for dx.  accumulate: dw (GFG_OUT_F32 only, else
 *   GFG_EINVAL) and dbias are added to.  M = 0: dw and dbias are zeros, or are
 *   left as they are.
 *   workspace: at least fp8_linear_backward_workspace_bytes(M, N, K) bytes, as above.
 *
 * fp8_quantize_weight_device: w [G][N][K] (32 or 16 bits) in blocks of 128 x 128:
 *   q [G][N][K], scale [G][ceil(N/128)][ceil(K/128)], and, unless both are NULL,
 *   the same codes and bytes transposed, q_t [G][K][N], scale_t
 *   [G][ceil(K/128)][ceil(N/128)] (N a multiple of 16).  The grouped GEMMs' B
 *   operand is one of these too.
 *
 * Alignment: x, dy, w and all codes 16 bytes, d, dx and dw 8, bias and dbias 4
 * (else GFG_EINVAL).  Two calls with the same operands give the same bytes.
 *
 * Sizes: M >= 0 and at most 128 * 65535 (0 is a no-op, but for the gradients
 * above), N in [1, 2^28], K a multiple of 16 up to 2^22, fewer than 2^31 scale
 * bytes, 2^37 elements of x and 2^24 tiles of 128 x 128; backward: also N a multiple of
 * 16 up to 2^22, and M at most 2^22; else GFG_EUNSUPPORTED.
 */
GFG_API int fp8_gemm(const void* a, const uint8_t* a_scale, int64_t a_scale_ld, const void* b, const uint8_t* b_scale,
                     const float* bias, void* d, int64_t M, int64_t N, int64_t K, int32_t out_dtype, void* stream);
GFG_API int64_t fp8_linear_workspace_bytes(int64_t M, int64_t K);
GFG_API int fp8_linear(const void* x, int32_t in_dtype, const void* b, const uint8_t* b_scale, const float* bias, void* d,
                       int64_t M, int64_t N, int64_t K, int32_t out_dtype, void* workspace, int64_t workspace_bytes,
                       void* stream);
GFG_API int64_t fp8_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K);
GFG_API int fp8_linear_backward(const void* dy, const void* x, int32_t in_dtype, const void* b_t, const uint8_t* b_t_scale,
                                void* dx, void* dw, float* dbias, int64_t M, int64_t N, int64_t K, int32_t dx_dtype,
                                int32_t dw_dtype, int32_t accumulate, void* workspace, int64_t workspace_bytes,
                                void* stream);
GFG_API int fp8_quantize_weight_device(const void* w, int32_t in_dtype, int32_t G, int64_t N, int64_t K, uint8_t* q,
                                       uint8_t* scale, uint8_t* q_t, uint8_t* scale_t, void* stream);

/*
 * Between two blocks of a network (GPU, asynchronous on `stream`): the norm after
 * a block, its gate, the residual sum and the norm before the next block, in one
 * pass over the rows.  With rstd(v) = 1 / sqrt(mean(v^2) + eps), per row m of H:
 *
 *   u      = y * rstd(y) * post_weight     or u = y without post_weight
 *   out    = alpha * residual + gate * u   (gate 1 where there is none, u = 0 without y)
 *   normed = out * rstd(out) * weight      of the unrounded out
 *
 *   y [M][H] (dtype: GFG_IN_*) or NULL ; residual, out [M][H] (residual_dtype:
 *   dtype, or GFG_IN_F32) ; normed [M][H] (dtype) ; post_weight, weight [H] float
 *   gate: GFG_GATE_NONE, GFG_GATE_CHANNEL (float [H]) or GFG_GATE_TOKEN (float [M])
 *   out may be residual itself, and may be NULL; without weight there is no normed.
 *   stats [2][M] float or NULL: rstd(y) (1 without y or post_weight) and rstd(out)
 *   (written where weight is given)
 *   residual_norm_fp8: normed as the operand of fp8_gemm and the grouped GEMMs, in
 *   place of 16 bits: q [M][H] e4m3, scale [ceil(H/128)][scale_ld] E8M0 (H a multiple
 *   of 16, q 8-byte aligned), quantized as in fp8_linear from the unrounded values
 *
 * residual_norm_backward: from dout [M][H] (residual_dtype) and dnormed [M][H]
 * (dtype), either may be NULL, and the forward call's out, y and stats.  With
 * zh = out * rstd(out), yh = y * rstd(y) (y without post_weight):
 *
 *   G  = dout + rstd(out) * (dnormed * weight - zh * mean(dnormed * weight * zh))
 *   dresidual = alpha * G ; du = gate * G
 *   dy = rstd(y) * (post_weight * du - yh * mean(post_weight * du * yh))  (du without post_weight)
 *   dweight = sum_m dnormed * zh ; dpost_weight = sum_m du * yh ; dgate = the sum
 *   of G * u over m (GFG_GATE_CHANNEL) or over the row (GFG_GATE_TOKEN)
 *
 *   Each output may be NULL.  accumulate: dweight, dpost_weight and a channel
 *   gate's dgate are added to.  M = 0 writes zeros to those (unless accumulated).
 *   workspace: residual_norm_backward_workspace_bytes(M, H) bytes of device memory,
 *   16-byte aligned, uninitialized (what M rows need serves fewer too); needed for
 *   dweight, dpost_weight and a channel gate's dgate.
 *
 * All sums and statistics are fp32 (so a row's squares have to sum up within
 * fp32's range); every output is rounded once.  Two calls give the same bytes.
 * Rows need no alignment beyond that of their elements.
 *
 * Sizes: M >= 0 (0 is a no-op but for the sums) and below 2^31, H in [8, 32768]
 * (else GFG_EUNSUPPORTED).
 */
enum gfg_gate { GFG_GATE_NONE = 0, GFG_GATE_CHANNEL = 1, GFG_GATE_TOKEN = 2 };
GFG_API int residual_norm(const void* y, const void* residual, const float* weight, const float* post_weight,
                          const float* gate, int32_t gate_kind, float alpha, float eps, void* out, void* normed,
                          float* stats, int64_t M, int64_t H, int32_t dtype, int32_t residual_dtype, void* stream);
GFG_API int residual_norm_fp8(const void* y, const void* residual, const float* weight, const float* post_weight,
                              const float* gate, int32_t gate_kind, float alpha, float eps, void* out, uint8_t* q,
                              uint8_t* scale, int64_t scale_ld, float* stats, int64_t M, int64_t H, int32_t dtype,
                              int32_t residual_dtype, void* stream);
GFG_API int64_t residual_norm_backward_workspace_bytes(int64_t M, int64_t H);
GFG_API int residual_norm_backward(const void* dout, const void* dnormed, const void* out, const void* y,
                                   const float* stats, const float* weight, const float* post_weight,
                                   const float* gate, int32_t gate_kind, float alpha, void* dresidual, void* dy,
                                   float* dweight, float* dpost_weight, float* dgate, int32_t accumulate, int64_t M,
                                   int64_t H, int32_t dtype, int32_t residual_dtype, void* workspace,
                                   int64_t workspace_bytes, void* stream);

/*
 * Training of the router (GPU, asynchronous on `stream`).  moe_balance_loss: how
 * unevenly the tokens of each sequence spread over the experts, with the counts.
 * A token counts if it has an id in [0, E) (padding has ids -1, say).  For
 * sequence s with n tokens that count, over those:
 *
 *   counts[s, e] = how often e is an id ;  f_e = counts[s, e] * E / (k n)
 *   P_e = mean of p_e: the softmax of the logits, or the sigmoids over their sum
 *   loss = 1/S sum_s (alpha * sum_e f_e P_e + z * mean(logsumexp(logits)^2))
 *
 * Logits of -infinity or NaN are of masked experts (p = 0), and so, in effect, is a
 * sigmoid below fp32's normal range (a logit below about -87).  A sequence without
 * such tokens adds 0.
 *
 *   logits [T][E] (GFG_IN_*) ; ids [T][k] int32 (moe_topk's) ; seq_offsets [S+1]
 *   int32, rising from 0 to T, or NULL with S = 1 ; tokens outside are in no sequence
 *   loss [1] float ; counts [S][E] int32
 *   factors [S][E+1] float: alpha f_e / (S n), then 2 z / (S n), for the gradient
 *   workspace: moe_balance_workspace_bytes(T, E, S) bytes of device memory, 16-byte
 *   aligned, uninitialized (what T tokens need serves fewer too)
 *
 * moe_router_backward: dlogits [T][E] (the logits' type) of
 *
 *   dloss * loss + sum over t, j of dweights[t, j] * weights[t, j]
 *
 * with moe_topk's weights (same score, renormalize and scale; the choice and the
 * bias have no gradient).  dweights [T][k] float or NULL ; factors (with seq_offsets
 * and S as above) and dloss [1] float, both or neither NULL.  Ids outside [0, E)
 * have no weight; an id that stands twice has both.  dlogits is 0 where p is.  The
 * gradient of renormalized weights holds for all scores that fp32 does (softmaxes down
 * to e^-103 of the token's largest, sigmoids of logits down to -88.7); smaller ones
 * have none.
 *
 * Equal dweights of renormalized weights (a single one above all) have a gradient
 * of exactly 0.  Counts are exact, the sums fp32 in a fixed order: two calls give the same bytes.
 * Sizes: T >= 0 (0: loss and counts are 0) and below 2^31, E in [1, 1024],
 * k in [1, 64], S in [1, 65535] (else GFG_EUNSUPPORTED).
 */
GFG_API int64_t moe_balance_workspace_bytes(int64_t T, int64_t E, int64_t S);
GFG_API int moe_balance_loss(const void* logits, int32_t in_dtype, const int32_t* ids, const int32_t* seq_offsets,
                             float* loss, int32_t* counts, float* factors, int64_t T, int64_t E, int64_t k, int64_t S,
                             int32_t score, float alpha, float z, void* workspace, int64_t workspace_bytes,
                             void* stream);
GFG_API int moe_router_backward(const void* logits, int32_t in_dtype, const int32_t* ids, const float* dweights,
                                const float* factors, const float* dloss, const int32_t* seq_offsets, void* dlogits,
                                int64_t T, int64_t E, int64_t k, int64_t S, int32_t score, int32_t renormalize,
                                float scale, void* stream);

/*
 * Launch settings (process-wide, read at every GEMM call; not synchronized
 * with calls in flight on other threads).
 *
 * grouped_fp8_set_tile_order: the order in which a launch walks its
 * (M tile, N tile) work items.  The items are split into num_xcd contiguous
 * ranges, one per XCD (the hardware deals workgroup w to XCD w % 8, so with
 * num_xcd = 8 each range stays in one XCD's L2), and inside a range they
 * follow a grouped-M order group_m M tiles wide.  This is the locality mapping
 * of the second reference page ("[Kernel][MI350] Add cache-aware 8-wave
 * BF16/FP16 GEMM", section "Changes": XCD remap and grouped-M traversal with
 * a shortened final group, composed), made a run-time choice for its ablation
 * (section "Performance", second table).  Defaults: num_xcd = 8, group_m = 0
 * (each kernel's own width).  Every setting gives the same bytes: only the
 * order of the tiles changes.  num_xcd in [1, 8], group_m in [0, 64], else
 * GFG_EINVAL.
 *
 * grouped_fp8_set_tile_shape: the output tile of the plain FP8 GEMM calls
 * (grouped_fp8_gemm_contiguous / _masked).  GFG_TILE_AUTO picks 256 x 256
 * (where its requirements hold) when R256 * 1.6 <= R128, R being the rounds
 * of each shape's tiles over the CUs (ceil(tiles / CUs)), and either
 * R256 >= 2 or K >= 4096 (contiguous layout) or at least two 256 x 256 tiles
 * per CU (masked layout, counted from M_max: masked_m is device memory); for
 * the contiguous layout the rows must also average at least two 128-row tiles
 * per expert; else 128 x 256.  GFG_TILE_256x256 needs N a multiple of 256 and
 * at most 2^22, K/128 even, scale rows a multiple of 4 and scale_a 4-byte
 * aligned; a call that misses them then returns GFG_EUNSUPPORTED.  Other
 * values: GFG_EINVAL.  Results of the two tiles agree to the parity
 * tolerance; they are not promised to agree bit for bit.  The int8 products
 * follow the setting too: GFG_TILE_AUTO takes their large tiles (256 or 192 rows
 * by 256 columns) where tiles of 128 x 128 would outnumber the CUs,
 * GFG_TILE_128x256 the smaller ones, GFG_TILE_256x256 the large ones (N at most
 * 2^22); their results do not depend on it.  The dense FP8 products follow it in
 * the same way: large tiles (256 x 256, an operand of at least 4 rows) where tiles of
 * 256 x 128 would outnumber the CUs, those where tiles of 128 x 128 would;
 * GFG_TILE_256x256 needs N at most 2^21 (2^20 with 32-bit outputs), else
 * GFG_EUNSUPPORTED; with a set shape fp8_linear and fp8_linear_backward launch
 * their quantizers and products apart.
 *
 * grouped_fp8_set_grid_limit: at most max_workgroups workgroups per GEMM
 * launch.  0, the default, is no limit: one per CU, fewer when there are fewer
 * tiles (the int8 products' smaller tiles: one per tile).  The grid of a GEMM
 * launch is then rounded up to a multiple of num_xcd.  Each workgroup walks
 * more tiles; the results do not change.  The limit covers the FP8, MX and int8
 * products (int8_linear and fp8_linear of a few tokens and a small
 * fp8_linear_backward then take a launch for each product) and, not
 * rounded up, the expert layer's two products, whose fp32 sums it may reorder;
 * not the quantizers, the router and its training, the norms and the layer's last
 * sum over a token's pairs.
 * Negative: GFG_EINVAL.
 */
enum gfg_tile_shape { GFG_TILE_AUTO = 0, GFG_TILE_128x256 = 1, GFG_TILE_256x256 = 2 };
GFG_API int grouped_fp8_set_tile_order(int32_t num_xcd, int32_t group_m);
GFG_API int grouped_fp8_set_tile_shape(int32_t shape);
GFG_API int grouped_fp8_set_grid_limit(int32_t max_workgroups);

/* Thread-local message describing the calling thread's last failure ("" if none). */
GFG_API const char* grouped_fp8_last_error(void);

/* Library version string. */
GFG_API const char* gfg_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GFG_H */
