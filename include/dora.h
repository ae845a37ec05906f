/*
 * dora.h -- C ABI of libdora: the DoRA weight-norm and compose hot path on
 * GB300 (sm_103a).
 *
 * Method source (cited below as "P1 ¶<opening words>"):
 *   P1 = web page "人工智能训练新突破：Anthropic团队破解大模型微调内存瓶颈难题"
 *        (techwalker.com, 2026-04-01), summarising arXiv:2603.22276.
 *
 * Notation: W0[out,in] frozen base weight, A[r,in] and B[out,r] the low-rank
 * adapter, s its scale, m[out] the DoRA magnitude; activations base = x W0^T
 * and lora = x A^T B^T (NOT pre-scaled by s) are [T,out].
 *
 *   n_i  = || W0_i + s (B A)_i ||                       (per output row)
 *   g_i  = m_i / n_i
 *   y    = base + (g-1)*base + g*s*lora                 (g broadcast over T)
 *   d_base = g*dy,  d_lora = s*g*dy,
 *   d_mag_j = sum_t dy[t,j] * (base[t,j] + s*lora[t,j]) / n_j   (n held constant)
 *
 * Conventions shared by every entry point:
 *   - Every data pointer is a DEVICE pointer owned by the caller.  The library
 *     never allocates, frees or synchronises; every call is asynchronous on
 *     `stream` (NULL = the legacy default stream).
 *   - Arrays are dense and row-major with the shapes given; no aliasing
 *     between any input and any output.
 *   - Argument errors are detected on the host before anything is launched and
 *     return a status with no side effect.  A failed launch returns
 *     DORA_ERR_CUDA.  Kernels that wait on on-chip barriers give up after a
 *     bounded time and record it in a device word read by dora_device_error().
 *   - Results are bitwise reproducible for a given shape on a given device.
 *   - Only sm_103 devices are accepted (DORA_ERR_ARCH otherwise).
 *   - The calls may be captured in a CUDA graph once the same call (same
 *     shapes and buffers) has run outside capture: the first call of a
 *     device sets up kernel attributes, and the first with a shape or a set
 *     of buffers builds the plan and tensor maps it then reuses.  A replay
 *     gives the same bits as the calls launched one by one.
 */
#ifndef DORA_H
#define DORA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t / CUstream. */
typedef struct CUstream_st *dora_stream_t;

typedef enum {
  DORA_OK = 0,
  DORA_ERR_NULL = 1,       /* a required pointer is NULL                          */
  DORA_ERR_SHAPE = 2,      /* a size is negative, zero where not allowed, or too large */
  DORA_ERR_ALIGN = 3,      /* a pointer or row stride breaks an alignment rule    */
  DORA_ERR_DTYPE = 4,      /* unknown activation dtype                            */
  DORA_ERR_WORKSPACE = 5,  /* workspace NULL, misaligned or smaller than required */
  DORA_ERR_ARCH = 6,       /* current device is not sm_103                        */
  DORA_ERR_CUDA = 7,       /* a CUDA runtime/driver call or launch failed         */
  DORA_ERR_DEVICE = 8      /* a kernel's bounded on-chip wait gave up (see dora_device_error) */
} dora_status;

typedef enum {
  DORA_F32 = 0,            /* activations and their gradients are float32  */
  DORA_BF16 = 1            /* activations and their gradients are bfloat16 */
} dora_dtype;

/* Human-readable name of a status code (static string, never NULL). */
const char *dora_status_str(dora_status st);

/* ------------------------------------------------------------------------ */
/* (a) factored per-output-row weight norm                                   */
/* ------------------------------------------------------------------------ */

/*
 * Bytes of device workspace dora_norm_factored needs for this shape.  Pure
 * host arithmetic (no CUDA call); an upper bound valid on any device.  It grows
 * as O((out + in)*r + r^2) -- rank-dependent factors only, never out*in
 * (P1 ¶第一个创新是"因式分解规范化"技术: memory O(out*in) -> O(out*r + r^2)).
 * Returns 0 for an invalid shape.
 */
size_t dora_norm_factored_workspace(int64_t out, int64_t in, int64_t r);

/*
 * norm[i] = || W0_i + s (B A)_i ||,  g[i] = m[i] / norm[i]   for i < out.
 *
 * P1 ¶第一个创新是"因式分解规范化"技术: the squared norm is evaluated as a base
 * term, a cross term and a Gram term,
 *     n_i^2 = ||W0_i||^2 + 2 s <U_i, B_i> + s^2 B_i G B_i^T,
 *     U = W0 A^T [out,r],  G = A A^T [r,r],
 * so the out x in adapted weight is never formed.  The contractions run on the
 * tensor cores with every fp32 operand split as x = h + l (h = bf16(x),
 * l = bf16(x - h)): each product as three bf16 products h*h + l*h + h*l with
 * fp32 accumulation (dropped terms <= 3 * 2^-18 of the product); n^2 is
 * clamped at 0 before the square root; g is an IEEE division with no epsilon
 * (n = 0 gives inf/NaN).  Two launches (the split of A, then one cooperative
 * launch with one CTA per SM whose CTAs wait on one another through counters
 * in the workspace); a device that cannot hold every CTA at once gets
 * DORA_ERR_CUDA.  Plans and encoded tensor maps are cached per shape and per
 * buffer set, so repeated calls cost a few microseconds of host time.
 *
 *   W0    float32 [out, in]    16-byte aligned, in % 4 == 0
 *   A     float32 [r, in]      16-byte aligned
 *   B     float32 [out, r]     16-byte aligned (any r >= 1)
 *   m     float32 [out]        4-byte aligned
 *   s     adapter scale (e.g. alpha/sqrt(r))
 *   norm  float32 [out]  out
 *   g     float32 [out]  out
 *   workspace  >= dora_norm_factored_workspace(out,in,r) bytes, 256-byte
 *              aligned, caller-owned scratch; contents on entry are ignored
 *   Sizes: out >= 0 (0 is a no-op), in >= 1, r >= 1, r <= 1024,
 *          out, in < 2^31.
 */
dora_status dora_norm_factored(const float *W0, const float *A, const float *B,
                               const float *m, float s,
                               int64_t out, int64_t in, int64_t r,
                               float *norm, float *g,
                               void *workspace, size_t workspace_bytes,
                               dora_stream_t stream);

/* ------------------------------------------------------------------------ */
/* (a') the same norm for bf16 weights                                       */
/* ------------------------------------------------------------------------ */

/*
 * n0sq[i] = sum_j W0[i,j]^2 for a bfloat16 W0 [rows, cols], fp32 result in a
 * fixed summation order.  W0 is frozen during fine-tuning, so its row norms
 * are computed once and passed to every dora_norm_factored_bf16 call (the
 * base term of P1 ¶第一个创新是"因式分解规范化"技术).
 *   W0    bfloat16 [rows, cols]  16-byte aligned, cols % 8 == 0
 *   n0sq  float32 [rows]         4-byte aligned
 *   Sizes: rows >= 0 (0 is a no-op), cols >= 1, both < 2^31.
 */
dora_status dora_row_sumsq_bf16(const void *W0, int64_t rows, int64_t cols, float *n0sq,
                                dora_stream_t stream);

/* Bytes of workspace dora_norm_factored_bf16 needs (host arithmetic; 0 for an
 * invalid shape).  O(out + (out + r) r) bytes: s/2 G in three bf16 pieces,
 * partial sums, and B padded to a 16-byte row when r % 8 != 0. */
size_t dora_norm_factored_bf16_workspace(int64_t out, int64_t in, int64_t r);

/*
 * The factored norm of dora_norm_factored for bfloat16 W0, A and B (the same
 * definition, P1 ¶第一个创新是"因式分解规范化"技术), with the base term taken from
 * n0sq:
 *     n_i^2 = n0sq[i] + 2 s <U_i, B_i> + s^2 B_i G B_i^T,   g_i = m_i / n_i.
 * Products of bf16 values are exact in fp32, so U = W0 A^T and G = A A^T are
 * single bf16 tensor-core products with fp32 accumulation; s/2 G enters as three
 * bf16 pieces whose sum carries it to fp32 precision.  No adapter or weight is
 * converted or copied (B only when r % 8 != 0).
 *
 *   W0    bfloat16 [out, in]   16-byte aligned, in % 8 == 0
 *   A     bfloat16 [r, in]     16-byte aligned
 *   B     bfloat16 [out, r]    16-byte aligned (any r >= 1)
 *   m     float32 [out]        4-byte aligned
 *   n0sq  float32 [out]        ||W0_i||^2 (dora_row_sumsq_bf16), 4-byte aligned
 *   s, norm, g, workspace, sizes: as dora_norm_factored (workspace from
 *   dora_norm_factored_bf16_workspace).
 */
dora_status dora_norm_factored_bf16(const void *W0, const void *A, const void *B,
                                    const float *m, const float *n0sq, float s,
                                    int64_t out, int64_t in, int64_t r,
                                    float *norm, float *g,
                                    void *workspace, size_t workspace_bytes,
                                    dora_stream_t stream);

/* ------------------------------------------------------------------------ */
/* (a'') gradient through the norm (the variant with the norm not detached)  */
/* ------------------------------------------------------------------------ */

/* Bytes of workspace dora_norm_factored_bwd needs (host arithmetic; 0 for an
 * invalid shape).  O((out + in) r + r^2) bytes, never out*in. */
size_t dora_norm_factored_bwd_workspace(int64_t out, int64_t in, int64_t r);

/*
 * The part of dL/dA and dL/dB that flows through the row norm n, for a loss
 * that sees n only through g = m / n.  P1 is silent on a gradient through the
 * norm (its backward holds n constant, which is what dora_compose_bwd does);
 * this entry point is the plain chain rule for callers that do not detach it.
 * With d_mag = dL/dm as dora_compose_bwd writes it, dL/dn_i = -g_i d_mag_i and,
 * for V = W0 + s B A and c_i = (dL/dn_i) / n_i,
 *
 *   dB = s c (.) (W0 A^T + s B G),         G = A A^T
 *   dA = s (c (.) B)^T W0 + s^2 H A,       H = B^T diag(c) B
 *
 * evaluated in factored form (the out x in matrix V is never formed) on the
 * tensor cores with the same bf16 three-product split (x = h + l, each
 * product h h + l h + h l, fp32 accumulation) as dora_norm_factored.
 * The outputs are ONLY the norm's share: the caller adds the gradients of its
 * own lora = x A^T B^T product.  dA and dB are overwritten.
 *
 *   W0, A, B   float32, as for dora_norm_factored (16-byte aligned, in % 4 == 0)
 *   norm, g    float32 [out]  the forward's outputs (dora_norm_factored)
 *   d_mag      float32 [out]  dL/dm (dora_compose_bwd)
 *   dA         float32 [r, in]   dB  float32 [out, r]   (4-byte aligned)
 *   workspace  >= dora_norm_factored_bwd_workspace(out, in, r) bytes, 256-byte aligned
 *   Sizes as dora_norm_factored; out == 0 writes zeros to dA (an empty sum).
 * Launches at most 11 kernels (A split, B padding when r % 4 != 0, the split of
 * s c (.) B transposed, two Gram passes and their reductions, the dB and dA
 * passes and the fixed-order sums of their stream-K parts); results are
 * bitwise reproducible.
 */
dora_status dora_norm_factored_bwd(const float *W0, const float *A, const float *B,
                                   const float *norm, const float *g, const float *d_mag,
                                   float s, int64_t out, int64_t in, int64_t r,
                                   float *dA, float *dB,
                                   void *workspace, size_t workspace_bytes,
                                   dora_stream_t stream);

/* ------------------------------------------------------------------------ */
/* (b) fused compose, forward                                                */
/* ------------------------------------------------------------------------ */

/*
 * y = base + (g-1)*base + g*s*lora, one pass over [T,out].
 *
 * P1 ¶第二个创新是"融合Triton内核"技术 (four elementwise kernels fused into one)
 * and ¶从技术架构角度来看 / ¶他们在一个Qwen2-VL-7B适配器上的测量 (stable form with
 * the correction (g-1) kept explicit, fp32 intermediates).  Every element is
 * computed in fp32 and rounded once (nearest even) to the activation dtype.
 *
 *   act   DORA_F32 or DORA_BF16: dtype of base, lora and y
 *   base, lora  [T, out] of `act`
 *   g     float32 [out]
 *   y     [T, out] of `act`
 *   Sizes: T >= 0, out >= 0 (either 0 is a no-op).  Any out and any element
 *   alignment are accepted; the 128-bit path is taken when out is a multiple
 *   of 16/sizeof(act) and base, lora and y are 16-byte aligned.
 */
dora_status dora_compose_fwd(dora_dtype act, const void *base, const void *lora,
                             const float *g, float s, int64_t T, int64_t out,
                             void *y, dora_stream_t stream);

/* ------------------------------------------------------------------------ */
/* (b) fused compose, backward                                               */
/* ------------------------------------------------------------------------ */

/*
 * Bytes of device workspace dora_compose_bwd needs (fp32 partial column sums
 * of d_mag).  Pure host arithmetic; an upper bound valid on any device.
 */
size_t dora_compose_bwd_workspace(int64_t T, int64_t out);

/*
 * d_base = g*dy,  d_lora = s*g*dy,
 * d_mag[j] = (sum_t dy[t,j]*(base[t,j] + s*lora[t,j])) / norm[j].
 *
 * P1 ¶研究团队还设计了一个智能的三层调度系统 (fused backward in training) and
 * ¶研究团队还进行了广泛的收敛等价性验证 (d_mag reduction order).  The row norm is
 * treated as a constant (no gradient into A or B).  d_base and d_lora are
 * rounded once to `act`; d_mag is float32, summed in a fixed order (per-thread
 * token runs, then a fixed-order sum of the per-run partials), so it is
 * bitwise reproducible.  d_mag is overwritten, not accumulated.
 *
 *   act        dtype of grad_out, base, lora, d_base, d_lora
 *   grad_out, base, lora   [T, out] of `act`
 *   g, norm    float32 [out]
 *   d_base, d_lora  [T, out] of `act`
 *   d_mag      float32 [out]
 *   workspace  >= dora_compose_bwd_workspace(T,out) bytes, 256-byte aligned
 *   Sizes: T >= 0, out >= 0 (out == 0 is a no-op; T == 0 gives d_mag = 0).
 */
dora_status dora_compose_bwd(dora_dtype act, const void *grad_out, const void *base,
                             const void *lora, const float *g, const float *norm,
                             float s, int64_t T, int64_t out,
                             void *d_base, void *d_lora, float *d_mag,
                             void *workspace, size_t workspace_bytes,
                             dora_stream_t stream);

/* ------------------------------------------------------------------------ */
/* (b') compose backward without a workspace                                 */
/* ------------------------------------------------------------------------ */

/* Size, in floats, of the library's fixed device scratch array (4 MiB). */
#define DORA_NOALLOC_SCRATCH_FLOATS (1 << 20)

/*
 * Same results as dora_compose_bwd, but allocation-free for the caller: no
 * workspace argument.  The paper has no counterpart to this entry point; it
 * exists for callers that cannot allocate device memory where they run the
 * backward -- code embedded in an application that owns a fixed device memory
 * pool and exposes no allocator, or services that forbid cudaMalloc after
 * start-up because it synchronises the device and fragments shared memory.
 *
 * The d_mag partial sums go to one file-scope device array of
 * DORA_NOALLOC_SCRATCH_FLOATS floats, held on every GPU that loads the library
 * until the process exits.  The first call on a device looks up that array's
 * device address (cudaGetSymbolAddress, with the device current); make that
 * first call before any stream capture.  A device reset (cudaDeviceReset)
 * gives the device a new context and invalidates the address: the next call
 * looks it up again, so after a reset, too, make one call before any capture.
 * Every partial sum the call reads is
 * written earlier in the same call, so nothing needs clearing between calls,
 * but all calls share the one array: calls that overlap on the GPU (different
 * streams, or concurrent host threads on one device) race and give wrong
 * d_mag.  The call itself allocates nothing (no cudaMalloc/cudaFree, no
 * allocating library routine).
 *
 * Arguments, layouts and errors as dora_compose_bwd, plus: out must not exceed
 * DORA_NOALLOC_SCRATCH_FLOATS (DORA_ERR_SHAPE otherwise).  The call launches
 * exactly the grid dora_compose_bwd launches, so d_mag is bitwise the same.
 * That grid's partial rows times out stay below 4096 x the SM count floats,
 * which fits the array on any device with up to 256 SMs (GB300 has 152); a
 * device where it would not fit gets DORA_ERR_SHAPE before any launch.
 */
dora_status dora_compose_bwd_noalloc(dora_dtype act, const void *grad_out, const void *base,
                                     const void *lora, const float *g, const float *norm,
                                     float s, int64_t T, int64_t out,
                                     void *d_base, void *d_lora, float *d_mag,
                                     dora_stream_t stream);

/* ------------------------------------------------------------------------ */
/* (d) the compose folded into its adjacent products                         */
/* ------------------------------------------------------------------------ */

/* Bytes of workspace dora_compose_lora_fwd and dora_linear_fwd need (host
 * arithmetic; 0 for an invalid shape): s B split into two bf16 [out, r]
 * matrices.  dora_compose_lora_fwd_bf16 needs none. */
size_t dora_compose_fused_workspace(int64_t out, int64_t r);

/*
 * y = base + (g-1)*base + g*s*lora with lora = xa B^T computed in the same
 * kernel: the compose moved into the epilogue of the lora up-projection, so
 * lora never reaches memory (P1 ¶第二个创新是"融合Triton内核"技术 and
 * ¶从技术架构角度来看: the stable form, fp32 intermediates).  xa = x A^T is the
 * caller's down-projection.  s B is split into bf16 hi + lo (residual <= 2^-17
 * of s B), so each product is exact; fp32 accumulation on the tensor cores;
 * y is rounded once (nearest even) to bf16.
 *
 *   base  bf16 [T, out]   xa  bf16 [T, r]   y  bf16 [T, out]  (16-byte aligned)
 *   B     float32 [out, r] (4-byte aligned)   g  float32 [out] (16-byte aligned)
 *   workspace  >= dora_compose_fused_workspace(out, r) bytes, 256-byte aligned
 *   Sizes: T, out >= 0 (either 0 is a no-op), r >= 1; out % 8 == 0 and
 *   r % 8 == 0 (16-byte rows for the tensor-memory copies).
 * Two launches: the split of s B, then the fused kernel, as clusters of two
 * CTAs (one 256 x 256 tile of y per pair, tcgen05.mma.cta_group::2) where
 * the device can hold such clusters, else as single CTAs (128 x 256 tiles).
 * The fused kernel is a programmatic dependent launch on the split (its
 * set-up overlaps it); stream order is unchanged for the caller.
 * Results are bitwise reproducible for a given shape and device.
 */
dora_status dora_compose_lora_fwd(const void *base, const void *xa, const float *B,
                                  const float *g, float s,
                                  int64_t T, int64_t out, int64_t r, void *y,
                                  void *workspace, size_t workspace_bytes,
                                  dora_stream_t stream);

/*
 * The same lora up-projection form for a bf16 B (adapters kept in bf16):
 * y = base + (g-1)*base + g*(s*acc) with acc = xa B^T, B used as it is as the
 * tensor-core operand (every product exact in fp32, fp32 accumulation), s
 * applied to the accumulator in the epilogue, y rounded once to bf16
 * (P1 ¶第二个创新是"融合Triton内核"技术, the stable form).  One product instead
 * of the fp32-B form's two, and no split of B: one launch, no workspace.
 *
 *   base  bf16 [T, out]   xa  bf16 [T, r]   B  bf16 [out, r]   y  bf16 [T, out]
 *   g  float32 [out]; all five 16-byte aligned
 *   Sizes: T, out >= 0 (either 0 is a no-op), r >= 1; out % 8 == 0 and
 *   r % 8 == 0.
 * One launch (an ordinary one: it reads base from its first instruction), as
 * clusters of two CTAs where the device holds them, else single CTAs.
 * Results are bitwise reproducible for a given shape and device.
 */
dora_status dora_compose_lora_fwd_bf16(const void *base, const void *xa, const void *B,
                                       const float *g, float s,
                                       int64_t T, int64_t out, int64_t r, void *y,
                                       dora_stream_t stream);

/*
 * The whole layer output y = g*(x W0^T + s xa B^T) as ONE tensor-core GEMM
 * over K = in + r ([x | xa] times [W0 | s B]^T), with the compose in its
 * epilogue: neither base nor lora is formed.  x [T, in] and W0 [out, in] are
 * bf16 (16-byte aligned, in % 8 == 0); the rest as dora_compose_lora_fwd.
 * Since base + s lora stays in fp32 until the single rounding of y, this is the
 * page's stable evaluation with one rounding fewer.  Launches as
 * dora_compose_lora_fwd.
 */
dora_status dora_linear_fwd(const void *x, const void *W0, const void *xa, const float *B,
                            const float *g, float s,
                            int64_t T, int64_t in, int64_t out, int64_t r, void *y,
                            void *workspace, size_t workspace_bytes,
                            dora_stream_t stream);

/* ------------------------------------------------------------------------ */
/* (e) the step's activations and frozen weight in 8 bits                    */
/* ------------------------------------------------------------------------ */

/*
 * The 8-bit form of a matrix [rows, cols]: q, one E4M3 byte per element
 * [rows, cols], and scale, one byte b per block, standing for 2^(b - 127),
 * [ceil(rows / block_rows), ceil(cols / 128)].  block_rows is 1 (an
 * activation: 128 columns of one row) or 128 (a frozen weight: 128 x 128).
 * An element's value is E4M3(q) 2^(b - 127), b from 1 to 254.
 *
 * The scale of a block is the smallest power of two that brings its largest
 * finite magnitude to at most 448, and at least 2^-117: every value is then
 * exact in bf16 (except that a float32 within half a step of 2^128 rounds to
 * infinity), rounding (nearest even) happens once, in E4M3, and a block of
 * zeros keeps zeros.  A NaN or an infinity becomes NaN and does not enter its
 * block's scale.
 *
 * The page keeps its activations in 16 bits; it names the memory that a step
 * holds from forward to backward as what limits it (P1 ¶目前最流行的模型微调技术
 * 叫做DoRA).  x and v = base + s lora in 8 bits are 2 bytes an element where x,
 * base and lora in bf16 are 6.
 */

/*
 * x into the 8-bit form, one pass.
 *   act    DORA_F32 or DORA_BF16: dtype of x
 *   x      [rows, cols] of `act`
 *   block_rows  1 or 128
 *   q      uint8 [rows, cols]  out
 *   scale  uint8 [ceil(rows / block_rows), ceil(cols / 128)]  out
 *   Sizes: rows, cols >= 0 (either 0 is a no-op), < 2^31.  Any cols and any
 *   element alignment are accepted; the 128-bit path (block_rows = 1) is taken
 *   when rows are whole 16-byte pieces of `act` and x and q are aligned to
 *   16 and 16 / sizeof(act) bytes.
 */
dora_status dora_q8_store(dora_dtype act, const void *x, int64_t rows, int64_t cols, int block_rows,
                          void *q, void *scale, dora_stream_t stream);

/* The values of an 8-bit form: x[i,j] = E4M3(q[i,j]) 2^(b - 127), one pass.
 * Arguments and sizes as dora_q8_store (x is written). */
dora_status dora_q8_load(dora_dtype act, const void *q, const void *scale, int64_t rows, int64_t cols,
                         int block_rows, void *x, dora_stream_t stream);

/*
 * dora_compose_fwd that also keeps v = base + s lora in the 8-bit form
 * (block_rows = 1) for dora_compose_bwd_q8, in the same pass.  y is bitwise
 * what dora_compose_fwd writes; v is rounded to fp32 after the product and
 * after the sum, then stored as dora_q8_store would store it.
 *   q, scale  uint8 [T, out] and [T, ceil(out / 128)]  out
 *   the rest as dora_compose_fwd
 */
dora_status dora_compose_fwd_q8(dora_dtype act, const void *base, const void *lora,
                                const float *g, float s, int64_t T, int64_t out,
                                void *y, void *q, void *scale, dora_stream_t stream);

/* Bytes of workspace dora_compose_bwd_q8 needs (as dora_compose_bwd_workspace). */
size_t dora_compose_bwd_q8_workspace(int64_t T, int64_t out);

/*
 * dora_compose_bwd from the kept v: d_base = g*dy, d_lora = s*g*dy (bitwise
 * dora_compose_bwd's), d_mag[j] = (sum_t dy[t,j] v[t,j]) / norm[j] with the
 * 8-bit v, in fp32 and a fixed order.  base and lora are not read.
 *   q, scale  uint8 [T, out] and [T, ceil(out / 128)] (dora_compose_fwd_q8)
 *   the rest as dora_compose_bwd
 */
dora_status dora_compose_bwd_q8(dora_dtype act, const void *grad_out, const void *q, const void *scale,
                                const float *g, const float *norm, float s, int64_t T, int64_t out,
                                void *d_base, void *d_lora, float *d_mag,
                                void *workspace, size_t workspace_bytes, dora_stream_t stream);

/* Bytes of workspace dora_lora_grad_q8 needs (host arithmetic; 0 for an invalid
 * shape): fp32 parts of the tiles of dA that several CTAs work on, at most 512
 * parts of 128 features by up to 192 columns (50 MB; 1024 up to 32 columns). */
size_t dora_lora_grad_q8_workspace(int64_t T, int64_t in, int64_t r);

/*
 * dA = dxa^T x: the gradient of the lora down-projection xa = x A^T from the
 * 8-bit x kept by the forward; fp32 accumulation and result.
 *   dxa    bf16 [T, r]   xq uint8 [T, in]   (16-byte aligned, r % 8 == 0, in % 16 == 0)
 *   xscale uint8 [T, ceil(in / 128)]
 *   dA     float32 [r, in]  16-byte aligned, overwritten
 *   workspace  >= dora_lora_grad_q8_workspace(T, in, r) bytes, 256-byte aligned
 *   Sizes: T, in >= 0 (in == 0 is a no-op, T == 0 writes zeros) and below
 *   2^31 - 1023, 1 <= r <= 1024.
 * x's values are exact in bf16, so every product is; sums are fp32, in chains
 * of at most 512 tokens that are added up with ordinary rounding.  One launch,
 * and one that joins the parts of tiles of dA that several CTAs worked on.
 */
dora_status dora_lora_grad_q8(const void *dxa, const void *xq, const void *xscale,
                              int64_t T, int64_t in, int64_t r, float *dA,
                              void *workspace, size_t workspace_bytes, dora_stream_t stream);

/* Bytes of workspace dora_matmul_q8 and dora_matmul_q8_t need: none at any size
 * (the parts of a tile meet on chip); the pointer may be NULL. */
size_t dora_matmul_q8_workspace(int64_t T, int64_t out, int64_t in);
size_t dora_matmul_q8_t_workspace(int64_t T, int64_t out, int64_t in);

/*
 * y = x W^T for x and the frozen W both in 8 bits (the base product of the
 * layer); fp32 accumulation, y rounded once to bf16.
 *   xq  uint8 [T, in]     xscale  uint8 [T, ceil(in / 128)]
 *   wq  uint8 [out, in]   wscale  uint8 [ceil(out / 128), ceil(in / 128)]  (block_rows = 128)
 *   y   bf16 [T, out];  xq, wq and y 16-byte aligned, out % 16 == 0, in % 16 == 0
 *   workspace  not used (dora_matmul_q8_workspace)
 *   Sizes: T, out >= 0 (either 0 is a no-op), in >= 1, below 2^31 - 1023.
 * The tensor core multiplies E4M3 by E4M3 and applies both scales (block-scaled
 * tcgen05.mma); one launch.  Up to 128 tokens the k range is split over a
 * cluster of up to 8 CTAs and summed in rank order, above that CTA pairs take
 * 256 features x 64 to 256 tokens.  The launch is a programmatic dependent one: its set-up
 * overlaps the launch before it, and it reads and writes nothing of the
 * caller's before that has completed.
 */
dora_status dora_matmul_q8(const void *xq, const void *xscale, const void *wq, const void *wscale,
                           int64_t T, int64_t out, int64_t in, void *y,
                           void *workspace, size_t workspace_bytes, dora_stream_t stream);

/*
 * dx = dy W for the same stored W (no transposed copy) and a dy in 8 bits
 * (block_rows = 1): dyq [T, out], dyscale [T, ceil(out / 128)], dx bf16 [T, in].
 * Alignment and errors as dora_matmul_q8.
 *   Sizes: T, in >= 0 (either 0 is a no-op), out >= 1.
 */
dora_status dora_matmul_q8_t(const void *dyq, const void *dyscale, const void *wq, const void *wscale,
                             int64_t T, int64_t out, int64_t in, void *dx,
                             void *workspace, size_t workspace_bytes, dora_stream_t stream);

/* ------------------------------------------------------------------------ */
/* (f) a frozen weight in 4 bits                                             */
/* ------------------------------------------------------------------------ */

/*
 * The 4-bit form of a matrix [rows, cols], cols a multiple of 32: q, one E2M1
 * value per element (0, .5, 1, 1.5, 2, 3, 4, 6 and a sign bit), two a byte with
 * the even column in the low half [rows, cols / 2], and scale, one byte b per 32
 * columns of a row, standing for 2^(b - 127) [rows, cols / 32].  An element's
 * value is E2M1(q) 2^(b - 127), b from 0 to 254; b = 255 makes its group NaN.
 * This is the layout of a microscaling (MX) FP4 matrix stored row by row.
 *
 * The scale that a store gives a group is the smallest power of two that brings
 * its largest magnitude to at most 6, and at least 2^-125: every value is then
 * exact in bf16, and rounding (nearest even) happens once, in E2M1.  E2M1 has no
 * NaN: a group that holds a NaN or an infinity is stored as zeros with b = 255.
 * A stack of matrices of one width is stored as one matrix of all their rows.
 */

/*
 * x into the 4-bit form, one pass.
 *   act    DORA_F32 or DORA_BF16: dtype of x
 *   x      [rows, cols] of `act`, 16-byte aligned
 *   q      uint8 [rows, cols / 2]  out, 16-byte aligned
 *   scale  uint8 [rows, cols / 32]  out
 *   Sizes: rows, cols >= 0 (either 0 is a no-op), < 2^31, cols % 32 == 0.
 */
dora_status dora_q4_store(dora_dtype act, const void *x, int64_t rows, int64_t cols,
                          void *q, void *scale, dora_stream_t stream);

/* The values of a 4-bit form: x[i,j] = E2M1(q[i,j]) 2^(b - 127), one pass; exact in
 * either `act`, but infinite from 2^128 on (b = 253 and 254).  Arguments and sizes
 * as dora_q4_store (x is written). */
dora_status dora_q4_load(dora_dtype act, const void *q, const void *scale, int64_t rows, int64_t cols,
                         void *x, dora_stream_t stream);

/* Bytes of workspace dora_matmul_q4 and dora_matmul_q4_t need, by the sizes alone: for
 * x W^T of 9 to 32 tokens (of 5 to 16 an expert: T / experts, rounded up; where in is no
 * multiple of 128, to 16 and to 8) 2 T in + 8 T ceil(in / 128), for x in pieces; for others, where k is cut in parts to fill the device, 4 T out (dy W:
 * 4 T in) a part; else 0, and the pointer may be NULL.  Nothing in it is kept from one
 * call to the next; calls that run at once need one each. */
size_t dora_matmul_q4_workspace(int64_t T, int64_t out, int64_t in, int64_t experts);
size_t dora_matmul_q4_t_workspace(int64_t T, int64_t out, int64_t in, int64_t experts);

/*
 * y = x W^T for a bf16 x and a frozen W in 4 bits; fp32 accumulation, y rounded
 * once to bf16.  With experts, W is a stack of them, the rows of x are sorted by
 * expert, and rows offsets[e] to offsets[e + 1] meet W[e]; rows of y that no
 * expert has are left as they were.
 *   x        bf16 [T, in]     y  bf16 [T, out]
 *   offsets  int32 [experts + 1] on the device (dora_expert_sort), not falling; or
 *            NULL with experts == 1: all rows.  Values are clamped to 0 .. T.
 *   wq       uint8 [experts, out, in / 2]   wscale  uint8 [experts, out, in / 32]
 *   x, wq, wscale and y 16-byte aligned, in % 32 == 0, out % 16 == 0
 *   workspace  dora_matmul_q4_workspace bytes, 256-byte aligned
 *   Sizes: T, out >= 0 (either 0 is a no-op), in >= 1, below 2^31 - 1023,
 *   1 <= experts <= 4096.
 * Both operands enter as they are, infinities and the smallest numbers too, however many
 * tokens there are; a result below 2^-126 may be flushed to zero.  A value of W from 2^128
 * on (b = 253 and 254) is infinite where W enters as bf16: in dy W, and in x W^T of more
 * tokens than x enters in pieces for.  Parts are summed in a fixed order: the same call
 * gives the same bits.  Of few tokens x enters as 8-bit
 * pieces, up to four; where those do not hold 32 neighbouring values (an infinity, values
 * more than 2^36 apart), the call is slower.
 * One launch, or two where there is a workspace.  They are programmatic dependent ones:
 * their set-up overlaps the launch before them, and they read (but for lines of W asked
 * into L2) and write nothing of the caller's before that has completed.
 */
dora_status dora_matmul_q4(const void *x, const int32_t *offsets, const void *wq, const void *wscale,
                           int64_t T, int64_t out, int64_t in, int64_t experts, void *y,
                           void *workspace, size_t workspace_bytes, dora_stream_t stream);

/*
 * dx = dy W for the same stored W (no transposed copy): dy bf16 [T, out], dx bf16
 * [T, in].  The rest as dora_matmul_q4.
 *   Sizes: T, in >= 0 (either 0 is a no-op), out >= 1.
 */
dora_status dora_matmul_q4_t(const void *dy, const int32_t *offsets, const void *wq, const void *wscale,
                             int64_t T, int64_t out, int64_t in, int64_t experts, void *dx,
                             void *workspace, size_t workspace_bytes, dora_stream_t stream);

/* ------------------------------------------------------------------------ */
/* (g) tokens sorted by expert and back                                      */
/* ------------------------------------------------------------------------ */

/*
 * The T * k entries of expert [T, k] (entry i = t * k + j) sorted by expert, stably:
 *   order    int32 [T * k]       the entry at each sorted row
 *   inverse  int32 [T, k]        the sorted row of each entry
 *   offsets  int32 [experts + 1] the rows of expert e are offsets[e] to offsets[e + 1]
 * An entry outside [0, experts) goes to no expert: its row comes at or behind
 * offsets[experts], after all that do.  An expert may be named twice by a token.
 *   index_bytes  4 or 8: expert is int32 or int64
 *   Sizes: T >= 0, k >= 1, T * k < 2^31 - 1024, 1 <= experts <= 4096.
 */
dora_status dora_expert_sort(int index_bytes, const void *expert, int64_t T, int64_t k, int64_t experts,
                             int32_t *order, int32_t *inverse, int32_t *offsets, dora_stream_t stream);

/*
 * xs[inverse[t,j]] = x[t] for every entry that has an expert: the tokens' rows sorted
 * by expert.  The other rows of xs are left as they were.  Its gradient is
 * dora_expert_return without weights.
 *   act  DORA_F32 or DORA_BF16: dtype of x [T, cols] and xs [T * k, cols]
 *   inverse, offsets  of dora_expert_sort.  An entry of inverse is a row of xs where
 *        it lies in 0 .. min(offsets[experts], T * k), else it has no expert.
 *   Sizes: T, cols >= 0 (either 0 is a no-op), cols < 2^31; the rest as dora_expert_sort.
 *   Any element alignment; 128-bit accesses where rows are whole 16-byte pieces.
 */
dora_status dora_expert_send(dora_dtype act, const void *x, const int32_t *inverse, const int32_t *offsets,
                             int64_t T, int64_t k, int64_t cols, int64_t experts, void *xs,
                             dora_stream_t stream);

/*
 * y[t] = sum_j weight[t,j] ys[inverse[t,j]] over the entries that have an expert, in
 * fp32 and in the order of j, rounded once; 0 where none has.
 *   ys  [T * k, cols] and y [T, cols] of `act`;  weight  float32 [T, k], or NULL:
 *   every one 1.  The rest as dora_expert_send.
 */
dora_status dora_expert_return(dora_dtype act, const void *ys, const int32_t *inverse, const int32_t *offsets,
                               const float *weight, int64_t T, int64_t k, int64_t cols, int64_t experts,
                               void *y, dora_stream_t stream);

/*
 * The gradient of dora_expert_return: d_ys[inverse[t,j]] = weight[t,j] dy[t] and
 * d_weight[t,j] = <dy[t], ys[inverse[t,j]]> (fp32, fixed order; 0 for an entry that has
 * no expert).  Rows of d_ys that no expert has are left as they were.
 *   dy [T, cols], ys and d_ys [T * k, cols] of `act`;  weight, d_weight  float32 [T, k]
 */
dora_status dora_expert_return_bwd(dora_dtype act, const void *dy, const void *ys, const int32_t *inverse,
                                   const int32_t *offsets, const float *weight, int64_t T, int64_t k,
                                   int64_t cols, int64_t experts, void *d_ys, float *d_weight,
                                   dora_stream_t stream);

/*
 * Zeros in the rows of x [rows, cols] (of `act`) that no expert has: those before
 * offsets[0] and from offsets[experts] on, for callers who read them.
 *   Sizes: rows >= 0 (0 is a no-op), below 2^31 - 1024; the rest as dora_expert_send.
 */
dora_status dora_expert_clear(dora_dtype act, void *x, const int32_t *offsets, int64_t rows, int64_t cols,
                              int64_t experts, dora_stream_t stream);

/* ------------------------------------------------------------------------ */
/* diagnostics                                                               */
/* ------------------------------------------------------------------------ */

/*
 * Reads (synchronously: waits for the device) and clears the current device's
 * error word.  *code = 0 when no kernel gave up waiting; otherwise a nonzero
 * code naming the wait that timed out.  Returns DORA_ERR_DEVICE in that case.
 */
dora_status dora_device_error(int *code);

/* Number of kernels this process has launched through the library. */
uint64_t dora_kernel_launches(void);

/*
 * Testing hook for the failure path; no counterpart in the paper.  With on != 0
 * the tensor-core kernels of later dora_norm_factored, dora_norm_factored_bwd,
 * dora_compose_lora_fwd, dora_linear_fwd, dora_lora_grad_q8, dora_matmul_q8,
 * dora_matmul_q8_t, dora_matmul_q4 and dora_matmul_q4_t calls on the current device
 * withhold all their operand loads, so their bounded waits expire after
 * wait_limit_ns (0 = the default of 2 s): the kernels then record a code in the
 * device error word (see dora_device_error), free their tensor memory and
 * exit, leaving the context usable; their outputs are garbage.
 * on = 0 restores normal operation.  Synchronises the device.
 */
dora_status dora_test_stall_loads(int on, uint64_t wait_limit_ns);

/*
 * Testing hook; no counterpart in the paper.  With allow = 0, later
 * dora_compose_lora_fwd and dora_linear_fwd calls run their fused kernel as
 * single CTAs (128 x 256 tiles), as on a device that cannot hold clusters of
 * two; allow != 0 (the default) restores CTA pairs where the device has them.
 * Process-wide; never fails.
 */
dora_status dora_test_fused_pairs(int allow);

#ifdef __cplusplus
}
#endif

#endif /* DORA_H */
