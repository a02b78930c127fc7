/*
 * wq4 — W4A16 mixed-input GEMM for NVIDIA GB300 (sm_103a), C ABI.
 *
 * Computes Y[M,N] = X[M,K] . dequant(Wq)[N,K]^T with X, the scales and Y in bf16 or fp16,
 * 4-bit weight codes, one scale (and zero point) per group of G consecutive K elements (G = 128
 * by default; or no scales) and fp32 accumulation.
 *
 * The problem statement follows "aphrodite-engine/kernels/quantization/machete/
 * machete_mainloop.cuh": its header comment (weights prepacked once, then Y = mm(X, B_prepacked);
 * the product computed as the transpose Y^t = W^t X^t so the narrow type is the MMA's A side),
 * get_conversion_mode (scale-only and scale-with-zero modes), Arguments (pointers, strides, group
 * size, zero pointer) and can_implement (the argument rules reproduced under "Errors" below).
 * The grouped variant follows "sm90_gemm_array_tma_warpspecialized_cooperative.hpp" (one GEMM per
 * group index L, all in one persistent launch).
 *
 * Conventions for every entry point:
 *  - Pointers named X, Wq, scales, zeros, Wp, Y and workspace are DEVICE pointers. Arrays of
 *    shapes and of per-problem pointers in the grouped call are HOST arrays.
 *  - The caller owns every buffer. The library allocates no device memory.
 *  - Calls that take a stream are asynchronous on it; NULL means the legacy default stream.
 *  - Arguments are checked before anything is launched; on a negative status nothing was
 *    launched and no buffer was touched.
 *  - dtype: WQ4_BF16 or WQ4_FP16; X, the scales and Y share it. qtype: WQ4_U4B8 (value =
 *    (code - 8) s), WQ4_U4_ZP (value = (code - z) s with a 4-bit zero point per group and row) or
 *    WQ4_U4_FZP (value = code s + zf with a float zero of the dtype per group and row, added after
 *    the scale: the scale-with-zero conversion of "machete_mainloop.cuh", transform_A_kblock;
 *    not with device-resident shapes or pointers).
 *  - group_size G: 64, or a multiple of 128 that divides K (G == K: one scale per row,
 *    channel-wise; "machete_mainloop.cuh", can_implement and load); other sizes give
 *    WQ4_ERR_UNSUPPORTED. N and K multiples of 128; M >= 0. The G passed to the GEMM calls must
 *    be the one the weight was prepacked with (the blob holds one scale set per 128-K record,
 *    two with G = 64).
 */
#ifndef WQ4_H_
#define WQ4_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st* wq4_stream_t;

enum {
    WQ4_OK = 0,
    WQ4_ERR_INVALID = -1,      /* bad shape, null pointer, zero pointer given/missing, bad enum */
    WQ4_ERR_ALIGN = -2,        /* a pointer is not 16-byte aligned (TMA rule) */
    WQ4_ERR_UNSUPPORTED = -3,  /* valid for the method, not built here (a group size that is not a
                                  multiple of 128 dividing K, N or K not multiples of 128, ...) */
    WQ4_ERR_WORKSPACE = -4,    /* workspace missing or smaller than the *_workspace_bytes answer */
    WQ4_ERR_CUDA = -5,         /* a CUDA runtime call failed (no device, launch failure, ...) */
    WQ4_ERR_TIMEOUT = -6,      /* a kernel's bounded pipeline wait ran out (see wq4_get_last_error) */
    WQ4_ERR_BOUNDS = -7        /* debug build only: a kernel's bounds check failed (wq4_last_violation) */
};
enum { WQ4_BF16 = 0, WQ4_FP16 = 1,
       WQ4_FP32 = 2 };             /* only where a call says so (wq4_block_mm, wq4_token_logprobs) */
enum { WQ4_U4B8 = 0, WQ4_U4_ZP = 1, WQ4_U4_FZP = 2 };

/* Library version (major * 10000 + minor * 100 + patch) and a text for a status code. */
int wq4_version(void);
const char* wq4_status_string(int status);

/* ------------------------------------------------------------------------------------------ *
 * Prepack ("machete_mainloop.cuh", header comment: weights reordered once into the layout the
 * mainloop consumes, so each thread fetches several MMAs' worth with one 128-bit load).
 * ------------------------------------------------------------------------------------------ */

/* Bytes of the prepacked blob for an N x K weight (256-byte header + one record per
 * 128-row x 128-K tile). Returns 0 if the shape is not supported. */
size_t wq4_prepacked_bytes(int N, int K, int group_size, int qtype);

/* Reorders a weight into the prepacked blob.
 *   Wq      [N][K/8] uint32, code of element k = 8j+i in bits [4i, 4i+4) of word j.
 *   scales  [K/G][N] dtype, N contiguous (one scale per group and row); NULL for a weight
 *           without scales (WQ4_U4B8 only: the value is code - 8, the direct conversion of
 *           "machete_mainloop.cuh", get_conversion_mode), stored as 1.0.
 *   zeros   WQ4_U4_ZP: [K/G][N/8] uint32, zero point of row n = 8j+i in bits [4i, 4i+4) of
 *           word j. WQ4_U4_FZP: [K/G][N] dtype, the float zero of each (group, row), N
 *           contiguous like the scales. Required for both (with scales); NULL for WQ4_U4B8.
 *   Wp_out  wq4_prepacked_bytes(...) bytes, 16-byte aligned; fully overwritten.
 * Integer work: the blob is a bit-exact permutation of the inputs. */
int wq4_prepack(const uint32_t* Wq, const void* scales, const void* zeros,
                int N, int K, int group_size, int dtype, int qtype,
                void* Wp_out, wq4_stream_t stream);

/* Exact inverse of wq4_prepack (a test and export aid), with the same G: group j of scales_out
 * [K/G][N] and zeros_out (wq4_prepack's zeros layout for the qtype) is read from its first 128-K
 * record. zeros_out must be NULL for U4B8; scales_out may be NULL (not written). */
int wq4_unprepack(const void* Wp, int N, int K, int group_size, int dtype, int qtype,
                  uint32_t* Wq_out, void* scales_out, void* zeros_out, wq4_stream_t stream);

/* ------------------------------------------------------------------------------------------ *
 * GEMM ("machete_mainloop.cuh": transform_A_kblock defines the dequantised value (code - zero)
 * times the group's scale; mma/load define one scale row per group of K).
 * ------------------------------------------------------------------------------------------ */

/* Workspace bytes wq4_mm needs on the current device for this shape (partial sums of K-split
 * tiles and their arrival counters) under the current options; 0 when the call takes the
 * decode kernel (at most 32 tokens, where that kernel applies: WQ4_OPT_DECODE), which uses none
 * (workspace may then be NULL). The workspace must be
 * zero-filled once when allocated; every completed call leaves its counters at zero again.
 * Calls that may overlap on the GPU need separate workspaces. */
int wq4_workspace_bytes(int M, int N, int K, int group_size, size_t* bytes);

/* wq4_workspace_bytes for a given qtype. WQ4_U4_FZP on the tensor-core path (not the decode
 * kernel) adds a table of activation sums that a pre-pass writes on the stream before the GEMM
 * (per token and zero group of 128 K, or 64 with G = 64, split into a high and a low 16-bit
 * part): (M rounded up to the token tile) x 2 x (zero groups rounded up to 64) x 2 bytes after the
 * plan's own bytes (256-byte aligned). For the other qtypes the answer equals wq4_workspace_bytes. */
int wq4_workspace_bytes_ex(int M, int N, int K, int group_size, int qtype, size_t* bytes);

/* Y = X . dequant(Wp)^T.
 *   X   [M][K] dtype row-major, 16-byte aligned.
 *   Wp  blob from wq4_prepack with the same N, K, group_size, dtype and qtype.
 *   Y   [M][N] dtype row-major, fully overwritten (fp32 sums rounded to nearest even).
 *   workspace / workspace_bytes: see wq4_workspace_bytes.
 * M == 0 is a no-op. Results are identical from run to run (fixed reduction order). */
int wq4_mm(const void* X, const void* Wp, void* Y, int M, int N, int K, int group_size,
           int dtype, int qtype, void* workspace, size_t workspace_bytes, wq4_stream_t stream);

/* Y = alpha * (X . dequant(W)^T) + beta * C + bias, the epilogue with a source operand of the
 * pages' kernels ("sm90_gemm_array_tma_warpspecialized_cooperative.hpp": the epilogue loads C
 * and combines it with alpha and beta) plus a bias per output column:
 *   C     [M][N] dtype, row-major, 16-byte aligned; read only when beta != 0 (may then be NULL
 *         only if beta == 0); C may be Y itself (in place: every element is read, then written,
 *         by the same thread).
 *   bias  [N] dtype, 16-byte aligned, or NULL.
 * Computed in fp32 (alpha * acc, then + beta * C, then + bias) and rounded to dtype once.
 * Everything else as wq4_mm (same workspace rule, same plans). */
int wq4_mm_ex(const void* X, const void* Wp, void* Y, int M, int N, int K, int group_size,
              int dtype, int qtype, float alpha, const void* C, float beta, const void* bias,
              void* workspace, size_t workspace_bytes, wq4_stream_t stream);

/* Workspace bytes for wq4_grouped_mm with these P problems (host arrays of shapes); the same
 * zero-fill rule as wq4_workspace_bytes. */
int wq4_grouped_workspace_bytes(int P, const int* M, const int* N, const int* K, int group_size,
                                size_t* bytes);

/* The same for a weight format: float zeros (WQ4_U4_FZP) add the activation-sum tables of the
 * problems' zero steps (see wq4_workspace_bytes_ex); other formats as wq4_grouped_workspace_bytes. */
int wq4_grouped_workspace_bytes_ex(int P, const int* M, const int* N, const int* K, int group_size,
                                   int qtype, size_t* bytes);

/* P independent problems Y_p = X_p . dequant(Wp_p)^T in one launch (P <= 64).
 *   M, N, K            host arrays of P shapes; M[p] == 0 skips problem p (its pointers are
 *                      not dereferenced and may be NULL).
 *   X, Wp, Y           host arrays of P device pointers, per-problem layouts as in wq4_mm.
 * All problems share group_size, dtype and qtype. When every non-empty problem has at most 32
 * tokens (decode-sized experts), the problems' row blocks go through the decode kernel in one
 * launch, as wq4_mm does for one problem: no workspace (the workspace queries answer 0). */
int wq4_grouped_mm(int P, const int* M, const int* N, const int* K,
                   const void* const* X, const void* const* Wp, void* const* Y,
                   int group_size, int dtype, int qtype,
                   void* workspace, size_t workspace_bytes, wq4_stream_t stream);

/* Same computation as wq4_mm, for callers that cannot allocate device memory or hand the
 * library a buffer: code that must not call cudaMalloc (for instance inside a section where
 * allocation would stall or break a stream capture, or a plugin whose host runtime owns every
 * device allocation). There is no counterpart in the pages: it only changes where the K-split
 * scratch lives. Instead of a caller workspace it uses one fixed 24 MiB array in the library's
 * device memory (every GPU that loads the library holds it until the process exits).
 * Plans: calls that wq4_mm sends to the decode kernel go there too (no scratch). A GEMM plan
 * whose K-split scratch fits the array is wq4_mm's own; one that would need more (for example
 * 4096 tokens x N = 4096, whose 192-token tiles need 30 MB) keeps every tile whole instead.
 * Results: bit-identical to wq4_mm's under the same options when the plan is wq4_mm's; with
 * tiles kept whole, the same fp32 sums added in another order (equal within rounding, not bit
 * for bit). WQ4_ERR_WORKSPACE only when an option forces a split (WQ4_OPT_GRID,
 * WQ4_OPT_SPLIT_ALL) whose scratch exceeds the array.
 * It allocates nothing: no cudaMalloc, no cudaFree, no allocating library call. The first call
 * on a device looks up the array's device address (cudaGetSymbolAddress) with that device
 * current, whatever the shape; make that first call before any stream capture. The array is
 * shared by all calls on a device and keeps the last call's contents; each call that uses it
 * clears the part that must start at zero (an async memset on `stream`). Calls that overlap on
 * the GPU (other streams, or concurrently running graphs) race on the array and must be
 * serialised by the caller. Arguments and errors as wq4_mm. */
int wq4_mm_static_scratch(const void* X, const void* Wp, void* Y, int M, int N, int K, int group_size,
                          int dtype, int qtype, wq4_stream_t stream);

/* Grouped GEMM whose token counts are known only on the device (tokens routed to experts by a
 * kernel on the same stream): the grouped call of "sm90_gemm_array_tma_warpspecialized_cooperative.hpp"
 * with its problem shapes in device memory.
 *   M_dev   DEVICE array of P int token counts, read when the work starts (stream order);
 *           each is clamped to [0, M_cap[p]].
 *   M_cap   HOST array: rows that X[p] and Y[p] hold (the capacity of each problem's buffers).
 *   N, K, X, Wp, Y, group_size, dtype, qtype as in wq4_grouped_mm; X[p] is [M_cap[p]][K[p]] and
 *           only its first M_dev[p] rows matter; rows of Y[p] beyond M_dev[p] are not written.
 *   workspace  wq4_grouped_device_m_workspace_bytes(P) bytes, 16-byte aligned (the tile table
 *           a set-up kernel writes before the GEMM); no zero fill needed.
 * The plan (token tile, grid) is made for the capacities, with every tile whole. */
int wq4_grouped_device_m_workspace_bytes(int P, size_t* bytes);
int wq4_grouped_mm_device_m(int P, const int* M_dev, const int* M_cap, const int* N, const int* K,
                            const void* const* X, const void* const* Wp, void* const* Y,
                            int group_size, int dtype, int qtype,
                            void* workspace, size_t workspace_bytes, wq4_stream_t stream);

/* Grouped GEMM whose per-problem pointers live in device memory (written by a kernel on the same
 * stream, for example the expert buffers of a token router): the grouped call of
 * "sm90_gemm_array_tma_warpspecialized_cooperative.hpp" with its pointer arrays in device memory
 * and any number of problems up to 4096.
 *   M, N, K   HOST arrays of P shapes (the plan needs them); M[p] == 0 skips problem p (its
 *             pointers are not read).
 *   X_dev, Wp_dev, Y_dev   DEVICE arrays of P device pointers (8-byte aligned arrays), read when
 *             the work starts (stream order); per-problem layouts as in wq4_mm.
 *   group_size, dtype, qtype   shared by every problem; float zeros (WQ4_U4_FZP) are not
 *             supported here (WQ4_ERR_UNSUPPORTED).
 *   workspace  wq4_grouped_dev_ptrs_workspace_bytes(...) bytes, 128-byte aligned, zero-filled
 *             before its first use (the K-split counters come first and are left at zero by
 *             every call that completes; the rest, the problem table and one 128-byte activation
 *             tensor map per problem, is rewritten by every call). Calls that share a workspace
 *             must be in stream order.
 * A set-up kernel on `stream` reads the pointers, checks each non-empty problem's pointers (non-null,
 * 16-byte aligned) and blob header, writes its descriptor and its activation tensor map (encoded
 * on the host for its shape, the X address replaced on the device); then the GEMM runs the
 * plan wq4_grouped_mm would make for these shapes, reading the problems from the table. A problem
 * that fails the device-side check is skipped (its Y is not written) and wq4_get_last_error then
 * reports WQ4_ERR_INVALID; the other problems are computed. Host-side argument errors as
 * wq4_grouped_mm, plus WQ4_ERR_ALIGN for a pointer array not 8-byte aligned or a workspace not
 * 128-byte aligned. Results are bit-identical to wq4_grouped_mm's for the same problems. */
int wq4_grouped_dev_ptrs_workspace_bytes(int P, const int* M, const int* N, const int* K, int group_size,
                                         size_t* bytes);
int wq4_grouped_mm_dev_ptrs(int P, const int* M, const int* N, const int* K,
                            const void* const* X_dev, const void* const* Wp_dev, void* const* Y_dev,
                            int group_size, int dtype, int qtype,
                            void* workspace, size_t workspace_bytes, wq4_stream_t stream);

/* ------------------------------------------------------------------------------------------ *
 * 8-bit rows: the projections of a model that stay in 8-bit float next to the 4-bit ones, what
 * feeds them and what reads the last one's answer.
 *
 * Quantised rows [T][D] are e4m3 codes Q, row t at Q + t ldq (ldq bytes, a multiple of 16), and one
 * fp32 scale per token and block of 128 columns, scales[b lds + t] (lds elements, a multiple of 4,
 * >= T): the value of element (t, d) is Q[t][d] scales[d / 128][t]. A last block of fewer than 128
 * columns has a scale of its own. Both pointers are 16-byte aligned. Padding (codes past D, scales
 * past T) is neither read nor written.
 *
 * A block's scale is max(max |y| / 448, 2^-126) and its codes are y / scale, the quotients in fp32 rounded
 * to nearest, the codes to nearest even (448 is the largest e4m3 value). A NaN becomes a NaN code and does not touch the scale; a block
 * with an infinity gets an infinite scale, and all its values read back as NaN.
 * ------------------------------------------------------------------------------------------ */

/* RMS norm with the residual's addition, into quantised rows:
 *     h = X + R        y = h / sqrt(mean(h^2) + eps) * weight        (fp32 throughout)
 *   X       [T][D] dtype (WQ4_BF16 or WQ4_FP16), row stride ldx elements.
 *   R       the residual, [T][D] dtype, row stride ldr; NULL: h = X.
 *   weight  [D] dtype.
 *   R_out   h rounded to dtype, the next layer's residual, row stride ldro, or NULL; needs R. May be X
 *           or R itself (same stride). The norm goes by the unrounded h.
 *   Y       y rounded to dtype (what wq4_mm reads), row stride ldy, or NULL. May be X or R itself (same
 *           stride) where R_out is not.
 *   Q, scales, ldq, lds   y as quantised rows, or both NULL; one of Y and Q at least is given.
 * eps is finite and >= 0. D <= 32768, any D >= 1; rows whose sizes, strides and pointers are multiples
 * of 16 bytes are read and written in 16-byte vectors. T == 0 is a no-op. */
int wq4_add_rmsnorm_quant(const void* X, long long ldx, const void* R, long long ldr, const void* weight, int T, int D,
                          float eps, int dtype, void* R_out, long long ldro, void* Y, long long ldy, void* Q,
                          long long ldq, float* scales, long long lds, wq4_stream_t stream);

/* Gated activation into quantised rows: y = silu(g) u with g = X[t][0..D), u = X[t][D..2D) and
 * silu(g) = g / (1 + exp(-g)), in fp32.
 *   X       [T][2 D] dtype (WQ4_BF16 or WQ4_FP16), row stride ldx elements.
 *   Q, scales, ldq, lds   quantised rows of D columns.
 * Any D >= 1 (up to 2^24). T == 0 is a no-op. */
int wq4_silu_mul_quant(const void* X, long long ldx, int T, int D, int dtype, void* Q, long long ldq, float* scales,
                       long long lds, wq4_stream_t stream);

/* Product of quantised rows with an 8-bit weight that has one scale per 128 x 128 block:
 *     Y[m][n] = sum over blocks b of x_scales[b][m] w_scales[n / 128][b] sum over k in b of X[m][k] W[n][k]
 * with fp32 accumulation, rounded once.
 *   X, x_scales   quantised rows [M][K] (ldx bytes, ldsx elements).
 *   W         [N][K] e4m3, row stride ldw bytes (a multiple of 16), 16-byte aligned: read as it is, there
 *             is nothing to prepack.
 *   w_scales  [ceil(N / 128)][ceil(K / 128)] fp32, row stride ldsw elements.
 *   Y         [M][N] dtype (WQ4_BF16, WQ4_FP16 or WQ4_FP32), row stride ldy elements.
 * Any M >= 0 and N >= 1; K a multiple of 16 (WQ4_ERR_UNSUPPORTED otherwise). Needs no workspace.
 * Results are identical from run to run (fixed reduction order). M == 0 is a no-op. */
int wq4_block_mm(const void* X, long long ldx, const float* x_scales, long long ldsx, const void* W, long long ldw,
                 const float* w_scales, long long ldsw, void* Y, long long ldy, int M, int N, int K, int dtype,
                 wq4_stream_t stream);

/* Log probabilities of given tokens, the entropy of each row's distribution and its most likely tokens,
 * from logits x (log p = x - log sum exp x), in fp32:
 *   logits        [T][V] dtype (WQ4_BF16, WQ4_FP16 or WQ4_FP32), row stride ld elements.
 *   tokens        [T] the token of each row whose log probability is asked for; one outside [0, V) gives
 *                 NaN. NULL, with logprobs, when there is none to ask for.
 *   logprobs      [T] log p of tokens[t], or NULL with tokens.
 *   entropy       [T] -sum p log p in nats, or NULL.
 *   top_ids, top_logprobs   [T][top_k] the top_k most likely tokens in order, the lower index first among
 *                 equal logits; both NULL with top_k == 0. top_k <= 32 and <= V.
 * Logits of -inf are tokens that cannot occur: log probability -inf, no part in the entropy, never listed;
 * a row with fewer than top_k others is filled up with id -1 and log probability -inf. A row of nothing
 * but -inf has log probabilities -inf and entropy 0. In a row that holds a NaN or +inf every log
 * probability and the entropy are NaN (ids still rank the values that are not NaN).
 * V <= 2^30. T == 0 is a no-op. */
int wq4_token_logprobs(const void* logits, long long ld, const long long* tokens, int T, int V, int dtype, int top_k,
                       float* logprobs, float* entropy, int* top_ids, float* top_logprobs, wq4_stream_t stream);

/* ------------------------------------------------------------------------------------------ *
 * Attention over a paged cache, for decoding with drafted tokens: what lies between a layer's projection to
 * queries, keys and values and its output projection, and what decides on the drafts.
 *
 * Sequences are ragged: sequence b's tokens of this step are rows starts[b] .. starts[b + 1] - 1 of every
 * per-token array. With drafts they form a tree: the first is the last token that is certain, every other one has
 * a parent among the ones before it. context[b] tokens of the sequence came before; the cache holds them
 * at places 0 .. context[b] - 1 of the sequence, and token i of this step at place context[b] + i.
 * ------------------------------------------------------------------------------------------ */

/* A paged cache of one layer: element (page, token of the page, head, feature) of the keys lies at
 * k + page k_page + token k_token + head k_head + feature, and so for the values; strides in elements of the
 * call's dtype. A slot is page * page_size + token of the page; pages * page_size < 2^31. */
typedef struct wq4_kv_cache {
    void *k, *v;
    long long k_page, k_token, k_head;
    long long v_page, v_token, v_head;
    int pages, page_size;
} wq4_kv_cache;

/* Queries, keys and values of T tokens, with a norm and a rotation on the way; keys and values go to their slots:
 *     x' = x / sqrt(mean(x^2) + eps) * weight                  (each head of q and k; fp32 throughout)
 *     (a, b) -> (a cos w - b sin w, b cos w + a sin w),  w = positions[t] inv_freq[i]
 * for the pairs i < rot_dim / 2 of features (i, i + rot_dim / 2), or (2 i, 2 i + 1) with interleaved = 1. The
 * angle is the exact product of position and frequency, however far the position is.
 *   Q, K, V   [T][q_heads or kv_heads][D] dtype (WQ4_BF16 or WQ4_FP16): element (t, h, d) at t ts + h hs + d; so
 *             views of one projection's rows will do. Rows do not overlap.
 *   q_weight, k_weight   [D] dtype; both NULL: no norm. With q_heads == 0 (keys and values only) q_weight is NULL.
 *   positions   [T] any 64-bit number, read with rot_dim > 0; inv_freq [rot_dim / 2] radians per position.
 *   Q_out     [T][q_heads][D] with strides of its own; may be Q itself (same strides).
 *   slots     [T]; a negative one: the token's key and value are not written (padding; its query is). One beyond
 *             the cache is not written either, and wq4_get_last_error reports WQ4_ERR_INVALID. Slots are
 *             distinct: of two tokens with the same slot either's elements may stay.
 * The rest of the cache is left as it is. D <= 1024, any D; multiples of 16 with 16-byte rows are fastest.
 * T == 0 is a no-op. */
int wq4_rope_append(const void* Q, long long q_ts, long long q_hs, const void* K, long long k_ts, long long k_hs,
                    const void* V, long long v_ts, long long v_hs, int T, int q_heads, int kv_heads, int D, int dtype,
                    const void* q_weight, const void* k_weight, float eps, const long long* positions,
                    const float* inv_freq, int rot_dim, int interleaved, void* Q_out, long long qo_ts, long long qo_hs,
                    const wq4_kv_cache* cache, const long long* slots, wq4_stream_t stream);

/* Attention of B sequences' tokens over their paged caches:
 *     out[t][h] = sum_j p_j V[j][h / (q_heads / kv_heads)],   p = softmax over j of scale q[t][h] . K[j][...]
 * over the places j of the sequence that the token sees: every place of its context and, among this
 * step's tokens, those its mask names, or without masks those before it and itself.
 *   Q, out    [T][q_heads][D] dtype, 16-byte aligned, strides multiples of 8 elements. q_heads is a multiple of
 *             kv_heads. out must not overlap Q.
 *   cache     this step's keys and values are in it (wq4_rope_append). k and v 16-byte aligned, strides multiples
 *             of 8; page_size a multiple of 16.
 *   page_table   [B][table_width] int, row stride ld_table: page i of sequence b holds its places from i page_size.
 *             Entries past a sequence's last place are not read. A sequence has at most 2^30 places. A table no wider
 *             than the longest sequence needs is soonest: its width is all that the choice of kernel knows of the lengths.
 *   starts    [B + 1] int, in DEVICE memory as page_table and context [B] int; 0 <= starts[b] <= starts[b + 1] <= T.
 *   max_tokens   the most tokens that one sequence has in this step.
 *   mask      [T][mask_words] 64-bit words: token i of a sequence sees token j of the same where bit j % 64 of
 *             word j / 64 is set (bits past its sequence's tokens count for nothing). mask_words >=
 *             ceil(max_tokens / 64). NULL: it sees tokens j <= i.
 *   lse       [T][q_heads] log of the sum of exp over the places seen, or NULL.
 * A token that sees nothing gets zeros and an lse of -inf. What lies in places that a token does not see, NaN and
 * infinities among it, does not reach its output. Rows of out and lse past starts[B] are left as they are.
 * Probabilities are rounded to dtype before they multiply the values (their sum is not); all sums are fp32.
 * (WQ4_FP16: those below 2^-27 of a row's largest to steps of 2^-37 of it.)
 * A page outside the cache, a table too narrow for a sequence, or starts that do not ascend within T and by at most
 * max_tokens give outputs that mean nothing, and wq4_get_last_error reports WQ4_ERR_INVALID; nothing
 * is read or written out of bounds.
 *   workspace   wq4_tree_attention_workspace_bytes(...) bytes on the current device, 16-byte aligned, zero-filled once
 *             when allocated (its first 4 bytes per SM have to be zero, the rest may hold anything); every completed
 *             call leaves it fit for the next. Calls that may overlap
 *             on the GPU need separate workspaces (two graphs captured with the same one as well).
 * D a multiple of 8, at most 256; max_tokens * q_heads / kv_heads at most 2^30 (WQ4_ERR_UNSUPPORTED otherwise). Results are identical from run to run for
 * the same lengths. B == 0 or T == 0 is a no-op. */
int wq4_tree_attention_workspace_bytes(int B, int max_tokens, int q_heads, int kv_heads, int D, size_t* bytes);
int wq4_tree_attention(const void* Q, long long q_ts, long long q_hs, const wq4_kv_cache* cache, const int* page_table,
                       int ld_table, int table_width, const int* starts, const int* context, int B, int T,
                       int max_tokens, int q_heads, int kv_heads, int D, int dtype, float scale,
                       const unsigned long long* mask, int mask_words, void* out, long long o_ts, long long o_hs,
                       float* lse, void* workspace, size_t workspace_bytes, wq4_stream_t stream);

/* Verification of drafted tokens: which of them the target model keeps, and the token that follows them, such that
 * what comes out is distributed as the target's own tokens are.
 * Row t of the logits answers token t. The walk through sequence b begins at its first token with p =
 * softmax(logits / temperature) of its row, and goes through the others j in order. Where j's parent is the node the
 * walk is at, j is tried: it is kept if uniforms[j] q(token_j) < p(token_j), and the walk goes on from j
 * with the p of its row; otherwise what the draft accounts for is taken from the target,
 * p = max(p - q, 0) / its sum (p stays where nothing is left). q is the node's row of draft_probs, the distribution that
 * each of its children was drawn from, independently and with replacement; without draft_probs a draft is certain: q = 1 at the token tried, 0 elsewhere. At the
 * end the next token is drawn from p: the first one at which the sum of p exceeds final_uniforms[b].
 *   logits    [T][V] dtype (WQ4_BF16, WQ4_FP16 or WQ4_FP32), row stride ld. -inf: a token that cannot occur.
 *   tokens    [T]; parents [T] int, the parent's place within the sequence (the first token's is not read); starts
 *             [B + 1] int as in wq4_tree_attention, all in DEVICE memory. A draft outside the vocabulary is
 *             not kept and takes nothing from p.
 *   draft_probs   [T][V] fp32, row stride ldp, or NULL.
 *   temperature   [B] fp32, 0: greedy (the whole of p at the row's first largest logit), or NULL: 1 everywhere.
 *   uniforms [T], final_uniforms [B]   random numbers of [0, 1).
 *   accepted  [B] int, the drafts kept; path [B][max(1, max_tokens - 1)] int, row stride ld_path: their places
 *             within the sequence in order, then -1; next_tokens [B].
 * The walk ends with next token -1 at a row that holds a NaN or +inf, or nothing but -inf, for a temperature that is
 * negative, NaN, infinite or so small that the scaled logits overflow, and for a sequence without tokens.
 * Probabilities are fp32, decisions are by sums over the vocabulary that are off by less than 2^-37 of them. Results are identical
 * from run to run; the sums' order hangs on B, V and the device, so that a sequence may go another way in another batch where a
 * random number lies as near to a border as that. starts that do not ascend within T and by at most max_tokens: as in wq4_tree_attention. V <= 400000. B == 0 is a no-op. */
int wq4_verify_drafts(const void* logits, long long ld, const long long* tokens, const int* parents, const int* starts,
                      int B, int T, int max_tokens, int V, int dtype, const float* draft_probs, long long ldp,
                      const float* temperature, const float* uniforms, const float* final_uniforms, int* accepted,
                      int* path, int ld_path, long long* next_tokens, wq4_stream_t stream);

/* ------------------------------------------------------------------------------------------ *
 * Errors and options.
 * ------------------------------------------------------------------------------------------ */

/* Synchronises the stream, then reports (and clears) what any wq4 kernel on the current device
 * recorded in the device status word: a failed bounds check of the debug build (WQ4_ERR_BOUNDS),
 * else a blob header that did not match its call or an index in device memory outside what it
 * indexes (WQ4_ERR_INVALID), else a pipeline timeout
 * (WQ4_ERR_TIMEOUT), else a kernel whose shared memory did not lie as it needs (WQ4_ERR_CUDA: its outputs are
 * undefined); with nothing recorded, a pending CUDA error (WQ4_ERR_CUDA), else WQ4_OK. A
 * call whose waits ran out stops early and leaves its outputs undefined; the context stays
 * usable, but a workspace it used must be zero-filled again before the next call (its split
 * counters may be left non-zero). The status word is shared by every stream on the device and is
 * read, then cleared: a kernel still running on another stream may record between the two, and
 * that record is lost, so call it while no other wq4 work is in flight to see everything. */
int wq4_get_last_error(wq4_stream_t stream);

/* Bounds checks: 1 when this library is the debug build (libwq4_debug.so, compiled with
 * WQ4_DEBUG=1), 0 for the release build, whose kernels carry no checks. The debug build's
 * kernels check, before each use, every tiled tensor copy's innermost coordinate (a 16-byte
 * multiple, the box inside the tensor), every weight record's range inside its blob, every
 * scheduled tile against its problem's M, N and K groups, the K-split workspace slots and
 * counters, and every output column against N. A failed check never faults or waits: the copy
 * reads the tensor's origin (or the blob's first record) instead, a store or workspace access is
 * skipped, the CTA stops at its next pipeline wait, and wq4_get_last_error reports
 * WQ4_ERR_BOUNDS; the call's outputs are then undefined. Slots, pages, lengths and tokens that the attention
 * operators read from device memory are checked in both builds (WQ4_ERR_INVALID). */
int wq4_debug_checks(void);

/* The first violation that the last WQ4_ERR_BOUNDS report read back: record[0] = the check site
 * (1 tile, 2 activation tile copy, 3 activation sums, 4 weight record, 5 epilogue C copy,
 * 6 K-split partial slot, 7 K-split counter, 8 output column, 9 decode weight stage, 10 decode
 * activation piece, 11 problem index, 12 block-scaled product operand copy, 13 block-scaled product
 * output), record[1..3] = the offending coordinate or index, then two
 * values whose meaning depends on the site (listed with the sites in csrc/wq4_check.h). record
 * must hold 4 ints. Returns 1 and clears the saved violation if there was one, 0 (record zeroed)
 * otherwise, WQ4_ERR_INVALID for a null record. */
int wq4_last_violation(int* record);

/* Process-wide tuning and test options (not thread-safe; set before launching):
 *   WQ4_OPT_TOKEN_TILE      force the token tile (16, 64, 128, 160 or 192); 0 = automatic
 *   WQ4_OPT_GRID            force the number of persistent CTAs; 0 = automatic
 *   WQ4_OPT_SPLIT_ALL       1 = every tile goes through the K-split path (tests)
 *   WQ4_OPT_TIMEOUT_CYCLES  bound of every pipeline wait in SM clock cycles; 0 = default
 *   WQ4_OPT_TRACE           1 = print each dispatch decision to stderr
 *   WQ4_OPT_A_IN_SMEM       1 = stage the dequantised operand in shared memory instead of tensor
 *                           memory (both give the same result; for comparison)
 *   WQ4_OPT_CLUSTER         0 = automatic, -1 = never, 2..8 = force the cluster split: each tile's
 *                           K range split over a cluster of that many CTAs whose partial sums are
 *                           added through distributed shared memory
 *   WQ4_OPT_DECODE          0 = automatic, -1 = never, 1 = whenever the shape allows: wq4_mm with at
 *                           most 32 tokens uses a warp-level-MMA kernel that keeps whole weight rows
 *                           per CTA (no workspace)
 *   WQ4_OPT_PDL             0 = both kernels are launched with programmatic dependent launch (a
 *                           call's set-up overlaps the end of the previous kernel on the stream;
 *                           it touches global memory only after that kernel has completed);
 *                           -1 = plain stream order
 *   WQ4_OPT_TEST_STALL      1 = (tests of the failure path) the GEMM, decode and block-scaled
 *                           product and attention kernels make one wait per CTA on a barrier
 *                           that nothing arrives on, and wq4_token_logprobs one per row that a cluster of
 *                           CTAs shares; it runs out after the WQ4_OPT_TIMEOUT_CYCLES bound,
 *                           the call stops early and wq4_get_last_error reports
 *                           WQ4_ERR_TIMEOUT. Kernels without a bounded wait (norm, gated
 *                           activation, log probabilities of a row per CTA, prepack) are as
 *                           ever. 0 = off
 *   WQ4_OPT_CONST_WEIGHTS   1 = the caller promises that no kernel still pending on the stream
 *                           writes a blob that a later call reads: the decode kernel then checks
 *                           the blob header and copies its first weights, and the tensor-core GEMM
 *                           (problems given on the host) its first ring of weight records, before
 *                           the kernel ahead has completed (activations, C and outputs keep stream
 *                           order). Results are undefined if the promise is broken. 0 = stream
 *                           order for every operand (default)
 *   WQ4_OPT_DECODE_DEPTH    weight ring slots of the decode kernel (one slot = one 16-row block x
 *                           1024 K); 0 = automatic, 2..16 = forced
 *   WQ4_OPT_DECODE_TRIGGER  0 = the decode kernel lets the next kernel on the stream start once its
 *                           activations have landed (default), 1 = at once
 *   WQ4_OPT_VERIFY_DEV_PTRS 1 = (tests) wq4_grouped_mm_dev_ptrs stops after its set-up kernels: it
 *                           synchronises the stream, reads back the activation tensor maps they
 *                           patched and compares each byte for byte with the map the host encoder
 *                           makes for the same address and row count; WQ4_OK when every map
 *                           matches, WQ4_ERR_UNSUPPORTED otherwise (the differing bytes printed
 *                           under WQ4_OPT_TRACE). The GEMM is not launched. 0 = off
 * Returns WQ4_ERR_INVALID for an unknown key or value. */
enum {
    WQ4_OPT_TOKEN_TILE = 1,
    WQ4_OPT_GRID = 2,
    WQ4_OPT_SPLIT_ALL = 3,
    WQ4_OPT_TIMEOUT_CYCLES = 4,
    WQ4_OPT_TRACE = 5,
    WQ4_OPT_A_IN_SMEM = 6,
    WQ4_OPT_CLUSTER = 7,
    WQ4_OPT_DECODE = 8,
    WQ4_OPT_PDL = 9,
    WQ4_OPT_TEST_STALL = 10,
    WQ4_OPT_CONST_WEIGHTS = 11,
    WQ4_OPT_DECODE_DEPTH = 12,
    WQ4_OPT_DECODE_TRIGGER = 13,
    WQ4_OPT_VERIFY_DEV_PTRS = 14
};
int wq4_set_option(int key, long long value);
long long wq4_get_option(int key);

#ifdef __cplusplus
}
#endif
#endif /* WQ4_H_ */
