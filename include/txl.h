/*
 * txl.h -- C ABI of libtxl.so: Transformer-XL relative multi-head attention over
 * [memory ++ current segment] on one NVIDIA GB300 (sm_103a).
 *
 * The operation (citations are page title and section):
 *   "跨窗口的相对位置编码" §3 and "Transformer-XL 和相对位置编码" §2.3.2 (terms (a)-(d)):
 *       A_ij = q_i.k_j + q_i.r_{i-j} + u.k_j + v.r_{i-j}
 *   "跨窗口的相对位置编码" §2, "Transformer-XL 和相对位置编码" §2.3.2:
 *       R_delta[2k] = sin(delta * 10000^(-2k/d_model)), R_delta[2k+1] = cos(same)
 *       r_delta = R_delta W_R                  (W_{k,R}; "TransformerXL 相对位置编码" §3.1 r_proj)
 *   "TransformerXL 相对位置编码" §2.4: distances beyond clamp_len count as clamp_len.
 *   "TransformerXL 相对位置编码" §4.2/§4.3: mask the summed score; keys span memory + current.
 *   "Transformer-XL 和相对位置编码" §2.3.1: K, V from [SG(memory) ∘ current], Q from current.
 *   "Transformer-XL架构解析" §1.1: the memory is a FIFO of mem_len positions.
 *
 * Conventions for every entry point:
 *  - Pointers named "device" are CUDA device addresses; the caller owns all memory.  The library
 *    never allocates, frees or synchronises.  Work is enqueued on `stream` (a cudaStream_t; NULL
 *    is the legacy default stream) on the calling thread's current device, and calls return as
 *    soon as it is enqueued.
 *  - Arguments are validated on the host before anything is launched; a non-TXL_OK status means
 *    nothing was enqueued (except TXL_ERR_CUDA, which reports a failed launch).
 *  - Element strides are in elements, not bytes.  The innermost index (d) is always contiguous.
 *  - No exceptions, no printing, no CPU fallback.
 */
#ifndef TXL_H
#define TXL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    TXL_OK = 0,
    TXL_ERR_INVALID_ARG = 1,   /* null pointer, non-positive size, inconsistent shapes       */
    TXL_ERR_UNSUPPORTED = 2,   /* valid request this build does not implement                 */
    TXL_ERR_ALIGNMENT = 3,     /* a base address or stride is not 16-byte aligned where needed */
    TXL_ERR_CUDA = 4,          /* a CUDA runtime/driver call failed                            */
    TXL_ERR_TIMEOUT = 5,       /* written to err_flag by a kernel whose bounded wait expired   */
    TXL_ERR_WORKSPACE = 6,     /* workspace missing or smaller than txl_rel_attn_workspace_size */
    TXL_ERR_PAGE = 7           /* written to a paged memory's err_flag: a position without a page */
} txl_status;

typedef enum { TXL_F32 = 0, TXL_BF16 = 1 } txl_dtype;

/* A [B][T][H][D] tensor in device memory: element (b,t,h,d) lives at
 * ptr + b*stride_b + t*stride_t + h*stride_h + d   (elements of the call's dtype). */
typedef struct {
    void* ptr;
    int64_t stride_b;
    int64_t stride_t;
    int64_t stride_h;
} txl_view;

/* K/V memory of M positions per batch entry ("Transformer-XL架构解析" §1.1: FIFO cache).
 * k and v are device [B][M][H][D] slot arrays with the strides below (shared by k and v).
 * Logical memory key j (0 <= j < M, j = M-1 newest) lives in physical slot (wp + j) mod M and
 * is valid iff j >= M - valid.  A freshly zeroed ring has wp = 0, valid = 0.  A plain
 * contiguous memory (oldest first) is described by wp = 0, valid = M.  M = 0 means no memory
 * (k, v may then be NULL). */
typedef struct {
    void* k;
    void* v;
    int64_t stride_b;
    int64_t stride_t;
    int64_t stride_h;
    int B, M, H, D;
    txl_dtype dtype;
    int wp;      /* next slot to write == slot of the oldest position once the ring is full */
    int valid;   /* number of valid positions, 0..M */
} txl_mem;

/* Human-readable name of a status code (static string). */
const char* txl_status_str(txl_status status);

/* Library ABI version (major*10000 + minor*100 + patch). */
int txl_version(void);

/*
 * txl_rel_pos_gen -- position key vectors of every distance the attention can see.
 *   r[delta][h][d] = sum_m R_delta[m] * W_R[m][h*d_head + d],  delta = 0 .. n_rows-1,
 * with R_delta the interleaved sinusoid above (fp32 angles, on chip; never stored).
 * Row index == distance.  For one attention call, n_rows = min(M+L, clamp_len+1).
 *   W_R : device [d_model][ld_w], dtype; columns 0 .. n_head*d_head-1 are used; no bias.
 *   r   : device [n_rows][n_head][ld_r], dtype; only d < d_head is written.
 * Limits: d_model even, 2 <= d_model <= 4096; ld_w >= n_head*d_head; ld_r >= d_head.
 * bf16: tensor-core path (fp32 accumulate, R rounded to bf16 before the product, output rounded
 *       to bf16 once); needs W_R 16-byte aligned and ld_w a multiple of 8.
 * f32 : fp32 SIMT path with R rounded once from double precision.
 */
txl_status txl_rel_pos_gen(int n_rows, int d_model, int n_head, int d_head,
                           const void* W_R, int64_t ld_w,
                           void* r, int64_t ld_r,
                           txl_dtype dtype, void* stream);

/*
 * txl_rel_attn_fwd -- one forward call of relative multi-head attention.
 * For every batch b, head h and query i (0 <= i < L, absolute position M+i) over keys
 * j in [memory(0..M-1) ++ current(M..M+L-1)]:
 *   delta = M + i - j,  delta_c = min(delta, clamp_len)
 *   visible(i, j) <=> (M - valid) <= j <= M + i
 *   s_ij  = scale * ( q_i.k_j + q_i.r[delta_c] + u_h.k_j + v_h.r[delta_c] )
 *   out_i = sum_j softmax_j(s_ij over visible j) * v_j          (masked keys weigh exactly 0)
 * Arguments:
 *   q      : view of [B][L][H][D] queries of the current segment (device).
 *   mem    : the memory (see txl_mem); may be NULL when there is no memory (M = 0).
 *   k_cur, v_cur : views of [B][L][H][D] keys/values of the current segment (device).
 *   u, v_bias : device fp32 [H][D] global content / position biases.
 *   r      : device [n_rows][H][ld_r] from txl_rel_pos_gen; n_rows >= min(M+L, clamp_len+1).
 *   scale  : logit scale; <= 0 selects 1/sqrt(D).
 *   out    : view of [B][L][H][D] outputs (device), dtype.
 *   workspace : device scratch of workspace_bytes (txl_rel_attn_workspace_size); may be NULL
 *            when that size is 0.
 *   err_flag : optional device int; a kernel whose bounded wait expires writes TXL_ERR_TIMEOUT
 *            there (and its outputs are then undefined).  Never cleared by the library.
 * Paths:
 *   bf16, D <= 128, every base and stride 16-byte aligned, and a ring whose wp and M are
 *   multiples of 128 (or wp == 0): the fused TMA + tcgen05 kernel (TMEM accumulators; the
 *   relative shift is an index remap; the score matrix never reaches HBM).
 *   otherwise (f32, other layouts, other rings): a warp-per-query SIMT kernel on the GPU.
 */
txl_status txl_rel_attn_fwd(int B, int L, int H, int D, int clamp_len,
                            const txl_view* q, const txl_mem* mem,
                            const txl_view* k_cur, const txl_view* v_cur,
                            const float* u, const float* v_bias,
                            const void* r, int64_t ld_r, int n_rows,
                            float scale, const txl_view* out, txl_dtype dtype,
                            void* workspace, size_t workspace_bytes,
                            int* err_flag, void* stream);

/* Bytes of device workspace txl_rel_attn_fwd needs for this shape (0 for every path of this
 * version; kept so callers can size it once). */
size_t txl_rel_attn_workspace_size(int B, int L, int H, int D, const txl_mem* mem,
                                   txl_dtype dtype);

/* Which kernel txl_rel_attn_fwd would run for these arguments: 1 = fused tcgen05 kernel,
 * 2 = SIMT kernel, or a negative txl_status if the arguments are rejected. */
int txl_rel_attn_path(int B, int L, int H, int D, const txl_view* q, const txl_mem* mem,
                      const txl_view* k_cur, const txl_view* v_cur, const void* r,
                      int64_t ld_r, const txl_view* out, txl_dtype dtype);

/*
 * txl_rel_attn_decode -- the same attention as txl_rel_attn_fwd for a few queries (1 <= L <= 16)
 * over a long memory: the incremental-generation case ("Transformer-XL架构解析" §3.2,
 * "Transformer-XL 和相对位置编码" §2.2: each new token attends to the cached memory and itself).
 * Arguments, layouts, masks, clamp and result are those of txl_rel_attn_fwd (f32 or bf16, any
 * ring), except:
 *   L         : 1 .. 16 queries per (b, h) (TXL_ERR_UNSUPPORTED above).
 *   workspace : device scratch, 16-byte aligned, of at least
 *               txl_rel_attn_decode_workspace_size(B, L, H, D, mem) bytes (TXL_ERR_WORKSPACE
 *               otherwise).  It holds per-chunk partial results between the two kernels of the
 *               call; its contents on entry do not matter and are overwritten.
 * The keys of every (b, h) are split into chunks of 256 processed by separate CTAs on the CUDA
 * cores (the work is bound by HBM bandwidth: about one flop per byte at L = 1), then the chunks
 * are merged (split-K softmax).  Calls that share a workspace must not overlap on the GPU.
 * With L >= 3, bf16, D <= 64 and inputs that txl_rel_attn_fwd's fused kernel takes (16-byte aligned
 * rows and strides; a ring's write pointer and length multiples of 128), the call runs that fused
 * tensor-core kernel instead (one query tile over every key, faster from three queries on) and
 * leaves the workspace untouched; the argument checks, the workspace check included, are the same.
 */
txl_status txl_rel_attn_decode(int B, int L, int H, int D, int clamp_len,
                               const txl_view* q, const txl_mem* mem,
                               const txl_view* k_cur, const txl_view* v_cur,
                               const float* u, const float* v_bias,
                               const void* r, int64_t ld_r, int n_rows,
                               float scale, const txl_view* out, txl_dtype dtype,
                               void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device workspace txl_rel_attn_decode needs: B*H*L*ceil((M+L)/256)*(D+2)*4
 * (0 when the shape is outside the decode path). */
size_t txl_rel_attn_decode_workspace_size(int B, int L, int H, int D, const txl_mem* mem);

/* Which kernels txl_rel_attn_decode (and txl_rel_attn_decode_noalloc) would run for these
 * arguments: 1 = the fused persistent tcgen05 kernel (L >= 3, see txl_rel_attn_decode), 4 = the
 * split-key decode kernels and their merge, or a negative txl_status if the arguments are rejected.
 * Nothing is launched; the workspace is not checked. */
int txl_rel_attn_decode_path(int B, int L, int H, int D, const txl_view* q, const txl_mem* mem,
                             const txl_view* k_cur, const txl_view* v_cur, const void* r,
                             int64_t ld_r, const txl_view* out, txl_dtype dtype);

/*
 * txl_rel_attn_decode_noalloc -- txl_rel_attn_decode without a caller workspace, for callers that
 * cannot obtain device memory at call time.  The pages have no counterpart to this entry point: it
 * is a service of this library.  Examples of such callers: a serving process whose device memory
 * is owned by a pre-sized arena that forbids allocations once it runs; a plugin reached through an
 * interface that passes only inputs and outputs; a per-token generation loop that cannot afford
 * cudaMalloc, which may synchronise the device.  Nothing here allocates: no cudaMalloc, cudaFree
 * or allocating library routine is called.
 * Arguments, layouts and results are those of txl_rel_attn_decode minus the workspace.  The
 * per-chunk partial results live instead in a fixed 8 MiB scratch array inside the library, which
 * every GPU that loads the library holds until the process exits:
 *   - B*H*L*ceil((M+L)/256)*(D+2)*4 must not exceed 8388608 bytes (TXL_ERR_WORKSPACE otherwise;
 *     use txl_rel_attn_decode with a workspace for such shapes);
 *   - the first call on a device looks up the array's device address (cudaGetSymbolAddress, with
 *     that device current) and caches it with the id of the current context; make that first
 *     call before any stream capture.  After cudaDeviceReset the device's new context has another
 *     id, and the first call in it looks the address up again (so that call, too, belongs before
 *     any capture);
 *   - every call shares the array.  Each call writes every partial it reads, so nothing has to
 *     start at zero, but calls that overlap on the GPU (two streams, or two host threads on
 *     different streams) race on it and their results are undefined: keep them ordered, for
 *     instance on one stream.
 * Calls that txl_rel_attn_decode sends to the fused kernel (L >= 3, see there) do so here as well
 * and do not touch the array (the size limit above still applies to them).
 */
txl_status txl_rel_attn_decode_noalloc(int B, int L, int H, int D, int clamp_len,
                                       const txl_view* q, const txl_mem* mem,
                                       const txl_view* k_cur, const txl_view* v_cur,
                                       const float* u, const float* v_bias,
                                       const void* r, int64_t ld_r, int n_rows,
                                       float scale, const txl_view* out, txl_dtype dtype,
                                       void* stream);

/*
 * txl_mem_push -- append L positions to the FIFO memory ("Transformer-XL架构解析" §1.1;
 * "Transformer-XL 和相对位置编码" §2.3.1: the cached states of the previous segment).
 * Copies k_new/v_new [B][L][H][D] (device views) into slots (wp + t) mod M for
 * t = max(0, L-M) .. L-1 (a segment longer than the memory keeps its last M positions), then
 * updates mem->wp = (wp + L) mod M and mem->valid = min(valid + L, M) on the host at enqueue
 * time.  The copy is ordered on `stream`; the attention for this segment must be enqueued
 * before the push if it should see the previous memory.  Bit-exact copy.
 */
txl_status txl_mem_push(txl_mem* mem, const txl_view* k_new, const txl_view* v_new, int L,
                        void* stream);

/*
 * txl_linear -- Y = X W: bf16 inputs, fp32 accumulation on the tensor cores, one rounding of each
 * output to bf16.  The content projections of the attention layer: q_proj, k_proj, v_proj and
 * o_proj of "TransformerXL 相对位置编码" §3.1 (linear maps without bias); Q = h W_q, K = h~ W_k,
 * V = h~ W_v of "Transformer-XL 和相对位置编码" §2.3.1.
 *   X : device [m][ld_x], columns 0..k-1 are read;  W : device [k][ld_w], columns 0..n-1 are read;
 *   Y : device [m][ld_y], columns 0..n-1 are written and nothing else.
 * Limits: m, n >= 0 (either 0: nothing to do), k >= 1; ld_x >= k, ld_w >= n, ld_y >= n; X and W
 * 16-byte aligned with ld_x, ld_w multiples of 8 (TXL_ERR_ALIGNMENT otherwise).  bf16 only
 * (TXL_ERR_UNSUPPORTED for TXL_F32).  err_flag: as txl_rel_attn_fwd.
 */
txl_status txl_linear(int m, int n, int k, const void* X, int64_t ld_x, const void* W, int64_t ld_w,
                      void* Y, int64_t ld_y, txl_dtype dtype, int* err_flag, void* stream);

/*
 * txl_rel_attn_layer -- one attention-layer step of Transformer-XL over hidden states:
 *   Q = h W_q and K = h~ W_k, V = h~ W_v over h~ = [SG(h_mem) o h], the memory-extended states
 *   ("Transformer-XL 和相对位置编码" §2.3.1); the relative attention of txl_rel_attn_fwd with the
 *   memory's keys first; y = concat_heads(attention) W_o ("TransformerXL 相对位置编码" §3.1); then
 *   the segment enters the memory (the FIFO of txl_mem_push; mem->wp and mem->valid advance).
 * The memory caches the projected keys and values of its positions (h_mem W_k, h_mem W_v) rather
 * than h_mem: with the weights fixed this is the same function (a row's projection does not depend
 * on when it is taken), and each position is projected once, when it enters the memory, instead of
 * once for every segment that attends to it.
 *   h      : device bf16 [B*L][ld_h], row b*L + t = position t of batch entry b, d_model columns.
 *   mem    : K/V memory as for txl_rel_attn_fwd (bf16, B, H, D matching), or NULL / M = 0.
 *   W_qkv  : device bf16 [d_model][3*H*D], columns [0,HD) = W_q, [HD,2HD) = W_k, [2HD,3HD) = W_v.
 *   W_o    : device bf16 [H*D][d_model].
 *   u, v_bias, r, ld_r, n_rows, clamp_len, scale : as txl_rel_attn_fwd (r from txl_rel_pos_gen).
 *   y      : device bf16 [B*L][ld_y], d_model columns written.
 *   workspace : device, >= txl_rel_attn_layer_workspace_size(B, L, H, D) bytes, 16-byte aligned
 *            (TXL_ERR_WORKSPACE if missing or smaller): the segment's q|k|v [B*L][3*H*D] and the
 *            attention output [B*L][H*D], bf16.  Its contents after the call are unspecified.
 * Limits: H*D and d_model multiples of 8; the limits of txl_linear and txl_rel_attn_fwd.  bf16
 * only.  Enqueues four launches on `stream` (projection, attention, output projection, push).
 */
txl_status txl_rel_attn_layer(int B, int L, int H, int D, int d_model, int clamp_len,
                              const void* h, int64_t ld_h, txl_mem* mem,
                              const void* W_qkv, const void* W_o,
                              const float* u, const float* v_bias,
                              const void* r, int64_t ld_r, int n_rows, float scale,
                              void* y, int64_t ld_y, void* workspace, size_t workspace_bytes,
                              int* err_flag, void* stream);

/* Bytes of device workspace txl_rel_attn_layer needs: B*L*H*D*8 (0 for an empty shape). */
size_t txl_rel_attn_layer_workspace_size(int B, int L, int H, int D);

/*
 * txl_rel_attn_layer_fused -- the layer step of txl_rel_attn_layer in three launches, with the memory
 * push folded into the projection.  The memory of mem_len positions lives in a ring of at least
 * mem_len + L slots (mem->M slots; mem->wp = slot of the oldest memory position, mem->valid = valid
 * memory positions, 0 .. mem_len): the q|k|v product writes the segment's K and V straight into the
 * L slots after the memory, (wp + mem_len + t) mod mem->M, and Q into the workspace; the fused
 * attention reads memory and segment keys from the ring (logical key j of [memory ++ segment] in
 * slot (wp + j) mod mem->M); the output product follows; then, instead of a copy, the window moves:
 * mem->wp += L (mod mem->M), mem->valid = min(valid + L, mem_len).  The function is that of
 * txl_rel_attn_layer with a memory of mem_len positions ("Transformer-XL 和相对位置编码" §2.3.1: the
 * cached states of the previous segment extend the keys and values; "TransformerXL 相对位置编码" §3.1:
 * projections without bias).
 *   h, W_qkv, W_o, u, v_bias, r, ld_r, n_rows, clamp_len, scale, y, ld_y, err_flag : as txl_rel_attn_layer
 *            (n_rows >= min(mem_len + L, clamp_len + 1)).
 *   mem    : device bf16 rings k, v, dense [B][mem->M][H][D]; a ring starts zeroed (wp = 0, valid = 0):
 *            slots past the valid memory are read (and masked), so they must hold finite values.
 *   workspace : device, >= txl_rel_attn_layer_fused_workspace_size(B, L, H, D) bytes, 16-byte aligned.
 * Limits (TXL_ERR_UNSUPPORTED otherwise; use txl_rel_attn_layer): bf16; D <= 64 and a multiple of 8;
 * H*D a multiple of 64; d_model a multiple of 8; L, mem_len, mem->M and mem->wp multiples of 128.
 */
txl_status txl_rel_attn_layer_fused(int B, int L, int H, int D, int d_model, int clamp_len,
                                    const void* h, int64_t ld_h, txl_mem* mem, int mem_len,
                                    const void* W_qkv, const void* W_o,
                                    const float* u, const float* v_bias,
                                    const void* r, int64_t ld_r, int n_rows, float scale,
                                    void* y, int64_t ld_y, void* workspace, size_t workspace_bytes,
                                    int* err_flag, void* stream);

/* Bytes of device workspace txl_rel_attn_layer_fused needs: B*L*H*D*4 (0 for an empty shape). */
size_t txl_rel_attn_layer_fused_workspace_size(int B, int L, int H, int D);

/*
 * txl_rel_attn_bwd -- gradients of one txl_rel_attn_fwd call for an upstream gradient d_out,
 * by the chain rule through the four-term score ("Transformer-XL 和相对位置编码" §2.3.2) and the
 * softmax: with q' = q + u, q'' = q + v_bias, P the attention weights and dS_ij =
 * scale P_ij (d_out_i . v_j - d_out_i . out_i),
 *   dq_i  = sum_j dS_ij (k_j + r[delta_ij])        dk_j = sum_i dS_ij q'_i      dv_j = sum_i P_ij d_out_i
 *   du    = sum dS_ij k_j     dv_bias = sum dS_ij r[delta_ij]     dr[delta] = sum_{delta_ij = delta} dS_ij q''_i
 * The memory's keys and values get no gradient: the memory is the stop-gradient part of the
 * extended sequence ("Transformer-XL 和相对位置编码" §2.3.1); dk_cur, dv_cur cover the current
 * segment's keys.  Arguments as txl_rel_attn_fwd, plus
 *   out    : the forward call's output (view, dtype);  d_out : upstream gradient (view, dtype).
 *   dq, dk_cur, dv_cur : device fp32 [B][L][H][D] (dense);  du, dv_bias : device fp32 [H][D];
 *   dr     : device fp32 [n_rows][H][D], every row written (rows no pair reaches are zero).
 *   workspace : device, >= txl_rel_attn_bwd_workspace_size(B, L, H, D) bytes, 16-byte aligned.
 * Scores are recomputed and P is never stored.  bf16 with D = 64 and 16-byte aligned rows and
 * strides (q, k, v, the memory, d_out, r): bf16 products on the tensor cores with fp32 accumulation
 * (c(q + u), c(q + v), P and dS rounded to bf16 as product operands, c = scale log2 e; pairs whose
 * distance reaches clamp_len summed in fp32), the row log-sum-exp taken by the fused forward kernel
 * when that kernel takes the inputs (written into the workspace).  With out, the gradients and dr
 * 16-byte aligned as well, the gradient products run as tcgen05 MMAs with TMEM accumulators (a
 * launch of query CTAs for dq and dr, and key CTAs for dk and dv); otherwise as mma.sync products.
 * Every other case: fp32 arithmetic on the CUDA cores.  Enqueues several launches.
 */
txl_status txl_rel_attn_bwd(int B, int L, int H, int D, int clamp_len,
                            const txl_view* q, const txl_mem* mem,
                            const txl_view* k_cur, const txl_view* v_cur,
                            const float* u, const float* v_bias,
                            const void* r, int64_t ld_r, int n_rows, float scale,
                            const txl_view* out, const txl_view* d_out,
                            float* dq, float* dk_cur, float* dv_cur, float* du, float* dv_bias,
                            float* dr, txl_dtype dtype, void* workspace, size_t workspace_bytes,
                            void* stream);

/* Which gradient kernel txl_rel_attn_bwd and txl_rel_attn_bwd_lse would run for these arguments
 * (the addresses of out, d_out and the gradient buffers count: their alignment chooses the kernel):
 * 1 = tcgen05 kernel, 2 = mma.sync kernel, 3 = SIMT kernels, or a negative txl_status if the
 * arguments are rejected.  No launch. */
int txl_rel_attn_bwd_path(int B, int L, int H, int D, const txl_view* q, const txl_mem* mem,
                          const txl_view* k_cur, const txl_view* v_cur, const void* r, int64_t ld_r,
                          const txl_view* out, const txl_view* d_out, const float* dq, const float* dk_cur,
                          const float* dv_cur, const float* dr, txl_dtype dtype);

/* Bytes of device workspace txl_rel_attn_bwd needs: B*L*H*(2 + 2*D)*4 (0 for an empty shape). */
size_t txl_rel_attn_bwd_workspace_size(int B, int L, int H, int D);

/*
 * txl_rel_attn_fwd_lse -- txl_rel_attn_fwd that also saves the statistics of its softmax, as a
 * forward pass does for its backward:
 *   lse : device fp32 [B][L][H] (4-byte aligned), lse[(b L + i) H + h] = m_i + log2 l_i, the
 *         log2-domain log-sum-exp of row i's visible scores in the units c s_ij (c = scale log2 e):
 *         m_i the row maximum, l_i the sum of the bf16 weights 2^(c s_ij - m_i) that the output's
 *         P.V multiplied (the output's own normaliser).
 * out is written exactly as txl_rel_attn_fwd writes it.  Only the fused tcgen05 kernel keeps the
 * statistics: bf16, D <= 64 and the inputs its path takes (txl_rel_attn_path = 1), else
 * TXL_ERR_UNSUPPORTED before any launch; lse NULL: TXL_ERR_INVALID_ARG; misaligned:
 * TXL_ERR_ALIGNMENT.  Other arguments and errors as txl_rel_attn_fwd.
 */
txl_status txl_rel_attn_fwd_lse(int B, int L, int H, int D, int clamp_len,
                                const txl_view* q, const txl_mem* mem,
                                const txl_view* k_cur, const txl_view* v_cur,
                                const float* u, const float* v_bias,
                                const void* r, int64_t ld_r, int n_rows,
                                float scale, const txl_view* out, float* lse, txl_dtype dtype,
                                void* workspace, size_t workspace_bytes,
                                int* err_flag, void* stream);

/*
 * txl_rel_attn_bwd_lse -- txl_rel_attn_bwd given the statistics txl_rel_attn_fwd_lse saved for
 * the same call (same inputs and output): on the tensor-core path the gradient kernels read lse
 * in place of taking the row log-sum-exp again (one pass over the keys fewer).  lse: device fp32
 * [B][L][H] (4-byte aligned, TXL_ERR_ALIGNMENT otherwise), read only; NULL gives
 * txl_rel_attn_bwd.  Paths that do not use the statistics ignore it.  Other arguments, results and
 * errors as txl_rel_attn_bwd.
 */
txl_status txl_rel_attn_bwd_lse(int B, int L, int H, int D, int clamp_len,
                                const txl_view* q, const txl_mem* mem,
                                const txl_view* k_cur, const txl_view* v_cur,
                                const float* u, const float* v_bias,
                                const void* r, int64_t ld_r, int n_rows, float scale,
                                const txl_view* out, const txl_view* d_out, const float* lse,
                                float* dq, float* dk_cur, float* dv_cur, float* du, float* dv_bias,
                                float* dr, txl_dtype dtype, void* workspace, size_t workspace_bytes,
                                void* stream);

/*
 * txl_rel_pos_bwd -- gradient of W_R from the gradient of the position rows:
 *   dW_R[m][h*d_head + d] = sum_delta R_delta[m] * dr[delta][h][d]
 * with R_delta the interleaved sinusoid of txl_rel_pos_gen (frequencies in double precision; the
 * angle of every fourth distance reduced modulo 2 pi in double precision, the other three offset from
 * it in fp32; then the fp32 sine or cosine: entries within 6e-7 of the exact sinusoid).  dr: device fp32 [n_rows][H][D] (as txl_rel_attn_bwd writes it);
 * dW_R: device fp32 [d_model][ld_dw], columns 0..H*D-1 written (zeroed, then partial sums over
 * ranges of distances added atomically: the fp32 summation order may differ from call to call).
 * d_model even, ld_dw >= H*D.  The products run on the tensor cores as three tf32 products per
 * step (R and dr each split into a tf32 part and the fp32 remainder; the remainder product dropped):
 * about 2^-21 relative error per product, fp32 accumulation.
 */
txl_status txl_rel_pos_bwd(int n_rows, int d_model, int n_head, int d_head, const float* dr,
                           float* dW_R, int64_t ld_dw, void* stream);

/*
 * txl_rel_attn_table_fwd -- the learned-table variant of relative attention ("TransformerXL 相对位置编码"
 * §3.1): bidirectional over one sequence of L positions (no memory, no causal mask).  The position
 * vector of a pair is row rel = clamp(i - j + max_len - 1, 0, 2*max_len - 2) of the projected table
 * r_table = pos_emb W_R (the distance shifted to a non-negative index and clamped, §2; project the
 * learned pos_emb [2*max_len - 1][d_model] with txl_linear, the projection commutes with the lookup):
 *   s_ij = scale*q_i.k_j + scale*q_i.r_rel + u_h.k_j + v_h.r_rel
 * (the scale on the first two terms only, as that page computes it), keys with key_mask[b][j] == 0
 * scored -1e9 (a row whose keys are all masked averages every value), out_i = softmax_j(s_ij) v_j.
 *   q, k, v, out : views of [B][L][H][D] (device, dtype).  u, v_bias : device fp32 [H][D].
 *   r_table : device [2*max_len - 1][H][ld_r], dtype.  key_mask : device uint8 [B][L] or NULL.
 *   scale   : <= 0 selects 1/sqrt(D).
 * Limits: 1 <= D <= 128, max_len >= 1.  bf16 with D <= 64, L <= max_len and 16-byte aligned bases
 * and strides (q, k, v, r_table): the persistent tcgen05 kernel of txl_rel_attn_fwd in a learned-table
 * mode (log2(e)(scale*q + u), log2(e)(scale*q + v) and P rounded to bf16 as product operands, fp32
 * accumulation in tensor memory; a masked key's score is about -1e30 there, which gives it the same
 * weight as -1e9: exactly 0 beside any unmasked key, equal weights in a fully masked row).  Other bf16
 * calls with D = 64 and 16-byte aligned
 * rows and strides (q, k, v, out, r_table): bf16 mma.sync products with fp32 accumulation (scale*q + u,
 * scale*q + v and P rounded to bf16).  Every other case: fp32 arithmetic on the CUDA cores.
 */
txl_status txl_rel_attn_table_fwd(int B, int L, int H, int D, int max_len,
                                  const txl_view* q, const txl_view* k, const txl_view* v,
                                  const float* u, const float* v_bias,
                                  const void* r_table, int64_t ld_r, const uint8_t* key_mask,
                                  float scale, const txl_view* out, txl_dtype dtype, void* stream);

/* Which kernel txl_rel_attn_table_fwd would run for these arguments: 1 = the persistent tcgen05
 * kernel (learned-table mode), 3 = the mma.sync tensor-core kernel, 2 = the CUDA-core kernel, or a
 * negative txl_status if the arguments are rejected.  Nothing is launched. */
int txl_rel_attn_table_path(int B, int L, int H, int D, int max_len,
                            const txl_view* q, const txl_view* k, const txl_view* v,
                            const void* r_table, int64_t ld_r, const uint8_t* key_mask,
                            const txl_view* out, txl_dtype dtype);

/*
 * Quantised K/V memory: the FIFO memory of txl_mem with its keys and values held as 4- or 8-bit
 * codes (a service of this library; the pages hold the memory in the compute type).  The channels
 * of a head are split into groups of 32 consecutive d (G = ceil(D/32); the last group is shorter
 * when D is not a multiple of 32).  With n = 2^bits - 1, a group x of one position is held as
 *     lo   = the largest bf16 that is not above min(x)
 *     step = the smallest bf16 that is not below (max(x) - lo) / n
 *     c_d  = the integer nearest to (x_d - lo) / step, ties to even (0 where step = 0)
 * and stands for x'_d = lo + step * c_d, so |x'_d - x_d| <= step / 2.  These definitions are met
 * exactly, whatever the input type.  A group with a NaN or an infinity, or one whose lo, step or
 * max - lo is not finite, is held with step = lo = NaN and stands for NaN throughout.
 *   rows : device, 16-byte aligned, dense [B][H][M][row] bytes, row = txl_qmem_row_bytes(D, bits).  A row
 *          holds the k codes of G groups in the order of d (4 bits: byte t holds d = 2t in its low and
 *          d = 2t + 1 in its high half; codes of d >= D are 0), the v codes likewise, then for each
 *          group four bf16: the k step, k lo, v step and v lo (zeros for one group more where G is
 *          odd).  That is G * bits / 2 + ceil(G / 2) units of 16 bytes; where their number is a
 *          multiple of eight, an unused unit follows (eight rows in shared memory must not begin in
 *          the same banks).  One position of a head is one contiguous piece, and so are its neighbours.
 *   bits : 4 or 8.  D <= 128.
 *   wp, valid : as in txl_mem (logical key j in slot (wp + j) mod M, valid iff j >= M - valid).
 * Slots that are not valid are never read, so the rows need no initial values.  M = 0 means no
 * memory (rows may then be NULL).
 */
typedef struct {
    void* rows;
    int B, M, H, D;
    int bits;
    int wp;
    int valid;
} txl_qmem;

/* Bytes of a row of a quantised memory (0 for an invalid shape): it takes B * H * M of them. */
size_t txl_qmem_row_bytes(int D, int bits);

/*
 * txl_qmem_push -- txl_mem_push into a quantised memory: quantises k_new/v_new [B][L][H][D] (device
 * views of dtype) into slots (wp + t) mod M for t = max(0, L-M) .. L-1, then updates mem->wp and
 * mem->valid on the host at enqueue time.  Other slots are left as they were.  Any strides; rows
 * that start on 16-byte boundaries are read 16 bytes at a time.
 */
txl_status txl_qmem_push(txl_qmem* mem, const txl_view* k_new, const txl_view* v_new, int L,
                         txl_dtype dtype, void* stream);

/*
 * txl_qmem_read -- what the memory stands for: logical positions j0 .. j0+n-1 (oldest first; all of
 * them valid: M - valid <= j0, j0 + n <= M, TXL_ERR_INVALID_ARG otherwise) into views k_out, v_out
 * of [B][n][H][D], dtype: one fp32 multiply-add, rounded to dtype.  Only d < D is written.
 */
txl_status txl_qmem_read(const txl_qmem* mem, int j0, int n, const txl_view* k_out,
                         const txl_view* v_out, txl_dtype dtype, void* stream);

/* txl_qmem_push and txl_qmem_read with their arguments in one struct, for bindings that pay per argument: k, v are
 * k_new, v_new or k_out, v_out; n is L or n; j0 is read by txl_qmem_read_call alone. */
typedef struct {
    txl_qmem* mem;
    txl_view k, v;
    int j0, n;
    int dtype;                 /* a txl_dtype */
    void* stream;
} txl_qmem_kv_args;
txl_status txl_qmem_push_call(const txl_qmem_kv_args* args);
txl_status txl_qmem_read_call(const txl_qmem_kv_args* args);

/*
 * txl_rel_attn_qmem -- txl_rel_attn_fwd with the memory's keys and values held in a txl_qmem: the
 * same scores, mask, clamp and softmax over k'_j, v'_j = what the memory stands for, and the current
 * segment's k_cur, v_cur as they are.  Arguments as txl_rel_attn_fwd (mem may be NULL), plus
 *   workspace : device scratch, 16-byte aligned, of at least txl_rel_attn_qmem_workspace_size(B, L,
 *            H, D, mem, dtype) bytes (TXL_ERR_WORKSPACE otherwise; may be NULL when that is 0).
 *            Calls that share a workspace must not overlap on the GPU.
 * L <= 16 (generation), two launches, or one where few positions are not clamped: the position terms
 * (q+v).r go into the workspace, then the codes are multiplied as they are (q and the weights, each group of 32
 * channels in units of its own, held to 22 bits, or to 2^-34 of the group's largest where that is more; fp32
 * calls keep sums to fp32's precision, bf16 ones to 15 bits).  A position whose step in a group of values is far
 * above the others' costs the group bits: its sums are then off by up to 2^-12 of that position's weighted step,
 * in fp32 2^-14 (what it stands for is off by up to half a step from what was pushed).
 * L > 16, bf16, four launches (three for D > 64): K and V of the memory's valid positions and of the segment,
 * and r, are written into the workspace once in 16 bits, and the fused tcgen05 kernels of txl_rel_attn_fwd run
 * over them, for q, k_cur, v_cur and r of any layout.  A (b, h) has fp16 operands and P, in units of powers of
 * two taken from the data, where fp16 has the range: all its values are finite, D times a bound of
 * |scale log2(e) (q+u)| times the largest |k'| is at most 2^15, the same for (q+v) and the head's r, and the
 * largest |v'| is at most 2^12 times the smallest that a group of 32 channels which is not zero has as its
 * largest.  Otherwise it has bf16 ones, as in txl_rel_attn_fwd.  (Where r's rows do not start on 16-byte
 * boundaries, all entries of a head have one type.)  Keys and values of the segment reach the queries from
 * their position on alone, whatever they are.  (A call without a memory, M = 0, is txl_rel_attn_fwd's.)
 * L > 16, fp32, one launch: codes are expanded tile by tile in shared memory, all arithmetic in fp32.
 * err_flag as for txl_rel_attn_fwd: every kernel that waits for copies sets it if a wait runs out.
 */
txl_status txl_rel_attn_qmem(int B, int L, int H, int D, int clamp_len,
                             const txl_view* q, const txl_qmem* mem,
                             const txl_view* k_cur, const txl_view* v_cur,
                             const float* u, const float* v_bias,
                             const void* r, int64_t ld_r, int n_rows,
                             float scale, const txl_view* out, txl_dtype dtype,
                             void* workspace, size_t workspace_bytes,
                             int* err_flag, void* stream);

/* txl_rel_attn_qmem with its arguments in one struct, for bindings that pay per argument. */
typedef struct {
    int B, L, H, D, clamp_len, n_rows;
    int dtype;                 /* a txl_dtype */
    float scale;
    txl_view q, k_cur, v_cur, out;
    const txl_qmem* mem;
    const float* u;
    const float* v_bias;
    const void* r;
    int64_t ld_r;
    void* workspace;
    size_t workspace_bytes;
    int* err_flag;
    void* stream;
} txl_rel_attn_qmem_args;
txl_status txl_rel_attn_qmem_call(const txl_rel_attn_qmem_args* args);

/* Bytes of device workspace txl_rel_attn_qmem needs.  L <= 16: B*H*L rows of M + L floats (a multiple of
 * four, and up to seven more).  L > 16: 0 without a memory or in fp32, else, with D rounded up to a
 * multiple of 8 in each row of a head, M rows of K and V in 16 bits, 3 L such rows, M + L rows of r and 144
 * bytes per (b, h). */
size_t txl_rel_attn_qmem_workspace_size(int B, int L, int H, int D, const txl_qmem* mem, txl_dtype dtype);

/* Which kernels txl_rel_attn_qmem would run for these arguments: 5 = the one that multiplies the codes
 * (L <= 16), 6 = the fp32 one of longer segments, 1 = the expanded memory, then the tcgen05 kernels, 1 or
 * 2 = the kernel of txl_rel_attn_path for a bf16 call without a memory, or a negative txl_status if the
 * arguments are rejected.  Nothing is launched; the workspace is not checked. */
int txl_rel_attn_qmem_path(int B, int L, int H, int D, const txl_view* q, const txl_qmem* mem,
                           const txl_view* k_cur, const txl_view* v_cur, const void* r,
                           int64_t ld_r, const txl_view* out, txl_dtype dtype);

/*
 * Paged K/V memory: the cached keys and values of B sequences of different lengths in pages of one pool (a service of
 * this library; the pages of the reference hold one length for the batch).  Slot s of sequence b is row s mod page_len
 * of page table[b][s / page_len]; a sequence uses its slots 0 .. length[b]-1.  Each slot holds a position (the
 * attention takes distances from it, so slots may be in any order, and positions may be missing), and the attention
 * weight that it has received so far.  The positions of a sequence are distinct and below next_pos[b], that of its next
 * one.  Lengths, positions and table are device memory: a captured graph of calls may be replayed, and each replay works
 * on what the memory then holds.
 *   k, v     : device, 16-byte aligned, [n_pages][H][page_len][ld] of dtype; ld >= D, rows of a multiple of 16 bytes.
 *              What a row holds at and past D is never used (pushes write zeros there).
 *   pos, weight : device [n_pages][page_len]; pos 8-byte aligned.
 *   table    : device [B][max_pages]; entries outside 0 .. n_pages-1 are no page.  A page that a push, an eviction or the
 *              sum of weights writes belongs to one sequence; pages that are only read may be shared.
 *   length, next_pos : device [B];  scratch : device, B * (H + 1) + 1 ints, zero (every call leaves it so).
 *   err_flag : optional device int: a call that meets a slot without a page writes TXL_ERR_PAGE there if it is 0 (never
 *              cleared by the library).  Such a slot counts as not there; a push that does not find pages for all new
 *              positions of a sequence leaves that sequence as it was, and its queries' outputs too.
 * Calls on one memory must not overlap on the GPU (one stream, or ordered streams), and no tensor that a call writes may
 * overlap one that it reads.
 * Limits (TXL_ERR_UNSUPPORTED): D <= 128; ld <= 65536; page_len a multiple of 16; B <= 4096; H <= 65535; n_pages * page_len and
 * max_pages * page_len, and the T of a push, below 2^31 - 2^20.  Positions are 0 .. 2^31 - 33.
 */
typedef struct {
    void* k;
    void* v;
    int* pos;
    float* weight;
    const int* table;
    int* length;
    int* next_pos;
    int* scratch;
    int* err_flag;
    int B, H, D, ld, n_pages, page_len, max_pages;
    int dtype;                 /* a txl_dtype */
} txl_paged;

/*
 * txl_paged_push -- new positions of every sequence: rows t < counts[b] of k_new, v_new [B][T][H][D] (device views of
 * the memory's dtype) into slots length[b] + t, with positions next_pos[b] + t and weight 0; then length[b] and next_pos[b]
 * advance by counts[b].  counts: device [B] (values outside 0 .. T count as 0 or T), or NULL for T each.  Rows past
 * counts[b] are not read.  Bit-exact copy; any strides.  T = 0: nothing to do.
 */
txl_status txl_paged_push(const txl_paged* mem, const txl_view* k_new, const txl_view* v_new, int T, const int* counts,
                          void* stream);

/* txl_paged_push with its arguments in one struct, for bindings that pay per argument. */
typedef struct {
    const txl_paged* mem;
    txl_view k_new, v_new;
    const int* counts;
    void* stream;
    int T;
} txl_paged_push_args;
txl_status txl_paged_push_call(const txl_paged_push_args* args);

/*
 * txl_rel_attn_paged -- relative attention of T = 1 .. 16 new tokens a sequence over a paged memory (incremental
 * generation, "Transformer-XL架构解析" §3.2: each new token attends to the cached memory and itself).  With k_new, v_new
 * the call first pushes them as txl_paged_push does; with both NULL the last counts[b] positions of each sequence are in
 * the memory already.  Query i < counts[b] of sequence b has position p_i = next_pos[b] - counts[b] + i (next_pos after
 * the push), slot j position p_j:
 *   visible(i, j) <=> p_j <= p_i,   delta = min(p_i - p_j, clamp_len, n_rows - 1)
 *   s_ij  = scale * ( q_i.k_j + q_i.r[delta] + u_h.k_j + v_h.r[delta] )
 *   out_i = sum_j softmax_j(s_ij over visible j) * v_j       (0 where nothing is visible)
 * Rows i >= counts[b] of out are left as they were (and those of q not read).
 *   u, v_bias, r, ld_r, scale : as txl_rel_attn_fwd;  n_rows >= 1 rows of r (no more than 2^30 distances, H * ld_r below 2^31).
 *   accumulate : not 0: weight[j] += sum over heads and queries of softmax_j(s_ij), for txl_paged_evict (a slot's weight
 *              is the sum over the calls since it entered).
 *   workspace : device scratch, 16-byte aligned, of at least txl_rel_attn_paged_workspace_size bytes (TXL_ERR_WORKSPACE).
 *              Calls that share a workspace must not overlap on the GPU.
 * T > 16: TXL_ERR_UNSUPPORTED.  More tokens over a memory that a sequence already has go through calls of 16; a first prompt takes
 * txl_rel_attn_fwd and txl_paged_push.
 * The slots of all (sequence, head) pairs are cut into equal shares for the blocks, whatever the lengths.  bf16: mma.sync
 * products; scale log2(e) (q + u), scale log2(e) (q + v) and the weights of the softmax are held to 16 bits (two bf16
 * each).  f32: fp32 arithmetic on the CUDA cores.  The result does not depend on the order in which blocks run.  A key or value
 * that a query does not see does not reach it, whatever it is.  One launch for one bf16 token, else two; one more with accumulate.
 */
typedef struct {
    int T, clamp_len, n_rows, accumulate;
    float scale;
    const txl_paged* mem;
    txl_view q, k_new, v_new, out;
    const int* counts;
    const float* u;
    const float* v_bias;
    const void* r;
    int64_t ld_r;
    void* workspace;
    size_t workspace_bytes;
    void* stream;
} txl_rel_attn_paged_args;
txl_status txl_rel_attn_paged(const txl_rel_attn_paged_args* args);

/* Bytes of device workspace txl_rel_attn_paged needs for n_rows distances (min(n_rows, clamp_len + 1) are enough): mostly
 * B*H*T floats a distance (not for one bf16 token), with accumulate H*T floats a slot of the pool (of B * max_pages pages, where those
 * are fewer), and parts of the sums (1280 T rows of D floats).  0 for an invalid shape. */
size_t txl_rel_attn_paged_workspace_size(const txl_paged* mem, int T, int n_rows, int accumulate);

/*
 * txl_paged_evict -- cut every sequence to `keep` positions: of a sequence with more, the length[b] - keep slots of
 * the least weight leave (of equal weights the older positions; NaN counts as the largest weight), but none of the last
 * `recent` positions (those >= next_pos[b] - recent).  The survivors in slots >= keep move, in order, into the
 * slots that became free in front (keys, values, position, weight), and length[b] = keep.  Other slots are left as
 * they were; next_pos does not change, so later tokens keep their distances.  keep >= 1, 0 <= recent <= keep.
 *   workspace : device scratch, 16-byte aligned, of txl_paged_evict_workspace_size(mem) bytes.
 * A sequence that has a slot without a page is left as it was.  Two launches.
 */
txl_status txl_paged_evict(const txl_paged* mem, int keep, int recent, void* workspace, size_t workspace_bytes,
                           void* stream);

/* Bytes of device workspace txl_paged_evict needs: two ints a sequence and slot of half the sequence's capacity (max_pages * page_len,
 * which the number of blocks that a sequence is given follows too: a table no wider than the sequences need serves both). */
size_t txl_paged_evict_workspace_size(const txl_paged* mem);

/*
 * 4-bit weights: a matrix W [k][n] held as codes of 4 bits; each column's entries k in groups of 32, 64 or 128 (the last
 * group shorter) share
 *     lo   = the largest bf16 that is not above the group's least entry
 *     step = the smallest bf16 that is not below (most - lo) / 15
 *     c    = the integer nearest to (w - lo) / step, ties to even (0 where step = 0)
 * and stand for w' = lo + step c (differences and quotients in double precision).  A group with a NaN or an infinity, or
 * whose step is not finite, stands for NaN throughout.
 *   data : device, 16-byte aligned, txl_q4_bytes(k, n, group) bytes: the codes as the kernels' lanes read them (64 columns
 *          by 64 k in 2 KB), then the groups' parameters.
 */
typedef struct {
    void* data;
    int k, n;
    int group;
} txl_q4;

/* Bytes of a matrix of 4-bit weights (0 for an invalid shape): k, n >= 1 and at most 2^21, group 32, 64 or 128. */
size_t txl_q4_bytes(int k, int n, int group);

/* Quantise device bf16 W [k][ld_w] (columns 0 .. n-1 are read; any alignment) into w->data. */
txl_status txl_q4_quantise(const txl_q4* w, const void* W, int64_t ld_w, void* stream);

/* What the codes stand for, rounded to bf16 once, into device bf16 W [k][ld_w] (columns 0 .. n-1 are written). */
txl_status txl_q4_expand(const txl_q4* w, void* W, int64_t ld_w, void* stream);

/*
 * txl_linear_q4 -- Y = X W' for bf16 X [m][ld_x] (columns 0 .. k-1 are read) and 4-bit weights: txl_linear with a quarter
 * of the weights' bytes, for the projections of a generated token.  Y bf16 [m][ld_y], columns 0 .. n-1 are written.
 * Up to 128 rows, and more of an X that txl_linear does not take (misaligned): 16 rows at a time straight from the codes
 * (products of the bf16 x and the exact codes, fp32 sums, one rounding; an entry whose fp32 sums are not finite is computed
 * again in double precision, so that any finite X and weights give the product, slower).  Every 16 rows expand the codes anew: from
 * about a hundred rows on txl_linear with the bf16 weights is faster.  Otherwise the weights are expanded to bf16 in the workspace and txl_linear's kernel runs.
 *   workspace : device scratch, 16-byte aligned, of at least txl_linear_q4_workspace_size(m, w) bytes (TXL_ERR_WORKSPACE;
 *            may be NULL when that is 0).  Calls that share a workspace must not overlap on the GPU.
 * Limits: m >= 0 (0: nothing to do), m <= 2^19; ld_x >= k, ld_y >= n.  err_flag as txl_linear.
 */
txl_status txl_linear_q4(int m, const txl_q4* w, const void* X, int64_t ld_x, void* Y, int64_t ld_y, void* workspace,
                         size_t workspace_bytes, int* err_flag, void* stream);

/* txl_linear_q4 with its arguments in one struct, for bindings that pay per argument. */
typedef struct {
    const txl_q4* w;
    const void* X;
    int64_t ld_x;
    void* Y;
    int64_t ld_y;
    void* workspace;
    size_t workspace_bytes;
    int* err_flag;
    void* stream;
    int m;
} txl_linear_q4_args;
txl_status txl_linear_q4_call(const txl_linear_q4_args* args);

/* Bytes of device workspace txl_linear_q4 needs: 0 for m <= 128, else 2 k (n rounded up to a multiple of 8). */
size_t txl_linear_q4_workspace_size(int m, const txl_q4* w);

/*
 * Checked build.  libtxl_checked.so is this library compiled with -DTXL_CHECKED (the package builds
 * it on request: transformer_xl_relative_gb300/_build.py --checked; the binding loads it when the
 * environment variable TXL_CHECKED is 1).  Its kernels range-check the indices they compute before
 * using them (the key row of every TMA key/value tile of the fused attention, the memory ring slot
 * of every key in the other attention kernels and of every pushed position, the remapped r row):
 * an index outside its range is counted in a device counter owned by the library and replaced by a
 * safe one, so the call completes (its results are then meaningless) and nothing traps or waits.
 * It stands in for a memory checker; the pages have no counterpart.
 *   txl_checked_build        : 1 in the checked build, 0 otherwise.
 *   txl_range_errors         : failed checks since the library was loaded or last cleared, into the
 *                              host int *count.  Synchronizes the current device (a debugging call).
 *                              TXL_ERR_UNSUPPORTED (and 0) in the normal build.
 *   txl_range_errors_clear   : resets the counter (synchronizes the current device).
 *   txl_selftest_range_check : enqueues one failing and one passing check on `stream`; the counter
 *                              gains exactly one.  TXL_ERR_UNSUPPORTED in the normal build.
 */
int txl_checked_build(void);
txl_status txl_range_errors(int* count);
txl_status txl_range_errors_clear(void);
txl_status txl_selftest_range_check(void* stream);

/* Self-test of the bounded waits used by every kernel: launches one CTA that waits on an
 * mbarrier nothing will signal, gives up after timeout_us microseconds (1 .. 10^7), writes
 * TXL_ERR_TIMEOUT to the device int err_flag and returns.  The context stays usable. */
txl_status txl_selftest_wait_timeout(int* err_flag, unsigned timeout_us, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TXL_H */
