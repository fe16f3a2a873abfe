/*
 * bqm.h - block-quantized matrix products on AMD Instinct MI355X (gfx950).  C ABI.
 *
 * What the library computes.  Decode streams every weight once per token, so its
 * speed is set by how many weight bytes cross HBM ("V100跑Qwen 27B：量化与KV Cache调优，
 * 从4到64 tok/s", lmnt.cn, section 1.2); the compact block formats Q4_0 and Q8_0 named
 * in that page's format table (section 4.1) cut those bytes.  Every product here is
 *     y = dequant(W) . x
 * with W stored in 32-weight blocks that each carry one binary16 scale d:
 *     Q4_0 weight = (nibble - 8) * d        Q8_0 weight = int8 * d.
 * A third format, MXFP4, carries a power of two per block and has its own products; and
 * bqm_route makes the expert ids and weights that the indexed products take.
 *
 * Interchange block layout (host or device bytes, what bqm_repack reads):
 *     Q4_0: 18 bytes per block = binary16 d (little endian), then 16 bytes; byte j
 *           holds weight j in its low nibble and weight j+16 in its high nibble.
 *     Q8_0: 34 bytes per block = binary16 d, then 32 signed bytes (weight j = byte j).
 *     A matrix W[N][K] is N rows of K/32 consecutive blocks.
 * The pages name the formats but do not print their bytes; this is the ggml layout.
 *
 * Packed (device) layout, what the products read: produced by bqm_repack, opaque to
 * callers except for its size, bqm_packed_bytes().  It separates the 16-byte aligned
 * code bytes from the scales so that every code load is a full 16-byte load.
 *
 * Conventions shared by every call:
 *   - Pointers are DEVICE pointers unless stated; the caller owns all memory.  The
 *     library allocates nothing and frees nothing (qmv_id_sum_noalloc keeps its slot rows
 *     in a fixed device array that is part of the library); work is queued on `stream` (a HIP
 *     stream; 0 = the null stream) and the call returns without synchronizing (only
 *     bqm_chain_prepare and bqm_chain_status wait, as their entries say).
 *   - Argument errors are found on the host before anything is launched: the call
 *     returns a non-zero bqm_status and leaves every output untouched.  A failed launch
 *     returns BQM_E_LAUNCH.  Faults inside a kernel surface at the caller's next
 *     synchronization, as for any HIP kernel.
 *   - Sizes may be zero (nothing is launched, except that N > 0 with K = 0 writes
 *     zeros, the value of an empty sum).  K must be a multiple of 32.
 *   - Pointers passed to the products must be 16-byte aligned (torch allocations are).
 *   - Outputs must not alias inputs (but for the linear layers' mul and residual).  Results are
 *     deterministic: no atomic updates of data, a fixed summation order, the same bits on every run
 *     with the same launch.
 *   - Host-side state, all safe to use from several threads: per device, the compute-unit
 *     count and the device address of qmv_id_sum_noalloc's array (cached once); per kernel,
 *     whether its static local memory fits (checked once); per workspace prepared by
 *     bqm_chain_prepare, whether the chain has a waiting GEMV (under a mutex).
 *   - Floating-point outputs are fp32 and satisfy, per output,
 *         |y - y_exact| <= 1e-3 * sum_i |w_i * x_i|
 *     (y_exact in exact arithmetic); integer and byte outputs are exact.
 */
#ifndef BQM_H
#define BQM_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  BQM_OK = 0,
  BQM_E_NULL = 1,        /* a required pointer is NULL                          */
  BQM_E_SHAPE = 2,       /* negative size, K % 32 != 0, or a size over a limit  */
  BQM_E_ALIGN = 3,       /* a pointer is not 16-byte aligned                    */
  BQM_E_UNSUPPORTED = 4, /* an unknown or refused format, type, score, activation */
  BQM_E_LAUNCH = 5       /* the HIP runtime refused a launch                    */
} bqm_status;

/* Block formats.  BQM_MXFP4 is taken by bqm_packed_bytes, bqm_repack, bqm_unpack, bqm_embed, bqm_linear
 * and bqm_linear_grouped, and has products of its own (the *_mxfp4 calls); the other calls with a fmt
 * argument refuse it with BQM_E_UNSUPPORTED. */
typedef enum { BQM_Q4_0 = 2, BQM_Q8_0 = 8, BQM_MXFP4 = 39 } bqm_fmt;

/* Element types of float rows (router logits, the rows of the MXFP4 quantizer and of the layers). */
typedef enum { BQM_F32 = 0, BQM_F16 = 1, BQM_BF16 = 30 } bqm_type;

/* Activations of bqm_linear and bqm_linear_grouped: z, max(z, 0), z / (1 + exp(-z)), z times the
 * normal distribution's share below z, and its tanh form z / (1 + exp(-2 sqrt(2 / pi) (z + 0.044715 z^3))). */
typedef enum { BQM_ACT_NONE = 0, BQM_ACT_RELU = 1, BQM_ACT_SILU = 2, BQM_ACT_GELU = 3, BQM_ACT_GELU_TANH = 4 } bqm_act;

/* Largest M accepted by qmv_q4_0 / qmv_q8_0, the small-batch decode width. */
#define BQM_QMV_MAX_M 8
/* Limits of qmv_id: token count, experts per token, number of experts (the per-expert
 * slot tables are built in LDS). */
#define BQM_QMV_ID_MAX_T 64
#define BQM_QMV_ID_MAX_TOPK 32
#define BQM_QMV_ID_MAX_E 4096
/* Token limit of qmm_id (top_k and E as for qmv_id). */
#define BQM_QMM_ID_MAX_T 16384

/* Bytes of the packed layout of a rows x K matrix in format fmt (0 for an unknown
 * format or a K that is not a multiple of 32).  Host function, no device work. */
size_t bqm_packed_bytes(int fmt, int64_t rows, int64_t K);

/* One-time layout transform: interchange blocks (w_interchange, rows x K/32 blocks,
 * 2-byte aligned) -> packed layout (w_packed, bqm_packed_bytes(fmt, rows, K) bytes,
 * 16-byte aligned).  Every byte of the packed buffer is written.  Precedent: weights
 * re-laid out once for the unit that runs them, like the interleaved repack on the page
 * "ik_llama.cpp 老工作站多 GPU 部署 Qwen3-235B-A22B 实战指南" (nxmr.cn), section on -rtr. */
int bqm_repack(int fmt, const void* w_interchange, void* w_packed, int64_t rows, int64_t K,
               hipStream_t stream);

/* Inverse of bqm_repack (packed -> interchange), byte exact.  For tests and export. */
int bqm_unpack(int fmt, const void* w_packed, void* w_interchange, int64_t rows, int64_t K,
               hipStream_t stream);

/* Decode GEMV and small-batch GEMV ("V100跑Qwen 27B" page, section 1.2: every weight read
 * once per token):
 *     Y[m][n] = sum_k dequant(W)[n][k] * X[m][k],   0 <= m < M <= 8, 0 <= n < N.
 * w_packed: packed N x K matrix.  X: fp32 [M][K] row-major.  Y: fp32 [M][N] row-major.
 * M = 0 or N = 0: nothing to do.  M > 8, or one workgroup's share of the rows reaching
 * 2 GiB of codes: BQM_E_SHAPE.  (A chain of one GEMV: see qmv_chain.) */
int qmv_q4_0(const void* w_packed, const float* X, float* Y, int M, int64_t N, int64_t K,
             hipStream_t stream);
int qmv_q8_0(const void* w_packed, const float* X, float* Y, int M, int64_t N, int64_t K,
             hipStream_t stream);

/* Expert-indexed GEMV, the mul_mat_id of the page "ik_llama.cpp 老工作站多 GPU 部署
 * Qwen3-235B-A22B 实战指南" (nxmr.cn), background and split-mode sections: a 3D expert
 * tensor W[E][N][K] and per-token expert ids.
 *     e = ids[t][s];  Y[t][s][n] = sum_k dequant(W)[e][n][k] * x_ts[k]
 *     x_ts = X + t * x_tok_stride + s * x_slot_stride      (strides in floats)
 * x_slot_stride = 0 broadcasts one input per token (gate/up projections); = K gives each
 * slot its own input (down projection).  A negative id marks a padding slot: its Y row is
 * written with zeros.  An id >= E is a contract violation: its Y row is filled with NaN
 * and nothing outside the arrays is read.  Each selected expert's rows are streamed once
 * per group of the slots routed to it: groups of up to 4 (fp32 vector products), or from
 * T >= 8 tokens with K a multiple of 128 groups of up to 16 (bf16 matrix-core products with
 * each input split into two bf16 parts but for a remainder below 2^-14 |x|; the result
 * meets the same 1e-3 * sum |w x| bound for inputs below 2^86 in magnitude).
 * w_packed: the expert tensor packed as ONE matrix of E*N rows (bqm_repack with
 * rows = E*N).  ids: int32 [T][top_k], device memory.  Y: fp32 [T][top_k][N].
 * fmt: BQM_Q4_0 or BQM_Q8_0.  Limits: T <= 64, top_k <= 32, E <= 4096. */
int qmv_id(int fmt, const void* w_packed, int E, int64_t N, int64_t K, const int32_t* ids, int T,
           int top_k, const float* X, int64_t x_tok_stride, int64_t x_slot_stride, float* Y,
           hipStream_t stream);

/* Fused expert gate+up, the fused MoE path (`-fmoe`, `fused_moe 1`) of the page
 * "ik_llama.cpp 老工作站多 GPU 部署 Qwen3-235B-A22B 实战指南" (nxmr.cn), recommended-command
 * section.  The page names the path without defining it; read as the SwiGLU feed-forward
 * of the models it runs:
 *     g = W_gate[e] x_ts,  u = W_up[e] x_ts,  Y[t][s][n] = silu(g[n]) * u[n],
 *     silu(z) = z / (1 + exp(-z))
 * One pass: each selected expert's gate and up rows are streamed once per group of its
 * slots (groups as for qmv_id), both sums share every input read.  w_gate and w_up: two expert
 * tensors of the same format and shape, each packed as one matrix of E*N rows.  Everything
 * else (ids, strides, padding and out-of-range ids, limits, errors) as qmv_id. */
int qmv_id_gate_up(int fmt, const void* w_gate, const void* w_up, int E, int64_t N, int64_t K,
                   const int32_t* ids, int T, int top_k, const float* X, int64_t x_tok_stride,
                   int64_t x_slot_stride, float* Y, hipStream_t stream);

/* Expert-indexed GEMV with the router-weighted sum over each token's slots: the output of
 * a mixture-of-experts feed-forward layer (the top-k routed experts of the page
 * "ik_llama.cpp 老工作站多 GPU 部署 Qwen3-235B-A22B 实战指南" (nxmr.cn), background
 * section), its small decode-time steps merged as the "llama.cpp-v100" README
 * (shadowgraph.io) describes in its kernels-and-runtime list: the weighting is done in the
 * product's store, the sum by one small kernel after it.  Read as
 *     Y_slots[t][s][n] = weights[t][s] * sum_k dequant(W)[e][n][k] * x_ts[k]
 *     Y[t][n]          = sum_{s < top_k} Y_slots[t][s][n]     (fp32, s ascending)
 * with e, x_ts, padding and out-of-range ids as in qmv_id: a padding slot's row is 0 (it
 * adds 0), an id >= E gives a NaN row (Y[t][n] is NaN).  Deterministic.
 * weights: fp32 [T][top_k], 4-byte aligned.  Y_slots: fp32 [T][top_k][N] (device memory
 * the caller owns; written as qmv_id's Y, scaled by the weights).  Y: fp32 [T][N], 16-byte
 * aligned, not overlapping Y_slots.  top_k = 0 writes Y = 0.  Limits and status codes as
 * qmv_id; a null or misaligned weights pointer: BQM_E_NULL / BQM_E_ALIGN. */
int qmv_id_sum(int fmt, const void* w_packed, int E, int64_t N, int64_t K, const int32_t* ids,
               const float* weights, int T, int top_k, const float* X, int64_t x_tok_stride,
               int64_t x_slot_stride, float* Y_slots, float* Y, hipStream_t stream);

/* qmv_id_sum for callers that cannot allocate device memory (code being captured into a HIP
 * graph, tight serving loops, harnesses that forbid hipMalloc): the same computation and
 * results as qmv_id_sum, without the Y_slots argument.  The weighted slot rows are kept in a
 * device array inside the library, BQM_NOALLOC_SLOT_FLOATS floats (4 MiB) per GPU, held
 * from the first call on that GPU until the process ends; the call itself allocates
 * nothing.  T * top_k * N above BQM_NOALLOC_SLOT_FLOATS: BQM_E_SHAPE.  Every call on one GPU
 * uses that GPU's array: calls that overlap in time on one GPU (other streams, other host
 * threads) race and must not be issued.  Other arguments, limits and status codes as
 * qmv_id_sum; BQM_E_LAUNCH also if the array's address cannot be obtained. */
#define BQM_NOALLOC_SLOT_FLOATS (1 << 20)
int qmv_id_sum_noalloc(int fmt, const void* w_packed, int E, int64_t N, int64_t K,
                       const int32_t* ids, const float* weights, int T, int top_k, const float* X,
                       int64_t x_tok_stride, int64_t x_slot_stride, float* Y, hipStream_t stream);

/* ---- chains of GEMVs in one launch ----------------------------------------------------
 * Decode runs one GEMV after another, each reading the previous one's output (through
 * the layers' other operations); launching them one by one pays a kernel start and drain
 * per GEMV.  The pages remove that per-launch cost by capturing decode in graphs and fusing
 * operators (page "v100llm：专为NVIDIA V100 GPU打造的高性能大模型推理引擎" (zingnex.cn),
 * section 4) and by merging the many small decode operators ("llama.cpp-v100" README
 * (shadowgraph.io), kernels-and-runtime list); here the GEMVs of a decode step share one
 * persistent launch.  A chain runs a list of GEMVs in order in ONE launch: a GEMV marked `wait`
 * starts only after every earlier GEMV of the chain has finished and its outputs are
 * visible device-wide (so its x may be an earlier GEMV's y); the weights of the next GEMV
 * are already streaming while the previous one finishes.  Every GEMV of a chain has the
 * same batch M (1..8).  Same arithmetic and tolerance as qmv_q4_0 / qmv_q8_0. */
typedef struct bqm_gemv {
  const void* w_packed;  /* packed N x K matrix (device)                              */
  const float* x;        /* [M][K] fp32 inputs (device), row-major, 16-byte aligned   */
  float* y;              /* [M][N] fp32 outputs (device), row-major                   */
  int64_t N, K;          /* 1 <= N <= 2^30; 32 <= K <= BQM_CHAIN_MAX_K, K % 32 == 0   */
  int32_t fmt;           /* BQM_Q4_0 or BQM_Q8_0, the same for every GEMV of a chain  */
  int32_t wait;          /* nonzero: start after all earlier GEMVs of the chain       */
  int32_t M;             /* batch, 1..8, the same for every GEMV of a chain           */
  int32_t reserved;      /* set to 0                                                  */
} bqm_gemv;

/* Largest K of a chain GEMV.  The chain keeps a 64-byte table row per GEMV and the staged
 * inputs in the LDS of each workgroup: bqm_chain_prepare returns BQM_E_SHAPE when the table
 * leaves no room for 32 blocks of K per input row (about 1900 GEMVs at M = 1; the inputs of
 * a long K are then staged in chunks). */
#define BQM_CHAIN_MAX_K 32768

/* Device bytes of the workspace of an n-GEMV chain (0 if n < 1). */
size_t bqm_chain_workspace_bytes(int n);

/* Validates the n host-side descriptors, then writes them, the staging plan and a zeroed
 * synchronization header into `workspace` (device memory, bqm_chain_workspace_bytes(n)
 * bytes, 16-byte aligned, owned by the caller).  A set-up call: it synchronizes `stream`
 * before it returns, so `descs` may be freed afterwards.  Errors: BQM_E_SHAPE (sizes, M
 * differing between GEMVs, a chain too long for the LDS), BQM_E_NULL, BQM_E_ALIGN,
 * BQM_E_UNSUPPORTED (mixed or unknown formats), BQM_E_LAUNCH. */
int bqm_chain_prepare(const bqm_gemv* descs, int n, void* workspace, hipStream_t stream);

/* Runs a prepared chain in one launch on `stream`; fmt, M and n must be those it was
 * prepared with (the kernel checks fmt, n and the class of M against the workspace and
 * otherwise computes nothing and records error 2).  A chain with a waiting GEMV runs as a
 * cooperative launch (all workgroups resident at once); one without (independent GEMVs,
 * split between the workgroups together) as an ordinary launch.  The workspace is left
 * ready for the next call; calls sharing one workspace must not overlap in time. */
int qmv_chain(int fmt, int M, void* workspace, int n, hipStream_t stream);

/* Synchronizes `stream` and returns the chain's error word: 0 = ok, 1 = a device-wide
 * wait timed out (results invalid; prepare again), 2 = fmt/M/n mismatch, -1 = copy failed. */
int bqm_chain_status(const void* workspace, hipStream_t stream);

/* Activation quantizer for the prefill product.  The prefill kernels the pages describe
 * work on Q8_0-format blocks ("llama.cpp-v100" README (shadowgraph.io): its SM70 kernels
 * adapted to Q8_0, computing-kernels item); the activations are read as taking the same
 * 32-wide int8 block shape with an fp32 scale, per row m and block b, in IEEE single
 * precision:  a = max_j |x_j|;  dx = a / 127 (correctly rounded);  dx == 0 gives all-zero
 * codes and dx = +0; otherwise Xq_j = round_half_away_from_zero(x_j / dx) clamped to
 * [-127, 127].  X: fp32 [M][K];  Xq: int8 [M][K];  dx: fp32 [M][K/32].  Bit exact. */
int bqm_quantize_q8_act(const float* X, int8_t* Xq, float* dx, int64_t M, int64_t K,
                        hipStream_t stream);

/* Prefill product with Q8_0 weights (the llama-bench pp512 shape of the page "llama.cpp
 * 0.9.0" analysis (ai-v5 LLMNews), section 2 table):
 *     isum[m][n][b] = sum_{j<32} qw[n][32b+j] * Xq[m][32b+j]        exact int32 (int8 MFMA)
 *     Y[m][n]       = sum_b (d_w[n][b] * dx[m][b]) * isum[m][n][b]    fp32, b ascending
 * The scale product d_w * dx comes from the matrix cores as an fp32 sum of six exact
 * partial products (d_w and dx split into bf16 parts); it may differ from the correctly
 * rounded product in the last bits, well within the float tolerance.
 * w_packed: packed Q8_0 N x K matrix.  Xq, dx: from bqm_quantize_q8_act.  Y: fp32 [M][N].
 * Operands are addressed with 32-bit offsets: M*K or N*K code bytes of 2 GiB or more give
 * BQM_E_SHAPE. */
int qmm_q8_0(const void* w_packed, const int8_t* Xq, const float* dx, float* Y, int64_t M,
             int64_t N, int64_t K, hipStream_t stream);

/* Prefill product with Q4_0 weights (the pp512 prompt-processing rows of Q4_0 (QAT)
 * models in the same section of the "llama.cpp 0.9.0" analysis page): the definition of
 * qmm_q8_0 with qw the nibble - 8 (weight j of a block in the low nibble of code byte j,
 * weight j + 16 in the high one).  The nibbles are widened to int8 on the way into local
 * memory, so the integer sums are exact and the scaling is that of qmm_q8_0.
 * w_packed: packed Q4_0 N x K matrix; the rest as for qmm_q8_0.  Same status codes. */
int qmm_q4_0(const void* w_packed, const int8_t* Xq, const float* dx, float* Y, int64_t M,
             int64_t N, int64_t K, hipStream_t stream);

/* Expert-indexed prefill product: the prefill expert matmul of the "llama.cpp-v100" README
 * (shadowgraph.io), kernels-and-runtime list, with qmv_id's routing (mul_mat_id, page
 * "ik_llama.cpp 老工作站多 GPU 部署 Qwen3-235B-A22B 实战指南" (nxmr.cn)):
 *     e = ids[t][s],  r = t * x_tok_rows + s * x_slot_rows,
 *     Y[t][s][n] = sum_b d_w[e][n][b] * dx[r][b] * sum_j qw[e][n][32b+j] * Xq[r][32b+j]
 * i.e. qmm_q8_0 / qmm_q4_0 of input row r with expert e's matrix, integer block sums exact,
 * the scaling as in qmm_q8_0.  The slots of each expert are gathered into row tiles (in
 * slot order), so each expert's rows are streamed once per 64 of its slots.
 * w_packed: expert tensor of format fmt packed as ONE matrix of E*N rows.  ids: int32
 * [T][top_k].  Xq, dx: quantized activations from bqm_quantize_q8_act, rows as indexed
 * above (x_tok_rows = 1, x_slot_rows = 0: one row per token; top_k, 1: one per slot).
 * Y: fp32 [T][top_k][N].  Padding slots (negative id) give zero rows, ids >= E NaN rows.
 * Limits: T <= BQM_QMM_ID_MAX_T, top_k <= 32, E <= 4096; the input rows the slots address,
 * and one expert's codes, below 2 GiB (else BQM_E_SHAPE). */
int qmm_id(int fmt, const void* w_packed, int E, int64_t N, int64_t K, const int32_t* ids, int T,
           int top_k, const int8_t* Xq, const float* dx, int64_t x_tok_rows, int64_t x_slot_rows,
           float* Y, hipStream_t stream);

/* ---- MXFP4 ----------------------------------------------------------------------------
 * The OCP microscaling format with 4-bit elements, the one block format that the matrix cores
 * of gfx950 multiply as it is stored: 32 e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 for the low
 * three bits, negative with the fourth) under one e8m0 scale byte e that stands for 2^(e - 127),
 * e = 255 for NaN.  Interchange block: 17 bytes, e first, then 16 bytes of which byte j holds code
 * j in its low nibble and code j + 16 in its high one (any alignment).  Packed: as for the other
 * formats, written by bqm_repack and also by bqm_quantize_mxfp4; one layout serves weights and
 * activations.  4.25 bits per weight, rows padded to 16 and K to 128 (codes) and 512 (scales). */

/* Rows of floats -> packed MXFP4.  Per row and block of 32, in the values of x_type: m = max |x|;
 * the scale is 2^s with s = floor(log2 m) - 2, at least -127 (m = 0: -127); each code is the e2m1
 * value nearest to x / 2^s, ties to the even code, values beyond 6 to 6, signs kept.  A block with
 * an infinity or a NaN gets the scale byte 255 and codes 0.  Bit exact.
 * X: [rows][K] of x_type (bqm_type) with x_stride elements from row to row; X 16-byte aligned,
 * rows 16-byte aligned or not.  packed: bqm_packed_bytes(BQM_MXFP4, rows, K) bytes, all written.
 * x_stride < K: BQM_E_SHAPE; an unknown type: BQM_E_UNSUPPORTED. */
int bqm_quantize_mxfp4(int x_type, const void* X, int64_t x_stride, void* packed, int64_t rows, int64_t K,
                       hipStream_t stream);

/* Packed MXFP4 -> rows of floats, each value rounded once to y_type (exact in fp32 and bf16 but for
 * scales above 2^125 whose values pass the type's range and become infinities; the values of a
 * block with scale byte 255 are NaN).  Y: [rows][K] with y_stride elements from row to row, the
 * elements between rows are left as they are. */
int bqm_dequantize_mxfp4(const void* packed, int y_type, void* Y, int64_t y_stride, int64_t rows, int64_t K,
                         hipStream_t stream);

/* Decode GEMV and small-batch GEMV with MXFP4 weights, qmv_q4_0's counterpart:
 *     Y[m][n] = sum_k dequant(W)[n][k] * X[m][k],   0 <= m < M <= 8, 0 <= n < N,   X and Y fp32.
 * Same tolerance and status codes; each input counts exactly down to a resolution of 2^-133, and each
 * weight as it is, also those beyond fp32's largest number (scales above 2^125).  K above BQM_MXFP4_MAX_K,
 * N above 2^29: BQM_E_SHAPE. */
#define BQM_MXFP4_MAX_K (1 << 23)
int qmv_mxfp4(const void* w_packed, const float* X, float* Y, int M, int64_t N, int64_t K, hipStream_t stream);

/* Prefill product of two packed MXFP4 matrices, qmm_q4_0's counterpart:
 *     Y[m][n] = sum_k dequant(W)[n][k] * dequant(X)[m][k]                 fp32
 * w_packed: packed N x K.  x_packed: packed M x K, from bqm_quantize_mxfp4.  Products of codes are
 * exact and block scales are powers of two; the sums are fp32.  Any M from one token on.  A block
 * of either operand with scale byte 255 makes the outputs of its row NaN.  K above
 * BQM_MXFP4_MAX_K: BQM_E_SHAPE (qmm_id_mxfp4 too, and where the activations' codes reach 2 GiB), and so
 * are outputs that take 2^22 tiles of 256 x 256 or more. */
int qmm_mxfp4(const void* w_packed, const void* x_packed, float* Y, int64_t M, int64_t N, int64_t K, hipStream_t stream);

/* Expert-indexed qmm_mxfp4, qmm_id's counterpart:
 *     e = ids[t][s],  r = t * x_tok_rows + s * x_slot_rows,
 *     Y[t][s][n] = sum_k dequant(W)[e][n][k] * dequant(X)[r][k]
 * w_packed: expert tensor packed as ONE matrix of E*N rows.  x_packed: packed x_rows x K; every
 * row that the slots address lies below x_rows (else BQM_E_SHAPE).  Padding slots (negative id) give
 * zero rows, ids >= E NaN rows.  Limits: T <= BQM_QMM_ID_MAX_T, top_k <= 32, E <= 4096. */
int qmm_id_mxfp4(const void* w_packed, int E, int64_t N, int64_t K, const int32_t* ids, int T, int top_k,
                 const void* x_packed, int64_t x_rows, int64_t x_tok_rows, int64_t x_slot_rows, float* Y,
                 hipStream_t stream);

/* ---- routing to experts ----------------------------------------------------------------
 * The ids and weights that qmv_id, qmv_id_gate_up, qmv_id_sum, qmm_id and qmm_id_mxfp4 take, from
 * a router's logits (the top-k routed experts of the page "ik_llama.cpp 老工作站多 GPU 部署
 * Qwen3-235B-A22B 实战指南" (nxmr.cn), background section).  Per token:
 *     score[e] = softmax over the E logits, or 1 / (1 + exp(-logit[e]))
 *     value[e] = logit[e] without a bias, score[e] + bias[e] with one
 * n_group > 1: the experts form n_group runs of E / n_group; a group's value is the sum of its
 * group_top (1 or 2) largest value[e] (of score[e] where group_top is 2 and there is no bias), and
 * only the experts of the topk_group groups with the largest take part.  The top_k experts with the
 * largest value are chosen, in descending order, ties (of groups too) to the lower index:
 *     ids[t][s] = e,   weights[t][s] = scale * score[e]  (/ the sum of the chosen scores with renorm)
 * Values are compared in 64 bits, so that neighbours come out in the order of the real numbers.
 * An expert whose logit (or bias) is -infinity is never chosen; slots that no expert is left
 * for get id -1 (a padding slot of the products) and weight 0.  Chosen scores that sum to 0 give
 * weights 0.  A NaN logit or bias, or with softmax a logit of +infinity, gives that token the ids
 * 0, 1, ... and NaN weights.
 * logits: [T][E] of l_type (bqm_type) with l_stride >= E elements from row to row.  bias: fp32 [E] or
 * NULL.  ids: int32 [T][top_k], weights: fp32 [T][top_k].  All pointers aligned to 16 bytes but
 * bias (4).  Limits: E <= 4096, top_k <= 32, n_group <= BQM_ROUTE_MAX_GROUPS dividing E,
 * 1 <= topk_group <= n_group, group_top 1 or 2 and at most E / n_group where n_group > 1,
 * T <= BQM_ROUTE_MAX_T.  E = 0: every id -1.  Unknown score or type: BQM_E_UNSUPPORTED. */
typedef enum { BQM_SOFTMAX = 0, BQM_SIGMOID = 1 } bqm_score;
#define BQM_ROUTE_MAX_GROUPS 64
#define BQM_ROUTE_MAX_T (1 << 22)
int bqm_route(int score, int l_type, const void* logits, int64_t l_stride, const float* bias, int T, int E,
              int n_group, int topk_group, int group_top, int top_k, int renorm, float scale, int32_t* ids,
              float* weights, hipStream_t stream);

/* ---- layers on float rows ---------------------------------------------------------------
 * What a model does around the products: tokens to rows, and a projection with everything that follows
 * it up to the next one, on rows as they are (no quantization of activations), in one launch each. */

/* Rows of a packed table by token id, times a scale (the embeddings, which the byte counts of the page
 * "V100跑Qwen 27B：量化与KV Cache调优，从4到64 tok/s" (lmnt.cn), section 4.1, leave out: gathered, not streamed):
 *     Y[t][k] = scale * dequant(W)[ids[t]][k]
 * computed in fp32 and rounded once to y_type.  fmt: any of the three.  w_packed: packed rows x K.  ids:
 * int32 [T]; a negative id gives a row of zeros, an id >= rows a row of NaN.  Y: [T][K] of y_type with
 * y_stride >= K elements from row to row, those between rows are left as they are.  Only the product has to be
 * a number of fp32: an MXFP4 weight beyond its largest number and a scale below its smallest count as they
 * are.  rows, T and K up to 2^30, y_stride too. */
int bqm_embed(int fmt, const void* w_packed, int64_t rows, int64_t K, const int32_t* ids, int64_t T, float scale,
              int y_type, void* Y, int64_t y_stride, hipStream_t stream);

/* Linear layer, from one token to long prompts:
 *     z[m][n] = bias[n] + sum_k dequant(W)[n][k] * X[m][k]
 *     Y[m][n] = act(z[m][n]) * mul[m][n] + residual[m][n]
 * fmt: any of the three.  X: [M][K] of x_type.  bias: fp32 [N] or NULL (0).  act: bqm_act.  mul, residual:
 * [M][N] of y_type, or NULL (1 and 0); mul makes a gated feed-forward's silu(gate) * up of the gate's
 * product.  Y: [M][N] of y_type; the elements between its rows are left as they are.  mul and residual
 * may be Y itself (same address and stride): each element is read before it is written.  Rows lie x_stride,
 * mul_stride, res_stride and y_stride elements apart, at least their length (a stride without a pointer is
 * ignored); X's rows have to start at multiples of 16 bytes, the others need not, and a bias at one of 4.
 * Arithmetic: codes and rows meet as they are (fp32 rows in three bf16 parts, exact down to a resolution of
 * 2^-133), block scales in fp32, sums in fp32; one rounding to y_type at the end.  z meets the tolerance of
 * the products for inputs below 2^116 in magnitude (a block's sum without its scale has to stay a
 * number of fp32).  K = 0: the sum is 0.  K and x_stride up to BQM_LINEAR_MAX_K, the other strides up to 2^30.
 * Sizes with ceil(M / 32) * ceil(N / 128) < 2^22 are taken; above that a call may need more workgroups than a
 * launch holds: BQM_E_SHAPE. */
#define BQM_LINEAR_MAX_K (1 << 20)
int bqm_linear(int fmt, const void* w_packed, int x_type, const void* X, int64_t x_stride, const float* bias, int act,
               const void* mul, int64_t mul_stride, const void* residual, int64_t res_stride, int y_type, void* Y,
               int64_t y_stride, int64_t M, int64_t N, int64_t K, hipStream_t stream);

/* The linear layer for rows that lie in the order of their experts (the mixture-of-experts layer of the page
 * "ik_llama.cpp 老工作站多 GPU 部署 Qwen3-235B-A22B 实战指南" (nxmr.cn), background section, after its tokens
 * were dealt to the experts): rows offsets[e] .. offsets[e + 1] - 1 are expert e's, any number of them, none
 * too, and take matrix e and bias e:
 *     z[r][n] = bias[e][n] + sum_k dequant(W)[e][n][k] * X[r][k],   Y as in bqm_linear.
 * w_packed: expert tensor packed as ONE matrix of E*N rows.  bias: fp32 [E][N] or NULL.  offsets: int32
 * [E + 1], device memory, not decreasing, from 0 or more up to R or less; rows of Y outside
 * offsets[0] .. offsets[E] are left as they are.  Offsets below 0 or above R count as 0 or R; where they
 * decrease, which rows of Y are written, and with what, is not defined (nothing outside Y's R rows is).
 * E <= BQM_QMV_ID_MAX_E.  Sizes with (min(E + R / 32, R) + 16) * ceil(N / 128) < 2^22 are taken: a group has row
 * tiles of its own, however few its rows.  The rest as bqm_linear with M = R. */
int bqm_linear_grouped(int fmt, const void* w_packed, int E, const int32_t* offsets, int x_type, const void* X,
                       int64_t x_stride, const float* bias, int act, const void* mul, int64_t mul_stride,
                       const void* residual, int64_t res_stride, int y_type, void* Y, int64_t y_stride, int64_t R,
                       int64_t N, int64_t K, hipStream_t stream);

/* Static English text for a status code. */
const char* bqm_strerror(int status);

#ifdef __cplusplus
}
#endif

#endif /* BQM_H */
