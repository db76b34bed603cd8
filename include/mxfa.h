/*
 * mxfa.h -- C ABI of libmxfa: MXFP8 block-scaled FlashAttention (forward and
 * backward) for NVIDIA GB300 (sm_103a), with its quantizers and the fused
 * RMSNorm+Quantize producer.
 *
 * Sources for what each call computes (web pages on one subject):
 *  [MX]   "Low-Precision FlashAttention-4: End-to-End Block-Scaled Attention
 *         on Blackwell" (kongchang.com), section "Why MXFP8" -- OCP MX: 32
 *         elements share one power-of-two (E8M0) scale, E4M3 payload.
 *  [TMEM] "MXFP8 FlashAttention-4 Hits 2.85 Petaflops in Meta's Production
 *         Training" (andresseo.expert), section "Inside the TMEM Bargain and
 *         Zero-Gather Jagged Pipeline" -- online P / dS quantization, square
 *         32x32 blocks for Q, K, dO in the backward pass, dQ reduction in
 *         FP16 with static scaling, split addressing for jagged inputs,
 *         fused RMSNorm / GEMM producers.
 *  [KDIM] "Meta's MXFP8 FlashAttention-4 kernel, tackling TMEM scale-factor
 *         constraints, hits up to 1.6x over BF16" (theclarity.today),
 *         paragraphs 1-3 -- scales along the MMA K dimension (D for Q and K,
 *         N for V); scales padded and permuted to 128-aligned layouts for TMA.
 *  [ITEMS] "Meta's FlashAttention-4 Achieves 2.85 PF/s with MXFP8 on Blackwell
 *         GPUs" (brifing.si), items 5 (jagged), 6 (backward), 7 (fused
 *         producers).
 *
 * Conventions for every call
 *  - All tensor pointers are DEVICE pointers owned by the caller; the library
 *    never allocates, frees or synchronises (except mxfa_get_device_status).
 *    Work is enqueued on the caller's stream (a cudaStream_t; 0 = legacy).
 *  - Attention tensors are token-major: x[token][head][d] with d contiguous
 *    (dense [B][S][H][D] is the varlen layout with B sequences of length S).
 *    D must be 128.
 *  - Payload pointers, scale pointers and bf16 outputs must be 16-byte
 *    aligned (else MXFA_ERR_MISALIGNED).
 *  - Arguments are checked before any launch; launch failures are reported
 *    as MXFA_ERR_CUDA.  Device-side failures (a bounded wait that expired,
 *    an index check that skipped an access) are recorded in a status word
 *    read by mxfa_get_device_status.  Nothing aborts the process.
 *
 * Scale-factor layouts
 *  compact (one E8M0 byte per block, logical order):
 *    ROW  [tokens][H*D/32]            1x32 along d
 *    COL  [sum ceil(len/32)][H*D]     32x1 along the tokens of a sequence
 *    SQ   [sum ceil(len/32)][H*D/32]  32x32 within a head
 *  packed (what the attention kernels read; rows padded per sequence to a
 *  multiple of 128 with value 0x7F, i.e. 2^0):
 *    tiles = sum over sequences of ceil(len/128); tile t of head h is entry
 *    (t * H + h).
 *    ROW  512-byte atom per entry: byte (r%32)*16 + (r/32)*4 + k for token r
 *         of the tile and d-block k  (the tensor core's 128x4 scale layout)
 *    COL  512-byte atom per entry: byte (d%32)*16 + (d/32)*4 + k for column d
 *         and 32-token block k of the tile
 *    SQ   16 bytes per entry: byte 4*k + c for token block k and d-block c
 */
#ifndef MXFA_H
#define MXFA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* mxfa_stream_t; /* same type as cudaStream_t */

typedef enum {
  MXFA_OK = 0,
  MXFA_ERR_INVALID_ARG = 1,   /* null pointer, bad size, bad enum        */
  MXFA_ERR_UNSUPPORTED = 2,   /* valid but not implemented (e.g. D!=128) */
  MXFA_ERR_MISALIGNED = 3,    /* pointer not 16-byte aligned             */
  MXFA_ERR_WORKSPACE_TOO_SMALL = 4,
  MXFA_ERR_CUDA = 5,          /* a CUDA call or kernel launch failed     */
  MXFA_ERR_TIMEOUT = 6,       /* a kernel's bounded wait expired         */
  MXFA_ERR_DEVICE_INDEX = 7   /* a kernel's index check skipped an access */
} mxfa_status;

typedef enum {
  MXFA_BLK_ROW = 0, /* 1x32 along d (MMA K = D: Q, K forward; V backward)    */
  MXFA_BLK_COL = 1, /* 32x1 along tokens of a sequence (MMA K = N: V forward) */
  MXFA_BLK_SQ = 2   /* 32x32, transpose-invariant (Q, K, dO backward)         */
} mxfa_block;

/* An MXFP8 operand as the attention kernels read it: E4M3 payload in the
 * source layout (compact, never padded) and E8M0 scales in the packed
 * layout of its block kind. */
typedef struct {
  const uint8_t* data;
  const uint8_t* sf;
} mxfa_mx;

/* Outputs of a quantizing call; sf_compact and sf_packed may be NULL. */
typedef struct {
  uint8_t* data;
  uint8_t* sf_compact;
  uint8_t* sf_packed;
} mxfa_mx_out;

/* The forward kernel moves its running row maximum only when it grows by
 * more than this many log2 units (O and l keep the stale maximum exactly). */
#define MXFA_FWD_RESCALE_THRESHOLD 8.0f

/* Options of the *_opts attention calls (the plain calls use the defaults).
 *  rescale_threshold  forward only: the running row maximum moves when it
 *          grows by more than this (log2 units, 0 <= t <= 8); 0 rescales at
 *          every increase.  P~ = 2^(s' - m) then stays below 2^t.  Default
 *          MXFA_FWD_RESCALE_THRESHOLD.
 *  p_scale MXFA_P_SCALE_BLOCK (default): each 32-element block of P gets the
 *          E8M0 scale of its own maximum (OCP rule).  MXFA_P_SCALE_CONST: one
 *          constant scale for every block ([ITEMS] item 4: constant scaling
 *          of softmax outputs, which lie in a known range): forward
 *          2^(ceil(t) - 8), so the largest possible P~, 2^ceil(t), maps to
 *          256 <= 448; backward 2^-8 (P <= 1 maps to <= 256).  Values below
 *          2^-9 of the scale round to zero. */
#define MXFA_P_SCALE_BLOCK 0
#define MXFA_P_SCALE_CONST 1
typedef struct {
  float rescale_threshold;
  int p_scale;
} mxfa_attn_opts;

const char* mxfa_status_string(mxfa_status s);
int mxfa_version(void);

/* Number of packed tiles: sum over sequences of ceil(len/128).  cu_seqlens
 * here is a HOST array of nseq+1 offsets; NULL means nseq sequences of
 * seqlen tokens.  Returns -1 on bad input. */
int64_t mxfa_packed_tiles(const int32_t* cu_seqlens_host, int nseq, int seqlen);
/* Bytes of a packed scale tensor for `tiles` packed tiles and H heads. */
size_t mxfa_sf_packed_bytes(mxfa_block blk, int64_t tiles, int H);

/* mxfa_quantize -- bf16 -> E4M3 payload + E8M0 scales ([MX]; orientation
 * per [KDIM] and [TMEM]).
 *  x          bf16 [tokens][H][D], D = 128
 *  blk        block kind
 *  cu_seqlens DEVICE int32[nseq+1] sequence offsets, or NULL for nseq
 *             sequences of max_seqlen tokens each (tokens = nseq*max_seqlen)
 *  max_seqlen longest sequence (sizes the grid)
 *  packed_tiles  mxfa_packed_tiles() of the same sequences (bounds the
 *             packed output; ignored when out->sf_packed is NULL)
 *  out        payload [tokens][H][D] and the compact and/or packed scales
 * Scale: floor(log2 amax) - 8 clamped to [0, 254]; payload RNE, saturating
 * at 448; a block holding Inf/NaN gets scale 0xFF and payload 0x7F. */
mxfa_status mxfa_quantize(const void* x, int64_t tokens, int H, int D, mxfa_block blk,
                          const int32_t* cu_seqlens, int nseq, int max_seqlen,
                          int64_t packed_tiles, const mxfa_mx_out* out, mxfa_stream_t stream);

/* mxfa_quantize_dual -- one read of x, two layouts: blk (MXFA_BLK_COL or
 * MXFA_BLK_SQ) into out, and MXFA_BLK_ROW into out_row, each byte for byte as
 * mxfa_quantize would write it ([ITEMS] item 7: quantization fused so that no
 * separate pass reads the tensor again).  COL + ROW serves V (forward, then
 * backward); SQ + ROW serves Q and K (backward, then forward).  Arguments as
 * mxfa_quantize; out_row and its payload are required, its scale pointers
 * nullable; another blk is MXFA_ERR_INVALID_ARG. */
mxfa_status mxfa_quantize_dual(const void* x, int64_t tokens, int H, int D, mxfa_block blk,
                               const int32_t* cu_seqlens, int nseq, int max_seqlen,
                               int64_t packed_tiles, const mxfa_mx_out* out,
                               const mxfa_mx_out* out_row, mxfa_stream_t stream);

/* mxfa_sf_pack -- compact scales -> packed scales for the same block kind,
 * values unchanged, padding rows 0x7F ([KDIM] paragraph 3, [ITEMS] item 5:
 * only the scale factors are scattered and padded; payload stays compact).
 * Arguments as mxfa_quantize. */
mxfa_status mxfa_sf_pack(const uint8_t* sf_compact, int64_t tokens, int H, int D, mxfa_block blk,
                         const int32_t* cu_seqlens, int nseq, int max_seqlen,
                         int64_t packed_tiles, uint8_t* sf_packed, mxfa_stream_t stream);

/* mxfa_sf_unpack -- packed scales -> compact scales: the inverse of
 * mxfa_sf_pack for every real row / block (padding bytes are not read).
 * It gives tests and tools a C-ABI round trip of the packed layout that the
 * tensor core reads; it is not on the training path.  Arguments as
 * mxfa_sf_pack with the roles of the two scale buffers exchanged. */
mxfa_status mxfa_sf_unpack(const uint8_t* sf_packed, int64_t tokens, int H, int D, mxfa_block blk,
                           const int32_t* cu_seqlens, int nseq, int max_seqlen,
                           int64_t packed_tiles, uint8_t* sf_compact, mxfa_stream_t stream);

/* mxfa_fwd -- dense forward ([KDIM] paragraphs 1-2, [TMEM]).
 *  q, k       ROW-quantized payload [B][S][H][128] + packed ROW scales
 *  v          COL-quantized payload + packed COL scales
 *  causal     mask key > query
 *  o          bf16 [B][S][H][128] (output)
 *  lse        fp32 [B][H][S] natural-log log-sum-exp (output)
 * P is quantized per 32 keys in registers; the row sum is taken before. */
mxfa_status mxfa_fwd(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v, int B, int S, int H,
                     int D, float softmax_scale, int causal, void* o, float* lse,
                     mxfa_stream_t stream);

/* mxfa_varlen_fwd -- jagged forward ([TMEM] split addressing, [ITEMS] 5).
 *  cu_seqlens_q/k  DEVICE int32[nseq+1]; q/o/lse follow cu_seqlens_q,
 *                  k/v follow cu_seqlens_k.  Lengths may be 0: a query
 *                  sequence whose key sequence is empty gets O = 0 and
 *                  lse = -inf (the empty softmax sum); an empty query
 *                  sequence writes nothing.  max_seqlen_k must be >= 1.
 *  ptiles_q/k      mxfa_packed_tiles() of the query / key sequences
 *  lse             fp32 [H][total_q]
 *  causal          top-left aligned (key index > query index masked) */
mxfa_status mxfa_varlen_fwd(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v,
                            const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int nseq,
                            int max_seqlen_q, int max_seqlen_k, int64_t total_q, int64_t total_k,
                            int64_t ptiles_q, int64_t ptiles_k, int H, int D, float softmax_scale,
                            int causal, void* o, float* lse, mxfa_stream_t stream);

/* mxfa_fwd_mxo, mxfa_varlen_fwd_mxo -- the forward passes above that also
 * emit O as MXFP8 for the output projection ([KDIM] paragraph 4: fused
 * producer and output epilogues).  The bf16 O they write is quantized in
 * 1x32 blocks along D, byte for byte as mxfa_quantize(MXFA_BLK_ROW)
 * quantizes that bf16 O:
 *  o_mx->data        E4M3 [tokens][H][128] (required, 16-byte aligned)
 *  o_mx->sf_compact  E8M0 [tokens][H * 4] (nullable, 4-byte aligned)
 *  o_mx->sf_packed   packed ROW atoms, ptiles_q * H * 512 bytes, rows past
 *                    a sequence's end 0x7F (nullable, 16-byte aligned)
 * Other arguments and errors as mxfa_fwd / mxfa_varlen_fwd; o_mx NULL is
 * MXFA_ERR_INVALID_ARG. */
mxfa_status mxfa_fwd_mxo(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v, int B, int S, int H,
                         int D, float softmax_scale, int causal, void* o, float* lse,
                         const mxfa_mx_out* o_mx, mxfa_stream_t stream);
mxfa_status mxfa_varlen_fwd_mxo(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v,
                                const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int nseq,
                                int max_seqlen_q, int max_seqlen_k, int64_t total_q,
                                int64_t total_k, int64_t ptiles_q, int64_t ptiles_k, int H, int D,
                                float softmax_scale, int causal, void* o, float* lse,
                                const mxfa_mx_out* o_mx, mxfa_stream_t stream);

/* mxfa_fwd_opts, mxfa_varlen_fwd_opts -- mxfa_fwd / mxfa_varlen_fwd with
 * options (see mxfa_attn_opts; NULL = defaults).  A threshold outside
 * [0, 8] or an unknown p_scale is MXFA_ERR_INVALID_ARG. */
mxfa_status mxfa_fwd_opts(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v, int B, int S, int H,
                          int D, float softmax_scale, int causal, const mxfa_attn_opts* opts,
                          void* o, float* lse, mxfa_stream_t stream);
mxfa_status mxfa_varlen_fwd_opts(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v,
                                 const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int nseq,
                                 int max_seqlen_q, int max_seqlen_k, int64_t total_q,
                                 int64_t total_k, int64_t ptiles_q, int64_t ptiles_k, int H, int D,
                                 float softmax_scale, int causal, const mxfa_attn_opts* opts,
                                 void* o, float* lse, mxfa_stream_t stream);

/* Workspace of the backward pass for total_q query tokens in nseq sequences:
 * one 2560-byte record per (64-query tile, head) -- the tile's scale atoms,
 * lse * log2(e) and Delta = rowsum(dO^ * O) -- for at most
 * ceil(total_q / 64) + nseq tiles, followed by the dQ accumulator
 * ([total_q][H][128], fp32 when dq_mode = 0, fp16 when 1). */
size_t mxfa_bwd_workspace_size(int64_t total_q, int nseq, int H, int D, int dq_mode);

/* mxfa_bwd -- dense backward, five GEMMs with recompute ([TMEM], [ITEMS] 6).
 *  q, k, dO   SQ-quantized payload + packed SQ scales (32x32 blocks serve
 *             both GEMM orientations)
 *  v          ROW-quantized payload + packed ROW scales
 *  o, dout    bf16 O and dO [B][S][H][128];  lse fp32 [B][H][S] from mxfa_fwd.
 *             Delta = rowsum(dO^ * O) takes the dequantized square-block dO^
 *             of dout_mx (the operand that also enters dP), so dout itself
 *             is checked but not read
 *  dq_mode    0: dQ reduced in fp32;  1: fp16 with static scale
 *             dq_static_scale (a power of two; partials are multiplied by it
 *             before the fp16 reduction and divided after)
 *  dq, dk, dv bf16 outputs [B][S][H][128]
 *  ws         caller-owned workspace of mxfa_bwd_workspace_size() bytes
 * P is recomputed from the square-block Q, K and lse, quantized 1x32 along
 * queries for dV; dS = P (dP - Delta) is quantized in 32x32 blocks. */
mxfa_status mxfa_bwd(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v, const mxfa_mx* dout_mx,
                     const void* o, const void* dout, const float* lse, int B, int S, int H, int D,
                     float softmax_scale, int causal, int dq_mode, float dq_static_scale, void* dq,
                     void* dk, void* dv, void* ws, size_t ws_bytes, mxfa_stream_t stream);

/* mxfa_varlen_bwd -- jagged backward; arguments as mxfa_varlen_fwd and
 * mxfa_bwd (lse [H][total_q]).  Keys of a sequence with no queries get
 * dK = dV = 0; queries of a sequence with no keys get dQ = 0. */
mxfa_status mxfa_varlen_bwd(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v,
                            const mxfa_mx* dout_mx, const void* o, const void* dout, const float* lse,
                            const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int nseq,
                            int max_seqlen_q, int max_seqlen_k, int64_t total_q, int64_t total_k,
                            int64_t ptiles_q, int64_t ptiles_k, int H, int D, float softmax_scale,
                            int causal, int dq_mode, float dq_static_scale, void* dq, void* dk,
                            void* dv, void* ws, size_t ws_bytes, mxfa_stream_t stream);

/* mxfa_bwd_opts, mxfa_varlen_bwd_opts -- mxfa_bwd / mxfa_varlen_bwd with
 * options (see mxfa_attn_opts; NULL = defaults; the backward reads only
 * p_scale, which selects the block or constant scale of its P^T). */
mxfa_status mxfa_bwd_opts(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v,
                          const mxfa_mx* dout_mx, const void* o, const void* dout, const float* lse,
                          int B, int S, int H, int D, float softmax_scale, int causal,
                          const mxfa_attn_opts* opts, int dq_mode, float dq_static_scale, void* dq,
                          void* dk, void* dv, void* ws, size_t ws_bytes, mxfa_stream_t stream);
mxfa_status mxfa_varlen_bwd_opts(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v,
                                 const mxfa_mx* dout_mx, const void* o, const void* dout,
                                 const float* lse, const int32_t* cu_seqlens_q,
                                 const int32_t* cu_seqlens_k, int nseq, int max_seqlen_q,
                                 int max_seqlen_k, int64_t total_q, int64_t total_k,
                                 int64_t ptiles_q, int64_t ptiles_k, int H, int D,
                                 float softmax_scale, int causal, const mxfa_attn_opts* opts,
                                 int dq_mode, float dq_static_scale, void* dq, void* dk, void* dv,
                                 void* ws, size_t ws_bytes, mxfa_stream_t stream);

/* mxfa_bwd_mxg, mxfa_varlen_bwd_mxg -- the backward passes above that also
 * emit the gradients as MXFP8 ([TMEM] page, section "What the Benchmarks
 * Show About Low-Precision Training": quantized gradients instead of bf16).
 * Each bf16 gradient they write is quantized in 1x32 blocks along D, byte
 * for byte as mxfa_quantize(MXFA_BLK_ROW) quantizes it.  dq_mx, dk_mx, dv_mx
 * are each nullable; for each given one:
 *  data        E4M3 [tokens][H][128] (required, 16-byte aligned)
 *  sf_compact  E8M0 [tokens][H * 4] (nullable, 4-byte aligned; required for
 *              dq_mx when its sf_packed is given)
 *  sf_packed   packed ROW atoms, ptiles * H * 512 bytes, rows past a
 *              sequence's end 0x7F (nullable, 16-byte aligned)
 * dK and dV are quantized in the kernel's epilogue, dQ in its final pass
 * (plus one scale-packing pass when dq_mx->sf_packed is given).  Other
 * arguments and errors as mxfa_bwd / mxfa_varlen_bwd. */
mxfa_status mxfa_bwd_mxg(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v,
                         const mxfa_mx* dout_mx, const void* o, const void* dout, const float* lse,
                         int B, int S, int H, int D, float softmax_scale, int causal, int dq_mode,
                         float dq_static_scale, void* dq, void* dk, void* dv, void* ws,
                         size_t ws_bytes, const mxfa_mx_out* dq_mx, const mxfa_mx_out* dk_mx,
                         const mxfa_mx_out* dv_mx, mxfa_stream_t stream);
mxfa_status mxfa_varlen_bwd_mxg(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v,
                                const mxfa_mx* dout_mx, const void* o, const void* dout,
                                const float* lse, const int32_t* cu_seqlens_q,
                                const int32_t* cu_seqlens_k, int nseq, int max_seqlen_q,
                                int max_seqlen_k, int64_t total_q, int64_t total_k,
                                int64_t ptiles_q, int64_t ptiles_k, int H, int D,
                                float softmax_scale, int causal, int dq_mode, float dq_static_scale,
                                void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                                const mxfa_mx_out* dq_mx, const mxfa_mx_out* dk_mx,
                                const mxfa_mx_out* dv_mx, mxfa_stream_t stream);

/* mxfa_rmsnorm_quant -- fused RMSNorm + MX quantization in one pass
 * ([TMEM] "fused producers", [ITEMS] item 7: FP8 out with dual scale layouts).
 *  x      bf16 [T][C], C in {256, 512, 1024, 2048}
 *  gamma  fp32 [C]
 *  y = (x * r) * gamma, r = 1/sqrt(mean(x^2) + eps), fp32, each operation
 *  correctly rounded; the sum of squares runs in a fixed order: lane l of a
 *  warp owns columns 8l + 256k + j, adds their squares k-outer, j-inner, then
 *  a butterfly over lane distances 16, 8, 4, 2, 1.
 *  seg_len  column and square blocks are anchored every seg_len rows
 *           (a multiple of 32; a multiple of 128 dividing T when packed
 *           scales are requested)
 *  H        head split of C for the packed layouts (C = H * 128)
 *  row/col/sq  outputs for 1x32, 32x1 and 32x32 blocks; each may be NULL
 *           (at least one must be given). */
mxfa_status mxfa_rmsnorm_quant(const void* x, const float* gamma, int64_t T, int64_t C, float eps,
                               int seg_len, int H, const mxfa_mx_out* row, const mxfa_mx_out* col,
                               const mxfa_mx_out* sq, mxfa_stream_t stream);

/* mxfa_bwd_noalloc -- mxfa_bwd for callers that cannot allocate device
 * memory.  The pages have no counterpart to this call: it is an interface
 * addition of this library.
 *  For code that must not call cudaMalloc (allocator or memory-pool hooks,
 *  runtimes that forbid device allocation after start-up, bindings without a
 *  device allocator), the workspace comes from a scratch array compiled into
 *  the library (mxfa_bwd_noalloc_scratch_bytes() = 32 MiB, 256-byte aligned,
 *  held by every GPU that loads the library until the process exits).  The
 *  call allocates nothing; inputs and outputs are as for mxfa_bwd.
 *  The first call on each device looks up the array's device address
 *  (cudaGetSymbolAddress, with that device current) and caches it: make that
 *  first call before any stream capture.
 *  Problems whose workspace (mxfa_bwd_workspace_size) exceeds the array are
 *  rejected with MXFA_ERR_WORKSPACE_TOO_SMALL before anything is launched.
 *  All calls share the one array and it keeps the last call's contents (the
 *  backward pass clears what must start at zero); calls that overlap on the
 *  GPU, e.g. on two streams, race on it. */
mxfa_status mxfa_bwd_noalloc(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v,
                             const mxfa_mx* dout_mx, const void* o, const void* dout,
                             const float* lse, int B, int S, int H, int D, float softmax_scale,
                             int causal, int dq_mode, float dq_static_scale, void* dq, void* dk,
                             void* dv, mxfa_stream_t stream);
size_t mxfa_bwd_noalloc_scratch_bytes(void);

/* mxfa_gemm_quant -- projection GEMM with the quantization fused into its
 * epilogue ([TMEM] "fused producers": projection GEMM epilogues emit FP8;
 * [ITEMS] item 7: GEMM+Quantize with dual scale-factor layouts in one pass).
 *  a   ROW-quantized A [M][K] (payload, and packed ROW scales with K / 128
 *      column groups, i.e. mxfa_quantize(MXFA_BLK_ROW) of a bf16 [M][K/128][128])
 *  b   ROW-quantized B [N][K] likewise (a weight stored [out][in])
 *  Y = A B^T (dequantized operands, fp32 accumulation), written as
 *  y_bf16  bf16 [M][N] (nullable)
 *  y_row   MXFP8 of Y in 1x32 blocks along N: payload [M][N], compact scales
 *          [M][N / 32], packed ROW atoms of (128-row tile, 128-column group),
 *          as mxfa_quantize(MXFA_BLK_ROW) lays them out for Y seen as
 *          [M][N / 128][128] (nullable; its scale pointers nullable)
 *  y_col   MXFP8 of Y in 32x1 blocks along M (blocks start at multiples of
 *          32 rows): payload [M][N], compact scales [M / 32][N], packed COL
 *          atoms (nullable; its scale pointers nullable)
 *  At least one output must be given.  M, N, K multiples of 128
 *  (else MXFA_ERR_UNSUPPORTED).  Each output block is quantized with the OCP
 *  rule of mxfa_quantize from the fp32 value of Y (not from its bf16 copy). */
mxfa_status mxfa_gemm_quant(const mxfa_mx* a, const mxfa_mx* b, int64_t M, int64_t N, int64_t K,
                            void* y_bf16, const mxfa_mx_out* y_row, const mxfa_mx_out* y_col,
                            mxfa_stream_t stream);

/* Lower-precision formats -- the next formats the pages name ([ITEMS] item
 * 12: MXFP6 and MXFP4; [KDIM] paragraph 1: Blackwell's block-scaled MMA runs
 * MXFP8, MXFP6, MXFP4 and NVFP4).
 * mxfa_quantize_lowp -- bf16 x[rows][cols] -> codes in 1x32 blocks along the
 * columns with E8M0 scales
 * (MXFP4 = E2M1, max 6, emax 2; MXFP6 = E2M3, max 7.5, emax 2, or E3M2, max
 * 28, emax 4: scale = floor(log2 amax) - emax, clamped to [0, 254]; codes
 * nearest-even, saturating; a block holding Inf / NaN gets scale 0xFF and
 * codes 0), or NVFP4 in 1x16 blocks: fp32 tensor scale st = amax / 2688
 * (448 * 6; 1 for an all-zero tensor), written to *tensor_scale (DEVICE),
 * E4M3 block scales E4M3(amax_block / (6 st)) and E2M1 codes of
 * x / (scale * st), every step one correctly rounded fp32 operation (NVFP4
 * inputs must be finite).
 *  q          [rows][cols] bytes: with MXFA_LOWP_CODES one code per byte in
 *             the low bits; with MXFA_LOWP_MMA (MX formats) the form the
 *             block-scaled MMA reads sub-byte operands in from shared memory:
 *             each run of 16 codes packed little-endian (code j at bit 4j for
 *             FP4, 6j for FP6) in the first 8 / 12 bytes of a 16-byte group,
 *             the rest zero -- still one byte of storage per element
 *  sf         scales [rows][cols / 32] (MX) or [rows][cols / 16] (NVFP4)
 *  sf_packed  MX only, nullable: packed atoms per (128-row tile, 128-column
 *             group) as the GEMM reads them (rows, cols multiples of 128)
 * cols must be a multiple of 32 (MX) or 16 (NVFP4). */
#define MXFA_LOWP_MXFP4 0
#define MXFA_LOWP_MXFP6_E2M3 1
#define MXFA_LOWP_MXFP6_E3M2 2
#define MXFA_LOWP_NVFP4 3
#define MXFA_LOWP_CODES 0
#define MXFA_LOWP_MMA 1
mxfa_status mxfa_quantize_lowp(const void* x, int64_t rows, int cols, int fmt, int q_layout, uint8_t* q,
                               uint8_t* sf, uint8_t* sf_packed, float* tensor_scale, mxfa_stream_t stream);

/* mxfa_gemm_quant_fmt -- mxfa_gemm_quant with the element format of each
 * operand: MXFA_ELEM_E4M3 (MXFP8), or MXFP6 / MXFP4 operands from
 * mxfa_quantize_lowp (MXFA_LOWP_MMA layout, packed scale atoms), which the tensor
 * core's mixed-format block-scaled MMA reads at the MXFP8 rate.  The output
 * options are those of mxfa_gemm_quant. */
#define MXFA_ELEM_E4M3 0
#define MXFA_ELEM_E2M3 1
#define MXFA_ELEM_E3M2 2
#define MXFA_ELEM_E2M1 3
mxfa_status mxfa_gemm_quant_fmt(const mxfa_mx* a, int a_fmt, const mxfa_mx* b, int b_fmt, int64_t M,
                                int64_t N, int64_t K, void* y_bf16, const mxfa_mx_out* y_row,
                                const mxfa_mx_out* y_col, mxfa_stream_t stream);

/* ------------------------------------------------------------ 4-bit KV cache
 * Serving: keys and values of the tokens so far, held as MXFP4 or NVFP4 in pages,
 * and the attention that reads them.  The web pages above have no counterpart to
 * these calls; the formats are those of mxfa_quantize_lowp.
 *
 * A cache (of one layer) is num_blocks pages of `page` rows (16, 32, 64 or 128)
 * for each of H key heads, D = 128:
 *  k, v        E2M1 codes [num_blocks][H][page][64], two to a byte, the even
 *              channel in the low nibble
 *  k_sf, v_sf  block scales [num_blocks][H][page][4] (MXFP4: E8M0 per 32
 *              channels) or [8] (NVFP4: E4M3 per 16 channels)
 *  k_scale, v_scale  NVFP4: DEVICE fp32, the (finite, positive) scale of the whole
 *              K and V cache, chosen by the caller before the first store; unused for
 *              MXFP4
 * All device pointers, owned by the caller, codes and scales 16-byte aligned.
 * A slot is block * page + row.  A cached value is code * scale (* k_scale or
 * v_scale).  MXFP4 scales are 2^X with X = floor(log2 amax) - 2 clamped to
 * [-23, 13], so that every cached value is a binary16 number: magnitudes
 * above 49152 saturate and blocks below 2^-21 lose precision, where
 * mxfa_quantize_lowp clamps to the whole range of E8M0.  NVFP4 scales are
 * E4M3(amax / (6 st)), codes E2M1(x / (scale st)), as mxfa_quantize_lowp's.  A block
 * holding Inf or NaN reads back as NaN (scale 0xFF or 0x7F, codes 0). */
#define MXFA_KV_MXFP4 0
#define MXFA_KV_NVFP4 1
typedef struct {
  uint8_t *k, *v;
  uint8_t *k_sf, *v_sf;
  const float *k_scale, *v_scale;
  int64_t num_blocks;
  int page, H, D, fmt;
} mxfa_kv_cache;

/* Bytes of the codes (of k or of v) and of the block scales of a cache. */
size_t mxfa_kv_codes_bytes(int64_t num_blocks, int page, int H);
size_t mxfa_kv_sf_bytes(int64_t num_blocks, int page, int H, int fmt);

/* mxfa_kv_plan -- block tables and slots of a step, from request lengths, on
 * the GPU and without a host read, so that a captured graph can be replayed.
 *  ctx_lens     int32 [R], tokens in the cache before the step
 *  new_lens     int32 [R], new tokens of the step; negative: the request is done
 *  block_table  int32 [R][max_blocks], the first ceil(ctx / page) entries of a
 *               row in use; new blocks are written behind them, other entries stay
 *  free_ring    int32 [ring_size], queue of free blocks; ring_size is at least the number of
 *               blocks, so that blocks given back never reach those still queued
 *  ring_in/out  int64 [3]: number of blocks ever taken, number ever put in (free
 *               blocks are the ring entries [taken, put) modulo ring_size), and (written
 *               only) the blocks that this step lacked
 *  tokens       rows of slots and positions
 *  cu_q         int32 [R + 1], prefix sums of max(new_lens, 0)
 *  kv_lens      int32 [R]: ctx + new; 0 for a done request
 *  slots        int64 [tokens], positions int32 [tokens]: token t of the step, the
 *               requests' tokens one after another; -1 for tokens past cu_q[R]
 * Blocks are taken in request order.  Where the free ones do not suffice, the
 * first request that would exceed them and all later ones that need a block get none:
 * their kv_lens stays ctx, their slots are -1 (mxfa_kv_append skips them), and
 * ring_out[2] > 0 says so.  Such a request's tokens stay in cu_q, so mxfa_kv_attn
 * computes their rows too, as if they were the last of the ctx stored ones: these rows mean
 * nothing.  The same holds for a request past max_blocks.
 * Where cu_q[R] exceeds `tokens`, all tokens are planned (blocks, kv_lens) and the last ones
 * get no slot.  A done request's blocks go back in request and table
 * order and can be taken from the next step on.  kv_lens may be ctx_lens and
 * ring_out may be ring_in (a step captured once and replayed); any other
 * buffers that overlap are MXFA_ERR_INVALID_ARG.  The new lengths sum to less than 2^31.
 * A request whose tokens exceed
 * max_blocks pages gets no block and is recorded as a failed index check.
 * R <= 16384, page as above, max_blocks * page <= 2^30 (else MXFA_ERR_UNSUPPORTED). */
mxfa_status mxfa_kv_plan(const int32_t* ctx_lens, const int32_t* new_lens, int R, int32_t* block_table,
                         int max_blocks, int32_t* free_ring, int64_t ring_size, const int64_t* ring_in,
                         int64_t* ring_out, int page, int64_t tokens, int32_t* cu_q, int32_t* kv_lens,
                         int64_t* slots, int32_t* positions, mxfa_stream_t stream);

/* mxfa_kv_append -- quantizes new tokens into their slots.
 *  k, v      bf16 rows of H * 128, consecutive tokens k_stride / v_stride elements
 *            apart (multiples of 8, at least H * 128), 16-byte aligned
 *  slots     DEVICE int64 [tokens]; negative: the token is skipped.  Slots of one call are
 *            distinct (two tokens with one slot leave it undefined); a slot past the
 *            cache is skipped and recorded as a failed index check
 * k, v and slots do not overlap the cache's codes and block scales, nor do these
 * overlap one another, k_scale or v_scale (MXFA_ERR_INVALID_ARG). */
mxfa_status mxfa_kv_append(const mxfa_kv_cache* cache, const void* k, const void* v, int64_t k_stride,
                           int64_t v_stride, int64_t tokens, const int64_t* slots, mxfa_stream_t stream);

/* mxfa_kv_load -- the cached values of slots as bf16 k, v [tokens][H][128] (MXFP4
 * exact, NVFP4 rounded to nearest), in any order and repeated at will; zeros
 * for a negative slot (and for one past the cache, which is recorded).  k and v overlap
 * neither each other nor slots nor the cache (MXFA_ERR_INVALID_ARG). */
mxfa_status mxfa_kv_load(const mxfa_kv_cache* cache, const int64_t* slots, int64_t tokens, void* k, void* v,
                         mxfa_stream_t stream);

/* Workspace of mxfa_kv_attn on the current device, for the same R, max_q, Hq and
 * cache, and max_k = max_blocks * page; 0 where short contexts need none (ws may
 * then be NULL). */
size_t mxfa_kv_attn_workspace_size(int R, int max_q, int64_t max_k, int Hq, int H);

/* mxfa_kv_attn -- attention of new query tokens over the cache.
 *  q            bf16 rows of Hq * 128, q_stride elements apart (a multiple of 8),
 *               Hq a multiple of the cache's H: query heads h G .. h G + G - 1 read
 *               key head h, G = Hq / H
 *  cu_q         DEVICE int32 [R + 1]; request r's queries are rows cu_q[r] ..
 *               cu_q[r + 1] - 1, at most max_q of them; rows outside are not written
 *  kv_lens      DEVICE int32 [R], keys of each request, its new tokens included
 *  block_table  DEVICE int32 [R][max_blocks]
 *  causal       1: query i of a request's n sees keys j <= kv - n + i; 0: all keys
 *  o            bf16 [total_q][Hq][128];  lse fp32 [Hq][total_q], natural log.  A query
 *               that sees no key gets O = 0 and lse = -inf; one with Inf or NaN
 *               that sees a key gets NaN.  Scores, times softmax_scale, stay within fp32's
 *               range; those past it count as infinite
 *  ws           mxfa_kv_attn_workspace_size() bytes, 16-byte aligned, not shared by calls
 *               that can run at the same time; its contents need not be kept
 * Keys past kv_lens or in no row's sight are not used, whatever they hold.  A block index
 * outside the cache (its keys count as not there) and offsets or lengths outside
 * their tables (the request is left out) are recorded as failed index checks.
 * o, lse and ws overlap neither each other nor an input, the cache's buffers among them
 * (MXFA_ERR_INVALID_ARG).
 * max_blocks * page <= 2^30, and <= 2^25 where max_q * G > 48 (else
 * MXFA_ERR_UNSUPPORTED). */
mxfa_status mxfa_kv_attn(const mxfa_kv_cache* cache, const void* q, int64_t q_stride, int64_t total_q,
                         const int32_t* cu_q, const int32_t* kv_lens, int R, const int32_t* block_table,
                         int max_blocks, int max_q, int Hq, float softmax_scale, int causal, void* o,
                         float* lse, void* ws, size_t ws_bytes, mxfa_stream_t stream);

/* mxfa_kv_attn_window -- mxfa_kv_attn (causal) where a query at position p (query i of a request's n:
 * p = kv - n + i) sees the last `window` keys, p - window + 1 .. p, and the first `sinks` ones,
 * j < sinks, j <= p.  window >= 1, sinks >= 0.  Pages without a key in a row's sight are not read, and
 * their table entries may be anything (pages given back by mxfa_kv_free).  The workspace is of
 * mxfa_kv_attn_window_workspace_size() bytes; everything else as mxfa_kv_attn, the limit of 2^25 keys
 * taken of window + sinks. */
size_t mxfa_kv_attn_window_workspace_size(int R, int max_q, int64_t max_k, int Hq, int H, int window, int sinks);
mxfa_status mxfa_kv_attn_window(const mxfa_kv_cache* cache, const void* q, int64_t q_stride, int64_t total_q,
                                const int32_t* cu_q, const int32_t* kv_lens, int R, const int32_t* block_table,
                                int max_blocks, int max_q, int Hq, float softmax_scale, int window, int sinks,
                                void* o, float* lse, void* ws, size_t ws_bytes, mxfa_stream_t stream);

/* mxfa_kv_attn_shared -- mxfa_kv_attn (causal) for requests that share prefixes: the keys of a group's
 * prefix are read once for the queries of all its requests, where that pays.
 *  group_starts DEVICE int32 [groups + 1], ascending: group g is requests group_starts[g] ..
 *               group_starts[g + 1] - 1; requests of no group are computed as by mxfa_kv_attn
 *  prefix_lens  DEVICE int32 [groups]: the first prefix_lens[g] keys of each request of the group are
 *               those of its first request, whose row of block_table they are read from; each
 *               request's further keys from its own row.  Any length, 0 included
 *  max_group_q  the most query tokens of a group
 *  share        MXFA_KV_SHARE_AUTO: prefixes are read once for a group where that is estimated to be faster, from the
 *               lengths and on the GPU (long prefixes, many requests of few tokens), and by each request
 *               for itself otherwise; _ALWAYS, _NEVER: one or the other
 * Each request with queries has at least the prefix before them (kv - n >= prefix).  One that has not,
 * and the requests of a group whose starts, queries or prefix are outside their bounds, are left out
 * and recorded as failed index checks.  (After a step that lacked blocks, ring_out[2] > 0, mxfa_kv_plan leaves some
 * kv_lens at the old contexts: those requests' rows mean nothing, and one that is no longer behind its prefix
 * by its kv_lens is left out and recorded here, where mxfa_kv_attn computes it.)
 * The workspace is of mxfa_kv_attn_shared_workspace_size_mode() bytes for
 * the same share, max_k = max_blocks * page: 1056 bytes a token and query head (results of prefixes and of what is
 * behind them, in fp32), or 8 with _NEVER, beside what mxfa_kv_attn needs, twice or once;
 * mxfa_kv_attn_shared_workspace_size() bytes suffice for any.  Everything else as mxfa_kv_attn.  groups may be 0. */
#define MXFA_KV_SHARE_AUTO 0
#define MXFA_KV_SHARE_ALWAYS 1
#define MXFA_KV_SHARE_NEVER 2
size_t mxfa_kv_attn_shared_workspace_size(int R, int groups, int64_t total_q, int max_q, int max_group_q, int64_t max_k,
                                          int Hq, int H);
size_t mxfa_kv_attn_shared_workspace_size_mode(int R, int groups, int64_t total_q, int max_q, int max_group_q, int64_t max_k,
                                               int Hq, int H, int share);
mxfa_status mxfa_kv_attn_shared(const mxfa_kv_cache* cache, const void* q, int64_t q_stride, int64_t total_q,
                                const int32_t* cu_q, const int32_t* kv_lens, int R, const int32_t* block_table,
                                int max_blocks, int max_q, int Hq, float softmax_scale, const int32_t* group_starts,
                                const int32_t* prefix_lens, int groups, int max_group_q, int share, void* o, float* lse,
                                void* ws, size_t ws_bytes, mxfa_stream_t stream);

/* ---------------------------------------------------------- rotary positions
 * The first `rot` of a head's 128 channels turn by their token's position p: pair i by the angle
 * t = p f_i,  (a, b) -> gain (a cos t - b sin t, b cos t + a sin t);  the others stay.  The pages have
 * no counterpart to these calls.
 *  turns   DEVICE int64 [rot / 2]: f_i / 2 pi in 2^-64ths of a turn, modulo 2^64 (negative where it is
 *          half a turn or more), so that the angle of any position is exact to 2^-32 turns
 *  rot     16, 32, .., 128
 *  layout  pairs (i, i + rot / 2) or (2 i, 2 i + 1) */
#define MXFA_ROPE_HALF 0
#define MXFA_ROPE_INTERLEAVED 1
typedef struct {
  const int64_t* turns;
  int rot, layout;
  double gain;
} mxfa_rotation;

/* mxfa_rope -- y = x turned (before mxfa_quantize, mxfa_kv_append or mxfa_kv_attn), or with inverse = 1
 * turned back with the same gain: the gradient of x from that of y.
 *  x, y       bf16 rows of H * 128, consecutive tokens x_stride / y_stride elements apart (multiples of
 *             8, at least H * 128), 16-byte aligned; y may be x (same stride), else they do not overlap
 *  positions  DEVICE int32 [tokens], as mxfa_kv_plan gives them; negative: the token's row of y stays
 * Each step is rounded once: c = fp32(gain cos t), s = fp32(gain sin t) (all but a few in ten thousand
 * correctly), the fp32 products a c and b s, their fp32 difference or sum, and bf16 of it.  y overlaps neither positions nor turns (MXFA_ERR_INVALID_ARG). */
mxfa_status mxfa_rope(const void* x, int64_t x_stride, void* y, int64_t y_stride, const int32_t* positions,
                      int64_t tokens, int H, int D, const mxfa_rotation* rot, int inverse, mxfa_stream_t stream);

/* mxfa_kv_append_rope -- a step's new tokens in one call: q_out = q turned, k turned and v into the
 * cache, byte for byte as mxfa_rope of q and k and mxfa_kv_append of the turned k and v.
 *  q, q_out   bf16 rows of Hq * 128, q_out may be q (same stride)
 *  positions  DEVICE int32 [tokens]; negative: the token is left out altogether
 *  slots      as mxfa_kv_append; a token without a slot still gets its q_out
 * Other arguments and errors as mxfa_kv_append and mxfa_rope. */
mxfa_status mxfa_kv_append_rope(const mxfa_kv_cache* cache, const void* q, int64_t q_stride, int Hq, const void* k,
                                int64_t k_stride, const void* v, int64_t v_stride, int64_t tokens,
                                const int32_t* positions, const int64_t* slots, const mxfa_rotation* rot, void* q_out,
                                int64_t q_out_stride, mxfa_stream_t stream);

/* ------------------------------------------------- pages shared by requests
 * refs int32 [num_blocks] (DEVICE, zeros at first) counts the owners of a block beside the first.  A
 * request that may share pages, or has given some up, is ended by mxfa_kv_free, not by a negative count in
 * mxfa_kv_plan, which gives back all blocks of its row whoever else owns them.  Shared pages are full:
 * a request goes on behind the tokens it was forked with, and one that is cut back to fewer (rejected
 * drafts) is cut back no further than that. */

/* mxfa_kv_fork -- requests that continue other ones: row dst[f] of block_table gets the first lens[f]
 * tokens of row src[f].  Whole pages are shared (refs + 1).  A last page that is not full would be
 * written by both, so it gets a new block from the ring, the k-th such fork the k-th free block.
 *  src, dst, lens  DEVICE int32 [F], F <= 16384; a row is dst of one fork only and src of none then;
 *               0 <= lens <= the tokens that row src holds
 *  from_blocks, to_blocks  int32 [F] (written): the block to copy and the new one, for mxfa_kv_copy_blocks
 *               in each layer's cache; -1, -1 where there is none
 *  lens_out     int32 [F] (written): tokens that row dst holds: lens, or where the ring had no block left
 *               (ring_out[2] counts them) the whole pages of it alone, with -1 behind them in the table
 *  free_ring, ring_in/out  as mxfa_kv_plan; ring_out may be ring_in
 * Other entries of row dst stay.  Forks outside their bounds give nothing (lens_out 0), and entries that are no
 * blocks are copied as -1 without an owner (a last page's takes no block of the ring: lens_out is the whole pages
 * alone); both are recorded as failed index checks.  Other buffers that overlap are MXFA_ERR_INVALID_ARG. */
mxfa_status mxfa_kv_fork(int32_t* block_table, int R, int max_blocks, const int32_t* src, const int32_t* dst,
                         const int32_t* lens, int F, int32_t* refs, int64_t num_blocks, const int32_t* free_ring,
                         int64_t ring_size, const int64_t* ring_in, int64_t* ring_out, int page, int32_t* from_blocks,
                         int32_t* to_blocks, int32_t* lens_out, mxfa_stream_t stream);

/* mxfa_kv_fork_gap -- mxfa_kv_fork of requests that have given pages up (behind a window, its sinks' pages kept):
 * entries gap_first[f] .. gap_end[f] - 1 of row src[f] are neither read nor shared, and are -1 in row dst[f].
 * mxfa_kv_fork would count an owner for them, although such a block is in the ring or another request's by then.
 *  gap_first, gap_end  DEVICE int32 [F], 0 <= gap_first <= gap_end <= lens / page (else the fork is outside its
 *               bounds); equal: none.  Both NULL: as mxfa_kv_fork */
mxfa_status mxfa_kv_fork_gap(int32_t* block_table, int R, int max_blocks, const int32_t* src, const int32_t* dst,
                             const int32_t* lens, const int32_t* gap_first, const int32_t* gap_end, int F, int32_t* refs,
                             int64_t num_blocks, const int32_t* free_ring, int64_t ring_size, const int64_t* ring_in,
                             int64_t* ring_out, int page, int32_t* from_blocks, int32_t* to_blocks, int32_t* lens_out,
                             mxfa_stream_t stream);

/* mxfa_kv_free -- pages given up: for each f, entries first[f] .. end[f] - 1 of row rows[f] (ended requests,
 * rejected continuations, pages behind a window) have one owner fewer; negative entries are skipped.  Blocks left
 * without an owner go to the ring in ascending order.  The table stays as it is: an entry given up is not given
 * up again, and a row that has some is forked by mxfa_kv_fork_gap.  ring_size is at least num_blocks (MXFA_ERR_INVALID_ARG); ring_out may be ring_in; ring_out[2] is ring_in[2].  Rows and ranges
 * outside the table, entries past num_blocks and blocks given up more often than owned are recorded as failed
 * index checks.  Other buffers that overlap are MXFA_ERR_INVALID_ARG. */
mxfa_status mxfa_kv_free(const int32_t* block_table, int R, int max_blocks, const int32_t* rows, const int32_t* first,
                         const int32_t* end, int F, int32_t* refs, int64_t num_blocks, int32_t* free_ring,
                         int64_t ring_size, const int64_t* ring_in, int64_t* ring_out, mxfa_stream_t stream);

/* mxfa_kv_copy_blocks -- block from_blocks[i] of the cache (all heads, codes and scales of K and V) over
 * to_blocks[i], n <= 8192; pairs with a negative one are skipped, ones past the cache skipped and
 * recorded.  All blocks are read before any is written, so a block may be read and written (a list of
 * moves); one that is written by several pairs holds the last one's.  mxfa_kv_fork's pairs, of which no
 * block is both, may be copied in pieces. */
mxfa_status mxfa_kv_copy_blocks(const mxfa_kv_cache* cache, const int32_t* from_blocks, const int32_t* to_blocks, int n,
                                mxfa_stream_t stream);

/* mxfa_tensor_peak_probe -- `ctas` CTAs (one per SM at most) each issue
 * `iters` x 4 back-to-back block-scaled MMAs (M = 128, N = 256, K = 32, E4M3,
 * operands resident in shared memory) and write the SM clock cycles they took
 * to cycles[ctas] (DEVICE, 8-byte aligned).  The pages have no counterpart: it
 * measures this GPU's dense MXFP8 tensor-pipe peak, the denominator of the
 * benchmark's roofline fractions (MACs per CTA = iters * 4 * 128 * 256 * 32). */
mxfa_status mxfa_tensor_peak_probe(int iters, int ctas, unsigned long long* cycles, mxfa_stream_t stream);

/* Synchronise `stream`, then return and clear the device status words:
 * MXFA_OK, MXFA_ERR_TIMEOUT or MXFA_ERR_DEVICE_INDEX (bit flags also in
 * *flags when flags is not NULL: 1 timeout, 2 index). */
mxfa_status mxfa_get_device_status(mxfa_stream_t stream, unsigned* flags);

#ifdef __cplusplus
}
#endif
#endif /* MXFA_H */
