// api.cu -- the C ABI (include/mxfa.h): argument checks, TMA descriptors and
// kernel launches.  No allocation, no synchronisation on the hot path.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "../../include/mxfa.h"
#include "mxfa_internal.h"

using namespace mxfa;

namespace mxfa {

int sm_count_current_device() {
  static std::atomic<int> count[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < kMaxDevices) {
    const int c = count[dev].load(std::memory_order_relaxed);
    if (c > 0) return c;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 0;
  if (dev >= 0 && dev < kMaxDevices) count[dev].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace mxfa

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// u8 tensor [tokens][H][128] as a 3-D map, box 128 x 1 x box_rows, 128B swizzle.
bool make_map_u8(CUtensorMap* m, const void* ptr, int64_t tokens, int H, int box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {128, cuuint64_t(H), cuuint64_t(tokens)};
  cuuint64_t strides[2] = {128, cuuint64_t(H) * 128};
  cuuint32_t box[3] = {128, 1, cuuint32_t(box_rows)};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// dQ accumulator [tokens][H][128] (fp32 or fp16) as a 3-D map, box 128 x 1 x 64.
bool make_map_acc(CUtensorMap* m, const void* ptr, int64_t tokens, int H, bool half) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t esz = half ? 2 : 4;
  cuuint64_t dims[3] = {128, cuuint64_t(H), cuuint64_t(tokens)};
  cuuint64_t strides[2] = {128 * esz, cuuint64_t(H) * 128 * esz};
  cuuint32_t box[3] = {128, 1, 64};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
                   const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// bf16 tensor [tokens][H][128] as a 3-D map for stores, box 64 x 1 x 32 (128-byte rows),
// 128B swizzle.
bool make_map_bf16_store(CUtensorMap* m, void* ptr, int64_t tokens, int H) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {128, cuuint64_t(H), cuuint64_t(tokens)};
  cuuint64_t strides[2] = {256, cuuint64_t(H) * 256};
  cuuint32_t box[3] = {64, 1, 32};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, ptr, dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// bf16 tensor [tokens][H][128] as a 3-D map for loads, box 128 x heads x 32
// (32 rows of `heads` adjacent heads), no swizzle; rows and heads past the
// tensor read 0.
bool make_map_bf16_rows(CUtensorMap* m, const void* ptr, int64_t tokens, int H, int heads) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {128, cuuint64_t(H), cuuint64_t(tokens)};
  cuuint64_t strides[2] = {256, cuuint64_t(H) * 256};
  cuuint32_t box[3] = {128, cuuint32_t(heads), 32};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

mxfa_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return MXFA_OK;
  if (e == cudaErrorInvalidValue) return MXFA_ERR_INVALID_ARG;
  return MXFA_ERR_CUDA;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Backward tile records: 2560 bytes per (64-query tile, head); sum over
// sequences of ceil(len / 64) is at most ceil(total / 64) + nseq.
size_t bwd_records_bytes(int64_t total_q, int nseq, int H) {
  const size_t n = size_t(ceil_div(total_q, 64) + nseq) * size_t(H) * 2560u;
  return (n + 255) & ~size_t(255);
}

// Shared checks of a sequence description.
mxfa_status check_seqs(const int32_t* cu, int nseq, int maxlen, int64_t tokens) {
  if (nseq <= 0 || maxlen < 0 || tokens < 0) return MXFA_ERR_INVALID_ARG;
  if (!cu && int64_t(nseq) * maxlen != tokens) return MXFA_ERR_INVALID_ARG;
  if (tokens >= (int64_t(1) << 31)) return MXFA_ERR_UNSUPPORTED;
  return MXFA_OK;
}

mxfa_status check_mx(const mxfa_mx* x) {
  if (!x || !x->data || !x->sf) return MXFA_ERR_INVALID_ARG;
  if (!aligned16(x->data) || !aligned16(x->sf)) return MXFA_ERR_MISALIGNED;
  return MXFA_OK;
}

// Options: NULL = defaults; otherwise checked.
mxfa_status read_opts(const mxfa_attn_opts* opts, float& thr, int& p_scale) {
  thr = MXFA_FWD_RESCALE_THRESHOLD;
  p_scale = MXFA_P_SCALE_BLOCK;
  if (!opts) return MXFA_OK;
  if (!(opts->rescale_threshold >= 0.0f && opts->rescale_threshold <= 8.0f)) return MXFA_ERR_INVALID_ARG;
  if (opts->p_scale != MXFA_P_SCALE_BLOCK && opts->p_scale != MXFA_P_SCALE_CONST) return MXFA_ERR_INVALID_ARG;
  thr = opts->rescale_threshold;
  p_scale = opts->p_scale;
  return MXFA_OK;
}

mxfa_status gemm_common(const mxfa_mx* a, int a_code, const mxfa_mx* b, int b_code, int64_t M, int64_t N,
                        int64_t K, void* y_bf16, const mxfa_mx_out* y_row, const mxfa_mx_out* y_col,
                        mxfa_stream_t stream);

mxfa_status fwd_common(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v, Seqs sq, Seqs sk,
                       int64_t total_q, int64_t total_k, int64_t ptq, int64_t ptk, int H, int D,
                       float scale, int causal, void* o, float* lse, const mxfa_mx_out* omx, bool dense,
                       mxfa_stream_t stream, const mxfa_attn_opts* opts = nullptr) {
  mxfa_status s;
  float thr;
  int p_scale;
  if ((s = read_opts(opts, thr, p_scale))) return s;
  if ((s = check_mx(q)) || (s = check_mx(k)) || (s = check_mx(v))) return s;
  if (!o || !lse || H <= 0) return MXFA_ERR_INVALID_ARG;
  if (omx && (!omx->data || !aligned16(omx->data) || (omx->sf_compact && !aligned4(omx->sf_compact)) ||
              (omx->sf_packed && !aligned16(omx->sf_packed))))
    return omx->data ? MXFA_ERR_MISALIGNED : MXFA_ERR_INVALID_ARG;
  if (D != 128) return MXFA_ERR_UNSUPPORTED;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return MXFA_ERR_INVALID_ARG;
  if (!aligned16(o)) return MXFA_ERR_MISALIGNED;
  if (ptq <= 0 || ptk <= 0) return MXFA_ERR_INVALID_ARG;
  if (total_q == 0) return MXFA_OK;
  FwdArgs a;
  memset(&a, 0, sizeof(a));
  if (!make_map_u8(&a.tm_q, q->data, total_q, H, 128) || !make_map_u8(&a.tm_k, k->data, total_k, H, 128) ||
      !make_map_u8(&a.tm_v, v->data, total_k, H, 128) || !make_map_bf16_store(&a.tm_o, o, total_q, H))
    return MXFA_ERR_CUDA;
  a.sfq = q->sf;
  a.sfk = k->sf;
  a.sfv = v->sf;
  a.sq = sq;
  a.sk = sk;
  a.total_q = total_q;
  a.ptiles_q = ptq;
  a.ptiles_k = ptk;
  a.H = H;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.rescale_thr = thr;
  // constant P scale: 2^(ceil(thr) - 8), the largest possible P~ = 2^ceil(thr) -> 256
  a.p_sc_const = p_scale == MXFA_P_SCALE_CONST ? uint32_t(127 + int(std::ceil(thr)) - 8) : 0u;
  a.causal = causal ? 1 : 0;
  a.o = static_cast<uint16_t*>(o);
  if (omx) {
    a.omx = omx->data;
    a.omx_sfc = omx->sf_compact;
    a.omx_sfp = omx->sf_packed;
  }
  a.lse = lse;
  a.dense_lse = dense ? 1 : 0;
  a.lse_hstride = dense ? sq.seqlen : total_q;
  // Staged TMA stores of O (and one K/V stage fewer) pay off when items are
  // short, the epilogue being a large share of each item, and cost 1-2% on
  // long ones: mean key length up to 2048.
  a.stage_o = total_k <= int64_t(sk.nseq) * 2048 ? 1 : 0;
  return from_cuda(launch_fwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

mxfa_status bwd_common(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v, const mxfa_mx* dmx,
                       const void* o, const void* dout, const float* lse, Seqs sq, Seqs sk,
                       int64_t total_q, int64_t total_k, int64_t ptq, int64_t ptk, int H, int D,
                       float scale, int causal, int dq_mode, float dq_static_scale, void* dq, void* dk,
                       void* dv, void* ws, size_t ws_bytes, const mxfa_mx_out* gmx[3], bool dense,
                       mxfa_stream_t stream, const mxfa_attn_opts* opts = nullptr) {
  mxfa_status s;
  float thr_unused;
  int p_scale;
  if ((s = read_opts(opts, thr_unused, p_scale))) return s;
  if ((s = check_mx(q)) || (s = check_mx(k)) || (s = check_mx(v)) || (s = check_mx(dmx))) return s;
  for (int i = 0; i < 3 && gmx; i++) {
    const mxfa_mx_out* m = gmx[i];
    if (!m) continue;
    if (!m->data) return MXFA_ERR_INVALID_ARG;
    if (i == 0 && m->sf_packed && !m->sf_compact) return MXFA_ERR_INVALID_ARG;
    if (!aligned16(m->data) || (m->sf_compact && !aligned4(m->sf_compact)) ||
        (m->sf_packed && !aligned16(m->sf_packed)))
      return MXFA_ERR_MISALIGNED;
  }
  if (!o || !dout || !lse || !dq || !dk || !dv || H <= 0) return MXFA_ERR_INVALID_ARG;
  if (D != 128) return MXFA_ERR_UNSUPPORTED;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return MXFA_ERR_INVALID_ARG;
  if (dq_mode != 0 && dq_mode != 1) return MXFA_ERR_INVALID_ARG;
  if (dq_mode == 1) {
    int e;
    if (!(dq_static_scale > 0.0f) || !std::isfinite(dq_static_scale) ||
        std::frexp(dq_static_scale, &e) != 0.5f)
      return MXFA_ERR_INVALID_ARG;  // must be a power of two
  }
  if (!aligned16(o) || !aligned16(dout) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) ||
      !aligned16(ws))
    return MXFA_ERR_MISALIGNED;
  if (ptq <= 0 || ptk <= 0) return MXFA_ERR_INVALID_ARG;
  if (!ws) return MXFA_ERR_INVALID_ARG;
  if (ws_bytes < mxfa_bwd_workspace_size(total_q, sq.nseq, H, D, dq_mode))
    return MXFA_ERR_WORKSPACE_TOO_SMALL;
  if (total_q == 0 || total_k == 0) return MXFA_OK;
  BwdArgs a;
  memset(&a, 0, sizeof(a));
  if (!make_map_u8(&a.tm_q, q->data, total_q, H, 64) || !make_map_u8(&a.tm_do, dmx->data, total_q, H, 64) ||
      !make_map_u8(&a.tm_k, k->data, total_k, H, 128) || !make_map_u8(&a.tm_v, v->data, total_k, H, 128) ||
      !make_map_bf16_store(&a.tm_dk, dk, total_k, H) || !make_map_bf16_store(&a.tm_dv, dv, total_k, H))
    return MXFA_ERR_CUDA;
  a.sfq = q->sf;
  a.sfk = k->sf;
  a.sfv = v->sf;
  a.sfdo = dmx->sf;
  a.do_q = dmx->data;
  a.o = static_cast<const uint16_t*>(o);
  a.dout = static_cast<const uint16_t*>(dout);
  a.lse = lse;
  a.sq = sq;
  a.sk = sk;
  a.total_q = total_q;
  a.total_k = total_k;
  a.ptiles_q = ptq;
  a.ptiles_k = ptk;
  a.H = H;
  a.scale = scale;
  // constant P^T scale 2^-8: P <= 1 maps to <= 256
  a.p_sc_const = p_scale == MXFA_P_SCALE_CONST ? 119u : 0u;
  a.causal = causal ? 1 : 0;
  a.dq_mode = dq_mode;
  a.dq_static_scale = dq_mode == 1 ? dq_static_scale : 1.0f;
  a.dq = static_cast<uint16_t*>(dq);
  a.dk = static_cast<uint16_t*>(dk);
  a.dv = static_cast<uint16_t*>(dv);
  if (gmx && gmx[0]) {
    a.dqmx = gmx[0]->data;
    a.dqmx_sfc = gmx[0]->sf_compact;
    a.dqmx_sfp = gmx[0]->sf_packed;
  }
  if (gmx && gmx[1]) {
    a.dkmx = gmx[1]->data;
    a.dkmx_sfc = gmx[1]->sf_compact;
    a.dkmx_sfp = gmx[1]->sf_packed;
  }
  if (gmx && gmx[2]) {
    a.dvmx = gmx[2]->data;
    a.dvmx_sfc = gmx[2]->sf_compact;
    a.dvmx_sfp = gmx[2]->sf_packed;
  }
  a.rec = static_cast<uint8_t*>(ws);
  a.dq_acc = static_cast<uint8_t*>(ws) + bwd_records_bytes(total_q, sq.nseq, H);
  if (!make_map_acc(&a.tm_dqacc, a.dq_acc, total_q, H, dq_mode == 1)) return MXFA_ERR_CUDA;
  a.dense_lse = dense ? 1 : 0;
  a.lse_hstride = dense ? sq.seqlen : total_q;
  return from_cuda(launch_bwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

const char* mxfa_status_string(mxfa_status s) {
  switch (s) {
    case MXFA_OK: return "ok";
    case MXFA_ERR_INVALID_ARG: return "invalid argument";
    case MXFA_ERR_UNSUPPORTED: return "unsupported configuration";
    case MXFA_ERR_MISALIGNED: return "pointer not 16-byte aligned";
    case MXFA_ERR_WORKSPACE_TOO_SMALL: return "workspace too small";
    case MXFA_ERR_CUDA: return "CUDA error";
    case MXFA_ERR_TIMEOUT: return "device wait timed out";
    case MXFA_ERR_DEVICE_INDEX: return "device index check failed";
  }
  return "unknown status";
}

int mxfa_version(void) { return 1; }

int64_t mxfa_packed_tiles(const int32_t* cu, int nseq, int seqlen) {
  if (nseq < 0) return -1;
  if (!cu) return seqlen < 0 ? -1 : int64_t(nseq) * ceil_div(seqlen, 128);
  int64_t t = 0;
  for (int i = 0; i < nseq; i++) {
    int64_t len = int64_t(cu[i + 1]) - cu[i];
    if (len < 0) return -1;
    t += ceil_div(len, 128);
  }
  return t;
}

size_t mxfa_sf_packed_bytes(mxfa_block blk, int64_t tiles, int H) {
  if (tiles < 0 || H <= 0) return 0;
  return size_t(tiles) * size_t(H) * (blk == MXFA_BLK_SQ ? 16u : 512u);
}

mxfa_status mxfa_quantize(const void* x, int64_t tokens, int H, int D, mxfa_block blk,
                          const int32_t* cu, int nseq, int max_seqlen, int64_t packed_tiles,
                          const mxfa_mx_out* out, mxfa_stream_t stream) {
  if (!x || !out || !out->data || H <= 0) return MXFA_ERR_INVALID_ARG;
  if (blk < MXFA_BLK_ROW || blk > MXFA_BLK_SQ) return MXFA_ERR_INVALID_ARG;
  if (D != 128) return MXFA_ERR_UNSUPPORTED;
  mxfa_status s = check_seqs(cu, nseq, max_seqlen, tokens);
  if (s) return s;
  if (!aligned16(x) || !aligned16(out->data)) return MXFA_ERR_MISALIGNED;
  if (out->sf_packed && packed_tiles <= 0) return MXFA_ERR_INVALID_ARG;
  QuantArgs a;
  memset(&a, 0, sizeof(a));
  a.x = static_cast<const uint16_t*>(x);
  a.tokens = tokens;
  a.H = H;
  a.D = D;
  a.mode = int(blk);
  a.seq = Seqs{cu, nseq, max_seqlen};
  a.packed_tiles = packed_tiles;
  a.data = out->data;
  a.sf_compact = out->sf_compact;
  a.sf_packed = out->sf_packed;
  if (tokens == 0) return MXFA_OK;
  return from_cuda(launch_quantize(a, reinterpret_cast<cudaStream_t>(stream)));
}

mxfa_status mxfa_quantize_dual(const void* x, int64_t tokens, int H, int D, mxfa_block blk,
                               const int32_t* cu, int nseq, int max_seqlen, int64_t packed_tiles,
                               const mxfa_mx_out* out, const mxfa_mx_out* out_row, mxfa_stream_t stream) {
  if (!x || !out || !out->data || !out_row || !out_row->data || H <= 0) return MXFA_ERR_INVALID_ARG;
  if (blk != MXFA_BLK_COL && blk != MXFA_BLK_SQ) return MXFA_ERR_INVALID_ARG;
  if (D != 128) return MXFA_ERR_UNSUPPORTED;
  mxfa_status s = check_seqs(cu, nseq, max_seqlen, tokens);
  if (s) return s;
  if (!aligned16(x) || !aligned16(out->data) || !aligned16(out_row->data)) return MXFA_ERR_MISALIGNED;
  if ((out->sf_packed || out_row->sf_packed) && packed_tiles <= 0) return MXFA_ERR_INVALID_ARG;
  QuantArgs a;
  memset(&a, 0, sizeof(a));
  a.x = static_cast<const uint16_t*>(x);
  a.tokens = tokens;
  a.H = H;
  a.D = D;
  a.mode = int(blk);
  a.seq = Seqs{cu, nseq, max_seqlen};
  a.packed_tiles = packed_tiles;
  a.data = out->data;
  a.sf_compact = out->sf_compact;
  a.sf_packed = out->sf_packed;
  a.row_data = out_row->data;
  a.row_sfc = out_row->sf_compact;
  a.row_sfp = out_row->sf_packed;
  if (tokens == 0) return MXFA_OK;
  // dense batches of at least one unit's heads take the streaming kernel (its
  // TMA row coordinate is a 32-bit integer)
  a.has_map = (!cu && H >= kQuantHeadsPerUnit && tokens < (int64_t(1) << 31) &&
               make_map_bf16_rows(&a.tm_x, x, tokens, H, kQuantHeadsPerUnit))
                  ? 1
                  : 0;
  return from_cuda(launch_quantize(a, reinterpret_cast<cudaStream_t>(stream)));
}

mxfa_status mxfa_sf_pack(const uint8_t* sf_compact, int64_t tokens, int H, int D, mxfa_block blk,
                         const int32_t* cu, int nseq, int max_seqlen, int64_t packed_tiles,
                         uint8_t* sf_packed, mxfa_stream_t stream) {
  if (!sf_compact || !sf_packed || H <= 0 || packed_tiles <= 0) return MXFA_ERR_INVALID_ARG;
  if (blk < MXFA_BLK_ROW || blk > MXFA_BLK_SQ) return MXFA_ERR_INVALID_ARG;
  if (D != 128) return MXFA_ERR_UNSUPPORTED;
  mxfa_status s = check_seqs(cu, nseq, max_seqlen, tokens);
  if (s) return s;
  PackArgs a;
  a.sf_compact = sf_compact;
  a.tokens = tokens;
  a.H = H;
  a.D = D;
  a.mode = int(blk);
  a.seq = Seqs{cu, nseq, max_seqlen};
  a.packed_tiles = packed_tiles;
  a.sf_packed = sf_packed;
  if (tokens == 0) return MXFA_OK;
  return from_cuda(launch_sf_pack(a, reinterpret_cast<cudaStream_t>(stream)));
}

mxfa_status mxfa_sf_unpack(const uint8_t* sf_packed, int64_t tokens, int H, int D, mxfa_block blk,
                           const int32_t* cu, int nseq, int max_seqlen, int64_t packed_tiles,
                           uint8_t* sf_compact, mxfa_stream_t stream) {
  if (!sf_compact || !sf_packed || H <= 0 || packed_tiles <= 0) return MXFA_ERR_INVALID_ARG;
  if (blk < MXFA_BLK_ROW || blk > MXFA_BLK_SQ) return MXFA_ERR_INVALID_ARG;
  if (D != 128) return MXFA_ERR_UNSUPPORTED;
  mxfa_status s = check_seqs(cu, nseq, max_seqlen, tokens);
  if (s) return s;
  PackArgs a;
  a.sf_compact = nullptr;
  a.tokens = tokens;
  a.H = H;
  a.D = D;
  a.mode = int(blk);
  a.seq = Seqs{cu, nseq, max_seqlen};
  a.packed_tiles = packed_tiles;
  a.sf_packed = const_cast<uint8_t*>(sf_packed);
  if (tokens == 0) return MXFA_OK;
  return from_cuda(launch_sf_unpack(a, sf_compact, reinterpret_cast<cudaStream_t>(stream)));
}

mxfa_status mxfa_fwd(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v, int B, int S, int H, int D,
                     float softmax_scale, int causal, void* o, float* lse, mxfa_stream_t stream) {
  if (B <= 0 || S <= 0) return MXFA_ERR_INVALID_ARG;
  const int64_t total = int64_t(B) * S;
  mxfa_status s = check_seqs(nullptr, B, S, total);
  if (s) return s;
  const int64_t pt = int64_t(B) * ceil_div(S, 128);
  return fwd_common(q, k, v, Seqs{nullptr, B, S}, Seqs{nullptr, B, S}, total, total, pt, pt, H, D,
                    softmax_scale, causal, o, lse, nullptr, true, stream);
}

mxfa_status mxfa_fwd_mxo(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v, int B, int S, int H,
                         int D, float softmax_scale, int causal, void* o, float* lse,
                         const mxfa_mx_out* o_mx, mxfa_stream_t stream) {
  if (B <= 0 || S <= 0 || !o_mx) return MXFA_ERR_INVALID_ARG;
  const int64_t total = int64_t(B) * S;
  mxfa_status s = check_seqs(nullptr, B, S, total);
  if (s) return s;
  const int64_t pt = int64_t(B) * ceil_div(S, 128);
  return fwd_common(q, k, v, Seqs{nullptr, B, S}, Seqs{nullptr, B, S}, total, total, pt, pt, H, D,
                    softmax_scale, causal, o, lse, o_mx, true, stream);
}

mxfa_status mxfa_varlen_fwd(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v, const int32_t* cu_q,
                            const int32_t* cu_k, int nseq, int max_sq, int max_sk, int64_t total_q,
                            int64_t total_k, int64_t ptq, int64_t ptk, int H, int D, float softmax_scale,
                            int causal, void* o, float* lse, mxfa_stream_t stream) {
  if (!cu_q || !cu_k) return MXFA_ERR_INVALID_ARG;
  mxfa_status s;
  if ((s = check_seqs(cu_q, nseq, max_sq, total_q)) || (s = check_seqs(cu_k, nseq, max_sk, total_k)))
    return s;
  if (max_sk <= 0) return MXFA_ERR_INVALID_ARG;
  return fwd_common(q, k, v, Seqs{cu_q, nseq, max_sq}, Seqs{cu_k, nseq, max_sk}, total_q, total_k, ptq,
                    ptk, H, D, softmax_scale, causal, o, lse, nullptr, false, stream);
}

mxfa_status mxfa_varlen_fwd_mxo(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v,
                                const int32_t* cu_q, const int32_t* cu_k, int nseq, int max_sq,
                                int max_sk, int64_t total_q, int64_t total_k, int64_t ptq, int64_t ptk,
                                int H, int D, float softmax_scale, int causal, void* o, float* lse,
                                const mxfa_mx_out* o_mx, mxfa_stream_t stream) {
  if (!cu_q || !cu_k || !o_mx) return MXFA_ERR_INVALID_ARG;
  mxfa_status s;
  if ((s = check_seqs(cu_q, nseq, max_sq, total_q)) || (s = check_seqs(cu_k, nseq, max_sk, total_k)))
    return s;
  if (max_sk <= 0) return MXFA_ERR_INVALID_ARG;
  return fwd_common(q, k, v, Seqs{cu_q, nseq, max_sq}, Seqs{cu_k, nseq, max_sk}, total_q, total_k, ptq,
                    ptk, H, D, softmax_scale, causal, o, lse, o_mx, false, stream);
}

mxfa_status mxfa_fwd_opts(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v, int B, int S, int H,
                          int D, float softmax_scale, int causal, const mxfa_attn_opts* opts, void* o,
                          float* lse, mxfa_stream_t stream) {
  if (B <= 0 || S <= 0) return MXFA_ERR_INVALID_ARG;
  const int64_t total = int64_t(B) * S;
  mxfa_status s = check_seqs(nullptr, B, S, total);
  if (s) return s;
  const int64_t pt = int64_t(B) * ceil_div(S, 128);
  return fwd_common(q, k, v, Seqs{nullptr, B, S}, Seqs{nullptr, B, S}, total, total, pt, pt, H, D,
                    softmax_scale, causal, o, lse, nullptr, true, stream, opts);
}

mxfa_status mxfa_varlen_fwd_opts(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v,
                                 const int32_t* cu_q, const int32_t* cu_k, int nseq, int max_sq,
                                 int max_sk, int64_t total_q, int64_t total_k, int64_t ptq, int64_t ptk,
                                 int H, int D, float softmax_scale, int causal,
                                 const mxfa_attn_opts* opts, void* o, float* lse, mxfa_stream_t stream) {
  if (!cu_q || !cu_k) return MXFA_ERR_INVALID_ARG;
  mxfa_status s;
  if ((s = check_seqs(cu_q, nseq, max_sq, total_q)) || (s = check_seqs(cu_k, nseq, max_sk, total_k)))
    return s;
  if (max_sk <= 0) return MXFA_ERR_INVALID_ARG;
  return fwd_common(q, k, v, Seqs{cu_q, nseq, max_sq}, Seqs{cu_k, nseq, max_sk}, total_q, total_k, ptq,
                    ptk, H, D, softmax_scale, causal, o, lse, nullptr, false, stream, opts);
}

size_t mxfa_bwd_workspace_size(int64_t total_q, int nseq, int H, int D, int dq_mode) {
  if (total_q < 0 || nseq <= 0 || H <= 0 || D <= 0) return 0;
  return bwd_records_bytes(total_q, nseq, H) + size_t(total_q) * H * D * (dq_mode == 1 ? 2u : 4u);
}

mxfa_status mxfa_bwd(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v, const mxfa_mx* dmx,
                     const void* o, const void* dout, const float* lse, int B, int S, int H, int D,
                     float softmax_scale, int causal, int dq_mode, float dq_static_scale, void* dq,
                     void* dk, void* dv, void* ws, size_t ws_bytes, mxfa_stream_t stream) {
  if (B <= 0 || S <= 0) return MXFA_ERR_INVALID_ARG;
  const int64_t total = int64_t(B) * S;
  mxfa_status s = check_seqs(nullptr, B, S, total);
  if (s) return s;
  const int64_t pt = int64_t(B) * ceil_div(S, 128);
  return bwd_common(q, k, v, dmx, o, dout, lse, Seqs{nullptr, B, S}, Seqs{nullptr, B, S}, total, total,
                    pt, pt, H, D, softmax_scale, causal, dq_mode, dq_static_scale, dq, dk, dv, ws,
                    ws_bytes, nullptr, true, stream);
}

mxfa_status mxfa_bwd_opts(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v, const mxfa_mx* dmx,
                          const void* o, const void* dout, const float* lse, int B, int S, int H, int D,
                          float softmax_scale, int causal, const mxfa_attn_opts* opts, int dq_mode,
                          float dq_static_scale, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                          mxfa_stream_t stream) {
  if (B <= 0 || S <= 0) return MXFA_ERR_INVALID_ARG;
  const int64_t total = int64_t(B) * S;
  mxfa_status s = check_seqs(nullptr, B, S, total);
  if (s) return s;
  const int64_t pt = int64_t(B) * ceil_div(S, 128);
  return bwd_common(q, k, v, dmx, o, dout, lse, Seqs{nullptr, B, S}, Seqs{nullptr, B, S}, total, total,
                    pt, pt, H, D, softmax_scale, causal, dq_mode, dq_static_scale, dq, dk, dv, ws,
                    ws_bytes, nullptr, true, stream, opts);
}

mxfa_status mxfa_varlen_bwd_opts(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v,
                                 const mxfa_mx* dmx, const void* o, const void* dout, const float* lse,
                                 const int32_t* cu_q, const int32_t* cu_k, int nseq, int max_sq,
                                 int max_sk, int64_t total_q, int64_t total_k, int64_t ptq, int64_t ptk,
                                 int H, int D, float softmax_scale, int causal,
                                 const mxfa_attn_opts* opts, int dq_mode, float dq_static_scale,
                                 void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                                 mxfa_stream_t stream) {
  if (!cu_q || !cu_k) return MXFA_ERR_INVALID_ARG;
  mxfa_status s;
  if ((s = check_seqs(cu_q, nseq, max_sq, total_q)) || (s = check_seqs(cu_k, nseq, max_sk, total_k)))
    return s;
  return bwd_common(q, k, v, dmx, o, dout, lse, Seqs{cu_q, nseq, max_sq}, Seqs{cu_k, nseq, max_sk},
                    total_q, total_k, ptq, ptk, H, D, softmax_scale, causal, dq_mode, dq_static_scale,
                    dq, dk, dv, ws, ws_bytes, nullptr, false, stream, opts);
}

mxfa_status mxfa_bwd_mxg(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v, const mxfa_mx* dmx,
                         const void* o, const void* dout, const float* lse, int B, int S, int H, int D,
                         float softmax_scale, int causal, int dq_mode, float dq_static_scale, void* dq,
                         void* dk, void* dv, void* ws, size_t ws_bytes, const mxfa_mx_out* dq_mx,
                         const mxfa_mx_out* dk_mx, const mxfa_mx_out* dv_mx, mxfa_stream_t stream) {
  if (B <= 0 || S <= 0) return MXFA_ERR_INVALID_ARG;
  const int64_t total = int64_t(B) * S;
  mxfa_status s = check_seqs(nullptr, B, S, total);
  if (s) return s;
  const int64_t pt = int64_t(B) * ceil_div(S, 128);
  const mxfa_mx_out* gmx[3] = {dq_mx, dk_mx, dv_mx};
  return bwd_common(q, k, v, dmx, o, dout, lse, Seqs{nullptr, B, S}, Seqs{nullptr, B, S}, total, total,
                    pt, pt, H, D, softmax_scale, causal, dq_mode, dq_static_scale, dq, dk, dv, ws,
                    ws_bytes, gmx, true, stream);
}

mxfa_status mxfa_varlen_bwd(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v, const mxfa_mx* dmx,
                            const void* o, const void* dout, const float* lse, const int32_t* cu_q,
                            const int32_t* cu_k, int nseq, int max_sq, int max_sk, int64_t total_q,
                            int64_t total_k, int64_t ptq, int64_t ptk, int H, int D, float softmax_scale,
                            int causal, int dq_mode, float dq_static_scale, void* dq, void* dk, void* dv,
                            void* ws, size_t ws_bytes, mxfa_stream_t stream) {
  if (!cu_q || !cu_k) return MXFA_ERR_INVALID_ARG;
  mxfa_status s;
  if ((s = check_seqs(cu_q, nseq, max_sq, total_q)) || (s = check_seqs(cu_k, nseq, max_sk, total_k)))
    return s;
  return bwd_common(q, k, v, dmx, o, dout, lse, Seqs{cu_q, nseq, max_sq}, Seqs{cu_k, nseq, max_sk},
                    total_q, total_k, ptq, ptk, H, D, softmax_scale, causal, dq_mode, dq_static_scale,
                    dq, dk, dv, ws, ws_bytes, nullptr, false, stream);
}

mxfa_status mxfa_varlen_bwd_mxg(const mxfa_mx* q, const mxfa_mx* k, const mxfa_mx* v, const mxfa_mx* dmx,
                                const void* o, const void* dout, const float* lse, const int32_t* cu_q,
                                const int32_t* cu_k, int nseq, int max_sq, int max_sk, int64_t total_q,
                                int64_t total_k, int64_t ptq, int64_t ptk, int H, int D,
                                float softmax_scale, int causal, int dq_mode, float dq_static_scale,
                                void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                                const mxfa_mx_out* dq_mx, const mxfa_mx_out* dk_mx,
                                const mxfa_mx_out* dv_mx, mxfa_stream_t stream) {
  if (!cu_q || !cu_k) return MXFA_ERR_INVALID_ARG;
  mxfa_status s;
  if ((s = check_seqs(cu_q, nseq, max_sq, total_q)) || (s = check_seqs(cu_k, nseq, max_sk, total_k)))
    return s;
  const mxfa_mx_out* gmx[3] = {dq_mx, dk_mx, dv_mx};
  return bwd_common(q, k, v, dmx, o, dout, lse, Seqs{cu_q, nseq, max_sq}, Seqs{cu_k, nseq, max_sk},
                    total_q, total_k, ptq, ptk, H, D, softmax_scale, causal, dq_mode, dq_static_scale,
                    dq, dk, dv, ws, ws_bytes, gmx, false, stream);
}

mxfa_status mxfa_rmsnorm_quant(const void* x, const float* gamma, int64_t T, int64_t C, float eps,
                               int seg_len, int H, const mxfa_mx_out* row, const mxfa_mx_out* col,
                               const mxfa_mx_out* sq, mxfa_stream_t stream) {
  if (!x || !gamma || T < 0 || seg_len <= 0 || H <= 0) return MXFA_ERR_INVALID_ARG;
  if (!row && !col && !sq) return MXFA_ERR_INVALID_ARG;
  if (C != 256 && C != 512 && C != 1024 && C != 2048) return MXFA_ERR_UNSUPPORTED;
  if (C % H != 0 || C / H != 128) return MXFA_ERR_UNSUPPORTED;
  if (seg_len % 32 != 0) return MXFA_ERR_UNSUPPORTED;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return MXFA_ERR_INVALID_ARG;
  const mxfa_mx_out* outs[3] = {row, col, sq};
  bool packed = false;
  for (const mxfa_mx_out* m : outs) {
    if (!m) continue;
    if (!m->data) return MXFA_ERR_INVALID_ARG;
    if (!aligned16(m->data)) return MXFA_ERR_MISALIGNED;
    if (m->sf_packed) packed = true;
  }
  if (packed && (seg_len % 128 != 0 || T % seg_len != 0)) return MXFA_ERR_UNSUPPORTED;
  if (!aligned16(x) || !aligned16(gamma)) return MXFA_ERR_MISALIGNED;
  RmsArgs a;
  memset(&a, 0, sizeof(a));
  a.x = static_cast<const uint16_t*>(x);
  a.gamma = gamma;
  a.T = T;
  a.C = int(C);
  a.eps = eps;
  a.seg_len = seg_len;
  a.H = H;
  a.D = 128;
  if (row) { a.row_data = row->data; a.row_sfc = row->sf_compact; a.row_sfp = row->sf_packed; }
  if (col) { a.col_data = col->data; a.col_sfc = col->sf_compact; a.col_sfp = col->sf_packed; }
  if (sq) { a.sq_data = sq->data; a.sq_sfc = sq->sf_compact; a.sq_sfp = sq->sf_packed; }
  if (T == 0) return MXFA_OK;
  return from_cuda(launch_rmsnorm_quant(a, reinterpret_cast<cudaStream_t>(stream)));
}

mxfa_status mxfa_gemm_quant_fmt(const mxfa_mx* a, int a_fmt, const mxfa_mx* b, int b_fmt, int64_t M,
                                int64_t N, int64_t K, void* y_bf16, const mxfa_mx_out* y_row,
                                const mxfa_mx_out* y_col, mxfa_stream_t stream) {
  // element formats -> the MMA kind's format codes
  auto code = [](int f) { return f == MXFA_ELEM_E4M3 ? 0 : f == MXFA_ELEM_E2M3 ? 3 : f == MXFA_ELEM_E3M2 ? 4 : 5; };
  for (int f : {a_fmt, b_fmt})
    if (f != MXFA_ELEM_E4M3 && f != MXFA_ELEM_E2M3 && f != MXFA_ELEM_E3M2 && f != MXFA_ELEM_E2M1)
      return MXFA_ERR_INVALID_ARG;
  return gemm_common(a, code(a_fmt), b, code(b_fmt), M, N, K, y_bf16, y_row, y_col, stream);
}

mxfa_status mxfa_gemm_quant(const mxfa_mx* a, const mxfa_mx* b, int64_t M, int64_t N, int64_t K,
                            void* y_bf16, const mxfa_mx_out* y_row, const mxfa_mx_out* y_col,
                            mxfa_stream_t stream) {
  return gemm_common(a, 0, b, 0, M, N, K, y_bf16, y_row, y_col, stream);
}

mxfa_status mxfa_quantize_lowp(const void* x, int64_t rows, int cols, int fmt, int q_layout, uint8_t* q,
                               uint8_t* sf, uint8_t* sf_packed, float* tensor_scale, mxfa_stream_t stream) {
  if (!x || !q || !sf || rows < 0 || cols <= 0) return MXFA_ERR_INVALID_ARG;
  if (fmt < MXFA_LOWP_MXFP4 || fmt > MXFA_LOWP_NVFP4) return MXFA_ERR_INVALID_ARG;
  if (q_layout != MXFA_LOWP_CODES && q_layout != MXFA_LOWP_MMA) return MXFA_ERR_INVALID_ARG;
  if (q_layout == MXFA_LOWP_MMA && fmt == MXFA_LOWP_NVFP4) return MXFA_ERR_UNSUPPORTED;
  if (cols % (fmt == MXFA_LOWP_NVFP4 ? 16 : 32) != 0) return MXFA_ERR_UNSUPPORTED;
  if (fmt == MXFA_LOWP_NVFP4 && (!tensor_scale || !aligned4(tensor_scale))) return MXFA_ERR_INVALID_ARG;
  if (sf_packed && (fmt == MXFA_LOWP_NVFP4 || rows % 128 != 0 || cols % 128 != 0)) return MXFA_ERR_UNSUPPORTED;
  if (!aligned16(x) || !aligned16(q) || (sf_packed && !aligned16(sf_packed))) return MXFA_ERR_MISALIGNED;
  if (rows * int64_t(cols) >= (int64_t(1) << 40)) return MXFA_ERR_UNSUPPORTED;
  LowpArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.rows = rows;
  a.cols = cols;
  a.fmt = fmt;
  a.q = q;
  a.q_mma = q_layout == MXFA_LOWP_MMA;
  a.sf = sf;
  a.sf_packed = sf_packed;
  a.tensor_scale = tensor_scale;
  return from_cuda(launch_lowp_quantize(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {
mxfa_status gemm_common(const mxfa_mx* a, int a_code, const mxfa_mx* b, int b_code, int64_t M, int64_t N,
                        int64_t K, void* y_bf16, const mxfa_mx_out* y_row, const mxfa_mx_out* y_col,
                        mxfa_stream_t stream) {
  mxfa_status s;
  if ((s = check_mx(a)) || (s = check_mx(b))) return s;
  if (M < 0 || N < 0 || K < 0) return MXFA_ERR_INVALID_ARG;
  if (M % 128 || N % 128 || K % 128) return MXFA_ERR_UNSUPPORTED;
  if (M >= (int64_t(1) << 31) || N >= (int64_t(1) << 24) || K >= (int64_t(1) << 24)) return MXFA_ERR_UNSUPPORTED;
  if (!y_bf16 && !y_row && !y_col) return MXFA_ERR_INVALID_ARG;
  if (y_bf16 && !aligned16(y_bf16)) return MXFA_ERR_MISALIGNED;
  for (const mxfa_mx_out* m : {y_row, y_col}) {
    if (!m) continue;
    if (!m->data) return MXFA_ERR_INVALID_ARG;
    if (!aligned16(m->data) || (m->sf_compact && !aligned4(m->sf_compact)) ||
        (m->sf_packed && !aligned16(m->sf_packed)))
      return MXFA_ERR_MISALIGNED;
  }
  if (M == 0 || N == 0) return MXFA_OK;
  if (K == 0) return MXFA_ERR_UNSUPPORTED;
  GemmArgs g;
  memset(&g, 0, sizeof(g));
  if (!make_map_u8(&g.tm_a, a->data, M, int(K / 128), 128) || !make_map_u8(&g.tm_b, b->data, N, int(K / 128), 128))
    return MXFA_ERR_CUDA;
  g.sfa = a->sf;
  g.sfb = b->sf;
  g.M = M;
  g.N = N;
  g.K = K;
  g.a_fmt = a_code;
  g.b_fmt = b_code;
  g.y_bf16 = static_cast<uint16_t*>(y_bf16);
  if (y_row) { g.row_data = y_row->data; g.row_sfc = y_row->sf_compact; g.row_sfp = y_row->sf_packed; }
  if (y_col) { g.col_data = y_col->data; g.col_sfc = y_col->sf_compact; g.col_sfp = y_col->sf_packed; }
  return from_cuda(launch_gemm_quant(g, reinterpret_cast<cudaStream_t>(stream)));
}
}  // namespace

namespace {

// Checks of a cache, shared by the calls that take one.
mxfa_status check_cache(const mxfa_kv_cache* c, KvPages& p) {
  if (!c || !c->k || !c->v || !c->k_sf || !c->v_sf) return MXFA_ERR_INVALID_ARG;
  if (c->fmt != MXFA_KV_MXFP4 && c->fmt != MXFA_KV_NVFP4) return MXFA_ERR_INVALID_ARG;
  if (c->num_blocks <= 0 || c->page <= 0 || c->H <= 0) return MXFA_ERR_INVALID_ARG;
  if (c->D != 128) return MXFA_ERR_UNSUPPORTED;
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return MXFA_ERR_UNSUPPORTED;
  if (c->num_blocks >= (int64_t(1) << 31) || c->H > 65536) return MXFA_ERR_UNSUPPORTED;
  if (c->fmt == MXFA_KV_NVFP4 && (!c->k_scale || !c->v_scale)) return MXFA_ERR_INVALID_ARG;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_sf) || !aligned16(c->v_sf)) return MXFA_ERR_MISALIGNED;
  if (c->fmt == MXFA_KV_NVFP4 && (!aligned4(c->k_scale) || !aligned4(c->v_scale))) return MXFA_ERR_MISALIGNED;
  p.k = c->k;
  p.v = c->v;
  p.k_sf = c->k_sf;
  p.v_sf = c->v_sf;
  p.k_scale = c->k_scale;
  p.v_scale = c->v_scale;
  p.blocks = c->num_blocks;
  p.page = c->page;
  p.page_shift = c->page == 16 ? 4 : c->page == 32 ? 5 : c->page == 64 ? 6 : 7;
  p.H = c->H;
  p.fmt = c->fmt;
  return MXFA_OK;
}

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// 0: [a, a + na) and [b, b + nb) do not meet; 1: they begin at one place; 2: they overlap
int overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  if (x == y) return 1;
  return x < y + nb && y < x + na ? 2 : 0;
}

struct Range {
  const void* at;
  size_t bytes;
};
bool meet(const Range& a, const Range& b) { return a.bytes && b.bytes && overlap(a.at, a.bytes, b.at, b.bytes) != 0; }
template <typename A, typename B>
bool any_meet(const A& a, const B& b) {
  for (const Range& x : a)
    for (const Range& y : b)
      if (meet(x, y)) return true;
  return false;
}

// The buffers of a (checked) cache: codes and block scales of K and V, then NVFP4's scales.
struct CacheRanges {
  Range r[6];
  const Range* begin() const { return r; }
  const Range* end() const { return r + 6; }
};
CacheRanges ranges_of(const KvPages& c) {
  const size_t rows = size_t(c.blocks) * size_t(c.H) * size_t(c.page), sf = c.fmt == MXFA_KV_NVFP4 ? 8 : 4;
  const size_t st = c.fmt == MXFA_KV_NVFP4 ? 4 : 0;
  return {{{c.k, rows * 64}, {c.v, rows * 64}, {c.k_sf, rows * sf}, {c.v_sf, rows * sf}, {c.k_scale, st}, {c.v_scale, st}}};
}

// Checks of an attention call over the cache, shared by its forms; what they have in common goes into `a`.
mxfa_status check_attn(const mxfa_kv_cache* cache, const void* q, int64_t q_stride, int64_t total_q, const int32_t* cu_q, const int32_t* kv_lens,
                       int R, const int32_t* block_table, int max_blocks, int max_q, int Hq, float softmax_scale, void* o, float* lse, void* ws,
                       KvAttnArgs& a) {
  memset(&a, 0, sizeof(a));
  mxfa_status s = check_cache(cache, a.c);
  if (s) return s;
  if (!q || !cu_q || !kv_lens || !block_table || !o || !lse) return MXFA_ERR_INVALID_ARG;
  if (total_q < 0 || R < 0 || max_blocks <= 0 || max_q < 0 || Hq <= 0 || Hq % a.c.H) return MXFA_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.0f) || !std::isfinite(softmax_scale)) return MXFA_ERR_INVALID_ARG;
  if (total_q > 1 && q_stride < int64_t(Hq) * 128) return MXFA_ERR_INVALID_ARG;
  if (total_q >= (int64_t(1) << 31) || total_q * Hq >= (int64_t(1) << 31) || R > (1 << 20) ||
      int64_t(max_blocks) * a.c.page > (int64_t(1) << 30))
    return MXFA_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(o) || !aligned16(ws) || (total_q > 1 && q_stride % 8)) return MXFA_ERR_MISALIGNED;
  if (!aligned4(cu_q) || !aligned4(kv_lens) || !aligned4(block_table) || !aligned4(lse)) return MXFA_ERR_MISALIGNED;
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.total_q = total_q;
  a.cu_q = cu_q;
  a.kv_lens = kv_lens;
  a.R = R;
  a.table = block_table;
  a.width = max_blocks;
  a.max_q = max_q;
  a.Hq = Hq;
  a.G = Hq / a.c.H;
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.o = static_cast<uint16_t*>(o);
  a.lse = lse;
  a.ws = static_cast<uint8_t*>(ws);
  return MXFA_OK;
}

// The workspace suffices, and what the call writes meets nothing else of it.
mxfa_status check_attn_buffers(const KvAttnArgs& a, size_t need, size_t ws_bytes, const int32_t* starts, const int32_t* prefix_lens, int groups) {
  if (need > 0 && !a.ws) return MXFA_ERR_INVALID_ARG;
  if (ws_bytes < need) return MXFA_ERR_WORKSPACE_TOO_SMALL;
  const size_t row = size_t(a.Hq) * 256, rows = size_t(a.total_q), R = size_t(a.R);
  const Range written[] = {{a.o, rows * row}, {a.lse, rows * size_t(a.Hq) * 4}, {a.ws, need}};
  const Range read[] = {{a.q, (rows - 1) * size_t(a.total_q > 1 ? a.q_stride : 0) * 2 + row}, {a.cu_q, R * 4 + 4}, {a.kv_lens, R * 4},
                        {a.table, R * size_t(a.width) * 4}, {starts, starts ? size_t(groups) * 4 + 4 : 0},
                        {prefix_lens, prefix_lens ? size_t(groups) * 4 : 0}};
  if (any_meet(written, read) || any_meet(written, ranges_of(a.c))) return MXFA_ERR_INVALID_ARG;
  if (meet(written[0], written[1]) || meet(written[0], written[2]) || meet(written[1], written[2])) return MXFA_ERR_INVALID_ARG;
  return MXFA_OK;
}

mxfa_status check_rotation(const mxfa_rotation* r, Rotation& x) {
  if (!r || !r->turns || r->rot <= 0 || r->rot > 128 || !std::isfinite(float(r->gain))) return MXFA_ERR_INVALID_ARG;
  if (r->layout != MXFA_ROPE_HALF && r->layout != MXFA_ROPE_INTERLEAVED) return MXFA_ERR_INVALID_ARG;
  if (r->rot % 16) return MXFA_ERR_UNSUPPORTED;
  if (!aligned8(r->turns)) return MXFA_ERR_MISALIGNED;
  x.turns = reinterpret_cast<const uint64_t*>(r->turns);
  x.rot = r->rot;
  x.inter = r->layout == MXFA_ROPE_INTERLEAVED ? 1 : 0;
  x.inverse = 0;
  x.gain = float(r->gain);
  x.gain_rest = float(r->gain - double(x.gain));
  return MXFA_OK;
}

// Rows of `heads` heads of 128 bf16, `stride` elements apart.
Range rows_range(const void* at, int64_t stride, int64_t tokens, int heads) {
  return {at, size_t(tokens - 1) * size_t(tokens > 1 ? stride : 0) * 2 + size_t(heads) * 256};
}
// Rows of a and of b, of one distance, that lie beside one another.
bool rows_apart(const Range& a, const Range& b, int64_t tokens, int64_t a_stride, int64_t b_stride, int a_heads, int b_heads) {
  if (tokens < 2 || a_stride != b_stride) return false;
  const int64_t period = a_stride * 2, an = int64_t(a_heads) * 256, bn = int64_t(b_heads) * 256;
  const int64_t far = static_cast<const char*>(b.at) - static_cast<const char*>(a.at);
  const int64_t off = (far % period + period) % period;  // of b's rows behind a's
  return off >= an && off + bn <= period;
}

mxfa_status check_pages(const void* table, int R, int max_blocks, int F, const void* refs, int64_t blocks, const void* ring, int64_t ring_size,
                        const void* ring_in, const void* ring_out) {
  if (!table || !refs || !ring || !ring_in || !ring_out) return MXFA_ERR_INVALID_ARG;
  if (R <= 0 || max_blocks <= 0 || F < 0 || blocks <= 0 || ring_size <= 0) return MXFA_ERR_INVALID_ARG;
  if (R > (1 << 20) || F > kKvPlanMaxRequests || int64_t(R) * max_blocks >= (int64_t(1) << 31) || blocks >= (int64_t(1) << 31) ||
      ring_size >= (int64_t(1) << 31))
    return MXFA_ERR_UNSUPPORTED;
  if (!aligned4(table) || !aligned4(refs) || !aligned4(ring) || !aligned8(ring_in) || !aligned8(ring_out)) return MXFA_ERR_MISALIGNED;
  return MXFA_OK;
}

// Whether a written buffer meets another one; `own` (nullable), the last written one, is the last read one in place.
template <size_t N, size_t M>
bool clash(const Range (&written)[N], const Range (&read)[M], const Range* own) {
  for (size_t i = 0; i < N; i++) {
    for (size_t j = 0; j < M; j++)
      if (!(own == &written[i] && j == M - 1) && meet(written[i], read[j])) return true;
    for (size_t j = i + 1; j < N; j++)
      if (meet(written[i], written[j])) return true;
  }
  return false;
}

}  // namespace

extern "C" {

size_t mxfa_kv_codes_bytes(int64_t num_blocks, int page, int H) {
  if (num_blocks < 0 || page <= 0 || H <= 0) return 0;
  return size_t(num_blocks) * size_t(page) * size_t(H) * 64u;
}

size_t mxfa_kv_sf_bytes(int64_t num_blocks, int page, int H, int fmt) {
  if (num_blocks < 0 || page <= 0 || H <= 0) return 0;
  return size_t(num_blocks) * size_t(page) * size_t(H) * (fmt == MXFA_KV_NVFP4 ? 8u : 4u);
}

mxfa_status mxfa_kv_plan(const int32_t* ctx_lens, const int32_t* new_lens, int R, int32_t* block_table,
                         int max_blocks, int32_t* free_ring, int64_t ring_size, const int64_t* ring_in,
                         int64_t* ring_out, int page, int64_t tokens, int32_t* cu_q, int32_t* kv_lens,
                         int64_t* slots, int32_t* positions, mxfa_stream_t stream) {
  if (R < 0 || max_blocks <= 0 || ring_size <= 0 || tokens < 0) return MXFA_ERR_INVALID_ARG;
  if (!free_ring || !ring_in || !ring_out || !cu_q) return MXFA_ERR_INVALID_ARG;
  if (R > 0 && (!ctx_lens || !new_lens || !block_table || !kv_lens)) return MXFA_ERR_INVALID_ARG;
  if (tokens > 0 && (!slots || !positions)) return MXFA_ERR_INVALID_ARG;
  if (page != 16 && page != 32 && page != 64 && page != 128) return MXFA_ERR_UNSUPPORTED;
  if (R > kKvPlanMaxRequests || tokens >= (int64_t(1) << 31) || ring_size >= (int64_t(1) << 31) ||
      int64_t(max_blocks) * page > (int64_t(1) << 30) || int64_t(R) * max_blocks >= (int64_t(1) << 31))
    return MXFA_ERR_UNSUPPORTED;
  for (const void* p : {static_cast<const void*>(ctx_lens), static_cast<const void*>(new_lens),
                        static_cast<const void*>(block_table), static_cast<const void*>(free_ring),
                        static_cast<const void*>(cu_q), static_cast<const void*>(kv_lens),
                        static_cast<const void*>(positions)})
    if (!aligned4(p)) return MXFA_ERR_MISALIGNED;
  if (!aligned8(ring_in) || !aligned8(ring_out) || !aligned8(slots)) return MXFA_ERR_MISALIGNED;
  const size_t lens = size_t(R) * 4;
  const int same_len = R > 0 ? overlap(ctx_lens, lens, kv_lens, lens) : 0;
  const int same_ring = overlap(ring_in, 24, ring_out, 24);
  if (same_len == 2 || same_ring == 2) return MXFA_ERR_INVALID_ARG;
  // every CTA reads the inputs while others write: no other two buffers may meet
  const size_t toks = size_t(tokens);
  const Range written[] = {{block_table, lens * size_t(max_blocks)}, {free_ring, size_t(ring_size) * 4}, {cu_q, lens + 4},
                           {slots, toks * 8}, {positions, toks * 4}, {ring_out, 24}, {kv_lens, lens}};
  const Range read[] = {{new_lens, lens}, {ctx_lens, lens}, {ring_in, 24}};
  for (const Range& w : written) {
    for (const Range& r : read) {
      const bool own = (w.at == kv_lens && r.at == ctx_lens && same_len) || (w.at == ring_out && r.at == ring_in && same_ring);
      if (!own && meet(w, r)) return MXFA_ERR_INVALID_ARG;
    }
    for (const Range& o : written)
      if (&o != &w && meet(w, o)) return MXFA_ERR_INVALID_ARG;
  }
  KvPlanArgs a;
  memset(&a, 0, sizeof(a));
  a.ctx = ctx_lens;
  a.add = new_lens;
  a.R = R;
  a.table = block_table;
  a.width = max_blocks;
  a.ring = free_ring;
  a.ring_size = ring_size;
  a.ring_in = ring_in;
  a.ring_out = ring_out;
  a.page_shift = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
  a.tokens = tokens;
  a.cu_q = cu_q;
  a.kv_lens = kv_lens;
  a.slots = slots;
  a.positions = positions;
  a.aliased = same_len == 1 || same_ring == 1;
  return from_cuda(launch_kv_plan(a, reinterpret_cast<cudaStream_t>(stream)));
}

mxfa_status mxfa_kv_append(const mxfa_kv_cache* cache, const void* k, const void* v, int64_t k_stride,
                           int64_t v_stride, int64_t tokens, const int64_t* slots, mxfa_stream_t stream) {
  KvRowsArgs a;
  memset(&a, 0, sizeof(a));
  mxfa_status s = check_cache(cache, a.c);
  if (s) return s;
  if (!k || !v || !slots || tokens < 0) return MXFA_ERR_INVALID_ARG;
  if (tokens > 1 && (k_stride < int64_t(a.c.H) * 128 || v_stride < int64_t(a.c.H) * 128)) return MXFA_ERR_INVALID_ARG;
  if (tokens >= (int64_t(1) << 31) || tokens * a.c.H >= (int64_t(1) << 31) - 128) return MXFA_ERR_UNSUPPORTED;
  if (!aligned16(k) || !aligned16(v) || !aligned8(slots) || (tokens > 1 && (k_stride % 8 || v_stride % 8)))
    return MXFA_ERR_MISALIGNED;
  if (tokens == 0) return MXFA_OK;
  // what is written (codes and block scales) meets neither what is read nor itself
  const CacheRanges own = ranges_of(a.c);
  const size_t row = size_t(a.c.H) * 256, steps = size_t(tokens) - 1;
  const Range read[] = {{k, steps * size_t(k_stride) * 2 + row}, {v, steps * size_t(v_stride) * 2 + row}, {slots, size_t(tokens) * 8}};
  for (int i = 0; i < 4; i++) {
    for (const Range& x : read)
      if (meet(own.r[i], x)) return MXFA_ERR_INVALID_ARG;
    for (int j = i + 1; j < 6; j++)
      if (meet(own.r[i], own.r[j])) return MXFA_ERR_INVALID_ARG;
  }
  a.k = const_cast<uint16_t*>(static_cast<const uint16_t*>(k));
  a.v = const_cast<uint16_t*>(static_cast<const uint16_t*>(v));
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.tokens = tokens;
  a.slots = slots;
  return from_cuda(launch_kv_append(a, reinterpret_cast<cudaStream_t>(stream)));
}

mxfa_status mxfa_kv_load(const mxfa_kv_cache* cache, const int64_t* slots, int64_t tokens, void* k, void* v,
                         mxfa_stream_t stream) {
  KvRowsArgs a;
  memset(&a, 0, sizeof(a));
  mxfa_status s = check_cache(cache, a.c);
  if (s) return s;
  if (!k || !v || !slots || tokens < 0) return MXFA_ERR_INVALID_ARG;
  if (tokens >= (int64_t(1) << 31) || tokens * a.c.H >= (int64_t(1) << 31) - 128) return MXFA_ERR_UNSUPPORTED;
  if (!aligned16(k) || !aligned16(v) || !aligned8(slots)) return MXFA_ERR_MISALIGNED;
  if (tokens == 0) return MXFA_OK;
  const size_t bytes = size_t(tokens) * size_t(a.c.H) * 256;
  const Range written[] = {{k, bytes}, {v, bytes}}, sr{slots, size_t(tokens) * 8};
  if (meet(written[0], written[1]) || meet(written[0], sr) || meet(written[1], sr)) return MXFA_ERR_INVALID_ARG;
  if (any_meet(written, ranges_of(a.c))) return MXFA_ERR_INVALID_ARG;
  a.k = static_cast<uint16_t*>(k);
  a.v = static_cast<uint16_t*>(v);
  a.tokens = tokens;
  a.slots = slots;
  return from_cuda(launch_kv_load(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t mxfa_kv_attn_workspace_size(int R, int max_q, int64_t max_k, int Hq, int H) {
  if (R < 0 || max_q < 0 || max_k < 0 || H <= 0 || Hq <= 0 || Hq % H) return 0;
  return kv_attn_workspace(R, max_q, max_k, Hq / H);
}

mxfa_status mxfa_kv_attn(const mxfa_kv_cache* cache, const void* q, int64_t q_stride, int64_t total_q,
                         const int32_t* cu_q, const int32_t* kv_lens, int R, const int32_t* block_table,
                         int max_blocks, int max_q, int Hq, float softmax_scale, int causal, void* o,
                         float* lse, void* ws, size_t ws_bytes, mxfa_stream_t stream) {
  KvAttnArgs a;
  const mxfa_status s = check_attn(cache, q, q_stride, total_q, cu_q, kv_lens, R, block_table, max_blocks, max_q, Hq, softmax_scale, o, lse, ws, a);
  if (s) return s;
  if (total_q == 0 || R == 0 || max_q == 0) return MXFA_OK;
  a.causal = causal ? 1 : 0;
  const int64_t max_k = int64_t(max_blocks) * a.c.page;
  if (!kv_attn_reaches(max_q, max_k, a.G)) return MXFA_ERR_UNSUPPORTED;
  const mxfa_status t = check_attn_buffers(a, kv_attn_workspace(R, max_q, max_k, a.G), ws_bytes, nullptr, nullptr, 0);
  return t ? t : from_cuda(launch_kv_attn(kAll, a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t mxfa_kv_attn_window_workspace_size(int R, int max_q, int64_t max_k, int Hq, int H, int window, int sinks) {
  if (R < 0 || max_q < 0 || max_k < 0 || H <= 0 || Hq <= 0 || Hq % H || window < 1 || sinks < 0) return 0;
  return kv_attn_workspace(R, max_q, kv_window_reach(max_q, max_k, window, sinks), Hq / H);
}

mxfa_status mxfa_kv_attn_window(const mxfa_kv_cache* cache, const void* q, int64_t q_stride, int64_t total_q,
                                const int32_t* cu_q, const int32_t* kv_lens, int R, const int32_t* block_table,
                                int max_blocks, int max_q, int Hq, float softmax_scale, int window, int sinks,
                                void* o, float* lse, void* ws, size_t ws_bytes, mxfa_stream_t stream) {
  KvAttnArgs a;
  const mxfa_status s = check_attn(cache, q, q_stride, total_q, cu_q, kv_lens, R, block_table, max_blocks, max_q, Hq, softmax_scale, o, lse, ws, a);
  if (s) return s;
  if (window < 1 || sinks < 0) return MXFA_ERR_INVALID_ARG;
  if (total_q == 0 || R == 0 || max_q == 0) return MXFA_OK;
  a.causal = 1;
  // no context is longer than 2^30 keys
  a.window = window < (1 << 30) ? window : 1 << 30;
  a.sinks = sinks < (1 << 30) ? sinks : 1 << 30;
  const int64_t max_k = kv_window_reach(max_q, int64_t(max_blocks) * a.c.page, a.window, a.sinks);
  if (!kv_attn_reaches(max_q, max_k, a.G)) return MXFA_ERR_UNSUPPORTED;
  const mxfa_status t = check_attn_buffers(a, kv_attn_workspace(R, max_q, max_k, a.G), ws_bytes, nullptr, nullptr, 0);
  return t ? t : from_cuda(launch_kv_attn(kWindow, a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t mxfa_kv_attn_shared_workspace_size(int R, int groups, int64_t total_q, int max_q, int max_group_q, int64_t max_k,
                                          int Hq, int H) {
  return mxfa_kv_attn_shared_workspace_size_mode(R, groups, total_q, max_q, max_group_q, max_k, Hq, H, MXFA_KV_SHARE_AUTO);
}

size_t mxfa_kv_attn_shared_workspace_size_mode(int R, int groups, int64_t total_q, int max_q, int max_group_q, int64_t max_k,
                                               int Hq, int H, int share) {
  if (share != MXFA_KV_SHARE_AUTO && share != MXFA_KV_SHARE_ALWAYS && share != MXFA_KV_SHARE_NEVER) return 0;
  if (R < 0 || groups < 0 || total_q < 0 || max_q < 0 || max_group_q < 0 || max_k < 0 || H <= 0 || Hq <= 0 || Hq % H) return 0;
  if (groups == 0) return kv_attn_workspace(R, max_q, max_k, Hq / H);
  return kv_shared_workspace(R, groups, total_q, max_q, max_group_q, max_k, Hq, Hq / H, share);
}

mxfa_status mxfa_kv_attn_shared(const mxfa_kv_cache* cache, const void* q, int64_t q_stride, int64_t total_q,
                                const int32_t* cu_q, const int32_t* kv_lens, int R, const int32_t* block_table,
                                int max_blocks, int max_q, int Hq, float softmax_scale, const int32_t* group_starts,
                                const int32_t* prefix_lens, int groups, int max_group_q, int share, void* o, float* lse,
                                void* ws, size_t ws_bytes, mxfa_stream_t stream) {
  KvAttnArgs a;
  const mxfa_status s = check_attn(cache, q, q_stride, total_q, cu_q, kv_lens, R, block_table, max_blocks, max_q, Hq, softmax_scale, o, lse, ws, a);
  if (s) return s;
  if (share != MXFA_KV_SHARE_AUTO && share != MXFA_KV_SHARE_ALWAYS && share != MXFA_KV_SHARE_NEVER) return MXFA_ERR_INVALID_ARG;
  if (groups < 0 || max_group_q < 0 || (groups > 0 && (!group_starts || !prefix_lens))) return MXFA_ERR_INVALID_ARG;
  if (!aligned4(group_starts) || !aligned4(prefix_lens)) return MXFA_ERR_MISALIGNED;
  if (groups > (1 << 20)) return MXFA_ERR_UNSUPPORTED;
  if (total_q == 0 || R == 0 || max_q == 0) return MXFA_OK;
  a.causal = 1;
  const int64_t max_k = int64_t(max_blocks) * a.c.page;
  if (!kv_attn_reaches(max_q, max_k, a.G) || (groups > 0 && !kv_attn_reaches(max_group_q, max_k, a.G))) return MXFA_ERR_UNSUPPORTED;
  const size_t need = mxfa_kv_attn_shared_workspace_size_mode(R, groups, total_q, max_q, max_group_q, max_k, Hq, a.c.H, share);
  const mxfa_status t = check_attn_buffers(a, need, ws_bytes, group_starts, prefix_lens, groups);
  if (t) return t;
  if (groups == 0) return from_cuda(launch_kv_attn(kAll, a, reinterpret_cast<cudaStream_t>(stream)));
  a.starts = group_starts;
  return from_cuda(launch_kv_attn_shared(a, prefix_lens, groups, max_group_q, share, reinterpret_cast<cudaStream_t>(stream)));
}

mxfa_status mxfa_rope(const void* x, int64_t x_stride, void* y, int64_t y_stride, const int32_t* positions,
                      int64_t tokens, int H, int D, const mxfa_rotation* rot, int inverse, mxfa_stream_t stream) {
  RopeArgs a;
  memset(&a, 0, sizeof(a));
  mxfa_status s = check_rotation(rot, a.rot);
  if (s) return s;
  if (!x || !y || !positions || tokens < 0 || H <= 0) return MXFA_ERR_INVALID_ARG;
  if (tokens > 1 && (x_stride < int64_t(H) * 128 || y_stride < int64_t(H) * 128)) return MXFA_ERR_INVALID_ARG;
  if (D != 128 || H > 65536 || tokens >= (int64_t(1) << 31) || tokens * H >= (int64_t(1) << 31)) return MXFA_ERR_UNSUPPORTED;
  if (!aligned16(x) || !aligned16(y) || !aligned4(positions) || (tokens > 1 && (x_stride % 8 || y_stride % 8))) return MXFA_ERR_MISALIGNED;
  if (tokens == 0) return MXFA_OK;
  const Range xr = rows_range(x, x_stride, tokens, H), yr = rows_range(y, y_stride, tokens, H);
  const bool in_place = x == y && (tokens == 1 || x_stride == y_stride);
  const Range read[] = {{positions, size_t(tokens) * 4}, {a.rot.turns, size_t(a.rot.rot) * 4}};
  if ((!in_place && meet(xr, yr)) || meet(yr, read[0]) || meet(yr, read[1])) return MXFA_ERR_INVALID_ARG;
  a.rot.inverse = inverse ? 1 : 0;
  a.x = static_cast<const uint16_t*>(x);
  a.y = static_cast<uint16_t*>(y);
  a.x_stride = x_stride;
  a.y_stride = y_stride;
  a.positions = positions;
  a.tokens = tokens;
  a.H = H;
  return from_cuda(launch_rope(a, reinterpret_cast<cudaStream_t>(stream)));
}

mxfa_status mxfa_kv_append_rope(const mxfa_kv_cache* cache, const void* q, int64_t q_stride, int Hq, const void* k,
                                int64_t k_stride, const void* v, int64_t v_stride, int64_t tokens,
                                const int32_t* positions, const int64_t* slots, const mxfa_rotation* rot, void* q_out,
                                int64_t q_out_stride, mxfa_stream_t stream) {
  KvAppendRopeArgs a;
  memset(&a, 0, sizeof(a));
  mxfa_status s = check_cache(cache, a.c);
  if (s || (s = check_rotation(rot, a.rot))) return s;
  if (!q || !k || !v || !positions || !slots || !q_out || tokens < 0 || Hq <= 0) return MXFA_ERR_INVALID_ARG;
  const int64_t kv_row = int64_t(a.c.H) * 128, q_row = int64_t(Hq) * 128;
  if (tokens > 1 && (k_stride < kv_row || v_stride < kv_row || q_stride < q_row || q_out_stride < q_row)) return MXFA_ERR_INVALID_ARG;
  if (Hq > 65536 || tokens >= (int64_t(1) << 31) || tokens * (int64_t(Hq) + 2 * int64_t(a.c.H)) >= (int64_t(1) << 31)) return MXFA_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned4(positions) || !aligned8(slots) ||
      (tokens > 1 && (q_stride % 8 || k_stride % 8 || v_stride % 8 || q_out_stride % 8)))
    return MXFA_ERR_MISALIGNED;
  if (tokens == 0) return MXFA_OK;
  // what is written (the turned q, codes and block scales) meets neither what is read nor itself, but for q in place
  const CacheRanges own = ranges_of(a.c);
  const Range out = rows_range(q_out, q_out_stride, tokens, Hq), qr = rows_range(q, q_stride, tokens, Hq);
  const Range read[] = {rows_range(k, k_stride, tokens, a.c.H), rows_range(v, v_stride, tokens, a.c.H), {positions, size_t(tokens) * 4},
                        {slots, size_t(tokens) * 8}, {a.rot.turns, size_t(a.rot.rot) * 4}};
  const bool in_place = q == q_out && (tokens == 1 || q_stride == q_out_stride);
  if (!in_place && meet(out, qr)) return MXFA_ERR_INVALID_ARG;
  for (const Range& x : read)
    // q in place may be a part of the projection that k and v are other parts of
    if (meet(out, x) && !(in_place && (&x == &read[0] || &x == &read[1]) && rows_apart(out, x, tokens, q_out_stride, &x == &read[0] ? k_stride : v_stride, Hq, a.c.H)))
      return MXFA_ERR_INVALID_ARG;
  for (int i = 0; i < 6; i++) {
    if (meet(own.r[i], out)) return MXFA_ERR_INVALID_ARG;
    if (i >= 4) continue;
    if (meet(own.r[i], qr)) return MXFA_ERR_INVALID_ARG;
    for (const Range& x : read)
      if (meet(own.r[i], x)) return MXFA_ERR_INVALID_ARG;
    for (int j = i + 1; j < 6; j++)
      if (meet(own.r[i], own.r[j])) return MXFA_ERR_INVALID_ARG;
  }
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.y = static_cast<uint16_t*>(q_out);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.y_stride = q_out_stride;
  a.tokens = tokens;
  a.Hq = Hq;
  a.positions = positions;
  a.slots = slots;
  return from_cuda(launch_kv_append_rope(a, reinterpret_cast<cudaStream_t>(stream)));
}

mxfa_status mxfa_kv_fork(int32_t* block_table, int R, int max_blocks, const int32_t* src, const int32_t* dst,
                         const int32_t* lens, int F, int32_t* refs, int64_t num_blocks, const int32_t* free_ring,
                         int64_t ring_size, const int64_t* ring_in, int64_t* ring_out, int page, int32_t* from_blocks,
                         int32_t* to_blocks, int32_t* lens_out, mxfa_stream_t stream) {
  return mxfa_kv_fork_gap(block_table, R, max_blocks, src, dst, lens, nullptr, nullptr, F, refs, num_blocks, free_ring, ring_size, ring_in,
                          ring_out, page, from_blocks, to_blocks, lens_out, stream);
}

mxfa_status mxfa_kv_fork_gap(int32_t* block_table, int R, int max_blocks, const int32_t* src, const int32_t* dst,
                             const int32_t* lens, const int32_t* gap_first, const int32_t* gap_end, int F, int32_t* refs,
                             int64_t num_blocks, const int32_t* free_ring, int64_t ring_size, const int64_t* ring_in,
                             int64_t* ring_out, int page, int32_t* from_blocks, int32_t* to_blocks, int32_t* lens_out,
                             mxfa_stream_t stream) {
  mxfa_status s = check_pages(block_table, R, max_blocks, F, refs, num_blocks, free_ring, ring_size, ring_in, ring_out);
  if (s) return s;
  if ((gap_first == nullptr) != (gap_end == nullptr)) return MXFA_ERR_INVALID_ARG;
  if (F > 0 && (!src || !dst || !lens || !from_blocks || !to_blocks || !lens_out)) return MXFA_ERR_INVALID_ARG;
  if (page != 16 && page != 32 && page != 64 && page != 128) return MXFA_ERR_UNSUPPORTED;
  if (int64_t(max_blocks) * page > (int64_t(1) << 30)) return MXFA_ERR_UNSUPPORTED;
  for (const void* p : {static_cast<const void*>(src), static_cast<const void*>(dst), static_cast<const void*>(lens),
                        static_cast<const void*>(gap_first), static_cast<const void*>(gap_end),
                        static_cast<const void*>(from_blocks), static_cast<const void*>(to_blocks), static_cast<const void*>(lens_out)})
    if (!aligned4(p)) return MXFA_ERR_MISALIGNED;
  const size_t list = size_t(F) * 4;
  const Range written[] = {{block_table, size_t(R) * size_t(max_blocks) * 4}, {refs, size_t(num_blocks) * 4}, {from_blocks, list},
                           {to_blocks, list}, {lens_out, list}, {ring_out, 24}};
  const size_t gaps = gap_first ? list : 0;
  const Range read[] = {{src, list}, {dst, list}, {lens, list}, {gap_first, gaps}, {gap_end, gaps}, {free_ring, size_t(ring_size) * 4}, {ring_in, 24}};
  if (clash(written, read, ring_in == ring_out ? &written[5] : nullptr)) return MXFA_ERR_INVALID_ARG;
  KvForkArgs a;
  memset(&a, 0, sizeof(a));
  a.table = block_table;
  a.R = R;
  a.width = max_blocks;
  a.src = src;
  a.dst = dst;
  a.lens = lens;
  a.gap_first = gap_first;
  a.gap_end = gap_end;
  a.F = F;
  a.refs = refs;
  a.blocks = num_blocks;
  a.ring = free_ring;
  a.ring_size = ring_size;
  a.ring_in = ring_in;
  a.ring_out = ring_out;
  a.page_shift = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
  a.from_blocks = from_blocks;
  a.to_blocks = to_blocks;
  a.lens_out = lens_out;
  return from_cuda(launch_kv_fork(a, reinterpret_cast<cudaStream_t>(stream)));
}

mxfa_status mxfa_kv_free(const int32_t* block_table, int R, int max_blocks, const int32_t* rows, const int32_t* first,
                         const int32_t* end, int F, int32_t* refs, int64_t num_blocks, int32_t* free_ring,
                         int64_t ring_size, const int64_t* ring_in, int64_t* ring_out, mxfa_stream_t stream) {
  mxfa_status s = check_pages(block_table, R, max_blocks, F, refs, num_blocks, free_ring, ring_size, ring_in, ring_out);
  if (s) return s;
  if (F > 0 && (!rows || !first || !end)) return MXFA_ERR_INVALID_ARG;
  if (ring_size < num_blocks) return MXFA_ERR_INVALID_ARG;
  if (max_blocks > (1 << 26)) return MXFA_ERR_UNSUPPORTED;
  if (!aligned4(rows) || !aligned4(first) || !aligned4(end)) return MXFA_ERR_MISALIGNED;
  const size_t list = size_t(F) * 4;
  const Range written[] = {{refs, size_t(num_blocks) * 4}, {free_ring, size_t(ring_size) * 4}, {ring_out, 24}};
  const Range read[] = {{block_table, size_t(R) * size_t(max_blocks) * 4}, {rows, list}, {first, list}, {end, list}, {ring_in, 24}};
  if (clash(written, read, ring_in == ring_out ? &written[2] : nullptr)) return MXFA_ERR_INVALID_ARG;
  KvFreeArgs a;
  memset(&a, 0, sizeof(a));
  a.table = block_table;
  a.R = R;
  a.width = max_blocks;
  a.rows = rows;
  a.first = first;
  a.end = end;
  a.F = F;
  a.refs = refs;
  a.blocks = num_blocks;
  a.ring = free_ring;
  a.ring_size = ring_size;
  a.ring_in = ring_in;
  a.ring_out = ring_out;
  return from_cuda(launch_kv_free(a, reinterpret_cast<cudaStream_t>(stream)));
}

mxfa_status mxfa_kv_copy_blocks(const mxfa_kv_cache* cache, const int32_t* from_blocks, const int32_t* to_blocks, int n,
                                mxfa_stream_t stream) {
  KvPages c;
  const mxfa_status s = check_cache(cache, c);
  if (s) return s;
  if (n < 0 || !from_blocks || !to_blocks) return MXFA_ERR_INVALID_ARG;
  if (!aligned4(from_blocks) || !aligned4(to_blocks)) return MXFA_ERR_MISALIGNED;
  if (n > kKvCopyMost) return MXFA_ERR_UNSUPPORTED;
  if (n == 0) return MXFA_OK;
  const CacheRanges own = ranges_of(c);
  const Range read[] = {{from_blocks, size_t(n) * 4}, {to_blocks, size_t(n) * 4}};
  for (int i = 0; i < 4; i++) {
    if (meet(own.r[i], read[0]) || meet(own.r[i], read[1])) return MXFA_ERR_INVALID_ARG;
    for (int j = i + 1; j < 6; j++)
      if (meet(own.r[i], own.r[j])) return MXFA_ERR_INVALID_ARG;
  }
  return from_cuda(launch_kv_copy(c, from_blocks, to_blocks, n, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"

extern "C" {

mxfa_status mxfa_tensor_peak_probe(int iters, int ctas, unsigned long long* cycles, mxfa_stream_t stream) {
  if (iters <= 0 || ctas <= 0 || !cycles) return MXFA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(cycles) & 7u) return MXFA_ERR_MISALIGNED;
  return from_cuda(launch_mma_peak(iters, ctas, cycles, reinterpret_cast<cudaStream_t>(stream)));
}

mxfa_status mxfa_get_device_status(mxfa_stream_t stream, unsigned* flags) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(st) != cudaSuccess) return MXFA_ERR_CUDA;
  unsigned f = read_status_quant(st) | read_status_fwd(st) | read_status_bwd(st) | read_status_gemm(st) | read_status_kv(st) |
               read_status_kv_attn(st) | read_status_kv_prefill(st) | read_status_rope(st) | read_status_kv_pages(st) |
               read_status_kv_shared(st);
  if (flags) *flags = f;
  if (f & 1u) return MXFA_ERR_TIMEOUT;
  if (f & 2u) return MXFA_ERR_DEVICE_INDEX;
  return MXFA_OK;
}

}  // extern "C"
