// kv_attn.cu -- attention over the 4-bit key/value cache for few query rows:
// decoding steps and drafted tokens.
//
//   o = softmax(scale q K^T) V,  lse = log sum exp(scale q K^T)
// per query row, K and V the cache rows of the request's block table, causal
// aligned to the end (query i of n sees keys j <= kv - n + i).
//
// Numbers.  A cached value is code x scale with both factors and the product
// exact in binary16 (MXFP4 scales are clamped to [2^-23, 2^13] by the store; an
// NVFP4 product has 6 significant bits in [2^-10, 2688]); NVFP4's fp32 scale of
// the whole cache joins the softmax scale (K) and the final factor (V).  q goes
// to binary16 with a power of two per row that puts its largest element in
// [2^14, 2^15): bf16 has 8 significant bits, so only elements 2^28 below the
// row's largest lose any.  The products accumulate in fp32.  P = 2^(s - m + 8)
// is rounded to binary16 (11 bits; relative 2^-11, against 2^-8 for the bf16
// result), where the offset 8 keeps weights down to 2^-32 of the largest from
// vanishing; m moves when a score exceeds it by more than 6, so P <= 2^14.
//
// Work.  The key tiles (128 keys) of all (request, key head, block of query
// rows) items form one line, with kItemTiles units more for each item, cut into
// equal runs, one per CTA: no CTA has more than one unit above another whatever the
// lengths.  An item inside one run is finished there; one cut by a border leaves
// partial (m, l, O) records that a second kernel joins in the order of the keys, so
// results do not depend on timing.  Where all contexts are short (kWholeTiles) there is
// no line: whole items go round the CTAs, whose tiles may then differ.  Each of the CTA's four warps takes 32 of a tile's keys with its own
// ring of asynchronous copies and its own softmax state, so warps never wait on
// one another inside an item.
//
// Fragments.  m16n8k16 with sixteen keys (then sixteen channels) as M and eight
// query rows as N, so that a group of up to eight heads fills the tensor core's
// tile: S^T = K Q^T, O^T += V^T P^T, with P^T's fragment from S^T's by an 8x8
// transpose (movmatrix).  The contraction order is free as long as both operands
// agree, so a lane's K fragments over all of D are the 32 consecutive channels
// (one 16-byte load, one MXFP4 block) of its key, and Q is laid out to match;
// its V fragments are 16 consecutive channels of four keys, two keys' codes
// merged into bytes before conversion so that the pair (key, key + 1) comes
// out of one conversion.
//
// What bounds it.  Latency: 3.7 warps a scheduler, each on one chain of dependent
// instructions (617 a warp for 32 keys and one tile of rows, a quarter of them
// conversions), keep the schedulers 55%, the ALUs 45% and HBM 54% busy; no unit is full.
// 64 requests of up to 8192 keys, 8 key heads, G = 4, MXFP4: 65 us, 3.8 TB/s (57% of a
// copy's rate); three of 97,000 to 130,000 keys, G = 8, NVFP4: 87 us, 4.4 TB/s.  Requests
// of 24 to 48 rows (3 to 6 tokens x 8) over up to 12288 keys: 107 us, 214 TFLOP/s; there
// every tile of rows adds 150 instructions, and a second block of rows converts the
// cache again.  Other forms, in their time: query rows as M 115 us for the first case
// where keys as M took 88; bulk copies 91 where these took 85; two chains of score
// products, no change.
//
// Windows and prefixes (KvKind).  With a window a row sees the first `sinks` keys and the
// last `window` ones: the tiles that hold neither are no part of the line, table entries of
// hidden keys are not read, and steps without a key in sight are left out.  16 requests of up
// to 32768 keys, window 4096, 4 sinks, 8 key heads, G = 4: 30 us (floor 10): the same chain,
// and 8 units a CTA to spread its start over.  Prefixes and what is behind them: kv_shared.cu.
#include "kv_fp4.cuh"
#include "mx_ptx.cuh"
#include "mxfa_internal.h"

namespace mxfa {

static __device__ unsigned g_status_kv_attn;

namespace kva {

constexpr int kStep = 32;                 // keys of one warp step
constexpr int kTile = 128;                // keys of one CTA step, by which work is counted and cut
constexpr int kStages = 3;
constexpr float kOffset = 8.0f;           // log2 offset of P
constexpr float kLazy = 6.0f;             // growth of a row maximum that moves m
constexpr int kMaxNt = 4;                 // blocks of at most 32 query rows
constexpr int kMinTiles = 4;              // least units of a run, as long as items are cut
// Contexts of at most as many tiles (1024 keys) are not cut at all: us for 1, 16 and 64
// requests of 512 keys 7.7, 8.2, 16.3 whole and 10.8, 13.0, 21.6 cut; of 1024 keys
// 11.8, 12.0, 24.6 and 11.4, 14.7, 29.8; of 2048 keys 19.4, 21.9, 40.7 and 11.6, 20.9, 44.5.
constexpr int kWholeTiles = 8;
// What an item costs beside its tiles (drain, merge), in tiles: 1, 2, 3 and 4 took 133,
// 116, 110.7 and 110.7 us for the drafted tokens above, 72.6, 66.8, 65.9 and 66.7 us for
// the 64 requests.
constexpr int kItemTiles = 3;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
// CTAs of an SM for NT 8-row tiles: 16, 12 or 8 warps, as 32 NT accumulator registers
// a thread allow.
__host__ __device__ constexpr int ctas_per_sm(int nt) { return nt == 1 ? 4 : nt == 2 ? 3 : 2; }

__host__ __device__ constexpr int sf_bytes(int fmt) { return fmt == 0 ? 4 : 8; }
__host__ __device__ constexpr int stage_bytes(int fmt) { return kStep * 64 * 2 + kStep * sf_bytes(fmt) * 2; }

// A warp's result of an item passes through the third stage of its ring, eight rows
// at a time: row r, 16-byte quad q at r * 512 + (q ^ (r / 2)) * 16 bytes, so that the
// stores of a quad's rows and two neighbours' channels fall on different banks; then
// m and l of all rows.  The first two stages receive the next item meanwhile.
__host__ __device__ constexpr int last_stage(int fmt) { return (kStages - 1) * stage_bytes(fmt); }
static_assert(8 * 512 + 8 * kMaxNt * 8 <= stage_bytes(0), "a stage holds eight rows, and m and l");
// Q's fragments of one tile of eight rows live in registers (staged through warp 0's
// third stage at the start of an item), those of more tiles in shared memory.  With
// the row scales that is 55,328 bytes for NVFP4 and NT = 1, of which four fit an SM.
__host__ __device__ constexpr int ring_bytes(int fmt) { return kWarps * kStages * stage_bytes(fmt); }
__host__ __device__ constexpr int smem_bytes(int fmt, int nt) {
  return ring_bytes(fmt) + (nt > 1 ? nt * 8 * 128 * 2 : 0) + nt * 8 * 4;
}

// Workspace: per CTA of the grid a header and two partial records.
struct Header {
  int r, rb, h;   // the item that begins in this CTA's run and ends behind it
  int parts;      // number of further CTAs that hold a part of it; 0: none
};
template <int NT>
struct Partial {
  float o[8 * NT][128];
  float m[8 * NT], l[8 * NT];
};
__host__ __device__ inline size_t header_bytes(int ctas) { return (size_t(ctas) * sizeof(Header) + 255) & ~size_t(255); }

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_sf(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}

// Key (0..7) held by row n of an 8-key score tile.  The swap of the pairs 2, 3 and
// 6, 7 puts the four lanes of a quad on keys of both parities, so that their
// 8-byte loads of V (64-byte rows, chunks swizzled by bit 2 of the key) cover all banks.
__device__ __forceinline__ int key_of(int n) { return n ^ ((n >> 1) & 1); }

struct Request {
  int q0, n;      // first query token and their number
  int kv;         // keys
  // kWindow, kTail: keys lo .. hi - 1 are in no row's sight; the tiles that hold nothing else,
  // `jump` keys of them from key `at` on, are left out of the line.  kTail, where prefixes are not
  // shared after all: hi = 0, and keys before lo are those of the group's first request
  int lo, hi, at, jump;
};
// Keys lo .. hi - 1 hidden from every row of a request.
__device__ __forceinline__ void hide(Request& x, int lo, int hi) {
  x.lo = lo, x.hi = hi;
  x.at = (lo + kTile - 1) / kTile * kTile;
  x.jump = max(0, hi / kTile * kTile - x.at);
}
template <int KIND>
__device__ __forceinline__ Request request_of(const KvAttnArgs& a, int r) {
  Request x;
  x.lo = x.hi = x.at = x.jump = 0;
  if constexpr (KIND == kPrefix) {  // checked by kv_shared_plan_kernel, whose result is 0 for a group that is none
    x.kv = __ldg(a.prefix + r);
    x.q0 = x.n = 0;
    if (x.kv <= 0) return x;
    x.q0 = __ldg(a.cu_q + __ldg(a.starts + r));
    const int n = __ldg(a.cu_q + __ldg(a.starts + r + 1)) - x.q0;
    x.n = int64_t(n) * a.G <= a.split_rows ? n : 0;
    return x;
  }
  const int64_t b = __ldg(a.cu_q + r), e = __ldg(a.cu_q + r + 1);
  const int kv = __ldg(a.kv_lens + r);
  const int64_t most = int64_t(a.width) << a.c.page_shift;
  if (b < 0 || e < b || e > a.total_q || e - b > a.max_q || kv < 0 || kv > most) {
    atomicOr(&g_status_kv_attn, DEV_BAD_INDEX);  // nothing of this request is computed
    x.q0 = x.n = x.kv = 0;
    return x;
  }
  x.q0 = int(b);
  x.n = (e - b) * a.G <= a.split_rows ? int(e - b) : 0;
  x.kv = kv;
  if constexpr (KIND == kWindow) {
    const int lo = int(max(int64_t(0), int64_t(kv) - (e - b) - a.window + 1));  // of the first token
    hide(x, min(a.sinks, lo), lo);
  }
  if constexpr (KIND == kTail) {
    const int p = __ldg(a.prefix + r);  // negative: of a group that is none
    if (p > 0 && e > b && kv - (e - b) < p) atomicOr(&g_status_kv_attn, DEV_BAD_INDEX);
    if (p < 0 || kv - (e - b) < p) x.n = 0;
    if (x.n > 0) {
      if (__ldg(a.share)) hide(x, 0, p);
      else x.lo = p;
    }
  }
  return x;
}
// Row of the block table whose keys the call's request r reads.
template <int KIND>
__device__ __forceinline__ int table_row(const KvAttnArgs& a, int r) {
  return KIND == kPrefix ? __ldg(a.starts + r) : r;
}
__device__ __forceinline__ int tiles_of(const Request& x) { return max(1, (x.kv - x.jump + kTile - 1) / kTile); }

// N = 4 or 8 channels from c of a finished row: `row` = token * Hq + head; m, l, o of its keys.  A record stays as
// it is, for kv_shared_join_kernel.
template <int KIND, int N>
__device__ __forceinline__ void finish(const KvAttnArgs& a, int64_t token, int head, int c, float m, float l, const float (&o)[N], float vst,
                                       bool record) {
  const int64_t row = token * a.Hq + head;
  if (kRecords<KIND> && record) {
    float4* dst = reinterpret_cast<float4*>(a.rows_o + row * 128 + c);
#pragma unroll
    for (int i = 0; i < N / 4; i++) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    if (c == 0) a.rows_ml[row] = make_float2(m, l);
    return;
  }
  const float f = l == 0.0f ? 1.0f : vst / l;
  uint32_t p[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; i++) p[i] = pack_bf16(o[2 * i] * f, o[2 * i + 1] * f);
  uint16_t* dst = a.o + row * 128 + c;
  if constexpr (N == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(p[0], p[1], p[2], p[3]);
  else *reinterpret_cast<uint2*>(dst) = make_uint2(p[0], p[1]);
  if (c == 0) a.lse[int64_t(head) * a.total_q + token] = l == 0.0f ? -INFINITY : (m - kOffset + log2f(l)) * 0.6931471805599453f;
}

// Units of work (tiles, and kItemTiles for each item) of request r.
template <int KIND, int ROWS>
__device__ __forceinline__ int64_t request_units(const KvAttnArgs& a, int r) {
  const Request x = request_of<KIND>(a, r);
  if (x.n == 0) return 0;
  return int64_t((x.n * a.G + ROWS - 1) / ROWS) * a.c.H * (tiles_of(x) + kItemTiles);
}

// Inclusive scan of `v` over the CTA; `total` gets the sum.
__device__ __forceinline__ int64_t cta_scan(int64_t v, int64_t* warp_sums, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; w++) {
    if (w < warp) v += warp_sums[w];
    total += warp_sums[w];
  }
  return v;
}

// One warp's softmax state and work on its keys of an item.  Lane (c, g) = (lane % 4,
// lane / 4) holds query rows 8 t + 2 c, + 1 and of them channels 16 g .. 16 g + 15.
template <int KIND, int FMT, int NT>
struct Worker {
  static constexpr int kSf = sf_bytes(FMT);
  uint32_t ring;        // this warp's stages
  int lane, c, g;
  float acc[NT][8][4];  // [.][j]: channels 16 g + 2 j (rows 2c, 2c + 1), 16 g + 2 j + 1 (the same)
  float m[NT][2], l[NT][2];
  uint4 qf[NT == 1 ? 4 : 1];  // Q's fragments of one tile

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < NT; t++) {
#pragma unroll
      for (int j = 0; j < 8; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) acc[t][j][e] = 0.0f;
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.0f;
    }
  }

  // Copies: two lanes per key and pass, a 32-byte sector at a time; pass i brings key
  // 16 i + lane / 2 of a step.  A warp's steps lie kTile keys apart, a multiple of every
  // page size, so a lane's rows within the pages stay the same for all steps of an
  // item, and an address is the lane's base plus block times the bytes of a block; from
  // pages of 32 rows on both passes are in one block, 16 rows apart.  Chunks of 16
  // bytes are swizzled by bit 2 of the key (see key_of).
  const uint8_t *k_src, *sf_src;  // of pass 0; lane % 2 brings the scales of K or of V
  int64_t v_from_k;
  uint32_t to0, to1, to_sf;       // in the stage, of pass 0
  uint32_t block_bytes;
  __device__ __forceinline__ void aim(const KvPages& p, int key0, int h) {
    const int half = lane & 1, key = lane >> 1, swz = ((key >> 2) & 1) << 1;
    to0 = ring + key * 64 + ((half ^ swz) << 4);
    to1 = ring + key * 64 + (((2 + half) ^ swz) << 4);
    to_sf = ring + kStep * 128 + (half * kStep + key) * kSf;
    block_bytes = uint32_t(p.H * p.page * 64);
    v_from_k = p.v - p.k;
    const int row = h * p.page + ((key0 + key) & (p.page - 1));
    k_src = p.k + row * 64 + half * 16;
    sf_src = (half ? p.v_sf : p.k_sf) + row * kSf;
  }
  __device__ __forceinline__ void copy_pass(uint32_t s, const uint8_t* k, const uint8_t* v, const uint8_t* sf, int i, int rows) {
    cp16(to0 + s + i * 1024, k + rows * 64);
    cp16(to1 + s + i * 1024, k + rows * 64 + 32);
    cp16(to0 + s + i * 1024 + kStep * 64, v + rows * 64);
    cp16(to1 + s + i * 1024 + kStep * 64, v + rows * 64 + 32);
    cp_sf<kSf>(to_sf + s + i * 16 * kSf, sf + rows * kSf);
  }
  // `b0`, `b1`: blocks of the two passes, within the cache (any block for rows that do not count)
  __device__ __forceinline__ void copy(int stage, bool small_pages, uint32_t b0, uint32_t b1) {
    const uint32_t s = stage * stage_bytes(FMT);
    const uint8_t* k = k_src + uint64_t(b0) * block_bytes;
    const uint8_t* sf = sf_src + uint64_t(b0) * (block_bytes / (64 / kSf));
    copy_pass(s, k, k + v_from_k, sf, 0, 0);
    if (KIND == kTail) {  // a prefix may end between the passes
      k = k_src + uint64_t(b1) * block_bytes;
      sf = sf_src + uint64_t(b1) * (block_bytes / (64 / kSf));
      copy_pass(s, k, k + v_from_k, sf, 1, small_pages ? 0 : 16);
    } else if (small_pages) {
      k = k_src + uint64_t(b1) * block_bytes;
      sf = sf_src + uint64_t(b1) * (block_bytes / (64 / kSf));
      copy_pass(s, k, k + v_from_k, sf, 1, 0);
    } else {
      copy_pass(s, k, k + v_from_k, sf, 1, 16);
    }
  }

  // Scores, softmax and P V of the 32 keys in `stage`.  MASKED: `seen` has a bit per key
  // of the step, and the row counts keys before limit[t][i], the first here being key0; of
  // these with a window the sinks and the last `window`.
  int window, sinks;
  __device__ __forceinline__ bool sees(int key, int limit) const {
    return key < limit && (KIND != kWindow || key >= limit - window || key < sinks);
  }
  template <bool MASKED>
  __device__ __forceinline__ void compute(int stage, uint32_t qs, const float (&cs)[NT][2], uint32_t seen,
                                          const int (&limit)[NT][2], int key0) {
    const uint32_t s = ring + stage * stage_bytes(FMT);
    const uint32_t sfk = s + kStep * 128, sfv = sfk + kStep * kSf;
    const int kg = key_of(g);
    float sc[NT][2][4];
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int u = 0; u < 2; u++)
#pragma unroll
        for (int e = 0; e < 4; e++) sc[t][u][e] = 0.0f;
    // V: a NaN block (scale byte 0xFF or 0x7F) reaches every row through 0 x NaN, so
    // where rows see different keys it is taken out of the product and put into the
    // rows that see its key; so are rows that are no keys and may hold anything.  Its
    // words are read ahead of K's products (drafted tokens 109 -> 108 us).
    const uint32_t vrow = ((((g >> 1) ^ (((c >> 1) & 1) << 1)) << 4) + ((g & 1) << 3));
    const int ka = key_of(2 * c), kb = key_of(2 * c + 1);
    uint2 va[2][2], vb[2][2];
    uint32_t bs[2][2];
#pragma unroll
    for (int u = 0; u < 2; u++) {
#pragma unroll
      for (int x = 0; x < 2; x++) {
        const int key = (2 * u + x) * 8;
        va[u][x] = lds8(s + kStep * 64 + (key + ka) * 64 + vrow);
        vb[u][x] = lds8(s + kStep * 64 + (key + kb) * 64 + vrow);
        uint32_t b0, b1;
        if (FMT == 0) {
          b0 = lds_u8(sfv + (key + ka) * 4 + (g >> 1));
          b1 = lds_u8(sfv + (key + kb) * 4 + (g >> 1));
          if (MASKED) {
            if (b0 == 0xFFu || !((seen >> (key + ka)) & 1u)) b0 = 0;
            if (b1 == 0xFFu || !((seen >> (key + kb)) & 1u)) b1 = 0;
          }
          bs[u][x] = e8m0_pair(b0, b1);
        } else {
          b0 = lds_u8(sfv + (key + ka) * 8 + g);
          b1 = lds_u8(sfv + (key + kb) * 8 + g);
          if (MASKED) {
            if ((b0 & 0x7Fu) == 0x7Fu || !((seen >> (key + ka)) & 1u)) b0 = 0;
            if ((b1 & 0x7Fu) == 0x7Fu || !((seen >> (key + kb)) & 1u)) b1 = 0;
          }
          bs[u][x] = e4m3_pair(b0 | (b1 << 8));
        }
      }
    }
    {
      uint32_t kw[2][2][4], ks[2][2][2];  // [16 keys][first or second eight][word or scale]
#pragma unroll
      for (int u = 0; u < 2; u++)
#pragma unroll
        for (int x = 0; x < 2; x++) {
          const int key = u * 16 + x * 8 + kg;
          const uint4 w = lds16(s + key * 64 + ((c ^ (((kg >> 2) & 1) << 1)) << 4));
          kw[u][x][0] = w.x, kw[u][x][1] = w.y, kw[u][x][2] = w.z, kw[u][x][3] = w.w;
          if (FMT == 0) {
            const uint32_t b = lds_u8(sfk + key * 4 + c);
            ks[u][x][0] = ks[u][x][1] = e8m0_pair(b, b);
          } else {
            const uint32_t b = e4m3_pair(lds_u16(sfk + key * 8 + 2 * c));
            ks[u][x][0] = __byte_perm(b, b, 0x1010);
            ks[u][x][1] = __byte_perm(b, b, 0x3232);
          }
        }
#pragma unroll
      for (int w = 0; w < 4; w++) {
        uint4 q[NT];
#pragma unroll
        for (int t = 0; t < NT; t++) q[t] = NT == 1 ? qf[NT == 1 ? w : 0] : lds16(qs + ((t * 4 + w) * 32 + lane) * 16);
#pragma unroll
        for (int u = 0; u < 2; u++) {
          uint32_t h0[4], h1[4];
          e2m1x8_to_f16(kw[u][0][w], h0);
          e2m1x8_to_f16(kw[u][1][w], h1);
#pragma unroll
          for (int i = 0; i < 4; i++) {
            h0[i] = hmul2(h0[i], ks[u][0][w >> 1]);
            h1[i] = hmul2(h1[i], ks[u][1][w >> 1]);
          }
          const uint32_t a0[4] = {h0[0], h1[0], h0[1], h1[1]}, a1[4] = {h0[2], h1[2], h0[3], h1[3]};
#pragma unroll
          for (int t = 0; t < NT; t++) {
            mma_f16(sc[t][u], a0, q[t].x, q[t].y);
            mma_f16(sc[t][u], a1, q[t].z, q[t].w);
          }
        }
      }
    }
    if (MASKED) {
#pragma unroll
      for (int u = 0; u < 2; u++)
#pragma unroll
        for (int x = 0; x < 2; x++) {
          const int key = u * 16 + x * 8 + kg;
          const bool there = (seen >> key) & 1u;
#pragma unroll
          for (int t = 0; t < NT; t++)
#pragma unroll
            for (int i = 0; i < 2; i++)
              if (!there || !sees(key0 + key, limit[t][i])) sc[t][u][2 * x + i] = -INFINITY;
        }
    }
    // a row's maximum moves only where a score passes it by more than kLazy (and
    // from -inf on), so its lanes are joined only then
    bool grow = false;
    float top[NT][2];
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int i = 0; i < 2; i++) {
        top[t][i] = fmaxf(fmax3(sc[t][0][i], sc[t][0][2 + i], sc[t][1][i]), sc[t][1][2 + i]) * cs[t][i];
        grow |= top[t][i] > m[t][i] + kLazy;
      }
    if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
      for (int t = 0; t < NT; t++)
#pragma unroll
        for (int i = 0; i < 2; i++) {
          float x = top[t][i];
#pragma unroll
          for (int o = 4; o <= 16; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
          if (x > m[t][i] + kLazy) {
            const float f = m[t][i] == -INFINITY ? 0.0f : ex2(m[t][i] - x);
            m[t][i] = x;
            l[t][i] *= f;
#pragma unroll
            for (int j = 0; j < 8; j++) {
              acc[t][j][i] *= f;
              acc[t][j][2 + i] *= f;
            }
          }
        }
    }
    uint32_t pf[NT][2][2];  // P^T fragments: [16 keys][first or second eight]
#pragma unroll
    for (int t = 0; t < NT; t++) {
      const float off0 = m[t][0] == -INFINITY ? 0.0f : kOffset - m[t][0];
      const float off1 = m[t][1] == -INFINITY ? 0.0f : kOffset - m[t][1];
#pragma unroll
      for (int u = 0; u < 2; u++)
#pragma unroll
        for (int x = 0; x < 2; x++) {
          const float p0 = ex2(fmaf(sc[t][u][2 * x], cs[t][0], off0));
          const float p1 = ex2(fmaf(sc[t][u][2 * x + 1], cs[t][1], off1));
          l[t][0] += p0;
          l[t][1] += p1;
          pf[t][u][x] = transpose8x8(pack_f16(p0, p1));
        }
    }
#pragma unroll
    for (int u = 0; u < 2; u++) {
#pragma unroll
      for (int w = 0; w < 2; w++) {
        uint32_t e0[4], o0[4], e1[4], o1[4];  // even and odd channels of the first and second eight keys
        {
          const uint32_t x = w ? va[u][0].y : va[u][0].x, y = w ? vb[u][0].y : vb[u][0].x;
          e2m1x8_to_f16((x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u), e0);
          e2m1x8_to_f16(((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), o0);
        }
        {
          const uint32_t x = w ? va[u][1].y : va[u][1].x, y = w ? vb[u][1].y : vb[u][1].x;
          e2m1x8_to_f16((x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u), e1);
          e2m1x8_to_f16(((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), o1);
        }
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const uint32_t a[4] = {hmul2(e0[j], bs[u][0]), hmul2(o0[j], bs[u][0]), hmul2(e1[j], bs[u][1]), hmul2(o1[j], bs[u][1])};
#pragma unroll
          for (int t = 0; t < NT; t++) mma_f16(acc[t][w * 4 + j], a, pf[t][u][0], pf[t][u][1]);
        }
      }
    }
    if (MASKED) {
      const float nan = __uint_as_float(0x7FC00000u);
      bool any;  // a NaN block in the row of this lane's key
      if (FMT == 0) {
        const uint32_t b = lds_u32(sfv + lane * 4);
        any = __vcmpeq4(b, 0xFFFFFFFFu) != 0;
      } else {
        const uint2 b = lds8(sfv + lane * 8);
        any = (__vcmpeq4(b.x & 0x7F7F7F7Fu, 0x7F7F7F7Fu) | __vcmpeq4(b.y & 0x7F7F7F7Fu, 0x7F7F7F7Fu)) != 0;
      }
      if (!__any_sync(0xFFFFFFFFu, any && ((seen >> lane) & 1u))) return;
#pragma unroll 1
      for (int key = 0; key < kStep; key++) {
        bool bad;  // in channels 16 g .. + 15
        if (FMT == 0) bad = lds_u8(sfv + key * 4 + (g >> 1)) == 0xFFu;
        else bad = (lds_u8(sfv + key * 8 + g) & 0x7Fu) == 0x7Fu;
        if (!bad || !((seen >> key) & 1u)) continue;
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
          for (int i = 0; i < 2; i++)
            if (sees(key0 + key, limit[t][i])) {
#pragma unroll
              for (int j = 0; j < 8; j++) acc[t][j][i] = acc[t][j][2 + i] = nan;
            }
      }
    }
  }
};

// Part of an item that a CTA computes: tiles t0 .. t0 + nt - 1 of the `tiles` of
// (request r, query rows row0 .. row0 + rows - 1 of it, key head h).
struct Item {
  int r, rb, h, t0, nt, tiles;
  int q0, row0, rows;
  int n, kv;
  int lo, hi, at, jump;  // as in Request
  int64_t last_unit;  // of the item, on the line
};

template <int KIND, int FMT, int NT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(NT)) kv_attn_kernel(KvAttnArgs a) {
  constexpr int ROWS = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t s_scan[kWarps];
  __shared__ int64_t s_before;
  __shared__ int s_r;
  float* s_cs = reinterpret_cast<float*>(smem + ring_bytes(FMT));
  uint8_t* s_q = NT > 1 ? smem + ring_bytes(FMT) + ROWS * 4 : smem + last_stage(FMT);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (kRecords<KIND> && !a.late) asm volatile("griddepcontrol.wait;" ::: "memory");  // for the prefixes' checks
  asm volatile("griddepcontrol.launch_dependents;");  // kv_join_kernel may take its place and wait
  // `late`: nothing is read of the kernel before this one, but its end is this one's, too.  One CTA waits for
  // it; the others make room.
  auto leave = [&] {
    if (kRecords<KIND> && a.late && blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  };
  Header* headers = reinterpret_cast<Header*>(a.ws);
  Partial<NT>* partials = reinterpret_cast<Partial<NT>*>(a.ws + header_bytes(gridDim.x));

  // the line of units and this CTA's run of it; or, where all contexts are short,
  // whole items one after another
  int64_t total = 0, pos = 0, end = 0, base = 0, run = 0, extra = 0;
  int r = 0;
  if (a.whole) {
    end = int64_t(a.R) * a.c.H;
    pos = blockIdx.x;
  } else {
    if (!kRecords<KIND> && tid == 0) headers[blockIdx.x].parts = 0;
    int64_t first_own = 0, first_upto = 0;  // of the first kThreads requests, the only ones most often
    for (int r0 = 0; r0 < a.R; r0 += kThreads) {
      int64_t sum;
      const int64_t own = r0 + tid < a.R ? request_units<KIND, ROWS>(a, r0 + tid) : 0;
      const int64_t upto = cta_scan(own, s_scan, sum);
      if (r0 == 0) {
        first_own = own;
        first_upto = upto;
      }
      total += sum;
    }
    const int64_t most = (total + kMinTiles - 1) / kMinTiles;
    const int64_t C = most < int64_t(gridDim.x) ? most : int64_t(gridDim.x);
    if (int64_t(blockIdx.x) >= C) {
      leave();
      return;
    }
    run = total / C, extra = total - run * C;  // the first `extra` CTAs take one unit more
    pos = run * blockIdx.x + min(extra, int64_t(blockIdx.x));
    end = pos + run + (int64_t(blockIdx.x) < extra ? 1 : 0);
    int64_t before = 0;
    for (int r0 = 0; r0 < a.R; r0 += kThreads) {
      int64_t sum = total, own = first_own, upto = first_upto;
      if (a.R > kThreads) {
        own = r0 + tid < a.R ? request_units<KIND, ROWS>(a, r0 + tid) : 0;
        upto = before + cta_scan(own, s_scan, sum);
      }
      if (upto - own <= pos && pos < upto) {
        s_r = r0 + tid;
        s_before = upto - own;
      }
      before += sum;
      if (pos < before) break;
    }
    __syncthreads();
    r = s_r;
    base = s_before;
  }

  // the next part of an item of this CTA, if there is one
  auto next = [&](Item& it) -> bool {
    while (pos < end && r < a.R) {
      if (a.whole) r = int(pos / a.c.H);
      const Request x = request_of<KIND>(a, r);
      it.tiles = tiles_of(x);
      it.q0 = x.q0, it.n = x.n, it.kv = x.kv;
      it.lo = x.lo, it.hi = x.hi, it.at = x.at, it.jump = x.jump;
      if (a.whole) {
        it.rb = 0, it.h = int(pos - int64_t(r) * a.c.H);
        it.t0 = 0, it.nt = x.n == 0 ? 0 : it.tiles;
        it.last_unit = 0;
        pos += gridDim.x;
      } else {
        const int nrb = (x.n * a.G + ROWS - 1) / ROWS, units = it.tiles + kItemTiles;
        const int64_t all = x.n == 0 ? 0 : int64_t(nrb) * a.c.H * units;
        if (pos >= base + all) {
          base += all;
          r++;
          continue;
        }
        const int64_t local = pos - base;
        const int item = local >> 32 ? int(local / units) : int(uint32_t(local) / uint32_t(units));
        const int u0 = int(local - int64_t(item) * units), u1 = int(min(int64_t(units), u0 + (end - pos)));
        it.rb = item / a.c.H, it.h = item - it.rb * a.c.H;
        it.t0 = max(0, u0 - kItemTiles);  // the first units of an item stand for its cost as such
        it.nt = max(0, u1 - kItemTiles) - it.t0;
        it.last_unit = base + int64_t(item + 1) * units - 1;
        pos += u1 - u0;
      }
      if (it.nt == 0) continue;
      it.r = r;
      it.row0 = it.rb * ROWS;
      it.rows = min(ROWS, x.n * a.G - it.row0);
      return true;
    }
    return false;
  };

  Worker<KIND, FMT, NT> wk;
  wk.window = a.window, wk.sinks = a.sinks;
  wk.ring = smem_u32(smem) + warp * kStages * stage_bytes(FMT);
  wk.lane = lane;
  wk.c = lane & 3;
  wk.g = lane >> 2;
  const float kst = FMT == 1 ? __ldg(a.c.k_scale) : 1.0f;
  const float vst = FMT == 1 ? __ldg(a.c.v_scale) : 1.0f;
  float* const mine = reinterpret_cast<float*>(smem + warp * kStages * stage_bytes(FMT) + last_stage(FMT));
  const bool small_pages = a.c.page == 16;
  const uint32_t last_block = uint32_t(a.c.blocks) - 1u;

  // copies of the current item: the blocks of the lane's two keys of a step, looked
  // up one step ahead
  int k_lo, k_end, steps;  // kWindow, kTail: places on the line, which leaves `jump` keys out at `jump_at`
  int jump_at = 0, jump = 0, hide_lo = 0, hide_hi = 0;
  constexpr bool kHides = KIND == kWindow || KIND == kTail;
  auto key_at = [&](int place) { return kHides && place >= jump_at ? place + jump : place; };
  auto in_sight = [&](int place) {
    if (!kHides) return place < k_end;
    const int key = key_at(place);
    return place < k_end && (key < hide_lo || key >= hide_hi);
  };
  const int32_t *table, *first_table = nullptr;  // kTail, prefixes not shared: of keys before hide_lo
  uint32_t b0 = 0, b1 = 0;
  auto look_up = [&](int step, uint32_t& b0, uint32_t& b1) {
    const int place = k_lo + (lane >> 1) + step * kTile, key = key_at(place);
    const bool second = in_sight(place + 16);
    if (KIND == kTail && first_table) {
      auto block = [&](int k) { return uint32_t(__ldg((k < hide_lo ? first_table : table) + (k >> a.c.page_shift))); };
      b0 = in_sight(place) ? block(key) : 0xFFFFFFFFu;
      b1 = second ? block(key + 16) : 0xFFFFFFFFu;
      return;
    }
    // where keys are hidden, a block of both passes may have only the second one's key in sight
    const bool first = in_sight(place) || (kHides && !small_pages && second);
    b0 = first ? uint32_t(__ldg(table + (key >> a.c.page_shift))) : 0xFFFFFFFFu;
    if (small_pages) b1 = second ? uint32_t(__ldg(table + (key >> 4) + 1)) : 0xFFFFFFFFu;
    else b1 = second ? b0 : 0xFFFFFFFFu;
  };
  // starts the copies of a step and returns a bit per visible key; rows that are none
  // (past the last key, or of a block outside the cache) bring some other row, unseen
  auto issue = [&](int step, int st) -> uint32_t {
    const int place = k_lo + (lane >> 1) + step * kTile;
    const bool live0 = b0 <= last_block && (!kHides || in_sight(place)), live1 = b1 <= last_block;
    wk.copy(st, small_pages, min(b0, last_block), min(b1, last_block));
    cp_commit();
    uint32_t seen = 0xFFFFFFFFu;
    if (!__all_sync(0xFFFFFFFFu, live0 && live1)) {
      // lanes 2k and 2k + 1 speak for keys k and 16 + k
      const uint32_t v0 = __ballot_sync(0xFFFFFFFFu, live0), v1 = __ballot_sync(0xFFFFFFFFu, live1);
      seen = __ballot_sync(0xFFFFFFFFu, ((lane < 16 ? v0 : v1) >> (2 * (lane & 15))) & 1u);
      if ((!live0 && in_sight(place)) || (!live1 && in_sight(place + 16))) atomicOr(&g_status_kv_attn, DEV_BAD_INDEX);
    }
    return seen;
  };
  static_assert(kStages == 3, "two steps in flight ahead of the one computed");
  uint32_t seen0 = 0, seen1 = 0;
  uint4 qv[NT > 2 ? 4 : 2];  // this thread's channels of the item's queries
  constexpr int kPasses = (ROWS * 8 + kThreads - 1) / kThreads;
  // starts an item: its first two steps, and its queries' loads
  auto begin = [&](const Item& it) {
    const int last_tok = (it.row0 + it.rows - 1) / a.G;
    const int keys = a.causal ? max(0, it.kv - it.n + last_tok + 1) : it.kv;  // that some row sees
    k_lo = it.t0 * kTile + warp * kStep;
    if (kHides) {
      jump_at = it.at, jump = it.jump, hide_lo = it.lo, hide_hi = it.hi;
      k_end = min((it.t0 + it.nt) * kTile, keys - jump);  // the last key is behind the hidden ones
    } else {
      k_end = min((it.t0 + it.nt) * kTile, keys);
    }
    steps = k_lo < k_end ? (k_end - k_lo + kTile - 1) / kTile : 0;
    table = a.table + int64_t(table_row<KIND>(a, it.r)) * a.width;
    if (KIND == kTail) first_table = it.hi < it.lo ? a.table + int64_t(__ldg(a.starts + it.r)) * a.width : nullptr;
    wk.aim(a.c, k_lo, it.h);
    // the first three steps' blocks at once, or each would be waited for
    uint32_t e0[3], e1[3];
#pragma unroll
    for (int s = 0; s < 3; s++) look_up(s, e0[s], e1[s]);
#pragma unroll
    for (int s = 0; s < 2; s++) {
      b0 = e0[s], b1 = e1[s];
      if (s < steps) (s == 0 ? seen0 : seen1) = issue(s, s);
      else cp_commit();
    }
    b0 = e0[2], b1 = e1[2];
    // eight threads per row, 16 channels each
#pragma unroll
    for (int pass = 0; pass < kPasses; pass++) {
      const int row = (pass * kThreads + tid) >> 3, part = tid & 7;
      qv[2 * pass] = qv[2 * pass + 1] = make_uint4(0, 0, 0, 0);
      if (row < it.rows) {
        const int rr = it.row0 + row, tok = rr / a.G, hd = rr - tok * a.G;
        const uint16_t* src = a.q + int64_t(it.q0 + tok) * a.q_stride + int64_t(it.h * a.G + hd) * 128 + part * 16;
        qv[2 * pass] = __ldg(reinterpret_cast<const uint4*>(src));
        qv[2 * pass + 1] = __ldg(reinterpret_cast<const uint4*>(src) + 1);
      }
    }
  };

  // further CTAs that hold a part of an item that begins here
  auto parts_behind = [&](const Item& x) {
    const int64_t larger = extra * (run + 1);  // units of the CTAs that take one more
    return int(x.last_unit < larger ? x.last_unit / (run + 1) : extra + (x.last_unit - larger) / run) - int(blockIdx.x);
  };

  Item it;
  if (!next(it)) {
    leave();
    return;
  }
  begin(it);
  for (bool more = true; more;) {
    // Q: binary16 with a power of two per row, in fragment order
#pragma unroll
    for (int pass = 0; pass < kPasses; pass++) {
      const int row = (pass * kThreads + tid) >> 3, part = tid & 7;
      const uint4 v0 = qv[2 * pass], v1 = qv[2 * pass + 1];
      const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
      uint32_t mx = 0;
#pragma unroll
      for (int e = 0; e < 8; e++) mx = max(mx, hmax2(abs2(w[e])));
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
      const float2 sc = q_row_scale(mx);
      const float f = sc.x, inv = sc.y;
      // channels 16 part + 0..15 belong to lane column c = part / 2, contraction steps
      // 4 (part % 2) .. + 3, four channels a step (b0, b1); a 16-byte word of lane
      // (c, row % 8) holds two steps
      if (row < ROWS) {
        uint4* dst = reinterpret_cast<uint4*>(s_q) + ((row >> 3) * 4 + (part & 1) * 2) * 32 + (row & 7) * 4 + (part >> 1);
#pragma unroll
        for (int st = 0; st < 2; st++)
          dst[st * 32] = make_uint4(pack_f16(bf_lo(w[4 * st]) * f, bf_hi(w[4 * st]) * f),
                                    pack_f16(bf_lo(w[4 * st + 1]) * f, bf_hi(w[4 * st + 1]) * f),
                                    pack_f16(bf_lo(w[4 * st + 2]) * f, bf_hi(w[4 * st + 2]) * f),
                                    pack_f16(bf_lo(w[4 * st + 3]) * f, bf_hi(w[4 * st + 3]) * f));
        // never 0: the score of a hidden key, -inf, is multiplied by it
        if (part == 0) s_cs[row] = fmaxf(a.scale_log2 * kst * inv, 1.17549435e-38f);
      }
    }
    __syncthreads();
    float cs[NT][2];
    int lim[NT][2];
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const int row = t * 8 + 2 * wk.c + i;
        cs[t][i] = s_cs[row];
        lim[t][i] = !a.causal || row >= it.rows ? it.kv : it.kv - it.n + (it.row0 + row) / a.G + 1;
        if (KIND == kWindow) lim[t][i] = max(lim[t][i], 0);
      }
    const int all_see = a.causal ? it.kv - it.n + it.row0 / a.G + 1 : it.kv;  // keys that every row sees
    // and with a window from here on
    const int all_from = KIND == kWindow ? max(0, it.kv - it.n + (it.row0 + it.rows - 1) / a.G + 1) - a.window : 0;
    wk.clear();
    const uint32_t qs = smem_u32(s_q);
    if (NT == 1) {
#pragma unroll
      for (int w = 0; w < 4; w++) wk.qf[NT == 1 ? w : 0] = lds16(qs + (w * 32 + lane) * 16);
      __syncthreads();  // the stage is free for copies
    }
    int stage = 0;  // every item begins with stage 0
#pragma unroll 1
    for (int step = 0; step < steps; step++) {
      // the stage of step - 1 is free: every lane has read it
      __syncwarp();
      uint32_t seen2 = 0;
      if (step + 2 < steps) {
        seen2 = issue(step + 2, stage == 0 ? 2 : stage - 1);
        look_up(step + 3, b0, b1);
      } else {
        cp_commit();
      }
      cp_wait<kStages - 1>();
      __syncwarp();
      const int key0 = key_at(k_lo + step * kTile);
      const bool behind = KIND == kWindow && key0 < all_from && key0 + kStep > a.sinks;
      if (kHides && seen0 == 0u) {
        // nothing: beside a few sinks, or before the window's first key
      } else if (seen0 != 0xFFFFFFFFu || key0 + kStep > all_see || behind) wk.template compute<true>(stage, qs, cs, seen0, lim, key0);
      else wk.template compute<false>(stage, qs, cs, seen0, lim, key0);
      seen0 = seen1;
      seen1 = seen2;
      stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    __syncwarp();
    // the next item's first copies run while this one's warps are joined
    const Item cur = it;
    more = next(it);
    if (more) begin(it);
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int i = 0; i < 2; i++) {
        float v = wk.l[t][i];
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        if (wk.g == 0) *reinterpret_cast<float2*>(mine + 1024 + (t * 8 + 2 * wk.c + i) * 2) = make_float2(wk.m[t][i], v);
      }
    const bool head_part = cur.t0 > 0, cut = cur.t0 + cur.nt < cur.tiles;
    // for the join: but not a request's whole rows without a prefix
    const bool record = KIND == kPrefix || (KIND == kTail && (cur.hi > 0 || cut || head_part));
    Partial<NT>* part = &partials[2 * blockIdx.x + (head_part ? 0 : 1)];
    const float* const theirs = reinterpret_cast<const float*>(smem + last_stage(FMT));  // of warp 0
    constexpr int kRing = kStages * stage_bytes(FMT) / 4;                                // floats from warp to warp
#pragma unroll
    for (int t = 0; t < NT; t++) {
      if (t > 0) __syncthreads();  // the previous eight rows are no longer read
#pragma unroll
      for (int i = 0; i < 2; i++) {
        float4* dst = reinterpret_cast<float4*>(mine) + (2 * wk.c + i) * 32;
#pragma unroll
        for (int j = 0; j < 8; j += 2)
          dst[(wk.g * 4 + (j >> 1)) ^ wk.c] =
              make_float4(wk.acc[t][j][i], wk.acc[t][j][2 + i], wk.acc[t][j + 1][i], wk.acc[t][j + 1][2 + i]);
      }
      __syncthreads();
      const int row = tid >> 4, quad = (tid & 15) * 2;  // eight channels a thread
      const int frow = t * 8 + row;
      float M = -INFINITY, L = 0.0f, w[kWarps];
      float2 ml[kWarps];
#pragma unroll
      for (int k = 0; k < kWarps; k++) {
        ml[k] = *reinterpret_cast<const float2*>(theirs + k * kRing + 1024 + frow * 2);
        M = fmaxf(M, ml[k].x);
      }
#pragma unroll
      for (int k = 0; k < kWarps; k++) {
        // without keys (m = -inf) l and O are 0, or NaN where every score was
        w[k] = ml[k].x == -INFINITY ? 1.0f : ex2(ml[k].x - M);
        L += w[k] * ml[k].y;
      }
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; j++) o[j] = 0.0f;
#pragma unroll
      for (int k = 0; k < kWarps; k++) {
        const float4* src = reinterpret_cast<const float4*>(theirs + k * kRing) + row * 32;
#pragma unroll
        for (int j = 0; j < 2; j++) {
          const float4 v = src[(quad + j) ^ (row >> 1)];
          o[4 * j] += w[k] * v.x;
          o[4 * j + 1] += w[k] * v.y;
          o[4 * j + 2] += w[k] * v.z;
          o[4 * j + 3] += w[k] * v.w;
        }
      }
      if (frow < cur.rows) {
        if (head_part || cut) {
          float4* dst = reinterpret_cast<float4*>(part->o[frow]) + quad;
          dst[0] = make_float4(o[0], o[1], o[2], o[3]);
          dst[1] = make_float4(o[4], o[5], o[6], o[7]);
          if (quad == 0) {
            part->m[frow] = M;
            part->l[frow] = L;
          }
        } else {
          const int rr = cur.row0 + frow, tok = rr / a.G, hd = cur.h * a.G + rr - tok * a.G;
          finish<KIND, 8>(a, cur.q0 + tok, hd, quad * 4, M, L, o, vst, record);
        }
        if (record && !head_part && quad == 0) {
          const int rr = cur.row0 + frow, tok = rr / a.G, hd = cur.h * a.G + rr - tok * a.G;
          a.places[int64_t(cur.q0 + tok) * a.Hq + hd] =
              make_uint2(blockIdx.x, kv_place(cut ? parts_behind(cur) + 1 : 0, frow, false, cur.hi > 0));
        }
      }
    }
    if (!kRecords<KIND> && cut && !head_part && tid == 0) {
      Header hd;
      hd.r = cur.r;
      hd.rb = cur.rb;
      hd.h = cur.h;
      hd.parts = parts_behind(cur);
      headers[blockIdx.x] = hd;
    }
    __syncthreads();  // the third stages and the row scales are free
  }
  leave();
}

// Joins the parts of the item that begins in CTA blockIdx.x's run and ends behind
// it.  Two warps per row, four channels a lane: one takes the first half of the parts and
// one the second, each in the order of the keys.
template <int KIND, int FMT, int NT>
__global__ void __launch_bounds__(256) kv_join_kernel(KvAttnArgs a, int ctas) {
  __shared__ float4 s_o[4][32];
  __shared__ float s_l[4];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for the end of kv_attn_kernel
  const Header hd = reinterpret_cast<const Header*>(a.ws)[blockIdx.x];
  if (hd.parts == 0) return;
  const Partial<NT>* partials = reinterpret_cast<const Partial<NT>*>(a.ws + header_bytes(ctas));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = warp >> 2;
  const int row = blockIdx.y * 4 + (warp & 3);
  const Request x = request_of<KIND>(a, hd.r);
  const int rr = hd.rb * 8 * NT + row;
  const bool live = rr < x.n * a.G;
  auto part = [&](int i) -> const Partial<NT>& { return partials[2 * (blockIdx.x + i) + (i == 0 ? 1 : 0)]; };
  const int count = live ? hd.parts + 1 : 0, mid = (count + 1) / 2;
  float M = -INFINITY;
  for (int i = lane; i < count; i += 32) M = fmaxf(M, part(i).m[row]);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
  float L = 0.0f;
  float4 s = make_float4(0, 0, 0, 0);
  const int last = half ? count : mid;
#pragma unroll 8
  for (int i = half ? mid : 0; i < last; i++) {
    const Partial<NT>& p = part(i);
    const float m = p.m[row];
    const float w = m == -INFINITY ? 1.0f : ex2(m - M);  // without keys l and O are 0, or NaN
    const float4 v = *reinterpret_cast<const float4*>(&p.o[row][lane * 4]);
    L += w * p.l[row];
    s.x += w * v.x;
    s.y += w * v.y;
    s.z += w * v.z;
    s.w += w * v.w;
  }
  if (half) {
    s_o[warp & 3][lane] = s;
    if (lane == 0) s_l[warp & 3] = L;
  }
  __syncthreads();
  if (half || !live) return;
  const float4 v = s_o[warp][lane];
  L += s_l[warp];
  const float vst = FMT == 1 ? __ldg(a.c.v_scale) : 1.0f;
  const int tok = rr / a.G, head = hd.h * a.G + rr - tok * a.G;
  float o[4] = {s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w};
  finish<KIND, 4>(a, x.q0 + tok, head, lane * 4, M, L, o, vst, false);
}

// Tiles of eight query rows in a block: as few blocks of at most 32 rows as there
// can be, of equal size (48 rows: two of 24; in their time 110 us for the drafted tokens
// above, where blocks of 32 took 132, as four tiles spill, and blocks of 16 took 125).
int row_tiles(int64_t rows) {
  const int64_t blocks = (rows + 8 * kMaxNt - 1) / (8 * kMaxNt);
  return int((rows + 8 * blocks - 1) / (8 * blocks));
}

template <int NT>
size_t workspace(int sms) {
  const int ctas = sms * ctas_per_sm(NT);
  return header_bytes(ctas) + size_t(ctas) * 2 * sizeof(Partial<NT>);
}

// `line_ws`: the prompts' workspace, whose line is made beside kv_attn_kernel; NULL: no prompts.
template <int KIND, int FMT, int NT>
cudaError_t launch(const KvAttnArgs& a, uint8_t* line_ws, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  constexpr int bytes = smem_bytes(FMT, NT);
  cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(kv_attn_kernel<KIND, FMT, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  });
  if (e != cudaSuccess) return e;
  const int ctas = sm_count_current_device() * ctas_per_sm(NT);
  if (ctas <= 0) return cudaErrorInvalidDevice;
  if (a.whole) {
    const int64_t items = int64_t(a.R) * a.c.H;
    const int64_t most = int64_t(ctas) * 16;
    const unsigned grid = unsigned(items < most ? items : most);
    if constexpr (kRecords<KIND>) return launch_early(kv_attn_kernel<KIND, FMT, NT>, dim3(grid), kThreads, bytes, st, a);
    kv_attn_kernel<KIND, FMT, NT><<<grid, kThreads, bytes, st>>>(a);
    return cudaGetLastError();
  }
  if constexpr (kRecords<KIND>) {
    if (a.late || !line_ws) return launch_early(kv_attn_kernel<KIND, FMT, NT>, dim3(unsigned(ctas)), kThreads, bytes, st, a);
  }
  kv_attn_kernel<KIND, FMT, NT><<<ctas, kThreads, bytes, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (line_ws && (e = launch_kv_prefill_line(KIND, a, line_ws, true, st)) != cudaSuccess) return e;
  if constexpr (kRecords<KIND>) return cudaSuccess;
  else return launch_early(kv_join_kernel<KIND, FMT, NT>, dim3(unsigned(ctas), 2 * NT), 256, 0, st, a, ctas);
}

template <int KIND, int FMT>
cudaError_t launch_fmt(const KvAttnArgs& a, int nt, uint8_t* line_ws, cudaStream_t st) {
  switch (nt) {
    case 1: return launch<KIND, FMT, 1>(a, line_ws, st);
    case 2: return launch<KIND, FMT, 2>(a, line_ws, st);
    case 3: return launch<KIND, FMT, 3>(a, line_ws, st);
    default: return launch<KIND, FMT, 4>(a, line_ws, st);
  }
}

cudaError_t launch_kind(int kind, const KvAttnArgs& a, int nt, uint8_t* line_ws, cudaStream_t st) {
  switch (kind * 2 + (a.c.fmt == 0 ? 0 : 1)) {
    case kAll * 2: return launch_fmt<kAll, 0>(a, nt, line_ws, st);
    case kAll * 2 + 1: return launch_fmt<kAll, 1>(a, nt, line_ws, st);
    case kWindow * 2: return launch_fmt<kWindow, 0>(a, nt, line_ws, st);
    case kWindow * 2 + 1: return launch_fmt<kWindow, 1>(a, nt, line_ws, st);
    case kPrefix * 2: return launch_fmt<kPrefix, 0>(a, nt, line_ws, st);
    case kPrefix * 2 + 1: return launch_fmt<kPrefix, 1>(a, nt, line_ws, st);
    case kTail * 2: return launch_fmt<kTail, 0>(a, nt, line_ws, st);
    default: return launch_fmt<kTail, 1>(a, nt, line_ws, st);
  }
}

size_t workspace_of(int nt) {
  const int sms = sm_count_current_device();
  switch (nt) {
    case 1: return workspace<1>(sms);
    case 2: return workspace<2>(sms);
    case 3: return workspace<3>(sms);
    default: return workspace<4>(sms);
  }
}

// Which kernels a call runs, by the most query rows (tokens x G) a request can have.
// Up to kFewRows: this file's alone, with tiles for that many rows.  Above: this
// file's for the requests of at most kMixedRows rows, with tiles for a single token
// (the decoding requests of a mixed batch), and kv_prefill.cu's for the others.
// Measured here / there, in us, with 8 key heads and MXFP4: 24 requests of 6000 keys
// with 24 rows each 70 / 114, 32 rows 85 / 115, 48 rows 123 / 116, 56 rows 153 / 116; 24
// to 48 rows over up to 12288 keys 111 / 118.  One prompt of 512 tokens with 48 requests
// of 4096 keys, these with 16 rows 195 / 232, 24 rows 237 / 232, 32 rows 281 / 233.
constexpr int kFewRows = 48, kMixedRows = 24;
struct Plan {
  int nt, split_rows;
  bool prefill;
  bool whole;  // one block of rows per request and no item worth cutting: no workspace
};
Plan plan_of(int max_q, int64_t max_k, int G) {
  const int64_t rows = int64_t(max_q < 1 ? 1 : max_q) * G;
  if (rows <= kFewRows) return Plan{row_tiles(rows), kFewRows, false, rows <= 8 * kMaxNt && max_k <= kWholeTiles * kTile};
  return Plan{row_tiles(G < kMixedRows ? G : kMixedRows), kMixedRows, true, false};
}

}  // namespace kva

// Whether a call's longest context is within what its kernels take: kv_prefill.cu's
// waits end after 2 s, and its longest one, for an item to pass, takes 2 us a tile of
// 128 keys: 0.6 s for 2^25 keys.
bool kv_attn_reaches(int max_q, int64_t max_k, int G) {
  return !kva::plan_of(max_q, max_k, G).prefill || max_k <= (int64_t(1) << 25);
}

// The most keys of a context that a row can see, and those its tiles hold beside them.
int64_t kv_window_reach(int max_q, int64_t max_k, int window, int sinks) {
  const int64_t tile = kva::kTile, sunk = (sinks + tile - 1) / tile * tile;
  const int64_t most = sunk + (int64_t(window) + max_q + 2 * tile - 3) / tile * tile;
  return most < max_k ? most : max_k;
}

size_t kv_attn_workspace(int R, int max_q, int64_t max_k, int G) {
  const kva::Plan p = kva::plan_of(max_q, max_k, G);
  if (p.whole) return 0;
  const size_t few = (kva::workspace_of(p.nt) + 255) & ~size_t(255);
  return p.prefill ? few + kv_prefill_workspace(R) : few;
}

bool kv_attn_few(int max_q, int64_t max_k, int G) { return !kva::plan_of(max_q, max_k, G).prefill; }

// The parts of a call's workspace: where the kernels of few and of many rows leave records.
KvRecords kv_attn_records(uint8_t* ws, int R, int max_q, int64_t max_k, int G) {
  const kva::Plan p = kva::plan_of(max_q, max_k, G);
  KvRecords x;
  x.many_ws = ws + ((kva::workspace_of(p.nt) + 255) & ~size_t(255));
  x.few = ws + kva::header_bytes(sm_count_current_device() * kva::ctas_per_sm(p.nt));
  x.few_rows = 8 * p.nt;
  x.split_rows = p.prefill ? p.split_rows : 1 << 30;
  x.many = p.prefill ? kv_prefill_records(x.many_ws, R) : nullptr;
  return x;
}

cudaError_t launch_kv_attn(int kind, const KvAttnArgs& args, cudaStream_t st) {
  clear_stale_error();
  KvAttnArgs a = args;
  // no request has more keys than a row of its table
  int64_t max_k = int64_t(a.width) << a.c.page_shift;
  if (kind == kWindow) max_k = kv_window_reach(a.max_q, max_k, a.window, a.sinks);
  const kva::Plan p = kva::plan_of(a.max_q, max_k, a.G);
  a.split_rows = p.split_rows;
  a.whole = p.whole;
  uint8_t* const line_ws = p.prefill ? kv_attn_records(a.ws, a.R, a.max_q, max_k, a.G).many_ws : nullptr;
  if (kind == kPrefix && p.prefill) {  // all groups, by the line that kv_shared_plan_kernel has made
    a.split_rows = 0;
    return launch_kv_prefill(kind, a, line_ws, st);
  }
  cudaError_t e;
  if (!p.prefill || a.G <= kva::kMixedRows) e = kva::launch_kind(kind, a, p.nt, line_ws, st);
  else e = launch_kv_prefill_line(kind, a, line_ws, false, st);
  return e != cudaSuccess || !p.prefill ? e : launch_kv_prefill(kind, a, line_ws, st);
}

unsigned read_status_kv_attn(cudaStream_t st) {
  unsigned v = 0, z = 0;
  cudaMemcpyFromSymbolAsync(&v, g_status_kv_attn, sizeof(v), 0, cudaMemcpyDeviceToHost, st);
  cudaMemcpyToSymbolAsync(g_status_kv_attn, &z, sizeof(z), 0, cudaMemcpyHostToDevice, st);
  cudaStreamSynchronize(st);
  return v;
}

}  // namespace mxfa
