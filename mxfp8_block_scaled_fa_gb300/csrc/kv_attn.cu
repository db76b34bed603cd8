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
// is rounded to binary16 (11 bits; relative 2^-12, against 2^-9 for the bf16
// result), where the offset 8 keeps weights down to 2^-32 of the largest from
// vanishing; m moves when a score exceeds it by more than 6, so P <= 2^14.
//
// Work.  The key tiles (128 keys) of all (request, key head, block of query
// rows) items form one line, cut into equal runs, one per CTA: no CTA has more
// than one tile above another whatever the lengths.  An item inside one run is
// finished there; one cut by a border leaves partial (m, l, O) records that a
// second kernel joins in the order of the keys, so results do not depend on
// timing.  Each of the CTA's four warps takes 32 of a tile's keys with its own
// ring of asynchronous copies and its own softmax state, so warps never wait on
// one another inside an item.
//
// Fragments.  m16n8k16 with the query rows as M.  The contraction order is free
// as long as both operands agree, so a lane's K fragments over all of D are
// the 32 consecutive channels (one 16-byte load, one MXFP4 block) of its key,
// and Q is laid out to match; its V fragments are 16 consecutive channels of
// four keys, two keys' codes merged into bytes before conversion so that the
// pair (key, key + 1) comes out of one conversion.
#include "mx_ptx.cuh"
#include "mxfa_internal.h"

namespace mxfa {

static __device__ unsigned g_status_kv_attn;

namespace kva {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 32;                 // keys of one warp step
constexpr int kTile = kStep * kWarps;     // keys of one CTA step
constexpr int kStages = 3;
constexpr float kOffset = 8.0f;           // log2 offset of P
constexpr float kLazy = 6.0f;             // growth of a row maximum that moves m
constexpr int kCtasPerSm = 3;
constexpr int kMinTiles = 4;              // least tiles of a run, as long as items are cut

__host__ __device__ constexpr int sf_bytes(int fmt) { return fmt == 0 ? 4 : 8; }
__host__ __device__ constexpr int stage_bytes(int fmt) { return kStep * 64 * 2 + kStep * sf_bytes(fmt) * 2; }

// Merge layout: row r, quarter c (32 channels) at r * 144 + c * 36 floats, so that
// the 128-bit stores of two rows' four lanes each fall on different banks.
constexpr int kMergeRow = 144;
__host__ __device__ constexpr int area_bytes(int fmt) {
  const int ring = kWarps * kStages * stage_bytes(fmt);
  const int merge = kWarps * 16 * kMergeRow * 4;
  return ring > merge ? ring : merge;
}
__host__ __device__ constexpr int smem_bytes(int fmt, int mt) {
  return area_bytes(fmt) + mt * 16 * 128 * 2 /* Q */ + kWarps * mt * 16 * 8 /* m, l */ + mt * 16 * 4 /* row scales */;
}

// Workspace: per CTA of the grid a header and two partial records.
struct Header {
  int r, rb, h;   // the item that begins in this CTA's run and ends behind it
  int parts;      // number of further CTAs that hold a part of it; 0: none
};
template <int MT>
struct Partial {
  float o[16 * MT][128];
  float m[16 * MT], l[16 * MT];
};
__host__ __device__ inline size_t header_bytes(int ctas) { return (size_t(ctas) * sizeof(Header) + 255) & ~size_t(255); }

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_sf(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(live ? N : 0) : "memory");
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
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t* h) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
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
// A pair of E8M0 bytes -> binary16 pair 2^(b - 127); 0xFF gives Inf, which times
// the code 0 it comes with is NaN; a zero-filled byte gives 0.
__device__ __forceinline__ uint32_t e8m0_pair(uint32_t lo, uint32_t hi) {
  return pack_f16(__uint_as_float(lo << 23), __uint_as_float(hi << 23));
}
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(two)));
  return r;
}

// Key (0..7) held by column n of an 8-key score tile.  The swap of the pairs 2, 3 and
// 6, 7 puts the four lanes of a quad on keys of both parities, so that their
// 8-byte loads of V (64-byte rows, chunks swizzled by bit 2 of the key) cover all banks.
__device__ __forceinline__ int key_of(int n) { return n ^ ((n >> 1) & 1); }

struct Request {
  int q0, n;      // first query token and their number
  int kv;         // keys
};
__device__ __forceinline__ Request request_of(const KvAttnArgs& a, int r) {
  Request x;
  const int64_t b = __ldg(a.cu_q + r), e = __ldg(a.cu_q + r + 1);
  const int kv = __ldg(a.kv_lens + r);
  const int64_t most = int64_t(a.width) << a.c.page_shift;
  if (b < 0 || e < b || e > a.total_q || e - b > a.max_q || kv < 0 || kv > most) {
    atomicOr(&g_status_kv_attn, DEV_BAD_INDEX);  // nothing of this request is computed
    x.q0 = x.n = x.kv = 0;
    return x;
  }
  x.q0 = int(b);
  x.n = int(e - b);
  x.kv = kv;
  return x;
}
__device__ __forceinline__ int tiles_of(const Request& x) { return max(1, (x.kv + kTile - 1) / kTile); }

// Tiles of all items of request r.
template <int ROWS>
__device__ __forceinline__ int64_t request_tiles(const KvAttnArgs& a, int r) {
  const Request x = request_of(a, r);
  if (x.n == 0) return 0;
  return int64_t((x.n * a.G + ROWS - 1) / ROWS) * a.c.H * tiles_of(x);
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

// One warp's softmax state and work on its keys of an item.
template <int FMT, int MT>
struct Worker {
  static constexpr int kSf = sf_bytes(FMT);
  uint32_t ring;        // this warp's stages
  int lane, c, g;
  float acc[MT][16][4];
  float m[MT][2], l[MT][2];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < MT; t++) {
#pragma unroll
      for (int j = 0; j < 16; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) acc[t][j][e] = 0.0f;
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.0f;
    }
  }

  // Issue the copies of 32 keys from key0 on; `block` is the block of key
  // key0 + lane (not `live`: the row is zero-filled and not visible).
  __device__ __forceinline__ void copy(const KvPages& p, int stage, int key0, int h, int64_t block, bool live) {
    const uint32_t s = ring + stage * stage_bytes(FMT);
    const int64_t row = ((live ? block : 0) * p.H + h) * p.page + ((key0 + lane) & (p.page - 1));
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int64_t rr = __shfl_sync(0xFFFFFFFFu, row, i * 8 + (lane >> 2));
      const bool ok = __shfl_sync(0xFFFFFFFFu, int(live), i * 8 + (lane >> 2)) != 0;
      const uint32_t dst = s + (i * 8 + (lane >> 2)) * 64 + (((lane & 3) ^ ((lane >> 4) << 1)) << 4);
      cp16(dst, p.k + rr * 64 + (lane & 3) * 16, ok);
      cp16(dst + kStep * 64, p.v + rr * 64 + (lane & 3) * 16, ok);
    }
    cp_sf<kSf>(s + kStep * 128 + lane * kSf, p.k_sf + row * kSf, live);
    cp_sf<kSf>(s + kStep * 128 + kStep * kSf + lane * kSf, p.v_sf + row * kSf, live);
  }

  // Scores, softmax and P V of the 32 keys in `stage`.  `seen` has a bit per key of
  // the step; limit[t][i]: keys of the row that count, relative to the first (both
  // only read if `masked`).
  __device__ __forceinline__ void compute(int stage, uint32_t qs, const float (&cs)[MT][2], uint32_t seen, bool masked,
                                          const int (&limit)[MT][2]) {
    const uint32_t s = ring + stage * stage_bytes(FMT);
    const uint32_t sfk = s + kStep * 128, sfv = sfk + kStep * kSf;
    float sc[MT][4][4];
#pragma unroll
    for (int t = 0; t < MT; t++)
#pragma unroll
      for (int n = 0; n < 4; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) sc[t][n][e] = 0.0f;
    {
      uint4 kw[4];
      uint32_t ks[4][2];
      const int kg = key_of(g);
#pragma unroll
      for (int n = 0; n < 4; n++) {
        const int key = n * 8 + kg;
        kw[n] = lds16(s + key * 64 + ((c ^ (((kg >> 2) & 1) << 1)) << 4));
        if (FMT == 0) {
          const uint32_t b = lds_u8(sfk + key * 4 + c);
          ks[n][0] = ks[n][1] = e8m0_pair(b, b);
        } else {
          const uint32_t b = e4m3_pair(lds_u16(sfk + key * 8 + 2 * c));
          ks[n][0] = __byte_perm(b, b, 0x1010);
          ks[n][1] = __byte_perm(b, b, 0x3232);
        }
      }
#pragma unroll
      for (int w = 0; w < 4; w++) {
        uint32_t a0[MT][4], a1[MT][4];
#pragma unroll
        for (int t = 0; t < MT; t++) {
          const uint4 x = lds16(qs + ((t * 8 + 2 * w) * 32 + lane) * 16);
          const uint4 y = lds16(qs + ((t * 8 + 2 * w + 1) * 32 + lane) * 16);
          a0[t][0] = x.x, a0[t][1] = x.y, a0[t][2] = x.z, a0[t][3] = x.w;
          a1[t][0] = y.x, a1[t][1] = y.y, a1[t][2] = y.z, a1[t][3] = y.w;
        }
#pragma unroll
        for (int n = 0; n < 4; n++) {
          const uint32_t word = w == 0 ? kw[n].x : w == 1 ? kw[n].y : w == 2 ? kw[n].z : kw[n].w;
          uint32_t hv[4];
          e2m1x8_to_f16(word, hv);
#pragma unroll
          for (int i = 0; i < 4; i++) hv[i] = hmul2(hv[i], ks[n][w >> 1]);
#pragma unroll
          for (int t = 0; t < MT; t++) {
            mma_f16(sc[t][n], a0[t], hv[0], hv[1]);
            mma_f16(sc[t][n], a1[t], hv[2], hv[3]);
          }
        }
      }
    }
    // scores in log2 units, masked
#pragma unroll
    for (int t = 0; t < MT; t++)
#pragma unroll
      for (int n = 0; n < 4; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          float x = sc[t][n][e] * cs[t][e >> 1];
          if (masked) {
            const int key = n * 8 + key_of(2 * c + (e & 1));
            if (!((seen >> key) & 1u) || key >= limit[t][e >> 1]) x = -INFINITY;
          }
          sc[t][n][e] = x;
        }
    uint32_t pf[MT][4][2];
    bool grow = false;
    float top[MT][2];
#pragma unroll
    for (int t = 0; t < MT; t++)
#pragma unroll
      for (int i = 0; i < 2; i++) {
        float x = fmaxf(sc[t][0][2 * i], sc[t][0][2 * i + 1]);
#pragma unroll
        for (int n = 1; n < 4; n++) x = fmax3(x, sc[t][n][2 * i], sc[t][n][2 * i + 1]);
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 2));
        top[t][i] = x;
        grow |= x > m[t][i] + kLazy;   // also from m = -inf on
      }
    if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
      for (int t = 0; t < MT; t++)
#pragma unroll
        for (int i = 0; i < 2; i++) {
          if (top[t][i] > m[t][i] + kLazy) {
            const float f = m[t][i] == -INFINITY ? 0.0f : ex2(m[t][i] - top[t][i]);
            m[t][i] = top[t][i];
            l[t][i] *= f;
#pragma unroll
            for (int j = 0; j < 16; j++) {
              acc[t][j][2 * i] *= f;
              acc[t][j][2 * i + 1] *= f;
            }
          }
        }
    }
#pragma unroll
    for (int t = 0; t < MT; t++)
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const float off = m[t][i] == -INFINITY ? 0.0f : kOffset - m[t][i];
#pragma unroll
        for (int n = 0; n < 4; n++) {
          const float p0 = ex2(sc[t][n][2 * i] + off), p1 = ex2(sc[t][n][2 * i + 1] + off);
          l[t][i] += p0 + p1;
          pf[t][n][i] = pack_f16(p0, p1);
        }
      }
    // V: a NaN block (scale byte 0xFF or 0x7F) reaches every row through 0 x NaN, so
    // where rows see different keys it is taken out of the product and put into the
    // rows that see its key
    const uint32_t vrow = ((((g >> 1) ^ (((c >> 1) & 1) << 1)) << 4) + ((g & 1) << 3));
    const int ka = key_of(2 * c), kb = key_of(2 * c + 1);
#pragma unroll
    for (int u = 0; u < 2; u++) {
      uint32_t bs[2];
      uint2 va[2], vb[2];
#pragma unroll
      for (int x = 0; x < 2; x++) {
        const int key = (2 * u + x) * 8;
        va[x] = lds8(s + kStep * 64 + (key + ka) * 64 + vrow);
        vb[x] = lds8(s + kStep * 64 + (key + kb) * 64 + vrow);
        uint32_t b0, b1;
        if (FMT == 0) {
          b0 = lds_u8(sfv + (key + ka) * 4 + (g >> 1));
          b1 = lds_u8(sfv + (key + kb) * 4 + (g >> 1));
          if (masked) {
            if (b0 == 0xFFu) b0 = 0;
            if (b1 == 0xFFu) b1 = 0;
          }
          bs[x] = e8m0_pair(b0, b1);
        } else {
          b0 = lds_u8(sfv + (key + ka) * 8 + g);
          b1 = lds_u8(sfv + (key + kb) * 8 + g);
          if (masked) {
            if ((b0 & 0x7Fu) == 0x7Fu) b0 = 0;
            if ((b1 & 0x7Fu) == 0x7Fu) b1 = 0;
          }
          bs[x] = e4m3_pair(b0 | (b1 << 8));
        }
      }
#pragma unroll
      for (int w = 0; w < 2; w++) {
        uint32_t b0e[4], b0o[4], b1e[4], b1o[4];
        {
          const uint32_t x = w ? va[0].y : va[0].x, y = w ? vb[0].y : vb[0].x;
          e2m1x8_to_f16((x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u), b0e);
          e2m1x8_to_f16(((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), b0o);
        }
        {
          const uint32_t x = w ? va[1].y : va[1].x, y = w ? vb[1].y : vb[1].x;
          e2m1x8_to_f16((x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u), b1e);
          e2m1x8_to_f16(((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), b1o);
        }
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const uint32_t e0 = hmul2(b0e[j], bs[0]), e1 = hmul2(b1e[j], bs[1]);
          const uint32_t o0 = hmul2(b0o[j], bs[0]), o1 = hmul2(b1o[j], bs[1]);
#pragma unroll
          for (int t = 0; t < MT; t++) {
            const uint32_t pa[4] = {pf[t][2 * u][0], pf[t][2 * u][1], pf[t][2 * u + 1][0], pf[t][2 * u + 1][1]};
            mma_f16(acc[t][w * 8 + 2 * j], pa, e0, e1);
            mma_f16(acc[t][w * 8 + 2 * j + 1], pa, o0, o1);
          }
        }
      }
    }
    if (masked) {
      // this lane's accumulators: channels 32c .. 32c + 31 of its rows
      const float nan = __uint_as_float(0x7FC00000u);
#pragma unroll 1
      for (int key = 0; key < kStep; key++) {
        bool lo, hi;  // NaN in channels 32c .. +15, 32c + 16 .. +31
        if (FMT == 0) {
          lo = hi = lds_u8(sfv + key * 4 + c) == 0xFFu;
        } else {
          const uint32_t b = lds_u16(sfv + key * 8 + 2 * c);
          lo = (b & 0x7Fu) == 0x7Fu;
          hi = (b & 0x7F00u) == 0x7F00u;
        }
        if (!(lo || hi) || !((seen >> key) & 1u)) continue;
#pragma unroll
        for (int t = 0; t < MT; t++)
#pragma unroll
          for (int i = 0; i < 2; i++)
            if (key < limit[t][i]) {
#pragma unroll
              for (int j = 0; j < 16; j++) {
                if (lo) acc[t][j][2 * i] = nan;
                if (hi) acc[t][j][2 * i + 1] = nan;
              }
            }
      }
    }
  }
};

template <int FMT, int MT>
__global__ void __launch_bounds__(kThreads, MT == 1 ? kCtasPerSm : 2) kv_attn_kernel(KvAttnArgs a) {
  constexpr int ROWS = 16 * MT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t s_scan[kWarps];
  __shared__ int64_t s_before;
  __shared__ int s_r;
  uint8_t* s_q = smem + area_bytes(FMT);
  float* s_ml = reinterpret_cast<float*>(s_q + ROWS * 256);  // [warp][row][m, l]
  float* s_cs = s_ml + kWarps * ROWS * 2;
  float* s_merge = reinterpret_cast<float*>(smem);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Header* headers = reinterpret_cast<Header*>(a.ws);
  Partial<MT>* partials = reinterpret_cast<Partial<MT>*>(a.ws + header_bytes(gridDim.x));
  if (tid == 0) headers[blockIdx.x].parts = 0;

  // the line of tiles and this CTA's run of it
  int64_t total = 0;
  for (int r0 = 0; r0 < a.R; r0 += kThreads) {
    int64_t sum;
    cta_scan(r0 + tid < a.R ? request_tiles<ROWS>(a, r0 + tid) : 0, s_scan, sum);
    total += sum;
  }
  const int64_t most = (total + kMinTiles - 1) / kMinTiles;
  const int64_t C = most < int64_t(gridDim.x) ? most : int64_t(gridDim.x);
  if (int64_t(blockIdx.x) >= C) return;
  const int64_t start = total * blockIdx.x / C, end = total * (blockIdx.x + 1) / C;
  if (start == end) return;
  {
    int64_t before = 0;
    for (int r0 = 0; r0 < a.R; r0 += kThreads) {
      int64_t sum;
      const int64_t own = r0 + tid < a.R ? request_tiles<ROWS>(a, r0 + tid) : 0;
      const int64_t upto = before + cta_scan(own, s_scan, sum);
      if (upto - own <= start && start < upto) {
        s_r = r0 + tid;
        s_before = upto - own;
      }
      before += sum;
      if (start < before) break;
    }
  }
  __syncthreads();
  int r = s_r;
  int64_t base = s_before;

  Worker<FMT, MT> wk;
  wk.ring = smem_u32(smem) + warp * kStages * stage_bytes(FMT);
  wk.lane = lane;
  wk.c = lane & 3;
  wk.g = lane >> 2;
  const float kst = FMT == 1 ? __ldg(a.c.k_scale) : 1.0f;
  const float vst = FMT == 1 ? __ldg(a.c.v_scale) : 1.0f;

  for (int64_t pos = start; pos < end && r < a.R;) {
    const Request x = request_of(a, r);
    const int tiles = tiles_of(x);
    const int nrb = (x.n * a.G + ROWS - 1) / ROWS;
    const int64_t all = x.n == 0 ? 0 : int64_t(nrb) * a.c.H * tiles;
    if (pos >= base + all) {
      base += all;
      r++;
      continue;
    }
    const int64_t local = pos - base;
    const int item = int(local / tiles), t0 = int(local - int64_t(item) * tiles);
    const int rb = item / a.c.H, h = item - rb * a.c.H;
    const int nt = int(min(int64_t(tiles - t0), end - pos));
    const int row0 = rb * ROWS, rows = min(ROWS, x.n * a.G - row0);
    const int first_tok = row0 / a.G, last_tok = (row0 + rows - 1) / a.G;
    // keys that some row of the block sees
    const int keys = a.causal ? max(0, x.kv - x.n + last_tok + 1) : x.kv;
    const int all_see = a.causal ? x.kv - x.n + first_tok + 1 : x.kv;
    const int k_lo = t0 * kTile + warp * kStep;
    const int k_end = min((t0 + nt) * kTile, keys);
    const int steps = k_lo < k_end ? (k_end - k_lo + kTile - 1) / kTile : 0;
    const int32_t* table = a.table + int64_t(r) * a.width;

    auto block_of = [&](int step) -> int {
      const int key = k_lo + step * kTile + lane;
      return step < steps && key < k_end ? __ldg(table + (key >> a.c.page_shift)) : -1;
    };
    uint32_t seen_ring[kStages];
    auto issue = [&](int step, int stage, int block) {
      const bool live = block >= 0 && block < a.c.blocks;
      const int key0 = k_lo + step * kTile;
      if (step < steps && key0 + lane < k_end && !live) atomicOr(&g_status_kv_attn, DEV_BAD_INDEX);
      if (step < steps) wk.copy(a.c, stage, key0, h, block, live);
      cp_commit();
      return __ballot_sync(0xFFFFFFFFu, live);
    };
    int nb[kStages];
#pragma unroll
    for (int i = 0; i < kStages; i++) nb[i] = block_of(i);
#pragma unroll
    for (int i = 0; i < kStages - 1; i++) seen_ring[i] = issue(i, i, nb[i]);
    int next_block = nb[kStages - 1];

    // Q of the item: binary16 with a power of two per row, in fragment order;
    // eight threads per row, 16 channels each
#pragma unroll
    for (int pass = 0; pass < MT; pass++) {
      const int i = pass * kThreads + tid;
      const int row = i >> 3, part = i & 7;
      uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
      if (row < rows) {
        const int rr = row0 + row, tok = rr / a.G, hd = rr - tok * a.G;
        const uint16_t* src = a.q + int64_t(x.q0 + tok) * a.q_stride + int64_t(h * a.G + hd) * 128 + part * 16;
        v0 = __ldg(reinterpret_cast<const uint4*>(src));
        v1 = __ldg(reinterpret_cast<const uint4*>(src) + 1);
      }
      const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
      uint32_t mx = 0;
#pragma unroll
      for (int e = 0; e < 8; e++) mx = max(mx, hmax2(abs2(w[e])));
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
      // 2^(14 - floor(log2 amax)), exponent field 268 - E, at most 2^126
      const int ex = int(mx >> 7);
      const int fe = mx == 0 ? 127 : min(253, 268 - ex);
      const float f = __uint_as_float(uint32_t(fe) << 23);
      const float inv = __uint_as_float(uint32_t(254 - fe) << 23);
      // channels 16 part + 0..15 belong to lane column c = part / 2, steps
      // 4 (part % 2) .. + 3, four channels a step: pairs a0/a2 (rows g), a1/a3 (rows g + 8)
      const int t = row >> 4, r16 = row & 15, cc = part >> 1;
#pragma unroll
      for (int st = 0; st < 4; st++) {
        const int ks = (part & 1) * 4 + st;
        uint32_t* dst = reinterpret_cast<uint32_t*>(s_q) + ((t * 8 + ks) * 32 + (r16 & 7) * 4 + cc) * 4 + (r16 >> 3);
        dst[0] = pack_f16(bf_lo(w[2 * st]) * f, bf_hi(w[2 * st]) * f);
        dst[2] = pack_f16(bf_lo(w[2 * st + 1]) * f, bf_hi(w[2 * st + 1]) * f);
      }
      if (part == 0) s_cs[row] = a.scale_log2 * kst * inv;
    }
    __syncthreads();
    float cs[MT][2];
    int lim[MT][2];
#pragma unroll
    for (int t = 0; t < MT; t++)
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const int row = t * 16 + wk.g + 8 * i;
        cs[t][i] = s_cs[row];
        lim[t][i] = !a.causal || row >= rows ? x.kv : x.kv - x.n + (row0 + row) / a.G + 1;
      }
    wk.clear();
    const uint32_t qs = smem_u32(s_q);
    for (int s0 = 0; s0 < steps; s0 += kStages) {
#pragma unroll
      for (int u = 0; u < kStages; u++) {
        const int step = s0 + u;
        if (step >= steps) break;
        // the stage of step - 1 is free: every lane has read it
        __syncwarp();
        seen_ring[(u + kStages - 1) % kStages] = issue(step + kStages - 1, (u + kStages - 1) % kStages, next_block);
        next_block = block_of(step + kStages);
        cp_wait<kStages - 1>();
        __syncwarp();
        const int key0 = k_lo + step * kTile;
        const uint32_t seen = seen_ring[u];
        const bool masked = seen != 0xFFFFFFFFu || key0 + kStep > all_see;
        int limit[MT][2];
#pragma unroll
        for (int t = 0; t < MT; t++)
#pragma unroll
          for (int i = 0; i < 2; i++) limit[t][i] = lim[t][i] - key0;
        wk.compute(u, qs, cs, seen, masked, limit);
      }
    }
    cp_wait<0>();
    // join the warps' states
#pragma unroll
    for (int t = 0; t < MT; t++)
#pragma unroll
      for (int i = 0; i < 2; i++) {
        float v = wk.l[t][i];
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
        if (wk.c == 0) {
          float* p = s_ml + (warp * ROWS + t * 16 + wk.g + 8 * i) * 2;
          p[0] = wk.m[t][i];
          p[1] = v;
        }
      }
    const bool head_part = t0 > 0, cut = t0 + nt < tiles;
    Partial<MT>* part = &partials[2 * blockIdx.x + (head_part ? 0 : 1)];
#pragma unroll
    for (int t = 0; t < MT; t++) {
      __syncthreads();  // the rings, or the previous sixteen rows, are no longer read
#pragma unroll
      for (int i = 0; i < 2; i++) {
        float* dst = s_merge + (warp * 16 + wk.g + 8 * i) * kMergeRow + wk.c * 36;
#pragma unroll
        for (int e = 0; e < 2; e++)
#pragma unroll
          for (int j = 0; j < 16; j += 4)
            *reinterpret_cast<float4*>(dst + e * 16 + j) = make_float4(wk.acc[t][j][2 * i + e], wk.acc[t][j + 1][2 * i + e],
                                                                       wk.acc[t][j + 2][2 * i + e], wk.acc[t][j + 3][2 * i + e]);
      }
      __syncthreads();
      const int row = tid >> 3, col = (tid & 7) * 16;  // sixteen channels a thread
      const int frow = t * 16 + row;
      float M = -INFINITY, L = 0.0f, w[kWarps];
#pragma unroll
      for (int k = 0; k < kWarps; k++) M = fmaxf(M, s_ml[(k * ROWS + frow) * 2]);
#pragma unroll
      for (int k = 0; k < kWarps; k++) {
        // without keys (m = -inf) l and O are 0, or NaN where every score was
        const float mk = s_ml[(k * ROWS + frow) * 2];
        w[k] = mk == -INFINITY ? 1.0f : ex2(mk - M);
        L += w[k] * s_ml[(k * ROWS + frow) * 2 + 1];
      }
      float o[16];
#pragma unroll
      for (int j = 0; j < 16; j++) o[j] = 0.0f;
#pragma unroll
      for (int k = 0; k < kWarps; k++) {
        const float* src = s_merge + (k * 16 + row) * kMergeRow + (col >> 5) * 36 + (col & 16);
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 v = *reinterpret_cast<const float4*>(src + j);
          o[j] += w[k] * v.x;
          o[j + 1] += w[k] * v.y;
          o[j + 2] += w[k] * v.z;
          o[j + 3] += w[k] * v.w;
        }
      }
      if (frow < rows) {
        if (head_part || cut) {
#pragma unroll
          for (int j = 0; j < 16; j += 4)
            *reinterpret_cast<float4*>(&part->o[frow][col + j]) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
          if ((tid & 7) == 0) {
            part->m[frow] = M;
            part->l[frow] = L;
          }
        } else {
          const int rr = row0 + frow, tok = rr / a.G, hd = h * a.G + rr - tok * a.G;
          const float f = L == 0.0f ? 1.0f : vst / L;
          uint4* dst = reinterpret_cast<uint4*>(a.o + (int64_t(x.q0 + tok) * a.Hq + hd) * 128 + col);
#pragma unroll
          for (int j = 0; j < 16; j += 8)
            dst[j >> 3] = make_uint4(pack_bf16(o[j] * f, o[j + 1] * f), pack_bf16(o[j + 2] * f, o[j + 3] * f),
                                     pack_bf16(o[j + 4] * f, o[j + 5] * f), pack_bf16(o[j + 6] * f, o[j + 7] * f));
          if ((tid & 7) == 0)
            a.lse[int64_t(hd) * a.total_q + x.q0 + tok] =
                L == 0.0f ? -INFINITY : (M - kOffset + log2f(L)) * 0.6931471805599453f;
        }
      }
    }
    if (cut && !head_part && tid == 0) {
      const int64_t last = base + int64_t(item + 1) * tiles - 1;  // the CTA of the item's last tile
      Header hd;
      hd.r = r;
      hd.rb = rb;
      hd.h = h;
      hd.parts = int(((last + 1) * C - 1) / total) - int(blockIdx.x);
      headers[blockIdx.x] = hd;
    }
    pos += nt;
    __syncthreads();  // Q and the row states are no longer read
  }
}

// Joins the parts of the item that begins in CTA blockIdx.x's run and ends behind
// it: one warp per row, four channels a lane, parts in the order of the keys.
template <int FMT, int MT>
__global__ void __launch_bounds__(128) kv_join_kernel(KvAttnArgs a, int ctas) {
  const Header hd = reinterpret_cast<const Header*>(a.ws)[blockIdx.x];
  if (hd.parts == 0) return;
  const Partial<MT>* partials = reinterpret_cast<const Partial<MT>*>(a.ws + header_bytes(ctas));
  const int row = blockIdx.y * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const Request x = request_of(a, hd.r);
  const int rr = hd.rb * 16 * MT + row;
  if (rr >= x.n * a.G) return;
  auto part = [&](int i) -> const Partial<MT>& { return partials[2 * (blockIdx.x + i) + (i == 0 ? 1 : 0)]; };
  float M = -INFINITY;
  for (int i = lane; i <= hd.parts; i += 32) M = fmaxf(M, part(i).m[row]);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
  float L = 0.0f;
  float4 s = make_float4(0, 0, 0, 0);
#pragma unroll 4
  for (int i = 0; i <= hd.parts; i++) {
    const Partial<MT>& p = part(i);
    const float m = p.m[row];
    const float w = m == -INFINITY ? 1.0f : ex2(m - M);  // without keys l and O are 0, or NaN
    const float4 v = *reinterpret_cast<const float4*>(&p.o[row][lane * 4]);
    L += w * p.l[row];
    s.x += w * v.x;
    s.y += w * v.y;
    s.z += w * v.z;
    s.w += w * v.w;
  }
  const float vst = FMT == 1 ? __ldg(a.c.v_scale) : 1.0f;
  const float f = L == 0.0f ? 1.0f : vst / L;
  const int tok = rr / a.G, head = hd.h * a.G + rr - tok * a.G;
  *reinterpret_cast<uint2*>(a.o + (int64_t(x.q0 + tok) * a.Hq + head) * 128 + lane * 4) =
      make_uint2(pack_bf16(s.x * f, s.y * f), pack_bf16(s.z * f, s.w * f));
  if (lane == 0)
    a.lse[int64_t(head) * a.total_q + x.q0 + tok] =
        L == 0.0f ? -INFINITY : (M - kOffset + log2f(L)) * 0.6931471805599453f;
}

template <int MT>
size_t workspace(int ctas) {
  return header_bytes(ctas) + size_t(ctas) * 2 * sizeof(Partial<MT>);
}

template <int FMT, int MT>
cudaError_t launch(const KvAttnArgs& a, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  constexpr int bytes = smem_bytes(FMT, MT);
  cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(kv_attn_kernel<FMT, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  });
  if (e != cudaSuccess) return e;
  const int ctas = sm_count_current_device() * (MT == 1 ? kCtasPerSm : 2);
  if (ctas <= 0) return cudaErrorInvalidDevice;
  kv_attn_kernel<FMT, MT><<<ctas, kThreads, bytes, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  kv_join_kernel<FMT, MT><<<dim3(unsigned(ctas), 4 * MT), 128, 0, st>>>(a, ctas);
  return cudaGetLastError();
}

}  // namespace kva

size_t kv_attn_workspace(int R, int max_q, int G) {
  (void)R;
  const int sms = sm_count_current_device();
  return int64_t(max_q) * G <= 16 ? kva::workspace<1>(sms * kva::kCtasPerSm) : kva::workspace<2>(sms * 2);
}

cudaError_t launch_kv_attn(const KvAttnArgs& a, cudaStream_t st) {
  clear_stale_error();
  if (int64_t(a.max_q) * a.G <= 16) return a.c.fmt == 0 ? kva::launch<0, 1>(a, st) : kva::launch<1, 1>(a, st);
  return a.c.fmt == 0 ? kva::launch<0, 2>(a, st) : kva::launch<1, 2>(a, st);
}

unsigned read_status_kv_attn(cudaStream_t st) {
  unsigned v = 0, z = 0;
  cudaMemcpyFromSymbolAsync(&v, g_status_kv_attn, sizeof(v), 0, cudaMemcpyDeviceToHost, st);
  cudaMemcpyToSymbolAsync(g_status_kv_attn, &z, sizeof(z), 0, cudaMemcpyHostToDevice, st);
  cudaStreamSynchronize(st);
  return v;
}

}  // namespace mxfa
