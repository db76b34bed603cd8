// rope.cu -- rotary positions: channels of q and k turned by their token's position, for training
// (and turned back, for the gradients), and fused with the store of k and v into the 4-bit cache.
//
//   pair i of the first rot channels, at position p:  a' = g (a cos t - b sin t),  b' = g (b cos t + a sin t),
//   t = p f_i; the pair is channels (i, i + rot / 2) or (2 i, 2 i + 1); the other channels stay.
// The gradient of (a, b) is the same turn by -t of the gradient of (a', b').
//
// Angles.  An fp32 product p f loses the angle for far positions (a position of 2^20 leaves 2^-4
// radians), and fp64 is slow here, so frequencies are whole numbers of 2^-64ths of a turn: p times one,
// modulo 2^64, is the fraction of a turn exactly (the frequency's own rounding, 2^-65 turns, grows to 2^-34 for
// p = 2^31), and its upper 32 bits, as a signed fraction of a half turn, are the argument of sincospi: within
// 2^-24 of pi radians, well below the bf16 results' 2^-9.
//
// A warp takes some heads of one token: its lanes compute the token's angles once, two pairs a lane, and pass them
// through shared memory; then sixteen lanes a head, eight channels a lane, whose partners in the half layout are
// rot / 16 lanes away.  Every element is read and written once.
#include "kv_rows.cuh"

namespace mxfa {

static __device__ unsigned g_status_rope;

namespace {

constexpr int kWarps = 4;

// The (cos, sin) of a token's pairs, times the gain, into a warp's `cs`.
__device__ __forceinline__ void angles(const Rotation& r, int pos, int lane, float2* cs) {
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const int pair = lane + 32 * i;
    if (2 * pair < r.rot) {
      const uint64_t turn = uint64_t(uint32_t(pos)) * __ldg(r.turns + pair);
      float s, c;
      sincospif(float(int32_t(turn >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31
      cs[pair] = make_float2(c * r.gain, (r.inverse ? -s : s) * r.gain);
    }
  }
  __syncwarp();
}

// A lane's cosines and sines: channels 8 l .. 8 l + 7 of a head, two to a register pair.
template <bool INTER>
struct Turn {
  float2 c[4], s[4];
  bool turned;
  int partner;
  __device__ __forceinline__ Turn(const float2* cs, int rot, int lane) {
    const int l = lane & 15;
    turned = 8 * l < rot;
    const bool second = !INTER && 16 * l >= rot;
    const int first = !turned ? 0 : INTER ? 4 * l : second ? 8 * l - rot / 2 : 8 * l;
    partner = !turned ? lane : second ? lane - rot / 16 : lane + rot / 16;
#pragma unroll
    for (int e = 0; e < (INTER ? 2 : 4); e++) {
      const float4 v = *reinterpret_cast<const float4*>(cs + first + 2 * e);
      if (INTER) {
        c[2 * e] = make_float2(v.x, v.x), c[2 * e + 1] = make_float2(v.z, v.z);
        s[2 * e] = make_float2(-v.y, v.y), s[2 * e + 1] = make_float2(-v.w, v.w);
      } else {
        c[e] = make_float2(v.x, v.z);
        s[e] = second ? make_float2(v.y, v.w) : make_float2(-v.y, -v.w);
      }
    }
  }
  // All lanes of the warp.
  __device__ __forceinline__ uint4 operator()(uint4 x) const {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t y[4];
#pragma unroll
    for (int e = 0; e < 4; e++) {
      // the other channel of each pair: beside it, or in the partner's word
      const uint32_t p = INTER ? w[e] : __shfl_sync(0xFFFFFFFFu, w[e], partner);
      const float2 own = make_float2(bf_lo(w[e]), bf_hi(w[e]));
      const float2 other = INTER ? make_float2(own.y, own.x) : make_float2(bf_lo(p), bf_hi(p));
      const float2 r = ffma2(own, c[e], fmul2(other, s[e]));
      y[e] = pack_bf16(r.x, r.y);
    }
    return turned ? make_uint4(y[0], y[1], y[2], y[3]) : x;
  }
};

// Sixteen bytes that nothing reads again soon, but that this thread may write (results in place).
__device__ __forceinline__ uint4 load_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// Heads h0 .. h1 - 1 of a token, N rows a lane group in flight.
template <bool INTER, int N>
__global__ void __launch_bounds__(kWarps * 32) rope_kernel(RopeArgs a) {
  __shared__ __align__(16) float2 s_cs[kWarps][64];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t item = int64_t(blockIdx.x) * kWarps + warp;
  const int64_t token = item / a.parts;
  if (token >= a.tokens) return;
  const int pos = __ldg(a.positions + token);
  if (pos < 0) return;
  const int h0 = int(item - token * a.parts) * a.heads_per_part, h1 = min(h0 + a.heads_per_part, a.H);
  const uint16_t* x = a.x + token * a.x_stride + (lane & 15) * 8;
  uint16_t* y = a.y + token * a.y_stride + (lane & 15) * 8;
  uint4 v[N];
  auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < N; i++) {
      v[i] = make_uint4(0, 0, 0, 0);
      if (h + 2 * i < h1) v[i] = load_stream(reinterpret_cast<const uint4*>(x + (h + 2 * i) * 128));
    }
  };
  int h = h0 + (lane >> 4);
  load(h);  // on their way while the angles are computed
  angles(a.rot, pos, lane, s_cs[warp]);
  const Turn<INTER> turn(s_cs[warp], a.rot.rot, lane);
  while (true) {
#pragma unroll
    for (int i = 0; i < N; i++) {
      const uint4 o = turn(v[i]);
      if (h + 2 * i < h1) __stcs(reinterpret_cast<uint4*>(y + (h + 2 * i) * 128), o);
    }
    h += 2 * N;
    if (h - (lane >> 4) >= h1) break;
    load(h);
  }
}

// The same for q, and k and v into the cache.  A warp has heads of q, or rows of K and V (those of K first).
template <int FMT, bool INTER, int N>
__global__ void __launch_bounds__(kWarps * 32) kv_append_rope_kernel(KvAppendRopeArgs a) {
  __shared__ __align__(16) float2 s_cs[kWarps][64];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l16 = lane & 15;
  const int64_t item = int64_t(blockIdx.x) * kWarps + warp;
  const int parts = a.q_parts + a.kv_parts;
  const int64_t token = item / parts;
  if (token >= a.tokens) return;
  const int pos = __ldg(a.positions + token);
  if (pos < 0) return;
  const int part = int(item - token * parts);
  const bool is_q = part < a.q_parts;
  int64_t slot = 0, block = 0;
  if (!is_q) {
    slot = __ldg(a.slots + token);
    block = slot >> a.c.page_shift;
    if (slot < 0) return;
    if (block >= a.c.blocks) {
      if (lane == 0) atomicOr(&g_status_rope, DEV_BAD_INDEX);
      return;
    }
  }
  const int all = is_q ? a.Hq : 2 * a.c.H;
  const int h0 = (is_q ? part : part - a.q_parts) * a.heads_per_part, h1 = min(h0 + a.heads_per_part, all);
  const uint16_t* q = a.q + token * a.q_stride;
  const uint16_t* k = a.k + token * a.k_stride;
  const uint16_t* v = a.v + token * a.v_stride;
  uint16_t* y = a.y + token * a.y_stride;
  uint4 x[N];
  auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < N; i++) {
      const int r = h + 2 * i;
      x[i] = make_uint4(0, 0, 0, 0);
      if (r < h1) {
        const uint16_t* src = is_q ? q + r * 128 : r < a.c.H ? k + r * 128 : v + (r - a.c.H) * 128;
        x[i] = load_stream(reinterpret_cast<const uint4*>(src + l16 * 8));
      }
    }
  };
  int h = h0 + (lane >> 4);
  load(h);  // on their way while the angles are computed
  angles(a.rot, pos, lane, s_cs[warp]);
  const Turn<INTER> turn(s_cs[warp], a.rot.rot, lane);
  while (true) {
#pragma unroll
    for (int i = 0; i < N; i++) {
      const int r = h + 2 * i;
      const uint4 o = turn(x[i]);
      if (is_q) {
        if (r < h1) *reinterpret_cast<uint4*>(y + r * 128 + l16 * 8) = o;
      } else {
        const bool is_v = r >= a.c.H;
        const int64_t at = (block * a.c.H + (is_v ? r - a.c.H : r)) * a.c.page + (slot & (a.c.page - 1));
        kv_store_row<FMT>(a.c, r < h1, is_v, at, l16, is_v ? x[i] : o);
      }
    }
    h += 2 * N;
    if (h - (lane >> 4) >= h1) break;
    load(h);
  }
}

// Heads a warp takes, `most` at most: fewer where there are few tokens, so that the call spreads over the GPU; many
// share a token's angles.  16384 tokens of 32 + 8 heads stored take 89, 74, 67 and 67 us with 8, 16, 32 and 64, of 32
// heads turned 47, 43, 44 and 44 us.
int heads_per_part(int64_t tokens, int heads, int most) {
  const int64_t warps = int64_t(sm_count_current_device()) * 32;
  for (int n = most; n > 2; n /= 2)
    if (tokens * ((heads + n - 1) / n) >= warps) return n;
  return 2;
}

template <bool INTER>
void rope_n(const RopeArgs& a, unsigned grid, cudaStream_t s) {
  if (a.heads_per_part > 4) rope_kernel<INTER, 4><<<grid, kWarps * 32, 0, s>>>(a);
  else rope_kernel<INTER, 1><<<grid, kWarps * 32, 0, s>>>(a);
}

template <int FMT, bool INTER>
void append_n(const KvAppendRopeArgs& a, unsigned grid, cudaStream_t s) {
  if (a.heads_per_part > 4) kv_append_rope_kernel<FMT, INTER, 4><<<grid, kWarps * 32, 0, s>>>(a);
  else kv_append_rope_kernel<FMT, INTER, 1><<<grid, kWarps * 32, 0, s>>>(a);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& args, cudaStream_t s) {
  clear_stale_error();
  RopeArgs a = args;
  a.heads_per_part = heads_per_part(a.tokens, a.H, 16);
  a.parts = (a.H + a.heads_per_part - 1) / a.heads_per_part;
  const int64_t grid = (a.tokens * a.parts + kWarps - 1) / kWarps;
  if (a.rot.inter) rope_n<true>(a, unsigned(grid), s);
  else rope_n<false>(a, unsigned(grid), s);
  return cudaGetLastError();
}

cudaError_t launch_kv_append_rope(const KvAppendRopeArgs& args, cudaStream_t s) {
  clear_stale_error();
  KvAppendRopeArgs a = args;
  a.heads_per_part = heads_per_part(a.tokens, a.Hq + 2 * a.c.H, 32);
  a.q_parts = (a.Hq + a.heads_per_part - 1) / a.heads_per_part;
  a.kv_parts = (2 * a.c.H + a.heads_per_part - 1) / a.heads_per_part;
  const int64_t grid = (a.tokens * (a.q_parts + a.kv_parts) + kWarps - 1) / kWarps;
  if (a.c.fmt == 0) a.rot.inter ? append_n<0, true>(a, unsigned(grid), s) : append_n<0, false>(a, unsigned(grid), s);
  else a.rot.inter ? append_n<1, true>(a, unsigned(grid), s) : append_n<1, false>(a, unsigned(grid), s);
  return cudaGetLastError();
}

unsigned read_status_rope(cudaStream_t st) {
  unsigned v = 0, z = 0;
  cudaMemcpyFromSymbolAsync(&v, g_status_rope, sizeof(v), 0, cudaMemcpyDeviceToHost, st);
  cudaMemcpyToSymbolAsync(g_status_rope, &z, sizeof(z), 0, cudaMemcpyHostToDevice, st);
  cudaStreamSynchronize(st);
  return v;
}

}  // namespace mxfa
