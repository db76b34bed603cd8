// rope.cu -- rotary positions: channels of q and k turned by their token's position, for training
// (and turned back, for the gradients), and fused with the store of k and v into the 4-bit cache.
//
//   pair i of the first rot channels, at position p:  a' = g (a cos t - b sin t),  b' = g (b cos t + a sin t),
//   t = p f_i; the pair is channels (i, i + rot / 2) or (2 i, 2 i + 1); the other channels stay.
// The gradient of (a, b) is the same turn by -t of the gradient of (a', b').
//
// Every step is one correctly rounded fp32 operation, as an elementwise program has them: c = fp32(g cos t) and
// s = fp32(g sin t), two products, their sum, and bf16 of it.  So what an elementwise form of the same steps turns and
// stores is the same codes here, where an fp32 step off would now and then move a 4-bit code by a quarter.
//
// Angles.  An fp32 product p f loses the angle for far positions (a position of 2^20 leaves 2^-4
// radians), and fp64 is slow here, so frequencies are whole numbers of 2^-64ths of a turn: p times one,
// modulo 2^64, is the fraction of a turn exactly (the frequency's own rounding, 2^-65 turns, grows to 2^-34 for
// p = 2^31).  Its quarter turn, the nearest of 64 equal parts of that and the rest b, |b| <= pi / 256, are whole numbers, too, and
//   cos(a + b) = cos a + (cos a (cos b - 1) - sin a sin b),  sin(a + b) = sin a + (sin a (cos b - 1) + cos a sin b)
// with cos a, sin a, b and the first sum in pairs of fp32 values and short series for b: off by 2^-35 at most
// before the rounding, so all but one in 3000 of the results are the correctly rounded ones.
//
// A warp takes some heads of one token: its lanes compute the token's angles once, two pairs a lane, and pass them
// through shared memory; then sixteen lanes a head, eight channels a lane, whose partners in the half layout are
// rot / 16 lanes away.  Every element is read and written once.
#include "kv_rows.cuh"

namespace mxfa {

static __device__ unsigned g_status_rope;

namespace {

constexpr int kWarps = 4;

// cos a, what it lacks of 53 bits, and sin a likewise: a = i pi / 128.
__device__ const float4 kParts[33] = {
    {0x1.0p+0f, 0x0.0p+0f, 0x0.0p+0f, 0x0.0p+0f},
    {0x1.ffd886p-1f, 0x1.099a1ap-30f, 0x1.92156p-6f, -0x1.0b933p-31f},
    {0x1.ff621ep-1f, 0x1.bcb6bep-28f, 0x1.91f66p-5f, -0x1.de44fep-30f},
    {0x1.fe9cdap-1f, 0x1.a03108p-26f, 0x1.2d520ap-4f, -0x1.a63cc2p-29f},
    {0x1.fd88dap-1f, 0x1.e89292p-28f, 0x1.917a6cp-4f, -0x1.eb25eap-31f},
    {0x1.fc2648p-1f, -0x1.e3cc06p-26f, 0x1.f564e6p-4f, -0x1.2ad19ep-29f},
    {0x1.fa7558p-1f, -0x1.eeb5d2p-30f, 0x1.2c8106p-3f, 0x1.d1cc28p-28f},
    {0x1.f8765p-1f, -0x1.63ad16p-27f, 0x1.5e2144p-3f, 0x1.22cff2p-29f},
    {0x1.f6297cp-1f, 0x1.feeb96p-26f, 0x1.8f8b84p-3f, -0x1.cb2cfap-30f},
    {0x1.f38f3ap-1f, 0x1.8c9cb2p-26f, 0x1.c0b826p-3f, 0x1.4fc9ecp-28f},
    {0x1.f0a7fp-1f, -0x1.1b73cap-27f, 0x1.f19f98p-3f, -0x1.37a83ap-29f},
    {0x1.ed740ep-1f, 0x1.da1258p-27f, 0x1.111d26p-2f, 0x1.58fb3cp-29f},
    {0x1.e9f416p-1f, -0x1.273a44p-26f, 0x1.294062p-2f, 0x1.dab3ep-27f},
    {0x1.e6288ep-1f, 0x1.891c22p-26f, 0x1.4135cap-2f, -0x1.7d134p-27f},
    {0x1.e2121p-1f, 0x1.3da1bap-27f, 0x1.58f9a8p-2f, -0x1.4a9c04p-27f},
    {0x1.ddb13cp-1f, -0x1.2667b8p-26f, 0x1.708854p-2f, -0x1.e0b74cp-27f},
    {0x1.d906bcp-1f, 0x1.e651a8p-26f, 0x1.87de2ap-2f, 0x1.abaa58p-28f},
    {0x1.d4134ep-1f, -0x1.d646d8p-26f, 0x1.9ef794p-2f, 0x1.d476c6p-29f},
    {0x1.ced7bp-1f, -0x1.786712p-26f, 0x1.b5d1p-2f, 0x1.3c2b98p-27f},
    {0x1.c954b2p-1f, 0x1.3411f4p-29f, 0x1.cc66eap-2f, -0x1.b38ee8p-28f},
    {0x1.c38b3p-1f, -0x1.cfe84ap-26f, 0x1.e2b5d4p-2f, -0x1.fe4272p-28f},
    {0x1.bd7c0ap-1f, 0x1.8df2a6p-26f, 0x1.f8ba4ep-2f, -0x1.01d952p-28f},
    {0x1.b72834p-1f, 0x1.465b9p-27f, 0x1.07387ap-1f, -0x1.b74004p-27f},
    {0x1.b090a6p-1f, -0x1.fabf8p-27f, 0x1.11eb36p-1f, -0x1.7c969cp-26f},
    {0x1.a9b662p-1f, 0x1.21d434p-26f, 0x1.1c73b4p-1f, -0x1.9465cep-27f},
    {0x1.a29a7ap-1f, 0x1.189e08p-31f, 0x1.26d054p-1f, 0x1.9ba25cp-26f},
    {0x1.9b3e04p-1f, 0x1.fce1dp-27f, 0x1.30ff8p-1f, -0x1.8f47e6p-28f},
    {0x1.93a224p-1f, 0x1.324c8p-26f, 0x1.3affa2p-1f, 0x1.240a18p-26f},
    {0x1.8bc806p-1f, 0x1.62a2e8p-26f, 0x1.44cf32p-1f, 0x1.424776p-27f},
    {0x1.83b0ep-1f, 0x1.7ff2eep-26f, 0x1.4e6cacp-1f, -0x1.070686p-27f},
    {0x1.7b5df2p-1f, 0x1.3557d8p-28f, 0x1.57d694p-1f, -0x1.6e626cp-26f},
    {0x1.72d084p-1f, -0x1.02000ep-26f, 0x1.610b76p-1f, -0x1.5c5a64p-26f},
    {0x1.6a09e6p-1f, 0x1.9fcef4p-27f, 0x1.6a09e6p-1f, 0x1.9fcef4p-27f}};

// An exact product's rounding error; sums whose first term is the larger one, or 0.
__device__ __forceinline__ float product_rest(float a, float b, float p) { return __fmaf_rn(a, b, -p); }
__device__ __forceinline__ float2 sum_of(float a, float b, float rest) {
  const float h = __fadd_rn(a, b);
  return make_float2(h, __fadd_rn(__fsub_rn(b, __fsub_rn(h, a)), rest));
}

// (cos, sin) of a turn's 2^-64ths, times the gain, each rounded once.
__device__ __forceinline__ float2 cos_sin(uint64_t turn, float gain, float gain_rest) {
  const unsigned quarter = unsigned((turn + (1ull << 61)) >> 62);
  const int64_t r = int64_t(turn - (uint64_t(quarter) << 62));      // |r| <= 2^61: an eighth of a turn
  const int part = int((r + (int64_t(1) << 55)) >> 56);              // -32 .. 32
  const int d = int((r - (int64_t(part) << 56)) >> 24);              // 2^-40ths of a turn
  const float dh = __int2float_rn(d), dl = __int2float_rn(d - __float2int_rn(dh));
  constexpr float kUnit = 0x1.921fb6p-38f, kUnitRest = -0x1.777a5cp-63f;  // 2 pi 2^-40
  const float b = __fmul_rn(dh, kUnit);
  const float b_rest = __fadd_rn(product_rest(dh, kUnit, b), __fmaf_rn(dh, kUnitRest, __fmul_rn(dl, kUnit)));
  const float b2 = __fmul_rn(b, b);
  const float sin_rest = __fmaf_rn(-__fmul_rn(b, b2), 1.0f / 6.0f, b_rest);                // sin b = b + this
  const float cos_less = __fmul_rn(__fmaf_rn(b2, 1.0f / 24.0f, -0.5f), b2);                // cos b - 1
  float4 t = __ldg(&kParts[abs(part)]);
  if (part < 0) t.z = -t.z, t.w = -t.w;
  const float p = __fmul_rn(t.z, b), q = __fmul_rn(t.x, b);
  const float cr = __fsub_rn(__fmaf_rn(t.x, cos_less, t.y), __fmaf_rn(t.w, b, __fmaf_rn(t.z, sin_rest, product_rest(t.z, b, p))));
  const float sr = __fadd_rn(__fmaf_rn(t.z, cos_less, t.w), __fmaf_rn(t.y, b, __fmaf_rn(t.x, sin_rest, product_rest(t.x, b, q))));
  const float2 c = sum_of(t.x, -p, cr), s = sum_of(t.z, q, sr);
  auto times_gain = [&](float2 x) {
    const float y = __fmul_rn(x.x, gain);
    return __fadd_rn(y, __fadd_rn(product_rest(x.x, gain, y), __fmaf_rn(x.y, gain, __fmul_rn(x.x, gain_rest))));
  };
  const float gc = times_gain(c), gs = times_gain(s);
  const float2 v = quarter & 1u ? make_float2(-gs, gc) : make_float2(gc, gs);
  return quarter & 2u ? make_float2(-v.x, -v.y) : v;
}

// The (cos, sin) of a token's pairs, times the gain, into a warp's `cs`.
__device__ __forceinline__ void angles(const Rotation& r, int pos, int lane, float2* cs) {
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const int pair = lane + 32 * i;
    if (2 * pair < r.rot) {
      const float2 v = cos_sin(uint64_t(uint32_t(pos)) * __ldg(r.turns + pair), r.gain, r.gain_rest);
      cs[pair] = make_float2(v.x, r.inverse ? -v.y : v.y);
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
      // rounded one by one: packed pairs of products and sums would be merged into a multiply-add, and some
      // bf16 results another (16384 tokens stored 2 us sooner at most)
      y[e] = pack_bf16(__fadd_rn(__fmul_rn(own.x, c[e].x), __fmul_rn(other.x, s[e].x)),
                       __fadd_rn(__fmul_rn(own.y, c[e].y), __fmul_rn(other.y, s[e].y)));
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

// The same for q, and k and v into the cache.  A warp has heads of q, or rows of K and V (those of K first), each in a loop of
// its own: one for both took 68 us instead of 61 for 16384 tokens of 32 + 8 heads.  The next rows on their way while
// these are turned: 79 (registers for fewer warps).
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
  auto load = [&](int h, auto&& at) {
#pragma unroll
    for (int i = 0; i < N; i++) {
      const int r = h + 2 * i;
      x[i] = make_uint4(0, 0, 0, 0);
      if (r < h1) x[i] = load_stream(reinterpret_cast<const uint4*>(at(r) + l16 * 8));
    }
  };
  int h = h0 + (lane >> 4);
  if (is_q) {
    auto at = [&](int r) { return q + r * 128; };
    load(h, at);  // on their way while the angles are computed
    angles(a.rot, pos, lane, s_cs[warp]);
    const Turn<INTER> turn(s_cs[warp], a.rot.rot, lane);
    while (true) {
#pragma unroll
      for (int i = 0; i < N; i++) {
        const int r = h + 2 * i;
        const uint4 o = turn(x[i]);
        if (r < h1) __stcs(reinterpret_cast<uint4*>(y + r * 128 + l16 * 8), o);
      }
      h += 2 * N;
      if (h - (lane >> 4) >= h1) break;
      load(h, at);
    }
    return;
  }
  auto at = [&](int r) { return r < a.c.H ? k + r * 128 : v + (r - a.c.H) * 128; };
  load(h, at);
  angles(a.rot, pos, lane, s_cs[warp]);
  const Turn<INTER> turn(s_cs[warp], a.rot.rot, lane);
  while (true) {
#pragma unroll
    for (int i = 0; i < N; i++) {
      const int r = h + 2 * i;
      const bool is_v = r >= a.c.H;
      uint4 o = x[i];
      if (r - (lane >> 4) < a.c.H) {  // of K, or the warp's other row is
        const uint4 t = turn(o);
        if (!is_v) o = t;
      }
      const int64_t to = (block * a.c.H + (is_v ? r - a.c.H : r)) * a.c.page + (slot & (a.c.page - 1));
      kv_store_row<FMT>(a.c, r < h1, is_v, to, l16, o);
    }
    h += 2 * N;
    if (h - (lane >> 4) >= h1) break;
    load(h, at);
  }
}

// Heads a warp takes, `most` at most: fewer where there are few tokens, so that the call spreads over the GPU; many
// share a token's angles.  16384 tokens of 32 + 8 heads stored take 65 and 61 us with 16 and 32 (89, 74, 67 and 67 with 8, 16,
// 32 and 64 while q, k and v had one loop), of 32 heads turned 47, 43, 44 and 44 us with 8 to 64.  For 32 warps an SM;
// for 64, 1024 to 4096 tokens of 32 + 8 heads take 9.4, 11.8 and 17.6 us instead of 7.9, 11.6 and 16.0, for 16, 1531 of 20 + 5 in
// NVFP4 12.4 instead of 10.5.
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
