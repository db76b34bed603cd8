// kv_cache.cu -- the 4-bit key/value cache in pages: the plan of a step (block
// tables and slots from request lengths), the store of new tokens (bf16 ->
// E2M1 codes with block scales) and the load of stored ones.
//
// A cache row is one token of one key head: 128 E2M1 codes, two to a byte with
// the even channel in the low nibble, and its block scales.
//   MXFP4  1x32 blocks, E8M0 byte X + 127 with X = floor(log2 amax) - 2 clamped
//          to [-23, 13], codes E2M1(x 2^-X).  Within the clamp this is the MX
//          rule of lowp_mx_kernel; the clamp keeps every value the cache can
//          hold (k 2^-24 up to 6 2^13) a binary16 number, so that the attention
//          multiplies code and scale in binary16 without rounding.
//   NVFP4  1x16 blocks, scale s = E4M3(amax / (6 st)), codes E2M1(x / (s st)),
//          every step one correctly rounded fp32 operation, under the caller's
//          fp32 scale st of the whole K or V cache.
// A block with Inf or NaN gets scale 0xFF (MXFP4) or 0x7F (NVFP4) and codes 0:
// it reads back as NaN.
#include <cooperative_groups.h>

#include "kv_rows.cuh"

namespace mxfa {

static __device__ unsigned g_status_kv;

// ------------------------------------------------------------------------ plan
// One step of a batch, from R context lengths c_r and R counts of new tokens
// n_r (n_r < 0: the request is done and gives its blocks back):
//   cu     prefix sums of max(n_r, 0)
//   grow_r = ceil((c_r + n_r) / page) - ceil(c_r / page) new blocks, taken in
//            request order from the ring [head, tail); a request is served if
//            the sum of grow up to and with it is at most tail - head, or if it
//            grows by nothing; otherwise it keeps c_r and its tokens get slot -1
//   token t of request r at position p = c_r + t - cu_r has slot
//            table[r][p / page] * page + p % page
// Every CTA scans all requests (three prefix sums, kept in shared memory) and
// then takes its share of table entries and tokens: nothing waits on another
// CTA, except that the lengths and the ring counters, which may be updated in
// place, are written after a barrier of the only cluster.  The work is a few
// kilobytes for a decoding step, bound by latency (16 requests: 4.4 us, the chain
// lengths, scans, ring, table, slots); a step with prompts writes 12 bytes per token
// (1024 requests, 24 prompts, 131072 tokens: 8.1 us; 15.2 us when the tokens' threads
// looked for the blocks of finished requests, too).
constexpr int kPlanThreads = 256;  // 16 / 1024 requests: 4.4 / 8.1 us; with 512 (and half the CTAs) 5.0 / 8.6, with 1024 6.9 / 12.0

__device__ __forceinline__ int pages_of(int len, int shift) { return int((int64_t(len) + (1 << shift) - 1) >> shift); }

struct PlanSums {
  int q;
  int grow;
  int back;
};

// Exclusive prefix sums over the CTA's threads; `total` gets the sums.
__device__ __forceinline__ PlanSums plan_scan(PlanSums v, PlanSums* warp_sums, PlanSums& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  PlanSums in = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xFFFFFFFFu, in.q, o), b = __shfl_up_sync(0xFFFFFFFFu, in.grow, o),
              c = __shfl_up_sync(0xFFFFFFFFu, in.back, o);
    if (lane >= o) {
      in.q += a;
      in.grow += b;
      in.back += c;
    }
  }
  if (lane == 31) warp_sums[warp] = in;
  __syncthreads();
  PlanSums before{0, 0, 0};
  total = PlanSums{0, 0, 0};
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; w++) {
    const PlanSums s = warp_sums[w];
    if (w < warp) {
      before.q += s.q;
      before.grow += s.grow;
      before.back += s.back;
    }
    total.q += s.q;
    total.grow += s.grow;
    total.back += s.back;
  }
  __syncthreads();
  return PlanSums{before.q + in.q - v.q, before.grow + in.grow - v.grow, before.back + in.back - v.back};
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(KvPlanArgs a) {
  // per request: first token (R + 1 entries), context length, and the rank of
  // its first ring entry: taken (>= 0), or -1 if it is not served, or given
  // back (-2 - rank)
  extern __shared__ int32_t plan_smem[];
  int32_t* s_cu = plan_smem;
  int32_t* s_ctx = plan_smem + a.R + 1;
  int32_t* s_rank = s_ctx + a.R;
  __shared__ PlanSums s_warp[kPlanThreads / 32];
  __shared__ int s_taken;
  const int tid = threadIdx.x;
  const int64_t head = a.ring_in[0], tail = a.ring_in[1];
  const int64_t room = tail - head;
  const int avail = room <= 0 ? 0 : int(room < a.ring_size ? room : a.ring_size);
  if (tid == 0) s_taken = 0;
  __syncthreads();
  PlanSums run{0, 0, 0};
  int taken = 0;
  int next_c = tid < a.R ? a.ctx[tid] : 0, next_n = tid < a.R ? a.add[tid] : 0;
  for (int r0 = 0; r0 < a.R; r0 += kPlanThreads) {
    const int r = r0 + tid;
    PlanSums v{0, 0, 0};
    int c = next_c, n = next_n;
    bool fits_table = true;
    if (r + kPlanThreads < a.R) {  // the next ones' are on their way during the scan
      next_c = a.ctx[r + kPlanThreads];
      next_n = a.add[r + kPlanThreads];
    }
    if (r < a.R) {
      c = max(c, 0);
      const int have = pages_of(c, a.page_shift);
      if (n < 0) {
        v.back = min(have, a.width);
      } else {
        v.q = n;
        const int64_t need = (int64_t(c) + n + (1 << a.page_shift) - 1) >> a.page_shift;
        fits_table = need <= a.width;
        v.grow = fits_table ? int(need) - have : 0;
      }
      if (!fits_table || (n < 0 && have > a.width)) atomicOr(&g_status_kv, DEV_BAD_INDEX);
    }
    PlanSums tot;
    const PlanSums ex = plan_scan(v, s_warp, tot);
    if (r < a.R) {
      const int before = run.grow + ex.grow;
      const bool in_room = before + v.grow <= avail;
      s_cu[r] = run.q + ex.q;
      s_ctx[r] = c;
      s_rank[r] = n < 0 ? -2 - (run.back + ex.back) : (fits_table && (v.grow == 0 || in_room)) ? before : -1;
      if (in_room) taken = max(taken, before + v.grow);
    }
    run.q += tot.q;
    run.grow += tot.grow;
    run.back += tot.back;
  }
  atomicMax(&s_taken, taken);
  if (tid == 0) s_cu[a.R] = run.q;
  __syncthreads();
  const int page = 1 << a.page_shift;
  const int64_t head0 = (head % a.ring_size + a.ring_size) % a.ring_size;
  const int64_t tail0 = (tail % a.ring_size + a.ring_size) % a.ring_size;
  auto wrap = [&](int64_t i) {  // into the ring; one subtraction unless a caller's counters are off
    if (i >= a.ring_size) i -= a.ring_size;
    return i < a.ring_size ? i : i % a.ring_size;
  };
  const int total = s_cu[a.R];
  // blocks given back, and (where not every token has a row below) blocks taken: one
  // CTA per request, four entries of a thread in flight
  for (int r = blockIdx.x; r < a.R; r += gridDim.x) {
    const int rank = s_rank[r];
    if (rank == -1 || (rank >= 0 && total <= a.tokens)) continue;
    const int have = pages_of(s_ctx[r], a.page_shift);
    int32_t* row = a.table + int64_t(r) * a.width;
    const bool take = rank >= 0;
    const int from = take ? have : 0;
    const int to = take ? pages_of(s_ctx[r] + s_cu[r + 1] - s_cu[r], a.page_shift) : min(have, a.width);
    const int64_t at = take ? head0 + rank - have : tail0 + (-2 - rank);  // ring place of entry 0
    for (int j0 = from + tid; j0 < to; j0 += 4 * kPlanThreads) {
      int32_t v[4];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int j = j0 + kPlanThreads * i;
        if (j < to) v[i] = take ? a.ring[wrap(at + j)] : row[j];
      }
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int j = j0 + kPlanThreads * i;
        if (j >= to) continue;
        if (take) row[j] = v[i];
        else a.ring[wrap(at + j)] = v[i];
      }
    }
  }
  // tokens; the first of a new page writes the page's table entry
  for (int64_t t = int64_t(blockIdx.x) * kPlanThreads + tid; t < a.tokens; t += int64_t(gridDim.x) * kPlanThreads) {
    int64_t slot = -1;
    int pos = -1;
    if (t < total) {
      int lo = 0, hi = a.R;  // the request with cu[lo] <= t < cu[lo + 1]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_cu[mid] <= int(t)) lo = mid;
        else hi = mid;
      }
      pos = s_ctx[lo] + int(t) - s_cu[lo];
      const int rank = s_rank[lo];
      if (rank >= 0) {
        const int have = pages_of(s_ctx[lo], a.page_shift), j = pos >> a.page_shift;
        int32_t b = -1;
        if (j >= 0 && j < a.width) {
          int32_t* entry = a.table + int64_t(lo) * a.width + j;
          if (j < have) {
            b = *entry;
          } else {
            b = a.ring[wrap(head0 + rank + j - have)];
            if ((pos & (page - 1)) == 0) *entry = b;
          }
        }
        if (b >= 0) slot = int64_t(b) * page + (pos & (page - 1));
      }
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
  }
  // offsets, lengths and counters: the first CTA, once every CTA of its cluster
  // has read the inputs (in place there is one cluster)
  cooperative_groups::this_cluster().sync();
  if (blockIdx.x == 0) {
    for (int r = tid; r <= a.R; r += kPlanThreads) {
      a.cu_q[r] = s_cu[r];
      if (r < a.R) {
        const int rank = s_rank[r];
        a.kv_lens[r] = rank < -1 ? 0 : s_ctx[r] + (rank >= 0 ? s_cu[r + 1] - s_cu[r] : 0);
      }
    }
    if (tid == 0) {
      a.ring_out[0] = head + s_taken;
      a.ring_out[1] = tail + run.back;
      a.ring_out[2] = run.grow - s_taken;
    }
  }
}

cudaError_t launch_kv_plan(const KvPlanArgs& a, cudaStream_t st) {
  clear_stale_error();
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (3 * kKvPlanMaxRequests + 1) * int(sizeof(int32_t)));
  });
  if (e != cudaSuccess) return e;
  // a cluster of 1, 2, 4 or 8 CTAs, one CTA per 256 tokens or 16 requests; many
  // clusters for long steps whose outputs are not their own inputs
  int64_t ctas = (a.tokens + kPlanThreads - 1) / kPlanThreads;
  const int64_t by_requests = (int64_t(a.R) + 15) / 16;
  ctas = ctas > by_requests ? ctas : by_requests;
  const int most = a.aliased ? 8 : 256;
  int grid = 1;
  while (grid < most && grid < ctas) grid *= 2;
  const size_t bytes = size_t(3 * int64_t(a.R) + 1) * sizeof(int32_t);
  if (grid == 1) {  // a cluster of its own
    kv_plan_kernel<<<1, kPlanThreads, bytes, st>>>(a);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = unsigned(grid < 8 ? grid : 8);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_plan_kernel, a);
}

// --------------------------------------------------------------- store and load
// Sixteen lanes per cache row of K or of V, eight channels a lane: 16 bytes of
// bf16 on one side, 4 bytes of codes on the other, and one lane of each block
// for its scale.  256 bytes of bf16 and 68 or 72 bytes of cache per row move.  32768
// tokens x 8 heads: store 41 us (MXFP4, 4.1 TB/s) and 71 us (NVFP4, 2.4 TB/s:
// instructions, 3.4 a cycle, with eight correctly rounded divisions a lane), load 36
// and 38 us (4.7 and 4.5 TB/s); a plain elementwise kernel that moves as many bytes
// takes 29 us (5.9 TB/s).  A token's rows in a page are 64 bytes each, a page of
// one head apart.
// Where row `r` of the call (token, head, K or V) lives in the cache; false if
// its slot is negative or out of range.
struct KvRow {
  int64_t token;
  int head;
  bool is_v;
  int64_t at;  // cache row
};
__device__ __forceinline__ bool kv_row(const KvRowsArgs& a, uint32_t r, KvRow& w) {
  const uint32_t th = r >> 1;
  w.is_v = r & 1;
  w.token = th / uint32_t(a.c.H);
  w.head = int(th - uint32_t(w.token) * uint32_t(a.c.H));
  const int64_t slot = __ldg(a.slots + w.token);
  const int64_t block = slot >> a.c.page_shift;
  w.at = (block * a.c.H + w.head) * a.c.page + (slot & (a.c.page - 1));
  if (slot < 0) return false;
  if (block >= a.c.blocks) {
    atomicOr(&g_status_kv, DEV_BAD_INDEX);
    return false;
  }
  return true;
}

// The rows of a CTA: sixteen lanes to each, N a lane group, whose loads are all in
// flight before the first is used.
template <int FMT, int N>
__global__ void __launch_bounds__(256) kv_append_kernel(KvRowsArgs a) {
  const int lane = threadIdx.x & 15;
  const uint32_t rows = uint32_t(a.tokens * a.c.H * 2);  // below 2^32 - 128
  KvRow w[N];
  uint4 x[N];
  bool live[N];
#pragma unroll
  for (int i = 0; i < N; i++) {
    const uint32_t r = blockIdx.x * uint32_t(16 * N) + i * 16u + (threadIdx.x >> 4);
    live[i] = r < rows && kv_row(a, r, w[i]);
    x[i] = make_uint4(0, 0, 0, 0);
    if (live[i]) {
      const uint16_t* src = w[i].is_v ? a.v + w[i].token * a.v_stride : a.k + w[i].token * a.k_stride;
      x[i] = ldg_stream(reinterpret_cast<const uint4*>(src + w[i].head * 128 + lane * 8));
    }
  }
#pragma unroll
  for (int i = 0; i < N; i++) {
    kv_store_row<FMT>(a.c, live[i], w[i].is_v, w[i].at, lane, x[i]);
  }
}

// A row without a slot reads as zeros.
template <int FMT, int N>
__global__ void __launch_bounds__(256) kv_load_kernel(KvRowsArgs a) {
  const int lane = threadIdx.x & 15;
  const uint32_t rows = uint32_t(a.tokens * a.c.H * 2);  // below 2^32 - 128
  KvRow w[N];
  uint32_t c[N], b[N];
  bool live[N], mine[N];
#pragma unroll
  for (int i = 0; i < N; i++) {
    const uint32_t r = blockIdx.x * uint32_t(16 * N) + i * 16u + (threadIdx.x >> 4);
    mine[i] = r < rows;
    live[i] = mine[i] && kv_row(a, r, w[i]);
    c[i] = b[i] = 0;
    if (live[i]) {
      c[i] = __ldg(reinterpret_cast<const uint32_t*>((w[i].is_v ? a.c.v : a.c.k) + w[i].at * 64) + lane);
      const uint8_t* sf = w[i].is_v ? a.c.v_sf : a.c.k_sf;
      b[i] = FMT == 0 ? __ldg(sf + w[i].at * 4 + (lane >> 2)) : __ldg(sf + w[i].at * 8 + (lane >> 1));
    }
  }
#pragma unroll
  for (int i = 0; i < N; i++) {
    if (!mine[i]) continue;
    uint32_t out[4] = {0, 0, 0, 0};
    if (live[i]) {
      float s, st = 1.0f;
      if (FMT == 0) {
        s = b[i] == 0xFFu ? __uint_as_float(0x7FC00000u) : __uint_as_float(b[i] << 23);
      } else {
        s = e4m3x2_to_float2(b[i]).x;
        st = __ldg(w[i].is_v ? a.c.v_scale : a.c.k_scale);
      }
      uint32_t h[4];
      e2m1x8_to_f16(c[i], h);
#pragma unroll
      for (int e = 0; e < 4; e++) {
        float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[e]));
        f.x = __fmul_rn(f.x, s);
        f.y = __fmul_rn(f.y, s);
        if (FMT == 1) {
          f.x = __fmul_rn(f.x, st);
          f.y = __fmul_rn(f.y, st);
        }
        out[e] = pack_bf16(f.x, f.y);
      }
    }
    uint16_t* dst = w[i].is_v ? a.v : a.k;
    __stcs(reinterpret_cast<uint4*>(dst + (w[i].token * a.c.H + w[i].head) * 128 + lane * 8),
           make_uint4(out[0], out[1], out[2], out[3]));
  }
}

// Four rows to a lane group once one row each fills the GPU (about 16 CTAs of 16
// rows an SM); below that, one row each spreads the work over more SMs.  Store, us, with
// one and with four rows, 8 heads: 64 tokens 1.9 and 3.0, 1024 tokens 3.0 and 3.6, 2048
// tokens 4.2 and 5.0, 8192 tokens 12.0 and 11.7, 32768 tokens 49.6 and 40.8.
bool many_rows(const KvRowsArgs& a) { return a.tokens * a.c.H * 2 >= int64_t(sm_count_current_device()) * 16 * 16; }

cudaError_t launch_kv_append(const KvRowsArgs& a, cudaStream_t s) {
  clear_stale_error();
  constexpr int N = 4;
  const bool many = many_rows(a);
  const int64_t per = many ? 16 * N : 16;
  const unsigned g = unsigned((a.tokens * a.c.H * 2 + per - 1) / per);
  if (a.c.fmt == 0) many ? kv_append_kernel<0, N><<<g, 256, 0, s>>>(a) : kv_append_kernel<0, 1><<<g, 256, 0, s>>>(a);
  else many ? kv_append_kernel<1, N><<<g, 256, 0, s>>>(a) : kv_append_kernel<1, 1><<<g, 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_load(const KvRowsArgs& a, cudaStream_t s) {
  clear_stale_error();
  constexpr int N = 4;
  const bool many = many_rows(a);
  const int64_t per = many ? 16 * N : 16;
  const unsigned g = unsigned((a.tokens * a.c.H * 2 + per - 1) / per);
  if (a.c.fmt == 0) many ? kv_load_kernel<0, N><<<g, 256, 0, s>>>(a) : kv_load_kernel<0, 1><<<g, 256, 0, s>>>(a);
  else many ? kv_load_kernel<1, N><<<g, 256, 0, s>>>(a) : kv_load_kernel<1, 1><<<g, 256, 0, s>>>(a);
  return cudaGetLastError();
}

unsigned read_status_kv(cudaStream_t st) {
  unsigned v = 0, z = 0;
  cudaMemcpyFromSymbolAsync(&v, g_status_kv, sizeof(v), 0, cudaMemcpyDeviceToHost, st);
  cudaMemcpyToSymbolAsync(g_status_kv, &z, sizeof(z), 0, cudaMemcpyHostToDevice, st);
  cudaStreamSynchronize(st);
  return v;
}

}  // namespace mxfa
