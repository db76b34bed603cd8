// kv_shared.cu -- attention over the 4-bit cache for requests that share prefixes.
//
// A softmax over the keys of a prefix and of what is behind it is joined from both parts' (m, l, O):
//   o = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i,  M = max m_i.
// So the prefix of a group is one attention problem for the queries of all its requests (kPrefix: the
// groups take the requests' places), the rest one of each request (kTail: keys before the prefix's
// end are hidden), by the kernels of kv_attn.cu and kv_prefill.cu, which leave records instead of results:
//   kv_shared_plan_kernel  checks the groups, writes the prefix of each request, the line that
//                          kv_prefill.cu works off for the groups, and clears the records' places
//                          (a request without a prefix has its results at once, unless it is cut)
//   kPrefix, kTail         neither needs the other's results, so the second starts where the first
//                          leaves SMs free
//   kv_shared_join_kernel  a warp a row: its records in the order of the keys
#include "kv_fp4.cuh"
#include "mx_ptx.cuh"
#include "mxfa_internal.h"

namespace mxfa {

static __device__ unsigned g_status_kv_shared;

namespace {

constexpr int kPlan = 512;
constexpr float kOffset = 8.0f;  // log2 offset of P in the records, as in kv_attn.cu and kv_prefill.cu

struct SharedArgs {
  const int32_t* prefix_lens;
  int groups, max_group_q;
  int32_t *gpre, *pre;
  int64_t* line;    // NULL: the groups are not kv_prefill.cu's
  uint4* places;    // of both passes, 16 bytes at a time
  int64_t words;
};

// The first CTA goes through the groups: prefix of group g at gpre[g] (0: none, or not as documented), behind them
// their number of items for kv_prefill.cu; the
// others take a request a thread: pre[r] (-1: of a group not as documented; 0: of none).
__global__ void __launch_bounds__(kPlan) kv_shared_plan_kernel(KvAttnArgs a, SharedArgs s) {
  __shared__ int64_t s_sum[kPlan / 32];
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto checked = [&](int g, int& n) -> int {  // -1: not as documented
    const int b = __ldg(a.starts + g), e = __ldg(a.starts + g + 1), p = __ldg(s.prefix_lens + g);
    n = 0;
    if (b < 0 || e < b || e > a.R || p < 0 || p > int64_t(a.width) << a.c.page_shift) return -1;
    const int q0 = __ldg(a.cu_q + b), q1 = __ldg(a.cu_q + e);
    if (q0 < 0 || q1 < q0 || q1 > a.total_q || q1 - q0 > s.max_group_q) return -1;
    n = q1 - q0;
    return e - b > 1 ? p : 0;  // a single request reads its own row
  };
  for (int64_t w = int64_t(blockIdx.x) * kPlan + tid; w < s.words; w += int64_t(gridDim.x) * kPlan) s.places[w] = make_uint4(0, 0, 0, 0);
  if (blockIdx.x > 0) {
    for (int r = (int(blockIdx.x) - 1) * kPlan + tid; r < a.R; r += (int(gridDim.x) - 1) * kPlan) {
      int lo = 0, hi = s.groups, n;  // the group with starts[lo] <= r < starts[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.starts + mid) <= r) lo = mid;
        else hi = mid;
      }
      const bool in = __ldg(a.starts + lo) <= r && r < __ldg(a.starts + lo + 1);
      s.pre[r] = in ? checked(lo, n) : 0;
    }
    return;
  }
  int64_t base = 0;
  int items = 0;
  for (int g0 = 0; g0 < s.groups; g0 += kPlan) {
    const int g = g0 + tid;
    int64_t u = 0;
    if (g < s.groups) {
      int n;
      const int p = checked(g, n);
      if (p < 0) atomicOr(&g_status_kv_shared, DEV_BAD_INDEX);
      s.gpre[g] = max(p, 0);
      if (p > 0) {
        u = kv_prefix_units(n, p, a.G, a.c.H);
        items = min(int64_t(items) + kv_prefix_items(n, a.G, a.c.H), int64_t(1) << 20);
      }
    }
    if (!s.line) continue;
    int64_t v = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t t = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += t;
    }
    if (lane == 31) s_sum[warp] = v;
    __syncthreads();
    int64_t before = base, all = 0;
    for (int w = 0; w < kPlan / 32; w++) {
      if (w < warp) before += s_sum[w];
      all += s_sum[w];
    }
    if (g < s.groups) s.line[g] = before + v - u;
    base += all;
    __syncthreads();
  }
  if (!s.line) return;
  // items, as many as the GPU can have runs for (the sum of saturated counts is below 2^30)
  items = __reduce_add_sync(0xFFFFFFFFu, items);
  if (lane == 0) s_sum[warp] = items;
  __syncthreads();
  if (tid == 0) {
    int64_t n = 0;
    for (int w = 0; w < kPlan / 32; w++) n += s_sum[w];
    s.gpre[s.groups] = int(min(n, int64_t(1) << 20));
    s.line[s.groups] = base;
  }
}

// One pass's records.
struct Pass {
  const uint8_t *few, *many;
  int few_rows;
  const float* rows_o;
  const float2* rows_ml;
  const uint2* places;
};

// Where a row's records of a pass are: part i's o, m and l.
struct Row {
  const uint8_t* at;      // record 2 cta + 1, the first part's
  const float* o;         // in one piece
  const float2* ml;
  int parts, rows, row;
  __device__ __forceinline__ Row(const Pass& p, uint2 place, int64_t r) {
    parts = place.y >> 16;
    row = (place.y >> 3) & 0xFF;
    rows = place.y & 4u ? kPrefillRows : p.few_rows;
    at = (place.y & 4u ? p.many : p.few) + (2 * int64_t(place.x) + 1) * rows * 520;
    o = p.rows_o + r * 128;
    ml = p.rows_ml + r;
  }
  __device__ __forceinline__ int count() const { return max(parts, 1); }
  __device__ __forceinline__ const uint8_t* record(int i) const { return i == 0 ? at : at + int64_t(2 * i - 1) * rows * 520; }
  __device__ __forceinline__ float2 ml_of(int i) const {
    const float* m = parts == 0 ? &ml->x : reinterpret_cast<const float*>(record(i) + rows * 512) + row;
    return make_float2(__ldcg(m), __ldcg(parts == 0 ? m + 1 : m + rows));
  }
  __device__ __forceinline__ const float4* o_at(int i) const {
    return reinterpret_cast<const float4*>(parts == 0 ? o : reinterpret_cast<const float*>(record(i)) + row * 128);
  }
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A warp a row, four channels a lane.
__global__ void __launch_bounds__(256) kv_shared_join_kernel(KvAttnArgs a, Pass prefix, Pass tail) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t r = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (r >= a.total_q * a.Hq) return;
  const uint2 pt = __ldcg(tail.places + r), pp = __ldcg(prefix.places + r);
  if (!(pt.y & 1u)) return;  // of no request
  const bool two = pt.y & 2u;
  if (two && !(pp.y & 1u)) {  // offsets that are none leave a request's rows outside its group's
    if (lane == 0) atomicOr(&g_status_kv_shared, DEV_BAD_INDEX);
    return;
  }
  const Row x(tail, pt, r), y(prefix, two ? pp : pt, r);
  const int ny = two ? y.count() : 0, n = ny + x.count();
  auto ml_of = [&](int i) { return i < ny ? y.ml_of(i) : x.ml_of(i - ny); };
  constexpr int N = 8;  // records in flight
  float4 v[N];
  auto load = [&](int i0) {
#pragma unroll
    for (int j = 0; j < N; j++) {
      const int i = min(i0 + j, n - 1);
      v[j] = __ldcg((i < ny ? y.o_at(i) : x.o_at(i - ny)) + lane);
    }
  };
  // a lane has the (m, l) of every 32nd record: of the first 32, most often all, they stay
  const float2 mine = lane < n ? ml_of(lane) : make_float2(-INFINITY, 0.0f);
  load(0);
  float M = mine.x;
  for (int i = lane + 32; i < n; i += 32) M = fmaxf(M, ml_of(i).x);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
  float L = 0.0f;
  float4 s = make_float4(0, 0, 0, 0);
  for (int i0 = 0; i0 < n; i0 += 32) {
    const float2 ml = i0 == 0 ? mine : i0 + lane < n ? ml_of(i0 + lane) : make_float2(-INFINITY, 0.0f);
    const float w = ml.x == -INFINITY ? 1.0f : ex2(ml.x - M);  // without keys l and O are 0, or NaN
    L += w * ml.y;
    const int end = min(32, n - i0);
    for (int j0 = 0; j0 < end; j0 += N) {
      if (i0 + j0 > 0) load(i0 + j0);
#pragma unroll
      for (int j = 0; j < N; j++) {
        const float u = __shfl_sync(0xFFFFFFFFu, w, j0 + j);
        if (j0 + j < end) {
          s.x += u * v[j].x;
          s.y += u * v[j].y;
          s.z += u * v[j].z;
          s.w += u * v[j].w;
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, o);
  const float vst = a.c.fmt == 1 ? __ldg(a.c.v_scale) : 1.0f;
  const float f = L == 0.0f ? 1.0f : vst / L;
  *reinterpret_cast<uint2*>(a.o + r * 128 + lane * 4) = make_uint2(pack_bf16(s.x * f, s.y * f), pack_bf16(s.z * f, s.w * f));
  const int64_t token = r / a.Hq;
  if (lane == 0) a.lse[(r - token * a.Hq) * a.total_q + token] = L == 0.0f ? -INFINITY : (M - kOffset + log2f(L)) * 0.6931471805599453f;
}

// Places in a call's workspace: for either pass its rows in one piece and its records, and what the plan writes.
struct Places {
  size_t o[2], ml[2], where, gpre, pre, pass[2], bytes;
};
Places places_of(int R, int groups, int64_t total_q, int max_q, int max_group_q, int64_t max_k, int Hq, int G) {
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t x = at;
    at += (n + 255) & ~size_t(255);
    return x;
  };
  const size_t rows = size_t(total_q) * size_t(Hq);
  Places p;
  for (int i = 0; i < 2; i++) {
    p.o[i] = take(rows * 512);
    p.ml[i] = take(rows * 8);
  }
  p.where = take(rows * 16);
  p.gpre = take(size_t(groups) * 4 + 4);
  p.pre = take(size_t(R) * 4);
  p.pass[0] = take(kv_attn_workspace(groups, max_group_q, max_k, G));
  p.pass[1] = take(kv_attn_workspace(R, max_q, max_k, G));
  p.bytes = at;
  return p;
}

}  // namespace

size_t kv_shared_workspace(int R, int groups, int64_t total_q, int max_q, int max_group_q, int64_t max_k, int Hq, int G) {
  return places_of(R, groups, total_q, max_q, max_group_q, max_k, Hq, G).bytes;
}

cudaError_t launch_kv_attn_shared(const KvAttnArgs& args, const int32_t* prefix_lens, int groups, int max_group_q, cudaStream_t st) {
  clear_stale_error();
  const int64_t max_k = int64_t(args.width) << args.c.page_shift, rows = args.total_q * args.Hq;
  uint8_t* const ws = args.ws;
  const Places p = places_of(args.R, groups, args.total_q, args.max_q, max_group_q, max_k, args.Hq, args.G);
  KvAttnArgs a[2] = {args, args};  // the groups as requests, whose keys are the prefixes; the requests behind them
  KvRecords rec[2];
  Pass pass[2];
  for (int i = 0; i < 2; i++) {
    a[i].ws = ws + p.pass[i];
    a[i].rows_o = reinterpret_cast<float*>(ws + p.o[i]);
    a[i].rows_ml = reinterpret_cast<float2*>(ws + p.ml[i]);
    a[i].places = reinterpret_cast<uint2*>(ws + p.where) + i * rows;
    a[i].prefix = reinterpret_cast<const int32_t*>(ws + (i ? p.pre : p.gpre));
  }
  a[0].R = groups;
  a[0].max_q = max_group_q;
  a[0].causal = 0;
  a[1].causal = 1;
  for (int i = 0; i < 2; i++) {
    rec[i] = kv_attn_records(a[i].ws, a[i].R, a[i].max_q, max_k, args.G);
    pass[i] = Pass{rec[i].few, rec[i].many, rec[i].few_rows, a[i].rows_o, a[i].rows_ml, a[i].places};
  }
  const bool few[2] = {kv_attn_few(max_group_q, max_k, args.G), kv_attn_few(args.max_q, max_k, args.G)};
  SharedArgs s{prefix_lens, groups, max_group_q, reinterpret_cast<int32_t*>(ws + p.gpre), reinterpret_cast<int32_t*>(ws + p.pre),
               few[0] ? nullptr : reinterpret_cast<int64_t*>(rec[0].many_ws), reinterpret_cast<uint4*>(ws + p.where), rows};
  const int64_t by_requests = 1 + (int64_t(args.R) + kPlan - 1) / kPlan, by_words = (rows + 4 * kPlan - 1) / (4 * kPlan);
  int64_t grid = by_requests > by_words ? by_requests : by_words;
  grid = grid < 2 ? 2 : grid < 1024 ? grid : 1024;
  kv_shared_plan_kernel<<<unsigned(grid), kPlan, 0, st>>>(args, s);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if ((e = launch_kv_attn(kPrefix, a[0], st)) != cudaSuccess) return e;
  a[1].late = few[1];  // one kernel, which needs nothing of the pass before
  if ((e = launch_kv_attn(kTail, a[1], st)) != cudaSuccess) return e;
  return launch_early(kv_shared_join_kernel, dim3(unsigned((rows + 7) / 8)), 256, 0, st, args, pass[0], pass[1]);
}

unsigned read_status_kv_shared(cudaStream_t st) {
  unsigned v = 0, z = 0;
  cudaMemcpyFromSymbolAsync(&v, g_status_kv_shared, sizeof(v), 0, cudaMemcpyDeviceToHost, st);
  cudaMemcpyToSymbolAsync(g_status_kv_shared, &z, sizeof(z), 0, cudaMemcpyHostToDevice, st);
  cudaStreamSynchronize(st);
  return v;
}

}  // namespace mxfa
