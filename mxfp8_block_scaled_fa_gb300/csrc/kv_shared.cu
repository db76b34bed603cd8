// kv_shared.cu -- attention over the 4-bit cache for requests that share prefixes.
//
// A softmax over the keys of a prefix and of what is behind it is joined from both parts' (m, l, O):
//   o = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i,  M = max m_i.
// So the prefix of a group is one attention problem for the queries of all its requests (kPrefix: the
// groups take the requests' places), the rest one of each request (kTail: keys before the prefix's
// end are hidden), by the kernels of kv_attn.cu and kv_prefill.cu, which leave records instead of results:
//   kv_shared_plan_kernel  checks the groups, decides whether sharing pays, writes the prefix of each request, the line
//                          that kv_prefill.cu works off for the groups, and clears the records' places
//   kPrefix, kTail         neither needs the other's results, so the second starts where the first
//                          leaves SMs free
//   kv_shared_join_kernel  a warp a row: its records in the order of the keys (a request without a prefix
//                          has its results before, unless it is cut)
//
// When it pays.  Read by each request, a prefix's tile of 128 keys takes its kernel's time per block of rows; shared, it
// takes that of the group's blocks, but records and join are more: 3 us and 0.6 ns a row, by the cases
// below.  In us, shared and not: 64 requests of 4 rows behind 8192 keys (8 key heads) 51 and 126; 6 x 5 requests of up to 15
// rows behind up to 3000 28 and 31; 16 of 4 rows behind 1024 27 and 25; 4 x 8 of 8 rows behind up to 4096 38 and 37; 3 x 30 of
// up to 25 rows behind up to 535 102 and 91; 3 x 8 of up to 636 rows behind up to 3454 157 and 132.  One that is not shared takes 5
// to 11 us (prompts 20 to 38) more than mxfa_kv_attn: the plan, a kernel without work, the second pass's masks.  With
// MXFA_KV_SHARE_NEVER, which has no such kernel, 3 to 10 (prompts 35).
#include "kv_fp4.cuh"
#include "mx_ptx.cuh"
#include "mxfa_internal.h"

#include "../../include/mxfa.h"

namespace mxfa {

static __device__ unsigned g_status_kv_shared;

namespace {

constexpr int kPlan = 512;
constexpr float kOffset = 8.0f;  // log2 offset of P in the records, as in kv_attn.cu and kv_prefill.cu

struct SharedArgs {
  const int32_t* prefix_lens;
  int groups, max_group_q;
  int mode;                 // MXFA_KV_SHARE_*
  int32_t *gpre, *pre, *first, *share;
  int64_t* line;            // NULL: the groups are not kv_prefill.cu's
  uint4* places;            // of both passes, 16 bytes at a time
  int64_t words;
  int few_rows[2], split_rows[2];  // of the passes' kernels
  float sms;
};

// SM microseconds of a tile of 128 keys for `rows` rows of one request (or group) and key head: kv_attn.cu's kernel by
// blocks of few_rows (0.54, 0.68, 0.82 and 0.96 for 8 to 32), kv_prefill.cu's by blocks of 256.
__device__ __forceinline__ float tile_cost(float rows, int few_rows, int split_rows) {
  if (rows > float(split_rows)) return ceilf(rows / float(kPrefillRows)) * 1.6f;
  return ceilf(rows / float(few_rows)) * (0.4f + 0.0175f * float(few_rows));
}

// The first CTA goes through the groups: prefix of group g at gpre[g] (0: none, not as documented, or not shared), behind them
// their number of items for kv_prefill.cu, and whether they are shared; the others take a request a thread: pre[r]
// (-1: of a group not as documented; 0: of none, or alone in its group) and the group's first request first[r].
__global__ void __launch_bounds__(kPlan) kv_shared_plan_kernel(KvAttnArgs a, SharedArgs s) {
  __shared__ int64_t s_sum[kPlan / 32];
  __shared__ float s_gain[kPlan / 32];
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int b, e, n;  // of the group that was checked: requests and query tokens
  auto checked = [&](int g) -> int {  // -1: not as documented
    b = __ldg(a.starts + g), e = __ldg(a.starts + g + 1);
    const int p = __ldg(s.prefix_lens + g);
    n = 0;
    if (b < 0 || e < b || e > a.R || p < 0 || p > int64_t(a.width) << a.c.page_shift) return -1;
    const int q0 = __ldg(a.cu_q + b), q1 = __ldg(a.cu_q + e);
    if (q0 < 0 || q1 < q0 || q1 > a.total_q || q1 - q0 > s.max_group_q) return -1;
    n = q1 - q0;
    return p;
  };
  auto common = [&](int g) -> int {  // a single request reads its own row
    const int p = checked(g);
    return p > 0 && e - b < 2 ? 0 : p;
  };
  for (int64_t w = int64_t(blockIdx.x) * kPlan + tid; w < s.words; w += int64_t(gridDim.x) * kPlan) s.places[w] = make_uint4(0, 0, 0, 0);
  if (blockIdx.x > 0) {
    for (int r = (int(blockIdx.x) - 1) * kPlan + tid; r < a.R; r += (int(gridDim.x) - 1) * kPlan) {
      int lo = 0, hi = s.groups;  // the group with starts[lo] <= r < starts[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.starts + mid) <= r) lo = mid;
        else hi = mid;
      }
      const bool in = __ldg(a.starts + lo) <= r && r < __ldg(a.starts + lo + 1);
      int p = in ? checked(lo) : 0;
      if (p > 0 && e - b == 1) {  // has no prefix for the kernels to come, but its queries behind one
        const int own = __ldg(a.cu_q + r + 1) - __ldg(a.cu_q + r);
        const bool short_of = own > 0 && int64_t(__ldg(a.kv_lens + r)) - own < p;
        if (short_of) atomicOr(&g_status_kv_shared, DEV_BAD_INDEX);
        p = short_of ? -1 : 0;
      }
      s.pre[r] = p;
      s.first[r] = p > 0 ? b : r;
    }
    return;
  }
  float gain = 0.0f;
  int first_p = 0, first_n = 0;  // of the first kPlan groups, most often all
  for (int g = tid; g < s.groups; g += kPlan) {
    const int p = common(g);
    if (g == tid) first_p = p, first_n = n;
    if (p < 0) atomicOr(&g_status_kv_shared, DEV_BAD_INDEX);
    if (p <= 0 || n == 0) continue;
    const float rows = float(n) * float(a.G), m = float(e - b);
    const float tiles = float(a.c.H) * float((p + kPrefillTile - 1) / kPrefillTile);
    gain += tiles * (m * tile_cost(rows / m, s.few_rows[1], s.split_rows[1]) - tile_cost(rows, s.few_rows[0], s.split_rows[0])) / s.sms -
            0.0006f * rows * float(a.c.H);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) gain += __shfl_xor_sync(0xFFFFFFFFu, gain, o);
  if (lane == 0) s_gain[warp] = gain;
  __syncthreads();
  gain = 0.0f;
  for (int w = 0; w < kPlan / 32; w++) gain += s_gain[w];
  const bool share = s.mode == MXFA_KV_SHARE_ALWAYS || (s.mode == MXFA_KV_SHARE_AUTO && gain > 3.0f);
  if (tid == 0) *s.share = share ? 1 : 0;
  int64_t base = 0;
  int items = 0;
  for (int g0 = 0; g0 < s.groups; g0 += kPlan) {
    const int g = g0 + tid;
    int64_t u = 0;
    if (g < s.groups) {
      const int p = !share ? 0 : g0 == 0 ? first_p : common(g);
      if (g0 == 0) n = first_n;
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
    int64_t k = 0;
    for (int w = 0; w < kPlan / 32; w++) k += s_sum[w];
    s.gpre[s.groups] = int(min(k, int64_t(1) << 20));
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

// Places in a call's workspace: for either pass its rows in one piece and its records, and what the plan writes.  Where
// nothing is shared (MXFA_KV_SHARE_NEVER) there is no first pass, and rows in one piece are results: of a row only
// the second pass's place is left, 8 bytes instead of 1056.
struct Places {
  size_t o[2], ml[2], where, gpre, pre, first, share, pass[2], bytes;
};
Places places_of(int R, int groups, int64_t total_q, int max_q, int max_group_q, int64_t max_k, int Hq, int G, int mode) {
  size_t at = 0;
  const bool never = mode == MXFA_KV_SHARE_NEVER;
  auto take = [&](size_t n) {
    const size_t x = at;
    at += (n + 255) & ~size_t(255);
    return x;
  };
  const size_t rows = size_t(total_q) * size_t(Hq);
  Places p;
  for (int i = 0; i < 2; i++) {
    p.o[i] = take(never ? 0 : rows * 512);
    p.ml[i] = take(never ? 0 : rows * 8);
  }
  p.where = take(rows * (never ? 8 : 16));
  p.gpre = take(size_t(groups) * 4 + 4);
  p.pre = take(size_t(R) * 4);
  p.first = take(size_t(R) * 4);
  p.share = take(4);
  p.pass[0] = take(never ? 0 : kv_attn_workspace(groups, max_group_q, max_k, G));
  p.pass[1] = take(kv_attn_workspace(R, max_q, max_k, G));
  p.bytes = at;
  return p;
}

}  // namespace

size_t kv_shared_workspace(int R, int groups, int64_t total_q, int max_q, int max_group_q, int64_t max_k, int Hq, int G,
                           int mode) {
  return places_of(R, groups, total_q, max_q, max_group_q, max_k, Hq, G, mode).bytes;
}

cudaError_t launch_kv_attn_shared(const KvAttnArgs& args, const int32_t* prefix_lens, int groups, int max_group_q, int mode, cudaStream_t st) {
  clear_stale_error();
  const int64_t max_k = int64_t(args.width) << args.c.page_shift, rows = args.total_q * args.Hq;
  uint8_t* const ws = args.ws;
  const bool never = mode == MXFA_KV_SHARE_NEVER;
  const Places p = places_of(args.R, groups, args.total_q, args.max_q, max_group_q, max_k, args.Hq, args.G, mode);
  KvAttnArgs a[2] = {args, args};  // the groups as requests, whose keys are the prefixes; the requests behind them
  KvRecords rec[2];
  Pass pass[2];
  for (int i = 0; i < 2; i++) {
    a[i].ws = ws + p.pass[i];
    a[i].rows_o = reinterpret_cast<float*>(ws + p.o[i]);
    a[i].rows_ml = reinterpret_cast<float2*>(ws + p.ml[i]);
    a[i].places = reinterpret_cast<uint2*>(ws + p.where) + (never ? 0 : i * rows);
    a[i].prefix = reinterpret_cast<const int32_t*>(ws + (i ? p.pre : p.gpre));
  }
  a[0].R = groups;
  a[0].max_q = max_group_q;
  a[0].causal = 0;
  a[1].causal = 1;
  a[1].starts = reinterpret_cast<const int32_t*>(ws + p.first);
  a[1].share = reinterpret_cast<const int32_t*>(ws + p.share);
  for (int i = 0; i < 2; i++) {
    rec[i] = kv_attn_records(a[i].ws, a[i].R, a[i].max_q, max_k, args.G);
    pass[i] = Pass{rec[i].few, rec[i].many, rec[i].few_rows, a[i].rows_o, a[i].rows_ml, a[i].places};
  }
  const bool few[2] = {kv_attn_few(max_group_q, max_k, args.G), kv_attn_few(args.max_q, max_k, args.G)};
  SharedArgs s;
  s.prefix_lens = prefix_lens;
  s.groups = groups;
  s.max_group_q = max_group_q;
  s.mode = mode;
  s.gpre = reinterpret_cast<int32_t*>(ws + p.gpre);
  s.pre = reinterpret_cast<int32_t*>(ws + p.pre);
  s.first = reinterpret_cast<int32_t*>(ws + p.first);
  s.share = reinterpret_cast<int32_t*>(ws + p.share);
  s.line = never || few[0] ? nullptr : reinterpret_cast<int64_t*>(rec[0].many_ws);
  s.places = reinterpret_cast<uint4*>(ws + p.where);
  s.words = never ? (rows + 1) / 2 : rows;
  for (int i = 0; i < 2; i++) {
    s.few_rows[i] = rec[i].few_rows;
    s.split_rows[i] = i == 0 && !few[0] ? 0 : rec[i].split_rows;  // the prompts' kernel takes all groups or none
  }
  s.sms = float(sm_count_current_device());
  const int64_t by_requests = 1 + (int64_t(args.R) + kPlan - 1) / kPlan, by_words = (rows + 4 * kPlan - 1) / (4 * kPlan);
  int64_t grid = by_requests > by_words ? by_requests : by_words;
  grid = grid < 2 ? 2 : grid < 1024 ? grid : 1024;
  kv_shared_plan_kernel<<<unsigned(grid), kPlan, 0, st>>>(args, s);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (!never && (e = launch_kv_attn(kPrefix, a[0], st)) != cudaSuccess) return e;
  a[1].late = few[1] && !never;  // one kernel, which needs nothing of the pass before
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
